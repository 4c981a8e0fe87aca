"""The feed-forward calls where rows, weights and outputs pass 2^31 elements and 2^32 bytes, on
operands whose FP32 sums are exact (test_gpu_ffn_kernels says why), compared in whole."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402

CHUNK = 4096
VALUES = torch.tensor([0.0, 1.0, -1.0, 2.0, -2.0])


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def e4m3(g, *shape):
    """E4M3 bytes of 0, +-1 and +-2."""
    v = VALUES.cuda()[torch.randint(0, 5, shape, device="cuda", generator=g)]
    return v.to(torch.float8_e4m3fn).view(torch.uint8)


def scales(g, *shape):
    return torch.exp2(torch.randint(-1, 2, shape, device="cuda", generator=g).float())


def quarters(g, *shape):
    """BF16 multiples of 1/4 up to 8, made chunk by chunk."""
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for c in t.split(CHUNK):
        c.copy_(torch.randint(-32, 33, c.shape, device="cuda", generator=g, dtype=torch.int8).bfloat16() / 4)
    return t


def value(q, s):
    """FP32 rows of E4M3 bytes and the scales of their blocks."""
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, -1)[..., :q.shape[-1]]


def new(*shape, dtype=torch.bfloat16):
    return torch.full(shape, 85 if dtype == torch.uint8 else -77, dtype=dtype, device="cuda")


def quantized(v):
    """The E4M3 values and scales of FP32 rows.  (Tensors by tensors: torch divides by a number, and a
    number by a tensor, by way of a rounded reciprocal.)"""
    m, n = v.shape
    b = torch.nn.functional.pad(v, (0, -n % 128)).view(m, -1, 128)
    a = b.abs().amax(-1).clamp_min(2.0 ** -100)
    most = torch.full_like(a, 448)
    q = (b * (most / a)[..., None]).to(torch.float8_e4m3fn).float()
    return q.view(m, -1)[:, :n], a / most


class Rows:
    """Two experts' rows of 16 elements, and the exact products with weights of `features` rows."""

    def __init__(self, counts, features, seed, slack=3, parts=1):
        g = gen(seed)
        self.M, self.M_cap, K = sum(counts), sum(counts) + slack, 16
        self.offs = torch.tensor([0, counts[0], self.M], dtype=torch.int32, device="cuda")
        self.split = counts[0]
        self.a, self.sa = e4m3(g, self.M_cap, K), scales(g, self.M_cap, 1)
        self.w = e4m3(g, 2, parts, features, K)
        self.sw = scales(g, 2, parts, -(-features // 128), 1)
        full = self.w.view(torch.float8_e4m3fn).float() * self.sw.repeat_interleave(128, 2)[:, :, :features]
        self.wt = full.reshape(2, parts * features, K).transpose(1, 2).contiguous()

    def chunks(self):
        """Row ranges within an expert, with their expert and products."""
        edges = sorted({0, self.split, self.M, *range(0, self.M, CHUNK)})
        for lo, hi in zip(edges, edges[1:]):
            g = int(lo >= self.split)
            yield slice(lo, hi), g, value(self.a[lo:hi], self.sa[lo:hi]) @ self.wt[g]


def same(got, want, what):
    got = got.view(torch.float8_e4m3fn).float() if got.dtype == torch.uint8 else got
    assert torch.equal(got.float(), want.float()), what


def behind(M, *outputs):
    for t in outputs:
        assert (t[M:].float() == (85 if t.dtype == torch.uint8 else -77)).all()


def test_dense_rows():
    N = 32784
    r = Rows([40000, 26001], N, 1)
    assert r.M * N > 1 << 31
    g = gen(2)
    bias, res, y, pre = quarters(g, 2, N).float(), quarters(g, r.M_cap, N), new(r.M_cap, N), new(r.M_cap, N)
    mx.mxfp4_fp8_block_gemm_act(r.a, r.sa, r.w[:, 0], r.sw[:, 0], y, r.offs, bias=bias, residual=res, pre=pre, act="relu")
    for at, e, p in r.chunks():
        p += bias[e]
        same(pre[at], p.bfloat16(), ("pre", at))
        same(y[at], (p.clamp_min(0) + res[at].float()).bfloat16(), ("y", at))
    behind(r.M, y, pre)


def test_gated_rows():
    I = 32784
    r = Rows([40000, 26001], I, 3, parts=2)
    assert r.M * I > 1 << 31
    bias = quarters(gen(4), 2, 2 * I).float()
    out, h, q, qs = new(r.M_cap, I), new(r.M_cap, 2 * I), new(r.M_cap, I, dtype=torch.uint8), \
        new(r.M_cap, -(-I // 128), dtype=torch.float32)
    ws = torch.empty(mx.mxfp4_fp8_gated_gemm_workspace(2, r.M_cap, I, 16), dtype=torch.uint8, device="cuda")
    mx.mxfp4_fp8_gated_gemm(r.a, r.sa, r.w, r.sw, r.offs, out=out, q=q, q_scales=qs, h=h, bias=bias, workspace=ws, act="relu")
    for at, e, p in r.chunks():
        p += bias[e]
        same(h[at], p.bfloat16(), ("h", at))
        v = p[:, :I].clamp_min(0) * p[:, I:]
        same(out[at], v.bfloat16(), ("out", at))
        b, s = quantized(v)
        same(qs[at], s, ("scales", at))
        same(q[at], b, ("q", at))
    behind(r.M, out, h, q, qs)


@pytest.mark.parametrize("in_place", [False, True])
def test_gated_gradient_rows(in_place):
    I = 32896
    r = Rows([40000, 26001], I, 5)
    h = quarters(gen(6), r.M_cap, 2 * I)
    h[r.M:] = -77
    was = h.clone() if in_place else h
    dh, out = h if in_place else new(r.M_cap, 2 * I), new(r.M_cap, I)
    q, qs = new(r.M_cap, 2 * I, dtype=torch.uint8), new(r.M_cap, 2 * I // 128, dtype=torch.float32)
    ws = torch.empty(mx.mxfp4_fp8_gated_gemm_backward_workspace(2, r.M_cap, I, 16), dtype=torch.uint8, device="cuda")
    mx.mxfp4_fp8_gated_gemm_backward(r.a, r.sa, r.w[:, 0], r.sw[:, 0], h, r.offs, dh=dh, dq=q, dq_scales=qs, out=out,
                                     workspace=ws, act="relu")
    for at, e, p in r.chunks():
        gate, up = was[at, :I].float(), was[at, I:].float()
        same(out[at], (gate.clamp_min(0) * up).bfloat16(), ("out", at))
        v = torch.cat([p * up * (gate > 0), p * gate.clamp_min(0)], 1)
        same(dh[at], v.bfloat16(), ("dh", at))
        b, s = quantized(v)
        same(qs[at], s, ("scales", at))
        same(q[at], b, ("q", at))
    behind(r.M, dh, out, q, qs)


def test_weights():
    """Experts' weights of 5.6 GB in all."""
    G, N, K = 21, 8208, 32784
    g = gen(7)
    w = torch.empty((G, N, K), dtype=torch.uint8, device="cuda")
    for i in range(G):
        w[i] = e4m3(g, N, K)
    kb = -(-K // 128)
    a, sa, sw = e4m3(g, 3 * G, K), scales(g, 3 * G, kb), scales(g, G, -(-N // 128), kb)
    counts = [2, 4] * (G // 2) + [3 * G - 6 * (G // 2)]
    at = [sum(counts[:i]) for i in range(G + 1)]
    y = new(3 * G, N)
    mx.mxfp4_fp8_block_gemm_act(a, sa, w, sw, y, torch.tensor(at, dtype=torch.int32, device="cuda"))
    gate = new(3 * G, N // 2)
    parts = (G, 2, N // 2, K)
    sg = scales(g, G, 2, -(-N // 256), kb)
    mx.mxfp4_fp8_gated_gemm(a, sa, w.view(parts), sg, torch.tensor(at, dtype=torch.int32, device="cuda"), out=gate, act="relu")
    for i in range(G):
        r = slice(at[i], at[i + 1])
        x = value(a[r], sa[r])
        raw = w[i].view(torch.float8_e4m3fn).float()
        wide = sw[i].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        same(y[r], (x @ (raw * wide).t().contiguous()).bfloat16(), i)
        wide = sg[i].repeat_interleave(128, 1)[:, :N // 2].reshape(N, kb).repeat_interleave(128, 1)[:, :K]
        p = x @ (raw * wide).t().contiguous()
        same(gate[r], (p[:, :N // 2].clamp_min(0) * p[:, N // 2:]).bfloat16(), i)


@pytest.mark.parametrize("in_place", [False, True])
def test_rows_and_biases(in_place):
    """Sums of at most 66001 multiples of 1/4 up to 8 are exact in FP32 in any order."""
    M, N = 66001, 32896
    g = gen(8)
    d, p = quarters(g, M + 3, N), quarters(g, M + 3, N)
    if in_place:
        d[M:] = -77
    was = d.clone() if in_place else d
    dp, db = d if in_place else new(M + 3, N), new(2, N, dtype=torch.float32)
    q, qs = new(M + 3, N, dtype=torch.uint8), new(M + 3, N // 128, dtype=torch.float32)
    ws = torch.empty(mx.mxfp4_act_rows_backward_workspace(2, M + 3, N), dtype=torch.uint8, device="cuda")
    mx.mxfp4_act_rows_backward(d, p, torch.tensor([0, 40000, M], dtype=torch.int32, device="cuda"), dpre=dp, q=q,
                               q_scales=qs, dbias=db, workspace=ws, act="relu")
    sums = torch.zeros((2, N), dtype=torch.float64, device="cuda")
    edges = sorted({0, 40000, M, *range(0, M, CHUNK)})
    for lo, hi in zip(edges, edges[1:]):
        v = was[lo:hi].float() * (p[lo:hi] > 0)
        same(dp[lo:hi], v.bfloat16(), lo)
        b, s = quantized(v)
        same(qs[lo:hi], s, lo)
        same(q[lo:hi], b, lo)
        sums[int(lo >= 40000)] += v.sum(0, dtype=torch.float64)
    assert torch.equal(db.double(), sums)
    behind(M, dp, q, qs)
