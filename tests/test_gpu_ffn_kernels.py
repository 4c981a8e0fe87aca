"""Every kernel of the feed-forward products (ffn_sizes, whose cover of the choice test_ffn_choice
checks), on operands whose sums are exact in FP32, so that each output is one number: the FP32
result rounded once.

Operands are 0, +-1 and +-2, scales 1/2, 1 and 2, biases and residuals multiples of 1/4 up to 8: a
sum is a multiple of 1/4 of at most 16 K < 2^19, 21 bits, whatever its order, and the matrix cores
hold a block's 128 products of at most 4 exactly.  With ReLU or no activation what follows is one
FP32 product (of an exact number by another), FP32 sums of 21-bit numbers, and the last rounding."""
from __future__ import annotations

import numpy as np
import pytest

from ffn_sizes import KERNELS, MANY

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402

VALUES = np.array([0, 1, -1, 2, -2], np.float32)
BYTES = np.array([0x00, 0x38, 0xB8, 0x40, 0xC0], np.uint8)
F = np.float32


def dev(v):
    return torch.from_numpy(np.ascontiguousarray(v)).cuda()


def shares(G, M, rng):
    """Rows of each expert: unequal, some zero, and the last one's end at M."""
    p = np.exp(0.7 * rng.normal(size=G)) * (rng.random(G) < 0.85)
    p = p if p.sum() else np.ones(G)
    return np.concatenate([[0], np.cumsum(rng.multinomial(M, p / p.sum()))]).astype(np.int32)


def scales(rng, *shape):
    return 2.0 ** rng.integers(-1, 2, shape).astype(F)


def quarters(rng, *shape):
    return (rng.integers(-32, 33, shape) / 4).astype(F)


def wide(s, rows, k):
    """Scales of 128-blocks along the last axis (and, for weights, of the one before) as factors."""
    s = s[..., np.arange(k) // 128]
    return s if rows is None else s[..., np.arange(rows) // 128, :]


def bf16(v):
    """FP32 -> BF16, nearest even, as FP32."""
    return torch.from_numpy(np.ascontiguousarray(v, F)).bfloat16().float().numpy()


def fp8(v):
    """FP32 rows -> the values of E4M3 bytes and the FP32 scales of 1x128 blocks."""
    m, n = v.shape
    pad = np.zeros((m, -(-n // 128) * 128), F)
    pad[:, :n] = v
    b = pad.reshape(m, -1, 128)
    a = np.maximum(np.abs(b).max(-1), F(2.0 ** -100))
    q = torch.from_numpy(b * (F(448) / a)[..., None]).to(torch.float8_e4m3fn).float().numpy()
    return q.reshape(m, -1)[:, :n], a / F(448)


class Outputs:
    """Buffers of a call, filled with something else before it, rows behind the last untouched."""

    def __init__(self, M, M_cap):
        self.M, self.M_cap, self.all = M, M_cap, []

    def new(self, n, dtype=torch.bfloat16):
        t = torch.full((self.M_cap, n), 0x55 if dtype == torch.uint8 else -77.0, dtype=dtype, device="cuda")
        self.all.append((t, t.clone()))
        return t

    def fp8(self, n):
        return self.new(n, torch.uint8), self.new(-(-n // 128), torch.float32)

    def check(self, t, want, what):
        got = t[:self.M]
        got = (got.view(torch.float8_e4m3fn) if got.dtype == torch.uint8 else got).float().cpu().numpy()
        bad = np.argwhere(got != want)            # (no NaN is among them: the sums are finite)
        assert not len(bad), (what, len(bad), bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])

    def behind(self):
        for t, before in self.all:
            assert torch.equal(t[self.M:], before[self.M:])


def operands(G, M_cap, parts, N, K, seed):
    rng = np.random.default_rng(seed)
    M = M_cap - min(3, M_cap // 2)
    offs = shares(G, M, rng)
    a, w = rng.integers(0, 5, (M_cap, K), dtype=np.int8), rng.integers(0, 5, (G, parts, N, K), dtype=np.int8)
    sa, sw = scales(rng, M_cap, -(-K // 128)), scales(rng, G, parts, -(-N // 128), -(-K // 128))
    av = VALUES[a[:M]] * wide(sa[:M], None, K)
    p = np.zeros((M, parts * N), F)
    for g in range(G):
        r = slice(offs[g], offs[g + 1])
        if offs[g] < offs[g + 1]:
            p[r] = av[r] @ (VALUES[w[g]] * wide(sw[g], N, K)).reshape(parts * N, K).T
    assert np.abs(p).max() < 2.0 ** 19 and (4 * p == np.rint(4 * p)).all()
    expert = np.searchsorted(offs, np.arange(M), side="right") - 1
    ab, wb = BYTES[a], BYTES[w]
    ab[M:], sa[M:] = 0x7F, np.nan                 # garbage behind the last row
    return rng, M, expert, p, (dev(ab), dev(sa), dev(wb), dev(sw), dev(offs))


def workspace(n):
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("act", ["relu", "none"])
@pytest.mark.parametrize("kind,e4m3,kernel,runs,G,M_cap,N,K", KERNELS + MANY)
def test_one_rounding(kind, e4m3, kernel, runs, G, M_cap, N, K, act):
    parts = 2 if kind == "gated" else 1
    rng, M, expert, p, (a, sa, w, sw, offs) = operands(G, M_cap, parts, N, K, N + K + len(act))
    relu = (lambda v: np.maximum(v, 0)) if act == "relu" else (lambda v: v)
    o = Outputs(M, M_cap)
    if kind == "gated":
        bias = quarters(rng, G, 2 * N)
        out, h = o.new(N), o.new(2 * N)
        q, qs = o.fp8(N) if e4m3 else (None, None)
        mx.mxfp4_fp8_gated_gemm(a, sa, w, sw, offs, out=out, q=q, q_scales=qs, h=h, bias=dev(bias), act=act,
                                workspace=workspace(mx.mxfp4_fp8_gated_gemm_workspace(G, M_cap, N, K)) if e4m3 else None)
        p += bias[expert]
        result = relu(p[:, :N]) * p[:, N:]
        o.check(h, bf16(p), "h")
        o.check(out, bf16(result), "out")
    elif kind == "gradient":
        hv = quarters(rng, M_cap, 2 * N)
        dh, out = o.new(2 * N), o.new(N)
        q, qs = o.fp8(2 * N) if e4m3 else (None, None)
        mx.mxfp4_fp8_gated_gemm_backward(
            a, sa, w[:, 0], sw[:, 0], dev(hv).bfloat16(), offs, dh=dh, dq=q, dq_scales=qs, out=out, act=act,
            workspace=workspace(mx.mxfp4_fp8_gated_gemm_backward_workspace(G, M_cap, N, K)) if e4m3 else None)
        gate, up = hv[:M, :N], hv[:M, N:]
        slope = (gate > 0).astype(F) if act == "relu" else np.ones_like(gate)
        result = np.concatenate([p * up * slope, p * relu(gate)], 1)
        o.check(dh, bf16(result), "dh")
        o.check(out, bf16(relu(gate) * up), "out")
    else:
        bias, res = quarters(rng, G, N), quarters(rng, M_cap, N)
        y, pre = o.new(N), o.new(N)
        mx.mxfp4_fp8_block_gemm_act(a, sa, w[:, 0], sw[:, 0], y, offs, bias=dev(bias), residual=dev(res).bfloat16(),
                                    pre=pre, act=act)
        p += bias[expert]
        o.check(pre, bf16(p), "pre")
        o.check(y, bf16(relu(p) + res[:M]), "y")
    if e4m3:
        bytes_, s = fp8(result)
        o.check(qs, s, "scales")
        o.check(q, bytes_, "E4M3")
    o.behind()
