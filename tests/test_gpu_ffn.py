"""The feed-forward operators against float64 (ffn_ref has the bounds and where they come from):
the gated product, its gradient, the product with bias, activation and residual, and the rows'
and biases' gradient, at every kernel."""
from __future__ import annotations

import numpy as np
import pytest

import ffn_ref as fr
from test_gpu_block_gemm import operands

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402

ACTS = ["silu", "gelu", "gelu_tanh", "relu", "none"]


def dev(v):
    return torch.from_numpy(np.ascontiguousarray(v)).cuda()


def bf16(v):
    """float64 -> BF16 (nearest even), as float64 and as a GPU tensor."""
    t = torch.from_numpy(np.asarray(v, np.float32)).bfloat16()
    return t.double().numpy(), t.cuda()


def full(shape, dtype=torch.bfloat16, value=-3.0):
    return torch.full(shape, value, dtype=dtype, device="cuda")


def setup(counts, N, K, slack, seed, parts=1):
    """Operands whose products are of about unit size, garbage past the last row."""
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(offs[-1])
    G, M_cap = len(counts), M + slack
    rng = np.random.default_rng(seed)
    a, sa, w, _ = operands(offs, M_cap, parts * N, K, seed)
    kb, nb = -(-K // 128), -(-N // 128)
    # (E4M3 bytes drawn evenly: values of root mean square 118)
    sa = (np.exp(rng.normal(size=(M_cap, kb))) / 118).astype(np.float32)
    sw = (np.exp(0.5 * rng.normal(size=(G, parts * nb, kb))) / (118 * np.sqrt(3 * K))).astype(np.float32)
    a[M:], sa[M:] = 0x7F, np.nan
    if parts > 1:
        w, sw = w.reshape(G, parts, N, K), sw.reshape(G, parts, nb, kb)
    return offs, M, M_cap, a, sa, w, sw, rng


def host(t, M, what):
    """The rows of an output as float64; the rows behind them have to be as they were."""
    assert (t[M:].double() == -3 if t.dtype != torch.uint8 else t[M:] == 0x55).all(), what
    return t[:M].double().cpu().numpy() if t.dtype != torch.uint8 else t[:M].cpu().numpy()


def fp8_out(M_cap, n):
    return full((M_cap, n), torch.uint8, 0x55), full((M_cap, -(-n // 128)), torch.float32)


def work(fn, *sizes):
    return torch.empty(max(16, fn(*sizes)), dtype=torch.uint8, device="cuda").fill_(0xFF)


def check_gated(counts, I, K, act="silu", bias=True, fp8=True, h=True, slack=3, seed=0):
    offs, M, M_cap, a, sa, w, sw, rng = setup(counts, I, K, slack, seed, 2)
    b = rng.normal(size=(len(counts), 2, I)).astype(np.float32) if bias else None
    out = full((M_cap, I))
    hb = full((M_cap, 2 * I)) if h else None
    q, qs = fp8_out(M_cap, I) if fp8 else (None, None)
    ws = work(mx.mxfp4_fp8_gated_gemm_workspace, len(counts), M_cap, I, K)
    mx.mxfp4_fp8_gated_gemm(dev(a), dev(sa), dev(w), dev(sw), dev(offs), out=out, q=q, q_scales=qs, h=hb,
                            bias=dev(b) if bias else None, workspace=ws, act=act)
    want_h, eh = fr.gated_h(a[:M], sa[:M], w, sw, offs, b)
    want, e = fr.gated_out(want_h, eh, act)
    got = host(out, M, "out"), host(hb, M, "h") if h else None
    if not M:
        return
    fr.check_bf16(got[0], want, e, "out")
    if h:
        fr.check_bf16(got[1], want_h, eh, "h")
    if fp8:
        fr.check_fp8(host(q, M, "q"), host(qs, M, "q_scales").astype(np.float32), want, e, "q")


def check_gradient(counts, I, K, act="silu", fp8=True, out=True, slack=3, seed=0, in_place=False):
    offs, M, M_cap, a, sa, w, sw, rng = setup(counts, I, K, slack, seed)
    hv, h = bf16(1.5 * rng.normal(size=(M_cap, 2 * I)))
    h[M:] = -3.0
    dh = h if in_place else full((M_cap, 2 * I))
    ob = full((M_cap, I)) if out else None
    q, qs = fp8_out(M_cap, 2 * I) if fp8 else (None, None)
    ws = work(mx.mxfp4_fp8_gated_gemm_backward_workspace, len(counts), M_cap, I, K)
    mx.mxfp4_fp8_gated_gemm_backward(dev(a), dev(sa), dev(w), dev(sw), h, dev(offs), dh=dh, dq=q, dq_scales=qs, out=ob,
                                     workspace=ws, act=act)
    d, ed = fr.product(a[:M], sa[:M], w, sw, offs)
    want, e, want_out, eo = fr.gated_gradient(d, ed, hv[:M], act)
    got = host(dh, M, "dh")
    fr.check_bf16(got, want, e, "dh")
    if out:
        fr.check_bf16(host(ob, M, "out"), want_out, eo, "out")
    if fp8:
        fr.check_fp8(host(q, M, "dq"), host(qs, M, "dq_scales").astype(np.float32), want, e, "dq")


def check_dense(counts, N, K, act="gelu", bias=True, residual=True, pre=True, slack=3, seed=0, in_place=False):
    offs, M, M_cap, a, sa, w, sw, rng = setup(counts, N, K, slack, seed)
    b = rng.normal(size=(len(counts), N)).astype(np.float32) if bias else None
    rv, r = bf16(rng.normal(size=(M_cap, N)))
    r[M:] = -3.0
    y = r if in_place else full((M_cap, N))
    p = full((M_cap, N)) if pre else None
    mx.mxfp4_fp8_block_gemm_act(dev(a), dev(sa), dev(w), dev(sw), y, dev(offs), bias=dev(b) if bias else None,
                                residual=r if residual else None, pre=p, act=act)
    want_p, ep = fr.product(a[:M], sa[:M], w, sw, offs, b)
    f = fr.act(want_p, act)[0]
    e = fr.SLOPE * ep + fr.act_error(want_p) * np.abs(f)
    want = f + rv[:M] if residual else f
    got = host(y, M, "y"), host(p, M, "pre") if pre else None
    if not M:
        return
    fr.check_bf16(got[0], want, e + 2.0 ** -23 * np.abs(want), "y")
    if pre:
        fr.check_bf16(got[1], want_p, ep, "pre")


SHAPES = [
    ([1], 8, 16), ([1], 256, 128), ([3], 24, 144), ([0, 1, 0, 2], 136, 272), ([16], 512, 1024), ([17], 512, 1024),
    ([0] * 5, 64, 64), ([33, 0, 5], 1000, 336), ([64, 65, 63], 384, 640), ([257], 1352, 1744), ([2, 0, 4, 1, 7, 0, 3, 8], 2048, 1040),
    ([16, 0, 5], 1032, 400),                      # waves that share K, 16 tokens
    ([121], 2040, 272),                           # the same, 32 tokens
    ([17, 0, 13], 4104, 144),                     # few rows an expert, one workgroup per CU
    ([3, 0, 9, 1, 0, 33, 2, 5], 4104, 272),       # the same, several
    ([1] * 40, 1032, 400), ([1, 0, 2, 1, 0, 1, 1, 1] * 12, 264, 4096),
    ([100, 0, 130], 4104, 272),                   # medium
    ([50, 51, 49, 0, 64, 1, 100, 85], 8200, 144),
    ([301, 300, 280], 1544, 528),
    ([900, 3], 12296, 144),                       # large
    ([356, 100, 0, 640, 1, 385], 12296, 400),     # large, with partial tiles of 100, 128, 1 and 129 rows
    ([1000, 129], 8208, 272), ([700, 260], 9984, 16),
    ([2500, 0, 700], 4104, 272),
    ([1] * 300, 520, 112),
]


@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_gated(counts, N, K):
    fp8 = N % 16 == 0
    check_gated(counts, N, K, act=ACTS[(N // 8 + K) % 5], fp8=fp8, seed=N + K)


@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_gradient(counts, N, K):
    if not sum(counts):
        counts = [0, 2, 0]
    check_gradient(counts, N, K, act=ACTS[(N // 8 + K + 1) % 5], fp8=False, seed=N + K)
    if N > 200 and N < 5000:
        check_gradient(counts, N // 128 * 128, K, act=ACTS[(N // 8 + K + 2) % 5], seed=N)


@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_dense(counts, N, K):
    check_dense(counts, N, K, act=ACTS[(N // 8 + K + 3) % 5], seed=N + K)


# sizes that the estimate of block_ffn.hip gives to kernels the above do not reach: groups of
# waves that share K (with blocks for all of them, and with fewer), pairs on a CU, wide tiles
GATED = [
    ([2], 512, 4096), ([17], 2064, 1040), ([40], 2048, 4096), ([21, 19], 3088, 2064), ([20, 30, 17], 2064, 2064), ([1, 0, 2], 1552, 2064), ([1, 0, 2], 1552, 4096), ([1, 0, 2], 3088, 4096),
    ([16, 20, 1, 0, 40, 16, 30, 7], 1024, 4096), ([130, 120, 139], 2064, 1040), ([130, 120, 150], 2064, 2064),
    ([20, 30, 0, 60, 10, 40, 17, 20], 1552, 4096), ([60, 64, 129, 1, 0, 70, 88, 90], 1552, 4096),
    ([300, 100, 200, 90, 207], 1552, 4096), ([50, 51, 49, 0, 64, 1, 100, 85], 2064, 128), ([30, 0, 57], 8208, 128),
    ([897], 1024, 272), ([600, 500], 4112, 272), ([900, 1000], 2064, 144),
]
OTHERS = [
    ([2], 256, 4096), ([17], 4112, 1040), ([40], 4096, 4096), ([30, 0, 31], 4112, 2064), ([1, 2], 4112, 2064), ([1, 2], 4112, 4096), ([1, 2], 8208, 4096),
    ([37], 8208, 4096), ([130, 120, 139], 4112, 1040), ([127], 12304, 4096), ([45, 0, 1, 0, 0], 1552, 4096),
    ([50, 51, 49, 0, 64, 1, 100, 85], 4112, 128), ([897], 2064, 272), ([1097], 1552, 272), ([75] * 20, 1032, 2064),
]


@pytest.mark.parametrize("counts,N,K", GATED)
def test_gated_every_kernel(counts, N, K):
    check_gated(counts, N, K, fp8=False, seed=N)
    check_gated(counts, N, K, act="gelu", h=False, seed=N + 1)


@pytest.mark.parametrize("counts,N,K", OTHERS)
def test_others_every_kernel(counts, N, K):
    check_gradient(counts, N, K, fp8=False, seed=N)
    check_gradient(counts, N // 128 * 128, K, act="gelu", seed=N + 1)
    check_dense(counts, N, K, seed=N + 2)


@pytest.mark.parametrize("K", [16, 144, 272, 400, 528, 656])
@pytest.mark.parametrize("counts,N", [([17], 4112), ([1, 2], 8208), ([140, 130, 129], 4112), ([70, 0, 64, 33], 4104)])
def test_few_blocks_of_k(counts, N, K):
    """One to six blocks of K, the last one partial: fewer than the waves or groups that share them."""
    check_dense(counts, N, K, seed=K + N)
    check_gated(counts, N // 32 * 16, K, seed=K + N)


@pytest.mark.parametrize("act", ACTS)
def test_activations(act):
    for M in (5, 300):                            # few rows, and a tile
        check_gated([M, 2], 272, 272, act=act, seed=M)
        check_gradient([M, 2], 256, 272, act=act, seed=M + 1)
        check_dense([M, 2], 264, 272, act=act, seed=M + 2)


@pytest.mark.parametrize("M", [3, 90, 2000])
def test_outputs_left_out(M):
    counts, N, K = [M, 1], 384, 272
    for kw in (dict(fp8=False, h=False), dict(fp8=True, h=False, bias=False), dict(fp8=False, h=True, bias=False)):
        check_gated(counts, N, K, seed=M, **kw)
    check_gradient(counts, N, K, out=False, fp8=False, seed=M)
    check_gradient(counts, N, K, out=False, fp8=True, seed=M)
    for kw in (dict(bias=False, residual=False, pre=False), dict(bias=True, residual=False), dict(bias=False, pre=False)):
        check_dense(counts, N, K, seed=M, **kw)


def test_fp8_alone():
    """q without out, dq without dh: the same bytes as with them."""
    for M, N in ((3, 256), (40, 2048), (700, 1024)):
        offs, _, M_cap, a, sa, w, sw, rng = setup([M, 5], N, 272, 2, M, 2)
        args = [dev(v) for v in (a, sa, w, sw, offs)]
        ws = work(mx.mxfp4_fp8_gated_gemm_workspace, 2, M_cap, N, 272)
        both, alone = fp8_out(M_cap, N), fp8_out(M_cap, N)
        mx.mxfp4_fp8_gated_gemm(*args, out=full((M_cap, N)), q=both[0], q_scales=both[1], workspace=ws)
        mx.mxfp4_fp8_gated_gemm(*args, q=alone[0], q_scales=alone[1], workspace=ws)
        assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])
        h = bf16(rng.normal(size=(M_cap, 2 * N)))[1]
        wt, swt = args[2][:, 0].contiguous(), args[3][:, 0].contiguous()
        ws = work(mx.mxfp4_fp8_gated_gemm_backward_workspace, 2, M_cap, N, 272)
        both, alone = fp8_out(M_cap, 2 * N), fp8_out(M_cap, 2 * N)
        mx.mxfp4_fp8_gated_gemm_backward(*args[:2], wt, swt, h, args[4], dh=full((M_cap, 2 * N)), dq=both[0],
                                         dq_scales=both[1], workspace=ws)
        mx.mxfp4_fp8_gated_gemm_backward(*args[:2], wt, swt, h, args[4], dq=alone[0], dq_scales=alone[1], workspace=ws)
        assert torch.equal(both[0], alone[0]) and torch.equal(both[1], alone[1])


@pytest.mark.parametrize("counts,N,K", [([7, 2], 256, 272), ([40, 3], 2056, 272), ([150, 130], 4104, 144), ([800], 12296, 128)])
def test_in_place(counts, N, K):
    check_gradient(counts, N, K, fp8=False, in_place=True, seed=N)
    check_dense(counts, N, K, in_place=True, seed=N)


@pytest.mark.parametrize("times", [8, 40])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 17, 40, 1, 9, 0, 5], 1040, 272), ([0, 200], 2064, 144), ([5], 512, 400)])
def test_capacity_far_above_the_rows(counts, N, K, times):
    slack = (times - 1) * sum(counts) + 7
    check_gated(counts, N, K, slack=slack, seed=times)
    check_gradient(counts, N // 128 * 128, K, slack=slack, seed=times)
    check_dense(counts, N, K, slack=slack, seed=times)


@pytest.mark.parametrize("I", [16, 48, 112, 128, 144, 240, 256, 272, 400])
def test_gated_widths_in_and_across_scale_blocks(I):
    for M in (6, 300):
        check_gated([M], I, 144, seed=I)


# ---- the rows' and biases' gradient ---------------------------------------------------------

def check_rows(counts, N, act, dpre=True, fp8=False, dbias=True, slack=3, seed=0, in_place=None):
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, G = int(offs[-1]), len(counts)
    M_cap = M + slack
    rng = np.random.default_rng(seed)
    dv, d = bf16(rng.normal(size=(M_cap, N)) * np.exp(rng.normal(size=(M_cap, 1))))
    pv, p = bf16(2 * rng.normal(size=(M_cap, N)))
    d[M:], p[M:] = float("nan") if in_place != "dout" else -3.0, float("nan") if in_place != "pre" else -3.0
    o = {"dout": d, "pre": p, None: full((M_cap, N)) if dpre else None}[in_place]
    q, qs = fp8_out(M_cap, N) if fp8 else (None, None)
    db = full((G, N), torch.float32) if dbias else None
    ws = work(mx.mxfp4_act_rows_backward_workspace, G, M_cap, N)
    mx.mxfp4_act_rows_backward(d, p if act != "none" else None, dev(offs), dpre=o, q=q, q_scales=qs, dbias=db,
                               workspace=ws, act=act)
    slope = fr.act(pv[:M], act)[1]
    es = fr.act_error(pv[:M]) if act not in ("none", "relu") else np.zeros((M, N))
    want = dv[:M] * slope
    e = np.abs(dv[:M]) * es + 2.0 ** -23 * np.abs(want)
    if o is not None and M:
        fr.check_bf16(host(o, M, "dpre"), want, e, "dpre")
    if fp8 and M:
        fr.check_fp8(host(q, M, "q"), host(qs, M, "q_scales").astype(np.float32), want, e, "q")
    if dbias:
        # a sum of at most 64 rows a thread (an expert's rows whole), 8 threads; or of 16, 8, a run of tiles, 16 runs
        got = db.double().cpu().numpy()
        for g in range(G):
            r = slice(offs[g], offs[g + 1])
            depth = 80 + counts[g] / 128
            bound = e[r].sum(0) + depth * 2.0 ** -24 * np.abs(want[r]).sum(0)
            assert (np.abs(got[g] - want[r].sum(0)) <= bound).all(), g


@pytest.mark.parametrize("counts,N", [
    ([1], 8), ([0, 3, 0], 264), ([5, 0, 120], 256), ([128], 1000), ([0, 0], 16), ([1] * 70, 48),
    ([130], 8), ([127, 128, 129, 1, 0], 264), ([1000, 0, 700], 520), ([250, 0, 249], 136), ([0, 300, 0, 1, 0, 200], 264), ([10] * 51, 520), ([400, 0, 0, 0, 0, 110], 72), ([0] * 70 + [300] + [0] * 70 + [5], 136),
    ([4500], 72), ([40] * 90, 256),
])
def test_rows_and_biases(counts, N):
    for i, act in enumerate(ACTS):
        check_rows(counts, N, act, seed=N + i, fp8=N % 16 == 0 and i % 2 == 0)


@pytest.mark.parametrize("M", [9, 700])
def test_rows_outputs_left_out(M):
    check_rows([M, 3], 272, "gelu", dbias=False, seed=1)
    check_rows([M, 3], 272, "silu", dpre=False, fp8=True, dbias=False, seed=2)
    check_rows([M, 3], 272, "none", dpre=False, seed=3)
    check_rows([M, 3], 272, "gelu_tanh", dpre=False, fp8=True, seed=4)
    for which in ("dout", "pre"):
        check_rows([M, 3], 272, "gelu", in_place=which, seed=5)


def test_no_rows_gives_zero_biases():
    for M_cap in (0, 5, 500):
        db = full((3, 40), torch.float32)
        x = torch.zeros((M_cap, 40), dtype=torch.bfloat16, device="cuda")
        mx.mxfp4_act_rows_backward(x, x, torch.zeros(4, dtype=torch.int32, device="cuda"), dbias=db, act="silu",
                                   workspace=work(mx.mxfp4_act_rows_backward_workspace, 3, M_cap, 40))
        assert (db == 0).all()


def test_large_and_special_arguments():
    """Derivatives far out (1 on the right, 0 on the left), at the largest BF16 numbers, at zeros
    of both signs, and NaN where a NaN or a zero times an infinity is."""
    x = np.array([0.0, -0.0, 3e38, -3e38, 100.0, -100.0, 1e19, -1e19, 40.0, -40.0, 1e-30, -1e-30, 20.0, -20.0, 5.0, -5.0])
    pv, p = bf16(x[None].repeat(2, 0))
    one = torch.ones((2, 16), dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    for act in ACTS:
        o = full((2, 16))
        mx.mxfp4_act_rows_backward(one, p, offs, dpre=o, act=act)
        with np.errstate(over="ignore", invalid="ignore"):
            want = fr.act(np.clip(pv, -1e4, 1e4), act)[1]
        got = o.double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18).all(), (act, got, want)
    nan = torch.full((2, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    for act in ("silu", "gelu", "gelu_tanh"):
        o = full((2, 16))
        mx.mxfp4_act_rows_backward(one, nan, offs, dpre=o, act=act)
        assert o.isnan().all(), act


# ---- together, on streams, in graphs --------------------------------------------------------

class Block:
    """A small feed-forward block, forward and gradient, as a program calls it."""

    def __init__(self, counts, H, I, seed=0):
        self.offs_np, self.M, self.M_cap, a, sa, w, sw, rng = setup(counts, I, H, 4, seed, 2)
        self.G, self.H, self.I = len(counts), H, I
        _, _, _, _, _, w2, sw2, _ = setup(counts, H, I, 4, seed + 1)
        self.a, self.sa, self.w, self.sw, self.w2, self.sw2 = (dev(v) for v in (a, sa, w, sw, w2, sw2))
        self.w2t, self.sw2t = self.w2.transpose(1, 2).contiguous(), self.sw2.transpose(1, 2).contiguous()
        flat, sflat = self.w.view(self.G, 2 * I, H), self.sw.view(self.G, -1, self.sw.shape[-1])
        self.wt, self.swt = flat.transpose(1, 2).contiguous(), sflat.transpose(1, 2).contiguous()
        self.b1 = dev(rng.normal(size=(self.G, 2 * I)).astype(np.float32))
        self.b2 = dev(rng.normal(size=(self.G, H)).astype(np.float32))
        self.offs = dev(self.offs_np)
        self.res = bf16(rng.normal(size=(self.M_cap, H)))[1]
        self.dout = bf16(rng.normal(size=(self.M_cap, H)))[1]
        z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")      # noqa: E731
        self.h, self.y, self.dh, self.act, self.dx = z(self.M_cap, 2 * I), z(self.M_cap, H), z(self.M_cap, 2 * I), \
            z(self.M_cap, I), z(self.M_cap, H)
        self.q, self.qs = mx.alloc_fp8_rows_f32_outputs(self.M_cap, I)
        self.dy, self.dys = mx.alloc_fp8_rows_f32_outputs(self.M_cap, H)
        self.dq, self.dqs = mx.alloc_fp8_rows_f32_outputs(self.M_cap, 2 * I)
        self.db1 = torch.zeros((self.G, 2 * I), device="cuda")
        self.db2 = torch.zeros((self.G, H), device="cuda")
        self.ws = work(lambda: max(mx.mxfp4_fp8_gated_gemm_workspace(self.G, self.M_cap, I, H),
                                   mx.mxfp4_fp8_gated_gemm_backward_workspace(self.G, self.M_cap, I, H),
                                   mx.mxfp4_act_rows_backward_workspace(self.G, self.M_cap, 2 * I),
                                   mx.mxfp4_act_rows_backward_workspace(self.G, self.M_cap, H)))

    def run(self, stream=None):
        mx.mxfp4_fp8_gated_gemm(self.a, self.sa, self.w, self.sw, self.offs, q=self.q, q_scales=self.qs, h=self.h,
                                bias=self.b1, workspace=self.ws, stream=stream)
        mx.mxfp4_fp8_block_gemm_act(self.q, self.qs, self.w2, self.sw2, self.y, self.offs, bias=self.b2,
                                    residual=self.res, stream=stream)
        mx.mxfp4_act_rows_backward(self.dout, None, self.offs, q=self.dy, q_scales=self.dys, dbias=self.db2,
                                   workspace=self.ws, stream=stream)
        mx.mxfp4_fp8_gated_gemm_backward(self.dy, self.dys, self.w2t, self.sw2t, self.h, self.offs, dh=self.dh,
                                         dq=self.dq, dq_scales=self.dqs, out=self.act, workspace=self.ws,
                                         stream=stream)
        mx.mxfp4_act_rows_backward(self.dh, None, self.offs, dbias=self.db1, workspace=self.ws, stream=stream)
        mx.mxfp4_fp8_block_gemm_act(self.dq, self.dqs, self.wt, self.swt, self.dx, self.offs, stream=stream)

    def outputs(self):
        return [t.clone() for t in (self.y, self.h, self.q, self.qs, self.dh, self.dq, self.dqs, self.act, self.dx,
                                    self.db1, self.db2)]

    def reference(self):
        """float64 y, dx, db1, db2 by automatic differentiation, without the roundings between."""
        import moe_ref as ref
        M, I, H = self.M, self.I, self.H
        val = lambda q, s: ref.e4m3(q.cpu().numpy()) * s.cpu().double().numpy()[..., np.arange(q.shape[-1]) // 128]      # noqa: E731
        x = torch.from_numpy(val(self.a[:M], self.sa[:M])).requires_grad_()
        nb = np.arange(I) // 128
        w = torch.from_numpy(val(self.w, self.sw[:, :, nb])).reshape(self.G, 2 * I, H)
        w2 = torch.from_numpy(val(self.w2, self.sw2[:, np.arange(H) // 128]))
        b1, b2 = self.b1.cpu().double().requires_grad_(), self.b2.cpu().double().requires_grad_()
        y = []
        for g in range(self.G):
            r = slice(int(self.offs_np[g]), int(self.offs_np[g + 1]))
            h = x[r] @ w[g].T + b1[g]
            y.append((torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ w2[g].T + b2[g])
        y = torch.cat(y) + self.res[:M].cpu().double()
        return (y, *torch.autograd.grad((y * self.dout[:M].cpu().double()).sum(), (x, b1, b2)))


@pytest.mark.parametrize("counts,H,I", [([3, 0, 2], 400, 256), ([60, 0, 33, 7], 528, 384), ([300, 41], 1040, 512)])
def test_block_forward_and_gradient(counts, H, I):
    """The calls in a row against float64.  The activations between the products are quantized
    once on the way forward, the gradients twice on the way back (relative rounding at most
    2^-4 of an element, 0.026 in the mean: y's block part 0.026, dx's sqrt(2) 0.026; biases'
    gradients db1 0.026 over its own sums, db2 from dout alone)."""
    b = Block(counts, H, I, seed=H)
    b.run()
    y, dx, db1, db2 = b.reference()
    y0 = b.res[:b.M].cpu().double()
    for got, want, bound in ((b.y[:b.M].cpu().double() - y0, y.detach() - y0, 0.045), (b.dx[:b.M].cpu().double(), dx, 0.06),
                             (b.db1.cpu().double(), db1, 0.06), (b.db2.cpu().double(), db2, 1e-5)):
        err = (got - want).norm() / want.norm()
        assert err <= bound, (err, bound)


def test_another_stream():
    b = Block([60, 0, 33, 7], 528, 384, seed=5)
    b.run()
    torch.cuda.synchronize()
    want = b.outputs()
    for t in (b.y, b.h, b.dh, b.act, b.dx, b.db1, b.db2):
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for got, exp in zip(b.outputs(), want):
        assert torch.equal(got, exp)


@pytest.mark.parametrize("counts", [[3, 0, 2], [300, 41]])
def test_graph_replays(counts):
    """Captured once, replayed with other inputs and eager work between: every replay as eager."""
    b = Block(counts, 528, 384, seed=6)
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for i in range(4):
        b.dout.copy_(torch.roll(b.dout, 1, 1))
        b.b1.add_(0.25)
        b.a[:b.M].copy_(torch.roll(b.a[:b.M], 1, 1))
        for t in (b.y, b.h, b.dh, b.act, b.dx, b.db1, b.db2):
            t.fill_(float(i))
        graph.replay()
        got = b.outputs()
        torch.cuda.synchronize()
        b.run()
        for g, w in zip(got, b.outputs()):
            assert torch.equal(g[:b.M] if len(g) == b.M_cap else g, w[:b.M] if len(w) == b.M_cap else w), i


def test_tensors_of_another_device_are_refused(monkeypatch):
    b = Block([3, 0, 2], 400, 256, seed=9)
    b.run()
    monkeypatch.setattr(mx, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="the current device is cuda:1"):
        b.run()


def test_same_bits_every_time():
    """No sum depends on the order in which workgroups run."""
    for counts in ([3, 0, 2], [60, 0, 33, 7], [300, 41]):
        b = Block(counts, 528, 384, seed=10)
        b.run()
        want = b.outputs()
        for _ in range(5):
            b.run()
            for got, exp in zip(b.outputs(), want):
                assert torch.equal(got, exp)


def test_two_calls_at_once():
    """Two blocks on two streams, each with buffers of its own."""
    blocks = [Block([60, 0, 33, 7], 528, 384, seed=7), Block([300, 41], 528, 384, seed=8)]
    want = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        want.append(b.outputs())
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        for b, s in zip(blocks, streams):
            b.run(stream=s)
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for got, exp in zip(b.outputs(), w):
            assert torch.equal(got, exp)
