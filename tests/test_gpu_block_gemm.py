"""The expert product with FP32 block scales against the float64 product of the same bytes.

    |y - exact| <= 2^-8 |exact| + (1 + 2^-8) (2^-10 + (K / 128 + 4) 2^-24) sum|terms| + 2^-133
(2^-8 |exact|: BF16; 2^-10: the matrix core's own rounding of a 64-term dot product, as
test_gpu_gemm measures it, with margin; the rest the FP32 sum over the blocks.)  Over all
outputs the 2-norm of the error stays below 2^-8 of the result's.
"""
from __future__ import annotations

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402


def operands(offs, M_cap, N, K, seed):
    rng = np.random.default_rng(seed)
    G = len(offs) - 1
    kb, nb = -(-K // 128), -(-N // 128)

    def codes(shape):
        b = rng.integers(0, 256, size=shape, dtype=np.int64)
        return np.where((b & 0x7F) == 0x7F, b - 1, b).astype(np.uint8)

    sa = np.exp(rng.normal(size=(M_cap, kb)) * 2).astype(np.float32)
    sw = (np.exp(rng.normal(size=(G, nb, kb))) * 0.01).astype(np.float32)
    return codes((M_cap, K)), sa, codes((G, N, K)), sw


def check(counts, N, K, slack=3, seed=0):
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(offs[-1])
    M_cap = M + slack
    a, sa, w, sw = operands(offs, M_cap, N, K, seed)
    a[M:] = 0x7F                                  # NaN bytes and scales past the last row are not used
    sa[M:] = np.nan
    y = torch.full((M_cap, N), -3.0, dtype=torch.bfloat16, device="cuda")
    dev = lambda v: torch.from_numpy(v).cuda()    # noqa: E731
    mx.mxfp4_fp8_block_gemm(dev(a), dev(sa), dev(w), dev(sw), y, dev(offs))
    exact, mag = ref.block_product(a[:M], sa[:M], w, sw, offs)
    got = y.double().cpu().numpy()
    assert (got[M:] == -3).all()
    got = got[:M]
    bound = 2.0 ** -8 * np.abs(exact) + (1 + 2.0 ** -8) * (2.0 ** -10 + (K / 128 + 4) * 2.0 ** -24) * mag + 2.0 ** -133
    bad = np.argwhere(~(np.abs(got - exact) <= bound))
    assert not len(bad), (len(bad), bad[:5], got[tuple(bad[0])], exact[tuple(bad[0])])
    if M:
        assert np.linalg.norm(got - exact) <= 2.0 ** -8 * np.linalg.norm(exact)


@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 16), ([1], 256, 128), ([3], 24, 144), ([0, 1, 0, 2], 136, 272), ([16], 512, 1024), ([17], 512, 1024),
    ([1] * 40, 256, 512), ([0] * 5, 64, 64), ([33, 0, 5], 1000, 336), ([64, 65, 63], 384, 640),
    ([128], 576, 1536), ([100, 1, 300, 0, 127], 520, 1040), ([257], 1352, 1744), ([511, 3], 256, 2048),
    ([700, 41], 640, 2064), ([1025], 264, 400), ([2, 0, 4, 1, 7, 0, 3, 8], 2048, 7168), ([5, 1, 0, 31, 12], 4096, 1040),
    ([300] * 3, 128, 112), ([1500], 768, 896),
])
def test_product(counts, N, K):
    check(counts, N, K)


@pytest.mark.parametrize("counts,N,K", [
    ([2500, 0, 700], 4104, 400),                  # large tiles, ragged in all three directions
    ([1100], 12288, 144),
    ([70, 0, 64, 33, 129, 1, 90, 128], 7176, 272),     # medium tiles, many of them
    ([301, 300, 280], 1544, 528),                 # medium tiles, few of them
    ([1, 0, 2, 1, 0, 1, 3, 0] * 10, 1032, 656),   # about a row per expert
    ([1] * 300, 520, 240),                        # more experts than a wave has lanes
    ([0] * 130 + [9] + [0] * 70 + [40], 264, 144),
])
def test_every_kernel(counts, N, K):
    check(counts, N, K, seed=N)


@pytest.mark.parametrize("K", [16, 144, 272, 400, 528])
@pytest.mark.parametrize("counts,N", [
    ([16, 0, 5], 1032),                           # waves that share K, 16 tokens
    ([121], 2040),                                # the same, 32 tokens
    ([17, 0, 13], 4104),                          # 32 x 128, one workgroup per CU
    ([3, 0, 9, 1, 0, 33, 2, 5], 4104),            # 32 x 128, several
    ([100, 0, 130], 4104),                        # 128 x 128, one workgroup per CU
    ([50, 51, 49, 0, 64, 1, 100, 85], 8200),      # 128 x 128, several
    ([500, 3], 12296),
    ([900, 3], 12296),                            # 256 x 256
])
def test_every_kernel_at_every_stage_count(counts, N, K):
    """One to five blocks of K, the last one partial: fewer and more than a kernel's buffers."""
    check(counts, N, K, seed=K + N)


@pytest.mark.parametrize("counts,N,K", [
    ([9, 8], 4104, 4096),
    ([9, 8, 7], 4104, 4096),                      # 32 x 128, one per CU
    ([1, 0, 2, 1, 0, 1, 1, 1] * 12, 264, 4096),   # 32 x 128, several workgroups per CU
    ([5], 520, 7184), ([40], 2048, 8192),
])
def test_deep(counts, N, K):
    """Rows a multiple of 4096 bytes apart, whose blocks are taken in turned order, and others."""
    check(counts, N, K, seed=N)


@pytest.mark.parametrize("M", [1, 2, 8, 15, 31, 32, 33, 47, 48, 96, 192, 255, 256, 320])
def test_row_counts(M):
    check([M], 384, 512, slack=0, seed=M)


@pytest.mark.parametrize("K", [16, 48, 112, 128, 144, 240, 256, 272, 384, 496, 512, 1136])
@pytest.mark.parametrize("M", [7, 300])
def test_widths(K, M):
    check([M], 136, K, seed=K)


@pytest.mark.parametrize("N", [8, 16, 56, 64, 120, 128, 136, 200, 248, 256, 264])
@pytest.mark.parametrize("M", [5, 300])
def test_features(N, M):
    check([M, 2], N, 272, seed=N)


def test_no_rows_and_no_experts_with_rows():
    y = torch.full((4, 64), -3.0, dtype=torch.bfloat16, device="cuda")
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")     # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")                          # noqa: E731
    mx.mxfp4_fp8_block_gemm(z(4, 128), f(4, 1), z(2, 64, 128), f(2, 1, 1), y, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert (y == -3).all()


def test_scales_of_zero_and_far_apart():
    """A zero scale takes its block out; scales 2^-60 and 2^60 keep their blocks' precision."""
    M, N, K = 40, 128, 512
    a, sa, w, sw = operands([0, M], M, N, K, 5)
    sa[:, 1] = 0
    sw[:, :, 2] = 2.0 ** -60
    sa[:, 2] = 2.0 ** 60
    offs = np.array([0, M], np.int32)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    dev = lambda v: torch.from_numpy(v).cuda()    # noqa: E731
    mx.mxfp4_fp8_block_gemm(dev(a), dev(sa), dev(w), dev(sw), y, dev(offs))
    exact, mag = ref.block_product(a, sa, w, sw, offs)
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - exact) <= 2.0 ** -8 * np.abs(exact) + 2.0 ** -9 * mag + 2.0 ** -133)


def test_activation_gradient_by_transposed_weights():
    """dX = dY W: the same entry point on the transposed weights and scales, against the
    float64 product and against differences of the float64 forward (which is linear)."""
    counts, N, K = [37, 0, 90], 256, 384
    offs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(offs[-1])
    dy, sdy, w, sw = operands(offs, M, N, K, 8)
    dy, sdy = dy[:, :N].copy(), np.abs(sdy[:, :N // 128]).copy()
    wt = np.ascontiguousarray(w.transpose(0, 2, 1))
    swt = np.ascontiguousarray(sw.transpose(0, 2, 1))
    dx = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    dev = lambda v: torch.from_numpy(v).cuda()    # noqa: E731
    mx.mxfp4_fp8_block_gemm(dev(dy), dev(sdy), dev(wt), dev(swt), dx, dev(offs))
    got = dx.double().cpu().numpy()
    exact, mag = ref.block_product(dy, sdy, wt, swt, offs)
    assert np.all(np.abs(got - exact) <= 2.0 ** -8 * np.abs(exact) + 2.0 ** -9 * mag + 2.0 ** -133)
    # f(X) = <dY, X W^T> is linear: its difference along unit vector (m, k) is dX[m, k]
    dyv = ref.e4m3(dy) * sdy.astype(np.float64)[:, np.arange(N) // 128]
    for m, k in ((0, 0), (36, 383), (37, 130), (126, 255)):
        g = int(np.searchsorted(offs, m, side="right")) - 1
        wv = ref.e4m3(w[g]) * sw[g].astype(np.float64)[np.arange(N) // 128][:, np.arange(K) // 128]
        step = np.zeros(K)
        step[k] = 1.0
        diff = (dyv[m] @ (wv @ step) - dyv[m] @ (wv @ -step)) / 2
        assert abs(got[m, k] - diff) <= 2.0 ** -8 * abs(diff) + 2.0 ** -9 * mag[m, k] + 2.0 ** -133
