"""Argument checks of the expert-layer entry points (CPU): every refusal happens before
anything is enqueued, with the documented status; the binding refuses tensors that do not
fit before a pointer reaches the library."""
import functools
import os

import pytest

import block_scaled_precision_bf16tofp4row_amd as mx

A = 0x7F0000000000                                # never read
B = A + 0x1000000
OK, NULL, SHAPE, ALIGN, HIP = (mx.MXFP4_OK, mx.MXFP4_ERR_NULL, mx.MXFP4_ERR_SHAPE, mx.MXFP4_ERR_ALIGN,
                               mx.MXFP4_ERR_HIP)


@pytest.fixture(scope="module")
def lib():
    return mx.load_library()


def _route(lib, l=A, f32=1, bias=A, mask=A, ids=B, w=B, T=3, E=32, ng=4, tg=2, gb=2, k=4, score=0, rn=1, scale=1.0):
    return lib.mxfp4_route_topk(l, f32, bias, mask, ids, w, T, E, ng, tg, gb, k, score, rn, scale, None)


def _route_back(lib, l=A, f32=1, ids=A, dw=A, dl=B, T=3, E=32, k=4, score=1, rn=1, scale=1.0):
    return lib.mxfp4_route_topk_backward(l, f32, ids, dw, dl, T, E, k, score, rn, scale, None)


def _map(lib, ids=A, offs=B, pos=B, src=None, ws=A, T=3, k=2, first=0, G=4, cap=6):
    return lib.mxfp4_expert_map(ids, offs, pos, src, ws, T, k, first, G, cap, None)


def _disp(lib, fn, x=A, pos=A, y=B, s=B, T=3, k=2, cap=6, K=128):
    return getattr(lib, fn)(x, pos, y, s, T, k, cap, K, None)


def _rows(lib, x=A, y=B, s=B, offs=A, G=2, M=4, K=128):
    return lib.mxfp4_bf16_to_fp8_rows_f32(x, y, s, offs, G, M, K, None)


def _gemm(lib, a=A, sa=A, w=A, sw=A, y=B, offs=A, G=2, M=4, N=64, K=128):
    return lib.mxfp4_fp8_block_gemm(a, sa, w, sw, y, offs, G, M, N, K, None)


def _comb(lib, y=A, pos=A, w=A, base=A, out=B, T=3, k=2, cap=6, K=64):
    return lib.mxfp4_combine_rows(y, pos, w, base, out, T, k, cap, K, None)


def _comb_back(lib, dout=A, y=A, pos=A, w=A, dy=B, dw=B, T=3, k=2, cap=6, K=64):
    return lib.mxfp4_combine_rows_backward(dout, y, pos, w, dy, dw, T, k, cap, K, None)


def _refuses(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_route_refusals(lib):
    c = functools.partial(_route, lib)
    _refuses(c, NULL, [dict(l=None), dict(ids=None), dict(w=None)])
    _refuses(c, SHAPE, [dict(T=-1), dict(T=1 << 31), dict(T=1 << 30, k=4), dict(E=0), dict(E=1028), dict(ng=0),
                        dict(ng=5), dict(ng=128, E=1024), dict(tg=0), dict(tg=5), dict(gb=0), dict(gb=3),
                        dict(gb=2, ng=32), dict(k=0), dict(k=17), dict(k=65, E=128, tg=4), dict(score=2),
                        dict(score=-1), dict(scale=float("inf")), dict(scale=float("nan"))])
    _refuses(c, ALIGN, [dict(l=A + 8), dict(bias=A + 4), dict(mask=A + 1), dict(ids=B + 4), dict(w=B + 8)])
    _refuses(c, OK, [dict(T=0), dict(T=0, bias=None, mask=None, f32=0)])
    b = functools.partial(_route_back, lib)
    _refuses(b, NULL, [dict(l=None), dict(ids=None), dict(dw=None), dict(dl=None)])
    _refuses(b, SHAPE, [dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(score=7),
                        dict(scale=float("nan"))])
    _refuses(b, ALIGN, [dict(l=A + 2), dict(ids=A + 4), dict(dw=A + 8), dict(dl=B + 2)])
    assert b(T=0) == OK


def test_map_refusals(lib):
    c = functools.partial(_map, lib)
    _refuses(c, NULL, [dict(ids=None), dict(offs=None), dict(pos=None), dict(T=1 << 20, ws=None)])
    _refuses(c, SHAPE, [dict(T=-1), dict(k=0), dict(k=65), dict(G=0), dict(G=1025), dict(first=-1), dict(cap=-1),
                        dict(cap=1 << 31), dict(T=1 << 30, k=2)])
    _refuses(c, ALIGN, [dict(ids=A + 4), dict(offs=B + 2), dict(pos=B + 8), dict(src=B + 4), dict(ws=A + 4)])
    assert mx.mxfp4_expert_map_workspace(1, 1, 1) == 0
    for T, k, G in ((1 << 20, 8, 1024), (4096, 8, 32), (700, 6, 5)):
        assert 0 <= mx.mxfp4_expert_map_workspace(T, k, G) <= 256 * G
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 65, 1), (1, 1, 0), (1, 1, 1025), (1 << 30, 2, 1)):
        assert mx.mxfp4_expert_map_workspace(*bad) == -1


@pytest.mark.parametrize("fn,step", [("mxfp4_dispatch_rows", 32), ("mxfp4_dispatch_fp8_rows", 16)])
def test_dispatch_refusals(lib, fn, step):
    c = functools.partial(_disp, lib, fn)
    _refuses(c, NULL, [dict(x=None), dict(pos=None), dict(y=None), dict(s=None)])
    _refuses(c, SHAPE, [dict(T=-1), dict(k=0), dict(k=65), dict(cap=-1), dict(cap=1 << 31), dict(K=0), dict(K=-step),
                        dict(K=128 + step // 2), dict(T=1 << 30), dict(T=1 << 30, k=1, K=1 << 21)])
    _refuses(c, ALIGN, [dict(x=A + 2), dict(pos=A + 4), dict(y=B + 8), dict(s=B + 4)])
    _refuses(c, OK, [dict(T=0), dict(cap=0), dict(T=0, K=step)])


def test_rows_and_product_refusals(lib):
    c = functools.partial(_rows, lib)
    _refuses(c, NULL, [dict(x=None), dict(y=None), dict(s=None), dict(offs=None)])
    _refuses(c, SHAPE, [dict(G=0), dict(M=-1), dict(K=0), dict(K=120), dict(M=1 << 31)])
    _refuses(c, ALIGN, [dict(x=A + 4), dict(y=B + 1), dict(s=B + 4), dict(offs=A + 2)])
    assert c(M=0) == OK
    g = functools.partial(_gemm, lib)
    _refuses(g, NULL, [dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(offs=None)])
    _refuses(g, SHAPE, [dict(G=0), dict(M=-1), dict(K=0), dict(K=24), dict(N=0), dict(N=-8), dict(N=12),
                        dict(K=(1 << 20) + 16), dict(N=(1 << 20) + 8), dict(M=1 << 31)])
    _refuses(g, ALIGN, [dict(a=A + 8), dict(sa=A + 4), dict(w=A + 1), dict(sw=A + 4), dict(y=B + 2), dict(offs=A + 1)])
    assert g(M=0) == OK


def test_combine_refusals(lib):
    c = functools.partial(_comb, lib)
    _refuses(c, NULL, [dict(y=None), dict(pos=None), dict(out=None)])
    _refuses(c, SHAPE, [dict(T=-1), dict(k=0), dict(k=65), dict(cap=-1), dict(K=0), dict(K=12), dict(T=1 << 30)])
    _refuses(c, ALIGN, [dict(y=A + 2), dict(pos=A + 4), dict(w=A + 4), dict(base=A + 8), dict(out=B + 2)])
    _refuses(c, OK, [dict(T=0), dict(T=0, w=None, base=None)])
    b = functools.partial(_comb_back, lib)
    _refuses(b, NULL, [dict(dout=None), dict(y=None), dict(pos=None), dict(w=None), dict(dy=None), dict(dw=None)])
    _refuses(b, SHAPE, [dict(T=-1), dict(k=0), dict(K=4), dict(cap=1 << 31)])
    _refuses(b, ALIGN, [dict(dout=A + 2), dict(y=A + 2), dict(pos=A + 4), dict(w=A + 4), dict(dy=B + 2),
                        dict(dw=B + 4)])
    assert b(T=0) == OK


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is present")
def test_valid_calls_without_a_device_report_hip_error(lib):
    assert _route(lib) == HIP and _route_back(lib) == HIP and _map(lib) == HIP and _map(lib, T=1 << 14) == HIP
    assert _disp(lib, "mxfp4_dispatch_rows") == HIP and _disp(lib, "mxfp4_dispatch_fp8_rows") == HIP
    assert _rows(lib) == HIP and _gemm(lib) == HIP and _comb(lib) == HIP and _comb_back(lib) == HIP


def test_binding_checks_tensors():
    """Sizes, types, contiguity and device, on CPU tensors (so nothing is launched)."""
    import torch
    T, E, k, G, K, cap = 3, 16, 2, 4, 256, 6
    f = torch.float32
    l, ids, w = torch.zeros(T, E), torch.zeros((T, k), dtype=torch.int32), torch.zeros(T, k)
    x = torch.zeros((T, K), dtype=torch.bfloat16)
    y = torch.zeros((cap, K), dtype=torch.bfloat16)
    offs = torch.zeros(G + 1, dtype=torch.int32)
    q, s = torch.zeros((cap, K), dtype=torch.uint8), torch.zeros((cap, K // 128))
    raises = functools.partial(pytest.raises, ValueError)
    with raises(match="logits has dtype"):
        mx.mxfp4_route_topk(l.half(), ids, w)
    with raises(match="bias holds"):
        mx.mxfp4_route_topk(l, ids, w, bias=torch.zeros(E - 1))
    with raises(match="row_mask holds"):
        mx.mxfp4_route_topk(l, ids, w, row_mask=torch.zeros(T - 1, dtype=torch.uint8))
    with raises(match="weights holds"):
        mx.mxfp4_route_topk(l, ids, w[:2])
    with raises(match="score must be"):
        mx.mxfp4_route_topk(A, A, A, T=0, E=E, k=k, score="tanh", stream=0)
    with raises(match="contiguous"):
        mx.mxfp4_route_topk(torch.zeros(E, T).t(), ids, w)
    with raises(match="must be a GPU tensor"):
        mx.mxfp4_route_topk(l, ids, w)
    with raises(match="dlogits has dtype"):
        mx.mxfp4_route_topk_backward(l.bfloat16(), ids, w, l)
    with raises(match="ids has dtype"):
        mx.mxfp4_expert_map(ids.long(), offs, ids, None)
    with raises(match="src holds"):
        mx.mxfp4_expert_map(ids, offs, ids, None, src=ids.view(-1), M_cap=7)
    with raises(match="workspace holds"):
        big = torch.zeros((1 << 13, 8), dtype=torch.int32)
        mx.mxfp4_expert_map(big, offs, big, torch.zeros(1, dtype=torch.int32))
    with raises(match="codes holds"):
        mx.mxfp4_dispatch_rows(x, ids, q[:, :64].contiguous(), q)
    with raises(match="y_scales has dtype"):
        mx.mxfp4_dispatch_fp8_rows(x, ids, q, q)
    with raises(match="y_scales holds"):
        mx.mxfp4_bf16_to_fp8_rows_f32(y, q, s[:5], offs)
    with raises(match="w_scales holds"):
        mx.mxfp4_fp8_block_gemm(q, s, torch.zeros((G, 136, K), dtype=torch.uint8), torch.zeros(G, 1, 2), y, offs)
    with raises(match="w holds"):
        mx.mxfp4_fp8_block_gemm(q, s, torch.zeros((3, 64, K), dtype=torch.uint8), torch.zeros(G, 1, 2), y, offs)
    with raises(match="base holds"):
        mx.mxfp4_combine_rows(y, ids, x, weights=w, base=x[:2])
    with raises(match="dweights has dtype"):
        mx.mxfp4_combine_rows_backward(x, y, ids, w, y, w.double())


def test_empty_tensors_are_no_null_pointers():
    """No tokens: the calls succeed and enqueue nothing (torch gives an empty tensor no address)."""
    import torch
    class Gpu:                                    # an empty tensor of a GPU, as far as the binding looks
        def __init__(self, shape, dtype):
            self.t = torch.empty(shape, dtype=dtype)
            self.shape, self.dtype, self.is_cuda = self.t.shape, dtype, True
        def __getattr__(self, n):
            return getattr(self.t, n)
    i, f, b, u = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    e = lambda d, *s: Gpu(s, d)                   # noqa: E731
    mx.mxfp4_route_topk(e(f, 0, 8), e(i, 0, 2), e(f, 0, 2), stream=0)
    mx.mxfp4_route_topk_backward(e(b, 0, 8), e(i, 0, 2), e(f, 0, 2), e(b, 0, 8), stream=0)
    mx.mxfp4_dispatch_rows(e(b, 0, 64), e(i, 0, 2), e(u, 0, 32), e(u, 0, 2), stream=0)
    mx.mxfp4_dispatch_fp8_rows(e(b, 0, 64), e(i, 0, 2), e(u, 0, 64), e(f, 0, 1), stream=0)
    mx.mxfp4_combine_rows(e(b, 0, 64), e(i, 0, 2), e(b, 0, 64), stream=0)
    mx.mxfp4_combine_rows_backward(e(b, 0, 64), e(b, 0, 64), e(i, 0, 2), e(f, 0, 2), e(b, 0, 64), e(f, 0, 2), stream=0)


def test_rows_longer_than_their_counters(lib):
    """A row's lanes are counted in 32 bits: longer rows are refused, not wrapped."""
    for K in (1 << 31, 1 << 37):
        for call in (functools.partial(_disp, lib, "mxfp4_dispatch_rows"),
                     functools.partial(_disp, lib, "mxfp4_dispatch_fp8_rows"), functools.partial(_comb, lib),
                     functools.partial(_comb_back, lib)):
            assert call(T=1, k=1, cap=1, K=K) == SHAPE, (call, K)
        assert _rows(lib, M=1, K=K) == SHAPE, K
