"""Argument checks of the feed-forward entry points (CPU): every refusal happens before
anything is enqueued, with the documented status; the binding refuses tensors that do not fit
before a pointer reaches the library."""
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


def _gated(lib, a=A, sa=A, w=A, sw=A, bias=A, out=B, q=B, qs=B, h=B, ws=B, offs=A, G=2, M=4, I=64, K=128, act=2):
    return lib.mxfp4_fp8_gated_gemm(a, sa, w, sw, bias, out, q, qs, h, ws, offs, G, M, I, K, act, None)


def _back(lib, a=A, sa=A, w=A, sw=A, h=A, dh=B, q=B, qs=B, out=B, ws=B, offs=A, G=2, M=4, I=128, K=128, act=2):
    return lib.mxfp4_fp8_gated_gemm_backward(a, sa, w, sw, h, dh, q, qs, out, ws, offs, G, M, I, K, act, None)


def _dense(lib, a=A, sa=A, w=A, sw=A, bias=A, res=A, pre=B, y=B, offs=A, G=2, M=4, N=64, K=128, act=0):
    return lib.mxfp4_fp8_block_gemm_act(a, sa, w, sw, bias, res, pre, y, offs, G, M, N, K, act, None)


def _rows(lib, dout=A, pre=A, dpre=B, q=B, qs=B, db=B, ws=B, offs=A, G=2, M=4, N=64, act=3):
    return lib.mxfp4_act_rows_backward(dout, pre, dpre, q, qs, db, ws, offs, G, M, N, act, None)


def _refuses(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


PRODUCT_SHAPES = [dict(G=0), dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=24), dict(K=(1 << 20) + 16), dict(act=-1),
                  dict(act=5)]


def test_gated_refusals(lib):
    c = functools.partial(_gated, lib)
    _refuses(c, NULL, [dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(offs=None), dict(q=None),
                       dict(qs=None), dict(out=None, q=None, qs=None), dict(ws=None, M=1, I=2048, K=7168)])
    _refuses(c, SHAPE, PRODUCT_SHAPES + [dict(I=0), dict(I=-8), dict(I=12), dict(I=72), dict(I=(1 << 19) + 16)])
    _refuses(c, ALIGN, [dict(a=A + 8), dict(sa=A + 4), dict(w=A + 1), dict(sw=A + 4), dict(bias=A + 4), dict(out=B + 2),
                        dict(q=B + 8), dict(qs=B + 4), dict(h=B + 2), dict(ws=B + 4), dict(offs=A + 2)])
    _refuses(c, OK, [dict(M=0), dict(M=0, I=72, q=None, qs=None), dict(M=0, ws=None, I=2048, K=7168), dict(M=0, out=None, h=None)])


def test_gated_backward_refusals(lib):
    c = functools.partial(_back, lib)
    _refuses(c, NULL, [dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(h=None), dict(offs=None),
                       dict(q=None), dict(qs=None), dict(dh=None, q=None, qs=None), dict(ws=None, M=1, I=256, K=4096)])
    _refuses(c, SHAPE, PRODUCT_SHAPES + [dict(I=0), dict(I=12), dict(I=64), dict(I=(1 << 19) + 128)])
    _refuses(c, ALIGN, [dict(a=A + 8), dict(sa=A + 4), dict(w=A + 1), dict(sw=A + 4), dict(h=A + 4), dict(dh=B + 2),
                        dict(q=B + 8), dict(qs=B + 4), dict(out=B + 2), dict(ws=B + 4), dict(offs=A + 2)])
    _refuses(c, OK, [dict(M=0), dict(M=0, I=72, q=None, qs=None), dict(M=0, dh=None, out=None)])


def test_dense_refusals(lib):
    c = functools.partial(_dense, lib)
    _refuses(c, NULL, [dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(offs=None)])
    _refuses(c, SHAPE, PRODUCT_SHAPES + [dict(N=0), dict(N=-8), dict(N=12), dict(N=(1 << 20) + 8)])
    _refuses(c, ALIGN, [dict(a=A + 8), dict(sa=A + 4), dict(w=A + 1), dict(sw=A + 4), dict(bias=A + 4), dict(res=A + 2),
                        dict(pre=B + 2), dict(y=B + 2), dict(offs=A + 1)])
    _refuses(c, OK, [dict(M=0), dict(M=0, bias=None, res=None, pre=None)])


def test_act_rows_refusals(lib):
    c = functools.partial(_rows, lib)
    _refuses(c, NULL, [dict(dout=None), dict(offs=None), dict(pre=None), dict(q=None), dict(qs=None),
                       dict(dpre=None, q=None, qs=None, db=None), dict(M=4096, ws=None)])
    _refuses(c, SHAPE, [dict(G=0), dict(M=-1), dict(M=1 << 31), dict(N=0), dict(N=12), dict(N=72), dict(N=(1 << 20) + 8),
                        dict(act=-1), dict(act=9)])
    _refuses(c, ALIGN, [dict(dout=A + 2), dict(pre=A + 2), dict(dpre=B + 2), dict(q=B + 8), dict(qs=B + 4),
                        dict(db=B + 4), dict(ws=B + 4), dict(offs=A + 2)])
    _refuses(c, OK, [dict(M=0, db=None), dict(M=0, db=None, pre=None, act=0)])


def test_workspaces():
    one = mx.mxfp4_fp8_gated_gemm_workspace
    back = mx.mxfp4_fp8_gated_gemm_backward_workspace
    assert one(1, 1, 2048, 7168) == 4 * 2048 and back(1, 1, 2048, 7168) == 8 * 2048
    rows = mx.mxfp4_act_rows_backward_workspace
    assert rows(3, 5, 64) == 0 and rows(8, 32768, 4096) == 4 * 4096 * (32768 // 32 + 7)
    # enough for every call of fewer rows
    for G in (1, 7, 40):
        for fn in (lambda M: one(G, M, 1040, 512), lambda M: back(G, M, 1024, 512), lambda M: rows(G, M, 1040)):      # noqa: E731
            sizes = [fn(M) for M in (0, 1, 3, 40, 128, 129, 500, 2000, 4000, 8000, 100000)]
            assert sizes == sorted(sizes), (G, sizes)
    assert one(8, 1 << 30, 2048, 7168) == back(8, 1 << 30, 2048, 7168) == 1 << 24
    for fn in (one, mx.mxfp4_fp8_gated_gemm_backward_workspace):
        for bad in ((0, 1, 64, 128), (1, -1, 64, 128), (1, 1, 12, 128), (1, 1, 64, 24), (1, 1, (1 << 19) + 8, 128)):
            assert fn(*bad) == -1, bad
    for bad in ((0, 1, 64), (1, -1, 64), (1, 1, 12), (1, 1, (1 << 20) + 8)):
        assert mx.mxfp4_act_rows_backward_workspace(*bad) == -1, bad


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is present")
def test_valid_calls_without_a_device_report_hip_error(lib):
    for c in (_gated, _back, _dense, _rows):
        for M in (1, 4, 300, 20000):
            assert c(lib, M=M) == HIP, (c, M)
    assert _rows(lib, M=0) == HIP                 # the zero bias gradients
    assert _rows(lib, pre=None, act=0) == HIP


def test_binding_checks_tensors():
    """Sizes, types, contiguity and device, on CPU tensors (so nothing is launched)."""
    import torch
    M, I, K, G = 4, 64, 256, 2
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)             # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)          # noqa: E731
    offs = torch.zeros(G + 1, dtype=torch.int32)
    a, sa, w, sw = u8(M, K), torch.zeros(M, 2), u8(G, 2 * I, K), torch.zeros(G, 2, 1, 2)
    raises = functools.partial(pytest.raises, ValueError)
    call = functools.partial(mx.mxfp4_fp8_gated_gemm, a, sa, w, sw, offs)
    for kw, match in ((dict(out=bf(M, I - 1)), "out holds"), (dict(out=u8(M, 2 * I)), "out has dtype"),
                      (dict(out=bf(M, I), h=bf(M, I)), "h holds"), (dict(out=bf(M, I), bias=torch.zeros(G, I)), "bias holds"),
                      (dict(q=u8(M, I), q_scales=torch.zeros(M, 1)[:3]), "q_scales holds"),
                      (dict(out=bf(I, M).t()), "out must be contiguous"), (dict(out=bf(M, I)), "must be a GPU tensor")):
        with raises(match=match):
            call(**kw)
    with raises(match="workspace holds"):
        call(q=u8(M, I), q_scales=torch.zeros(M, 1), workspace=u8(16))
    with raises(match="act must be one of"):
        mx.mxfp4_fp8_gated_gemm(1, 1, 1, 1, 1, out=1, act="swish", G=1, M_cap=0, I=16, K=16)
    with raises(match="w_scales holds"):
        mx.mxfp4_fp8_gated_gemm(a, sa, w, torch.zeros(G, 1, 1, 2), offs, out=bf(M, I))
    for bad in (u8(2, I + 1, K), u8(G, 2 * I + 1, K), u8(G, 2 * I, K - 16), u8(G + 1, 2 * I, K)):
        with raises(match="w has shape"):
            mx.mxfp4_fp8_gated_gemm(a, sa, bad, sw, offs, out=bf(M, I))
    for bad in (u8(I, K), u8(G, I, K - 16), u8(G + 1, I, K)):
        with raises(match="w has shape"):
            mx.mxfp4_fp8_block_gemm_act(a, sa, bad, sw, bf(M, I), offs)
    back = functools.partial(mx.mxfp4_fp8_gated_gemm_backward, a, sa, u8(G, I, K), torch.zeros(G, 1, 2))
    with raises(match="h holds"):
        back(bf(M, I), offs, dh=bf(M, 2 * I))
    with raises(match="dh holds"):
        back(bf(M, 2 * I), offs, dh=bf(M, I))
    with raises(match="must be a GPU tensor"):
        back(bf(M, 2 * I), offs, dh=bf(M, 2 * I))
    dense = functools.partial(mx.mxfp4_fp8_block_gemm_act, a, sa, u8(G, I, K), torch.zeros(G, 1, 2))
    for kw, match in ((dict(bias=torch.zeros(I)), "bias holds"), (dict(residual=bf(M - 1, I)), "residual holds"),
                      (dict(pre=torch.zeros(M, I)), "pre has dtype"), (dict(), "must be a GPU tensor")):
        with raises(match=match):
            dense(bf(M, I), offs, **kw)
    rows = functools.partial(mx.mxfp4_act_rows_backward, bf(M, I))
    for kw, match in ((dict(dbias=torch.zeros(I)), "dbias holds"), (dict(dpre=bf(M, 8)), "dpre holds"),
                      (dict(q=u8(M, I), q_scales=torch.zeros(M - 1, 1)), "q_scales holds"),
                      (dict(dpre=bf(M, I)), "must be a GPU tensor")):
        with raises(match=match):
            rows(bf(M, I), offs, act="gelu", **kw)
