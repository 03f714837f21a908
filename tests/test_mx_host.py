"""Host-side checks of the microscaled entry points (no GPU needed): every bad argument is
refused with the documented status before anything is enqueued."""
import ctypes

import pytest

import bit_group_quantized_qgemv_gb300 as q

EINVAL, ENULL, EALIGN = -1, -2, -3
L = q.lib


def ptr(v=0x10000):
    return ctypes.c_void_p(v)


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values(), None)


P = ptr()
QUANTIZE = dict(bits=4, x=P, m=3, k=64, codes=P, scales=P)
DEQUANTIZE = dict(bits=8, codes=P, scales=P, m=3, k=64, y=P)
NORM = dict(x=P, residual=P, gamma=P, eps=1e-5, m=3, k=64, h=P, codes=P, scales=P)
MATVEC = dict(codes=P, scales=P, x=P, y=P, m=3, n=5, k=64, residual=P)
GEMM = dict(codes=P, scales=P, x=P, xs=P, y=P, m=30, n=5, k=64, residual=P)
GATED = dict(gc=P, gs=P, uc=P, us=P, x=P, xs=P, m=30, i=64, k=64, h=P, hc=P, hs=P)
CALLS = [(L.qgemv_mx_quantize, QUANTIZE, ("x", "codes", "scales"), ("x", "codes"), ()),
         (L.qgemv_mx_dequantize, DEQUANTIZE, ("codes", "scales", "y"), ("codes", "y"), ()),
         (L.qgemv_residual_rmsnorm_mxfp8, NORM, ("x", "gamma", "h", "codes", "scales"),
          ("x", "residual", "gamma", "h", "codes"), ()),
         (L.qgemv_mxfp4, MATVEC, ("codes", "scales", "x", "y"), ("codes", "x"), ("y", "residual")),
         (L.qgemv_mx_gemm, GEMM, ("codes", "scales", "x", "xs", "y"), ("codes", "x"), ("y", "residual")),
         (L.qgemv_mx_swiglu, GATED, ("gc", "gs", "uc", "us", "x", "xs"), ("gc", "uc", "x", "hc"), ("h",))]


@pytest.mark.parametrize("fn,d,required,by16,by2", CALLS, ids=lambda v: getattr(v, "__name__", ""))
def test_pointers_and_rows(fn, d, required, by16, by2):
    for name in required:
        assert call(fn, d, **{name: None}) == ENULL, name
    for name in by16:
        assert call(fn, d, **{name: ptr(0x10008)}) == EALIGN, name
    for name in by2:
        assert call(fn, d, **{name: ptr(0x10001)}) == EALIGN, name
    for kw in (dict(k=0), dict(k=16), dict(k=48), dict(k=65), dict(k=-32), dict(k=2 ** 30 + 32), dict(m=-1),
               dict(m=2 ** 30 + 1, k=32), dict(m=2 ** 30, k=512)):
        assert call(fn, d, **kw) == EINVAL, kw
    # a null pointer before a bad size, a bad size before a bad address
    assert call(fn, d, **{required[0]: None, "k": 48}) == ENULL
    assert call(fn, d, **{by16[0]: ptr(0x10004), "k": 48}) == EINVAL


def test_sizes():
    for bits in (0, 2, 5, 16, -4):
        assert call(L.qgemv_mx_quantize, QUANTIZE, bits=bits) == EINVAL
        assert call(L.qgemv_mx_dequantize, DEQUANTIZE, bits=bits) == EINVAL
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(L.qgemv_residual_rmsnorm_mxfp8, NORM, eps=eps) == EINVAL
    for kw in (dict(m=0), dict(m=9), dict(n=0), dict(n=-1), dict(k=28704), dict(n=2 ** 30 + 1, k=32)):
        assert call(L.qgemv_mxfp4, MATVEC, **kw) == EINVAL, kw
    for fn, d, name in ((L.qgemv_mx_gemm, GEMM, "n"), (L.qgemv_mx_swiglu, GATED, "i")):
        for kw in ({name: 0}, {name: -32}, {name: 2 ** 30 + 1, "k": 32}):
            assert call(fn, d, **kw) == EINVAL, kw
    for i in (1, 31, 33, 48):                     # a whole number of blocks where the result is MXFP8
        assert call(L.qgemv_mx_swiglu, GATED, i=i) == EINVAL
    for kw in (dict(h=None, hc=None, hs=None), dict(hc=None), dict(hs=None)):
        assert call(L.qgemv_mx_swiglu, GATED, **kw) == ENULL, kw


def test_no_rows():
    """Nothing to do: the arrays of rows may be missing, the weights and the norm's may not."""
    for fn, d, gone in ((L.qgemv_mx_quantize, QUANTIZE, ("x", "codes", "scales")),
                        (L.qgemv_mx_dequantize, DEQUANTIZE, ("codes", "scales", "y")),
                        (L.qgemv_residual_rmsnorm_mxfp8, NORM, ("x", "residual", "h", "codes", "scales")),
                        (L.qgemv_mx_gemm, GEMM, ("x", "xs", "y", "residual")),
                        (L.qgemv_mx_swiglu, GATED, ("x", "xs", "h", "hc", "hs"))):
        assert call(fn, d, m=0, **{n: None for n in gone}) == 0
        assert call(fn, d, m=0, k=48) == EINVAL
    assert call(L.qgemv_residual_rmsnorm_mxfp8, NORM, m=0, gamma=None) == ENULL
    assert call(L.qgemv_mx_gemm, GEMM, m=0, codes=None) == ENULL
    assert call(L.qgemv_mx_swiglu, GATED, m=0, us=None) == ENULL


def test_no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for fn, d, *_ in CALLS:
        assert call(fn, d) == -5
