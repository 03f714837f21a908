"""ctypes binding of libqgemv.so: argument marshalling only.

Each function takes torch tensors that already live on the GPU, passes their
device pointers and shapes to the C ABI of the same name (include/qgemv.h)
on the current torch stream, and raises ``QgemvError`` on a non-zero status.
Every step of the computation runs in the library's CUDA kernels; there is
no fallback: if the library cannot be loaded, importing fails loudly.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import build as _build

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_L = ctypes.c_longlong

_SIGS = {
    "qgemv_w4g64": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "qgemv_w2g64": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "qgemv_w8g64": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "rmsnorm_qgemv": (_I, [_P, _P, _P, _P, _P, _F, _P, _I, _I, _P]),
    "swiglu_qgemv": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _I, _I, _P]),
    "moe_qgemv_combine": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _P, _P,
                               _P, _P, _P, _P]),
    "moe_qgemv_combine_traced": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _P, _P,
                                      _P, _P, _P, _P, _I, ctypes.POINTER(_I), _P]),
    "qgemv_moe_workspace_bytes": (ctypes.c_size_t, [_I, _I]),
    "moe_qgemv_combine_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _P, _P,
                                       _P, _P, _P]),
    "qgemv_noalloc_max_scratch": (ctypes.c_size_t, []),
    "decode_attention_seq1": (_I, [_P, _P, _I, _I, _I, _P]),
    "qgemv_decode_stack_workspace_bytes": (ctypes.c_size_t, [_P]),
    "qgemv_decode_stack": (_I, [_P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "qgemv_strerror": (ctypes.c_char_p, [_I]),
    "qgemv_last_cuda_error": (_I, []),
    "qgemv_device_status": (_I, [ctypes.POINTER(ctypes.c_uint)]),
    "qgemv_version": (_I, []),
    "qgemv_selftest_wait_timeout": (_I, [ctypes.c_uint, ctypes.c_void_p]),
    "qgemv_lm_head_argmax": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _P, _P]),
    "qgemv_argmax_scratch_bytes": (ctypes.c_size_t, []),
    "qgemv_moe_router": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "qgemv_residual_rmsnorm": (_I, [_P, _P, _P, _F, _I, _P, _P, _P]),
    "qgemv_sample_topk": (_I, [_P, _I, _I, _F, _P, _P, _P, _P, _P]),
    "qgemv_lut4": (_I, [_P, _P, _I, _I, _P, _P, _I, _I, _P, _P]),
    "qgemv_lm_head_sample": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _F, _P, _P, _P, _P, _P]),
    "qgemv_plan_gemv": (_I, [_I, _I, _I, _I, _I, _I, _P]),
    "qgemv_qk_norm_rope_append": (_I, [_P, _P, _L, _I, _I, _P, _P, _P, _I, _I, _P, _P, _F, _P, _L,
                                       _P, _P, _P, _P]),
    "qgemv_paged_attention": (_I, [_P, _P, _L, _I, _I, _P, _I, _F, _P, _L, _P, _P, ctypes.c_size_t,
                                   _P, _P]),
    "qgemv_paged_attention_workspace_bytes": (ctypes.c_size_t, [_P, _I, _I, _I]),
    "qgemv_attention_mass": (_I, [_P, _P, _L, _I, _I, _P, _I, _F, _P, _P, _P, _P, _P]),
    "qgemv_cache_evict": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "qgemv_mx_quantize": (_I, [_I, _P, _I, _I, _P, _P, _P]),
    "qgemv_mx_dequantize": (_I, [_I, _P, _P, _I, _I, _P, _P]),
    "qgemv_residual_rmsnorm_mxfp8": (_I, [_P, _P, _P, _F, _I, _I, _P, _P, _P, _P]),
    "qgemv_mxfp4": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "qgemv_mx_gemm": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "qgemv_mx_swiglu": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
}


class GemvPlan(ctypes.Structure):
    """qgemv_gemv_plan (include/qgemv.h)."""
    _fields_ = [(n, ctypes.c_int) for n in
                ("path", "passes", "m_pad", "cluster", "chunk_k", "stages", "smem_bytes")]


#: QGEMV_PATH_* of include/qgemv.h, by value.
GEMV_PATHS = ("generic", "stream", "mma", "mma_passes", "batch", "batch_passes")

#: Names the C header declares (the binding exposes each one).
EXPORTED = tuple(_SIGS)


class QgemvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({strerror(status)})")


def _load():
    path = os.environ.get("QGEMV_LIB") or _build.LIB
    if not os.path.exists(path):
        raise ImportError(
            f"libqgemv.so not found at {path}; build it first with "
            "`python -m bit_group_quantized_qgemv_gb300.build` (needs nvcc)")
    handle = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


lib = _load()


def strerror(status: int) -> str:
    return lib.qgemv_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise QgemvError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _cuda(t, dtypes, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_CODES = (torch.int32, getattr(torch, "uint32", torch.int32))
_F16 = (torch.float16,)
_HALF, _F32, _I32 = torch.float16, torch.float32, torch.int32


def _weight(w, name):
    codes, scales, biases = w
    return (_cuda(codes, _CODES, name + ".codes"), _cuda(scales, _F16, name + ".scales"),
            _cuda(biases, _F16, name + ".biases"))


def _plain(fn, bits, w, x, y, residual, stream):
    codes, scales, biases = _weight(w, "w")
    x = _cuda(x, _F16, "x")
    N = codes.shape[-2]
    K = codes.shape[-1] * 32 // bits
    M = 1 if x.dim() == 1 else x.shape[0]
    if y is None:
        y = torch.empty((N,) if x.dim() == 1 else (M, N), dtype=torch.float16, device=x.device)
    _cuda(y, _F16, "y")
    _cuda(residual, _F16, "residual")
    st = fn(_ptr(codes), _ptr(scales), _ptr(biases), _ptr(x), _ptr(y), M, N, K,
            _ptr(residual), _stream(stream))
    _check(st, fn.__name__)
    return y


def qgemv_w4g64(w, x, y=None, residual=None, stream=None):
    """y = W x (+ residual) for a 4-bit g64 weight w = (codes, scales, biases)."""
    return _plain(lib.qgemv_w4g64, 4, w, x, y, residual, stream)


def qgemv_w2g64(w, x, y=None, residual=None, stream=None):
    """y = W x (+ residual) for a 2-bit g64 weight w = (codes, scales, biases)."""
    return _plain(lib.qgemv_w2g64, 2, w, x, y, residual, stream)


def residual_rmsnorm(x, gamma, residual=None, eps=1e-5, h=None, xn=None, stream=None):
    """qgemv_residual_rmsnorm: h = x + residual (fp16; x itself when residual
    is None), xn = RMSNorm(h) * gamma (fp16).  Returns (h, xn)."""
    x = _cuda(x, _F16, "x")
    gamma = _cuda(gamma, _F16, "gamma")
    _cuda(residual, _F16, "residual")
    K = x.shape[-1]
    if residual is not None and h is None:
        h = torch.empty(K, dtype=torch.float16, device=x.device)
    if xn is None:
        xn = torch.empty(K, dtype=torch.float16, device=x.device)
    st = lib.qgemv_residual_rmsnorm(_ptr(x), _ptr(residual), _ptr(gamma), float(eps), K, _ptr(h),
                                    _ptr(xn), _stream(stream))
    _check(st, "qgemv_residual_rmsnorm")
    return (h if residual is not None else x), xn


def moe_router(w, x, top_k=4, shared=0, logits=None, idx=None, wt=None, stream=None):
    """MoE routing on the GPU (qgemv_moe_router): logits = Wr x (4-bit g64),
    idx = shared expert + top routed experts, wt = softmax of their logits.
    Returns (idx int32 [top_k], wt float32 [top_k], logits fp16 [E])."""
    codes, scales, biases = _weight(w, "w")
    x = _cuda(x, _F16, "x")
    E = codes.shape[-2]
    H = codes.shape[-1] * 8
    if logits is None:
        logits = torch.empty(E, dtype=torch.float16, device=x.device)
    if idx is None:
        idx = torch.empty(top_k, dtype=torch.int32, device=x.device)
    if wt is None:
        wt = torch.empty(top_k, dtype=torch.float32, device=x.device)
    _cuda(logits, _F16, "logits")
    _cuda(idx, (torch.int32,), "idx")
    _cuda(wt, (torch.float32,), "wt")
    st = lib.qgemv_moe_router(_ptr(codes), _ptr(scales), _ptr(biases), _ptr(x), E, H, int(top_k),
                              int(shared), _ptr(logits), _ptr(idx), _ptr(wt), _stream(stream))
    _check(st, "qgemv_moe_router")
    return idx, wt, logits


def argmax_scratch_bytes() -> int:
    return int(lib.qgemv_argmax_scratch_bytes())


def plan_gemv(bits, M, N, K, sms, aligned16=True):
    """The kernels qgemv_w4g64 / w2g64 / w8g64 take for a shape
    (qgemv_plan_gemv; host-only): a dict with the path name and its plan."""
    out = GemvPlan()
    _check(lib.qgemv_plan_gemv(int(bits), int(M), int(N), int(K), int(sms), int(bool(aligned16)),
                               ctypes.byref(out)), "qgemv_plan_gemv")
    d = {n: getattr(out, n) for n, _ in GemvPlan._fields_}
    d["path"] = GEMV_PATHS[d["path"]]
    return d


def lm_head_argmax(w, x, logits=None, scratch=None, token=None, stream=None):
    """Greedy lm_head (qgemv_lm_head_argmax): logits = W x (4-bit g64) and
    token = the lowest index of the largest logit, both on the device.
    `scratch` (uint8, argmax_scratch_bytes(), zero before first use; left
    zero) may be kept across calls; a fresh zeroed one is made if None.
    Returns (token int32 [1], logits fp16 [N])."""
    codes, scales, biases = _weight(w, "w")
    x = _cuda(x, _F16, "x")
    N = codes.shape[-2]
    K = codes.shape[-1] * 8  # 4-bit: 8 codes per 32-bit word
    if logits is None:
        logits = torch.empty(N, dtype=torch.float16, device=x.device)
    if scratch is None:
        scratch = torch.zeros(argmax_scratch_bytes(), dtype=torch.uint8, device=x.device)
    if token is None:
        token = torch.empty(1, dtype=torch.int32, device=x.device)
    _cuda(logits, _F16, "logits")
    _cuda(token, (torch.int32,), "token")
    st = lib.qgemv_lm_head_argmax(_ptr(codes), _ptr(scales), _ptr(biases), _ptr(x), _ptr(logits),
                                  N, K, _ptr(scratch), _ptr(token), _stream(stream))
    _check(st, "qgemv_lm_head_argmax")
    return token, logits


def _sample_outputs(device, top_k, u, token, want_topk, topk_idx, topk_prob):
    u = _cuda(u, (torch.float32,), "u")
    if token is None:
        token = torch.empty(1, dtype=torch.int32, device=device)
    _cuda(token, (torch.int32,), "token")
    if want_topk:
        if topk_idx is None:
            topk_idx = torch.empty(top_k, dtype=torch.int32, device=device)
        if topk_prob is None:
            topk_prob = torch.empty(top_k, dtype=torch.float32, device=device)
    _cuda(topk_idx, (torch.int32,), "topk_idx")
    _cuda(topk_prob, (torch.float32,), "topk_prob")
    return u, token, topk_idx, topk_prob


def sample_topk(logits, top_k, temperature, u, token=None, want_topk=False, topk_idx=None,
                topk_prob=None, stream=None):
    """Top-k sampling on the device (qgemv_sample_topk) from fp16 logits [N];
    u: fp32 [1] on the device (the caller's random number in [0, 1)).
    Returns (token int32 [1], topk_idx int32 [top_k] or None, topk_prob fp32
    [top_k] or None); the candidate outputs are made when want_topk."""
    logits = _cuda(logits, _F16, "logits")
    u, token, topk_idx, topk_prob = _sample_outputs(logits.device, top_k, u, token, want_topk,
                                                    topk_idx, topk_prob)
    st = lib.qgemv_sample_topk(_ptr(logits), logits.numel(), int(top_k), float(temperature),
                               _ptr(u), _ptr(token), _ptr(topk_idx), _ptr(topk_prob),
                               _stream(stream))
    _check(st, "qgemv_sample_topk")
    return token, topk_idx, topk_prob


def lm_head_sample(w, x, top_k, temperature, u, logits=None, token=None, want_topk=False,
                   topk_idx=None, topk_prob=None, stream=None):
    """lm_head matvec (4-bit g64) then top-k sampling (qgemv_lm_head_sample).
    Returns (token, logits, topk_idx, topk_prob) as sample_topk."""
    codes, scales, biases = _weight(w, "w")
    x = _cuda(x, _F16, "x")
    N = codes.shape[-2]
    K = codes.shape[-1] * 8  # 4-bit: 8 codes per 32-bit word
    if logits is None:
        logits = torch.empty(N, dtype=torch.float16, device=x.device)
    _cuda(logits, _F16, "logits")
    u, token, topk_idx, topk_prob = _sample_outputs(x.device, top_k, u, token, want_topk,
                                                    topk_idx, topk_prob)
    st = lib.qgemv_lm_head_sample(_ptr(codes), _ptr(scales), _ptr(biases), _ptr(x),
                                  _ptr(logits), N, K, int(top_k), float(temperature), _ptr(u),
                                  _ptr(token), _ptr(topk_idx), _ptr(topk_prob), _stream(stream))
    _check(st, "qgemv_lm_head_sample")
    return token, logits, topk_idx, topk_prob


def qgemv_lut4(codes, lut, x, rows_per_lut=1, y=None, residual=None, stream=None):
    """LUT / palettised 4-bit GEMV (qgemv_lut4): y[n] = sum_k
    lut[n // rows_per_lut][q[n][k]] x[k] (+ residual[n]).  codes: int32/uint32
    view [N][K/8] on the device; lut: fp16 [n_luts][16]; x: fp16 [K]."""
    codes = _cuda(codes, _CODES, "codes")
    lut = _cuda(lut, _F16, "lut")
    x = _cuda(x, _F16, "x")
    if lut.dim() != 2 or lut.shape[1] != 16:
        raise ValueError("lut must be fp16 [n_luts][16]")
    N, K = codes.shape[-2], codes.shape[-1] * 8
    if y is None:
        y = torch.empty(N, dtype=torch.float16, device=x.device)
    _cuda(y, _F16, "y")
    residual = _cuda(residual, _F16, "residual")
    st = lib.qgemv_lut4(_ptr(codes), _ptr(lut), lut.shape[0], int(rows_per_lut), _ptr(x), _ptr(y),
                        N, K, _ptr(residual), _stream(stream))
    _check(st, "qgemv_lut4")
    return y


def qgemv_w8g64(w, x, y=None, residual=None, stream=None):
    """y = W x (+ residual) for an 8-bit g64 weight w = (codes, scales, biases)."""
    return _plain(lib.qgemv_w8g64, 8, w, x, y, residual, stream)


def rmsnorm_qgemv(w, x, norm_weight, eps=1e-5, y=None, stream=None):
    codes, scales, biases = _weight(w, "w")
    x = _cuda(x, _F16, "x")
    _cuda(norm_weight, _F16, "norm_weight")
    N, K = codes.shape[-2], codes.shape[-1] * 8
    if y is None:
        y = torch.empty(N, dtype=torch.float16, device=x.device)
    st = lib.rmsnorm_qgemv(_ptr(codes), _ptr(scales), _ptr(biases), _ptr(x), _ptr(norm_weight),
                           float(eps), _ptr(y), N, K, _stream(stream))
    _check(st, "rmsnorm_qgemv")
    return y


def swiglu_qgemv(gate, up, x, norm_weight=None, eps=1e-5, h=None, stream=None):
    gc, gs, gb = _weight(gate, "gate")
    uc, us, ub = _weight(up, "up")
    x = _cuda(x, _F16, "x")
    _cuda(norm_weight, _F16, "norm_weight")
    I, K = gc.shape[-2], gc.shape[-1] * 8
    if h is None:
        h = torch.empty(I, dtype=torch.float16, device=x.device)
    st = lib.swiglu_qgemv(_ptr(gc), _ptr(gs), _ptr(gb), _ptr(uc), _ptr(us), _ptr(ub), _ptr(x),
                          _ptr(norm_weight), float(eps), _ptr(h), I, K, _stream(stream))
    _check(st, "swiglu_qgemv")
    return h


def moe_workspace_bytes(top_k: int, inter: int) -> int:
    return int(lib.qgemv_moe_workspace_bytes(int(top_k), int(inter)))


def moe_qgemv_combine(gu, dn, expert_idx, expert_w, x, residual=None, y=None, workspace=None,
                      err_flag=None, stream=None):
    """gu = (codes [E][2I][H/8], scales, biases), dn = (codes [E][H][I/8], ...)."""
    gc, gs, gb = _weight(gu, "gu")
    dc, ds, db = _weight(dn, "dn")
    _cuda(expert_idx, (torch.int32,), "expert_idx")
    _cuda(expert_w, (torch.float32,), "expert_w")
    x = _cuda(x, _F16, "x")
    _cuda(residual, _F16, "residual")
    E, I2, H8 = gc.shape
    I, H = I2 // 2, H8 * 8
    top_k = expert_idx.numel()
    if y is None:
        y = torch.empty(H, dtype=torch.float16, device=x.device)
    if workspace is None:
        workspace = torch.empty(top_k * I, dtype=torch.float32, device=x.device)
    _cuda(workspace, (torch.float32,), "workspace")
    _cuda(err_flag, (torch.int32,), "err_flag")
    st = lib.moe_qgemv_combine(_ptr(gc), _ptr(gs), _ptr(gb), _ptr(dc), _ptr(ds), _ptr(db), E, H,
                               I, _ptr(expert_idx), _ptr(expert_w), top_k, _ptr(x),
                               _ptr(residual), _ptr(y), _ptr(workspace), _ptr(err_flag),
                               _stream(stream))
    _check(st, "moe_qgemv_combine")
    return y


def moe_qgemv_combine_traced(gu, dn, expert_idx, expert_w, x, residual=None, trace_ctas=256,
                             err_flag=None, stream=None):
    """moe_qgemv_combine that also returns what each CTA of its two kernels
    read and used: (y, trace uint32 [2][trace_ctas][top_k][4], ctas launched
    per phase).  Trace records: idx read, weight bits read, expert used (-1:
    skipped), weight bits used (0: skipped)."""
    gc, gs, gb = _weight(gu, "gu")
    dc, ds, db = _weight(dn, "dn")
    _cuda(expert_idx, (torch.int32,), "expert_idx")
    _cuda(expert_w, (torch.float32,), "expert_w")
    x = _cuda(x, _F16, "x")
    _cuda(residual, _F16, "residual")
    E, I2, H8 = gc.shape
    I, H = I2 // 2, H8 * 8
    top_k = expert_idx.numel()
    y = torch.empty(H, dtype=torch.float16, device=x.device)
    workspace = torch.empty(top_k * I, dtype=torch.float32, device=x.device)
    trace = torch.full((2, trace_ctas, top_k, 4), -1, dtype=torch.int32, device=x.device)
    _cuda(err_flag, (torch.int32,), "err_flag")
    launched = (_I * 2)(0, 0)
    st = lib.moe_qgemv_combine_traced(_ptr(gc), _ptr(gs), _ptr(gb), _ptr(dc), _ptr(ds), _ptr(db),
                                      E, H, I, _ptr(expert_idx), _ptr(expert_w), top_k, _ptr(x),
                                      _ptr(residual), _ptr(y), _ptr(workspace), _ptr(err_flag),
                                      _ptr(trace), trace_ctas, launched, _stream(stream))
    _check(st, "moe_qgemv_combine_traced")
    return y, trace, (int(launched[0]), int(launched[1]))


def moe_qgemv_combine_noalloc(gu, dn, expert_idx, expert_w, x, residual=None, y=None,
                              err_flag=None, stream=None):
    """moe_qgemv_combine without a workspace: the library's fixed scratch array
    stands in for it (see include/qgemv.h for its size limit and sharing)."""
    gc, gs, gb = _weight(gu, "gu")
    dc, ds, db = _weight(dn, "dn")
    _cuda(expert_idx, (torch.int32,), "expert_idx")
    _cuda(expert_w, (torch.float32,), "expert_w")
    x = _cuda(x, _F16, "x")
    _cuda(residual, _F16, "residual")
    E, I2, H8 = gc.shape
    I, H = I2 // 2, H8 * 8
    if y is None:
        y = torch.empty(H, dtype=torch.float16, device=x.device)
    _cuda(err_flag, (torch.int32,), "err_flag")
    st = lib.moe_qgemv_combine_noalloc(_ptr(gc), _ptr(gs), _ptr(gb), _ptr(dc), _ptr(ds),
                                       _ptr(db), E, H, I, _ptr(expert_idx), _ptr(expert_w),
                                       expert_idx.numel(), _ptr(x), _ptr(residual), _ptr(y),
                                       _ptr(err_flag), _stream(stream))
    _check(st, "moe_qgemv_combine_noalloc")
    return y


def noalloc_max_scratch_bytes() -> int:
    return int(lib.qgemv_noalloc_max_scratch())


def decode_attention_seq1(qkv, n_q, n_kv, head_dim, out=None, stream=None):
    qkv = _cuda(qkv, _F16, "qkv")
    if out is None:
        out = torch.empty(n_q * head_dim, dtype=torch.float16, device=qkv.device)
    st = lib.decode_attention_seq1(_ptr(qkv), _ptr(out), int(n_q), int(n_kv), int(head_dim),
                                   _stream(stream))
    _check(st, "decode_attention_seq1")
    return out


_LAYER_FIELDS = ["qkv_codes", "qkv_scales", "qkv_biases", "attn_norm", "o_codes", "o_scales",
                 "o_biases", "mlp_norm", "gate_codes", "gate_scales", "gate_biases", "up_codes",
                 "up_scales", "up_biases", "down_codes", "down_scales", "down_biases"]


class StackLayer(ctypes.Structure):
    """qgemv_stack_layer: device pointers of one layer."""
    _fields_ = [(f, ctypes.c_void_p) for f in _LAYER_FIELDS]


class StackShape(ctypes.Structure):
    """qgemv_stack_shape."""
    _fields_ = [("hidden", _I), ("n_q", _I), ("n_kv", _I), ("head_dim", _I), ("inter", _I),
                ("n_layers", _I), ("eps", _F)]


def stack_shape(hidden, n_q, n_kv, head_dim, inter, n_layers, eps=1e-5) -> StackShape:
    return StackShape(hidden, n_q, n_kv, head_dim, inter, n_layers, eps)


def decode_stack_workspace_bytes(shape: StackShape) -> int:
    return int(lib.qgemv_decode_stack_workspace_bytes(ctypes.byref(shape)))


def stack_layers(layers):
    """Descriptors for a list of layers, each a dict with weight triples
    'qkv', 'o', 'gate', 'up', 'down' and fp16 vectors 'attn_norm',
    'mlp_norm' (CUDA tensors)."""
    arr = (StackLayer * len(layers))()
    for i, L in enumerate(layers):
        d = arr[i]
        for name in ("qkv", "o", "gate", "up", "down"):
            c, sc, b = _weight(L[name], name)
            setattr(d, name + "_codes", c.data_ptr())
            setattr(d, name + "_scales", sc.data_ptr())
            setattr(d, name + "_biases", b.data_ptr())
        d.attn_norm = _cuda(L["attn_norm"], _F16, "attn_norm").data_ptr()
        d.mlp_norm = _cuda(L["mlp_norm"], _F16, "mlp_norm").data_ptr()
    return arr


def decode_stack(layers, shape: StackShape, x, y=None, workspace=None, stream=None):
    """One token through the layer stack in one call (qgemv_decode_stack).
    `layers` is a list of layer dicts or a prebuilt stack_layers() array."""
    arr = layers if isinstance(layers, ctypes.Array) else stack_layers(layers)
    x = _cuda(x, _F16, "x")
    if y is None:
        y = torch.empty(shape.hidden, dtype=torch.float16, device=x.device)
    nbytes = decode_stack_workspace_bytes(shape)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    st = lib.qgemv_decode_stack(arr, ctypes.byref(shape), _ptr(x), _ptr(y), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "qgemv_decode_stack")
    return y


class KVCacheStruct(ctypes.Structure):
    """qgemv_kv_cache (include/qgemv.h)."""
    _fields_ = ([(n, _P) for n in ("k", "v", "page_table", "kv_len")] +
                [(n, _I) for n in ("n_pages", "page_size", "n_kv", "head_dim", "n_seqs",
                                   "max_pages")])


class KVCache:
    """Handle of a paged key/value cache (kv_cache()); it keeps its tensors alive."""

    def __init__(self, k, v, page_table, kv_len):
        self.k, self.v = _cuda(k, _F16, "k"), _cuda(v, _F16, "v")
        self.page_table = _cuda(page_table, (_I32,), "page_table")
        self.kv_len = _cuda(kv_len, (_I32,), "kv_len")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must both be [n_pages][n_kv][page_size][head_dim]")
        if page_table.dim() != 2 or kv_len.shape != page_table.shape[:1]:
            raise ValueError("page_table must be [n_seqs][max_pages] and kv_len [n_seqs]")
        self.device, self.index = k.device, k.get_device()
        for name, t in (("v", v), ("page_table", page_table), ("kv_len", kv_len)):
            if t.device != self.device:
                raise ValueError(f"{name} is on {t.device}, k on {self.device}")
        n_pages, self.n_kv, self.page_size, self.head_dim = k.shape
        self.n_seqs, self.max_pages = page_table.shape
        self.capacity = self.max_pages * self.page_size
        self.starts = (self.n_seqs + 1,)                       # shape of q_start
        self.entries = (self.n_seqs, self.n_kv, self.capacity)  # shape of mass and entry_pos
        self.scale = self.head_dim ** -0.5
        self.workspace_sizes = {}
        self.struct = KVCacheStruct(k.data_ptr(), v.data_ptr(), page_table.data_ptr(),
                                    kv_len.data_ptr(), n_pages, self.page_size, self.n_kv,
                                    self.head_dim, self.n_seqs, self.max_pages)
        self.ref = ctypes.byref(self.struct)


def kv_cache(k, v, page_table, kv_len) -> KVCache:
    """Handle of a paged cache: k, v fp16 [n_pages][n_kv][page_size][head_dim],
    page_table int32 [n_seqs][max_pages], kv_len int32 [n_seqs] (entries of
    each sequence, the new tokens of a call included; read when the kernels
    run), all on one GPU."""
    return KVCache(k, v, page_table, kv_len)


# The current device, and a device's current stream, without making objects.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(call, cache, stream, *args):
    """A call for another stream or device than the current ones: again with
    them current, so that its kernels run there and what it allocates belongs
    to the stream they run on."""
    if stream is None:
        with torch.cuda.device(cache.index):
            return call(cache, *args)
    if stream.device != cache.device:
        raise ValueError(f"stream is on {stream.device}, the cache on {cache.device}")
    with torch.cuda.stream(stream):
        return call(cache, *args)


def _at(cache, t, dtype, name, shape=None):
    """Address of a contiguous tensor on the cache's device, of the given
    shape; None for None."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.get_device() != cache.index or not t.is_contiguous() or
            (shape is not None and t.shape != shape)):
        _cuda(t, (dtype,), name)
        if t.get_device() != cache.index:
            raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _token_rows(cache, t, name, rows=None, width=None):
    """fp16 rows of tokens, [tokens][width] or [tokens][heads][head_dim], whose
    row stride is free: (address, tokens, width, row stride)."""
    if t.get_device() != cache.index:
        raise ValueError(f"{name} must be a CUDA tensor on {cache.device}")
    if t.dtype is not torch.float16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.float16")
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        n, w = shape
        inner = stride[1] == 1
    elif len(shape) == 3:
        n, w = shape[0], shape[1] * shape[2]
        inner = stride[2] == 1 and (stride[1] == shape[2] or shape[1] == 1)
    else:
        inner = False
    if not inner:
        raise ValueError(f"{name} must be rows of tokens, contiguous within a row")
    if (width is not None and w != width) or (rows is not None and n != rows):
        raise ValueError(f"{name} has {n} rows of {w}, expected {rows} of {width}")
    return t.data_ptr(), n, w, stride[0] if n > 1 else w


def _heads(cache, width, extra, name):
    n = width // cache.head_dim - extra
    if width % cache.head_dim or n < 1:
        raise ValueError(f"{name} has rows of {width}, not whole heads of {cache.head_dim}")
    return n


def qk_norm_rope_append(cache, qkv, q_start, positions, inv_freq=None, interleaved=False,
                        q_norm=None, k_norm=None, eps=1e-6, q_out=None, entry_pos=None,
                        entry_mass=None, err_flag=None, stream=None):
    """qgemv_qk_norm_rope_append: per-head norms and rotation of the queries and
    keys in qkv [tokens][(n_q + 2 n_kv) head_dim], keys and values into the
    cache.  inv_freq: fp32 [rotary_dim / 2], None for no rotation.  Returns
    q_out [tokens][n_q head_dim]."""
    if stream is not None or _current_device() != cache.index:
        return _elsewhere(qk_norm_rope_append, cache, stream, qkv, q_start, positions, inv_freq,
                          interleaved, q_norm, k_norm, eps, q_out, entry_pos, entry_mass, err_flag)
    x, T, width, stride = _token_rows(cache, qkv, "qkv")
    hd = cache.head_dim
    n_q = _heads(cache, width, 2 * cache.n_kv, "qkv")
    if q_out is None:
        q_out = torch.empty(T, n_q * hd, dtype=torch.float16, device=cache.device)
    y, _, _, y_stride = _token_rows(cache, q_out, "q_out", T, n_q * hd)
    rc = lib.qgemv_qk_norm_rope_append(
        cache.ref, x, stride, T, n_q, _at(cache, q_start, _I32, "q_start", cache.starts),
        _at(cache, positions, _I32, "positions", (T,)), _at(cache, inv_freq, _F32, "inv_freq"),
        0 if inv_freq is None else 2 * inv_freq.numel(), interleaved,
        _at(cache, q_norm, _HALF, "q_norm", (hd,)), _at(cache, k_norm, _HALF, "k_norm", (hd,)), eps,
        y, y_stride, _at(cache, entry_pos, _I32, "entry_pos", cache.entries),
        _at(cache, entry_mass, _F32, "entry_mass", cache.entries),
        _at(cache, err_flag, _I32, "err_flag"), _raw_stream(cache.index))
    if rc:
        _check(rc, "qgemv_qk_norm_rope_append")
    return q_out


def paged_attention_workspace_bytes(cache, n_tokens, n_q, max_q) -> int:
    """Workspace with which paged_attention is fastest for these sizes."""
    if _current_device() != cache.index:
        return _elsewhere(paged_attention_workspace_bytes, cache, None, n_tokens, n_q, max_q)
    key = (int(n_tokens), int(n_q), int(max_q))
    n = cache.workspace_sizes.get(key)
    if n is None:
        n = int(lib.qgemv_paged_attention_workspace_bytes(cache.ref, *key))
        if len(cache.workspace_sizes) >= 1024:
            cache.workspace_sizes.clear()
        cache.workspace_sizes[key] = n
    return n


def paged_attention(cache, q, q_start, max_q=None, scale=None, out=None, want_lse=False, lse=None,
                    workspace=None, err_flag=None, stream=None):
    """qgemv_paged_attention: causal attention of each sequence's new tokens over
    its cache; q [tokens][n_q head_dim].  max_q: the largest number of new
    tokens in a sequence (default: all).  scale: default head_dim ** -0.5.
    Returns (out, lse fp32 [tokens][n_q] or None)."""
    if stream is not None or _current_device() != cache.index:
        return _elsewhere(paged_attention, cache, stream, q, q_start, max_q, scale, out, want_lse,
                          lse, workspace, err_flag)
    x, T, width, stride = _token_rows(cache, q, "q")
    n_q = _heads(cache, width, 0, "q")
    max_q = max(T, 1) if max_q is None else int(max_q)
    if out is None:
        out = torch.empty(T, width, dtype=torch.float16, device=cache.device)
    y, _, _, y_stride = _token_rows(cache, out, "out", T, width)
    if lse is None and want_lse:
        lse = torch.empty(T, n_q, dtype=torch.float32, device=cache.device)
    if workspace is None:
        n = paged_attention_workspace_bytes(cache, T, n_q, max_q)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=cache.device)
    else:
        if workspace.get_device() != cache.index or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the cache's device")
        n = workspace.numel() * workspace.element_size()
    rc = lib.qgemv_paged_attention(
        cache.ref, x, stride, T, n_q, _at(cache, q_start, _I32, "q_start", cache.starts), max_q,
        cache.scale if scale is None else scale, y, y_stride, _at(cache, lse, _F32, "lse", (T, n_q)),
        workspace.data_ptr() if n else None, n, _at(cache, err_flag, _I32, "err_flag"),
        _raw_stream(cache.index))
    if rc:
        _check(rc, "qgemv_paged_attention")
    return out, lse


def attention_mass(cache, q, q_start, lse, max_q=None, scale=None, mass=None, mass_out=None,
                   err_flag=None, stream=None):
    """qgemv_attention_mass: mass (fp32 [n_seqs][n_kv][capacity], None: zeros) plus
    the attention weight every cached entry receives from the new tokens; q
    and lse as paged_attention took and gave them.  Returns mass_out (a new
    array is zero behind each sequence's length; it may be mass itself)."""
    if stream is not None or _current_device() != cache.index:
        return _elsewhere(attention_mass, cache, stream, q, q_start, lse, max_q, scale, mass,
                          mass_out, err_flag)
    x, T, width, stride = _token_rows(cache, q, "q")
    n_q = _heads(cache, width, 0, "q")
    if mass_out is None:
        mass_out = torch.zeros(cache.entries, dtype=torch.float32, device=cache.device)
    rc = lib.qgemv_attention_mass(
        cache.ref, x, stride, T, n_q, _at(cache, q_start, _I32, "q_start", cache.starts),
        max(T, 1) if max_q is None else int(max_q), cache.scale if scale is None else scale,
        _at(cache, lse, _F32, "lse", (T, n_q)), _at(cache, mass, _F32, "mass", cache.entries),
        _at(cache, mass_out, _F32, "mass_out", cache.entries),
        _at(cache, err_flag, _I32, "err_flag"), _raw_stream(cache.index))
    if rc:
        _check(rc, "qgemv_attention_mass")
    return mass_out


def cache_evict(cache, mass, entry_pos, next_pos, keep, n_sink=0, n_recent=0, kept=None,
                mass_out=None, pos_out=None, kv_len_out=None, err_flag=None, stream=None):
    """qgemv_cache_evict: cut every sequence to its `keep` entries of largest mass
    (positions below n_sink and the last n_recent before next_pos first), each
    head for itself; rows of the cache move in place.  Returns (kept int32
    [n_seqs][n_kv][keep], mass_out, pos_out, kv_len_out); kv_len_out is the new
    length, to be written into the cache's kv_len before the next call."""
    if stream is not None or _current_device() != cache.index:
        return _elsewhere(cache_evict, cache, stream, mass, entry_pos, next_pos, keep, n_sink,
                          n_recent, kept, mass_out, pos_out, kv_len_out, err_flag)
    keep, S, dev = int(keep), cache.n_seqs, cache.device
    if kept is None:
        kept = torch.empty(S, cache.n_kv, max(keep, 0), dtype=torch.int32, device=dev)
    if mass_out is None:
        mass_out = torch.zeros(cache.entries, dtype=torch.float32, device=dev)
    if pos_out is None:
        pos_out = torch.zeros(cache.entries, dtype=torch.int32, device=dev)
    if kv_len_out is None:
        kv_len_out = torch.empty(S, dtype=torch.int32, device=dev)
    rc = lib.qgemv_cache_evict(
        cache.ref, _at(cache, mass, _F32, "mass", cache.entries),
        _at(cache, entry_pos, _I32, "entry_pos", cache.entries),
        _at(cache, next_pos, _I32, "next_pos", (S,)), keep, int(n_sink), int(n_recent),
        _at(cache, kept, _I32, "kept", (S, cache.n_kv, max(keep, 0))),
        _at(cache, mass_out, _F32, "mass_out", cache.entries),
        _at(cache, pos_out, _I32, "pos_out", cache.entries),
        _at(cache, kv_len_out, _I32, "kv_len_out", (S,)), _at(cache, err_flag, _I32, "err_flag"),
        _raw_stream(cache.index))
    if rc:
        _check(rc, "qgemv_cache_evict")
    return kept, mass_out, pos_out, kv_len_out


# ------------------------------------------------- microscaled (MX) operators

_U8 = torch.uint8
_E4M3 = torch.float8_e4m3fn
_CODES4, _CODES8, _BYTES = _CODES, (_U8, _E4M3), (_U8,)


class _NoCalls:
    """In place of a module that is not there: what needs it says so, all else works."""

    def __init__(self, path):
        self._path = path

    def __getattr__(self, name):
        raise ImportError(f"{self._path} not found: the microscaled operators need it "
                          "(build.py makes it, with a C compiler and Python's headers)")


def _load_calls():
    """The module that looks at a call's tensors and makes the call (csrc/mx_calls.c)."""
    path = _build.CALLS
    if not os.path.exists(path):
        return _NoCalls(path)
    loader = importlib.machinery.ExtensionFileLoader("_mx_calls", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_mx_calls", loader))
    loader.exec_module(module)
    names = ("qgemv_mx_quantize", "qgemv_mx_dequantize", "qgemv_residual_rmsnorm_mxfp8",
             "qgemv_mxfp4", "qgemv_mx_gemm", "qgemv_mx_swiglu")
    module.bind(*[ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names],
                _HALF, _U8, _E4M3, _I32, _CODES4[1], _current_device, _raw_stream)
    return module


_calls = _load_calls()


def _mx_elsewhere(call, t, stream, *args):
    """A call for another stream or device than the current ones: again with them
    current, so that what it allocates belongs to the stream it runs on."""
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    if stream is None:
        with torch.cuda.device(t.get_device()):
            return call(*args)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.stream(stream):
        return call(*args)


def _mx_unfit(call, args, what, **tensors):
    """What to do where _calls found that something does not fit: the call on its tensors'
    device, or the error.  tensors: name = (tensor, types, shape), the first one's device is
    the call's."""
    t = next(iter(tensors.values()))[0]
    if t.is_cuda and _current_device() != t.get_device():
        return _mx_elsewhere(call, t, None, *args)
    for name, (t, dtypes, shape) in tensors.items():
        if t is None:
            continue
        _cuda(t, dtypes, name)
        if t.get_device() != _current_device():
            raise ValueError(f"{name} is on {t.device}, not on cuda:{_current_device()}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise QgemvError(-1, what)  # sizes that the library refuses


def _mx_lead(t, name):
    """All sizes of a tensor but the last, and the last."""
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one axis")
    return t.shape[:-1], t.shape[-1]


def _mx_weight(w, name):
    """{name: (tensor, types, shape)} of an MXFP4 weight, for _mx_unfit."""
    codes, scales = w
    if codes.dim() != 2:
        raise ValueError(f"{name}.codes must be [rows][k / 8]")
    n, words = codes.shape
    return {name + ".codes": (codes, _CODES4, codes.shape),
            name + ".scales": (scales, _BYTES, (n, words // 4))}


def _mx_rows(x, k):
    """The same of MXFP8 rows of k columns."""
    lead, _ = _mx_lead(x[0], "x.codes")
    return {"x.codes": (x[0], _CODES8, (*lead, k)), "x.scales": (x[1], _BYTES, (*lead, k // 32))}


def mx_quantize(x, bits=8, codes=None, scales=None, stream=None):
    """qgemv_mx_quantize: fp16 rows [..., k] in microscaled form, blocks of 32 along
    k (k a multiple of 32).  bits 4: MXFP4, codes int32 [..., k / 8]; bits 8: MXFP8,
    codes uint8 [..., k] (e4m3; a float8_e4m3fn tensor may be given).  Returns
    (codes, scales uint8 [..., k / 32])."""
    if stream is not None:
        return _mx_elsewhere(mx_quantize, x, stream, x, bits, codes, scales)
    if codes is None or scales is None:
        lead, k = _mx_lead(x, "x")
        if codes is None:
            codes = torch.empty((*lead, k if bits == 8 else k // 8),
                                dtype=_U8 if bits == 8 else _I32, device=x.device)
        if scales is None:
            scales = torch.empty((*lead, k // 32), dtype=_U8, device=x.device)
    rc = _calls.quantize(x, bits, codes, scales)
    if rc == 0:
        return codes, scales
    if rc is None:
        if bits not in (4, 8):
            raise ValueError(f"bits must be 4 or 8, not {bits}")
        lead, k = _mx_lead(x, "x")
        kind, per = (_CODES8, 1) if bits == 8 else (_CODES4, 8)
        return _mx_unfit(mx_quantize, (x, bits, codes, scales), "qgemv_mx_quantize",
                         x=(x, _F16, x.shape), codes=(codes, kind, (*lead, k // per)),
                         scales=(scales, _BYTES, (*lead, k // 32)))
    _check(rc, "qgemv_mx_quantize")


def mx_dequantize(codes, scales, out=None, stream=None):
    """qgemv_mx_dequantize: the fp16 values [..., k] of MXFP4 (int32 codes) or MXFP8
    (uint8 or float8_e4m3fn codes) rows."""
    if stream is not None:
        return _mx_elsewhere(mx_dequantize, codes, stream, codes, scales, out)
    if out is None:
        lead, k = _mx_lead(codes, "codes")
        out = torch.empty((*lead, 8 * k if codes.dtype in _CODES4 else k), dtype=_HALF,
                          device=codes.device)
    rc = _calls.dequantize(codes, scales, out)
    if rc == 0:
        return out
    if rc is None:
        lead, k = _mx_lead(codes, "codes")
        k = 8 * k if codes.dtype in _CODES4 else k
        return _mx_unfit(mx_dequantize, (codes, scales, out), "qgemv_mx_dequantize",
                         codes=(codes, _CODES4 + _CODES8, codes.shape),
                         scales=(scales, _BYTES, (*lead, k // 32)), out=(out, _F16, (*lead, k)))
    _check(rc, "qgemv_mx_dequantize")


def residual_rmsnorm_mxfp8(x, gamma, residual=None, eps=1e-5, h=None, codes=None, scales=None,
                           stream=None):
    """qgemv_residual_rmsnorm_mxfp8: h = x + residual (fp16 rows [..., k]; x itself
    when residual is None), RMSNorm(h) * gamma as MXFP8.  h may be x or residual.
    Returns (h, codes uint8 [..., k], scales uint8 [..., k / 32])."""
    if stream is not None:
        return _mx_elsewhere(residual_rmsnorm_mxfp8, x, stream, x, gamma, residual, eps, h, codes,
                             scales)
    if residual is None:
        h = x
    elif h is None:
        h = torch.empty_like(x)
    if codes is None:
        codes = torch.empty(x.shape, dtype=_U8, device=x.device)
    if scales is None:
        lead, k = _mx_lead(x, "x")
        scales = torch.empty((*lead, k // 32), dtype=_U8, device=x.device)
    rc = _calls.norm(x, gamma, residual, eps, h, codes, scales)
    if rc == 0:
        return h, codes, scales
    if rc is None:
        lead, k = _mx_lead(x, "x")
        return _mx_unfit(residual_rmsnorm_mxfp8, (x, gamma, residual, float(eps), h, codes, scales),
                         "qgemv_residual_rmsnorm_mxfp8", x=(x, _F16, x.shape),
                         gamma=(gamma, _F16, (k,)), residual=(residual, _F16, x.shape),
                         h=(h, _F16, x.shape), codes=(codes, _CODES8, x.shape),
                         scales=(scales, _BYTES, (*lead, k // 32)))
    _check(rc, "qgemv_residual_rmsnorm_mxfp8")


def qgemv_mxfp4(w, x, y=None, residual=None, stream=None):
    """y = W x (+ residual) for an MXFP4 weight w = (codes int32 [n][k / 8], scales
    uint8 [n][k / 32]) and one to eight fp16 rows x ([k] or [m][k]).  x counts exactly,
    but for the last bit of values below 2^-13 in blocks of 32 with one of 32768 or more."""
    if stream is not None:
        return _mx_elsewhere(qgemv_mxfp4, x, stream, w, x, y, residual)
    codes, scales = w
    if y is None:
        lead, _ = _mx_lead(x, "x")
        y = torch.empty((*lead, codes.shape[0]), dtype=_HALF, device=x.device)
    rc = _calls.matvec(codes, scales, x, y, residual)
    if rc == 0:
        return y
    if rc is None:
        tensors = _mx_weight(w, "w")
        (lead, _), n, k = _mx_lead(x, "x"), codes.shape[0], 8 * codes.shape[1]
        return _mx_unfit(qgemv_mxfp4, (w, x, y, residual), "qgemv_mxfp4", x=(x, _F16, (*lead, k)),
                         **tensors, y=(y, _F16, (*lead, n)), residual=(residual, _F16, (*lead, n)))
    _check(rc, "qgemv_mxfp4")


def mx_gemm(w, x, y=None, residual=None, stream=None):
    """qgemv_mx_gemm: y = W x (+ residual, which may be y) for an MXFP4 weight w =
    (codes int32 [n][k / 8], scales uint8 [n][k / 32]) and any number of MXFP8 rows
    x = (codes uint8 [..., k], scales uint8 [..., k / 32]).  Returns y fp16 [..., n]."""
    codes, scales = w
    xc, xs = x
    if stream is not None:
        return _mx_elsewhere(mx_gemm, xc, stream, w, x, y, residual)
    if y is None:
        lead, _ = _mx_lead(xc, "x.codes")
        y = torch.empty((*lead, codes.shape[0]), dtype=_HALF, device=xc.device)
    rc = _calls.gemm(codes, scales, xc, xs, y, residual)
    if rc == 0:
        return y
    if rc is None:
        tensors = _mx_weight(w, "w")
        (lead, _), n, k = _mx_lead(xc, "x.codes"), codes.shape[0], 8 * codes.shape[1]
        return _mx_unfit(mx_gemm, (w, x, y, residual), "qgemv_mx_gemm", **_mx_rows(x, k), **tensors,
                         y=(y, _F16, (*lead, n)), residual=(residual, _F16, (*lead, n)))
    _check(rc, "qgemv_mx_gemm")


def mx_swiglu(gate, up, x, h=None, codes=None, scales=None, stream=None):
    """qgemv_mx_swiglu: silu(Wg x) * (Wu x) for MXFP4 weights gate, up (each (codes,
    scales), [n][k]) and MXFP8 rows x = (codes, scales).  With h (fp16 [..., n]) alone the
    result goes there and h is returned; else it leaves as MXFP8, what mx_gemm takes:
    returns (codes uint8 [..., n], scales uint8 [..., n / 32]) (and fills h where given)."""
    gc, gs = gate
    uc, us = up
    xc, xs = x
    if stream is not None:
        return _mx_elsewhere(mx_swiglu, xc, stream, gate, up, x, h, codes, scales)
    held = h is None or codes is not None or scales is not None
    if held and (codes is None or scales is None):
        lead, _ = _mx_lead(xc, "x.codes")
        if codes is None:
            codes = torch.empty((*lead, gc.shape[0]), dtype=_U8, device=xc.device)
        if scales is None:
            scales = torch.empty((*lead, gc.shape[0] // 32), dtype=_U8, device=xc.device)
    rc = _calls.gated(gc, gs, uc, us, xc, xs, h, codes, scales)
    if rc == 0:
        return (codes, scales) if held else h
    if rc is None:
        tensors = _mx_weight(gate, "gate")
        (lead, _), n, k = _mx_lead(xc, "x.codes"), gc.shape[0], 8 * gc.shape[1]
        if uc.shape != gc.shape:
            raise ValueError(f"up.codes has shape {tuple(uc.shape)}, gate.codes {tuple(gc.shape)}")
        return _mx_unfit(mx_swiglu, (gate, up, x, h, codes, scales), "qgemv_mx_swiglu",
                         **_mx_rows(x, k), **tensors, **_mx_weight(up, "up"),
                         h=(h, _F16, (*lead, n)), codes=(codes, _CODES8, (*lead, n)),
                         scales=(scales, _BYTES, (*lead, n // 32)))
    _check(rc, "qgemv_mx_swiglu")


def device_status() -> int:
    """Read and clear the device-side status word (synchronises the device)."""
    flags = ctypes.c_uint(0)
    _check(lib.qgemv_device_status(ctypes.byref(flags)), "qgemv_device_status")
    return int(flags.value)


def selftest_wait_timeout(limit_us: int = 2000, stream=None) -> None:
    """Enqueue the bounded-wait self-test (qgemv_selftest_wait_timeout): a
    wait that nothing satisfies gives up after limit_us and sets bit 0 of
    the device status word."""
    _check(lib.qgemv_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "qgemv_selftest_wait_timeout")


def last_cuda_error() -> int:
    return int(lib.qgemv_last_cuda_error())


def version() -> int:
    return int(lib.qgemv_version())
