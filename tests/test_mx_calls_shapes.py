"""The module that makes the calls of the microscaled operators (csrc/mx_calls.c), without a
GPU: scales of another layout than their rows', with as many of them, do not reach the library."""
import subprocess
import sys
import textwrap


def test_scales_of_another_shape():
    # (in a process of its own: the module is bound once, to the library)
    code = textwrap.dedent("""
        import ctypes, importlib.machinery, importlib.util, math
        import torch
        from bit_group_quantized_qgemv_gb300 import _binding as b
        loader = importlib.machinery.ExtensionFileLoader("_mx_calls", b._build.CALLS)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_mx_calls", loader))
        loader.exec_module(m)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        types = [(I, P, I, I, P, P, P), (I, P, P, I, I, P, P), (P, P, P, F, I, I, P, P, P, P),
                 (P, P, P, P, I, I, I, P, P), (P, P, P, P, P, I, I, I, P, P), (P, P, P, P, P, P, I, I, I, P, P, P, P)]
        kept = [ctypes.CFUNCTYPE(I, *ts)(lambda *args: 7) for ts in types]
        m.bind(*[ctypes.cast(c, P).value for c in kept], torch.float16, torch.uint8, torch.float8_e4m3fn, torch.int32,
               torch.uint32, lambda: 0, lambda index: 0)

        class T:                                         # a contiguous tensor on GPU 0
            def __init__(self, dtype, *shape): self.dtype, self.shape = dtype, shape
            def get_device(self): return 0
            def is_contiguous(self): return True
            def numel(self): return math.prod(self.shape)
            def size(self, i): return self.shape[i]
            def data_ptr(self): return 0x1000
        H, U, W = torch.float16, torch.uint8, torch.int32
        x, c8, c4, s, st = T(H, 5, 96), T(U, 5, 96), T(W, 5, 12), T(U, 5, 3), T(U, 3, 5)
        wc, ws, wt, y = T(W, 64, 12), T(U, 64, 3), T(U, 3, 64), T(H, 5, 64)
        hc, hs, ht = T(U, 5, 64), T(U, 5, 2), T(U, 2, 5)
        flat = [T(U, 15), T(U, 192), T(U, 10)]
        calls = {
            "quantize 8": lambda s=s: m.quantize(x, 8, c8, s), "quantize 4": lambda s=s: m.quantize(x, 4, c4, s),
            "dequantize 8": lambda s=s: m.dequantize(c8, s, x), "dequantize 4": lambda s=s: m.dequantize(c4, s, x),
            "norm": lambda s=s: m.norm(x, T(H, 96), None, 0.5, x, c8, s), "rows": lambda s=s: m.gemm(wc, ws, c8, s, y, None),
            "gated rows": lambda s=s: m.gated(wc, ws, wc, ws, c8, s, y, None, None)}
        for name, call in calls.items():
            assert call() == 7 and call(T(U, 5, 1, 3)) == 7 and call(T(U, 1, 5, 3)) == 7, name
            assert call(st) is None and call(T(U, 15)) is None and call(T(U, 5, 3, 1)) is None, name
        calls = {
            "matvec": lambda s=ws, c=wc: m.matvec(c, s, x, y, None), "gemm": lambda s=ws, c=wc: m.gemm(c, s, c8, T(U, 5, 3), y, None),
            "gate": lambda s=ws, c=wc: m.gated(c, s, wc, ws, c8, T(U, 5, 3), y, None, None),
            "up": lambda s=ws, c=wc: m.gated(wc, ws, c, s, c8, T(U, 5, 3), y, None, None)}
        for name, call in calls.items():
            assert call() == 7, name
            assert call(wt) is None and call(T(U, 192)) is None and call(T(U, 64, 3, 1)) is None, name
            # a stack of weights is not one weight
            assert call(T(U, 4, 16, 3), T(W, 4, 16, 12)) is None and call(ws, T(W, 4, 16, 12)) is None, name
            assert call(T(U, 24), T(W, 768)) is None, name
        gated = lambda s: m.gated(wc, ws, wc, ws, c8, T(U, 5, 3), None, hc, s)
        assert gated(hs) == 7 and gated(ht) is None and gated(T(U, 10)) is None
        print("done")
    """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stderr[-2000:]
