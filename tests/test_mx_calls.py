"""The module that makes the calls of the microscaled operators (csrc/mx_calls.c), without a
GPU: stand-ins for tensors and for the C functions, what reaches these, and what does not."""
import subprocess
import sys
import textwrap


def test_calls():
    # (in a process of its own: the module is bound once, to the library)
    code = textwrap.dedent("""
        import ctypes, importlib.machinery, importlib.util
        import bit_group_quantized_qgemv_gb300 as q
        from bit_group_quantized_qgemv_gb300 import _binding as b
        import torch
        loader = importlib.machinery.ExtensionFileLoader("_mx_calls", b._build.CALLS)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_mx_calls", loader))
        loader.exec_module(m)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        types = [(I, P, I, I, P, P, P), (I, P, P, I, I, P, P), (P, P, P, F, I, I, P, P, P, P),
                 (P, P, P, P, I, I, I, P, P), (P, P, P, P, P, I, I, I, P, P), (P, P, P, P, P, P, I, I, I, P, P, P, P)]
        seen, kept = [], []
        def function(ts):
            def f(*args):
                seen.append(args)
                return 7
            c = ctypes.CFUNCTYPE(I, *ts)(f)
            kept.append(c)
            return ctypes.cast(c, P).value
        m.bind(*[function(t) for t in types], torch.float16, torch.uint8, torch.float8_e4m3fn, torch.int32, torch.uint32,
               lambda: 1, lambda index: 0x500 + index)

        class T:                                         # a tensor on GPU 1
            at = 0x1000
            def __init__(self, dtype, *shape, device=1, contiguous=True):
                self.dtype, self.shape, self.index, self.ok = dtype, shape, device, contiguous
                T.at += 0x1000
                self.p = T.at
            def get_device(self): return self.index
            def is_contiguous(self): return self.ok
            def numel(self):
                n = 1
                for s in self.shape: n *= s
                return n
            def size(self, i): return self.shape[i]
            def data_ptr(self): return self.p
        H, U, W, E = torch.float16, torch.uint8, torch.int32, torch.float8_e4m3fn
        def got(r, *want):
            assert r == 7 and seen[-1] == want, (r, seen[-1], want)
            seen.clear()
        def none(r):
            assert r is None and not seen, (r, seen)
        x, c8, c4, s = T(H, 3, 5, 96), T(U, 3, 5, 96), T(W, 3, 5, 12), T(U, 3, 5, 3)
        got(m.quantize(x, 8, c8, s), 8, x.p, 15, 96, c8.p, s.p, 0x501)
        got(m.quantize(x, 4, c4, s), 4, x.p, 15, 96, c4.p, s.p, 0x501)
        got(m.quantize(x, 8, T(E, 3, 5, 96), s), 8, x.p, 15, 96, T.at, s.p, 0x501)
        got(m.dequantize(c8, s, x), 8, c8.p, s.p, 15, 96, x.p, 0x501)
        got(m.dequantize(c4, s, x), 4, c4.p, s.p, 15, 96, x.p, 0x501)
        empty = T(H, 0, 96)
        got(m.quantize(empty, 8, T(U, 0, 96), T(U, 0, 3)), 8, empty.p, 0, 96, T.at - 0x1000, T.at, 0x501)
        for bad in (m.quantize(x, 4, c8, s), m.quantize(x, 8, c4, s), m.quantize(x, 5, c8, s), m.quantize(c8, 8, c8, s),
                    m.quantize(x, 8, c8, T(U, 3, 5, 2)), m.quantize(x, 8, T(U, 3, 5, 96, device=0), s),
                    m.quantize(x, 8, T(U, 3, 5, 96, contiguous=False), s), m.quantize(T(H, 3, 5, 96, device=0), 8, c8, s),
                    m.quantize(T(H, 3, 5, 96, device=-1), 8, c8, s), m.quantize(x, 8, T(U, 5, 3, 12, 8), s),
                    m.quantize(T(H, 2, 48), 8, T(U, 2, 48), T(U, 3)), m.quantize(None, 8, c8, s), m.quantize(x, "8", c8, s),
                    m.quantize(x, 8, 3, s), m.quantize(T(H, 2 ** 27, 64), 8, T(U, 2 ** 27, 64), T(U, 2 ** 27, 3)),
                    m.quantize(T(H, 2 ** 31, 32), 8, T(U, 2 ** 31, 32), T(U, 2 ** 31, 1)), m.quantize(x, 8),
                    m.dequantize(c8, s, T(H, 3, 5, 64)), m.dequantize(x, s, x), m.dequantize(c4, s, T(H, 5, 3, 96, device=0))):
            none(bad)
        g, r, h = T(H, 96), T(H, 3, 5, 96), T(H, 3, 5, 96)
        got(m.norm(x, g, r, 0.5, h, c8, s), x.p, r.p, g.p, 0.5, 15, 96, h.p, c8.p, s.p, 0x501)
        got(m.norm(x, g, None, 0.25, x, c8, s), x.p, None, g.p, 0.25, 15, 96, None, c8.p, s.p, 0x501)
        for bad in (m.norm(x, T(H, 64), r, 0.5, h, c8, s), m.norm(x, g, r, 0.5, None, c8, s), m.norm(x, g, r, "e", h, c8, s),
                    m.norm(x, g, T(H, 15, 96, device=0), 0.5, h, c8, s), m.norm(x, g, r, 0.5, c8, c8, s)):
            none(bad)
        wc, ws, y, x2 = T(W, 7, 12), T(U, 7, 3), T(H, 2, 7), T(H, 2, 96)
        got(m.matvec(wc, ws, x2, y, None), wc.p, ws.p, x2.p, y.p, 2, 7, 96, None, 0x501)
        got(m.matvec(wc, ws, x2, y, y), wc.p, ws.p, x2.p, y.p, 2, 7, 96, y.p, 0x501)
        y15 = T(H, 3, 5, 7)
        got(m.gemm(wc, ws, c8, s, y15, y15), wc.p, ws.p, c8.p, s.p, y15.p, 15, 7, 96, y15.p, 0x501)
        for bad in (m.matvec(wc, ws, T(H, 2, 64), y, None), m.matvec(wc, ws, x2, T(H, 7, 2), None), m.matvec(wc, T(U, 7, 2), x2, y, None),
                    m.matvec(T(torch.int64, 7, 12), ws, x2, y, None), m.matvec(wc, ws, x2, y, T(H, 7)),
                    m.gemm(wc, ws, c8, T(U, 15), y15, None), m.gemm(wc, ws, x, s, y15, None), m.gemm(T(W, 7, 13), ws, c8, s, y15, None)):
            none(bad)
        uc, us = T(W, 64, 12), T(U, 64, 3)
        gc, gs = T(torch.uint32, 64, 12), T(U, 64, 3)
        hh, hc, hs = T(H, 3, 5, 64), T(U, 3, 5, 64), T(U, 3, 5, 2)
        got(m.gated(gc, gs, uc, us, c8, s, hh, hc, hs), gc.p, gs.p, uc.p, us.p, c8.p, s.p, 15, 64, 96, hh.p, hc.p, hs.p, 0x501)
        got(m.gated(gc, gs, uc, us, c8, s, hh, None, None), gc.p, gs.p, uc.p, us.p, c8.p, s.p, 15, 64, 96, hh.p, None, None, 0x501)
        got(m.gated(gc, gs, uc, us, c8, s, None, hc, hs), gc.p, gs.p, uc.p, us.p, c8.p, s.p, 15, 64, 96, None, hc.p, hs.p, 0x501)
        for bad in (m.gated(gc, gs, T(W, 32, 12), us, c8, s, hh, hc, hs), m.gated(gc, gs, uc, us, c8, s, hh, hc, None),
                    m.gated(gc, gs, uc, us, c8, s, hc, hc, hs), m.gated(wc, ws, wc, ws, c8, s, None, T(U, 3, 5, 7), T(U, 0))):
            none(bad)
        print("done")
    """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stderr[-2000:]
