"""Cases of the microscaled (MX) operators: what they compute, on which sizes.

Weights are MXFP4, activations MXFP8 or fp16: blocks of 32 values along k share a
scale 2^(byte - 127), a value is its code times that.  Codes of 4 bits are e2m1
(0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign; eight to an int32, the lowest four bits
first), codes of 8 bits e4m3 (up to 448).  Five operators, the gated block of a layer:

* ``quantize``  fp16 rows to MXFP4 or MXFP8 and back (``mx_quantize``, ``mx_dequantize``);
* ``norm``      residual addition, RMS norm, the result in MXFP8 (``residual_rmsnorm_mxfp8``);
* ``matvec``    MXFP4 weights times one to eight fp16 rows (``qgemv_mxfp4``);
* ``product``   MXFP4 weights times any number of MXFP8 rows (``mx_gemm``);
* ``gated``     silu(gate) * up of MXFP8 rows, out as MXFP8 or fp16 (``mx_swiglu``).

What is held in 8 bits is returned as the values it stands for.
"""
import math

import torch

own = False

EPS = 1.0e-5
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # One token's activations on their way into a product: nothing but latency.
        dict(name="quantize_row", op="quantize", bits=8, m=1, k=4096),
        # A weight matrix as it is loaded: the gate projection of the 8B shape.
        dict(name="quantize_weight", op="quantize", bits=4, m=14336, k=4096),
        # The norm in front of a decode step's products.
        dict(name="norm_one", op="norm", m=1, k=4096, res=True),
        # The same for a prompt.
        dict(name="norm_prompt", op="norm", m=2048, k=4096, res=True),
        # Batch-1 decoding: the output projection of the 8B shape.
        dict(name="matvec_one", op="matvec", m=1, n=4096, k=4096, res=True),
        # The vocabulary projection of the 0.6B shape.
        dict(name="matvec_head", op="matvec", m=1, n=151936, k=1024, res=False),
        # Five drafted tokens through a down projection.
        dict(name="matvec_down", op="matvec", m=5, n=4096, k=14336, res=True),
        # A decode step of 48 sequences: the fused QKV projection.
        dict(name="product_batch", op="product", m=48, n=6144, k=4096, res=False),
        # Sizes that fit no tile.
        dict(name="product_odd", op="product", m=777, n=1003, k=1120, res=True),
        # A long prompt through a down projection.
        dict(name="product_prompt", op="product", m=4096, n=4096, k=14336, res=True),
        # A decode step of 16 sequences through gate and up, on to the down projection.
        dict(name="gated_step", op="gated", m=16, n=14336, k=4096, out8=True),
        # A prompt through gate and up.
        dict(name="gated_prompt", op="gated", m=2048, n=14336, k=4096, out8=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "norm", "matvec", "matvec", "product", "product", "gated", "gated"])
    k = 32 * (log(1, 512) if rng.random() < 0.5 else 4 * log(1, 128))
    if op in ("quantize", "norm"):
        m = log(1, max(1, 40000000 // k) if rng.random() < 0.5 else 200)
        return dict(op="quantize", bits=rng.choice([4, 8]), m=m, k=k) if op == "quantize" else dict(op="norm", m=m, k=k, res=rng.random() < 0.7)
    if op == "matvec":
        return dict(op="matvec", m=rng.randint(1, 8), n=log(1, min(160000, 150000000 // k)), k=k, res=rng.random() < 0.5)
    n = log(1, min(30000, 60000000 // k))
    if op == "gated" and rng.random() < 0.7:
        n = (n + 31) // 32 * 32
    m = log(1, 64) if rng.random() < 0.4 else log(16, max(17, min(4096, 100000000000 // (n * k))))
    if op == "product":
        return dict(op="product", m=m, n=n, k=k, res=rng.random() < 0.5)
    return dict(op="gated", m=m, n=n, k=k, out8=n % 32 == 0 and rng.random() < 0.7)


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":
        return {"bytes": m * k * (4 + 2 * (case["bits"] / 8 + 1 / 32)), "flops": 2 * m * k}
    if op == "norm":
        return {"bytes": m * k * ((4 if case["res"] else 2) + 2 * case["res"] + 2 * 33 / 32 + 2) + 2 * k, "flops": 6 * m * k}
    n = case["n"]
    if op == "gated":
        return {"bytes": 2 * n * k * 17 / 32 + m * k * 33 / 32 + m * n * (2 * 33 / 32 + 2 if case["out8"] else 2), "flops": 4 * m * n * k}
    return {"bytes": n * k * 17 / 32 + m * k * (33 / 32 if op == "product" else 2) + m * n * (4 if case["res"] else 2), "flops": 2 * m * n * k}


# ------------------------------------------------------ formats, 32 bits


def _power(e):
    """2^e as fp32 from its bits, -127 <= e <= 127."""
    return torch.where(e > -127, (e.int() + 127) << 23, torch.full_like(e.int(), 1 << 22)).view(torch.float32)


def _blocks(x, bits):
    """fp32 rows [m][k] in blocks of 32, and the exponents of their scales."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    # floor(log2): the exponent of a float is exact, a logarithm is not
    e = torch.where(top > 0, torch.frexp(top).exponent - 1 - (2 if bits == 4 else 8), -127)
    return b, torch.clamp(e, -127, 127)


def _round(v, bits):
    """Codes of values that are divided by their scale."""
    if bits == 8:
        return torch.clamp(v, -448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    a = v.abs()
    # a tie goes to the even code: above the odd steps' middles, from the even ones' on
    code = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int()
    return code + 8 * torch.signbit(v).int()


def _quantize(x, bits):
    """fp32 rows to codes (int32 [m][k / 8] or uint8 [m][k]) and scales (uint8 [m][k / 32])."""
    b, e = _blocks(x, bits)
    code = _round(b * _power(-e), bits).reshape(x.shape)
    scales = (e.squeeze(-1) + 127).to(torch.uint8)
    if bits == 8:
        return code, scales
    shift = 4 * torch.arange(8, device=x.device)
    packed = (code.view(x.shape[0], -1, 8).long() << shift).sum(-1)
    return (packed - ((packed >> 31) << 32)).int(), scales


def _values(codes, scales):
    """The fp32 values of codes and scales."""
    if codes.dtype == torch.uint8:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + [-t for t in E2M1], device=codes.device)
        shift = 4 * torch.arange(8, dtype=torch.int32, device=codes.device)
        v = table[((codes.unsqueeze(-1) >> shift) & 15).long()].flatten(-2)
    return (v.reshape(v.shape[0], -1, 32) * _power(scales.int().unsqueeze(-1) - 127)).reshape(v.shape)


# ----------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, m, k, dev = case["op"], case["m"], case["k"], "cuda"

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=dev) * scale

    def activations():
        # some channels are far larger than the others, as behind a norm
        return normal(m, k) * torch.exp(0.7 * normal(k))

    def weight(n):
        parts = [_quantize((normal(min(8192, n - i), k, scale=k ** -0.5)).half().float(), 4) for i in range(0, n, 8192)]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])

    def codes8(rows, cols):
        return torch.zeros(rows, cols, dtype=torch.uint8, device=dev), torch.zeros(rows, cols // 32, dtype=torch.uint8, device=dev)

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float16, device=dev)

    st = dict(case=case)
    if op == "quantize":
        x = normal(m, k, scale=k ** -0.5) if case["bits"] == 4 else activations()
        st.update(x=x.half(), values=zeros(m, k))
        st["held"] = codes8(m, k) if case["bits"] == 8 else (torch.zeros(m, k // 8, dtype=torch.int32, device=dev), torch.zeros(m, k // 32, dtype=torch.uint8, device=dev))
    elif op == "norm":
        st.update(x=activations().half(), res=(normal(m, k) * 2).half() if case["res"] else None, gamma=(1 + normal(k, scale=0.1)).half(),
                  h=zeros(m, k), held=codes8(m, k), values=zeros(m, k))
    else:
        n = case["n"]
        st["w"] = weight(n)
        x = activations()
        st["x"] = x.half() if op == "matvec" else _quantize(x, 8)
        st["y"] = zeros(m, n)
        if op == "gated":
            st["up"] = weight(n)
            st["held"] = codes8(m, n) if case["out8"] else None
        else:
            st["res"] = normal(m, n).half() if case["res"] else None
    return st


# ------------------------------------------------------------- plain form


def _plain(st):
    c = st["case"]
    if c["op"] == "quantize":
        codes, scales = _quantize(st["x"].float(), c["bits"])
        return [_values(codes, scales).half()]
    if c["op"] == "norm":
        h = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).half()
        f = h.float()
        n = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * st["gamma"].float()
        return [h, _values(*_quantize(n, 8)).half()]
    x = st["x"].float() if c["op"] == "matvec" else _values(*st["x"])
    y = torch.matmul(x, _values(*st["w"]).t())
    if c["op"] == "gated":
        h = y / (1 + torch.exp(-y)) * torch.matmul(x, _values(*st["up"]).t())
        return [_values(*_quantize(h, 8)).half()] if c["out8"] else [h.half()]
    return [(y if st["res"] is None else y + st["res"].float()).half()]


def run(st):
    if not own:
        return _plain(st)
    import bit_group_quantized_qgemv_gb300 as q
    c = st["case"]
    if c["op"] == "quantize":
        codes, scales = st["held"]
        q.mx_quantize(st["x"], c["bits"], codes=codes, scales=scales)
        return [q.mx_dequantize(codes, scales, out=st["values"])]
    if c["op"] == "norm":
        codes, scales = st["held"]
        h, codes, scales = q.residual_rmsnorm_mxfp8(st["x"], st["gamma"], residual=st["res"], eps=EPS, h=st["h"], codes=codes, scales=scales)
        return [h, q.mx_dequantize(codes, scales, out=st["values"])]
    if c["op"] == "matvec":
        return [q.qgemv_mxfp4(st["w"], st["x"], y=st["y"], residual=st["res"])]
    if c["op"] == "product":
        return [q.mx_gemm(st["w"], st["x"], y=st["y"], residual=st["res"])]
    if not c["out8"]:
        return [q.mx_swiglu(st["w"], st["up"], st["x"], h=st["y"])]
    codes, scales = q.mx_swiglu(st["w"], st["up"], st["x"], codes=st["held"][0], scales=st["held"][1])
    return [q.mx_dequantize(codes, scales, out=st["y"])]


# ---------------------------------------------------- definition, 64 bits


def _exact_mx(x, bits):
    """Values of a microscaled format for 64-bit rows: the step of the grid at each value, then that many steps."""
    emax, emin, mant, top = (2, 0, 1, 6.0) if bits == 4 else (8, -6, 3, 448.0)
    b = x.view(x.shape[0], x.shape[1] // 32, 32)
    most = b.abs().max(-1, keepdim=True).values
    lead = torch.floor(torch.log2(torch.where(most > 0, most, 1.0)))
    lead = lead + (torch.exp2(lead + 1) <= most).double() - (torch.exp2(lead) > most).double()
    scale = torch.where(most > 0, torch.exp2(torch.clamp(lead - emax, -127, 127)), 0.0)
    v = b / torch.where(scale > 0, scale, 1.0)
    own_lead = torch.floor(torch.log2(torch.clamp(v.abs(), min=2.0 ** emin)))
    own_lead = own_lead + (torch.exp2(own_lead + 1) <= v.abs()).double()
    step = torch.exp2(torch.clamp(own_lead, min=emin) - mant)
    return (torch.clamp(torch.round(v / step) * step, -top, top) * scale).view(x.shape)


def _exact_values(codes, scales):
    """Values of held codes, from their bits."""
    if codes.dtype == torch.uint8:
        c = codes.long()
        e, f, s = (c >> 3) & 15, c & 7, c >> 7
        v = torch.where(e > 0, (8 + f).double() * torch.exp2(e.double() - 10), f.double() * 2.0 ** -9)
    else:
        c = torch.stack([(codes.long() >> (4 * i)) & 15 for i in range(8)], -1).view(codes.shape[0], -1)
        e, f, s = (c >> 1) & 3, c & 1, c >> 3
        v = torch.where(e > 0, (2 + f).double() * torch.exp2(e.double() - 2), f.double() * 0.5)
    return (1 - 2 * s.double()) * v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return [_exact_mx(st["x"].double(), case["bits"])]
    if case["op"] == "norm":
        h = st["x"].double() if st["res"] is None else (st["x"].double() + st["res"].double())
        f = h.half().double()
        return [h, _exact_mx(f / torch.sqrt((f * f).sum(-1, keepdim=True) / case["k"] + EPS) * st["gamma"].double(), 8)]
    x = st["x"].double() if case["op"] == "matvec" else _exact_values(*st["x"])

    def times(w):
        parts = [x @ _exact_values(w[0][i:i + 8192], w[1][i:i + 8192]).T for i in range(0, case["n"], 8192)]
        return torch.cat(parts, 1)

    y = times(st["w"])
    if case["op"] == "gated":
        h = y * torch.sigmoid(y) * times(st["up"])
        return [_exact_mx(h, 8) if case["out8"] else h]
    return [y if st["res"] is None else y + st["res"].double()]
