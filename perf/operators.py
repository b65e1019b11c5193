"""What the ragged expert products and the 4-bit operators are measured on.

Five operators of the layer's experts, each as a user of the package calls it:

  product       y[r] = W_e x[r] for the rows r of expert e, 16-bit operands
  gradients     the same product's backward: dx[r] = W_e^T dy[r] and
                dW_e = sum over the rows of e of dy[r] x[r]^T
  quantize      rows to microscaled 4-bit values and back (the values that the
                codes stand for are what is returned)
  dequantize    stored 4-bit values to bf16 or fp32
  product_fp4   the grouped product of 4-bit rows and 4-bit weights

The rows of all experts lie in one buffer in expert order: expert e holds
sizes[e] rows (any number, none included) from starts[e] on, either back to
back or, as `moe_dispatch` leaves them, each expert from a multiple of 128.

Formats. An element is one of 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign.
  mx  blocks of 32, scale 2^(floor(log2 amax) - 2), its exponent held in 8 bits
  nv  blocks of 16, scale amax / (6 g) rounded to an 8-bit float (4 exponent
      and 3 mantissa bits, at most 448), g the tensor's 32-bit scale
An element is the nearest representable number to x / (scale * g), ties to the
even code, at most 6. A tensor's g is amax / 2688 (at least 2^-100).
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ALIGN = 128


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step of 8 tokens: the routed rows on their way to 4 bits
        dict(name="quantize_nv_decode", op="quantize", fmt="nv", groups=1, rows=64, cols=2048, dtype="bf16"),
        # a prefill's routed rows, 4096 tokens to 8 experts each
        dict(name="quantize_mx_rows", op="quantize", fmt="mx", groups=1, rows=32768, cols=2048, dtype="bf16"),
        # all down projections of a layer from fp32 masters, a scale per expert
        dict(name="quantize_nv_weights", op="quantize", fmt="nv", groups=64, rows=2048, cols=1024, dtype="fp32"),
        # an odd number of rows of an uncommon width, read back to fp32
        dict(name="dequantize_mx_odd", op="dequantize", fmt="mx", groups=1, rows=999, cols=1056, dtype="fp32"),
        # a layer's stored gate/up projections read back to bf16
        dict(name="dequantize_nv_weights", op="dequantize", fmt="nv", groups=64, rows=2048, cols=2048, dtype="bf16"),
        # decode: 8 tokens, 64 rows over 64 experts; weights are all that is read
        dict(name="product_decode", op="product", experts=64, rows=64, n=2048, k=2048, spread="even", pad=False,
             out="bf16"),
        # prefill of 4096 tokens under a skewed router, rows back to back
        dict(name="product_prefill", op="product", experts=64, rows=32768, n=2048, k=2048, spread="zipf", pad=False,
             out="bf16"),
        # a training step of 16384 tokens through the gate/up projection, fp32 weight gradients
        dict(name="gradients_train", op="gradients", experts=64, rows=131072, n=2048, k=2048, spread="zipf",
             pad=False, out="fp32"),
        # a small layer of odd sizes in padded groups
        dict(name="gradients_odd", op="gradients", experts=7, rows=1001, n=1048, k=520, spread="even", pad=True,
             out="bf16"),
        # decode on 4-bit experts
        dict(name="fp4_nv_decode", op="product_fp4", fmt="nv", experts=64, rows=64, n=2048, k=2048, spread="even",
             pad=False, out="bf16"),
        # a small layer of odd sizes in the other format
        dict(name="fp4_mx_odd", op="product_fp4", fmt="mx", experts=24, rows=5003, n=1416, k=1056, spread="zipf",
             pad=False, out="fp32"),
        # a large batch through the gate/up projection
        dict(name="fp4_nv_batch", op="product_fp4", fmt="nv", experts=64, rows=131072, n=2048, k=2048, spread="even",
             pad=True, out="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "dequantize", "product", "gradients", "product_fp4"])
    if op in ("quantize", "dequantize"):
        groups = rng.choice([1, 1, _logint(rng, 2, 64)])
        cols = 32 * _logint(rng, 1, 128)
        rows = _logint(rng, 1, max(2, min(131072, (1 << 27) // (groups * cols))))
        return dict(op=op, fmt=rng.choice(["nv", "mx"]), groups=groups, rows=rows, cols=cols,
                    dtype=rng.choice(["bf16", "fp32"]))
    unit = 32 if op == "product_fp4" else 8
    n = 8 * _logint(rng, 1, 512)
    k = unit * _logint(rng, 1, 4096 // unit)
    experts = _logint(rng, 1, max(1, min(128, (1 << 28) // (n * k))))
    rows = _logint(rng, 1, min(131072, (1 << 39) // (n * k)))
    case = dict(op=op, experts=experts, rows=rows, n=n, k=k, spread=rng.choice(["even", "zipf", "one"]),
                pad=rng.random() < 0.3, out=rng.choice(["bf16", "fp32"]))
    if op == "product_fp4":
        case["fmt"] = rng.choice(["nv", "mx"])
    return case


def _shares(case):
    """Each expert's share of the rows: equal, a Zipf law, or all to one expert."""
    e = case["experts"]
    if case["spread"] == "even":
        p = [1.0] * e
    elif case["spread"] == "zipf":
        p = [(i + 1) ** -1.2 for i in range(e)]
    else:
        p = [0.0] * e
        p[e // 2] = 1.0
    s = sum(p)
    return [v / s for v in p]


def work(case):
    """Each input read once and each output written once; two operations a
    multiply-add. Weights count for the experts that rows are expected to reach."""
    if case["op"] in ("quantize", "dequantize"):
        count = case["groups"] * case["rows"] * case["cols"]
        held = count // 2 + count // (16 if case["fmt"] == "nv" else 32)
        wide = count * (2 if case["dtype"] == "bf16" else 4)
        if case["op"] == "dequantize":
            return {"bytes": held + wide, "flops": 2 * count}
        return {"bytes": 2 * wide + held, "flops": 8 * count}
    m, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
    reached = sum(1.0 - (1.0 - p) ** m for p in _shares(case))
    out = 2 if case["out"] == "bf16" else 4
    if case["op"] == "product":
        return {"bytes": int(2 * m * k + 2 * reached * n * k + out * m * n), "flops": 2 * m * n * k}
    if case["op"] == "gradients":
        return {"bytes": int(2 * m * (n + k) + 2 * reached * n * k + 2 * m * k + out * e * n * k),
                "flops": 4 * m * n * k}
    per = 0.5 + (1 / 16 if case["fmt"] == "nv" else 1 / 32)
    return {"bytes": int(per * m * k + per * reached * n * k + out * m * n), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ 4-bit values, plain form


def _pow2(e):
    """2^e in fp64 for whole e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _plain_tensor_scale(x3):
    amax = x3.float().abs().flatten(1).amax(dim=1)
    # a tensor divisor: division by a Python number is a product with its reciprocal on a GPU
    return torch.clamp(amax / torch.full_like(amax, 2688.0), min=2.0 ** -100)


def _plain_block_scale(amax, g, fmt):
    """The blocks' scales as fp64 numbers, from their largest magnitudes."""
    amax = amax.double()
    if fmt == "mx":
        exp = torch.frexp(amax).exponent - 3
        return _pow2(torch.where(amax > 0, exp, torch.full_like(exp, -127)).clamp(-127, 127))
    q = (amax / (6.0 * g.double())).clamp(max=448.0)
    exp = (torch.frexp(q).exponent - 1).clamp(min=-6)
    step = _pow2(exp - 3)
    return torch.clamp(torch.round(q / step) * step, max=448.0)


def _plain_codes(x2, g, fmt):
    """x2 [rows, cols] and its tensor scale g: (codes with the sign in bit 3,
    block scales as fp64). Borders between neighbours are compared in fp64, where
    border * scale * g is exact."""
    size = 16 if fmt == "nv" else 32
    rows, cols = x2.shape
    xb = x2.float().reshape(rows, cols // size, size)
    mag = xb.abs()
    scale = _plain_block_scale(mag.amax(dim=-1), g, fmt)
    step = (scale * (g.double() if fmt == "nv" else 1.0)).unsqueeze(-1)
    mag = mag.double()
    code = torch.zeros(mag.shape, dtype=torch.uint8, device=x2.device)
    for i, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        at = border * step
        code += (mag > at) if i % 2 == 0 else (mag >= at)  # a tie goes to the even code
    code = torch.where(step > 0, code, torch.zeros_like(code))
    return (code + 8 * (xb < 0).to(torch.uint8)).reshape(rows, cols), scale


def _grid(device):
    return torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=device)


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _scale_bytes(scale, fmt):
    if fmt == "mx":
        return (torch.frexp(scale).exponent - 1 + 127).to(torch.uint8)
    return scale.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_values(packed, scale_bytes, g, fmt):
    """The fp32 values of packed codes [rows, cols / 2]."""
    rows, half = packed.shape
    codes = torch.stack((packed & 15, packed >> 4), dim=-1).reshape(rows, 2 * half)
    v = _grid(packed.device)[codes.int()]
    size = 16 if fmt == "nv" else 32
    if fmt == "mx":
        s = _pow2(scale_bytes.int() - 127).float()
    else:
        s = scale_bytes.view(torch.float8_e4m3fn).float()
    v = (v.reshape(rows, -1, size) * s.unsqueeze(-1)).reshape(rows, 2 * half)
    return v * g if fmt == "nv" else v


def _quantize_plain_3d(x3, g, fmt):
    """Packed codes and scale bytes of [groups, rows, cols], one group at a time."""
    codes, scales = [], []
    for i in range(x3.shape[0]):
        c, s = _plain_codes(x3[i], g[i], fmt)
        codes.append(_pack(c))
        scales.append(_scale_bytes(s, fmt))
    return torch.stack(codes), torch.stack(scales)


# ------------------------------------------------------------------ inputs


def _rows(gen, rows, cols, dtype):
    """Rows as they leave a pre-norm: unit root mean square."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    return (x * torch.rsqrt(x.pow(2).mean(dim=-1, keepdim=True) + 1e-5)).to(dtype)


def _weights(gen, experts, n, k, dtype):
    w = torch.empty(experts, n, k, dtype=dtype, device="cuda")
    for e in range(experts):
        w[e] = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    return w


def _layout(case, seed):
    """Rows per expert, first row of each expert, rows of the buffer."""
    g = torch.Generator().manual_seed(7919 * seed + 13)
    pick = torch.multinomial(torch.tensor(_shares(case)), case["rows"], replacement=True, generator=g)
    sizes = torch.bincount(pick, minlength=case["experts"]).tolist()
    starts, at = [], 0
    for s in sizes:
        starts.append(at)
        at += (s + _ALIGN - 1) // _ALIGN * _ALIGN if case["pad"] else s
    if case["pad"]:  # the buffer is sized for any split of the rows
        at = (case["rows"] + case["experts"] * (_ALIGN - 1) + _ALIGN - 1) // _ALIGN * _ALIGN
    return sizes, starts, at


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(104729 * seed + 7)
    st = dict(case)
    if case["op"] in ("quantize", "dequantize"):
        shape = (case["groups"], case["rows"], case["cols"])
        dt = _DT[case["dtype"]] if case["op"] == "quantize" else torch.bfloat16
        if case["groups"] > 1:
            x = _weights(gen, *shape, dt)
        else:
            x = _rows(gen, case["rows"], case["cols"], dt).reshape(shape)
        st["x"] = x
        if case["op"] == "dequantize":
            st["g"] = _plain_tensor_scale(x)
            st["codes"], st["scales"] = _quantize_plain_3d(x, st["g"], case["fmt"])
            del st["x"]
        else:
            size = 16 if case["fmt"] == "nv" else 32
            st["codes"] = torch.empty(shape[0], shape[1], shape[2] // 2, dtype=torch.uint8, device="cuda")
            st["scales"] = torch.empty(shape[0], shape[1], shape[2] // size, dtype=torch.uint8, device="cuda")
            st["g"] = torch.empty(shape[0], device="cuda")
        st["values"] = torch.empty(shape, dtype=_DT[case["dtype"]], device="cuda")
        return st

    sizes, starts, total = _layout(case, seed)
    experts, n, k = case["experts"], case["n"], case["k"]
    out = _DT[case["out"]]
    st["sizes"], st["starts"] = sizes, starts
    offsets = [0]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    st["group_start"] = (torch.tensor(starts + [total], dtype=torch.int32, device="cuda") if case["pad"] else None)
    x = _rows(gen, total, k, torch.bfloat16)
    w = _weights(gen, experts, n, k, torch.bfloat16)
    if own:
        import sparse_moe_transformer_route_b200 as moe
        st["shape"] = moe.grouped_shape(total, experts, n, k, out)
        st["ws"] = moe.grouped_workspace(st["shape"])
    if case["op"] == "product_fp4":
        fmt = case["fmt"]
        st["xg"] = _plain_tensor_scale(x.unsqueeze(0))
        st["wg"] = _plain_tensor_scale(w)
        xq, xs = _quantize_plain_3d(x.unsqueeze(0), st["xg"], fmt)
        st["xq"], st["xs"] = xq[0], xs[0]
        st["wq"], st["wscale"] = _quantize_plain_3d(w, st["wg"], fmt)
        st["y"] = torch.zeros(total, n, dtype=out, device="cuda")
        return st
    st["x"], st["w"] = x, w
    if case["op"] == "product":
        st["y"] = torch.zeros(total, n, dtype=out, device="cuda")
    else:
        st["dy"] = torch.randn(total, n, generator=gen, device="cuda").to(torch.bfloat16)
        st["dx"] = torch.zeros(total, k, dtype=torch.bfloat16, device="cuda")
        st["dw"] = torch.empty(experts, n, k, dtype=out, device="cuda")
        if own:
            import sparse_moe_transformer_route_b200 as moe
            st["shape_dx"] = moe.grouped_shape(total, experts, n, k, torch.bfloat16)
    return st


# ------------------------------------------------------------------ one pass


def _run_own(st):
    import sparse_moe_transformer_route_b200 as moe

    op = st["op"]
    if op in ("quantize", "dequantize"):
        fmt = moe.MOE_NVFP4 if st["fmt"] == "nv" else moe.MOE_MXFP4
        g = st["g"] if st["fmt"] == "nv" else None
        if op == "quantize":
            if g is not None:
                moe.moe_tensor_scale_microscaled(st["x"], g)
            moe.moe_quantize_microscaled(fmt, st["x"], g, st["codes"], st["scales"])
        moe.moe_dequantize_microscaled(fmt, st["codes"], st["scales"], g, st["values"])
        return (st["values"], g) if (op == "quantize" and g is not None) else st["values"]
    gs, off = st["group_start"], st["offsets"]
    if op == "product":
        moe.moe_grouped_gemm(st["shape"], st["x"], gs, off, st["w"], st["y"], st["ws"])
        return st["y"]
    if op == "gradients":
        moe.moe_grouped_gemm_dgrad(st["shape_dx"], st["dy"], gs, off, st["w"], st["dx"], st["ws"])
        moe.moe_grouped_gemm_wgrad(st["shape"], st["dy"], st["x"], gs, off, st["dw"], st["ws"])
        return st["dx"], st["dw"]
    fmt, xg, wg = (moe.MOE_NVFP4, st["xg"], st["wg"]) if st["fmt"] == "nv" else (moe.MOE_MXFP4, None, None)
    moe.moe_grouped_gemm_microscaled(st["shape"], fmt, st["xq"], st["xs"], xg, gs, off, st["wq"], st["wscale"], wg,
                                     st["y"], st["ws"])
    return st["y"]


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "quantize":
        g = _plain_tensor_scale(st["x"])
        out = torch.empty_like(st["values"])
        for i in range(st["x"].shape[0]):
            c, s = _plain_codes(st["x"][i], g[i], st["fmt"])
            out[i] = _plain_values(_pack(c), _scale_bytes(s, st["fmt"]), g[i], st["fmt"]).to(out.dtype)
        return (out, g) if st["fmt"] == "nv" else out
    if op == "dequantize":
        out = torch.empty_like(st["values"])
        for i in range(out.shape[0]):
            out[i] = _plain_values(st["codes"][i], st["scales"][i], st["g"][i], st["fmt"]).to(out.dtype)
        return out
    groups = [(e, a, a + s) for e, (a, s) in enumerate(zip(st["starts"], st["sizes"])) if s > 0]
    if op == "product":
        y = torch.zeros_like(st["y"])
        for e, lo, hi in groups:
            y[lo:hi] = (st["x"][lo:hi].float() @ st["w"][e].float().t()).to(y.dtype)
        return y
    if op == "gradients":
        dx, dw = torch.zeros_like(st["dx"]), torch.zeros_like(st["dw"])
        for e, lo, hi in groups:
            dy = st["dy"][lo:hi].float()
            dx[lo:hi] = (dy @ st["w"][e].float()).to(dx.dtype)
            dw[e] = (dy.t() @ st["x"][lo:hi].float()).to(dw.dtype)
        return dx, dw
    one = torch.ones((), device="cuda")
    y = torch.zeros_like(st["y"])
    for e, lo, hi in groups:
        x = _plain_values(st["xq"][lo:hi], st["xs"][lo:hi], one, st["fmt"])
        w = _plain_values(st["wq"][e], st["wscale"][e], one, st["fmt"])
        r = x @ w.t()
        if st["fmt"] == "nv":
            r = r * (st["xg"][0] * st["wg"][e])
        y[lo:hi] = r.to(y.dtype)
    return y


# ------------------------------------------------------------------ the definition in 64 bits


def _two_to(e):
    """2^e for whole e held in fp64, from a table."""
    table = torch.tensor([2.0 ** i for i in range(-200, 201)], dtype=torch.float64, device=e.device)
    return table[e.long() + 200]


def _exact_read(packed, scale_bytes, g, fmt):
    """The real values of stored codes: sign, exponent and mantissa fields spelt out."""
    def element(c):
        c = c.double()
        sign = 1.0 - 2.0 * torch.floor(c / 8.0)
        c = torch.remainder(c, 8.0)
        exp, man = torch.floor(c / 2.0), torch.remainder(c, 2.0)
        return sign * torch.where(exp > 0, (1.0 + man / 2.0) * _two_to(exp - 1.0), man / 2.0)

    low = element(packed % 16)
    high = element(torch.div(packed, 16, rounding_mode="floor"))
    v = torch.stack((low, high), dim=2).flatten(1)
    b = scale_bytes.double()
    if fmt == "mx":
        return v * _two_to(b - 127.0).repeat_interleave(32, dim=1)
    exp, man = torch.floor(b / 8.0), torch.remainder(b, 8.0)
    s = torch.where(exp > 0, (1.0 + man / 8.0) * _two_to(exp - 7.0), man * 2.0 ** -9)
    return v * s.repeat_interleave(16, dim=1) * (1.0 if g is None else g.double())


def _exact_round_trip(x2, g32, g64, fmt):
    """x2 through its 4-bit form: round to a multiple of the binade's step. g32 is
    the scale that the format stores (32 bits), which the blocks are divided by."""
    x = x2.double()
    size = 32 if fmt == "mx" else 16
    top = x.abs().unflatten(1, (-1, size)).amax(dim=2)
    if fmt == "mx":
        e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=2.0 ** -200))), torch.full_like(top, -125.0))
        e = torch.where(_two_to(e + 1.0) <= top, e + 1.0, e)  # log2 may fall short of a power of two
        e = torch.where(_two_to(e) > top, e - 1.0, e)
        s = _two_to((e - 2.0).clamp(min=-127.0))
        unit = s
    else:
        t = top / (g32.double() * 6.0)
        low = _two_to(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))).clamp(max=8.0) - 3.0)
        s = (torch.round(t / low) * low).clamp(max=448.0)
        unit = s * g32.double()
    unit = unit.repeat_interleave(size, dim=1)
    q = torch.where(unit > 0, x.abs() / unit.clamp(min=1e-300), torch.zeros_like(x)).clamp(max=6.0)
    ulp = torch.where(q >= 4.0, 2.0, torch.where(q >= 2.0, 1.0, 0.5)).double()
    v = torch.round(q / ulp) * ulp
    wide = s.repeat_interleave(size, dim=1) * (1.0 if fmt == "mx" else g64)
    return torch.sign(x) * v * wide


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt = case["op"], case.get("fmt")
    if op == "quantize":
        out = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
        scales = []
        for i in range(case["groups"]):
            big = st["x"][i].double().abs().max()
            scales.append((big / torch.full_like(big, 2688.0)).clamp(min=2.0 ** -100))
            g32 = scales[-1].float()
            out[i] = _exact_round_trip(st["x"][i], g32, g32.double(), fmt)
        return (out, torch.stack(scales)) if fmt == "nv" else out
    if op == "dequantize":
        out = torch.empty(st["values"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["groups"]):
            out[i] = _exact_read(st["codes"][i], st["scales"][i], st["g"][i], fmt)
        return out
    spans = [(e, slice(a, a + s)) for e, (a, s) in enumerate(zip(st["starts"], st["sizes"]))]
    if op == "product":
        y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
        for e, rows in spans:
            y[rows] = torch.einsum("rk,nk->rn", st["x"][rows].double(), st["w"][e].double())
        return y
    if op == "gradients":
        dx = torch.zeros(st["dx"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(st["dw"].shape, dtype=torch.float64, device="cuda")
        for e, rows in spans:
            dy = st["dy"][rows].double()
            dx[rows] = torch.einsum("rn,nk->rk", dy, st["w"][e].double())
            dw[e] = torch.einsum("rn,rk->nk", dy, st["x"][rows].double())
        return dx, dw
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    for e, rows in spans:
        x = _exact_read(st["xq"][rows], st["xs"][rows], st["xg"][0], fmt)
        w = _exact_read(st["wq"][e], st["wscale"][e], st["wg"][e], fmt)
        y[rows] = torch.einsum("rk,nk->rn", x, w)
    return y
