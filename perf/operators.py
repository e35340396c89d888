"""Workloads of the block-scaled (MX) operators and of the fused RMS norm, each with its plain form.

Five kinds of case, by case["op"]:

  quantize     a matrix to MX codes with one power-of-two scale per 32 values, along its rows or
               (transpose) along its columns, returned as the values that the codes stand for
  norm         h = x + residual, y = h / rms(h) * weight, with y in MX codes, in 16 bits, or both
  norm_grad    the gradients of that norm with respect to h and to the weight
  product      act(A x B^T) of MX operands, dense or with its rows grouped by expert
  linear_grad  both gradients of a linear layer whose products run on MX operands

MX format (OCP Microscaling v1.0): a block of 32 consecutive values shares the scale 2^(s - 127),
s = 127 + floor(log2(max |x|)) - emax, kept to [0, 254]; an element is x / scale rounded to nearest
even and saturated. e2m1 (4 bits): emax 2, largest 6; e4m3 (8 bits): emax 8, largest 448.
Storage: codes row-major, two e2m1 codes to a byte with the even element in the low half, rows
padded with zero codes to whole blocks; scales as (rows / 64, blocks / 16, 64, 16), rounded up.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32
# format: (bits, fraction bits, smallest exponent, emax, largest magnitude)
FORMATS = {"e2m1": (4, 1, 0, 2, 6.0), "e4m3": (8, 3, -6, 8, 448.0)}
EPS = 1e-5


def listed():
    return [
        # the activations of 16 decoding tokens on their way into a product: latency
        dict(name="quantize_tokens", op="quantize", rows=16, cols=4096, type="bf16", fmt="e4m3", transpose=False),
        # a weight matrix laid out once for serving
        dict(name="quantize_weight", op="quantize", rows=8192, cols=8192, type="bf16", fmt="e2m1", transpose=False),
        # the operand of a weight gradient: blocks run along an odd number of tokens
        dict(name="quantize_transposed", op="quantize", rows=5001, cols=4104, type="f16", fmt="e4m3", transpose=True),
        # one decoding token between two layers
        dict(name="norm_token", op="norm", rows=1, cols=4096, type="bf16", residual=True, out="mx", fmt="e4m3"),
        # the tokens of a prompt or a training step
        dict(name="norm_prompt", op="norm", rows=16768, cols=4096, type="bf16", residual=True, out="mx", fmt="e4m3"),
        # a width that is no power of two, both outputs, no residual
        dict(name="norm_odd", op="norm", rows=2047, cols=5000, type="f16", residual=False, out="both", fmt="e2m1"),
        # a training step's backward pass, with the gradient of the residual stream coming in
        dict(name="norm_grad_step", op="norm_grad", rows=8192, cols=8192, type="bf16", residual=True),
        # a few odd rows in 32 bits, the norm at the end of a network
        dict(name="norm_grad_odd", op="norm_grad", rows=333, cols=2050, type="f32", residual=False),
        # one decoding token through a layer with 4-bit weights
        dict(name="product_token", op="product", m=1, n=8192, k=8192, groups=0, a="e4m3", b="e2m1", act="none", c=False),
        # the largest dense product, 4 bits on both sides
        dict(name="product_square", op="product", m=8192, n=8192, k=8192, groups=0, a="e2m1", b="e2m1", act="none", c=False),
        # a prompt's tokens over ragged experts with 4-bit weights, one of them without tokens
        dict(name="product_experts", op="product", m=16768, n=4096, k=4096, groups=8, a="e4m3", b="e2m1", act="silu", c=False),
        # the backward pass of a linear layer in a training step: three quantisations, two products
        dict(name="linear_grad_step", op="linear_grad", m=4096, n=4096, k=2048, fmt="e4m3"),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        v = max(lo, min(hi, (v + step - 1) // step * step))
        return v - step if v == 3072 else v

    op = rng.choice(["quantize", "norm", "norm_grad", "product", "product", "linear_grad"])
    kind, fmt = rng.choice(["bf16", "f16", "f32"]), rng.choice(["e2m1", "e4m3"])
    if op == "quantize":
        return dict(op=op, rows=size(1, 8192), cols=size(32, 8192), type=kind, fmt=fmt, transpose=rng.random() < 0.5)
    if op == "norm":
        return dict(op=op, rows=size(1, 16384), cols=size(64, 4096), type=kind, residual=rng.random() < 0.5,
                    out=rng.choice(["mx", "plain", "both"]), fmt=fmt)
    if op == "norm_grad":
        return dict(op=op, rows=size(1, 8192), cols=size(64, 8192), type=kind, residual=rng.random() < 0.5)
    if op == "product":
        a, b = rng.choice([("e4m3", "e2m1"), ("e2m1", "e2m1"), ("e4m3", "e4m3")])
        groups = rng.choice([0, 0, rng.randint(2, 16)])
        # (fewer and smaller experts than the dense sizes would allow: each has weights of its own)
        return dict(op=op, m=size(1, 8192), n=size(128, 4096 if groups else 8192, 8), k=size(32, 4096 if groups else 8192),
                    groups=groups, a=a, b=b, act=rng.choice(["none", "silu", "gelu_tanh"]), c=rng.random() < 0.3)
    return dict(op=op, m=size(16, 4096), n=size(128, 4096, 8), k=size(128, 2048, 8), fmt=fmt)


def offsets(case):
    """The rows of each expert, from the case alone: uneven, and the second expert has none."""
    g, m = case["groups"], case["m"]
    r = random.Random(1000 * m + g)
    w = [0.0 if i == 1 else r.random() ** 2 + 0.02 for i in range(g)]
    cu, acc = [0], 0.0
    for x in w:
        acc += x
        cu.append(int(round(m * acc / sum(w))))
    cu[-1] = m
    return cu


def ceil(a, b):
    return -(-a // b)


def mx_bytes(rows, k, fmt):
    return rows * ceil(k, BLOCK) * (BLOCK * FORMATS[fmt][0] // 8 + 1)


def work(case):
    op = case["op"]
    if op in ("quantize", "norm", "norm_grad"):
        r, c, e = case["rows"], case["cols"], TYPES[case["type"]].itemsize
    if op == "quantize":
        q = mx_bytes(c, r, case["fmt"]) if case["transpose"] else mx_bytes(r, c, case["fmt"])
        return {"bytes": r * c * e + q + r * c * 2, "flops": 3 * r * c}
    if op == "norm":
        n = 1 + (2 if case["residual"] else 0) + (1 if case["out"] != "mx" else 0)  # x; residual and h; y
        q = mx_bytes(r, c, case["fmt"]) + r * c * 2 if case["out"] != "plain" else 0
        return {"bytes": n * r * c * e + q + c * e + r * 4, "flops": 8 * r * c}
    if op == "norm_grad":
        return {"bytes": (3 + (1 if case["residual"] else 0)) * r * c * e + c * (e + 4) + r * 4, "flops": 10 * r * c}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "product":
        outs = 1 if case["act"] == "none" or not case["c"] else 2
        cu = offsets(case) if case["groups"] else [0, m]
        used = sum(b > a for a, b in zip(cu, cu[1:]))
        return {"bytes": mx_bytes(m, k, case["a"]) + used * mx_bytes(n, k, case["b"]) + 2 * m * n * (outs + case["c"]),
                "flops": 2 * m * n * k}
    return {"bytes": 2 * (m * n + m * k) + mx_bytes(k, n, case["fmt"]) + 2 * m * k + 2 * n * k, "flops": 4 * m * n * k}


# ---- inputs


def floor_log2(a):
    """floor(log2 a) of positive values; frexp gives a fraction in [1/2, 1)."""
    return torch.frexp(a)[1] - 1


def blocks_of(x):
    """(..., k) as (..., blocks, 32), padded with zeros."""
    k = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, ceil(k, BLOCK) * BLOCK - k))
    return x.reshape(*x.shape[:-1], -1, BLOCK)


def mx_round(x, fmt):
    """x (..., k) as element values (..., blocks, 32) and scale exponents (..., blocks, 1)."""
    bits, frac, emin, emax, top = FORMATS[fmt]
    b = blocks_of(x)
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, floor_log2(a) - emax, torch.full_like(a, -127, dtype=torch.int32)).clamp(-127, 127)
    v = torch.ldexp(b, -e)
    step = (torch.frexp(v)[1] - 1).clamp(min=emin) - frac  # of the element's spacing, as an exponent
    v = torch.ldexp(torch.round(torch.ldexp(v, -step)), step).clamp(-top, top)
    return v, e


def mx_values(x, fmt):
    v, e = mx_round(x, fmt)
    return torch.ldexp(v, e).flatten(-2)[..., : x.shape[-1]]


def mx_store(x, fmt):
    """The codes and scales of x (..., rows, k) in the storage order that the file's head describes."""
    v, e = mx_round(x, fmt)
    if fmt == "e4m3":
        codes = v.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
        c = torch.searchsorted(mags, v.abs()).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
        c = c.flatten(-2)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    s = (e.squeeze(-1) + 127).to(torch.uint8)
    rows, blocks = s.shape[-2:]
    s = torch.nn.functional.pad(s, (0, ceil(blocks, 16) * 16 - blocks, 0, ceil(rows, 64) * 64 - rows))
    s = s.reshape(*s.shape[:-2], ceil(rows, 64), 64, ceil(blocks, 16), 16).transpose(-3, -2)
    return codes.contiguous(), s.contiguous()


def activations(g, shape, kind):
    """Normal values over channels of uneven size, a few of them far larger, as between a model's layers."""
    x = torch.randn(*shape, generator=g, device="cuda")
    ch = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    ch = torch.where(torch.rand(shape[-1], generator=g, device="cuda") < 0.005, 16 * ch, ch)
    return (x * ch).to(TYPES[kind])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        s["x"] = activations(g, (case["rows"], case["cols"]), case["type"])
    elif op == "norm":
        shape = (case["rows"], case["cols"])
        s["x"] = activations(g, shape, case["type"])
        s["r"] = activations(g, shape, case["type"]) if case["residual"] else None
        s["w"] = (1 + 0.2 * torch.randn(case["cols"], generator=g, device="cuda")).to(TYPES[case["type"]])
    elif op == "norm_grad":
        shape, kind = (case["rows"], case["cols"]), TYPES[case["type"]]
        s["h"] = activations(g, shape, case["type"])
        s["w"] = (1 + 0.2 * torch.randn(case["cols"], generator=g, device="cuda")).to(kind)
        s["dy"] = torch.randn(*shape, generator=g, device="cuda").to(kind)
        s["dres"] = torch.randn(*shape, generator=g, device="cuda").to(kind) if case["residual"] else None
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(-1) + EPS).float()  # the forward pass keeps it
    elif op == "product":
        m, n, k, G = case["m"], case["n"], case["k"], case["groups"]
        s["A"] = mx_store(activations(g, (m, k), "f32"), case["a"])
        s["B"] = mx_store(torch.randn(*((G, n, k) if G else (n, k)), generator=g, device="cuda") / math.sqrt(k), case["b"])
        s["C"] = torch.randn(m, n, generator=g, device="cuda").bfloat16() if case["c"] else None
        s["cu"] = torch.tensor(offsets(case), dtype=torch.int32, device="cuda") if G else None
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["dY"] = torch.randn(m, n, generator=g, device="cuda").bfloat16()
        s["X"] = activations(g, (m, k), "bf16")
        w = torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)
        s["WT"] = mx_store(w.t().contiguous(), case["fmt"])  # W^T (k, n), blocks along n
    if own:
        keep(s)
    return s


def keep(s):
    """What a program keeps beside its inputs: output buffers, operand handles and plans."""
    import gemm_epilogue_persistent_amd as gep
    case, op = s["case"], s["case"]["op"]
    new = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    if op == "quantize":
        shape = (case["cols"], case["rows"]) if case["transpose"] else (case["rows"], case["cols"])
        s["q"], s["v"] = gep.mx_empty(*shape, case["fmt"]), new(shape, torch.bfloat16)
    elif op == "norm":
        x = s["x"]
        s["out_h"] = torch.empty_like(x) if case["residual"] else None
        s["out_y"] = torch.empty_like(x) if case["out"] != "mx" else None
        s["rstd"] = new((x.shape[0],), torch.float32)
        if case["out"] != "plain":
            s["q"], s["v"] = gep.mx_empty(*x.shape, case["fmt"]), new(x.shape, torch.bfloat16)
        else:
            s["q"] = None
    elif op == "norm_grad":
        h = s["h"]
        s["dx"], s["dw"] = torch.empty_like(h), new((h.shape[1],), torch.float32)
        s["work"] = new((gep.rmsnorm_backward_workspace(*h.shape),), torch.uint8)
    elif op == "product":
        k, (m, n) = case["k"], (case["m"], case["n"])
        s["a"], s["b"] = gep.MxTensor(*s["A"], case["a"], k), gep.MxTensor(*s["B"], case["b"], k)
        post = case["act"] != "none"
        s["D"] = new((m, n), torch.bfloat16) if case["c"] or not post else None
        s["P"] = new((m, n), torch.bfloat16) if post else None
        s["plan"] = gep.MxPlan(s["a"], s["b"], s["C"], s["D"], s["P"], act=case["act"], cu_seqlens_m=s["cu"])
    else:
        m, n, k, fmt = case["m"], case["n"], case["k"], case["fmt"]
        s["w"] = gep.MxTensor(*s["WT"], fmt, n)
        s["dy_n"], s["dy_m"], s["x_m"] = gep.mx_empty(m, n, fmt), gep.mx_empty(n, m, fmt), gep.mx_empty(k, m, fmt)
        s["dX"], s["dW"] = new((m, k), torch.bfloat16), new((n, k), torch.bfloat16)
        s["plan_x"] = gep.MxPlan(s["dy_n"], s["w"], None, s["dX"])
        s["plan_w"] = gep.MxPlan(s["dy_m"], s["x_m"], None, s["dW"])


# ---- one pass


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import gemm_epilogue_persistent_amd as gep
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        gep.mx_quantize(s["x"], case["fmt"], out=s["q"], transpose=case["transpose"])
        return {"values": gep.mx_dequantize(s["q"], out=s["v"])}
    if op == "norm":
        gep.rmsnorm(s["x"], s["w"], residual=s["r"], eps=EPS, h=s["out_h"], y=s["out_y"], q=s["q"], rstd=s["rstd"])
        v = gep.mx_dequantize(s["q"], out=s["v"]) if s["q"] is not None else None
        return {"h": s["out_h"], "rstd": s["rstd"], "values": v, "y": s["out_y"]}
    if op == "norm_grad":
        gep.rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dx=s["dx"], dw=s["dw"], dres=s["dres"], workspace=s["work"])
        return {"dw": s["dw"], "dx": s["dx"]}
    if op == "product":
        s["plan"].run(s["a"], s["b"], s["C"], s["D"], s["P"], cu_seqlens_m=s["cu"])
        return {"d": s["D"], "post": s["P"]}
    gep.mx_quantize(s["dY"], case["fmt"], out=s["dy_n"])
    gep.mx_quantize(s["dY"], case["fmt"], out=s["dy_m"], transpose=True)
    gep.mx_quantize(s["X"], case["fmt"], out=s["x_m"], transpose=True)
    s["plan_x"].run(s["dy_n"], s["w"], None, s["dX"])
    s["plan_w"].run(s["dy_m"], s["x_m"], None, s["dW"])
    return {"dw": s["dW"], "dx": s["dX"]}


def mx_load(stored, fmt, k):
    """The values (..., rows, k) in 32 bits of codes and scales."""
    codes, tiles = stored
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        table = torch.cat([table, -table])
        v = table[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(-2)
    s = tiles.transpose(-3, -2).flatten(-2).flatten(-3, -2)
    s = torch.ldexp(torch.ones((), device=codes.device), s[..., : codes.shape[-2], : v.shape[-1] // BLOCK].int() - 127)
    return (v.unflatten(-1, (-1, BLOCK)) * s.unsqueeze(-1)).flatten(-2)[..., :k]


def activation(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        x = s["x"].float()
        return {"values": mx_values(x.t() if case["transpose"] else x, case["fmt"]).bfloat16()}
    if op == "norm":
        h = s["x"]
        if s["r"] is not None:
            h = (s["x"].float() + s["r"].float()).to(h.dtype)
        f = h.float()
        rstd = torch.rsqrt(f.square().mean(-1) + EPS)
        y = f * rstd[:, None] * s["w"].float()
        return {"h": h if s["r"] is not None else None, "rstd": rstd,
                "values": mx_values(y, case["fmt"]).bfloat16() if case["out"] != "plain" else None,
                "y": y.to(h.dtype) if case["out"] != "mx" else None}
    if op == "norm_grad":
        h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
        n = h * rstd
        p = dy * s["w"].float()
        dx = rstd * (p - n * (p * n).mean(-1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dw": (dy * n).sum(0), "dx": dx.to(s["h"].dtype)}
    if op == "product":
        k, G = case["k"], case["groups"]
        a, b = mx_load(s["A"], case["a"], k), mx_load(s["B"], case["b"], k)
        if G:
            # rows of each expert side by side, short ones filled up with zeros
            cu, rows = s["cu"].long(), torch.arange(case["m"], device=a.device)
            group = torch.searchsorted(cu[1:].contiguous(), rows, right=True)
            at = rows - cu[group]
            longest = max(y - x for x, y in zip(offsets(case), offsets(case)[1:]))
            side = torch.zeros(G, longest, k, device=a.device)
            side[group, at] = a
            x = torch.matmul(side, b.transpose(1, 2).contiguous())[group, at]
        else:
            x = a @ b.t()
        if s["C"] is not None:
            x = x + s["C"].float()
        post = case["act"] != "none"
        return {"d": x.bfloat16() if case["c"] or not post else None,
                "post": activation(x, case["act"]).bfloat16() if post else None}
    fmt, dy = case["fmt"], s["dY"].float()
    dx = mx_values(dy, fmt) @ mx_load(s["WT"], fmt, case["n"]).t()
    dw = mx_values(dy.t(), fmt) @ mx_values(s["X"].float().t(), fmt).t()
    return {"dw": dw.bfloat16(), "dx": dx.bfloat16()}


# ---- the definitions in 64 bits


def representable(fmt, device):
    """Every magnitude of the format, ascending, so that the index's last bit is the fraction's."""
    bits, frac, emin, emax, top = FORMATS[fmt]
    mags = [math.ldexp(i, emin - frac) for i in range(1 << frac)]
    for e in range(emin, emax + 1):
        mags += [math.ldexp((1 << frac) + i, e - frac) for i in range(1 << frac)]
    return torch.tensor([v for v in mags if v <= top], dtype=torch.float64, device=device)


def nearest(x, fmt):
    """x (..., k) in 64 bits as the nearest MX values: ties to the even code, larger ones to the largest."""
    mags = representable(fmt, x.device)
    between = (mags[1:] + mags[:-1]) / 2
    k, out = x.shape[-1], []
    for part in x.split(max(1, (1 << 26) // max(1, k)), 0):
        b = torch.zeros(*part.shape[:-1], ceil(k, BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
        b[..., :k] = part
        b = b.reshape(*b.shape[:-1], -1, BLOCK)
        a = b.abs().max(-1, keepdim=True).values
        e = torch.log2(a.clamp(min=1e-300)).floor()
        e = torch.where(torch.exp2(e) > a, e - 1, torch.where(torch.exp2(e + 1) <= a, e + 1, e))
        scale = torch.exp2((e - FORMATS[fmt][3]).clamp(-127, 127))
        v = b.abs() / scale
        below, above = torch.bucketize(v, between), torch.bucketize(v, between, right=True)
        at = torch.where(below == above, below, below + below % 2)  # on a border: the even one of the two
        v = mags[at] * scale * torch.sign(b)
        out.append(v.reshape(*part.shape[:-1], -1)[..., :k])
    return torch.cat(out, 0)


def decode(stored, fmt, rows, k):
    """Codes and scales of one matrix by the bit fields of the format, in 64 bits."""
    bits, frac, emin, emax, top = FORMATS[fmt]
    codes, tiles = stored
    c = codes.long()
    if bits == 4:
        c = torch.stack([c % 16, c // 16], -1).reshape(rows, -1)
    sign = 1.0 - 2.0 * (c >> (bits - 1)).double()
    c = c % (1 << (bits - 1))
    e, f = c >> frac, (c % (1 << frac)).double() / (1 << frac)
    v = sign * torch.where(e == 0, f * 2.0**emin, (1 + f) * torch.exp2((e - 1 + emin).double()))
    r = torch.arange(rows, device=c.device)[:, None]
    b = (torch.arange(v.shape[1], device=c.device) // BLOCK)[None, :]
    scale = tiles[r // 64, b // 16, r % 64, b % 16].double()
    return (v * torch.exp2(scale - 127))[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        return {"values": nearest(x.t().contiguous() if case["transpose"] else x, case["fmt"])}
    if op == "norm":
        h = s["x"].double()
        if s["r"] is not None:
            h = (h + s["r"].double()).to(s["x"].dtype).double()
        rstd = 1 / torch.sqrt((h * h).sum(1) / case["cols"] + EPS)
        y = s["w"].double() * (h * rstd.unsqueeze(1))
        return {"h": h if s["r"] is not None else None, "rstd": rstd,
                "values": nearest(y, case["fmt"]) if case["out"] != "plain" else None, "y": y if case["out"] != "mx" else None}
    if op == "norm_grad":
        # y_j = w_j h_j r with r = (mean h^2 + eps)^(-1/2), so dr/dh_i = -r^3 h_i / n
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["w"].double(), s["rstd"].double().unsqueeze(1)
        dx = r * w * dy - h * r**3 / case["cols"] * (dy * w * h).sum(1, keepdim=True)
        if s["dres"] is not None:
            dx += s["dres"].double()
        return {"dw": (dy * h * r).sum(0), "dx": dx}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = decode(s["A"], case["a"], m, k)
        x = torch.empty(m, n, dtype=torch.float64, device="cuda")
        if case["groups"]:
            cu = offsets(case)
            for g in range(case["groups"]):
                if cu[g + 1] > cu[g]:
                    x[cu[g]:cu[g + 1]] = a[cu[g]:cu[g + 1]] @ decode((s["B"][0][g], s["B"][1][g]), case["b"], n, k).t()
        else:
            x = a @ decode(s["B"], case["b"], n, k).t()
        if case["c"]:
            x += s["C"].double()
        p = x
        if case["act"] == "silu":
            p = x * torch.sigmoid(x)
        elif case["act"] == "gelu_tanh":
            p = x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x**3))
        post = case["act"] != "none"
        return {"d": x if case["c"] or not post else None, "post": p if post else None}
    m, n, k, fmt = case["m"], case["n"], case["k"], case["fmt"]
    dy, x = s["dY"].double(), s["X"].double()
    dx = nearest(dy, fmt) @ decode(s["WT"], fmt, k, n).t()
    dw = nearest(dy.t().contiguous(), fmt) @ nearest(x.t().contiguous(), fmt).t()
    return {"dw": dw, "dx": dx}
