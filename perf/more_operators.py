"""Workloads of the 8-bit operators with a scale per 128 values, of activation checkpoints in that format and
of the router's balance loss, each with its plain form.

Six kinds of case, by case["op"]:

  quantize     a matrix to 8-bit codes with a scale per 128 values of a row, or per 128 x 128 tile, and the
               same of its transpose, returned as the values that the codes stand for
  product      act(A B^T + C) of such operands, dense or with its rows grouped by expert
  linear_grad  both gradients of a linear layer whose products run on such operands
  act          y = act(x), quantised for the next product, and x itself kept in 8 bits
  act_grad     from those 8 bits: dx = dy act'(x), quantised along rows and columns or plain, and act(x) again,
               quantised along columns for the weight's gradient
  balance      per-expert counts, a router's balance loss and its gradient

Format: codes are OCP e4m3. Of a block, r = 448 / max |x| in fp32, 2^126 at most, cut to 13 significant bits (so that x r is
exact in fp32 for 16-bit x); a code is x r rounded to nearest even, scale = 1 / r in fp32, the value code * scale. Storage: codes row-major, rows padded with zero codes to 16
bytes; scales in fp32, (rows / 64, blocks / 4, 64, 4) rounded up, or of tiles (rows / 128, blocks) with the blocks
rounded up to a multiple of 4.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128
TOP = 448.0
MOST = 2.0**126


def listed():
    return [
        # the activations of 16 decoding tokens on their way into a product: latency
        dict(name="quantize_tokens", op="quantize", rows=16, cols=4096, type="bf16", tiles=False, back=False),
        # a weight laid out for the forward and the backward product after an optimizer's step
        dict(name="quantize_weight", op="quantize", rows=8192, cols=8192, type="bf16", tiles=True, back=True),
        # a gradient on its way into both products of a backward pass: an odd number of tokens
        dict(name="quantize_both", op="quantize", rows=5001, cols=4104, type="f16", tiles=False, back=True),
        # one decoding token through a layer
        dict(name="product_token", op="product", m=1, n=8192, k=8192, groups=0, b="tiles", act="none", c=False),
        # the largest dense product
        dict(name="product_square", op="product", m=8192, n=8192, k=8192, groups=0, b="tiles", act="none", c=False),
        # a prompt's tokens over ragged experts, one of them without tokens
        dict(name="product_experts", op="product", m=16768, n=4096, k=4096, groups=8, b="tiles", act="silu", c=False),
        # the backward pass of a linear layer in a training step: two quantisations, two products
        dict(name="linear_grad_step", op="linear_grad", m=4096, n=4096, k=2048),
        # the activation between a training step's two products
        dict(name="act_step", op="act", rows=16768, cols=4096, type="bf16", act="silu", plain=False),
        # a step's backward pass through it: everything that its four products take
        dict(name="act_grad_step", op="act_grad", rows=8192, cols=8192, type="bf16", act="gelu_tanh", plain=False),
        # odd sizes in 32 bits, the gradient for a product in 16 bits or more
        dict(name="act_grad_odd", op="act_grad", rows=333, cols=2050, type="f32", act="relu_sq", plain=True),
        # a few tokens over eight experts
        dict(name="balance_tokens", op="balance", batch=1, tokens=16, experts=8, k=2, type="f32", scores="softmax", mask=False),
        # a step's padded sequences over many experts, a loss for each sequence
        dict(name="balance_sequences", op="balance", batch=8, tokens=4096, experts=256, k=8, type="bf16", scores="sigmoid", mask=True),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, (v + step - 1) // step * step))

    op = rng.choice(["quantize", "product", "product", "linear_grad", "act", "act_grad", "balance", "balance"])
    kind, act = rng.choice(["bf16", "f16", "f32"]), rng.choice(["relu", "relu_sq", "gelu_tanh", "silu"])
    if op == "quantize":
        return dict(op=op, rows=size(1, 8192), cols=size(16, 8192), type=kind, tiles=rng.random() < 0.4, back=rng.random() < 0.6)
    if op == "product":
        groups = rng.choice([0, 0, rng.randint(2, 16)])
        # (fewer and smaller experts than the dense sizes would allow: each has weights of its own)
        most = 4096 if groups else 8192
        return dict(op=op, m=size(1, 8192), n=size(64, most, 8), k=size(16, most), groups=groups,
                    b=rng.choice(["tiles", "tiles", "rows"]), act=rng.choice(["none", "none", act]), c=rng.random() < 0.3)
    if op == "linear_grad":
        return dict(op=op, m=size(16, 4096), n=size(128, 4096, 8), k=size(128, 2048, 8))
    if op == "balance":
        experts = size(3, 512)
        return dict(op=op, batch=rng.choice([1, 1, rng.randint(2, 8)]), tokens=size(1, 4096), experts=experts,
                    k=rng.randint(1, min(8, experts - 1)), type=kind, scores=rng.choice(["softmax", "sigmoid"]), mask=rng.random() < 0.5)
    return dict(op=op, rows=size(1, 8192), cols=size(16, 8192), type=kind, act=act, plain=rng.random() < 0.4)


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


def lengths(case):
    """The tokens of each sequence, from the case alone: the first of several is full, the others may be short or empty."""
    r = random.Random(1000 * case["tokens"] + case["batch"])
    return [case["tokens"] if i == 0 and case["batch"] > 1 else r.randint(0, case["tokens"]) for i in range(case["batch"])]


def ceil(a, b):
    return -(-a // b)


def stored_bytes(rows, k, tiles):
    return rows * k + 4 * ceil(k, BLOCK) * (ceil(rows, BLOCK) if tiles else rows)


def work(case):
    op = case["op"]
    if op in ("quantize", "act", "act_grad"):
        r, c, e = case["rows"], case["cols"], TYPES[case["type"]].itemsize
    if op == "quantize":
        q = stored_bytes(r, c, case["tiles"]) + (stored_bytes(c, r, case["tiles"]) if case["back"] else 0)
        return {"bytes": r * c * e + q + 2 * r * c * (1 + case["back"]), "flops": 3 * r * c}
    if op == "act":
        n = 2 * (stored_bytes(r, c, False) + 2 * r * c)  # what is kept, what goes on; and their values
        return {"bytes": r * c * e + n + (r * c * e if case["plain"] else 0), "flops": 16 * r * c}
    if op == "act_grad":
        out = r * c * e if case["plain"] else stored_bytes(r, c, False) + stored_bytes(c, r, False) + 4 * r * c
        return {"bytes": r * c * e + stored_bytes(r, c, False) + out + stored_bytes(c, r, False) + 2 * r * c, "flops": 30 * r * c}
    if op == "balance":
        n, e = case["batch"] * case["tokens"], case["experts"]
        return {"bytes": 2 * n * e * TYPES[case["type"]].itemsize + 8 * n * case["k"] + n * case["mask"] + 8 * case["batch"] * e,
                "flops": 20 * n * e}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "product":
        outs = 1 if case["act"] == "none" or not case["c"] else 2
        cu = offsets(case) if case["groups"] else [0, m]
        used = sum(b > a for a, b in zip(cu, cu[1:]))
        return {"bytes": stored_bytes(m, k, False) + used * stored_bytes(n, k, case["b"] == "tiles") + 2 * m * n * (outs + case["c"]),
                "flops": 2 * m * n * k}
    return {"bytes": 2 * (m * n + m * k) + stored_bytes(k, n, True) + 2 * m * k + 2 * n * k, "flops": 4 * m * n * k}


# ---- the format


def whole_blocks(x, tiles):
    """x (..., rows, k) as (..., row blocks, rows of one, blocks, 128), padded with zeros."""
    rows, k = x.shape[-2:]
    tall = BLOCK if tiles else 1
    x = torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -rows % tall))
    return x.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, tall))


def e4m3(v):
    """v in 64 bits, at most 448 in magnitude, rounded to nearest even in e4m3: 8 steps a binade, 2^-9 at the least."""
    steps = torch.tensor([2.0**e for e in range(-9, 6)], dtype=v.dtype, device=v.device)
    step = steps[torch.frexp(v)[1].clamp(min=-5).int() + 5]  # of v in [2^(e - 1), 2^e): 2^(e - 4)
    return torch.round(v / step) * step


def factor(top):
    """What a block of largest magnitude `top` is multiplied with: quotient in 64 bits, rounded to 32, cut."""
    r = torch.full_like(top, TOP, dtype=torch.float64).div(top.double()).float().clamp(max=MOST)
    return r.view(torch.int32).bitwise_and(-(1 << 11)).view(torch.float32).double()


def to_blocks(x, tiles):
    """x (..., rows, k): its elements and scales, both in whole blocks. Products in 64 bits: a rounded one could
    pass the border between two elements, which many 16-bit values lie on."""
    b = whole_blocks(x.float(), tiles)
    r = factor(b.abs().amax((-3, -1), keepdim=True))
    return e4m3((b.double() * r).clamp(-TOP, TOP)), (1 / r).float()


def values_of(x, tiles=False):
    """x as the values in 32 bits that its codes and scales stand for."""
    v, s = to_blocks(x, tiles)
    v = (v.float() * s).flatten(-2).flatten(-3, -2)
    return v[..., : x.shape[-2], : x.shape[-1]]


def store(x, tiles=False):
    """The codes and scales of x (..., rows, k) in the storage order that the file's head describes."""
    v, s = to_blocks(x, tiles)
    rows, k = x.shape[-2:]
    codes = v.flatten(-2).flatten(-3, -2)[..., :rows, : ceil(k, 16) * 16]
    codes = codes.float().to(torch.float8_e4m3fn).view(torch.uint8)
    s = s.squeeze(-1).squeeze(-2)  # (..., rows or row blocks, blocks)
    s = torch.nn.functional.pad(s, (0, -s.shape[-1] % 4, 0, 0 if tiles else -rows % 64))
    if not tiles:
        s = s.unflatten(-1, (-1, 4)).unflatten(-3, (-1, 64)).transpose(-3, -2)
    return codes.contiguous(), s.contiguous()


def load(stored, k):
    """The values (..., rows, k) in 32 bits of codes and scales."""
    codes, s = stored
    rows = codes.shape[-2]
    if s.dim() == codes.dim() + 2:
        s = s.transpose(-3, -2).flatten(-2).flatten(-3, -2)
    else:
        s = s.repeat_interleave(BLOCK, -2)
    s = s.repeat_interleave(BLOCK, -1)[..., :rows, :k]
    return codes.view(torch.float8_e4m3fn).float()[..., :k] * s


# ---- inputs


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
        shape = (case["rows"], case["cols"])
        s["x"] = (torch.randn(*shape, generator=g, device="cuda") / 64).to(TYPES[case["type"]]) if case["tiles"] else activations(g, shape, case["type"])
    elif op == "product":
        m, n, k, G = case["m"], case["n"], case["k"], case["groups"]
        s["A"] = store(activations(g, (m, k), "f32"))
        s["B"] = store(torch.randn(*((G, n, k) if G else (n, k)), generator=g, device="cuda") / math.sqrt(k), case["b"] == "tiles")
        s["C"] = torch.randn(m, n, generator=g, device="cuda").bfloat16() if case["c"] else None
        s["cu"] = torch.tensor(offsets(case), dtype=torch.int32, device="cuda") if G else None
    elif op == "linear_grad":
        m, n, k = case["m"], case["n"], case["k"]
        s["dY"] = torch.randn(m, n, generator=g, device="cuda").bfloat16()
        s["X"] = activations(g, (m, k), "bf16")
        s["WT"] = store(torch.randn(k, n, generator=g, device="cuda") / math.sqrt(k), True)  # W^T (k, n)
    elif op == "act":
        s["x"] = activations(g, (case["rows"], case["cols"]), case["type"])
    elif op == "act_grad":
        shape = (case["rows"], case["cols"])
        s["saved"] = store(activations(g, shape, "f32"))  # the forward pass keeps it
        s["dy"] = torch.randn(*shape, generator=g, device="cuda").to(TYPES[case["type"]])
    else:
        b, t, e = case["batch"], case["tokens"], case["experts"]
        taste = torch.randn(e, generator=g, device="cuda")  # some experts are liked by most tokens
        s["logits"] = (1.5 * torch.randn(b, t, e, generator=g, device="cuda") + taste).to(TYPES[case["type"]])
        s["chosen"] = torch.topk(s["logits"].float(), case["k"], -1).indices
        at = torch.arange(t, device="cuda")
        s["mask"] = at < torch.tensor(lengths(case), device="cuda")[:, None] if case["mask"] else None
        s["grad"] = torch.full((), float(t), device="cuda")  # (the loss is scaled up, as for 16-bit gradients)
    if own:
        keep(s)
    return s


def keep(s):
    """What a program keeps beside its inputs: output buffers, operand handles and plans."""
    import gemm_epilogue_persistent_amd as gep
    case, op = s["case"], s["case"]["op"]
    new = lambda shape, t=torch.bfloat16: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    if op in ("quantize", "act", "act_grad"):
        shape, back = (case["rows"], case["cols"]), (case["cols"], case["rows"])
    if op == "quantize":
        s["q"], s["v"] = gep.fp8_empty(*shape, tiles=case["tiles"]), new(shape)
        s["qt"], s["vt"] = (gep.fp8_empty(*back, tiles=case["tiles"]), new(back)) if case["back"] else (None, None)
    elif op == "product":
        k, shape = case["k"], (case["m"], case["n"])
        s["a"], s["b"] = gep.Fp8Tensor(*s["A"], k), gep.Fp8Tensor(*s["B"], k)
        post = case["act"] != "none"
        s["D"] = new(shape) if case["c"] or not post else None
        s["P"] = new(shape) if post else None
        s["plan"] = gep.Fp8Plan(s["a"], s["b"], s["C"], s["D"], s["P"], act=case["act"], cu_seqlens_m=s["cu"])
    elif op == "linear_grad":
        m, n, k = case["m"], case["n"], case["k"]
        s["w"] = gep.Fp8Tensor(*s["WT"], n)
        s["dy_n"], s["dy_m"], s["x_m"] = gep.fp8_empty(m, n), gep.fp8_empty(n, m), gep.fp8_empty(k, m)
        s["dX"], s["dW"] = new((m, k)), new((n, k))
        s["plan_x"] = gep.Fp8Plan(s["dy_n"], s["w"], None, s["dX"])
        s["plan_w"] = gep.Fp8Plan(s["dy_m"], s["x_m"], None, s["dW"])
    elif op == "act":
        s["kept"], s["q"] = gep.fp8_empty(*shape), gep.fp8_empty(*shape)
        s["vk"], s["vq"], s["y"] = new(shape), new(shape), torch.empty_like(s["x"]) if case["plain"] else None
    elif op == "act_grad":
        s["kept"], s["yt"], s["vyt"] = gep.Fp8Tensor(*s["saved"], case["cols"]), gep.fp8_empty(*back), new(back)
        s["dx"] = torch.empty_like(s["dy"]) if case["plain"] else None
        s["q"], s["qt"] = (None, None) if case["plain"] else (gep.fp8_empty(*shape), gep.fp8_empty(*back))
        s["vq"], s["vqt"] = (None, None) if case["plain"] else (new(shape), new(back))
    else:
        b, t, e = case["batch"], case["tokens"], case["experts"]
        s["balance"], s["dlogits"] = gep.balance_empty(e, batch=b), torch.empty_like(s["logits"])
        s["work"] = new((gep.router_balance_workspace(b, t, e),), torch.uint8)


# ---- one pass


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import gemm_epilogue_persistent_amd as gep
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        gep.fp8_quantize(s["x"], out=s["q"], out_t=s["qt"])
        return {"values": gep.fp8_dequantize(s["q"], out=s["v"]),
                "values_t": gep.fp8_dequantize(s["qt"], out=s["vt"]) if case["back"] else None}
    if op == "product":
        s["plan"].run(s["a"], s["b"], s["C"], s["D"], s["P"], cu_seqlens_m=s["cu"])
        return {"d": s["D"], "post": s["P"]}
    if op == "linear_grad":
        gep.fp8_quantize(s["dY"], out=s["dy_n"], out_t=s["dy_m"])
        gep.fp8_quantize(s["X"], out_t=s["x_m"])
        s["plan_x"].run(s["dy_n"], s["w"], None, s["dX"])
        s["plan_w"].run(s["dy_m"], s["x_m"], None, s["dW"])
        return {"dw": s["dW"], "dx": s["dX"]}
    if op == "act":
        gep.fp8_act(s["x"], case["act"], saved=s["kept"], q=s["q"], y=s["y"])
        return {"saved": gep.fp8_dequantize(s["kept"], out=s["vk"]), "q": gep.fp8_dequantize(s["q"], out=s["vq"]), "y": s["y"]}
    if op == "act_grad":
        gep.fp8_act_backward(s["dy"], s["kept"], case["act"], dx=s["dx"], q=s["q"], qt=s["qt"], yt=s["yt"])
        out = {"dx": s["dx"], "yt": gep.fp8_dequantize(s["yt"], out=s["vyt"])}
        if not case["plain"]:
            out["q"], out["qt"] = gep.fp8_dequantize(s["q"], out=s["vq"]), gep.fp8_dequantize(s["qt"], out=s["vqt"])
        return out
    b = gep.router_balance(s["logits"], s["chosen"], out=s["balance"], scores=case["scores"], mask=s["mask"], coef=0.01, workspace=s["work"])
    gep.router_balance_backward(s["logits"], b, grad=s["grad"], dlogits=s["dlogits"])
    return {"counts": b.counts, "cu_seqlens": b.cu_seqlens, "dlogits": s["dlogits"], "loss": b.loss, "probs": b.probs}


def activation(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "relu_sq":
        return x.clamp(min=0).square()
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def slope(x, act):
    if act == "relu":
        return (x > 0).float()
    if act == "relu_sq":
        return 2 * x.clamp(min=0)
    if act == "silu":
        p = 1 / (1 + torch.exp(-x))
        return p * (1 + x * (1 - p))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "quantize":
        x = s["x"].float()
        return {"values": values_of(x, case["tiles"]).bfloat16(),
                "values_t": values_of(x.t(), case["tiles"]).bfloat16() if case["back"] else None}
    if op == "product":
        k, G = case["k"], case["groups"]
        a, b = load(s["A"], k), load(s["B"], k)
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
    if op == "linear_grad":
        dy, x = s["dY"].float(), s["X"].float()
        dx = values_of(dy) @ load(s["WT"], case["n"]).t()
        dw = values_of(dy.t()) @ values_of(x.t()).t()
        return {"dw": dw.bfloat16(), "dx": dx.bfloat16()}
    if op == "act":
        x = s["x"].float()
        y = activation(x, case["act"])
        return {"saved": values_of(x).bfloat16(), "q": values_of(y).bfloat16(), "y": y.to(s["x"].dtype) if case["plain"] else None}
    if op == "act_grad":
        x, dy = load(s["saved"], case["cols"]), s["dy"].float()
        dx = dy * slope(x, case["act"])
        out = {"dx": dx.to(s["dy"].dtype) if case["plain"] else None, "yt": values_of(activation(x, case["act"]).t()).bfloat16()}
        if not case["plain"]:
            out["q"], out["qt"] = values_of(dx).bfloat16(), values_of(dx.t()).bfloat16()
        return out
    b, e = case["batch"], case["experts"]
    x = s["logits"].float()
    valid = s["mask"] if s["mask"] is not None else torch.ones(x.shape[:2], dtype=torch.bool, device=x.device)
    n = valid.sum(1)
    hits = (s["chosen"] + torch.arange(b, device=x.device)[:, None, None] * e)[valid].flatten()
    counts = torch.bincount(hits, minlength=b * e).view(b, e)
    # loss = coef / B sum_b sum_e f_be P_be, f = E counts / (k n), P the mean score
    some = n.clamp(min=1)[:, None].float()
    f = counts.float() * e / (case["k"] * some)
    # (the gradient only knows differences of the counts: those to the least are exact)
    more = (counts - counts.amin(1, keepdim=True)).float() * e / (case["k"] * some)
    if case["scores"] == "softmax":
        u = torch.exp(x - x.amax(-1, keepdim=True))
    else:
        u = 1 / (1 + torch.exp(-x))
    p = u / u.sum(-1, keepdim=True) * valid[..., None]
    mean = p.double().sum(1).float() / some
    w = (more / some * (0.01 / b) * s["grad"])[:, None, :]
    d = p * (w - (p * w).sum(-1, keepdim=True))
    if case["scores"] == "sigmoid":
        d = d * (1 - u)
    total = counts.sum(0).cumsum(0)
    return {"counts": counts.int(), "cu_seqlens": torch.nn.functional.pad(total, (1, 0)).int(), "dlogits": d.to(s["logits"].dtype),
            "loss": 0.01 / b * (f * mean).sum(), "probs": mean}


# ---- the definitions in 64 bits


def representable(device):
    """Every magnitude of e4m3, ascending, so that the index's last bit is the fraction's."""
    mags = [i * 2.0**-9 for i in range(8)] + [(8 + i) * 2.0 ** (e - 3) for e in range(-6, 9) for i in range(8)]
    return torch.tensor([v for v in mags if v <= TOP], dtype=torch.float64, device=device)


def nearest(x, tiles=False):
    """x (rows, k) in 64 bits as the nearest values of the format: ties to the even code. Factor and scale are numbers of 32 bits."""
    mags = representable(x.device)
    between = (mags[1:] + mags[:-1]) / 2
    rows, k = x.shape
    tall, out = BLOCK if tiles else 1, []
    for part in x.split(max(tall, (1 << 26) // max(1, k) // BLOCK * BLOCK), 0):
        r = part.shape[0]
        b = torch.zeros(ceil(r, tall) * tall, ceil(k, BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
        b[:r, :k] = part
        b = b.reshape(-1, tall, b.shape[1] // BLOCK, BLOCK)
        top = b.abs().permute(0, 2, 1, 3).flatten(2).max(-1).values[:, None, :, None]
        f = (torch.full_like(top, TOP) / top).float().clamp(max=MOST).double()
        m, e = torch.frexp(f)
        f = torch.floor(m * 8192) / 8192 * torch.exp2(e.double())
        scale = torch.reciprocal(f).float().double()
        v = b.abs() * f
        below, above = torch.bucketize(v, between), torch.bucketize(v, between, right=True)
        at = torch.where(below == above, below, below + below % 2)  # on a border: the even one of the two
        out.append((mags[at] * scale * torch.sign(b)).reshape(-1, b.shape[2] * BLOCK)[:r, :k])
    return torch.cat(out, 0)


def decode(stored, rows, k):
    """Codes and scales of one matrix by the bit fields of the format, in 64 bits."""
    codes, s = stored
    c = codes[:, :k].long()
    e, f = (c >> 3) % 16, (c % 8).double() / 8
    v = (1.0 - 2.0 * (c >> 7).double()) * torch.where(e == 0, f * 2.0**-6, (1 + f) * torch.exp2((e - 7).double()))
    r, b = torch.arange(rows, device=c.device)[:, None], (torch.arange(k, device=c.device) // BLOCK)[None, :]
    return v * (s[r // BLOCK, b] if s.dim() == 2 else s[r // 64, b // 4, r % 64, b % 4]).double()


def act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x**3))
    if act == "none":
        return x
    y = torch.where(x > 0, x, torch.zeros_like(x))
    return y * y if act == "relu_sq" else y


def slope64(x, act):
    if act == "relu":
        return (x > 0).double()
    if act == "relu_sq":
        return 2 * torch.where(x > 0, x, torch.zeros_like(x))
    u, du = x, 1.0
    if act == "gelu_tanh":  # y = x s(u), y' = s + x s (1 - s) u'
        c = 2 * math.sqrt(2 / math.pi)
        u, du = c * (x + 0.044715 * x**3), c * (1 + 3 * 0.044715 * x * x)
    return torch.sigmoid(u) + x * torch.sigmoid(u) * torch.sigmoid(-u) * du


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        return {"values": nearest(x, case["tiles"]), "values_t": nearest(x.t().contiguous(), case["tiles"]) if case["back"] else None}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = decode(s["A"], m, k)
        x = torch.empty(m, n, dtype=torch.float64, device="cuda")
        if case["groups"]:
            cu = offsets(case)
            for g in range(case["groups"]):
                if cu[g + 1] > cu[g]:
                    x[cu[g]:cu[g + 1]] = a[cu[g]:cu[g + 1]] @ decode((s["B"][0][g], s["B"][1][g]), n, k).t()
        else:
            x = a @ decode(s["B"], n, k).t()
        if case["c"]:
            x += s["C"].double()
        post = case["act"] != "none"
        return {"d": x if case["c"] or not post else None, "post": act64(x, case["act"]) if post else None}
    if op == "linear_grad":
        m, n, k = case["m"], case["n"], case["k"]
        dy, x = s["dY"].double(), s["X"].double()
        dx = nearest(dy) @ decode(s["WT"], k, n).t()
        dw = nearest(dy.t().contiguous()) @ nearest(x.t().contiguous()).t()
        return {"dw": dw, "dx": dx}
    if op == "act":
        x = s["x"].double()
        y = act64(x, case["act"])
        return {"saved": nearest(x), "q": nearest(y), "y": y if case["plain"] else None}
    if op == "act_grad":
        x, dy = decode(s["saved"], case["rows"], case["cols"]), s["dy"].double()
        dx = dy * slope64(x, case["act"])
        out = {"dx": dx if case["plain"] else None, "yt": nearest(act64(x, case["act"]).t().contiguous())}
        if not case["plain"]:
            out["q"], out["qt"] = nearest(dx), nearest(dx.t().contiguous())
        return out
    # by the chain rule on L = coef E / B sum_b 1 / (k n^2) sum_e counts_be sum_t p_bte
    b, t, e, k = case["batch"], case["tokens"], case["experts"], case["k"]
    x = s["logits"].double()
    n = torch.tensor([float(v) for v in (lengths(case) if case["mask"] else [t] * b)], dtype=torch.float64, device="cuda")
    inside = (torch.arange(t, device="cuda")[None, :] < n[:, None]).double()
    one_hot = torch.zeros(b, t, e, dtype=torch.float64, device="cuda").scatter_add_(2, s["chosen"], torch.ones_like(s["chosen"], dtype=torch.float64))
    counts = (one_hot * inside[:, :, None]).sum(1)
    p = torch.softmax(x, -1) if case["scores"] == "softmax" else torch.sigmoid(x) / torch.sigmoid(x).sum(-1, keepdim=True)
    c = torch.where(n > 0, 0.01 * e / b / (k * n * n), torch.zeros_like(n))[:, None]
    sums = (p * inside[:, :, None]).sum(1)
    # dL / dp, less its smallest value in each sequence: p sums to one, so what is the same for all experts has no effect
    back = (c * (counts - counts.amin(1, keepdim=True)) * s["grad"].double())[:, None, :]
    d = (back - (back * p).sum(-1, keepdim=True)) * p * inside[:, :, None]
    if case["scores"] == "sigmoid":
        d = d * torch.sigmoid(-x)
    return {"counts": None, "cu_seqlens": None, "dlogits": d, "loss": (c * counts * sums).sum(),
            "probs": torch.where(n > 0, 1 / n, torch.zeros_like(n))[:, None] * sums}
