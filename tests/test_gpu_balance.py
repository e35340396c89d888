"""Per-expert counts, balance loss and its gradient against the definition in 64 bits.

Tolerances: a score is off by at most 2^-20 of itself (two exponentials of 2^-22, the sum of up to 2048 of them in a tree
of at most 32 + 6 levels, two quotients: 46 half steps of 2^-24 in all, below 2^-18.4 / 2^-24 = 48; taken as 2^-18); a mean
adds the tokens that one lane sums one after another and the tree above them; a gradient p (w - sum p w) is
off by the scores' error times |w| + sum p |w|, then half a step of its type. Counts are equal.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_persistent_amd as gep
from test_gpu_fp8 import SENTINEL, TYPES, announce

pytestmark = pytest.mark.gpu

ERR = 2.0 ** -18


def definition(x, chosen, mask, scores, coef, grad=1.0):
    """x (B, T, E) float64, on the CPU."""
    B, T, E = x.shape
    k = chosen.shape[-1]
    valid = mask if mask is not None else torch.ones(B, T, dtype=torch.bool)
    u = x if scores == "softmax" else torch.nn.functional.logsigmoid(x)
    top = u.amax(-1, keepdim=True)
    p = torch.exp(u - torch.where(top == -np.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total == 0, torch.zeros_like(p), p / total)
    p = torch.where(valid[..., None], p, torch.zeros_like(p))
    n = valid.sum(1).double()
    some = n.clamp(min=1)
    counts = torch.zeros(B, E, dtype=torch.int64)
    for b in range(B):
        ids = chosen[b][valid[b]].flatten().long()
        ids = ids[(ids >= 0) & (ids < E)]
        counts[b] = torch.bincount(ids, minlength=E)
    P = p.sum(1) / some[:, None]
    f = E * counts.double() / (k * some[:, None])
    loss = coef / max(B, 1) * (f * P).sum()
    w = grad * coef / max(B, 1) * (f / some[:, None])
    w = (w - w.amin(1, keepdim=True))[:, None, :]
    mean = (p * w).sum(-1, keepdim=True)
    d = p * (w - mean)
    size = p * (w.abs() + (p * w.abs()).sum(-1, keepdim=True))
    if scores == "sigmoid":
        d, size = d * torch.sigmoid(-x), size * torch.sigmoid(-x)
    d = torch.where(valid[..., None], d, torch.zeros_like(d))
    return dict(counts=counts, n=valid.sum(1), probs=P, loss=loss, d=d, size=torch.where(valid[..., None], size, torch.zeros_like(size)))


def check(b, d, want, kind, T, k):
    assert torch.equal(b.counts.cpu().long(), want["counts"])
    assert torch.equal(b.valid.cpu().long(), want["n"])
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), want["counts"].sum(0).cumsum(0)])
    assert torch.equal(b.cu_seqlens.cpu().long(), cu)
    err = ERR + (T + 20) * 2.0 ** -24
    probs = b.probs.double().cpu()
    assert ((probs - want["probs"]).abs() <= err * want["probs"] + 1e-38).all()
    assert abs(b.loss.double().item() - want["loss"].item()) <= (err + 2048 * 2.0 ** -24) * abs(want["loss"].item())
    if d is not None:
        f = torch.finfo(TYPES[kind])
        g = d.double().cpu()
        tol = 2 * ERR * want["size"] * (1 + f.eps) + f.eps / 2 * want["d"].abs() + f.smallest_normal * f.eps + 1e-38
        assert torch.isfinite(g).all()
        bad = (g - want["d"]).abs() > tol
        assert not bad.any(), f"{bad.sum()} of {bad.numel()} out, worst {((g - want['d']).abs() / tol).max():.4g}"


def inputs(seed, B, T, E, k, kind, masked, index):
    g = torch.Generator().manual_seed(seed)
    x = (2 * torch.randn(B, T, E, generator=g) + torch.randn(E, generator=g)).to(TYPES[kind])
    chosen = torch.topk(x.float() + torch.rand(B, T, E, generator=g), k, -1).indices.to(index)
    drop = torch.rand(B, T, k, generator=g) < 0.1  # (dropped choices: -1, or past the end)
    chosen = torch.where(drop, torch.where(torch.rand(B, T, k, generator=g) < 0.5, -1, E).to(index), chosen)
    mask = torch.rand(B, T, generator=g) < 0.7 if masked else None
    return x, chosen, mask


def run(x, chosen, mask, scores, coef=0.01, grad=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    lg, mk = x.cuda(), dev(mask)
    b = gep.router_balance(lg, chosen.cuda(), scores=scores, coef=coef, mask=mk)
    d = gep.router_balance_backward(lg, b, grad=None if grad is None else torch.tensor([grad], device="cuda"))
    return b, d


EXPERTS = [1, 2, 7, 8, 9, 16, 31, 60, 64, 100, 128, 160, 256, 257, 384, 512, 513, 1000, 1024, 1025, 2048]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("E", EXPERTS)
def test_experts(E, kind, scores):
    announce(f"balance experts {E} {kind} {scores}")
    for B, T, masked in ((1, 1, False), (1, 37, True), (3, 130, True), (1, 700, False)):
        k = min(E, 1 + (E + T) % 6)
        x, chosen, mask = inputs(E * 7 + T, B, T, E, k, kind, masked, torch.int64 if T % 2 else torch.int32)
        b, d = run(x, chosen, mask, scores, grad=64.0)
        check(b, d, definition(x.double(), chosen, mask, scores, 0.01, 64.0), kind, T, k)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,T,E,k", [(1, 20000, 64, 6), (8, 3001, 128, 8), (70, 33, 8, 2), (1, 5000, 8, 1), (2, 1500, 2048, 3)])
def test_many_tokens(B, T, E, k, scores):
    """Several workgroups a sequence, and their join."""
    announce(f"balance {B}x{T} over {E} {scores}")
    x, chosen, mask = inputs(B + T, B, T, E, k, "f32", B > 1, torch.int64)
    b, d = run(x, chosen, mask, scores, coef=1.0)
    check(b, d, definition(x.double(), chosen, mask, scores, 1.0), "f32", T, k)
    c, e = run(x, chosen, mask, scores, coef=1.0)
    assert torch.equal(b.probs, c.probs) and torch.equal(b.loss, c.loss) and torch.equal(d, e)


def test_two_dimensions_strides_and_in_place():
    announce("balance strides")
    x, chosen, mask = inputs(3, 2, 50, 60, 4, "f32", True, torch.int64)
    want = definition(x.double(), chosen, mask, "softmax", 1.0)
    buf = torch.full((2, 70, 97), SENTINEL, device="cuda")
    view = buf[:, 5:55, 7:67]
    view.copy_(x)
    out = torch.full((2, 61, 80), SENTINEL, device="cuda")
    b = gep.router_balance(view, chosen.cuda(), mask=mask.cuda())
    d = gep.router_balance_backward(view, b, dlogits=out[:, 3:53, 1:61])
    check(b, d, want, "f32", 50, 4)
    out[:, 3:53, 1:61] = SENTINEL
    assert (out == SENTINEL).all()
    # one sequence as a matrix
    b2 = gep.router_balance(view[1], chosen[1].cuda(), mask=mask[1].cuda())
    w2 = definition(x[1:].double(), chosen[1:], mask[1:], "softmax", 1.0)
    d2 = gep.router_balance_backward(view[1], b2)
    assert d2.shape == (50, 60)
    check(b2, d2.unsqueeze(0), w2, "f32", 50, 4)
    # the gradient in the place of the logits
    gep.router_balance_backward(view, b, dlogits=view)
    assert ((view.double().cpu() - want["d"]).abs() <= 2 * ERR * want["size"] + 2.0 ** -23 * want["d"].abs() + 1e-38).all()
    buf[:, 5:55, 7:67] = SENTINEL
    assert (buf == SENTINEL).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_masked_logits(scores):
    """Infinities and the type's lowest value in masked places, rows that a mask leaves empty, NaN in padding."""
    announce(f"balance masked logits {scores}")
    for kind in TYPES:
        x, chosen, mask = inputs(11, 2, 40, 24, 3, kind, True, torch.int64)
        low = torch.finfo(TYPES[kind]).min
        x[0, 3, 5:] = -float("inf")
        x[0, 4] = -float("inf")
        x[0, 5] = low
        x[0, 6, :20] = low
        x[1, 7, 1:] = -90.0
        x[1, 7, 0] = -100.0
        x[1, 8] = -1000.0
        x[1, 9, 2] = 80.0
        x[0, 10], x[1, 11] = float("nan"), float("inf")
        mask[0, 3:10], mask[1, 7:10] = True, True
        mask[0, 10], mask[1, 11] = False, False
        b, d = run(x, chosen, mask, scores, grad=1024.0)
        clean = torch.where(mask[..., None], x, torch.zeros_like(x)).double()
        clean[0, 4] = -np.inf
        check(b, d, definition(clean, chosen, mask, scores, 0.01, 1024.0), kind, 40, 3)
        assert (d[0, 4] == 0).all() and (d[0, 10] == 0).all() and (d[1, 11] == 0).all()


def test_nothing_counts():
    """A sequence without tokens, a batch of only such, no tokens at all."""
    announce("balance nothing counts")
    x, chosen, mask = inputs(2, 3, 20, 9, 2, "f32", True, torch.int64)
    mask[1] = False
    b, d = run(x, chosen, mask, "softmax")
    check(b, d, definition(x.double(), chosen, mask, "softmax", 0.01), "f32", 20, 2)
    assert (d[1] == 0).all() and (b.probs[1] == 0).all()
    b, d = run(x, chosen, torch.zeros_like(mask), "sigmoid")
    assert b.loss.item() == 0 and (d == 0).all() and not b.counts.any() and not b.cu_seqlens.any()
    for shape in ((0, 9), (3, 0, 9), (0, 5, 9)):
        out = gep.balance_empty(9, batch=shape[0] if len(shape) == 3 else 1)
        for t in (out.loss, out.counts, out.cu_seqlens, out.probs, out.valid):
            t.fill_(7)
        lg = torch.zeros(shape, device="cuda")
        gep.router_balance(lg, torch.zeros(shape[:-1] + (2,), dtype=torch.int64, device="cuda"), out=out)
        for t in (out.loss, out.counts, out.cu_seqlens, out.probs, out.valid):
            assert not t.any()
        assert gep.router_balance_backward(lg, out).shape == shape


def test_even_choice():
    """Every expert chosen equally often: the loss is coef, the gradient exactly 0; all of one: E P."""
    announce("balance even choice")
    E, T = 8, 64
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1))
    chosen = (torch.arange(T * 2) % E).view(T, 2)
    b, d = run(x, chosen, None, "softmax", coef=3.0)
    assert abs(b.loss.item() - 3.0) < 1e-5 and (d == 0).all()
    b, _ = run(x, torch.full((T, 1), 5), None, "softmax", coef=1.0)
    assert abs(b.loss.item() - E * torch.softmax(x.double(), -1)[:, 5].mean().item()) < 1e-5
    assert b.cu_seqlens.cpu().tolist() == [0] * 6 + [T] * 3
    # the same index twice counts twice
    b, _ = run(x, torch.full((T, 2), 5), None, "softmax")
    assert b.counts.cpu()[0].tolist() == [0, 0, 0, 0, 0, 2 * T, 0, 0]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_gradient_is_the_difference(scores):
    announce(f"balance differences {scores}")
    x, chosen, mask = inputs(5, 2, 6, 5, 2, "f32", True, torch.int64)
    _, d = run(x, chosen, mask, scores, coef=1.0, grad=2.0)
    x64, h = x.double(), 1e-5
    for at in np.ndindex(2, 6, 5):
        up, down = x64.clone(), x64.clone()
        up[at] += h
        down[at] -= h
        diff = 2.0 * (definition(up, chosen, mask, scores, 1.0)["loss"] - definition(down, chosen, mask, scores, 1.0)["loss"]) / (2 * h)
        # (third derivatives of order 1: 1e-10; cancellation 1e-16 / 1e-5)
        assert abs(d[at].double().item() - diff.item()) < 1e-6


def test_streams_graphs_and_buffers():
    """On a stream of its own; replayed; with buffers that are used again; the grouped products take the offsets."""
    announce("balance streams and graphs")
    x, chosen, mask = inputs(9, 4, 500, 96, 4, "bf16", True, torch.int32)
    want = definition(x.double(), chosen, mask, "sigmoid", 0.01)
    lg, ch, mk = x.cuda(), chosen.cuda(), mask.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = gep.router_balance(lg, ch, scores="sigmoid", coef=0.01, mask=mk, stream=s)
    d = gep.router_balance_backward(lg, b, stream=s)
    s.synchronize()
    check(b, d, want, "bf16", 500, 4)
    out, ws = gep.balance_empty(96, batch=4), torch.empty(gep.router_balance_workspace(4, 500, 96), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    e = torch.empty_like(lg)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gep.router_balance(lg, ch, out=out, scores="sigmoid", coef=0.01, mask=mk, workspace=ws)
        gep.router_balance_backward(lg, out, dlogits=e)
    for _ in range(4):
        ws.fill_(255)
        e.fill_(SENTINEL)
        out.probs.fill_(SENTINEL)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(out, e, want, "bf16", 500, 4)
        assert torch.equal(out.probs, b.probs) and torch.equal(e, d)
    lg.copy_(torch.zeros_like(lg))
    g.replay()
    torch.cuda.synchronize()
    check(out, e, definition(torch.zeros_like(x).double(), chosen, mask, "sigmoid", 0.01), "bf16", 500, 4)


def test_refusals():
    x = torch.zeros(2, 5, 8, device="cuda")
    c = torch.zeros(2, 5, 2, dtype=torch.int64, device="cuda")
    m = torch.ones(2, 5, dtype=torch.bool, device="cuda")
    for args, kw in (((x, c[0]), {}), ((x, c.transpose(0, 1)), {}), ((x[..., ::2], c), {}), ((x, c), dict(scores="relu")),
                     ((x, c), dict(mask=m[:1])), ((x, c), dict(mask=m.t().contiguous().t())), ((x, c), dict(out=gep.balance_empty(8))),
                     ((x, c), dict(out=gep.balance_empty(9, batch=2))), ((x, c.cpu()), {}), ((x[0, 0], c[0, 0]), {}),
                     ((x, c), dict(workspace=torch.zeros(64, device="cuda"))), ((x.cpu(), c.cpu()), {})):
        with pytest.raises(ValueError):
            gep.router_balance(*args, **kw)
    for args, kw in (((x.double(), c), {}), ((x, c.float()), {}), ((x, c), dict(mask=m.int())), ((x, c), dict(out=x))):
        with pytest.raises(TypeError):
            gep.router_balance(*args, **kw)
    for args, kw in (((x, torch.zeros(2, 5, 9, dtype=torch.int64, device="cuda")), {}), ((x, c[..., :0].contiguous()), {}),
                     ((x, c), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
                     ((x.expand(2, 5, 8)[:, :1].expand(2, 5, 8), c), {})):
        with pytest.raises(gep.GemmError):
            gep.router_balance(*args, **kw)
    b = gep.router_balance(x, c)
    for args, kw in (((x[:1], b), {}), ((x, gep.balance_empty(8, batch=2)), {}), ((x, b), dict(grad=torch.ones(2, device="cuda"))),
                     ((x, b), dict(dlogits=x[:1])), ((x, b), dict(grad=torch.ones(1, device="cuda").double()))):
        with pytest.raises(ValueError):
            gep.router_balance_backward(*args, **kw)
    with pytest.raises(TypeError):
        gep.router_balance_backward(x, b, dlogits=x.bfloat16())
    with pytest.raises(TypeError):
        gep.router_balance_backward(x, x)
    with pytest.raises(ValueError):
        gep.balance_empty(0)


@pytest.mark.parametrize("experts,dtype", [(8, torch.float32), (60, torch.bfloat16)])
def test_tokens_outermost(experts, dtype):
    """Logits (tokens, batch, experts), whose sequences alternate row by row, give what contiguous ones give."""
    announce(f"balance with alternating sequences {experts}")
    base = torch.randn(70, 3, experts, device="cuda").to(dtype)
    logits = base.transpose(0, 1)
    chosen = torch.randint(0, experts, (3, 70, 2), device="cuda")
    want = gep.router_balance(logits.contiguous(), chosen)
    got = gep.router_balance(logits, chosen)
    for name in ("loss", "probs", "counts", "cu_seqlens", "valid"):
        assert torch.equal(getattr(got, name), getattr(want, name))
    d = gep.router_balance_backward(logits, got, dlogits=torch.empty_like(base).transpose(0, 1))
    assert torch.equal(d, gep.router_balance_backward(logits.contiguous(), want))


def test_most_tokens():
    """2^31 - 1 tokens of one choice each: numbers past the last token pass 31 bits."""
    announce("balance of 2^31 - 1 tokens")
    n = 2 ** 31 - 1
    logits, chosen = torch.zeros(n, 1, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    b = gep.router_balance(logits, chosen)
    assert b.counts.item() == n and b.valid.item() == n and b.cu_seqlens.tolist() == [0, n]
    # (a workgroup adds 2^23 ones, which fp32 holds; the 256 workgroups' sums are added in four chains of 64, each sum rounded by
    # 2^-24 of itself at most and all but the last one's exact; P, f and their product are rounded once each)
    assert abs(b.loss.item() - 1) <= 2.0 ** -20
    logits.fill_(1)
    gep.router_balance_backward(logits, b, dlogits=logits)
    assert not logits.any()


@pytest.mark.parametrize("E,T", [(8, 1024), (8, 1025), (8, 4096), (8, 4097), (64, 128), (64, 129), (64, 512), (64, 513), (512, 17), (512, 64),
                                 (512, 65), (600, 16), (600, 17)])
def test_one_workgroup(E, T):
    """Around the numbers of tokens up to which one workgroup of 256 or 1024 threads takes them."""
    announce(f"balance one workgroup {T} over {E}")
    x, chosen, mask = inputs(E + T, 1, T, E, 3, "f32", True, torch.int32)
    b, d = run(x, chosen, mask, "softmax", coef=1.0)
    check(b, d, definition(x.double(), chosen, mask, "softmax", 1.0), "f32", T, 3)
