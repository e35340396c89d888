"""The FP8 operators, the checkpoints and the router together (examples/fp8_experts.py), on streams, in graphs and at
large sizes.

Tolerance of the layers. An e4m3 element is off by at most 2^-4 of itself, in the root mean square by 2^-4 / sqrt(3) =
0.036 at the widest (values far below their block's largest, which are off by more of themselves, weigh little in
a norm). The errors of a product's terms are independent of their signs, so a product whose operands are off by ea and eb in
the Frobenius norm is off by sqrt(ea^2 + eb^2): 0.051 for one. y passes through two products and the activation, whose
slope is below 1.1: sqrt(2) x 0.051 x 1.1 = 0.079; a gradient through at most three, with the activation's
derivative taken at a point that is itself off by 0.051 + 0.036: below 0.13. 0.15 covers them.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp8_ref as R
import gemm_epilogue_persistent_amd as gep
from test_gpu_fp8 import announce

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layers():
    spec = importlib.util.spec_from_file_location("fp8_experts", os.path.join(ROOT, "examples", "fp8_experts.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,d,f", [(1, 256, 512), (77, 264, 520), (300, 512, 1024)])
def test_mlp(layers, tokens, d, f):
    announce(f"fp8 MLP {tokens} x {d} x {f}")
    t, dy, _ = layers.inputs(tokens, d, f, 0, seed=tokens)
    layer = layers.Fp8Mlp(t["w1"], t["w2"])
    y, saved = layer.forward(t["x"])
    grads = layer.backward(dy, saved)
    leaves = {k: v.float().cpu().requires_grad_() for k, v in t.items()}
    want = layers.reference_mlp(**leaves)
    want.backward(dy.float().cpu())
    assert layers.relative(y.cpu(), want.detach()) <= 0.15
    for name, got in zip(("x", "w1", "w2"), grads):
        assert layers.relative(got.cpu(), leaves[name].grad) <= 0.15, name


@pytest.mark.parametrize("tokens,d,f,experts,k", [(3, 128, 256, 4, 2), (130, 264, 392, 8, 2), (200, 256, 512, 5, 1)])
def test_experts(layers, tokens, d, f, experts, k):
    """The router's offsets lead the grouped products, its loss and gradient beside them."""
    announce(f"fp8 experts {tokens} x {d} x {f} over {experts}")
    t, dy, logits = layers.inputs(tokens, d, f, experts, seed=tokens)
    layer = layers.Fp8Experts(t["w1"], t["w2"], k)
    y, loss, saved = layer.forward(t["x"], logits)
    grads = layer.backward(dy, torch.full((), 2.0, device="cuda"), saved)
    leaves = {n: v.float().cpu().requires_grad_() for n, v in dict(t, logits=logits).items()}
    want, balance = layers.reference_experts(k=k, **leaves)
    ((want * dy.float().cpu()).sum() + 2 * balance).backward()
    assert layers.relative(y.cpu(), want.detach()) <= 0.15
    assert abs(loss.item() - balance.item()) <= 1e-5 * balance.item()
    for name, got in zip(("x", "w1", "w2"), grads):
        assert layers.relative(got.cpu(), leaves[name].grad) <= 0.15, name
    assert layers.relative(grads[3].cpu(), leaves["logits"].grad) <= 1e-4
    counts = torch.bincount(torch.topk(logits.cpu(), k, -1).indices.flatten(), minlength=experts)
    assert torch.equal(saved[1].cu_seqlens.cpu().long()[1:], counts.cumsum(0))


def test_graph_replays(layers):
    """A layer's passes captured into a graph: every replay, with eager work between them and new inputs, equals the
    eager result bit for bit."""
    announce("fp8 graph")
    t, dy, _ = layers.inputs(130, 256, 512, 0, seed=9)
    layer = layers.Fp8Mlp(t["w1"], t["w2"])
    et, edy, logits = layers.inputs(64, 256, 384, 6, seed=3)
    experts = layers.Fp8Experts(et["w1"], et["w2"], 2)
    x, g, ex, eg, el = t["x"].clone(), dy.clone(), et["x"].clone(), edy.clone(), logits.clone()
    one = torch.ones((), device="cuda")
    deep, deep_b = gep.fp8_quantize(torch.randn(40, 4096, device="cuda")), gep.fp8_quantize(torch.randn(64, 4096, device="cuda"), tiles=True)
    D = torch.empty(40, 64, device="cuda")
    plan = gep.Fp8Plan(deep, deep_b, None, D, tile="32", split=4)
    assert plan.workspace_bytes > 0

    def both():
        y, saved = layer.forward(x)
        grads = layer.backward(g, saved)
        z, loss, kept = experts.forward(ex, el)
        more = experts.backward(eg, one, kept)
        plan.run(deep, deep_b, None, D)
        return (y, *grads, z, loss, *more, D)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (9, 10, 11):
        new, dnew, _ = layers.inputs(130, 256, 512, 0, seed=seed)
        enew, ednew, lnew = layers.inputs(64, 256, 384, 6, seed=seed)
        x.copy_(new["x"])
        g.copy_(dnew)
        ex.copy_(enew["x"])
        eg.copy_(ednew)
        el.copy_(lnew)
        want = [v.clone() for v in both()]
        D.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(out, want):
            assert torch.equal(got, w)


def test_other_stream_allocations():
    """What a call on a given stream allocates is ordered with that stream, whatever the current one still
    has to do."""
    announce("fp8 allocations on another stream")
    x = torch.randn(200, 512, device="cuda")
    b = gep.fp8_quantize(torch.randn(64, 512, device="cuda"), tiles=True)
    logits, chosen = torch.randn(3000, 16, device="cuda"), torch.randint(0, 16, (3000, 2), device="cuda")
    want_q = gep.fp8_quantize(x)
    want_v, want_y, want_d = gep.fp8_dequantize(want_q), gep.fp8_act(x, "silu"), gep.fp8_gemm(want_q, b)
    want_b = gep.router_balance(logits, chosen)
    want_g = gep.router_balance_backward(logits, want_b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(int(5e7))  # the current stream is busy for a while
    q = gep.fp8_quantize(x, stream=s)
    v, y, d = gep.fp8_dequantize(q, stream=s), gep.fp8_act(x, "silu", stream=s), gep.fp8_gemm(q, b, stream=s)
    bal = gep.router_balance(logits, chosen, stream=s)
    g = gep.router_balance_backward(logits, bal, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(q.codes, want_q.codes) and torch.equal(q.scales, want_q.scales)
    for got, want in ((v, want_v), (y, want_y), (d, want_d), (g, want_g), (bal.probs, want_b.probs), (bal.cu_seqlens, want_b.cu_seqlens)):
        assert torch.equal(got, want)


def test_plan_workspaces_overlap():
    """Runs of one plan on two streams at once, and two graphs of it replayed at once, after the plan is gone."""
    announce("fp8 plan on two streams and in two graphs")
    a = [gep.fp8_quantize(torch.randn(40, 4096, device="cuda")) for _ in range(2)]
    b = gep.fp8_quantize(torch.randn(64, 4096, device="cuda"), tiles=True)
    want, got = [torch.empty(40, 64, device="cuda") for _ in range(2)], [torch.empty(40, 64, device="cuda") for _ in range(2)]
    plan = gep.Fp8Plan(a[0], b, None, want[0], tile="32", split=8)
    for i in range(2):
        plan.run(a[i], b, None, want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(50):
        for i in range(2):
            plan.run(a[i], b, None, got[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            for _ in range(20):
                plan.run(a[i], b, None, got[i])
    del plan
    for _ in range(3):
        for t in got:
            t.fill_(-1)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        for i in range(2):
            assert torch.equal(got[i], want[i])


def test_balance_graphs_side_by_side():
    """Two graphs of the balance loss, each with what it allocated, replayed at once."""
    announce("balance in two graphs")
    logits = [torch.randn(4000, 64, device="cuda") for _ in range(2)]
    chosen = [torch.topk(t, 4, -1).indices for t in logits]
    want = [gep.router_balance(*a) for a in zip(logits, chosen)]
    streams, graphs, got = [torch.cuda.Stream() for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)], [None, None]
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            for _ in range(20):
                got[i] = gep.router_balance(logits[i], chosen[i])
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for name in ("loss", "probs", "counts", "cu_seqlens"):
                assert torch.equal(getattr(got[i], name), getattr(want[i], name))


def sampled(x, rows, cols, q, qt):
    """Codes and scales of some rows and columns of a large matrix against the definition's."""
    nb, nbt = -(-x.shape[1] // 128), -(-x.shape[0] // 128)
    for m, t, some, blocks in ((q, x, rows, nb), (qt, x.t(), cols, nbt)):
        for r in some:
            codes, scales = R.quantize(t[r:r + 1].double().cpu().numpy())
            assert np.array_equal(m.codes[r:r + 1].cpu().numpy(), codes)
            b = np.arange(blocks)
            assert np.array_equal(m.scales[r // 64].cpu().numpy()[b // 4, r % 64, b % 4], scales[0])


def test_large_matrix():
    """More than 2^31 bytes of codes in both directions; the same through a checkpoint."""
    announce("fp8 quantise 70001 x 32784 bf16")
    rows, cols = 70001, 32784
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    q, qt = gep.fp8_empty(rows, cols), gep.fp8_empty(cols, rows)
    gep.fp8_quantize(x, out=q, out_t=qt)
    sampled(x, (0, 1, 64, 35000, 65530, 69999, 70000), (0, 5, 16384, 32767, 32783), q, qt)
    kept, r2, yt = gep.fp8_empty(rows, cols), gep.fp8_empty(rows, cols), gep.fp8_empty(cols, rows)
    gep.fp8_act(x, "relu", saved=kept, q=r2)
    assert torch.equal(kept.codes, q.codes) and torch.equal(kept.scales, q.scales)
    dx = torch.empty_like(x)
    gep.fp8_act_backward(x, kept, "relu", dx=dx, yt=yt)
    for r in (0, 35000, 70000):
        v = gep.fp8_dequantize(gep.Fp8Tensor(kept.codes[r:r + 1], kept.scales[r // 64:r // 64 + 1].roll(-(r % 64), 2).contiguous(), cols),
                               dtype=torch.float32)
        assert torch.equal(dx[r:r + 1], torch.where(v > 0, x[r:r + 1], torch.zeros_like(x[r:r + 1])))


def test_many_rows_and_columns():
    """Very long and very narrow matrices: the last rows and tiles of the last launch."""
    announce("fp8 quantise 2^24 + 5 x 16 and 1 x 2^28 + 77")
    x = torch.empty((1 << 24) + 5, 16, dtype=torch.bfloat16, device="cuda").normal_()
    q = gep.fp8_quantize(x)
    v = gep.fp8_dequantize(q, dtype=torch.float32)
    top = x.float().abs().amax(1, keepdim=True)
    assert ((v - x.float()).abs() <= 2.0 ** -4 * x.float().abs() + 2.0 ** -10 / 447 * top).all()
    y = torch.empty(1, (1 << 28) + 77, device="cuda").uniform_(-3, 3)
    got = gep.fp8_empty(y.shape[1], 1)
    gep.fp8_quantize(y, out_t=got)
    want = gep.fp8_quantize(y.view(-1, 1))
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
