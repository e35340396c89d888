"""The MX operators and the norm together (examples/mx_mlp.py), on streams and in graphs.

Tolerance of the layer. An element of an e4m3 block is off by at most 2^-4 of itself, an e2m1 one by at
most 1/4 of itself, or by half the spacing of the smallest values, 2^-10 and 1/4 of the block's scale.
The errors of a product's K terms are independent of the terms' signs, so in the Frobenius norm a
product with operands off by ea and eb (relative, root mean square, uniform in half a step: 1 / sqrt(3)
of the largest) is off by sqrt(ea^2 + eb^2) of a product of unrelated factors. e4m3: ea = 2^-4 / sqrt(3) =
0.036 at the widest, so one product 0.051; y is a residual plus two products in a row (0.072 of a
term smaller than y), a gradient passes through at most three (0.088) with the activation's derivative,
which a perturbed argument changes by at most 1.1 of it. 0.15 covers them.
"""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import gemm_epilogue_persistent_amd as gep

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def announce(name):
    print(f"[case] {name}", flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def mlp():
    spec = importlib.util.spec_from_file_location("mx_mlp", os.path.join(ROOT, "examples", "mx_mlp.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,d,f", [(1, 256, 512), (77, 264, 520), (300, 512, 1024)])
def test_layer(mlp, tokens, d, f):
    announce(f"layer {tokens} x {d} x {f}")
    t, dy = mlp.inputs(tokens, d, f, seed=tokens)
    layer = mlp.MxMlp(t["weight"], t["w1"], t["w2"])
    y, saved = layer.forward(t["x"], t["residual"], save=True)
    grads = layer.backward(dy, saved)
    leaves = {k: v.float().cpu().requires_grad_() for k, v in t.items()}
    want = mlp.reference(**leaves)
    want.backward(dy.float().cpu())
    assert mlp.relative(y.cpu(), want.detach()) <= 0.15
    for name, got in zip(("x", "weight", "w1", "w2"), grads):
        assert mlp.relative(got.cpu(), leaves[name].grad) <= 0.15, name
    assert torch.equal(leaves["x"].grad, leaves["residual"].grad)


def test_experts(mlp):
    """A grouped layer gives each expert's rows what its own dense product gives, up to the order of
    the sums (2^-23 of the terms' magnitudes and half a bf16 step each)."""
    announce("experts")
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(150, 384, generator=g, device="cuda").bfloat16()
    w = torch.randn(4, 264, 384, generator=g, device="cuda").bfloat16()
    weight = torch.ones(384, device="cuda", dtype=torch.bfloat16)
    off = [0, 70, 70, 71, 150]
    experts = mlp.MxExperts(weight, w)
    got = experts.forward(x, torch.tensor(off, dtype=torch.int32, device="cuda"))
    n = torch.empty_like(x)
    q = gep.mx_empty(150, 384, "e4m3")
    gep.rmsnorm(x, weight, y=n, q=q)
    v = gep.mx_dequantize(q, dtype=torch.float32).double().cpu()
    for i in range(4):
        rows = slice(off[i], off[i + 1])
        wv = gep.mx_dequantize(experts.w1.group(i), dtype=torch.float32).double().cpu()
        pre = v[rows] @ wv.t()
        # (32 x 2^-13 of the largest product of each block of 32, see test_gpu_mx.py)
        blocks = v[rows].abs().unflatten(1, (12, 32)).amax(-1) @ wv.abs().unflatten(1, (12, 32)).amax(-1).t()
        bound = 385 * 2.0 ** -24 * (v[rows].abs() @ wv.abs().t()) + 32 * 2.0 ** -13 * blocks
        want = pre * torch.sigmoid(pre)
        err = (got[rows].double().cpu() - want).abs()
        assert (err <= (1.1 * bound + 2.0 ** -20 * (want.abs() + pre.abs())) * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()).all()


def test_graph_replays(mlp):
    """A layer's passes captured into a graph: every replay, with eager work between them and new inputs,
    equals the eager result bit for bit."""
    announce("graph")
    t, dy = mlp.inputs(130, 256, 512, seed=9)
    layer = mlp.MxMlp(t["weight"], t["w1"], t["w2"])
    x, r, g = t["x"].clone(), t["residual"].clone(), dy.clone()
    # (K split over workgroups too: its plan owns a workspace)
    a, b = gep.mx_quantize(t["w1"][:40], "e4m3"), gep.mx_quantize(t["w1"][40:104], "e2m1")
    D = torch.empty(40, 64, device="cuda")
    deep = gep.mx_quantize(torch.randn(40, 4096, device="cuda"), "e4m3")
    deep_b = gep.mx_quantize(torch.randn(64, 4096, device="cuda"), "e2m1")
    plan = gep.MxPlan(deep, deep_b, None, D, tile="32", split=4)
    assert plan.workspace_bytes > 0

    def both():
        y, saved = layer.forward(x, r, save=True)
        grads = layer.backward(g, saved)
        plan.run(deep, deep_b, None, D)
        return (y, *grads, gep.mx_gemm(a, b), D)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (9, 10, 11):
        new, dnew = mlp.inputs(130, 256, 512, seed=seed)
        x.copy_(new["x"])
        r.copy_(new["residual"])
        g.copy_(dnew)
        want = [v.clone() for v in both()]
        D.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(out, want):
            assert torch.equal(got, w)


def test_other_stream_allocations():
    """What a call on a given stream allocates is ordered with that stream, whatever the current one still
    has to do."""
    announce("allocations on another stream")
    x = torch.randn(200, 512, device="cuda")
    w = torch.ones(512, device="cuda")
    b = gep.mx_quantize(torch.randn(64, 512, device="cuda"), "e4m3")
    want_q = gep.mx_quantize(x, "e4m3")
    want_v, want_n = gep.mx_dequantize(want_q), gep.rmsnorm(x, w)
    want_d = gep.mx_gemm(want_q, b)
    rstd = torch.rand(200, device="cuda") + 0.5
    want_dx, want_dw = gep.rmsnorm_backward(x, x, w, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(int(5e7))  # the current stream is busy for a while
    q = gep.mx_quantize(x, "e4m3", stream=s)
    v, n = gep.mx_dequantize(q, stream=s), gep.rmsnorm(x, w, stream=s)
    d = gep.mx_gemm(q, b, stream=s)
    dx, dw = gep.rmsnorm_backward(x, x, w, rstd, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(q.codes, want_q.codes) and torch.equal(q.scales, want_q.scales)
    for got, want in ((v, want_v), (n, want_n), (d, want_d), (dx, want_dx), (dw, want_dw)):
        assert torch.equal(got, want)


def test_plan_workspace_on_other_streams():
    """A plan's workspace that another stream used is not handed out again before that stream is done."""
    announce("workspace on other streams")
    a = gep.mx_quantize(torch.randn(40, 4096, device="cuda"), "e4m3")
    b = gep.mx_quantize(torch.randn(64, 4096, device="cuda"), "e4m3")
    D, E = torch.empty(40, 64, device="cuda"), torch.empty(40, 64, device="cuda")
    plan = gep.MxPlan(a, b, None, D, tile="32", split=8)
    plan.run(a, b, None, D)
    nbytes = plan.workspace_bytes
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(int(2e7))
        plan.run(a, b, None, E)  # the current stream
    plan.run(a, b, None, E, stream=s)
    address = plan._workspace.data_ptr()
    del plan
    other = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    assert other.data_ptr() != address
    torch.cuda.synchronize()
    assert torch.equal(D, E)


def test_many_narrow_rows():
    """More rows than one launch of the norm takes; the last ones are right and nothing is left out."""
    announce("norm of 2^24 + 5 rows of 8")
    rows, cols = (1 << 24) + 5, 8
    x = torch.randn(rows, cols, device="cuda").half()
    w = torch.linspace(0.5, 1.5, cols, device="cuda").half()
    y, rstd = torch.full_like(x, 77.0), torch.full((rows,), 77.0, device="cuda")
    gep.rmsnorm(x, w, y=y, rstd=rstd)
    f = x.double()
    r = torch.rsqrt(f.square().mean(1) + 1e-5)
    # rstd: half an fp32 step of the rounded 64-bit value and its own 2^-50; y: half a step of f16
    assert ((rstd.double() - r).abs() <= 2.0 ** -23 * r).all()
    want = f * r[:, None] * w.double()
    assert ((y.double() - want).abs() <= 2.0 ** -11 * want.abs() * (1 + 2.0 ** -10) + 2.0 ** -25).all()


def test_many_columns_transposed():
    """More tiles than one launch of the transposed quantiser takes: the codes of x^T from x and from x^T."""
    announce("transposed quantiser, 2^29 + 77 columns")
    cols = (1 << 29) + 77
    x = torch.empty(1, cols, device="cuda").uniform_(-3, 3)
    got = gep.mx_empty(cols, 1, "e2m1")
    gep.mx_quantize(x, "e2m1", out=got, transpose=True)
    want = gep.mx_quantize(x.view(cols, 1), "e2m1")
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_norm_of_large_and_small_values(kind):
    """Squares past fp32's range and below it: y is still the quotient (rstd to half a step, y to 2^-22
    and half a step of its type), while rstd itself is an fp32 number."""
    announce(f"norm of large and small values {kind}")
    g = torch.Generator().manual_seed(2)
    x = torch.randn(6, 300, generator=g, dtype=torch.float64)
    x *= torch.tensor([1e25, 1e30, 1e20, 1e-20, 1e-25, 1e-30], dtype=torch.float64)[:, None]
    x = x.to(kind)
    w = torch.ones(300, dtype=kind)
    rstd = torch.empty(6, device="cuda")
    y = gep.rmsnorm(x.cuda(), w.cuda(), eps=0.0, rstd=rstd).double().cpu().numpy()
    f = x.double().numpy()
    r = 1 / np.sqrt((f ** 2).mean(1))
    half = torch.finfo(kind).eps / 2
    assert (np.abs(rstd.double().cpu().numpy() - r) <= 2.0 ** -23 * r).all()
    want = f * r[:, None]
    assert (np.abs(y - want) <= (half + 2.0 ** -22) * np.abs(want) + torch.finfo(kind).tiny).all()


def test_norm_output_refusals():
    x, w, r = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda"), torch.zeros(4, 64, device="cuda")
    h = torch.empty_like(x)
    for kw in (dict(y=x), dict(residual=r, y=r), dict(residual=r, h=h, y=h)):
        with pytest.raises(gep.GemmError):
            gep.rmsnorm(x, w, **kw)


def test_plan_workspace_of_a_busy_stream():
    """A plan made on a stream that still writes into a block freed there runs on another stream: its
    partial sums lie elsewhere."""
    announce("workspace beside a busy stream")
    a = gep.mx_quantize(torch.randn(40, 4096, device="cuda"), "e4m3")
    b = gep.mx_quantize(torch.randn(64, 4096, device="cuda"), "e4m3")
    D, E = torch.empty(40, 64, device="cuda"), torch.empty(40, 64, device="cuda")
    nbytes = 8 * 40 * 64 * 4
    gep.MxPlan(a, b, None, D, tile="32", split=8).run(a, b, None, D)
    s = torch.cuda.Stream()
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(int(2e7))
    block.fill_(255)
    del block
    plan = gep.MxPlan(a, b, None, D, tile="32", split=8)
    assert plan.workspace_bytes == nbytes
    for _ in range(50):
        plan.run(a, b, None, E, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(D, E)


def test_plan_workspaces_overlap():
    """Runs of one plan on two streams at once, and two graphs of it replayed at once, after the plan is gone."""
    announce("one plan on two streams and in two graphs")
    a = [gep.mx_quantize(torch.randn(40, 4096, device="cuda"), "e4m3") for _ in range(2)]
    b = gep.mx_quantize(torch.randn(64, 4096, device="cuda"), "e4m3")
    want, got = [torch.empty(40, 64, device="cuda") for _ in range(2)], [torch.empty(40, 64, device="cuda") for _ in range(2)]
    plan = gep.MxPlan(a[0], b, None, want[0], tile="32", split=8)
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
