"""Layers whose products run on 8-bit operands with a scale per 128 values, as in a training step: a dense MLP and a
mixture of experts with its router's balance loss. What the backward pass needs of the activations is kept in those 8 bits.

    MLP       y = W2 silu(W1 x)
    experts   y_t = sum over the k experts e that token t chose of g_te W2_e silu(W1_e x_t),
              loss = the balance loss of the choice

Run it with `python examples/fp8_experts.py` from the repository's root (an MI355X is needed): the error of
the outputs and of each gradient against fp32 arithmetic on the unquantised values, and the time of each pass.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_epilogue_persistent_amd as gep  # noqa: E402


def both_ways(w):
    """A weight (n, k) as tiles, and its transpose: the operands of the forward and of the backward product."""
    q, t = gep.fp8_empty(*w.shape, tiles=True, device=w.device), gep.fp8_empty(*w.shape[::-1], tiles=True, device=w.device)
    gep.fp8_quantize(w, out=q, out_t=t)
    return q, t


class Fp8Mlp:
    """w1 (f, d) and w2 (d, f) in bf16."""

    def __init__(self, w1, w2):
        (self.w1, self.w1t), (self.w2, self.w2t) = both_ways(w1), both_ways(w2)

    def forward(self, x):
        """(y, what backward takes: 8 bits a value of x and of the first product)."""
        m, d, f = *x.shape, self.w1.rows
        qx, kept, qa = gep.fp8_empty(m, d), gep.fp8_empty(m, f), gep.fp8_empty(m, f)
        gep.fp8_quantize(x, out=qx)
        gep.fp8_act(gep.fp8_gemm(qx, self.w1), "silu", saved=kept, q=qa)
        return gep.fp8_gemm(qa, self.w2), (qx, kept)

    def backward(self, dy, saved):
        """Gradients of x, w1 and w2 from dy (tokens, d): four products, each on 8-bit operands."""
        qx, kept = saved
        m, d, f = *dy.shape, self.w1.rows
        q, qt = gep.fp8_empty(m, d), gep.fp8_empty(d, m)
        gep.fp8_quantize(dy, out=q, out_t=qt)
        da = gep.fp8_gemm(q, self.w2t)
        dq, dqt, at, xt = gep.fp8_empty(m, f), gep.fp8_empty(f, m), gep.fp8_empty(f, m), gep.fp8_empty(d, m)
        gep.fp8_act_backward(da, kept, "silu", q=dq, qt=dqt, yt=at)
        gep.fp8_act_backward(None, qx, "none", yt=xt)  # the input's blocks along the tokens
        return gep.fp8_gemm(dq, self.w1t), gep.fp8_gemm(dqt, xt), gep.fp8_gemm(qt, at)


class Fp8Experts:
    """w1 (experts, f, d) and w2 (experts, d, f) in bf16; each token goes to k experts."""

    def __init__(self, w1, w2, k, coef=0.01):
        self.k, self.coef = k, coef
        n, f, d = w1.shape
        new = lambda rows, cols: gep.fp8_empty(rows, cols, tiles=True, groups=n, device=w1.device)  # noqa: E731
        self.w1, self.w1t, self.w2, self.w2t = new(f, d), new(d, f), new(d, f), new(f, d)
        for e in range(n):
            gep.fp8_quantize(w1[e], out=self.w1.group(e), out_t=self.w1t.group(e))
            gep.fp8_quantize(w2[e], out=self.w2.group(e), out_t=self.w2t.group(e))

    def forward(self, x, logits):
        """(y, balance loss, what backward takes). x (tokens, d) bf16, logits (tokens, experts) fp32."""
        t, k = x.shape[0], self.k
        gate, chosen = torch.topk(torch.softmax(logits, -1), k, -1)
        balance = gep.router_balance(logits, chosen, coef=self.coef)
        cu = balance.cu_seqlens
        order = torch.argsort(chosen.flatten(), stable=True)  # the rows in the order of their experts
        place = torch.argsort(order).view(t, k)               # where a token's rows went
        rows = t * k
        qx, kept, qa = gep.fp8_empty(rows, x.shape[1]), gep.fp8_empty(rows, self.w1.rows), gep.fp8_empty(rows, self.w1.rows)
        gep.fp8_quantize(x[order // k], out=qx)
        gep.fp8_act(gep.fp8_gemm(qx, self.w1, cu_seqlens_m=cu), "silu", saved=kept, q=qa)
        out = gep.fp8_gemm(qa, self.w2, cu_seqlens_m=cu)
        y = (out[place].float() * gate[..., None]).sum(1).to(x.dtype)
        return y, balance.loss, (logits, balance, gate, order, place, qx, kept)

    def backward(self, dy, dloss, saved):
        """Gradients of x, w1, w2 and, of the balance loss, the logits (the gates are taken as they are). The experts' weight
        gradients, which sum over runs of tokens of any length, are 16-bit products."""
        logits, balance, gate, order, place, qx, kept = saved
        k, cu, n = self.k, balance.cu_seqlens, balance.experts
        rows, f, d = kept.rows, kept.k, dy.shape[1]
        dout = (dy[order // k].float() * gate.flatten()[order, None]).to(dy.dtype)
        da = gep.fp8_gemm(gep.fp8_quantize(dout), self.w2t, cu_seqlens_m=cu)
        dpre, a, dq = torch.empty_like(da), torch.empty_like(da), gep.fp8_empty(rows, f)
        gep.fp8_act_backward(da, kept, "silu", dx=dpre, q=dq, y=a)
        dx = gep.fp8_gemm(dq, self.w1t, cu_seqlens_m=cu)[place].float().sum(1).to(dy.dtype)
        dw1, dw2 = torch.empty(n, f, d, dtype=dy.dtype, device=dy.device), torch.empty(n, d, f, dtype=dy.dtype, device=dy.device)
        for w, left, right in ((dw1, dpre, gep.fp8_dequantize(qx)), (dw2, dout, a)):
            gep.Plan(left.t(), right.t(), None, w, cu_seqlens_k=cu).run(left.t(), right.t(), None, w, cu_seqlens_k=cu)
        return dx, dw1, dw2, gep.router_balance_backward(logits, balance, grad=dloss)


def reference_mlp(x, w1, w2):
    return torch.nn.functional.silu(x @ w1.t()) @ w2.t()


def reference_experts(x, logits, w1, w2, k, coef=0.01):
    """(y, balance loss) in fp32 with torch's own operations and gradients; the gates without one."""
    p = torch.softmax(logits, -1)
    gate, chosen = torch.topk(p.detach(), k, -1)
    full = torch.zeros_like(p).scatter(1, chosen, gate)
    h = torch.nn.functional.silu(torch.einsum("td,efd->tef", x, w1))
    y = torch.einsum("tef,edf,te->td", h, w2, full)
    counts = torch.zeros_like(p).scatter(1, chosen, 1.0).sum(0)
    t, e = p.shape
    return y, coef * (e * counts / (k * t) * p.mean(0)).sum()


def inputs(tokens, d, f, experts, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()  # noqa: E731
    lead = (experts,) if experts else ()
    t = dict(x=new(tokens, d), w1=new(*lead, f, d, scale=d ** -0.5), w2=new(*lead, d, f, scale=f ** -0.5))
    return t, new(tokens, d), torch.randn(tokens, max(experts, 1), generator=g, device="cuda")


def relative(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


def timed(call, n=20):
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        call()
    start.record()
    for _ in range(n):
        call()
    end.record()
    end.synchronize()
    return start.elapsed_time(end) / n * 1e3


def main(tokens=4096, d=2048, f=4096, experts=8, k=2):
    t, dy, _ = inputs(tokens, d, f, 0)
    layer = Fp8Mlp(t["w1"], t["w2"])
    y, saved = layer.forward(t["x"])
    grads = layer.backward(dy, saved)
    leaves = {n: v.float().requires_grad_() for n, v in t.items()}
    want = reference_mlp(**leaves)
    want.backward(dy.float())
    print(f"MLP      y relative error {relative(y, want.detach()):.4f}, " +
          ", ".join(f"d{n} {relative(g, leaves[n].grad):.4f}" for n, g in zip(("x", "w1", "w2"), grads)))
    print(f"MLP      {tokens} tokens: forward {timed(lambda: layer.forward(t['x'])):.0f} us, "
          f"backward {timed(lambda: layer.backward(dy, saved)):.0f} us")
    t, dy, logits = inputs(256, 512, 512, experts)
    small = Fp8Experts(t["w1"], t["w2"], k)
    y, loss, saved = small.forward(t["x"], logits)
    grads = small.backward(dy, torch.ones((), device="cuda"), saved)
    leaves = {n: v.float().requires_grad_() for n, v in dict(t, logits=logits).items()}
    want, balance = reference_experts(k=k, **leaves)
    ((want * dy.float()).sum() + balance).backward()
    print(f"experts  y relative error {relative(y, want.detach()):.4f}, loss {loss.item():.6f} ({balance.item():.6f}), " +
          ", ".join(f"d{n} {relative(g, leaves[n].grad):.4f}" for n, g in zip(("x", "w1", "w2", "logits"), grads)))
    t, dy, logits = inputs(tokens, d, f, experts)
    layer = Fp8Experts(t["w1"], t["w2"], k)
    saved = layer.forward(t["x"], logits)[2]
    one = torch.ones((), device="cuda")
    print(f"experts  {tokens} tokens, {k} of {experts} each: forward {timed(lambda: layer.forward(t['x'], logits)):.0f} us, "
          f"backward {timed(lambda: layer.backward(dy, one, saved)):.0f} us")


if __name__ == "__main__":
    main()
