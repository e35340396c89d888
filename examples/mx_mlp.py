"""A residual MLP layer on block-scaled (MX) operands: the fused RMS norm, the quantiser and the
products run together as in a model's layer, for prompts, for single tokens and for training.

    h = x + residual      n = h / rms(h) * weight      y = h + W2 silu(W1 n)

Run it with `python examples/mx_mlp.py` from the repository's root (an MI355X is needed): the
error of the outputs and of each gradient against fp32 arithmetic on the unquantised values, and
the time of each pass.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gemm_epilogue_persistent_amd as gep  # noqa: E402


class MxMlp:
    """Weights w1 (f, d) and w2 (d, f) in bf16, laid out once as MX matrices in the order that each
    product reads them. weight: the norm's, (d,) bf16. fmt: the activations' and gradients' format;
    weight_fmt: the weights' (e2m1 for serving in 4 bits)."""

    def __init__(self, weight, w1, w2, fmt="e4m3", weight_fmt="e4m3", eps=1e-5, training=True):
        self.weight, self.fmt, self.eps = weight, fmt, eps
        self.w1 = gep.mx_quantize(w1, weight_fmt)
        self.w2 = gep.mx_quantize(w2, weight_fmt)
        if training:
            self.w1t = gep.mx_quantize(w1, weight_fmt, transpose=True)  # (d, f): blocks along f
            self.w2t = w2.t().contiguous()  # (f, d): the product that ends in the activation's derivative runs in bf16

    def forward(self, x, residual=None, save=False):
        """(y, what backward takes). x, residual: (tokens, d) bf16."""
        m, d = x.shape
        f = self.w1.rows
        new = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device=x.device)  # noqa: E731
        h = x if residual is None else new(m, d)
        q = gep.mx_empty(m, d, self.fmt, device=x.device)
        n = new(m, d) if save else None
        rstd = torch.empty(m, dtype=torch.float32, device=x.device) if save else None
        gep.rmsnorm(x, self.weight, residual=residual, eps=self.eps, h=None if residual is None else h, y=n, q=q, rstd=rstd)
        pre, a = new(m, f) if save else None, new(m, f)
        gep.mx_gemm(q, self.w1, D=pre, PostAct=a, act="silu")
        y = gep.mx_gemm(gep.mx_quantize(a, self.fmt), self.w2, D=new(m, d), C=h)
        return y, (h, n, rstd, pre) if save else None

    def backward(self, dy, saved):
        """Gradients of x (and of the residual), the norm's weight, w1 and w2 from dy (tokens, d)."""
        h, n, rstd, pre = saved
        fmt = self.fmt
        dpre, a = torch.empty_like(pre), torch.empty_like(pre)
        gep.gemm_dact(dy, self.w2t, pre, dpre, PostAct=a, act="silu")
        # weight gradients sum over tokens: both operands have their blocks along them
        dw2 = gep.mx_gemm(gep.mx_quantize(dy, fmt, transpose=True), gep.mx_quantize(a, fmt, transpose=True))
        dw1 = gep.mx_gemm(gep.mx_quantize(dpre, fmt, transpose=True), gep.mx_quantize(n, fmt, transpose=True))
        dn = gep.mx_gemm(gep.mx_quantize(dpre, fmt), self.w1t)
        dx, dweight = gep.rmsnorm_backward(dn, h, self.weight, rstd, dres=dy)
        return dx, dweight, dw1, dw2


class MxExperts:
    """The first product of a mixture of experts on rows sorted by expert: one matrix per expert,
    (experts, f, d), in MX codes; offsets: int32 (experts + 1,) on the GPU."""

    def __init__(self, weight, w1, fmt="e4m3", weight_fmt="e2m1", eps=1e-5):
        self.weight, self.fmt, self.eps = weight, fmt, eps
        self.w1 = gep.mx_empty(w1.shape[1], w1.shape[2], weight_fmt, groups=w1.shape[0], device=w1.device)
        for g in range(w1.shape[0]):
            gep.mx_quantize(w1[g], weight_fmt, out=self.w1.group(g))

    def forward(self, x, offsets):
        q = gep.rmsnorm(x, self.weight, eps=self.eps, q=gep.mx_empty(*x.shape, self.fmt, device=x.device))
        a = torch.empty(x.shape[0], self.w1.rows, dtype=torch.bfloat16, device=x.device)
        return gep.mx_gemm(q, self.w1, PostAct=a, act="silu", cu_seqlens_m=offsets)


def reference(x, residual, weight, w1, w2, eps=1e-5):
    """The layer in fp32 with torch's own operations and gradients."""
    h = x + residual
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * weight
    return h + torch.nn.functional.silu(n @ w1.t()) @ w2.t()


def inputs(tokens, d, f, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()  # noqa: E731
    return dict(x=new(tokens, d), residual=new(tokens, d), weight=(1 + new(d, scale=0.1)).bfloat16(),
                w1=new(f, d, scale=d ** -0.5), w2=new(d, f, scale=f ** -0.5)), new(tokens, d)


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


def main(tokens=4096, d=2048, f=8192):
    t, dy = inputs(tokens, d, f)
    layer = MxMlp(t["weight"], t["w1"], t["w2"])
    y, saved = layer.forward(t["x"], t["residual"], save=True)
    grads = layer.backward(dy, saved)
    leaves = {k: v.float().requires_grad_() for k, v in t.items()}
    want = reference(**leaves)
    want.backward(dy.float())
    print(f"y         relative error {relative(y, want.detach()):.4f}")
    for name, got in zip(("x", "weight", "w1", "w2"), grads):
        print(f"d{name:8s} relative error {relative(got, leaves[name].grad):.4f}")
    for fmt in ("e4m3", "e2m1"):
        serve = MxMlp(t["weight"], t["w1"], t["w2"], weight_fmt=fmt, training=False)
        one = serve.forward(t["x"][:1], t["residual"][:1])[0]
        print(f"one token, {fmt} weights: relative error {relative(one, want.detach()[:1]):.4f}, "
              f"{timed(lambda: serve.forward(t['x'][:1], t['residual'][:1])):.0f} us")
    print(f"{tokens} tokens: forward {timed(lambda: layer.forward(t['x'], t['residual'], save=True)):.0f} us, "
          f"backward {timed(lambda: layer.backward(dy, saved)):.0f} us")


if __name__ == "__main__":
    main()
