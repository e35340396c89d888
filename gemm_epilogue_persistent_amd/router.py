"""The router's side of the grouped products: per-expert counts with their offsets, the balance loss of a batch and its
gradient (binding of include/router_mi355x.h; argument checks and marshalling only).

    b = router_balance(logits, chosen, coef=0.01, mask=mask)     # b.loss, b.counts, b.cu_seqlens, b.probs
    dlogits = router_balance_backward(logits, b, grad=g)

Of `batch` sequences, each with n unmasked tokens that make k choices each:
P_e = mean over its tokens of p_e, f_e = experts counts_e / (k n), loss = coef / batch sum f_e P_e, with p the softmax of
the logits or their sigmoids divided by the sum of them.
"""
import torch

from . import _abi
from .mx import _FLOAT_DT, _MOST, _allocating, _launch

SCORES = {"softmax": 0, "sigmoid": 1}


class RouterBalance:
    """What router_balance gives: loss float32 (), counts int32 (batch, experts), cu_seqlens int32 (experts + 1), the
    offsets of the experts' rows over all sequences; probs float32 (batch, experts), the mean scores; valid
    int32 (batch), the unmasked tokens. It also remembers the call (k, scores, coef, mask) for the backward pass."""

    __slots__ = ("loss", "counts", "cu_seqlens", "probs", "valid", "batch", "experts", "device", "call")

    def __repr__(self):
        return f"RouterBalance(batch {self.batch}, {self.experts} experts, {self.device})"


def balance_empty(experts, batch=1, device="cuda"):
    """Storage of the results of router_balance, zeros."""
    return _storage(int(experts), int(batch), device, torch.zeros)


def _storage(experts, batch, device, fill):
    if experts < 1 or batch < 0:
        raise ValueError("at least one expert and no negative batch expected")
    b = RouterBalance()
    new = lambda shape, dtype: fill(shape, dtype=dtype, device=device)  # noqa: E731
    b.loss, b.counts, b.cu_seqlens = new((), torch.float32), new((batch, experts), torch.int32), new((experts + 1,), torch.int32)
    b.probs, b.valid = new((batch, experts), torch.float32), new((batch,), torch.int32)
    b.batch, b.experts, b.device, b.call = batch, experts, b.loss.device, None
    return b


def router_balance_workspace(batch, tokens, experts):
    """Bytes of device memory that router_balance takes as its workspace."""
    n = _abi.load().router_balance_workspace(*(_abi.int32(k, v) for k, v in (("batch", batch), ("tokens", tokens), ("experts", experts))))
    if n < 0:
        raise ValueError("sizes outside what router_balance takes")
    return n


def _logits(name, t, shape=None, device=None, dtype=None):
    """Checks of logits (tokens, experts) or (batch, tokens, experts); (batch, tokens, experts) and both strides."""
    have = t.shape
    if len(have) not in (2, 3) or not t.is_cuda:
        raise ValueError(f"{name}: (tokens, experts) or (batch, tokens, experts) on the GPU expected")
    if t.dtype not in _FLOAT_DT or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if shape is not None and have != shape:
        raise ValueError(f"{name} has shape {tuple(have)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    b, n, e = have if len(have) == 3 else (1, *have)
    if b > _MOST or n > _MOST or e > _MOST:
        raise ValueError(f"{name}: more than 2^31 - 1 sequences, tokens or experts")
    if e < 1:
        raise ValueError(f"{name}: no experts")
    step = t.stride()
    if e > 1 and step[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return (b, n, e), step[-2] if n > 1 else e, step[0] if b > 1 else 0


def router_balance(logits, chosen, out=None, scores="softmax", coef=1.0, mask=None, workspace=None, stream=None):
    """Counts and balance loss of logits (tokens, experts) or (batch, tokens, experts), 16- or 32-bit floats with contiguous
    rows; batch: a loss for each sequence, whose mean is returned. chosen: (..., k) int32 or int64,
    contiguous, the experts that each token goes to (an index outside the experts is no choice). mask: (...) bool,
    contiguous; tokens where it is False count nowhere. workspace: uint8 of router_balance_workspace(batch,
    tokens, experts) bytes that nothing else uses meanwhile (allocated if None). Returns `out`, a RouterBalance
    (allocated if None)."""
    (b, n, e), ld, ldb = _logits("logits", logits)
    dev = logits.device
    if scores not in SCORES:
        raise ValueError(f"unknown scores {scores!r}")
    lead = logits.shape[:-1]
    if chosen.dim() != len(lead) + 1 or chosen.shape[:-1] != lead or chosen.device != dev or not chosen.is_contiguous():
        raise ValueError(f"chosen: contiguous {tuple(lead) + ('k',)} on {dev} expected")
    if chosen.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"chosen: int32 or int64 expected, not {chosen.dtype}")
    k = chosen.shape[-1]
    if mask is not None:
        if mask.dtype != torch.bool:
            raise TypeError(f"mask: bool expected, not {mask.dtype}")
        if mask.shape != lead or mask.device != dev or not mask.is_contiguous():
            raise ValueError(f"mask: contiguous {tuple(lead)} on {dev} expected")
    if out is None or workspace is None:
        with _allocating(stream), torch.cuda.device(dev):
            out = _storage(e, b, dev, torch.empty) if out is None else out
            workspace = torch.empty(router_balance_workspace(b, n, e), dtype=torch.uint8, device=dev) if workspace is None else workspace
    if not isinstance(out, RouterBalance):
        raise TypeError("out: a RouterBalance expected")
    if out.batch != b or out.experts != e or out.device != dev:
        raise ValueError(f"out is of batch {out.batch} and {out.experts} experts on {out.device}, expected {b} and {e} on {dev}")
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous uint8 tensor on the logits' GPU expected")
    a = _abi.ROUTER_BALANCE_ARGS.pack(
        b, n, e, _abi.int32("k", k), _FLOAT_DT[logits.dtype], SCORES[scores], chosen.element_size(), float(coef), logits.data_ptr(), chosen.data_ptr(),
        mask.data_ptr() if mask is not None else 0, out.counts.data_ptr(), out.valid.data_ptr(), out.cu_seqlens.data_ptr(),
        out.probs.data_ptr(), out.loss.data_ptr(), workspace.data_ptr(), workspace.numel(), ld, ldb)
    _launch(dev, stream, _abi.load().router_balance, a)
    out.call = (lead, k, scores, float(coef), mask)
    return out


def router_balance_backward(logits, balance, grad=None, dlogits=None, stream=None):
    """The gradient of grad * balance.loss with respect to the logits, which `balance` was made of (with the same mask,
    whose memory is read again). grad: a float32 tensor of one element on the GPU (None: 1). Returns dlogits, of the logits'
    type (allocated if None; may be the logits themselves)."""
    if not isinstance(balance, RouterBalance):
        raise TypeError("balance: a RouterBalance expected")
    if balance.call is None:
        raise ValueError("balance: no results of router_balance")
    lead, k, scores, coef, mask = balance.call
    (b, n, e), ld, ldb = _logits("logits", logits)
    dev = logits.device
    if logits.shape[:-1] != lead or e != balance.experts or dev != balance.device:
        raise ValueError(f"logits: {tuple(lead) + (balance.experts,)} on {balance.device} expected, as in the forward pass")
    if grad is not None and (grad.dtype != torch.float32 or grad.numel() != 1 or grad.device != dev):
        raise ValueError(f"grad: one float32 on {dev} expected")
    if dlogits is None:
        with _allocating(stream):
            dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    _, ldd, lddb = _logits("dlogits", dlogits, logits.shape, dev, logits.dtype)
    a = _abi.ROUTER_BALANCE_BACKWARD_ARGS.pack(
        b, n, e, k, _FLOAT_DT[logits.dtype], SCORES[scores], coef, logits.data_ptr(), mask.data_ptr() if mask is not None else 0,
        balance.counts.data_ptr(), balance.valid.data_ptr(), grad.data_ptr() if grad is not None else 0, dlogits.data_ptr(),
        ld, ldb, ldd, lddb)
    _launch(dev, stream, _abi.load().router_balance_backward, a)
    return dlogits
