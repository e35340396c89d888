"""The balance loss's scores far below a row's largest one, its sums row by row, and its mean scores under bounds that follow
from how the tokens are shared out.

Tolerances, in half steps h = 2^-24. A score p = e^d / sum, d a difference that fp32 holds: the exponential 3 (one step of the
instruction, and its own last rounding), the sum of a row whose other terms are below e^-20 1, the quotient 1, their product
1: 6. A sigmoid's e^x / (1 + e^x) 3 more: a reciprocal within a step and a product: 9; where a row is scaled by its largest
logit, the product with 1 - s(x), which has 3 of the exponential, 1 of the sum and 2 of the reciprocal: 12. The mean of one token is that. A
gradient p (w - sum p w) of a weight that is exact: the score's, those of the sum, which is a score's, and 6 for its four products and differences.
"""
import numpy as np
import pytest
import torch

import gemm_epilogue_persistent_amd as gep
import test_gpu_balance as balance
from test_gpu_balance import definition, inputs, run
from test_gpu_fp8 import announce

pytestmark = pytest.mark.gpu

H = 2.0 ** -24


def relative(got, want):
    """Largest error relative to the value, of those above 2^-125 (smaller ones may be 0)."""
    some = want.abs() > 2.0 ** -125
    assert ((got - want).abs()[~some] <= 2.0 ** -124).all()
    return ((got - want).abs()[some] / want.abs()[some]).max().item()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 60, 300, 2048])
def test_far_below_the_largest(E, scores):
    """Rows of one token each: the largest logit 0 (softmax) or 100 (a sigmoid of 1), the others from -21 to -87, a multiple of
    2^-8, so that differences are exact: their scores are e^x, to a few steps of themselves."""
    announce(f"balance far below the largest {E} {scores}")
    B = 64
    g = torch.Generator().manual_seed(E)
    x = -21 - torch.randint(0, 66 * 256, (B, 1, E), generator=g).double() / 256
    top = torch.randint(0, E, (B, 1, 1), generator=g)
    x.scatter_(2, top, 0.0 if scores == "softmax" else 100.0)
    # the largest's own count is the least, so that the gradient of the others is p w: w is a power of two times a whole number
    chosen = (top + 1) % E
    want = definition(x, chosen, None, scores, 1.0)
    b, d = run(x.float(), chosen, None, scores, coef=1.0)
    assert relative(b.probs.double().cpu(), want["probs"]) <= (6 if scores == "softmax" else 9) * H
    if E & (E - 1) == 0:
        got = d.double().cpu()
        # (of a sigmoid of 100, 1 - s is e^-100: below fp32)
        others = torch.ones_like(x, dtype=torch.bool).scatter(2, top, False)
        assert relative(got[others], want["d"][others]) <= (18 if scores == "softmax" else 24) * H


@pytest.mark.parametrize("top", [-0.5, -5.0, -12.0, -20.0, -30.0, -36.0, -39.5, -41.0, -70.0, -86.0])
def test_small_sigmoids_beside_smaller_ones(top):
    """Sigmoid rows whose largest logit is small and whose others lie below e^-87, where fp32 ends: the scores are e^(x - top)
    all the same. Multiples of 1 / 4: differences are exact."""
    announce(f"balance small sigmoids {top}")
    low = [v / 4 for v in range(-4 * 110, -4 * 80) if v / 4 > top - 85]
    for E in (2, 24, 260):
        rows = []
        for i, v in enumerate(low):
            row = np.full(E, v)
            row[i % E] = top
            row[(i + 1) % E] = v
            if E > 2:
                row[(i + 2) % E] = -np.inf
            rows.append(row)
        x = torch.tensor(np.array(rows))[:, None, :]
        chosen = (torch.arange(len(low)) + 1).remainder(E)[:, None, None]
        want = definition(x, chosen, None, "sigmoid", 1.0)
        b, d = run(x.float(), chosen, None, "sigmoid", coef=1.0, grad=float(len(low)))
        # (a row's sum: 8 values of a lane one after another, and 6 levels of the tree)
        levels = 14 * H
        assert relative(b.probs.double().cpu(), want["probs"]) <= 12 * H + levels
        # (relative to p (w + sum p w): two scores, 6 as above, 6 of 1 - s(x), and 4 of the weight, coef experts / (batch k))
        want = definition(x, chosen, None, "sigmoid", 1.0, float(len(low)))
        assert ((d.double().cpu() - want["d"]).abs() <= (40 * H + 2 * levels) * want["size"] + 2.0 ** -124).all()


def test_negative_infinity_beside_small_sigmoids():
    announce("balance -inf beside small sigmoids")
    x = torch.full((3, 4, 9), -np.inf, dtype=torch.float64)
    x[0, 0, 3] = -100.0
    x[0, 1, 3], x[0, 1, 4] = -30.0, -np.inf
    x[1, 2] = -95.0
    x[2, 3, :2] = torch.tensor([-0.25, -99.0])
    chosen = torch.randint(0, 9, (3, 4, 2), generator=torch.Generator().manual_seed(1))
    b, d = run(x.float(), chosen, None, "sigmoid", coef=1.0, grad=64.0)
    balance.check(b, d, definition(x, chosen, None, "sigmoid", 1.0, 64.0), "f32", 4, 2)
    assert (d[0, 2] == 0).all() and b.probs[0, 3].item() == 0.5


SHARED = [(1, 20000, 64, 6), (8, 3001, 128, 8), (70, 33, 8, 2), (1, 5000, 8, 1), (2, 1500, 2048, 3), (300, 77, 16, 2), (1, 70000, 8, 2),
          (1, 1025, 512, 2), (3, 4097, 257, 4), (1, 64, 64, 2)]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,T,E,k", SHARED)
def test_every_row_once(B, T, E, k, scores):
    """Each token has one expert of score 1, all others 0: the sums are whole numbers, which fp32 adds exactly, so that a row
    taken twice, left out or taken for its neighbour changes a mean."""
    announce(f"balance every row once {B}x{T} over {E} {scores}")
    g = torch.Generator().manual_seed(B + T)
    best = torch.randint(0, E, (B, T), generator=g)
    mask = torch.rand(B, T, generator=g) < 0.8 if B > 1 else None
    x = torch.full((B, T, E), -200.0).scatter_(2, best[..., None], 100.0)
    chosen = torch.randint(0, E, (B, T, k), generator=g)
    b, d = run(x, chosen, mask, scores)
    keep = torch.ones(B, T, dtype=torch.bool) if mask is None else mask
    for s in range(B):
        n = keep[s].sum()
        want = torch.bincount(best[s][keep[s]], minlength=E).float() / n.float()
        assert torch.equal(b.probs[s].cpu(), want)
        assert torch.equal(b.counts[s].cpu().long(), torch.bincount(chosen[s][keep[s]].flatten(), minlength=E))
    assert not d.any()


def chain(B, T, E):
    """Additions that a mean score passes through: the tokens of a group of lanes one after another, the groups of a wave, the waves of a
    workgroup; the workgroups that a wave of the join adds, and its eight waves."""
    lanes = 1
    while lanes < 64 and lanes * 8 < E:
        lanes *= 2
    threads = 1024 if E <= 512 else 256
    groups = threads // lanes
    per = -(-(-(-T // max(1, 256 // B))) // groups) * groups
    if B == 1 and T <= 4 * groups:
        return 16 + 6 + 16  # (one workgroup of 256 or 1024 threads: four tokens a group, or sixteen)
    return per // groups + 6 + threads // 64 + -(-(-(-T // per)) // 4) + 8


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B,T,E,k", SHARED)
def test_mean_scores(B, T, E, k, scores):
    """The error of a score (the file of the other tests: 46 half steps, and the difference to the largest logit, which lies below 32
    in magnitude: 32 more, its half step relative to e^d), then a half step for each addition on the way and 2 for the mean."""
    announce(f"balance mean scores {B}x{T} over {E} {scores}")
    x, chosen, mask = inputs(B + T, B, T, E, k, "f32", B > 1, torch.int64)
    want = definition(x.double(), chosen, mask, scores, 1.0)
    b, _ = run(x, chosen, mask, scores, coef=1.0)
    tol = (80 + chain(B, T, E)) * H
    assert ((b.probs.double().cpu() - want["probs"]).abs() <= tol * want["probs"]).all()
    # (the loss: the factors f, their products and 2048 sums in a tree of 9 levels and 64 workgroups' shares)
    assert abs(b.loss.double().item() - want["loss"].item()) <= (tol + (8 + 9 + -(-B * (-(-E // 64)) // 256) + 16) * H) * want["loss"].item()


@pytest.mark.parametrize("B,T,E", [(4096, 3, 8), (65535, 1, 8), (3000, 2, 130), (1000, 5, 2048), (2001, 2, 1), (90, 3, 60), (1025, 2, 100), (17, 4, 128)])
def test_many_sequences(B, T, E):
    """Counts, offsets and losses of thousands of short sequences."""
    announce(f"balance of {B} sequences of {T} tokens over {E}")
    x, chosen, mask = inputs(B, B, T, E, min(E, 2), "f32", True, torch.int32)
    want = definition(x.double(), chosen, mask, "softmax", 0.01, 64.0)
    b, d = run(x, chosen, mask, "softmax", grad=64.0)
    balance.check(b, d, want, "f32", T, min(E, 2))
