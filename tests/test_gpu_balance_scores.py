"""The balance loss's scores far below a row's largest one.

Tolerances, in half steps h = 2^-24. A score p = e^d / sum, d a difference that fp32 holds: the exponential 3 (one step of the
instruction, and its own last rounding), the sum of a row whose other terms are below e^-20 1, the quotient 1, their product
1: 6. A sigmoid's e^x / (1 + e^x) 3 more: a reciprocal within a step and a product: 9. The mean of one token is that. A
gradient p (w - sum p w) of a weight that is exact: the score's, those of the sum, which is a score's, and 6 for its four products and differences.
"""
import pytest
import torch

from test_gpu_balance import definition, run
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
