"""Seeded random sweep of the FP8 products, the quantisers, the activations and the balance loss: sizes, types, tiles, groups,
splits, epilogues, masks and strides drawn together, each case against the 64-bit formulas and bounds of the parametrised
tests. The case is printed before each GPU call. GEP_SWEEP_CASES sets the number of cases of each kind (default 60; case i draws
from seed 100 + i, so a larger count adds cases).
"""
import os
import random

import numpy as np
import pytest
import torch

import gemm_epilogue_persistent_amd as gep
import test_gpu_balance as balance
import test_gpu_fp8 as fp8
from test_gpu_fp8 import TILES, TYPES, announce

pytestmark = pytest.mark.gpu

CASES = int(os.environ.get("GEP_SWEEP_CASES", "60"))
ACTS = ["none", "relu", "relu_sq", "gelu_tanh", "silu"]


def spread(r, lo, hi):
    """Whole numbers whose logarithm is spread evenly."""
    return min(hi, int(lo * ((hi + 1) / lo) ** r.random()))


@pytest.mark.parametrize("i", range(CASES))
def test_products(i):
    r = random.Random(100 + i)
    M, N, K = spread(r, 1, 600), 8 * spread(r, 1, 75), spread(r, 1, 3000)
    tiles, tile = r.random() < 0.5, r.choice(TILES + ["auto"])
    sizes, split = None, 1
    if r.random() < 0.4:
        cuts = sorted(r.randint(0, M) for _ in range(r.choice([1, 2, 5, 70]) - 1))
        sizes = np.diff([0] + cuts + [M]).tolist()
    elif tile in TILES[1:] and K > 512 and r.random() < 0.4:
        split = r.choice([2, 3, 8])
    kinds = list(TYPES)
    c, d, post = r.choice([None] + kinds), r.choice([None] + kinds), r.choice([None] + kinds)
    if d is None and post is None:
        d = r.choice(kinds)
    act = r.choice(ACTS) if post else "none"
    if act == "relu_sq" and post == "f16":
        post = "bf16"  # (products of 3000 terms pass 256, and their squares F16's range)
    announce(f"fp8 sweep product {i}: {M}x{N}x{K} tiles {tiles} tile {tile} groups {sizes and len(sizes)} split {split} {c} {d} {post} {act}")
    fp8.run_product(M, N, K, tile, tiles, c, d, post, act, sizes, seed=1000 + 100 * i, split=split)


@pytest.mark.parametrize("i", range(CASES))
def test_quantisers(i):
    r = random.Random(100 + i)
    rows, cols, kind, tiles = spread(r, 1, 700), spread(r, 1, 1500), r.choice(list(TYPES)), r.random() < 0.5
    pad, at = r.randint(0, 9), r.randint(0, 5)
    announce(f"fp8 sweep quantiser {i}: {rows}x{cols} {kind} tiles {tiles} pad {pad} at {at}")
    x = torch.empty(rows * (cols + pad) + at + 1, dtype=TYPES[kind], device="cuda").fill_(float("nan"))
    x = x[at:at + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    x.copy_(fp8.values(1000 + i, rows, cols, kind))
    x64 = x.double().cpu().numpy()
    q, qt = fp8.dirty(rows, cols, tiles), fp8.dirty(cols, rows, tiles)
    gep.fp8_quantize(x, out=q, out_t=qt)
    fp8.check_quantized(q, x64, tiles)
    fp8.check_quantized(qt, x64.T, tiles)
    one, turned = fp8.dirty(rows, cols, tiles), fp8.dirty(rows, cols, tiles)
    gep.fp8_quantize(x, out=one)
    fp8.check_quantized(one, x64, tiles)
    gep.fp8_quantize(x.t().contiguous().t(), out=turned)  # (columns contiguous)
    fp8.check_quantized(turned, x64, tiles)


@pytest.mark.parametrize("i", range(CASES))
def test_balances(i):
    r = random.Random(100 + i)
    B, E = r.choice([1, 1, 2, 9]), spread(r, 1, 2048)
    T, k = spread(r, 1, max(1, min(6000, 2_000_000 // (B * E)))), r.randint(1, min(E, 8))
    kind, scores = r.choice(list(TYPES)), r.choice(["softmax", "sigmoid"])
    masked, index = r.random() < 0.5, r.choice([torch.int32, torch.int64])
    announce(f"fp8 sweep balance {i}: {B}x{T} over {E} k {k} {kind} {scores} masked {masked}")
    x, chosen, mask = balance.inputs(1000 + i, B, T, E, k, kind, masked, index)
    b, d = balance.run(x, chosen, mask, scores)
    balance.check(b, d, balance.definition(x.double(), chosen, mask, scores, 0.01), kind, T, k)
