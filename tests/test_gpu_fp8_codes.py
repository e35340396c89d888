"""8-bit matrices whose codes hold e4m3's NaN (0x7F and 0xFF), which the quantiser never writes but others may."""
import pytest
import torch

import gemm_epilogue_persistent_amd as gep
from test_gpu_fp8 import TILES, announce, dirty, operand, stored
from test_gpu_fp8_act import ACTS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
def test_nan_codes(act):
    """e4m3 has a NaN code of its own: an element of it is NaN, as the inverse says, and so are its gradient and, but for
    ReLU, whose NaN is 0, its value. Its neighbours are what they are without it."""
    announce(f"fp8 act NaN codes {act}")
    codes, scales = operand(5, 140, 300)
    clean = stored(codes, scales, 300)
    bad = codes.copy()
    bad[3, 17], bad[139, 299], bad[64, 128] = 0x7F, 0xFF, 0x7F
    kept = stored(bad, scales, 300)
    dy = torch.randn(140, 300, generator=torch.Generator().manual_seed(2)).cuda()
    got = [torch.empty(140, 300, device="cuda") for _ in range(4)]
    gep.fp8_act_backward(dy, clean, act, dx=got[0], y=got[1])
    gep.fp8_act_backward(dy, kept, act, dx=got[2], y=got[3])
    nan = gep.fp8_dequantize(kept, dtype=torch.float32).isnan()
    assert nan.sum() == 3 and torch.equal(nan.nonzero().cpu(), torch.tensor([[3, 17], [64, 128], [139, 299]]))
    assert torch.equal(got[2][~nan], got[0][~nan]) and torch.equal(got[3][~nan], got[1][~nan])
    assert got[2][nan].isnan().all()
    assert (got[3][nan] == 0).all() if act in ("relu", "relu_sq") else got[3][nan].isnan().all()
    # in 8 bits the block is NaN
    q, yt = dirty(140, 300), dirty(300, 140)
    gep.fp8_act_backward(dy, kept, act, q=q, yt=yt)
    blocks = torch.zeros(140, 300, dtype=torch.bool, device="cuda")
    blocks[3, :128], blocks[64, 128:256], blocks[139, 256:] = True, True, True
    assert torch.equal(gep.fp8_dequantize(q).isnan(), blocks)
    if act not in ("relu", "relu_sq"):
        turned = torch.zeros(300, 140, dtype=torch.bool, device="cuda")
        turned[17, :128], turned[128, :128], turned[299, 128:] = True, True, True
        assert torch.equal(gep.fp8_dequantize(yt).isnan(), turned)


@pytest.mark.parametrize("tiles", [True, False])
@pytest.mark.parametrize("tile", TILES)
def test_nan_codes_in_products(tile, tiles):
    """A NaN element of A makes its row NaN, one of B its column, and nothing else."""
    announce(f"fp8 product with NaN codes tile {tile} {'tiles' if tiles else 'rows'}")
    M, N, K = 140, 272, 700
    (ca, sa), (cb, sb) = operand(1, M, K), operand(2, N, K, tiles)
    clean = torch.empty(M, N, device="cuda")
    gep.fp8_gemm(stored(ca, sa, K), stored(cb, sb, K, tiles), D=clean, tile=tile, split=1)
    ca[130, 699], ca[7, 0], cb[260, 555] = 0x7F, 0xFF, 0x7F
    got = torch.empty(M, N, device="cuda")
    gep.fp8_gemm(stored(ca, sa, K), stored(cb, sb, K, tiles), D=got, tile=tile, split=1)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[130], bad[7], bad[:, 260] = True, True, True
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], clean[~bad])
