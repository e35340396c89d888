"""The 128 x 128 tiles of the quantiser and of the activation's backward pass along the rows and down the columns (columns of a
multiple of 8 tiles where rows of codes are no whole lines of 128 bytes), and over several launches (2^22 tiles each)."""
import numpy as np
import pytest
import torch

import fp8_ref as R
import gemm_epilogue_persistent_amd as gep
from test_gpu_fp8 import announce, check_quantized, dirty, stored, values
from test_gpu_fp8_act import ordinary

pytestmark = pytest.mark.gpu

DOWN = [(1000, 200), (1024, 520), (1000, 1), (897, 136), (2048, 72)]
ALONG = [(1000, 256), (1024, 120), (1025, 200), (896, 200), (1030, 264)]


@pytest.mark.parametrize("tiles", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", DOWN + ALONG)
def test_quantise(rows, cols, kind, tiles):
    announce(f"fp8 tile order {rows}x{cols} {kind} {'tiles' if tiles else 'rows'}")
    x = values(rows + cols, rows, cols, kind)
    x64 = x.double().numpy()
    q, qt = dirty(rows, cols, tiles), dirty(cols, rows, tiles)
    gep.fp8_quantize(x.cuda(), out=q, out_t=qt)
    check_quantized(q, x64, tiles)
    check_quantized(qt, x64.T, tiles)
    if tiles:
        check_quantized(gep.fp8_quantize(x.cuda(), tiles=True), x64, True)


@pytest.mark.parametrize("rows,cols", DOWN + ALONG)
def test_activation_backward(rows, cols):
    announce(f"fp8 tile order of the activation's backward pass {rows}x{cols}")
    x = ordinary(rows, rows, cols, "bf16").double().numpy()
    codes, scales = R.quantize(x)
    dy = torch.randn(rows, cols, generator=torch.Generator().manual_seed(3)).bfloat16()
    q, qt, dx = dirty(rows, cols), dirty(cols, rows), torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    gep.fp8_act_backward(dy.cuda(), stored(codes, scales, cols), "relu", dx=dx, q=q, qt=qt)
    want = dy.double().numpy() * (R.values(codes, scales, cols) > 0)  # (16-bit values, and zeros with their sign: exact)
    check_quantized(q, want)
    check_quantized(qt, want.T)
    assert np.array_equal(dx.double().cpu().numpy(), want)


TALL = (1 << 29) + 1000  # 2^22 + 8 tiles of 128 rows


def test_down_past_one_launch():
    announce("fp8 quantise and act backward 2^29 + 1000 x 1")
    x = torch.empty(TALL, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(7))
    q, qt = gep.fp8_empty(TALL, 1, tiles=True), gep.fp8_empty(1, TALL, tiles=True)
    gep.fp8_quantize(x, out=q, out_t=qt)
    kept = gep.fp8_quantize(x)
    dx, yt = torch.full_like(x, 77.0), gep.fp8_empty(1, TALL)
    gep.fp8_act_backward(x, kept, "relu", dx=dx, yt=yt)
    last = (1 << 22) * 128
    for s in (slice(0, 512), slice(last // 2, last // 2 + 256), slice(last - 512, last), slice(last, TALL)):
        v = x[s].double().cpu().numpy()
        b = torch.arange(s.start // 128, -(-s.stop // 128), device="cuda")
        codes, scales = R.quantize(v, True)
        assert np.array_equal(q.codes[s].cpu().numpy(), codes) and np.array_equal(q.scales[b, 0].cpu().numpy(), scales[:, 0])
        codes, scales = R.quantize(v.T, True)
        assert np.array_equal(qt.codes[:, s].cpu().numpy(), codes[:, :len(v)])
        assert np.array_equal(qt.scales[0][b].cpu().numpy(), scales[0])
        codes, scales = R.quantize(v)
        xh = R.values(codes, scales, 1).astype(np.float32).astype(np.float64)
        assert np.array_equal(dx[s].double().cpu().numpy(), v * (xh > 0))
        # (a column of x^ in blocks of 128: scales are exact, a code may be a neighbour where fp32's product with r lies on a border)
        codes, scales = R.quantize(np.where(xh > 0, xh, 0).T)
        assert np.array_equal(yt.scales[0][b // 4, 0, b % 4].cpu().numpy(), scales[0])
        assert np.abs(yt.codes[:, s].cpu().numpy().astype(int) - codes[:, :len(v)]).max() <= 1
