"""Large 8-bit results, and launches of more tiles than one grid takes (2^22), value by value or in samples."""
import numpy as np
import pytest
import torch

import fp8_ref as R
import gemm_epilogue_persistent_amd as gep
from test_gpu_fp8 import announce

pytestmark = pytest.mark.gpu


def rows_equal(m, some, want):
    """Rows `some` of the FP8 matrix m (a scale per 128 values of a row) are the definition's of want(row) (k values, float64)."""
    nb = -(-m.k // 128)
    b = np.arange(nb)
    for r in some:
        codes, scales = R.quantize(want(r)[None, :])
        assert np.array_equal(m.codes[r:r + 1].cpu().numpy(), codes), r
        assert np.array_equal(m.scales[r // 64].cpu().numpy()[b // 4, r % 64, b % 4], scales[0]), r


def test_large_activation():
    """More than 2^31 bytes of codes of act(x) and of the transposed checkpoint."""
    announce("fp8 act 70001 x 32784 bf16")
    rows, cols = 70001, 32784
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(4))
    kept, q = gep.fp8_empty(rows, cols), gep.fp8_empty(rows, cols)
    gep.fp8_act(x, "relu", saved=kept, q=q)
    rows_equal(q, (0, 63, 64, 35000, 65536, 65537, 69999, 70000), lambda r: np.maximum(x[r].double().cpu().numpy(), 0.0) + 0.0)
    rows_equal(kept, (0, 65537, 70000), lambda r: x[r].double().cpu().numpy())
    qt, yt = gep.fp8_empty(cols, rows), gep.fp8_empty(cols, rows)
    dy = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    gep.fp8_act_backward(dy, kept, "relu", q=q, qt=qt, yt=yt)

    def column(c):  # x^, as fp32 holds it
        codes = kept.codes[:, c:c + 1].cpu().numpy()
        s = kept.scales[:, c // 512, :, (c // 128) % 4].reshape(-1)[:rows].cpu().numpy()
        return R.values(codes, s[:, None], 1)[:, 0].astype(np.float32).astype(np.float64)

    for c in (0, 17, 30000, 32767, 32768, 32783):
        xh = column(c)
        # (act(x^) is x^ or 0, 4 bits times a scale of 24: rounded once to fp32, as here; its product with r is rounded once more, so
        # a code may be the neighbour's where the exact one lies on a border)
        codes, scales = R.quantize(np.where(xh > 0, xh, 0)[None, :])
        got = yt.codes[c:c + 1].cpu().numpy()
        b = np.arange(scales.shape[1])
        assert np.array_equal(yt.scales[c // 64].cpu().numpy()[b // 4, c % 64, b % 4], scales[0])
        assert np.abs(got.astype(int) - codes).max() <= 1 and (got != codes).mean() < 1e-3
        d = dy[:, c].double().cpu().numpy() * (xh > 0)  # (16-bit values, and zeros with their sign: exact)
        rows_equal(qt, (c,), lambda r: d)


WIDE = (1 << 29) + 77  # 2^22 + 1 tiles of 128 columns


@pytest.fixture
def wide():
    yield torch.empty(1, WIDE, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(6))
    torch.cuda.empty_cache()


def sections(n):
    """Runs of columns at the ends, around the last tile of the first launch, and in the last one."""
    last = (1 << 22) * 128
    return [slice(0, 512), slice(last // 2, last // 2 + 256), slice(last - 512, last), slice(last, n)]


@pytest.mark.parametrize("tiles", [True, False])
def test_quantise_past_one_launch(wide, tiles):
    announce(f"fp8 quantise 1 x 2^29 + 77 {'tiles' if tiles else 'rows'}, both directions")
    q, qt = gep.fp8_empty(1, WIDE, tiles=tiles), gep.fp8_empty(WIDE, 1, tiles=tiles)
    for m in (q, qt):
        m.codes.fill_(0x55)
    gep.fp8_quantize(wide, out=q, out_t=qt)
    for s in sections(WIDE):
        x = wide[:, s].double().cpu().numpy()
        codes, scales = R.quantize(x, tiles)
        n, b = x.shape[1], np.arange(s.start // 128, -(-s.stop // 128))
        assert np.array_equal(q.codes[:, s].cpu().numpy(), codes[:, :n])
        at = torch.from_numpy(b).cuda()
        got = q.scales[0][at] if tiles else q.scales[0][at // 4, 0, at % 4]
        assert np.array_equal(got.cpu().numpy(), scales[0])
        codes, scales = R.quantize(x.T, tiles)
        assert np.array_equal(qt.codes[s].cpu().numpy(), codes)
        got = qt.scales[b[0]:b[-1] + 1, 0] if tiles else qt.scales.view(-1, 64, 4)[s.start // 64:-(-s.stop // 64), :, 0].reshape(-1)[:n]
        assert np.array_equal(got.cpu().numpy(), scales[:, 0])


def test_activation_backward_past_one_launch(wide):
    announce("fp8 act backward 1 x 2^29 + 77")
    kept = gep.fp8_quantize(wide)
    dx, qt, yt = torch.full_like(wide, 77.0), gep.fp8_empty(WIDE, 1), gep.fp8_empty(WIDE, 1)
    gep.fp8_act_backward(wide, kept, "relu", dx=dx, qt=qt, yt=yt)
    for s in sections(WIDE):
        x = wide[:, s].double().cpu().numpy()
        codes, scales = R.quantize(x)
        xh = R.values(codes, scales, x.shape[1]).astype(np.float32).astype(np.float64)
        d = x * (xh > 0)
        assert np.array_equal(dx[:, s].double().cpu().numpy(), d)
        # (a column of one value: its code is 448 / the value cut to 13 bits, times the value: no border near)
        for m, v in ((qt, d), (yt, np.where(xh > 0, xh, 0))):
            codes, scales = R.quantize(v.T)
            assert np.array_equal(m.codes[s].cpu().numpy(), codes)
            got = m.scales.view(-1, 64, 4)[s.start // 64:-(-s.stop // 64), :, 0].reshape(-1)[:x.shape[1]]
            assert np.array_equal(got.cpu().numpy(), scales[:, 0])
