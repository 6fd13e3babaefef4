"""8-bit append, tiles whose scale grows: the stored values against the rows that
were given, and scales that grow from the smallest to the largest."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
from oracle import quantized as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE = pytest.mark.parametrize("code", ["int8", "e4m3"])


def values(p):
    scales = p.scales.cpu().numpy().astype(np.float64)
    return oq.decode(p.codes.view(torch.uint8).cpu().numpy(), p.code) * scales[..., None, None], scales


def append(p, codes, scales, k, v, slots):
    """One call, and the same by the oracle: equal bit for bit."""
    oq.append(codes, scales, k.numpy(), v.numpy(), slots, p.code)
    pk.pa_reshape_and_cache_q8(k.to(DEV), v.to(DEV), p, torch.tensor(slots, device=DEV))
    odd = not (torch.isfinite(k).all() and torch.isfinite(v).all())
    assert pk.pa_get_device_error() == (pk.PA_DEVERR_NONFINITE if odd else 0)
    assert np.array_equal(p.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(p.codes.view(torch.uint8).cpu().numpy(), codes)


@CODE
@pytest.mark.parametrize("factor", [1.0, 1.1, 2.0, 3.7, 64.0, 1e4])
def test_error_after_growth(factor, code):
    """16 rows in 16 calls, each up to `factor` times the one before; small and
    large elements in every row. By 1e4 the last rows pass fp32: an infinity is
    reported and stored as the largest code, which the oracle's codes hold; the
    bound is for the finite ones."""
    g = torch.Generator().manual_seed(int(factor * 10))
    p = pk.Q8Pool(2, 2, 128, code)
    codes, scales = np.zeros(p.codes.shape, np.uint8), np.zeros(p.scales.shape, np.float32)
    given, grew = np.zeros((2, 2, 16, 128)), np.zeros((2, 2))
    for r in range(16):
        rows = [torch.randn(1, 2, 128, generator=g) * torch.exp2(-9 * torch.rand(1, 2, 128, generator=g)) *
                factor ** (r * (0.5 + 0.5 * float(torch.rand(1, generator=g)))) for _ in range(2)]
        old = scales[1].copy()
        append(p, codes, scales, *rows, [16 + r])
        given[0, :, r], given[1, :, r] = rows[0][0].double().numpy(), rows[1][0].double().numpy()
        grew += (scales[1] > old) & (r > 0)
    got, s = values(p)
    given, here = np.where(np.isfinite(given), given, 0), np.isfinite(given)
    err, mag, s = np.where(here, np.abs(got[1] - given), 0), np.abs(given), s[1][..., None, None]
    if code == "int8":
        lim = s / 2 * (1 + grew[..., None, None])
    else:
        lim = np.where(grew[..., None, None] > 0, 2.0 ** -4 * mag + 2.0 ** -9 * s, np.maximum(2.0 ** -4 * mag, 2.0 ** -10 * s))
    assert np.all(err <= lim + 2.0 ** -22 * mag)
    if factor >= 2:
        assert grew.min() >= 3


@CODE
@pytest.mark.parametrize("small", [2.0 ** -99, 1e-20])
@pytest.mark.parametrize("large", [2.0 ** 27, 2.0 ** 29, 1e20, 3.4e38])
def test_tiny_scale_then_large_rows(large, small, code):
    """No finite value is cut off, whatever the tile's scale was before."""
    g = torch.Generator().manual_seed(1)
    p = pk.Q8Pool(2, 1, 64, code)
    codes, scales = np.zeros(p.codes.shape, np.uint8), np.zeros(p.scales.shape, np.float32)
    low = [small * (0.5 + 0.5 * torch.rand(3, 1, 64, generator=g)) for _ in range(2)]
    append(p, codes, scales, *low, [0, 1, 2])
    high = [large * (2 * torch.rand(2, 1, 64, generator=g) - 1) for _ in range(2)]
    high[0][0, 0, 0], high[1][1, 0, 5] = large, -large
    append(p, codes, scales, *high, [3, 7])
    got, s = values(p)
    for kv in range(2):
        x = high[kv][:, 0].double().numpy()
        step = s[0, kv, 0] / 2 if code == "int8" else np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s[0, kv, 0])
        assert np.all(np.abs(got[0, kv, 0, [3, 7]] - x) <= step + 2.0 ** -22 * np.abs(x))
