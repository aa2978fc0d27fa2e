"""Edges of the training-step operators on the GPU."""
import math

import numpy as np
import pytest
import torch

from test_checkpoint_gpu import code_values, np64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


# ------------------------------------------------- largest values of a checkpoint
def held_block(x):
    """What one block (float64, finite) stands for: the nearest e4m3 value times
    2^e, but no more than the largest of them that is a float32 number."""
    table = code_values()
    e = -117
    while np.abs(x).max() > 448.0 * 2.0 ** e:
        e += 1
    table = table[table * 2.0 ** e < 2.0 ** 128]
    z = np.abs(x) / 2.0 ** e
    lo = np.searchsorted(table, z, side="right") - 1
    hi = np.minimum(lo + 1, len(table) - 1)
    down, up = z - table[lo], table[hi] - z
    pick = np.where((up < down) | ((up == down) & (lo % 2 == 1)), hi, lo)
    return np.copysign(table[pick], x) * 2.0 ** e


BF16_MAX, F32_MAX = (2 - 2.0 ** -7) * 2.0 ** 127, (2 - 2.0 ** -23) * 2.0 ** 127
TOPS = [1.75 * 2.0 ** 127, 1.765625 * 2.0 ** 127, 1.875 * 2.0 ** 127, 1.9296875 * 2.0 ** 127, 1.9375 * 2.0 ** 127, BF16_MAX]


@pytest.mark.parametrize("top", TOPS + [F32_MAX, (1.9375 - 2.0 ** -23) * 2.0 ** 127], ids=lambda t: t.hex())
def test_largest_values_stay_finite(mm, top):
    """Up to the largest finite input a held value is finite and off by at most 2^-4."""
    print(f"[case] checkpoint of {top.hex()}", flush=True)
    rng = np.random.default_rng(61)
    x = rng.standard_normal((32, 32)) * 2.0 ** 120
    x[3, 4], x[17, 30], x[31, 0] = top, -top, top / 2
    for dtype in (F32, BF16) if top in TOPS else (F32,):
        t = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
        saved = mm.muon_checkpoint_write([t])
        want = held_block(np64(t))
        assert np.isfinite(want.astype(np.float32)).all()
        for out in (F32, BF16):
            got = np64(mm.muon_checkpoint_read(saved, dtype=out)[0])
            np.testing.assert_array_equal(got, want)
        assert abs(got[3, 4] - top) <= top / 16 and abs(got[17, 30] + top) <= top / 16
        dy = torch.zeros((32, 8), dtype=BF16, device="cuda")
        dy[3, 0] = dy[17, 1] = 1.0
        G = torch.full((8, 32), math.nan, device="cuda")
        mm.muon_checkpoint_grad([(dy, saved[0], G)])
        np.testing.assert_array_equal(np64(G)[:2], want[[3, 17]])
    # beside them a NaN and infinities stay NaN
    t[5, 5], t[6, 6], t[7, 7] = math.nan, math.inf, -math.inf
    got = np64(mm.muon_checkpoint_read(mm.muon_checkpoint_write([t]))[0])
    assert np.isnan(got[[5, 6, 7], [5, 6, 7]]).all() and np.isnan(got).sum() == 3
