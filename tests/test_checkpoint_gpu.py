"""8-bit activation checkpoints on the GPU: held values equal to the format's
definition bit for bit, and the weight gradient against float64 sums of the
held values."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


def code_values():
    """The 127 non-negative finite values of e4m3, by code."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


def held(x):
    """What a checkpoint of x (float64 array of float32 or bfloat16 values) stands for."""
    T, C = x.shape
    table = code_values()
    out = np.empty_like(x)
    for t in range(0, T, 32):
        for c in range(0, C, 32):
            b = x[t:t + 32, c:c + 32]
            fin = np.isfinite(b)
            top = np.abs(b[fin]).max() if fin.any() else 0.0
            e = -117
            while top > 448.0 * 2.0 ** e:
                e += 1
            z = np.where(fin, np.abs(b), 0) / 2.0 ** e
            lo = np.clip(np.searchsorted(table, z, side="right") - 1, 0, 126)
            hi = np.minimum(lo + 1, 126)
            down, up = z - table[lo], table[hi] - z
            pick = np.where((up < down) | ((up == down) & (lo % 2 == 1)), hi, lo)
            v = np.where(fin, np.copysign(table[pick], b) * 2.0 ** e, np.nan)
            out[t:t + 32, c:c + 32] = v
    return out


def activation(tokens, cols, dtype, pad=0, seed=0, special=False):
    rng = np.random.default_rng([11, seed, tokens, cols])
    x = rng.standard_normal((tokens, cols + pad)) * np.exp(rng.standard_normal((1, cols + pad)))
    if special:
        x[:32] *= 1e-30                               # a block row far down
        x[32:64] *= 1e30
        x[64:96, :40] = 0
        x[96:128, :5] = 448.0 * 2.0 ** rng.integers(-3, 3, (x[96:128].shape[0], 5))
        flat = rng.integers(0, tokens, 24), rng.integers(0, cols, 24)
        x[flat] = rng.choice([np.inf, -np.inf, np.nan, -0.0, 3e38, 1e-44], 24)
        # halves between neighbouring codes, at a top of exactly 448
        x[128:160, :32] = np.outer(np.ones(x[128:160].shape[0]), (code_values()[64:96] + code_values()[65:97]) / 2)
        x[128:160, 0] = 448.0
    t = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    return t[:, :cols]


def np64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("tokens,cols", [(1, 1), (1, 300), (31, 33), (32, 32), (33, 31), (64, 256), (100, 257), (5, 700),
                                         (257, 513)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
def test_held_values(mm, tokens, cols, dtype, pad):
    print(f"[case] checkpoint {tokens} x {cols} {dtype} pad {pad}", flush=True)
    x = activation(tokens, cols, dtype, pad)
    want = held(np64(x))
    saved = mm.muon_checkpoint_write([x])
    for out in (BF16, F32):
        got = mm.muon_checkpoint_read(saved, dtype=out)[0]
        assert got.dtype == out
        np.testing.assert_array_equal(np64(got), want)
    # into a padded tensor: the padding stays
    wide = torch.full((tokens, cols + 5), 7.0, dtype=BF16, device="cuda")
    mm.muon_checkpoint_read(saved, xs=[wide[:, 2:2 + cols]])
    np.testing.assert_array_equal(np64(wide[:, 2:2 + cols]), want)
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + cols:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_special_values(mm, dtype):
    print(f"[case] checkpoint special values {dtype}", flush=True)
    x = activation(170, 100, dtype, special=True)
    got = np64(mm.muon_checkpoint_read(mm.muon_checkpoint_write([x]))[0])
    want = held(np64(x))
    np.testing.assert_array_equal(got, want)
    finite = np.isfinite(want)
    np.testing.assert_array_equal(np.signbit(got[finite]), np.signbit(want[finite]))


def test_list_of_activations(mm):
    print("[case] 70 checkpoints in one call", flush=True)
    xs = [activation(1 + 7 * i, 5 + 11 * i, BF16 if i % 2 else F32, seed=i) for i in range(70)]
    xs[3] = xs[3][:0]
    saved = mm.muon_checkpoint_write(xs)
    for x, got in zip(xs, mm.muon_checkpoint_read(saved)):
        np.testing.assert_array_equal(np64(got), held(np64(x)))
    again = mm.muon_checkpoint_write(xs[::-1], saved[::-1])
    for x, got in zip(xs[::-1], mm.muon_checkpoint_read(again, dtype=F32)):
        np.testing.assert_array_equal(np64(got), held(np64(x)))


def upstream(tokens, outs, pad, seed=0):
    rng = np.random.default_rng([12, seed, tokens, outs])
    t = torch.from_numpy((0.01 * rng.standard_normal((tokens, outs + pad))).astype(np.float32)).to(BF16).cuda()
    return t[:, :outs]


def check_grad(dy, x_held, got, old=None):
    """Exact products summed in float32 in any order: at most one half step per
    summand of the sum of magnitudes, then one rounding to G's type."""
    d, g = np64(dy), np64(got)
    want, size = d.T @ x_held, np.abs(d).T @ np.abs(x_held)
    if old is not None:
        want, size = want + old, size + np.abs(old)
    half = 2.0 ** -24 if got.dtype == F32 else 2.0 ** -8
    err = (d.shape[0] + 32) * 2.0 ** -24 * size + half * (1 + half) * np.abs(want) + 1e-38
    bad = ~(np.abs(g - want) <= err)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside"


GRADS = [(1, 1, 1, 0), (1, 300, 33, 0), (31, 7, 64, 0), (32, 256, 256, 0), (33, 255, 300, 0), (100, 257, 31, 3),
         (777, 300, 257, 8), (640, 64, 520, 5), (2100, 130, 260, 0), (3001, 77, 100, 8), (4096, 256, 256, 0),
         (8192, 501, 300, 0), (6000, 520, 270, 8)]  # several tiles, each cut into many shares


@pytest.mark.parametrize("tokens,outs,cols,pad", GRADS)
@pytest.mark.parametrize("g_type", [F32, BF16])
def test_grad(mm, tokens, outs, cols, pad, g_type):
    print(f"[case] gradient {tokens} x {outs} x {cols} pad {pad} {g_type}", flush=True)
    x = activation(tokens, cols, BF16)
    saved = mm.muon_checkpoint_write([x])[0]
    xh = np64(mm.muon_checkpoint_read([saved], dtype=F32)[0])
    dy = upstream(tokens, outs, pad)
    G = torch.full((outs, cols), math.nan, dtype=g_type, device="cuda")
    mm.muon_checkpoint_grad([(dy, saved, G)])
    check_grad(dy, xh, G)
    old = np64(G)
    mm.muon_checkpoint_grad([(dy, saved, G)], accumulate=True)
    check_grad(dy, xh, G, old)


@pytest.mark.parametrize("outs", range(1, 9))
@pytest.mark.parametrize("tokens", [2, 33, 300])
def test_grad_of_narrow_rows(mm, tokens, outs):
    """Rows of a few elements: a 16-byte read spans several of them, and near dY's end none may be one."""
    print(f"[case] gradient {tokens} x {outs} x 40", flush=True)
    x = activation(tokens, 40, BF16)
    saved = mm.muon_checkpoint_write([x])[0]
    xh = np64(mm.muon_checkpoint_read([saved], dtype=F32)[0])
    room = torch.full((tokens * outs + 64,), math.nan, dtype=BF16, device="cuda")
    dy = room[32:32 + tokens * outs].view(tokens, outs)  # NaN before the first element and behind the last
    dy.copy_(upstream(tokens, outs, 0))
    G = torch.empty((outs, 40), device="cuda")
    mm.muon_checkpoint_grad([(dy, saved, G)])
    check_grad(dy, xh, G)


def test_grad_no_tokens(mm):
    saved = mm.muon_checkpoint_write([torch.empty((0, 40), dtype=BF16, device="cuda")])[0]
    G = torch.full((24, 40), 3.0, device="cuda")
    dy = torch.empty((0, 24), dtype=BF16, device="cuda")
    mm.muon_checkpoint_grad([(dy, saved, G)], accumulate=True)
    assert (G == 3).all()
    mm.muon_checkpoint_grad([(dy, saved, G)])
    assert (G == 0).all()


def test_grad_list_shares_a_checkpoint(mm):
    print("[case] 30 gradients in one call", flush=True)
    mats, parts = [], []
    for i in range(10):
        tokens, cols = 40 + 97 * i, 30 + 60 * i
        saved = mm.muon_checkpoint_write([activation(tokens, cols, BF16, seed=i)])[0]
        xh = np64(mm.muon_checkpoint_read([saved], dtype=F32)[0])
        for j, outs in enumerate((16, 72 + i, 300)):
            dy = upstream(tokens, outs, 0, seed=j)
            mats.append((dy, saved, torch.empty((outs, cols), device="cuda", dtype=F32 if j else BF16)))
            parts.append(xh)
    mm.muon_checkpoint_grad(mats)
    first = [g.clone() for _, _, g in mats]
    for (dy, _, g), xh in zip(mats, parts):
        check_grad(dy, xh, g)
    mm.muon_checkpoint_grad(mats)
    assert all(torch.equal(a, g) for a, (_, _, g) in zip(first, mats))


def test_grad_keeps_other_rows_out(mm):
    """Rows of dY and x past the tokens, and columns past the widths, are never summed."""
    tokens, outs, cols = 45, 70, 90
    x = torch.full((64, 128), math.nan, dtype=BF16, device="cuda")
    dy = torch.full((64, 96), math.nan, dtype=BF16, device="cuda")
    x[:tokens, :cols] = activation(tokens, cols, BF16)
    dy[:tokens, :outs] = upstream(tokens, outs, 0)
    saved = mm.muon_checkpoint_write([x[:tokens, :cols]])[0]
    xh = np64(mm.muon_checkpoint_read([saved], dtype=F32)[0])
    G = torch.empty((outs, cols), device="cuda")
    mm.muon_checkpoint_grad([(dy[:tokens, :outs], saved, G)])
    check_grad(dy[:tokens, :outs], xh, G)
    # a NaN or infinity inside reaches its own row or column of G only
    inside = dy[:tokens, :outs].clone()
    inside[tokens - 1, 5] = math.inf
    mm.muon_checkpoint_grad([(inside, saved, G)])
    bad = ~torch.isfinite(G)
    assert bad[5].all() and bad.sum() == cols
