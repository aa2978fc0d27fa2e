"""The tests' float64 formulas of the norms and rotations: the gradient against
differences, the rotation against complex products (no GPU)."""
import numpy as np
import pytest

import matrix_muon_step_amd as mm
import rotate_ref as ref


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D,R", [(8, 8), (24, 16), (16, 0)])
def test_gradient_against_differences(D, R, interleaved, norm):
    rng = np.random.default_rng(D + R)
    rotary = mm.MuonRotary(R, interleaved=interleaved)
    x, dz = rng.standard_normal((5, 3, D)), rng.standard_normal((5, 3, D))
    w = 1 + 0.3 * rng.standard_normal(D) if norm else None
    u = ref.angles(ref.places([3, 2]), rotary)
    dx, dw, _, _ = ref.backward(dz, x, u, rotary, norm, w, 1e-3)

    def loss(x, w):
        return (ref.forward(x, u, rotary, norm, w, 1e-3)[0] * dz).sum()

    h = 1e-5
    for t, a, d in ((0, 0, 0), (1, 2, 3), (4, 1, D - 1), (2, 0, D // 2)):
        e = np.zeros_like(x)
        e[t, a, d] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[t, a, d]) < 1e-7
    if norm:
        for d in (0, D // 2, D - 1):
            e = np.zeros(D)
            e[d] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[d]) < 1e-7


def test_rotation_is_a_complex_product():
    rotary = mm.MuonRotary(8, base=100.0, interleaved=True)
    x = np.random.default_rng(0).standard_normal((3, 2, 8))
    p = np.array([[0, 7, -123456789012]])
    z = ref.turn(x, ref.angles(p, rotary), rotary)
    want = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * np.outer(p[0].astype(np.longdouble), 100.0 ** -(np.arange(4) / 4))[:, None])
    assert np.abs(z[:2, ..., 0::2] - want.real[:2]).max() < 1e-12 and np.abs(z[:2, ..., 1::2] - want.imag[:2]).max() < 1e-12
    assert np.abs(np.abs(want[2]) - np.hypot(z[2, ..., 0::2], z[2, ..., 1::2])).max() < 1e-12


def test_rotary_arguments():
    r = mm.MuonRotary(16, sections=[2, 0, 6])
    assert r.axes == 3 and r.pair_axes == (0, 0, 2, 2, 2, 2, 2, 2) and r.frequencies[1] == 10000.0 ** (-1 / 8)
    assert mm.MuonRotary(8, pair_axes=[0, 1, 0, 1]).axes == 2
    assert mm.MuonRotary(0).axes == 1
    for bad in (dict(rotary_dim=12), dict(rotary_dim=136), dict(rotary_dim=-8), dict(rotary_dim=8, frequencies=[1.0]),
                dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, base=float("nan")), dict(rotary_dim=8, sections=[4, 1]),
                dict(rotary_dim=8, sections=[5, -1]), dict(rotary_dim=8, sections=[]), dict(rotary_dim=8, pair_axes=[0, 1]),
                dict(rotary_dim=8, pair_axes=[0, 1, 2, -1]), dict(rotary_dim=8, sections=[4], pair_axes=[0] * 4),
                dict(rotary_dim=16, sections=[2, 2, 2, 1, 1]), dict(rotary_dim=8.5)):
        with pytest.raises(ValueError):
            mm.MuonRotary(**bad)
    with pytest.raises(mm.MuonError):
        mm.muon_qk_norm_rotate_backward_workspace_bytes(12)
    with pytest.raises(mm.MuonError):
        mm.muon_qk_norm_rotate_backward_workspace_bytes(136)
