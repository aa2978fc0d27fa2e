"""The weights' gradients of muon_qk_norm_rotate over long sums: float32 runs
stay short however many tokens and heads there are, so the error stays that of
rotate_ref.backward (64 terms of a run, then float64)."""
import numpy as np
import pytest
import torch

import rotate_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


# many short sequences; long ones; more heads than a run has terms in one piece
@pytest.mark.parametrize("lengths,heads,dim,rotary", [([8] * 4096, 64, 128, 8), ([8] * 8192, 32, 128, 128), ([16384] * 4, 64, 64, 40),
                                                      ([300, 20], 4096, 128, 8), ([61], 4096, 128, 128)],
                         ids=["short", "short-wide", "long", "heads", "heads-wide"])
def test_terms_of_one_sign(mm, lengths, heads, dim, rotary):
    """Every token and head adds the same products, where float32 sums drift one way: at position 0 the gradient
    is their number times one head's."""
    print(f"[case] {len(lengths)} x {lengths[0]} {heads} x {dim} R {rotary}", flush=True)
    T, n = sum(lengths), sum(lengths) * heads
    rng = np.random.default_rng([23, heads, dim, rotary])
    x, dz = (torch.from_numpy(rng.standard_normal(dim).astype(np.float32) * s).to(BF16).cuda() for s in (3.0, 0.1))
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(dim)).astype(np.float32)).cuda()
    p, r = mm.muon_packing_create(lengths), mm.MuonRotary(rotary)
    at = torch.zeros(T, dtype=torch.int32, device="cuda")
    q, up = x.expand(T, heads, dim), dz.expand(T, heads, dim)
    got = mm.muon_qk_norm_rotate_backward(up, up[:, :1], q, q[:, :1], p, r, positions=at, q_weight=w, k_weight=w)
    one = [t.float().cpu().numpy().astype(np.float64).reshape(1, 1, dim) for t in (dz, x)]
    dx, dw, _, ew = ref.backward(*one, ref.angles(np.zeros((1, 1), dtype=np.int64), r), r, True, w.cpu().numpy(), 1e-6)
    for name, terms, d in (("d_q_weight", n, got[2]), ("d_k_weight", T, got[3])):
        off = np.abs(d.cpu().numpy().astype(np.float64) - terms * dw) / (terms * ew)
        assert (off <= 1).all(), f"{name}: {(off > 1).sum()} of {dim} outside, worst {off.max():.2f} of the bound"
    assert torch.equal(got[0], got[0][:1, :1].expand(T, heads, dim))
    again = mm.muon_qk_norm_rotate_backward(up, up[:, :1], q, q[:, :1], p, r, positions=at, q_weight=w, k_weight=w)
    assert torch.equal(again[2], got[2]) and torch.equal(again[3], got[3])
