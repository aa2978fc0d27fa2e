"""muon_qk_norm_rotate and its gradient on tensors of more than 256 MiB, which
are written past the caches: every element against the float64 formulas of
rotate_ref, formed on the GPU."""
import math

import pytest
import torch

import rotate_ref as ref

pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64
LARGE = 256 << 20
EPS = 1e-6


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


def turn(x, u, rotary, back=False):
    lo, hi = ref.pairs_of(rotary)
    c, s = torch.cos(u)[:, None], torch.sin(u)[:, None] * (-1 if back else 1)
    z = x.clone()
    z[..., lo] = x[..., lo] * c - x[..., hi] * s
    z[..., hi] = x[..., hi] * c + x[..., lo] * s
    return z


def both(x, rotary):
    lo, hi = ref.pairs_of(rotary)
    e = x.abs()
    z = e.clone()
    z[..., lo] = z[..., hi] = e[..., lo] + e[..., hi]
    return z


def inside(got, want, err, what):
    off = ((got.double() - want).abs() / err).amax().item()     # NaN where an element is
    assert off <= 1, f"{what}: worst {off:.2f} of the bound"


def check_forward(z, x, u, r, w, what):
    """As rotate_ref.forward; w None: no norm."""
    x, D = x.double(), x.shape[-1]
    y = x if w is None else x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.double()
    want = turn(y, u, r)
    inside(z, want, (D + 20) * ref.F32 * both(y, r) + ref.BF * (1 + 2 * ref.BF) * want.abs() + 2.0 ** -133, what)


def check_backward(dx, dw, dz, x, u, r, w, what):
    """As rotate_ref.backward."""
    dz, D = dz.double(), dz.shape[-1]
    g, spread = turn(dz, u, r, back=True), both(dz, r)
    if w is None:
        inside(dx, g, 10 * ref.F32 * spread + ref.BF * (1 + 2 * ref.BF) * g.abs() + 2.0 ** -133, "d" + what)
        return
    x, w = x.double(), w.double()
    root = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
    n, rel = x * root, (D + 20) * ref.F32
    want = root * (w * g - n * (w * g * n).mean(dim=-1, keepdim=True))
    size = ((w * n).abs() * spread).mean(dim=-1, keepdim=True)
    err = root * (w.abs() * (10 * ref.F32 * spread + rel * g.abs()) + n.abs() * (2 * rel + 10 * ref.F32) * size)
    inside(dx, want, err + ref.BF * (1 + 2 * ref.BF) * want.abs() + 2.0 ** -133, "d" + what)
    want = (g * n).sum(dim=(0, 1))
    err = ((10 * ref.F32 * spread + (rel + 64 * ref.F32) * g.abs()) * n.abs()).sum(dim=(0, 1))
    inside(dw, want, err + 2 * ref.F32 * want.abs() + 1e-30, f"d_{what}_weight")


# 16-byte and 8-byte runs of a lane, heads that are turned in part
@pytest.mark.parametrize("heads,kv_heads,dim,rotary", [(24, 8, 128, 128), (60, 28, 40, 24)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_more_than_the_caches(mm, heads, kv_heads, dim, rotary, interleaved, norm):
    print(f"[case] {heads}/{kv_heads} x {dim} R {rotary} interleaved {interleaved} norm {norm}", flush=True)
    lengths = [16000, 0, 1, 130, 3001]
    T, rows = sum(lengths), sum(lengths) + 3
    assert 2 * T * (heads + kv_heads) * dim * 2 > LARGE
    gen = torch.Generator(device="cuda").manual_seed(heads + rotary)

    def draw(h, scale):
        x = (scale * torch.randn((rows, h, dim), generator=gen, device="cuda")).to(BF16)
        x[T:] = math.nan
        return x

    q, k, dq, dk = draw(heads, 3.0), draw(kv_heads, 0.5), draw(heads, 0.1), draw(kv_heads, 0.1)
    w = [1 + 0.3 * torch.randn(dim, generator=gen, device="cuda") if norm else None for _ in range(2)]
    p, r = mm.muon_packing_create(lengths), mm.MuonRotary(rotary, interleaved=interleaved)
    kw = dict(norm=norm, q_weight=w[0], k_weight=w[1], eps=EPS)
    z = mm.muon_qk_norm_rotate(q, k, p, r, **kw)
    g = mm.muon_qk_norm_rotate_backward(dq, dk, q if norm else None, k if norm else None, p, r, **kw)
    place = torch.cat([torch.arange(n, device="cuda") for n in lengths])
    u = place.double()[:, None] * torch.tensor(r.frequencies, dtype=F64, device="cuda")
    for i, (what, x, up) in enumerate((("q", q, dq), ("k", k, dk))):
        check_forward(z[i][:T], x[:T], u, r, w[i], what)
        check_backward(g[i][:T], g[2 + i], up[:T], x[:T], u, r, w[i], what)
        assert (z[i][T:] == 0).all() and (g[i][T:] == 0).all()
    # the same bits over the inputs, whose rows behind the last sequence stay
    again = [t.clone() for t in (dq, dk)]
    mm.muon_qk_norm_rotate_backward(*again, q, k, p, r, **kw, dq=again[0], dk=again[1])
    mm.muon_qk_norm_rotate(q, k, p, r, **kw, q_out=q, k_out=k)
    for got, want in zip([q, k] + again, z + g[:2]):
        assert torch.equal(got[:T], want[:T]) and torch.isnan(got[T:]).all()
