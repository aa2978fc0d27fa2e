"""muon_attention and muon_attention_backward on the GPU against the float64
formulas (attention_ref), element by element within the error that the
kernels' roundings can make."""
import math

import numpy as np
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


def inputs(lengths, heads, kv_heads, dim, behind=0, seed=0, sharp=2.0, layout="fused"):
    """q, k, v, do as bfloat16 GPU tensors.  Rows behind the last sequence are NaN."""
    rng = np.random.default_rng([7, seed, sum(lengths), heads, dim])
    T = sum(lengths)
    rows = T + behind

    def draw(h, scale):
        x = rng.standard_normal((rows, h, dim)) * scale
        x[T:] = np.nan
        return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()

    q, k, v, do = draw(heads, sharp), draw(kv_heads, 1.0), draw(kv_heads, 1.0), draw(heads, 0.1)
    if layout == "fused":      # views of one projection output
        both = torch.cat([q, k, v], dim=1)
        q, k, v = both[:, :heads], both[:, heads:heads + kv_heads], both[:, heads + kv_heads:]
    elif layout == "heads":    # head-major buffers
        q, k, v, do = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, do))
    elif layout == "wide":     # padded rows and heads
        def widen(x):
            big = torch.full((x.shape[0], x.shape[1], x.shape[2] + 24), math.nan, dtype=x.dtype, device=x.device)
            big[:, :, 8:8 + x.shape[2]] = x
            return big[:, :, 8:8 + x.shape[2]]
        q, k, v, do = (widen(x) for x in (q, k, v, do))
    return q, k, v, do


def host(x, T):
    return x[:T].float().cpu().numpy().astype(np.float64)


def close(got, want, err, what):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= err)
    worst = np.nanmax(np.where(err > 0, np.abs(got - want) / np.where(err > 0, err, 1), 0)) if got.size else 0
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {worst:.2f} of the bound"


def check_forward(mm, lengths, heads, kv_heads, dim, behind=0, layout="fused", seed=0, scale=None, sharp=2.0):
    print(f"[case] forward {lengths} {heads}/{kv_heads} x {dim} {layout}", flush=True)
    T = sum(lengths)
    q, k, v, _ = inputs(lengths, heads, kv_heads, dim, behind, seed, sharp, layout)
    top = torch.full((heads,), -math.inf, device="cuda")
    o, lse = mm.muon_attention(q, k, v, mm.muon_packing_create(lengths), scale=scale, max_logit=top)
    torch.cuda.synchronize()
    sc = dim ** -0.5 if scale is None else scale
    ro, rl, rt, eo, el, et = ref.forward(host(q, T), host(k, T), host(v, T), lengths, sc)
    close(host(o, T), ro, eo, "o")
    close(lse[:, :T].cpu().numpy(), rl, el, "lse")
    close(top.cpu().numpy(), rt, et, "max_logit")
    assert (o[T:] == 0).all() and (lse[:, T:] == 0).all()


def check_backward(mm, lengths, heads, kv_heads, dim, behind=0, layout="fused", seed=0, sharp=2.0):
    print(f"[case] backward {lengths} {heads}/{kv_heads} x {dim} {layout}", flush=True)
    T = sum(lengths)
    q, k, v, do = inputs(lengths, heads, kv_heads, dim, behind, seed, sharp, layout)
    packing = mm.muon_packing_create(lengths)
    o, lse = mm.muon_attention(q, k, v, packing)
    dq, dk, dv = mm.muon_attention_backward(do, q, k, v, o, lse, packing)
    torch.cuda.synchronize()
    r = ref.backward(host(do, T), host(q, T), host(k, T), host(v, T), host(o, T), lse[:, :T].cpu().numpy(), lengths,
                     dim ** -0.5)
    for name, got, want, err in zip(("dq", "dk", "dv"), (dq, dk, dv), r[:3], r[3:]):
        close(host(got, T), want, err, name)
        assert (got[T:] == 0).all(), name


LENGTHS = [[1], [2], [31], [32], [33], [63], [64], [65], [127], [128], [129], [200], [257], [1, 1, 1], [0, 5, 0],
           [3, 64, 1, 130, 0, 17], [300, 1, 129]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 64), (4, 2, 128)])
def test_forward_lengths(mm, lengths, heads, kv_heads, dim):
    check_forward(mm, lengths, heads, kv_heads, dim, behind=3)


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 64), (4, 2, 128)])
def test_backward_lengths(mm, lengths, heads, kv_heads, dim):
    check_backward(mm, lengths, heads, kv_heads, dim, behind=3)


SHAPES = [(1, 1, 8), (3, 3, 16), (3, 1, 24), (8, 2, 32), (5, 5, 40), (6, 3, 56), (25, 25, 64), (8, 8, 72), (8, 1, 80),
          (16, 8, 96), (9, 3, 120), (12, 4, 128)]


@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
@pytest.mark.parametrize("layout", ["plain", "fused", "heads", "wide"])
def test_layouts(mm, heads, kv_heads, dim, layout):
    check_forward(mm, [70, 1, 150], heads, kv_heads, dim, layout=layout)
    check_backward(mm, [70, 1, 150], heads, kv_heads, dim, layout=layout)


def test_many_tiles(mm):
    """More key tiles than the pair kernel takes (heads of 64 and fewer)."""
    lengths = [1, 130, 40, 0, 257, 64, 128, 33] * 6
    check_forward(mm, lengths, 10, 10, 64)
    check_backward(mm, lengths, 10, 10, 64, behind=2)
    check_backward(mm, lengths, 16, 8, 40)
    check_backward(mm, lengths, 20, 10, 40, behind=1)
    check_backward(mm, lengths, 27, 9, 64, layout="fused")


@pytest.mark.parametrize("lengths", [[1025], [1100, 3, 64], [1151, 0, 1], [2000]], ids=str)
@pytest.mark.parametrize("heads,kv_heads,dim", [(3, 3, 64), (4, 2, 128), (2, 1, 40), (2, 2, 104)])
def test_split_keys(mm, lengths, heads, kv_heads, dim):
    """Few rows of long sequences: their keys are split over two wave groups."""
    check_forward(mm, lengths, heads, kv_heads, dim, behind=1, sharp=4.0)
    check_backward(mm, lengths, heads, kv_heads, dim, behind=1)


def test_long_sequence(mm):
    check_forward(mm, [1500, 700], 4, 1, 128)
    check_backward(mm, [1500, 700], 4, 1, 128)
    check_forward(mm, [2100], 2, 2, 64)
    check_backward(mm, [2100], 2, 2, 64)
