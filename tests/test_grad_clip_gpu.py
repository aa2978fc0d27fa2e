"""muon_grad_norm and muon_grad_clip on the GPU against float64."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}      # half a step, relative
TINY = {BF16: 2.0 ** -134, F32: 2.0 ** -150}   # half the smallest step


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


def tensors(sizes, types, seed=0, scale=1.0, shift=0):
    rng = np.random.default_rng([17, seed, len(sizes)])
    out = []
    for i, n in enumerate(sizes):
        x = rng.standard_normal(n + shift) * scale * (1 + i % 3)
        out.append(torch.from_numpy(x.astype(np.float32)).to(types[i % len(types)]).cuda()[shift:])
    return out


def wide(t):
    return t.double().cpu().numpy().astype(np.longdouble).ravel()


def norm_of(grads):
    """The norm in 80 bits, and what float64 sums of n squares may be off: n half steps of the sum."""
    total = sum((wide(g) ** 2).sum() for g in grads) if grads else np.longdouble(0)
    n = sum(g.numel() for g in grads)
    norm = np.sqrt(total)
    return norm, float(norm) * (n + 8) * 2.0 ** -53


def check_clip(mm, grads, max_norm, out_types=None, in_place=False):
    """A clip against the formula; returns the outputs."""
    norm, err = norm_of(grads)
    old = [wide(g) for g in grads]
    # values from here on count every element of a gradient: NaN where the call leaves one out
    outs = None if in_place else [torch.full(g.shape, math.nan, dtype=out_types[i % len(out_types)], device="cuda")
                                  for i, g in enumerate(grads)]
    got = mm.muon_grad_clip(grads, max_norm, outs=outs)
    assert got.dtype == F64 and got.shape == ()
    assert abs(np.longdouble(got.item()) - norm) <= err
    factor = max_norm / norm if norm > max_norm else np.longdouble(1)
    results = grads if in_place else outs
    for x, y in zip(old, results):
        want = x * factor
        # the product rounded to float32, then to out's type; the factor carries the norm's error
        step = HALF[F32] + (HALF[y.dtype] * (1 + HALF[F32]) if y.dtype != F32 else 0.0)
        off = np.abs(wide(y) - want)
        assert (off <= np.abs(want) * (step + 2 * err / max(float(norm), 1e-300)) + TINY[F32] + TINY[y.dtype]).all()
    if not in_place:
        for x, g in zip(old, grads):
            assert (wide(g) == x).all()
    return results


SIZES = [[1], [7], [8], [9], [255, 3], [2048], [8191], [8192], [8193], [3, 0, 5, 8192 * 3 + 1], [65536, 256, 256, 1],
         [100003, 8192, 1, 4096]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F32, BF16)], ids=["f32", "bf16", "both"])
def test_sizes(mm, sizes, types):
    print(f"[case] clip {sizes} {types}", flush=True)
    for shift in (0, 1, 3):
        for outs in ((F32,), (BF16,), (BF16, F32)):
            check_clip(mm, tensors(sizes, types, shift=shift), 0.5, outs)
        check_clip(mm, tensors(sizes, types, shift=shift), 1e6, (F32, BF16))
        check_clip(mm, tensors(sizes, types, shift=shift), 0.5, in_place=True)


def test_many_tensors(mm):
    """More tensors than a launch takes, and more chunks than its work-groups."""
    print("[case] many tensors", flush=True)
    rng = np.random.default_rng(3)
    sizes = [int(n) for n in rng.integers(0, 20000, size=301)]
    check_clip(mm, tensors(sizes, (F32, BF16)), 1.0, (BF16, F32))
    check_clip(mm, tensors(sizes, (F32, BF16)), 1.0, in_place=True)
    big = [5, 8192 * 2100 + 77] + [64] * 200 + [8192 * 4097 + 3]
    check_clip(mm, tensors(big, (BF16, F32)), 1.0, (F32,))


def test_matrices_and_norm_alone(mm):
    print("[case] matrices", flush=True)
    grads = [g.view(37, 11) for g in tensors([407] * 5, (F32, BF16))]
    norm, err = norm_of(grads)
    got = mm.muon_grad_norm(grads)
    assert got.shape == () and abs(np.longdouble(got.item()) - norm) <= err
    into = torch.full((1,), math.nan, dtype=F64, device="cuda")
    assert mm.muon_grad_norm(grads, norm=into) is into and into.item() == got.item()
    # a tensor given twice counts twice
    twice = mm.muon_grad_norm(grads + grads[:1])
    assert abs(np.longdouble(twice.item()) - norm_of(grads + grads[:1])[0]) <= 2 * err
    assert mm.muon_grad_norm([]).item() == 0.0
    assert mm.muon_grad_norm([torch.empty(0, device="cuda")]).item() == 0.0
    assert mm.muon_grad_clip([], 1.0).item() == 0.0
    zero = torch.zeros(100, device="cuda")
    assert mm.muon_grad_clip([zero], 1.0).item() == 0.0 and (zero == 0).all()


def test_norm_given(mm):
    """Two shards: each one's norm, joined by the program, then clipped by the joint one."""
    print("[case] shards", flush=True)
    a, b = tensors([5000, 33], (F32,), seed=1), tensors([70000], (BF16,), seed=2)
    whole = [t.clone() for t in a + b]
    mm.muon_grad_clip(whole, 2.0)
    joint = torch.sqrt(mm.muon_grad_norm(a).square() + mm.muon_grad_norm(b).square())
    assert mm.muon_grad_clip(a, 2.0, norm=joint) is joint
    mm.muon_grad_clip(b, 2.0, norm=joint.view(1))
    for x, y in zip(a + b, whole):
        # the norms may differ by some steps of float64, a value then by one rounding
        assert ((x.double() - y.double()).abs() <= 2 * HALF[x.dtype] * y.double().abs()).all()
    for bad in (math.nan, math.inf, -1.0, 0.0, 1.99):
        kept = [t.clone() for t in a]
        mm.muon_grad_clip(a, 2.0, norm=torch.tensor(bad, dtype=F64, device="cuda"))
        assert all(torch.equal(x, y) for x, y in zip(a, kept))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite(mm, bad):
    """The norm tells, the values stay as they are."""
    print(f"[case] clip with {bad}", flush=True)
    for dtype in (F32, BF16):
        grads = tensors([20000, 9], (dtype,))
        grads[0][12345] = bad
        kept = [g.clone() for g in grads]
        outs = [torch.empty_like(g) for g in grads]
        for norm in (mm.muon_grad_clip(grads, 1.0, outs=outs), mm.muon_grad_clip(grads, 1.0), mm.muon_grad_norm(grads)):
            assert math.isnan(norm.item()) if math.isnan(bad) else norm.item() == math.inf
        for g, k, o in zip(grads, kept, outs):
            assert torch.equal(g.nan_to_num(1.5), k.nan_to_num(1.5)) and torch.equal(o.nan_to_num(1.5), k.nan_to_num(1.5))


def test_range(mm):
    """Squares that float32 cannot hold, on either side."""
    print("[case] largest and smallest values", flush=True)
    top = torch.full((3000,), 3.0e38, device="cuda")
    check_clip(mm, [top], 1.0, (F32,))
    check_clip(mm, [top], 1e37, (F32, BF16))
    low = torch.full((3000,), 1e-40, device="cuda")
    assert (low > 0).all()
    check_clip(mm, [low], 1e-39, (F32,))
    check_clip(mm, [low, top], 1.0, (F32,))
    check_clip(mm, [torch.full((9,), 3.3e38, dtype=BF16, device="cuda")], 1e-30, (F32,))


def test_more_elements_than_32_bits(mm):
    print("[case] 2^31 + 70001 elements", flush=True)
    n = (1 << 31) + 70001
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[5], g[n // 2], g[n - 1] = 3.0, 4.0, 12.0
    norm = mm.muon_grad_clip([g], 6.5)
    assert norm.item() == 13.0
    assert [g[i].item() for i in (5, n // 2, n - 1)] == [1.5, 2.0, 6.0] and int(torch.count_nonzero(g)) == 3


def test_repeats_and_streams(mm):
    """The same bits in every run, on any stream, with a workspace of the caller's or not."""
    print("[case] repeats", flush=True)
    grads = tensors([100000, 8193, 5] * 40, (F32, BF16))
    want = mm.muon_grad_norm(grads).item()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.full((mm.muon_grad_norm_workspace_bytes(),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        for workspace in (None, ws):
            got = mm.muon_grad_norm(grads, workspace=workspace, stream=stream)
            torch.cuda.synchronize()
            assert got.item() == want
    outs = [torch.empty_like(g) for g in grads]
    assert mm.muon_grad_clip(grads, 1.0, outs=outs, stream=side) is not None
    torch.cuda.synchronize()
    kept = [o.clone() for o in outs]
    mm.muon_grad_clip(grads, 1.0, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_captured(mm):
    """Two captured calls that share a workspace, replayed with other work between."""
    print("[case] captured clips", flush=True)
    a, b = tensors([30000, 17], (F32,), seed=5), tensors([8192 * 9 + 1] * 99, (BF16,), seed=6)
    oa, ob = [torch.empty_like(t) for t in a], [torch.empty(t.shape, device="cuda") for t in b]
    ws = torch.empty(mm.muon_grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mm.muon_grad_clip(a, 1.0, outs=oa, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        na = mm.muon_grad_clip(a, 1.0, outs=oa, workspace=ws)
        nb = mm.muon_grad_clip(b, 3.0, outs=ob, workspace=ws)
    for i in range(4):
        for t in a + b:
            t.mul_(1.0 + 0.5 * i)
        for t in oa + ob:
            t.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        ea, eb = [torch.empty_like(t) for t in oa], [torch.empty_like(t) for t in ob]
        assert mm.muon_grad_clip(a, 1.0, outs=ea).item() == na.item()
        assert mm.muon_grad_clip(b, 3.0, outs=eb).item() == nb.item()
        assert all(torch.equal(x, y) for x, y in zip(oa + ob, ea + eb))


def test_refusals(mm):
    g = torch.ones(64, device="cuda")
    for bad in ([g.cpu()], [g.double()], [g[::2]], [g, g], [g, g[32:]]):
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_grad_clip(bad, 1.0)
    for outs in ([], [g[:32]], [g.half()], [g.to(BF16).cpu()], [g.view(8, 8)]):
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_grad_clip([g], 1.0, outs=outs)
    with pytest.raises(mm.MuonError):                                   # in place, of another type
        mm.muon_grad_clip([g], 1.0, outs=[g.view(BF16)[:64]])
    for max_norm in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(mm.MuonError):
            mm.muon_grad_clip([g], max_norm)
    for norm in (g[:1], torch.zeros(2, dtype=F64, device="cuda"), torch.zeros((), dtype=F64)):
        with pytest.raises(ValueError):
            mm.muon_grad_clip([g], 1.0, norm=norm)
        with pytest.raises(ValueError):
            mm.muon_grad_norm([g], norm=norm)
    for ws in (torch.empty(64, dtype=torch.uint8, device="cuda"), torch.empty(1 << 15, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(mm.MuonError):
            mm.muon_grad_norm([g], workspace=ws)
    shared = torch.ones(64, dtype=F64, device="cuda")
    with pytest.raises(mm.MuonError):                                   # the norm inside an output
        mm.muon_grad_clip([g], 1.0, outs=[shared.view(F32)[:64]], norm=shared[3:4])
    assert (g == 1).all()
