"""muon_qk_norm_rotate and its gradient on the GPU against the float64 formulas
(rotate_ref), element by element within the error that the roundings can make."""
import math

import numpy as np
import pytest
import torch

import rotate_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


def draw(rng, rows, T, heads, dim, scale):
    x = rng.standard_normal((rows, heads, dim)) * scale
    x[T:] = np.nan
    return torch.from_numpy(x.astype(np.float32)).to(BF16).cuda()


def inputs(lengths, heads, kv_heads, dim, behind=0, seed=0, layout="fused"):
    """q, k, and gradients of the outputs; rows behind the last sequence are NaN."""
    rng = np.random.default_rng([11, seed, sum(lengths), heads, dim])
    T = sum(lengths)
    ts = [draw(rng, T + behind, T, h, dim, s) for h, s in ((heads, 3.0), (kv_heads, 0.5), (heads, 0.1), (kv_heads, 0.1))]
    if layout == "fused":
        q, k = torch.cat(ts[:2] + [ts[1]], dim=1).split([heads, kv_heads, kv_heads], dim=1)[:2]
        ts[:2] = [q, k]
    elif layout == "heads":
        ts = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in ts]
    elif layout == "wide":
        for i, x in enumerate(ts):
            big = torch.full((x.shape[0], x.shape[1], dim + 24), math.nan, dtype=BF16, device="cuda")
            big[:, :, 8:8 + dim] = x
            ts[i] = big[:, :, 8:8 + dim]
    w = [(1 + 0.3 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2)]
    return ts, [torch.from_numpy(x).cuda() for x in w]


def host(x, T=None):
    return x[:T].float().cpu().numpy().astype(np.float64)


def close(got, want, err, what):
    bad = ~(np.abs(got - want) <= err)
    worst = np.nanmax(np.abs(got - want) / err) if got.size else 0
    assert got.shape == want.shape and not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {worst:.2f} of the bound"


def check(mm, lengths, heads, kv_heads, dim, rotary=None, norm=True, weights=True, positions=None, behind=0, layout="fused",
          eps=1e-6, seed=0):
    print(f"[case] {lengths} {heads}/{kv_heads} x {dim} R {rotary and rotary.rotary_dim} norm {norm} {layout}", flush=True)
    T = sum(lengths)
    ts, w = inputs(lengths, heads, kv_heads, dim, behind, seed, layout)
    w = w if norm and weights else [None, None]
    p = mm.muon_packing_create(lengths)
    kw = dict(positions=positions, norm=norm, q_weight=w[0], k_weight=w[1], eps=eps)
    outs = mm.muon_qk_norm_rotate(ts[0], ts[1], p, rotary, **kw)
    grads = mm.muon_qk_norm_rotate_backward(ts[2], ts[3], ts[0] if norm else None, ts[1] if norm else None, p, rotary, **kw)
    torch.cuda.synchronize()
    r = rotary or mm.MuonRotary(0)
    at = ref.places(lengths, r.axes) if positions is None else positions.cpu().numpy().reshape(r.axes, -1)[:, :T]
    u = ref.angles(at, r)
    for i, name in enumerate("qk"):
        x, dz = host(ts[i], T), host(ts[2 + i], T)
        wi = None if w[i] is None else w[i].cpu().numpy().astype(np.float64)
        z, e = ref.forward(x, u, r, norm, wi, eps)
        close(host(outs[i], T), z, e, name)
        dx, dw, ex, ew = ref.backward(dz, x, u, r, norm, wi, eps)
        close(host(grads[i], T), dx, ex, "d" + name)
        if wi is not None:
            close(host(grads[2 + i]), dw, ew, f"d_{name}_weight")
        else:
            assert grads[2 + i] is None
        assert (outs[i][T:] == 0).all() and (grads[i][T:] == 0).all()


LENGTHS = [[1], [7], [8], [9], [127], [128], [129], [300, 1, 129], [1, 1, 1], [0, 5, 0], [3, 64, 1, 130, 0, 17]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 64), (4, 2, 128)])
def test_lengths(mm, lengths, heads, kv_heads, dim):
    check(mm, lengths, heads, kv_heads, dim, mm.MuonRotary(dim), behind=3)


SHAPES = [(1, 1, 8, 8), (3, 3, 16, 16), (3, 1, 24, 24), (8, 2, 32, 16), (5, 5, 40, 40), (6, 3, 56, 24), (25, 25, 64, 64),
          (8, 8, 72, 64), (8, 1, 80, 80), (16, 8, 96, 48), (9, 3, 120, 120), (12, 4, 128, 128), (12, 4, 128, 64),
          (300, 7, 64, 64), (1, 40, 128, 8), (2, 2, 128, 0), (7, 3, 8, 0)]


@pytest.mark.parametrize("heads,kv_heads,dim,rotary", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_shapes(mm, heads, kv_heads, dim, rotary, interleaved):
    r = mm.MuonRotary(rotary, interleaved=interleaved)
    for i, layout in enumerate(("plain", "fused", "heads", "wide")):
        check(mm, [20, 1, 33], heads, kv_heads, dim, r, norm=i != 1, weights=i != 2, layout=layout, behind=i)


@pytest.mark.parametrize("interleaved", [False, True])
def test_without_rotation(mm, interleaved):
    check(mm, [20, 40], 4, 2, 64, None)
    check(mm, [20, 40], 4, 2, 64, None, weights=False)
    check(mm, [20, 40], 4, 2, 64, None, norm=False)


def test_many_pieces(mm):
    """More pieces than the backward pass has work-groups."""
    check(mm, [1] * 70 + [4000, 900, 130, 5], 3, 1, 64, mm.MuonRotary(64))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_positions(mm, axes, dtype):
    """Positions of the program's own on several axes, far and negative ones among them, strided."""
    T, rows = 90, 95
    rng = np.random.default_rng(axes)
    at = rng.integers(-3, 1 << 20, size=(axes, rows + 6))
    at[:, 3], at[:, 4], at[:, 5] = (1 << 31) - 1, -(1 << 31), 0
    if dtype == torch.int64:
        at[0, 7], at[-1, 8] = 1 << 33, -(1 << 33)
    p = torch.from_numpy(at).to(dtype).cuda()[:, 2:2 + rows]
    sections = {1: [32], 2: [5, 27], 3: [8, 12, 12], 4: [1, 2, 28, 1]}[axes]
    check(mm, [40, 50], 4, 2, 64, mm.MuonRotary(64, sections=sections), positions=p, behind=5)
    pair_axes = [i % axes for i in range(20)]
    check(mm, [90], 2, 2, 40, mm.MuonRotary(40, pair_axes=pair_axes, interleaved=True), positions=p, behind=5)
    if axes == 1:
        check(mm, [90], 2, 2, 40, mm.MuonRotary(40), positions=p[0], behind=5)
    check(mm, [40, 50], 4, 2, 64, mm.MuonRotary(64, sections=sections), positions=p[:1].expand(axes, rows), behind=5)


def test_frequencies(mm):
    """Frequencies of the program's own: none, negative, whole turns, the largest."""
    f = [0.0, -1.0, 2 * math.pi, math.pi / 2, 1024.0, -1024.0, 1e-300, 1e-5]
    check(mm, [300], 3, 2, 16, mm.MuonRotary(16, frequencies=f))
    q = torch.ones((1, 1, 16), dtype=BF16, device="cuda")
    p = mm.muon_packing_create([1])
    for bad in (math.nan, math.inf, 1025.0, -1e30):
        with pytest.raises(mm.MuonError):
            mm.muon_qk_norm_rotate(q, q.clone(), p, mm.MuonRotary(16, frequencies=[bad] + f[1:]))


def test_sizes_of_values(mm):
    """Heads of zeros, of the largest and of the smallest numbers; NaN and infinities stay in their head."""
    print("[case] sizes of values", flush=True)
    D = 64
    p, r = mm.muon_packing_create([6]), mm.MuonRotary(D)
    x = torch.randn((6, 3, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    plain = x.to(BF16)
    sized = plain.clone()
    sized[0, 0] = 0
    sized[1, 1] = (x[1, 1] * 2.0 ** 100).to(BF16)
    sized[2, 2] = (x[2, 2].sign() * 3.38e38).to(BF16)
    sized[3, 0] = (x[3, 0] * 2.0 ** -100).to(BF16)
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    up = (0.01 * x.flip(0)).to(BF16)
    for eps in (1e-6, 2.0 ** -126, 1e-30):
        kw = dict(q_weight=w, k_weight=w, eps=eps)
        z, zk = mm.muon_qk_norm_rotate(sized, sized, p, r, **kw, q_out=torch.empty_like(sized))
        dx, _, dw, _ = mm.muon_qk_norm_rotate_backward(up, up, sized, sized, p, r, **kw)
        u = ref.angles(ref.places([6]), r)
        want, err = ref.forward(host(sized), u, r, True, host(w), eps)
        close(host(z), want, err, "z")
        assert torch.equal(z, zk)
        want, want_w, err, err_w = ref.backward(host(up), host(sized), u, r, True, host(w), eps)
        fits = np.abs(want) < 3.38e38                    # 1 / sqrt(eps) of a head of zeros may not
        close(np.where(fits, host(dx), 0), np.where(fits, want, 0), err, "dx")
        if eps == 1e-6:
            close(host(dw), want_w, err_w, "dw")
    base = mm.muon_qk_norm_rotate(plain, plain, p, r)[0]
    for bad in (math.nan, math.inf, -math.inf):
        sized = plain.clone()
        sized[4, 1, 7] = bad
        z = mm.muon_qk_norm_rotate(sized, sized, p, r)[0]
        assert torch.isnan(z[4, 1, 7])
        z[4, 1] = base[4, 1]
        assert torch.equal(z, base)


def test_in_place_and_outputs(mm):
    """Inputs as outputs; outputs in a fused buffer, the rest of which stays as it was."""
    print("[case] outputs in place", flush=True)
    H, K, D, T, rows = 4, 2, 64, 69, 80
    p, r = mm.muon_packing_create([64, 5]), mm.MuonRotary(D)
    (q, k, dq, dk), w = inputs([64, 5], H, K, D, behind=rows - T)
    kw = dict(q_weight=w[0], k_weight=w[1])
    z = mm.muon_qk_norm_rotate(q, k, p, r, **kw)
    g = mm.muon_qk_norm_rotate_backward(dq, dk, q, k, p, r, **kw)
    buf = torch.full((rows, H + K + 1, D), 7.0, dtype=BF16, device="cuda")
    views = buf[:, :H], buf[:, H:H + K]
    got = mm.muon_qk_norm_rotate(q, k, p, r, **kw, q_out=views[0], k_out=views[1])
    assert got[0] is views[0] and all(torch.equal(a[:T], b[:T]) for a, b in zip(views, z))
    mm.muon_qk_norm_rotate_backward(dq, dk, q, k, p, r, **kw, dq=views[0], dk=views[1])
    assert all(torch.equal(a[:T], b[:T]) for a, b in zip(views, g))
    assert (buf[T:] == 7).all() and (buf[:, H + K:] == 7).all()
    for up, x in ((True, False), (False, True)):         # over the upstream gradients, over the inputs
        a, b = [t.clone() for t in (dq, dk)], [t.clone() for t in (q, k)]
        to = a if up else b
        mm.muon_qk_norm_rotate_backward(*a, *b, p, r, **kw, dq=to[0], dk=to[1])
        assert all(torch.equal(s[:T], t[:T]) for s, t in zip(to, g))
    fused = torch.cat([q, k], dim=1)
    kept = fused.clone()
    mm.muon_qk_norm_rotate(fused[:, :H], fused[:, H:], p, r, **kw, q_out=fused[:, :H], k_out=fused[:, H:])
    assert torch.equal(fused[:T, :H], z[0][:T]) and torch.equal(fused[:T, H:], z[1][:T])
    assert torch.equal(fused[T:].view(torch.int16), kept[T:].view(torch.int16))
    # without a norm the gradient undoes the rotation up to the roundings, and reads no input
    x = torch.full_like(q, math.nan)
    turned = mm.muon_qk_norm_rotate(dq, dk, p, r, norm=False)
    back = mm.muon_qk_norm_rotate_backward(*turned, x, x[:, :K], p, r, norm=False)
    assert (back[0][:T].float() - dq[:T].float()).abs().max() <= 4 * ref.BF * dq[:T].float().abs().max()


def test_empty(mm):
    print("[case] no tokens", flush=True)
    for lengths in ([], [0, 0]):
        p = mm.muon_packing_create(lengths)
        q = torch.full((3, 2, 64), math.nan, dtype=BF16, device="cuda")
        w = torch.ones(64, device="cuda")
        z = mm.muon_qk_norm_rotate(q, q, p, mm.MuonRotary(64), q_weight=w, k_weight=w)
        assert all((t == 0).all() for t in z)
        g = mm.muon_qk_norm_rotate_backward(q, q, q, q, p, mm.MuonRotary(64), q_weight=w, k_weight=w)
        assert all((t == 0).all() for t in g)


def test_one_weight_only(mm):
    print("[case] a weight of the queries alone", flush=True)
    (q, k, dq, dk), w = inputs([50], 4, 2, 64)
    p, r = mm.muon_packing_create([50]), mm.MuonRotary(64)
    both = mm.muon_qk_norm_rotate_backward(dq, dk, q, k, p, r, q_weight=w[0], k_weight=w[1])
    none = mm.muon_qk_norm_rotate_backward(dq, dk, q, k, p, r)
    one = mm.muon_qk_norm_rotate_backward(dq, dk, q, k, p, r, q_weight=w[0])
    assert torch.equal(one[0], both[0]) and torch.equal(one[2], both[2]) and one[3] is None
    assert torch.equal(one[1], none[1])
    # one weight for both
    shared = mm.muon_qk_norm_rotate_backward(dq, dk, q, k, p, r, q_weight=w[0], k_weight=w[0])
    assert torch.equal(shared[2], both[2]) and not torch.equal(shared[1], both[1])


def test_offsets_past_32_bits(mm):
    """Rows and heads more than 2^31 elements apart."""
    print("[case] far rows and heads", flush=True)
    H, D = 2, 64
    p, r = mm.muon_packing_create([3]), mm.MuonRotary(D)
    buf = torch.zeros((1 << 31) + (1 << 23) + D, dtype=BF16, device="cuda")
    far = buf.as_strided((3, H, D), (1 << 22, 1 << 31, 1))
    (q, _, dq, _), _ = inputs([3], H, H, D)
    far.copy_(q)
    want = mm.muon_qk_norm_rotate(q, q, p, r)[0]
    assert torch.equal(mm.muon_qk_norm_rotate(far, q, p, r)[0], want)
    mm.muon_qk_norm_rotate(q, q, p, r, q_out=far)
    assert torch.equal(far.contiguous(), want) and int(torch.count_nonzero(buf)) <= 3 * H * D


def test_streams_and_graphs(mm):
    """Two captured calls (forward, and backward with a workspace that both graphs' calls share), replayed with
    eager work between, on the capturing stream's and another's."""
    print("[case] captured", flush=True)
    (q, k, dq, dk), w = inputs([300, 77], 6, 3, 64)
    p, r = mm.muon_packing_create([300, 77]), mm.MuonRotary(64)
    kw = dict(q_weight=w[0], k_weight=w[1])
    ws = torch.empty(mm.muon_qk_norm_rotate_backward_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            z = mm.muon_qk_norm_rotate(q, k, p, r, **kw)
            results.append(z + mm.muon_qk_norm_rotate_backward(dq, dk, q, k, p, r, **kw, workspace=ws))
        graphs.append(g)
    for i in range(4):
        for t in (q, k, dq, dk):
            t.mul_(1.0 + 0.25 * i)
        for ts in results:
            for t in ts:
                t.fill_(math.nan)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        want = mm.muon_qk_norm_rotate(q, k, p, r, **kw, stream=side) + mm.muon_qk_norm_rotate_backward(
            dq, dk, q, k, p, r, **kw, workspace=ws, stream=side)
        torch.cuda.synchronize()
        for ts in results:
            assert all(torch.equal(a, b) for a, b in zip(ts, want))


def test_refusals(mm):
    (q, k, dq, dk), w = inputs([20], 4, 2, 64, layout="plain")
    p, r = mm.muon_packing_create([20]), mm.MuonRotary(64)
    pos = torch.zeros((1, 20), dtype=torch.int64, device="cuda")
    bad = [dict(q=q.float()), dict(q=q[:19]), dict(k=k[:, :, :32]), dict(k=k.cpu()), dict(q=q.transpose(0, 1)),
           dict(q=q[:19], k=k[:19]), dict(q_weight=w[0].half()), dict(q_weight=w[0][:32]), dict(k_weight=w[0].cpu()),
           dict(norm=False, q_weight=w[0]), dict(eps=0.0), dict(eps=math.nan), dict(eps=-1.0), dict(eps=math.inf),
           dict(rotary=mm.MuonRotary(72)), dict(positions=pos.float()), dict(positions=pos[:, :19]), dict(positions=pos.cpu()),
           dict(positions=pos.expand(2, 20)), dict(rotary=mm.MuonRotary(64, sections=[16, 16]), positions=pos),
           dict(q_out=q[:, :, :32]), dict(q_out=k), dict(k_out=q[:, :2]), dict(q_out=torch.empty_like(q).cpu()),
           dict(q_out=q.flip(0)[:19]), dict(q_out=dq, k_out=dq[:, 1:3])]
    for change in bad:
        args = dict(q=q, k=k, packing=p, rotary=r, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        args.update(change)
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_qk_norm_rotate(**args)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    for change in (dict(q=None), dict(k=None), dict(d_q_weight=w[1]), dict(q=q[:, :3]), dict(dq=dk), dict(dk=q[:, :2]),
                   dict(q_weight=w[0], workspace=small), dict(q_weight=w[0], d_q_weight=w[0]),
                   dict(q_weight=w[0], k_weight=w[1], d_q_weight=w[1]), dict(d_k_out=dk[:5])):
        args = dict(d_q_out=dq, d_k_out=dk, q=q, k=k, packing=p, rotary=r)
        args.update(change)
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_qk_norm_rotate_backward(**args)
    p.close()
    with pytest.raises(RuntimeError):
        mm.muon_qk_norm_rotate(q, k, p, r)
