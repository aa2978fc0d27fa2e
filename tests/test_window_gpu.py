"""Attention with a window and first tokens that stay visible, and its backward
pass, on the GPU against the float64 formulas (window_ref), element by element
within the error that the kernels' roundings can make."""
import math

import numpy as np
import pytest
import torch

import window_ref as ref
from test_attention_gpu import close, host, inputs

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


def check(mm, lengths, heads, kv_heads, dim, window, sinks, behind=0, layout="fused", seed=0, sharp=2.0, backward=True):
    print(f"[case] {lengths} {heads}/{kv_heads} x {dim} window {window} sinks {sinks} {layout}", flush=True)
    T, scale = sum(lengths), dim ** -0.5
    q, k, v, do = inputs(lengths, heads, kv_heads, dim, behind, seed, sharp, layout)
    packing = mm.muon_packing_create(lengths)
    top = torch.full((heads,), -math.inf, device="cuda")
    o, lse = mm.muon_attention(q, k, v, packing, max_logit=top, window=window, sinks=sinks)
    torch.cuda.synchronize()
    r = ref.forward(host(q, T), host(k, T), host(v, T), lengths, scale, window, sinks)
    close(host(o, T), r[0], r[3], "o")
    close(lse[:, :T].cpu().numpy(), r[1], r[4], "lse")
    close(top.cpu().numpy(), r[2], r[5], "max_logit")
    assert (o[T:] == 0).all() and (lse[:, T:] == 0).all()
    if not backward:
        return
    grads = mm.muon_attention_backward(do, q, k, v, o, lse, packing, window=window, sinks=sinks)
    torch.cuda.synchronize()
    r = ref.backward(host(do, T), host(q, T), host(k, T), host(v, T), host(o, T), lse[:, :T].cpu().numpy(), lengths, scale,
                     window, sinks)
    for name, got, want, err in zip(("dq", "dk", "dv"), grads, r[:3], r[3:]):
        close(host(got, T), want, err, name)
        assert (got[T:] == 0).all(), name


LENGTHS = [[1], [2], [33], [64], [65], [129], [200], [257], [0, 5, 0], [3, 64, 1, 130, 0, 17], [300, 1, 129]]
WINDOWS = [(1, 0), (1, 3), (2, 1), (31, 0), (64, 4), (65, 64), (100, 33), (130, 0), (17, 128)]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 64), (4, 2, 128)])
def test_lengths(mm, lengths, heads, kv_heads, dim):
    for window, sinks in WINDOWS:
        check(mm, lengths, heads, kv_heads, dim, window, sinks, behind=3)


@pytest.mark.parametrize("window", [1, 5, 63, 64, 65, 127, 128, 129, 191, 192, 193, 400, 449, 450])
@pytest.mark.parametrize("sinks", [0, 1, 4, 32, 40, 64, 65, 97, 128])
def test_windows(mm, window, sinks):
    check(mm, [450, 190], 2, 1, 64, window, sinks)
    check(mm, [450, 190], 2, 1, 128, window, sinks)


SHAPES = [(1, 1, 8), (3, 1, 24), (8, 2, 32), (5, 5, 40), (25, 25, 64), (8, 8, 72), (8, 1, 80), (16, 8, 96), (9, 3, 120),
          (12, 4, 128)]


@pytest.mark.parametrize("heads,kv_heads,dim", SHAPES)
@pytest.mark.parametrize("layout", ["plain", "fused", "heads", "wide"])
def test_layouts(mm, heads, kv_heads, dim, layout):
    check(mm, [70, 1, 150], heads, kv_heads, dim, 40, 3, layout=layout, behind=1)


@pytest.mark.parametrize("lengths", [[1023], [1024], [1025], [2049, 3, 1100], [3000]], ids=str)
@pytest.mark.parametrize("heads,kv_heads,dim", [(3, 3, 64), (4, 1, 128), (2, 1, 40)])
def test_several_chunks(mm, lengths, heads, kv_heads, dim):
    """Sequences whose rows beyond the window fill several work items of the first tokens' gradients."""
    for window, sinks in ((5, 4), (300, 40), (1000, 128), (1024, 1), (1025, 70)):
        check(mm, lengths, heads, kv_heads, dim, window, sinks, sharp=1.0)


def test_split_keys(mm):
    """Few rows of long sequences with wide windows: their keys are split over two wave groups."""
    for dim, kv in ((64, 2), (128, 1), (40, 2), (104, 1)):
        for window, sinks in ((900, 4), (1100, 0), (1100, 128), (1300, 65)):
            check(mm, [2300, 5], 2, kv, dim, window, sinks, behind=1, sharp=3.0)


def test_many_tiles(mm):
    """More key tiles than the pair kernel takes (heads of 64 and fewer)."""
    lengths = [1, 130, 40, 0, 257, 64, 128, 33] * 6
    for window, sinks in ((20, 2), (100, 40), (128, 0)):
        check(mm, lengths, 10, 10, 64, window, sinks)
        check(mm, lengths, 20, 10, 40, window, sinks, behind=1)


@pytest.mark.parametrize("dim", [64, 40])
def test_many_tiles_of_long_sequences(mm, dim):
    """The same with sums of the first tokens that are joined, and some that are not."""
    check(mm, [3000, 7, 400], 14, 14, dim, 90, 4, sharp=1.0)
    check(mm, [2600], 17, 17, dim, 300, 70, behind=1, sharp=1.0)


def test_windows_that_hide_nothing(mm):
    """muon_attention's bits, with any number of first tokens."""
    print("[case] windows over everything", flush=True)
    lens = [300, 7, 129]
    q, k, v, do = inputs(lens, 4, 2, 64)
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(q, k, v, p)
    want = (o, lse) + mm.muon_attention_backward(do, q, k, v, o, lse, p)
    for window, sinks in ((300, 0), (301, 4), (1 << 40, 128), (None, 4)):
        o, lse = mm.muon_attention(q, k, v, p, window=window, sinks=sinks)
        got = (o, lse) + mm.muon_attention_backward(do, q, k, v, o, lse, p, window=window, sinks=sinks)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_that_see_themselves(mm):
    """A window of one: o is v, lse the row's own logit, and only v has a gradient beyond rounding."""
    print("[case] window 1", flush=True)
    lens = [140, 1]
    q, k, v, do = inputs(lens, 4, 2, 64)
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(q, k, v, p, window=1)
    assert torch.equal(o, v.repeat_interleave(2, dim=1))
    dq, dk, dv = mm.muon_attention_backward(do, q, k, v, o, lse, p, window=1)
    # ds is p times the difference of two float32 sums of the same 64 products
    size = (do.float().abs() * o.float().abs()).sum(dim=2) * 66 * 2.0 ** -23
    assert (dq.float().abs() <= 1.02 * 64 ** -0.5 * size[..., None] * k.float().abs().repeat_interleave(2, dim=1) + 1e-30).all()
    want = do.float().view(141, 2, 2, 64).sum(dim=2)
    assert ((dv.float() - want).abs() <= 2.0 ** -7 * do.float().abs().view(141, 2, 2, 64).sum(dim=2)).all()


def test_repeats_and_isolation(mm):
    """The same bits in every run; values that are not finite stay in their sequence, and those of hidden keys'
    k leave rows that do not see them as they are."""
    print("[case] repeats and isolation", flush=True)
    lens, window, sinks = [500, 330, 700], 100, 5
    q, k, v, do = inputs(lens, 4, 2, 128, layout="plain")
    p = mm.muon_packing_create(lens)

    def run(q, k, v, do):
        o, lse = mm.muon_attention(q, k, v, p, window=window, sinks=sinks)
        return (o, lse.t()) + mm.muon_attention_backward(do, q, k, v, o, lse, p, window=window, sinks=sinks)

    want = run(q, k, v, do)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, run(q, k, v, do)))
    for bad in (math.nan, math.inf):
        x = [t.clone() for t in (q, k, v, do)]
        for t in x:
            t[620, :, 5] = bad
        got = run(*x)
        for rows in (slice(0, 500), slice(830, 1530)):
            assert all(torch.equal(a[rows], b[rows]) for a, b in zip(want, got))
        assert not torch.isfinite(got[0][620]).all()
    x = k.clone()
    x[600] = math.nan                        # row 100 of the second sequence: seen by its rows 100 to 199
    o, lse = mm.muon_attention(q, x, v, p, window=window, sinks=sinks)
    for rows in (slice(500, 600), slice(700, 830)):
        assert torch.equal(o[rows], want[0][rows]) and torch.equal(lse.t()[rows], want[1][rows])
    assert torch.isnan(o[600:700]).all()


def test_max_logit_is_of_visible_pairs(mm):
    print("[case] max_logit", flush=True)
    q = torch.ones((300, 2, 64), dtype=BF16, device="cuda")
    k = torch.ones((300, 1, 64), dtype=BF16, device="cuda")
    k[:, :, 0] = torch.linspace(0, -30, 300, device="cuda").to(BF16)[:, None]
    k[10] = 50.0                             # seen by rows 10 to 19
    q[10:20] = -1.0
    p = mm.muon_packing_create([300])
    for sinks, want in ((0, 63.0), (11, 3200.0)):
        top = torch.full((1,), -math.inf, device="cuda")
        mm.muon_attention(q, k, k, p, scale=1.0, max_logit=top, window=10, sinks=sinks)
        s = (q[:, 0].double() @ k[:, 0].double().t()).cpu().numpy()
        assert abs(top.item() - s[ref.seen(300, 10, sinks)].max()) <= 1e-2 and top.item() >= want - 64


def test_max_logit_of_many_items(mm):
    """Joined in the workspace: the largest of several calls, per head and per group, NaN and infinities among them,
    with a workspace or (through the C interface) without."""
    print("[case] max_logit of many items", flush=True)
    import ctypes

    from matrix_muon_step_amd import binding as bd
    lens, H, K, D, window, sinks = [700, 1, 300, 129], 60, 20, 64, 50, 2
    q, k, v, _ = inputs(lens, H, K, D, layout="plain")
    q[710, 7, 3] = math.nan
    q[5, 8], k[3, 2] = 0, 1.0
    q[5, 8, 0], k[3, 2, 0] = math.inf, 1.0               # row 5 sees key 3: +infinity
    p = mm.muon_packing_create(lens)
    T = sum(lens)
    want = np.array([ref.logits(host(q, T)[r, h], host(k, T)[r, h // 3], D ** -0.5, ref.seen(n, window, sinks)).max()
                     for h in range(H) for r, n in list(ref.spans(lens))]).reshape(H, -1)
    want = np.where(np.isnan(want).any(axis=1), np.nan, want.max(axis=1))
    err = 4 * 66 * 2.0 ** -24 * np.abs(np.nan_to_num(want, posinf=0.0)) + 1e-3
    o, lse = torch.empty_like(q), torch.empty((H, T), device="cuda")
    for entries, expect in ((H, want), (K, want.reshape(K, 3).max(axis=1))):
        for start in (-math.inf, 5.0):
            top = torch.full((entries,), start, device="cuda")
            mm.muon_attention(q, k, v, p, max_logit=top, window=window, sinks=sinks, o=o, lse=lse)
            again = torch.full((entries,), start, device="cuda")
            args = bd.muon_attention_t(*[bd._heads_tensor("", t, T, None)[0] for t in (q, k, v, o)], lse.data_ptr(), T,
                                       again.data_ptr(), entries, H, K, D, D ** -0.5)
            assert mm.lib().muon_window_attention_workspace_bytes(ctypes.byref(args), window, sinks, ctypes.c_void_p(p._h)) > 0
            assert mm.lib().muon_window_attention(ctypes.byref(args), window, sinks, ctypes.c_void_p(p._h), None, 0,
                                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == mm.MUON_OK
            torch.cuda.synchronize()
            assert torch.equal(top.view(torch.int32), again.view(torch.int32))
            got, w = top.cpu().numpy().astype(np.float64), np.fmax(expect, start)
            w = np.where(np.isnan(expect), np.nan, w)
            assert (np.isnan(got) == np.isnan(w)).all() and (np.isposinf(got) == np.isposinf(w)).all()
            fine = np.isfinite(w)
            e = err.reshape(entries, -1).max(axis=1)
            assert (np.abs(got[fine] - w[fine]) <= e[fine]).all()


def test_streams_and_graphs(mm):
    """Captured forward and backward calls of two layers that share a workspace, replayed with eager work between."""
    print("[case] captured", flush=True)
    lens, kw = [1500, 77], dict(window=60, sinks=3)
    q, k, v, do = inputs(lens, 4, 2, 64)
    p = mm.muon_packing_create(lens)
    ws = torch.empty(mm.muon_attention_backward_workspace_bytes(q, k, p, **kw), dtype=torch.uint8, device="cuda")
    assert ws.numel() > mm.muon_attention_backward_workspace_bytes(q, k, p)

    def layer(stream=None):
        o, lse = mm.muon_attention(q, k, v, p, **kw, stream=stream)
        return (o, lse) + mm.muon_attention_backward(do, q, k, v, o, lse, p, **kw, workspace=ws, stream=stream)

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer()
        graphs.append((g, out))
    side = torch.cuda.Stream()
    for i in range(4):
        for t in (q, k, v, do):
            t.mul_(1.0 + 0.1 * i)
        ws.fill_(255)
        for g, out in graphs:
            for t in out:
                t.fill_(math.nan)
            g.replay()
        torch.cuda.synchronize()
        want = layer(side)
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_far_offsets(mm):
    """Key rows more than 2^31 elements behind the first ones, which stay visible."""
    print("[case] offsets past 32 bits", flush=True)
    n, D, stride = 1100, 64, 1 << 21
    q, k, v, do = inputs([n], 1, 1, D, layout="plain")
    buf = torch.empty(n * stride, dtype=BF16, device="cuda")
    far = [buf.as_strided((n, 1, D), (stride, stride, 1), i * 64) for i in range(3)]
    for a, b in zip(far, (k, v, q)):
        a.copy_(b)
    p = mm.muon_packing_create([n])
    kw = dict(window=50, sinks=2)
    o, lse = mm.muon_attention(q, k, v, p, **kw)
    want = (o, lse) + mm.muon_attention_backward(do, q, k, v, o, lse, p, **kw)
    o, lse = mm.muon_attention(far[2], far[0], far[1], p, **kw)
    got = (o, lse) + mm.muon_attention_backward(do, far[2], far[0], far[1], o, lse, p, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(mm):
    q, k, v, do = inputs([20], 4, 2, 64, layout="plain")
    p = mm.muon_packing_create([20])
    o, lse = mm.muon_attention(q, k, v, p)
    for bad in (dict(window=0), dict(window=-1), dict(window=2.5), dict(window=1 << 64), dict(window=4, sinks=-1),
                dict(window=4, sinks=129), dict(sinks=-1), dict(sinks=129), dict(window=4, sinks=0.5)):
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_attention(q, k, v, p, **bad)
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_attention_backward(do, q, k, v, o, lse, p, **bad)
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_attention_backward_workspace_bytes(q, k, p, **bad)
    small = torch.empty(mm.muon_attention_backward_workspace_bytes(q, k, p), dtype=torch.uint8, device="cuda")
    with pytest.raises(mm.MuonError):
        mm.muon_attention_backward(do, q, k, v, o, lse, p, window=4, sinks=2, workspace=small)
