"""The training-step operators on the GPU as programs use them: the largest
logits, isolation of sequences, outputs in place, streams, graphs, offsets past
32 bits, and one attention layer's step from its input to QK-Clip."""
import math

import numpy as np
import pytest
import torch

import attention_ref as ref
from test_attention_gpu import close, host, inputs
from test_checkpoint_gpu import activation, check_grad, np64, upstream

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import matrix_muon_step_amd as m

    m.lib()
    return m


# ----------------------------------------------------------- largest logits
def test_max_logit_runs_over_calls_and_groups(mm):
    print("[case] max_logit over calls and groups", flush=True)
    lens, H, K, D = [40, 90], 6, 2, 64
    per_head = torch.full((H,), -math.inf, device="cuda")
    per_group = torch.full((K,), -math.inf, device="cuda")
    want, err = np.full(H, -np.inf), np.zeros(H)
    p = mm.muon_packing_create(lens)
    for seed in range(3):
        q, k, v, _ = inputs(lens, H, K, D, seed=seed)
        mm.muon_attention(q, k, v, p, max_logit=per_head)
        mm.muon_attention(q, k, v, p, max_logit=per_group)
        r = ref.forward(host(q, 130), host(k, 130), host(v, 130), lens, D ** -0.5)
        want, err = np.maximum(want, r[2]), np.maximum(err, r[5])
        close(per_head.cpu().numpy(), want, err, "per head")
        close(per_group.cpu().numpy(), want.reshape(K, -1).max(axis=1), err.reshape(K, -1).max(axis=1), "per group")
    # a start above every logit stays
    high = torch.full((H,), 1e6, device="cuda")
    mm.muon_attention(q, k, v, p, max_logit=high)
    assert (high == 1e6).all()


def test_max_logit_negative_and_not_finite(mm):
    print("[case] max_logit of negative, NaN and infinite logits", flush=True)
    D = 64
    p = mm.muon_packing_create([5])
    q = torch.ones((5, 4, D), dtype=BF16, device="cuda")
    k = -torch.ones((5, 4, D), dtype=BF16, device="cuda")
    v = torch.ones((5, 4, D), dtype=BF16, device="cuda")
    q[2, 1, 3] = math.nan
    q[4, 2] = 0
    q[4, 2, 0], k[:, 2, 0] = math.inf, 1.0      # +inf logits in the last row
    k[3, 3] = -2.0                              # one key lower still
    top = torch.tensor([-math.inf, -3.0, -math.inf, -8.0], device="cuda")
    mm.muon_attention(q, k, v, p, scale=0.5, max_logit=top)
    got = top.cpu().numpy()
    assert got[0] == -32.0 and np.isnan(got[1]) and got[2] == np.inf and got[3] == -8.0
    # NaN stays, whatever comes after; QK-Clip leaves such a head alone
    mm.muon_attention(v, v, v, p, scale=0.5, max_logit=top)
    assert np.isnan(top.cpu().numpy()[1])


# ------------------------------------------------- isolation and outputs
def test_sequences_do_not_mix(mm):
    """NaN and infinities of one sequence, and rows behind the last, reach no other sequence's rows."""
    print("[case] isolation", flush=True)
    lens, H, K, D = [50, 33, 70], 4, 2, 128
    T = sum(lens)
    q, k, v, do = inputs(lens, H, K, D, behind=9, layout="plain")
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(q, k, v, p)
    grads = mm.muon_attention_backward(do, q, k, v, o, lse, p)
    for bad in (math.nan, math.inf):
        x = [t.clone() for t in (q, k, v, do)]
        for t in x:
            t[60, :, 5] = bad                   # inside the second sequence
        o2, lse2 = mm.muon_attention(x[0], x[1], x[2], p)
        g2 = mm.muon_attention_backward(x[3], x[0], x[1], x[2], o2, lse2, p)
        for rows in (slice(0, 50), slice(83, T)):
            assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])
            for a, b in zip(grads, g2):
                assert torch.equal(a[rows], b[rows])
        assert not torch.isfinite(o2[60]).all()


def test_outputs_in_place(mm):
    """Outputs given by the caller: views of one fused buffer, rows behind the
    last sequence and everything between the views left as they were."""
    print("[case] outputs in place", flush=True)
    lens, H, K, D = [64, 5], 4, 2, 64
    T, rows = 69, 80
    q, k, v, do = inputs(lens, H, K, D, behind=rows - T)
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(q, k, v, p)
    want = mm.muon_attention_backward(do, q, k, v, o, lse, p)
    buf = torch.full((rows, H + 2 * K + 1, D), 7.0, dtype=BF16, device="cuda")
    out_o = torch.full((rows, H, D), 7.0, dtype=BF16, device="cuda")
    out_l = torch.full((H, rows + 3), 7.0, device="cuda")
    mm.muon_attention(q, k, v, p, o=out_o, lse=out_l[:, :rows])
    assert torch.equal(out_o[:T], o[:T]) and (out_o[T:] == 7).all()
    assert torch.equal(out_l[:, :T], lse[:, :T]) and (out_l[:, T:] == 7).all()
    views = buf[:, :H], buf[:, H:H + K], buf[:, H + K:H + 2 * K]
    got = mm.muon_attention_backward(do, q, k, v, out_o, out_l[:, :rows], p, dq=views[0], dk=views[1], dv=views[2])
    for a, b, w in zip(got, views, want):
        assert a.data_ptr() == b.data_ptr() and torch.equal(b[:T], w[:T])
    assert (buf[T:] == 7).all() and (buf[:, H + 2 * K:] == 7).all()


def test_refusals_of_the_binding(mm):
    q, k, v, do = inputs([20], 4, 2, 64, layout="plain")
    p = mm.muon_packing_create([20])
    o, lse = mm.muon_attention(q, k, v, p)
    bad = [dict(q=q.float()), dict(q=q[:19]), dict(k=k[:, :, :32]), dict(k=k.cpu()), dict(v=v[:10]), dict(q=q[:, :3]),
           dict(q=q.transpose(1, 2)), dict(o=torch.empty_like(q)[:, :2]), dict(o=q), dict(lse=lse.double()),
           dict(lse=lse[:2]), dict(max_logit=torch.zeros(3, device="cuda")), dict(scale=0.0), dict(scale=math.nan)]
    for change in bad:
        args = dict(q=q, k=k, v=v, packing=p)
        args.update(change)
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_attention(**args)
    for change in (dict(do=do[:5]), dict(o=o[:, :2]), dict(dq=torch.empty_like(k)), dict(dk=k), dict(dv=torch.empty_like(q)),
                   dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), dict(lse=lse.half())):
        args = dict(do=do, q=q, k=k, v=v, o=o, lse=lse, packing=p)
        args.update(change)
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_attention_backward(**args)
    for n in ([-1], [1 << 25]):
        with pytest.raises(mm.MuonError):
            mm.muon_packing_create(n)
    p.close()
    p.close()
    with pytest.raises(RuntimeError):
        mm.muon_attention(q, k, v, p)
    x = torch.zeros((20, 30), dtype=BF16, device="cuda")
    c = mm.muon_checkpoint_write([x])[0]
    G = torch.zeros((16, 30), device="cuda")
    dy = torch.zeros((20, 16), dtype=BF16, device="cuda")
    for args in ([x.half()], [x.t()], [x[0]], [x.cpu()]):
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_checkpoint_write(args)
    for args in ((dy[:19], c, G), (dy.float(), c, G), (dy, c, G.t()), (dy, c, G.half()), (dy, c, G[:8]),
                 (dy, mm.MuonCheckpoint(c.data[:100], 20, 30), G), (dy, c, G[:, :29])):
        with pytest.raises((ValueError, mm.MuonError)):
            mm.muon_checkpoint_grad([args])
    with pytest.raises(mm.MuonError):
        mm.muon_checkpoint_grad([(dy, c, G), (dy, c, G)])


def test_empty_calls(mm):
    p = mm.muon_packing_create([])
    q = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    o, lse = mm.muon_attention(q, q, q, p)
    assert o.shape == q.shape and lse.shape == (4, 0)
    mm.muon_attention_backward(q, q, q, q, o, lse, p)
    q = torch.full((3, 4, 64), 2.0, dtype=BF16, device="cuda")
    o, lse = mm.muon_attention(q, q, q, mm.muon_packing_create([0, 0]))
    assert (o == 0).all() and (lse == 0).all()
    assert mm.muon_checkpoint_write([]) == [] and mm.muon_checkpoint_read([]) == []
    mm.muon_checkpoint_grad([])


# -------------------------------------------------------- streams and graphs
def layer(mm, x, w, packing, do, H, K, D, top, out=None):
    """One layer's operators around library projections: everything a graph holds."""
    qkv = (x @ w).view(x.shape[0], H + 2 * K, D)
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    saved = mm.muon_checkpoint_write([x])[0]
    o, lse = mm.muon_attention(q, k, v, packing, max_logit=top)
    d = torch.empty_like(qkv)
    mm.muon_attention_backward(do, q, k, v, o, lse, packing, dq=d[:, :H], dk=d[:, H:H + K], dv=d[:, H + K:])
    dy = d.view(x.shape[0], -1)
    parts = dy[:, :H * D], dy[:, H * D:(H + K) * D], dy[:, (H + K) * D:]
    grads = [torch.empty((p.shape[1], x.shape[1]), device=x.device) for p in parts]
    mm.muon_checkpoint_grad([(p, saved, g) for p, g in zip(parts, grads)])
    return o, lse, d, grads


def layer_inputs(T, width, H, K, D, seed):
    rng = np.random.default_rng([31, seed, T])
    make = lambda *s, scale=1.0: torch.from_numpy((scale * rng.standard_normal(s)).astype(np.float32)).to(BF16).cuda()  # noqa: E731
    return make(T, width), make(width, (H + 2 * K) * D, scale=width ** -0.5), make(T, H, D, scale=0.1)


def flat(r):
    return [r[0], r[1], r[2], *r[3]]


def test_layer_on_other_streams_at_once(mm):
    print("[case] two streams at once, one packing", flush=True)
    lens, H, K, D = [130, 1, 300], 4, 2, 64
    p = mm.muon_packing_create(lens)
    data = [layer_inputs(431, 256, H, K, D, s) for s in (0, 1)]
    tops = [torch.full((H,), -math.inf, device="cuda") for _ in range(2)]
    want = [flat(layer(mm, x, w, p, do, H, K, D, t)) for (x, w, do), t in zip(data, tops)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                x, w, do = data[i]
                got[i] = flat(layer(mm, x, w, p, do, H, K, D, tops[i]))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # the stream as an argument, and by its handle
    q = torch.randn((431, H, D), device="cuda").to(BF16)
    torch.cuda.synchronize()
    ref_o, _ = mm.muon_attention(q, q, q, p)
    for s in (streams[0], streams[0].cuda_stream):
        o, _ = mm.muon_attention(q, q, q, p, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(o, ref_o)


def test_layer_in_graphs(mm):
    """Two captured layers, replayed several times in turn with new inputs and
    eager work between, give the eager bits every time."""
    print("[case] captured layers", flush=True)
    H, K, D = 4, 2, 64
    cases = []
    for seed, lens in enumerate(([200, 57], [3000])):
        T = sum(lens)
        p = mm.muon_packing_create(lens)
        x, w, do = layer_inputs(T, 192, H, K, D, seed)
        top = torch.full((H,), -math.inf, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(mm, x, w, p, do, H, K, D, top)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = flat(layer(mm, x, w, p, do, H, K, D, top))
        cases.append((p, x, w, do, top, g, out, T))
    for turn in range(4):
        for p, x, w, do, top, g, out, T in cases:
            nx, _, ndo = layer_inputs(T, 192, H, K, D, 10 + turn)
            x.copy_(nx)
            do.copy_(ndo)
            top.fill_(-math.inf)
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out] + [top.clone()]
            top.fill_(-math.inf)
            want = flat(layer(mm, x, w, p, do, H, K, D, top)) + [top]
            assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


def test_packing_is_not_created_while_capturing(mm):
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        x += 1
        with pytest.raises(mm.MuonError):
            mm.muon_packing_create([5])
    g.replay()
    torch.cuda.synchronize()
    assert (x == 1).all()


def test_same_bits_every_time(mm):
    print("[case] repeatable", flush=True)
    lens, H, K, D = [700, 1, 515], 8, 2, 128
    p = mm.muon_packing_create(lens)
    x, w, do = layer_inputs(sum(lens), 320, H, K, D, 5)
    first = None
    for _ in range(4):
        top = torch.full((K,), -math.inf, device="cuda")
        got = flat(layer(mm, x, w, p, do, H, K, D, top)) + [top]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


# --------------------------------------------------- gradients by differences
def test_gradients_by_differences(mm):
    """The kernels' gradients along random directions against differences of the
    float64 forward pass: off by no more than the elements' own bounds add up to."""
    print("[case] differences", flush=True)
    lens, H, K, D = [40, 23], 4, 2, 32
    T = 63
    q, k, v, do = inputs(lens, H, K, D, layout="plain", sharp=1.0)
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(q, k, v, p)
    got = mm.muon_attention_backward(do, q, k, v, o, lse, p)
    x = [host(t, T) for t in (q, k, v)]
    g = host(do, T)
    exact = ref.forward(*x, lens, D ** -0.5)
    with_held = ref.backward(g, *x, host(o, T), lse.cpu().numpy(), lens, D ** -0.5)
    with_exact = ref.backward(g, *x, exact[0], exact[1], lens, D ** -0.5)
    rng = np.random.default_rng(41)
    step = 1e-5
    for i in range(3):
        # the held o and lse are rounded: their effect on the gradient is the formula's
        bound = with_held[3 + i] + np.abs(with_held[i] - with_exact[i])
        for _ in range(4):
            d = rng.standard_normal(x[i].shape)
            up, down = ([a + (s * step * d if j == i else 0) for j, a in enumerate(x)] for s in (1, -1))
            slope = ((ref.forward(*up, lens, D ** -0.5)[0] - ref.forward(*down, lens, D ** -0.5)[0]) * g).sum() / (2 * step)
            assert abs((host(got[i], T) * d).sum() - slope) <= (bound * np.abs(d)).sum() + 1e-6


# ------------------------------------------------------ offsets past 32 bits
def test_attention_offsets_past_32_bits(mm):
    """Rows and heads more than 2^32 bytes apart."""
    print("[case] attention, offsets past 32 bits", flush=True)
    lens, H, D = [900, 300], 2, 64
    T = 1200
    small = inputs(lens, H, H, D, layout="plain")
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(*small[:3], p)
    want = mm.muon_attention_backward(small[3], *small[:3], o, lse, p)
    for shape, view in (((T, 1 << 22), lambda b: b[:, :H * D].unflatten(1, (H, D))),              # 8 MB between rows
                        ((H, 1 << 32), lambda b: b[:, :T * D].unflatten(1, (T, D)).transpose(0, 1))):  # 8 GB between heads
        wide = []
        for t in small:
            b = view(torch.empty(shape, dtype=BF16, device="cuda"))
            b.copy_(t)
            wide.append(b)
        ob = view(torch.empty(shape, dtype=BF16, device="cuda"))
        got_o, got_l = mm.muon_attention(*wide[:3], p, o=ob)
        assert torch.equal(got_o, o) and torch.equal(got_l, lse)
        dq = view(torch.empty(shape, dtype=BF16, device="cuda"))
        got = mm.muon_attention_backward(wide[3], *wide[:3], ob, got_l, p, dq=dq)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del wide, ob, dq, got, got_o
        torch.cuda.empty_cache()


def test_checkpoint_offsets_past_32_bits(mm):
    """An activation of more than 2^32 bytes, its checkpoint, and its gradient."""
    print("[case] checkpoint, offsets past 32 bits", flush=True)
    T, C = 70000, 65536
    x = torch.zeros((T, C), dtype=BF16, device="cuda")
    rows = [0, 1, 33333, 65535, 65600, T - 1]
    g = torch.Generator(device="cuda").manual_seed(5)
    for r in rows:
        x[r] = torch.randn(C, generator=g, device="cuda").to(BF16)
    saved = mm.muon_checkpoint_write([x])
    back = mm.muon_checkpoint_read(saved)[0]
    for r in rows:
        assert (back[r] - x[r]).abs().max() <= x[r].abs().max() / 16 and (back[r] != 0).any()
    assert int(torch.count_nonzero(back[2:33333])) == 0
    outs = 24
    dy = torch.zeros((T, outs), dtype=BF16, device="cuda")
    for i, r in enumerate(rows):
        dy[r, i] = 1.0 + i
    G = torch.empty((outs, C), device="cuda")
    mm.muon_checkpoint_grad([(dy, saved[0], G)])
    for i, r in enumerate(rows):
        assert torch.equal(G[i], (1.0 + i) * back[r].float())
    assert int(torch.count_nonzero(G[len(rows):])) == 0
    del x, back, saved, G
    torch.cuda.empty_cache()


# --------------------------------------------------------- one training step
def test_attention_layer_step(mm):
    """From a layer's input to clipped weights: attention with the largest
    logits, its backward pass, the projections' gradients from 8-bit
    checkpoints, the Muon step and QK-Clip."""
    print("[case] one layer's training step", flush=True)
    lens, H, K, D, width = [90, 200, 14], 6, 2, 32, 128
    T, scale, tau = sum(lens), 32 ** -0.5, 2.0
    rng = np.random.default_rng(51)
    W = {n: torch.from_numpy((rng.standard_normal((h * D, width)) * s).astype(np.float32)).cuda()
         for n, h, s in (("q", H, 0.4), ("k", K, 0.4), ("v", K, 0.1))}
    x = torch.from_numpy(rng.standard_normal((T, width)).astype(np.float32)).to(BF16).cuda()
    p = mm.muon_packing_create(lens)

    def project(n, h):
        return (x.float() @ W[n].t()).to(BF16).view(T, h, D)

    q, k, v = project("q", H), project("k", K), project("v", K)
    saved = mm.muon_checkpoint_write([x])[0]
    top = torch.full((K,), -math.inf, device="cuda")
    o, lse = mm.muon_attention(q, k, v, p, scale=scale, max_logit=top)
    do = o.float().mul(1e-3).to(BF16)        # gradient of 5e-4 |o|^2
    dq, dk, dv = mm.muon_attention_backward(do, q, k, v, o, lse, p, scale=scale)
    grads = {n: torch.empty_like(W[n]) for n in W}
    mm.muon_checkpoint_grad([(d.view(T, -1), saved, grads[n]) for n, d in (("q", dq), ("k", dk), ("v", dv))])
    xh = np64(mm.muon_checkpoint_read([saved], dtype=F32)[0])
    for n, d in (("q", dq), ("k", dk), ("v", dv)):
        check_grad(d.view(T, -1), xh, grads[n])
    before = {n: W[n].clone() for n in W}
    B = {n: torch.zeros_like(W[n]) for n in W}
    mm.muon_step([(W[n], grads[n], B[n]) for n in W], mu=0.9, lr=0.0)
    assert all(torch.equal(W[n], before[n]) and torch.equal(B[n], grads[n]) for n in W)
    # one max logit per key head clips its query heads' rows and its own
    mm.muon_qk_clip([(W["q"], D * H // K, top), (W["k"], D, top)], tau)
    s = top.cpu().numpy()
    assert (s > tau).all()
    for n, h in (("q", H // K * D), ("k", D)):
        for g in range(K):
            rows = slice(g * h, (g + 1) * h)
            want = before[n][rows].double() * math.sqrt(tau / float(s[g]))
            assert torch.allclose(W[n][rows].double(), want, rtol=1e-6, atol=0)
    # the clipped weights' largest logit is tau, up to the roundings of q and k to bfloat16
    after = torch.full((K,), -math.inf, device="cuda")
    mm.muon_attention(project("q", H), project("k", K), v, p, scale=scale, max_logit=after)
    qn = (np64(q) ** 2).sum(axis=2).max() ** 0.5
    kn = (np64(k) ** 2).sum(axis=2).max() ** 0.5
    slack = scale * qn * kn * tau / s.min() * 4 * 2.0 ** -8
    assert (np.abs(after.cpu().numpy() - tau) <= slack).all()
