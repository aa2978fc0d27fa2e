"""Edges of the training-step operators on the GPU."""
import math

import numpy as np
import pytest
import torch

import attention_ref as ref
from test_attention_gpu import host, inputs
from test_checkpoint_gpu import activation, check_grad, code_values, np64, upstream

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


# ------------------------------------------------- gradients without tokens among others
def grad_set(mm, sizes, pad, g_type, seed=0):
    mats = []
    for i, (tokens, outs, cols) in enumerate(sizes):
        saved = mm.muon_checkpoint_write([activation(max(tokens, 1), cols, BF16, seed=seed + i)[:tokens]])[0]
        dy = upstream(max(tokens, 1), outs, pad, seed=seed + i)[:tokens]
        mats.append((dy, saved, torch.full((outs, cols), math.nan, dtype=g_type, device="cuda")))
    return mats


SETS = [[(777, 300, 257), (640, 64, 520)],             # a work-group per tile
        [(8192, 501, 300)],                             # tiles cut into shares
        [(100, 256, 256), (33, 40, 700), (31, 264, 96)]]
EMPTY = [(0, 24, 40), (0, 300, 257), (0, 7, 513)]


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("g_type", [F32, BF16])
@pytest.mark.parametrize("which", range(len(SETS)))
def test_empty_gradients_among_others(mm, which, g_type, pad):
    """First, in the middle and last: zeros, and the others' bits unchanged."""
    print(f"[case] gradients {SETS[which]} with empty ones {g_type} pad {pad}", flush=True)
    mats = grad_set(mm, SETS[which], pad, g_type)
    mm.muon_checkpoint_grad(mats)
    want = [G.clone() for _, _, G in mats]
    for (dy, saved, G) in mats:
        check_grad(dy, np64(mm.muon_checkpoint_read([saved], dtype=F32)[0]), G)
    empty = grad_set(mm, EMPTY, pad, g_type)
    mixed = [empty[0], mats[0], empty[1], *mats[1:], empty[2]]
    for _, _, G in mixed:
        G.fill_(math.nan)
    mm.muon_checkpoint_grad(mixed)
    assert all((G == 0).all() for _, _, G in empty)
    assert all(torch.equal(G, w) for (_, _, G), w in zip(mats, want))
    for _, _, G in empty:
        G.fill_(3.0)
    old = [np64(G) for _, _, G in mats]
    mm.muon_checkpoint_grad(mixed, accumulate=True)
    assert all((G == 3).all() for _, _, G in empty)
    for (dy, saved, G), o in zip(mats, old):
        check_grad(dy, np64(mm.muon_checkpoint_read([saved], dtype=F32)[0]), G, o)


@pytest.mark.parametrize("outs", [8, 7, 300])
def test_only_empty_gradients(mm, outs):
    print(f"[case] {outs} outs of no tokens", flush=True)
    mats = grad_set(mm, [(0, outs, 40), (0, outs, 700)], 0, F32)
    assert mm.muon_checkpoint_grad_workspace_bytes(mats) == 0
    mm.muon_checkpoint_grad(mats)
    assert all((G == 0).all() for _, _, G in mats)


def test_many_gradients_mostly_empty_in_a_graph(mm):
    """Several launches, some with empty matrices only, captured and replayed."""
    print("[case] 60 gradients, 54 of them empty, in a graph", flush=True)
    sizes = [(0, 8 + i, 40 + 3 * i) for i in range(60)]
    for i, size in ((0, (300, 100, 64)), (20, (33, 7, 96)), (23, (5, 300, 40)), (24, (64, 64, 64)), (40, (700, 33, 130)),
                    (47, (1, 1, 1))):
        sizes[i] = size
    mats = grad_set(mm, sizes, 0, F32)
    mm.muon_checkpoint_grad(mats)
    want = [G.clone() for _, _, G in mats]
    for (dy, saved, G), (tokens, _, _) in zip(mats, sizes):
        if tokens:
            check_grad(dy, np64(mm.muon_checkpoint_read([saved], dtype=F32)[0]), G)
        else:
            assert (G == 0).all()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mm.muon_checkpoint_grad(mats)
    for _ in range(3):
        for _, _, G in mats:
            G.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(G, w) for (_, _, G), w in zip(mats, want))
    mm.muon_checkpoint_grad([m for m, size in zip(mats, sizes) if not size[0]], accumulate=True)
    assert all(torch.equal(G, w) for (_, _, G), w in zip(mats, want))


@pytest.mark.parametrize("outs,cols", [(1, 1), (7, 513), (64, 512), (300, 257), (129, 1024), (1, 65536)])
@pytest.mark.parametrize("g_type", [F32, BF16])
def test_zeros_end_with_the_matrix(mm, outs, cols, g_type):
    print(f"[case] zeros {outs} x {cols} {g_type}", flush=True)
    room = torch.full((outs * cols + 64,), 7.0, dtype=g_type, device="cuda")
    G = room[32:32 + outs * cols].view(outs, cols)
    saved = mm.muon_checkpoint_write([torch.empty((0, cols), dtype=BF16, device="cuda")])[0]
    some = grad_set(mm, [(40, 16, 32)], 0, g_type)
    mm.muon_checkpoint_grad([(torch.empty((0, outs), dtype=BF16, device="cuda"), saved, G), *some])
    assert (G == 0).all() and (room[:32] == 7).all() and (room[32 + outs * cols:] == 7).all()
    check_grad(some[0][0], np64(mm.muon_checkpoint_read([some[0][1]], dtype=F32)[0]), some[0][2])


# ------------------------------------------------- the end of an aligned dY
@pytest.mark.parametrize("outs", [1, 2, 3, 5, 6, 7, 9, 14, 70, 129, 250, 259])
@pytest.mark.parametrize("tokens", [2, 32, 45, 1000, 6000])
def test_grad_at_the_end_of_aligned_rows(mm, tokens, outs):
    """Widths that end inside a 16-byte chunk: the last token's elements all
    count, and nothing behind them does."""
    print(f"[case] gradient {tokens} x {outs} x 40, aligned", flush=True)
    stride = -(-outs // 8) * 8
    x = activation(tokens, 40, BF16)
    x[-1] = 1.0                                        # the last token counts as much as all others together
    saved = mm.muon_checkpoint_write([x])[0]
    xh = np64(mm.muon_checkpoint_read([saved], dtype=F32)[0])
    room = torch.full((tokens + 2, stride), math.nan, dtype=BF16, device="cuda")
    dy = room[1:tokens + 1, :outs]
    dy.copy_(upstream(tokens, outs, 0))
    dy[-1] = torch.arange(1, outs + 1, device="cuda").to(BF16)
    assert dy.data_ptr() % 16 == 0
    G = torch.full((outs, 40), math.nan, device="cuda")
    mm.muon_checkpoint_grad([(dy, saved, G)])
    check_grad(dy, xh, G)


# ------------------------------------------------------------ largest logits
def test_max_logit_entry_that_is_nan(mm):
    """A NaN of either sign in max_logit stays one, whatever the logits' sign."""
    print("[case] max_logit with NaN entries", flush=True)
    D = 64
    p = mm.muon_packing_create([5])
    q = torch.ones((5, 4, D), dtype=BF16, device="cuda")
    k = torch.ones((5, 4, D), dtype=BF16, device="cuda")
    k[:, 2:] = -1.0
    bits = np.array([0xFFC00000, 0x7FC00000, 0xFFC00000, 0x7F800001], dtype=np.uint32).view(np.int32)
    top = torch.from_numpy(bits).cuda().view(F32)
    mm.muon_attention(q, k, q, p, max_logit=top)
    assert torch.isnan(top).all(), top
    per_group = torch.from_numpy(bits[:2].copy()).cuda().view(F32)
    mm.muon_attention(q, k[:, 1:3], q[:, :2], p, max_logit=per_group)
    assert torch.isnan(per_group).all(), per_group


# ------------------------------------------------------------------- streams
@pytest.mark.parametrize("use", ["read", "write", "grad", "attention"])
def test_memory_in_use_on_another_stream_is_not_handed_out(mm, use):
    """A checkpoint or packing that is dropped while a call on another stream
    is still to run keeps its memory until that call is done."""
    print(f"[case] dropped while in use by {use}", flush=True)
    tokens, cols = 5000, 300
    x = activation(tokens, cols, BF16)
    if use == "attention":
        q = torch.ones((tokens, 2, 64), dtype=BF16, device="cuda")
        made = mm.muon_packing_create([1] * tokens)
        data = made._table
    else:
        made = mm.muon_checkpoint_write([x])[0]
        data = made.data
    at, size = data.data_ptr(), data.numel()
    dy, G = upstream(tokens, 64, 0), torch.zeros((64, cols), device="cuda")
    again = torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                  # what follows waits some 50 ms
        if use == "read":
            mm.muon_checkpoint_read([made], xs=[again])
        elif use == "write":
            mm.muon_checkpoint_write([x], [made])
        elif use == "grad":
            mm.muon_checkpoint_grad([(dy, made, G)])
        else:
            mm.muon_attention(q, q, q, made)
    del made, data
    new = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert not side.query(), "the side stream was done too early to tell"
    assert new.data_ptr() != at
    torch.cuda.synchronize()


# ------------------------------------------------------------ largest logits, wave by wave
@pytest.mark.parametrize("n,D", [(300, 64), (1100, 64), (1100, 128)])
def test_max_logit_in_any_row(mm, n, D):
    """The largest logit counts whichever row of a work item has it (one head
    for each 16th row), in short sequences and in split ones."""
    print(f"[case] largest logit in any of {n} rows, heads of {D}", flush=True)
    rows = list(range(0, n, 16)) + [n - 1]
    H = len(rows)
    q = torch.ones((n, H, D), dtype=BF16, device="cuda")
    k = torch.ones((n, H, D), dtype=BF16, device="cuda")
    for h, r in enumerate(rows):
        q[r, h] = 1.0 + (h + 1) / 128.0 if h < 127 else 2.0
    for heads in (1, 3, H):                            # few heads: split; many: not
        want = [D * float(q[rows[h], h, 0]) for h in range(heads)]
        top = torch.full((heads,), -math.inf, device="cuda")
        mm.muon_attention(q[:, :heads], k[:, :heads], k[:, :heads], mm.muon_packing_create([n]), scale=1.0, max_logit=top)
        np.testing.assert_array_equal(top.cpu().numpy(), np.array(want, dtype=np.float32))


def test_max_logit_next_to_the_largest_float(mm):
    """Logits that are finite while their base-2 form is not: the largest is still theirs."""
    print("[case] max_logit near 2^128", flush=True)
    D = 64
    p = mm.muon_packing_create([70])
    q = torch.zeros((70, 3, D), dtype=BF16, device="cuda")
    k = torch.zeros((70, 3, D), dtype=BF16, device="cuda")
    q[:, 0, 3], k[66, 0, 3] = 2.0 ** 64, 2.0 ** 63     # 2^127 * 1.9 = 0.95 * 2^128
    q[:, 1, 3], k[0, 1, 3] = 2.0 ** 64, 2.0 ** 62      # half of it: finite in base 2 too
    q[:, 2, 3], k[5, 2, 3] = 2.0 ** 64, 2.0 ** 64      # infinite
    top = torch.full((3,), -math.inf, device="cuda")
    mm.muon_attention(q, k, torch.ones_like(q), p, scale=1.9, max_logit=top)
    s = np.float32(1.9)
    np.testing.assert_array_equal(top.cpu().numpy(), np.array([s * np.float32(2.0 ** 127), s * np.float32(2.0 ** 126), np.inf],
                                                              dtype=np.float32))


# ------------------------------------------- not finite, on every kernel variant
# (lengths, heads, kv heads, head size): keys split over two wave groups, and
# more key tiles than the pair kernel takes
VARIANTS = {"split": ([1100, 40], 2, 2, 64), "split128": ([40, 1100], 4, 2, 128), "three": ([64] * 50 + [130], 11, 11, 64),
            "three40": ([70] * 50 + [130], 11, 11, 40)}


@pytest.mark.parametrize("name", VARIANTS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_variants_keep_sequences_apart(mm, name, bad):
    lens, H, K, D = VARIANTS[name]
    print(f"[case] isolation {name} {bad}", flush=True)
    T = sum(lens)
    q, k, v, do = inputs(lens, H, K, D, behind=9, layout="plain")
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(q, k, v, p)
    grads = mm.muon_attention_backward(do, q, k, v, o, lse, p)
    assert all(torch.isfinite(t).all() for t in (o[:T], lse[:, :T], *(g[:T] for g in grads)))
    start = np.concatenate([[0], np.cumsum(lens)])
    for seq in {0, len(lens) // 2, len(lens) - 1}:
        for at in {0, lens[seq] // 2, lens[seq] - 1}:
            row = int(start[seq]) + at
            x = [t.clone() for t in (q, k, v, do)]
            for t in x:
                t[row, :, 5] = bad
            o2, lse2 = mm.muon_attention(x[0], x[1], x[2], p)
            g2 = mm.muon_attention_backward(x[3], x[0], x[1], x[2], o2, lse2, p)
            for rows in (slice(0, int(start[seq])), slice(int(start[seq + 1]), None)):
                assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])
                for a, b in zip(grads, g2):
                    assert torch.equal(a[rows], b[rows])
            assert not torch.isfinite(o2[row]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pos", [0, 10, 70, 700, 1000, 1050, 1099])
def test_split_keys_not_finite_logits(mm, pos, D):
    """One key of a long sequence gives a NaN, an infinite or a -infinite logit
    (each in a head of its own), in a tile of either wave group: rows before it
    and the largest logits follow the formulas."""
    print(f"[case] split keys, key {pos} not finite, heads of {D}", flush=True)
    n = 1100
    p = mm.muon_packing_create([n])
    q = torch.ones((n, 5, D), dtype=BF16, device="cuda")
    k = -torch.ones((n, 5, D), dtype=BF16, device="cuda")
    v = torch.ones((n, 5, D), dtype=BF16, device="cuda")
    k[pos, 0, 3] = math.nan
    k[pos, 1, 3] = math.inf
    k[pos, 2, 3] = -math.inf
    k[:, 3, 3] = -math.inf
    top = torch.full((5,), -math.inf, device="cuda")
    o, lse = mm.muon_attention(q, k, v, p, scale=0.5, max_logit=top)
    got, one = lse.cpu().numpy().astype(np.float64), -0.5 * D
    t = top.cpu().numpy()
    # the base logit is exact; the one with an element of infinite size is that infinity
    assert np.isnan(t[0]) and t[1] == np.inf and t[2] == one and t[3] == -np.inf and t[4] == one
    i = np.arange(n)
    count = {0: i + 1.0, 1: i + 1.0, 2: np.where(i >= pos, i, i + 1.0), 4: i + 1.0}
    for h, c in count.items():
        rows = i < pos if h < 2 else c > 0
        want = one + np.log(c[rows])
        # the logits are exact, their sum is a sum of ones: log2, a product and an addition in float32
        assert (np.abs(got[h, rows] - want) <= 4 * ref.F32 * (np.abs(want) + 1) + 2.0 ** -20).all(), h
        assert (host(o[:, h][torch.from_numpy(rows).cuda()], n) == 1).all(), h
        assert np.isnan(got[h, ~rows]).all() if h < 2 else np.isneginf(got[h, ~rows]).all(), h
    assert np.isneginf(got[3]).all()


# ---------------------------------------------------------------- workspaces
@pytest.mark.parametrize("lens", [[5], [200, 57], [1100]], ids=str)
def test_backward_in_a_workspace_of_the_asked_size(mm, lens):
    print(f"[case] backward of {lens} in the caller's workspace", flush=True)
    q, k, v, do = inputs(lens, 4, 2, 64)
    p = mm.muon_packing_create(lens)
    o, lse = mm.muon_attention(q, k, v, p)
    want = mm.muon_attention_backward(do, q, k, v, o, lse, p)
    need = mm.muon_attention_backward_workspace_bytes(q, k, p)
    room = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    got = mm.muon_attention_backward(do, q, k, v, o, lse, p, workspace=room[256:256 + need])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (room[:256] == 7).all() and (room[256 + need:] == 7).all()
    with pytest.raises(mm.MuonError):
        mm.muon_attention_backward(do, q, k, v, o, lse, p, workspace=room[256:255 + need])
