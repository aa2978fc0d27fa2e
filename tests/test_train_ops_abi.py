"""Host-side checks of the training-step operators (no GPU): every refusal is
raised before anything is enqueued.  Attention calls take a packing, which
only a GPU can hold a table for, so these tests hand them a host-side one of
the same layout whose table is never read."""
import ctypes
import math

import pytest

import matrix_muon_step_amd as mm
from matrix_muon_step_amd import binding as bd

BASE = 1 << 36  # fake, 256-byte aligned device addresses, far apart; never dereferenced


def lengths(*n):
    return (ctypes.c_int64 * max(1, len(n)))(*n), len(n)


class packing_s(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("tokens", ctypes.c_int64), ("n_tiles", ctypes.c_int64),
                ("by_query", ctypes.c_void_p), ("by_key", ctypes.c_void_p), ("lo", ctypes.c_size_t),
                ("hi", ctypes.c_size_t), ("longest", ctypes.c_int64)]


def packing(tokens=100, tiles=1):
    # of a device that is not there: what passes every check ends at that one
    return packing_s(77, tokens, tiles, BASE, BASE + 64, BASE, BASE + 4096, tokens)


# ---------------------------------------------------------------- packings
def test_packing_bytes():
    L = mm.lib()
    assert L.muon_packing_bytes(*lengths()) == 256
    assert L.muon_packing_bytes(*lengths(0, 0)) == 256
    assert L.muon_packing_bytes(*lengths(1)) == 256
    assert L.muon_packing_bytes(*lengths(128 * 100)) == 100 * 32 // 256 * 256 + 256 * (100 * 32 % 256 > 0)
    assert L.muon_packing_bytes(*lengths(*[1] * 1000)) >= 1000 * 32


@pytest.mark.parametrize("n", [(-1,), (5, -2, 3), ((1 << 24) + 1,), (1 << 24,) * 65])
def test_packing_refuses_lengths(n):
    L = mm.lib()
    n = n if isinstance(n, tuple) else (n,)
    assert L.muon_packing_bytes(*lengths(*n)) == 0 and mm.muon_last_error()
    out = ctypes.c_void_p(7)
    st = L.muon_packing_create(*lengths(*n), ctypes.c_void_p(BASE), 1 << 30, None, ctypes.byref(out))
    assert st in (mm.MUON_ERR_INVALID_ARG, mm.MUON_ERR_UNSUPPORTED) and out.value is None


def test_packing_refuses_tables():
    L = mm.lib()
    out = ctypes.c_void_p()
    args = lengths(5, 7)
    assert L.muon_packing_create(*args, None, 1 << 20, None, ctypes.byref(out)) == mm.MUON_ERR_WORKSPACE
    assert L.muon_packing_create(*args, ctypes.c_void_p(BASE), 8, None, ctypes.byref(out)) == mm.MUON_ERR_WORKSPACE
    assert L.muon_packing_create(*args, ctypes.c_void_p(BASE + 16), 1 << 20, None, ctypes.byref(out)) == mm.MUON_ERR_WORKSPACE
    assert L.muon_packing_create(*args, ctypes.c_void_p(BASE), 1 << 20, None, None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_packing_create(None, 2, ctypes.c_void_p(BASE), 1 << 20, None, ctypes.byref(out)) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_packing_create(None, -1, ctypes.c_void_p(BASE), 1 << 20, None, ctypes.byref(out)) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_packing_destroy(None) == mm.MUON_OK


def test_empty_packing_needs_no_gpu():
    L = mm.lib()
    out = ctypes.c_void_p()
    assert L.muon_packing_create(*lengths(0, 0), ctypes.c_void_p(BASE), 256, None, ctypes.byref(out)) == mm.MUON_OK
    a = forward()
    for f in ("q", "k", "v", "o"):
        setattr(a, f, bd.muon_heads_t(0, 0, 0))
    a.lse = None
    assert L.muon_attention(ctypes.byref(a), out, None) == mm.MUON_OK       # nothing to do
    a.heads = 3
    assert L.muon_attention(ctypes.byref(a), out, None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_packing_destroy(out) == mm.MUON_OK


# --------------------------------------------------------------- attention
def heads_at(i, heads, dim=64, token_stride=None):
    return bd.muon_heads_t(BASE * (2 + i), token_stride or heads * dim, dim)


def forward(heads=4, kv=2, dim=64):
    return bd.muon_attention_t(heads_at(0, heads, dim), heads_at(1, kv, dim), heads_at(2, kv, dim), heads_at(3, heads, dim),
                               BASE * 20, 128, BASE * 21, heads, heads, kv, dim, 0.125)


def backward(heads=4, kv=2, dim=64):
    g = bd.muon_attention_grad_t()
    for i, (f, h) in enumerate((("q", heads), ("k", kv), ("v", kv), ("o", heads), ("d_o", heads), ("dq", heads),
                                ("dk", kv), ("dv", kv))):
        setattr(g, f, heads_at(i, h, dim))
    g.lse, g.lse_stride = BASE * 20, 128
    g.heads, g.kv_heads, g.head_dim, g.scale = heads, kv, dim, 0.125
    return g


def call_forward(a, p=None):
    return mm.lib().muon_attention(ctypes.byref(a), ctypes.byref(p or packing()), None)


def call_backward(g, ws=BASE * 30, ws_bytes=1 << 30, p=None):
    return mm.lib().muon_attention_backward(ctypes.byref(g), ctypes.byref(p or packing()), ctypes.c_void_p(ws), ws_bytes, None)


def view(**kw):
    def change(name):
        def f(a):
            t = getattr(a, name)
            for k, v in kw.items():
                setattr(t, k, v if not callable(v) else v(getattr(t, k)))
        return f
    return change


SHAPES = [
    (dict(heads=0), mm.MUON_ERR_INVALID_ARG), (dict(kv_heads=0), mm.MUON_ERR_INVALID_ARG),
    (dict(heads=5), mm.MUON_ERR_INVALID_ARG), (dict(heads=8192), mm.MUON_ERR_UNSUPPORTED),
    (dict(head_dim=0), mm.MUON_ERR_UNSUPPORTED), (dict(head_dim=12), mm.MUON_ERR_UNSUPPORTED),
    (dict(head_dim=136), mm.MUON_ERR_UNSUPPORTED), (dict(scale=0.0), mm.MUON_ERR_INVALID_ARG),
    (dict(scale=-1.0), mm.MUON_ERR_INVALID_ARG), (dict(scale=math.nan), mm.MUON_ERR_INVALID_ARG),
    (dict(scale=math.inf), mm.MUON_ERR_INVALID_ARG), (dict(lse=0), mm.MUON_ERR_INVALID_ARG),
    (dict(lse=BASE * 20 + 2), mm.MUON_ERR_ALIGN), (dict(lse_stride=99), mm.MUON_ERR_INVALID_ARG),
]
VIEWS = [
    (dict(data=0), mm.MUON_ERR_INVALID_ARG), (dict(data=lambda p: p + 8), mm.MUON_ERR_ALIGN),
    (dict(token_stride=132), mm.MUON_ERR_ALIGN), (dict(head_stride=68), mm.MUON_ERR_ALIGN),
    (dict(token_stride=-64), mm.MUON_ERR_INVALID_ARG), (dict(head_stride=-64), mm.MUON_ERR_INVALID_ARG),
    (dict(token_stride=1 << 23), mm.MUON_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("make,call", [(forward, call_forward), (backward, call_backward)], ids=["forward", "backward"])
@pytest.mark.parametrize("change,status", SHAPES, ids=str)
def test_attention_refuses_shapes(make, call, change, status):
    a = make()
    for k, v in change.items():
        setattr(a, k, v)
    assert call(a) == status and mm.muon_last_error()


@pytest.mark.parametrize("change,status", VIEWS, ids=str)
def test_attention_refuses_views(change, status):
    for name in ("q", "k", "v", "o"):
        a = forward()
        view(**change)(name)(a)
        assert call_forward(a) == status, name
    for name in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv"):
        g = backward()
        view(**change)(name)(g)
        assert call_backward(g) == status, name


@pytest.mark.parametrize("make,call", [(forward, call_forward), (backward, call_backward)], ids=["forward", "backward"])
def test_attention_refuses_more_than_a_launch(make, call):
    """Fewer than 2^32 lanes to a launch: 2^23 items of up to 512."""
    assert call(make(), p=packing(tiles=1 << 21)) == mm.MUON_ERR_UNSUPPORTED    # 4 heads
    # one fewer passes on to the device check
    assert call(make(), p=packing(tiles=(1 << 21) - 1)) in (mm.MUON_ERR_HIP, mm.MUON_ERR_INVALID_ARG)
    assert "items" not in mm.muon_last_error()


def test_attention_null_arguments():
    L = mm.lib()
    assert L.muon_attention(None, ctypes.byref(packing()), None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_attention(ctypes.byref(forward()), None, None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_attention_backward(None, ctypes.byref(packing()), None, 0, None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_attention_backward(ctypes.byref(backward()), None, None, 0, None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_attention_backward_workspace_bytes(None, ctypes.byref(packing())) == 0
    assert L.muon_attention_backward_workspace_bytes(ctypes.byref(backward()), None) == 0


def test_max_logit_arguments():
    for n, status in ((3, mm.MUON_ERR_INVALID_ARG), (0, mm.MUON_ERR_INVALID_ARG)):
        a = forward()
        a.logit_heads = n
        assert call_forward(a) == status
    a = forward()
    a.max_logit += 2
    assert call_forward(a) == mm.MUON_ERR_ALIGN
    a = forward()
    a.max_logit = a.o.data + 16
    assert call_forward(a) == mm.MUON_ERR_ALIAS
    a = forward()
    a.max_logit = a.lse
    assert call_forward(a) == mm.MUON_ERR_ALIAS


def test_attention_workspace():
    g = backward()
    need = mm.lib().muon_attention_backward_workspace_bytes(ctypes.byref(g), ctypes.byref(packing()))
    assert need >= 100 * 4 * 8
    assert call_backward(g, ws=0) == mm.MUON_ERR_WORKSPACE
    assert call_backward(g, ws=BASE * 30 + 128) == mm.MUON_ERR_WORKSPACE
    assert call_backward(g, ws_bytes=need - 1) == mm.MUON_ERR_WORKSPACE
    for name in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv"):
        assert call_backward(g, ws=getattr(g, name).data) == mm.MUON_ERR_ALIAS, name
    assert call_backward(g, ws=g.lse) == mm.MUON_ERR_ALIAS
    assert call_backward(g, ws=BASE) == mm.MUON_ERR_ALIAS          # the packing's table


OVERLAPS = [("o", "q"), ("o", "k"), ("o", "v")]


@pytest.mark.parametrize("out,other", OVERLAPS)
def test_attention_output_overlaps(out, other):
    a = forward()
    getattr(a, out).data = getattr(a, other).data
    assert call_forward(a) == mm.MUON_ERR_ALIAS
    a = forward()
    getattr(a, out).data = getattr(a, other).data + 2 * 64 * 2     # a head further
    assert call_forward(a) == mm.MUON_ERR_ALIAS


@pytest.mark.parametrize("out", ["dq", "dk", "dv"])
@pytest.mark.parametrize("other", ["q", "k", "v", "o", "d_o", "dq", "dk", "dv"])
def test_gradient_overlaps(out, other):
    if out == other:
        return
    g = backward()
    getattr(g, out).data = getattr(g, other).data
    assert call_backward(g) == mm.MUON_ERR_ALIAS
    g = backward()
    getattr(g, out).data = g.lse
    assert call_backward(g) == mm.MUON_ERR_ALIAS


def test_output_overlaps_itself():
    for ts, hs in ((64, 64), (0, 64), (256, 0), (192, 64), (64, 64 * 99)):
        a = forward()
        a.o.token_stride, a.o.head_stride = ts, hs
        assert call_forward(a) == mm.MUON_ERR_ALIAS, (ts, hs)


def test_interleaved_outputs_are_no_overlap():
    """dq, dk and dv as views of one fused buffer pass the overlap checks (the
    call then ends at the device check)."""
    def fused(g, shift=0):
        width = (4 + 2 + 2) * 64
        for name, at in (("dq", 0), ("dk", 4 * 64), ("dv", 6 * 64)):
            setattr(g, name, bd.muon_heads_t(BASE * 9 + 2 * (at + (shift if name == "dk" else 0)), width, 64))
    g = backward()
    fused(g)
    assert call_backward(g) in (mm.MUON_ERR_HIP, mm.MUON_ERR_INVALID_ARG) and "overlap" not in mm.muon_last_error()
    fused(g, 8)                                                     # dk's last head reaches into dv
    assert call_backward(g) == mm.MUON_ERR_ALIAS
    g = backward()                                                  # head by head: [k | v] pairs
    for name, at in (("dk", 0), ("dv", 64)):
        setattr(g, name, bd.muon_heads_t(BASE * 9 + 2 * at, 2 * 128, 128))
    assert call_backward(g) in (mm.MUON_ERR_HIP, mm.MUON_ERR_INVALID_ARG) and "overlap" not in mm.muon_last_error()


# -------------------------------------------------------------- checkpoints
def item(**kw):
    v = dict(x=BASE * 2, x_stride=100, x_dtype=mm.MUON_BF16, reserved=0, data=BASE * 3, tokens=40, cols=100)
    v.update(kw)
    return bd.muon_checkpoint_t(*[v[n] for n, _ in bd.muon_checkpoint_t._fields_])


ITEMS = [
    (dict(tokens=-1), mm.MUON_ERR_INVALID_ARG), (dict(cols=0), mm.MUON_ERR_INVALID_ARG),
    (dict(cols=70000, x_stride=70000), mm.MUON_ERR_UNSUPPORTED), (dict(tokens=(1 << 30) + 1), mm.MUON_ERR_UNSUPPORTED),
    (dict(x_dtype=5), mm.MUON_ERR_INVALID_ARG), (dict(x_stride=99), mm.MUON_ERR_INVALID_ARG),
    (dict(x=0), mm.MUON_ERR_INVALID_ARG), (dict(data=0), mm.MUON_ERR_INVALID_ARG), (dict(x=BASE * 2 + 1), mm.MUON_ERR_ALIGN),
    (dict(x=BASE * 2 + 2, x_dtype=mm.MUON_F32), mm.MUON_ERR_ALIGN), (dict(data=BASE * 3 + 128), mm.MUON_ERR_ALIGN),
    # 2^24 work-groups of 256 lanes
    (dict(tokens=1 << 29, cols=1, x_stride=1), mm.MUON_ERR_UNSUPPORTED),
    (dict(tokens=1 << 21, cols=65536, x_stride=65536), mm.MUON_ERR_UNSUPPORTED),
    (dict(data=BASE * 2), mm.MUON_ERR_ALIAS), (dict(x=BASE * 3 + 512), mm.MUON_ERR_ALIAS),
]


@pytest.mark.parametrize("change,status", ITEMS, ids=str)
def test_checkpoint_refusals(change, status):
    arr = (bd.muon_checkpoint_t * 2)(item(x=BASE * 7, data=BASE * 8), item(**change))
    for f in (mm.lib().muon_checkpoint_write, mm.lib().muon_checkpoint_read):
        assert f(arr, 2, None) == status and mm.muon_last_error()


def test_checkpoint_lists():
    L = mm.lib()
    for f in (L.muon_checkpoint_write, L.muon_checkpoint_read):
        assert f(None, 0, None) == mm.MUON_OK
        assert f(None, 1, None) == mm.MUON_ERR_INVALID_ARG
        assert f((bd.muon_checkpoint_t * 1)(item()), -1, None) == mm.MUON_ERR_INVALID_ARG
        assert f((bd.muon_checkpoint_t * 1)(item(tokens=0, x=0, data=0)), 1, None) == mm.MUON_OK
    # one data written by two items; one x written by two
    assert L.muon_checkpoint_write((bd.muon_checkpoint_t * 2)(item(), item(x=BASE * 5)), 2, None) == mm.MUON_ERR_ALIAS
    assert L.muon_checkpoint_read((bd.muon_checkpoint_t * 2)(item(), item(data=BASE * 5)), 2, None) == mm.MUON_ERR_ALIAS


def test_checkpoint_bytes():
    assert mm.muon_checkpoint_bytes(32, 32) == 1280
    assert mm.muon_checkpoint_bytes(33, 32) == 2304
    assert mm.muon_checkpoint_bytes(0, 5) == 256
    assert mm.muon_checkpoint_bytes(1 << 30, 65536) == (1 << 46) + (1 << 36)
    for bad in ((-1, 5), (5, 0), (5, 65537), ((1 << 30) + 1, 5)):
        with pytest.raises(mm.MuonError):
            mm.muon_checkpoint_bytes(*bad)


def grad(**kw):
    v = dict(dy=BASE * 2, dy_stride=64, data=BASE * 3, tokens=40, cols=100, G=BASE * 4, outs=60, g_dtype=mm.MUON_F32,
             accumulate=0)
    v.update(kw)
    return bd.muon_checkpoint_grad_t(*[v[n] for n, _ in bd.muon_checkpoint_grad_t._fields_])


GRADS = [
    (dict(tokens=-1), mm.MUON_ERR_INVALID_ARG), (dict(cols=0), mm.MUON_ERR_INVALID_ARG),
    (dict(outs=0), mm.MUON_ERR_INVALID_ARG), (dict(outs=70000, dy_stride=70000), mm.MUON_ERR_UNSUPPORTED),
    (dict(cols=70000), mm.MUON_ERR_UNSUPPORTED), (dict(dy_stride=59), mm.MUON_ERR_INVALID_ARG),
    (dict(dy_stride=1 << 23), mm.MUON_ERR_UNSUPPORTED), (dict(g_dtype=2), mm.MUON_ERR_INVALID_ARG),
    (dict(accumulate=2), mm.MUON_ERR_INVALID_ARG), (dict(dy=0), mm.MUON_ERR_INVALID_ARG),
    (dict(data=0), mm.MUON_ERR_INVALID_ARG), (dict(G=0), mm.MUON_ERR_INVALID_ARG), (dict(dy=BASE * 2 + 1), mm.MUON_ERR_ALIGN),
    (dict(data=BASE * 3 + 64), mm.MUON_ERR_ALIGN), (dict(G=BASE * 4 + 8), mm.MUON_ERR_ALIGN),
    (dict(G=BASE * 2), mm.MUON_ERR_ALIAS), (dict(G=BASE * 3), mm.MUON_ERR_ALIAS), (dict(G=BASE * 9), mm.MUON_ERR_ALIAS),
]


@pytest.mark.parametrize("change,status", GRADS, ids=str)
def test_gradient_refusals(change, status):
    arr = (bd.muon_checkpoint_grad_t * 2)(grad(dy=BASE * 7, data=BASE * 8, G=BASE * 9), grad(**change))
    assert mm.lib().muon_checkpoint_grad(arr, 2, None, 0, None) == status and mm.muon_last_error()


def test_gradient_workspace_and_lists():
    L = mm.lib()
    assert L.muon_checkpoint_grad(None, 0, None, 0, None) == mm.MUON_OK
    assert L.muon_checkpoint_grad(None, 1, None, 0, None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_checkpoint_grad((bd.muon_checkpoint_grad_t * 1)(grad()), -1, None, 0, None) == mm.MUON_ERR_INVALID_ARG
    small = (bd.muon_checkpoint_grad_t * 1)(grad())
    assert L.muon_checkpoint_grad_workspace_bytes(small, 1) == 0 and mm.muon_last_error() == ""
    long = (bd.muon_checkpoint_grad_t * 1)(grad(tokens=100000, cols=256, outs=256, dy_stride=256))
    need = L.muon_checkpoint_grad_workspace_bytes(long, 1)
    assert need > 0
    call = lambda ws, n: L.muon_checkpoint_grad(long, 1, ctypes.c_void_p(ws), n, None)  # noqa: E731
    assert call(0, need) == mm.MUON_ERR_WORKSPACE
    assert call(BASE * 5, need - 1) == mm.MUON_ERR_WORKSPACE
    assert call(BASE * 5 + 16, need) == mm.MUON_ERR_WORKSPACE
    assert call(BASE * 4, need) == mm.MUON_ERR_ALIAS
    bad = (bd.muon_checkpoint_grad_t * 1)(grad(outs=0))
    assert L.muon_checkpoint_grad_workspace_bytes(bad, 1) == 0 and mm.muon_last_error()
