"""Host-side checks of the gradient norm, of the norms and rotations of queries
and keys, and of windowed attention (no GPU): every refusal is raised before
anything is enqueued."""
import ctypes
import math

import pytest

import matrix_muon_step_amd as mm
from matrix_muon_step_amd import binding as bd

BASE = 1 << 36  # fake, 256-byte aligned device addresses, far apart; never dereferenced


# ------------------------------------------------------------ gradient norm
def gradients(*changes, n=2):
    arr = (bd.muon_gradient_t * n)()
    for i in range(n):
        arr[i] = bd.muon_gradient_t(BASE * (2 * i + 2), BASE * (2 * i + 3), 100, mm.MUON_F32, mm.MUON_BF16)
    for i, field, value in changes:
        setattr(arr[i], field, value)
    return arr


def grad_norm(arr, n=2, norm=BASE * 50, ws=BASE * 60, ws_bytes=1 << 20):
    return mm.lib().muon_grad_norm(arr, n, ctypes.c_void_p(norm), ctypes.c_void_p(ws), ws_bytes, None)


def grad_clip(arr, n=2, max_norm=1.0, norm=BASE * 50, given=0, ws=BASE * 60, ws_bytes=1 << 20):
    return mm.lib().muon_grad_clip(arr, n, max_norm, ctypes.c_void_p(norm), given, ctypes.c_void_p(ws), ws_bytes, None)


def test_gradient_workspace():
    need = mm.muon_grad_norm_workspace_bytes()
    assert need > 0 and need % 256 == 0
    for call in (grad_norm, grad_clip):
        assert call(gradients(), ws=0) == mm.MUON_ERR_WORKSPACE
        assert call(gradients(), ws=BASE * 60 + 16) == mm.MUON_ERR_WORKSPACE
        assert call(gradients(), ws_bytes=need - 1) == mm.MUON_ERR_WORKSPACE
        assert call(gradients(), ws=BASE * 2) == mm.MUON_ERR_ALIAS
        assert call(gradients(), norm=BASE * 60 + 64) == mm.MUON_ERR_ALIAS
        assert call(gradients(), norm=0) == mm.MUON_ERR_INVALID_ARG
        assert call(gradients(), norm=BASE * 50 + 4) == mm.MUON_ERR_ALIGN
        assert call(None, n=2) == mm.MUON_ERR_INVALID_ARG
        assert call(gradients(), n=-1) == mm.MUON_ERR_INVALID_ARG


@pytest.mark.parametrize("field,value,status", [
    ("count", -1, mm.MUON_ERR_INVALID_ARG), ("count", (1 << 40) + 1, mm.MUON_ERR_UNSUPPORTED), ("g", 0, mm.MUON_ERR_INVALID_ARG),
    ("g_dtype", 2, mm.MUON_ERR_INVALID_ARG), ("g_dtype", -1, mm.MUON_ERR_INVALID_ARG), ("g", BASE * 2 + 2, mm.MUON_ERR_ALIGN),
    ("g", BASE * 50, mm.MUON_ERR_ALIAS), ("g", BASE * 60 + 64, mm.MUON_ERR_ALIAS)], ids=str)
def test_gradients_refused(field, value, status):
    for i in (0, 1):
        assert grad_norm(gradients((i, field, value))) == status and mm.muon_last_error()
        assert grad_clip(gradients((i, field, value))) == status and mm.muon_last_error()


@pytest.mark.parametrize("field,value,status", [
    ("out", 0, mm.MUON_ERR_INVALID_ARG), ("out", BASE * 3 + 1, mm.MUON_ERR_ALIGN), ("out_dtype", 7, mm.MUON_ERR_INVALID_ARG),
    ("out", BASE * 2, mm.MUON_ERR_ALIAS),            # in place, of another type
    ("out", BASE * 2 + 398, mm.MUON_ERR_ALIAS), ("out", BASE * 4 - 198, mm.MUON_ERR_ALIAS), ("out", BASE * 5, mm.MUON_ERR_ALIAS)],
    ids=str)
def test_clip_outputs_refused(field, value, status):
    assert grad_clip(gradients((0, field, value))) == status and mm.muon_last_error()


def test_clip_in_place_and_arguments():
    same = gradients((0, "out", BASE * 2), (0, "out_dtype", mm.MUON_F32), (1, "g", BASE * 2))
    assert grad_clip(same) == mm.MUON_ERR_ALIAS      # a tensor clipped in place and read again
    for max_norm in (0.0, -1.0, math.inf, math.nan):
        assert grad_clip(gradients(), max_norm=max_norm) == mm.MUON_ERR_INVALID_ARG
    # a given norm is read: it may lie in no output, and needs no workspace
    assert grad_clip(gradients(), norm=BASE * 3 + 16, given=1, ws=0) == mm.MUON_ERR_ALIAS
    assert grad_clip(gradients(), norm=0, given=1, ws=0) == mm.MUON_ERR_INVALID_ARG


# ------------------------------------------------- norms and rotations
class packing_s(ctypes.Structure):
    """A packing's host side, of a device that is not there: what passes every check ends at that one."""
    _fields_ = [("device", ctypes.c_int), ("tokens", ctypes.c_int64), ("n_tiles", ctypes.c_int64),
                ("by_query", ctypes.c_void_p), ("by_key", ctypes.c_void_p), ("lo", ctypes.c_size_t),
                ("hi", ctypes.c_size_t), ("longest", ctypes.c_int64), ("chunks", ctypes.c_int64)]


def packing(tokens=100, tiles=1, longest=None):
    longest = tokens if longest is None else longest
    return packing_s(77, tokens, tiles, BASE, BASE + 64, BASE, BASE + 4096, longest, -(-longest // 256))


PASSED = (mm.MUON_ERR_HIP, mm.MUON_ERR_INVALID_ARG)   # no GPU, or not the packing's


def passed(status):
    return status in PASSED and ("device" in mm.muon_last_error() or "hip" in mm.muon_last_error().lower())


def heads_at(i, heads, dim=64):
    return bd.muon_heads_t(BASE * (2 + i), heads * dim, dim)


KEEP = []


def rotate(heads=4, kv=2, dim=64, rotary=None):
    r = rotary or mm.MuonRotary(dim)
    KEEP.append(r)
    return bd.muon_qk_rotate_t(heads_at(0, heads, dim), heads_at(1, kv, dim), heads_at(2, heads, dim), heads_at(3, kv, dim),
                               BASE * 20, BASE * 21, BASE * 22, 128, 64, heads, kv, dim, 1, 1e-6, r._t)


def call_rotate(a, p=None):
    return mm.lib().muon_qk_norm_rotate(ctypes.byref(a), ctypes.byref(p or packing()), None)


def call_rotate_back(a, p=None, up_q=None, up_k=None, dqw=BASE * 23, dkw=BASE * 24, ws=BASE * 30, ws_bytes=1 << 30):
    up_q = up_q or heads_at(4, a.heads, a.head_dim)
    up_k = up_k or heads_at(5, a.kv_heads, a.head_dim)
    return mm.lib().muon_qk_norm_rotate_backward(ctypes.byref(a), ctypes.byref(up_q), ctypes.byref(up_k),
                                                 ctypes.c_void_p(dqw), ctypes.c_void_p(dkw), ctypes.byref(p or packing()),
                                                 ctypes.c_void_p(ws), ws_bytes, None)


ROTATE = [
    (dict(heads=0), mm.MUON_ERR_INVALID_ARG), (dict(kv_heads=-1), mm.MUON_ERR_INVALID_ARG),
    (dict(heads=4097), mm.MUON_ERR_UNSUPPORTED), (dict(kv_heads=4097), mm.MUON_ERR_UNSUPPORTED),
    (dict(head_dim=12), mm.MUON_ERR_UNSUPPORTED), (dict(head_dim=0), mm.MUON_ERR_UNSUPPORTED),
    (dict(head_dim=136), mm.MUON_ERR_UNSUPPORTED), (dict(eps=0.0), mm.MUON_ERR_INVALID_ARG),
    (dict(eps=math.nan), mm.MUON_ERR_INVALID_ARG), (dict(eps=math.inf), mm.MUON_ERR_INVALID_ARG),
    (dict(eps=1e-39), mm.MUON_ERR_INVALID_ARG), (dict(norm=0), mm.MUON_ERR_INVALID_ARG),
    (dict(q_weight=BASE * 20 + 2), mm.MUON_ERR_ALIGN), (dict(k_weight=BASE * 20 + 1), mm.MUON_ERR_ALIGN),
    (dict(positions=BASE * 22 + 4), mm.MUON_ERR_ALIGN), (dict(position_bits=16), mm.MUON_ERR_INVALID_ARG),
    (dict(position_stride=99), mm.MUON_ERR_INVALID_ARG), (dict(position_stride=1 << 41), mm.MUON_ERR_INVALID_ARG),
    (dict(positions=BASE * 4), mm.MUON_ERR_ALIAS), (dict(q_weight=BASE * 5 + 64), mm.MUON_ERR_ALIAS),
]


@pytest.mark.parametrize("call", [call_rotate, call_rotate_back])
@pytest.mark.parametrize("change,status", ROTATE, ids=str)
def test_rotate_refuses(call, change, status):
    a = rotate()
    for k, v in change.items():
        setattr(a, k, v)
    assert call(a) == status and mm.muon_last_error()


def test_rotate_passes_on():
    for call in (call_rotate, call_rotate_back):
        assert passed(call(rotate()))
        a = rotate()
        a.q_out, a.k_out = a.q, a.k                     # over the inputs
        assert passed(call(a))
        a = rotate()
        a.k_weight = a.q_weight                         # one weight for both
        assert passed(call(a))
        a = rotate(kv=3)                                # queries and keys need not be grouped
        assert passed(call(a))
        a = rotate(rotary=mm.MuonRotary(64, sections=[8, 12, 12]))
        a.position_stride = 0                           # one row of positions for all axes
        assert passed(call(a))
    a = rotate()
    assert passed(call_rotate_back(a, up_q=a.q_out, up_k=a.k_out))
    a.norm, a.q_weight, a.k_weight, a.q.data, a.k.data = 0, 0, 0, 0, 0
    assert passed(call_rotate_back(a, dqw=0, dkw=0, ws=0, ws_bytes=0))
    assert call_rotate(a) == mm.MUON_ERR_INVALID_ARG    # the forward pass reads them


@pytest.mark.parametrize("name", ["q", "k", "q_out", "k_out"])
def test_rotate_refuses_views(name):
    for call in (call_rotate, call_rotate_back):
        for field, value, status in (("data", 0, mm.MUON_ERR_INVALID_ARG), ("data", BASE * 9 + 8, mm.MUON_ERR_ALIGN),
                                     ("token_stride", 132, mm.MUON_ERR_ALIGN), ("token_stride", -64, mm.MUON_ERR_INVALID_ARG),
                                     ("head_stride", 1 << 50, mm.MUON_ERR_UNSUPPORTED),
                                     ("token_stride", 1 << 23, mm.MUON_ERR_UNSUPPORTED)):
            a = rotate()
            setattr(getattr(a, name), field, value)
            assert call(a) == status, (field, value)
    # an output that overlaps an input it is not, by one row, or another output
    a = rotate()
    a.q_out.data = a.q.data + 2 * a.q.token_stride
    assert call_rotate(a) == mm.MUON_ERR_ALIAS and call_rotate_back(a) == mm.MUON_ERR_ALIAS
    a = rotate()
    a.k_out.data = a.q_out.data
    assert call_rotate(a) == mm.MUON_ERR_ALIAS and call_rotate_back(a) == mm.MUON_ERR_ALIAS
    a = rotate()
    a.q_out.head_stride = 32                            # and itself
    assert call_rotate(a) == mm.MUON_ERR_ALIAS


def test_rotate_refuses_rotary():
    for field, value, status in (("rotary_dim", 72, mm.MUON_ERR_UNSUPPORTED), ("rotary_dim", -8, mm.MUON_ERR_UNSUPPORTED),
                                 ("rotary_dim", 12, mm.MUON_ERR_UNSUPPORTED), ("axes", 0, mm.MUON_ERR_INVALID_ARG),
                                 ("axes", 5, mm.MUON_ERR_INVALID_ARG), ("frequency", None, mm.MUON_ERR_INVALID_ARG)):
        a = rotate()
        setattr(a.rotary, field, value)
        assert call_rotate(a) == status and call_rotate_back(a) == status, field
    a = rotate(rotary=mm.MuonRotary(64, sections=[16, 16]))
    a.rotary.axes = 1                                   # a pair's axis that is not there
    assert call_rotate(a) == mm.MUON_ERR_INVALID_ARG
    a = rotate(rotary=mm.MuonRotary(64, frequencies=[1.0] * 31 + [2000.0]))
    assert call_rotate(a) == mm.MUON_ERR_INVALID_ARG
    a = rotate()
    a.rotary.axis = None                                # all of the first
    assert passed(call_rotate(a))


def test_rotate_backward_arguments():
    L = mm.lib()
    need = mm.muon_qk_norm_rotate_backward_workspace_bytes(64)
    assert call_rotate_back(rotate(), ws=0) == mm.MUON_ERR_WORKSPACE
    assert call_rotate_back(rotate(), ws_bytes=need - 1) == mm.MUON_ERR_WORKSPACE
    assert call_rotate_back(rotate(), ws=BASE * 30 + 64) == mm.MUON_ERR_WORKSPACE
    assert call_rotate_back(rotate(), ws=BASE * 4) == mm.MUON_ERR_ALIAS
    assert call_rotate_back(rotate(), dqw=BASE * 20) == mm.MUON_ERR_ALIAS
    assert call_rotate_back(rotate(), dqw=BASE * 24 + 4) == mm.MUON_ERR_ALIAS
    assert call_rotate_back(rotate(), dqw=BASE * 23 + 2) == mm.MUON_ERR_ALIGN
    assert passed(call_rotate_back(rotate(), dqw=0, dkw=0, ws=0, ws_bytes=0))
    assert passed(call_rotate_back(rotate(), dqw=0))
    a = rotate()
    a.k_weight = 0
    assert call_rotate_back(a) == mm.MUON_ERR_INVALID_ARG and passed(call_rotate_back(a, dkw=0))
    up = heads_at(4, 4)
    up.data = rotate().k_out.data
    assert call_rotate_back(rotate(), up_q=up) == mm.MUON_ERR_ALIAS
    for args in ((None, ctypes.byref(up), ctypes.byref(up)), (ctypes.byref(rotate()), None, ctypes.byref(up)),
                 (ctypes.byref(rotate()), ctypes.byref(up), None)):
        assert L.muon_qk_norm_rotate_backward(*args, None, None, ctypes.byref(packing()), None, 0, None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_qk_norm_rotate(None, ctypes.byref(packing()), None) == mm.MUON_ERR_INVALID_ARG
    assert L.muon_qk_norm_rotate(ctypes.byref(rotate()), None, None) == mm.MUON_ERR_INVALID_ARG


# -------------------------------------------------------- windowed attention
def attention(heads=4, kv=2, dim=64):
    return bd.muon_attention_t(heads_at(0, heads, dim), heads_at(1, kv, dim), heads_at(2, kv, dim), heads_at(3, heads, dim),
                               BASE * 20, 128, BASE * 21, heads, heads, kv, dim, 0.125)


def attention_grad(heads=4, kv=2, dim=64):
    g = bd.muon_attention_grad_t()
    for i, (f, h) in enumerate((("q", heads), ("k", kv), ("v", kv), ("o", heads), ("d_o", heads), ("dq", heads),
                                ("dk", kv), ("dv", kv))):
        setattr(g, f, heads_at(i, h, dim))
    g.lse, g.lse_stride = BASE * 20, 128
    g.heads, g.kv_heads, g.head_dim, g.scale = heads, kv, dim, 0.125
    return g


def call_window(a, window=10, sinks=4, p=None, ws=0, ws_bytes=0):
    return mm.lib().muon_window_attention(ctypes.byref(a), window, sinks, ctypes.byref(p or packing()), ctypes.c_void_p(ws),
                                          ws_bytes, None)


def forward_bytes(a, window=10, sinks=4, p=None):
    return mm.lib().muon_window_attention_workspace_bytes(ctypes.byref(a), window, sinks, ctypes.byref(p or packing()))


def window_bytes(g, window=10, sinks=4, p=None):
    return mm.lib().muon_window_attention_backward_workspace_bytes(ctypes.byref(g), window, sinks, ctypes.byref(p or packing()))


def call_window_back(g, window=10, sinks=4, p=None, ws=BASE * 30, ws_bytes=1 << 30):
    return mm.lib().muon_window_attention_backward(ctypes.byref(g), window, sinks, ctypes.byref(p or packing()),
                                                   ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("make,call", [(attention, call_window), (attention_grad, call_window_back)])
def test_window_refuses(make, call):
    for window, sinks, status in ((0, 0, mm.MUON_ERR_INVALID_ARG), (-5, 0, mm.MUON_ERR_INVALID_ARG),
                                  (10, -1, mm.MUON_ERR_INVALID_ARG), (10, 129, mm.MUON_ERR_UNSUPPORTED)):
        assert call(make(), window, sinks) == status and mm.muon_last_error()
        assert window_bytes(attention_grad(), window, sinks) == 0
    for window, sinks in ((1, 0), (1, 128), (99, 4), (100, 0), (1 << 62, 128)):
        assert passed(call(make(), window, sinks))
    for field, value, status in (("heads", 0, mm.MUON_ERR_INVALID_ARG), ("head_dim", 12, mm.MUON_ERR_UNSUPPORTED),
                                 ("scale", math.nan, mm.MUON_ERR_INVALID_ARG), ("lse", 0, mm.MUON_ERR_INVALID_ARG),
                                 ("lse_stride", 99, mm.MUON_ERR_INVALID_ARG)):
        a = make()
        setattr(a, field, value)
        assert call(a) == status
    a = make()
    a.k.data = 0
    assert call(a) == mm.MUON_ERR_INVALID_ARG


def test_window_workspace():
    g = attention_grad()
    base = mm.lib().muon_attention_backward_workspace_bytes(ctypes.byref(g), ctypes.byref(packing()))
    assert window_bytes(g, 10, 0) == window_bytes(g, 100, 128) == window_bytes(g, 1 << 62, 5) == base
    for sinks in (1, 4, 32, 33, 128):
        for tokens in (100, 256, 257, 5000):
            p = packing(tokens)
            rows = mm.lib().muon_attention_backward_workspace_bytes(ctypes.byref(g), ctypes.byref(p))
            sums = -(-tokens // 256) * 2 * 8 * sinks * 64
            assert window_bytes(g, 10, sinks, p) == rows + (sums + 255) // 256 * 256
    need = window_bytes(g)
    assert need > base
    assert call_window_back(g, ws_bytes=need - 1) == mm.MUON_ERR_WORKSPACE
    assert call_window_back(g, ws=0) == mm.MUON_ERR_WORKSPACE
    assert call_window_back(g, ws=BASE * 30 + 64) == mm.MUON_ERR_WORKSPACE
    # the sums' end counts as the workspace's too
    assert call_window_back(g, ws=g.dk.data - need + 256) == mm.MUON_ERR_ALIAS
    assert passed(call_window_back(g, ws=g.dk.data - need))
    assert mm.lib().muon_window_attention(None, 4, 0, ctypes.byref(packing()), None, 0, None) == mm.MUON_ERR_INVALID_ARG
    assert mm.lib().muon_window_attention(ctypes.byref(attention()), 4, 0, None, None, 0, None) == mm.MUON_ERR_INVALID_ARG


def test_window_forward_workspace():
    """Room for the work items' largest logits, where there are many of them."""
    a, many = attention(), packing(tokens=100, tiles=1000)
    assert forward_bytes(a, p=many) == 4000 * 4 // 256 * 256 + 256 and mm.muon_last_error() == ""
    assert forward_bytes(a) == 0 and mm.muon_last_error() == ""            # few items
    assert forward_bytes(a, 100, p=many) == 0 and mm.muon_last_error() == ""   # nothing hidden
    none = attention()
    none.max_logit = 0
    assert forward_bytes(none, p=many) == 0 and mm.muon_last_error() == ""
    for window, sinks in ((0, 0), (10, -1), (10, 129)):
        assert forward_bytes(a, window, sinks, many) == 0 and mm.muon_last_error()
    a.heads = 5
    assert forward_bytes(a, p=many) == 0 and mm.muon_last_error()
    assert mm.lib().muon_window_attention_workspace_bytes(None, 1, 0, ctypes.byref(many)) == 0 and mm.muon_last_error()
    a = attention()
    need = forward_bytes(a, p=many)
    assert passed(call_window(a, p=many)) and passed(call_window(a, p=many, ws=BASE * 30, ws_bytes=need))
    assert call_window(a, p=many, ws=BASE * 30, ws_bytes=need - 1) == mm.MUON_ERR_WORKSPACE
    assert call_window(a, p=many, ws=BASE * 30 + 64, ws_bytes=need + 64) == mm.MUON_ERR_WORKSPACE
    for other in (a.q.data, a.v.data, a.o.data, a.lse, a.max_logit, BASE):
        assert call_window(a, p=many, ws=other // 256 * 256, ws_bytes=need) == mm.MUON_ERR_ALIAS
    # one that is not used overlaps nothing
    assert passed(call_window(a, ws=a.q.data, ws_bytes=0))


def test_window_workspace_of_few_key_heads():
    """Room for float32 sums where several work-groups share a key tile, within what the header says."""
    def extra(heads, kv, dim, tiles, tokens, window=1000):
        g, p = attention_grad(heads, kv, dim), packing(tokens, tiles)
        return window_bytes(g, window, 0, p) - mm.lib().muon_attention_backward_workspace_bytes(ctypes.byref(g), ctypes.byref(p))

    for heads, kv, dim, tiles in ((8, 1, 128, 32), (32, 8, 128, 16), (16, 2, 40, 10), (24, 3, 64, 32)):
        more = extra(heads, kv, dim, tiles, 128 * tiles)
        assert 0 < more <= tiles * 1024 * dim * heads
    assert extra(8, 8, 128, 32, 4096) == 0                 # no heads to share out
    assert extra(32, 8, 128, 200, 25600) == 0              # enough key tiles
    assert extra(8, 1, 128, 32, 4096, window=4096) == 0    # nothing hidden
