"""Edges of the training-step operators on the host (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import matrix_muon_step_amd as mm
from test_train_ops_abi import backward, call_backward, call_forward, forward, grad, item

from matrix_muon_step_amd import binding as bd


# ------------------------------------------------- gradients without tokens among others
def workspace(*mats):
    arr = (bd.muon_checkpoint_grad_t * len(mats))(*mats)
    need = mm.lib().muon_checkpoint_grad_workspace_bytes(arr, len(mats))
    assert mm.muon_last_error() == ""
    return need


SETS = {"tiles": [dict(tokens=777, cols=7168, outs=2048, dy_stride=2048)],
        "small": [dict(tokens=40, cols=100, outs=60)] * 3,
        "shares": [dict(tokens=16384, cols=1600, outs=6400, dy_stride=6400)],
        "both": [dict(tokens=8192, cols=300, outs=501, dy_stride=501), dict(tokens=100, cols=256, outs=256, dy_stride=256)]}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("size", [dict(cols=7168, outs=2048, dy_stride=2048), dict(cols=65536, outs=65536, dy_stride=65536)],
                         ids=["expert", "largest"])
def test_a_gradient_without_tokens_changes_no_layout(name, accumulate, size):
    """The workspace follows the layout: a matrix of no tokens (an expert that
    none was routed to) leaves it as it is, wherever it stands."""
    mats = [grad(accumulate=accumulate, **m) for m in SETS[name]]
    none = grad(tokens=0, accumulate=accumulate, **size)
    want = workspace(*mats)
    assert workspace(none, *mats) == workspace(*mats, none) == workspace(mats[0], none, *mats[1:]) == want
    assert workspace(none, none) == 0


# ------------------------------------------------------------ scales
@pytest.mark.parametrize("make,call", [(forward, call_forward), (backward, call_backward)], ids=["forward", "backward"])
def test_scales_without_a_base_two_form_are_refused(make, call):
    """scale * log2(e) has to be a float32 number: with an infinite one a logit of 0 is NaN."""
    a = make()
    for scale in (2.36e38, 3.4e38):                    # 2^128 / log2(e) is 2.3586e38
        a.scale = scale
        assert call(a) == mm.MUON_ERR_UNSUPPORTED and "scale" in mm.muon_last_error()
    for scale in (2.35e38, 1e-45):                     # pass on to the device check
        a.scale = scale
        assert call(a) in (mm.MUON_ERR_HIP, mm.MUON_ERR_INVALID_ARG) and "scale" not in mm.muon_last_error()


# ------------------------------------------------------------ extents
@pytest.mark.parametrize("tokens,stride", [(1 << 24, 1 << 40), (1 << 23, 1 << 40), (1 << 28, 1 << 35), (1 << 28, (1 << 28) + 1)])
def test_extents_past_64_bits_are_refused(tokens, stride):
    """An x whose extent in bytes wraps would pass the overlap checks."""
    arr = (bd.muon_checkpoint_t * 1)(item(tokens=tokens, x_stride=stride, cols=8))
    for f in (mm.lib().muon_checkpoint_write, mm.lib().muon_checkpoint_read):
        assert f(arr, 1, None) == mm.MUON_ERR_UNSUPPORTED and "x_stride" in mm.muon_last_error()
    # as far as it goes, the overlap is seen: data inside x
    inside = item(tokens=1 << 16, x_stride=1 << 40, cols=8, data=item().x + (1 << 40))
    arr = (bd.muon_checkpoint_t * 1)(inside)
    assert mm.lib().muon_checkpoint_write(arr, 1, None) == mm.MUON_ERR_ALIAS


# ------------------------------------------------------------ the binding
def test_current_stream_without_torch_internals(monkeypatch):
    """Where torch lacks the call that gives the current stream's handle, its documented one serves."""
    class Stream:
        cuda_stream = 4711

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream() if device == 2 else None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 4710 + index // 2, raising=False)
    with bd._on(None, None) as st:
        assert st.cuda_stream == 4711
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    for device in (None, torch.device("cuda", 2)):
        with bd._on(device, None) as st:
            assert st.cuda_stream == 4711


def test_checkpoint_size_follows_its_fields():
    """The check of the data's size is that of the tokens and columns that the call will use."""
    c = mm.MuonCheckpoint(None, 32, 32)
    assert c._bytes() == mm.muon_checkpoint_bytes(32, 32)
    c.tokens = 320
    assert c._bytes() == mm.muon_checkpoint_bytes(320, 32)
    c.cols = 64
    assert c._bytes() == c._bytes() == mm.muon_checkpoint_bytes(320, 64)
    c.tokens = -1
    with pytest.raises(mm.MuonError):
        c._bytes()
    empty = mm.MuonCheckpoint(None, 0, 0)
    with pytest.raises(mm.MuonError):
        empty._bytes()


@pytest.mark.parametrize("n", [(1 << 64) + 5, 5 - (1 << 64), 1 << 63, 3.7, 1e30, float("nan"), "7"])
def test_numbers_that_64_bits_do_not_hold(n):
    """Neither their low bits nor their whole part is taken for them."""
    with pytest.raises(ValueError):
        mm.muon_packing_create([3, n])
    with pytest.raises(ValueError):
        mm.muon_checkpoint_bytes(n, 5)
    with pytest.raises(ValueError):
        mm.muon_checkpoint_bytes(5, n)


def test_numbers_of_other_integer_types():
    for n in (np.int32(33), torch.tensor(33), 33.0):
        assert mm.muon_checkpoint_bytes(n, n) == mm.muon_checkpoint_bytes(33, 33)


def test_packings_are_on_gpus_only(monkeypatch):
    """"cpu" is not taken for the current GPU."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: pytest.fail("went on to a GPU"))
    for device in ("cpu", torch.device("cpu"), "meta"):
        with pytest.raises(ValueError):
            mm.muon_packing_create([3], device=device)


def test_backward_workspace_by_its_shapes():
    """What the library asks for, for an empty packing (the only one that needs
    no GPU), and the refusals."""
    table, h = (ctypes.c_char * 512)(), ctypes.c_void_p()
    at = (ctypes.addressof(table) + 255) // 256 * 256
    assert mm.lib().muon_packing_create((ctypes.c_int64 * 1)(0), 1, ctypes.c_void_p(at), 256, None, ctypes.byref(h)) == mm.MUON_OK
    p = mm.MuonPacking(h.value, [0], None, None, 0)
    q, k = torch.empty((0, 6, 64)), torch.empty((0, 2, 64))
    assert mm.muon_attention_backward_workspace_bytes(q, k, p) == 64 * 6 * 2 * 4
    with pytest.raises(mm.MuonError):
        mm.muon_attention_backward_workspace_bytes(k, q, p)
    with pytest.raises(mm.MuonError):
        mm.muon_attention_backward_workspace_bytes(q[:, :, :12], k, p)
    p.close()
    with pytest.raises(RuntimeError):
        mm.muon_attention_backward_workspace_bytes(q, k, p)
