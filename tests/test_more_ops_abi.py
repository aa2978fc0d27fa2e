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
