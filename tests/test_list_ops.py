"""CPU tests of the list operators' host side: refusals, layout sizes, handles, the oracle.

No test here launches a kernel: pointers are fake numbers, and calls that pass validation are
made only where no GPU is visible (they then stop at the first HIP call)."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import newton_schulz_02_amd as nm
from oracle.grad_oracle import clip_coef, clip_grads, grad_norm
from tests.test_abi import _gpu_visible

BASE = 1 << 40


def grads(*sizes, dtype=nm.MUON_BF16, step=1 << 34):
    arr = (nm.muon_grad * max(1, len(sizes)))()
    for i, n in enumerate(sizes):
        arr[i] = nm.muon_grad(BASE + i * step, n, dtype, 0)
    return arr


def adamw(*sizes, param=nm.MUON_BF16, grad=nm.MUON_BF16, master=False):
    arr = (nm.adamw_tensor * max(1, len(sizes)))()
    for i, n in enumerate(sizes):
        at = BASE + i * (1 << 36)
        arr[i] = nm.adamw_tensor(at, at + (1 << 33), at + (2 << 33), at + (3 << 33), at + (4 << 33) if master else 0,
                                 n, param, grad, 1.0, 0)
    return arr


def size_of(fn, arr, count):
    out = ctypes.c_size_t(0)
    return getattr(nm.lib(), fn)(arr, count, ctypes.byref(out)), out.value


@pytest.mark.parametrize("mutate,code", [
    (lambda a: setattr(a[0], "grad", 0), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "n", -1), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "n", (1 << 40) + 1), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "dtype", 3), nm.MUON_EINVAL),
    (lambda a: setattr(a[1], "reserved", 1), nm.MUON_EINVAL),
    (lambda a: setattr(a[1], "grad", a[1].grad + 1), nm.MUON_EINVAL),
    (lambda a: setattr(a[1], "grad", 2 ** 64 - 8), nm.MUON_EINVAL),  # ends past the address space
    (lambda a: setattr(a[1], "grad", a[0].grad), nm.MUON_EALIAS),  # the same gradient twice
    (lambda a: setattr(a[1], "grad", a[0].grad + 2 * 99), nm.MUON_EALIAS),  # one element shared
])
def test_grad_list_refusals(mutate, code):
    arr = grads(100, 100)
    mutate(arr)
    assert size_of("muon_grad_list_size", arr, 2)[0] == code
    lst = nm.muon_grad_list()
    assert nm.lib().muon_grad_list_init(arr, 2, ctypes.c_void_p(1 << 32), 1 << 30, None, ctypes.byref(lst)) == code
    assert nm.last_error()


@pytest.mark.parametrize("mutate,code", [
    (lambda a: setattr(a[0], "param", 0), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "m", 0), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "param_dtype", 0), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "grad_dtype", 9), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "n", -5), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "decay", math.nan), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "reserved", 2), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "v", a[0].v + 2), nm.MUON_EINVAL),
    (lambda a: (setattr(a[0], "param_dtype", nm.MUON_F32), setattr(a[0], "master", BASE + (5 << 33))), nm.MUON_EINVAL),
    (lambda a: setattr(a[0], "grad", a[0].param), nm.MUON_EALIAS),
    (lambda a: setattr(a[0], "v", a[0].m), nm.MUON_EALIAS),
    (lambda a: setattr(a[1], "param", a[0].param), nm.MUON_EALIAS),  # the same parameter twice
    (lambda a: setattr(a[1], "m", a[0].v + 4 * 99), nm.MUON_EALIAS),
    (lambda a: setattr(a[0], "master", a[1].v), nm.MUON_EALIAS),
    (lambda a: setattr(a[1], "grad", a[0].m), nm.MUON_EALIAS),
])
def test_adamw_list_refusals(mutate, code):
    arr = adamw(100, 100)
    mutate(arr)
    assert size_of("adamw_list_size", arr, 2)[0] == code
    lst = nm.adamw_list()
    assert nm.lib().adamw_list_init(arr, 2, ctypes.c_void_p(1 << 32), 1 << 30, None, ctypes.byref(lst)) == code


def test_shared_gradients_of_adamw_and_empty_tensors_are_allowed():
    arr = adamw(100, 100, 0)
    arr[1].grad = arr[0].grad
    arr[2].param = arr[2].grad = arr[2].m = arr[2].v = 0
    assert size_of("adamw_list_size", arr, 3)[0] == nm.MUON_OK
    g = grads(7, 0)
    g[1].grad = 0
    assert size_of("muon_grad_list_size", g, 2)[0] == nm.MUON_OK
    # Neighbours that touch do not overlap.
    g = grads(7, 9)
    g[1].grad = g[0].grad + 14
    assert size_of("muon_grad_list_size", g, 2)[0] == nm.MUON_OK


def test_sizes_and_counts():
    for fn, make in (("muon_grad_list_size", grads), ("adamw_list_size", adamw)):
        rc, empty = size_of(fn, None, 0)
        assert rc == nm.MUON_OK
        rc, one = size_of(fn, make(1), 1)
        assert rc == nm.MUON_OK and one % 256 == 0
        # The layout grows with the number of tensors, and by far less than one byte in 200 of theirs.
        rc, large = size_of(fn, make(1 << 30), 1)
        assert rc == nm.MUON_OK and one < large < one + (1 << 31) // 200
        rc, many = size_of(fn, make(*[1] * 1000), 1000)
        assert rc == nm.MUON_OK and empty <= one < many < 200_000
        assert size_of(fn, make(1), -1)[0] == nm.MUON_EINVAL
        assert size_of(fn, make(1), (1 << 20) + 1)[0] == nm.MUON_EINVAL
        assert size_of(fn, None, 1)[0] == nm.MUON_EINVAL
        assert getattr(nm.lib(), fn)(make(1), 1, None) == nm.MUON_EINVAL


def test_workspace_refusals():
    lst = nm.muon_grad_list()
    arr = grads(100)
    need = size_of("muon_grad_list_size", arr, 1)[1]
    init = nm.lib().muon_grad_list_init
    assert init(arr, 1, None, need, None, ctypes.byref(lst)) == nm.MUON_EINVAL
    assert init(arr, 1, ctypes.c_void_p(BASE + 64), need, None, ctypes.byref(lst)) == nm.MUON_EINVAL
    assert init(arr, 1, ctypes.c_void_p(1 << 32), need - 1, None, ctypes.byref(lst)) == nm.MUON_ENOSPC
    assert init(arr, 1, ctypes.c_void_p(1 << 32), need, None, None) == nm.MUON_EINVAL
    # A workspace that reaches into the tensor, or starts inside it.
    for at in (BASE, (BASE - need) // 256 * 256 + 256):
        assert init(arr, 1, ctypes.c_void_p(at), need, None, ctypes.byref(lst)) == nm.MUON_EALIAS
    many = adamw(1 << 20)
    need = size_of("adamw_list_size", many, 1)[1]
    alist = nm.adamw_list()
    assert nm.lib().adamw_list_init(many, 1, ctypes.c_void_p(many[0].v + 256), need, None,
                                    ctypes.byref(alist)) == nm.MUON_EALIAS


def test_calls_refuse_a_handle_that_no_init_filled():
    """An uninitialised, foreign or changed handle reaches no kernel."""
    lib = nm.lib()
    clip = nm.muon_clip(BASE, 1.0, 0)
    hp = nm.adamw_hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1)
    for fill in (0, 0xFFFFFFFFFFFFFFFF, 0x6d756f6e67726164, 0x6d756f6e6164616d):
        g, a = nm.muon_grad_list(), nm.adamw_list()
        for i in range(8):
            g.opaque[i] = a.opaque[i] = fill
        assert lib.muon_grad_norm(ctypes.byref(g), 0, ctypes.c_void_p(BASE), None) == nm.MUON_EINVAL
        assert lib.muon_grad_clip(ctypes.byref(g), ctypes.byref(clip), None) == nm.MUON_EINVAL
        assert lib.muon_grad_clip_norm(ctypes.byref(g), 0, 1.0, ctypes.c_void_p(BASE), None) == nm.MUON_EINVAL
        assert lib.adamw_list_step(ctypes.byref(a), ctypes.byref(hp), None, None) == nm.MUON_EINVAL
        assert "init" in nm.last_error()
    assert lib.muon_grad_norm(None, 0, ctypes.c_void_p(BASE), None) == nm.MUON_EINVAL
    assert lib.adamw_list_step(None, ctypes.byref(hp), None, None) == nm.MUON_EINVAL


@pytest.mark.skipif(_gpu_visible(), reason="valid call with fake pointers: only without a GPU")
def test_valid_layout_without_gpu_reports_hip_error():
    lst = nm.muon_grad_list()
    arr = grads(100)
    assert nm.lib().muon_grad_list_init(arr, 1, ctypes.c_void_p(1 << 32), 1 << 20, None,
                                        ctypes.byref(lst)) == nm.MUON_EHIP


def test_clipped_muon_step_refusals():
    from tests.test_abi import HP, mats

    def run(norm=1 << 30, max_norm=1.0, reserved=0, arr=None):
        clip = nm.muon_clip(norm, max_norm, reserved)
        return nm.lib().muon_step_clipped(arr or mats((8, 8), (8, 16)), 2, ctypes.byref(HP), ctypes.byref(clip),
                                          ctypes.c_void_p(1 << 32), 1 << 39, None)

    a = mats((8, 8), (8, 16))
    assert run(norm=0) == nm.MUON_EINVAL and run(norm=(1 << 30) + 2) == nm.MUON_EINVAL
    assert run(max_norm=-1.0) == nm.MUON_EINVAL and run(max_norm=math.inf) == nm.MUON_EINVAL
    assert run(max_norm=math.nan) == nm.MUON_EINVAL and run(reserved=1) == nm.MUON_EINVAL
    for out, n in ((a[0].param, 8 * 8 * 2), (a[1].momentum, 8 * 16 * 2)):
        assert run(norm=out) == nm.MUON_EALIAS and run(norm=out + n - 4) == nm.MUON_EALIAS
    for at in (1 << 32, (1 << 32) + (1 << 39) - 4):
        assert run(norm=at) == nm.MUON_EALIAS  # in the workspace
    if not _gpu_visible():  # just outside: valid, and stops at the first HIP call
        assert run(norm=a[0].param - 4) == nm.MUON_EHIP and run(norm=a[0].param + 8 * 8 * 2) == nm.MUON_EHIP
    bad = mats((8, 8), (8, 16))
    bad[1].rows = -1
    assert run(arr=bad) == nm.MUON_EINVAL
    # No clip: muon_step's own refusals.
    assert nm.lib().muon_step_clipped(bad, 2, ctypes.byref(HP), None, ctypes.c_void_p(1 << 32), 1 << 40,
                                      None) == nm.MUON_EINVAL


def test_binding_refusals():
    b, f, h = (torch.zeros(4, 6, dtype=t) for t in (torch.bfloat16, torch.float32, torch.float16))
    with pytest.raises(ValueError, match="contiguous"):
        nm.GradClip([b.t()])
    with pytest.raises(ValueError, match="contiguous"):
        nm.GradClip([f[:, :3]])
    with pytest.raises(TypeError, match="float16"):
        nm.GradClip([f, h])
    with pytest.raises(ValueError, match="one GPU"):
        nm.GradClip([f])
    with pytest.raises(ValueError, match="one GPU"):
        nm.AdamWStep([b], [b.clone()], [f], [f.clone()])
    with pytest.raises(ValueError, match="same length"):
        nm.adamw_array([b], [b], [f], [])
    with pytest.raises(ValueError, match="same length"):
        nm.adamw_array([b], [b], [f], [f], masters=[None, None])
    with pytest.raises(ValueError, match="shape"):
        nm.adamw_array([b], [b], [f], [f.reshape(6, 4)])
    with pytest.raises(TypeError, match="v must be float32"):
        nm.adamw_array([b], [b], [f], [b])
    with pytest.raises(TypeError, match="master must be float32"):
        nm.adamw_array([b], [b], [f], [f], masters=[b])
    with pytest.raises(ValueError, match="kind of norm"):
        nm._norm_kind(2)


# --- the oracle ---------------------------------------------------------------------------

def test_oracle_norm_by_hand():
    assert grad_norm([[3.0], [], [4.0]]) == 5.0
    assert grad_norm([[3.0, -7.0], [4.0]], "inf") == 7.0
    assert grad_norm([]) == 0.0 and grad_norm([[]], "inf") == 0.0
    assert grad_norm([[3e200], [4e200]]) == pytest.approx(5e200, rel=1e-15)
    assert grad_norm([[3e-200], [4e-200]]) == pytest.approx(5e-200, rel=1e-15)
    for kind in ("l2", "inf"):
        assert math.isinf(grad_norm([[1.0, -math.inf]], kind))
        assert math.isnan(grad_norm([[math.inf], [math.nan]], kind))


def test_oracle_clip_by_hand():
    assert clip_coef(1.0, 2.0) == 1.0
    assert clip_coef(4.0 - 1e-6, 1.0) == 0.25
    assert clip_coef(math.inf, 1.0) == 0.0 and math.isnan(clip_coef(math.nan, 1.0))
    np.testing.assert_array_equal(clip_grads([[8.0, -4.0]], 4.0 - 1e-6, 1.0)[0], [2.0, -1.0])
