"""GPU: AdamW's state follows the betas that the caller gives, not their fp32 roundings.

Tolerances, u = 2^-24 (half a step of fp32), r = 1 - beta:
  m  r is rounded (u), so is its product with g (u) and the sum with the low part of beta times m
     (u of r|g|, and of |m| 2^-24, since that part is below 2^-24); the last product and sum are one
     rounding: u (|m'| + 3 r|g| + 2^-22 |m|).
  v  r, r g and r g g are three roundings, the rest as for m: u (v' + 4 r g^2 + 2^-22 v).
  each, and the smallest denormal per rounding.  The parameter's bounds are those of
  test_gpu_parity, with betas as exact as here.
A beta rounded to fp32 is up to u off, so u r^-1 relative in r: 1.3e-5 at 0.999."""

from __future__ import annotations

import ctypes
import types

import numpy as np
import pytest
import torch

import newton_schulz_02_amd as nm
from oracle import adamw_step as oracle_adamw
from tests.gpu_helpers import DEV, log, to64
from tests.test_gpu_list_ops import KINDS
from tests.test_gpu_parity import adamw_bounds

pytestmark = pytest.mark.gpu

U = 2.0 ** -24 * (1 + 2.0 ** -20)
TINY = 4 * 2.0 ** -149
BETAS = [(0.9, 0.999), (0.9, 0.9999), (0.95, 0.95), (0.99, 0.999999), (0.0, 0.5), (0.3, 1 - 2.0 ** -30)]
N = 4099


def state(seed, kind="f32/f32", m=1e-2, v=1e-4, g=1e-2):
    pt, gt, master = KINDS[kind]
    gen = torch.Generator(DEV).manual_seed(seed)

    def normal(std):
        return torch.randn(N, device=DEV, generator=gen) * std

    p = normal(0.5).to(pt)
    return p, normal(g).to(gt), normal(m), normal(1.0).square() * v, p.float() * (1 + 2.0 ** -10) if master else None


def check_state(m0, v0, g0, m1, v1, b1, b2):
    g0, m0, v0 = to64(g0), to64(m0), to64(v0)
    want_m, want_v = b1 * m0 + (1 - b1) * g0, b2 * v0 + (1 - b2) * g0 * g0
    em, ev = np.abs(to64(m1) - want_m), np.abs(to64(v1) - want_v)
    assert np.all(em <= U * (np.abs(want_m) + 3 * (1 - b1) * np.abs(g0) + 2.0 ** -22 * np.abs(m0)) + TINY)
    assert np.all(ev <= U * (want_v + 4 * (1 - b2) * g0 * g0 + 2.0 ** -22 * v0) + TINY)


# From a zero state the result is r g and r g^2; without gradients it is the decayed state alone.
STARTS = {"zero state": dict(m=0.0, v=0.0), "no gradient": dict(g=0.0), "both": {}}


@pytest.mark.parametrize("start", list(STARTS))
@pytest.mark.parametrize("betas", BETAS)
@pytest.mark.parametrize("kind", list(KINDS))
def test_list_state_follows_the_betas(kind, betas, start):
    log(f"adamw list {kind} betas {betas} {start}")
    p, g, m, v, w = state(3, kind, **STARTS[start])
    at, m0, v0 = (w if w is not None else p).clone(), m.clone(), v.clone()
    hp = types.SimpleNamespace(lr=1e-3, beta1=betas[0], beta2=betas[1], eps=1e-8, weight_decay=0.1)
    nm.AdamWStep([p], [g], [m], [v], masters=[w], **vars(hp))(7)
    check_state(m0, v0, g, m, v, *betas)
    want, _, _ = oracle_adamw(to64(at), to64(g), to64(m0), to64(v0), t=7, **vars(hp))
    bound = adamw_bounds(to64(at), to64(g), to64(m0), to64(v0), 7, hp)[0]
    if w is None and p.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    assert np.all(np.abs(to64(p if w is None else w) - want) <= bound)


@pytest.mark.parametrize("start", list(STARTS))
@pytest.mark.parametrize("betas", BETAS)
def test_packed_state_follows_the_betas(betas, start):
    log(f"adamw packed betas {betas} {start}")
    p, g, m, v, _ = state(4, **STARTS[start])
    m0, v0 = m.clone(), v.clone()
    nm.adamw_step(p, g, m, v, beta1=betas[0], beta2=betas[1], step=3)
    check_state(m0, v0, g, m, v, *betas)


def fma32(a, b, c):
    """fp32 multiply-add: the product of two fp32 values is exact in fp64."""
    return (np.float64(a) * b + c).astype(np.float32)


def test_float_betas_are_taken_as_they_are():
    """adamw_step and adamw_list_step of the library: betas in fp32, 1 - beta their exact
    difference from 1, bit for bit; the 64-bit forms do the same for betas that are floats."""
    log("adamw float betas")
    b1, b2 = np.float32(0.9), np.float32(0.999)
    one = np.float32(1)
    lib, stream = nm.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    results = []
    for wide in (False, True):
        hp = (nm.adamw_hparams_double if wide else nm.adamw_hparams)(1e-3, float(b1), float(b2), 1e-8, 0.1, 5)
        packed, listed = state(5)[:4], state(5)[:4]
        lst = nm.AdamWStep(*([t] for t in listed))
        g0, m0, v0 = (t.cpu().numpy() for t in packed[1:])
        args = [ctypes.c_void_p(t.data_ptr()) for t in packed]
        assert (lib.adamw_step_double if wide else lib.adamw_step)(*args, N, ctypes.byref(hp), stream) == nm.MUON_OK
        assert (lib.adamw_list_step_double if wide else lib.adamw_list_step)(
            ctypes.byref(lst.list), ctypes.byref(hp), None, stream) == nm.MUON_OK
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(packed, listed))
        np.testing.assert_array_equal(packed[2].cpu().numpy(), fma32(b1, m0, (one - b1) * g0))
        np.testing.assert_array_equal(packed[3].cpu().numpy(), fma32(b2, v0, (one - b2) * g0 * g0))
        results.append(packed)
    # The rates that are not betas are rounded to fp32 in either form.
    assert torch.equal(results[0][2], results[1][2]) and torch.equal(results[0][3], results[1][3])
    assert torch.equal(results[0][0], results[1][0])


@pytest.mark.parametrize("betas", [(0.5, 0.75), (0.9, 0.999)])
def test_an_infinite_state_stays_infinite(betas):
    """Whether beta is a float or not: beta inf + r g is infinite, not NaN."""
    log(f"adamw infinite state {betas}")
    for step in ("list", "packed"):
        p, g, m, v, _ = state(6)
        p0 = p.clone()
        v[::3] = float("inf")
        m[1::3] = float("-inf")
        if step == "list":
            nm.AdamWStep([p], [g], [m], [v], beta1=betas[0], beta2=betas[1], weight_decay=0.0)(2)
        else:
            nm.adamw_step(p, g, m, v, beta1=betas[0], beta2=betas[1], weight_decay=0.0, step=2)
        assert bool((v[::3] == float("inf")).all()) and bool((m[1::3] == float("-inf")).all())
        assert torch.equal(p[::3], p0[::3])  # no finite m moves it
        assert bool((p[1::3] == float("inf")).all())
