"""GPU: muon_step with clipped gradients, and the whole update of a training step as it is used:
the global norm over matrices and other parameters, then Muon and AdamW that clip by it.

Tolerances: the momentum's as in gpu_helpers (one storage ulp of beta M + c G, plus 2^-22 of the
magnitudes, which covers the 5 * 2^-24 of the clip coefficient and its product with G); the
updates' as in gpu_helpers.TOL; AdamW's as in test_gpu_list_ops."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import newton_schulz_02_amd as nm
from newton_schulz_02_amd import workloads as W
from oracle import muon_step as oracle_step
from oracle.grad_oracle import clip_coef, grad_norm
from tests.gpu_helpers import DEV, TOL, log, momentum_ok, relf, to64
from tests.test_gpu_list_ops import BF16, F32, Adam, norm_close

pytestmark = pytest.mark.gpu


def _muon(shapes, dtype, seed):
    wl = W.custom("clipped", shapes, dtype=dtype, seed=seed)
    items = list(W.generate(wl))
    dev = [[t.to(DEV) for t in (w, g, m)] for _, w, g, m in items]
    step = nm.MuonStep([x[0] for x in dev], [x[1] for x in dev], [x[2] for x in dev], lr=wl.lr, beta=wl.beta,
                       coeffs=wl.coeffs, steps=wl.steps, eps=wl.eps)
    return wl, items, dev, step


def _check(wl, items, dev, coef):
    for (spec, w0, g, m0), (w1, g1, m1) in zip(items, dev):
        assert torch.equal(g1.cpu(), g)  # gradients unchanged
        cg = torch.from_numpy(coef * to64(g))
        assert momentum_ok(m0, cg, m1, wl.beta, spec.dtype), f"{spec.rows}x{spec.cols}: momentum"
        want, _ = oracle_step(to64(w0), cg.numpy(), to64(m0), lr=wl.lr, beta=wl.beta, coeffs=wl.coeffs,
                              steps=wl.steps, eps=wl.eps)
        err = relf(to64(w1) - to64(w0), want - to64(w0))
        log(f"  {spec.rows}x{spec.cols} {spec.dtype}: relF {err:.3e}")
        assert err <= TOL[spec.dtype]


# Aligned and odd sizes: the vector and the element path of the momentum kernel.
SHAPES = [(256, 512), (129, 77), (300, 200), (1, 40)]


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("norm,max_norm", [(5.0, 1.0), (0.2, 1.0), (1.0, 0.0)])
def test_clipped_muon_step(dtype, norm, max_norm):
    log(f"clipped muon {dtype} {norm} {max_norm}")
    wl, items, dev, step = _muon(SHAPES, dtype, 5)
    step(clip=(torch.tensor(norm, device=DEV), max_norm))
    step.check()
    _check(wl, items, dev, clip_coef(norm, max_norm))


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_a_norm_below_the_limit_is_the_unclipped_step(dtype):
    log(f"unclipped muon {dtype}")
    _, _, a, sa = _muon(SHAPES, dtype, 6)
    _, _, b, sb = _muon(SHAPES, dtype, 6)
    sa()
    sb(clip=(torch.tensor([0.5], device=DEV), 0.75))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for xa, xb in zip(a, b) for x, y in zip(xa, xb))
    nm.muon_step([x[0] for x in a], [x[1] for x in a], [x[2] for x in a])
    nm.muon_step([x[0] for x in b], [x[1] for x in b], [x[2] for x in b], clip=(torch.tensor(0.5, device=DEV), 0.75))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for xa, xb in zip(a, b) for x, y in zip(xa, xb))


def test_norm_muon_and_adamw_of_one_step():
    """One training step's update on each of two streams: Muon on matrices, AdamW on an embedding
    with a master and on fp32 vectors, all clipped by the norm of all gradients."""
    log("one step's update")
    wl, items, dev, step = _muon(SHAPES, W.BF16, 7)
    rest = Adam([1000 * 33, 77, 4096], ["master/bf16", "f32/f32", "f32/f32"], 8)
    adam = rest.step()
    grads = [x[1] for x in dev] + rest.g
    want = grad_norm([to64(g) for g in grads])
    lst = nm.GradClip(grads)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    limit = want / 3
    norm = lst.norm()
    side.wait_stream(torch.cuda.current_stream())
    step(clip=(norm, limit))
    adam(5, clip=(norm, limit), stream=side)
    torch.cuda.synchronize()
    step.check()
    assert norm_close(norm, want)
    # The limit reaches the kernels as fp32, half a step of which the tolerances' 5 u do not
    # contain: the oracle takes the rounded one.
    coef = clip_coef(want, float(np.float32(limit)))
    assert coef < 0.34
    _check(wl, items, dev, coef)
    rest.check(5, coef)


def test_clipped_step_refusals_of_the_binding():
    _, _, _, step = _muon([(64, 64)], W.BF16, 9)
    with pytest.raises(ValueError, match="norm must be"):
        step(clip=(torch.ones(()), 1.0))
    with pytest.raises(nm.MuonError):
        step(clip=(torch.ones((), device=DEV), -1.0))
