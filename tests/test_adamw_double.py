"""CPU tests of the AdamW entry points with 64-bit hyperparameters: refusals."""

from __future__ import annotations

import ctypes
import math

import pytest

import newton_schulz_02_amd as nm
from tests.test_abi import _gpu_visible

BASE = 1 << 40


@pytest.mark.parametrize("change", [dict(lr=math.nan), dict(lr=1e300), dict(eps=math.inf), dict(weight_decay=-math.inf),
                                    dict(beta1=1.0), dict(beta2=-1e-300), dict(beta2=1.0), dict(step=0),
                                    dict(reserved=1)])
def test_adamw_double_refusals(change):
    hp = nm.adamw_hparams_double(1e-3, 0.9, 0.999, 1e-8, 0.1, 1, 0)
    for name, x in change.items():
        setattr(hp, name, x)
    p = [ctypes.c_void_p(BASE + (i << 20)) for i in range(4)]
    assert nm.lib().adamw_step_double(*p, 16, ctypes.byref(hp), None) == nm.MUON_EINVAL
    assert nm.lib().adamw_step_double(*p, 16, None, None) == nm.MUON_EINVAL
    assert nm.lib().adamw_list_step_double(None, ctypes.byref(hp), None, None) == nm.MUON_EINVAL
    if not _gpu_visible():  # betas that fp32 cannot hold below 1 are valid
        good = nm.adamw_hparams_double(1e-3, 0.9, 1 - 2.0 ** -50, 1e-8, 0.1, 1, 0)
        assert nm.lib().adamw_step_double(*p, 16, ctypes.byref(good), None) == nm.MUON_EHIP
