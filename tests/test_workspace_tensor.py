"""CPU tests: which tensors are accepted as a workspace."""

from __future__ import annotations

import pytest
import torch

import newton_schulz_02_amd as nm


def _refuses(workspace, what):
    m = torch.zeros(64, 64)
    steps = (lambda: nm.MuonStep([m], [m.clone()], [m.clone()], workspace=workspace),
             lambda: nm.ShampooStep([m], [m.clone()], [m.clone()], [m.clone()], workspace=workspace))
    for step in steps:
        with pytest.raises(ValueError, match=what):
            step()
    with pytest.raises(ValueError, match=what):
        nm._check_workspace(workspace, 1 << 20)


def test_a_workspace_with_more_elements_than_memory_is_refused():
    """One byte seen 16 million times: the kernels would write behind it."""
    _refuses(torch.zeros(1, dtype=torch.uint8).expand(1 << 24), "contiguous")
    _refuses(torch.zeros(1 << 24, dtype=torch.uint8)[::2], "contiguous")


def test_a_short_workspace_is_refused():
    _refuses(torch.zeros(256, dtype=torch.uint8), "needs")


def test_a_contiguous_part_is_accepted():
    nm._check_workspace(torch.zeros(1 << 20, dtype=torch.uint8)[256:], (1 << 20) - 256)
    m = torch.zeros(64, 64)
    nm.MuonStep([m], [m.clone()], [m.clone()], workspace=torch.zeros(1 << 24, dtype=torch.uint8)[256:])
