"""CPU tests of the hash that versions the tuning tables: which sources it covers."""

from __future__ import annotations

import shutil

import pytest

from newton_schulz_02_amd import build


@pytest.fixture
def sources(tmp_path, monkeypatch):
    copy = tmp_path / "csrc"
    shutil.copytree(build.CSRC, copy)
    monkeypatch.setattr(build, "CSRC", copy)
    return copy


@pytest.mark.parametrize("name", ["kernels_list.hip", "list_math.h", "list_plan.h", "list_types.h"])
def test_the_list_operators_do_not_make_saved_tables_stale(sources, name):
    before = build.kernel_hash()
    with open(sources / name, "a") as f:
        f.write("// changed\n")
    assert build.kernel_hash() == before


@pytest.mark.parametrize("name", ["kernels_gemm.hip", "kernels_gemm_wide.hip", "split_fixup.h", "split_protocol.h",
                                  "tile_order.h", "muon_internal.h", "planner.h"])
def test_the_tuned_kernels_do(sources, name):
    before = build.kernel_hash()
    with open(sources / name, "a") as f:
        f.write("// changed\n")
    assert build.kernel_hash() != before


def test_no_tuned_kernel_includes_a_list_source(sources):
    """Directly or through another header."""
    seen, todo = set(), ["kernels_gemm.hip", "kernels_gemm_wide.hip"]
    while todo:
        name = todo.pop()
        if name in seen or not (sources / name).is_file():
            continue
        seen.add(name)
        todo += [line.split('"')[1] for line in (sources / name).read_text().splitlines()
                 if line.startswith('#include "')]
    assert "muon_internal.h" in seen and not seen & build.LIST_SOURCES
