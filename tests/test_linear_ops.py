"""CPU tests of the 8-bit linear operators' host side: refusals, workspace sizes, the oracle.

No test here launches a kernel: pointers are fake numbers, and calls that pass validation are
made only where no GPU is visible (they then stop at the first HIP call)."""

from __future__ import annotations

import ctypes
import shutil
import subprocess

import numpy as np
import pytest
import torch

import newton_schulz_02_amd as nm
from newton_schulz_02_amd import build
from oracle import linear_oracle as lo
from tests.test_abi import _gpu_visible

BASE = 1 << 40
FAR = 1 << 36  # apart from each other


def view(rows, cols, *, at=BASE, ld=None, dtype=nm.MUON_BF16):
    return nm.muon_view(at, rows, cols, cols if ld is None else ld, dtype, 0)


def codes(rows, cols, *, at=BASE + FAR, block=0):
    return nm.muon_codes(at, at + FAR // 2, rows, cols, block, 0)


def ref(x):
    return None if x is None else ctypes.byref(x)


WS = ctypes.c_void_p(1 << 46)


def quantize(x, c, transpose=0, ws=WS, size=1 << 40):
    return nm.lib().muon_quantize(ref(x), transpose, ref(c), ws, size, None)


def dequantize(c, out):
    return nm.lib().muon_dequantize(ref(c), ref(out), None)


def matmul(a, b, out, ws=WS, size=1 << 40):
    return nm.lib().muon_int8_matmul(ref(a), ref(b), ref(out), ws, size, None)


def linear(x, w, out, ws=WS, size=1 << 40):
    return nm.lib().muon_int8_linear(ref(x), ref(w), ref(out), ws, size, None)


def wgrad(dy, x, out, accumulate=0, ws=WS, size=1 << 40):
    return nm.lib().muon_weight_grad(ref(dy), ref(x), ref(out), accumulate, ws, size, None)


def good(call):
    """A call that passes validation: without a GPU it stops at the first HIP call."""
    if _gpu_visible():
        return
    assert call() == nm.MUON_EHIP, nm.last_error()


OUT = BASE + 4 * FAR


@pytest.mark.parametrize("call,code", [
    (lambda: quantize(None, codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), None), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8, at=0), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8, at=BASE + 1), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8, at=BASE + 2, dtype=nm.MUON_F32), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8, dtype=3), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8, ld=7), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8, ld=0), codes(4, 8)), nm.MUON_EINVAL),  # one row repeated
    (lambda: quantize(view(4, 8, ld=-8), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(-1, 8), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, (1 << 30) + 1), codes(4, (1 << 30) + 1)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8, at=2 ** 64 - 16), codes(4, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(1 << 30, 8, ld=1 << 32, dtype=nm.MUON_F32), codes(1 << 30, 8)), nm.MUON_EINVAL),  # 2^64 bytes
    (lambda: quantize(view(1 << 30, 8, ld=(1 << 32) + 1), codes(1 << 30, 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), codes(8, 4)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), codes(4, 8), 1), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), codes(8, 4), 2), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), codes(8, 4, block=128), 1), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), codes(4, 8, block=64)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), codes(4, 8, at=BASE + FAR + 8)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), nm.muon_codes(OUT, 0, 4, 8, 0, 0)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), nm.muon_codes(OUT, OUT + 4096, 4, 8, 0, 1)), nm.MUON_EINVAL),
    (lambda: quantize(view(4, 8), nm.muon_codes(OUT, OUT + 256, 4, 8, 0, 0)), nm.MUON_EALIAS),  # scales in the codes
    (lambda: quantize(view(4, 8), codes(4, 8, at=BASE)), nm.MUON_EALIAS),
    (lambda: quantize(view(300, 512), codes(512, 300), 1, ws=None), nm.MUON_EINVAL),
    (lambda: quantize(view(300, 512), codes(512, 300), 1, ws=ctypes.c_void_p((1 << 46) + 64)), nm.MUON_EINVAL),
    (lambda: quantize(view(300, 512), codes(512, 300), 1, size=512 * 4 - 1), nm.MUON_ENOSPC),
    (lambda: quantize(view(300, 512), codes(512, 300), 1, ws=ctypes.c_void_p(BASE + 256)), nm.MUON_EALIAS),
    (lambda: quantize(view(300, 512), codes(512, 300), 1, ws=ctypes.c_void_p(BASE + FAR)), nm.MUON_EALIAS),
    (lambda: dequantize(None, view(4, 8, at=OUT)), nm.MUON_EINVAL),
    (lambda: dequantize(codes(4, 8), None), nm.MUON_EINVAL),
    (lambda: dequantize(codes(4, 8), view(4, 9, at=OUT)), nm.MUON_EINVAL),
    (lambda: dequantize(codes(4, 8), view(4, 8, at=BASE + FAR)), nm.MUON_EALIAS),
    (lambda: dequantize(codes(4, 8), view(4, 8, at=BASE + FAR + FAR // 2)), nm.MUON_EALIAS),
    (lambda: matmul(None, codes(4, 8), view(4, 4)), nm.MUON_EINVAL),
    (lambda: matmul(codes(4, 8), codes(4, 9, at=OUT), view(4, 4)), nm.MUON_EINVAL),
    (lambda: matmul(codes(4, 8, block=128), codes(4, 8, at=OUT), view(4, 4)), nm.MUON_EINVAL),
    (lambda: matmul(codes(4, 8), codes(4, 8, at=OUT, block=128), view(4, 4)), nm.MUON_EINVAL),
    (lambda: matmul(codes(4, 131072), codes(4, 131072, at=OUT), view(4, 4)), nm.MUON_EINVAL),  # sums leave 32 bits
    (lambda: matmul(codes(4, 8), codes(5, 8, at=OUT), view(4, 4)), nm.MUON_EINVAL),
    (lambda: matmul(codes(4, 8), codes(5, 8, at=OUT), None), nm.MUON_EINVAL),
    (lambda: matmul(codes(4, 8), codes(5, 8, at=OUT), view(4, 5, at=OUT)), nm.MUON_EALIAS),
    (lambda: matmul(codes(1, 8), codes((1 << 26) + 1, 8, at=OUT), view(1, (1 << 26) + 1)), nm.MUON_EINVAL),
    (lambda: matmul(codes(1 << 20, 8), codes(1 << 20, 8, at=OUT), view(1 << 20, 1 << 20)), nm.MUON_EINVAL),
    (lambda: linear(None, codes(4, 8), view(4, 4, at=OUT)), nm.MUON_EINVAL),
    (lambda: linear(view(4, 8), None, view(4, 4, at=OUT)), nm.MUON_EINVAL),
    (lambda: linear(view(4, 8), codes(4, 8), None), nm.MUON_EINVAL),
    (lambda: linear(view(4, 9), codes(4, 8), view(4, 4, at=OUT)), nm.MUON_EINVAL),
    (lambda: linear(view(4, 8), codes(4, 8), view(4, 4)), nm.MUON_EALIAS),
    (lambda: linear(view(100, 8), codes(4, 8), view(100, 4, at=OUT), ws=None), nm.MUON_EINVAL),
    (lambda: linear(view(100, 8), codes(4, 8), view(100, 4, at=OUT), size=100 * 128), nm.MUON_ENOSPC),
    (lambda: linear(view(100, 8), codes(4, 8), view(100, 4, at=OUT), ws=ctypes.c_void_p(OUT + 256)), nm.MUON_EALIAS),
    (lambda: wgrad(None, codes(64, 8, block=128), view(16, 8, at=OUT)), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 16), None, view(16, 8, at=OUT)), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 16), codes(64, 8, block=128), None), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 16), codes(64, 8), view(16, 8, at=OUT)), nm.MUON_EINVAL),  # codes by row
    (lambda: wgrad(view(64, 16), codes(65, 8, block=128), view(16, 8, at=OUT)), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 16), codes(64, 8, block=128), view(8, 16, at=OUT)), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 16), codes(64, 8, block=128), view(16, 8, at=OUT), 2), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 16), codes(64, 8, block=128), view(16, 8)), nm.MUON_EALIAS),
    (lambda: wgrad(view(64, 16), codes(64, 8, block=128), view(16, 8, at=BASE + FAR)), nm.MUON_EALIAS),
    (lambda: wgrad(view(1, 1 << 24), codes(1, 8, block=128), view(1 << 24, 8, at=OUT)), nm.MUON_EINVAL),
    (lambda: wgrad(view(1, 8), codes(1, 1 << 24, block=128), view(8, 1 << 24, at=OUT)), nm.MUON_EINVAL),
    (lambda: quantize(view(1 << 20, 1 << 19), codes(1 << 19, 1 << 20, at=1 << 44), 1, size=1 << 45), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 15), codes(64, 8, block=128), view(15, 8, at=OUT), ws=None), nm.MUON_EINVAL),
    (lambda: wgrad(view(64, 15), codes(64, 8, block=128), view(15, 8, at=OUT), size=64 * 16 * 2 - 1), nm.MUON_ENOSPC),
    (lambda: wgrad(view(64, 15), codes(64, 8, block=128), view(15, 8, at=OUT), ws=ctypes.c_void_p(BASE)), nm.MUON_EALIAS),
])
def test_refusals(call, code):
    assert call() == code
    assert nm.last_error()


def test_calls_that_are_not_refused_reach_the_device():
    good(lambda: quantize(view(4, 8), codes(4, 8), ws=None, size=0))
    good(lambda: quantize(view(0, 8, at=0), nm.muon_codes(0, 0, 0, 8, 0, 0), ws=None, size=0))
    good(lambda: quantize(view(300, 512), codes(512, 300), 1))
    good(lambda: dequantize(codes(4, 8, block=128), view(4, 8, ld=20, at=OUT)))
    good(lambda: matmul(codes(4, 131071), codes(4, 131071, at=OUT), view(4, 4), ws=None, size=0))
    good(lambda: linear(view(1, 4096), codes(4, 4096), view(1, 4, at=OUT), ws=None, size=0))
    good(lambda: wgrad(view(64, 16), codes(64, 8, block=128), view(16, 8, at=OUT), ws=None, size=0))
    # x and out are columns of one wider buffer: they do not overlap, though their ranges do.
    good(lambda: linear(view(9, 16, ld=48), codes(32, 16), view(9, 32, ld=48, at=BASE + 32)))
    good(lambda: linear(view(9, 16, ld=48, at=BASE + 64), codes(32, 16), view(9, 32, ld=48)))


def test_rows_of_one_buffer_that_do_overlap_are_refused():
    assert linear(view(9, 16, ld=48), codes(32, 16), view(9, 32, ld=48, at=BASE + 30)) == nm.MUON_EALIAS
    assert linear(view(9, 16, ld=48), codes(32, 16), view(9, 32, ld=48, at=BASE + 34)) == nm.MUON_EALIAS  # its next row
    assert linear(view(9, 16, ld=48), codes(32, 16), view(9, 32, ld=47, at=BASE + 32)) == nm.MUON_EALIAS


def size_of(fn, *args):
    out = ctypes.c_size_t(0)
    rc = getattr(nm.lib(), fn)(*args, ctypes.byref(out))
    return rc, out.value


def test_workspace_sizes():
    assert size_of("muon_quantize_size", ref(view(300, 512)), 0) == (0, 0)
    rc, n = size_of("muon_quantize_size", ref(view(300, 512)), 1)
    assert rc == 0 and n % (512 * 4) == 0 and 512 * 4 <= n <= 32 * 512 * 4
    assert size_of("muon_int8_matmul_size", ref(codes(4, 8)), ref(codes(4, 8, at=OUT)))[0] == 0
    rc, n = size_of("muon_int8_linear_size", ref(view(100, 130)), ref(codes(4, 130)))
    assert rc == 0 and n >= 100 * 256 + 400
    assert size_of("muon_int8_linear_size", ref(view(1, 4096)), ref(codes(4, 4096))) == (0, 0)
    rc, n = size_of("muon_weight_grad_size", ref(view(64, 15)), ref(codes(64, 8, block=128)))
    assert rc == 0 and n >= 64 * 16 * 2
    for fn, args in (("muon_quantize_size", (None, 0)), ("muon_int8_matmul_size", (None, ref(codes(4, 8)))),
                     ("muon_int8_linear_size", (None, ref(codes(4, 8)))),
                     ("muon_weight_grad_size", (None, ref(codes(4, 8, block=128))))):
        assert size_of(fn, *args)[0] == nm.MUON_EINVAL
    assert nm.lib().muon_quantize_size(ref(view(4, 8)), 0, None) == nm.MUON_EINVAL


@pytest.mark.parametrize("tokens,outputs,ld,inputs,pieces", [(777, 517, 524, 1031, 3), (8192, 768, 768, 768, 7),
                                                             (512, 768, 768, 768, 1), (4096, 4096, 4096, 4096, 1)])
def test_pieces_of_a_weight_gradient(tokens, outputs, ld, inputs, pieces):
    """The plans whose times the cost model's comment gives: each piece has its partial results in the workspace."""
    rc, n = size_of("muon_weight_grad_size", ref(view(tokens, outputs, ld=ld)), ref(codes(tokens, inputs, block=128)))
    assert rc == 0 and n == (pieces * outputs * inputs * 4 if pieces > 1 else 0)


@pytest.mark.parametrize("call,kind", [
    (lambda x: nm.quantize(x), ValueError),
    (lambda x: nm.Codes.empty(4, 8, device="cpu"), ValueError),
    (lambda x: nm.Codes(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4), 8), ValueError),
    (lambda x: nm.Codes(torch.zeros(4, 128), torch.zeros(4), 8), ValueError),
    (lambda x: nm.Codes(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(5), 8), ValueError),
    (lambda x: nm.Codes(torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4), 200, block=True), ValueError),
    (lambda x: nm._view_arg("x", x[0]), ValueError),
    (lambda x: nm._view_arg("x", x.t()), ValueError),
    (lambda x: nm._view_arg("x", x[:1].expand(3, 8)), ValueError),
    (lambda x: nm._view_arg("x", x.half()), TypeError),
])
def test_binding_refusals(call, kind):
    with pytest.raises(kind):
        call(torch.zeros(4, 8))


def leaf(*shape):
    return torch.zeros(*shape).requires_grad_()


CALLS_WITH_A_GRADIENT = [
    lambda x: nm.quantize(x),
    lambda x: nm.quantize(x, block=True),
    lambda x: nm.quantize(x * 2.0, transpose=True),  # not a leaf
    lambda x: nm.quantize(torch.zeros(4, 8), out=x),
    lambda x: nm.dequantize(x.detach(), out=x),
    lambda x: nm.int8_matmul(x, x.detach()),
    lambda x: nm.int8_matmul(x.detach(), x),
    lambda x: nm.int8_linear(x, x.detach()),
    lambda x: nm.int8_linear(x.detach(), x.detach(), out=x),
    lambda x: nm.weight_grad(x, x.detach()),
    lambda x: nm.weight_grad(x.detach(), x.detach(), out=x, accumulate=True),
    lambda x: nm.Codes(torch.zeros(4, 128, dtype=torch.int8), leaf(4), 8),
]


@pytest.mark.parametrize("call", CALLS_WITH_A_GRADIENT)
def test_operands_that_need_a_gradient_are_refused(call):
    """The calls record no graph: a gradient would be lost without a word."""
    with pytest.raises(ValueError, match="needs a gradient"):
        call(leaf(4, 8))
    with torch.no_grad(), pytest.raises(ValueError, match="on a GPU"):  # as of any tensor here
        call(leaf(4, 8))


@pytest.mark.parametrize("call", CALLS_WITH_A_GRADIENT[:-1])
def test_operands_with_a_tangent_are_refused(call):
    with torch.autograd.forward_ad.dual_level():
        x = torch.autograd.forward_ad.make_dual(torch.zeros(4, 8), torch.ones(4, 8))
        x.detach = lambda: torch.zeros(4, 8)  # keeps a tangent otherwise
        with torch.no_grad(), pytest.raises(ValueError, match="needs a gradient"):
            call(x)


def test_a_function_may_call_the_operators():
    """Inside a torch.autograd.Function gradients are off: the call goes on to its other checks."""
    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            with pytest.raises(ValueError, match="on a GPU"):
                nm.quantize(x, block=True)
            return x.clone()

        @staticmethod
        def backward(ctx, dy):
            with pytest.raises(ValueError, match="on a GPU"):
                nm.weight_grad(dy, dy)
            return dy

    x = leaf(4, 8)
    Layer.apply(x).sum().backward()
    assert x.grad.eq(1).all()


def test_views_of_single_rows_and_columns():
    x = torch.zeros(6, 8)
    for t, want in ((x[:, 2:5], (6, 3, 8)), (x[:1].expand(1, 8), (1, 8, 8)), (x[:, :1], (6, 1, 8)),
                    (x[::2], (3, 8, 16)), (x[2:2], (0, 8, 8))):
        v = nm._view_arg("x", t)
        assert (v.rows, v.cols, v.ld) == want and v.dtype == nm.MUON_F32


@pytest.mark.parametrize("name", sorted(build.LINEAR_SOURCES))
def test_the_linear_operators_do_not_make_saved_tuning_tables_stale(name, tmp_path, monkeypatch):
    import shutil

    copy = tmp_path / "csrc"
    shutil.copytree(build.CSRC, copy)
    monkeypatch.setattr(build, "CSRC", copy)
    before = build.kernel_hash()
    with open(copy / name, "a") as f:
        f.write("// changed\n")
    assert build.kernel_hash() == before


# --- the oracle ----------------------------------------------------------------------------------

def test_oracle_codes():
    q, s = lo.row_codes([[254.0, 1.0, -3.0, 0.0], [0.0, 0.0, 0.0, 0.0], [1.0, np.inf, 0.0, 0.0], [127.0, 0.5, 1.5, -2.5]])
    assert q.tolist() == [[127, 0, -2, 0], [0, 0, 0, 0], [0, 0, 0, 0], [127, 0, 2, -2]]
    assert s[0] == 2.0 and s[1] == 0.0 and np.isnan(s[2]) and s[3] == 1.0
    x = np.zeros((1, 130))
    x[0, :4] = [127.0, 0.5, 1.5, -3.0]
    x[0, 128:] = [127.5, 1.0]
    q, s = lo.block_codes(x)
    assert s.tolist() == [[1.0, 2.0]]
    assert q[0, :4].tolist() == [127, 0, 2, -3] and q[0, 128:].tolist() == [64, 0]


def test_oracle_block_values_are_bf16_numbers():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 300)) * 10.0 ** rng.integers(-30, 30, (50, 1))
    values = lo.decode(*lo.block_codes(x), True)
    t = torch.from_numpy(values)
    assert torch.equal(t.to(torch.bfloat16).double(), t)
    top = np.repeat(np.abs(np.pad(x, ((0, 0), (0, 84)))).reshape(50, 3, 128).max(axis=2), 128, axis=1)[:, :300]
    # A step is less than 2 / 127 of the largest value, a rounding half a step.
    assert (np.abs(values - x) <= top / 127.0).all()


def test_oracle_gradient_is_the_difference_quotient():
    """L(W) = sum(dy * (x W^T)) is linear in W: its differences are the gradient."""
    rng = np.random.default_rng(2)
    x, dy, w = rng.standard_normal((7, 130)), rng.standard_normal((7, 5)), rng.standard_normal((5, 130))
    codes_, scale = lo.block_codes(x)
    kept = lo.decode(codes_, scale, True)
    dw, _ = lo.weight_grad(dy, codes_, scale)
    loss = lambda m: float((dy * (kept @ m.T)).sum())  # noqa: E731
    for i, j in ((0, 0), (4, 129), (2, 77)):
        e = np.zeros_like(w)
        e[i, j] = 1.0
        assert abs((loss(w + e) - loss(w - e)) / 2 - dw[i, j]) < 1e-10


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_row_distances_of_any_size_are_looked_at_without_overflow(tmp_path):
    """The host's checks, compiled to stop at a signed overflow: ld is free where there is one row (or
    none), and refused beyond [cols, 2^32] otherwise."""
    (tmp_path / "main.cpp").write_text("""
        #include "linear_plan.h"
        int main() {
          std::string err;
          muon::QuantPlan p;
          for (int64_t ld : {INT64_MAX, INT64_MIN, int64_t(1) << 62, -(int64_t(1) << 61), int64_t(1) << 33, int64_t(7)})
            for (int32_t dtype : {MUON_BF16, MUON_F32})
              for (int64_t rows = 0; rows < 3; ++rows) {
                const muon_view x = {reinterpret_cast<void*>(uintptr_t(1) << 40), rows, 8, ld, dtype, 0};
                if (muon::plan_quantize(&x, 0, nullptr, &p, &err) != (rows > 1 ? MUON_EINVAL : MUON_OK)) return 1;
              }
          return 0;
        }""")
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", f"-I{build.CSRC}",
                    str(tmp_path / "main.cpp"), str(build.CSRC / "linear_plan.cpp"), "-o", str(tmp_path / "main")],
                   check=True, timeout=120)
    run = subprocess.run([str(tmp_path / "main")], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stderr
