"""GPU: the 8-bit operators of linear layers against float64.

Tolerances.  U = 2^-24 is half a step of fp32, B = 2^-8 half a step of bf16.
  codes    are equal to the oracle's: they are defined exactly.  A row's scale is one fp32
           division (U, or half the smallest denormal); a block's is a power of two.
  values   a block's are exact in either type.  A row's are one fp32 product of the scale that the
           codes have (U) and for bf16 one rounding more.
  products the sum is exact; it is rounded to fp32, and so are its products with the two scales
           (3 U), then to bf16.  The scales are those that the codes have.
  weight gradients  the products of bf16 values are exact; a sum of n terms in fp32 in any order is
           off by at most 2 U n times the sum of the terms' magnitudes (2 U an addition, so that
           one that truncates is covered).  Products of fp32 values are rounded (1 more).  The old
           gradient's addition is U on the result, and bf16 one rounding more.  Whole numbers
           whose sums stay below 2^24 come out exactly, whatever the order."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import newton_schulz_02_amd as nm
from oracle import linear_oracle as lo
from oracle.grad_oracle import grad_norm
from tests.gpu_helpers import DEV, log, to64

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [BF16, F32]


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def normal(rows, cols, dtype, seed, pad=0, shift=0):
    """rows x cols normal values of rows of different sizes, as columns [shift, shift + cols) of a
    buffer that is NaN elsewhere."""
    g = gen(seed)
    wide = torch.full((rows, cols + pad + shift), float("nan"), device=DEV, dtype=dtype)
    x = wide[:, shift:shift + cols]
    x.copy_(torch.randn(rows, cols, device=DEV, generator=g) * torch.rand(rows, 1, device=DEV, generator=g).mul(8).exp())
    return x


def out_in(rows, cols, dtype, pad, fill=7.0):
    wide = torch.full((rows + 1, cols + pad), fill, device=DEV, dtype=dtype)
    return wide, wide[:rows, :cols]


def untouched(wide, rows, cols, fill=7.0):
    return bool((wide[rows:] == fill).all()) and bool((wide[:, cols:] == fill).all())


def check_codes(c, x, block):
    q, s = (lo.block_codes if block else lo.row_codes)(to64(x))
    got = c.q[:, :x.shape[1]].cpu().numpy()
    assert np.array_equal(got, q), f"{np.count_nonzero(got != q)} codes differ"
    assert not c.q[:, x.shape[1]:].any()  # the padding
    have = to64(c.scale).reshape(s.shape)
    if block:
        assert np.array_equal(have, s, equal_nan=True)
    else:
        assert np.array_equal(np.isnan(have), np.isnan(s))
        fine = ~np.isnan(s)
        assert (np.abs(have - s)[fine] <= s[fine] * U * (1 + 1e-6) + 2.0 ** -150).all()


# Lengths around the vector, block, wave and workgroup sizes of the kernels, and past each variant's.
SHAPES = [(1, 1), (3, 7), (1, 8), (5, 127), (4, 128), (2, 129), (130, 64), (9, 511), (3, 2048), (2, 2049), (7, 4096),
          (2, 8192), (1, 8200), (2, 12289), (3, 33000), (1, 131071), (257, 385), (1000, 96)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes(rows, cols, dtype):
    for pad, shift in ((0, 0), (5, 3)):
        x = normal(rows, cols, dtype, rows + cols, pad, shift)
        log(f"codes {rows}x{cols} {dtype} +{pad}")
        check_codes(nm.quantize(x), x, False)
        check_codes(nm.quantize(x, block=True), x, True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (300, 1), (63, 65), (64, 256), (129, 257), (2049, 40), (40, 2049), (513, 1025)])
def test_codes_of_columns(rows, cols, dtype):
    x = normal(rows, cols, dtype, rows, 3, 1)
    c = nm.quantize(x, transpose=True)
    assert c.shape == (cols, rows)
    check_codes(c, x.t(), False)


def ties(dtype):
    """Rows whose values lie in the middle between two codes, or next to it."""
    rows = []
    for top in (127.0, 254.0, 63.5, 127.0 * 2.0 ** -60, 127.0 * 2.0 ** 100):
        half = torch.arange(-126.5, 127.0, 1.0, dtype=torch.float64) * (top / 127.0)
        row = torch.cat([torch.tensor([top], dtype=torch.float64), half])
        rows += [row, row * (1 + 2.0 ** -23), row * (1 - 2.0 ** -23)]
        rows[-1][0] = rows[-2][0] = top
    # Largest values whose quotients are rounded.
    for top in (1.0, 3.0, 191.0 / 64):
        rows.append(torch.cat([torch.tensor([top], dtype=torch.float64),
                               torch.arange(-126.5, 127.0, 1.0, dtype=torch.float64) * (top / 127.0)]))
    return torch.stack(rows).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties(dtype):
    x = ties(dtype)
    check_codes(nm.quantize(x), x, False)
    check_codes(nm.quantize(x, block=True), x, True)
    check_codes(nm.quantize(x.t().contiguous(), transpose=True), x, False)
    w = nm.quantize(torch.eye(x.shape[1], device=DEV) * 127.0)  # codes 127 on the diagonal, scale 1
    y = nm.int8_linear(x[:16], w, F32)  # few rows: the codes are made inside the product
    c = nm.quantize(x[:16])
    assert torch.equal(y, (c.q[:, :x.shape[1]].int() * 127).float() * c.scale[:, None])


@pytest.mark.parametrize("exponent", [-99, -20, 0, 60, 127])
def test_every_bf16_quotient(exponent):
    """Each of the 128 mantissas as a row's largest value, with all values down to 2^-11 of it."""
    tops = (torch.arange(128, 256, dtype=torch.float64) * 2.0 ** (exponent - 7))[:, None]
    values = (torch.arange(128, 256, dtype=torch.float64) * 2.0 ** -7)[None, :] * \
        (2.0 ** torch.arange(exponent - 11, exponent + 1, dtype=torch.float64))[:, None]
    row = values.reshape(1, -1)
    x = torch.cat([tops, torch.where(row <= tops, row, -0.0 * row), -torch.where(row <= tops, row, 0.0 * row)], dim=1)
    x = x.to(BF16).to(DEV)
    check_codes(nm.quantize(x), x, False)
    check_codes(nm.quantize(x.t().contiguous(), transpose=True), x, False)
    check_codes(nm.quantize(x.float()), x, False)


@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_values(dtype):
    big, tiny = torch.finfo(dtype).max, 2.0 ** -133 if dtype == BF16 else 2.0 ** -149
    x = torch.zeros(12, 300, dtype=dtype, device=DEV)
    x[1, 299] = big
    x[2, :] = torch.linspace(-1, 1, 300, device=DEV).to(dtype) * big
    x[3, 5] = tiny
    x[4, :] = tiny
    x[4, 1] = -2 * tiny
    x[5, :] = torch.linspace(-1, 1, 300, device=DEV).to(dtype) * 2.0 ** -120
    x[6, 7] = float("nan")
    x[6, 200] = 3.0
    x[7, 150] = float("inf")
    x[8, 299] = -float("inf")
    x[8, 0] = 1.0
    x[9, :] = 1.0
    x[9, 100] = 2.0 ** 60
    x[10, :] = -0.0
    x[11, :] = torch.linspace(-1, 1, 300, device=DEV).to(dtype) * 2.0 ** -101
    check_codes(nm.quantize(x), x, False)
    check_codes(nm.quantize(x, block=True), x, True)
    check_codes(nm.quantize(x.t().contiguous(), transpose=True), x, False)
    kept = nm.quantize(x, block=True)
    want = lo.decode(*lo.block_codes(to64(x)), True)
    for t in TYPES:
        assert np.array_equal(to64(kept.dequantize(t)), want, equal_nan=True)


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 130, 0), (17, 1031, 3), (300, 256, 8), (2, 8200, 1)])
def test_dequantize(rows, cols, pad, block, out):
    x = normal(rows, cols, F32, 3)
    c = nm.quantize(x, block=block)
    wide, y = out_in(rows, cols, out, pad)
    assert nm.dequantize(c, out=y) is y
    assert untouched(wide, rows, cols)
    want = lo.decode(to64(c.q[:, :cols]), to64(c.scale), block)
    if block:
        assert np.array_equal(to64(y), want)
    else:
        rel = U if out == F32 else (1 + U) * (1 + B) - 1
        assert (np.abs(to64(y) - want) <= np.abs(want) * rel).all()
    assert torch.equal(y, c.dequantize(out))


def check_product(y, a, b):
    """y against the 64-bit product of codes a and b (exact there: sums stay below 2^53)."""
    k = a.shape[1]
    sums = a.q[:, :k].double() @ b.q[:, :k].double().t()
    want = sums * a.scale.double()[:, None] * b.scale.double()[None, :]
    rel = (1 + U) ** 3 * (1 + (B if y.dtype == BF16 else 0.0)) - 1
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    bad = (y.double() - want).abs() > want.abs() * rel
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} results are off"


# (rows, columns of the result, summed columns): few rows with codes made inside and before, tiles
# of 128 and of 256 with ragged ends, odd and even numbers of k-steps, one k-step and none.
PRODUCTS = [(1, 1, 1), (1, 15, 128), (1, 257, 4096), (2, 100, 1031), (3, 33, 2000), (5, 1000, 300), (16, 64, 3000),
            (16, 517, 8200), (7, 40, 131071), (17, 1, 1), (17, 130, 127), (100, 200, 129), (128, 128, 384),
            (129, 127, 1024), (300, 700, 640), (4000, 3333, 200), (3800, 3601, 384), (20, 10, 131071), (40000, 3, 5)]


@pytest.mark.parametrize("rows,cols,k", PRODUCTS)
def test_products(rows, cols, k):
    log(f"product {rows}x{cols}x{k}")
    for dtype, out, pad in ((BF16, BF16, 0), (F32, F32, 5), (BF16, F32, 0), (F32, BF16, 8)):
        x = normal(rows, k, dtype, 5, pad, pad // 5)
        a, b = nm.quantize(x), nm.quantize(normal(cols, k, dtype, 6))
        wide, y = out_in(rows, cols, out, pad)
        nm.int8_matmul(a, b, out=y)
        assert untouched(wide, rows, cols)
        check_product(y, a, b)
        wide, z = out_in(rows, cols, out, pad)
        nm.int8_linear(x, b, out=z)
        assert untouched(wide, rows, cols)
        assert torch.equal(y, z)


def test_sums_reach_the_ends_of_32_bits():
    k = 131071
    a = nm.Codes(torch.full((2, k + 1), 127, dtype=torch.int8, device=DEV), torch.ones(2, device=DEV), k)
    a.q[1] = -127
    a.q[:, k:] = 0
    for rows in (2, 40):
        c = nm.Codes(a.q[:1].expand(rows, -1).contiguous(), torch.ones(rows, device=DEV), k)
        y = nm.int8_matmul(c, a, F32)
        want = torch.tensor([127.0 * 127.0 * k, -127.0 * 127.0 * k], dtype=torch.float64, device=DEV).float()
        assert torch.equal(y, want.expand(rows, 2))


@pytest.mark.parametrize("rows", [3, 40])
def test_lost_rows_and_channels_of_products(rows):
    x, w = normal(rows, 300, BF16, 1), normal(50, 300, BF16, 2)
    x[1, 7] = float("inf")
    x[2] = 0
    w[4, 9] = float("nan")
    w[5] = 0
    a, b = nm.quantize(x), nm.quantize(w)
    y = nm.int8_matmul(a, b)
    check_product(y, a, b)
    assert y[1].isnan().all() and y[:, 4].isnan().all() and int(y.isnan().sum()) == 50 + rows - 1
    assert (y[2, :4] == 0).all() and (y[0, 5] == 0).all()
    assert torch.equal(nm.int8_linear(x, b), y) or torch.equal(nm.int8_linear(x, b).nan_to_num(9.0), y.nan_to_num(9.0))


def whole(rows, cols, most, dtype, seed, pad=0, shift=0):
    wide = torch.full((rows, cols + pad + shift), float("nan"), device=DEV, dtype=dtype)
    x = wide[:, shift:shift + cols]
    return x.copy_(torch.randint(-most, most + 1, (rows, cols), device=DEV, generator=gen(seed)))


# (tokens, outputs, inputs): one token, tokens around the k-steps of 16 and 64, pieces of tokens,
# tiles of 128 and of 256 with ragged ends.
GRADS = [(1, 1, 1), (1, 8, 128), (15, 9, 3), (16, 130, 129), (63, 16, 257), (64, 128, 128), (65, 127, 130),
         (129, 300, 70), (1000, 64, 200), (1025, 264, 129), (20000, 8, 5), (4097, 130, 640), (130, 4000, 3500),
         (64, 3801, 3600), (300, 3592, 3600)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,outputs,inputs", GRADS)
def test_weight_grads_of_whole_numbers(tokens, outputs, inputs, dtype):
    """Exact: |dy| <= 7 and |x| <= 7, so sums stay below 49 * 20000 < 2^20."""
    log(f"weight grad {tokens}x{outputs}x{inputs} {dtype}")
    for pad, shift in ((0, 0), (9, 3)):
        dy = whole(tokens, outputs, 7, dtype, 1, pad, shift)
        x = whole(tokens, inputs, 7, BF16, 2)
        kept = nm.quantize(x, block=True)
        want = dy.double().t().contiguous() @ x.double()
        wide, dw = out_in(outputs, inputs, F32, pad)
        nm.weight_grad(dy, kept, out=dw)
        assert untouched(wide, outputs, inputs)
        assert torch.equal(dw.double(), want)
        nm.weight_grad(dy, kept, out=dw, accumulate=True)
        assert untouched(wide, outputs, inputs)
        assert torch.equal(dw.double(), 2 * want)
    wide, dw = out_in(outputs, inputs, BF16, 1, 3.0)
    nm.weight_grad(dy, kept, out=dw, accumulate=True)
    assert untouched(wide, outputs, inputs, 3.0)
    assert torch.equal(dw, (want + 3.0).to(BF16))
    assert torch.equal(nm.weight_grad(dy, kept, BF16), want.to(BF16))


@pytest.mark.parametrize("outputs,inputs,shift", [(1024, 2048, 0), (1021, 2048, 1), (3592, 3600, 0)])
def test_weight_grads_of_any_number_of_steps(outputs, inputs, shift):
    """1 to 13 steps of 64 tokens: rounds of six and every rest, in each kind of tile.  Exact."""
    for steps in range(1, 14):
        log(f"weight grad {steps} steps of {outputs}x{inputs}")
        tokens = 64 * steps - 3 * (steps % 2)
        dy, x = whole(tokens, outputs, 7, BF16, steps, 0, shift), whole(tokens, inputs, 7, BF16, 20 + steps)
        want = dy.float().t().contiguous() @ x.float()  # below 49 * 832: exact
        assert torch.equal(nm.weight_grad(dy, nm.quantize(x, block=True)), want)


@pytest.mark.parametrize("rows,cols", [(130, 200), (2048, 4096), (4096, 4096)])
def test_products_of_any_number_of_steps(rows, cols):
    """2 to 14 steps of 64 columns: rounds of five and every rest, in each tile.  With 127 in each row the
    codes are the values, and sums stay below 127^2 + 49 * 896 < 2^24: exact."""
    for k in range(128, 128 * 8, 128):
        log(f"int8 product {rows}x{cols}x{k}")
        a, b = whole(rows, k, 7, BF16, k), whole(cols, k, 7, BF16, k + 1)
        a[:, 0] = b[:, 0] = 127
        got = nm.int8_matmul(nm.quantize(a), nm.quantize(b), F32)
        assert torch.equal(got, a.float() @ b.float().t().contiguous())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,outputs,inputs", [(1, 5, 300), (100, 64, 257), (1500, 136, 384), (640, 3640, 3520)])
def test_weight_grads(tokens, outputs, inputs, dtype):
    dy = normal(tokens, outputs, dtype, 1)
    kept = nm.quantize(normal(tokens, inputs, dtype, 2), block=True)
    x = kept.dequantize(F32).double()
    want, size = dy.double().t().contiguous() @ x, dy.double().abs().t().contiguous() @ x.abs()
    sums = 2 * U * (tokens + (1 if dtype == F32 else 0)) * size
    assert ((nm.weight_grad(dy, kept).double() - want).abs() <= sums).all()
    for out in TYPES:
        old = normal(outputs, inputs, out, 3)
        dw = old.clone()
        nm.weight_grad(dy, kept, out=dw, accumulate=True)
        total = old.double() + want
        bound = (sums + total.abs() * U) * (1 + U)
        if out == BF16:
            bound = bound * (1 + B) + total.abs() * B
        assert ((dw.double() - total).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [5, 64, 70, 1030])
def test_weight_grads_with_infinities(tokens, dtype):
    """An infinity or a NaN reaches its own row (dy) or block of columns (x) of dw, and no other;
    tokens behind the last one add nothing to it."""
    dy, x = whole(tokens, 40, 3, dtype, 1), whole(tokens, 300, 3, BF16, 2)
    x[tokens - 1, :5] = 2
    dy[tokens - 1, 3] = float("inf")
    dy[0, 7] = float("nan")
    x[2, 130] = float("inf")
    x[:, 290] = 0
    kept = nm.quantize(x, block=True)
    dw = nm.weight_grad(dy, kept)
    decoded = kept.dequantize(F32)
    assert decoded[2, 128:256].isnan().all() and int(decoded.isnan().sum()) == 128
    want = torch.from_numpy(to64(dy).T @ to64(decoded)).to(DEV)
    assert torch.equal(dw.isnan(), want.isnan()) and torch.equal(dw.isinf(), want.isinf())
    fine = want.isfinite()
    assert torch.equal(dw[fine].double(), want[fine])
    assert torch.isinf(dw[3, :5]).all() and not dw[[0, 1, 2] + list(range(8, 40))][:, :128].isnan().any()


@pytest.mark.parametrize("tokens,outputs,inputs", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0)])
def test_no_elements(tokens, outputs, inputs):
    x, dy = torch.zeros(tokens, inputs, device=DEV), torch.ones(tokens, outputs, device=DEV)
    w = torch.ones(outputs, inputs, device=DEV)
    assert nm.quantize(w, transpose=True).shape == (inputs, outputs)
    wq, kept = nm.quantize(w), nm.quantize(x, block=True)
    assert kept.dequantize().shape == (tokens, inputs)
    for y in (nm.int8_linear(x, wq), nm.int8_matmul(nm.quantize(x), wq, F32),
              nm.int8_linear(torch.zeros(tokens * 9, inputs, device=DEV), wq)):
        assert y.shape[1] == outputs and not y.any()
    for d in (dy, dy.to(BF16)):
        dw = torch.full((outputs, inputs), 3.0, device=DEV)
        nm.weight_grad(d, kept, out=dw, accumulate=True)
        assert (dw == 3.0).all()  # no token: nothing is added
        if tokens == 0:
            nm.weight_grad(d, kept, out=dw)
            assert not dw.any()


def layer_pass(x, w, dy, grad, stream=None):
    """Forward and backward of one layer; grad is added to."""
    kept = nm.quantize(x, block=True, stream=stream)
    y = nm.int8_linear(x, nm.quantize(w, stream=stream), stream=stream)
    dx = nm.int8_linear(dy, nm.quantize(w, transpose=True, stream=stream), stream=stream)
    nm.weight_grad(dy, kept, out=grad, accumulate=True, stream=stream)
    return y, dx


def test_a_training_step():
    """Two micro-batches through a layer, the gradients' norm, clipping and a Muon step."""
    tokens, outputs, inputs = 200, 136, 264
    w = (torch.randn(outputs, inputs, device=DEV, generator=gen(1)) * 0.05).to(F32)
    grad = torch.zeros(outputs, inputs, device=DEV)
    want = np.zeros((outputs, inputs))
    size = np.zeros((outputs, inputs))
    for batch in range(2):
        x, dy = normal(tokens, inputs, BF16, 10 + batch), normal(tokens, outputs, BF16, 20 + batch)
        y, dx = layer_pass(x, w, dy, grad)
        wq = lo.row_codes(to64(w))
        y64 = lo.product(lo.row_codes(to64(x)), wq)
        dx64 = lo.product(lo.row_codes(to64(dy)), lo.row_codes(to64(w).T))
        # The scales are rounded too: 5 U, and the result to bf16.
        rel = (1 + U) ** 5 * (1 + B) * (1 + 1e-6) - 1
        assert (np.abs(to64(y) - y64) <= np.abs(y64) * rel).all()
        assert (np.abs(to64(dx) - dx64) <= np.abs(dx64) * rel).all()
        dw, mag = lo.weight_grad(to64(dy), *lo.block_codes(to64(x)))
        want += dw
        size += mag
    bound = 2 * U * (2 * tokens + 2) * size
    assert (np.abs(to64(grad) - want) <= bound).all()
    clip = nm.GradClip([grad])
    norm = clip.norm()
    assert abs(float(norm) - grad_norm([to64(grad)])) <= U * float(norm) * (1 + 1e-6)
    before, moment = w.clone(), torch.zeros_like(w)
    nm.MuonStep([w], [grad], [moment], lr=0.02)(clip=(norm, 1.0))
    scale = 1.0 / (grad_norm([to64(grad)]) + 1e-6)
    # M = c G, with c as the clip's own test has it (4 roundings) and its product with G.
    assert (np.abs(to64(moment) - scale * to64(grad)) <= 6 * U * np.abs(scale * to64(grad)) + 2.0 ** -149).all()
    assert torch.isfinite(w).all() and not torch.equal(w, before)


def test_input_gradient_is_the_difference_quotient():
    """y = xq wq^T is linear in xq: differences of sum(dy * y) are dx, with the same codes of w."""
    w, dy = normal(40, 130, F32, 1), normal(6, 40, F32, 2)
    wt, gq = nm.quantize(w, transpose=True), nm.quantize(dy)
    dx = to64(nm.int8_matmul(gq, wt, F32))
    values, g = to64(wt.dequantize(F32)).T, to64(gq.dequantize(F32))  # outputs x inputs, tokens x outputs
    loss = lambda x: float((g * (x @ values.T)).sum())  # noqa: E731
    x = np.random.default_rng(3).standard_normal((6, 130))
    for i, j in ((0, 0), (5, 129), (3, 64)):
        e = np.zeros_like(x)
        e[i, j] = 1.0
        terms = float(np.abs(g[i]) @ np.abs(values[:, j]))
        # Codes and scales give values of one rounding each (2 U a term); the quotient's own error is
        # that of a 64-bit sum of the whole loss.
        noise = 1e-13 * float((np.abs(g) * (np.abs(x) @ np.abs(values).T)).sum())
        assert abs((loss(x + e) - loss(x - e)) / 2 - dx[i, j]) <= 6 * U * terms + noise


def test_results_do_not_change_from_run_to_run():
    x, w, dy = normal(1500, 264, BF16, 1), normal(136, 264, BF16, 2), normal(1500, 136, BF16, 3)
    runs = []
    for _ in range(3):
        grad = torch.zeros(136, 264, device=DEV)
        runs.append((*layer_pass(x, w, dy, grad), grad))
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))


@pytest.mark.parametrize("handle", [False, True])
def test_named_streams(handle):
    """Calls on a stream that is named, whose operands and results are dropped right after."""
    want, got = [], []
    side = torch.cuda.Stream()
    for i in range(6):
        x, w, dy = normal(900, 264, BF16, i), normal(135, 264, BF16, 9), normal(900, 135, BF16, 30 + i)
        grad = torch.zeros(135, 264, device=DEV)
        want.append((*layer_pass(x, w, dy, grad), grad))
        torch.cuda.synchronize()
        grad = torch.zeros(135, 264, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        got.append((*layer_pass(x, w, dy, grad, stream=side.cuda_stream if handle else side), grad))
        del x, w, dy, grad
        torch.full((900, 264), float("nan"), device=DEV, dtype=BF16)  # takes what was given back
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(p, q))


def test_graphs():
    """Two graphs of the same calls, replayed in turn on new values, with eager work between."""
    sizes = (700, 135, 264)
    graphs = []
    for g in range(2):
        x, w, dy = normal(sizes[0], sizes[2], BF16, 1), normal(sizes[1], sizes[2], BF16, 2), normal(sizes[0], sizes[1], BF16, 3)
        grad = torch.zeros(sizes[1], sizes[2], device=DEV)
        layer_pass(x, w, dy, grad)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer_pass(x, w, dy, grad)
            few = nm.int8_linear(x[:3], nm.quantize(w))
        graphs.append((graph, x, w, dy, grad, out, few))
    for turn in range(3):
        for k, (graph, x, w, dy, grad, out, few) in enumerate(graphs):
            x.copy_(normal(*x.shape, BF16, 40 + 2 * turn + k))
            dy.copy_(normal(*dy.shape, BF16, 60 + 2 * turn + k))
            grad.fill_(1.0)
            graph.replay()
            other = torch.ones_like(grad)
            want = layer_pass(x, w, dy, other)
            torch.cuda.synchronize()
            assert torch.equal(grad, other) and all(torch.equal(p, q) for p, q in zip(out, want))
            assert torch.equal(few, nm.int8_linear(x[:3], nm.quantize(w)))


def test_a_graph_of_named_streams():
    """A captured layer whose calls name their streams, the weight gradient's one that joins in the
    capture; replayed on new values, with eager calls between."""
    x, w, dy = normal(700, 264, BF16, 1), normal(135, 264, BF16, 2), normal(700, 135, BF16, 3)
    grad = torch.zeros(135, 264, device=DEV)
    layer_pass(x, w, dy, grad)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        kept = nm.quantize(x, block=True, stream=main)
        side.wait_stream(main)
        nm.weight_grad(dy, kept, out=grad, accumulate=True, stream=side)
        y = nm.int8_linear(x, nm.quantize(w, stream=main), stream=main)
        dx = nm.int8_linear(dy, nm.quantize(w, transpose=True, stream=main), stream=main)
        main.wait_stream(side)
    for turn in range(4):
        x.copy_(normal(*x.shape, BF16, 40 + turn))
        dy.copy_(normal(*dy.shape, BF16, 60 + turn))
        grad.fill_(1.0)
        graph.replay()
        other = torch.ones_like(grad)
        want = layer_pass(x, w, dy, other)
        torch.cuda.synchronize()
        assert torch.equal(grad, other) and torch.equal(y, want[0]) and torch.equal(dx, want[1])


def test_calls_of_several_threads():
    """Threads with a stream each: the same results as one after another."""
    import threading

    data = [(normal(300 + 7 * i, 264, BF16, i), normal(135, 264, BF16, 9), normal(300 + 7 * i, 135, BF16, 30 + i)) for i in range(4)]
    want = []
    for x, w, dy in data:
        grad = torch.zeros(135, 264, device=DEV)
        want.append((*layer_pass(x, w, dy, grad), grad))
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            x, w, dy = data[i]
            for _ in range(20):
                grad = torch.zeros(135, 264, device=DEV)
                got[i] = (*layer_pass(x, w, dy, grad), grad)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for p, q in zip(want, got):
        assert q is not None and all(torch.equal(a, b) for a, b in zip(p, q))


def test_codes_are_written_in_place():
    x = normal(50, 300, BF16, 1)
    for block in (False, True):
        c = nm.Codes.empty(50, 300, block=block, device=DEV)
        at = c.q.data_ptr()
        assert nm.quantize(x, block=block, out=c) is c and c.q.data_ptr() == at
        check_codes(c, x, block)
    with pytest.raises(ValueError):
        nm.quantize(x, out=nm.Codes.empty(50, 299, device=DEV))
    with pytest.raises(ValueError):
        nm.quantize(x, out=c)  # codes by block
    with pytest.raises(ValueError):
        nm.quantize(x, block=True, transpose=True)


def test_refused_calls_on_the_gpu_leave_the_output():
    x, w = normal(4, 300, BF16, 1), nm.quantize(normal(8, 300, BF16, 2))
    y = torch.full((4, 8), 5.0, device=DEV, dtype=BF16)
    kept = nm.quantize(x, block=True)
    for call in (lambda: nm.int8_linear(x[:, :299], w, out=y), lambda: nm.int8_matmul(kept, w, out=y),
                 lambda: nm.int8_linear(x, w, F32, out=y), lambda: nm.int8_linear(x, w, out=y.t()),
                 lambda: nm.weight_grad(y, w, accumulate=True), lambda: nm.weight_grad(y[:3], kept),
                 lambda: nm.int8_linear(x, w, out=y.expand(4, 8)[:, :7]), lambda: nm.int8_linear(x.half(), w, out=y),
                 lambda: nm.int8_linear(x.cpu(), w, out=y), lambda: nm.dequantize(kept, out=x[:, :299]),
                 lambda: nm.weight_grad(torch.ones(1, 1, device=DEV).expand(4, 8), kept)):
        with pytest.raises((ValueError, TypeError, nm.MuonError)):
            call()
    assert (y == 5.0).all()


def test_profile_names_the_launches():
    x, w = normal(100, 300, BF16, 1), normal(80, 300, BF16, 2)
    nm.profile_begin()
    nm.weight_grad(normal(100, 80, BF16, 3), nm.quantize(x, block=True))
    nm.int8_linear(x, nm.quantize(w))
    nm.int8_linear(x[:2], nm.quantize(w))
    nm.quantize(w, transpose=True)
    nm.quantize(x).dequantize()
    stats = nm.profile_end()
    for name in ("quantize_rows", "quantize_blocks", "quantize_columns", "dequantize", "int8_product", "int8_few", "weight_grad"):
        assert stats[name]["launches"] >= 1


def test_more_than_2_31_elements():
    """The last rows of operands and results behind 2^31 elements are those of a call on them alone."""
    rows, cols = 70003, 32776
    x = torch.empty(rows, cols, device=DEV, dtype=BF16).normal_(generator=gen(1))
    tail = x[-200:]
    c, kept = nm.quantize(x), nm.quantize(x, block=True)
    for got, block in ((c, False), (kept, True)):
        part = nm.quantize(tail, block=block)
        assert torch.equal(got.q[-200:], part.q) and torch.equal(got.scale[-200:], part.scale)
        del part
    w = nm.quantize(normal(40, cols, BF16, 2))
    assert torch.equal(nm.int8_matmul(c, w)[-200:], nm.int8_matmul(nm.quantize(tail), w))
    few = nm.quantize(normal(3, cols, BF16, 3))
    assert torch.equal(nm.int8_matmul(few, c)[:, -200:], nm.int8_matmul(few, nm.quantize(tail)))
    # Only the last 200 tokens' dy is not zero; whole numbers, so that sums are exact in any order.
    x[-200:] = whole(200, cols, 7, BF16, 4)
    kept = nm.quantize(x, block=True)
    values = kept.dequantize()
    assert torch.equal(values[-200:], tail)
    dy = torch.zeros(rows, 24, device=DEV, dtype=BF16)
    dy[-200:] = whole(200, 24, 7, BF16, 5)
    want = nm.weight_grad(dy[-200:], nm.quantize(tail, block=True))
    assert torch.equal(nm.weight_grad(dy, kept), want)
    assert torch.equal(nm.weight_grad(dy.float(), kept), want)


def test_results_behind_2_31_elements():
    a, b = nm.quantize(normal(70001, 130, BF16, 1)), nm.quantize(normal(32771, 130, BF16, 2))
    y = nm.int8_matmul(a, b)
    assert torch.equal(y[-130:], nm.int8_matmul(nm.quantize(normal(70001, 130, BF16, 1)[-130:]), b))
    del y, a, b
    dy, x = whole(66, 70008, 3, BF16, 1), whole(66, 32771, 3, BF16, 2)
    kept = nm.quantize(x, block=True)
    dw = nm.weight_grad(dy, kept, BF16)
    assert torch.equal(dw[-9:], (dy[:, -9:].double().t().contiguous() @ x.double()).to(BF16))
    del dw
    t = nm.quantize(whole(40000, 54001, 7, BF16, 3), transpose=True)
    assert torch.equal(t.q[-70:, :40000].t(), nm.quantize(whole(40000, 54001, 7, BF16, 3)[:, -70:], transpose=True).q[:, :40000].t())


def same_codes(c, part, lo, hi):
    return torch.equal(c.q[lo:hi], part.q) and torch.equal(c.scale[lo:hi], part.scale)


@pytest.mark.parametrize("cols", [1, 2049])
def test_more_rows_than_workgroups(cols):
    """A launch of codes by row has at most 2^20 workgroups, of four rows (a wave each) or one; longer
    operands go round three times here.  A part of one round at a time gives the same."""
    turn = (4 if cols == 1 else 1) << 20
    rows = 2 * turn + 19
    x = torch.empty(rows, cols, device=DEV, dtype=BF16).normal_(generator=gen(1))
    c = nm.quantize(x)
    for at in range(0, rows, turn):
        hi = min(rows, at + turn)
        log(f"rows {at} to {hi} of {cols}")
        assert same_codes(c, nm.quantize(x[at:hi]), at, hi)
    check_codes(nm.quantize(x[-100:]), x[-100:], False)


def test_more_blocks_than_workgroups():
    """The same of codes by block (2^30 runs of 8 values in 2^20 workgroups) and of reading them."""
    rows, turn = (1 << 26) + 100, 1 << 25
    x = torch.empty(rows, 128, device=DEV, dtype=BF16).normal_(generator=gen(1))
    c = nm.quantize(x, block=True)
    values = c.dequantize(BF16)
    for at in range(0, rows, turn):
        hi = min(rows, at + turn)
        log(f"rows {at} to {hi}")
        part = nm.quantize(x[at:hi], block=True)
        assert same_codes(c, part, at, hi)
        assert torch.equal(values[at:hi], part.dequantize(BF16))
        del part
    check_codes(nm.quantize(x[-100:], block=True), x[-100:], True)


def test_more_unaligned_rows_than_workgroups():
    """Rows of dy that are copied to aligned ones first, 2^28 runs of 8 values in a round."""
    tokens, outputs = (1 << 24) + 50, 121
    dy = torch.zeros(tokens, outputs, device=DEV, dtype=BF16)
    x = torch.zeros(tokens, 3, device=DEV, dtype=BF16)
    ends = torch.cat([torch.arange(60), torch.arange(tokens - 110, tokens)]).to(DEV)
    dy[ends], x[ends] = whole(170, outputs, 7, BF16, 1), whole(170, 3, 7, BF16, 2)
    x[60:-110] = 5.0
    want = dy[ends].double().t().contiguous() @ x[ends].double()
    assert torch.equal(nm.weight_grad(dy, nm.quantize(x, block=True)).double(), want)


class Layer(torch.autograd.Function):
    """A linear layer as a user of autograd has it: y = x W^T, in 8 bits both ways."""

    @staticmethod
    def forward(ctx, x, w):
        ctx.kept = nm.quantize(x, block=True)
        ctx.save_for_backward(w)
        return nm.int8_linear(x, nm.quantize(w))

    @staticmethod
    def backward(ctx, dy):
        (w,) = ctx.saved_tensors
        return nm.int8_linear(dy, nm.quantize(w, transpose=True)), nm.weight_grad(dy, ctx.kept, BF16)


def test_a_layer_for_autograd():
    x, w, dy = normal(200, 264, BF16, 1), normal(136, 264, BF16, 2), normal(200, 136, BF16, 3)
    want = nm.int8_linear(x, nm.quantize(w))
    dx = nm.int8_linear(dy, nm.quantize(w, transpose=True))
    dw = nm.weight_grad(dy, nm.quantize(x, block=True), BF16)
    x, w = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = Layer.apply(x, w)
    y.backward(dy)
    assert torch.equal(y, want) and torch.equal(x.grad, dx) and torch.equal(w.grad, dw)


def test_operands_that_need_a_gradient_are_refused():
    x, w = normal(4, 300, F32, 1), nm.quantize(normal(8, 300, F32, 2))
    leaf, y = x.clone().requires_grad_(), torch.full((4, 8), 5.0, device=DEV)
    kept, learned = nm.quantize(x, block=True), nm.quantize(normal(8, 300, F32, 2))
    learned.scale.requires_grad_()
    for call in (lambda: nm.int8_linear(leaf, w, out=y), lambda: nm.int8_linear(x, learned, out=y), lambda: learned.dequantize(),
                 lambda: nm.int8_matmul(nm.quantize(x), learned, out=y), lambda: nm.quantize(leaf * 2),
                 lambda: nm.weight_grad(leaf[:, :5], kept)):
        with pytest.raises(ValueError, match="needs a gradient"):
            call()
    assert (y == 5.0).all()
    with torch.no_grad():
        assert torch.equal(nm.int8_linear(leaf, learned), nm.int8_linear(x, w))
