"""GPU: the global gradient norm, clipping and AdamW over lists against float64.

Tolerances.  u = 2^-24 is half a step of fp32.
  norm   its squares and sum are 64-bit, the result is rounded to fp32 once: u relative (or half
         the smallest denormal), plus the sum's own error, far below it.
  clip   the norm's rounding, 1e-6 as fp32, their sum, the quotient and the product with g are
         one rounding each: 5 u relative; a bf16 result is rounded once more, 2^-8 at most (or
         half its smallest denormal, 2^-134; fp32: 2^-150).
  AdamW  the bounds of the packed fp32 step (tests/test_gpu_parity.py), whose 4 * 2^-22 on each
         use of g also covers the 5 u of the clip coefficient and product; a bf16 param adds
         one rounding of the result, 2^-8 relative at most."""

from __future__ import annotations

import types

import numpy as np
import pytest
import torch

import newton_schulz_02_amd as nm
from oracle import adamw_step as oracle_adamw
from oracle.grad_oracle import clip_coef, clip_grads, grad_norm
from tests.gpu_helpers import DEV, log, to64
from tests.test_gpu_parity import adamw_bounds

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def norm_close(got: torch.Tensor, want: float) -> bool:
    got = float(got)
    return abs(got - want) <= U * want * (1 + 1e-6) + 2.0 ** -150


def clip_bound(want: np.ndarray, dtype) -> np.ndarray:
    rel, tiny = (2.0 ** -8, 2.0 ** -134) if dtype == BF16 else (0.0, 2.0 ** -150)
    return np.abs(want) * (rel + 5 * U) * (1 + 1e-6) + tiny + 2.0 ** -150


# Lists as (numel, dtype); every tensor lies in a buffer of its own, `shift` elements behind a
# 256-byte boundary, with guards around it.
LISTS = {
    "empty": [],
    "no elements": [(0, BF16), (0, F32)],
    "one": [(1, F32)],
    "ones": [(1, BF16)] * 130,
    "tails": [(n, t) for n in (1, 7, 8, 9, 255, 257, 2047, 2049, 4095, 4097, 8191, 8193) for t in (BF16, F32)],
    "with empties": [(0, F32), (5000, BF16), (0, BF16), (0, BF16), (3, F32), (0, F32)],
    "layer vectors": [(4096, F32)] * 65,
    "many": [(1 + 37 * i % 5003, BF16 if i % 3 else F32) for i in range(700)],
    "long": [(20_000_003, BF16), (11, F32)],
    "long fp32": [(9_500_001, F32), (1, BF16), (64, F32)],
}


def make(spec, seed, shift=0, std=1e-2):
    """(views, guarded buffers): the views' values are normal, the guards NaN."""
    gen = torch.Generator(DEV).manual_seed(seed)
    views, bufs = [], []
    for i, (n, t) in enumerate(spec):
        off = 128 + (shift + i if shift else 0)
        buf = torch.full((off + n + 128,), float("nan"), device=DEV, dtype=t)
        view = buf[off:off + n]
        view.copy_(torch.randn(n, device=DEV, generator=gen) * std)
        views.append(view)
        bufs.append((buf, off, n))
    return views, bufs


def guards_whole(bufs) -> bool:
    return all(bool(torch.isnan(b[:o]).all()) and bool(torch.isnan(b[o + n:]).all()) for b, o, n in bufs)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("name", list(LISTS))
def test_norm(name, shift):
    log(f"norm {name} shift {shift}")
    views, bufs = make(LISTS[name], 3, shift)
    host = [to64(v) for v in views]
    lst = nm.GradClip(views, device=DEV)
    for kind in ("l2", "inf"):
        want = grad_norm(host, kind)
        first, second = lst.norm(kind), lst.norm(kind)
        log(f"  {kind}: {float(first)!r} want {want!r}")
        assert norm_close(first, want) if kind == "l2" else float(first) == want
        assert torch.equal(first, second)
        assert torch.equal(nm.grad_norm(views, kind, device=DEV), first)
    assert guards_whole(bufs)
    assert all(np.array_equal(to64(v), h) for v, h in zip(views, host))


@pytest.mark.parametrize("std", [1e-25, 1e-41, 3e18, 1e30])
def test_norm_of_values_whose_squares_leave_fp32(std):
    log(f"norm std {std}")
    views, _ = make([(5000, F32), (777, BF16)], 5, std=std)
    want = grad_norm([to64(v) for v in views])
    got = nm.GradClip(views).norm()
    log(f"  {float(got)!r} want {want!r}")
    assert want > 0 and norm_close(got, want)


def test_norm_above_fp32_is_infinite():
    log("norm above fp32")
    views = [torch.full((100,), 3e38, device=DEV)]
    lst = nm.GradClip(views)
    assert torch.isinf(lst.norm()) and float(lst.norm("inf")) == float(np.float32(3e38))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad,at", [("nan", 0), ("nan", 9998), ("inf", 5000), ("-inf", 9999), ("both", 17)])
def test_norm_and_clip_of_infinities_and_nan(bad, at, dtype):
    log(f"norm of {bad} at {at} {dtype}")
    views, bufs = make([(100, F32), (10000, dtype), (33, BF16)], 6)
    views[1][at] = float("nan" if bad in ("nan", "both") else bad)
    if bad == "both":
        views[2][5] = float("inf")
    for kind in ("l2", "inf"):
        got = nm.GradClip(views).norm(kind)
        assert torch.isnan(got) if bad in ("nan", "both") else float(got) == float("inf")
    host = [to64(v) for v in views]
    norm = nm.GradClip(views).clip_norm(1.0)
    want = clip_grads(host, float(norm), 1.0)  # all NaN, or 0 and NaN at the infinity
    for v, w in zip(views, want):
        np.testing.assert_array_equal(to64(v), w)
    assert guards_whole(bufs)


@pytest.mark.parametrize("kind,max_norm", [("l2", 1.0), ("inf", 1e-3), ("l2", 0.0), ("l2", 1e-30)])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("name", list(LISTS))
def test_clip(name, shift, kind, max_norm):
    log(f"clip {name} shift {shift} {kind} {max_norm}")
    views, bufs = make(LISTS[name], 4, shift, std=1.0)
    host = [to64(v) for v in views]
    want = grad_norm(host, kind)
    lst = nm.GradClip(views, device=DEV)
    norm = lst.clip_norm(max_norm, kind)
    assert norm_close(norm, want)
    for v, w in zip(views, clip_grads(host, want, max_norm)):
        assert np.all(np.abs(to64(v) - w) <= clip_bound(w, v.dtype))
    assert guards_whole(bufs)


def test_clip_by_a_norm_in_hand_and_one_shot_forms():
    log("clip by a norm in hand")
    spec = LISTS["many"]
    views, bufs = make(spec, 8, 1)
    host = [to64(v) for v in views]
    norm = torch.tensor([7.5], device=DEV)
    nm.GradClip(views).clip(norm, 2.0)
    for v, w in zip(views, clip_grads(host, 7.5, 2.0)):
        assert np.all(np.abs(to64(v) - w) <= clip_bound(w, v.dtype))
    again, _ = make(spec, 8, 1)
    nm.grad_clip(again, norm, 2.0)
    assert all(torch.equal(a, b) for a, b in zip(views, again))
    both, _ = make(spec, 8, 1)
    alone, _ = make(spec, 8, 1)
    n = nm.clip_grad_norm(both, 0.1)
    nm.grad_clip(alone, n, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(both, alone))
    assert guards_whole(bufs)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_clip_into_denormals(dtype):
    """Products below the normal range keep the type's denormals (c itself is normal)."""
    log(f"clip into denormals {dtype}")
    views, bufs = make([(5001, dtype), (40000, dtype)], 12, 1, std=1e-30)
    host = [to64(v) for v in views]
    nm.GradClip(views).clip(torch.tensor(1e10, device=DEV), 1.0)
    for v, w in zip(views, clip_grads(host, 1e10, 1.0)):
        assert np.all(np.abs(to64(v) - w) <= clip_bound(w, v.dtype))
        assert 0 < np.abs(to64(v)).max() < 2.0 ** -126
    assert guards_whole(bufs)


def test_a_norm_below_the_limit_leaves_every_bit():
    log("clip below the limit")
    views, _ = make(LISTS["many"], 9)
    views[3][0] = -0.0
    before = [v.clone() for v in views]
    norm = nm.GradClip(views).clip_norm(1e6)
    assert 0 < float(norm) < 1e6
    assert all(torch.equal(v.view(torch.int16 if v.dtype == BF16 else torch.int32),
                           b.view(torch.int16 if b.dtype == BF16 else torch.int32)) for v, b in zip(views, before))


def test_offsets_past_32_bits():
    """A tensor of more than 2^32 bytes and 2^31 elements: the norm counts all of it, clipping
    reaches its end."""
    n = (1 << 31) + 4099
    log(f"norm and clip of {n} bf16 elements")
    g = torch.full((n,), 0.5, device=DEV, dtype=BF16)
    lst = nm.GradClip([g])
    norm = lst.norm()
    assert norm_close(norm, 0.5 * np.sqrt(float(n)))
    lst.clip(torch.tensor(8.0, device=DEV), 4.0)  # c = 4 / (8 + 1e-6): 0.25 after the bf16 rounding
    assert bool((g[-5000:] == 0.25).all()) and bool((g[:5000] == 0.25).all())
    assert int((g == 0.25).sum(dtype=torch.int64)) == n


# --- AdamW ----------------------------------------------------------------------------------

KINDS = {"f32/f32": (F32, F32, False), "f32/bf16": (F32, BF16, False), "bf16/bf16": (BF16, BF16, False),
         "bf16/f32": (BF16, F32, False), "master/bf16": (BF16, BF16, True), "master/f32": (BF16, F32, True)}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


class Adam:
    """A list of parameters with its state, each buffer guarded; kinds: one per tensor.  apart:
    the buffers of one tensor lie differently towards the 16 bytes of an access."""

    def __init__(self, sizes, kinds, seed, shift=0, first=False, apart=False):
        self.kinds = [KINDS[k] for k in kinds]
        self.bufs = []

        def part(dtypes, at, std):
            views, bufs = make(list(zip(sizes, dtypes)), at, shift + 3 * (at - seed) if apart else shift, std)
            self.bufs += bufs
            return views

        n = len(sizes)
        self.p = part([k[0] for k in self.kinds], seed, 0.5)
        self.g = part([k[1] for k in self.kinds], seed + 1, 1e-2)
        self.m = part([F32] * n, seed + 2, 0.0 if first else 1e-2)
        self.v = part([F32] * n, seed + 3, 0.0 if first else 1e-2)
        self.w = part([F32] * n, seed + 4, 0.0)
        for v in self.v:
            v.square_()
        for p, w in zip(self.p, self.w):
            w.copy_(p.float() * (1 + 2.0 ** -10))  # a master between two bf16 values
        self.masters = [w if k[2] else None for w, k in zip(self.w, self.kinds)]
        self.decays = [1.0 if i % 3 else 0.0 for i in range(n)]
        self.host = [[to64(t) for t in (p, g, m, v, w)] for p, g, m, v, w in zip(self.p, self.g, self.m, self.v, self.w)]

    def step(self, **kw):
        return nm.AdamWStep(self.p, self.g, self.m, self.v, masters=self.masters, decays=self.decays, **HP, **kw)

    def check(self, step, coef=1.0):
        for i, ((p0, g0, m0, v0, w0), (pt, _, master), d) in enumerate(zip(self.host, self.kinds, self.decays)):
            if p0.size == 0:
                continue
            at = w0 if master else p0
            hp = types.SimpleNamespace(**{**HP, "weight_decay": HP["weight_decay"] * d})
            want, m1, v1 = oracle_adamw(at, coef * g0, m0, v0, t=step, lr=hp.lr, beta1=hp.beta1, beta2=hp.beta2,
                                        eps=hp.eps, weight_decay=hp.weight_decay)
            bp, bm, bv = adamw_bounds(at, coef * g0, m0, v0, step, hp)
            assert np.all(np.abs(to64(self.m[i]) - m1) <= bm), f"m of tensor {i}"
            assert np.all(np.abs(to64(self.v[i]) - v1) <= bv), f"v of tensor {i}"
            if master:
                assert np.all(np.abs(to64(self.w[i]) - want) <= bp), f"master of tensor {i}"
                # The param is its master, rounded once.
                assert torch.equal(self.p[i], self.w[i].to(pt)), f"param of tensor {i}"
            else:
                if pt == BF16:
                    bp = bp + 2.0 ** -8 * (np.abs(want) + bp)
                assert np.all(np.abs(to64(self.p[i]) - want) <= bp), f"param of tensor {i}"
                np.testing.assert_array_equal(to64(self.w[i]), w0)
            np.testing.assert_array_equal(to64(self.g[i]), g0)
        assert guards_whole(self.bufs)


SIZES = {
    "tails": [1, 3, 4, 5, 0, 1023, 1025, 2047, 2048, 2049, 4099],
    "vectors": [4096] * 9,
    "long": [3_000_001, 17],
}


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("kind", list(KINDS))
def test_adamw_list(kind, sizes, shift):
    log(f"adamw {kind} {sizes} shift {shift}")
    a = Adam(SIZES[sizes], [kind] * len(SIZES[sizes]), 11, shift)
    a.step()(7)
    a.check(7)


@pytest.mark.parametrize("kind", list(KINDS))
def test_adamw_buffers_that_lie_differently(kind):
    log(f"adamw {kind}, buffers apart")
    a = Adam([5, 2048, 4099, 6143, 100_000], [kind] * 5, 17, 1, apart=True)
    a.step()(2)
    a.check(2)


def test_adamw_offsets_past_32_bits():
    """More than 2^31 elements, and more chunks than workgroups: every element is updated, once."""
    n = (1 << 31) + 4099
    log(f"adamw of {n} elements")
    p = torch.full((n,), 1.0, device=DEV, dtype=BF16)
    g = torch.full((n,), 0.5, device=DEV, dtype=BF16)
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    small = [torch.full((5,), x, device=DEV, dtype=t) for x, t in ((1.0, BF16), (0.5, BF16), (0.0, F32), (0.0, F32))]
    for buf in ((p, g, m, v), small):
        nm.AdamWStep([buf[0]], [buf[1]], [buf[2]], [buf[3]], lr=0.25, weight_decay=0.0)(1)
    # The first step moves by lr: 1 - 0.25 m/sqrt(v) = 0.75 after the bf16 rounding.
    assert float(small[0][0]) == 0.75 and float(small[2][0]) != 0.0
    for big, one in zip((p, m, v), (small[0], small[2], small[3])):
        assert int((big == one[0]).sum(dtype=torch.int64)) == n


@pytest.mark.parametrize("norm,max_norm", [(4.0, 1.0), (0.5, 1.0), (1.0, 0.0)])
def test_adamw_list_of_all_kinds_with_clipping(norm, max_norm):
    log(f"adamw mixed, clip {norm} {max_norm}")
    sizes = [(1 + 997 * i) % 9001 for i in range(40)]
    kinds = [list(KINDS)[i % len(KINDS)] for i in range(40)]
    a = Adam(sizes, kinds, 21, 1)
    a.step()(3, clip=(torch.tensor(norm, device=DEV), max_norm))
    a.check(3, clip_coef(norm, max_norm))


def test_adamw_first_step_and_one_shot():
    log("adamw first step")
    a, b = (Adam([300, 5000], ["master/bf16", "f32/f32"], 31, first=True) for _ in range(2))
    a.step()(1)
    a.check(1)
    nm.adamw_list_step(b.p, b.g, b.m, b.v, masters=b.masters, decays=b.decays, step=1, **HP)
    assert all(torch.equal(x, y) for x, y in zip(a.p + a.m + a.v + a.w, b.p + b.m + b.v + b.w))


def test_adamw_of_zero_gradients_and_state():
    """A row that no token reached: g = m = v = 0 only decays."""
    log("adamw zero")
    p = torch.full((1000,), 2.0, device=DEV)
    z = [torch.zeros_like(p) for _ in range(3)]
    nm.AdamWStep([p], z[:1], z[1:2], z[2:], **HP)(1)
    assert bool((p == p[0]).all()) and abs(float(p[0]) - 2.0 * (1 - 1e-4)) <= 4 * U * 2.0
    assert all(not bool(t.any()) for t in z)


def test_adamw_list_equals_the_packed_step():
    """One fp32 tensor with fp32 gradients: the packed adamw_step's arithmetic, bit for bit."""
    log("adamw packed")
    a = Adam([100_003], ["f32/f32"], 41)
    a.decays = [1.0]
    p, g, m, v = (t[0].clone() for t in (a.p, a.g, a.m, a.v))
    step = a.step()
    for t in (1, 2, 3):
        step(t)
        nm.adamw_step(p, g, m, v, step=t, **HP)
    assert torch.equal(a.p[0], p) and torch.equal(a.m[0], m) and torch.equal(a.v[0], v)


def test_adamw_learning_rate_of_a_call_stays():
    log("adamw lr")
    a, b = (Adam([777], ["f32/f32"], 51) for _ in range(2))
    step = a.step()
    step(1, lr=0.25)
    step(2)
    other = nm.AdamWStep(b.p, b.g, b.m, b.v, masters=b.masters, decays=b.decays, **{**HP, "lr": 0.25})
    other(1)
    other(2)
    assert torch.equal(a.p[0], b.p[0])


# --- streams, graphs, several lists ------------------------------------------------------------

def test_two_lists_on_two_streams():
    log("lists on two streams")
    spec = LISTS["many"]
    ref, lists, sides = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(2):
        views, _ = make(spec, 60 + k, std=1.0)
        nm.clip_grad_norm(views, 1.0)
        ref.append([v.clone() for v in views])
    states = [make(spec, 60 + k, std=1.0)[0] for k in range(2)]
    torch.cuda.synchronize()
    for k in range(2):
        lists.append(nm.GradClip(states[k], stream=sides[k]))
    norms = [lists[k].clip_norm(1.0, stream=sides[k]) for k in range(2)]
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(states[k], ref[k]))
        assert norm_close(norms[k], grad_norm([to64(v) for v in make(spec, 60 + k, std=1.0)[0]]))


def test_a_list_used_on_another_stream_than_its_own():
    log("list on another stream")
    views, _ = make(LISTS["tails"], 70)
    want = grad_norm([to64(v) for v in views])
    lst = nm.GradClip(views)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [lst.norm(stream=side) for _ in range(3)]
    by_handle = lst.norm(stream=side.cuda_stream)
    del lst  # its workspace stays until the side stream has passed
    junk = [torch.full((1 << 20,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    side.synchronize()
    assert all(norm_close(g, want) for g in got + [by_handle])
    del junk


def test_a_call_on_another_stream_waits_for_the_layout():
    """The layout is queued behind long work on its own stream; the call on a side stream comes
    after it all the same."""
    log("layout behind long work")
    views, _ = make(LISTS["tails"], 71)
    want = grad_norm([to64(v) for v in views])
    a = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        b = a @ a
    lst = nm.GradClip(views)
    got = [lst.norm(stream=side), lst.norm(stream=side)]
    side.synchronize()
    assert all(norm_close(g, want) for g in got)
    del b


def test_clip_and_adamw_in_a_graph():
    """Captured once and replayed with new values, with eager work in between."""
    log("graph")
    kinds, sizes = ["master/bf16", "bf16/f32", "f32/f32"], [50_001, 4097, 130]
    a, b = (Adam(sizes, kinds, 81) for _ in range(2))
    la, sa, lb, sb = nm.GradClip(a.g), a.step(), nm.GradClip(b.g), b.step()
    norm = torch.zeros((), device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.clip_norm(0.5, out=norm)
        sa(4, clip=(norm, 0.25))
    for k in range(4):
        for x, y in zip(a.g, b.g):
            new = torch.randn(x.numel(), device=DEV) * (k + 1)
            x.copy_(new)
            y.copy_(new)
        graph.replay()
        n = lb.clip_norm(0.5)
        sb(4, clip=(n, 0.25))
        torch.cuda.synchronize()
        assert torch.equal(norm, n)
        for x, y in zip(a.g + a.p + a.m + a.v + a.w, b.g + b.p + b.m + b.v + b.w):
            assert torch.equal(x, y)


def test_two_graphs_and_eager_calls_share_a_list():
    """One after another on one stream: each leaves the list as it found it."""
    log("two graphs, one list")
    views, _ = make(LISTS["many"] + LISTS["long"], 85, std=1.0)
    lst = nm.GradClip(views)
    a, b, e = (torch.zeros((), device=DEV) for _ in range(3))
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        lst.norm(out=a)
    with torch.cuda.graph(graphs[1]):
        lst.norm("inf", out=b)
    for k in range(4):
        for v in views:
            v.mul_(0.5 + k)
        graphs[k % 2].replay()
        graphs[1 - k % 2].replay()
        lst.norm(out=e)
        torch.cuda.synchronize()
        host = [to64(v) for v in views]
        assert torch.equal(a, e) and norm_close(a, grad_norm(host)) and float(b) == grad_norm(host, "inf")


def test_twenty_thousand_tensors():
    log("20000 tensors")
    flat = torch.randn(70_000, device=DEV)
    sizes = [1 + i % 6 for i in range(20_000)]
    views = list(flat[:sum(sizes)].split(sizes))
    host = to64(flat)
    norm = nm.clip_grad_norm(views, 2.0)
    assert norm_close(norm, grad_norm([host[:sum(sizes)]]))
    want = clip_grads([host[:sum(sizes)]], grad_norm([host[:sum(sizes)]]), 2.0)[0]
    assert np.all(np.abs(to64(flat)[:sum(sizes)] - want) <= clip_bound(want, F32))
    np.testing.assert_array_equal(to64(flat)[sum(sizes):], host[sum(sizes):])


def test_a_list_laid_out_inside_a_graph():
    """The layout travels in kernel arguments, so even a one-shot call may be captured."""
    log("one-shot in a graph")
    views, _ = make(LISTS["many"], 90, std=1.0)
    other = [v.clone() for v in views]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = nm.clip_grad_norm(views, 1.0)
        inside = nm.GradClip(views)
        inside.clip(norm, 1e30)
    with pytest.raises(RuntimeError, match="inside a graph capture"):
        inside.norm()  # its table exists only in replays
    for k in range(3):
        for v, o in zip(views, other):
            new = torch.randn(v.numel(), device=DEV) * (k + 1)
            v.copy_(new)
            o.copy_(new)
        graph.replay()
        n = nm.clip_grad_norm(other, 1.0)
        torch.cuda.synchronize()
        assert torch.equal(norm, n) and all(torch.equal(v, o) for v, o in zip(views, other))


def test_refusals_on_the_gpu():
    log("refusals")
    g = torch.ones(10, device=DEV)
    lst = nm.GradClip([g])
    with pytest.raises(nm.MuonError) as e:
        nm.GradClip([g, g])
    assert e.value.status == nm.MUON_EALIAS
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(nm.MuonError):
            lst.clip_norm(bad)
    with pytest.raises(ValueError, match="norm must be"):
        lst.clip(torch.ones(2, device=DEV), 1.0)
    with pytest.raises(ValueError, match="norm must be"):
        lst.clip(torch.ones(()), 1.0)
    with pytest.raises(ValueError, match="norm must be"):
        lst.norm(out=torch.zeros((), device=DEV, dtype=torch.float64))
    with pytest.raises(ValueError, match="workspace"):
        nm.GradClip([g], workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="workspace is on"):
        nm.GradClip([g], workspace=torch.empty(1 << 20, dtype=torch.uint8))
    inside = lst.workspace[4096:4100].view(F32)
    for call in (lambda: lst.norm(out=inside), lambda: lst.clip(inside, 1.0), lambda: lst.clip_norm(1.0, out=inside)):
        with pytest.raises(nm.MuonError) as e:
            call()
        assert e.value.status == nm.MUON_EALIAS
    p, m, v = torch.ones(10, device=DEV), torch.zeros(10, device=DEV), torch.zeros(10, device=DEV)
    with pytest.raises(nm.MuonError):
        nm.AdamWStep([p], [g], [m], [v])(0)
    with pytest.raises(nm.MuonError):
        nm.AdamWStep([p], [g], [m], [v], beta1=1.0)(1)
    torch.cuda.synchronize()
    assert bool((g == 1).all()) and bool((p == 1).all())


def test_profile_names():
    log("profile")
    views, _ = make([(5000, F32)], 1, std=1.0)
    lst = nm.GradClip(views)
    nm.profile_begin()
    lst.clip_norm(1.0)
    prof = nm.profile_end()
    assert {"grad_norm", "grad_clip"} <= set(prof)
    assert prof["grad_norm"]["bytes"] == 20000 and prof["grad_clip"]["bytes"] == 40000
