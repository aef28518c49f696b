"""GPU: the list operators in graph captures and on streams of their own.  Tolerances as in
test_gpu_list_ops."""

from __future__ import annotations

import ctypes

import pytest
import torch

import newton_schulz_02_amd as nm
from oracle.grad_oracle import grad_norm
from tests.gpu_helpers import DEV, log, to64
from tests.test_gpu_list_ops import LISTS, make, norm_close

pytestmark = pytest.mark.gpu


def test_a_list_of_one_capture_is_refused_in_another():
    """The second capture would record calls on a table that only replays of the first write.
    Nothing of the refused calls is recorded."""
    log("list of another capture")
    views, _ = make(LISTS["tails"], 100, std=1.0)
    p, m, v = ([torch.zeros_like(x, dtype=torch.float32) for x in views] for _ in range(3))
    norm, other = torch.zeros((), device=DEV), torch.ones((), device=DEV)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        lst = nm.GradClip(views)
        adam = nm.AdamWStep(p, views, m, v)
        lst.norm(out=norm)
    with torch.cuda.graph(graphs[1]):
        other.add_(1.0)
        calls = [lambda: lst.norm(out=other), lambda: lst.norm(), lambda: lst.clip(norm, 1.0),
                 lambda: lst.clip_norm(1.0, out=other), lambda: adam(1)]
        for call in calls:
            with pytest.raises(RuntimeError, match="inside a graph capture"):
                call()
        # The library's own check, for callers without the binding.
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert nm.lib().muon_grad_norm(ctypes.byref(lst.list), 0, ctypes.c_void_p(other.data_ptr()),
                                       stream) == nm.MUON_EINVAL
        assert "inside a graph capture" in nm.last_error()
        hp = nm.adamw_hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1)
        assert nm.lib().adamw_list_step(ctypes.byref(adam.list), ctypes.byref(hp), None, stream) == nm.MUON_EINVAL
    for k in range(3):
        graphs[1].replay()  # before the first one: only the addition
        graphs[0].replay()
        torch.cuda.synchronize()
        assert float(other) == 2.0 + k
        assert norm_close(norm, grad_norm([to64(x) for x in views]))
        for x in views:
            x.mul_(0.5)
    assert not any(bool(t.any()) for t in p + m + v)


def test_a_captured_list_on_streams_beside_its_capture():
    """Refused on a stream that has not joined the capture; used on one that has."""
    log("list and a side stream of a capture")
    views, _ = make(LISTS["tails"], 101, std=1.0)
    norm, apart = torch.zeros((), device=DEV), torch.zeros((), device=DEV)
    side, stranger = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)  # joins before the layout, which the call waits for all the same
        lst = nm.GradClip(views)
        for out in (apart, None):
            with pytest.raises(RuntimeError, match="inside a graph capture"):
                lst.norm(out=out, stream=stranger)
        lst.norm(out=norm, stream=side)
        main.wait_stream(side)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert norm_close(norm, grad_norm([to64(x) for x in views])) and float(apart) == 0.0
        for x in views:
            x.mul_(0.5)


def test_norms_of_one_list_on_streams_in_turn():
    """Called on three streams with no waits of the caller's own: each norm comes after the last
    one, whose counts and partial results lie in the same workspace."""
    log("norms in turn")
    views, _ = make(LISTS["long"] + LISTS["many"], 102, std=1.0)
    host = [to64(x) for x in views]
    want = {kind: grad_norm(host, kind) for kind in ("l2", "inf")}
    lst = nm.GradClip(views)
    torch.cuda.synchronize()
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for k in range(30):
        kind = ("l2", "inf")[k % 2]
        outs.append((kind, lst.norm(kind, stream=streams[k * 7 % 3])))
    torch.cuda.synchronize()
    for kind, got in outs:
        assert norm_close(got, want[kind])


def test_norms_of_one_list_on_branches_of_a_capture():
    log("norms on branches")
    views, _ = make(LISTS["long"], 103, std=1.0)
    lst = nm.GradClip(views)
    outs = [torch.zeros((), device=DEV) for _ in range(4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for k, out in enumerate(outs):
            lst.norm(out=out, stream=side if k % 2 else None)
        main.wait_stream(side)
    for k in range(4):
        graph.replay()
        eager = lst.norm()
        torch.cuda.synchronize()
        want = grad_norm([to64(x) for x in views])
        assert all(torch.equal(out, eager) for out in outs) and norm_close(eager, want)
        for x in views:
            x.mul_(0.5)


@pytest.mark.parametrize("spec", ["long", "tails"])  # counted in groups, and by one count
def test_overlapping_norms_leave_the_list_usable(spec):
    """Through the library, which orders nothing: the values of norms that overlap are undefined,
    but the next ones, after a synchronisation, are right."""
    log(f"overlapping norms, {spec}")
    views, _ = make(LISTS[spec], 104, std=1.0)
    want = grad_norm([to64(x) for x in views])
    lst = nm.GradClip(views)
    outs = torch.zeros(8, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(10):
        for k in range(8):
            rc = nm.lib().muon_grad_norm(ctypes.byref(lst.list), 0, ctypes.c_void_p(outs.data_ptr() + 4 * k),
                                         ctypes.c_void_p(streams[k % 4].cuda_stream))
            assert rc == nm.MUON_OK
        torch.cuda.synchronize()
        assert norm_close(lst.norm(), want) and norm_close(lst.norm(), want)
        torch.cuda.synchronize()


def busy(stream):
    """Queue some 20 ms of work on a stream."""
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device=DEV)
        for _ in range(30):
            a = a @ a * 2.0 ** -12
    return a


def places(numel, dtype, count=64):
    """Addresses that the allocator gives tensors of the current stream now; nothing is written."""
    return {t.data_ptr() for t in [torch.empty(numel, dtype=dtype, device=DEV) for _ in range(count)]}


def test_a_dropped_norm_stays_until_its_named_stream_has_read_it():
    """clip=(norm, limit) on a side stream that is still busy, the norm dropped at once: its
    memory is not given away before the side stream gets there."""
    log("norm dropped while a stream is busy")
    views, _ = make([(5000, torch.float32)], 105, std=1.0)
    p, m, v = ([torch.zeros(5000, device=DEV)] for _ in range(3))
    w, g, mom = (torch.zeros(64, 64, device=DEV) for _ in range(3))
    lst, adam, muon = nm.GradClip(views), nm.AdamWStep(p, views, m, v), nm.MuonStep([w], [g], [mom])
    side = torch.cuda.Stream()
    calls = [lambda n: adam(1, clip=(n, 1.0), stream=side), lambda n: lst.clip(n, 1.0, stream=side),
             lambda n: muon(side, clip=(n, 1.0)), lambda n: lst.norm(out=n, stream=side)]
    for call in calls:
        norm = torch.full((), 2.0, device=DEV)
        at = norm.data_ptr()
        torch.cuda.synchronize()
        keep = busy(side)
        call(norm)
        del norm
        assert at not in places((), torch.float32)
        assert not side.query()  # the side stream was still busy
        side.synchronize()
        del keep


def test_a_dropped_list_keeps_its_workspace_until_its_streams_have_passed():
    log("list dropped while a stream is busy")
    views, _ = make(LISTS["tails"], 106, std=1.0)
    want = grad_norm([to64(x) for x in views])
    lst = nm.GradClip(views)
    at, size = lst.workspace.data_ptr(), lst.workspace.numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = busy(side)
    norm = lst.norm(stream=side)
    del lst
    assert at not in places(size, torch.uint8)
    assert not side.query()
    side.synchronize()
    assert norm_close(norm, want)
    del keep


def test_an_expanded_workspace_is_refused():
    log("expanded workspace")
    g = torch.ones(10, device=DEV)
    for bad in (torch.zeros(1, dtype=torch.uint8, device=DEV).expand(1 << 20),
                torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            nm.GradClip([g], workspace=bad)
        with pytest.raises(ValueError, match="contiguous"):
            nm.AdamWStep([g], [g.clone()], [g.clone()], [g.clone()], workspace=bad)


@pytest.mark.parametrize("own", [False, True])  # eager norms on the default stream, or one of their own
def test_eager_and_captured_norms_of_one_list(own):
    """Eager norms before the capture, between captures and between replays."""
    log("eager and captured norms")
    views, _ = make(LISTS["long"], 107, std=1.0)
    lst = nm.GradClip(views)
    outs = [torch.zeros((), device=DEV) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.stream(torch.cuda.Stream() if own else torch.cuda.current_stream()):
        for graph, out in zip(graphs, outs):
            first = lst.norm()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                lst.norm(out=out)
        for k in range(4):
            graphs[k % 2].replay()
            eager = lst.norm()
            graphs[1 - k % 2].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
            assert norm_close(eager, grad_norm([to64(x) for x in views]))
            for x in views:
                x.mul_(0.5)
        assert float(first) > 0.0
