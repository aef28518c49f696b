"""CPU tests of how the list classes deal with streams and graph captures, with the stream calls
replaced by recorders: no test here launches a kernel."""

from __future__ import annotations

import ctypes
import types

import pytest
import torch

import newton_schulz_02_amd as nm


class Stream:
    """Stands in for a stream: its handle, the capture it takes part in, and what was asked of it."""

    def __init__(self, handle, capture=0):
        self.cuda_stream, self.capture, self.waits, self.device = handle, capture, [], torch.device("cuda", 0)

    def wait_event(self, event):
        self.waits.append(event)

    def record_event(self):
        return ("event of", self.cuda_stream, self.capture)


def laid_out(home, cls=nm.GradClip):
    """A list laid out on `home`, without a device."""
    lst = object.__new__(cls)
    lst.device, lst.count = torch.device("cuda", 0), 0
    lst._home, lst._capture, lst._laid_out = home.cuda_stream, home.capture, home.record_event()
    lst._ordered = {lst._home}
    lst._current_device = lambda: 0
    lst._norm_last, lst._norm_streams = None, set()
    lst.workspace = types.SimpleNamespace(record_stream=lambda s: None)
    lst.list = lst._list = None
    return lst


@pytest.fixture
def streams(monkeypatch):
    """Streams by handle; the library's and torch's answers on them."""
    known = {}

    def make(handle, capture=0):
        known[handle] = Stream(handle, capture)
        return known[handle]

    monkeypatch.setattr(nm, "_capture_of", lambda handle: known[handle].capture)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: known[handle])
    return make


def calls():
    seen = []

    def fn(*args):
        seen.append(args)
        return nm.MUON_OK
    return fn, seen


def use(lst, stream):
    fn, seen = calls()
    lst._call(fn, (), stream, lst._handle(stream))
    return seen


def test_a_captured_list_is_for_streams_of_its_capture(streams):
    home = streams(1, capture=7)
    lst = laid_out(home)
    assert use(lst, home) and not home.waits
    # A branch of the same capture waits for the layout, each time.
    branch = streams(2, capture=7)
    assert use(lst, branch) and use(lst, branch)
    assert branch.waits == [lst._laid_out] * 2
    # Nothing is asked of a stream outside, and no call is made.
    for other in (streams(3), streams(4, capture=8)):
        with pytest.raises(RuntimeError, match="inside a graph capture"):
            use(lst, other)
        assert not other.waits
    # The same stream in a later capture, and after both.
    for capture in (8, 0):
        home.capture = capture
        with pytest.raises(RuntimeError, match="inside a graph capture"):
            use(lst, home)


def test_an_eager_list_waits_once_for_its_layout(streams):
    lst = laid_out(streams(1))
    side = streams(2)
    assert use(lst, side) and use(lst, side)
    assert side.waits == [lst._laid_out]
    graph = streams(3, capture=7)  # cannot wait for what is outside
    assert use(lst, graph) and not graph.waits


def norm(lst, stream):
    fn, seen = calls()
    with pytest.MonkeyPatch.context() as patch:
        patch.setattr(nm, "lib", lambda: types.SimpleNamespace(muon_grad_norm=fn))
        lst.norm(out=Value(), stream=stream)
    assert len(seen) == 1


def waited(stream, lst):
    """Streams that `stream` was made to wait for (the layout aside), and forget them."""
    out = [e[1] for e in stream.waits if e is not lst._laid_out]
    stream.waits.clear()
    return out


def test_norms_of_a_list_come_one_after_another(streams):
    a, b, c = (streams(k) for k in (1, 2, 3))
    lst = laid_out(a)
    norm(lst, a)
    norm(lst, a)
    assert not a.waits
    norm(lst, b)
    assert waited(b, lst) == [1]
    norm(lst, b)
    assert not b.waits
    norm(lst, c)
    assert waited(c, lst) == [2]
    norm(lst, a)
    assert waited(a, lst) == [3]


def test_norms_inside_a_capture_and_outside_do_not_wait_for_each_other(streams):
    a, b, c, d = (streams(k) for k in (1, 2, 3, 4))
    lst = laid_out(a)
    norm(lst, a)
    b.capture = c.capture = 7
    norm(lst, b)
    assert waited(b, lst) == []
    norm(lst, c)  # a branch of the same capture
    assert waited(c, lst) == [2]
    norm(lst, d)  # eager: the eager norm before it was on a
    assert waited(d, lst) == [1]
    norm(lst, c)
    assert waited(c, lst) == [2]  # b's capture goes on
    d.capture = 9  # d's eager norm was before this capture, so nothing can wait for it
    norm(lst, a)
    assert waited(a, lst) == []
    b.capture = c.capture = d.capture = 0
    norm(lst, b)
    assert set(waited(b, lst)) == {1, 3, 4}
    norm(lst, a)
    assert waited(a, lst) == [2]


def test_a_branch_waits_for_a_norm_that_its_origin_captured(streams):
    """The origin stream held the last norm before the capture, too."""
    a, b = streams(1), streams(2)
    lst = laid_out(a)
    norm(lst, a)
    a.capture = b.capture = 7
    norm(lst, a)
    norm(lst, b)
    assert waited(b, lst) == [1]


class Value:
    """Stands in for a norm on the device."""

    def __init__(self):
        self.dtype, self.device, self.kept = torch.float32, torch.device("cuda", 0), []

    def numel(self):
        return 1

    def data_ptr(self):
        return 1 << 30

    def record_stream(self, stream):
        self.kept.append(stream.cuda_stream)


@pytest.mark.parametrize("call", ["norm", "clip", "clip_norm", "adamw", "muon"])
def test_a_norm_used_on_a_named_stream_is_kept_until_then(streams, monkeypatch, call):
    ok = types.SimpleNamespace(**{name: lambda *a: nm.MUON_OK for name in (
        "muon_grad_norm", "muon_grad_clip", "muon_grad_clip_norm", "adamw_list_step_double", "muon_step_clipped")})
    monkeypatch.setattr(nm, "lib", lambda: ok)
    a, b = streams(1), streams(2)
    grads, adam, muon = laid_out(a), laid_out(a, nm.AdamWStep), object.__new__(nm.MuonStep)
    adam.hp = nm.adamw_hparams_double()
    muon.arr, muon.count, muon.hp, muon.device = None, 0, nm.make_hparams(), torch.device("cuda", 0)
    muon.workspace = torch.zeros(1)
    run = {"norm": lambda x, s: grads.norm(out=x, stream=s), "clip": lambda x, s: grads.clip(x, 1.0, stream=s),
           "clip_norm": lambda x, s: grads.clip_norm(1.0, out=x, stream=s),
           "adamw": lambda x, s: adam(1, clip=(x, 1.0), stream=s), "muon": lambda x, s: muon(s, clip=(x, 1.0))}[call]
    for stream in (a, b):
        x = Value()
        run(x, stream)
        assert x.kept == [stream.cuda_stream]


def test_a_stream_of_another_device_is_refused(streams):
    a, b = streams(1), streams(2)
    b.device = torch.device("cuda", 1)
    lst = laid_out(a)
    for call in (lambda: use(lst, b), lambda: norm(lst, b)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()
    assert not b.waits


def test_a_refused_update_leaves_the_learning_rate(streams, monkeypatch):
    rates, answers = [], [nm.MUON_OK, nm.MUON_EINVAL, nm.MUON_OK]

    def step(lst, hp, clip, stream):
        rates.append(hp._obj.lr)
        return answers.pop(0)

    lib = types.SimpleNamespace(adamw_list_step_double=step, muon_strerror=lambda c: b"", muon_last_error=lambda: b"")
    monkeypatch.setattr(nm, "lib", lambda: lib)
    a = streams(1)
    adam = laid_out(a, nm.AdamWStep)
    adam.hp = nm.adamw_hparams_double(0.5)
    adam(1, lr=0.25, stream=a)
    with pytest.raises(nm.MuonError):
        adam(2, lr=float("nan"), stream=a)
    adam(2, stream=a)
    assert rates[0] == rates[2] == 0.25


def test_stream_capture_arguments():
    out = ctypes.c_uint64(5)
    assert nm.lib().muon_stream_capture(None, None) == nm.MUON_EINVAL
    assert nm.lib().muon_stream_capture(None, ctypes.byref(out)) == nm.MUON_OK and out.value == 0  # the null stream
