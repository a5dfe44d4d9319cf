"""Where a plan's runs are ordered, on fakes of streams, events and the library."""
import pytest

from huffman_decode_df11_b200 import linear

HOME, SIDE, THIRD = 11, 12, 13


class _Fake:
    """The calls of one plan: what it asked the library and the streams for, in order."""

    def __init__(self, monkeypatch, capture=0):
        self.log, self.captures, self.done, self.current = [], {HOME: capture}, 0, HOME
        fake = self

        class Event:
            cuda_event = 77

            def __init__(self, external=False):
                self.external = external

            def record(self):
                fake.log.append(("record", fake.current, self.external))

        class Stream:
            def __init__(self, handle):
                self.handle = handle

            def wait_event(self, event):
                fake.log.append(("wait", self.handle))

        class Work:
            def record_stream(self, s):
                fake.log.append(("record_stream", s.handle))

            def data_ptr(self):
                return 0

        class Lib:
            def df11_capture_id(self, handle):
                return fake.captures.get(handle, 0)

            def df11_event_done(self, event):
                return fake.done

            def df11_decode_linear(self, *args):
                fake.log.append(("run", args[-1]))
                return 0

        class Device:
            index = 0

        monkeypatch.setattr(linear, "_on_stream", Stream)
        monkeypatch.setattr(linear, "_stream_handle", lambda s: self.current if s is None else s)
        monkeypatch.setattr(linear.torch.cuda, "Event", Event)
        monkeypatch.setattr(linear.torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(linear.torch.cuda, "is_current_stream_capturing",
                            lambda: bool(self.captures.get(self.current, 0)))
        self.plan = linear.LinearPlan([], [], [])
        p = self.plan
        p._n, p._lib, p._work, p._device, p._descs, p._ops = 1, Lib(), Work(), Device(), None, None
        p._streams = {HOME}
        if hasattr(p, "_mark"):
            p._mark()
        self.made, self.log = list(self.log), []

    def run(self, stream=None):
        self.log = []
        self.plan.run(stream=stream)
        return self.log


def test_the_first_run_on_another_stream_waits(monkeypatch):
    f = _Fake(monkeypatch)
    assert f.made == [("record", HOME, True)]
    assert f.run() == [("run", HOME)]
    assert f.run(SIDE) == [("wait", SIDE), ("record_stream", SIDE), ("run", SIDE)]
    assert f.run(SIDE) == [("run", SIDE)]
    assert f.run(THIRD) == [("wait", THIRD), ("record_stream", THIRD), ("run", THIRD)]


def test_no_wait_once_the_earlier_work_is_done(monkeypatch):
    f = _Fake(monkeypatch)
    f.done = 1
    assert f.run(SIDE) == [("record_stream", SIDE), ("run", SIDE)]
    f.captures[THIRD] = 5
    assert f.run(THIRD) == [("run", THIRD)]


@pytest.mark.parametrize("stream", [HOME, SIDE])
def test_a_captured_run_waits_wherever_it_is(monkeypatch, stream):
    # a graph may be replayed on another stream than the one it was captured on
    f = _Fake(monkeypatch)
    f.run(stream)
    f.captures[stream] = 5
    for _ in range(2):
        assert f.run(stream) == [("wait", stream), ("run", stream)]
    f.done = 1
    assert f.run(stream) == [("run", stream)]


def test_a_plan_made_in_a_capture(monkeypatch):
    f = _Fake(monkeypatch, capture=5)
    assert f.made == [("record", HOME, False)]
    assert f.run() == [("run", HOME)]
    f.captures[SIDE] = 5                    # forked within the capture
    assert f.run(SIDE) == [("wait", SIDE), ("run", SIDE)]
    f.captures = {SIDE: 6}                  # another one cannot wait for its event
    assert f.run(SIDE) == [("run", SIDE)]
    f.captures = {}
    assert f.run(THIRD) == [("record_stream", THIRD), ("run", THIRD)]


def test_a_plan_for_one_call_marks_nothing(monkeypatch):
    f = _Fake(monkeypatch)
    monkeypatch.setattr(linear.torch.cuda, "Event", None)
    p = linear._OneRun([], [], [])
    p._mark()
    assert p._born is None and f.plan._born is not None


def test_the_library_s_answers_without_a_device():
    from huffman_decode_df11_b200 import lib
    assert lib().df11_event_done(None) == -1
    assert lib().df11_capture_id(None) == 0


def test_the_event_of_a_graph_s_wait_lives_as_long_as_the_plan(monkeypatch):
    import weakref
    f = _Fake(monkeypatch)
    event = weakref.ref(f.plan._born)
    f.captures[SIDE] = 5
    assert ("wait", SIDE) in f.run(SIDE)     # a node of the graph's that names the event
    f.captures, f.done = {}, 1
    f.run()
    assert f.plan._born is None and event() is not None
    del f.plan
    assert event() is None
