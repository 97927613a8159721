"""Lookups whose backward adds to one gradient buffer, on several streams: each sum waits for the one before it.

Without a GPU: the kernels are replaced by the formula on the host, and streams and events by ones that log."""
import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma

LOG = []


class Stream:
    def __init__(self, name):
        self.name = name

    def wait_event(self, event):
        LOG.append(("wait", self.name, event.after))

    def wait_stream(self, other):
        LOG.append(("wait for all of", self.name, other.name))


class Event:
    after = None

    def __init__(self, **kw):
        pass

    def record(self, stream):
        LOG.append(("event",))
        self.after = stream.name, sum(e[0] == "add" for e in LOG)


@pytest.fixture
def fake(monkeypatch):
    """fake(names): the streams that are current in the order of the sums; fake.captured: whether they are captured."""
    LOG.clear()
    here = {"names": [], "captured": []}

    def lookup(ids, table, scale=1.0, padding=None, out=None, dtype=None, stream=None):
        return table[ids] * scale

    def grad(ids, dy, buf, scale=1.0, padding=None, accumulate=False, ws=None, stream=None):
        LOG.append(("add", here["names"][0].name))
        here["names"].pop(0)
        if here["captured"]:
            here["captured"].pop(0)
        return buf.index_add_(0, ids, dy * scale)

    monkeypatch.setattr(ma, "embedding_lookup", lookup)
    monkeypatch.setattr(ma, "embedding_grad", grad)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: here["names"][0].name)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: bool(here["captured"] and here["captured"][0]))
    monkeypatch.setattr(torch.cuda, "synchronize", lambda index=None: LOG.append(("synchronize",)))
    monkeypatch.setattr(ma, "_LAST_SUM", {})
    monkeypatch.setattr(ma, "_SUM_STREAMS", {})
    streams = {}

    def use(names, captured=(), known=None):
        """known: the streams that lookups ran on before the backward pass (by default those of the sums)."""
        for n in names if known is None else known:
            ma._SUM_STREAMS.setdefault(-1, {}).setdefault(n, Stream(n))  # -1: a host tensor's device
        here["names"] = [streams.setdefault(n, Stream(n)) for n in names]
        here["captured"] = list(captured)

    return use


def passes(lookups, calls=1):
    """`calls` backward passes over `lookups` lookups each, into one buffer."""
    table, buf = torch.ones((5, 4), requires_grad=True), torch.zeros((5, 4))
    ids = torch.tensor([0, 3, 3])
    for _ in range(calls):
        sum(ma.embedding(ids, table, grad=buf).sum() for _ in range(lookups)).backward()
    return buf


def test_sums_on_two_streams_wait_for_one_another(fake):
    fake("aba")
    buf = passes(3)
    assert buf[3].tolist() == [6.0] * 4
    assert [e for e in LOG if e[0] != "event"] == [("add", "a"), ("wait", "b", ("a", 1)), ("add", "b"),
                                                   ("wait", "a", ("b", 2)), ("add", "a")]


def test_sums_on_one_stream_wait_for_nothing_and_record_nothing(fake):
    fake("aaaa")
    passes(2, calls=2)
    assert LOG == [("add", "a")] * 4


def test_the_first_sum_on_a_second_stream_within_a_pass(fake):
    # a stream that no lookup was on before the backward pass (made within it): the sum before it has no event
    fake("abab", known="a")
    passes(4)
    assert [e for e in LOG if e[0] != "event"] == [
        ("add", "a"), ("wait for all of", "b", "a"), ("add", "b"), ("wait", "a", ("b", 2)), ("add", "a"),
        ("wait", "b", ("a", 3)), ("add", "b")]


def test_the_first_sum_on_a_second_stream_in_a_later_pass(fake):
    fake("aab", known="a")
    passes(1, calls=3)
    assert [e for e in LOG if e[0] != "event"] == [("add", "a"), ("add", "a"), ("synchronize",), ("add", "b")]


def test_the_first_captured_sum_waits_for_no_eager_one(fake):
    fake("ab", [False, True], known="a")
    passes(1, calls=2)
    assert [e for e in LOG if e[0] != "event"] == [("add", "a"), ("add", "b")]


def test_a_later_backward_pass_waits_too(fake):
    fake("ab")
    passes(1, calls=2)
    assert ("wait", "b", ("a", 1)) in LOG


def test_inside_a_capture_only_sums_of_the_same_pass_are_waited_for(fake):
    # an event recorded outside a capture cannot be waited for inside it, nor one inside it outside
    fake("abab" "cd", [False, False, True, True, False, False])
    passes(2, calls=3)
    waits = [e[1:] for e in LOG if e[0] == "wait"]
    assert waits == [("b", ("a", 1)), ("b", ("a", 3)), ("d", ("c", 5))]
