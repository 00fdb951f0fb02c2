"""What FvattnCache and FvattnPlan keep between calls, with the device calls replaced by fakes: lengths,
first errors, buffers."""
import pytest
import torch

import top_routed_block_b200 as fv


class Calls:
    """Stands in for the device calls: writes the next of the given status words, as they do."""

    def __init__(self, monkeypatch):
        self.append, self.attend = [], []
        monkeypatch.setattr(fv, "fvattn_cache_append", self._append)
        monkeypatch.setattr(fv, "fvattn_cache_attend", self._attend)
        self.captured = False
        monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.captured)

    def _append(self, K, V, pages, table, start, *, dev_status, **kw):
        dev_status[0] = self.append.pop(0) if self.append else 0
        return dev_status

    def _attend(self, Q, pages, table, lens, *, dev_status, **kw):
        dev_status[0] = self.attend.pop(0) if self.attend else 0
        return Q, None, dev_status


@pytest.fixture
def calls(monkeypatch):
    return Calls(monkeypatch)


def cache(B=3):
    return fv.FvattnCache(B, 2, 64, 64, 256, device="cpu")


def rows(B, T):
    return torch.zeros(B, 2, T, 64, dtype=torch.bfloat16)


def test_lengths_are_what_was_appended(calls):
    """The kernel holds a count inside [0, T]; the lengths follow it."""
    c = cache()
    c.append(rows(3, 10), rows(3, 10))
    assert c.lens.tolist() == [10, 10, 10]
    given = torch.tensor([11, -4, 3], dtype=torch.int32)
    c.append(rows(3, 10), rows(3, 10), new_lens=given)
    assert c.lens.tolist() == [20, 10, 13] and given.tolist() == [11, -4, 3]
    c.append(rows(3, 1), rows(3, 1), new_lens=torch.tensor([-(2 ** 31), 2 ** 31 - 1, 0], dtype=torch.int32))
    assert c.lens.tolist() == [20, 11, 13]


@pytest.mark.parametrize("call,codes", [
    ("append", [0, -8, 0, 0]), ("attend", [-7, 0]), ("attend", [0, -8, 0]), ("append", [-8]),
    ("append", [0, -8] + [0] * 700), ("attend", [0] * 127 + [-8]), ("append", [0] * 128 + [-8, 0, -7]), ("attend", [0] * 300 + [-8] + [0] * 126),
])
def test_errors_stay_until_they_are_reported(calls, call, codes):
    c = cache()
    c.check()
    getattr(calls, call).extend(codes)
    for _ in codes:
        c.append(rows(3, 1), rows(3, 1))
        c.attend(rows(3, 1))
    assert c.status.tolist() == ([codes[-1], 0] if call == "append" else [0, codes[-1]])
    with pytest.raises(fv.FvattnError) as e:
        c.check()
    assert e.value.status == min(codes)
    c.append(rows(3, 1), rows(3, 1))
    c.attend(rows(3, 1))
    c.check()


def test_errors_of_captured_calls_stay(calls):
    """A captured call writes the same word at every replay and keeps its errors itself; calls outside the graph, also
    many of them, have other words."""
    c = cache()
    c.append(rows(3, 1), rows(3, 1))
    c.check()
    calls.captured = True
    calls.append, calls.attend = [0, -8, 0, 0], [0, -7, 0, 0]
    words = set()
    for _ in range(4):
        c.append(rows(3, 1), rows(3, 1))
        c.attend(rows(3, 1))
        words.add((c._last[0].data_ptr(), c._last[1].data_ptr()))
    assert len(words) == 1
    calls.captured = False
    for _ in range(300):
        c.attend(rows(3, 1))
        assert all(c._last[1].data_ptr() not in w for w in words)
    with pytest.raises(fv.FvattnError) as e:
        c.check()
    assert e.value.status == -8
    c.check()


def test_a_plan_allocates_the_turned_tensors_once(monkeypatch):
    given = []

    def rope(Q, K, positions, axes, *, out_q=None, out_k=None, stream=None):
        given.append((out_q, out_k))
        return (torch.empty_like(Q) if out_q is None else out_q, torch.empty_like(K) if out_k is None else out_k)

    monkeypatch.setattr(fv, "fvattn_rope", rope)
    monkeypatch.setattr(fv, "fvattn_route", lambda Q, K, *a, **kw: None)
    monkeypatch.setattr(fv, "fvattn_sparse_fwd", lambda Q, K, *a, **kw: (Q, K))
    plan = fv.FvattnPlan(1, 2, 100, 64, 64, device="cpu")
    x = torch.zeros(1, 2, 100, 64, dtype=torch.bfloat16)
    first = plan(x, x, x, 0.9, positions=x, rope=x)
    assert plan.turned == first and given == [(None, None)]
    plan(x, x, x, 0.9)
    assert plan.turned is None
    again = plan(x, x, x, 0.9, positions=x, rope=x)
    assert given[1][0] is first[0] and given[1][1] is first[1] and again[0] is first[0] and plan.turned[1] is first[1]
