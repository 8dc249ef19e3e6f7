"""Which scratch the binding hands to an attention call (host logic; the
allocator is a stand-in, so no GPU is needed)."""
import ctypes

import pytest

import block_quantized_gemv_q8_gb300 as qx


class Allocator:
    """Hands out addresses, and knows which of them are still held."""

    def __init__(self):
        self.made, self.live = [], set()

    def __call__(self, index, stream, nbytes):
        outer = self

        class Owner:
            def __init__(self, n):
                self.n = n
                outer.live.add(n)

            def __del__(self):
                outer.live.discard(self.n)

        self.made.append((index, stream, nbytes))
        n = 4096 * len(self.made)
        return n, Owner(n)


@pytest.fixture
def pool():
    allocate = Allocator()
    return qx._Scratch(allocate), allocate


def test_a_stream_keeps_its_buffer_until_a_call_needs_more(pool):
    scratch, a = pool
    first = scratch.get(0, 7, 0, 1000)
    assert scratch.get(0, 7, 0, 10) == scratch.get(0, 7, 0, 1000) == first
    assert scratch.get(0, 8, 0, 10) != first and scratch.get(1, 7, 0, 10) != first
    more = scratch.get(0, 7, 0, 1001)
    assert more != first and first not in a.live and scratch.get(0, 7, 0, 1000) == more
    assert a.made == [(0, 7, 1000), (0, 8, 10), (1, 7, 10), (0, 7, 1001)]


def test_a_capture_has_a_buffer_of_its_own(pool):
    """Neither the stream's, which later calls may replace, nor another capture's, which was cleared for its own graph."""
    scratch, a = pool
    eager = scratch.get(0, 7, 0, 1000)
    g1 = scratch.get(0, 7, 21, 100)
    assert g1 != eager and scratch.get(0, 7, 21, 50) == g1  # one for the calls of a capture
    assert scratch.get(0, 9, 21, 50) not in (eager, g1)     # but another on a branch of it
    g2 = scratch.get(0, 7, 22, 100)
    assert g2 not in (eager, g1)
    assert scratch.get(0, 7, 0, 1000) == eager and eager in a.live
    assert scratch.get(0, 7, 0, 5000) not in (eager, g1, g2) and g2 in a.live


def test_a_capture_that_needs_more_gets_another_cleared_buffer(pool):
    scratch, a = pool
    small = scratch.get(0, 7, 5, 100)
    large = scratch.get(0, 7, 5, 200)
    assert large != small and scratch.get(0, 7, 5, 100) == large


def test_captures_that_are_over_are_let_go(pool):
    scratch, a = pool
    for capture in range(1, 50):
        scratch.get(0, 7, capture, 100)
    assert len(a.live) == 1
    # two captures in turn: each call finds a buffer that its own graph clears
    x, y, z = scratch.get(0, 7, 60, 100), scratch.get(0, 8, 61, 100), scratch.get(0, 7, 60, 100)
    assert len({x, y, z}) == 3


def test_outside_of_captures_there_is_no_capture():
    qx.build_library()
    assert qx.lib().qx_stream_capture_id(ctypes.c_void_p(None)) == 0


def test_the_caches_of_a_stack_share_a_streams_scratch(monkeypatch):
    """Each object had one of its own: 144 MB for every layer of a stack."""
    qx.build_library()
    allocate = Allocator()
    monkeypatch.setattr(qx.PagedKV, "_scratch", qx._Scratch(allocate))

    def cache():
        kv = object.__new__(qx.PagedKV)
        kv.heads, kv.head_dim, kv.n_seqs, kv._index, kv._needs = 8, 128, 1, 0, {}
        return kv

    layers = [cache() for _ in range(4)]
    assert len({kv.scratch(300, 32, 7) for kv in layers}) == 1
    assert len({kv.scratch(1, 32, 7) for kv in layers}) == 1
    assert len({kv.scratch(1, 32, 7, 5) for kv in layers}) == 1  # and a graph's
    assert [m[:2] for m in allocate.made] == [(0, 7), (0, 7)] and allocate.made[1][2] < allocate.made[0][2]


@pytest.mark.parametrize("status", [qx.QX_ERR_DEVICE_TIMEOUT, qx.QX_ERR_RANGE, qx.QX_OK])
def test_scratch_of_calls_that_gave_up_is_not_used_again(monkeypatch, status):
    """A wait that ran out leaves arrival counters that are not zero; a page out of range does not."""
    class Lib:
        qx_device_check = staticmethod(lambda stream: status)

    allocate = Allocator()
    monkeypatch.setattr(qx.PagedKV, "_scratch", qx._Scratch(allocate))
    monkeypatch.setattr(qx, "lib", lambda: Lib)
    old = [qx.PagedKV._scratch.get(0, 7, capture, 100) for capture in (0, 3)]
    assert qx.qx_device_check(stream=0) == status
    new = [qx.PagedKV._scratch.get(0, 7, capture, 100) for capture in (0, 3)]
    assert set(old).isdisjoint(new) if status == qx.QX_ERR_DEVICE_TIMEOUT else old == new
