"""GPU tests of attention calls in captured graphs, several on one cache: each
graph has scratch of its own, cleared by itself, whatever is captured, replayed
or called around it."""
import pytest
import torch

import block_quantized_gemv_q8_gb300 as qx
from .test_gpu_layer import BF16, F16, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()
    qx.lib()
    assert qx.qx_device_check() == qx.QX_OK


class Call:
    """An attention call on the tokens of a batch, or on some of them with a cache of their own."""

    def __init__(self, b, kv=None, q=None, expect=None, **mask):
        self.b, self.kv, self.q, self.mask = b, kv or b.kv, b.q if q is None else q, mask
        self.out = torch.empty_like(self.q)
        self.expected = expect if expect is not None else b.expect(b.dim ** -0.5, **mask)

    def __call__(self):
        qx.qx_attn_paged(self.kv, self.q, out=self.out, **self.mask)

    def wrong(self):
        self.out.fill_(float("nan"))

    def check(self, what):
        torch.cuda.synchronize()
        self.b.check(self.out, None, self.expected, what)


def captured(call, stream=None):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        call()
    return g


def sizes():
    """Calls whose rows are shared by several CTAs, by the split kernel and by the tensor cores, and of other sizes."""
    lens = [([1], [3000]), ([1, 1, 1], [900, 3000, 70]), ([150], [2000]), ([3, 200], [700, 1500])]
    return [Call(Batch(q, kv, 8, 2, 128, 16, (BF16, F16)[n % 2], seed=n)) for n, (q, kv) in enumerate(lens)]


def test_graphs_replayed_in_another_order_than_captured():
    """No call before the first capture, so every buffer is one of a graph's."""
    calls = sizes()
    shared = calls[0].b.kv  # all on one cache object's scratch: the later ones' caches borrow it
    for c in calls[1:]:
        c.kv._scratch = shared._scratch
    graphs = [captured(c) for c in calls]
    for order in ([3, 2, 1, 0], [1, 3, 0, 2], [0, 0, 1, 2, 3]):
        for n in order:
            calls[n].wrong()
            graphs[n].replay()
            calls[n].check(f"graph {n}")
    del graphs[0]
    for n in (2, 1):
        calls[n + 1].wrong()
        graphs[n].replay()
        calls[n + 1].check(f"graph {n + 1}, the first one gone")


def test_a_graph_of_two_calls_of_one_cache():
    b = Batch([1, 1], [3000, 500], 8, 2, 64, 32, BF16, seed=3)
    one, two = Call(b), Call(b, window=300, sinks=2)
    g = captured(lambda: (one(), two(), one()))
    for _ in range(3):
        one.wrong(), two.wrong()
        g.replay()
        one.check("first"), two.check("second")


def test_a_larger_call_after_the_capture_takes_nothing_from_the_graph():
    """Warm-up, capture and a larger call on one stream; what is allocated there afterwards stays as it is."""
    small, large = Call(Batch([1], [5000], 8, 2, 128, 16, BF16, seed=1)), Call(Batch([300, 4], [2500, 2000], 32, 2, 128, 16, BF16, seed=2))
    large.kv._scratch = small.kv._scratch
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        small()
    g = captured(small, stream=s)
    with torch.cuda.stream(s):
        large()
        large.check("larger call")
        fill = [torch.full((1 << 20,), n, dtype=torch.int32, device="cuda") for n in range(24)]
        for _ in range(3):
            small.wrong()
            g.replay()
            small.check("replay")
    torch.cuda.synchronize()
    assert all((t == n).all() for n, t in enumerate(fill))


def test_graphs_replayed_beside_each_other_and_beside_calls():
    a, b = Call(Batch([1] * 3, [4000, 3000, 20], 8, 2, 128, 16, BF16, seed=4)), Call(Batch([140], [3000], 8, 2, 128, 16, BF16, seed=5))
    c = Call(Batch([1, 2], [2500, 2600], 8, 2, 128, 16, F16, seed=6))
    b.kv._scratch = c.kv._scratch = a.kv._scratch
    ga, gb = captured(a), captured(b)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for call in (a, b, c):
        call.wrong()
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, run in zip(streams, (ga.replay, gb.replay, c)):
            with torch.cuda.stream(stream):
                run()
    for call in (a, b, c):
        call.check("beside the others")


def test_the_stream_argument_under_capture():
    b = Batch([1, 1], [3000, 500], 8, 2, 128, 16, BF16, seed=8)
    call = Call(b)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qx.qx_attn_paged(b.kv, b.q, out=call.out, stream=s)
    qx.qx_attn_paged(b.kv, b.q, stream=s)  # the stream's own scratch, not the graph's
    for _ in range(2):
        call.wrong()
        g.replay()
        call.check("replay")


@pytest.mark.parametrize("shared,tails", [(300, [5, 40, 1]), (5000, [9] * 8)])
def test_shared_prefix_in_a_graph(shared, tails):
    b = Batch([1] * len(tails), [shared + t for t in tails], 8, 2, 128, 16, BF16, seed=7)
    for n in range(1, len(tails)):
        b.keys[n][:shared], b.values[n][:shared] = b.keys[0][:shared], b.values[0][:shared]
        for i in range(-(-shared // 16)):
            m, src, dst = min(16, shared - 16 * i), int(b.table_host[0, i]), int(b.table_host[n, i])
            b.k[dst, :, :m], b.v[dst, :, :m] = b.k[src, :, :m], b.v[src, :, :m]
    expected, out = b.expect(128 ** -0.5), torch.empty_like(b.q)
    g = captured(lambda: qx.qx_attn_shared(b.kv, b.q, shared, out=out))
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        b.check(out, None, expected)


def test_calls_after_a_wait_that_ran_out():
    """They start from new scratch, and a captured graph clears its own."""
    a, b = Call(Batch([1, 1], [3000, 900], 8, 2, 128, 16, BF16, seed=9)), Call(Batch([150], [2000], 8, 2, 128, 16, BF16, seed=10))
    a(), b()
    g = captured(lambda: (a(), b()))
    # what calls that gave up could leave: counters that are not zero
    scratch = a.kv._scratch
    for _, _, buf in list(scratch._streams.values()) + [h for held in scratch._captures.values() for h in held.values()]:
        buf[:qx.QX_ATTN_COUNTER_BYTES].view(torch.int32).fill_(3)
    qx.qx_debug_timeout_probe(5_000_000)
    assert qx.qx_device_check() == qx.QX_ERR_DEVICE_TIMEOUT
    for run in (lambda: (a(), b()), g.replay, lambda: (a(), b())):
        a.wrong(), b.wrong()
        run()
        a.check("a"), b.check("b")
