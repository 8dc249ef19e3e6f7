"""GPU tests of shared prefixes whose prefix and tails are two kernels beside
each other and a third that joins them: long prefixes, or many rows behind
shorter ones, for few tokens a sequence."""
import pytest
import torch

import block_quantized_gemv_q8_gb300 as qx
from . import layer_reference as ref
from .test_gpu_layer import BF16, F16, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()
    qx.lib()
    assert qx.qx_device_check() == qx.QX_OK


def shared_batch(shared, tails, q_lens, hq, hkv, dim, page, dtype, seed):
    """Sequences that begin with the first one's keys, whole pages of them in common."""
    b = Batch(q_lens, [shared + t for t in tails], hq, hkv, dim, page, dtype, seed=seed)
    for n in range(1, len(tails)):
        b.keys[n][:shared], b.values[n][:shared] = b.keys[0][:shared], b.values[0][:shared]
        i, m = shared // page, shared % page
        if m:
            src, dst = int(b.table_host[0, i]), int(b.table_host[n, i])
            b.k[dst, :, :m], b.v[dst, :, :m] = b.k[src, :, :m], b.v[src, :, :m]
        b.table_host[n, :i] = b.table_host[0, :i]
    b.table.copy_(torch.from_numpy(b.table_host))
    return b


# prefix blocks shared out evenly (from 12 of 128 keys on) or not; group sizes; sequences beyond a tile
CASES = [(5000, 8, (32, 8, 128), 64, BF16), (4200, 3, (14, 2, 64), 16, F16), (6000, 40, (16, 1, 64), 32, BF16),
         (1000, 256, (32, 8, 128), 16, BF16), (1300, 300, (14, 14, 64), 64, F16), (8200, 5, (12, 2, 128), 256, BF16)]


@pytest.mark.parametrize("shared,seqs,heads,page,dtype", CASES)
def test_prefix_and_tails_beside_each_other(shared, seqs, heads, page, dtype):
    """Appends and attention in turn, back to back: each call sees the append before it, and only that."""
    hq, hkv, dim = heads
    tails = [1 + (37 * n) % 150 for n in range(seqs)]
    b = shared_batch(shared, tails, [1] * seqs, hq, hkv, dim, page, dtype, seed=shared)
    g = torch.Generator(device="cuda").manual_seed(5)
    steps = []
    for _ in range(2):  # two variants of every sequence's last key and value
        x = torch.empty((seqs, hq + 2 * hkv, dim), device="cuda").normal_(generator=g).to(dtype)
        for n in range(seqs):
            b.keys[n][-1], b.values[n][-1] = ref.f64(x[n, hq:hq + hkv]), ref.f64(x[n, hq + hkv:])
        steps.append((x, b.expect(dim ** -0.5, q=x[:, :hq])))
    outs, lses = [], []
    for i in range(12):
        x, _ = steps[i % 2]
        q = qx.qx_rope_append(b.kv, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])
        lse = torch.empty((seqs, hq), device="cuda")
        outs.append(qx.qx_attn_shared(b.kv, q, shared, lse=lse))
        lses.append(lse)
    for i in range(12):
        b.check(outs[i], lses[i], steps[i % 2][1], f"call {i}")
        assert torch.equal(outs[i].view(torch.int16), outs[i % 2].view(torch.int16)) and torch.equal(lses[i], lses[i % 2])


@pytest.mark.parametrize("heads", [(32, 8, 128), (14, 2, 64)])
@pytest.mark.parametrize("shared,tails,q_lens", [
    (5000, [0, 3, 200, 1, 9], [1, 5, 0, 1, 3]),      # an idle sequence, tokens inside the prefix, no tail at all
    (1000, [n % 7 for n in range(200)], [n % 3 for n in range(200)])])
def test_idle_sequences_and_tokens_inside_the_prefix(heads, shared, tails, q_lens):
    hq, hkv, dim = heads
    b = shared_batch(shared, tails, q_lens, hq, hkv, dim, 16, BF16, seed=9)
    expected = b.expect(dim ** -0.5)
    first = None
    for _ in range(4):
        lse = torch.full((b.T, hq), 7.0, device="cuda")
        out = torch.full((b.T, hq, dim), float("nan"), device="cuda")
        qx.qx_attn_shared(b.kv, b.q, shared, out=out, lse=lse)
        b.check(out, lse, expected)
        assert first is None or torch.equal(out, first)
        first = out


def test_prefix_and_tails_of_two_streams():
    """Each stream's scratch is its own, beside each other and in any order."""
    a = shared_batch(5000, [9, 40, 3], [1] * 3, 32, 8, 128, 64, BF16, seed=1)
    b = shared_batch(1000, list(range(1, 241)), [1] * 240, 32, 8, 128, 16, BF16, seed=2)
    want = [x.expect(128 ** -0.5) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[qx.qx_attn_shared(x.kv, x.q, n, stream=s) for x, n, s in ((a, 5000, streams[0]), (b, 1000, streams[1]))] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in outs:
        for x, out, expected in zip((a, b), pair, want):
            x.check(out, None, expected)
