"""GPU tests of what the operators between the weight products do at their
edges: what is out of range, what is not a number, what a type can hardly hold."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_q8_gb300 as qx
from . import layer_reference as ref
from .test_gpu_layer import BF16, F16, F32, Batch, check_norm, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()
    qx.lib()
    assert qx.qx_device_check() == qx.QX_OK


@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (80, 40), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src", [F32, BF16])
def test_a_position_beyond_the_rotation_is_not_written(dim, rot, interleaved, src):
    """Neither the token's key and value nor its queries, rotated elements or others."""
    b = Batch([1, 2, 1], [20, 34, 5], 4, 2, dim, 16, BF16)
    x = torch.randn(4, 8, dim, device="cuda").to(src)
    cos, sin = table_of(rot // 2, 33)  # position 33, sequence 1's last, has no row
    q_out = torch.full((4, 4, dim), 3.0, dtype=BF16, device="cuda")
    before = b.k.clone(), b.v.clone()
    qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:6], x[:, 6:], cos, sin, interleaved, q_out)
    assert qx.qx_device_check() == qx.QX_ERR_RANGE
    assert (q_out[2] == 3.0).all() and (q_out[[0, 1, 3]] != 3.0).any(-1).all()
    for cache, was in zip((b.k, b.v), before):
        same = cache.view(torch.int16) == was.view(torch.int16)
        for seq, pos in ((0, 19), (1, 32), (2, 4)):
            page, slot = int(b.table_host[seq, pos // 16]), pos % 16
            assert not same[page, :, slot].all()
            same[page, :, slot] = True
        assert same.all(), "only the good tokens' slots may change"
    # without a rotation the table does not matter
    qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:6], x[:, 6:], q_out=q_out)
    assert qx.qx_device_check() == qx.QX_OK and torch.equal(q_out, x[:, :4].to(BF16))


@pytest.mark.parametrize("limit_ns", [1_000_000, 20_000_000])
def test_a_warp_that_gives_up_takes_the_others_along(limit_ns):
    """Its unit comes before the others' limit: they have it, and leave with the one that has not."""
    got = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    qx.qx_debug_agree_probe(limit_ns, got)
    assert qx.qx_device_check() == qx.QX_ERR_DEVICE_TIMEOUT
    assert got.tolist() == [0, 1, 1, 1]
    assert qx.qx_device_check() == qx.QX_OK


def not_numbers(b, out, lse, rows):
    """Rows `rows` (of [tokens, heads]) are not a number, their log-sum-exp neither; the others are right."""
    assert qx.qx_device_check() == qx.QX_OK
    o, l, mass, top = b.expect(b.dim ** -0.5)
    got, gl = ref.f64(out), ref.f64(lse)
    assert np.isnan(got[rows]).all() and np.isnan(gl[rows]).all()
    good = ~rows
    assert (np.abs(got - o) <= ref.attention_bound(o, mass, top, b.dim, b.dtype, out.dtype))[good].all()
    assert (np.abs(gl - l) <= ref.lse_bound(l, top, b.dim))[good].all()


NAN_BATCHES = [([1], [1]), ([1], [7000]), ([1, 1], [20, 700]), ([3, 2], [50, 3000]), ([140, 1], [140, 90]), ([130], [4000])]


@pytest.mark.parametrize("dim", [64, 128, 80])
@pytest.mark.parametrize("q_lens,kv_lens", NAN_BATCHES)
def test_a_query_that_is_not_a_number(dim, q_lens, kv_lens):
    b = Batch(q_lens, kv_lens, 4, 2, dim, 16, BF16, seed=1)
    rows = np.zeros((b.T, 4), dtype=bool)
    rows[-1, 1] = rows[0, 2] = True
    lse = torch.empty((b.T, 4), device="cuda")
    clean = b.q.clone()
    b.q[torch.from_numpy(rows).cuda()] = float("nan")
    out = qx.qx_attn_paged(b.kv, b.q, lse=lse)
    b.q.copy_(clean)
    not_numbers(b, out, lse, rows)


@pytest.mark.parametrize("dim", [64, 128, 80])
@pytest.mark.parametrize("q_lens,kv_lens", NAN_BATCHES)
@pytest.mark.parametrize("which", ["one", "all"])
def test_keys_that_are_not_numbers(dim, q_lens, kv_lens, which):
    """One of the first sequence's keys, or all of them, of one key head."""
    b = Batch(q_lens, kv_lens, 4, 2, dim, 16, F16, seed=2)
    clean = b.k.clone()
    last = kv_lens[0] - q_lens[0]  # the position of its first token: every token sees the keys up to it
    for j in (range(last + 1) if which == "all" else [last]):
        b.k[int(b.table_host[0, j // 16]), 1, j % 16] = float("nan")
    rows = np.zeros((b.T, 4), dtype=bool)
    rows[:q_lens[0], 2:] = True
    lse = torch.empty((b.T, 4), device="cuda")
    out = qx.qx_attn_paged(b.kv, b.q, lse=lse)
    b.k.copy_(clean)
    not_numbers(b, out, lse, rows)


@pytest.mark.parametrize("q_lens", [[1], [3], [130]])
@pytest.mark.parametrize("dim", [64, 128, 32])
@pytest.mark.parametrize("nats", [12.75, 17.6])
def test_unlikely_keys_beside_likely_ones_in_f16(q_lens, dim, nats):
    """Every sixteenth key is a likely one whose value is zero: the output is what
    f16 holds of the others' probabilities, 2^-18.4 or 2^-25.4 of the largest."""
    n = 20000
    b = Batch(q_lens, [n], 4, 2, dim, 64, F16, seed=7)
    b.q.zero_()
    b.q[..., 0] = 8.0
    keys, values = np.zeros((n, 2, dim)), 1000.0 * (b.values[0] + 0.5)
    keys[::16, :, 0], values[::16] = nats, 0.0
    for i in range(-(-n // 64)):
        m, page = min(64, n - 64 * i), int(b.table_host[0, i])
        for cache, host in ((b.k, keys), (b.v, values)):
            cache[page, :, :m] = torch.from_numpy(host[64 * i:64 * i + m]).to(F16).transpose(0, 1).cuda()
    b.keys[0], b.values[0] = (ref.f64(torch.from_numpy(x).to(F16)) for x in (keys, values))
    for out_dtype in (F16, F32):
        lse = torch.empty((b.T, 4), device="cuda")
        out = torch.empty((b.T, 4, dim), dtype=out_dtype, device="cuda")
        qx.qx_attn_paged(b.kv, b.q, scale=0.125, out=out, lse=lse)
        b.check(out, lse, b.expect(0.125), f"{q_lens} {dim} {nats} {out_dtype}")


def test_block_norm_refuses_output_rows_that_overlap():
    y, r, w = torch.randn(4, 64, device="cuda"), torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    one, close = torch.empty(64, device="cuda").expand(4, 64), torch.empty(256, device="cuda").as_strided((4, 64), (56, 1))
    wide = torch.randn(4, 128, device="cuda")
    for bad in (dict(r_out=one), dict(r_out=close), dict(w_pre=w, x_out=one), dict(w_pre=w, x_out=close)):
        with pytest.raises(qx.QxError) as e:
            qx.qx_block_norm(y, r, **bad)
        assert e.value.status == qx.QX_ERR_SHAPE
    with pytest.raises(qx.QxError):  # in place, but in rows that lie otherwise
        qx.qx_block_norm(y, wide[:, :64], r_out=wide.view(-1)[:256].view(4, 64))
    # one row for all as an input, one row of any stride as an output
    r2, _ = qx.qx_block_norm(y, r[:1].expand(4, 64))
    assert torch.equal(r2, r[:1] + y)
    r2, _ = qx.qx_block_norm(y[:1], r[:1], r_out=torch.empty(64, device="cuda").as_strided((1, 64), (0, 1)))
    assert torch.equal(r2, r[:1] + y[:1]) and qx.qx_device_check() == qx.QX_OK


@pytest.mark.parametrize("dim", [64, 128, 80])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_lens,kv_lens,at,window,sinks", [
    ([4], [40], 38, 0, 0), ([3, 2], [700, 30], 698, 0, 0), ([3], [6000], 5998, 0, 0), ([6], [300], 257, 40, 0), ([6], [300], 2, 40, 5),
    ([140], [140], 100, 0, 0), ([140, 1], [400, 9], 300, 0, 0), ([150], [600], 430, 60, 3), ([130], [7000], 6990, 0, 0),
    ([150], [600], 430, 60, 20), ([140, 3], [400, 9], 5, 0, 0), ([64, 64], [64, 192], 63, 0, 0), ([400], [400], 399, 0, 0), ([300], [300], 17, 30, 2)])
def test_a_value_that_some_rows_do_not_see(dim, out_dtype, value, q_lens, kv_lens, at, window, sinks):
    """Rows whose mask hides the key of an infinite or undefined value are as if it were not there."""
    b = Batch(q_lens, kv_lens, 4, 2, dim, 16, BF16, seed=3)
    b.v[int(b.table_host[0, at // 16]), 0, at % 16, 5:9] = value
    lse = torch.empty((b.T, 4), device="cuda")
    out = torch.empty((b.T, 4, dim), dtype=out_dtype, device="cuda")
    qx.qx_attn_paged(b.kv, b.q, window=window, sinks=sinks, out=out, lse=lse)
    assert qx.qx_device_check() == qx.QX_OK
    o, l, mass, top = b.expect(dim ** -0.5, window, sinks)
    pos = np.arange(kv_lens[0] - q_lens[0], kv_lens[0])
    sees = (at <= pos) & ((window == 0) | (at > pos - window) | (at < sinks))
    hit = np.zeros(o.shape, dtype=bool)
    hit[:q_lens[0], :2, 5:9] = sees[:, None, None]
    got = ref.f64(out)
    assert np.array_equal(np.isfinite(got), ~hit)
    # (the reference's rows that see it hold a finite value there: they are not compared in those elements)
    err = np.where(hit, 0.0, np.abs(np.where(hit, 0.0, got) - o))
    assert (err <= ref.attention_bound(o, mass, top, dim, BF16, out_dtype)).all()
    assert (np.abs(ref.f64(lse) - l) <= ref.lse_bound(l, top, dim)).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shared,tails,q_lens,at", [(300, [3, 9], [3, 9], 302), (300, [4, 100], [8, 100], 298), (5000, [6, 6], [3, 3], 5004),
                                                    (5000, [200, 1], [200, 1], 5100)])
def test_a_value_that_some_rows_do_not_see_behind_a_prefix(dim, shared, tails, q_lens, at):
    kv_lens = [shared + t for t in tails]
    b = Batch(q_lens, kv_lens, 4, 2, dim, 16, BF16, seed=4)
    for n in range(1, len(kv_lens)):
        b.keys[n][:shared], b.values[n][:shared] = b.keys[0][:shared], b.values[0][:shared]
        for i in range(-(-shared // 16)):
            m, src, dst = min(16, shared - 16 * i), int(b.table_host[0, i]), int(b.table_host[n, i])
            b.k[dst, :, :m], b.v[dst, :, :m] = b.k[src, :, :m], b.v[src, :, :m]
    owners = range(len(kv_lens)) if at < shared else [0]
    for n in owners:
        b.v[int(b.table_host[n, at // 16]), 1, at % 16, 11] = float("nan")
    lse = torch.empty((b.T, 4), device="cuda")
    out = qx.qx_attn_shared(b.kv, b.q, shared, lse=lse)
    assert qx.qx_device_check() == qx.QX_OK
    o, l, mass, top = b.expect(dim ** -0.5)
    hit = np.zeros(o.shape, dtype=bool)
    for t, n, pos in ref.tokens(kv_lens, b.q_start_host):
        hit[t, 2:, 11] = n in owners and pos >= at
    got = ref.f64(out)
    assert np.array_equal(np.isfinite(got), ~hit)
    err = np.where(hit, 0.0, np.abs(np.where(hit, 0.0, got) - o))
    assert (err <= ref.attention_bound(o, mass, top, dim, BF16, BF16)).all()
    assert (np.abs(ref.f64(lse) - l) <= ref.lse_bound(l, top, dim)).all()


def stream_of(t):
    """The stream whose memory a tensor is, by the allocator's own account."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("number", [False, True])
def test_outputs_are_memory_of_the_calls_stream(number):
    b = Batch([1, 2], [20, 33], 4, 2, 64, 16, BF16)
    x, w = torch.randn(3, 8, 64, device="cuda"), torch.ones(512, device="cuda")
    y = x.view(3, 512)
    s = torch.cuda.Stream()
    stream = s.cuda_stream if number else s
    s.wait_stream(torch.cuda.current_stream())
    outs = [qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:6], x[:, 6:], stream=stream), qx.qx_attn_paged(b.kv, b.q, stream=stream),
            qx.qx_attn_shared(b.kv, b.q, 0, stream=stream), *qx.qx_block_norm(y, y, w_pre=w, stream=stream)]
    assert [stream_of(t) for t in outs] == [s.cuda_stream] * 5
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(outs[0], x[:, :4].to(BF16)) and torch.equal(outs[3], y + y)
    assert stream_of(qx.qx_attn_paged(b.kv, b.q)) == torch.cuda.current_stream().cuda_stream
    assert qx.qx_device_check() == qx.QX_OK


@pytest.mark.parametrize("heads", [(14, 2, 64), (12, 2, 128), (5, 1, 128), (10, 1, 64), (3, 3, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_the_same_inputs_give_the_same_bits(heads, dtype):
    """Whatever other kernels left in shared memory, where a tile's rows are not all tokens' rows."""
    hq, hkv, dim = heads
    for q_lens, kv_lens in (([150, 40], [2000, 300]), ([700], [900]), ([70] * 9, list(range(70, 700, 70)))):
        b = Batch(q_lens, kv_lens, hq, hkv, dim, 16, dtype, seed=6)
        first = None
        for n in range(8):
            y = torch.randn((2000, 4096), device="cuda") * 10.0 ** (n - 4)  # (a ring of rows in shared memory)
            qx.qx_block_norm(y, y, w_pre=torch.ones(4096, device="cuda"))
            lse = torch.empty((b.T, hq), device="cuda")
            out = qx.qx_attn_paged(b.kv, b.q, lse=lse)
            if first is None:
                first = out, lse
                b.check(out, lse, b.expect(dim ** -0.5))
            assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])


@pytest.mark.parametrize("act,res", [(BF16, F16), (F32, F16), (F16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", [(3, 1000), (1300, 2048), (2, 14336)])
def test_block_norm_of_other_pairs_of_types(act, res, rows, cols):
    g = torch.Generator(device="cuda").manual_seed(cols)
    make = lambda *shape, dt=F32: torch.empty(shape, device="cuda").normal_(generator=g).to(dt)  # noqa: E731
    y, r, gate, w1, w2 = make(rows, cols, dt=act), make(rows, cols, dt=res), make(rows, cols, dt=act), make(cols), make(cols)
    r2, x = qx.qx_block_norm(y, r, w_post=w1, gate=gate, alpha=0.7, w_pre=w2)
    assert r2.dtype == res and x.dtype == act
    some = slice(0, 40)
    check_norm(y[some], r[some], w1, gate[some], 0.7, w2, 1e-5, r2[some], x[some])
