"""GPU tests of the operators between the weight products: rotation and append
to the paged cache, attention over it, and the norms around a block, each
against a plain 64-bit implementation (tests/layer_reference.py) within bounds
that follow from the roundings the header states."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_q8_gb300 as qx
from . import layer_reference as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()
    qx.lib()
    assert qx.qx_device_check() == qx.QX_OK


def table_of(angles, n_pos):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(angles) / max(1, angles))
    return torch.from_numpy(np.cos(a)).float().cuda(), torch.from_numpy(np.sin(a)).float().cuda()


class Batch:
    """A paged cache with random pages; what no sequence has written holds NaN,
    and table entries past a sequence's last page point outside the cache."""

    def __init__(self, q_lens, kv_lens, hq, hkv, dim, page=16, dtype=BF16, layout="hnd", seed=0, std=1.0, spare_pages=3):
        rng = np.random.default_rng(seed)
        self.q_lens, self.kv_lens, self.hq, self.hkv, self.dim, self.page, self.dtype = q_lens, kv_lens, hq, hkv, dim, page, dtype
        need = [-(-kv // page) for kv in kv_lens]
        n_pages = sum(need) + spare_pages
        order = rng.permutation(n_pages).astype(np.int32)
        table = np.full((len(kv_lens), max(need + [1]) + 1), n_pages + 7, dtype=np.int32)
        shape = (n_pages, hkv, page, dim) if layout == "hnd" else (n_pages, page, hkv, dim)
        k, v = (torch.full(shape, float("nan"), dtype=dtype) for _ in range(2))
        if layout != "hnd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        self.keys, self.values, at = [], [], 0
        for b, kv in enumerate(kv_lens):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            kk, vv = (torch.from_numpy(rng.standard_normal((kv, hkv, dim)) * std).to(dtype) for _ in range(2))
            self.keys.append(ref.f64(kk))
            self.values.append(ref.f64(vv))
            for i in range(need[b]):
                n = min(page, kv - i * page)
                k[int(table[b, i]), :, :n] = kk[i * page:i * page + n].transpose(0, 1)
                v[int(table[b, i]), :, :n] = vv[i * page:i * page + n].transpose(0, 1)
        strided = (lambda t: t.cuda()) if layout == "hnd" else (lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2))
        self.k, self.v = strided(k), strided(v)
        self.table_host = table
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        self.q_start_host = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.q_start = torch.from_numpy(self.q_start_host).cuda()
        self.T = int(self.q_start_host[-1])
        self.q = torch.from_numpy(rng.standard_normal((self.T, hq, dim))).to(dtype).cuda()
        self.kv = qx.PagedKV(self.k, self.v, self.table, self.kv_len, self.q_start)

    def expect(self, scale, window=0, sinks=0, q=None):
        q = ref.f64(self.q if q is None else q)
        parts = []
        for b, kv in enumerate(self.kv_lens):
            t0, t1 = self.q_start_host[b], self.q_start_host[b + 1]
            pos = np.arange(kv - (t1 - t0), kv)
            parts.append(ref.attention(q[t0:t1], self.keys[b], self.values[b], pos, scale, window, sinks))
        return [np.concatenate([p[i] for p in parts]) for i in range(4)]

    def check(self, out, lse, expected, what=""):
        o, l, mass, top = expected
        assert qx.qx_device_check() == qx.QX_OK
        got = ref.f64(out)
        assert np.isfinite(got).all(), f"{what}: {np.argwhere(~np.isfinite(got))[:4]}"
        err, tol = np.abs(got - o), ref.attention_bound(o, mass, top, self.dim, self.dtype, out.dtype)
        assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.3g} of the bound at {np.unravel_index(np.argmax(err / tol), err.shape)}"
        if lse is not None:
            gl = ref.f64(lse)
            seen = np.isfinite(l)
            assert np.array_equal(gl == -np.inf, ~seen), what
            assert (np.abs(gl[seen] - l[seen]) <= ref.lse_bound(l, top, self.dim)[seen]).all(), what


HEADS = [(32, 8, 128), (14, 2, 64), (3, 3, 64), (16, 1, 64), (12, 2, 128), (4, 2, 80), (2, 1, 256), (2, 2, 8), (40, 1, 128)]
MASKS = [(0, 0), (40, 4), (100, 0), (1, 0), (17, 33), (300, 130)]
BATCHES = [
    ([1], [1]), ([1], [2]), ([1], [300]),
    ([1, 1, 1], [17, 64, 333]),
    ([1, 1, 1, 1], [0, 5, 0, 129]),                # padding sequences: no key
    ([5, 1, 130, 0, 33], [5, 77, 200, 40, 20]),    # an idle sequence, and one with 13 padding tokens
    ([64, 64], [64, 192]),
    ([3, 4, 2], [700, 3, 1500]),
    ([257], [400]),
]


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_attention_shapes(heads, batch):
    q_lens, kv_lens = BATCHES[batch]
    hq, hkv, dim = heads
    for i, (window, sinks) in enumerate(MASKS):
        page, dtype = (16, 64, 32, 128, 256, 16)[i], (BF16, F16)[(i + batch) % 2]
        b = Batch(q_lens, kv_lens, hq, hkv, dim, page, dtype, ("hnd", "nhd")[(i + batch) % 2], seed=100 * batch + i)
        lse = torch.full((b.T, hq), 7.0, device="cuda")
        out = torch.full((b.T, hq, dim), float("nan"), dtype=(dtype, F32)[i % 2], device="cuda")
        qx.qx_attn_paged(b.kv, b.q, window=window, sinks=sinks, out=out, lse=lse)
        b.check(out, lse, b.expect(dim ** -0.5, window, sinks), f"heads {heads} page {page} window {window} sinks {sinks}")


@pytest.mark.parametrize("heads", [(32, 8, 128), (28, 4, 64)])
@pytest.mark.parametrize("window,sinks", [(100, 4), (150, 200), (0, 0), (64, 0)])
def test_prefill_of_more_tiles_than_the_gpu_holds(heads, window, sinks):
    """Each SM takes several tile pairs one after another."""
    hq, hkv, dim = heads
    q_lens = [1700, 3, 900, 40] if window else [700, 300, 1, 500]
    kv_lens = [1700, 90, 1500, 300] if window else [700, 400, 60, 500]
    if not window:
        hq, hkv = 8 * hkv * 4, 4 * hkv
    b = Batch(q_lens, kv_lens, hq, hkv, dim, 16, BF16, seed=12)
    lse = torch.empty((b.T, hq), device="cuda")
    out = qx.qx_attn_paged(b.kv, b.q, window=window, sinks=sinks, lse=lse)
    b.check(out, lse, b.expect(dim ** -0.5, window, sinks), f"{heads} window {window}")


@pytest.mark.parametrize("heads", [(32, 8, 128), (14, 2, 64), (6, 6, 64), (16, 1, 128)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([100, 0, 37, 200, 130], [4000, 60, 37, 2100, 90]),  # an idle sequence; one with 40 padding tokens
    ([129], [6000]), ([33] * 20, list(range(33, 1733, 85))), ([400, 300], [3, 2000])])
def test_few_pairs_over_long_contexts(heads, q_lens, kv_lens):
    """Key blocks shared out over the SMs: rows in several parts, in one, and in none."""
    hq, hkv, dim = heads
    for i, (window, sinks) in enumerate([(0, 0), (1800, 5), (1500, 0)]):
        b = Batch(q_lens, kv_lens, hq, hkv, dim, (16, 64, 256)[i], (BF16, F16, BF16)[i], ("hnd", "nhd", "hnd")[i], seed=20 + i)
        lse = torch.full((b.T, hq), 7.0, device="cuda")
        out = torch.full((b.T, hq, dim), float("nan"), dtype=(b.dtype, F32, b.dtype)[i], device="cuda")
        exp = b.expect(dim ** -0.5, window, sinks)
        for _ in range(2):
            qx.qx_attn_paged(b.kv, b.q, window=window, sinks=sinks, out=out, lse=lse)
            b.check(out, lse, exp, f"{heads} window {window} sinks {sinks}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [5000]), ([300], [2500]), ([1, 1, 200], [3000, 1, 900])])
@pytest.mark.parametrize("std", [0.0, 1.0, 30.0])
def test_attention_score_ranges(dtype, q_lens, kv_lens, std):
    """Equal scores, ordinary ones, and ones so far apart that a running maximum leaps."""
    b = Batch(q_lens, kv_lens, 4, 1, 128, 64, dtype, seed=5, std=std)
    lse = torch.empty((b.T, 4), device="cuda")
    out = qx.qx_attn_paged(b.kv, b.q, lse=lse)
    b.check(out, lse, b.expect(128 ** -0.5), f"std {std}")
    out = qx.qx_attn_paged(b.kv, b.q, scale=-0.3, window=777, sinks=9, lse=lse)
    b.check(out, lse, b.expect(-0.3, 777, 9), f"std {std}, negative scale")


@pytest.mark.parametrize("dim", [64, 128, 32])
def test_rising_scores(dim):
    """Each key scores higher than all before it: every block moves the maximum."""
    b = Batch([1, 150], [2000, 1100], 2, 1, dim, 16, F16, seed=9)
    for n, kv in enumerate(b.kv_lens):
        up = np.zeros((kv, 1, dim))
        up[:, 0, 0] = np.linspace(-60, 60, kv)
        up = torch.from_numpy(up).to(F16)
        b.keys[n] = ref.f64(up)
        for i in range(-(-kv // 16)):
            m = min(16, kv - 16 * i)
            b.k[int(b.table_host[n, i]), :, :m] = up[16 * i:16 * i + m].transpose(0, 1).cuda()
    b.q.fill_(0)
    b.q[..., 0] = 4.0
    for sign in (1.0, -1.0):
        lse = torch.empty((b.T, 2), device="cuda")
        out = qx.qx_attn_paged(b.kv, b.q, scale=sign, lse=lse)
        b.check(out, lse, b.expect(sign), f"sign {sign}")


@pytest.mark.parametrize("heads", [(32, 8, 128), (14, 2, 64)])
@pytest.mark.parametrize("page,sinks", [(16, 16), (16, 1), (16, 17), (32, 5), (64, 64), (64, 3), (64, 65), (128, 7)])
def test_first_keys_beside_a_window(heads, page, sinks):
    """First keys that share the window's page, its block or neither, and pages
    between them and the window that hold NaN and are given back."""
    hq, hkv, dim = heads
    for n, (q_lens, kv_lens, window) in enumerate([([150, 2], [700, 300], 90), ([200], [200], 70), ([130, 40], [131, 200], 1),
                                                   ([140], [333], 150), ([129], [900], 640)]):
        b = Batch(q_lens, kv_lens, hq, hkv, dim, page, (BF16, F16)[n % 2], seed=40 + n)
        for s, (m, kv) in enumerate(zip(q_lens, kv_lens)):
            first = max(0, kv - m + 1 - window)
            for i in range(-(-kv // page)):
                if page * i >= sinks and page * (i + 1) <= first:
                    b.k[int(b.table_host[s, i])] = float("nan")
                    b.v[int(b.table_host[s, i])] = float("nan")
                    b.table[s, i] = -1
        lse = torch.empty((b.T, hq), device="cuda")
        out = qx.qx_attn_paged(b.kv, b.q, window=window, sinks=sinks, lse=lse)
        b.check(out, lse, b.expect(dim ** -0.5, window, sinks), f"{heads} page {page} sinks {sinks} window {window} {q_lens}")


@pytest.mark.parametrize("heads", [(32, 8, 128), (14, 2, 64), (2, 2, 80)])
def test_pages_outside_the_window_may_be_given_back(heads):
    hq, hkv, dim = heads
    for q_lens, kv_lens in (([1, 1], [1000, 700]), ([140, 3], [1000, 700])):
        b = Batch(q_lens, kv_lens, hq, hkv, dim, 16, BF16, seed=3)
        window, sinks = 200, 20
        for n, (m, kv) in enumerate(zip(q_lens, kv_lens)):
            first = max(0, kv - m + 1 - window)  # the first key that the first token's window holds
            for i in range(-(-kv // 16)):
                if 16 * i >= sinks and 16 * (i + 1) <= first:
                    b.k[int(b.table_host[n, i])] = float("nan")
                    b.v[int(b.table_host[n, i])] = float("nan")
                    b.table[n, i] = -1
        out = qx.qx_attn_paged(b.kv, b.q, window=window, sinks=sinks)
        b.check(out, None, b.expect(dim ** -0.5, window, sinks), f"{heads} {q_lens}")


@pytest.mark.parametrize("heads", [(32, 8, 128), (14, 2, 64), (16, 1, 64), (2, 2, 80)])
@pytest.mark.parametrize("shared,tails,q_lens", [
    (100, [1, 30, 7], [1, 1, 1]), (512, [1, 2, 3, 300], [1, 1, 1, 1]), (1000, list(range(1, 41)), [1] * 40),
    (0, [5, 9], [1, 1]), (77, [0, 3], [1, 1]), (640, [150, 20, 60], [150, 5, 60]), (3000, [4], [4]),
    (50, [3, 10], [20, 10])])
def test_shared_prefix(heads, shared, tails, q_lens):
    hq, hkv, dim = heads
    kv = [shared + t for t in tails]
    for page, dtype in ((16, BF16), (64, F16)):
        b = Batch(q_lens, kv, hq, hkv, dim, page, dtype, seed=11)
        for n in range(1, len(kv)):  # the first sequence's prefix in all
            b.keys[n][:shared], b.values[n][:shared] = b.keys[0][:shared], b.values[0][:shared]
            for i in range(-(-shared // page)):
                m = min(page, shared - i * page)
                src, dst = int(b.table_host[0, i]), int(b.table_host[n, i])
                b.k[dst, :, :m], b.v[dst, :, :m] = b.k[src, :, :m], b.v[src, :, :m]
        lse = torch.empty((b.T, hq), device="cuda")
        out = qx.qx_attn_shared(b.kv, b.q, shared, lse=lse)
        exp = b.expect(dim ** -0.5)
        b.check(out, lse, exp, f"{heads} shared {shared} page {page}")
        # whole pages of the prefix in common: entries of the others' tables
        # that lead to it are the first one's
        whole = shared // page
        b.table[1:, :whole] = b.table[:1, :whole]
        out = qx.qx_attn_shared(b.kv, b.q, shared, lse=lse, out=torch.empty((b.T, hq, dim), device="cuda"))
        b.check(out, lse, exp, f"{heads} shared {shared} page {page}, pages in common")


def test_attention_is_reproducible_and_leaves_its_scratch_fit():
    for q_lens, kv_lens in (([1] * 5, [3000, 40, 900, 2000, 1]), ([200, 1, 30], [2000, 10, 3000])):
        b = Batch(q_lens, kv_lens, 8, 2, 128, 32, BF16, seed=2)
        first = qx.qx_attn_paged(b.kv, b.q).clone()
        for _ in range(20):
            assert torch.equal(qx.qx_attn_paged(b.kv, b.q).view(torch.int16), first.view(torch.int16))
        # another shape on the same scratch in between
        qx.qx_attn_paged(b.kv, b.q, window=50)
        assert torch.equal(qx.qx_attn_paged(b.kv, b.q).view(torch.int16), first.view(torch.int16))
        b.check(first, None, b.expect(128 ** -0.5))


def test_strided_queries_and_other_streams():
    b = Batch([1, 40, 1], [100, 90, 513], 14, 2, 64, 16, F16, seed=4)
    wide = torch.zeros((b.T, 18, 64), dtype=F16, device="cuda")
    wide[:, :14] = b.q
    exp = b.expect(64 ** -0.5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [qx.qx_attn_paged(b.kv, wide[:, :14], stream=s, out=torch.empty_like(b.q)) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    for o in outs:
        b.check(o, None, exp)
    with torch.cuda.stream(streams[0]):
        o = qx.qx_attn_paged(b.kv, wide[:, :14])
    torch.cuda.synchronize()
    b.check(o, None, exp)


def test_captured_step_follows_the_lengths():
    """Append and attention captured once, replayed while kv_len grows in place."""
    b = Batch([1, 1], [40, 71], 8, 2, 64, 16, BF16, seed=6)
    cos, sin = table_of(32, 200)
    new = torch.randn(2, 12, 64, device="cuda")
    q_rot = torch.empty((2, 8, 64), dtype=BF16, device="cuda")
    out = torch.empty_like(q_rot)

    def step():
        qx.qx_rope_append(b.kv, new[:, :8], new[:, 8:10], new[:, 10:], cos, sin, q_out=q_rot)
        qx.qx_attn_paged(b.kv, q_rot, out=out)

    step()  # also writes its key over each sequence's last one
    torch.cuda.synchronize()
    for n in range(2):
        page, slot = int(b.table_host[n, (b.kv_lens[n] - 1) // 16]), (b.kv_lens[n] - 1) % 16
        b.keys[n][-1], b.values[n][-1] = ref.f64(b.k[page, :, slot]), ref.f64(b.v[page, :, slot])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        kv = [int(x) + 1 for x in b.kv_len.cpu()]
        for n in range(2):  # the step's key goes to position kv - 1
            page = (kv[n] - 1) // 16
            if b.table_host[n, page] >= b.k.shape[0]:
                spare = sorted(set(range(b.k.shape[0])) - set(b.table_host.reshape(-1).tolist()))
                b.table_host[n, page] = spare[0]
        b.table.copy_(torch.from_numpy(b.table_host))
        b.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        new.normal_()
        g.replay()
        torch.cuda.synchronize()
        for n in range(2):
            c, s = ref.f64(cos)[kv[n] - 1], ref.f64(sin)[kv[n] - 1]
            want = ref.rotate(ref.f64(new[n, 8:10]), c, s, False)
            page, slot = int(b.table_host[n, (kv[n] - 1) // 16]), (kv[n] - 1) % 16
            got = ref.f64(b.k[page, :, slot])
            assert (np.abs(got - want) <= 2.0 ** -7 * (np.abs(want) + 1)).all()
            have = max(0, len(b.keys[n]))
            b.keys[n] = np.concatenate([b.keys[n][:kv[n] - 1], got[None]])
            b.values[n] = np.concatenate([b.values[n][:kv[n] - 1], ref.f64(b.v[page, :, slot])[None]])
            assert have <= kv[n]
        b.kv_lens = kv
        b.check(out, None, b.expect(64 ** -0.5, q=q_rot))


def test_attention_over_a_cache_of_more_than_2_31_elements():
    n_pages, page, hkv, dim = 70000, 256, 1, 128  # 2.29e9 elements, 4.6 GB each
    k, v = (torch.empty((n_pages, hkv, page, dim), dtype=BF16, device="cuda") for _ in range(2))
    use = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in use[0].tolist():
        k[i].normal_(generator=g)
        v[i].normal_(generator=g)
    for m in (1, 90):
        kv = qx.PagedKV(k, v, use, torch.tensor([700], dtype=torch.int32, device="cuda"),
                        torch.tensor([0, m], dtype=torch.int32, device="cuda"))
        q = torch.randn((m, 4, dim), device="cuda").to(BF16)
        out = qx.qx_attn_paged(kv, q)
        kk, vv = (ref.f64(c[use[0].long(), 0].reshape(-1, 1, dim)[:700]) for c in (k, v))
        o, _, mass, top = ref.attention(ref.f64(q), kk, vv, np.arange(700 - m, 700), dim ** -0.5)
        assert qx.qx_device_check() == qx.QX_OK
        assert (np.abs(ref.f64(out) - o) <= ref.attention_bound(o, mass, top, dim, BF16, BF16)).all()


@pytest.mark.parametrize("heads", [(32, 8, 128), (14, 2, 64), (2, 2, 80)])
@pytest.mark.parametrize("q_lens", [[1, 1], [150, 2]])
def test_pages_and_lengths_out_of_range_are_reported(heads, q_lens):
    hq, hkv, dim = heads
    b = Batch(q_lens, [500, 300], hq, hkv, dim, 16, BF16, seed=8)
    good = b.expect(dim ** -0.5)
    b.table[1, 2] = b.k.shape[0]  # one past the last page
    out = qx.qx_attn_paged(b.kv, b.q)
    assert qx.qx_device_check() == qx.QX_ERR_RANGE
    assert qx.qx_device_check() == qx.QX_OK
    n = int(b.q_start_host[1])  # the other sequence's rows are right
    o, _, mass, top = good
    assert (np.abs(ref.f64(out[:n]) - o[:n]) <= ref.attention_bound(o, mass, top, dim, BF16, BF16)[:n]).all()
    b.table.copy_(torch.from_numpy(b.table_host))
    b.kv_len[1] = 16 * b.table.shape[1] + 1  # longer than its row of the table
    qx.qx_attn_paged(b.kv, b.q)
    assert qx.qx_device_check() == qx.QX_ERR_RANGE
    b.kv_len[1] = 300
    out = qx.qx_attn_paged(b.kv, b.q)
    b.check(out, None, good)


def test_attention_takes_no_tokens_and_leaves_foreign_rows():
    b = Batch([2, 1], [10, 20], 4, 2, 64, 16, BF16)
    assert qx.qx_attn_paged(b.kv, b.q[:0]).shape == (0, 4, 64)
    more = torch.cat([b.q, b.q[:2]])  # two rows that belong to no sequence
    out = torch.full((5, 4, 64), 3.0, dtype=BF16, device="cuda")
    qx.qx_attn_paged(b.kv, more, out=out)
    b.check(out[:3], None, b.expect(0.125))
    assert (out[3:] == 3.0).all()


# ---------------------------------------------------------------------------
# rotation and append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("src", [F32, F16, BF16])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,dim,rot", [(32, 8, 128, 128), (14, 2, 64, 64), (4, 1, 80, 40), (1, 1, 8, 8), (2, 2, 256, 64),
                                            (3, 3, 96, 0), (0, 2, 64, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append(src, dtype, hq, hkv, dim, rot, interleaved):
    for n, (q_lens, kv_lens) in enumerate([([1], [1]), ([1, 1, 1], [40, 0, 17]), ([20, 0, 3, 9], [25, 30, 3, 5]), ([300], [300])]):
        layout, page = ("hnd", "nhd")[n % 2], (16, 32)[n % 2]
        b = Batch(q_lens, kv_lens, max(hq, hkv), hkv, dim, page, dtype, layout, seed=n)
        rng = np.random.default_rng(n)
        x = torch.from_numpy(rng.standard_normal((b.T, hq + 2 * hkv, dim))).to(src).cuda()
        cos, sin = table_of(rot // 2, 320) if rot else (None, None)
        before = b.k.clone(), b.v.clone()
        q_out = torch.full((b.T, hq, dim), float("nan"), dtype=dtype, device="cuda") if hq else None
        got_q = qx.qx_rope_append(b.kv, x[:, :hq] if hq else None, x[:, hq:hq + hkv], x[:, hq + hkv:], cos, sin, interleaved, q_out)
        assert qx.qx_device_check() == qx.QX_OK
        want_k, want_v = ref.f64(before[0]), ref.f64(before[1])
        xs, u = ref.f64(x), ref.ROUND[dtype]
        # one rounding to the cache's type, and two f32 products of at most |a| + |b| with their sum
        bound = lambda w: u * np.abs(w) + 2.0 ** -22 * (np.abs(xs).max() * 2) + 2.0 ** -25  # noqa: E731
        for t, s, pos in ref.tokens(kv_lens, b.q_start_host):
            turn = lambda z: ref.rotate(z, ref.f64(cos)[pos], ref.f64(sin)[pos], interleaved) if rot else z  # noqa: E731
            if hq:
                want = np.zeros((hq, dim)) if pos < 0 else turn(xs[t, :hq])
                assert (np.abs(ref.f64(got_q[t]) - want) <= bound(want)).all(), (t, pos)
            if pos >= 0:
                at, slot = int(b.table_host[s, pos // page]), pos % page
                want_k[at, :, slot], want_v[at, :, slot] = turn(xs[t, hq:hq + hkv]), xs[t, hq + hkv:]
        for cache, want in ((b.k, want_k), (b.v, want_v)):
            got = ref.f64(cache)
            assert np.array_equal(np.isnan(got), np.isnan(want))
            ok = ~np.isnan(want)
            assert (np.abs(got[ok] - want[ok]) <= bound(want[ok])).all()


def test_rope_append_of_one_token_with_any_token_stride():
    """One token's rows may be a view whose token stride is no multiple of 8."""
    b = Batch([1], [30], 4, 2, 64, 16, F16)
    base = torch.randn(9 * 512, device="cuda")
    x = torch.as_strided(base, (1, 8, 64), (7, 64, 1))
    cos, sin = table_of(32, 64)
    q = qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:6], x[:, 6:], cos, sin)
    assert qx.qx_device_check() == qx.QX_OK
    want = ref.rotate(ref.f64(base[:256].view(4, 64)), ref.f64(cos)[29], ref.f64(sin)[29], False)
    assert (np.abs(ref.f64(q[0]) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -20).all()
    got = ref.f64(b.v[int(b.table_host[0, 1]), :, 13])
    assert (np.abs(got - ref.f64(base[384:512].view(2, 64))) <= 2.0 ** -11 * np.abs(got) + 2.0 ** -20).all()


def test_rope_append_reports_what_is_out_of_range():
    b = Batch([1, 1], [20, 33], 4, 2, 64, 16, BF16)
    x = torch.randn(2, 8, 64, device="cuda")
    cos, sin = table_of(32, 33)
    args = (b.kv, x[:, :4], x[:, 4:6], x[:, 6:])
    qx.qx_rope_append(*args, cos, sin)
    assert qx.qx_device_check() == qx.QX_OK
    qx.qx_rope_append(*args, cos[:32].contiguous(), sin[:32].contiguous())  # position 32 has no row
    assert qx.qx_device_check() == qx.QX_ERR_RANGE
    b.table[0, 1] = -5
    before = b.k.clone()
    qx.qx_rope_append(*args, cos, sin)
    assert qx.qx_device_check() == qx.QX_ERR_RANGE
    page, slot = int(b.table_host[1, 2]), 0
    same = b.k.view(torch.int16) == before.view(torch.int16)
    same[page, :, slot] = True
    assert same.all(), "only the good token's slot may change"
    b.kv_len[0] = 16 * b.table.shape[1] + 1
    qx.qx_rope_append(*args, cos, sin)
    assert qx.qx_device_check() == qx.QX_ERR_RANGE


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("act,res", [(F32, F32), (BF16, F32), (F16, F32), (BF16, BF16), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (1, 1), (3, 7), (77, 896), (5, 1000), (2, 14336), (4, 32768), (2, 32767), (3, 8200),
                                       (1, 9001), (300, 64)])
def test_block_norm(act, res, rows, cols):
    rng = np.random.default_rng(cols)
    make = lambda *shape, dt=F32, std=1.0: torch.from_numpy(rng.standard_normal(shape) * std).to(dt).cuda()  # noqa: E731
    y, r = make(rows, cols, dt=act, std=0.5), make(rows, cols, dt=res, std=2.0)
    w1, w2 = make(cols), make(cols)
    gates = {"none": None, "channel": make(cols, dt=act), "row": make(rows, cols, dt=act)}
    for post, gname, pre, alpha in ((True, "none", True, 1.0), (True, "row", True, 0.3), (False, "channel", True, -1.5),
                                    (True, "channel", False, 1.0), (False, "none", True, 0.0)):
        gate = gates[gname]
        r2, x = qx.qx_block_norm(y, r, w_post=w1 if post else None, gate=gate, alpha=alpha, w_pre=w2 if pre else None, eps=1e-6)
        check_norm(y, r, w1 if post else None, gate, alpha, w2 if pre else None, 1e-6, r2, x)


@pytest.mark.parametrize("act,res", [(F32, F32), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("rows,cols", [(3000, 4096), (700, 8192), (6000, 96), (2500, 1000), (1300, 4104), (2500, 1544)])
def test_block_norm_of_many_rows(act, res, rows, cols):
    """More rows than the GPU holds at a time, in every combination of operands."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    make = lambda *shape, dt=F32, std=1.0: torch.empty(shape, dtype=dt, device="cuda").normal_(0, std, generator=g)  # noqa: E731
    y, r, w1, w2 = make(rows, cols, dt=act), make(rows, cols, dt=res, std=2.0), make(cols), make(cols)
    some = torch.randperm(rows, generator=g, device="cuda")[:40]
    for gate in (None, make(cols, dt=act), make(rows, cols, dt=act)):
        for post, pre in ((w1, w2), (None, w2), (w1, None)):
            r2, x = qx.qx_block_norm(y, r, w_post=post, gate=gate, alpha=0.7, w_pre=pre)
            part = gate if gate is None or gate.dim() == 1 else gate[some]
            check_norm(y[some], r[some], post, part, 0.7, pre, 1e-5, r2[some], None if pre is None else x[some])
    r2, x = qx.qx_block_norm(None, r, w_pre=w2, r_out=torch.empty_like(r), x_out=torch.empty(rows, cols, dtype=act, device="cuda"))
    check_norm(None, r[some], None, None, 1.0, w2, 1e-5, r2[some], x[some])
    assert qx.qx_device_check() == qx.QX_OK


def check_norm(y, r, w_post, gate, alpha, w_pre, eps, r2, x):
    torch.cuda.synchronize()
    host = [None if t is None else ref.f64(t) for t in (y, r, w_post, gate, w_pre)]
    want_r, want_x, size = ref.block_norm(host[0], host[1], host[2], host[3], np.float64(np.float32(alpha)), host[4], np.float64(np.float32(eps)))
    # f32 arithmetic: a sum of at most 2^15 squares over a CTA (each partial
    # sum's rounding, at most 48 of them one after another), a root, a
    # division and a few products: 64 roundings bound it
    f32 = 64 * 2.0 ** -24
    assert (np.abs(ref.f64(r2) - want_r) <= ref.ROUND[r2.dtype] * np.abs(want_r) + f32 * size + 2.0 ** -25).all()
    if w_pre is not None:
        inv = np.abs(host[4]) / np.sqrt((want_r ** 2).mean(1, keepdims=True) + eps)
        assert (np.abs(ref.f64(x) - want_x) <= ref.ROUND[x.dtype] * np.abs(want_x) + 2 * f32 * (size * inv) + 2.0 ** -25).all()


def test_block_norm_strides_aliases_and_first_norm():
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((9, 2500), device="cuda", generator=g)
    w = torch.randn(1200, device="cuda", generator=g)
    for first in (0, 8, 3):  # aligned and odd starts of strided rows
        y, r = wide[:, first:first + 1200], wide[:, 1200 + first:2400 + first]
        r2, x = qx.qx_block_norm(y, r, w_post=w, w_pre=w, alpha=0.5)
        check_norm(y, r, w, None, 0.5, w, 1e-5, r2, x)
    # the residual and the block's output overwritten in place
    y, r = wide[:, :1200].contiguous(), wide[:, 1200:2400].contiguous()
    y0, r0 = y.clone(), r.clone()
    r2, x = qx.qx_block_norm(y, r, w_post=w, w_pre=w, r_out=r, x_out=y)
    assert r2.data_ptr() == r.data_ptr() and x.data_ptr() == y.data_ptr()
    check_norm(y0, r0, w, None, 1.0, w, 1e-5, r2, x)
    # the first norm of a stack: no block before it
    r2, x = qx.qx_block_norm(None, r0, w_pre=w)
    assert r2.data_ptr() == r0.data_ptr()
    check_norm(None, r0, None, None, 1.0, w, 1e-5, r0, x)
    # zero rows, and rows of zeros
    r2, x = qx.qx_block_norm(y0[:0], r0[:0], w_pre=w)
    assert x.shape == (0, 1200)
    z = torch.zeros((2, 1200), device="cuda")
    r2, x = qx.qx_block_norm(z, z, w_post=w, w_pre=w)
    assert (r2 == 0).all() and (x == 0).all()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_binding_refuses_what_it_cannot_serve():
    b = Batch([1, 1], [20, 33], 4, 2, 64, 16, BF16)
    x = torch.randn(2, 8, 64, device="cuda")
    cos, sin = table_of(32, 40)
    with pytest.raises(TypeError):
        qx.qx_attn_paged(b.kv, b.q.float())
    with pytest.raises(ValueError):
        qx.qx_attn_paged(b.kv, b.q.cpu())
    with pytest.raises(ValueError):
        qx.qx_attn_paged(b.kv, b.q[:, :, :32])
    with pytest.raises(ValueError):
        qx.qx_attn_paged(b.kv, b.q.transpose(0, 1).contiguous().transpose(0, 1)[:, ::2])
    with pytest.raises(ValueError):
        qx.qx_attn_paged(b.kv, b.q, out=torch.empty((2, 4, 63), device="cuda"))
    with pytest.raises(qx.QxError) as e:
        qx.qx_attn_paged(b.kv, b.q, out=torch.empty((2, 4, 64), dtype=F16, device="cuda"))
    assert e.value.status == qx.QX_ERR_FMT
    with pytest.raises(qx.QxError) as e:
        qx.qx_attn_paged(b.kv, b.q[:, :3].contiguous())  # 3 query heads over 2 key heads
    assert e.value.status == qx.QX_ERR_SHAPE
    for bad in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan"))):
        with pytest.raises(qx.QxError) as e:
            qx.qx_attn_paged(b.kv, b.q, **bad)
        assert e.value.status == qx.QX_ERR_ARG
    with pytest.raises(qx.QxError) as e:
        qx.qx_attn_shared(b.kv, b.q, -1)
    assert e.value.status == qx.QX_ERR_ARG
    with pytest.raises(ValueError):
        qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:5], x[:, 6:], cos, sin)
    with pytest.raises(TypeError):
        qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:6], x[:, 6:].double(), cos, sin)
    with pytest.raises(TypeError):
        qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:6], x[:, 6:], cos.double(), sin.double())
    with pytest.raises(qx.QxError) as e:
        qx.qx_rope_append(b.kv, x[:, :4], x[:, 4:6], x[:, 6:], cos[:, :30].contiguous(), sin[:, :30].contiguous())
    assert e.value.status == qx.QX_ERR_SHAPE
    with pytest.raises(ValueError):
        qx.PagedKV(b.k, b.v[:, :1], b.table, b.kv_len, b.q_start)
    with pytest.raises(TypeError):
        qx.PagedKV(b.k, b.v, b.table.long(), b.kv_len, b.q_start)
    with pytest.raises(ValueError):
        qx.PagedKV(b.k, b.v, b.table, b.kv_len, b.q_start[:2])
    odd = qx.PagedKV(b.k[:, :, :12], b.v[:, :, :12], b.table, b.kv_len, b.q_start)
    with pytest.raises(qx.QxError) as e:
        qx.qx_attn_paged(odd, b.q)
    assert e.value.status == qx.QX_ERR_SHAPE
    y = torch.randn(4, 64, device="cuda")
    with pytest.raises(ValueError):
        qx.qx_block_norm(y, y[:3])
    with pytest.raises(TypeError):
        qx.qx_block_norm(y, y, w_pre=torch.ones(64, dtype=F16, device="cuda"))
    with pytest.raises(qx.QxError) as e:
        qx.qx_block_norm(y, y, w_pre=torch.ones(64, device="cuda"), eps=-1.0)
    assert e.value.status == qx.QX_ERR_ARG
    assert qx.qx_device_check() == qx.QX_OK
