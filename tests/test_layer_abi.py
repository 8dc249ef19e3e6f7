"""Refusals of the entry points between the weight products, from the host,
before anything is launched (no GPU needed; the addresses are never used)."""
import ctypes

import pytest

import block_quantized_gemv_q8_gb300 as qx

A16 = 1 << 20


@pytest.fixture(scope="module")
def lib():
    qx.build_library()
    return qx.lib()


def kv(**change):
    a = dict(k=A16, v=A16, dtype=qx.QX_BF16, n_heads=2, head_dim=64, page_size=16, n_pages=4, page_stride=2048, head_stride=1024,
             slot_stride=64, table=A16, table_stride=3, kv_len=A16, q_start=A16, n_seqs=1)
    a.update(change)
    return qx._Kv(**a)


BAD_KV = [(dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(table=None), "ARG"), (dict(kv_len=None), "ARG"),
          (dict(q_start=None), "ARG"), (dict(dtype=qx.QX_F32), "FMT"), (dict(dtype=5), "FMT"), (dict(n_heads=0), "SHAPE"),
          (dict(head_dim=0), "SHAPE"), (dict(head_dim=60), "SHAPE"), (dict(head_dim=264), "SHAPE"), (dict(page_size=8), "SHAPE"),
          (dict(page_size=48), "SHAPE"), (dict(page_size=1 << 17), "SHAPE"), (dict(n_pages=0), "SHAPE"),
          (dict(n_pages=1 << 31), "SHAPE"), (dict(table_stride=0), "SHAPE"), (dict(n_seqs=0), "SHAPE"),
          (dict(page_stride=-8), "SHAPE"), (dict(slot_stride=1 << 41), "SHAPE"), (dict(slot_stride=56), "SHAPE"),
          (dict(head_stride=0), "SHAPE"), (dict(page_stride=8), "SHAPE"), (dict(slot_stride=68), "ALIGN"),
          (dict(head_stride=1001), "ALIGN"), (dict(k=A16 + 8), "ALIGN"), (dict(v=A16 + 2), "ALIGN")]


@pytest.mark.parametrize("change,status", BAD_KV, ids=lambda v: str(v))
def test_cache_descriptors(lib, change, status):
    want = getattr(qx, "QX_ERR_" + status)
    c, P = kv(**change), ctypes.c_void_p
    q = qx._Qkv(1, 2, qx.QX_F32, A16, A16, A16, 128, 128, 128)
    assert lib.qx_rope_append(ctypes.byref(c), ctypes.byref(q), P(A16), P(A16), 9, 64, 0, P(A16), None) == want
    assert lib.qx_attn_paged(ctypes.byref(c), P(A16), 1, 2, 128, 1.0, 0, 0, P(A16), qx.QX_BF16, None, P(A16), None) == want
    assert lib.qx_attn_shared(ctypes.byref(c), P(A16), 1, 2, 128, 1.0, 0, P(A16), qx.QX_BF16, None, P(A16), None) == want


def test_rope_append_refusals(lib):
    c, P = kv(), ctypes.c_void_p

    def call(cos=A16, sin=A16, n_pos=9, rot=64, out=A16, cache=None, null_in=False, **change):
        a = dict(n_tokens=1, n_q_heads=2, dtype=qx.QX_F32, q=A16, k=A16, v=A16, q_stride=128, k_stride=128, v_stride=128)
        a.update(change)
        i = qx._Qkv(**a)
        return lib.qx_rope_append(ctypes.byref(c) if cache is None else None, None if null_in else ctypes.byref(i), P(cos), P(sin),
                                  n_pos, rot, 0, P(out), None)

    for bad in (dict(cache=0), dict(null_in=True), dict(q=None), dict(k=None), dict(v=None), dict(cos=None), dict(sin=None), dict(out=None)):
        assert call(**bad) == qx.QX_ERR_ARG, bad
    assert call(dtype=2) == qx.QX_ERR_FMT
    for bad in (dict(rot=4), dict(rot=72), dict(rot=-8), dict(n_pos=-1), dict(n_tokens=-1), dict(n_q_heads=-1), dict(q_stride=-8)):
        assert call(**bad) == qx.QX_ERR_SHAPE, bad
    for bad in (dict(q=A16 + 4), dict(k=A16 + 8), dict(v=A16 + 2), dict(cos=A16 + 4), dict(sin=A16 + 4), dict(out=A16 + 2),
                dict(q_stride=130), dict(k_stride=65), dict(v_stride=4)):
        assert call(**bad) == qx.QX_ERR_ALIGN, bad
    assert call(n_tokens=0) == qx.QX_OK


def test_attention_refusals(lib):
    c, P = kv(), ctypes.c_void_p

    def call(shared=False, q=A16, n=1, hq=4, stride=256, scale=1.0, window=0, sinks=0, out=A16, dtype=qx.QX_BF16, lse=None, scratch=A16):
        mask = (window,) if shared else (window, sinks)
        f = lib.qx_attn_shared if shared else lib.qx_attn_paged
        return f(ctypes.byref(c), P(q), n, hq, stride, scale, *mask, P(out), dtype, P(lse), P(scratch), None)

    for shared in (False, True):
        for bad in (dict(q=None), dict(out=None), dict(scratch=None), dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan"))):
            assert call(shared, **bad) == qx.QX_ERR_ARG, bad
        for bad in (dict(hq=3), dict(hq=0), dict(hq=2 * 129), dict(n=-1), dict(n=1 << 31), dict(stride=-8), dict(n=2, stride=248)):
            assert call(shared, **bad) == qx.QX_ERR_SHAPE, bad
        for bad in (dict(dtype=qx.QX_F16), dict(dtype=3)):
            assert call(shared, **bad) == qx.QX_ERR_FMT, bad
        for bad in (dict(q=A16 + 2), dict(out=A16 + 8), dict(stride=252), dict(lse=A16 + 1), dict(scratch=A16 + 16)):
            assert call(shared, **bad) == qx.QX_ERR_ALIGN, bad
        assert call(shared, n=0, q=None, out=None, scratch=None) == qx.QX_OK
    assert call(sinks=-1) == qx.QX_ERR_ARG


def test_scratch_sizes(lib):
    size = lib.qx_attn_scratch_bytes
    assert size(1, 4, 2, 64, 1) > 0 and size(0, 4, 2, 64, 1) > 0
    assert size(64, 32, 8, 128, 64) >= size(1, 32, 8, 128, 1)
    for bad in ((-1, 4, 2, 64, 1), (1, 3, 2, 64, 1), (1, 0, 2, 64, 1), (1, 4, 0, 64, 1), (1, 4, 2, 60, 1), (1, 4, 2, 64, 0),
                (1, 4, 2, 512, 1), (1, 129, 1, 64, 1)):
        assert size(*bad) == 0, bad


def test_block_norm_refusals(lib):
    def call(**change):
        a = dict(rows=1, cols=64, dtype=qx.QX_F32, res_dtype=qx.QX_F32, y=A16, r=A16, w_post=A16, w_pre=A16, alpha=1.0, eps=1e-5, r_out=A16,
                 x=A16, y_stride=64, r_stride=64, r_out_stride=64, x_stride=64)
        a.update(change)
        return lib.qx_block_norm(ctypes.byref(qx._Norm(**a)), None)

    assert lib.qx_block_norm(None, None) == qx.QX_ERR_ARG
    for bad in (dict(r=None), dict(w_pre=None), dict(x=None), dict(r_out=None, x=None, w_pre=None), dict(y=None), dict(eps=-1.0),
                dict(eps=float("nan")), dict(alpha=float("inf")), dict(y=None, w_post=None, gate=A16)):
        assert call(**bad) == qx.QX_ERR_ARG, bad
    for bad in (dict(dtype=2), dict(res_dtype=8)):
        assert call(**bad) == qx.QX_ERR_FMT, bad
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=32769), dict(y_stride=-1)):
        assert call(**bad) == qx.QX_ERR_SHAPE, bad
    for bad in (dict(y=A16 + 2), dict(r=A16 + 1), dict(w_pre=A16 + 2), dict(w_post=A16 + 3), dict(x=A16 + 2), dict(r_out=A16 + 1)):
        assert call(**bad) == qx.QX_ERR_ALIGN, bad
    assert call(rows=0) == qx.QX_OK


def test_new_status_has_a_name(lib):
    assert qx.qx_status_string(qx.QX_ERR_RANGE).startswith("QX_ERR_RANGE")


def test_scratch_sizes_serve_every_smaller_call(lib):
    """A caller may size once for the largest of every argument."""
    size, last = lib.qx_attn_scratch_bytes, 0
    for dim in range(8, 257, 8):
        assert size(300, 32, 8, dim, 4) >= last, dim
        last = size(300, 32, 8, dim, 4)
    for tokens in (0, 1, 2, 3, 263, 264, 265, 266, 4095, 4096, 4097, 100000):
        for heads in (8, 16, 32, 64):
            most = size(tokens, heads, 8, 128, 9)
            assert all(size(t, h, hk, d, n) <= most for t in (0, tokens // 2, max(0, tokens - 1), tokens) for h in (8, heads)
                       for hk in (1, 8) for d in (8, 64, 80, 128) for n in (1, 9)), (tokens, heads)


def test_agree_probe_refusals(lib):
    P = ctypes.c_void_p
    for limit, got in ((10, A16), (1 << 40, A16), (1_000_000, None)):
        assert lib.qx_debug_agree_probe(limit, P(got), None) == qx.QX_ERR_ARG


def test_block_norm_refuses_output_rows_that_overlap(lib):
    def call(**change):
        a = dict(rows=2, cols=64, dtype=qx.QX_BF16, res_dtype=qx.QX_F32, y=A16, r=2 * A16, w_pre=A16, alpha=1.0, eps=1e-5, r_out=3 * A16,
                 x=4 * A16, y_stride=64, r_stride=64, r_out_stride=64, x_stride=64)
        a.update(change)
        return lib.qx_block_norm(ctypes.byref(qx._Norm(**a)), None)

    for bad in (dict(r_out_stride=0), dict(r_out_stride=63), dict(x_stride=0), dict(x_stride=56), dict(r_out=None, x_stride=8)):
        assert call(**bad) == qx.QX_ERR_SHAPE, bad
    # in place, each row over its own
    for bad in (dict(r_out=2 * A16, r_stride=128), dict(r_out=2 * A16, r_out_stride=72), dict(x=A16, y_stride=0), dict(x=A16, y_stride=72)):
        assert call(**bad) == qx.QX_ERR_SHAPE, bad
