"""GPU tests of attention over an 8-bit cache whose scales lie far apart or far from
one, each row against a plain 64-bit implementation within its own bound."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_q8_gb300 as qx
from . import layer_reference as ref
from .test_gpu_layer_q8 import BF16, F16, F32, BatchQ8
from .test_gpu_layer_q8_edges import CALLS

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -80  # what the bound takes a row's value scales for at least


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()
    qx.lib()
    assert qx.qx_device_check() == qx.QX_OK


def slots(b, s):
    """Page and slot of each key of sequence s."""
    j = np.arange(b.kv_lens[s])
    return torch.from_numpy(b.table_host[s, j // b.page]).long().cuda(), torch.from_numpy(j % b.page).cuda()


def scales_of(b, w, s):
    page, slot = slots(b, s)
    return getattr(b, w + "_scale")[page, :, slot].cpu().numpy()


def set_heads(b, w, s, scales, zero=None):
    """Gives the heads of sequence s these scales [keys, heads], and codes of zero where `zero` [keys] says so."""
    page, slot = slots(b, s)
    codes = np.rint(b.held[w][s] / scales_of(b, w, s)[..., None].astype(np.float64))
    if zero is not None:
        codes[zero] = 0
        getattr(b, w)[page, :, slot] = torch.from_numpy(codes).to(torch.int8).cuda()
    scales = scales.astype(np.float32)
    getattr(b, w + "_scale")[page, :, slot] = torch.from_numpy(scales).cuda()
    b.held[w][s] = codes * scales[..., None].astype(np.float64)


def check(b, scale=None, window=0, sinks=0, what=""):
    """Outputs (in f32) and log-sum-exps of every row.

    A product p d is rounded to f16 (2^-11 at most), or held to 2^-32 of D = the
    row's largest p times its largest value scale (or 2^-80), and meets codes of
    128 at most.  Scores as in attention_bound.  Exponents: an argument is below
    256 and rounds by 2^-17; a row's base rises by 256 in all, and its rescalings'
    arguments round by 2^-24 of that together: below 2^-15 with the joins'.  The
    sum of the p loses those below 2^-38 of the largest."""
    scale = b.dim ** -0.5 if scale is None else scale
    out, lse = torch.empty(b.T, b.hq, b.dim, device="cuda"), torch.empty(b.T, b.hq, device="cuda")
    qx.qx_attn_paged_q8(b.kv, b.q, scale=scale, window=window, sinks=sinks, out=out, lse=lse)
    assert qx.qx_device_check() == qx.QX_OK
    got, got_lse, q, group = ref.f64(out), ref.f64(lse), ref.f64(b.q), b.hq // b.hkv
    for s, kv in enumerate(b.kv_lens):
        t0, t1 = b.q_start_host[s], b.q_start_host[s + 1]
        pos, j = np.arange(kv - (t1 - t0), kv)[:, None], np.arange(kv)[None]
        see = (j <= pos) & ((j > pos - window) | (j < sinks) if window else True)
        dv = np.abs(scales_of(b, "v", s).astype(np.float64))
        for h in range(b.hq):
            z = (q[t0:t1, h] @ b.held["k"][s][:, h // group].T) * scale
            top = np.where(see, np.abs(z), 0).max(1)
            z = np.where(see, z, -np.inf)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            l = p.sum(1, keepdims=True)
            p /= l
            v = b.held["v"][s][:, h // group]
            want, mass, want_lse = p @ v, p @ np.abs(v), (m + np.log(l))[:, 0]
            rel = 2.0 ** -15 + 16 * (b.dim + 2) * 2.0 ** -24 * (1.0 + top) / 4 + kv * 2.0 ** -38
            largest = p.max(1) * np.maximum(np.where(see, dv[:, h // group], 0).max(1), LEAST)
            tol = (2.0 ** -11 + rel)[:, None] * mass + (kv * 2.0 ** -32 * 128 * largest)[:, None] + 2.0 ** -23 * np.abs(want)
            err = np.abs(got[t0:t1, h] - want)
            assert (err <= tol).all(), f"{what} sequence {s} head {h}: {np.max(err / tol):.3g} of the bound"  # (no numbers, too)
            assert (np.abs(got_lse[t0:t1, h] - want_lse) <= rel + 2.0 ** -15 + 2.0 ** -22 * np.abs(want_lse)).all(), f"{what} sequence {s} head {h}"


PATTERNS = {"first half": lambda j, n: j < n // 2, "second half": lambda j, n: j >= n // 2, "thirty-twos": lambda j, n: j // 32 % 2 == 0,
            "one by one": lambda j, n: j * 7 % 5 < 2, "the last": lambda j, n: j < n - 1}
CASES = CALLS + [((32, 8, 128), [1] * 6, [5000, 300, 64, 1, 2000, 130]), ((28, 4, 64), [150, 3], [3000, 90])]


@pytest.mark.parametrize("heads,q_lens,kv_lens", CASES, ids=lambda v: str(v))
@pytest.mark.parametrize("low,high", [(0.0, 60), (0.0, 100), (-80, 47), (-80, 100), (-40, 85), (0, 100), (-70, 60)], ids=str)
def test_sums_where_value_scales_lie_far_apart(heads, q_lens, kv_lens, low, high):
    """Keys of like scores, of which some have values of 2^low (0.0: of zero) and the others 2^high:
    the first ones' probabilities count as much as the others'."""
    for i, (name, lows) in enumerate(PATTERNS.items()):
        b = BatchQ8(q_lens, kv_lens, *heads, 16, (BF16, F16)[i % 2], seed=30 + i)
        for s, kv in enumerate(kv_lens):
            d = scales_of(b, "v", s).astype(np.float64)
            least = 0.0 * d if isinstance(low, float) else d / d.min() * 2.0 ** low
            set_heads(b, "v", s, np.where(lows(np.arange(kv), kv)[:, None], least, d / d.max() * 2.0 ** high))
        check(b, what=name)
        if name == "thirty-twos":
            check(b, window=70, sinks=3, what=name + ", window")


@pytest.mark.parametrize("heads,q_lens,kv_lens", CASES, ids=lambda v: str(v))
def test_value_scales_of_one_size(heads, q_lens, kv_lens):
    """From 2^-80 to 2^100 relative to themselves; smaller ones as if they were 2^-80."""
    for i, power in enumerate((-80, 100, -70, -100, -120)):
        b = BatchQ8(q_lens, kv_lens, *heads, 16, (BF16, F16)[i % 2], seed=40 + i, k_std=3.0)
        for s in range(len(kv_lens)):
            d = scales_of(b, "v", s).astype(np.float64)
            set_heads(b, "v", s, d / (d.max() if power > 0 else d.min()) * 2.0 ** power)
        check(b, what=f"2^{power}")


@pytest.mark.parametrize("heads,tokens", [((8, 2, 128), 1), ((14, 2, 64), 1), ((8, 1, 128), 64), ((4, 2, 80), 1)], ids=str)
def test_many_small_probabilities_of_small_value_scales(heads, tokens):
    """20000 keys of 2^-18 of the largest probability each, all value scales at 2^-80."""
    kv = 20000
    b = BatchQ8([tokens], [kv], *heads, 64, BF16, seed=50, spread=0.2)
    b.q.fill_(1.0)
    scales = np.zeros((kv, b.hkv))
    codes = np.zeros((kv, b.hkv, b.dim))
    codes[7] = 127
    scales[7] = 18 * np.log(2) / (127 * b.dim * b.dim ** -0.5)
    b.held["k"][0] = codes * scales_of(b, "k", 0)[..., None].astype(np.float64)
    page, slot = slots(b, 0)
    b.k[page, :, slot] = torch.from_numpy(codes).to(torch.int8).cuda()
    set_heads(b, "k", 0, scales)
    d = scales_of(b, "v", 0).astype(np.float64)
    set_heads(b, "v", 0, d / d.min() * LEAST)
    check(b)


@pytest.mark.parametrize("heads,q_lens,kv_lens", CASES, ids=lambda v: str(v))
def test_value_scales_that_rise_from_key_to_key(heads, q_lens, kv_lens):
    """Keys that a row does not see yet, or not any more, have larger values: the row is within the
    bound of those that it sees."""
    for i, rise in enumerate((lambda j: j // 16, lambda j: j % 128 // 32, lambda j: 60 - j // 16, lambda j: 4 * (j % 64 > 40))):
        b = BatchQ8(q_lens, kv_lens, *heads, 16, (F16, BF16)[i % 2], seed=70 + i, k_std=2.0)
        for s, kv in enumerate(kv_lens):
            power = np.clip(rise(np.arange(kv)), -70, 90)
            set_heads(b, "v", s, scales_of(b, "v", s).astype(np.float64) * 2.0 ** power[:, None])
        check(b)
        check(b, window=50, sinks=2, what="window")
