"""GPU tests of attention over an 8-bit cache whose key scales, times the scores'
scale or times a row's products alone, leave f32's range though the scores do not."""
import numpy as np
import pytest
import torch

import block_quantized_gemv_q8_gb300 as qx
from .test_gpu_layer_q8 import BF16, F16, BatchQ8
from .test_gpu_layer_q8_edges import CALLS
from .test_gpu_layer_q8_ranges import check, scales_of, set_heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()
    qx.lib()
    assert qx.qx_device_check() == qx.QX_OK


@pytest.mark.parametrize("heads,q_lens,kv_lens", CALLS, ids=lambda v: str(v))
@pytest.mark.parametrize("sign", [1, -1])
def test_products_of_nothing(heads, q_lens, kv_lens, sign):
    """Queries of zeros over keys of very large scales, and keys whose codes are zeros among others: scores of zero."""
    for i, dtype in enumerate((BF16, F16)):
        b = BatchQ8(q_lens, kv_lens, *heads, 16, dtype, seed=60 + i)
        for s, kv in enumerate(kv_lens):
            nothing = np.arange(kv) % 3 == 1
            set_heads(b, "k", s, np.where(nothing[:, None], np.float32(3e38), scales_of(b, "k", s)), nothing)
        check(b, scale=sign * 0.9, what="codes of zeros")
        b = BatchQ8(q_lens, kv_lens, *heads, 16, dtype, seed=62 + i)
        b.q.zero_()
        for s, kv in enumerate(kv_lens):
            set_heads(b, "k", s, np.full((kv, b.hkv), 3e38))
        check(b, scale=sign * 5.0, what="queries of zeros")


@pytest.mark.parametrize("heads,q_lens,kv_lens", CALLS, ids=lambda v: str(v))
@pytest.mark.parametrize("power", [122, 100, -100, -110])
def test_scales_that_make_up_for_one_another(heads, q_lens, kv_lens, power):
    """Key scales of 2^power with scores' scales of about its inverse, of either sign."""
    for i, dtype in enumerate((BF16, F16)):
        b = BatchQ8(q_lens, kv_lens, *heads, 32, dtype, seed=64 + i)
        for s in range(len(kv_lens)):
            set_heads(b, "k", s, scales_of(b, "k", s).astype(np.float64) * 64 * 2.0 ** power)
        for sign in (1, -1):
            check(b, scale=sign * 2.0 ** -(power + 4 if power > 0 else power + 8), what=f"{dtype} {sign}")


@pytest.mark.parametrize("heads,q_lens,kv_lens", CALLS, ids=lambda v: str(v))
def test_large_queries_beside_large_scales(heads, q_lens, kv_lens):
    """Queries of 2^110 over keys of 2^-110, and keys of no codes whose scale is 2^40."""
    b = BatchQ8(q_lens, kv_lens, *heads, 16, BF16, seed=66)
    b.q = (b.q.double() * 2.0 ** 110).to(BF16)
    for s, kv in enumerate(kv_lens):
        nothing = np.arange(kv) % 5 == 2
        set_heads(b, "k", s, np.where(nothing[:, None], 2.0 ** 40, scales_of(b, "k", s).astype(np.float64) * 2.0 ** -110), nothing)
    check(b)
