"""GPU tests of attention over an 8-bit cache in batches of unlike sequences: a CTA's
tiles come and go, and chunks run beside single tokens."""
import pytest

import block_quantized_gemv_q8_gb300 as qx
from .test_gpu_layer_q8 import BF16, F16, BatchQ8
from .test_gpu_layer_q8_ranges import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()
    qx.lib()
    assert qx.qx_device_check() == qx.QX_OK


@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (8, 1, 128)], ids=str)
def test_tiles_that_come_and_go(heads):
    """Pairs of one tile and of two, of odd and even numbers of key blocks, one after another in a CTA."""
    tile = 128 // (heads[0] // heads[1])
    q_lens = [(tile // 2, 2 * tile, tile, tile + 3, 5, 2 * tile - 1)[b % 6] for b in range(240)]
    kv_lens = [q + (70, 0, 300, 129, 500, 257, 900)[b % 7] for b, q in enumerate(q_lens)]
    for i, dtype in enumerate((BF16, F16)):
        b = BatchQ8(q_lens, kv_lens, *heads, (16, 64)[i], dtype, seed=80 + i)
        check(b)
        check(b, window=100, sinks=3, what="window")


@pytest.mark.parametrize("heads", [(8, 2, 128), (14, 2, 64), (2, 2, 64)], ids=str)
@pytest.mark.parametrize("chunk,singles", [(512, 63), (256, 255), (1000, 200), (40, 3)])
def test_a_chunk_beside_single_tokens(heads, chunk, singles):
    """Whichever kernel the batch's mean rows choose."""
    kv_lens = [1 + 37 * i % 700 for i in range(singles)]
    at = singles // 2
    b = BatchQ8([1] * at + [chunk] + [1] * (singles - at), kv_lens[:at] + [chunk + 600] + kv_lens[at:], *heads, 16, F16, seed=82)
    check(b)
