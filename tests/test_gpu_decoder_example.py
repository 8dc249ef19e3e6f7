"""The decoder example: a prompt taken at once, in chunks, and token by token
gives the same hidden states, with a window and behind a shared prefix too.

The weight products are the same W4A8 arithmetic on every path (their f32 sums
differ by their order), the cache holds the same bf16 keys and values up to a
unit in the last place, and the attention rounds its probabilities to bf16, so
outputs of norm about 1 agree within 2 % in the 2-norm of a row."""
import os
import sys

import pytest
import torch

import block_quantized_gemv_q8_gb300 as qx

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu
SMALL = dict(hidden=1024, ffn=2048, q_heads=8, kv_heads=2, head_dim=128, layers=2, max_keys=512, page=16)


def near(a, b):
    assert qx.qx_device_check() == qx.QX_OK
    d = ((a - b).norm(dim=-1) / b.norm(dim=-1)).max().item()
    assert d < 0.02, d


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qx.build_library()


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_chunks_and_steps_agree_with_the_whole_prompt(window, sinks):
    from decoder_layer import Decoder
    h = torch.randn(300, 1024, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    whole = Decoder(**SMALL, window=window, sinks=sinks)
    whole.batch([300])
    want = whole.forward(h.clone())
    parts = Decoder(**SMALL, window=window, sinks=sinks)
    got, at = [], 0
    for n in (130, 1, 7, 158, 1, 1, 2):
        parts.batch([n])
        got.append(parts.forward(h[at:at + n].clone()))
        at += n
    near(torch.cat(got), want)


def test_batch_of_sequences_and_a_shared_prefix():
    from decoder_layer import Decoder
    g = torch.Generator(device="cuda").manual_seed(2)
    prefix = torch.randn(200, 1024, device="cuda", generator=g)
    tails = torch.randn(3, 9, 1024, device="cuda", generator=g)
    want = []
    for b in range(3):
        one = Decoder(**SMALL)
        one.batch([209])
        want.append(one.forward(torch.cat([prefix, tails[b]]))[200:])
    many = Decoder(**SMALL, seqs=3)
    # the first sequence takes the prefix; the others' tables lead to its pages (12 whole ones) and a copy of the last
    many.batch([200, 0, 0])
    many.forward(prefix.clone())
    for b in (1, 2):
        for kv in many.kv:
            for c in (kv.k, kv.v):
                c[int(many.table[b, 12])] = c[int(many.table[0, 12])]
        many.table[b, :12] = many.table[0, :12]
        many.kv_len[b] = 200
    got = []
    for i in range(9):
        many.batch([1, 1, 1])
        got.append(many.forward(tails[:, i].clone(), shared_len=200))
    near(torch.stack(got, 1), torch.stack(want))
