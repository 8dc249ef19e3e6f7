"""A decoder stack on the library: block-quantised weight products with the
operators between them, for prefill and for captured decode steps.

    python examples/decoder_layer.py            # Llama-3.1-8B shapes, 4 layers, random weights

A layer is, in the order of its launches,

    q, k, v = Wq x, Wk x, Wv x            qx_gemv_multi, or qx_gemm_prefill for several rows
    q, cache <- rotate(q, k), v           qx_rope_append
    a = attention(q, cache)               qx_attn_paged, or qx_attn_shared behind a shared prefix
    y = Wo a                              qx_gemv / qx_gemm_prefill
    h, x = h + y, norm(h + y)             qx_block_norm
    g, u = Wg x, Wu x                     qx_gemv_multi / qx_gemm_prefill
    y = Wd (silu(g) u)                    qx_gemv / qx_gemm_prefill
    h, x = h + y, norm(h + y)             qx_block_norm, with the next layer's weight

Weights are Q4_K; activations are f32 and quantised to int8 at each product,
the cache is bf16.
"""
from __future__ import annotations

import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_quantized_gemv_q8_gb300 as qx  # noqa: E402


class Decoder:
    """`layers` decoder layers over one paged cache each, with random Q4_K weights."""

    def __init__(self, hidden=4096, ffn=14336, q_heads=32, kv_heads=8, head_dim=128, layers=4, seqs=1, max_keys=4096, page=64,
                 theta=500000.0, window=0, sinks=0, seed=0):
        import synth
        dev = torch.device("cuda")
        self.hidden, self.ffn, self.hq, self.hk, self.dim = hidden, ffn, q_heads, kv_heads, head_dim
        self.window, self.sinks, self.seqs = window, sinks, seqs

        def weight(rows, cols, i):
            w = torch.from_numpy(synth.weights(synth.Q4_K, rows, cols, seed=seed * 1000 + i)).to(dev)
            return w, rows, cols

        self.layers = []
        gen = torch.Generator(device=dev).manual_seed(seed)
        norm = lambda: torch.rand(hidden, device=dev, generator=gen) + 0.5  # noqa: E731
        qd, kd = q_heads * head_dim, kv_heads * head_dim
        for n in range(layers):
            i = 10 * n
            self.layers.append(dict(
                q=weight(qd, hidden, i), k=weight(kd, hidden, i + 1), v=weight(kd, hidden, i + 2), o=weight(hidden, qd, i + 3),
                gate=weight(ffn, hidden, i + 4), up=weight(ffn, hidden, i + 5), down=weight(hidden, ffn, i + 6),
                attn_norm=norm(), ffn_norm=norm()))
        self.last_norm = norm()
        # Random weights of this recipe grow the activations; the residual scale keeps the stack in range.
        self.alpha = 0.05
        angle = torch.arange(max_keys, device=dev, dtype=torch.float64)[:, None] * theta ** (
            -torch.arange(0, head_dim, 2, device=dev, dtype=torch.float64) / head_dim)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        # the batch: one row of the page table a sequence (here each sequence owns its pages)
        pages = -(-max_keys // page)
        self.table = torch.arange(seqs * pages, dtype=torch.int32, device=dev).view(seqs, pages)
        self.kv_len = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.q_start = torch.zeros(seqs + 1, dtype=torch.int32, device=dev)
        self.kv = []
        for _ in range(layers):
            k, v = (torch.zeros((seqs * pages, kv_heads, page, head_dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
            self.kv.append(qx.PagedKV(k, v, self.table, self.kv_len, self.q_start))

    def batch(self, tokens):
        """Announce `tokens[b]` new tokens of each sequence (lengths on the GPU grow in place)."""
        t = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        self.kv_len += t
        self.q_start[1:] = torch.cumsum(t, 0)

    def _product(self, names, layer, x):
        """Several products over the same rows of x."""
        Ws = [layer[n] for n in names]
        cols = Ws[0][2]
        if x.shape[0] == 1:
            ys = qx.qx_gemv_multi([qx.QX_Q4_K] * len(Ws), [w[0] for w in Ws], [w[1] for w in Ws], cols, x[0],
                                  mode=qx.QX_MODE_W4A8_FUSED | qx.QX_FLAG_PDL)
            return [y[None] for y in ys]
        act = qx.qx_quantize_act_q8(x)
        return [qx.qx_gemm_prefill(qx.QX_Q4_K, w, rows, cols, act) for w, rows, _ in Ws]

    def forward(self, h, shared_len=0):
        """h: f32 [tokens, hidden], the tokens that batch() announced; returns the normed output of the stack."""
        h, x = qx.qx_block_norm(None, h, w_pre=self.layers[0]["attn_norm"], x_out=torch.empty_like(h))
        for n, layer in enumerate(self.layers):
            T, kv = x.shape[0], self.kv[n]
            q, k, v = self._product(("q", "k", "v"), layer, x)
            q = qx.qx_rope_append(kv, q.view(T, self.hq, self.dim), k.view(T, self.hk, self.dim), v.view(T, self.hk, self.dim), self.cos,
                                  self.sin, interleaved=True)
            a = torch.empty((T, self.hq, self.dim), device=x.device)
            if shared_len:
                qx.qx_attn_shared(kv, q, shared_len, out=a)
            else:
                qx.qx_attn_paged(kv, q, window=self.window, sinks=self.sinks, out=a)
            y, = self._product(("o",), layer, a.view(T, self.hq * self.dim))
            h, x = qx.qx_block_norm(y, h, alpha=self.alpha, w_pre=layer["ffn_norm"])
            gate, up = self._product(("gate", "up"), layer, x)
            y, = self._product(("down",), layer, torch.nn.functional.silu(gate) * up)
            w = self.layers[n + 1]["attn_norm"] if n + 1 < len(self.layers) else self.last_norm
            h, x = qx.qx_block_norm(y, h, alpha=self.alpha, w_pre=w)
        return x


def main():
    prompt, steps = 2000, 64
    d = Decoder(max_keys=prompt + steps + 8)
    h = torch.randn(prompt, d.hidden, device="cuda")
    d.batch([prompt])
    d.forward(h)  # warm-up: the cache is written again below
    torch.cuda.synchronize()
    t = time.perf_counter()
    out = d.forward(h)
    torch.cuda.synchronize()
    print(f"prefill of {prompt} tokens, {len(d.layers)} layers: {(time.perf_counter() - t) * 1e3:.2f} ms")
    # decode: one captured step, replayed while the lengths grow in place
    x = out[-1:].clone()
    d.batch([1])
    d.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = d.forward(x)
    t = time.perf_counter()
    for _ in range(steps):
        graph.replay()
        x.copy_(y)
        d.kv_len += 1
    torch.cuda.synchronize()
    print(f"decode: {(time.perf_counter() - t) / steps * 1e3:.3f} ms a token ({len(d.layers)} layers, contexts of {prompt} to "
          f"{prompt + steps} keys)")
    assert qx.qx_device_check() == qx.QX_OK and torch.isfinite(y).all()


if __name__ == "__main__":
    main()
