"""Plain 64-bit references of the operators between the weight products, one
sequence and one row at a time, on host arrays, and how far a kernel's result
may be from them."""
import numpy as np
import torch

# unit roundoff (round to nearest): half a unit in the last place, relative
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def tokens(kv_len, q_start):
    """(token, sequence, position) of every token of the batch."""
    for b, kv in enumerate(kv_len):
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            yield q_start[b] + i, b, kv - n + i


def rotate(x, c, s, interleaved):
    """x [heads, dim] turned by the angles whose cosines and sines are c, s [rot / 2]."""
    x, half = x.copy(), len(c)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    x[:, a], x[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return x


def attention(q, keys, values, positions, scale, window=0, sinks=0):
    """q [tokens, hq, d] against the sequence's keys and values [kv, hk, d] (64 bits).

    Returns out, lse, the weighted sum of |v| and the largest |score| of each row."""
    T, hq, d = q.shape
    g = hq // keys.shape[1] if keys.shape[1] else 1
    out, mass = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, top = np.full((T, hq), -np.inf), np.zeros((T, hq))
    positions, j = np.asarray(positions)[:, None], np.arange(len(keys))[None]
    see = j <= positions
    if window:
        see &= (j > positions - window) | (j < sinks)
    rows = see.any(1)
    if not rows.any():
        return out, lse, mass, top
    see = see[rows]
    for h in range(hq):
        k, v = keys[:, h // g], values[:, h // g]
        s = np.where(see, (q[rows, h] @ k.T) * scale, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(1, keepdims=True)
        out[rows, h], mass[rows, h] = (p / l) @ v, (p / l) @ np.abs(v)
        lse[rows, h], top[rows, h] = (m + np.log(l))[:, 0], np.where(see, np.abs(s), 0).max(1)
    return out, lse, mass, top


def attention_bound(out, mass, top, dim, cache_dtype, out_dtype):
    """|kernel - exact| of an output: the probabilities rounded to the cache's
    type before they meet v (u each, of the weighted sum of |v|); each score's
    f32 sum and scaling (dim + 2 roundings of a term no larger than the
    largest score's order, taken as 16 times it) turned into a relative error
    of p; the exponential and the f32 sums (2^-18 together); the output's own
    rounding; and subnormal results (2^-24 for f16's spacing there)."""
    u = ROUND[cache_dtype]
    rel = u + 2.0 ** -18 + 16 * (dim + 2) * 2.0 ** -24 * (1.0 + top)[..., None] / 4
    return rel * mass + ROUND[out_dtype] * (1 + 2 * rel) * np.abs(out) + 2.0 ** -24


def lse_bound(lse, top, dim):
    return 2.0 ** -18 + 16 * (dim + 2) * 2.0 ** -24 * (1.0 + top) / 4 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def block_norm(y, r, w_post, gate, alpha, w_pre, eps):
    u = 0.0
    if y is not None:
        u = y
        if w_post is not None:
            u = u * w_post / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        if gate is not None:
            u = u * gate
        u = alpha * u
    r2 = r + u
    return r2, None if w_pre is None else r2 * w_pre / np.sqrt((r2 * r2).mean(1, keepdims=True) + eps), np.abs(r) + np.abs(u)
