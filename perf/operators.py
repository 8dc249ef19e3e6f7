"""What a decoder layer runs between its weight products, as measurable cases.

Four operators: keys and values appended to a paged cache with the position
rotation applied on the way ("append"); attention over that cache with a
sliding window and a few first tokens that stay visible ("attn"); the same for
a batch whose sequences share a long prefix ("shared"); and the norms after and
before a block fused with its gate and residual scale ("norm").  `run` computes
them in plain torch operations in 32 bits, or, where `own` is true, through
this repository's package.

Head layouts: 32 query and 8 key heads of 128 (q 4096 rows, k and v 1024 rows:
the Llama-3.1-8B projections) and 14 and 2 heads of 64 (896 and 128 rows: the
Qwen2-0.5B projections), and other groupings of the same head sizes.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of one conversation: the call's latency
        dict(name="append 1 token", op="append", seqs=1, q_min=1, q_max=1, kv_min=2047, kv_max=2047, page=64, hq=32, hkv=8,
             dim=128, rot=128, interleaved=True, src="f32", dtype="bf16"),
        # a decode step of 64 conversations of mixed length on a small model
        dict(name="append 64 tokens", op="append", seqs=64, q_min=1, q_max=1, kv_min=1, kv_max=4000, page=32, hq=14, hkv=2,
             dim=64, rot=64, interleaved=False, src="f32", dtype="f16"),
        # three long prompts in one prefill call
        dict(name="append 3 prompts", op="append", seqs=3, q_min=1500, q_max=4001, kv_min=1500, kv_max=4001, page=64, hq=32,
             hkv=8, dim=128, rot=128, interleaved=True, src="f32", dtype="bf16"),
        # one token of one short conversation on a small model: the call's latency
        dict(name="decode 1 x 1023", op="attn", seqs=1, q_min=1, q_max=1, kv_min=1023, kv_max=1023, page=32, hq=14, hkv=2, dim=64,
             window=0, sinks=0, dtype="f16"),
        # a decode step of 64 long conversations, the window and four sinks visible
        dict(name="decode 64, window 4096", op="attn", seqs=64, q_min=1, q_max=1, kv_min=100, kv_max=16000, page=64, hq=32, hkv=8,
             dim=128, window=4096, sinks=4, dtype="bf16"),
        # chunks of several prompts behind earlier context, small model, small pages
        dict(name="prefill 5 chunks", op="attn", seqs=5, q_min=37, q_max=1000, kv_min=600, kv_max=6000, page=16, hq=14, hkv=2,
             dim=64, window=0, sinks=0, dtype="f16"),
        # a long prompt in one call, the window and four sinks visible
        dict(name="prefill 8191, window 1024", op="attn", seqs=1, q_min=8191, q_max=8191, kv_min=8191, kv_max=8191, page=64, hq=32,
             hkv=8, dim=128, window=1024, sinks=4, dtype="bf16"),
        # a few answers sampled in parallel from one prompt
        dict(name="shared 2000, 16 seqs", op="shared", seqs=16, shared=2000, tail_min=1, tail_max=300, page=16, hq=32, hkv=8,
             dim=128, dtype="bf16"),
        # a full decode batch behind one long system prompt or document
        dict(name="shared 32768, 256 seqs", op="shared", seqs=256, shared=32768, tail_min=5, tail_max=500, page=64, hq=32, hkv=8,
             dim=128, dtype="bf16"),
        # between two blocks of a decode step: the call's latency
        dict(name="norm 1 x 4096", op="norm", rows=1, cols=4096, gate="none", post=True, alpha=1.0, dtype="f32", res="f32"),
        # a decode batch on a small model, gated for each row and channel
        dict(name="norm 77 x 896", op="norm", rows=77, cols=896, gate="row", post=True, alpha=0.7, dtype="f16", res="f32"),
        # between two blocks of a prefill
        dict(name="norm 8192 x 4096", op="norm", rows=8192, cols=4096, gate="channel", post=True, alpha=0.5, dtype="bf16", res="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _padded(case):
    """Values of the plain form's largest temporary."""
    if case["op"] in ("append", "norm"):
        return 0
    q, kv = _lens(case)
    if case["op"] == "shared":
        return len(q) * max(kv) * case["hq"]
    return len(q) * max(max(q) * max(kv) * case["hq"], max(kv) * case["hkv"] * case["dim"])


def _draw(rng):
    op = rng.choice(["append", "attn", "attn", "shared", "norm"])
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=rng.choice([896, 1024, 2048, 4096, 4864, 14336, 64 * rng.randint(2, 200)]),
                    gate=rng.choice(["none", "row", "channel"]), post=rng.random() < 0.8, alpha=round(rng.uniform(0.1, 1.5), 3),
                    dtype=rng.choice(["f32", "bf16", "f16"]), res=rng.choice(["f32", "f32", "bf16"]))
    hq, hkv, dim = rng.choice([(32, 8, 128), (14, 2, 64), (8, 8, 128), (16, 1, 64), (32, 4, 128), (12, 2, 128)])
    c = dict(op=op, page=rng.choice([16, 32, 64, 128, 256]), hq=hq, hkv=hkv, dim=dim, dtype=rng.choice(["bf16", "f16"]))
    if op == "shared":
        c.update(seqs=_log(rng, 2, 256), shared=_log(rng, 100, 32768), tail_min=1, tail_max=_log(rng, 1, 2000))
        return c
    if rng.random() < 0.5:  # decode, one token or a few
        c.update(seqs=_log(rng, 1, 256), q_min=1, q_max=rng.choice([1, 1, 1, 4]))
        kv = _log(rng, 1, 131072)
    else:
        c.update(seqs=_log(rng, 1, 16), q_min=1, q_max=_log(rng, 8, 8192))
        kv = _log(rng, 1, 16384)
    kv = max(kv, c["q_max"])
    c.update(kv_min=max(c["q_max"], int(kv * rng.uniform(0.1, 1.0))), kv_max=kv)
    if op == "append":
        c.update(rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5, src=rng.choice(["f32", c["dtype"]]))
    else:
        c.update(window=rng.choice([0, _log(rng, 16, 8192)]), sinks=0)
        if c["window"]:
            c["sinks"] = rng.choice([0, 1, 4, 4, 17])
    return c


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _cost(c))
    while True:
        c = _draw(rng)
        if _cost(c) <= most[c["op"]] and _padded(c) <= 2_300_000_000:
            return c


def _spread(n, lo, hi):
    """n whole numbers spread over lo .. hi, the largest first: a batch's lengths go by the case alone."""
    return [hi - int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(n)]


def _lens(case):
    """The new tokens of each sequence, and its keys with those counted."""
    n = case["seqs"]
    if case["op"] == "shared":
        return [1] * n, [case["shared"] + t for t in _spread(n, case["tail_min"], case["tail_max"])]
    q = _spread(n, case["q_min"], case["q_max"])
    kv = _spread(n, case["kv_min"], case["kv_max"])
    if case["op"] == "append" and case["q_max"] > 4:
        return q, [max(a, b) for a, b in zip(q, kv)]
    kv = kv[n // 2:] + kv[:n // 2]  # the longest chunk is not always behind the longest context
    return q, [max(a, b) for a, b in zip(q, kv)]


def work(case):
    if case["op"] == "norm":
        n, e, r = case["rows"] * case["cols"], BYTES[case["dtype"]], BYTES[case["res"]]
        gate = {"none": 0, "row": n * e, "channel": case["cols"] * e}[case["gate"]]
        return {"bytes": n * (2 * e + 2 * r) + gate + case["cols"] * 4 * (1 + case["post"]), "flops": n * 10}
    q, kv = _lens(case)
    T, hq, hkv, d = sum(q), case["hq"], case["hkv"], case["dim"]
    if case["op"] == "append":
        n = T * (hq + 2 * hkv) * d
        return {"bytes": n * (BYTES[case["src"]] + 2) + T * case["rot"] * 4, "flops": T * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "shared":
        keys, pairs = case["shared"] + sum(k - case["shared"] for k in kv), sum(kv)
    else:
        keys = pairs = 0
        for a, b in zip(q, kv):
            p = np.arange(b - a, b, dtype=np.int64)
            if not case["window"]:
                keys, pairs = keys + b, pairs + int((p + 1).sum())
                continue
            low = np.maximum(0, p - case["window"] + 1)
            first = np.minimum(case["sinks"], low)
            keys, pairs = keys + b - int(low[0]) + int(min(case["sinks"], low[0])), pairs + int((p + 1 - low + first).sum())
    return {"bytes": keys * hkv * d * 4 + T * hq * d * 4, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="f32", mean=0.0, std=1.0):
        x = torch.empty(shape, dtype=DTYPES[dtype], device="cuda")
        return x.normal_(mean, std, generator=g)

    s = {"case": case}
    if case["op"] == "norm":
        rows, cols, dt = case["rows"], case["cols"], case["dtype"]
        s["y"], s["r"] = normal(rows, cols, dtype=dt, std=0.5), normal(rows, cols, dtype=case["res"], std=2.0)
        s["w_post"] = normal(cols, mean=1.0, std=0.2) if case["post"] else None
        s["w_pre"] = normal(cols, mean=1.0, std=0.2)
        s["gate"] = {"none": None, "row": (rows, cols), "channel": (cols,)}[case["gate"]]
        if s["gate"] is not None:
            s["gate"] = normal(*s["gate"], dtype=dt)
        s["r_out"], s["x"] = torch.empty_like(s["r"]), torch.empty_like(s["y"])
        return s
    q, kv = _lens(case)
    page, hq, hkv, d, dt = case["page"], case["hq"], case["hkv"], case["dim"], case["dtype"]
    shared = case.get("shared", 0) // page  # pages that all sequences have
    need = np.array([-(-k // page) for k in kv])
    wide, first = int(need.max()), np.concatenate([[0], np.cumsum(need - shared)]) + shared
    at = np.zeros((len(kv), wide), dtype=np.int64)
    for b in range(len(kv)):
        at[b, :shared] = np.arange(shared)
        at[b, shared:need[b]] = np.arange(first[b], first[b + 1])
    order = torch.randperm(int(first[-1]), generator=g, device="cuda").to(torch.int32)  # pages lie anywhere in the cache
    s["table"] = order[torch.from_numpy(at).cuda()].contiguous()
    s["k"], s["v"] = (normal(int(first[-1]), hkv, page, d, dtype=dt) for _ in range(2))
    if case["op"] == "shared" and case["shared"] % page:
        # the page in which the prefix ends is a copy of its own in each sequence
        for c in (s["k"], s["v"]):
            c[s["table"][:, shared].long(), :, :case["shared"] % page] = c[s["table"][0, shared].long(), :, :case["shared"] % page]
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        # the rows of one product: q, k and v lie beside each other
        qkv = normal(sum(q), hq + 2 * hkv, d, dtype=case["src"])
        s["q"], s["new_k"], s["new_v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        half = case["rot"] // 2
        angle = torch.arange(max(kv), device="cuda", dtype=torch.float64)[:, None] * 500000.0 ** (
            -torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    else:
        s["q"] = normal(sum(q), hq, d, dtype=dt)
    s["out"] = torch.empty(sum(q), hq, d, dtype=DTYPES[dt], device="cuda")
    s["q_max"] = max(q)
    if own:
        import block_quantized_gemv_q8_gb300 as qx
        s["kv"] = qx.PagedKV(s["k"], s["v"], s["table"], s["kv_len"], s["q_start"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return {"append": _append, "attn": _attn, "shared": _shared, "norm": _norm}[op](state)


def _run_own(s, op):
    import block_quantized_gemv_q8_gb300 as qx
    c = s["case"]
    if op == "append":
        q = qx.qx_rope_append(s["kv"], s["q"], s["new_k"], s["new_v"], s["cos"], s["sin"], interleaved=c["interleaved"], q_out=s["out"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if op == "attn":
        return qx.qx_attn_paged(s["kv"], s["q"], window=c["window"], sinks=c["sinks"], out=s["out"])
    if op == "shared":
        return qx.qx_attn_shared(s["kv"], s["q"], c["shared"], out=s["out"])
    r, x = qx.qx_block_norm(s["y"], s["r"], w_post=s["w_post"], gate=s["gate"], alpha=c["alpha"], w_pre=s["w_pre"], eps=EPS,
                            r_out=s["r_out"], x_out=s["x"])
    return {"r": r, "x": x}


def _positions(s, tokens):
    """The sequence and the position of each token."""
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"], t, right=True) - 1
    return seq, s["kv_len"][seq] - s["q_start"][seq + 1] + t


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _append(s):
    c, page = s["case"], s["case"]["page"]
    seq, pos = _positions(s, s["q"].shape[0])
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    at, slot = s["table"][seq, pos // page].long(), (pos % page).long()
    s["k"][at, :, slot] = _rotate(s["new_k"], cos, sin, c["rot"], c["interleaved"]).to(s["k"].dtype)
    s["v"][at, :, slot] = s["new_v"].to(s["v"].dtype)
    return {"q": _rotate(s["q"], cos, sin, c["rot"], c["interleaved"]).to(s["out"].dtype), "k": s["k"], "v": s["v"]}


def _pages(cache, table):
    """The pages of a table, in order and in 32 bits: [..., heads, keys, dim]."""
    x = cache[table.long()].float().transpose(-4, -3)
    return x.reshape(*x.shape[:-3], x.shape[-3] * x.shape[-2], x.shape[-1])


def _weights(scores, seen):
    """Softmax over the last axis where `seen`; rows that see nothing get zeros."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = (scores - top).exp()
    return p / p.sum(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)


def _attn(s):
    c, q, n = s["case"], s["q"], s["case"]["seqs"]
    T, hq, d = q.shape
    hkv, G, most = c["hkv"], hq // c["hkv"], s["q_max"]
    k, v = _pages(s["k"], s["table"]), _pages(s["v"], s["table"])  # [seq, hkv, keys, d]
    seq, pos = _positions(s, T)
    row = torch.arange(T, device="cuda") - s["q_start"][seq]
    grid = torch.zeros(n, most, hq, d, device="cuda")
    grid[seq, row] = q.float()
    at = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
    at[seq, row] = pos
    grid = grid.view(n, most, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, G * most, d)
    scores = (grid @ k.transpose(-1, -2)) * (1 / math.sqrt(d))
    j, at = torch.arange(k.shape[2], device="cuda")[None, None], at[:, :, None]
    seen = j <= at
    if c["window"]:
        seen = seen & ((j > at - c["window"]) | (j < c["sinks"]))
    scores = scores.view(n, hkv, G, most, -1)
    o = _weights(scores, seen[:, None, None]).view(n, hkv, G * most, -1) @ v
    o = o.view(n, hkv, G, most, d).permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)
    return o[seq, row].to(q.dtype)


def _shared(s):
    c, q, n = s["case"], s["q"].float(), s["case"]["seqs"]
    hkv, d, page = c["hkv"], c["dim"], c["page"]
    G, L, first = c["hq"] // hkv, c["shared"], c["shared"] // page  # `first`: the pages that all have
    q = q.view(n, hkv, G, d) * (1 / math.sqrt(d))
    k, v = (_pages(s[w], s["table"][0, :-(-L // page)])[:, :L] for w in ("k", "v"))  # [hkv, L, d]
    kt, vt = (_pages(s[w], s["table"][:, first:])[:, :, L - first * page:] for w in ("k", "v"))  # [seq, hkv, tail, d]
    qs = q.transpose(0, 1).reshape(hkv, n * G, d)
    sp = (qs @ k.transpose(-1, -2)).view(hkv, n, G, L).transpose(0, 1)
    st = q @ kt.transpose(-1, -2)
    j = torch.arange(L + kt.shape[2], device="cuda")
    p = _weights(torch.cat((sp, st), -1), (j < s["kv_len"][:, None])[:, None, None])
    o = (p[..., :L].transpose(0, 1).reshape(hkv, n * G, L) @ v).view(hkv, n, G, d).transpose(0, 1) + p[..., L:] @ vt
    return o.reshape(n, hkv * G, d).to(s["out"].dtype)


def _norm(s):
    c, u = s["case"], s["y"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["r"].float() + c["alpha"] * u
    x = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["w_pre"]
    return {"r": r.to(s["r"].dtype), "x": x.to(s["y"].dtype)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        y, r = s["y"].double(), s["r"].double()
        if case["post"]:
            y = s["w_post"].double() * y / (y.square().mean(1, keepdim=True) + EPS).sqrt()
        gate = 1.0 if s["gate"] is None else s["gate"].double()
        r = r + gate * y * case["alpha"]
        return {"r": r, "x": s["w_pre"].double() * r / (r.square().mean(1, keepdim=True) + EPS).sqrt()}
    lens, kv, page, d = *_lens(case), case["page"], case["dim"]
    if case["op"] == "append":
        q, nk, k, v = s["q"].double(), s["new_k"].double(), s["k"].double(), s["v"].double()
        half, t = case["rot"] // 2, 0
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        for n, (m, e) in enumerate(zip(lens, kv)):
            p = torch.arange(e - m, e, device="cuda")
            w = torch.complex(s["cos"][p].double(), s["sin"][p].double())[:, None]
            for x in (q[t:t + m], nk[t:t + m]):
                z = torch.complex(x[..., a], x[..., b]) * w
                x[..., a], x[..., b] = z.real, z.imag
            at = s["table"][n].long()[p // page]
            k[at, :, p % page], v[at, :, p % page] = nk[t:t + m], s["new_v"][t:t + m].double()
            t += m
        return {"q": q, "k": k, "v": v}
    G, t = case["hq"] // case["hkv"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for n, (m, e) in enumerate(zip(lens, kv)):
        p, j = torch.arange(e - m, e, device="cuda")[:, None], torch.arange(e, device="cuda")[None]
        hide = j > p
        if case.get("window"):
            hide |= (j <= p - case["window"]) & (j >= case["sinks"])
        at = s["table"][n, :-(-e // page)].long()
        for h in range(case["hkv"]):
            k, v = (s[w][at, h].reshape(-1, d)[:e].double() for w in ("k", "v"))
            q = s["q"][t:t + m, h * G:(h + 1) * G].double()
            z = torch.einsum("tgd,kd->gtk", q, k).div_(math.sqrt(d)).masked_fill_(hide, -math.inf)
            out[t:t + m, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", torch.softmax(z, -1), v)
        t += m
    return out
