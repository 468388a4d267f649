"""Measured cases of a serving step over a paged cache, and of its rotary positions.

A step takes a batch of requests, each with some new tokens (a chunk of its prompt,
or one token that it generated), packed one request after the other:

- ``append``: pages for the new tokens, and for every token its position and its slot
  of the cache (block tables and slot maps from request lengths);
- ``rope_append``: rotary positions on the projected queries and keys, the keys and
  values written to their slots;
- ``chunk``: the new tokens' attention over the pages, each token seeing the keys up to
  its own (under a sliding window with sinks: the last ones and the first);
- ``step``: the three in a row;
- ``rope_train``: the same rotary positions in training, forward and backward, between
  the projection and the attention's layout.

``run`` computes each in its plain form (elementary torch operations in 32 bits,
rounded once) while ``own`` is false, and calls the package's operators while it
is true.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")
ALL = 1 << 30  # a window that reaches every key


def listed():
    return [
        # A few chats, one token each: the smallest bookkeeping, where latency counts.
        {"name": "append_b8", "op": "append", "B": 8, "chunks": 0, "chunk": 1, "max_ctx": 3000,
         "page_size": 64, "max_pages": 64, "spare": 100, "pad": 0},
        # A large server's batch: 16 prompts in chunks of 509 between 1008 single tokens, long
        # tables, the token arrays padded to the size that a graph was captured with.
        {"name": "append_b1024_mixed", "op": "append", "B": 1024, "chunks": 16, "chunk": 509,
         "max_ctx": 30000, "page_size": 32, "max_pages": 1024, "spare": 5000, "pad": 40},
        # A training step of a grouped-query layer on one long sequence, whole heads rotated.
        {"name": "rope_train_gqa_s8192", "op": "rope_train", "B": 1, "S": 8192, "Hq": 32, "Hkv": 8,
         "D": 128, "R": 128, "style": 1, "grads": "bf16"},
        # A small multi-head model on packed rows of an odd length, half of each head rotated
        # in neighbouring pairs, gradients in 32 bits.
        {"name": "rope_train_mha_s1001_d64", "op": "rope_train", "B": 4, "S": 1001, "Hq": 12,
         "Hkv": 12, "D": 64, "R": 32, "style": 0, "grads": "fp32"},
        # One token each of 64 requests.
        {"name": "rope_append_t64", "op": "rope_append", "T": 64, "Hq": 32, "Hkv": 8, "D": 128,
         "R": 128, "style": 1, "page_size": 64, "num_pages": 512},
        # The tokens of several prompts at once.
        {"name": "rope_append_t8192", "op": "rope_append", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128,
         "R": 64, "style": 1, "page_size": 64, "num_pages": 512},
        # The smallest attention: one token of one chat with a two-head model.
        {"name": "chunk_1_of_300_d64", "op": "chunk", "B": 1, "chunks": 0, "chunk": 1, "min_ctx": 299,
         "max_ctx": 299, "Hq": 2, "Hkv": 2, "D": 64, "page_size": 32, "window": ALL, "sinks": 0},
        # Four whole prompts: bound by arithmetic.
        {"name": "chunk_prompts_4x2048", "op": "chunk", "B": 4, "chunks": 4, "chunk": 2048,
         "min_ctx": 0, "max_ctx": 0, "Hq": 32, "Hkv": 8, "D": 128, "page_size": 64, "window": ALL,
         "sinks": 0},
        # The last chunk of one long prompt: few rows against many keys.
        {"name": "chunk_500_of_16k", "op": "chunk", "B": 1, "chunks": 1, "chunk": 500,
         "min_ctx": 16000, "max_ctx": 16000, "Hq": 32, "Hkv": 8, "D": 128, "page_size": 64,
         "window": ALL, "sinks": 0},
        # A full serving batch: 62 single tokens of ragged lengths up to 16384 and two chunks.
        {"name": "chunk_mixed_b64", "op": "chunk", "B": 64, "chunks": 2, "chunk": 512, "min_ctx": 1000,
         "max_ctx": 16383, "Hq": 32, "Hkv": 8, "D": 128, "page_size": 64, "window": ALL, "sinks": 0},
        # Long chunks of two streams under the window and sinks of a streaming model.
        {"name": "chunk_window_2x2000_of_30k", "op": "chunk", "B": 2, "chunks": 2, "chunk": 2000,
         "min_ctx": 20000, "max_ctx": 30000, "Hq": 24, "Hkv": 8, "D": 64, "page_size": 32,
         "window": 4096, "sinks": 4},
        # A whole step of a layer, bookkeeping included: 30 single tokens and two chunks.
        {"name": "step_b32", "op": "step", "B": 32, "chunks": 2, "chunk": 250, "min_ctx": 100,
         "max_ctx": 4000, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "style": 0, "page_size": 64,
         "window": ALL, "sinks": 0, "spare": 40, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "rope_train", "rope_append", "chunk", "chunk", "step"])
    D = rng.choice([64, 128, 256] if op in ("rope_train", "rope_append") else [64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7])
    Hq = Hkv * min(group, 32 // Hkv)
    page = rng.choice([32, 64, 96, 128])
    style = rng.choice([0, 1])
    R = rng.choice([D, D, D // 2, 16, 48])
    if op == "append":
        B = _log_int(rng, 1, 1024)
        max_ctx = _log_int(rng, 40, 30000)
        chunk = _log_int(rng, 1, 600)
        return {"op": op, "B": B, "chunks": rng.randint(0, min(B, 16)), "chunk": chunk,
                "max_ctx": max_ctx, "page_size": page, "max_pages": (max_ctx + chunk) // page + 2,
                "spare": rng.randint(0, 3000), "pad": rng.choice([0, 1, 31, 100])}
    if op == "rope_train":
        return {"op": op, "B": rng.choice([1, 2, 3]), "S": _log_int(rng, 1, 2700), "Hq": Hq, "Hkv": Hkv,
                "D": D, "R": R, "style": style,
                "grads": rng.choice(["bf16", "fp32"])}
    if op == "rope_append":
        T = _log_int(rng, 1, 8192)
        return {"op": op, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R,
                "style": style, "page_size": page, "num_pages": T // page + rng.randint(2, 100)}
    # Attention: up to 500 new tokens in chunks, contexts up to 16000.
    B = _log_int(rng, 1, 64 if op == "chunk" else 32)
    chunks = rng.randint(0, min(B, 3))
    chunk = max(1, _log_int(rng, 1, 500) // max(chunks, 1))
    max_ctx = _log_int(rng, 1, 16000 if op == "chunk" and B <= 32 else 4000)
    windowed = rng.choice([False, False, True])
    c = {"op": op, "B": B, "chunks": chunks, "chunk": chunk, "min_ctx": rng.randint(0, max_ctx // 2),
         "max_ctx": max_ctx, "Hq": Hq, "Hkv": Hkv, "D": D, "page_size": page,
         "window": _log_int(rng, 1, 4096) if windowed else ALL,
         "sinks": rng.choice([0, 1, 4, rng.randint(5, 300)]) if windowed else 0}
    if op == "step":
        c.update(R=R, style=style, spare=rng.randint(0, 300), pad=rng.choice([0, 5]))
    return c


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _to_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _rope_table(max_pos, R):
    """cos and sin of each position's angles (a long context's base), rounded from 64 bits."""
    freq = 500000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.stack([torch.cos(angle), torch.sin(angle)], -1).float()


def _new_lens(c):
    return [c["chunk"]] * c["chunks"] + [1] * (c["B"] - c["chunks"])


def _contexts(c):
    """Cached tokens of each request: spread evenly, so that every seed has the same work."""
    lo, hi = c.get("min_ctx", c["max_ctx"] // 8), c["max_ctx"]
    return np.linspace(lo, hi, c["B"]).astype(np.int64) if c["B"] > 1 else np.array([hi])


def _requests(c, rng):
    """Cached and new tokens of each request, in an order and pairing of the seed's own (a
    chunk keeps the context that its place in the spread gives it)."""
    ctx, new = _contexts(c), np.array(_new_lens(c))
    places = np.linspace(0, c["B"] - 1, c["chunks"] + 2)[1:-1].astype(int)  # of the chunks
    places = np.unique(places)
    singles = np.setdiff1d(np.arange(c["B"]), places)
    if len(places) < c["chunks"]:
        extra = c["chunks"] - len(places)
        places, singles = np.concatenate([places, singles[:extra]]), singles[extra:]
    ctx = ctx[np.concatenate([places, singles])]
    order = rng.permutation(c["B"])
    return ctx[order], new[order]


def _held_pages(c, ctx, rng, spare):
    """A table whose rows hold the pages of their contexts, from a pool with ``spare`` more
    pages than the step needs."""
    ps, M, B = c["page_size"], c["max_pages"], c["B"]
    pages = -(-ctx // ps)
    total = int(sum(-(-(int(x) + n) // ps) for x, n in zip(ctx, c["new"])))
    P = total + spare + 1
    ids = rng.permutation(P)
    base = np.concatenate([[0], np.cumsum(pages)])[:-1]
    slot = np.arange(M)[None, :]
    have = slot < pages[:, None]
    table = np.where(have, ids[np.where(have, base[:, None] + slot, 0)], -1)
    return table, np.bincount(table[table >= 0], minlength=P)


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    rng = np.random.default_rng(seed)
    op = c["op"]
    s = {"case": c}
    N = (c.get("Hq", 0) + 2 * c.get("Hkv", 0)) * c.get("D", 0)
    if op == "rope_train":
        B, S, Hq, Hkv, D = (c[n] for n in ("B", "S", "Hq", "Hkv", "D"))
        dtype = torch.bfloat16 if c["grads"] == "bf16" else torch.float32
        s["qkv"] = _normal(g, B, S, N)
        s["table"] = _rope_table(S, c["R"])
        s["dq"] = _normal(g, B, Hq, S, D, dtype=dtype)
        s["dk"] = _normal(g, B, Hkv, S, D, dtype=dtype)
        s["dv"] = _normal(g, B, Hkv, S, D, dtype=dtype)
        return s
    if op == "rope_append":
        T, P, ps = c["T"], c["num_pages"], c["page_size"]
        s["qkv"] = _normal(g, T, N)
        s["table"] = _rope_table(20000, c["R"])
        s["positions"] = _to_gpu(rng.integers(0, 20000, T))
        s["slots"] = _to_gpu(rng.permutation(P * ps)[:T])
        s["k_cache"] = _normal(g, P, c["Hkv"], ps, c["D"])
        s["v_cache"] = _normal(g, P, c["Hkv"], ps, c["D"])
        return s
    ctx, new = _requests(c, rng)
    c["ctx"], c["new"] = ctx, new
    ps = c["page_size"]
    c["cu"] = np.concatenate([[0], np.cumsum(new)])
    c["T"] = int(new.sum()) + c.get("pad", 0)
    if op == "chunk":
        # The step's pages are there and written: lengths count the new tokens.
        length = ctx + new
        c["max_pages"] = int(-(-length.max() // ps)) + 1
        c["new"] = np.zeros_like(new)
        table, refs = _held_pages(c, length, rng, 2)
        c["new"] = new
        s["seqlens"], s["cu"] = _to_gpu(length), _to_gpu(c["cu"])
        s["q"] = _normal(g, c["T"], c["Hq"], c["D"])
    else:
        if op == "step":
            c["max_pages"] = int(-(-(ctx + new).max() // ps)) + 1
            s["qkv"] = _normal(g, c["T"], N)
            s["rope"] = _rope_table(c["max_ctx"] + c["chunk"] + 1, c["R"])
        table, refs = _held_pages(c, ctx, rng, c["spare"])
        s["refs"], s["seqlens"], s["new"] = _to_gpu(refs), _to_gpu(ctx), _to_gpu(new)
    s["table"] = _to_gpu(table)
    if op in ("chunk", "step"):
        s["k_cache"] = _normal(g, refs.size, c["Hkv"], ps, c["D"])
        s["v_cache"] = _normal(g, refs.size, c["Hkv"], ps, c["D"])
        # The plain form's plan: requests with the same number of new tokens, at most eight
        # chunks at once (new tokens, longest request, rows, lengths, first tokens).
        length, s["groups"] = ctx + new, []
        for n in sorted(set(new.tolist())):
            same = np.nonzero(new == n)[0]
            step = len(same) if n == 1 else 8
            for rows in [same[i:i + step] for i in range(0, len(same), step)]:
                s["groups"].append((n, int(length[rows].max())) + tuple(
                    torch.from_numpy(a[rows]).cuda() for a in (np.arange(c["B"]), length, c["cu"])))
    if own and op == "chunk":
        # One plan serves the layers of a step; a step's own is part of its pass.
        import tensor_attn_fwd_gb300 as attn
        s["plan"] = attn.attn_chunk_plan(s["cu"], s["seqlens"], c["T"], c["Hq"], c["Hkv"], c["D"],
                                         c["max_pages"] * ps, c["window"], c["sinks"])
    return s


# ------------------------------------------------------------------ plain forms
def _plain_append(s):
    c = s["case"]
    ps, T = c["page_size"], c["T"]
    table, refs, length, new = s["table"], s["refs"], s["seqlens"], s["new"]
    B, M = table.shape
    P = refs.numel()
    end = length + new
    takes = (length >= 0) & (end <= M * ps) & (new > 0)
    slot = torch.arange(M, device="cuda")[None, :]
    lo, hi = length // ps, torch.where(takes, (end + ps - 1) // ps, 0)
    missing = (slot >= lo[:, None]) & (slot < hi[:, None]) & (table < 0)
    need = missing.sum(1)
    n_free = (refs == 0).sum()
    takes &= need.cumsum(0) <= n_free
    missing &= takes[:, None]
    rank = (missing.reshape(-1).cumsum(0) - 1).view(B, M)
    order = torch.argsort((refs != 0).int(), stable=True).int()  # free ids first, ascending
    table = torch.where(missing, order[rank.clamp(min=0, max=P - 1)], table)
    given = torch.where(missing, table, 0).reshape(-1)
    refs = refs.index_add(0, given, missing.reshape(-1).int())
    out_len = torch.where(takes, end, length)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)])
    t = torch.arange(T, device="cuda")
    row = torch.searchsorted(cu, t, right=True) - 1
    mine = (row < B) & takes[row.clamp(max=B - 1)]
    row = row.clamp(max=B - 1)
    pos = torch.where(mine, length[row] + t - cu[row], 0)
    page = table.view(-1)[row * M + pos // ps]
    slots = torch.where(mine, page * ps + pos % ps, -1)
    counts = torch.stack([need.sum(), n_free]).int()
    return {"table": table, "refs": refs, "seqlens": out_len, "cu": cu.int(), "positions": pos.int(),
            "slots": slots.int(), "counts": counts}


def _rotate(x, cs, style, sign=1.0):
    """The first R dims of each head turned by its token's angles; x [..., heads, D] in 32
    bits, cs [..., R/2, 2]."""
    R = 2 * cs.shape[-2]
    cos, sin = cs[..., None, :, 0], sign * cs[..., None, :, 1]
    turned, rest = x[..., :R], x[..., R:]
    if style == 0:
        a, b = turned[..., 0::2], turned[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., : R // 2], turned[..., R // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, rest], -1)


def _plain_rope_train(s):
    c = s["case"]
    B, S, Hq, Hkv, D = (c[n] for n in ("B", "S", "Hq", "Hkv", "D"))
    bf16 = torch.bfloat16
    x = s["qkv"].float().view(B, S, Hq + 2 * Hkv, D)
    cs = s["table"][:S]
    y = _rotate(x[:, :, : Hq + Hkv], cs, c["style"]).to(bf16).transpose(1, 2)
    out = {"q": y[:, :Hq].contiguous(), "k": y[:, Hq:].contiguous(),
           "v": x[:, :, Hq + Hkv:].to(bf16).transpose(1, 2).contiguous()}
    d = torch.cat([s["dq"], s["dk"]], 1).float().transpose(1, 2)
    d = torch.cat([_rotate(d, cs, c["style"], -1.0), s["dv"].float().transpose(1, 2)], 2)
    out["dqkv"] = d.to(bf16).reshape(B, S, -1)
    return out


def _plain_rope_append(s, qkv, rope, positions, slots, used):
    """``used`` leading tokens have slots."""
    c = s["case"]
    Hq, Hkv, D, ps = (c[n] for n in ("Hq", "Hkv", "D", "page_size"))
    x = qkv.float().view(-1, Hq + 2 * Hkv, D)
    y = _rotate(x[:, : Hq + Hkv], rope[positions.long()], c["style"]).to(torch.bfloat16)
    slot = slots[:used].long()
    page, at = slot // ps, slot % ps
    s["k_cache"][page, :, at] = y[:used, Hq:]
    s["v_cache"][page, :, at] = x[:used, Hq + Hkv:].to(torch.bfloat16)
    return y[:, :Hq].contiguous()


def _softmax(x):
    """exp(x - lse) and lse over the last axis; rows of -inf give 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    e = e / torch.where(total == 0, torch.ones_like(total), total)
    return e, (m + torch.log(total)).squeeze(-1)


def _plain_chunk(s, q, table):
    """Requests with as many new tokens as each other at once."""
    c = s["case"]
    Hq, Hkv, D, ps = (c[n] for n in ("Hq", "Hkv", "D", "page_size"))
    window, sinks, M = c["window"], c["sinks"], c["max_pages"]
    G = Hq // Hkv
    o = torch.zeros(c["T"], Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(c["T"], Hq, device="cuda")
    for n, most, b, L, first_t in s["groups"]:
        rows = b.numel()
        t = first_t[:, None] + torch.arange(n, device="cuda")
        if window >= ALL:
            slot = torch.arange(-(-most // ps), device="cuda").expand(rows, -1)
        else:  # the slots that the window and the sinks reach
            ns = min(M, -(-sinks // ps))
            nw = min(M, (window + n + ps - 2) // ps + 1)
            first = ((L - n - window + 1).clamp(min=0) // ps).clamp(min=ns)[:, None]
            slot = torch.cat([torch.arange(ns, device="cuda").expand(rows, ns),
                              first + torch.arange(nw, device="cuda")], 1)
        key = (slot[:, :, None] * ps + torch.arange(ps, device="cuda")).view(rows, 1, -1)
        p = (L[:, None] - n + torch.arange(n, device="cuda"))[:, :, None]
        seen = (key <= p) & ((key > p - window) | (key < sinks))
        page = torch.gather(table[b].long(), 1, slot.clamp(max=M - 1)).clamp(min=0)
        k = s["k_cache"][page].permute(0, 2, 1, 3, 4).reshape(rows, Hkv, -1, D).float()
        x = q[t].view(rows, n, Hkv, G, D).permute(0, 2, 3, 1, 4).float()
        x = torch.matmul(x.reshape(rows, Hkv, G * n, D), k.transpose(-1, -2))
        del k
        x = x.view(rows, Hkv, G, n, -1).mul_(1.0 / math.sqrt(D))
        w, z = _softmax(x.masked_fill_(~seen[:, None, None], NEG))
        del x
        v = s["v_cache"][page].permute(0, 2, 1, 3, 4).reshape(rows, Hkv, -1, D).float()
        y = torch.matmul(w.view(rows, Hkv, G * n, -1), v)
        del w, v
        y = y.view(rows, Hkv, G, n, D).permute(0, 3, 1, 2, 4).reshape(rows, n, Hq, D)
        o[t] = y.to(torch.bfloat16)
        lse[t] = z.permute(0, 3, 1, 2).reshape(rows, n, Hq)
    return {"o": o, "lse": lse}


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "append":
        return _plain_append(s)
    if op == "rope_train":
        return _plain_rope_train(s)
    if op == "rope_append":
        q = _plain_rope_append(s, s["qkv"], s["table"], s["positions"], s["slots"], c["T"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "chunk":
        return _plain_chunk(s, s["q"], s["table"])
    out = _plain_append(s)
    out["q"] = _plain_rope_append(s, s["qkv"], s["rope"], out["positions"], out["slots"],
                                  int(c["cu"][-1]))
    out.update(_plain_chunk(s, out["q"], out["table"]))
    out.update(k_cache=s["k_cache"], v_cache=s["v_cache"])
    return out


# ------------------------------------------------------------------ the package's operators
def _own_append(attn, s):
    names = ("table", "refs", "seqlens", "cu", "positions", "slots", "counts")
    return dict(zip(names, attn.attn_pages_append(s["table"], s["refs"], s["seqlens"], s["new"],
                                                  s["case"]["T"], s["case"]["page_size"])))


def _own_chunk(attn, s, q, table, plan):
    """Tokens behind the last request are left as they were: as zeros, here."""
    c = s["case"]
    if c.get("pad", 0) == 0:
        o, lse = attn.attn_chunk_paged(q, s["k_cache"], s["v_cache"], table, plan)
    else:
        o, lse = attn.attn_chunk_paged(q, s["k_cache"], s["v_cache"], table, plan,
                                       o=torch.zeros_like(q),
                                       lse=torch.zeros(c["T"], c["Hq"], device="cuda"))
    return {"o": o, "lse": lse}


def _own(s):
    import tensor_attn_fwd_gb300 as attn
    c = s["case"]
    op = c["op"]
    if op == "append":
        return _own_append(attn, s)
    if op == "rope_train":
        q, k, v = attn.attn_rope_split(s["qkv"], s["table"], c["Hq"], c["Hkv"], style=c["style"])
        dqkv = attn.attn_rope_split_bwd(s["dq"], s["dk"], s["dv"], s["table"], style=c["style"])
        return {"q": q, "k": k, "v": v, "dqkv": dqkv}
    if op == "rope_append":
        q = attn.attn_rope_append(s["qkv"], s["table"], s["positions"], s["slots"], s["k_cache"],
                                  s["v_cache"], c["Hq"], style=c["style"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "chunk":
        return _own_chunk(attn, s, s["q"], s["table"], s["plan"])
    out = _own_append(attn, s)
    plan = attn.attn_chunk_plan(out["cu"], out["seqlens"], c["T"], c["Hq"], c["Hkv"], c["D"],
                                c["max_pages"] * c["page_size"], c["window"], c["sinks"])
    out["q"] = attn.attn_rope_append(s["qkv"], s["rope"], out["positions"], out["slots"],
                                     s["k_cache"], s["v_cache"], c["Hq"], style=c["style"])
    out.update(_own_chunk(attn, s, out["q"], out["table"], plan))
    out.update(k_cache=s["k_cache"], v_cache=s["v_cache"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def _attention_work(c):
    """Keys that some token of a request sees are read once; (token, key) pairs are counted."""
    ctx, new = _requests(c, np.random.default_rng(0))
    keys = pairs = 0
    for x, n in zip(ctx.tolist(), new.tolist()):
        p = x + np.arange(n, dtype=np.int64)
        first = np.maximum(p - c["window"] + 1, 0)
        pairs += int((p + 1 - first + np.minimum(first, c["sinks"])).sum())
        keys += x + n - int(first[0]) + min(int(first[0]), c["sinks"])
    T = int(new.sum())
    q = T * c["Hq"] * c["D"] * 2
    return 2 * keys * c["Hkv"] * c["D"] * 2 + 2 * q + T * c["Hq"] * 4, 4 * pairs * c["Hq"] * c["D"]


def _append_bytes(c):
    ctx, new = _requests(c, np.random.default_rng(0))
    T = int(new.sum()) + c["pad"]
    M = c.get("max_pages", (int((ctx + new).max()) + c["page_size"] - 1) // c["page_size"] + 1)
    P = int(sum(-(-(int(x) + n) // c["page_size"]) for x, n in zip(ctx, new))) + c["spare"] + 1
    return 4 * (2 * c["B"] * M + 2 * P + 4 * c["B"] + 2 * T)


def _rope_bytes(c, T):
    """The projected rows read and written once."""
    return T * (2 * (c["Hq"] + 2 * c["Hkv"]) * c["D"] * 2 + c["R"] * 4)


def work(case):
    c = case
    op = c["op"]
    if op == "append":
        return {"bytes": _append_bytes(c), "flops": 0}
    if op == "rope_append":
        return {"bytes": _rope_bytes(c, c["T"]) + 8 * c["T"], "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["R"]}
    if op == "rope_train":
        T, N = c["B"] * c["S"], (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        size = 2 if c["grads"] == "bf16" else 4
        return {"bytes": T * N * (2 + 2 + size + 2) + c["S"] * c["R"] * 4,
                "flops": 6 * T * (c["Hq"] + c["Hkv"]) * c["R"]}
    b, f = _attention_work(c)
    if op == "step":
        T = c["chunks"] * (c["chunk"] - 1) + c["B"] + c["pad"]
        b += _append_bytes(c) + _rope_bytes(c, T) + 8 * T
        f += 3 * T * (c["Hq"] + c["Hkv"]) * c["R"]
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ 64 bits
def _exact_append(s):
    c = s["case"]
    ps, T = c["page_size"], c["T"]
    table, refs = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    length, new = s["seqlens"].tolist(), s["new"].tolist()
    free = [int(p) for p in np.nonzero(refs == 0)[0]]
    counts, out_len, cu = [0, len(free)], list(length), [0]
    positions, slots = np.zeros(T, dtype=np.int64), np.full(T, -1, dtype=np.int64)
    for b, (x, n) in enumerate(zip(length, new)):
        at = cu[-1]
        cu.append(at + n)
        if n == 0 or x < 0 or x + n > table.shape[1] * ps:
            continue
        want = [j for j in range(x // ps, (x + n - 1) // ps + 1) if table[b, j] < 0]
        counts[0] += len(want)
        if counts[0] > counts[1]:
            continue
        for j in want:
            table[b, j] = free.pop(0)
            refs[table[b, j]] = 1
        out_len[b] = x + n
        for i in range(n):
            positions[at + i] = x + i
            slots[at + i] = table[b, (x + i) // ps] * ps + (x + i) % ps
    return {"table": table, "refs": refs, "seqlens": np.array(out_len), "cu": np.array(cu),
            "positions": positions, "slots": slots, "counts": np.array(counts)}


def _exact_turn(x, cs, style):
    """Heads [..., H, D] of 64 bits, their first dims as complex numbers times cs [...]."""
    R = 2 * cs.shape[-1]
    y = x.clone()
    if style == 0:
        z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2).contiguous())
        y[..., :R] = torch.view_as_real(z * cs.unsqueeze(-2)).reshape(*x.shape[:-1], R)
    else:
        z = torch.complex(x[..., : R // 2], x[..., R // 2: R]) * cs.unsqueeze(-2)
        y[..., : R // 2], y[..., R // 2: R] = z.real, z.imag
    return y


def _exact_rope_train(s):
    c = s["case"]
    B, S, Hq, Hkv, D = (c[n] for n in ("B", "S", "Hq", "Hkv", "D"))
    cs = torch.view_as_complex(s["table"][:S].double())
    x = s["qkv"].double().reshape(B, S, -1, D)
    out = {"q": _exact_turn(x[:, :, :Hq], cs, c["style"]).permute(0, 2, 1, 3),
           "k": _exact_turn(x[:, :, Hq:Hq + Hkv], cs, c["style"]).permute(0, 2, 1, 3),
           "v": x[:, :, Hq + Hkv:].permute(0, 2, 1, 3)}
    parts = [_exact_turn(s[n].double().permute(0, 2, 1, 3), cs.conj().resolve_conj(), c["style"])
             for n in ("dq", "dk")]
    out["dqkv"] = torch.cat(parts + [s["dv"].double().permute(0, 2, 1, 3)], 2).reshape(B, S, -1)
    return out


def _exact_rope_append(s, qkv, rope, positions, slots, kc, vc):
    c = s["case"]
    Hq, Hkv, D, ps = (c[n] for n in ("Hq", "Hkv", "D", "page_size"))
    x = qkv.double().reshape(qkv.shape[0], -1, D)
    cs = torch.view_as_complex(rope.double())[positions.long()]
    k = _exact_turn(x[:, Hq:Hq + Hkv], cs, c["style"])
    for t, slot in enumerate(slots.tolist()):
        if slot >= 0:
            kc[slot // ps, :, slot % ps] = k[t]
            vc[slot // ps, :, slot % ps] = x[t, Hq + Hkv:]
    return _exact_turn(x[:, :Hq], cs, c["style"])


def _exact_chunk(s, q, table, kc, vc):
    c = s["case"]
    Hq, Hkv, D, ps = (c[n] for n in ("Hq", "Hkv", "D", "page_size"))
    G, window, sinks = Hq // Hkv, c["window"], c["sinks"]
    o = torch.zeros(c["T"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["T"], Hq, dtype=torch.float64, device="cuda")
    for b, (x, n) in enumerate(zip(c["ctx"].tolist(), c["new"].tolist())):
        pages = table[b].long()
        for i0 in range(0, n, 256):
            i1 = min(n, i0 + 256)
            start = max(0, x + i0 - window + 1)
            t = torch.cat([torch.arange(0, min(sinks, start), device="cuda"),
                           torch.arange(start, x + i1, device="cuda")])
            pos = torch.arange(x + i0, x + i1, device="cuda")[:, None]
            seen = (t <= pos) & ((pos - t < window) | (t < sinks))
            rows = slice(int(c["cu"][b]) + i0, int(c["cu"][b]) + i1)
            for h in range(Hkv):
                k, v = kc[pages[t // ps], h, t % ps].double(), vc[pages[t // ps], h, t % ps].double()
                heads = slice(h * G, (h + 1) * G)
                y = torch.einsum("nrd,kd->rnk", q[rows, heads].double(), k) / math.sqrt(D)
                y = torch.where(seen, y, NEG)
                z = torch.logsumexp(y, -1)
                o[rows, heads] = torch.einsum("rnk,kd->nrd", torch.exp(y - z[..., None]), v)
                lse[rows, heads] = z.T
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "append":
        return _exact_append(s)
    if op == "rope_train":
        return _exact_rope_train(s)
    if op == "chunk":
        return _exact_chunk(s, s["q"], s["table"], s["k_cache"], s["v_cache"])
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    if op == "rope_append":
        q = _exact_rope_append(s, s["qkv"], s["table"], s["positions"], s["slots"], kc, vc)
        return {"q": q, "k_cache": kc, "v_cache": vc}
    out = _exact_append(s)
    table = torch.from_numpy(out["table"]).cuda()
    positions, slots = torch.from_numpy(out["positions"]).cuda(), torch.from_numpy(out["slots"]).cuda()
    # q, the cached keys and values are rounded to 16 bits before the attention reads them.
    out["q"] = _exact_rope_append(s, s["qkv"], s["rope"], positions, slots, kc, vc)
    bf16 = torch.bfloat16
    out.update(_exact_chunk(s, out["q"].to(bf16), table, kc.to(bf16), vc.to(bf16)))
    out.update(k_cache=kc, v_cache=vc)
    return out
