"""Measured cases of the bounded-cache operators.

Two families that a streaming server or a long-context trainer runs together:
attention with a sliding window and sinks (training step, prefill of a chunk,
decode of one token over a paged cache), and the bookkeeping of the pages that
such a cache is made of (fork, free, compact, and the page copies they list).

``run`` computes each in its plain form (elementary torch operations in 32 bits,
rounded once) while ``own`` is false, and calls the package's operators while it
is true.  ``exact`` gives the same outputs from the definitions in 64 bits.

Visibility: query row i stands at position p = i + Sk - Sq and sees key j when
j <= p and (j > p - window or j < sinks).  Tables hold page ids (-1: no page),
``refs[p]`` counts the holders of page p (0: free).
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")


def listed():
    return [
        # A training step (forward, then backward) of a grouped-query layer on one
        # long sequence: the window and four sinks of a streaming model.
        {"name": "train_gqa_s8192_w1024", "op": "train", "B": 1, "Hq": 32, "Hkv": 8, "Sq": 8192,
         "Sk": 8192, "D": 128, "window": 1024, "sinks": 4},
        # A small multi-head model trained on packed rows of an odd length.
        {"name": "train_mha_s1000_w200_d64", "op": "train", "B": 4, "Hq": 16, "Hkv": 16, "Sq": 1000,
         "Sk": 1000, "D": 64, "window": 200, "sinks": 0},
        # A 512-token chunk of a long prompt against what the cache holds so far.
        {"name": "chunk_gqa_512_of_16384_w4096", "op": "prefill", "B": 1, "Hq": 32, "Hkv": 8,
         "Sq": 512, "Sk": 16384, "D": 128, "window": 4096, "sinks": 128},
        # The smallest call: one short prompt of a two-head model, where latency counts.
        {"name": "prefill_mha_s128_w32_d64", "op": "prefill", "B": 1, "Hq": 2, "Hkv": 2, "Sq": 128,
         "Sk": 128, "D": 64, "window": 32, "sinks": 1},
        # A full serving batch, ragged lengths up to 16384, one token each.
        {"name": "decode_b64_w4096", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "D": 128,
         "page_size": 64, "max_len": 16384, "window": 4096, "sinks": 4},
        # One user's chat far into its stream: split over the window.
        {"name": "decode_b1_w1024", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page_size": 64, "max_len": 30000, "window": 1024, "sinks": 4},
        # Eight beams of one prompt reordered after a step.
        {"name": "fork_8_beams", "op": "fork", "groups": 1, "beams": 8, "Hkv": 8, "D": 128,
         "page_size": 64, "max_pages": 64, "num_pages": 640, "max_len": 3000, "room": 1},
        # 64 prompts of eight samples each: every group re-forked from its survivors.
        {"name": "fork_64x8_beams", "op": "fork", "groups": 64, "beams": 8, "Hkv": 8, "D": 128,
         "page_size": 64, "max_pages": 256, "num_pages": 8192, "max_len": 4000, "room": 33},
        # The window moved on in a small batch: pages it has passed are given up.
        {"name": "free_b8", "op": "free", "B": 8, "max_pages": 48, "page_size": 64, "window": 1024,
         "sinks": 4},
        # A large batch with long tables, finished rows among them.
        {"name": "free_b1024", "op": "free", "B": 1024, "max_pages": 2048, "page_size": 32,
         "window": 4096, "sinks": 128},
        # A small pool packed before its tail is handed back.
        {"name": "compact_p300", "op": "compact", "B": 7, "max_pages": 40, "num_pages": 300,
         "Hkv": 2, "D": 64, "page_size": 32, "live": 0.5},
        # A server's pool, half of it scattered over all ids.
        {"name": "compact_p16384", "op": "compact", "B": 256, "max_pages": 64, "num_pages": 16384,
         "Hkv": 4, "D": 128, "page_size": 64, "live": 0.55},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["train", "prefill", "decode", "fork", "free", "compact"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4])
    sinks = rng.choice([0, 1, 4, rng.randint(5, 300)])
    if op == "train":
        S = _log_int(rng, 100, 3000)
        B = rng.choice([1, 2])
        # From a window of 8: with one visible key dQ and dK are zero but for rounding.
        return {"op": op, "B": B, "Hq": Hkv * group, "Hkv": Hkv, "Sq": S, "Sk": S, "D": D,
                "window": _log_int(rng, 8, min(S, 1024)), "sinks": sinks}
    if op == "prefill":
        Sq = _log_int(rng, 1, 2048)
        Sk = Sq + rng.choice([0, _log_int(rng, 1, 12000)])
        return {"op": op, "B": rng.choice([1, 2]), "Hq": Hkv * group, "Hkv": Hkv, "Sq": Sq,
                "Sk": Sk, "D": D, "window": _log_int(rng, 1, min(Sk, 4096)), "sinks": sinks}
    if op == "decode":
        max_len = _log_int(rng, 40, 16384)
        return {"op": op, "B": _log_int(rng, 1, 64), "Hq": Hkv * group, "Hkv": Hkv,
                "D": rng.choice([64, 128, 256]), "page_size": rng.choice([32, 64, 96, 128]),
                "max_len": max_len, "window": _log_int(rng, 1, max_len), "sinks": sinks}
    if op == "fork":
        groups, beams = _log_int(rng, 1, 64), rng.randint(1, 8)
        page = rng.choice([32, 64, 96])
        max_len = _log_int(rng, 40, 4000)
        room = rng.randint(0, 100)
        max_pages = (max_len + room) // page + 2
        spare = room // page + 3
        return {"op": op, "groups": groups, "beams": beams, "Hkv": Hkv, "D": D, "page_size": page,
                "max_pages": max_pages, "max_len": max_len, "room": room,
                "num_pages": groups * (max_len // page + 1 + 3 * beams) + groups * beams * spare}
    if op == "free":
        B = _log_int(rng, 1, 1024)
        page = rng.choice([32, 64, 128])
        max_pages = _log_int(rng, 2, 2048)
        return {"op": op, "B": B, "max_pages": max_pages, "page_size": page,
                "window": _log_int(rng, 1, max_pages * page), "sinks": sinks}
    B = _log_int(rng, 1, 256)
    num_pages = _log_int(rng, 50, 8000)
    return {"op": op, "B": B, "max_pages": _log_int(rng, 2, 64), "num_pages": num_pages, "Hkv": Hkv,
            "D": D, "page_size": rng.choice([32, 64]), "live": rng.uniform(0.05, 0.95)}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _to_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _fork_tables(c, rng):
    """Rows of ``groups`` prompts with ``beams`` beams each: a beam shares its
    group's prompt pages and holds one to three pages of its own."""
    G, K, ps, M = c["groups"], c["beams"], c["page_size"], c["max_pages"]
    ids = rng.permutation(c["num_pages"])
    rows = G * K
    most = c["max_len"]
    length = np.repeat(rng.integers(max(1, most // 2), most + 1, G), K)
    pages = -(-length // ps)
    tail = np.minimum(np.repeat(rng.integers(1, 4, G), K), pages)  # pages of the beam's own
    shared = pages - tail
    group = np.arange(rows) // K
    shared_of = shared[::K]
    base = np.concatenate([[0], np.cumsum(shared_of)])[:-1]
    slot = np.arange(M)[None, :]
    own_base = int(shared_of.sum()) + np.concatenate([[0], np.cumsum(tail)])[:-1]
    at = np.where(slot < shared[:, None], base[group][:, None] + slot,
                  own_base[:, None] + slot - shared[:, None])
    have = slot < pages[:, None]
    table = np.where(have, ids[np.where(have, at, 0)], -1)
    refs = np.bincount(table[table >= 0], minlength=c["num_pages"])
    # Survivors: the beams that a selection keeps, several children for the best.
    parents = group * K + np.minimum(rng.integers(0, K, rows), rng.integers(0, K, rows))
    return table, refs, length, parents


def _free_tables(c, rng):
    """Long rows whose first half is shared by pairs; an eighth of them finished."""
    B, M, ps = c["B"], c["max_pages"], c["page_size"]
    length = rng.integers(0, M * ps + 1, B)
    length[rng.random(B) < 0.125] = 0
    held = rng.integers((length + ps - 1) // ps, M + 1)  # pages reserved past the keys too
    slot = np.arange(M)[None, :]
    owner = np.where(slot < M // 2, np.arange(B)[:, None] // 2, (B + 1) // 2 + np.arange(B)[:, None])
    ids = rng.permutation(((B + 1) // 2 + B) * M)
    table = np.where(slot < held[:, None], ids[owner * M + slot], -1)
    refs = np.bincount(table[table >= 0], minlength=ids.size)
    return table, refs, length


def _compact_tables(c, rng):
    """Rows over the live pages of a pool, live ids scattered over all of it."""
    P, B, M = c["num_pages"], c["B"], c["max_pages"]
    n = max(1, int(P * c["live"]))
    live = rng.permutation(P)[:n]
    # Every live page once while the table has entries, the rest shared prefixes.
    flat = np.where(np.arange(B * M) < n, np.arange(B * M) % n, rng.integers(0, n, B * M))
    table = live[rng.permutation(flat).reshape(B, M)]
    table = np.where(rng.random((B, M)) < 0.1, -1, table)  # pages that a window has passed
    refs = np.bincount(table[table >= 0], minlength=P)
    return table, refs


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    rng = np.random.default_rng(seed)
    op = c["op"]
    s = {"case": c}
    if op in ("train", "prefill"):
        s["q"] = _normal(g, c["B"], c["Hq"], c["Sq"], c["D"])
        s["k"] = _normal(g, c["B"], c["Hkv"], c["Sk"], c["D"])
        s["v"] = _normal(g, c["B"], c["Hkv"], c["Sk"], c["D"])
        if op == "train":
            s["dout"] = _normal(g, c["B"], c["Hq"], c["Sq"], c["D"])
    elif op == "decode":
        B, ps, most = c["B"], c["page_size"], c["max_len"]
        length = rng.integers(max(1, most // 4), most + 1, B) if B > 1 else np.array([most])
        M = -(-most // ps)
        P = B * M + 3
        s["q"] = _normal(g, B, c["Hq"], 1, c["D"])
        s["k_cache"] = _normal(g, P, c["Hkv"], ps, c["D"])
        s["v_cache"] = _normal(g, P, c["Hkv"], ps, c["D"])
        s["table"] = _to_gpu(rng.permutation(P)[: B * M].reshape(B, M))
        s["seqlens"] = _to_gpu(length)
    elif op == "fork":
        table, refs, length, parents = _fork_tables(c, rng)
        s.update(table=_to_gpu(table), refs=_to_gpu(refs), seqlens=_to_gpu(length),
                 parents=_to_gpu(parents))
    elif op == "free":
        table, refs, length = _free_tables(c, rng)
        s.update(table=_to_gpu(table), refs=_to_gpu(refs), seqlens=_to_gpu(length))
    else:
        table, refs = _compact_tables(c, rng)
        s.update(table=_to_gpu(table), refs=_to_gpu(refs))
    if op in ("fork", "compact"):
        s["k_cache"] = _normal(g, c["num_pages"], c["Hkv"], c["page_size"], c["D"])
        s["v_cache"] = _normal(g, c["num_pages"], c["Hkv"], c["page_size"], c["D"])
    return s


# ------------------------------------------------------------------ plain forms
def _visible(Sq, Sk, window, sinks):
    p = torch.arange(Sq, device="cuda")[:, None] + (Sk - Sq)
    j = torch.arange(Sk, device="cuda")[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def _softmax(x):
    """exp(x - lse) and lse over the last axis; rows of -inf give 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == NEG, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    e = e / torch.where(total == 0, torch.ones_like(total), total)
    return e, (m + torch.log(total)).squeeze(-1)


def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, Sq, Sk, D = (c[n] for n in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    scale = 1.0 / math.sqrt(D)
    n = Hq // Hkv
    q = s["q"].float().view(B, Hkv, n * Sq, D)  # the heads of a group beside each other
    k, v = s["k"].float(), s["v"].float()
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, Hkv, n, Sq, Sk) * scale
    x = x.masked_fill_(~_visible(Sq, Sk, c["window"], c["sinks"]), NEG)
    p, lse = _softmax(x)
    del x
    o = torch.matmul(p.view(B, Hkv, n * Sq, Sk), v)
    out = {"o": o.view(B, Hq, Sq, D).to(torch.bfloat16), "lse": lse.view(B, Hq, Sq)}
    if c["op"] == "train":
        do = s["dout"].float().view(B, Hkv, n * Sq, D)
        p = p.view(B, Hkv, n * Sq, Sk)
        out["dv"] = torch.matmul(p.transpose(-1, -2), do).to(torch.bfloat16)
        ds = torch.matmul(do, v.transpose(-1, -2))
        ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out["dq"] = torch.matmul(ds, k).view(B, Hq, Sq, D).to(torch.bfloat16)
        out["dk"] = torch.matmul(ds.transpose(-1, -2), q).to(torch.bfloat16)
    return out


def _plain_decode(s):
    c = s["case"]
    B, Hq, Hkv, D, ps = (c[n] for n in ("B", "Hq", "Hkv", "D", "page_size"))
    window, sinks = c["window"], c["sinks"]
    M = s["table"].shape[1]
    # The slots of a row that the window and the sinks can reach, gathered.
    length = s["seqlens"].long()[:, None]
    ns = min(M, -(-sinks // ps))
    nw = min(M, (window + ps - 2) // ps + 1)
    first = ((length - window).clamp(min=0) // ps).clamp(min=ns)
    slot = torch.cat([torch.arange(ns, device="cuda").expand(B, ns),
                      first + torch.arange(nw, device="cuda")], 1)
    key = (slot[:, :, None] * ps + torch.arange(ps, device="cuda")).view(B, -1)
    seen = (key < length) & ((key >= length - window) | (key < sinks))
    page = torch.gather(s["table"].long(), 1, slot.clamp(max=M - 1))
    n = key.shape[1]
    k = s["k_cache"][page].permute(0, 2, 1, 3, 4).reshape(B, Hkv, n, D).float()
    v = s["v_cache"][page].permute(0, 2, 1, 3, 4).reshape(B, Hkv, n, D).float()
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    p, lse = _softmax(x.masked_fill(~seen[:, None, None, :], NEG))
    return {"o": torch.matmul(p, v).view(B, Hq, D).to(torch.bfloat16), "lse": lse.view(B, Hq)}


def _plain_copy(s, src, dst):
    """Page dst[i] takes page src[i] in both caches.  A pair of -1 repeats the first
    pair (or copies page 0 onto itself when there is none)."""
    use = dst >= 0
    first = torch.where(use.any(), use.int().argmax(), torch.zeros_like(use.int().argmax()))
    src0, dst0 = src[first].clamp(min=0), dst[first].clamp(min=0)
    src, dst = torch.where(use, src, src0).long(), torch.where(use, dst, dst0).long()
    s["k_cache"].index_copy_(0, dst, s["k_cache"].index_select(0, src))
    s["v_cache"].index_copy_(0, dst, s["v_cache"].index_select(0, src))


def _count(ids, use, n):
    """How often each page id occurs among the used entries."""
    out = torch.zeros(n, dtype=torch.int32, device="cuda")
    return out.index_add_(0, ids.clamp(min=0).reshape(-1), use.reshape(-1).int())


def _plain_free(s):
    c = s["case"]
    ps = c["page_size"]
    length = s["seqlens"][:, None]
    lo = torch.arange(s["table"].shape[1], device="cuda", dtype=torch.int32)[None, :] * ps
    keep = (lo < length) & ((lo + ps > length - c["window"]) | (lo < c["sinks"]))
    table = torch.where(keep, s["table"], -1)
    gone = (s["table"] >= 0) & ~keep
    return {"table": table, "refs": s["refs"] - _count(s["table"], gone, s["refs"].numel())}


def _plain_fork(s):
    c = s["case"]
    ps, room = c["page_size"], c["room"]
    old, refs, parents = s["table"], s["refs"], s["parents"].long()
    P, M = refs.numel(), old.shape[1]
    R = parents.numel()
    here = parents >= 0
    length = torch.where(here, s["seqlens"][parents.clamp(min=0)], 0)
    rows = torch.where(here[:, None], old[parents.clamp(min=0)], -1)
    slot = torch.arange(M, device="cuda")[None, :]
    lo = (length // ps)[:, None]
    hi = torch.where(here, (length + room + ps - 1) // ps, 0)[:, None]
    fixed = (slot < lo) & (rows >= 0)
    free_slot = (slot >= lo) & (slot < hi)
    # Holders of a page that are not a slot to be written.
    held = refs - _count(old, old >= 0, P) + _count(rows, fixed, P)
    at = torch.arange(R * M, device="cuda").view(R, M)
    mine = free_slot & (rows >= 0)
    lowest = torch.full((P,), R * M, device="cuda").scatter_reduce_(
        0, rows.clamp(min=0).long().reshape(-1),
        torch.where(mine, at, R * M).reshape(-1), "amin")
    keep = mine & (lowest[rows.clamp(min=0).long()] == at) & (held[rows.clamp(min=0).long()] == 0)
    fresh = free_slot & ~keep
    rank = (fresh.reshape(-1).cumsum(0) - 1).view(R, M)
    order = torch.argsort((refs != 0).int(), stable=True).int()  # free ids first, ascending
    given = order[rank.clamp(min=0, max=P - 1)]
    table = torch.where(fixed | keep, rows, torch.where(fresh, given, -1))
    copied = fresh & (slot * ps < length[:, None]) & (rows >= 0)
    last = lo.clamp(max=M - 1)
    moved = copied.gather(1, last).squeeze(1)
    src = torch.where(moved, rows.gather(1, last).squeeze(1), -1)
    dst = torch.where(moved, table.gather(1, last).squeeze(1), -1)
    new_refs = held + _count(table, keep | fresh, P)
    counts = torch.stack([fresh.sum(), (refs == 0).sum()]).int()
    _plain_copy(s, src, dst)
    return {"table": table, "refs": new_refs, "seqlens": length, "src": src, "dst": dst,
            "counts": counts, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    P = refs.numel()
    ids = torch.arange(P, device="cuda", dtype=torch.int32)
    live = refs > 0
    n = live.sum().int()
    mover = live & (ids >= n)
    hole = ~live & (ids < n)
    # k-th mover to k-th hole; the lists end in -1.
    half = torch.arange(P // 2, device="cuda")
    src = torch.argsort((~mover).int(), stable=True)[: P // 2].int()
    dst = torch.argsort((~hole).int(), stable=True)[: P // 2].int()
    src = torch.where(half < mover.sum(), src, -1)
    dst = torch.where(half < mover.sum(), dst, -1)
    rank = (mover.cumsum(0) - 1).clamp(min=0, max=max(P // 2 - 1, 0))
    to = torch.where(mover, dst[rank], ids)
    new_table = torch.where(table >= 0, to[table.clamp(min=0).long()], -1)
    new_refs = torch.zeros_like(refs).index_add_(0, to, torch.where(live, refs, 0))
    _plain_copy(s, src, dst)
    return {"table": new_table, "refs": new_refs, "src": src, "dst": dst, "num_live": n.view(1),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------------------------ the package's operators
def _own(s):
    import tensor_attn_fwd_gb300 as attn
    c = s["case"]
    op = c["op"]
    if op in ("train", "prefill"):
        o, lse = attn.attn_window_fwd(s["q"], s["k"], s["v"], c["window"], c["sinks"])
        out = {"o": o, "lse": lse}
        if op == "train":
            out["dq"], out["dk"], out["dv"] = attn.attn_window_bwd(
                s["q"], s["k"], s["v"], o, lse, s["dout"], c["window"], c["sinks"])
        return out
    if op == "decode":
        o, lse = attn.decode_window_paged(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                          s["seqlens"], c["window"], c["sinks"])
        return {"o": o, "lse": lse}
    if op == "free":
        table, refs = attn.attn_pages_free(s["table"], s["refs"], s["seqlens"], c["page_size"],
                                           c["window"], c["sinks"])
        return {"table": table, "refs": refs}
    if op == "fork":
        table, refs, seqlens, src, dst, counts = attn.attn_pages_fork(
            s["table"], s["refs"], s["seqlens"], s["parents"], c["page_size"], c["room"])
        attn.attn_pages_copy(s["k_cache"], s["v_cache"], src, dst)
        return {"table": table, "refs": refs, "seqlens": seqlens, "src": src, "dst": dst,
                "counts": counts, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    table, refs, src, dst, num_live = attn.attn_pages_compact(s["table"], s["refs"])
    attn.attn_pages_copy(s["k_cache"], s["v_cache"], src, dst)
    return {"table": table, "refs": refs, "src": src, "dst": dst, "num_live": num_live,
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("train", "prefill"):
        return _plain_attention(state)
    if op == "decode":
        return _plain_decode(state)
    if op == "free":
        return _plain_free(state)
    if op == "fork":
        return _plain_fork(state)
    return _plain_compact(state)


# ------------------------------------------------------------------ work
def _pairs(Sq, Sk, window, sinks):
    """Visible (row, key) pairs of one head."""
    p = np.arange(Sq, dtype=np.int64) + (Sk - Sq)
    first = np.maximum(p - window + 1, 0)
    n = np.where(p >= 0, p + 1 - first, 0) + np.where(p >= 0, np.minimum(first, sinks), 0)
    return int(n.sum())


def work(case):
    c = case
    op = c["op"]
    if op in ("train", "prefill"):
        B, Hq, Hkv, Sq, Sk, D = (c[n] for n in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
        pairs = B * Hq * _pairs(Sq, Sk, c["window"], c["sinks"])
        qn, kn = B * Hq * Sq * D * 2, B * Hkv * min(Sk, Sq + c["window"] + c["sinks"]) * D * 2
        fwd = 2 * qn + 2 * kn + B * Hq * Sq * 4
        if op == "prefill":
            return {"bytes": fwd, "flops": 4 * D * pairs}
        # The step reads q, k, v and dout and writes o, lse, dq, dk and dv.
        return {"bytes": fwd + 2 * qn + 2 * kn, "flops": 14 * D * pairs}
    if op == "decode":
        B, D = c["B"], c["D"]
        # Lengths are spread evenly over the upper three quarters (one row: max_len).
        length = np.linspace(max(1, c["max_len"] // 4), c["max_len"], 64) if B > 1 else np.array([c["max_len"]])
        seen = np.minimum(length, c["window"] + np.minimum(c["sinks"], np.maximum(length - c["window"], 0)))
        rows = float(seen.mean()) * B
        return {"bytes": int(4 * D * c["Hkv"] * rows + B * c["Hq"] * (4 * D + 4)),
                "flops": int(4 * D * c["Hq"] * rows)}
    page = 2 * c.get("Hkv", 0) * c["page_size"] * c.get("D", 0) * 2  # K and V
    if op == "fork":
        rows = c["groups"] * c["beams"]
        # Most children beyond a page's first holder copy it: beams - 1 of a group in the
        # limit, about 0.6 of them with parents drawn as here.
        copies = int(0.6 * c["groups"] * (c["beams"] - 1))
        return {"bytes": 2 * 4 * rows * c["max_pages"] + 2 * 4 * c["num_pages"] + 2 * page * copies,
                "flops": 0}
    if op == "free":
        entries = c["B"] * c["max_pages"]
        return {"bytes": 2 * 4 * entries + 2 * 4 * ((c["B"] + 1) // 2 + c["B"]) * c["max_pages"],
                "flops": 0}
    n = min(c["live"] * c["num_pages"], 0.9 * c["B"] * c["max_pages"])
    moves = int(n * (1 - n / c["num_pages"]))
    return {"bytes": int(2 * 4 * c["B"] * c["max_pages"] + 2 * 4 * c["num_pages"] + 2 * page * moves),
            "flops": 0}


# ------------------------------------------------------------------ 64 bits
def _exact_rows(q, k, v, do, rows, keys, seen, scale, acc):
    """One block of query rows of one KV head against the keys it can see."""
    x = torch.einsum("nrd,kd->nrk", q[:, rows], k[keys]) * scale
    x = torch.where(seen, x, NEG)
    lse = torch.logsumexp(x, -1)
    p = torch.where(seen, torch.exp(x - torch.where(lse == NEG, 0.0, lse)[..., None]), 0.0)
    o = torch.einsum("nrk,kd->nrd", p, v[keys])
    acc["o"][:, rows] = o
    acc["lse"][:, rows] = lse
    if do is None:
        return
    g = do[:, rows]
    ds = p * (torch.einsum("nrd,kd->nrk", g, v[keys]) - (g * o).sum(-1)[..., None]) * scale
    acc["dv"].index_add_(0, keys, torch.einsum("nrk,nrd->kd", p, g))
    acc["dk"].index_add_(0, keys, torch.einsum("nrk,nrd->kd", ds, q[:, rows]))
    acc["dq"][:, rows] = torch.einsum("nrk,kd->nrd", ds, k[keys])


def _exact_attention(s):
    c = s["case"]
    B, Hq, Hkv, Sq, Sk, D = (c[n] for n in ("B", "Hq", "Hkv", "Sq", "Sk", "D"))
    n, step = Hq // Hkv, 256
    train = c["op"] == "train"
    f = dict(dtype=torch.float64, device="cuda")
    out = {"o": torch.zeros(B, Hq, Sq, D, **f), "lse": torch.full((B, Hq, Sq), NEG, **f)}
    if train:
        out.update(dq=torch.zeros(B, Hq, Sq, D, **f), dk=torch.zeros(B, Hkv, Sk, D, **f),
                   dv=torch.zeros(B, Hkv, Sk, D, **f))
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * n, (h + 1) * n)
            acc = {"o": out["o"][b, heads], "lse": out["lse"][b, heads]}
            if train:
                acc.update(dq=out["dq"][b, heads], dk=out["dk"][b, h], dv=out["dv"][b, h])
            q, k, v = s["q"][b, heads].double(), s["k"][b, h].double(), s["v"][b, h].double()
            do = s["dout"][b, heads].double() if train else None
            for r0 in range(0, Sq, step):
                r1 = min(Sq, r0 + step)
                last = r1 - 1 + Sk - Sq
                if last < 0:
                    continue
                start = max(0, r0 + Sk - Sq - c["window"] + 1)
                keys = torch.cat([torch.arange(0, min(c["sinks"], start, last + 1), device="cuda"),
                                  torch.arange(start, last + 1, device="cuda")])
                pos = torch.arange(r0, r1, device="cuda")[:, None] + Sk - Sq
                seen = (keys <= pos) & ((pos - keys < c["window"]) | (keys < c["sinks"]))
                _exact_rows(q, k, v, do, slice(r0, r1), keys, seen, 1.0 / math.sqrt(D), acc)
    return out


def _exact_decode(s):
    c = s["case"]
    B, Hq, Hkv, D, ps = (c[n] for n in ("B", "Hq", "Hkv", "D", "page_size"))
    out = {"o": torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda"),
           "lse": torch.zeros(B, Hq, dtype=torch.float64, device="cuda")}
    for b, length in enumerate(s["seqlens"].tolist()):
        start = max(0, length - c["window"])
        t = torch.cat([torch.arange(0, min(c["sinks"], start), device="cuda"),
                       torch.arange(start, length, device="cuda")])
        page = s["table"][b].long()[t // ps]
        k = s["k_cache"][page, :, t % ps].double()  # [keys, Hkv, D]
        v = s["v_cache"][page, :, t % ps].double()
        q = s["q"][b, :, 0].double().view(Hkv, Hq // Hkv, D)
        x = torch.einsum("gnd,kgd->gnk", q, k) / math.sqrt(D)
        lse = torch.logsumexp(x, -1)
        out["o"][b] = torch.einsum("gnk,kgd->gnd", torch.exp(x - lse[..., None]), v).reshape(Hq, D)
        out["lse"][b] = lse.reshape(Hq)
    return out


def _exact_copies(s, pairs):
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    for a, b in pairs:
        kc[b] = s["k_cache"][a]
        vc[b] = s["v_cache"][a]
    return {"k_cache": kc, "v_cache": vc}


def _exact_free(s):
    c = s["case"]
    ps = c["page_size"]
    table, refs = s["table"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()
    for b, length in enumerate(s["seqlens"].tolist()):
        for slot in np.nonzero(table[b] >= 0)[0].tolist():
            keys = range(slot * ps, min((slot + 1) * ps, length))
            if not (len(keys) and (keys[-1] >= length - c["window"] or keys[0] < c["sinks"])):
                refs[table[b, slot]] -= 1
                table[b, slot] = -1
    return {"table": table, "refs": refs}


def _exact_fork(s):
    c = s["case"]
    ps, room, M = c["page_size"], c["room"], c["max_pages"]
    old, length = s["table"].cpu().numpy(), s["seqlens"].tolist()
    parents = s["parents"].tolist()
    refs = s["refs"].cpu().numpy().copy()
    free = [int(p) for p in np.nonzero(refs == 0)[0]]
    counts = [0, len(free)]
    np.subtract.at(refs, old[old >= 0], 1)
    R = len(parents)
    table = np.full((R, M), -1, dtype=np.int64)
    lens = [length[p] if p >= 0 else 0 for p in parents]
    for r, p in enumerate(parents):
        n = lens[r] // ps if p >= 0 else 0
        table[r, :n] = old[p, :n]
        np.add.at(refs, table[r][table[r] >= 0], 1)
    shared = refs.copy()
    taken, src, dst = set(), [-1] * R, [-1] * R
    for r, p in enumerate(parents):
        if p < 0:
            continue
        for slot in range(lens[r] // ps, min(M, -(-(lens[r] + room) // ps))):
            page = int(old[p, slot])
            if page >= 0 and shared[page] == 0 and page not in taken:
                taken.add(page)
            else:
                new = free.pop(0)
                counts[0] += 1
                if page >= 0 and slot * ps < lens[r]:
                    src[r], dst[r] = page, new
                taken.add(page)
                page = new
            table[r, slot] = page
            refs[page] += 1
    out = {"table": table, "refs": refs, "seqlens": np.array(lens), "src": np.array(src),
           "dst": np.array(dst), "counts": np.array(counts)}
    out.update(_exact_copies(s, [(a, b) for a, b in zip(src, dst) if b >= 0]))
    return out


def _exact_compact(s):
    table, refs = s["table"].cpu().numpy(), s["refs"].cpu().numpy()
    live = np.nonzero(refs > 0)[0].tolist()
    n = len(live)
    holes = [p for p in range(n) if refs[p] == 0]
    movers = [p for p in live if p >= n]
    to = np.arange(refs.size + 1)
    to[-1] = -1  # an entry of -1 stays
    to[movers] = holes
    new_refs = np.zeros_like(refs)
    new_refs[to[live]] = refs[live]
    pad = [-1] * (refs.size // 2 - len(movers))
    out = {"table": to[table], "refs": new_refs, "src": np.array(movers + pad),
           "dst": np.array(holes + pad), "num_live": np.array([n])}
    out.update(_exact_copies(s, list(zip(movers, holes))))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("train", "prefill"):
        return _exact_attention(s)
    if op == "decode":
        return _exact_decode(s)
    if op == "fork":
        return _exact_fork(s)
    if op == "free":
        return _exact_free(s)
    return _exact_compact(s)
