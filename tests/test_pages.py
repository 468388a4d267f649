"""Pages of a cache: attn_pages_fork, attn_pages_free, attn_pages_compact and
attn_pages_copy against the rules written out in Python, entry by entry, and a
stream that runs them together with the projection, the windowed prefill and the
windowed decode."""
import math

import numpy as np
import pytest
import torch

import tensor_attn_fwd_gb300 as attn


# ------------------------------------------------------------------ the rules
def plain_free(table, refs, lens, page, window, sinks, room=0):
    table, refs = table.copy(), refs.copy()
    B, M = table.shape
    for b in range(B):
        n = min(int(lens[b]), M * page)
        for s in range(M):
            e = table[b, s]
            if not -1 <= e < len(refs):
                e = -1
            keep = (n >= 0 and s * page < n + room
                    and ((s + 1) * page > n - window or s * page < sinks))
            if not keep and e >= 0:
                refs[e] -= 1
            table[b, s] = e if keep else -1
    return table, refs


def plain_fork(table, refs, lens, parents, page, room):
    B, M = table.shape
    R, P = len(parents), len(refs)

    def entry(p, s):
        return table[p, s] if -1 <= table[p, s] < P else -1

    free = [p for p in range(P) if refs[p] == 0]
    n_free, needed = len(free), 0
    refs = refs.copy()
    for b in range(B):
        for s in range(M):
            if entry(b, s) >= 0:
                refs[entry(b, s)] -= 1
    out = np.full((R, M), -1)
    parents = [p if -1 <= p < B else -1 for p in parents]
    length = [min(max(int(lens[p]), 0), M * page) if p >= 0 else 0 for p in parents]
    for r, p in enumerate(parents):
        for s in range(length[r] // page if p >= 0 else 0):
            out[r, s] = entry(p, s)
            if out[r, s] >= 0:
                refs[out[r, s]] += 1
    others = refs.copy()
    src, dst, seen = [-1] * R, [-1] * R, set()
    for r, p in enumerate(parents):
        if p < 0:
            continue
        n = length[r]
        for s in range(n // page, min(M, -(-(n + room) // page))):
            e = entry(p, s)
            if e >= 0 and e not in seen and others[e] == 0:
                out[r, s] = e
            else:
                needed += 1
                new = free.pop(0) if free else -1
                out[r, s] = new
                if s * page < n and e >= 0 and new >= 0:
                    src[r], dst[r] = e, new
                if s * page < n and new < 0:
                    length[r] = s * page
            if e >= 0:
                seen.add(e)
            if out[r, s] >= 0:
                refs[out[r, s]] = 1
    return out, refs, np.array(length), np.array(src), np.array(dst), np.array([needed, n_free])


def plain_compact(table, refs):
    P = len(refs)
    live = [p for p in range(P) if refs[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    movers = [p for p in live if p >= n]
    to = {p: p for p in live}
    to.update(zip(movers, holes))
    out = np.array([[to.get(int(e), -1) for e in row] for row in table])
    new = np.zeros_like(refs)
    for p in live:
        new[to[p]] = refs[p]
    pad = [-1] * (P // 2 - len(movers))
    return out, new, np.array(movers + pad), np.array(holes + pad), np.array([n])


# ------------------------------------------------------------------ inputs
def cache_tables(rng, B, M, P, page, fill, shared, extern=0):
    """A consistent cache: rows of ragged lengths over a shuffled pool, some rows
    continuing another's prefix, ``extern`` pages with a holder outside the table."""
    ids = rng.permutation(P).tolist()
    table = np.full((B, M), -1)
    lens = rng.integers(0, int(M * page * fill) + 1, B)
    lens[rng.random(B) < 0.2] //= page
    lens[rng.random(B) < 0.2] *= page
    lens = np.minimum(lens, M * page)
    for b in range(B):
        n = -(-int(lens[b]) // page)
        take = 0
        if b and rng.random() < shared:  # a beam of an earlier row: all its pages, or a prefix
            a = int(rng.integers(0, b))
            if rng.random() < 0.5:
                lens[b] = lens[a]
                table[b] = table[a]
                continue
            take = min(int(lens[a]) // page, n)
            table[b, :take] = table[a, :take]
        for s in range(take, n):
            if not ids:
                lens[b] = s * page
                break
            table[b, s] = ids.pop()
    refs = np.bincount(table[table >= 0].ravel(), minlength=P)
    held = np.nonzero(refs)[0]
    for p in rng.choice(held, min(extern, len(held)), replace=False) if len(held) else []:
        refs[p] += 1
    return table, refs, lens


def gpu(*arrays):
    out = [torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda() for a in arrays]
    return out if len(out) > 1 else out[0]


def same(got, want, what):
    for g, w, name in zip(got, want, what):
        assert np.array_equal(g.cpu().numpy(), np.asarray(w)), name


# B, M, P, page: one entry; small; one row; wide; over the one-cluster limit (both ways)
SIZES = [(1, 1, 1, 1), (3, 5, 20, 4), (1, 300, 400, 32), (70, 9, 700, 64), (1500, 3, 5000, 32),
         (40, 1700, 70000, 16), (3, 4, 140001, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("window,sinks,room", [(1, 0, 0), (40, 3, 0), (10 ** 9, 0, 7), (100, 70, 33)])
def test_free(size, window, sinks, room):
    B, M, P, page = size
    rng = np.random.default_rng(B + M)
    table, refs, lens = cache_tables(rng, B, M, P, page, 1.0, 0.3)
    lens[rng.random(B) < 0.2] = -1
    want = plain_free(table, refs, lens, page, window, sinks, room)
    t, r, n = gpu(table, refs, lens)
    got = attn.attn_pages_free(t, r, n, page, window, sinks, room)
    assert attn.attn_debug_status() == attn.ATTN_OK
    same(got, want, ("table", "refs"))
    same((t, r), (table, refs), ("the input table", "the input refs"))
    got = attn.attn_pages_free(t, r, n, page, window, sinks, room, block_table_out=t, refs_out=r)
    assert got[0] is t and got[1] is r
    same(got, want, ("table in place", "refs in place"))


@pytest.mark.gpu
def test_free_without_a_window_gives_up_what_lies_behind():
    t, r, n = gpu([[4, 0, 2], [3, 1, -1]], [1] * 5, [33, 64])
    table, refs = attn.attn_pages_free(t, r, n, 32)
    same((table, refs), ([[4, 0, -1], [3, 1, -1]], [1, 1, 0, 1, 1]), ("table", "refs"))


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("room", [0, 1, 90])
@pytest.mark.parametrize("kind", ["same", "beams", "fewer", "more"])
def test_fork(size, room, kind):
    B, M, P, page = size
    rng = np.random.default_rng(7 * B + M + room)
    table, refs, lens = cache_tables(rng, B, M, P, page, 0.8, 0.5, extern=B // 2)
    parents = {"same": np.arange(B), "beams": rng.integers(-1, B, B),
               "fewer": rng.integers(0, B, max(1, B // 3)),
               "more": rng.integers(0, B, 2 * B + 1)}[kind]
    want = plain_fork(table, refs, lens, parents, page, room)
    got = attn.attn_pages_fork(*gpu(table, refs, lens, parents), page, room)
    status = attn.attn_debug_status()
    assert status == (attn.ATTN_ERR_NO_PAGES if want[5][0] > want[5][1] else attn.ATTN_OK)
    same(got, want, ("table", "refs", "seqlens", "src", "dst", "counts"))


@pytest.mark.gpu
def test_fork_copies_what_is_written_twice():
    # Row 0 has one full page and three keys of a second; both new rows continue it.
    args = gpu([[5, 2, -1]], [0, 0, 1, 0, 0, 1], [7], [0, 0])
    table, refs, lens, src, dst, counts = attn.attn_pages_fork(*args, 4, room=2)
    same((table, refs, lens, src, dst, counts),
         ([[5, 2, 0], [5, 1, 3]], [1, 1, 1, 1, 0, 2], [7, 7], [-1, 2], [-1, 1], [3, 4]),
         ("table", "refs", "lens", "src", "dst", "counts"))


@pytest.mark.gpu
def test_fork_without_pages_ends_the_rows_and_says_so():
    args = gpu([[1, 0]], [1, 1], [6], [0, 0, 0])
    table, refs, lens, src, dst, counts = attn.attn_pages_fork(*args, 4)
    assert attn.attn_debug_status() == attn.ATTN_ERR_NO_PAGES
    same((table, refs, lens, src, dst, counts),
         ([[1, 0], [1, -1], [1, -1]], [1, 3], [6, 4, 4], [-1] * 3, [-1] * 3, [2, 0]),
         ("table", "refs", "lens", "src", "dst", "counts"))


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("fill", [0.0, 0.4, 1.0])
def test_compact(size, fill):
    B, M, P, page = size
    rng = np.random.default_rng(B * M + P)
    table, refs, lens = cache_tables(rng, B, M, P, page, fill, 0.3, extern=2)
    want = plain_compact(table, refs)
    got = attn.attn_pages_compact(*gpu(table, refs))
    assert attn.attn_debug_status() == attn.ATTN_OK
    same(got, want, ("table", "refs", "src", "dst", "num_live"))
    again = attn.attn_pages_compact(got[0], got[1])  # nothing is left to move
    same(again, (want[0], want[1], [-1] * (P // 2), [-1] * (P // 2), want[4]),
         ("table", "refs", "src", "dst", "num_live"))


@pytest.mark.gpu
@pytest.mark.parametrize("alive", ["all", "none", "head", "tail", "odd"])
@pytest.mark.parametrize("P", [1, 2, 1023, 1025, 200000])
def test_compact_pools(alive, P):
    p = np.arange(P)
    refs = {"all": p * 0 + 1, "none": p * 0, "head": p < P // 3, "tail": p >= P - P // 3,
            "odd": p % 2}[alive].astype(int) * (p % 5 + 1)
    table = np.where(refs > 0, p, -1)[None, -4000:]
    want = plain_compact(table, refs)
    same(attn.attn_pages_compact(*gpu(table, refs)), want, ("table", "refs", "src", "dst", "live"))
    assert attn.attn_debug_status() == attn.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("page_shape,dtype", [((2, 32, 64), torch.bfloat16), ((3, 1, 8), torch.bfloat16),
                                              ((1, 33, 16), torch.uint8), ((8, 64, 128), torch.bfloat16)])
def test_copy(page_shape, dtype):
    P = 37
    rng = np.random.default_rng(1)
    k, v = (torch.randint(0, 250, (P, *page_shape), device="cuda").to(dtype) for _ in range(2))
    ids = rng.permutation(P)
    src, dst = ids[:15].copy(), ids[15:30].copy()
    src[3] = dst[3] = -1
    src[5] = src[6]  # one page copied twice
    kw, vw = k.clone(), v.clone()
    for a, b in zip(src, dst):
        if a >= 0:
            kw[b], vw[b] = k[a], v[a]
    s, d = gpu(src, dst)
    attn.attn_pages_copy(k, v, s, d)
    assert attn.attn_debug_status() == attn.ATTN_OK
    assert torch.equal(k, kw) and torch.equal(v, vw)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    attn.attn_pages_copy(k, v, none, none)
    assert torch.equal(k, kw) and torch.equal(v, vw)


@pytest.mark.gpu
def test_copy_many_pairs():
    P = 140000  # more pairs than one grid holds
    k = torch.arange(P * 8, device="cuda").remainder(251).to(torch.bfloat16).view(P, 8)
    v = k + 1
    src = torch.arange(0, P, 2, dtype=torch.int32, device="cuda")
    dst = src + 1
    kw, vw = k.clone(), v.clone()
    kw[1::2], vw[1::2] = k[::2], v[::2]
    attn.attn_pages_copy(k, v, src, dst)
    assert torch.equal(k, kw) and torch.equal(v, vw)


@pytest.mark.gpu
def test_bad_entries_are_reported_and_read_as_no_page():
    bad = attn.ATTN_ERR_INVALID_ARG
    table, refs, lens = np.array([[0, 7, 2], [1, -2, -1]]), np.array([1, 1, 1, 0, 0]), np.array([9, 3])
    got = attn.attn_pages_free(*gpu(table, refs, lens), 4, 3, 1)
    assert attn.attn_debug_status() == bad
    same(got, plain_free(table, refs, lens, 4, 3, 1), ("table", "refs"))
    got = attn.attn_pages_fork(*gpu(table, refs, lens, [1, 2, 0, -5]), 4, 1)
    assert attn.attn_debug_status() == bad
    same(got, plain_fork(table, refs, lens, [1, 2, 0, -5], 4, 1), ("table", "refs", "lens", "src", "dst", "n"))
    got = attn.attn_pages_compact(*gpu(table, refs))
    assert attn.attn_debug_status() == bad
    same(got, plain_compact(table, refs), ("table", "refs", "src", "dst", "live"))
    attn.attn_pages_compact(*gpu([[3, 0]], refs))  # page 3 counts no holder
    assert attn.attn_debug_status() == bad
    k = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    v = k + 1
    for s, d in ((0, 4), (-1, 2), (5, 1), (1, -7)):
        attn.attn_pages_copy(k, v, *gpu([s], [d]))
        assert attn.attn_debug_status() == bad
    assert bool((k == 0).all()) and bool((v == 1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B,P", [(12, 400), (300, 8000), (2000, 60000)])  # each launch form
def test_graph_and_stream(B, P):
    rng = np.random.default_rng(3)
    table, refs, lens = cache_tables(rng, B, 20, P, 32, 0.7, 0.5)
    args = gpu(table, refs, lens, rng.integers(0, B, B))
    want = attn.attn_pages_fork(*args, 32, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn.attn_pages_fork(*args, 32, 5, stream=side)
    side.synchronize()
    same(got, [w.cpu().numpy() for w in want], ["stream"] * 6)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = attn.attn_pages_fork(*args, 32, 5)
        packed = attn.attn_pages_compact(got[0], got[1])
        left = attn.attn_pages_free(packed[0], packed[1], got[2], 32, 64, 4)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    same(got, [w.cpu().numpy() for w in want], ["graph"] * 6)
    w2 = plain_compact(want[0].cpu().numpy(), want[1].cpu().numpy())
    same(packed, w2, ["graph"] * 5)
    same(left, plain_free(w2[0], w2[1], want[2].cpu().numpy(), 32, 64, 4), ["graph"] * 2)


# ------------------------------------------------------------------ together
@pytest.mark.gpu
def test_a_stream_over_pages_follows_the_prefill():
    """Two prompts, four beams each: projection, windowed prefill, then one token a
    step over a pool that the window keeps small, with beams re-forked and the pool
    packed on the way.  The last rows match the windowed prefill of each beam's whole
    history within the roundings of both (2^-8 each on O and on P; fp32 sums)."""
    torch.manual_seed(0)
    Hq, Hkv, D, hidden, page, window, sinks = 4, 2, 64, 128, 32, 70, 5
    prompts, beams, S0, steps = 2, 4, 150, 90
    B, M = prompts * beams, (S0 + steps) // page + 2
    per_row = -(-sinks // page) + window // page + 3
    P = prompts * (S0 // page + 2) + 2 * B * per_row
    w = (torch.randn((Hq + 2 * Hkv) * D, hidden) / math.sqrt(hidden)).to(torch.bfloat16).cuda()
    rope = attn.attn_rope_table(S0 + steps, D)
    kc, vc = (torch.full((P, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))

    def put(table, lens, k, v):
        """Keys and values of one new token a row, at position lens."""
        at = lens.long()
        ids = table.gather(1, (at // page)[:, None])[:, 0].long()
        assert bool((ids >= 0).all())
        kc[ids, :, at % page] = k[:, :, 0]
        vc[ids, :, at % page] = v[:, :, 0]

    # The prompts, one row each; every page of a prompt is written once.
    x0 = torch.randn(prompts, S0, hidden, device="cuda").to(torch.bfloat16)
    q, k, v = attn.attn_qkv_rope(x0, w, rope, Hq, Hkv)
    attn.attn_window_fwd(q, k, v, window, sinks)
    empty = gpu(np.full((1, M), -1), np.zeros(P), [0], [-1] * prompts)
    table, refs, lens, _, _, _ = attn.attn_pages_fork(*empty, page)
    ids = torch.arange(prompts, dtype=torch.int32, device="cuda")
    table, refs, lens, _, _, _ = attn.attn_pages_fork(table, refs, lens, ids, page, room=S0)
    for t in range(S0):
        put(table, lens + t, k[:, :, t:t + 1], v[:, :, t:t + 1])
    lens = lens + S0
    hist = [(q[p], k[p], v[p]) for p in range(prompts) for _ in range(beams)]  # per beam
    parents = gpu(np.arange(B) // beams)
    for step in range(steps):
        # Continue each beam's parent, with a page for the coming token.
        table, refs, lens, src, dst, counts = attn.attn_pages_fork(table, refs, lens, parents, page,
                                                                   room=1)
        attn.attn_pages_copy(kc, vc, src, dst)
        if step % 17 == 5:
            table, refs, src, dst, live = attn.attn_pages_compact(table, refs)
            attn.attn_pages_copy(kc, vc, src, dst)
            kc[int(live):], vc[int(live):] = float("nan"), float("nan")
        x = torch.randn(B, 1, hidden, device="cuda").to(torch.bfloat16)
        q, k, v = attn.attn_qkv_rope(x, w, rope, Hq, Hkv, positions=lens.view(B, 1))
        put(table, lens, k, v)
        lens = lens + 1
        o, lse = attn.decode_window_paged(q, kc, vc, table, lens, window, sinks)
        table, refs = attn.attn_pages_free(table, refs, lens, page, window, sinks)
        if step:  # the prompts' beams start as copies of their prompt
            hist = [hist[p] for p in parents.tolist()]
        hist = [tuple(torch.cat([h, t[b]], 1) for h, t in zip(hist[b], (q, k, v))) for b in range(B)]
        parents = gpu(np.arange(B) // beams * beams
                      + np.random.default_rng(step).integers(0, beams, B))
        if step % 20 == 0:
            assert attn.attn_debug_status() == attn.ATTN_OK
    assert attn.attn_debug_status() == attn.ATTN_OK
    assert int((refs > 0).sum()) <= B * per_row
    for b in range(B):
        ow, lw = attn.attn_window_fwd(*(t[None].contiguous() for t in hist[b]), window, sinks)
        ow, lw = ow[0, :, -1].double(), lw[0, :, -1].double()
        qb, kb, vb = (t.double().abs() for t in hist[b])
        assert bool(((o[b].double() - ow).abs()
                     <= 2 * (2.0 ** -8 + 2.0 ** -11) * (ow.abs() + vb.amax())).all())
        scores = (qb[:, -1:] @ kb.repeat_interleave(Hq // Hkv, 0).transpose(1, 2)).amax() / math.sqrt(D)
        assert bool(((lse[b].double() - lw).abs()
                     <= 2 * ((D + 8) * 2.0 ** -24 * scores + 2.0 ** -18)).all())


# ------------------------------------------------------------------ refusals (no GPU)
A, A2, A3 = 0x10000000, 0x20000000, 0x30000000


def _lib():
    from tensor_attn_fwd_gb300 import build as attn_build
    attn_build.build()
    return attn.load_library()


def c_free(t=A, r=A, n=A, to=A2, ro=A2, B=2, M=4, P=8, page=32, window=8, sinks=1, room=0):
    return _lib().attn_pages_free(t, r, n, to, ro, B, M, P, page, window, sinks, room, None)


def c_fork(t=A, r=A, n=A, p=A, to=A2, ro=A2, no=A2, s=A2, d=A3, c=A2, w=A2, B=2, R=2, M=4, P=8, page=32,
           room=0):
    return _lib().attn_pages_fork(t, r, n, p, to, ro, no, s, d, c, w, B, R, M, P, page, room, None)


def c_compact(t=A, r=A, to=A2, ro=A2, s=A2, d=A3, n=A2, w=A2, B=2, M=4, P=8):
    return _lib().attn_pages_compact(t, r, to, ro, s, d, n, w, B, M, P, None)


def c_copy(k=A, v=A2, s=A, d=A, n=3, P=8, size=1024):
    return _lib().attn_pages_copy(k, v, s, d, n, P, size, None)


INV, UNS, MIS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_MISALIGNED


@pytest.mark.parametrize("call,kw,code", [(f, kw, c) for f in (c_free, c_fork, c_compact) for kw, c in [
    (dict(t=None), INV), (dict(r=None), INV), (dict(to=None), INV), (dict(ro=None), INV),
    (dict(B=0), INV), (dict(M=0), INV), (dict(P=0), INV), (dict(B=1 << 20, M=1 << 12), UNS),
    (dict(P=(1 << 30) + 1), UNS), (dict(t=A + 1), MIS), (dict(ro=A2 + 2), MIS),
]] + [
    (c_free, dict(n=None), INV), (c_free, dict(window=0), INV), (c_free, dict(sinks=-1), INV),
    (c_free, dict(room=-1), INV), (c_free, dict(page=0), INV), (c_free, dict(M=1 << 20, page=1 << 11), UNS),
    (c_free, dict(n=A + 3), MIS),
    (c_fork, dict(p=None), INV), (c_fork, dict(w=None), INV), (c_fork, dict(R=0), INV),
    (c_fork, dict(room=-1), INV), (c_fork, dict(to=A), INV), (c_fork, dict(ro=A), INV),
    (c_fork, dict(no=A), INV), (c_fork, dict(d=A2, s=A2), INV), (c_fork, dict(R=1 << 30), UNS),
    (c_fork, dict(p=A + 2), MIS), (c_fork, dict(c=A2 + 1), MIS),
    (c_compact, dict(to=A), INV), (c_compact, dict(ro=A), INV), (c_compact, dict(s=None), INV),
    (c_compact, dict(n=None), INV), (c_compact, dict(w=None), INV), (c_compact, dict(s=A3), INV),
    (c_compact, dict(w=A2 + 1), MIS),
    (c_copy, dict(k=None), INV), (c_copy, dict(v=None), INV), (c_copy, dict(s=None), INV),
    (c_copy, dict(n=-1), INV), (c_copy, dict(P=0), INV), (c_copy, dict(size=0), INV),
    (c_copy, dict(size=1000), UNS), (c_copy, dict(size=1 << 50), UNS), (c_copy, dict(k=A + 8), MIS),
    (c_copy, dict(d=A + 1), MIS)])
def test_c_rejects(call, kw, code):
    assert call(**kw) == code


def test_copy_of_nothing_needs_no_lists():
    assert c_copy(n=0, s=None, d=None) == attn.ATTN_OK


def test_workspace():
    import ctypes
    n = ctypes.c_longlong(0)
    assert _lib().attn_pages_workspace(8, 3, ctypes.byref(n)) == attn.ATTN_OK and n.value >= 2 * 8 + 3
    assert _lib().attn_pages_workspace(0, 3, ctypes.byref(n)) == INV
    assert _lib().attn_pages_workspace(8, -1, ctypes.byref(n)) == INV
    assert _lib().attn_pages_workspace(8, 1, None) == INV
    assert "pages" in attn.attn_status_string(attn.ATTN_ERR_NO_PAGES)


def test_python_rejects_cpu_tensors():
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_pages_free(t, t[0], t[0], 32)
    with pytest.raises(ValueError):
        attn.attn_pages_fork(t, t[0], t[0], t[0], 32)
    with pytest.raises(ValueError):
        attn.attn_pages_compact(t, t[0])
    with pytest.raises(ValueError):
        attn.attn_pages_copy(t, t, t[0], t[0])


@pytest.mark.gpu
def test_python_rejects():
    t, r, n = gpu([[0, 1], [2, 3]], [1] * 4, [8, 8])
    k = torch.zeros(4, 2, 8, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: attn.attn_pages_free(t.long(), r, n, 4),
                lambda: attn.attn_pages_free(t, r, n[:1], 4),
                lambda: attn.attn_pages_free(t.t(), r, n, 4),
                lambda: attn.attn_pages_free(t, r, n, 4, window=0),
                lambda: attn.attn_pages_free(t, r, n, 4, room=-1),
                lambda: attn.attn_pages_free(t, r, n, 4, refs_out=r[:3]),
                lambda: attn.attn_pages_fork(t, r, n, n.float(), 4),
                lambda: attn.attn_pages_fork(t, r, n, n, 4, room=-1),
                lambda: attn.attn_pages_copy(k, k[:3], r, r),
                lambda: attn.attn_pages_copy(k, k.clone(), r, r[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(attn.AttnError):
        attn.attn_pages_free(t, r, n, 0)
    with pytest.raises(attn.AttnError):
        attn.attn_pages_fork(t, r, n, n[:0], 4)
    with pytest.raises(attn.AttnError):
        attn.attn_pages_copy(k[:, :, :3].contiguous(), k[:, :, :3].contiguous(), r, r)  # 12-byte pages
