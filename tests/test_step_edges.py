"""A serving step at the edges of what the documentation allows: large tables that are copied
beside the call's own work, rows that are refused, large scores, the bounds-checked build."""
import ctypes
import math

import numpy as np
import pytest
import torch

import tensor_attn_fwd_gb300 as attn
from tensor_attn_fwd_gb300 import build as attn_build

from test_step import (A, APPEND, BF, INV, M2, M4, MIS, append_case, check, dense, gpu, plain_append,
                       pool, reference, run_chunk, same, status_ok)


# ------------------------------------------------------------------ refusals (no GPU)
@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INV) for n in ("cu", "sl", "slots", "plan")],
    *[({n: M2}, MIS) for n in ("cu", "sl", "slots")], (dict(plan=M4), MIS),
    *[({n: 0}, INV) for n in ("B", "T", "Hq", "Hkv", "D", "mk", "window")], (dict(sinks=-1), INV),
])
def test_plan_with_slots_rejects(kw, code):
    d = dict(cu=A, sl=A, slots=A, plan=A, B=2, T=8, Hq=4, Hkv=2, D=64, mk=128, window=9, sinks=0)
    d.update(kw)
    assert attn.load_library().attn_chunk_plan_slots(*d.values(), None) == code


def test_plan_with_slots_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.attn_chunk_plan(i, i[:3], 4, 4, 2, 64, 128, slots=i)


# ------------------------------------------------------------------ large tables
def busy(stream):
    """A few milliseconds of matrix products on another stream."""
    a = torch.ones(4096, 4096, dtype=torch.bfloat16, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(20):
            torch.mm(a, a)
    a.record_stream(stream)


# Rows, slots, pages, page size, new tokens: tables and counts that CTAs of their own copy while
# the others hand out pages (131072 entries or pages and more).
LARGE = [(1024, 1024, 40000, 32, 40), (300, 700, 30000, 64, 200), (131, 1001, 150001, 32, 9),
         (2000, 130, 200000, 96, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,M,P,ps,most", LARGE)
@pytest.mark.parametrize("reserved", [0.0, 0.01])
def test_append_of_large_tables(B, M, P, ps, most, reserved):
    # Slots of tokens in pages that rows had before (partly filled, or reserved) do not depend
    # on when the copies are made: the results' memory holds other pages that look right.
    rng = np.random.default_rng(B + M)
    table, refs, lens, new = append_case(rng, B, M, P, ps, most, reserved)
    T = int(new.sum()) + 5
    want = plain_append(table, refs, lens, new, T, ps)
    assert want[6][0] <= want[6][1]
    inputs = gpu(table, refs, lens, new)
    wrong = gpu((np.arange(B * M) * 7 % P).reshape(B, M), np.full(P, 5), np.full(B, 11))
    other = torch.cuda.Stream()
    for i in range(12):
        out = [x.clone() for x in wrong]
        if i % 3 == 1:
            busy(other)
        same(attn.attn_pages_append(*inputs, T, ps, block_table_out=out[0], refs_out=out[1],
                                    seqlens_out=out[2]), want)
        # Table and counts in place, lengths not.
        here, out = [x.clone() for x in inputs], wrong[2].clone()
        if i % 3 == 2:
            busy(other)
        same(attn.attn_pages_append(*here, T, ps, block_table_out=here[0], refs_out=here[1],
                                    seqlens_out=out), want)
        assert torch.equal(here[2], inputs[2])
    # Everything in place.
    same(attn.attn_pages_append(*inputs, T, ps, block_table_out=inputs[0], refs_out=inputs[1],
                                seqlens_out=inputs[2]), want)
    status_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("B,M,P,ps,most", LARGE)
@pytest.mark.parametrize("bad", [-2, "P"])
def test_append_reports_a_bad_entry_that_it_replaces(B, M, P, ps, most, bad):
    # An entry that is no page, where a row's new tokens come: read as -1, and reported also where
    # the page that takes its place is written to the same memory.
    rng = np.random.default_rng(B)
    table, refs, lens, new = append_case(rng, B, M, P, ps, most)
    rows = [b for b in range(B) if new[b] > 0 and table[b, (lens[b] + new[b] - 1) // ps] < 0]
    b = rows[len(rows) // 2]
    table[b, (lens[b] + new[b] - 1) // ps] = P if bad == "P" else bad
    T = int(new.sum())
    want = plain_append(table, refs, lens, new, T, ps)
    inputs = gpu(table, refs, lens, new)
    for _ in range(8):
        here, out = [x.clone() for x in inputs], torch.zeros_like(inputs[2])
        same(attn.attn_pages_append(*here, T, ps, block_table_out=here[0], refs_out=here[1],
                                    seqlens_out=out), want)
        assert attn.attn_debug_status() == INV
    same(attn.attn_pages_append(*inputs, T, ps), want)
    assert attn.attn_debug_status() == INV


# ------------------------------------------------------------------ shared pages
def append_of_sharing_rows(table, refs, lens, new, T, ps):
    """plain_append, where rows whose new keys would go to a page of several holders take none
    of their tokens and need no pages, as finished rows; and which rows those are."""
    B, M = table.shape
    shares = np.zeros(B, dtype=bool)
    for b in range(B):
        x, n = int(lens[b]), int(new[b])
        if n > 0 and x >= 0 and x + n <= M * ps:
            e = table[b, x // ps:(x + n - 1) // ps + 1]
            shares[b] = bool((refs[e[e >= 0]] > 1).any())
    out = list(plain_append(table, refs, np.where(shares, -1, lens), new, T, ps))
    out[2] = np.where(shares, lens, out[2])
    return out, shares


@pytest.mark.gpu
@pytest.mark.parametrize("B,M,P,ps,most", APPEND[2:] + LARGE[:2])
@pytest.mark.parametrize("reserved", [0.0, 0.3])
def test_append_refuses_rows_that_share_a_page_to_be_written(B, M, P, ps, most, reserved):
    rng = np.random.default_rng(B + 3)
    table, refs, lens, new = append_case(rng, B, M, P, ps, most, reserved)
    # Second holders of some pages: of those that are written, and of full ones.
    held = np.nonzero(refs == 1)[0]
    refs[held[rng.random(held.size) < 0.5 / (most // ps + 2)]] = 2
    b = int(np.argmax((new > 0) & (lens % ps != 0)))
    refs[table[b, lens[b] // ps]] = 3
    T = int(new.sum())
    want, shares = append_of_sharing_rows(table, refs, lens, new, T, ps)
    assert shares[b] and (new[~shares] > 0).any()
    inputs = gpu(table, refs, lens, new)
    same(attn.attn_pages_append(*inputs, T, ps), want)
    assert attn.attn_debug_status() == INV
    same(attn.attn_pages_append(*inputs, T, ps, block_table_out=inputs[0], refs_out=inputs[1],
                                seqlens_out=inputs[2]), want)
    assert attn.attn_debug_status() == INV


@pytest.mark.gpu
def test_append_of_rows_that_share_full_pages():
    # Samples of one prompt: full pages of several holders are no obstacle.
    table = np.array([[0, 1, 2, -1], [0, 1, 3, -1], [0, 1, -1, -1]])
    refs, lens, new = np.array([3, 3, 1, 1, 0, 0, 0]), np.array([70, 71, 64]), np.array([1, 40, 32])
    want = plain_append(table, refs, lens, new, 73, 32)
    assert (want[2] == lens + new).all()
    same(attn.attn_pages_append(*gpu(table, refs, lens, new), 73, 32), want)
    status_ok()


# ------------------------------------------------------------------ steps with refused requests
@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 4)])
def test_step_with_refused_requests(D, window, sinks):
    """Requests without pages for their tokens, past their slots, finished, and with an empty
    table: none of their tokens sees a key, nothing is reported for them, and the others
    are as without them."""
    Hq, Hkv, ps, M, T = 8, 2, 32, 24, 420
    rng = np.random.default_rng(D)
    ctxs, new = [500, 300, 740, 90, 400, 0, 8, 333], [1, 200, 40, 60, 1, 70, 33, 1]
    lens = np.array(ctxs)
    lens[3] = -5  # finished
    pages = -(-np.maximum(lens, 0) // ps)
    table, at = np.full((8, M), -1), 0
    ids = rng.permutation(200)
    for b in range(8):
        table[b, :pages[b]] = ids[at:at + pages[b]]
        at += pages[b]
    refs = np.bincount(table[table >= 0], minlength=200)
    refs[np.nonzero(refs == 0)[0][8:]] = 1  # eight free pages: a part of the rows' needs
    kc, vc = (torch.randn(200, Hkv, ps, D, device="cuda").to(BF) for _ in range(2))
    tab, ref_counts, ln, nw = gpu(table, refs, lens, new)
    if window:  # pages that the window has passed are gone
        tab, ref_counts = attn.attn_pages_free(tab, ref_counts, ln, ps, window, sinks)
        ref_counts.copy_(torch.from_numpy(refs).cuda())
    rope = attn.attn_rope_table(M * ps, D)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda").to(BF)
    tab, ref_counts, ln, cu, pos, slots, counts = attn.attn_pages_append(tab, ref_counts, ln, nw, T, ps)
    assert attn.attn_debug_status() != attn.ATTN_OK  # no pages, or past its slots: either first
    taken = (ln.cpu().numpy() > lens) & (lens >= 0)
    assert taken.tolist() == [True, True, False, False, True, False, False, False]
    plan = attn.attn_chunk_plan(cu, ln, T, Hq, Hkv, D, M * ps, window, sinks, slots=slots)
    q = attn.attn_rope_append(qkv, rope, pos, slots, kc, vc, Hq)
    o = torch.full((T, Hq, D), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    attn.attn_chunk_paged(q, kc, vc, tab, plan, o=o, lse=lse)
    status_ok()
    seen = tab.cpu().numpy().astype(np.int64)
    seen[seen < 0] = 0  # (of keys that the window has passed)
    ref = reference(q, [c if t else -n for c, t, n in zip(ctxs, taken, new)], new, seen, kc, vc,
                    window or 1 << 30, sinks, 1 / math.sqrt(D))
    check((o, lse), ref, sum(new))
    first = np.cumsum([0] + new)
    for b in range(8):
        rows = slice(first[b], first[b + 1])
        assert bool((ref[1][rows] == -math.inf).all()) == (not taken[b])
    assert bool((o[sum(new):] == 7).all()) and bool((lse[sum(new):] == 7).all())
    # Where all are taken the slots change nothing.
    cu1, ln1 = gpu(np.array([0, 1, 201]), np.array([501, 500]))
    with_slots = attn.attn_chunk_plan(cu1, ln1, 201, Hq, Hkv, D, M * ps, window, sinks,
                                      slots=slots[:201])
    without = attn.attn_chunk_plan(cu1, ln1, 201, Hq, Hkv, D, M * ps, window, sinks)
    a, b = (attn.attn_chunk_paged(q[:201], kc, vc, tab[:2].contiguous(), p) for p in (with_slots, without))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    status_ok()
    for bad in (slots[:-1], slots.long(), slots.cpu()):
        with pytest.raises(ValueError):
            attn.attn_chunk_plan(cu, ln, T, Hq, Hkv, D, M * ps, slots=bad)


@pytest.mark.gpu
def test_refused_requests_in_a_graph():
    """A captured step: a request waits for pages, sees nothing meanwhile, and goes on when
    another's are free."""
    Hq, Hkv, D, ps, B, M, P, T = 4, 2, 64, 32, 2, 8, 7, 100
    rope = attn.attn_rope_table(M * ps, D)
    table, refs, lens, new = gpu(np.full((B, M), -1), np.zeros(P), np.zeros(B), np.zeros(B))
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda").to(BF)
    kc, vc = (torch.zeros(P, Hkv, ps, D, dtype=BF, device="cuda") for _ in range(2))
    o, lse = torch.zeros(T, Hq, D, dtype=BF, device="cuda"), torch.zeros(T, Hq, device="cuda")

    def step():
        _, _, _, cu, pos, slots, _ = attn.attn_pages_append(
            table, refs, lens, new, T, ps, block_table_out=table, refs_out=refs, seqlens_out=lens)
        plan = attn.attn_chunk_plan(cu, lens, T, Hq, Hkv, D, M * ps, slots=slots)
        q = attn.attn_rope_append(qkv, rope, pos, slots, kc, vc, Hq)
        attn.attn_chunk_paged(q, kc, vc, table, plan, o=o, lse=lse)
        return q

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            q = step()
    torch.cuda.synchronize()
    length = [0, 0]
    for news, takes in (([60, 40], [1, 1]), ([70, 30], [1, 0]), ([1, 30], [1, 0]), (None, None),
                        ([0, 30], [0, 1])):
        if news is None:  # the first request ends; its pages are free
            lens[0] = -1000
            attn.attn_pages_free(table, refs, lens, ps, 1 << 30, 0, block_table_out=table,
                                 refs_out=refs)
            length[0] = 0
            continue
        qkv.normal_()
        new.copy_(gpu(np.array(news)))
        g.replay()
        torch.cuda.synchronize()
        assert attn.attn_debug_status() == (
            attn.ATTN_OK if all(t or not n for t, n in zip(takes, news)) else attn.ATTN_ERR_NO_PAGES)
        ref = reference(q, [x if t else -n for x, t, n in zip(length, takes, news)], news,
                        np.maximum(table.cpu().numpy(), 0).astype(np.int64), kc, vc, 1 << 30, 0, 0.125)
        check((o, lse), ref, sum(news))
        length = [x + n * t for x, t, n in zip(length, takes, news)]
        assert lens.tolist()[1] == length[1]


# ------------------------------------------------------------------ large scores
@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), (300, 5)])
def test_chunk_large_scores_choose_one_key(D, window, sinks):
    """Scores of thousands, whose maximum moves far from tile to tile: the result is the best
    key's V where that key is clearly the best.

    A score is a sum of D products in 32 bits, off by at most E = (D + 16) 2^-23 of the sum of
    its terms' sizes, scale and LSE's roundings included; the LSE of a row moves by no
    more than its scores.  Where the best score leads by 2 E + 25, the others' weights are e^-25
    of the best's each, 6000 of them 1e-7 in all.  The best's own is rounded to bf16 once
    (2^-8; its 32-bit value is what the sum holds), and so is the result."""
    ctxs, news, Hkv, G = [600, 130, 5500, 0], [1, 70, 33, 9], 2, 4
    table, lens, kc, vc = pool(ctxs, news, 32, Hkv, D)
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn(sum(news), Hkv * G, D, generator=g, device="cuda").to(BF) * 30
    kc *= 20
    o, lse = run_chunk(q, news, lens, table, kc, vc, window, sinks, scale=1.0)
    status_ok()
    ref = reference(q, ctxs, news, table, kc, vc, window, sinks, 1.0)
    t0 = clear = rows = 0
    for b, (c, n) in enumerate(zip(ctxs, news)):
        k, v = (x.double() for x in dense(table[b], kc, vc, c + n))
        x = q[t0:t0 + n].double().view(n, Hkv, G, D)
        p, j = torch.arange(c, c + n, device="cuda")[:, None], torch.arange(c + n, device="cuda")
        seen = (j <= p) & ((j > p - window) | (j < sinks))
        s = torch.einsum("nhgd,khd->nhgk", x, k).masked_fill(~seen[:, None, None], -math.inf)
        terms = torch.einsum("nhgd,khd->nhgk", x.abs(), k.abs())
        off = (D + 16) * 2.0 ** -23 * terms.masked_fill(~seen[:, None, None], 0).amax(-1)
        assert bool(((lse[t0:t0 + n].double() - ref[1][t0:t0 + n]).abs()
                     <= off.view(n, -1)).all())
        top = s.topk(min(2, c + n), -1)
        lead = top.values[..., 0] - (top.values[..., 1] if c + n > 1 else -math.inf)
        best = top.indices[..., 0]  # [n, Hkv, G]
        want = v[best, torch.arange(Hkv, device="cuda")[None, :, None]]
        pick = lead > 2 * off + 25
        err = (o[t0:t0 + n].double().view(n, Hkv, G, D) - want).abs() - 2.0 ** -6.99 * want.abs() - 1e-6
        assert float(err[pick].max()) <= 0
        assert bool(torch.isfinite(o[t0:t0 + n]).all())
        clear, rows, t0 = clear + int(pick.sum()), rows + pick.numel(), t0 + n
    assert clear >= 0.9 * rows


# ------------------------------------------------------------------ the bounds-checked build
@pytest.fixture(scope="module")
def dbg():
    lib = ctypes.CDLL(attn_build.build(debug=True))
    i, p = ctypes.c_int, ctypes.c_void_p
    lib.attn_chunk_plan_slots.argtypes = [p] * 4 + [i] * 8 + [p]
    lib.attn_chunk_paged.argtypes = [p] * 8 + [i] * 8 + [ctypes.c_float, p]
    lib.attn_debug_status.argtypes = [p]
    return lib


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctxs,news,G,window,sinks,offset", [
    ([9000, 12, 900, 40], [60, 100, 1, 1], 3, 1 << 30, 0, 8),   # cut and whole items
    ([5, 300, 0, 2000, 77], [300, 257, 1, 129, 0], 4, 200, 7, 0),
    ([30, 0, 500], [1, 1, 1], 1, 1 << 30, 0, 0),
    ([100, 900], [9, 140], 130, 1 << 30, 0, 8),                 # more heads than a tile's rows
])
def test_debug_build_chunk_matches_release(dbg, ctxs, news, G, D, window, sinks, offset):
    """Every store of the attention of new tokens checked against its buffer: none outside, and
    the release library's bits; rows behind the last request left as they were."""
    Hkv, ps, spare = 2, 64, 3
    table, lens, kc, vc = pool(ctxs, news, ps, Hkv, D)
    T, Hq, B = sum(news) + spare, Hkv * G, len(news)
    q = torch.randn(T, Hq, D, device="cuda").to(BF)
    want = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in (((T, Hq, D), BF), ((T, Hq), torch.float32))]
    run_chunk(q, news, lens, table, kc, vc, window, sinks, o=want[0], lse=want[1])
    status_ok()
    n, size = ctypes.c_longlong(), ctypes.c_longlong()
    lib = attn.load_library()
    assert lib.attn_chunk_plan_size(B, T, Hq, Hkv, D, ctypes.byref(n)) == 0
    assert lib.attn_chunk_workspace(D, ctypes.byref(size)) == 0
    plan = torch.empty(n.value, dtype=torch.int32, device="cuda")
    ws = torch.empty(size.value, device="cuda")
    cu, ln, tab, slots = gpu(np.concatenate([[0], np.cumsum(news)]), lens, table, np.zeros(T))
    buf = torch.full((q.numel() + offset,), 7.0, dtype=BF, device="cuda")
    o, lse = buf[offset:].view_as(q), torch.full((T, Hq), 7.0, device="cuda")
    stream, M = torch.cuda.current_stream().cuda_stream, table.shape[1]
    assert dbg.attn_chunk_plan_slots(cu.data_ptr(), ln.data_ptr(), slots.data_ptr(), plan.data_ptr(), B, T,
                                     Hq, Hkv, D, M * ps, window, sinks, stream) == 0
    assert dbg.attn_chunk_paged(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), tab.data_ptr(),
                                plan.data_ptr(), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), B, T, Hq,
                                Hkv, kc.shape[0], ps, M, D, 1 / math.sqrt(D), stream) == 0
    assert dbg.attn_debug_status(None) == attn.ATTN_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert bool((o[T - spare:] == 7).all())
