"""A serving step at the edges of what the documentation allows: large tables that are copied
beside the call's own work, rows that are refused, large scores, the bounds-checked build."""
import numpy as np
import pytest
import torch

import tensor_attn_fwd_gb300 as attn

from test_step import APPEND, INV, append_case, gpu, plain_append, same, status_ok


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
