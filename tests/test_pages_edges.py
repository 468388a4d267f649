"""Page calls at the edges of what the documentation allows: limits, inconsistent tables,
finished rows, and the results' layout."""
import numpy as np
import pytest
import torch

import tensor_attn_fwd_gb300 as attn

from test_pages import UNS, c_fork, cache_tables, gpu, plain_fork, plain_free, same


# ------------------------------------------------------------------ limits (no GPU)
@pytest.mark.parametrize("R", [(1 << 30) + 1, (1 << 31) - 1])
def test_fork_refuses_more_rows_than_its_loops_count(R):
    # One slot a row: R * max_pages is below 2^31, but a row number past 2^30 plus the
    # threads of a grid is not.
    assert c_fork(R=R, M=1) == UNS


# ------------------------------------------------------------------ inconsistent input
@pytest.mark.gpu
@pytest.mark.parametrize("pair", [(-2, -5), (-1, -3), (-2, -1), (-(2 ** 31), -1)])
def test_copy_reports_every_pair_that_is_no_page(pair):
    # Only -1, -1 is an unused place of the list.
    k = torch.arange(32, device="cuda").to(torch.bfloat16).view(4, 8)
    v = k + 1
    kw, vw = k.clone(), v.clone()
    attn.attn_pages_copy(k, v, *gpu([pair[0], -1], [pair[1], -1]))
    assert attn.attn_debug_status() == attn.ATTN_ERR_INVALID_ARG
    assert torch.equal(k, kw) and torch.equal(v, vw)


# B, P: one CTA; one cluster; a cooperative grid
FORMS = [(12, 500), (300, 9000), (2000, 70000)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,P", FORMS)
@pytest.mark.parametrize("room", [0, 40])
def test_fork_reports_entries_whose_page_counts_no_holder(B, P, room):
    # Such a page is in the free list: kept in a row it would be handed to another as well.
    rng = np.random.default_rng(B + room)
    table, refs, lens = cache_tables(rng, B, 20, P, 32, 0.7, 0.5)
    named = np.unique(table[table >= 0])
    refs[rng.choice(named, 5 + len(named) // 10, replace=False)] = 0
    refs[rng.choice(named, 2, replace=False)] = -3
    parents = rng.integers(-1, B, B)
    consistent = np.where((table >= 0) & (refs[table] > 0), table, -1)
    want = plain_fork(consistent, refs, lens, parents, 32, room)
    assert want[5][0] <= want[5][1]
    got = attn.attn_pages_fork(*gpu(table, refs, lens, parents), 32, room)
    assert attn.attn_debug_status() == attn.ATTN_ERR_INVALID_ARG
    same(got, want, ("table", "refs", "seqlens", "src", "dst", "counts"))


# ------------------------------------------------------------------ finished rows
@pytest.mark.gpu
@pytest.mark.parametrize("B,P", FORMS)
@pytest.mark.parametrize("kind", ["same", "beams"])
def test_fork_keeps_finished_rows_finished(B, P, kind):
    # free, fork with room, free: a finished row takes no pages and keeps its mark.
    rng = np.random.default_rng(B)
    page, room = 32, 40
    table, refs, lens = cache_tables(rng, B, 20, P, page, 0.7, 0.5)
    done = rng.random(B) < 0.3
    done[0] = True
    lens[done] = -rng.integers(1, 1000, done.sum())
    parents = np.arange(B) if kind == "same" else rng.integers(-1, B, B)
    for freed_first in (False, True):
        t, r = (plain_free(table, refs, lens, page, 10 ** 9, 0) if freed_first else (table, refs))
        live = np.where((parents >= 0) & (lens[parents] < 0), -1, parents)
        want = list(plain_fork(t, r, lens, live, page, room))
        want[2] = np.where((parents >= 0) & (lens[parents] < 0), lens[parents], want[2])
        got = attn.attn_pages_fork(*gpu(t, r, lens, parents), page, room)
        assert attn.attn_debug_status() == attn.ATTN_OK
        same(got, want, ("table", "refs", "seqlens", "src", "dst", "counts"))
        again = attn.attn_pages_free(got[0], got[1], got[2], page, room=room)
        same(again, plain_free(want[0], want[1], want[2], page, 10 ** 9, 0, room), ("table", "refs"))
        assert bool((again[0][torch.from_numpy(want[2] < 0).cuda()] == -1).all())
    # A length as low as it gets.
    args = gpu([[0, 1], [2, -1]], [1, 1, 1, 0, 0, 0], [-(2 ** 31), 3], [0, 1])
    got = attn.attn_pages_fork(*args, 4, room=2)
    same(got, ([[-1, -1], [2, 3]], [0, 0, 1, 1, 0, 0], [-(2 ** 31), 3], [-1, -1], [-1, -1], [1, 3]),
         ("table", "refs", "seqlens", "src", "dst", "counts"))
