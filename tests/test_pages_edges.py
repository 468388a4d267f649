"""Page calls at the edges of what the documentation allows: limits, inconsistent tables,
finished rows, and the results' layout."""
import numpy as np
import pytest
import torch

import tensor_attn_fwd_gb300 as attn

from test_pages import A, A2, A3, UNS, c_fork, cache_tables, gpu, plain_fork, same  # noqa: F401


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
