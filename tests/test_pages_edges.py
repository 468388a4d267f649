"""Page calls at the edges of what the documentation allows: limits, inconsistent tables,
finished rows, and the results' layout."""
import numpy as np
import pytest
import torch

import tensor_attn_fwd_gb300 as attn

from test_pages import A, A2, A3, UNS, c_fork, gpu, plain_fork, same  # noqa: F401


# ------------------------------------------------------------------ limits (no GPU)
@pytest.mark.parametrize("R", [(1 << 30) + 1, (1 << 31) - 1])
def test_fork_refuses_more_rows_than_its_loops_count(R):
    # One slot a row: R * max_pages is below 2^31, but a row number past 2^30 plus the
    # threads of a grid is not.
    assert c_fork(R=R, M=1) == UNS
