"""The compiled binding (csrc/binding.cpp) of the windowed and page calls."""
import pytest
import torch

import tensor_attn_fwd_gb300 as attn


def _tensors():
    q = torch.randn(1, 2, 8, 64, device="cuda").to(torch.bfloat16)
    k = torch.randn(1, 1, 300, 64, device="cuda").to(torch.bfloat16)
    cache = torch.randn(8, 1, 64, 64, device="cuda").to(torch.bfloat16)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    refs = torch.ones(8, dtype=torch.int32, device="cuda")
    lens = torch.full((1,), 200, dtype=torch.int32, device="cuda")
    parents = torch.zeros(1, dtype=torch.int32, device="cuda")
    return q, k, cache, table, refs, lens, parents


@pytest.mark.gpu
@pytest.mark.parametrize("n", [-1, -(2 ** 31) - 1, 2 - 2 ** 32, 64 - 2 ** 32, 64 - 2 ** 40, -(2 ** 63), -(10 ** 30)])
def test_no_negative_number_passes_for_a_positive_one(n):
    q, k, cache, table, refs, lens, parents = _tensors()
    q1 = q[:, :, :1].contiguous()
    for call in (lambda: attn.attn_window_fwd(q, k, k, 100, num_splits=n),
                 lambda: attn.decode_window(q1, k, k, 100, num_splits=n),
                 lambda: attn.decode_window_paged(q1, cache, cache, table, lens, 100, num_splits=n),
                 lambda: attn.attn_pages_free(table, refs, lens, n, 100),
                 lambda: attn.attn_pages_fork(table, refs, lens, parents, n)):
        with pytest.raises(attn.AttnError, match="INVALID_ARG"):
            call()
