"""Windowed attention at the edges of what the documentation allows: workspace sizes and
what they refuse."""
import ctypes

import pytest
import torch

import tensor_attn_fwd_gb300 as attn

from test_window import _lib

INV, UNS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED


# ------------------------------------------------------------------ workspaces
# B, Hq, Hkv, Sq, D: one item; even and odd groups of heads; few and many rounds
WORKSPACES = [(1, 2, 1, 8, 64), (1, 2, 2, 8, 64), (1, 4, 2, 300, 128), (1, 3, 1, 300, 128), (2, 6, 2, 513, 64),
              (1, 4, 1, 129, 256), (3, 5, 5, 200, 256), (1, 80, 40, 600, 64), (2, 45, 45, 500, 128),
              (1, 90, 30, 250, 256), (1, 152, 76, 200, 64)]


def workspace_floats(B, Hq, Hkv, Sq, D, splits, n_sm):
    """fp32 O and LSE of every row of the items that the last round of CTAs holds."""
    if splits == 1:
        return 0
    pairs = D < 256 and Hq // Hkv % 2 == 0  # an item: a 128-row tile of two heads
    tile_rows = 128 if pairs or D == 256 else 256
    items = B * (Hq // 2 if pairs else Hq) * -(-Sq // tile_rows)
    return items % n_sm * splits * (128 if D == 256 else 256) * (D + 1)


def check_workspaces(n_sm):
    for case in WORKSPACES:
        for splits in (1, 2, 3, 32):
            n = ctypes.c_longlong(-1)
            assert _lib().attn_window_fwd_workspace(*case, splits, ctypes.byref(n)) == attn.ATTN_OK
            assert n.value == workspace_floats(*case, splits, n_sm), (case, splits)


def test_forward_workspace_without_a_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    check_workspaces(1)  # a device of unknown size counts as one SM: every round is full


@pytest.mark.gpu
def test_forward_workspace_holds_the_partials_of_the_last_round():
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    check_workspaces(n_sm)
    assert any(workspace_floats(*case, 2, n_sm) for case in WORKSPACES)


# B, Hq, Hkv, Sq, D: too many elements; too many 128-row tiles; too many heads
@pytest.mark.parametrize("case", [(1, 1 << 10, 1, 1 << 30, 128), (1 << 20, 1 << 10, 1, 129, 64),
                                  (1 << 21, 1 << 10, 1, 8, 64), (1, 2, 1, (1 << 30) + 1, 64),
                                  (2 ** 31 - 1, 2 ** 31 - 1, 1, 2 ** 31 - 1, 128)])
@pytest.mark.parametrize("splits", [1, 2])
def test_forward_workspace_refuses_the_sizes_that_the_call_refuses(case, splits):
    n = ctypes.c_longlong(-1)
    assert _lib().attn_window_fwd_workspace(*case, splits, ctypes.byref(n)) == UNS
    A = 0x10000000
    B, Hq, Hkv, Sq, D = case
    assert _lib().attn_window_fwd(A, A, A, A, A, A, B, Hq, Hkv, Sq, 1000, D, 10, 1, splits, 0.1, None) == UNS


# B, Hq, Hkv, Sq, Sk, D
@pytest.mark.parametrize("case", [(1, 1 << 10, 1, 1 << 30, 8, 128), (1, 1 << 10, 1 << 10, 8, 1 << 30, 128),
                                  (1, 1 << 10, 1, 1 << 21, 8, 64), (1 << 20, 1 << 10, 1 << 10, 1, 200, 64),
                                  (1 << 21, 1 << 10, 1, 1, 8, 64), (1, 2, 1, 8, (1 << 30) + 1, 64),
                                  (2 ** 31 - 1, 2 ** 31 - 1, 1, 2 ** 31 - 1, 2 ** 31 - 1, 128),
                                  (1, 2, 1, 8, 8, 256)])
def test_backward_workspace_refuses_the_sizes_that_the_call_refuses(case):
    n = ctypes.c_longlong(-1)
    assert _lib().attn_window_bwd_workspace(*case, 10, 1, ctypes.byref(n)) == UNS
    A = 0x10000000
    assert _lib().attn_window_bwd(*[A] * 10, *case, 10, 1, 0.1, None) == UNS


# ------------------------------------------------------------------ products past 64 bits
@pytest.mark.parametrize("call", ["attn_fwd", "attn_window_fwd"])
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk", [(1 << 30, 1 << 30, 1, 1 << 30, 8), (1 << 30, 1 << 30, 1, 1 << 28, 8),
                                            (1 << 29, 1 << 30, 1 << 30, 1 << 30, 1 << 30)])
def test_sizes_whose_product_wraps_are_refused(call, B, Hq, Hkv, Sq, Sk):
    A = 0x10000000
    if call == "attn_fwd":
        status = _lib().attn_fwd(A, A, A, A, A, B, Hq, Hkv, Sq, Sk, 64, 1, 0.1, None)
    else:
        status = _lib().attn_window_fwd(A, A, A, A, A, None, B, Hq, Hkv, Sq, Sk, 64, 10, 1, 1, 0.1, None)
    assert status == UNS
