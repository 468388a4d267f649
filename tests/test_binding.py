"""The compiled binding (csrc/binding.cpp) of the windowed and page calls."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import tensor_attn_fwd_gb300 as attn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# A stand-in for the library's launches, which says whether its caller held Python's lock.
STAND_IN = r"""
#include <Python.h>
#define F(name) int name() { return PyGILState_Check() ? 4 : 0; }
F(attn_window_fwd) F(attn_window_bwd) F(attn_decode_window) F(attn_decode_window_paged)
F(attn_pages_free) F(attn_pages_fork) F(attn_pages_compact) F(attn_pages_copy)
"""
CALLS = r"""
import ctypes, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # found before libattn.so's own
sys.path[:0] = [sys.argv[2], sys.argv[2] + "/tests"]
import torch
import tensor_attn_fwd_gb300 as attn
from test_binding import _tensors
q, k, cache, table, refs, lens, parents = _tensors()
q1 = q[:, :, :1].contiguous()
o, lse = attn.attn_window_fwd(q, k, k, 100, num_splits=1)
for call in (lambda: attn.attn_window_fwd(q, k, k, 100),
             lambda: attn.attn_window_fwd(q, k, k, 100, num_splits=2, o=o, lse=lse),
             lambda: attn.attn_window_bwd(q, k, k, o, lse, q, 100),
             lambda: attn.decode_window(q1, k, k, 100),
             lambda: attn.decode_window_paged(q1, cache, cache, table, lens, 100),
             lambda: attn.attn_pages_free(table, refs, lens, 64, 100),
             lambda: attn.attn_pages_fork(table, refs, lens, parents, 64),
             lambda: attn.attn_pages_compact(table, refs),
             lambda: attn.attn_pages_copy(cache, cache, table[0], table[0])):
    call()
"""


@pytest.mark.gpu
def test_launches_do_not_hold_the_interpreters_lock(tmp_path):
    # A launch can wait for the GPU; the other threads, and host functions in a stream that
    # need the lock, have to go on meanwhile.
    src, lib = tmp_path / "stand_in.c", tmp_path / "stand_in.so"
    src.write_text(STAND_IN)
    subprocess.run(["gcc", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], str(src),
                    "-o", str(lib)], check=True)
    r = subprocess.run([sys.executable, "-c", CALLS, str(lib), ROOT], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.gpu
@pytest.mark.parametrize("B,M,P", [(1, 1, 1), (3, 5, 21), (7, 9, 130), (50, 33, 5001), (300, 5, 9999)])
def test_page_results_begin_at_16_bytes_and_do_not_overlap(B, M, P):
    # One allocation, from which the next calls read and write in vectors.
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    parents = torch.arange(B, dtype=torch.int32, device="cuda")
    for results in (attn.attn_pages_free(table, refs, lens, 4),
                    attn.attn_pages_fork(table, refs, lens, parents, 4),
                    attn.attn_pages_compact(table, refs)):
        spans = []
        for t in results:
            assert t.data_ptr() % 16 == 0
            spans.append((t.storage_offset(), t.storage_offset() + t.numel()))
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        assert spans[-1][1] * 4 <= results[0].untyped_storage().nbytes()
