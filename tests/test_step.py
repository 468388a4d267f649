"""A serving step over a paged cache: slots of new tokens, rotary positions, attention of
the new tokens; each against its formula in 64 bits, and a run of them together."""
import math

import numpy as np
import pytest
import torch

import tensor_attn_fwd_gb300 as attn

INV, UNS, MIS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_MISALIGNED
BF = torch.bfloat16
F64 = torch.float64


@pytest.fixture(scope="module")
def lib():
    return attn.load_library()


def gpu(*arrays):
    out = [torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda() for a in arrays]
    return out if len(out) > 1 else out[0]


def status_ok():
    assert attn.attn_debug_status() == attn.ATTN_OK


# ================================================================== refusals (no GPU)
# Fake, never-dereferenced device addresses: validation fails before any launch.
A = 0x10000000       # 16-byte aligned
M4 = 0x10000004      # 4-byte aligned
M2 = 0x10000002


def c_append(lib, bt=A, refs=A, sl=A, nl=A + 256, bto=A, ro=A, slo=A, cu=A, pos=A, slots=A, cnt=A, ws=A,
             B=2, T=8, M=4, P=16, ps=32):
    return lib.attn_pages_append(bt, refs, sl, nl, bto, ro, slo, cu, pos, slots, cnt, ws, B, T, M, P,
                                 ps, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INV) for n in ("bt", "refs", "sl", "nl", "bto", "ro", "slo", "cu", "pos", "slots",
                                 "cnt", "ws")],
    *[({n: M2}, MIS) for n in ("bt", "refs", "sl", "nl", "bto", "ro", "slo", "cu", "pos", "slots",
                               "cnt", "ws")],
    *[({n: 0}, INV) for n in ("B", "T", "M", "P", "ps")],
    *[({n: -1}, INV) for n in ("B", "T", "M", "P", "ps")],
    (dict(B=1 << 16, M=1 << 15), UNS),       # table slots past int
    (dict(M=1 << 20, ps=1 << 11), UNS),      # keys of a row past 2^30
    (dict(P=(1 << 30) + 1), UNS),
    (dict(P=1 << 26, ps=32), UNS),           # cache slots past int
    (dict(T=(1 << 30) + 1), UNS),
])
def test_append_rejects(lib, kw, code):
    assert c_append(lib, **kw) == code


def test_append_rejects_lengths_over_new_ones(lib):
    assert c_append(lib, nl=A + 64, slo=A + 64) == INV


def test_append_workspace_rejects(lib):
    import ctypes
    n = ctypes.c_longlong(-1)
    assert lib.attn_pages_append_workspace(0, 1, ctypes.byref(n)) == INV
    assert lib.attn_pages_append_workspace(1, 0, ctypes.byref(n)) == INV
    assert lib.attn_pages_append_workspace(1, 1, None) == INV
    assert lib.attn_pages_append_workspace(10, 3, ctypes.byref(n)) == 0 and n.value >= 10 + 9


def c_split(lib, qkv=A, ld=512, tab=A, pos=None, q=A, k=A, v=A, B=1, S=4, Hq=4, Hkv=2, D=64, R=64,
            mp=16, style=0):
    return lib.attn_rope_split(qkv, ld, tab, pos, q, k, v, B, S, Hq, Hkv, D, R, mp, style, None)


def c_split_bwd(lib, qkv=A, ld=512, tab=A, pos=None, q=A, k=A, v=A, fp32=0, B=1, S=4, Hq=4, Hkv=2,
                D=64, R=64, mp=16, style=0):
    return lib.attn_rope_split_bwd(q, k, v, fp32, tab, pos, qkv, ld, B, S, Hq, Hkv, D, R, mp, style,
                                   None)


def c_rope_append(lib, qkv=A, ld=512, tab=A, pos=A, slots=A, q=A, k=A, v=A, S=4, Hq=4, Hkv=2, D=64,
                  R=64, mp=16, P=4, ps=32, style=0, B=1):
    return lib.attn_rope_append(qkv, ld, tab, pos, slots, q, k, v, S * B, Hq, Hkv, D, R, mp, P, ps,
                                style, None)


ROPE_BAD = [
    *[({n: None}, INV) for n in ("qkv", "tab", "q", "k", "v")],
    *[({n: M4}, MIS) for n in ("qkv", "tab", "q", "k", "v")],
    *[({n: 0}, INV) for n in ("S", "Hq", "Hkv", "D", "R", "mp", "B")],
    (dict(pos=M2), MIS),
    (dict(Hq=3), INV), (dict(style=2), INV), (dict(style=-1), INV),
    (dict(ld=504), INV),                     # shorter than the heads
    (dict(ld=516), UNS),                     # rows off 16 bytes
    (dict(R=128), INV), (dict(R=24), UNS), (dict(R=8), UNS),
    (dict(D=96, ld=768), UNS),
    (dict(S=(1 << 30) + 1, mp=(1 << 30) + 1), UNS),
    (dict(ld=1 << 39, S=16), UNS),
    (dict(Hq=1 << 25, Hkv=1, ld=1 << 40), UNS),
]


@pytest.mark.parametrize("kw,code", ROPE_BAD)
def test_rope_rejects(lib, kw, code):
    assert c_split(lib, **kw) == code
    assert c_split_bwd(lib, **kw) == code
    assert c_rope_append(lib, **kw) == code


def test_rope_rejects_more(lib):
    assert c_split(lib, S=17) == INV and c_split_bwd(lib, S=17) == INV  # table shorter than s
    assert c_split_bwd(lib, fp32=2) == INV
    assert c_rope_append(lib, pos=None) == INV and c_rope_append(lib, slots=None) == INV
    assert c_rope_append(lib, slots=M2) == MIS
    assert c_rope_append(lib, P=0) == INV and c_rope_append(lib, ps=0) == INV
    assert c_rope_append(lib, P=1 << 26) == UNS  # slots past int


@pytest.mark.parametrize("kw,code", [
    (dict(t=None), INV), (dict(t=M4), MIS), (dict(mp=0), INV), (dict(R=0), INV), (dict(R=3), INV),
    (dict(base=1.0), INV), (dict(base=math.inf), INV), (dict(base=math.nan), INV),
    (dict(factor=0.0), INV), (dict(factor=-1.0), INV), (dict(factor=math.inf), INV),
    (dict(factor=math.nan), INV), (dict(amp=0.0), INV), (dict(amp=math.nan), INV),
    (dict(orig=-1), INV), (dict(orig=10, low=2.0, high=2.0), INV),
    (dict(orig=10, low=-1.0), INV), (dict(orig=10, high=math.inf), INV),
    (dict(orig=10, low=math.nan), INV), (dict(mp=1 << 30, R=1 << 12), UNS),
])
def test_rope_table_scaled_rejects(lib, kw, code):
    d = dict(t=A, mp=16, R=64, base=1e4, factor=2.0, low=1.0, high=4.0, orig=0, amp=1.0)
    d.update(kw)
    assert lib.attn_rope_table_scaled(d["t"], d["mp"], d["R"], d["base"], d["factor"], d["low"],
                                      d["high"], d["orig"], d["amp"], None) == code


def c_plan(lib, cu=A, sl=A, plan=A, B=2, T=8, Hq=4, Hkv=2, D=64, mk=128, window=1 << 30, sinks=0):
    return lib.attn_chunk_plan(cu, sl, plan, B, T, Hq, Hkv, D, mk, window, sinks, None)


def c_chunk(lib, q=A, k=A, v=A, bt=A, plan=A, o=A, lse=A, ws=A, B=2, T=8, Hq=4, Hkv=2, P=8, ps=32,
            M=4, D=64, scale=0.1):
    return lib.attn_chunk_paged(q, k, v, bt, plan, o, lse, ws, B, T, Hq, Hkv, P, ps, M, D, scale, None)


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INV) for n in ("cu", "sl", "plan")],
    (dict(cu=M2), MIS), (dict(sl=M2), MIS), (dict(plan=M4), MIS),
    *[({n: 0}, INV) for n in ("B", "T", "Hq", "Hkv", "D", "mk", "window")],
    (dict(sinks=-1), INV), (dict(Hq=3), INV), (dict(D=512), UNS), (dict(D=96), UNS),
    (dict(mk=(1 << 30) + 1), UNS), (dict(T=1 << 30), UNS),
    (dict(B=1 << 26, T=1, Hkv=2), UNS),      # items past the plan's count
])
def test_chunk_plan_rejects(lib, kw, code):
    assert c_plan(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    *[({n: None}, INV) for n in ("q", "k", "v", "bt", "plan", "o", "lse", "ws")],
    *[({n: M4}, MIS) for n in ("q", "k", "v", "plan", "o", "lse", "ws")],
    (dict(bt=M2), MIS),
    *[({n: 0}, INV) for n in ("B", "T", "Hq", "Hkv", "D", "P", "ps", "M")],
    (dict(Hq=3), INV), (dict(D=512), UNS), (dict(ps=48), UNS), (dict(scale=0.0), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
    (dict(P=1 << 25, ps=32), UNS),           # rows of the caches past a coordinate
    (dict(M=1 << 20, ps=1 << 11), UNS),
])
def test_chunk_rejects(lib, kw, code):
    assert c_chunk(lib, **kw) == code


def test_chunk_sizes_reject(lib):
    import ctypes
    n = ctypes.c_longlong(-1)
    assert lib.attn_chunk_plan_size(1, 1, 4, 2, 64, None) == INV
    assert lib.attn_chunk_plan_size(1, 1, 4, 3, 64, ctypes.byref(n)) == INV
    assert lib.attn_chunk_plan_size(1, 1, 4, 2, 512, ctypes.byref(n)) == UNS
    assert lib.attn_chunk_workspace(64, None) == INV
    assert lib.attn_chunk_workspace(0, ctypes.byref(n)) == INV
    assert lib.attn_chunk_workspace(512, ctypes.byref(n)) == UNS


def test_python_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(2, 3, 512, dtype=BF)
    with pytest.raises(ValueError):
        attn.attn_pages_append(i.view(2, 2), i, i[:2], i[:2], 4, 32)
    with pytest.raises(ValueError):
        attn.attn_rope_split(x, torch.zeros(4, 32, 2), 4, 2)
    with pytest.raises(ValueError):
        attn.attn_rope_append(x[0], torch.zeros(4, 32, 2), i, i, x.view(1, 2, 24, 64),
                              x.view(1, 2, 24, 64), 4)
    with pytest.raises(ValueError):
        attn.attn_chunk_plan(i, i[:3], 4, 4, 2, 64, 128)
    with pytest.raises(ValueError):
        attn.attn_chunk_paged(x, x.view(1, 2, 24, 64), x.view(1, 2, 24, 64), i.view(2, 2), i)


# ================================================================== append
def plain_append(table, refs, lens, new, T, ps):
    table, refs = table.copy(), refs.copy()
    B, M = table.shape
    table[(table < -1) | (table >= refs.size)] = -1
    free = [int(p) for p in np.nonzero(refs == 0)[0]]
    counts, out, cu = [0, len(free)], lens.copy(), [0]
    pos, slots = np.zeros(T, dtype=np.int64), np.full(T, -1, dtype=np.int64)
    total = 0
    for b in range(B):
        n, x = max(int(new[b]), 0), int(lens[b])
        t0, total = total, total + n
        cu.append(min(total, T))
        if n == 0 or x < 0 or x + n > M * ps:
            continue
        want = [j for j in range(x // ps, (x + n - 1) // ps + 1) if table[b, j] < 0]
        counts[0] += len(want)
        if counts[0] > counts[1] or total > T:
            continue
        for j in want:
            table[b, j] = free.pop(0)
            refs[table[b, j]] = 1
        out[b] = x + n
        for i in range(n):
            pos[t0 + i] = x + i
            slots[t0 + i] = table[b, (x + i) // ps] * ps + (x + i) % ps
    return table, refs, out, np.array(cu), pos, slots, np.array(counts)


APPEND_NAMES = ("table", "refs", "seqlens", "cu", "positions", "slots", "counts")


def same(got, want):
    for g, w, name in zip(got, want, APPEND_NAMES):
        assert g.dtype == torch.int32
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)


def append_case(rng, B, M, P, ps, most_new, reserved=0.0):
    lens = rng.integers(0, M * ps - most_new + 1, B)
    new = rng.integers(0, most_new + 1, B)
    pages = -(-lens // ps)
    ids = rng.permutation(P)
    table = np.full((B, M), -1)
    at = 0
    for b in range(B):
        n = min(int(pages[b]), 3)  # the last pages: those before are passed by a window
        table[b, pages[b] - n:pages[b]] = ids[at:at + n]
        at += n
        for j in range(pages[b], M):  # reserved pages, with holes
            if rng.random() < reserved and at < P // 2:
                table[b, j] = ids[at]
                at += 1
    assert at <= P
    refs = np.bincount(table[table >= 0], minlength=P)
    return table, refs, lens, new


# rows, slots, pages, page size, new tokens: one CTA; a cluster; one with CTAs that copy; rows of
# many slots; many pages a warp; more rows than threads
APPEND = [(1, 1, 1, 32, 32), (1, 5, 40, 32, 1), (7, 9, 100, 64, 70), (64, 16, 1000, 96, 300),
          (300, 33, 6000, 32, 9), (900, 100, 20000, 128, 500), (2500, 20, 60000, 32, 200),
          (12, 300, 3000, 32, 4000), (40, 20, 1200001, 32, 100), (20000, 3, 70001, 32, 40),
          (2, 129, 700, 32, 4000), (60, 128, 8192, 64, 130), (1000, 8, 8192, 64, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,M,P,ps,most", APPEND)
@pytest.mark.parametrize("reserved", [0.0, 0.5])
@pytest.mark.parametrize("pad", [0, 37])
def test_append(B, M, P, ps, most, reserved, pad):
    rng = np.random.default_rng(B + M + pad)
    table, refs, lens, new = append_case(rng, B, M, P, ps, most, reserved)
    T = max(int(new.sum()) + pad, 1)
    want = plain_append(table, refs, lens, new, T, ps)
    inputs = gpu(table, refs, lens, new)
    kept = [t.clone() for t in inputs]
    same(attn.attn_pages_append(*inputs, T, ps), want)
    if want[6][0] <= want[6][1]:
        status_ok()
    else:
        assert attn.attn_debug_status() == attn.ATTN_ERR_NO_PAGES
    assert all(torch.equal(a, b) for a, b in zip(inputs, kept))
    # In place.
    got = attn.attn_pages_append(*inputs, T, ps, block_table_out=inputs[0], refs_out=inputs[1],
                                 seqlens_out=inputs[2])
    assert got[0] is not None and got[0].data_ptr() == inputs[0].data_ptr()
    same(got, want)
    attn.attn_debug_status()


@pytest.mark.gpu
@pytest.mark.parametrize("B,M,P,ps,most", APPEND[2:])
def test_append_without_enough_pages(B, M, P, ps, most):
    # Rows take all or none, in order; those that need no page still take their tokens.
    rng = np.random.default_rng(B)
    table, refs, lens, new = append_case(rng, B, M, P, ps, most)
    free = np.nonzero(refs == 0)[0]
    refs[free[len(free) // 5:]] = 1
    need = plain_append(table, refs, lens, new, int(new.sum()), ps)[6]
    keep = max(1, need[0] // 2)
    refs[np.nonzero(refs == 0)[0][keep:]] = 1
    want = plain_append(table, refs, lens, new, int(new.sum()), ps)
    assert want[6][0] > want[6][1]
    took = want[2] != lens
    assert not took[new > 0].all()
    same(attn.attn_pages_append(*gpu(table, refs, lens, new), int(new.sum()), ps), want)
    assert attn.attn_debug_status() == attn.ATTN_ERR_NO_PAGES


@pytest.mark.gpu
@pytest.mark.parametrize("B,M,P,ps,most", APPEND[2:])
def test_append_finished_and_bad_rows(B, M, P, ps, most):
    rng = np.random.default_rng(B + 1)
    table, refs, lens, new = append_case(rng, B, M, P, ps, most)
    lens[rng.random(B) < 0.2] = -(1 << 30)
    same(attn.attn_pages_append(*gpu(table, refs, lens, new), int(new.sum()), ps),
         plain_append(table, refs, lens, new, int(new.sum()), ps))
    status_ok()
    for what in ("negative", "capacity", "tokens", "entry", "huge"):
        t, n, T = table.copy(), new.copy(), int(new.sum())
        n[B // 2] = max(n[B // 2], 1)
        T = int(n.sum())
        ln = np.maximum(lens, 0)
        if what == "negative":
            n[B // 2] = -5
            T = int(np.maximum(n, 0).sum())
        elif what == "capacity":
            ln[B // 2] = M * ps
        elif what == "tokens":
            T = max(T - 1 - int(n[-1]), 1)
        elif what == "entry":
            t[B // 2, 0] = P
            t[B // 3, M - 1] = -2
        else:
            n[:] = (1 << 31) - 1  # sums far past int
            T = 100
        want = plain_append(t, refs, ln, n, T, ps)
        same(attn.attn_pages_append(*gpu(t, refs, ln, n), T, ps), want)
        assert attn.attn_debug_status() == INV, what


@pytest.mark.gpu
def test_append_python_checks():
    table, refs, lens, new = gpu(np.full((2, 3), -1), np.zeros(9), np.zeros(2), np.ones(2))
    for bad in [dict(tokens=0), dict(tokens="x"), dict(new=new[:1]), dict(lens=lens.long()),
                dict(out=refs)]:
        d = dict(tokens=2, new=new, lens=lens, out=None)
        d.update(bad)
        with pytest.raises((ValueError, TypeError)):
            attn.attn_pages_append(table, refs, d["lens"], d["new"], d["tokens"], 32,
                                   block_table_out=d["out"])
    with pytest.raises(attn.AttnError):
        attn.attn_pages_append(table, refs, lens, new, 2, 0)


@pytest.mark.gpu
def test_append_decode_loop_in_a_graph():
    # Captured once with its inputs as outputs, replayed: one token a row and replay.
    B, M, P, ps = 5, 4, 30, 32
    table, refs, lens = gpu(np.full((B, M), -1), np.zeros(P), np.arange(B) * 7)
    new = gpu(np.ones(B))
    t0, r0, l0 = (x.cpu().numpy() for x in (table, refs, lens))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        attn.attn_pages_append(table.clone(), refs.clone(), lens.clone(), new, B, ps)  # warm-up
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = attn.attn_pages_append(table, refs, lens, new, B, ps, block_table_out=table,
                                         refs_out=refs, seqlens_out=lens)
    for _ in range(70):
        want = plain_append(t0, r0, l0, np.ones(B, dtype=np.int64), B, ps)
        g.replay()
        torch.cuda.synchronize()
        same(out, want)
        t0, r0, l0 = want[:3]
    status_ok()


# ================================================================== rotary positions
def turn(x, cs, style, sign=1):
    """x [..., H, D] in 64 bits, cs [..., R/2, 2] of the tokens: the first R dims turned."""
    R = 2 * cs.shape[-2]
    c, s = cs[..., None, :, 0], sign * cs[..., None, :, 1]
    y = x.clone()
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if style == 0 else (i, i + R // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def near(got, want, size):
    """Rounded once to bf16 (half a step: 2^-8 of the value), after at most four roundings
    in 32 bits of terms as large as ``size``."""
    assert got.dtype == BF
    err = (got.double().cpu() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + 4 * 2.0 ** -24 * size).all()), float(err.max())


ROPE = [  # B, S, Hq, Hkv, D, R
    (1, 1, 1, 1, 64, 16), (2, 5, 4, 2, 64, 64), (1, 33, 6, 3, 64, 48), (2, 17, 8, 1, 128, 128),
    (3, 7, 12, 12, 128, 32), (1, 9, 5, 1, 128, 112), (1, 6, 4, 2, 256, 256), (2, 3, 2, 2, 256, 64),
    (1, 1000, 3, 1, 128, 64)]


def rope_inputs(B, S, Hq, Hkv, D, R, seed=0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, S, (Hq + 2 * Hkv) * D, generator=g).to(BF)
    max_pos = 4 * S + 50
    pos = torch.randint(0, max_pos, (B, S), generator=g, dtype=torch.int32)
    table = attn.attn_rope_table(max_pos, R)
    return g, qkv, pos, table


@pytest.mark.gpu
@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("shape", ROPE)
@pytest.mark.parametrize("given", [False, True])
def test_rope_split_and_gradient(shape, style, given):
    B, S, Hq, Hkv, D, R = shape
    g, qkv, pos, table = rope_inputs(*shape)
    cs = table.double().cpu()[pos.long() if given else torch.arange(S).expand(B, S)]
    x = qkv.double().view(B, S, -1, D)
    arg = pos.cuda() if given else None
    q, k, v = attn.attn_rope_split(qkv.cuda(), table, Hq, Hkv, positions=arg, style=style)
    near(q, turn(x[:, :, :Hq], cs, style).transpose(1, 2), 8)
    near(k, turn(x[:, :, Hq:Hq + Hkv], cs, style).transpose(1, 2), 8)
    assert torch.equal(v.cpu(), qkv.view(B, S, -1, D)[:, :, Hq + Hkv:].transpose(1, 2))
    for dtype in (BF, torch.float32):
        dq, dk, dv = (torch.randn(B, h, S, D, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        got = attn.attn_rope_split_bwd(dq.cuda(), dk.cuda(), dv.cuda(), table, positions=arg,
                                       style=style)
        want = torch.cat([turn(t.double().transpose(1, 2), cs, style, -1) for t in (dq, dk)]
                         + [dv.double().transpose(1, 2)], 2).reshape(B, S, -1)
        near(got, want, 8)
    status_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("style", [0, 1])
def test_rope_gradient_against_differences(style):
    # The map is linear: sum(d * f(x + e)) - sum(d * f(x - e)) = 2 <f^T d, e>, here with the
    # formula's f in 64 bits and the kernel's f^T d, for single elements e.
    B, S, Hq, Hkv, D, R = 1, 4, 2, 1, 64, 32
    g, qkv, pos, _ = rope_inputs(B, S, Hq, Hkv, D, R)
    table = attn.attn_rope_table_scaled(70, R, 1e4, 4.0, 1.0, 8.0, 32, amplitude=1.25)
    cs = table.double().cpu()[pos.long()]
    d = [torch.randn(B, h, S, D, generator=g) for h in (Hq, Hkv, Hkv)]
    grad = attn.attn_rope_split_bwd(*(t.cuda() for t in d), table, positions=pos.cuda(), style=style)
    x = qkv.double()

    def f(x):
        y = x.view(B, S, -1, D)
        y = torch.cat([turn(y[:, :, :Hq + Hkv], cs, style), y[:, :, Hq + Hkv:]], 2).transpose(1, 2)
        return sum(float((a.double() * b).sum())
                   for a, b in zip(d, (y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:])))

    for i in range(0, x.numel(), 13):
        e = torch.zeros(x.numel(), dtype=F64)
        e[i] = 1.0
        e = e.view_as(x)
        want = (f(x + e) - f(x - e)) / 2
        got = float(grad.double().cpu().view(-1)[i])
        assert abs(got - want) <= 2.0 ** -8 * abs(want) + 1e-5, (i, got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("shape", ROPE)
def test_rope_append(shape, style):
    B, S, Hq, Hkv, D, R = shape
    T, P, ps = B * S, B * S // 32 + 3, 32
    g, qkv, pos, table = rope_inputs(*shape, seed=1)
    qkv, pos = qkv.view(T, -1), pos.view(T)
    slots = torch.randperm(P * ps, generator=g)[:T].int()
    slots[::7] = -1
    caches = [torch.randn(P, Hkv, ps, D, generator=g).to(BF).cuda() for _ in range(2)]
    want = [c.double().cpu() for c in caches]
    q = attn.attn_rope_append(qkv.cuda(), table, pos.cuda(), slots.cuda(), *caches, Hq, style=style)
    status_ok()
    x = qkv.double().view(T, -1, D)
    cs = table.double().cpu()[pos.long()]
    near(q, turn(x[:, :Hq], cs, style), 8)
    k = turn(x[:, Hq:Hq + Hkv], cs, style)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[0][s // ps, :, s % ps] = k[t]
            want[1][s // ps, :, s % ps] = x[t, Hq + Hkv:]
    near(caches[0], want[0], 8)
    assert torch.equal(caches[1].double().cpu(), want[1])


@pytest.mark.gpu
def test_rope_rows_of_a_wider_matrix():
    # Rows that are parts of longer ones (a projection beside others), read and written.
    B, S, Hq, Hkv, D, R = 2, 5, 4, 2, 64, 64
    _, qkv, _, table = rope_inputs(B, S, Hq, Hkv, D, R)
    N = qkv.shape[-1]
    wide = torch.full((B, S, N + 72), float("nan"), dtype=BF, device="cuda")
    wide[..., 8:8 + N] = qkv.cuda()
    part = wide[..., 8:8 + N]
    for a, b in zip(attn.attn_rope_split(part, table, Hq, Hkv),
                    attn.attn_rope_split(qkv.cuda(), table, Hq, Hkv)):
        assert torch.equal(a, b)
    d = [torch.randn(B, h, S, D, device="cuda").to(BF) for h in (Hq, Hkv, Hkv)]
    want = attn.attn_rope_split_bwd(*d, table)
    got = attn.attn_rope_split_bwd(*d, table, dqkv=part)
    assert got.data_ptr() == part.data_ptr() and torch.equal(got, want)
    assert bool(torch.isnan(wide[..., :8]).all()) and bool(torch.isnan(wide[..., 8 + N:]).all())
    caches = [torch.zeros(1, Hkv, 32, D, dtype=BF, device="cuda") for _ in range(4)]
    slots, pos = gpu(np.arange(B * S), np.arange(B * S) % 7)
    qa = attn.attn_rope_append(want.view(B * S, N), table, pos, slots, *caches[:2], Hq)
    qb = attn.attn_rope_append(part.reshape(B * S, N), table, pos, slots, *caches[2:], Hq)
    qc = attn.attn_rope_append(wide.view(B * S, -1)[:, 8:8 + N], table, pos, slots, *caches[2:], Hq)
    assert torch.equal(qa, qb) and torch.equal(qa, qc)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    status_ok()
    for bad in (wide[..., 4:4 + N], wide[..., ::2], wide.transpose(0, 1)[..., :N], wide[:, :, :N + 8]):
        with pytest.raises((ValueError, attn.AttnError)):
            attn.attn_rope_split(bad, table, Hq, Hkv)


@pytest.mark.gpu
def test_rope_bad_positions_and_slots():
    T, Hq, Hkv, D, P, ps = 6, 2, 1, 64, 2, 32
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(BF)
    table = attn.attn_rope_table(10, D)
    caches = [torch.zeros(P, Hkv, ps, D, dtype=BF, device="cuda") for _ in range(2)]
    pos = torch.tensor([0, -1, 10, 9, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    slots = torch.tensor([0, 1, 2, 3, 4, 5], dtype=torch.int32)
    q = attn.attn_rope_append(qkv.cuda(), table, pos.cuda(), slots.cuda(), *caches, Hq)
    assert attn.attn_debug_status() == INV
    cs = table.double().cpu()[pos.long().clamp(0, 9)]
    near(q, turn(qkv.double().view(T, -1, D)[:, :Hq], cs, 0), 8)
    before = [c.clone() for c in caches]
    slots = torch.tensor([P * ps, -2, 2 ** 31 - 1, -2 ** 31, -1, -1], dtype=torch.int32)
    attn.attn_rope_append(qkv.cuda(), table, slots.cuda() * 0, slots.cuda(), *caches, Hq)
    assert attn.attn_debug_status() == INV
    assert all(torch.equal(a, b) for a, b in zip(caches, before))
    with pytest.raises(ValueError):
        attn.attn_rope_split(qkv.cuda().view(1, T, -1), table, 3, 1)  # 256 columns, five heads
    with pytest.raises(ValueError):
        attn.attn_rope_append(qkv.cuda(), table, slots[:3].cuda(), slots.cuda(), *caches, Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(), dict(factor=8.0), dict(factor=0.5, amplitude=2.0),
    dict(factor=8.0, low=1.0, high=4.0, original_pos=8192),
    dict(factor=32.0, low=1.0, high=32.0, original_pos=4096, amplitude=0.1 * math.log(32) + 1)])
@pytest.mark.parametrize("R,base", [(128, 500000.0), (48, 10000.0), (2, 10.0)])
def test_rope_table_scaled(kw, R, base):
    max_pos = 40000
    got = attn.attn_rope_table_scaled(max_pos, R, base, **kw)
    i = np.arange(R // 2, dtype=np.longdouble)
    theta = np.longdouble(base) ** (-2 * i / R)
    factor = np.longdouble(kw.get("factor", 1.0))
    keep = 0 * theta
    if kw.get("original_pos", 0):
        turns = kw["original_pos"] * theta / (2 * np.longdouble(np.pi))
        keep = np.clip((turns - kw["low"]) / (kw["high"] - kw["low"]), 0, 1)
    theta = theta * (keep + (1 - keep) / factor)
    angle = np.arange(max_pos, dtype=np.longdouble)[:, None] * theta
    amp = float(np.float32(kw.get("amplitude", 1.0)))
    want = np.stack([np.cos(angle), np.sin(angle)], -1) * amp
    # Half a step of fp32, and the angle in 64 bits: about 2^-51 of up to 2^18 radians here.
    err = np.abs(got.double().cpu().numpy() - want.astype(np.float64))
    assert float((err - 2.0 ** -24 * np.abs(want).astype(np.float64)).max()) <= amp * 2.0 ** -32
    if not kw:
        assert torch.equal(got, attn.attn_rope_table(max_pos, R, base))


# ================================================================== attention of new tokens
def pool(ctxs, news, ps, Hkv, D, seed=0, extra=3, spare_slots=1):
    """Scattered pages for requests of ctx + new keys, K and V, and the block table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = np.array(ctxs) + np.array(news)
    pages = -(-np.maximum(lens, 0) // ps)
    M = int(pages.max()) + spare_slots
    P = int(pages.sum()) + extra
    ids = rng.permutation(P)
    table = np.full((len(lens), M), -1)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    k, v = (torch.randn(P, Hkv, ps, D, generator=g, device="cuda", dtype=BF) for _ in range(2))
    return table, lens, k, v


def dense(table_row, kc, vc, n):
    """Keys [0, n) of a request: [n, Hkv, D]."""
    ps = kc.shape[2]
    t = torch.arange(n, device="cuda")
    page = torch.from_numpy(table_row).cuda()[t // ps]
    return kc[page, :, t % ps], vc[page, :, t % ps]


def reference(q, ctxs, news, table, kc, vc, window, sinks, scale):
    """O and LSE in 64 bits, and sum p |v| (the scale of O's error)."""
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    o = torch.zeros(T, Hq, D, dtype=F64, device="cuda")
    size = torch.zeros_like(o)
    lse = torch.full((T, Hq), -math.inf, dtype=F64, device="cuda")
    t0 = 0
    for b, (c, n) in enumerate(zip(ctxs, news)):
        L = max(c + n, 0)
        if n and L:
            k, v = (x.double() for x in dense(table[b], kc, vc, L))
            p = torch.arange(c, c + n, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None, :]
            seen = (j <= p) & ((j > p - window) | (j < sinks))
            unseen = ~seen.any(0)
            k, v = k.masked_fill(unseen[:, None, None], 0), v.masked_fill(unseen[:, None, None], 0)
            x = q[t0:t0 + n].double().view(n, Hkv, G, D)
            s = torch.einsum("nhgd,khd->hgnk", x, k) * scale
            s = s.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[..., None])
            o[t0:t0 + n] = torch.einsum("hgnk,khd->nhgd", w, v).reshape(n, Hq, D)
            size[t0:t0 + n] = torch.einsum("hgnk,khd->nhgd", w, v.abs()).reshape(n, Hq, D)
            lse[t0:t0 + n] = z.permute(2, 0, 1).reshape(n, Hq)
        t0 += n
    return o, lse, size


def check(got, ref, rows, off=None):
    """P is rounded to bf16 (half a step, 2^-8 of each weight) and O once more; scores are
    sums of D products in 32 bits, off by up to D * 2^-23 of the terms' sum, about 0.64 sqrt(D):
    2^-13 at D = 128 and 2^-11.6 at D = 256, which moves the LSE by as much and the weights by
    twice that (they are divided by their sum)."""
    (o, lse), (ro, rl, size) = got, ref
    assert o.dtype == BF and lse.dtype == torch.float32
    if off is None:
        off = 2.0 ** -12 if o.shape[-1] <= 128 else 2.0 ** -11
    o, lse, ro, rl, size = o[:rows].double(), lse[:rows].double(), ro[:rows], rl[:rows], size[:rows]
    err = (o - ro).abs() - 2.0 ** -8 * ro.abs() - (2.0 ** -8 + 2 * off) * size
    assert bool((err <= 0).all()), float(err.max())
    empty = rl == -math.inf
    assert bool((lse[empty] == -math.inf).all()) and bool((o[empty] == 0).all())
    assert float((lse - rl)[~empty].abs().max() if (~empty).any() else 0) <= off


def run_chunk(q, news, lens, table, kc, vc, window=None, sinks=0, scale=None, **kw):
    cu = np.concatenate([[0], np.cumsum(news)])
    cu, lens, table = gpu(cu, lens, table)
    Hkv, ps = kc.shape[1:3]
    plan = attn.attn_chunk_plan(cu, lens, q.shape[0], q.shape[1], Hkv, q.shape[2],
                                table.shape[1] * ps, window, sinks)
    return attn.attn_chunk_paged(q, kc, vc, table, plan, scale, **kw)


def case(ctxs, news, Hkv, G, D, ps, window=None, sinks=0, seed=0):
    table, lens, kc, vc = pool(ctxs, news, ps, Hkv, D, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(sum(news), Hkv * G, D, generator=g, device="cuda", dtype=BF)
    got = run_chunk(q, news, lens, table, kc, vc, window, sinks)
    status_ok()
    check(got, reference(q, ctxs, news, table, kc, vc, window or 1 << 30, sinks, 1 / math.sqrt(D)),
          sum(news))


CHUNK = [
    ([0], [1]), ([0], [2]), ([299], [1]), ([31], [1]), ([127], [1]), ([128], [1]), ([0], [31]),
    ([0], [32]), ([0], [33]), ([0], [64]), ([0], [65]), ([0], [300]), ([1000], [37]), ([96], [200]),
    ([3, 500, 0, 129], [1, 1, 40, 7]), ([0, 50, 0, 0], [5, 0, 0, 3]), ([2000] + [5] * 9, [1] * 10)]


@pytest.mark.gpu
@pytest.mark.parametrize("ctxs,news", CHUNK)
@pytest.mark.parametrize("Hkv,G,D,ps", [(2, 4, 128, 64), (1, 1, 64, 32), (2, 3, 64, 96),
                                        (1, 8, 128, 128), (3, 1, 128, 32), (2, 2, 256, 64),
                                        (1, 5, 256, 96), (1, 1, 256, 128)])
def test_chunk(ctxs, news, Hkv, G, D, ps):
    case(ctxs, news, Hkv, G, D, ps)


@pytest.mark.gpu
@pytest.mark.parametrize("G", [2, 5, 7, 16, 33, 64, 65, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_groups(G, D):
    # Rows of a tile are tokens x heads: heads that do not divide 128, and more than 128.
    case([0, 200, 70], [9, 1, 130], 2, G, D, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (20, 0), (20, 40), (128, 4), (129, 300),
                                          (1000, 128), (5000, 7)])
@pytest.mark.parametrize("D,ps", [(64, 32), (128, 64), (128, 96), (256, 64), (256, 32)])
def test_chunk_window(window, sinks, D, ps):
    case([0, 700, 1500, 333, 64], [150, 1, 90, 257, 64], 2, 4, D, ps, window, sinks)


@pytest.mark.gpu
def test_chunk_many_requests():
    # More items than parts, and parts that begin anywhere: every request's work is cut
    # somewhere in some of these.
    rng = np.random.default_rng(5)
    for _ in range(4):
        B = 200
        ctxs = rng.integers(0, 1500, B).tolist()
        news = np.where(rng.random(B) < 0.1, rng.integers(0, 200, B), 1).tolist()
        case(ctxs, news, 2, 4, 64, 32, seed=int(rng.integers(1000)))


@pytest.mark.gpu
@pytest.mark.parametrize("news", [[1], [500], [128], [70]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_long_cache(news, D):
    # One request over all the CTAs: many partial results of an item.
    case([40000], news, 1, 4, D, 64)


@pytest.mark.gpu
def test_chunk_more_tokens_than_keys():
    # Tokens before the first key (lengths shorter than the new tokens) see nothing.
    news = [10, 40, 3, 200]
    lens = [4, 0, -7, 130]
    ctxs = [max(x, 0) - n for x, n in zip(lens, news)]
    table, _, kc, vc = pool([0] * 4, [200] * 4, 32, 2, 64)
    q = torch.randn(sum(news), 8, 64, device="cuda", dtype=BF)
    got = run_chunk(q, news, lens, table, kc, vc)
    status_ok()
    ref = reference(q, ctxs, news, table, kc, vc, 1 << 30, 0, 0.125)
    assert bool((ref[1] == -math.inf).any())
    check(got, ref, sum(news))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), (100, 5), (300, 0)])
def test_chunk_unseen_memory_may_hold_anything(D, fill, window, sinks):
    ctxs, news, ps, Hkv = [900, 0, 431], [30, 77, 1], 64, 2
    table, lens, kc, vc = pool(ctxs, news, ps, Hkv, D)
    q = torch.randn(sum(news), 8, D, device="cuda", dtype=BF)
    ref = reference(q, ctxs, news, table, kc, vc, window, sinks, 1 / math.sqrt(D))
    seen = torch.zeros(kc.shape[0], ps, dtype=torch.bool)
    cut = table.copy()
    for b, (c, n) in enumerate(zip(ctxs, news)):
        for j in range(c + n):
            if j >= c - window + 1 or j < sinks:
                seen[table[b, j // ps], j % ps] = True
        for s in range(table.shape[1]):  # pages without a seen key are gone
            lo, hi = s * ps, min((s + 1) * ps, c + n)
            if not any(j >= c - window + 1 or j < sinks for j in range(lo, hi)):
                cut[b, s] = [-1, 1 << 30, -77][s % 3]
    for x in (kc, vc):
        x.masked_fill_(~seen.cuda()[:, None, :, None], fill)
    got = run_chunk(q, news, lens, cut, kc, vc, window, sinks)
    status_ok()
    check(got, ref, sum(news))


@pytest.mark.gpu
def test_chunk_tokens_behind_the_last_request():
    ctxs, news = [100, 3], [5, 1]
    table, lens, kc, vc = pool(ctxs, news, 32, 1, 64)
    q = torch.randn(50, 4, 64, device="cuda", dtype=BF)
    o = torch.full((50, 4, 64), 7.0, device="cuda", dtype=BF)
    lse = torch.full((50, 4), 7.0, device="cuda")
    got = run_chunk(q, news, lens, table, kc, vc, o=o, lse=lse)
    assert got[0].data_ptr() == o.data_ptr()
    check(got, reference(q, ctxs, news, table, kc, vc, 1 << 30, 0, 0.125), 6)
    assert bool((o[6:] == 7).all()) and bool((lse[6:] == 7).all())
    status_ok()


@pytest.mark.gpu
def test_chunk_extreme_scores():
    # Large scores: one key takes the whole weight, and the running maximum moves.
    ctxs, news = [600, 130], [1, 70]
    table, lens, kc, vc = pool(ctxs, news, 32, 2, 64)
    q = torch.randn(71, 8, 64, device="cuda", dtype=BF) * 30
    kc *= 20
    got = run_chunk(q, news, lens, table, kc, vc, scale=1.0)
    ref = reference(q, ctxs, news, table, kc, vc, 1 << 30, 0, 1.0)
    # Scores of about 2e4 are off by 2^-16 of their terms' sum: up to 0.5 for D = 64; rows
    # whose best key is not clearly the best are left out.
    o, lse = got
    assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse).all())
    assert float(((lse.double() - ref[1]) / ref[1].abs()).abs().max()) <= 2.0 ** -15
    status_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("climb", [True, False])
def test_chunk_moving_maximum(D, climb):
    # Scores that climb with the keys, or jump, by more than 8 in base 2 from tile to tile, at
    # other places in each row.  (Their terms add up to 155, the noise's to less than 25: off by
    # D * 2^-23 of that.)
    ctxs, news = [1000, 700, 2000], [60, 1, 13]
    table, lens, kc, vc = pool(ctxs, news, 64, 2, D)
    g = torch.Generator(device="cuda").manual_seed(D)
    u = torch.sign(torch.randn(D, generator=g, device="cuda"))
    steps = torch.arange(64, device="cuda") * 5.0 if climb else \
        torch.rand(64, generator=g, device="cuda") * 150
    for b, (c, n) in enumerate(zip(ctxs, news)):
        for slot in range(-(-(c + n) // 64)):
            page = int(table[b, slot])
            kc[page] = (kc[page].float() * 0.1 + steps[slot] / D * u).to(BF)
    gain = torch.rand(sum(news), 8, 1, generator=g, device="cuda")
    q = (gain * u + 0.1 * torch.randn(sum(news), 8, D, generator=g, device="cuda")).to(BF)
    got = run_chunk(q, news, lens, table, kc, vc, scale=1.0)
    status_ok()
    check(got, reference(q, ctxs, news, table, kc, vc, 1 << 30, 0, 1.0), sum(news),
          off=D * 2.0 ** -23 * 180)


@pytest.mark.gpu
def test_chunk_bad_page_is_reported():
    table, lens, kc, vc = pool([100], [1], 32, 1, 64)
    q = torch.randn(1, 4, 64, device="cuda", dtype=BF)
    for bad in (-1, kc.shape[0], 1 << 30, -(1 << 31)):
        t = table.copy()
        t[0, 1] = bad
        o, _ = run_chunk(q, [1], lens, t, kc, vc)
        assert attn.attn_debug_status() == INV
        t[0, 1] = 0
        assert torch.equal(o, run_chunk(q, [1], lens, t, kc, vc)[0])
        status_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [-1, 2, 4, 8], [0, 4, 9, 8], [0, 1, 2, 9], [7, 0, 8, 8]])
def test_chunk_bad_bounds_are_reported(cu):
    table, lens, kc, vc = pool([50] * 3, [3] * 3, 32, 1, 64)
    q = torch.randn(8, 4, 64, device="cuda", dtype=BF)
    cu, lens, table = gpu(cu, lens, table)
    plan = attn.attn_chunk_plan(cu, lens, 8, 4, 1, 64, table.shape[1] * 32)
    assert attn.attn_debug_status() == INV
    attn.attn_chunk_paged(q, kc, vc, table, plan)
    status_ok()


@pytest.mark.gpu
def test_chunk_overlapping_requests_stay_in_the_plan():
    # Every request claims all tokens, again and again: more items than a plan holds.
    T, B = 600, 64
    cu = gpu(np.array([0, T] * (B // 2) + [0]))
    lens = gpu(np.full(B, 700))
    guard = torch.full((1 << 20,), 77, dtype=torch.int32, device="cuda")
    import ctypes
    n = ctypes.c_longlong()
    assert attn.load_library().attn_chunk_plan_size(B, T, 8, 2, 64, ctypes.byref(n)) == 0
    attn.attn_chunk_plan(cu, lens, T, 8, 2, 64, 1024, plan=guard)
    assert attn.attn_debug_status() == INV
    assert bool((guard[n.value:] == 77).all())


@pytest.mark.gpu
def test_chunk_refuses_a_plan_of_other_sizes():
    table, lens, kc, vc = pool([100], [4], 32, 1, 64)
    q = torch.randn(4, 4, 64, device="cuda", dtype=BF)
    cu, lens, table = gpu(np.array([0, 4]), lens, table)
    keys = table.shape[1] * 32
    o, lse = torch.full_like(q, 7.0), torch.full((4, 4), 7.0, device="cuda")
    for other in [(5, 4, 1, 64, keys), (4, 2, 1, 64, keys), (4, 4, 2, 64, keys), (4, 4, 1, 128, keys),
                  (4, 4, 1, 64, keys + 32)]:
        plan = attn.attn_chunk_plan(cu, lens, *other, plan=torch.zeros(100000, dtype=torch.int32,
                                                                      device="cuda"))
        status_ok()
        attn.attn_chunk_paged(q, kc, vc, table, plan, o=o, lse=lse)
        assert attn.attn_debug_status() == INV
    attn.attn_chunk_paged(q, kc, vc, table, torch.zeros_like(plan), o=o, lse=lse)
    assert attn.attn_debug_status() == INV
    assert bool((o == 7).all()) and bool((lse == 7).all())
    for bad in (plan[:20], plan.long(), plan.view(-1, 2)):
        with pytest.raises(ValueError):
            attn.attn_chunk_paged(q, kc, vc, table, bad)
    with pytest.raises(attn.AttnError):
        attn.attn_chunk_paged(q, kc, vc, table, plan[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_output_off_32_bytes(D):
    # Whole and cut items, to an output that is aligned to 16 bytes alone.
    ctxs, news = [9000, 12, 900, 40], [60, 100, 1, 1]
    table, lens, kc, vc = pool(ctxs, news, 64, 2, D)
    q = torch.randn(sum(news), 6, D, device="cuda", dtype=BF)
    want = run_chunk(q, news, lens, table, kc, vc)
    buf = torch.full((q.numel() + 16,), 7.0, dtype=BF, device="cuda")
    assert buf.data_ptr() % 32 == 0
    o = buf[8:8 + q.numel()].view_as(q)
    got = run_chunk(q, news, lens, table, kc, vc, o=o)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((buf[:8] == 7).all()) and bool((buf[-8:] == 7).all())
    status_ok()


@pytest.mark.gpu
def test_chunk_same_bits_each_time():
    ctxs, news = [5000, 12, 900], [60, 100, 1]
    table, lens, kc, vc = pool(ctxs, news, 64, 2, 128)
    q = torch.randn(sum(news), 8, 128, device="cuda", dtype=BF)
    first = run_chunk(q, news, lens, table, kc, vc)
    for _ in range(20):
        again = run_chunk(q, news, lens, table, kc, vc)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
def test_chunk_same_bits_of_long_items():
    # Twice as many items as CTAs, of more than 2^10 K/V tiles, a few of them four tiles longer:
    # whether two of those meet in a CTA may not decide how the work is cut.
    B, ps = 2 * torch.cuda.get_device_properties(0).multi_processor_count, 128
    M = 1100
    kc, vc = (torch.randn(M, 1, ps, 64, device="cuda", dtype=BF) for _ in range(2))
    table = gpu(np.tile(np.arange(M), (B, 1)))  # one cache for all
    lens = np.full(B, 1040 * ps)
    lens[np.random.default_rng(0).permutation(B)[:18]] += 4 * ps
    q = torch.randn(B, 1, 64, device="cuda", dtype=BF)
    cu, lens = gpu(np.arange(B + 1), lens)
    first = None
    for _ in range(12):
        plan = attn.attn_chunk_plan(cu, lens, B, 1, 1, 64, M * ps)
        got = attn.attn_chunk_paged(q, kc, vc, table, plan)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    status_ok()


@pytest.mark.gpu
def test_chunk_two_streams_and_shared_plan():
    # One plan, two layers at once on streams of their own.
    ctxs, news = [3000, 700], [50, 1]
    table, lens, k0, v0 = pool(ctxs, news, 64, 2, 64)
    k1, v1 = torch.randn_like(k0), torch.randn_like(v0)
    q = torch.randn(51, 8, 64, device="cuda", dtype=BF)
    cu, lens, tab = gpu(np.array([0, 50, 51]), lens, table)
    plan = attn.attn_chunk_plan(cu, lens, 51, 8, 2, 64, tab.shape[1] * 64)
    want = [attn.attn_chunk_paged(q, k, v, tab, plan) for k, v in ((k0, v0), (k1, v1))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [attn.attn_chunk_paged(q, k, v, tab, plan, stream=s)
               for s, (k, v) in zip(streams, ((k0, v0), (k1, v1)))]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    status_ok()


@pytest.mark.gpu
def test_chunk_offsets_past_32_bits():
    # A cache of 2^31 elements and more each for K and V: pages at its far end.
    Hkv, ps, D = 8, 64, 128
    P = (1 << 31) // (Hkv * ps * D) + 40
    kc = torch.zeros(P, Hkv, ps, D, device="cuda", dtype=BF)
    vc = torch.zeros(P, Hkv, ps, D, device="cuda", dtype=BF)
    ctxs, news = [900, 5], [40, 1]
    table = np.arange(P - 32, P).reshape(2, 16)[:, ::-1].copy()
    kc[P - 32:].normal_()
    vc[P - 32:].normal_()
    q = torch.randn(41, 32, D, device="cuda", dtype=BF)
    got = run_chunk(q, news, [940, 6], table, kc, vc)
    check(got, reference(q, ctxs, news, table, kc, vc, 1 << 30, 0, 1 / math.sqrt(D)), 41)
    # ... and written there.
    qkv = torch.randn(2, (32 + 16) * D, device="cuda", dtype=BF)
    rope = attn.attn_rope_table(8, D)
    slots = gpu(np.array([(P - 1) * ps + 63, (P - 1) * ps]))
    attn.attn_rope_append(qkv, rope, gpu(np.zeros(2)), slots, kc, vc, 32)
    rows = qkv.view(2, 48, D)
    assert torch.equal(kc[P - 1, :, [63, 0]].transpose(0, 1), rows[:, 32:40])
    assert torch.equal(vc[P - 1, :, [63, 0]].transpose(0, 1), rows[:, 40:])
    status_ok()


# ================================================================== together
@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(None, 0), (150, 4)])
@pytest.mark.parametrize("D,R,style", [(64, 32, 0), (128, 128, 1), (256, 64, 1)])
def test_serving_steps(window, sinks, D, R, style):
    """Prompts in chunks and generated tokens side by side, two layers, over pages that the
    window gives up: each step's attention against the whole history in 64 bits."""
    Hq, Hkv, ps, B, M, P = 8, 2, 32, 4, 24, 60
    g = torch.Generator(device="cuda").manual_seed(7)
    rope = attn.attn_rope_table_scaled(M * ps, R, 10000.0, 4.0, 1.0, 8.0, 200)
    table, refs, lens = gpu(np.full((B, M), -1), np.zeros(P), np.zeros(B))
    caches = [[torch.full((P, Hkv, ps, D), float("nan"), dtype=BF, device="cuda") for _ in range(2)]
              for _ in range(2)]
    history = [[[] for _ in range(B)] for _ in range(2)]  # layer, request: rotated k and v rows
    plans = [[100, 1, 0, 33], [100, 1, 64, 1], [37, 1, 64, 1], [1, 1, 1, 1], [1, 1, 130, 1], [1, 1, 1, 1]]
    length = [0] * B
    for new in plans:
        T = sum(new) + 3
        table, refs, lens, cu, pos, slots, counts = attn.attn_pages_append(
            table, refs, lens, gpu(np.array(new)), T, ps)
        plan = attn.attn_chunk_plan(cu, lens, T, Hq, Hkv, D, M * ps, window, sinks)
        for layer in range(2):
            qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda", dtype=BF)
            kc, vc = caches[layer]
            q = attn.attn_rope_append(qkv, rope, pos, slots, kc, vc, Hq, style=style)
            got = attn.attn_chunk_paged(q, kc, vc, table, plan)
            status_ok()
            x = qkv.double().cpu().view(T, -1, D)
            t0 = 0
            for b, n in enumerate(new):
                cs = rope.double().cpu()[length[b]:length[b] + n]
                k = turn(x[t0:t0 + n, Hq:Hq + Hkv], cs, style)
                near(q[t0:t0 + n], turn(x[t0:t0 + n, :Hq], cs, style), 8)
                # What the cache holds: rounded.
                history[layer][b].append((k.to(BF), x[t0:t0 + n, Hq + Hkv:].to(BF)))
                t0 += n
            kd = [torch.cat([h[0] for h in row]) for row in history[layer]]
            vd = [torch.cat([h[1] for h in row]) for row in history[layer]]
            # The same attention over contiguous pages of the history.
            n_pages = [-(-k.shape[0] // ps) + 1 for k in kd]
            flat = [torch.zeros(sum(n_pages), Hkv, ps, D, dtype=BF, device="cuda") for _ in range(2)]
            tab, at = np.zeros((B, max(n_pages)), dtype=np.int64), 0
            for b in range(B):
                tab[b, :n_pages[b]] = np.arange(at, at + n_pages[b])
                for dst, src in zip(flat, (kd[b], vd[b])):
                    pad = torch.zeros(n_pages[b] * ps, Hkv, D, dtype=BF)
                    pad[:src.shape[0]] = src
                    dst[at:at + n_pages[b]] = pad.view(-1, ps, Hkv, D).transpose(1, 2).cuda()
                at += n_pages[b]
            ref = reference(q, length, new, tab, *flat, window or 1 << 30, sinks, 1 / math.sqrt(D))
            check(got, ref, sum(new))
        length = [a + n for a, n in zip(length, new)]
        assert lens.tolist() == length
        if window is not None:
            table, refs = attn.attn_pages_free(table, refs, lens, ps, window, sinks)
    # Single tokens: the decode that the library had gives the same.
    q1 = torch.randn(B, Hq, 1, D, generator=g, device="cuda", dtype=BF)
    plan = attn.attn_chunk_plan(gpu(np.arange(B + 1)), lens, B, Hq, Hkv, D, M * ps, window, sinks)
    o, lse = attn.attn_chunk_paged(q1.view(B, Hq, D), *caches[0], table, plan)
    od, ld = attn.decode_window_paged(q1, *caches[0], table, lens, window or 1 << 30, sinks)
    assert float((lse - ld).abs().max()) <= 2.0 ** -11
    # Each rounds its weights and its result once (2^-8 each, of values up to about 4).
    assert float((o.float() - od.float()).abs().max()) <= 4 * 4 * 2.0 ** -8
    status_ok()


@pytest.mark.gpu
def test_steps_of_forked_rows():
    """Three samples of one prompt: forked with its pages shared, then tokens of their own, with
    and without pages that the fork reserved."""
    Hq, Hkv, D, ps, M, P, n = 4, 2, 64, 32, 8, 40, 70
    rope = attn.attn_rope_table(M * ps, D)
    kc, vc = (torch.full((P, Hkv, ps, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(3)

    def step(table, refs, lens, news):
        T = sum(news)
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda", dtype=BF)
        length = lens.tolist()
        table, refs, lens, cu, pos, slots, _ = attn.attn_pages_append(
            table, refs, lens, gpu(np.array(news)), T, ps)
        plan = attn.attn_chunk_plan(cu, lens, T, Hq, Hkv, D, M * ps)
        q = attn.attn_rope_append(qkv, rope, pos, slots, kc, vc, Hq)
        got = attn.attn_chunk_paged(q, kc, vc, table, plan)
        status_ok()
        tab = table.cpu().numpy().astype(np.int64)
        check(got, reference(q, length, news, tab, kc, vc, 1 << 30, 0, 0.125), T)
        return table, refs, lens

    table, refs, lens = step(*gpu(np.full((1, M), -1), np.zeros(P), np.zeros(1)), [n])
    kept = kc[table[0, :2].long()].clone()
    for room in (0, 40):
        t, r, ln, src, dst, _ = attn.attn_pages_fork(table, refs, lens, gpu(np.zeros(3)), ps, room=room)
        attn.attn_pages_copy(kc, vc, src, dst)
        for news in ([1, 1, 1], [5, 0, 60], [1, 90, 1]):
            t, r, ln = step(t, r, ln, news)
        tab = t.cpu().numpy()
        assert (tab[:, :2] == tab[0, 0:2]).all()  # full pages of the prompt: shared
        own = tab[:, 2:][tab[:, 2:] >= 0]
        assert len(set(own.tolist())) == own.size
        np.testing.assert_array_equal(
            r.cpu().numpy(), np.bincount(tab[tab >= 0], minlength=P))
    assert torch.equal(kc[table[0, :2].long()], kept)


@pytest.mark.gpu
def test_step_in_a_graph():
    """A whole step captured once and replayed with other lengths."""
    Hq, Hkv, D, ps, B, M, P, T = 8, 2, 64, 32, 3, 20, 64, 40
    rope = attn.attn_rope_table(M * ps, D)
    table, refs, lens = gpu(np.full((B, M), -1), np.zeros(P), np.zeros(B))
    new = gpu(np.zeros(B))
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda", dtype=BF)
    kc, vc = (torch.zeros(P, Hkv, ps, D, dtype=BF, device="cuda") for _ in range(2))
    o = torch.zeros(T, Hq, D, dtype=BF, device="cuda")
    lse = torch.zeros(T, Hq, device="cuda")

    def step():
        _, _, _, cu, pos, slots, _ = attn.attn_pages_append(
            table, refs, lens, new, T, ps, block_table_out=table, refs_out=refs, seqlens_out=lens)
        plan = attn.attn_chunk_plan(cu, lens, T, Hq, Hkv, D, M * ps)
        q = attn.attn_rope_append(qkv, rope, pos, slots, kc, vc, Hq)
        attn.attn_chunk_paged(q, kc, vc, table, plan, o=o, lse=lse)
        return q

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()  # no tokens: nothing changes
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            q = step()
    torch.cuda.synchronize()
    length = [0] * B
    for news in ([20, 5, 0], [1, 30, 9], [1, 1, 1], [0, 0, 0], [40, 0, 0], [2, 1, 30]):
        qkv.normal_()
        new.copy_(gpu(np.array(news)))
        o.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        status_ok()
        ref = reference(q, length, news, table.cpu().numpy().astype(np.int64), kc, vc, 1 << 30, 0, 0.125)
        check((o, lse), ref, sum(news))
        assert bool((o[sum(news):] == 7).all())
        length = [a + n for a, n in zip(length, news)]
        assert lens.tolist() == length
