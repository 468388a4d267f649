"""Attention with a sliding window and sinks: attn_window_fwd, attn_window_bwd,
decode_window and decode_window_paged against the formula in 64 bits.

Bounds, element by element, from the roundings that the kernels make (u = 2^-8,
half a bf16 step relative to the value; fp32 sums of the products add less than
w = 2^-12 relative to the sum of magnitudes at these sizes):
  O     P is rounded to bf16 for the second product, O once at the end:
        u |O| + (u + w) sum_j P |V|
  LSE   scores are fp32 sums of D products, each within 2^-24 of the running sum of
        magnitudes: (D + 8) 2^-24 max_j scale sum_d |q k| + 2^-18
  dV    u |dV| + (u + w) sum_i P |dO|
  dS    dS is rounded to bf16; Delta reads the rounded O:
        e_dS = (u + w) |dS| + P (sum_d |dO| e_O + w sum_d |dO| |V|)
  dQ    u |dQ| + scale sum_j e_dS |K| + w scale sum_j |dS| |K|; dK alike
"""
import ctypes
import itertools
import math
import threading

import pytest
import torch

import tensor_attn_fwd_gb300 as attn

U, W = 2.0 ** -8, 2.0 ** -12
NEG = float("-inf")


def visible(Sq, Sk, window, sinks):
    p = torch.arange(Sq)[:, None] + Sk - Sq
    j = torch.arange(Sk)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def reference(q, k, v, window, sinks, scale, do=None):
    """The outputs in 64 bits and their bounds: dicts of tensors."""
    q, k, v = (t.double().cpu() for t in (q, k, v))
    B, Hq, Sq, D = q.shape
    Hkv, Sk = k.shape[1:3]
    n = Hq // Hkv
    kx, vx = (t.repeat_interleave(n, 1) for t in (k, v))
    seen = visible(Sq, Sk, window, sinks)
    x = (q @ kx.transpose(-1, -2)) * scale
    x = x.masked_fill(~seen, NEG)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse.masked_fill(lse == NEG, 0.0)[..., None]).masked_fill(~seen, 0.0)
    o = p @ vx
    mag = (q.abs() @ kx.abs().transpose(-1, -2)).masked_fill(~seen, 0.0).amax(-1) * scale
    ref = {"o": o, "lse": lse}
    tol = {"o": U * o.abs() + (U + W) * (p @ vx.abs()), "lse": (D + 8) * 2.0 ** -24 * mag + 2.0 ** -18}
    if do is not None:
        do = do.double().cpu()

        def shared(t):  # the sum over the query heads of a KV head
            return t.view(B, Hkv, n, Sk, D).sum(2)

        pt = p.transpose(-1, -2)
        ds = p * (do @ vx.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        e_ds = (U + W) * ds.abs() + p * ((do.abs() * tol["o"]).sum(-1, keepdim=True)
                                         + W * (do.abs() @ vx.abs().transpose(-1, -2)))
        both = e_ds + W * ds.abs()
        ref["dv"] = shared(pt @ do)
        ref["dq"] = scale * (ds @ kx)
        ref["dk"] = scale * shared(ds.transpose(-1, -2) @ q)
        tol["dv"] = U * ref["dv"].abs() + (U + W) * shared(pt @ do.abs())
        tol["dq"] = U * ref["dq"].abs() + scale * (both @ kx.abs())
        tol["dk"] = U * ref["dk"].abs() + scale * shared(both.transpose(-1, -2) @ q.abs())
    return ref, tol


def check(name, got, ref, tol):
    got = got.double().cpu()
    assert got.shape == ref.shape, name
    empty = ref == NEG
    assert torch.equal(got == NEG, empty), f"{name}: rows without keys"
    err = torch.where(empty, 0.0, got - ref.masked_fill(empty, 0.0)).abs()
    assert bool(torch.isfinite(err).all()), f"{name}: not finite"
    over = (err - tol - 1e-30).max().item()
    assert over <= 0, f"{name}: {over:.3e} over the bound (worst error {err.max().item():.3e})"


def inputs(B, Hq, Hkv, Sq, Sk, D, seed, grad=False):
    g = torch.Generator().manual_seed(seed)
    shapes = [(B, Hq, Sq, D), (B, Hkv, Sk, D), (B, Hkv, Sk, D)] + ([(B, Hq, Sq, D)] if grad else [])
    return [torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in shapes]


# B, Hq, Hkv, Sq, Sk, D, window, sinks
SHAPES = [
    (1, 1, 1, 1, 1, 64, 1, 0),              # one row, one key
    (1, 2, 1, 1, 1, 128, 5, 3),             # a window and sinks longer than the sequence
    (1, 2, 1, 1, 1000, 128, 999, 0),        # one row of a long cache
    (2, 4, 2, 129, 129, 64, 1, 0),          # a row sees itself alone
    (1, 4, 4, 128, 128, 64, 32, 1),         # one tile
    (1, 2, 2, 300, 300, 128, 128, 0),       # row pairs, window of one tile
    (1, 4, 1, 257, 257, 64, 100, 130),      # sinks past the first tile
    (1, 3, 1, 500, 500, 128, 70, 4),        # an odd group: row pairs
    (1, 2, 1, 700, 700, 64, 129, 200),
    (1, 1, 1, 900, 900, 64, 130, 129),      # a gap in the tiles of a row pair
    (1, 5, 1, 1030, 1030, 128, 1, 1),       # far apart: one sink, one key
    (2, 2, 2, 100, 700, 64, 300, 7),        # a chunk against a longer cache
    (1, 4, 2, 300, 129, 128, 40, 3),        # rows before the first key
    (1, 2, 2, 300, 100, 64, 10, 0),         # whole tiles of such rows, row pairs
    (1, 2, 2, 200, 200, 64, 10000, 0),      # the window covers everything
    (1, 2, 2, 200, 200, 64, 2, 10000),      # the sinks do
    (1, 2, 2, 640, 640, 64, 128, 128),      # everything on tile borders
    (1, 6, 2, 1100, 1100, 128, 257, 513),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward_match_the_formula(shape):
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    q, k, v, do = inputs(B, Hq, Hkv, Sq, Sk, D, 11 * Sq + Sk + window, grad=True)
    scale = 1.0 / math.sqrt(D)
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks)
    grads = attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
    assert attn.attn_debug_status() == attn.ATTN_OK
    ref, tol = reference(q, k, v, window, sinks, scale, do)
    check("o", o, ref["o"], tol["o"])
    check("lse", lse, ref["lse"], tol["lse"])
    for name, got in zip(("dq", "dk", "dv"), grads):
        check(name, got, ref[name], tol[name])


# The same shapes at the head dimension that has a kernel of its own (no backward).
SHAPES_256 = [s[:5] + (256,) + s[6:] for s in SHAPES[:17]]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES_256 + [(1, 2, 1, 40, 3000, 256, 1500, 300)])
@pytest.mark.parametrize("splits", [1, 2, 5, None])
def test_forward_of_head_dimension_256(shape, splits):
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    splits = splits if splits is None else min(splits, -(-Sk // 128))
    q, k, v = inputs(B, Hq, Hkv, Sq, Sk, D, Sq + 5 * Sk)
    want, tol = reference(q, k, v, window, sinks, 1.0 / math.sqrt(D))
    unseen = ~visible(Sq, Sk, window, sinks).any(0)
    k[:, :, unseen.cuda()] = float("nan")
    v[:, :, unseen.cuda()] = float("inf")
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=splits)
    assert attn.attn_debug_status() == attn.ATTN_OK
    check("o", o, want["o"], tol["o"])
    check("lse", lse, want["lse"], tol["lse"])


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Sk,D", [(2, 4, 2, 333, 333, 128), (1, 3, 3, 200, 700, 64),
                                              (1, 2, 1, 300, 129, 64), (1, 4, 2, 300, 500, 256)])
def test_a_window_over_everything_is_the_causal_forward(B, Hq, Hkv, Sq, Sk, D):
    q, k, v = inputs(B, Hq, Hkv, Sq, Sk, D, 5)
    want = attn.attn_fwd_bf16o(q, k, v, causal=True)
    for window, sinks in ((Sk, 0), (2 ** 31 + 5, 0), (1, Sk), (7, 2 ** 40)):
        got = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=1)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES + [(1, 4, 2, 40, 3000, 64, 1500, 300)])
@pytest.mark.parametrize("splits", [2, 3, 7, None])
def test_forward_in_splits(shape, splits):
    # Also splits without a tile, splits of sinks alone, and row pairs whose tiles' runs differ.
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    if splits is not None and splits > -(-Sk // 128):
        pytest.skip("more splits than key tiles")
    q, k, v = inputs(B, Hq, Hkv, Sq, Sk, D, Sq + 3 * Sk)
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=splits)
    assert attn.attn_debug_status() == attn.ATTN_OK
    ref, tol = reference(q, k, v, window, sinks, 1.0 / math.sqrt(D))
    check("o", o, ref["o"], tol["o"])
    check("lse", lse, ref["lse"], tol["lse"])


@pytest.mark.gpu
def test_gradients_are_the_differences_of_the_forward():
    # Directional differences of L = sum(dO O) in 64 bits along random directions.
    B, Hq, Hkv, S, D, window, sinks = 1, 4, 2, 90, 64, 17, 3
    q, k, v, do = inputs(B, Hq, Hkv, S, S, D, 3, grad=True)
    scale = 1.0 / math.sqrt(D)
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks)
    grads = attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
    _, tol = reference(q, k, v, window, sinks, scale, do)
    h = 1e-4
    g = torch.Generator().manual_seed(1)
    for i, name in enumerate(("dq", "dk", "dv")):
        base = [t.double().cpu() for t in (q, k, v)]
        d = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        loss = []
        for sign in (1, -1):
            at = list(base)
            at[i] = base[i] + sign * h * d
            loss.append((reference(*at, window, sinks, scale)[0]["o"] * do.double().cpu()).sum())
        diff = ((loss[0] - loss[1]) / (2 * h)).item()
        got = (grads[i].double().cpu() * d).sum().item()
        # The gradient's bound along d, and the difference's own h^2 term.
        assert abs(got - diff) <= (tol[name] * d.abs()).sum().item() + 1e-4 * abs(diff), name


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 8, 1, 1300, 1300, 128, 60, 5), (2, 2, 1, 900, 1000, 64, 1, 257),
                                   (1, 4, 4, 2000, 2000, 64, 129, 128)])
def test_sink_tiles_whose_rows_are_split(shape):
    # Sequences long against their window: the tiles with sinks are cut into parts.
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    q, k, v, do = inputs(B, Hq, Hkv, Sq, Sk, D, Sq, grad=True)
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks)
    ref, tol = reference(q, k, v, window, sinks, 1.0 / math.sqrt(D), do)
    grads = attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
    assert attn.attn_debug_status() == attn.ATTN_OK
    for name, got in zip(("dq", "dk", "dv"), grads):
        check(name, got, ref[name], tol[name])
    n = ctypes.c_longlong(0)
    assert _lib().attn_window_bwd_workspace(*shape, ctypes.byref(n)) == attn.ATTN_OK
    assert n.value > B * Hq * Sq  # Delta, and partial sums
    # A workspace of the caller's: only its own floats are written, whatever they held.
    ws = torch.full((n.value + 4096,), float("nan"), device="cuda")
    again = attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks, workspace=ws)
    assert bool(torch.isnan(ws[n.value:]).all())
    for a, b in zip(grads, again):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks, workspace=ws[: n.value - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 4, 2, 70, 1024, 128, 100, 5), (2, 2, 2, 300, 900, 64, 130, 128),
                                   (1, 3, 1, 40, 700, 128, 1, 0), (1, 2, 1, 1, 300, 64, 37, 200),
                                   (1, 2, 1, 129, 2000, 64, 500, 300)])
@pytest.mark.parametrize("splits", [1, 2])
def test_keys_that_no_row_sees_may_be_anything(shape, splits):
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    q, k, v, do = inputs(B, Hq, Hkv, Sq, Sk, D, 8, grad=True)
    want = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=splits)
    gwant = attn.attn_window_bwd(q, k, v, *want, do, window, sinks)
    unseen = ~visible(Sq, Sk, window, sinks).any(0)
    assert bool(unseen.any())
    k2, v2 = k.clone(), v.clone()
    k2[:, :, unseen.cuda()] = float("nan")
    v2[:, :, unseen.cuda()] = float("-inf")
    got = attn.attn_window_fwd(q, k2, v2, window, sinks, num_splits=splits)
    ggot = attn.attn_window_bwd(q, k2, v2, *got, do, window, sinks)
    assert attn.attn_debug_status() == attn.ATTN_OK
    for a, b in zip(got + ggot, want + gwant):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_outputs_rows_behind_the_tensor_stay():
    B, Hq, Hkv, S, D, window, sinks = 1, 2, 1, 201, 64, 33, 2
    q, k, v, do = inputs(B, Hq, Hkv, S, S, D, 9, grad=True)

    def guarded(shape, dtype):
        n = math.prod(shape)
        buf = torch.full((n + 4096,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[:n].view(shape)

    ob, o = guarded(q.shape, torch.bfloat16)
    lb, lse = guarded(q.shape[:3], torch.float32)
    attn.attn_window_fwd(q, k, v, window, sinks, o=o, lse=lse)
    gs = [guarded(t.shape, torch.bfloat16) for t in (q, k, v)]
    attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks, dq=gs[0][1], dk=gs[1][1], dv=gs[2][1])
    for buf, view in [(ob, o), (lb, lse)] + gs:
        assert bool((buf[view.numel():] == 7.0).all())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    # q, o, dout and dq of 2.2e9 elements: the last rows of the last head against the same
    # rows computed as a chunk of their own (each within the bounds: twice them apart).
    B, Hq, Hkv, S, D, window, sinks = 1, 32, 1, 530000, 128, 100, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    q, do = (torch.randn(B, Hq, S, D, generator=g, device="cuda", dtype=torch.bfloat16)
             for _ in range(2))
    k, v = (torch.randn(B, Hkv, S, D, generator=g, device="cuda", dtype=torch.bfloat16)
            for _ in range(2))
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks)
    dq, dk, dv = attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
    assert attn.attn_debug_status() == attn.ATTN_OK
    n = 300  # rows; their keys: the sinks, and the last n + window
    seen = torch.cat([torch.arange(sinks), torch.arange(S - n - window, S)]).cuda()
    kt, vt = k[:, :, seen], v[:, :, seen]
    rows = [t[:, -1:, -n:].contiguous() for t in (q, do)]
    ref, tol = reference(rows[0], kt, vt, window, sinks, 1.0 / math.sqrt(D), rows[1])
    check("o", o[:, -1:, -n:], ref["o"], tol["o"])
    check("lse", lse[:, -1:, -n:], ref["lse"], tol["lse"])
    check("dq", dq[:, -1:, -n:], ref["dq"], tol["dq"])
    # The last key's gradients come from the last row of every head.
    ref, tol = reference(q[:, :, -1:], kt, vt, window, sinks, 1.0 / math.sqrt(D), do[:, :, -1:])
    check("dk", dk[:, :, -1], ref["dk"][:, :, -1], tol["dk"][:, :, -1])
    check("dv", dv[:, :, -1], ref["dv"][:, :, -1], tol["dv"][:, :, -1])


# ------------------------------------------------------------------ decode
def paged(k, v, page, seed, spare=3):
    """A paged copy of contiguous caches: (k_cache, v_cache, table), pages shuffled."""
    B, Hkv, Sk, D = k.shape
    M = -(-Sk // page)
    P = B * M + spare
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(P, generator=g)[: B * M].view(B, M)
    out = []
    for t in (k, v):
        pad = torch.zeros(B, Hkv, M * page, D, dtype=t.dtype, device=t.device)
        pad[:, :, :Sk] = t
        cache = torch.full((P, Hkv, page, D), float("nan"), dtype=t.dtype, device=t.device)
        cache[ids.view(-1).cuda()] = (pad.view(B, Hkv, M, page, D).transpose(1, 2)
                                      .reshape(B * M, Hkv, page, D))
        out.append(cache)
    return out[0], out[1], ids.int().cuda().contiguous()


def decode_reference(q, k, v, lens, window, sinks, scale):
    outs, tols = {"o": [], "lse": []}, {"o": [], "lse": []}
    B, Hq, _, D = q.shape
    for b, n in enumerate(lens):
        if n == 0:
            z = torch.zeros(1, Hq, 1, D, dtype=torch.float64)
            r, t = {"o": z, "lse": z[..., 0] + NEG}, {"o": z, "lse": z[..., 0]}
        else:
            r, t = reference(q[b:b + 1], k[b:b + 1, :, :n], v[b:b + 1, :, :n], window, sinks, scale)
        for name in outs:
            outs[name].append(r[name][:, :, 0])
            tols[name].append(t[name][:, :, 0])
    return {n: torch.cat(x) for n, x in outs.items()}, {n: torch.cat(x) for n, x in tols.items()}


# Hq, Hkv, D, window, sinks, lengths
DECODES = [
    (1, 1, 64, 1, 0, [1, 2, 33, 64]),
    (4, 1, 128, 40, 4, [0, 1, 39, 40, 41, 44, 45, 76, 300]),
    (8, 2, 64, 100, 33, [5, 32, 33, 132, 133, 134, 517]),
    (6, 2, 256, 64, 1, [64, 65, 96, 97, 400]),
    (17, 1, 128, 31, 70, [31, 70, 101, 102, 230]),      # a group wider than one MMA tile
    (4, 4, 128, 10 ** 6, 0, [1, 100, 333]),             # a window over everything
    (2, 1, 64, 3, 10 ** 6, [1, 100, 333]),              # sinks over everything
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", DECODES)
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 16, None])
def test_decode_matches_the_formula(case, splits):
    Hq, Hkv, D, window, sinks, lens = case
    B, Sk = len(lens), max(lens)
    q, k, v = inputs(B, Hq, Hkv, 1, Sk, D, 17 * Hq + D) if B else None
    scale = 1.0 / math.sqrt(D)
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # Keys past a sequence's length, and those that its window has passed, are garbage.
    kg, vg = k.clone(), v.clone()
    for b, n in enumerate(lens):
        hidden = torch.ones(Sk, dtype=torch.bool)
        hidden[:n] = ~visible(1, n, window, sinks)[0] if n else hidden[:0]
        kg[b, :, hidden.cuda()] = float("nan")
        vg[b, :, hidden.cuda()] = float("-inf")
    ref, tol = decode_reference(q, k, v, lens, window, sinks, scale)
    o, lse = attn.decode_window(q, kg, vg, window, sinks, seqlens=seqlens, num_splits=splits)
    assert attn.attn_debug_status() == attn.ATTN_OK
    check("o", o, ref["o"], tol["o"])
    check("lse", lse, ref["lse"], tol["lse"])
    for page in (32, 96):
        kc, vc, table = paged(kg, vg, page, seed=page)
        # Pages without a seen key are not read: their entries are no pages.
        slot = torch.arange(table.shape[1])
        for b, n in enumerate(lens):
            live = (slot * page < n) & (((slot + 1) * page > n - window) | (slot * page < sinks))
            table[b, ~live.cuda()] = -1
        op, lp = attn.decode_window_paged(q, kc, vc, table, seqlens, window, sinks,
                                          num_splits=splits)
        assert attn.attn_debug_status() == attn.ATTN_OK
        assert torch.equal(op, o) and torch.equal(lp, lse) or splits is None
        check("o", op, ref["o"], tol["o"])
        check("lse", lp, ref["lse"], tol["lse"])


@pytest.mark.gpu
def test_decode_without_lengths_is_the_forward_of_the_last_row():
    B, Hq, Hkv, Sk, D, window, sinks = 2, 8, 2, 777, 128, 130, 9
    q, k, v = inputs(B, Hq, Hkv, 1, Sk, D, 4)
    ref, tol = reference(q, k, v, window, sinks, 1.0 / math.sqrt(D))
    o, lse = attn.decode_window(q, k, v, window, sinks)
    check("o", o, ref["o"][:, :, 0], tol["o"][:, :, 0])
    check("lse", lse, ref["lse"][:, :, 0], tol["lse"][:, :, 0])


@pytest.mark.gpu
def test_decode_of_a_cache_past_32_bits():
    P, Hkv, page, D, window, sinks = 33000, 8, 64, 128, 200, 3  # 2.2e9 elements a cache
    kc = torch.empty(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    q, k, v = inputs(1, 16, Hkv, 1, 320, D, 12)
    table = torch.tensor([[P - 1, 7, P - 2, 5, P - 3]], dtype=torch.int32, device="cuda")
    for s, p in enumerate(table[0].tolist()):
        kc[p], vc[p] = k[0, :, s * page:(s + 1) * page], v[0, :, s * page:(s + 1) * page]
    seqlens = torch.tensor([311], dtype=torch.int32, device="cuda")
    ref, tol = decode_reference(q, k, v, [311], window, sinks, 1.0 / math.sqrt(D))
    o, lse = attn.decode_window_paged(q, kc, vc, table, seqlens, window, sinks)
    check("o", o, ref["o"], tol["o"])
    check("lse", lse, ref["lse"], tol["lse"])
    src = torch.tensor([P - 1, 5], dtype=torch.int32, device="cuda")
    dst = torch.tensor([9, P - 4], dtype=torch.int32, device="cuda")
    attn.attn_pages_copy(kc, vc, src, dst)
    for a, b in ((P - 1, 9), (5, P - 4)):
        assert torch.equal(kc[a], kc[b]) and torch.equal(vc[a], vc[b])


@pytest.mark.gpu
def test_decode_reports_a_bad_page_it_reaches():
    q, k, v = inputs(1, 2, 1, 1, 128, 64, 2)
    kc, vc, table = paged(k, v, 32, 1, spare=0)
    seqlens = torch.tensor([128], dtype=torch.int32, device="cuda")
    table[0, 1] = 99  # passed by the window: never looked at
    attn.decode_window_paged(q, kc, vc, table, seqlens, 40, 3)
    assert attn.attn_debug_status() == attn.ATTN_OK
    table[0, 3] = 4
    attn.decode_window_paged(q, kc, vc, table, seqlens, 40, 3)
    assert attn.attn_debug_status() == attn.ATTN_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [1, 12])
def test_streams_and_two_graphs_at_once(splits):
    Hq, Hkv, D, Sk, window, sinks = 8, 2, 128, 4096, 2000, 4
    sets = [inputs(1, Hq, Hkv, 1, Sk, D, s) for s in (1, 2)]
    want = [attn.decode_window(*s, window, sinks, num_splits=splits) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = attn.decode_window(*sets[0], window, sinks, num_splits=splits, stream=side)
    side.synchronize()
    assert torch.equal(on_side[0], want[0][0]) and torch.equal(on_side[1], want[0][1])
    graphs, outs = [], []
    for s in sets:  # both captured on one stream
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(attn.decode_window(*s, window, sinks, num_splits=splits))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 3])
def test_two_prefill_graphs_at_once(D, splits):
    window, sinks = 500, 4
    sets = [inputs(1, 4, 2, 200, 1500, D, s) for s in (1, 2)]
    want = [attn.attn_window_fwd(*s, window, sinks, num_splits=splits) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for s in sets:  # both captured on one stream
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(attn.attn_window_fwd(*s, window, sinks, num_splits=splits))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 6, 2, 2100, 2100, 64, 700, 4), (3, 8, 4, 1500, 2000, 128, 900, 130),
                                   (2, 5, 5, 3000, 3000, 64, 4000, 0), (4, 4, 2, 1300, 1300, 256, 400, 3)])
def test_heads_of_many_rounds_match_a_call_of_their_own(shape):
    # More items than SMs, in every order of the schedule: a KV head's rows come out the
    # same bits as when it is called alone.
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    q, k, v = inputs(B, Hq, Hkv, Sq, Sk, D, 3)
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=1)
    G = Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            one = [t[b:b + 1, h * n:(h + 1) * n].contiguous() for t, n in ((q, G), (k, 1), (v, 1))]
            o1, l1 = attn.attn_window_fwd(*one, window, sinks, num_splits=1)
            assert torch.equal(o1, o[b:b + 1, h * G:(h + 1) * G])
            assert torch.equal(l1, lse[b:b + 1, h * G:(h + 1) * G])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 80, 40, 600, 900, 64, 200, 5), (2, 45, 45, 500, 500, 128, 130, 0),
                                   (1, 90, 30, 250, 700, 256, 300, 140), (1, 88, 44, 500, 500, 128, 700, 0),
                                   (1, 152, 76, 200, 400, 64, 100, 3)])  # full rounds on 152 SMs
@pytest.mark.parametrize("splits", [2, 3, None])
def test_splits_of_the_last_round(shape, splits):
    # More items than SMs: those of the last round are cut, the others are not.
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    q, k, v = inputs(B, Hq, Hkv, Sq, Sk, D, 9)
    k, v = k.clone(), v.clone()
    unseen = ~visible(Sq, Sk, window, sinks).any(0)
    heads = [0, 1, Hkv // 2, Hkv - 1]
    G = Hq // Hkv
    of = [h * G + g for h in heads for g in range(G)]
    want, tol = reference(q[:, of], k[:, heads], v[:, heads], window, sinks, 1.0 / math.sqrt(D))
    k[:, :, unseen.cuda()] = float("nan")
    v[:, :, unseen.cuda()] = float("nan")
    whole, whole_lse = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=1)
    o, lse = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=splits)
    assert attn.attn_debug_status() == attn.ATTN_OK
    check("o", o[:, of], want["o"], tol["o"])
    check("lse", lse[:, of], want["lse"], tol["lse"])
    assert bool(torch.isfinite(o).all())
    # The rest agree with one split: two results of that bound, and whole rounds alike.
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 256 if D < 256 and G % 2 else 128
    tiles = -(-Sq // rows)
    items = B * Hkv * tiles * (G // 2 if rows == 128 and D < 256 else G)
    differ = (lse != whole_lse).sum().item()
    assert differ <= items % n_sm * (128 if D == 256 else 256)
    assert (o.float() - whole.float()).abs().max().item() <= 2 * tol["o"].max().item()


@pytest.mark.gpu
def test_threads_on_streams_of_their_own():
    shapes = [(1, 4, 2, 300, 300, 64, 70, 4), (1, 2, 2, 40, 2000, 128, 900, 3),
              (2, 6, 2, 500, 500, 64, 33, 130), (1, 8, 1, 700, 700, 128, 128, 0)]

    def work(shape, out, stream):
        B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
        with torch.cuda.stream(stream):
            q, k, v, do = inputs(B, Hq, Hkv, Sq, Sk, D, Sq, grad=True)
            for _ in range(5):
                o, lse = attn.attn_window_fwd(q, k, v, window, sinks)
                grads = attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
                dec = attn.decode_window(q[:, :, -1:].contiguous(), k, v, window, sinks)
            out.append((o, lse) + grads + dec)
            stream.synchronize()

    want = [[] for _ in shapes]
    for shape, out in zip(shapes, want):
        work(shape, out, torch.cuda.current_stream())
    got = [[] for _ in shapes]
    threads = [threading.Thread(target=work, args=(s, g, torch.cuda.Stream()))
               for s, g in zip(shapes, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, g in zip(want, got):
        for a, b in zip(w[0], g[0]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_training_step_in_a_graph_repeats_its_bits():
    B, Hq, Hkv, S, D, window, sinks = 1, 4, 2, 400, 64, 100, 4
    q, k, v, do = inputs(B, Hq, Hkv, S, S, D, 6, grad=True)

    def step():
        o, lse = attn.attn_window_fwd(q, k, v, window, sinks)
        return (o, lse) + attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks)

    want = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 4, 2, 301, 301, 64, 100, 4), (1, 4, 1, 129, 777, 128, 300, 5),
                                   (1, 3, 3, 300, 129, 64, 40, 200), (1, 2, 1, 1300, 1300, 128, 60, 5),
                                   (1, 2, 1, 200, 640, 256, 300, 5)])
def test_debug_build_stores_in_bounds_and_matches(shape):
    # Every output store checked against its buffer (a stray one is skipped and reported).
    from tensor_attn_fwd_gb300 import build as attn_build
    dbg = ctypes.CDLL(attn_build.build(debug=True))
    for name in ("attn_window_fwd", "attn_window_fwd_workspace", "attn_window_bwd", "attn_decode_window",
                 "attn_debug_status"):
        fn, like = getattr(dbg, name), getattr(attn.load_library(), name)
        fn.argtypes, fn.restype = like.argtypes, like.restype
    B, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    q, k, v, do = inputs(B, Hq, Hkv, Sq, Sk, D, 21, grad=True)
    scale, stream = 1.0 / math.sqrt(D), torch.cuda.current_stream().cuda_stream
    n = ctypes.c_longlong(0)
    assert dbg.attn_window_fwd_workspace(B, Hq, Hkv, Sq, D, 2, ctypes.byref(n)) == attn.ATTN_OK
    floats = n.value
    if D < 256:
        attn.load_library().attn_window_bwd_workspace(*shape, ctypes.byref(n))
    ws = torch.empty(max(floats, n.value), device="cuda")
    for splits in (1, 2):
        want = attn.attn_window_fwd(q, k, v, window, sinks, num_splits=splits)
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        assert dbg.attn_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                   lse.data_ptr(), ws.data_ptr(), B, Hq, Hkv, Sq, Sk, D, window,
                                   sinks, splits, scale, stream) == attn.ATTN_OK
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    if D < 256:
        want = attn.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
        got = [torch.empty_like(t) for t in want]
        assert dbg.attn_window_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                   lse.data_ptr(), do.data_ptr(), *(t.data_ptr() for t in got),
                                   ws.data_ptr(), *shape, scale, stream) == attn.ATTN_OK
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    qd = q[:, :, -1:].contiguous()
    for splits in (1, 9):
        want = attn.decode_window(qd, k, v, window, sinks, num_splits=splits)
        got = [torch.empty_like(t) for t in want]
        assert dbg.attn_decode_window(qd.data_ptr(), k.data_ptr(), v.data_ptr(), None,
                                      got[0].data_ptr(), got[1].data_ptr(), B, Hq, Hkv, Sk, D,
                                      window, sinks, splits, scale, stream) == attn.ATTN_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert dbg.attn_debug_status(None) == attn.ATTN_OK


# ------------------------------------------------------------------ refusals (no GPU)
A, M = 0x10000000, 0x10000004


def _lib():
    from tensor_attn_fwd_gb300 import build as attn_build
    attn_build.build()
    return attn.load_library()


def fwd(q=A, k=A, v=A, o=A, lse=A, B=1, Hq=2, Hkv=1, Sq=8, Sk=8, D=64, window=4, sinks=1,
        scale=0.125, ws=None, ns=1):
    return _lib().attn_window_fwd(q, k, v, o, lse, ws, B, Hq, Hkv, Sq, Sk, D, window, sinks, ns, scale,
                                  None)


def bwd(q=A, k=A, v=A, o=A, lse=A, do=A, dq=A, dk=A, dv=A, ws=A, B=1, Hq=2, Hkv=1, Sq=8, Sk=8, D=64,
        window=4, sinks=1, scale=0.125):
    return _lib().attn_window_bwd(q, k, v, o, lse, do, dq, dk, dv, ws, B, Hq, Hkv, Sq, Sk, D, window,
                                  sinks, scale, None)


COMMON = [
    (dict(q=None), attn.ATTN_ERR_INVALID_ARG),
    (dict(lse=None), attn.ATTN_ERR_INVALID_ARG),
    (dict(window=0), attn.ATTN_ERR_INVALID_ARG),
    (dict(window=-1), attn.ATTN_ERR_INVALID_ARG),
    (dict(sinks=-1), attn.ATTN_ERR_INVALID_ARG),
    (dict(Hq=3, Hkv=2), attn.ATTN_ERR_INVALID_ARG),
    (dict(Sq=0), attn.ATTN_ERR_INVALID_ARG),
    (dict(scale=float("inf")), attn.ATTN_ERR_INVALID_ARG),
    (dict(D=96), attn.ATTN_ERR_UNSUPPORTED),
    (dict(Sk=(1 << 30) + 1), attn.ATTN_ERR_UNSUPPORTED),
    (dict(v=M), attn.ATTN_ERR_MISALIGNED),
    (dict(o=M), attn.ATTN_ERR_MISALIGNED),
]


@pytest.mark.parametrize("call,kw,code", [(f, kw, c) for f in (fwd, bwd) for kw, c in COMMON] + [
    (fwd, dict(ns=0), attn.ATTN_ERR_INVALID_ARG),
    (fwd, dict(ns=-3, ws=A), attn.ATTN_ERR_INVALID_ARG),
    (fwd, dict(ns=2, Sk=300), attn.ATTN_ERR_INVALID_ARG),        # no workspace
    (fwd, dict(ns=4, Sk=300, ws=A), attn.ATTN_ERR_INVALID_ARG),  # three key tiles
    (fwd, dict(ns=2, Sk=300, ws=M), attn.ATTN_ERR_MISALIGNED),
    (fwd, dict(ns=2, Sk=300, ws=A, Sq=1 << 30), attn.ATTN_ERR_UNSUPPORTED),
    (bwd, dict(D=256), attn.ATTN_ERR_UNSUPPORTED),
    (bwd, dict(ws=None), attn.ATTN_ERR_INVALID_ARG),
    (bwd, dict(dk=M), attn.ATTN_ERR_MISALIGNED)])
def test_prefill_and_backward_reject(call, kw, code):
    assert call(**kw) == code


def test_forward_split_rule():
    n = ctypes.c_int(0)
    rule = _lib().attn_window_fwd_num_splits
    assert rule(1, 2, 1, 8, 8, 64, 4, 1, None) == attn.ATTN_ERR_INVALID_ARG
    assert rule(1, 2, 1, 8, 8, 64, 0, 1, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert rule(1, 2, 1, 8, 1 << 20, 64, 500, 1, ctypes.byref(n)) == attn.ATTN_OK and n.value >= 1
    big = 2**31 - 1  # too large for attn_window_fwd: still a count
    assert rule(big, big, 1, big, big, big, 5, 1, ctypes.byref(n)) == attn.ATTN_OK and n.value == 1


def test_forward_workspace():
    n = ctypes.c_longlong(-1)
    size = _lib().attn_window_fwd_workspace
    assert size(1, 2, 1, 8, 64, 1, None) == attn.ATTN_ERR_INVALID_ARG
    assert size(1, 2, 1, 8, 64, 0, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert size(1, 3, 2, 8, 64, 2, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert size(1, 2, 1, 8, 96, 2, ctypes.byref(n)) == attn.ATTN_ERR_UNSUPPORTED
    assert size(1, 4, 1, 1 << 30, 64, 2, ctypes.byref(n)) == attn.ATTN_ERR_UNSUPPORTED
    assert size(1, 2, 1, 8, 64, 1, ctypes.byref(n)) == attn.ATTN_OK and n.value == 0
    assert size(1, 2, 1, 8, 64, 3, ctypes.byref(n)) == attn.ATTN_OK and n.value >= 0


def test_decode_split_rule():
    n = ctypes.c_int(0)
    rule = _lib().attn_decode_window_num_splits
    assert rule(1, 2, 1, 100, 64, 4, 1, None) == attn.ATTN_ERR_INVALID_ARG
    assert rule(1, 2, 1, 0, 64, 4, 1, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert rule(1, 2, 1, 100, 64, 0, 1, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert rule(1, 3, 2, 100, 64, 4, 1, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert rule(1, 2, 1, 1 << 30, 64, 20, 1, ctypes.byref(n)) == attn.ATTN_OK and n.value == 1
    assert rule(1, 2, 1, 1 << 30, 64, 1 << 30, 1 << 30, ctypes.byref(n)) == attn.ATTN_OK
    assert 1 <= n.value <= 16


def test_backward_workspace():
    n = ctypes.c_longlong(0)
    size = _lib().attn_window_bwd_workspace
    assert size(1, 2, 1, 8, 8, 64, 4, 1, None) == attn.ATTN_ERR_INVALID_ARG
    assert size(1, 2, 1, 8, 8, 64, 0, 1, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert size(1, 3, 2, 8, 8, 64, 4, 1, ctypes.byref(n)) == attn.ATTN_ERR_INVALID_ARG
    assert size(1, 2, 1, 8, 8, 96, 4, 1, ctypes.byref(n)) == attn.ATTN_ERR_UNSUPPORTED
    assert size(1, 2, 1, 9, 9, 64, 4, 0, ctypes.byref(n)) == attn.ATTN_OK and n.value >= 2 * 9


def dec(q=A, k=A, v=A, sl=A, o=A, lse=A, B=1, Hq=4, Hkv=1, Sk=64, D=128, window=8, sinks=1, ns=4,
        scale=0.1):
    return _lib().attn_decode_window(q, k, v, sl, o, lse, B, Hq, Hkv, Sk, D, window, sinks, ns, scale,
                                     None)


def decp(q=A, k=A, v=A, sl=A, o=A, lse=A, B=1, Hq=4, Hkv=1, D=128, window=8, sinks=1, ns=4, scale=0.1,
         bt=A, num_pages=8, page=64, max_pages=4):
    return _lib().attn_decode_window_paged(q, k, v, bt, sl, o, lse, B, Hq, Hkv, num_pages, page,
                                           max_pages, D, window, sinks, ns, scale, None)


@pytest.mark.parametrize("call,kw,code", list(itertools.chain.from_iterable(
    [(f, kw, c) for kw, c in [
        (dict(o=None), attn.ATTN_ERR_INVALID_ARG),
        (dict(lse=None), attn.ATTN_ERR_INVALID_ARG),
        (dict(ns=17), attn.ATTN_ERR_INVALID_ARG),
        (dict(ns=-1), attn.ATTN_ERR_INVALID_ARG),
        (dict(window=0), attn.ATTN_ERR_INVALID_ARG),
        (dict(sinks=-3), attn.ATTN_ERR_INVALID_ARG),
        (dict(ns=0), attn.ATTN_ERR_INVALID_ARG),
        (dict(ns=10 ** 6), attn.ATTN_ERR_INVALID_ARG),
        (dict(D=96), attn.ATTN_ERR_UNSUPPORTED),
        (dict(B=70000), attn.ATTN_ERR_UNSUPPORTED),
        (dict(k=M), attn.ATTN_ERR_MISALIGNED),
        (dict(o=M), attn.ATTN_ERR_MISALIGNED),
        (dict(lse=M), attn.ATTN_ERR_MISALIGNED),
        (dict(sl=A + 1), attn.ATTN_ERR_MISALIGNED),
    ]] for f in (dec, decp))) + [
        (decp, dict(sl=None), attn.ATTN_ERR_INVALID_ARG),
        (decp, dict(bt=None), attn.ATTN_ERR_INVALID_ARG),
        (decp, dict(page=48), attn.ATTN_ERR_UNSUPPORTED),
        (decp, dict(max_pages=1 << 25), attn.ATTN_ERR_UNSUPPORTED)])
def test_decode_rejects(call, kw, code):
    assert call(**kw) == code


def test_python_rejects():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        attn.attn_window_fwd(q, q, q, 4)  # CPU tensors
    with pytest.raises(ValueError):
        attn.attn_window_bwd(q, q, q, q, q, q, 4)
    with pytest.raises(ValueError):
        attn.decode_window(q[:, :, :1], q, q, 4)


@pytest.mark.gpu
def test_python_rejects_shapes_types_and_reach():
    q, k, v = inputs(1, 2, 1, 8, 8, 64, 1)
    o, lse = attn.attn_window_fwd(q, k, v, 4)
    for bad in (dict(window=0), dict(window=-2), dict(window=4, sinks=-1)):
        with pytest.raises(ValueError):
            attn.attn_window_fwd(q, k, v, **bad)
    for splits in (0, 2, 2**30):  # one key tile
        with pytest.raises((ValueError, RuntimeError)):
            attn.attn_window_fwd(q, k, v, 4, num_splits=splits)
    with pytest.raises(ValueError):
        attn.attn_window_fwd(q.float(), k, v, 4)
    with pytest.raises(ValueError):
        attn.attn_window_fwd(q.transpose(1, 2), k, v, 4)
    with pytest.raises(ValueError):
        attn.attn_window_bwd(q, k, v, o.float(), lse, q, 4)   # o is bf16
    with pytest.raises(ValueError):
        attn.attn_window_bwd(q, k, v, o, None, q, 4)
    with pytest.raises(ValueError):
        attn.decode_window(q, k, v, 4)                        # eight query rows
    with pytest.raises(ValueError):
        attn.decode_window(q[:, :, :1].contiguous(), k, v, 4,
                           seqlens=torch.tensor([8], device="cuda"))  # int64 lengths
