// window.cuh -- which 128-key tiles a 128-row query tile needs under a sliding
// window with sinks, and the reverse.  Query row i stands at position
// p = i + off, off = Sk - Sq, and sees key j iff
//   j <= p and (j > p - window or j < sinks).
// window and sinks are clamped to [1, Sk] and [0, Sk] by the host, so no sum
// below leaves the range of int (sequences are at most 2^30 long).
#pragma once

#include <cstdint>
#include <type_traits>

#include "ptx.cuh"

namespace attn {

// Division of 0 <= n < 2^31 by a fixed d >= 1 with one multiplication (Granlund and
// Montgomery, "Division by Invariant Integers using Multiplication", 1994).
struct FixedDiv {
  uint32_t mul, shift;
  FixedDiv() = default;
  explicit FixedDiv(uint32_t d) : shift(d > 1 ? 32 - __builtin_clz(d - 1) : 0) {
    mul = static_cast<uint32_t>((((1ull << shift) - d) << 32) / d + 1);
  }
  __host__ __device__ __forceinline__ int div(int n) const {
    const uint32_t x = static_cast<uint32_t>(n);
    return static_cast<int>((static_cast<uint32_t>((static_cast<uint64_t>(x) * mul) >> 32) + x) >> shift);
  }
};

// KV tiles [b, s) and [w, e) in that order, or none (e = 0).  Of a whole query tile
// b = 0 and s <= w < e: [0, s) holds sinks and [w, e) runs from its first row's window
// start to its last row's position (sink tiles that meet it are counted to it).  A
// run of steps of such a list (steps()) has the same form; without tiles of one part
// b = s = 0, or w = e = s.  e - 1 is always the last tile.
struct TileRange {
  int b, s, w, e;
  __device__ __forceinline__ int first() const { return b < s ? b : w; }
  __device__ __forceinline__ int next(int j) const { return j + 1 == s ? w : j + 1; }
  __device__ __forceinline__ bool has(int j) const {
    return (j >= b && j < s) || (j >= w && j < e);
  }
  __host__ __device__ __forceinline__ int count() const { return s - b + e - w; }
  __device__ __forceinline__ int tile(int step) const {
    return step < s - b ? b + step : step - (s - b) + w;
  }
  // Steps [x, y) of a whole list, y clamped to its end.
  __device__ __forceinline__ TileRange steps(int x, int y) const {
    y = min(y, count());
    if (x >= y) return {0, 0, 0, 0};
    if (x >= s) return {0, 0, w + x - s, w + y - s};
    if (y <= s) return {x, y, y, y};
    return {x, s, w, w + y - s};
  }
};

__host__ __device__ __forceinline__ TileRange window_kv_tiles(int Sq, int Sk, int window, int sinks,
                                                     int row_first) {
  TileRange r = {0, 0, 0, 0};
  const int row_last = min(row_first + 127, Sq - 1);
  const int hi = row_last + Sk - Sq + 1;  // keys [0, hi) up to the last row's position
  if (row_first >= Sq || hi <= 0) return r;
  r.e = (hi + 127) / 128;
  r.w = max(row_first + Sk - Sq - window + 1, 0) / 128;
  r.s = min((min(sinks, hi) + 127) / 128, r.w);
  return r;
}

// Order of the forward's items (per_group of them at each tile of a KV head, n_bg KV
// heads).  First the tiles whose rows all have their whole window, which take equally
// long: KV head by KV head, so that the items in flight share K/V in L2.  Then the
// `ramp` tiles below, longest first across the heads, which balances the
// CTAs: with all of them in the first order a window of all of S = 4096 keys (16/8
// heads of 128) took 76.3 us instead of 51.5, and one of 512 keys at B2 S4096 32/8 heads
// 80.1 instead of 71.1.
//
// Every role of a CTA works an item out for itself, between two items, so the divisions
// are multiplications (as divisions they cost 0.7 us an item).
//
// With splits, the last round of items, which does not fill the CTAs, is cut along the
// keys into num_splits parts each, so that it takes a part of the time: the first
// `unsplit` items are left whole, a multiple of the CTAs, and the `rem` others are
// counted split by split (slot: their number).
struct WindowItem {
  int split, slot;  // slot -1: whole
  int bg, member, tile;
};
struct WindowOrder {
  int tiles, n_bg, per_group, num_splits, unsplit, rem, ramp, ctas;
  FixedDiv by_rem, by_group, by_whole, by_bg, by_num_splits;

  // rows: query rows of a tile; ctas: that run at once.
  static WindowOrder make(int Sq, int Sk, int window, int rows, int n_bg, int per_group,
                          int num_splits, int ctas) {
    WindowOrder o;
    o.tiles = (Sq + rows - 1) / rows;
    o.n_bg = n_bg;
    o.per_group = per_group;
    const int items = n_bg * per_group * o.tiles;
    o.unsplit = num_splits == 1 ? items : items / ctas * ctas;
    o.rem = items - o.unsplit;
    o.num_splits = o.rem == 0 ? 1 : num_splits;
    o.ctas = o.total() < ctas ? o.total() : ctas;  // of the launch
    // Tiles that hold a row with less than its window before it.
    const long long short_rows = static_cast<long long>(window) - 1 - (Sk - Sq);
    const long long n = short_rows <= 0 ? 0 : (short_rows + rows - 1) / rows;
    o.ramp = n < o.tiles ? static_cast<int>(n) : o.tiles;
    o.by_rem = FixedDiv(o.rem > 0 ? o.rem : 1);
    o.by_group = FixedDiv(per_group);
    o.by_whole = FixedDiv(o.tiles > o.ramp ? o.tiles - o.ramp : 1);
    o.by_bg = FixedDiv(n_bg);
    o.by_num_splits = FixedDiv(o.num_splits);
    return o;
  }
  int total() const { return unsplit + rem * num_splits; }
  __host__ __device__ __forceinline__ WindowItem item(int idx) const {
    WindowItem x;
    x.split = 0;
    x.slot = -1;
    if (idx >= unsplit) {
      x.split = by_rem.div(idx - unsplit);
      x.slot = idx - unsplit - x.split * rem;
      idx = unsplit + x.slot;
    }
    const int rest = by_group.div(idx);
    x.member = idx - rest * per_group;
    const int whole = tiles - ramp;
    if (rest < n_bg * whole) {
      x.bg = by_whole.div(rest);
      x.tile = tiles - 1 - (rest - x.bg * whole);
    } else {
      const int t = by_bg.div(rest - n_bg * whole);
      x.bg = rest - n_bg * (whole + t);
      x.tile = ramp - 1 - t;
    }
    return x;
  }
  // An item's part of a tile's list: its split-th equal run of steps.
  __device__ __forceinline__ TileRange steps_of(const TileRange& r, const WindowItem& x) const {
    if (x.slot < 0) return r;
    const int chunk = by_num_splits.div(r.count() + num_splits - 1);
    return r.steps(x.split * chunk, x.split * chunk + chunk);
  }
};

// Where the rows of split items go: partials in [split][slot][item_rows], and the row
// of O (b * Hq + h) * Sq + i, or -1, that row `row` of a split's [slot][item_rows] is.
// An item of 256 rows is a tile of two heads (head_pairs), or two tiles of one.
struct WindowRows {
  WindowOrder order;
  int Sq, head_pairs, item_rows;
  __device__ __forceinline__ int operator()(int row) const {
    const int slot = item_rows == 256 ? row >> 8 : row >> 7, r = row - slot * item_rows;
    const WindowItem x = order.item(order.unsplit + slot);
    const int head = ((x.bg * order.per_group + x.member) << head_pairs) + (head_pairs ? r >> 7 : 0);
    const int i = head_pairs ? x.tile * 128 + (r & 127) : x.tile * item_rows + r;
    return i < Sq ? head * Sq + i : -1;
  }
};

// The tiles of two neighbouring query tiles as one list (it may hold a tile that
// neither needs).
__device__ __forceinline__ TileRange tile_union(const TileRange& x, const TileRange& y) {
  if (x.e == 0) return y;
  if (y.e == 0) return x;
  TileRange u;
  const bool xs = x.b < x.s, ys = y.b < y.s;
  u.b = xs && ys ? min(x.b, y.b) : (xs ? x.b : y.b);
  u.s = max(x.s, y.s);
  const bool xw = x.w < x.e, yw = y.w < y.e;
  u.w = xw && yw ? min(x.w, y.w) : (xw ? x.w : y.w);
  u.e = max(x.e, y.e);
  if (!xw && !yw) {
    u.w = u.e = u.s;
  } else if (u.s >= u.w) {  // the parts meet: one run from the lower begin
    if (u.b < u.s) u.w = min(u.w, u.b);
    u.b = u.s = 0;
  }
  return u;
}

// The kernels' masks.  kUnseen is kWindow for calls with keys that no row sees (a
// chunk against a longer sequence), which have to be kept from the products; the work
// for it in the MMA warp's loop costs a training step, which has none, 2.4 %.
enum Mask { kNoWindow = 0, kWindow = 1, kUnseen = 2 };
// A kernel's parameters: the windowed kernels' have members more.  The plain ones read none
// of them, but a longer parameter block alone changes what the compiler makes of a kernel:
// where it cost something (the plain dQ kernel 2 to 4 %, with 134 registers for 140; the
// forward of D <= 128 0.3 to 1 %) the plain form is not given them.
template <Mask WIN, typename Plain, typename Windowed>
using ParamsOf = std::conditional_t<WIN == kNoWindow, Plain, Windowed>;

// Keys [sinks, unseen_end) are seen by no row: the first row's window starts at
// unseen_end.
__host__ __device__ __forceinline__ int unseen_end(int Sq, int Sk, int window) {
  return Sk - Sq - window + 1 > 0 ? Sk - Sq - window + 1 : 0;
}
inline bool has_unseen(int Sq, int Sk, int window, int sinks) {
  return sinks < unseen_end(Sq, Sk, window);
}
// Their rows of a K or V tile of keys [key0, key0 + 128) in shared memory (128-byte
// swizzled sub-tiles of 64 dims) become zero: memory that no row sees may hold NaN, and
// a weight of 0 times NaN is NaN.  A whole warp, which afterwards may issue MMAs on
// the tile; nothing to do but for the two tiles at the ends of the range.
template <int D>
__device__ __forceinline__ void zero_unseen_rows(uint8_t* tile, int key0, int sinks, int end,
                                                 int lane) {
  // (Tiles wholly inside the range are read by nobody.)
  if (key0 != (sinks & ~127) && key0 != (end & ~127)) return;
  const int r0 = max(sinks - key0, 0), r1 = min(end - key0, 128);
  if (r0 >= r1) return;
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  for (int i = lane; i < (r1 - r0) * kChunks; i += 32) {
    const int r = r0 + i / kChunks, c = i % kChunks;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * (128 * 128) + r * 128 + (c & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

// Masks of 32 columns as bits: one test per column, where the comparisons of the
// visibility rule cost several instructions each (a masked 128-key step of the
// forward took 3.4 us with them).
__device__ __forceinline__ uint32_t bits_below(int n) {  // bits [0, n), n clamped to [0, 32]
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}
// Bits [lo, hi), and of those below lo the first `sinks`.
__device__ __forceinline__ uint32_t window_bits(int lo, int hi, int sinks) {
  return bits_below(hi) & (~bits_below(lo) | bits_below(sinks));
}

// Query tiles [m0, m1) of 128 rows that see a key of key tile n (m1 <= m0: none):
// from the row at the tile's first key to the last row whose window reaches its
// last key, or to the end where the tile holds a sink.
struct QTileRange {
  int m0, m1;
};

__device__ __forceinline__ QTileRange window_q_tiles(int Sq, int Sk, int window, int sinks, int n) {
  const int off = Sk - Sq;
  const int mtiles = (Sq + 127) / 128;
  QTileRange r;
  r.m0 = min(max(128 * n - off, 0) / 128, mtiles);
  r.m1 = mtiles;
  if (128 * n >= sinks) {
    const int last = min(128 * n + 127, Sk - 1) - off + window - 1;
    r.m1 = last < 0 ? 0 : min(mtiles, last / 128 + 1);
  }
  return r;
}

}  // namespace attn
