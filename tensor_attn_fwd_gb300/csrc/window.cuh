// window.cuh -- which 128-key tiles a 128-row query tile needs under a sliding
// window with sinks, and the reverse.  Query row i stands at position
// p = i + off, off = Sk - Sq, and sees key j iff
//   j <= p and (j > p - window or j < sinks).
// window and sinks are clamped to [1, Sk] and [0, Sk] by the host, so no sum
// below leaves the range of int (sequences are at most 2^30 long).
#pragma once

#include <cstdint>

namespace attn {

// KV tiles [0, s) and [w, e) with s <= w < e, or none (e = 0).  The window part of
// a tile's rows runs from its first row's window start to its last row's
// position; sink tiles that meet it are counted to it (s = w: one run).
struct TileRange {
  int s, w, e;
  __device__ __forceinline__ int first() const { return s > 0 ? 0 : w; }
  __device__ __forceinline__ int next(int j) const { return j + 1 == s ? w : j + 1; }
  __device__ __forceinline__ bool has(int j) const { return j < s || (j >= w && j < e); }
  __device__ __forceinline__ int count() const { return e > 0 ? s + e - w : 0; }
  __device__ __forceinline__ int tile(int step) const { return step < s ? step : step - s + w; }
};

__device__ __forceinline__ TileRange window_kv_tiles(int Sq, int Sk, int window, int sinks,
                                                     int row_first) {
  TileRange r = {0, 0, 0};
  const int row_last = min(row_first + 127, Sq - 1);
  const int hi = row_last + Sk - Sq + 1;  // keys [0, hi) up to the last row's position
  if (row_first >= Sq || hi <= 0) return r;
  r.e = (hi + 127) / 128;
  r.w = max(row_first + Sk - Sq - window + 1, 0) / 128;
  r.s = min((min(sinks, hi) + 127) / 128, r.w);
  return r;
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
