// attn_bwd.cu -- attention backward (dQ, dK, dV) on sm_103a tensor cores.
//
// Source: "A Thread-Register Decoupled GPU Execution Model for Efficient Tensor
// Computation", Methodology and Evaluation (the FlashAttention backward: more
// GEMMs than the forward, more live tensors, operand transposes and score
// recomputation).  For O = softmax(S) V with S = scale * Q K^T (+ mask) and an
// upstream gradient dO:
//   P = exp(S - LSE)   Delta_i = sum_d dO_id O_id   dP = dO V^T
//   dS = P * (dP - Delta)   dV = P^T dO   dK = scale * dS^T Q   dQ = scale * dS K
// (dK and dV sum over the query heads that share a KV head).
//
// Three kernels, enqueued in order on the caller's stream:
//   delta kernel  Delta = rowsum(dO * O) into caller workspace.
//   dK/dV kernel  one CTA per 128-key tile of one KV head.  It loops over every
//                 (query head of the group, 128-row query tile) that sees those
//                 keys: S^T = K Q^T and dP^T = V dO^T (smem x smem) into TMEM;
//                 the gradient warps (one thread per key) turn them into P^T
//                 and dS^T (bf16, written back into TMEM over S^T / dP^T); then
//                 dV += P^T dO and dK += dS^T Q accumulate in TMEM.  No atomics.
//                 Per step the MMA warp issues dV(s) as soon as P^T(s) is in
//                 TMEM and S^T(s+1) right behind it (it overwrites P^T(s) only
//                 after dV has read it), so the gradient warps' dS^T(s) overlaps
//                 dV(s) and S^T(s+1); then dK(s) once dS^T(s) is in TMEM and
//                 dP^T(s+1), which overlap the exponentials of step s+1.
//   dQ kernel     persistent (one CTA per SM) over the 128-row query tiles,
//                 highest first: S = Q K^T and dP = dO V^T recomputed for each
//                 visible KV tile, dS written into TMEM, dQ += dS K accumulated
//                 in one of two TMEM buffers (a tile's epilogue overlaps the
//                 next tile's products; its Q and dO load once the current
//                 tile's last S and dP are done).  S(s+1) is issued as soon as
//                 the gradient warps have read S(s), so it overlaps their work
//                 on step s; K and V stream through separate rings (K is
//                 needed until dQ(s), V only until dP(s)).
// Roles (320 threads): warps 0-7 gradient math (two warpgroups, each owning 64
// of a tile's 128 columns: the backward needs no row reductions, so the split
// is free), warp 8 MMA issue, warp 9 TMA.  Each warpgroup writes its bf16
// P / dS values into its own half of the S / dP columns, so neither can
// overwrite scores the other has not read yet.
// The Q/dO (dK/dV kernel) or K/V (dQ kernel) tiles stream through a two-stage
// ring; the fixed operand tiles are loaded once.  All waits are bounded.
//
// The windowed instantiations (Mask; window.cuh) walk the tiles that a sliding window
// with sinks leaves, take a bf16 O and write bf16 gradients.  They run dQ first, which
// computes Delta in two warps of its own, then dK/dV, whose key tiles with sinks are
// cut into parts (SinkSplit), then the parts' sum.  8192 rows, 32/8 heads, D = 128,
// window 1024, sinks 4: 408 us (dQ 165, dK/dV 240).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "window.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int kBwdThreads = 320;
constexpr int kBwdMmaWarp = 8;
constexpr int kBwdLoadWarp = 9;
constexpr int kGradThreads = 256;
constexpr int kDqDeltaWarp = 10;  // windowed dQ: warps 10 and 11 compute Delta
constexpr int kDqWinThreads = 384;
// Query tiles of few key tiles compute Delta a second time (see the dQ kernel).
constexpr int kExactDeltaSteps = 4;
constexpr uint32_t kDqDeltaBytes = 3 * 128 * sizeof(float);  // two tiles' Delta, one's sums
constexpr int kStages = 2;
constexpr uint32_t kSub = 128 * 128;  // [128 rows x 64 bf16] 128B-swizzled sub-tile
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kKStages = 3;  // dQ kernel: K ring
constexpr int kVStages = 2;  // dQ kernel: V ring

template <int D>
struct BwdCfg {
  static constexpr uint32_t kTile = (D / 64) * kSub;  // one 128 x D bf16 tile
  // dK/dV smem: two fixed tiles, kStages x (two streamed tiles), then scalars/barriers
  static constexpr uint32_t kFixed = 2 * kTile;
  static constexpr uint32_t kRing = kStages * 2 * kTile;
  // Per gradient warp: -LSE2 and -Delta of its 64 columns for the current step.
  static constexpr uint32_t kScalars = 8 * 2 * 64 * 4;
  static constexpr uint32_t kBarBytes = 256;
  static constexpr size_t kSmem = 1024 + kFixed + kRing + kScalars + kBarBytes;
  // dQ smem: Q and dO fixed, a K ring and a V ring, barriers.
  static constexpr size_t kSmemDq =
      1024 + kFixed + size_t(kKStages + kVStages) * kTile + kBarBytes;
  static_assert(kSmem <= 232448 && kSmemDq + kDqDeltaBytes <= 232448, "shared memory per CTA");
  static constexpr uint32_t kColS = 0, kColDP = 128, kColA0 = 256, kColA1 = 256 + D;
  static constexpr uint32_t kIdescSS = idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t kIdescTS = idesc_bf16_f32(128, D, false, true);
};

struct BwdBars {
  uint64_t fixed_full;
  uint64_t full[kKStages], empty[kKStages];     // dK/dV: Q+dO stages; dQ: K stages
  uint64_t full_v[kVStages], empty_v[kVStages];  // dQ: V stages
  uint64_t s_full;    // S (or S^T) of the current step is in TMEM
  uint64_t dp_full;   // dP (or dP^T) of the current step is in TMEM
  uint64_t p_ready;   // dK/dV: P^T written; dQ: S read (its columns are free)
  uint64_t ds_full;   // dS (or dS^T) written
  uint64_t acc_full;  // all accumulating MMAs have completed
  uint64_t mma_done;
  // persistent dQ kernel: Q/dO buffer reusable; dQ accumulator b complete / read out
  uint64_t q_empty, acc_full2[2], acc_free[2];
  // windowed dQ: Delta of a tile is in shared memory / has been read (two buffers)
  uint64_t delta_full[2], delta_free[2];
  // ... and the sums of P dP of warps 4-7 / those of warps 0-7 are in shared memory
  uint64_t part_full, total_full;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(BwdBars) <= 256, "barrier block too large");

struct BwdParams {
  const float* lse;    // [B,Hq,Sq] natural log
  const float* delta;  // [B,Hq,Sq]
  float* out0;         // dkdv: dK [B,Hkv,Sk,D]; dq: dQ [B,Hq,Sq,D]
  float* out1;         // dkdv: dV
  int* status;
  int B, Hq, Hkv, Sq, Sk, causal;
  float scale, scale_log2;
  // Named by code that the plain dQ kernel does not reach (BwdWindowParams has its own).
  static constexpr int window = 0, sinks = 0;
};
// The windowed kernels': the visibility of window.cuh, and bf16 gradients (out0, out1 point
// at bf16).
struct BwdWindowParams : BwdParams {
  int window, sinks;
  // dQ, which runs first: it computes Delta from O and dO for its tiles and
  // leaves it in delta_out for dK/dV.
  const __nv_bfloat16 *o, *dout;
  float* delta_out;
  // Windowed dK/dV: the first split_tiles key tiles (those with sinks, which every
  // later row sees) are cut along their steps into `parts` CTAs each.  Part i of
  // such a tile writes fp32 partials, [part][tile][B * Hkv][128][D], dK's then dV's,
  // to `partials`; bwd_sum_parts_kernel adds them in order.
  int split_tiles, parts;
  float* partials;
  // Windowed: B * Hq, B * Hkv, Hq / Hkv, parts.  (As divisions they cost dQ's roles,
  // which find their next tile between two, about as much as the forward's.)
  FixedDiv by_q_planes, by_kv_planes, by_group, by_parts;
};
// dQ's parameters.  (dK/dV takes the windowed ones in either form: as it is compiled, the
// plain kernel is 0.6 to 1 % slower with the others.)
template <Mask WIN>
using DqArgs = ParamsOf<WIN, BwdParams, BwdWindowParams>;

// Read-only global load issued where it stands in the program.
__device__ __forceinline__ float ld_nc_f32(const float* ptr) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(ptr) : "memory");
  return v;
}

__device__ __forceinline__ void bwd_record(int* status) {
  if (status != nullptr) atomicCAS(status, 0, ATTN_ERR_TIMEOUT);
}

__device__ __forceinline__ bool bwd_wait(uint64_t* bar, uint32_t parity, BwdBars* bars);

// The wait for a whole converged warp (the TMA and MMA roles run as whole warps
// and issue from one elected lane); the vote keeps the outcome uniform.  Used
// once per work item.  Inside a step those warps wait without a vote (a vote
// per wait costs several per cent): each lane keeps its outcome, issue
// continues with in-bounds addresses, and one vote per step makes the stop
// decision uniform; a lane still polling is waited for by the next elect.sync.
__device__ __forceinline__ bool bwd_wait_w(uint64_t* bar, uint32_t parity, BwdBars* bars) {
  return __all_sync(0xffffffffu, bwd_wait(bar, parity, bars));
}

__device__ __forceinline__ bool bwd_wait(uint64_t* bar, uint32_t parity, BwdBars* bars) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(a, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&bars->abort)) return false;
    if (globaltimer() - t0 > ATTN_WAIT_NS) {
      *reinterpret_cast<volatile int*>(&bars->abort) = 1;
      return false;
    }
  }
}

// First 128-row query tile that can see key tile n (bottom-right causal).
__device__ __forceinline__ int first_q_tile(const BwdParams& p, int n) {
  if (!p.causal) return 0;
  const int row = 128 * n - (p.Sk - p.Sq);
  return row <= 0 ? 0 : row / 128;
}

// KV tiles a query tile needs (as in the forward).
__device__ __forceinline__ int kv_tiles_for(const BwdParams& p, int m) {
  const int row_first = 128 * m;
  if (row_first >= p.Sq) return 0;
  int nvis = p.Sk;
  if (p.causal) {
    const int row_last = min(row_first + 127, p.Sq - 1);
    nvis = min(p.Sk, row_last + p.Sk - p.Sq + 1);
    if (nvis <= 0) return 0;
  }
  return (nvis + 127) / 128;
}

// ------------------------------------------------------------------ Delta
template <int D>
__global__ void __launch_bounds__(256) bwd_delta_kernel(const __nv_bfloat16* __restrict__ dout,
                                                        const float* __restrict__ o,
                                                        float* __restrict__ delta, int rows) {
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  constexpr int DPL = D / 32;
  const __nv_bfloat16* dr = dout + static_cast<size_t>(row) * D + lane * DPL;
  const float* orow = o + static_cast<size_t>(row) * D + lane * DPL;
  float acc = 0.f;
#pragma unroll
  for (int e = 0; e < DPL; ++e) acc = fmaf(__bfloat162float(dr[e]), orow[e], acc);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  if (lane == 0) delta[row] = acc;
}

// Delta of 32 consecutive rows by one warp: lane l returns row row0 + l's.  D / 8 lanes
// read a row's O and dO in 16-byte loads, 256 / D rows at a time; the lanes' partial
// sums are reduced and spread by exchanging halves (each exchange halves the values
// a lane carries).  Rows from `rows` on read the last row.
template <int D>
__device__ __forceinline__ float warp_delta(const __nv_bfloat16* o, const __nv_bfloat16* dout,
                                            long long row0, long long rows, int lane) {
  constexpr int L = D / 8;        // lanes a row
  constexpr int R = 32 / L;       // rows at a time
  constexpr int N = 32 / R;       // values a lane starts with (= L)
  float acc[N];
#pragma unroll
  for (int i0 = 0; i0 < N; i0 += 4) {
    uint4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long row = min(row0 + (i0 + i) * R + lane / L, rows - 1);
      a[i] = __ldg(reinterpret_cast<const uint4*>(o) + row * L + lane % L);
      b[i] = __ldg(reinterpret_cast<const uint4*>(dout) + row * L + lane % L);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, y[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // a bf16 is the upper half of its float
        sum = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), sum);
        sum = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), sum);
      }
      acc[i0 + i] = sum;
    }
  }
  // Lane l ends with value l % L of its group of L lanes: row (l % L) * R + l / L.
#pragma unroll
  for (int m = L / 2; m > 0; m >>= 1) {
    const bool upper = lane & m;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float give = upper ? acc[i] : acc[i + m];
      const float keep = upper ? acc[i + m] : acc[i];
      acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
  return __shfl_sync(0xffffffffu, acc[0], (lane % R) * L + lane / R);
}

// ------------------------------------------------------------------ shared pieces
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                          int row0, int plane) {
#pragma unroll
  for (int s = 0; s < D / 64; ++s) tma_load_3d(dst + s * kSub, map, bar, s * 64, row0, plane);
}

// One 128x128 SS product into TMEM column d_col (called by the whole MMA warp): a b^T (K-major tiles, D deep).
template <int D>
__device__ __forceinline__ void mma_ss_tile(uint32_t tmem, uint32_t d_col, uint32_t a_smem,
                                            uint32_t b_smem) {
  using C = BwdCfg<D>;
  constexpr uint64_t kDesc = sdesc_sw128(0, 16, 1024);
  constexpr uint32_t kHi = static_cast<uint32_t>(kDesc >> 32);
  constexpr uint32_t kLo = static_cast<uint32_t>(kDesc);
  const uint32_t a = kLo + (a_smem >> 4);
  const uint32_t b = kLo + (b_smem >> 4);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kSub + (kk & 3) * 32) >> 4;
    const uint64_t ad = desc_from_words(a + off, kHi);
    const uint64_t bd = desc_from_words(b + off, kHi);
    if (kk == 0)
      mma_ss_w<0>(tmem + d_col, ad, bd, C::kIdescSS);
    else
      mma_ss_w<1>(tmem + d_col, ad, bd, C::kIdescSS);
  }
}

// acc (+)= A(tmem, 128 x 128 bf16 at column a_col) x B(smem tile, MN-major)
// (called by the whole MMA warp).
template <int D>
__device__ __forceinline__ void mma_ts_acc(uint32_t tmem, uint32_t acc_col, uint32_t a_col,
                                           uint32_t b_smem, bool first) {
  using C = BwdCfg<D>;
  constexpr uint64_t kDesc = sdesc_sw128(0, kSub, 1024);
  constexpr uint32_t kHi = static_cast<uint32_t>(kDesc >> 32);
  constexpr uint32_t kLo = static_cast<uint32_t>(kDesc);
  const uint32_t b = kLo + (b_smem >> 4);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint64_t bd = desc_from_words(b + kk * (2048 >> 4), kHi);
    // bf16 A: rows 0-63 packed at columns [0,32), rows 64-127 at [64,96).
    const uint32_t ac = a_col + kk * 8 + (kk >= 4 ? 32 : 0);
    if (first && kk == 0)
      mma_ts_w<0>(tmem + acc_col, tmem + ac, bd, C::kIdescTS);
    else
      mma_ts_w<1>(tmem + acc_col, tmem + ac, bd, C::kIdescTS);
  }
}

// Read columns [c_begin, c_end) of this thread's fp32 accumulator row from
// TMEM, scale them and store them to global memory (valid rows only).  Rows
// are D floats apart and lane l holds row l of its warp's 32; lane pairs swap
// half their segments (pair_transpose8) so that each store writes 64
// contiguous bytes of one row.  All 32 lanes must call it.
template <int D>
__device__ __forceinline__ void store_acc_row(uint32_t taddr, float* dst, float mul, bool valid,
                                              int c_begin, int c_end, int lane, const float* base,
                                              size_t bytes, int* status) {
  const int pb = lane & 1;
  const bool partner_valid = __shfl_xor_sync(0xffffffffu, valid, 1);
  const bool even_valid = pb ? partner_valid : valid, odd_valid = pb ? valid : partner_valid;
  float* even_row = dst - pb * D;
  const bool v8 = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
  for (int c = c_begin; c < c_end; c += 32) {
    uint32_t w[32];
    tmem_ld32(taddr + c, w);
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * mul);
    pair_transpose8(w, lane);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float* e = even_row + c + 8 * (2 * m + pb);
      float* o = even_row + D + c + 8 * (2 * m + pb);
      if (even_valid && store_in_bounds(e, 32, base, bytes, status)) st_global_8w(e, &w[16 * m], v8);
      if (odd_valid && store_in_bounds(o, 32, base, bytes, status)) st_global_8w(o, &w[16 * m + 8], v8);
    }
  }
}

// The same for a bf16 gradient (each fp32 sum rounded to nearest even once); the
// lanes of a pair write 32 contiguous bytes each.
template <int D>
__device__ __forceinline__ void store_acc_row16(uint32_t taddr, __nv_bfloat16* dst, float mul,
                                                bool valid, int c_begin, int c_end, int lane,
                                                const void* base, size_t bytes, int* status) {
  const int pb = lane & 1;
  const bool partner_valid = __shfl_xor_sync(0xffffffffu, valid, 1);
  const bool even_valid = pb ? partner_valid : valid, odd_valid = pb ? valid : partner_valid;
  __nv_bfloat16* even_row = dst - pb * D;
  const bool v8 = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;
#pragma unroll 1
  for (int c = c_begin; c < c_end; c += 32) {
    uint32_t w[16];
    {
      uint32_t a[32];
      tmem_ld32(taddr + c, a);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16x2(__uint_as_float(a[2 * i]) * mul, __uint_as_float(a[2 * i + 1]) * mul);
    }
    pair_transpose8(w, lane);
    __nv_bfloat16* e = even_row + c + 16 * pb;
    __nv_bfloat16* o = even_row + D + c + 16 * pb;
    if (even_valid && store_in_bounds(e, 32, base, bytes, status)) st_global_8w(e, &w[0], v8);
    if (odd_valid && store_in_bounds(o, 32, base, bytes, status)) st_global_8w(o, &w[8], v8);
  }
}

// ------------------------------------------------------------------ dK / dV
template <int D, Mask WIN = kNoWindow>
__global__ void __launch_bounds__(kBwdThreads, 1)
    bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ CUtensorMap tmDO, const BwdWindowParams p) {
  using C = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTile;
  uint8_t* sRing = smem + C::kFixed;  // stage st: Q at +0, dO at +kTile
  float* sScal = reinterpret_cast<float*>(smem + C::kFixed + C::kRing);  // [st][2][128]
  BwdBars* bars = reinterpret_cast<BwdBars*>(smem + C::kFixed + C::kRing + C::kScalars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Work: key tile n of KV head (b, g); CTAs are numbered n-major so the
  // largest work (low n under a causal mask) is scheduled first.
  const int BH = p.B * p.Hkv;
  int n;
  if constexpr (WIN)
    n = p.by_kv_planes.div(blockIdx.x);
  else
    n = blockIdx.x / BH;
  const int bg = blockIdx.x - n * BH;
  int part = -1;  // windowed: this CTA's part of a split tile
  if constexpr (WIN) {
    if (n < p.split_tiles * p.parts) {
      const int tile = p.by_parts.div(n);
      part = n - tile * p.parts;
      n = tile;
    } else {
      n -= p.split_tiles * (p.parts - 1);
    }
  }
  const int group = p.Hq / p.Hkv;
  const int mtiles = (p.Sq + 127) / 128;
  int m0 = min(first_q_tile(p, n), mtiles);
  int per_head = mtiles - m0;
  if constexpr (WIN) {
    const QTileRange qr = window_q_tiles(p.Sq, p.Sk, p.window, p.sinks, n);
    m0 = qr.m0;
    per_head = max(qr.m1 - qr.m0, 0);
  }
  int nsteps = group * per_head;
  int s_base = 0;  // first of the tile's steps that this CTA takes
  if constexpr (WIN) {
    if (part >= 0) {
      const int chunk = p.by_parts.div(nsteps + p.parts - 1);
      s_base = min(part * chunk, nsteps);
      nsteps = min(chunk, nsteps - s_base);
    }
  }

  if (threadIdx.x == 0) {
    mbar_init(&bars->fixed_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->p_ready, kGradThreads / 32);  // one arrival per gradient warp
    mbar_init(&bars->ds_full, kGradThreads / 32);
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kBwdMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  bool ok = true;
  // Windowed: a dependent of dQ, which leaves Delta.  Only the gradient warps, which read
  // it, wait for dQ: the first products run beside dQ's end.  (The call's inputs are
  // complete: dQ let its dependents start after its own wait for what came before.)
  if constexpr (WIN) grid_launch_dependents();

  if (warp == kBwdLoadWarp) {
    if (nsteps > 0) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&bars->fixed_full, 2 * C::kTile);
        load_tile<D>(sK, &tmK, &bars->fixed_full, 128 * n, bg);
        load_tile<D>(sV, &tmV, &bars->fixed_full, 128 * n, bg);
      }
      __syncwarp();
      for (int s = 0; s < nsteps && ok; ++s) {
        const int st = s % kStages;
        bool good = true;
        if (s >= kStages) good = bwd_wait(&bars->empty[st], ((s / kStages) - 1) & 1, bars);
        const int head = bg * group + (s_base + s) / per_head;  // b * Hq + h
        const int m = m0 + (s_base + s) % per_head;
        uint8_t* dst = sRing + st * 2 * C::kTile;
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars->full[st], 2 * C::kTile);
          load_tile<D>(dst, &tmQ, &bars->full[st], 128 * m, head);
          load_tile<D>(dst + C::kTile, &tmDO, &bars->full[st], 128 * m, head);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, good);
      }
      if (!ok) bwd_record(p.status);
      for (int s = max(0, nsteps - kStages); s < nsteps; ++s)
        (void)mbar_wait(&bars->full[s % kStages], (s / kStages) & 1);
      (void)mbar_wait(&bars->fixed_full, 0);
    }
  } else if (warp == kBwdMmaWarp) {
    if (nsteps > 0) {
      ok = bwd_wait_w(&bars->fixed_full, 0, bars);
      if constexpr (WIN == kUnseen) {
        const int unseen = unseen_end(p.Sq, p.Sk, p.window);
        zero_unseen_rows<D>(sK, 128 * n, p.sinks, unseen, lane);
        zero_unseen_rows<D>(sV, 128 * n, p.sinks, unseen, lane);
      }
      const uint32_t k_addr = smem_u32(sK), v_addr = smem_u32(sV);
      // S^T = K Q^T of step s (its Q/dO stage must have landed) and dP^T = V dO^T.
      auto issue_s = [&](int s) -> bool {  // this lane's wait outcome
        const int st = s % kStages;
        const bool got = bwd_wait(&bars->full[st], (s / kStages) & 1, bars);
        mma_ss_tile<D>(tmem, C::kColS, k_addr, smem_u32(sRing + st * 2 * C::kTile));
        tc_commit_w(&bars->s_full);
        return got;
      };
      auto issue_dp = [&](int s) {  // after issue_s(s), which waited for the stage
        const int st = s % kStages;
        mma_ss_tile<D>(tmem, C::kColDP, v_addr, smem_u32(sRing + st * 2 * C::kTile) + C::kTile);
        tc_commit_w(&bars->dp_full);
      };
      if (ok) {
        const bool got = issue_s(0);
        issue_dp(0);
        ok = __all_sync(0xffffffffu, got);
      }
      // One vote after the loop: after a timed-out wait the abort flag makes
      // every later wait give up after a few polls (operands stay in bounds).
      bool good = true;
      for (int s = 0; s < nsteps && ok; ++s) {
        const int st = s % kStages;
        const uint32_t q_addr = smem_u32(sRing + st * 2 * C::kTile);
        const uint32_t do_addr = q_addr + C::kTile;
        // dV += P^T dO as soon as P^T is in TMEM (B operands MN-major: their
        // rows are the K dimension), then at once S^T(s+1): it overwrites P^T(s)
        // only after dV has read it (same-thread tcgen05 order), and the
        // gradient warps need S^T(s) no more; they compute dS^T(s) meanwhile.
        good &= bwd_wait(&bars->p_ready, s & 1, bars);
        tc_fence_after();
        mma_ts_acc<D>(tmem, C::kColA1, C::kColS, do_addr, s == 0);
        if (s + 1 < nsteps) good &= issue_s(s + 1);
        // dK += dS^T Q once dS^T is in TMEM; then the stage is free, and
        // dP^T(s+1) may overwrite dS^T(s).
        good &= bwd_wait(&bars->ds_full, s & 1, bars);
        tc_fence_after();
        mma_ts_acc<D>(tmem, C::kColA0, C::kColDP, q_addr, s == 0);
        tc_commit_w(&bars->empty[st]);
        if (s + 1 < nsteps) issue_dp(s + 1);
      }
      ok = ok && __all_sync(0xffffffffu, good);
      if (ok) tc_commit_w(&bars->acc_full);
      if (!ok) bwd_record(p.status);
      tc_commit_w(&bars->mma_done);
      (void)mbar_wait(&bars->mma_done, 0);
    }
  } else {
    // Gradient warps: thread r owns key 128n + r (TMEM lane r); warpgroup
    // `half` handles columns [64*half, 64*half + 64).
    const int quad = warp & 3;
    const int half = warp >> 2;
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    const int key = 128 * n + r;
    const bool key_valid = key < p.Sk;
    // LSE and Delta of a step's 64 columns (2 per lane), loaded one step ahead:
    // the loads stay in flight through the previous step's work (volatile asm
    // keeps them ahead of that work's tcgen05 operations).  Rows past Sq load
    // row Sq - 1 (in bounds) and are zeroed when staged.
    float pre_l[2] = {0.f, 0.f}, pre_d[2] = {0.f, 0.f};
    // The step being fetched: its query tile, and its head as b * Hq + h (counted, as a
    // division a step costs 0.5 to 3 % of a windowed backward).
    int pre_m = 0, next_m = m0, next_head = bg * group;
    if (s_base > 0) {
      next_m += s_base % per_head;
      next_head += s_base / per_head;
    }
    auto fetch = [&]() {
      const size_t base = static_cast<size_t>(next_head) * p.Sq;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = min(128 * next_m + 64 * half + 32 * u + lane, p.Sq - 1);
        pre_l[u] = ld_nc_f32(p.lse + base + row);
        pre_d[u] = ld_nc_f32(p.delta + base + row);
      }
      pre_m = next_m;
      if (++next_m == m0 + per_head) {
        next_m = m0;
        ++next_head;
      }
    };
    if constexpr (WIN) grid_dependency_wait();
    if (nsteps > 0) fetch();
    for (int s = 0; s < nsteps && ok; ++s) {
      const int m = pre_m;
      // This step's -LSE (log2 domain) and -Delta for the warpgroup's 64
      // columns, in the warp's own buffer (no cross-warp barrier, so an
      // aborting warp cannot strand others); read back as broadcast float4.
      float* nl2 = sScal + warp * 128;
      float* ndl = nl2 + 64;
      __syncwarp();  // every lane is done with the previous step's values
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool rv = 128 * m + 64 * half + 32 * u + lane < p.Sq;
        nl2[32 * u + lane] = rv ? -pre_l[u] * kLog2e : 0.f;
        ndl[32 * u + lane] = rv ? -pre_d[u] : 0.f;
      }
      __syncwarp();
      if (s + 1 < nsteps) fetch();
      // Visible columns (query rows 128m + col) of this key: [c_lo, c_hi) --
      // row >= key - (Sk - Sq) under the causal mask, row < Sq.
      const int row_lo = WIN || p.causal ? key - (p.Sk - p.Sq) : -0x40000000;
      const int c_lo = max(row_lo - 128 * m, 0);
      int c_hi = key_valid ? min(p.Sq - 128 * m, 128) : 0;
      // Windowed: rows up to the last whose window reaches the key, sinks to the end.
      if (WIN && key >= p.sinks) c_hi = min(c_hi, row_lo + p.window - 128 * m);
      const bool need_mask = __any_sync(0xffffffffu, c_lo > 64 * half || c_hi < 64 * half + 64);
      ok = __all_sync(0xffffffffu, bwd_wait(&bars->s_full, s & 1, bars));
      if (!ok) break;
      tc_fence_after();
      // P^T for this warpgroup's 64 columns: kept in registers for dS^T and
      // written (bf16) into its own half of the S^T columns.
      const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2);
      float pv[64];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int c = 2 * half + cc;
        const uint32_t bits = WIN ? window_bits(c_lo - 32 * c, c_hi - 32 * c, 0) : 0u;
        uint32_t sr[32];
        tmem_ld32(tmem + lane_addr + C::kColS + 32 * c, sr);
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 nl = *reinterpret_cast<const float4*>(nl2 + 32 * cc + e);
          float x[4];
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sl2,
                           f2_pack(nl.x, nl.y)),
                    x[0], x[1]);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[e + 2]), __uint_as_float(sr[e + 3])), sl2,
                           f2_pack(nl.z, nl.w)),
                    x[2], x[3]);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float pu = ex2(x[u]);
            if (need_mask) {
              const int col = 32 * c + e + u;
              if constexpr (WIN)
                pu = (bits >> (e + u) & 1u) ? pu : 0.f;
              else
                pu = (col >= c_lo && col < c_hi) ? pu : 0.f;
            }
            pv[32 * cc + e + u] = pu;
          }
          pk[e >> 1] = pack_bf16x2(pv[32 * cc + e], pv[32 * cc + e + 1]);
          pk[(e >> 1) + 1] = pack_bf16x2(pv[32 * cc + e + 2], pv[32 * cc + e + 3]);
        }
        tmem_st16(tmem + lane_addr + C::kColS + 64 * half + 16 * cc, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_warp(&bars->p_ready);
      // dS^T = P^T (dP^T - Delta), into this warpgroup's half of the dP^T columns.
      ok = __all_sync(0xffffffffu, bwd_wait(&bars->dp_full, s & 1, bars));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int c = 2 * half + cc;
        uint32_t dr[32];
        tmem_ld32(tmem + lane_addr + C::kColDP + 32 * c, dr);
        uint32_t dk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 nd = *reinterpret_cast<const float4*>(ndl + 32 * cc + e);
          float d[4];
          f2_unpack(f2_mul(f2_pack(pv[32 * cc + e], pv[32 * cc + e + 1]),
                           f2_add(f2_pack(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1])),
                                  f2_pack(nd.x, nd.y))),
                    d[0], d[1]);
          f2_unpack(f2_mul(f2_pack(pv[32 * cc + e + 2], pv[32 * cc + e + 3]),
                           f2_add(f2_pack(__uint_as_float(dr[e + 2]), __uint_as_float(dr[e + 3])),
                                  f2_pack(nd.z, nd.w))),
                    d[2], d[3]);
          dk[e >> 1] = pack_bf16x2(d[0], d[1]);
          dk[(e >> 1) + 1] = pack_bf16x2(d[2], d[3]);
        }
        tmem_st16(tmem + lane_addr + C::kColDP + 64 * half + 16 * cc, dk);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_warp(&bars->ds_full);
    }
    if (ok) {
      const size_t kv_row = (static_cast<size_t>(bg) * p.Sk + key) * D;
      float* dk_row = p.out0 + kv_row;
      float* dv_row = p.out1 + kv_row;
      const size_t kv_bytes =
          static_cast<size_t>(p.B) * p.Hkv * p.Sk * D * (WIN ? sizeof(__nv_bfloat16) : sizeof(float));
      if constexpr (WIN) {
        __nv_bfloat16* dk16 = reinterpret_cast<__nv_bfloat16*>(p.out0) + kv_row;
        __nv_bfloat16* dv16 = reinterpret_cast<__nv_bfloat16*>(p.out1) + kv_row;
        if (part >= 0) {
          // Partials of every row of the tile (those past Sk are never read).
          const size_t plane = static_cast<size_t>(p.split_tiles) * BH * 128 * D;
          const size_t part_bytes = 2 * p.parts * plane * sizeof(float);
          float* dk_part = p.partials + part * plane +
                           (static_cast<size_t>(n * BH + bg) * 128 + r) * D;
          float* dv_part = dk_part + p.parts * plane;
          if (nsteps == 0) {
            for (int c = half * D / 2; c < (half + 1) * D / 2; c += 4) {
              *reinterpret_cast<float4*>(dk_part + c) = make_float4(0.f, 0.f, 0.f, 0.f);
              *reinterpret_cast<float4*>(dv_part + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
          } else {
            ok = __all_sync(0xffffffffu, bwd_wait(&bars->acc_full, 0, bars));
            if (ok) {
              tc_fence_after();
              store_acc_row<D>(tmem + lane_addr + C::kColA0, dk_part, p.scale, true, half * D / 2,
                               (half + 1) * D / 2, lane, p.partials, part_bytes, p.status);
              store_acc_row<D>(tmem + lane_addr + C::kColA1, dv_part, 1.f, true, half * D / 2,
                               (half + 1) * D / 2, lane, p.partials, part_bytes, p.status);
            }
          }
        } else if (nsteps == 0) {
          if (key_valid && store_in_bounds(dk16, D * 2, p.out0, kv_bytes, p.status) &&
              store_in_bounds(dv16, D * 2, p.out1, kv_bytes, p.status)) {
            for (int c = half * D / 2; c < (half + 1) * D / 2; c += 8) {
              *reinterpret_cast<uint4*>(dk16 + c) = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(dv16 + c) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        } else {
          ok = __all_sync(0xffffffffu, bwd_wait(&bars->acc_full, 0, bars));
          if (ok) {
            tc_fence_after();
            store_acc_row16<D>(tmem + lane_addr + C::kColA0, dk16, p.scale, key_valid,
                               half * D / 2, (half + 1) * D / 2, lane, p.out0, kv_bytes, p.status);
            store_acc_row16<D>(tmem + lane_addr + C::kColA1, dv16, 1.f, key_valid, half * D / 2,
                               (half + 1) * D / 2, lane, p.out1, kv_bytes, p.status);
          }
        }
      } else if (nsteps == 0) {
        // No query row sees these keys: their gradients are zero.
        if (key_valid && store_in_bounds(dk_row, D * 4, p.out0, kv_bytes, p.status) &&
            store_in_bounds(dv_row, D * 4, p.out1, kv_bytes, p.status)) {
          for (int c = half * D / 2; c < (half + 1) * D / 2; c += 4) {
            *reinterpret_cast<float4*>(dk_row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(dv_row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      } else {
        ok = __all_sync(0xffffffffu, bwd_wait(&bars->acc_full, 0, bars));
        if (ok) {
          tc_fence_after();
          store_acc_row<D>(tmem + lane_addr + C::kColA0, dk_row, p.scale, key_valid,
                           half * D / 2, (half + 1) * D / 2, lane, p.out0, kv_bytes, p.status);
          store_acc_row<D>(tmem + lane_addr + C::kColA1, dv_row, 1.f, key_valid,
                           half * D / 2, (half + 1) * D / 2, lane, p.out1, kv_bytes, p.status);
        }
      }
    }
    if (!ok) bwd_record(p.status);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kBwdMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dK and dV of the split key tiles: the sum of their parts, in order, rounded once.
// A thread per four dims of a row.
template <int D>
__global__ void __launch_bounds__(256)
    bwd_sum_parts_kernel(const float* __restrict__ partials, __nv_bfloat16* __restrict__ dk,
                         __nv_bfloat16* __restrict__ dv, int split_tiles, int parts, int BH,
                         int Sk, int* status) {
  grid_dependency_wait();
  grid_launch_dependents();
  const size_t plane = static_cast<size_t>(split_tiles) * BH * 128 * D;
  const size_t at = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  const int row = static_cast<int>(at / D);  // (tile * BH + bg) * 128 + key of the tile
  const int tile = row / (128 * BH), bg = (row / 128) % BH;
  const int key = 128 * tile + (row & 127);
  if (at >= plane || key >= Sk) return;
  const size_t to = (static_cast<size_t>(bg) * Sk + key) * D + at % D;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float* src = partials + i * parts * plane + at;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < parts; ++q) {
      const float4 y = *reinterpret_cast<const float4*>(src + q * plane);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    __nv_bfloat16* out = i ? dv : dk;
    if (store_in_bounds(out + to, 8, out, static_cast<size_t>(BH) * Sk * D * 2, status))
      *reinterpret_cast<uint2*>(out + to) =
          make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  }
}

// ------------------------------------------------------------------ dQ
// Persistent: min(#query tiles, #SMs) CTAs, each walking the query tiles
// (highest tile first, i.e. longest under a causal mask) in the order c,
// 2G-1-c, 2G+c, ... (G CTAs), which balances a descending cost list.  Across
// its tiles a CTA keeps one TMEM allocation and its barrier phases; the next
// tile's Q and dO load as soon as the current tile's last S and dP products
// are done, and the dQ accumulator alternates between two TMEM buffers so that
// one tile's epilogue overlaps the next tile's products.
__device__ __forceinline__ int dq_tile_index(int round, int cta, int grid) {
  return round * grid + ((round & 1) ? (grid - 1 - cta) : cta);
}

// The KV tiles of query tile m: step s reads tile kv_tile(s), s < nsteps.
template <Mask WIN>
struct DqTiles {
  int nsteps;
  TileRange r;
  __device__ __forceinline__ DqTiles(const DqArgs<WIN>& p, int m) {
    if constexpr (WIN) {
      r = window_kv_tiles(p.Sq, p.Sk, p.window, p.sinks, 128 * m);
      nsteps = r.count();
    } else {
      nsteps = kv_tiles_for(p, m);
    }
  }
  __device__ __forceinline__ int kv_tile(int s) const {
    if constexpr (WIN)
      return r.tile(s);
    else
      return s;
  }
};

template <int D, Mask WIN = kNoWindow>
__global__ void __launch_bounds__(WIN ? kDqWinThreads : kBwdThreads, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmDO, const DqArgs<WIN> p) {
  using C = BwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sDO = smem + C::kTile;
  uint8_t* sK = smem + C::kFixed;                // K ring: kKStages tiles
  uint8_t* sV = sK + kKStages * C::kTile;        // V ring: kVStages tiles
  BwdBars* bars = reinterpret_cast<BwdBars*>(sV + kVStages * C::kTile);
  float* sDelta = reinterpret_cast<float*>(sV + kVStages * C::kTile + C::kBarBytes);  // [2][128]
  float* sPart = sDelta + 2 * 128;                                                        // [128]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Work: query tile m of head (b, h), numbered m-major with the highest m first.
  const int BH = p.B * p.Hq;
  const int mtiles = (p.Sq + 127) / 128;
  const int total = BH * mtiles;
  const int group = p.Hq / p.Hkv;
  // Query tile m of head bh (b * Hq + h) of item idx.
  auto tile_of = [&](int idx, int& m, int& bh) {
    if constexpr (WIN) {
      const int rank = p.by_q_planes.div(idx);
      m = mtiles - 1 - rank;
      bh = idx - rank * BH;
    } else {
      m = mtiles - 1 - idx / BH;
      bh = idx % BH;
    }
  };

  if (threadIdx.x == 0) {
    mbar_init(&bars->fixed_full, 1);  // this tile's Q and dO have landed
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&bars->full_v[s], 1);
      mbar_init(&bars->empty_v[s], 1);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->p_ready, kGradThreads / 32);  // one arrival per gradient warp
    mbar_init(&bars->ds_full, kGradThreads / 32);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->acc_full2[b], 1);
      mbar_init(&bars->acc_free[b], kGradThreads / 32);
      if constexpr (WIN) {
        mbar_init(&bars->delta_full[b], 2);
        mbar_init(&bars->delta_free[b], kGradThreads / 32);
        if (b == 0) {
          mbar_init(&bars->part_full, kGradThreads / 64);
          mbar_init(&bars->total_full, kGradThreads / 64);
        }
      }
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kBwdMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  bool ok = true;
  if constexpr (WIN) {  // launched as a dependent of the kernel before (the forward)
    grid_dependency_wait();
    grid_launch_dependents();
  }

  if (warp == kBwdLoadWarp) {
    uint32_t G = 0;   // first global step of the current tile
    uint32_t gl = 0;  // steps whose K and V copies were issued
    int kt = 0;       // tiles with work so far (Q/dO loads issued)
    for (int rnd = 0; ok; ++rnd) {
      const int idx = dq_tile_index(rnd, blockIdx.x, gridDim.x);
      if (idx >= total) break;
      int m, bh;
      tile_of(idx, m, bh);
      const DqTiles<WIN> tiles(p, m);
      const int nsteps = tiles.nsteps;
      if (nsteps == 0) continue;
      int bkv;  // b * Hkv + KV head
      if constexpr (WIN)
        bkv = p.by_group.div(bh);
      else
        bkv = (bh / p.Hq) * p.Hkv + (bh % p.Hq) / group;
      // Q and dO of this tile once the previous tile's last S and dP are done.
      if (kt > 0 && !(ok = __all_sync(0xffffffffu, bwd_wait(&bars->q_empty, (kt - 1) & 1, bars))))
        break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&bars->fixed_full, 2 * C::kTile);
        load_tile<D>(sQ, &tmQ, &bars->fixed_full, 128 * m, bh);
        load_tile<D>(sDO, &tmDO, &bars->fixed_full, 128 * m, bh);
      }
      __syncwarp();
      ++kt;
      // K(s) and V(s) in use order; K(s) is held until dQ(s), V(s) until dP(s).
      for (int s = 0; s < nsteps && ok; ++s) {
        const uint32_t g = G + s;
        const int sk = g % kKStages, sv = g % kVStages;
        bool good = true;
        if (g >= uint32_t(kKStages))
          good = bwd_wait(&bars->empty[sk], ((g / kKStages) - 1) & 1, bars);
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars->full[sk], C::kTile);
          load_tile<D>(sK + sk * C::kTile, &tmK, &bars->full[sk], 128 * tiles.kv_tile(s), bkv);
        }
        __syncwarp();
        if (g >= uint32_t(kVStages))
          good &= bwd_wait(&bars->empty_v[sv], ((g / kVStages) - 1) & 1, bars);
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars->full_v[sv], C::kTile);
          load_tile<D>(sV + sv * C::kTile, &tmV, &bars->full_v[sv], 128 * tiles.kv_tile(s), bkv);
        }
        __syncwarp();
        gl = g + 1;
        ok = __all_sync(0xffffffffu, good);
      }
      G += nsteps;
    }
    if (!ok) bwd_record(p.status);
    // Every copy this warp issued lands before the CTA can exit (older copies
    // have landed: their slots were released after their use).
    for (uint32_t g = (gl > uint32_t(kKStages) ? gl - kKStages : 0); g < gl; ++g)
      (void)mbar_wait(&bars->full[g % kKStages], (g / kKStages) & 1);
    for (uint32_t g = (gl > uint32_t(kVStages) ? gl - kVStages : 0); g < gl; ++g)
      (void)mbar_wait(&bars->full_v[g % kVStages], (g / kVStages) & 1);
    if (kt > 0) (void)mbar_wait(&bars->fixed_full, (kt - 1) & 1);
  } else if (warp == kBwdMmaWarp) {
    const uint32_t q_addr = smem_u32(sQ), do_addr = smem_u32(sDO);
    const uint32_t k_base = smem_u32(sK), v_base = smem_u32(sV);
    const int unseen = WIN == kUnseen ? unseen_end(p.Sq, p.Sk, p.window) : 0;
    // Step g's products; `tile` is its KV tile.
    auto issue_s = [&](uint32_t g, int tile) -> bool {  // S = Q K^T; this lane's wait outcome
      const int sk = g % kKStages;
      const bool got = bwd_wait(&bars->full[sk], (g / kKStages) & 1, bars);
      if constexpr (WIN == kUnseen)
        zero_unseen_rows<D>(sK + sk * C::kTile, 128 * tile, p.sinks, unseen, lane);
      mma_ss_tile<D>(tmem, C::kColS, q_addr, k_base + sk * C::kTile);
      tc_commit_w(&bars->s_full);
      return got;
    };
    auto issue_dp = [&](uint32_t g, int tile) -> bool {  // dP = dO V^T; V(g) is free afterwards
      const int sv = g % kVStages;
      const bool got = bwd_wait(&bars->full_v[sv], (g / kVStages) & 1, bars);
      if constexpr (WIN == kUnseen)
        zero_unseen_rows<D>(sV + sv * C::kTile, 128 * tile, p.sinks, unseen, lane);
      mma_ss_tile<D>(tmem, C::kColDP, do_addr, v_base + sv * C::kTile);
      tc_commit_w(&bars->dp_full);
      tc_commit_w(&bars->empty_v[sv]);
      return got;
    };
    uint32_t G = 0;  // first global step of the current tile
    int kt = 0;      // tiles with work so far
    bool good = true;  // one vote per tile, as in the dK/dV kernel's loop
    for (int rnd = 0; ok; ++rnd) {
      const int idx = dq_tile_index(rnd, blockIdx.x, gridDim.x);
      if (idx >= total) break;
      int m, bh;
      tile_of(idx, m, bh);
      const DqTiles<WIN> tiles(p, m);
      const int nsteps = tiles.nsteps;
      if (nsteps == 0) continue;
      const int buf = kt & 1;
      const uint32_t acc_col = buf ? C::kColA1 : C::kColA0;
      good &= bwd_wait(&bars->fixed_full, kt & 1, bars);  // this tile's Q and dO
      // The epilogue of tile kt-2 has read this accumulator buffer.
      if (kt >= 2) good &= bwd_wait(&bars->acc_free[buf], ((kt >> 1) - 1) & 1, bars);
      // S(G) overwrites the S columns once the previous step's S has been read.
      if (G > 0) good &= bwd_wait(&bars->p_ready, (G - 1) & 1, bars);
      tc_fence_after();
      good &= issue_s(G, tiles.kv_tile(0));
      good &= issue_dp(G, tiles.kv_tile(0));
      if (nsteps == 1) tc_commit_w(&bars->q_empty);  // last S and dP of the tile issued
      for (int s = 0; s < nsteps; ++s) {
        const uint32_t g = G + s;
        // S(g+1) as soon as the gradient warps have read S(g) ...
        if (s + 1 < nsteps) {
          good &= bwd_wait(&bars->p_ready, g & 1, bars);
          tc_fence_after();
          good &= issue_s(g + 1, tiles.kv_tile(s + 1));
        }
        // ... dQ += dS K once dS(g) is in TMEM (K MN-major: its rows are the K dim) ...
        good &= bwd_wait(&bars->ds_full, g & 1, bars);
        tc_fence_after();
        mma_ts_acc<D>(tmem, acc_col, C::kColDP, k_base + (g % kKStages) * C::kTile, s == 0);
        tc_commit_w(&bars->empty[g % kKStages]);
        // ... then dP(g+1), which overwrites dS(g) after dQ has read it.  After
        // the tile's last dP, Q and dO may be replaced by the next tile's.
        if (s + 1 < nsteps) {
          good &= issue_dp(g + 1, tiles.kv_tile(s + 1));
          if (s + 2 == nsteps) tc_commit_w(&bars->q_empty);
        }
      }
      tc_commit_w(&bars->acc_full2[buf]);
      G += nsteps;
      ++kt;
      ok = __all_sync(0xffffffffu, good);
    }
    if (!ok) bwd_record(p.status);
    // Every MMA this warp issued completes before TMEM is released.
    tc_commit_w(&bars->mma_done);
    (void)mbar_wait(&bars->mma_done, 0);
  } else if (WIN && warp >= kDqDeltaWarp) {
    if constexpr (WIN) {
      // Delta, a tile or two ahead of the gradient warps: 64 rows a warp, from global
      // memory, to shared memory for them and to delta_out for dK/dV.  (By the gradient
      // warps themselves, at a tile's start, the loads' latency cost more than a kernel
      // of its own for Delta: 8192 rows, 32 heads, D = 128: 561 against 552 us a step.)
      int kt = 0;
      for (int rnd = 0; ok; ++rnd) {
        const int idx = dq_tile_index(rnd, blockIdx.x, gridDim.x);
        if (idx >= total) break;
        int m, bh;
        tile_of(idx, m, bh);
        const int nsteps = DqTiles<WIN>(p, m).nsteps;
        const int buf = kt & 1;
        if (nsteps > 0 && kt >= 2) {
          ok = __all_sync(0xffffffffu, bwd_wait(&bars->delta_free[buf], ((kt >> 1) - 1) & 1, bars));
          if (!ok) break;
        }
  #pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int r = 64 * (warp - kDqDeltaWarp) + 32 * i;
          const long long row0 = static_cast<long long>(bh) * p.Sq + 128 * m + r;
          const float dlt =
              warp_delta<D>(p.o, p.dout, row0, static_cast<long long>(BH) * p.Sq, lane);
          if ((nsteps == 0 || nsteps > kExactDeltaSteps) && 128 * m + r + lane < p.Sq)
            p.delta_out[row0 + lane] = dlt;
          if (nsteps > 0) sDelta[128 * buf + r + lane] = dlt;
        }
        if (nsteps > 0) {
          mbar_arrive_warp(&bars->delta_full[buf]);
          ++kt;
        }
      }
    }
    if (!ok) bwd_record(p.status);
  } else {
    // Gradient warps: thread r owns query row 128m + r (TMEM lane r); warpgroup
    // `half` handles keys [64*half, 64*half + 64) of each tile.
    const int quad = warp & 3;
    const int half = warp >> 2;
    const int r = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2);
    const size_t q_bytes =
        static_cast<size_t>(p.B) * p.Hq * p.Sq * D * (WIN ? sizeof(__nv_bfloat16) : sizeof(float));
    uint32_t G = 0;  // first global step of the current tile
    int kt = 0;      // tiles with work so far
    int exact_tiles = 0;  // windowed: those whose Delta was added up here
    for (int rnd = 0; ok; ++rnd) {
      const int idx = dq_tile_index(rnd, blockIdx.x, gridDim.x);
      if (idx >= total) break;
      int m, bh;
      tile_of(idx, m, bh);
      const DqTiles<WIN> tiles(p, m);
      const int nsteps = tiles.nsteps;
      const int row = 128 * m + r;
      const bool row_valid = row < p.Sq;
      float* dq_row = p.out0 + (static_cast<size_t>(bh) * p.Sq + row) * D;
      __nv_bfloat16* dq16 =
          reinterpret_cast<__nv_bfloat16*>(p.out0) + (static_cast<size_t>(bh) * p.Sq + row) * D;
      if (nsteps == 0) {
        // No key is visible to these rows: their gradient is zero.
        if constexpr (WIN) {
          if (row_valid && store_in_bounds(dq16, D * 2, p.out0, q_bytes, p.status))
            for (int c = half * D / 2; c < (half + 1) * D / 2; c += 8)
              *reinterpret_cast<uint4*>(dq16 + c) = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        if (row_valid && store_in_bounds(dq_row, D * 4, p.out0, q_bytes, p.status))
          for (int c = half * D / 2; c < (half + 1) * D / 2; c += 4)
            *reinterpret_cast<float4*>(dq_row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        continue;
      }
      const float lse2 = row_valid ? __ldg(p.lse + static_cast<size_t>(bh) * p.Sq + row) * kLog2e
                                   : 0.f;
      float dlt = 0.f;
      if constexpr (WIN) {
        const int buf = kt & 1;
        ok = __all_sync(0xffffffffu, bwd_wait(&bars->delta_full[buf], (kt >> 1) & 1, bars));
        if (!ok) break;
        dlt = row_valid ? sDelta[128 * buf + r] : 0.f;
        mbar_arrive_warp(&bars->delta_free[buf]);
      } else {
        dlt = row_valid ? __ldg(p.delta + static_cast<size_t>(bh) * p.Sq + row) : 0.f;
      }
      const uint64_t nl2 = f2_pack(-lse2, -lse2);
      uint64_t ndl = f2_pack(-dlt, -dlt);
      // Delta from a bf16 O is off by O's rounding (and P's in it), which a row of few
      // keys shows: at a window of 8 dQ and dK are 2.7e-3 off, 1.63 times what their own
      // rounding alone would make, and still 1.5 times at 64.  So where a tile has few
      // steps (and windows are that short) sum_j P dP, which is Delta, is added up on
      // the way: dK/dV uses it, and here the last step, which holds most keys of the
      // tile's later rows.  (2.4e-3 then, at each window.)  The steps before it, which
      // hold most keys of its first rows, keep the Delta from O.
      const bool exact = WIN && nsteps <= kExactDeltaSteps;
      uint64_t p_dp = f2_pack(0.f, 0.f);
      const int key_hi = WIN || p.causal ? min(p.Sk - 1, row + p.Sk - p.Sq) : p.Sk - 1;
      const int win_lo = row + p.Sk - p.Sq - p.window + 1;  // windowed: the window's first key
      for (int s = 0; s < nsteps && ok; ++s) {
        const uint32_t g = G + s;
        ok = __all_sync(0xffffffffu, bwd_wait(&bars->s_full, g & 1, bars));
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld32(tmem + lane_addr + C::kColS + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(sr));
        tmem_ld32(tmem + lane_addr + C::kColS + 64 * half + 32,
                  *reinterpret_cast<uint32_t(*)[32]>(sr + 32));
        // S(g) is in registers: its columns may be overwritten by S(g+1).
        tc_fence_before();
        mbar_arrive_warp(&bars->p_ready);
        // Keys 128s + 64*half + e are visible for e < n_vis (causal limit, Sk).
        const int key0 = 128 * tiles.kv_tile(s) + 64 * half;
        int n_vis;  // (Written as in each form it measured best.)
        if constexpr (WIN)
          n_vis = row_valid ? min(max(key_hi - key0 + 1, 0), 64) : 0;
        else
          n_vis = row_valid ? min(max(key_hi - (128 * s + 64 * half) + 1, 0), 64) : 0;
        // Windowed: of those, only e < n_sink or e >= n_skip.
        const int n_sink = p.sinks - key0, n_skip = win_lo - key0;
        const bool need_mask =
            __any_sync(0xffffffffu, n_vis < 64 || (WIN && n_skip > 0 && n_sink < 64));
        uint32_t bits[2] = {0u, 0u};
        if constexpr (WIN) {
          bits[0] = window_bits(n_skip, n_vis, n_sink);
          bits[1] = window_bits(n_skip - 32, n_vis - 32, n_sink - 32);
        }
        float pv[64];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[e]), __uint_as_float(sr[e + 1])), sl2, nl2),
                    x0, x1);
          float p0 = ex2(x0), p1 = ex2(x1);
          if (need_mask) {
            if constexpr (WIN) {
              p0 = (bits[e >> 5] >> (e & 31) & 1u) ? p0 : 0.f;
              p1 = (bits[e >> 5] >> ((e & 31) + 1) & 1u) ? p1 : 0.f;
            } else {
              p0 = e < n_vis ? p0 : 0.f;
              p1 = e + 1 < n_vis ? p1 : 0.f;
            }
          }
          pv[e] = p0;
          pv[e + 1] = p1;
        }
        ok = __all_sync(0xffffffffu, bwd_wait(&bars->dp_full, g & 1, bars));
        if (!ok) break;
        tc_fence_after();
        if constexpr (WIN) {
          if (exact) {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              uint32_t dr[32];
              tmem_ld32(tmem + lane_addr + C::kColDP + 64 * half + 32 * cc, dr);
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                p_dp = f2_fma(f2_pack(pv[32 * cc + e], pv[32 * cc + e + 1]),
                              f2_pack(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1])), p_dp);
            }
            if (s + 1 == nsteps) {
              // The two warpgroups' halves of the sum: 4-7 to 0-3, the total back.
              float a, b;
              f2_unpack(p_dp, a, b);
              dlt = a + b;
              if (half == 1) {
                sPart[r] = dlt;
                mbar_arrive_warp(&bars->part_full);
                ok = __all_sync(0xffffffffu, bwd_wait(&bars->total_full, exact_tiles & 1, bars));
                if (!ok) break;
                dlt = sPart[r];
              } else {
                ok = __all_sync(0xffffffffu, bwd_wait(&bars->part_full, exact_tiles & 1, bars));
                if (!ok) break;
                dlt += sPart[r];
                sPart[r] = dlt;
                mbar_arrive_warp(&bars->total_full);
                if (row_valid) p.delta_out[static_cast<size_t>(bh) * p.Sq + row] = dlt;
              }
              ++exact_tiles;
              ndl = f2_pack(-dlt, -dlt);
            }
          }
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t dr[32];
          tmem_ld32(tmem + lane_addr + C::kColDP + 64 * half + 32 * cc, dr);
          uint32_t dk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float d0, d1;
            f2_unpack(f2_mul(f2_pack(pv[32 * cc + e], pv[32 * cc + e + 1]),
                             f2_add(f2_pack(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1])),
                                    ndl)),
                      d0, d1);
            dk[e >> 1] = pack_bf16x2(d0, d1);
          }
          tmem_st16(tmem + lane_addr + C::kColDP + 64 * half + 16 * cc, dk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars->ds_full);
      }
      if (!ok) break;
      // Epilogue: dQ * scale from this tile's accumulator buffer, which the
      // MMA warp may reuse for tile kt+2 once every gradient warp has read it.
      const int buf = kt & 1;
      ok = __all_sync(0xffffffffu, bwd_wait(&bars->acc_full2[buf], (kt >> 1) & 1, bars));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + lane_addr + (buf ? C::kColA1 : C::kColA0);
      if constexpr (WIN)
        store_acc_row16<D>(acc, dq16, p.scale, row_valid, half * D / 2, (half + 1) * D / 2, lane,
                           p.out0, q_bytes, p.status);
      else
        store_acc_row<D>(acc, dq_row, p.scale, row_valid, half * D / 2, (half + 1) * D / 2, lane,
                         p.out0, q_bytes, p.status);
      tc_fence_before();
      mbar_arrive_warp(&bars->acc_free[buf]);
      G += nsteps;
      ++kt;
    }
    if (!ok) bwd_record(p.status);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kBwdMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The sink tiles' parts (see BwdWindowParams).  A key tile with sinks is seen by every
// later row, group * ceil(Sq/128) steps, where the others take about group *
// (window/128 + 2): on one CTA it outlasts all of them (8192 rows, window 1024, 32/8
// heads: 432 us for dK/dV, of which 0.4 of the CTAs' time was idle).  It is cut into
// parts of at least a common tile's steps and half an SM's share of all steps, below
// which finer parts balance no better.  At most 32 (the sum's loop).
struct SinkSplit {
  int tiles, parts;
};
SinkSplit sink_split(int B, int Hq, int Hkv, int Sq, int Sk, int window, int sinks) {
  const long long mtiles = (Sq + 127) / 128, ntiles = (Sk + 127) / 128;
  const long long tiles = (sinks + 127) / 128;
  const long long reach = window / 128 + 2;
  const long long common = reach < mtiles ? reach : mtiles, group = Hq / Hkv;
  const long long share =
      group * B * Hkv * ((ntiles - tiles) * common + tiles * mtiles) / (2 * sm_count());
  const long long least = group * common > share ? group * common : share;
  const long long parts = tiles == 0 ? 1 : (group * mtiles + least - 1) / least;
  if (parts <= 1) return {0, 1};
  return {static_cast<int>(tiles), static_cast<int>(parts < 32 ? parts : 32)};
}

// o, dq, dk and dv are fp32, or bf16 in the windowed form (window > 0), whose
// `delta` is followed by the partials of the split sink tiles.
template <int D, Mask WIN>
cudaError_t launch_bwd_impl(const void* q, const void* k, const void* v, const void* o,
                            const float* lse, const void* dout, void* dq, void* dk, void* dv,
                            float* delta, int B, int Hq, int Hkv, int Sq, int Sk, int causal,
                            int window, int sinks, float scale, cudaStream_t stream, int* status) {
  using C = BwdCfg<D>;
  cudaError_t e = cudaSuccess;
  if constexpr (!WIN) {
    const int rows = B * Hq * Sq;
    bwd_delta_kernel<D><<<(rows + 7) / 8, 256, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(dout), static_cast<const float*>(o), delta, rows);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  CUtensorMap tmQ, tmK, tmV, tmDO;
  if (!encode_bf16_map(&tmQ, q, D, Sq, B * Hq, 128) ||
      !encode_bf16_map(&tmK, k, D, Sk, B * Hkv, 128) ||
      !encode_bf16_map(&tmV, v, D, Sk, B * Hkv, 128) ||
      !encode_bf16_map(&tmDO, dout, D, Sq, B * Hq, 128))
    return cudaErrorInvalidValue;
  if ((e = ensure_smem_attr(reinterpret_cast<const void*>(bwd_dkdv_kernel<D, WIN>),
                            static_cast<int>(C::kSmem))) != cudaSuccess)
    return e;
  if ((e = ensure_smem_attr(reinterpret_cast<const void*>(bwd_dq_kernel<D, WIN>),
                            static_cast<int>(C::kSmemDq + (WIN ? kDqDeltaBytes : 0)))) !=
      cudaSuccess)
    return e;
  BwdWindowParams p = {};
  p.lse = lse;
  p.delta = delta;
  p.status = status;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Sq = Sq;
  p.Sk = Sk;
  p.causal = causal;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  const int q_tiles = B * Hq * ((Sq + 127) / 128);
  const int q_ctas = q_tiles < sm_count() ? q_tiles : sm_count();
  const int kv_tiles = (Sk + 127) / 128;
  if constexpr (WIN) {
    // dQ first (it computes Delta), each kernel the programmatic dependent of the last.
    const SinkSplit split = sink_split(B, Hq, Hkv, Sq, Sk, window, sinks);
    p.window = window;
    p.sinks = sinks;
    p.o = static_cast<const __nv_bfloat16*>(o);
    p.dout = static_cast<const __nv_bfloat16*>(dout);
    p.delta_out = delta;
    p.split_tiles = split.tiles;
    p.parts = split.parts;
    p.partials = delta + window_bwd_delta_floats(B, Hq, Sq);
    p.by_q_planes = FixedDiv(B * Hq);
    p.by_kv_planes = FixedDiv(B * Hkv);
    p.by_group = FixedDiv(Hq / Hkv);
    p.by_parts = FixedDiv(p.parts);
    p.out0 = static_cast<float*>(dq);
    p.out1 = nullptr;
    if ((e = launch_programmatic(bwd_dq_kernel<D, WIN>, dim3(q_ctas), dim3(kDqWinThreads),
                                 C::kSmemDq + kDqDeltaBytes, stream, tmQ, tmK, tmV, tmDO, p)) !=
        cudaSuccess)
      return e;
    p.out0 = static_cast<float*>(dk);
    p.out1 = static_cast<float*>(dv);
    const int kv_ctas = B * Hkv * (kv_tiles + p.split_tiles * (p.parts - 1));
    if ((e = launch_programmatic(bwd_dkdv_kernel<D, WIN>, dim3(kv_ctas), dim3(kBwdThreads),
                                 C::kSmem, stream, tmQ, tmK, tmV, tmDO, p)) != cudaSuccess)
      return e;
    if (p.split_tiles == 0) return cudaSuccess;
    const size_t vecs = static_cast<size_t>(p.split_tiles) * B * Hkv * 128 * (D / 4);
    return launch_programmatic(bwd_sum_parts_kernel<D>,
                               dim3(static_cast<unsigned>((vecs + 255) / 256)), dim3(256), 0,
                               stream, p.partials, static_cast<__nv_bfloat16*>(dk),
                               static_cast<__nv_bfloat16*>(dv), p.split_tiles, p.parts, B * Hkv,
                               Sk, status);
  } else {
    p.out0 = static_cast<float*>(dk);
    p.out1 = static_cast<float*>(dv);
    bwd_dkdv_kernel<D><<<B * Hkv * kv_tiles, kBwdThreads, C::kSmem, stream>>>(tmQ, tmK, tmV, tmDO,
                                                                            p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    p.out0 = static_cast<float*>(dq);
    p.out1 = nullptr;
    bwd_dq_kernel<D><<<q_ctas, kBwdThreads, C::kSmemDq, stream>>>(tmQ, tmK, tmV, tmDO, p);
    return cudaGetLastError();
  }
}

}  // namespace

cudaError_t launch_attn_bwd(const void* q, const void* k, const void* v, const float* o,
                            const float* lse, const void* dout, float* dq, float* dk, float* dv,
                            float* delta, int B, int Hq, int Hkv, int Sq, int Sk, int D,
                            int causal, float scale, cudaStream_t stream, int* status) {
  if (D == 128)
    return launch_bwd_impl<128, kNoWindow>(q, k, v, o, lse, dout, dq, dk, dv, delta, B, Hq, Hkv, Sq,
                                       Sk, causal, 0, 0, scale, stream, status);
  return launch_bwd_impl<64, kNoWindow>(q, k, v, o, lse, dout, dq, dk, dv, delta, B, Hq, Hkv, Sq, Sk,
                                    causal, 0, 0, scale, stream, status);
}

long long window_bwd_workspace_floats(int B, int Hq, int Hkv, int Sq, int Sk, int D, int window,
                                      int sinks) {
  const SinkSplit split = sink_split(B, Hq, Hkv, Sq, Sk, window, sinks);
  return window_bwd_delta_floats(B, Hq, Sq) +
         2ll * split.tiles * split.parts * B * Hkv * 128 * D;
}

cudaError_t launch_attn_window_bwd(const void* q, const void* k, const void* v, const void* o,
                                   const float* lse, const void* dout, void* dq, void* dk,
                                   void* dv, float* delta, int B, int Hq, int Hkv, int Sq, int Sk,
                                   int D, int window, int sinks, float scale, cudaStream_t stream,
                                   int* status) {
  const auto launch = has_unseen(Sq, Sk, window, sinks)
                          ? (D == 128 ? launch_bwd_impl<128, kUnseen> : launch_bwd_impl<64, kUnseen>)
                          : (D == 128 ? launch_bwd_impl<128, kWindow> : launch_bwd_impl<64, kWindow>);
  return launch(q, k, v, o, lse, dout, dq, dk, dv, delta, B, Hq, Hkv, Sq, Sk, 1, window, sinks,
                scale, stream, status);
}

}  // namespace attn
