// rope.cu -- rotary positions on projected rows, beside the projection that has them in
// its epilogue (qkv_rope.cu): between a projection of any kind and the attention's layout,
// in training (split and its gradient), and into the pages of a cache in serving (append).
//
// A row of qkv holds Hq query heads, Hkv key heads and Hkv value heads of D dims.  The
// first R dims of a query or key head at position p are R/2 pairs (a, b), dims (2i, 2i+1)
// (style 0) or (i, i + R/2) (style 1), turned by the angle p * theta_i:
//   a' = a cos - b sin,   b' = a sin + b cos,
// from a table of (cos, sin) rows; dims from R on, and value heads, are copied.  The map
// is linear, so the gradient is its transpose: the same with sin negated, and the
// scatter of the heads turned round.
//
// Bound by memory: each element is read and written once.  A thread owns a unit of 16
// dims of a head, two 16-byte vectors that hold whole pairs in either style, at the same
// place of several heads of its token, so that it reads its eight (cos, sin) once.  What
// counts is loads on their way: six units of a thread at once, issued ahead of the position and
// the angles that depend on it, in CTAs of 128 threads; and stores that are let go first
// (8192 tokens, 32/8 heads of 128: split 31.6 us, 6.4 TB/s, its gradient 33.9, append 33.3; with a
// CTA of 256 threads a token, two units at once, behind the angles, 51.2, 53.0 and 51.0;
// four units at once 34.9, 33.8 and 35.1; without the streaming stores 36.2, 36.6, 38.1).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "window.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int kThreads = 128;
constexpr int kPerThread = 4;  // a thread's units, at least (where a token has so many)

__device__ __forceinline__ void record_status(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

enum Form { kSplit, kAppend, kGrad };

struct RopeParams {
  // Rows of Hq + 2 Hkv heads: read (split, append: qkv), or written (gradient: dqkv).
  __nv_bfloat16* rows;
  long long ld;  // elements from one row to the next
  const float* table;    // [max_pos, R/2, 2]
  const int* positions;  // [tokens], or null: s
  const int* slots;      // append: [tokens]
  // Split: [B,H,S,D]; append: q [tokens,Hq,D] and the caches; gradient: dq, dk, dv.
  void *q, *k, *v;
  int tokens, S, Hq, Hkv, D, R, max_pos;
  int group;  // threads of a token
  int page_size;
  long long num_slots;  // append: num_pages * page_size
  FixedDiv by_seq, by_page;
  int* status;
};

// A unit's two vectors as they are in memory, and as floats.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    a = __ldcs(reinterpret_cast<const uint4*>(p));
    b = __ldcs(reinterpret_cast<const uint4*>(q));
  }
  static __device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void get(float (&x)[8], float (&y)[8]) const {
    widen(a, x);
    widen(b, y);
  }
};
template <>
struct Raw<float> {
  float4 a, b, c, d;
  __device__ __forceinline__ void load(const float* p, const float* q) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    c = __ldcs(reinterpret_cast<const float4*>(q));
    d = __ldcs(reinterpret_cast<const float4*>(q) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8], float (&y)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    y[0] = c.x, y[1] = c.y, y[2] = c.z, y[3] = c.w, y[4] = d.x, y[5] = d.y, y[6] = d.z, y[7] = d.w;
  }
};
// Rounded once, to nearest even.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  const uint4 w = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                             pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  __stcs(reinterpret_cast<uint4*>(p), w);
}

// A pair turned, every product and sum rounded by itself (not fused): the bits that the formula
// gives in 32-bit arithmetic, whoever computes it.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
  a = x;
}

// p.group threads to a token.  TG: the type of dq, dk and dv.
template <Form FORM, int STYLE, typename TG>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  using TIn = std::conditional_t<FORM == kGrad, TG, __nv_bfloat16>;
  constexpr int N = sizeof(TIn) == 2 ? 6 : 3;  // units on their way at once
  grid_dependency_wait();
  grid_launch_dependents();
  const int me = threadIdx.x & (p.group - 1);
  const int t = blockIdx.x * (kThreads / p.group) + threadIdx.x / p.group;
  if (t >= p.tokens) return;
  const int units = p.D / 16, turned = p.R / 16;
  const int u = me & (units - 1);  // (D is a power of two)
  const int heads = p.Hq + 2 * p.Hkv;
  const int step = p.group / units;
  int b = 0, s = t;
  if (FORM != kAppend) {
    b = p.by_seq.div(t);
    s = t - b * p.S;
  }
  // This unit's two vectors of a rotated head, and of one that is copied.
  const bool turns = u < turned;
  const int o0 = STYLE == 1 && turns ? 8 * u : 16 * u;
  const int o1 = STYLE == 1 && turns ? p.R / 2 + 8 * u : 16 * u + 8;
  int slot = -1;
  if (FORM == kAppend) slot = __ldg(p.slots + t);
  int pos = s;
  if (p.positions != nullptr) pos = __ldg(p.positions + t);
  long long page = -1;
  int at = 0;
  float cs[8], sn[8];

  // Where head h begins on the other side than the projected row.
  const auto other = [&](int h) -> size_t {
    const bool is_q = h < p.Hq;
    const int g = is_q ? h : h >= p.Hq + p.Hkv ? h - p.Hq - p.Hkv : h - p.Hq;
    const int H = is_q ? p.Hq : p.Hkv;
    if (FORM == kAppend && !is_q) return ((page * H + g) * p.page_size + at) * p.D;
    if (FORM == kAppend) return (static_cast<size_t>(t) * H + g) * p.D;
    return ((static_cast<size_t>(b) * H + g) * p.S + s) * p.D;
  };
  const auto base = [&](int h) { return h < p.Hq ? p.q : h >= p.Hq + p.Hkv ? p.v : p.k; };
  __nv_bfloat16* const row = p.rows + t * p.ld;
  const int h_first = me / units;
  for (int h0 = h_first; h0 < heads; h0 += N * step) {
    Raw<TIn> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * step;
      if (h < heads) {
        const bool is_v = h >= p.Hq + p.Hkv;
        // A value head's vectors lie side by side.
        const int a0 = is_v ? 16 * u : o0, a1 = is_v ? 16 * u + 8 : o1;
        const TIn* from = FORM == kGrad ? static_cast<const TIn*>(base(h)) + other(h)
                                        : reinterpret_cast<const TIn*>(row) + h * p.D;
        raw[i].load(from + a0, from + a1);
      }
    }
    if (h0 == h_first) {  // behind the first loads, which need neither
      if (FORM == kAppend) {
        if (slot >= 0 && slot < p.num_slots) {
          page = p.by_page.div(slot);
          at = slot - static_cast<int>(page) * p.page_size;
        } else if (slot != -1) {
          record_status(p.status, ATTN_ERR_INVALID_ARG);
        }
      }
      if (turns) {
        if (pos < 0 || pos >= p.max_pos) {
          record_status(p.status, ATTN_ERR_INVALID_ARG);
          pos = min(max(pos, 0), p.max_pos - 1);
        }
        const float4* angles =
            reinterpret_cast<const float4*>(p.table + static_cast<size_t>(pos) * p.R + 16 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 w = __ldg(angles + i);
          cs[2 * i] = w.x, sn[2 * i] = w.y, cs[2 * i + 1] = w.z, sn[2 * i + 1] = w.w;
        }
        if (FORM == kGrad)
#pragma unroll
          for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int h = h0 + i * step;
      const bool is_v = h >= p.Hq + p.Hkv;
      if (h >= heads || (FORM == kAppend && h >= p.Hq && page < 0)) continue;
      float x[8], y[8];
      raw[i].get(x, y);
      if (turns && !is_v) {
        if constexpr (STYLE == 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e) turn(x[e], y[e], cs[e], sn[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            turn(x[2 * e], x[2 * e + 1], cs[e], sn[e]);
            turn(y[2 * e], y[2 * e + 1], cs[4 + e], sn[4 + e]);
          }
        }
      }
      const int a0 = is_v ? 16 * u : o0, a1 = is_v ? 16 * u + 8 : o1;
      __nv_bfloat16* to = FORM == kGrad ? row + h * p.D
                                        : static_cast<__nv_bfloat16*>(base(h)) + other(h);
      store8(to + a0, x);
      store8(to + a1, y);
    }
  }
}

template <Form FORM, typename TG = float>
cudaError_t launch_rope(RopeParams p, int style, cudaStream_t stream) {
  const long long units = (p.Hq + 2ll * p.Hkv) * (p.D / 16);
  p.group = 32;
  while (p.group < kThreads && 2 * kPerThread * p.group <= units) p.group *= 2;
  const int tokens = kThreads / p.group;  // of a CTA
  return launch_programmatic(style == 0 ? rope_kernel<FORM, 0, TG> : rope_kernel<FORM, 1, TG>,
                             dim3((p.tokens + tokens - 1) / tokens), dim3(kThreads), 0, stream, p);
}

// The frequencies' scaling, as internal.h's RopeScaling; one thread per table entry.  In
// 64 bits: the angle of a far position needs more than 32.  Bound by that arithmetic (an exp and a
// sincos an entry): 131,072 positions of 128 dims 1.0 ms, scaled by parts 1.4, their bytes
// 10 us.  A model makes its table once.
__global__ void rope_table_scaled_kernel(float* table, int max_pos, int R, double log_base,
                                         const RopeScaling sc) {
  const long long n = static_cast<long long>(max_pos) * (R / 2);
  for (long long idx = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; idx < n;
       idx += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int i = static_cast<int>(idx % (R / 2));
    const long long pos = idx / (R / 2);
    double theta = exp(-2.0 * i / R * log_base);
    // Turns over the original context decide how far the frequency is lowered.
    double keep = 0.0;
    if (sc.original > 0) {
      const double turns = sc.original * theta * 0.15915494309189535;  // 1 / (2 pi)
      keep = fmin(fmax((turns - sc.low) / (sc.high - sc.low), 0.0), 1.0);
    }
    theta *= keep + (1.0 - keep) / sc.factor;
    double sn, cs;
    sincos(static_cast<double>(pos) * theta, &sn, &cs);
    table[2 * idx] = static_cast<float>(cs * sc.amplitude);
    table[2 * idx + 1] = static_cast<float>(sn * sc.amplitude);
  }
}

}  // namespace

cudaError_t launch_rope_table_scaled(float* table, int max_pos, int R, double base,
                                     const RopeScaling& scaling, cudaStream_t stream) {
  const long long n = static_cast<long long>(max_pos) * (R / 2);
  const int blocks = static_cast<int>(n / 256 + 1 < 4096 ? n / 256 + 1 : 4096);
  rope_table_scaled_kernel<<<blocks, 256, 0, stream>>>(table, max_pos, R, std::log(base), scaling);
  return cudaGetLastError();
}

cudaError_t launch_rope_split(const void* qkv, long long ld, const float* table,
                              const int* positions, void* q, void* k, void* v, int B, int S, int Hq,
                              int Hkv, int D, int R, int max_pos, int style, cudaStream_t stream,
                              int* status) {
  RopeParams p = {};
  p.rows = static_cast<__nv_bfloat16*>(const_cast<void*>(qkv));
  p.ld = ld;
  p.table = table;
  p.positions = positions;
  p.q = q;
  p.k = k;
  p.v = v;
  p.tokens = B * S;
  p.S = S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.R = R;
  p.max_pos = max_pos;
  p.by_seq = FixedDiv(S);
  p.status = status;
  return launch_rope<kSplit>(p, style, stream);
}

cudaError_t launch_rope_split_bwd(const void* dq, const void* dk, const void* dv, int fp32,
                                  const float* table, const int* positions, void* dqkv,
                                  long long ld, int B, int S, int Hq, int Hkv, int D, int R,
                                  int max_pos, int style, cudaStream_t stream, int* status) {
  RopeParams p = {};
  p.rows = static_cast<__nv_bfloat16*>(dqkv);
  p.ld = ld;
  p.table = table;
  p.positions = positions;
  p.q = const_cast<void*>(dq);
  p.k = const_cast<void*>(dk);
  p.v = const_cast<void*>(dv);
  p.tokens = B * S;
  p.S = S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.R = R;
  p.max_pos = max_pos;
  p.by_seq = FixedDiv(S);
  p.status = status;
  return fp32 ? launch_rope<kGrad, float>(p, style, stream)
              : launch_rope<kGrad, __nv_bfloat16>(p, style, stream);
}

cudaError_t launch_rope_append(const void* qkv, long long ld, const float* table,
                               const int* positions, const int* slots, void* q, void* k_cache,
                               void* v_cache, int T, int Hq, int Hkv, int D, int R, int max_pos,
                               int num_pages, int page_size, int style, cudaStream_t stream,
                               int* status) {
  RopeParams p = {};
  p.rows = static_cast<__nv_bfloat16*>(const_cast<void*>(qkv));
  p.ld = ld;
  p.table = table;
  p.positions = positions;
  p.slots = slots;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.tokens = T;
  p.S = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.R = R;
  p.max_pos = max_pos;
  p.page_size = page_size;
  p.num_slots = static_cast<long long>(num_pages) * page_size;
  p.by_page = FixedDiv(page_size);
  p.status = status;
  return launch_rope<kAppend>(p, style, stream);
}

}  // namespace attn
