// pages.cu -- bookkeeping of a paged KV cache on the device: free, fork, compact,
// and the page copies that fork and compact list.
//
// A block table [rows, max_pages] (int32) names the page of each slot of a row
// (-1: none); refs[p] counts the holders of page p (0: free).  All results are
// functions of the inputs alone: pages are handed out lowest id first, in the
// order of (row, slot), and the atomics below add and take minima of integers, so
// their order changes nothing.  The host never reads back, so the calls can be
// captured in a graph between decode steps.
//
// Each operation is a few phases with a barrier between them:
//   free     1 copy refs              2 give up the references
//   fork     1 copy refs, count free  2 count holders, list free pages, copy the
//            read-only slots          3 count the pages each row needs
//            4 hand them out
//   compact  1 count live             2 list holes and movers   3 renumber
//   append   at its struct
// What a call costs beyond the tables' bytes is latency: round trips to L2 that follow
// each other, and the barriers.  So the number of CTAs that take part grows with the
// call (us for fork / compact / free, graph replays):
//   one CTA, lists and counters in shared memory (run_small; fork and compact):
//     8 x 48 slots, 600 pages 5.0 / 2.8; 32 x 64, 4000 6.8 / 5.3; 64 x 64, 6000 9.3 / 11.6
//   one cluster of 16 CTAs and the hardware's barrier, up to 2^15 elements:
//     64 x 64, 6000 - / 8.0 / 4.9; 128 x 128, 16000 11.1 / 8.2 / 5.0; 256 x 128, 30000
//     13.5 / 10.0 / 5.0; 256 x 256, 60000 17.6 / 13.2 / 5.0 (clusters of 8: 24.9 / 18.9 / 7.7)
//   a cooperative grid of 1024 elements a CTA, at most one CTA an SM: 128 x 128, 16000
//     14.0 / 9.7 / 4.9; 256 x 128, 30000 14.3 / 10.2 / 5.0; 256 x 256, 60000 14.1 / 10.3
//     / 5.0; 1024 x 2048, 2 M 44.5 / 35.6 / 11.0 (a launch per phase: 64.4 / 52.0 / 12.5).
//     Bound there by the L2's rate of scattered 4-byte atomics.  (Free grows with what is
//     given up: of 2 M entries none 8.2, half 11.7, 1.4 M 14.5, nearly all 15.9, and 16 to
//     18 with inputs that are not in L2.)
// The forms were compared with divisions in fork.  As multiplications they save it 0.4 to
// 1.5 us up to 2^20 slots (8 x 48 4.5, 32 x 64 5.8, 64 x 64 7.7, 256 x 128 12.4, 1024 x
// 512 with 500000 pages 18.6); from 2^21 on it takes 8 % longer (48.0), the atomics
// meeting in denser bursts.
// All of the above before fork looked up whether each entry's page has holders
// (old_entry): with that, on inputs of its own, 8 x 48 4.5, 32 x 64 6.0, 64 x 64 8.1, 128 x
// 128 10.9, 256 x 128 13.2, 256 x 256 13.4, 1024 x 512 25, 1024 x 2048 56 to 62; without
// it 4.5, 6.0, 8.0, 10.8, 13.0, 13.2, 23, 53.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "window.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
// The largest calls (elements of arrays) of one CTA, and of one cluster.
constexpr long long kSmallForkEntries = 8192, kSmallForkPages = 6144, kSmallForkSlots = 8192;
constexpr long long kSmallCompactEntries = 8192, kSmallCompactPages = 4096;
constexpr long long kSmallAppendEntries = 8192, kSmallAppendPages = 8192, kSmallAppendTokens = 4096;
constexpr long long kSmallAppendSlots = 128;  // of a row's new tokens
constexpr long long kClusterWork = 1 << 15;
constexpr int kClusterCtas = 16;  // past the portable 8: the kernels opt in
constexpr int kMaxCopiers = 6;    // append: clusters that copy the table

__device__ __forceinline__ void record_status(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// This CTA's part [begin, end) of n things shared out over the grid.
struct Part {
  int begin, end;
  // The parts begin at multiples of `align` (a power of two).
  __device__ __forceinline__ explicit Part(int n, int align = 1) {
    const int chunk = ((n + gridDim.x - 1) / gridDim.x + align - 1) & ~(align - 1);
    begin = static_cast<int>(min(static_cast<long long>(blockIdx.x) * chunk, static_cast<long long>(n)));
    end = min(begin + chunk, n);
  }
};

// Sum of one value per thread over the CTA (kWarps warps); every thread gets it.
__device__ __forceinline__ int block_sum(int x, int* smem) {
  x = __reduce_add_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = x;
  __syncthreads();
  const int total = __reduce_add_sync(0xffffffffu, smem[threadIdx.x & 31]);
  __syncthreads();
  return total;
}

// Exclusive prefix sum of one value per thread over the CTA; total: their sum.
__device__ __forceinline__ int block_scan(int x, int* smem, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) smem[warp] = incl;
  __syncthreads();
  int w = smem[lane], wincl = w;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, wincl, off);
    if (lane >= off) wincl += y;
  }
  total = __shfl_sync(0xffffffffu, wincl, 31);
  const int before = __shfl_sync(0xffffffffu, wincl - w, warp);
  __syncthreads();
  return before + incl - x;
}

// Sum of counts[0, n) by the whole CTA.
__device__ __forceinline__ int sum_counts(const int* counts, int n, int* smem) {
  int x = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) x += counts[i];
  return block_sum(x, smem);
}

// Place of element i in a shared array that threads read in runs: a word of padding
// every 32 keeps the runs of a warp in different banks.
__host__ __device__ __forceinline__ constexpr int pad(int i) { return i + (i >> 5); }

// A table entry: a page, or -1 (an entry that is neither is reported and read as -1).
__device__ __forceinline__ int checked_entry(int e, int num_pages, int* status) {
  if (e >= num_pages || e < -1) {
    record_status(status, ATTN_ERR_INVALID_ARG);
    return -1;
  }
  return e;
}

// All phases of a call.  kCluster: one cluster and its barrier; kGrid: a cooperative
// grid and its (every CTA is resident, and each enters every barrier).
enum Span { kCluster, kGrid };
template <typename Op, Span SPAN>
__global__ void __launch_bounds__(kThreads, 1) pages_phases_kernel(const Op op) {
  __shared__ int smem[32];
  if constexpr (SPAN == kCluster) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  for (int ph = 0; ph < Op::kPhases; ++ph) {
    op.run(ph, smem);
    if (ph + 1 == Op::kPhases) break;
    if constexpr (SPAN == kCluster)
      cluster_sync();
    else
      cooperative_groups::this_grid().sync();
  }
}

// A small call: one CTA.
template <typename Op>
__global__ void __launch_bounds__(kThreads, 1) pages_small_kernel(const Op op) {
  __shared__ int smem[32];
  extern __shared__ int lists[];
  grid_dependency_wait();
  grid_launch_dependents();
  op.run_small(smem, lists);
}

// ------------------------------------------------------------------ free
struct FreeOp {
  static constexpr int kPhases = 2;
  const int *table, *refs, *seqlens;
  int *table_out, *refs_out;
  int B, M, P, page_size, window, sinks, room;
  int refs_vec, table_vec;  // 16-byte accesses are aligned
  FixedDiv by_row;          // M, or M / 4 with table_vec
  int* status;

  // Slots s, s + 1, ... of a row of `len` keys, holding e: the pages kept, or -1 for
  // those given up.
  template <int N>
  __device__ __forceinline__ void settle(int (&e)[N], int s, int len) const {
    bool drop[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      e[i] = checked_entry(e[i], P, status);
      // A slot is kept when the row goes on and the slot holds a key that the next
      // decode reads (the window of seqlens, the sinks) or that is still to come.
      const int lo = (s + i) * page_size;
      const bool keep = len >= 0 && lo < static_cast<long long>(len) + room &&
                        (lo + page_size > len - window || lo < sinks);
      drop[i] = !keep && e[i] >= 0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (drop[i]) {
        atomicSub(refs_out + e[i], 1);  // (its result unused: a reduction in L2)
        e[i] = -1;
      }
  }
  __device__ __forceinline__ int length(int b) const { return min(seqlens[b], M * page_size); }

  __device__ void run(int ph, int*) const {
    const unsigned tid = blockIdx.x * kThreads + threadIdx.x, n_threads = gridDim.x * kThreads;
    // Four at a time where the arrays allow it: the whole of refs in 16-byte vectors,
    // and the tables if their rows are multiples of four slots.
    if (ph == 0) {
      if (refs == refs_out) return;
      const unsigned vecs = refs_vec ? P / 4 : 0;
      for (unsigned i = tid; i < vecs; i += n_threads)
        reinterpret_cast<int4*>(refs_out)[i] = reinterpret_cast<const int4*>(refs)[i];
      for (unsigned p = 4 * vecs + tid; p < static_cast<unsigned>(P); p += n_threads)
        refs_out[p] = refs[p];
      return;
    }
    const unsigned entries = static_cast<unsigned>(B) * M;  // < 2^31: i cannot wrap
    if (table_vec) {
      const unsigned row_vecs = M / 4;
      for (unsigned i = tid; i < entries / 4; i += n_threads) {
        const int b = by_row.div(i), s = 4 * (i - b * row_vecs), len = length(b);
        const int4 x = reinterpret_cast<const int4*>(table)[i];
        int e[4] = {x.x, x.y, x.z, x.w};
        settle(e, s, len);
        reinterpret_cast<int4*>(table_out)[i] = make_int4(e[0], e[1], e[2], e[3]);
      }
    } else {
      for (unsigned i = tid; i < entries; i += n_threads) {
        const int b = by_row.div(i);
        int e[1] = {table[i]};
        settle(e, i - b * M, length(b));
        table_out[i] = e[0];
      }
    }
  }
};

// ------------------------------------------------------------------ fork
struct ForkOp {
  static constexpr int kPhases = 4;
  const int *table, *refs, *seqlens, *parents;
  int *table_out, *refs_out, *seqlens_out, *src, *dst, *counts;
  int *lowest, *free_list, *need, *cta_free, *cta_need;  // workspace
  unsigned* live;  // workspace: bit p of word p / 32: page p has holders
  int B, R, M, P, page_size, room;
  FixedDiv by_page, by_row, by_writable;  // page_size, M, small_slots
  int* status;

  // An entry of the old table: a page, or -1.  One that is neither, or whose page counts
  // no holder (it is in the free list), is reported and read as -1.  (From bits, which
  // stay in L1: 1024 x 2048 slots of 2 M pages take 62 us, 53 without the look-up and 70
  // with refs itself; 256 x 256 of 60000 13.3, 13.1 and 14.0.)
  __device__ __forceinline__ int old_entry(size_t i, int* report) const {
    const int e = checked_entry(table[i], P, report);
    if (e < 0 || (live[e >> 5] >> (e & 31) & 1u)) return e;
    record_status(report, ATTN_ERR_INVALID_ARG);
    return -1;
  }

  // Slots of a row that hold keys or shall: ceil((len + room) / page_size), at most M.
  // (M * page_size <= 2^30 and the host clamps room to it.)
  __device__ __forceinline__ int slots_for(int len) const {
    const unsigned keys = min(static_cast<unsigned>(len) + room, static_cast<unsigned>(M) * page_size);
    return by_page.div(static_cast<int>(keys + page_size - 1));
  }

  // New row r: its parent (-1: a row without pages), length, and slots to be written
  // [lo, hi).  A finished row's (length below 0) stays one.
  struct Row {
    int parent, len, lo, hi;
  };
  __device__ __forceinline__ Row row(int r) const {
    Row x;
    x.parent = parents[r];
    if (x.parent >= B || x.parent < -1) {
      record_status(status, ATTN_ERR_INVALID_ARG);
      x.parent = -1;
    }
    x.len = x.parent < 0 ? 0 : min(seqlens[x.parent], M * page_size);
    if (x.len < 0) x.parent = -1;
    x.lo = x.parent < 0 ? 0 : by_page.div(x.len);
    x.hi = x.parent < 0 ? 0 : slots_for(x.len);
    return x;
  }
  // A page of a slot to be written stays with the lowest (row, slot) that has it
  // there, if nobody else holds it.  refs_out holds the other holders until phase 3,
  // in which only that (row, slot) changes it.
  __device__ __forceinline__ bool keeps(int e, int at) const {
    return e >= 0 && lowest[e] == at && refs_out[e] == 0;
  }

  __device__ void run(int ph, int* smem) const {
    const int tid = blockIdx.x * kThreads + threadIdx.x, n_threads = gridDim.x * kThreads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Part pages(P, 32), rows(R);
    if (ph == 0) {
      int n = 0;
      for (int p0 = pages.begin; p0 < pages.end; p0 += kThreads) {
        const int p = p0 + threadIdx.x;
        const int c = p < pages.end ? refs[p] : -1;
        n += c == 0;
        const unsigned bits = __ballot_sync(0xffffffffu, c > 0);
        if (p < pages.end) {
          refs_out[p] = c;
          lowest[p] = INT_MAX;
          if (lane == 0) live[p >> 5] = bits;
        }
      }
      n = block_sum(n, smem);
      if (threadIdx.x == 0) cta_free[blockIdx.x] = n;
      for (int r = tid; r < R; r += n_threads) seqlens_out[r] = row(r).len;
    } else if (ph == 1) {
      // refs_out: the holders that are no slots of the old table ...
      const unsigned entries = static_cast<unsigned>(B) * M, new_entries = static_cast<unsigned>(R) * M;
      for (unsigned i = tid; i < entries; i += n_threads) {
        const int e = old_entry(i, status);
        if (e >= 0) atomicSub(refs_out + e, 1);
      }
      // ... and the read-only slots of the new one.
      for (unsigned i = tid; i < new_entries; i += n_threads) {
        const int r = by_row.div(i), s = i - r * M;
        const Row x = row(r);
        int e = -1;
        if (s < x.hi || s < x.lo) e = old_entry(static_cast<size_t>(x.parent) * M + s, nullptr);
        if (s < x.lo) {
          if (e >= 0) atomicAdd(refs_out + e, 1);
        } else if (e >= 0) {
          atomicMin(lowest + e, static_cast<int>(i));
          e = -1;
        }
        table_out[i] = e;
      }
      int at = sum_counts(cta_free, blockIdx.x, smem);
      for (int p0 = pages.begin; p0 < pages.end; p0 += kThreads) {
        const int p = p0 + threadIdx.x;
        const int is_free = p < pages.end && refs[p] == 0;
        int total;
        const int k = at + block_scan(is_free, smem, total);
        if (is_free) free_list[k] = p;
        at += total;
      }
    } else if (ph == 2) {
      // A warp per row: the pages it needs, then this CTA's rows' offsets.
      for (int r = rows.begin + warp; r < rows.end; r += kWarps) {
        const Row x = row(r);
        int n = 0;
        for (int s = x.lo + lane; s < x.hi; s += 32) {
          const int e = old_entry(static_cast<size_t>(x.parent) * M + s, nullptr);
          n += !keeps(e, r * M + s);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) need[r] = n;
      }
      __syncthreads();
      int at = 0;
      for (int r0 = rows.begin; r0 < rows.end; r0 += kThreads) {
        const int r = r0 + threadIdx.x;
        const int n = r < rows.end ? need[r] : 0;
        int total;
        const int k = at + block_scan(n, smem, total);
        if (r < rows.end) need[r] = k;
        at += total;
      }
      if (threadIdx.x == 0) cta_need[blockIdx.x] = at;
    } else {
      const int n_free = sum_counts(cta_free, gridDim.x, smem);
      const int base = sum_counts(cta_need, blockIdx.x, smem);
      if (blockIdx.x == gridDim.x - 1) {
        const int n = base + cta_need[blockIdx.x];
        if (threadIdx.x == 0) {
          counts[0] = n;
          counts[1] = n_free;
          if (n > n_free) record_status(status, ATTN_ERR_NO_PAGES);
        }
      }
      for (int r = rows.begin + warp; r < rows.end; r += kWarps) {
        const Row x = row(r);
        int k = base + need[r];
        int from = -1, to = -1;  // the row's copy: its first writable slot may hold keys
        for (int s0 = x.lo; s0 < x.hi; s0 += 32) {
          const int s = s0 + lane;
          const bool mine = s < x.hi;
          const int at = r * M + s;
          const int e =
              mine ? old_entry(static_cast<size_t>(x.parent) * M + s, nullptr) : -1;
          const bool keep = mine && keeps(e, at);
          const unsigned fresh = __ballot_sync(0xffffffffu, mine && !keep);
          int page = e;
          if (mine && !keep) {
            const int mine_k = k + __popc(fresh & ((1u << lane) - 1u));
            page = mine_k < n_free ? free_list[mine_k] : -1;
            const bool holds_keys = s * page_size < x.len;
            if (holds_keys && e >= 0 && page >= 0) {
              from = e;
              to = page;
            }
            // No page left: the row ends before the slot's keys.
            if (holds_keys && page < 0) seqlens_out[r] = s * page_size;
          }
          if (mine) {
            if (page >= 0) refs_out[page] = 1;
            table_out[at] = page;
          }
          k += __popc(fresh);
        }
        // Only slot lo, lane 0's in the first round, can hold keys.
        if (lane == 0) {
          src[r] = from;
          dst[r] = to;
        }
      }
    }
  }

  // One CTA, everything but the tables in shared memory.  The slots to be written are
  // numbered r * W + j, j < W = room / page_size + 2, which is their order, so each
  // thread takes a run of them and one prefix sum ranks the pages they need.
  __host__ __device__ static int small_slots(int room, int page_size) { return room / page_size + 2; }
  static size_t small_bytes(int P, int R) {
    return (pad(P) + 2ll * P + 2ll * R) * sizeof(int);
  }
  __device__ void run_small(int* smem, int* lists) const {
    int* held = lists;       // holders other than slots to be written; then refs_out
    // Lowest (r, slot) that would write the page; kFree: it has no holder.  Of the pages
    // in slots to be written, at the end: kStays, or of those that had no holder kGiven.
    int* low = held + pad(P);
    constexpr int kFree = INT_MAX - 1, kStays = -1, kGiven = -2;
    int* free_at = low + P;  // free pages, ascending
    int* parent = free_at + P;
    int* len = parent + R;
    const int t = threadIdx.x;
    const int per = (P + kThreads - 1) / kThreads;  // pages of a thread, in one run
    const int p0 = min(t * per, P), p1 = min(p0 + per, P);
    int n = 0;
    for (int p = t; p < P; p += kThreads) {
      const int c = refs[p];
      held[pad(p)] = c;
      low[p] = c > 0 ? INT_MAX : kFree;
    }
    for (int r = t; r < R; r += kThreads) {
      const Row x = row(r);
      parent[r] = x.parent;
      len[r] = x.len;
    }
    __syncthreads();
    for (int p = p0; p < p1; ++p) n += held[pad(p)] == 0;
    int n_free;
    int k = block_scan(n, smem, n_free);
    for (int p = p0; p < p1; ++p)
      if (held[pad(p)] == 0) free_at[k++] = p;
    __syncthreads();
    const auto old_entry = [&](int i, int* report) {  // as in run
      const int e = checked_entry(table[i], P, report);
      if (e < 0) return e;
      const int l = low[e];
      if (l != kFree && l != kGiven) return e;
      record_status(report, ATTN_ERR_INVALID_ARG);
      return -1;
    };
    const unsigned entries = B * M, new_entries = R * M;
    for (unsigned i = t; i < entries; i += kThreads) {
      const int e = old_entry(i, status);
      if (e >= 0) atomicSub(held + pad(e), 1);
    }
    const auto slot_begin = [&](int r) { return parent[r] < 0 ? 0 : by_page.div(len[r]); };
    const auto slot_end = [&](int r) { return parent[r] < 0 ? 0 : slots_for(len[r]); };
    for (unsigned i = t; i < new_entries; i += kThreads) {
      const int r = by_row.div(i), s = i - r * M;
      const int lo = slot_begin(r);
      int e = -1;
      if (s < lo || s < slot_end(r)) e = old_entry(parent[r] * M + s, nullptr);
      if (s < lo) {
        if (e >= 0) atomicAdd(held + pad(e), 1);
      } else if (e >= 0) {
        atomicMin(low + e, static_cast<int>(i));
        e = -1;
      }
      table_out[i] = e;
    }
    __syncthreads();
    const int W = small_slots(room, page_size), slots = R * W;
    const int run = (slots + kThreads - 1) / kThreads;
    const int f0 = min(t * run, slots), f1 = min(f0 + run, slots);
    // Slot f's entry; -2 if it is past its row's end.  `stays`: its page is its own.
    const auto entry = [&](int f, int& r, int& s, bool& stays) {
      r = by_writable.div(f);
      s = slot_begin(r) + f - r * W;
      stays = false;
      if (s >= slot_end(r)) return -2;
      const int e = old_entry(parent[r] * M + s, nullptr);
      stays = e >= 0 && low[e] == r * M + s && held[pad(e)] == 0;
      return e;
    };
    n = 0;
    int r, s;
    bool stays;
    for (int f = f0; f < f1; ++f) n += entry(f, r, s, stays) != -2 && !stays;
    int needed;
    k = block_scan(n, smem, needed);  // its barrier: nobody reads held as it was any more
    // A row without slots to write has nothing to copy; the others set theirs below.
    for (int f = f0; f < f1; ++f) {
      int e = entry(f, r, s, stays);
      // Only a row's first slot to write can hold keys already.
      const bool first = f == r * W, holds_keys = first && e != -2 && s * page_size < len[r];
      const int from = e;
      int length = len[r];
      bool copied = false;
      if (e != -2) {
        if (!stays) {
          e = k < n_free ? free_at[k] : -1;
          ++k;
          copied = holds_keys && from >= 0 && e >= 0;
          if (holds_keys && e < 0) length = s * page_size;  // no page left for the keys
        }
        table_out[r * M + s] = e;
        if (e >= 0) low[e] = stays ? kStays : kGiven;  // one holder, and nobody's lowest
      }
      if (first) {
        src[r] = copied ? from : -1;
        dst[r] = copied ? e : -1;
        seqlens_out[r] = length;
      }
    }
    if (t == 0) {
      counts[0] = needed;
      counts[1] = n_free;
      if (needed > n_free) record_status(status, ATTN_ERR_NO_PAGES);
    }
    __syncthreads();
    for (int p = t; p < P; p += kThreads) refs_out[p] = low[p] < 0 ? 1 : held[pad(p)];
  }
};

// ------------------------------------------------------------------ compact
struct CompactOp {
  static constexpr int kPhases = 3;
  const int *table, *refs;
  int *table_out, *refs_out, *src, *dst, *num_live;
  int *rank, *cta_live;  // workspace
  int B, M, P;
  int* status;

  // Live pages in [begin, end), by the whole CTA.
  __device__ __forceinline__ int live_in(int begin, int end, int* smem) const {
    int n = 0;
    for (int p = begin + threadIdx.x; p < end; p += kThreads) n += refs[p] > 0;
    return block_sum(n, smem);
  }
  // Live pages below id n_live: those that stay.
  __device__ __forceinline__ int staying(int n_live, int* smem) const {
    const int chunk = (P + gridDim.x - 1) / gridDim.x;
    const int cta = n_live / chunk;  // the CTA part that n_live lies in (or past the last)
    return sum_counts(cta_live, min(cta, static_cast<int>(gridDim.x)), smem) +
           live_in(min(cta * chunk, P), n_live, smem);
  }

  __device__ void run(int ph, int* smem) const {
    const int tid = blockIdx.x * kThreads + threadIdx.x, n_threads = gridDim.x * kThreads;
    const Part pages(P);
    if (ph == 0) {
      const int n = live_in(pages.begin, pages.end, smem);
      if (threadIdx.x == 0) cta_live[blockIdx.x] = n;
      return;
    }
    const int n_live = sum_counts(cta_live, gridDim.x, smem);
    const int stay = staying(n_live, smem);
    const int moves = n_live - stay;  // as many holes below n_live as live pages from it on
    if (ph == 1) {
      int before = sum_counts(cta_live, blockIdx.x, smem);
      for (int p0 = pages.begin; p0 < pages.end; p0 += kThreads) {
        const int p = p0 + threadIdx.x;
        const int c = p < pages.end ? refs[p] : 0;
        int total;
        const int k = before + block_scan(c > 0, smem, total);  // live pages below p
        before += total;
        if (p >= pages.end) continue;
        if (p < n_live) {
          if (c > 0)
            refs_out[p] = c;
          else
            dst[p - k] = p;
        } else {
          refs_out[p] = 0;
          if (c > 0) {
            src[k - stay] = p;
            rank[p] = k - stay;
          }
        }
      }
      for (int i = moves + tid; i < P / 2; i += n_threads) src[i] = dst[i] = -1;
      if (tid == 0) *num_live = n_live;
    } else {
      for (int i = tid; i < moves; i += n_threads) refs_out[dst[i]] = refs[src[i]];
      const unsigned entries = static_cast<unsigned>(B) * M;
      for (unsigned i = tid; i < entries; i += n_threads) {
        int e = checked_entry(table[i], P, status);
        if (e >= 0 && refs[e] <= 0) {  // an entry of a page that counts no holder
          record_status(status, ATTN_ERR_INVALID_ARG);
          e = -1;
        }
        table_out[i] = e >= n_live ? dst[rank[e]] : e;
      }
    }
  }

  // One CTA: the new id of every page in shared memory, a run of pages per thread.
  static size_t small_bytes(int P) { return (pad(P) + P / 2) * sizeof(int); }
  __device__ void run_small(int* smem, int* lists) const {
    int* to = lists;       // the page's count, then its new id (-1: not live)
    int* holes = to + pad(P);   // free ids below n_live, ascending
    const int t = threadIdx.x;
    const int per = (P + kThreads - 1) / kThreads;
    const int p0 = min(t * per, P), p1 = min(p0 + per, P);
    for (int p = t; p < P; p += kThreads) to[pad(p)] = refs[p];
    __syncthreads();
    int n = 0;
    for (int p = p0; p < p1; ++p) n += to[pad(p)] > 0;
    int n_live;
    const int before = block_scan(n, smem, n_live);  // live pages below p0
    n = 0;
    for (int p = p0; p < min(p1, n_live); ++p) n += to[pad(p)] > 0;
    const int stay = block_sum(n, smem), moves = n_live - stay;
    int k = before;
    for (int p = p0; p < p1; ++p) {
      if (to[pad(p)] > 0)
        ++k;
      else if (p < n_live)
        holes[p - k] = p;
    }
    __syncthreads();
    k = before;
    for (int p = p0; p < p1; ++p) {
      const int c = to[pad(p)];
      int id = -1;
      if (c > 0) {
        id = p < n_live ? p : holes[k - stay];
        if (p >= n_live) {
          src[k - stay] = p;
          dst[k - stay] = id;
        }
        refs_out[id] = c;
        ++k;
      }
      if (p >= n_live) refs_out[p] = 0;
      to[pad(p)] = id;
    }
    for (int i = moves + t; i < P / 2; i += kThreads) src[i] = dst[i] = -1;
    if (t == 0) *num_live = n_live;
    __syncthreads();
    const unsigned entries = B * M;
    for (unsigned i = t; i < entries; i += kThreads) {
      const int e = checked_entry(table[i], P, status);
      const int id = e >= 0 ? to[pad(e)] : -1;
      if (e >= 0 && id < 0) record_status(status, ATTN_ERR_INVALID_ARG);  // counts no holder
      table_out[i] = id;
    }
  }
};

// ------------------------------------------------------------------ append
// Pages, positions and slots for a step's new tokens.  The workers, a cluster of CTAs, take
// equal parts of the pages and of the rows:
//   1 count the free pages; count the pages that each row lacks, its tokens; look for rows that
//     would write into a page of several holders
//   2 list the free pages that are needed; decide which rows take their tokens
//   3 hand the pages out  4 positions and slots of the tokens
// and further CTAs copy refs and the table meanwhile, but for the pages and entries that are
// the workers'.  Nothing orders their stores before the workers' loads, so the workers take
// entries that named a page before the call from `table`, and from `table_out` only those that
// they wrote.
// Token sums are clamped to T + 1 (a sum that saturates stays associative).
//
// Latency, again: each phase is a few dependent trips to L2.  1024 rows of 1024 slots, 560,000
// pages and 9152 tokens take 16.0 us; with lengths updated in place, where the workers copy
// the table themselves before they begin, 21.5.  Where all fits one CTA's shared
// memory (run_small), there are no phases: 8 rows 3.5 us instead of 10.2, 64 rows of 128 slots
// with 2048 tokens 7.9 instead of 12.0.  But its tokens take turns, and a row's slots one thread:
// 15360 tokens took 19.2 us instead of 12.7, one row of 500 new slots 30.4 instead of 19.6.
struct AppendOp {
  const int *table, *refs, *seqlens, *new_lens;
  int *table_out, *refs_out, *seqlens_out, *cu, *positions, *slots, *counts;
  // Workspace: the free pages that are needed, ascending; of each worker's warps the free
  // pages, and of each worker the free and needed pages and the tokens; per row the needed
  // pages before it, its first token (both in its worker's rows), and its length before (-1:
  // it takes no tokens).
  int *free_list, *warp_free, *cta_free, *cta_need, *cta_tokens, *need, *first, *len;
  int B, M, P, T, page_size, workers;
  FixedDiv by_page, by_row;  // page_size; M, or M / 4 with table_vec
  int refs_vec, table_vec;   // 16-byte accesses are aligned
  int* status;

  struct Row {
    int len, n;
    int lo, hi;  // slots of the new tokens
  };
  __device__ __forceinline__ Row row(int r, int* report) const {
    return row(seqlens[r], new_lens[r], report);
  }
  __device__ __forceinline__ Row row(int length, int n, int* report) const {
    Row x = {length, n, 0, 0};
    if (x.n < 0) {
      record_status(report, ATTN_ERR_INVALID_ARG);
      x.n = 0;
    }
    const long long end = static_cast<long long>(x.len) + x.n;
    if (x.n == 0 || x.len < 0) return x;
    if (end > static_cast<long long>(M) * page_size) {
      record_status(report, ATTN_ERR_INVALID_ARG);
      return x;
    }
    x.lo = by_page.div(x.len);
    x.hi = by_page.div(static_cast<int>(end) - 1) + 1;
    return x;
  }
  __device__ __forceinline__ int tokens(int n) const { return min(n, T + 1); }
  __device__ __forceinline__ int add_tokens(int a, int b) const {
    return static_cast<int>(min(static_cast<unsigned>(a) + b, static_cast<unsigned>(T) + 1));
  }
  // Exclusive prefix of the token counts over the CTA, as block_scan.
  __device__ __forceinline__ int token_scan(int x, int* smem, int& total) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl = add_tokens(incl, y);
    }
    const int excl = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 31) smem[warp] = incl;
    __syncthreads();
    int wincl = smem[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, wincl, off);
      if (lane >= off) wincl = add_tokens(wincl, y);
    }
    total = __shfl_sync(0xffffffffu, wincl, 31);
    const int before = __shfl_sync(0xffffffffu, wincl, max(warp - 1, 0));
    __syncthreads();
    return add_tokens(warp > 0 ? before : 0, lane > 0 ? excl : 0);
  }

  // Entries [i, i + N) of row b's slots from s on, copied (checked); entries that lack a
  // page of the row's new tokens are a worker's.
  template <int N>
  __device__ __forceinline__ void copy(int b, int s, const int (&e)[N], int* to) const {
    const Row x = row(b, nullptr);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int page = checked_entry(e[i], P, status);
      if (page >= 0 || s + i < x.lo || s + i >= x.hi) to[i] = page;
    }
  }
  // The table, by CTA `part` of `parts`.
  __device__ void copy_table(int part, int parts) const {
    const unsigned tid = part * kThreads + threadIdx.x, n_threads = parts * kThreads;
    const unsigned entries = static_cast<unsigned>(B) * M;
    if (table_vec) {
      for (unsigned i = tid; i < entries / 4; i += n_threads) {
        const int4 x = reinterpret_cast<const int4*>(table)[i];
        const int e[4] = {x.x, x.y, x.z, x.w};
        const int b = by_row.div(i), s = 4 * (i - b * (M / 4));
        const Row r = row(b, nullptr);
        if (s + 4 <= r.lo || s >= r.hi) {
          reinterpret_cast<int4*>(table_out)[i] =
              make_int4(checked_entry(x.x, P, status), checked_entry(x.y, P, status),
                        checked_entry(x.z, P, status), checked_entry(x.w, P, status));
        } else {
          copy(b, s, e, table_out + 4 * static_cast<size_t>(i));
        }
      }
    } else {
      for (unsigned i = tid; i < entries; i += n_threads) {
        const int e[1] = {table[i]};
        const int b = by_row.div(i);
        copy(b, i - b * M, e, table_out + i);
      }
    }
  }

  // Pages [begin, end) of one of the workers' warps, numbered over all of them.
  __device__ __forceinline__ void warp_pages(int w, int& begin, int& end) const {
    const int warps = workers * kWarps;
    const int chunk = ((P + warps - 1) / warps + 127) & ~127;
    begin = static_cast<int>(min(static_cast<long long>(w) * chunk, static_cast<long long>(P)));
    end = static_cast<int>(min(static_cast<long long>(begin) + chunk, static_cast<long long>(P)));
  }
  // The free pages among this warp's [begin, end), 128 at a time, four to a lane as bits:
  // f(round, bits), with several rounds' loads on their way at once.
  template <typename F>
  __device__ __forceinline__ void each_free(int begin, int end, F f) const {
    constexpr int kAtOnce = 8;
    const int lane = threadIdx.x & 31;
    for (int i0 = 0; begin + 128 * i0 < end; i0 += kAtOnce) {
      int4 c[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int p = begin + 128 * (i0 + i) + 4 * lane;
        c[i] = make_int4(1, 1, 1, 1);
        if (refs_vec && p + 4 <= end) {
          c[i] = *reinterpret_cast<const int4*>(refs + p);
        } else if (p < end) {
          c[i].x = refs[p];
          if (p + 1 < end) c[i].y = refs[p + 1];
          if (p + 2 < end) c[i].z = refs[p + 2];
          if (p + 3 < end) c[i].w = refs[p + 3];
        }
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (begin + 128 * (i0 + i) < end)
          f(i0 + i, (c[i].x == 0) | (c[i].y == 0) << 1 | (c[i].z == 0) << 2 | (c[i].w == 0) << 3);
    }
  }
  // The counts of pages that have holders (free pages are the workers'), by CTA `part` of `parts`.
  __device__ void copy_refs(int part, int parts) const {
    if (refs_out == refs) return;
    const unsigned tid = part * kThreads + threadIdx.x, n_threads = parts * kThreads;
    const unsigned vecs = refs_vec ? P / 4 : 0;
    for (unsigned i = tid; i < vecs; i += n_threads) {
      const int4 c = reinterpret_cast<const int4*>(refs)[i];
      if (c.x != 0 && c.y != 0 && c.z != 0 && c.w != 0) {
        reinterpret_cast<int4*>(refs_out)[i] = c;
      } else {
        const int e[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (e[j] != 0) refs_out[4 * i + j] = e[j];
      }
    }
    for (unsigned p = 4 * vecs + tid; p < static_cast<unsigned>(P); p += n_threads) {
      const int c = refs[p];
      if (c != 0) refs_out[p] = c;
    }
  }
  static constexpr int kKept = 16;  // rounds of each_free whose bits a warp keeps

  // What a worker's CTA shares between its threads.
  struct Shared {
    int sums[32];
    // Of rows: their slots, how many of them lack a page (later the number of their first page,
    // or -1), and which, as far as a word says it.
    int lo[kThreads], hi[kThreads], lacking[kThreads];
    unsigned mask[kThreads];
    uint8_t shares[kThreads];  // would write into a page of several holders
    int starts[kThreads];
    uint8_t free_bits[kWarps][kKept * 32];  // four pages each
  };
  // What a thread keeps from phase to phase where the worker's rows are no more than its
  // threads: its row.
  struct Mine {
    Row x;
    int lacking, k, t;
    bool shares;
  };
  // The slots of the row at place i of `lo` and `hi`, eight lanes to a row, or all to a row
  // of more slots: f(place, slot, lanes) with `lanes` the mask of those that share the row, in
  // turns of eight or 32 slots; slots from hi on are nobody's (-1).
  template <typename F>
  __device__ __forceinline__ void each_slot(const Shared& sh, int i, F f) const {
    const int lane = threadIdx.x & 31;
    const int lo = sh.lo[i], hi = sh.hi[i];
    if (hi - lo <= 8) {
      if (lo < hi) f(i, lo + (lane & 7) < hi ? lo + (lane & 7) : -1, 0xffu << (lane & 24));
    }
    __syncwarp();
    for (unsigned left = __ballot_sync(0xffffffffu, hi - lo > 8 && (lane & 7) == 0); left != 0;
         left &= left - 1) {
      const int l = __ffs(left) - 1;
      const int ii = __shfl_sync(0xffffffffu, i, l), end = sh.hi[ii];
      for (int s = sh.lo[ii] + lane; s - lane < end; s += 32) f(ii, s < end ? s : -1, 0xffffffffu);
    }
  }
  static constexpr int kRowsAtOnce = kThreads / 8;
  __device__ __forceinline__ int entry(int r, int s, int* report) const {
    return checked_entry(table[static_cast<size_t>(r) * M + s], P, report);
  }

  // Worker w of the pages and rows.
  __device__ void run(int ph, int w, Mine& my, Shared& sh) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (B + workers - 1) / workers;
    const int r_begin = min(w * per, B), r_end = min(r_begin + per, B);
    const bool one = r_end - r_begin <= kThreads;  // a row a thread
    int p_begin, p_end;
    warp_pages(w * kWarps + warp, p_begin, p_end);
    if (ph == 0) {
      // The first rows' lengths, on their way with the pages' counts.
      int length = 0, more = 0;
      if (r_begin + static_cast<int>(threadIdx.x) < r_end) {
        length = seqlens[r_begin + threadIdx.x];
        more = new_lens[r_begin + threadIdx.x];
      }
      int n = 0;
      each_free(p_begin, p_end, [&](int i, unsigned bits) {
        if (bits != 0 && refs_out != refs) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (bits >> j & 1u) refs_out[p_begin + 128 * i + 4 * lane + j] = 0;
        }
        if (i < kKept) sh.free_bits[warp][32 * i + lane] = static_cast<uint8_t>(bits);
        n += __popc(bits);
      });
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) warp_free[w * kWarps + warp] = sh.sums[warp] = n;
      __syncthreads();
      if (warp == 0) {
        const int all = __reduce_add_sync(0xffffffffu, sh.sums[lane]);
        if (lane == 0) cta_free[w] = all;
      }
      int at = 0, tok = 0;
      for (int r0 = r_begin; r0 < r_end; r0 += kThreads) {
        const int r = r0 + threadIdx.x;
        Row x = {0, 0, 0, 0};
        if (r < r_end) x = r0 == r_begin ? row(length, more, nullptr) : row(r, nullptr);
        sh.lo[threadIdx.x] = x.lo;
        sh.hi[threadIdx.x] = x.hi;
        sh.lacking[threadIdx.x] = 0;
        sh.shares[threadIdx.x] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < min(kThreads, r_end - r0); i0 += kRowsAtOnce)
          each_slot(sh, i0 + (threadIdx.x >> 3), [&](int i, int s, unsigned lanes) {
            // (Bad entries are reported here: in place, a page may be in one's stead by the time
            // that a CTA that copies looks.)
            const int page = s >= 0 ? entry(r0 + i, s, status) : 0;
            const unsigned votes = __ballot_sync(lanes, page < 0);
            if (s >= 0 && page >= 0 && refs[page] > 1) sh.shares[i] = 1;
            if (lane == __ffs(lanes) - 1) {
              sh.lacking[i] += __popc(votes);
              sh.mask[i] = votes >> (__ffs(lanes) - 1);  // (of one turn; see `word`)
            }
          });
        __syncthreads();
        int total, tok_total;
        const bool shares = sh.shares[threadIdx.x] != 0;
        const int lacking = shares ? 0 : sh.lacking[threadIdx.x];
        const int k = at + block_scan(lacking, sh.sums, total);
        const int t = add_tokens(tok, token_scan(tokens(x.n), sh.sums, tok_total));
        if (one) {
          my.x = x;
          my.lacking = lacking;
          my.k = k;
          my.t = t;
          my.shares = shares;
        } else if (r < r_end) {
          need[r] = k;
          first[r] = t;
          len[r] = shares ? -1 : 0;  // (for the next phase)
        }
        at += total;
        tok = add_tokens(tok, tok_total);
      }
      if (threadIdx.x == 0) {
        cta_need[w] = at;
        cta_tokens[w] = tok;
      }
      return;
    }
    // What the workers before this one have, and all of them (at most 32 workers).
    int free_before = 0, free_all = 0, need_before = 0, need_all = 0, first_token = 0;
    const int warp_has = ph == 1 ? warp_free[w * kWarps + lane] : 0;
    if (ph == 1 || !one) {
      const int f = lane < workers ? cta_free[lane] : 0, q = lane < workers ? cta_need[lane] : 0;
      int t = lane < w ? cta_tokens[lane] : 0;
      free_all = __reduce_add_sync(0xffffffffu, f);
      need_all = __reduce_add_sync(0xffffffffu, q);
      free_before = __reduce_add_sync(0xffffffffu, lane < w ? f : 0);
      need_before = __reduce_add_sync(0xffffffffu, lane < w ? q : 0);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) t = add_tokens(t, __shfl_xor_sync(0xffffffffu, t, off));
      first_token = t;
    }
    if (ph == 1) {
      const int wanted = min(need_all, free_all);
      int at = free_before + __reduce_add_sync(0xffffffffu, lane < warp ? warp_has : 0);
      const int rounds = (p_end - p_begin + 127) / 128;
      if (at < wanted && rounds <= kKept) {
        // A run of each lane's own, so that one prefix sum ranks them.
        const uint8_t* mine = sh.free_bits[warp] + lane * rounds;
        int n = 0;
        for (int i = 0; i < rounds; ++i) n += __popc(mine[i]);
        int k = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, k, off);
          if (lane >= off) k += y;
        }
        k += at - n;
        for (int i = 0; i < rounds; ++i)
          for (unsigned bits = mine[i]; bits != 0; bits &= bits - 1) {
            if (k < wanted) free_list[k] = p_begin + 4 * (lane * rounds + i) + __ffs(bits) - 1;
            ++k;
          }
      } else if (at < wanted) {
        each_free(p_begin, p_end, [&](int i, unsigned bits) {
          if (at >= wanted || !__any_sync(0xffffffffu, bits != 0)) return;
          const unsigned below = (1u << lane) - 1u;
          int k = at;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const unsigned votes = __ballot_sync(0xffffffffu, bits >> j & 1u);
            k += __popc(votes & below);
            at += __popc(votes);
          }
          for (; bits != 0; bits &= bits - 1) {
            if (k < wanted) free_list[k] = p_begin + 128 * i + 4 * lane + __ffs(bits) - 1;
            ++k;
          }
        });
      }
      // Which rows take their tokens: those whose pages and whose places in the step's T
      // suffice.  (Each row's lengths are read for the last time here, by the thread that
      // writes the new one: the two arrays may be one.)
      for (int r = r_begin + threadIdx.x; r < r_end; r += kThreads) {
        const Row x = one ? row(my.x.len, new_lens[r], status) : row(r, status);
        const int after = need_before + (one             ? my.k + my.lacking
                                         : r + 1 < r_end ? need[r + 1]
                                                         : cta_need[w]);
        const int t = add_tokens(first_token, one ? my.t : first[r]);
        const int end = add_tokens(t, tokens(x.n));
        const bool shares = one ? my.shares : len[r] < 0;
        bool takes = x.lo < x.hi && !shares;
        if (end > T || shares) {
          record_status(status, ATTN_ERR_INVALID_ARG);
          takes = false;
        }
        takes = takes && after <= free_all;
        cu[r + 1] = min(end, T);
        len[r] = takes ? x.len : -1;
        if (one) {
          sh.lacking[threadIdx.x] = takes ? need_before + my.k : -1;
          seqlens_out[r] = takes ? x.len + x.n : x.len;
        }
      }
      if (w == 0 && threadIdx.x == 0) {
        cu[0] = 0;
        counts[0] = need_all;
        counts[1] = free_all;
        if (need_all > free_all) record_status(status, ATTN_ERR_NO_PAGES);
      }
      return;
    }
    // Pages for the rows' slots that lack one (-1 for those of rows that take none).
    for (int r0 = r_begin; r0 < r_end; r0 += kThreads) {
      const int r = r0 + threadIdx.x;
      if (!one) {
        Row x = {0, 0, 0, 0};
        int k0 = -1;
        if (r < r_end) {
          x = row(r, nullptr);
          if (len[r] >= 0) k0 = need_before + need[r];
        }
        __syncthreads();
        sh.lo[threadIdx.x] = x.lo;
        sh.hi[threadIdx.x] = x.hi;
        sh.lacking[threadIdx.x] = k0;
        __syncthreads();
      }
      for (int i0 = 0; i0 < min(kThreads, r_end - r0); i0 += kRowsAtOnce)
        each_slot(sh, i0 + (threadIdx.x >> 3), [&](int i, int s, unsigned lanes) {
          const int leader = __ffs(lanes) - 1;
          // One turn's slots are known from phase 1.
          const bool word = one && sh.hi[i] - sh.lo[i] <= __popc(lanes);
          const bool lacking =
              word ? sh.mask[i] >> (lane - leader) & 1u : s >= 0 && entry(r0 + i, s, nullptr) < 0;
          const unsigned votes = __ballot_sync(lanes, lacking);
          const int k = sh.lacking[i];
          __syncwarp(lanes);
          if (lane == leader && k >= 0) sh.lacking[i] = k + __popc(votes);
          __syncwarp(lanes);
          if (lacking) {
            const int page = k >= 0 ? free_list[k + __popc(votes & ((1u << lane) - 1u))] : -1;
            table_out[static_cast<size_t>(r0 + i) * M + s] = page;
            if (page >= 0) refs_out[page] = 1;
          }
        });
    }
    if (one) return;
    __syncthreads();
    for (int r = r_begin + threadIdx.x; r < r_end; r += kThreads) {
      const int x = seqlens[r];
      seqlens_out[r] = len[r] >= 0 ? x + new_lens[r] : x;
    }
  }
  // Positions and slots of the tokens, shared out over the workers.
  __device__ void run_tokens(int w, Shared& sh) const {
    int* const starts = sh.starts;
    // Every step-th row's first token, for a search that seldom leaves the CTA.
    const int step = (B + kStarts - 1) / kStarts, n = (B + step - 1) / step;
    for (int i = threadIdx.x; i < n; i += kThreads) starts[i] = cu[i * step];
    __syncthreads();
    for (int t = w * kThreads + threadIdx.x; t < T; t += workers * kThreads) {
      // The last row whose tokens begin at or before t (rows before it may have none).
      int lo = 0, hi = n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (starts[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
      lo *= step;
      hi = min(lo + step, B);
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
      int pos = 0, slot = -1;
      const int from = len[lo], t0 = cu[lo], t1 = cu[lo + 1];
      if (t < t1 && from >= 0) {
        pos = from + t - t0;
        const int s = by_page.div(pos);
        const size_t at = static_cast<size_t>(lo) * M + s;
        int page = checked_entry(table[at], P, nullptr);
        if (page < 0) page = table_out[at];  // a worker's (in place: already read)
        slot = page * page_size + pos - s * page_size;
      }
      positions[t] = pos;
      slots[t] = slot;
    }
  }
  static constexpr int kStarts = kThreads;

  // One CTA, everything in shared memory between one trip for the inputs and the stores: a thread
  // per row, and one prefix sum for its tokens, its lacking pages and a run of free pages.
  static size_t small_bytes(long long entries, int P, int B) {
    return (entries + pad(P) + P + 2ll * B + 1) * sizeof(int);
  }
  __device__ void run_small(unsigned long long* sums, int* lists) const {
    const int t = threadIdx.x, entries = B * M;
    int* const page_of = lists;           // the table
    int* const held = page_of + entries;  // refs
    int* const free_at = held + pad(P);   // free pages, ascending
    int* const begin = free_at + P;       // rows' first tokens (B + 1)
    int* const taken = begin + B + 1;     // rows' lengths before, or -1
    const int length = t < B ? seqlens[t] : 0, more = t < B ? new_lens[t] : 0;
    for (int i = t; i < entries; i += kThreads) page_of[i] = checked_entry(table[i], P, status);
    for (int p = t; p < P; p += kThreads) held[pad(p)] = refs[p];
    const Row x = row(length, more, status);
    __syncthreads();
    const int per = (P + kThreads - 1) / kThreads;  // pages of a thread, in one run
    const int p0 = min(t * per, P), p1 = min(p0 + per, P);
    int n_free = 0, lacking = 0;
    for (int p = p0; p < p1; ++p) n_free += held[pad(p)] == 0;
    bool shares = false;
    for (int s = x.lo; s < x.hi; ++s) {
      const int page = page_of[t * M + s];
      lacking += page < 0;
      shares |= page >= 0 && held[pad(page)] > 1;
    }
    if (shares) lacking = 0;
    // (Fields of 30, 17 and 17 bits: rows <= 2^10, tokens clamped to T + 1 < 2^13, entries and
    // pages <= 2^13.)
    const unsigned long long mine = static_cast<unsigned long long>(tokens(x.n)) |
                                    static_cast<unsigned long long>(lacking) << 30 |
                                    static_cast<unsigned long long>(n_free) << 47;
    unsigned long long incl = mine;
    const int lane = t & 31, warp = t >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    unsigned long long warps = sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, warps, off);
      if (lane >= off) warps += y;
    }
    const unsigned long long all = __shfl_sync(0xffffffffu, warps, 31);
    unsigned long long before = __shfl_sync(0xffffffffu, warps, max(warp - 1, 0));
    before = (warp > 0 ? before : 0) + incl - mine;
    const auto token_field = [&](unsigned long long v) {
      return min(static_cast<int>(v & ((1u << 30) - 1)), T + 1);
    };
    const auto field = [](unsigned long long v, int at) {
      return static_cast<int>(v >> at & 0x1ffff);
    };
    int f = field(before, 47);
    for (int p = p0; p < p1; ++p)
      if (held[pad(p)] == 0) free_at[f++] = p;
    const int free_all = field(all, 47), need_all = field(all, 30);
    int k = field(before, 30);
    const int t0 = token_field(before), t1 = token_field(before + mine);
    if (t < B && (t1 > T || shares)) record_status(status, ATTN_ERR_INVALID_ARG);
    const bool takes =
        t < B && x.lo < x.hi && !shares && t1 <= T && k + lacking <= free_all;
    if (t < B) {
      begin[t] = min(t0, T);
      taken[t] = takes ? x.len : -1;
      cu[t] = min(t0, T);
      seqlens_out[t] = takes ? x.len + x.n : length;
    }
    if (t == B - 1) begin[B] = cu[B] = min(t1, T);
    if (t == 0) {
      counts[0] = need_all;
      counts[1] = free_all;
      if (need_all > free_all) record_status(status, ATTN_ERR_NO_PAGES);
    }
    __syncthreads();
    if (takes)
      for (int s = x.lo; s < x.hi; ++s)
        if (page_of[t * M + s] < 0) {
          const int page = free_at[k++];
          page_of[t * M + s] = page;
          held[pad(page)] = 1;
        }
    __syncthreads();
    for (int i = t; i < entries; i += kThreads) table_out[i] = page_of[i];
    for (int p = t; p < P; p += kThreads) refs_out[p] = held[pad(p)];
    for (int i = t; i < T; i += kThreads) {
      int lo = 0, hi = B;  // the last row whose tokens begin at or before i
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (begin[mid] <= i)
          lo = mid;
        else
          hi = mid;
      }
      int pos = 0, slot = -1;
      if (i < begin[lo + 1] && taken[lo] >= 0) {
        pos = taken[lo] + i - begin[lo];
        const int s = by_page.div(pos);
        slot = page_of[lo * M + s] * page_size + pos - s * page_size;
      }
      positions[i] = pos;
      slots[i] = slot;
    }
  }
};

__global__ void __launch_bounds__(kThreads, 1) pages_append_small_kernel(const AppendOp op) {
  __shared__ unsigned long long sums[32];
  extern __shared__ int lists[];
  grid_dependency_wait();
  grid_launch_dependents();
  op.run_small(sums, lists);
}

// A cluster of workers and further CTAs that copy (without those the workers do).
__global__ void __launch_bounds__(kThreads, 1) pages_append_kernel(const AppendOp op) {
  __shared__ AppendOp::Shared sh;
  grid_dependency_wait();
  grid_launch_dependents();
  const int w = blockIdx.x;
  if (w >= op.workers) {
    op.copy_refs(w - op.workers, gridDim.x - op.workers);
    op.copy_table(w - op.workers, gridDim.x - op.workers);
    return;
  }
  if (static_cast<int>(gridDim.x) == op.workers) {
    op.copy_refs(w, op.workers);
    op.copy_table(w, op.workers);
  }
  AppendOp::Mine my = {};
  for (int ph = 0; ph < 3; ++ph) {
    op.run(ph, w, my, sh);
    cluster_sync();
  }
  op.run_tokens(w, sh);
}

// ------------------------------------------------------------------ copies
// A CTA per 32 KB of a page, every load in flight before the first store, both marked
// as used once (evict-first).  Bound by HBM: 4000 pages of 2 x 64 KB in 161.7 us, 6484
// GB/s, 96 % of a plain copy's rate; without the marks 166.1, 16 KB a CTA 170.2, a
// persistent grid of 8 CTAs an SM 169.7.
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;  // 16-byte vectors a thread: 32 KB a CTA

__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(uint4* k, uint4* v, const int* __restrict__ src, const int* __restrict__ dst,
                      int num_pages, long long page_vecs, int chunks, int* status) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int pair = blockIdx.y;
  const int from = __ldg(src + pair), to = __ldg(dst + pair);
  if (from == -1 && to == -1) return;
  if (from < 0 || to < 0 || from >= num_pages || to >= num_pages) {
    if (threadIdx.x == 0) record_status(status, ATTN_ERR_INVALID_ARG);
    return;
  }
  uint4* base = blockIdx.x < chunks ? k : v;
  const long long c = static_cast<long long>(blockIdx.x % chunks) * (kCopyThreads * kCopyVecs);
  const uint4* a = base + from * page_vecs;
  uint4* b = base + to * page_vecs;
  uint4 x[kCopyVecs];
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const long long at = c + i * kCopyThreads + threadIdx.x;
    if (at < page_vecs) x[i] = __ldcs(a + at);
  }
#pragma unroll
  for (int i = 0; i < kCopyVecs; ++i) {
    const long long at = c + i * kCopyThreads + threadIdx.x;
    if (at < page_vecs) __stcs(b + at, x[i]);
  }
}

// ------------------------------------------------------------------ host side
template <typename Op>
cudaError_t launch_small(const Op& op, size_t smem, cudaStream_t stream) {
  if (smem > 48 * 1024) {
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(pages_small_kernel<Op>),
                                           static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_programmatic(pages_small_kernel<Op>, dim3(1), dim3(kThreads), smem, stream, op);
}

// work: elements of the largest array.
template <typename Op>
cudaError_t launch_phases(const Op& op, long long work, cudaStream_t stream) {
  if (work <= kClusterWork) {
    const auto kernel = pages_phases_kernel<Op, kCluster>;
    const cudaError_t e = allow_large_cluster(reinterpret_cast<const void*>(kernel));
    if (e != cudaSuccess) return e;
    return launch_programmatic_cluster(kernel, dim3(kClusterCtas), dim3(kThreads), 0, stream,
                                       kClusterCtas, op);
  }
  const long long ctas = (work + kThreads - 1) / kThreads;
  const int most = sm_count() < kPagesMaxCtas ? sm_count() : kPagesMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_phases_kernel<Op, kGrid>, op);
  return e != cudaSuccess ? e : cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

cudaError_t launch_pages_free(const int* table, const int* refs, const int* seqlens,
                              int* table_out, int* refs_out, int B, int M, int P, int page_size,
                              int window, int sinks, int room, cudaStream_t stream, int* status) {
  FreeOp op{table, refs, seqlens, table_out, refs_out, B, M, P, page_size, window, sinks, room};
  op.refs_vec = aligned16(refs) && aligned16(refs_out);
  op.table_vec = M % 4 == 0 && aligned16(table) && aligned16(table_out);
  op.by_row = FixedDiv(op.table_vec ? M / 4 : M);
  op.status = status;
  const long long entries = static_cast<long long>(B) * M;
  return launch_phases(op, entries > P ? entries : P, stream);
}

cudaError_t launch_pages_fork(const int* table, const int* refs, const int* seqlens,
                              const int* parents, int* table_out, int* refs_out, int* seqlens_out,
                              int* src, int* dst, int* counts, int* workspace, int B, int R, int M,
                              int P, int page_size, int room, cudaStream_t stream, int* status) {
  ForkOp op{table, refs, seqlens, parents, table_out, refs_out, seqlens_out, src, dst, counts};
  op.lowest = workspace;
  op.free_list = op.lowest + P;
  op.cta_free = op.free_list + P;
  op.cta_need = op.cta_free + kPagesMaxCtas;
  op.need = op.cta_need + kPagesMaxCtas;
  op.live = reinterpret_cast<unsigned*>(op.need + R);
  op.B = B;
  op.R = R;
  op.M = M;
  op.P = P;
  op.page_size = page_size;
  op.room = room < M * page_size ? room : M * page_size;  // further keys have no slots
  op.by_page = FixedDiv(page_size);
  op.by_row = FixedDiv(M);
  op.by_writable = FixedDiv(ForkOp::small_slots(op.room, page_size));
  op.status = status;
  const long long entries = static_cast<long long>(B > R ? B : R) * M;
  if (entries <= kSmallForkEntries && P <= kSmallForkPages &&
      static_cast<long long>(R) * ForkOp::small_slots(op.room, page_size) <= kSmallForkSlots)
    return launch_small(op, ForkOp::small_bytes(P, R), stream);
  return launch_phases(op, entries > P ? entries : P, stream);
}

cudaError_t launch_pages_append(const int* table, const int* refs, const int* seqlens,
                                const int* new_lens, int* table_out, int* refs_out,
                                int* seqlens_out, int* cu, int* positions, int* slots, int* counts,
                                int* workspace, int B, int T, int M, int P, int page_size,
                                cudaStream_t stream, int* status) {
  AppendOp op{table, refs, seqlens, new_lens, table_out, refs_out, seqlens_out,
              cu, positions, slots, counts};
  op.free_list = workspace;
  op.warp_free = op.free_list + P;
  op.cta_free = op.warp_free + kClusterCtas * kWarps;
  op.cta_need = op.cta_free + kClusterCtas;
  op.cta_tokens = op.cta_need + kClusterCtas;
  op.need = op.cta_tokens + kClusterCtas;
  op.first = op.need + B;
  op.len = op.first + B;
  op.B = B;
  op.M = M;
  op.P = P;
  op.T = T;
  op.page_size = page_size;
  op.by_page = FixedDiv(page_size);
  op.refs_vec = aligned16(refs) && aligned16(refs_out);
  op.table_vec = M % 4 == 0 && aligned16(table) && aligned16(table_out);
  op.by_row = FixedDiv(op.table_vec ? M / 4 : M);
  op.status = status;
  const long long entries = static_cast<long long>(B) * M;
  if (entries <= kSmallAppendEntries && P <= kSmallAppendPages && B <= kThreads &&
      T <= kSmallAppendTokens && T <= kSmallAppendSlots * page_size) {
    const size_t smem = AppendOp::small_bytes(entries, P, B);
    const auto small = pages_append_small_kernel;
    const cudaError_t e =
        ensure_smem_attr(reinterpret_cast<const void*>(small), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_programmatic(small, dim3(1), dim3(kThreads), smem, stream, op);
  }
  op.workers = kClusterCtas;
  const auto kernel = pages_append_kernel;
  const cudaError_t e = allow_large_cluster(reinterpret_cast<const void*>(kernel));
  if (e != cudaSuccess) return e;
  // Eight entries or pages a thread for clusters that copy.  They read the rows' lengths whenever they
  // run, so that lengths updated in place leave the copy to the workers.
  long long copiers = (entries > P ? entries : P) / (8ll * kThreads * kClusterCtas);
  if (copiers > kMaxCopiers) copiers = kMaxCopiers;
  if (seqlens_out == seqlens) copiers = 0;
  return launch_programmatic_cluster(kernel, dim3(static_cast<unsigned>((1 + copiers) * kClusterCtas)),
                                     dim3(kThreads), 0, stream, kClusterCtas, op);
}

cudaError_t launch_pages_compact(const int* table, const int* refs, int* table_out, int* refs_out,
                                 int* src, int* dst, int* num_live, int* workspace, int B, int M,
                                 int P, cudaStream_t stream, int* status) {
  CompactOp op{table, refs, table_out, refs_out, src, dst, num_live};
  op.rank = workspace;
  op.cta_live = workspace + P;
  op.B = B;
  op.M = M;
  op.P = P;
  op.status = status;
  const long long entries = static_cast<long long>(B) * M;
  if (entries <= kSmallCompactEntries && P <= kSmallCompactPages)
    return launch_small(op, CompactOp::small_bytes(P), stream);
  return launch_phases(op, entries > P ? entries : P, stream);
}

cudaError_t launch_pages_copy(void* k, void* v, const int* src, const int* dst, int n,
                              int num_pages, long long page_bytes, cudaStream_t stream,
                              int* status) {
  const long long vecs = page_bytes / 16;
  const int chunks =
      static_cast<int>((vecs + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs));
  // At most 65535 pairs in the grid's y.
  for (int at = 0; at < n; at += 65535) {
    const int m = n - at < 65535 ? n - at : 65535;
    const cudaError_t e = launch_programmatic(
        pages_copy_kernel, dim3(2 * chunks, m, 1), dim3(kCopyThreads), 0, stream,
        static_cast<uint4*>(k), static_cast<uint4*>(v), src + at, dst + at, num_pages, vecs, chunks,
        status);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace attn
