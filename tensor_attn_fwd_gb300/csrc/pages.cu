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
constexpr long long kClusterWork = 1 << 15;
constexpr int kClusterCtas = 16;  // past the portable 8: the kernels opt in

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
