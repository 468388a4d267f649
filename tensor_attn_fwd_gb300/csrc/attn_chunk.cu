// attn_chunk.cu -- attention of a step's new tokens over a paged cache: a plan of the
// work, built on the GPU from the requests' lengths, and the kernels that carry it out.
//
// Request b has n_b new tokens (packed one request after the other) and seqlens[b] keys in
// its pages, the new tokens' own among them.  Its token i stands at p = seqlens[b] - n_b + i
// and sees key j iff  j <= p  and  (j > p - window  or  j < sinks); in one pass over the
// keys (Background, Equ. 1 of the page that attn_fwd.cu cites)
//   O = softmax(Q K^T * scale) V,   LSE = ln sum_j exp(S_ij).
//
// Rows.  The query heads of a KV head read the same K/V, so a query tile's 128 rows are
// tokens x heads of one KV head: row r is token r / slice_heads, head r % slice_heads (one
// TMA box of [tokens][heads][64 dims] lays them out so).  A request with one new token
// fills a few rows, a prompt all of them.
//
// Items.  An item is two such tiles of a request and KV head, which stream the same K/V
// tiles of 128 keys: the tensor core works on one tile while the other's softmax runs.
// An item whose tokens fit one tile takes both tile slots for it, which share out its K/V
// tiles by turns (two softmax states, merged at the end), for the same overlap.
//
// Plan.  Requests differ in their numbers of tokens and keys, so the items' K/V tiles are
// put in one line and cut into equal parts, one for each CTA; an item that is cut leaves
// partial results, which a second kernel merges by their LSE (attn_combine's formula).
// The plan depends on the lengths alone: one serves all layers of a step.
//
// Pages.  A K/V tile is loaded as boxes of 32, 64 or 128 keys (what divides the page), each
// found through the block table; boxes that no row sees are filled with zeros by a load
// past the cache's end, and their table entries are not read.
//
// Roles, tensor memory and the online softmax are attn_fwd.cu's.
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

constexpr int kMagic = 0x43484b31;
constexpr int kMaxKeys = 1 << 30;  // of a request
// A piece's cost around its K/V tiles, in tiles.
constexpr int kOverhead = 1;
// An item is cut no closer than this to its ends (in tiles): a cut costs partial results.
constexpr int kSnap = 2;
// Cost that is worth a CTA of its own.
constexpr int kMinShare = 4;

__device__ __forceinline__ void record_status(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// The plan's header.
struct PlanHeader {
  int magic, B, T, Hq, Hkv, D, max_keys, window, sinks, ctas;
  int n_pieces, n_cuts;
  int pad[kChunkHeader - 12];
};
static_assert(sizeof(PlanHeader) == kChunkHeader * sizeof(int), "header size");

// A run of K/V tiles of an item.
struct alignas(16) Piece {
  int token, tokens;  // first packed token, their number (1 to 2 tiles' worth)
  int pos;            // the first one's position
  int row;            // request
  int head;           // KV head * slices + slice
  int begin, end;     // K/V tiles, in the order of the item's list
  int part;           // slot of its partial result; -1: it is the whole item
};
static_assert(sizeof(Piece) == kChunkRecord * sizeof(int), "record size");
// An item in pieces: partial results [part, part + parts).
struct alignas(16) Cut {
  int token, tokens, head, part, parts;
  int pad[3];
};
static_assert(sizeof(Cut) == kChunkRecord * sizeof(int), "record size");

// The K/V tiles that `tokens` tokens from position `pos` on see: sink tiles [0, s), then
// [w, e); e = 0: none.
struct KvTiles {
  int s, w, e;
  int lo, hi;  // keys: some row sees [lo, hi) and [0, sinks)
  __device__ __forceinline__ KvTiles(int pos, int tokens, int window, int sinks) {
    hi = max(pos + tokens, 0);
    lo = max(pos - window + 1, 0);
    e = (hi + 127) / 128;
    w = min(lo / 128, e);
    s = min((min(sinks, hi) + 127) / 128, w);
  }
  __device__ __forceinline__ int count() const { return s + e - w; }
  __device__ __forceinline__ int tile(int k) const { return k < s ? k : k - s + w; }
};

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// Exclusive prefix sum of one value per thread over the CTA; total: their sum.
template <typename X>
__device__ __forceinline__ X scan(X x, X* smem, X& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  X incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const X y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) smem[warp] = incl;
  __syncthreads();
  const X w = smem[lane];
  X wincl = w;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const X y = __shfl_up_sync(0xffffffffu, wincl, off);
    if (lane >= off) wincl += y;
  }
  total = __shfl_sync(0xffffffffu, wincl, 31);
  const X before = __shfl_sync(0xffffffffu, wincl - w, warp);
  __syncthreads();
  return before + incl - x;
}

struct PlanParams {
  const int *cu, *seqlens;
  int* plan;
  int B, T, Hq, Hkv, D, max_keys, window, sinks, ctas;
  int heads, item_tokens;  // KV heads x slices; tokens of an item
  long long max_items;
  int* status;
};

__global__ void __launch_bounds__(kPlanThreads, 1) chunk_plan_kernel(const PlanParams p) {
  __shared__ long long smem[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const ChunkLayout at(p.B, p.max_items, p.ctas);
  PlanHeader* const header = reinterpret_cast<PlanHeader*>(p.plan);
  int* const begins = p.plan + at.begins;
  Cut* const cuts = reinterpret_cast<Cut*>(p.plan + at.cuts);
  int* const tiles = p.plan + at.tiles;  // a KV head's items of the requests before
  Piece* const pieces = reinterpret_cast<Piece*>(p.plan + at.pieces);
  const int tid = threadIdx.x;

  // Packed tokens of a request (bad bounds: none).
  const auto tokens_of = [&](int b, int* report) {
    const int t0 = p.cu[b], t1 = p.cu[b + 1];
    if (t0 >= 0 && t0 <= t1 && t1 <= p.T) return t1 - t0;
    record_status(report, ATTN_ERR_INVALID_ARG);
    return 0;
  };
  long long n_tiles = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    const long long n = b < p.B ? (tokens_of(b, p.status) + p.item_tokens - 1) / p.item_tokens : 0;
    long long total;
    const long long before = n_tiles + scan(n, smem, total);
    // (Past the plan's capacity they are not used.)
    if (b < p.B) tiles[b] = static_cast<int>(min(before, 1ll << 30));
    n_tiles += total;
  }
  if (tid == 0) tiles[p.B] = static_cast<int>(min(n_tiles, 1ll << 30));
  __syncthreads();
  // Overlapping requests could need more items than the plan holds.
  const bool fits = n_tiles * p.heads <= p.max_items;
  if (!fits) record_status(p.status, ATTN_ERR_INVALID_ARG);
  const int items = fits ? static_cast<int>(n_tiles) * p.heads : 0;

  // Item i: request by request, in each KV head by KV head, its tokens ascending.
  const auto item = [&](int i, Piece& x) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (static_cast<long long>(tiles[mid]) * p.heads <= i)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int first = tiles[lo], n = tiles[lo + 1] - first;
    const int rest = i - first * p.heads;
    const int t0 = p.cu[lo], n_tok = p.cu[lo + 1] - t0;
    const int len = min(max(p.seqlens[lo], 0), p.max_keys);
    x.row = lo;
    x.head = rest / n;
    const int from = (rest - x.head * n) * p.item_tokens;
    x.token = t0 + from;
    x.tokens = min(p.item_tokens, n_tok - from);
    x.pos = len - n_tok + from;
    x.begin = 0;
    x.end = KvTiles(x.pos, x.tokens, p.window, p.sinks).count();
    x.part = -1;
  };
  long long cost = 0;
  for (int i = tid; i < items; i += kPlanThreads) {
    Piece x;
    item(i, x);
    cost += x.end + kOverhead;
  }
  long long all;
  scan(cost, smem, all);
  const long long want = (all + kMinShare - 1) / kMinShare;
  const int n = want < p.ctas ? static_cast<int>(max(want, 1ll)) : p.ctas;

  // Part c of the line begins at all * c / n.
  long long line = 0;
  int before_cuts = 0, before_items = 0;  // so far: cuts, and items that are cut
  for (int i0 = 0; i0 < items; i0 += kPlanThreads) {
    const int i = i0 + tid;
    Piece x = {};
    int w = 0;
    if (i < items) {
      item(i, x);
      w = x.end + kOverhead;
    }
    long long total;
    const long long from = line + scan(static_cast<long long>(w), smem, total);
    line += total;
    // Parts that begin in this item, at their K/V tile (near its ends: at the end).
    const int c0 = max(1, static_cast<int>((from * n + all - 1) / max(all, 1ll)));
    const int steps = x.end;
    const auto cut_at = [&](int c) {
      const int off = static_cast<int>(all * c / n - from);
      const int k = static_cast<int>(static_cast<long long>(off) * steps / max(w, 1));
      return k < kSnap ? 0 : (steps - k < kSnap ? steps : k);
    };
    int n_cuts = 0;
    if (w > 0) {
      int last = 0;
      for (int c = c0; c < n && all * c / n < from + w; ++c) {
        const int k = cut_at(c);
        if (k > last && k < steps) {
          ++n_cuts;
          last = k;
        }
      }
    }
    // Cuts in the low half, cut items in the high one (at most one of each a CTA).
    long long sums;
    const long long rank = scan(static_cast<long long>(n_cuts) | (n_cuts > 0 ? 1ll << 32 : 0ll),
                                smem, sums);
    const int cuts_before = before_cuts + static_cast<int>(rank & 0xffffffff);
    const int items_before = before_items + static_cast<int>(rank >> 32);
    before_cuts += static_cast<int>(sums & 0xffffffff);
    before_items += static_cast<int>(sums >> 32);
    if (w > 0) {
      int piece = i + cuts_before;
      int part = n_cuts > 0 ? cuts_before + items_before : -1;
      if (n_cuts > 0) {
        Cut cut = {x.token, x.tokens, x.head, part, n_cuts + 1, {0, 0, 0}};
        cuts[items_before] = cut;
      }
      int last = 0;
      for (int c = c0; c < n && all * c / n < from + w; ++c) {
        const int k = cut_at(c);
        if (k > last && k < steps) {
          x.begin = last;
          x.end = k;
          x.part = part++;
          pieces[piece++] = x;
          last = k;
        }
        begins[c] = k < steps || steps == 0 ? (k == 0 ? i + cuts_before : piece)
                                            : i + cuts_before + n_cuts + 1;
      }
      x.begin = last;
      x.end = steps;
      x.part = part;
      pieces[piece] = x;
    }
  }
  const int n_pieces = items + before_cuts;
  for (int c = tid; c <= p.ctas; c += kPlanThreads) {
    if (c == 0) begins[c] = 0;
    if (c >= n || items == 0) begins[c] = c == 0 ? 0 : n_pieces;
  }
  if (tid == 0) {
    PlanHeader h = {kMagic, p.B, p.T, p.Hq, p.Hkv, p.D, p.max_keys, p.window, p.sinks, p.ctas,
                    n_pieces, before_items, {0, 0, 0, 0}};
    *header = h;
  }
}

// ------------------------------------------------------------------ attention
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr uint32_t kSubBytes = 128 * 128;  // one [128 rows x 64 bf16] swizzled sub-tile
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kLaunchRegs = 168;  // 65536 / 384, rounded down to a multiple of 8
constexpr uint32_t kRegsSoftmax = 200;
constexpr uint32_t kRegsOther = 104;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther == kThreads * kLaunchRegs,
              "register split must use exactly the launch allocation");
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kSub = D / 64;
  static constexpr uint32_t kTileBytes = kSub * kSubBytes;  // 128 x D bf16
  static constexpr int kStages = (D == 128) ? 5 : 9;
  static constexpr uint32_t kColS0 = 0, kColS1 = 128;
  static constexpr uint32_t kColO0 = 256, kColO1 = 256 + D;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kBarBytes = 512;
  static constexpr uint32_t kStatBytes = 2 * 128 * 2 * sizeof(float);
  // No room is left to align the tiles: the kernel has no static shared memory, so that the
  // dynamic one begins at a multiple of 1024 (and it looks).
  static constexpr size_t kSmemBytes =
      2 * size_t(kTileBytes) + size_t(kStages) * kTileBytes + kBarBytes + kStatBytes;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t kv_full[10], kv_empty[10];
  uint64_t s_full[2], p_full[2][2], o_full[2];
  // Items of one tile: the two states of a warp's 32 rows are there to be merged; merged.
  uint64_t merge_ready[4], merge_done[4];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block too large");

struct ChunkParams {
  const int* plan;
  const int* block_table;
  __nv_bfloat16* o;
  float *lse, *part_o, *part_lse;
  size_t o_bytes, lse_bytes, part_o_bytes, part_lse_bytes;  // bounds checks of debug builds
  int o_v8, part_v8;  // 32-byte stores
  int* status;
  int B, T, Hq, Hkv, D, num_pages, page_size, max_pages;
  int group, slices, slice_heads, tile_tokens;
  int box_keys, page_rows;  // keys of a K/V box; rows of the caches (num_pages * Hkv * page_size)
  int ctas;
  long long begins, cuts, pieces;  // the plan's layout
  FixedDiv by_page, by_heads, by_slices;
  float scale_log2;  // scale * log2(e)
};

// Does the plan belong to this call?
__device__ __forceinline__ bool plan_fits(const ChunkParams& p) {
  const PlanHeader* h = reinterpret_cast<const PlanHeader*>(p.plan);
  return h->magic == kMagic && h->B == p.B && h->T == p.T && h->Hq == p.Hq && h->Hkv == p.Hkv &&
         h->D == p.D && h->max_keys == p.max_pages * p.page_size && h->ctas == p.ctas;
}

// What all roles know of the plan: this CTA's pieces.
struct Work {
  const Piece* pieces;
  int begin, end;
  int window, sinks;
};

__device__ __forceinline__ Piece load_piece(const Piece* x) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(x));
  const int4 b = __ldg(reinterpret_cast<const int4*>(x) + 1);
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Bounded wait that also gives up as soon as another role has aborted.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Bars* bars) {
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
// The same for a whole converged warp, with a uniform outcome.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Bars* bars) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, bars));
}

// ------------------------------------------------------------------ producer
// K tiles run ahead of V tiles by one step (two in items of one tile, whose slots take
// them by turns): K_0 (K_1), then pairs V_k, K_k+1 (K_k+2) that complete on V_k's barrier,
// which the MMA warp waits for once.
template <int D>
__device__ void load_role(const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                          const ChunkParams& p, const Work& work, uint8_t* sQ, uint8_t* sKV,
                          Bars* bars, int lane) {
  using C = Cfg<D>;
  uint32_t kv_ctr = 0, q_ctr = 0;
  bool ok = true;
  const uint64_t pol_q = policy_evict_first();
  const uint64_t pol_kv = policy_evict_last();
  const int boxes = 128 / p.box_keys;      // of a K/V tile
  const int batch = 32 / boxes;            // tiles whose boxes the lanes look up at once
  const int my_tile = lane / boxes, my_box = lane % boxes;
  const uint32_t box_bytes = p.box_keys * 128;
  const uint32_t q_bytes = p.slice_heads * p.tile_tokens * 128 * C::kSub;
  bool bad_page = false;
  for (int i = work.begin; i < work.end && ok; ++i) {
    const Piece x = load_piece(work.pieces + i);
    const int n = x.end - x.begin;
    if (n <= 0) continue;
    const bool dual = x.tokens <= p.tile_tokens;
    const KvTiles kv(x.pos, x.tokens, work.window, work.sinks);
    const int g = p.by_slices.div(x.head);
    const int h0 = g * p.group + (x.head - g * p.slices) * p.slice_heads;
    const int* table = p.block_table + static_cast<size_t>(x.row) * p.max_pages;
    // Row of the caches where this lane's box of tiles [k0, k0 + batch) begins; past their
    // end where no row sees a key of it.
    const auto look_up = [&](int k0) {
      const int k = x.begin + k0 + my_tile;
      if (k >= x.end) return p.page_rows;
      const int key = kv.tile(k) * 128 + my_box * p.box_keys;
      if (key >= kv.hi || (key + p.box_keys <= kv.lo && key >= work.sinks)) return p.page_rows;
      const int slot = p.by_page.div(key);
      int page = __ldg(table + slot);
      if (page < 0 || page >= p.num_pages) {
        bad_page = true;
        page = 0;
      }
      return (page * p.Hkv + g) * p.page_size + key - slot * p.page_size;
    };
    int cur = look_up(0), nxt = look_up(batch), cur0 = 0;
    if (q_ctr > 0 && !(ok = wait_warp(&bars->q_empty, (q_ctr - 1) & 1, bars))) break;
    if (elect_one()) {
      mbar_arrive_expect_tx(&bars->q_full, dual ? q_bytes : 2 * q_bytes);
      for (int t = 0; t < (dual ? 1 : 2); ++t)
#pragma unroll
        for (int s = 0; s < C::kSub; ++s)
          tma_load_3d_hint(sQ + t * C::kTileBytes + s * kSubBytes, tmQ, &bars->q_full, s * 64, h0,
                           x.token + t * p.tile_tokens, pol_q);
    }
    __syncwarp();
    ++q_ctr;
    auto take_stage = [&](uint32_t& st) -> bool {
      st = kv_ctr % C::kStages;
      bool g = true;
      if (kv_ctr >= uint32_t(C::kStages))
        g = wait_or_abort(&bars->kv_empty[st], ((kv_ctr / C::kStages) - 1) & 1, bars);
      ++kv_ctr;
      return g;
    };
    // Tile k of the piece (all lanes call it; k is in the current batch or the next).
    auto load_tile = [&](const CUtensorMap* tm, uint32_t st, uint64_t* bar, int k) {
      for (int b = 0; b < boxes; ++b) {
        const int at = k - cur0;
        const int row = at < batch ? __shfl_sync(0xffffffffu, cur, at * boxes + b)
                                   : __shfl_sync(0xffffffffu, nxt, (at - batch) * boxes + b);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < C::kSub; ++s)
            tma_load_3d_hint(sKV + st * C::kTileBytes + s * kSubBytes + b * box_bytes, tm, bar,
                             s * 64, row, 0, pol_kv);
        }
        __syncwarp();
      }
    };
    auto expect = [&](uint64_t* bar, uint32_t bytes) {
      if (elect_one()) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
    };
    const int ahead = dual ? 2 : 1;
    for (int k = 0; k < min(ahead, n) && ok; ++k) {
      uint32_t st;
      const bool g = take_stage(st);
      expect(&bars->kv_full[st], C::kTileBytes);
      load_tile(tmK, st, &bars->kv_full[st], k);
      ok = __all_sync(0xffffffffu, g);
    }
    for (int k = 0; k < n && ok; ++k) {
      // V_k and K_k+ahead lie in this batch or the next.
      if (k == cur0 + batch) {
        cur0 = k;
        cur = nxt;
        nxt = look_up(k + batch);
      }
      uint32_t sv, sk = 0;
      const bool pair = k + ahead < n;
      bool good = take_stage(sv);
      if (pair) good &= take_stage(sk);
      expect(&bars->kv_full[sv], pair ? 2 * C::kTileBytes : C::kTileBytes);
      load_tile(tmV, sv, &bars->kv_full[sv], k);
      if (pair) {
        load_tile(tmK, sk, &bars->kv_full[sv], k + ahead);
        if (elect_one()) mbar_arrive(&bars->kv_full[sk]);
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, good);
    }
  }
  if (bad_page) record_status(p.status, ATTN_ERR_INVALID_ARG);
  if (!ok) record_status(p.status, ATTN_ERR_TIMEOUT);
  // Let every copy that this thread issued land before the CTA can exit.  Those of stages
  // reused since have landed (the MMA warp released them after it saw them, and with a V
  // the K that counts on its barrier).
  const uint32_t last = kv_ctr;
  for (uint32_t c = (last > uint32_t(C::kStages) ? last - C::kStages : 0); c < last; ++c)
    (void)mbar_wait(&bars->kv_full[c % C::kStages], (c / C::kStages) & 1);
  if (q_ctr > 0) (void)mbar_wait(&bars->q_full, (q_ctr - 1) & 1);
}

// ------------------------------------------------------------------ MMA issuer
// Rows [r0, r1) of a V tile become zero.  A whole warp, which afterwards may issue MMAs.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int r1, int lane) {
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  for (int i = lane; i < (r1 - r0) * kChunks; i += 32) {
    const int r = r0 + i / kChunks, c = i % kChunks;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * kSubBytes + r * 128 + (c & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D>
__device__ void mma_role(const ChunkParams& p, const Work& work, uint8_t* sQ, uint8_t* sKV,
                         Bars* bars, uint32_t tmem, int lane) {
  using C = Cfg<D>;
  constexpr uint64_t kDescK = sdesc_sw128(0, 16, 1024);         // Q and K: K-major
  constexpr uint64_t kDescV = sdesc_sw128(0, kSubBytes, 1024);  // V: MN-major
  constexpr uint32_t kHi = static_cast<uint32_t>(kDescK >> 32);
  static_assert(static_cast<uint32_t>(kDescV >> 32) == kHi, "same SBO/swizzle words");
  constexpr uint32_t kLoK = static_cast<uint32_t>(kDescK);
  constexpr uint32_t kLoV = static_cast<uint32_t>(kDescV);
  constexpr uint32_t kTile16 = C::kTileBytes >> 4;
  const uint32_t q_lo = kLoK + (smem_u32(sQ) >> 4);
  const uint32_t k_lo = kLoK + (smem_u32(sKV) >> 4);
  const uint32_t v_lo = kLoV + (smem_u32(sKV) >> 4);
  uint32_t kv_ctr = 0, q_ctr = 0;
  uint32_t p_phase = 0;  // bit t: slot t's
  bool ok = true;

  // S_t = Q_q K^T over D in steps of 16 (K-major operands, 128B swizzle).
  auto issue_s = [&](int t, int q, uint32_t kst) {
    const uint32_t a0 = q_lo + q * kTile16;
    const uint32_t b0 = k_lo + kst * kTile16;
    const uint32_t d = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk >> 2) * kSubBytes + (kk & 3) * 32) >> 4;
      const uint64_t a = desc_from_words(a0 + off, kHi);
      const uint64_t b = desc_from_words(b0 + off, kHi);
      if (kk == 0)
        mma_ss_w<0>(d, a, b, C::kIdescQK);
      else
        mma_ss_w<1>(d, a, b, C::kIdescQK);
    }
    tc_commit_w(&bars->s_full[t]);
  };
  // O_t (+)= P_t V (P from TMEM, V MN-major), as the halves of P arrive.
  auto issue_pv = [&](int t, uint32_t vst, bool first) -> bool {
    const uint32_t b0 = v_lo + vst * kTile16;
    const uint32_t d = tmem + (t ? C::kColO1 : C::kColO0);
    const uint32_t a = tmem + (t ? C::kColS1 : C::kColS0);
    bool good = true;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      good &= wait_or_abort(&bars->p_full[t][half], p_phase >> t & 1, bars);
      tc_fence_after();
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) {
        const int kk = half * 4 + k4;
        const uint64_t bd = desc_from_words(b0 + kk * (2048 >> 4), kHi);
        if (first && kk == 0)
          mma_ts_w<0>(d, a + kk * 8, bd, C::kIdescPV);
        else
          mma_ts_w<1>(d, a + kk * 8, bd, C::kIdescPV);
      }
    }
    p_phase ^= 1u << t;
    return good;
  };
  // Per-lane outcome (no vote: one vote per piece makes the decision to stop uniform).
  auto acquire_kv = [&](uint32_t& st) -> bool {
    st = kv_ctr % C::kStages;
    const bool got = wait_or_abort(&bars->kv_full[st], (kv_ctr / C::kStages) & 1, bars);
    ++kv_ctr;
    return got;
  };
  auto next_stage = [&] {  // landed with a V: counted on its barrier
    const uint32_t st = kv_ctr % C::kStages;
    ++kv_ctr;
    return st;
  };

  for (int i = work.begin; i < work.end && ok; ++i) {
    const Piece x = load_piece(work.pieces + i);
    const int n = x.end - x.begin;
    if (n <= 0) continue;
    const bool dual = x.tokens <= p.tile_tokens;
    const KvTiles kv(x.pos, x.tokens, work.window, work.sinks);
    // Keys that no row sees may hold anything, and a weight of 0 times NaN is NaN: their
    // rows of V become zero (those of whole boxes are loaded as zeros).
    auto clear_unseen = [&](uint32_t vst, int k) {
      const int j = kv.tile(x.begin + k), key0 = 128 * j;
      if (j != kv.e - 1 && j != kv.w && j != kv.s - 1) return;
      uint8_t* tile = sKV + vst * C::kTileBytes;
      const int lo = max(work.sinks - key0, 0), hi = min(kv.lo - key0, 128);
      if (lo < hi) zero_rows<D>(tile, lo, hi, lane);
      if (kv.hi < key0 + 128) zero_rows<D>(tile, kv.hi - key0, 128, lane);
      fence_proxy_async_smem();
      __syncwarp();
    };
    if (!(ok = wait_warp(&bars->q_full, q_ctr & 1, bars))) break;
    ++q_ctr;
    bool good = true;
    if (dual) {
      // Slot k & 1 takes tile k.
      for (int k = 0; k < min(2, n); ++k) {
        uint32_t kst;
        good &= acquire_kv(kst);
        tc_fence_after();
        issue_s(k, 0, kst);
        tc_commit_w(&bars->kv_empty[kst]);
      }
      if (n <= 2) tc_commit_w(&bars->q_empty);
      for (int k = 0; k < n; ++k) {
        uint32_t vst, nst = 0;
        const int t = k & 1;
        const bool more = k + 2 < n;
        good &= acquire_kv(vst);
        if (more) nst = next_stage();
        clear_unseen(vst, k);
        good &= issue_pv(t, vst, k < 2);
        if (more) {
          issue_s(t, 0, nst);
          tc_commit_w(&bars->kv_empty[nst]);
          if (k + 3 == n) tc_commit_w(&bars->q_empty);
        } else {
          tc_commit_w(&bars->o_full[t]);
        }
        tc_commit_w(&bars->kv_empty[vst]);
      }
    } else {
      uint32_t kst;
      good &= acquire_kv(kst);
      tc_fence_after();
      issue_s(0, 0, kst);
      issue_s(1, 1, kst);
      tc_commit_w(&bars->kv_empty[kst]);
      if (n == 1) tc_commit_w(&bars->q_empty);
      for (int k = 0; k < n; ++k) {
        uint32_t vst, nst = 0;
        const bool more = k + 1 < n;
        good &= acquire_kv(vst);
        if (more) nst = next_stage();
        clear_unseen(vst, k);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          good &= issue_pv(t, vst, k == 0);
          if (more)
            issue_s(t, t, nst);
          else
            tc_commit_w(&bars->o_full[t]);
        }
        tc_commit_w(&bars->kv_empty[vst]);
        if (more) {
          tc_commit_w(&bars->kv_empty[nst]);
          if (k + 2 == n) tc_commit_w(&bars->q_empty);
        }
      }
    }
    ok = __all_sync(0xffffffffu, good);
  }
  if (!ok) record_status(p.status, ATTN_ERR_TIMEOUT);
  // Every MMA this thread issued must finish before TMEM is released.
  tc_commit_w(&bars->mma_done);
  (void)mbar_wait(&bars->mma_done, 0);
}

// ------------------------------------------------------------------ softmax
template <int D>
__device__ void softmax_role(const ChunkParams& p, const Work& work, Bars* bars, float2* stats,
                             uint32_t tmem, int warp, int lane) {
  using C = Cfg<D>;
  const int t = warp >> 2;
  const int quad = warp & 3;
  const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t tS = tmem + lane_addr + (t ? C::kColS1 : C::kColS0);
  const uint32_t tO = tmem + lane_addr + (t ? C::kColO1 : C::kColO0);
  const uint32_t tOther = tmem + lane_addr + (t ? C::kColO0 : C::kColO1);
  const float sl2 = p.scale_log2;
  const uint64_t pol_o = policy_evict_first();  // output rows are written once
  const int tile_row = quad * 32 + lane;
  const int row_token = p.by_heads.div(tile_row);  // of the tile's
  const int row_head = tile_row - row_token * p.slice_heads;
  uint32_t s_phase = 0, o_phase = 0, merge_phase = 0;
  bool ok = true;

  for (int i = work.begin; i < work.end && ok; ++i) {
    const Piece x = load_piece(work.pieces + i);
    const int n = x.end - x.begin;
    const bool dual = x.tokens <= p.tile_tokens;
    const KvTiles kv(x.pos, x.tokens, work.window, work.sinks);
    const int g = p.by_slices.div(x.head);
    const int slice_head = (x.head - g * p.slices) * p.slice_heads + row_head;
    const int token = row_token + (dual ? 0 : t * p.tile_tokens);  // of the item's
    const bool row_valid =
        row_token < p.tile_tokens && token < x.tokens && slice_head < p.group;
    const bool warp_valid = __any_sync(0xffffffffu, row_valid);
    // This slot's tiles of the piece: all, or every second one.
    const int k0 = dual ? t : 0, dk = dual ? 2 : 1;
    // Last key that the row sees, and first of its window (rows that are nobody's: all keys,
    // which spares their warp the masks).
    const int limit = row_valid ? x.pos + token : kMaxKeys;
    const int win_lo = row_valid ? limit - work.window + 1 : -kMaxKeys;

    // Where the row's results go.
    const bool part = x.part >= 0;
    const int row_at = dual ? tile_row : t * 128 + tile_row;  // in the partial result
    const size_t at = part ? static_cast<size_t>(x.part) * 256 + row_at
                           : static_cast<size_t>(x.token + token) * p.Hq + g * p.group + slice_head;
    float* const lse_ptr = (part ? p.part_lse : p.lse) + at;
    const size_t lse_bytes = part ? p.part_lse_bytes : p.lse_bytes;

    float m = -INFINITY;  // reference maximum (log2 domain)
    float l = 0.f;
    for (int k = k0; k < n; k += dk) {
      ok = wait_warp(&bars->s_full[t], s_phase, bars);
      if (!ok) break;
      s_phase ^= 1;
      if (!warp_valid) {
        // Nobody reads these rows of P V.
        tc_fence_before();
        mbar_arrive_warp(&bars->p_full[t][0]);
        mbar_arrive_warp(&bars->p_full[t][1]);
        continue;
      }
      tc_fence_after();

      // S row: columns 0..63 are loaded and waited for, 64..127 stay in
      // flight while the first half is masked and reduced.
      uint32_t sa[64], sb[64];
      tmem_ld64(tS, sa);
      tmem_ld64_nowait(tS + 64, sb);
      const int key0 = kv.tile(x.begin + k) * 128;
      const bool need_mask = __any_sync(
          0xffffffffu, key0 + 127 > limit || (key0 < win_lo && key0 + 127 >= work.sinks));
      auto mask_half = [&](uint32_t(&y)[64], int h) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int c0 = key0 + 64 * h + 32 * q;
          const uint32_t bits = window_bits(win_lo - c0, limit + 1 - c0, work.sinks - c0);
          if (__any_sync(0xffffffffu, bits != 0xffffffffu)) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(bits >> c & 1u)) y[32 * q + c] = __float_as_uint(-INFINITY);
          }
        }
      };
      if (need_mask) mask_half(sa, 0);
      // Row maximum: 4 independent chains of 3-input max.
      float ch[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ch[e] = max3(ch[e], __uint_as_float(sa[c + e]), __uint_as_float(sa[c + 4 + e]));
      tmem_ld_wait64(sb);
      if (need_mask) mask_half(sb, 1);
#pragma unroll
      for (int c = 0; c < 64; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ch[e] = max3(ch[e], __uint_as_float(sb[c + e]), __uint_as_float(sb[c + 4 + e]));
      const float m_tile = max3(ch[0], ch[1], fmaxf(ch[2], ch[3])) * sl2;

      bool rescale = false;
      float alpha = 1.f;
      if (k == k0) {
        m = m_tile;
      } else if (row_valid && m_tile - m > kRescaleThreshold) {  // false when both are -inf
        alpha = ex2(m - m_tile);
        m = m_tile;
        l *= alpha;
        rescale = true;
      }
      if (__any_sync(0xffffffffu, rescale)) {
        // The slot's last P V is complete: S was committed after it.
        const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t orow[32];
          tmem_ld32(tO + c, orow);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(orow[e]), __uint_as_float(orow[e + 1])), a2),
                      x0, x1);
            orow[e] = __float_as_uint(x0);
            orow[e + 1] = __float_as_uint(x1);
          }
          tmem_st32(tO + c, orow);
        }
      }
      // p = 2^(s * scale * log2 e - m), two columns per paired FMA/ADD.
      const float base = (m == -INFINITY) ? 0.f : m;
      const uint64_t sc2 = f2_pack(sl2, sl2);
      const uint64_t nb2 = f2_pack(-base, -base);
      uint64_t acc2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc2[e] = f2_pack(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t* src = c < 2 ? &sa[32 * c] : &sb[32 * (c - 2)];
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x0, x1;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(src[2 * e]), __uint_as_float(src[2 * e + 1])),
                           sc2, nb2),
                    x0, x1);
          const float p0 = ex2(x0);
          const float p1 = ex2(x1);
          acc2[e & 3] = f2_add(acc2[e & 3], f2_pack(p0, p1));
          pk[e] = pack_bf16x2(p0, p1);
        }
        tmem_st16(tS + 16 * c, pk);
        if (c & 1) {
          // Keys [64*(c/2), 64*(c/2)+64) of P (and any O rescale) are in TMEM.
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(&bars->p_full[t][c >> 1]);
        }
      }
      float rsum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, b;
        f2_unpack(acc2[e], a, b);
        rsum += a + b;
      }
      l += rsum;
    }
    if (!ok) break;

    const bool has_own = n > k0;  // (one tile in all: slot 1 of a dual item has none)
    if (has_own) {
      ok = wait_warp(&bars->o_full[t], o_phase, bars);
      if (!ok) break;
      o_phase ^= 1;
    }
    if (!warp_valid) continue;
    tc_fence_after();
    // Weights of the slot's O (and of the other's): O = (w O_t + w' O_t') / l.
    float w_own = 1.f, w_other = 0.f;
    bool has_other = false;
    if (dual && n > 0) {
      stats[t * 128 + tile_row] = make_float2(m, l);
      mbar_arrive_warp(&bars->merge_ready[quad]);
      ok = wait_warp(&bars->merge_ready[quad], merge_phase, bars);
      if (!ok) break;
      tc_fence_after();
      const float2 y = stats[(1 - t) * 128 + tile_row];
      const float both = fmaxf(m, y.x);
      w_own = m == -INFINITY ? 0.f : ex2(m - both);
      w_other = y.x == -INFINITY ? 0.f : ex2(y.x - both);
      l = l * w_own + y.y * w_other;
      m = both;
      has_other = n > 1 - t;
    }
    const float inv_l = l > 0.f ? 1.f / l : 0.f;
    w_own *= inv_l;
    w_other *= inv_l;
    // Lane pairs swap half their segments (pair_transpose8), so that each store writes 64
    // contiguous bytes of a row.  A merged row's halves are each written by one slot.
    const int pb = lane & 1;
    const int c_begin = dual ? t * (D / 2) : 0, c_end = dual ? (t + 1) * (D / 2) : D;
    const unsigned valid = __ballot_sync(0xffffffffu, row_valid);
    const bool even_valid = valid >> (lane & ~1) & 1u, odd_valid = valid >> (lane | 1) & 1u;
    const size_t other_at = __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(at), 1);
    const size_t even_at = pb ? other_at : at, odd_at = pb ? at : other_at;
#pragma unroll 1
    for (int c = c_begin; c < c_end; c += 32) {
      uint32_t w[32];
      if (has_own) {
        tmem_ld32(tO + c, w);
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * w_own);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = 0u;
      }
      if (has_other) {
        uint32_t y[32];
        tmem_ld32(tOther + c, y);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          w[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), w_other, __uint_as_float(w[e])));
      }
      if (part) {
        pair_transpose8(w, lane);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float* e32 = p.part_o + even_at * D + c + 8 * (2 * q + pb);
          float* d32 = p.part_o + odd_at * D + c + 8 * (2 * q + pb);
          if (even_valid && store_in_bounds(e32, 32, p.part_o, p.part_o_bytes, p.status))
            st_global_8w(e32, &w[16 * q], p.part_v8);
          if (odd_valid && store_in_bounds(d32, 32, p.part_o, p.part_o_bytes, p.status))
            st_global_8w(d32, &w[16 * q + 8], p.part_v8);
        }
      } else {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          v[e] = pack_bf16x2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
        pair_transpose8(v, lane);
        __nv_bfloat16* e16 = p.o + even_at * D + c + 16 * pb;
        __nv_bfloat16* d16 = p.o + odd_at * D + c + 16 * pb;
        if (even_valid && store_in_bounds(e16, 32, p.o, p.o_bytes, p.status))
          st_global_8w_hint(e16, &v[0], p.o_v8, pol_o);
        if (odd_valid && store_in_bounds(d16, 32, p.o, p.o_bytes, p.status))
          st_global_8w_hint(d16, &v[8], p.o_v8, pol_o);
      }
    }
    if (row_valid && (!dual || t == 0) &&
        store_in_bounds(lse_ptr, 4, part ? p.part_lse : p.lse, lse_bytes, p.status))
      *lse_ptr = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    if (dual && n > 0) {
      // The other slot has read this one's O before it is written again.
      tc_fence_before();
      mbar_arrive_warp(&bars->merge_done[quad]);
      ok = wait_warp(&bars->merge_done[quad], merge_phase, bars);
      merge_phase ^= 1;
    }
  }
  if (!ok) record_status(p.status, ATTN_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ kernel
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_chunk_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const ChunkParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023) != 0) {  // the swizzled tiles need it
    if (threadIdx.x == 0) record_status(p.status, ATTN_ERR_UNSUPPORTED);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * C::kTileBytes;
  Bars* bars = reinterpret_cast<Bars*>(sKV + C::kStages * C::kTileBytes);
  float2* stats = reinterpret_cast<float2*>(sKV + C::kStages * C::kTileBytes + C::kBarBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t][0], 4);  // one arrival per softmax warp of the slot
      mbar_init(&bars->p_full[t][1], 4);
      mbar_init(&bars->o_full[t], 1);
    }
    for (int q = 0; q < 4; ++q) {
      mbar_init(&bars->merge_ready[q], 2);  // one per slot
      mbar_init(&bars->merge_done[q], 2);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // A programmatic dependent: global memory is touched from here on.
  grid_dependency_wait();
  grid_launch_dependents();

  const bool fits = plan_fits(p);
  if (!fits && threadIdx.x == 0) record_status(p.status, ATTN_ERR_INVALID_ARG);
  const PlanHeader* header = reinterpret_cast<const PlanHeader*>(p.plan);
  Work work;
  work.pieces = reinterpret_cast<const Piece*>(p.plan + p.pieces);
  work.begin = fits ? p.plan[p.begins + blockIdx.x] : 0;
  work.end = fits ? p.plan[p.begins + blockIdx.x + 1] : 0;
  work.window = header->window;
  work.sinks = header->sinks;

  if (warp < 8) {
    setmaxnreg_inc<kRegsSoftmax>();
    softmax_role<D>(p, work, bars, stats, tmem, warp, lane);
  } else {
    setmaxnreg_dec<kRegsOther>();
    if (warp == kMmaWarp) {
      mma_role<D>(p, work, sQ, sKV, bars, tmem, lane);
    } else if (warp == kLoadWarp) {
      load_role<D>(&tmQ, &tmK, &tmV, p, work, sQ, sKV, bars, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ merge
// A CTA column per cut item (grid x), its rows shared out over the warps of grid y: rows'
// partial results weighted by their LSE, in the order of the keys.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) chunk_merge_kernel(const ChunkParams p) {
  constexpr int DPL = D / 32;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  if (!plan_fits(p)) return;
  const PlanHeader* header = reinterpret_cast<const PlanHeader*>(p.plan);
  if (static_cast<int>(blockIdx.x) >= header->n_cuts) return;
  const Cut cut = reinterpret_cast<const Cut*>(p.plan + p.cuts)[blockIdx.x];
  const bool dual = cut.tokens <= p.tile_tokens;
  const int g = p.by_slices.div(cut.head);
  for (int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); row < (dual ? 128 : 256);
       row += gridDim.y * kMergeWarps) {
    const int t = row >> 7, tile_row = row & 127;
    const int row_token = p.by_heads.div(tile_row);
    const int head = (cut.head - g * p.slices) * p.slice_heads + tile_row - row_token * p.slice_heads;
    const int token = row_token + t * p.tile_tokens;
    if (row_token >= p.tile_tokens || token >= cut.tokens || head >= p.group) continue;
    const size_t to = static_cast<size_t>(cut.token + token) * p.Hq + g * p.group + head;
    const float* lse = p.part_lse + static_cast<size_t>(cut.part) * 256 + row;
    const float* o = p.part_o + (static_cast<size_t>(cut.part) * 256 + row) * D + lane * DPL;
    float M = -INFINITY;
    for (int s = lane; s < cut.parts; s += 32) M = fmaxf(M, lse[s * 256]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float out[DPL];
#pragma unroll
    for (int e = 0; e < DPL; ++e) out[e] = 0.f;
    float total = 0.f;
    if (M != -INFINITY) {
      for (int s = 0; s < cut.parts; ++s) {
        const float w = ex2((lse[s * 256] - M) * kLog2e);
        total += w;
        const float* src = o + static_cast<size_t>(s) * 256 * D;
#pragma unroll
        for (int e = 0; e < DPL; e += 2) {
          const float2 y = *reinterpret_cast<const float2*>(src + e);
          out[e] = fmaf(w, y.x, out[e]);
          out[e + 1] = fmaf(w, y.y, out[e + 1]);
        }
      }
      const float inv = 1.f / total;
#pragma unroll
      for (int e = 0; e < DPL; ++e) out[e] *= inv;
    }
    __nv_bfloat16* dst = p.o + to * D + lane * DPL;
    if (store_in_bounds(dst, 2 * DPL, p.o, p.o_bytes, p.status)) {
#pragma unroll
      for (int e = 0; e < DPL; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(out[e], out[e + 1]);
    }
    if (lane == 0 && store_in_bounds(p.lse + to, 4, p.lse, p.lse_bytes, p.status))
      p.lse[to] = M == -INFINITY ? -INFINITY : M + logf(total);
  }
}

template <int D>
cudaError_t launch_impl(const void* q, const void* k, const void* v, const ChunkParams& p,
                        cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap tmQ, tmK, tmV;
  if (!encode_bf16_map(&tmQ, q, D, p.Hq, p.T, p.slice_heads, p.tile_tokens) ||
      !encode_bf16_map(&tmK, k, D, p.page_rows, 1, p.box_keys) ||
      !encode_bf16_map(&tmV, v, D, p.page_rows, 1, p.box_keys))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(attn_chunk_kernel<D>),
                                   static_cast<int>(C::kSmemBytes));
  if (e != cudaSuccess) return e;
  e = launch_programmatic(attn_chunk_kernel<D>, dim3(p.ctas), dim3(kThreads), C::kSmemBytes, stream,
                          tmQ, tmK, tmV, p);
  if (e != cudaSuccess) return e;
  return launch_programmatic(chunk_merge_kernel<D>, dim3(p.ctas, 8), dim3(32 * kMergeWarps), 0,
                             stream, p);
}

}  // namespace

cudaError_t launch_chunk_plan(const int* cu, const int* seqlens, int* plan, int B, int T, int Hq,
                              int Hkv, int D, int max_keys, int window, int sinks,
                              cudaStream_t stream, int* status) {
  const ChunkTiling tiling(Hq, Hkv);
  PlanParams p = {cu, seqlens, plan, B, T, Hq, Hkv, D, max_keys, window, sinks, sm_count()};
  p.heads = Hkv * tiling.slices;
  p.item_tokens = 2 * tiling.tile_tokens;
  p.max_items = tiling.max_items(B, T, Hkv);
  p.status = status;
  return launch_programmatic(chunk_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
}

cudaError_t launch_attn_chunk(const void* q, const void* k_cache, const void* v_cache,
                              const int* plan, const PagedKV& paged, void* o, float* lse,
                              float* workspace, int B, int T, int Hq, int Hkv, int D, float scale,
                              cudaStream_t stream, int* status) {
  const ChunkTiling tiling(Hq, Hkv);
  ChunkParams p = {};
  p.plan = plan;
  p.block_table = paged.block_table;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.ctas = sm_count();
  const size_t part_rows = 2ull * p.ctas * 256;
  p.part_o = workspace;
  p.part_lse = workspace + part_rows * D;
  p.o_bytes = static_cast<size_t>(T) * Hq * D * 2;
  p.lse_bytes = static_cast<size_t>(T) * Hq * sizeof(float);
  p.part_o_bytes = part_rows * D * sizeof(float);
  p.part_lse_bytes = part_rows * sizeof(float);
  p.o_v8 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
  p.part_v8 = (reinterpret_cast<uintptr_t>(workspace) & 31u) == 0;
  p.status = status;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.num_pages = paged.num_pages;
  p.page_size = paged.page_size;
  p.max_pages = paged.max_pages;
  p.group = tiling.group;
  p.slices = tiling.slices;
  p.slice_heads = tiling.slice_heads;
  p.tile_tokens = tiling.tile_tokens;
  p.box_keys = paged.page_size % 128 == 0 ? 128 : paged.page_size % 64 == 0 ? 64 : 32;
  p.page_rows = paged.num_pages * Hkv * paged.page_size;
  const ChunkLayout layout(B, tiling.max_items(B, T, Hkv), p.ctas);
  p.begins = layout.begins;
  p.cuts = layout.cuts;
  p.pieces = layout.pieces;
  p.by_page = FixedDiv(paged.page_size);
  p.by_heads = FixedDiv(tiling.slice_heads);
  p.by_slices = FixedDiv(tiling.slices);
  p.scale_log2 = scale * 1.4426950408889634f;
  return D == 128 ? launch_impl<128>(q, k_cache, v_cache, p, stream)
                  : launch_impl<64>(q, k_cache, v_cache, p, stream);
}

}  // namespace attn
