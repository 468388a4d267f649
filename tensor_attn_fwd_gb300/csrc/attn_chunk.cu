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
// At D = 256 tensor memory holds one tile's O, and an item is one tile, whose K/V tiles of 64
// keys the slots take by turns.  Both add to the one O, so they share each row's reference
// maximum: it goes from slot to slot with the tiles.  (Scored by both slots, each adding up half
// of O's dims, four prompts of 2048 tokens took 183 us instead of 125, 16/4 heads.)
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
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "window.cuh"

namespace attn {
namespace {

using namespace ptx;

constexpr int kMagic = 0x43484b31;
constexpr int kMaxKeys = 1 << 30;  // of a request
// Costs of an item in the line: per K/V tile with one query tile and with two, and around its
// tiles (its start and its epilogue).  Alike for one tile and two: 64 requests with 8 prompts
// among them 447 us instead of 347; 1 around them: 64 single tokens of up to 16384 keys, D 64,
// 187 instead of 177.  (Measured with one cache for all requests, so that K and V come from L2,
// us for a tile and around an item: two query tiles 1.43 and 3.7 at D = 128, 1.25 and 2.6 at 64;
// one 0.81 and 3.0, 0.68 and 2.7; at D = 256, one tile by 64 keys, 0.91 and 3.0, which is near
// enough to the others' ratios to share the constants.)
constexpr int kCostOne = 2, kCostTwo = 3, kOverhead = 5;
// An item is cut no closer than this to its ends (in tiles), since a cut costs partial results:
// 100 tokens of 1000 19.0 us, with 4 22.6; one of 300 8.0, with 1 10.3.
constexpr int kSnap = 2;
// What cuts cost the CTAs that have them: whole items are dealt out if that is as good.  (Never
// dealt: four prompts of 2048 tokens 132 us instead of 108, sixteen of 512 79 instead of 59.)
constexpr int kCutCost = 12;
// Cost that is worth a CTA of its own: with 16 a token of 16000 keys takes 24.3 us instead of
// 22.6, with 24 one of 300 11.9 instead of 8.1.
constexpr int kMinShare = 8;

__device__ __forceinline__ void record_status(int* status, int code) {
  if (status != nullptr) atomicCAS(status, 0, code);
}

// The plan's header.
struct PlanHeader {
  int magic, B, T, Hq, Hkv, D, max_keys, window, sinks, ctas;
  int n_pieces;
  int pad[kChunkHeader - 11];
};
static_assert(sizeof(PlanHeader) == kChunkHeader * sizeof(int), "header size");

// A run of K/V tiles of an item.
enum : uint16_t {
  kRagged = 1,  // the item's last K/V tile reaches past the request's keys
  kShared = 2,  // the request's K/V is read by several items
};
struct alignas(16) Piece {
  int token;          // first packed token
  uint16_t tokens;    // their number (1 to 2 tiles' worth)
  uint16_t flags;     // kRagged, kShared
  int pos;            // the first one's position
  int row;            // request
  int head;           // KV head * slices + slice
  int begin, end;     // K/V tiles, in the order of the item's list
  int part;           // slot of its partial result; -1: it is the whole item
};
static_assert(sizeof(Piece) == kChunkRecord * sizeof(int), "record size");
// An item in pieces: its partial results are those of slots [part, part + parts).
struct alignas(16) Cut {
  int token, tokens, head, part, parts;  // parts = 0: an unused record
  int pad[3];
};
static_assert(sizeof(Cut) == kChunkRecord * sizeof(int), "record size");

// The K/V tiles that `tokens` tokens from position `pos` on see: sink tiles [0, s), then
// [w, e); e = 0: none.
struct KvTiles {
  int s, w, e;
  int lo, hi;  // keys: some row sees [lo, hi) and [0, sinks)
  __device__ __forceinline__ KvTiles(int pos, int tokens, int window, int sinks, int tile_keys) {
    const int shift = tile_keys == 128 ? 7 : 6;
    hi = max(pos + tokens, 0);
    lo = max(pos - window + 1, 0);
    e = (hi + tile_keys - 1) >> shift;
    w = min(lo >> shift, e);
    s = min((min(sinks, hi) + tile_keys - 1) >> shift, w);
  }
  __device__ __forceinline__ int count() const { return s + e - w; }
  __device__ __forceinline__ int tile(int k) const { return k < s ? k : k - s + w; }
};

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;
constexpr int kCostLevels = 2048;

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
  const int* slots;  // of the tokens, or null: every request has taken its own
  int* plan;
  int B, T, Hq, Hkv, D, max_keys, window, sinks, ctas;
  int heads, tile_tokens, item_tokens;  // KV heads x slices; tokens of a query tile, of an item
  int tile_keys;
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
  Piece* const firsts = reinterpret_cast<Piece*>(p.plan + at.firsts);
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
    // (A request that has not taken its tokens has keys, but none that they see.)
    const bool taken = p.slots == nullptr || p.slots[t0] >= 0;
    const int len = taken ? min(max(p.seqlens[lo], 0), p.max_keys) : 0;
    x.row = lo;
    x.head = rest / n;
    const int from = (rest - x.head * n) * p.item_tokens;
    x.token = t0 + from;
    x.tokens = static_cast<uint16_t>(min(p.item_tokens, n_tok - from));
    x.pos = len - n_tok + from;
    const bool ragged = len % p.tile_keys != 0 &&
                        (x.pos + x.tokens - 1) / p.tile_keys == (len - 1) / p.tile_keys;
    x.flags = (ragged ? kRagged : 0) | (n > 1 ? kShared : 0);
    x.begin = 0;
    x.end = KvTiles(x.pos, x.tokens, p.window, p.sinks, p.tile_keys).count();
    x.part = -1;
  };
  __shared__ int counts[kCostLevels];  // items of each cost, then ranks
  __shared__ unsigned long long loads[kChunkMaxCtas];
  for (int i = tid; i < kCostLevels; i += kPlanThreads) counts[i] = 0;
  for (int i = tid; i < kChunkMaxCtas; i += kPlanThreads) loads[i] = 0;
  __syncthreads();
  const auto cost_of = [&](const Piece& x) {
    return x.end * (x.tokens > p.tile_tokens ? kCostTwo : kCostOne) + kOverhead;
  };
  long long cost = 0;
  for (int i = tid; i < items; i += kPlanThreads) {
    Piece x;
    item(i, x);
    cost += cost_of(x);
    if (items >= 2 * p.ctas) atomicAdd(counts + min(cost_of(x), kCostLevels - 1), 1);
  }
  long long all;
  scan(cost, smem, all);
  const long long want = (all + kMinShare - 1) / kMinShare;
  const int n = want < p.ctas ? static_cast<int>(max(want, 1ll)) : p.ctas;

  // Many items: whole ones, longest first, dealt out forth and back over the CTAs.  (Items of
  // equal cost in any order, which changes no CTA's load and no result.  The costs past the
  // last level are not told apart: with one of them nothing is dealt.)
  bool dealt = false;
  if (items >= 2 * p.ctas && n == p.ctas) {
    __syncthreads();
    static_assert(kCostLevels == 2 * kPlanThreads, "two levels a thread");
    const bool exact = counts[kCostLevels - 1] == 0;
    const int high = kCostLevels - 1 - 2 * tid;
    const long long here = counts[high] + counts[high - 1];
    long long total;
    const int before = static_cast<int>(scan(here, smem, total));
    const int of_high = counts[high];
    __syncthreads();
    counts[high] = before;
    counts[high - 1] = before + of_high;
    __syncthreads();
    const int rounds = items / n, extra = items - rounds * n;  // the last round may be short
    const auto begin_of = [&](int c) {
      return c * rounds + (rounds & 1 ? max(c - (n - extra), 0) : min(c, extra));
    };
    for (int i = tid; i < items; i += kPlanThreads) {
      Piece x;
      item(i, x);
      const int rank = atomicAdd(counts + min(cost_of(x), kCostLevels - 1), 1);
      const int round = rank / n, j = rank - round * n;
      const int c = round & 1 ? n - 1 - j : j;
      pieces[begin_of(c) + round] = x;
      atomicAdd(loads + c, static_cast<unsigned long long>(cost_of(x)));
    }
    __syncthreads();
    // Taken if no CTA has much more than its share; otherwise the line is cut.
    long long most = tid < n ? static_cast<long long>(loads[tid]) : 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
    if ((tid & 31) == 0) smem[tid >> 5] = most;
    __syncthreads();
    most = smem[tid & 31];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
    __syncthreads();
    dealt = exact && most <= all / n + kCutCost;
    if (dealt)
      for (int c = tid; c < n; c += kPlanThreads) begins[c] = begin_of(c);
  }

  // Part c of the line begins at all * c / n.
  long long line = 0;
  int before_cuts = 0, before_items = 0;  // so far: cuts, and items that are cut
  for (int i0 = 0; i0 < items && !dealt; i0 += kPlanThreads) {
    const int i = i0 + tid;
    Piece x = {};
    int w = 0;
    if (i < items) {
      item(i, x);
      w = cost_of(x);
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
      if (steps < 2 * kSnap) return 2 * k < steps ? 0 : steps;
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
      int part = n_cuts > 0 ? cuts_before + items_before : -1;  // cut items have a slot more than cuts
      if (n_cuts > 0) cuts[items_before] = {x.token, x.tokens, x.head, part, n_cuts + 1, {0, 0, 0}};
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
  __syncthreads();
  for (int c = tid; c <= p.ctas; c += kPlanThreads) {
    if (c == 0 && !dealt) begins[c] = 0;
    if (c >= n || items == 0) begins[c] = c == 0 ? 0 : n_pieces;
    if (c >= before_items && c < p.ctas) cuts[c] = {};
    // The parts' first pieces once more, where they can be read without their numbers.
    if (c < p.ctas) {
      const int i = c < n && items > 0 ? begins[c] : n_pieces;
      if (i < n_pieces) firsts[c] = pieces[i];
    }
  }
  if (tid == 0) {
    PlanHeader h = {kMagic, p.B, p.T, p.Hq, p.Hkv, p.D, p.max_keys, p.window, p.sinks, p.ctas,
                    n_pieces, {0, 0, 0, 0, 0}};
    *header = h;
  }
}

// ------------------------------------------------------------------ attention
constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;
constexpr int kLoadKWarp = 9, kLoadVWarp = 10;
constexpr float kRescaleThreshold = 8.0f;
constexpr uint32_t kLaunchRegs = 168;  // 65536 / 384, rounded down to a multiple of 8
constexpr uint32_t kRegsSoftmax = 192;
constexpr uint32_t kRegsOther = 120;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther == kThreads * kLaunchRegs,
              "register split must use exactly the launch allocation");
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr bool kBoth = D == 256;  // one query tile, whose one O both slots add to
  static constexpr int kSub = D / 64;      // swizzled sub-tiles of 64 dims
  static constexpr int kKeys = kBoth ? 64 : 128;  // of a K/V tile
  static constexpr uint32_t kQSubBytes = 128 * 128, kSubBytes = kKeys * 128;
  static constexpr uint32_t kQTileBytes = kSub * kQSubBytes;
  static constexpr int kQTiles = kBoth ? 1 : 2;
  static constexpr uint32_t kTileBytes = kSub * kSubBytes;  // K or V
  static constexpr int kStages = (D == 64) ? 9 : 5;
  static constexpr int kCols = kBoth ? 128 : D;  // of O that a slot writes
  static constexpr uint32_t kColS0 = 0, kColS1 = 128;
  static constexpr uint32_t kColO0 = 256, kColO1 = 256 + kCols;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kBarBytes = 512;
  static constexpr uint32_t kStatBytes = 2 * 128 * 2 * sizeof(float);
  // No room is left to align the tiles: the kernel has no static shared memory, so that the
  // dynamic one begins at a multiple of 1024 (and it looks).
  static constexpr size_t kKvOffset = size_t(kQTiles) * kQTileBytes;
  static constexpr size_t kBarOffset = kKvOffset + size_t(kStages) * kTileBytes;
  static constexpr size_t kSmemBytes = kBarOffset + kBarBytes + kStatBytes;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, kKeys, false, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
};

struct Bars {
  uint64_t q_full[2], q_empty[2];  // of each Q tile
  uint64_t kv_full[10], kv_empty[10];
  uint64_t s_full[2], p_full[2][2], o_full[2];
  // Items of one tile: the two states of a warp's 32 rows are there to be merged; merged.
  uint64_t merge_ready[4], merge_done[4];
  uint64_t max_ready[2][4];  // one O: the rows' reference maxima, of each slot's last tile
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
  int o_v8;  // 32-byte stores
  int* status;
  int B, T, Hq, Hkv, D, num_pages, page_size, max_pages;
  int group, slices, slice_heads, tile_tokens;
  int box_keys, page_rows;  // keys of a K/V box; rows of the caches (num_pages * Hkv * page_size)
  int ctas;
  long long begins, firsts, cuts, pieces;  // the plan's layout
  FixedDiv by_page, by_heads, by_slices;
  float scale_log2;  // scale * log2(e)
};

// Does the plan belong to this call?
__device__ __forceinline__ bool plan_fits(const ChunkParams& p) {
  const PlanHeader* h = reinterpret_cast<const PlanHeader*>(p.plan);
  return h->magic == kMagic && h->B == p.B && h->T == p.T && h->Hq == p.Hq && h->Hkv == p.Hkv &&
         h->D == p.D && h->max_keys == p.max_pages * p.page_size && h->ctas == p.ctas;
}

// What a role knows of the plan: this CTA's pieces.  (Read by each for itself: held in common,
// it costs the softmax warps registers that they do not have.)
struct Work {
  const Piece* pieces;
  int begin, end;
  int window, sinks;
};
__device__ __forceinline__ int load_int(const int* x) {
  int y;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(y) : "l"(x));
  return y;
}
__device__ __forceinline__ Piece load_piece(const Piece* x) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(x));
  const int4 b = __ldg(reinterpret_cast<const int4*>(x) + 1);
  return {a.x, static_cast<uint16_t>(a.y), static_cast<uint16_t>(a.y >> 16), a.z, a.w,
          b.x, b.y, b.z, b.w};
}
// (All loads at once: one after the other they held up the first K tile by a microsecond.)
__device__ __forceinline__ Work load_work(const ChunkParams& p) {
  const PlanHeader* h = reinterpret_cast<const PlanHeader*>(p.plan);
  Work work;
  work.pieces = reinterpret_cast<const Piece*>(p.plan + p.pieces);
  work.begin = load_int(p.plan + p.begins + blockIdx.x);
  work.end = load_int(p.plan + p.begins + blockIdx.x + 1);
  work.window = load_int(&h->window);
  work.sinks = load_int(&h->sinks);
  if (!plan_fits(p)) work.end = work.begin;
  return work;
}

// The fields that the softmax warps need only after a piece's tiles, read once more (from L1):
// kept, they would not fit the registers.
struct PieceEnd {
  int token, head, part;
};
__device__ __forceinline__ PieceEnd load_piece_end(const Piece* x) {
  PieceEnd y;
  asm volatile("ld.global.nc.b32 %0, [%3];\n\tld.global.nc.b32 %1, [%3+16];\n\t"
               "ld.global.nc.b32 %2, [%3+28];"
               : "=r"(y.token), "=r"(y.head), "=r"(y.part) : "l"(x));
  return y;
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

// ------------------------------------------------------------------ producers
// Two warps share a ring of stages, one for Q and K, one for V.  K tiles run ahead of V tiles by
// one step, or two in items of one tile, whose slots take them by turns: K_0 (K_1), then V_k,
// K_k+1 (K_k+2), which is the order in which the MMA warp needs them and in which they take
// the stages.  (What bounds them is the issue of the copies, four a tile of 64-key pages at D =
// 128.  One warp for K and V: four prompts of 2048 tokens 150 us instead of 131, 64 single tokens
// of up to 16384 keys at D = 64 223 instead of 183.)
template <int D>
__device__ void load_role(const CUtensorMap* tmQ, const CUtensorMap* tm, const ChunkParams& p,
                          const Work& work, const Piece& first, uint8_t* sQ, uint8_t* sKV,
                          Bars* bars, int lane, bool loads_v) {
  using C = Cfg<D>;
  uint32_t before = 0;         // tiles of the pieces before
  uint32_t q_uses[2] = {0, 0};  // of each Q tile, so far
  int q_tile = 1;              // items of one tile take the Q tiles by turns: one is loaded while
                               // the other is in use
  bool ok = true;
  const uint64_t pol_q = policy_evict_first();
  // K and V that several items read are kept in L2; those that one reads are let go, or a
  // batch of single tokens would push the others out.
  const uint64_t pol_keep = policy_evict_last();
  const int boxes = C::kKeys / p.box_keys;  // of a K/V tile
  const int batch = 32 / boxes;            // tiles whose boxes the lanes look up at once
  const int my_tile = lane / boxes, my_box = lane % boxes;
  const uint32_t box_bytes = p.box_keys * 128;
  const uint32_t q_bytes = p.slice_heads * p.tile_tokens * 128 * C::kSub;
  bool bad_page = false;
  // A piece, and the rows of the caches where this lane's boxes of two batches of its tiles
  // begin.  The next one's are on their way while a piece is loaded.
  struct Ahead {
    Piece x;
    int g, cur, nxt;
  };
  // Row of the caches where this lane's box of tiles [k0, k0 + batch) begins; past their end
  // where no row sees a key of it.
  const auto look_up = [&](const Piece& x, int g, int k0) {
    const int k = x.begin + k0 + my_tile;
    if (k >= x.end) return p.page_rows;
    const KvTiles kv(x.pos, x.tokens, work.window, work.sinks, C::kKeys);
    const int key = kv.tile(k) * C::kKeys + my_box * p.box_keys;
    if (key >= kv.hi || (key + p.box_keys <= kv.lo && key >= work.sinks)) return p.page_rows;
    const int slot = p.by_page.div(key);
    int page = __ldg(p.block_table + static_cast<size_t>(x.row) * p.max_pages + slot);
    if (page < 0 || page >= p.num_pages) {
      bad_page = true;
      page = 0;
    }
    return (page * p.Hkv + g) * p.page_size + key - slot * p.page_size;
  };
  // (Read before what says whether there is one: the first K tile waits for it.)
  const auto look_ahead = [&](int i) {
    Ahead a = {};
    if (i >= work.end) return a;
    a.x = i == work.begin ? first : load_piece(work.pieces + i);
    a.g = p.by_slices.div(a.x.head);
    a.cur = look_up(a.x, a.g, 0);
    a.nxt = look_up(a.x, a.g, batch);
    return a;
  };
  Ahead ahead_of = look_ahead(work.begin);
  uint32_t last = 0;  // this warp's last tile, as a count of all
  for (int i = work.begin; i < work.end && ok; ++i) {
    const Piece x = ahead_of.x;
    const int g = ahead_of.g;
    int cur = ahead_of.cur, nxt = ahead_of.nxt, cur0 = 0;
    const int n = x.end - x.begin;
    if (n <= 0) {
      ahead_of = look_ahead(i + 1);
      continue;
    }
    const bool dual = !C::kBoth && x.tokens <= p.tile_tokens;
    const uint64_t pol_kv = x.flags & kShared ? pol_keep : pol_q;
    const int ahead = min(C::kBoth || dual ? 2 : 1, n);
    // Tile k of this warp's kind into its stage.
    auto load = [&](int k) {
      // V_k lies in the batch of tile k or the one before.
      if (k == cur0 + batch) {
        cur0 = k;
        cur = nxt;
        nxt = look_up(x, g, k + batch);
      }
      const uint32_t at = before + (loads_v      ? ahead + k + min(k, n - ahead)
                                    : k < ahead ? k
                                                : 2 * k - ahead + 1);
      const uint32_t st = at % C::kStages;
      bool got = true;
      if (at >= uint32_t(C::kStages))
        got = wait_or_abort(&bars->kv_empty[st], (at / C::kStages - 1) & 1, bars);
      int row[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        row[b] = __shfl_sync(0xffffffffu, cur, (k - cur0) * boxes + b);
      if (elect_one()) {
        uint64_t* bar = &bars->kv_full[st];
        uint8_t* to = sKV + st * C::kTileBytes;
        mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b < boxes) {
#pragma unroll
            for (int s = 0; s < C::kSub; ++s)
              tma_load_3d_hint(to + s * C::kSubBytes + b * box_bytes, tm, bar, s * 64, row[b], 0,
                               pol_kv);
          }
      }
      last = at + 1;
      ok = __all_sync(0xffffffffu, got);
    };
    if (dual) q_tile ^= 1;
    auto load_q = [&](int t, int token) {
      if (q_uses[t] > 0) ok = wait_warp(&bars->q_empty[t], (q_uses[t] - 1) & 1, bars);
      if (!ok) return;
      if (elect_one()) {
        const int h0 = g * p.group + (x.head - g * p.slices) * p.slice_heads;
        mbar_arrive_expect_tx(&bars->q_full[t], q_bytes);
#pragma unroll
        for (int s = 0; s < C::kSub; ++s)
          tma_load_3d_hint(sQ + t * C::kQTileBytes + s * C::kQSubBytes, tmQ, &bars->q_full[t], s * 64, h0,
                           token, pol_q);
      }
      __syncwarp();
      ++q_uses[t];
    };
    if (!loads_v) {
      if (dual) {
        if (q_tile == 0)
          load_q(0, x.token);
        else
          load_q(1, x.token);
      }
      for (int k = 0; k < ahead && ok; ++k) load(k);
      if (!dual && ok) load_q(0, x.token);
      if (!C::kBoth && !dual && ok) load_q(1, x.token + p.tile_tokens);
      if (!ok) break;
    }
    ahead_of = look_ahead(i + 1);
    for (int k = loads_v ? 0 : ahead; k < n && ok; ++k) load(k);
    before += 2 * n;
  }
  if (bad_page) record_status(p.status, ATTN_ERR_INVALID_ARG);
  if (!ok) record_status(p.status, ATTN_ERR_TIMEOUT);
  // Let every copy land before the CTA can exit: each stage's last one, whichever warp's (the MMA
  // warp released those before it after it saw them).
  const uint32_t all = ok ? before : last;
  for (uint32_t c = all > uint32_t(C::kStages) ? all - C::kStages : 0; c < all; ++c)
    (void)mbar_wait(&bars->kv_full[c % C::kStages], (c / C::kStages) & 1);
#pragma unroll
  for (int t = 0; t < 2; ++t)
    if (q_uses[t] > 0) (void)mbar_wait(&bars->q_full[t], (q_uses[t] - 1) & 1);
}

// ------------------------------------------------------------------ MMA issuer
// Rows [r0, r1) of a V tile become zero.  A whole warp, which afterwards may issue MMAs.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int r1, int lane) {
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  for (int i = lane; i < (r1 - r0) * kChunks; i += 32) {
    const int r = r0 + i / kChunks, c = i % kChunks;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * Cfg<D>::kSubBytes + r * 128 + (c & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D>
__device__ void mma_role(const ChunkParams& p, const Work& work, uint8_t* sQ, uint8_t* sKV,
                         Bars* bars, uint32_t tmem, int lane) {
  using C = Cfg<D>;
  constexpr uint64_t kDescK = sdesc_sw128(0, 16, 1024);         // Q and K: K-major
  constexpr uint64_t kDescV = sdesc_sw128(0, C::kSubBytes, 1024);  // V: MN-major
  constexpr uint32_t kHi = static_cast<uint32_t>(kDescK >> 32);
  static_assert(static_cast<uint32_t>(kDescV >> 32) == kHi, "same SBO/swizzle words");
  constexpr uint32_t kLoK = static_cast<uint32_t>(kDescK);
  constexpr uint32_t kLoV = static_cast<uint32_t>(kDescV);
  constexpr uint32_t kQTile16 = C::kQTileBytes >> 4, kTile16 = C::kTileBytes >> 4;
  uint32_t q_lo = kLoK + (smem_u32(sQ) >> 4);
  uint32_t k_lo = kLoK + (smem_u32(sKV) >> 4);
  uint32_t v_lo = kLoV + (smem_u32(sKV) >> 4);
  uint32_t q_phase = 0;  // bit t: Q tile t's
  int q_tile = C::kBoth ? 0 : 1;  // of items of one tile (see load_role)
  uint32_t p_phase = 0;  // bit t: slot t's
  bool ok = true;

  // S_t = Q_q K^T over D in steps of 16 (K-major operands, 128B swizzle).
  auto issue_s = [&](int t, int q, uint32_t kst) {
    const uint32_t a0 = q_lo + q * kQTile16;
    const uint32_t b0 = k_lo + kst * kTile16;
    const uint32_t d = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint64_t a =
          desc_from_words(a0 + (((kk >> 2) * C::kQSubBytes + (kk & 3) * 32) >> 4), kHi);
      const uint64_t b =
          desc_from_words(b0 + (((kk >> 2) * C::kSubBytes + (kk & 3) * 32) >> 4), kHi);
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
    const uint32_t d = tmem + (t && !C::kBoth ? C::kColO1 : C::kColO0);
    const uint32_t a = tmem + (t ? C::kColS1 : C::kColS0);
    bool good = true;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      good &= wait_or_abort(&bars->p_full[t][half], p_phase >> t & 1, bars);
      tc_fence_after();
#pragma unroll
      for (int k4 = 0; k4 < C::kKeys / 32; ++k4) {
        const int kk = half * (C::kKeys / 32) + k4;
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
  uint32_t stage = 0, stage_phase = 0;
  auto acquire_kv = [&](uint32_t& st) -> bool {
    const bool got = wait_or_abort(&bars->kv_full[stage], stage_phase, bars);
    st = stage;
    stage = st + 1 == C::kStages ? 0 : st + 1;
    if (stage == 0) stage_phase ^= 1;
    return got;
  };

  for (int i = work.begin; i < work.end && ok; ++i) {
    const Piece x = load_piece(work.pieces + i);
    const int n = x.end - x.begin;
    if (n <= 0) continue;
    const bool dual = !C::kBoth && x.tokens <= p.tile_tokens;
    const KvTiles kv(x.pos, x.tokens, work.window, work.sinks, C::kKeys);
    // Keys that no token sees may hold anything, and a weight of 0 times NaN is NaN: their
    // rows of V become zero (those of whole boxes are loaded as zeros).  Keys behind an item's
    // last position, but not the request's, are later tokens'.  Of the item's tiles these are the
    // last, where the window begins and where the sinks end: `clear` is the next of them.
    const int last_tile = x.flags & kRagged ? kv.count() - 1 : kMaxKeys;
    const auto next_clear = [&](int k) {
      if (k <= kv.s - 1 && work.sinks % C::kKeys != 0) return kv.s - 1;
      if (k <= kv.s && kv.lo % C::kKeys != 0) return kv.s;
      return last_tile;
    };
    int clear = next_clear(x.begin);
    auto clear_unseen = [&](uint32_t vst, int k) {
      const int key0 = C::kKeys * kv.tile(k);
      uint8_t* tile = sKV + vst * C::kTileBytes;
      const int lo = max(work.sinks - key0, 0), hi = min(kv.lo - key0, C::kKeys);
      if (lo < hi) zero_rows<D>(tile, lo, hi, lane);
      if (k == last_tile) zero_rows<D>(tile, kv.hi - key0, C::kKeys, lane);
      fence_proxy_async_smem();
      __syncwarp();
      clear = k < last_tile ? next_clear(k + 1) : kMaxKeys;
    };
    if (dual) q_tile ^= 1;
    const uint32_t q_mine = dual ? 1u << q_tile : C::kBoth ? 1u : 3u;
    for (int t = 0; t < 2 && ok; ++t)
      if (q_mine >> t & 1) ok = wait_warp(&bars->q_full[t], q_phase >> t & 1, bars);
    if (!ok) break;
    q_phase ^= q_mine;
    bool good = true;
    int k = x.begin;  // the tile whose V comes next
    // Turn t of a round: slot t adds P V of a tile and scores its next one.  With two query
    // tiles both slots take each K/V tile, with one (DUAL) every second tile is a slot's.  (Two
    // instances: the time between the MMAs' issues is lost to the tensor core, and with one
    // for both a step of two tiles took 7 % longer.)
    const auto run = [&](auto dual_constant) {
      constexpr bool DUAL = decltype(dual_constant)::value;
      const auto release_q = [&] {  // after the last scores
        if (!DUAL) tc_commit_w(&bars->q_empty[0]);
        tc_commit_w(&bars->q_empty[DUAL ? q_tile : 1]);
      };
      // (What the operands' addresses make is worked out here: kept for both instances, it
      // would not fit the registers.)
      asm volatile("" : "+r"(q_lo), "+r"(k_lo), "+r"(v_lo), "+r"(tmem));
      uint32_t vst = 0, kst = 0;
      good &= acquire_kv(kst);
      tc_fence_after();
      issue_s(0, DUAL ? q_tile : 0, kst);
      if (DUAL && n > 1) {
        tc_commit_w(&bars->kv_empty[kst]);
        good &= acquire_kv(kst);
        tc_fence_after();
      }
      if (!DUAL || n > 1) issue_s(1, DUAL ? q_tile : 1, kst);
      tc_commit_w(&bars->kv_empty[kst]);
      if (n <= (DUAL ? 2 : 1)) release_q();
      for (int left = n; left > 0;) {  // tiles whose P V is to come
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool more = left > (DUAL ? 2 : 1);
          if (DUAL || t == 0) {
            good &= acquire_kv(vst);
            if (k == clear) clear_unseen(vst, k);
          }
          good &= issue_pv(t, vst, k < x.begin + (DUAL && !C::kBoth ? 2 : 1));
          if (C::kBoth) tc_commit_w(&bars->o_full[t]);
          if (more) {
            if (DUAL || t == 0) {
              good &= acquire_kv(kst);
              tc_fence_after();
            }
            issue_s(t, DUAL ? q_tile : t, kst);
          } else if (!C::kBoth) {
            tc_commit_w(&bars->o_full[t]);
          }
          if (DUAL || t == 1) {
            tc_commit_w(&bars->kv_empty[vst]);
            if (more) tc_commit_w(&bars->kv_empty[kst]);
            if (left == (DUAL ? 3 : 2)) release_q();
            ++k;
            --left;
            if (DUAL && left == 0) break;
          }
        }
      }
    };
    if constexpr (C::kBoth) {
      run(std::true_type{});
    } else {
      if (dual)
        run(std::true_type{});
      else
        run(std::false_type{});
    }
    ok = __all_sync(0xffffffffu, good);
  }
  if (!ok) record_status(p.status, ATTN_ERR_TIMEOUT);
  // Every MMA this thread issued must finish before TMEM is released.
  tc_commit_w(&bars->mma_done);
  (void)mbar_wait(&bars->mma_done, 0);
}

// A partial result: the rows' O (by their own sum) in fp32, four columns of all 128 rows of a
// query tile beside each other, so that a warp's 32 rows are stored and read in whole lines.
template <int D>
__device__ __forceinline__ size_t part_at(int part, int tile, int column, int tile_row) {
  return ((static_cast<size_t>(Cfg<D>::kQTiles * part + tile) * (D / 4) + column / 4) * 128 +
          tile_row) * 4;
}
template <int D>
__device__ __forceinline__ int part_lse_at(int part, int tile, int tile_row) {
  return (Cfg<D>::kQTiles * part + tile) * 128 + tile_row;
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&w)[32]) { tmem_ld32(at, w); }
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t (&w)[64]) { tmem_ld64(at, w); }

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
  // One O: the tiles of the pieces before, this slot's and the other's, and those of the other
  // whose maxima this warp could wait for.
  uint32_t own_pv = 0, other_pv = 0, other_max = 0;
  bool ok = true;

  for (int i = work.begin; i < work.end && ok; ++i) {
    const Piece x = load_piece(work.pieces + i);
    const bool dual = !C::kBoth && x.tokens <= p.tile_tokens;
    const int kv_head = p.by_slices.div(x.head);
    const int slice_head = (x.head - kv_head * p.slices) * p.slice_heads + row_head;
    const int token = row_token + (C::kBoth || dual ? 0 : t * p.tile_tokens);  // of the item's
    const bool row_valid =
        row_token < p.tile_tokens && token < x.tokens && slice_head < p.group;
    const bool warp_valid = __any_sync(0xffffffffu, row_valid);
    const int first_token = __shfl_sync(0xffffffffu, token, 0);
    // Last key that the row sees (nobody's rows take their warp's first one's: no masks more),
    // and the first of its window.
    const int limit = x.pos + (row_valid ? token : first_token);
    const int win_lo = limit - work.window + 1;
    // This slot's tiles of the piece: all, or every second one.
    const bool turns = C::kBoth || dual;
    const int k_first = x.begin + (turns ? t : 0), dk = turns ? 2 : 1;
    int k = k_first;
    int sink_tiles, skip;  // tiles from sink_tiles on lie `skip` further on
    {
      const KvTiles kv(x.pos, x.tokens, work.window, work.sinks, C::kKeys);
      sink_tiles = kv.s;
      skip = kv.w - kv.s;
    }

    float m = -INFINITY;  // reference maximum (log2 domain)
    float l = 0.f;
    bool first = true;
    for (; k < x.end; k += dk) {
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
      if constexpr (C::kKeys == 128) tmem_ld64_nowait(tS + 64, sb);
      const int key0 = (k < sink_tiles ? k : k + skip) * C::kKeys;
      const bool need_mask = __any_sync(
          0xffffffffu, key0 + C::kKeys > limit + 1 || (key0 < win_lo && key0 + C::kKeys > work.sinks));
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
      if constexpr (C::kKeys == 128) {
        tmem_ld_wait64(sb);
        if (need_mask) mask_half(sb, 1);
#pragma unroll
        for (int c = 0; c < 64; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            ch[e] = max3(ch[e], __uint_as_float(sb[c + e]), __uint_as_float(sb[c + 4 + e]));
      }
      const float m_tile = max3(ch[0], ch[1], fmaxf(ch[2], ch[3])) * sl2;

      bool rescale = false;
      float alpha = 1.f;
      if constexpr (C::kBoth) {
        // One O has one reference: that of the tile before, from the other slot, or this tile's
        // maximum.  It goes on to the other slot ahead of the exponentials.
        const int j = k - x.begin;
        if (j > 1) ok = wait_warp(&bars->o_full[t], (own_pv + (j >> 1) - 1) & 1, bars);
        if (!ok) break;
        float m_row = m_tile;
        if (j > 0) {
          ok = wait_warp(&bars->max_ready[1 - t][quad], (other_max + ((j - 1) >> 1)) & 1, bars);
          if (!ok) break;
          m_row = stats[(1 - t) * 128 + tile_row].x;
          if (row_valid && m_tile - m_row > kRescaleThreshold) {
            alpha = ex2(m_row - m_tile);
            m_row = m_tile;
            rescale = true;
          }
        }
        if (m_row != m) l *= ex2(m - m_row);
        m = m_row;
        stats[t * 128 + tile_row].x = m;
        mbar_arrive_warp(&bars->max_ready[t][quad]);
      } else if (first) {
        first = false;
        m = m_tile;
      } else if (row_valid && m_tile - m > kRescaleThreshold) {  // false when both are -inf
        alpha = ex2(m - m_tile);
        m = m_tile;
        l *= alpha;
        rescale = true;
      }
      if (__any_sync(0xffffffffu, rescale)) {
        // The slot's last P V is complete: S was committed after it.  That of the other slot,
        // in one O, is waited for.  (The one before it is complete: the other slot
        // waited for it before it handed its maxima on.)
        if constexpr (C::kBoth) {
          ok = wait_warp(&bars->o_full[1 - t], (other_pv + ((k - x.begin - 1) >> 1)) & 1, bars);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t tAll = C::kBoth ? tmem + lane_addr + C::kColO0 : tO;
        const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t orow[32];
          tmem_ld32(tAll + c, orow);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(orow[e]), __uint_as_float(orow[e + 1])), a2),
                      x0, x1);
            orow[e] = __float_as_uint(x0);
            orow[e + 1] = __float_as_uint(x1);
          }
          tmem_st32(tAll + c, orow);
        }
      }
      // p = 2^(s * scale * log2 e - m), two columns per paired FMA/ADD.  P is rounded to bf16, the
      // type that its product with a bf16 V takes (twice the time in tf32, and twice the room in
      // tensor memory); its sum is of the values in 32 bits.  That makes the error of O 2.0e-3 to
      // 2.3e-3 (2-norm, relative) where one rounding of O alone has 1.6e-3.
      const float base = (m == -INFINITY) ? 0.f : m;
      const uint64_t sc2 = f2_pack(sl2, sl2);
      const uint64_t nb2 = f2_pack(-base, -base);
      uint64_t acc2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc2[e] = f2_pack(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < C::kKeys / 32; ++c) {
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
        constexpr int kHalf = C::kKeys / 64;
        if (c % kHalf == kHalf - 1) {
          // Half of P's keys (and any O rescale) are in TMEM.
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(&bars->p_full[t][c / kHalf]);
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

    const int n = x.end - x.begin;
    const bool has_own = C::kBoth ? n > 0 : k != k_first;  // (one tile in all: slot 1 has none)
    if (!C::kBoth && has_own) {
      ok = wait_warp(&bars->o_full[t], o_phase, bars);
      if (!ok) break;
      o_phase ^= 1;
    }
    const int own_n = (n + 1 - t) >> 1, other_n = (n + t) >> 1;  // tiles taken by turns
    own_pv += own_n;
    other_pv += other_n;
    if (!warp_valid) continue;
    other_max += other_n;
    tc_fence_after();
    // Weights of the slot's O (and of the other's): O = (w O_t + w' O_t') / l.
    float w_own = 1.f, w_other = 0.f;
    bool has_other = false;
    if (turns && n > 0) {
      stats[t * 128 + tile_row] = make_float2(m, l);
      mbar_arrive_warp(&bars->merge_ready[quad]);
      ok = wait_warp(&bars->merge_ready[quad], merge_phase, bars);
      if (!ok) break;
      const float2 y = stats[(1 - t) * 128 + tile_row];
      const float both = fmaxf(m, y.x);
      w_own = m == -INFINITY ? 0.f : ex2(m - both);
      w_other = y.x == -INFINITY ? 0.f : ex2(y.x - both);
      l = l * w_own + y.y * w_other;
      m = both;
      if constexpr (C::kBoth) {
        // O is relative to the last tile's reference, which is the highest.
        const bool own_last = ((n - 1) & 1) == t;
        ok = wait_warp(&bars->o_full[(n - 1) & 1], ((own_last ? own_pv : other_pv) - 1) & 1, bars);
        if (!ok) break;
        w_own = 1.f;
        w_other = 0.f;
      }
      tc_fence_after();
      has_other = !C::kBoth && n > 1 - t;
    }
    const float inv_l = l > 0.f ? 1.f / l : 0.f;
    w_own *= inv_l;
    w_other *= inv_l;
    const float own_lse = l > 0.f ? m + log2f(l) : -INFINITY;  // log2 domain
    const PieceEnd to = load_piece_end(work.pieces + i);
    const auto row_of = [&] {  // of O and LSE
      const int kv_head = p.by_slices.div(to.head);
      return static_cast<size_t>(to.token + row_token +
                                 (C::kBoth || dual ? 0 : t * p.tile_tokens)) * p.Hq +
             kv_head * p.group + (to.head - kv_head * p.slices) * p.slice_heads + row_head;
    };
    const int c_off = C::kBoth ? t * C::kCols : 0;  // dim of the slot's first column
    const bool writes_lse = row_valid && (!(C::kBoth || dual) || t == 0);
    // Lane pairs swap half their segments (pair_transpose8), so that each store writes 64
    // contiguous bytes of a row.
    const int pb = lane & 1;
    const unsigned valid = __ballot_sync(0xffffffffu, row_valid);
    const bool even_valid = valid >> (lane & ~1) & 1u, odd_valid = valid >> (lane | 1) & 1u;
    const auto store_columns = [&](int c, uint32_t* w, __nv_bfloat16* even, __nv_bfloat16* odd) {
      uint32_t v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        v[e] = pack_bf16x2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
      pair_transpose8(v, lane);
      if (even_valid && store_in_bounds(even + c, 32, p.o, p.o_bytes, p.status))
        st_global_8w_hint(even + c, &v[0], p.o_v8, pol_o);
      if (odd_valid && store_in_bounds(odd + c, 32, p.o, p.o_bytes, p.status))
        st_global_8w_hint(odd + c, &v[8], p.o_v8, pol_o);
    };
    const auto pair_rows = [&](size_t at, __nv_bfloat16*& even, __nv_bfloat16*& odd) {
      const size_t other = __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(at), 1);
      even = p.o + (pb ? other : at) * D + c_off + 16 * pb;
      odd = p.o + (pb ? at : other) * D + c_off + 16 * pb;
    };
    // The other slot has read O, or its part of it, before it is written again.
    const auto release_o = [&] {
      tc_fence_before();
      mbar_arrive_warp(&bars->merge_done[quad]);
      ok = wait_warp(&bars->merge_done[quad], merge_phase, bars);
      merge_phase ^= 1;
    };
    if (!dual && to.part < 0 && n > 0) {  // (or of one, which the slots share out by columns)
      // A whole item of two tiles: 64 columns of O at a time, the next ones on their way.  (The
      // time of an item around its tiles is that of this.)
      uint32_t wa[64], wb[64];
      tmem_ld64(tO, wa);
      if constexpr (C::kCols == 128) tmem_ld64_nowait(tO + 64, wb);
      const size_t at = row_of();
      __nv_bfloat16 *even, *odd;
      pair_rows(at, even, odd);
      const auto scaled = [&](uint32_t(&w)[64], int c) {
#pragma unroll
        for (int e = 0; e < 64; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * w_own);
        store_columns(c, &w[0], even, odd);
        store_columns(c + 32, &w[32], even, odd);
      };
      scaled(wa, 0);
      if constexpr (C::kCols == 128) {
        tmem_ld_wait64(wb);
        scaled(wb, 64);
      }
      if (writes_lse && store_in_bounds(p.lse + at, 4, p.lse, p.lse_bytes, p.status))
        p.lse[at] = own_lse * kLn2;
      if (C::kBoth) release_o();
      continue;
    }
    // Columns [c, c + N) of the row's result of this piece.
    const auto own_columns = [&](int c, auto& w) {
      constexpr int N = sizeof(w) / sizeof(w[0]);
      if (has_own) {
        load_columns(tO + c, w);
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * w_own);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) w[e] = 0u;
      }
      if (N == 32 && has_other) {
        uint32_t y[N];
        load_columns(tOther + c, y);
#pragma unroll
        for (int e = 0; e < N; ++e)
          w[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), w_other, __uint_as_float(w[e])));
      }
    };
    // The columns that this warp writes (of an item of one tile, whose slots are merged, each
    // slot writes half), N at a time.
    const auto finish = [&](auto n_constant, int c_begin, int c_end) {
      constexpr int N = decltype(n_constant)::value;
      const int tile = C::kBoth || dual ? 0 : t;
      if (to.part >= 0) {
#pragma unroll 1
        for (int c = c_begin; c < c_end; c += N) {
          uint32_t w[N];
          own_columns(c, w);
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            float* y = p.part_o + part_at<D>(to.part, tile, c_off + c + e, tile_row);
            if (store_in_bounds(y, 16, p.part_o, p.part_o_bytes, p.status))
              *reinterpret_cast<uint4*>(y) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
          }
        }
        float* y = p.part_lse + part_lse_at<D>(to.part, tile, tile_row);
        if (writes_lse && store_in_bounds(y, 4, p.part_lse, p.part_lse_bytes, p.status)) *y = own_lse;
        return;
      }
      const size_t at = row_of();
      __nv_bfloat16 *even, *odd;
      pair_rows(at, even, odd);
#pragma unroll 1
      for (int c = c_begin; c < c_end; c += N) {
        uint32_t w[N];
        own_columns(c, w);
#pragma unroll
        for (int e = 0; e < N; e += 32) store_columns(c + e, &w[e], even, odd);
      }
      if (writes_lse && store_in_bounds(p.lse + at, 4, p.lse, p.lse_bytes, p.status))
        p.lse[at] = own_lse * kLn2;
    };
    if (dual)
      finish(std::integral_constant<int, 32>{}, t * (D / 2), (t + 1) * (D / 2));
    else
      finish(std::integral_constant<int, 64>{}, 0, C::kCols);
    if (turns && n > 0) release_o();
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
  uint8_t* sKV = smem + C::kKvOffset;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kBarOffset);
  float2* stats = reinterpret_cast<float2*>(smem + C::kBarOffset + C::kBarBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
    }
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
      mbar_init(&bars->max_ready[0][q], 1);
      mbar_init(&bars->max_ready[1][q], 1);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == kLoadKWarp && lane == 0) {
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

  if (threadIdx.x == 0 && !plan_fits(p)) record_status(p.status, ATTN_ERR_INVALID_ARG);
  if (warp < 8) {
    setmaxnreg_inc<kRegsSoftmax>();
    softmax_role<D>(p, load_work(p), bars, stats, tmem, warp, lane);
  } else {
    setmaxnreg_dec<kRegsOther>();
    if (warp == kMmaWarp) {
      mma_role<D>(p, load_work(p), sQ, sKV, bars, tmem, lane);
    } else if (warp == kLoadKWarp || warp == kLoadVWarp) {
      const bool loads_v = warp == kLoadVWarp;
      const Piece first = load_piece(reinterpret_cast<const Piece*>(p.plan + p.firsts) + blockIdx.x);
      load_role<D>(&tmQ, loads_v ? &tmV : &tmK, p, load_work(p), first, sQ, sKV, bars, lane, loads_v);
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
// A cut item (grid x, or none), 16 columns (y) of a query tile (z), a row to a thread: the
// partial results weighted by their LSE, summed in the order of the keys.  A thread's loads of
// up to four pieces are on their way at once, so that it takes few trips to L2.
//
// The plan is older than the attention kernel, which has waited for it, so it is read ahead of the
// wait for that kernel, and CTAs without an item leave.  (Not the first: the kernel has to end
// after the one before, on which the next kernel in the stream relies.)
constexpr int kMergeColumns = 16;
template <int D>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const ChunkParams p) {
  const Cut cut = reinterpret_cast<const Cut*>(p.plan + p.cuts)[blockIdx.x];
  const int tile = blockIdx.z, tile_row = threadIdx.x, c = blockIdx.y * kMergeColumns;
  const bool mine = plan_fits(p) && cut.parts > 0 && tile * p.tile_tokens < cut.tokens;
  if (!mine && (blockIdx.x | blockIdx.y | blockIdx.z) != 0) return;
  const int g = p.by_slices.div(cut.head);
  const int row_token = p.by_heads.div(tile_row);
  const int head = (cut.head - g * p.slices) * p.slice_heads + tile_row - row_token * p.slice_heads;
  const int token = row_token + tile * p.tile_tokens;
  grid_dependency_wait();
  if (!mine || row_token >= p.tile_tokens || token >= cut.tokens || head >= p.group) return;
  float top = -INFINITY, total = 0.f;  // of the weights 2^(lse - top), their sum
  float sum[kMergeColumns];
#pragma unroll
  for (int e = 0; e < kMergeColumns; ++e) sum[e] = 0.f;
  for (int s0 = 0; s0 < cut.parts; s0 += 4) {
    const int n = min(4, cut.parts - s0);
    float lse[4];
    float4 x[4][kMergeColumns / 4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int part = cut.part + s0 + min(s, n - 1);
      lse[s] = s < n ? p.part_lse[part_lse_at<D>(part, tile, tile_row)] : -INFINITY;
#pragma unroll
      for (int q = 0; q < kMergeColumns / 4; ++q)
        x[s][q] = *reinterpret_cast<const float4*>(
            p.part_o + part_at<D>(part, tile, c + 4 * q, tile_row));
    }
    const float higher = fmaxf(fmaxf(fmaxf(lse[0], lse[1]), fmaxf(lse[2], lse[3])), top);
    if (higher == -INFINITY) continue;
    const float scale = ex2(top - higher);
    top = higher;
    total *= scale;
#pragma unroll
    for (int e = 0; e < kMergeColumns; ++e) sum[e] *= scale;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float w = ex2(lse[s] - top);
      total += w;
#pragma unroll
      for (int q = 0; q < kMergeColumns / 4; ++q) {
        sum[4 * q] = fmaf(w, x[s][q].x, sum[4 * q]);
        sum[4 * q + 1] = fmaf(w, x[s][q].y, sum[4 * q + 1]);
        sum[4 * q + 2] = fmaf(w, x[s][q].z, sum[4 * q + 2]);
        sum[4 * q + 3] = fmaf(w, x[s][q].w, sum[4 * q + 3]);
      }
    }
  }
  const float inv = total > 0.f ? 1.f / total : 0.f;
  uint32_t y[kMergeColumns / 2];
#pragma unroll
  for (int e = 0; e < kMergeColumns / 2; ++e)
    y[e] = pack_bf16x2(sum[2 * e] * inv, sum[2 * e + 1] * inv);
  const size_t at = static_cast<size_t>(cut.token + token) * p.Hq + g * p.group + head;
  if (store_in_bounds(p.o + at * D + c, 2 * kMergeColumns, p.o, p.o_bytes, p.status))
    st_global_8w(p.o + at * D + c, y, p.o_v8);
  if (c == 0 && store_in_bounds(p.lse + at, 4, p.lse, p.lse_bytes, p.status))
    p.lse[at] = total > 0.f ? (top + log2f(total)) * kLn2 : -INFINITY;
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
  // (Items of so few tiles are never cut.)
  if (e != cudaSuccess || p.max_pages * p.page_size <= (2 * kSnap - 1) * C::kKeys) return e;
  return launch_programmatic(chunk_merge_kernel<D>, dim3(p.ctas, D / kMergeColumns, C::kQTiles),
                             dim3(128), 0, stream, p);
}

}  // namespace

int chunk_ctas() { return sm_count() < kChunkMaxCtas ? sm_count() : kChunkMaxCtas; }

cudaError_t launch_chunk_plan(const int* cu, const int* seqlens, const int* slots, int* plan, int B,
                              int T, int Hq, int Hkv, int D, int max_keys, int window, int sinks,
                              cudaStream_t stream, int* status) {
  const ChunkTiling tiling(Hq, Hkv);
  PlanParams p = {cu, seqlens, slots, plan, B, T, Hq, Hkv, D, max_keys, window, sinks, chunk_ctas()};
  p.heads = Hkv * tiling.slices;
  p.tile_tokens = tiling.tile_tokens;
  p.item_tokens = tiling.item_tokens(D);
  p.tile_keys = chunk_tile_keys(D);
  p.max_items = tiling.max_items(B, T, Hkv, D);
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
  p.ctas = chunk_ctas();
  const size_t part_rows = 2ull * p.ctas * chunk_part_rows(D);
  p.part_o = workspace;
  p.part_lse = workspace + part_rows * D;
  p.o_bytes = static_cast<size_t>(T) * Hq * D * 2;
  p.lse_bytes = static_cast<size_t>(T) * Hq * sizeof(float);
  p.part_o_bytes = part_rows * D * sizeof(float);
  p.part_lse_bytes = part_rows * sizeof(float);
  p.o_v8 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0;
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
  if (p.box_keys > chunk_tile_keys(D)) p.box_keys = chunk_tile_keys(D);
  p.page_rows = paged.num_pages * Hkv * paged.page_size;
  const ChunkLayout layout(B, tiling.max_items(B, T, Hkv, D), p.ctas);
  p.begins = layout.begins;
  p.firsts = layout.firsts;
  p.cuts = layout.cuts;
  p.pieces = layout.pieces;
  p.by_page = FixedDiv(paged.page_size);
  p.by_heads = FixedDiv(tiling.slice_heads);
  p.by_slices = FixedDiv(tiling.slices);
  p.scale_log2 = scale * 1.4426950408889634f;
  const auto launch = D == 256 ? launch_impl<256> : D == 128 ? launch_impl<128> : launch_impl<64>;
  return launch(q, k_cache, v_cache, p, stream);
}

}  // namespace attn
