// api.cu -- the C ABI of libattn.so: argument validation, status codes and the
// per-device state (SM count, kernel attributes, device status word).  Every
// entry point validates before launching; nothing here allocates device
// memory or synchronises, except attn_debug_status().
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "kernel_attrs.h"
#include "window.cuh"

namespace attn {
namespace {

constexpr int kMaxDevices = SharedMemoryLimits::kMaxDevices;

// Written by kernels whose bounded wait expired (ATTN_ERR_TIMEOUT).
__device__ int g_status_word = 0;

std::mutex g_mutex;
int g_sm_count[kMaxDevices] = {0};
int* g_status_ptr[kMaxDevices] = {nullptr};

SharedMemoryLimits g_smem_limits;

int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
  return dev;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes are int on the ABI; keep every product the kernels form in range.
constexpr long long kMaxElems = 1ll << 40;
constexpr int kMaxSeq = 1 << 30;

}  // namespace

int sm_count() {
  const int dev = current_device();
  if (dev < 0) return 1;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_sm_count[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 1;
    g_sm_count[dev] = n;
  }
  return g_sm_count[dev];
}

int* status_word_device_ptr() {
  const int dev = current_device();
  if (dev < 0) return nullptr;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_status_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess) return nullptr;
    g_status_ptr[dev] = static_cast<int*>(p);
  }
  return g_status_ptr[dev];
}

cudaError_t ensure_smem_attr(const void* kernel, int bytes) {
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mutex);
  return g_smem_limits.allow(kernel, dev, bytes, [](const void* f, int n) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
  });
}

cudaError_t allow_large_cluster(const void* kernel) {
  static const void* seen[kMaxDevices][16] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mutex);
  int i = 0;
  while (i < 16 && seen[dev][i] != nullptr && seen[dev][i] != kernel) ++i;
  if (i < 16 && seen[dev][i] == kernel) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && i < 16) seen[dev][i] = kernel;  // (table full: set again next time)
  return e;
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qres;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &qres) == cudaSuccess &&
        qres == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

}  // namespace

bool encode_bf16_map(CUtensorMap* map, const void* base, int D, int rows, int planes,
                     int box_rows) {
  auto fn = get_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(D) * 2 * cuuint64_t(rows)};
  const cuuint32_t box[3] = {64, cuuint32_t(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace attn

using namespace attn;

extern "C" {

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ATTN_OK";
    case ATTN_ERR_INVALID_ARG: return "ATTN_ERR_INVALID_ARG: invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED: unsupported configuration";
    case ATTN_ERR_MISALIGNED: return "ATTN_ERR_MISALIGNED: pointer not 16-byte aligned";
    case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA: CUDA runtime error";
    case ATTN_ERR_TIMEOUT: return "ATTN_ERR_TIMEOUT: a kernel wait expired";
    case ATTN_ERR_BOUNDS: return "ATTN_ERR_BOUNDS: a kernel store fell outside its output (debug build)";
    case ATTN_ERR_NO_PAGES: return "ATTN_ERR_NO_PAGES: no free pages left";
    default: return "unknown attn status";
  }
}

int attn_version(void) { return (1 << 16) | 0; }

namespace {

// The argument checks of the prefill entry points; ATTN_OK or the status to return.
int fwd_check_args(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale) {
  if (!q || !k || !v || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (Sq > kMaxSeq || Sk > kMaxSeq) return ATTN_ERR_UNSUPPORTED;
  // (Then no product below overflows.)
  if (static_cast<long long>(B) * Hq > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hq * Sq > kMaxElems / D ||
      static_cast<long long>(B) * Hkv * Sk > kMaxElems / D)
    return ATTN_ERR_UNSUPPORTED;
  // Work items (B*Hq*ceil(Sq/256), or ceil(Sq/128) at D = 256) are indexed with int.
  if (static_cast<long long>(B) * Hq * ((Sq + 127) / 128) > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

int fwd_common(const void* q, const void* k, const void* v, void* o, int o_bf16, float* lse,
               int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale,
               void* stream) {
  const int chk = fwd_check_args(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale);
  if (chk != ATTN_OK) return chk;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e = launch_attn_fwd(q, k, v, o, o_bf16, lse, B, Hq, Hkv, Sq, Sk, D, causal,
                                        scale, static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int attn_fwd(const void* q, const void* k, const void* v, float* o, float* lse, int B, int Hq,
             int Hkv, int Sq, int Sk, int D, int causal, float scale, void* stream) {
  return fwd_common(q, k, v, o, 0, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale, stream);
}

int attn_fwd_bf16o(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                   int Hq, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                   void* stream) {
  return fwd_common(q, k, v, o, 1, lse, B, Hq, Hkv, Sq, Sk, D, causal, scale, stream);
}

int attn_fwd_splitkv(const void* q, const void* k, const void* v, float* o_part,
                     float* lse_part, int B, int Hq, int Hkv, int Sq, int Sk, int D, int causal,
                     int num_splits, float scale, void* stream) {
  if (!q || !k || !v || !o_part || !lse_part) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (Sq > kMaxSeq || Sk > kMaxSeq) return ATTN_ERR_UNSUPPORTED;
  // Every split covers at least one 128-key tile.
  if (num_splits < 1 || num_splits > (Sk + 127) / 128) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_splits) * B * Hq * Sq * D > kMaxElems ||
      static_cast<long long>(B) * Hkv * Sk * D > kMaxElems)
    return ATTN_ERR_UNSUPPORTED;
  // Work items B*Hq*ceil(Sq/256)*num_splits are indexed with int.
  if (static_cast<long long>(B) * Hq * ((Sq + 255) / 256) * num_splits > (1ll << 30))
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o_part) ||
      !aligned16(lse_part))
    return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e =
      launch_attn_fwd_splitkv(q, k, v, o_part, lse_part, B, Hq, Hkv, Sq, Sk, D, causal,
                              num_splits, scale, static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

namespace {
// Items that splits cut (the last round's), at most: see WindowOrder.
long long window_split_items(long long B, int Hq, int Hkv, int Sq, int D) {
  const long long items = window_items(B, Hq, Hkv, Sq, D), n_sm = sm_count();
  return items % n_sm;
}
bool window_splits_fit(int B, int Hq, int Hkv, int Sq, int D, int num_splits) {
  const long long rem = window_split_items(B, Hq, Hkv, Sq, D);
  return static_cast<long long>(B) * Hq * Sq <= (1ll << 30) &&
         window_items(B, Hq, Hkv, Sq, D) + rem * num_splits <= (1ll << 30) &&
         rem * num_splits * window_item_rows(D) * D <= kMaxElems;
}
}  // namespace

int attn_window_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                    float* workspace, int B, int Hq, int Hkv, int Sq, int Sk, int D, int window,
                    int sinks, int num_splits, float scale, void* stream) {
  if (window < 1 || sinks < 0 || num_splits < 1) return ATTN_ERR_INVALID_ARG;
  if (num_splits > 1 && !workspace) return ATTN_ERR_INVALID_ARG;
  const int chk = fwd_check_args(q, k, v, o, lse, B, Hq, Hkv, Sq, Sk, D, 1, scale);
  if (chk != ATTN_OK) return chk;
  if (num_splits > 1) {
    // Every split of the longest row has a key tile; rows and items are counted with int.
    if (num_splits > (Sk + 127) / 128) return ATTN_ERR_INVALID_ARG;
    if (!window_splits_fit(B, Hq, Hkv, Sq, D, num_splits)) return ATTN_ERR_UNSUPPORTED;
    if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  }
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  // A window or sinks past the last key mean all keys; clamped, the kernels' sums fit int.
  const cudaError_t e =
      launch_attn_window_fwd(q, k, v, o, lse, workspace, B, Hq, Hkv, Sq, Sk, D,
                             window < Sk ? window : Sk, sinks < Sk ? sinks : Sk, num_splits,
                             scale, static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_window_fwd_num_splits(int B, int Hq, int Hkv, int Sq, int Sk, int D, int window,
                               int sinks, int* num_splits) {
  if (num_splits == nullptr || B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || D <= 0 ||
      Hq % Hkv != 0 || window < 1 || sinks < 0)
    return ATTN_ERR_INVALID_ARG;
  *num_splits = 1;
  // (Up to three tiles, one split is always best by the estimate below.)
  if (static_cast<long long>(window) + sinks <= 128 || Sk <= 384) return ATTN_OK;
  if (Sq > kMaxSeq || Sk > kMaxSeq || static_cast<long long>(B) * Hq > (1ll << 30) ||
      !window_splits_fit(B, Hq, Hkv, Sq, D, 32))
    return ATTN_OK;
  const long long n_sm = sm_count();
  window = window < Sk ? window : Sk;
  sinks = sinks < Sk ? sinks : Sk;
  const WindowOrder order = window_order(B, Hq, Hkv, Sq, Sk, D, window, 2);
  if (order.rem == 0) return ATTN_OK;
  // Key tiles of the last round's longest item, its first.
  const int tile_rows = D == 256 || window_head_pairs(Hq, Hkv) ? 128 : 256;
  const int row0 = order.item(order.unsplit).tile * tile_rows;
  const TileRange r0 = window_kv_tiles(Sq, Sk, window, sinks, row0);
  const TileRange r1 = window_kv_tiles(Sq, Sk, window, sinks, row0 + tile_rows - 128);
  const long long tiles = r0.count() > r1.count() ? r0.count() : r1.count();
  // Estimated time of the last round, in ns: 1400 for a step of an item, 3500 around it,
  // and for the merge 3500 and the partials' way to L2 and back at 5 bytes a ps.
  // Measured (us, all of one round) against it, D = 128, 32/8 heads: Sq 512, 34 tiles:
  // 1 split 51.9 (est. 52), 2 37.2 (38); Sq 512, 10 tiles: 1 20.0 (17), 2 21.1 (20);
  // Sq 128, 34 tiles: 4 22.8 (23), 8 19.4 (20), 16 26.4 (more than one round).
  // D = 256, where an item is one tile of a head, measured alike: 16/4 heads, Sq 512, 34
  // tiles: 1 56.0, 2 36.9, 3 50.0; Sq 128: 7 20.6, 8 22.3; 32 items of 4 tiles: 1 12.3,
  // 2 13.6; 24 items of 34: 6 22.1, 7 30.7.
  // D = 64, whose step takes about 1200, 32/8 heads: Sq 512, 34 tiles: 1 45.9, 2 31.7, 3
  // 40.6; Sq 512, 10 tiles: 1 17.5, 2 17.3; Sq 128, 34 tiles: 6 16.9, 8 16.2, 12 20.6; Sq 1280:
  // 2 72.6, 8 60.2, 12 58.9, 16 60.0.  The rule takes 2, 2, 9 and 17: the same estimate serves.
  const long long rows = 1ll * order.rem * window_item_rows(D), all = 1ll * B * Hq * Sq;
  const long long partial_ns = 2 * (rows < all ? rows : all) * D * 4 / 5000;  // of one split
  long long best_ns = tiles * 1400 + 3500;
  for (long long ns = 2; ns <= tiles && ns <= 32 && ns * order.rem <= n_sm; ++ns) {
    const long long t = (tiles + ns - 1) / ns * 1400 + 7000 + ns * partial_ns;
    if (t < best_ns) {
      *num_splits = static_cast<int>(ns);
      best_ns = t;
    }
  }
  return ATTN_OK;
}

int attn_window_fwd_workspace(int B, int Hq, int Hkv, int Sq, int D, int num_splits,
                              long long* floats) {
  if (floats == nullptr || B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || D <= 0 || num_splits < 1 ||
      Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
  if (Sq > kMaxSeq || static_cast<long long>(B) * Hq > (1ll << 30) ||
      static_cast<long long>(B) * Hq * Sq > kMaxElems / D ||
      static_cast<long long>(B) * Hq * ((Sq + 127) / 128) > (1ll << 30) ||
      (num_splits > 1 && !window_splits_fit(B, Hq, Hkv, Sq, D, num_splits)))
    return ATTN_ERR_UNSUPPORTED;
  *floats = num_splits == 1 ? 0
                            : window_split_items(B, Hq, Hkv, Sq, D) * num_splits *
                                  window_item_rows(D) * (D + 1);
  return ATTN_OK;
}

int attn_fwd_num_splits(int B, int Hq, int Hkv, int Sq, int Sk, int D, int* num_splits) {
  if (num_splits == nullptr) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || D <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  const int n_sm = sm_count();
  if (n_sm <= 0) return ATTN_ERR_CUDA;
  long long ns = 1;
  if (D == 64 || D == 128) {
    // Work items without splitting (two 128-row query tiles each).
    const long long base = fwd_items_per_split(B, Hq, Hkv, Sq);
    const long long kv_tiles = (Sk + 127) / 128;
    // Splitting pays when it removes more KV steps from every item than the
    // combine and the partials cost: a cache long against the chunk
    // (Sk > 2 Sq) or at least 16 KV tiles.  Measured counter-examples: causal
    // or not, B1 H16 S1024 D64 (one pass 14.0 us, 2 splits 14.8) and B1 Hq32
    // Hkv8 Sq512 Sk1024 (16.2 vs 18.2).
    const bool worth = Sk > 2ll * Sq || kv_tiles >= 16;
    if (worth && base * 5 < static_cast<long long>(n_sm) * 4) {
      // Too few to fill the GPU: as many splits as still fit every item in one
      // round on the SMs (a second round would cost as much as it saves), each
      // split keeping at least four 128-key tiles.
      ns = n_sm / base > 1 ? n_sm / base : 1;
      const long long cap = kv_tiles / 4 > 1 ? kv_tiles / 4 : 1;
      if (ns > cap) ns = cap;
    }
  }
  *num_splits = static_cast<int>(ns);
  return ATTN_OK;
}

}  // extern "C"

int attn::decode_check_args(const void* q, const void* k, const void* v, int B, int Hq, int Hkv,
                            int Sk, int D, int num_splits, float scale, bool paged) {
  if (!q || !k || !v) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sk <= 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > Sk) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  // The kernels split [0, Sk) with int arithmetic.
  if (Sk > kMaxSeq) return ATTN_ERR_UNSUPPORTED;
  if (!paged && static_cast<long long>(B) * Hkv * Sk * D > kMaxElems) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_splits) * B * Hq * D > kMaxElems) return ATTN_ERR_UNSUPPORTED;
  // Output rows (and tensor-map planes) are indexed with int.
  if (static_cast<long long>(B) * Hq > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
  const int head_slices = (Hq / Hkv + 15) / 16;  // query heads per decode CTA: 16
  if (B > 65535 || static_cast<long long>(Hkv) * head_slices > 65535)
    return ATTN_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

extern "C" {

namespace {

int decode_common(const void* q, const void* k, const void* v, const int* seqlens,
                  float* o_part, float* lse_part, int B, int Hq, int Hkv, int Sk, int D,
                  int num_splits, float scale, void* stream, const PagedKV* paged = nullptr) {
  if (!o_part || !lse_part) return ATTN_ERR_INVALID_ARG;
  const int chk = decode_check_args(q, k, v, B, Hq, Hkv, Sk, D, num_splits, scale,
                                    paged != nullptr);
  if (chk != ATTN_OK) return chk;
  if (!aligned16(o_part) || !aligned16(lse_part)) return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e =
      launch_decode_splitkv(q, k, v, o_part, lse_part, B, Hq, Hkv, Sk, D, num_splits, scale,
                            static_cast<cudaStream_t>(stream), status, seqlens, paged);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int attn_decode_splitkv(const void* q, const void* k, const void* v, float* o_part,
                        float* lse_part, int B, int Hq, int Hkv, int Sk, int D, int num_splits,
                        float scale, void* stream) {
  return decode_common(q, k, v, nullptr, o_part, lse_part, B, Hq, Hkv, Sk, D, num_splits, scale,
                       stream);
}

int attn_decode_splitkv_varlen(const void* q, const void* k, const void* v, const int* seqlens,
                               float* o_part, float* lse_part, int B, int Hq, int Hkv, int Sk,
                               int D, int num_splits, float scale, void* stream) {
  if (!seqlens) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(seqlens) & 3u) != 0) return ATTN_ERR_MISALIGNED;
  return decode_common(q, k, v, seqlens, o_part, lse_part, B, Hq, Hkv, Sk, D, num_splits, scale,
                       stream);
}

int attn_decode_fused(const void* q, const void* k, const void* v, const int* seqlens, float* o,
                      float* lse, float* o_part, float* lse_part, int* counters, int B, int Hq,
                      int Hkv, int Sk, int D, int num_splits, float scale, void* stream) {
  if (!o_part || !lse_part || !o || !lse || !counters) return ATTN_ERR_INVALID_ARG;
  const int chk = decode_check_args(q, k, v, B, Hq, Hkv, Sk, D, num_splits, scale, false);
  if (chk != ATTN_OK) return chk;
  if (!aligned16(o_part) || !aligned16(lse_part) || !aligned16(o) || !aligned16(lse))
    return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(counters) & 3u) != 0) return ATTN_ERR_MISALIGNED;
  if (seqlens != nullptr && (reinterpret_cast<uintptr_t>(seqlens) & 3u) != 0)
    return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const FusedCombine fused{o, lse, counters};
  const cudaError_t e =
      launch_decode_splitkv(q, k, v, o_part, lse_part, B, Hq, Hkv, Sk, D, num_splits, scale,
                            static_cast<cudaStream_t>(stream), status, seqlens, nullptr, &fused);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_decode_fused_counters(int B, int Hq, int Hkv, int* count) {
  if (count == nullptr) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  const long long n = static_cast<long long>(B) * Hkv * ((Hq / Hkv + 15) / 16);
  if (n > (1ll << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  *count = static_cast<int>(n);
  return ATTN_OK;
}

namespace {

// The paged decode entry points' checks of the cache description; ATTN_OK or
// the status to return.  On success *paged describes the cache and *capacity is
// max_pages * page_size.
int paged_check_args(const int* block_table, const int* seqlens, int Hkv, int num_pages,
                     int page_size, int max_pages, int D, int B, PagedKV* paged, int* capacity) {
  if (!block_table || !seqlens) return ATTN_ERR_INVALID_ARG;
  if (num_pages <= 0 || page_size <= 0 || max_pages <= 0) return ATTN_ERR_INVALID_ARG;
  if (page_size % 32 != 0) return ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(block_table) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(seqlens) & 3u) != 0)
    return ATTN_ERR_MISALIGNED;
  const long long cap = static_cast<long long>(max_pages) * page_size;
  if (cap > kMaxSeq) return ATTN_ERR_UNSUPPORTED;
  if (Hkv > 0 && static_cast<long long>(num_pages) * Hkv > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
  if (Hkv > 0 && D > 0 &&
      static_cast<long long>(num_pages) * Hkv * page_size * D > kMaxElems)
    return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * max_pages > (1ll << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  *paged = PagedKV{block_table, page_size, max_pages, num_pages};
  *capacity = static_cast<int>(cap);
  return ATTN_OK;
}

}  // namespace

int attn_decode_fused_paged(const void* q, const void* k_cache, const void* v_cache,
                            const int* block_table, const int* seqlens, float* o, float* lse,
                            float* o_part, float* lse_part, int* counters, int B, int Hq, int Hkv,
                            int num_pages, int page_size, int max_pages, int D, int num_splits,
                            float scale, void* stream) {
  PagedKV paged;
  int capacity = 0;
  const int pchk = paged_check_args(block_table, seqlens, Hkv, num_pages, page_size, max_pages,
                                    D, B, &paged, &capacity);
  if (pchk != ATTN_OK) return pchk;
  if (!o_part || !lse_part || !o || !lse || !counters) return ATTN_ERR_INVALID_ARG;
  // The contiguous-size checks apply to the capacity; the cache itself is
  // num_pages pages, checked above.
  const int chk = decode_check_args(q, k_cache, v_cache, B, Hq, Hkv, capacity, D, num_splits,
                                    scale, true);
  if (chk != ATTN_OK) return chk;
  if (!aligned16(o_part) || !aligned16(lse_part) || !aligned16(o) || !aligned16(lse))
    return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(counters) & 3u) != 0) return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const FusedCombine fused{o, lse, counters};
  const cudaError_t e = launch_decode_splitkv(q, k_cache, v_cache, o_part, lse_part, B, Hq, Hkv,
                                              capacity, D, num_splits, scale,
                                              static_cast<cudaStream_t>(stream), status, seqlens,
                                              &paged, &fused);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

namespace {

// Sk: the cache's capacity; paged: its layout, or nullptr (contiguous, [B,Hkv,Sk,D]).
int decode_window_common(const void* q, const void* k, const void* v, const int* seqlens,
                         const PagedKV* paged, void* o, float* lse, int B, int Hq, int Hkv, int Sk,
                         int D, int window, int sinks, int num_splits, float scale,
                         void* stream) {
  if (!o || !lse || window < 1 || sinks < 0 || num_splits > kWindowDecodeSplits)
    return ATTN_ERR_INVALID_ARG;
  // (Splits without a block of their own are empty: there may be more splits than keys.)
  const int chk = decode_check_args(q, k, v, B, Hq, Hkv, Sk, D,
                                    num_splits < 1 ? num_splits : 1, scale, paged != nullptr);
  if (chk != ATTN_OK) return chk;
  if (!aligned16(o) || !aligned16(lse)) return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(seqlens) & 3u) != 0) return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e = launch_decode_window(
      q, k, v, seqlens, paged, o, lse, B, Hq, Hkv, Sk, D, window < Sk ? window : Sk,
      sinks < Sk ? sinks : Sk, num_splits, scale, static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int attn_decode_window(const void* q, const void* k, const void* v, const int* seqlens, void* o,
                       float* lse, int B, int Hq, int Hkv, int Sk, int D, int window, int sinks,
                       int num_splits, float scale, void* stream) {
  return decode_window_common(q, k, v, seqlens, nullptr, o, lse, B, Hq, Hkv, Sk, D, window, sinks,
                              num_splits, scale, stream);
}

int attn_decode_window_num_splits(int B, int Hq, int Hkv, int Sk, int D, int window, int sinks,
                                  int* num_splits) {
  if (num_splits == nullptr || B <= 0 || Hq <= 0 || Hkv <= 0 || Sk <= 0 || D <= 0 ||
      Hq % Hkv != 0 || window < 1 || sinks < 0)
    return ATTN_ERR_INVALID_ARG;
  const long long n_sm = sm_count();
  if (n_sm <= 0) return ATTN_ERR_CUDA;
  const long long reach = static_cast<long long>(window) + sinks;
  const long long blocks = ((reach < Sk ? reach : Sk) + 31) / 32;
  // CTAs of one split.  Measured (us; 32 query heads a KV head's group of 4, keys seen):
  const long long base = static_cast<long long>(B) * Hkv * ((Hq / Hkv + 15) / 16);
  long long ns;
  if (D == 64) {
    // Two CTAs an SM or more: base 128, 4100 keys: 1 split 32.1, 2 23.6, 4 30.4.
    ns = 2 * n_sm / base;
  } else if (D == 256) {
    // One CTA an SM: base 64, 2052 keys: 1 split 34.3, 2 27.5, 3 37.0.
    ns = n_sm / base;
  } else if (base * 5 >= n_sm * 4) {
    ns = 1;  // base 128, 4100 keys: 1 split 44.4, 2 44.9
  } else if (base >= 16) {
    // About one CTA an SM, to a power of two: base 64, 1028 keys: 2 splits 10.2, 4 9.9, 6
    // 16.3; base 32: 2 10.0, 4 8.0, 8 8.7; base 96, 4100 keys: 1 40.8, 2 35.6, 4 42.3.
    ns = 1ll << std::lround(std::log2(static_cast<double>((n_sm + base - 1) / base)));
  } else {
    ns = n_sm / base;
  }
  // CTAs a little past one or two rounds of resident ones (3, 2 or 1 an SM) and long
  // walks: with splits the last round is as short as its CTAs.  D 128, 4100 keys: base
  // 312: 1 split 122.3, 2 110.8, 3 105.5; 384: 128.5, 119.5, 124.9; 416: 130.2, 129.8;
  // 640: 206.8, 197.2, 195.1; 2052 keys: base 312: 68.1, 64.9, 64.3; 1028 keys: 38.2,
  // 39.9.  D 64, 4100 keys: base 480: 101.9, 89.9, 86.1.  D 256: base 160: 144, 130, 122.
  const long long slots = n_sm * (D == 64 ? 3 : D == 128 ? 2 : 1);
  const long long rounds = base / slots, extra = base % slots;
  if ((rounds == 1 || rounds == 2) && extra > 0 && extra * 20 <= slots * 7 &&
      blocks >= 64 * rounds)
    ns = extra * 20 <= slots * 3 ? 3 : 2;
  // A split keeps two blocks (base 8, 260 keys: 1 split 6.8, 4 5.4, 8 5.6), and clusters
  // past 12 pay only for few and long walks (base 8, 1028 keys: 8 splits 6.7, 12 6.2, 16 7.8;
  // base 1, 16388 keys: 12 16.9, 16 15.0).
  const long long most = base <= 4 && blocks >= 256 ? kWindowDecodeSplits : 12;
  if (ns > most) ns = most;
  if (ns > blocks / 2) ns = blocks / 2;
  *num_splits = ns > 1 ? static_cast<int>(ns) : 1;
  return ATTN_OK;
}

int attn_decode_window_paged(const void* q, const void* k_cache, const void* v_cache,
                             const int* block_table, const int* seqlens, void* o, float* lse,
                             int B, int Hq, int Hkv, int num_pages, int page_size, int max_pages,
                             int D, int window, int sinks, int num_splits, float scale,
                             void* stream) {
  PagedKV paged;
  int capacity = 0;
  const int pchk = paged_check_args(block_table, seqlens, Hkv, num_pages, page_size, max_pages,
                                    D, B, &paged, &capacity);
  if (pchk != ATTN_OK) return pchk;
  return decode_window_common(q, k_cache, v_cache, seqlens, &paged, o, lse, B, Hq, Hkv, capacity,
                              D, window, sinks, num_splits, scale, stream);
}

int attn_decode_splitkv_paged(const void* q, const void* k_cache, const void* v_cache,
                              const int* block_table, const int* seqlens, float* o_part,
                              float* lse_part, int B, int Hq, int Hkv, int num_pages,
                              int page_size, int max_pages, int D, int num_splits, float scale,
                              void* stream) {
  PagedKV paged;
  int capacity = 0;
  const int pchk = paged_check_args(block_table, seqlens, Hkv, num_pages, page_size, max_pages,
                                    D, B, &paged, &capacity);
  if (pchk != ATTN_OK) return pchk;
  // The contiguous-size checks of decode_common apply to the capacity; the
  // cache itself is num_pages pages, checked above.
  return decode_common(q, k_cache, v_cache, seqlens, o_part, lse_part, B, Hq, Hkv, capacity, D,
                       num_splits, scale, stream, &paged);
}

namespace {

// The backward's sizes (positive ones) are within its limits.
bool bwd_sizes_fit(int B, int Hq, int Hkv, int Sq, int Sk, int D) {
  if (Sq > kMaxSeq || Sk > kMaxSeq) return false;
  if (static_cast<long long>(B) * Hq > (1ll << 30)) return false;  // (no product below overflows)
  if (static_cast<long long>(B) * Hq * Sq > kMaxElems / D ||
      static_cast<long long>(B) * Hkv * Sk > kMaxElems / D)
    return false;
  if (static_cast<long long>(B) * Hq * ((Sq + 127) / 128) > (1ll << 30) ||
      static_cast<long long>(B) * Hkv * ((Sk + 127) / 128) > (1ll << 30))
    return false;
  // Delta rows are indexed with int.
  if (static_cast<long long>(B) * Hq * Sq > (1ll << 30)) return false;
  return D == 64 || D == 128;
}

// The argument checks of the backward entry points; ATTN_OK or the status to return.
int bwd_check_args(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dout, const void* dq, const void* dk, const void* dv,
                   const float* delta_ws, int B, int Hq, int Hkv, int Sq, int Sk, int D,
                   int causal, float scale) {
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !delta_ws)
    return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || D <= 0) return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (!bwd_sizes_fit(B, Hq, Hkv, Sq, Sk, D)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(delta_ws))
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

}  // namespace

int attn_bwd(const void* q, const void* k, const void* v, const float* o, const float* lse,
             const void* dout, float* dq, float* dk, float* dv, float* delta_ws, int B, int Hq,
             int Hkv, int Sq, int Sk, int D, int causal, float scale, void* stream) {
  const int chk = bwd_check_args(q, k, v, o, lse, dout, dq, dk, dv, delta_ws, B, Hq, Hkv, Sq, Sk,
                                 D, causal, scale);
  if (chk != ATTN_OK) return chk;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e =
      launch_attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, delta_ws, B, Hq, Hkv, Sq, Sk, D, causal,
                      scale, static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_window_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                    const void* dout, void* dq, void* dk, void* dv, float* workspace, int B,
                    int Hq, int Hkv, int Sq, int Sk, int D, int window, int sinks, float scale,
                    void* stream) {
  if (window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  const int chk = bwd_check_args(q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Sq, Sk,
                                 D, 1, scale);
  if (chk != ATTN_OK) return chk;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e = launch_attn_window_bwd(
      q, k, v, o, lse, dout, dq, dk, dv, workspace, B, Hq, Hkv, Sq, Sk, D,
      window < Sk ? window : Sk, sinks < Sk ? sinks : Sk, scale, static_cast<cudaStream_t>(stream),
      status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_window_bwd_workspace(int B, int Hq, int Hkv, int Sq, int Sk, int D, int window, int sinks,
                              long long* floats) {
  if (floats == nullptr || B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || D <= 0 ||
      window < 1 || sinks < 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (!bwd_sizes_fit(B, Hq, Hkv, Sq, Sk, D)) return ATTN_ERR_UNSUPPORTED;
  *floats = window_bwd_workspace_floats(B, Hq, Hkv, Sq, Sk, D, window < Sk ? window : Sk,
                                        sinks < Sk ? sinks : Sk);
  return ATTN_OK;
}

int attn_rope_table(float* table, int max_pos, int D, float base, void* stream) {
  if (!table) return ATTN_ERR_INVALID_ARG;
  if (max_pos <= 0 || D <= 0 || D % 2 != 0) return ATTN_ERR_INVALID_ARG;
  if (!(base > 1.f) || !std::isfinite(base)) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pos) * D > kMaxElems) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(table)) return ATTN_ERR_MISALIGNED;
  const cudaError_t e = launch_rope_table(table, max_pos, D, static_cast<double>(base),
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_qkv_rope(const void* x, const void* w, const float* rope_table, const int* positions,
                  void* q, void* k, void* v, int B, int S, int hidden, int Hq, int Hkv, int D,
                  int max_pos, int style, void* stream) {
  if (!x || !w || !rope_table || !q || !k || !v) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || S <= 0 || hidden <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_pos <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (style != 0 && style != 1) return ATTN_ERR_INVALID_ARG;
  if (positions == nullptr && max_pos < S) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
  if (hidden % 8 != 0) return ATTN_ERR_UNSUPPORTED;  // TMA row pitch: a multiple of 16 bytes
  const long long T = static_cast<long long>(B) * S;
  const long long N = static_cast<long long>(Hq + 2ll * Hkv) * D;
  if (T > (1ll << 30) || N > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
  if (T * hidden > kMaxElems || N * hidden > kMaxElems || T * N > kMaxElems)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(x) || !aligned16(w) || !aligned16(rope_table) || !aligned16(q) ||
      !aligned16(k) || !aligned16(v))
    return ATTN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(positions) & 3u) != 0) return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e = launch_qkv_rope(x, w, rope_table, positions, q, k, v, B, S, hidden, Hq,
                                        Hkv, D, max_pos, style,
                                        static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_decode_num_splits(int B, int Hq, int Hkv, int Sk, int D, int* num_splits) {
  if (num_splits == nullptr) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sk <= 0 || D <= 0 || Hq % Hkv != 0)
    return ATTN_ERR_INVALID_ARG;
  const int n_sm = sm_count();
  if (n_sm <= 0) return ATTN_ERR_CUDA;
  // CTAs without splitting: (batch, KV head, 16-head slice of the group).
  const long long base = static_cast<long long>(B) * Hkv * ((Hq / Hkv + 15) / 16);
  long long ns = 1;
  if (base * 5 < static_cast<long long>(n_sm) * 4) {
    // Too few to stream at full bandwidth.  At D = 256 a decode CTA takes a
    // whole SM, so the CTAs must fit in one wave: floor(SMs / base).  Otherwise
    // about one CTA per SM (two at D = 64, whose CTAs are lighter), rounded to
    // the nearest power of two: with power-of-two caches the splits then cut the
    // keys into whole 128-key groups (four warps x 32 keys), and the measured
    // optimum sat there (B1 Hq32 Hkv8 Sk32768: 16 splits 27.5 us, 19 splits
    // 28.2; B4 Hq32 Hkv4 Sk32768 D64: 16 splits 28.9, 10 splits 30.4).
    if (D == 256) {
      ns = n_sm / base > 1 ? n_sm / base : 1;
    } else {
      const long long ctas = (D == 64 ? 2ll : 1ll) * n_sm;
      const double t = static_cast<double>((ctas + base - 1) / base);
      ns = 1ll << std::lround(std::log2(t));
    }
    // Each split keeps at least 128 KB of K and V per KV head (128 keys at
    // D = 256, 256 at D = 128, 512 at D = 64): single-sequence B1 Hq32 Hkv8 Sk4096 gets 16
    // splits, 8.9 us against the 13.4 of an earlier 1024-key floor, and
    // B1 Hq32 Hkv8 Sk8192 D64 16 splits (11.1 us; 32 splits 13.9).  At most 32
    // splits, the combine's one pass over a warp of partials: with one or two
    // CTAs per split more only lengthen the combine's serial loop over them
    // (B1 Hq8 Hkv1 Sk16384: 64 splits 16.7 us, 32 13.4).
    if (ns > 32) ns = 32;
    const long long min_keys = 32768 / D;
    const long long cap = Sk / min_keys > 1 ? Sk / min_keys : 1;
    if (ns > cap) ns = cap;
  }
  *num_splits = static_cast<int>(ns);
  return ATTN_OK;
}

int attn_combine(const float* o_part, const float* lse_part, float* o, float* lse, int B, int Hq,
                 int D, int num_splits, void* stream) {
  if (!o_part || !lse_part || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || D <= 0 || num_splits < 1) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(num_splits) * B * Hq * D > kMaxElems ||
      static_cast<long long>(B) * Hq > (1ll << 30))
    return ATTN_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(o_part) || !aligned16(lse_part) || !aligned16(o) || !aligned16(lse))
    return ATTN_ERR_MISALIGNED;
  const cudaError_t e = launch_combine(o_part, lse_part, o, lse, B * Hq, D, num_splits,
                                       static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The checks that the page tables share; ATTN_OK or the status to return.
int pages_check_args(const int* block_table, const int* refs, const int* block_table_out,
                     const int* refs_out, int B, int max_pages, int num_pages, int page_size) {
  if (!block_table || !refs || !block_table_out || !refs_out) return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0) return ATTN_ERR_INVALID_ARG;
  // Slots of the table are numbered, and keys counted, with int.
  if (static_cast<long long>(B) * max_pages > (1ll << 31) - 1 ||
      static_cast<long long>(max_pages) * page_size > kMaxSeq || num_pages > kMaxSeq)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned4(block_table) || !aligned4(refs) || !aligned4(block_table_out) ||
      !aligned4(refs_out))
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

}  // namespace

int attn_pages_free(const int* block_table, const int* refs, const int* seqlens,
                    int* block_table_out, int* refs_out, int B, int max_pages, int num_pages,
                    int page_size, int window, int sinks, int room, void* stream) {
  if (!seqlens || window < 1 || sinks < 0 || room < 0) return ATTN_ERR_INVALID_ARG;
  const int chk = pages_check_args(block_table, refs, block_table_out, refs_out, B, max_pages,
                                   num_pages, page_size);
  if (chk != ATTN_OK) return chk;
  if (!aligned4(seqlens)) return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  // Past the rows' capacity a window reaches every key: clamped, the sums fit int.
  const cudaError_t e = launch_pages_free(
      block_table, refs, seqlens, block_table_out, refs_out, B, max_pages, num_pages, page_size,
      window < kMaxSeq ? window : kMaxSeq, sinks, room, static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_pages_fork(const int* block_table, const int* refs, const int* seqlens,
                    const int* parents, int* block_table_out, int* refs_out, int* seqlens_out,
                    int* src, int* dst, int* counts, int* workspace, int B, int R, int max_pages,
                    int num_pages, int page_size, int room, void* stream) {
  if (!seqlens || !parents || !seqlens_out || !src || !dst || !counts || !workspace)
    return ATTN_ERR_INVALID_ARG;
  if (R <= 0 || room < 0) return ATTN_ERR_INVALID_ARG;
  const int chk = pages_check_args(block_table, refs, block_table_out, refs_out, B, max_pages,
                                   num_pages, page_size);
  if (chk != ATTN_OK) return chk;
  // (A row's number and the rows in flight at once are added as ints.)
  if (static_cast<long long>(R) * max_pages > (1ll << 31) - 1 || R > kMaxSeq)
    return ATTN_ERR_UNSUPPORTED;
  // The phases read their inputs after other CTAs have written outputs.
  if (block_table_out == block_table || refs_out == refs || seqlens_out == seqlens ||
      seqlens_out == parents || src == parents || dst == parents || src == dst)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned4(seqlens) || !aligned4(parents) || !aligned4(seqlens_out) || !aligned4(src) ||
      !aligned4(dst) || !aligned4(counts) || !aligned4(workspace))
    return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e = launch_pages_fork(
      block_table, refs, seqlens, parents, block_table_out, refs_out, seqlens_out, src, dst, counts,
      workspace, B, R, max_pages, num_pages, page_size, room, static_cast<cudaStream_t>(stream),
      status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_pages_compact(const int* block_table, const int* refs, int* block_table_out,
                       int* refs_out, int* src, int* dst, int* num_live, int* workspace, int B,
                       int max_pages, int num_pages, void* stream) {
  if (!num_live || !workspace || (num_pages > 1 && (!src || !dst))) return ATTN_ERR_INVALID_ARG;
  const int chk = pages_check_args(block_table, refs, block_table_out, refs_out, B, max_pages,
                                   num_pages, 1);
  if (chk != ATTN_OK) return chk;
  if (block_table_out == block_table || refs_out == refs || (src != nullptr && src == dst))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned4(src) || !aligned4(dst) || !aligned4(num_live) || !aligned4(workspace))
    return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e = launch_pages_compact(
      block_table, refs, block_table_out, refs_out, src, dst, num_live, workspace, B, max_pages,
      num_pages, static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_pages_workspace(int num_pages, int R, long long* entries) {
  if (entries == nullptr || num_pages < 1 || R < 0) return ATTN_ERR_INVALID_ARG;
  *entries = pages_workspace(num_pages, R);
  return ATTN_OK;
}

int attn_pages_copy(void* k_cache, void* v_cache, const int* src, const int* dst, int n,
                    int num_pages, long long page_bytes, void* stream) {
  if (!k_cache || !v_cache || n < 0 || num_pages <= 0 || page_bytes <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (n > 0 && (!src || !dst)) return ATTN_ERR_INVALID_ARG;
  if (page_bytes % 16 != 0 || num_pages > kMaxSeq) return ATTN_ERR_UNSUPPORTED;
  if (page_bytes > (2ll * kMaxElems) / num_pages) return ATTN_ERR_UNSUPPORTED;
  if (page_bytes > (1ll << 40)) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned4(src) || !aligned4(dst))
    return ATTN_ERR_MISALIGNED;
  if (n == 0) return ATTN_OK;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e = launch_pages_copy(k_cache, v_cache, src, dst, n, num_pages, page_bytes,
                                          static_cast<cudaStream_t>(stream), status);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_wait_selftest(unsigned long long limit_ns, unsigned long long* waited_ns, void* stream) {
  if (limit_ns < 1000ull || limit_ns > 1000000000ull) return ATTN_ERR_INVALID_ARG;
  if (waited_ns != nullptr && (reinterpret_cast<uintptr_t>(waited_ns) & 7u) != 0)
    return ATTN_ERR_MISALIGNED;
  int* status = status_word_device_ptr();
  if (status == nullptr) return ATTN_ERR_CUDA;
  const cudaError_t e =
      launch_wait_selftest(limit_ns, status, reinterpret_cast<uint64_t*>(waited_ns),
                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int attn_debug_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return ATTN_ERR_CUDA;
  int value = 0;
  if (cudaMemcpyFromSymbol(&value, g_status_word, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int)) != cudaSuccess) return ATTN_ERR_CUDA;
  return value;
}

}  // extern "C"
