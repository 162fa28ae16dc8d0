// extern "C" entry points of libbtq: host-side argument checks, then the
// launchers in calib.hip, select.hip, compress.hip, decompress.hip, rows.hip,
// matmul8.hip, heads.hip, kvcache.hip and attention.hip.
// The contract of each call is documented in include/btq.h.
#include <math.h>

#include <mutex>

#include "btq.h"
#include "common.hpp"

// Scratch of btq_calib_update_noalloc: a file-scope device array, one copy
// on each GPU the library runs on, held until the process ends. Host code
// never uses this name as an address (on the host it is only a stand-in);
// it passes the device address that hipGetSymbolAddress returns for the
// current device.
static __device__ __align__(256) float scratch[BTQ_NOALLOC_SCRATCH_BYTES / sizeof(float)];

namespace {

constexpr int64_t kMaxP = 65535;
constexpr int64_t kMaxH = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 62;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// P in [1,kMaxP], H in [1,kMaxH], T >= t_min, P*T*H < 2^62.
int check_dims(int64_t P, int64_t T, int64_t H, int64_t t_min) {
  if (P < 1 || P > kMaxP || H < 1 || H > kMaxH || T < t_min) return BTQ_ERR_SHAPE;
  if (T > 0 && T > kMaxElems / (P * H)) return BTQ_ERR_SHAPE;
  return BTQ_OK;
}

int check_k(int64_t H, int64_t k) { return (k < 0 || k > H) ? BTQ_ERR_SHAPE : BTQ_OK; }

int hip_status(hipError_t e) { return e == hipSuccess ? BTQ_OK : BTQ_ERR_HIP; }

// Packed row pitch: at least the row's code bytes, and P*T*pitch < 2^62.
int check_pitch(int64_t P, int64_t T, int64_t H, int64_t k, int64_t pitch) {
  if (pitch < (H - k + 1) / 2 || pitch > kMaxElems) return BTQ_ERR_SHAPE;
  if (T > 0 && pitch > 0 && T > kMaxElems / (P * pitch)) return BTQ_ERR_SHAPE;
  return BTQ_OK;
}

constexpr int kMaxDevices = 256;
std::mutex g_scratch_mu;
void* g_scratch_addr[kMaxDevices];   // `scratch` on each device, looked up once

// The current device's address of `scratch`: looked up on the first call on
// that device, with it current, and kept.
int scratch_address(float** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return BTQ_ERR_HIP;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_addr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) {
      (void)hipGetLastError();
      return BTQ_ERR_HIP;
    }
    g_scratch_addr[dev] = p;
  }
  *out = static_cast<float*>(g_scratch_addr[dev]);
  return BTQ_OK;
}

}  // namespace

extern "C" {

int64_t btq_packed_row_bytes(int64_t H, int64_t k) {
  if (H < 1 || k < 0 || k > H) return -1;
  return (H - k + 1) / 2;
}

int64_t btq_packed_pitch(int64_t H, int64_t k) {
  const int64_t b = btq_packed_row_bytes(H, k);
  return b < 0 ? -1 : (b + 127) / 128 * 128;
}

size_t btq_calib_workspace_bytes(int64_t P, int64_t T, int64_t H) {
  if (check_dims(P, T, H, 1) != BTQ_OK) return 0;
  const btq::CalibPlan plan = btq::calib_plan(P, T, H);
  return (size_t)(2 * plan.nchunk * P * H) * sizeof(float);
}

size_t btq_select_workspace_bytes(int64_t P, int64_t H, int64_t k) {
  if (P < 1 || P > kMaxP || H < 1 || H > kMaxH || check_k(H, k) != BTQ_OK) return 0;
  return (size_t)(P * H) * sizeof(float);   // per-shard widths; the shared score uses H
}

int btq_calib_update(const uint16_t* x, int64_t P, int64_t T, int64_t H, float momentum,
                     int first_batch, float* run_min, float* run_max, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int st = check_dims(P, T, H, 1);
  if (st != BTQ_OK) return st;
  if (!x || !run_min || !run_max) return BTQ_ERR_ARG;
  if (!(momentum >= 0.0f && momentum < 1.0f)) return BTQ_ERR_ARG;   // also rejects NaN
  if (!aligned(x, 2) || !aligned(run_min, 4) || !aligned(run_max, 4)) return BTQ_ERR_ALIGN;
  const size_t need = btq_calib_workspace_bytes(P, T, H);
  if (need > 0 && !workspace) return BTQ_ERR_ARG;
  if (workspace_bytes < need) return BTQ_ERR_WORKSPACE;
  if (!aligned(workspace, 4)) return BTQ_ERR_ALIGN;
  const float a = momentum;
  const float c = 1.0f - a;   // one fp32 subtraction
  return hip_status(btq::launch_calib(x, P, T, H, a, c, first_batch != 0, run_min, run_max,
                                      (float*)workspace, (hipStream_t)stream));
}

int btq_calib_update_noalloc(const uint16_t* x, int64_t P, int64_t T, int64_t H, float momentum,
                             int first_batch, float* run_min, float* run_max, void* stream) {
  int st = check_dims(P, T, H, 1);
  if (st != BTQ_OK) return st;
  if (!x || !run_min || !run_max) return BTQ_ERR_ARG;
  if (!(momentum >= 0.0f && momentum < 1.0f)) return BTQ_ERR_ARG;   // also rejects NaN
  if (!aligned(x, 2) || !aligned(run_min, 4) || !aligned(run_max, 4)) return BTQ_ERR_ALIGN;
  // the same kernels with as many token chunks as the scratch holds partials for
  const btq::CalibPlan plan =
      btq::calib_plan_capped(P, T, H, (int64_t)(BTQ_NOALLOC_SCRATCH_BYTES / sizeof(float)));
  if (plan.nchunk < 1) return BTQ_ERR_SCRATCH;
  float* ws = nullptr;
  st = scratch_address(&ws);
  if (st != BTQ_OK) return st;
  const float a = momentum;
  const float c = 1.0f - a;
  return hip_status(btq::launch_calib_plan(x, P, T, H, a, c, first_batch != 0, run_min, run_max,
                                           ws, plan, (hipStream_t)stream));
}

namespace {

// Shared checks of the selection calls' parameter and map outputs.
int check_select_outputs(const float* run_min, const float* run_max, int64_t P, int64_t H,
                         int64_t k, const float* scale, const float* rscale,
                         const uint8_t* zero_point, const int32_t* outlier_idx,
                         const int32_t* fmap, const int32_t* cmap) {
  if (P < 1 || P > kMaxP || H < 1 || H > kMaxH) return BTQ_ERR_SHAPE;
  int st = check_k(H, k);
  if (st != BTQ_OK) return st;
  if (!run_min || !run_max || !scale || !rscale || !zero_point || !fmap) return BTQ_ERR_ARG;
  if ((k > 0 && !outlier_idx) || (k < H && !cmap)) return BTQ_ERR_ARG;
  if (!aligned(run_min, 4) || !aligned(run_max, 4) || !aligned(scale, 4) ||
      !aligned(rscale, 4) || !aligned(outlier_idx, 4) || !aligned(fmap, 4) || !aligned(cmap, 4))
    return BTQ_ERR_ALIGN;
  return BTQ_OK;
}

int check_workspace(int64_t P, int64_t H, int64_t k, const void* workspace, size_t bytes) {
  if (!workspace) return BTQ_ERR_ARG;
  if (bytes < btq_select_workspace_bytes(P, H, k)) return BTQ_ERR_WORKSPACE;
  if (!aligned(workspace, 4)) return BTQ_ERR_ALIGN;
  return BTQ_OK;
}

}  // namespace

int btq_select_outliers(const float* run_min, const float* run_max, int64_t P, int64_t H,
                        int64_t k, float* scale, float* rscale, uint8_t* zero_point,
                        int32_t* outlier_idx, int32_t* fmap, int32_t* cmap, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return btq_select_outliers_rule(run_min, run_max, P, H, k, BTQ_SCORE_SUM, scale, rscale,
                                  zero_point, outlier_idx, fmap, cmap, workspace,
                                  workspace_bytes, stream);
}

int btq_select_outliers_rule(const float* run_min, const float* run_max, int64_t P, int64_t H,
                             int64_t k, int score_rule, float* scale, float* rscale,
                             uint8_t* zero_point, int32_t* outlier_idx, int32_t* fmap,
                             int32_t* cmap, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int st = check_select_outputs(run_min, run_max, P, H, k, scale, rscale, zero_point, outlier_idx,
                                fmap, cmap);
  if (st != BTQ_OK) return st;
  if (score_rule != BTQ_SCORE_SUM && score_rule != BTQ_SCORE_MAX) return BTQ_ERR_ARG;
  st = check_workspace(P, H, k, workspace, workspace_bytes);
  if (st != BTQ_OK) return st;
  return hip_status(btq::launch_select(run_min, run_max, P, H, k, scale, rscale, zero_point,
                                       outlier_idx, fmap, cmap, (float*)workspace,
                                       score_rule == BTQ_SCORE_MAX, (hipStream_t)stream));
}

int btq_select_outliers_per_shard(const float* run_min, const float* run_max, int64_t P,
                                  int64_t H, int64_t k, float* scale, float* rscale,
                                  uint8_t* zero_point, int32_t* outlier_idx, int32_t* fmap,
                                  int32_t* cmap, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  int st = check_select_outputs(run_min, run_max, P, H, k, scale, rscale, zero_point, outlier_idx,
                                fmap, cmap);
  if (st != BTQ_OK) return st;
  st = check_workspace(P, H, k, workspace, workspace_bytes);
  if (st != BTQ_OK) return st;
  return hip_status(btq::launch_select_per_shard(run_min, run_max, P, H, k, scale, rscale,
                                                 zero_point, outlier_idx, fmap, cmap,
                                                 (float*)workspace, (hipStream_t)stream));
}

int btq_select_features(const float* run_min, const float* run_max, int64_t P, int64_t H,
                        int64_t k, const int32_t* features, float* scale, float* rscale,
                        uint8_t* zero_point, int32_t* outlier_idx, int32_t* fmap, int32_t* cmap,
                        void* stream) {
  int st = check_select_outputs(run_min, run_max, P, H, k, scale, rscale, zero_point, outlier_idx,
                                fmap, cmap);
  if (st != BTQ_OK) return st;
  if (k > 0 && !features) return BTQ_ERR_ARG;
  if (!aligned(features, 4)) return BTQ_ERR_ALIGN;
  for (int64_t i = 0; i < k; ++i) {   // distinct, ascending, inside [0, H)
    const int64_t h = features[i];
    if (h < 0 || h >= H || (i > 0 && h <= features[i - 1])) return BTQ_ERR_ARG;
  }
  const hipStream_t s = (hipStream_t)stream;
  if (k > 0) {
    const hipError_t e = hipMemcpyAsync(outlier_idx, features, (size_t)k * sizeof(int32_t),
                                        hipMemcpyHostToDevice, s);
    if (e != hipSuccess) return BTQ_ERR_HIP;
  }
  return hip_status(btq::launch_select_set(run_min, run_max, P, H, k, scale, rscale, zero_point,
                                           outlier_idx, fmap, cmap, s));
}

int btq_compress_pack_ex(const uint16_t* x, int64_t P, int64_t T, int64_t H, int64_t k,
                         const float* rscale, const uint8_t* zero_point,
                         const int32_t* outlier_idx, const int32_t* cmap, int sets,
                         uint8_t* packed, int64_t packed_pitch, uint16_t* outliers,
                         void* stream) {
  int st = check_dims(P, T, H, 0);
  if (st != BTQ_OK) return st;
  st = check_k(H, k);
  if (st != BTQ_OK) return st;
  st = check_pitch(P, T, H, k, packed_pitch);
  if (st != BTQ_OK) return st;
  if (sets != BTQ_SETS_SHARED && sets != BTQ_SETS_PER_SHARD) return BTQ_ERR_ARG;
  if (!rscale || !zero_point || (k > 0 && !outlier_idx) || (k < H && !cmap)) return BTQ_ERR_ARG;
  if (T > 0 && (!x || (k < H && !packed) || (k > 0 && !outliers))) return BTQ_ERR_ARG;
  if (!aligned(x, 2) || !aligned(rscale, 4) || !aligned(outlier_idx, 4) || !aligned(cmap, 4) ||
      !aligned(outliers, 2))
    return BTQ_ERR_ALIGN;
  if (T == 0) return BTQ_OK;
  return hip_status(btq::launch_compress(x, P, T, H, k, rscale, zero_point, outlier_idx, cmap,
                                         packed, packed_pitch, outliers,
                                         sets == BTQ_SETS_PER_SHARD, (hipStream_t)stream));
}

int btq_compress_pack(const uint16_t* x, int64_t P, int64_t T, int64_t H, int64_t k,
                      const float* rscale, const uint8_t* zero_point, const int32_t* outlier_idx,
                      const int32_t* cmap, uint8_t* packed, uint16_t* outliers, void* stream) {
  return btq_compress_pack_ex(x, P, T, H, k, rscale, zero_point, outlier_idx, cmap,
                              BTQ_SETS_SHARED, packed, btq_packed_row_bytes(H, k), outliers,
                              stream);
}

int btq_compress_pack_per_shard(const uint16_t* x, int64_t P, int64_t T, int64_t H, int64_t k,
                                const float* rscale, const uint8_t* zero_point,
                                const int32_t* outlier_idx, const int32_t* cmap, uint8_t* packed,
                                uint16_t* outliers, void* stream) {
  return btq_compress_pack_ex(x, P, T, H, k, rscale, zero_point, outlier_idx, cmap,
                              BTQ_SETS_PER_SHARD, packed, btq_packed_row_bytes(H, k), outliers,
                              stream);
}

int btq_decompress_reduce_ex(const uint8_t* packed, int64_t packed_pitch,
                             const uint16_t* outliers, int64_t P, int64_t T, int64_t H, int64_t k,
                             const float* scale, const uint8_t* zero_point, const int32_t* fmap,
                             int sets, void* y, int y_type, void* stream) {
  int st = check_dims(P, T, H, 0);
  if (st != BTQ_OK) return st;
  st = check_k(H, k);
  if (st != BTQ_OK) return st;
  st = check_pitch(P, T, H, k, packed_pitch);
  if (st != BTQ_OK) return st;
  if (sets != BTQ_SETS_SHARED && sets != BTQ_SETS_PER_SHARD) return BTQ_ERR_ARG;
  if (y_type != BTQ_Y_F32 && y_type != BTQ_Y_BF16) return BTQ_ERR_ARG;
  if (!scale || !zero_point || !fmap) return BTQ_ERR_ARG;
  if (T > 0 && (!y || (k < H && !packed) || (k > 0 && !outliers))) return BTQ_ERR_ARG;
  const bool bf16 = y_type == BTQ_Y_BF16;
  if (!aligned(outliers, 2) || !aligned(scale, 4) || !aligned(fmap, 4) ||
      !aligned(y, bf16 ? 2 : 4))
    return BTQ_ERR_ALIGN;
  if (T == 0) return BTQ_OK;
  return hip_status(btq::launch_decompress(packed, packed_pitch, outliers, P, T, H, k, scale,
                                           zero_point, fmap, sets == BTQ_SETS_PER_SHARD, y, bf16,
                                           (hipStream_t)stream));
}

int btq_decompress_reduce(const uint8_t* packed, const uint16_t* outliers, int64_t P, int64_t T,
                          int64_t H, int64_t k, const float* scale, const uint8_t* zero_point,
                          const int32_t* fmap, float* y, void* stream) {
  return btq_decompress_reduce_ex(packed, btq_packed_row_bytes(H, k), outliers, P, T, H, k, scale,
                                  zero_point, fmap, BTQ_SETS_SHARED, y, BTQ_Y_F32, stream);
}

int btq_decompress_reduce_bf16(const uint8_t* packed, const uint16_t* outliers, int64_t P,
                               int64_t T, int64_t H, int64_t k, const float* scale,
                               const uint8_t* zero_point, const int32_t* fmap, uint16_t* y,
                               void* stream) {
  return btq_decompress_reduce_ex(packed, btq_packed_row_bytes(H, k), outliers, P, T, H, k, scale,
                                  zero_point, fmap, BTQ_SETS_SHARED, y, BTQ_Y_BF16, stream);
}

int btq_decompress_reduce_per_shard(const uint8_t* packed, const uint16_t* outliers, int64_t P,
                                    int64_t T, int64_t H, int64_t k, const float* scale,
                                    const uint8_t* zero_point, const int32_t* fmap, float* y,
                                    void* stream) {
  return btq_decompress_reduce_ex(packed, btq_packed_row_bytes(H, k), outliers, P, T, H, k, scale,
                                  zero_point, fmap, BTQ_SETS_PER_SHARD, y, BTQ_Y_F32, stream);
}

namespace {

bool value_type(int t) { return t == BTQ_T_F32 || t == BTQ_T_BF16; }
size_t value_align(int t) { return t == BTQ_T_F32 ? 4 : t == BTQ_T_BF16 ? 2 : 1; }

// Largest K whose sum of K products of two codes (at most 2^14 each) stays
// inside int32.
constexpr int64_t kMaxSumK = 131071;

// Row strides of a [P,T,K] tensor: not negative, and P, T steps of them stay
// inside 2^62 elements.
int check_strides(int64_t P, int64_t T, int64_t shard, int64_t pitch) {
  if (shard < 0 || pitch < 0) return BTQ_ERR_SHAPE;
  if (shard > kMaxElems / P || (T > 0 && pitch > kMaxElems / T)) return BTQ_ERR_SHAPE;
  return BTQ_OK;
}

int check_matmul(int64_t as_shard, const int8_t* w, const float* w_scale, const float* bias,
                 int64_t P, int64_t T, int64_t N, int64_t K, const void* y, int y_type) {
  int st = check_dims(P, T, K, 0);
  if (st == BTQ_OK) st = check_dims(P, T, N, 0);
  if (st == BTQ_OK) st = check_dims(P, N, K, 0);
  if (st != BTQ_OK) return st;
  if (N > kMaxH || N < 1 || K > kMaxSumK) return BTQ_ERR_SHAPE;
  if (as_shard < 0 || as_shard > kMaxElems / P) return BTQ_ERR_SHAPE;
  if (!value_type(y_type) || !w || !w_scale || (T > 0 && !y)) return BTQ_ERR_ARG;
  if (!aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(y, value_align(y_type)))
    return BTQ_ERR_ALIGN;
  return BTQ_OK;
}

// Workspace of btq_int8_linear: the codes with rows padded to 16 bytes, then
// the scales. Its bytes stay inside 2^62 too (short rows grow up to 20 times).
int64_t code_pitch(int64_t K) { return (K + 15) / 16 * 16; }
int64_t code_row_bytes(int64_t K) { return code_pitch(K) + (int64_t)sizeof(float); }
int check_linear_workspace(int64_t P, int64_t T, int64_t K) {
  return K < 1 || K > kMaxSumK ? BTQ_ERR_SHAPE : check_dims(P, T, code_row_bytes(K), 0);
}

// ---- heads, the paged cache and attention ----

// Heads of one tensor: strides >= 0 whose largest element stays inside 2^62.
int check_head_rows(int64_t P, int64_t T, int64_t H, int64_t D, int64_t shard, int64_t pitch,
                    int64_t head) {
  if (shard < 0 || pitch < 0 || head < 0) return BTQ_ERR_SHAPE;
  const int64_t most = kMaxElems / 4;
  if (P > 1 && shard > most / P) return BTQ_ERR_SHAPE;
  if (T > 1 && pitch > most / T) return BTQ_ERR_SHAPE;
  if (H > 1 && head > most / H) return BTQ_ERR_SHAPE;
  return D > most ? BTQ_ERR_SHAPE : BTQ_OK;
}

// Heads that a call writes, too: no element may belong to two of them, or lanes would
// write it in no order. From the smallest stride on, each is at least what those before
// it span.
int check_out_rows(int64_t P, int64_t T, int64_t H, int64_t D, int64_t shard, int64_t pitch,
                   int64_t head) {
  const int st = check_head_rows(P, T, H, D, shard, pitch, head);
  if (st != BTQ_OK) return st;
  int64_t stride[3] = {head, pitch, shard}, count[3] = {H, T, P}, span = D;
  for (int i = 0; i < 3; ++i) {
    int least = i;
    for (int j = i + 1; j < 3; ++j)
      if (count[j] > 1 && (count[least] <= 1 || stride[j] < stride[least])) least = j;
    if (count[least] <= 1) return BTQ_OK;
    if (stride[least] < span) return BTQ_ERR_SHAPE;
    span += stride[least] * (count[least] - 1);
    stride[least] = stride[i], count[least] = count[i];
  }
  return BTQ_OK;
}

int check_rope(const float* cos, const float* sin, int64_t rows, int64_t dim, int64_t D, int rope) {
  if (rope != BTQ_ROPE_HALF && rope != BTQ_ROPE_PAIRS) return BTQ_ERR_ARG;
  if (!cos != !sin) return BTQ_ERR_ARG;
  if (!cos) return BTQ_OK;
  if (rows < 1 || rows > (int64_t(1) << 31) || dim < 2 || dim % 2 != 0 || dim > D)
    return BTQ_ERR_SHAPE;
  return aligned(cos, 4) && aligned(sin, 4) ? BTQ_OK : BTQ_ERR_ALIGN;
}

bool head_features(int64_t D) { return D >= 32 && D <= 256 && D % 32 == 0; }
constexpr int64_t kMaxPlaces = int64_t(1) << 30;
constexpr int64_t kMaxKvBlocks = int64_t(1) << 23;   // thread blocks of a launch over places

// Sizes of the batch, its cache and table.
int check_kv_sizes(int64_t P, int64_t T, int64_t Hk, int64_t D, int64_t B, int64_t max_pages,
                   int64_t page_size) {
  if (P < 1 || P > kMaxP || T < 0 || T > kMaxPlaces || Hk < 1 || Hk > kMaxP || B < 0 ||
      B > kMaxPlaces || !head_features(D))
    return BTQ_ERR_SHAPE;
  if (page_size < 32 || page_size > 65536 || (page_size & (page_size - 1)) != 0 || max_pages < 0 ||
      max_pages > kMaxPlaces / page_size)
    return BTQ_ERR_SHAPE;
  // a grid over all places that the rows can touch
  return (T / 32 + 2 * B) > kMaxKvBlocks / (P * Hk) ? BTQ_ERR_SHAPE : BTQ_OK;
}

int check_kv(int64_t P, int64_t T, int64_t Hk, int64_t D, const int32_t* starts,
             const int32_t* lengths, int64_t B, const int32_t* table, int64_t max_pages,
             const uint8_t* cache, int64_t pages, int64_t page_size) {
  const int st = check_kv_sizes(P, T, Hk, D, B, max_pages, page_size);
  if (st != BTQ_OK) return st;
  if (pages < 1 || pages > kMaxElems / (P * Hk * (page_size / 32) * btq_kv_block_bytes(D)) ||
      pages >= (int64_t(1) << 31))
    return BTQ_ERR_SHAPE;
  if (B > 0 && T > 0 && (!starts || !lengths || (max_pages > 0 && !table) || !cache))
    return BTQ_ERR_ARG;
  if (!aligned(starts, 4) || !aligned(lengths, 4) || !aligned(table, 4) || !aligned(cache, 16))
    return BTQ_ERR_ALIGN;
  return BTQ_OK;
}

btq::KvArgs kv_args(int64_t P, int64_t T, int64_t Hk, int64_t D, const int32_t* starts,
                    const int32_t* lengths, int64_t B, const int32_t* table, int64_t max_pages,
                    const uint8_t* cache, int64_t pages, int64_t page_size) {
  int shift = 0;
  while ((int64_t(32) << shift) < page_size) ++shift;
  if (max_pages == 0) table = starts;   // (an address that may be read; no entry counts)
  return {P, T, (int)B, (int)Hk, (int)D, starts, lengths, table, max_pages,
          (int)(max_pages * page_size), const_cast<uint8_t*>(cache), pages, shift};
}

int check_attention_sizes(int64_t P, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B,
                          int64_t max_pages, int64_t page_size, int64_t max_length) {
  const int st = check_kv_sizes(P, T, Hk, D, B, max_pages, page_size);
  if (st != BTQ_OK) return st;
  if (Hq < 1 || Hq > kMaxP / 2 || Hq % Hk != 0 || max_length < 0 || max_length > kMaxPlaces)
    return BTQ_ERR_SHAPE;
  const int64_t G = Hq / Hk;
  return T > kMaxPlaces / 2 / G ? BTQ_ERR_SHAPE : BTQ_OK;
}
btq::AttnPlan plan_attention(int64_t P, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t B,
                             int64_t max_pages, int64_t page_size, int64_t max_length) {
  const int64_t places = max_pages * page_size;
  return btq::attn_plan(P, T, (int)Hq, (int)Hk, (int)D, (int)B,
                        max_length == 0 || max_length > places ? places : max_length);
}

}  // namespace

int btq_quantize_rows(const void* x, int x_type, int64_t x_shard, int64_t x_pitch, int64_t P,
                      int64_t T, int64_t K, int8_t* q, float* scale, void* stream) {
  int st = check_dims(P, T, K, 0);
  if (st == BTQ_OK) st = check_strides(P, T, x_shard, x_pitch);
  if (st != BTQ_OK) return st;
  if (!value_type(x_type) || (T > 0 && (!x || !q || !scale))) return BTQ_ERR_ARG;
  if (!aligned(x, value_align(x_type)) || !aligned(scale, 4)) return BTQ_ERR_ALIGN;
  if (T == 0) return BTQ_OK;
  return hip_status(btq::launch_quantize_rows(x, x_type, x_shard, x_pitch, P, T, K, q, K, scale,
                                              (hipStream_t)stream));
}

int btq_int8_matmul(const int8_t* a, int64_t a_shard, int64_t a_pitch, const float* a_scale,
                    int64_t as_shard, const int8_t* w, const float* w_scale, const float* bias,
                    int64_t P, int64_t T, int64_t N, int64_t K, void* y, int y_type,
                    void* stream) {
  int st = check_matmul(as_shard, w, w_scale, bias, P, T, N, K, y, y_type);
  if (st == BTQ_OK) st = check_strides(P, T, a_shard, a_pitch);
  if (st != BTQ_OK) return st;
  if (T > 0 && (!a || !a_scale)) return BTQ_ERR_ARG;
  if (!aligned(a_scale, 4)) return BTQ_ERR_ALIGN;
  if (T == 0) return BTQ_OK;
  const btq::MatmulArgs m = {a, a_shard, a_pitch, a_scale, as_shard, w, w_scale, bias,
                             P, T, N, K, y, y_type};
  return hip_status(btq::launch_int8_matmul(m, (hipStream_t)stream));
}

size_t btq_int8_linear_workspace_bytes(int64_t P, int64_t T, int64_t K) {
  if (check_linear_workspace(P, T, K) != BTQ_OK) return 0;
  return (size_t)(P * T * code_row_bytes(K));
}

int btq_int8_linear(const void* x, int x_type, int64_t x_shard, int64_t x_pitch, const int8_t* w,
                    const float* w_scale, const float* bias, int64_t P, int64_t T, int64_t N,
                    int64_t K, void* y, int y_type, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int st = check_matmul(0, w, w_scale, bias, P, T, N, K, y, y_type);
  if (st == BTQ_OK) st = check_strides(P, T, x_shard, x_pitch);
  if (st == BTQ_OK) st = check_linear_workspace(P, T, K);
  if (st != BTQ_OK) return st;
  if (!value_type(x_type) || (T > 0 && (!x || !workspace))) return BTQ_ERR_ARG;
  if (!aligned(x, value_align(x_type)) || !aligned(workspace, 16)) return BTQ_ERR_ALIGN;
  if (workspace_bytes < btq_int8_linear_workspace_bytes(P, T, K)) return BTQ_ERR_WORKSPACE;
  if (T == 0) return BTQ_OK;
  const int64_t pitch = code_pitch(K);
  const int64_t rows = x_shard == 0 ? 1 : P;   // shards of activations
  int8_t* q = (int8_t*)workspace;
  float* scale = (float*)(q + P * T * pitch);
  const btq::MatmulArgs m = {q, rows == 1 ? 0 : T * pitch, pitch, scale, rows == 1 ? 0 : T,
                             w, w_scale, bias, P, T, N, K, y, y_type};
  if (btq::small_linear_ok(x, x_type, x_shard, x_pitch, m))
    return hip_status(btq::launch_small_linear(x, x_shard, x_pitch, m, (hipStream_t)stream));
  st = hip_status(btq::launch_quantize_rows(x, x_type, x_shard, x_pitch, rows, T, K, q, pitch,
                                            scale, (hipStream_t)stream));
  if (st != BTQ_OK) return st;
  return hip_status(btq::launch_int8_matmul(m, (hipStream_t)stream));
}

int btq_block_norm(const void* y, int y_type, const void* residual, int r_type, int64_t T,
                   int64_t H, int post, const float* post_weight, const float* post_bias,
                   float post_eps, const void* gate, int gate_type, int64_t gate_rows,
                   float alpha, int pre, const float* pre_weight, const float* pre_bias,
                   float pre_eps, void* residual_out, void* n, int n_type, float* n_scale,
                   void* stream) {
  int st = check_dims(1, T, H, 0);
  if (st != BTQ_OK) return st;
  if (gate && (gate_rows < 1 || T % gate_rows != 0)) return BTQ_ERR_SHAPE;
  if (post < BTQ_NORM_NONE || post > BTQ_NORM_LAYER || pre < BTQ_NORM_NONE ||
      pre > BTQ_NORM_LAYER)
    return BTQ_ERR_ARG;
  if (!value_type(y_type) || !value_type(r_type) || !value_type(gate_type)) return BTQ_ERR_ARG;
  if (!value_type(n_type) && n_type != BTQ_T_INT8) return BTQ_ERR_ARG;
  if ((post_weight && post == BTQ_NORM_NONE) || (post_bias && post != BTQ_NORM_LAYER) ||
      (pre_weight && pre == BTQ_NORM_NONE) || (pre_bias && pre != BTQ_NORM_LAYER))
    return BTQ_ERR_ARG;
  if (!(post_eps >= 0.0f && post_eps < INFINITY) || !(pre_eps >= 0.0f && pre_eps < INFINITY) ||
      !(alpha > -INFINITY && alpha < INFINITY))
    return BTQ_ERR_ARG;
  if (T > 0 && (!residual || (!y && (post != BTQ_NORM_NONE || gate)) || (!residual_out && !n)))
    return BTQ_ERR_ARG;
  if ((n && n_type == BTQ_T_INT8) ? (T > 0 && !n_scale) : n_scale != nullptr) return BTQ_ERR_ARG;
  const size_t r_align = value_align(r_type);
  if (!aligned(y, value_align(y_type)) || !aligned(residual, r_align) ||
      !aligned(residual_out, r_align) || !aligned(gate, value_align(gate_type)) ||
      !aligned(n, value_align(n_type)) || !aligned(post_weight, 4) || !aligned(post_bias, 4) ||
      !aligned(pre_weight, 4) || !aligned(pre_bias, 4) || !aligned(n_scale, 4))
    return BTQ_ERR_ALIGN;
  if (T == 0) return BTQ_OK;
  const btq::NormArgs a = {y, residual, y_type, r_type, T, H, post, pre, post_weight, post_bias,
                           pre_weight, pre_bias, post_eps, pre_eps, gate, gate_type,
                           gate ? T / gate_rows : 1, alpha, residual_out, n, n_type, n_scale};
  return hip_status(btq::launch_block_norm(a, (hipStream_t)stream));
}

int64_t btq_kv_block_bytes(int64_t D) { return head_features(D) ? 32 * D + 256 : 0; }

int btq_head_norm_rope(const void* x, int x_type, int64_t x_shard, int64_t x_pitch, int64_t x_head,
                       int64_t P, int64_t T, int64_t q_heads, int64_t k_heads, int64_t D, int norm,
                       const float* q_weight, int64_t qw_shard, int64_t qw_head,
                       const float* k_weight, int64_t kw_shard, int64_t kw_head, float eps,
                       const int32_t* positions, const float* cos_table, const float* sin_table,
                       int64_t rope_rows, int64_t rope_dim, int rope, void* y, int y_type,
                       int64_t y_shard, int64_t y_pitch, int64_t y_head, void* stream) {
  if (q_heads < 0 || k_heads < 0 || q_heads > kMaxP || k_heads > kMaxP || q_heads + k_heads < 1 ||
      D < 1 || D > 65536)
    return BTQ_ERR_SHAPE;
  const int64_t H = q_heads + k_heads;
  int st = check_dims(P, T, H * D, 0);
  if (st == BTQ_OK) st = check_head_rows(P, T, H, D, x_shard, x_pitch, x_head);
  if (st == BTQ_OK) st = check_out_rows(P, T, H, D, y_shard, y_pitch, y_head);
  if (st == BTQ_OK) st = check_head_rows(P, 1, H, D, qw_shard, 0, qw_head);
  if (st == BTQ_OK) st = check_head_rows(P, 1, H, D, kw_shard, 0, kw_head);
  if (st == BTQ_OK) st = check_rope(cos_table, sin_table, rope_rows, rope_dim, D, rope);
  if (st != BTQ_OK) return st;
  if (!value_type(x_type) || !value_type(y_type) || norm < BTQ_NORM_NONE || norm > BTQ_NORM_LAYER ||
      !(eps >= 0.0f && eps < INFINITY))
    return BTQ_ERR_ARG;
  if (T > 0 && (!x || !y || (cos_table && !positions))) return BTQ_ERR_ARG;
  if (!aligned(x, value_align(x_type)) || !aligned(y, value_align(y_type)) ||
      !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(positions, 4))
    return BTQ_ERR_ALIGN;
  if (T == 0) return BTQ_OK;
  const btq::HeadArgs a = {
      {const_cast<void*>(x), x_type, x_shard, x_pitch, x_head},
      {y, y_type, y_shard, y_pitch, y_head},
      P, T, (int)q_heads, (int)k_heads, (int)D, norm, q_weight, k_weight,
      qw_shard, qw_head, kw_shard, kw_head, eps, positions,
      {cos_table, sin_table, rope_rows, (int)rope_dim, rope}};
  return hip_status(btq::launch_head_norm_rope(a, (hipStream_t)stream));
}

int btq_kv_append(const void* k, const void* v, int x_type, int64_t k_shard, int64_t k_pitch,
                  int64_t k_head, int64_t v_shard, int64_t v_pitch, int64_t v_head, int64_t P,
                  int64_t T, int64_t Hk, int64_t D, const int32_t* seq_starts,
                  const int32_t* lengths, int64_t B, const int32_t* page_table, int64_t max_pages,
                  const float* cos_table, const float* sin_table, int64_t rope_rows,
                  int64_t rope_dim, int rope, uint8_t* cache, int64_t pages, int64_t page_size,
                  void* stream) {
  int st = check_kv(P, T, Hk, D, seq_starts, lengths, B, page_table, max_pages, cache, pages,
                    page_size);
  if (st == BTQ_OK) st = check_head_rows(P, T, Hk, D, k_shard, k_pitch, k_head);
  if (st == BTQ_OK) st = check_head_rows(P, T, Hk, D, v_shard, v_pitch, v_head);
  if (st == BTQ_OK) st = check_rope(cos_table, sin_table, rope_rows, rope_dim, D, rope);
  if (st != BTQ_OK) return st;
  if (!value_type(x_type) || (T > 0 && B > 0 && (!k || !v))) return BTQ_ERR_ARG;
  if (!aligned(k, value_align(x_type)) || !aligned(v, value_align(x_type))) return BTQ_ERR_ALIGN;
  if (T == 0 || B == 0) return BTQ_OK;
  return hip_status(btq::launch_kv_append(
      {const_cast<void*>(k), x_type, k_shard, k_pitch, k_head},
      {const_cast<void*>(v), x_type, v_shard, v_pitch, v_head},
      {cos_table, sin_table, rope_rows, (int)rope_dim, rope},
      kv_args(P, T, Hk, D, seq_starts, lengths, B, page_table, max_pages, cache, pages, page_size),
      (hipStream_t)stream));
}

int btq_kv_gather(const int32_t* seq_starts, const int32_t* lengths, int64_t B,
                  const int32_t* page_table, int64_t max_pages, const uint8_t* cache,
                  int64_t pages, int64_t page_size, int64_t P, int64_t T, int64_t Hk, int64_t D,
                  void* k, void* v, int y_type, int64_t k_shard, int64_t k_pitch, int64_t k_head,
                  int64_t v_shard, int64_t v_pitch, int64_t v_head, void* stream) {
  int st = check_kv(P, T, Hk, D, seq_starts, lengths, B, page_table, max_pages, cache, pages,
                    page_size);
  if (st == BTQ_OK)
    st = k ? check_out_rows(P, T, Hk, D, k_shard, k_pitch, k_head)
           : check_head_rows(P, T, Hk, D, k_shard, k_pitch, k_head);
  if (st == BTQ_OK)
    st = v ? check_out_rows(P, T, Hk, D, v_shard, v_pitch, v_head)
           : check_head_rows(P, T, Hk, D, v_shard, v_pitch, v_head);
  if (st != BTQ_OK) return st;
  if (!value_type(y_type) || (T > 0 && B > 0 && !k && !v)) return BTQ_ERR_ARG;
  if (!aligned(k, value_align(y_type)) || !aligned(v, value_align(y_type))) return BTQ_ERR_ALIGN;
  if (T == 0 || B == 0) return BTQ_OK;
  return hip_status(btq::launch_kv_gather(
      {k, y_type, k_shard, k_pitch, k_head}, {v, y_type, v_shard, v_pitch, v_head},
      kv_args(P, T, Hk, D, seq_starts, lengths, B, page_table, max_pages, cache, pages, page_size),
      (hipStream_t)stream));
}

size_t btq_kv_attention_workspace_bytes(int64_t P, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                        int64_t B, int64_t max_pages, int64_t page_size,
                                        int64_t max_length) {
  if (check_attention_sizes(P, T, Hq, Hk, D, B, max_pages, page_size, max_length) != BTQ_OK ||
      T == 0 || B == 0)
    return 0;
  return plan_attention(P, T, Hq, Hk, D, B, max_pages, page_size, max_length).workspace;
}

int btq_kv_attention(const void* q, int64_t q_shard, int64_t q_pitch, int64_t q_head, int64_t P,
                     int64_t T, int64_t Hq, int64_t Hk, int64_t D, const int32_t* seq_starts,
                     const int32_t* lengths, int64_t B, const int32_t* page_table,
                     int64_t max_pages, const uint8_t* cache, int64_t pages, int64_t page_size,
                     float scale, int causal, int64_t window, int64_t max_length, void* out,
                     int out_type, float* lse, void* workspace, size_t workspace_bytes,
                     void* stream) {
  int st = check_attention_sizes(P, T, Hq, Hk, D, B, max_pages, page_size, max_length);
  if (st == BTQ_OK)
    st = check_kv(P, T, Hk, D, seq_starts, lengths, B, page_table, max_pages, cache, pages,
                  page_size);
  if (st == BTQ_OK) st = check_head_rows(P, T, Hq, D, q_shard, q_pitch, q_head);
  if (st != BTQ_OK) return st;
  if (window < 0) return BTQ_ERR_SHAPE;
  if (!value_type(out_type) || !(scale > 0.0f && scale <= 0x1p127f)) return BTQ_ERR_ARG;
  if (T > 0 && B > 0 && (!q || !out)) return BTQ_ERR_ARG;
  if (!aligned(q, 2) || !aligned(out, out_type == BTQ_T_F32 ? 8 : 4) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return BTQ_ERR_ALIGN;
  if (T == 0 || B == 0) return BTQ_OK;
  const btq::AttnPlan plan = plan_attention(P, T, Hq, Hk, D, B, max_pages, page_size, max_length);
  if (plan.workspace > 0 && !workspace) return BTQ_ERR_ARG;
  if (workspace_bytes < plan.workspace) return BTQ_ERR_WORKSPACE;
  const btq::HeadRows rows = {const_cast<void*>(q), BTQ_T_BF16, q_shard, q_pitch, q_head};
  const btq::AttnArgs a = {
      rows, btq::on16(rows),
      kv_args(P, T, Hk, D, seq_starts, lengths, B, page_table, max_pages, cache, pages, page_size),
      (int)Hq, (int)(Hq / Hk), (uint32_t)(((uint64_t(1) << 32) + Hq / Hk - 1) / (Hq / Hk)),
      scale * 1.4426950408889634f, causal != 0, (int)(window > kMaxPlaces ? 0 : window), out, out_type, lse, (float*)workspace, plan.splits,
      plan.begin};
  return hip_status(btq::launch_kv_attention(a, plan, (hipStream_t)stream));
}

const char* btq_status_str(int status) {
  switch (status) {
    case BTQ_OK: return "ok";
    case BTQ_ERR_ARG: return "invalid argument (null pointer, unknown option, or a factor out of range)";
    case BTQ_ERR_SHAPE: return "invalid shape (a size, a stride or the packed pitch out of range)";
    case BTQ_ERR_ALIGN: return "pointer not aligned to its element type";
    case BTQ_ERR_WORKSPACE: return "workspace too small";
    case BTQ_ERR_HIP: return "HIP call failed";
    case BTQ_ERR_SCRATCH:
      return "P*H too large for the no-alloc scratch (2*P*H*4 bytes must fit BTQ_NOALLOC_SCRATCH_BYTES)";
    default: return "unknown btq status";
  }
}

const char* btq_version(void) { return "0.5.0"; }

}  // extern "C"
