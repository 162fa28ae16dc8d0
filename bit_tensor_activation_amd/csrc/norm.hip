// btq_block_norm: the norms after one block and before the next, with the
// gate, the residual scale and the residual sum between them.
#include "common.hpp"

namespace btq {
namespace {

constexpr int kNone = 0, kLayer = 2;   // btq_norm

__device__ __forceinline__ float load_value(const void* p, int type, int64_t i) {
  return type == kBf16 ? bf16_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

__device__ __forceinline__ void store_value(void* p, int type, int64_t i, float v) {
  if (type == kBf16)
    ((uint16_t*)p)[i] = (uint16_t)f32_to_bf16(v);
  else
    ((float*)p)[i] = v;
}

// ---- general kernel: any size and alignment ----
//
// One block a row. Each statistic is a pass over the row, recomputed from the
// inputs (which the caches hold after the first pass); the last pass writes.
// It covers rows too long for the register kernel.
constexpr int kGenThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* lds) {
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, float* lds) {
  for (int m = 32; m; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = __uint_as_float(v);
  __syncthreads();
  return max(max(__float_as_uint(lds[0]), __float_as_uint(lds[1])),
             max(__float_as_uint(lds[2]), __float_as_uint(lds[3])));
}

__global__ __launch_bounds__(kGenThreads) void norm_general_kernel(NormArgs a) {
  __shared__ float lds[4];
  const float inv_h = 1.0f / (float)a.H;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.H;
    const int64_t grow = t / a.gate_each * a.H;
    float mean_u = 0.0f, rstd_u = 1.0f, mean_r = 0.0f, rstd_r = 1.0f;

    // value(h) summed over the row
    auto sum = [&](auto value) {
      float s = 0.0f;
      for (int64_t h = threadIdx.x; h < a.H; h += kGenThreads) s += value(h);
      return block_sum(s, lds);
    };
    auto y = [&](int64_t h) { return load_value(a.y, a.y_type, row + h); };
    auto r = [&](int64_t h) {
      const float res = load_value(a.residual, a.r_type, row + h);
      if (!a.y) return res;
      float u = y(h);
      if (a.post != kNone) {
        u = (u - mean_u) * rstd_u;
        if (a.post_weight) u *= a.post_weight[h];
        if (a.post_bias) u += a.post_bias[h];
      }
      if (a.gate) u *= load_value(a.gate, a.gate_type, grow + h);
      return res + a.alpha * u;
    };
    if (a.post != kNone) {
      if (a.post == kLayer) mean_u = sum(y) * inv_h;
      const float var = sum([&](int64_t h) {
        const float d = y(h) - mean_u;
        return d * d;
      }) * inv_h;
      rstd_u = 1.0f / sqrtf(var + a.post_eps);
    }
    if (a.pre != kNone && a.n) {
      if (a.pre == kLayer) mean_r = sum(r) * inv_h;
      const float var = sum([&](int64_t h) {
        const float d = r(h) - mean_r;
        return d * d;
      }) * inv_h;
      rstd_r = 1.0f / sqrtf(var + a.pre_eps);
    }
    auto n = [&](int64_t h, float rv) {
      if (a.pre == kNone) return rv;
      float v = (rv - mean_r) * rstd_r;
      if (a.pre_weight) v *= a.pre_weight[h];
      if (a.pre_bias) v += a.pre_bias[h];
      return v;
    };
    RowScale rs = {1.0f, 0.0f};
    if (a.n && a.n_type == kInt8) {
      uint32_t m = 0;
      for (int64_t h = threadIdx.x; h < a.H; h += kGenThreads)
        m = max(m, __float_as_uint(n(h, r(h))) & 0x7fffffffu);
      rs = row_scale(block_max(m, lds));
      if (threadIdx.x == 0) a.n_scale[t] = rs.scale;
    }
    for (int64_t h = threadIdx.x; h < a.H; h += kGenThreads) {
      const float rv = r(h);
      if (a.n) {
        const float v = n(h, rv);
        if (a.n_type == kInt8)
          ((int8_t*)a.n)[row + h] = (int8_t)code_bits(v, rs.mul);
        else
          store_value(a.n, a.n_type, row + h, v);
      }
      if (a.residual_out) store_value(a.residual_out, a.r_type, row + h, rv);
    }
  }
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  norm_general_kernel<<<dim3((unsigned)(a.T < kMaxBlocks ? a.T : kMaxBlocks)), kGenThreads, 0,
                        s>>>(a);
  return hipGetLastError();
}

}  // namespace btq
