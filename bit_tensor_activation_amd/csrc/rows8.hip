// btq_quantize_rows: per-row 8-bit codes.
#include "common.hpp"

namespace btq {
namespace {

__device__ __forceinline__ float load_value(const void* p, int type, int64_t i) {
  return type == kBf16 ? bf16_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

// ---- general kernel: any size, stride and alignment; one block a row ----
constexpr int kGenThreads = 256;

__global__ __launch_bounds__(kGenThreads) void rows_general_kernel(
    const void* __restrict__ x, int x_type, int64_t x_shard, int64_t x_pitch, int64_t rows,
    int64_t T, int64_t K, int8_t* __restrict__ q, int64_t q_pitch, float* __restrict__ scale) {
  __shared__ uint32_t lds[4];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row / T * x_shard + row % T * x_pitch;
    uint32_t m = 0;
    for (int64_t k = threadIdx.x; k < K; k += kGenThreads)
      m = max(m, __float_as_uint(load_value(x, x_type, base + k)) & 0x7fffffffu);
    for (int o = 32; o; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
    __syncthreads();
    const RowScale rs = row_scale(max(max(lds[0], lds[1]), max(lds[2], lds[3])));
    if (threadIdx.x == 0) scale[row] = rs.scale;
    for (int64_t k = threadIdx.x; k < K; k += kGenThreads)
      q[row * q_pitch + k] = (int8_t)code_bits(load_value(x, x_type, base + k), rs.mul);
  }
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;

}  // namespace

hipError_t launch_quantize_rows(const void* x, int x_type, int64_t x_shard, int64_t x_pitch,
                                int64_t P, int64_t T, int64_t K, int8_t* q, int64_t q_pitch,
                                float* scale, hipStream_t s) {
  const int64_t rows = P * T;
  rows_general_kernel<<<dim3((unsigned)(rows < kMaxBlocks ? rows : kMaxBlocks)), kGenThreads, 0,
                        s>>>(x, x_type, x_shard, x_pitch, rows, T, K, q, q_pitch, scale);
  return hipGetLastError();
}

}  // namespace btq
