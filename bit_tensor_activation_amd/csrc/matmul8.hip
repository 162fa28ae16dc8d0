// btq_int8_matmul: products of 8-bit codes on the matrix cores, int32 sums,
// scaled by token and output channel.
//
// Every kernel feeds the weights as the matrix instruction's first operand
// and the activations as its second. The result then holds, in each lane, one
// token and runs of 4 consecutive output channels, which store as vectors.
// The order of k inside an instruction does not matter (integer sums are
// exact), as long as both operands take it alike.
#include "common.hpp"

namespace btq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// 16 bytes k..k+15 of a row of K, zero past its end. Any alignment; nothing
// past the row is read.
__device__ __forceinline__ v4i load_chunk(const int8_t* __restrict__ row, int64_t k, int64_t K) {
  v4i v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k + i < K) d[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
    v = v4i{(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
  }
  return v;
}

// y = sum * a_scale * w_scale (+ bias), each step one fp32 operation.
__device__ __forceinline__ float scaled(int sum, float sa, float sw, float b, bool has_bias) {
  const float v = (float)sum * sa * sw;
  return has_bias ? v + b : v;
}

// ---- general kernel: any size, stride and alignment ----
//
// 64 tokens x 64 channels a block, 4 waves of 32x32, 64 bytes of k a step
// through LDS (rows padded to 80 bytes).
constexpr int kGenTile = 64, kGenK = 64, kGenRow = 80;

__global__ __launch_bounds__(256) void matmul_general_kernel(MatmulArgs g, int64_t tiles_t,
                                                             int64_t tiles_n, int64_t tiles) {
  __shared__ __align__(16) int8_t la[kGenTile * kGenRow];
  __shared__ __align__(16) int8_t lw[kGenTile * kGenRow];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wt = (wave & 1) * 32, wn = (wave >> 1) * 32;
  const int lr = threadIdx.x >> 2, lk = (threadIdx.x & 3) * 16;   // this thread's chunk
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t p = tile / (tiles_t * tiles_n);
    const int64_t t0 = tile / tiles_n % tiles_t * kGenTile;
    const int64_t n0 = tile % tiles_n * kGenTile;
    const int8_t* arow = g.a + p * g.a_shard + min(t0 + lr, g.T - 1) * g.a_pitch;
    const int8_t* wrow = g.w + (p * g.N + min(n0 + lr, g.N - 1)) * g.K;
    v16i acc = {};
    for (int64_t k0 = 0; k0 < g.K; k0 += kGenK) {
      const v4i va = load_chunk(arow, k0 + lk, g.K), vw = load_chunk(wrow, k0 + lk, g.K);
      __syncthreads();
      *(v4i*)(la + lr * kGenRow + lk) = va;
      *(v4i*)(lw + lr * kGenRow + lk) = vw;
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kGenK; kk += 32) {
        const int off = kk + (lane >> 5) * 16;
        const v4i fa = *(const v4i*)(la + (wt + (lane & 31)) * kGenRow + off);
        const v4i fw = *(const v4i*)(lw + (wn + (lane & 31)) * kGenRow + off);
        acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw, fa, acc, 0, 0, 0);
      }
    }
    const int64_t t = t0 + wt + (lane & 31);
    if (t < g.T) {
      const float sa = g.a_scale[p * g.as_shard + t];
      const int64_t out = (p * g.T + t) * g.N;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int64_t n = n0 + wn + 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
        if (n < g.N) {
          const float v = scaled(acc[i], sa, g.w_scale[p * g.N + n],
                                 g.bias ? g.bias[p * g.N + n] : 0.0f, g.bias != nullptr);
          if (g.y_type == kBf16)
            ((uint16_t*)g.y)[out + n] = (uint16_t)f32_to_bf16(v);
          else
            ((float*)g.y)[out + n] = v;
        }
      }
    }
  }
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;

}  // namespace

hipError_t launch_int8_matmul(const MatmulArgs& a, hipStream_t s) {
  const int64_t tt = (a.T + kGenTile - 1) / kGenTile, tn = (a.N + kGenTile - 1) / kGenTile;
  const int64_t tiles = a.P * tt * tn;
  matmul_general_kernel<<<dim3((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks)), 256, 0, s>>>(
      a, tt, tn, tiles);
  return hipGetLastError();
}

}  // namespace btq
