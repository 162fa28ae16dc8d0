// The calls that work row by row: btq_block_norm (the norms after one block and
// before the next, with the gate, the residual scale and the residual sum
// between them) and btq_quantize_rows (8-bit codes with a scale for each row).
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

// ---- general kernels: any size, stride and alignment ----
//
// One block a row. Each statistic is a pass over the row, recomputed from the
// inputs (which the caches hold after the first pass); the last pass writes.
// They cover rows too long for the register kernels. A thread adds H/256 terms
// one after another, up to 2^22 of them, so the sums are held in 64 bits: in 32
// the terms would be lost beside the sum. The passes wait for their loads, not
// for the additions (T=1024 H=65536, us: rms 1087 with either, layer 1466
// against 1457).
constexpr int kGenThreads = 256;

__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* lds) {
  for (int m = 32; m; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return max(max(lds[0], lds[1]), max(lds[2], lds[3]));
}

__global__ __launch_bounds__(kGenThreads) void norm_general_kernel(NormArgs a) {
  __shared__ double sums[4];
  __shared__ uint32_t maxima[4];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.H;
    const int64_t grow = t / a.gate_each * a.H;
    float mean_u = 0.0f, rstd_u = 1.0f, mean_r = 0.0f, rstd_r = 1.0f;

    // value(h) averaged over the row
    auto average = [&](auto value) {
      double s = 0.0;
      for (int64_t h = threadIdx.x; h < a.H; h += kGenThreads) s += value(h);
      return (float)(block_sum(s, sums) / (double)a.H);
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
      if (a.post == kLayer) mean_u = average(y);
      const float var = average([&](int64_t h) {
        const float d = y(h) - mean_u;
        return d * d;
      });
      rstd_u = 1.0f / sqrtf(var + a.post_eps);
    }
    if (a.pre != kNone && a.n) {
      if (a.pre == kLayer) mean_r = average(r);
      const float var = average([&](int64_t h) {
        const float d = r(h) - mean_r;
        return d * d;
      });
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
      rs = row_scale(block_max(m, maxima));
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

__global__ __launch_bounds__(kGenThreads) void rows_general_kernel(
    const void* __restrict__ x, int x_type, int64_t x_shard, int64_t x_pitch, int64_t rows,
    int64_t T, int64_t K, int8_t* __restrict__ q, int64_t q_pitch, float* __restrict__ scale) {
  __shared__ uint32_t maxima[4];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t base = row / T * x_shard + row % T * x_pitch;
    uint32_t m = 0;
    for (int64_t k = threadIdx.x; k < K; k += kGenThreads)
      m = max(m, __float_as_uint(load_value(x, x_type, base + k)) & 0x7fffffffu);
    const RowScale rs = row_scale(block_max(m, maxima));
    if (threadIdx.x == 0) scale[row] = rs.scale;
    for (int64_t k = threadIdx.x; k < K; k += kGenThreads)
      q[row * q_pitch + k] = (int8_t)code_bits(load_value(x, x_type, base + k), rs.mul);
  }
}

// ---- register kernels: a row stays in registers from its load to its store ----
//
// G lanes share a row, and each holds E = 8*NV of its elements. The row is
// read once and written once; each statistic is a sum over registers, six lane
// moves and (G > 64) one LDS exchange. A layer norm takes its variance from
// the deviations in a second sum, so a large mean costs no precision.
// Bound by HBM: the norm at T=16384 H=8192 (fp32 y, bf16 residual and n, 1.34 GB)
// takes 228 us, 5.9 TB/s; at T=2048 H=4096 16 us; codes of 32768 x 8192 bf16
// 141 us, 5.7 TB/s. One row alone takes 4.5 us, most of it the launch and the
// two sums' latency. Row lengths choose G: a row's lanes hold at most 32
// elements each (16 would halve the loads in flight, 64 spill), and more than 64
// lanes pay an LDS exchange.
// A lane takes runs of 8 elements. Every access goes through a buffer
// descriptor over the row, which is checked dword by dword: what lies past the
// row loads as 0 and is not stored. That needs rows on 4 bytes (kAligned), not
// on the 16 of the vectors. Else (bf16 rows of odd H, codes of H not a multiple
// of 4) bf16 loads read the dwords the row lies in, shift by its odd half and
// clear what belongs to the next row (never past the dword of the row's last
// element), and stores go by address, at any byte.
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// A row of `n` elements of `size` bytes.
template <bool kAligned>
struct Row {
  char* p;
  uint32_t skip;   // bytes of the first dword before the row
  rsrc_t r;
  __device__ __forceinline__ Row(const void* base, int64_t first, int n, int size) {
    p = (char*)base + first * size;
    skip = kAligned ? 0 : (uint32_t)(uintptr_t)p & 3;
    r = make_rsrc(p - skip, kAligned ? (uint32_t)(n * size) : (skip + n * size + 3) & ~3u);
  }
};

template <int G, int NV, bool kAligned>
struct RowMap {
  using R = Row<kAligned>;
  static constexpr int E = 8 * NV;
  int i;   // lane of the row's group
  int H;
  __device__ __forceinline__ int at(int v, int j) const { return (v * G + i) * 8 + j; }
  // raw words of 8 elements: 8 for fp32 (always on 4 bytes), 4 for bf16
  template <int kType>
  __device__ __forceinline__ void load(const R& r, int v, uint32_t (&w)[8]) const {
    constexpr int kWords = kType == kF32 ? 8 : 4;
    const int h = at(v, 0);
#pragma unroll
    for (int q = 0; q < kWords / 4; ++q) {
      const v4u a =
          __builtin_amdgcn_raw_buffer_load_b128(r.r, (uint32_t)(h * kWords / 2 + 16 * q), 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * q + j] = a[j];
    }
    if constexpr (!kAligned && kType == kBf16) {
      w[4] = __builtin_amdgcn_raw_buffer_load_b32(r.r, (uint32_t)(h * 2 + 16), 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = __builtin_amdgcn_alignbyte(w[j + 1], w[j], r.skip);
        if (h + 2 * j + 1 >= H) w[j] &= h + 2 * j >= H ? 0u : 0xffffu;
      }
    }
  }
  template <int kType>
  static __device__ __forceinline__ float value(const uint32_t (&w)[8], int j) {
    if constexpr (kType == kF32) return __uint_as_float(w[j]);
    return j & 1 ? __uint_as_float(w[j / 2] & 0xffff0000u) : __uint_as_float(w[j / 2] << 16);
  }
  // 8 elements of kSize bytes, packed in w. The streaming hint leaves the caches
  // to what is read (norm T=16384 H=8192: 255 -> 238 us, T=512: 11.4 -> 9.8);
  // on the loads it costs where the data is in the cache.
  template <int kSize>
  __device__ __forceinline__ void put(const R& r, int v, const uint32_t* w) const {
    const int h = at(v, 0);
    if constexpr (kAligned || kSize == 4) {
      const uint32_t off = (uint32_t)(h * kSize);
      if constexpr (kSize == 1) {
        __builtin_amdgcn_raw_buffer_store_b64(v2u{w[0], w[1]}, r.r, off, 0, 0);
      } else {
#pragma unroll
        for (int q = 0; q < kSize / 2; ++q)
          __builtin_amdgcn_raw_buffer_store_b128(
              v4u{w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]}, r.r, off + 16u * q, 0, kStream);
      }
    } else if (h + 8 <= H) {
      __builtin_memcpy(r.p + (int64_t)h * kSize, w, 8 * kSize);
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (h + j < H) {
          if constexpr (kSize == 2)
            ((uint16_t*)r.p)[h + j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
          if constexpr (kSize == 1) r.p[h + j] = (char)(w[j / 4] >> (8 * (j & 3)));
        }
    }
  }
  template <int kType>
  __device__ __forceinline__ void store(const R& r, int v, const float (&f)[8]) const {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < (kType == kF32 ? 8 : 4); ++j)
      w[j] = kType == kF32 ? __float_as_uint(f[j]) : f32_to_bf16x2(f[2 * j & 7], f[2 * j + 1 & 7]);
    put<kType == kF32 ? 4 : 2>(r, v, w);
  }
  __device__ __forceinline__ void store_codes(const R& r, int v, const float (&f)[8],
                                              float mul) const {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = code_bits(f[j], mul);
    const uint32_t w[2] = {c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                           c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24};
    put<1>(r, v, w);
  }
};

// One value a lane combined over the G lanes of a row; all lanes get it.
// `slot` is LDS that no other exchange in flight uses.
template <int G, typename F>
__device__ __forceinline__ uint32_t row_combine(uint32_t x, uint32_t* slot, F f) {
  x = wave_combine(x, f);
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = x;
    lds_barrier();
    x = slot[0];
#pragma unroll
    for (int w = 1; w < G / 64; ++w) x = f(x, slot[w]);
  }
  return x;
}
template <int G>
__device__ __forceinline__ float row_sum(float x, uint32_t* slot) {
  return __uint_as_float(row_combine<G>(__float_as_uint(x), slot, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ uint32_t row_max(uint32_t x, uint32_t* slot) {
  return row_combine<G>(x, slot, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// Statistics of the row in v, which is 0 past H: its mean (layer) and
// 1/sqrt(var + eps).
template <int G, int NV, bool kAligned>
__device__ __forceinline__ void row_stats(const RowMap<G, NV, kAligned>& m, const float (&v)[8 * NV],
                                          int H, bool layer, float eps, uint32_t* slot,
                                          float* mean, float* rstd) {
  const float inv_h = 1.0f / (float)H;
  float s = 0.0f;
  *mean = 0.0f;
  if (layer) {
#pragma unroll
    for (int e = 0; e < 8 * NV; ++e) s += v[e];
    *mean = row_sum<G>(s, slot) * inv_h;
    s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8 * NV; ++e) {
      const float d = m.at(e / 8, e % 8) < H ? v[e] - *mean : 0.0f;
      s = __builtin_fmaf(d, d, s);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8 * NV; ++e) s = __builtin_fmaf(v[e], v[e], s);
  }
  *rstd = 1.0f / sqrtf(row_sum<G>(s, slot + 16) * inv_h + eps);
}

// f = norm of 8 elements of the row. kAhead: their weights are in w already.
// kClear: what was 0 past H stays 0, for the sums of a norm that follows.
// There -mean is left of a deviation, and a weight that loads as 0 does not
// clear it: there may be none, and mean*rstd may be Inf. (Clearing the deviations
// in row_stats instead keeps a second copy of the row: 139 registers against
// 98, T=4096 H=5000 41.5 against 37 us.)
template <bool kAhead, bool kClear, int G, int NV, bool kAligned>
__device__ __forceinline__ void row_norm(const RowMap<G, NV, kAligned>& m, int v, float (&f)[8],
                                         float mean, float rstd, const float* weight,
                                         const uint32_t (&ahead)[8], const float* bias) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (f[j] - (kClear && m.at(v, j) >= m.H ? 0.0f : mean)) * rstd;
  if (weight) {
    if constexpr (!kAhead) m.template load<kF32>(Row<kAligned>(weight, 0, m.H, 4), v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= __uint_as_float(kAhead ? ahead[j] : w[j]);
  }
  if (bias) {
    m.template load<kF32>(Row<kAligned>(bias, 0, m.H, 4), v, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += __uint_as_float(w[j]);
  }
}

template <int G, int NV, bool kAligned, int kY, int kR>
__global__ __launch_bounds__(G == 64 ? 256 : G) void norm_row_kernel(NormArgs a) {
  constexpr int E = 8 * NV;
  constexpr int kRows = G == 64 ? 4 : 1;   // rows of a block
  // 5 exchanges a row, in two sets: a wave may enter the next row's while
  // another still reads this one's, but never the one after that
  __shared__ uint32_t lds[2][5 * 16];
  RowMap<G, NV, kAligned> m;
  m.i = threadIdx.x % G;
  const int H = m.H = (int)a.H;
  int set = 0;
  const int sub = __builtin_amdgcn_readfirstlane((int)threadIdx.x / G);
  for (int64_t t = (int64_t)blockIdx.x * kRows + sub; t < a.T;
       t += (int64_t)gridDim.x * kRows, set ^= 1) {
    uint32_t* slot = lds[set];
    const int64_t row = t * H;
    constexpr int ysz = kY == kF32 ? 4 : 2, rsz = kR == kF32 ? 4 : 2;
    const Row<kAligned> rr(a.residual, row, H, rsz);
    float u[E];
    uint32_t res[NV][8];
    // The kernel for few rows loads the weights and the gate with them: nothing
    // is left to wait for after the sums (T=1 H=8192: 4.6 -> 4.2 us). With many
    // rows the registers do more as further waves.
    constexpr bool kAhead = G == 1024 && NV == 1;
    uint32_t pw_ahead[8], nw_ahead[8], gw_ahead[8];
    const Row<kAligned> rg(a.gate, a.gate ? t / a.gate_each * H : 0, H,
                           a.gate_type == kF32 ? 4 : 2);
    if (a.y) {
      const Row<kAligned> ry(a.y, row, H, ysz);
      uint32_t yw[NV][8];
#pragma unroll
      for (int v = 0; v < NV; ++v) m.template load<kY>(ry, v, yw[v]);
#pragma unroll
      for (int v = 0; v < NV; ++v) m.template load<kR>(rr, v, res[v]);
      if constexpr (kAhead) {
        if (a.post_weight)
          m.template load<kF32>(Row<kAligned>(a.post_weight, 0, H, 4), 0, pw_ahead);
        if (a.gate && a.gate_type == kF32) m.template load<kF32>(rg, 0, gw_ahead);
        if (a.gate && a.gate_type == kBf16) m.template load<kBf16>(rg, 0, gw_ahead);
        if (a.pre_weight)
          m.template load<kF32>(Row<kAligned>(a.pre_weight, 0, H, 4), 0, nw_ahead);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = m.template value<kY>(yw[e / 8], e % 8);
      float mean = 0.0f, rstd = 1.0f;
      if (a.post != kNone)
        row_stats(m, u, H, a.post == kLayer, a.post_eps, slot, &mean, &rstd);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = u[v * 8 + j];
        if (a.post != kNone)
          row_norm<kAhead, true>(m, v, f, mean, rstd, a.post_weight, pw_ahead, a.post_bias);
        if (a.gate) {
          uint32_t w[8];
          if (a.gate_type == kF32) {
            if (!kAhead) m.template load<kF32>(rg, v, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= m.template value<kF32>(kAhead ? gw_ahead : w, j);
          } else {
            if (!kAhead) m.template load<kBf16>(rg, v, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= m.template value<kBf16>(kAhead ? gw_ahead : w, j);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[v * 8 + j] = m.template value<kR>(res[v], j) + a.alpha * f[j];
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) m.template load<kR>(rr, v, res[v]);
      if (kAhead && a.pre_weight)
        m.template load<kF32>(Row<kAligned>(a.pre_weight, 0, H, 4), 0, nw_ahead);
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = m.template value<kR>(res[e / 8], e % 8);
    }
    if (a.residual_out) {
      const Row<kAligned> ro(a.residual_out, row, H, rsz);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = u[v * 8 + j];
        m.template store<kR>(ro, v, f);
      }
    }
    if (!a.n) continue;
    float mean = 0.0f, rstd = 1.0f;
    if (a.pre != kNone) {
      row_stats(m, u, H, a.pre == kLayer, a.pre_eps, slot + 32, &mean, &rstd);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = u[v * 8 + j];
        row_norm<kAhead, false>(m, v, f, mean, rstd, a.pre_weight, nw_ahead, a.pre_bias);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[v * 8 + j] = f[j];
      }
    }
    const Row<kAligned> rn(a.n, row, H, a.n_type == kF32 ? 4 : a.n_type == kBf16 ? 2 : 1);
    RowScale rs = {1.0f, 0.0f};
    if (a.n_type == kInt8) {
      uint32_t big = 0;
#pragma unroll
      for (int e = 0; e < E; ++e)
        big = max(big, m.at(e / 8, e % 8) < H ? __float_as_uint(u[e]) & 0x7fffffffu : 0u);
      rs = row_scale(row_max<G>(big, slot + 64));
      if (m.i == 0) a.n_scale[t] = rs.scale;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = u[v * 8 + j];
      if (a.n_type == kInt8)
        m.store_codes(rn, v, f, rs.mul);
      else if (a.n_type == kBf16)
        m.template store<kBf16>(rn, v, f);
      else
        m.template store<kF32>(rn, v, f);
    }
  }
}

// 8-bit codes of a row: the largest |x| from the bits, then the codes.
template <int G, int NV, bool kAligned, int kX>
__global__ __launch_bounds__(G == 64 ? 256 : G) void rows_code_kernel(
    const void* __restrict__ x, int64_t x_shard, int64_t x_pitch, uint32_t rows, uint32_t T, int K,
    int8_t* __restrict__ q, int64_t q_pitch, float* __restrict__ scale) {
  constexpr uint32_t kRows = G == 64 ? 4 : 1;
  constexpr int sz = kX == kF32 ? 4 : 2;
  __shared__ uint32_t lds[2][16];   // two rows' exchanges, as in norm_row_kernel
  RowMap<G, NV, kAligned> m;
  m.i = threadIdx.x % G;
  m.H = K;
  int set = 0;
  const uint32_t sub = (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x / G);
  for (uint32_t row = blockIdx.x * kRows + sub; row < rows; row += gridDim.x * kRows, set ^= 1) {
    const int64_t base = (int64_t)(row / T) * x_shard + (int64_t)(row % T) * x_pitch;
    const Row<kAligned> rx(x, base, K, sz);
    uint32_t w[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) m.template load<kX>(rx, v, w[v]);
    uint32_t big = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        big = max(big, __float_as_uint(m.template value<kX>(w[v], j)) & 0x7fffffffu);
    const RowScale rs = row_scale(row_max<G>(big, lds[set]));
    if (m.i == 0) scale[row] = rs.scale;
    const Row<kAligned> rq(q, row * q_pitch, K, 1);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = m.template value<kX>(w[v], j);
      m.store_codes(rq, v, f, rs.mul);
    }
  }
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;
// The longest rows that stay in registers: 32 elements a lane of 1024.
constexpr int64_t kMaxRow = 32768;

struct CodeArgs {
  const void* x;
  int64_t x_shard, x_pitch, P, T, K;
  int8_t* q;
  int64_t q_pitch;
  float* scale;
};

template <int G, int NV, bool kAligned, int kX>
hipError_t launch_codes(const CodeArgs& c, hipStream_t s) {
  constexpr int per = G == 64 ? 4 : 1;
  const int64_t rows = c.P * c.T, blocks = (rows + per - 1) / per;
  rows_code_kernel<G, NV, kAligned, kX>
      <<<dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), G == 64 ? 256 : G, 0, s>>>(
          c.x, c.x_shard, c.x_pitch, (uint32_t)rows, (uint32_t)c.T, (int)c.K, c.q, c.q_pitch,
          c.scale);
  return hipGetLastError();
}

template <bool kAligned, int kX>
hipError_t launch_codes_sized(const CodeArgs& c, hipStream_t s) {
  if (c.K <= 512) return launch_codes<64, 1, kAligned, kX>(c, s);
  if (c.K <= 1024) return launch_codes<64, 2, kAligned, kX>(c, s);
  if (c.K <= 2048) return launch_codes<256, 1, kAligned, kX>(c, s);
  if (c.K <= 4096) return launch_codes<256, 2, kAligned, kX>(c, s);
  if (c.K <= 8192) return launch_codes<256, 4, kAligned, kX>(c, s);
  if (c.K <= 16384) return launch_codes<1024, 2, kAligned, kX>(c, s);
  return launch_codes<1024, 4, kAligned, kX>(c, s);
}

template <int G, int NV, bool kAligned, int kY, int kR>
hipError_t launch_rows(const NormArgs& a, hipStream_t s) {
  constexpr int rows = G == 64 ? 4 : 1;
  const int64_t blocks = (a.T + rows - 1) / rows;
  norm_row_kernel<G, NV, kAligned, kY, kR>
      <<<dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), G == 64 ? 256 : G, 0, s>>>(a);
  return hipGetLastError();
}

template <int G, int NV, bool kAligned>
hipError_t launch_types(const NormArgs& a, hipStream_t s) {
  if (a.y_type == kF32)
    return a.r_type == kF32 ? launch_rows<G, NV, kAligned, kF32, kF32>(a, s)
                            : launch_rows<G, NV, kAligned, kF32, kBf16>(a, s);
  return a.r_type == kF32 ? launch_rows<G, NV, kAligned, kBf16, kF32>(a, s)
                          : launch_rows<G, NV, kAligned, kBf16, kBf16>(a, s);
}

template <bool kAligned>
hipError_t launch_sized(const NormArgs& a, hipStream_t s) {
  const int64_t H = a.H;
  if (H <= 512) return launch_types<64, 1, kAligned>(a, s);
  if (H <= 1024) return launch_types<64, 2, kAligned>(a, s);
  if (H <= 2048) return launch_types<256, 1, kAligned>(a, s);
  if (H <= 4096) return launch_types<256, 2, kAligned>(a, s);
  // few rows leave most of the chip idle, so a row takes more lanes (H=8192:
  // T=64 5.1 against 6.3 us, T=256 7.4 against 8.7, T=1024 24.2 against 17.8)
  if (H <= 8192 && a.T > 256) return launch_types<256, 4, kAligned>(a, s);
  if (H <= 8192) return launch_types<1024, 1, kAligned>(a, s);
  if constexpr (kAligned) {
    if (H > 16384) return launch_types<1024, 4, kAligned>(a, s);
  }
  return launch_types<1024, 2, kAligned>(a, s);
}

// Rows of `pitch` elements start on 4 bytes.
bool on4(const void* p, int64_t pitch, int type) {
  const int64_t size = type == kF32 ? 4 : type == kBf16 ? 2 : 1;
  return ((uintptr_t)p & 3) == 0 && pitch * size % 4 == 0;
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  if (a.H <= kMaxRow) {
    // (fp32 tensors are on 4 bytes)
    const bool aligned = on4(a.y, a.H, a.y_type) && on4(a.residual, a.H, a.r_type) &&
                         on4(a.gate, a.gate ? a.H : 0, a.gate_type) &&
                         on4(a.residual_out, a.H, a.r_type) && on4(a.n, a.n ? a.H : 0, a.n_type);
    if (aligned) return launch_sized<true>(a, s);
    if (a.H <= kMaxRow / 2) return launch_sized<false>(a, s);
  }
  norm_general_kernel<<<dim3((unsigned)(a.T < kMaxBlocks ? a.T : kMaxBlocks)), kGenThreads, 0,
                        s>>>(a);
  return hipGetLastError();
}

hipError_t launch_quantize_rows(const void* x, int x_type, int64_t x_shard, int64_t x_pitch,
                                int64_t P, int64_t T, int64_t K, int8_t* q, int64_t q_pitch,
                                float* scale, hipStream_t s) {
  const int64_t rows = P * T;
  if (K <= kMaxRow && rows < (int64_t(1) << 31)) {
    const CodeArgs c = {x, x_shard, x_pitch, P, T, K, q, q_pitch, scale};
    if (on4(x, x_shard, x_type) && on4(x, x_pitch, x_type) && (x_type == kF32 || K % 2 == 0) &&
        on4(q, q_pitch, kInt8) && K % 4 == 0)
      return x_type == kF32 ? launch_codes_sized<true, kF32>(c, s)
                            : launch_codes_sized<true, kBf16>(c, s);
    return x_type == kF32 ? launch_codes_sized<false, kF32>(c, s)
                          : launch_codes_sized<false, kBf16>(c, s);
  }
  rows_general_kernel<<<dim3((unsigned)(rows < kMaxBlocks ? rows : kMaxBlocks)), kGenThreads, 0,
                        s>>>(x, x_type, x_shard, x_pitch, rows, T, K, q, q_pitch, scale);
  return hipGetLastError();
}

}  // namespace btq
