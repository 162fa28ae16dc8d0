// btq_head_norm_rope: the norm of each query and key head over its features, and
// the rotation by its token's position, in one pass.
//
//   y = turn((x - mean) / sqrt(mean((x - mean)^2) + eps) * w), mean only for layer.
// Bound by bytes: x is read and y written once, weights and the tables' rows come from
// L2. A head's features stay in its lanes' registers between the sums and the store, so
// the sums cost 3 lane exchanges at D = 128. P=4 T=8192 18 heads D=128 bf16: 57 us, 302 MB
// at 5.3 TB/s, a large copy's rate. One token of 8 + 1 heads: 4.2 us in a graph, 2.7 of
// them the kernel.
#include "common.hpp"

namespace btq {
namespace {

constexpr int kNone = 0, kLayer = 2;   // btq_norm
constexpr int kHalf = 0;               // btq_rope

__device__ __forceinline__ float head_value(const void* p, int type, int64_t i) {
  return type == kBf16 ? bf16_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}
__device__ __forceinline__ void put_head_value(void* p, int type, int64_t i, float v) {
  if (type == kBf16)
    ((uint16_t*)p)[i] = (uint16_t)f32_to_bf16(v);
  else
    ((float*)p)[i] = v;
}

__device__ __forceinline__ const float* head_weight(const HeadArgs& a, int64_t p, int h) {
  if (h < a.Hq) return a.q_weight ? a.q_weight + p * a.qw_shard + h * a.qw_head : nullptr;
  return a.k_weight ? a.k_weight + p * a.kw_shard + (h - a.Hq) * a.kw_head : nullptr;
}

// ---- general kernel: any size, stride and alignment; a wave a head, which reads it
// again for each sum (from L1) ----
__device__ __forceinline__ float wave_sum(float x) {
  return __uint_as_float(wave_combine(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__global__ __launch_bounds__(256) void head_general_kernel(HeadArgs a, int64_t items) {
  const int lane = threadIdx.x & 63;
  const int H = a.Hq + a.Hk;
  for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < items;
       item += (int64_t)gridDim.x * 4) {
    const int h = (int)(item % H);
    const int64_t t = item / H % a.T, p = item / H / a.T;
    const int64_t xb = p * a.x.shard + t * a.x.pitch + h * a.x.head;
    const int64_t yb = p * a.y.shard + t * a.y.pitch + h * a.y.head;
    const float* w = head_weight(a, p, h);
    float mean = 0.0f, rstd = 1.0f;
    auto x = [&](int i) { return head_value(a.x.p, a.x.type, xb + i); };
    if (a.norm != kNone) {
      if (a.norm == kLayer) {
        float s = 0.0f;
        for (int i = lane; i < a.D; i += 64) s += x(i);
        mean = wave_sum(s) / (float)a.D;
      }
      float s = 0.0f;
      for (int i = lane; i < a.D; i += 64) {
        const float d = x(i) - mean;
        s = __builtin_fmaf(d, d, s);
      }
      rstd = 1.0f / sqrtf(wave_sum(s) / (float)a.D + a.eps);
    }
    auto normed = [&](int i) {
      float v = x(i);
      if (a.norm != kNone) v = (v - mean) * rstd;
      return w ? v * w[i] : v;
    };
    // y may be x: a lane reads both features of a pair before it writes them,
    // and the sums above have read the whole head
    const int dim = a.rope.cos ? a.rope.dim : 0, half = dim / 2;
    const int pos = dim ? a.positions[t] : 0;
    for (int j = lane; j < half; j += 64) {
      const int i0 = a.rope.style == kHalf ? j : 2 * j, i1 = a.rope.style == kHalf ? j + half : 2 * j + 1;
      float c = __uint_as_float(0x7fc00000u), s = c;
      if (in_table(a.rope, pos)) {
        c = a.rope.cos[(int64_t)pos * half + j];
        s = a.rope.sin[(int64_t)pos * half + j];
      }
      const float u = normed(i0), v = normed(i1);
      put_head_value(a.y.p, a.y.type, yb + i0, u * c - v * s);
      put_head_value(a.y.p, a.y.type, yb + i1, v * c + u * s);
    }
    for (int i = dim + lane; i < a.D; i += 64)
      put_head_value(a.y.p, a.y.type, yb + i, normed(i));
  }
}

// ---- vector kernel: L lanes a head, 16 features a lane, in two runs of 8 ----
//
// The runs are those whose features turn into each other (8*i and dim/2 + 8*i
// where halves pair, neighbours else), so a pair never leaves its lane, and both
// styles read the same 8 entries of a token's cos and sin.
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

template <int kType>
__device__ __forceinline__ void load8(const void* base, int64_t first, float (&f)[8]) {
  if constexpr (kType == kF32) {
    const v4u* p = (const v4u*)((const float*)base + first);
    const v4u a = p[0], b = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(a[j]), f[4 + j] = __uint_as_float(b[j]);
  } else {
    const v4u a = *(const v4u*)((const uint16_t*)base + first);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(a[j] << 16);
      f[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
  }
}
template <int kType>
__device__ __forceinline__ void store8(void* base, int64_t first, const float (&f)[8]) {
  if constexpr (kType == kF32) {
    v4u* p = (v4u*)((float*)base + first);
    p[0] = v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    p[1] = v4u{__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])};
  } else {
    *(v4u*)((uint16_t*)base + first) =
        v4u{f32_to_bf16x2(f[0], f[1]), f32_to_bf16x2(f[2], f[3]), f32_to_bf16x2(f[4], f[5]),
            f32_to_bf16x2(f[6], f[7])};
  }
}

// The sum over groups of L lanes, in each of them.
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  auto add = [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  };
  uint32_t x = __float_as_uint(v);
  if constexpr (L >= 2) x = add(x, dpp<0xb1>(x));
  if constexpr (L >= 4) x = add(x, dpp<0x4e>(x));
  if constexpr (L >= 8) x = add(x, dpp<0x141>(x));
  if constexpr (L >= 16) x = add(x, dpp<0x140>(x));
  if constexpr (L >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = add(s[0], s[1]);
  }
  if constexpr (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = add(s[0], s[1]);
  }
  return __uint_as_float(x);
}

template <int L, int kX, int kY>
__global__ __launch_bounds__(256) void head_vector_kernel(HeadArgs a, uint32_t items) {
  const int H = a.Hq + a.Hk;
  const uint32_t i = threadIdx.x % L;
  const uint32_t item = blockIdx.x * (256 / L) + threadIdx.x / L;
  const bool live = item < items && (int)i < a.D / 16;
  // idle lanes keep to the last head's first run; they take part in the sums as 0
  const uint32_t it = item < items ? item : items - 1;
  const uint32_t t = it / (uint32_t)H;
  const int h = (int)(it - t * (uint32_t)H);
  const int64_t p = blockIdx.y;
  const int dim = a.rope.cos ? a.rope.dim : 0;
  const bool turn = (int)(16 * i) < dim;
  const int run = live ? (int)i : 0;
  int f0 = 16 * run, f1 = f0 + 8;
  if (a.rope.style == kHalf && 16 * run < dim) f0 = 8 * run, f1 = dim / 2 + 8 * run;
  const int64_t xb = p * a.x.shard + (int64_t)t * a.x.pitch + h * a.x.head;
  float u[8], v[8], c[8], s[8];
  load8<kX>(a.x.p, xb + f0, u);
  load8<kX>(a.x.p, xb + f1, v);
  if (turn && live) {
    const int pos = a.positions[t];
    if (in_table(a.rope, pos)) {
      const int64_t at = (int64_t)pos * (dim / 2) + 8 * run;
      load8<kF32>(a.rope.cos, at, c);
      load8<kF32>(a.rope.sin, at, s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = s[j] = __uint_as_float(0x7fc00000u);
    }
  }
  const float* w = head_weight(a, p, h);
  if (a.norm != kNone) {
    const float inv = 1.0f / (float)a.D;
    float mean = 0.0f, q = 0.0f;
    if (a.norm == kLayer) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m += u[j] + v[j];
      mean = group_sum<L>(live ? m : 0.0f) * inv;
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] -= mean, v[j] -= mean;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(u[j], u[j], __builtin_fmaf(v[j], v[j], q));
    const float rstd = 1.0f / sqrtf(group_sum<L>(live ? q : 0.0f) * inv + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] *= rstd, v[j] *= rstd;
  }
  if (!live) return;
  if (w) {
    float wu[8], wv[8];
    load8<kF32>(w, f0, wu);
    load8<kF32>(w, f1, wv);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] *= wu[j], v[j] *= wv[j];
  }
  if (turn) {
    if (a.rope.style == kHalf) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = u[j], y = v[j];
        u[j] = x * c[j] - y * s[j];
        v[j] = y * c[j] + x * s[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = u[2 * j], y = u[2 * j + 1], z = v[2 * j], q = v[2 * j + 1];
        u[2 * j] = x * c[j] - y * s[j];
        u[2 * j + 1] = y * c[j] + x * s[j];
        v[2 * j] = z * c[4 + j] - q * s[4 + j];
        v[2 * j + 1] = q * c[4 + j] + z * s[4 + j];
      }
    }
  }
  const int64_t yb = p * a.y.shard + (int64_t)t * a.y.pitch + h * a.y.head;
  store8<kY>(a.y.p, yb + f0, u);
  store8<kY>(a.y.p, yb + f1, v);
}

template <int L, int kX, int kY>
hipError_t launch_vector(const HeadArgs& a, hipStream_t s) {
  const int64_t items = a.T * (a.Hq + a.Hk), blocks = (items * L + 255) / 256;
  head_vector_kernel<L, kX, kY><<<dim3((unsigned)blocks, (unsigned)a.P), 256, 0, s>>>(
      a, (uint32_t)items);
  return hipGetLastError();
}

template <int L>
hipError_t launch_types(const HeadArgs& a, hipStream_t s) {
  if (a.x.type == kF32)
    return a.y.type == kF32 ? launch_vector<L, kF32, kF32>(a, s) : launch_vector<L, kF32, kBf16>(a, s);
  return a.y.type == kF32 ? launch_vector<L, kBf16, kF32>(a, s) : launch_vector<L, kBf16, kBf16>(a, s);
}

bool weight_on16(const float* w, int64_t shard, int64_t head) {
  return ((uintptr_t)w & 15) == 0 && shard % 4 == 0 && head % 4 == 0;
}

}  // namespace

hipError_t launch_head_norm_rope(const HeadArgs& a, hipStream_t s) {
  const int64_t items = a.T * (a.Hq + a.Hk);
  const int dim = a.rope.cos ? a.rope.dim : 0;
  if (a.D % 16 == 0 && a.D <= 1024 && dim % 16 == 0 && on16(a.x) && on16(a.y) &&
      weight_on16(a.q_weight, a.qw_shard, a.qw_head) &&
      weight_on16(a.k_weight, a.kw_shard, a.kw_head) && ((uintptr_t)a.rope.cos & 15) == 0 &&
      ((uintptr_t)a.rope.sin & 15) == 0 && items < (int64_t(1) << 25)) {   // (2^31 threads)
    if (a.D <= 32) return launch_types<2>(a, s);
    if (a.D <= 64) return launch_types<4>(a, s);
    if (a.D <= 128) return launch_types<8>(a, s);
    if (a.D <= 256) return launch_types<16>(a, s);
    return launch_types<64>(a, s);
  }
  const int64_t all = a.P * items, blocks = (all + 3) / 4;
  head_general_kernel<<<dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), 256, 0, s>>>(a, all);
  return hipGetLastError();
}

}  // namespace btq
