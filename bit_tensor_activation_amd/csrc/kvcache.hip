// btq_kv_append and btq_kv_gather: rows of new keys and values into the paged
// 4-bit cache, and what the cache holds back into rows.
//
//   scale = (hi - lo)/15 up to bf16,  z = rint(-lo/scale),  code = rint(x/scale) + z
// Bound by bytes, 4*D read and D + 8 written for a token of a head. A thread block takes
// the 32 tokens of a cache block, so that blocks which the call fills are written in whole
// lines and nothing else touches the bytes that two tokens share. P=8, 8 sequences of
// 2048 new tokens, D=128, rotated: 22 us, 67 MB read and 18 written at 3.8 TB/s (a block's
// conversion waits for its loads; only the CU's other blocks run meanwhile); gather of
// as much 16 us, 5.3 TB/s. 64 sequences of one new token: 5.9 and 3.1 us.
#include "common.hpp"

namespace btq {
namespace {

constexpr int kHalf = 0;   // btq_rope
constexpr int kThreads = 256;
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// The block (32 tokens of a head) that a thread block works on.
struct Place {
  int64_t at;      // its byte offset in the cache, -1: no page
  int64_t row;     // batch row of its token 0 (which may lie before the sequence's)
  int from, to;    // its tokens among the batch's rows
  int first;       // place of token 0 in its sequence
};
__device__ __forceinline__ bool find_place(const KvArgs& a, int64_t item, int64_t shard, int head,
                                           Place* o) {
  int64_t sub;
  SeqRange s;
  const int b = find_sequence(a, 1, 5, 2 * kBlockTokens, item, &sub, &s);
  if (b < 0) return false;
  const int block = (s.first() >> 5) + (int)sub;
  o->first = block * kBlockTokens;
  o->from = max(s.first() - o->first, 0);
  o->to = min(s.length - o->first, kBlockTokens);
  if (o->from >= o->to) return false;
  o->row = (int64_t)s.begin + o->first - s.first();
  o->at = kv_block(a, b, shard, head, block);
  return true;
}

template <bool kVector>
__device__ __forceinline__ void load_tile(const HeadRows& r, int64_t base, int D, const Place& at,
                                          float* tile, int pitch) {
  const int runs = D / 8;
  for (int i = threadIdx.x; i < kBlockTokens * runs; i += kThreads) {
    const int t = i / runs, f = (i - t * runs) * 8;
    if (t < at.from || t >= at.to) continue;
    const int64_t e = base + (at.row + t) * r.pitch + f;
    float v[8];
    if (r.type == kBf16) {
      uint32_t w[4];
      if constexpr (kVector) {
        const v4u x = *(const v4u*)((const uint16_t*)r.p + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = x[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = ((const uint16_t*)r.p)[e + 2 * j] |
                 (uint32_t)((const uint16_t*)r.p)[e + 2 * j + 1] << 16;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = ((const float*)r.p)[e + j];
    }
    float* o = tile + t * pitch + f;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v[j];
  }
}

// f combined over groups of 8 lanes.
template <typename F>
__device__ __forceinline__ uint32_t combine8(uint32_t x, F f) {
  x = f(x, dpp<0xb1>(x));
  x = f(x, dpp<0x4e>(x));
  return f(x, dpp<0x141>(x));
}

// Codes of E features a lane, 8 lanes a row; returns the row's word.
// The quotient x/scale is the correctly rounded one: q = x*r with r the rounded
// 1/scale, then one step of its residual (Markstein's theorem). A product with r
// alone would miss the ties that bf16 rows have (x and scale hold 8 bits each).
template <int E>
__device__ __forceinline__ uint32_t quantize(const float (&x)[E], uint32_t (&code)[E]) {
  float lo = 0.0f, hi = 0.0f;
  uint32_t big = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    big = max(big, __float_as_uint(x[e]) & 0x7fffffffu);
  }
  lo = __uint_as_float(combine8(__float_as_uint(lo), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
  }));
  hi = __uint_as_float(combine8(__float_as_uint(hi), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
  big = combine8(big, [](uint32_t a, uint32_t b) { return max(a, b); });
  const float range = hi - lo;
  // rounded up to bf16, so 15 steps span the range and no code is cut off
  uint32_t sb = (__float_as_uint(range / 15.0f) + 0xffffu) & 0xffff0000u;
  const bool bad = big >= 0x7f800000u || !(range < INFINITY);
  if (sb < 0x00800000u) sb = 0x3f800000u;   // below the normal numbers: scale 1, codes 0
  const float scale = __uint_as_float(sb), r = 1.0f / scale;
  auto steps = [&](float v) {
    const float q = v * r;
    return rintf(__builtin_fmaf(__builtin_fmaf(-q, scale, v), r, q));
  };
  const float z = fminf(steps(-lo), 15.0f);
#pragma unroll
  for (int e = 0; e < E; ++e)
    code[e] = bad ? 0u : (uint32_t)fminf(fmaxf(steps(x[e]) + z, 0.0f), 15.0f);
  return bad ? kNanWord : sb | (__float_as_uint(128.0f + z) >> 16);
}

// ---- the usual form: 8 lanes a token, its features in registers ----
//
// A lane holds two runs of W features of a key, those that turn into each other (W*i
// and dim/2 + W*i where halves pair, neighbours else), and 2*W neighbouring features of
// a value; where D is no multiple of 64 some of the 8 lanes are idle. Codes of values
// turn in LDS: a thread merges a dword of 4 features of each of 8 tokens into 4 rows of
// 8 tokens, 12 instructions for 32 codes. Takes rows and tables on 16 bytes, and a
// number of turned features that whole lanes have.
// P=8, 16384 tokens, half of them turned: D = 128 55 -> 22 us by the general kernel and here,
// 96 45 -> 20.
// (D = 192 takes 8 lanes of 24 features or 6 of 32: all of a head turned 31 against 42 us,
// 64 features of it, which only the second form takes, 41 and 98 by the general kernel.)
constexpr int head_run(int D) { return D % 64 == 0 ? D / 16 : D == 32 ? 4 : D == 96 ? 8 : 16; }
template <int W, int kType>
__device__ __forceinline__ void load_run(const void* base, int64_t first, float (&x)[W]) {
#pragma unroll
  for (int e = 0; e < W; e += 4) {
    if constexpr (kType == kF32) {
      const v4u w = *(const v4u*)((const float*)base + first + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[e + j] = __uint_as_float(w[j]);
    } else {
      const v2u w = *(const v2u*)((const uint16_t*)base + first + e);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[e + 2 * j] = __uint_as_float(w[j] << 16);
        x[e + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

template <int D, int W, int kType>
__global__ __launch_bounds__(kThreads) void kv_append_heads_kernel(HeadRows k, HeadRows v,
                                                                   RopeArgs rope, KvArgs a,
                                                                   uint32_t first_item) {
  constexpr int kLanes = D / (2 * W), kPitch = D / 4 + 1;
  __shared__ uint32_t codes[kBlockTokens * kPitch];
  const int64_t shard = blockIdx.y, item = first_item + blockIdx.z;
  const int head = blockIdx.x;
  Place at;
  if (!find_place(a, item, shard, head, &at)) return;
  const int t = threadIdx.x / 8, in_row = threadIdx.x % 8;
  const bool busy = kLanes == 8 || in_row < kLanes;
  const int sub = busy ? in_row : 0;                   // (idle lanes read what is there)
  const bool token = t >= at.from && t < at.to, mine = token && busy;
  const int64_t row = at.row + (token ? t : at.from);
  const bool turn = rope.cos && 2 * W * sub < rope.dim, halves = turn && rope.style == kHalf;
  const int f0 = halves ? W * sub : 2 * W * sub, f1 = halves ? rope.dim / 2 + f0 : f0 + W;
  float x[W], y[W], c[W], s[W], u[W], w[W];
  const int64_t kb = shard * k.shard + row * k.pitch + head * k.head;
  const int64_t vb = shard * v.shard + row * v.pitch + head * v.head + 2 * W * sub;
  load_run<W, kType>(k.p, kb + f0, x);
  load_run<W, kType>(k.p, kb + f1, y);
  const int64_t pos = at.first + (token ? t : at.from);
  // (the place of a row that is dropped may be negative: its loads come before that is known)
  const bool known = in_table(rope, pos);
  if (turn) {
    const int64_t e = (known ? pos : 0) * (rope.dim / 2) + W * sub;
    load_run<W, kF32>(rope.cos, e, c);
    load_run<W, kF32>(rope.sin, e, s);
  }
  load_run<W, kType>(v.p, vb, u);
  load_run<W, kType>(v.p, vb + W, w);
  if (at.at < 0) return;
  if (!busy) {
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = y[e] = u[e] = w[e] = 0.0f;
  }
  uint8_t* block = a.cache + at.at;
  // this thread's part of the values' block: features 4*fq .. of tokens 8*group ..
  const int fq = threadIdx.x / 4, group = threadIdx.x % 4;
  uint32_t mask = 0, old[(D + 255) / 256][4];
  {
    const int from = max(at.from - 8 * group, 0), to = min(at.to - 8 * group, 8);
    if (from < to) mask = (to == 8 ? 0xffffffffu : (1u << (4 * to)) - 1) & (0xffffffffu << (4 * from));
  }
  if (mask && ~mask) {
#pragma unroll
    for (int i = 0; i < (D + 255) / 256; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * (fq + 64 * i) < D)
          old[i][r] = *(const uint32_t*)(block + 16 * D + (4 * (fq + 64 * i) + r) * 16 + group * 4);
  }

  if (turn && busy) {
    if (!known) {
#pragma unroll
      for (int e = 0; e < W; ++e) c[e] = s[e] = __uint_as_float(0x7fc00000u);
    }
    if (halves) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float p = x[e], q = y[e];
        x[e] = p * c[e] - q * s[e];
        y[e] = q * c[e] + p * s[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const float p = x[e], q = x[e + 1], m = y[e], n = y[e + 1];
        x[e] = p * c[e / 2] - q * s[e / 2];
        x[e + 1] = q * c[e / 2] + p * s[e / 2];
        y[e] = m * c[(W + e) / 2] - n * s[(W + e) / 2];
        y[e + 1] = n * c[(W + e) / 2] + m * s[(W + e) / 2];
      }
    }
  }
  float z[2 * W];
  uint32_t code[2 * W];
#pragma unroll
  for (int e = 0; e < W; ++e) z[e] = x[e], z[W + e] = y[e];
  const uint32_t kw = quantize<2 * W>(z, code);
  if (mine) {
    uint8_t* out = block + t * (D / 2);
#pragma unroll
    for (int e = 0; e < 2 * W; e += 4)
      *(uint16_t*)(out + (e < W ? f0 + e : f1 + e - W) / 2) =
          (uint16_t)(code[e] | code[e + 1] << 4 | code[e + 2] << 8 | code[e + 3] << 12);
    if (sub == 0) *(uint32_t*)(block + 32 * D + t * 4) = kw;
  }
#pragma unroll
  for (int e = 0; e < W; ++e) z[e] = u[e], z[W + e] = w[e];
  const uint32_t vw = quantize<2 * W>(z, code);
  if (mine && sub == 0) *(uint32_t*)(block + 32 * D + 128 + t * 4) = vw;
  if (busy) {
#pragma unroll
    for (int e = 0; e < 2 * W; e += 4)
      codes[t * kPitch + (2 * W * sub + e) / 4] =
          code[e] | code[e + 1] << 8 | code[e + 2] << 16 | code[e + 3] << 24;
  }
  lds_barrier();
  if (!mask) return;
#pragma unroll
  for (int i = 0; i < (D + 255) / 256; ++i) {
    const int q = fq + 64 * i;
    if (4 * q >= D) break;
    uint32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      p[j] = codes[(8 * group + 2 * j) * kPitch + q] | codes[(8 * group + 2 * j + 1) * kPitch + q] << 4;
    const uint32_t a0 = __builtin_amdgcn_perm(p[1], p[0], 0x05010400u);
    const uint32_t a1 = __builtin_amdgcn_perm(p[1], p[0], 0x07030602u);
    const uint32_t b0 = __builtin_amdgcn_perm(p[3], p[2], 0x05010400u);
    const uint32_t b1 = __builtin_amdgcn_perm(p[3], p[2], 0x07030602u);
    const uint32_t rows[4] = {
        __builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
        __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u)};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *(uint32_t*)(block + 16 * D + (4 * q + r) * 16 + group * 4) =
          ~mask ? (rows[r] & mask) | (old[i][r] & ~mask) : rows[r];
  }
}

template <int D, bool kVector>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(HeadRows k, HeadRows v, RopeArgs rope,
                                                             KvArgs a,
                                                             uint32_t first_item) {
  constexpr int E = D / 8, kPitch = D + 4;
  __shared__ float tile[2][kBlockTokens * kPitch];
  __shared__ uint32_t codes[kBlockTokens * (E * 2 + 1)];   // a row of D bytes and 4 more
  const int64_t shard = blockIdx.y, item = first_item + blockIdx.z;
  const int head = blockIdx.x;
  Place at;
  if (!find_place(a, item, shard, head, &at) || at.at < 0) return;
  load_tile<kVector>(k, shard * k.shard + head * k.head, D, at, tile[0], kPitch);
  load_tile<kVector>(v, shard * v.shard + head * v.head, D, at, tile[1], kPitch);
  __syncthreads();

  uint8_t* block = a.cache + at.at;
  const int t = threadIdx.x / 8, sub = threadIdx.x % 8, f0 = sub * E;
  const bool mine = t >= at.from && t < at.to;
  uint32_t code[E];
  float x[E];
  {
    const float* row = tile[0] + t * kPitch;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = row[f0 + e];
    if (rope.cos) {
      const int half = rope.dim / 2;
      const int64_t pos = at.first + t;
      const bool known = in_table(rope, pos);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = f0 + e;
        if (i < rope.dim && mine) {
          const bool second = rope.style == kHalf ? i >= half : e & 1;
          const int j = rope.style == kHalf ? (second ? i - half : i) : i / 2;
          const float other = row[rope.style == kHalf ? (second ? i - half : i + half) : i ^ 1];
          float c = __uint_as_float(0x7fc00000u), s = c;
          if (known) c = rope.cos[pos * half + j], s = rope.sin[pos * half + j];
          x[e] = second ? x[e] * c + other * s : x[e] * c - other * s;
        }
      }
    }
    const uint32_t word = quantize<E>(x, code);
    if (mine) {
      uint8_t* out = block + t * (D / 2) + sub * (E / 2);
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *(uint16_t*)(out + e / 2) = (uint16_t)(code[e] | code[e + 1] << 4 | code[e + 2] << 8 |
                                               code[e + 3] << 12);
      if (sub == 0) *(uint32_t*)(block + 32 * D + t * 4) = word;
    }
  }
  {
    const float* row = tile[1] + t * kPitch;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = row[f0 + e];
    const uint32_t word = quantize<E>(x, code);
    if (mine && sub == 0) *(uint32_t*)(block + 32 * D + 128 + t * 4) = word;
    uint32_t* out = codes + t * (E * 2 + 1) + sub * (E / 4);
#pragma unroll
    for (int e = 0; e < E; e += 4)
      out[e / 4] = code[e] | code[e + 1] << 8 | code[e + 2] << 16 | code[e + 3] << 24;
  }
  __syncthreads();
  // 16 tokens of a feature a thread: 8 bytes, in which only this batch's tokens change
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    const int d = i >> 1, first = (i & 1) * 16;
    uint64_t bits = 0, mask = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int token = first + j;
      const uint64_t c = ((const uint8_t*)(codes + token * (E * 2 + 1)))[d];
      if (token >= at.from && token < at.to) {
        bits |= c << (4 * j);
        mask |= (uint64_t)15 << (4 * j);
      }
    }
    if (!mask) continue;
    uint64_t* out = (uint64_t*)(block + 16 * D + d * 16 + first / 2);
    if (~mask) bits |= *out & ~mask;
    *out = bits;
  }
}

// 4 features of every 32 of a row, n in all: 8 lanes store 32 neighbouring ones.
template <bool kVector>
__device__ __forceinline__ void store_row(const HeadRows& r, int64_t row, int sub, const float* v, int n) {
#pragma unroll
  for (int j = 0; j < n; j += 4) {
    const int64_t e = row + 8 * j + 4 * sub;
    if (r.type == kF32) {
      float* o = (float*)r.p + e;
      if constexpr (kVector) {
        *(v4u*)o = v4u{__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                       __float_as_uint(v[j + 3])};
      } else {
        for (int i = 0; i < 4; ++i) o[i] = v[j + i];
      }
    } else {
      uint16_t* o = (uint16_t*)r.p + e;
      const v2u w = {f32_to_bf16x2(v[j], v[j + 1]), f32_to_bf16x2(v[j + 2], v[j + 3])};
      if constexpr (kVector) {
        *(v2u*)o = w;
      } else {
        for (int i = 0; i < 4; ++i) o[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

template <int D, bool kVector>
__global__ __launch_bounds__(kThreads) void kv_gather_kernel(HeadRows k, HeadRows v, KvArgs a,
                                                             uint32_t first_item) {
  constexpr int E = D / 8;
  __shared__ uint32_t codes[kBlockTokens * (E * 2 + 1)];
  const int64_t shard = blockIdx.y, item = first_item + blockIdx.z;
  const int head = blockIdx.x;
  Place at;
  if (!find_place(a, item, shard, head, &at)) return;
  const uint8_t* block = a.cache + at.at;
  if (at.at >= 0) {
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      const int d = i >> 1, first = (i & 1) * 16;
      const uint64_t bits = *(const uint64_t*)(block + 16 * D + d * 16 + first / 2);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        ((uint8_t*)(codes + (first + j) * (E * 2 + 1)))[d] = (uint8_t)(bits >> (4 * j) & 15);
    }
  }
  __syncthreads();
  const int t = threadIdx.x / 8, sub = threadIdx.x % 8;
  if (t < at.from || t >= at.to) return;
  float kx[E], vx[E];
#pragma unroll
  for (int e = 0; e < E; ++e) kx[e] = vx[e] = 0.0f;
  if (at.at >= 0) {   // a place without a page holds zeros
    const uint32_t kw = *(const uint32_t*)(block + 32 * D + t * 4);
    const uint32_t vw = *(const uint32_t*)(block + 32 * D + 128 + t * 4);
    const float ks = __uint_as_float(kw & 0xffff0000u), kz = __uint_as_float(kw << 16) - 128.0f;
    const float vs = __uint_as_float(vw & 0xffff0000u), vz = __uint_as_float(vw << 16) - 128.0f;
    const uint8_t* kr = block + t * (D / 2) + sub * 2;
    const uint32_t* vr = codes + t * (E * 2 + 1) + sub;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const uint32_t c = *(const uint16_t*)(kr + 4 * e), d = vr[2 * e];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        kx[e + j] = ((float)(c >> (4 * j) & 15) - kz) * ks;
        vx[e + j] = ((float)(d >> (8 * j) & 15) - vz) * vs;
      }
    }
  }
  const int64_t row = at.row + t;
  if (k.p) store_row<kVector>(k, shard * k.shard + row * k.pitch + head * k.head, sub, kx, E);
  if (v.p) store_row<kVector>(v, shard * v.shard + row * v.pitch + head * v.head, sub, vx, E);
}

// Launches over the blocks of 32 places that T rows of B sequences can touch
// (find_sequence), as many at once as a grid's third axis holds.
template <typename F>
hipError_t each_launch(const KvArgs& a, F f) {
  const int64_t items = a.T / kBlockTokens + 2 * (int64_t)a.B;
  for (int64_t i = 0; i < items; i += 65535)
    f(dim3(a.Hk, (unsigned)a.P, (unsigned)(items - i < 65535 ? items - i : 65535)), (uint32_t)i);
  return hipGetLastError();
}

#define BTQ_FOR_HEAD(D, CALL)            \
  switch (D) {                           \
    case 32: return CALL(32);            \
    case 64: return CALL(64);            \
    case 96: return CALL(96);            \
    case 128: return CALL(128);          \
    case 160: return CALL(160);          \
    case 192: return CALL(192);          \
    case 224: return CALL(224);          \
    default: return CALL(256);           \
  }

template <int D, int W>
hipError_t append_heads(const HeadRows& k, const HeadRows& v, const RopeArgs& rope, const KvArgs& a,
                        hipStream_t s) {
  return each_launch(a, [&](dim3 grid, uint32_t first) {
    if (k.type == kF32)
      kv_append_heads_kernel<D, W, kF32><<<grid, kThreads, 0, s>>>(k, v, rope, a, first);
    else
      kv_append_heads_kernel<D, W, kBf16><<<grid, kThreads, 0, s>>>(k, v, rope, a, first);
  });
}
template <int D, bool kVector>
hipError_t append(const HeadRows& k, const HeadRows& v, const RopeArgs& rope, const KvArgs& a,
                  hipStream_t s) {
  return each_launch(a, [&](dim3 grid, uint32_t first) {
    kv_append_kernel<D, kVector><<<grid, kThreads, 0, s>>>(k, v, rope, a, first);
  });
}
template <int D, bool kVector>
hipError_t gather(const HeadRows& k, const HeadRows& v, const KvArgs& a, hipStream_t s) {
  return each_launch(a, [&](dim3 grid, uint32_t first) {
    kv_gather_kernel<D, kVector><<<grid, kThreads, 0, s>>>(k, v, a, first);
  });
}

}  // namespace

hipError_t launch_kv_append(const HeadRows& k, const HeadRows& v, const RopeArgs& rope,
                            const KvArgs& a, hipStream_t s) {
  const bool vec = on16(k) && on16(v);
  const bool on = vec && (!rope.cos || (((uintptr_t)rope.cos & 15) == 0 && ((uintptr_t)rope.sin & 15) == 0));
  // runs of W features take turned ones that are those of whole lanes
  auto runs = [&](int W) { return on && (!rope.cos || rope.dim % (2 * W) == 0); };
  if (a.D == 192 && !runs(head_run(192)) && runs(16)) return append_heads<192, 16>(k, v, rope, a, s);
#define BTQ_CALL(N)                                                      \
  (runs(head_run(N)) ? append_heads<N, head_run(N)>(k, v, rope, a, s)    \
   : vec             ? append<N, true>(k, v, rope, a, s)                 \
                     : append<N, false>(k, v, rope, a, s))
  BTQ_FOR_HEAD(a.D, BTQ_CALL)
#undef BTQ_CALL
}

hipError_t launch_kv_gather(const HeadRows& k, const HeadRows& v, const KvArgs& a, hipStream_t s) {
  const bool vec = on16(k) && on16(v);
#define BTQ_CALL(N) (vec ? gather<N, true>(k, v, a, s) : gather<N, false>(k, v, a, s))
  BTQ_FOR_HEAD(a.D, BTQ_CALL)
#undef BTQ_CALL
}

}  // namespace btq
