// btq_kv_attention: queries over the keys and values of a paged 4-bit cache.
//
// Rows of the problem are (query, head) pairs that share a key head: G = Hq/Hk
// heads of n queries give n*G columns c of S = K Q^T, for each
//   t[key] = scale * sum_d q[d]*(code[key,d] - z[key])*s[key],  p = exp(t - max),
//   out = sum_key p*s'[key]*(code'[key,:] - z'[key]) / sum_key p.
// A nibble or-ed into the mantissa of bf16 128 is the exact bf16 128 + code, 7
// instructions for the 8 codes of a dword. So both products run on the matrix
// cores on 128 + code, and 128 + z is taken off after: from S as a product with
// the sum of q, from out as one more row of V^T that holds 128 + z', whose
// product sees the same rounded p*s' as the codes do. Scores are exact to fp32
// rounding; p*s' is rounded to bf16, as a weight of the second product.
//
// S is computed transposed (keys down, columns across), so that the 4 values of a
// column that a lane holds of two 16-key tiles are the 8 consecutive keys of the
// second product's operand: keys are dealt to tile rows to make it so, and
// nothing moves between lanes but the running maximum. One wave takes 128 keys
// (4 blocks) a step: 16-byte loads of K and V from HBM to registers, no LDS.
#include "kv.hpp"

namespace btq {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

constexpr int kTile = 128;                     // keys of a wave's step
constexpr int kTileBlocks = kTile / kBlockTokens;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ v4f mfma(v8b a, v8b b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 8 codes of a dword as bf16 128 + code, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ v8b codes_to_bf16(uint32_t w) {
  v4u r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
  return __builtin_bit_cast(v8b, r);
}
// 8 bf16 in that order.
__device__ __forceinline__ v8b deal(v4u w) {
  v4u r;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    r[2 * j] = __builtin_amdgcn_perm(w[2 + j], w[j], 0x05040100u);
    r[2 * j + 1] = __builtin_amdgcn_perm(w[2 + j], w[j], 0x07060302u);
  }
  return __builtin_bit_cast(v8b, r);
}

// x of lane kLane of each row of 16 lanes.
template <int kLane>
__device__ __forceinline__ uint32_t row_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x150 + kLane, 0xf, 0xf, true);
}

// x combined over the 4 lanes that hold one column.
template <typename F>
__device__ __forceinline__ float column_combine(float v, F f) {
  const uint32_t x = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  const uint32_t y = __float_as_uint(f(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(y, y, false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_max(float v) {
  return column_combine(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float column_sum(float v) {
  return column_combine(v, [](float a, float b) { return a + b; });
}

// A launch item: columns [col0, col0 + ncols) of a sequence and a key head.
struct Item {
  int b, head;
  int64_t shard;
  SeqRange seq;
  int col0;
};

// The keys of split `split`, in tiles: an equal share of the tiles that the item's
// columns see, no split shorter than kMinTiles.
constexpr int kMinTiles = 4;
struct KeyTiles {
  int begin, end;   // this split's
  int splits;       // those that have any
};
__device__ __forceinline__ KeyTiles key_tiles(int lo, int hi, int split, int splits) {
  const int t0 = lo / kTile, t1 = (hi + kTile - 1) / kTile;
  const int n = max(t1 - t0, 0);
  const int each = max((n + splits - 1) / splits, kMinTiles);
  KeyTiles k;
  k.begin = min(t0 + split * each, t1);
  k.end = min(k.begin + each, t1);
  k.splits = max((n + each - 1) / each, 1);
  return k;
}
// Keys that some column of [col0, col1) sees: [lo, hi).
__device__ __forceinline__ void keys_seen(const AttnArgs& a, const SeqRange& s, int col0, int col1,
                                          int* lo, int* hi) {
  const int first = s.first() + col0 / a.G, last = s.first() + (col1 - 1) / a.G;
  *hi = clamp_int(a.causal ? last + 1 : s.length, 0, s.length);
  *lo = a.window ? min(max(first + 1 - a.window, 0), *hi) : 0;
}

template <int D, int NT, bool kKeys>
struct AttnShape {
  static constexpr int C = 16 * NT;                    // columns of a wave
  static constexpr int kCols = kKeys ? C : 4 * C;      // of a block
  static constexpr int kShift = (kKeys ? 4 : 6) + (NT == 1 ? 0 : NT == 2 ? 1 : 2);
};

// Partial results of a split: [item][split][column] rows of D sums, then as many
// (maximum, sum of p) pairs.
struct Partial {
  float* sums;
  float* stats;
};
__device__ __forceinline__ Partial partial(const AttnArgs& a, int64_t unit, int64_t units, int split,
                                           int cols, int D) {
  const int64_t row = (unit * a.splits + split) * cols;
  return {a.ws + row * D, a.ws + units * a.splits * cols * D + row * 2};
}

__device__ __forceinline__ void store_out2(const AttnArgs& a, int64_t at, float x, float y) {
  if (a.out_type == kBf16)
    *(uint32_t*)((uint16_t*)a.out + at) = f32_to_bf16x2(x, y);
  else
    *(float2*)((float*)a.out + at) = make_float2(x, y);
}
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, const Item& it, int col) {
  return ((it.shard * a.kv.T + it.seq.begin + col / a.G) * a.Hq + it.head * a.G + col % a.G);
}
// Factor of sums relative to the maximum m2 when they join others under m. Where
// no score was above -Inf the sum of p is 0, or NaN if the scores were.
__device__ __forceinline__ float share(float m2, float sum, float m) {
  return m2 == kNegInf ? sum : exp2f(m2 - m);
}
__device__ __forceinline__ float lse_of(float m2, float l) {
  return l > 0.0f || l != l ? 0.6931471805599453f * (m2 + log2f(l)) : kNegInf;
}

template <int D, int NT, bool kKeys>
__global__ __launch_bounds__(256, 2) void attention_kernel(AttnArgs a, int64_t first_block,
                                                           int64_t items) {
  using S = AttnShape<D, NT, kKeys>;
  constexpr int NS = D / 32, ND = D / 16, C = S::C;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cl = lane & 15, g = lane >> 4;   // column (or tile row) and quarter of the wave

  const int64_t heads = a.kv.P * a.kv.Hk, id = first_block + blockIdx.x;
  const int64_t hk = id % heads, rest = id / heads;
  const int split = (int)(rest / items);
  // the last items of a causal batch see the most keys: they go first
  const int64_t item_id = items - 1 - rest % items;
  Item it;
  it.shard = hk / a.kv.Hk;
  it.head = (int)(hk % a.kv.Hk);
  int64_t sub;
  it.b = find_sequence(a.kv, a.G, S::kShift, 1, item_id, &sub);
  if (it.b < 0) return;
  it.seq = seq_range(a.kv, it.b);
  const int cols = it.seq.n * a.G;
  if (sub >= ((int64_t)cols + S::kCols - 1) / S::kCols) return;
  it.col0 = (int)sub * S::kCols + (kKeys ? 0 : wave * C);
  if (it.col0 >= cols) return;   // (a whole wave; no barrier follows where waves take columns)

  const int col1 = min(it.col0 + C, cols);
  int klo, khi;
  keys_seen(a, it.seq, it.col0, col1, &klo, &khi);
  const KeyTiles kt = key_tiles(klo, khi, split, a.splits);
  if (split >= kt.splits) return;

  // the queries: operand B of the first product, and their sums
  v8b q[NT][NS];
  float qsum[NT];
  int lo[NT], hi[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = it.col0 + n * 16 + cl;
    const int qi = col / a.G, pos = it.seq.first() + qi;
    hi[n] = a.causal ? min(pos + 1, it.seq.length) : it.seq.length;
    lo[n] = a.window ? max(pos + 1 - a.window, 0) : 0;
    const bool live = col < cols;
    const uint16_t* row = (const uint16_t*)a.q.p + it.shard * a.q.shard +
                          (it.seq.begin + (int64_t)(live ? qi : 0)) * a.q.pitch +
                          (it.head * (int64_t)a.G + (live ? col % a.G : 0)) * a.q.head + g * (D / 4);
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      v4u w;
      if (a.q_on16) {
        w = *(const v4u*)(row + 8 * s);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = row[8 * s + 2 * j] | (uint32_t)row[8 * s + 2 * j + 1] << 16;
      }
      if (!live) w = v4u{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sum += __uint_as_float(w[j] << 16) + __uint_as_float(w[j] & 0xffff0000u);
      q[n][s] = deal(w);
    }
    qsum[n] = column_sum(sum);
  }
  // keys that every column sees, for the tiles that need no mask
  const int all_hi = a.causal ? it.seq.first() + it.col0 / a.G + 1 : it.seq.length;
  const int all_lo = a.window ? it.seq.first() + (col1 - 1) / a.G + 1 - a.window : 0;

  v4f o[NT][ND], oz[NT];
  float m2[NT], l[NT];   // running maximum times scale*log2(e), sum of p of this lane's keys
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    oz[n] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < ND; ++d) o[n][d] = v4f{0, 0, 0, 0};
    m2[n] = kNegInf;
    l[n] = 0.0f;
  }

  constexpr int kStep = kKeys ? 4 : 1;
  for (int tile = kt.begin + (kKeys ? wave : 0); tile < kt.end; tile += kStep) {
    const int64_t vb = kv_block(a.kv, it.b, it.shard, it.head, tile * kTileBlocks + g);
    const int64_t kb = kv_block(a.kv, it.b, it.shard, it.head, tile * kTileBlocks + cl / 4);
    // a block without a page reads the cache's first one; the mask hides it
    const uint8_t* vp = a.kv.cache + (vb < 0 ? 0 : vb);
    const uint8_t* kp = a.kv.cache + (kb < 0 ? 0 : kb) + g * (D / 8) + (cl & 3) * (D / 2);
    uint32_t k[4][2][NS];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __builtin_memcpy(k[s][h], kp + (8 * s + 4 * h) * (D / 2), 4 * NS);
    // words of keys and values 2*cl and 2*cl + 1 of the lane's block
    uint32_t kw[2], vw[2];
    __builtin_memcpy(kw, vp + 32 * D + cl * 8, 8);
    __builtin_memcpy(vw, vp + 32 * D + 128 + cl * 8, 8);
    v4u v[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) v[d] = *(const v4u*)(vp + 16 * D + (d * 16 + cl) * 16);

    const int key0 = tile * kTile;
    const bool full = key0 >= all_lo && key0 + kTile <= all_hi && __ballot(vb < 0) == 0;

    // scores of 32 keys a lane and column: step s, half h, value i is the key
    // 8s + 4h + i of the lane's block
    float t[NT][4][2][4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4f acc[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NS; ++w) {
          const v8b kc = codes_to_bf16(k[s][h][w]);
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n] = mfma(kc, q[n][w], acc[n]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) t[n][s][h][i] = acc[n][i];
      }
    auto each_key = [&](auto f) {
      f(std::integral_constant<int, 0>{}); f(std::integral_constant<int, 1>{});
      f(std::integral_constant<int, 2>{}); f(std::integral_constant<int, 3>{});
      f(std::integral_constant<int, 4>{}); f(std::integral_constant<int, 5>{});
      f(std::integral_constant<int, 6>{}); f(std::integral_constant<int, 7>{});
      f(std::integral_constant<int, 8>{}); f(std::integral_constant<int, 9>{});
      f(std::integral_constant<int, 10>{}); f(std::integral_constant<int, 11>{});
      f(std::integral_constant<int, 12>{}); f(std::integral_constant<int, 13>{});
      f(std::integral_constant<int, 14>{}); f(std::integral_constant<int, 15>{});
    };
    each_key([&](auto pair) {
      constexpr int kPair = decltype(pair)::value;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        constexpr int kKey0 = 2 * kPair;
        const int key = kKey0 + j;
        const uint32_t w = row_lane<kPair>(kw[j]);
        const float ks = __uint_as_float(w & 0xffff0000u), kz = __uint_as_float(w << 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float& x = t[n][key >> 3][(key >> 2) & 1][key & 3];
          x = __builtin_fmaf(-kz, qsum[n], x) * ks;
        }
      }
    });
    if (!full) {
      const int base = key0 + g * kBlockTokens;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int from = vb < 0 ? kBlockTokens : lo[n] - base, to = hi[n] - base;
#pragma unroll
        for (int key = 0; key < 32; ++key) {
          float& x = t[n][key >> 3][(key >> 2) & 1][key & 3];
          x = key >= from && key < to ? x : kNegInf;
        }
      }
    }
    // the running maximum is raised only when a new one is 8 powers of 2 above it:
    // p then stays below 2^8, and the sums are rarely rescaled
    float alpha[NT];
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float m = kNegInf;
#pragma unroll
      for (int key = 0; key < 32; ++key) m = fmaxf(m, t[n][key >> 3][(key >> 2) & 1][key & 3]);
      alpha[n] = column_max(m) * a.scale2;
      raise |= alpha[n] > m2[n] + 8.0f || (m2[n] == kNegInf && alpha[n] > kNegInf);
    }
    if (__ballot(raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m = fmaxf(m2[n], alpha[n]);
        const float f = m == kNegInf ? 1.0f : exp2f(m2[n] - m);
        m2[n] = m;
        l[n] *= f;
        oz[n] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[n][d] *= f;
      }
    }
    // p, and the second product 8 keys of each block at a time
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float off = m2[n] == kNegInf ? 0.0f : m2[n];
#pragma unroll
      for (int key = 0; key < 32; ++key) {
        float& x = t[n][key >> 3][(key >> 2) & 1][key & 3];
        x = __builtin_amdgcn_exp2f(__builtin_fmaf(x, a.scale2, -off));   // hidden: 0
        l[n] += x;
      }
    }
    uint32_t zrow[16];
    each_key([&](auto pair) {
      constexpr int kPair = decltype(pair)::value;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = 2 * kPair + j;
        const uint32_t w = row_lane<kPair>(vw[j]);
        const float vs = __uint_as_float(w & 0xffff0000u);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float& x = t[n][key >> 3][(key >> 2) & 1][key & 3];
          // a hidden value's scale may be NaN
          x = !full && x == 0.0f ? 0.0f : x * vs;
        }
        // 128 + z of keys i (low half) and 4 + i; whatever stands in a place that
        // holds no value, it is a number
        uint32_t& pair_z = zrow[(key >> 3) * 4 + (key & 3)];
        if ((key & 4) == 0)
          pair_z = (w & 0xfu) | 0x43004300u;
        else
          pair_z |= (w & 0xfu) << 16;
      }
    });
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v8b p[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        v4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16x2(t[n][s][0][i], t[n][s][1][i]);
        p[n] = __builtin_bit_cast(v8b, w);
      }
      const v4u zw = {zrow[4 * s], zrow[4 * s + 1], zrow[4 * s + 2], zrow[4 * s + 3]};
      const v8b z = __builtin_bit_cast(v8b, zw);
#pragma unroll
      for (int n = 0; n < NT; ++n) oz[n] = mfma(z, p[n], oz[n]);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const v8b vc = codes_to_bf16(v[d][s]);
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][d] = mfma(vc, p[n], o[n][d]);
      }
    }
  }

  const int64_t unit = item_id * heads + hk, units = items * heads;
  if constexpr (!kKeys) {
    const Partial part = partial(a, unit, units, split, S::kCols, D);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = it.col0 + n * 16 + cl;
      const float sum = column_sum(l[n]);
      if (col >= cols) continue;
      const int pc = wave * C + n * 16 + cl;
      const float f = kt.splits > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      const int64_t at = kt.splits > 1 ? 0 : out_row(a, it, col);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const v4f x = (o[n][d] - oz[n]) * f;
        const int f0 = d * 16 + g * 4;
        if (kt.splits > 1) {
          *(v4f*)(part.sums + (int64_t)pc * D + f0) = x;
        } else {
          store_out2(a, at * D + f0, x[0], x[1]);
          store_out2(a, at * D + f0 + 2, x[2], x[3]);
        }
      }
      if (g == 0) {
        if (kt.splits > 1) {
          part.stats[2 * pc] = m2[n];
          part.stats[2 * pc + 1] = sum;
        } else if (a.lse) {
          a.lse[at] = lse_of(m2[n], sum);
        }
      }
    }
  } else {
    // the waves' sums, each relative to the common maximum, added in their order
    __shared__ float stat[4][C][2];
    constexpr int kChunk = NT == 1 ? (D < 128 ? D : 128) : NT == 2 ? (D < 64 ? D : 64) : 32;
    __shared__ float sums[4][C][kChunk + 4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float sum = column_sum(l[n]);
      if (g == 0) {
        stat[wave][n * 16 + cl][0] = m2[n];
        stat[wave][n * 16 + cl][1] = sum;
      }
    }
    __syncthreads();
    float f[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = n * 16 + cl;
      const float m = fmaxf(fmaxf(stat[0][c][0], stat[1][c][0]), fmaxf(stat[2][c][0], stat[3][c][0]));
      f[n] = share(m2[n], stat[wave][c][1], m);
    }
    const Partial part = partial(a, unit, units, split, S::kCols, D);
    for (int d0 = 0; d0 < D; d0 += kChunk) {
      if (d0) __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          if (d * 16 < d0 || d * 16 >= d0 + kChunk) continue;
          const v4f x = (o[n][d] - oz[n]) * f[n];
          *(v4f*)&sums[wave][n * 16 + cl][d * 16 - d0 + g * 4] = f[n] == 0.0f ? v4f{0, 0, 0, 0} : x;
        }
      __syncthreads();
      const int width = min(kChunk, D - d0);
      for (int i = threadIdx.x; i < C * width / 2; i += 256) {
        const int c = i / (width / 2), d = (i - c * (width / 2)) * 2;
        const int col = it.col0 + c;
        if (col >= cols) continue;
        const float m = fmaxf(fmaxf(stat[0][c][0], stat[1][c][0]), fmaxf(stat[2][c][0], stat[3][c][0]));
        float sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float mw = stat[w][c][0];
          sum += stat[w][c][1] * share(mw, stat[w][c][1], m);
          x += sums[w][c][d];
          y += sums[w][c][d + 1];
        }
        if (kt.splits > 1) {
          *(float2*)(part.sums + (int64_t)c * D + d0 + d) = make_float2(x, y);
          if (d0 + d == 0) {
            part.stats[2 * c] = m;
            part.stats[2 * c + 1] = sum;
          }
        } else {
          const int64_t at = out_row(a, it, col);
          const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
          store_out2(a, at * D + d0 + d, x * r, y * r);
          if (a.lse && d0 + d == 0) a.lse[at] = lse_of(m, sum);
        }
      }
    }
  }
}

// Joins the splits of an item's columns, in their order.
template <int D, int NT, bool kKeys>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int64_t first_block,
                                                             int64_t items) {
  using S = AttnShape<D, NT, kKeys>;
  constexpr int C = S::C;
  const int64_t heads = a.kv.P * a.kv.Hk, id = first_block + blockIdx.x;
  const int64_t hk = id % heads, item_id = id / heads;
  Item it;
  it.shard = hk / a.kv.Hk;
  it.head = (int)(hk % a.kv.Hk);
  int64_t sub;
  it.b = find_sequence(a.kv, a.G, S::kShift, 1, item_id, &sub);
  if (it.b < 0) return;
  it.seq = seq_range(a.kv, it.b);
  const int cols = it.seq.n * a.G;
  if (sub >= ((int64_t)cols + S::kCols - 1) / S::kCols) return;
  it.col0 = (int)sub * S::kCols;
  const int64_t unit = id, units = items * heads;
  for (int i = threadIdx.x; i < S::kCols * D / 2; i += 256) {
    const int c = i / (D / 2), d = (i - c * (D / 2)) * 2, col = it.col0 + c;
    if (col >= cols) return;
    // the same splits as the wave that had this column
    const int col0 = it.col0 + c / C * C;
    int klo, khi;
    keys_seen(a, it.seq, col0, min(col0 + C, cols), &klo, &khi);
    const KeyTiles kt = key_tiles(klo, khi, 0, a.splits);
    if (kt.splits <= 1) continue;
    float m = kNegInf;
    for (int s = 0; s < kt.splits; ++s)
      m = fmaxf(m, partial(a, unit, units, s, S::kCols, D).stats[2 * c]);
    float sum = 0.0f, x = 0.0f, y = 0.0f;
    for (int s = 0; s < kt.splits; ++s) {
      const Partial part = partial(a, unit, units, s, S::kCols, D);
      const float ms = part.stats[2 * c];
      const float f = share(ms, part.stats[2 * c + 1], m);
      const float2 v = *(const float2*)(part.sums + (int64_t)c * D + d);
      sum += part.stats[2 * c + 1] * f;
      x += v.x * f;
      y += v.y * f;
    }
    const int64_t at = out_row(a, it, col);
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
    store_out2(a, at * D + d, x * r, y * r);
    if (a.lse && d == 0) a.lse[at] = lse_of(m, sum);
  }
}

constexpr int64_t kMaxLaunch = int64_t(1) << 23;   // blocks of a launch

template <int D, int NT, bool kKeys>
hipError_t launch_shape(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
  const int64_t units = plan.items * a.kv.P * a.kv.Hk, blocks = units * plan.splits;
  for (int64_t b = 0; b < blocks; b += kMaxLaunch)
    attention_kernel<D, NT, kKeys>
        <<<dim3((unsigned)(blocks - b < kMaxLaunch ? blocks - b : kMaxLaunch)), 256, 0, s>>>(
            a, b, plan.items);
  if (plan.splits > 1)
    for (int64_t b = 0; b < units; b += kMaxLaunch)
      attention_join_kernel<D, NT, kKeys>
          <<<dim3((unsigned)(units - b < kMaxLaunch ? units - b : kMaxLaunch)), 256, 0, s>>>(
              a, b, plan.items);
  return hipGetLastError();
}

template <int D>
hipError_t launch_head(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
  if (plan.by_keys) return launch_shape<D, 1, true>(a, plan, s);
  return launch_shape<D, 2, false>(a, plan, s);
}

}  // namespace

AttnPlan attn_plan(int64_t P, int64_t T, int Hq, int Hk, int D, int B, int64_t max_length) {
  AttnPlan p;
  const int G = Hq / Hk;
  // columns of a sequence on average: a block's waves share out the keys of 16
  // columns, or take 32 columns each
  p.by_keys = T * G <= (int64_t)32 * B;
  p.tiles_of = p.by_keys ? 1 : 2;
  const int64_t cols = p.by_keys ? 16 : 128;
  p.items = T * G / cols + B;
  // blocks that fill the chip twice; a split has kMinTiles tiles at least
  const int64_t work = p.items < T * G ? p.items : T * G;
  const int64_t units = (work < 1 ? 1 : work) * P * Hk;
  int64_t most = (max_length + kTile * kMinTiles - 1) / (kTile * kMinTiles);
  int64_t want = (1024 + units - 1) / units;
  if (want > most) want = most;
  p.splits = (int)(want < 1 ? 1 : want);
  p.workspace = p.splits > 1 ? (size_t)(p.items * P * Hk * p.splits * cols) * (D + 2) * 4 : 0;
  return p;
}

hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
  switch (a.kv.D) {
    case 32: return launch_head<32>(a, plan, s);
    case 64: return launch_head<64>(a, plan, s);
    case 96: return launch_head<96>(a, plan, s);
    case 128: return launch_head<128>(a, plan, s);
    case 160: return launch_head<160>(a, plan, s);
    case 192: return launch_head<192>(a, plan, s);
    case 224: return launch_head<224>(a, plan, s);
    default: return launch_head<256>(a, plan, s);
  }
}

}  // namespace btq
