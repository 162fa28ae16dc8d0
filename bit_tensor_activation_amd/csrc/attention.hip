// btq_kv_attention: queries over the keys and values of a paged 4-bit cache.
//
// Rows of the problem are (query, head) pairs that share a key head: G = Hq/Hk
// heads of n queries give n*G columns c of S = K Q^T, for each
//   t[key] = scale * sum_d q[d]*(code[key,d] - z[key])*s[key],  p = exp(t - max),
//   out = sum_key p*s'[key]*(code'[key,:] - z'[key]) / sum_key p.
// Both products run on the matrix cores on the codes themselves, and z is taken off
// after: from S as a product with the sum of q, from out as one more row of V^T
// that holds 128 + z', whose product sees the same rounded p*s' as the codes do. A
// nibble or-ed into the mantissa of bf16 128 is the exact bf16 128 + code, 7
// instructions for the 8 codes of a dword. (Where many columns share the conversion,
// keys take 4 more to the exact fp16 code - z.) p*s' is rounded to bf16, as a weight
// of the second product. Codes as 8-bit floats, which a nibble in a byte of its own
// is, with queries as sums of two, take 3 instructions, but those products are summed
// to fewer bits: lse was off by 3.5e-6 of itself, and 1e-7 this way, which costs
// up to 7% (64 sequences of up to 4095 tokens 40 -> 43 us).
//
// S is computed transposed (keys down, columns across), so that the 4 values of a
// column that a lane holds of two 16-key tiles are the 8 consecutive keys of the
// second product's operand: keys are dealt to tile rows to make it so, and
// nothing moves between lanes but the running maximum.
//
// Two kernels. attention_keys_kernel, for few columns a sequence, is bound by the
// cache's bytes: each wave streams blocks of 32 tokens from HBM to registers (no
// LDS) and a block's waves share out the keys. attention_columns_kernel, for many,
// is bound by instructions: a block's waves take columns of their own and share
// the conversion of the codes through LDS.
#include "common.hpp"

namespace btq {
namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef uint16_t v2s __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ v4f mfma(v8b a, v8b b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 8 codes of a dword as bf16 128 + code, in the order 0 4 1 5 2 6 3 7. `magic` is
// 0x43004300 in a register: and-or takes one constant only.
__device__ __forceinline__ v4u codes_to_bf16(uint32_t w, uint32_t magic) {
  v4u r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = ((w >> (4 * j)) & 0x000f000fu) | magic;
  return r;
}
__device__ __forceinline__ v8b as_bf16(v4u w) { return __builtin_bit_cast(v8b, w); }
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

// The thread's number, computed where it stands: what follows from it is not kept in
// registers over the loops around.
__device__ __forceinline__ int thread_here() {
  int t = threadIdx.x;
  settle(t);
  return t;
}

// x of lane kLane of each row of 16 lanes.
template <int kLane>
__device__ __forceinline__ uint32_t row_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x150 + kLane, 0xf, 0xf, true);
}

template <int kLane>
__device__ __forceinline__ float from_lane(float x) {
  return __uint_as_float(row_lane<kLane>(__float_as_uint(x)));
}

// x of lane kLane of each quad.
template <int kLane>
__device__ __forceinline__ float from_quad(float x) {
  return __uint_as_float(dpp<0x55 * kLane>(__float_as_uint(x)));
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

// Keys of a wave behind which it takes 128 + z off the sums. Those hold up to 143 for a
// value of some steps, and every instruction rounds the whole of it: taken off at the end
// only, the error grew with a wave's keys, to 3.1e-2 of a row at 131072 of them. 3e-4 of a
// row, whatever their number, is what is left (the weights' rounding makes 1.7e-3). It costs
// the columns' kernel 2 to 3% at D = 128 (2048 new tokens over 32768: 2330 -> 2395 us; as much
// with 8 times as many keys, so it is not the subtractions), others up to 2% at D = 256.
constexpr int kOffsetKeys = 1024;

// Keeps a uniform branch a branch: without it the compiler turns short ones into
// selects that every pass pays for.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

template <int N>
struct Int {
  static constexpr int value = N;
};
template <int kBegin, int kEnd, int kStep, typename F>
__device__ __forceinline__ void static_for(F f) {
  if constexpr (kBegin < kEnd) {
    f(Int<kBegin>{});
    static_for<kBegin + kStep, kEnd, kStep>(f);
  }
}

// ---- what a wave keeps of its columns: 16*NT of them, column n*16 + lane%16 in
// the 4 lanes of that number ----
//
// NT is 1 in the keys' kernel, which alone calls take() and weights(); the columns' kernel has
// 1 or 2 and raises its maximum between its own instructions.
// Queries are operand B of the first product: bf16 as they come, or, for keys as
// fp16, fp16 taken by a power of 2 to a largest of 2^13 or more: exact down to 2^-27
// of that.
template <int D, int NT>
struct Columns {
  static constexpr int NS = D / 32, ND = D / 16;
  v8h q[NT][NS];             // bits of either type
  float qsum[NT];
  int lo[NT], hi[NT];        // keys that the column sees
  v4f o[NT][ND], oz[NT];     // sums of p*s'*(128 + code) of 4 features, and of p*s'*(128 + z')
  float m2[NT], l[NT];       // running maximum times scale*log2(e); sum of p of this lane's keys
  int all_lo, all_hi;        // keys that every column sees
  int any_lo, any_hi;        // keys that some column sees

  // Columns [col0, col0 + 16*NT) of a sequence, of which those below cols exist, and
  // their queries as they are, this lane's quarter of the features. Of W = 8 columns
  // lanes 8 .. 15 have the same ones as lanes 0 .. 7.
  template <int W = 16 * NT>
  __device__ __forceinline__ void fetch(const AttnArgs& a, const SeqRange& s, int64_t shard, int head,
                                        int col0, int cols, v4u (&w)[NT][NS]) {
    const int lane = thread_here() & 63, cl = lane & 15, g = lane >> 4;
    // (col0 the same in all lanes; col/G by a product, exact below 2^32/G)
    const int first = col0 / a.G, rest = col0 - first * a.G;
    auto query = [&](int col) {
      const uint32_t x = (uint32_t)(rest + col - col0);
      return first + (int)(a.G == 1 ? x : __umulhi(x, a.G_inverse));
    };
    const int last = query(min(col0 + W, cols) - 1);
    all_hi = a.causal ? min(s.first() + first + 1, s.length) : s.length;
    all_lo = a.window ? s.first() + last + 1 - a.window : 0;
    any_hi = a.causal ? clamp_int(s.first() + last + 1, 0, s.length) : s.length;
    any_lo = a.window ? max(s.first() + first + 1 - a.window, 0) : 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = col0 + n * 16 + (W < 16 ? cl % W : cl);
      const bool live = col < cols;
      const int qi = query(live ? col : col0), pos = s.first() + qi;
      hi[n] = a.causal ? min(pos + 1, s.length) : s.length;
      lo[n] = a.window ? max(pos + 1 - a.window, 0) : 0;
      const uint16_t* row = (const uint16_t*)a.q.p + shard * a.q.shard +
                            (s.begin + (int64_t)qi) * a.q.pitch +
                            (head * (int64_t)a.G + (live ? col : col0) - (int64_t)qi * a.G) * a.q.head +
                            g * (D / 4);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (a.q_on16) {
          w[n][i] = *(const v4u*)(row + 8 * i);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[n][i][j] = row[8 * i + 2 * j] | (uint32_t)row[8 * i + 2 * j + 1] << 16;
        }
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      oz[n] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < ND; ++d) o[n][d] = v4f{0, 0, 0, 0};
      m2[n] = kNegInf;
      l[n] = 0.0f;
    }
  }
  // Takes the zero points off what is summed so far (kOffsetKeys).
  __device__ __forceinline__ void take_off() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int d = 0; d < ND; ++d) o[n][d] -= oz[n];
      oz[n] = v4f{0, 0, 0, 0};
    }
  }
  // (a column that does not exist repeats the first one; its results go nowhere)
  __device__ __forceinline__ void take(const v4u (&w)[NT][NS]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float sum = 0.0f;
      v2s top = {0, 0};   // largest |q| of the even and of the odd features, as bits
#pragma unroll
      for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum += __uint_as_float(w[n][i][j] << 16) + __uint_as_float(w[n][i][j] & 0xffff0000u);
          top = __builtin_elementwise_max(top, __builtin_bit_cast(v2s, (uint32_t)w[n][i][j] & 0x7fff7fffu));
        }
        q[n][i] = __builtin_bit_cast(v8h, deal(w[n][i]));
      }
      // NaN and Inf in a query make all its scores NaN
      qsum[n] = column_sum(max(top[0], top[1]) < 0x7f80 ? sum : __uint_as_float(0x7fc00000u));
    }
  }
  // The largest finite |q| of the lane's features, as fp32 bits.
  static __device__ __forceinline__ uint32_t top_of(const v4u (&w)[NT][NS]) {
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = (h ? w[n][i][j] : w[n][i][j] << 16) & 0x7fff0000u;
            top = max(top, x < 0x7f800000u ? x : 0u);
          }
    return top;
  }
  // q*up as fp16. NaN and Inf in a query make all its scores NaN.
  __device__ __forceinline__ void take_halves(float up, const v4u (&w)[NT][NS]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const v4u x = __builtin_bit_cast(v4u, deal(w[n][i]));
        v4u y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f[h] = __uint_as_float(h ? x[j] & 0xffff0000u : x[j] << 16);
            f[h] = fabsf(f[h]) < INFINITY ? f[h] * up : __uint_as_float(0x7fc00000u);
          }
          y[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[0], f[1]));
        }
        q[n][i] = __builtin_bit_cast(v8h, y);
      }
  }
  // Scores t (value k is a key of the lane's) to weights p; l and the sums follow
  // the running maximum. It is raised only when a new one is 8 powers of 2 above
  // it: p stays below 2^8, and the sums are rarely rescaled.
  template <int kValues>
  __device__ __forceinline__ void weights(float scale2, float (&t)[NT][kValues]) {
    float top[NT];
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float m = t[n][0];
#pragma unroll
      for (int k = 1; k < kValues; ++k) m = fmaxf(m, t[n][k]);
      top[n] = column_max(m) * scale2;
      raise |= top[n] > m2[n] + 8.0f || (m2[n] == kNegInf && top[n] > kNegInf);
    }
    if (__ballot(raise)) {
      keep_branch();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m = fmaxf(m2[n], top[n]);
        const float f = m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m2[n] - m);
        m2[n] = m;
        l[n] *= f;
        oz[n] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[n][d] *= f;
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float off = m2[n] == kNegInf ? 0.0f : m2[n];
#pragma unroll
      for (int k = 0; k < kValues; ++k) {
        t[n][k] = __builtin_amdgcn_exp2f(__builtin_fmaf(t[n][k], scale2, -off));   // hidden: 0
        l[n] += t[n][k];
      }
    }
  }
};

// The 8 weights p*s' of a lane's keys 0 .. 7 (values 4*h + i) as operand B.
__device__ __forceinline__ v8b weights_to_bf16(const float* p) {
  v4u w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16x2(p[i], p[4 + i]);
  return as_bf16(w);
}

// Keys that some column of [col0, col1) sees: [lo, hi).
__device__ __forceinline__ void keys_seen(const AttnArgs& a, const SeqRange& s, int col0, int col1,
                                          int* lo, int* hi) {
  const int first = s.first() + col0 / a.G, last = s.first() + (col1 - 1) / a.G;
  *hi = clamp_int(a.causal ? last + 1 : s.length, 0, s.length);
  *lo = a.window ? min(max(first + 1 - a.window, 0), *hi) : 0;
}

// ---- results ----
__device__ __forceinline__ void store_out2(const AttnArgs& a, int64_t at, float x, float y) {
  if (a.out_type == kBf16)
    *(uint32_t*)((uint16_t*)a.out + at) = f32_to_bf16x2(x, y);
  else
    *(float2*)((float*)a.out + at) = make_float2(x, y);
}
// Row of out and lse of a column. (col/G by a product where that is exact.)
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, const SeqRange& s, int64_t shard,
                                           int head, int col) {
  const int q = a.G == 1 ? col
                         : (int64_t)col * a.G < (int64_t(1) << 32) ? (int)__umulhi((uint32_t)col, a.G_inverse)
                                                                   : col / a.G;
  return (shard * a.kv.T + s.begin + q) * a.Hq + head * a.G + (col - q * a.G);
}
// Factor of sums relative to the maximum m2 when they join others under m. Where
// no score was above -Inf the sum of p is 0, or NaN if the scores were.
__device__ __forceinline__ float share(float m2, float sum, float m) {
  return m2 == kNegInf ? sum : __builtin_amdgcn_exp2f(m2 - m);
}
__device__ __forceinline__ float lse_of(float m2, float l) {
  return l > 0.0f || l != l ? 0.6931471805599453f * (m2 + log2f(l)) : kNegInf;
}
// Partial results of `cols` columns: rows of D sums, then (maximum, sum of p) pairs.
struct Partial {
  float* sums;
  float* stats;
};
__device__ __forceinline__ Partial partial(const AttnArgs& a, int64_t slot, int64_t slots, int cols,
                                           int D) {
  return {a.ws + slot * cols * D, a.ws + slots * cols * D + slot * cols * 2};
}

// ---- few columns: waves share out the keys ----
//
// A wave takes 128 keys (4 blocks) a step: 16-byte loads of keys and values,
// 17 KB in flight a wave while the step before is computed, its page numbers a
// step earlier.
constexpr int kTile = 128;
constexpr int kTileBlocks = kTile / kBlockTokens;

//
// A group has W = 16 columns, or 8 where sequences have no more on average. Those
// take the matrix instruction's 16 columns twice: as 0 .. 7 for one step of 32 keys and
// as 8 .. 15 for the next, with zeros for queries (and later weights) in the other half,
// so both steps' scores add up in one accumulator and a lane has half as many to
// turn into weights (some 770 -> 660 vector instructions a tile at D = 128). The halves' sums join at
// the end.
template <int D, int W>
struct KeysWave {
  static constexpr int NT = 1;
  static constexpr int NS = D / 32, ND = D / 16;
  Columns<D, NT> c;
  const AttnArgs& a;
  int b, head;
  int64_t shard;
  uint32_t magic;
  // words of the lane's keys and values: KW pairs, h-th of a pair 4 keys further
  static constexpr int KW = W == 8 ? 2 : 1;
  uint32_t k[4][2][NS], kw[KW][2], vw[KW][2];
  v4u v[ND];
  v8h q_high[W == 8 ? NS : 1];   // W = 8: queries as columns 8 .. 15; c.q has the others

  __device__ __forceinline__ explicit KeysWave(const AttnArgs& args) : a(args) {
    magic = 0x43004300u;
    opaque(magic);
  }
  // Page number of block `i` of a tile, and its place in the cache. A block that is
  // not there reads the cache's first one, and the mask hides it.
  __device__ __forceinline__ int page(int tile, int i) const {
    const int slot = (tile * kTileBlocks + i) >> a.kv.page_shift;
    return a.kv.table[(int64_t)b * a.kv.max_pages + min(slot, (int)a.kv.max_pages - 1)];
  }
  __device__ __forceinline__ bool place(int tile, int end, int i, int page, int64_t* at) const {
    const int block = tile * kTileBlocks + i, shift = a.kv.page_shift;
    const bool there = tile < end && (block >> shift) < a.kv.max_pages && page >= 0 && page < a.kv.pages;
    const int64_t in_page = block & ((1 << shift) - 1);
    *at = there ? ((((shard * a.kv.pages + page) * a.kv.Hk + head) << shift) + in_page) *
                      kv_block_bytes(D)
                : 0;
    return there;
  }

  // Tiles begin, begin + step, .. of [begin, end) of columns [col0, ..) of a sequence.
  // The page numbers, the queries and the first tile load one behind the other.
  __device__ __forceinline__ void run(const SeqRange& seq, int col0, int cols, int begin, int end,
                                      int step) {
    c.clear();
    if (begin >= end) return;
    const int lane = thread_here() & 63, cl = lane & 15, g = lane >> 4;
    int pk = page(begin, cl / 4), pv = page(begin, g);
    v4u raw[NT][NS];
    c.template fetch<W>(a, seq, shard, head, col0, cols, raw);
    int64_t kat, vat;
    place(begin, end, cl / 4, pk, &kat);
    bool there = place(begin, end, g, pv, &vat);
    pk = page(begin + step, cl / 4), pv = page(begin + step, g);
    load_keys(kat);
    load_words(vat, kw, vw);
    load_values(vat);
    c.take(raw);
    if constexpr (W == 8) {
      const uint32_t low = cl < 8 ? 0xffffffffu : 0u;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const v4u x = __builtin_bit_cast(v4u, c.q[0][i]);
        c.q[0][i] = __builtin_bit_cast(v8h, x & low);
        q_high[i] = __builtin_bit_cast(v8h, x & ~low);
      }
    }
    // whether columns see different keys
    const int uneven = c.all_lo > c.any_lo || c.all_hi < c.any_hi ? 2 : 0;
    int done = 0;
    for (int tile = begin; tile < end; tile += step) {
      if (++done % (kOffsetKeys / kTile) == 0) {
        keep_branch();
        c.take_off();
      }
      const int key0 = tile * kTile;
      const bool full = key0 >= c.all_lo && key0 + kTile <= c.all_hi && __ballot(!there) == 0;
      place(tile + step, end, cl / 4, pk, &kat);
      const bool there_next = place(tile + step, end, g, pv, &vat);
      pk = page(tile + 2 * step, cl / 4), pv = page(tile + 2 * step, g);
      uint32_t kw_next[KW][2], vw_next[KW][2];
      load_words(vat, kw_next, vw_next);
      compute(kat, vat, key0, there, uniform(full ? 0 : 1 | uneven));
#pragma unroll
      for (int p = 0; p < KW; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j) kw[p][j] = kw_next[p][j], vw[p][j] = vw_next[p][j];
      there = there_next;
    }
    if constexpr (W == 8) join_halves();
  }
  // Columns 8 .. 15 added to 0 .. 7, whose they are.
  __device__ __forceinline__ void join_halves() {
    auto other = [](float x) { return __uint_as_float(dpp<0x128>(__float_as_uint(x))); };
    const float m = fmaxf(c.m2[0], other(c.m2[0]));
    // (where there was no score above -Inf the sums are 0 or NaN)
    const float f = c.m2[0] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(c.m2[0] - m);
    auto join = [&](float& x) {
      x *= f;
      x += other(x);
    };
    c.m2[0] = m;
    join(c.l[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float z = c.oz[0][i];
      join(z);
      c.oz[0][i] = z;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        float x = c.o[0][d][i];
        join(x);
        c.o[0][d][i] = x;
      }
    }
  }
  __device__ __forceinline__ void load_keys(int64_t at) {
    const int lane = threadIdx.x & 63, cl = lane & 15, g = lane >> 4;
    const uint8_t* p = a.kv.cache + at + g * (D / 8) + (cl & 3) * (D / 2);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) __builtin_memcpy(k[s][h], p + (8 * s + 4 * h) * (D / 2), 4 * NS);
  }
  // The first key of the lane's words, of its block: that of step cl/4, or, of pair p, of
  // step 2*p + cl/8.
  static __device__ __forceinline__ int word_key(int cl, int p) {
    return (W == 8 ? 16 * p + (cl & 8) : 8 * (cl >> 2)) + (cl & 3);
  }
  __device__ __forceinline__ void load_words(int64_t at, uint32_t (&x)[KW][2], uint32_t (&y)[KW][2]) {
    const int cl = threadIdx.x & 15;
    const uint32_t* from = (const uint32_t*)(a.kv.cache + at + 32 * D);
#pragma unroll
    for (int p = 0; p < KW; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[p][h] = from[word_key(cl, p) + 4 * h];
        y[p][h] = from[word_key(cl, p) + 4 * h + 32];
      }
  }
  __device__ __forceinline__ void load_values(int64_t at) {
    const uint8_t* p = a.kv.cache + at + 16 * D + (threadIdx.x & 15) * 16;
#pragma unroll
    for (int d = 0; d < ND; ++d) v[d] = *(const v4u*)(p + d * 256);
  }

  // One tile; the next one's keys load when the first product is done with these,
  // its values after the second.
  __device__ __forceinline__ void compute(int64_t kat, int64_t vat, int key0, bool there, int mask) {
    // Passes of KS steps of 32 keys, of which a lane has scores of KL.
    constexpr int KS = W == 8 ? 4 : 2, KL = 2;
    const int cl = threadIdx.x & 15;
    const int base = key0 + ((threadIdx.x & 63) >> 4) * kBlockTokens;
    // of the lane's keys and values; a step's products take them from the lanes
    // that have them. Whatever stands in a place that holds nothing, z' is a number.
    float ks[KW][2], kz[KW][2], vs[KW][2];
    uint32_t vz[KW];
#pragma unroll
    for (int p = 0; p < KW; ++p) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ks[p][h] = __uint_as_float(kw[p][h] & 0xffff0000u);
        kz[p][h] = -__uint_as_float(kw[p][h] << 16);
        vs[p][h] = __uint_as_float(vw[p][h] & 0xffff0000u);
      }
      vz[p] = (vw[p][0] & 0xfu) | (vw[p][1] & 0xfu) << 16 | magic;
    }
    if (mask) {   // places that no column sees may hold anything
      keep_branch();
#pragma unroll
      for (int p = 0; p < KW; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = base + word_key(cl, p) + 4 * h;
          if (!there || key < c.any_lo || key >= c.any_hi) vs[p][h] = 0.0f;
        }
    }
    // A value of the lane's key 4*h + i of its step s of the pass
    static_for<0, 4, KS>([&](auto pass) {
      constexpr int S0 = decltype(pass)::value;
      auto of_key = [&](const float (&x)[KW][2], auto index, auto value) {
        constexpr int s = decltype(index)::value, h = decltype(value)::value / 4, i = decltype(value)::value % 4;
        if constexpr (W == 8)
          return from_quad<i>(x[s][h]);
        else
          return from_lane<4 * (S0 + s) + i>(x[0][h]);
      };
      // Value 8*s + 4*h + i: key 4*h + i of the block's step S0 + s, or 2*s and, in lanes
      // 8 .. 15, 2*s + 1
      float t[1][8 * KL];
      static_for<0, KL, 1>([&](auto index) {
        constexpr int s = decltype(index)::value;
        // both halves together: a product waits for the one before it in its own
        v4f acc[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
#pragma unroll
        for (int w = 0; w < NS; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v8b kc = as_bf16(codes_to_bf16(k[W == 8 ? 2 * s : S0 + s][h][w], magic));
            acc[h] = mfma(kc, __builtin_bit_cast(v8b, c.q[0][w]), acc[h]);
          }
        if constexpr (W == 8) {
#pragma unroll
          for (int w = 0; w < NS; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const v8b kc = as_bf16(codes_to_bf16(k[2 * s + 1][h][w], magic));
              acc[h] = mfma(kc, __builtin_bit_cast(v8b, q_high[w]), acc[h]);
            }
        }
        static_for<0, 8, 1>([&](auto value) {
          constexpr int h = decltype(value)::value / 4, i = decltype(value)::value % 4;
          t[0][8 * s + 4 * h + i] = (acc[h][i] + of_key(kz, index, value) * c.qsum[0]) * of_key(ks, index, value);
        });
      });
      if constexpr (S0 + KS == 4) {
        issue_fence();
        load_keys(kat);
        issue_fence();
      }
      auto hide = [&](float with) {
        const int first = base + 8 * S0 + (W == 8 ? (threadIdx.x & 8) : 0);
        const int from = there ? c.lo[0] - first : 32, to = c.hi[0] - first;
#pragma unroll
        for (int v = 0; v < 8 * KL; ++v) {
          const int key = W == 8 ? (v >> 3) * 16 + (v & 7) : v;
          t[0][v] = key >= from && key < to ? t[0][v] : with;
        }
      };
      if (mask) {
        keep_branch();
        hide(kNegInf);
      }
      c.weights(a.scale2, t);
      static_for<0, KL, 1>([&](auto index) {
        static_for<0, 8, 1>([&](auto value) {
          t[0][8 * decltype(index)::value + decltype(value)::value] *= of_key(vs, index, value);
        });
      });
      if (mask & 2) {   // the scale of a value that only others see may be NaN
        keep_branch();
        hide(0.0f);
      }
      static_for<0, KS, 1>([&](auto index) {
        constexpr int s = decltype(index)::value;
        constexpr int L = W == 8 ? 8 * (s % 2) : 4 * (S0 + s), p = W == 8 ? s / 2 : 0;
        const v8b z = as_bf16(v4u{row_lane<L>(vz[p]), row_lane<L + 1>(vz[p]), row_lane<L + 2>(vz[p]),
                                  row_lane<L + 3>(vz[p])});
        v8b weight = weights_to_bf16(&t[0][8 * (W == 8 ? s / 2 : s)]);
        if constexpr (W == 8) {
          const uint32_t mine = (threadIdx.x & 8) == (s % 2 ? 8u : 0u) ? 0xffffffffu : 0u;
          weight = as_bf16(__builtin_bit_cast(v4u, weight) & mine);
        }
        c.oz[0] = mfma(z, weight, c.oz[0]);
#pragma unroll
        for (int d = 0; d < ND; ++d)
          c.o[0][d] = mfma(as_bf16(codes_to_bf16(v[d][S0 + s], magic)), weight, c.o[0][d]);
      });
    });
    issue_fence();
    load_values(vat);
    issue_fence();
  }
};

// Tiles of a sequence's columns, from its rows' first key to their last; one at
// least where there are columns, so that rows that see nothing are written too.
// (All column tiles count the same; a mask hides what a causal one does not see.)
struct SeqTiles {
  int first, tiles, groups;   // first tile, tiles, column groups of 2^shift
  // A group's length in the flat order: its tiles, and what it costs a block to begin
  // with another group and to join its sums.
  int begin;
  __device__ __forceinline__ int length() const { return tiles + begin; }
};
__device__ __forceinline__ SeqTiles seq_tiles(const AttnArgs& a, const SeqRange& s, int shift) {
  SeqTiles r;
  const int64_t cols = (int64_t)s.n * a.G;
  r.groups = (int)((cols + (1 << shift) - 1) >> shift);
  const int hi = s.length;
  const int lo = a.window ? min(max(s.first() + 1 - a.window, 0), max(hi - 1, 0)) : 0;
  r.first = lo / kTile;
  r.tiles = max((hi + kTile - 1) / kTile - r.first, 1);
  r.begin = a.begin;
  return r;
}

// The work of a launch laid out flat: head after head, sequence after sequence,
// column group after group, tile after tile.
struct Flat {
  int64_t per_head;   // tiles of a head
  int b;              // the sequence that holds position `at` of a head, and
  int64_t begin;      // where its tiles begin
};
template <int kThreads>
__device__ __forceinline__ int64_t flat_total(const AttnArgs& a, int shift, int64_t* lds, int64_t* mine,
                                              int* b0, int* b1) {
  const int each = (a.kv.B + kThreads - 1) / kThreads;
  *b0 = min((int)threadIdx.x * each, a.kv.B);
  *b1 = min(*b0 + each, a.kv.B);
  int64_t sum = 0;
  for (int b = *b0; b < *b1; ++b) {
    const SeqTiles t = seq_tiles(a, seq_range(a.kv, b), shift);
    sum += (int64_t)t.groups * t.length();
  }
  int64_t inc = sum;   // inclusive sum over the wave
  for (int d = 1; d < 64; d *= 2) {
    const int64_t v = __shfl_up(inc, d);
    if ((int)(threadIdx.x & 63) >= d) inc += v;
  }
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < (int)threadIdx.x >> 6) before += lds[w];
    total += lds[w];
  }
  *mine = before + inc - sum;
  return total;
}
template <int kThreads>
__device__ __forceinline__ void flat_find(const AttnArgs& a, int shift, int64_t at, int64_t mine, int b0,
                                          int b1, Flat* out) {
  for (int b = b0; b < b1; ++b) {
    const SeqTiles t = seq_tiles(a, seq_range(a.kv, b), shift);
    const int64_t n = (int64_t)t.groups * t.length();
    if (at >= mine && at < mine + n) {
      out->b = b;
      out->begin = mine;
    }
    mine += n;
  }
}
constexpr int64_t kStreamBlocks = 256;   // one a CU
// a/b, in 32 bits where they fit (a 64-bit division takes some 150 instructions).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if ((uint64_t)(a | b) >> 32 == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}
// The flat order is cut into equal shares, of 4 tiles and a beginning at least.
__device__ __forceinline__ int64_t flat_share(int64_t all, int begin) {
  const int64_t n = (all + kStreamBlocks - 1) / kStreamBlocks;
  return n < begin + 4 ? begin + 4 : n;
}

// The sums of the team's first `waves` waves (the others had no tile), each relative
// to the common maximum, added in the waves' order; to `out` where they are whole,
// else to a partial result.
template <int D, int W, int kTeam, bool kStream>
__device__ __forceinline__ void join_team(const AttnArgs& a, const Columns<D, 1>& c, const SeqRange& seq,
                                          int64_t shard, int head, int col0, int cols, int waves, bool whole,
                                          const Partial& part) {
  constexpr int C = W, kVec = D / 4;
  __shared__ float2 stat[kTeam][C];       // maximum and sum of p
  __shared__ float factor[C];             // 1/sum of all, or 1
  __shared__ v4f sums[kTeam][C][kVec + 1];
  const int tid = thread_here(), lane = tid & 63, wave = tid >> 6, cl = lane & 15, g = lane >> 4;
  const int live = min(C, cols - col0);
  const float own = column_sum(c.l[0]);
  if (g == 0 && cl < C) stat[wave][cl] = make_float2(c.m2[0], own);
  lds_barrier();
  if (wave < waves && cl < live) {
    float m = kNegInf;
    for (int w = 0; w < waves; ++w) m = fmaxf(m, stat[w][cl].x);
    const float f = share(c.m2[0], own, m);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) sums[wave][cl][d * 4 + g] = (c.o[0][d] - c.oz[0]) * f;
    if (wave == 0 && g == 0) {
      float sum = 0.0f;
      for (int w = 0; w < waves; ++w) sum += stat[w][cl].y * share(stat[w][cl].x, stat[w][cl].y, m);
      factor[cl] = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      if (!whole)
        *(float2*)(part.stats + 2 * cl) = make_float2(m, sum);
      else if (a.lse)
        a.lse[out_row(a, seq, shard, head, col0 + cl)] = lse_of(m, sum);
    }
  }
  lds_barrier();
  for (int i = tid; i < live * kVec; i += 64 * kTeam) {
    const int col = i / kVec, d = i - col * kVec;
    v4f x = sums[0][col][d];
    for (int w = 1; w < waves; ++w) x += sums[w][col][d];
    if (whole) {
      x *= factor[col];
      const int64_t at = out_row(a, seq, shard, head, col0 + col) * D + 4 * d;
      store_out2(a, at, x[0], x[1]);
      store_out2(a, at + 2, x[2], x[3]);
    } else {
      *(v4f*)(part.sums + (int64_t)col * D + 4 * d) = x;
    }
  }
  if (kStream) lds_barrier();   // the next segment writes stat and sums again
}

// A group of columns that goes on past the end of the block it begins in. The cuts
// of all blocks lie behind their partial results.
struct Cut {
  int32_t parts;   // blocks that it lies in; 0: none
  int32_t b, hk, group;
};
template <int D, int C>
__device__ __forceinline__ Cut* cuts(const AttnArgs& a) {
  return (Cut*)(a.ws + 2 * kStreamBlocks * C * (D + 2));
}

// kStream: the flat order is cut into equal shares, one a block, so a batch of any
// lengths fills the chip evenly; a group of columns that a cut divides leaves
// partial results (slot 2*block + 1 where it begins in the block, else 2*block),
// which attention_join_kernel adds. Else a block takes one group of columns.
template <int D, int W, int kTeam, bool kStream>
__global__ __launch_bounds__(64 * kTeam, D <= 128 ? 2 : 1) void attention_keys_kernel(AttnArgs a,
                                                                                     uint32_t first_item) {
  constexpr int kShift = W == 8 ? 3 : 4;
  const int wave = uniform((int)threadIdx.x >> 6);
  KeysWave<D, W> w(a);
  if constexpr (!kStream) {
    w.head = blockIdx.x;
    w.shard = blockIdx.y;
    int64_t sub;
    SeqRange seq;
    w.b = find_sequence(a.kv, a.G, kShift, part_extra(a.G, kShift), first_item + blockIdx.z, &sub, &seq);
    if (w.b < 0) return;
    const int cols = seq.n * a.G;
    if ((sub << kShift) >= cols) return;
    const int col0 = (int)sub << kShift;
    int lo, hi;
    keys_seen(a, seq, col0, min(col0 + W, cols), &lo, &hi);
    const int t0 = lo / kTile, t1 = (hi + kTile - 1) / kTile;
    w.run(seq, col0, cols, t0 + wave, t1, kTeam);
    join_team<D, W, kTeam, kStream>(a, w.c, seq, w.shard, w.head, col0, cols, clamp_int(t1 - t0, 1, kTeam),
                                    true, Partial{});
  } else {
    __shared__ int64_t scan[kTeam];
    __shared__ Flat found;
    int64_t mine;
    int b0, b1;
    const int64_t per_head =
        uniform(flat_total<64 * kTeam>(a, kShift, scan, &mine, &b0, &b1));
    const int64_t all = per_head * a.kv.P * a.kv.Hk, each = flat_share(all, a.begin);
    const int64_t x0 = blockIdx.x * each, x1 = min(x0 + each, all);
    Cut* cut = cuts<D, W>(a) + blockIdx.x;
    if (x0 >= x1) {
      if (threadIdx.x == 0) cut->parts = 0;
      return;
    }
    int hk = (int)divide(x0, per_head);
    flat_find<64 * kTeam>(a, kShift, x0 - hk * per_head, mine, b0, b1, &found);
    __syncthreads();
    w.b = __builtin_amdgcn_readfirstlane(found.b);
    int64_t begin = hk * per_head + uniform(found.begin);   // of sequence w.b of head hk
    int parts = 0, cut_group = 0;
    for (int64_t x = x0; x < x1;) {
      const SeqRange seq = uniform(seq_range(a.kv, w.b));
      const SeqTiles st = seq_tiles(a, seq, kShift);
      const int64_t n = (int64_t)st.groups * st.length();
      if (x >= begin + n) {   // on to the next sequence, or the next head's first
        begin += n;
        if (++w.b == a.kv.B) w.b = 0, ++hk;
        continue;
      }
      const int group = (int)divide(x - begin, st.length());
      const int64_t unit = begin + (int64_t)group * st.length(), tiles = unit + st.begin;
      const int t0 = (int)(max(x, tiles) - tiles), t1 = (int)(min(x1, unit + st.length()) - tiles);
      x = unit + st.length();
      if (t1 <= t0) continue;   // a share that ends in a beginning leaves it to the next
      const int cols = seq.n * a.G, col0 = group << kShift;
      w.shard = hk / a.kv.Hk;
      w.head = hk % a.kv.Hk;
      w.run(seq, col0, cols, st.first + t0 + wave, st.first + t1, kTeam);
      join_team<D, W, kTeam, kStream>(
          a, w.c, seq, w.shard, w.head, col0, cols, min(t1 - t0, kTeam), t1 - t0 == st.tiles,
          partial(a, 2 * (int64_t)blockIdx.x + (t0 == 0), 2 * kStreamBlocks, W, D));
      if (x > x1 && t0 == 0) {
        parts = (int)(divide(x - 1, each) - blockIdx.x) + 1;
        cut_group = group;
      }
    }
    // (the last group that this block began, if it goes on)
    if (threadIdx.x == 0) *cut = {parts, w.b, hk, cut_group};
  }
}

// Adds the partial results of a cut group: blockIdx.x is the block that it begins
// in, blockIdx.y a part of its columns. Threads by (team, column, 4 features), the
// blocks of a cut shared out over teams.
constexpr int kJoinThreads = 512;
template <int D>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttnArgs a) {
  constexpr int C = 16, kVec = D / 4;
  constexpr int kSpan = C / 4;                                       // columns of a block
  constexpr int kItems = kSpan * kVec;
  constexpr int kTeams = kJoinThreads / kItems;
  static_assert(kTeams >= 2, "threads");
  __shared__ v4f sums[kTeams][kItems];
  __shared__ float stat[kTeams][kItems][2];
  const Cut cut = cuts<D, C>(a)[blockIdx.x];
  if (cut.parts == 0) return;
  const SeqRange seq = uniform(seq_range(a.kv, cut.b));
  const int cols = seq.n * a.G, first = blockIdx.y * kSpan, col0 = (cut.group << 4) + first;
  if (col0 >= cols) return;
  const int64_t slots = 2 * kStreamBlocks;
  // (threads behind the last whole team have no part)
  const int team = threadIdx.x / kItems, i = threadIdx.x - team * kItems;
  const int c = i / kVec, d = (i - c * kVec) * 4;
  const bool live = team < kTeams && col0 + c < cols;
  // relative to a running maximum, 8 blocks at a time
  float m = kNegInf, l = 0.0f;
  v4f x = {0, 0, 0, 0};
  if (live) {
    const int span = (cut.parts + kTeams - 1) / kTeams, end = min((team + 1) * span, cut.parts);
    for (int p0 = team * span; p0 < end; p0 += 8) {
      float ms[8], ls[8];
      v4f ys[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = min(p0 + j, end - 1);
        const Partial q = partial(a, 2 * ((int64_t)blockIdx.x + p) + (p == 0), slots, C, D);
        const float2 st = *(const float2*)(q.stats + 2 * (first + c));
        ms[j] = p0 + j < end ? st.x : kNegInf;
        ls[j] = p0 + j < end ? st.y : 0.0f;
        ys[j] = *(const v4f*)(q.sums + (int64_t)(first + c) * D + d);
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, ms[j]);
      float f = share(m, l, top);
      l *= f;
      x *= f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f = share(ms[j], ls[j], top);
        l += ls[j] * f;
        if (p0 + j < end) x += ys[j] * f;
      }
      m = top;
    }
  }
  if (team < kTeams) {
    sums[team][i] = x;
    stat[team][i][0] = m;
    stat[team][i][1] = l;
  }
  __syncthreads();
  if (live && team == 0) {
    float top = m;
#pragma unroll
    for (int t = 1; t < kTeams; ++t) top = fmaxf(top, stat[t][i][0]);
    float f = share(m, l, top);
    m = top;
    l *= f;
    x *= f;
#pragma unroll
    for (int t = 1; t < kTeams; ++t) {
      f = share(stat[t][i][0], stat[t][i][1], top);
      l += stat[t][i][1] * f;
      x += sums[t][i] * f;
    }
    const int64_t at = out_row(a, seq, cut.hk / a.kv.Hk, (int)(cut.hk % a.kv.Hk), col0 + c);
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    store_out2(a, at * D + d, x[0] * r, x[1] * r);
    store_out2(a, at * D + d + 2, x[2] * r, x[3] * r);
    if (a.lse && d == 0) a.lse[at] = lse_of(m, l);
  }
}

// ---- many columns: a block's 4 waves take 16*NT columns each ----
//
// A tile of 64 keys (2 blocks, each loaded by 2 waves) goes from HBM through
// registers to LDS, in the order in which the matrix instructions' operands are read:
// 64 lanes of 16 consecutive bytes. Keys go as the exact fp16 code - z (a nibble or-ed
// into the mantissa of 1024, less 1024 + z), values as bf16 128 + code. Two tiles of
// LDS: while one is used the next is converted, and the one after is on its way from
// memory. A score takes one multiply-add from the product to the exponent, which
// is relative to the maximum of the tiles before.
// A matrix instruction that waits for its unit holds up the vector instructions of
// the SIMD's other waves (measured: a wave of the one kind and a wave of the other
// take as long as both one after the other), so the two overlap only where one wave
// alternates them; 2 multiply-adds behind each cost next to nothing.
constexpr int kColsTile = 64;
constexpr int kRing = 4;

template <int D, int NT>
struct ColsShape {
  static constexpr int NS = D / 32, ND = D / 16, C = 16 * NT, kCols = 4 * C;
  static constexpr int kShift = NT == 1 ? 6 : 7;
  static constexpr int VN = (D + 127) / 128;   // rows of values a thread
  struct Buffer {
    v4u k[4 * NS][64], v[2 * ND][64];
    float ks[64], vs[64];                      // scales: of keys in powers of 2 of p
    uint16_t vz[64];
    int there[2];
  };
};

// The keys of split `split`, in tiles: an equal share of the tiles that the item's
// columns see, no split shorter than kMinTiles.
constexpr int kMinTiles = 8;
struct KeyTiles {
  int begin, end;   // this split's
  int splits;       // those that have any
};
__device__ __forceinline__ KeyTiles key_tiles(int lo, int hi, int split, int splits) {
  const int t0 = lo / kColsTile, t1 = (hi + kColsTile - 1) / kColsTile;
  const int n = max(t1 - t0, 0);
  const int each = max((n + splits - 1) / splits, kMinTiles);
  KeyTiles k;
  k.begin = min(t0 + split * each, t1);
  k.end = min(k.begin + each, t1);
  k.splits = max((n + each - 1) / each, 1);
  return k;
}
template <int D, int NT>
__global__ __launch_bounds__(256, 2) void attention_columns_kernel(AttnArgs a, uint32_t first_item,
                                                                   uint32_t items) {
  using S = ColsShape<D, NT>;
  constexpr int NS = S::NS, ND = S::ND, C = S::C;
  __shared__ typename S::Buffer buf[2];
  __shared__ uint32_t tops[4];
  const int tid = threadIdx.x, lane = tid & 63, cl = lane & 15, g = lane >> 4;
  const int wave = uniform(tid >> 6);

  const int head = blockIdx.x;
  const int64_t shard = blockIdx.y, heads = a.kv.P * a.kv.Hk, hk = shard * a.kv.Hk + head;
  const uint32_t id = first_item + blockIdx.z;
  const int split = (int)(id / items);
  // the last items of a causal batch see the most keys: they go first
  const int64_t item = items - 1 - (id - split * items);
  int64_t sub;
  SeqRange seq;
  const int b = find_sequence(a.kv, a.G, S::kShift, part_extra(a.G, S::kShift), item, &sub, &seq);
  if (b < 0) return;
  const int cols = seq.n * a.G;
  if ((sub << S::kShift) >= cols) return;
  const int block_col = (int)sub << S::kShift;
  int klo, khi;
  keys_seen(a, seq, block_col, min(block_col + S::kCols, cols), &klo, &khi);
  const KeyTiles kt = key_tiles(klo, khi, split, a.splits);
  if (split >= kt.splits) return;

  const int col0 = block_col + wave * C;
  const bool live = col0 < cols;    // a wave without columns loads and waits with the others
  Columns<D, NT> c;
  float unit;                       // from the first product to powers of 2 of p
  {
    v4u raw[NT][NS];
    c.fetch(a, seq, shard, head, live ? col0 : block_col, cols, raw);
    c.clear();
    const uint32_t top = wave_combine(c.top_of(raw), [](uint32_t x, uint32_t y) { return max(x, y); });
    if (lane == 0) tops[wave] = top;
    lds_barrier();
    const uint32_t all = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    // 2^(13 - exponent of the block's largest |q|), within the powers that have a reciprocal
    const float up = __uint_as_float((uint32_t)(254 + 13 - clamp_int((int)(all >> 23), 20, 254)) << 23);
    unit = a.scale2 / up;
    c.take_halves(up, raw);
  }
  uint32_t magic = 0x43004300u, magic16 = 0x64006400u;
  opaque(magic);
  opaque(magic16);

  // Loads: waves 2*j and 2*j + 1 take block j of a tile; a thread takes a quarter of a
  // key's row and its word, rows of values, and the word of a value.
  const int block = wave >> 1, krow = lane & 31, quarter = 2 * (wave & 1) + (lane >> 5);
  const int kfrag = block * 2 + (krow >> 2 & 1), kslot = quarter * 16 + (krow >> 3) * 4 + (krow & 3);
  const int vrow = (wave & 1) * 64 + lane;
  uint32_t kreg[NS], kword, vword;
  v4u vreg[S::VN];
  int page, there = 0;              // the page number is looked up a tile ahead
  auto look_up = [&](int tile) {
    const int slot = min((2 * tile + block) >> a.kv.page_shift, (int)a.kv.max_pages - 1);
    page = a.kv.table[(int64_t)b * a.kv.max_pages + slot];
  };
  int loaded = 0;                   // first place of the block loaded last
  auto load = [&](int tile) {
    const int t = min(tile, kt.end - 1), shift = a.kv.page_shift, at = 2 * t + block, p = uniform(page);
    there = (at >> shift) < a.kv.max_pages && p >= 0 && p < a.kv.pages;
    // (the mask hides what a block without a page seems to hold)
    const int64_t offset = there ? ((((shard * a.kv.pages + p) * a.kv.Hk + head) << shift) +
                                    (at & ((1 << shift) - 1))) * kv_block_bytes(D)
                                 : 0;
    loaded = at * kBlockTokens;
    look_up(tile + 1);
    const uint8_t* from = a.kv.cache + offset;
    __builtin_memcpy(kreg, from + (uint32_t)(krow * (D / 2) + quarter * (D / 8)), 4 * NS);
    kword = *(const uint32_t*)(from + (uint32_t)(32 * D + krow * 4));
    vword = *(const uint32_t*)(from + (uint32_t)(32 * D + 128 + krow * 4));
#pragma unroll
    for (int i = 0; i < S::VN; ++i)
      vreg[i] = *(const v4u*)(from + (uint32_t)(16 * D + min(vrow + 128 * i, D - 1) * 16));
  };
  // Piece i of a tile's conversion: a dword of 8 codes of a key, or of a feature's values.
  constexpr int kPieces = NS + 4 * S::VN;
  auto write_piece = [&](typename S::Buffer& o, int i) {
    if (i < NS) {
      const v2h zero = __builtin_bit_cast(v2h, (kword & 0xfu) * 0x10001u | magic16);   // 1024 + z, twice
      const v4u x = codes_to_bf16(kreg[i], magic16);   // 1024 + code, in the same order
      v4u y;
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, (uint32_t)x[j]) - zero);
      o.k[kfrag * NS + i][kslot] = y;
    } else {
      const int r = (i - NS) >> 2, q = (i - NS) & 3, d = vrow + 128 * r;
      if (D % 128 == 0 || d < D) o.v[block * ND + (d >> 4)][q * 16 + (d & 15)] = codes_to_bf16(vreg[r][q], magic);
    }
  };
  auto write_words = [&](typename S::Buffer& o) {
    if (quarter == 0) {
      o.ks[block * 32 + krow] = __uint_as_float(kword & 0xffff0000u) * unit;
    } else if (quarter == 2) {
      // a place that holds nothing gets scale 0, so that it stays a number
      const bool held = there && loaded + krow < seq.length;
      o.vs[block * 32 + krow] = held ? __uint_as_float(vword & 0xffff0000u) : 0.0f;
      o.vz[block * 32 + (krow & 24) + (krow & 3) * 2 + (krow >> 2 & 1)] = (uint16_t)(0x4300u | (vword & 0xfu));
      if (krow == 0) o.there[block] = there;
    }
  };
  auto compute = [&](const typename S::Buffer& in, typename S::Buffer& next, int key0, int mask) {
    float t[NT][16], off[NT];
    auto hide = [&](float with) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int key = key0 + (k >> 3) * 32 + g * 8 + (k & 7);
          const bool seen = key >= c.lo[n] && key < c.hi[n] && (mask >> (1 + (k >> 3)) & 1);
          t[n][k] = seen ? t[n][k] : with;
        }
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) off[n] = c.m2[n] == kNegInf ? 0.0f : c.m2[n];
    // Fragment f of the keys, 4*NS of them, then of the values: kAhead of them are on
    // their way from LDS. Each is a slot of NT matrix instructions with a few others
    // behind, fenced so that they stay there (see the header of this kernel).
    v4u ring[kRing];
    auto read = [&](int f) {
      if (f < 4 * NS)
        ring[f % kRing] = in.k[f][lane];
      else if (f < 8 * NS)
        ring[f % kRing] = in.v[f - 4 * NS][lane];
    };
#pragma unroll
    for (int f = 0; f < kRing - 1; ++f) read(f);
    v4f ks[2], acc[2][NT];
    ks[0] = *(const v4f*)&in.ks[g * 8];
    // group j*2 + h: keys 8*g + 4*h .. of block j
    auto scores = [&](int group, int i) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        t[n][4 * group + i] = __builtin_fmaf(acc[group & 1][n][i], ks[group & 1][i], -off[n]);
    };
#pragma unroll
    for (int group = 0; group < 4; ++group) {
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[group & 1][n] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < NS; ++w) {
        const int f = group * NS + w;
        read(f + kRing - 1);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[group & 1][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
              __builtin_bit_cast(v8h, ring[f % kRing]), c.q[n][w], acc[group & 1][n], 0, 0, 0);
        if (group > 0 && NS >= 4 && w < 4) scores(group - 1, w);
        issue_fence();
      }
      if (NS < 4 && group > 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) scores(group - 1, i);
      if (group < 3) ks[(group + 1) & 1] = *(const v4f*)&in.ks[((group + 1) >> 1) * 32 + g * 8 + ((group + 1) & 1) * 4];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) scores(3, i);
    if (mask & 1) {
      keep_branch();
      hide(kNegInf);
    }
    // the running maximum, as in Columns::weights, but t is relative to it already
    float top[NT];
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float m = t[n][0];
#pragma unroll
      for (int k = 1; k < 16; ++k) m = fmaxf(m, t[n][k]);
      top[n] = column_max(m);
      raise |= top[n] > 8.0f || (c.m2[n] == kNegInf && top[n] > kNegInf);
    }
    if (__ballot(raise)) {
      keep_branch();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool first = c.m2[n] == kNegInf;
        const float up = first ? (top[n] == kNegInf ? 0.0f : top[n]) : fmaxf(top[n], 0.0f);
        const float f = first ? 1.0f : __builtin_amdgcn_exp2f(-up);   // (nothing to scale at first)
        c.m2[n] = first ? top[n] : c.m2[n] + up;
        c.l[n] *= f;
        c.oz[n] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) c.o[n][d] *= f;
#pragma unroll
        for (int k = 0; k < 16; ++k) t[n][k] -= up;
      }
    }
    v4f vs[4];
    v4u z[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) vs[k] = *(const v4f*)&in.vs[(k >> 1) * 32 + g * 8 + (k & 1) * 4];
#pragma unroll
    for (int j = 0; j < 2; ++j) z[j] = *(const v4u*)&in.vz[j * 32 + g * 8];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        t[n][k] = __builtin_amdgcn_exp2f(t[n][k]);   // hidden: 0
        c.l[n] += t[n][k];
        t[n][k] *= vs[k >> 2][k & 3];
      }
    if (mask & 1) {   // the scale of a hidden value may be NaN
      keep_branch();
      hide(0.0f);
    }
    write_words(next);
    v8b p[2][NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) p[0][n] = weights_to_bf16(&t[n][0]);
    issue_fence();
    // the second product, and between its instructions the conversion of the next tile
    // (behind the last one nobody reads it)
#pragma unroll
    for (int f = 0; f < 4 * NS; ++f) {
      const int j = f / ND, d = f % ND;
      read(4 * NS + f + kRing - 1);
#pragma unroll
      for (int n = 0; n < NT; ++n) c.o[n][d] = mfma(as_bf16(ring[f % kRing]), p[j][n], c.o[n][d]);
      if (f % 2 == 0 && f / 2 < kPieces) write_piece(next, f / 2);
      if (f == 1)
#pragma unroll
        for (int n = 0; n < NT; ++n) p[1][n] = weights_to_bf16(&t[n][8]);
      if (d == ND - 1)
#pragma unroll
        for (int n = 0; n < NT; ++n) c.oz[n] = mfma(as_bf16(z[j]), p[j][n], c.oz[n]);
      issue_fence();
    }
#pragma unroll
    for (int i = 2 * NS; i < kPieces; ++i) write_piece(next, i);
  };

  if (kt.begin < kt.end) {
    look_up(kt.begin);
    load(kt.begin);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) write_piece(buf[0], i);
    write_words(buf[0]);
    load(kt.begin + 1);
    lds_barrier();
  }
  for (int tile = kt.begin; tile < kt.end; ++tile) {
    const int even = (tile - kt.begin) & 1;
    const int key0 = tile * kColsTile;
    const int blocks = uniform(buf[even].there[0] | buf[even].there[1] << 1);
    const bool full = blocks == 3 && key0 >= c.all_lo && key0 + kColsTile <= c.all_hi;
    compute(buf[even], buf[even ^ 1], key0, blocks << 1 | (full ? 0 : 1));
    if ((tile - kt.begin + 1) % (kOffsetKeys / kColsTile) == 0) {
      keep_branch();
      c.take_off();
    }
    load(tile + 2);
    lds_barrier();
  }
  if (!live) return;

  const int64_t slot = (item * heads + hk) * a.splits + split;
  const Partial part = partial(a, slot, items * heads * a.splits, S::kCols, D);
  const bool whole = kt.splits == 1;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = col0 + n * 16 + cl;
    const float sum = column_sum(c.l[n]);
    if (col >= cols) continue;
    const int pc = wave * C + n * 16 + cl;
    const float f = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = out_row(a, seq, shard, head, col);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const v4f x = (c.o[n][d] - c.oz[n]) * f;
      const int f0 = d * 16 + g * 4;
      if (whole) {
        store_out2(a, at * D + f0, x[0], x[1]);
        store_out2(a, at * D + f0 + 2, x[2], x[3]);
      } else {
        *(v4f*)(part.sums + (int64_t)pc * D + f0) = x;
      }
    }
    if (g == 0) {
      if (!whole) {
        part.stats[2 * pc] = c.m2[n];
        part.stats[2 * pc + 1] = sum;
      } else if (a.lse) {
        a.lse[at] = lse_of(c.m2[n], sum);
      }
    }
  }
}

// Adds the splits of an item's columns, in their order.
template <int D, int NT>
__global__ __launch_bounds__(256) void attention_splits_kernel(AttnArgs a, uint32_t first_item,
                                                               uint32_t items) {
  using S = ColsShape<D, NT>;
  const int head = blockIdx.x;
  const int64_t shard = blockIdx.y, heads = a.kv.P * a.kv.Hk, item = first_item + blockIdx.z;
  const int64_t id = item * heads + shard * a.kv.Hk + head;
  int64_t sub;
  SeqRange seq;
  const int b = find_sequence(a.kv, a.G, S::kShift, part_extra(a.G, S::kShift), item, &sub, &seq);
  if (b < 0) return;
  const int cols = seq.n * a.G;
  if ((sub << S::kShift) >= cols) return;
  const int block_col = (int)sub << S::kShift;
  int klo, khi;
  keys_seen(a, seq, block_col, min(block_col + S::kCols, cols), &klo, &khi);
  const KeyTiles kt = key_tiles(klo, khi, 0, a.splits);
  if (kt.splits == 1) return;
  auto part = [&](int s) {
    return partial(a, id * a.splits + s, items * heads * a.splits, S::kCols, D);
  };
  const int live = min(S::kCols, cols - block_col);
  for (int i = threadIdx.x; i < live * (D / 4); i += 256) {
    const int c = i / (D / 4), d = (i - c * (D / 4)) * 4;
    float m = kNegInf;
    for (int s = 0; s < kt.splits; ++s) m = fmaxf(m, part(s).stats[2 * c]);
    float sum = 0.0f;
    v4f x = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < kt.splits; ++s) {
      const Partial p = part(s);
      const float l = p.stats[2 * c + 1], f = share(p.stats[2 * c], l, m);
      sum += l * f;
      x += *(const v4f*)(p.sums + (int64_t)c * D + d) * f;
    }
    const int64_t at = out_row(a, seq, shard, head, block_col + c);
    const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
    store_out2(a, at * D + d, x[0] * r, x[1] * r);
    store_out2(a, at * D + d + 2, x[2] * r, x[3] * r);
    if (a.lse && d == 0) a.lse[at] = lse_of(m, sum);
  }
}

// Calls f(first, n) for items in launches of as many as a grid's third axis holds.
template <typename F>
hipError_t each_launch(int64_t items, F f) {
  for (int64_t i = 0; i < items; i += 65535) f((uint32_t)i, (unsigned)(items - i < 65535 ? items - i : 65535));
  return hipGetLastError();
}

// 4 waves a block: a SIMD that has one wave is kept busy by its instructions (some 2 us a
// tile of 128 keys at D = 128), so 8 of them, us against 4, take 26 against 27 for 128
// groups of 4000 keys, but 22 against 20 for 256 of 2000 and 37 against 31 for 512.
template <int D, int W>
hipError_t launch_keys(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
  return each_launch(plan.items, [&](uint32_t first, unsigned n) {
    attention_keys_kernel<D, W, 4, false><<<dim3(a.kv.Hk, (unsigned)a.kv.P, n), 256, 0, s>>>(a, first);
  });
}
template <int D>
hipError_t launch_stream(const AttnArgs& a, hipStream_t s) {
  // 8 waves a block as far as their registers go: fewer, longer shares leave less to join
  constexpr int kTeam = D <= 128 ? 8 : 4;
  attention_keys_kernel<D, 16, kTeam, true><<<dim3(kStreamBlocks), 64 * kTeam, 0, s>>>(a, 0);
  attention_join_kernel<D><<<dim3(kStreamBlocks, 4), kJoinThreads, 0, s>>>(a);
  return hipGetLastError();
}
template <int D>
hipError_t launch_columns(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
  constexpr int NT = D <= 128 ? 2 : 1;
  const uint32_t items = (uint32_t)plan.items;
  const hipError_t e = each_launch(plan.items * plan.splits, [&](uint32_t first, unsigned n) {
    attention_columns_kernel<D, NT><<<dim3(a.kv.Hk, (unsigned)a.kv.P, n), 256, 0, s>>>(a, first, items);
  });
  if (e != hipSuccess || plan.splits == 1) return e;
  return each_launch(plan.items, [&](uint32_t first, unsigned n) {
    attention_splits_kernel<D, NT><<<dim3(a.kv.Hk, (unsigned)a.kv.P, n), 256, 0, s>>>(a, first, items);
  });
}

template <int D>
hipError_t launch_head(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
  switch (plan.kind) {
    case kAttnKeys:
      if constexpr (D <= 128)
        if (plan.columns == 8) return launch_keys<D, 8>(a, plan, s);
      return launch_keys<D, 16>(a, plan, s);
    case kAttnStream: return launch_stream<D>(a, s);
    default: return launch_columns<D>(a, plan, s);
  }
}

}  // namespace

AttnPlan attn_plan(int64_t P, int64_t T, int Hq, int Hk, int D, int B, int64_t max_length) {
  AttnPlan p = {};
  const int G = Hq / Hk;
  const int64_t heads = P * Hk, columns = T * G;
  p.splits = 1;
  // Columns of a sequence, on average, up to which the keys' kernels are faster. D = 128, 8
  // heads on one, P = 8, us by keys against by columns: 64 sequences of 3000 keys with 96
  // columns each 155 against 182, with 128 204 against 195, with 192 302 against 287; one
  // of 16000 with 128 columns 39 against 154. Over short contexts the groups' beginnings
  // weigh more: 64 of 300 keys with 64 columns 36 against 40, with 96 49 against 42.
  // With one head on one the same limits hold (3000 keys, 128 columns: 203 against 249, 192:
  // 300 against 298; 300 keys, 64: 36 against 41, 96: 51 against 44), at D = 64 the long one is
  // low (192: 194 against 230) and at D = 256 the short one high (64: 93 against 66; long, 128:
  // 535 against 540).
  const int64_t few = max_length > 512 ? 128 : 64;
  if (columns <= few * B) {
    p.items = (columns + (int64_t)B * part_extra(G, 4)) / 16;
    // groups of columns that exist, as far as the host knows: each row has one at least
    const int64_t rows = T < B ? T : B;
    const int64_t units = (rows > columns / 16 ? rows : columns / 16) * heads;
    // A block takes a group of columns whole where that leaves none much longer than an
    // equal share of a full chip, which costs a second launch and a beginning for every
    // cut. D = 128, us whole against in shares: 128 groups of 2000 keys 15 against 18, of
    // up to 4000 24 against 31, 256 of 4000 29 against 34, of up to 6000 37 against 36,
    // 512 of up to 8000 73 against 67; 64 groups of 4000 26 against 21. (Other D: not measured.)
    const int64_t longest = units >= 128 ? 4096 : 2048;
    if (max_length <= longest || units >= 4096) {
      p.kind = kAttnKeys;
      // (in equal shares with D = 128 they take all 256 registers: one sequence of 131071
      // keys 37.4 us, 36.0 with 16 columns)
      if (D <= 128 && columns <= (int64_t)8 * B) {
        p.columns = 8;
        p.items = (columns + (int64_t)B * part_extra(G, 3)) / 8;
      }
    } else {
      p.kind = kAttnStream;
      // some 5 us, or 12 tiles of 8 waves; with fewer groups than that a block has one
      // beginning or two, all alike
      p.begin = units <= kStreamBlocks / 2 ? 0 : 12;
      p.workspace = (size_t)(2 * kStreamBlocks * 16) * (D + 2) * 4 + kStreamBlocks * sizeof(Cut);
    }
    return p;
  }
  p.kind = kAttnColumns;
  const int64_t cols = D <= 128 ? 128 : 64;
  p.items = (columns + (int64_t)B * part_extra(G, D <= 128 ? 7 : 6)) / cols;
  // blocks that fill the chip
  const int64_t units = (columns + cols - 1) / cols * heads;
  const int64_t most = (max_length + kColsTile * kMinTiles - 1) / (kColsTile * kMinTiles);
  int64_t want = (512 + units - 1) / units;
  if (want > most) want = most;
  if (want > 1) {
    p.splits = (int)want;
    p.workspace = (size_t)(p.items * heads * want * cols) * (D + 2) * 4;
  }
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
