// Internal helpers shared by the libbtq kernels (gfx950, wave64).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace btq {

constexpr int kWave = 64;

// bf16 bit pattern -> fp32 (exact: the bf16 bits are the high half).
__device__ __forceinline__ float bf16_to_f32(uint32_t bits16) {
  return __uint_as_float(bits16 << 16);
}

// Orders LDS traffic between the lanes of one wavefront. The waves of a
// block work on separate LDS regions and never wait for each other, so a
// block-wide barrier is not needed. The fences keep the compiler from moving
// LDS accesses across this point. The hardware runs one wave's LDS
// instructions in issue order.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Block barrier that orders LDS only. __syncthreads() also orders global
// memory, which makes every wave wait for all of its loads in flight
// (vmcnt(0)) before the barrier, also where only LDS needs ordering.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Keeps the scheduler from moving instructions across this point. The fast
// kernels issue their setup loads first and their token-row loads second: the
// vector-memory counter retires in issue order, so a wait for a setup load
// then never includes the row loads behind it.
__device__ __forceinline__ void issue_fence() { __builtin_amdgcn_sched_barrier(0); }

// Marks a register as redefined here (an empty asm that reads and writes it).
// The fast kernels apply it to the per-lane constants that come straight from
// setup loads, once, before their main loop: the completion wait then happens
// there, and the loop body never has to wait for a setup load again.
template <typename V>
__device__ __forceinline__ void settle(V& v) {
  asm volatile("" : "+v"(v));
}

// Hides a value's origin from the optimizer (an empty asm that reads and
// writes it, with no side effects), so it cannot rewrite the computation of
// the value's uses in terms of that origin.
template <typename V>
__device__ __forceinline__ void opaque(V& v) {
  asm("" : "+v"(v));
}

// Raw buffer resources (gfx9 format). A wave builds a descriptor over the
// part of a tensor it touches, so every offset stays 32-bit. The hardware
// range check then handles ragged edges: a load at or past num_records
// returns 0, and a store there is dropped. Lanes that have nothing to do
// point their offset at kOOB instead of branching. That keeps the memory
// instructions out of divergent control flow, where the compiler has to
// wait for all loads in flight at every join. Every descriptor this library
// builds spans fewer than 2^31 bytes, so any offset >= kOOB is out of range.
using rsrc_t = __amdgpu_buffer_rsrc_t;
constexpr int kRsrcWord3 = 0x00020000;   // dword3: 32-bit data format, raw (no swizzle)
constexpr uint32_t kOOB = 0x80000000u;

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           kRsrcWord3);
}

// Cache policy for streaming (read-once / write-once) buffer accesses:
// the non-temporal hint (bit 1 of the gfx94x/gfx950 cache-policy operand).
constexpr int kStream = 2;

// XCD-aware block order. MI355X deals workgroups round-robin over its 8
// XCDs, and each XCD has its own L2. A unit is a group of `per_unit`
// consecutive logical blocks whose writes share cache lines: all tiles of
// one block of token rows. This mapping runs a whole unit on one XCD, so the
// partial lines its blocks write merge in one L2 before they reach HBM.
// Returns false for the padding blocks of the last round.
constexpr int kXcds = 8;
__device__ __forceinline__ bool xcd_unit_block(int64_t b, int64_t per_unit, int64_t units,
                                               int64_t* unit, int64_t* sub) {
  const int64_t xcd = b % kXcds;
  const int64_t slot = b / kXcds;
  *unit = (slot / per_unit) * kXcds + xcd;
  *sub = slot % per_unit;
  return *unit < units;
}
__host__ __forceinline__ int64_t xcd_grid(int64_t per_unit, int64_t units) {
  return (units + kXcds - 1) / kXcds * kXcds * per_unit;
}

// Geometry of one wave-tile of the int4 slot axis. A tile owns the slots
// [jstart, jend), 8 per lane, so that no two tiles share a packed byte. It
// also owns every feature h in [hs, he): its int4 features plus the BF16
// features that fall between them. Tile 0 starts at h = 0 and the last
// tile ends at h = H.
constexpr int kLaneSlots = 8;                    // slots per lane = one packed dword
constexpr int kTileSlots = kWave * kLaneSlots;   // 512 slots per wave-tile

struct TileGeom {
  int jstart, jend;   // slot range
  int hs, he;         // feature range
  int ilo, nout;      // BF16 features idx[ilo .. ilo+nout) lie in [hs, he)
};

__device__ __forceinline__ TileGeom tile_geom(const int32_t* __restrict__ cmap, int c,
                                              int ntiles, int Hq, int H) {
  TileGeom g;
  g.jstart = c * kTileSlots;
  g.jend = min(Hq, g.jstart + kTileSlots);
  g.hs = (c == 0) ? 0 : cmap[g.jstart];
  g.he = (c == ntiles - 1) ? H : cmap[g.jend];
  // h0 has exactly h0 - j0 BF16 features below it when cmap[j0] = h0
  g.ilo = g.hs - g.jstart;
  g.nout = (g.he - g.jend) - g.ilo;
  return g;
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, 0xf, 0xf, true);
}

// x combined over the 64 lanes, in all of them: neighbours in 4, halves of 8,
// halves of 16, then rows of 16 and halves of the wave by swaps. A few cycles a
// step, where a shuffle through LDS takes over a hundred.
template <typename F>
__device__ __forceinline__ uint32_t wave_combine(uint32_t x, F f) {
  x = f(x, dpp<0xb1>(x));    // quad_perm 1,0,3,2
  x = f(x, dpp<0x4e>(x));    // quad_perm 2,3,0,1
  x = f(x, dpp<0x141>(x));   // row_half_mirror
  x = f(x, dpp<0x140>(x));   // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return f(b[0], b[1]);
}

// ---- values of the calls around the codec ----
enum ValueType { kF32 = 0, kBf16 = 1, kInt8 = 2 };   // btq_type

// fp32 -> bf16 bits, round to nearest even; NaN stays NaN (made quiet).
__device__ __forceinline__ uint32_t f32_to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  const uint32_t r = (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
  return (u & 0x7fffffffu) > 0x7f800000u ? (u >> 16) | 0x40u : r;
}

// Two at once (v_cvt_pk_bf16_f32): `lo` in the low half.
__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 v = __builtin_convertvector((f2{lo, hi}), b2);
  return __builtin_bit_cast(uint32_t, v);
}

// The 8-bit scale of a row from the largest |x| of the row as fp32 bits
// (bits order as values do, and Inf and NaN come above every finite value).
// code = rint(x*mul). mul is 127/m raised by 2^-21 of itself: that outweighs
// the three roundings of x*mul (each at most 2^-24), so an exact tie lands
// above the half and rounds away from zero. For bf16 x no other value comes
// that near to a tie: x*127/m = 127*mx/(ma*2^j) with mx, ma < 256 differs
// from (2n+1)/2 by 0 or by at least 1/(254*255) of itself.
struct RowScale {
  float scale, mul;
};
__device__ __forceinline__ RowScale row_scale(uint32_t absmax_bits) {
  const float m = __uint_as_float(absmax_bits);
  RowScale r;
  r.scale = m / 127.0f;
  r.mul = 127.0f / m * (1.0f + 0x1p-21f);
  if (absmax_bits >= 0x7f800000u) {
    r.scale = __uint_as_float(0x7fc00000u);
    r.mul = 0.0f;
  } else if (r.scale < 0x1p-126f) {
    r.scale = 1.0f;
    r.mul = 0.0f;
  }
  return r;
}

// The code in the low byte: adding 1.5*2^23 leaves the rounded integer, in
// two's complement, in the low mantissa bits. A row with mul 0 may hold Inf
// or NaN; its codes are 0 whatever x is.
__device__ __forceinline__ uint32_t code_bits(float x, float mul) {
  const uint32_t b = __float_as_uint(__builtin_fmaf(x, mul, 12582912.0f));
  return mul == 0.0f ? 0u : b & 0xffu;
}

// ---- host-side launchers (one per kernel family), called by abi.hip ----
struct CalibPlan {
  int64_t nchunk;          // token-axis chunks reduced in parallel
  int64_t rows_per_chunk;
};
CalibPlan calib_plan(int64_t P, int64_t T, int64_t H);
// The same plan with at most as many chunks as fit max_ws_floats floats of
// partials (nchunk 0: not even one chunk fits).
CalibPlan calib_plan_capped(int64_t P, int64_t T, int64_t H, int64_t max_ws_floats);
hipError_t launch_calib(const uint16_t* x, int64_t P, int64_t T, int64_t H, float a, float c,
                        int first, float* run_min, float* run_max, float* ws, hipStream_t s);
// ws holds 2*plan.nchunk*P*H floats.
hipError_t launch_calib_plan(const uint16_t* x, int64_t P, int64_t T, int64_t H, float a, float c,
                             int first, float* run_min, float* run_max, float* ws,
                             const CalibPlan& plan, hipStream_t s);

hipError_t launch_select(const float* run_min, const float* run_max, int64_t P, int64_t H,
                         int64_t k, float* scale, float* rscale, uint8_t* zp, int32_t* idx,
                         int32_t* fmap, int32_t* cmap, float* ws_score, bool score_max,
                         hipStream_t s);
// One BF16 set per shard: idx [P,k], fmap [P,H], cmap [P,H-k]; ws_width
// holds P*H floats.
hipError_t launch_select_per_shard(const float* run_min, const float* run_max, int64_t P,
                                   int64_t H, int64_t k, float* scale, float* rscale, uint8_t* zp,
                                   int32_t* idx, int32_t* fmap, int32_t* cmap, float* ws_width,
                                   hipStream_t s);
// The same outputs for a given BF16 set: idx is a device copy of k distinct
// features in ascending order.
hipError_t launch_select_set(const float* run_min, const float* run_max, int64_t P, int64_t H,
                             int64_t k, float* scale, float* rscale, uint8_t* zp,
                             const int32_t* idx, int32_t* fmap, int32_t* cmap, hipStream_t s);

// rscale [P,H], zp [P,H]; per_shard: idx [P,k] and cmap [P,H-k] hold one
// set per shard, else idx [k] and cmap [H-k].
hipError_t launch_compress(const uint16_t* x, int64_t P, int64_t T, int64_t H, int64_t k,
                           const float* rscale, const uint8_t* zp, const int32_t* idx,
                           const int32_t* cmap, uint8_t* packed, int64_t pitch, uint16_t* outl,
                           bool per_shard, hipStream_t s);

// scale [P,H], zp [P,H]; fmap [P,H] when per_shard, else [H]. y is fp32,
// or bf16 bits when bf16.
hipError_t launch_decompress(const uint8_t* packed, int64_t pitch, const uint16_t* outl, int64_t P,
                             int64_t T, int64_t H, int64_t k, const float* scale,
                             const uint8_t* zp, const int32_t* fmap, bool per_shard, void* y,
                             bool bf16, hipStream_t s);

// Per-row 8-bit codes: x fp32 or bf16 [P,T,K] with row strides in elements,
// q [P,T,q_pitch] (bytes past K are not written), scale [P,T].
hipError_t launch_quantize_rows(const void* x, int x_type, int64_t x_shard, int64_t x_pitch,
                                int64_t P, int64_t T, int64_t K, int8_t* q, int64_t q_pitch,
                                float* scale, hipStream_t s);

struct MatmulArgs {
  const int8_t* a;
  int64_t a_shard, a_pitch;
  const float* a_scale;
  int64_t as_shard;
  const int8_t* w;          // [P,N,K]
  const float* w_scale;     // [P,N]
  const float* bias;        // [P,N] or null
  int64_t P, T, N, K;
  void* y;                  // [P,T,N]
  int y_type;
};
hipError_t launch_int8_matmul(const MatmulArgs& a, hipStream_t s);

// btq_int8_linear in one launch, for products so small that launches count.
// small_linear_ok: whether the sizes and x (bf16, row strides in elements) suit
// it; m.a and m.a_scale are not used.
bool small_linear_ok(const void* x, int x_type, int64_t x_shard, int64_t x_pitch,
                     const MatmulArgs& m);
hipError_t launch_small_linear(const void* x, int64_t x_shard, int64_t x_pitch,
                               const MatmulArgs& m, hipStream_t s);

struct NormArgs {
  const void* y;            // null: no block output
  const void* residual;
  int y_type, r_type;
  int64_t T, H;
  int post, pre;            // btq_norm
  const float *post_weight, *post_bias, *pre_weight, *pre_bias;
  float post_eps, pre_eps;
  const void* gate;         // null: 1
  int gate_type;
  int64_t gate_each;        // tokens that share one gate row
  float alpha;
  void* residual_out;
  void* n;
  int n_type;
  float* n_scale;
};
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);

// Rows of heads: head h of token t of shard p starts at element
// p*shard + t*pitch + h*head, its D features are contiguous.
struct HeadRows {
  void* p;
  int type;
  int64_t shard, pitch, head;
};
struct RopeArgs {
  const float *cos, *sin;   // [rows, dim/2]; null: no rotation
  int64_t rows;
  int dim, style;           // btq_rope
};
// Whether the tables have a row for a position. cos and sin of one that they have not
// are NaN, so that nothing computed from it passes for a result.
__device__ __forceinline__ bool in_table(const RopeArgs& r, int64_t pos) {
  return pos >= 0 && pos < r.rows;
}

struct HeadArgs {
  HeadRows x, y;
  int64_t P, T;
  int Hq, Hk, D;
  int norm;                 // btq_norm
  const float *q_weight, *k_weight;
  int64_t qw_shard, qw_head, kw_shard, kw_head;
  float eps;
  const int32_t* positions;
  RopeArgs rope;
};
// Every head starts on 16 bytes.
inline bool on16(const HeadRows& r) {
  const int64_t n = r.type == kF32 ? 4 : 8;
  return ((uintptr_t)r.p & 15) == 0 && r.shard % n == 0 && r.pitch % n == 0 && r.head % n == 0;
}
hipError_t launch_head_norm_rope(const HeadArgs& a, hipStream_t s);

// A batch of sequences and the paged cache that holds them.
struct KvArgs {
  int64_t P, T;
  int B, Hk, D;
  const int32_t *starts, *lengths, *table;   // [B+1], [B], [B,max_pages]
  int64_t max_pages;
  int capacity;             // max_pages * page size
  uint8_t* cache;
  int64_t pages;
  int page_shift;           // a page holds 2^page_shift blocks
};
hipError_t launch_kv_append(const HeadRows& k, const HeadRows& v, const RopeArgs& rope,
                            const KvArgs& a, hipStream_t s);
hipError_t launch_kv_gather(const HeadRows& k, const HeadRows& v, const KvArgs& a, hipStream_t s);

struct AttnArgs {
  HeadRows q;               // bf16
  bool q_on16;              // every head starts on 16 bytes
  KvArgs kv;
  int Hq, G;                // query heads, those of one key head
  uint32_t G_inverse;       // 2^32/G rounded up; of G = 1 it would not fit, and nothing reads it
  float scale2;             // scale * log2(e)
  int causal, window;       // window 0: none
  void* out;                // [P,T,Hq*D]
  int out_type;
  float* lse;               // [P,T,Hq] or null
  float* ws;
  int splits, begin;        // of the plan
};
// How a call of these sizes runs (attention.hip).
enum AttnKind { kAttnKeys, kAttnStream, kAttnColumns };
struct AttnPlan {
  AttnKind kind;
  int splits;               // kAttnColumns: of the keys
  int begin;                // kAttnStream: what a group of columns costs to begin, in tiles
  int columns;              // kAttnKeys: of a group, 8 or (0) 16
  int64_t items;            // groups of columns of one head that are set aside
  size_t workspace;
};
AttnPlan attn_plan(int64_t P, int64_t T, int Hq, int Hk, int D, int B, int64_t max_length);
hipError_t launch_kv_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t s);

// ---- the paged 4-bit cache: its layout, the batch's, and the search for a work
// item's sequence ----

// A block holds 32 tokens of one head: keys [32][D/2], values [D][16], then a
// word for each key and one for each value. In a byte the even feature (keys)
// or token (values) is the low nibble. The word: the scale's bf16 bits in the
// high half, those of 128 + z in the low half (exact: z is at most 15); a code c
// stands for scale*(c - z). 128 + c is what a nibble becomes when it is or-ed
// into the mantissa of bf16 128, so a kernel that multiplies by 128 + c corrects
// by the same 128 + z.
//
// Values lie transposed so that the matrix instructions of attention find 8
// tokens of a feature in one dword (and 8 features of a key, which keys hold so
// anyway): no operand goes through LDS or another lane.
constexpr int kBlockTokens = 32;
__host__ __device__ constexpr int64_t kv_block_bytes(int D) { return 32 * D + 256; }
constexpr uint32_t kZeroWord = 0x4300u;          // 128 + 0
constexpr uint32_t kNanWord = 0x7fc04300u;       // scale NaN, z 0

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return min(max(v, lo), hi); }

// The rows [begin, end) of sequence b in the batch, and its tokens in the cache
// with them. Whatever the arrays hold, rows stay in [0, T) and places below the
// table's end.
struct SeqRange {
  int begin, n;
  int length;
  __device__ __forceinline__ int first() const { return length - n; }   // place of the first row
};
__device__ __forceinline__ SeqRange cut_range(const KvArgs& a, int start, int next, int length) {
  SeqRange s;
  s.begin = clamp_int(start, 0, (int)a.T);
  s.n = clamp_int(next, s.begin, (int)a.T) - s.begin;
  s.length = clamp_int(length, 0, a.capacity);
  return s;
}
__device__ __forceinline__ SeqRange seq_range(const KvArgs& a, int b) {
  return cut_range(a, a.starts[b], a.starts[b + 1], a.lengths[b]);
}

// Values that are the same in all lanes, in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}
__device__ __forceinline__ SeqRange uniform(const SeqRange& s) {
  return {uniform(s.begin), uniform(s.n), uniform(s.length)};
}

// Work items lie sequence after sequence. An item covers 2^shift of a sequence's
// rows*mul, and b's begin at floor((begin*mul + b*extra) / 2^shift). That leaves
// each sequence as many as it needs with extra 2^shift less the largest power of 2 up to
// 2^shift that divides mul (part_extra), for parts that begin at the first row, and with
// 2*2^shift for parts that begin at a multiple of 2^shift in the sequence. The grid then
// follows from T and the number of sequences, which the host knows; of parts no item is
// without work where each sequence has one row.
__host__ __device__ inline int part_extra(int mul, int shift) {
  const int two = mul & -mul, all = 1 << shift;
  return all - (two < all ? two : all);
}
// Returns the sequence of `item` (a whole wave asks for one item) with its rows and
// length, and leaves the item's number in it; or -1. 64 sequences a step; the last
// step has loaded the rows and lengths of all it looks at, so they cost no load of
// their own after it.
__device__ __forceinline__ int find_sequence(const KvArgs& a, int mul, int shift, int extra,
                                             int64_t item, int64_t* sub, SeqRange* range) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.B;
  for (;;) {
    const int step = (hi - lo + 63) >> 6;
    const int b = lo + lane * step;
    const int at = min(b, a.B - 1);
    // (cut as cut_range does, so that items are numbered by the rows that there are)
    const int start = clamp_int(a.starts[at], 0, (int)a.T), next = a.starts[at + 1], length = a.lengths[at];
    const int64_t first = ((int64_t)start * mul + (int64_t)b * extra) >> shift;
    const int n = __popcll(__ballot(b < hi && first <= item));
    if (n == 0) return -1;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) {
      *sub = item - (((int64_t)__builtin_amdgcn_readlane(start, n - 1) * mul + (int64_t)lo * extra) >> shift);
      if (*sub < 0) return -1;   // lane n - 1 is none of those counted: starts do not ascend
      *range = cut_range(a, __builtin_amdgcn_readlane(start, n - 1),
                         __builtin_amdgcn_readlane(next, n - 1),
                         __builtin_amdgcn_readlane(length, n - 1));
      break;
    }
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Byte offset of a sequence's block in the cache, or -1 where it has no page.
__device__ __forceinline__ int64_t kv_block(const KvArgs& a, int b, int64_t shard, int head,
                                            int block) {
  const int slot = block >> a.page_shift;
  if (block < 0 || slot >= a.max_pages) return -1;
  const int page = a.table[(int64_t)b * a.max_pages + slot];
  if (page < 0 || page >= a.pages) return -1;
  const int in_page = block & ((1 << a.page_shift) - 1);
  return ((((shard * a.pages + page) * a.Hk + head) << a.page_shift) + in_page) *
         kv_block_bytes(a.D);
}

}  // namespace btq
