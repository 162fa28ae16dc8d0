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

}  // namespace btq
