// btq_int8_matmul: products of 8-bit codes on the matrix cores, int32 sums,
// scaled by token and output channel.
//
// Every kernel feeds the weights as the matrix instruction's first operand
// and the activations as its second. The result then holds, in each lane, one
// token and runs of 4 consecutive output channels, which store as vectors.
// The order of k inside an instruction does not matter (integer sums are
// exact), as long as both operands take it alike.
#include <type_traits>

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

// y = sum * a_scale * w_scale + bias (0 without one), each step one fp32
// operation.
__device__ __forceinline__ float scaled(int sum, float sa, float sw, float b) {
  return (float)sum * sa * sw + b;
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
                                 g.bias ? g.bias[p * g.N + n] : 0.0f);
          if (g.y_type == kBf16)
            ((uint16_t*)g.y)[out + n] = (uint16_t)f32_to_bf16(v);
          else
            ((float*)g.y)[out + n] = v;
        }
      }
    }
  }
}

// ---- results of a block, written through buffer descriptors: what lies past
// the last token or channel is dropped, and its scales load as 0 ----
typedef float v4f __attribute__((ext_vector_type(4)));

struct OutTile {
  rsrc_t y;                 // from the block's first token and channel
  const float *sw, *bias;   // LDS: the block's channels
  int cols;                 // channels of the block that exist
};

template <bool kBf>
__device__ __forceinline__ rsrc_t out_rsrc(const MatmulArgs& g, int64_t p, int64_t t0, int64_t n0,
                                           int rows, int cols) {
  constexpr int sz = kBf ? 2 : 4;
  return make_rsrc((char*)g.y + ((p * g.T + t0) * g.N + n0) * sz,
                   (uint32_t)((rows - 1) * (int)g.N + cols) * sz);
}

// A block's scales and biases to LDS, where the epilogue reads them without
// waiting for its own stores (vector loads and stores retire in one order).
__device__ __forceinline__ void stage_scales(const MatmulArgs& g, int64_t p, int64_t t0,
                                             int64_t n0, int rows, int cols, int rt, int rn,
                                             float* sa, float* sw, float* bias) {
  for (int i = threadIdx.x; i < rt; i += blockDim.x)
    sa[i] = i < rows ? g.a_scale[p * g.as_shard + t0 + i] : 0.0f;
  for (int i = threadIdx.x; i < rn; i += blockDim.x) {
    sw[i] = i < cols ? g.w_scale[p * g.N + n0 + i] : 0.0f;
    bias[i] = g.bias && i < cols ? g.bias[p * g.N + n0 + i] : 0.0f;
  }
}

// 32 tokens x 32*MN channels of one wave: scaled, rounded, turned in LDS and
// stored by rows. A product's lane l holds the token l%32 and, in acc[4g + j],
// channel 8g + 4(l/32) + j: stored as they are, rows would go out in pieces of
// 16 bytes. Through LDS (the wave's own `turn`, rows padded by 16 bytes, so
// that the writes, 32 rows at a time, spread over the banks) a store covers
// runs of 64*MN bytes of bf16.
// t, n: the first token and channel within the block; rows, cols: those of the
// block that exist. kVec: N is a multiple of 8 and y of 16 bytes.
template <int MN, bool kBf>
constexpr int kTurnRow = 32 * MN * (kBf ? 2 : 4) + 16;
template <int MN, bool kBf>
constexpr int kTurnBytes = 32 * kTurnRow<MN, kBf>;

template <int MN, bool kVec, bool kBf>
__device__ __forceinline__ void store_rows(const v16i* const (&acc)[MN], const OutTile& o,
                                           int8_t* turn, float sa, int t, int n, int rows, int N) {
  constexpr int sz = kBf ? 2 : 4, kRow = kTurnRow<MN, kBf>;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  int8_t* to = turn + (lane & 31) * kRow;
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = 32 * i + 8 * g + 4 * h;
      const v4f w = *(const v4f*)(o.sw + n + c), b = *(const v4f*)(o.bias + n + c);
      v4f f;
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = scaled((*acc[i])[4 * g + j], sa, w[j], b[j]);
      if constexpr (kBf) {
        typedef uint32_t v2u __attribute__((ext_vector_type(2)));
        *(v2u*)(to + c * 2) = v2u{f32_to_bf16x2(f[0], f[1]), f32_to_bf16x2(f[2], f[3])};
      } else {
        *(v4f*)(to + c * 4) = f;
      }
    }
  wave_lds_sync();
  if constexpr (kVec) {
    constexpr int kLanes = 32 * MN * sz / 16;   // that share a row
    constexpr int kPass = 64 / kLanes;          // rows a pass
    const int c = lane % kLanes * (16 / sz);
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += kPass) {
      const int r = r0 + lane / kLanes;
      const v4i v = *(const v4i*)(turn + r * kRow + c * sz);
      const bool ok = t + r < rows && n + c < o.cols;
      __builtin_amdgcn_raw_buffer_store_b128(
          v, o.y, ok ? (uint32_t)((t + r) * N + n + c) * (uint32_t)sz : kOOB, 0, 0);
    }
  } else {
    constexpr int kCols = MN < 2 ? 32 : 64;   // a pass: 64 columns of a row, or 32 of two
#pragma unroll 4
    for (int e = 0; e < 32 * 32 * MN; e += 64) {
      const int at = e + lane, r = at / kCols / (32 * MN / kCols),
                c = at % kCols + at / kCols % (32 * MN / kCols) * kCols;
      const bool ok = t + r < rows && n + c < o.cols;
      const uint32_t off = ok ? (uint32_t)((t + r) * N + n + c) * (uint32_t)sz : kOOB;
      if constexpr (kBf)
        __builtin_amdgcn_raw_buffer_store_b16(*(const uint16_t*)(turn + r * kRow + c * sz), o.y,
                                              off, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b32(*(const uint32_t*)(turn + r * kRow + c * sz), o.y,
                                              off, 0, 0);
    }
  }
  wave_lds_sync();
}

// ---- tile kernel: K a multiple of 16, rows on 16-byte boundaries ----
//
// A block of 4 waves (2x2) makes 64*MN channels x 64*MT tokens; a wave
// 32*MN x 32*MT in 32x32x32 products. k goes in steps of 128 bytes, two steps
// in LDS: one is read while the next one lands by direct loads to LDS. In LDS
// a row's eight 16-byte chunks are permuted by c ^ (row & 7) (the loads
// permute their addresses: a direct load writes its lanes in a line), so the
// 8 rows that one LDS cycle serves lie in different banks.
// A step is 4 slices of 32 bytes. The next slice's operands are read while
// the matrix cores run the present one. The barrier stands before the last
// slice: its operands are in registers by then, so the buffer is free for the
// step after the next, and its products hide the first reads of the next step.
constexpr int kStep = 128;

// 16 bytes a lane from rsrc[off + soff] straight to LDS: lane i of the wave to
// byte to + 16*i. `to`, an LDS address, is the same in all lanes. Written as
// assembly because the compiler, which cannot tell the two steps' buffers
// apart, would wait for these loads before every later LDS read; the kernel
// orders them itself, with wait_loads and a barrier before the first read.
__device__ __forceinline__ void load_to_lds(rsrc_t r, uint32_t to, uint32_t off, uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(to), "v"(off), "s"(r), "s"(soff)
      : "m0", "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Waits until at most kLoads of this wave's vector loads are in flight (and,
// for kLds, none of its LDS reads).
template <int kLoads, bool kLds>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((kLoads & 15) | (kLoads >> 4) << 14 | 7 << 4 | (kLds ? 0 : 15) << 8);
}

template <int MN, int MT, bool kVec, bool kBf>
__global__ __launch_bounds__(256, MN* MT == 16 ? 1 : 2) void matmul_tile_kernel(
    MatmulArgs g, int tiles_t, int tiles_n, int tiles) {
  constexpr int RN = 64 * MN, RT = 64 * MT, kLoads = 2 * MN + 2 * MT;
  constexpr int kStage = (RN + RT) * kStep;
  __shared__ __align__(1024) int8_t lds[2 * kStage];
  __shared__ __align__(16) float l_sa[RT], l_sw[RN], l_bias[RN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = (wave >> 1) * 32 * MN, wt = (wave & 1) * 32 * MT;

  // Each XCD takes one run of tiles, and walks it 4 tiles of channels by many
  // of tokens, so the blocks that run together share operands in its L2.
  int tile;
  {
    const int b = blockIdx.x, xcd = b % kXcds, slot = b / kXcds;
    const int each = tiles / kXcds, more = tiles % kXcds;
    tile = xcd * each + min(xcd, more) + slot;
  }
  const int per_p = tiles_t * tiles_n;
  const int p = tile / per_p;
  int in = tile % per_p;
  const int group = in / (4 * tiles_t);
  in -= group * 4 * tiles_t;
  const int height = min(4, tiles_n - group * 4);
  const int64_t n0 = (int64_t)(group * 4 + in % height) * RN;
  const int64_t t0 = (int64_t)(in / height) * RT;

  const int nrows = (int)min((int64_t)RN, g.N - n0), trows = (int)min((int64_t)RT, g.T - t0);
  const int K = (int)g.K, pitch = (int)g.a_pitch;
  const rsrc_t rw = make_rsrc(g.w + (p * g.N + n0) * g.K, (uint32_t)(nrows * K));
  const rsrc_t ra = make_rsrc(g.a + p * g.a_shard + t0 * g.a_pitch,
                              (uint32_t)((trows - 1) * pitch + K));
  const int lrow = tid >> 3, chunk = ((tid & 7) ^ (lrow >> 1 & 7)) * 16;
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < 2 * MN; ++i)
    off[i] = (uint32_t)(min(lrow + 32 * i, nrows - 1) * K + chunk);
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i)
    off[2 * MN + i] = (uint32_t)(min(lrow + 32 * i, trows - 1) * pitch + chunk);

  const int steps = (K + kStep - 1) / kStep;
  const uint32_t to = lds_address(lds) + wave * 1024;
  // load i of a step
  auto fetch = [&](int step, int i) {
    const bool in_row = step * kStep + chunk < K;
    load_to_lds(i < 2 * MN ? rw : ra, to + (step & 1) * kStage + i * 32 * kStep,
                in_row ? off[i] : kOOB, step * kStep);
  };
  v4i fw[2][MN], fa[2][MT];
  const int frow = (lane & 31) * kStep;
  // operand i of a slice
  auto read = [&](int step, int slice, int i) {
    const int pos = ((2 * slice + (lane >> 5)) ^ (lane >> 1 & 7)) * 16;
    const int8_t* from = lds + (step & 1) * kStage + frow + pos;
    if (i < MN)
      fw[slice & 1][i] = *(const v4i*)(from + (wn + 32 * i) * kStep);
    else
      fa[slice & 1][i - MN] = *(const v4i*)(from + (RN + wt + 32 * (i - MN)) * kStep);
  };
  v16i acc[MN][MT] = {};
  // The products of a slice, in turn with the reads of the slice after it and
  // loads d0..d1 of step `ds`. The fences keep this order.
  auto slice = [&](int set, auto has_read, int rstep, int rslice, auto has_load, int ds, int d0,
                   int d1) {
    constexpr int kM = MN * MT, kR = MN + MT;
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      acc[m / MT][m % MT] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
          fw[set][m / MT], fa[set][m % MT], acc[m / MT][m % MT], 0, 0, 0);
      if constexpr (decltype(has_read)::value) {
#pragma unroll
        for (int r = 0; r < kR; ++r)
          if (r * kM / kR / 2 == m || (r * kM / kR / 2 >= kM && m == kM - 1))
            read(rstep, rslice, r);
      }
      if constexpr (decltype(has_load)::value) {
#pragma unroll
        for (int d = 0; d < kLoads; ++d)
          if (d >= d0 && d < d1 && (d - d0) * kM / (d1 - d0) == m) fetch(ds, d);
      }
      issue_fence();
    }
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  constexpr int kEarly = kLoads / 2;   // loads that go out right after the barrier
  // One step; next, next2: the steps after it exist.
  auto body = [&](int step, auto next, auto next2) {
    slice(0, yes, step, 1, next, step + 1, kEarly, kLoads);
    slice(1, yes, step, 2, no, 0, 0, 1);
    slice(0, yes, step, 3, no, 0, 0, 1);
    if constexpr (decltype(next)::value) {
      wait_loads<0, true>();
      __builtin_amdgcn_s_barrier();
      issue_fence();
    }
    slice(1, next, step + 1, 0, next2, step + 2, 0, kEarly);
  };

#pragma unroll
  for (int i = 0; i < kLoads; ++i) fetch(0, i);
  stage_scales(g, p, t0, n0, trows, nrows, RT, RN, l_sa, l_sw, l_bias);
  wait_loads<0, true>();
  __builtin_amdgcn_s_barrier();
  issue_fence();
  if (steps > 1) {
#pragma unroll
    for (int i = 0; i < kEarly; ++i) fetch(1, i);
  }
#pragma unroll
  for (int i = 0; i < MN + MT; ++i) read(0, 0, i);
  int step = 0;
  for (; step + 2 < steps; ++step) body(step, yes, yes);
  if (step + 1 < steps) body(step++, yes, no);
  body(step, no, no);

  lds_barrier();   // the other waves are done with the operands
  const OutTile o = {out_rsrc<kBf>(g, p, t0, n0, trows, nrows), l_sw, l_bias, nrows};
  static_assert(4 * kTurnBytes<MN, kBf> <= 2 * kStage, "the turn fits the operands' LDS");
  int8_t* turn = lds + wave * kTurnBytes<MN, kBf>;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const v16i* part[MN];
#pragma unroll
    for (int i = 0; i < MN; ++i) part[i] = &acc[i][j];
    store_rows<MN, kVec, kBf>(part, o, turn, l_sa[wt + 32 * j + (lane & 31)], wt + 32 * j, wn,
                              trows, (int)g.N);
  }
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;

template <int MN, int MT>
hipError_t launch_tiles(const MatmulArgs& a, hipStream_t s) {
  const int64_t tt = (a.T + 64 * MT - 1) / (64 * MT), tn = (a.N + 64 * MN - 1) / (64 * MN);
  const dim3 grid((unsigned)(a.P * tt * tn));
  const bool bf = a.y_type == kBf16, vec = a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0;
  const int itt = (int)tt, itn = (int)tn, n = (int)(a.P * tt * tn);
  if (vec && bf)
    matmul_tile_kernel<MN, MT, true, true><<<grid, 256, 0, s>>>(a, itt, itn, n);
  else if (vec)
    matmul_tile_kernel<MN, MT, true, false><<<grid, 256, 0, s>>>(a, itt, itn, n);
  else if (bf)
    matmul_tile_kernel<MN, MT, false, true><<<grid, 256, 0, s>>>(a, itt, itn, n);
  else
    matmul_tile_kernel<MN, MT, false, false><<<grid, 256, 0, s>>>(a, itt, itn, n);
  return hipGetLastError();
}

// Direct 16-byte loads need every row on a 16-byte boundary; a block's rows of
// a, w and y must each span less than 2^31 bytes.
bool rows_aligned(const MatmulArgs& a) {
  return a.K % 16 == 0 && a.a_pitch % 16 == 0 && a.a_shard % 16 == 0 &&
         ((uintptr_t)a.a & 15) == 0 && ((uintptr_t)a.w & 15) == 0 &&
         a.a_pitch < (int64_t(1) << 22) && a.N < (int64_t(1) << 20);
}

}  // namespace

hipError_t launch_int8_matmul(const MatmulArgs& a, hipStream_t s) {
  const int64_t t128 = (a.T + 127) / 128, n128 = (a.N + 127) / 128;
  if (rows_aligned(a) && a.P * t128 * n128 <= kMaxBlocks) {
    if (a.P * ((t128 + 1) / 2) * ((n128 + 1) / 2) >= 256) return launch_tiles<4, 4>(a, s);
    return launch_tiles<2, 2>(a, s);
  }
  const int64_t tt = (a.T + kGenTile - 1) / kGenTile, tn = (a.N + kGenTile - 1) / kGenTile;
  const int64_t tiles = a.P * tt * tn;
  matmul_general_kernel<<<dim3((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks)), 256, 0, s>>>(
      a, tt, tn, tiles);
  return hipGetLastError();
}

}  // namespace btq
