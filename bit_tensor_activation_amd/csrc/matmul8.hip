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
// For k below 16, rows or strides too large for 32-bit offsets, and more tiles
// than a grid holds: 64 tokens x 64 channels a block, 4 waves of 32x32, 64 bytes
// of k a step through LDS (rows padded to 80 bytes).
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

// The lane, counted anew: cheaper at a kernel's end than a register held
// through its loop.
__device__ __forceinline__ int lane_id() {
  return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
}

// 4 channels c.. of one token to its turned row.
template <bool kBf>
__device__ __forceinline__ void store_turn(int8_t* row, int c, v4i sum, float sa, v4f w, v4f b) {
  v4f f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = scaled(sum[j], sa, w[j], b[j]);
  if constexpr (kBf) {
    typedef uint32_t v2u __attribute__((ext_vector_type(2)));
    *(v2u*)(row + c * 2) = v2u{f32_to_bf16x2(f[0], f[1]), f32_to_bf16x2(f[2], f[3])};
  } else {
    *(v4f*)(row + c * 4) = f;
  }
}

// `count` turned rows from LDS to y, by kThreads threads. Stored with the
// streaming hint: y does not push the operands out of the caches (P=8 T=2048
// N=4096: K=512 71.0 -> 63.5 us; with btq_compress_pack reading y next, K=2048
// 194.5 -> 191.3 us for both).
template <int kThreads, int MN, bool kVec, bool kBf>
__device__ __forceinline__ void store_turned(int thread, int count, const int8_t* turn,
                                             const OutTile& o, int t, int n, int rows, int N) {
  constexpr int sz = kBf ? 2 : 4, kRow = kTurnRow<MN, kBf>;
  constexpr int kRun = kVec ? 16 / sz : 1;         // elements of a store
  constexpr int kStores = 32 * MN / kRun;          // of a row
  const auto put = [&](const int8_t* from, uint32_t off) {
    if constexpr (kVec)
      __builtin_amdgcn_raw_buffer_store_b128(*(const v4i*)from, o.y, off, 0, kStream);
    else if constexpr (kBf)
      __builtin_amdgcn_raw_buffer_store_b16(*(const uint16_t*)from, o.y, off, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(*(const uint32_t*)from, o.y, off, 0, 0);
  };
  if constexpr (kThreads % kStores == 0) {   // a thread keeps its columns
    constexpr int kPass = kThreads / kStores;
    const int c = thread % kStores * kRun;
    int r = thread / kStores;
    const bool in_cols = n + c < o.cols;
    uint32_t off = (uint32_t)((t + r) * N + n + c) * (uint32_t)sz;
    const int8_t* from = turn + r * kRow + c * sz;
#pragma unroll 4
    for (; r < count; r += kPass, off += (uint32_t)(kPass * N * sz), from += kPass * kRow)
      put(from, in_cols && t + r < rows ? off : kOOB);
  } else {
#pragma unroll 4
    for (int e = thread; e < count * kStores; e += kThreads) {
      const int r = e / kStores, c = e % kStores * kRun;
      const bool ok = t + r < rows && n + c < o.cols;
      put(turn + r * kRow + c * sz, ok ? (uint32_t)((t + r) * N + n + c) * (uint32_t)sz : kOOB);
    }
  }
}

template <int MN, bool kVec, bool kBf>
__device__ __forceinline__ void store_rows(const v16i* const (&acc)[MN], const OutTile& o,
                                           int8_t* turn, float sa, int t, int n, int rows, int N) {
  constexpr int kRow = kTurnRow<MN, kBf>;
  const int lane = lane_id(), h = lane >> 5;
  int8_t* to = turn + (lane & 31) * kRow;
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = 32 * i + 8 * g + 4 * h;
      const v4f w = *(const v4f*)(o.sw + n + c), b = *(const v4f*)(o.bias + n + c);
      const v16i& x = *acc[i];
      store_turn<kBf>(to, c, v4i{x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]}, sa, w, b);
    }
  wave_lds_sync();
  store_turned<64, MN, kVec, kBf>(lane, 32, turn, o, t, n, rows, N);
  wave_lds_sync();
}

// ---- tile kernel ----
//
// A block of 4 waves (WN x WT) makes RN channels x RT tokens; a wave 32*MN x
// 32*MT of them in 32x32x32 products. k goes in steps of 128 bytes, S of them in
// LDS: one is read while the others land by direct loads to LDS. In LDS a row's
// eight 16-byte chunks are permuted by c ^ (row/2 & 7) (the loads permute their
// addresses: a direct load writes its lanes in a line), so the 16 rows that one
// LDS cycle serves lie in different banks (two rows share the 64 banks; with
// c ^ (row & 7) half of the reads' cycles were conflicts).
// A step is 4 slices of 32 bytes. The next slice's operands are read while
// the matrix cores run the present one. The barrier stands before the last
// slice: its operands are in registers by then, so the buffer is free for a
// later step, and its products hide the first reads of the next step.
// Large products are bound by the chip's power: 8192^3 takes 434 us, 2.5 POPS,
// the matrix cores busy 0.71 of the cycles at 1.67 GHz; products of few tokens
// by the weights' bytes (T=64 N=8192 P=8 K=4096: 58 us, 4.9 TB/s); short sums by
// their results' bytes (T=2048 N=4096 P=8 K=256: 48 us for 134 MB).
constexpr int kStep = 128;

// kBytes (4 or 16) a lane from rsrc[off + soff] straight to LDS: lane i of the
// wave to byte to + kBytes*i. `to`, an LDS address, is the same in all lanes.
// Written as assembly because the compiler, which cannot tell the steps'
// buffers apart, would wait for these loads before every later LDS read; the
// kernel orders them itself, with wait_loads and a barrier before the first
// read. (m0 is reserved and nothing else in these kernels uses it.)
// kNt: with the streaming hint.
template <int kBytes, bool kNt = false>
__device__ __forceinline__ void load_to_lds(rsrc_t r, uint32_t to, uint32_t off, uint32_t soff) {
  static_assert(kBytes == 16 || (kBytes == 4 && !kNt));
  if constexpr (kNt)
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen nt lds"
        :
        : "s"(to), "v"(off), "s"(r), "s"(soff)
        : "memory");
  else if constexpr (kBytes == 16)
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(to), "v"(off), "s"(r), "s"(soff)
        : "memory");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %1, %2, %3 offen lds"
        :
        : "s"(to), "v"(off), "s"(r), "s"(soff)
        : "memory");
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

// A block's share of the product: RN channels x RT tokens of shard p, and the
// loads of its operands, 256 threads together, into S buffers of LDS.
// kNt: the channels' loads stream past the caches. kCodes: the block makes the
// tokens' codes and scales itself; only the channels are loaded.
template <int RN, int RT, int S, bool kNt, bool kCodes = false>
struct Block {
  static constexpr int kTokens = kCodes ? 0 : RT;   // rows of tokens in a step
  static constexpr int kLoads = (RN + kTokens) / 32, kStage = (RN + kTokens) * kStep;
  struct Lds {
    __align__(1024) int8_t operands[S * kStage];
    // whole loads of 64
    __align__(16) float sa[(RT + 63) / 64 * 64], sw[(RN + 63) / 64 * 64], bias[(RN + 63) / 64 * 64];
  };
  int p, nrows, trows, K, chunk, wave;
  int64_t n0, t0;
  const int8_t *w, *a;      // the block's first rows
  rsrc_t rw, ra;
  uint32_t to, off[kLoads];

  __device__ __forceinline__ Block(const MatmulArgs& g, int tiles_t, int tiles_n, int tiles,
                                   Lds& lds) {
    // Each XCD takes one run of tiles, and walks it 4 tiles of channels by
    // many of tokens, so the blocks that run together share operands in its L2.
    const int b = blockIdx.x, xcd = b % kXcds;
    const int tile = xcd * (tiles / kXcds) + min(xcd, tiles % kXcds) + b / kXcds;
    const int per_p = tiles_t * tiles_n;
    p = tile / per_p;
    int in = tile % per_p;
    const int group = in / (4 * tiles_t);
    in -= group * 4 * tiles_t;
    const int height = min(4, tiles_n - group * 4);
    n0 = (int64_t)(group * 4 + in % height) * RN;
    t0 = (int64_t)(in / height) * RT;
    nrows = (int)min((int64_t)RN, g.N - n0);
    trows = (int)min((int64_t)RT, g.T - t0);
    K = (int)g.K;
    const int pitch = (int)g.a_pitch, tid = threadIdx.x, row = tid >> 3;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    w = g.w + (p * g.N + n0) * g.K;
    rw = make_rsrc(w, (uint32_t)(nrows * K));
    if constexpr (!kCodes) {
      a = g.a + p * g.a_shard + t0 * g.a_pitch;
      ra = make_rsrc(a, (uint32_t)((trows - 1) * pitch + K));
    }
    chunk = ((tid & 7) ^ (row >> 1 & 7)) * 16;
#pragma unroll
    for (int i = 0; i < RN / 32; ++i)
      off[i] = (uint32_t)(min(row + 32 * i, nrows - 1) * K + chunk);
#pragma unroll
    for (int i = 0; i < kTokens / 32; ++i)
      off[RN / 32 + i] = (uint32_t)(min(row + 32 * i, trows - 1) * pitch + chunk);
    to = lds_address(lds.operands) + wave * 1024;
    // The scales and biases go to LDS first, where the epilogue reads them
    // without waiting for its own stores (vector loads and stores retire in
    // one order). One wave loads 64 of them at a time.
    if constexpr (!kCodes) stage(g.a_scale + p * g.as_shard + t0, trows, lds.sa, RT);
    stage(g.w_scale + p * g.N + n0, nrows, lds.sw, RN);
    if (g.bias)
      stage(g.bias + p * g.N + n0, nrows, lds.bias, RN);
    else
      for (int i = tid; i < RN; i += 256) lds.bias[i] = 0.0f;
  }
  __device__ __forceinline__ void stage(const float* from, int n, float* dst, int size) const {
    const rsrc_t r = make_rsrc(from, (uint32_t)n * 4u);
    for (int i = wave * 64; i < size; i += 256)
      load_to_lds<4>(r, lds_address(dst + i), (uint32_t)(i + (threadIdx.x & 63)) * 4u, 0);
  }
  // Load i of a step into buffer `buf`. Past the end of a row (and for the
  // steps past the last, which keep the counts of loads in flight the same)
  // the address is out of range: nothing is read.
  __device__ __forceinline__ void fetch(int step, int buf, int i) const {
    const bool in_row = step * kStep + chunk < K;
    const uint32_t at = to + buf * kStage + i * 32 * kStep, from = in_row ? off[i] : kOOB;
    if (i < RN / 32)
      load_to_lds<16, kNt>(rw, at, from, step * kStep);
    else
      load_to_lds<16>(ra, at, from, step * kStep);
  }
  // The same load to registers, for rows on any byte: of a step that ends
  // inside the rows,
  __device__ __forceinline__ v4i load_whole(int step, int i) const {
    v4i v;
    __builtin_memcpy(&v, (i < RN / 32 ? w : a) + (off[i] + (uint32_t)(step * kStep)), 16);
    return v;
  }
  // and of any step: 16 bytes that end inside the row, shifted down to where
  // they belong.
  __device__ __forceinline__ v4i load(int step, int i) const {
    const int k = step * kStep;
    if (k + kStep <= K) return load_whole(step, i);
    const int past = max(k + chunk + 16 - K, 0);   // bytes of the chunk past the row
    if (past >= 16) return v4i{0, 0, 0, 0};
    v4i v;
    __builtin_memcpy(&v, (i < RN / 32 ? w : a) + (off[i] + (uint32_t)(k - past)), 16);
    const unsigned __int128 bits = __builtin_bit_cast(unsigned __int128, v) >> (8 * past);
    return __builtin_bit_cast(v4i, bits);
  }
  static __device__ __forceinline__ void put(Lds& lds, int buf, int i, v4i v) {
    *(v4i*)(lds.operands + buf * kStage + i * 32 * kStep + threadIdx.x * 16) = v;
  }
  __device__ __forceinline__ int steps() const { return (K + kStep - 1) / kStep; }
  // Operand rows row..row+31 of slice `slice` in buffer `buf`: this lane's 16
  // bytes. Channels come first, tokens from row RN.
  static __device__ __forceinline__ v4i read(const Lds& lds, int buf, int slice, int row) {
    const int lane = threadIdx.x & 63;
    const int pos = ((2 * slice + (lane >> 5)) ^ (lane >> 1 & 7)) * 16;
    return *(const v4i*)(lds.operands + buf * kStage + (lane & 31) * kStep + pos + row * kStep);
  }
};

// kLoad: kDirect or kDirectNt where K and every row lie on 16 bytes. kAnyByte
// (S = 2): the next step's operands wait in registers while this one is
// multiplied.
enum Load { kDirect, kDirectNt, kAnyByte };

template <int WN, int WT, int MN, int MT, int S, Load kLoad, bool kVec, bool kBf>
__global__ __launch_bounds__(256, MN* MT == 16 ? 1 : 2) void matmul_tile_kernel(
    MatmulArgs g, int tiles_t, int tiles_n, int tiles) {
  static_assert(WN * WT == 4 && (kLoad != kAnyByte || S == 2));
  constexpr int RN = 32 * MN * WN, RT = 32 * MT * WT;
  using B = Block<RN, RT, S, kLoad == kDirectNt>;
  constexpr int kLoads = B::kLoads;
  __shared__ typename B::Lds lds;
  const B b(g, tiles_t, tiles_n, tiles, lds);
  const int wn = b.wave / WT * 32 * MN, wt = b.wave % WT * 32 * MT;
  v4i fw[2][MN], fa[2][MT];
  // operand i of a slice
  auto read = [&](int buf, int slice, int i) {
    if (i < MN)
      fw[slice & 1][i] = B::read(lds, buf, slice, wn + 32 * i);
    else
      fa[slice & 1][i - MN] = B::read(lds, buf, slice, RN + wt + 32 * (i - MN));
  };
  v16i acc[MN][MT] = {};
  // The products of a slice, in turn with the reads of the slice after it and
  // with also(d0) .. also(d1 - 1). The fences keep this order.
  auto slice = [&](int set, int rbuf, int rslice, int d0, int d1, auto also) {
    constexpr int kM = MN * MT, kR = MN + MT;
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      acc[m / MT][m % MT] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
          fw[set][m / MT], fa[set][m % MT], acc[m / MT][m % MT], 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kR; ++r)
        if (min(r * kM / kR / 2, kM - 1) == m) read(rbuf, rslice, r);
#pragma unroll
      for (int d = 0; d < kLoads; ++d)
        if (d >= d0 && d < d1 && (d - d0) * kM / (d1 - d0) == m) also(d);
      issue_fence();
    }
  };
  const auto nothing = [](int) {};
  const int steps = b.steps();
  int buf = 0;
  if constexpr (kLoad != kAnyByte) {
    // half of a step's loads go out right after the barrier that frees their
    // buffer, the other half a slice later: together they would hold up the
    // products that follow (8192^3: 2319 against 2439 TOPS)
    constexpr int kEarly = kLoads / 2;
#pragma unroll
    for (int q = 0; q < S; ++q)
#pragma unroll
      for (int i = 0; i < (q == S - 1 ? kEarly : kLoads); ++i) b.fetch(q, q, i);
    wait_loads<(S - 2) * kLoads + kEarly, true>();
    __builtin_amdgcn_s_barrier();
    issue_fence();
#pragma unroll
    for (int i = 0; i < MN + MT; ++i) read(0, 0, i);
    for (int step = 0; step < steps; ++step) {
      const int next = S == 2 ? buf ^ 1 : buf + 1 == S ? 0 : buf + 1;
      const int last = S == 2 ? next : buf == 0 ? S - 1 : buf - 1;   // buffer of step + S - 1
      slice(0, buf, 1, kEarly, kLoads, [&](int d) { b.fetch(step + S - 1, last, d); });
      slice(1, buf, 2, 0, 0, nothing);
      slice(0, buf, 3, 0, 0, nothing);
      wait_loads<(S - 2) * kLoads, true>();   // the next step is in LDS
      __builtin_amdgcn_s_barrier();           // for all waves, and this buffer is free
      issue_fence();
      slice(1, next, 0, 0, kEarly, [&](int d) { b.fetch(step + S, buf, d); });
      buf = next;
    }
  } else {
    v4i next_rows[kLoads];
    if (b.K >= kStep) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) next_rows[i] = b.load_whole(0, i);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) B::put(lds, 0, i, next_rows[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        B::put(lds, 0, i, b.load(0, i));
        issue_fence();
      }
    }
    wait_loads<0, true>();   // also the scales
    lds_barrier();
#pragma unroll
    for (int i = 0; i < MN + MT; ++i) read(0, 0, i);
    // the next step's loads go out over two slices and into the other buffer
    // over the third
    int step = 0;
    for (; step + 1 < b.K / kStep; ++step) {
      const auto load = [&](int d) { next_rows[d] = b.load_whole(step + 1, d); };
      slice(0, buf, 1, 0, kLoads / 2, load);
      slice(1, buf, 2, kLoads / 2, kLoads, load);
      slice(0, buf, 3, 0, kLoads, [&](int d) { B::put(lds, buf ^ 1, d, next_rows[d]); });
      lds_barrier();
      slice(1, buf ^ 1, 0, 0, 0, nothing);
      buf ^= 1;
    }
    for (; step < steps; ++step) {   // the next step is the row's end, or past it
      slice(0, buf, 1, 0, 0, nothing);
      slice(1, buf, 2, 0, 0, nothing);
      slice(0, buf, 3, 0, 0, nothing);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        B::put(lds, buf ^ 1, i, b.load(step + 1, i));
        issue_fence();
      }
      lds_barrier();
      slice(1, buf ^ 1, 0, 0, 0, nothing);
      buf ^= 1;
    }
  }

  wait_loads<0, true>();   // no load may land in what is written next
  lds_barrier();
  const OutTile o = {out_rsrc<kBf>(g, b.p, b.t0, b.n0, b.trows, b.nrows), lds.sw, lds.bias,
                     b.nrows};
  static_assert(4 * kTurnBytes<MN, kBf> <= sizeof(lds.operands), "the turn fits");
  int8_t* turn = lds.operands + b.wave * kTurnBytes<MN, kBf>;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const v16i* part[MN];
#pragma unroll
    for (int i = 0; i < MN; ++i) part[i] = &acc[i][j];
    store_rows<MN, kVec, kBf>(part, o, turn, lds.sa[wt + 32 * j + (lane_id() & 31)],
                              wt + 32 * j, wn, b.trows, (int)g.N);
  }
}

// The end of the kernels whose waves split k: sums added through LDS, scaled
// and stored.
template <int MN, int MT, bool kVec, bool kBf, typename B>
__device__ __forceinline__ void finish_split(const MatmulArgs& g, const B& b,
                                             typename B::Lds& lds, const v16i (&acc)[MN][MT]) {
  wait_loads<0, true>();   // no load may land in what is written next
  lds_barrier();
  const OutTile o = {out_rsrc<kBf>(g, b.p, b.t0, b.n0, b.trows, b.nrows), lds.sw, lds.bias,
                     b.nrows};
  // wave v finishes the channels 8v .. 8v+7 of every product: acc[4v .. 4v+3]
  const int lane = threadIdx.x & 63, h = lane >> 5;
  constexpr int kSums = 4 * MN * MT * 4 * 64 * 16;
  static_assert(kSums + MT * kTurnBytes<MN, kBf> <= sizeof(lds.operands), "the sums fit");
  v4i* sums = (v4i*)lds.operands;
  int8_t* turn = lds.operands + kSums;
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sums[((b.wave * MN * MT + i * MT + j) * 4 + v) * 64 + lane] =
            v4i{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2],
                acc[i][j][4 * v + 3]};
  lds_barrier();
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      v4i sum = sums[((i * MT + j) * 4 + b.wave) * 64 + lane];
#pragma unroll
      for (int q = 1; q < 4; ++q)
        sum += sums[((q * MN * MT + i * MT + j) * 4 + b.wave) * 64 + lane];
      const int t = 32 * j + (lane & 31), c = 32 * i + 8 * b.wave + 4 * h;
      const float sa = lds.sa[t];
      const v4f w = *(const v4f*)(o.sw + c), bias = *(const v4f*)(o.bias + c);
      store_turn<kBf>(turn + t * kTurnRow<MN, kBf>, c, sum, sa, w, bias);
    }
  lds_barrier();
  store_turned<256, MN, kVec, kBf>((int)threadIdx.x, 32 * MT, turn, o, 0, 0, b.trows, (int)g.N);
}

// ---- few tokens or few tiles: the waves of a block split k ----
//
// The product then costs less than reading the weights, and what counts is
// bytes in flight on every CU. The block is 32*MN channels x 32*MT tokens, so
// that few channels still make many blocks; its four waves share the loads as
// above and each multiplies one of a step's four slices. Their int32 sums are
// added through LDS at the end, exact in any order. T=8 N=1024 P=8 K=8192 (67 MB
// of weights, 256 blocks): 12.9 us, 5.2 TB/s; 128 channels a block leave 64
// blocks and take 25.6.
template <int MN, int MT, int S, Load kLoad, bool kVec, bool kBf>
__global__ __launch_bounds__(256, 2) void matmul_split_kernel(MatmulArgs g, int tiles_t,
                                                              int tiles_n, int tiles) {
  constexpr int RN = 32 * MN, RT = 32 * MT;
  using B = Block<RN, RT, S, kLoad == kDirectNt>;
  constexpr int kLoads = B::kLoads;
  __shared__ typename B::Lds lds;
  const B b(g, tiles_t, tiles_n, tiles, lds);
  v16i acc[MN][MT] = {};
  v4i fw[MN], fa[MT];
  auto read = [&](int buf) {
#pragma unroll
    for (int i = 0; i < MN; ++i) fw[i] = B::read(lds, buf, b.wave, 32 * i);
#pragma unroll
    for (int i = 0; i < MT; ++i) fa[i] = B::read(lds, buf, b.wave, RN + 32 * i);
  };
  auto multiply = [&]() {
#pragma unroll
    for (int i = 0; i < MN; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
  };
  const int steps = b.steps();
  int buf = 0;
  if constexpr (kLoad != kAnyByte) {
#pragma unroll
    for (int q = 0; q < S - 1; ++q)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) b.fetch(q, q, i);
    for (int step = 0; step < steps; ++step) {
      wait_loads<(S - 2) * kLoads, false>();   // this step is in LDS
      __builtin_amdgcn_s_barrier();            // for all waves, and the last step's buffer is free
      issue_fence();
      read(buf);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) b.fetch(step + S - 1, buf == 0 ? S - 1 : buf - 1, i);
      multiply();
      issue_fence();
      buf = buf + 1 == S ? 0 : buf + 1;
    }
  } else {
    // steps on their way in registers, and as many in LDS
    constexpr int kDeep = MN * MT == 1 ? 4 : 2;
    v4i rows[kDeep][kLoads];
#pragma unroll
    for (int q = 0; q < kDeep; ++q)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) rows[q][i] = b.load(q, i);
    for (int step = 0; step < steps; step += kDeep) {
#pragma unroll
      for (int q = 0; q < kDeep; ++q) {
        if (step + q >= steps) break;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) B::put(lds, q, i, rows[q][i]);
        lds_barrier();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) rows[q][i] = b.load(step + kDeep + q, i);
        read(q);
        multiply();
      }
    }
  }
  finish_split<MN, MT, kVec, kBf>(g, b, lds, acc);
}

// ---- activations quantized by the block: one launch for a small linear layer ----
//
// For calls that the second launch and the codes' way through memory would
// lengthen most: 32 channels x kTokens tokens a block, waves splitting k as
// above. A wave reads 16/NVEC rows of x, all at once (NVEC vectors of 8 a lane),
// takes their largest values and leaves codes and scales in LDS, while the first
// steps of the weights land. Every block of channels quantizes its tokens
// again, from L2. Both sides of the rule (at most two blocks a CU), one launch
// against two, us: one call after another the host's part counts and one launch
// always takes less (P=8 T=1 N=1024 K=1024: 7.4 against 10.0; T=32 N=4096 K=512:
// 7.3 against 10.0; P=8 T=32 N=2048 K=512: 8.1 against 10.1). In a graph it takes
// less up to about 24 rows a block (P=8 T=1 N=1024 K=1024: 4.1 against 5.7; P=3
// T=77 N=999 K=1000: 7.7 against 8.9; T=24 N=4096 K=512: 5.5 with either) and
// more where a block quantizes 32 rows of short k (T=32 N=4096 K=512: 6.3 against
// 5.5; with two blocks a CU, P=8 T=32 N=2048 K=512, 8.3 against 6.3; P=2 T=16
// N=8192 K=2048, 16 rows, 9.7 against 8.6).
template <Load kLoad, int NVEC, bool kBf>
__global__ __launch_bounds__(256, 2) void linear_small_kernel(MatmulArgs g, const uint16_t* x,
                                                              int64_t x_shard, int64_t x_pitch,
                                                              int tiles_t, int tiles_n, int tiles) {
  constexpr int kRows = 16 / NVEC, kTokens = 4 * kRows, S = 6;
  constexpr int kCodeRow = NVEC * 512 + 16;   // 16: rows start in different banks
  using B = Block<32, kTokens, S, false, true>;
  typedef uint32_t v2u __attribute__((ext_vector_type(2)));
  typedef unsigned short v2h __attribute__((ext_vector_type(2)));
  __shared__ typename B::Lds lds;
  __shared__ __align__(16) int8_t codes[kTokens * kCodeRow];
  const B b(g, tiles_t, tiles_n, tiles, lds);
  const int lane = threadIdx.x & 63;
  v4i raw[kRows][NVEC];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (4 * r + b.wave >= b.trows) break;
    const int64_t t = b.t0 + 4 * r + b.wave;
    const rsrc_t rx = make_rsrc(x + b.p * x_shard + t * x_pitch, (uint32_t)b.K * 2u);
#pragma unroll
    for (int v = 0; v < NVEC; ++v)
      raw[r][v] = __builtin_bit_cast(
          v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, (uint32_t)(v * 64 + lane) * 16u, 0, 0));
  }
  issue_fence();
  constexpr int kDeep = 4;   // steps on their way in registers (kAnyByte)
  v4i rows[kDeep];
#pragma unroll
  for (int q = 0; q < (kLoad == kAnyByte ? kDeep : S - 1); ++q) {
    if constexpr (kLoad == kAnyByte)
      rows[q] = b.load(q, 0);
    else
      b.fetch(q, q, 0);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (4 * r + b.wave >= b.trows) break;
    v2h big = {0, 0};
#pragma unroll
    for (int v = 0; v < NVEC; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        big = __builtin_elementwise_max(
            big, __builtin_bit_cast(v2h, (uint32_t)raw[r][v][j] & 0x7fff7fffu));
    const uint32_t most = wave_combine((uint32_t)max(big[0], big[1]) << 16,
                                       [](uint32_t p, uint32_t q) { return max(p, q); });
    const RowScale rs = row_scale(most);
    const int t = 4 * r + b.wave;
    if (lane == 0) lds.sa[t] = rs.scale;
#pragma unroll
    for (int v = 0; v < NVEC; ++v) {
      uint32_t c[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t d = (uint32_t)raw[r][v][j];
        c[2 * j] = code_bits(__uint_as_float(d << 16), rs.mul);
        c[2 * j + 1] = code_bits(__uint_as_float(d & 0xffff0000u), rs.mul);
      }
      *(v2u*)(codes + t * kCodeRow + (v * 64 + lane) * 8) =
          v2u{c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
              c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24};
    }
  }
  lds_barrier();
  const int8_t* code = codes + min(lane & 31, b.trows - 1) * kCodeRow + b.wave * 32 +
                       (lane >> 5) * 16;
  v16i acc[1][1] = {};
  auto multiply = [&](int buf, int step) {
    acc[0][0] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
        B::read(lds, buf, b.wave, 0), *(const v4i*)(code + step * kStep), acc[0][0], 0, 0, 0);
  };
  const int steps = b.steps();
  if constexpr (kLoad == kAnyByte) {
    for (int step = 0; step < steps; step += kDeep) {
#pragma unroll
      for (int q = 0; q < kDeep; ++q) {
        if (step + q >= steps) break;   // codes end with the row
        B::put(lds, q, 0, rows[q]);
        lds_barrier();
        rows[q] = b.load(step + kDeep + q, 0);
        multiply(q, step + q);
      }
    }
  } else {
    int buf = 0;
    for (int step = 0; step < steps; ++step) {
      wait_loads<S - 2, false>();
      __builtin_amdgcn_s_barrier();
      issue_fence();
      b.fetch(step + S - 1, buf == 0 ? S - 1 : buf - 1, 0);
      multiply(buf, step);
      issue_fence();
      buf = buf + 1 == S ? 0 : buf + 1;
    }
  }
  finish_split<1, 1, false, kBf>(g, b, lds, acc);
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;
// Blocks of 256 threads that a grid may have, one for each tile.
constexpr int64_t kMaxTiles = int64_t(1) << 23;

hipError_t launch_general(const MatmulArgs& a, hipStream_t s) {
  const int64_t tt = (a.T + kGenTile - 1) / kGenTile, tn = (a.N + kGenTile - 1) / kGenTile;
  const int64_t tiles = a.P * tt * tn;
  matmul_general_kernel<<<dim3((unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks)), 256, 0, s>>>(
      a, tt, tn, tiles);
  return hipGetLastError();
}

// A kernel over RN x RT tiles; kernel(vec, bf16, grid, tiles of t, of n, of all).
template <int RN, int RT, typename F>
hipError_t launch_tiled(const MatmulArgs& a, hipStream_t s, F kernel) {
  const int64_t tt = (a.T + RT - 1) / RT, tn = (a.N + RN - 1) / RN, n = a.P * tt * tn;
  if (n >= kMaxTiles) return launch_general(a, s);
  const bool bf = a.y_type == kBf16, vec = a.N % 8 == 0 && ((uintptr_t)a.y & 15) == 0;
  const auto run = [&](auto v, auto b) { kernel(v, b, dim3((unsigned)n), (int)tt, (int)tn, (int)n); };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  if (vec)
    bf ? run(yes, yes) : run(yes, no);
  else
    bf ? run(no, yes) : run(no, no);
  return hipGetLastError();
}

template <int WN, int WT, int MN, int MT, int S, Load kLoad = kDirect>
hipError_t launch_tiles(const MatmulArgs& a, hipStream_t s) {
  return launch_tiled<32 * MN * WN, 32 * MT * WT>(
      a, s, [&](auto v, auto b, dim3 grid, int tt, int tn, int n) {
        matmul_tile_kernel<WN, WT, MN, MT, S, kLoad, decltype(v)::value, decltype(b)::value>
            <<<grid, 256, 0, s>>>(a, tt, tn, n);
      });
}

template <int MN, int MT, int S, Load kLoad = kDirect>
hipError_t launch_split(const MatmulArgs& a, hipStream_t s) {
  return launch_tiled<32 * MN, 32 * MT>(
      a, s, [&](auto v, auto b, dim3 grid, int tt, int tn, int n) {
        matmul_split_kernel<MN, MT, S, kLoad, decltype(v)::value, decltype(b)::value>
            <<<grid, 256, 0, s>>>(a, tt, tn, n);
      });
}

// A block's rows of a, w and y must each span less than 2^31 bytes (there are
// 256 of them at most).
bool spans_ok(const MatmulArgs& a) {
  return a.a_pitch < (int64_t(1) << 22) && a.N < (int64_t(1) << 20);
}

// Direct 16-byte loads need every row on a 16-byte boundary.
bool rows_aligned(const MatmulArgs& a) {
  return a.K % 16 == 0 && a.a_pitch % 16 == 0 && a.a_shard % 16 == 0 &&
         ((uintptr_t)a.a & 15) == 0 && ((uintptr_t)a.w & 15) == 0;
}

// The tile whose blocks, in rounds over the chip's 256 CUs, cost least. A cost
// is the time of a round with `few` (at most 256) or `full` (512, two a CU)
// blocks in units of a round of 256 x 256 tiles, measured at K=4096: T=64 ..
// 4096, N=4096 .. 8192, P=1 and 8. One tile for all sizes loses up to 5x (T=128
// N=4096 K=4096: 8.3 us with 32 x 64 tiles, 41.5 us with 256 x 256; T=8192
// N=8192 K=8192: 450 us with 256 x 256, 560 us with 128 x 128). Rows on any
// byte cost more for each load, so large tiles pay sooner (K=4095 N=4096 T=256:
// 22 us with 32 x 64, 46 with 128 x 128; 8192 x 8192: 742 with 256 x 256, 881
// with 128 x 128, 1199 with 128 x 64; with the loads spread over the slices
// 675 with 256 x 256).
enum Tile { k256x256, k128x128, k128x64, k64x64, k32x64, k32x32, kTiles };

Tile choose_tile(const MatmulArgs& a, bool direct) {
  struct Cost {
    int n, t;
    float few, full;
  };
  constexpr Cost direct_cost[kTiles] = {{256, 256, 1.0f, 2.0f},  {128, 128, 0.37f, 0.62f},
                                        {128, 64, 0.26f, 0.42f}, {64, 64, 0.17f, 0.30f},
                                        {32, 64, 0.13f, 0.22f},  {32, 32, 0.11f, 0.16f}};
  constexpr Cost any_cost[kTiles] = {{256, 256, 1.0f, 2.0f},  {128, 128, 0.50f, 0.59f},
                                     {128, 64, 0.39f, 0.43f}, {64, 64, 9.0f, 9.0f},   // not built
                                     {32, 64, 0.15f, 0.24f},  {32, 32, 0.10f, 0.15f}};
  const Cost* tiles = direct ? direct_cost : any_cost;
  Tile best = k256x256;
  float least = 0.0f;
  for (int i = 0; i < kTiles; ++i) {
    const int64_t blocks =
        a.P * ((a.T + tiles[i].t - 1) / tiles[i].t) * ((a.N + tiles[i].n - 1) / tiles[i].n);
    float cost = blocks <= 256 ? tiles[i].few : (float)((blocks + 511) / 512) * tiles[i].full;
    if (i == k256x256) {
      cost = (float)((blocks + 255) / 256);
      // With short sums a block mostly waits for its first loads and its
      // stores, which a second block on the CU covers: at P=8 T=2048 N=4096
      // 256 x 256 and 128 x 128 tiles take 55.3 and 51.8 us for K=256, 67.2
      // and 64.6 us for K=512, 88.8 and 94.2 us for K=1024.
      cost *= a.K <= 512 ? 1.3f : a.K <= 1024 ? 1.15f : 1.0f;
    }
    if (i == 0 || cost < least) best = (Tile)i, least = cost;
  }
  return best;
}

// Vectors of 8 a lane for rows of K, and the tokens of a block.
int small_vectors(int64_t K) { return K <= 1024 ? 2 : K <= 2048 ? 4 : K <= 4096 ? 8 : 16; }

template <Load kLoad, int NVEC>
hipError_t launch_small(const void* x, int64_t x_shard, int64_t x_pitch, const MatmulArgs& m,
                        hipStream_t s) {
  constexpr int kTokens = 64 / NVEC;
  const int64_t tt = (m.T + kTokens - 1) / kTokens, tn = (m.N + 31) / 32, n = m.P * tt * tn;
  if (m.y_type == kBf16)
    linear_small_kernel<kLoad, NVEC, true><<<dim3((unsigned)n), 256, 0, s>>>(
        m, (const uint16_t*)x, x_shard, x_pitch, (int)tt, (int)tn, (int)n);
  else
    linear_small_kernel<kLoad, NVEC, false><<<dim3((unsigned)n), 256, 0, s>>>(
        m, (const uint16_t*)x, x_shard, x_pitch, (int)tt, (int)tn, (int)n);
  return hipGetLastError();
}

template <Load kLoad>
hipError_t launch_small_rows(const void* x, int64_t x_shard, int64_t x_pitch, const MatmulArgs& m,
                             hipStream_t s) {
  switch (small_vectors(m.K)) {
    case 2: return launch_small<kLoad, 2>(x, x_shard, x_pitch, m, s);
    case 4: return launch_small<kLoad, 4>(x, x_shard, x_pitch, m, s);
    case 8: return launch_small<kLoad, 8>(x, x_shard, x_pitch, m, s);
    default: return launch_small<kLoad, 16>(x, x_shard, x_pitch, m, s);
  }
}

}  // namespace

hipError_t launch_int8_matmul(const MatmulArgs& a, hipStream_t s) {
  if (spans_ok(a) && rows_aligned(a)) {
    const int64_t n32 = a.P * ((a.N + 31) / 32);
    const int64_t n128 = a.P * ((a.N + 127) / 128), n64 = a.P * ((a.N + 63) / 64);
    // Few tokens: the weights are read once, and the tile only has to keep
    // every CU loading. 128 channels a block share the activations best; with
    // fewer than one such block a CU, smaller ones fill the chip (T=64 P=8 K=8192
    // N=1024: 15.7 us with 32 channels, 27.9 with 128; P=4 N=8192 K=4096: 29.0
    // and 24.4; P=2 N=8192 K=8192: 29.1 with 32, 25.9 with 64, 33.8 with 128). For up to 32 tokens
    // and long k, 64 channels by split waves read more steadily than 128 (T=16
    // N=8192 P=8 K=4096: 54.7 against 63.2 us; K=1024: 15.1 against 13.5).
    // Weights as large as the 256 MB last-level cache cannot be there from an
    // earlier call and are not kept for a later one: loaded with the streaming
    // hint (N=8192 P=8 K=4096: T=64 63.8 -> 58.0 us, T=16 55.2 -> 48.9). Half
    // of that lost by it (N=8192 P=4 K=4096, found there again: 24.4 -> 33.5).
    const bool nt = a.P * a.N * a.K >= (int64_t(1) << 28);
    if (a.T <= 32) {
      if (n128 >= 512 && a.K <= 2048)
        return nt ? launch_tiles<4, 1, 1, 1, 3, kDirectNt>(a, s)
                  : launch_tiles<4, 1, 1, 1, 3>(a, s);
      if (n64 >= 512)
        return nt ? launch_split<2, 1, 6, kDirectNt>(a, s) : launch_split<2, 1, 6>(a, s);
      return launch_split<1, 1, 6>(a, s);
    }
    if (a.T <= 64) {
      if (n128 >= 256)
        return nt ? launch_tiles<4, 1, 1, 2, 3, kDirectNt>(a, s)
                  : launch_tiles<4, 1, 1, 2, 3>(a, s);
      if (n64 >= 256) return launch_split<2, 2, 6>(a, s);
      if (n32 >= 256) return launch_split<1, 2, 6>(a, s);
      return launch_split<1, 1, 6>(a, s);
    }
    switch (choose_tile(a, true)) {
      case k256x256: return launch_tiles<2, 2, 4, 4, 2>(a, s);
      case k128x128:   // one block a CU: more steps in flight
        return n128 * ((a.T + 127) / 128) <= 256 ? launch_tiles<2, 2, 2, 2, 4>(a, s)
                                                 : launch_tiles<2, 2, 2, 2, 2>(a, s);
      case k128x64: return launch_tiles<4, 1, 1, 2, 3>(a, s);
      case k64x64: return launch_split<2, 2, 6>(a, s);
      case k32x64: return launch_split<1, 2, 6>(a, s);
      default: return launch_split<1, 1, 6>(a, s);
    }
  }
  if (spans_ok(a) && a.K >= 16) {   // rows on any byte
    switch (choose_tile(a, false)) {
      case k256x256: return launch_tiles<2, 2, 4, 4, 2, kAnyByte>(a, s);
      case k128x128: return launch_tiles<2, 2, 2, 2, 2, kAnyByte>(a, s);
      case k128x64: return launch_tiles<4, 1, 1, 2, 2, kAnyByte>(a, s);
      case k32x64: return launch_split<1, 2, 4, kAnyByte>(a, s);
      default: return launch_split<1, 1, 4, kAnyByte>(a, s);
    }
  }
  return launch_general(a, s);
}

bool small_linear_ok(const void* x, int x_type, int64_t x_shard, int64_t x_pitch,
                     const MatmulArgs& m) {
  if (x_type != kBf16 || m.K < 16 || m.K > 8192 || m.K % 2 || m.N >= (int64_t(1) << 20))
    return false;
  if (((uintptr_t)x & 3) || x_shard % 2 || x_pitch % 2) return false;   // rows on 4 bytes
  const int64_t tokens = 64 / small_vectors(m.K);
  return m.P * ((m.N + 31) / 32) * ((m.T + tokens - 1) / tokens) <= 512;
}

hipError_t launch_small_linear(const void* x, int64_t x_shard, int64_t x_pitch,
                               const MatmulArgs& m, hipStream_t s) {
  return m.K % 16 == 0 && ((uintptr_t)m.w & 15) == 0
             ? launch_small_rows<kDirect>(x, x_shard, x_pitch, m, s)
             : launch_small_rows<kAnyByte>(x, x_shard, x_pitch, m, s);
}

}  // namespace btq
