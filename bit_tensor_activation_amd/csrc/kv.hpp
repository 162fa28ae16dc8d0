// What the paged 4-bit cache's kernels share: its layout, the batch's layout and
// the search for a work item's sequence.
#pragma once

#include "common.hpp"

namespace btq {

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
// rows*mul, so b's begin at most at floor(starts[b]*mul / 2^shift) + b*extra, and
// that many are set aside: with extra 1 for parts that begin at the first row, 2
// for parts that begin at a multiple of 2^shift in the sequence. The grid then
// follows from T and the number of sequences, which the host knows.
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
    const int start = a.starts[at], next = a.starts[at + 1], length = a.lengths[at];
    const int64_t first = (((int64_t)start * mul) >> shift) + (int64_t)b * extra;
    const int n = __popcll(__ballot(b < hi && first <= item));
    if (n == 0) return -1;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) {
      *sub = item - (((int64_t)__builtin_amdgcn_readlane(start, n - 1) * mul) >> shift) -
             (int64_t)lo * extra;
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
