// The search of the attention group for a work item's sequence, on the CPU: the device
// code of common.hpp (cut out of it into search.inc), run for a wave of 64 lanes that
// take turns. Prints "all ok", or what went wrong.
//
// For any seq_starts and lengths an item's columns or places have to lie inside the
// batch, and for ascending ones every row has to belong to exactly one item.
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <random>
#include <vector>

#define __device__
#define __host__
#define __forceinline__ inline
using std::max;
using std::min;

namespace {
constexpr int kLanes = 64;
struct { int x; } threadIdx;
ucontext_t g_main, g_lane[kLanes];
std::vector<char> g_stack[kLanes];
int64_t g_value[2][kLanes];   // what the lanes bring to an exchange, and to the next
int g_turn[kLanes];
std::function<void()> g_body;
int g_running;

void lane_main() {
  g_body();
  g_turn[threadIdx.x] = -1;
  swapcontext(&g_lane[threadIdx.x], &g_main);
}
// Every lane hands in x, and reads all when the last has.
const int64_t* exchange(int64_t x) {
  const int lane = threadIdx.x, at = g_turn[lane]++ & 1;
  g_value[at][lane] = x;
  swapcontext(&g_lane[lane], &g_main);
  return g_value[at];
}
void run_wave(std::function<void()> body) {
  g_body = body;
  for (int i = 0; i < kLanes; ++i) {
    g_stack[i].resize(65536);
    getcontext(&g_lane[i]);
    g_lane[i].uc_stack.ss_sp = g_stack[i].data();
    g_lane[i].uc_stack.ss_size = g_stack[i].size();
    g_lane[i].uc_link = nullptr;
    g_turn[i] = 0;
    makecontext(&g_lane[i], lane_main, 0);
  }
  for (bool any = true; any;) {
    any = false;
    for (int i = 0; i < kLanes; ++i) {
      if (g_turn[i] < 0) continue;
      threadIdx.x = i;
      swapcontext(&g_main, &g_lane[i]);
      any = true;
    }
  }
}
uint64_t __ballot(bool x) {
  const int64_t* v = exchange(x);
  uint64_t r = 0;
  for (int i = 0; i < kLanes; ++i) r |= (uint64_t)(v[i] & 1) << i;
  return r;
}
int read_lane(int x, int lane) { return (int)exchange(x)[lane]; }
}  // namespace
#define __popcll __builtin_popcountll
#define __builtin_amdgcn_readlane(x, lane) read_lane(x, lane)
#define __builtin_amdgcn_readfirstlane(x) read_lane(x, 0)

namespace btq {
#include "search.inc"
}
using namespace btq;

namespace {
int g_bad = 0;
void report(const char* what, const KvArgs& a, int mul, int shift, int64_t item, int64_t sub) {
  if (g_bad++ > 5) return;
  printf("%s: T=%d B=%d mul=%d shift=%d item=%d sub=%d starts", what, (int)a.T, a.B, mul, shift, (int)item, (int)sub);
  for (int i = 0; i <= min(a.B, 12); ++i) printf(" %d", a.starts[i]);
  printf("\n");
}
int find(const KvArgs& a, int mul, int shift, int extra, int64_t item, int64_t* sub, SeqRange* s) {
  int found = -2;
  run_wave([&] {
    int64_t n = 0;
    SeqRange r = {};
    const int b = find_sequence(a, mul, shift, extra, item, &n, &r);
    if (threadIdx.x == 0) found = b, *sub = n, *s = r;
  });
  return found;
}

// Groups of 2^shift columns of G a row, as attention takes them.
void columns(const KvArgs& a, int G, int shift, bool ascending) {
  std::vector<int> seen(a.T * G);
  const int extra = part_extra(G, shift);
  for (int64_t item = 0; item < ((a.T * G + (int64_t)a.B * extra) >> shift); ++item) {
    int64_t sub;
    SeqRange s;
    if (find(a, G, shift, extra, item, &sub, &s) < 0) continue;
    const int64_t first = sub << shift, cols = (int64_t)s.n * G;
    if (first >= cols) continue;
    if (first < 0 || s.begin < 0 || s.begin + s.n > a.T) {
      report("columns outside", a, G, shift, item, sub);
      continue;
    }
    for (int64_t c = first; c < min(first + (1 << shift), cols); ++c) ++seen[s.begin * G + c];
  }
  if (!ascending) return;
  for (int b = 0; b < a.B; ++b) {
    const SeqRange s = seq_range(a, b);
    for (int c = 0; c < s.n * G; ++c)
      if (seen[s.begin * G + c] != 1) {
        report("a column's items are not one", a, G, shift, seen[s.begin * G + c], c);
        return;
      }
  }
}
// Blocks of 32 places, as append and gather take them.
void places(const KvArgs& a, bool ascending) {
  std::vector<int> seen(a.T);
  for (int64_t item = 0; item < a.T / kBlockTokens + 2 * a.B; ++item) {
    int64_t sub;
    SeqRange s;
    if (find(a, 1, 5, 2 * kBlockTokens, item, &sub, &s) < 0) continue;
    const int64_t first = ((s.first() >> 5) + sub) * kBlockTokens;
    const int64_t from = max<int64_t>(s.first() - first, 0), to = min<int64_t>(s.length - first, kBlockTokens);
    for (int64_t t = from; t < to; ++t) {
      const int64_t row = s.begin + first - s.first() + t;
      if (row < 0 || row >= a.T) {
        report("a row outside", a, 1, 5, item, sub);
        break;
      }
      ++seen[row];
    }
  }
  if (!ascending) return;
  for (int b = 0; b < a.B; ++b) {
    const SeqRange s = seq_range(a, b);
    for (int i = 0; i < s.n; ++i)
      if (seen[s.begin + i] != 1) {
        report("a row's items are not one", a, 1, 5, seen[s.begin + i], i);
        return;
      }
  }
}
void check(std::vector<int32_t> starts, std::vector<int32_t> lengths, int T, int G, bool ascending) {
  KvArgs a = {};
  a.T = T;
  a.B = (int)lengths.size();
  a.starts = starts.data();
  a.lengths = lengths.data();
  a.capacity = 1 << 20;
  for (int shift = 3; shift <= 7; ++shift) columns(a, G, shift, ascending);
  places(a, ascending);
}
}  // namespace

int main(int argc, char** argv) {
  const bool any_order = argc > 1 && argv[1][0] == 'u';
  std::mt19937 g(7);
  if (any_order) check({0, 8, 8, 0, 1, 2, 3, 4, 5}, std::vector<int32_t>(8, 9), 8, 8, false);
  for (int i = 0; i < 150; ++i) {
    const int B = i % 20 == 0 ? 70 + g() % 80 : 1 + g() % 9, T = 1 + g() % 40, G = 1 + g() % 17;
    std::vector<int32_t> starts(B + 1), lengths(B);
    for (int32_t& x : lengths) x = (int)(g() % 100);
    for (int32_t& x : starts) x = any_order && i % 3 == 0 ? (int32_t)g() : (int)(g() % (T + 20)) - (i % 2 ? 10 : 0);
    if (!any_order || i % 3 == 1) std::sort(starts.begin(), starts.end());
    if (any_order && i % 3 == 1) std::reverse(starts.begin(), starts.end());
    if (!any_order && i % 2 == 0)
      for (int32_t& x : starts) x = min(x, T);
    check(starts, lengths, T, G, !any_order);
  }
  if (g_bad) return printf("%d wrong\n", g_bad), 1;
  printf("all ok\n");
  return 0;
}
