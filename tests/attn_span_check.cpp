// Host check of attn_span.h: the tiles of sequences of every length up to 2^31 -
// 1, and the table entries that a wavefront fetches for them, two of its tiles
// ahead, in both forms of the kernel (every tile, every eighth one). Prints
// "ok <fetches>" or the first failure.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "attn_span.h"

using namespace nvfp4;

static uint64_t rng = 0x9E3779B97F4A7C15ull;
static uint32_t next_u32() {
  rng = rng * 6364136223846793005ull + 1442695040888963407ull;
  return (uint32_t)(rng >> 33);
}

static long fetches = 0;
static void fail(const char* what, int len, int64_t window, int page, int key) {
  std::printf("%s: len %d window %lld page %d key %d\n", what, len, (long long)window, page, key);
  std::exit(1);
}

static void fetch(int key, int page, int shift, int blocks, int len, int64_t window) {
  for (int ahead = 0; ahead < TK; ++ahead, ++fetches) {
    int in = -1;
    const int pi = page_of(key, ahead, page, shift, blocks, in);
    if (pi < 0 || pi >= blocks || in < 0 || in >= page) fail("outside the table", len, window, page, key);
    const int64_t k = (int64_t)(uint32_t)key + ahead;
    if (k < len && (int64_t)pi * page + in != k) fail("another key", len, window, page, key);
  }
}

static void check(int len, int64_t window, int Q, int page) {
  const int64_t blocks64 = (((int64_t)1 << 31) - 1) / page;   // a row of nearly 2^31 keys
  const int blocks = (int)blocks64;
  const int64_t cap64 = blocks64 * page;
  const int cap = (int)(cap64 < 0x7FFFFFFF ? cap64 : 0x7FFFFFFF);
  const int shift = (page & (page - 1)) == 0 ? __builtin_ctz((unsigned)page) : -1;
  const Span s = span_of(len, cap, Q, window);
  const int want = len < 0 ? 0 : len > cap ? cap : len;
  int64_t first = window ? (int64_t)want - Q - window + 1 : 0;
  if (first < 0) first = 0;
  if (s.len != want || s.n < 1 || s.base < 0 || s.base % TK || s.base > first ||
      first - s.base >= TK || (int64_t)s.base + (int64_t)s.n * TK < want ||
      (s.n > 1 && (int64_t)s.base + (int64_t)(s.n - 1) * TK >= want))
    fail("span", len, window, page, s.base);
  for (int step = 1; step <= 8; step += 7)
    for (int back = 1; back <= 20 && back <= s.n; ++back) {
      // a tile near the sequence's end, and what is fetched while it is computed
      const int key = (int)((int64_t)s.base + (int64_t)(s.n - back) * TK);
      const int nxt = tile_after(key, step), nxt2 = tile_after(nxt, step);
      fetch(key, page, shift, blocks, s.len, window);
      fetch(nxt, page, shift, blocks, s.len, window);
      fetch(nxt2, page, shift, blocks, s.len, window);
    }
}

int main() {
  const int pages[] = {1, 3, 16, 20, 100, 1024, 65536, 1000000, 1 << 20};
  const int64_t windows[] = {0, 1, 31, 33, 1000, 0x7FFFFFFF};
  for (int page : pages)
    for (int64_t window : windows)
      for (int Q : {1, 3, 64}) {
        for (int d = 0; d < 80; ++d) check(0x7FFFFFFF - d, window, Q, page);
        for (int len : {-0x7FFFFFFF - 1, -1, 0, 1, 31, 32, 33, 64, 1000}) check(len, window, Q, page);
        for (int i = 0; i < 50; ++i) check((int)next_u32(), window, Q, page);
      }
  std::printf("ok %ld\n", fetches);
  return 0;
}
