// Host check of attn_span.h for every tile that the kernels have, 16, 32 and 64 keys:
// the tiles of sequences of every length up to 2^31 - 1, and the table entries that a
// wavefront fetches for them, two of its tiles ahead, in both forms of the kernel (every
// tile, every eighth one), key by key and run by run. Prints "ok <fetches>" or the
// first failure.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "attn_span.h"

using namespace nvfp4;

static uint64_t rng = 0xD1B54A32D192ED03ull;
static uint32_t next_u32() {
  rng = rng * 6364136223846793005ull + 1442695040888963407ull;
  return (uint32_t)(rng >> 33);
}

static long fetches = 0;
static void fail(const char* what, int tile, int len, int64_t window, int page, int key) {
  std::printf("%s: tile %d len %d window %lld page %d key %d\n", what, tile, len,
              (long long)window, page, key);
  std::exit(1);
}

template <int TILE>
static void fetch(int key, int page, int shift, int blocks, int len, int64_t window) {
  int first = 0, first_in = 0;
  for (int ahead = 0; ahead < TILE; ++ahead, ++fetches) {
    int in = -1;
    const int pi = page_of(key, ahead, page, shift, blocks, in);
    if (pi < 0 || pi >= blocks || in < 0 || in >= page)
      fail("outside the table", TILE, len, window, page, key);
    const int64_t k = (int64_t)(uint32_t)key + ahead;
    if (k < len && (int64_t)pi * page + in != k) fail("another key", TILE, len, window, page, key);
    // a run of 16 keys (of 64 in pages of as many) is looked up once
    const int run = page % 64 == 0 && TILE == 64 ? 64 : 16;
    if (page % 16 == 0) {
      if (ahead % run == 0) {
        first = pi;
        first_in = in;
      } else if (pi != first || in != first_in + ahead % run) {
        fail("a run in two pages", TILE, len, window, page, key);
      }
    }
    // and a quad of keys, in pages of whole quads
    if (page % 4 == 0 && ahead % 4 != 0 && in % 4 != ahead % 4)
      fail("a quad in two pages", TILE, len, window, page, key);
  }
}

template <int TILE>
static void check(int len, int64_t window, int Q, int page) {
  const int64_t blocks64 = (((int64_t)1 << 31) - 1) / page;   // a row of nearly 2^31 keys
  const int blocks = (int)blocks64;
  const int64_t cap64 = blocks64 * page;
  const int cap = (int)(cap64 < 0x7FFFFFFF ? cap64 : 0x7FFFFFFF);
  const int shift = (page & (page - 1)) == 0 ? __builtin_ctz((unsigned)page) : -1;
  const Span s = span_of<TILE>(len, cap, Q, window);
  const int want = len < 0 ? 0 : len > cap ? cap : len;
  int64_t first = window ? (int64_t)want - Q - window + 1 : 0;
  if (first < 0) first = 0;
  if (s.len != want || s.n < 1 || s.base < 0 || s.base % TILE || s.base > first ||
      first - s.base >= TILE || (int64_t)s.base + (int64_t)s.n * TILE < want ||
      (s.n > 1 && (int64_t)s.base + (int64_t)(s.n - 1) * TILE >= want))
    fail("span", TILE, len, window, page, s.base);
  for (int step : {1, 8})
    for (int back = 1; back <= 20 && back <= s.n; ++back) {
      // a tile near the sequence's end, and what is fetched while it is computed
      const int key = (int)((int64_t)s.base + (int64_t)(s.n - back) * TILE);
      const int nxt = tile_after<TILE>(key, step), nxt2 = tile_after<TILE>(nxt, step);
      fetch<TILE>(key, page, shift, blocks, s.len, window);
      fetch<TILE>(nxt, page, shift, blocks, s.len, window);
      fetch<TILE>(nxt2, page, shift, blocks, s.len, window);
    }
}

template <int TILE>
static void all() {
  for (int page : {1, 3, 16, 20, 64, 100, 1024, 65536, 1000000, 1 << 20})
    for (int64_t window : {(int64_t)0, (int64_t)1, (int64_t)63, (int64_t)65, (int64_t)1000,
                           (int64_t)0x7FFFFFFF})
      for (int Q : {1, 3, 64}) {
        for (int d = 0; d < 2 * TILE + 3; d += TILE > 16 ? 3 : 1)
          check<TILE>(0x7FFFFFFF - d, window, Q, page);
        for (int len : {-0x7FFFFFFF - 1, -1, 0, 1, TILE - 1, TILE, TILE + 1, 2 * TILE, 1000})
          check<TILE>(len, window, Q, page);
        for (int i = 0; i < 20; ++i) check<TILE>((int)next_u32(), window, Q, page);
      }
}

int main() {
  all<16>();
  all<32>();
  all<64>();
  std::printf("ok %ld\n", fetches);
  return 0;
}
