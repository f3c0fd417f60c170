// attn_span.h -- the tiles of a sequence in attention over a paged cache, and
// the place of a key in its table: also built for the host, where a test walks
// them at the far end of the lengths.
#pragma once

#include <stdint.h>

#include "segments.h"   // NVFP4_HD

namespace nvfp4 {

constexpr int TK = 32;   // keys per tile

// The tiles of one sequence: keys base .. len - 1, with a window from a tile's
// start on. cap: the keys that its table row can name.
struct Span {
  int len, base, n;   // n >= 1: an empty sequence has one tile, of which nobody sees a key
};
NVFP4_HD inline Span span_of(int len, int cap, int64_t Q, int64_t window) {
  Span s;
  s.len = len < 0 ? 0 : len > cap ? cap : len;
  const int64_t lo = window ? (int64_t)s.len - Q - window + 1 : 0;
  s.base = lo <= 0 ? 0 : (int)lo & ~(TK - 1);
  s.n = s.len > s.base ? (s.len - s.base - 1) / TK + 1 : 1;
  return s;
}

// The first key of the tile `step` tiles after the one at `key`. A wavefront
// reads the table two of its tiles ahead, past the sequence's last one too: there
// the key may pass 2^31 and is a 32-bit number without a sign (as in page_of).
NVFP4_HD inline int tile_after(int key, int step) {
  return (int)((uint32_t)key + (uint32_t)(step * TK));
}

// The entry of a sequence's table row (its last one for keys past the row) that
// holds a key, and the key's place in the page.
NVFP4_HD inline int page_of(int key, int ahead, int page, int page_shift, int max_blocks,
                            int& in) {
  const uint32_t k = (uint32_t)key + (uint32_t)ahead;
  const uint32_t pi = page_shift >= 0 ? k >> page_shift : k / (uint32_t)page;
  in = (int)(k - pi * (uint32_t)page);
  return (int)(pi < (uint32_t)max_blocks ? pi : (uint32_t)max_blocks - 1u);
}

}  // namespace nvfp4
