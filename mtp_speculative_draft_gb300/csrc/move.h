// How kv_beam_reorder cuts its rows into tiles (plain C++, no CUDA).
#pragma once

#include <algorithm>
#include <cstdint>

namespace mtp {

constexpr int kMoveThreads = 256;
constexpr int kMoveWords = 16;  // 16-byte words a thread

struct MovePlan {
  int shift;      // a tile has 2^shift 16-byte words of a beam
  int rows;       // rows a tile
  int64_t tiles;  // tiles of max_len rows
};

// `wide`: the wider head size; `lists`: prompts times KV heads times K or V times
// layers.  A tile of every beam fits the CTA's registers: 64 KB, a power of two a
// beam (a row each of 64 beams of 256 dims).
inline MovePlan move_plan(int beams, int wide, int64_t lists, int max_len, int sms) {
  MovePlan p;
  p.shift = 12;
  static_assert(kMoveThreads * kMoveWords == 1 << 12, "16-byte words of a CTA");
  while ((beams << p.shift) > 1 << 12) --p.shift;
  auto tiles = [&](int rows) { return ((int64_t)max_len + rows - 1) / rows; };
  // smaller tiles where there is not a CTA an SM: 5 beams' 17 rows of 64 dims in one
  // layer 2.1 us, not 3.1
  while (p.shift > 0 && 4 << (p.shift - 1) >= wide && lists * tiles((4 << p.shift) / wide) < sms) --p.shift;
  p.rows = std::min(max_len, (4 << p.shift) / wide);
  p.tiles = tiles(p.rows);
  return p;
}

}  // namespace mtp
