// How the experts' products are run.  Host code without HIP.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "rows_plan.hpp"

namespace externd {

constexpr int kMoeGroup = 16;      // slots that go through an expert's weights together
constexpr int kMoeFewSlots = 64;   // most slots whose choices the first product makes: a lane a slot

inline int64_t moe_most_groups(int64_t slots, int64_t experts) {
  return std::min(slots, std::min(slots, experts) + slots / kMoeGroup);
}

// Whether the first product makes the choice itself: a wave a token of its workgroups' eight, a lane a slot.
inline bool moe_few(int64_t tokens, int64_t top, int64_t experts) {
  return tokens <= 8 && tokens * top <= kMoeFewSlots && experts <= 256;
}

// Waves that share a tile of a product: as many as bring the launch to sixteen a compute unit.
inline int waves_a_tile(int64_t tiles, int64_t groups, int cus, int least, int most) {
  int sw = least;
  while (sw < most && tiles * groups * sw < (int64_t)cus * 16) sw *= 2;
  return sw;
}

struct MoeForms {
  int up;          // waves that share a tile of the first product: 4, 8 or 16
  int one;         // one token: waves of each of its experts, 1 to 16; else 0
  int down;        // more tokens: waves that share a tile of the second product, 1 to 16
  int down_tiles;  // that many tiles a wave at once
};
inline MoeForms moe_forms(int64_t tokens, int64_t top, int64_t experts, int64_t rows, int64_t cols, int64_t up_ld, int64_t down_ld, int cus) {
  const int64_t groups = moe_most_groups(tokens * top, experts);
  MoeForms f = {};
  f.up = waves_a_tile(rows_tiles(rows, rows_apart_bits(up_ld)), groups, cus, 4, 16);
  if (tokens == 1) {
    f.one = top == 1 ? 16 : top == 2 ? 8 : top <= 4 ? 4 : top <= 8 ? 2 : 1;
    return f;
  }
  const int64_t tiles = rows_tiles(cols, rows_apart_bits(down_ld));
  f.down = waves_a_tile(tiles, groups, cus, 1, 16);
  f.down_tiles = f.down == 1 && tiles * groups >= (int64_t)cus * 32 ? 2 : 1;
  return f;
}

}  // namespace externd
