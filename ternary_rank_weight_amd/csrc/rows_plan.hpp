// Which weight rows the tiles of rows_core.hpp take.  Host code without HIP.
#pragma once
#include <stdint.h>

namespace externd {

// The bits of how far apart a tile's rows are taken, for rows of ldw entries.
inline int rows_apart_bits(int64_t ldw) {
  int bits = 3;
  while (bits > 0 && ldw % ((int64_t)16 >> bits) == 0) --bits;
  return bits;
}
inline int64_t rows_tiles(int64_t rows, int apart_bits) {
  const int64_t group = (int64_t)16 << apart_bits;
  return ((rows + group - 1) / group) << apart_bits;
}

}  // namespace externd
