// Which 16-byte pieces (4 floats) of a row a tile of columns may load whole.
// Plain C++, so that the rule can be checked on the host.
#pragma once

#include <cstdint>

namespace nm {

// Whether columns c0 .. c0 + width of a row of C floats may be loaded in whole
// pieces: rows lie on 16 bytes (ldb % 4 == 0) and the piece that C ends inside,
// if the tile reaches it, ends within the row's `readable` columns.
constexpr bool whole_pieces(int c0, int width, int C, int64_t ldb, int64_t readable) {
  const int64_t end = int64_t(c0) + width, last = (int64_t(C) + 3) / 4 * 4;
  return (ldb & 3) == 0 && (end < last ? end : last) <= readable;
}

// The piece loaded for column c, a multiple of 4: the last one again past C.
constexpr int piece_start(int c, int C) {
  const int last = (C - 1) & ~3;
  return c < last ? c : last;
}

}  // namespace nm
