// Which tiles a product of the orthogonalised updates takes. Plain C++: the
// choice is the host's, and a test on the host holds it to what it should be.
#pragma once

#include <stdint.h>

namespace sparcml {

constexpr uint32_t kPad = 64;  // sides are padded with zeros to this
constexpr uint32_t up(uint32_t v, uint32_t to) { return (v + to - 1) / to * to; }

// Tiles of I x J, or those of I x I on and below the diagonal.
constexpr uint32_t tiles_of(uint32_t I, uint32_t J, bool sym) { return sym ? I * (I + 1) / 2 : I * J; }

// Tiles of m x n, or of a symmetric m x m, that are `side` wide and high.
constexpr uint32_t tiles_by(uint32_t m, uint32_t n, bool sym, uint32_t side) {
  return tiles_of(up(m, side) / side, up(n, side) / side, sym);
}

// The side of a product's tiles, 64, 128 or 256, from the tiles that all of its
// matrices have together. The larger the tile, the fewer bytes a product takes;
// the smaller, the more CUs share the work. 64 x 64 tiles where all run at once,
// two to a CU (one matrix of 1000 x 1537: 250 us, against 456 with 128 x 128;
// six of 1024 x 1024, 816 such tiles: 702 against 651). Else by turns of the 256
// CUs: a 256 x 256 tile does the work of four of 128 x 128 in 1 / 1.2 of the
// time (12 of 2048 x 2048, 8 turns' worth each: 6.2 ms against 7.2), but 273
// of them take two turns where 975 smaller ones take four (three matrices of
// 3085 x 6855: 11.1 ms against 9.4).
constexpr uint64_t turns_of(uint64_t tiles) { return (tiles + 255) / 256; }
constexpr uint32_t tile_side(uint64_t tiny, uint64_t small, uint64_t large) {
  return tiny <= 512 ? 64 : 4 * turns_of(large) * 10 <= turns_of(small) * 12 ? 256 : 128;
}

}  // namespace sparcml
