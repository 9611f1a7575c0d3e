// Which bytes the main loop of w8_ring.h copies from memory: plain integers, so that a
// program on the host can replay every copy's range.
#pragma once

#include <cstdint>

namespace awq {

// One operand from its next k-tile on: `bytes` to the end of its last valid row, which
// the hardware checks every copy against, and the k-tiles left.
struct RingRange {
  int bytes, shorter, left;   // shorter: what a k-tile takes off
  constexpr void advance() { bytes = --left > 0 ? bytes - shorter : 0; }
};
// Where the next k-tile lies: 128 bytes on in every row, or in the next panel of every
// row's 128 bytes, which is as long as this one.
enum class RingKind { kRows, kPanels };
// `valid` rows of `row` bytes.
constexpr RingRange ring_range(RingKind kind, int valid, int row, int tiles) {
  // an empty range stays empty: below 0 the hardware would take it for one of 4 GiB
  return {valid * row, kind == RingKind::kRows && valid ? 128 : 0, tiles};
}

// A lane's 16 bytes in even (j = 0) and odd (1) copies of a wave, 8 rows each from row
// wave_row: rows of 8 chunks as swz64 has them.
constexpr int ring_offset(int wave_row, int lane, int j, int row) {
  return (wave_row + (lane >> 3)) * row + ((lane & 7) ^ ((lane >> 4) + 4 * j)) * 16;
}

// The rows of A that wave w of a gated pair's tile copies: 64 channels from n0 + 64·(w / 2)
// of the first layer (even w) or of the second, of which `valid` are there.
struct PairRows {
  int64_t first;
  int valid;
};
constexpr PairRows pair_rows(int64_t n0, int wave, int64_t N) {
  const int64_t first = n0 + 64 * (wave >> 1), left = N - first;
  return {left > 0 ? first : N - 1, left < 0 ? 0 : left < 64 ? int(left) : 64};
}

}  // namespace awq
