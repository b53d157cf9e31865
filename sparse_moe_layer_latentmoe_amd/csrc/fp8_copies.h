// Where the LDS-tiled 8-bit product's copies read, as plain integers (so that
// a host program can walk them too).
//
// A buffer load's bound is compared with its vector offset; what happens to
// the scalar offset in that comparison is not relied upon.  So a copy either
// stays inside its array with both offsets (weights), or carries its whole
// distance from the bounded base in the vector offset (scales), where what
// lies past the end reads as 0.
#pragma once
#include <cstddef>
#include <cstdint>

namespace lmoe {

constexpr int kFp8CopyRows = 8;  // weight rows of one copy instruction

// First row, counted from the tile's first, that the copy of rows row .. row
// + 7 reads: units past the matrix's last row read its last eight (their
// columns are not stored).  rows_left: rows from the tile's first to the
// matrix's end, a multiple of 8.
constexpr int fp8_weight_unit(int row, int rows_left) {
  return row < rows_left - kFp8CopyRows ? row : rows_left - kFp8CopyRows;
}

// The two offsets of lane `lane` in that copy, in bytes of a matrix whose rows
// have K codes, for block kb: chunk is the lane's 16-byte piece of the 128.
constexpr uint32_t fp8_weight_lane(int lane, uint32_t chunk, uint32_t K) {
  return (uint32_t)(lane >> 3) * K + chunk;
}
constexpr int fp8_weight_scalar(int row, int rows_left, int kb, int K) {
  return kb * 128 + fp8_weight_unit(row, rows_left) * K;
}

// Token scales of blocks 8 g .. 8 g + 7 of a row that starts `row` bytes from
// the base: lane's place in copy instruction i.
constexpr uint32_t fp8_xscale_lane(uint32_t row, int lane, int i, int g) {
  return row + (uint32_t)(g * 32 + ((lane & 7) ^ ((i & 1) << 2)) * 4);
}

// Weight scales: places 64 i .. 64 i + 63 of the tile's 128-row block b, in
// rows of KB scales.
constexpr uint32_t fp8_wscale_lane(int lane, int b, int i, int KB) {
  return (uint32_t)(b * KB + i * 64 + lane) * 4u;
}

}  // namespace lmoe
