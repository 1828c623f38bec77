// Where the tiles of the product of 8-bit integers read their operands, as
// arithmetic that a host test can go through as well.
//
// A stage takes 64 bytes of k of 256 rows of each operand, in chunks of 16.
// The contraction is cut into whole turns of the ring.  No address lies outside
// its array, whichever way a buffer load compares its scalar offset with the
// descriptor's range: the intrinsic leaves that open, and only the vector
// offset's own comparison is relied on (for w's rows behind the last one, and
// for scales).
//   w [V,d]: stages are 64 bytes apart, but the last one of a row ends with the row
//     and later ones repeat it.  A row shorter than a stage repeats its last
//     chunk instead.
//   x: panels of whole blocks of 256 rows; a chunk that w's stages show a second
//     time is zero there, so that it adds nothing.  Rows behind the last one
//     hold anything: their sums are never stored.
#pragma once

namespace kd {

constexpr long kInt8Stage = 64, kInt8Chunk = 16, kInt8Turn = 4 * kInt8Stage, kInt8Rows = 256;

constexpr long int8_turns(long d) { return (d + kInt8Turn - 1) / kInt8Turn; }
constexpr long int8_panel_rows(long T) { return (T + kInt8Rows - 1) / kInt8Rows * kInt8Rows; }

// w: the byte of a row at which stage s begins, and that of chunk c in a stage
constexpr long int8_stage_at(long s, long d) {
  const long at = s * kInt8Stage, last = d - kInt8Stage;
  return last <= 0 ? 0 : at < last ? at : last;
}
constexpr long int8_chunk_at(long c, long d) { return c * kInt8Chunk < d ? c * kInt8Chunk : d - kInt8Chunk; }

// x: the byte of a row that chunk c of stage s holds, or -1 for zeros
constexpr long int8_x_at(long s, long c, long d) {
  if (s * kInt8Stage >= d) return -1;
  if (d < kInt8Stage) return c * kInt8Chunk < d ? c * kInt8Chunk : -1;
  const long at = int8_stage_at(s, d) + c * kInt8Chunk;
  return at < s * kInt8Stage ? -1 : at;
}

}  // namespace kd
