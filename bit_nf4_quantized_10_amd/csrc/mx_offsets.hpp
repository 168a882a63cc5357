// Byte offsets into an MXFP4 matrix's codes that a load takes in two parts, a lane's own
// and a scalar one.  Plain C++, so that a host program can run through all of them.
#pragma once

#include <stdint.h>

namespace qn {

struct MxOffset {
  uint32_t lane, scalar;
};

// Block 16 chunk + 4 step + g of a row of nb blocks, 16 bytes each; rows past the last and
// blocks past the row's end are masked (from 2^31 on, past any matrix).  The mask stands in
// the lane's part, since a buffer's range check need not count the scalar part: past the
// last row's end that one alone would lead up to 240 bytes out of the matrix.  Nor does the
// scalar part itself pass the matrix's end, which a check that subtracts it could not bear.
constexpr MxOffset mx_code_offset(int row, int rows, int nb, int chunk, int step, int g) {
  return MxOffset{(row < rows && 16 * chunk + 4 * step + g < nb ? (static_cast<uint32_t>(row) * static_cast<uint32_t>(nb) + g) * 16u : 0x80000000u) +
                      64u * step,
                  256u * chunk};
}

// The scalar part of the copies of a stage, eight blocks of every row: past the last block
// (of `last` of them) all lanes are masked, and it stays at the last stage that holds one.
constexpr uint32_t mx_stage_offset(int stage, int last) { return 128u * (stage < (last - 1) / 8 ? stage : (last - 1) / 8); }

}  // namespace qn
