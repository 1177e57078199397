// Where the forward on 8-bit rows reads: a lane's own offset keeps every access
// inside its operand, or is past any buffer's end, whatever the scalar offset adds
// (the range check of a buffer load need not count that one).  A row may end inside
// what a step reads; behind the last row nothing follows.
#pragma once
#include <stdint.h>

namespace qlk {

constexpr uint32_t kPast = 0x80000000u;   // an offset past the end of any operand

// Tiles: a step is a line of 128 bytes of a row, in eight 16-byte pieces XOR-swizzled
// by (row >> 1) & 7.  The piece that `lane` brings to row `row` of a tile that starts
// at row `first` of [rows, K], in the first step; `back`: in the line's second half.
struct LinePiece {
  uint32_t off;
  bool back;
};
constexpr LinePiece line_piece(int row, int lane, int first, int rows, int K) {
  const int piece = (lane & 7) ^ ((row >> 1) & 7);
  return {first + row < rows ? (uint32_t)((int64_t)(first + row) * K + piece * 16) : kPast, piece >= 4};
}
// The lane's offset in a step; ends: the one that K ends in the middle of.
constexpr uint32_t line_at(const LinePiece& p, bool ends) { return ends && p.back ? kPast : p.off; }

// Single tokens: load q of a run of 256 columns takes 64 of them from column kc + 256
// run on, out of `cols` that follow kc.  Past those it reads the row's start instead,
// which meets zeros of X.
constexpr uint32_t run_at(int q, int run, int cols, int kc) {
  return 256 * run + 64 * q < cols ? (uint32_t)(kc + 256 * run + 64 * q) : 0u;
}

}  // namespace qlk
