// Sizes and places of the cross entropy's scratch, which are arithmetic alone.
#pragma once

#include <stdint.h>

namespace ra {

constexpr uint64_t kCeTile = 256;                  // rows and columns of the logits that a tile has
constexpr uint64_t kCePieceBytes = 256ull << 20;   // of g, at most (but kCeLeastPiece columns)
constexpr uint64_t kCeLeastPiece = 1024;

inline uint64_t round_up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

// Where the scratch's parts start, in bytes from its own start.
struct CePlan {
  uint64_t rows_pad, cols_pad;  // hidden's copy: whole tiles of rows, rows of whole 16-byte lines
  uint64_t slots;               // forward: partial sums per row
  uint64_t piece, pieces;       // backward: columns of a piece of g (whole tiles), and how many there are
  uint64_t index, where, target, lse, dloss, logit;  // per row
  uint64_t hidden, weight;                           // copies (weight: only where it is not read in place)
  uint64_t partial;                                  // forward
  uint64_t g, dhidden;                               // backward
  uint64_t bytes;
};
constexpr uint64_t kCeHeader = 256;

inline CePlan ce_plan(uint64_t rows, uint64_t cols, uint64_t vocab, bool packed, bool backward) {
  CePlan p = {};
  p.rows_pad = round_up(rows ? rows : 1, kCeTile);
  p.cols_pad = round_up(cols, 8);
  p.slots = (vocab + 255) / 256 * 2;
  const uint64_t most = kCePieceBytes / (2 * p.rows_pad) / kCeTile * kCeTile;
  p.piece = most < kCeLeastPiece ? kCeLeastPiece : most;
  if (p.piece > round_up(vocab, kCeTile)) p.piece = round_up(vocab, kCeTile);
  p.pieces = (vocab + p.piece - 1) / p.piece;
  uint64_t at = kCeHeader;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  p.index = take(p.rows_pad * 4);
  p.where = take(p.rows_pad * 4);
  p.target = take(p.rows_pad * 4);
  p.hidden = take(p.rows_pad * p.cols_pad * 2);
  p.weight = packed ? take(vocab * p.cols_pad * 2) : 0;
  if (backward) {
    p.lse = take(p.rows_pad * 4);
    p.dloss = take(p.rows_pad * 4);
    p.g = take(p.rows_pad * p.piece * 2);
    p.dhidden = take(p.rows_pad * p.cols_pad * 4);
  } else {
    p.logit = take(p.rows_pad * 4);
    p.partial = take(p.rows_pad * p.slots * 8);
  }
  p.bytes = at;
  return p;
}

}  // namespace ra
