// Sizes and places of the cross entropy's scratch, which are arithmetic alone.
#pragma once

#include <stdint.h>

namespace ra {

constexpr uint64_t kCeTile = 256;                  // rows and columns of a result that a tile has
constexpr uint64_t kCePieceBytes = 192ull << 20;   // of g, at most (but kCeLeastPiece columns)
constexpr uint64_t kCeLeastPiece = 1024;
constexpr uint64_t kCePairs = 76;                  // pairs of CTAs: one on each two of the 152 SMs
constexpr uint64_t kCeMostParts = 1216;            // CTAs of the first kernel
constexpr uint64_t kCeMostSplits = 64;             // of the words that dh sums over

inline uint64_t round_up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

// Where the scratch's parts start, in bytes from its first multiple of 256.
struct CePlan {
  uint64_t rows_pad, cols_pad;  // hidden's copy: whole tiles of rows, rows of whole blocks of 64
  uint64_t part_rows, parts;    // rows of a CTA of the first kernel, and how many there are
  uint64_t words;               // of a tile of logits: 256, or as many less as share them out evenly
  uint64_t slots;               // forward: partial sums per row
  uint64_t piece, pieces;       // backward: columns of a piece of g (whole tiles), and how many there are
  uint64_t splits;              // backward: shares of a piece's words that dh is summed over apart
  uint64_t counters, tops, index, where, target, lse, dloss, logit;
  uint64_t hidden, weight;      // copies (weight: only where it is not read in place)
  uint64_t partial;             // forward
  uint64_t g[2], dhidden;       // backward
  uint64_t bytes;
};
constexpr uint64_t kCeHeader = 256;

inline CePlan ce_plan(uint64_t rows, uint64_t cols, uint64_t vocab, bool packed, bool backward) {
  CePlan p = {};
  p.rows_pad = round_up(rows ? rows : 1, kCeTile);
  p.cols_pad = round_up(cols, 64);
  p.part_rows = round_up((rows + kCeMostParts - 1) / kCeMostParts, 8);
  if (p.part_rows == 0) p.part_rows = 8;
  p.parts = rows ? (rows + p.part_rows - 1) / p.part_rows : 1;
  // Pieces of about one size, so that no launch is a small one. With few rows all words are one piece, although they are read
  // a second time from HBM then: pieces whose words stay in L2 (61 x 1024 x 50257 bf16: 2 pieces 97 us a call, 4 121, one 79)
  // pay more for their launches' ends.
  uint64_t most = kCePieceBytes / (2 * p.rows_pad) / kCeTile;
  if (most < kCeLeastPiece / kCeTile) most = kCeLeastPiece / kCeTile;
  const uint64_t tiles = (vocab + kCeTile - 1) / kCeTile;
  p.pieces = (tiles + most - 1) / most;
  if (p.pieces) {
    const uint64_t each = (tiles + p.pieces - 1) / p.pieces;
    p.piece = each * kCeTile;
    p.pieces = (tiles + each - 1) / each;
    // few rows make few tiles of dh, each a sum over all words of a piece: as many shares as keep a tile's work below
    // half of a pair's, in blocks of 64 summed elements. Storing a tile's results counts as 3 of them (61 x 1024 x 50257 /
    // 200 x 1024 x 50257 / 500 x 768 x 32000 bf16, us a call: 1: 82.8 / 86.3 / 73.2, 2: 81.0 / 85.1 / 73.2, 3: 78.5 / 86.9 /
    // 72.7, 4: 78.2 / 89.2 / 72.7, 6: 80.6 / 91.7 / 75.5).
    constexpr uint64_t kCeStore = 3;
    const uint64_t across = (cols + kCeTile - 1) / kCeTile, words = p.piece / 64;
    const uint64_t dh = p.rows_pad / kCeTile * across;
    const uint64_t work = dh * words + (words / 4) * across * ((rows + 63) / 64 + kCeStore) + p.rows_pad / kCeTile * (words / 4) * ((cols + 63) / 64 + kCeStore);
    const uint64_t most_words = work / (2 * kCePairs) + 1;
    p.splits = (words + most_words - 1) / most_words;
    if (p.splits > words / 8) p.splits = words / 8;  // none below 512 words
    if (p.splits > kCeMostSplits) p.splits = kCeMostSplits;
    if (p.splits < 1) p.splits = 1;
  }
  p.words = kCeTile;
  if (!backward || p.pieces == 1) {
    // where the pairs take few tiles each, narrower ones that make a whole number for every pair
    const uint64_t high = p.rows_pad / kCeTile, turns = (high * tiles + kCePairs - 1) / kCePairs;
    const uint64_t most_tiles = turns * kCePairs / high;
    if (turns && turns <= 8) p.words = round_up((vocab + most_tiles - 1) / most_tiles, 32);
    if (p.words > kCeTile) p.words = kCeTile;
    if (p.words < 64) p.words = 64;
  }
  p.slots = (vocab + p.words - 1) / p.words * 2;
  uint64_t at = kCeHeader;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  p.counters = take((p.pieces + 1) * 4);
  p.tops = take(p.parts * 4);
  p.index = take(p.rows_pad * 4);
  p.where = take(p.rows_pad * 4);
  p.target = take(p.rows_pad * 4);
  p.hidden = take(p.rows_pad * p.cols_pad * 2);
  p.weight = packed ? take(vocab * p.cols_pad * 2) : 0;
  if (backward) {
    p.lse = take(p.rows_pad * 4);
    p.dloss = take(p.rows_pad * 4);
    p.g[0] = take(p.rows_pad * p.piece * 2);
    p.g[1] = p.pieces > 1 ? take(p.rows_pad * p.piece * 2) : p.g[0];
    p.dhidden = take(p.splits * rows * p.cols_pad * 4);
  } else {
    p.logit = take(p.rows_pad * 4);
    p.partial = take(p.rows_pad * p.slots * 8);
  }
  p.bytes = at + 255;
  return p;
}

}  // namespace ra
