// Sizes and places of the embedding gradient's scratch, which are arithmetic alone.
#pragma once

#include <stdint.h>

namespace ra {

constexpr uint64_t kEmbOneSort = 32768;      // tokens that a cluster sorts, at most: their places take 15 bits of a word
constexpr uint64_t kEmbOneVocab = 1u << 17;  // and their numbers, or `vocab` for none, the other 17
constexpr uint64_t kEmbSortTile = 4096;      // tokens that a CTA takes at a time where there are more
constexpr uint64_t kEmbSortCtas = 304;       // CTAs of a sorting pass, at most: each reads the counts of all
constexpr uint64_t kEmbSumWarps = 8;         // of a CTA that adds up

struct EmbPlan {
  bool one;              // a cluster sorts
  uint32_t bits, passes; // of a digit, and digits of a number
  uint64_t tiles, ctas;  // of 4096 tokens, one behind the other in each CTA of a sorting pass (not one)
  uint64_t span, spans;  // sorted places that a CTA adds up, a share to each warp, and how many such spans there are
  uint64_t across;       // CTAs side by side on a row
  uint64_t keys[2], places[2], counts, tickets, partial;  // in bytes from the scratch's start
  uint64_t bytes;
};

// `per_lane`: columns of a lane, 8 or 4.
inline EmbPlan emb_plan(uint64_t rows, uint64_t cols, uint64_t vocab, uint64_t per_lane) {
  EmbPlan p = {};
  p.one = rows <= kEmbOneSort && vocab < kEmbOneVocab;
  uint32_t bits = 1;
  while (bits < 32 && vocab >> bits) ++bits;
  p.passes = (bits + 7) / 8;
  p.bits = (bits + p.passes - 1) / p.passes;
  p.tiles = ((rows + kEmbSortTile - 1) / kEmbSortTile + kEmbSortCtas - 1) / kEmbSortCtas;
  p.ctas = p.tiles ? (rows + kEmbSortTile * p.tiles - 1) / (kEmbSortTile * p.tiles) : 0;
  p.across = (cols + 32 * per_lane - 1) / (32 * per_lane);
  // short spans where they fill the device once (4 CTAs an SM), longer ones where there are more: a span's ends cost it
  // a partial sum
  p.span = kEmbSumWarps * 8;
  while (p.span < kEmbSumWarps * 32 && (rows + p.span - 1) / p.span * p.across > 152 * 4) p.span *= 2;
  p.spans = (rows + p.span - 1) / p.span;
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes_) {
    const uint64_t here = at;
    at += (bytes_ + 255) / 256 * 256;
    return here;
  };
  for (int i = 0; i < (p.one ? 1 : 2); ++i) p.keys[i] = take(rows * 4), p.places[i] = take(rows * 4);
  p.counts = p.one ? 0 : take(p.ctas * 256 * 4);
  p.tickets = take(p.spans * p.across * 4);
  p.partial = take(p.spans * 2 * p.across * 32 * per_lane * 4);
  p.bytes = at + 16;
  return p;
}

}  // namespace ra
