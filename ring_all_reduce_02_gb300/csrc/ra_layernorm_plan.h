// Launch shapes of layer norm that are arithmetic alone.
#pragma once

#include <stdint.h>

namespace ra {

// Clusters of CTAs to launch where each takes every so manyth row and the device holds `fit` of them at once (a second
// wave would take as long again); never more than there are rows. Rows that share a phase are `phases` apart (1 on
// the 16-byte grid), and a cluster's rows have to: the number is a multiple of it, unless each cluster has one row.
// 0: there is no such number, the device holds too few.
inline uint64_t late_clusters(uint64_t fit, uint64_t rows, uint64_t phases) {
  return rows <= fit ? rows : fit / phases * phases;
}

}  // namespace ra
