// slice_edges.h -- a slice of a row in pieces of 16 bytes as they lie in memory, and which of them leave the matrix.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PULSE_BOTH_SIDES __host__ __device__ __forceinline__
#else
#define PULSE_BOTH_SIDES inline
#endif

namespace pulse {

struct SliceEdges {
  uint32_t pieces;
  bool low, high;  // the first piece begins before the matrix, the last one ends behind it
};

// `count` elements from element `at` of a matrix that spans `span` elements (from its first to its last, gaps between rows
// included), `lead` elements into a piece of `piece`. A slice can be shorter than a piece, and a matrix too: then rows other
// than the first and the last have such pieces, and one piece can leave at both ends. Pieces between the first and the last
// are of the slice alone.
PULSE_BOTH_SIDES SliceEdges slice_edges(uint64_t at, uint32_t count, uint32_t lead, uint32_t piece, uint64_t span) {
  SliceEdges e;
  e.pieces = (lead + count + piece - 1) / piece;
  e.low = e.pieces != 0 && at < lead;
  e.high = e.pieces != 0 && at + uint64_t(e.pieces) * piece > span + lead;
  return e;
}

}  // namespace pulse
