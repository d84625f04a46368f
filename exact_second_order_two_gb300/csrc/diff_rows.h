// Which query rows a part of the CUDA-core dK/dV pass walks over.  Host code as
// well, so that the arithmetic can be checked at sizes too long to run.
#pragma once

#ifdef __CUDACC__
#define FBOB_HD __host__ __device__ __forceinline__
#else
#define FBOB_HD inline
#endif

namespace fbob {

struct RowRange {
  int first, end;
};

// Rows of head g of a group, in the part that takes the tiles t0 .. t1 - 1 of the
// group's heads (per_head tiles of `tile` rows each, from row `start` on, N rows).
// The heads behind g count in t1: their tiles are left out before they are
// turned into rows, which all of a group's heads together need not fit in 31
// bits.
FBOB_HD RowRange part_rows(int t0, int t1, int g, int per_head, int start, int N, int tile) {
  const int from = t0 - g * per_head, to = t1 - g * per_head;
  const int end = start + (to < per_head ? to : per_head) * tile;
  return {start + (from > 0 ? from : 0) * tile, end < N ? end : N};
}

}  // namespace fbob
