// What the join of the shared-prefix attention reads for one head, from the entry that the
// attention kernel left for it.  Host and device: the bounds are checked on the CPU.
//
// An entry holds the first and the last slot with a partial of the head's group, and the row of its
// first query among the slot's rows.  A call that gave up waiting leaves entries as the workspace held
// them, which is anything; whatever they say, the reads stay within the workspace.
#pragma once

#if defined(__CUDACC__)
#define ARKV_JOIN_FN __host__ __device__ __forceinline__
#else
#define ARKV_JOIN_FN inline
#endif

namespace arkv {

struct JoinSpan {
    int first, last;   // slots, none if last < first; 0 <= first <= slots, last < slots
    int row;           // 0 .. row_tiles * tile_rows - group
};

ARKV_JOIN_FN JoinSpan join_span(int first, int last, int row, int slots, int row_tiles, int tile_rows, int group) {
    JoinSpan s;
    s.first = first < 0 ? 0 : first > slots ? slots : first;
    s.last = last < slots ? last : slots - 1;
    const int most = row_tiles * tile_rows - group;
    s.row = row < 0 ? 0 : row > most ? most : row;
    return s;
}

}  // namespace arkv
