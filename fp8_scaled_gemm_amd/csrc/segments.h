// Row blocks of ragged sequences, found on the device (gfx950 only).
//
// Sequence b owns the rows start[b] * mult .. start[b + 1] * mult - 1 of a
// launch; a workgroup handles a block of `rows` of them.  How many blocks a
// sequence has is known on the device only, so sequence b is given the block
// numbers from base(b) = floor(start[b] * mult / rows) + b on.  That leaves
// room for all of its blocks,
//   base(b + 1) - base(b) >= floor(n mult / rows) + 1 >= ceil(n mult / rows),
// needs floor(total * mult / rows) + sequences numbers in all, and finds the
// sequence of a block by counting the bases that are not above it: no prefix
// sums, and no lengths on the host.  Numbers in the gaps find nothing to do.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8g {

// Number of bases that are <= id among start[0 .. count): the sequence's index
// plus one.  All 64 lanes take part; the result is uniform.
template <class Start>
__device__ __forceinline__ int find_block(Start start, int count, int mult, int rows_log2, int id) {
    const int lane = threadIdx.x & 63;
    int found = 0;
    for (int c = 0; c < count; c += 64) {
        const int b = c + lane;
        const bool below = b < count && (int)(((int64_t)start(b) * mult) >> rows_log2) + b <= id;
        const int n = __popcll(__ballot(below));
        found += n;
        if (n < 64) break;
    }
    return __builtin_amdgcn_readfirstlane(found);
}

}  // namespace fp8g
