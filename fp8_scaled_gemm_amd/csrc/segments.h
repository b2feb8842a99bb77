// Row blocks of ragged sequences, found on the device, and division by a number
// that a launch knows (gfx950 only).
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

// The sequence of a block, its [start, end) and a word of its own.
struct Sequence {
    int index, start, end, word;      // index -1: the block belongs to none
};

// start(b), b <= count, ascending; word(b), b < count, read alongside so that
// one round trip to memory finds everything.  All 64 lanes take part; the
// result is uniform.
template <class Start, class Word>
__device__ __forceinline__ Sequence find_sequence(Start start, Word word, int count, int mult, int rows_log2, int id) {
    const int lane = threadIdx.x & 63;
    Sequence s = {-1, 0, 0, 0};
    for (int c = 0; c < count; c += 64) {
        const int b = c + lane;
        int at = 0, end = 0, w = 0;
        if (b < count) at = start(b), end = start(b + 1), w = word(b);
        const bool below = b < count && (int)(((int64_t)at * mult) >> rows_log2) + b <= id;
        const int n = __popcll(__ballot(below));      // bases ascend: the lowest n lanes
        if (n > 0) {
            s.index = c + n - 1;
            s.start = __builtin_amdgcn_readlane(at, n - 1);
            s.end = __builtin_amdgcn_readlane(end, n - 1);
            s.word = __builtin_amdgcn_readlane(w, n - 1);
        }
        if (n < 64) break;
    }
    s.index = __builtin_amdgcn_readfirstlane(s.index);
    return s;
}

// n / d for n < 2^31 by a multiply: (mulhi(n, mul) + n) >> shift
struct FastDiv {
    uint32_t mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f;
    f.shift = 0;
    while ((1ull << f.shift) < d) f.shift++;
    f.mul = (uint32_t)((((1ull << f.shift) - d) << 32) / d + 1);
    return f;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, FastDiv f) { return (__umulhi(n, f.mul) + n) >> f.shift; }

}  // namespace fp8g
