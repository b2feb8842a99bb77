// Host-side argument checks that the ABI files of the block's operators share.
#pragma once

#include <stdint.h>

namespace fp8g {

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

// a * b * c, or -1 past 2^60
inline int64_t mul3(int64_t a, int64_t b, int64_t c) {
    const int64_t lim = (int64_t)1 << 60;
    if (a == 0 || b == 0 || c == 0) return 0;
    if (a > lim / b) return -1;
    const int64_t ab = a * b;
    if (ab > lim / c) return -1;
    return ab * c;
}

// `count` runs of `width` bytes, `stride` bytes apart
struct Rows {
    uintptr_t at;
    uint64_t count, width, stride;
};
inline Rows rows_of(const void* p, int64_t count, int64_t width, int64_t stride) {
    return Rows{reinterpret_cast<uintptr_t>(p), (uint64_t)count, (uint64_t)width, (uint64_t)stride};
}
inline Rows bytes_of(const void* p, int64_t bytes) { return rows_of(p, 1, bytes, bytes); }

inline bool overlaps(const Rows& a, const Rows& b) {
    if (!a.count || !b.count || !a.width || !b.width) return false;
    const uintptr_t a_end = a.at + (a.count - 1) * a.stride + a.width, b_end = b.at + (b.count - 1) * b.stride + b.width;
    if (a_end <= b.at || b_end <= a.at) return false;
    if (a.count > 1 && b.count > 1 && a.stride == b.stride) {
        // side by side in the same rows (q and k of one projection): their
        // places modulo the stride decide
        const uint64_t off = a.at < b.at ? (b.at - a.at) % a.stride : (a.stride - (a.at - b.at) % a.stride) % a.stride;
        return !(off >= a.width && off + b.width <= a.stride);
    }
    return true;
}

}  // namespace fp8g
