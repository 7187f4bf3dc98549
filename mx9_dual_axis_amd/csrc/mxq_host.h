// Host-side argument checks shared by the C-ABI files.
#pragma once

#include <stdint.h>

namespace {

constexpr uint64_t kMaxThreads = 0xFFFFFFFFull - 256;   // grid.x * block.x must fit 32 bits

struct Span {
    uintptr_t p;
    uint64_t n;   // bytes
};

inline bool overlap(const Span& a, const Span& b) {
    return a.n != 0 && b.n != 0 && a.p < b.p + b.n && b.p < a.p + a.n;
}

inline bool any_overlap(const Span* s, int k) {
    for (int i = 0; i < k; ++i)
        for (int j = i + 1; j < k; ++j)
            if (overlap(s[i], s[j])) return true;
    return false;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// No device buffer spans more bytes than a 48-bit virtual address space.
constexpr uint64_t kMaxSpan = uint64_t(1) << 48;
constexpr uint64_t kTooLarge = ~uint64_t(0);

// Bytes spanned by a [rows, cols] matrix with row pitch ld (elements), or
// kTooLarge when that exceeds kMaxSpan (computed without overflow).
inline uint64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t esz) {
    if (rows <= 0 || cols <= 0) return 0;
    const unsigned __int128 b =
        (static_cast<unsigned __int128>(rows - 1) * uint64_t(ld) + uint64_t(cols)) * uint64_t(esz);
    return b > kMaxSpan ? kTooLarge : uint64_t(b);
}

}  // namespace
