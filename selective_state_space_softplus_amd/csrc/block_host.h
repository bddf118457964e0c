// block_host.h -- argument checks shared by the host sides of the block's operators.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "ss_block.h"

#define SS_EXPORT extern "C" __attribute__((visibility("default")))

namespace ss_block {

constexpr int64_t kMaxElems = int64_t(1) << 46;   // keeps every index product far from int64 overflow

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};

inline Range range_of(const void* p, int64_t count, size_t elem) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + uintptr_t(count) * elem : lo};
}

inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
inline bool same(Range a, Range b) { return a.lo == b.lo && a.hi == b.hi; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t elem_size(int dtype) { return dtype == SS_BF16 ? 2 : 4; }
inline bool dtype_ok(int dtype) { return dtype == SS_F32 || dtype == SS_BF16; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
inline int status(hipError_t e) { return e == hipSuccess ? SS_OK : SS_ERR_HIP; }

// Every size at least 1 and their product at most 2^46 (no product that could overflow is formed).
inline bool sizes_ok(std::initializer_list<int64_t> sizes) {
    int64_t most = kMaxElems;
    for (int64_t s : sizes) {
        if (s <= 0 || s > most) return false;
        most /= s;
    }
    return true;
}

// No output overlaps an input or another output.
template <size_t NI, size_t NO>
bool apart(const Range (&ins)[NI], const Range (&outs)[NO]) {
    for (size_t i = 0; i < NO; i++) {
        for (const Range& r : ins)
            if (overlaps(r, outs[i])) return false;
        for (size_t j = i + 1; j < NO; j++)
            if (overlaps(outs[i], outs[j])) return false;
    }
    return true;
}

}  // namespace ss_block
