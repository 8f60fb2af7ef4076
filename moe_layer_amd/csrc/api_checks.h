// Argument checks shared by the C ABI of the operators around the layer
// (rows_api.hip, sorted_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "moe.h"

namespace moe {

namespace {

constexpr int32_t kMaxRows = 1 << 30;   // row indices plus a block stay in 32 bits
constexpr int32_t kMaxCols = 1 << 20;   // and byte counts in 64

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
    const void* p;
    int64_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + uintptr_t(b.bytes) && b0 < a0 + uintptr_t(a.bytes);
}
// any output over an input or another output; each of the first `in_place` outputs
// may be one of the first `in_place` inputs itself
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins, int in_place) {
    int i = 0;
    for (const Span& o : outs) {
        int k = 0;
        for (const Span& n : ins) {
            const bool itself = i < in_place && k < in_place && o.p == n.p && o.bytes == n.bytes;
            if (overlap(o, n) && !itself) return true;
            ++k;
        }
        int j = 0;
        for (const Span& other : outs)
            if (j++ > i && overlap(o, other)) return true;
        ++i;
    }
    return false;
}

}  // namespace

}  // namespace moe
