// Division by kernel arguments without a divide.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace li {

// Division of a non-negative int32 by a fixed one (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// t / d = (h + ((t - h) >> 1)) >> (l - 1) for h = floor(m t / 2^32); d = 1 apart.
struct FixedDiv {
    uint32_t m = 0;
    int32_t shift = -1;                 // l - 1, -1 for d = 1
    __host__ FixedDiv() {}
    __host__ explicit FixedDiv(uint32_t d) {
        if (d <= 1) return;
        int l = 0;
        while (((uint64_t)1 << l) < d) ++l;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1);
        shift = l - 1;
    }
    __device__ __forceinline__ int32_t div(int32_t t) const {
        if (shift < 0) return t;
        const uint32_t h = __umulhi(m, (uint32_t)t);
        return (int32_t)((h + (((uint32_t)t - h) >> 1)) >> shift);
    }
};

}  // namespace li
