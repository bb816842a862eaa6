// Division by a constant of a launch, for the host (which finds the multiplier)
// and the kernels.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define NVFP4_BOTH __host__ __device__ __forceinline__
#else
#define NVFP4_BOTH inline
#endif

namespace nvfp4 {

// Division of a 31-bit number by a constant of the launch: n / d =
// (n * mul) >> 32 >> shift, exact for n < 2^31 (mul = ceil(2^(32 + shift) /
// d) with 2^shift >= d; then mul d - 2^(32 + shift) < d <= 2^shift, and the
// error n (mul d - 2^(32 + shift)) / (d 2^(32 + shift)) stays below 1 / d).
struct DivBy {
    uint32_t d;
    uint64_t mul;
    uint32_t shift;

    static DivBy of(uint32_t d)
    {
        uint32_t s = 0;
        while (((uint64_t)1 << s) < d)
            ++s;
        const uint64_t one = (uint64_t)1 << s;
        // ceil(2^32 * 2^s / d) in 64 bits: s <= 31
        return DivBy{d, ((one << 32) + d - 1) / d, s};
    }
    NVFP4_BOTH uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> 32 >> shift); }
};

}  // namespace nvfp4
