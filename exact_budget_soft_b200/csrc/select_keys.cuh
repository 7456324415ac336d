// select_keys.cuh -- scores as ordered keys, and ranges of keys as bounds of scores
// (host and device: the host tests compile this file by itself).
#pragma once
#include <cmath>
#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define SEL_BOTH __host__ __device__ __forceinline__
#else
#define SEL_BOTH inline
#endif

namespace lapsum {

SEL_BOTH uint32_t sel_bits(float f) {
#ifdef __CUDA_ARCH__
    return __float_as_uint(f);
#else
    uint32_t u;
    std::memcpy(&u, &f, 4);
    return u;
#endif
}
SEL_BOTH float sel_float(uint32_t u) {
#ifdef __CUDA_ARCH__
    return __uint_as_float(u);
#else
    float f;
    std::memcpy(&f, &u, 4);
    return f;
#endif
}

// Order-preserving key of the selection, ASCENDING with the score: -0 and +0
// share a key, a NaN gets 0, below -inf (0x007fffff).
SEL_BOTH uint32_t sel_key(float f) {
    const uint32_t u = sel_bits(f + 0.0f);   // -0 + 0 = +0
    const uint32_t k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return f != f ? 0u : k;
}

// The score of a key.
SEL_BOTH float sel_value(uint32_t key) {
    return sel_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// A range of keys as bounds of scores: of a score f, f >= lo says that its key is in
// the range or above, f > hi that it is above (a range that takes in NaN, the key 0,
// says so: its passes compare keys).  No score has the key 0x7fffffff: as a bound it
// would be -0, which no zero is above, so a range that ends there ends one key lower.
struct SelRange {
    float lo, hi;
    bool nan;
    SEL_BOTH SelRange(uint32_t first, uint32_t span) {
        constexpr uint32_t MINUS_INF = 0x007fffffu, MINUS_ZERO = 0x7fffffffu;
        const uint32_t last = first + span;
        nan = first == 0u;
        lo = first <= MINUS_INF ? -INFINITY : sel_value(first);
        hi = last < MINUS_INF ? -INFINITY : sel_value(last == MINUS_ZERO ? last - 1u : last);   // beyond +inf: a NaN, nothing is above
    }
};

}  // namespace lapsum
