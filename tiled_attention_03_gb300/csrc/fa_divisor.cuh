// fa_divisor.cuh -- division by a number that the host knows, as a product (internal).
#pragma once

#include <cstdint>

namespace fa {

// Division of 0 <= n < 2^31 by d as a product: mul = ceil(2^s / d), s = 31 + ceil(log2 d).
struct Divisor {
    uint32_t mul;
    int shift;
    __device__ __forceinline__ int of(int n) const {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
    }
};
inline Divisor divisor(int64_t d) {
    int l = 0;
    while ((int64_t{1} << l) < d) ++l;
    return Divisor{static_cast<uint32_t>(((uint64_t{1} << (31 + l)) + d - 1) / d), 31 + l};
}

}  // namespace fa
