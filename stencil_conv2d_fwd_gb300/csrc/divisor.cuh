// Division by a number that the host knows.
#pragma once

#include <cstdint>

namespace sc {

// n / d for n below 2^31 by one multiplication: m = ceil(2^(31 + s) / d), s = ceil(log2 d).
struct Divisor {
    uint32_t d, m, s;
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const
    {
        return (uint32_t)((unsigned long long)n * m >> 31 >> s);
    }
};
inline Divisor make_divisor(int d)
{
    uint32_t s = 0;
    while ((1u << s) < (uint32_t)d) ++s;
    return Divisor{(uint32_t)d, (uint32_t)(((1ull << (31 + s)) + d - 1) / d), s};
}

}  // namespace sc
