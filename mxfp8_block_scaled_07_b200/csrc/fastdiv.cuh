#pragma once
#include <cstdint>

namespace mx {

// Quotients by a divisor known at launch: n / d = (n * mul) >> (31 + shift) for 0 <= n < 2^31, with shift =
// ceil(log2 d) and mul = ceil(2^(31 + shift) / d) < 2^32: the error of mul adds less than 1 / d to the quotient.
// (A 64-bit division is a subroutine of some 70 instructions; two of them per 16-byte store are what these
// kernels' time went into.)
struct FastDiv {
    uint32_t d, mul, shift;
    static FastDiv of(int64_t d) {
        uint32_t s = 0;
        while ((int64_t(1) << s) < d) ++s;
        return {static_cast<uint32_t>(d), static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d), s};
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> (31 + shift));
    }
};

}  // namespace mx
