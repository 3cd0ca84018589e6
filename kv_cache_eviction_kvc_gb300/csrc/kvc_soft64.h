// kvc_soft64.h -- the fp64 addition of a utility update by integer arithmetic,
// rounded as IEEE 754 asks (to nearest, ties to even).
//
// fp64 instructions are scarce on this part (tens of clocks of an SM for a
// warp's addition), integer ones are not: an addition here is about 40 of them.
// (A multiply-add is about 150: measured slower than the hardware's two
// operations, so the EMA rule keeps those.)  Only for the operands that
// utilities are made of, positive normal numbers far from the ends of the
// range; the caller keeps the hardware's addition for the rest.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVC_HD __host__ __device__ __forceinline__
#else
#define KVC_HD inline
#endif

namespace kvc {

constexpr uint64_t kOne52 = 1ull << 52;

// A positive normal number between 2^-700 and 2^700, as bits.
KVC_HD bool soft_normal(uint64_t b) { return (b >> 52) - 323u <= 1400u; }

// A positive normal fp32 number (as bits) as fp64 bits.
KVC_HD uint64_t soft_widen(uint32_t b)
{
    return ((uint64_t)b << 29) + ((uint64_t)(1023 - 127) << 52);
}

// a + b of two positive normal numbers.
KVC_HD uint64_t soft_add(uint64_t a, uint64_t b)
{
    const uint64_t x = a > b ? a : b, y = a > b ? b : a;
    const int d = (int)(x >> 52) - (int)(y >> 52);
    // three bits below the last: the larger's are zero, the smaller's lowest
    // stands for all that is shifted out
    const uint64_t mx = ((x & (kOne52 - 1)) | kOne52) << 3, my = ((y & (kOne52 - 1)) | kOne52) << 3;
    const int s = d < 60 ? d : 60;
    uint64_t sum = mx + (my >> s | ((my & ((1ull << s) - 1)) != 0 ? 1 : 0));
    uint64_t e = x >> 52;
    if (sum >> 56) {
        sum = (sum >> 1) | (sum & 1);
        e++;
    }
    const uint64_t q = sum >> 3, r = sum & 7;
    // (a mantissa that rounds up to 2^53 carries into the exponent)
    return (e << 52) + (q - kOne52) + (r + (q & 1) > 4 ? 1 : 0);
}

}  // namespace kvc
