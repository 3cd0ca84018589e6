// kvc_soft64.h -- the two fp64 operations of a utility update, by integer
// arithmetic, rounded as IEEE 754 asks (to nearest, ties to even).
//
// fp64 instructions are scarce on this part (measured: a warp's addition every
// 88 clocks of an SM), integer ones are not: an addition here is about 40 of
// them, a multiply-add of a product about 110.  Only for the operands
// that utilities are made of (zero and positive normal numbers far from the
// ends of the range); the caller keeps the hardware's operation for the rest.
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

KVC_HD int soft_clz(uint64_t x)
{
#ifdef __CUDA_ARCH__
    return __clzll((long long)x);
#else
    return __builtin_clzll(x);
#endif
}

KVC_HD uint64_t soft_mulhi(uint64_t a, uint64_t b)
{
#ifdef __CUDA_ARCH__
    return __umul64hi(a, b);
#else
    return (uint64_t)((unsigned __int128)a * b >> 64);
#endif
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

// hi:lo shifted right by s (0..127), bits shifted out left in the lowest.
KVC_HD void soft_shr(uint64_t &hi, uint64_t &lo, int s)
{
    if (s >= 64) {
        lo = hi | (lo != 0 ? 1 : 0);
        hi = 0;
        s -= 64;
    }
    if (s == 0) return;
    const uint64_t out = lo << (64 - s);
    lo = lo >> s | hi << (64 - s) | (out != 0 ? 1 : 0);
    hi >>= s;
}

// b x of a positive normal b and a positive normal fp32 x (as bits), rounded.
KVC_HD uint64_t soft_mul(uint64_t b, uint32_t x)
{
    const uint64_t m = (b & (kOne52 - 1)) | kOne52, f = (x & 0x7fffffu) | 0x800000u;
    // 77 bits at most: the product's upper 45 and lower 32
    const uint64_t lo = (m & 0xffffffffu) * f, up = (m >> 32) * f + (lo >> 32);
    const int over = (int)(up >> 44);                        // 2^76 and above
    const uint64_t low = up << 32 | (lo & 0xffffffffu);
    const int drop = 23 + over;
    const uint64_t q = up << (32 - drop) | (lo & 0xffffffffu) >> drop;
    const uint64_t rem = low & ((1ull << drop) - 1), half = 1ull << (drop - 1);
    const uint64_t e = (b >> 52) + (x >> 23) - 127 + over;
    return (e << 52) + (q - kOne52) + (rem + (q & 1) > half ? 1 : 0);
}

// a m + p, rounded once; a and m positive normal numbers, p one or zero.
KVC_HD uint64_t soft_fma(uint64_t a, uint64_t m, uint64_t p)
{
    const uint64_t ma = (a & (kOne52 - 1)) | kOne52, mm = (m & (kOne52 - 1)) | kOne52;
    // the product's 106 bits at 124 or 125 downwards, p's 53 at 124 downwards
    uint64_t xh = soft_mulhi(ma << 11, mm << 9), xl = (ma << 11) * (mm << 9);
    uint64_t ph = p ? ((p & (kOne52 - 1)) | kOne52) << 8 : 0, pl = 0;
    // exponents of bit 124, biased by 1023
    const int ex = (int)(a >> 52) + (int)(m >> 52) - 1023, ep = p ? (int)(p >> 52) : ex;
    const int d = ex - ep, s = d < 0 ? -d : d;
    if (d >= 0) soft_shr(ph, pl, s < 127 ? s : 127);
    else soft_shr(xh, xl, s < 127 ? s : 127);
    const uint64_t l = xl + pl, h = xh + ph + (l < xl ? 1 : 0);
    // the highest bit is 124, 125 or 126 (60 .. 62 of the upper word)
    const int top = 63 - soft_clz(h), drop = top - 52;
    const uint64_t q = h >> drop, rem = (h & ((1ull << drop) - 1)) << 1 | (l != 0 ? 1 : 0);
    const uint64_t half = 1ull << drop;
    const uint64_t e = (uint64_t)((d >= 0 ? ex : ep) + top - 60);
    return (e << 52) + (q - kOne52) + (rem + (q & 1) > half ? 1 : 0);
}

}  // namespace kvc
