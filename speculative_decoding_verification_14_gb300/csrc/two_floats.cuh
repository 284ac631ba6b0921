// two_floats.cuh -- numbers kept in two floats, h + l with |l| at most half a unit of h's last place: sums and
// products by the exact transformations of Knuth, Dekker and (with a fused multiply-add) Ogita, Rump and Oishi, and
// exp and ln by series.  A 64-bit operation costs this GPU some 140 cycles where a row's loss waits for it (a chain
// of fifty took 4 us a row); these take a few float instructions each.  Plain C++ too, so that a host can test it.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define SV_TWO __host__ __device__ __forceinline__
#else
#define SV_TWO inline
#endif

namespace sv {

struct Two {
    float h, l;
};

SV_TWO float two_mul_rn(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fmul_rn(a, b);
#else
    volatile float p = a * b;
    return p;
#endif
}
// a + b
SV_TWO Two two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return Two{s, (a - (s - t)) + (b - t)};
}
// the same for |a| >= |b| or a = 0
SV_TWO Two two_fast(float a, float b) {
    const float s = a + b;
    return Two{s, b - (s - a)};
}
SV_TWO Two two_add(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    return two_fast(s.h, s.l + (a.l + b.l));
}
SV_TWO Two two_mul(Two a, Two b) {
    const float p = two_mul_rn(a.h, b.h);
    const float e = fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, two_mul_rn(a.l, b.h));
    return fabsf(p) <= 3.4028235e38f ? two_fast(p, e) : Two{p, 0.0f};
}
SV_TWO Two two_neg(Two a) { return Two{-a.h, -a.l}; }
SV_TWO Two two_div(Two a, Two b) {
    const float q = a.h / b.h;
    const float r = fmaf(-q, b.h, a.h) + fmaf(-q, b.l, a.l);
    return two_fast(q, r / b.h);
}

// exp: x = n ln 2 + r, |r| < 0.35, and 1 + r + r^2 / 2 + r^3 (1/6 + r / 24 + ...), the series to r^9 with its first three
// terms in two floats: 2^-28 of itself at worst (20 million arguments on a host).  ln 2 as 2839 / 4096, whose products with n are exact, and the rest.  Below -86 (which
// float's normal numbers end at): 0, above 88 infinity.
SV_TWO Two two_exp(Two x) {
    if (!(x.h > -86.0f))
        return Two{x.h == x.h ? 0.0f : x.h, 0.0f};
    if (x.h > 88.0f)
        return Two{INFINITY, 0.0f};
    const float n = rintf(x.h * 1.44269504f);
    Two r = two_sum(fmaf(n, -2839.0f / 4096.0f, x.h), fmaf(n, -3.19461850e-5f, x.l));
    const float s = two_mul_rn(r.h, r.h), sl = fmaf(r.h, r.h, -s) + 2.0f * two_mul_rn(r.h, r.l);
    float q = fmaf(r.h, 1.0f / 362880.0f, 1.0f / 40320.0f);
    q = fmaf(r.h, q, 1.0f / 5040.0f);
    q = fmaf(r.h, q, 1.0f / 720.0f);
    q = fmaf(r.h, q, 1.0f / 120.0f);
    q = fmaf(r.h, q, 1.0f / 24.0f);
    q = fmaf(r.h, q, 1.0f / 6.0f);
    const Two a = two_fast(1.0f, r.h), b = two_sum(0.5f * s, two_mul_rn(two_mul_rn(s, r.h), q));
    const Two c = two_add(Two{a.h, a.l}, Two{b.h, b.l + (r.l + 0.5f * sl)});
    const uint32_t bits = (uint32_t)(127 + (int)n) << 23;
    float scale;
#ifdef __CUDA_ARCH__
    scale = __uint_as_float(bits);
#else
    std::memcpy(&scale, &bits, 4);
#endif
    return Two{c.h * scale, c.l * scale};
}

// ln of a normal x > 0: x = 2^e m, m from 0.7 to 1.42, ln m = 2 artanh((m - 1) / (m + 1)), the quotient in two floats and
// the series of artanh to its eleventh power: 2^-29 at worst.
SV_TWO Two two_log(Two x) {
    int32_t bits;
#ifdef __CUDA_ARCH__
    bits = __float_as_int(x.h);
#else
    std::memcpy(&bits, &x.h, 4);
#endif
    const int e = (bits - 0x3f3504f3) >> 23;  // m from sqrt(1/2) on
    const int32_t down = bits - (e << 23), half1 = (127 - e / 2) << 23, half2 = (127 - (e - e / 2)) << 23;
    float m, s1, s2;
#ifdef __CUDA_ARCH__
    m = __int_as_float(down), s1 = __int_as_float(half1), s2 = __int_as_float(half2);
#else
    std::memcpy(&m, &down, 4), std::memcpy(&s1, &half1, 4), std::memcpy(&s2, &half2, 4);
#endif
    const float ml = x.l * s1 * s2;
    const Two den = two_sum(m, 1.0f);
    const float num = m - 1.0f;  // exact
    const Two s = two_div(Two{num, ml}, Two{den.h, den.l + ml});
    const float p = two_mul_rn(s.h, s.h);
    float q = fmaf(p, 1.0f / 11.0f, 1.0f / 9.0f);
    q = fmaf(p, q, 1.0f / 7.0f);
    q = fmaf(p, q, 0.2f);
    q = fmaf(p, q, 1.0f / 3.0f);
    const Two t = two_fast(2.0f * s.h, 2.0f * fmaf(two_mul_rn(s.h, p), q, s.l));
    const float fe = (float)e;
    return two_add(Two{fe * (2839.0f / 4096.0f), fe * 3.19461850e-5f}, t);
}

}  // namespace sv
