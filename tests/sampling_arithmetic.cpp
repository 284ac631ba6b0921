// The sampling kernels' arithmetic on weights (sampling_weights.cuh), run on the host and
// measured against long doubles: 64 bits and more, good to 2^-60 here.  Built without
// contraction, as the header writes its fused operations out.  Prints a line "name value"
// for each figure the tests ask about.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>

using std::max;
using std::min;
#define __CUDACC__
#define __device__
#define __forceinline__ inline
struct float2 {
    float x, y;
};
static inline float2 make_float2(float x, float y) { return {x, y}; }
static inline uint32_t __float_as_uint(float f) {
    uint32_t u;
    std::memcpy(&u, &f, 4);
    return u;
}
static inline int __float_as_int(float f) { return (int)__float_as_uint(f); }
static inline float __uint_as_float(uint32_t u) {
    float f;
    std::memcpy(&f, &u, 4);
    return f;
}
static inline float __int_as_float(int i) { return __uint_as_float((uint32_t)i); }
static inline long long __double_as_longlong(double d) {
    long long i;
    std::memcpy(&i, &d, 8);
    return i;
}
static inline unsigned long long __umul64hi(unsigned long long a, unsigned long long b) {
    return (unsigned long long)(((unsigned __int128)a * b) >> 64);
}
static inline float __fdiv_rn(float a, float b) { return a / b; }
static inline int __float2int_rn(float f) { return (int)lrintf(f); }
static inline long long __float2ll_rn(float f) { return llrintf(f); }
#include "../speculative_decoding_verification_14_gb300/csrc/sampling_weights.cuh"
#undef __CUDACC__

using namespace sv;

static std::mt19937_64 gen(7);

// floor(u x) and ceil(p x) against 128-bit products; the largest difference
static void shares() {
    const float us[] = {0.0f, -0.0f, 0x1p-149f, 0x1.8p-130f, 0x1p-24f, 0.3f, 0.5f, 0x1.fffffep-1f};
    uint64_t off = 0, zero = 0;
    for (int i = 0; i < 2000; ++i) {
        const uint64_t x = gen() >> (2 + gen() % 60);
        for (float u : us) {
            int e;
            const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(u), &e), 24);
            const unsigned __int128 y = (unsigned __int128)m * x;
            const int sh = 24 - e;
            const uint64_t want = sh >= 128 ? 0 : (uint64_t)(y >> sh), got = floor_scaled(u, x);
            off = max(off, want > got ? want - got : got - want);
            if (u == 0.0f)
                zero = max<uint64_t>(zero, got);
        }
        const double p = (double)(gen() >> 11) * 0x1p-53;
        if (p > 0.0) {
            int e;
            const uint64_t m = (uint64_t)std::ldexp(std::frexp(p, &e), 53);
            const int sh = 53 - e;
            const unsigned __int128 y = (unsigned __int128)m * x;
            const uint64_t want = (uint64_t)(y >> sh) + ((y & (((unsigned __int128)1 << sh) - 1)) != 0);
            const uint64_t got = ceil_scaled(p, x);
            off = max(off, want > got ? want - got : got - want);
        }
    }
    std::printf("shares_off %llu\nzero_share %llu\n", (unsigned long long)off, (unsigned long long)zero);
}

// a row's scale at an ordinary temperature, a logit of it, and the logit's weight
struct Sample {
    RowScale s;
    float l;
    long double w;
    Sample() {
        std::normal_distribution<double> normal;
        const float T = (float)(0.2 + 1.4 * (double)(gen() >> 11) * 0x1p-53);
        s.lmax = (float)(10.0 + 3.0 * normal(gen));
        s.fix = kMaxFix;
        set_temperature(s, T);
        l = s.lmax - (float)std::fabs(normal(gen)) * 9.0f * T;
        w = std::exp(((long double)l - (long double)s.lmax) / (long double)T);
    }
};

// how far a weight is off, as a share of itself, and the range of its 44 bits
static void weights() {
    long double worst = 0, least = 2, most = 0;
    for (int i = 0; i < 4000000; ++i) {
        const Sample x;
        int down;
        const unsigned long long u = weight_parts(x.s, kPow2Steps, x.l, down);
        if (down > kMaxFix)
            continue;
        worst = max(worst, std::fabs(std::ldexp((long double)u, -kMaxFix - down) / x.w - 1));
        least = min(least, std::ldexp((long double)u, -kMaxFix));
        most = max(most, std::ldexp((long double)u, -kMaxFix));
    }
    std::printf("weight_off %.9Lg\nleast_parts %.9Lg\nmost_parts %.9Lg\n", worst, least, most);
}

// how far a sum of four equal weights is off, as a share of itself: all errors agree
static void sums() {
    static float2 steps[kSteps * 16];
    long double worst = 0;
    const Units units(kMaxFix);
    for (int j = 0; j < kSteps * 16; ++j)
        steps[j] = kPow2Steps[j >> 4];
    for (int i = 0; i < 4000000; ++i) {
        const Sample x;
        if (!(std::fabs(x.s.lmax * x.s.ch) < 128.0f) || x.w < 0x1p-10L)  // small ones' share is their units'
            continue;
        SumScale t(x.s);
        t.steps = steps + (i & 15);
        WeightSum sum;
        unsigned long long n = 0;
        for (int j = 0; j < 4; ++j)
            sum.add(sum_weight(t, x.l));
        sum.into(n, units);
        n += sum.rest(kMaxFix);
        worst = max(worst, std::fabs(std::ldexp((long double)n, -kMaxFix - 2) / x.w - 1));
    }
    std::printf("sum_off %.9Lg\n", worst);
}

// how many parts a search takes to one key, and how often a part was not a smaller one inside the whole,
// whatever part the search names (2048 is what it names when it finds none)
static void key_ranges() {
    int most = 0, outside = 0;
    for (int i = 0; i < 200000; ++i) {
        KeyRange r;
        r.lo = (uint32_t)gen() >> gen() % 32;
        r.hi = max(r.lo, (uint32_t)gen() >> gen() % 32);
        if (i == 0)
            r = {0, 0xffffffffu};
        int n = 0;
        for (; r.lo != r.hi && n < 40; ++n) {
            const int shift = r.shift(2048);
            const uint32_t choice[4] = {(uint32_t)(gen() % 2048), 2048u, 0xffffffffu, 0u};
            const uint32_t last = (r.hi - r.lo) >> shift, at = choice[gen() % 4];
            const KeyRange p = r.part(at, shift);
            outside += last >= 2048 || p.lo > p.hi || p.lo < r.lo || p.hi > r.hi || p.hi - p.lo >= r.hi - r.lo;
            // the keys that count as that part are those in it
            outside += at <= last && ((r.hi - p.hi) >> shift != at || (r.hi - p.lo) >> shift != at);
            r = p;
        }
        most = max(most, n);
    }
    std::printf("key_range_rounds %d\nkey_ranges_outside %d\n", most, outside);
}

int main() {
    key_ranges();
    weights();
    sums();
    shares();
    return 0;
}
