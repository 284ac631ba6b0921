// sampling_weights.cuh -- the sampling kernels' arithmetic on weights, in plain floats
// and integers: no instruction of its own, so that it also runs on a host.
//
// Which tokens a filter keeps and which one a uniform draws are
// decided on running sums of w = exp((l - l_max)/T).  Around a border of a
// wide row two neighbouring sums are 1e-6 of the whole apart and less, so float sums
// would pick other tokens than the definition does, and sums taken in another
// order other ones again.  The kernels therefore take every weight to
// 2^-39 of itself as a 64-bit integer W = w 2^F: integer sums have no rounding and no
// order.  F = 43 for V <= 2^19 and less beyond, so that V weights fit 62 bits.
#pragma once

#include <cstdint>

namespace sv {

constexpr int kMaxFix = 43;

// Fractional bits of the integer weights of a row of V entries.
inline int weight_bits(int64_t V) {
    int lg = 0;
    while (((int64_t)1 << lg) < V)
        ++lg;
    return 62 - lg < kMaxFix ? 62 - lg : kMaxFix;
}

#ifdef __CUDACC__

// 2^(j/128) as the sum of two floats, to 2^-49.
constexpr int kSteps = 128;
__device__ const float2 kPow2Steps[kSteps] = {
    {0x1.000000p+0f, 0x0p+0f}, {0x1.0163dap+0f, 0x1.3f6666p-25f}, {0x1.02c9a4p+0f, -0x1.887fa0p-28f},
    {0x1.04315ep+0f, 0x1.0dcff0p-25f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0706b2p+0f, 0x1.3bbedcp-25f},
    {0x1.087452p+0f, -0x1.e2990ep-26f}, {0x1.09e3ecp+0f, 0x1.58de70p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x1.0cc922p+0f, 0x1.6e48fep-25f}, {0x1.0e3ec4p+0f, -0x1.a585ccp-25f}, {0x1.0fb66ap+0f, 0x1.ffda64p-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.12abdcp+0f, 0x1.b0c730p-30f}, {0x1.1429aap+0f, 0x1.d525bcp-25f},
    {0x1.15a98cp+0f, 0x1.14b1cap-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.18af94p+0f, -0x1.dcdc86p-26f},
    {0x1.1a35bep+0f, 0x1.6df96ep-25f}, {0x1.1bbe08p+0f, 0x1.011734p-26f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.1ed502p+0f, 0x1.7e6c8ep-27f}, {0x1.2063b8p+0f, 0x1.0c519ap-25f}, {0x1.21f49ap+0f, -0x1.d0446ep-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.251ce4p+0f, 0x1.f654c8p-25f}, {0x1.26b456p+0f, 0x1.789f38p-26f},
    {0x1.284dfep+0f, 0x1.f56380p-28f}, {0x1.29e9e0p+0f, -0x1.5c0424p-25f}, {0x1.2b87fep+0f, -0x1.e4a4cep-25f},
    {0x1.2d285ap+0f, 0x1.b900c2p-26f}, {0x1.2ecafap+0f, 0x1.27c5eap-25f}, {0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {0x1.321710p+0f, -0x1.d993e8p-27f}, {0x1.33c08cp+0f, -0x1.b37d20p-25f}, {0x1.356c56p+0f, -0x1.b5803cp-30f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.38cae6p+0f, 0x1.a0bb0cp-25f}, {0x1.3a7db4p+0f, -0x1.634c02p-25f},
    {0x1.3c32dcp+0f, 0x1.89d472p-27f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.3fa450p+0f, 0x1.2b2006p-26f},
    {0x1.4160a2p+0f, 0x1.f72e2ap-28f}, {0x1.431f5ep+0f, -0x1.abd5dap-26f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.46a41ep+0f, 0x1.a3a00ap-25f}, {0x1.486a2cp+0f, -0x1.47d866p-25f}, {0x1.4a32b0p+0f, -0x1.e50584p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.4dcb2ap+0f, -0x1.8088bcp-26f}, {0x1.4f9b28p+0f, -0x1.2c5a6cp-25f},
    {0x1.516daap+0f, 0x1.67b320p-27f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f}, {0x1.551a4cp+0f, 0x1.4bb242p-25f},
    {0x1.56f474p+0f, -0x1.295b04p-25f}, {0x1.58d12ep+0f, -0x1.6d0700p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.5c9268p+0f, 0x1.4b28d6p-25f}, {0x1.5e76f2p+0f, -0x1.4a5bd6p-25f}, {0x1.605e1cp+0f, -0x1.a248fep-26f},
    {0x1.6247ecp+0f, -0x1.f8b550p-25f}, {0x1.643464p+0f, -0x1.66679cp-25f}, {0x1.662388p+0f, 0x1.2a9112p-27f},
    {0x1.68155ep+0f, -0x1.766ad2p-25f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.6c0128p+0f, -0x1.5e84a8p-25f},
    {0x1.6dfb24p+0f, -0x1.cd72e8p-27f}, {0x1.6ff7e0p+0f, -0x1.ab9ae0p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.73f9a4p+0f, 0x1.14b02ep-25f}, {0x1.75feb6p+0f, -0x1.37b306p-25f}, {0x1.780694p+0f, 0x1.fbcba8p-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.7c1ed0p+0f, 0x1.30c132p-28f}, {0x1.7e2f34p+0f, -0x1.261634p-25f},
    {0x1.804276p+0f, -0x1.783cbep-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.8471a4p+0f, 0x1.88f1ecp-26f},
    {0x1.868d9ap+0f, -0x1.2edb44p-26f}, {0x1.88ac7ep+0f, -0x1.9d665ap-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.8cf322p+0f, -0x1.29576ep-25f}, {0x1.8f1aeap+0f, -0x1.baa232p-26f}, {0x1.9145b0p+0f, 0x1.723ff8p-25f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.95a44cp+0f, 0x1.790a42p-25f}, {0x1.97d82ap+0f, -0x1.0d8d84p-31f},
    {0x1.9a0f18p+0f, -0x1.e6bf08p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.9e8632p+0f, -0x1.873738p-26f},
    {0x1.a0c668p+0f, -0x1.2886a6p-26f}, {0x1.a309bep+0f, 0x1.8945a6p-25f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.a799e2p+0f, -0x1.99e994p-25f}, {0x1.a9e6b6p+0f, -0x1.50c048p-25f}, {0x1.ac36bcp+0f, -0x1.606432p-31f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b0e072p+0f, 0x1.31b6ccp-25f}, {0x1.b33a2cp+0f, -0x1.ec3a82p-26f},
    {0x1.b59728p+0f, 0x1.bcab28p-25f}, {0x1.b7f770p+0f, -0x1.a09438p-25f}, {0x1.ba5b04p+0f, -0x1.ebdf36p-25f},
    {0x1.bcc1eap+0f, -0x1.f687c6p-25f}, {0x1.bf2c26p+0f, -0x1.0a387ep-26f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x1.c40ab6p+0f, -0x1.7c2c98p-39f}, {0x1.c67f12p+0f, 0x1.cafa2ap-25f}, {0x1.c8f6dap+0f, -0x1.7f230ap-25f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.cdf0b6p+0f, -0x1.544780p-25f}, {0x1.d072d4p+0f, 0x1.40f130p-25f},
    {0x1.d2f870p+0f, 0x1.01b13ep-25f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.d80e32p+0f, -0x1.26cf8ep-25f},
    {0x1.da9e60p+0f, 0x1.ed9942p-27f}, {0x1.dd3220p+0f, -0x1.9fc974p-25f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.e26462p+0f, -0x1.614bdap-25f}, {0x1.e502eep+0f, 0x1.e2cffep-26f}, {0x1.e7a520p+0f, -0x1.0e2ce0p-26f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.ecf482p+0f, 0x1.b1ccfep-25f}, {0x1.efa1bep+0f, 0x1.cc2b44p-25f},
    {0x1.f252b4p+0f, -0x1.1288aep-25f}, {0x1.f50766p+0f, -0x1.246eb0p-26f}, {0x1.f7bfdap+0f, 0x1.b397c2p-25f},
    {0x1.fa7c18p+0f, 0x1.9e90d8p-28f}, {0x1.fd3c22p+0f, 0x1.71ee3ep-25f}};

// What turns a row's logits into weights: t = (l_max g - l g) c, c = log2(e)/(T g).
struct RowScale {
    float lmax;
    float ch, cl;  // c as the sum of two floats
    float g;       // 1; kShrink from T = kFarT on
    int fix;       // F
};

// At temperatures that weigh differences of 2^127 and more, logits and T are both taken smaller: the
// difference is a float then, and c a normal one.  What a logit below 2^-62 loses is nothing over such a T.
constexpr float kFarT = 0x1p100f, kShrink = 0x1p-64f;

// t as the sum of two floats; t >= 0, +inf for l = -inf.  The difference
// l_max - l is taken with its rounding error, so t is good to 2^-45 of itself.
__device__ __forceinline__ void exponent_of(const RowScale& s, float l, float& th, float& tl) {
    const float m = s.lmax * s.g;
    l *= s.g;
    const float d = m - l;
    const float bv = d - m;
    const float dl = (m - (d - bv)) - (l + bv);
    th = d * s.ch;
    tl = fmaf(d, s.ch, -th);
    tl = fmaf(d, s.cl, tl);
    tl = fmaf(dl, s.ch, tl);
}

// 2^-t as u 2^(-43 - down), 0.997 * 2^43 <= u < 2^44, within 2^-39 of itself up to t = 32 (of
// what lies beyond, rounding to 2^-43 leaves eleven bits at most); down = 64 from t = 60 on.  A
// table and a polynomial, after P. T. P. Tang, "Table-driven implementation of the exponential
// function in IEEE floating-point arithmetic", ACM TOMS 15 (1989):
//   -t = k/128 + r,  |r| <= 1/256:  2^-t = 2^floor(k/128) * 2^((k mod 128)/128) * e^z,
//   z = r ln 2 = zh + zl, |zh| < 2^-8.5, |zl| < 2^-19 up to t = 32,
//   e^z - 1 = zh + q + zl (1 + zh + q + zl/2),  q = zh^2/2 + zh^3/6 + zh^4/24 < 2^-18.
// What rounds, in units of 2^-42 of the weight: q twice 0.5; what is added to it 1, and its factor 0.9;
// their product with the table's value 1.4, and the sum with what zh's leaves 1.4; t's lower part 0.9,
// zl's 0.25, the last bit 0.25: 7.1 in all, 8 being 2^-39.  (With 64 steps the parts behind zh are four
// times as large: 2^-37.4 at worst.)  The worst of 300 million is 2^-39.9.
__device__ __forceinline__ unsigned long long weight_parts(const RowScale& s, const float2* pow2, float l,
                                                           int& down) {
    float th, tl;
    exponent_of(s, l, th, tl);
    down = 64;
    if (!(th < 60.0f))
        return 0;
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
    constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.9046542121259336e-9f;
    const float m = fmaf(th, -128.0f, kMagic);
    const int k = __float_as_int(m) - __float_as_int(kMagic);
    const float r = fmaf(m - kMagic, -0.0078125f, -th);  // exact
    const float zh = r * kLn2h;
    float zl = fmaf(r, kLn2h, -zh);
    zl = fmaf(r, kLn2l, zl);
    zl = fmaf(tl, -kLn2h, zl);
    const float half = zh * (0.5f * zh);
    const float q = fmaf(half, zh * fmaf(zh, 1.0f / 12.0f, 1.0f / 3.0f), half);
    const float2 p = pow2[k & (kSteps - 1)];
    const float ah = p.x * zh;
    const float small = fmaf(p.x, zh, -ah) + fmaf(p.y, zh, p.y);  // below 2^-24
    const float slope = (1.0f + zh) + fmaf(0.5f, zl, q);
    const float b = fmaf(p.x, fmaf(zl, slope, q), small);
    const float v = p.x + ah;               // p.x >= 1 > |ah|
    const float e = (ah - (v - p.x)) + b;
    // v + e in units of 2^-43: the multiple of 2^-21 from the bits of v + 4, what is left
    // (below 2^-21) from the bits of a sum with 1.5 * 2^-20
    const float v4 = (v + e) + 4.0f;
    const float left = e + (v - (v4 - 4.0f));
    constexpr float kMagicLow = 1.430511474609375e-6f;  // 1.5 * 2^-20
    const int low = __float_as_int(left + kMagicLow) - __float_as_int(kMagicLow);
    down = -(k >> 7);  // >= 0
    return ((unsigned long long)(uint32_t)(__float_as_int(v4) - __float_as_int(4.0f)) << 22) + (long long)low;
}

__device__ __forceinline__ unsigned long long rounded_shift(unsigned long long x, int n) {
    return n > 62 ? 0 : n ? (x + (1ull << (n - 1))) >> n : x;
}

// round(2^F 2^-t)
__device__ __forceinline__ unsigned long long weight_fixed(const RowScale& s, const float2* pow2, float l) {
    int down;
    const unsigned long long u = weight_parts(s, pow2, l, down);
    return rounded_shift(u, down + kMaxFix - s.fix);
}

// round(2^F n 2^-t) for n <= V entries with one logit: many small ones are not rounded
// away one by one (n u < 2^63 in units of 2^-F)
__device__ __forceinline__ unsigned long long mass_fixed(const RowScale& s, const float2* pow2, float l,
                                                         uint32_t n) {
    int down;
    const unsigned long long u = weight_parts(s, pow2, l, down);
    return rounded_shift(rounded_shift(u, kMaxFix - s.fix) * n, down);
}

// g and c of a temperature
__device__ __forceinline__ void set_temperature(RowScale& s, float T) {
    constexpr float kLog2eh = 1.44269502162933349609375f, kLog2el = 1.9259629911266174e-8f;
    s.g = T < kFarT ? 1.0f : kShrink;
    T *= s.g;
    s.ch = __fdiv_rn(kLog2eh, T);
    s.cl = __fdiv_rn(fmaf(-s.ch, T, kLog2eh) + kLog2el, T);
}

// floor(u x) and ceil(p x) with no rounding before the last step.
__device__ __forceinline__ unsigned long long scaled(uint64_t mant, int sh, unsigned long long x,
                                                     bool up) {
    // mant x / 2^sh, mant < 2^53, x < 2^63, 0 <= sh
    const unsigned long long hi = __umul64hi(mant, x), lo = mant * x;
    if (sh >= 128)
        return (up && (hi | lo)) ? 1 : 0;
    unsigned long long q;
    bool rest;
    if (sh >= 64) {
        q = sh == 64 ? hi : hi >> (sh - 64);
        rest = lo || (sh > 64 && (hi << (128 - sh)));
    } else if (sh) {
        q = (hi << (64 - sh)) | (lo >> sh);
        rest = (lo << (64 - sh)) != 0;
    } else {
        q = lo;
        rest = false;
    }
    return q + (up && rest ? 1 : 0);
}
__device__ __forceinline__ unsigned long long floor_scaled(float u, unsigned long long x) {
    const uint32_t b = __float_as_uint(u) & 0x7fffffffu;  // 0 <= u < 1; -0 is 0
    const int ex = (int)(b >> 23);
    const uint32_t m = ex ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    return scaled(m, 150 - (ex ? ex : 1), x, false);
}
__device__ __forceinline__ unsigned long long ceil_scaled(double p, unsigned long long x) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(p);  // 0 < p < 1
    const int ex = (int)(b >> 52);
    const unsigned long long f = b & 0xfffffffffffffull;
    return scaled(ex ? f | 0x10000000000000ull : f, 1075 - (ex ? ex : 1), x, true);
}

// Keys lo..hi, and the parts that a search splits them into, counted from hi down: 2^shift
// keys each, `parts` of them at most.  Whatever part a search names, it is less than the whole and inside
// it: what goes on until one key is left ends after three of 2048 parts, also where the row changes under it.
struct KeyRange {
    uint32_t lo, hi;

    __device__ __forceinline__ int shift(uint32_t parts) const {
        int n = 0;
        while (((hi - lo) >> n) >= parts)
            ++n;
        return n;
    }
    __device__ __forceinline__ KeyRange part(uint32_t i, int n) const {
        const uint32_t top = hi - (min(i, (hi - lo) >> n) << n), width = (1u << n) - 1;
        return {top - lo > width ? top - width : lo, top};
    }
};

// ---------------------------------------------------- sums of weights -----

// A weight for sums, in half the instructions of weight_fixed, below kFarT: 2^(p - M), p = l c,
// M = l_max c, without the difference l_max - l.
//   M = Mk/128 + Mr, |Mr| <= 1/256;  p = k/128 + r + Mr, |r| <= 1/256, p - k/128 exact;
//   2^(p - M) = 2^floor((k - Mk)/128) T[(k - Mk) mod 128] (1 + y),  y = e^z - 1 in one float.
// y rounds at 2^-33 to either side, three times, and with ln 2 a weight is 2^-30.6 off at most:
// a sum of many entries does not show it (the lists' entries, few, take weight_fixed).  T in two floats, a copy for each of 16 lanes,
// so that lanes' reads do not meet in a bank.  For |M| < 128.
struct SumScale {
    float ch, cl, floor_l, mh, ml;  // mh + ml: Mr
    int k0;                         // Mk
    const float2* steps;

    __device__ __forceinline__ explicit SumScale(const RowScale& s) : ch(s.ch), cl(s.cl), floor_l(s.lmax - 70.0f / s.ch) {
        const float m = s.lmax * s.ch, l = fmaf(s.lmax, s.ch, -m) + s.lmax * s.cl, k = rintf(m * 128.0f);
        const float rest = fmaf(k, -0.0078125f, m);  // exact
        mh = rest + l;
        ml = l - (mh - rest);
        k0 = (int)k;
    }
};
// the weight as the table's part and the rest
__device__ __forceinline__ float2 sum_weight(const SumScale& s, float l) {
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
    l = fmaxf(l, s.floor_l);
    const float p = l * s.ch;
    const float pl = fmaf(l, s.cl, -s.ml) + fmaf(l, s.ch, -p);
    const float m = fmaf(p - s.mh, 128.0f, kMagic);
    const int k = __float_as_int(m) - __float_as_int(kMagic) - s.k0;
    const float r = (fmaf(m - kMagic, -0.0078125f, p) - s.mh) + pl;
    const float y = r * fmaf(r, fmaf(r, fmaf(r, 0.00961812911f, 0.0555041087f), 0.240226507f), 0.693147181f);
    const float2 t = s.steps[(k & 127) << 4];
    const float two = __int_as_float(((k & ~127) << 16) + (127 << 23));  // 2^floor(k/128)
    return make_float2(t.x * two, fmaf(t.x, y, t.y) * two);
}
// What WeightSum's parts are worth in units of 2^-F.
struct Units {
    float one, back;   // 2^n, n = min(F, 37), and 2^-n
    uint32_t hi, low;  // 2^(F - 20), 2^(F - n)
    __device__ __forceinline__ explicit Units(int F)
        : one((float)(1ull << min(F, 37))), back(1.0f / one), hi(1u << (F - 20)), low(1u << (F - min(F, 37))) {}
};
// A sum of weights.  Of four at a time, the table's parts go to a float of 2^-20 units,
// whose bits count them, and what that and the rests (|e^z - 1| < 2^-8.5) leave to one
// below 2^-6.5.  An integer takes its 2^-37 units, and what is less stays for the next four:
// a row's many small weights are not rounded away one by one.
struct WeightSum {
    static constexpr float kBase = 8.0f;
    float hi = kBase, lo = 0.0f;
    __device__ __forceinline__ void add(float2 w) {
        const float s = hi + w.x, taken = s - hi;
        lo += w.y + (w.x - taken);
        hi = s;
    }
    __device__ __forceinline__ void into(unsigned long long& x, const Units& u) {
        const int units = __float2int_rn(lo * u.one);
        x += (unsigned long long)(__float_as_uint(hi) - __float_as_uint(kBase)) * u.hi;
        x += (long long)units * (int)u.low;
        lo = fmaf((float)units, -u.back, lo);
        hi = kBase;
    }
    __device__ __forceinline__ long long rest(int F) const { return __float2ll_rn(lo * (float)(1ull << F)); }
};

#endif  // __CUDACC__

}  // namespace sv
