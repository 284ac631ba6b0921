// sampling_common.cuh -- arithmetic shared by the sampling and log-probability
// kernels: the order of logits as integers, softmax weights as integers, and
// reductions over a CTA.
//
// Weights.  Which tokens a filter keeps and which one a uniform draws are
// decided on running sums of w = exp((l - l_max)/T).  Around a border of a
// wide row two neighbouring sums are 1e-6 of the whole apart and less, so float sums
// would pick other tokens than the definition does, and sums taken in another
// order other ones again.  The kernels therefore take every weight to
// 2^-39 of itself as a 64-bit integer W = w 2^F: integer sums have no rounding and no
// order.  F = 43 for V <= 2^19 and less beyond, so that V weights fit 62 bits.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace sv {

constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr int kMaxFix = 43;

// Fractional bits of the integer weights of a row of V entries.
inline int weight_bits(int64_t V) {
    int lg = 0;
    while (((int64_t)1 << lg) < V)
        ++lg;
    return 62 - lg < kMaxFix ? 62 - lg : kMaxFix;
}

#ifdef __CUDACC__

// 2^(j/64) as the sum of two floats, j = 0..63.
__device__ const float2 kPow2Steps[64] = {
    {0x1.000000p+0f, 0x0p+0f}, {0x1.02c9a4p+0f, -0x1.887fa0p-28f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {0x1.087452p+0f, -0x1.e2990ep-26f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.0e3ec4p+0f, -0x1.a585ccp-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.1429aap+0f, 0x1.d525bcp-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f},
    {0x1.1a35bep+0f, 0x1.6df96ep-25f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, {0x1.2063b8p+0f, 0x1.0c519ap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.26b456p+0f, 0x1.789f38p-26f}, {0x1.29e9e0p+0f, -0x1.5c0424p-25f},
    {0x1.2d285ap+0f, 0x1.b900c2p-26f}, {0x1.306fe0p+0f, 0x1.4636e2p-25f}, {0x1.33c08cp+0f, -0x1.b37d20p-25f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3a7db4p+0f, -0x1.634c02p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f},
    {0x1.4160a2p+0f, 0x1.f72e2ap-28f}, {0x1.44e086p+0f, 0x1.8624b4p-30f}, {0x1.486a2cp+0f, -0x1.47d866p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.4f9b28p+0f, -0x1.2c5a6cp-25f}, {0x1.5342b6p+0f, -0x1.2c5610p-25f},
    {0x1.56f474p+0f, -0x1.295b04p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.5e76f2p+0f, -0x1.4a5bd6p-25f},
    {0x1.6247ecp+0f, -0x1.f8b550p-25f}, {0x1.662388p+0f, 0x1.2a9112p-27f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f},
    {0x1.6dfb24p+0f, -0x1.cd72e8p-27f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f}, {0x1.75feb6p+0f, -0x1.37b306p-25f},
    {0x1.7a1148p+0f, -0x1.829fd0p-25f}, {0x1.7e2f34p+0f, -0x1.261634p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.868d9ap+0f, -0x1.2edb44p-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.8f1aeap+0f, -0x1.baa232p-26f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.97d82ap+0f, -0x1.0d8d84p-31f}, {0x1.9c4918p+0f, 0x1.51f848p-27f},
    {0x1.a0c668p+0f, -0x1.2886a6p-26f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f}, {0x1.a9e6b6p+0f, -0x1.50c048p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b33a2cp+0f, -0x1.ec3a82p-26f}, {0x1.b7f770p+0f, -0x1.a09438p-25f},
    {0x1.bcc1eap+0f, -0x1.f687c6p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.c67f12p+0f, 0x1.cafa2ap-25f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.d072d4p+0f, 0x1.40f130p-25f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f},
    {0x1.da9e60p+0f, 0x1.ed9942p-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f}, {0x1.e502eep+0f, 0x1.e2cffep-26f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.efa1bep+0f, 0x1.cc2b44p-25f}, {0x1.f50766p+0f, -0x1.246eb0p-26f},
    {0x1.fa7c18p+0f, 0x1.9e90d8p-28f}};

// Order of logits as unsigned integers: a larger logit has a larger key, and
// -0 has the key of +0.
__device__ __forceinline__ uint32_t logit_key(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kKeyMinusInf = 0x007fffffu;  // logit_key(-inf)

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What turns a row's logits into weights: t = (l_max - l) c, c = log2(e)/T.
struct RowScale {
    float lmax;
    float ch, cl;  // c as the sum of two floats
    int fix;       // F
};

// t as the sum of two floats; t >= 0, +inf for l = -inf.  The difference
// l_max - l is taken with its rounding error, so t is good to 2^-45 of itself.
__device__ __forceinline__ void exponent_of(const RowScale& s, float l, float& th, float& tl) {
    const float d = s.lmax - l;
    const float bv = d - s.lmax;
    const float dl = (s.lmax - (d - bv)) - (l + bv);
    th = d * s.ch;
    tl = fmaf(d, s.ch, -th);
    tl = fmaf(d, s.cl, tl);
    tl = fmaf(dl, s.ch, tl);
}

// 2^-t as u 2^(-43 - down), 2^43 <= u < 2^44, within 2^-39 of itself; down = 64 from t = 60 on.
//   -t = k/64 + r,  |r| <= 1/128:  2^-t = 2^floor(k/64) * 2^((k mod 64)/64) * (1 + y),
//   y = e^z - 1 for z = r ln 2 as z + z^2/2 + z^3/6 + z^4/24, |z| < 2^-7.5, its first
// term in two floats; the terms behind it are below 2^-16 and take one (2^-40).
__device__ __forceinline__ unsigned long long weight_parts(const RowScale& s, const float2* pow2, float l,
                                                           int& down) {
    float th, tl;
    exponent_of(s, l, th, tl);
    down = 64;
    if (!(th < 60.0f))
        return 0;
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
    constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.9046542121259336e-9f;
    const float m = fmaf(th, -64.0f, kMagic);
    const int k = __float_as_int(m) - __float_as_int(kMagic);
    const float r = fmaf(m - kMagic, -0.015625f, -th);  // exact
    const float zh = r * kLn2h;
    float zl = fmaf(r, kLn2h, -zh);
    zl = fmaf(r, kLn2l, zl);
    zl = fmaf(tl, -kLn2h, zl);
    const float z = zh + zl;
    const float q = z * z * fmaf(z, fmaf(z, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f);
    const float2 p = pow2[k & 63];
    const float ah = p.x * zh;
    float b = fmaf(p.x, zh, -ah);
    b = fmaf(p.x, zl + q, b);
    b = fmaf(p.y, zh, b) + p.y;
    const float v = p.x + ah;               // p.x >= 1 > |ah|
    const float e = (ah - (v - p.x)) + b;
    // v + e in units of 2^-43: the multiple of 2^-21 from the bits of v + 4, what is left
    // (below 2^-21) from the bits of a sum with 1.5 * 2^-20
    const float v4 = (v + e) + 4.0f;
    const float left = e + (v - (v4 - 4.0f));
    constexpr float kMagicLow = 1.430511474609375e-6f;  // 1.5 * 2^-20
    const int low = __float_as_int(left + kMagicLow) - __float_as_int(kMagicLow);
    down = -(k >> 6);  // >= 0
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

// 2^-t as a float (2^-22 of itself): what probabilities are written from.
__device__ __forceinline__ float weight_float(const RowScale& s, float l) {
    float th, tl;
    exponent_of(s, l, th, tl);
    if (!(th < 150.0f))
        return 0.0f;
    const float e = ex2_approx(-th);
    return fmaf(e, tl * -0.6931472f, e);
}

// c = log2(e)/T as the sum of two floats
__device__ __forceinline__ void split_scale(float T, float& ch, float& cl) {
    constexpr float kLog2eh = 1.44269502162933349609375f, kLog2el = 1.9259629911266174e-8f;
    ch = __fdiv_rn(kLog2eh, T);
    cl = __fdiv_rn(fmaf(-ch, T, kLog2eh) + kLog2el, T);
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
    const uint32_t b = __float_as_uint(u);  // 0 <= u < 1
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

__device__ __forceinline__ uint4 load_stream(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Entry e of a 16-byte vector of ES-byte logits, widened exactly to float.
template <int ES>
__device__ __forceinline__ float vector_entry(const uint4& v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (ES == 4)
        return __uint_as_float(w[e]);
    else
        return __uint_as_float((e & 1) ? (w[e >> 1] & 0xffff0000u) : (w[e >> 1] << 16));
}
template <int ES>
__device__ __forceinline__ float scalar_entry(const void* row, int64_t i) {
    if constexpr (ES == 4)
        return static_cast<const float*>(row)[i];
    else
        return __uint_as_float((uint32_t)static_cast<const unsigned short*>(row)[i] << 16);
}

// The largest of two floats, NaN if one is a NaN.
__device__ __forceinline__ float max_nan(float x, float y) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
    return d;
}

// The largest of a vector's logits, whatever NaNs it holds; NaN if it holds one.
template <int ES>
__device__ __forceinline__ float vector_max(const uint4& v) {
    if constexpr (ES == 4) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        uint32_t m, x;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(v.z), "r"(v.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
}
template <int ES>
__device__ __forceinline__ float vector_max_nan(const uint4& v) {
    if constexpr (ES == 4) {
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                       max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
        uint32_t m, x;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(v.x), "r"(v.y));
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(v.z), "r"(v.w));
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
}

// Sums of 2^((l - m) c) against two maxima, joined into the first: a new maximum, or a
// NaN, which stays.
__device__ __forceinline__ void join_sums(float& m, float& s, float m1, float s1, float c) {
    const float grown = max_nan(m, m1), inf = __int_as_float(0x7f800000);
    s = (m > -inf ? s * ex2_approx((m - grown) * c) : 0.0f) + (m1 > -inf ? s1 * ex2_approx((m1 - grown) * c) : 0.0f);
    m = grown;
}

// the same over groups of N lanes
template <int N>
__device__ __forceinline__ void join_lanes(float& m, float& s, float c) {
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
        const float m1 = __shfl_xor_sync(kAllLanes, m, o), s1 = __shfl_xor_sync(kAllLanes, s, o);
        join_sums(m, s, m1, s1, c);
    }
}

// sum of 2^((l - m) c) over a vector's logits: differences (a bfloat16 operand is
// widened inside the subtraction), products and sums two at a time
template <int ES>
__device__ __forceinline__ float exp_sum(const uint4& v, float m, float c) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    unsigned long long cc, sum = 0;
    asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
#pragma unroll
    for (int j = 0; j < 8 / ES; ++j) {
        float lo, hi;
        if constexpr (ES == 2) {
            asm("{\n\t.reg .b16 l, h;\n\t"
                "mov.b32 {l, h}, %2;\n\t"
                "add.rn.f32.bf16 %0, l, %3;\n\t"
                "add.rn.f32.bf16 %1, h, %3;\n\t}"
                : "=f"(lo), "=f"(hi)
                : "r"(w[j]), "f"(-m));
        } else {
            lo = __uint_as_float(w[2 * j]) - m;
            hi = __uint_as_float(w[2 * j + 1]) - m;
        }
        unsigned long long t;
        asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tmul.rn.f32x2 %0, d, %3;\n\t}" : "=l"(t) : "f"(lo), "f"(hi), "l"(cc));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(t));
        asm("mov.b64 %0, {%1, %2};" : "=l"(t) : "f"(ex2_approx(lo)), "f"(ex2_approx(hi)));
        if (j)
            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(t));
        else
            sum = t;
    }
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(sum));
    return lo + hi;
}

// The largest logit of each of a thread's steps through the slice (the first pass goes
// kDeep vectors a step, and so do later ones), to quarters and in eight bits: later
// passes leave out the steps that hold nothing for them.  Long slices' steps share the
// 16 codes.
constexpr int kDeep = 4;
struct StepCodes {
    uint8_t code[16];
};
__device__ __forceinline__ uint32_t step_code(float l) {  // grows with l; NaN: the largest
    const float x = fmaf(l, 4.0f, 64.0f);
    return x < 0.0f ? 0u : x < 255.0f ? (uint32_t)x : 255u;
}
// One CTA's part of a row: ids s0..s1-1, and its 16-byte vectors.  Number k holds the
// ids from k E - off on, where off is the place of the row's first logit in its own
// vector.  What they leave at the part's ends (the row's ends: parts meet between
// vectors) is taken one by one.  NT: threads of the CTA.
template <int ES, int NT>
struct Slice {
    static constexpr int E = 16 / ES;
    const unsigned char* base;  // the row's first logit
    uint32_t s0, s1, off, k0, k1;

    Slice() = default;
    // part `rank` of parts of `slice` ids (a multiple of E, and together V + E - 1 at least)
    __device__ __forceinline__ Slice(const unsigned char* row, int64_t V, int64_t slice, int rank) : base(row) {
        off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u) / ES;
        const int64_t v0 = rank * slice - off, v1 = v0 + slice;
        s0 = (uint32_t)(v0 < 0 ? 0 : v0 < V ? v0 : V);
        s1 = (uint32_t)(v1 < V ? v1 : V);
        k0 = (s0 + off + E - 1) / E;
        k1 = max((s1 + off) / E, k0);
    }

    __device__ __forceinline__ const uint4* vectors() const {
        return reinterpret_cast<const uint4*>(base - (size_t)off * ES);
    }
    __device__ __forceinline__ uint32_t head_end() const { return min(k0 * E - off, s1); }
    __device__ __forceinline__ uint32_t tail_start() const { return min(max(k1 * E - off, head_end()), s1); }

    // which of the 16 codes is step s's: s >> code_shift()
    __device__ __forceinline__ int code_shift() const {
        const uint32_t steps = (k1 - k0 + kDeep * NT - 1) / (kDeep * NT);
        return steps <= 16 ? 0 : 28 - __clz(steps - 1);
    }

    // vec(w, id of its first logit) for every vector of the slice, one(id) for every
    // other logit.  The next D vectors are loaded before D are worked on; `Rolled` keeps
    // one copy of vec's code.
    template <int D, bool Rolled, class Vec, class One>
    __device__ __forceinline__ void walk(Vec&& vec, One&& one) const {
        walk_steps<D, Rolled>(vec, [](uint32_t) {}, one);
    }
    // The same step by step: a thread's step s is D of its vectors, and done(s) follows it.
    template <int D, bool Rolled, class Vec, class Done, class One>
    __device__ __forceinline__ void walk_steps(Vec&& vec, Done&& done, One&& one) const {
        const int tid = threadIdx.x;
        const uint4* p = vectors() + k0 + tid;
        uint4 next[D];
        const auto load = [&](uint32_t k) {
#pragma unroll
            for (int j = 0; j < D; ++j)
                if (k + j * NT < k1)
                    next[j] = load_stream(p + j * NT);
            p += D * NT;
        };
        load(k0 + tid);
        uint32_t s = 0;
#pragma unroll 1
        for (uint32_t k = k0 + tid; k < k1; k += D * NT, ++s) {
            uint4 w[D];
#pragma unroll
            for (int j = 0; j < D; ++j)
                w[j] = next[j];
            load(k + D * NT);
            if constexpr (Rolled) {
#pragma unroll 1
                for (int j = 0; j < D && k + j * NT < k1; ++j) {
                    vec(w[0], (k + j * NT) * E - off);
#pragma unroll
                    for (int i = 0; i + 1 < D; ++i)
                        w[i] = w[i + 1];
                }
            } else {
#pragma unroll
                for (int j = 0; j < D; ++j)
                    if (k + j * NT < k1)
                        vec(w[j], (k + j * NT) * E - off);
            }
            done(s);
        }
        edges(one);
    }

    // one(id) for the entries beside the vectors
    template <class One>
    __device__ __forceinline__ void edges(One&& one) const {
        const uint32_t head = head_end() - s0, edge = head + (s1 - tail_start());
#pragma unroll 1
        for (uint32_t j = threadIdx.x; j < edge; j += NT)
            one(j < head ? s0 + j : tail_start() + (j - head));
    }

    // the codes that are at least `least`: a bit each
    __device__ __forceinline__ static uint32_t marks(const StepCodes* codes, uint32_t least) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            m |= (uint32_t)(codes->code[i] >= least) << i;
        return m;
    }
    // walk(), but of the marked steps alone.  Each thread goes from one such step to its
    // next: a warp waits for as many loads as its busiest lane has.
    template <int D, class Vec, class One>
    __device__ __forceinline__ void walk_marked(uint32_t marks, Vec&& vec, One&& one) const {
        const int tid = threadIdx.x, shift = code_shift();
        const uint32_t mine = k1 - k0 > tid ? k1 - k0 - tid : 0, steps = (mine + D * NT - 1) / (D * NT);
        const uint4* p = vectors() + k0 + tid;
        const auto following = [&](uint32_t s) {
            while (s < steps && !((marks >> (s >> shift)) & 1))
                ++s;
            return s;
        };
        uint4 next[D];
        const auto load = [&](uint32_t s) {
#pragma unroll
            for (int j = 0; j < D; ++j)
                if ((s * D + j) * NT < mine)
                    next[j] = load_stream(p + (s * D + j) * NT);
        };
        uint32_t s = following(0);
        load(s);
#pragma unroll 1
        while (s < steps) {
            uint4 w[D];
#pragma unroll
            for (int j = 0; j < D; ++j)
                w[j] = next[j];
            const uint32_t at = s;
            s = following(s + 1);
            load(s);
#pragma unroll 1
            for (int j = 0; j < D && (at * D + j) * NT < mine; ++j) {
                vec(w[0], (k0 + tid + (at * D + j) * NT) * E - off);
#pragma unroll
                for (int i = 0; i + 1 < D; ++i)
                    w[i] = w[i + 1];
            }
        }
        edges(one);
    }

    // skip(id of its first logit) for the vectors of the other steps
    template <int D, class Skip>
    __device__ __forceinline__ void pass_unmarked(uint32_t marks, Skip&& skip) const {
        const int shift = code_shift();
        uint32_t s = 0;
#pragma unroll 1
        for (uint32_t k = k0 + threadIdx.x; k < k1; k += D * NT, ++s)
            if (!((marks >> (s >> shift)) & 1)) {
#pragma unroll
                for (int j = 0; j < D; ++j)
                    if (k + j * NT < k1)
                        skip((k + j * NT) * E - off);
            }
    }

    // fn(l, id) for every entry of the slice
    template <class F>
    __device__ __forceinline__ void each(F&& fn) const {
        walk<4, true>(
            [&](const uint4& w, uint32_t id) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    fn(vector_entry<ES>(w, e), id + e);
            },
            [&](uint32_t id) { fn(scalar_entry<ES>(base, id), id); });
    }
};

#endif  // __CUDACC__

}  // namespace sv
