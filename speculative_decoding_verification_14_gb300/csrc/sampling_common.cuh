// sampling_common.cuh -- shared by the sampling and log-probability kernels: the order
// of logits as integers, loads and vectors of logits, sums in floats, and the walk over
// a CTA's slice of a row.  Weights as integers: sampling_weights.cuh.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sampling_weights.cuh"

namespace sv {

constexpr uint32_t kAllLanes = 0xffffffffu;

#ifdef __CUDACC__

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

// 2^-t as a float (2^-22 of itself): what probabilities are written from.
__device__ __forceinline__ float weight_float(const RowScale& s, float l) {
    float th, tl;
    exponent_of(s, l, th, tl);
    if (!(th < 150.0f))
        return 0.0f;
    const float e = ex2_approx(-th);
    return fmaf(e, tl * -0.6931472f, e);
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
// 16 codes.  Codes tell logits from -16 to 47.75 apart; rows beyond, or of small scale, get one code and
// are looked at whole (256 rows of 151936 bfloat16 with l_max about 60: draw under top-p 85 us
// instead of 69, filter 61 instead of 57).
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
