// distill.cu -- distillation of a drafter from the target's top log-probabilities: the loss of
// each row of draft logits, and its gradient.
//
// For a row z at temperature T, q = softmax(z / T), and the teacher's tokens x_k with
// log-probabilities a_k, t_k = exp(a_k):
//   top:   t_k over their sum, r = 0
//   tail:  r = max(0, 1 - sum t_k), an outcome of draft mass q_rest = sum of q off the list
//   loss   sum t_k (ln t_k - ln q(x_k)) + r (ln r - ln q_rest)
//   d/dz_v ((sum t_k + r) q_v - t_v) / T on the list, (... q_v - r q_v / q_rest) / T off it
//
// Design: clusters of C CTAs take the rows in turn.  Each CTA's slice of the row is copied
// to shared memory once (cp.async.bulk) and stays there: the sums and the gradient are both taken from it, so that a
// row is read once and its gradient written once whatever is asked for; the next row comes into L2 meanwhile.  The
// listed entries are taken out of the slice (-inf in their place) before the sums: what is summed then is the mass off
// the list, without the cancellation of S - sum of listed weights, and against a logit off the list, so that q_v / q_rest
// is right where the whole tail underflows next to a listed entry.  The CTAs exchange these sums and the listed
// logits through distributed shared memory.  Seven warps walk the slice; beside them the teacher has the list and makes
// of the sums what the gradient is written from, and the first CTA's scribe has r and the loss, in two floats: float32
// would lose what 1 - sum t_k or a small loss leaves (up to 5e-5 of it), and 64-bit arithmetic takes 140 cycles an
// operation (with it, by the teacher, 256 x 8 rows of 128256 bfloat16 took 334 us).
//
// What bounds it: 256 x 8 rows of 128256, 20 entries, loss and gradient: bfloat16 224 us for 1.05 GB (4.7 TB/s, 0.69 of
// a copy's rate), float32 416 us (0.75); 64 x 4 of 151936 bfloat16 46 us (0.50).  A CTA's turn of some 20 thousand
// cycles is 2.5 waiting for the copy, 1.5 at the barriers before the sums, 4 summing, 6 between the sums and the
// gradient (joins, the exchange, the teacher), 6 writing; three CTAs an SM (their slices fill its shared memory) hide
// most of one another's, and no pipe is above 30 %.  Tried: rows one by one, a cluster each, 279 and 485 us; four CTAs
// an SM with smaller slices 259 and 462, two with larger ones 234 and 410; 256 or 320 walkers an SM at fewer
// registers 246 and 261.
// Three CTAs of 288 threads leave 72 registers a thread, which is less than the scribe needs, who alone keeps two rows'
// lists: the compiler reports 130 bytes of spills, 206 read back.
//
// A wait that runs out (2 s for other CTAs, 10 s for a copy) ends the cluster's work: the CTA that gave up says so with
// its next sums, no CTA that hears of it waits or copies any more, and the rows left get NaN and SV_ERR_TIMEOUT.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/spec_verify.h"
#include "distill_plan.h"
#include "losses_common.cuh"
#include "losses_selftest.h"
#include "sampling_common.cuh"
#include "sv_context.h"
#include "two_floats.cuh"

namespace {

using namespace sv;

constexpr int kNT = kDistillThreads;
constexpr int kNW = kNT / 32;
constexpr int kMaxC = 16;
constexpr int kMaxList = kDistillMaxList;
constexpr uint32_t kCopyPiece = 16384;
// ex2.approx gives 5.0e-8 of itself too little in the mean over a period of its argument (measured, 2^22 arguments;
// 4 to 7e-8 in each sixty-fourth of it): a sum of many is corrected by it where two floats are kept
constexpr float kPowerBias = 5.0e-8f;

struct Args {
    const void* logits;
    int64_t stride;
    const float* top_logprobs;
    const int32_t* top_tokens;
    const int32_t* accept_len;  // or NULL: every row
    const float* grad_loss;     // or NULL: 1
    float* loss;                // or NULL
    void* grad;                 // or NULL
    int64_t grad_stride;
    int32_t* status;
    uint32_t* err_word;
    int64_t V, rows;
    int rows_per_seq, C, n, tail;
    int selftest;          // SV_SELFTEST_DISTILL_COPY or _EXCHANGE: in the last CTA of this row; 0 for neither
    int64_t selftest_row;
    uint32_t vectors;  // per CTA
    float iT, iTl, ch, cl;  // 1 / T and log2(e) / T in two parts each, the latter's both above 0
};

// what a CTA's slice gives off the list: a sum of weights, 2^-38 a unit in two halves, and what they are against; hi is
// -1 from a CTA that has given up
struct CtaPart {
    float hi, lo, m;
};

// what a row's gradients are written from: k 2^((z - m) c) off the list, g (total q - t) on it
struct Answer {
    float m, k, M, iS, total, g;
    float mu, su;
    int kind;      // an SV_ code, or -1: no teacher
    bool nothing;  // r is what rounding left
};

struct Shared {
    unsigned long long warp_sum[kNW];
    uint64_t bar, exchange[2];
    CtaPart part[2][kMaxC];
    Answer answer;
    float a[kMaxList];
    int32_t token[kMaxList];
    float z[2][kMaxList];  // the draft logits of the list
    float warp_max[kNW];
    float r[2], total[2];  // from the first CTA
    float list_max, list_sum;
    uint32_t listed;  // whether a token is
    uint32_t flags;   // 1 << code
    // Whether a wait of this CTA, or of one that told it so, has run out before a turn: of even turns and of odd ones,
    // each written in the turn before.  From then on it waits no more, copies nothing, and its rows have no answers.
    uint32_t dead[2];
};

__device__ __forceinline__ void store_cluster(uint32_t addr, float x) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

__device__ __forceinline__ unsigned long long two(float x, float y) {
    unsigned long long t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(t) : "f"(x), "f"(y));
    return t;
}

// 2^((z - m) c) of logits 2j and 2j + 1 of a vector, c = log2(e) / T in one float or (Fine) two: what
// rounding leaves of c moves every weight the same way, by up to |(z - m) / T| 2^-25
template <int ES, bool Fine>
__device__ __forceinline__ unsigned long long exp_two(const uint4& v, int j, float m, unsigned long long ch,
                                                      unsigned long long cl) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
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
    unsigned long long d = two(lo, hi), y;
    if constexpr (Fine) {
        // both parts are above 0: a difference of -inf gives -inf
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(d), "l"(cl));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(y) : "l"(d), "l"(ch));
    } else {
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(d), "l"(ch));
    }
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(y));
    return two(ex2_approx(lo), ex2_approx(hi));
}

// their sum over a vector
template <int ES>
__device__ __forceinline__ float exp_vector_sum(const uint4& v, float m, unsigned long long ch, unsigned long long cl) {
    unsigned long long s = exp_two<ES, true>(v, 0, m, ch, cl);
#pragma unroll
    for (int j = 1; j < 8 / ES; ++j)
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s) : "l"(exp_two<ES, true>(v, j, m, ch, cl)));
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(s));
    return lo + hi;
}

// times k, in the logits' type (bfloat16 rounds more away than the rest of c would add)
template <int ES>
__device__ __forceinline__ uint4 exp_scaled(const uint4& v, float m, unsigned long long ch, unsigned long long cl,
                                            float k) {
    uint32_t out[4];
    const unsigned long long kk = two(k, k);
#pragma unroll
    for (int j = 0; j < 8 / ES; ++j) {
        unsigned long long t = exp_two<ES, ES == 4>(v, j, m, ch, cl);
        float lo, hi;
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(t) : "l"(kk));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(t));
        if constexpr (ES == 2) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out[j]) : "f"(hi), "f"(lo));
        } else {
            out[2 * j] = __float_as_uint(lo);
            out[2 * j + 1] = __float_as_uint(hi);
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int ES>
__device__ __forceinline__ void store_entry(unsigned char* row, int64_t i, float x) {
    if constexpr (ES == 4)
        reinterpret_cast<float*>(row)[i] = x;
    else
        reinterpret_cast<__nv_bfloat16*>(row)[i] = __float2bfloat16_rn(x);
}

// A CTA's slice of a row as vectors v0 .. v1 - 1 of 16 bytes; vector k holds the ids from k E - off on.
template <int ES>
struct Part {
    static constexpr int E = 16 / ES;
    uint32_t off, v0, v1;
    int64_t V;
    __device__ __forceinline__ Part(const unsigned char* base, int64_t n, uint32_t vectors, int rank) : V(n) {
        off = (uint32_t)(reinterpret_cast<uintptr_t>(base) & 15u) / ES;
        const int64_t all = (n + off + E - 1) / E, a = (int64_t)rank * vectors, b = a + vectors;
        v0 = (uint32_t)(a < all ? a : all);
        v1 = (uint32_t)(b < all ? b : all);
    }
    // vectors that lie inside the row as a whole
    __device__ __forceinline__ bool whole(uint32_t k) const {
        return (int64_t)k * E >= off && (int64_t)(k + 1) * E <= V + off;
    }
};

// the largest of a warp's lanes; NaN if one is
__device__ __forceinline__ float warp_max(float x) {
    float m;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
    return m;
}
// The largest logit of a slice's vectors that fall to this warp; NaN if one is.
template <int ES>
__device__ __forceinline__ float slice_max(const uint4* slice, uint32_t vectors) {
    float m = -__int_as_float(0x7f800000);
    if constexpr (ES == 2) {
        uint32_t x = 0xff80ff80u;  // -inf, -inf
        for (uint32_t k = threadIdx.x; k < vectors; k += kNT) {
            const uint4 w = slice[k];
            uint32_t y, z;
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w.x), "r"(w.y));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(w.z), "r"(w.w));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(y), "r"(z));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(y));
        }
        m = max_nan(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    } else {
        for (uint32_t k = threadIdx.x; k < vectors; k += kNT)
            m = max_nan(m, vector_max_nan<ES>(slice[k]));
    }
    return warp_max(m);
}

// the sum over a warp's lanes
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x = two_add(x, Two{__shfl_xor_sync(kAllLanes, x.h, o), __shfl_xor_sync(kAllLanes, x.l, o)});
    return x;
}
// x + y, where a y beyond float is an infinity that stays (x and y are above -inf)
__device__ __forceinline__ Two two_finite(Two x, Two y) {
    const float inf = __int_as_float(0x7f800000);
    return x.h < inf && y.h < inf ? two_add(x, y) : Two{inf, 0.0f};
}
// (x - y) / T; an infinity stays one
__device__ __forceinline__ Two over(float x, float y, Two iT) {
    const Two d = two_sum(x, -y);
    return fabsf(d.h) <= 3.4028235e38f ? two_mul(d, iT) : Two{d.h, 0.0f};
}

// Writes f(local vector) as the gradient's vectors of this part.
template <int ES, typename F>
__device__ __forceinline__ void write_part(const Part<ES>& p, unsigned char* grad, F f) {
    constexpr int E = 16 / ES;
    const bool same = (uint32_t)(reinterpret_cast<uintptr_t>(grad) & 15u) / ES == p.off;
    // the row's ends, and rows whose gradient lies otherwise to 16 bytes than they do: entry by entry
    const auto by_entry = [&](uint32_t k) {
        const uint4 w = f(k - p.v0);
        const int64_t id = (int64_t)k * E - p.off;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (id + e >= 0 && id + e < p.V)
                store_entry<ES>(grad, id + e, vector_entry<ES>(w, e));
    };
    if (same) {
        uint4* vectors = reinterpret_cast<uint4*>(grad - (size_t)p.off * ES) + p.v0;
        const uint32_t w0 = p.v0 < p.v1 && !p.whole(p.v0) ? 1u : 0u;
        const uint32_t n = p.v1 - p.v0, w1 = n > w0 && !p.whole(p.v1 - 1) ? n - 1 : n;
#pragma unroll 4
        for (uint32_t i = w0 + threadIdx.x; i < w1; i += kNT)
            vectors[i] = f(i);
        if (threadIdx.x == 0 && w0)
            by_entry(p.v0);
        if (threadIdx.x == 32 && w1 < n)
            by_entry(p.v1 - 1);
    } else {
        for (uint32_t k = p.v0 + threadIdx.x; k < p.v1; k += kNT)
            by_entry(k);
    }
}

// the warps that walk the slice
__device__ __forceinline__ void sync_walkers() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(kNT) : "memory");
}

// the whole vectors of a part: first, and bytes of all
template <int ES>
__device__ __forceinline__ uint32_t whole_vectors(const Part<ES>& p, uint32_t& first) {
    uint32_t w0 = p.v0, w1 = p.v1;
    if (w0 < w1 && !p.whole(w0))
        ++w0;
    if (w0 < w1 && !p.whole(w1 - 1))
        --w1;
    first = w0;
    return (w1 - w0) * 16u;
}

template <int ES>
__global__ void __launch_bounds__(kNT + 64, kDistillCtas) sv_distill_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(128) uint4 slice[];
    __shared__ Shared sh;
    constexpr int E = 16 / ES;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.C, n = a.n;
    const uint32_t rank = blockIdx.x % C, clusters = gridDim.x / C;
    const float inf = __int_as_float(0x7f800000);
    const bool teacher = warp == kNW;     // the list, and what follows from the slices' sums
    const bool scribe = warp == kNW + 1;  // of the first CTA: what the list leaves, and the loss
    const unsigned long long ch = two(a.ch, a.ch), cl = two(a.cl, a.cl);
    const auto row_base = [&](int64_t row) { return static_cast<const unsigned char*>(a.logits) + row * a.stride * ES; };
    const auto is_live = [&](int64_t row) {
        if (!a.accept_len)
            return true;
        const int64_t seq = row / a.rows_per_seq;
        return row - seq * a.rows_per_seq < a.accept_len[seq];
    };

    if (teacher && lane == 0) {
        sh.listed = 0;
        sh.flags = 0;
        sh.dead[0] = sh.dead[1] = 0;
        barrier_init(&sh.bar, 1);
        for (int i = 0; i < 2; ++i)
            barrier_init(&sh.exchange[i], (uint32_t)C + 1);  // every CTA's sums, and the first one's r
        barrier_init_fence();
    }
    __syncwarp();
    cluster_arrive();
    int64_t row = blockIdx.x / C;
    // What the next row needs, ahead of it: a walker's listed token, the others' tokens and log-probabilities.
    int32_t tokens[kMaxList / 32];
    float logprobs[kMaxList / 32];
    bool next_live = is_live(row);
    const auto fetch = [&](int64_t r) {
        if (warp < kNW) {
            tokens[0] = tid < n ? a.top_tokens[r * n + tid] : -1;
        } else {
#pragma unroll
            for (int j = 0; j < kMaxList / 32; ++j)
                if (lane + 32 * j < n) {
                    tokens[j] = a.top_tokens[r * n + lane + 32 * j];
                    logprobs[j] = a.top_logprobs[r * n + lane + 32 * j];
                }
        }
    };
    fetch(row);
    cluster_wait();  // every CTA of the cluster runs: its memory may be written

    // The first CTA's scribe: a row's list in two floats, ahead of the row,
    struct {
        Two r, ts, t[kMaxList / 32];  // what the list leaves, its sum, its shares
        float a[kMaxList / 32], shift;
        uint32_t tokens;  // bit j: a token in place lane + 32 j
    } list;
    const auto read_list = [&] {
        float top = -inf;
        list.tokens = 0;
#pragma unroll
        for (int j = 0; j < kMaxList / 32; ++j) {
            const bool there = lane + 32 * j < n && tokens[j] >= 0 && tokens[j] < a.V;
            list.tokens |= (uint32_t)there << j;
            list.a[j] = there && logprobs[j] < inf ? logprobs[j] : -inf;
            top = fmaxf(top, list.a[j]);
        }
        top = warp_max(top);
        list.shift = !a.tail && top > -inf ? top : 0.0f;
        list.ts = Two{0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kMaxList / 32; ++j) {
            list.t[j] = Two{0.0f, 0.0f};
            if (32 * j < n) {
                list.t[j] = two_exp(two_sum(list.a[j], -list.shift));
                list.ts = two_add(list.ts, list.t[j]);
            }
        }
        list.ts = warp_sum(list.ts);
        list.r = Two{0.0f, 0.0f};
        if (a.tail) {
            list.r = two_add(Two{1.0f, 0.0f}, two_neg(list.ts));
            if (!(list.r.h > 0.0f))
                list.r = Two{0.0f, 0.0f};
        } else if (list.ts.h > 0.0f) {
#pragma unroll
            for (int j = 0; j < kMaxList / 32; ++j)
                if (32 * j < n)
                    list.t[j] = two_div(list.t[j], list.ts);
        }
    };
    // and its loss from the parts' sums and the list's logits, while the walkers have the next row's sums to take.
    struct {
        int64_t row;
        Two r, ts, t[kMaxList / 32];
        CtaPart part;
        float z[kMaxList / 32], a[kMaxList / 32], shift, mu, M, su;
        int code;
    } owed;
    owed.row = -1;
    if (scribe && rank == 0)
        read_list();
    const auto settle = [&] {
        if (owed.row < 0)
            return;
        Two loss{0.0f, 0.0f};
        if (owed.code == SV_OK && a.loss) {
            const Two iT{a.iT, a.iTl};
            Two off{0.0f, 0.0f}, on{0.0f, 0.0f};
            if (owed.part.m > -inf) {
                const Two s = two_sum(owed.part.hi * (1.0f / 64.0f), owed.part.lo * 3.6379788e-12f);
                off = two_mul(two_mul(s, Two{1.0f, kPowerBias}), two_exp(over(owed.part.m, owed.M, iT)));
            }
            // sums of t (a - shift - z / T), and of the listed weights
#pragma unroll
            for (int j = 0; j < kMaxList / 32; ++j) {
                if (32 * j >= n)
                    break;
                const Two y = over(owed.z[j], owed.M, iT);
                on = two_add(on, two_exp(y));
                if (owed.t[j].h > 0.0f) {
                    const Two d = two_add(two_sum(owed.a[j], -owed.shift), two_neg(y));
                    loss = two_finite(loss, two_mul(owed.t[j], d));
                }
            }
            off = warp_sum(off);
            on = warp_sum(on);
            const bool infinite = __any_sync(kAllLanes, loss.h == inf);
            loss = warp_sum(loss);
            const Two ls = two_log(two_add(on, off));
            if (a.tail)
                loss = two_add(loss, two_mul(owed.ts, ls));
            else
                loss = two_add(loss, two_add(ls, two_neg(two_log(owed.ts))));
            if (owed.r.h > 0.0f) {  // a tail too small beside M for its weight still has a logarithm
                const Two lu = off.h > 1e-30f ? two_log(off)
                               : owed.su > 0.0f ? two_add(over(owed.mu, owed.M, iT), two_log(Two{owed.su, 0.0f}))
                                                : Two{-inf, 0.0f};
                const Two d = two_add(two_log(owed.r), two_add(ls, two_neg(lu)));
                loss = two_finite(loss, two_mul(owed.r, d));
            }
            if (infinite || !(loss.h < inf))
                loss.h = inf, loss.l = 0.0f;
        }
        owed.code = owed.code < 0 ? SV_OK : owed.code;
        if (lane == 0) {
            if (a.loss)
                a.loss[owed.row] = owed.code ? __int_as_float(0x7fffffff) : loss.h + loss.l;
            if (a.status)
                a.status[owed.row] = owed.code;
            if (owed.code)
                atomicOr(a.err_word, 1u << owed.code);
        }
        owed.row = -1;
    };

    // Every CTA of a row arrives at all the others and waits for them, whatever it sees of the row: CTAs that see
    // different lists or lengths, which a program changes under the call, still end.  What others write has a place
    // for even turns and one for odd ones: a CTA is at most one turn ahead of another.
    uint32_t loads = 0;
    for (uint32_t turn = 0; row < a.rows; ++turn, row += clusters) {
        const uint32_t odd = turn & 1u, phase = (turn >> 1) & 1u;
        const unsigned char* base = row_base(row);
        unsigned char* grad = a.grad ? static_cast<unsigned char*>(a.grad) + row * a.grad_stride * ES : nullptr;
        const Part<ES> p(base, a.V, a.vectors, (int)rank);
        const bool more = row + clusters < a.rows;
        const bool live = __syncthreads_and(next_live);  // one answer for the CTA, whose last row is done with
        const bool dead = sh.dead[odd] != 0;
        if (teacher) {
            if (live && !dead && lane == 0) {
                uint32_t first;
                const uint32_t bytes = whole_vectors(p, first);
                barrier_expect(&sh.bar, bytes);
                const unsigned char* src = base - (size_t)p.off * ES + (size_t)first * 16;
                unsigned char* dst = reinterpret_cast<unsigned char*>(slice + (first - p.v0));
                for (uint32_t at = 0; at < bytes; at += kCopyPiece)
                    copy_bulk(dst + at, src + at, min(kCopyPiece, bytes - at), &sh.bar);
            }
            __syncwarp();
            // shares against the largest (top) or as they are (tail)
            uint32_t flags = 0;
            float top = -inf;
#pragma unroll
            for (int j = 0; j < kMaxList / 32; ++j) {
                const int k = lane + 32 * j;
                if (k >= n)
                    break;
                const int32_t y = tokens[j];
                float lp = logprobs[j];
                if (y < 0 || y >= a.V)
                    lp = -inf;
                else if (!(lp < inf))
                    flags |= 1u << SV_ERR_NONFINITE, lp = -inf;
                sh.a[k] = lp;
                sh.token[k] = y;
                top = fmaxf(top, lp);
            }
            __syncwarp();
            if (more) {
                next_live = is_live(row + clusters);
                fetch(row + clusters);
            }
            const float weight = grad && a.grad_loss ? a.grad_loss[row] : 1.0f;
            float shift = 0.0f, sum = 1.0f;
            if (!a.tail) {
                top = warp_max(top);
                shift = top > -inf ? top : 0.0f;
                sum = 0.0f;
#pragma unroll
                for (int j = 0; j < kMaxList / 32; ++j)
                    if (lane + 32 * j < n)
                        sum += expf(sh.a[lane + 32 * j] - shift);
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    sum += __shfl_xor_sync(kAllLanes, sum, o);
            }
            sh.list_max = shift;
            sh.list_sum = sum;
            // a token listed twice
            for (int k = lane; k < n; k += 32) {
                const int32_t y = sh.token[k];
                if (y >= 0)
                    for (int j = 0; j < k; ++j)
                        if (sh.token[j] == y)
                            flags |= 1u << SV_ERR_TOKEN_RANGE;
            }
            if (flags)
                atomicOr(&sh.flags, flags);
            __syncwarp();
            if (live && more && next_live && !dead && lane == 0) {  // the next row comes into L2 meanwhile
                const unsigned char* after = row_base(row + clusters);
                const Part<ES> q(after, a.V, a.vectors, (int)rank);
                uint32_t first;
                const uint32_t bytes = whole_vectors(q, first);
                if (bytes)
                    prefetch_bulk(after - (size_t)q.off * ES + (size_t)first * 16, bytes);
            }
            __syncwarp();
            if (dead || (!barrier_try_cluster(&sh.exchange[odd], phase) &&
                         !barrier_wait_cluster(&sh.exchange[odd], phase, kWaitNs)) ||
                (a.selftest == SV_SELFTEST_DISTILL_EXCHANGE && row == a.selftest_row && (int)rank == C - 1)) {
                atomicOr(&sh.flags, 1u << SV_ERR_TIMEOUT);
                sh.dead[odd ^ 1u] = 1;
            }
            __syncwarp();
            if (!live) {
                if (rank == 0 && lane == 0) {
                    if (a.loss)
                        a.loss[row] = 0.0f;
                    if (a.status)
                        a.status[row] = SV_OK;
                }
                if (lane == 0)
                    sh.flags = 0;
                continue;
            }
            const CtaPart part = sh.part[odd][lane % C];
            float mu = part.m, M = -inf, z[kMaxList / 32];
#pragma unroll
            for (int j = 0; j < kMaxList / 32; ++j) {
                const int k = lane + 32 * j;
                z[j] = k < n && sh.token[k] >= 0 ? sh.z[odd][k] : -inf;
                M = max_nan(M, z[j]);
            }
            mu = warp_max(mu);
            M = max_nan(mu, warp_max(M));
            const bool has = lane < C && part.m > -inf;
            float su = has ? fmaf(part.hi, 1.0f / 64.0f, part.lo * 3.6379788e-12f) * expf((part.m - mu) * a.iT) : 0.0f;
            float S = 0.0f;
#pragma unroll
            for (int j = 0; j < kMaxList / 32; ++j)
                if (32 * j < n)
                    S += z[j] > -inf ? expf((z[j] - M) * a.iT) : 0.0f;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                su += __shfl_xor_sync(kAllLanes, su, o);
                S += __shfl_xor_sync(kAllLanes, S, o);
            }
            if (__any_sync(kAllLanes, part.hi < 0.0f) && lane == 0) {
                atomicOr(&sh.flags, 1u << SV_ERR_TIMEOUT);
                sh.dead[odd ^ 1u] = 1;
            }
            __syncwarp();
            flags = sh.flags;
            const bool answer = flags || sh.listed;
            const int code = flags ? __ffs(flags) - 1
                             : answer && (!(M > -inf && M < inf) || !(sum > 0.0f)) ? SV_ERR_NONFINITE : SV_OK;
            const bool good = answer && code == SV_OK;
            // the draft's mass off the list
            const float wu = good && mu > -inf ? su * expf((mu - M) * a.iT) : 0.0f;
            S += wu;
            const float iS = __fdividef(1.0f, S), rest = wu * iS;
            // what rounding leaves of a list that holds all the mass there is, is no outcome
            float r = sh.r[odd], total = sh.total[odd];
            const bool nothing = rest < 1.17549435e-38f && r <= 9.5367432e-7f;
            if (nothing) {
                total -= r;
                r = 0.0f;
            }
            __syncwarp();
            if (lane == 0) {
                const float g = weight * a.iT;
                sh.answer = Answer{mu > -inf ? mu : 0.0f, su > 0.0f ? __fdividef(g * (total * rest - r), su) : 0.0f, M, iS,
                                   total, g, mu, su, answer ? code : -1, nothing};
                sh.listed = 0;  // for the next row
                sh.flags = 0;
            }
            __syncthreads();
            continue;
        }
        if (scribe) {
            if (rank == 0) {
                if (lane < C) {
                    store_cluster(cluster_addr(&sh.r[odd], lane), list.r.h);
                    store_cluster(cluster_addr(&sh.total[odd], lane), a.tail ? two_add(list.ts, list.r).h : 1.0f);
                    barrier_arrive_cluster(cluster_addr(&sh.exchange[odd], lane));
                }
                __syncwarp();
                if (more)
                    fetch(row + clusters);
                settle();
            }
            if (more)
                next_live = is_live(row + clusters);
            if (live && rank == 0) {
                if (!dead && !barrier_try_cluster(&sh.exchange[odd], phase))
                    barrier_wait_cluster(&sh.exchange[odd], phase, kWaitNs);  // the teacher says if it ran out
                __syncwarp();
                owed.part = lane < C ? sh.part[odd][lane] : CtaPart{0.0f, 0.0f, -inf};
                owed.r = list.r, owed.ts = list.ts, owed.shift = list.shift;
#pragma unroll
                for (int j = 0; j < kMaxList / 32; ++j) {
                    owed.t[j] = list.t[j], owed.a[j] = list.a[j];
                    owed.z[j] = (list.tokens >> j) & 1u ? sh.z[odd][lane + 32 * j] : -inf;
                }
            }
            if (live) {
                __syncthreads();  // what the teacher makes of the sums
                if (rank == 0) {
                    owed.row = row;
                    owed.mu = sh.answer.mu, owed.M = sh.answer.M, owed.su = sh.answer.su;
                    owed.code = sh.answer.kind;
                    if (sh.answer.nothing)
                        owed.r = Two{0.0f, 0.0f};
                }
            }
            if (rank == 0 && more)
                read_list();
            continue;
        }

        // the walkers
        int32_t x = tokens[0];  // listed token number tid
        float mine = -inf;      // and its logit, where it is of this slice
        bool own = false;
        if (live && !dead) {
            if (tid < 2 * E && p.v0 < p.v1) {  // the row's ends, where vectors are not whole
                const uint32_t k = tid < E ? p.v0 : p.v1 - 1;
                const int64_t id = (int64_t)k * E - p.off + tid % E;
                if (!p.whole(k)) {
                    const float z = id >= 0 && id < a.V ? scalar_entry<ES>(base, id) : -inf;
                    store_entry<ES>(reinterpret_cast<unsigned char*>(slice + (k - p.v0)), tid % E, z);
                }
            }
            if (x < -1 || x >= a.V) {
                atomicOr(&sh.flags, 1u << SV_ERR_TOKEN_RANGE);
                x = -1;
            }
            if (x >= 0)
                sh.listed = 1;
        }
        if (more) {
            next_live = is_live(row + clusters);
            fetch(row + clusters);
        }
        if (!live || dead) {
            if (warp == 0 && lane < C) {
                if (live)
                    store_cluster(cluster_addr(&sh.part[odd][rank].hi, lane), -1.0f);
                barrier_arrive_cluster(cluster_addr(&sh.exchange[odd], lane));
            }
            __syncwarp();
            if (live)
                __syncthreads();  // the others' warps wait for the teacher's answer
            const uint32_t v = !live ? 0u : ES == 4 ? 0x7fffffffu : 0x7fff7fffu;
            if (grad)
                write_part<ES>(p, grad, [&](uint32_t) { return make_uint4(v, v, v, v); });
            continue;
        }
        if (!barrier_wait(&sh.bar, loads & 1u, kCopyWaitNs) ||
            (a.selftest == SV_SELFTEST_DISTILL_COPY && row == a.selftest_row && (int)rank == C - 1)) {
            atomicOr(&sh.flags, 1u << SV_ERR_TIMEOUT);
            sh.dead[odd ^ 1u] = 1;
        }
        ++loads;
        sync_walkers();  // also the row's ends are in
        const uint32_t vectors = sh.listed ? p.v1 - p.v0 : 0;  // without a list there is nothing to sum
        // the listed entries leave the slice
        if (x >= 0) {
            const int64_t at = (int64_t)x + p.off;
            own = at >= (int64_t)p.v0 * E && at < (int64_t)p.v1 * E;
            if (own) {
                unsigned char* s8 = reinterpret_cast<unsigned char*>(slice);
                const int64_t i = at - (int64_t)p.v0 * E;
                mine = scalar_entry<ES>(s8, i);
                store_entry<ES>(s8, i, -inf);
                for (int c = 0; c < C; ++c)
                    store_cluster(cluster_addr(&sh.z[odd][tid], c), mine);
            }
        }
        sync_walkers();
        // Sums off the list against the largest of one vector per thread: a thread's stays below 2^12 unless that
        // misses the slice's largest by far (or there is a NaN), and then they are taken again against the largest
        // of all.  A sum that follows a growing maximum would be multiplied by powers that are each off by 2^-22.
        float m;
        for (uint32_t span = kNT;; span = vectors) {
            m = slice_max<ES>(slice, min(span, vectors));
            if (lane == 0)
                sh.warp_max[warp] = m;
            sync_walkers();
#pragma unroll
            for (int w = 0; w < kNW; ++w)
                m = max_nan(m, sh.warp_max[w]);
            float s = 0.0f;
            if (m > -inf) {
#pragma unroll 2
                for (uint32_t k = tid; k < vectors; k += kNT)
                    s += exp_vector_sum<ES>(slice[k], m, ch, cl);
            }
            // Threads' sums join as integers, 2^-38 a unit: in 12 and 26 bits behind the point, whose sums over a
            // warp stay below 2^29 and 2^31
            const bool fits = s < 4096.0f && (m > -inf || span >= vectors);
            const uint32_t whole = (uint32_t)(s * 4096.0f);
            const uint32_t part = (uint32_t)((s - (float)whole * (1.0f / 4096.0f)) * 274877906944.0f);
            const uint32_t hi = __reduce_add_sync(kAllLanes, whole), lo = __reduce_add_sync(kAllLanes, part);
            const bool all = __all_sync(kAllLanes, fits);
            if (lane == 0)
                sh.warp_sum[warp] = all ? ((unsigned long long)hi << 26) + lo : ~0ull;
            sync_walkers();
            if (span >= vectors)
                break;
            bool again = false;
#pragma unroll
            for (int w = 0; w < kNW; ++w)
                again |= sh.warp_sum[w] == ~0ull;
            if (!again)
                break;
            sync_walkers();  // before these are written again
        }
        if (warp == 0 && lane < C) {
            unsigned long long sum = 0;
#pragma unroll
            for (int w = 0; w < kNW; ++w)
                sum += sh.warp_sum[w];
            const uint32_t to = cluster_addr(&sh.part[odd][rank], lane);
            store_cluster(to, (sh.flags >> SV_ERR_TIMEOUT) & 1u ? -1.0f : (float)(uint32_t)(sum >> 32));
            store_cluster(to + 4, (float)(uint32_t)sum);
            store_cluster(to + 8, m);
            barrier_arrive_cluster(cluster_addr(&sh.exchange[odd], lane));
        }
        __syncthreads();  // what the teacher makes of the sums
        if (grad) {
            const Answer w = sh.answer;
            if (w.kind == SV_OK) {
                write_part<ES>(p, grad, [&](uint32_t i) { return exp_scaled<ES>(slice[i], w.m, ch, cl, w.k); });
                sync_walkers();  // the listed entries' gradients come after the others'
                if (own) {
                    const float q = expf((mine - w.M) * a.iT) * w.iS, t = expf(sh.a[tid] - sh.list_max) / sh.list_sum;
                    store_entry<ES>(grad, x, w.g * (w.total * q - t));
                }
            } else {  // zeros without a teacher, else NaN
                const uint32_t v = w.kind < 0 ? 0u : ES == 4 ? 0x7fffffffu : 0x7fff7fffu;
                write_part<ES>(p, grad, [&](uint32_t) { return make_uint4(v, v, v, v); });
            }
        }
        // what was written into the slice comes before the copies that fill it next
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (scribe && rank == 0)
        settle();
    // no CTA leaves before the others have written into it for the last time
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (tid == 0 && (sh.dead[0] | sh.dead[1])) {
        if (loads)
            barrier_wait(&sh.bar, (loads - 1) & 1u, kCopyWaitNs);  // the last copy that was issued
        atomicOr(a.err_word, 1u << SV_ERR_TIMEOUT);
    }
}

// Attributes of the kernels on a device, once.
bool setup(int device) {
    static std::atomic<unsigned long long> done{0};
    const unsigned long long bit = 1ull << (device & 63);
    if (device < 64 && (done.load(std::memory_order_acquire) & bit))
        return true;
    for (const void* fn : {(const void*)sv_distill_kernel<2>, (const void*)sv_distill_kernel<4>})
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kDistillSmem) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            (void)cudaGetLastError();
            return false;
        }
    if (device < 64)
        done.fetch_or(bit, std::memory_order_release);
    return true;
}

// How many clusters of a shape run at once: asked once for each shape.
int resident(const void* fn, int device, int es, const cudaLaunchConfig_t& like) {
    struct Known {
        int device, es, C, smem, clusters;
    };
    static std::mutex mutex;
    static Known known[64];
    static int count = 0;
    const int C = (int)like.attrs[0].val.clusterDim.x, smem = (int)like.dynamicSmemBytes;
    std::lock_guard<std::mutex> lock(mutex);
    for (int i = 0; i < (count < 64 ? count : 64); ++i)
        if (known[i].device == device && known[i].es == es && known[i].C == C && known[i].smem == smem)
            return known[i].clusters;
    cudaLaunchConfig_t cfg = like;
    cfg.gridDim = dim3((unsigned)C, 1, 1);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return 0;
    }
    known[count++ % 64] = Known{device, es, C, smem, n};
    return n;
}

}  // namespace

extern "C" {

int spec_distill_get_plan(sv_ctx* ctx, int B, int rows_per_seq, int64_t V, int logits_dtype, sv_plan* out) {
    if (!ctx)
        return SV_ERR_INVALID_ARG;
    return spec_distill_plan_for(ctx->num_sms, ctx->sampling_max_cluster, B, rows_per_seq, V, logits_dtype,
                                 ctx->ovr_cluster, out);
}

int spec_distill_run(sv_ctx* ctx, const void* draft_logits, int logits_dtype, int64_t logits_stride,
                     const float* top_logprobs, const int32_t* top_tokens, int n, const int32_t* accept_len, int B,
                     int rows_per_seq, int64_t V, float temperature, int tail, const float* grad_loss, float* loss,
                     void* grad_logits, int64_t grad_stride, int32_t* status, void* stream) {
    if (!ctx || !draft_logits || !top_logprobs || !top_tokens || (!loss && !grad_logits) ||
        (logits_dtype != SV_F32 && logits_dtype != SV_BF16))
        return SV_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 40;
    if (B < 1 || B > ctx->max_B || rows_per_seq < 1 || rows_per_seq > ctx->max_K + 1 || V < 1 || V > ctx->max_V ||
        V > ((int64_t)1 << 31) - 1 || n < 1 || n > kMaxList || logits_stride < V || logits_stride > most ||
        (double)B * (double)rows_per_seq * (double)logits_stride >= 1099511627776.0)  // 2^40
        return SV_ERR_INVALID_ARG;
    // 2^-100 .. 2^100: differences of any two logits over T, and their exponents, stay what they are
    if (!(temperature >= 7.8886091e-31f) || !(temperature <= 1.2676506e30f) || (tail != 0 && tail != 1))
        return SV_ERR_INVALID_ARG;
    const int es = logits_dtype == SV_BF16 ? 2 : 4;
    if (!aligned(draft_logits, es) || !aligned(top_logprobs, 4) || !aligned(top_tokens, 4) ||
        !aligned(accept_len, 4) || !aligned(grad_loss, 4) || !aligned(loss, 4) || !aligned(grad_logits, es) ||
        !aligned(status, 4))
        return SV_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)B * rows_per_seq;
    if (grad_logits) {
        if (grad_stride < V || grad_stride > most || (double)rows * (double)grad_stride >= 1099511627776.0)
            return SV_ERR_INVALID_ARG;
        // in place, or apart: rows that overlap others would be read after they were written
        if (!(grad_logits == draft_logits && (rows == 1 || logits_stride == grad_stride)) &&
            rows_meet(draft_logits, logits_stride * es, grad_logits, grad_stride * es, rows, V * es))
            return SV_ERR_INVALID_ARG;
    }
    sv_plan plan;
    const int rc = spec_distill_get_plan(ctx, B, rows_per_seq, V, logits_dtype, &plan);
    if (rc != SV_OK)
        return rc;
    Args a;
    std::memset(&a, 0, sizeof a);
    a.logits = draft_logits;
    a.stride = logits_stride;
    a.top_logprobs = top_logprobs;
    a.top_tokens = top_tokens;
    a.accept_len = accept_len;
    a.grad_loss = grad_loss;
    a.loss = loss;
    a.grad = grad_logits;
    a.grad_stride = grad_stride;
    a.status = status;
    a.err_word = ctx->d_err;
    a.V = V;
    a.rows = rows;
    a.rows_per_seq = rows_per_seq;
    a.C = plan.cluster;
    a.n = n;
    a.tail = tail;
    a.vectors = (uint32_t)(plan.slice * es / 16);
    a.iT = (float)(1.0 / (double)temperature);
    a.iTl = (float)(1.0 / (double)temperature - (double)a.iT);
    const double c = 1.4426950408889634074 / (double)temperature;
    a.ch = (float)c;
    if ((double)a.ch > c)
        a.ch = std::nextafterf(a.ch, 0.0f);
    a.cl = (float)(c - (double)a.ch);
    if (!(a.cl >= 1.17549435e-38f))  // a difference of -inf times it is -inf
        a.cl = 1.17549435e-38f;
    a.selftest = losses_selftest(ctx);
    a.selftest_row = rows / 2;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.blockDim = dim3(kNT + 64, 1, 1);
    cfg.dynamicSmemBytes = (size_t)plan.smem_bytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    DeviceGuard guard(ctx->device);
    if (!setup(ctx->device))
        return SV_ERR_CUDA;
    const auto kernel = es == 2 ? sv_distill_kernel<2> : sv_distill_kernel<4>;
    int64_t clusters = rows;
    if (plan.grid > ctx->num_sms) {  // as many as run at once, which take the rows in turn
        const int most_clusters = resident((const void*)kernel, ctx->device, es, cfg);
        if (most_clusters < 1)
            return SV_ERR_CUDA;
        clusters = rows < most_clusters ? rows : most_clusters;
    }
    cfg.gridDim = dim3((unsigned)(clusters * plan.cluster), 1, 1);
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SV_ERR_CUDA;
    }
    return SV_OK;
}

}  // extern "C"
