// logprobs.cu -- log-probabilities of the tokens a verify emitted, their
// ranks, and the largest entries of their rows.
//
// For a row l reached by the verify and its token x:
//   logprob = (l_x - l_max)/T - ln sum exp((l - l_max)/T)
//   rank    = 1 + #{l > l_x}
//   top n   = the n largest entries by descending logit and ascending id
//
// Design: one cluster of C CTAs per row, a slice of the vocabulary per CTA;
// rows from accept_len on are not read.  One pass takes the maximum, the sum
// (rescaled when a thread's maximum grows), the count above l_x, and every
// thread's largest entry, and of each step of four vectors in eight bits.  The n-th
// largest of a CTA's thread maxima bounds its n-th largest entry from below: only threads
// whose maximum reaches that bound look at their entries again, in those steps that
// may hold one (without the eight bits, at all of them: 90 instead of 71 us below), and
// hand them to a short list.  Each CTA sends its n best to the first one, which orders them.
//
// What bounds it: waiting for the pass's loads (four vectors a thread, one step ahead, four CTAs
// an SM: nearly four warps wait for each one that issues, and no pipe is above 30 %), and the chain after it:
// 256 x 8 rows of 128256 bfloat16, 56% of them live, top 20: 67 us for 296 MB, 4.4 TB/s;
// 37 x 3 rows of 50257 float32 14 us; 8 x 5 rows of 32000 bfloat16 9 us, a launch and
// sixteen barriers for the bound.  Where fewer tokens than n are left beside a finite mask, the mask's
// value is the bound, and each of the n best takes a walk of its own: 150 rows of 50257, top 20, 190 us
// instead of 25.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_verify.h"
#include "sampling_common.cuh"
#include "sv_context.h"

namespace cg = cooperative_groups;

namespace {

using namespace sv;

constexpr int kNT = 256;
constexpr int kNW = kNT / 32;
constexpr int kMaxC = 16;
constexpr int kMaxTop = 32;
constexpr int kList = 1024;

struct Args {
    const void* logits;
    int64_t stride;
    const int32_t* tokens;
    const int32_t* accept_len;  // or NULL: every row
    float* logprob;
    int32_t* rank;
    float* top_logprobs;
    int32_t* top_tokens;
    int32_t* status;
    uint32_t* err_word;
    int64_t V, slice;
    int rows_per_seq, C, top_n;
    float T, ch;
};

struct Shared {
    unsigned long long list[kList];         // key << 32 | ~id
    unsigned long long best[kMaxC][kMaxTop];  // first CTA: every CTA's n best, 0 behind the last
    float part_max[kMaxC], part_sum[kMaxC];
    uint32_t part_above[kMaxC];
    float warp_max[kNW], warp_sum[kNW];
    uint32_t warp_above[kNW];
    uint32_t list_n;
    unsigned long long warp_best[kNW];
};

__device__ __forceinline__ unsigned long long order_of(float l, uint32_t id) {
    return ((unsigned long long)logit_key(l) << 32) | (uint32_t)~id;
}

// x - y, or at temperatures from kFarT on (x - y) kShrink
template <bool Far>
__device__ __forceinline__ float apart(float x, float y) {
    return Far ? x * kShrink - y * kShrink : x - y;
}

// `Far`: T from kFarT on, where logits may lie further apart than a float holds.  a.T and a.ch
// are those of the smaller logits then.
template <int ES, bool Far>
__global__ void __launch_bounds__(kNT, 4) sv_logprobs_kernel(const __grid_constant__ Args a) {
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int E = 16 / ES;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.C, rank = (int)cluster.block_rank(), n = a.top_n;
    const int64_t row = blockIdx.x / C, seq = row / a.rows_per_seq;
    const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fffffff);

    const auto leave = [&](int code) {  // a row with no answer
        if (rank == 0) {
            if (tid == 0) {
                a.logprob[row] = nan;
                if (a.rank)
                    a.rank[row] = 0;
                if (a.status)
                    a.status[row] = code;
                if (code)
                    atomicOr(a.err_word, 1u << code);
            }
            if (tid < n) {
                a.top_logprobs[row * n + tid] = nan;
                a.top_tokens[row * n + tid] = -1;
            }
        }
    };
    const int32_t x = a.tokens[row];  // both loads at once
    const bool dead = a.accept_len && row - seq * a.rows_per_seq >= a.accept_len[seq];
    if (dead || x < 0 || x >= a.V) {
        leave(dead ? SV_OK : SV_ERR_TOKEN_RANGE);
        // where a program changes these under the call, CTAs of a row may differ: none leaves while
        // another may still write into it
        if (C > 1) {
            cluster.sync();
            cluster.sync();
        }
        return;
    }
    const unsigned char* base = static_cast<const unsigned char*>(a.logits) + row * a.stride * ES;
    const float lx = scalar_entry<ES>(base, x);
    const Slice<ES, kNT> v(base, a.V, a.slice, rank);

    cluster.barrier_arrive();

    // the pass over the slice
    float m = -inf, s = 0.0f;
    uint32_t above = 0;
    const auto merge = [&](float& m0, float& s0, float m1, float s1) {
        if constexpr (Far) {
            const float grown = max_nan(m0, m1);
            s0 = (m0 > -inf ? s0 * ex2_approx(apart<true>(m0, grown) * a.ch) : 0.0f) +
                 (m1 > -inf ? s1 * ex2_approx(apart<true>(m1, grown) * a.ch) : 0.0f);
            m0 = grown;
        } else {
            join_sums(m0, s0, m1, s1, a.ch);
        }
    };
    const auto grow = [&](float top) { merge(m, s, top, 0.0f); };
    StepCodes codes;
    const int shift = v.code_shift();
    if (shift) {  // else every step has a code of its own
#pragma unroll
        for (int i = 0; i < 16; ++i)
            codes.code[i] = 0;
    }
    float step = -inf;  // the step's largest
    v.template walk_steps<kDeep, false>(
        [&](const uint4& w, uint32_t) {
            const float top = vector_max_nan<ES>(w);
            step = max_nan(step, top);
            if (!(top <= m))
                grow(top);
            if (top > lx) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    above += vector_entry<ES>(w, e) > lx;
            }
            if (top > -inf) {  // else m may be -inf too
                if constexpr (Far) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        s += ex2_approx(apart<true>(vector_entry<ES>(w, e), m) * a.ch);
                } else {
                    s += exp_sum<ES>(w, m, a.ch);
                }
            }
        },
        [&](uint32_t i) {
            const uint8_t x = (uint8_t)step_code(step);
            if (shift == 0 || x > codes.code[i >> shift])
                codes.code[i >> shift] = x;
            step = -inf;
        },
        [&](uint32_t id) {
            const float l = scalar_entry<ES>(base, id);
            above += l > lx;
            if (!(l <= m))
                grow(l);
            if (l > -inf)
                s += ex2_approx(apart<Far>(l, m) * a.ch);
        });
    const float mine = m;

    // join the threads, then the CTAs
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float m1 = __shfl_xor_sync(kAllLanes, m, o), s1_ = __shfl_xor_sync(kAllLanes, s, o);
        merge(m, s, m1, s1_);
    }
    above = __reduce_add_sync(kAllLanes, above);
    if (lane == 0) {
        sh.warp_max[warp] = m;
        sh.warp_sum[warp] = s;
        sh.warp_above[warp] = above;
    }
    if (tid == 0)
        sh.list_n = 0;
    __syncthreads();
    cluster.barrier_wait();  // every CTA of the cluster runs: its memory may be written
    if (tid == 0) {
        for (int w = 1; w < kNW; ++w) {
            merge(m, s, sh.warp_max[w], sh.warp_sum[w]);
            above += sh.warp_above[w];
        }
        *cluster.map_shared_rank(&sh.part_max[rank], 0) = m;
        *cluster.map_shared_rank(&sh.part_sum[rank], 0) = s;
        *cluster.map_shared_rank(&sh.part_above[rank], 0) = above;
    }

    // the CTA's n largest
    if (n) {
        // bound: the largest key that n threads' maxima reach (bf16: its upper half says all)
        const uint32_t key = logit_key(mine);
        uint32_t bound = 0;
        for (int bit = 31; bit >= (ES == 2 ? 16 : 0); --bit) {
            const uint32_t t = bound | (1u << bit);
            if (__syncthreads_count(key >= t) >= n)
                bound = t;
        }
        if (bound <= kKeyMinusInf)
            bound = kKeyMinusInf + 1;
        if (key >= bound) {
            const auto offer = [&](float l, uint32_t id) {
                if (logit_key(l) >= bound) {
                    const uint32_t at = atomicAdd(&sh.list_n, 1u);
                    if (at < (uint32_t)kList)
                        sh.list[at] = order_of(l, id);
                }
            };
            const float least = key_logit(bound);
            v.template walk_marked<kDeep>(
                v.marks(&codes, step_code(least)),
                [&](const uint4& w, uint32_t id) {
                    if (vector_max<ES>(w) >= least) {
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            offer(vector_entry<ES>(w, e), id + e);
                    }
                },
                [&](uint32_t id) { offer(scalar_entry<ES>(base, id), id); });
        }
        __syncthreads();
        const uint32_t got = sh.list_n;
        unsigned long long* best = cluster.map_shared_rank(sh.best[rank], 0);
        if (got <= (uint32_t)kList) {
            // an entry's place is the number of entries before it
            for (uint32_t i = tid; i < got; i += kNT) {
                const unsigned long long o = sh.list[i];
                int place = 0;
                for (uint32_t j = 0; j < got && place < n; ++j)
                    place += sh.list[j] > o;
                if (place < n)
                    best[place] = o;
            }
            for (int i = (int)got + tid; i < n; i += kNT)
                best[i] = 0;
        } else {
            // many equal logits at the bound: one entry after the other
            unsigned long long last = ~0ull;
            for (int r = 0; r < n; ++r) {
                unsigned long long o = 0;
                for (uint32_t i = v.s0 + tid; i < v.s1; i += kNT) {
                    const unsigned long long y = order_of(scalar_entry<ES>(base, i), i);
                    if (y < last && y > o && (uint32_t)(y >> 32) > kKeyMinusInf)
                        o = y;
                }
                for (int k = 16; k; k >>= 1) {
                    const unsigned long long y = __shfl_xor_sync(kAllLanes, o, k);
                    o = y > o ? y : o;
                }
                if (lane == 0)
                    sh.warp_best[warp] = o;
                __syncthreads();
                for (int w = 0; w < kNW; ++w)
                    o = sh.warp_best[w] > o ? sh.warp_best[w] : o;
                if (tid == 0)
                    best[r] = o;
                last = o;
                __syncthreads();
            }
        }
    }
    cluster.sync();
    if (rank)
        return;
    m = sh.part_max[0];
    s = sh.part_sum[0];
    above = sh.part_above[0];
    for (int r = 1; r < C; ++r) {
        merge(m, s, sh.part_max[r], sh.part_sum[r]);
        above += sh.part_above[r];
    }
    if (!(m > -inf && m < inf)) {
        leave(SV_ERR_NONFINITE);
        return;
    }
    const float ls = logf(s);
    const auto value = [&](float l) {
        // by halves: l - m may be no float where (l - m) / T is one
        return Far ? fmaf(apart<true>(l, m), 1.0f / a.T, -ls) : fmaf(0.5f * l - 0.5f * m, 2.0f / a.T, -ls);
    };
    if (tid == 0) {
        a.logprob[row] = value(lx);
        if (a.rank)
            a.rank[row] = (int32_t)min(above + 1, 0x7fffffffu);
        if (a.status)
            a.status[row] = SV_OK;
    }
    // order the CTAs' best
    int listed = 0;
    for (int i0 = 0; i0 < C * n; i0 += kNT) {
        const int i = i0 + tid;
        const unsigned long long o = i < C * n ? sh.best[i / n][i % n] : 0;
        listed += __syncthreads_count(o != 0);
        if (!o)
            continue;
        int place = 0;
        for (int r = 0; r < C; ++r)
            for (int j = 0; j < n && sh.best[r][j] > o; ++j)
                ++place;
        if (place < n) {
            a.top_logprobs[row * n + place] = value(key_logit((uint32_t)(o >> 32)));
            a.top_tokens[row * n + place] = (int32_t)~(uint32_t)o;
        }
    }
    if (tid >= listed && tid < n) {
        a.top_logprobs[row * n + tid] = nan;
        a.top_tokens[row * n + tid] = -1;
    }
}

}  // namespace

namespace sv {

bool logprobs_setup() {
    for (const void* fn : {(const void*)sv_logprobs_kernel<2, false>, (const void*)sv_logprobs_kernel<4, false>,
                           (const void*)sv_logprobs_kernel<2, true>, (const void*)sv_logprobs_kernel<4, true>})
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return false;
        }
    return true;
}

}  // namespace sv

extern "C" {

int spec_logprobs_get_plan(sv_ctx* ctx, int B, int rows_per_seq, int64_t V, int logits_dtype,
                           sv_plan* out) {
    if (!ctx)
        return SV_ERR_INVALID_ARG;
    return spec_logprobs_plan_for(ctx->num_sms, ctx->sampling_max_cluster, B, rows_per_seq, V,
                                  logits_dtype, ctx->ovr_cluster, out);
}

int spec_logprobs_run(sv_ctx* ctx, const void* target_logits, int logits_dtype,
                      int64_t logits_stride, const int32_t* tokens, const int32_t* accept_len,
                      int B, int rows_per_seq, int64_t V, float temperature, int top_n,
                      float* logprob, int32_t* rank, float* top_logprobs, int32_t* top_tokens,
                      int32_t* status, void* stream) {
    if (!ctx || !target_logits || !tokens || !logprob ||
        (logits_dtype != SV_F32 && logits_dtype != SV_BF16))
        return SV_ERR_INVALID_ARG;
    if (B < 1 || B > ctx->max_B || rows_per_seq < 1 || rows_per_seq > ctx->max_K + 1 || V < 1 ||
        V > ctx->max_V || V > ((int64_t)1 << 31) || logits_stride < V ||
        logits_stride > ((int64_t)1 << 40) ||
        (double)B * (double)rows_per_seq * (double)logits_stride >= 1099511627776.0)  // 2^40
        return SV_ERR_INVALID_ARG;
    if (!(temperature >= 1.17549435e-38f) || !std::isfinite(temperature) || top_n < 0 ||
        top_n > kMaxTop || (top_n && (!top_logprobs || !top_tokens)))
        return SV_ERR_INVALID_ARG;
    const int es = logits_dtype == SV_BF16 ? 2 : 4;
    if (!aligned(target_logits, es) || !aligned(tokens, 4) || !aligned(accept_len, 4) ||
        !aligned(logprob, 4) || !aligned(rank, 4) || !aligned(top_logprobs, 4) ||
        !aligned(top_tokens, 4) || !aligned(status, 4))
        return SV_ERR_INVALID_ARG;
    sv_plan plan;
    const int rc = spec_logprobs_get_plan(ctx, B, rows_per_seq, V, logits_dtype, &plan);
    if (rc != SV_OK)
        return rc;
    Args a;
    std::memset(&a, 0, sizeof a);
    a.logits = target_logits;
    a.stride = logits_stride;
    a.tokens = tokens;
    a.accept_len = accept_len;
    a.logprob = logprob;
    a.rank = rank;
    a.top_logprobs = top_logprobs;
    a.top_tokens = top_tokens;
    a.status = status;
    a.err_word = ctx->d_err;
    a.V = V;
    a.slice = plan.slice;
    a.rows_per_seq = rows_per_seq;
    a.C = plan.cluster;
    a.top_n = top_n;
    const bool far = temperature >= kFarT;
    a.T = far ? temperature * kShrink : temperature;
    a.ch = (float)(1.4426950408889634074 / (double)a.T);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)plan.grid, 1, 1);
    cfg.blockDim = dim3(kNT, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    DeviceGuard guard(ctx->device);
    const auto kernel = far ? (es == 2 ? sv_logprobs_kernel<2, true> : sv_logprobs_kernel<4, true>)
                            : (es == 2 ? sv_logprobs_kernel<2, false> : sv_logprobs_kernel<4, false>);
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SV_ERR_CUDA;
    }
    return SV_OK;
}

}  // extern "C"
