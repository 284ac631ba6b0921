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
// Design: one cluster of C CTAs per row.  Each CTA's slice of the row is copied to shared memory
// once (cp.async.bulk) and stays there: the sums and the gradient are both taken from it, so that a
// row is read once and its gradient written once whatever is asked for.  The listed entries are taken
// out of the slice (-inf in their place) before the sums: what is summed then is the mass off the
// list, without the cancellation of S - sum of listed weights, and against the maximum off the list, so
// that q_v / q_rest is right where the whole tail underflows next to a listed entry.  The CTAs
// exchange (maximum, sum) of both parts through distributed shared memory; r and the loss, where
// float32 would lose what 1 - sum t_k or a small loss leaves, are taken in 64 bits by the first CTA
// from a few numbers per row.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_verify.h"
#include "distill_plan.h"
#include "losses_common.cuh"
#include "sampling_common.cuh"
#include "sv_context.h"

namespace cg = cooperative_groups;

namespace {

using namespace sv;

constexpr int kNT = kDistillThreads;
constexpr int kNW = kNT / 32;
constexpr int kMaxC = 16;
constexpr int kMaxList = kDistillMaxList;
constexpr uint32_t kCopyPiece = 16384;

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
    int64_t V;
    int rows_per_seq, C, n, tail;
    uint32_t vectors;  // per CTA
    float T, ch;       // log2(e) / T
};

struct Shared {
    double t[kMaxList];  // first CTA: the list's shares
    float a[kMaxList];
    int32_t token[kMaxList];
    float z[kMaxList];  // first CTA: the draft logits of the list
    float4 part[kMaxC];  // every CTA's (maximum, sum) off the list and on it
    float2 warp_off[kNW], warp_on[kMaxList / 32];
    float r, total;  // from the first CTA
    double r64, log_sum;  // first CTA: r, and ln sum exp(a - largest a)
    float list_max, list_sum;
    uint32_t flags;  // bit 0: a listed token; above: 1 << code
    uint64_t bar;
};

// 2^((z - m) c) times k for a vector's logits, in the logits' type
template <int ES>
__device__ __forceinline__ uint4 exp_scaled(const uint4& v, float m, float c, float k) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[4];
    unsigned long long cc, kk;
    asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
    asm("mov.b64 %0, {%1, %1};" : "=l"(kk) : "f"(k));
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
        asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tmul.rn.f32x2 %0, d, %3;\n\t}"
            : "=l"(t)
            : "f"(ex2_approx(lo)), "f"(ex2_approx(hi)), "l"(kk));
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

// Writes f(k, local vector) as the gradient's vectors of this part.
template <int ES, typename F>
__device__ __forceinline__ void write_part(const Part<ES>& p, unsigned char* grad, F f) {
    constexpr int E = 16 / ES;
    const bool same = (uint32_t)(reinterpret_cast<uintptr_t>(grad) & 15u) / ES == p.off;
    uint4* vectors = reinterpret_cast<uint4*>(grad - (size_t)p.off * ES);
    for (uint32_t k = p.v0 + threadIdx.x; k < p.v1; k += kNT) {
        const uint4 w = f(k - p.v0);
        if (same && p.whole(k)) {
            vectors[k] = w;
        } else {
            // the row's ends, and rows whose gradient lies otherwise to 16 bytes than they do: entry by entry
            const int64_t id = (int64_t)k * E - p.off;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (id + e >= 0 && id + e < p.V)
                    store_entry<ES>(grad, id + e, vector_entry<ES>(w, e));
        }
    }
}

template <int ES>
__global__ void __launch_bounds__(kNT, 3) sv_distill_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(128) uint4 slice[];
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    constexpr int E = 16 / ES;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.C, rank = (int)cluster.block_rank(), n = a.n;
    const int64_t row = blockIdx.x / C, seq = row / a.rows_per_seq;
    const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fffffff);
    const unsigned char* base = static_cast<const unsigned char*>(a.logits) + row * a.stride * ES;
    unsigned char* grad = a.grad ? static_cast<unsigned char*>(a.grad) + row * a.grad_stride * ES : nullptr;
    const Part<ES> p(base, a.V, a.vectors, rank);

    // every way through the kernel passes both barriers of the cluster once: CTAs of a row that see
    // different lists or lengths, which a program changes under the call, still end
    cluster.barrier_arrive();
    const bool live = !a.accept_len || row - seq * a.rows_per_seq < a.accept_len[seq];
    bool answer = live;  // the row has a teacher
    int code = SV_OK;
    float M = 0.0f, S = 1.0f, mu = -inf, su = 0.0f, r = 0.0f, total = 1.0f;
    float mine = -inf;  // listed logit of token number tid, where it is of this slice
    bool own = false;
    if (live) {
        if (tid == 0) {
            sh.flags = 0;
            barrier_init(&sh.bar, 1);
            barrier_init_fence();
            uint32_t w0 = p.v0, w1 = p.v1;
            if (w0 < w1 && !p.whole(w0))
                ++w0;
            if (w0 < w1 && !p.whole(w1 - 1))
                --w1;
            const uint32_t bytes = (w1 - w0) * 16u;
            barrier_expect(&sh.bar, bytes);
            const unsigned char* src = base - (size_t)p.off * ES + (size_t)w0 * 16;
            unsigned char* dst = reinterpret_cast<unsigned char*>(slice + (w0 - p.v0));
            for (uint32_t at = 0; at < bytes; at += kCopyPiece)
                copy_bulk(dst + at, src + at, min(kCopyPiece, bytes - at), &sh.bar);
        }
        if (tid < 2 * E && p.v0 < p.v1) {  // the row's ends, where vectors are not whole
            const uint32_t k = tid < E ? p.v0 : p.v1 - 1;
            const int64_t id = (int64_t)k * E - p.off + tid % E;
            if (!p.whole(k)) {
                const float z = id >= 0 && id < a.V ? scalar_entry<ES>(base, id) : -inf;
                store_entry<ES>(reinterpret_cast<unsigned char*>(slice + (k - p.v0)), tid % E, z);
            }
        }
        // the list
        int32_t x = -1;
        uint32_t flags = 0;
        if (tid < n) {
            x = a.top_tokens[row * n + tid];
            float lp = a.top_logprobs[row * n + tid];
            if (x < -1 || x >= a.V) {
                flags = 1u << SV_ERR_TOKEN_RANGE;
                x = -1;
            }
            if (x >= 0) {
                flags |= 1u;
                if (!(lp < inf)) {
                    flags |= 1u << SV_ERR_NONFINITE;
                    lp = -inf;
                }
            } else {
                lp = -inf;
            }
            sh.token[tid] = x;
            sh.a[tid] = lp;
        }
        __syncthreads();
        if (tid < n && x >= 0) {
            bool twice = false;
            for (int j = 0; j < tid; ++j)
                twice |= sh.token[j] == x;
            if (twice) {
                flags |= 1u << SV_ERR_TOKEN_RANGE;
                x = -1;
            }
        }
        if (flags)
            atomicOr(&sh.flags, flags);
        if (warp == 0) {
            float top = -inf;
            for (int k = lane; k < n; k += 32)
                top = fmaxf(top, sh.a[k]);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(kAllLanes, top, o));
            // shares against the largest (top) or as they are (tail)
            const float shift = a.tail ? 0.0f : top > -inf ? top : 0.0f;
            float sum = 0.0f;
            for (int k = lane; k < n; k += 32)
                sum += expf(sh.a[k] - shift);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                sum += __shfl_xor_sync(kAllLanes, sum, o);
            if (lane == 0) {
                sh.list_max = shift;
                sh.list_sum = a.tail ? 1.0f : sum;
            }
            if (rank == 0) {
                double s = 0.0;
                for (int k = lane; k < n; k += 32) {
                    const double t = exp((double)sh.a[k] - (double)shift);
                    sh.t[k] = t;
                    s += t;
                }
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    s += __shfl_xor_sync(kAllLanes, s, o);
                const double rest = a.tail ? fmax(0.0, 1.0 - s) : 0.0;
                if (lane == 0) {
                    sh.r64 = rest;
                    sh.log_sum = a.tail ? 0.0 : log(s);
                }
                const float r_ = (float)rest, total_ = a.tail ? (float)(s + rest) : 1.0f;
                for (int k = lane; k < n; k += 32)
                    if (!a.tail)
                        sh.t[k] /= s;
                cluster.barrier_wait();  // every CTA of the cluster runs: its memory may be written
                if (lane < C) {
                    *cluster.map_shared_rank(&sh.r, lane) = r_;
                    *cluster.map_shared_rank(&sh.total, lane) = total_;
                }
            } else {
                cluster.barrier_wait();
            }
        } else {
            cluster.barrier_wait();
        }
        if (!barrier_wait(&sh.bar, 0, kCopyWaitNs))
            atomicOr(&sh.flags, 1u << SV_ERR_TIMEOUT);
        __syncthreads();
        // the listed entries leave the slice
        if (tid < n && x >= 0) {
            const int64_t at = (int64_t)x + p.off;
            own = at >= (int64_t)p.v0 * E && at < (int64_t)p.v1 * E;
            if (own) {
                unsigned char* s8 = reinterpret_cast<unsigned char*>(slice);
                const int64_t i = at - (int64_t)p.v0 * E;
                mine = scalar_entry<ES>(s8, i);
                store_entry<ES>(s8, i, -inf);
                *cluster.map_shared_rank(&sh.z[tid], 0) = mine;
            }
        }
        __syncthreads();
        answer = sh.flags & 1u;
        // sums off the list
        float m = -inf, s = 0.0f;
        if (sh.flags)  // without a list there is nothing to sum
            for (uint32_t k = tid; k < p.v1 - p.v0; k += kNT) {
                const uint4 w = slice[k];
                const float top = vector_max_nan<ES>(w);
                if (!(top <= m))
                    join_sums(m, s, top, 0.0f, a.ch);
                if (top > -inf)  // else m may be -inf too
                    s += exp_sum<ES>(w, m, a.ch);
            }
        join_lanes<32>(m, s, a.ch);
        if (lane == 0)
            sh.warp_off[warp] = make_float2(m, s);
        if (warp < kMaxList / 32) {
            float mo = mine, so = own ? 1.0f : 0.0f;
            join_lanes<32>(mo, so, a.ch);
            if (lane == 0)
                sh.warp_on[warp] = make_float2(mo, so);
        }
        __syncthreads();
        if (warp == 0) {
            const float2 off = lane < kNW ? sh.warp_off[lane] : make_float2(-inf, 0.0f);
            const float2 on = lane < kMaxList / 32 ? sh.warp_on[lane] : make_float2(-inf, 0.0f);
            float m0 = off.x, s0 = off.y, m1 = on.x, s1 = on.y;
            join_lanes<8>(m0, s0, a.ch);
            join_lanes<8>(m1, s1, a.ch);
            m0 = __shfl_sync(kAllLanes, m0, 0), s0 = __shfl_sync(kAllLanes, s0, 0);
            m1 = __shfl_sync(kAllLanes, m1, 0), s1 = __shfl_sync(kAllLanes, s1, 0);
            if (lane < C)
                *cluster.map_shared_rank(&sh.part[rank], lane) = make_float4(m0, s0, m1, s1);
        }
    } else {
        cluster.barrier_wait();
    }
    cluster.sync();

    if (live && answer) {
        float4 part = lane < C ? sh.part[lane] : make_float4(-inf, 0.0f, -inf, 0.0f);
        join_lanes<16>(part.x, part.y, a.ch);
        join_lanes<16>(part.z, part.w, a.ch);
        mu = __shfl_sync(kAllLanes, part.x, 0), su = __shfl_sync(kAllLanes, part.y, 0);
        M = __shfl_sync(kAllLanes, part.z, 0), S = __shfl_sync(kAllLanes, part.w, 0);
        join_sums(M, S, mu, su, a.ch);
        const uint32_t flags = sh.flags >> 1;
        if (flags)
            code = __ffs(flags);
        else if (!(M > -inf && M < inf) || !(sh.list_sum > 0.0f))
            code = SV_ERR_NONFINITE;
        r = sh.r;
        total = sh.total;
    } else if (live && sh.flags) {
        code = __ffs(sh.flags >> 1);  // a list of nothing but errors
        answer = true;
    }
    const bool good = answer && code == SV_OK;
    // the draft's mass off the list
    const float wu = good && mu > -inf ? su * ex2_approx((mu - M) * a.ch) : 0.0f;
    const float rest = wu / S;
    // what rounding leaves of a list that holds all the mass there is, is no outcome
    const bool nothing = rest < 1.17549435e-38f && r <= 9.5367432e-7f;
    if (nothing) {
        total -= r;
        r = 0.0f;
    }

    if (grad) {
        if (!answer) {
            write_part<ES>(p, grad, [](uint32_t) { return make_uint4(0, 0, 0, 0); });
        } else {
            const float g = (a.grad_loss ? a.grad_loss[row] : 1.0f) / a.T;
            const float k = !good ? nan : su > 0.0f ? g * ((total * rest - r) / su) : 0.0f;
            const float m = good && mu > -inf ? mu : 0.0f;
            if (good)
                write_part<ES>(p, grad, [&](uint32_t i) { return exp_scaled<ES>(slice[i], m, a.ch, k); });
            else
                write_part<ES>(p, grad, [&](uint32_t) {
                    const uint32_t w = ES == 4 ? 0x7fffffffu : 0x7fff7fffu;
                    return make_uint4(w, w, w, w);
                });
            __syncthreads();  // the listed entries' gradients come after the others'
            if (good && own) {
                const float q = expf((mine - M) / a.T) / S, t = expf(sh.a[tid] - sh.list_max) / sh.list_sum;
                store_entry<ES>(grad, sh.token[tid], g * (total * q - t));
            }
        }
    }
    if (rank == 0 && warp == 0) {
        double loss = 0.0;
        if (good && a.loss) {
            const double iT = 1.0 / (double)a.T, ls = log((double)S);
            for (int k = lane; k < n; k += 32) {
                const double t = sh.t[k];
                if (t > 0.0)
                    loss += t * (((double)sh.a[k] - (double)sh.list_max - sh.log_sum) -
                                 (((double)sh.z[k] - (double)M) * iT - ls));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1)
                loss += __shfl_xor_sync(kAllLanes, loss, o);
            const double r64 = nothing ? 0.0 : sh.r64;
            if (r64 > 0.0)
                loss += r64 * (log(r64) - (((double)mu - (double)M) * iT + log((double)su) - ls));
        }
        if (lane == 0) {
            if (a.loss)
                a.loss[row] = code ? nan : (float)loss;
            if (a.status)
                a.status[row] = code;
            if (code)
                atomicOr(a.err_word, 1u << code);
        }
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
    a.rows_per_seq = rows_per_seq;
    a.C = plan.cluster;
    a.n = n;
    a.tail = tail;
    a.vectors = (uint32_t)(plan.slice * es / 16);
    a.T = temperature;
    a.ch = (float)(1.4426950408889634074 / (double)temperature);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)plan.grid, 1, 1);
    cfg.blockDim = dim3(kNT, 1, 1);
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
    if (cudaLaunchKernelEx(&cfg, es == 2 ? sv_distill_kernel<2> : sv_distill_kernel<4>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return SV_ERR_CUDA;
    }
    return SV_OK;
}

}  // extern "C"
