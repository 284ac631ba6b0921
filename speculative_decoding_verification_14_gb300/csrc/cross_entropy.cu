// cross_entropy.cu -- softmax cross entropy of a vocabulary head z = h W^T over rows of hidden states,
// without keeping the logits, and its gradients.
//
//   loss = lse - z_y,  lse = ln sum_v exp z_v
//   d_v = g (exp(z_v - lse) - [v = y]), of the label g (exp(-loss) - 1) where the losses are given,  grad_h = sum_v d_v W_v,  grad_W_v = sum over rows of d_v h
//
// Rows that count are packed first (those below accept_len with a label), so that the products' work is
// theirs alone and nothing that a padded row holds reaches the head's gradient.
// Loss: one product whose tiles leave (maximum, sum) of each row's 256 logits without the label's, and a join of those
// with it: small losses keep their digits (1e-5 relative beside what the logits are off; 0.8 us of a loss of 5 rows).
// Gradients: piece by piece of the vocabulary, the logits once more, now written as bfloat16 d (how much a piece is:
// kPieceBytes); then d W into float32 sums of the hidden states' gradient, and
// d^T h, which is that piece's rows of the head's gradient.  d is rounded to bfloat16 (2^-8 of itself at most) since the
// tensor cores take it so: the rest of d as a second operand would be two more products beside four.  Its errors are
// independent from entry to entry, but a row's label may be most of its gradient (against 64 bits both are off by 2.2e-3
// to 2.6e-3 of their norm, 1.7e-3 of which is their own rounding).  A logit's sum is a float in tensor memory, which
// the tensor cores cut and do not round, the same way in every row: at D of 4096 loss and lse are off by 2.3e-6 of
// themselves, at 1024 by 6e-7, at 100 by 1e-7, logits by 4.1e-6, 9.8e-7, 1e-7 in the mean.  Products of one sign lose more,
// 1.4e-5 and 2.2e-6 (a sum that has grown takes less of each), and sums of few products nothing: no factor puts it
// back for all.  Sums begun anew every so many products would, for a tile's 256 x 256 more additions each time.
// The launches of a call begin while the ones before them end.
//
// What bounds it (replayed): with many rows the tensor cores.  8192 rows of 128256 x 4096, loss and both gradients,
// 20.3 to 21.5 ms: its products, 4 of 8.6 TFLOP, one of them the logits' second, take 95 % of the rate that a library
// product reaches in a burst, and what the clock leaves of that under the power limit; 2048 rows, the loss, 1.25 ms (0.90).
// 256 rows of 151936 x 2048, the hidden states' gradient, 368 us: three products, each over all of the weight, whose 622 MB
// no L2 holds from one to the next: 3 x 92 us at a copy's rate, where the products are 3 x 83.  Few rows read the weight at 5.2 TB/s once it flows: 5 rows of 32000 x 1024, the
// loss, 22.5 us (10 for 65 MB): 4 until the rows are packed, 4 until the first tile is there, 12 for the weight, 3 for
// the last tile's statistics.  40 rows, both gradients, 96 us: four such passes, over the weight or its gradient.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_verify.h"
#include "cross_entropy.h"
#include "distill_plan.h"
#include "losses_selftest.h"
#include "matrix_product.cuh"
#include "sv_context.h"
#include "two_floats.cuh"

namespace {

using namespace sv;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- rows that count

struct Rows {
    const __nv_bfloat16* hidden;
    int64_t stride;
    const int32_t* labels;
    const int32_t* accept_len;  // or NULL
    const float* lse;           // backward: rows whose lse is not finite have no gradient
    const float* loss_in;       // or NULL
    const float* grad_loss;     // or NULL
    int64_t R, V, D, depth;
    int rows_per_seq;
    const int32_t* counts;      // rows that count of each kCountRows; NULL for few rows
    // packed
    int32_t* index;
    int32_t* state;  // the number of rows that count, and whether a wait of this call has run out
    int32_t* label;
    float* packed_lse;
    float* packed_loss;
    float* scale;
    __nv_bfloat16* packed;
    // of rows that do not count
    float* loss;
    float* lse_out;
    int32_t* status;
    uint32_t* err_word;
    __nv_bfloat16* grad_hidden;
    int64_t grad_stride;
};

constexpr int kRowsPerBlock = 8;

// 0: counts; 1: does not; otherwise an error's code
__device__ __forceinline__ int row_kind(const Rows& a, int64_t row) {
    const int64_t seq = row / a.rows_per_seq;
    if (a.accept_len && row - seq * a.rows_per_seq >= a.accept_len[seq])
        return 1;
    const int32_t y = a.labels[row];
    if (y == -1)
        return 1;
    if (y < 0 || y >= a.V)
        return SV_ERR_TOKEN_RANGE;
    if (a.lse && !(fabsf(a.lse[row]) <= 3.4028235e38f))
        return SV_ERR_NONFINITE;
    if (a.loss_in && !(a.loss_in[row] == a.loss_in[row]))
        return SV_ERR_NONFINITE;
    return 0;
}

// Of many rows, those that count in each kCountRows.
__global__ void __launch_bounds__(256) sv_ce_count_kernel(const __grid_constant__ Rows a) {
    __shared__ int n;
    if (threadIdx.x == 0)
        n = 0;
    __syncthreads();
    int mine = 0;
    for (int64_t i = threadIdx.x, r = blockIdx.x * kCountRows + i; i < kCountRows && r < a.R; i += blockDim.x, r += blockDim.x)
        mine += row_kind(a, r) == 0;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0)
        atomicAdd(&n, mine);
    __syncthreads();
    if (threadIdx.x == 0)
        const_cast<int32_t*>(a.counts)[blockIdx.x] = n;
}

// Eight rows a block.  A block counts the rows before its own, which is R^2 / 16 looks at a row; of many rows, those of
// its own kCountRows, and adds up the numbers before.  The launch for the numbers costs 1.5 us of a loss call with 2048
// rows of 256 x 64 and lengths (15.5 -> 17.0) and gains at 4096 (19.0 -> 17.3), without lengths at 16384 (17.6 -> 18.7
// at 8192, 26.1 -> 23.8); 2^20 rows with lengths are 1.08 ms instead of 150.
// Blocks behind the last row clear the packed rows that fill up the
// last block of depth.
__global__ void __launch_bounds__(256) sv_ce_rows_kernel(const __grid_constant__ Rows a) {
    __shared__ int before;
    __shared__ int kinds[kRowsPerBlock];
    launch_next();
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.x * kRowsPerBlock, end = r0 < a.R ? r0 : a.R;
    if (tid == 0)
        before = 0;
    if (tid == 0 && blockIdx.x == 0)
        a.state[1] = 0;
    __syncthreads();
    int n = 0;
    int64_t from = 0;
    if (a.counts) {
        from = end / kCountRows * kCountRows;
        for (int64_t c = tid; c < end / kCountRows; c += blockDim.x)
            n += a.counts[c];
    }
    for (int64_t r = from + tid; r < end; r += blockDim.x)
        n += row_kind(a, r) == 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if ((tid & 31) == 0 && n)
        atomicAdd(&before, n);
    if (tid < kRowsPerBlock)
        kinds[tid] = r0 + tid < a.R ? row_kind(a, r0 + tid) : 1;
    __syncthreads();
    if (r0 >= a.R) {  // one row of filling per block
        const int64_t at = before + (int64_t)blockIdx.x - (a.R + kRowsPerBlock - 1) / kRowsPerBlock;
        if (at < (before + kBlockK - 1) / kBlockK * (int64_t)kBlockK)
            for (int64_t d = tid; d < a.depth; d += blockDim.x)
                a.packed[at * a.depth + d] = __float2bfloat16_rn(0.0f);
        return;
    }
    // a row a warp
    const int warp = tid >> 5, lane = tid & 31;
    const int64_t row = r0 + warp;
    if (row < a.R) {
        int64_t at = before;
        for (int i = 0; i < warp; ++i)
            at += kinds[i] == 0;
        const int kind = kinds[warp];
        if (kind == 0) {
            const __nv_bfloat16* src = a.hidden + row * a.stride;
            __nv_bfloat16* dst = a.packed + at * a.depth;
            int64_t done = 0;
            if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
                done = a.D / 8 * 8;
#pragma unroll 4
                for (int64_t d = lane; d < a.D / 8; d += 32)
                    reinterpret_cast<uint4*>(dst)[d] = reinterpret_cast<const uint4*>(src)[d];
            }
            for (int64_t d = done + lane; d < a.D; d += 32)
                dst[d] = src[d];
            if (lane == 0) {
                a.index[at] = (int32_t)row;
                a.label[at] = a.labels[row];
                if (a.packed_lse) {
                    if (a.status)
                        a.status[row] = SV_OK;
                    a.packed_lse[at] = a.lse[row];
                    if (a.loss_in)
                        a.packed_loss[at] = a.loss_in[row];
                    a.scale[at] = a.grad_loss ? a.grad_loss[row] : 1.0f;
                }
            }
        } else {
            const float x = kind == 1 ? 0.0f : __int_as_float(0x7fffffff);
            if (lane == 0) {
                if (a.loss)
                    a.loss[row] = x;
                if (a.lse_out)
                    a.lse_out[row] = x;
                if (a.status)
                    a.status[row] = kind == 1 ? SV_OK : kind;
                if (kind != 1)
                    atomicOr(a.err_word, 1u << kind);
            }
            if (a.grad_hidden)
                for (int64_t d = lane; d < a.D; d += 32)
                    a.grad_hidden[row * a.grad_stride + d] = __float2bfloat16_rn(x);
        }
        if (lane == 0 && row == a.R - 1)
            a.state[0] = (int32_t)(at + (kind == 0));
    }
}

// ---------------------------------------------------------------- tiles

struct Tiles {
    CUtensorMap a, b, c;  // c: what is written
    int32_t* state;  // the rows that count, and whether a wait of this call has run out
    const int32_t* label;
    const int32_t* index;
    int32_t* status;  // of the gradients' call, or NULL
    uint32_t* err_word;
    int64_t selftest;  // a tile's number, or -1
    int64_t V, D;
    int64_t first_tile, tiles;  // vocabulary tiles of this launch
    int64_t rows;               // of the workspace
    int a_rows;                 // the most that count, up to a tile's
    // loss
    float2* stats;
    float* label_logit;
    // gradients
    const float* lse;
    const float* loss;  // or NULL
    const float* scale;
    float* sums;
    int64_t depth;
    int splits, add;
    __nv_bfloat16* out;
    int64_t out_stride;
    int out_vectors;  // rows of out lie on 16 bytes: written through c, else entry by entry
};

// What a launch needs of the one before it is read behind wait_previous(), which run_tiles calls once its own
// barriers and tensor memory are set up.
// the row of a tile that this thread has in tensor memory
__device__ __forceinline__ int64_t tile_row(int64_t tile) {
    uint32_t rank;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    return tile * kTile + rank * kHalf + (threadIdx.x & 127);
}

// Behind a wait that ran out no row of the call has an answer.
__device__ __noinline__ void timed_out(int32_t* status, const int32_t* index, const int32_t* state) {
    if (status)
        for (int64_t r = threadIdx.x; r < *state; r += blockDim.x)
            status[index[r]] = SV_ERR_TIMEOUT;
}

// (maximum, sum of exponentials) of each row's logits in each tile of the vocabulary, the label's left out: a loss
// near 0 is the others' sum beside the label's weight, which is lost in a sum that begins with that weight
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsMm, 1)
    sv_ce_stats_kernel(const __grid_constant__ Tiles p) {
    int64_t n = 0;
    const auto shape = [&](int64_t count) {
        n = count;
        return MatrixShape{(n + kTile - 1) / kTile, p.tiles, (p.D + kBlockK - 1) / kBlockK, 1};
    };
    run_tiles<false, false>(&p.a, &p.b, p.a_rows, shape, 0, 0, p.err_word, 1u << SV_ERR_TIMEOUT, p.state, p.selftest,
                            [&](int64_t rt, int64_t ct, int, auto load) {
        const int64_t row = tile_row(rt), c0 = ct * kTile;
        const bool there = row < n;
        const int64_t y = there ? p.label[row] - c0 : -1;
        float m = -__int_as_float(0x7f800000), s = 0.0f, zy = 0.0f;
        for (int c = 0; c < kTile; c += 32) {
            float v[32];
            load(c, v);
            const int left = (int)(p.V - c0 - c < 32 ? p.V - c0 - c : 32);  // columns of the vocabulary
            if (left <= 0)
                break;
            if (y >= c && y < c + 32) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (y == c + e) {
                        zy = v[e];
                        v[e] = -__int_as_float(0x7f800000);
                    }
            }
            float top = m;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (e >= left)
                    v[e] = -__int_as_float(0x7f800000);
                // a NaN has to reach the sum
                asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(v[e]));
            }
            const float base = top > -__int_as_float(0x7f800000) ? top : 0.0f;
            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < 32; ++e)
                part[e & 3] += ex2((v[e] - base) * kLog2e);
            s = s * ex2((m - base) * kLog2e) + ((part[0] + part[1]) + (part[2] + part[3]));
            m = top;
            if (!(top == top))
                s = top;
        }
        if (there) {
            p.stats[ct * p.rows + row] = make_float2(m, s);
            if (y >= 0 && y < kTile)
                p.label_logit[row] = zy;
        }
    });
}

// d of a piece of the vocabulary, bfloat16; zeros in rows and columns that only fill up tiles.  The label's is p - 1: of
// an lse, whose last place is 1e-6 to 4e-6 of p, or, without that cancellation, exp(-loss) - 1.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsMm, 1)
    sv_ce_probs_kernel(const __grid_constant__ Tiles p) {
    TileStore store;
    int64_t n = 0;
    const auto shape = [&](int64_t count) {
        n = count;
        return MatrixShape{(n + kTile - 1) / kTile, p.tiles, (p.D + kBlockK - 1) / kBlockK, 1};
    };
    const bool gave_up = run_tiles<false, false>(&p.a, &p.b, p.a_rows, shape, p.first_tile * kTile, 0, p.err_word, 1u << SV_ERR_TIMEOUT, p.state, p.selftest,
                            [&](int64_t rt, int64_t ct, int, auto load) {
        const int64_t row = tile_row(rt), c0 = (p.first_tile + ct) * kTile;
        const bool there = row < n;
        const int64_t y = there ? p.label[row] - c0 : -1;
        const float lse = there ? p.lse[row] : 0.0f, g = there ? p.scale[row] : 0.0f;
        const bool given = p.loss != nullptr;
        const float dy = given && y >= 0 && y < kTile ? expm1f(-p.loss[row]) : 0.0f;
        // rows behind those that fill up the last block of depth are read by nobody
        const int64_t warp_row = row - (threadIdx.x & 31);
        if (warp_row >= (n + kBlockK - 1) / kBlockK * kBlockK)
            return;
        for (int c = 0; c < kTile; c += 64) {
            float v[64];
            load(c, *reinterpret_cast<float(*)[32]>(v));
            load(c + 32, *reinterpret_cast<float(*)[32]>(v + 32));
            const int left = there ? (int)(p.V - c0 - c < 64 ? p.V - c0 - c : 64) : 0;
#pragma unroll
            for (int e = 0; e < 64; ++e)
                v[e] = ex2((v[e] - lse) * kLog2e);
            if (y >= c && y < c + 64) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (y == c + e)
                        v[e] = given ? dy : v[e] - 1.0f;
            }
#pragma unroll
            for (int e = 0; e < 64; ++e)
                v[e] = e < left ? v[e] * g : 0.0f;
            store.put(&p.c, (int)(ct * kTile + c), (int)warp_row, v);
        }
    });
    if (threadIdx.x >= 128)
        store.finish();
    if (__builtin_expect(gave_up, 0))
        timed_out(p.status, p.index, p.state);
}

// a piece's part of the hidden states' gradient: float32 sums, those of a split apart
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsMm, 1)
    sv_ce_hidden_kernel(const __grid_constant__ Tiles p) {
    int64_t n = 0;
    const auto shape = [&](int64_t count) {
        n = count;
        return MatrixShape{(n + kTile - 1) / kTile, (p.D + kTile - 1) / kTile, p.tiles * (kTile / kBlockK), p.splits};
    };
    const bool gave_up = run_tiles<false, true>(&p.a, &p.b, p.a_rows, shape, 0, p.first_tile * kTile, p.err_word, 1u << SV_ERR_TIMEOUT, p.state, p.selftest,
                           [&](int64_t rt, int64_t ct, int split, auto load) {
        const int64_t row = tile_row(rt), c0 = ct * kTile;
        float* out = p.sums + ((int64_t)split * p.rows + row) * p.depth + c0;
        for (int c = 0; c < kTile && c0 + c < p.D; c += 32) {
            float v[32];
            load(c, v);
            if (row >= n)
                continue;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (c0 + c + 4 * q < p.depth) {
                    float4* to = reinterpret_cast<float4*>(out + c) + q;
                    float4 x = p.add ? *to : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    x.x += v[4 * q], x.y += v[4 * q + 1], x.z += v[4 * q + 2], x.w += v[4 * q + 3];
                    *to = x;
                }
        }
    });
    if (__builtin_expect(gave_up, 0))
        timed_out(p.status, p.index, p.state);
}

// a piece's rows of the head's gradient
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsMm, 1)
    sv_ce_weight_kernel(const __grid_constant__ Tiles p) {
    TileStore store;
    int64_t n = 0;
    const auto shape = [&](int64_t count) {
        n = count;
        return MatrixShape{p.tiles, (p.D + kTile - 1) / kTile, (n + kBlockK - 1) / kBlockK, 1};
    };
    const bool gave_up = run_tiles<true, true>(&p.a, &p.b, p.a_rows, shape, 0, 0, p.err_word, 1u << SV_ERR_TIMEOUT, p.state, p.selftest,
                          [&](int64_t rt, int64_t ct, int, auto load) {
        const int64_t v_id = p.first_tile * kTile + tile_row(rt), c0 = ct * kTile;
        if (p.out_vectors) {
            for (int c = 0; c < kTile && c0 + c < p.D; c += 64) {
                float v[64];
                load(c, *reinterpret_cast<float(*)[32]>(v));
                load(c + 32, *reinterpret_cast<float(*)[32]>(v + 32));
                if (v_id - (threadIdx.x & 31) < p.V)  // what lies beyond the head is left out by the copy
                    store.put(&p.c, (int)(c0 + c), (int)(v_id - (threadIdx.x & 31)), v);
            }
            return;
        }
        __nv_bfloat16* out = p.out + v_id * p.out_stride + c0;
        for (int c = 0; c < kTile && c0 + c < p.D; c += 32) {
            float v[32];
            load(c, v);
            if (v_id < p.V)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (c0 + c + e < p.D)
                        out[c + e] = __float2bfloat16_rn(v[e]);
        }
    });
    if (threadIdx.x >= 128)
        store.finish();
    if (__builtin_expect(gave_up, 0))
        timed_out(p.status, p.index, p.state);
}

// ---------------------------------------------------------------- joins

struct Join {
    const int2* state;  // the rows that count, and whether a wait of this call has run out
    const int32_t* index;
    int64_t rows, tiles, D, depth;
    const float2* stats;
    const float* label_logit;
    float* loss;
    float* lse;
    int32_t* status;
    uint32_t* err_word;
    const float* sums;
    int splits;
    __nv_bfloat16* grad_hidden;
    int64_t grad_stride;
};

// Eight rows a block, their tiles over 32 threads each: first the largest maximum m, then the sum s of the others'
// weights against it, in two floats, and with the label's logit z:
//   z >= m: loss = ln(1 + s exp(m - z)),          lse = z + loss
//   z < m:  loss = (m - z) + ln(s + exp(z - m)),  lse = m + ln(s + exp(z - m))
// Nothing cancels, so a loss is as good relative to itself as the logits' differences are.
__global__ void __launch_bounds__(256) sv_ce_join_kernel(const __grid_constant__ Join a) {
    __shared__ float part[8][8], rest[8][8];  // of a warp's four shares
    launch_next();
    wait_previous();
    const int at = threadIdx.x & 7, share = threadIdx.x >> 3;
    const int64_t row = (int64_t)blockIdx.x * 8 + at;
    const int2 state = *a.state;
    const int64_t n = state.x;
    if ((int64_t)blockIdx.x * 8 >= n)
        return;
    const float inf = __int_as_float(0x7f800000);
    const float2* stats = a.stats + row;
    const float z = row < n ? a.label_logit[row] : 0.0f;
    const int64_t to = row < n ? a.index[row] : 0;
    float m = -inf;
    Two s{0.0f, 0.0f};
    if (row < n) {
#pragma unroll 4
        for (int64_t t = share; t < a.tiles; t += 32)
            asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(stats[t * a.rows].x));
    }
#pragma unroll
    for (int o = 8; o < 32; o *= 2)
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(__shfl_xor_sync(0xffffffffu, m, o)));
    part[share >> 2][at] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(part[i][at]));
    if (row < n && m > -inf && m < inf) {
#pragma unroll 4
        for (int64_t t = share; t < a.tiles; t += 32) {
            const float2 x = stats[t * a.rows];
            const Two y = two_sum(s.h, x.y * expf(x.x - m));
            s = Two{y.h, s.l + y.l};
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o *= 2)
        s = two_add(s, Two{__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.l, o)});
    __syncthreads();
    part[share >> 2][at] = s.h;
    rest[share >> 2][at] = s.l;
    __syncthreads();
    if (share || row >= n)
        return;
    s = Two{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s = two_add(s, Two{part[i][at], rest[i][at]});
    const float nan = __int_as_float(0x7fffffff);
    float most = m;
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(z));
    const bool lost = state.y != 0, good = !lost && most > -inf && most < inf;
    const float ls = z >= m ? log1pf(s.h * expf(m - z)) : logf(s.h + (s.l + expf(z - m)));
    a.loss[to] = good ? (z >= m ? ls : (m - z) + ls) : nan;
    a.lse[to] = good ? most + ls : nan;
    if (a.status)
        a.status[to] = good ? SV_OK : lost ? SV_ERR_TIMEOUT : SV_ERR_NONFINITE;
    if (!good && !lost)
        atomicOr(a.err_word, 1u << SV_ERR_NONFINITE);
}

// Four columns a thread: the splits' sums, rounded once.
__global__ void __launch_bounds__(256) sv_ce_hidden_join_kernel(const __grid_constant__ Join a) {
    launch_next();
    wait_previous();
    const int64_t row = blockIdx.x, d = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
    const int2 state = *a.state;
    if (row >= state.x || d >= a.D)
        return;
    const float4* from = reinterpret_cast<const float4*>(a.sums + row * a.depth + d);
    const int64_t apart = a.rows * a.depth / 4;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) {
        const float4 y = from[s * apart];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    if (state.y)
        x.x = x.y = x.z = x.w = __int_as_float(0x7fffffff);
    __nv_bfloat16* out = a.grad_hidden + (int64_t)a.index[row] * a.grad_stride + d;
    if (d + 4 <= a.D && (reinterpret_cast<uintptr_t>(out) & 7u) == 0) {
        uint2 w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x.y), "f"(x.x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x.w), "f"(x.z));
        *reinterpret_cast<uint2*>(out) = w;
    } else {
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < a.D)
                out[e] = __float2bfloat16_rn(v[e]);
    }
}

// ---------------------------------------------------------------- host

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeFn>(f);
}

// A bfloat16 matrix [rows, columns] as boxes of 64 columns and `box` rows; what lies beyond is zeros.
bool tensor_map(CUtensorMap* map, const void* base, int64_t rows, int64_t columns, int64_t stride, int box) {
    const EncodeFn encode = encoder();
    if (!encode)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)columns, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {64, (cuuint32_t)box}, steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*TilesFn)(const Tiles);

// Attributes of the kernels on a device, and how many pairs run at once.
int matrix_pairs(int device) {
    static std::atomic<int> pairs[64];
    if (device < 0 || device >= 64)
        return 0;
    int n = pairs[device].load(std::memory_order_acquire);
    if (n)
        return n;
    int least = 1 << 30;
    for (TilesFn fn : {sv_ce_stats_kernel, sv_ce_probs_kernel, sv_ce_hidden_kernel, sv_ce_weight_kernel}) {
        if (cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMm) != cudaSuccess) {
            (void)cudaGetLastError();
            return 0;
        }
        cudaLaunchConfig_t cfg;
        std::memset(&cfg, 0, sizeof cfg);
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(kThreadsMm, 1, 1);
        cfg.dynamicSmemBytes = kSmemMm;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, (const void*)fn, &cfg) != cudaSuccess || clusters < 1) {
            (void)cudaGetLastError();
            return 0;
        }
        least = clusters < least ? clusters : least;
    }
    pairs[device].store(least, std::memory_order_release);
    return least;
}

// A launch that may begin while the one before it, of the same call, ends: it waits for that one's results itself.
template <typename Args>
bool launch_after(void (*fn)(const Args), const Args& args, dim3 grid, int threads, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, args) == cudaSuccess)
        return true;
    (void)cudaGetLastError();
    return false;
}

bool launch_tiles(TilesFn fn, const Tiles& p, int64_t most, int pairs, cudaStream_t stream) {
    const int64_t n = most < pairs ? most : pairs;
    return launch_after(fn, p, dim3((unsigned)(2 * (n < 1 ? 1 : n)), 1, 1), kThreadsMm, kSmemMm, stream);
}

int check(const sv_ctx* ctx, const void* hidden, int dtype, int64_t hidden_stride, const void* weight,
          int64_t weight_stride, const int32_t* labels, const int32_t* accept_len, int B, int rows_per_seq, int64_t V,
          int64_t D, const void* workspace, size_t workspace_bytes, bool grad, CrossEntropyPlan* plan) {
    if (!ctx || !hidden || !weight || !labels || !workspace || (dtype != SV_F32 && dtype != SV_BF16))
        return SV_ERR_INVALID_ARG;
    const int64_t most = (int64_t)1 << 40;
    if (B < 1 || B > ctx->max_B || rows_per_seq < 1 || rows_per_seq > ctx->max_K + 1 || V < 1 || V > ctx->max_V ||
        V > ((int64_t)1 << 31) - 1 || D < 1 || D > ((int64_t)1 << 20) || (int64_t)B * rows_per_seq > kMaxRowsCe ||
        hidden_stride < D || hidden_stride > most || weight_stride < D || weight_stride > ((int64_t)1 << 32) ||
        (double)B * rows_per_seq * (double)hidden_stride >= 1099511627776.0 ||  // 2^40
        (double)V * (double)weight_stride >= 1099511627776.0)
        return SV_ERR_INVALID_ARG;
    if (dtype != SV_BF16)
        return SV_ERR_UNSUPPORTED;
    // the copy engine takes the weight's rows on 16 bytes
    if (!aligned(hidden, 2) || !aligned(weight, 16) || (V > 1 && weight_stride % 8) || !aligned(labels, 4) ||
        !aligned(accept_len, 4) || !aligned(workspace, 256))
        return SV_ERR_INVALID_ARG;
    *plan = cross_entropy_plan(ctx->num_sms, (int64_t)B * rows_per_seq, V, D, grad);
    return workspace_bytes < plan->total ? SV_ERR_INVALID_ARG : SV_OK;
}

// The stride the copy engine is given: a single row's is its length on 16 bytes, whatever the call's is.
int64_t rows_apart(int64_t V, int64_t D, int64_t weight_stride) { return V > 1 ? weight_stride : round_up(D, 8); }

Rows pack_args(const CrossEntropyPlan& plan, unsigned char* ws, const void* hidden, int64_t stride,
               const int32_t* labels, const int32_t* accept_len, int B, int rows_per_seq, int64_t V, int64_t D,
               uint32_t* err_word) {
    Rows r;
    std::memset(&r, 0, sizeof r);
    r.hidden = static_cast<const __nv_bfloat16*>(hidden);
    r.stride = stride;
    r.labels = labels;
    r.accept_len = accept_len;
    r.R = (int64_t)B * rows_per_seq;
    r.V = V;
    r.D = D;
    r.depth = plan.depth;
    r.rows_per_seq = rows_per_seq;
    r.index = reinterpret_cast<int32_t*>(ws + plan.index);
    r.state = r.index + plan.rows;
    r.label = reinterpret_cast<int32_t*>(ws + plan.label);
    r.packed = reinterpret_cast<__nv_bfloat16*>(ws + plan.hidden);
    r.err_word = err_word;
    if (r.R > (accept_len ? kCountFromLengths : kCountFrom))
        r.counts = reinterpret_cast<const int32_t*>(ws + plan.counts);
    return r;
}

// The first of a call's launches, which begin when what came before them on the stream has ended; `fill`: the blocks
// that clear packed rows.
bool launch_rows(const Rows& r, int fill, cudaStream_t stream) {
    if (r.counts)
        sv_ce_count_kernel<<<(unsigned)((r.R + kCountRows - 1) / kCountRows), 256, 0, stream>>>(r);
    sv_ce_rows_kernel<<<(unsigned)((r.R + kRowsPerBlock - 1) / kRowsPerBlock + fill), 256, 0, stream>>>(r);
    return cudaGetLastError() == cudaSuccess;
}

}  // namespace

extern "C" {

int spec_cross_entropy_workspace(sv_ctx* ctx, int B, int rows_per_seq, int64_t V, int64_t D, int grad, size_t* bytes) {
    if (!ctx)
        return SV_ERR_INVALID_ARG;
    return spec_cross_entropy_workspace_for(ctx->num_sms, B, rows_per_seq, V, D, grad, bytes);
}

int spec_cross_entropy_run(sv_ctx* ctx, const void* hidden, int dtype, int64_t hidden_stride, const void* weight,
                           int64_t weight_stride, const int32_t* labels, const int32_t* accept_len, int B,
                           int rows_per_seq, int64_t V, int64_t D, float* loss, float* lse, int32_t* status,
                           void* workspace, size_t workspace_bytes, void* stream) {
    CrossEntropyPlan plan;
    const int rc = check(ctx, hidden, dtype, hidden_stride, weight, weight_stride, labels, accept_len, B, rows_per_seq,
                         V, D, workspace, workspace_bytes, false, &plan);
    if (rc != SV_OK)
        return rc;
    if (!loss || !lse || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(status, 4))
        return SV_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->device);
    const int pairs = matrix_pairs(ctx->device);
    if (!pairs)
        return SV_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    Rows r = pack_args(plan, ws, hidden, hidden_stride, labels, accept_len, B, rows_per_seq, V, D, ctx->d_err);
    r.loss = loss;
    r.lse_out = lse;
    r.status = status;
    Tiles p;
    std::memset(&p, 0, sizeof p);
    if (!tensor_map(&p.a, r.packed, plan.rows, D, plan.depth, box_rows(r.R)) ||
        !tensor_map(&p.b, weight, V, D, rows_apart(V, D, weight_stride), kHalf))
        return SV_ERR_CUDA;
    p.state = r.state;
    p.selftest = losses_selftest(ctx) == SV_SELFTEST_LOGITS ? 0 : -1;
    p.label = r.label;
    p.err_word = ctx->d_err;
    p.V = V;
    p.D = D;
    p.tiles = plan.vocab_tiles;
    p.rows = plan.rows;
    p.a_rows = (int)(r.R < kTile ? r.R : kTile);
    p.stats = reinterpret_cast<float2*>(ws + plan.stats);
    p.label_logit = reinterpret_cast<float*>(ws + plan.label_logit);
    Join j;
    std::memset(&j, 0, sizeof j);
    j.state = reinterpret_cast<const int2*>(r.state);
    j.index = r.index;
    j.rows = plan.rows;
    j.tiles = plan.vocab_tiles;
    j.stats = p.stats;
    j.label_logit = p.label_logit;
    j.loss = loss;
    j.lse = lse;
    j.status = status;
    j.err_word = ctx->d_err;
    if (!launch_rows(r, 0, st) ||
        !launch_tiles(sv_ce_stats_kernel, p, plan.rows / kTile * plan.vocab_tiles, pairs, st))
        return SV_ERR_CUDA;
    return launch_after(sv_ce_join_kernel, j, dim3((unsigned)((r.R + 7) / 8), 1, 1), 256, 0, st) ? SV_OK : SV_ERR_CUDA;
}

int spec_cross_entropy_grad_of_loss(sv_ctx* ctx, const void* hidden, int dtype, int64_t hidden_stride,
                                    const void* weight, int64_t weight_stride, const int32_t* labels,
                                    const int32_t* accept_len, const float* lse, const float* loss,
                                    const float* grad_loss, int B, int rows_per_seq, int64_t V, int64_t D,
                                    void* grad_hidden, int64_t grad_hidden_stride, void* grad_weight,
                                    int64_t grad_weight_stride, int32_t* status, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    CrossEntropyPlan plan;
    const int rc = check(ctx, hidden, dtype, hidden_stride, weight, weight_stride, labels, accept_len, B, rows_per_seq,
                         V, D, workspace, workspace_bytes, true, &plan);
    if (rc != SV_OK)
        return rc;
    const int64_t R = (int64_t)B * rows_per_seq, most = (int64_t)1 << 40;
    if (!lse || (!grad_hidden && !grad_weight) || !aligned(lse, 4) || !aligned(loss, 4) || !aligned(grad_loss, 4) ||
        !aligned(grad_hidden, 2) || !aligned(grad_weight, 2) || !aligned(status, 4) ||
        (grad_hidden && (grad_hidden_stride < D || grad_hidden_stride > most ||
                         (double)R * (double)grad_hidden_stride >= 1099511627776.0)) ||
        (grad_weight && (grad_weight_stride < D || grad_weight_stride > most ||
                         (double)V * (double)grad_weight_stride >= 1099511627776.0)) ||
        (grad_hidden && rows_meet(hidden, hidden_stride * 2, grad_hidden, grad_hidden_stride * 2, R, D * 2)) ||
        (grad_weight && rows_meet(weight, weight_stride * 2, grad_weight, grad_weight_stride * 2, V, D * 2)))
        return SV_ERR_INVALID_ARG;
    DeviceGuard guard(ctx->device);
    const int pairs = matrix_pairs(ctx->device);
    if (!pairs)
        return SV_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    Rows r = pack_args(plan, ws, hidden, hidden_stride, labels, accept_len, B, rows_per_seq, V, D, ctx->d_err);
    r.lse = lse;
    r.loss_in = loss;
    r.grad_loss = grad_loss;
    r.packed_lse = reinterpret_cast<float*>(ws + plan.lse);
    r.packed_loss = reinterpret_cast<float*>(ws + plan.loss);
    r.scale = reinterpret_cast<float*>(ws + plan.scale);
    r.status = status;
    r.grad_hidden = static_cast<__nv_bfloat16*>(grad_hidden);
    r.grad_stride = grad_hidden_stride;
    __nv_bfloat16* probs = reinterpret_cast<__nv_bfloat16*>(ws + plan.probs);
    const int64_t width = plan.piece_tiles * kTile;
    Tiles logits, hid, wgt;
    std::memset(&logits, 0, sizeof logits);
    logits.state = r.state;
    logits.label = r.label;
    logits.index = r.index;
    logits.status = status;
    logits.err_word = ctx->d_err;
    logits.V = V;
    logits.D = D;
    logits.rows = plan.rows;
    logits.a_rows = (int)(R < kTile ? R : kTile);
    logits.lse = r.packed_lse;
    logits.loss = loss ? r.packed_loss : nullptr;
    logits.scale = r.scale;
    logits.sums = reinterpret_cast<float*>(ws + plan.sums);
    logits.depth = plan.depth;
    logits.splits = plan.splits;
    logits.out = static_cast<__nv_bfloat16*>(grad_weight);
    logits.out_stride = grad_weight_stride;
    // the copy engine writes whole 16 bytes: beyond D too, where that ends inside some; and its strides end at 2^40 bytes
    logits.out_vectors = aligned(grad_weight, 16) && grad_weight_stride % 8 == 0 && D % 8 == 0 &&
                         grad_weight_stride < ((int64_t)1 << 39);
    hid = wgt = logits;
    const int selftest = losses_selftest(ctx);
    logits.selftest = selftest == SV_SELFTEST_PROBS ? 0 : -1;
    hid.selftest = selftest == SV_SELFTEST_HIDDEN ? 0 : -1;
    wgt.selftest = selftest == SV_SELFTEST_WEIGHT ? 0 : -1;
    if (!tensor_map(&logits.a, r.packed, plan.rows, D, plan.depth, box_rows(R)) ||
        !tensor_map(&logits.b, weight, V, D, rows_apart(V, D, weight_stride), kHalf) ||
        !tensor_map(&hid.a, probs, plan.rows, width, width, box_rows(R)) ||
        !tensor_map(&hid.b, weight, V, D, rows_apart(V, D, weight_stride), kBlockK) ||
        !tensor_map(&wgt.a, probs, plan.rows, width, width, kBlockK) ||
        !tensor_map(&wgt.b, r.packed, plan.rows, D, plan.depth, kBlockK) ||
        !tensor_map(&logits.c, probs, plan.rows, width, width, 32) ||
        (grad_weight && logits.out_vectors && !tensor_map(&wgt.c, grad_weight, V, D, grad_weight_stride, 32)))
        return SV_ERR_CUDA;
    if (!launch_rows(r, kBlockK, st))
        return SV_ERR_CUDA;
    const int64_t row_tiles = plan.rows / kTile, depth_tiles = (D + kTile - 1) / kTile;
    for (int64_t piece = 0; piece < plan.pieces; ++piece) {
        const int64_t first = piece * plan.piece_tiles;
        const int64_t tiles = plan.vocab_tiles - first < plan.piece_tiles ? plan.vocab_tiles - first : plan.piece_tiles;
        for (Tiles* t : {&logits, &hid, &wgt}) {
            t->first_tile = first;
            t->tiles = tiles;
            t->add = piece > 0;
        }
        if (!launch_tiles(sv_ce_probs_kernel, logits, row_tiles * tiles, pairs, st) ||
            (grad_hidden && !launch_tiles(sv_ce_hidden_kernel, hid, row_tiles * depth_tiles * plan.splits, pairs, st)) ||
            (grad_weight && !launch_tiles(sv_ce_weight_kernel, wgt, tiles * depth_tiles, pairs, st)))
            return SV_ERR_CUDA;
    }
    if (grad_hidden) {
        Join j;
        std::memset(&j, 0, sizeof j);
        j.state = reinterpret_cast<const int2*>(r.state);
        j.index = r.index;
        j.rows = plan.rows;
        j.D = D;
        j.depth = plan.depth;
        j.sums = logits.sums;
        j.splits = plan.splits;
        j.grad_hidden = r.grad_hidden;
        j.grad_stride = grad_hidden_stride;
        if (!launch_after(sv_ce_hidden_join_kernel, j, dim3((unsigned)R, (unsigned)((D + 1023) / 1024), 1), 256, 0, st))
            return SV_ERR_CUDA;
    }
    return SV_OK;
}

int spec_cross_entropy_grad(sv_ctx* ctx, const void* hidden, int dtype, int64_t hidden_stride, const void* weight,
                            int64_t weight_stride, const int32_t* labels, const int32_t* accept_len, const float* lse,
                            const float* grad_loss, int B, int rows_per_seq, int64_t V, int64_t D, void* grad_hidden,
                            int64_t grad_hidden_stride, void* grad_weight, int64_t grad_weight_stride, int32_t* status,
                            void* workspace, size_t workspace_bytes, void* stream) {
    return spec_cross_entropy_grad_of_loss(ctx, hidden, dtype, hidden_stride, weight, weight_stride, labels, accept_len,
                                           lse, nullptr, grad_loss, B, rows_per_seq, V, D, grad_hidden,
                                           grad_hidden_stride, grad_weight, grad_weight_stride, status, workspace,
                                           workspace_bytes, stream);
}

}  // extern "C"
