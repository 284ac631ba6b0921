// matrix_product.cuh -- tiles of a bfloat16 matrix product on the tensor cores, for kernels that do
// something with each tile instead of writing it.
//
// A pair of CTAs (a cluster of two) computes a tile of 256 x 256: each holds 128 rows of A and 128 rows
// of B per stage, in 64 elements of depth, and the products of all of them go to the tensor memory of
// the CTA that holds the rows of A (tcgen05.mma, cta_group::2).  Pairs are persistent and take tiles in
// turn.  One thread of each CTA issues the copies (cp.async.bulk.tensor, 128-byte swizzle) that fill its
// ring of stages, one thread of the first CTA the products, and four warps of each CTA take the finished
// tile out of tensor memory, where two tiles have room: the next one's products run meanwhile.
// A CTA's operands of a stage come to 32 KB for 128 x 256 x 64 products, 64 bytes a cycle at the tensor cores' full rate;
// one CTA by itself with 128 x 256 would need 96.  Six stages are in flight.
// An operand lies in memory with its depth contiguous, or with its rows contiguous ("turned": the
// probabilities as [v, r] and the weight as [d, v] are read from [r, v] and [v, d] as they lie).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cross_entropy.h"
#include "losses_common.cuh"

namespace sv {

constexpr int kStagesMm = 6;
constexpr int kOperandBytes = kHalf * kBlockK * 2;  // one operand of one stage: 16 KB
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kThreadsMm = 256;  // warps: copies, products, tensor memory, none, four for tiles
constexpr int kTmemColumns = 512;
constexpr int kStoreBytes = 32 * 128;  // 32 rows of 64 bfloat16 columns on their way out
constexpr int kSmemMm = kStagesMm * kStageBytes + 8 * kStoreBytes + 1024;  // two for each tile warp; and the
                                                                           // distance to a multiple of 1024

struct MatrixBarriers {
    uint64_t full[kStagesMm], empty[kStagesMm], tile_full[2], tile_empty[2], done;
    long long fills[2];  // stages that either CTA has issued its copies for
    uint32_t tmem, failed;
};

// A wait for copies has their own limit, one for what follows from copies, or from products of them, that and kWaitNs.
constexpr unsigned long long kProductWaitNs = kCopyWaitNs + kWaitNs;

// Whoever gives up says so to all warps of the pair, which then give up at their next wait that is not over.
__device__ __forceinline__ void give_up(volatile uint32_t* failed) {
    uint32_t rank;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    *failed = 1;
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(const_cast<uint32_t*>(failed), rank ^ 1u)), "r"(1u)
                 : "memory");
}
// Waits for a phase, at most `limit` ns.
static __device__ __noinline__ bool matrix_wait_slow(uint64_t* bar, uint32_t parity, unsigned long long limit,
                                                     volatile uint32_t* failed) {
    const unsigned long long t0 = global_ns();
    while (!*failed) {
        for (int i = 0; i < 64; ++i)
            if (barrier_try_cluster(bar, parity))
                return true;
        if (global_ns() - t0 > limit)
            give_up(failed);
    }
    return false;
}
__device__ __forceinline__ bool matrix_wait(uint64_t* bar, uint32_t parity, unsigned long long limit,
                                            volatile uint32_t* failed) {
    return barrier_try_cluster(bar, parity) || matrix_wait_slow(bar, parity, limit, failed);
}

// After a pair has given up, and all its warps know and wait for one another: the copies issued have landed and the
// products issued are done before either CTA leaves, as far as kCopyWaitNs and kWaitNs see.  One CTA may have issued
// copies of a stage whose other half the other one then left out, up to a ring's worth: the first CTA, on whose
// barriers both halves arrive, takes the half that never comes off what the barrier expects.
static __device__ __noinline__ void matrix_drain(MatrixBarriers& bars, uint32_t second_bytes, int32_t* state,
                                                 uint32_t* err_word, uint32_t timeout_bit) {
    uint32_t rank;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    if (rank == 1 && threadIdx.x == 0)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(&bars.fills[1], 0)), "l"(bars.fills[1]) : "memory");
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0 && rank == 0) {
        const long long own = bars.fills[0], other = bars.fills[1], most = own > other ? own : other;
        for (long long j = own; j < other; ++j)
            barrier_expect(&bars.full[j % kStagesMm], second_bytes);
        for (long long j = other; j < own; ++j)
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(
                             shared_addr(&bars.full[j % kStagesMm])),
                         "r"(second_bytes)
                         : "memory");
        for (long long j = most > kStagesMm ? most - kStagesMm : 0; j < most; ++j)
            barrier_wait(&bars.full[j % kStagesMm], (uint32_t)(j / kStagesMm) & 1u, kCopyWaitNs);
    }
    if (threadIdx.x == 32) {  // of the first CTA: the thread that issued the products
        if (rank == 0)
            asm volatile(
                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                    shared_addr(&bars.done)),
                "h"((uint16_t)3)
                : "memory");
        barrier_wait(&bars.done, 0, kWaitNs);
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0) {
        *(volatile int32_t*)(state + 1) = 1;
        atomicOr(err_word, timeout_bit);
    }
}

__device__ __forceinline__ void copy_tile(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

// Shared-memory descriptor of an operand: 128-byte swizzle.  Depth contiguous: rows of 128 bytes, groups of
// eight rows 1024 apart.  Turned: 64 rows of the operand side by side in 128 bytes, groups of eight
// depths 1024 apart, the next 64 rows 8192 on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool turned) {
    uint64_t d = (uint64_t)((addr & 0x3ffffu) >> 4);
    d |= (uint64_t)((turned ? 8192u : 16u) >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// bf16 x bf16 -> f32, 256 x 256
__host__ __device__ constexpr uint32_t product_desc(bool turned_a, bool turned_b) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((turned_a ? 1u : 0u) << 15) | ((turned_b ? 1u : 0u) << 16) |
           ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}
__device__ __forceinline__ void product(uint32_t tmem, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
}
// the products issued so far arrive on this barrier of both CTAs when they are done
__device__ __forceinline__ void products_arrive(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            shared_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// 32 columns of this warp's 32 rows
__device__ __forceinline__ void load_columns(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}

// 64 columns of a tile warp's 32 rows, rounded to bfloat16, out through shared memory: a thread has a row, whose
// 16-byte parts go to places swizzled as the copy engine takes them (no two lanes of eight in a bank), and one lane
// hands the box to it.  Lane 0 of each warp waits for its own copies alone; two boxes take turns.
struct TileStore {
    uint32_t at;  // this warp's two boxes
    int turn = 0;
    __device__ __forceinline__ TileStore() {
        extern __shared__ unsigned char dynamic[];
        at = ((shared_addr(dynamic) + 1023u) & ~1023u) + kStagesMm * kStageBytes +
             ((threadIdx.x >> 5) & 3) * 2 * kStoreBytes;
    }
    __device__ __forceinline__ void put(const CUtensorMap* map, int x, int y, const float (&v)[64]) {
        const int lane = threadIdx.x & 31;
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
        const uint32_t box = at + turn * kStoreBytes, row = box + lane * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[e]) : "f"(v[8 * q + 2 * e + 1]), "f"(v[8 * q + 2 * e]));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((q ^ (lane & 7)) << 4)), "r"(w[0]),
                         "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                         "r"(box), "r"(x), "r"(y)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        turn ^= 1;
    }
    // all of it is in memory
    __device__ __forceinline__ void finish() {
        if ((threadIdx.x & 31) == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
};

// What a pair computes: `rows` x `columns` tiles, each over blocks k0 .. k1 - 1 of its split of the depth.
struct MatrixShape {
    int64_t row_tiles, column_tiles, blocks;
    int splits;
    __device__ __forceinline__ int64_t tiles() const { return row_tiles * column_tiles * splits; }
    // Pairs that run at the same time share operands in L2: eight row tiles at a time, columns within them.
    __device__ __forceinline__ void tile(int64_t i, int64_t& row, int64_t& column, int& split) const {
        const int64_t one = row_tiles * column_tiles;
        split = (int)(i / one);
        i -= split * one;
        const int64_t group = i / (8 * column_tiles), first = group * 8, in = i - first * column_tiles;
        const int64_t height = row_tiles - first < 8 ? row_tiles - first : 8;
        row = first + in % height;
        column = in / height;
    }
    __device__ __forceinline__ void depth(int split, int64_t& k0, int64_t& k1) const {
        k0 = blocks * split / splits;
        k1 = blocks * (split + 1) / splits;
    }
};

// Runs the pair's tiles, of a shape that is asked for once the launch before has ended.  a_rows: the
// most rows that A can have (its box has 128 of them, or as many as there are, rounded up to eight): where they fit one
// CTA, what the other would copy is left out, and its rows of the tile mean nothing.  b0: row (column for a turned
// operand) at which B begins in its map, kb: depth likewise.  finish(row tile, column tile, split, load) is called by the four tile warps of each CTA
// for each tile; load(c, v) gives columns c .. c + 31 of the thread's row, and has to be called by whole warps;
// without a single block of depth the tile is all zeros and load gives them.
// state: the rows that count, which the shape is asked with, and whether a wait has run out, kept in memory from launch to
// launch and read in one load.  A pair whose wait ran out, and every pair of a
// launch behind one where that happened, does no more products: load gives NaN for each tile that is left, so that none
// keeps what an earlier call wrote.  Such a pair says so there and in the error word, and run_tiles returns true.
// selftest: the number of a tile at which the tile warps do as if their wait for it had run out; -1 for none.
template <bool TurnedA, bool TurnedB, typename Shape, typename Finish>
__device__ __forceinline__ bool run_tiles(const CUtensorMap* map_a, const CUtensorMap* map_b, int a_rows,
                                          Shape shape_of, int64_t b0, int64_t kb, uint32_t* err_word, uint32_t timeout_bit,
                                          int32_t* state, int64_t selftest, Finish finish) {
    extern __shared__ unsigned char dynamic[];
    __shared__ MatrixBarriers bars;
    const uint32_t stage0 = (shared_addr(dynamic) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    volatile uint32_t* failed = &bars.failed;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStagesMm; ++s) {
            barrier_init(&bars.full[s], 1);
            barrier_init(&bars.empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            barrier_init(&bars.tile_full[t], 1);
            barrier_init(&bars.tile_empty[t], 8);  // four warps of two CTAs
        }
        barrier_init(&bars.done, 1);
        bars.failed = 0;
        barrier_init_fence();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_addr(&bars.tmem)),
                     "r"(kTmemColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *(volatile uint32_t*)&bars.tmem;
    launch_next();
    wait_previous();
    int32_t count, lost;
    asm volatile("ld.global.v2.s32 {%0, %1}, [%2];" : "=r"(count), "=r"(lost) : "l"(state) : "memory");
    const MatrixShape shape = shape_of((int64_t)count);
    const uint32_t second_bytes = TurnedA || a_rows > kHalf ? kStageBytes : kOperandBytes;  // the second CTA's copies
    const uint32_t stage_bytes = second_bytes + (TurnedA || a_rows > kHalf ? kStageBytes : kOperandBytes + box_rows(a_rows) * 128u);
    const bool late = lost != 0;
    if (late && threadIdx.x == 0)
        give_up(failed);

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool go = !late;
            long long fills = 0;
            for (int64_t i = pair; go && i < shape.tiles(); i += pairs) {
                int64_t row, column, k0, k1;
                int split;
                shape.tile(i, row, column, split);
                shape.depth(split, k0, k1);
                const int ra = (int)(row * kTile + rank * kHalf), rb = (int)(b0 + column * kTile + rank * kHalf);
                for (int64_t k = k0; k < k1; ++k) {
                    if (!matrix_wait(&bars.empty[stage], phase ^ 1u, kProductWaitNs, failed)) {
                        go = false;
                        break;
                    }
                    ++fills;
                    // both CTAs' copies arrive on the first one's barrier
                    const uint32_t bar = cluster_addr(&bars.full[stage], 0);
                    if (rank == 0)
                        barrier_expect(&bars.full[stage], stage_bytes);
                    const uint32_t at = stage0 + stage * kStageBytes, bt = at + kOperandBytes;
                    const int da = (int)(k * kBlockK), db = (int)(kb + k * kBlockK);
                    if constexpr (TurnedA) {
                        copy_tile(at, map_a, ra, da, bar);
                        copy_tile(at + kOperandBytes / 2, map_a, ra + 64, da, bar);
                    } else if (rank == 0 || a_rows > kHalf) {
                        copy_tile(at, map_a, da, ra, bar);
                    }
                    if constexpr (TurnedB) {
                        copy_tile(bt, map_b, rb, db, bar);
                        copy_tile(bt + kOperandBytes / 2, map_b, rb + 64, db, bar);
                    } else {
                        copy_tile(bt, map_b, db, rb, bar);
                    }
                    if (++stage == kStagesMm)
                        stage = 0, phase ^= 1u;
                }
            }
            // until every stage was read: the last arrivals on this CTA's barriers are in
            for (int s = 0; go && s < kStagesMm; ++s) {
                go = matrix_wait(&bars.empty[stage], phase ^ 1u, kProductWaitNs, failed);
                if (++stage == kStagesMm)
                    stage = 0, phase ^= 1u;
            }
            bars.fills[rank] = fills;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            int stage = 0, t = 0;
            uint32_t phase = 0, tphase = 0;
            bool go = !late;
            for (int64_t i = pair; go && i < shape.tiles(); i += pairs) {
                int64_t row, column, k0, k1;
                int split;
                shape.tile(i, row, column, split);
                shape.depth(split, k0, k1);
                if (k0 == k1)
                    continue;
                if (!matrix_wait(&bars.tile_empty[t], tphase ^ 1u, kWaitNs, failed))
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + t * kTile;
                for (int64_t k = k0; k < k1; ++k) {
                    if (!matrix_wait(&bars.full[stage], phase, kCopyWaitNs, failed)) {
                        go = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t at = stage0 + stage * kStageBytes;
                    const uint64_t a = operand_desc(at, TurnedA), b = operand_desc(at + kOperandBytes, TurnedB);
#pragma unroll
                    for (int j = 0; j < kBlockK / 16; ++j)  // 16 of depth: 32 bytes, or two groups of eight
                        product(d, a + j * (TurnedA ? 2048 >> 4 : 32 >> 4), b + j * (TurnedB ? 2048 >> 4 : 32 >> 4),
                                product_desc(TurnedA, TurnedB), k > k0 || j > 0);
                    products_arrive(&bars.empty[stage]);
                    if (++stage == kStagesMm)
                        stage = 0, phase ^= 1u;
                }
                if (!go)
                    break;
                products_arrive(&bars.tile_full[t]);
                if (++t == 2)
                    t = 0, tphase ^= 1u;
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        int t = 0;
        uint32_t tphase = 0;
        bool there = !late;
        for (int64_t i = pair; i < shape.tiles(); i += pairs) {
            int64_t row, column, k0, k1;
            int split;
            shape.tile(i, row, column, split);
            shape.depth(split, k0, k1);
            if (there && k0 < k1) {
                there = __all_sync(0xffffffffu, matrix_wait(&bars.tile_full[t], tphase, kProductWaitNs, failed));
                if (i == selftest) {
                    give_up(failed);
                    there = false;
                }
            }
            if (!there || k0 == k1) {
                const float fill = there ? 0.0f : __int_as_float(0x7fffffff);
                finish(row, column, split, [fill](int, float(&v)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        v[e] = fill;
                });
                continue;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t at = tmem + t * kTile + ((uint32_t)((warp & 3) * 32) << 16);
            finish(row, column, split, [at](int c, float(&v)[32]) { load_columns(at + c, v); });
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                barrier_arrive_cluster(cluster_addr(&bars.tile_empty[t], 0));
            if (++t == 2)
                t = 0, tphase ^= 1u;
        }
    }
    // neither CTA leaves while the other may still write into it
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const bool gave_up = *failed != 0;  // the same in both
    if (__builtin_expect(gave_up, 0))
        matrix_drain(bars, second_bytes, state, err_word, timeout_bit);
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns) : "memory");
    return gave_up;
}

}  // namespace sv
