// sampling.cu -- drawing tokens, and truncating logits, under temperature,
// top-k, top-p and min-p.
//
// For a row l of V logits and a temperature T > 0, w_v = exp((l_v - l_max)/T),
// S = sum w.  Entry v is kept when l_v > -inf and
//   top-k: fewer than k entries are larger than l_v;
//   top-p: the mass of the entries larger than l_v is below top_p S;
//   min-p: w_v >= min_p;
// every filter looks at the untruncated row and keeps or drops equal logits
// together, so the kept set is {l >= cut}.  With E the kept mass, the draw
// lays the kept entries out by descending logit and ascending id and takes the
// first whose running sum exceeds u E.  The kept set is a prefix of that
// order, so the cut and the draw are one search: for the place where a count
// or a mass is crossed.  T = 0 keeps the lowest id of the largest logits.
//
// Design: one cluster of C CTAs per row, a slice of the vocabulary per CTA.
//  A. One pass counts the entries by the upper 16 bits of their logits in shared
//     memory (one 32-bit add per entry, 3 instructions to find its place) and takes
//     the maximum.
//  B. Each CTA adds up the cluster's counts at its share of the places, weighs the
//     places that hold something, and finds whether the cut lies there; then the same
//     for the draw.
//  C. bfloat16 places are single values: their masses are exact, and what is left
//     is to find which of the equal entries was drawn.  float32: a second pass sums and
//     lists exactly around the places found.
//  D. Probabilities or truncated logits are written in a last pass.
// Rows with logits outside the window of places that matter, or crowded where the
// list should hold them, go the general way (sampling_general.cuh).
//
// What bounds it: instructions, shared-memory adds and waits, not bytes.  A CTA of 64128
// bfloat16 entries (256 rows of 128256, two CTAs a row, 3.4 CTAs on an SM) spends 36 of its
// 72 thousand cycles counting (about seven instructions an entry, and an add that
// takes some 3.5 turns for 32 lanes whose places fall on the banks as they come), 3 on its
// start, 5 on the exchange, 7 on weighing, 8 on two searches and 8 on finding the drawn entry.
// Four CTAs of 256 threads fit an SM (43 KB, 64 registers).  Parts of a fixed size
// are why rows are cut no finer than the planner does.  A row alone is a chain
// of some twenty barriers through code fetched for the first time: 46 thousand cycles
// for 32000 float32 entries, which is why most loops here are not unrolled.
// Per launch on one GB300 (replayed back to back, inputs larger than L2): 256 rows of
// 128256 bfloat16 under top-p 54 us (65.7 MB, 1.2 TB/s); 2048 of them truncated
// 241 us (1.05 GB in and out, 4.4 TB/s); 256 rows of 128256 float32 under every filter
// with their probabilities 94 us (263 MB, 2.8 TB/s); one of 32000 float32 21 us.
// What rows beside these cost: beyond the counted magnitudes 256 rows of 128256 bfloat16 take
// 660 us instead of 58, 150 of 50257 float32 84 instead of 67; float32 rows at T = 0, counted and then
// walked twice more, 71 us for 256 of 128256 (bfloat16 34); a float32 row in a batch of 150 whose
// stretches miss the cut or hold too many entries, less than one in a hundred, adds some 240 us to its launch.
#include "sampling_row.cuh"

#include "sampling_general.cuh"
#include "sv_context.h"

namespace {

// the logit of least magnitude at place D (bfloat16: the only one)
__device__ __forceinline__ float place_value(int D) {
    const int s = kMags + 1 - D, i = s >= 0 ? s : -1 - s;
    const uint32_t b = i ? (uint32_t)(kMag0 - 1 + i) : 0u;
    return __uint_as_float((b | (s < 0 ? 0x8000u : 0u)) << 16);
}

// the place of a logit
__device__ __forceinline__ int place_of(float l) {
    const uint32_t b = __float_as_uint(l);
    const int m = (int)((b & 0x7fffffffu) >> 16);
    const int i = min(max(m, kMag0 - 1), kMag0 + kMags) - (kMag0 - 1);
    return kMags + 1 - ((b >> 31) ? -1 - i : i);
}

// the two places below the window: they hold +0 and -0, which are one logit
__device__ __forceinline__ bool is_tiny(int D) { return D == kFirstTiny || D == kFirstTiny + 1; }
__device__ __forceinline__ bool inside(int D) { return D >= 1 && D <= kPlaces - 2 && !is_tiny(D); }

// a float32 place's largest or smallest logit; inside the window
__device__ __forceinline__ float place_end(int D, bool largest) {
    const float l = place_value(D);
    return largest == (l > 0.0f) ? __uint_as_float(__float_as_uint(l) | 0xffffu) : l;
}

// a logit that stands for place D: bfloat16 the only one, float32 the middle one
template <int ES>
__device__ __forceinline__ float place_logit(float lmax, int D) {
    const float l = place_value(D);
    if constexpr (ES == 4)
        return fminf(__uint_as_float(__float_as_uint(l) | 0x8000u), lmax);
    return l;
}

// mass of n entries at place D: bfloat16 exactly, float32 by the middle one's float weight;
// one of those at l_max's place is l_max, which weighs 1: at low temperatures the middle weighs
// nothing, and a row's mass is never 0
template <int ES>
__device__ __forceinline__ unsigned long long place_mass(const RowScale& s, const float2* pow2, int D, uint32_t n) {
    if (n == 0)
        return 0;
    const float l = place_logit<ES>(s.lmax, D);
    if constexpr (ES == 2)
        return mass_fixed(s, pow2, l, n);
    const float w = ex2_approx((l - s.lmax) * s.ch), one = (float)(1ull << s.fix);
    const bool top = ((__float_as_uint(l) ^ __float_as_uint(s.lmax)) >> 16) == 0;
    return __float2ull_rn(top ? one + (float)(n - 1) * (w * one) : (float)n * (w * one));
}

// Counts the two logits whose upper 16 bits x holds.  Each place's byte
// offset is 4 i or 4 (-1 - i), both logits' in the halves of one word.
// Logits above -127 alone are counted: what is missing lies below.
__device__ __forceinline__ void count_pair(Shared* sh, uint32_t x) {
    constexpr uint32_t lo = (kMag0 - 1) * 0x10001u, hi = (kMag0 + kMags) * 0x10001u;
    constexpr int far = 4 * (-1 - (kMags + 1));
    const uint32_t m = x & 0x7fff7fffu;
    uint32_t sign, i;
    asm("max.u16x2 %0, %1, %2;" : "=r"(i) : "r"(m), "r"(lo));
    asm("min.u16x2 %0, %1, %2;" : "=r"(i) : "r"(i), "r"(hi));
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(sign) : "r"(x), "r"(0u), "r"(0xbb99u));  // sign of each half
    const uint32_t o = (((i - lo) << 2) ^ sign) & 0xfffcfffcu;
    const int o0 = (int)(short)(o & 0xffffu), o1 = (int)o >> 16;
    char* zero = reinterpret_cast<char*>(sh->count + kMags + 2);
    if (o0 != far)
        atomicAdd(reinterpret_cast<uint32_t*>(zero + o0), 1u);
    if (o1 != far)
        atomicAdd(reinterpret_cast<uint32_t*>(zero + o1), 1u);
}

// A.  The CTA's counts, and the codes of its steps; returns its largest key, 0xffffffff
// for a NaN.
template <int ES>
__device__ __noinline__ uint32_t count_pass(Shared* sh, StepCodes* codes) {
    sh = here();
    const View<ES> v(sh);
    const int shift = v.code_shift();
    float lmax = __int_as_float(0xff800000);
    float step = lmax;           // float32: a step's largest
    // float32 under top-p: the row's sum, too, in floats
    const bool sum = ES == 4 && sh->sum_T > 0.0f;
    const float ch = __fdiv_rn(1.44269502162933349609375f, sum ? sh->sum_T : 1.0f);
    float m = lmax, t = 0.0f;
    uint32_t two = 0xff80ff80u;  // bfloat16: of each half
#pragma unroll
    for (int i = 0; i < 16; ++i)
        codes->code[i] = 0;
    v.template walk_steps<kDeep, false>(
        [&](const uint4& w, uint32_t) {
            if constexpr (ES == 2) {
                count_pair(sh, w.x);
                count_pair(sh, w.y);
                count_pair(sh, w.z);
                count_pair(sh, w.w);
                uint32_t m, x;
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w.x), "r"(w.y));
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w.z), "r"(w.w));
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x));
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(two) : "r"(two), "r"(m));
            } else {
                count_pair(sh, __byte_perm(w.x, w.y, 0x7632));
                count_pair(sh, __byte_perm(w.z, w.w, 0x7632));
                const float top = vector_max_nan<4>(w);
                step = max_nan(step, top);
                if (sum) {
                    if (!(top <= m))
                        join_sums(m, t, top, 0.0f, ch);
                    if (top > __int_as_float(0xff800000))
                        t += exp_sum<4>(w, m, ch);
                }
            }
        },
        [&](uint32_t s) {
            if constexpr (ES == 2) {
                step = max_nan(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
                two = 0xff80ff80u;
            }
            const uint8_t x = (uint8_t)step_code(step);
            if (shift == 0 || x > codes->code[s >> shift])
                codes->code[s >> shift] = x;
            lmax = max_nan(lmax, step);
            step = __int_as_float(0xff800000);
        },
        [&](uint32_t id) {  // a lone logit, paired with -inf, which is not counted
            const float l = scalar_entry<ES>(v.base, id);
            count_pair(sh, (__float_as_uint(l) >> 16) | 0xff800000u);
            lmax = max_nan(lmax, l);
            if (sum)
                join_sums(m, t, l, 1.0f, ch);
        });
    if (sum) {
        join_lanes<32>(m, t, ch);
        if ((threadIdx.x & 31) == 0) {
            sh->warp_top[threadIdx.x >> 5] = m;
            sh->warp_noise[threadIdx.x >> 5] = t;
        }
    }
    uint32_t key = lmax == lmax ? logit_key(lmax) : 0xffffffffu;
    key = __reduce_max_sync(kAllLanes, key);
    if ((threadIdx.x & 31) == 0)
        sh->warp_max[threadIdx.x >> 5] = key;
    __syncthreads();
    return __reduce_max_sync(kAllLanes, sh->warp_max[threadIdx.x & (kNW - 1)]);
}

// Chunks of places per CTA, and this CTA's first and last.
__device__ __forceinline__ int chunks_per(int C) { return (kChunks + C - 1) / C; }
__device__ __forceinline__ int first_chunk(int C, int rank) { return min(rank * chunks_per(C), kChunks); }

// A CTA's chunks lie behind its shared memory.
__device__ __forceinline__ Chunk* chunks(Shared* sh) { return reinterpret_cast<Chunk*>(sh + 1); }

// Entries at place D over the cluster, once they are merged: of a place of this CTA's
// range, and of any.
__device__ __forceinline__ uint32_t own_count(const Shared* sh, int D) { return sh->count[kPlaces - 1 - D]; }
__device__ __forceinline__ uint32_t any_count(Shared* sh, int D) {
    const int r = D / 32 / chunks_per(sh->args.C);
    return peer(sh->count, r)[kPlaces - 1 - D];
}

// Adds the other CTAs' counts at this CTA's range of places to its own: nobody else
// reads them there.  A thread takes four places at a time, of every CTA.
__device__ __noinline__ void merge_counts(Shared* sh) {
    sh = here();
    const int C = sh->args.C, rank = cta_rank(), first = first_chunk(C, rank) * 32;
    const int n = first_chunk(C, rank + 1) * 8 - first / 4, per = (n + kNT - 1) / kNT;
    uint4* own = reinterpret_cast<uint4*>(sh->count + kPlaces - first) - n;
    int i = 0, g = 0, r = rank;
#pragma unroll 1
    for (int t = 0; t < per * (C - 1); t += 4) {
        uint4 x[4];
        int at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i == 0) {
                g = threadIdx.x;
                r = r + 1 < C ? r + 1 : 0;
            }
            i = i + 1 < per ? i + 1 : 0;
            at[j] = t + j < per * (C - 1) && g < n ? g : -1;
            if (at[j] >= 0)
                x[j] = *peer(own + g, r);
            g += kNT;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at[j] >= 0) {
                const uint4 s = own[at[j]];
                own[at[j]] = make_uint4(s.x + x[j].x, s.y + x[j].y, s.z + x[j].z, s.w + x[j].w);
            }
    }
    __syncthreads();
}

// B.  Masses and counts of the CTA's chunks of places, and what lies above each in this
// CTA; the CTA's sums to every CTA.  float32: with the square of how far the places'
// sums may be off, their entries' weights being spread over the places' width.
template <int ES>
__device__ __noinline__ void weigh_places(Shared* sh) {
    sh = here();
    const RowScale scale = sh->scale;
    const int C = sh->args.C, rank = cta_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = first_chunk(C, rank), c1 = first_chunk(C, rank + 1);
    float noise = 0.0f;
#pragma unroll 1
    for (int c = c0 + warp; c < c1; c += kNW) {
        const int D = c * 32 + lane;
        uint32_t n = own_count(sh, D);
        unsigned long long m = 0;
        if (__any_sync(kAllLanes, n)) {
            m = place_mass<ES>(scale, sh->pow2, D, n);
            if (ES == 4 && n) {
                // width 2^-7 of the place's power of two, 2^-25 below the window; 1 / sqrt(12)
                const float l = place_logit<ES>(scale.lmax, D);
                const uint32_t b = __float_as_uint(l) & 0x7f800000u;
                const float width = is_tiny(D) ? 0x1p-25f : __uint_as_float(b - (7u << 23));
                const float e = ex2_approx((l - scale.lmax) * scale.ch) * (width * 0.28867513f * scale.ch);
                noise = fmaf(e * e, (float)n, noise);
            }
            n = __reduce_add_sync(kAllLanes, n);
            m = warp_sum(m);
        }
        if (lane == 0) {
            chunks(sh)[c - c0].mass = m;
            chunks(sh)[c - c0].cnt = n;
        }
    }
    if constexpr (ES == 4) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            noise += __shfl_xor_sync(kAllLanes, noise, o);
        if (lane == 0)
            sh->warp_noise[warp] = noise;
    }
    __syncthreads();
    if (warp == 0) {
        const int q = (c1 - c0 + 31) / 32, i0 = min(lane * q, c1 - c0), i1 = min(i0 + q, c1 - c0);
        unsigned long long m = 0;
        uint32_t n = 0;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            m += chunks(sh)[i].mass;
            n += chunks(sh)[i].cnt;
        }
        const Prefix x = warp_prefix(m, n);
        m = x.before_mass;
        n = x.before_count;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            chunks(sh)[i].above_mass = m;
            chunks(sh)[i].above_cnt = n;
            m += chunks(sh)[i].mass;
            n += chunks(sh)[i].cnt;
        }
        m = __shfl_sync(kAllLanes, x.mass, 31);
        n = __shfl_sync(kAllLanes, x.count, 31);
        if (lane < C) {
            *peer(&sh->part_mass[rank], lane) = m;
            *peer(&sh->part_cnt[rank], lane) = n;
        }
        if constexpr (ES == 4) {
            noise = sh->warp_noise[lane & (kNW - 1)];
#pragma unroll
            for (int o = kNW / 2; o; o >>= 1)
                noise += __shfl_xor_sync(kAllLanes, noise, o);
            if (lane < C)
                *peer(&sh->part_noise[rank], lane) = noise;
        }
    }
    the_cluster().sync();
}

struct Wanted {
    uint32_t k;            // count to reach, 0: none
    unsigned long long p;  // mass to reach, 0: none; with `draw` a mass to exceed
    int limit;             // the last place min-p keeps, kNoPlace: none
    bool draw;
};

// Finds the places where the conditions end, in every CTA's `place[set]`, and
// returns the first.  The thread whose chunk of places holds one hands it to a warp,
// which goes through the chunk.
template <int ES>
__device__ __noinline__ Found search_places(Shared* sh, int set, const Wanted s) {
    sh = here();
    const int C = sh->args.C, rank = cta_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = first_chunk(C, rank), c1 = first_chunk(C, rank + 1);
    static_assert(kChunks <= kNT, "a thread per chunk");
    const unsigned long long above_m = warp_sum(lane < rank ? sh->part_mass[lane] : 0ull);
    const uint32_t above_n = __reduce_add_sync(kAllLanes, lane < rank ? sh->part_cnt[lane] : 0u);
    if (tid < c1 - c0) {
        const unsigned long long before_m = above_m + chunks(sh)[tid].above_mass;
        const uint32_t before_n = above_n + chunks(sh)[tid].above_cnt;
        const unsigned long long after_m = before_m + chunks(sh)[tid].mass;
        const uint32_t after_n = before_n + chunks(sh)[tid].cnt;
        const Hit h = {c0 + tid, before_n, before_m};
        if (s.k && before_n < s.k && after_n >= s.k)
            sh->hit[set][kByCount] = h;
        if (s.draw ? before_m <= s.p && after_m > s.p : s.p && before_m < s.p && after_m >= s.p)
            sh->hit[set][kByMass] = h;
        if (s.limit / 32 == c0 + tid)
            sh->hit[set][kByLimit] = h;
    }
    __syncthreads();
    if (warp < kConds && sh->hit[set][warp].chunk >= 0) {
        const Hit h = sh->hit[set][warp];
        Found f;
        f.bin = h.chunk * 32 + lane;
        f.count = own_count(sh, f.bin);
        f.mass = place_mass<ES>(sh->scale, sh->pow2, f.bin, f.count);
        const Prefix x = warp_prefix(f.mass, f.count);
        f.above_mass = h.above_mass + x.before_mass;
        f.above_count = h.above_count + x.before_count;
        const unsigned long long em = h.above_mass + x.mass;
        const uint32_t en = h.above_count + x.count;
        const bool here = warp == kByCount ? f.above_count < s.k && en >= s.k
                          : warp == kByLimit ? f.bin == s.limit
                          : s.draw ? f.above_mass <= s.p && em > s.p
                                   : f.above_mass < s.p && em >= s.p;
        // the lane that has it stores here, the others pass it on
        const uint32_t who = __ballot_sync(kAllLanes, here);
        if (who) {
            const int from = __ffs(who) - 1;
            f.bin = h.chunk * 32 + from;
            f.count = __shfl_sync(kAllLanes, f.count, from);
            f.above_count = __shfl_sync(kAllLanes, f.above_count, from);
            f.mass = __shfl_sync(kAllLanes, f.mass, from);
            f.above_mass = __shfl_sync(kAllLanes, f.above_mass, from);
            if (lane < C)
                *peer(&sh->place[set][warp], lane) = f;
        }
    }
    the_cluster().sync();
    Found f = sh->place[set][0];
    for (int c = 1; c < kConds; ++c)
        if (sh->place[set][c].bin < f.bin)
            f = sh->place[set][c];
    return f;
}

// The entry number r by ascending id at place D (bfloat16); the CTA that holds it
// returns its id in one thread, every other thread returns -1.  Each CTA gathers
// the ids of its entries there; in the one that holds it, the id with as many smaller ones
// as are left is it.
__device__ __noinline__ int64_t find_entry(Shared* sh, const StepCodes* codes, int D, unsigned long long r) {
    sh = here();
    const View<2> v(sh);
    const int C = sh->args.C, rank = cta_rank(), tid = threadIdx.x;
    const float l = place_value(D);
    const uint32_t bits = __float_as_uint(l) >> 16, two = bits * 0x10001u;
    const unsigned short* q = reinterpret_cast<const unsigned short*>(v.base);
    const uint32_t least = step_code(l);
    constexpr uint32_t kIds = kPlaces;
    uint32_t* ids = sh->count;  // the counts are done with
    const auto found = [&](uint32_t id) {
        const uint32_t at = atomicAdd(&sh->list_n[0], 1u);
        if (at < kIds)
            ids[at] = id;
    };
    v.walk_marked<kDeep>(
        v.marks(codes, least),
        [&](const uint4& w, uint32_t id) {
            uint32_t m;
            const uint32_t x[4] = {w.x ^ two, w.y ^ two, w.z ^ two, w.w ^ two};
            asm("min.u16x2 %0, %1, %2;" : "=r"(m) : "r"(x[0]), "r"(x[1]));
            asm("min.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x[2]));
            asm("min.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x[3]));
            if ((m & 0xffffu) == 0 || (m >> 16) == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if ((x[j] & 0xffffu) == 0)
                        found(id + 2 * j);
                    if ((x[j] >> 16) == 0)
                        found(id + 2 * j + 1);
                }
            }
        },
        [&](uint32_t id) {
            if (q[id] == bits)
                found(id);
        });
    __syncthreads();
    const uint32_t n = sh->list_n[0];
    if (C > 1) {
        if (tid < C)
            *peer(&sh->part_list[0][rank], tid) = n;
        the_cluster().sync();
#pragma unroll 1
        for (int c = 0; c < rank; ++c) {
            if (r < sh->part_list[0][c])
                return -1;
            r -= sh->part_list[0][c];
        }
    }
    if (r >= n)
        return -1;
    if (n > kIds) {
        // a stretch of ids per thread: how many it holds, then which one
        const uint32_t per = (v.s1 - v.s0 + kNT - 1) / kNT;
        const uint32_t e0 = min(v.s0 + tid * per, v.s1), e1 = min(e0 + per, v.s1);
        uint32_t mine = 0;
        for (uint32_t e = e0; e < e1; ++e)
            mine += q[e] == bits;
        const Prefix x = cta_prefix(sh, 0, mine);
        if (r < x.before_count || r >= x.before_count + mine)
            return -1;
        uint32_t left = (uint32_t)r - x.before_count, e = e0;
        while (e < e1 && (q[e] != bits || left-- != 0))
            ++e;
        return e < e1 ? (int64_t)e : -1;
    }
    if (n <= (uint32_t)kNT) {
        const uint32_t id = tid < n ? ids[tid] : 0;
        uint32_t before = 0;
        for (uint32_t j = 0; j < n; ++j)
            before += ids[j] < id;
        return tid < n && before == r ? (int64_t)id : -1;
    }
    // the largest x with at most r ids below it
    uint32_t x = 0;
    for (int bit = 31 - __clz(v.s1); bit >= 0; --bit) {
        const uint32_t t = x | 1u << bit;
        uint32_t below = 0;
        for (uint32_t i = tid; i < n; i += kNT)
            below += ids[i] < t;
        if (cta_sum(sh, below) <= r)
            x = t;
    }
    return tid == 0 ? (int64_t)x : -1;
}

// A stretch of places around one of interest: lane r looks at r places to either
// side.  It reaches so far that `margin` of the row's mass lies on either side of the
// place in the middle, as far as the list holds the entries; all entries from the largest
// on, where the list holds those.
__device__ __noinline__ void band_around(Shared* sh, int which, const Found f, unsigned long long margin) {
    sh = here();
    const int lane = threadIdx.x & 31, D = f.bin - 16 + lane;
    const uint32_t n = D >= 1 && D <= kPlaces - 2 ? any_count(sh, D) : 0;
    const Prefix x = warp_prefix(place_mass<4>(sh->scale, sh->pow2, D, n), n);
    const int r = lane & 15;
    // the middle place is lane 16
    const uint32_t mid = __shfl_sync(kAllLanes, x.before_count, 16);
    const uint32_t up = mid - __shfl_sync(kAllLanes, x.before_count, 16 - r);
    const uint32_t down = __shfl_sync(kAllLanes, x.count, 16 + r) - mid;
    const unsigned long long up_mass =
        __shfl_sync(kAllLanes, x.before_mass, 16) - __shfl_sync(kAllLanes, x.before_mass, 16 - r);
    const unsigned long long down_mass =
        __shfl_sync(kAllLanes, x.mass, 16 + r) - __shfl_sync(kAllLanes, x.mass, 16);
    const bool fits_top = f.above_count + down <= (uint32_t)kList, fits = up + down <= (uint32_t)kList;
    const uint32_t top = __ballot_sync(kAllLanes, fits_top) & 0xffffu;
    const uint32_t top_far = __ballot_sync(kAllLanes, fits_top && down_mass >= margin) & 0xffffu;
    const uint32_t part = __ballot_sync(kAllLanes, fits) & 0xffffu;
    const uint32_t part_far = __ballot_sync(kAllLanes, fits && down_mass >= margin && up_mass >= margin) & 0xffffu;
    Band b = {0.0f, 0.0f, 0, (top | part) != 0, top != 0};
    if (b.on) {
        const uint32_t far = top ? top_far : part_far;
        const int reach = far ? __ffs(far) - 1 : 31 - __clz(top ? top : part);
        const int first = top ? 1 : max(f.bin - reach, 1), last = min(f.bin + reach, kPlaces - 2);
        b.above_count = top ? 0 : f.above_count - __shfl_sync(kAllLanes, up, reach);
        b.hi = top ? sh->scale.lmax : place_end(first, true);
        b.lo = place_end(last, false);
        b.on = !is_tiny(first) && !is_tiny(last);
    }
    if (threadIdx.x == 0)
        sh->band[which] = b;
    __syncthreads();
}

// The first CTA's list, with the other CTAs' behind its own.
__device__ __noinline__ void pull_list(Shared* sh, int which) {
    sh = here();
    unsigned long long* to = list_at(sh, which);
    const int C = sh->args.C;
    const int lane = threadIdx.x & 31;
    const uint32_t n = __reduce_add_sync(kAllLanes, lane < C ? sh->part_list[which][lane] : 0u);
    for (uint32_t i = sh->part_list[which][0] + threadIdx.x; i < n && i < (uint32_t)kList; i += kNT) {
        int r = 0;
        uint32_t j = i;
        while (j >= sh->part_list[which][r])
            j -= sh->part_list[which][r++];
        to[i] = peer(to, r)[j];
    }
    if (threadIdx.x == 0)
        sh->list_n[which] = min(n, (uint32_t)kList);
    __syncthreads();
}

// The sums of the second pass: the row; what lies above the cut's stretch; above the
// draw's.  With the stretches' entries in the CTA's lists.
struct Sums {
    unsigned long long x[3];
};

__device__ __forceinline__ SumScale sum_scale(Shared* sh, const RowScale& s) {
    SumScale t(s);
    float2* steps = reinterpret_cast<float2*>(sh->hi);  // behind the second list: 16 KB
    for (int i = threadIdx.x; i < kSteps * 16; i += kNT)
        steps[i] = sh->pow2[i >> 4];
    t.steps = steps + (threadIdx.x & 15);
    __syncthreads();
    return t;
}
// What a pass adds to: all, and of each stretch that is no list from the largest on what
// lies above it.  With what goes to the lists; a stretch that is off, or whose entries the
// list has, reaches from infinity on.
struct Above {
    float chi, clo, dhi, dlo;
    __device__ __forceinline__ Above(const Shared* sh, bool list) {
        const float inf = __int_as_float(0x7f800000);
        chi = sh->band[0].hi;
        dhi = sh->band[1].hi;
        clo = list ? sh->band[0].lo : inf;
        dlo = list ? sh->band[1].lo : inf;
    }
    __device__ __forceinline__ void take(Shared* sh, float l, uint32_t id) const {
        if (l >= clo && l <= chi)
            offer(&sh->list_n[0], list_at(sh, 0), l, id);
        if (l >= dlo && l <= dhi)
            offer(&sh->list_n[1], list_at(sh, 1), l, id);
    }
};

// by weight_fixed, of the whole slice (|l_max c| from 128 on: l_max 17.7 at T = 0.2; the open draw of
// 150 rows of 50257 takes 99 us there and 78 at T = 1) or its entries beside the vectors
__device__ __noinline__ Sums sum_each(Shared* sh, bool list, bool edges) {
    sh = here();
    View<4> v(sh);
    const Above a(sh, list);
    Sums s = {{0, 0, 0}};
    const auto one = [&](float l, uint32_t id) {
        const unsigned long long x = weight_fixed(sh->scale, sh->pow2, l);
        s.x[0] += x;
        s.x[1] += l > a.chi ? x : 0;
        s.x[2] += l > a.dhi ? x : 0;
        a.take(sh, l, id);
    };
    const uint32_t head = edges ? v.head_end() : v.s1, tail = edges ? v.tail_start() : v.s1;
    const uint32_t n = head - v.s0 + (v.s1 - tail);
#pragma unroll 1
    for (uint32_t j = threadIdx.x; j < n; j += kNT) {
        const uint32_t id = j < head - v.s0 ? v.s0 + j : tail + (j - (head - v.s0));
        one(scalar_entry<4>(v.base, id), id);
    }
    return s;
}

__device__ __noinline__ Sums sum_exact(Shared* sh, bool list) {
    sh = here();
    const RowScale scale = sh->scale;
    const bool fits = fabsf(scale.lmax * scale.ch) < 128.0f;
    Sums s = sum_each(sh, list, fits);
    if (!fits)
        return s;
    const View<4> v(sh);
    const Above a(sh, list);
    const SumScale t = sum_scale(sh, scale);
    const Units units(scale.fix);
    WeightSum all, over_c, over_d;
    v.walk<1, true>(
        [&](const uint4& w, uint32_t id) {
            const float l[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
            bool listed = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = sum_weight(t, l[e]);
                all.add(x);
                if (l[e] > a.chi)
                    over_c.add(x);
                else
                    listed |= l[e] >= a.clo;
                if (l[e] > a.dhi)
                    over_d.add(x);
                else
                    listed |= l[e] >= a.dlo;
            }
            all.into(s.x[0], units);
            if (a.chi < __int_as_float(0x7f800000))
                over_c.into(s.x[1], units);
            if (a.dhi < __int_as_float(0x7f800000))
                over_d.into(s.x[2], units);
            if (listed) {
                uint4 x = w;
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    a.take(sh, __uint_as_float(x.x), id + e);
                    x = make_uint4(x.y, x.z, x.w, 0);
                }
            }
        },
        [](uint32_t) {});
    s.x[0] += all.rest(scale.fix);
    s.x[1] += over_c.rest(scale.fix);
    s.x[2] += over_d.rest(scale.fix);
    return s;
}

// The cut's entries alone.
__device__ __noinline__ void list_entries(Shared* sh, const StepCodes* codes) {
    sh = here();
    const View<4> v(sh);
    const float low = sh->band[0].lo;
    const uint32_t least = step_code(low);
    const auto take = [&](float l, uint32_t id) {
        if (l >= low)
            offer(&sh->list_n[0], list_at(sh, 0), l, id);
    };
    v.walk_marked<kDeep>(
        v.marks(codes, least),
        [&](const uint4& w, uint32_t id) {
            if (vector_max<4>(w) >= low) {
                take(__uint_as_float(w.x), id);
                take(__uint_as_float(w.y), id + 1);
                take(__uint_as_float(w.z), id + 2);
                take(__uint_as_float(w.w), id + 3);
            }
        },
        [&](uint32_t id) { take(scalar_entry<4>(v.base, id), id); });
}

// How far the first pass's float sum may be off, as a share of itself: 2^-n.  A weight
// is off by (l_max - l)/T * 2.5 * 2^-24 + 2^-22, which keeps below 2^-17 of the sum for
// any V.  Each of a thread's vectors may raise its maximum, which rescales its sum by a
// power good to 2^-22 with two roundings of 2^-24 beside it: 2^-14 holds for 64 vectors
// a thread and the joins of threads and CTAs.
__device__ __forceinline__ int fast_bits(const Shared* sh) {
    const uint32_t vectors = (sh->args.slice / 4 + kNT) / kNT;
    return vectors <= 64 ? 14 : max(14 - (26 - __clz(vectors - 1)), 0);
}

// The lists of the second pass in the first CTA, and what they say of the cut and the
// draw; leaves in sh->ok 1: found, 0: not in the lists, 2: too near a border for
// these sums.  `first`: the lists are new.
__device__ __noinline__ void settle(Shared* sh, bool by_mass, bool summed, bool first) {
    sh = here();
    const int tid = threadIdx.x, C = sh->args.C;
    const bool draw = sh->args.u != nullptr;
    if (summed) {
        const int warp = tid >> 5, lane = tid & 31;
        if (warp < 3) {
            const unsigned long long x = warp_sum(lane < C ? sh->sums[warp][lane] : 0ull);
            if (lane == 0)
                sh->sums[warp][0] = x;
        }
        __syncthreads();
    }
    if (sh->band[0].on && tid == kNT - 1) {  // a thread that has nothing to pull, mostly
        if (!summed)
            sh->sums[0][0] = by_mass ? __float2ull_rn(sh->fast_sum * (float)(1ull << sh->scale.fix)) : 0;
        const unsigned long long whole = sh->sums[0][0];
        sh->want = {sh->set.k, sh->want_limit, sh->band[0].above_count, logit_key(sh->band[0].lo),
                    by_mass ? ceil_scaled(sh->set.top_p, whole) : 0, sh->sums[1][0],
                    summed ? 0 : whole >> fast_bits(sh)};
    }
    if (first && sh->band[0].on)
        pull_list(sh, 0);
    if (first && sh->band[1].on)
        pull_list(sh, 1);
    __syncthreads();
    int ok = 3;  // 3: the draw is not in this list
    if (sh->band[0].on) {
        if (sh->want_limit > logit_key(sh->band[0].hi)) {
            ok = 0;
        } else if (sh->list_n[0] <= (uint32_t)kFew) {
            ok = resolve_few(sh, 0, true, draw);
        } else {
            if (first)
                sort_list(sh, 0);
            ok = cut_in_sorted(sh);
            if (ok == 1 && draw)
                ok = draw_in_sorted(sh, 0, sh->want.above_mass, floor_scaled(sh->set.u, sh->kept_mass)) ? 1 : 3;
        }
    } else if (tid == 0) {
        sh->kept_mass = sh->sums[0][0];
        sh->cut_key = kKeyMinusInf + 1;
        sh->kept = 0;
    }
    __syncthreads();
    if (ok == 3 && draw) {
        if (!sh->band[1].on) {
            ok = 0;
        } else if (sh->list_n[1] <= (uint32_t)kFew) {
            if (tid == 0)
                sh->want = {0, 0, 0, 0, 0, sh->sums[2][0], 0};
            __syncthreads();
            ok = resolve_few(sh, 1, false, true);
        } else {
            sort_list(sh, 1);
            ok = draw_in_sorted(sh, 1, sh->sums[2][0], floor_scaled(sh->set.u, sh->kept_mass)) ? 1 : 0;
        }
        ok = ok == 3 ? 0 : ok;
    }
    if (tid == 0)
        sh->ok = ok == 3 ? 1 : ok;
    __syncthreads();
}

// C, float32.  Leaves the cut, what is kept, the row's sum in the first CTA's
// sums[0][0], and the drawn entry there; false when the stretches do not hold them.
// `fine`: integer sums at once.
__device__ __noinline__ bool exact_pass(Shared* sh, const StepCodes* codes, bool by_mass, bool fine) {
    sh = here();
    const int rank = cta_rank(), tid = threadIdx.x;
    for (bool first = true;; first = false, fine = true) {
        Sums s = {{0, 0, 0}};
        if (fine)
            s = sum_exact(sh, first);
        else
            list_entries(sh, codes);
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const unsigned long long x = warp_sum(s.x[j]);
            if ((tid & 31) == 0)
                sh->warp_mass[j][tid >> 5] = x;
        }
        __syncthreads();
        const int warp = tid >> 5, lane = tid & 31;
        if (warp < 3) {
            const unsigned long long x = warp_sum(lane < kNW ? sh->warp_mass[warp][lane] : 0ull);
            if (lane == 0)
                *peer(&sh->sums[warp][rank], 0) = x;
        } else if (warp < 5 && lane == 0) {
            *peer(&sh->part_list[warp - 3][rank], 0) = sh->list_n[warp - 3];
        }
        the_cluster().sync();
        if (rank == 0)
            settle(sh, by_mass, fine, first);
        share_cut(sh);
        const uint32_t ok = sh->ok;
        if (ok != 2)
            return ok;
        the_cluster().sync();  // everyone has read `ok`
    }
}

// Of everything from -127 down, the entries above -inf.
template <int ES>
__device__ __noinline__ uint32_t count_far(Shared* sh) {
    sh = here();
    const View<ES> v(sh);
    uint32_t n = 0;
    v.each([&](float l, uint32_t) { n += place_of(l) == kPlaces - 1 && l > __int_as_float(0xff800000); });
    return cta_sum(sh, n);
}

// Whether the slice holds logits below the window other than zeros (bfloat16).
__device__ __noinline__ uint32_t any_tiny(Shared* sh) {
    sh = here();
    const View<2> v(sh);
    bool any = false;
    v.each([&](float l, uint32_t) { any = any || (l != 0.0f && is_tiny(place_of(l))); });
    return __syncthreads_or(any);
}

// a count of every CTA's, added up over the cluster
__device__ __forceinline__ uint32_t cluster_sum(Shared* sh, uint32_t x) {
    const int C = sh->args.C;
    the_cluster().sync();  // everyone has read `part_tiny`
    if ((int)threadIdx.x < C)
        *peer(&sh->part_tiny[cta_rank()], threadIdx.x) = x;
    the_cluster().sync();
    x = 0;
#pragma unroll 1
    for (int r = 0; r < C; ++r)
        x += sh->part_tiny[r];
    return x;
}

// A row whose answer does not depend on logits outside the window of places goes
// through the following parts; each returns false, in every CTA, for the others.
//
// bfloat16: the places' sums are exact, and so are the cut and the draw.
// float32: they place the cut and the draw to within a few places.  A second
// pass takes the sums of the row and of what lies above the two stretches of
// places around them, and lists the stretches' entries, among which the exact cut and
// draw are found; where a stretch turns out not to hold them, the row is left to
// the general way.  Few entries above the cut are listed whole, and need no
// sum but the row's for top-p: the first pass has it in floats, to 2^-14, and where an
// entry lies nearer to top-p's border than that, a pass takes it in integers.

// The counts and the scale of the weights.
template <int ES>
__device__ __noinline__ bool count_places(Shared* sh, StepCodes* codes) {
    sh = here();
    const int tid = threadIdx.x, C = sh->args.C, rank = cta_rank();
    uint32_t key = count_pass<ES>(sh, codes);
    the_cluster().barrier_wait();  // every CTA runs: its memory may be written
    if (tid < C) {
        *peer(&sh->part_max[rank], tid) = key;
        *peer(&sh->part_tiny[rank], tid) = sh->count[kMags + 1] + sh->count[kMags + 2];
    }
    if (rank == 0 && tid > 64 && tid < 64 + C)  // a warp that has nothing else to do
        *peer(&sh->set, tid - 64) = sh->set;
    if (ES == 4 && tid < 32 && sh->sum_T > 0.0f) {
        float m = sh->warp_top[tid & (kNW - 1)], t = sh->warp_noise[tid & (kNW - 1)];
        join_lanes<kNW>(m, t, __fdiv_rn(1.44269502162933349609375f, sh->sum_T));
        if (tid < C) {
            *peer(&sh->part_top[rank], tid) = m;
            *peer(&sh->part_sum[rank], tid) = t;
        }
    }
    the_cluster().sync();
    const int lane = tid & 31;
    key = __reduce_max_sync(kAllLanes, lane < C ? sh->part_max[lane] : 0u);
    const uint32_t tiny = __reduce_add_sync(kAllLanes, lane < C ? sh->part_tiny[lane] : 0u);  // below the window
    RowScale scale;
    scale.fix = sh->args.fix;
    scale.lmax = key_logit(key);
    const float T = sh->set.T;
    set_temperature(scale, T > 0.0f ? T : 1.0f);
    if (tid == 0)
        sh->scale = scale;
    if (ES == 4 && tid < 32 && sh->set.top_p < 1.0) {
        const bool in = lane < C;
        float m = in ? sh->part_top[lane] : __int_as_float(0xff800000), t = in ? sh->part_sum[lane] : 0.0f;
        join_lanes<kMaxC>(m, t, scale.ch);
        if (tid == 0)
            sh->fast_sum = t;
    }
    __syncthreads();
    if (sh->set.code || key == 0xffffffffu || !inside(place_of(scale.lmax)))
        return false;
    if (T == 0.0f)
        return ES == 2;
    // logits from -127 down must weigh nothing
    if (scale.g != 1.0f || !((scale.lmax + 127.0f) * scale.ch >= 61.0f))
        return false;
    // bfloat16 logits below the window are taken for 0: their weights are off by
    // 2^-24/T of themselves, which must not show in the sum (>= 1 at l_max) at 2^-39
    return !(ES == 2 && tiny && (float)tiny * weight_float(scale, 0.0f) > T * 3.0517578e-5f &&
             cluster_sum(sh, any_tiny(sh)));
}

// T = 0 (bfloat16): the first entry at the largest value's place.
__device__ __noinline__ void take_largest(Shared* sh, const StepCodes* codes) {
    sh = here();
    const int64_t id = find_entry(sh, codes, place_of(sh->scale.lmax), 0);
    if (id >= 0) {
        put_token(sh, (int32_t)id, 1.0f);
#pragma unroll 1
        for (int r = 0; r < sh->args.C; ++r)
            *peer(&sh->token, r) = (uint32_t)id;
    }
    if (sh->args.probs || sh->args.out) {
        the_cluster().sync();
        write_out<2>(sh, codes, kKeepToken, sh->scale.lmax, 0.0f, sh->token);
    }
    put_rest(sh, SV_OK, 1, 1, 1);
}

// The places' masses, the place of the cut, and what it keeps.
template <int ES>
__device__ __noinline__ bool find_cut(Shared* sh) {
    sh = here();
    const int tid = threadIdx.x, C = sh->args.C;
    if (C > 1)
        merge_counts(sh);
    weigh_places<ES>(sh);
    const int lane = tid & 31;
    const unsigned long long whole = warp_sum(lane < C ? sh->part_mass[lane] : 0ull);
    const uint32_t near = __reduce_add_sync(kAllLanes, lane < C ? sh->part_cnt[lane] : 0u);
    Wanted s = {sh->set.k, sh->set.top_p < 1.0 ? ceil_scaled(sh->set.top_p, whole) : 0, kNoPlace, false};
    if (sh->set.has_min) {
        // the smallest float l with l - l_max >= T ln(min_p); bfloat16: the smallest of those
        float limit = __double2float_ru((double)sh->scale.lmax + sh->set.dmin);
        if (tid == 0)
            sh->want_limit = logit_key(limit);
        if (ES == 2 && limit > 0.0f && (__float_as_uint(limit) & 0xffffu))
            limit = __uint_as_float((__float_as_uint(limit) & 0xffff0000u) + 0x10000u);
        s.limit = place_of(limit);
        if (!inside(s.limit))
            return false;
    }
    if (tid == 0) {
        sh->whole = sh->mass = whole;
        sh->near = sh->kept_n = near;
        sh->cut = -3.402823466e38f;
        sh->cut_at.bin = kNoPlace;
    }
    if (s.k || s.p || s.limit < kNoPlace) {
        const Found f = search_places<ES>(sh, 0, s);
        if (is_tiny(f.bin))
            return false;
        if (tid == 0 && f.bin < kNoPlace) {
            sh->cut_at = f;
            sh->mass = f.above_mass + f.mass;
            if (ES == 2) {
                sh->kept_n = f.above_count + f.count;
                sh->cut = place_value(f.bin);
            }
        }
    }
    __syncthreads();
    if (sh->cut_at.bin == kNoPlace && (int64_t)sh->near < sh->args.V) {
        // everything is kept: those from -127 down that are not -inf as well
        if (sh->set.k)
            return false;
        const uint32_t far = cluster_sum(sh, count_far<ES>(sh));
        if (tid == 0)
            sh->kept_n += far;
        __syncthreads();
    }
    return true;
}

// bfloat16: the drawn place, and which of its entries it is.
__device__ __noinline__ bool draw_value(Shared* sh, const StepCodes* codes) {
    sh = here();
    const Wanted w = {0, floor_scaled(sh->set.u, sh->mass), kNoPlace, true};
    const Found d = search_places<2>(sh, 1, w);
    if (is_tiny(d.bin))
        return false;
    const float l = place_value(d.bin);
    // of the place's entries, each with the same share of its mass; products below 2^62
    const int cut = max(34 - __clzll(d.mass) - __clz(d.count), 0);
    const unsigned long long at = ((w.p - d.above_mass) >> cut) * d.count / max(d.mass >> cut, 1ull);
    const int64_t id = find_entry(sh, codes, d.bin, min((uint32_t)at, d.count - 1));
    if (id >= 0)
        put_token(sh, (int32_t)id, weight_float(sh->scale, l) * inverse_mass(sh->scale, sh->mass));
    return true;
}

// float32: the stretches around the cut and the draw, and the second pass.
__device__ __noinline__ bool settle_exactly(Shared* sh, const StepCodes* codes) {
    sh = here();
    const int tid = threadIdx.x;
    const bool by_mass = sh->set.top_p < 1.0, draw = sh->args.u != nullptr;
    // four standard deviations of the places' sum, and what their middles miss
    float noise = (tid & 15) < sh->args.C ? sh->part_noise[tid & 15] : 0.0f;
#pragma unroll
    for (int o = kMaxC / 2; o; o >>= 1)
        noise += __shfl_xor_sync(kAllLanes, noise, o);
    const float deviations = 4.0f * sqrtf(noise) * (float)(1ull << sh->scale.fix);  // may be infinite
    const unsigned long long margin = __float2ull_rn(fminf(deviations, (float)sh->whole)) + (sh->whole >> 12);
    if (sh->cut_at.bin < kNoPlace) {
        band_around(sh, 0, sh->cut_at, margin);
        if (!sh->band[0].on)
            return false;
    }
    if (draw && !sh->band[0].from_top) {
        const Wanted w = {0, floor_scaled(sh->set.u, sh->mass), kNoPlace, true};
        const Found h = search_places<4>(sh, 1, w);
        if (!sh->band[0].on || place_end(h.bin, true) > sh->band[0].hi) {
            band_around(sh, 1, h, margin);
            if (!sh->band[1].on)
                return false;
        }
    }
    the_cluster().barrier_arrive();
    // a float sum will do to tell whether an entry listed whole lies above top-p's
    // border; not where it becomes part of the answer, or entries weigh too little (a filter's
    // `mass`: 256 rows of 128256 float32 under top-k 200 and top-p take 188 us with it, 104 without)
    const bool fine =
        !sh->band[0].from_top || sh->args.mass ||
        (by_mass && sh->cut_at.bin < kNoPlace && place_mass<4>(sh->scale, sh->pow2, sh->cut_at.bin, 1) < sh->whole >> 15);
    the_cluster().barrier_wait();  // every CTA has read the places around: lists may lie over them
    if (!exact_pass(sh, codes, by_mass, fine))
        return false;
    if (tid == 0) {
        sh->whole = sh->sums[0][0];
        sh->mass = sh->kept_mass;
        if (sh->band[0].on)
            sh->kept_n = sh->kept;
        sh->cut = key_logit(sh->cut_key);
        if (draw && cta_rank() == 0)
            put_token(sh, (int32_t)sh->token,
                      weight_float(sh->scale, key_logit(sh->token_key)) * inverse_mass(sh->scale, sh->mass));
    }
    __syncthreads();
    return true;
}

// The whole call, or false.
template <int ES>
__device__ __forceinline__ bool by_place(Shared* sh) {
    StepCodes codes;
    if (!count_places<ES>(sh, &codes))
        return false;
    if constexpr (ES == 2) {
        if (sh->set.T == 0.0f) {
            take_largest(sh, &codes);
            return true;
        }
    }
    if (!find_cut<ES>(sh))
        return false;
    if constexpr (ES == 2) {
        if (sh->args.u && !draw_value(sh, &codes))
            return false;
    } else {
        if (!settle_exactly(sh, &codes))
            return false;
    }
    write_out<ES>(sh, &codes, kKeepFrom, sh->cut, inverse_mass(sh->scale, sh->mass), 0);
    put_rest(sh, SV_OK, sh->kept_n, sh->mass, sh->whole);
    return true;
}

template <int ES>
__device__ __noinline__ void general_row(Shared* sh, int code) {
    sh = here();
    General<ES> g(sh);
    g.run(code);
}

__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// What the row's parts need to know: where it lies, and its settings; what only the
// later parts need, by a thread that nothing waits for before the counts are taken.
template <int ES>
__device__ __forceinline__ void set_up(Shared* sh, const Args& a) {
    const int tid = threadIdx.x;
    const uint32_t row = blockIdx.x / a.C;
    {
        // the part's first 32 KB are on their way while the counts are zeroed
        const int64_t first = cta_rank() * a.slice, n = min(a.V - first, a.slice) * ES;
        if (tid * 128 < n)
            prefetch(static_cast<const unsigned char*>(a.logits) + ((int64_t)row * a.stride + first) * ES + tid * 128);
    }
    if (tid == 0) {
        const Slice<ES, kNT> v(static_cast<const unsigned char*>(a.logits) + (int64_t)row * a.stride * ES, a.V, a.slice,
                              cta_rank());
        sh->args = a;
        sh->row = row;
        sh->base = v.base;
        sh->s0 = v.s0;
        sh->s1 = v.s1;
        sh->off = v.off;
        sh->k0 = v.k0;
        sh->k1 = v.k1;
        sh->want_limit = 0;
        const float inf = __int_as_float(0x7f800000);
        sh->band[0] = sh->band[1] = {inf, inf, 0, false, false};
    } else if (tid == 32) {
        const int64_t seq = row / (uint32_t)a.rows_per_seq;
        const float T = a.set.temperatures ? a.set.temperatures[seq] : a.set.temperature;
        const double top_p = a.set.top_ps ? (double)a.set.top_ps[seq] : a.set.top_p;
        sh->sum_T = top_p < 1.0 ? T : 0.0f;
        if (cta_rank() == 0) {
            const int32_t k = a.set.top_ks ? a.set.top_ks[seq] : a.set.top_k;
            sh->set.T = T;
            sh->set.k = k > 0 ? (uint32_t)k : 0;
            sh->set.top_p = top_p;
        }
    } else if (tid >= 64 && tid < 64 + 2 * kConds) {
        sh->hit[(tid - 64) / kConds][(tid - 64) % kConds].chunk = -1;
        sh->place[(tid - 64) / kConds][(tid - 64) % kConds].bin = kNoPlace;
    } else if (tid >= 96 && tid < 98) {
        sh->list_n[tid - 96] = 0;
    } else if (tid >= kNT - kSteps) {
        sh->pow2[tid - (kNT - kSteps)] = kPow2Steps[tid - (kNT - kSteps)];
    }
    uint4* z = reinterpret_cast<uint4*>(sh->count);
    for (int i = tid; i < kPlaces / 4; i += kNT)
        z[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (tid == 32 && cta_rank() == 0) {
        const int64_t seq = row / (uint32_t)a.rows_per_seq;
        const double min_p = a.set.min_ps ? (double)a.set.min_ps[seq] : a.set.min_p;
        const float T = sh->set.T, u = a.u ? a.u[row * a.u_stride] : 0.0f;
        sh->set.u = u;
        sh->set.has_min = min_p > 0.0;
        sh->set.code = !(T == 0.0f || (T >= 1.17549435e-38f && T <= 3.402823466e38f)) || !(sh->set.top_p > 0.0) || !(min_p < 1.0)
                       ? SV_ERR_INVALID_ARG
                   : !(u >= 0.0f && u < 1.0f) ? SV_ERR_UNIFORM_RANGE
                                              : SV_OK;
        if (min_p > 0.0)
            sh->set.dmin = (double)T * log(min_p);
    }
}

template <int ES>
__global__ void __launch_bounds__(kNT, 4) sv_sample_kernel(const __grid_constant__ Args a) {
    Shared* sh = here();
    the_cluster().barrier_arrive();
    set_up<ES>(sh, a);
    if (by_place<ES>(sh)) {
        the_cluster().sync();  // no CTA leaves while another may still read its memory
        return;
    }
    the_cluster().sync();  // every CTA is done with what it was told
    if (sh->args.general_rows && cta_rank() == 0 && threadIdx.x == 0)
        atomicAdd(sh->args.general_rows, 1u);
    general_row<ES>(sh, sh->set.code);
}

// with a CTA's chunks of places
size_t shared_size(int cluster) {
    return sizeof(Shared) + (size_t)((kChunks + cluster - 1) / cluster) * sizeof(Chunk);
}
static_assert(4 * (sizeof(Shared) + kChunks * sizeof(Chunk) + 1024) <= 233472, "four CTAs per SM");

int launch(sv_ctx* ctx, Args& a, int B, int rows, int64_t V, int dtype, cudaStream_t stream) {
    sv_plan plan;
    const int rc = spec_sample_get_plan(ctx, B, rows, V, dtype, &plan);
    if (rc != SV_OK)
        return rc;
    const int es = dtype == SV_BF16 ? 2 : 4;
    a.err_word = ctx->d_err;
    a.general_rows = ctx->general_rows;
    a.V = V;
    a.slice = plan.slice;
    a.C = plan.cluster;
    a.rows_per_seq = rows;
    a.fix = weight_bits(V);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)plan.grid, 1, 1);
    cfg.blockDim = dim3(kNT, 1, 1);
    cfg.dynamicSmemBytes = shared_size(plan.cluster);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)plan.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    DeviceGuard guard(ctx->device);
    if (cudaLaunchKernelEx(&cfg, es == 2 ? sv_sample_kernel<2> : sv_sample_kernel<4>, a) !=
        cudaSuccess) {
        (void)cudaGetLastError();
        return SV_ERR_CUDA;
    }
    return SV_OK;
}

// The checks that the draw and the filter share.
int check(const sv_ctx* ctx, const void* logits, int dtype, int64_t stride, int B, int rows,
          int64_t V, const sv_sampling* s) {
    if (!ctx || !logits || !s || (dtype != SV_F32 && dtype != SV_BF16))
        return SV_ERR_INVALID_ARG;
    if (B < 1 || B > ctx->max_B || rows < 1 || rows > ctx->max_K + 1 || V < 1 || V > ctx->max_V ||
        V > ((int64_t)1 << 31) || stride < V || stride > ((int64_t)1 << 40))
        return SV_ERR_INVALID_ARG;
    if ((double)B * (double)rows * (double)stride >= 1099511627776.0)  // 2^40
        return SV_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == SV_BF16 ? 2 : 4) || !aligned(s->temperatures, 4) ||
        !aligned(s->top_ks, 4) || !aligned(s->top_ps, 4) || !aligned(s->min_ps, 4))
        return SV_ERR_INVALID_ARG;
    if (!s->temperatures && !(s->temperature == 0.0f || (s->temperature >= 1.17549435e-38f &&
                                                         std::isfinite(s->temperature))))
        return SV_ERR_INVALID_ARG;
    if ((!s->top_ps && !(s->top_p > 0.0)) || (!s->min_ps && !(s->min_p < 1.0)))
        return SV_ERR_INVALID_ARG;
    return SV_OK;
}

// Whether one of n rows of x_bytes shares memory with one of n rows of y_bytes.  Rows of a kind do
// not overlap, so that where neither end of two rows meets, the lower one meets no later one.
bool meet(const void* x, int64_t x_stride, const void* y, int64_t y_stride, int64_t n, int64_t x_bytes,
          int64_t y_bytes) {
    const char *x0 = static_cast<const char*>(x), *y0 = static_cast<const char*>(y);
    if (y0 >= x0 + (n - 1) * x_stride + x_bytes || x0 >= y0 + (n - 1) * y_stride + y_bytes)
        return false;
    for (int64_t i = 0, j = 0; i < n && j < n;) {
        const char *a = x0 + i * x_stride, *b = y0 + j * y_stride;
        if (a < b + y_bytes && b < a + x_bytes)
            return true;
        ++(a < b ? i : j);
    }
    return false;
}

}  // namespace

namespace sv {

int sampling_setup() {
    for (const void* fn : {(const void*)sv_sample_kernel<2>, (const void*)sv_sample_kernel<4>}) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared_size(1)) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return 0;
        }
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return 8;
        }
    }
    return logprobs_setup() ? 16 : 8;
}

}  // namespace sv

extern "C" {

int spec_sample_get_plan(sv_ctx* ctx, int B, int rows_per_seq, int64_t V, int logits_dtype,
                         sv_plan* out) {
    if (!ctx)
        return SV_ERR_INVALID_ARG;
    return spec_sample_plan_for(ctx->num_sms, ctx->sampling_max_cluster, B, rows_per_seq, V,
                                logits_dtype, ctx->ovr_cluster, out);
}

int spec_sample_set_telemetry(sv_ctx* ctx, uint32_t* general_rows) {
    if (!ctx || !aligned(general_rows, 4))
        return SV_ERR_INVALID_ARG;
    ctx->general_rows = general_rows;
    return SV_OK;
}

int spec_sample_run(sv_ctx* ctx, const void* logits, int logits_dtype, int64_t logits_stride,
                    const float* uniforms, int64_t uniforms_stride, int B, int rows_per_seq,
                    int64_t V, const sv_sampling* settings, int32_t* tokens, int64_t tokens_stride,
                    float* probs, int64_t probs_stride, float* p_token, int32_t* kept,
                    int32_t* status, void* stream) {
    const int rc = check(ctx, logits, logits_dtype, logits_stride, B, rows_per_seq, V, settings);
    if (rc != SV_OK)
        return rc;
    const int64_t most = (int64_t)1 << 40;
    if (!uniforms || !tokens || uniforms_stride < 1 || uniforms_stride > most ||
        tokens_stride < 1 || tokens_stride > most || !aligned(uniforms, 4) || !aligned(tokens, 4) ||
        !aligned(probs, 4) || !aligned(p_token, 4) || !aligned(kept, 4) || !aligned(status, 4) ||
        (probs && (probs_stride < V || probs_stride > most)))
        return SV_ERR_INVALID_ARG;
    if (probs && meet(logits, logits_stride * (logits_dtype == SV_BF16 ? 2 : 4), probs, probs_stride * 4,
                      (int64_t)B * rows_per_seq, V * (logits_dtype == SV_BF16 ? 2 : 4), V * 4))
        return SV_ERR_INVALID_ARG;
    Args a;
    std::memset(&a, 0, sizeof a);
    a.logits = logits;
    a.stride = logits_stride;
    a.u = uniforms;
    a.u_stride = uniforms_stride;
    a.tokens = tokens;
    a.token_stride = tokens_stride;
    a.probs = probs;
    a.probs_stride = probs_stride;
    a.p_token = p_token;
    a.kept = kept;
    a.status = status;
    a.set = *settings;
    return launch(ctx, a, B, rows_per_seq, V, logits_dtype, static_cast<cudaStream_t>(stream));
}

int spec_filter_run(sv_ctx* ctx, const void* logits, int logits_dtype, int64_t logits_stride,
                    int B, int rows_per_seq, int64_t V, const sv_sampling* settings,
                    void* out_logits, int64_t out_stride, int32_t* kept, float* mass,
                    int32_t* status, void* stream) {
    const int rc = check(ctx, logits, logits_dtype, logits_stride, B, rows_per_seq, V, settings);
    if (rc != SV_OK)
        return rc;
    const int es = logits_dtype == SV_BF16 ? 2 : 4;
    if (!out_logits || !aligned(out_logits, es) || out_stride < V ||
        out_stride > ((int64_t)1 << 40) || !aligned(kept, 4) || !aligned(mass, 4) ||
        !aligned(status, 4))
        return SV_ERR_INVALID_ARG;
    // in place, or apart: rows that overlap others would be read after they were written
    const int64_t n = (int64_t)B * rows_per_seq;
    if (!(logits == out_logits && (n == 1 || logits_stride == out_stride)) &&
        meet(logits, logits_stride * es, out_logits, out_stride * es, n, V * es, V * es))
        return SV_ERR_INVALID_ARG;
    Args a;
    std::memset(&a, 0, sizeof a);
    a.logits = logits;
    a.stride = logits_stride;
    a.out = out_logits;
    a.out_stride = out_stride;
    a.kept = kept;
    a.mass = mass;
    a.status = status;
    a.set = *settings;
    return launch(ctx, a, B, rows_per_seq, V, logits_dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
