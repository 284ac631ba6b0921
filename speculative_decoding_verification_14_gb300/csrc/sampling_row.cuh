// sampling_row.cuh -- what every part of the sampling kernel works on: a row's
// arguments and state in shared memory, the walk over a CTA's slice of the row,
// prefix sums, lists of entries, and the rows written at the end.  Included by
// sampling.cu alone.
//
// The parts a row goes through are functions of their own, and what they hand on
// lies in shared memory: the kernel stays within 64 registers a thread, and its
// code short -- a small call spends much of its time fetching code.  They get a
// copy of the kernel's arguments there too.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_verify.h"
#include "sampling_common.cuh"

namespace cg = cooperative_groups;

namespace {

using namespace sv;

constexpr int kNT = 256;
constexpr int kNW = kNT / 32;
constexpr int kBins = 2048;
constexpr int kList = 1024;  // entries of a list
constexpr int kFew = 128;    // entries compared each with each instead of sorted
constexpr int kMaxC = 16;

struct Args {
    const void* logits;
    int64_t stride;
    const float* u;  // NULL: no draw
    int64_t u_stride;
    int32_t* tokens;
    int64_t token_stride;
    float* probs;  // or NULL
    int64_t probs_stride;
    float* p_token;
    void* out;  // truncated logits, or NULL
    int64_t out_stride;
    float* mass;
    int32_t* kept;
    int32_t* status;
    uint32_t* err_word;
    uint32_t* general_rows;  // counter of rows that go the general way, or NULL
    sv_sampling set;
    int64_t V, slice;
    int rows_per_seq, C, fix;
};

enum Cond { kByCount, kByMass, kByLimit, kConds };

struct Found {
    int bin;  // kBins or kNoPlace: none
    uint32_t count, above_count;
    unsigned long long mass, above_mass;
};

// Rows are counted by the upper 16 bits of their logits, which are a bfloat16
// logit's value and a float32 logit's to 2^-8: a place for every magnitude from
// 2^-25 up to 127 of either sign, and one each for what is smaller and larger.
// A place i is 0 below the window, 1..kMags inside it and kMags + 1 above; its
// signed index is i, or -1 - i for negative logits, so that it grows with the
// logit.  Searches run by descending logit: D = kMags + 1 - index.
constexpr int kMag0 = (127 - 25) << 7;
constexpr int kMags = 4094;
constexpr int kPlaces = 2 * (kMags + 2);
constexpr int kChunks = kPlaces / 32;  // places a warp takes at once
constexpr int kFirstTiny = kMags + 1;  // D of the two places below the window
constexpr int kNoPlace = kPlaces;

struct Hit {  // the chunk of places that holds the end of a condition, and what lies above it
    int chunk;
    uint32_t above_count;
    unsigned long long above_mass;
};

struct Chunk {  // 32 places: their sums, and what lies above them in the CTA
    unsigned long long mass, above_mass;
    uint32_t cnt, above_cnt;
};

struct Band {  // a stretch of places that a list may hold
    float lo, hi;  // its logits; +inf: none
    uint32_t above_count;
    bool on, from_top;
};

// What a cut is by: top-k (0: off), the mass top-p has to reach (0: off), the least
// key min-p keeps; what lies above the list; the list's lowest key; and by how much the
// sums may be off.
struct Cut {
    uint32_t k, limit_key, above_count, low;
    unsigned long long p, above_mass, slack;
};

// A row's settings, as the first CTA of the cluster has read them: all CTAs take the same turns,
// also where a program changes a setting or a uniform under the call.
struct alignas(16) Settings {
    float T, u;
    uint32_t k;     // top-k, 0: off
    int code;
    double top_p;   // >= 1: off
    double dmin;    // T ln(min_p)
    bool has_min;
};

// A CTA's shared memory, followed by its chunks of places.  Four CTAs share an SM, and
// leave a good part of it to the first-level cache, where the threads' saved registers are.
struct alignas(16) Shared {
    union {
        struct {
            uint32_t lo[kBins], hi[kBins], cnt[kBins];
            unsigned long long list[kList];  // key << 32 | ~id
        };
        uint32_t count[kPlaces];
    };
    float2 pow2[kSteps];
    Args args;
    // the CTA's slice of the row
    const unsigned char* base;  // the row's first logit
    uint32_t row, s0, s1, off, k0, k1;
    Settings set;
    float sum_T;    // as this CTA has read them: T where float32's first pass takes the float sum, else 0
    // what its parts have found
    RowScale scale;
    Found cut_at;   // the place where the cut lies
    unsigned long long whole, mass;  // of the row; of what is kept
    uint32_t near, kept_n;  // entries counted; kept
    float cut;
    Cut want;  // for the lists
    Hit hit[2][kConds];  // of the search for the cut and of that for the draw
    Found place[2][kConds];
    Found found[kConds];
    unsigned long long part_mass[kMaxC];
    uint32_t part_cnt[kMaxC], part_max[kMaxC], part_tiny[kMaxC], part_list[2][kMaxC];
    float part_noise[kMaxC], part_top[kMaxC], part_sum[kMaxC];
    float fast_sum;  // of the row, against its maximum (float32 under top-p)
    unsigned long long sums[3][kMaxC];
    unsigned long long warp_mass[3][kNW];
    uint32_t warp_cnt[kNW], warp_max[kNW];
    float warp_noise[kNW], warp_top[kNW];
    unsigned long long few[kFew];  // weights of a short list
    unsigned long long list_mass;  // in all
    uint32_t list_n[2];
    Band band[2];  // of the cut and of the draw
    uint32_t want_limit;  // the least key min-p keeps
    // what the first CTA (or the CTA that finds it) tells the others
    uint32_t ok, cut_key, kept, token, token_key;
    unsigned long long kept_mass;
};

// The CTA's own.  Functions of their own ask for it again: what they are handed is an
// address of any kind to them, and its atomics and loads would be slower.
__device__ __forceinline__ Shared* here() {
    extern __shared__ __align__(16) unsigned char shared_bytes[];
    return reinterpret_cast<Shared*>(shared_bytes);
}
__device__ __forceinline__ cg::cluster_group the_cluster() { return cg::this_cluster(); }
__device__ __forceinline__ int cta_rank() { return (int)the_cluster().block_rank(); }
template <class T>
__device__ __forceinline__ T* peer(T* p, int r) {
    return the_cluster().map_shared_rank(p, r);
}

__device__ __noinline__ unsigned long long weight_call(RowScale s, const float2* pow2, float l) {
    return weight_fixed(s, pow2, l);
}

// sum over the warp of integers below 2^62, in three parts so that the lanes' sums fit 32 bits
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long m) {
    const uint32_t a = __reduce_add_sync(kAllLanes, (uint32_t)m & 0x1fffffu);
    const uint32_t b = __reduce_add_sync(kAllLanes, (uint32_t)(m >> 21) & 0x1fffffu);
    const uint32_t c = __reduce_add_sync(kAllLanes, (uint32_t)(m >> 42));
    return a + ((unsigned long long)b << 21) + ((unsigned long long)c << 42);
}

struct Prefix {
    unsigned long long before_mass, mass;  // before this thread; up to it, or in all
    uint32_t before_count, count;
};

// inclusive prefixes over the warp
__device__ __noinline__ Prefix warp_prefix(unsigned long long m, uint32_t n) {
    const int lane = threadIdx.x & 31;
    Prefix p;
    p.mass = m;
    p.count = n;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long pm = __shfl_up_sync(kAllLanes, p.mass, o);
        const uint32_t pn = __shfl_up_sync(kAllLanes, p.count, o);
        if (lane >= o) {
            p.mass += pm;
            p.count += pn;
        }
    }
    p.before_mass = p.mass - m;
    p.before_count = p.count - n;
    return p;
}

// exclusive prefixes over the CTA's threads, and the totals
__device__ __noinline__ Prefix cta_prefix(Shared* sh, unsigned long long m, uint32_t n) {
    sh = here();
    const int warp = threadIdx.x >> 5;
    Prefix p = warp_prefix(m, n);
    __syncthreads();
    if ((threadIdx.x & 31) == 31) {
        sh->warp_mass[0][warp] = p.mass;
        sh->warp_cnt[warp] = p.count;
    }
    __syncthreads();
    p.mass = 0;
    p.count = 0;
#pragma unroll 1
    for (int w = 0; w < kNW; ++w) {
        if (w < warp) {
            p.before_mass += sh->warp_mass[0][w];
            p.before_count += sh->warp_cnt[w];
        }
        p.mass += sh->warp_mass[0][w];
        p.count += sh->warp_cnt[w];
    }
    return p;
}

// sum over the CTA's threads
__device__ __forceinline__ uint32_t cta_sum(Shared* sh, uint32_t x) {
    x = __reduce_add_sync(kAllLanes, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sh->warp_cnt[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0;
#pragma unroll 1
    for (int w = 0; w < kNW; ++w)
        x += sh->warp_cnt[w];
    return x;
}

// ------------------------------------------------------------- the slice -----

template <int ES>
struct View : Slice<ES, kNT> {
    __device__ __forceinline__ explicit View(const Shared* sh) {
        this->base = sh->base;
        this->s0 = sh->s0;
        this->s1 = sh->s1;
        this->off = sh->off;
        this->k0 = sh->k0;
        this->k1 = sh->k1;
    }
};

// --------------------------------------------------------------- lists -----

// The lists lie over the bins and places, which are done with when they are made.
__device__ __forceinline__ unsigned long long* list_at(Shared* sh, int which) {
    return which ? reinterpret_cast<unsigned long long*>(sh->lo) : sh->list;
}

// an entry for a list (of this or another CTA)
__device__ __forceinline__ void offer(uint32_t* n, unsigned long long* list, float l, uint32_t id) {
    const uint32_t at = atomicAdd(n, 1u);
    if (at < (uint32_t)kList)
        list[at] = ((unsigned long long)logit_key(l) << 32) | (uint32_t)~id;
}

// Sorts a list of this CTA: descending logits, ascending ids.
__device__ __noinline__ void sort_list(Shared* sh, int which) {
    sh = here();
    unsigned long long* list = list_at(sh, which);
    const int tid = threadIdx.x;
    if (tid == 0 && sh->list_n[which] > (uint32_t)kList)
        sh->list_n[which] = kList;
    __syncthreads();
    const int n = (int)sh->list_n[which];
    int size = 2;
    while (size < n)
        size <<= 1;
    for (int i = n + tid; i < size; i += kNT)
        list[i] = 0;
    __syncthreads();
    for (int len = 2; len <= size; len <<= 1)
        for (int gap = len >> 1; gap; gap >>= 1) {
            for (int i = tid; i < size / 2; i += kNT) {
                const int x = 2 * i - (i & (gap - 1)), y = x + gap;
                const unsigned long long vx = list[x], vy = list[y];
                if ((vx < vy) == ((x & len) == 0)) {  // descending runs first
                    list[x] = vy;
                    list[y] = vx;
                }
            }
            __syncthreads();
        }
}

// Mass before this thread's share of a sorted list's entries, and in all.
__device__ __noinline__ Prefix list_prefix(Shared* sh, int which) {
    sh = here();
    const unsigned long long* list = list_at(sh, which);
    const int n = (int)sh->list_n[which], own = (n + kNT - 1) / kNT;
    const int i0 = min(own * (int)threadIdx.x, n), i1 = min(i0 + own, n);
    unsigned long long m = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i)
        m += weight_call(sh->scale, sh->pow2, key_logit((uint32_t)(list[i] >> 32)));
    return cta_prefix(sh, m, 0);
}

// whether the cut lies in a list of n entries and this mass: 1, 0, or 2: the sums do not tell
__device__ __forceinline__ int cut_inside(const Cut& c, int n, unsigned long long mass) {
    if ((c.k && c.above_count >= c.k) || (c.p && c.above_count && c.above_mass >= c.p))
        return 0;
    if (c.limit_key >= c.low || (c.k && c.above_count + (uint32_t)n >= c.k))
        return 1;
    if (!c.p || c.above_mass + mass + c.slack < c.p)
        return 0;
    return c.above_mass + mass >= c.p + c.slack ? 1 : 2;
}

// The last group of equal logits in the first list that every filter keeps: the
// cut, the kept mass and count, left in `sh`.  Returns 1 when the cut lies in the list:
// some filter ends with it; 0 when it does not; 2 when the sums do not tell.
__device__ __noinline__ int cut_in_sorted(Shared* sh) {
    sh = here();
    const Cut& c = sh->want;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = (int)sh->list_n[0], own = (n + kNT - 1) / kNT;
    const int i0 = min(own * tid, n), i1 = min(i0 + own, n);
    const Prefix x = list_prefix(sh, 0);
    unsigned long long at = c.above_mass + x.before_mass;
    int last = -1;
    bool near = false;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = (uint32_t)(sh->list[i] >> 32);
        const bool start = i == 0 || (uint32_t)(sh->list[i - 1] >> 32) != key;
        if (start && key >= c.limit_key && (!c.k || c.above_count + i < c.k)) {
            if (!c.p || at < c.p)
                last = i;
            if (c.p && c.above_count + i > 0 && (at < c.p ? c.p - at : at - c.p) < c.slack)
                near = true;
        }
        at += weight_call(sh->scale, sh->pow2, key_logit(key));
    }
    // conditions fail for good once they fail: the last start over all threads
    last = __reduce_max_sync(kAllLanes, last);
    const bool any_near = __syncthreads_or(near);
    if (lane == 0)
        sh->warp_max[warp] = (uint32_t)(last + 1);
    __syncthreads();
    int g = 0;
#pragma unroll 1
    for (int i = 0; i < kNW; ++i)
        g = max(g, (int)sh->warp_max[i]);
    --g;  // -1: nothing of the list is kept
    const uint32_t key = g >= 0 ? (uint32_t)(sh->list[g] >> 32) : c.limit_key;
    if (tid == 0 && g < 0) {
        sh->cut_key = key;
        sh->kept = c.above_count;
        sh->kept_mass = c.above_mass;
    }
    at = c.above_mass + x.before_mass;
    for (int i = i0; i < i1 && g >= 0; ++i) {
        const uint32_t y = (uint32_t)(sh->list[i] >> 32);
        at += weight_call(sh->scale, sh->pow2, key_logit(y));
        if (y == key && (i == n - 1 || (uint32_t)(sh->list[i + 1] >> 32) != key)) {
            sh->cut_key = key;
            sh->kept = c.above_count + i + 1;
            sh->kept_mass = at;
        }
    }
    __syncthreads();
    return any_near ? 2 : cut_inside(c, n, x.mass);
}

// The first entry of a sorted list whose running sum exceeds `target`, left in
// `sh`; whether the list holds it.
__device__ __noinline__ bool draw_in_sorted(Shared* sh, int which, unsigned long long above_mass,
                                            unsigned long long target) {
    sh = here();
    const unsigned long long* list = list_at(sh, which);
    const int n = (int)sh->list_n[which], own = (n + kNT - 1) / kNT;
    const int i0 = min(own * (int)threadIdx.x, n), i1 = min(i0 + own, n);
    const Prefix x = list_prefix(sh, which);
    unsigned long long at = above_mass + x.before_mass;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const uint32_t key = (uint32_t)(list[i] >> 32);
        const unsigned long long w = weight_call(sh->scale, sh->pow2, key_logit(key));
        if (at <= target && at + w > target) {
            sh->token = ~(uint32_t)list[i];
            sh->token_key = key;
        }
        at += w;
    }
    __syncthreads();
    return above_mass <= target && above_mass + x.mass > target;
}

// The same for a list of at most kFew entries in any order, a few threads comparing an
// entry with all: what is larger than it, and what comes before it.  `cut`: find the cut
// (else all of the list counts as kept); `draw`: then the draw at u E, the kept mass E
// being the cut's or, without one, sh->kept_mass.
__device__ __noinline__ int resolve_few(Shared* sh, int which, bool cut, bool draw) {
    sh = here();
    const Cut& c = sh->want;
    const int tid = threadIdx.x, warp = tid >> 5, n = (int)sh->list_n[which];
    const unsigned long long* list = list_at(sh, which);
    if (tid < n)
        sh->few[tid] = weight_call(sh->scale, sh->pow2, key_logit((uint32_t)(list[tid] >> 32)));
    __syncthreads();
    // 2, 4 or 8 threads to an entry
    const int lg = n > 64 ? 1 : n > 32 ? 2 : 3, at = tid >> lg;
    static_assert(kFew << 1 == kNT);
    const unsigned long long mine = at < n ? list[at] : 0;
    const uint32_t key = (uint32_t)(mine >> 32);
    unsigned long long larger = 0, before = 0;
    uint32_t count = 0;
    if (at < n) {
#pragma unroll 4
        for (int j = tid & ((1 << lg) - 1); j < n; j += 1 << lg) {
            const unsigned long long o = list[j], x = sh->few[j];
            if (o > mine)
                before += x;
            if ((uint32_t)(o >> 32) > key) {
                larger += x;
                ++count;
            }
        }
    }
#pragma unroll 1
    for (int o = 1 << lg >> 1; o; o >>= 1) {
        larger += __shfl_xor_sync(kAllLanes, larger, o);
        before += __shfl_xor_sync(kAllLanes, before, o);
        count += __shfl_xor_sync(kAllLanes, count, o);
    }
    larger += c.above_mass;
    before += c.above_mass;
    count += c.above_count;
    const bool has = at < n && (tid & ((1 << lg) - 1)) == 0;
    const unsigned long long w = has ? sh->few[at] : 0;
    bool kept = has;
    int ok = 1;
    if (cut) {
        bool near = false;
        kept = has && key >= c.limit_key && (!c.k || count < c.k);
        if (kept && c.p) {
            near = count > 0 && (larger < c.p ? c.p - larger : larger - c.p) < c.slack;
            kept = larger < c.p;
        }
        // the least key kept, how many, their mass, and the list's
        const uint32_t least = __reduce_min_sync(kAllLanes, kept ? key : 0xffffffffu);
        const unsigned long long list_mass = warp_sum(w), kept_mass = warp_sum(kept ? w : 0ull);
        const uint32_t number = __popc(__ballot_sync(kAllLanes, kept));
        if ((tid & 31) == 0) {
            sh->warp_max[warp] = least;
            sh->warp_mass[0][warp] = list_mass;
            sh->warp_mass[1][warp] = kept_mass;
            sh->warp_cnt[warp] = number;
        }
        const bool any_near = __syncthreads_or(near);
        if (warp == 0) {
            const bool in = tid < kNW;
            const uint32_t x = __reduce_min_sync(kAllLanes, in ? sh->warp_max[tid] : 0xffffffffu);
            const uint32_t sum = __reduce_add_sync(kAllLanes, in ? sh->warp_cnt[tid] : 0u);
            const unsigned long long all = warp_sum(in ? sh->warp_mass[0][tid] : 0ull);
            const unsigned long long mass = warp_sum(in ? sh->warp_mass[1][tid] : 0ull);
            if (tid == 0) {
                sh->cut_key = sum ? x : c.limit_key;
                sh->kept = c.above_count + sum;
                sh->kept_mass = c.above_mass + mass;
                sh->list_mass = all;
            }
        }
        __syncthreads();
        ok = any_near ? 2 : cut_inside(c, n, sh->list_mass);
    }
    if (ok == 1 && draw) {
        const unsigned long long target = floor_scaled(sh->set.u, sh->kept_mass);
        const bool it = kept && before <= target && before + w > target;
        if (it) {
            sh->token = ~(uint32_t)mine;
            sh->token_key = key;
        }
        ok = __syncthreads_or(it) ? 1 : 3;  // 3: above the list, or below it
    }
    return ok;
}

// what the first CTA has found, to the others
__device__ __forceinline__ void share_cut(Shared* sh) {
    const int tid = threadIdx.x;
    if (cta_rank() == 0 && tid > 0 && tid < sh->args.C) {
        *peer(&sh->cut_key, tid) = sh->cut_key;
        *peer(&sh->kept, tid) = sh->kept;
        *peer(&sh->kept_mass, tid) = sh->kept_mass;
        *peer(&sh->ok, tid) = sh->ok;
    }
    the_cluster().sync();
}

// -------------------------------------------------------------- outputs -----

enum Keep { kKeepFrom, kKeepToken, kBadRow };  // logits from `cut` on; one id; a row without an answer

// Probabilities (`Probs`) or truncated logits, of the entries from `cut` on (`From`), of one
// token, or of a row without an answer (`bad`).  Steps (see StepCodes; NULL: all are looked at) and
// vectors none of whose logits reaches `cut` are written without looking further.  inv:
// 2^F over the kept mass.
template <int ES, bool Probs, bool From>
__device__ __noinline__ void write_rows(Shared* sh, const StepCodes* codes, bool bad, float cut, float inv,
                                        uint32_t token) {
    sh = here();
    const RowScale scale = sh->scale;
    const Args& a = sh->args;
    const View<ES> v(sh);
    constexpr int E = View<ES>::E;
    const int64_t row = sh->row;
    float* p = a.probs + row * a.probs_stride;
    unsigned char* o = static_cast<unsigned char*>(a.out) + row * a.out_stride * ES;
    bad = !From && bad;
    const auto keep = [&](float l, uint32_t id) { return From ? l >= cut : id == token; };
    const auto prob = [&](float l, uint32_t id) {
        return bad ? __int_as_float(0x7fffffff)
                   : keep(l, id) ? (From ? weight_float(scale, l) * inv : 1.0f) : 0.0f;
    };
    const auto logit = [&](float l, uint32_t id) {
        return bad || keep(l, id) ? __float_as_uint(l) : 0xff800000u;
    };
    const auto one = [&](uint32_t id) {
        const float l = scalar_entry<ES>(v.base, id);
        if constexpr (Probs) {
            p[id] = prob(l, id);
        } else {
            const uint32_t h = logit(l, id);
            if constexpr (ES == 4)
                reinterpret_cast<uint32_t*>(o)[id] = h;
            else
                reinterpret_cast<unsigned short*>(o)[id] = (unsigned short)(h >> 16);
        }
    };
    // vectors of logits go to 16-byte places, or are written one by one
    const uintptr_t start = Probs ? reinterpret_cast<uintptr_t>(p - v.off) : reinterpret_cast<uintptr_t>(o - v.off * ES);
    if (start & 15u) {
#pragma unroll 1
        for (uint32_t i = v.s0 + threadIdx.x; i < v.s1; i += kNT)
            one(i);
        return;
    }
    const uint32_t marks = codes && !bad ? v.marks(codes, step_code(cut)) : 0xffffu;
    const auto nothing = [&](uint32_t id) {
        if constexpr (Probs) {
            float4* q = reinterpret_cast<float4*>(p + id);
#pragma unroll
            for (int e = 0; e < E / 4; ++e)
                q[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        } else {
            const uint32_t x = ES == 4 ? 0xff800000u : 0xff80ff80u;
            *reinterpret_cast<uint4*>(o + (size_t)id * ES) = make_uint4(x, x, x, x);
        }
    };
    v.template walk_marked<kDeep>(
        marks,
        [&](const uint4& w, uint32_t id) {
            if (!bad && !(vector_max<ES>(w) >= cut)) {
                nothing(id);
                return;
            }
            if constexpr (Probs) {
                float4* q = reinterpret_cast<float4*>(p + id);
#pragma unroll
                for (int e = 0; e < E / 4; ++e)
                    q[e] = make_float4(prob(vector_entry<ES>(w, 4 * e), id + 4 * e),
                                       prob(vector_entry<ES>(w, 4 * e + 1), id + 4 * e + 1),
                                       prob(vector_entry<ES>(w, 4 * e + 2), id + 4 * e + 2),
                                       prob(vector_entry<ES>(w, 4 * e + 3), id + 4 * e + 3));
            } else {
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (ES == 4)
                        h[j] = logit(vector_entry<ES>(w, j), id + j);
                    else
                        h[j] = (logit(vector_entry<ES>(w, 2 * j), id + 2 * j) >> 16) |
                               (logit(vector_entry<ES>(w, 2 * j + 1), id + 2 * j + 1) & 0xffff0000u);
                }
                *reinterpret_cast<uint4*>(o + (size_t)id * ES) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        },
        one);
    v.template pass_unmarked<kDeep>(marks, nothing);
}

// whichever the call wants
template <int ES>
__device__ __forceinline__ void write_out(Shared* sh, const StepCodes* codes, Keep how, float cut, float inv,
                                          uint32_t token) {
    const bool from = how == kKeepFrom, bad = how == kBadRow;
    if (sh->args.probs)
        from ? write_rows<ES, true, true>(sh, codes, bad, cut, inv, token)
             : write_rows<ES, true, false>(sh, codes, bad, cut, inv, token);
    else if (sh->args.out)
        from ? write_rows<ES, false, true>(sh, codes, bad, cut, inv, token)
             : write_rows<ES, false, false>(sh, codes, bad, cut, inv, token);
}

__device__ __forceinline__ void put_token(const Shared* sh, int32_t id, float p) {
    const Args& a = sh->args;
    if (a.tokens)
        a.tokens[sh->row * a.token_stride] = id;
    if (a.p_token)
        a.p_token[sh->row] = p;
}

// the row's other answers; the kept share of the row is mass / whole
__device__ __forceinline__ void put_rest(const Shared* sh, int code, uint32_t kept, unsigned long long mass,
                                         unsigned long long whole) {
    const Args& a = sh->args;
    if (cta_rank() == 0 && threadIdx.x == 0) {
        if (a.mass)
            a.mass[sh->row] = code ? __int_as_float(0x7fffffff) : (float)((double)mass / (double)whole);
        if (a.kept)
            a.kept[sh->row] = (int32_t)min(kept, 0x7fffffffu);
        if (a.status)
            a.status[sh->row] = code;
        if (code)
            atomicOr(a.err_word, 1u << code);
    }
}

// 2^F / mass as a float: three roundings
__device__ __forceinline__ float inverse_mass(const RowScale& s, unsigned long long mass) {
    return __fdiv_rn((float)(1ull << s.fix), (float)mass);
}

}  // namespace
