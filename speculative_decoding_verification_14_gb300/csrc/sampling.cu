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
//  A. a pass for l_max;
//  B. a pass that adds every entry's count and integer weight into 2048 bins
//     over t = (l_max - l) c, 32 to the octave, in shared memory; the cluster
//     adds its CTAs' bins up, each CTA a range of them, and finds the bin where
//     the first filter ends (the cut) and then the one that u E falls into;
//  C. the entries of such a bin go to a list in the first CTA, which sorts it
//     and finds the exact place.  A bin with more entries than the list holds
//     is split by the logits' keys, 2048 ways, until it fits or is one value.
//  D. probabilities or truncated logits are written in a last pass.
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
constexpr int kBins = 2048;
constexpr int kList = 1024;  // entries of the list
constexpr int kOwn = kList / kNT;  // of them per thread
constexpr int kMaxC = 16;
constexpr float kBinsPerOctave = 32.0f;

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
    sv_sampling set;
    int64_t V, slice;
    int rows_per_seq, C, fix;
};

enum Cond { kByCount, kByMass, kByLimit, kConds };

struct Found {
    int bin;  // kBins: none
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

struct alignas(16) Shared {
    union {
        struct {
            uint32_t lo[kBins], hi[kBins], cnt[kBins];
            unsigned long long list[kList];  // key << 32 | ~id
        };
        uint32_t count[kPlaces];
    };
    float2 pow2[64];
    unsigned long long chunk_mass[kChunks];
    uint32_t chunk_cnt[kChunks];
    struct {
        int chunk;
        uint32_t above_count;
        unsigned long long above_mass;
    } hit[2][kConds];  // of the search for the cut and of that for the draw
    Found place[2][kConds];
    unsigned long long part_mass[kMaxC];
    uint32_t part_cnt[kMaxC];
    uint32_t part_max[kMaxC];
    uint32_t part_tiny[kMaxC];
    unsigned long long warp_mass[kNW];
    uint32_t warp_cnt[kNW];
    uint32_t warp_max[kNW];
    Found found[kConds];
    uint32_t list_n[2];
    unsigned long long sums[3][kMaxC];
    uint32_t ok;
    // what the first CTA (or the CTA that finds it) tells the others
    uint32_t cut_key;
    uint32_t kept;
    unsigned long long kept_mass;
    uint32_t token;
    uint32_t token_key;
};

template <int ES>
struct Kernel {
    const Args& a;
    cg::cluster_group cluster;
    Shared& sh;
    int tid, lane, warp, rank, C;
    int64_t row;
    const unsigned char* base;  // the row's first logit
    uint32_t s0, s1;            // this CTA's slice, by ids
    // The slice's 16-byte vectors: number k holds the ids from k E - off on, where off is the
    // place of the row's first logit in its own vector.  What they leave at the
    // slice's ends (the row's ends: slices meet between vectors) is taken one by one.
    uint32_t off, k0, k1;
    RowScale scale;

    static constexpr int E = 16 / ES;

    __device__ Kernel(const Args& args, Shared& shared)
        : a(args), cluster(cg::this_cluster()), sh(shared) {
        tid = threadIdx.x;
        lane = tid & 31;
        warp = tid >> 5;
        C = a.C;
        rank = (int)cluster.block_rank();
        row = blockIdx.x / C;
        base = static_cast<const unsigned char*>(a.logits) + row * a.stride * ES;
        off = (uint32_t)(reinterpret_cast<uintptr_t>(base) & 15u) / ES;
        const int64_t v0 = rank * a.slice - off, v1 = v0 + a.slice;
        s0 = (uint32_t)(v0 < 0 ? 0 : v0 < a.V ? v0 : a.V);
        s1 = (uint32_t)(v1 < a.V ? v1 : a.V);
        k0 = (s0 + off + E - 1) / E;
        k1 = (s1 + off) / E;
        if (k1 < k0)
            k1 = k0;
        scale.fix = a.fix;
    }

    __device__ __forceinline__ const uint4* vectors() const {
        return reinterpret_cast<const uint4*>(base - (size_t)off * ES);
    }
    __device__ __forceinline__ uint32_t head_end() const { return min(k0 * E - off, s1); }
    __device__ __forceinline__ uint32_t tail_start() const { return max(k1 * E - off, head_end()); }

    // vec(w, id of its first logit) for every vector of the slice, one(id) for every other logit
    template <int D, class Vec, class One>
    __device__ __forceinline__ void walk(Vec&& vec, One&& one) const {
        const uint4* p = vectors() + k0 + tid;
        for (uint32_t k = k0 + tid; k < k1; k += D * kNT, p += D * kNT) {
            uint4 w[D];
#pragma unroll
            for (int j = 0; j < D; ++j)
                if (k + j * kNT < k1)
                    w[j] = load_stream(p + j * kNT);
#pragma unroll
            for (int j = 0; j < D; ++j)
                if (k + j * kNT < k1)
                    vec(w[j], (k + j * kNT) * E - off);
        }
        for (uint32_t i = s0 + tid; i < head_end(); i += kNT)
            one(i);
        for (uint32_t i = tail_start() + tid; i < s1; i += kNT)
            one(i);
    }

    // fn(l, id) for every entry of the slice
    template <class F>
    __device__ __forceinline__ void each(F&& fn) const {
        walk<4>(
            [&](const uint4& w, uint32_t id) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    fn(vector_entry<ES>(w, e), id + e);
            },
            [&](uint32_t id) { fn(scalar_entry<ES>(base, id), id); });
    }

    // the linear bin of a logit; larger logits, smaller bins
    __device__ __forceinline__ int bin_of(float l) const {
        const float t = (scale.lmax - l) * scale.ch * kBinsPerOctave;
        return t < (float)(kBins - 1) ? (int)t : kBins - 1;
    }

    template <class Map>
    __device__ void histogram(Map&& map) {
        for (int b = tid; b < kBins; b += kNT)
            sh.lo[b] = sh.hi[b] = sh.cnt[b] = 0;
        if (tid < kConds)
            sh.found[tid].bin = kBins;
        if (tid == 0)
            sh.list_n[0] = 0;
        __syncthreads();
        each([&](float l, uint32_t) {
            const int b = map(l);
            if (b < 0)
                return;
            const unsigned long long w = weight_fixed(scale, sh.pow2, l);
            const uint32_t wl = (uint32_t)w;
            const uint32_t old = atomicAdd(&sh.lo[b], wl);
            const uint32_t h = (uint32_t)(w >> 32) + (old + wl < old);
            if (h)
                atomicAdd(&sh.hi[b], h);
            atomicAdd(&sh.cnt[b], 1u);
        });
        cluster.sync();
        // this CTA's range of the bins, added up over the cluster
        const int per = (kBins + C - 1) / C, b0 = rank * per;
        const int b1 = b0 + per < kBins ? b0 + per : kBins;
        for (int b = b0 + tid; b < b1; b += kNT) {
            unsigned long long m = 0;
            uint32_t n = 0;
            for (int r = 0; r < C; ++r) {
                m += ((unsigned long long)cluster.map_shared_rank(sh.hi, r)[b] << 32) +
                     cluster.map_shared_rank(sh.lo, r)[b];
                n += cluster.map_shared_rank(sh.cnt, r)[b];
            }
            sh.lo[b] = (uint32_t)m;
            sh.hi[b] = (uint32_t)(m >> 32);
            sh.cnt[b] = n;
        }
        __syncthreads();
    }

    // exclusive prefixes over the CTA's threads of (mass, count); totals returned in m, n
    __device__ void scan(unsigned long long& m, uint32_t& n, unsigned long long& before_m,
                         uint32_t& before_n) {
        unsigned long long im = m;
        uint32_t in = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long pm = __shfl_up_sync(kAllLanes, im, o);
            const uint32_t pn = __shfl_up_sync(kAllLanes, in, o);
            if (lane >= o) {
                im += pm;
                in += pn;
            }
        }
        __syncthreads();
        if (lane == 31) {
            sh.warp_mass[warp] = im;
            sh.warp_cnt[warp] = in;
        }
        __syncthreads();
        before_m = im - m;
        before_n = in - n;
        m = 0;
        n = 0;
        for (int w = 0; w < kNW; ++w) {
            if (w < warp) {
                before_m += sh.warp_mass[w];
                before_n += sh.warp_cnt[w];
            }
            m += sh.warp_mass[w];
            n += sh.warp_cnt[w];
        }
    }

    struct Search {
        unsigned long long above_mass;  // of the entries above the searched range
        uint32_t above_count;
        uint32_t k;            // count to reach, 0: none
        double top_p;          // >= 1: none
        unsigned long long p;  // mass to reach (from top_p when `whole`)
        int limit_bin;         // bin of the min-p limit, kBins: none
        bool draw;             // p is a mass to exceed: u E
    };

    // Finds, for each condition, the bin where it ends, in every CTA's `found`;
    // returns the range's totals.
    __device__ void search(Search& s, bool whole, unsigned long long& total, uint32_t& total_n) {
        const int per = (kBins + C - 1) / C, b0 = rank * per;
        const int b1 = b0 + per < kBins ? b0 + per : kBins;
        const int q = (per + kNT - 1) / kNT;
        const int t0 = b0 + tid * q, t1 = t0 + q < b1 ? t0 + q : b1;
        unsigned long long m = 0, before_m;
        uint32_t n = 0, before_n;
        for (int b = t0; b < t1; ++b) {
            m += ((unsigned long long)sh.hi[b] << 32) + sh.lo[b];
            n += sh.cnt[b];
        }
        scan(m, n, before_m, before_n);
        if (tid < C) {
            *cluster.map_shared_rank(&sh.part_mass[rank], tid) = m;
            *cluster.map_shared_rank(&sh.part_cnt[rank], tid) = n;
        }
        cluster.sync();
        total = 0;
        total_n = 0;
        before_m += s.above_mass;
        before_n += s.above_count;
        for (int r = 0; r < C; ++r) {
            if (r < rank) {
                before_m += sh.part_mass[r];
                before_n += sh.part_cnt[r];
            }
            total += sh.part_mass[r];
            total_n += sh.part_cnt[r];
        }
        if (whole && s.top_p < 1.0)
            s.p = ceil_scaled(s.top_p, total);
        const bool by_mass = s.draw || s.top_p < 1.0;
        for (int b = t0; b < t1; ++b) {
            Found f;
            f.bin = b;
            f.count = sh.cnt[b];
            f.mass = ((unsigned long long)sh.hi[b] << 32) + sh.lo[b];
            f.above_count = before_n;
            f.above_mass = before_m;
            before_n += f.count;
            before_m += f.mass;
            if (s.k && f.above_count < s.k && before_n >= s.k)
                tell(kByCount, f);
            if (by_mass && (s.draw ? f.above_mass <= s.p && before_m > s.p
                                   : f.above_mass < s.p && before_m >= s.p))
                tell(kByMass, f);
            if (b == s.limit_bin)
                tell(kByLimit, f);
        }
        cluster.sync();
    }

    __device__ void tell(int cond, const Found& f) {
        for (int r = 0; r < C; ++r)
            *cluster.map_shared_rank(&sh.found[cond], r) = f;
    }

    // the condition that ends first
    __device__ Found first() const {
        Found f = sh.found[0];
        for (int c = 1; c < kConds; ++c)
            if (sh.found[c].bin < f.bin)
                f = sh.found[c];
        return f;
    }

    // the largest key with bin >= b (or the smallest with bin <= b): bins fall as keys grow
    __device__ uint32_t key_at(int b, bool largest) const {
        uint32_t lo = kKeyMinusInf + 1, hi = logit_key(scale.lmax);
        while (lo < hi) {
            if (largest) {
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                if (bin_of(key_logit(mid)) >= b)
                    lo = mid;
                else
                    hi = mid - 1;
            } else {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (bin_of(key_logit(mid)) <= b)
                    hi = mid;
                else
                    lo = mid + 1;
            }
        }
        return lo;
    }

    // Narrows the entries of found bin f to a key range [klo, khi] that fits
    // the list, or is a single key.
    __device__ void narrow(Search s, Found& f, uint32_t limit_key, uint32_t& klo, uint32_t& khi,
                           bool& split) {
        khi = key_at(f.bin, true);
        klo = key_at(f.bin, false);
        while (f.count > kList && klo != khi) {
            split = true;
            int sh_ = 0;
            while (((khi - klo) >> sh_) >= (uint32_t)kBins)
                ++sh_;
            const uint32_t top = khi, bottom = klo;
            cluster.sync();  // everyone has read `found`
            histogram([&](float l) {
                const uint32_t k = logit_key(l);
                return k <= top && k >= bottom ? (int)((top - k) >> sh_) : -1;
            });
            s.above_mass = f.above_mass;
            s.above_count = f.above_count;
            s.limit_bin = kBins;
            if (!s.draw && limit_key >= bottom && limit_key <= top)
                s.limit_bin = (int)((top - limit_key) >> sh_);
            unsigned long long m;
            uint32_t n;
            search(s, false, m, n);
            const Found g = first();  // a condition that ends in a range ends in a part of it
            f = g;
            khi = top - ((uint32_t)g.bin << sh_);
            const uint32_t low = sh_ ? khi - ((1u << sh_) - 1) : khi;
            klo = low > bottom && low <= khi ? low : bottom;
        }
    }

    // The lists lie over the bins and places, which are done with when they are made.
    __device__ __forceinline__ unsigned long long* list_at(int which) const {
        return which ? reinterpret_cast<unsigned long long*>(sh.lo) : sh.list;
    }

    __device__ __forceinline__ void offer(uint32_t* n, unsigned long long* list, float l, uint32_t id) const {
        const uint32_t at = atomicAdd(n, 1u);
        if (at < (uint32_t)kList)
            list[at] = ((unsigned long long)logit_key(l) << 32) | ~id;
    }

    // Sorts a list of this CTA: descending logits, ascending ids.
    __device__ void sort(int which) {
        unsigned long long* list = list_at(which);
        if (tid == 0 && sh.list_n[which] > (uint32_t)kList)
            sh.list_n[which] = kList;
        __syncthreads();
        const int n = (int)sh.list_n[which];
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

    // Entries with klo <= key <= khi into the first CTA's list, sorted there.
    __device__ void gather(uint32_t klo, uint32_t khi) {
        cluster.sync();  // everyone has read `found`
        if (rank == 0 && tid == 0)
            sh.list_n[0] = 0;
        cluster.sync();
        uint32_t* n = cluster.map_shared_rank(&sh.list_n[0], 0);
        unsigned long long* list = cluster.map_shared_rank(sh.list, 0);
        each([&](float l, uint32_t id) {
            const uint32_t k = logit_key(l);
            if (k >= klo && k <= khi)
                offer(n, list, l, id);
        });
        cluster.sync();
        if (rank == 0)
            sort(0);
    }

    // weights of this thread's entries of a list, what lies before them and in all
    __device__ void list_scan(int which, unsigned long long w[kOwn], unsigned long long& before,
                              unsigned long long& total) {
        unsigned long long m = 0, bm;
        uint32_t n = 0, bn;
        for (int j = 0; j < kOwn; ++j) {
            const int i = kOwn * tid + j;
            w[j] = i < (int)sh.list_n[which]
                       ? weight_fixed(scale, sh.pow2, key_logit((uint32_t)(list_at(which)[i] >> 32)))
                       : 0;
            m += w[j];
        }
        scan(m, n, bm, bn);
        before = bm;
        total = m;
    }

    // The last group of equal logits in the first list that every filter keeps
    // (first CTA): the cut, the kept mass and count.  Returns 1 when the cut lies in
    // the list: some filter ends with it, `low` being the lowest key it covers; 0 when it
    // does not; 2 when sums off by up to `slack` do not tell.
    __device__ int cut_in_list(const Search& s, const Found& f, uint32_t limit_key, uint32_t low,
                               unsigned long long slack) {
        const int n = (int)sh.list_n[0];
        unsigned long long w[kOwn], before, total;
        list_scan(0, w, before, total);
        unsigned long long at = f.above_mass + before;
        int last = -1;
        bool near = false;
        for (int j = 0; j < kOwn; ++j) {
            const int i = kOwn * tid + j;
            if (i < n) {
                const uint32_t k = (uint32_t)(sh.list[i] >> 32);
                const bool start = i == 0 || (uint32_t)(sh.list[i - 1] >> 32) != k;
                if (start && k >= limit_key && (!s.k || f.above_count + i < s.k)) {
                    if (s.top_p >= 1.0 || at < s.p)
                        last = i;
                    if (s.top_p < 1.0 && f.above_count + i > 0 && (at < s.p ? s.p - at : at - s.p) < slack)
                        near = true;
                }
            }
            at += w[j];
        }
        // conditions fail for good once they fail: the last start over all threads
        last = __reduce_max_sync(kAllLanes, last);
        const bool any_near = __syncthreads_or(near);
        if (lane == 0)
            sh.warp_max[warp] = (uint32_t)(last + 1);
        __syncthreads();
        int g = 0;
        for (int i = 0; i < kNW; ++i)
            g = (int)sh.warp_max[i] > g ? (int)sh.warp_max[i] : g;
        --g;  // -1: nothing of the list is kept
        const uint32_t key = g >= 0 ? (uint32_t)(sh.list[g] >> 32) : limit_key;
        unsigned long long at2 = f.above_mass + before;
        if (tid == 0 && g < 0) {
            sh.cut_key = key;
            sh.kept = f.above_count;
            sh.kept_mass = f.above_mass;
        }
        for (int j = 0; j < kOwn; ++j) {
            const int i = kOwn * tid + j;
            at2 += w[j];
            if (g >= 0 && i < n && (uint32_t)(sh.list[i] >> 32) == key &&
                (i == n - 1 || (uint32_t)(sh.list[i + 1] >> 32) != key)) {
                sh.cut_key = key;
                sh.kept = f.above_count + i + 1;
                sh.kept_mass = at2;
            }
        }
        __syncthreads();
        if (any_near)
            return 2;
        if ((s.k && f.above_count >= s.k) || (s.top_p < 1.0 && f.above_count && f.above_mass >= s.p))
            return 0;
        if (limit_key >= low || (s.k && f.above_count + (uint32_t)n >= s.k))
            return 1;
        if (s.top_p >= 1.0 || f.above_mass + total + slack < s.p)
            return 0;
        return f.above_mass + total >= s.p + slack ? 1 : 2;
    }

    // what the first CTA has found, to the others
    __device__ void share_cut() {
        if (rank == 0 && tid > 0 && tid < C) {
            *cluster.map_shared_rank(&sh.cut_key, tid) = sh.cut_key;
            *cluster.map_shared_rank(&sh.kept, tid) = sh.kept;
            *cluster.map_shared_rank(&sh.kept_mass, tid) = sh.kept_mass;
            *cluster.map_shared_rank(&sh.ok, tid) = sh.ok;
        }
        cluster.sync();
    }

    // The first entry of a list whose running sum exceeds `target` (first CTA);
    // whether the list holds it.
    __device__ bool draw_in_list(int which, unsigned long long above_mass, unsigned long long target) {
        const int n = (int)sh.list_n[which];
        unsigned long long w[kOwn], at, total;
        list_scan(which, w, at, total);
        at += above_mass;
        for (int j = 0; j < kOwn; ++j) {
            const int i = kOwn * tid + j;
            if (i < n && at <= target && at + w[j] > target) {
                sh.token = ~(uint32_t)list_at(which)[i];
                sh.token_key = (uint32_t)(list_at(which)[i] >> 32);
            }
            at += w[j];
        }
        __syncthreads();
        return above_mass <= target && above_mass + total > target;
    }

    // The entry number r, by ascending id, among those with this key.
    __device__ void draw_among_equals(uint32_t key, unsigned long long r) {
        const uint32_t per = (s1 - s0 + kNT - 1) / kNT;
        const uint32_t e0 = min(s0 + tid * per, s1), e1 = min(e0 + per, s1);
        uint32_t n = 0, before;
        unsigned long long m = 0, bm;
        for (uint32_t e = e0; e < e1; ++e)
            n += logit_key(scalar_entry<ES>(base, e)) == key;
        const uint32_t mine = n;
        scan(m, n, bm, before);
        cluster.sync();
        if (tid < C)
            *cluster.map_shared_rank(&sh.part_cnt[rank], tid) = n;
        cluster.sync();
        for (int c = 0; c < rank; ++c)
            before += sh.part_cnt[c];
        if (r >= before && r < (unsigned long long)before + mine) {
            uint32_t left = (uint32_t)(r - before);
            for (uint32_t e = e0; e < e1; ++e)
                if (logit_key(scalar_entry<ES>(base, e)) == key && left-- == 0) {
                    *cluster.map_shared_rank(&sh.token, 0) = e;
                    *cluster.map_shared_rank(&sh.token_key, 0) = key;
                    break;
                }
        }
        cluster.sync();
    }

    // Probabilities and truncated logits; keep(l, id) says what stays.  A vector
    // none of whose logits reaches `cut` is written without looking further.
    template <class Keep>
    __device__ void write(Keep&& keep, float cut, float inv, bool bad) {
        const float nan = __int_as_float(0x7fffffff);
        const auto prob = [&](float l, uint32_t id) {
            return bad ? nan : keep(l, id) ? (inv > 0.0f ? weight_float(scale, l) * inv : 1.0f) : 0.0f;
        };
        const auto logit = [&](float l, uint32_t id) {
            return bad || keep(l, id) ? __float_as_uint(l) : 0xff800000u;
        };
        float* p = a.probs ? a.probs + row * a.probs_stride : nullptr;
        unsigned char* o = a.out ? static_cast<unsigned char*>(a.out) + row * a.out_stride * ES : nullptr;
        if (!p && !o)
            return;
        const auto one = [&](uint32_t id) {
            const float l = scalar_entry<ES>(base, id);
            if (p)
                p[id] = prob(l, id);
            if (o) {
                const uint32_t h = logit(l, id);
                if constexpr (ES == 4)
                    reinterpret_cast<uint32_t*>(o)[id] = h;
                else
                    reinterpret_cast<unsigned short*>(o)[id] = (unsigned short)(h >> 16);
            }
        };
        // vectors of logits go to 16-byte places of both outputs, or are written one by one
        const bool even = (!p || (reinterpret_cast<uintptr_t>(p - off) & 15u) == 0) &&
                          (!o || (reinterpret_cast<uintptr_t>(o - off * ES) & 15u) == 0);
        if (!even) {
            for (uint32_t i = s0 + tid; i < s1; i += kNT)
                one(i);
            return;
        }
        walk<4>(
            [&](const uint4& w, uint32_t id) {
                float m = vector_entry<ES>(w, 0);
#pragma unroll
                for (int e = 1; e < E; ++e)
                    m = fmaxf(m, vector_entry<ES>(w, e));
                const bool any = bad || m >= cut;
                if (p) {
                    float4* q = reinterpret_cast<float4*>(p + id);
                    if (!any) {
#pragma unroll
                        for (int e = 0; e < E / 4; ++e)
                            q[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    } else {
#pragma unroll
                        for (int e = 0; e < E / 4; ++e)
                            q[e] = make_float4(prob(vector_entry<ES>(w, 4 * e), id + 4 * e),
                                               prob(vector_entry<ES>(w, 4 * e + 1), id + 4 * e + 1),
                                               prob(vector_entry<ES>(w, 4 * e + 2), id + 4 * e + 2),
                                               prob(vector_entry<ES>(w, 4 * e + 3), id + 4 * e + 3));
                    }
                }
                if (o) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (ES == 4)
                            h[j] = any ? logit(vector_entry<ES>(w, j), id + j) : 0xff800000u;
                        else
                            h[j] = any ? (logit(vector_entry<ES>(w, 2 * j), id + 2 * j) >> 16) |
                                             (logit(vector_entry<ES>(w, 2 * j + 1), id + 2 * j + 1) & 0xffff0000u)
                                       : 0xff80ff80u;
                    }
                    *reinterpret_cast<uint4*>(o + (size_t)id * ES) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            },
            one);
    }

    // -------------------------------------------------------- by places -----

    // the logit of least magnitude at place D (bfloat16: the only one)
    __device__ __forceinline__ static float place_value(int D) {
        const int s = kMags + 1 - D, i = s >= 0 ? s : -1 - s;
        const uint32_t b = i ? (uint32_t)(kMag0 - 1 + i) : 0u;
        return __uint_as_float((b | (s < 0 ? 0x8000u : 0u)) << 16);
    }

    // the place of a logit
    __device__ __forceinline__ static int place_of(float l) {
        const uint32_t b = __float_as_uint(l);
        const int m = (int)((b & 0x7fffffffu) >> 16);
        const int i = min(max(m, kMag0 - 1), kMag0 + kMags) - (kMag0 - 1);
        return kMags + 1 - ((b >> 31) ? -1 - i : i);
    }

    // a float32 place's largest or smallest logit; inside the window
    __device__ __forceinline__ static float place_end(int D, bool largest) {
        const float l = place_value(D);
        return largest == (l > 0.0f) ? __uint_as_float(__float_as_uint(l) | 0xffffu) : l;
    }

    // weight of the logits at place D: bfloat16 exactly, float32 by its middle
    __device__ __forceinline__ unsigned long long place_weight(int D) const {
        float l = place_value(D);
        if constexpr (ES == 4)
            l = fminf(__uint_as_float(__float_as_uint(l) | 0x8000u), scale.lmax);
        return weight_fixed(scale, sh.pow2, l);
    }

    // Counts the two logits whose upper 16 bits x holds.  Each place's byte
    // offset is 4 i or 4 (-1 - i), both logits' in the halves of one word.
    // Logits above -127 alone are counted: what is missing lies below.
    __device__ __forceinline__ void count_pair(uint32_t x) {
        constexpr uint32_t lo = (kMag0 - 1) * 0x10001u, hi = (kMag0 + kMags) * 0x10001u;
        constexpr int far = 4 * (-1 - (kMags + 1));
        const uint32_t m = x & 0x7fff7fffu;
        uint32_t sign, i;
        asm("max.u16x2 %0, %1, %2;" : "=r"(i) : "r"(m), "r"(lo));
        asm("min.u16x2 %0, %1, %2;" : "=r"(i) : "r"(i), "r"(hi));
        asm("prmt.b32 %0, %1, %2, %3;" : "=r"(sign) : "r"(x), "r"(0u), "r"(0xbb99u));  // sign of each half
        const uint32_t o = (((i - lo) << 2) ^ sign) & 0xfffcfffcu;
        const int o0 = (int)(short)(o & 0xffffu), o1 = (int)o >> 16;
        char* zero = reinterpret_cast<char*>(sh.count + kMags + 2);
        if (o0 != far)
            atomicAdd(reinterpret_cast<uint32_t*>(zero + o0), 1u);
        if (o1 != far)
            atomicAdd(reinterpret_cast<uint32_t*>(zero + o1), 1u);
    }

    // entries at N places, over the cluster
    template <int N>
    __device__ __forceinline__ void place_counts(const int (&D)[N], uint32_t (&n)[N]) const {
#pragma unroll
        for (int j = 0; j < N; ++j)
            n[j] = 0;
        for (int r = 0; r < C; ++r) {
            const uint32_t* count = cluster.map_shared_rank(sh.count, r);
            uint32_t x[N];
#pragma unroll
            for (int j = 0; j < N; ++j)
                x[j] = count[kPlaces - 1 - D[j]];
#pragma unroll
            for (int j = 0; j < N; ++j)
                n[j] += x[j];
        }
    }
    __device__ __forceinline__ uint32_t place_count(int D) const {
        const int d[1] = {D};
        uint32_t n[1];
        place_counts<1>(d, n);
        return n[0];
    }

    struct Wanted {
        uint32_t k;            // count to reach, 0: none
        unsigned long long p;  // mass to reach, 0: none; with `draw` a mass to exceed
        int limit;             // the last place min-p keeps, kNoPlace: none
        bool draw;
    };

    // Finds the places where the conditions end, in every CTA's `place[set]`, and
    // returns the first.  The thread whose chunk of places holds one hands it to a warp,
    // which goes through the chunk; m, n: the chunk's sums, before_m, before_n: what
    // lies above it.
    __device__ Found search_places(int set, const Wanted& s, int chunk, unsigned long long m, uint32_t n,
                                   unsigned long long before_m, uint32_t before_n) {
        const auto hit = [&](int c) {
            sh.hit[set][c].chunk = chunk;
            sh.hit[set][c].above_mass = before_m;
            sh.hit[set][c].above_count = before_n;
        };
        if (chunk >= 0) {
            if (s.k && before_n < s.k && before_n + n >= s.k)
                hit(kByCount);
            if (s.draw ? before_m <= s.p && before_m + m > s.p
                       : s.p && before_m < s.p && before_m + m >= s.p)
                hit(kByMass);
            if (s.limit / 32 == chunk)
                hit(kByLimit);
        }
        __syncthreads();
        if (warp < kConds && sh.hit[set][warp].chunk >= 0) {
            const int D = sh.hit[set][warp].chunk * 32 + lane;
            Found f;
            f.bin = D;
            f.count = place_count(D);
            f.mass = f.count ? f.count * place_weight(D) : 0;
            unsigned long long im = f.mass;
            uint32_t in = f.count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long pm = __shfl_up_sync(kAllLanes, im, o);
                const uint32_t pn = __shfl_up_sync(kAllLanes, in, o);
                if (lane >= o) {
                    im += pm;
                    in += pn;
                }
            }
            f.above_mass = sh.hit[set][warp].above_mass + im - f.mass;
            f.above_count = sh.hit[set][warp].above_count + in - f.count;
            const unsigned long long em = f.above_mass + f.mass;
            const uint32_t en = f.above_count + f.count;
            const bool here = warp == kByCount ? f.above_count < s.k && en >= s.k
                              : warp == kByLimit ? D == s.limit
                              : s.draw ? f.above_mass <= s.p && em > s.p
                                       : f.above_mass < s.p && em >= s.p;
            if (here)
                for (int r = 0; r < C; ++r)
                    *cluster.map_shared_rank(&sh.place[set][warp], r) = f;
        }
        cluster.sync();
        Found f = sh.place[set][0];
        for (int c = 1; c < kConds; ++c)
            if (sh.place[set][c].bin < f.bin)
                f = sh.place[set][c];
        return f;
    }

    // which of a vector's eight logits equal the bits `two` holds twice
    __device__ __forceinline__ static uint32_t matches(const uint4& w, uint32_t two) {
        const uint32_t x[4] = {w.x ^ two, w.y ^ two, w.z ^ two, w.w ^ two};
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            mask |= ((x[j] & 0xffffu) == 0 ? 1u << (2 * j) : 0u) | ((x[j] >> 16) == 0 ? 2u << (2 * j) : 0u);
        return mask;
    }

    // The entry number r by ascending id at place D (bfloat16); the CTA that holds it
    // returns its id in one thread, every other thread returns -1.  Each warp
    // counts in a stretch of the slice, then the warp that holds the entry looks again.
    __device__ int64_t find(int D, unsigned long long r) {
        uint32_t n = 0, in;
        if (lane < C)
            n = cluster.map_shared_rank(sh.count, lane)[kPlaces - 1 - D];
        in = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t p = __shfl_up_sync(kAllLanes, in, o);
            if (lane >= o)
                in += p;
        }
        const uint32_t owners = __ballot_sync(kAllLanes, r >= in - n && r < in);
        if (!owners || __ffs(owners) - 1 != rank)
            return -1;
        uint32_t left = (uint32_t)(r - __shfl_sync(kAllLanes, in - n, rank));
        const uint32_t bits = __float_as_uint(place_value(D)) >> 16, two = bits * 0x10001u;
        const unsigned short* q = reinterpret_cast<const unsigned short*>(base);
        // what lies before the first vector: less than one
        for (uint32_t i = s0; i < head_end(); ++i)
            if (q[i] == bits && left-- == 0)
                return tid == 0 ? (int64_t)i : -1;
        constexpr int L = 8;
        const uint4* p = vectors();
        const uint32_t per = (k1 - k0 + kNW - 1) / kNW;
        const uint32_t g0 = min(k0 + warp * per, k1), g1 = min(g0 + per, k1);
        uint32_t mine = 0;
        for (uint32_t g = g0 + lane; g < g1; g += 32 * L) {
            uint4 w[L];
#pragma unroll
            for (int j = 0; j < L; ++j)
                if (g + 32 * j < g1)
                    w[j] = load_stream(p + g + 32 * j);
#pragma unroll
            for (int j = 0; j < L; ++j)
                if (g + 32 * j < g1)
                    mine += __popc(matches(w[j], two));
        }
        mine = __reduce_add_sync(kAllLanes, mine);
        __syncthreads();
        if (lane == 0)
            sh.warp_cnt[warp] = mine;
        __syncthreads();
        int holder = -1;
        for (int w = 0; w < kNW; ++w) {
            if (left < sh.warp_cnt[w]) {
                holder = w;
                break;
            }
            left -= sh.warp_cnt[w];
        }
        if (holder < 0) {
            if (tid == 0)
                for (uint32_t i = tail_start(); i < s1; ++i)
                    if (q[i] == bits && left-- == 0)
                        return i;
            return -1;
        }
        if (holder != warp)
            return -1;
        for (uint32_t b = g0; b < g1; b += 32 * L) {
            uint32_t mask[L];
            uint4 w[L];
#pragma unroll
            for (int j = 0; j < L; ++j)
                if (b + lane + 32 * j < g1)
                    w[j] = load_stream(p + b + lane + 32 * j);
#pragma unroll
            for (int j = 0; j < L; ++j)
                mask[j] = b + lane + 32 * j < g1 ? matches(w[j], two) : 0;
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const uint32_t c = __popc(mask[j]), all = __reduce_add_sync(kAllLanes, c);
                if (left >= all) {
                    left -= all;
                    continue;
                }
                uint32_t ic = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(kAllLanes, ic, o);
                    if (lane >= o)
                        ic += x;
                }
                if (left >= ic - c && left < ic)
                    return (int64_t)(b + lane + 32 * j) * E - off + __fns(mask[j], 0, left - (ic - c) + 1);
                return -1;
            }
        }
        return -1;
    }

    // A stretch of places around one of interest, as far as the list holds its
    // entries: lane r looks at r places to either side.
    struct Band {
        bool on, from_top;
        float lo, hi;          // its logits
        uint32_t above_count;  // entries above it
    };
    __device__ Band band_around(const Found& f) const {
        Band b;
        const int D = f.bin - 16 + lane;
        const uint32_t n = place_count(D >= 1 && D <= kPlaces - 2 ? D : kPlaces - 1);  // the last: not counted, 0
        uint32_t in = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t p = __shfl_up_sync(kAllLanes, in, o);
            if (lane >= o)
                in += p;
        }
        const int r = lane & 15;
        const uint32_t upto = __shfl_sync(kAllLanes, in, 16 + r);
        const uint32_t over = __shfl_sync(kAllLanes, in - n, 16 - r);  // above the stretch, of these
        const uint32_t mid = __shfl_sync(kAllLanes, in - n, 16);
        const uint32_t whole = __ballot_sync(kAllLanes, f.above_count + (upto - mid) <= (uint32_t)kList) & 0xffffu;
        const uint32_t part = __ballot_sync(kAllLanes, upto - over <= (uint32_t)kList) & 0xffffu;
        b.from_top = whole != 0;
        b.on = (whole | part) != 0;
        if (!b.on)
            return b;
        const int reach = 31 - __clz(whole ? whole : part);
        const int first = whole ? 1 : max(f.bin - reach, 1), last = min(f.bin + reach, kPlaces - 2);
        b.above_count = whole ? 0 : f.above_count - (mid - __shfl_sync(kAllLanes, over, reach));
        b.hi = whole ? scale.lmax : place_end(first, true);
        b.lo = place_end(last, false);
        // the two places below the window hold +0 and -0, which are one logit
        if (first == kFirstTiny + 1 || first == kFirstTiny || last == kFirstTiny || last == kFirstTiny + 1)
            b.on = false;
        return b;
    }

    // sums over the cluster of three integers of every thread
    __device__ void sum3(unsigned long long (&x)[3]) {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            unsigned long long v = x[j];
            uint32_t n = 0, bn;
            unsigned long long bv;
            scan(v, n, bv, bn);
            if (tid < C)
                *cluster.map_shared_rank(&sh.sums[j][rank], tid) = v;
        }
        cluster.sync();
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            x[j] = 0;
            for (int r = 0; r < C; ++r)
                x[j] += sh.sums[j][r];
        }
    }

    // The whole call for a row whose answer does not depend on logits outside the
    // window of places; false (in every CTA) for the others.
    //
    // bfloat16: the places' sums are exact, and so are the cut and the draw.
    // float32: they place the cut and the draw to within a few places.  A second
    // pass takes the sums of the row and of what lies above the two stretches of
    // places around them, and lists the stretches' entries, among which the exact cut and
    // draw are found; where a stretch turns out not to hold them, the row is left to
    // the general way.  Few entries above the cut are listed whole, and need no
    // sum but the row's for top-p: it is taken in floats, to 2^-17, and where an entry
    // lies nearer to top-p's border than that, once more in integers.
    __device__ bool by_place(float T, int32_t top_k, double top_p, double min_p, float u) {
        {
            uint4* z = reinterpret_cast<uint4*>(sh.count);
            for (int i = tid; i < kPlaces / 4; i += kNT)
                z[i] = make_uint4(0, 0, 0, 0);
            if (tid < 2)
                sh.list_n[tid] = 0;
            if (tid < 2 * kConds) {
                sh.hit[tid / kConds][tid % kConds].chunk = -1;
                sh.place[tid / kConds][tid % kConds].bin = kNoPlace;
            }
        }
        __syncthreads();
        float lmax = __int_as_float(0xff800000);
        uint32_t two = 0xff80ff80u;  // bfloat16: the largest of each half
        walk<4>(
            [&](const uint4& w, uint32_t) {
                if constexpr (ES == 2) {
                    count_pair(w.x);
                    count_pair(w.y);
                    count_pair(w.z);
                    count_pair(w.w);
                    uint32_t m, x;
                    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(w.x), "r"(w.y));
                    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w.z), "r"(w.w));
                    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(x));
                    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(two) : "r"(two), "r"(m));
                } else {
                    count_pair(__byte_perm(w.x, w.y, 0x7632));
                    count_pair(__byte_perm(w.z, w.w, 0x7632));
                    lmax = max_nan(max_nan(lmax, __uint_as_float(w.x)), __uint_as_float(w.y));
                    lmax = max_nan(max_nan(lmax, __uint_as_float(w.z)), __uint_as_float(w.w));
                }
            },
            [&](uint32_t id) {  // a lone logit, paired with -inf, which is not counted
                const float l = scalar_entry<ES>(base, id);
                count_pair((__float_as_uint(l) >> 16) | 0xff800000u);
                lmax = max_nan(lmax, l);
            });
        if constexpr (ES == 2)
            lmax = max_nan(lmax, max_nan(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u)));
        // the largest key; above all of them: a NaN
        uint32_t key = lmax == lmax ? logit_key(lmax) : 0xffffffffu;
        key = __reduce_max_sync(kAllLanes, key);
        if (lane == 0)
            sh.warp_max[warp] = key;
        __syncthreads();
        for (int w = 0; w < kNW; ++w)
            key = max(key, sh.warp_max[w]);
        meet();
        if (tid < C) {
            *cluster.map_shared_rank(&sh.part_max[rank], tid) = key;
            *cluster.map_shared_rank(&sh.part_tiny[rank], tid) = sh.count[kMags + 1] + sh.count[kMags + 2];
        }
        cluster.sync();
        uint32_t tiny = 0;  // entries below the window
        for (int r = 0; r < C; ++r) {
            key = max(key, sh.part_max[r]);
            tiny += sh.part_tiny[r];
        }
        scale.lmax = key_logit(key);
        const int D0 = place_of(scale.lmax);
        if (key == 0xffffffffu || D0 < 1 || D0 > kPlaces - 2 || D0 == kFirstTiny || D0 == kFirstTiny + 1)
            return false;
        if (T == 0.0f) {
            if constexpr (ES == 4)
                return false;
            const int64_t id = find(D0, 0);
            if (id >= 0) {
                a_token(id, 1.0f);
                for (int r = 0; r < C; ++r)
                    *cluster.map_shared_rank(&sh.token, r) = (uint32_t)id;
            }
            if (a.probs || a.out) {
                cluster.sync();
                const uint32_t token = sh.token;
                write([=](float, uint32_t i) { return i == token; }, scale.lmax, 0.0f, false);
            }
            finish(SV_OK, 1, 1.0f);
            return true;
        }
        split_scale(T, scale.ch, scale.cl);
        // logits from -127 down must weigh nothing
        if (!((scale.lmax + 127.0f) * scale.ch >= 61.0f))
            return false;
        // bfloat16 logits below the window are taken for 0: their weights are off by
        // 2^-24/T of themselves, which must not show in the sum (>= 1 at l_max)
        if (ES == 2 && tiny && (float)tiny * weight_float(scale, 0.0f) > T * 3.0517578e-5f) {  // 2^-39 / 2^-24
            // unless they are zeros
            bool other = false;
            each([&](float l, uint32_t) { other = other || (l != 0.0f && fabsf(l) < 2.9802322e-8f); });
            const uint32_t any = __syncthreads_or(other);
            cluster.sync();  // everyone has read `part_tiny`
            if (tid < C)
                *cluster.map_shared_rank(&sh.part_tiny[rank], tid) = any;
            cluster.sync();
            for (int r = 0; r < C; ++r)
                if (sh.part_tiny[r])
                    return false;
        }

        // sums of each chunk of places, a chunk per warp
        const int per = (kChunks + C - 1) / C;
        const int c0 = min(rank * per, kChunks), c1 = min(c0 + per, kChunks);
        constexpr int L = 4;
        for (int c = c0 + warp; c < c1; c += L * kNW) {
            int D[L];
            uint32_t n[L];
#pragma unroll
            for (int j = 0; j < L; ++j)
                D[j] = min(c + j * kNW, kChunks - 1) * 32 + lane;
            place_counts<L>(D, n);
#pragma unroll
            for (int j = 0; j < L; ++j) {
                if (c + j * kNW >= c1)
                    break;
                unsigned long long m = 0;
                uint32_t all = 0;
                if (__any_sync(kAllLanes, n[j])) {
                    if (n[j])
                        m = n[j] * place_weight(D[j]);
                    all = __reduce_add_sync(kAllLanes, n[j]);
                    // 62 bits in three parts, so that the lanes' sums fit 32
                    m = (unsigned long long)__reduce_add_sync(kAllLanes, (uint32_t)m & 0x1fffffu) +
                        ((unsigned long long)__reduce_add_sync(kAllLanes, (uint32_t)(m >> 21) & 0x1fffffu) << 21) +
                        ((unsigned long long)__reduce_add_sync(kAllLanes, (uint32_t)(m >> 42)) << 42);
                }
                if (lane == 0) {
                    sh.chunk_mass[c + j * kNW - c0] = m;
                    sh.chunk_cnt[c + j * kNW - c0] = all;
                }
            }
        }
        __syncthreads();
        static_assert(kChunks <= kNT, "a thread per chunk");
        const bool has = tid < c1 - c0;
        const unsigned long long m = has ? sh.chunk_mass[tid] : 0;
        const uint32_t n = has ? sh.chunk_cnt[tid] : 0;
        unsigned long long tm = m, before_m, whole = 0;
        uint32_t tn = n, before_n, near = 0;
        scan(tm, tn, before_m, before_n);
        if (tid < C) {
            *cluster.map_shared_rank(&sh.part_mass[rank], tid) = tm;
            *cluster.map_shared_rank(&sh.part_cnt[rank], tid) = tn;
        }
        cluster.sync();
        for (int r = 0; r < C; ++r) {
            if (r < rank) {
                before_m += sh.part_mass[r];
                before_n += sh.part_cnt[r];
            }
            whole += sh.part_mass[r];
            near += sh.part_cnt[r];
        }
        const int chunk = has ? c0 + tid : -1;

        // the cut
        Wanted s;
        s.k = top_k > 0 ? (uint32_t)top_k : 0;
        s.p = top_p < 1.0 ? ceil_scaled(top_p, whole) : 0;
        s.limit = kNoPlace;
        s.draw = false;
        uint32_t limit_key = 0;
        if (min_p > 0.0) {
            // the smallest float l with l - l_max >= T ln(min_p); bfloat16: the smallest of those
            float limit = __double2float_ru((double)scale.lmax + (double)T * log(min_p));
            limit_key = logit_key(limit);
            if (ES == 2 && limit > 0.0f && (__float_as_uint(limit) & 0xffffu))
                limit = __uint_as_float((__float_as_uint(limit) & 0xffff0000u) + 0x10000u);
            s.limit = place_of(limit);
            if (s.limit < 1 || s.limit > kPlaces - 2 || s.limit == kFirstTiny || s.limit == kFirstTiny + 1)
                return false;
        }
        Found f;
        f.bin = kNoPlace;
        if (s.k || s.p || s.limit < kNoPlace)
            f = search_places(0, s, chunk, m, n, before_m, before_n);
        unsigned long long mass = whole;  // kept
        int64_t kept = near;
        float cut = -3.402823466e38f;
        if (f.bin < kNoPlace) {
            if (f.bin == kFirstTiny || f.bin == kFirstTiny + 1)
                return false;
            mass = f.above_mass + f.mass;
            if constexpr (ES == 2) {
                kept = f.above_count + f.count;
                cut = place_value(f.bin);
            }
        } else if ((uint64_t)near < (uint64_t)a.V) {
            // everything is kept: those from -127 down that are not -inf as well
            if (s.k)
                return false;
            uint32_t more = 0;
            each([&](float l, uint32_t) { more += place_of(l) == kPlaces - 1 && l > __int_as_float(0xff800000); });
            more = __reduce_add_sync(kAllLanes, more);
            __syncthreads();
            if (lane == 0)
                sh.warp_cnt[warp] = more;
            __syncthreads();
            more = 0;
            for (int w = 0; w < kNW; ++w)
                more += sh.warp_cnt[w];
            cluster.sync();
            if (tid < C)
                *cluster.map_shared_rank(&sh.part_cnt[rank], tid) = more;
            cluster.sync();
            for (int r = 0; r < C; ++r)
                kept += sh.part_cnt[r];
        }
        const bool by_draw = a.u != nullptr;

        if constexpr (ES == 4) {
            Band c, d;
            c.on = c.from_top = d.on = d.from_top = false;
            c.above_count = 0;
            if (f.bin < kNoPlace) {
                c = band_around(f);
                if (!c.on)
                    return false;
            }
            // float sums will do to tell whether an entry listed whole lies above top-p's
            // border; not where they become part of the answer, or entries weigh too little
            bool fine = !c.from_top || a.mass || (s.p && place_weight(f.bin) < whole >> 15);
            if (by_draw && !c.from_top) {
                Wanted w;
                w.k = 0;
                w.limit = kNoPlace;
                w.draw = true;
                w.p = floor_scaled(u, mass);
                const Found h = search_places(1, w, chunk, m, n, before_m, before_n);
                if (!c.on || place_end(h.bin, true) > c.hi) {
                    d = band_around(h);
                    if (!d.on)
                        return false;
                }
            }
            cluster.sync();  // the lists lie over the places
            const bool sums = top_p < 1.0 || !c.on || a.mass || !c.from_top;
            uint32_t *nc = cluster.map_shared_rank(&sh.list_n[0], 0), *nd = cluster.map_shared_rank(&sh.list_n[1], 0);
            unsigned long long *lc = cluster.map_shared_rank(list_at(0), 0),
                               *ld = cluster.map_shared_rank(list_at(1), 0);
            const float inf = __int_as_float(0x7f800000);
            const float clo = c.on ? c.lo : inf, chi = c.on ? c.hi : inf;
            const float dlo = d.on ? d.lo : inf, dhi = d.on ? d.hi : inf;
            const float low = fminf(clo, dlo);
            const auto list = [&](float l, uint32_t id) {
                if (l >= clo && l <= chi)
                    offer(nc, lc, l, id);
                if (l >= dlo && l <= dhi)
                    offer(nd, ld, l, id);
            };
            unsigned long long sum[3];  // the row; above the cut's stretch; above the draw's
            unsigned long long slack = 0;
            bool listed = false;
            for (;;) {
                sum[0] = sum[1] = sum[2] = 0;
                if (sums && fine) {
                    each([&](float l, uint32_t id) {
                        const unsigned long long x = weight_fixed(scale, sh.pow2, l);
                        sum[0] += x;
                        sum[1] += l > chi ? x : 0;
                        sum[2] += l > dhi ? x : 0;
                        if (l >= low && !listed)
                            list(l, id);
                    });
                } else if (sums) {
                    const float one = (float)(1ull << scale.fix);
                    const auto fast = [&](float l) { return ex2_approx((l - scale.lmax) * scale.ch); };
                    walk<4>(
                        [&](const uint4& w, uint32_t id) {
                            float t = 0.0f, top = -inf;
#pragma unroll
                            for (int e = 0; e < E; ++e) {
                                t += fast(vector_entry<ES>(w, e));
                                top = fmaxf(top, vector_entry<ES>(w, e));
                            }
                            sum[0] += __float2ull_rn(t * one);
                            if (top >= clo) {
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    list(vector_entry<ES>(w, e), id + e);
                            }
                        },
                        [&](uint32_t id) {
                            const float l = scalar_entry<ES>(base, id);
                            sum[0] += __float2ull_rn(fast(l) * one);
                            list(l, id);
                        });
                } else {
                    each([&](float l, uint32_t id) {
                        if (l >= clo)
                            offer(nc, lc, l, id);
                    });
                }
                sum3(sum);
                whole = sum[0];
                slack = sums && !fine ? whole >> 17 : 0;
                if (rank == 0) {
                    int ok = 1;  // 0: not in the lists, 2: too near a border for these sums
                    Search q;
                    q.k = s.k;
                    q.top_p = top_p;
                    q.p = top_p < 1.0 ? ceil_scaled(top_p, whole) : 0;
                    Found g;
                    g.above_mass = sum[1];
                    g.above_count = c.above_count;
                    if (c.on) {
                        if (!listed)
                            sort(0);
                        ok = limit_key <= logit_key(c.hi) ? cut_in_list(q, g, limit_key, logit_key(c.lo), slack) : 0;
                    } else if (tid == 0) {
                        sh.kept_mass = whole;
                        sh.cut_key = kKeyMinusInf + 1;
                        sh.kept = 0;
                    }
                    __syncthreads();
                    if (ok == 1 && by_draw) {
                        const unsigned long long target = floor_scaled(u, sh.kept_mass);
                        if (c.on && target >= sum[1]) {
                            ok = draw_in_list(0, sum[1], target);
                        } else {
                            if (d.on)
                                sort(1);
                            ok = d.on && draw_in_list(1, sum[2], target);
                        }
                    }
                    if (tid == 0)
                        sh.ok = ok;
                    __syncthreads();
                }
                share_cut();
                const uint32_t ok = sh.ok;
                if (ok == 0)
                    return false;
                if (ok == 1)
                    break;
                fine = true;
                listed = true;
                cluster.sync();  // everyone has read `ok`
            }
            mass = sh.kept_mass;
            if (c.on)
                kept = sh.kept;
            cut = key_logit(sh.cut_key);
        }
        const float inv = (float)((double)(1ull << scale.fix) / (double)mass);
        if (by_draw) {
            if constexpr (ES == 2) {
                s.k = 0;
                s.limit = kNoPlace;
                s.draw = true;
                s.p = floor_scaled(u, mass);
                const Found d = search_places(1, s, chunk, m, n, before_m, before_n);
                if (d.bin == kFirstTiny || d.bin == kFirstTiny + 1)
                    return false;
                const float l = place_value(d.bin);
                const int64_t id = find(d.bin, (s.p - d.above_mass) / weight_fixed(scale, sh.pow2, l));
                if (id >= 0)
                    a_token(id, weight_float(scale, l) * inv);
            } else if (rank == 0 && tid == 0) {
                a_token(sh.token, weight_float(scale, key_logit(sh.token_key)) * inv);
            }
        }
        write([&](float l, uint32_t) { return l >= cut; }, cut, inv, false);
        finish(SV_OK, (uint32_t)kept, (float)((double)mass / (double)whole));
        return true;
    }

    // the first use of another CTA's memory waits until every CTA runs
    bool met = false;
    __device__ void meet() {
        if (!met)
            cluster.barrier_wait();
        met = true;
    }

    __device__ void a_token(int64_t id, float p) {
        if (a.tokens)
            a.tokens[row * a.token_stride] = (int32_t)id;
        if (a.p_token)
            a.p_token[row] = p;
    }

    __device__ void finish(int code, uint32_t kept, float mass) {
        if (rank == 0 && tid == 0) {
            if (a.mass)
                a.mass[row] = mass;
            if (a.kept)
                a.kept[row] = (int32_t)kept;
            if (a.status)
                a.status[row] = code;
            if (code)
                atomicOr(a.err_word, 1u << code);
        }
    }

    __device__ void run() {
        const int64_t seq = row / a.rows_per_seq;
        const float T = a.set.temperatures ? a.set.temperatures[seq] : a.set.temperature;
        const int32_t top_k = a.set.top_ks ? a.set.top_ks[seq] : a.set.top_k;
        const double top_p = a.set.top_ps ? (double)a.set.top_ps[seq] : a.set.top_p;
        const double min_p = a.set.min_ps ? (double)a.set.min_ps[seq] : a.set.min_p;
        const float u = a.u ? a.u[row * a.u_stride] : 0.0f;
        int code = SV_OK;
        if (!(T == 0.0f || (T >= 1.17549435e-38f && T <= 3.402823466e38f)) || !(top_p > 0.0) ||
            !(min_p < 1.0))
            code = SV_ERR_INVALID_ARG;
        else if (!(u >= 0.0f && u < 1.0f))
            code = SV_ERR_UNIFORM_RANGE;
        if (tid < 64)
            sh.pow2[tid] = kPow2Steps[tid];

        cluster.barrier_arrive();
        if (!code && by_place(T, top_k, top_p, min_p, u)) {
            cluster.sync();  // no CTA leaves while another may still read its memory
            return;
        }
        if (met)
            cluster.sync();  // every CTA is done with what it was told
        general(code, T, top_k, top_p, min_p, u);
    }

    // The call for any row, and for an erroneous one.
    __device__ __forceinline__ void general(int code, float T, int32_t top_k, double top_p, double min_p, float u) {
        // A. the largest logit (NaN if there is one), over the cluster
        float m = __int_as_float(0xff800000);
        each([&](float l, uint32_t) { m = max_nan(m, l); });
#pragma unroll
        for (int o = 16; o; o >>= 1)
            m = max_nan(m, __shfl_xor_sync(kAllLanes, m, o));
        if (lane == 0)
            sh.warp_max[warp] = __float_as_uint(m);
        __syncthreads();
        for (int w = 0; w < kNW; ++w)
            m = max_nan(m, __uint_as_float(sh.warp_max[w]));
        meet();
        if (tid < C)
            *cluster.map_shared_rank(&sh.part_max[rank], tid) = __float_as_uint(m);
        cluster.sync();
        for (int r = 0; r < C; ++r)
            m = max_nan(m, __uint_as_float(sh.part_max[r]));
        if (!code && !(m >= -3.402823466e38f && m <= 3.402823466e38f))
            code = SV_ERR_NONFINITE;
        scale.lmax = m;
        if (code) {
            const float nan = __int_as_float(0x7fffffff);
            write([](float, uint32_t) { return false; }, 0.0f, 0.0f, true);
            if (rank == 0 && tid == 0)
                a_token(-1, nan);
            finish(code, 0, nan);
            cluster.sync();
            return;
        }
        if (T == 0.0f) {
            uint32_t id = 0xffffffffu;
            each([&](float l, uint32_t i) {
                if (l == m)
                    id = min(id, i);
            });
            id = __reduce_min_sync(kAllLanes, id);
            __syncthreads();
            if (lane == 0)
                sh.warp_cnt[warp] = id;
            __syncthreads();
            for (int w = 0; w < kNW; ++w)
                id = min(id, sh.warp_cnt[w]);
            if (tid < C)
                *cluster.map_shared_rank(&sh.part_cnt[rank], tid) = id;
            cluster.sync();
            for (int r = 0; r < C; ++r)
                id = min(id, sh.part_cnt[r]);
            write([=](float, uint32_t i) { return i == id; }, m, 0.0f, false);
            if (rank == 0 && tid == 0)
                a_token(id, 1.0f);
            finish(SV_OK, 1, 1.0f);
            cluster.sync();
            return;
        }
        split_scale(T, scale.ch, scale.cl);

        // B. bins over the whole row
        const auto linear = [&](float l) {
            return logit_key(l) > kKeyMinusInf ? bin_of(l) : -1;
        };
        histogram(linear);
        Search s;
        s.above_mass = 0;
        s.above_count = 0;
        s.k = top_k > 0 ? (uint32_t)top_k : 0;
        s.top_p = top_p;
        s.p = 0;
        s.draw = false;
        s.limit_bin = kBins;
        uint32_t limit_key = 0;
        if (min_p > 0.0) {
            // the smallest float l with l - l_max >= T ln(min_p)
            const float limit = __double2float_ru((double)m + (double)T * log(min_p));
            limit_key = logit_key(limit);
            if (limit_key > kKeyMinusInf)
                s.limit_bin = bin_of(limit);
        }
        unsigned long long whole, E;
        uint32_t n, kept;
        search(s, true, whole, n);
        const Found f = first();
        uint32_t cut_key = kKeyMinusInf + 1, klo = 1, khi = 0;
        bool split = false;
        Found g = f;
        if (f.bin < kBins) {
            narrow(s, g, limit_key, klo, khi, split);
            if (g.count <= kList) {
                gather(klo, khi);
                if (rank == 0)
                    cut_in_list(s, g, limit_key, klo, 0);
                share_cut();
                cut_key = sh.cut_key;
                kept = sh.kept;
                E = sh.kept_mass;
            } else {  // one value: the conditions hold at its start, or the limit is above it
                const bool in = klo >= limit_key;
                cut_key = in ? klo : limit_key;
                kept = g.above_count + (in ? g.count : 0);
                E = g.above_mass + (in ? g.mass : 0);
            }
        } else {
            kept = n;
            E = whole;
        }

        // C. the draw
        const float inv = (float)((double)(1ull << scale.fix) / (double)E);
        if (a.u) {
            const unsigned long long target = floor_scaled(u, E);
            if (f.bin < kBins && g.count <= kList && target >= g.above_mass) {
                if (rank == 0)
                    draw_in_list(0, g.above_mass, target);  // the cut's list holds it
            } else if (f.bin < kBins && g.count > kList && target >= g.above_mass) {
                const unsigned long long w = weight_fixed(scale, sh.pow2, key_logit(klo));
                draw_among_equals(klo, (target - g.above_mass) / w);
            } else {
                cluster.sync();
                if (split)
                    histogram(linear);
                else if (tid < kConds)
                    sh.found[tid].bin = kBins;
                cluster.sync();
                Search d;
                d.above_mass = 0;
                d.above_count = 0;
                d.k = 0;
                d.top_p = 1.0;
                d.p = target;
                d.limit_bin = kBins;
                d.draw = true;
                unsigned long long dm;
                uint32_t dn;
                search(d, true, dm, dn);
                Found h = first();
                narrow(d, h, 0, klo, khi, split);
                if (h.count <= kList) {
                    gather(klo, khi);
                    if (rank == 0)
                        draw_in_list(0, h.above_mass, target);
                } else {
                    const unsigned long long w = weight_fixed(scale, sh.pow2, key_logit(klo));
                    draw_among_equals(klo, (target - h.above_mass) / w);
                }
            }
            if (rank == 0 && tid == 0)
                a_token(sh.token, weight_float(scale, key_logit(sh.token_key)) * inv);
        }
        // D. rows out
        const float cut = key_logit(cut_key);
        write([&](float l, uint32_t) { return l >= cut; }, cut, inv, false);
        finish(SV_OK, kept, (float)((double)E / (double)whole));
        cluster.sync();  // no CTA leaves while another may still write into it
    }
};

template <int ES>
__global__ void __launch_bounds__(kNT, 4) sv_sample_kernel(const __grid_constant__ Args a) {
    __shared__ Shared sh;
    Kernel<ES> k(a, sh);
    k.run();
}

int launch(sv_ctx* ctx, Args& a, int B, int rows, int64_t V, int dtype, cudaStream_t stream) {
    sv_plan plan;
    const int rc = spec_sample_get_plan(ctx, B, rows, V, dtype, &plan);
    if (rc != SV_OK)
        return rc;
    const int es = dtype == SV_BF16 ? 2 : 4;
    a.err_word = ctx->d_err;
    a.V = V;
    a.slice = plan.slice;
    a.C = plan.cluster;
    a.rows_per_seq = rows;
    a.fix = weight_bits(V);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)plan.grid, 1, 1);
    cfg.blockDim = dim3(kNT, 1, 1);
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

}  // namespace

namespace sv {

int sampling_setup() {
    for (const void* fn : {(const void*)sv_sample_kernel<2>, (const void*)sv_sample_kernel<4>})
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
            (void)cudaGetLastError();
            return 8;
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
    const int64_t last = (int64_t)B * rows_per_seq - 1;
    const char *i0 = static_cast<const char*>(logits), *o0 = static_cast<char*>(out_logits);
    const char *i1 = i0 + (last * logits_stride + V) * es, *o1 = o0 + (last * out_stride + V) * es;
    if (o0 < i1 && i0 < o1 && !(i0 == o0 && (last == 0 || logits_stride == out_stride)))
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
