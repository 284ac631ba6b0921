// sampling_general.cuh -- the sampling kernel's way for any row: for the few that
// counting by places does not settle (sampling.cu), and for erroneous ones.
//
// A pass for l_max; a pass that adds every entry's count and integer weight
// into 2048 bins over t = (l_max - l) c, 32 to the octave; the bin where the first filter
// ends, and the one that u E falls into; the entries of such a bin in a sorted list
// of the first CTA.  A bin with more entries than the list holds is split by the
// logits' keys, 2048 ways, until it fits or is one value.
#pragma once

#include "sampling_row.cuh"

namespace {

constexpr float kBinsPerOctave = 32.0f;

template <int ES>
struct General {
    Shared* sh;
    View<ES> v;
    int tid, lane, warp, rank, C;
    RowScale scale;

    __device__ __forceinline__ explicit General(Shared* s)
        : sh(s), v(s), tid(threadIdx.x), lane(tid & 31), warp(tid >> 5), rank(cta_rank()), C(s->args.C) {
        scale.fix = s->args.fix;
        scale.g = 1.0f;
    }

    // the linear bin of a logit; larger logits, smaller bins
    __device__ __forceinline__ int bin_of(float l) const {
        const float t = (scale.lmax * scale.g - l * scale.g) * scale.ch * kBinsPerOctave;
        return t < (float)(kBins - 1) ? (int)t : kBins - 1;
    }

    template <class Map>
    __device__ __forceinline__ void histogram(Map&& map) {
        for (int b = tid; b < kBins; b += kNT)
            sh->lo[b] = sh->hi[b] = sh->cnt[b] = 0;
        if (tid < kConds)
            sh->found[tid].bin = kBins;
        if (tid == 0)
            sh->list_n[0] = 0;
        __syncthreads();
        v.each([&](float l, uint32_t) {
            const int b = map(l);
            if (b < 0)
                return;
            const unsigned long long w = weight_fixed(scale, sh->pow2, l);
            const uint32_t wl = (uint32_t)w;
            const uint32_t old = atomicAdd(&sh->lo[b], wl);
            const uint32_t h = (uint32_t)(w >> 32) + (old + wl < old);
            if (h)
                atomicAdd(&sh->hi[b], h);
            atomicAdd(&sh->cnt[b], 1u);
        });
        the_cluster().sync();
        // this CTA's range of the bins, added up over the cluster
        const int per = (kBins + C - 1) / C, b0 = rank * per;
        const int b1 = b0 + per < kBins ? b0 + per : kBins;
        for (int b = b0 + tid; b < b1; b += kNT) {
            unsigned long long m = 0;
            uint32_t n = 0;
            for (int r = 0; r < C; ++r) {
                m += ((unsigned long long)peer(sh->hi, r)[b] << 32) +
                     peer(sh->lo, r)[b];
                n += peer(sh->cnt, r)[b];
            }
            sh->lo[b] = (uint32_t)m;
            sh->hi[b] = (uint32_t)(m >> 32);
            sh->cnt[b] = n;
        }
        __syncthreads();
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
    __device__ __forceinline__ void search(Search& s, bool whole, unsigned long long& total, uint32_t& total_n) {
        const int per = (kBins + C - 1) / C, b0 = rank * per;
        const int b1 = b0 + per < kBins ? b0 + per : kBins;
        const int q = (per + kNT - 1) / kNT;
        const int t0 = b0 + tid * q, t1 = t0 + q < b1 ? t0 + q : b1;
        unsigned long long m = 0, before_m;
        uint32_t n = 0, before_n;
        for (int b = t0; b < t1; ++b) {
            m += ((unsigned long long)sh->hi[b] << 32) + sh->lo[b];
            n += sh->cnt[b];
        }
        {
            const Prefix x = cta_prefix(sh, m, n);
            m = x.mass;
            n = x.count;
            before_m = x.before_mass;
            before_n = x.before_count;
        }
        if (tid < C) {
            *peer(&sh->part_mass[rank], tid) = m;
            *peer(&sh->part_cnt[rank], tid) = n;
        }
        the_cluster().sync();
        total = 0;
        total_n = 0;
        before_m += s.above_mass;
        before_n += s.above_count;
        for (int r = 0; r < C; ++r) {
            if (r < rank) {
                before_m += sh->part_mass[r];
                before_n += sh->part_cnt[r];
            }
            total += sh->part_mass[r];
            total_n += sh->part_cnt[r];
        }
        if (whole && s.top_p < 1.0)
            s.p = ceil_scaled(s.top_p, total);
        const bool by_mass = s.draw || s.top_p < 1.0;
        for (int b = t0; b < t1; ++b) {
            Found f;
            f.bin = b;
            f.count = sh->cnt[b];
            f.mass = ((unsigned long long)sh->hi[b] << 32) + sh->lo[b];
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
        the_cluster().sync();
    }

    __device__ __forceinline__ void tell(int cond, const Found& f) {
        for (int r = 0; r < C; ++r)
            *peer(&sh->found[cond], r) = f;
    }

    // the condition that ends first
    __device__ Found first() const {
        Found f = sh->found[0];
        for (int c = 1; c < kConds; ++c)
            if (sh->found[c].bin < f.bin)
                f = sh->found[c];
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

    // Narrows the entries of found bin f to keys that fit the list, or to a single key.
    __device__ __forceinline__ KeyRange narrow(Search s, Found& f, uint32_t limit_key, bool& split) {
        KeyRange keys;
        keys.lo = key_at(f.bin, false);
        keys.hi = max(key_at(f.bin, true), keys.lo);
        while (f.count > kList && keys.lo != keys.hi) {
            split = true;
            const int n = keys.shift(kBins);
            the_cluster().sync();  // everyone has read `found`
            histogram([&](float l) {
                const uint32_t k = logit_key(l);
                return k <= keys.hi && k >= keys.lo ? (int)((keys.hi - k) >> n) : -1;
            });
            s.above_mass = f.above_mass;
            s.above_count = f.above_count;
            s.limit_bin = kBins;
            if (!s.draw && limit_key >= keys.lo && limit_key <= keys.hi)
                s.limit_bin = (int)((keys.hi - limit_key) >> n);
            unsigned long long m;
            uint32_t count;
            search(s, false, m, count);
            f = first();  // a condition that ends in a range ends in a part of it
            keys = keys.part((uint32_t)f.bin, n);
        }
        return keys;
    }

    // Entries with such keys into the first CTA's list, sorted there.
    __device__ __forceinline__ void gather(KeyRange keys) {
        the_cluster().sync();  // everyone has read `found`
        if (rank == 0 && tid == 0)
            sh->list_n[0] = 0;
        the_cluster().sync();
        uint32_t* n = peer(&sh->list_n[0], 0);
        unsigned long long* list = peer(sh->list, 0);
        v.each([&](float l, uint32_t id) {
            const uint32_t k = logit_key(l);
            if (k >= keys.lo && k <= keys.hi)
                offer(n, list, l, id);
        });
        the_cluster().sync();
        if (rank == 0)
            sort_list(sh, 0);
    }

    // The entry number r, by ascending id, among those with this key.
    __device__ __forceinline__ void draw_among_equals(uint32_t key, unsigned long long r) {
        const uint32_t per = (v.s1 - v.s0 + kNT - 1) / kNT;
        const uint32_t e0 = min(v.s0 + tid * per, v.s1), e1 = min(e0 + per, v.s1);
        uint32_t n = 0;
        for (uint32_t e = e0; e < e1; ++e)
            n += logit_key(scalar_entry<ES>(v.base, e)) == key;
        const uint32_t mine = n;
        const Prefix x = cta_prefix(sh, 0, n);
        uint32_t before = x.before_count;
        n = x.count;
        the_cluster().sync();
        if (tid < C)
            *peer(&sh->part_cnt[rank], tid) = n;
        the_cluster().sync();
        for (int c = 0; c < rank; ++c)
            before += sh->part_cnt[c];
        if (r >= before && r < (unsigned long long)before + mine) {
            uint32_t left = (uint32_t)(r - before);
            for (uint32_t e = e0; e < e1; ++e)
                if (logit_key(scalar_entry<ES>(v.base, e)) == key && left-- == 0) {
                    *peer(&sh->token, 0) = e;
                    *peer(&sh->token_key, 0) = key;
                    break;
                }
        }
        the_cluster().sync();
    }

    __device__ __forceinline__ void run(int code) {
        const float T = sh->set.T;
        // A. the largest logit (NaN if there is one), over the cluster
        float m = __int_as_float(0xff800000);
        v.each([&](float l, uint32_t) { m = max_nan(m, l); });
#pragma unroll
        for (int o = 16; o; o >>= 1)
            m = max_nan(m, __shfl_xor_sync(kAllLanes, m, o));
        if (lane == 0)
            sh->warp_max[warp] = __float_as_uint(m);
        __syncthreads();
        for (int w = 0; w < kNW; ++w)
            m = max_nan(m, __uint_as_float(sh->warp_max[w]));
        if (tid < C)
            *peer(&sh->part_max[rank], tid) = __float_as_uint(m);
        the_cluster().sync();
        for (int r = 0; r < C; ++r)
            m = max_nan(m, __uint_as_float(sh->part_max[r]));
        if (!code && !(m >= -3.402823466e38f && m <= 3.402823466e38f))
            code = SV_ERR_NONFINITE;
        scale.lmax = m;
        if (code) {
            write_out<ES>(sh, nullptr, kBadRow, 0.0f, 0.0f, 0);
            if (rank == 0 && tid == 0)
                put_token(sh, -1, __int_as_float(0x7fffffff));
            put_rest(sh, code, 0, 0, 1);
            the_cluster().sync();
            return;
        }
        if (T == 0.0f) {
            uint32_t id = 0xffffffffu;
            v.each([&](float l, uint32_t i) {
                if (l == m)
                    id = min(id, i);
            });
            id = __reduce_min_sync(kAllLanes, id);
            __syncthreads();
            if (lane == 0)
                sh->warp_cnt[warp] = id;
            __syncthreads();
            for (int w = 0; w < kNW; ++w)
                id = min(id, sh->warp_cnt[w]);
            if (tid < C)
                *peer(&sh->part_cnt[rank], tid) = id;
            the_cluster().sync();
            for (int r = 0; r < C; ++r)
                id = min(id, sh->part_cnt[r]);
            write_out<ES>(sh, nullptr, kKeepToken, m, 0.0f, id);
            if (rank == 0 && tid == 0)
                put_token(sh, (int32_t)id, 1.0f);
            put_rest(sh, SV_OK, 1, 1, 1);
            the_cluster().sync();
            return;
        }
        set_temperature(scale, T);
        if (tid == 0)
            sh->scale = scale;  // read behind the next barrier

        // B. bins over the whole row
        const auto linear = [&](float l) {
            return logit_key(l) > kKeyMinusInf ? bin_of(l) : -1;
        };
        histogram(linear);
        Search s;
        s.above_mass = 0;
        s.above_count = 0;
        s.k = sh->set.k;
        s.top_p = sh->set.top_p;
        s.p = 0;
        s.draw = false;
        s.limit_bin = kBins;
        uint32_t limit_key = 0;
        if (sh->set.has_min) {
            // the smallest float l with l - l_max >= T ln(min_p)
            const float limit = __double2float_ru((double)m + sh->set.dmin);
            limit_key = logit_key(limit);
            if (limit_key > kKeyMinusInf)
                s.limit_bin = bin_of(limit);
        }
        unsigned long long whole, E;
        uint32_t n, kept;
        search(s, true, whole, n);
        const Found f = first();
        uint32_t cut_key = kKeyMinusInf + 1, klo = 0;
        bool split = false;
        Found g = f;
        if (f.bin < kBins) {
            const KeyRange keys = narrow(s, g, limit_key, split);
            klo = keys.lo;
            if (g.count <= kList) {
                gather(keys);
                if (rank == 0) {
                    if (tid == 0)
                        sh->want = {s.k, limit_key, g.above_count, klo, s.top_p < 1.0 ? s.p : 0, g.above_mass, 0};
                    __syncthreads();
                    cut_in_sorted(sh);
                }
                share_cut(sh);
                cut_key = sh->cut_key;
                kept = sh->kept;
                E = sh->kept_mass;
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
        const float inv = inverse_mass(scale, E);
        if (sh->args.u) {
            const unsigned long long target = floor_scaled(sh->set.u, E);
            if (f.bin < kBins && g.count <= kList && target >= g.above_mass) {
                if (rank == 0)
                    draw_in_sorted(sh, 0, g.above_mass, target);  // the cut's list holds it
            } else if (f.bin < kBins && g.count > kList && target >= g.above_mass) {
                const unsigned long long w = weight_call(scale, sh->pow2, key_logit(klo));
                draw_among_equals(klo, (target - g.above_mass) / max(w, 1ull));
            } else {
                the_cluster().sync();
                if (split)
                    histogram(linear);
                else if (tid < kConds)
                    sh->found[tid].bin = kBins;
                the_cluster().sync();
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
                const KeyRange keys = narrow(d, h, 0, split);
                if (h.count <= kList) {
                    gather(keys);
                    if (rank == 0)
                        draw_in_sorted(sh, 0, h.above_mass, target);
                } else {
                    const unsigned long long w = weight_call(scale, sh->pow2, key_logit(keys.lo));
                    draw_among_equals(keys.lo, (target - h.above_mass) / max(w, 1ull));
                }
            }
            if (rank == 0 && tid == 0)
                put_token(sh, (int32_t)sh->token, weight_float(scale, key_logit(sh->token_key)) * inv);
        }
        // D. rows out
        write_out<ES>(sh, nullptr, kKeepFrom, key_logit(cut_key), inv, 0);
        put_rest(sh, SV_OK, kept, E, whole);
        the_cluster().sync();  // no CTA leaves while another may still write into it
    }
};

}  // namespace
