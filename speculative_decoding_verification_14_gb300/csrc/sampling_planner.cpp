// sampling_planner.cpp -- maps the rows of a sampling, filter or
// log-probability call onto thread-block clusters: one cluster per row, a
// slice of the vocabulary per CTA.
#include "../../include/spec_verify.h"
#include "sv_internal.h"

namespace {

// The largest power of two of CTAs per row that the GPU holds for every row
// at once (ctas_per_sm of `threads` each) and that leaves a CTA at least
// min_slice entries, min_full where the SMs have several CTAs each.
int plan_rows(int num_sms, int max_cluster, int B, int rows_per_seq, int64_t V, int dtype,
              int ovr_cluster, int threads, int ctas_per_sm, int64_t min_slice, int64_t min_full,
              sv_plan* out) {
    using namespace sv;
    if (!out || num_sms < 1 || max_cluster < 1 || B < 1 || rows_per_seq < 1 ||
        rows_per_seq > kMaxRows || V < 1 || V > ((int64_t)1 << 31) ||
        (dtype != SV_F32 && dtype != SV_BF16) || ovr_cluster < 0 || ovr_cluster > kMaxCluster)
        return SV_ERR_INVALID_ARG;
    if (ovr_cluster > max_cluster)
        return SV_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)B * rows_per_seq;
    int C = 1;
    if (ovr_cluster) {
        C = ovr_cluster;
    } else {
        for (int c = max_cluster < kMaxCluster ? max_cluster : kMaxCluster; c > 1; c /= 2)
            if (rows * c <= (int64_t)ctas_per_sm * num_sms &&
                ceil_div(V, c) >= (rows * c > num_sms ? min_full : min_slice)) {
                C = c;
                break;
            }
    }
    if (rows * C > 0x7fffffff)
        return SV_ERR_UNSUPPORTED;
    out->cluster = C;
    out->group = 1;
    out->threads = threads;
    out->smem_bytes = 0;
    // slices are cut between 16-byte vectors: a row may begin up to seven entries into one
    out->slice = round_up(ceil_div(V + 7, C), kSliceAlign);
    out->grid = rows * C;
    out->bulk_copy = ((V * (dtype == SV_BF16 ? 2 : 4)) % 16) == 0 ? 1 : 0;
    out->prefetch_next = 0;
    out->stages = 0;
    return SV_OK;
}

}  // namespace

// A sampling row's work beside its passes grows with the CTAs: 64 rows of 151936
// bfloat16 take 38.9 us with eight CTAs a row and 38.3 with four, 256 of 128256 64 us
// with four and 56 with two; 150 rows of 50257 float32 82 us with four and 68 with two.
// Between those sizes it is not always the best: of 8 to 153 rows of 32000 to 151936 under top-k and
// top-p, 67 of 104 are within 5 % of the best count.  The others: 77 to 152 rows of 32000, 25.5 us with
// one CTA a row and 21.2 to 22.5 with two; 20 to 39 rows, up to 14 % better with twice as many; 152
// rows of 128256 float32 or 151936, whose four CTAs a row do not all fit at once, 73 us and 49 with two.
extern "C" int spec_sample_plan_for(int num_sms, int max_cluster, int B, int rows_per_seq,
                                    int64_t V, int logits_dtype, int ovr_cluster, sv_plan* out) {
    return plan_rows(num_sms, max_cluster, B, rows_per_seq, V, logits_dtype, ovr_cluster, 256, 4,
                     2048, 24576, out);
}

// A log-probability row's does less: 37 x 3 rows of 50257 float32 take 14.2 us with
// four CTAs a row and 16.7 with one; 8 x 5 of 32000 bfloat16 10.7 us with eight and 9.3
// with four.  Where rows times CTAs come to all that the SMs hold (38 rows of sixteen, 76 of eight, 152
// of four), clusters do not all fit at once: 152 rows of 32000 bfloat16 take 15.9 us and 10.8 with two.
extern "C" int spec_logprobs_plan_for(int num_sms, int max_cluster, int B, int rows_per_seq,
                                      int64_t V, int logits_dtype, int ovr_cluster,
                                      sv_plan* out) {
    return plan_rows(num_sms, max_cluster, B, rows_per_seq, V, logits_dtype, ovr_cluster, 256, 4,
                     2048, 4096, out);
}
