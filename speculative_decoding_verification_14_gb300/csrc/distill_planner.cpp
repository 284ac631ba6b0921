// distill_planner.cpp -- maps the rows of a distillation call onto thread-block clusters: one
// cluster per row, a slice of the vocabulary in each CTA's shared memory.
#include "distill_plan.h"

#include "../../include/spec_verify.h"
#include "sv_internal.h"

namespace sv {

bool rows_meet(const void* x, int64_t x_stride, const void* y, int64_t y_stride, int64_t n, int64_t bytes) {
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
    if (y0 >= x0 + (uintptr_t)((n - 1) * x_stride + bytes) || x0 >= y0 + (uintptr_t)((n - 1) * y_stride + bytes))
        return false;
    // where neither of two rows meets, the lower one meets no later one of the other kind
    for (int64_t i = 0, j = 0; i < n && j < n;) {
        const uintptr_t a = x0 + (uintptr_t)(i * x_stride), b = y0 + (uintptr_t)(j * y_stride);
        if (a < b + (uintptr_t)bytes && b < a + (uintptr_t)bytes)
            return true;
        ++(a < b ? i : j);
    }
    return false;
}

}  // namespace sv

extern "C" int spec_distill_plan_for(int num_sms, int max_cluster, int B, int rows_per_seq, int64_t V,
                                     int logits_dtype, int ovr_cluster, sv_plan* out) {
    using namespace sv;
    if (!out || num_sms < 1 || max_cluster < 1 || B < 1 || rows_per_seq < 1 || rows_per_seq > kMaxRows || V < 1 ||
        V > ((int64_t)1 << 31) - 1 || (logits_dtype != SV_F32 && logits_dtype != SV_BF16) || ovr_cluster < 0 ||
        ovr_cluster > kMaxCluster)
        return SV_ERR_INVALID_ARG;
    if (ovr_cluster > max_cluster)
        return SV_ERR_UNSUPPORTED;
    const int es = logits_dtype == SV_BF16 ? 2 : 4, entries = 16 / es;
    const int64_t rows = (int64_t)B * rows_per_seq;
    // a row may begin up to seven entries into a vector
    const int64_t vectors = ceil_div(V + entries - 1, entries);
    const int most = max_cluster < kMaxCluster ? max_cluster : kMaxCluster;
    int C = 0;
    if (ovr_cluster) {
        C = ovr_cluster;
    } else {
        for (C = 1; C < most && ceil_div(vectors, C) * 16 > kDistillFullSmem;)  // the least of which an SM takes three
            ++C;
        // few rows: more CTAs for each, down to 512 vectors a slice
        while (2 * C <= most && rows * 2 * C <= num_sms && ceil_div(vectors, 2 * C) >= 512)
            C *= 2;
    }
    const int64_t per = ceil_div(vectors, C);
    if (per * 16 > kDistillSmem || rows * C > 0x7fffffff)
        return SV_ERR_UNSUPPORTED;
    out->cluster = C;
    out->group = 1;
    out->threads = kDistillThreads + 64;
    out->smem_bytes = (int)(per * 16);
    out->slice = per * entries;
    out->grid = rows * C;
    out->bulk_copy = 1;
    out->prefetch_next = 0;
    out->stages = 1;
    return SV_OK;
}
