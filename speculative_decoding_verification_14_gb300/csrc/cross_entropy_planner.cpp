// cross_entropy_planner.cpp -- pieces of the vocabulary, splits and workspace of the cross-entropy
// calls; the losses' self-test.
#include "cross_entropy.h"

#include <atomic>

#include "../../include/spec_verify.h"
#include "losses_selftest.h"
#include "sv_internal.h"

namespace sv {

namespace {
std::atomic<const sv_ctx*> tested{nullptr};
std::atomic<int> tested_wait{0};
}  // namespace

int losses_selftest(const sv_ctx* ctx) {
    return tested.load(std::memory_order_acquire) == ctx ? tested_wait.load(std::memory_order_relaxed) : SV_SELFTEST_OFF;
}

CrossEntropyPlan cross_entropy_plan(int num_sms, int64_t R, int64_t V, int64_t D, bool grad) {
    CrossEntropyPlan p{};
    p.rows = round_up(R, kTile);
    p.depth = round_up(D, 8);
    p.vocab_tiles = ceil_div(V, kTile);
    // the largest pieces whose probabilities stay within kPieceBytes, or of one tile, all of nearly the same size
    const int64_t fit = kPieceBytes / (p.rows * kTile * 2);
    p.pieces = ceil_div(p.vocab_tiles, fit < 1 ? 1 : fit);
    p.piece_tiles = ceil_div(p.vocab_tiles, p.pieces);
    p.pieces = ceil_div(p.vocab_tiles, p.piece_tiles);
    // few tiles of the hidden states' gradient: the piece's depth is split, down to two tiles a part
    const int64_t tiles = p.rows / kTile * ceil_div(D, kTile), pairs = num_sms / 2 > 0 ? num_sms / 2 : 1;
    int64_t splits = pairs / tiles;
    if (splits > kMaxSplits)
        splits = kMaxSplits;
    if (splits > p.piece_tiles / 2)
        splits = p.piece_tiles / 2;
    p.splits = splits < 1 ? 1 : (int)splits;
    size_t at = 0;
    const auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += (size_t)round_up(bytes, 256);
        return here;
    };
    p.counts = R > kCountFromLengths ? take(ceil_div(R, kCountRows) * 4) : 0;
    p.index = take(p.rows * 4 + 8);  // and the number of rows that count, and whether a wait ran out
    p.label = take(p.rows * 4);
    p.hidden = take(p.rows * p.depth * 2);
    if (grad) {
        p.lse = take(p.rows * 4);
        p.loss = take(p.rows * 4);
        p.scale = take(p.rows * 4);
        p.probs = take(p.rows * p.piece_tiles * kTile * 2);
        p.sums = take((int64_t)p.splits * p.rows * p.depth * 4);
    } else {
        p.stats = take(p.vocab_tiles * p.rows * 8);
        p.label_logit = take(p.rows * 4);
    }
    p.total = at;
    return p;
}

}  // namespace sv

extern "C" int spec_losses_selftest(sv_ctx* ctx, int wait) {
    if (!ctx || wait < SV_SELFTEST_OFF || wait > SV_SELFTEST_DISTILL_EXCHANGE)
        return SV_ERR_INVALID_ARG;
    sv::tested.store(nullptr, std::memory_order_release);
    sv::tested_wait.store(wait, std::memory_order_relaxed);
    if (wait != SV_SELFTEST_OFF)
        sv::tested.store(ctx, std::memory_order_release);
    return SV_OK;
}

extern "C" int spec_cross_entropy_workspace_for(int num_sms, int B, int rows_per_seq, int64_t V, int64_t D, int grad,
                                                size_t* bytes) {
    using namespace sv;
    if (!bytes || num_sms < 1 || B < 1 || rows_per_seq < 1 || rows_per_seq > kMaxRows || V < 1 ||
        V > ((int64_t)1 << 31) - 1 || D < 1 || D > ((int64_t)1 << 20) || (grad != 0 && grad != 1) ||
        (int64_t)B * rows_per_seq > kMaxRowsCe)
        return SV_ERR_INVALID_ARG;
    const int64_t R = (int64_t)B * rows_per_seq;
    *bytes = cross_entropy_plan(num_sms, R, V, D, false).total;
    if (grad) {  // serves both calls
        const size_t with = cross_entropy_plan(num_sms, R, V, D, true).total;
        *bytes = with > *bytes ? with : *bytes;
    }
    return SV_OK;
}
