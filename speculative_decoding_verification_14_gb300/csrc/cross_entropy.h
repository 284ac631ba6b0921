// cross_entropy.h -- sizes and workspace of the cross-entropy calls, shared by their planner and their
// kernels.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

namespace sv {

constexpr int kTile = 256;             // rows and columns of a CTA pair's tile
constexpr int kHalf = kTile / 2;       // of one CTA's operands
constexpr int kBlockK = 64;            // depth of a stage: 128 bytes, one swizzle atom
// A piece of the vocabulary is as many tiles as this holds of all rows' d, one at least (beyond 524288 rows that is more).
// Measured, replayed, with 32, 64, 128, 256 MB and 1 GB: 256 rows of 151936 x 2048, the hidden states' gradient, 445, 406,
// 367, 368, 368 us; 1024 rows of 128256 x 1024, both, 981, 800, 724, 681, 681 us; 8192 rows of 128256 x 4096, both, 27.8,
// 23.4, 20.8, 20.4, 20.0 ms; 65536 rows of it 928, 505, 299, 216, 172 ms, where the float32 sums of the hidden states'
// gradient, read and written once a piece, begin to count.  Pieces that L2 would hold lose more than they save.
constexpr int64_t kPieceBytes = (int64_t)1 << 28;
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxRowsCe = (int64_t)1 << 20;
constexpr int64_t kCountRows = 1024;  // have a number of their own of those that count, in calls of more rows than
constexpr int64_t kCountFrom = 8192;
constexpr int64_t kCountFromLengths = 2048;  // where a look at a row divides by the rows of a sequence

// rows of the box that A's copies have
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr int box_rows(int64_t rows) { return rows >= kHalf ? kHalf : (int)((rows + 7) / 8 * 8); }

// What a call keeps in its workspace: offsets in bytes.
struct CrossEntropyPlan {
    int64_t rows;        // R rounded up to a tile
    int64_t depth;       // D rounded up to 16 bytes: the packed rows' stride
    int64_t vocab_tiles;
    int64_t piece_tiles; // of one piece of the vocabulary
    int64_t pieces;
    int splits;          // of a piece's depth in the hidden states' gradient
    size_t counts;                      // int32 of each kCountRows rows
    size_t index, label, lse, loss, scale;  // [rows]: source row, label, lse, loss, grad_loss
    size_t hidden;                      // bf16 [rows, depth]
    size_t stats, label_logit;          // float2 [vocab_tiles, rows], float [rows]
    size_t probs;                       // bf16 [rows, piece_tiles * kTile]
    size_t sums;                        // float [splits, rows, depth]
    size_t total;
};

CrossEntropyPlan cross_entropy_plan(int num_sms, int64_t R, int64_t V, int64_t D, bool grad);

}  // namespace sv
