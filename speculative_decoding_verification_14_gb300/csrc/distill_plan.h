// distill_plan.h -- constants shared by the distillation kernel and its planner, and the check that
// rows read and rows written do not meet.  Not part of the public ABI.
#pragma once

#include <cstdint>

namespace sv {

constexpr int kDistillThreads = 224;     // that walk a slice; two warps beside them have the list and the loss
constexpr int kDistillCtas = 3;           // that fit an SM
constexpr int kDistillMaxList = 128;
constexpr int kDistillSmem = 221184;      // a CTA's slice at most (216 KB, beside the fixed state)
constexpr int kDistillFullSmem = 73728;   // a slice of which three CTAs fit an SM

// Whether one of n rows of `bytes` at x shares memory with one at y.  Rows of a kind do not overlap.
bool rows_meet(const void* x, int64_t x_stride, const void* y, int64_t y_stride, int64_t n, int64_t bytes);

}  // namespace sv
