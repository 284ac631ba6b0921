// losses_selftest.h -- which wait of the losses' kernels a call on this context takes, once it is over, for one
// that ran out (spec_losses_selftest): SV_SELFTEST_OFF but for one context at a time.  Not part of the public ABI.
#pragma once

struct sv_ctx;

namespace sv {

int losses_selftest(const sv_ctx* ctx);

}  // namespace sv
