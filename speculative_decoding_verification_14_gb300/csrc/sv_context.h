// sv_context.h -- the context behind sv_ctx and the host-side helpers that every
// entry point shares.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

struct sv_ctx {
    int device = 0;
    int max_B = 0, max_K = 0;
    int64_t max_V = 0;
    int num_sms = 0, smem_optin = 0, max_cluster = 8;
    int greedy_max_cluster = 8;
    int sampling_max_cluster = 8;  // sampling and log-probability kernels
    uint32_t* d_err = nullptr;
    int ovr_cluster = 0, ovr_group = 0, ovr_threads = 0;  // spec_verify_set_plan_override
    uint32_t* al_hist = nullptr;  // caller's accepted-length counters (device), or none
    int al_bins = 0;
    uint32_t* general_rows = nullptr;  // caller's counter of slow sampling rows (device), or none
    // staging for the host-buffer entry point
    unsigned char* d_stage = nullptr;
    size_t stage_bytes = 0;
};

namespace sv {

// Sets the attributes of the sampling and log-probability kernels on the
// current device.  Returns the largest cluster they may use, 0 when a CUDA
// call failed.
int sampling_setup();
bool logprobs_setup();

// Makes `dev` current for a scope.
struct DeviceGuard {
    int prev = -1;
    bool switched = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) {
            switched = cudaSetDevice(dev) == cudaSuccess;
        }
    }
    ~DeviceGuard() {
        if (switched)
            cudaSetDevice(prev);
    }
};

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace sv
