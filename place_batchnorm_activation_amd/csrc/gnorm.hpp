// Host launchers of the group norm (groupnorm.hip); arguments are validated by the C ABI
// layer (api_gnorm.cpp) before any of these is called.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "block.hpp"

namespace iabn {

// The first three as of the gated unit (block.hpp's GluAct).
enum GnAct { kGnSilu = 0, kGnGelu = 1, kGnGeluTanh = 2, kGnIdentity = 3, kGnLeaky = 4 };

struct GnArgs {
    const void *x, *dy;
    void* out;                                    // y, or dx
    int64_t ldx, lddy, ldo;
    int64_t N, HW, C, G;
    const float *weight, *bias;
    int act;
    float param, eps;
    float* stats;                                 // [N, G, 2]: mean and rstd
    float *dweight, *dbias;
};

size_t gn_workspace_bytes(int64_t N, int64_t HW, int64_t C, int64_t G, int64_t cus);
void launch_gn_forward(const GnArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s);
void launch_gn_backward(const GnArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s);

}  // namespace iabn
