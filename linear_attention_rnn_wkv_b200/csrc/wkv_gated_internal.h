// Launchers of the gated linear recurrence (wkv_gated_scan.cu) and the gated group norm
// (wkv_group_norm.cu), called by the C ABI after it has validated every argument.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

namespace wkvb {

// Steps from one saved state to the next (the forward's `carry`, read by the backward).
constexpr int kGatedCarrySteps = 128;

struct GatedScanShape {
    int64_t B, T, C;
    int io;  // 0 fp32, 1 bf16
};

// Whether one launch's grid holds the shape.
bool gated_scan_fits(const GatedScanShape& s);

cudaError_t launch_gated_scan_forward(const GatedScanShape& s, const void* g, const void* x, const float* state_in,
                                      void* y, float* state_out, float* carry, cudaStream_t stream);
cudaError_t launch_gated_scan_backward(const GatedScanShape& s, const void* g, const void* x, const float* carry,
                                       const void* gy, const float* gstate_out, void* gg, void* gx, float* gstate_in,
                                       cudaStream_t stream);
// n row-channels
cudaError_t launch_gated_scan_step(int64_t n, int io, const void* g, const void* x, float* state, void* y,
                                   cudaStream_t s);

}  // namespace wkvb
