// Launchers of the gated linear recurrence (wkv_gated_scan.cu) and the gated group norm
// (wkv_group_norm.cu), called by the C ABI after it has validated every argument.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

#include "wkv_internal.h"

namespace wkvb {

// Steps from one saved state to the next (the forward's `carry`, read by the backward).
constexpr int kGatedCarrySteps = 64;

struct GatedScanShape {
    int64_t B, T, C;
    int io;  // 0 fp32, 1 bf16
};

// Whether one launch's grid holds the shape.
bool gated_scan_fits(const GatedScanShape& s);

// The scan's bounded waits; for tests, the rank in its cluster of a block that withholds its sums, or the
// fetch of its first tile (-1: none).
struct GatedScanWaits {
    uint32_t spin_limit = kSpinLimitDefault;
    int drop_sums = -1, drop_tile = -1;
};

cudaError_t launch_gated_scan_forward(const GatedScanShape& s, const void* g, const void* x, const float* state_in,
                                      void* y, float* state_out, float* carry, cudaStream_t stream,
                                      const GatedScanWaits& waits = {});
cudaError_t launch_gated_scan_backward(const GatedScanShape& s, const void* g, const void* x, const float* carry,
                                       const void* gy, const float* gstate_out, void* gg, void* gx, float* gstate_in,
                                       cudaStream_t stream, const GatedScanWaits& waits = {});
// n row-channels
cudaError_t launch_gated_scan_step(int64_t n, int io, const void* g, const void* x, float* state, void* y,
                                   cudaStream_t s);

// Activations of the group norm (the C ABI's wkv_act).
enum : int { kActNone = 0, kActSilu = 1, kActSigmoid = 2 };

struct GroupNormShape {
    int64_t rows, C, groups;
    int io;  // 0 fp32, 1 bf16
    float eps;
    int act;
};

// Scratch of the backward's weight and bias sums.
size_t group_norm_workspace_bytes(const GroupNormShape& s);
cudaError_t launch_group_norm_forward(const GroupNormShape& s, const void* x, const void* z, const float* weight,
                                      const float* bias, void* y, cudaStream_t stream);
// workspace may be null when neither gweight nor gbias is wanted
cudaError_t launch_group_norm_backward(const GroupNormShape& s, const void* x, const void* z, const float* weight,
                                       const float* bias, const void* gy, void* gx, void* gz, float* gweight, float* gbias,
                                       void* workspace, cudaStream_t stream);

}  // namespace wkvb
