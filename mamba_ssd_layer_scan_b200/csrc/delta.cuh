// Internal interface of the gated delta rule's kernels (delta_*.cu).
#pragma once

#include "common.cuh"

namespace ssd {

constexpr float kL2Eps = 1e-6f;   // under the root of q's and k's norms

struct DeltaArgs {
    const void *q, *k, *v;      // (batch, L, G, N), same, (batch, L, H, P)
    const float *g, *beta;      // (batch, L, H); g nullable (no decay)
    const float *init;          // (nseq or batch, H, P, N), nullable
    void *o;                    // (batch, L, H, P)
    float *final_state;         // like init, nullable
    int64_t batch, L;
    int H, G, P, N;
    float scale;
    int l2norm;
    const int32_t *cu;          // packed sequences (batch 1): nseq + 1 offsets, else null
    int nseq;
};

// The recurrence token by token, any supported shape and type, state rows in registers.
// `status` (nullable): a nonzero word makes the kernel return without touching anything.
bool delta_recurrent_supported(int N);
cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool is_bf16, const int *status,
                                   cudaStream_t st);

}  // namespace ssd
