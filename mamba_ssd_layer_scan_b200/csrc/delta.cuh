// Internal interface of the gated delta rule's kernels (delta_*.cu).
#pragma once

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace ssd {

constexpr float kL2Eps = 1e-6f;   // under the root of q's and k's norms

// Kernels of one call that follow one another: a kernel launched with launch_after() may start while
// the one before it still runs, and reads nothing of it before wait_before() returns (every CTA
// calls it); let_next_start() in the earlier kernel allows it.
__device__ __forceinline__ void wait_before()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Lets `kern` have `smem` bytes of dynamic shared memory on the current device; what it was given
// before is remembered, the call takes a microsecond or two.
inline cudaError_t allow_smem(const void *kern, size_t smem)
{
    if (smem <= 40 * 1024) return cudaSuccess;   // with the static part it fits anyway
    constexpr int kKernels = 32, kDevices = 16;
    static std::atomic<const void *> kernels[kKernels];
    static std::atomic<int> given[kKernels][kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> *mine = nullptr;
    for (int i = 0; i < kKernels && dev < kDevices && !mine; ++i) {
        const void *at = kernels[i].load();
        if (!at && kernels[i].compare_exchange_strong(at, kern)) at = kern;
        if (at == kern) mine = &given[i][dev];
    }
    if (mine && mine->load() >= (int)smem) return cudaSuccess;
    static std::mutex one;   // no call may take back what another one has been given
    const std::lock_guard<std::mutex> hold(one);
    if (mine && mine->load() >= (int)smem) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && mine) mine->store((int)smem);
    return e;
}

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         Args... args)
{
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

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
    int *clear;                 // a status word that the call's first kernel clears; nullable
};

// The recurrence token by token, any supported shape and type, state rows in registers.
// `status` (nullable): a nonzero word makes the kernel return without touching anything.
bool delta_recurrent_supported(int N);
cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool is_bf16, const int *status,
                                   cudaStream_t st);

// The chunked form: chunks of kDeltaChunk tokens on warp-level bf16 matrix instructions (bf16
// inputs, N 64 or 128, P a multiple of 16).
constexpr int kDeltaChunk = 32;
bool delta_chunk_supported(bool is_bf16, int P, int N);

// The chunked form on tcgen05 (delta_tc.cu): bf16, P and N 64 or 128.  A bounded wait that gives up
// sets a bit of `status`, the workspace's status word.
constexpr int kDeltaTcChunk = 64;
constexpr int kDeltaTcItem = 25 * 1024;   // bytes of the workspace per chunk and head
bool delta_tc_supported(int P, int N);
cudaError_t launch_delta_tc(const DeltaArgs &a, char *items, int64_t nchunks, const int2 *tab,
                            const int32_t *cstart, int *status, cudaStream_t st);

// What delta_prep_kernel leaves of one chunk of one head, 8.5 KB in the workspace: row-major 32 x 32
// bf16 triangles in two parts each.
struct DeltaItem {
    static constexpr int kTri = kDeltaChunk * kDeltaChunk * 2;   // bytes of one part
    static constexpr int kInvHi = 0, kInvLo = kTri, kVec = 2 * kTri;
    // floats at kVec: ek[32], sw[32], eq[32], the chunk's decay
    static constexpr int kAttHi = kVec + 512, kAttLo = kAttHi + kTri, kBytes = kAttLo + kTri;
};

cudaError_t launch_delta_prep(const DeltaArgs &a, char *items, bool for_backward, int64_t nchunks,
                              const int2 *tab, cudaStream_t st);
// What the backward's kernels hand on through the workspace, and its outputs.  Spans are of 64
// tokens (n64 per batch row), tiles the P / 16 runs of 16 rows of a head, chunks of 32 tokens.
struct DeltaBwd {
    const bf16 *dout;      // (batch, L, H, P)
    const float *dfinal;   // (batch, H, P, N), nullable
    int64_t n64;
    float *states;         // (batch, n64 + 1, H, P, N): entering each span; last: the final state
    bf16 *dstates;         // (batch, n64, H, P, N): the gradient of the state leaving each span
    float *wfrag;          // W in accumulator layout, per (batch, chunk, H, tile): 16 x 32
    float *dot_oo, *dot_vv, *dot_vw;   // (batch, chunk, H, tile, 32): <dO, O>, <dV, V>, <dV, W>
    float *dot_ss;         // (batch, n64 + 1, H, tile): <dS, S> at the start, then behind each span
    float *dq_part, *dk_part;          // (batch, L, G * runs, N)
    int runs;              // runs of heads per group, `run_heads` each (the last may be shorter)
    int run_heads;
    bf16 *dq, *dk, *dv;    // outputs
    float *dg, *dbeta, *dinit;         // dg, dinit nullable
};

// bwd: nullable; with it the forward is run for the backward (see delta_chunk.cu).
cudaError_t launch_delta_chain(const DeltaArgs &a, const DeltaBwd *bwd, const char *items,
                               int64_t nchunks, const int2 *tab, const int32_t *cstart,
                               const int *status, cudaStream_t st);
cudaError_t launch_delta_adjoint(const DeltaArgs &a, const DeltaBwd &w, const char *items,
                                 int64_t nchunks, cudaStream_t st);
// dq and dk of each span and run of heads, then their sums over the runs; dg and dbeta.
cudaError_t launch_delta_grads(const DeltaArgs &a, const DeltaBwd &w, int64_t nchunks,
                               cudaStream_t st);

}  // namespace ssd
