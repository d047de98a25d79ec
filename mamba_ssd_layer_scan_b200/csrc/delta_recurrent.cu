// The gated delta rule token by token:
//
//     S <- exp(g) S,   u = beta (v - S k),   S <- S + u k^T,   o = scale S q
//
// The rows p of a state are independent, so a warp takes kRows of them (8; 4 or 2 where the launch would
// leave SM quarters without a warp) through all tokens of a
// sequence with the rows in registers (lane l holds elements l V .. l V + V - 1 of each).  Both dot
// products of a token are taken of the state as it stands -- S_new q = exp(g) S q + u (k . q) --
// so that a token costs one reduction: the 2 kRows sums are folded over the lanes together, each
// step halving the sums a lane carries (16 shuffles where kRows separate sums take 80).
//
// One token per sequence (decode) is HBM-bound on the float32 state, read and written once (128
// sequences x 80 heads of 64 x 128: 96-101 us, 6.7 TB/s; one sequence of 24 heads 4 us).  Many
// tokens are bound by the latency of that reduction; the chunked kernels take over where they can.
#include "delta.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 4;

template <int V> __device__ __forceinline__ void load_state(const float *p, float (&r)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 v = __ldcs(reinterpret_cast<const float4 *>(p + i));
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    } else if constexpr (V == 2) {
        const float2 v = __ldcs(reinterpret_cast<const float2 *>(p));
        r[0] = v.x; r[1] = v.y;
    } else {
        r[0] = __ldcs(p);
    }
}
template <int V> __device__ __forceinline__ void store_state(float *p, const float (&r)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            __stcs(reinterpret_cast<float4 *>(p + i),
                   make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]));
    } else if constexpr (V == 2) {
        __stcs(reinterpret_cast<float2 *>(p), make_float2(r[0], r[1]));
    } else {
        __stcs(p, r[0]);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// grid.x = ceil(P / (kRows kWarps)) * H * sequences
template <typename T, int V, int kRows>
__global__ void __launch_bounds__(kWarps * 32)
delta_recurrent_kernel(const DeltaArgs a, const int *status)
{
    constexpr int N = 32 * V;
    if (status && *status) return;
    if (a.clear && blockIdx.x + threadIdx.x == 0) *a.clear = 0;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int pblocks = (a.P + kRows * kWarps - 1) / (kRows * kWarps);
    const int h = (int)((blockIdx.x / pblocks) % a.H);
    const int64_t seq = blockIdx.x / pblocks / a.H;
    const int p0 = ((int)(blockIdx.x % pblocks) * kWarps + warp) * kRows;
    if (p0 >= a.P) return;
    const int rows = min(kRows, a.P - p0);
    int64_t t = seq * a.L, end = t + a.L;
    if (a.cu) {
        t = a.cu[seq];
        end = a.cu[seq + 1];
    }

    float s[kRows][V];
    const int64_t at = ((seq * a.H + h) * a.P + p0) * N + lane * V;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (a.init && r < rows) {
            load_state<V>(a.init + at + (int64_t)r * N, s[r]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) s[r][i] = 0.f;
        }
    }

    const int g = h / (a.H / a.G);
    // the row whose sums this lane ends up with, the same as kSame - 1 neighbours
    constexpr int kSame = 16 / kRows;
    const int row = lane / kSame % kRows;
    const bool on = row < rows;
    const T *kp = static_cast<const T *>(a.k) + (t * a.G + g) * N + lane * V;
    const T *qp = static_cast<const T *>(a.q) + (t * a.G + g) * N + lane * V;
    const T *vp = static_cast<const T *>(a.v) + (t * a.H + h) * a.P + p0 + row;
    T *op = static_cast<T *>(a.o) + (t * a.H + h) * a.P + p0 + row;
    const float *gp = a.g ? a.g + t * a.H + h : nullptr;
    const float *bp = a.beta + t * a.H + h;

    // the next token's operands are fetched while the current one is worked on
    T kn[V], qn[V], vn = from_f32<T>(0.f);
    float gn = 0.f, bn = 0.f;
    auto fetch = [&]() {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            kn[i] = kp[i];
            qn[i] = qp[i];
        }
        if (on) vn = *vp;
        if (gp) gn = *gp;
        bn = *bp;
        kp += (int64_t)a.G * N;
        qp += (int64_t)a.G * N;
        vp += (int64_t)a.H * a.P;
        bp += a.H;
        if (gp) gp += a.H;
    };
    if (t < end) fetch();
    for (; t < end; ++t) {
        float k[V], q[V], kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            k[i] = to_f32(kn[i]);
            q[i] = to_f32(qn[i]);
            kk = fmaf(k[i], k[i], kk);
            qq = fmaf(q[i], q[i], qq);
            kq = fmaf(k[i], q[i], kq);
        }
        const float v = to_f32(vn), beta = bn, decay = gp ? expf(gn) : 1.f;
        if (t + 1 < end) fetch();

        // lane: sum index bit 4 (0: S k, 1: S q), then the row's bits; the lowest are duplicates
        float c[2 * kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x = fmaf(s[r][i], k[i], x);
                y = fmaf(s[r][i], q[i], y);
            }
            c[r] = x;
            c[kRows + r] = y;
        }
#pragma unroll
        for (int n = kRows, o = 16; n > 0; n >>= 1, o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float mine = up ? c[n + i] : c[i], other = up ? c[i] : c[n + i];
                c[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
        }
        float dot = c[0];
#pragma unroll
        for (int o = kSame / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        kq = warp_sum(kq);
        float rk = 1.f, rq = a.scale;
        if (a.l2norm) {
            rk = rsqrtf(warp_sum(kk) + kL2Eps);
            rq *= rsqrtf(warp_sum(qq) + kL2Eps);
        }
        // u times k's norm, so that the update takes k as it is
        dot *= decay;
        float u = beta * (v - dot * rk) * rk;
        const float ku = __shfl_xor_sync(0xffffffffu, u, 16);
        if (lane >= 16 && on && lane % kSame == 0) *op = from_f32<T>(rq * fmaf(ku, kq, dot));
        op += (int64_t)a.H * a.P;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float ur = __shfl_sync(0xffffffffu, u, kSame * r);
#pragma unroll
            for (int i = 0; i < V; ++i) s[r][i] = fmaf(decay, s[r][i], ur * k[i]);
        }
    }
    if (a.final_state) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (r < rows) store_state<V>(a.final_state + at + (int64_t)r * N, s[r]);
    }
}

template <typename T, int V>
cudaError_t launch_sized(const DeltaArgs &a, const int *status, cudaStream_t st)
{
    const int64_t states = (a.cu ? a.nseq : a.batch) * a.H;
    auto go = [&](auto kern, int rows) {
        const int pblocks = (a.P + rows * kWarps - 1) / (rows * kWarps);
        kern<<<(unsigned)(states * pblocks), kWarps * 32, 0, st>>>(a, status);
        return cudaGetLastError();
    };
    // fewer rows to a warp shorten its token while the launch has few warps for an SM quarter (float32,
    // heads of 64 x 128, us with 8, 4 and 2 rows: 1500 tokens, 8 heads 785, 606, 556; 500 tokens, 37 heads
    // 264, 204, 240; 74 heads 264, 253, 324; 148 heads 344, 367, 591; one token, 128 x 80 heads 100, 101, 152)
    constexpr int64_t kQuarters = 148 * 4;
    if (states * a.P <= 2 * kQuarters) return go(delta_recurrent_kernel<T, V, 2>, 2);
    if (states * a.P <= 8 * kQuarters) return go(delta_recurrent_kernel<T, V, 4>, 4);
    return go(delta_recurrent_kernel<T, V, 8>, 8);
}

template <typename T>
cudaError_t launch_typed(const DeltaArgs &a, const int *status, cudaStream_t st)
{
    switch (a.N) {
    case 32: return launch_sized<T, 1>(a, status, st);
    case 64: return launch_sized<T, 2>(a, status, st);
    case 128: return launch_sized<T, 4>(a, status, st);
    case 256: return launch_sized<T, 8>(a, status, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

bool delta_recurrent_supported(int N) { return N == 32 || N == 64 || N == 128 || N == 256; }

cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool is_bf16, const int *status,
                                   cudaStream_t st)
{
    return is_bf16 ? launch_typed<bf16>(a, status, st) : launch_typed<float>(a, status, st);
}

}  // namespace ssd
