// Root-mean-square norm of the block's rows, forward and backward:
//
//     h = x + residual (rounded to its storage type, which is what the residual stream keeps)
//     y = h r w,   r = 1 / sqrt(mean(h^2) + eps)          w (dim) float32
//
// gated by silu(z) before the norm (h = x silu(z)) or behind it (y = h r w silu(z)); y in the
// input's type, or as e4m3 values with one float32 scale amax / 448 per group of a row.
// Backward, with n = h r, dn = dy (times silu(z) for the gate behind the norm), per row:
//
//     dh = r dn w - h r^3 sum(dn w h) / dim,    dw = sum over rows of dn n
//
// HBM-bound: each row is read once into registers, reduced once -- sum(h^2) together with the
// row's largest |h w| (forward, one scale per row) or with sum(dn w h) (backward) -- and written.
// A row of up to 32 vectors belongs to 8, 16 or 32 lanes of a warp, a longer one to a whole CTA;
// the CTAs walk the rows with their slice of w in registers.
#include "api.cuh"
#include "common.cuh"

namespace ssd {
namespace {

constexpr int kRowThreads = 256;   // CTA of the lanes-per-row variants
constexpr int kMaxDim = 16384;
constexpr int kMaxRowThreads = 512;
constexpr int kBwdCtas = 592;      // most CTAs of the backward: four per SM, each with a row of
                                   // partial weight gradients
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1e-30f;

struct NormArgs {
    const void *x, *residual, *z, *dy, *dres;
    const float *w;
    void *y, *res_out, *dx, *dz;
    uint8_t *y8;
    float *scales, *dw_part;
    int64_t rows;
    int dim, gate, quant;
    float eps;
};

// VEC elements of T from / to global memory in one access.
template <typename T, int VEC> struct Pack;
template <> struct Pack<float, 1> {
    float v;
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v; }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = f[0]; }
};
template <> struct Pack<bf16, 1> {
    bf16 v;
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = __float2bfloat16_rn(f[0]); }
};
template <> struct __align__(16) Pack<float, 4> {
    float4 v;
    __device__ __forceinline__ void get(float (&f)[4]) const
    {
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
    __device__ __forceinline__ void set(const float (&f)[4])
    {
        v = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <> struct __align__(16) Pack<bf16, 8> {
    __nv_bfloat162 v[4];
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __bfloat1622float2(v[i]);
            f[2 * i] = p.x; f[2 * i + 1] = p.y;
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    }
};

template <typename T, int VEC>
__device__ __forceinline__ void load(const void *base, int64_t at, float (&f)[VEC])
{
    reinterpret_cast<const Pack<T, VEC> *>(static_cast<const T *>(base) + at)->get(f);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(void *base, int64_t at, const float (&f)[VEC])
{
    Pack<T, VEC> p;
    p.set(f);
    *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(base) + at) = p;
}
template <int VEC> __device__ __forceinline__ void load_w(const float *w, float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        f[0] = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(w + i);
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        }
    }
}

// Larger of two values, NaN if either is (so that a row with a NaN keeps it in its scale).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int VEC> __device__ __forceinline__ void store_e4m3(uint8_t *to, const float (&f)[VEC])
{
    if constexpr (VEC == 1) {
        *to = (uint8_t)e4m3x2(f[0], 0.f);
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint32_t *>(to) =
            (uint32_t)e4m3x2(f[0], f[1]) | ((uint32_t)e4m3x2(f[2], f[3]) << 16);
    } else {
        uint2 v;
        v.x = (uint32_t)e4m3x2(f[0], f[1]) | ((uint32_t)e4m3x2(f[2], f[3]) << 16);
        v.y = (uint32_t)e4m3x2(f[4], f[5]) | ((uint32_t)e4m3x2(f[6], f[7]) << 16);
        *reinterpret_cast<uint2 *>(to) = v;
    }
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// Reduces a (a sum) and b (a sum, or a maximum when kMax) over the threads of a row.  TPR: lanes
// per row, 0 for the whole CTA; `buf` alternates between two halves from row to row, so that one
// barrier per row is enough.
template <int TPR, bool kMax>
__device__ __forceinline__ void reduce_row(float &a, float &b, float2 *red, int buf)
{
    constexpr int W = TPR == 0 ? 32 : TPR;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const float other = __shfl_xor_sync(0xffffffffu, b, o);
        b = kMax ? max_nan(b, other) : b + other;
    }
    if constexpr (TPR == 0) {
        const int warps = blockDim.x / 32;
        float2 *r = red + buf * (kMaxRowThreads / 32);
        if (threadIdx.x % 32 == 0) r[threadIdx.x / 32] = make_float2(a, b);
        __syncthreads();
        a = 0.f;
        b = 0.f;
        for (int i = 0; i < warps; ++i) {
            const float2 v = r[i];
            a += v.x;
            b = kMax ? max_nan(b, v.y) : b + v.y;
        }
    }
}

template <int TPR> __device__ __forceinline__ int threads_per_row()
{
    return TPR == 0 ? (int)blockDim.x : TPR;
}

// A thread's elements of its row: vectors j * threads + lane of VEC elements, j < NV.
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(TPR == 0 ? kMaxRowThreads : kRowThreads)
rms_norm_kernel(const NormArgs a)
{
    __shared__ float2 red[2 * (kMaxRowThreads / 32)];
    const int tpr = threads_per_row<TPR>();
    const int rows_per_cta = TPR == 0 ? 1 : kRowThreads / tpr;
    const int lane = TPR == 0 ? threadIdx.x : threadIdx.x % tpr;
    const int dim = a.dim;
    const float inv_dim = 1.f / (float)dim;
    float w[NV][VEC];
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = (j * tpr + lane) * VEC;
        on[j] = e < dim;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[j][i] = 0.f;
        if (on[j]) load_w<VEC>(a.w + e, w[j]);
    }
    int buf = 0;
    const int64_t step = (int64_t)gridDim.x * rows_per_cta;
    const int64_t first = (int64_t)blockIdx.x * rows_per_cta;
    const int sub = TPR == 0 ? 0 : threadIdx.x / tpr;
    for (int64_t base = first; base < a.rows; base += step, buf ^= 1) {
        const int64_t row = base + sub;
        const bool live = row < a.rows;   // the others take part in the shuffles only
        float h[NV][VEC], gate[NV][VEC];
        float ss = 0.f, top = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t at = row * dim + (j * tpr + lane) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[j][i] = 0.f;
            if (live && on[j]) {
                load<T, VEC>(a.x, at, h[j]);
                if (a.residual) {
                    float r[VEC];
                    load<T, VEC>(a.residual, at, r);
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        h[j][i] = to_f32(from_f32<T>(h[j][i] + r[i]));
                    store<T, VEC>(a.res_out, at, h[j]);
                }
                if (a.gate) {
                    load<T, VEC>(a.z, at, gate[j]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float s = silu(gate[j][i]);
                        if (a.gate == 1) h[j][i] *= s;
                        else gate[j][i] = s;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                ss = fmaf(h[j][i], h[j][i], ss);
                float v = h[j][i] * w[j][i];
                if (a.gate == 2 && live && on[j]) v *= gate[j][i];
                h[j][i] = v;
                top = max_nan(top, fabsf(v));
            }
        }
        const bool per_row = a.quant == dim;
        reduce_row<TPR, true>(ss, top, red, buf);
        const float r = rsqrtf(fmaf(ss, inv_dim, a.eps));
        float scale = fmaxf(top * r / kE4m3Max, kMinScale);
        if (top != top) scale = top;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = (j * tpr + lane) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[j][i] *= r;
            if (a.quant && !per_row) {   // one scale per `quant` elements: quant / VEC lanes
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < VEC; ++i) m = max_nan(m, fabsf(h[j][i]));
                for (int o = a.quant / VEC / 2; o > 0; o >>= 1)
                    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                scale = fmaxf(m / kE4m3Max, kMinScale);
                if (m != m) scale = m;
            }
            if (!live || !on[j]) continue;
            if (a.quant) {
                if (e % a.quant == 0) a.scales[row * (dim / a.quant) + e / a.quant] = scale;
                const float inv = 1.f / scale;
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[j][i] *= inv;
                store_e4m3<VEC>(a.y8 + row * dim + e, h[j]);
            } else {
                store<T, VEC>(a.y, row * dim + e, h[j]);
            }
        }
    }
}

template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(TPR == 0 ? kMaxRowThreads : kRowThreads)
rms_norm_bwd_kernel(const NormArgs a)
{
    __shared__ float2 red[2 * (kMaxRowThreads / 32)];
    const int tpr = threads_per_row<TPR>();
    const int rows_per_cta = TPR == 0 ? 1 : kRowThreads / tpr;
    const int lane = TPR == 0 ? threadIdx.x : threadIdx.x % tpr;
    const int dim = a.dim;
    const float inv_dim = 1.f / (float)dim;
    float w[NV][VEC], dw[NV][VEC];
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = (j * tpr + lane) * VEC;
        on[j] = e < dim;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[j][i] = dw[j][i] = 0.f;
        if (on[j]) load_w<VEC>(a.w + e, w[j]);
    }
    int buf = 0;
    const int64_t step = (int64_t)gridDim.x * rows_per_cta;
    const int64_t first = (int64_t)blockIdx.x * rows_per_cta;
    const int sub = TPR == 0 ? 0 : threadIdx.x / tpr;
    for (int64_t base = first; base < a.rows; base += step, buf ^= 1) {
        const int64_t row = base + sub;
        const bool live = row < a.rows;
        // x and z stay as loaded; dn w h and h h are reduced, then dn and h are formed again
        float x[NV][VEC], z[NV][VEC], dy[NV][VEC];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t at = row * dim + (j * tpr + lane) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] = dy[j][i] = z[j][i] = 0.f;
            if (live && on[j]) {
                load<T, VEC>(a.x, at, x[j]);
                load<T, VEC>(a.dy, at, dy[j]);
                if (a.gate) load<T, VEC>(a.z, at, z[j]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float h = x[j][i], dn = dy[j][i];
                if (a.gate) {
                    const float s = z[j][i] * sigmoid(z[j][i]);
                    if (a.gate == 1) h *= s;
                    else dn *= s;
                }
                ss = fmaf(h, h, ss);
                dot = fmaf(dn * w[j][i], h, dot);
            }
        }
        reduce_row<TPR, false>(ss, dot, red, buf);
        const float r = rsqrtf(fmaf(ss, inv_dim, a.eps));
        const float c = dot * inv_dim * r * r * r;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!live || !on[j]) continue;
            const int64_t at = row * dim + (j * tpr + lane) * VEC;
            float dx[VEC], dz[VEC];
            float dres[VEC];
            if (a.dres) load<T, VEC>(a.dres, at, dres);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float h = x[j][i], dn = dy[j][i], s = 0.f, slope = 0.f;
                if (a.gate) {   // silu and its derivative
                    const float g = sigmoid(z[j][i]);
                    s = z[j][i] * g;
                    slope = g * fmaf(z[j][i], 1.f - g, 1.f);
                    if (a.gate == 1) h *= s;
                    else dn *= s;
                }
                const float n = h * r;
                const float dh = fmaf(r * dn, w[j][i], -h * c);
                dw[j][i] = fmaf(dn, n, dw[j][i]);
                dx[i] = a.gate == 1 ? dh * s : a.dres ? dh + dres[i] : dh;
                dz[i] = (a.gate == 1 ? dh * x[j][i] : dy[j][i] * n * w[j][i]) * slope;
            }
            store<T, VEC>(a.dx, at, dx);
            if (a.gate) store<T, VEC>(a.dz, at, dz);
        }
    }
    // this CTA's partial weight gradient: one row of `dw_part`
    if constexpr (TPR == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (on[j])
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    a.dw_part[(int64_t)blockIdx.x * dim + (j * tpr + lane) * VEC + i] = dw[j][i];
    } else {   // the CTA's rows are added up in order
        extern __shared__ float part[];   // rows_per_cta x dim
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (on[j])
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    part[sub * dim + (j * tpr + lane) * VEC + i] = dw[j][i];
        __syncthreads();
        for (int e = threadIdx.x; e < dim; e += kRowThreads) {
            float s = 0.f;
            for (int k = 0; k < rows_per_cta; ++k) s += part[k * dim + e];
            a.dw_part[(int64_t)blockIdx.x * dim + e] = s;
        }
    }
}

// dw[e] = the sum of n rows of partial sums: 32 columns per CTA, the rows dealt to 8 warps, the
// warps' sums added in order, so repeated calls give the same bits.
__global__ void __launch_bounds__(256)
rms_norm_dw_kernel(const float *part, float *dw, int n, int dim)
{
    __shared__ float sums[8][32];
    const int col = blockIdx.x * 32 + threadIdx.x % 32, warp = threadIdx.x / 32;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    if (col < dim) {
        int r = warp;
        for (; r + 24 < n; r += 32) {
            s0 += part[(int64_t)r * dim + col];
            s1 += part[(int64_t)(r + 8) * dim + col];
            s2 += part[(int64_t)(r + 16) * dim + col];
            s3 += part[(int64_t)(r + 24) * dim + col];
        }
        for (; r < n; r += 8) s0 += part[(int64_t)r * dim + col];
    }
    sums[warp][threadIdx.x % 32] = (s0 + s1) + (s2 + s3);
    __syncthreads();
    if (warp == 0 && col < dim) {
        float s = 0.f;
        for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
        dw[col] = s;
    }
}

int sm_count()
{
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

int64_t bwd_ctas(int64_t rows, int rows_per_cta)
{
    const int64_t need = (rows + rows_per_cta - 1) / rows_per_cta;
    return need < kBwdCtas ? need : kBwdCtas;
}

template <typename T, int VEC, int NV, int TPR>
cudaError_t launch(const NormArgs &a, bool bwd, int threads, float *dw, cudaStream_t st)
{
    const int per_cta = TPR == 0 ? 1 : kRowThreads / TPR;
    const int64_t need = (a.rows + per_cta - 1) / per_cta;
    if (!bwd) {
        // enough CTAs to fill every SM's threads; each walks the rows with w in registers
        const int64_t most = (int64_t)sm_count() * (2048 / threads);
        rms_norm_kernel<T, VEC, NV, TPR>
            <<<(unsigned)(need < most ? need : most), threads, 0, st>>>(a);
        return cudaGetLastError();
    }
    const int64_t ctas = bwd_ctas(a.rows, per_cta);
    const size_t smem = TPR == 0 ? 0 : (size_t)per_cta * a.dim * sizeof(float);
    rms_norm_bwd_kernel<T, VEC, NV, TPR><<<(unsigned)ctas, threads, smem, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    rms_norm_dw_kernel<<<(a.dim + 31) / 32, 256, 0, st>>>(a.dw_part, dw, (int)ctas, a.dim);
    return cudaGetLastError();
}

// Threads of a CTA that takes one row of `vecs` vectors, NV per thread.
int row_threads(int vecs, int nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; }

// Rows of up to 32 vectors on 8, 16 or 32 lanes (no barrier), up to 128 vectors on a warp with
// four each, longer ones on a CTA with as few vectors per thread as its 512 threads allow.
template <typename T, int VEC>
cudaError_t launch_sized(const NormArgs &a, bool bwd, float *dw, cudaStream_t st)
{
    const int vecs = (a.dim + VEC - 1) / VEC;
    constexpr int kMost = 32 / VEC;   // vectors per thread that hold 32 elements
    if (vecs <= 8) return launch<T, VEC, 1, 8>(a, bwd, kRowThreads, dw, st);
    if (vecs <= 16) return launch<T, VEC, 1, 16>(a, bwd, kRowThreads, dw, st);
    if (vecs <= 32) return launch<T, VEC, 1, 32>(a, bwd, kRowThreads, dw, st);
    if (vecs <= 128) return launch<T, VEC, 4, 32>(a, bwd, kRowThreads, dw, st);
    if (vecs <= kMaxRowThreads) return launch<T, VEC, 1, 0>(a, bwd, row_threads(vecs, 1), dw, st);
    if (vecs <= 2 * kMaxRowThreads)
        return launch<T, VEC, 2, 0>(a, bwd, row_threads(vecs, 2), dw, st);
    if (vecs <= 4 * kMaxRowThreads)
        return launch<T, VEC, 4, 0>(a, bwd, row_threads(vecs, 4), dw, st);
    if constexpr (kMost > 4)
        return launch<T, VEC, kMost, 0>(a, bwd, row_threads(vecs, kMost), dw, st);
    return cudaErrorInvalidValue;   // not reached: kMaxDim elements fit
}

cudaError_t launch_norm(const NormArgs &a, bool is_bf16, bool bwd, float *dw, cudaStream_t st)
{
    if (is_bf16)
        return a.dim % 8 ? launch_sized<bf16, 1>(a, bwd, dw, st)
                         : launch_sized<bf16, 8>(a, bwd, dw, st);
    return a.dim % 4 ? launch_sized<float, 1>(a, bwd, dw, st)
                     : launch_sized<float, 4>(a, bwd, dw, st);
}

ssd_status check_norm(const ssd_norm_desc *d)
{
    if (!d) return api_fail(SSD_ERR_INVALID_ARG, "norm description is NULL");
    if (d->rows < 0) return api_fail(SSD_ERR_INVALID_ARG, "rows must be >= 0");
    if (d->dtype != SSD_F32 && d->dtype != SSD_BF16)
        return api_fail(SSD_ERR_INVALID_ARG, "dtype must be SSD_F32 or SSD_BF16");
    if (d->gate < SSD_GATE_NONE || d->gate > SSD_GATE_POST)
        return api_fail(SSD_ERR_INVALID_ARG, "gate must be an ssd_gate (got %d)", d->gate);
    if (!(d->eps >= 0.f)) return api_fail(SSD_ERR_INVALID_ARG, "eps must be >= 0");
    if (d->dim < 1 || d->dim > kMaxDim)
        return api_fail(SSD_ERR_UNSUPPORTED, "dim must be in 1..%d (got %lld)", kMaxDim,
                        (long long)d->dim);
    if (d->rows > (int64_t)1 << 40)
        return api_fail(SSD_ERR_UNSUPPORTED, "rows must be <= 2^40");
    const int q = d->quant_group;
    if (q != 0 && q != d->dim && !((q == 32 || q == 64 || q == 128) && d->dim % q == 0))
        return api_fail(SSD_ERR_UNSUPPORTED, "quant_group must be 0, dim, or 32, 64 or 128 dividing "
                        "dim (got %d for dim %lld)", q, (long long)d->dim);
    return SSD_OK;
}

// What the vector path (rows of whole 16-byte vectors) reads and writes must start on 16 bytes;
// otherwise elements of `size` bytes on their own size.
bool rows_aligned(const ssd_norm_desc *d, const void *p, int size = 0)
{
    const int e = d->dtype == SSD_BF16 ? 2 : 4;
    const bool vec = d->dim % (16 / e) == 0;
    return !p || api_aligned(p, vec ? 16 : size ? size : e);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_rms_norm(const ssd_norm_desc *d, const void *x, const void *residual,
                        const void *z, const float *weight, void *y, float *scales,
                        void *residual_out, void *stream)
{
    ssd_status st = check_norm(d);
    if (st != SSD_OK) return st;
    if ((d->gate != SSD_GATE_NONE) != (z != nullptr))
        return api_fail(SSD_ERR_INVALID_ARG, "z goes with a gate, and a gate with z");
    if ((residual == nullptr) != (residual_out == nullptr))
        return api_fail(SSD_ERR_INVALID_ARG, "residual and residual_out go together");
    if (residual && z)
        return api_fail(SSD_ERR_UNSUPPORTED, "a residual and a gate cannot be combined");
    if (d->rows == 0) return SSD_OK;
    if (!x || !weight || !y || (d->quant_group && !scales))
        return api_fail(SSD_ERR_INVALID_ARG,
                        "x, weight, y (and scales with quant_group) must be non-NULL");
    if (!rows_aligned(d, x) || !rows_aligned(d, residual) || !rows_aligned(d, z) ||
        !rows_aligned(d, residual_out) || !rows_aligned(d, y, d->quant_group ? 1 : 0) ||
        !rows_aligned(d, weight, 4) || !api_aligned(scales, 4))
        return api_fail(SSD_ERR_INVALID_ARG, "rows of whole 16-byte vectors and the weight must be "
                        "16-byte aligned, others aligned to their elements");
    NormArgs a = {};
    a.x = x;
    a.residual = residual;
    a.z = z;
    a.w = weight;
    a.y = y;
    a.y8 = static_cast<uint8_t *>(y);
    a.scales = scales;
    a.res_out = residual_out;
    a.rows = d->rows;
    a.dim = (int)d->dim;
    a.gate = d->gate;
    a.quant = d->quant_group;
    a.eps = d->eps;
    cudaError_t e = launch_norm(a, d->dtype == SSD_BF16, false, nullptr,
                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "RMS norm launch");
}

size_t ssd_rms_norm_bwd_workspace_size(const ssd_norm_desc *d)
{
    if (check_norm(d) != SSD_OK) return 0;
    return api_round256((size_t)kBwdCtas * d->dim * sizeof(float));
}

ssd_status ssd_rms_norm_bwd(const ssd_norm_desc *d, const void *x, const void *z,
                            const float *weight, const void *dy, const void *dresidual, void *dx,
                            void *dz, float *dweight, void *workspace, size_t workspace_bytes,
                            void *stream)
{
    ssd_status st = check_norm(d);
    if (st != SSD_OK) return st;
    if (d->quant_group)
        return api_fail(SSD_ERR_UNSUPPORTED, "the backward takes no quant_group");
    if ((d->gate != SSD_GATE_NONE) != (z != nullptr) || (z == nullptr) != (dz == nullptr))
        return api_fail(SSD_ERR_INVALID_ARG, "z and dz go with a gate, and a gate with them");
    if (dresidual && z)
        return api_fail(SSD_ERR_UNSUPPORTED, "a residual and a gate cannot be combined");
    if (!dweight || !api_aligned(dweight, 4))
        return api_fail(SSD_ERR_INVALID_ARG, "dweight must be non-NULL and aligned");
    cudaStream_t cst = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (d->rows == 0) {
        e = cudaMemsetAsync(dweight, 0, (size_t)d->dim * sizeof(float), cst);
        return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "clear dweight");
    }
    if (!x || !weight || !dy || !dx || !workspace)
        return api_fail(SSD_ERR_INVALID_ARG, "x, weight, dy, dx and workspace must be non-NULL");
    if (!rows_aligned(d, x) || !rows_aligned(d, z) || !rows_aligned(d, dy) ||
        !rows_aligned(d, dresidual) || !rows_aligned(d, dx) || !rows_aligned(d, dz) ||
        !rows_aligned(d, weight, 4))
        return api_fail(SSD_ERR_INVALID_ARG, "rows of whole 16-byte vectors and the weight must be "
                        "16-byte aligned, others aligned to their elements");
    if (!api_aligned(workspace, 256))
        return api_fail(SSD_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (workspace_bytes < ssd_rms_norm_bwd_workspace_size(d))
        return api_fail(SSD_ERR_INVALID_ARG, "workspace too small: need %zu bytes, got %zu",
                        ssd_rms_norm_bwd_workspace_size(d), workspace_bytes);
    NormArgs a = {};
    a.x = x;
    a.z = z;
    a.dy = dy;
    a.dres = dresidual;
    a.w = weight;
    a.dx = dx;
    a.dz = dz;
    a.dw_part = static_cast<float *>(workspace);
    a.rows = d->rows;
    a.dim = (int)d->dim;
    a.gate = d->gate;
    a.eps = d->eps;
    e = launch_norm(a, d->dtype == SSD_BF16, true, dweight, cst);
    return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "RMS norm backward launch");
}

}  // extern "C"
