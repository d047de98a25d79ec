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
// the CTAs walk the rows with their slice of w in registers and the next rows on their way.
// Measured (bf16): 16384 x 2560 with a residual 64 us, 80 % of the copy bandwidth, its backward 73 us;
// 8191 x 5120 gated, e4m3 by groups of 128, 50 us (65 %, issue slots); 98304 x 64 gated backward 20.5 us.
// The backward of rows above 8192 values holds weights, their gradients and up to three operands in
// registers that do not suffice (0.2 to 2 KB a thread go to local memory; value by value above 4096
// already): 8192 rows of 16384 run at 60 to 79 % of the copy bandwidth, gated 48 to 53 %, of 16383 at 18 %,
// gated 20 %.
#include <algorithm>
#include <atomic>

#include "api.cuh"
#include "common.cuh"
#include "delta.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace {

using namespace sm100;

constexpr int kRowThreads = 256;   // CTA of the lanes-per-row variants
constexpr int kMaxDim = 16384;
constexpr int kMaxRowThreads = 512;
constexpr int kBwdCtas = 608;      // most CTAs of the backward: four per SM, each with a row of
                                   // partial weight gradients (a multiple of 32)
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1e-30f;

// What a launch computes besides the norm: the kernels' variants.
enum : int { kPlain, kResidual, kPre, kPost };
enum : int { kNoQuant, kPerRow, kPerGroup };

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
template <> struct __align__(8) Pack<float, 2> {
    float2 v;
    __device__ __forceinline__ void get(float (&f)[2]) const { f[0] = v.x; f[1] = v.y; }
    __device__ __forceinline__ void set(const float (&f)[2]) { v = make_float2(f[0], f[1]); }
};
template <> struct __align__(4) Pack<bf16, 2> {
    __nv_bfloat162 v;
    __device__ __forceinline__ void get(float (&f)[2]) const
    {
        const float2 p = __bfloat1622float2(v);
        f[0] = p.x; f[1] = p.y;
    }
    __device__ __forceinline__ void set(const float (&f)[2]) { v = __floats2bfloat162_rn(f[0], f[1]); }
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
template <typename T> __device__ __forceinline__ void store_one(void *base, int64_t at, float f)
{
    static_cast<T *>(base)[at] = from_f32<T>(f);
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
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint16_t *>(to) = e4m3x2(f[0], f[1]);
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

// 1 / (1 + 2^(-z log2(e))), each step to about 2^-22; far from 0 exactly 0 or 1.
__device__ __forceinline__ float sigmoid(float z)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// x <- x y for a thread's vector (y: another vector, or one factor), and the two halves of the sum
// of squares.
template <int VEC> __device__ __forceinline__ void times(float (&x)[VEC], const float (&y)[VEC])
{
    if constexpr (VEC == 1) x[0] *= y[0];
    else
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
            unpair(mul2(pair(x[i], x[i + 1]), pair(y[i], y[i + 1])), x[i], x[i + 1]);
}
template <int VEC> __device__ __forceinline__ void plus(float (&x)[VEC], const float (&y)[VEC])
{
    if constexpr (VEC == 1) x[0] += y[0];
    else
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
            unpair(add2(pair(x[i], x[i + 1]), pair(y[i], y[i + 1])), x[i], x[i + 1]);
}
template <int VEC> __device__ __forceinline__ void times(float (&x)[VEC], float f)
{
    if constexpr (VEC == 1) x[0] *= f;
    else
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
            unpair(mul2(pair(x[i], x[i + 1]), pair(f, f)), x[i], x[i + 1]);
}
template <int VEC>
__device__ __forceinline__ void add_products(uint64_t &sum, const float (&x)[VEC],
                                             const float (&y)[VEC])
{
    if constexpr (VEC == 1) sum = fma2(pair(x[0], 0.f), pair(y[0], 0.f), sum);
    else
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
            sum = fma2(pair(x[i], x[i + 1]), pair(y[i], y[i + 1]), sum);
}
__device__ __forceinline__ float both(uint64_t p)
{
    float x, y;
    unpair(p, x, y);
    return x + y;
}

// Reduces a (a sum) and b (a sum or a maximum, or not at all) over the threads of a row.  TPR: lanes
// per row, 0 for the whole CTA; `buf` alternates between two halves from row to row, so that one
// barrier per row is enough.
enum : int { kAlone, kSum, kMax };
template <int kOther> __device__ __forceinline__ void reduce_step(float &a, float &b, int o)
{
    a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (kOther != kAlone) {
        const float other = __shfl_xor_sync(0xffffffffu, b, o);
        b = kOther == kMax ? max_nan(b, other) : b + other;
    }
}
template <int TPR, int kOther>
__device__ __forceinline__ void reduce_row(float &a, float &b, float2 *red, int buf)
{
    constexpr int W = TPR == 0 ? 32 : TPR;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) reduce_step<kOther>(a, b, o);
    if constexpr (TPR == 0) {   // every warp reduces the warps' results (at most 16) again
        const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
        float2 *r = red + buf * (kMaxRowThreads / 32);
        if (lane == 0) r[threadIdx.x / 32] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane % 16 < warps ? r[lane % 16] : make_float2(0.f, 0.f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) reduce_step<kOther>(a, b, o);
    }
}

// How a CTA walks the rows, and this thread's share of a row: vectors j * threads + lane of VEC
// elements, j < NV.  Rows of whole 16-byte vectors are taken in these; other rows in pairs, those that
// start at an odd element one element earlier, so that a pair is aligned and only the row's ends are
// taken one by one (3e7 bf16 values in rows of 7001 with a residual: 82 us, element by element 283, in
// rows of 7000 52), the next row's in registers; element by element where a tensor starts between
// pairs.  The operands' vectors of 16 bytes come some rows ahead through a ring in shared memory
// (cp.async); a thread reads what it copied itself, so the ring needs no barrier.
// With the next row in registers instead, 16384 x 2560 ran at 72 % (residual) and its backward
// at 33 % of the copy bandwidth: too few warps fitted.
__host__ __device__ constexpr int rows_ahead(int nv) { return nv == 1 ? 3 : nv == 2 ? 2 : 1; }
template <typename T, int VEC, int NV, int TPR, int kOps> struct Walk {
    static constexpr bool kRing = sizeof(T) * VEC == 16;
    int tpr, lane, sub, dim, shift;
    int64_t row, step, rows;
    bool on[NV];     // some of vector j is in the row; all of it
    bool full[NV];
    uint32_t slot;   // this thread's first slot in the ring
    int turn;
    // without a ring: this row's vectors and, where a thread has few of them, the next row's
    static constexpr bool kNext = !kRing && NV * VEC * sizeof(T) <= 32;
    Pack<T, VEC> now[kOps][kRing ? 1 : NV], then[kOps][kNext ? NV : 1];
    const void *op[kOps];

    __device__ __forceinline__ Walk(const NormArgs &a, char *ring) : dim(a.dim), rows(a.rows), turn(0)
    {
        tpr = TPR == 0 ? (int)blockDim.x : TPR;
        lane = TPR == 0 ? threadIdx.x : threadIdx.x % tpr;
        sub = TPR == 0 ? 0 : threadIdx.x / tpr;
        const int per_cta = TPR == 0 ? 1 : kRowThreads / tpr;
        step = (int64_t)gridDim.x * per_cta;   // even where a thread has several rows of odd width
        row = (int64_t)blockIdx.x * per_cta + sub;
        shift = VEC == 2 ? (int)(row & dim & 1) : 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            full[j] = col(j) >= 0 && col(j) + VEC <= dim;
            on[j] = VEC == 2 ? col(j) < dim : full[j];
        }
        slot = smem_u32(ring) + threadIdx.x * 16;
    }
    __device__ __forceinline__ int col(int j) const { return (j * tpr + lane) * VEC - shift; }
    __device__ __forceinline__ int64_t at(int j) const { return row * dim + col(j); }
    // of a vector at the row's end: whether element i is in the row
    __device__ __forceinline__ bool in(int j, int i) const
    {
        return (unsigned)(col(j) + i) < (unsigned)dim;
    }
    __device__ __forceinline__ uint32_t place(int o, int j) const
    {
        return slot + ((turn * kOps + o) * NV + j) * blockDim.x * 16;
    }
    // copies of the row `ahead` turns on into the present turn's slots
    __device__ __forceinline__ void prefetch(int ahead)
    {
        if constexpr (kRing) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                if (row + ahead * step >= rows || !on[j]) continue;
#pragma unroll
                for (int o = 0; o < kOps; ++o)
                    cp16(place(o, j), static_cast<const T *>(op[o]) + at(j) + ahead * step * dim, true);
            }
            cp_commit();
        }
    }
    // All vectors of a row, whatever is missing as zeros.  A pair across the row's end is read whole --
    // its other half is the neighbouring row's -- but for the tensor's last element.
    __device__ __forceinline__ void fetch(int64_t r, Pack<T, VEC> (*to)[NV]) const
    {
        const int64_t end = rows * dim;
#pragma unroll
        for (int o = 0; o < kOps; ++o)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int64_t i = r * dim + col(j);
                const T *from = static_cast<const T *>(op[o]) + i;
                float f[VEC] = {};
                Pack<T, VEC> p;
                p.set(f);
                if (r < rows && on[j]) {
                    if (VEC == 1 || i + VEC <= end) {
                        p = *reinterpret_cast<const Pack<T, VEC> *>(from);
                    } else {
                        f[0] = to_f32(*from);
                        p.set(f);
                    }
                }
                to[o][j] = p;
            }
    }
    __device__ __forceinline__ void start()
    {
        if constexpr (kRing) {
            for (int i = 0; i < rows_ahead(NV); ++i) {
                prefetch(i);
                turn = turn + 1 == rows_ahead(NV) ? 0 : turn + 1;
            }
        } else if constexpr (kNext) {
            fetch(row, then);
        }
    }
    // this row's vectors are there
    __device__ __forceinline__ void arrived()
    {
        if constexpr (kRing) {
            cp_wait<rows_ahead(NV) - 1>();
        } else if constexpr (kNext) {
#pragma unroll
            for (int o = 0; o < kOps; ++o)
#pragma unroll
                for (int j = 0; j < NV; ++j) now[o][j] = then[o][j];
            fetch(row + step, then);
        } else {
            fetch(row, now);
        }
    }
    // this thread's vector j of operand o
    __device__ __forceinline__ Pack<T, VEC> get(int o, int j) const
    {
        Pack<T, VEC> p;
        if constexpr (kRing) {
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(place(o, j)) : "memory");
            memcpy(&p, &v, 16);
        } else {
            p = now[o][j];
            if (VEC == 2 && !full[j]) {
                float f[VEC];
                p.get(f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = in(j, i) ? f[i] : 0.f;
                p.set(f);
            }
        }
        return p;
    }
    // the next row; call it once this row's vectors have been used
    __device__ __forceinline__ void next()
    {
        if constexpr (kRing) {
            prefetch(rows_ahead(NV));
            turn = turn + 1 == rows_ahead(NV) ? 0 : turn + 1;
        }
        row += step;
    }
    // the CTA's rows; the last ones may lie behind the end for some threads, which then only take
    // part in the reductions
    __device__ __forceinline__ bool more() const { return row - sub < rows; }
    __device__ __forceinline__ bool live() const { return row < rows; }
    __device__ __forceinline__ void put(void *to, int j, const float (&f)[VEC]) const
    {
        if (VEC != 2 || full[j]) {
            Pack<T, VEC> p;
            p.set(f);
            *reinterpret_cast<Pack<T, VEC> *>(static_cast<T *>(to) + at(j)) = p;
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (in(j, i)) store_one<T>(to, at(j) + i, f[i]);
        }
    }
    // this thread's weights, zeros outside the row
    __device__ __forceinline__ void weights(const float *w, float (&f)[NV][VEC]) const
    {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[j][i] = VEC == 2 && in(j, i) ? w[col(j) + i] : 0.f;
            if constexpr (VEC != 2) {
                if (on[j]) load_w<VEC>(w + col(j), f[j]);
            }
        }
    }
};

__host__ __device__ constexpr int norm_ops(int mode) { return mode == kPlain ? 1 : 2; }
__host__ __device__ constexpr int norm_bwd_ops(int mode) { return mode == kPlain ? 2 : 3; }

template <typename T, int VEC, int NV, int TPR, int kMode, int kQuant>
__global__ void __launch_bounds__(TPR == 0 ? kMaxRowThreads : kRowThreads)
rms_norm_kernel(const NormArgs a)
{
    __shared__ float2 red[2 * (kMaxRowThreads / 32)];
    extern __shared__ __align__(16) char ring[];
    const int dim = a.dim;
    const float inv_dim = 1.f / (float)dim;
    Walk<T, VEC, NV, TPR, norm_ops(kMode)> w(a, ring);
    w.op[0] = a.x;
    if constexpr (kMode != kPlain) w.op[1] = kMode == kResidual ? a.residual : a.z;
    w.start();
    float wt[NV][VEC];
    w.weights(a.w, wt);
    for (int buf = 0; w.more(); buf ^= 1) {
        const bool live = w.live();
        float h[NV][VEC];
        float top = 0.f;
        uint64_t sums = 0;
        w.arrived();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float other[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[j][i] = other[i] = 0.f;
            if (live && w.on[j]) {
                w.get(0, j).get(h[j]);
                if constexpr (kMode != kPlain) w.get(1, j).get(other);
                if constexpr (kMode == kResidual) {
                    Pack<T, VEC> sum;
                    plus(h[j], other);
                    sum.set(h[j]);
                    sum.get(h[j]);
                    w.put(a.res_out, j, h[j]);
                }
            }
            if constexpr (kMode == kPre || kMode == kPost) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) other[i] *= sigmoid(other[i]);
            }
            if constexpr (kMode == kPre) times(h[j], other);
            add_products(sums, h[j], h[j]);
            times(h[j], wt[j]);
            if constexpr (kMode == kPost) times(h[j], other);
            if constexpr (kQuant == kPerRow) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) top = max_nan(top, fabsf(h[j][i]));
            }
        }
        float ss = both(sums);
        reduce_row<TPR, kQuant == kPerRow ? kMax : kAlone>(ss, top, red, buf);
        const float r = rsqrtf(fmaf(ss, inv_dim, a.eps));
        float scale = max_nan(top * r * (1.f / kE4m3Max), kMinScale);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = w.col(j);
            times(h[j], r);
            if constexpr (kQuant != kNoQuant) {
                if constexpr (kQuant == kPerGroup) {   // 32, 64 or 128 elements: their lanes
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) m = max_nan(m, fabsf(h[j][i]));
                    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    if (VEC == 4 || a.quant > 32)
                        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    if (a.quant > (VEC == 4 ? 32 : 64))
                        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    if (VEC == 4 && a.quant > 64)
                        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    scale = max_nan(m * (1.f / kE4m3Max), kMinScale);
                }
                if (!live || !w.on[j]) continue;
                if constexpr (kQuant == kPerRow) {
                    if (j == 0 && w.lane == 0) a.scales[w.row] = scale;
                } else if ((e & (a.quant - 1)) == 0) {
                    const int shift = 31 - __clz(a.quant);
                    a.scales[w.row * (dim >> shift) + (e >> shift)] = scale;
                }
                float inv;   // of a scale between 1e-30 and 1e36: to 2^-23
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
                times(h[j], inv);
                uint8_t *to = a.y8 + w.at(j);
                if (VEC != 2 || w.full[j]) {
                    store_e4m3<VEC>(to, h[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (w.in(j, i)) to[i] = (uint8_t)e4m3x2(h[j][i], 0.f);
                }
            } else {
                if (!live || !w.on[j]) continue;
                w.put(a.y, j, h[j]);
            }
        }
        w.next();
    }
}

// The same walk.  The operands stay in registers as loaded (bf16 in half of them) and are taken
// apart again behind the reduction; the gate's sigmoid is formed again, too.
template <typename T, int VEC, int NV, int TPR, int kMode>
__global__ void __launch_bounds__(TPR == 0 ? kMaxRowThreads : kRowThreads)
rms_norm_bwd_kernel(const NormArgs a)
{
    __shared__ float2 red[2 * (kMaxRowThreads / 32)];
    extern __shared__ __align__(16) char ring[];
    constexpr bool kGated = kMode == kPre || kMode == kPost;
    const int dim = a.dim;
    const float inv_dim = 1.f / (float)dim;
    Walk<T, VEC, NV, TPR, norm_bwd_ops(kMode)> w(a, ring);
    w.op[0] = a.x;
    w.op[1] = a.dy;
    if constexpr (kMode != kPlain) w.op[2] = kGated ? a.z : a.dres;
    w.start();
    float wt[NV][VEC], dw[NV][VEC] = {};
    w.weights(a.w, wt);
    for (int buf = 0; w.more(); buf ^= 1) {
        const bool live = w.live();
        Pack<T, VEC> xp[NV], yp[NV], tp[NV];
        uint64_t sums = 0, dots = 0;
        w.arrived();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!live || !w.on[j]) continue;
            xp[j] = w.get(0, j);
            yp[j] = w.get(1, j);
            if constexpr (kMode != kPlain) tp[j] = w.get(2, j);
            float x[VEC], dy[VEC], z[VEC];
            xp[j].get(x);
            yp[j].get(dy);
            if constexpr (kGated) tp[j].get(z);
            if constexpr (kGated) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) z[i] *= sigmoid(z[i]);
                if constexpr (kMode == kPre) times(x, z);
                else times(dy, z);
            }
            add_products(sums, x, x);
            times(dy, wt[j]);
            add_products(dots, dy, x);
        }
        float ss = both(sums), dot = both(dots);
        reduce_row<TPR, kSum>(ss, dot, red, buf);
        const float r = rsqrtf(fmaf(ss, inv_dim, a.eps));
        const float c = dot * inv_dim * r * r * r;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!live || !w.on[j]) continue;
            float x[VEC], dy[VEC], t[VEC], dx[VEC], dz[VEC];
            xp[j].get(x);
            yp[j].get(dy);
            if constexpr (kMode != kPlain) tp[j].get(t);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float h = x[i], dn = dy[i], s = 0.f, slope = 0.f;
                if constexpr (kGated) {   // silu and its derivative
                    const float g = sigmoid(t[i]);
                    s = t[i] * g;
                    slope = g * fmaf(t[i], 1.f - g, 1.f);
                    if constexpr (kMode == kPre) h *= s;
                    else dn *= s;
                }
                const float n = h * r;
                const float dh = fmaf(r * dn, wt[j][i], -h * c);
                dw[j][i] = fmaf(dn, n, dw[j][i]);
                dx[i] = kMode == kPre ? dh * s : kMode == kResidual ? dh + t[i] : dh;
                if constexpr (kGated)
                    dz[i] = (kMode == kPre ? dh * x[i] : dy[i] * n * wt[j][i]) * slope;
            }
            w.put(a.dx, j, dx);
            if constexpr (kGated) w.put(a.dz, j, dz);
        }
        w.next();
    }
    let_next_start();
    // this CTA's partial weight gradient: one row of `dw_part`
    if constexpr (TPR == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (w.on[j])
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (VEC != 2 || w.in(j, i))
                        a.dw_part[(int64_t)blockIdx.x * dim + w.col(j) + i] = dw[j][i];
    } else {   // the CTA's rows are added up in order, in the ring's place
        constexpr int kPer = kRowThreads / (TPR == 0 ? kRowThreads : TPR);
        float *part = reinterpret_cast<float *>(ring);   // kPer x dim
        cp_wait<0>();
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (w.on[j])
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (VEC != 2 || w.in(j, i)) part[w.sub * dim + w.col(j) + i] = dw[j][i];
        __syncthreads();
        for (int e = threadIdx.x; e < dim; e += kRowThreads) {
            float s = 0.f;
            for (int k = 0; k < kPer; ++k) s += part[k * dim + e];
            a.dw_part[(int64_t)blockIdx.x * dim + e] = s;
        }
    }
}

// dw[e] = the sum of n rows of partial sums: 32 columns per CTA, the rows dealt to 32 warps, the
// warps' sums added in order, so repeated calls give the same bits.  (Dealt to 8 warps it took
// 25 us for 592 rows of 2560: the loads' latency, 19 times over.)
__global__ void __launch_bounds__(1024)
rms_norm_dw_kernel(const float *part, float *dw, int n, int dim)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, col = blockIdx.x * 32 + lane;
    float s[4] = {};
    wait_before();
    if (col < dim) {
        const float *p = part + col;
#pragma unroll
        for (int k = 0; k < kBwdCtas / 32; k += 4) {   // all loads at once
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = warp + (k + i) * 32;
                s[i] += k + i < kBwdCtas / 32 && r < n ? p[(int64_t)r * dim] : 0.f;
            }
        }
    }
    sums[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    float t = sums[lane][warp];   // column `warp`, a lane per row warp
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0 && blockIdx.x * 32 + warp < dim) dw[blockIdx.x * 32 + warp] = t;
}

// Of the current device; asked once per device.
int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) != cudaSuccess) return n;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed))) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Launches a walk of `rows` rows, per_cta at a time, on as many CTAs as the GPU holds at once.  `smem_most`
// is what the kernel's widest rows take: every call sets that limit, so that calls of several host
// threads, of rows of different widths, never lower it between another one's set and launch.
template <typename K>
cudaError_t launch_walk(K kern, const NormArgs &a, int per_cta, int threads, size_t smem,
                        size_t smem_most, int64_t most, int64_t *ctas, cudaStream_t st)
{
    cudaError_t e;
    if (smem > 40 * 1024) {   // with the static part this may pass 48 KB
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_most);
        if (e != cudaSuccess) return e;
    }
    int64_t grid = (a.rows + per_cta - 1) / per_cta;
    const int64_t sms = sm_count();
    if (grid > sms) {
        int per_sm = 1;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
        if (e != cudaSuccess) return e;
        if (grid > sms * per_sm) grid = sms * (per_sm > 0 ? per_sm : 1);
    }
    if (grid > most) grid = most;
    if (grid * per_cta < a.rows && grid > 1) grid &= ~int64_t(1);   // rows of odd width: see Walk
    if (ctas) *ctas = grid;
    kern<<<(unsigned)grid, threads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int VEC, int NV, int TPR, int kMode>
cudaError_t launch(const NormArgs &a, bool bwd, int threads, float *dw, cudaStream_t st)
{
    const int per_cta = TPR == 0 ? 1 : kRowThreads / TPR;
    constexpr size_t kSlots = sizeof(T) * VEC == 16 ? (size_t)rows_ahead(NV) * NV * 16 : 0;
    const size_t slots = kSlots * threads;   // bytes of an operand's ring
    constexpr size_t kMost = kSlots * (TPR == 0 ? kMaxRowThreads : kRowThreads);
    static_assert(TPR == 0 || kMost * 3 <= 40 * 1024, "needs no limit of its own");
    if (!bwd) {
        const size_t smem = slots * norm_ops(kMode);
        auto go = [&](auto kern) {
            return launch_walk(kern, a, per_cta, threads, smem, kMost * norm_ops(kMode), 1 << 30, nullptr,
                               st);
        };
        if (!a.quant) return go(rms_norm_kernel<T, VEC, NV, TPR, kMode, kNoQuant>);
        if (a.quant == a.dim) return go(rms_norm_kernel<T, VEC, NV, TPR, kMode, kPerRow>);
        if constexpr (VEC > 2)   // a group of 32 or more divides dim: whole vectors
            return go(rms_norm_kernel<T, VEC, NV, TPR, kMode, kPerGroup>);
        return cudaErrorInvalidValue;
    }
    size_t smem = slots * norm_bwd_ops(kMode);
    const size_t part = TPR == 0 ? 0 : (size_t)per_cta * a.dim * sizeof(float);
    smem = std::max(smem, part);
    int64_t ctas = 0;
    cudaError_t e = launch_walk(rms_norm_bwd_kernel<T, VEC, NV, TPR, kMode>, a, per_cta, threads,
                                smem, kMost * norm_bwd_ops(kMode), kBwdCtas, &ctas, st);
    if (e != cudaSuccess) return e;
    return launch_after(rms_norm_dw_kernel, (a.dim + 31) / 32, 1024, 0, st, a.dw_part, dw, (int)ctas,
                        a.dim);
}

// Threads of a CTA that takes one row of `vecs` vectors, NV per thread.
int row_threads(int vecs, int nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; }

// Rows of up to 32 vectors on 8, 16 or 32 lanes (no barrier), longer ones on a CTA with as few
// vectors per thread as its 512 threads allow.
template <typename T, int kMode>
cudaError_t launch_vectors(const NormArgs &a, bool bwd, float *dw, cudaStream_t st)
{
    constexpr int VEC = 16 / sizeof(T);
    const int vecs = a.dim / VEC;
    if (vecs <= 8) return launch<T, VEC, 1, 8, kMode>(a, bwd, kRowThreads, dw, st);
    if (vecs <= 16) return launch<T, VEC, 1, 16, kMode>(a, bwd, kRowThreads, dw, st);
    if (vecs <= 32) return launch<T, VEC, 1, 32, kMode>(a, bwd, kRowThreads, dw, st);
    if (vecs <= kMaxRowThreads)
        return launch<T, VEC, 1, 0, kMode>(a, bwd, row_threads(vecs, 1), dw, st);
    if (vecs <= 2 * kMaxRowThreads)
        return launch<T, VEC, 2, 0, kMode>(a, bwd, row_threads(vecs, 2), dw, st);
    if (vecs <= 4 * kMaxRowThreads)
        return launch<T, VEC, 4, 0, kMode>(a, bwd, row_threads(vecs, 4), dw, st);
    if constexpr (VEC == 4)
        return launch<T, VEC, 8, 0, kMode>(a, bwd, row_threads(vecs, 8), dw, st);
    return cudaErrorInvalidValue;   // not reached: kMaxDim elements fit
}

// The same in pairs (a row of odd width may take one more): up to 128 of them on a warp.
template <typename T, int kMode>
cudaError_t launch_pairs(const NormArgs &a, bool bwd, float *dw, cudaStream_t st)
{
    const int pairs = a.dim / 2 + a.dim % 2;
    if (pairs <= 8) return launch<T, 2, 1, 8, kMode>(a, bwd, kRowThreads, dw, st);
    if (pairs <= 32) return launch<T, 2, 1, 32, kMode>(a, bwd, kRowThreads, dw, st);
    if (pairs <= 64) return launch<T, 2, 2, 32, kMode>(a, bwd, kRowThreads, dw, st);
    if (pairs <= 128) return launch<T, 2, 4, 32, kMode>(a, bwd, kRowThreads, dw, st);
    if (pairs <= 2 * kMaxRowThreads)
        return launch<T, 2, 2, 0, kMode>(a, bwd, row_threads(pairs, 2), dw, st);
    if (pairs <= 4 * kMaxRowThreads)
        return launch<T, 2, 4, 0, kMode>(a, bwd, row_threads(pairs, 4), dw, st);
    if (pairs <= 8 * kMaxRowThreads)
        return launch<T, 2, 8, 0, kMode>(a, bwd, row_threads(pairs, 8), dw, st);
    return launch<T, 2, 16, 0, kMode>(a, bwd, row_threads(pairs, 16), dw, st);
}

template <typename T, int kMode>
cudaError_t launch_elements(const NormArgs &a, bool bwd, float *dw, cudaStream_t st)
{
    if (a.dim <= 256) return launch<T, 1, 8, 32, kMode>(a, bwd, kRowThreads, dw, st);
    if (a.dim <= 8 * kMaxRowThreads)
        return launch<T, 1, 8, 0, kMode>(a, bwd, row_threads(a.dim, 8), dw, st);
    return launch<T, 1, 32, 0, kMode>(a, bwd, row_threads(a.dim, 32), dw, st);
}

template <typename T, int kMode>
cudaError_t launch_sized(const NormArgs &a, bool bwd, float *dw, cudaStream_t st)
{
    if (a.dim % (16 / sizeof(T)) == 0) return launch_vectors<T, kMode>(a, bwd, dw, st);
    // (a null pointer is aligned)
    const int n = 2 * sizeof(T);
    const bool pairs = api_aligned(a.x, n) && api_aligned(a.residual, n) && api_aligned(a.z, n) &&
                       api_aligned(a.dy, n) && api_aligned(a.dres, n) && api_aligned(a.dx, n) &&
                       api_aligned(a.dz, n) && api_aligned(a.res_out, n) &&
                       api_aligned(a.y, bwd || !a.quant ? n : 2);
    return pairs ? launch_pairs<T, kMode>(a, bwd, dw, st) : launch_elements<T, kMode>(a, bwd, dw, st);
}

template <typename T>
cudaError_t launch_mode(const NormArgs &a, bool bwd, float *dw, cudaStream_t st)
{
    if (a.gate == SSD_GATE_PRE) return launch_sized<T, kPre>(a, bwd, dw, st);
    if (a.gate == SSD_GATE_POST) return launch_sized<T, kPost>(a, bwd, dw, st);
    if (bwd ? a.dres : a.residual) return launch_sized<T, kResidual>(a, bwd, dw, st);
    return launch_sized<T, kPlain>(a, bwd, dw, st);
}

cudaError_t launch_norm(const NormArgs &a, bool is_bf16, bool bwd, float *dw, cudaStream_t st)
{
    return is_bf16 ? launch_mode<bf16>(a, bwd, dw, st) : launch_mode<float>(a, bwd, dw, st);
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
