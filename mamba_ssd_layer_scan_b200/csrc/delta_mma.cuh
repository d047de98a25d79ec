// Warp-level bf16 matrix products of the gated delta rule's chunked kernels: fragments, the split
// of a float32 into bf16 parts, shared-memory tiles; sums in two floats.
#pragma once

#include "sm100.cuh"

namespace ssd {

// D (16 x 8, float32) += A (16 x 16, bf16) B (16 x 8, bf16).  Lane l holds of D rows l/4 and
// l/4 + 8, columns 2 (l % 4) + {0, 1}; of A the same rows, columns 2 (l % 4) + {0, 1, 8, 9}; of B
// rows (k) 2 (l % 4) + {0, 1, 8, 9}, column l/4.  Two neighbouring D tiles are thus an A operand.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4_trans(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%4], {%0, %1, %2, %3};"
                 ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(addr) : "memory");
}

// a + b = s + err exactly
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &err)
{
    s = a + b;
    const float bb = s - a;
    err = (a - (s - bb)) + (b - bb);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// x and y as bf16 pairs: hi the roundings, lo the roundings of what they leave.  hi + lo is x to
// 2^-16 of it: products with an exact bf16 operand then keep float32's usual accuracy.
__device__ __forceinline__ void split2(uint64_t xy, uint32_t &hi, uint32_t &lo)
{
    float x, y;
    sm100::unpair(xy, x, y);
    hi = sm100::pack_bf16x2(x, y);
    sm100::unpair(sm100::fma2(sm100::pair(bf16_lo(hi), bf16_hi(hi)), sm100::pair(-1.f, -1.f), xy),
                  x, y);
    lo = sm100::pack_bf16x2(x, y);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    split2(sm100::pair(x, y), hi, lo);
}

// Three parts: hi + mid + lo is x to 2^-24 of it.
__device__ __forceinline__ void split3(uint64_t xy, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const uint64_t minus = sm100::pair(-1.f, -1.f);
    float x, y;
    sm100::unpair(xy, x, y);
    hi = sm100::pack_bf16x2(x, y);
    xy = sm100::fma2(sm100::pair(bf16_lo(hi), bf16_hi(hi)), minus, xy);
    sm100::unpair(xy, x, y);
    mid = sm100::pack_bf16x2(x, y);
    sm100::unpair(sm100::fma2(sm100::pair(bf16_lo(mid), bf16_hi(mid)), minus, xy), x, y);
    lo = sm100::pack_bf16x2(x, y);
}

// The two parts one at a time.
__device__ __forceinline__ uint32_t round2(uint64_t xy)
{
    float x, y;
    sm100::unpair(xy, x, y);
    return sm100::pack_bf16x2(x, y);
}
__device__ __forceinline__ uint32_t rest2(uint64_t xy)
{
    uint32_t hi, lo;
    split2(xy, hi, lo);
    return lo;
}

// The A operand made of two neighbouring D tiles.
__device__ __forceinline__ void split_a(const float (&t0)[4], const float (&t1)[4],
                                        uint32_t (&hi)[4], uint32_t (&lo)[4])
{
    split2(t0[0], t0[1], hi[0], lo[0]);
    split2(t0[2], t0[3], hi[1], lo[1]);
    split2(t1[0], t1[1], hi[2], lo[2]);
    split2(t1[2], t1[3], hi[3], lo[3]);
}
__device__ __forceinline__ void split_a(const float (&t0)[4], const float (&t1)[4],
                                        uint32_t (&hi)[4], uint32_t (&mid)[4], uint32_t (&lo)[4])
{
    split3(sm100::pair(t0[0], t0[1]), hi[0], mid[0], lo[0]);
    split3(sm100::pair(t0[2], t0[3]), hi[1], mid[1], lo[1]);
    split3(sm100::pair(t1[0], t1[1]), hi[2], mid[2], lo[2]);
    split3(sm100::pair(t1[2], t1[3]), hi[3], mid[3], lo[3]);
}
__device__ __forceinline__ void round_a(const float (&t0)[4], const float (&t1)[4],
                                        uint32_t (&hi)[4])
{
    hi[0] = sm100::pack_bf16x2(t0[0], t0[1]);
    hi[1] = sm100::pack_bf16x2(t0[2], t0[3]);
    hi[2] = sm100::pack_bf16x2(t1[0], t1[1]);
    hi[3] = sm100::pack_bf16x2(t1[2], t1[3]);
}

// 16 bytes from global to shared memory; zeros where `on` is false (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

}  // namespace ssd
