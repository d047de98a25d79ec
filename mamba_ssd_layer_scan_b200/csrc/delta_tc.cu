// The gated delta rule's forward in chunks of 64 tokens on tcgen05 (bf16, headdim 64 or 128,
// dstate 64 or 128).  With the terms of delta_chunk.cu, per chunk and state row p (a TMEM lane):
//
//     X = S K^T,  R = V^T - ek X,  W = R Inv^T,  S' = E S + (sw W) K,  O = eq (S Q^T) + W Att^T
//
// delta_tc_prep_kernel, parallel over chunks and heads, writes Inv, Att and the factors of the rows
// as the shared-memory image that the second kernel copies.  delta_tc_kernel takes 128 state rows --
// one head of 128, or two heads of 64 of one group -- through a sequence.  Every product has p on
// the accumulator's lanes, so each result, taken from TMEM by the thread that owns the row and
// written back as bf16, is the next product's A operand; the B operands (K, Q, Inv, Att) lie in
// shared memory, K serving both as rows (X) and as columns (S').  S, R, sw W and Inv enter as two bf16
// parts each, so that final states are 3e-6 off (float32 sums alone leave 3e-7).  Att W, which goes to the
// output alone, is a product of float32 operands cut to 10 bits, W read where its product left it.  (Of
// bf16 operands it was off by as much as the output's own rounding for each of the two, 0.0033 for 0.0017
// in all; in two bf16 parts each it took half as much again and the parts' making: packed 16384 tokens x
// 80 heads 487 us, this form 446, bf16 420.)  The state itself stays in registers, float32.  Two heads
// that share a CTA multiply all 128 rows by each head's triangles and read their own result: 2 x 64
// columns cost the same as a block-diagonal product, and what is not finite in one head stays there.
//
// Bound: the chain of a chunk, three products deep (500-700 cycles each) with the rows' splits and the
// hand-overs between them, 5400 cycles: 2 x 4096 tokens x 32 heads of 128 take 179 us, 64 chunks of 2.8 us,
// behind 60 us for the triangles; 16384 packed tokens x 80 heads of 64 270 us behind 158 us.  64 tokens
// to a chunk: of 32 the same products would have half the columns, and the hand-overs twice their share.
#include "delta.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace {

using namespace sm100;

constexpr int kC = kDeltaTcChunk;      // 64 tokens
constexpr int kTile = kC * 128;        // bytes of a 64 x 64 bf16 tile, rows 128-byte swizzled
constexpr float kLog2e = 1.4426950408889634f;   // and what it leaves of log2(e)
constexpr float kLog2eLow = 1.9259629911266175e-8f;

// A float cut to 10 bits of mantissa is smaller by a quantity spread evenly over [0, 2^(e-10)): in a sum
// by 2^-11 ln 2 of it, with mantissas as evenly spread as logarithms are.  Att and W are both cut.
constexpr float kCutBoth = 1.f + 2 * 0.693147f / 2048;

template <int I> struct Int { static constexpr int value = I; };

// ---------------------------------------------------------------- the triangles
// A triangle, 64 x 64 bf16 in 6 KB: columns 0-31 of all rows, then columns 32-63 of rows 32-63, in
// rows of 64 bytes, 64-byte swizzled; in float32 (Att) 12 KB, in rows of 128 bytes, 128-byte swizzled.
// An item, per chunk and head: Inv in two parts, Att, and the factors -ek, sw, eq (64 floats each) and E
// (four times).
constexpr int kMat = 6 * 1024, kMatRight = 4 * 1024, kAttRight = 8 * 1024;
constexpr int kMats = 4 * kMat, kItemAtt = 2 * kMat, kItemVec = kMats, kVecFloats = 3 * kC + 4;
constexpr int kItem = kDeltaTcItem, kItemUsed = kItemVec + kVecFloats * 4;
static_assert(kItemUsed <= kItem && kItemUsed % 16 == 0 && kItem % 1024 == 0, "an item");
// Byte offset of the 16-byte piece `c` (8 columns) of row `r` of a triangle.
__device__ __forceinline__ uint32_t tri_at(int r, int c)
{
    return (c < 4 ? r * 64 : kMatRight + (r - 32) * 64) + (((c ^ (r >> 1)) & 3) << 4);
}
// Of the 8 columns `n` of a row of the one in float32, from the place of the row's first 8 (128-byte
// aligned apart from the swizzle).
__device__ __forceinline__ uint32_t att_at(uint32_t first, int n)
{
    return (first ^ ((n & 3) << 5)) + (n < 4 ? 0 : kAttRight - 32 * 128);
}

constexpr int kPrepWarps = 4, kPrepThreads = 2 * kPrepWarps * 32, kPrepQuad = 4;
// what the builders need of a head: log2(e) cs and its low part, both negated, kb, w
constexpr int kCs = 0, kCl = kC, kKb = 2 * kC, kW = 3 * kC, kGateFloats = 4 * kC;
constexpr int kPrepGates = 2 * kMats,   // K and Q lie there first
              kPrepNorms = kPrepGates + 2 * kPrepQuad * kGateFloats * 4,
              kPrepSmem = kPrepNorms + 2 * kC * 4;
static_assert(kPrepGates >= 4 * kTile, "K and Q of 128 columns");

// Byte offset of 16-byte piece `c` of row `r` in a tile of 128-byte rows, 128-byte swizzled.
__device__ __forceinline__ uint32_t sw_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t v)
{
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t at, float a, float b)
{
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float4 lds128(uint32_t at)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float f32(uint32_t v) { return __uint_as_float(v); }
__device__ __forceinline__ uint64_t pair_u(uint32_t x, uint32_t y) { return pair(f32(x), f32(y)); }
// Two pairs of floats from shared memory.
__device__ __forceinline__ void lds_pairs(uint32_t at, uint64_t (&p)[2])
{
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(p[0]), "=l"(p[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint64_t lds_pair(uint32_t at)
{
    uint64_t p;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(p) : "r"(at) : "memory");
    return p;
}
// Shared to global memory by the TMA unit; its source may be written again after the wait.
__device__ __forceinline__ void bulk_store(void *to, uint32_t from, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                 ::"l"(to), "r"(from), "r"(bytes) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
// A head's gates in a chunk, a warp; lane l has tokens 2 l and 2 l + 1.  First the running sums of g
// (times log2(e), hi + lo) and beta.
struct Gates {
    float hi[2], lo[2], beta[2];
};
__device__ __forceinline__ Gates sum_gates(const DeltaArgs &a, int64_t row0, int len, int h)
{
    const int lane = threadIdx.x % 32, i = 2 * lane;
    Gates s = {};
    float g[2] = {};
#pragma unroll
    for (int y = 0; y < 2; ++y)
        if (i + y < len) {
            const int64_t at = (row0 + i + y) * a.H + h;
            if (a.g) g[y] = a.g[at];
            s.beta[y] = a.beta[at];
        }
#pragma unroll
    for (int y = 0; y < 2; ++y) g[y] = g[y] < -200.f ? -200.f : g[y];
    // sums in two floats: differences behind a token that wipes the state out (-200) stay accurate
    float cs[2], cl[2];
    cs[0] = g[0];
    two_sum(g[0], g[1], cs[1], cl[1]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {   // over the lanes' second tokens
        const float up = __shfl_up_sync(0xffffffffu, cs[1], o);
        const float ul = __shfl_up_sync(0xffffffffu, cl[1], o);
        if (lane >= o) {
            float t, e;
            two_sum(cs[1], up, t, e);
            cs[1] = t;
            cl[1] += ul + e;
        }
    }
    float before = __shfl_up_sync(0xffffffffu, cs[1], 1);
    float beforel = __shfl_up_sync(0xffffffffu, cl[1], 1);
    if (lane == 0) before = beforel = 0.f;
    two_sum(before, g[0], cs[0], cl[0]);
    cl[0] += beforel;
#pragma unroll
    for (int y = 0; y < 2; ++y) {   // the product's rounding kept as well
        s.hi[y] = cs[y] * kLog2e;
        s.lo[y] = fmaf(cs[y], kLog2e, -s.hi[y]) + fmaf(cs[y], kLog2eLow, cl[y] * kLog2e);
    }
    return s;
}
// Then the factors that come of them: `gates` for the builders, `vec` (global) for the chain.
__device__ __forceinline__ void make_factors(const Gates &s, int len, const float *norms, float *gates,
                                             float *vec)
{
    const int lane = threadIdx.x % 32, i = 2 * lane;
    const float(&hi)[2] = s.hi;
    const float(&lo)[2] = s.lo;
    const float end = __shfl_sync(0xffffffffu, hi[1], 31);
    const float endl = __shfl_sync(0xffffffffu, lo[1], 31);
    // in the blocks below the diagonal exp(cs_i - cs_j) is taken by way of the last token of j's
    // block of 16
    const float m = __shfl_sync(0xffffffffu, hi[1], lane | 7);
    const float ml = __shfl_sync(0xffffffffu, lo[1], lane | 7);
    float ek[2], sw[2], eq[2], kb[2], w[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const bool on = i + y < len;
        const float rk = norms[i + y], ex = ex2(hi[y] + lo[y]);
        kb[y] = on ? rk * s.beta[y] : 0.f;
        ek[y] = on ? -ex * rk : 0.f;
        sw[y] = ex2((end - hi[y]) + (endl - lo[y])) * kb[y];
        eq[y] = on ? ex * norms[kC + i + y] : 0.f;
        w[y] = ex2((m - hi[y]) + (ml - lo[y])) * kb[y];
    }
    auto put = [&](float *to, float x, float y) {
        *reinterpret_cast<float2 *>(to + i) = make_float2(x, y);
    };
    put(gates + kCs, -hi[0], -hi[1]);
    put(gates + kCl, -lo[0], -lo[1]);
    put(gates + kKb, kb[0], kb[1]);
    put(gates + kW, w[0], w[1]);
    put(vec, ek[0], ek[1]);
    put(vec + kC, sw[0], sw[1]);
    put(vec + 2 * kC, eq[0], eq[1]);
    if (lane < 4) vec[3 * kC + lane] = ex2(end + endl);
}

// 16 rows (block b) of a head's A or Att from their products with the keys: accumulators g, rows
// lane / 4 and 8 behind, columns 8 n + 2 (lane % 4) + {0, 1}.  Below the diagonal block A goes as
// two bf16 parts to where Inv's will be; the diagonal block in float32, 8 columns of a row in the
// place of each part.
template <bool kAtt>
__device__ __forceinline__ void build_rows(const float (&g)[8][4], int b, const float *norms,
                                           uint32_t gates, uint32_t tri)
{
    const int lane = threadIdx.x % 32, j0 = 2 * (lane % 4);
    const bool odd = lane & 4;   // this lane's rows
    int r[2];
    uint32_t to[2];   // Att's: of the first of two values, the second's is to ^ 4
    float ri[2], c[2], l[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        r[y] = b * 16 + lane / 4 + y * 8;
        // rows r and r ^ 1 have their 16-byte pieces in the same banks: they store in opposite orders
        to[y] = tri + kItemAtt + r[y] * 128 + (((j0 / 4 ^ r[y]) & 7) << 4) + (j0 % 4 + r[y] % 2) * 4;
        ri[y] = kAtt ? norms[kC + r[y]] * kCutBoth : norms[r[y]];
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(c[y]) : "r"(gates + (kCs + r[y]) * 4));
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(l[y]) : "r"(gates + (kCl + r[y]) * 4));
    }
#pragma unroll
    for (int bb = 0; bb < 4; ++bb) {
        if (bb > b) break;
        if (bb < b) {
            float mc, ml;
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(mc) : "r"(gates + (kCs + bb * 16 + 15) * 4));
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(ml) : "r"(gates + (kCl + bb * 16 + 15) * 4));
            uint64_t u[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float f = ri[y] * ex2((mc - c[y]) + (ml - l[y]));
                u[y] = pair(f, f);
            }
#pragma unroll
            for (int n = 2 * bb; n < 2 * bb + 2; ++n) {
                const uint64_t w = lds_pair(gates + (kW + n * 8 + j0) * 4);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint64_t v = mul2(mul2(pair(g[n][2 * y], g[n][2 * y + 1]), w), u[y]);
                    if constexpr (kAtt) {
                        float x, z;
                        unpair(v, x, z);
                        sts32(att_at(to[y], n), __float_as_uint(odd ? z : x));
                        sts32(att_at(to[y], n) ^ 4, __float_as_uint(odd ? x : z));
                    } else {
                        const uint32_t at = tri + tri_at(r[y], n) + j0 * 2;
                        uint32_t hi, lo;
                        split2(v, hi, lo);
                        sts32(at, hi);
                        sts32(at + kMat, lo);
                    }
                }
            }
        } else {
#pragma unroll
            for (int n = 2 * bb; n < 2 * bb + 2; ++n) {
                const int j = n * 8 + j0;
                const uint64_t cj = lds_pair(gates + (kCs + j) * 4);
                const uint64_t lj = lds_pair(gates + (kCl + j) * 4);
                const uint64_t kb = lds_pair(gates + (kKb + j) * 4);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float d0, d1;
                    unpair(add2(add2(pair(-c[y], -c[y]), cj), add2(pair(-l[y], -l[y]), lj)), d0, d1);
                    const uint64_t d = mul2(mul2(pair(ex2(d0), ex2(d1)), kb), pair(ri[y], ri[y]));
                    float x, z;
                    unpair(mul2(pair(g[n][2 * y], g[n][2 * y + 1]), d), x, z);
                    const int end = r[y] + (kAtt ? 1 : 0);   // columns before it
                    x = j < end ? x : 0.f;
                    z = j + 1 < end ? z : 0.f;
                    if constexpr (kAtt) {
                        sts32(att_at(to[y], n), __float_as_uint(odd ? z : x));
                        sts32(att_at(to[y], n) ^ 4, __float_as_uint(odd ? x : z));
                    } else {
                        sts64(tri + n % 2 * kMat + tri_at(r[y], 2 * bb + j0 / 4) + j0 % 4 * 4, x, z);
                    }
                }
            }
        }
    }
}

// Inv from A, in place: a pair of warps per head (blk: which), barrier `id` their own.  16 x 16 diagonal
// blocks by substitution, a lane per column; the blocks below, of 16 and then of 32, as
// -T22 A21 T11 in warp-level matrix products.
__device__ __forceinline__ void solve_head(uint32_t tri, int blk, int id)
{
    const int lane = threadIdx.x % 32, own = blk * 2 + lane / 16;
    // -T A U for 16 rows of T at `rows` (kT / 16 blocks of them side by side, the last one
    // lower triangular), A and U of kU columns
    auto merge = [&](auto blocks, int m0, int skip, int r1, int c0, float (&Z)[4][4]) {
        constexpr int kB = decltype(blocks)::value;   // blocks of 16
        float Y[4][4] = {};
#pragma unroll
        for (int s = 0; s < kB; ++s) {
            if (s > skip) break;
            uint32_t ah[4], al[4], bh[4], bl[4];
            const uint32_t at = tri + tri_at(m0 + lane % 16, r1 / 8 + s * 2 + lane / 16);
            ldsm4(ah, at);
            ldsm4(al, at + kMat);
#pragma unroll
            for (int n = 0; n < kB; ++n) {
                const uint32_t bt = tri + tri_at(r1 + s * 16 + lane % 8 + (lane / 8 & 1) * 8,
                                                c0 / 8 + n * 2 + lane / 16);
                ldsm4_trans(bh, bt);
                ldsm4_trans(bl, bt + kMat);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_16816(Y[2 * n + m], ah, bh[2 * m], bh[2 * m + 1]);
                    mma_16816(Y[2 * n + m], al, bh[2 * m], bh[2 * m + 1]);
                    mma_16816(Y[2 * n + m], ah, bl[2 * m], bl[2 * m + 1]);
                }
            }
        }
#pragma unroll
        for (int s = 0; s < kB; ++s) {
            uint32_t ah[4], al[4], bh[4], bl[4];
            split_a(Y[2 * s], Y[2 * s + 1], ah, al);
#pragma unroll
            for (int n = 0; n <= s; ++n) {
                const uint32_t bt = tri + tri_at(c0 + s * 16 + lane % 8 + (lane / 8 & 1) * 8,
                                                c0 / 8 + n * 2 + lane / 16);
                ldsm4_trans(bh, bt);
                ldsm4_trans(bl, bt + kMat);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_16816(Z[2 * n + m], ah, bh[2 * m], bh[2 * m + 1]);
                    mma_16816(Z[2 * n + m], al, bh[2 * m], bh[2 * m + 1]);
                    mma_16816(Z[2 * n + m], ah, bl[2 * m], bl[2 * m + 1]);
                }
            }
        }
    };
    auto store_merged = [&](auto blocks, int m0, int c0, const float (&Z)[4][4]) {
#pragma unroll
        for (int n = 0; n < 2 * decltype(blocks)::value; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t hi, lo;
                split2(-Z[n][2 * k], -Z[n][2 * k + 1], hi, lo);
                const uint32_t at =
                    tri + tri_at(m0 + lane / 4 + k * 8, c0 / 8 + n) + lane % 4 * 4;
                sts32(at, hi);
                sts32(at + kMat, lo);
            }
    };
    {
        // a column of a 16 x 16 block's inverse: x_i = [i = column] - sum_{k < i} A_ik x_k
        const int r0 = own * 16, col = lane % 16;
        float v[16];
#pragma unroll
        for (int m = 0; m < 16; ++m) {
            float s0 = m == col ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int k = 0; k < m; k += 4) {
                const float4 A =
                    lds128(tri + k / 8 * kMat + tri_at(r0 + m, own * 2 + k / 4 % 2));
                s0 = fmaf(-A.x, v[k], s0);
                if (k + 1 < m) s1 = fmaf(-A.y, v[k + 1], s1);
                if (k + 2 < m) s0 = fmaf(-A.z, v[k + 2], s0);
                if (k + 3 < m) s1 = fmaf(-A.w, v[k + 3], s1);
            }
            v[m] = s0 + s1;
        }
        __syncwarp();
        // rows m and m + 1, two columns to a lane: even lanes store row m, odd ones row m + 1
        const int odd = lane & 1;
#pragma unroll
        for (int m = 0; m < 16; m += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? v[m] : v[m + 1], 1);
            uint32_t hi, lo;
            split2(odd ? other : v[m], odd ? v[m + 1] : other, hi, lo);
            const uint32_t at =
                tri + tri_at(r0 + m + odd, own * 2 + col / 8) + (lane % 8 & ~1) * 2;
            sts32(at, hi);
            sts32(at + kMat, lo);
        }
        __syncwarp();
        float Z[4][4] = {};   // the block of 16 below the diagonal, inside this block of 32
        merge(Int<1>{}, blk * 32 + 16, 0, blk * 32 + 16, blk * 32, Z);
        __syncwarp();
        store_merged(Int<1>{}, blk * 32 + 16, blk * 32, Z);
    }
    named_bar_sync(id, 64);
    float Z[4][4] = {};   // the block of 32 below
    merge(Int<2>{}, 32 + blk * 16, blk, 32, 0, Z);
    named_bar_sync(id, 64);   // the block has been read
    store_merged(Int<2>{}, 32 + blk * 16, 0, Z);
}

// grid: chunks * batch * G * runs of `run_heads` heads; two groups of 4 warps.  A warp has 16 rows of
// the products with the keys in registers for all heads of the run: of K K^T in the first group,
// which builds A and turns it into Inv, of Q K^T in the second, which builds Att and makes the
// factors of the next four heads meanwhile.
template <int N>
__global__ void __launch_bounds__(kPrepThreads, 3)
delta_tc_prep_kernel(const DeltaArgs a, char *items, int64_t nchunks, int run_heads, const int2 *tab)
{
    extern __shared__ __align__(128) char smem[];
    let_next_start();
    const int hpg = a.H / a.G, runs = (hpg + run_heads - 1) / run_heads;
    int64_t id = blockIdx.x;
    if (id == 0 && threadIdx.x == 0 && a.clear) *a.clear = 0;
    const int run = (int)(id % runs);
    id /= runs;
    const int grp = (int)(id % a.G);
    id /= a.G;
    const int64_t c = id % nchunks, b = id / nchunks;
    int64_t t0;
    int len;
    chunk_span(tab, c, kC, a.L, t0, len);
    if (len <= 0) return;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32 % kPrepWarps;
    const bool att = tid >= kPrepWarps * 32;
    const int64_t row0 = b * a.L + t0;
    const uint32_t base = smem_u32(smem);
    float *norms = reinterpret_cast<float *>(smem + kPrepNorms);   // of keys; of queries, times scale

    {   // K and Q, 64 columns (a tile each) at a time
        constexpr int kPer = N / 8, kRows = kPrepThreads / kPer;
        const int r = tid / kPer, col = tid % kPer;
        const int64_t first = ((row0 + r) * a.G + grp) * N + col * 8;
        const bf16 *kg = static_cast<const bf16 *>(a.k), *qg = static_cast<const bf16 *>(a.q);
#pragma unroll
        for (int i = 0; i < kC; i += kRows) {
            const bool on = r + i < len;
            const int64_t off = on ? first + (int64_t)i * a.G * N : 0;
            const uint32_t at = base + col / 8 * 2 * kTile + sw_at(r + i, col % 8);
            cp16(at, kg + off, on);
            cp16(at + kTile, qg + off, on);
        }
        cp_commit();
    }
    const int h_begin = run * run_heads, h_end = min(hpg, h_begin + run_heads);
    Gates first = {};   // while the copies are on their way
    if (att && h_begin + warp < h_end) first = sum_gates(a, row0, len, grp * hpg + h_begin + warp);
    cp_wait<0>();
    __syncthreads();
    {   // half a row per thread: keys, then queries
        const int row = tid / 2;
        float ss = 0.f;
        if (a.l2norm) {
            uint64_t sum[2] = {};
#pragma unroll
            for (int j = 0; j < N / 16; ++j) {
                const int col = tid % 2 * (N / 16) + j;
                const float4 w =
                    lds128(base + (col / 8 * 2 + row / kC) * kTile + sw_at(row % kC, col % 8));
                const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t u = __float_as_uint(f[k]);
                    const uint64_t y = pair(bf16_lo(u), bf16_hi(u));
                    sum[k % 2] = fma2(y, y, sum[k % 2]);
                }
            }
            float y, z;
            unpair(add2(sum[0], sum[1]), y, z);
            ss = y + z;
        }
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        const float r = a.l2norm ? rsqrtf(ss + kL2Eps) : 1.f;
        if (tid % 2 == 0) norms[row] = row < kC ? r : r * a.scale;
    }
    // the later blocks have more columns: spread over the SM's quarters
    const int blk = att ? kPrepWarps - 1 - warp : warp;
    float g[8][4] = {};
#pragma unroll
    for (int s = 0; s < N / 16; ++s) {
        const uint32_t tile = base + s / 4 * 2 * kTile;
        uint32_t fa[4], fb[4];
        ldsm4(fa, tile + att * kTile + sw_at(blk * 16 + lane % 16, s % 4 * 2 + lane / 16));
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n > blk) break;
            ldsm4(fb, tile + sw_at(n * 16 + lane % 8 + lane / 16 * 8, s % 4 * 2 + (lane / 8 & 1)));
            mma_16816(g[2 * n], fa, fb[0], fb[1]);
            mma_16816(g[2 * n + 1], fa, fb[2], fb[3]);
        }
    }
    __syncthreads();   // K's and Q's place is the triangles' now

    const int64_t item0 = (b * nchunks + c) * a.H + grp * hpg;
    auto gates_of = [&](int hq) { return kPrepGates + ((hq - h_begin) & kPrepQuad) * kGateFloats * 4; };
    auto make_gates = [&](int hq, const Gates &sums) {   // of heads hq .. hq + 3: a warp each
        const int hl = hq + warp;
        if (hl < h_end)
            make_factors(sums, len, norms,
                         reinterpret_cast<float *>(smem + gates_of(hq)) + warp * kGateFloats,
                         reinterpret_cast<float *>(items + (item0 + hl) * kItem + kItemVec));
    };
    if (att) make_gates(h_begin, first);
    for (int hp = h_begin; hp < h_end; hp += 2) {
        const int hq = h_begin + ((hp - h_begin) & ~(kPrepQuad - 1));
        const int here = min(2, h_end - hp);   // heads of this pair
        if (tid == 0) bulk_store_wait();
        __syncthreads();
        const uint32_t gates = base + gates_of(hq) + (hp - hq) * kGateFloats * 4;
        for (int x = 0; x < here; ++x) {
            if (att) build_rows<true>(g, blk, norms, gates + x * kGateFloats * 4, base + x * kMats);
            else build_rows<false>(g, blk, norms, gates + x * kGateFloats * 4, base + x * kMats);
        }
        if (att) {
            if (hp > hq || hp + 2 >= h_end) {
                const int next = hq + kPrepQuad;
                if (next + warp < h_end)
                    make_gates(next, sum_gates(a, row0, len, grp * hpg + next + warp));
            }
        } else {
            named_bar_sync(3, kPrepWarps * 32);
            if (warp / 2 < here) solve_head(base + warp / 2 * kMats, warp % 2, 1 + warp / 2);
        }
        fence_async_smem();
        __syncthreads();
        if (tid == 0)
            for (int x = 0; x < here; ++x)
                bulk_store(items + (item0 + hp + x) * kItem, base + x * kMats, kMats);
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------- the chain
constexpr int kRowWarps = 8, kMma = kRowWarps, kLoadKq = kMma + 1, kLoadV = kMma + 2;   // and items
constexpr int kTcThreads = (kMma + 4) * 32;
constexpr int kKqStages = 2;

// TMEM columns.  S's operand parts share the columns of its update; W of the first head those of
// X.  The Att product of the second head takes the place of the operands of the state's update, once
// that is done.
constexpr uint32_t kColS = 0, kColX = 128, kColW1 = 192, kColAw = 256, kColQ = 320, kColVt = 384,
                   kColOp = 448;

template <int N, int HP> struct TcSmem {
    static constexpr int kHalf = 2 * kTile;               // 64 columns of K, then of Q
    static constexpr int kStage = N / 64 * kHalf;
    static constexpr int kv = kKqStages * kStage, kTris = kv + 2 * 2 * kTile,
                         kIdent = kTris + 2 * HP * kItem, kBars = kIdent + 16 * 128;
    static constexpr int kTotal = kBars + 256;
};

struct TcBars {   // 256 bytes at most
    uint64_t kq_full[kKqStages], kq_empty[kKqStages], v_full[2], v_empty[2], tri_full[2],
        tri_empty[2], s_ready, x_done, r_ready, w_done, w_ready, ds_done, aw_done, o_read, drain;
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ void arrive_warp(uint64_t *bar)
{
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}
// ---------------------------------------------------------------- the rows' warps
template <int N, int P, int HP>
__device__ __forceinline__ void row_warps(const DeltaArgs &a, TcBars &bar, uint32_t base,
                                          uint32_t tmem, int64_t seq, int64_t row0, int64_t len_all,
                                          int nchunks, int h0, int heads)
{
    using L = TcSmem<N, HP>;
    constexpr int NS = N / 2;   // state columns of this thread
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, quad = warp % 4, half = warp / 4;
    const int r = quad * 32 + lane;
    const bool here = r / P < heads;          // rows of a head that is there
    const int x = here ? r / P : 0, h = h0 + x, p = r % P;
    const uint32_t t0 = tmem + ((uint32_t)quad << 21);
    const uint32_t col_w = t0 + (x ? kColW1 : kColX) + half * 32;
    const uint32_t col_aw = t0 + (x ? kColOp : kColAw) + half * 32;
    volatile int *abort = &bar.abort;

    uint64_t S[NS / 2];   // pairs of columns
    const int64_t srow = ((seq * a.H + h) * P + p) * N + half * NS;
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.init && here) v = *reinterpret_cast<const float4 *>(a.init + srow + i);
        S[i / 2] = pair(v.x, v.y);
        S[i / 2 + 1] = pair(v.z, v.w);
    }
    const uint32_t vecs = base + L::kTris + x * kItem + kItemVec;
    auto vec_of = [&](int c) { return vecs + (c & 1) * HP * kItem; };
    // S <- E S + the update that chunk c's products left
    auto take_update = [&](int c) {
        if (!wait_all(&bar.ds_done, c & 1, abort)) return false;
        tc_fence_after();
        uint64_t E[2];
        lds_pairs(vec_of(c) + 3 * kC * 4, E);   // E, four times
#pragma unroll
        for (int i = 0; i < NS; i += 32) {
            uint32_t d[32];
            tmem_ld32(t0 + kColS + half * NS + i, d);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 2)
                S[(i + j) / 2] = fma2(E[0], S[(i + j) / 2], pair_u(d[j], d[j + 1]));
        }
        return true;
    };
    // the output of chunk c, read and rounded: tokens 2 j, 2 j + 1 of this half in out[j]
    uint32_t out[16];
    auto read_out = [&](int c) {
        if (!wait_all(&bar.aw_done, c & 1, abort)) return false;
        tc_fence_after();
        const uint32_t eq = vec_of(c) + (2 * kC + half * 32) * 4;
        uint32_t q[32], w[32];
        tmem_ld32(t0 + kColQ + half * 32, q);
        tmem_ld32(col_aw, w);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            uint64_t e[2];
            lds_pairs(eq + j * 4, e);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float y, z;
                unpair(fma2(e[k], pair_u(q[j + 2 * k], q[j + 2 * k + 1]),
                            pair_u(w[j + 2 * k], w[j + 2 * k + 1])), y, z);
                out[j / 2 + k] = pack_bf16x2(y, z);
            }
        }
        tc_fence_before();
        arrive_warp(&bar.o_read);
        if (lane == 0) mbar_arrive(&bar.tri_empty[c & 1]);
        return true;
    };
    // neighbouring lanes have neighbouring p, and exchange halves of a pair of tokens, so that an
    // even lane stores the first token's two values, an odd one the second's
    auto store_out = [&](int c) {
        const int64_t left = len_all - (int64_t)c * kC - half * 32;
        const int odd = lane & 1, len = here ? (int)(left < 32 ? left : 32) - odd : 0;
        bf16 *to = static_cast<bf16 *>(a.o) +
                   ((row0 + (int64_t)c * kC + half * 32 + odd) * a.H + h) * P + (p & ~1);
        const int64_t step = 2 * (int64_t)a.H * P;
        const uint32_t pick = odd ? 0x3276 : 0x5410;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, out[j], 1);
            if (2 * j < len)
                *reinterpret_cast<uint32_t *>(to) = __byte_perm(out[j], other, pick);
            to += step;
        }
    };

    for (int c = 0; c < nchunks; ++c) {
        if (c > 0 && !take_update(c - 1)) return;
#pragma unroll
        for (int i = 0; i < NS; i += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) split2(S[i / 2 + j], hi[j], lo[j]);
            tmem_st8(t0 + kColS + half * NS + i / 2, hi);
            tmem_st8(t0 + kColS + half * NS + NS / 2 + i / 2, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(&bar.s_ready);
        if (c > 0 && !read_out(c - 1)) return;

        if (!wait_all(&bar.tri_full[c & 1], (c >> 1) & 1, abort)) return;
        if (!wait_all(&bar.x_done, c & 1, abort)) return;
        tc_fence_after();
        const uint32_t vec = vec_of(c) + half * 32 * 4;
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
            uint32_t xs[16], vs[16], hi[8], lo[8];
            tmem_ld16(t0 + kColX + half * 32 + i, xs);
            tmem_ld16(t0 + kColVt + half * 32 + i, vs);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                uint64_t e[2];   // -ek
                lds_pairs(vec + (i + j) * 4, e);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    split2(fma2(e[k], pair_u(xs[j + 2 * k], xs[j + 2 * k + 1]),
                                pair_u(vs[j + 2 * k], vs[j + 2 * k + 1])),
                           hi[j / 2 + k], lo[j / 2 + k]);
            }
            tmem_st8(t0 + kColOp + half * 16 + i / 2, hi);
            tmem_st8(t0 + kColOp + 32 + half * 16 + i / 2, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(&bar.r_ready);

        if (!wait_all(&bar.w_done, c & 1, abort)) return;
        tc_fence_after();
        uint32_t ws[32];
        tmem_ld32(col_w, ws);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 16) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                uint64_t s[2];
                lds_pairs(vec + (kC + i + j) * 4, s);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    split2(mul2(s[k], pair_u(ws[i + j + 2 * k], ws[i + j + 2 * k + 1])),
                           hi[j / 2 + k], lo[j / 2 + k]);
            }
            tmem_st8(t0 + kColOp + half * 16 + i / 2, hi);
            tmem_st8(t0 + kColOp + 32 + half * 16 + i / 2, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        arrive_warp(&bar.w_ready);
        if (c > 0) store_out(c - 1);   // while the state's update is on its way
    }
    if (!take_update(nchunks - 1)) return;
    if (a.final_state && here) {
#pragma unroll
        for (int i = 0; i < NS; i += 4) {
            float4 v;
            unpair(S[i / 2], v.x, v.y);
            unpair(S[i / 2 + 1], v.z, v.w);
            *reinterpret_cast<float4 *>(a.final_state + srow + i) = v;
        }
    }
    if (read_out(nchunks - 1)) store_out(nchunks - 1);
}

// ---------------------------------------------------------------- the matrix products' warp
template <int N, int HP>
__device__ __forceinline__ void issue_products(TcBars &bar, uint32_t base, uint32_t tmem, int nchunks,
                                               int heads)
{
    using L = TcSmem<N, HP>;
    constexpr int NS = N / 2;
    volatile int *abort = &bar.abort;
    // what loops and addresses depend on, where the compiler knows it is the same in all lanes
    const uint32_t on = elect_one();
    tmem = __reduce_max_sync(0xffffffffu, tmem);
    nchunks = __reduce_max_sync(0xffffffffu, nchunks);
    heads = __reduce_max_sync(0xffffffffu, heads);
    constexpr uint32_t id64 = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t id_v = idesc_bf16_f32(128, 16, true, false);
    constexpr uint32_t id_s = idesc_bf16_f32(128, N, false, true);
    // descriptors; their lowest 14 bits are an address / 16, so that offsets are added to them
    const uint64_t vd = smem_desc_sw128(base + L::kv, kTile, 1024);
    const uint64_t identd = smem_desc_sw128(base + L::kIdent, 0, 1024);
    const uint64_t kq0 = smem_desc_sw128(base, 0, 1024);
    const uint64_t kc0 = smem_desc_sw128(base, L::kHalf, 1024);
    const uint64_t tri0 = smem_desc_sw64(base + L::kTris, 512);
    const uint64_t att0 = smem_desc_sw128(base + L::kTris + kItemAtt, 0, 1024);

    auto products_v = [&](int c) {   // V^T, 16 tokens at a time, through the identity
        if (!wait_all(&bar.v_full[c & 1], (c >> 1) & 1, abort)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
            warp_mma_bf16(on, tmem + kColVt + k * 16, vd + (((c & 1) * 2 * kTile + k * 2048) >> 4), identd,
                     id_v, 0);
        warp_mma_commit(on, &bar.v_empty[c & 1]);
        return true;
    };
    if (!products_v(0)) return;
    for (int c = 0; c < nchunks; ++c) {
        const int stage = c % kKqStages, buf = c & 1;
        const uint64_t kd = kq0 + stage * (L::kStage >> 4);
        if (!wait_all(&bar.kq_full[stage], (c / kKqStages) & 1, abort)) return;
        // W of the chunk before, in X's columns, has been read
        if (c > 0 && !wait_all(&bar.aw_done, (c - 1) & 1, abort)) return;
        if (!wait_all(&bar.s_ready, c & 1, abort)) return;
        tc_fence_after();
        // the parts of S times 16 rows of K (or Q, `rows` bytes behind)
        auto with_s = [&](auto part, uint32_t d, uint32_t rows, bool first) {
#pragma unroll
            for (int k = 0; k < N / 16; ++k)
                warp_mma_bf16_ts(on, tmem + d, tmem + kColS + k * 16 / NS * NS +
                                          decltype(part)::value * (NS / 2) + k * 16 % NS / 2,
                            kd + ((k / 4 * L::kHalf + rows + k % 4 * 32) >> 4), id64, !first || k > 0);
        };
        with_s(Int<0>{}, kColX, 0, true);
        with_s(Int<1>{}, kColX, 0, false);
        warp_mma_commit(on, &bar.x_done);
        if (c > 0 && !wait_all(&bar.o_read, (c - 1) & 1, abort)) return;
        tc_fence_after();
        with_s(Int<0>{}, kColQ, kC * 128, true);
        with_s(Int<1>{}, kColQ, kC * 128, false);

        if (!wait_all(&bar.tri_full[buf], (c >> 1) & 1, abort)) return;
        if (!wait_all(&bar.r_ready, c & 1, abort)) return;
        tc_fence_after();
        // a triangle: tokens 16 k on take the written values of tokens 16 k .. 16 k + 15
        auto with_tri = [&](uint32_t d, uint32_t op, int step, uint64_t mat, bool first) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                warp_mma_bf16_ts(on, tmem + d + k * 16, tmem + op + k / 2 * step + k % 2 * 8,
                                 mat + ((k / 2 * kMatRight + k % 2 * (16 * 64 + 32)) >> 4),
                                 idesc_bf16_f32(128, 64 - 16 * k, false, false), !first || k > 0);
        };
        const uint64_t tris = tri0 + buf * (HP * kItem >> 4);
#pragma unroll 1
        for (int x = 0; x < HP; ++x) {
            if (x >= heads) break;
            const uint32_t d = x ? kColW1 : kColX;
            const uint64_t tri = tris + x * (kItem >> 4);
            with_tri(d, kColOp, 16, tri, true);
            with_tri(d, kColOp + 32, 16, tri, false);
            with_tri(d, kColOp, 16, tri + (kMat >> 4), false);
        }
        warp_mma_commit(on, &bar.w_done);

        if (!wait_all(&bar.w_ready, c & 1, abort)) return;
        tc_fence_after();
        const uint64_t kc = kc0 + stage * (L::kStage >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            warp_mma_bf16_ts(on, tmem + kColS, tmem + kColOp + k * 8, kc + k % 4 * (2048 >> 4), id_s, k > 0);
        warp_mma_commit(on, &bar.ds_done);
        warp_mma_commit(on, &bar.kq_empty[stage]);
        // Att times W, 8 tokens at a time
#pragma unroll 1   // (a chunk's instructions do not fit the cache otherwise: packed 471 us for 446)
        for (int x = 0; x < HP; ++x) {
            if (x >= heads) break;
            if (x) {   // its columns are free
                if (!wait_all(&bar.ds_done, c & 1, abort)) return;
                tc_fence_after();
            }
            const uint64_t att = att0 + ((buf * HP + x) * kItem >> 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                warp_mma_tf32_ts(on, tmem + (x ? kColOp : kColAw) + k / 2 * 16,
                                 tmem + (x ? kColW1 : kColX) + k * 8,
                                 att + ((k / 4 * (kAttRight - 32 * 128) + k / 2 * 16 * 128 + k % 4 * 32) >> 4),
                                 idesc_tf32_f32(128, 64 - k / 2 * 16), k > 0);
        }
        warp_mma_commit(on, &bar.tri_empty[buf]);
        warp_mma_commit(on, &bar.aw_done);   // last: the CTA's last wait is for it
        if (c + 1 < nchunks && !products_v(c + 1)) return;
    }
}

// ---------------------------------------------------------------- copies
// K and Q, zeros past the sequence's end.
template <int N, int HP>
__device__ __forceinline__ void load_kq(const DeltaArgs &a, TcBars &bar, uint32_t base, int64_t t0,
                                        int64_t len_all, int nchunks, int grp)
{
    using L = TcSmem<N, HP>;
    constexpr int kPer = N / 8, kRows = 32 / kPer;   // 16-byte pieces of a row, rows at a time
    const int lane = threadIdx.x % 32, r = lane / kPer, col = lane % kPer;
    const int64_t step = (int64_t)kRows * a.G * N;
    const int64_t first = ((t0 + r) * a.G + grp) * N + col * 8;
    const bf16 *kg = static_cast<const bf16 *>(a.k) + first;
    const bf16 *qg = static_cast<const bf16 *>(a.q) + first;
    for (int c = 0; c < nchunks; ++c) {
        const int stage = c % kKqStages;
        if (c >= kKqStages &&
            !wait_all(&bar.kq_empty[stage], (c / kKqStages - 1) & 1, &bar.abort)) return;
        const uint32_t to = base + stage * L::kStage + col / 8 * L::kHalf;
        const int64_t left = len_all - (int64_t)c * kC - r;   // rows of this lane's first one on
#pragma unroll 8
        for (int i = 0; i < kC; i += kRows) {
            const bool on = i < left;
            const uint32_t at = to + sw_at(r + i, col % 8);
            cp16(at, on ? kg : static_cast<const bf16 *>(a.k), on);
            cp16(at + kC * 128, on ? qg : static_cast<const bf16 *>(a.q), on);
            kg += step;
            qg += step;
        }
        cp_commit();
        cp_wait<0>();
        fence_async_smem();
        mbar_arrive(&bar.kq_full[stage]);
    }
}

template <int N, int P, int HP>
__device__ __forceinline__ void load_v(const DeltaArgs &a, TcBars &bar, uint32_t base, int64_t t0,
                                       int64_t len_all, int nchunks, int h0, int heads)
{
    using L = TcSmem<N, HP>;
    const int lane = threadIdx.x % 32, r = lane / 16, col = lane % 16;
    const int64_t step = (int64_t)2 * a.H * P;
    const bf16 *vg = static_cast<const bf16 *>(a.v) + ((t0 + r) * a.H + h0) * P + col * 8;
    const uint32_t to0 = base + L::kv + col / 8 * kTile;
    for (int c = 0; c < nchunks; ++c) {
        if (c >= 2 && !wait_all(&bar.v_empty[c & 1], ((c >> 1) - 1) & 1, &bar.abort)) return;
        const uint32_t to = to0 + (c & 1) * 2 * kTile;
        const int64_t left = col < heads * P / 8 ? len_all - (int64_t)c * kC - r : 0;
#pragma unroll 8
        for (int i = 0; i < kC; i += 2) {
            const bool on = i < left;
            cp16(to + sw_at(r + i, col % 8), on ? vg : static_cast<const bf16 *>(a.v), on);
            vg += step;
        }
        cp_commit();
        cp_wait<0>();
        fence_async_smem();
        mbar_arrive(&bar.v_full[c & 1]);
    }
}

// The items of the CTA's heads, chunk `first` on: one thread.
template <int N, int HP>
__device__ __forceinline__ void load_items(const DeltaArgs &a, TcBars &bar, char *smem,
                                           const char *items, int64_t first, int nchunks, int h0,
                                           int heads)
{
    using L = TcSmem<N, HP>;
    wait_before();   // only this thread reads what the first kernel wrote
    for (int c = 0; c < nchunks; ++c) {
        const int buf = c & 1;
        if (c >= 2 && !mbar_wait(&bar.tri_empty[buf], ((c >> 1) - 1) & 1, &bar.abort)) return;
        mbar_arrive_expect_tx(&bar.tri_full[buf], heads * kItemUsed);
        const char *from = items + ((first + c) * a.H + h0) * kItem;
        for (int x = 0; x < heads; ++x)
            bulk_load(smem + L::kTris + (buf * HP + x) * kItem, from + x * (int64_t)kItem, kItemUsed,
                      &bar.tri_full[buf]);
    }
}

// grid: sequences * G * ceil(heads of a group / HP)
template <int N, int P>
__global__ void __launch_bounds__(kTcThreads, 1)
delta_tc_kernel(const DeltaArgs a, const char *items, int64_t nchunks_all, const int32_t *cstart,
                int *status)
{
    constexpr int HP = 128 / P;
    using L = TcSmem<N, HP>;
    extern __shared__ char raw[];
    if (cstart && *status) {   // inconsistent offsets
        wait_before();
        return;
    }
    char *smem = reinterpret_cast<char *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    TcBars &bar = *reinterpret_cast<TcBars *>(smem + L::kBars);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int hpg = a.H / a.G, runs = (hpg + HP - 1) / HP;
    const int run = blockIdx.x % runs, grp = blockIdx.x / runs % a.G;
    int64_t seq = blockIdx.x / runs / a.G;
    int64_t t0 = seq * a.L, len_all = a.L, first = seq * nchunks_all;
    if (cstart) {
        // the longest sequences start first: this CTA takes the one of its rank
        if (a.nseq <= kTcThreads) {
            int *pick = &bar.abort;
            if (tid < a.nseq) {
                const int mine = a.cu[tid + 1] - a.cu[tid];
                int before = 0;
                for (int s = 0; s < a.nseq; ++s) {
                    const int other = a.cu[s + 1] - a.cu[s];
                    before += other > mine || (other == mine && s < tid);
                }
                if (before == seq) *pick = tid;
            }
            __syncthreads();
            seq = *pick;
            __syncthreads();
        }
        t0 = a.cu[seq];
        len_all = a.cu[seq + 1] - t0;
        first = cstart[seq];
    }
    const int nchunks = (int)((len_all + kC - 1) / kC);
    const int h0 = grp * hpg + run * HP, heads = hpg - run * HP < HP ? hpg - run * HP : HP;

    if (nchunks == 0) {   // an empty sequence: its state passes through
        if (a.final_state) {
            const int64_t at = (seq * a.H + h0) * P * N;
            for (int i = tid; i < heads * P * N; i += kTcThreads)
                a.final_state[at + i] = a.init ? a.init[at + i] : 0.f;
        }
        wait_before();
        return;
    }
    if (tid == 0) {
        bar.abort = 0;
        for (int i = 0; i < kKqStages; ++i) {
            mbar_init(&bar.kq_full[i], 32);
            mbar_init(&bar.kq_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.v_full[i], 32);
            mbar_init(&bar.v_empty[i], 1);
            mbar_init(&bar.tri_full[i], 1);
            mbar_init(&bar.tri_empty[i], 1 + kRowWarps);
        }
        mbar_init(&bar.s_ready, kRowWarps);
        mbar_init(&bar.x_done, 1);
        mbar_init(&bar.r_ready, kRowWarps);
        mbar_init(&bar.w_done, 1);
        mbar_init(&bar.w_ready, kRowWarps);
        mbar_init(&bar.ds_done, 1);
        mbar_init(&bar.aw_done, 1);
        mbar_init(&bar.o_read, kRowWarps);
        mbar_init(&bar.drain, 1);
        fence_mbar_init();
    }
    if (warp == kMma) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    if (tid < 256) {   // the 16 x 16 identity, in the first 32 bytes of 16 rows
        const int r = tid / 16, col = tid % 16;
        *reinterpret_cast<bf16 *>(smem + L::kIdent + sw_at(r, col / 8) + col % 8 * 2) =
            from_f32<bf16>(r == col ? 1.f : 0.f);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem, base = smem_u32(smem);

    if (warp < kRowWarps) {
        row_warps<N, P, HP>(a, bar, base, tmem, seq, t0, len_all, nchunks, h0, heads);
    } else if (warp == kMma) {
        issue_products<N, HP>(bar, base, tmem, nchunks, heads);
    } else if (warp == kLoadKq) {
        load_kq<N, HP>(a, bar, base, t0, len_all, nchunks, grp);
    } else if (warp == kLoadV) {
        load_v<N, P, HP>(a, bar, base, t0, len_all, nchunks, h0, heads);
    } else if (lane == 0) {
        load_items<N, HP>(a, bar, smem, items, first, nchunks, h0, heads);
    }
    __syncwarp();
    __syncthreads();
    if (warp == kMma) {
        if (bar.abort) {   // let the products and copies in flight end
            if (lane == 0) {
                mma_commit(&bar.drain);
                mbar_wait_drain(&bar.drain, 0);
                atomicOr(status, 4);
            }
            drain_sleep();
            __syncwarp();
        }
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

bool delta_tc_supported(int P, int N) { return (P == 64 || P == 128) && (N == 64 || N == 128); }

cudaError_t launch_delta_tc(const DeltaArgs &a, char *items, int64_t nchunks, const int2 *tab,
                            const int32_t *cstart, int *status, cudaStream_t st)
{
    const int64_t batch = a.cu ? 1 : a.batch, hpg = a.H / a.G;
    // heads per CTA of the first kernel: up to 16 share a chunk's products with its keys, fewer
    // where the launch would leave SMs empty
    int run = hpg < 16 ? (int)hpg : 16;
    auto ctas = [&] { return nchunks * batch * a.G * ((hpg + run - 1) / run); };
    while (run > kPrepQuad && ctas() < 2 * 444) run = (run + 1) / 2;
    if (ctas() > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto prep = [&](auto kern) {
        const cudaError_t e = allow_smem(reinterpret_cast<const void *>(kern), kPrepSmem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)ctas(), kPrepThreads, kPrepSmem, st>>>(a, items, nchunks, run, tab);
        return cudaGetLastError();
    };
    cudaError_t e = a.N == 128 ? prep(delta_tc_prep_kernel<128>) : prep(delta_tc_prep_kernel<64>);
    if (e != cudaSuccess) return e;
    const int hp = 128 / a.P;
    const unsigned grid = (unsigned)((a.cu ? a.nseq : a.batch) * a.G * ((hpg + hp - 1) / hp));
    auto go = [&](auto kern, int smem) {
        // to an address that is a multiple of 1024
        return launch_after(kern, grid, kTcThreads, smem + 1024, st, a, items, nchunks, cstart, status);
    };
    if (a.P == 64)
        return a.N == 128 ? go(delta_tc_kernel<128, 64>, TcSmem<128, 2>::kTotal)
                          : go(delta_tc_kernel<64, 64>, TcSmem<64, 2>::kTotal);
    return a.N == 128 ? go(delta_tc_kernel<128, 128>, TcSmem<128, 1>::kTotal)
                      : go(delta_tc_kernel<64, 128>, TcSmem<64, 1>::kTotal);
}

}  // namespace ssd
