// The gated delta rule in chunks of 32 tokens (bf16 inputs).
//
// With cs the chunk's running sum of g, e_i = exp(cs_i), E = e_last, k and q as normalised where
// that is asked for, and S the state that enters the chunk, the values that the tokens write are
//
//     W = Inv (V - e K S^T),   Inv = (I + A)^-1,   A_ij = exp(cs_i - cs_j) (k_i . k_j) beta_j, j < i
//     O = scale e Q S^T + Att W,                   Att_ij = scale exp(cs_i - cs_j) (q_i . k_j) beta_j, j <= i
//     S' = E S + sum_j (E / e_j) beta_j W_j k_j^T
//
// Two kernels.  delta_prep_kernel, parallel over chunks and heads, writes Inv - I, Att and the
// factors of the rows (norms, decays, beta) -- everything that does not need the state.
// delta_chain_kernel walks a sequence's chunks with the state in registers.  The rows p of a state
// are independent of one another, and of U, O and the products with them too: a warp owns 16 rows
// (the transposed products W^T = R^T Inv^T, S K^T, ... have p on the accumulators' rows), and the
// layout in which one product leaves its accumulators is the A operand of the next, so the whole
// chain of a chunk runs inside a warp with no exchange between warps at all.  They share the tiles
// of K, Q, V and the triangles, which two more warps bring one chunk ahead by cp.async (with the
// copies issued by the computing warps a chunk took 3.9 us for 2.3, at 2 x 2048 tokens x 24 heads).
//
// Accuracy: K, Q and V enter as they are; the state, the residual, W, Inv and Att, which are float32,
// enter as two bf16 parts each (2^-17 of one is left), so that final states are 3e-6 off (float32 sums
// alone leave 3e-7) and the output by little more than its own rounding.
// The backward's dg is a small difference of these products: what two parts leave of the values that
// are written, of dS in dS K^T and of W in Att W came to 1e-5 and more of dg for one call in eighty of a
// few tokens and heads (2.7e-5 at worst of 1800 such calls).  There these take three parts, and that is
// 7e-6 at worst; 44 and 32 matrix instructions more in the two chains, about 30 us of 445 at 2 x 2048 x 24
// heads.
//
// Bound: with many heads the rate of the warp-level matrix instructions (one m16n8k16 in 8 cycles per
// SM quarter), where the tcgen05 form takes over; with few, where a warp has its SM quarter to itself,
// the latency of its chain, 1.5 us a chunk: 129 tokens x 8 heads 18 us, 2048 tokens x 8 heads 104 us.
// The backward's chains at 2 x 2048 x 24 heads: 142 and 178 us.
#include "delta.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace {

using namespace sm100;

constexpr int C = kDeltaChunk;
constexpr int kPrepWarps = 4;
constexpr int kPrepHeads = 16;     // most heads of a group per CTA of the prep kernel
constexpr int kLoadWarps = 2;      // of a CTA of the chains, behind the warps that compute
constexpr int kMaxRows = 112;      // of a CTA of the chains: nine warps, of which a thread has 168 registers
constexpr float kMinDecay = -200.f;    // exp of it is 0 in float32
constexpr float kMinBeta = 1e-20f;

__device__ __forceinline__ float warp_sum4(float v)   // over 4 neighbouring lanes
{
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// grid: (chunks, batch, G * head runs).  kBwd: beta kept away from 0, where the backward divides by it
// (a token of beta 1e-20 writes nothing either).
template <int N, bool kBwd>
__global__ void __launch_bounds__(kPrepWarps * 32)
delta_prep_kernel(const DeltaArgs a, char *items, int64_t nchunks, const int2 *tab, int run_heads)
{
    constexpr int kPitch = N + 8;   // elements; 16 bytes more than a row: no bank conflicts
    __shared__ __align__(16) bf16 ks[C * kPitch], qs[C * kPitch];
    __shared__ float kk[C][C + 1], qk[C][C + 1];
    __shared__ __align__(16) float As[kPrepWarps][C][C + 4];
    __shared__ float rqs[C];

    if (blockIdx.x + blockIdx.y + blockIdx.z + threadIdx.x == 0 && a.clear) *a.clear = 0;
    const int64_t c = blockIdx.x, b = blockIdx.y;
    const int hpg = a.H / a.G, runs = (hpg + run_heads - 1) / run_heads;
    const int g = blockIdx.z / runs, run = blockIdx.z % runs;
    int64_t t0;
    int len;
    chunk_span(tab, c, C, a.L, t0, len);
    if (len <= 0) return;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int64_t row0 = b * a.L + t0;

    const bf16 *kg = static_cast<const bf16 *>(a.k) + (row0 * a.G + g) * N;
    const bf16 *qg = static_cast<const bf16 *>(a.q) + (row0 * a.G + g) * N;
    for (int i = tid; i < C * (N / 8); i += kPrepWarps * 32) {
        const int r = i / (N / 8), col = i % (N / 8) * 8;
        const int64_t off = r < len ? (int64_t)r * a.G * N + col : 0;
        cp16(smem_u32(ks + r * kPitch + col), kg + off, r < len);
        cp16(smem_u32(qs + r * kPitch + col), qg + off, r < len);
    }
    cp_commit();
    cp_wait<0>();
    __syncthreads();

    {   // K K^T (warps 0, 1) and Q K^T (warps 2, 3), 16 rows each
        const bf16 *rows = warp < 2 ? ks : qs;
        const int m0 = (warp & 1) * 16;
        float acc[4][4] = {};
#pragma unroll
        for (int s = 0; s < N / 16; ++s) {
            uint32_t fa[4], fb[4];
            ldsm4(fa, smem_u32(rows + (m0 + lane % 16) * kPitch + s * 16 + lane / 16 * 8));
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                ldsm4(fb, smem_u32(ks + (n * 16 + lane % 8 + lane / 16 * 8) * kPitch + s * 16 +
                                   (lane / 8 & 1) * 8));
                mma_16816(acc[2 * n], fa, fb[0], fb[1]);
                mma_16816(acc[2 * n + 1], fa, fb[2], fb[3]);
            }
        }
        float (*out)[C + 1] = warp < 2 ? kk : qk;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                out[m0 + lane / 4 + r / 2 * 8][n * 8 + lane % 4 * 2 + r % 2] = acc[n][r];
    }
    if (a.l2norm) {   // |q|^2 of 8 tokens per warp, 4 lanes to a token (|k|^2: kk's diagonal)
        const int r = warp * 8 + lane / 4;
        float s = 0.f;
        for (int i = lane % 4 * 2; i < N; i += 8) {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(qs + r * kPitch + i);
            s = fmaf(bf16_lo(v), bf16_lo(v), s);
            s = fmaf(bf16_hi(v), bf16_hi(v), s);
        }
        s = warp_sum4(s);
        if (lane % 4 == 0) rqs[r] = rsqrtf(s + kL2Eps);
    }
    __syncthreads();

    // a head per warp; lane j is token j: column j of the triangles
    const bool on = lane < len;
    const float rk = a.l2norm ? rsqrtf(kk[lane][lane] + kL2Eps) : 1.f;
    const float rq = (a.l2norm ? rqs[lane] : 1.f) * a.scale;
    float (*A)[C + 4] = As[warp];
    const int h_end = min(hpg, (run + 1) * run_heads);
    for (int hl = run * run_heads + warp; hl < h_end; hl += kPrepWarps) {
        const int h = g * hpg + hl;
        const int64_t at = (row0 + lane) * a.H + h;
        float gt = on && a.g ? a.g[at] : 0.f;
        float beta = on ? a.beta[at] : 0.f;
        if (gt < kMinDecay) gt = kMinDecay;
        if (kBwd && on && fabsf(beta) < kMinBeta) beta = kMinBeta;
        // running sum of g in two floats: differences behind a token that wipes the state out
        // (-200) stay accurate
        float cs = gt, cl = 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float up = __shfl_up_sync(0xffffffffu, cs, o);
            const float ul = __shfl_up_sync(0xffffffffu, cl, o);
            if (lane >= o) {
                float s, e;
                two_sum(cs, up, s, e);
                cs = s;
                cl += ul + e;
            }
        }
        const float cs_end = __shfl_sync(0xffffffffu, cs, 31);
        const float cl_end = __shfl_sync(0xffffffffu, cl, 31);
        const float e = __expf(cs + cl);
        char *item = items + ((b * nchunks + c) * a.H + h) * DeltaItem::kBytes;
        float *vec = reinterpret_cast<float *>(item + DeltaItem::kVec);
        vec[lane] = on ? e * rk : 0.f;
        vec[C + lane] = on ? __expf((cs_end - cs) + (cl_end - cl)) * rk * beta : 0.f;
        vec[2 * C + lane] = on ? e * rq : 0.f;
        if (lane == 31) vec[3 * C] = e;   // tokens past the end have g = 0

        float x[C], att[C];
        const float kb = rk * beta;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const float ci = __shfl_sync(0xffffffffu, cs, i), li = __shfl_sync(0xffffffffu, cl, i);
            const float ri = __shfl_sync(0xffffffffu, rk, i), qi = __shfl_sync(0xffffffffu, rq, i);
            const float d = lane <= i ? __expf((ci - cs) + (li - cl)) * kb : 0.f;
            A[i][lane] = lane < i ? kk[i][lane] * ri * d : 0.f;
            att[i] = lane <= i ? qk[i][lane] * qi * d : 0.f;
            x[i] = 0.f;
        }
        __syncwarp();
        // column `lane` of Inv by forward substitution: x_i = [i = lane] - sum_{k < i} A_ik x_k
#pragma unroll
        for (int i = 0; i < C; ++i) {
            float s0 = i == lane ? 1.f : 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int k = 0; k < i; k += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&A[i][k]);
                s0 = fmaf(-v.x, x[k], s0);
                s1 = fmaf(-v.y, x[k + 1], s1);
                s2 = fmaf(-v.z, x[k + 2], s2);
                s3 = fmaf(-v.w, x[k + 3], s3);
            }
            x[i] = (s0 + s1) + (s2 + s3);
        }
        __syncwarp();
        // rows i and i + 1, two columns to a lane: even lanes store row i, odd ones row i + 1
#pragma unroll
        for (int i = 0; i < C; i += 2) {
            const float x0 = i == lane ? 0.f : x[i], x1 = i + 1 == lane ? 0.f : x[i + 1];
            const bool odd = lane & 1;
            const float xo = __shfl_xor_sync(0xffffffffu, odd ? x0 : x1, 1);
            const float ao = __shfl_xor_sync(0xffffffffu, odd ? att[i] : att[i + 1], 1);
            const int off = ((i + odd) * C + (lane & ~1)) * 2;
            uint32_t hi, lo;
            split2(odd ? xo : x0, odd ? x1 : xo, hi, lo);
            *reinterpret_cast<uint32_t *>(item + DeltaItem::kInvHi + off) = hi;
            *reinterpret_cast<uint32_t *>(item + DeltaItem::kInvLo + off) = lo;
            split2(odd ? ao : att[i], odd ? att[i + 1] : ao, hi, lo);
            *reinterpret_cast<uint32_t *>(item + DeltaItem::kAttHi + off) = hi;
            *reinterpret_cast<uint32_t *>(item + DeltaItem::kAttLo + off) = lo;
        }
    }
}

// Shared-memory stage of one chunk: K and Q of the group, then the head's V (and dO, for the
// backward), its triangles and its factors.  Rows are 16 bytes longer than their data.
struct ChainStage {
    int kpitch, vpitch, head, tri, vec, state, w, total;   // bytes; from tri on offsets in the head's part
    static constexpr int kTriPitch = C * 2 + 16;
    static constexpr int kTri = C * kTriPitch;
    // bwd: with dO; adjoint: also the state behind a span, and W (in
    // accumulator layout)
    __host__ __device__ ChainStage(int rows, int N, bool bwd, bool adjoint = false)
        : kpitch(N * 2 + 16), vpitch(rows * 2 + 16), head(2 * C * kpitch),
          tri((bwd ? 2 : 1) * C * (rows * 2 + 16)), vec(tri + 4 * kTri), state(vec + 512),
          w(state + (adjoint ? rows * state_pitch(N) : 0)),
          total(head + w + (adjoint ? rows * C * 4 : 0))
    {
    }
    static __host__ __device__ constexpr int state_pitch(int N) { return N * 4 + 32; }
};
// The adjoint chain reads the states and W through its stage where a CTA has one warp of rows, bound by
// what a chunk waits for (2 x 2048 tokens x 24 heads, dS in two parts: 183 -> 162 us); with more rows the space is
// worth more as a second CTA on the SM.
__host__ __device__ constexpr bool adjoint_staged(int rows) { return rows == 16; }

// The CTA's share of a launch: see delta_chain_kernel.
struct ChainSlice {
    int64_t b, seq;
    int h, g, pb, rows;
    __device__ ChainSlice(const DeltaArgs &a, int rows_, bool packed) : rows(rows_)
    {
        const int splits = a.P / rows, blocks = a.H * splits;
        pb = (int)(blockIdx.x % splits) * rows;
        h = (int)(blockIdx.x % blocks) / splits;
        seq = blockIdx.x / blocks;
        g = h / (a.H / a.G);
        b = packed ? 0 : seq;
    }
};

// Issues the copies of chunk c into the stage at shared address s: the load warps.
template <int N, bool kBwd>
__device__ __forceinline__ void load_stage(const DeltaArgs &a, const ChainStage &lay,
                                           const ChainSlice &w, const char *items,
                                           const bf16 *dout, int64_t nchunks, const int2 *tab,
                                           int64_t c, uint32_t s)
{
    int64_t t0;
    int len;
    chunk_span(tab, c, C, a.L, t0, len);
    const int64_t row0 = w.b * a.L + t0;
    const int tid = threadIdx.x % (kLoadWarps * 32);
    constexpr int nthr = kLoadWarps * 32;
    const bf16 *kg = static_cast<const bf16 *>(a.k) + (row0 * a.G + w.g) * N;
    const bf16 *qg = static_cast<const bf16 *>(a.q) + (row0 * a.G + w.g) * N;
    for (int i = tid; i < C * (N / 8); i += nthr) {
        const int r = i / (N / 8), col = i % (N / 8);
        const bool on = r < len;
        const int64_t off = on ? (int64_t)r * a.G * N + col * 8 : 0;
        cp16(s + r * lay.kpitch + col * 16, kg + off, on);
        cp16(s + (C + r) * lay.kpitch + col * 16, qg + off, on);
    }
    const uint32_t sh = s + lay.head;
    const int64_t vat = (row0 * a.H + w.h) * a.P + w.pb;
    const bf16 *vg = static_cast<const bf16 *>(a.v) + vat;
    const int pieces = w.rows / 8;
    for (int i = tid; i < C * pieces; i += nthr) {
        const int r = i / pieces, col = i % pieces;
        const bool on = r < len;
        const int64_t off = on ? (int64_t)r * a.H * a.P + col * 8 : 0;
        cp16(sh + r * lay.vpitch + col * 16, vg + off, on);
        if (kBwd) cp16(sh + (C + r) * lay.vpitch + col * 16, dout + vat + off, on);
    }
    const char *item = items + ((w.b * nchunks + c) * a.H + w.h) * DeltaItem::kBytes;
    constexpr int kTris = 4;
    for (int i = tid; i < kTris * C * 4 + 32; i += nthr) {
        if (i < kTris * C * 4) {   // Inv's two parts, Att's: rows of four 16-byte pieces
            const int m = i / (C * 4), r = i / 4 % C, col = i % 4;
            const int src = m < 2 ? m * DeltaItem::kTri : DeltaItem::kAttHi + (m - 2) * DeltaItem::kTri;
            cp16(sh + lay.tri + m * ChainStage::kTri + r * ChainStage::kTriPitch + col * 16,
                 item + src + r * C * 2 + col * 16, true);
        } else {
            const int j = i - kTris * C * 4;
            cp16(sh + lay.vec + j * 16, item + DeltaItem::kVec + j * 16, true);
        }
    }
}

// Rows p and p + 8 of a float32 P x N matrix as accumulators, `m` at (row p, this lane's column).
template <int N> __device__ __forceinline__ void load_acc(const float *m, float (&S)[N / 8][4])
{
#pragma unroll
    for (int n = 0; n < N / 8; ++n) {
        const float2 u = *reinterpret_cast<const float2 *>(m + n * 8);
        const float2 v = *reinterpret_cast<const float2 *>(m + 8 * N + n * 8);
        S[n][0] = u.x; S[n][1] = u.y; S[n][2] = v.x; S[n][3] = v.y;
    }
}
template <int N> __device__ __forceinline__ void store_acc(float *m, const float (&S)[N / 8][4])
{
#pragma unroll
    for (int n = 0; n < N / 8; ++n) {
        *reinterpret_cast<float2 *>(m + n * 8) = make_float2(S[n][0], S[n][1]);
        *reinterpret_cast<float2 *>(m + 8 * N + n * 8) = make_float2(S[n][2], S[n][3]);
    }
}

// Writes a 16 x 32 accumulator (rows p, columns tokens) rounded to bf16 as 32 rows of 16 values,
// through this warp's columns of a tile that nobody reads any more.
__device__ __forceinline__ void store_tokens(const float (&O)[4][4], uint32_t tile, int pitch,
                                             uint32_t frag, bf16 *to, int64_t stride, int len,
                                             int lane)
{
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        uint32_t fo[4];
        round_a(O[2 * n], O[2 * n + 1], fo);
        stsm4_trans(frag + n * 16 * pitch, fo);
    }
    __syncwarp();
#pragma unroll
    for (int i = lane; i < C * 2; i += 32) {   // 32 bytes of a row: two lanes
        const int r = i / 2, half = i % 2;
        if (r < len) {
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(tile + r * pitch + half * 16) : "memory");
            *reinterpret_cast<uint4 *>(to + (int64_t)r * stride + half * 8) = v;
        }
    }
}

// Sums v[i] over the eight lanes of equal lane % 4, i = dot * 8 + (token tile) * 2 + e for kDots
// dots; afterwards lane l has, in v[0] and v[1] (e), the sums of token tile (l >> 2) & 3, and of
// dot l >> 4 for two dots (one dot: v[0] holds e = l >> 4).
template <int kDots> __device__ __forceinline__ void fold_tokens(float (&v)[kDots * 8], int lane)
{
    if constexpr (kDots == 2) {
#pragma unroll
        for (int n = 8, o = 16; n > 1; n >>= 1, o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float mine = up ? v[n + i] : v[i], other = up ? v[i] : v[n + i];
                v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
        }
    } else {
#pragma unroll
        for (int n = 4, o = 8; n > 1; n >>= 1, o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float mine = up ? v[n + i] : v[i], other = up ? v[i] : v[n + i];
                v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
        }
        const bool up = lane & 16;
        const float mine = up ? v[1] : v[0], other = up ? v[0] : v[1];
        v[0] = mine + __shfl_xor_sync(0xffffffffu, other, 16);
    }
}

// A CTA has `rows` rows p of a head: rows / 16 warps.  grid: (sequences * H * P / rows).  kBwd: the
// forward once more for the backward, which keeps the state every 64 tokens, W, and the dot products of
// o and its gradient instead of o.
template <int N, bool kBwd>
__global__ void __launch_bounds__((kMaxRows / 16 + kLoadWarps) * 32)
delta_chain_kernel(const DeltaArgs a, const DeltaBwd w, const char *items, int64_t nchunks,
                   const int2 *tab, const int32_t *cstart, const int *status, int rows)
{
    extern __shared__ __align__(128) char smem[];
    if (status && *status) {
        wait_before();
        return;
    }
    constexpr int NT = N / 8;
    const int P = a.P;
    const ChainStage lay(rows, N, kBwd);
    const ChainSlice slice(a, rows, cstart != nullptr);
    const int tid = threadIdx.x, lane = tid % 32, pl = tid / 32 * 16;   // this warp's rows of the CTA's
    const int p0 = slice.pb + pl, h = slice.h;
    const int64_t b = slice.b, seq = slice.seq;
    const int64_t c_begin = cstart ? cstart[seq] : 0, c_end = cstart ? cstart[seq + 1] : nchunks;

    const uint32_t base = smem_u32(smem);
    if (pl >= rows) {   // the load warps: a chunk ahead of the others
        wait_before();   // the others read nothing of the kernel before
        for (int64_t c = c_begin; c <= c_end; ++c) {
            if (c < c_end)
                load_stage<N, kBwd>(a, lay, slice, items, w.dout, nchunks, tab, c,
                                    base + ((c - c_begin) & 1) * lay.total);
            cp_commit();
            cp_wait<0>();
            __syncthreads();   // chunk c has arrived; chunk c - 1 is done with
        }
        return;
    }
    float S[NT][4] = {};
    const int64_t pn = (int64_t)(p0 + lane / 4) * N + lane % 4 * 2;   // this lane, in a P x N state
    const int64_t srow = (seq * a.H + h) * P * N + pn;
    if (a.init) load_acc<N>(a.init + srow, S);

    // fragment addresses inside a stage
    const int row_nn = lane % 8 + lane / 16 * 8, col_nn = (lane / 8 & 1) * 16;   // rows on n
    const int row_kk = lane % 8 + (lane / 8 & 1) * 8, col_kk = lane / 16 * 16;   // rows on k
    for (int64_t c = c_begin; c < c_end; ++c) {
        const int stage = (int)(c - c_begin) & 1;
        __syncthreads();   // this chunk has arrived; everyone is done with the other stage

        const uint32_t ks = base + stage * lay.total, qs = ks + C * lay.kpitch;
        const uint32_t vs = ks + lay.head;
        const uint32_t inv = vs + lay.tri, att = inv + 2 * ChainStage::kTri;
        const float *vec =
            reinterpret_cast<const float *>(smem + stage * lay.total + lay.head + lay.vec);
        const int64_t item = (b * nchunks + c) * a.H + h;
        if (kBwd && c % 2 == 0)
            store_acc<N>(w.states + ((b * (w.n64 + 1) + c / 2) * a.H + h) * P * N + pn, S);

        // S K^T and S Q^T (columns: tokens)
        float X[4][4] = {}, O[4][4] = {};
#pragma unroll
        for (int s = 0; s < N / 16; ++s) {
            uint32_t hi[4], lo[4], fb[4];
            split_a(S[2 * s], S[2 * s + 1], hi, lo);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                ldsm4(fb, ks + (n * 16 + row_nn) * lay.kpitch + s * 32 + col_nn);
                mma_16816(X[2 * n], hi, fb[0], fb[1]);
                mma_16816(X[2 * n + 1], hi, fb[2], fb[3]);
                mma_16816(X[2 * n], lo, fb[0], fb[1]);
                mma_16816(X[2 * n + 1], lo, fb[2], fb[3]);
                ldsm4(fb, qs + (n * 16 + row_nn) * lay.kpitch + s * 32 + col_nn);
                mma_16816(O[2 * n], hi, fb[0], fb[1]);
                mma_16816(O[2 * n + 1], hi, fb[2], fb[3]);
                mma_16816(O[2 * n], lo, fb[0], fb[1]);
                mma_16816(O[2 * n + 1], lo, fb[2], fb[3]);
            }
        }
        // R = V - e K S^T, in place of S K^T; the output's part from the state takes its factor
        const uint32_t vaddr = vs + pl * 2 + row_nn * lay.vpitch + col_nn;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint32_t fv[4];
            ldsm4_trans(fv, vaddr + n * 16 * lay.vpitch);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int t = 2 * n + m;
                const float2 ek = *reinterpret_cast<const float2 *>(vec + t * 8 + lane % 4 * 2);
                const float2 eq =
                    *reinterpret_cast<const float2 *>(vec + 2 * C + t * 8 + lane % 4 * 2);
                X[t][0] = fmaf(-ek.x, X[t][0], bf16_lo(fv[2 * m]));
                X[t][1] = fmaf(-ek.y, X[t][1], bf16_hi(fv[2 * m]));
                X[t][2] = fmaf(-ek.x, X[t][2], bf16_lo(fv[2 * m + 1]));
                X[t][3] = fmaf(-ek.y, X[t][3], bf16_hi(fv[2 * m + 1]));
                O[t][0] *= eq.x; O[t][1] *= eq.y; O[t][2] *= eq.x; O[t][3] *= eq.y;
            }
        }
        // W = R + (Inv - I) R: blocks of 16 tokens on and below the diagonal
        float W[4][4];
        {
            uint32_t hi[2][4], lo[2][4];
            split_a(X[0], X[1], hi[0], lo[0]);
            split_a(X[2], X[3], hi[1], lo[1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) W[t][r] = X[t][r];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int s = 0; s <= n; ++s) {
                    uint32_t fh[4], fl[4];
                    const uint32_t at =
                        inv + (n * 16 + row_nn) * ChainStage::kTriPitch + s * 32 + col_nn;
                    ldsm4(fh, at);
                    ldsm4(fl, at + ChainStage::kTri);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        mma_16816(W[2 * n + m], hi[s], fh[2 * m], fh[2 * m + 1]);
                        mma_16816(W[2 * n + m], lo[s], fh[2 * m], fh[2 * m + 1]);
                        mma_16816(W[2 * n + m], hi[s], fl[2 * m], fl[2 * m + 1]);
                    }
                }
        }
        // O += Att W
        {
            uint32_t hi[2][4], lo[2][4], rest[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if constexpr (kBwd) split_a(W[2 * s], W[2 * s + 1], hi[s], lo[s], rest[s]);
                else split_a(W[2 * s], W[2 * s + 1], hi[s], lo[s]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int s = 0; s <= n; ++s) {
                    uint32_t fb[4], fl[4];
                    const uint32_t at =
                        att + (n * 16 + row_nn) * ChainStage::kTriPitch + s * 32 + col_nn;
                    ldsm4(fb, at);
                    ldsm4(fl, at + ChainStage::kTri);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        mma_16816(O[2 * n + m], hi[s], fb[2 * m], fb[2 * m + 1]);
                        mma_16816(O[2 * n + m], lo[s], fb[2 * m], fb[2 * m + 1]);
                        mma_16816(O[2 * n + m], hi[s], fl[2 * m], fl[2 * m + 1]);
                        if constexpr (kBwd) {
                            mma_16816(O[2 * n + m], rest[s], fb[2 * m], fb[2 * m + 1]);
                            mma_16816(O[2 * n + m], lo[s], fl[2 * m], fl[2 * m + 1]);
                        }
                    }
                }
        }
        if constexpr (kBwd) {
            float d[8];   // <dO, O> over this warp's rows, per token
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t fd[4];
                ldsm4_trans(fd, vaddr + (C + n * 16) * lay.vpitch);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int t = 2 * n + m;
                    d[2 * t] = fmaf(bf16_lo(fd[2 * m]), O[t][0], bf16_lo(fd[2 * m + 1]) * O[t][2]);
                    d[2 * t + 1] =
                        fmaf(bf16_hi(fd[2 * m]), O[t][1], bf16_hi(fd[2 * m + 1]) * O[t][3]);
                }
            }
            fold_tokens<1>(d, lane);
            const int64_t tile = item * (P / 16) + p0 / 16;
            w.dot_oo[tile * C + (lane >> 2 & 3) * 8 + lane % 4 * 2 + (lane >> 4)] = d[0];
            float4 *wf = reinterpret_cast<float4 *>(w.wfrag + tile * (16 * C)) + lane;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                wf[t * 32] = make_float4(W[t][0], W[t][1], W[t][2], W[t][3]);
        }
        // S = E S + (E / e beta W)^T K
        const float E = vec[3 * C];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[n][r] *= E;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 sw = *reinterpret_cast<const float2 *>(vec + C + t * 8 + lane % 4 * 2);
            W[t][0] *= sw.x; W[t][1] *= sw.y; W[t][2] *= sw.x; W[t][3] *= sw.y;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint32_t hi[4], lo[4], rest[4];
            if constexpr (kBwd) split_a(W[2 * s], W[2 * s + 1], hi, lo, rest);
            else split_a(W[2 * s], W[2 * s + 1], hi, lo);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                uint32_t fb[4];
                ldsm4_trans(fb, ks + (s * 16 + row_kk) * lay.kpitch + n * 32 + col_kk);
                mma_16816(S[2 * n], hi, fb[0], fb[1]);
                mma_16816(S[2 * n + 1], hi, fb[2], fb[3]);
                mma_16816(S[2 * n], lo, fb[0], fb[1]);
                mma_16816(S[2 * n + 1], lo, fb[2], fb[3]);
                if constexpr (kBwd) {
                    mma_16816(S[2 * n], rest, fb[0], fb[1]);
                    mma_16816(S[2 * n + 1], rest, fb[2], fb[3]);
                }
            }
        }
        if constexpr (!kBwd) {
            int64_t t0;
            int len;
            chunk_span(tab, c, C, a.L, t0, len);
            store_tokens(O, vs + pl * 2, lay.vpitch, vaddr,
                         static_cast<bf16 *>(a.o) + ((b * a.L + t0) * a.H + h) * P + p0,
                         (int64_t)a.H * P, len, lane);
        }
    }
    __syncthreads();   // the load warps' last one
    let_next_start();
    if (kBwd)
        store_acc<N>(w.states + ((b * (w.n64 + 1) + w.n64) * a.H + h) * P * N + pn, S);
    else if (a.final_state)
        store_acc<N>(a.final_state + srow, S);
}

// The adjoint recurrence, chunk by chunk from the end, in the same layout (dS in registers, rows p
// per warp).  With Y = beta dL/dU, the gradient of the written values:
//
//     Y  = Att^T dO + sw K dS'^T,    dV = Inv^T Y,
//     dS = E dS' + (eq dO)^T Q - (ek dV)^T K
//
// sw, ek and eq are the factors of the forward (decays, norms, beta, scale).  It writes dV, the dot
// products of each token's dV with V and W, every 64 tokens dS' (bf16) and <dS', S'>, and dS of
// the initial state.
template <int N>
__global__ void __launch_bounds__((kMaxRows / 16 + kLoadWarps) * 32)
delta_adjoint_kernel(const DeltaArgs a, const DeltaBwd w, const char *items, int64_t nchunks,
                     int rows)
{
    extern __shared__ __align__(128) char smem[];
    wait_before();
    constexpr int NT = N / 8;
    const int P = a.P;
    const bool staged = adjoint_staged(rows);
    const ChainStage lay(rows, N, true, staged);
    const ChainSlice slice(a, rows, false);
    const int tid = threadIdx.x, lane = tid % 32, pl = tid / 32 * 16;
    const int p0 = slice.pb + pl, h = slice.h;
    const int64_t b = slice.b;

    const uint32_t base = smem_u32(smem);
    if (pl >= rows) {   // the load warps
        for (int64_t c = nchunks - 1; c >= -1; --c) {
            const uint32_t to = base + ((nchunks - 1 - c) & 1) * lay.total;
            if (c >= 0) load_stage<N, true>(a, lay, slice, items, w.dout, nchunks, nullptr, c, to);
            if (c >= 0 && staged) {   // 16 rows
                const int i0 = tid % (kLoadWarps * 32);
                const uint32_t head = to + lay.head;
                const int64_t item = (b * nchunks + c) * a.H + h;
                const float *wf = w.wfrag + (item * (P / 16) + slice.pb / 16) * (16 * C);
                for (int i = i0; i < 16 * C / 4; i += kLoadWarps * 32)
                    cp16(head + lay.w + i * 16, wf + i * 4, true);
                if (c % 2 == 1 || c == nchunks - 1) {
                    const float *sn = w.states + (((b * (w.n64 + 1) + c / 2 + 1) * a.H + h) * P +
                                                  slice.pb) * (int64_t)N;
                    for (int i = i0; i < 16 * N / 4; i += kLoadWarps * 32)
                        cp16(head + lay.state + i / (N / 4) * lay.state_pitch(N) + i % (N / 4) * 16,
                             sn + i * 4, true);
                }
            }
            cp_commit();
            cp_wait<0>();
            __syncthreads();
        }
        return;
    }
    float D[NT][4] = {};
    const int64_t pn = (int64_t)(p0 + lane / 4) * N + lane % 4 * 2;
    const int64_t srow = (b * a.H + h) * P * N + pn;
    if (w.dfinal) load_acc<N>(w.dfinal + srow, D);

    const int row_nn = lane % 8 + lane / 16 * 8, col_nn = (lane / 8 & 1) * 16;   // rows on n
    const int row_kk = lane % 8 + (lane / 8 & 1) * 8, col_kk = lane / 16 * 16;   // rows on k
    for (int64_t c = nchunks - 1; c >= 0; --c) {
        const int stage = (int)(nchunks - 1 - c) & 1;
        __syncthreads();

        const uint32_t ks = base + stage * lay.total, qs = ks + C * lay.kpitch;
        const uint32_t vs = ks + lay.head;
        const uint32_t inv = vs + lay.tri, att = inv + 2 * ChainStage::kTri;
        const char *part = smem + stage * lay.total + lay.head;
        const float *vec = reinterpret_cast<const float *>(part + lay.vec);
        const int64_t item = (b * nchunks + c) * a.H + h;
        const int64_t tile = item * (P / 16) + p0 / 16;
        float4 wf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            wf[t] = staged ? *reinterpret_cast<const float4 *>(part + lay.w + (t * 32 + lane) * 16)
                           : reinterpret_cast<const float4 *>(w.wfrag + tile * (16 * C))[t * 32 + lane];

        if (c % 2 == 1 || c == nchunks - 1) {   // the end of a span of 64 tokens
            const int64_t span = (b * w.n64 + c / 2) * a.H + h;
            // this lane's first row and the one 8 below
            const float *sn = w.states + ((b * (w.n64 + 1) + c / 2 + 1) * a.H + h) * P * N + pn;
            int below = 8 * N;
            if (staged) {
                sn = reinterpret_cast<const float *>(part + lay.state + lane / 4 * lay.state_pitch(N)) +
                     lane % 4 * 2;
                below = 8 * lay.state_pitch(N) / 4;
            }
            bf16 *ds = w.dstates + span * P * N + pn;
            float f = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 u = *reinterpret_cast<const float2 *>(sn + n * 8);
                const float2 v = *reinterpret_cast<const float2 *>(sn + below + n * 8);
                f = fmaf(D[n][0], u.x, fmaf(D[n][1], u.y, fmaf(D[n][2], v.x, fmaf(D[n][3], v.y, f))));
                *reinterpret_cast<uint32_t *>(ds + n * 8) = pack_bf16x2(D[n][0], D[n][1]);
                *reinterpret_cast<uint32_t *>(ds + 8 * N + n * 8) = pack_bf16x2(D[n][2], D[n][3]);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
            if (lane == 0)
                w.dot_ss[((b * (w.n64 + 1) + c / 2 + 1) * a.H + h) * (P / 16) + p0 / 16] = f;
        }

        // dS' K^T (columns: tokens)
        float Y[4][4] = {};
#pragma unroll
        for (int s = 0; s < N / 16; ++s) {
            uint32_t hi[4], lo[4], rest[4], fb[4];
            split_a(D[2 * s], D[2 * s + 1], hi, lo, rest);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                ldsm4(fb, ks + (n * 16 + row_nn) * lay.kpitch + s * 32 + col_nn);
                mma_16816(Y[2 * n], hi, fb[0], fb[1]);
                mma_16816(Y[2 * n + 1], hi, fb[2], fb[3]);
                mma_16816(Y[2 * n], lo, fb[0], fb[1]);
                mma_16816(Y[2 * n + 1], lo, fb[2], fb[3]);
                mma_16816(Y[2 * n], rest, fb[0], fb[1]);
                mma_16816(Y[2 * n + 1], rest, fb[2], fb[3]);
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 sw = *reinterpret_cast<const float2 *>(vec + C + t * 8 + lane % 4 * 2);
            Y[t][0] *= sw.x; Y[t][1] *= sw.y; Y[t][2] *= sw.x; Y[t][3] *= sw.y;
        }
        // Y += dO^T Att: blocks of 16 tokens on and below Att's diagonal.  dO^T, read transposed,
        // is an A operand as it is.
        const uint32_t vaddr = vs + pl * 2 + row_nn * lay.vpitch + col_nn;
        const uint32_t daddr = vaddr + C * lay.vpitch;
        uint32_t fd[2][4];
        ldsm4_trans(fd[0], daddr);
        ldsm4_trans(fd[1], daddr + 16 * lay.vpitch);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int n = 0; n <= s; ++n) {
                uint32_t fh[4], fl[4];
                const uint32_t at =
                    att + (s * 16 + row_kk) * ChainStage::kTriPitch + n * 32 + col_kk;
                ldsm4_trans(fh, at);
                ldsm4_trans(fl, at + ChainStage::kTri);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_16816(Y[2 * n + m], fd[s], fh[2 * m], fh[2 * m + 1]);
                    mma_16816(Y[2 * n + m], fd[s], fl[2 * m], fl[2 * m + 1]);
                }
            }
        // dV = Y + (Inv - I)^T Y
        float V[4][4];
        {
            uint32_t hi[2][4], lo[2][4];
            split_a(Y[0], Y[1], hi[0], lo[0]);
            split_a(Y[2], Y[3], hi[1], lo[1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) V[t][r] = Y[t][r];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int n = 0; n <= s; ++n) {
                    uint32_t fh[4], fl[4];
                    const uint32_t at =
                        inv + (s * 16 + row_kk) * ChainStage::kTriPitch + n * 32 + col_kk;
                    ldsm4_trans(fh, at);
                    ldsm4_trans(fl, at + ChainStage::kTri);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        mma_16816(V[2 * n + m], hi[s], fh[2 * m], fh[2 * m + 1]);
                        mma_16816(V[2 * n + m], lo[s], fh[2 * m], fh[2 * m + 1]);
                        mma_16816(V[2 * n + m], hi[s], fl[2 * m], fl[2 * m + 1]);
                    }
                }
        }
        // per token: <dV, V> and <dV, W> over this warp's rows
        {
            float d[16];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t fv[4];
                ldsm4_trans(fv, vaddr + n * 16 * lay.vpitch);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int t = 2 * n + m;
                    d[2 * t] = fmaf(bf16_lo(fv[2 * m]), V[t][0], bf16_lo(fv[2 * m + 1]) * V[t][2]);
                    d[2 * t + 1] =
                        fmaf(bf16_hi(fv[2 * m]), V[t][1], bf16_hi(fv[2 * m + 1]) * V[t][3]);
                    d[8 + 2 * t] = fmaf(wf[t].x, V[t][0], wf[t].z * V[t][2]);
                    d[8 + 2 * t + 1] = fmaf(wf[t].y, V[t][1], wf[t].w * V[t][3]);
                }
            }
            fold_tokens<2>(d, lane);
            float *to = (lane & 16 ? w.dot_vw : w.dot_vv) + tile * C;
            *reinterpret_cast<float2 *>(to + (lane >> 2 & 3) * 8 + lane % 4 * 2) =
                make_float2(d[0], d[1]);
        }
        int64_t t0;
        int len;
        chunk_span(nullptr, c, C, a.L, t0, len);
        store_tokens(V, vs + pl * 2, lay.vpitch, vaddr,
                     w.dv + ((b * a.L + t0) * a.H + h) * P + p0, (int64_t)a.H * P, len, lane);

        // dS = E dS' + (eq dO)^T Q - (ek dV)^T K
        const float E = vec[3 * C];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) D[n][r] *= E;
        float Z[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 ek = *reinterpret_cast<const float2 *>(vec + t * 8 + lane % 4 * 2);
            const float2 eq = *reinterpret_cast<const float2 *>(vec + 2 * C + t * 8 + lane % 4 * 2);
            const uint32_t x = fd[t / 2][t % 2 * 2], y = fd[t / 2][t % 2 * 2 + 1];
            Z[t][0] = eq.x * bf16_lo(x); Z[t][1] = eq.y * bf16_hi(x);
            Z[t][2] = eq.x * bf16_lo(y); Z[t][3] = eq.y * bf16_hi(y);
            V[t][0] *= -ek.x; V[t][1] *= -ek.y; V[t][2] *= -ek.x; V[t][3] *= -ek.y;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint32_t zh[4], zl[4], vh[4], vl[4];
            split_a(Z[2 * s], Z[2 * s + 1], zh, zl);
            split_a(V[2 * s], V[2 * s + 1], vh, vl);
            const uint32_t at = (s * 16 + row_kk) * lay.kpitch + col_kk;
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                uint32_t fq[4], fk[4];
                ldsm4_trans(fq, qs + at + n * 32);
                ldsm4_trans(fk, ks + at + n * 32);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma_16816(D[2 * n + m], zh, fq[2 * m], fq[2 * m + 1]);
                    mma_16816(D[2 * n + m], vh, fk[2 * m], fk[2 * m + 1]);
                    mma_16816(D[2 * n + m], zl, fq[2 * m], fq[2 * m + 1]);
                    mma_16816(D[2 * n + m], vl, fk[2 * m], fk[2 * m + 1]);
                }
            }
        }
    }
    __syncthreads();   // the load warps' last one
    let_next_start();
    if (w.dinit) store_acc<N>(w.dinit + srow, D);
    float f = 0.f;   // <dS, S> at the start
    if (a.init) {
        float S[NT][4];
        load_acc<N>(a.init + srow, S);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) f = fmaf(D[n][r], S[n][r], f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    }
    if (lane == 0) w.dot_ss[(b * (w.n64 + 1) * a.H + h) * (P / 16) + p0 / 16] = f;
}

// Rows of a head per CTA: all of them (half of 128), or fewer where the launch would leave SMs empty.
int chain_rows(const DeltaArgs &a, int64_t nseq)
{
    int rows = a.P > kMaxRows ? a.P / 2 : a.P;
    while (nseq * a.H * (a.P / rows) < 148 && rows % 32 == 0) rows /= 2;
    return rows;
}

}  // namespace

bool delta_chunk_supported(bool is_bf16, int P, int N)
{
    return is_bf16 && (N == 64 || N == 128) && P % 16 == 0 && P <= 128;
}

cudaError_t launch_delta_prep(const DeltaArgs &a, char *items, bool for_backward, int64_t nchunks,
                              const int2 *tab, cudaStream_t st)
{
    // fewer heads per CTA where the launch would leave SMs empty (at 1 x 64 tokens x 24 heads 16 heads
    // to a CTA took 28 us, 4 of them 8)
    const int64_t batch = tab ? 1 : a.batch, hpg = a.H / a.G;
    int run = hpg < kPrepHeads ? (int)hpg : kPrepHeads;
    auto runs = [&] { return (hpg + run - 1) / run; };
    while (run > kPrepWarps && nchunks * batch * a.G * runs() < 592) run = (run + 1) / 2;
    const dim3 grid((unsigned)nchunks, (unsigned)batch, (unsigned)(a.G * runs()));
    const dim3 block(kPrepWarps * 32);
    auto go = [&](auto kern) {
        kern<<<grid, block, 0, st>>>(a, items, nchunks, tab, run);
        return cudaGetLastError();
    };
    if (a.N == 128)
        return for_backward ? go(delta_prep_kernel<128, true>) : go(delta_prep_kernel<128, false>);
    return for_backward ? go(delta_prep_kernel<64, true>) : go(delta_prep_kernel<64, false>);
}

cudaError_t launch_delta_chain(const DeltaArgs &a, const DeltaBwd *bwd, const char *items,
                               int64_t nchunks, const int2 *tab, const int32_t *cstart,
                               const int *status, cudaStream_t st)
{
    const int64_t nseq = cstart ? a.nseq : a.batch;
    const int rows = chain_rows(a, nseq);
    const unsigned grid = (unsigned)(nseq * a.H * (a.P / rows));
    const unsigned threads = (unsigned)((rows / 16 + kLoadWarps) * 32);
    const int smem = 2 * ChainStage(rows, a.N, bwd != nullptr).total;
    const DeltaBwd w = bwd ? *bwd : DeltaBwd{};
    auto go = [&](auto kern) {
        return launch_after(kern, grid, threads, smem, st, a, w, items, nchunks, tab, cstart, status, rows);
    };
    if (bwd) return a.N == 128 ? go(delta_chain_kernel<128, true>) : go(delta_chain_kernel<64, true>);
    return a.N == 128 ? go(delta_chain_kernel<128, false>) : go(delta_chain_kernel<64, false>);
}

cudaError_t launch_delta_adjoint(const DeltaArgs &a, const DeltaBwd &w, const char *items,
                                 int64_t nchunks, cudaStream_t st)
{
    const int rows = chain_rows(a, a.batch);
    const unsigned grid = (unsigned)(a.batch * a.H * (a.P / rows));
    const unsigned threads = (unsigned)((rows / 16 + kLoadWarps) * 32);
    const int smem = 2 * ChainStage(rows, a.N, true, adjoint_staged(rows)).total;
    auto go = [&](auto kern) {
        return launch_after(kern, grid, threads, smem, st, a, w, items, nchunks, rows);
    };
    return a.N == 128 ? go(delta_adjoint_kernel<128>) : go(delta_adjoint_kernel<64>);
}

}  // namespace ssd
