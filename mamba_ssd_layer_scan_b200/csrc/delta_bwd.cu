// The gated delta rule's gradients of q, k, g and beta, once the two chains (delta_chunk.cu) have
// left the states, their gradients, W and dV.
//
// Per span of 64 tokens and head, with D_ij = exp(cs_i - cs_j), S the state entering the span, dS'
// the gradient of the state leaving it, and q, k as stored (rq, rk the norms' inverses, or 1):
//
//     M1_ij = D_ij scale beta_j rq_i rk_j (dO_i . W_j)   j <= i
//     M2_ij = D_ij beta_j rk_i rk_j (dV_i . W_j)         j < i
//     rq dq = eq dO S + M1 K
//     rk dk = sw W dS' - ek dV S + M1^T Q - (M2 + M2^T) K
//
// with eq = e rq scale, ek = e rk, sw = (E / e) rk beta.  The gradients of the stored rows follow
// from those of the normalised ones, y = q rq: dq = t - y (y . t), t = rq d(y).
//
// The decay's gradient at a token is <dS, S> before it, S having decayed; within a span of n tokens it
// telescopes from either end, with x_s = <dO_s, O_s> - <dV_s, V_s>:
//
//     dg_t = <dS', S'> + sum over s >= t of x_s = <dS, S> - sum over s < t of x_s
//     dbeta_t = <dV_t, W_t> / beta_t
//
// where the dot products come from the chains in float32 (the gradients' kernel takes 97 us at 2 x 2048
// tokens x 24 heads, latency of a head's loads and barriers, with two CTAs to an SM).  The errors of the two
// sums add up over n - t and t terms that partly cancel; weighted by t / n and (n - t) / n they give 0.6 of
// the first one's error alone (dg at 2 x 2048 x 24 heads: 4e-6, 2-norm).
#include "delta.cuh"
#include "delta_mma.cuh"

namespace ssd {
namespace {

using namespace sm100;

constexpr int kSpan = 64;
constexpr int kGradThreads = 256;

// Tiles of 128- or 256-byte rows, 16-byte piece c of row r at piece c ^ (r % 8): no bank conflicts, and
// two CTAs to an SM for P = 64.  W and M1 are held in two bf16 parts: rounded to one they left dq and dk
// 0.0029 off (2-norm) where their own rounding is 0.0017; now 0.0017 and 0.0019, what dS, S, dV and M2,
// rounded to bf16, add.  The triangles lie where the states were.
struct GradSmem {
    static constexpr int mpitch = kSpan * 2;
    int kpitch, vpitch, k, q, dout, w, wlo, dv, s, ds, m1, m1lo, m2, vec, total;
    __host__ __device__ GradSmem(int P, int N) : kpitch(N * 2), vpitch(P <= 64 ? 128 : 256)
    {
        k = 0;
        q = k + kSpan * kpitch;
        dout = q + kSpan * kpitch;
        w = dout + kSpan * vpitch;
        wlo = w + kSpan * vpitch;
        dv = wlo + kSpan * vpitch;
        s = dv + kSpan * vpitch;
        ds = s + P * kpitch;
        m1 = s;
        m1lo = m1 + kSpan * mpitch;
        m2 = m1lo + kSpan * mpitch;
        const int states = ds + P * kpitch, triangles = m2 + kSpan * mpitch;
        vec = states > triangles ? states : triangles;
        total = vec + 8 * kSpan * 4;
    }
};
__device__ __forceinline__ uint32_t swizzled(int row, int pitch, int piece)
{
    return row * pitch + ((piece ^ (row & 7)) << 4);
}

// grid: (spans, batch, G * runs); 8 warps
template <int N>
__global__ void __launch_bounds__(kGradThreads, 2)
delta_grad_kernel(const DeltaArgs a, const DeltaBwd w)
{
    extern __shared__ __align__(128) char smem[];
    wait_before();
    constexpr int NT = N / 16;   // n8 tiles of a warp's half of the columns
    const GradSmem lay(a.P, N);
    const int P = a.P, H = a.H, hpg = a.H / a.G;
    const int64_t span = blockIdx.x, b = blockIdx.y;
    const int g = blockIdx.z / w.runs, run = blockIdx.z % w.runs;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int mt = warp % 4 * 16, nh = warp / 4;   // this warp's 16 tokens and half of the columns
    const int64_t t0 = span * kSpan, row0 = b * a.L + t0, nchunks = (a.L + kDeltaChunk - 1) / kDeltaChunk;
    const int len = (int)(a.L - t0 < kSpan ? a.L - t0 : kSpan);
    const uint32_t base = smem_u32(smem);
    float *vec = reinterpret_cast<float *>(smem + lay.vec);
    float *cs = vec, *ek = vec + kSpan, *sw = vec + 2 * kSpan, *eq = vec + 3 * kSpan,
          *rks = vec + 4 * kSpan, *rqs = vec + 5 * kSpan, *kb = vec + 6 * kSpan,
          *cl = vec + 7 * kSpan;

    const bf16 *kg = static_cast<const bf16 *>(a.k) + (row0 * a.G + g) * N;
    const bf16 *qg = static_cast<const bf16 *>(a.q) + (row0 * a.G + g) * N;
    for (int i = tid; i < kSpan * (N / 8); i += kGradThreads) {
        const int r = i / (N / 8), col = i % (N / 8);
        const bool on = r < len;
        const int64_t off = on ? (int64_t)r * a.G * N + col * 8 : 0;
        cp16(base + lay.k + swizzled(r, lay.kpitch, col), kg + off, on);
        cp16(base + lay.q + swizzled(r, lay.kpitch, col), qg + off, on);
    }
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    {   // inverse norms: 4 lanes to a token
        const int r = tid / 4;
        float kk = 0.f, qq = 0.f;
        for (int i = tid % 4 * 2; i < N; i += 8) {
            const uint32_t at = swizzled(r, lay.kpitch, i / 8) + i % 8 * 2;
            const uint32_t x = *reinterpret_cast<const uint32_t *>(smem + lay.k + at);
            const uint32_t y = *reinterpret_cast<const uint32_t *>(smem + lay.q + at);
            kk = fmaf(bf16_lo(x), bf16_lo(x), fmaf(bf16_hi(x), bf16_hi(x), kk));
            qq = fmaf(bf16_lo(y), bf16_lo(y), fmaf(bf16_hi(y), bf16_hi(y), qq));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            kk += __shfl_xor_sync(0xffffffffu, kk, o);
            qq += __shfl_xor_sync(0xffffffffu, qq, o);
        }
        if (tid % 4 == 0) {
            rks[r] = a.l2norm ? rsqrtf(kk + kL2Eps) : 1.f;
            rqs[r] = (a.l2norm ? rsqrtf(qq + kL2Eps) : 1.f) * a.scale;
        }
    }

    float dq[NT][4] = {}, dk[NT][4] = {};
    // the row and piece of a fragment's address that are this lane's (rows on n, on k; A)
    const int row_nn = lane % 8 + lane / 16 * 8, col_nn = lane / 8 & 1;
    const int row_kk = lane % 8 + (lane / 8 & 1) * 8, col_kk = lane / 16;
    const int row_a = lane % 16, col_a = lane / 16;
    const int h_end = min(hpg, (run + 1) * w.run_heads);
    for (int hl = run * w.run_heads; hl < h_end; ++hl) {
        const int h = g * hpg + hl;
        __syncthreads();   // everyone is done with the previous head's tiles
        const int64_t vat = (row0 * H + h) * P;
        const int pieces = P / 8;
        for (int i = tid; i < kSpan * pieces; i += kGradThreads) {
            const int r = i / pieces, col = i % pieces;
            const bool on = r < len;
            const int64_t off = vat + (on ? (int64_t)r * H * P + col * 8 : 0);
            const uint32_t at = swizzled(r, lay.vpitch, col);
            cp16(base + lay.dout + at, w.dout + off, on);
            cp16(base + lay.dv + at, w.dv + off, on);
        }
        // W of 16 rows p and 16 tokens at a time, as the chain's accumulators hold it; zeros past the end
        for (int i = warp; i < P / 4; i += kGradThreads / 32) {
            const int tile = i / 4, n = i % 4;
            const int64_t c = span * 2 + n / 2;
            float4 t[2] = {};
            if (c < nchunks) {
                const float *wf = w.wfrag + (((b * nchunks + c) * H + h) * (P / 16) + tile) *
                                                (16 * kDeltaChunk);
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    t[m] = reinterpret_cast<const float4 *>(wf)[(n % 2 * 2 + m) * 32 + lane];
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                split2(t[m].x, t[m].y, hi[2 * m], lo[2 * m]);
                split2(t[m].z, t[m].w, hi[2 * m + 1], lo[2 * m + 1]);
            }
            const uint32_t at = swizzled(n * 16 + row_nn, lay.vpitch, tile * 2 + col_nn);
            stsm4_trans(base + lay.w + at, hi);
            stsm4_trans(base + lay.wlo + at, lo);
        }
        const bf16 *dsg = w.dstates + ((b * w.n64 + span) * H + h) * P * N;
        for (int i = tid; i < P * (N / 8); i += kGradThreads)
            cp16(base + lay.ds + swizzled(i / (N / 8), lay.kpitch, i % (N / 8)), dsg + i * 8, true);
        cp_commit();
        const float *sg = w.states + ((b * (w.n64 + 1) + span) * H + h) * P * N;
        for (int i = tid; i < P * (N / 8); i += kGradThreads) {   // rounded to the operand's bf16
            const float4 u = *reinterpret_cast<const float4 *>(sg + i * 8);
            const float4 v = *reinterpret_cast<const float4 *>(sg + i * 8 + 4);
            uint4 o;
            o.x = pack_bf16x2(u.x, u.y);
            o.y = pack_bf16x2(u.z, u.w);
            o.z = pack_bf16x2(v.x, v.y);
            o.w = pack_bf16x2(v.z, v.w);
            *reinterpret_cast<uint4 *>(smem + lay.s +
                                       swizzled(i / (N / 8), lay.kpitch, i % (N / 8))) = o;
        }
        if (warp == 0) {   // the span's decays: lane has tokens lane and lane + 32
            // running sums of g in two floats, as the forward's kernels take them
            float hi[2], lo[2], beta[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = lane + 32 * x;
                const int64_t at = (row0 + t) * H + h;
                hi[x] = t < len && a.g ? a.g[at] : 0.f;
                lo[x] = 0.f;
                beta[x] = t < len ? a.beta[at] : 0.f;
                if (hi[x] < -200.f) hi[x] = -200.f;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float up = __shfl_up_sync(0xffffffffu, hi[x], o);
                    const float ul = __shfl_up_sync(0xffffffffu, lo[x], o);
                    if (lane >= o) {
                        float e;
                        two_sum(hi[x], up, hi[x], e);
                        lo[x] += ul + e;
                    }
                }
            }
            const float mid = __shfl_sync(0xffffffffu, hi[0], 31);
            const float midl = __shfl_sync(0xffffffffu, lo[0], 31);
            float e;
            two_sum(hi[1], mid, hi[1], e);
            lo[1] += midl + e;
            const float end = __shfl_sync(0xffffffffu, hi[1], 31);
            const float endl = __shfl_sync(0xffffffffu, lo[1], 31);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = lane + 32 * x;
                const bool on = t < len;
                const float e = __expf(hi[x] + lo[x]);
                cs[t] = hi[x];
                cl[t] = lo[x];
                ek[t] = on ? e * rks[t] : 0.f;
                sw[t] = on ? __expf((end - hi[x]) + (endl - lo[x])) * rks[t] * beta[x] : 0.f;
                eq[t] = on ? e * rqs[t] : 0.f;
                kb[t] = on ? rks[t] * beta[x] : 0.f;
            }
        }
        cp_wait<0>();
        __syncthreads();

        // products with the states, then scaled row by row: x, y = tiles of rows (dO, dV, or W's two parts)
        auto with_state = [&](uint32_t x, uint32_t y, uint32_t st, const float *f, float sign,
                              float (&to)[NT][4]) {
            float acc[NT][4] = {};
            for (int s = 0; s < P / 16; ++s) {
                uint32_t fa[4], fl[4], fb[4];
                const uint32_t at = swizzled(mt + row_a, lay.vpitch, s * 2 + col_a);
                ldsm4(fa, base + x + at);
                if (y) ldsm4(fl, base + y + at);
#pragma unroll
                for (int n = 0; n < NT / 2; ++n) {
                    ldsm4_trans(fb, base + st + swizzled(s * 16 + row_kk, lay.kpitch,
                                                         nh * N / 16 + n * 2 + col_kk));
                    mma_16816(acc[2 * n], fa, fb[0], fb[1]);
                    mma_16816(acc[2 * n + 1], fa, fb[2], fb[3]);
                    if (y) {
                        mma_16816(acc[2 * n], fl, fb[0], fb[1]);
                        mma_16816(acc[2 * n + 1], fl, fb[2], fb[3]);
                    }
                }
            }
            const float f0 = sign * f[mt + lane / 4], f1 = sign * f[mt + lane / 4 + 8];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                to[n][0] = fmaf(f0, acc[n][0], to[n][0]);
                to[n][1] = fmaf(f0, acc[n][1], to[n][1]);
                to[n][2] = fmaf(f1, acc[n][2], to[n][2]);
                to[n][3] = fmaf(f1, acc[n][3], to[n][3]);
            }
        };
        with_state(lay.dout, 0, lay.s, eq, 1.f, dq);
        with_state(lay.w, lay.wlo, lay.ds, sw, 1.f, dk);
        with_state(lay.dv, 0, lay.s, ek, -1.f, dk);
        __syncthreads();   // the states' place is the triangles' now

        {   // M1 (warps 0-3) and M2 (warps 4-7): 16 rows, the columns up to the diagonal
            const uint32_t rows = base + (nh ? lay.dv : lay.dout);
            const uint32_t out = nh ? lay.m2 : lay.m1;
            const float *ri = nh ? rks : rqs;
            float acc[8][4] = {};
            for (int s = 0; s < P / 16; ++s) {
                uint32_t fa[4], fb[4];
                ldsm4(fa, rows + swizzled(mt + row_a, lay.vpitch, s * 2 + col_a));
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (n * 16 > mt) break;
                    const uint32_t at = swizzled(n * 16 + row_nn, lay.vpitch, s * 2 + col_nn);
                    ldsm4(fb, base + lay.w + at);
                    mma_16816(acc[2 * n], fa, fb[0], fb[1]);
                    mma_16816(acc[2 * n + 1], fa, fb[2], fb[3]);
                    ldsm4(fb, base + lay.wlo + at);
                    mma_16816(acc[2 * n], fa, fb[0], fb[1]);
                    mma_16816(acc[2 * n + 1], fa, fb[2], fb[3]);
                }
            }
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                if (n * 8 >= mt + 16) break;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int i = mt + lane / 4 + r * 8, j = n * 8 + lane % 4 * 2;
                    const float f = ri[i], ci = cs[i], li = cl[i];
                    const bool on0 = nh ? j < i : j <= i, on1 = nh ? j + 1 < i : j + 1 <= i;
                    const float d0 = (ci - cs[j]) + (li - cl[j]), d1 = (ci - cs[j + 1]) + (li - cl[j + 1]);
                    const float x = on0 ? acc[n][2 * r] * f * __expf(d0) * kb[j] : 0.f;
                    const float y = on1 ? acc[n][2 * r + 1] * f * __expf(d1) * kb[j + 1] : 0.f;
                    const uint32_t at = swizzled(i, lay.mpitch, n) + j % 8 * 2;
                    uint32_t hi, lo;
                    split2(x, y, hi, lo);
                    *reinterpret_cast<uint32_t *>(smem + out + at) = hi;
                    if (!nh) *reinterpret_cast<uint32_t *>(smem + lay.m1lo + at) = lo;
                }
            }
        }
        __syncthreads();

        // products with the triangles; K's and Q's columns as B operands
        auto with_rows = [&](const uint32_t (&fa)[4], uint32_t rows, int s, float (&to)[NT][4]) {
            uint32_t fb[4];
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                ldsm4_trans(fb, base + rows + swizzled(s * 16 + row_kk, lay.kpitch,
                                                       nh * N / 16 + n * 2 + col_kk));
                mma_16816(to[2 * n], fa, fb[0], fb[1]);
                mma_16816(to[2 * n + 1], fa, fb[2], fb[3]);
            }
        };
        for (int s = 0; s < 4; ++s) {
            uint32_t fa[4];
            if (s * 16 <= mt) {   // tokens up to these
                const uint32_t at = swizzled(mt + row_a, lay.mpitch, s * 2 + col_a);
                ldsm4(fa, base + lay.m1 + at);
                with_rows(fa, lay.k, s, dq);
                ldsm4(fa, base + lay.m1lo + at);
                with_rows(fa, lay.k, s, dq);
                ldsm4(fa, base + lay.m2 + at);
#pragma unroll
                for (int r = 0; r < 4; ++r) fa[r] ^= 0x80008000u;
                with_rows(fa, lay.k, s, dk);
            }
            if (s * 16 >= mt) {   // tokens from these on: transposed
                const uint32_t at = swizzled(s * 16 + row_nn, lay.mpitch, mt / 8 + col_nn);
                ldsm4_trans(fa, base + lay.m1 + at);
                with_rows(fa, lay.q, s, dk);
                ldsm4_trans(fa, base + lay.m1lo + at);
                with_rows(fa, lay.q, s, dk);
                ldsm4_trans(fa, base + lay.m2 + at);
#pragma unroll
                for (int r = 0; r < 4; ++r) fa[r] ^= 0x80008000u;
                with_rows(fa, lay.k, s, dk);
            }
        }
    }
    let_next_start();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int t = mt + lane / 4 + r * 8;
            if (t >= len) continue;
            const int64_t at = ((row0 + t) * (a.G * w.runs) + blockIdx.z) * N + nh * (N / 2) +
                               n * 8 + lane % 4 * 2;
            *reinterpret_cast<float2 *>(w.dq_part + at) = make_float2(dq[n][2 * r], dq[n][2 * r + 1]);
            *reinterpret_cast<float2 *>(w.dk_part + at) = make_float2(dk[n][2 * r], dk[n][2 * r + 1]);
        }
}

// A warp per (token, group): sums the runs in order and undoes the norms.
template <int N>
__device__ __forceinline__ void qk_row(const DeltaArgs &a, const DeltaBwd &w, int64_t row)
{
    constexpr int V = N / 32;
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float *part = (which ? w.dk_part : w.dq_part) + row * w.runs * N + lane * V;
        const bf16 *x = static_cast<const bf16 *>(which ? a.k : a.q) + row * N + lane * V;
        bf16 *out = (which ? w.dk : w.dq) + row * N + lane * V;
        float t[V] = {}, y[V];
        for (int r = 0; r < w.runs; ++r)
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] += part[(int64_t)r * N + i];
        if (a.l2norm) {
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] = to_f32(x[i]);
                ss = fmaf(y[i], y[i], ss);
                dot = fmaf(y[i], t[i], dot);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
            }
            const float c = dot / (ss + kL2Eps);
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] = fmaf(-c, y[i], t[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = from_f32<bf16>(t[i]);
    }
}

// A warp per (span, head): dbeta, and dg by a reverse running sum; lane has tokens 2 l, 2 l + 1.
__device__ __forceinline__ void gate_span(const DeltaArgs &a, const DeltaBwd &w, int64_t nchunks,
                                          int64_t item)
{
    const int lane = threadIdx.x % 32;
    const int h = (int)(item % a.H);
    const int64_t span = item / a.H % w.n64, b = item / a.H / w.n64;
    const int tiles = a.P / 16;
    const int64_t c = span * 2 + lane / 16;   // this lane's chunk
    float oo[2] = {}, vv[2] = {}, vw[2] = {}, ss = 0.f;
    if (c < nchunks) {
        const int64_t at = ((b * nchunks + c) * a.H + h) * tiles * kDeltaChunk + lane % 16 * 2;
        for (int i = 0; i < tiles; ++i) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                oo[x] += w.dot_oo[at + i * kDeltaChunk + x];
                vv[x] += w.dot_vv[at + i * kDeltaChunk + x];
                vw[x] += w.dot_vw[at + i * kDeltaChunk + x];
            }
        }
    }
    const float *at_begin = w.dot_ss + ((b * (w.n64 + 1) + span) * a.H + h) * tiles;
    const float *at_end = at_begin + (int64_t)a.H * tiles;
    float begin = 0.f;
    for (int i = 0; i < tiles; ++i) {
        begin += at_begin[i];
        ss += at_end[i];
    }
    const float d1 = oo[1] - vv[1], d0 = oo[0] - vv[0];
    float sum = d0 + d1, before = d0 + d1;   // of this lane's tokens and all behind, or before, them
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float dn = __shfl_down_sync(0xffffffffu, sum, o);
        const float up = __shfl_up_sync(0xffffffffu, before, o);
        if (lane + o < 32) sum += dn;
        if (lane >= o) before += up;
    }
    const float left = a.L - span * kSpan < kSpan ? (float)(a.L - span * kSpan) : (float)kSpan;
    float behind = __shfl_down_sync(0xffffffffu, sum, 1);   // from token 2 l + 2 on
    before = __shfl_up_sync(0xffffffffu, before, 1);        // up to token 2 l - 1
    if (lane == 31) behind = 0.f;
    if (lane == 0) before = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int64_t t = span * kSpan + lane * 2 + x;
        if (t >= a.L) continue;
        const int64_t at = (b * a.L + t) * a.H + h;
        float beta = a.beta[at];
        if (fabsf(beta) < 1e-20f) beta = 1e-20f;   // as the chains took it
        w.dbeta[at] = vw[x] / beta;
        const float from_end = ss + (behind + (x == 0 ? d0 + d1 : d1));
        const float from_begin = begin - (x == 0 ? before : before + d0);
        const float f = (float)(lane * 2 + x) / left;
        if (w.dg) w.dg[at] = fmaf(f, from_end - from_begin, from_begin);
    }
}

// The last kernel: a warp per item, (b, t, g) rows of dq and dk first, then (b, span, h).
template <int N>
__global__ void __launch_bounds__(256)
delta_finish_kernel(const DeltaArgs a, const DeltaBwd w, int64_t nchunks, int64_t rows, int64_t spans)
{
    wait_before();
    const int64_t item = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (item < rows) qk_row<N>(a, w, item);
    else if (item < rows + spans) gate_span(a, w, nchunks, item - rows);
}

}  // namespace

cudaError_t launch_delta_grads(const DeltaArgs &a, const DeltaBwd &w, int64_t nchunks,
                               cudaStream_t st)
{
    const int smem = GradSmem(a.P, a.N).total;
    const dim3 grid((unsigned)w.n64, (unsigned)a.batch, (unsigned)(a.G * w.runs));
    cudaError_t e =
        launch_after(a.N == 128 ? delta_grad_kernel<128> : delta_grad_kernel<64>, grid, kGradThreads,
                     smem, st, a, w);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.batch * a.L * a.G, spans = a.batch * w.n64 * a.H;
    return launch_after(a.N == 128 ? delta_finish_kernel<128> : delta_finish_kernel<64>,
                        (unsigned)((rows + spans + 7) / 8), 256, 0, st, a, w, nchunks, rows, spans);
}

}  // namespace ssd
