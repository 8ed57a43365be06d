// vp_linear_ce.cu -- softmax cross entropy of hidden . W^T without keeping the logits,
// forward and backward on tcgen05 tensor cores (formulas: vp_ce.cuh; the GEMMs, their
// order and their bounds: vp_gemm.cuh).
//
// Forward: tiles of 256 rows x 256 vocabulary rows; eight epilogue warps read a tile from TMEM, cap its
//   logits, and leave for each row and 128 columns (max, sum of exponentials, sum of logits) and the
//   target's logit; ce_join_kernel makes them the row's loss. 2 N V D flops.
// Backward, a piece of the vocabulary at a time: the piece's logits again, dz in the epilogue (through
//   the cap's slope) as one or two bf16 values, then dhidden += dz . W_c and dW_c = dz^T . h. 6 N V D
//   flops, 10 with dz as a pair everywhere, 6.5 to 6.9 with a pair where it counts (the default).
// Bound: the tensor cores, and the power they draw. 8192 x 75968 x 4096: forward 2.5 ms after
//   a pause (1.9 PFLOP/s); back to back, under the power cap, backward 9.9 to 10.2 and both 13.3 ms (1.62 PFLOP/s). Few rows: the bytes of W, read three times, and dW written (16 rows: 102, 107, 99 and 96 us, 92
//   each at the copy rate). Short K (D of 512 and less): the epilogues' instructions.
#include "vp_ce.cuh"
#include "vp_gemm.cuh"
#include "vp_stats.cuh"

namespace vp {

// A tensor-core step adds 16 products to the running fp32 sum and cuts off what lies below its last
// bit, towards zero, so a logit comes out short: over sums of independent terms by 2^-26 of itself a
// step on average (measured on GB300 as the slope of 98304 logits' errors: 0.86, 0.90, 0.96, 1.01, 1.03 and
// 1.06 times 2^-26 a step at D = 512, 1024, .., 16384, the same to 1 % at variances of 1, 6.25, 25 and 100).
// The epilogues give that mean back, for 16384 columns at most. It is a mean and no more: terms of one
// sign lose 1.9 to 5.4 times as much, and a sum that nothing is cut off of (one product, say) comes out long by what is
// given back, 2^-18 of itself at D = 4096 and 2^-16 at most. Either is within the bound of the steps themselves,
// 2^-23 of the running sum each.
constexpr int64_t kCutOffMostD = 16384;
static float cut_off(int64_t D) { return 1.f + (float)(std::min(D, kCutOffMostD) / 16) * 1.490116119384765625e-08f; }
__device__ __forceinline__ void scale_all(float (&v)[32], float s) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float2 p = __fmul2_rn(make_float2(v[i], v[i + 1]), f2(s));
        v[i] = p.x;
        v[i + 1] = p.y;
    }
}

template <bool kCap>
struct CeEpi {
    static constexpr bool kPdl = true, kWide = true;
    int N, n_t;
    float scale;        // cut_off(D)
    bool sum;           // the sum of the logits, which only label smoothing asks for
    int64_t vocab_start;
    const int64_t *targets;
    CeRules q;
    float4 *tiles;      // [N][n_t]
    float *tgt;         // [N]
    __device__ __forceinline__ void operator()(int row, int col0, int ncol, uint32_t taddr) const {
        const bool valid = row < N;
        const int64_t tg = valid ? targets[row] : -1;
        const int64_t t = tg - vocab_start - col0;
        const int tloc = (tg >= 0 && t >= 0 && t < ncol) ? (int)t : -1;
        float m = kNegBig, S = 0.f, zt = 0.f;
        float2 Z = f2(0.f);                              // times 2^-33 (kCeScale)
#pragma unroll 1
        for (int c = 0; c < kWideEpiCols / 32; ++c) {
            float v[32];
            tmem_ld32(taddr + c * 32, v);
            const int n = ncol - c * 32;                 // columns of the vocabulary left
            if (n <= 0) continue;
            scale_all(v, scale);
            if (kCap) soft_cap(q, v);
            if ((uint32_t)(tloc - c * 32) < 32u) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (c * 32 + i == tloc) zt = v[i];
            }
            if (n < 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    Z.x += i < n ? v[i] * kCeScale : 0.f;
                    if (i >= n) v[i] = -INFINITY;
                }
            } else if (sum) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) Z = __ffma2_rn(make_float2(v[i], v[i + 1]), f2(kCeScale), Z);
            }
            float cm = m;
#pragma unroll
            for (int i = 0; i < 32; ++i) cm = fmaxf(cm, v[i]);
            if (cm > m) {
                S *= ex2_approx((m - cm) * kLog2e);
                m = cm;
            }
            float2 s2 = f2(0.f);
            const ExpCentre k = exp_centre(m);
#pragma unroll
            for (int i = 0; i < 32; i += 2) s2 = __fadd2_rn(s2, ce_exp2(k, make_float2(v[i], v[i + 1])));
            S = fmaf(s2.x + s2.y, k.f, S);
        }
        if (!valid) return;
        tiles[(int64_t)row * n_t + col0 / kCeTileCols] = make_float4(m, S, Z.x + Z.y, 0.f);
        if (tloc >= 0) tgt[row] = zt;
    }
};

// A warp's 32 rows of kVecs 16-byte vectors, row i in lane i, turned in shared memory so that kVecs lanes have a
// row's vectors behind one another: use(row, vector, value). Straight from the lanes every store would touch half a
// sector of each of 32 rows (dW of 75968 x 4096 from 16 tokens took 256 us so, 150 by whole lines; its bytes are 92). The
// vectors' places are swapped by row so that neither side meets a bank twice.
constexpr int kStageVecs = 32 * 8;                       // of each epilogue warp: 4 KB
template <int kVecs, class Use>
__device__ __forceinline__ void turn_rows(uint4 *stage, const uint4 (&v)[kVecs], Use use) {
    static_assert(kVecs == 4 || kVecs == 8, "64 or 128 bytes of a row");
    const int lane = threadIdx.x & 31;
    auto at = [](int r, int j) { return r * kVecs + (j ^ (kVecs == 8 ? r & 7 : (r >> 1) & 3)); };
    __syncwarp();                                        // the last rows have been read
#pragma unroll
    for (int j = 0; j < kVecs; ++j) stage[at(lane, j)] = v[j];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int r = (32 / kVecs) * i + lane / kVecs, j = lane % kVecs;
        use(r, j, stage[at(r, j)]);
    }
}
// .. and to the rows `first` .. of a bf16 matrix
template <int kVecs>
__device__ __forceinline__ void store_rows(uint4 *stage, const uint4 (&v)[kVecs], __nv_bfloat16 *dst, int64_t ld, int first,
                                           int M) {
    turn_rows(stage, v, [&](int r, int j, const uint4 &x) {
        if (first + r < M) stg_stream(dst + r * ld + 8 * j, x);
    });
}

// Which values of dz the mixed precision carries as a pair. One bf16 value is off by up to 2^-8 of
// itself, so what the values up to a threshold of a row add to the error of dhidden is 2^-8 sqrt(sum of
// their squares) |W|, and with a threshold of t times the row's own scale s (for a cross entropy the values
// add up to about 2 s, s = |g| (1 - p_t), through the cap's slope at the target) that is below
// 2^-8 sqrt(2 t) s |W|: for t = 1/16 about a third of what the output's own rounding adds. The values of a
// row whose first half is larger, its target's first of all, are pairs. Which 32 x 64 pieces of dz hold one is noted, and the
// gradient GEMMs take the second halves of no other k-blocks. A z-loss multiplies every softmax, and the scale,
// by 1 + 2 zeta lse; beyond 4 the threshold grows with it, so that no row has pairs by the hundred.
constexpr float kPairShare = 1.f / 16.f;
constexpr int kFlagRows = 32, kFlagCols = 64;

// dz of 128 columns of a tile of the piece that starts at shard column v0, as bf16 (and, with
// lo_off != 0, what that rounding took away as a second one).
template <bool kCap>
struct DzCeEpi {
    static constexpr bool kPdl = true, kWide = true;
    int N, V, v0, ldz;
    float scale;        // cut_off(D)
    int64_t vocab_start;
    const int64_t *targets;
    CeRules q;
    const RowStat *stats;
    const float *g;
    __nv_bfloat16 *dz;
    int32_t *err;
    int64_t lo_off;
    uint8_t *flags;     // [N / 32][ldz / 64], or NULL: no notes
    float *limits;      // [N]: from where on a row's values are pairs; or NULL
    __device__ __forceinline__ void operator()(int row, int col0, int ncol, uint32_t taddr) const {
        const bool valid = row < N;
        const RowStat s = load_rowstat(stats + (valid ? row : 0));
        const int64_t tg = valid ? targets[row] : -1;
        const int64_t tl = tg - vocab_start;                // target column in the shard
        const bool outside = tg >= 0 && (tl < 0 || tl >= V) && !(s.flags & kRowSharded);
        int mode = (s.flags & (kRowNanInf | kRowEmpty | kRowBadTarget)) || outside ? 2 : 0;   // 1 zeros, 2 NaN
        if (tg < 0) mode = 1;
        if (valid && outside && err && col0 == 0 && v0 == 0) atomicOr(err, VP_ERRBIT_TARGET_);
        const int64_t tcol = tg >= 0 ? tl - v0 - col0 : -1;   // target column within this tile
        const CeGradRow gr = ce_grad_row<true>(q, s, valid ? g[row] : 0.f);
        // the record's c is log p of the target
        float limit = kPairShare * fabsf(gr.g) * fmaxf(q.smooth - expm1f(s.c_hi), 9.5367431640625e-07f) *
                      fmaxf(1.f, 0.25f * fabsf(1.f + gr.a1));
        if (kCap) {
            const float zt = (s.m + s.logS_hi + s.c_hi) * q.inv_cap;
            limit *= fmaxf(fmaf(-zt, zt, 1.f), 9.5367431640625e-07f);
        }
        if (limits && valid && col0 == 0) limits[row] = limit;
        __shared__ uint4 stage[kWideEpiWarps][kStageVecs];
        uint4 *mine = stage[(threadIdx.x >> 5) - 2];
        const int first = row - (threadIdx.x & 31);           // the warp's first row
        float most = 0.f;                                     // of the row's 64 columns
#pragma unroll 1
        for (int c = 0; c < kWideEpiCols; c += 32) {
            float v[32], slope[32];
            tmem_ld32(taddr + c, v);
            scale_all(v, scale);
            if (kCap) soft_cap<32, true>(q, v, slope);
            const uint32_t at = tcol >= 0 && tcol < kWideEpiCols ? (uint32_t)((int)tcol - c) : 32u;
            float dt = 0.f;                                   // the target's column
            if (at < 32u) {
                float zt = 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i == (int)at) zt = v[i];
                dt = ce_grad_target(q, gr, zt);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 d = ce_grad2(gr, make_float2(v[i], v[i + 1]));
                v[i] = d.x;
                v[i + 1] = d.y;
            }
            if (at < 32u) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i == (int)at) v[i] = dt;
            }
            if (kCap) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 d = __fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(slope[i], slope[i + 1]));
                    v[i] = d.x;
                    v[i + 1] = d.y;
                }
            }
            if (mode || c + 32 > ncol) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = mode == 1 || c + i >= ncol ? 0.f : mode == 2 ? qnan() : v[i];
            }
            uint4 hi[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) hi[k] = Elem<__nv_bfloat16>::pack(v + 8 * k);
            __nv_bfloat16 *dst = dz + (int64_t)first * ldz + col0 + c;
            store_rows(mine, hi, dst, ldz, first, N);
            if (lo_off) {
                uint4 lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float h[8];                               // what the rounding took away is exact in fp32
                    Elem<__nv_bfloat16>::unpack(hi[k], h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        most = fmaxf(most, fabsf(h[i]));  // as pair_add_kernel sees them
                        h[i] = v[8 * k + i] - h[i];
                    }
                    lo[k] = Elem<__nv_bfloat16>::pack(h);
                }
                store_rows(mine, lo, dst + lo_off, ldz, first, N);
            }
            if (flags && c % 64) {
                const bool pair = __any_sync(0xffffffffu, valid && most > limit);
                if ((row & 31) == 0 && valid)
                    flags[(int64_t)(row / kFlagRows) * (ldz / kFlagCols) + (col0 + c) / kFlagCols] = pair;
                most = 0.f;
            }
        }
    }
};

// The logits of hidden rows [N, D] and rows of W [nv, D], on CTA pairs.
template <class Epi>
static cudaError_t ce_logits_gemm(const void *h, const void *w, int N, int nv, int D, const Epi &epi, cudaStream_t stream) {
    CUtensorMap ta, tb;
    if (!make_map(&ta, h, N, D, D, kLBM) || !make_map(&tb, w, nv, D, D, kPBHalf)) return cudaErrorInvalidValue;
    return launch_gemm_pair<Epi>(ta, tb, N, nv, D, epi, stream, 0, kHintLogits);
}

struct CeFwdLayout {
    size_t tiles, tgt, total;
};
static CeFwdLayout ce_fwd_layout(int64_t N, int64_t V) {
    CeFwdLayout L;
    L.tiles = 0;
    L.tgt = up256((size_t)N * ((V + kCeTileCols - 1) / kCeTileCols) * sizeof(float4));
    L.total = L.tgt + up256((size_t)N * sizeof(float));
    return L;
}
size_t linear_ce_workspace_bytes(int64_t N, int64_t V) { return ce_fwd_layout(N, V).total; }

cudaError_t launch_linear_ce_fwd(const CeArgs &a) {
    const CeFwdLayout L = ce_fwd_layout(a.N, a.V);
    const int n_t = (int)((a.V + kCeTileCols - 1) / kCeTileCols);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    float4 *tiles = reinterpret_cast<float4 *>(ws + L.tiles);
    float *tgt = reinterpret_cast<float *>(ws + L.tgt);
    const CeRules q = ce_rules(a.opt);
    auto gemm = [&](const auto &epi) {
        return ce_logits_gemm(a.hidden, a.weight, (int)a.N, (int)a.V, (int)a.D, epi, a.stream);
    };
    const cudaError_t e = q.cap > 0.f
                              ? gemm(CeEpi<true>{(int)a.N, n_t, cut_off(a.D), a.parts || q.smooth > 0.f, a.vocab_start, a.targets, q, tiles, tgt})
                              : gemm(CeEpi<false>{(int)a.N, n_t, cut_off(a.D), a.parts || q.smooth > 0.f, a.vocab_start, a.targets, q, tiles, tgt});
    if (e != cudaSuccess) return e;
    return launch_ce_join(CeTiles{tiles, tgt, n_t, (int)a.V}, n_t, a);
}

// From the notes, the k-blocks whose second halves the gradient GEMMs take: for each 256 rows of dz the
// 64-column blocks (dhidden), and for each 256 columns the 64-row blocks (dW), in order. One CTA for a list.
__global__ void __launch_bounds__(256)
pair_list_kernel(const uint8_t *__restrict__ flags, int row_groups, int pitch, int col_groups, int n_rows, int *__restrict__ count,
                 int *__restrict__ list, int pitch_rows, int pitch_cols) {
    __shared__ uint32_t s_n[8];
    pdl_enter<true>();   // no global access before this
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool by_rows = (int)blockIdx.x < n_rows;
    const int b = by_rows ? blockIdx.x : blockIdx.x - n_rows;
    const int n = by_rows ? col_groups : (row_groups + 1) / 2;
    int *out = list + (by_rows ? (int64_t)b * pitch_rows : (int64_t)n_rows * pitch_rows + (int64_t)b * pitch_cols);
    uint32_t done = 0;
    for (int k0 = 0; k0 < n; k0 += 256) {
        const int k = k0 + tid;
        bool any = false;
        if (k < n) {
            // 8 groups of rows and one of columns, or 2 and 4 (one word: the pitch is a multiple of 4; the last may
            // hold groups behind the vocabulary, which nothing has written)
            const int r0 = by_rows ? 8 * b : 2 * k;
            const int in_word = col_groups - 4 * b;
            const uint32_t mask = by_rows || in_word >= 4 ? 0xffffffffu : (1u << (8 * in_word)) - 1u;
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (r0 + i >= row_groups || (!by_rows && i >= 2)) continue;
                const uint8_t *f = flags + (int64_t)(r0 + i) * pitch;
                seen |= by_rows ? f[k] : *reinterpret_cast<const uint32_t *>(f + 4 * b);
            }
            any = (seen & mask) != 0;
        }
        const uint32_t votes = __ballot_sync(0xffffffffu, any);
        if (lane == 0) s_n[warp] = __popc(votes);
        __syncthreads();
        uint32_t before = done;
        for (int w = 0; w < 8; ++w) {
            if (w < warp) before += s_n[w];
            done += s_n[w];
        }
        if (any) out[before + __popc(votes & ((1u << lane) - 1u))] = k;
        __syncthreads();
    }
    if (tid == 0) count[blockIdx.x] = (int)done;
}

// dhidden's share of the second halves, without a GEMM: a row's values above its limit are few (those of a cross entropy
// add up to about twice its scale, so some 32 at most, 64 with a large z-loss, and one or two as a rule), so their second halves times their rows of W are
// added to the row's sum as they are. A CTA for a row and 2048 columns: it goes through the row's noted blocks, 32 at a time,
// in order, so a row's sum does not depend on the rows beside it.
constexpr int kAddThreads = 256, kAddBlocks = 32;
__global__ void __launch_bounds__(kAddThreads)
pair_add_kernel(const __nv_bfloat16 *__restrict__ dz, int64_t lo_off, int ldz, const uint8_t *__restrict__ flags, int pitch,
                int col_groups, const float *__restrict__ limits, const __nv_bfloat16 *__restrict__ W, int D,
                float *__restrict__ acc) {
    __shared__ int s_block[kAddThreads];
    __shared__ uint32_t s_n[kAddThreads / 32];
    __shared__ uint2 s_mask[kAddBlocks];
    __shared__ float s_lo[kAddBlocks][kFlagCols];
    pdl_enter<true>();   // no global access before this
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x;
    const int d = (blockIdx.y * kAddThreads + tid) * 8;
    const float limit = limits[row];
    const uint8_t *f = flags + row / kFlagRows * pitch;
    const __nv_bfloat16 *hi = dz + row * ldz;
    float sum[8] = {};
    bool some = false;                                   // the same for the CTA
    for (int g0 = 0; g0 < col_groups; g0 += kAddThreads) {
        const bool noted = g0 + tid < col_groups && f[g0 + tid];
        const uint32_t votes = __ballot_sync(0xffffffffu, noted);
        if (lane == 0) s_n[warp] = __popc(votes);
        __syncthreads();
        int before = __popc(votes & ((1u << lane) - 1u)), n = 0;
        for (int w = 0; w < kAddThreads / 32; ++w) {
            if (w < warp) before += s_n[w];
            n += s_n[w];
        }
        if (noted) s_block[before] = g0 + tid;
        __syncthreads();
        for (int b0 = 0; b0 < n; b0 += kAddBlocks) {
            const int nb = min(kAddBlocks, n - b0);
            for (int b = warp; b < nb; b += kAddThreads / 32) {
                const int64_t at = (int64_t)s_block[b0 + b] * kFlagCols + 2 * lane;
                const uint32_t h = __ldg(reinterpret_cast<const uint32_t *>(hi + at)), l = __ldg(reinterpret_cast<const uint32_t *>(hi + lo_off + at));
                float x, y;
                Elem<__nv_bfloat16>::unpack2(h, x, y);
                const uint32_t even = __ballot_sync(0xffffffffu, fabsf(x) > limit), odd = __ballot_sync(0xffffffffu, fabsf(y) > limit);
                if (lane == 0) s_mask[b] = make_uint2(even, odd);
                Elem<__nv_bfloat16>::unpack2(l, s_lo[b][2 * lane], s_lo[b][2 * lane + 1]);
            }
            __syncthreads();
            for (int b = 0; b < nb; ++b) {
                const uint2 mask = s_mask[b];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    for (uint32_t m = half ? mask.y : mask.x; m; m &= m - 1) {
                        const int e = 2 * (__ffs(m) - 1) + half;
                        some = true;
                        if (d >= D) continue;
                        float w[8];
                        Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4 *>(W + ((int64_t)s_block[b0 + b] * kFlagCols + e) * D + d)), w);
#pragma unroll
                        for (int k = 0; k < 8; ++k) sum[k] = fmaf(s_lo[b][e], w[k], sum[k]);
                    }
                }
            }
            __syncthreads();
        }
    }
    if (!some || d >= D) return;
    float4 *p = reinterpret_cast<float4 *>(acc + row * D + d);
    float4 a = p[0], b = p[1];
    a.x += sum[0]; a.y += sum[1]; a.z += sum[2]; a.w += sum[3];
    b.x += sum[4]; b.y += sum[5]; b.z += sum[6]; b.w += sum[7];
    p[0] = a;
    p[1] = b;
}

// dhidden's tiles: the sum over a share of the k-blocks, kept apart for each share; ld is a multiple of 64.
struct SplitAccEpi {
    static constexpr bool kPdl = true, kWide = true;
    int M, ld;
    bool first;
    float *acc;          // [splits][M][ld]
    __device__ __forceinline__ void operator()(int row, int col0, int ncol, uint32_t taddr, int split) const {
        __shared__ uint4 stage[kWideEpiWarps][kStageVecs];
        uint4 *mine = stage[(threadIdx.x >> 5) - 2];
        const int top = row - (int)(threadIdx.x & 31);
#pragma unroll 1
        for (int c = 0; c < ncol; c += 32) {
            float v[32];
            tmem_ld32(taddr + c, v);
            uint4 u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = Elem<float>::pack(v + 4 * j);
            float *dst = acc + ((int64_t)split * M + top) * ld + col0 + c;
            turn_rows(mine, u, [&](int r, int j, const uint4 &x) {
                if (top + r >= M) return;
                uint4 *p = reinterpret_cast<uint4 *>(dst + (int64_t)r * ld + 4 * j);
                float f[4], o[4];
                Elem<float>::unpack(x, f);
                if (!first) {
                    Elem<float>::unpack(*p, o);
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[k] += o[k];
                }
                *p = Elem<float>::pack(f);
            });
        }
    }
};

// dW's tiles, rounded; ld is a multiple of 64.
struct StoreRowsEpi {
    static constexpr bool kPdl = true, kWide = true;
    int M, ld;
    int64_t row0;
    __nv_bfloat16 *out;
    __device__ __forceinline__ void operator()(int row, int col0, int ncol, uint32_t taddr, int) const {
        __shared__ uint4 stage[kWideEpiWarps][kStageVecs];
        uint4 *mine = stage[(threadIdx.x >> 5) - 2];
        const int first = row - (threadIdx.x & 31);
        // a chunk's columns come out of TMEM while the one before is stored
        uint32_t f[2][32];
        tmem_ld32_issue(taddr, f[0]);
        tmem_ld32_issue(taddr + 32, f[1]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kWideEpiCols; c += 64) {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = Elem<__nv_bfloat16>::pack(reinterpret_cast<const float *>(f[k / 4]) + 8 * (k % 4));
            if (c + 64 < kWideEpiCols) {
                tmem_ld32_issue(taddr + c + 64, f[0]);
                tmem_ld32_issue(taddr + c + 96, f[1]);
            }
            if (c < ncol) store_rows(mine, v, out + (row0 + first) * (int64_t)ld + col0 + c, ld, first, M);
            if (c + 64 < kWideEpiCols) tmem_wait_ld();
        }
    }
};

// The shares' sums, added in order and rounded once.
__global__ void __launch_bounds__(256)
split_sum_kernel(const float *__restrict__ acc, int64_t n, int splits, __nv_bfloat16 *__restrict__ out) {
    pdl_enter<true>();   // no global access before this
    const int64_t i = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);   // n is a multiple of 64
    if (i >= n) return;
    float v[8] = {};
    for (int s = 0; s < splits; ++s) {
        const float4 a = *reinterpret_cast<const float4 *>(acc + s * n + i), b = *reinterpret_cast<const float4 *>(acc + s * n + i + 4);
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    *reinterpret_cast<uint4 *>(out + i) = Elem<__nv_bfloat16>::pack(v);
}

// Columns of the vocabulary a piece: dz twice over near 1 GB, so that few rows take the whole vocabulary at
// once; 8192 at least.
static int64_t ce_piece(int64_t N, int64_t V) {
    const int64_t fit = ((int64_t)1 << 28) / N / 256 * 256, all = (V + 255) / 256 * 256;
    return std::min(all, std::clamp<int64_t>(fit, 8192, 1 << 22));
}

// Shares of dhidden's k-blocks: its output tiles are few where N and D are, and the GPU's pairs of SMs then
// stand still (1000 x 75968 x 2048, dz as a pair: 690 us with whole sums on 32 of 76 pairs, 340 with seven shares). The waves of tiles that a split makes, counted in whole tiles, with 1 % of them for
// each share's sums, which are written and read once more.
// dW's tiles are few where V and D are (backward of 4392 x 1597 x 256: 84 us with
// dW on 7 of 76 pairs, 50 with shares; 65536 x 256 x 1024: 883 and 261).
static int ce_splits(int64_t rows, int64_t K, int64_t D, int pairs) {
    const int64_t tiles = ((rows + 255) / 256) * ((D + 255) / 256);
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= 16 && s <= K / 512; ++s) {
        const double cost = (double)((tiles * s + pairs - 1) / pairs) / s + 0.01 * s;
        if (cost < least) least = cost, best = s;
    }
    return best;
}

// Whether dhidden's second halves are added by pair_add_kernel, about 15 ns a row, and not by the GEMM, 2 V D flops a row
// in those k-blocks that any of 256 rows notes (a quarter of 75968 columns, half of 20000). Backward, in us, so and
// otherwise: 8192 x 75968 x 4096 10210 and 10680, 2048 x 32000 x 2048 645 and 708, 8192 x 20000 x 1024 1021 and 1028; but
// 6427 x 4122 x 832 281 and 256, 256 x 32000 x 1024 102 and 97. Under a cap a row's values are not bounded by its scale: there the GEMM adds them.
static bool ce_apart(int64_t N, int64_t V, int64_t D, double cap) { return cap <= 0.0 && N >= 1024 && V * D >= 1 << 25; }

// Whether the mixed precision looks for the blocks that count: finding them is a launch, which costs more than all
// second halves where the table and the products are small (backward, in us, without and with: 64 x 5003 x 512 30 and 32,
// 2000 x 2000 x 256 41 and 44; but 64 x 16000 x 512 45 and 42, 16 x 16000 x 512 44 and 38, where they read the table once more).
static bool ce_lists(int64_t N, int64_t V, int64_t D) { return V * D > 1 << 22 || N * V * D > 1 << 30; }

struct CeBwdLayout {
    size_t dz, acc, acc_w, flags, limits, count, list, total;
    int64_t vc;
    int splits, splits_w, row_groups, col_groups, n_rows, n_cols, pitch_rows, pitch_cols;
};
static CeBwdLayout ce_bwd_layout(int64_t N, int64_t V, int64_t D, int pairs) {
    CeBwdLayout L;
    L.vc = ce_piece(N, V);
    L.splits = ce_splits(N, L.vc, D, pairs);
    // shares of dW only where its sums are small beside what they add up, and V is one piece
    L.splits_w = L.vc >= V && 2 * ((V + 255) / 256) * ((D + 255) / 256) <= pairs ? ce_splits(V, N, D, pairs) : 1;
    L.row_groups = (int)((N + kFlagRows - 1) / kFlagRows);
    L.col_groups = (int)(L.vc / kFlagCols);
    L.n_rows = (int)((N + 255) / 256);
    L.n_cols = (int)(L.vc / 256);
    L.pitch_rows = L.col_groups;
    L.pitch_cols = (L.row_groups + 1) / 2;
    L.dz = 0;
    L.acc = up256((size_t)2 * N * L.vc * 2);
    L.acc_w = L.acc + up256((size_t)L.splits * N * D * 4);
    L.flags = L.acc_w + (L.splits_w > 1 ? up256((size_t)L.splits_w * V * D * 4) : 0);
    L.limits = L.flags + up256((size_t)L.row_groups * L.col_groups);
    L.count = L.limits + up256((size_t)N * 4);
    L.list = L.count + up256((size_t)(L.n_rows + L.n_cols) * 4);
    L.total = L.list + up256(((size_t)L.n_rows * L.pitch_rows + (size_t)L.n_cols * L.pitch_cols) * 4);
    return L;
}
static int sm_pairs() {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return std::max(1, sms / 2);
}
size_t linear_ce_bwd_workspace_bytes(int64_t N, int64_t V, int64_t D) {
    return N ? ce_bwd_layout(N, V, D, sm_pairs()).total : 0;
}

cudaError_t launch_linear_ce_bwd(const CeArgs &a) {
    const CeBwdLayout L = ce_bwd_layout(a.N, a.V, a.D, sm_pairs());
    const int64_t vc = L.vc;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    __nv_bfloat16 *dz = reinterpret_cast<__nv_bfloat16 *>(ws + L.dz);
    const bool chain = a.precision != VP_GRAD_FAST_, mixed = a.precision == VP_GRAD_MIXED_ && ce_lists(a.N, a.V, a.D);
    const __nv_bfloat16 *dz_lo = dz + a.N * vc;            // behind dz_hi
    float *acc = reinterpret_cast<float *>(ws + L.acc);
    uint8_t *flags = mixed ? ws + L.flags : nullptr;
    const bool apart = mixed && a.dhidden && ce_apart(a.N, a.V, a.D, a.opt.cap);
    float *limits = apart ? reinterpret_cast<float *>(ws + L.limits) : nullptr;
    int *count = reinterpret_cast<int *>(ws + L.count), *list = reinterpret_cast<int *>(ws + L.list);
    const SplitK of_rows{L.splits, mixed ? count : nullptr, list, L.pitch_rows};
    const SplitK of_cols{L.splits_w, mixed ? count + L.n_rows : nullptr, list + (int64_t)L.n_rows * L.pitch_rows, L.pitch_cols};
    const __nv_bfloat16 *h = static_cast<const __nv_bfloat16 *>(a.hidden);
    const __nv_bfloat16 *W = static_cast<const __nv_bfloat16 *>(a.weight);
    const RowStat *stats = static_cast<const RowStat *>(a.stats);
    const int N = (int)a.N, V = (int)a.V, D = (int)a.D;
    const CeRules q = ce_rules(a.opt);
    cudaError_t e;
    CUtensorMap tm_h;
    if (!make_map_mn(&tm_h, h, N, D, D)) return cudaErrorInvalidValue;
    for (int64_t v0 = 0; v0 < V; v0 += vc) {
        const int nv = (int)(V - v0 < vc ? V - v0 : vc);
        auto gemm = [&](const auto &epi) {
            return ce_logits_gemm(h, W + v0 * D, N, nv, D, epi, a.stream);
        };
        const int64_t lo_off = chain ? a.N * vc : 0;
        e = q.cap > 0.f ? gemm(DzCeEpi<true>{N, V, (int)v0, (int)vc, cut_off(D), a.vocab_start, a.targets, q, stats, a.g, dz, a.err, lo_off, flags, limits})
                        : gemm(DzCeEpi<false>{N, V, (int)v0, (int)vc, cut_off(D), a.vocab_start, a.targets, q, stats, a.g, dz, a.err, lo_off, flags, limits});
        if (e != cudaSuccess) return e;
        if (mixed) {
            const int cols = (nv + 63) / 64, tiles = (nv + 255) / 256;
            e = launch_pdl(pair_list_kernel, dim3(L.n_rows + tiles), dim3(256), 0, a.stream, flags, L.row_groups, L.col_groups,
                           cols, L.n_rows, count, list, L.pitch_rows, L.pitch_cols);
            if (e != cudaSuccess) return e;
        }
        auto product = [&](auto kinds, bool chain, const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &ta2, int M, int Nn,
                           int K, const auto &epi, int group, const SplitK &ks) {
            using Epi = std::decay_t<decltype(epi)>;
            constexpr bool kAMn = decltype(kinds)::value;
            return chain ? launch_gemm_pair_impl<Epi, kAMn, true, false, true>(ta, tb, ta2, tb, M, Nn, K, K, epi, a.stream,
                                                                              (group + 1) / 2, kHintK2, ks)
                         : launch_gemm_pair_impl<Epi, kAMn, true, false, false>(ta, tb, ta, tb, M, Nn, K, 0, epi, a.stream,
                                                                               (group + 1) / 2, kHintK2, ks);
        };
        if (a.dhidden) {
            CUtensorMap ta, ta2, tb;
            if (!make_map(&ta, dz, N, nv, vc, kLBM) || !make_map(&ta2, dz_lo, N, nv, vc, kLBM) ||
                !make_map_mn(&tb, W + v0 * D, nv, D, D))
                return cudaErrorInvalidValue;
            // a short last piece has fewer k-blocks than there are shares; their sums stay as they are
            SplitK ks = of_rows;
            ks.splits = std::min(ks.splits, (nv + kLBK - 1) / kLBK);
            e = product(std::false_type(), chain && !apart, ta, tb, ta2, N, D, nv, SplitAccEpi{N, D, v0 == 0, acc}, kGradGroupM, ks);
            if (e != cudaSuccess) return e;
            if (apart) {
                e = launch_pdl(pair_add_kernel, dim3((unsigned)N, (unsigned)((D + 8 * kAddThreads - 1) / (8 * kAddThreads))),
                               dim3(kAddThreads), 0, a.stream, dz, lo_off, (int)vc, flags, L.col_groups, (nv + kFlagCols - 1) / kFlagCols,
                               limits, W + v0 * D, D, acc);
                if (e != cudaSuccess) return e;
            }
        }
        if (a.dW) {
            CUtensorMap ta, ta2;
            if (!make_map_mn(&ta, dz, N, nv, vc) || !make_map_mn(&ta2, dz_lo, N, nv, vc)) return cudaErrorInvalidValue;
            if (L.splits_w > 1)
                e = product(std::true_type(), chain, ta, tm_h, ta2, nv, D, N, SplitAccEpi{nv, D, true, reinterpret_cast<float *>(ws + L.acc_w)},
                            kWGroupM, of_cols);
            else
                e = product(std::true_type(), chain, ta, tm_h, ta2, nv, D, N,
                            StoreRowsEpi{nv, D, v0, static_cast<__nv_bfloat16 *>(a.dW)}, kWGroupM, of_cols);
            if (e != cudaSuccess) return e;
        }
    }
    auto sum = [&](size_t shares, int64_t n, int splits, void *out) {
        return launch_pdl(split_sum_kernel, dim3((unsigned)((n / 8 + 255) / 256)), dim3(256), 0, a.stream,
                          reinterpret_cast<const float *>(ws + shares), n, splits, static_cast<__nv_bfloat16 *>(out));
    };
    if (a.dW && L.splits_w > 1 && (e = sum(L.acc_w, a.V * a.D, L.splits_w, a.dW)) != cudaSuccess) return e;
    return a.dhidden ? sum(L.acc, a.N * a.D, L.splits, a.dhidden) : cudaSuccess;
}

cudaError_t read_linear_ce_fault(uint32_t *value, bool clear) { return read_tu_fault(value, clear); }

}  // namespace vp
