// vp_ce.cuh -- softmax cross entropy with label smoothing, z-loss and soft-capped
// logits: the formulas, and the join of a row's pieces, shared by the forms on
// logits (vp_ce.cu) and on hidden . W^T (vp_linear_ce.cu).
//
//   z_j  = x_j, or c tanh(x_j / c) with a cap c
//   lse  = m + log S, m the largest z_j of the row, S = sum_j e^{z_j - m}
//   loss = lse - (1 - e) z_t - (e / V) sum_j z_j + zeta lse^2
//        = log S - (1 - e) (z_t - m) - (e / V) W + zeta lse^2,   W = sum_j (z_j - m)
//   d loss / d z_j = p_j (1 + 2 zeta lse) - (1 - e) [j = t] - e / V,   p_j = e^{z_j - m} / S
//   d z_j / d x_j  = 1 - (z_j / c)^2
// The centred form keeps its digits under a large common offset of the logits,
// which cancels in every term but zeta's.
#pragma once

#include <type_traits>

#include "vp_device.cuh"
#include "vp_launch.h"

namespace vp {

struct CeRules {
    float smooth;                // e
    float share;                 // e / V, V the whole vocabulary's
    float zeta;
    float cap, inv_cap;          // c, 1 / c (cap 0: none)
};

// Sums W are carried times 2^-24: a row may span more than the largest float, and
// the factor is exact for all that counts.
constexpr float kCeScale = 5.9604644775390625e-08f;
constexpr double kCeUnscale = 16777216.0;

// t = tanh(y) and slope = 1 - t^2. Below 5/8: y (1 + s P(s)), s = y^2, P of degree 4 by
// interpolation of tanh(y) / y at Chebyshev points (relative error 7.3e-8, all roundings
// included); above: (1 - e) / (1 + e) and 4 e / (1 + e)^2 with e = e^{-2 |y|}, which do
// not cancel there (relative error about 3e-7). A value takes its formula whatever its
// neighbours are: the vote only spares a warp the second one when none of its values needs it.
constexpr float kTanhSplit = 0.625f;
template <int n>
__device__ __forceinline__ void soft_cap(const CeRules &q, const float (&x)[n], float (&z)[n], float *slope) {
    bool far = false;
    float y[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        y[i] = x[i] * q.inv_cap;
        const float s = y[i] * y[i];
        float p = fmaf(s, -0.005657135043293238f, 0.020588191226124763f);
        p = fmaf(s, p, -0.05372010916471481f);
        p = fmaf(s, p, 0.13331113755702972f);
        p = fmaf(s, p, -0.3333325982093811f);
        const float t = fmaf(y[i] * s, p, y[i]);
        z[i] = t * q.cap;
        if (slope) slope[i] = fmaf(-t, t, 1.f);
        far |= !(fabsf(y[i]) < kTanhSplit);
    }
    if (__any_sync(__activemask(), far)) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            float e, r;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(y[i]) * (-2.f * kLog2e)));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
            if (!(fabsf(y[i]) < kTanhSplit)) {
                z[i] = copysignf((1.f - e) * r, y[i]) * q.cap;
                if (slope) slope[i] = 4.f * e * r * r;
            }
        }
    }
}

// g (a p - e / V), a = 1 + a1: a column's gradient before the cap's slope. At the target
// 1 - e is taken away in a form that does not cancel as p -> 1: p - 1 = e^{log p} - 1.
__device__ __forceinline__ float ce_grad(const CeRules &q, float p, float a1, float g) {
    return g * fmaf(a1, p, p - q.share);
}
__device__ __forceinline__ float ce_grad_target(const CeRules &q, float p, float lp, float a1, float g) {
    const float pm1 = lp > -0.5f ? expm1_small(lp) : p - 1.f;
    return g * (pm1 + fmaf(a1, p, q.smooth - q.share));
}

// What a row's pieces come to.
struct CeRow {
    float M;
    DF S, W;              // W times 2^-24
    float zt;
    uint32_t flags;       // VP_PART_* of the pieces; kCeMinusInf where W is -inf
    int owners;           // pieces that hold the target
    uint32_t n;           // columns
};
constexpr uint32_t kCeMinusInf = 1u << 30;

// Pieces of a row: vp_partial records, at [k * sk + r * sr].
struct CePieces {
    const PartialRec *parts;
    int64_t sk, sr;
    __device__ __forceinline__ float max_of(int64_t r, int k) const { return parts[k * sk + r * sr].m; }
    __device__ __forceinline__ float target(int64_t, float zt) const { return zt; }
    __device__ __forceinline__ void add(int64_t r, int k, float M, CeRow &o) const {
        const PartialRec p = parts[k * sk + r * sr];
        o.flags |= p.flags;
        if (p.flags & kPartHasTarget) {
            ++o.owners;
            o.zt = p.z_t;
        }
        const float S = (float)p.S;
        if (S != S) o.flags |= kPartNanInf;
        else if (S > 0.f) {
            const float a = expf(p.m - M);
            df_add(o.S, a * S);
            df_add(o.S, a * (float)(p.S - (double)S));
        }
        // S_b: the piece's columns
        const double W = p.W * (1.0 / kCeUnscale);
        if (W == -INFINITY) o.flags |= kCeMinusInf;
        else if (W == W) {
            const float hi = (float)W, d = fmaf(M, -kCeScale, p.m * kCeScale);
            df_add(o.W, hi);
            df_add(o.W, (float)(W - (double)hi));
            df_add(o.W, (float)p.S_b * d);
        }
        o.n += (uint32_t)p.S_b;
    }
};

// Pieces of a row that one GEMM tile of 256 columns left: (m, S, sum z, -), and the target's
// logit in an array of its own.
struct CeTiles {
    const float4 *tiles;        // [N][n_t]
    const float *zt;            // [N]
    int n_t, V;
    __device__ __forceinline__ float max_of(int64_t r, int k) const { return tiles[r * n_t + k].x; }
    __device__ __forceinline__ float target(int64_t r, float) const { return zt[r]; }
    __device__ __forceinline__ void add(int64_t r, int k, float M, CeRow &o) const {
        const float4 p = tiles[r * n_t + k];
        if (p.y != p.y) o.flags |= kPartNanInf;
        else if (p.y > 0.f) df_add(o.S, p.y * expf(p.x - M));
        const int n = min(256, V - 256 * k);
        const float w = p.z * kCeScale;
        if (w == -INFINITY) o.flags |= kCeMinusInf;
        else if (w == w) {
            df_add(o.W, w);
            df_add(o.W, -(float)n * (M * kCeScale));
        }
        o.n += (uint32_t)n;
    }
};

static CeRules ce_rules(const CeOptions &o) {
    CeRules q;
    q.smooth = (float)o.smooth;
    q.share = (float)(o.smooth / (double)o.vocab_total);
    q.zeta = (float)o.zeta;
    q.cap = (float)o.cap;
    q.inv_cap = o.cap > 0.0 ? (float)(1.0 / (double)q.cap) : 0.f;
    return q;
}

struct CeJoinArgs {
    int64_t N, V, vocab_start;
    const int64_t *targets;      // not needed where the pieces are gathered shards
    float *loss;
    RowStat *stats;
    int32_t *err;
    PartialRec *parts;           // the shard's records, where they are wanted instead
    double smooth, zeta;
};

// One warp for four rows, a lane for every 32nd piece, in a fixed order; then one lane for
// each of the CTA's 32 rows takes the logarithm in 64 bits: a whole warp's worth of that narrow
// pipe for 32 rows, not for one.
constexpr int kCeJoinRows = 32;
enum CeJoin { kCeLoss, kCeRecords, kCeShards };   // losses; the shard's records; losses of gathered shards
template <class Src, CeJoin kind>
__global__ void __launch_bounds__(256)
ce_join_kernel(const Src src, int K, const CeJoinArgs a) {
    __shared__ CeRow rows[kCeJoinRows];
    pdl_enter<false>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * kCeJoinRows;
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + warp * 4 + i;
        if (r >= a.N) break;
        CeRow o{kNegBig, {0.f, 0.f}, {0.f, 0.f}, 0.f, 0u, 0, 0u};
        for (int k = lane; k < K; k += 32) o.M = fmaxf(o.M, src.max_of(r, k));
        o.M = warp_max(o.M);
        for (int k = lane; k < K; k += 32) src.add(r, k, o.M, o);
        const unsigned holders = __ballot_sync(0xffffffffu, o.owners > 0);
        o.zt = __shfl_sync(0xffffffffu, o.zt, holders ? __ffs(holders) - 1 : 0);
        o.owners = __reduce_add_sync(0xffffffffu, o.owners);
        o.flags = __reduce_or_sync(0xffffffffu, o.flags);
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            df_add(o.S, shfl_xor(o.S, m));
            df_add(o.W, shfl_xor(o.W, m));
        }
        o.n = __reduce_add_sync(0xffffffffu, o.n);
        if (lane == 0) rows[warp * 4 + i] = o;
    }
    __syncthreads();
    if (warp != 0 || r0 + lane >= a.N) return;
    const int64_t r = r0 + lane;
    const CeRow o = rows[lane];
    const double S = df_value(o.S);
    const double W = (o.flags & kCeMinusInf) ? -INFINITY : df_value(o.W) * kCeUnscale;
    const bool nan = (o.flags & kPartNanInf) || S != S;
    bool ignored, bad;
    float zt = o.zt;
    if (kind == kCeShards) {
        ignored = (o.flags & kPartIgnored) != 0;
        bad = !ignored && o.owners != 1;
    } else {
        const int64_t t = a.targets[r], loc = t - a.vocab_start;
        ignored = t < 0;
        bad = !ignored && (loc < 0 || loc >= a.V);
        zt = ignored || bad ? 0.f : src.target(r, zt);
    }
    if (kind == kCeRecords) {
        uint32_t pf = nan ? kPartNanInf : 0u;
        if (ignored) pf |= kPartIgnored;
        else if (!bad) pf |= kPartHasTarget;
        a.parts[r] = PartialRec{S > 0.0 ? o.M : kNegBig, 0.f, nan ? (double)qnan() : S, (double)o.n, W, zt, pf};
        return;
    }
    uint32_t flags = 0;
    if (nan) flags |= kRowNanInf;
    else if (S == 0.0) flags |= kRowEmpty;
    const double logS = log(nan ? (double)qnan() : S), lse = (double)o.M + logS;
    const bool broken = flags != 0;
    if (kind == kCeShards) flags |= kRowSharded | (bad ? kRowBadTarget : 0u);
    store_rowstat(a.stats + r, o.M, logS, 0.0, flags);
    if (bad && a.err) atomicOr(a.err, VP_ERRBIT_TARGET_);
    double loss = logS + a.zeta * lse * lse;
    if (a.smooth < 1.0) loss -= (1.0 - a.smooth) * ((double)zt - (double)o.M);
    if (a.smooth > 0.0) loss -= a.smooth * (W / (double)o.n);
    a.loss[r] = ignored ? 0.f : (bad || broken) ? qnan() : (float)loss;
}

// A row's K pieces made its loss and record, or the shard's record (a.parts), or, of gathered
// shards, the whole row's loss and record.
template <class Src>
static cudaError_t launch_ce_join(const Src &src, int K, const CeArgs &a, bool shards) {
    const CeJoinArgs j{a.N, a.V, a.vocab_start, a.targets, a.loss, static_cast<RowStat *>(a.stats), a.err,
                       static_cast<PartialRec *>(a.parts), a.opt.smooth, a.opt.zeta};
    const dim3 grid((unsigned)((a.N + kCeJoinRows - 1) / kCeJoinRows));
    if (a.parts) return launch_pdl(ce_join_kernel<Src, kCeRecords>, grid, dim3(256), 0, a.stream, src, K, j);
    if constexpr (std::is_same<Src, CePieces>::value)
        if (shards) return launch_pdl(ce_join_kernel<Src, kCeShards>, grid, dim3(256), 0, a.stream, src, K, j);
    return launch_pdl(ce_join_kernel<Src, kCeLoss>, grid, dim3(256), 0, a.stream, src, K, j);
}

}  // namespace vp
