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

// Sums W and sums of logits are carried times 2^-33: below 2^32 columns that lie up to twice the
// largest float apart do not overflow, and the factor is exact for all that counts.
constexpr float kCeScale = 1.16415321826934814453125e-10f;
constexpr double kCeUnscale = 8589934592.0;

// z = c t and slope = 1 - t^2, t = tanh(y), y = x / c, of n (even) values. Below |y| = 5/8:
// t = y (1 + s P(s)), s = y^2, P of degree 4 by interpolation of tanh(y) / y at Chebyshev
// points (relative error 7.3e-8, all roundings included); above: (1 - e) / (1 + e) and
// 4 e / (1 + e)^2 with e = e^{-2 |y|}, which do not cancel there (about 3e-7). A value takes
// its formula whatever its neighbours are: the vote only spares a warp the second one when
// none of its values needs it. Pairs of values go through f32x2 instructions.
constexpr float kTanhSplit = 0.625f;
template <int n, bool kSlope>
__device__ __forceinline__ void soft_cap(const CeRules &q, float (&x)[n], float (&slope)[n]) {
    static_assert(n % 2 == 0, "pairs");
    float far = 0.f;
    float2 y[n / 2];
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
        y[i] = __fmul2_rn(make_float2(x[2 * i], x[2 * i + 1]), f2(q.inv_cap));
        far = fmaxf(far, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
        const float2 s = __fmul2_rn(y[i], y[i]);
        float2 p = __ffma2_rn(s, f2(-0.005657135043293238f), f2(0.020588191226124763f));
        p = __ffma2_rn(s, p, f2(-0.05372010916471481f));
        p = __ffma2_rn(s, p, f2(0.13331113755702972f));
        p = __ffma2_rn(s, p, f2(-0.3333325982093811f));
        const float2 t = __ffma2_rn(__fmul2_rn(y[i], s), p, y[i]);
        const float2 z = __fmul2_rn(t, f2(q.cap));
        x[2 * i] = z.x;
        x[2 * i + 1] = z.y;
        if (kSlope) {
            slope[2 * i] = fmaf(-t.x, t.x, 1.f);
            slope[2 * i + 1] = fmaf(-t.y, t.y, 1.f);
        }
    }
    if (__any_sync(__activemask(), far >= kTanhSplit)) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float v = i % 2 ? y[i / 2].y : y[i / 2].x;
            float e, r;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(v) * (-2.f * kLog2e)));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
            if (fabsf(v) >= kTanhSplit) {
                x[i] = copysignf((1.f - e) * r, v) * q.cap;
                if (kSlope) slope[i] = 4.f * e * r * r;
            }
        }
    }
}
template <int n>
__device__ __forceinline__ void soft_cap(const CeRules &q, float (&x)[n]) {
    float none[n];
    soft_cap<n, false>(q, x, none);
}
__device__ __forceinline__ float soft_cap1(const CeRules &q, float x, float *slope = nullptr) {
    float v[2] = {x, 0.f}, m[2];
    soft_cap<2, true>(q, v, m);
    if (slope) *slope = m[0];
    return v[0];
}

__device__ __forceinline__ float ex2_approx(float a) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(a));
    return y;
}

// Exponentials against a centre k: e^{z - k} = 2^{z l - c} f with l = fl(log2 e), c = fl(k l), so that
// one FMA makes the argument of the hardware's 2^x. z l is exact inside the FMA, and f = 2^{c - k l}
// takes back what rounding k l did to every term alike; left over is (z - k) (log2 e - l), 2e-8 of
// z - k, and the argument's own rounding. What rounding did is up to 64 at |k| = 2^30: no term is above 2^64
// and f not below 2^-64. Beyond that (rows masked by the type's lowest value, say) floats lie 128 or more
// apart, so z is k or has no weight: l = 2 and c = 2 k serve as well, or l = 1 where 2 k could overflow.
struct ExpCentre {
    float l, c, f;
};
constexpr float kFarCentre = 1073741824.f, kLargeCentre = 1.2676506002282294e30f;   // 2^30 and 2^100
__device__ __forceinline__ ExpCentre far_centre(float k, float f) {
    const float l = fabsf(k) < kLargeCentre ? 2.f : 1.f;
    return {l, k * l, f};
}
// 2^-r, r what rounding a product took away: 1 - r ln 2 is off by r^2 / 4, 2^-24 up to 2^-11
constexpr float kSmallDrift = 4.8828125e-4f;
__device__ __forceinline__ ExpCentre exp_centre(float k) {
    if (fabsf(k) > kFarCentre) return far_centre(k, 1.f);
    const float c = k * kLog2e, r = fmaf(k, kLog2e, -c);
    return {kLog2e, c, fabsf(r) <= kSmallDrift ? fmaf(r, -0.6931471805599453f, 1.f) : ex2_approx(-r)};
}
// k = a + b + b_lo, b >= 0 a row's log S: its exponential goes into f where the sum is rounded by much. That is
// rare; in the gradient's larger kernels it is called (kCall), since inline its branch costs capped bf16 rows 3 %
// (8192 x 75968: 461 us, 449 so, 445 without it), and inline in those of one warp, where the call costs 15 %
// (65536 x 256, capped: 41 us, 36 so).
__device__ __forceinline__ ExpCentre large_centre(float a, float pa, float ea, float pb, float eb) {
    const float f = ex2_approx(-pb) * fmaf(eb, -0.6931471805599453f, 1.f);
    return fabsf(a) > kFarCentre ? far_centre(a, f) : ExpCentre{kLog2e, pa, ex2_approx(-ea) * f};
}
static __device__ __noinline__ ExpCentre large_centre_call(float a, float pa, float ea, float pb, float eb) {
    return large_centre(a, pa, ea, pb, eb);
}
template <bool kCall>
__device__ __forceinline__ ExpCentre exp_centre(float a, float b, float b_lo) {
    const float pa = a * kLog2e, ea = fmaf(a, kLog2e, -pa);
    const float pb = b * kLog2e, eb = fmaf(b_lo, kLog2e, fmaf(b, 1.925963033500011e-08f, fmaf(b, kLog2e, -pb)));
    const DF s = two_sum(pa, pb);
    const float r = s.lo + (ea + eb);
    if (fabsf(r) <= kSmallDrift) return {kLog2e, s.hi, fmaf(r, -0.6931471805599453f, 1.f)};
    return kCall ? large_centre_call(a, pa, ea, pb, eb) : large_centre(a, pa, ea, pb, eb);
}
// 2^{z l - c}
__device__ __forceinline__ float ce_exp(const ExpCentre &k, float z) { return ex2_approx(fmaf(z, k.l, -k.c)); }
__device__ __forceinline__ float2 ce_exp2(const ExpCentre &k, float2 z) {
    const float2 a = __ffma2_rn(z, f2(k.l), f2(-k.c));
    return make_float2(ex2_approx(a.x), ex2_approx(a.y));
}

// Constants of a row's gradient: dz = ga 2^{z l - c} - gs for every column but the target's.
struct CeGradRow {
    ExpCentre k;
    float ga, gs, g, a1, m, logS_hi, logS_lo;
};
template <bool kCall>
__device__ __forceinline__ CeGradRow ce_grad_row(const CeRules &q, const RowStat &s, float g) {
    const ExpCentre k = exp_centre<kCall>(s.m, s.logS_hi, s.logS_lo);
    const float a1 = 2.f * q.zeta * (s.m + (s.logS_hi + s.logS_lo));
    return {k, g * (1.f + a1) * k.f, g * q.share, g, a1, s.m, s.logS_hi, s.logS_lo};
}
__device__ __forceinline__ float2 ce_grad2(const CeGradRow &r, float2 z) {
    return __ffma2_rn(f2(r.ga), ce_exp2(r.k, z), f2(-r.gs));
}
// The target's column: 1 - e is taken away in a form that does not cancel as p -> 1,
// p - 1 = e^{log p} - 1.
__device__ __forceinline__ float ce_grad_target(const CeRules &q, const CeGradRow &r, float z) {
    const DF l = df_sub(df_diff(z, r.m), r.logS_hi, r.logS_lo);
    const float lp = l.hi + l.lo, p = exp_split(l.hi, l.lo);
    const float pm1 = lp > -0.5f ? expm1_small(lp) : p - 1.f;
    return r.g * (pm1 + fmaf(r.a1, p, q.smooth - q.share));
}

// What a piece of a row, or the whole of it, comes to.
struct CeRow {
    float M;
    DF S, W;              // W times 2^-33
    float zt;
    uint32_t flags;       // VP_PART_* of the pieces; kCeMinusInf where W is -inf
    int owners;           // pieces that hold the target
    uint32_t n;           // columns
};
constexpr uint32_t kCeMinusInf = 1u << 30;

// A piece of a row as its record says it: n columns, the largest m, sum S and sum W (times 2^-33).
struct CePiece {
    float m;
    DF S, W;
    float zt;
    uint32_t flags, n;
};

// o's centre moved up to M
__device__ __forceinline__ void ce_recentre(CeRow &o, float M) {
    if (M == o.M) return;
    const float a = expf(o.M - M);
    o.S.hi *= a;
    o.S.lo *= a;
    df_add(o.W, (float)o.n * fmaf(M, -kCeScale, o.M * kCeScale));
    o.M = M;
}
// o and a piece whose maximum is not above o's
__device__ __forceinline__ void ce_add(CeRow &o, const CePiece &p) {
    o.flags |= p.flags;
    if (p.flags & kPartHasTarget) o.zt = p.zt, ++o.owners;
    if (p.S.hi != p.S.hi) o.flags |= kPartNanInf;
    else if (p.S.hi > 0.f) {
        const float a = expf(p.m - o.M);
        df_add(o.S, a * p.S.hi);
        df_add(o.S, a * p.S.lo);
    }
    if (p.W.hi == p.W.hi) {
        df_add(o.W, p.W);
        df_add(o.W, (float)p.n * fmaf(o.M, -kCeScale, p.m * kCeScale));
    }
    o.n += p.n;
}

// A slice of a row of logits: 32 bytes, written and read 16 at a time.
struct alignas(16) CeSlice {
    float m, S, S_lo, W, W_lo, zt;
    uint32_t flags, n;
};
struct CeSlices {
    const CeSlice *slices;      // [N][K]
    int K;
    __device__ __forceinline__ float target(int64_t, float zt) const { return zt; }
    __device__ __forceinline__ CePiece piece(int64_t r, int k) const {
        const uint4 *p = reinterpret_cast<const uint4 *>(slices + r * K + k);
        const uint4 a = p[0], b = p[1];
        return {__uint_as_float(a.x), {__uint_as_float(a.y), __uint_as_float(a.z)},
                {__uint_as_float(a.w), __uint_as_float(b.x)}, __uint_as_float(b.y), b.z, b.w};
    }
};

// vp_partial records of gathered shards: [K][N].
struct CeShards {
    const PartialRec *parts;
    int64_t N;
    __device__ __forceinline__ float target(int64_t, float zt) const { return zt; }
    __device__ __forceinline__ CePiece piece(int64_t r, int k) const {
        const PartialRec p = parts[k * N + r];
        const double W = p.W / kCeUnscale;
        const bool minus_inf = W == -INFINITY;
        return {p.m, df_from(p.S), minus_inf ? DF{0.f, 0.f} : df_from(W), p.z_t,
                p.flags | (minus_inf ? kCeMinusInf : 0u), (uint32_t)p.S_b};          // S_b: its columns
    }
};

// What a GEMM's epilogue left of 128 columns of a row: (m, S, sum of z times 2^-33, -), and the target's
// logit in an array of its own.
constexpr int kCeTileCols = 128;
struct CeTiles {
    const float4 *tiles;        // [N][n_t]
    const float *zt;            // [N]
    int n_t, V;
    __device__ __forceinline__ float target(int64_t r, float) const { return zt[r]; }
    __device__ __forceinline__ CePiece piece(int64_t r, int k) const {
        const float4 p = tiles[r * n_t + k];
        const int n = min(kCeTileCols, V - kCeTileCols * k);
        const bool minus_inf = p.z == -INFINITY;
        DF W{minus_inf ? 0.f : p.z, 0.f};
        if (p.z == p.z) df_add(W, -(float)n * (p.x * kCeScale));                         // sum of (z - m)
        return {p.x, {p.y, 0.f}, W, 0.f, minus_inf ? kCeMinusInf : 0u, (uint32_t)n};
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

enum CeJoin { kCeLoss, kCeRecords, kCeGathered };   // losses; the shard's records; losses of gathered shards

// A row's loss and record, or the shard's record.
template <CeJoin kind>
__device__ __forceinline__ void ce_finish(const CeRow &o, int64_t r, const CeJoinArgs &a) {
    const double S = df_value(o.S);
    const double W = (o.flags & kCeMinusInf) ? -INFINITY : df_value(o.W) * kCeUnscale;
    const bool nan = (o.flags & kPartNanInf) || S != S;
    bool ignored, bad;
    if (kind == kCeGathered) {
        ignored = (o.flags & kPartIgnored) != 0;
        bad = !ignored && o.owners != 1;
    } else {
        const int64_t t = a.targets[r], loc = t - a.vocab_start;
        ignored = t < 0;
        bad = !ignored && (loc < 0 || loc >= a.V);
    }
    const float zt = ignored || bad ? 0.f : o.zt;
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
    if (kind == kCeGathered) flags |= kRowSharded | (bad ? kRowBadTarget : 0u);
    // c: log p of the target, by which the backward knows the scale of the row's gradient
    const double lpt = ((double)zt - (double)o.M) - logS;
    store_rowstat(a.stats + r, o.M, logS, ignored || bad || broken ? 0.0 : fmax(lpt, -1e30), flags);
    if (bad && a.err) atomicOr(a.err, VP_ERRBIT_TARGET_);
    double loss = logS + a.zeta * lse * lse;
    if (a.smooth < 1.0) loss -= (1.0 - a.smooth) * ((double)zt - (double)o.M);
    if (a.smooth > 0.0) loss -= a.smooth * (W / (double)o.n);
    a.loss[r] = ignored ? 0.f : (bad || broken) ? qnan() : (float)loss;
}

// kLanes lanes for a row, each for every kLanes-th piece in a fixed order, four at once: 8 lanes where a row has
// up to 32 pieces, a warp up to 256 (6427 rows of 33: 14 us, 32 with a CTA for each), beyond that the CTA's 256 lanes, for `per` rows one after the other. Then one lane for each of
// the CTA's rows takes the logarithm in 64 bits, a warp's worth of that narrow pipe for all of them and not
// for one. Lanes and order follow from the number of pieces alone; how many rows a CTA has does not change
// a row's result: one where there are few rows (16 rows of 594 pieces: 19 us with a warp for a row, 8 us so),
// eight where there are many.
constexpr int kCeJoinThreads = 256, kCeJoinAhead = 4, kCeJoinMany = 8;
template <class Src, CeJoin kind, int kLanes>
__global__ void __launch_bounds__(kCeJoinThreads)
ce_join_kernel(const Src src, int K, int per, const CeJoinArgs a) {
    static_assert(kLanes <= 32 || kLanes == kCeJoinThreads, "within a warp, or the whole CTA");
    constexpr int kWarpLanes = kLanes < 32 ? kLanes : 32, kParts = kLanes / kWarpLanes;   // warps of a row
    constexpr int kSide = kCeJoinThreads / kLanes;                                        // rows side by side
    __shared__ CeRow rows[kLanes <= 32 ? kSide : kCeJoinMany * kParts];
    pdl_enter<true>();
    const int lane = threadIdx.x & 31, k0 = threadIdx.x % kLanes;
    const int n_rows = kSide * per;
    const int64_t r0 = (int64_t)blockIdx.x * n_rows;
    for (int t = 0; t < per; ++t) {
        const int mine = t * kSide + threadIdx.x / kLanes;
        const int64_t row = r0 + mine < a.N ? r0 + mine : a.N - 1;   // a lane without a row of its own goes along
        CeRow o{kNegBig, {0.f, 0.f}, {0.f, 0.f}, 0.f, 0u, 0, 0u};
        for (int k = k0; k < K; k += kLanes * kCeJoinAhead) {
            CePiece p[kCeJoinAhead];
            float M = o.M;
#pragma unroll
            for (int i = 0; i < kCeJoinAhead; ++i)
                if (k + i * kLanes < K) p[i] = src.piece(row, k + i * kLanes);
#pragma unroll
            for (int i = 0; i < kCeJoinAhead; ++i)
                if (k + i * kLanes < K) M = fmaxf(M, p[i].m);
            ce_recentre(o, M);
#pragma unroll
            for (int i = 0; i < kCeJoinAhead; ++i)
                if (k + i * kLanes < K) ce_add(o, p[i]);
        }
        float M = o.M;
#pragma unroll
        for (int m = kWarpLanes / 2; m > 0; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
        ce_recentre(o, M);
#pragma unroll
        for (int m = kWarpLanes / 2; m > 0; m >>= 1) {
            const int owners = __shfl_xor_sync(0xffffffffu, o.owners, m);
            const float zt = __shfl_xor_sync(0xffffffffu, o.zt, m);
            if (owners > o.owners) o.zt = zt;
            o.owners += owners;
            o.flags |= __shfl_xor_sync(0xffffffffu, o.flags, m);
            o.n += __shfl_xor_sync(0xffffffffu, o.n, m);
            df_add(o.S, shfl_xor(o.S, m));
            df_add(o.W, shfl_xor(o.W, m));
        }
        if (threadIdx.x % kWarpLanes == 0) rows[mine * kParts + threadIdx.x % kLanes / 32] = o;
    }
    __syncthreads();
    if (threadIdx.x >= n_rows || r0 + lane >= a.N) return;               // n_rows is 32 at most
    CeRow o = rows[lane * kParts];
    for (int w = 1; w < kParts; ++w) {                                   // the row's warps, in order
        CeRow p = rows[lane * kParts + w];
        const float top = fmaxf(o.M, p.M);
        ce_recentre(o, top);
        ce_recentre(p, top);
        if (p.owners > o.owners) o.zt = p.zt;
        o.owners += p.owners;
        o.flags |= p.flags;
        o.n += p.n;
        df_add(o.S, p.S);
        df_add(o.W, p.W);
    }
    if (kind != kCeGathered && a.targets[r0 + lane] >= 0) o.zt = src.target(r0 + lane, o.zt);
    ce_finish<kind>(o, r0 + lane, a);
}

static CeJoinArgs ce_join_args(const CeArgs &a) {
    return {a.N, a.V, a.vocab_start, a.targets, a.loss, static_cast<RowStat *>(a.stats), a.err,
            static_cast<PartialRec *>(a.parts), a.opt.smooth, a.opt.zeta};
}

// A row's K pieces made its loss and record, or the shard's record (a.parts), or, of gathered
// shards, the whole row's loss and record.
template <class Src>
static cudaError_t launch_ce_join(const Src &src, int K, const CeArgs &a) {
    const CeJoinArgs j = ce_join_args(a);
    const int lanes = K <= 32 ? 8 : K <= 256 ? 32 : kCeJoinThreads;
    const int per = lanes == kCeJoinThreads && a.N > 1216 ? kCeJoinMany : 1;   // eight CTAs on every SM take 1216 rows at once
    const int rows = kCeJoinThreads / lanes * per;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((a.N + rows - 1) / rows)), dim3(kCeJoinThreads), 0, a.stream, src, K, per, j);
    };
    auto sized = [&](auto k) {
        constexpr CeJoin kind = decltype(k)::value;
        return lanes == 8 ? go(ce_join_kernel<Src, kind, 8>)
                          : lanes == 32 ? go(ce_join_kernel<Src, kind, 32>) : go(ce_join_kernel<Src, kind, kCeJoinThreads>);
    };
    if constexpr (std::is_same<Src, CeShards>::value) {
        return sized(std::integral_constant<CeJoin, kCeGathered>());
    } else {
        if (a.parts) return sized(std::integral_constant<CeJoin, kCeRecords>());
        return sized(std::integral_constant<CeJoin, kCeLoss>());
    }
}

}  // namespace vp
