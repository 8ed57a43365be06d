// vp_linear_ce.cu -- softmax cross entropy of hidden . W^T without keeping the logits,
// forward and backward on tcgen05 tensor cores (formulas: vp_ce.cuh; the GEMMs, their
// order and their bounds: vp_gemm.cuh).
//
// Forward: tiles of 256 rows x 256 vocabulary rows; the epilogue reads a tile from TMEM, caps
//   its logits, and leaves per row the tile's (max, sum of exponentials, sum of logits) and the
//   target's logit; ce_join_kernel makes them the row's loss. 2 N V D flops.
// Backward, a piece of the vocabulary at a time: the piece's logits again, dz in the
//   epilogue (through the cap's slope) as one or two bf16 values, then dhidden += dz . W_c and
//   dW_c = dz^T . h. 6 N V D flops, 10 with dz as a pair.
// Bound: the tensor cores, and the power they draw.
#include "vp_ce.cuh"
#include "vp_gemm.cuh"
#include "vp_stats.cuh"

namespace vp {

template <bool kCap>
struct CeEpi {
    int N, n_t;
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
        float m = kNegBig, S = 0.f, zt = 0.f, Z0 = 0.f, Z1 = 0.f;
#pragma unroll 1
        for (int c = 0; c < kLBN / 32; ++c) {
            float v[32];
            tmem_ld32(taddr + c * 32, v);
            const int n = ncol - c * 32;                 // columns of the vocabulary left
            if (n <= 0) continue;
            if (kCap) soft_cap(q, v);
            float cm = kNegBig;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                if (c * 32 + i == tloc) zt = v[i];
                if (c * 32 + i + 1 == tloc) zt = v[i + 1];
                Z0 += i < n ? v[i] : 0.f;
                Z1 += i + 1 < n ? v[i + 1] : 0.f;
                if (i >= n) v[i] = -INFINITY;
                if (i + 1 >= n) v[i + 1] = -INFINITY;
                cm = fmaxf(cm, fmaxf(v[i], v[i + 1]));
            }
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
        tiles[(int64_t)row * n_t + col0 / kLBN] = make_float4(m, S, Z0 + Z1, 0.f);
        if (tloc >= 0) tgt[row] = zt;
    }
};

// dz of a 256-column tile of the piece that starts at shard column v0, as bf16 (and, with
// lo_off != 0, what that rounding took away as a second one: store_dz).
template <bool kCap>
struct DzCeEpi {
    int N, V, v0, ldz;
    int64_t vocab_start;
    const int64_t *targets;
    CeRules q;
    const RowStat *stats;
    const float *g;
    __nv_bfloat16 *dz;
    int32_t *err;
    int64_t lo_off;
    __device__ __forceinline__ void operator()(int row, int col0, int ncol, uint32_t taddr) const {
        const bool valid = row < N;
        const RowStat s = load_rowstat(stats + (valid ? row : 0));
        const int64_t tg = valid ? targets[row] : -1;
        const int64_t tl = tg - vocab_start;                // target column in the shard
        const bool outside = tg >= 0 && (tl < 0 || tl >= V) && !(s.flags & kRowSharded);
        int mode = (s.flags & (kRowNanInf | kRowEmpty | kRowBadTarget)) || outside ? 2 : 0;   // 1 zeros, 2 NaN
        if (tg < 0) mode = 1;
        if (valid && outside && err && col0 == 0 && v0 == 0) atomicOr(err, VP_ERRBIT_TARGET_);
        const int64_t tl0 = tg >= 0 ? tl : -1;
        const int64_t tcol = tl0 - v0 - col0;               // target column within this tile
        const CeGradRow gr = ce_grad_row(q, s, valid ? g[row] : 0.f);
#pragma unroll 1
        for (int c = 0; c < kLBN / 32; ++c) {
            float v[32], slope[32];
            tmem_ld32(taddr + c * 32, v);
            if (kCap) soft_cap<32, true>(q, v, slope);
            const int64_t at = tcol - c * 32;
            float zt = 0.f;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                if (i == at) zt = v[i];
                if (i + 1 == at) zt = v[i + 1];
                float2 d = ce_grad2(gr, make_float2(v[i], v[i + 1]));
                v[i] = d.x;
                v[i + 1] = d.y;
            }
            if (at >= 0 && at < 32) {
                const float d = ce_grad_target(q, gr, zt);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i == at) v[i] = d;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (kCap) v[i] *= slope[i];
                if (mode == 1 || c * 32 + i >= ncol) v[i] = 0.f;
                else if (mode == 2) v[i] = qnan();
            }
            if (valid) store_dz(dz + (int64_t)row * ldz + col0 + c * 32, v, lo_off);
        }
    }
};

struct CeFwdLayout {
    size_t tiles, tgt, total;
};
static CeFwdLayout ce_fwd_layout(int64_t N, int64_t V) {
    CeFwdLayout L;
    L.tiles = 0;
    L.tgt = up256((size_t)N * ((V + kLBN - 1) / kLBN) * sizeof(float4));
    L.total = L.tgt + up256((size_t)N * sizeof(float));
    return L;
}
size_t linear_ce_workspace_bytes(int64_t N, int64_t V) { return ce_fwd_layout(N, V).total; }

cudaError_t launch_linear_ce_fwd(const CeArgs &a) {
    const CeFwdLayout L = ce_fwd_layout(a.N, a.V);
    const int n_t = (int)((a.V + kLBN - 1) / kLBN);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    float4 *tiles = reinterpret_cast<float4 *>(ws + L.tiles);
    float *tgt = reinterpret_cast<float *>(ws + L.tgt);
    const CeRules q = ce_rules(a.opt);
    auto gemm = [&](const auto &epi) {
        return launch_logits_gemm(a.hidden, a.weight, (int)a.N, (int)a.V, (int)a.D, epi, a.stream, kFwdPairs);
    };
    const cudaError_t e = q.cap > 0.f
                              ? gemm(CeEpi<true>{(int)a.N, n_t, a.vocab_start, a.targets, q, tiles, tgt})
                              : gemm(CeEpi<false>{(int)a.N, n_t, a.vocab_start, a.targets, q, tiles, tgt});
    if (e != cudaSuccess) return e;
    return launch_ce_join(CeTiles{tiles, tgt, n_t, (int)a.V}, n_t, a);
}

struct CeBwdLayout {
    size_t dz, acc, total;
};
static CeBwdLayout ce_bwd_layout(int64_t N, int64_t V, int64_t D) {
    const int64_t vc = chunk_cols(N, V);
    CeBwdLayout L;
    L.dz = 0;
    L.acc = up256((size_t)2 * N * vc * 2);
    L.total = L.acc + up256((size_t)N * D * 4);
    return L;
}
size_t linear_ce_bwd_workspace_bytes(int64_t N, int64_t V, int64_t D) { return ce_bwd_layout(N, V, D).total; }

cudaError_t launch_linear_ce_bwd(const CeArgs &a) {
    const CeBwdLayout L = ce_bwd_layout(a.N, a.V, a.D);
    const int64_t vc = chunk_cols(a.N, a.V);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    __nv_bfloat16 *dz = reinterpret_cast<__nv_bfloat16 *>(ws + L.dz);
    const int64_t lo_off = a.precision == VP_GRAD_EXACT_ ? a.N * vc : 0;   // dz_lo follows dz_hi
    float *acc = a.dhidden ? reinterpret_cast<float *>(ws + L.acc) : nullptr;
    const __nv_bfloat16 *h = static_cast<const __nv_bfloat16 *>(a.hidden);
    const __nv_bfloat16 *W = static_cast<const __nv_bfloat16 *>(a.weight);
    const RowStat *stats = static_cast<const RowStat *>(a.stats);
    const int N = (int)a.N, V = (int)a.V, D = (int)a.D;
    const CeRules q = ce_rules(a.opt);
    cudaError_t e;
    CUtensorMap tm_h_mn;
    if (!make_map_mn(&tm_h_mn, h, N, D, D)) return cudaErrorInvalidValue;
    for (int64_t v0 = 0; v0 < V; v0 += vc) {
        const int nv = (int)(V - v0 < vc ? V - v0 : vc);
        auto gemm = [&](const auto &epi) {
            return launch_logits_gemm(h, W + v0 * D, N, nv, D, epi, a.stream, kGemmPairs);
        };
        e = q.cap > 0.f ? gemm(DzCeEpi<true>{N, V, (int)v0, (int)vc, a.vocab_start, a.targets, q, stats, a.g, dz, a.err, lo_off})
                        : gemm(DzCeEpi<false>{N, V, (int)v0, (int)vc, a.vocab_start, a.targets, q, stats, a.g, dz, a.err, lo_off});
        if (e != cudaSuccess) return e;
        e = chunk_gradient_gemms(tm_h_mn, W, N, D, v0, nv, vc, dz, lo_off ? dz + lo_off : nullptr, acc,
                                 static_cast<__nv_bfloat16 *>(a.dhidden), static_cast<__nv_bfloat16 *>(a.dW), v0 + vc >= V,
                                 a.stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t read_linear_ce_fault(uint32_t *value, bool clear) { return read_tu_fault(value, clear); }

}  // namespace vp
