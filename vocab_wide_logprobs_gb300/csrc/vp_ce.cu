// vp_ce.cu -- softmax cross entropy of logits, forward and backward (formulas: vp_ce.cuh).
//
// Forward: one CTA for a slice of 1024 16-byte vectors of a row (8192 bf16 or 4096 fp32
//   logits), read once into registers, four loads of a thread on their way together. The
//   slice's maximum is known before its first exponential, so nothing is rescaled; the
//   CTA leaves a record (max, sum of exponentials, sum of centred logits, the target's
//   logit) and ce_join_kernel makes a row's records its loss. A single row is then spread
//   over as many SMs as it has slices, and a row's arithmetic depends on V, its type and
//   its address modulo 16 only.
// Backward: the same slices, one read and one write; dx may be x.
// Bound: DRAM bytes; with a cap on the logits the forward's issue slots.
#include "vp_ce.cuh"

namespace vp {

constexpr int kCeThreads = 256, kCeVecs = 4;
constexpr int kCeSliceVecs = kCeThreads * kCeVecs;

static int64_t ce_slices(bool bf16, int64_t V) {
    const int64_t per = (int64_t)kCeSliceVecs * (bf16 ? 8 : 4);
    return (V + per - 1) / per;
}

int64_t ce_workspace_bytes(bool bf16, int64_t N, int64_t V) {
    return N * ce_slices(bf16, V) * (int64_t)sizeof(PartialRec);
}

// S += sum of e^{z - m}, W += sum of (z - m) 2^-24 over n values
template <typename T, int n>
__device__ __forceinline__ void ce_sums(const float (&z)[n], float m, float &S, float &W) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
        if constexpr (Elem<T>::kPrecise) {
            const DF t = df_diff(z[i], m);
            S += exp_split(t.hi, t.lo);
        } else {
            S += Elem<T>::exp(z[i] - m);
        }
        W += fmaf(z[i], kCeScale, -m * kCeScale);
    }
}

template <typename T, bool kCap>
__global__ void __launch_bounds__(kCeThreads)
ce_fwd_kernel(const T *__restrict__ x, int V, Rows rows, const CeRules q, const int64_t *__restrict__ targets,
              int64_t vocab_start, int slices, int64_t total, PartialRec *__restrict__ parts) {
    constexpr int kVec = Elem<T>::kVec, kWarps = kCeThreads / 32;
    __shared__ float s_max[kWarps];
    __shared__ DF s_S[kWarps], s_W[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_enter<true>();   // no global access before this
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const int64_t r = tile / slices;
        const int s = (int)(tile - r * slices);
        const T *in = x + rows.off(r);
        const int head = head_count(in, V), nv = (V - head) / kVec, tail0 = head + nv * kVec;
        const int v0 = s * kCeSliceVecs, v1 = min(nv, v0 + kCeSliceVecs);
        uint4 u[kCeVecs];
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k) {
            const int i = v0 + tid + k * kCeThreads;
            if (i < v1) u[k] = ldg_stream(reinterpret_cast<const uint4 *>(in + head) + i);
        }
        // the first slice also takes the elements before the first vector and behind the last
        const int extra = s == 0 ? head + V - tail0 : 0;
        float ze[1] = {0.f}, zt[1] = {0.f};
        if (tid < extra) ze[0] = Elem<T>::load1(in + (tid < head ? tid : tail0 + tid - head));
        bool has_target = false;
        if (tid == 0) {
            const int64_t t = targets[r], loc = t - vocab_start;
            has_target = t >= 0 && loc >= 0 && loc < V &&
                         (loc < head || loc >= tail0 ? s == 0 : loc >= head + (int64_t)v0 * kVec && loc < head + (int64_t)v1 * kVec);
            if (has_target) zt[0] = Elem<T>::load1(in + loc);
        }

        float z[kCeVecs][kVec];
        float m = kNegBig;
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k) {
            if (v0 + tid + k * kCeThreads < v1) {
                Elem<T>::unpack(u[k], z[k]);
                if (kCap) soft_cap(q, z[k], z[k], nullptr);
#pragma unroll
                for (int e = 0; e < kVec; ++e) m = fmaxf(m, z[k][e]);
            }
        }
        if (kCap) soft_cap(q, ze, ze, nullptr);
        if (tid < extra) m = fmaxf(m, ze[0]);
        m = warp_max(m);
        if (lane == 0) s_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_max[w]);

        float S = 0.f, W = 0.f;
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k)
            if (v0 + tid + k * kCeThreads < v1) ce_sums<T>(z[k], m, S, W);
        if (tid < extra) ce_sums<T>(ze, m, S, W);
        // a masked column (-inf) makes the sum of logits -inf, which double-floats do not carry
        const bool minus_inf = __syncthreads_or(W == -INFINITY);
        DF Sd{S, 0.f}, Wd{minus_inf ? 0.f : W, 0.f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            df_add(Sd, shfl_xor(Sd, o));
            df_add(Wd, shfl_xor(Wd, o));
        }
        if (lane == 0) {
            s_S[warp] = Sd;
            s_W[warp] = Wd;
        }
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < kWarps; ++w) {
                df_add(Sd, s_S[w]);
                df_add(Wd, s_W[w]);
            }
            if (kCap) soft_cap(q, zt, zt, nullptr);
            parts[tile] = PartialRec{m, 0.f, df_value(Sd), (double)(max(v1 - v0, 0) * kVec + extra),
                                     minus_inf ? -INFINITY : df_value(Wd) * kCeUnscale, zt[0],
                                     has_target ? kPartHasTarget : 0u};
        }
    }
}

template <typename T, bool kCap>
__global__ void __launch_bounds__(kCeThreads)
ce_grad_kernel(const T *x, int V, Rows rows, const CeRules q, const RowStat *__restrict__ stats,
               const float *__restrict__ g_in, const int64_t *__restrict__ targets, int64_t vocab_start, T *dx,
               int32_t *__restrict__ err, int slices, int64_t total) {
    constexpr int kVec = Elem<T>::kVec;
    const int tid = threadIdx.x;
    pdl_enter<true>();   // no global access before this
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const int64_t r = tile / slices;
        const int s = (int)(tile - r * slices);
        const T *in = x + rows.off(r);
        T *out = dx + r * (int64_t)V;
        const int hin = head_count(in, V), hout = head_count(out, V);
        const int v0 = s * kCeSliceVecs;
        const int v1 = hin == hout ? min((V - hin) / kVec, v0 + kCeSliceVecs) : 0;
        uint4 u[kCeVecs];
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k) {
            const int i = v0 + tid + k * kCeThreads;
            if (i < v1) u[k] = ldg_stream(reinterpret_cast<const uint4 *>(in + hin) + i);
        }
        const RowStat st = load_rowstat(stats + r);
        float g = g_in[r];
        int64_t loc = -1;
        int mode = (st.flags & (kRowNanInf | kRowEmpty | kRowBadTarget)) ? 2 : 0;   // 1 zeros, 2 NaN
        const int64_t t = targets[r];
        if (t < 0) {
            mode = 1;
        } else {
            loc = t - vocab_start;
            if (loc < 0 || loc >= V) {
                loc = -1;
                if (!(st.flags & kRowSharded)) {      // else the target lies in another shard
                    mode = 2;
                    if (err && s == 0 && tid == 0) atomicOr(err, VP_ERRBIT_TARGET_);
                }
            }
        }
        const float a1 = 2.f * q.zeta * (st.m + (st.logS_hi + st.logS_lo));
        const float constant = mode == 1 ? 0.f : qnan();

        // n consecutive columns from j0 on
        auto columns = [&](auto &v, int64_t j0) {
            constexpr int n = sizeof(v) / sizeof(float);
            float slope[n];
            if (kCap) soft_cap(q, v, v, slope);
#pragma unroll
            for (int e = 0; e < n; ++e) {
                float lp, p;
                if constexpr (Elem<T>::kPrecise) {
                    const DF l = df_sub(df_diff(v[e], st.m), st.logS_hi, st.logS_lo);
                    lp = l.hi;
                    p = exp_split(l.hi, l.lo);
                    if (j0 + e == loc) lp = l.hi + l.lo;
                } else {
                    lp = (v[e] - st.m) - st.logS_hi;
                    p = Elem<T>::exp(lp);
                    if (j0 + e == loc) lp -= st.logS_lo;
                }
                float d = j0 + e == loc ? ce_grad_target(q, p, lp, a1, g) : ce_grad(q, p, a1, g);
                if (kCap) d *= slope[e];
                v[e] = mode ? constant : d;
            }
        };
        auto one = [&](int64_t j) {
            float v[1] = {Elem<T>::load1(in + j)};
            columns(v, j);
            Elem<T>::store1(out + j, v[0]);
        };
        if (hin == hout) {
            const int tail0 = hin + (V - hin) / kVec * kVec;
            if (s == 0 && tid < hin + V - tail0) one(tid < hin ? tid : tail0 + tid - hin);
#pragma unroll
            for (int k = 0; k < kCeVecs; ++k) {
                const int i = v0 + tid + k * kCeThreads;
                if (i < v1) {
                    float v[kVec];
                    Elem<T>::unpack(u[k], v);
                    columns(v, hin + (int64_t)i * kVec);
                    stg_stream(reinterpret_cast<uint4 *>(out + hin) + i, Elem<T>::pack(v));
                }
            }
        } else {   // input and output rows lie differently modulo 16 bytes
            const int64_t e0 = (int64_t)s * kCeSliceVecs * kVec, e1 = min((int64_t)V, e0 + (int64_t)kCeSliceVecs * kVec);
            for (int64_t j = e0 + tid; j < e1; j += kCeThreads) one(j);
        }
    }
}

static unsigned ce_grid(int64_t total) { return (unsigned)(total < 2147483647 ? total : 2147483647); }

cudaError_t launch_ce_fwd(const CeArgs &a) {
    const int slices = (int)ce_slices(a.bf16, a.V);
    const int64_t total = a.N * slices;
    const CeRules q = ce_rules(a.opt);
    const Rows rows{a.R, a.s_o, a.s_i};
    PartialRec *work = static_cast<PartialRec *>(a.workspace);
    auto go = [&](auto kernel, auto *x) {
        return launch_pdl(kernel, dim3(ce_grid(total)), dim3(kCeThreads), 0, a.stream, x, (int)a.V, rows, q, a.targets,
                          a.vocab_start, slices, total, work);
    };
    const float *xf = static_cast<const float *>(a.x);
    const __nv_bfloat16 *xb = static_cast<const __nv_bfloat16 *>(a.x);
    cudaError_t e = a.bf16 ? (q.cap > 0.f ? go(ce_fwd_kernel<__nv_bfloat16, true>, xb) : go(ce_fwd_kernel<__nv_bfloat16, false>, xb))
                           : (q.cap > 0.f ? go(ce_fwd_kernel<float, true>, xf) : go(ce_fwd_kernel<float, false>, xf));
    if (e != cudaSuccess) return e;
    return launch_ce_join(CePieces{work, 1, slices}, slices, a, false);
}

// Losses of gathered shards: parts [K, N], shard-major.
cudaError_t launch_ce_merge(const CeArgs &a, const void *parts, int64_t K) {
    return launch_ce_join(CePieces{static_cast<const PartialRec *>(parts), a.N, 1}, (int)K, a, true);
}

cudaError_t launch_ce_bwd(const CeArgs &a) {
    const int slices = (int)ce_slices(a.bf16, a.V);
    const int64_t total = a.N * slices;
    const CeRules q = ce_rules(a.opt);
    const Rows rows{a.R, a.s_o, a.s_i};
    auto go = [&](auto kernel, auto *x, auto *dx) {
        return launch_pdl(kernel, dim3(ce_grid(total)), dim3(kCeThreads), 0, a.stream, x, (int)a.V, rows, q,
                          static_cast<const RowStat *>(a.stats), a.g, a.targets, a.vocab_start, dx, a.err, slices, total);
    };
    const float *xf = static_cast<const float *>(a.x);
    const __nv_bfloat16 *xb = static_cast<const __nv_bfloat16 *>(a.x);
    float *df = static_cast<float *>(a.dx);
    __nv_bfloat16 *db = static_cast<__nv_bfloat16 *>(a.dx);
    return a.bf16 ? (q.cap > 0.f ? go(ce_grad_kernel<__nv_bfloat16, true>, xb, db) : go(ce_grad_kernel<__nv_bfloat16, false>, xb, db))
                  : (q.cap > 0.f ? go(ce_grad_kernel<float, true>, xf, df) : go(ce_grad_kernel<float, false>, xf, df));
}

}  // namespace vp
