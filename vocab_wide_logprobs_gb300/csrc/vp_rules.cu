// vp_rules.cu -- the rules a sampler puts on logits (penalties for repeated
// tokens, sparse biases, a packed mask of allowed tokens, a temperature), their
// gradient, and the logprobs of the ruled distribution with their gradient.
//
// Row r, column j (id v = vocab_start + j), c_p and c_o the occurrences of v
// among the row's prompt and output ids:
//   z = x;                       c_p + c_o > 0:  z = z > 0 ? z / rep : z * rep
//   c_o > 0:  z -= freq c_o + pres;     v in the bias list:  z += bias(v)
//   y = allowed(j) ? z / T : -inf
//   f = dy/dx = allowed(j) ? (c_p + c_o > 0 ? (x > 0 ? 1 / rep : rep) : 1) / T : 0
//
// Shape: a CTA takes a slice of kSlice columns of one row. Its thread t holds
// the octets (8 consecutive columns) t, t + 256, ... of the slice in registers,
// loaded before anything else so that they arrive while the CTA builds its
// tables in shared memory: a word per column with the number of output
// occurrences and a prompt bit, a word with the last bias entry, and a bit per
// column that is set where either is. Integer atomics only, so the order of
// the ids does not matter. The pass over the octets then looks at one byte of
// that bitmap and one byte of the mask per octet; only columns with a bit set
// read the tables.
//
// The ruled logprobs' forward writes one vp_partial record per (slice, row),
// as a vocabulary shard would, and merge_stats_kernel joins a row's slices.
// The slices depend on V alone, so a row's results do not depend on N.
#include "vp_launch.h"
#include "vp_device.cuh"

namespace vp {

constexpr int kRuleThreads = 256;
constexpr int kOctsPerThread = 4;
constexpr int kSlice = kRuleThreads * kOctsPerThread * 8;   // 8192 columns
constexpr uint32_t kPromptBit = 0x80000000u;

enum RuleOp { kProcFwd = 0, kProcBwd = 1, kLogpFwd = 2, kLogpBwd = 3 };

// Raw bits of 8 elements: one 16-byte vector of bf16, two of fp32.
template <typename T> struct Oct {
    static constexpr int kVecs = sizeof(T) / 2;
    uint4 u[kVecs];
};

// Plain (coherent) loads: y may be x.
__device__ __forceinline__ uint4 ld_once(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

__device__ __forceinline__ float ld_elem(const float *p) { return *reinterpret_cast<const volatile float *>(p); }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16 *p) {
    return __uint_as_float((uint32_t) * reinterpret_cast<const volatile unsigned short *>(p) << 16);
}

// n valid elements at p (vec: n == 8 and p is 16-byte aligned); the rest is 0.
template <typename T>
__device__ __forceinline__ void load_oct(Oct<T> &o, const T *p, int n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
        for (int i = 0; i < Oct<T>::kVecs; ++i) o.u[i] = ld_once(reinterpret_cast<const uint4 *>(p) + i);
        return;
    }
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? ld_elem(p + i) : 0.f;
#pragma unroll
    for (int i = 0; i < Oct<T>::kVecs; ++i) o.u[i] = Elem<T>::pack(v + i * Elem<T>::kVec);
}

template <typename T>
__device__ __forceinline__ void unpack_oct(const Oct<T> &o, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < Oct<T>::kVecs; ++i) Elem<T>::unpack(o.u[i], v + i * Elem<T>::kVec);
}

template <typename T>
__device__ __forceinline__ void store_oct(T *p, const float (&v)[8], int n, bool vec) {
    if (vec && n >= 8) {
#pragma unroll
        for (int i = 0; i < Oct<T>::kVecs; ++i)
            stg_stream(reinterpret_cast<uint4 *>(p) + i, Elem<T>::pack(v + i * Elem<T>::kVec));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) Elem<T>::store1(p + i, v[i]);
}

struct RuleKernelArgs {
    const void *x, *dy;
    void *out;
    int64_t N, n_slices, vocab_start;
    int V;
    Rows xrows, orows;
    RuleSet q;
    const int64_t *targets;
    const RowStat *stats;
    const float *g;
    PartialRec *parts;
    int32_t *err;
};

// The rules of one row, read and checked once per CTA.
struct RowRules {
    bool ok;
    int64_t first, n_prompt, n_total, bias_first, n_bias;
    float rep, freq, pres, inv_t;
    const uint8_t *mask;      // the row's mask bytes, NULL: everything allowed
};

__device__ __forceinline__ bool span_ok(int64_t first, int64_t n, int64_t total) {
    // n < 2^31: occurrences are counted in 31 bits
    return first >= 0 && n >= 0 && n <= 0x7fffffff && n <= total && first <= total - n;
}

__device__ RowRules row_rules(const RuleSet &q, int64_t r) {
    RowRules w{true, 0, 0, 0, 0, 0, 1.f, 0.f, 0.f, 1.f, nullptr};
    if (q.spans) {
        w.first = q.spans[3 * r];
        w.n_prompt = q.spans[3 * r + 1];
        w.n_total = q.spans[3 * r + 2];
        w.ok = span_ok(w.first, w.n_total, q.n_ids) && w.n_prompt >= 0 && w.n_prompt <= w.n_total;
        if (q.repetition) {
            w.rep = q.repetition[r];
            w.ok = w.ok && w.rep > 0.f && w.rep < pinf();
        }
        if (q.frequency) w.freq = q.frequency[r];
        if (q.presence) w.pres = q.presence[r];
    }
    if (q.bias_spans) {
        w.bias_first = q.bias_spans[2 * r];
        w.n_bias = q.bias_spans[2 * r + 1];
        w.ok = w.ok && span_ok(w.bias_first, w.n_bias, q.n_bias);
    }
    if (q.temperature) {
        const float t = q.temperature[r];
        w.ok = w.ok && t > 0.f && t < pinf();
        w.inv_t = 1.f / t;
    }
    if (q.mask) {
        const int64_t m = q.mask_rows ? q.mask_rows[r] : r;
        w.ok = w.ok && m >= -1 && m < q.n_masks;
        if (w.ok && m >= 0) w.mask = reinterpret_cast<const uint8_t *>(q.mask + m * q.mask_stride);
    }
    if (!w.ok) w.n_total = w.n_bias = 0;
    return w;
}

template <typename T, int kOp>
__global__ void __launch_bounds__(kRuleThreads) rules_kernel(const RuleKernelArgs a) {
    extern __shared__ uint32_t tables[];                 // counts [kSlice], then (with a bias list) entries [kSlice]
    __shared__ uint32_t touched[kSlice / 32];
    __shared__ float red_m[kRuleThreads / 32];
    __shared__ double red_s[kRuleThreads / 32];
    __shared__ uint32_t red_flags;
    __shared__ float target_z;
    pdl_enter<kOp != kLogpFwd>();

    const int tid = threadIdx.x;
    const int64_t total = a.N * a.n_slices;
    uint32_t *const counts = tables, *const entries = tables + kSlice;
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const int64_t r = tile / a.n_slices;
        const int slice = (int)(tile - r * a.n_slices);
        const int s0 = slice * kSlice;
        const int width = min(kSlice, a.V - s0);          // columns of this slice
        const T *xrow = static_cast<const T *>(a.x) + a.xrows.off(r) + s0;
        const bool xvec = ((uintptr_t)xrow & 15u) == 0;

        // ---- the slice's logits (dy for the gradient of the rules), in flight from here
        Oct<T> raw[kOctsPerThread];
        const T *main_row = kOp == kProcBwd ? static_cast<const T *>(a.dy) + r * a.V + s0 : xrow;
        const bool mvec = kOp == kProcBwd ? ((uintptr_t)main_row & 15u) == 0 : xvec;
#pragma unroll
        for (int k = 0; k < kOctsPerThread; ++k) {
            const int c = (k * kRuleThreads + tid) * 8;
            load_oct(raw[k], main_row + c, width - c, mvec);
        }
        const RowRules w = row_rules(a.q, r);
        uint32_t allow[kOctsPerThread];
#pragma unroll
        for (int k = 0; k < kOctsPerThread; ++k) {
            const int c = (k * kRuleThreads + tid) * 8;
            allow[k] = w.mask && c < width ? __ldg(w.mask + ((s0 + c) >> 3)) : 0xffu;
        }
        if (!w.ok && slice == 0 && tid == 0 && a.err) atomicOr(a.err, VP_ERRBIT_RULES_);

        // ---- tables
        const bool listed = w.n_total > 0 || w.n_bias > 0;   // uniform in the CTA
        if (listed) {
            for (int i = tid; i < kSlice / 32; i += kRuleThreads) touched[i] = 0u;
            if (w.n_total > 0)
                for (int i = tid; i < kSlice / 4; i += kRuleThreads)
                    reinterpret_cast<uint4 *>(counts)[i] = make_uint4(0u, 0u, 0u, 0u);
            if (w.n_bias > 0)
                for (int i = tid; i < kSlice / 4; i += kRuleThreads)
                    reinterpret_cast<uint4 *>(entries)[i] = make_uint4(0u, 0u, 0u, 0u);
            __syncthreads();
            const uint64_t base = (uint64_t)a.vocab_start + (uint64_t)s0;
            const int64_t *ids = a.q.ids + w.first;
            constexpr int kUnroll = 4;
            for (int64_t i0 = tid; i0 < w.n_total; i0 += kUnroll * kRuleThreads) {
                int64_t id[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int64_t i = i0 + u * kRuleThreads;
                    id[u] = i < w.n_total ? __ldg(ids + i) : -1;
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const uint64_t l = (uint64_t)id[u] - base;
                    if (id[u] < 0 || l >= (uint64_t)width) continue;
                    if (i0 + u * kRuleThreads < w.n_prompt) atomicOr(&counts[l], kPromptBit);
                    else atomicAdd(&counts[l], 1u);
                    atomicOr(&touched[l >> 5], 1u << (l & 31));
                }
            }
            for (int64_t i = tid; i < w.n_bias; i += kRuleThreads) {
                const int64_t id = __ldg(a.q.bias_ids + w.bias_first + i);
                const uint64_t l = (uint64_t)id - base;
                if (id < 0 || l >= (uint64_t)width) continue;
                atomicMax(&entries[l], (uint32_t)i + 1u);
                atomicOr(&touched[l >> 5], 1u << (l & 31));
            }
            __syncthreads();
        }

        // z and f of column l (0 <= l < width) whose bit is set, from x
        auto ruled = [&](int l, float x, float &f) {
            float z = x;
            f = 1.f;
            if (w.n_total > 0) {
                const uint32_t c = counts[l];
                if (c) {
                    z = x > 0.f ? x / w.rep : x * w.rep;
                    f = x > 0.f ? 1.f / w.rep : w.rep;
                }
                const uint32_t n = c & ~kPromptBit;
                if (n) z = z - w.freq * (float)n - w.pres;
            }
            if (w.n_bias > 0) {
                const uint32_t e = entries[l];
                if (e) z += __ldg(a.q.bias_values + w.bias_first + (e - 1));
            }
            return z;
        };

        if constexpr (kOp == kProcFwd || kOp == kProcBwd) {
            T *orow = static_cast<T *>(a.out) + (kOp == kProcFwd ? a.orows.off(r) : r * a.V) + s0;
            const bool ovec = ((uintptr_t)orow & 15u) == 0;
#pragma unroll
            for (int k = 0; k < kOctsPerThread; ++k) {
                const int o = k * kRuleThreads + tid, c = o * 8;
                if (c >= width) break;
                float v[8];
                unpack_oct(raw[k], v);
                const uint32_t hit = listed ? reinterpret_cast<const uint8_t *>(touched)[o] : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (hit >> i & 1u) {
                        float f;
                        if (kOp == kProcFwd) v[i] = ruled(c + i, v[i], f);
                        else { ruled(c + i, ld_elem(xrow + c + i), f); v[i] *= f; }
                    }
                    v[i] *= w.inv_t;
                    if (!(allow[k] >> i & 1u)) v[i] = kOp == kProcFwd ? -pinf() : 0.f;
                    if (!w.ok) v[i] = qnan();
                }
                store_oct(orow + c, v, width - c, ovec);
            }
        } else if constexpr (kOp == kLogpFwd) {
            float z[kOctsPerThread][8];
            float m = kNegBig;
            uint32_t flags = w.ok ? 0u : kPartNanInf;
            const int64_t tg = a.targets[r];
            const int64_t tl = tg - a.vocab_start - s0;      // the target's column in this slice, if any
            const bool has_target = tg >= 0 && tl >= 0 && tl < width;
#pragma unroll
            for (int k = 0; k < kOctsPerThread; ++k) {
                const int o = k * kRuleThreads + tid, c = o * 8;
                unpack_oct(raw[k], z[k]);
                const uint32_t hit = listed ? reinterpret_cast<const uint8_t *>(touched)[o] : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float f;
                    if (hit >> i & 1u) z[k][i] = ruled(c + i, z[k][i], f);
                    z[k][i] *= w.inv_t;
                    if (!(allow[k] >> i & 1u) || c + i >= width) z[k][i] = -pinf();
                    if (!(z[k][i] < pinf())) flags = kPartNanInf;      // NaN or +inf
                    m = fmaxf(m, z[k][i]);
                    if (has_target && c + i == (int)tl) target_z = z[k][i];
                }
            }
            m = warp_max(m);
            if (tid == 0) red_flags = 0u;
            if ((tid & 31) == 0) red_m[tid >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kRuleThreads / 32; ++i) m = fmaxf(m, red_m[i]);
            if (flags) atomicOr(&red_flags, flags);
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kOctsPerThread; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += Elem<T>::exp(z[k][i] - m);
            double sd = warp_sum((double)s);
            if ((tid & 31) == 0) red_s[tid >> 5] = sd;
            __syncthreads();
            if (tid == 0) {
                sd = 0.0;
                for (int i = 0; i < kRuleThreads / 32; ++i) sd += red_s[i];
                flags = red_flags;
                if (tg < 0) flags |= kPartIgnored;
                if (has_target) flags |= kPartHasTarget;
                a.parts[(int64_t)slice * a.N + r] = PartialRec{m, kNegBig, sd, 0.0, 0.0, has_target ? target_z : 0.f, flags};
            }
        } else {
            const RowStat st = load_rowstat(a.stats + r);
            const int64_t tg = a.targets[r];
            const int64_t tl = tg - a.vocab_start - s0;
            const bool ignored = tg < 0;
            const bool nan_row = !ignored && (!w.ok || (st.flags & (kRowNanInf | kRowEmpty | kRowBadTarget)) != 0);
            const int target = !ignored && tl >= 0 && tl < width ? (int)tl : -1;
            const float g = ignored ? 0.f : a.g[r];
            T *orow = static_cast<T *>(a.out) + r * a.V + s0;
            const bool ovec = ((uintptr_t)orow & 15u) == 0;
#pragma unroll
            for (int k = 0; k < kOctsPerThread; ++k) {
                const int o = k * kRuleThreads + tid, c = o * 8;
                if (c >= width) break;
                float v[8];
                unpack_oct(raw[k], v);
                const uint32_t hit = listed ? reinterpret_cast<const uint8_t *>(touched)[o] : 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float f = 1.f;
                    if (hit >> i & 1u) v[i] = ruled(c + i, v[i], f);
                    const float d = ((v[i] * w.inv_t - st.m) - st.logS_hi) - st.logS_lo;     // log p
                    f *= w.inv_t * g;
                    v[i] = c + i == target ? -f * expm1f(d) : -f * Elem<T>::exp(d);
                    if (!(allow[k] >> i & 1u) || ignored) v[i] = 0.f;
                    if (nan_row) v[i] = qnan();
                }
                store_oct(orow + c, v, width - c, ovec);
            }
        }
        if (tile + gridDim.x < total) __syncthreads();    // the tables are used again
    }
}

int64_t rule_slices(int64_t V) { return (V + kSlice - 1) / kSlice; }

template <typename T, int kOp>
static cudaError_t launch_rules_t(const RuleKernelArgs &k, cudaStream_t stream) {
    const size_t smem = (k.q.bias_spans ? 2 : k.q.spans ? 1 : 0) * (size_t)kSlice * 4;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(rules_kernel<T, kOp>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             2 * kSlice * 4);
        if (e != cudaSuccess) return e;
    }
    const int64_t total = k.N * k.n_slices;
    return launch_pdl(rules_kernel<T, kOp>, dim3((unsigned)(total < 0x7fffffff ? total : 0x7fffffff)), dim3(kRuleThreads),
                      smem, stream, k);
}

template <int kOp>
static cudaError_t launch_rules(const RuleArgs &a) {
    RuleKernelArgs k{a.x, a.dy, a.out, a.N, rule_slices(a.V), a.vocab_start, (int)a.V, Rows{a.R, a.s_o, a.s_i},
                     Rows{a.R, a.out_s_o, a.out_s_i}, a.rules, a.targets, static_cast<const RowStat *>(a.stats), a.g,
                     static_cast<PartialRec *>(a.parts), a.err};
    // no rule that reads the ids: the spans are not looked at
    if (!k.q.repetition && !k.q.frequency && !k.q.presence) k.q.spans = nullptr;
    return a.bf16 ? launch_rules_t<__nv_bfloat16, kOp>(k, a.stream) : launch_rules_t<float, kOp>(k, a.stream);
}

cudaError_t launch_process_fwd(const RuleArgs &a) { return launch_rules<kProcFwd>(a); }
cudaError_t launch_process_bwd(const RuleArgs &a) { return launch_rules<kProcBwd>(a); }
cudaError_t launch_processed_logprobs_bwd(const RuleArgs &a) { return launch_rules<kLogpBwd>(a); }

cudaError_t launch_processed_logprobs_fwd(const RuleArgs &a, float *logp, void *stats) {
    cudaError_t e = launch_rules<kLogpFwd>(a);
    if (e != cudaSuccess) return e;
    return launch_logprobs_merge(MergeArgs{a.parts, rule_slices(a.V), a.N, logp, stats, nullptr, a.err, a.stream});
}

}  // namespace vp
