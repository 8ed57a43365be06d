// vp_ce.cu -- softmax cross entropy of logits, forward and backward (formulas: vp_ce.cuh).
//
// Forward: one CTA for a slice of 2048 16-byte vectors of a row (16384 bf16 or 8192 fp32
//   logits; smaller CTAs for rows that they hold), read once into registers, eight loads of a thread on their way together. The
//   slice's maximum is known before its first exponential, so nothing is rescaled; the
//   CTA leaves a record (max, sum of exponentials, sum of centred logits, the target's
//   logit) and ce_join_kernel makes a row's records its loss. A single row is then spread
//   over as many SMs as it has slices, and a row's arithmetic depends on V, its type and
//   its address modulo 16 only.
// Backward: slices of 1024 vectors (2048 with a cap), one read and one write; dx may be x.
// Bound: DRAM bytes; with a cap on bf16 logits the issue slots, of which the cap takes some 6 a column.
//   8192 x 75968 bf16, at 6.79 TB/s 183 and 367 us: forward 204, 213 to 225 with the sum that label smoothing asks
//   for, backward 355; capped 338 and 450. 4096 x 75968 fp32: forward 181 to 193, backward 345 to 349; capped 249 and 372.
#include <algorithm>

#include "vp_ce.cuh"

namespace vp {

constexpr int kCeThreads = 256;
constexpr int kCeFwdVecs = 8;                    // vectors of a thread
// Threads of a CTA: fewer for a row that they can hold, so that more rows are on their way on an SM than four. The
// number depends on V alone, as the order of a row's sums does. Forward and backward against 256 threads, in us: 65536 x 256
// bf16 43 + 22 against 212 + 120, 65536 x 2048 83 + 78 against 237 + 144, 65536 x 4096 fp32 168 + 302 against 245 + 301,
// 16384 x 4100 bf16 40 + 46 against 66 + 49; few rows of 250 vectors, whose threads then have four, 6.7 against 5.4.
static int ce_threads(bool bf16, int64_t V) {
    const int64_t most = (V + (bf16 ? 7 : 3)) / (bf16 ? 8 : 4);       // vectors
    return most <= 128 ? 32 : most <= 64 * kCeFwdVecs ? 64 : most <= 128 * kCeFwdVecs ? 128 : kCeThreads;
}
constexpr int64_t kCeFewRows = 608;              // four for each of GB300's 152 SMs; the workspace's size, asked for on any host, follows from it
constexpr int ce_grad_vecs(bool cap) { return cap ? 8 : 4; }

static int64_t ce_slices(bool bf16, int vecs, int64_t V) {
    const int64_t per = (int64_t)ce_threads(bf16, V) * vecs * (bf16 ? 8 : 4);
    return (V + per - 1) / per;
}

// Few rows of one slice are finished where they are summed, the same way as in the join; of many the logarithms in 64
// bits, one CTA's at a time, would cost more than a launch that takes 32 at once.
static bool ce_whole(int64_t N, int n_slices) { return n_slices == 1 && N <= kCeFewRows; }

int64_t ce_workspace_bytes(bool bf16, int64_t N, int64_t V) {
    const int64_t n_slices = ce_slices(bf16, kCeFwdVecs, V);
    return ce_whole(N, (int)n_slices) ? 0 : N * n_slices * (int64_t)sizeof(CeSlice);
}

// A tile's row and slice, and a row's offset, without 64-bit divisions where the sizes allow: a thread
// has 32 elements or fewer, and a division costs as much as all of them.
__device__ __forceinline__ int64_t tile_row(int64_t tile, int n_slices, int &slice) {
    if (tile <= 0xffffffffll) {
        const uint32_t r = (uint32_t)tile / (uint32_t)n_slices;
        slice = (int)((uint32_t)tile - r * (uint32_t)n_slices);
        return r;
    }
    const int64_t r = tile / n_slices;
    slice = (int)(tile - r * n_slices);
    return r;
}
__device__ __forceinline__ int64_t row_offset(const Rows &rows, int64_t r) {
    return r < rows.R ? r * rows.s_i : rows.off(r);
}

// Bytes b .. b + 15 of two vectors behind one another, b a multiple of 2.
__device__ __forceinline__ uint4 shifted(const uint4 &x, const uint4 &y, uint32_t b) {
    uint32_t w[5];                                       // from word b / 4 on
    switch (b >> 2) {                                    // the same for a whole row
        case 0: w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w; w[4] = y.x; break;
        case 1: w[0] = x.y; w[1] = x.z; w[2] = x.w; w[3] = y.x; w[4] = y.y; break;
        case 2: w[0] = x.z; w[1] = x.w; w[2] = y.x; w[3] = y.y; w[4] = y.z; break;
        default: w[0] = x.w; w[1] = y.x; w[2] = y.y; w[3] = y.z; w[4] = y.w; break;
    }
    if (b & 2)
        return make_uint4(__funnelshift_r(w[0], w[1], 16), __funnelshift_r(w[1], w[2], 16), __funnelshift_r(w[2], w[3], 16),
                          __funnelshift_r(w[3], w[4], 16));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest of the values of a vector (NaN left out, as fmaxf does).
template <typename T>
__device__ __forceinline__ float vec_max(const uint4 &u, float m) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&u);
        const __nv_bfloat162 x = __hmax2(__hmax2(b[0], b[1]), __hmax2(b[2], b[3]));
        return fmaxf(m, fmaxf(__low2float(x), __high2float(x)));
    } else {
        return fmaxf(fmaxf(m, fmaxf(__uint_as_float(u.x), __uint_as_float(u.y))),
                     fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
}

// kSum: with the sum of the centred logits, which only label smoothing asks for. kWhole: rows of one slice, finished
// here (a kernel of its own: the 64-bit logarithm would take registers from the sums).
template <typename T, bool kCap, bool kSum, bool kWhole, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
ce_fwd_kernel(const T *__restrict__ x, int V, Rows rows, const CeRules q, const int64_t *__restrict__ targets,
              int64_t vocab_start, int n_slices, int64_t total, CeSlice *__restrict__ slices,
              const CeJoinArgs join) {
    constexpr int kVec = Elem<T>::kVec, kWarps = kThreads / 32, kCeVecs = kCeFwdVecs, kCeSliceVecs = kThreads * kCeVecs;
    __shared__ float s_max[kWarps];
    __shared__ DF s_S[kWarps], s_W[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_enter<true>();   // no global access before this
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        int s;
        const int64_t r = tile_row(tile, n_slices, s);
        const T *in = x + row_offset(rows, r);
        const int head = head_count(in, V), nv = (V - head) / kVec, tail0 = head + nv * kVec;
        const int v0 = s * kCeSliceVecs, v1 = min(nv, v0 + kCeSliceVecs);
        uint4 u[kCeVecs];
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k) {
            const int i = v0 + tid + k * kThreads;
            if (i < v1) u[k] = ldg_stream(reinterpret_cast<const uint4 *>(in + head) + i);
        }
        // the first slice also takes the elements before the first vector and behind the last
        const int extra = s == 0 ? head + V - tail0 : 0;
        float ze = 0.f, zt = 0.f;
        if (tid < extra) ze = Elem<T>::load1(in + (tid < head ? tid : tail0 + tid - head));
        bool has_target = false;
        if (tid == 0) {
            const int64_t t = targets[r], loc = t - vocab_start;
            has_target = t >= 0 && loc >= 0 && loc < V &&
                         (loc < head || loc >= tail0
                              ? s == 0
                              : loc >= head + (int64_t)v0 * kVec && loc < head + (int64_t)v1 * kVec);
            if (has_target) zt = Elem<T>::load1(in + loc);
        }

        // the maximum: of the raw values, since the cap is monotonic
        float m = kNegBig;
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k)
            if (v0 + tid + k * kThreads < v1) m = vec_max<T>(u[k], m);
        if (tid < extra) m = fmaxf(m, ze);
        m = warp_max(m);
        if (lane == 0) s_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_max[w]);
        if (kCap) m = soft_cap1(q, m);
        const ExpCentre centre = exp_centre(m);

        float2 S = f2(0.f), W = f2(0.f);
        const float2 mw = f2(-m * kCeScale);
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k) {
            if (v0 + tid + k * kThreads < v1) {
                float z[kVec];
                Elem<T>::unpack(u[k], z);
                if (kCap) soft_cap(q, z);
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    const float2 zz = make_float2(z[e], z[e + 1]);
                    S = __fadd2_rn(S, ce_exp2(centre, zz));
                    if (kSum) W = __fadd2_rn(W, __ffma2_rn(zz, f2(kCeScale), mw));
                }
            }
        }
        if (kCap) ze = soft_cap1(q, ze);
        if (tid < extra) {
            S.x += ce_exp(centre, ze);
            if (kSum) W.x += fmaf(ze, kCeScale, mw.x);
        }
        DF Sd = two_sum(S.x, S.y), Wd{0.f, 0.f};
        bool minus_inf = false;
        if (kSum) {
            // a masked column (-inf) makes the sum of logits -inf, which double-floats do not carry
            minus_inf = __syncthreads_or(W.x == -INFINITY || W.y == -INFINITY);
            if (!minus_inf) Wd = two_sum(W.x, W.y);
        }
        if constexpr (Elem<T>::kPrecise) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                df_add(Sd, shfl_xor(Sd, o));
                if (kSum) df_add(Wd, shfl_xor(Wd, o));
            }
        } else {
            // bf16 logits: a lane's two sums and the five steps in fp32, at most half a step of fp32 each;
            // double-floats here cost as many instructions as 25 of the 64 columns
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                Sd.hi += __shfl_xor_sync(0xffffffffu, Sd.hi, o);
                if (kSum) Wd.hi += __shfl_xor_sync(0xffffffffu, Wd.hi, o);
            }
            Sd.lo = Wd.lo = 0.f;
        }
        if (lane == 0) {
            s_S[warp] = Sd;
            s_W[warp] = Wd;
        }
        __syncthreads();
        if (warp == 0) {
            if (kCap) zt = soft_cap1(q, zt);
            if (lane == 0) {
                for (int w = 1; w < kWarps; ++w) {
                    df_add(Sd, s_S[w]);
                    if (kSum) df_add(Wd, s_W[w]);
                }
                const float S_all = Sd.hi * centre.f;
                CeSlice o{m, S_all, fmaf(Sd.hi, centre.f, -S_all) + Sd.lo * centre.f, Wd.hi, Wd.lo, zt,
                          (has_target ? kPartHasTarget : 0u) | (minus_inf ? kCeMinusInf : 0u),
                          (uint32_t)(max(v1 - v0, 0) * kVec + extra)};
                if (!(S_all < INFINITY)) o.S = qnan(), o.S_lo = 0.f;     // a NaN, or +inf without a cap
                if constexpr (kWhole) {
                    CeRow c{m, {0.f, 0.f}, {0.f, 0.f}, 0.f, 0u, 0, 0u};
                    ce_add(c, {o.m, {o.S, o.S_lo}, {o.W, o.W_lo}, o.zt, o.flags, o.n});
                    if (join.parts) ce_finish<kCeRecords>(c, r, join);
                    else ce_finish<kCeLoss>(c, r, join);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(slices + tile);
                    dst[0] = reinterpret_cast<const uint4 *>(&o)[0];
                    dst[1] = reinterpret_cast<const uint4 *>(&o)[1];
                }
            }
        }
    }
}

// dx may be x, so the gradient's loads are ordinary ones, not those of read-only memory. A thread reads an element
// before it writes it, and no other thread reads it.
__device__ __forceinline__ uint4 load_own(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ float load_own1(const float *p) { return *p; }
__device__ __forceinline__ float load_own1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// kSame: every row of the input lies as its row of the output modulo 16 bytes
template <typename T, bool kCap, bool kSame, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 32 ? 32 : (kCap ? 4 : 5) * (kCeThreads / kThreads))
ce_grad_kernel(const T *x, int V, Rows rows, const CeRules q, const RowStat *__restrict__ stats,
               const float *__restrict__ g_in, const int64_t *__restrict__ targets, int64_t vocab_start, T *dx,
               int32_t *__restrict__ err, int n_slices, int slice_vecs, int64_t total) {
    constexpr int kVec = Elem<T>::kVec, kCeVecs = ce_grad_vecs(kCap);
    const int tid = threadIdx.x;
    pdl_enter<true>();   // no global access before this
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
        int s;
        const int64_t r = tile_row(tile, n_slices, s);
        const T *in = x + row_offset(rows, r);
        T *out = dx + r * (int64_t)V;
        const int hin = head_count(in, V), hout = head_count(out, V);
        const int v0 = s * slice_vecs;
        const bool same = kSame || hin == hout;
        const int v1 = same ? min((V - hin) / kVec, v0 + slice_vecs) : 0;
        uint4 u[kCeVecs];
#pragma unroll
        for (int k = 0; k < kCeVecs; ++k) {
            const int i = v0 + tid + k * kThreads;
            if (i < v1) u[k] = load_own(reinterpret_cast<const uint4 *>(in + hin) + i);
        }
        const RowStat st = load_rowstat(stats + r);
        int mode = (st.flags & (kRowNanInf | kRowEmpty | kRowBadTarget)) ? 2 : 0;   // 1 zeros, 2 NaN
        int loc = -1;
        const int64_t t = targets[r];
        if (t < 0) {
            mode = 1;
        } else if (t - vocab_start >= 0 && t - vocab_start < V) {
            loc = (int)(t - vocab_start);
        } else if (!(st.flags & kRowSharded)) {      // else the target lies in another shard
            mode = 2;
            if (err && s == 0 && tid == 0) atomicOr(err, VP_ERRBIT_TARGET_);
        }
        const CeGradRow row = ce_grad_row<(kThreads > 32)>(q, st, g_in[r]);
        const float constant = mode == 1 ? 0.f : qnan();

        auto one = [&](int j) {
            float z = load_own1(in + j), slope = 1.f;
            if (kCap) z = soft_cap1(q, z, &slope);
            float d = j == loc ? ce_grad_target(q, row, z) : ce_grad2(row, make_float2(z, 0.f)).x;
            if (kCap) d *= slope;
            Elem<T>::store1(out + j, mode ? constant : d);
        };
        // the gradients of a vector of columns from j0 on
        auto vector = [&](const uint4 &raw, int j0) {
            float z[kVec], slope[kVec], d[kVec];
            Elem<T>::unpack(raw, z);
            if (kCap) soft_cap<kVec, true>(q, z, slope);
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
                float2 v = ce_grad2(row, make_float2(z[e], z[e + 1]));
                if (kCap) v = __fmul2_rn(v, make_float2(slope[e], slope[e + 1]));
                d[e] = v.x;
                d[e + 1] = v.y;
            }
            const uint32_t at = (uint32_t)(loc - j0);          // the target's place in this vector
            if (at < (uint32_t)kVec) {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (e == (int)at) d[e] = ce_grad_target(q, row, z[e]) * (kCap ? slope[e] : 1.f);
            }
            if (mode) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) d[e] = constant;
            }
            return Elem<T>::pack(d);
        };
        if (same) {
            const int tail0 = hin + (V - hin) / kVec * kVec;
            if (s == 0 && tid < hin + V - tail0) one(tid < hin ? tid : tail0 + tid - hin);
            uint4 *vout = reinterpret_cast<uint4 *>(out + hin);
#pragma unroll
            for (int k = 0; k < kCeVecs; ++k) {
                const int i = v0 + tid + k * kThreads;
                if (i < v1) stg_stream(vout + i, vector(u[k], hin + i * kVec));
            }
        } else if constexpr (!kSame) {
            // Input and output rows lie differently modulo 16 bytes (an odd vocabulary out of padded rows): whole
            // vectors of the output, each out of the two of the input that its columns lie in. The first and last ones,
            // whose two would reach out of the row, go column by column, as do the ends.
            const int nv = (V - hout) / kVec, o1 = min(nv, v0 + slice_vecs);
            const uint32_t b = (uint32_t)((uintptr_t)(in + hout) & 15u);
            const uint4 *base = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint8_t *>(in + hout) - b);
            const uint4 *first = reinterpret_cast<const uint4 *>(in), *last = reinterpret_cast<const uint4 *>(in + V);
            const int tail0 = hout + nv * kVec;
            if (s == 0 && tid < hout + V - tail0) one(tid < hout ? tid : tail0 + tid - hout);
            uint4 *vout = reinterpret_cast<uint4 *>(out + hout);
#pragma unroll 2
            for (int k = 0; k < kCeVecs; ++k) {
                const int i = v0 + tid + k * kThreads;
                if (i >= o1) break;
                if (base + i < first || base + i + 2 > last) {
                    for (int e = 0; e < kVec; ++e) one(hout + i * kVec + e);
                } else {
                    vout[i] = vector(shifted(__ldg(base + i), __ldg(base + i + 1), b), hout + i * kVec);
                }
            }
        }
    }
}

// CTAs of a call: one a slice, but of one warp no more than run at once, which then go from row to row: the GPU begins
// about one a nanosecond (65536 x 256 bf16: 83 + 67 us with one for each row). Larger ones are slower so: their rows' loads
// would no longer go on beside one another (65536 x 4096 bf16: 106 + 174 against 101 + 153).
static unsigned ce_grid(int64_t total, int threads) {
    if (threads == 32) {
        int dev = 0, sms = 0;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        total = std::min<int64_t>(total, (int64_t)std::max(1, sms) * 32);
    }
    return (unsigned)(total < 2147483647 ? total : 2147483647);
}

template <typename T>
static cudaError_t ce_fwd(const CeArgs &a) {
    const int n_slices = (int)ce_slices(a.bf16, kCeFwdVecs, a.V);
    const int64_t total = a.N * n_slices;
    const CeRules q = ce_rules(a.opt);
    CeSlice *work = static_cast<CeSlice *>(a.workspace);
    const bool whole = ce_whole(a.N, n_slices);
    const int threads = ce_threads(a.bf16, a.V);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(ce_grid(total, threads)), dim3(threads), 0, a.stream, static_cast<const T *>(a.x),
                          (int)a.V, Rows{a.R, a.s_o, a.s_i}, q, a.targets, a.vocab_start, n_slices, total, work,
                          ce_join_args(a));
    };
    const bool sum = a.parts || q.smooth > 0.f;      // a shard's records are merged with any smoothing
    auto pick = [&](auto cap, auto summed) {
        constexpr bool kCap = decltype(cap)::value, kSum = decltype(summed)::value;
        auto sized = [&](auto n) {
            constexpr int kThreads = decltype(n)::value;
            return whole ? go(ce_fwd_kernel<T, kCap, kSum, true, kThreads>) : go(ce_fwd_kernel<T, kCap, kSum, false, kThreads>);
        };
        return threads == 32    ? sized(std::integral_constant<int, 32>())
               : threads == 64  ? sized(std::integral_constant<int, 64>())
               : threads == 128 ? sized(std::integral_constant<int, 128>())
                                : sized(std::integral_constant<int, kCeThreads>());
    };
    const std::true_type yes;
    const std::false_type no;
    const cudaError_t e = q.cap > 0.f ? (sum ? pick(yes, yes) : pick(yes, no)) : (sum ? pick(no, yes) : pick(no, no));
    return e != cudaSuccess || whole ? e : launch_ce_join(CeSlices{work, n_slices}, n_slices, a);
}

cudaError_t launch_ce_fwd(const CeArgs &a) { return a.bf16 ? ce_fwd<__nv_bfloat16>(a) : ce_fwd<float>(a); }

cudaError_t launch_ce_merge(const CeArgs &a, const void *parts, int64_t K) {
    return launch_ce_join(CeShards{static_cast<const PartialRec *>(parts), a.N}, (int)K, a);
}

cudaError_t launch_ce_bwd(const CeArgs &a) {
    const int threads = ce_threads(a.bf16, a.V);
    // vectors of a thread: fewer where that leaves SMs without a slice (a gradient is the same in any slice; capped bf16, 107 x 30162
    // out of odd rows 9.5 us against 11.7, 7 x 87716 3.8 against 4.7)
    int vecs = ce_grad_vecs(a.opt.cap > 0.0);
    while (vecs > 1 && a.N * ce_slices(a.bf16, vecs, a.V) < kCeFewRows) vecs /= 2;
    const int slices = (int)ce_slices(a.bf16, vecs, a.V);
    const int64_t total = a.N * slices;
    const CeRules q = ce_rules(a.opt);
    const Rows rows{a.R, a.s_o, a.s_i};
    auto go = [&](auto kernel, auto *x, auto *dx) {
        return launch_pdl(kernel, dim3(ce_grid(total, threads)), dim3(threads), 0, a.stream, x, (int)a.V, rows, q,
                          static_cast<const RowStat *>(a.stats), a.g, a.targets, a.vocab_start, dx, a.err, slices,
                          threads * vecs, total);
    };
    const float *xf = static_cast<const float *>(a.x);
    const __nv_bfloat16 *xb = static_cast<const __nv_bfloat16 *>(a.x);
    float *df = static_cast<float *>(a.dx);
    __nv_bfloat16 *db = static_cast<__nv_bfloat16 *>(a.dx);
    const int64_t es = a.bf16 ? 2 : 4;
    const bool same = ((uintptr_t)a.x - (uintptr_t)a.dx) % 16 == 0 && (a.s_i - a.V) * es % 16 == 0 &&
                      (a.R >= a.N || (a.s_o - a.R * a.V) * es % 16 == 0);
    auto pick = [&](auto tag, auto *x, auto *dx) {
        using T = std::remove_reference_t<decltype(tag)>;
        auto wide = [&](auto cap, auto alike) {
            constexpr bool kCap = decltype(cap)::value, kSame = decltype(alike)::value;
            return threads == 32    ? go(ce_grad_kernel<T, kCap, kSame, 32>, x, dx)
                   : threads == 64  ? go(ce_grad_kernel<T, kCap, kSame, 64>, x, dx)
                   : threads == 128 ? go(ce_grad_kernel<T, kCap, kSame, 128>, x, dx)
                                    : go(ce_grad_kernel<T, kCap, kSame, kCeThreads>, x, dx);
        };
        const std::true_type yes;
        const std::false_type no;
        return q.cap > 0.f ? (same ? wide(yes, yes) : wide(yes, no)) : (same ? wide(no, yes) : wide(no, no));
    };
    return a.bf16 ? pick(__nv_bfloat16(), xb, db) : pick(float(), xf, df);
}

}  // namespace vp
