// vp_rules.cu -- the rules a sampler puts on logits (penalties for repeated
// tokens, sparse biases, a packed mask of allowed tokens, a temperature), their
// gradient, and the logprobs of the ruled distribution with their gradient.
//
// Row r, column j (id v = vocab_start + j), c_p and c_o the occurrences of v
// among the row's prompt and output ids:
//   z = x;                       c_p + c_o > 0:  z = z > 0 ? z (1 / rep) : z rep
//   c_o > 0:  z -= freq c_o + pres;     v in the bias list:  z += bias(v)
//   y = allowed(j) ? z (1 / T) : -inf
//   f = dy/dx = allowed(j) ? (c_p + c_o > 0 ? (x > 0 ? 1 / rep : rep) : 1) / T : 0
//
// Shape. A tile is a slice of 4096 columns of one row; a CTA works through
// consecutive tiles (a row's slices follow one another, its rules are read once).
// One bulk copy brings the next tile to shared memory while this one is worked on.
// Thread t owns the 16-byte vectors t, t + kThreads, ... of a tile. Of the ids the
// CTA builds tables for the tile: a word per column (half a word where fewer than
// 2^15 ids are given) with the number of output occurrences and a prompt bit, a
// word with the last bias entry, and a bit per column that is set where either
// is. Integer atomics only, so the order of the ids does not matter.
//   - The vector pass treats every column as if no list named it: a few packed
//     instructions per vector, one byte (fp32: four bits) of the mask for each.
//   - The columns that a list names (a few in a hundred) and the target are
//     walked apart: in the ruled logprobs' forward they are taken out of the
//     vector pass and their exponentials summed as integers, elsewhere they
//     overwrite what the vector pass stored. Looking the tables up vector by
//     vector instead had nearly every warp go through the slow path for a lane
//     or two.
// The walk clears the entries that it has read, so the tables are zero again.
// Of a row whose slices a CTA has several of, the ids are counted by slice and then
// sorted by slice, for as many slices at a time as the list in shared memory holds:
// going through all of them for every slice cost more than everything else, with long
// histories most of all (2048 x 75968 bf16, histories of 16384 to 17407 ids: processing
// 556 us, 1134 with only those rows sorted whose ids all fit).
//
// The ruled logprobs' forward writes one vp_partial record per (slice, row),
// as a vocabulary shard would, and rules_join_kernel joins a row's slices.
// The slices depend on V alone, so a row's results do not depend on N.
#include <atomic>
#include <type_traits>

#include "vp_device.cuh"
#include "vp_gemm_host.cuh"
#include "vp_launch.h"
#include "vp_tma.cuh"
#include "vp_waits.h"

namespace vp {

constexpr uint32_t kPromptBit = 0x80000000u;

enum RuleOp { kProcFwd = 0, kProcBwd = 1, kLogpFwd = 2, kLogpBwd = 3 };

// A tile's threads and size. Five CTAs an SM (fp32: four) are what the registers are
// held to; the kernels come out with fewer and run up to eight. Ruled logprobs' forward
// on GB300, us, 8192 x 75968 bf16 with 1000 ids a row: five 591, four 710, six 679,
// seven and eight 691; 1024 x 75968 fp32: four 136, three 153, five 151. (Tiles of 8192
// columns, tried when the kernel was new, took 1.37 times as long.)
template <typename E, int kN> struct Tile {
    using T = E;
    static constexpr int kThreads = kN, kWarps = kThreads / 32;
    static constexpr int kVec = Elem<T>::kVec;                // columns of a 16-byte vector
    static constexpr int kWidth = 4096;                       // columns of a tile
    static constexpr int kVecs = kWidth / kVec / kThreads;    // vectors of a thread
    static constexpr int kCtas = kThreads > 256 ? 1 : kThreads > 128 ? 3 : sizeof(T) == 4 ? 4 : 5;   // of an SM, if their shared memory fits
    static constexpr int kWords = kWidth / 32;                // words of the bitmap
    static constexpr uint32_t kAll = kVec == 8 ? 0xffu : 0xfu;
};
constexpr int kRuleThreads = 128;
// Rules on logits whose histories are longer than a tile: going through the ids is
// most of the work, and four warps are few for it (64 x 151936 fp32 with up to 16384
// ids a row: 97 us with 128 threads, 81 with 256; 1024 x 75968 bf16 with 1000 ids: 91
// and 113).
constexpr int kRuleThreadsLong = 256;
// ... of so few rows with histories that every tile has an SM of its own (us, one row
// of 151936 bf16, ids of the row: 700: 11 with 512 threads and 11 with 128; 4000: 13
// and 20; 32768: 23, and 36 with 256; 131072: 51 and 92).
constexpr int kRuleThreadsFew = 512;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// The CTAs of an SM that the registers are held to, and the pairs of ids of a thread on
// their way at once. Together they decide what registers a kernel comes out with, and
// so how many CTAs run: measured op by op, and again whenever the kernel changes. The
// ruled logprobs' backward (8192 x 75968 bf16 with 1000 ids a row, us): 7 CTAs and 3
// pairs 513, 2 pairs 525, 4 547; 6 and 2 546; 5 and 2 556. Off the boundaries (1024 x
// 75967): 5 and 2 143, 7 and 2 155, 7 and 3 159. Processing there: 5 and 6 114, with 3
// to 5 pairs or 6 to 7 CTAs 136 to 142.
template <typename T, int kOp, int kN, bool kAligned> constexpr int rule_ctas() {
    return kOp == kLogpBwd && sizeof(T) == 2 && kAligned ? 7 : Tile<T, kN>::kCtas;
}
template <int kOp, int kN, bool kAligned> constexpr uint32_t rule_pairs() {
    return kN > kRuleThreads || kOp == kProcBwd ? 8 : kOp == kLogpBwd ? kAligned ? 3 : 2 : 6;
}

// Orders this thread's earlier stores to shared memory before later bulk copies there.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A tile in shared memory lies as it does in memory modulo 16 bytes: column c at byte
// phase + c sizeof(T) of its buffer, phase that of the tile's address. The whole
// 16-byte blocks come as one bulk copy, issued by one thread and awaited by all; the
// up to 15 bytes before and after them are stored by the threads whose vectors reach
// into them.
template <typename T>
struct TileSource {
    const T *p;
    uint32_t phase;
    int first, last, width;   // columns [first, last) are whole blocks
    __device__ __forceinline__ TileSource(const T *src, int w)
        : p(src), phase((uint32_t)(uintptr_t)src & 15u), width(w) {
        first = min(w, (int)(((16u - phase) & 15u) / sizeof(T)));
        last = first + (w - first) / Elem<T>::kVec * Elem<T>::kVec;
    }
    __device__ __forceinline__ bool bulk() const { return last > first; }
    __device__ __forceinline__ T *at(T *buffer, int c) const { return buffer + phase / sizeof(T) + c; }
};

template <class L>
__device__ __forceinline__ void stage_edges(const TileSource<typename L::T> &t, typename L::T *buffer) {
    constexpr int kVec = L::kVec;
    bool wrote = false;
    if (t.first > 0 && threadIdx.x == 0) {                // block 0 is read with vector 0
        for (int c = 0; c < t.first; ++c) *t.at(buffer, c) = t.p[c];
        wrote = true;
    }
    if (t.last < t.width) {                               // block b with vector b and, phase or not, the one before
        const int b = (int)(t.phase / sizeof(typename L::T) + t.last) / kVec, me = (int)threadIdx.x;
        if (me == b % L::kThreads || (t.phase && b > 0 && me == (b - 1) % L::kThreads)) {
            for (int c = t.last; c < t.width; ++c) *t.at(buffer, c) = t.p[c];
            wrote = true;
        }
    }
    if (wrote) fence_async_proxy();                       // a bulk copy may write there later
}

// Bytes t .. t + 15 (t < 16, a multiple of 2) of a and b, one after the other.
__device__ __forceinline__ uint4 bytes_at(const uint4 &a, const uint4 &b, uint32_t t) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (t & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (t & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = (t & 3u) * 8u;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Vector o of a staged tile.
template <bool kAligned, typename T>
__device__ __forceinline__ uint4 staged_vec(const T *buffer, uint32_t phase, int o) {
    const uint4 *b = reinterpret_cast<const uint4 *>(buffer) + o;
    return kAligned ? b[0] : bytes_at(b[0], b[1], phase);
}

// Stores a warp's 32 neighbouring vectors (this lane's n columns, n <= 0: none) at p.
// Where p is off a 16-byte boundary (the whole tile's is, by the same phase), each
// lane stores the aligned block that begins in the vector before its own; the ends of
// the 32 vectors, and of the tile, go column by column. Called by whole warps.
template <bool kAligned, typename T>
__device__ __forceinline__ void store_vec(T *p, const uint4 &u, int n, uint32_t phase) {
    constexpr int kVec = Elem<T>::kVec;
    const T *e = reinterpret_cast<const T *>(&u);
    if (kAligned || phase == 0) {
        if (n >= kVec) {
            stg_stream(p, u);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (i < n) p[i] = e[i];
        }
        return;
    }
    uint4 before;
    before.x = __shfl_up_sync(0xffffffffu, u.x, 1);
    before.y = __shfl_up_sync(0xffffffffu, u.y, 1);
    before.z = __shfl_up_sync(0xffffffffu, u.z, 1);
    before.w = __shfl_up_sync(0xffffffffu, u.w, 1);
    const int lane = threadIdx.x & 31;
    const int split = (int)((16u - phase) / sizeof(T));   // this vector's columns in the block that begins before it
    const bool whole = n >= kVec, block = whole && lane > 0;
    if (block) stg_stream(reinterpret_cast<char *>(p) - phase, bytes_at(before, u, 16u - phase));
    // the next vector's block is not stored where it is not whole or in another warp
    const int from = block ? split : 0, to = lane == 31 || n - kVec < kVec ? n : split;
    if (from < to) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i >= from && i < to) p[i] = e[i];
    }
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
    bool tabled;              // a penalty reads the ids; without one the spans are only checked
    int row_ids;              // capacity of the list of a row's ids
    bool narrow;              // occurrences counted in 15 bits: fewer ids than that in all
};

// The rules of one row, read and checked when a CTA comes to it, and what else
// its tiles share.
struct RowRules {
    bool ok;
    uint32_t n_prompt, n_total, n_bias;
    float rep, inv_rep, freq, pres, inv_t;
    const int64_t *ids, *bias_ids;
    const float *bias_values;
    const uint8_t *mask;      // the row's mask bytes, NULL: everything allowed
    int target;               // the target's column of this call, -1: not in it
    bool ignored;             // no target (logprobs)
    bool nan_row;             // the row's outputs are NaN
    float m, log_s, scale;    // logprobs backward: log p = (v / T - m) - log_s; scale = -g / T. Elsewhere scale = 1 / T
    // The row's first element in x and in the output: offsets from the kernel's arguments, so that the
    // compiler sees global memory. The ruled logprobs' forward keeps an address of x instead: off the
    // boundaries 64 registers rather than 96, 1024 x 75967 bf16 in 108 us rather than 126 (at them the same).
    int64_t x_off, out_off;
    const void *x;
};

// What z is divided by is multiplied by as its fp32 reciprocal, which has to fit (from
// 2^-127 on: also its product with log2 e); at most half a step more than a quotient.
__device__ __forceinline__ bool divisor_ok(float d) { return d >= 0x1p-127f && d < pinf(); }

__device__ __forceinline__ bool span_ok(int64_t first, int64_t n, int64_t total) {
    // n < 2^31: occurrences are counted in 31 bits
    return first >= 0 && n >= 0 && n <= 0x7fffffff && n <= total && first <= total - n;
}

template <typename T, int kOp>
__device__ RowRules row_rules(const RuleKernelArgs &a, int64_t r) {
    const RuleSet &q = a.q;
    RowRules w{};
    w.ok = true;
    w.rep = w.inv_rep = w.inv_t = 1.f;
    if (q.spans) {
        const int64_t first = q.spans[3 * r], n_prompt = q.spans[3 * r + 1], n = q.spans[3 * r + 2];
        w.ok = span_ok(first, n, q.n_ids) && n_prompt >= 0 && n_prompt <= n;
        w.ids = q.ids + first;
        w.n_prompt = (uint32_t)n_prompt;
        w.n_total = a.tabled ? (uint32_t)n : 0u;
        if (q.repetition) {
            w.rep = q.repetition[r];
            w.inv_rep = 1.f / w.rep;
            w.ok = w.ok && divisor_ok(w.rep);
        }
        if (q.frequency) w.freq = q.frequency[r];
        if (q.presence) w.pres = q.presence[r];
    }
    if (q.bias_spans) {
        const int64_t first = q.bias_spans[2 * r], n = q.bias_spans[2 * r + 1];
        w.ok = w.ok && span_ok(first, n, q.n_bias);
        w.bias_ids = q.bias_ids + first;
        w.bias_values = q.bias_values + first;
        w.n_bias = (uint32_t)n;
    }
    if (q.temperature) {
        const float t = q.temperature[r];
        w.ok = w.ok && divisor_ok(t);
        w.inv_t = 1.f / t;
    }
    if (q.mask) {
        const int64_t m = q.mask_rows ? q.mask_rows[r] : r;
        w.ok = w.ok && m >= -1 && m < q.n_masks;
        if (w.ok && m >= 0) w.mask = reinterpret_cast<const uint8_t *>(q.mask + m * q.mask_stride);
    }
    if (!w.ok) w.n_total = w.n_bias = 0u;
    w.target = -1;
    w.nan_row = !w.ok;
    w.scale = w.inv_t;
    w.x_off = a.xrows.off(r);
    w.x = static_cast<const T *>(a.x) + w.x_off;
    w.out_off = kOp == kProcFwd ? a.orows.off(r) : r * a.V;
    if (kOp >= kLogpFwd) {
        const int64_t tg = a.targets[r], tl = tg - a.vocab_start;
        w.ignored = tg < 0;
        if (tg >= 0 && tl >= 0 && tl < a.V) w.target = (int)tl;
    }
    if (kOp == kLogpBwd) {
        const RowStat st = load_rowstat(a.stats + r);
        w.nan_row = !w.ignored && (!w.ok || (st.flags & (kRowNanInf | kRowEmpty | kRowBadTarget)) != 0);
        w.scale = w.ignored ? 0.f : -a.g[r] * w.inv_t;
        w.m = st.m;
        w.log_s = st.logS_hi;
    }
    return w;
}

// The exponential of an element type, of t = u log p: bf16 takes the hardware's
// 2^t (u = log2 e), fp32 e^t (u = 1).
template <typename T> struct Scaled;
template <> struct Scaled<__nv_bfloat16> {
    static constexpr float kUnit = kLog2e;
    static __device__ __forceinline__ float exp(float t) {
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
        return y;
    }
};
template <> struct Scaled<float> {
    static constexpr float kUnit = 1.f;
    static __device__ __forceinline__ float exp(float t) { return expf(t); }
};
// ... of both values of a pair
template <typename T>
__device__ __forceinline__ float2 scaled_exp2(float2 t) {
    return make_float2(Scaled<T>::exp(t.x), Scaled<T>::exp(t.y));
}

// Columns of a vector whose bit in `on` is clear become `off` (the bits of a
// value, twice for bf16). bf16 takes the vector's keep words, two for each four bits,
// from a table in shared memory.
template <typename T>
__device__ __forceinline__ uint4 keep_vec(uint4 u, uint32_t on, uint32_t off, const uint2 *keep_words) {
    if (sizeof(T) == 2) {
        const uint2 k = keep_words[on & 15u], l = keep_words[on >> 4];
        return make_uint4((u.x & k.x) | (off & ~k.x), (u.y & k.y) | (off & ~k.y), (u.z & l.x) | (off & ~l.x),
                          (u.w & l.y) | (off & ~l.y));
    }
    return make_uint4(on & 1u ? u.x : off, on & 2u ? u.y : off, on & 4u ? u.z : off, on & 8u ? u.w : off);
}

template <typename T> __device__ __forceinline__ uint32_t minus_inf_bits() {
    return sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
}

// The largest of a vector's values; NaN is passed over.
template <typename T> __device__ __forceinline__ float vec_max(const uint4 &u) {
    if (sizeof(T) == 2) {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&u);
        const __nv_bfloat162 m = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}

// Listed columns of a tile that are kept as a list; with more of them the bitmap
// is walked instead. A CTA that has several slices of a row, at most kSegment, sorts the
// row's ids among them by slice, into a list whose capacity the launch chooses.
constexpr int kListed = 512, kSegment = 64, kRowIdsLeast = 2048, kRowIdsMost = 32768;
// The listed columns' exponentials are summed as integers, in units of 2^-48 of
// the tile's largest, so that the order they are found in does not matter.
constexpr float kFixed = 281474976710656.f;   // 2^48

__device__ __forceinline__ float redux_max(float v) {      // NaN is passed over
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// Sum over the warp of integers below 2^58 - 2^53.
__device__ __forceinline__ unsigned long long redux_sum(unsigned long long v) {
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x7ffffffu);
    const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 27));
    return ((unsigned long long)hi << 27) + lo;
}

template <class L>
struct RuleSmem {
    using T = typename L::T;
    T stage[2][L::kWidth + L::kVec];                      // a tile, and its phase
    uint2 keep_words[16];
    alignas(16) uint8_t allowed[2][L::kWidth / 8];        // the tile's mask bits
    uint64_t full[2];
    unsigned long long listed_sum[2][L::kWarps];
    uint32_t touched[L::kWords];
    float red_top[2][L::kWarps], red_all[2][L::kWarps], red_s[2][L::kWarps], target_v[2];
    uint32_t n_listed[2];
    int seg_n;                                            // counted slices
    uint32_t seg_first;                                   // row_ids[0] is the id of this number, of the counted ones
    uint32_t segment[kSegment + 1];                       // where a slice's ids begin in row_ids; counters before that
    uint16_t listed[kListed];
    // counts [kWidth], with a bias list entries [kWidth], then the row's ids follow
};

template <typename T, int kOp, int kN, bool kAligned>
__global__ void __launch_bounds__(Tile<T, kN>::kThreads, (rule_ctas<T, kOp, kN, kAligned>()))
rules_kernel(const __grid_constant__ RuleKernelArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using L = Tile<T, kN>;
    constexpr int kThreads = L::kThreads, kVec = L::kVec, kVecs = L::kVecs, kSlice = L::kWidth,
                  kWords = L::kWords, kWarps = L::kWarps;
    RuleSmem<L> &sm = *reinterpret_cast<RuleSmem<L> *>(smem_raw);
    uint32_t *const counts = reinterpret_cast<uint32_t *>(smem_raw + sizeof(RuleSmem<L>));
    uint32_t *const entries = counts + (a.tabled ? a.narrow ? kSlice / 2 : kSlice : 0);
    // column of the slice, bit 15: prompt
    uint16_t *const row_ids = reinterpret_cast<uint16_t *>(entries + (a.q.bias_spans ? kSlice : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint8_t *const touched8 = reinterpret_cast<const uint8_t *>(sm.touched);
    const bool biased = a.q.bias_spans != nullptr;

    // the tables are cleared once; a tile clears what it touched
    for (int i = tid; i < kWords; i += kThreads) sm.touched[i] = 0u;
    for (int i = tid; i < (int)(entries - counts + (biased ? kSlice : 0)) / 4; i += kThreads)
        reinterpret_cast<uint4 *>(counts)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 16)
        sm.keep_words[tid] = make_uint2((tid & 1 ? 0xffffu : 0u) | (tid & 2 ? 0xffff0000u : 0u),
                                        (tid & 4 ? 0xffffu : 0u) | (tid & 8 ? 0xffff0000u : 0u));
    if (tid < 2) sm.n_listed[tid] = 0u;
    if (tid == 0) {
        mbar_init(&sm.full[0], 1);
        mbar_init(&sm.full[1], 1);
        fence_mbar_init();
    }
    pdl_enter<kOp != kLogpFwd>();

    const int64_t total = a.N * a.n_slices;
    const int64_t per = total / gridDim.x, more = total - per * gridDim.x;
    int64_t tile = blockIdx.x * per + min((int64_t)blockIdx.x, more);
    const int64_t end = tile + per + (blockIdx.x < more ? 1 : 0);
    int64_t r = tile / a.n_slices;
    int slice = (int)(tile - r * a.n_slices);
    const uint64_t policy = policy_evict_first();
    uint32_t parity = 0u;                                // next_phase
    bool arrived = true, fresh = true, sorted = false;   // fresh: the CTA's first tile of this row
    int seg0 = 0, seg_to = -1;                           // ... was this slice; row_ids holds ids up to the seg_to-th from it, -1: none

    // brings a tile of a row to a buffer; what to know of it there
    struct Staged { uint32_t phase; bool bulk; };
    auto stage = [&](int buf, const RowRules &w, int sl) {
        const int s0 = sl * kSlice, width = min(kSlice, a.V - s0);
        const T *p = s0 + (kOp == kLogpFwd   ? static_cast<const T *>(w.x)
                           : kOp == kProcBwd ? static_cast<const T *>(a.dy) + w.out_off
                                             : static_cast<const T *>(a.x) + w.x_off);
        auto copy = [&](T *to, const T *from, int n) {
            const uint32_t bytes = (uint32_t)n * (uint32_t)sizeof(T);
            mbar_arrive_expect_tx(&sm.full[buf], bytes);
            bulk_g2s(to, from, bytes, &sm.full[buf], policy);
        };
        if (kAligned && width == kSlice) {                // whole blocks and no edges
            if (tid == 0 && arrived) copy(sm.stage[buf], p, kSlice);
            return Staged{0u, true};
        }
        const TileSource<T> t(p, width);
        if (tid == 0 && arrived && t.bulk()) copy(t.at(sm.stage[buf], t.first), t.p + t.first, t.last - t.first);
        stage_edges<L>(t, sm.stage[buf]);
        return Staged{t.phase, t.bulk()};
    };
    // this thread's mask bits of a tile, vector k in byte k % 4 of word k / 4
    struct Allow { uint32_t b[(kVecs + 3) / 4]; };
    auto mask_bits = [&](const RowRules &w, int sl) {
        Allow m;
#pragma unroll
        for (int k = 0; k < (kVecs + 3) / 4; ++k) m.b[k] = w.mask ? 0u : 0x01010101u * L::kAll;
        if (w.mask) {
            const int o = (sl * kSlice + tid * kVec) >> 3, n = (a.V - 1) / 8 + 1, sh = kVec == 8 ? 0 : (tid & 1) * 4;
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                const int at = o + k * (kThreads * kVec / 8);
                if (at < n) m.b[k / 4] |= ((uint32_t)__ldg(w.mask + at) >> sh & L::kAll) << (8 * (k % 4));
            }
        }
        return m;
    };
    RowRules w = row_rules<T, kOp>(a, r), next_w = w;
    __syncthreads();                                     // the barriers are set up, the tables clear
    Staged staged = stage(0, w, slice);
    Allow allow = mask_bits(w, slice);

    for (int buf = 0; tile < end; ++tile, buf ^= 1) {
        const int s0 = slice * kSlice;
        const int width = min(kSlice, a.V - s0);          // columns of this slice
        const T *xrow = static_cast<const T *>(a.x) + w.x_off + s0;
        const T *const buffer = sm.stage[buf];
        const uint32_t phase = kAligned ? 0u : staged.phase;
        const T *const st = buffer + phase / sizeof(T);   // column 0
        if (!w.ok && slice == 0 && tid == 0 && a.err) atomicOr(a.err, VP_ERRBIT_RULES_);
        // the target's column in this slice, if it lies here
        const int target = kOp >= kLogpFwd && w.target >= s0 && w.target - s0 < width ? w.target - s0 : -1;

        // ---- the next tile (every thread is done with the other buffer)
        const bool row_ends = slice + 1 == a.n_slices;
        const int next_slice = row_ends ? 0 : slice + 1;
        Allow next_allow = allow;
        Staged next_staged = staged;
        if (tile + 1 < end) {
            if (row_ends) {
                next_w = row_rules<T, kOp>(a, r + 1);
                next_staged = stage(buf ^ 1, next_w, 0);
                next_allow = mask_bits(next_w, 0);
            } else {
                next_staged = stage(buf ^ 1, w, next_slice);
                next_allow = mask_bits(w, next_slice);
            }
        }

        // f(column past base, index) for the ids of the row's history whose columns lie below reach;
        // 4 to 16 ids of a thread on their way at once
        auto each = [&](uint64_t base, uint64_t reach, auto f) {
            const uint32_t head = min(w.n_total, (uint32_t)((uintptr_t)w.ids >> 3 & 1u));   // to a 16-byte boundary
            const uint32_t pairs = (w.n_total - head) / 2u;
            auto one = [&](uint32_t i, uint64_t id) {
                const uint64_t l = id - base;             // negative ids come out far above any reach
                if (l < reach) f((uint32_t)l, i);
            };
            constexpr uint32_t kUnroll = rule_pairs<kOp, kN, kAligned>();
            const ulonglong2 *const p = reinterpret_cast<const ulonglong2 *>(w.ids + head);
#pragma unroll 1
            for (uint32_t i0 = tid; i0 < pairs; i0 += kUnroll * kThreads) {
                ulonglong2 id[kUnroll];
#pragma unroll
                for (uint32_t u = 0; u < kUnroll; ++u) {
                    const uint32_t i = i0 + u * kThreads;
                    id[u] = i < pairs ? __ldg(p + i) : make_ulonglong2(~0ull, ~0ull);
                }
#pragma unroll
                for (uint32_t u = 0; u < kUnroll; ++u) {
                    const uint32_t i = head + 2u * (i0 + u * kThreads);
                    one(i, id[u].x);
                    one(i + 1u, id[u].y);
                }
            }
            if (tid == 0 && head) one(0u, (uint64_t)__ldg(w.ids));
            if (tid == 1 && (w.n_total - head) % 2u) one(w.n_total - 1u, (uint64_t)__ldg(w.ids + w.n_total - 1u));
        };
        const uint64_t base = (uint64_t)a.vocab_start + (uint64_t)s0;

        // ---- a row that this CTA has several slices of: its ids are counted by slice once, and sorted by
        // slice for as many slices at a time as row_ids has room for
        if (fresh) {
            fresh = false;
            seg0 = slice;
            seg_to = -1;
            sorted = false;
            const int seg_n = (int)min(end - tile, a.n_slices - (int64_t)slice);
            if (w.n_total != 0u && seg_n > 1 && seg_n <= kSegment) {
                seg_to = 0;
                if (tid == 0) sm.seg_n = seg_n;
                for (int i = tid; i <= kSegment; i += kThreads) sm.segment[i] = 0u;
                __syncthreads();
                each(base, (uint64_t)min((int64_t)seg_n * kSlice, (int64_t)a.V - s0),
                     [&](uint32_t l, uint32_t) { atomicAdd(&sm.segment[l / kSlice + 1], 1u); });
                __syncthreads();
                if (warp == 0) {                          // counts to beginnings
                    uint32_t lo = sm.segment[1 + lane], hi = sm.segment[33 + lane];
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const uint32_t a0 = __shfl_up_sync(0xffffffffu, lo, d), b0 = __shfl_up_sync(0xffffffffu, hi, d);
                        if (lane >= d) { lo += a0; hi += b0; }
                    }
                    hi += __shfl_sync(0xffffffffu, lo, 31);
                    sm.segment[1 + lane] = lo;
                    sm.segment[33 + lane] = hi;
                }
                __syncthreads();
            }
        }
        const int k = slice - seg0;
        if (k == seg_to) {
            // The next slices whose ids fit: none are placed yet, so segment holds their beginnings. Where not
            // even one slice's fit, its ids are gone through for itself.
            const uint32_t first = sm.segment[k], last = first + (uint32_t)a.row_ids;
#pragma unroll 1
            for (const int n = sm.seg_n; seg_to < n && sm.segment[seg_to + 1] <= last; ++seg_to) {}
            sorted = seg_to > k;
            __syncthreads();
            if (sorted) {                                 // the beginnings move to the ends as the ids are placed
                if (tid == 0) sm.seg_first = first;
                each(base, (uint64_t)min((int64_t)(seg_to - k) * kSlice, (int64_t)a.V - s0), [&](uint32_t l, uint32_t i) {
                    const uint32_t at = atomicAdd(&sm.segment[k + l / kSlice], 1u) - first;
                    row_ids[at] = (uint16_t)(l % kSlice | (i < w.n_prompt ? 0x8000u : 0u));
                });
                __syncthreads();
            } else {
                if (tid == 0) sm.segment[k] = sm.segment[k + 1];
                ++seg_to;
            }
        }

        // ---- tables (the target is listed too, without an entry)
        const bool listed = (w.n_total | w.n_bias) != 0u || target >= 0;    // uniform in the CTA
        if (listed) {
            auto mark = [&](uint32_t c) {
                const uint32_t bit = 1u << (c & 31);
                if (atomicOr(&sm.touched[c >> 5], bit) & bit) return;
                const uint32_t at = atomicAdd(&sm.n_listed[buf], 1u);
                if (at < (uint32_t)kListed) sm.listed[at] = (uint16_t)c;
                if (kOp == kProcBwd) asm volatile("prefetch.global.L2 [%0];" ::"l"(xrow + c));
            };
            auto enter = [&](uint32_t c, bool prompt) {
                if (a.narrow) {
                    const uint32_t sh = (c & 1) * 16;
                    if (prompt) atomicOr(&counts[c >> 1], 0x8000u << sh);
                    else atomicAdd(&counts[c >> 1], 1u << sh);
                } else {
                    if (prompt) atomicOr(&counts[c], kPromptBit);
                    else atomicAdd(&counts[c], 1u);
                }
                mark(c);
            };
            if (tid == kThreads - 1 && target >= 0) mark((uint32_t)target);
            if (sorted) {
                // row_ids begins with the first of these slices, whose own beginning is the end of the one before
                const uint32_t first = sm.seg_first, to = sm.segment[k] - first;
                // from the second warp on: the first is late, it has issued the next tile's copy
                for (uint32_t i = (k ? sm.segment[k - 1] - first : 0u) + (tid + kThreads - 32) % kThreads; i < to;
                     i += kThreads)
                    enter(row_ids[i] & 0x7fffu, row_ids[i] >> 15);
            } else {
                each(base, (uint64_t)width, [&](uint32_t l, uint32_t i) { enter(l, i < w.n_prompt); });
            }
#pragma unroll 1
            for (uint32_t i = tid; i < w.n_bias; i += kThreads) {
                const uint64_t l = (uint64_t)__ldg(w.bias_ids + i) - base;
                if (l >= (uint64_t)width) continue;
                atomicMax(&entries[(uint32_t)l], i + 1u);
                mark((uint32_t)l);
            }
        }
        if (staged.bulk && arrived) {
            if (!mbar_wait(&sm.full[buf], next_phase(parity, buf))) {
                // Late: flagged, and this thread waits for no later tile. The first one begins no more copies
                // (the barrier's arrival is spent, its phase open) and sees those under way land before it goes
                // on, so that the CTA keeps its shared memory until then. What it computes from here on is void.
                arrived = false;
                atomicOr(&g_linear_fault, 1u);
                mbar_wait(&sm.full[buf], next_phase(parity, buf));
                if (tile + 1 < end && next_staged.bulk) mbar_wait(&sm.full[buf ^ 1], next_phase(parity, buf ^ 1));
            }
            parity ^= 1u << buf;
        }
        if (listed) {
            if (w.mask) {                                 // this thread's mask bits, for the walk
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const uint32_t b = allow.b[k / 4] >> (8 * (k % 4)) & L::kAll;
                    const int o = k * kThreads + tid;
                    if (kVec == 8) {
                        sm.allowed[buf][o] = (uint8_t)b;
                    } else {                              // four bits each: a pair of lanes makes a byte
                        const uint32_t both = b | __shfl_down_sync(0xffffffffu, b, 1) << 4;
                        if (!(tid & 1)) sm.allowed[buf][o >> 1] = (uint8_t)both;
                    }
                }
            }
            __syncthreads();                              // the tables, and what other threads copied
        }
        const uint32_t n_listed = listed ? sm.n_listed[buf] : 0u;
        // f(column) for each listed column, by some thread
        auto walk = [&](auto f) {
            if (n_listed <= (uint32_t)kListed) {
                for (uint32_t i = tid; i < n_listed; i += kThreads) f((int)sm.listed[i]);
            } else if (kThreads > kRuleThreads) {         // long histories fill tiles: neighbouring lanes, neighbouring columns
#pragma unroll 4
                for (int i = warp; i < kWords; i += kWarps)
                    if (sm.touched[i] >> lane & 1u) f(i * 32 + lane);
            } else {
                for (int i = tid; i < kWords; i += kThreads)
                    for (uint32_t bits = sm.touched[i]; bits; bits &= bits - 1) f(i * 32 + __ffs(bits) - 1);
            }
        };
        // after the walk's last use of the bitmap
        auto clear = [&]() {
            if (n_listed <= (uint32_t)kListed) {
                for (uint32_t i = tid; i < n_listed; i += kThreads) sm.touched[sm.listed[i] >> 5] = 0u;
            } else {
                for (int i = tid; i < kWords; i += kThreads) sm.touched[i] = 0u;
            }
        };

        // v before the temperature, and f, of a listed column l from x; clears the column's entries if told to
        auto ruled = [&](int l, float x, float &f, bool last) {
            uint32_t c = 0u;
            if (a.tabled) {
                if (a.narrow) {
                    uint16_t *const h = reinterpret_cast<uint16_t *>(counts) + l;
                    c = (*h & 0x7fffu) | (uint32_t)(*h >> 15) << 31;
                    if (last) *h = 0;
                } else {
                    c = counts[l];
                    if (last) counts[l] = 0u;
                }
            }
            const uint32_t n = c & ~kPromptBit;
            f = c == 0u ? 1.f : x > 0.f ? w.inv_rep : w.rep;
            float v = x * f;
            if (n) v = fmaf(-w.freq, (float)n, v) - w.pres;
            if (biased) {
                const uint32_t e = entries[l];
                if (last) entries[l] = 0u;
                if (e) v += __ldg(w.bias_values + (e - 1));
            }
            return v;
        };
        auto allowed = [&](int l) { return !w.mask || (sm.allowed[buf][l >> 3] >> (l & 7) & 1); };

        if constexpr (kOp == kLogpFwd) {
            // Exponentials of u (v - top) / T, top the largest v before the temperature:
            // v - top is exact where it matters and cannot overflow upwards. Each thread
            // sums against its own top; warps and CTA join in a fixed order. NaN or +inf
            // make the sum NaN.
            const float c1 = w.inv_t * Scaled<T>::kUnit;
            float top = kNegBig, ltop = kNegBig, s = 0.f;   // ltop: of the listed columns, whoever finds them
            auto listed_value = [&](int l, bool last) {
                float f, v = ruled(l, to_float(st[l]), f, last);
                return allowed(l) ? v : -pinf();
            };
            walk([&](int l) {
                const float v = listed_value(l, false);
                if (!(v < pinf())) s = qnan();
                ltop = fmaxf(ltop, v);
                if (l == target) sm.target_v[buf] = v;
            });
            uint4 u[kVecs];
            auto read = [&](auto whole) {                 // whole: a tile of full width
                constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int o = k * kThreads + tid, n = kWhole ? kVec : width - o * kVec;
                    const uint32_t off = minus_inf_bits<T>();
                    u[k] = make_uint4(off, off, off, off);
                    if (n > 0) {
                        u[k] = staged_vec<kAligned>(buffer, phase, o);
                        uint32_t on = allow.b[k / 4] >> (8 * (k % 4)) & L::kAll;
                        if (listed)
                            on &= ~(kVec == 8 ? (uint32_t)touched8[o] : (uint32_t)touched8[o >> 1] >> ((tid & 1) * 4));
                        if (n < kVec) on &= (1u << n) - 1u;
                        if (on != L::kAll) u[k] = keep_vec<T>(u[k], on, off, sm.keep_words);
                    }
                    top = fmaxf(top, vec_max<T>(u[k]));
                }
            };
            if (kAligned && width == kSlice) read(std::bool_constant<kAligned>());
            else read(std::false_type());
            float2 e = make_float2(s, 0.f);
#pragma unroll
            for (int k = 0; k < kVecs; ++k) {
                float v[kVec];
                Elem<T>::unpack(u[k], v);
#pragma unroll
                for (int i = 0; i < kVec; i += 2) {
                    const float2 d = __fadd2_rn(make_float2(v[i], v[i + 1]), f2(-top));
                    e = __fadd2_rn(e, scaled_exp2<T>(__fmul2_rn(d, f2(c1))));
                }
            }
            s = e.x + e.y;
            const float wtop = redux_max(top);
            s *= Scaled<T>::exp((top - wtop) * c1);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (listed) ltop = redux_max(ltop);
            if (lane == 0) {
                sm.red_top[buf][warp] = wtop;
                sm.red_all[buf][warp] = fmaxf(wtop, ltop);
                sm.red_s[buf][warp] = s;
            }
            __syncthreads();                              // and every thread is done with the bitmap
            float m = sm.red_all[buf][0];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) m = fmaxf(m, sm.red_all[buf][i]);
            if (listed) {
                unsigned long long sum = 0ull;
                walk([&](int l) { sum += __float2ull_rn(Scaled<T>::exp((listed_value(l, true) - m) * c1) * kFixed); });
                sum = redux_sum(sum);                     // a lane's: at most 32 columns, each at most 2^48
                if (lane == 0) sm.listed_sum[buf][warp] = sum;
                if (n_listed > (uint32_t)kListed) __syncthreads();   // the walk reads every word of the bitmap
                clear();
                if (tid == 0) sm.n_listed[buf] = 0u;
                __syncthreads();                          // the sum is whole, the tables are clear
            }
            if (tid == kThreads - 1) {                    // of a warp that short lists leave idle
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) t += sm.red_s[buf][i] * Scaled<T>::exp((sm.red_top[buf][i] - m) * c1);
                if (listed) {
                    unsigned long long sum = 0ull;
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) sum += sm.listed_sum[buf][i];
                    t += __ull2float_rn(sum) * (1.f / kFixed);
                }
                uint32_t flags = !w.ok || t != t ? kPartNanInf : 0u;
                if (w.ignored) flags |= kPartIgnored;
                if (target >= 0) flags |= kPartHasTarget;
                // the record's maximum is after the temperature: what its rounding takes away (exact in the
                // FMA) goes into the sum
                float mz = kNegBig;
                if (t != 0.f) {
                    mz = fmaxf(m * w.inv_t, kNegBig);
                    const float d = fmaf(m, w.inv_t, -mz);
                    t *= fabsf(d) < 1e-3f ? fmaf(d, fmaf(0.5f, d, 1.f), 1.f) : expf(d);
                }
                // ... and the target's is kept beside it: without either a common offset of the logits would reach the
                // logprob (10^4 at a temperature of 0.7: 5e-4)
                const float v = target >= 0 ? sm.target_v[buf] : 0.f, zt = v * w.inv_t;
                const float rest = fabsf(zt) < pinf() ? fmaf(v, w.inv_t, -zt) : 0.f;
                a.parts[(int64_t)slice * a.N + r] = PartialRec{mz, kNegBig, (double)t, 0.0, (double)rest, zt, flags};
            }
        } else {
            T *orow = static_cast<T *>(a.out) + w.out_off + s0;
            const uint32_t ophase = (uint32_t)(uintptr_t)orow & 15u;
            const bool constant = w.nan_row || w.ignored;
            auto pass = [&](auto whole) {                 // whole: a tile of full width
                constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
                for (int k = 0; k < kVecs; ++k) {
                    const int o = k * kThreads + tid, n = kWhole ? kVec : width - o * kVec;
                    uint4 u = make_uint4(0u, 0u, 0u, 0u);
                    if (n > 0) {
                        u = staged_vec<kAligned>(buffer, phase, o);
                        float v[kVec];
                        Elem<T>::unpack(u, v);
#pragma unroll
                        for (int i = 0; i < kVec; i += 2) {
                            float2 d = make_float2(v[i], v[i + 1]);
                            if constexpr (kOp == kLogpBwd) {
                                d = __fadd2_rn(__ffma2_rn(d, f2(w.inv_t), f2(-w.m)), f2(-w.log_s));
                                if (Scaled<T>::kUnit != 1.f) d = __fmul2_rn(d, f2(Scaled<T>::kUnit));
                                d = scaled_exp2<T>(d);
                            }
                            d = __fmul2_rn(d, f2(w.scale));
                            v[i] = d.x;
                            v[i + 1] = d.y;
                        }
                        if (constant) {
#pragma unroll
                            for (int i = 0; i < kVec; ++i) v[i] = w.nan_row ? qnan() : 0.f;
                        }
                        u = Elem<T>::pack(v);
                        const uint32_t on = allow.b[k / 4] >> (8 * (k % 4)) & L::kAll;
                        if (on != L::kAll && !constant)
                            u = keep_vec<T>(u, on, kOp == kProcFwd ? minus_inf_bits<T>() : 0u, sm.keep_words);
                    }
                    store_vec<kAligned>(orow + o * kVec, u, n, ophase);
                }
            };
            if (kAligned && width == kSlice) pass(std::bool_constant<kAligned>());
            else pass(std::false_type());
            __syncthreads();                              // the vector pass's stores come before the walk's
            if (listed) {
                walk([&](int l) {
                    const float staged = to_float(st[l]);
                    float f, v = ruled(l, kOp == kProcBwd ? to_float(xrow[l]) : staged, f, true);
                    if (kOp == kProcFwd) {
                        v *= w.inv_t;
                    } else if (kOp == kProcBwd) {
                        v = staged * (f * w.inv_t);
                    } else {
                        const float d = fmaf(v, w.inv_t, -w.m) - w.log_s;
                        v = (l == target ? expm1f(d) : Scaled<T>::exp(d * Scaled<T>::kUnit)) * (f * w.scale);
                    }
                    if (!allowed(l)) v = kOp == kProcFwd ? -pinf() : 0.f;
                    if (!constant) Elem<T>::store1(orow + l, v);
                });
                if (n_listed > (uint32_t)kListed) __syncthreads();   // the walk reads every word of the bitmap
                clear();
                if (tid == 0) sm.n_listed[buf] = 0u;
                __syncthreads();                          // the tables are clear
            }
        }
        if (row_ends) {
            ++r;
            w = next_w;
            fresh = true;
        }
        allow = next_allow;
        staged = next_staged;
        slice = next_slice;
    }
}

// Joins a row's records (slice-major) into its logprob and vp_rowstat: one warp per
// row, lanes over the slices, the records' order fixed. What vp_logprobs_merge
// does for shards, with the exponentials of the sums in fp32 (the sums are fp32
// sums): its fp64 ones took 25 us for 8192 rows of 10 slices.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(kJoinWarps * 32)
rules_join_kernel(const PartialRec *__restrict__ parts, int K, int64_t N, float *__restrict__ logp,
                  RowStat *__restrict__ stats, int32_t *__restrict__ err) {
    pdl_enter<true>();
    const int64_t r = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= N) return;   // warp-uniform
    float M = kNegBig, zt = 0.f, rest = 0.f;             // the target's ruled logit: zt + rest
    uint32_t flags = 0u;
    for (int k = lane; k < K; k += 32) {
        const PartialRec &p = parts[(int64_t)k * N + r];
        M = fmaxf(M, p.m);
        flags |= p.flags;
        if (p.flags & kPartHasTarget) {
            zt = p.z_t;
            rest = (float)p.W;
        }
    }
    M = warp_max(M);
    const unsigned holders = __ballot_sync(0xffffffffu, (flags & kPartHasTarget) != 0u);   // one slice at most
    flags = __reduce_or_sync(0xffffffffu, flags);
    const int holder = holders ? __ffs(holders) - 1 : 0;
    zt = __shfl_sync(0xffffffffu, zt, holder);
    rest = __shfl_sync(0xffffffffu, rest, holder);
    double S = 0.0;
    for (int k = lane; k < K; k += 32) {
        const PartialRec &p = parts[(int64_t)k * N + r];
        if (p.S > 0.0) S += (double)(expf(p.m - M) * (float)p.S);   // a slice without weight is skipped
    }
    S = warp_sum(S);
    if (lane != 0) return;
    uint32_t rf = kRowSharded;
    if (flags & kPartNanInf) { S = (double)qnan(); rf |= kRowNanInf; }
    else if (S == 0.0) rf |= kRowEmpty;
    const double log_s = log(S);
    const bool ignored = (flags & kPartIgnored) != 0u, lost = !ignored && !holders;
    if (lost) rf |= kRowBadTarget;
    store_rowstat(stats + r, M, log_s, 0.0, rf);
    if (lost && err) atomicOr(err, VP_ERRBIT_TARGET_);
    const bool bad = lost || (rf & (kRowNanInf | kRowEmpty)) != 0u;
    logp[r] = ignored ? 0.f : bad ? qnan() : (float)(((double)zt - (double)M) + (double)rest - log_s);
}

// slices (records) of the ruled logprobs' forward
int64_t rule_slices(int64_t V) {
    constexpr int64_t width = Tile<float, kRuleThreads>::kWidth;
    return (V + width - 1) / width;
}

template <typename T, int kOp, int kN, bool kAligned>
static cudaError_t launch_rules_t(RuleKernelArgs k, cudaStream_t stream) {
    using L = Tile<T, kN>;
    // resident CTAs per SM for each choice of tables and capacity of row_ids, asked once per device
    static std::atomic<int> resident[64][6][5];
    k.n_slices = ((int64_t)k.V + L::kWidth - 1) / L::kWidth;
    // fewer than 2^15 ids in all (a training batch's sequences): no id occurs more often
    k.narrow = k.q.n_ids < 0x8000;
    const int tables = (k.tabled ? k.narrow ? 1 : 2 : 0) + (k.q.bias_spans ? 3 : 0);
    // Room for the average row's ids: long histories take shared memory from other CTAs, but going
    // through 16384 ids for every slice takes longer than the slice.
    int step = 0;
    if (k.tabled)
        while (step < 4 && (int64_t)(kRowIdsLeast << step) * k.N < k.q.n_ids) ++step;
    static_assert(kRowIdsLeast << 4 == kRowIdsMost, "five capacities");
    k.row_ids = k.tabled ? kRowIdsLeast << step : 0;
    auto bytes = [](int tables, int ids) {
        return (int)sizeof(RuleSmem<L>) + (tables % 3) * L::kWidth * 2 + (tables / 3) * L::kWidth * 4 + ids * 2;
    };
    const int smem = bytes(tables, k.row_ids);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> &known = resident[dev & 63][tables][step];
    int per_sm = known.load(std::memory_order_relaxed);
    if (!per_sm) {
        const auto kernel = rules_kernel<T, kOp, kN, kAligned>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(5, kRowIdsMost));
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, L::kThreads, smem);
        if (e != cudaSuccess) return e;
        per_sm = per_sm < 1 ? 1 : per_sm;
        known.store(per_sm, std::memory_order_relaxed);
    }
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const int64_t total = k.N * k.n_slices, most = (int64_t)sms * per_sm;
    return launch_pdl(rules_kernel<T, kOp, kN, kAligned>, dim3((unsigned)(total < most ? total : most)), dim3(L::kThreads),
                      (size_t)smem, stream, k);
}

// Whether every row of a matrix begins at a 16-byte boundary.
template <typename T>
static bool rows_aligned(const void *p, int64_t N, const Rows &rows) {
    const auto whole = [](int64_t stride) { return stride * (int64_t)sizeof(T) % 16 == 0; };
    return (uintptr_t)p % 16 == 0 && (rows.R < 2 || N < 2 || whole(rows.s_i)) && (rows.R >= N || whole(rows.s_o));
}

// Rows that all begin at 16-byte boundaries have a kernel of their own, without the
// shifts and with no check per vector in tiles of full width (us, 8192 x 75968 bf16
// with 1000 ids a row, forward / backward of the ruled logprobs: 591 / 513; when the
// kernel was split, with 16 ids of a thread on their way, 584 / 562 against 605 / 628
// with a check per vector and 648 / 632 with the choice made tile by tile in one
// kernel). 1024 x 75968 and 75967, the latter off the boundaries: 89 / 77 and 108 / 143.
template <typename T, int kOp>
static cudaError_t launch_rules_t(const RuleKernelArgs &k, cudaStream_t stream) {
    const Rows packed{1, k.V, 0};
    const bool aligned = rows_aligned<T>(kOp == kProcBwd ? k.dy : k.x, k.N, kOp == kProcBwd ? packed : k.xrows) &&
                         (kOp == kLogpFwd || rows_aligned<T>(k.out, k.N, kOp == kProcFwd ? k.orows : packed));
    if constexpr (kOp == kProcFwd) {
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (k.tabled && k.N <= sms / rule_slices(k.V))
            return aligned ? launch_rules_t<T, kOp, kRuleThreadsFew, true>(k, stream)
                           : launch_rules_t<T, kOp, kRuleThreadsFew, false>(k, stream);
        if (k.tabled && k.q.n_ids > Tile<T, kRuleThreads>::kWidth * k.N)
            return aligned ? launch_rules_t<T, kOp, kRuleThreadsLong, true>(k, stream)
                           : launch_rules_t<T, kOp, kRuleThreadsLong, false>(k, stream);
    }
    return aligned ? launch_rules_t<T, kOp, kRuleThreads, true>(k, stream)
                   : launch_rules_t<T, kOp, kRuleThreads, false>(k, stream);
}

template <int kOp>
static cudaError_t launch_rules(const RuleArgs &a) {
    RuleKernelArgs k{a.x, a.dy, a.out, a.N, 0, a.vocab_start, (int)a.V, Rows{a.R, a.s_o, a.s_i},
                     Rows{a.R, a.out_s_o, a.out_s_i}, a.rules, a.targets, static_cast<const RowStat *>(a.stats), a.g,
                     static_cast<PartialRec *>(a.parts), a.err,
                     a.rules.spans && (a.rules.repetition || a.rules.frequency || a.rules.presence), 0, false};
    return a.bf16 ? launch_rules_t<__nv_bfloat16, kOp>(k, a.stream) : launch_rules_t<float, kOp>(k, a.stream);
}

cudaError_t read_rules_fault(uint32_t *value, bool clear) { return read_tu_fault(value, clear); }

cudaError_t launch_process_fwd(const RuleArgs &a) { return launch_rules<kProcFwd>(a); }
cudaError_t launch_process_bwd(const RuleArgs &a) { return launch_rules<kProcBwd>(a); }
cudaError_t launch_processed_logprobs_bwd(const RuleArgs &a) { return launch_rules<kLogpBwd>(a); }

cudaError_t launch_processed_logprobs_fwd(const RuleArgs &a, float *logp, void *stats) {
    cudaError_t e = launch_rules<kLogpFwd>(a);
    if (e != cudaSuccess) return e;
    return launch_pdl(rules_join_kernel, dim3((unsigned)((a.N + kJoinWarps - 1) / kJoinWarps)), dim3(kJoinWarps * 32), 0,
                      a.stream, static_cast<const PartialRec *>(a.parts), (int)rule_slices(a.V), a.N, logp,
                      static_cast<RowStat *>(stats), a.err);
}

}  // namespace vp
