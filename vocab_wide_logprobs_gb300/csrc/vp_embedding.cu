// vp_embedding.cu -- rows of the vocabulary's table for token ids, and the table's gradient.
//
//   forward   y_n = s W[id_n]; an id < 0 (padding) or of another shard gives a zero row
//   backward  dW[v] = s sum_{n: id_n = v} dy_n, or that added to what dW holds
//
// Forward: a warp for a piece of 32 x 4 vectors of 8 columns of one row, so that the four
//   loads of a lane are on their way together. Bound: DRAM bytes (8192 rows of 4096, fp32 to bf16: 22 us; rows
//   asked for again come from L2).
// Backward of more than 128 tokens, three or four launches (up to there one: table_grad_few_kernel):
//   1. token_sort_kernel: the tokens of each id behind one another, in the order of their
//      positions. Each CTA owns some of the ids, goes over all N and counts, notes and
//      places its own: no CTA waits for another, no atomic decides an order. From 32768 tokens on
//      token_deal_kernel gives each CTA its own first (8192 ids 7 us, 65536 13, skewed ones 8 and 18).
//   2. table_grad_kernel: windows of the sorted tokens, each summed in fp32 in order; a
//      run of one id that lies in a window is written at once, the ends of runs that cross
//      windows are left as fp32 partial sums. More CTAs write zeros to rows no token asks for.
//   3. table_join_kernel: the partial sums of such runs, in the order of the windows, as
//      double-floats.
//   Every sum's order follows from the ids alone, so the result is the same every time, and
//   an id that takes half of a batch is spread over as many CTAs as it has windows.
//   Bound: DRAM bytes of dy and dW: 8192 tokens, 75968 x 4096 bf16: 8 + 95 + 7 us, of which the middle one moves
//   689 MB (7.2 TB/s); 65536 tokens, 75968 x 1024 fp32: 20 + 73 + 6, 445 MB (6.1 TB/s).
#include <algorithm>
#include <atomic>

#include "vp_device.cuh"
#include "vp_launch.h"

namespace vp {

constexpr int kEmbVec = 8;   // columns of a vector: 16 bytes of bf16, 32 of fp32

// Columns c .. c + 7 (vectors) or c, c + step, .. (single elements) of a row, as they lie in memory: a caller starts
// several rows' loads before it takes the first one's values.
template <typename T, bool kVector>
struct Row8 {
    uint4 u[kVector ? kEmbVec * sizeof(T) / 16 : 1];
    T e[kVector ? 1 : kEmbVec];
    __device__ __forceinline__ void load(const T *row, int c, int step, int D) {
        if constexpr (kVector) {
#pragma unroll
            for (int h = 0; h < (int)(kEmbVec * sizeof(T) / 16); ++h) u[h] = __ldg(reinterpret_cast<const uint4 *>(row + c + h * Elem<T>::kVec));
        } else {
#pragma unroll
            for (int k = 0; k < kEmbVec; ++k) e[k] = c + k * step < D ? __ldg(row + c + k * step) : T(0.f);
        }
    }
    // what a kernel also writes: not through the read-only path
    __device__ __forceinline__ void load_own(const T *row, int c, int step, int D) {
        if constexpr (kVector) {
#pragma unroll
            for (int h = 0; h < (int)(kEmbVec * sizeof(T) / 16); ++h)
                u[h] = *reinterpret_cast<const uint4 *>(row + c + h * Elem<T>::kVec);
        } else {
#pragma unroll
            for (int k = 0; k < kEmbVec; ++k) e[k] = c + k * step < D ? row[c + k * step] : T(0.f);
        }
    }
    __device__ __forceinline__ void get(float (&v)[kEmbVec]) const {
        if constexpr (kVector) {
#pragma unroll
            for (int h = 0; h < (int)(kEmbVec * sizeof(T) / 16); ++h) Elem<T>::unpack(u[h], v + h * Elem<T>::kVec);
        } else {
#pragma unroll
            for (int k = 0; k < kEmbVec; ++k) v[k] = (float)e[k];
        }
    }
};

template <typename T, bool kVector>
__device__ __forceinline__ void store8(T *row, int c, int step, int D, const float (&v)[kEmbVec]) {
    if constexpr (kVector) {
        if constexpr (sizeof(T) == 2) {
            stg_stream(row + c, Elem<T>::pack(v));
        } else {
            stg_stream(row + c, Elem<float>::pack(v));
            stg_stream(row + c + 4, Elem<float>::pack(v + 4));
        }
    } else {
#pragma unroll
        for (int e = 0; e < kEmbVec; ++e)
            if (c + e * step < D) Elem<T>::store1(row + c + e * step, v[e]);
    }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
constexpr int kEmbThreads = 128, kEmbUnroll = 4;
constexpr int kEmbPiece = 32 * kEmbUnroll * kEmbVec;   // columns of a warp's piece

template <typename TI, typename TO, bool kVector>
__global__ void __launch_bounds__(kEmbThreads)
embedding_fwd_kernel(const TI *__restrict__ table, int64_t pitch, int V, int D, const int64_t *__restrict__ ids,
                     int64_t vocab_start, float scale, bool sharded, TO *__restrict__ out, int32_t *__restrict__ err,
                     int pieces, int64_t total) {
    pdl_enter<true>();   // no global access before this
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kEmbThreads / 32);
    for (int64_t i = (int64_t)blockIdx.x * (kEmbThreads / 32) + (threadIdx.x >> 5); i < total; i += step) {
        const int64_t n = i / pieces;
        const int c0 = (int)(i - n * pieces) * kEmbPiece;
        const int64_t id = ids[n], local = id - vocab_start;
        const bool here = id >= 0 && local >= 0 && local < V;
        const bool wrong = id >= 0 && !here && !sharded;
        if (wrong && err && c0 == 0 && lane == 0) atomicOr(err, VP_ERRBIT_TARGET_);
        const TI *row = table + (here ? local : 0) * pitch;
        TO *dst = out + n * (int64_t)D;
        Row8<TI, kVector> u[kEmbUnroll];
#pragma unroll
        for (int k = 0; k < kEmbUnroll; ++k) {
            const int c = kVector ? c0 + (k * 32 + lane) * kEmbVec : c0 + k * 32 * kEmbVec + lane;
            if (here && c < D) u[k].load(row, c, 32, D);
        }
#pragma unroll
        for (int k = 0; k < kEmbUnroll; ++k) {
            const int c = kVector ? c0 + (k * 32 + lane) * kEmbVec : c0 + k * 32 * kEmbVec + lane;
            if (c >= D) continue;
            float v[kEmbVec];
            u[k].get(v);
#pragma unroll
            for (int e = 0; e < kEmbVec; ++e) v[e] = here ? v[e] * scale : wrong ? qnan() : 0.f;
            store8<TO, kVector>(dst, c, 32, D, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBins = 1024;               // ids of a CTA's range: a thread each in the scan, 128 KB of counters

constexpr int kSortAhead = 4;                    // ids of a lane on their way at once
constexpr int kStash = 768;                      // own tokens that a warp remembers for the second pass, at most
constexpr uint32_t kStashSpan = 1u << 22;        // and how long a stretch they can come from (10 + 22 bits)
static_assert(kSortMaxBins <= 1 << 10, "a bin's 10 bits");
static_assert(kSortWarps * (kSortMaxBins + kStash) * 4 <= 226 * 1024, "shared memory");

// Quotients by d >= 2 of x < 2^31 without a division: the high half of x m, shifted by s, where 2^s < d <= 2^(s + 1)
// and m = ceil(2^(32 + s) / d) < 2^32. m d exceeds 2^(32 + s) by less than d, so x m / 2^(32 + s) exceeds x / d by less than
// x / 2^(32 + s) <= 1 / 2^(s + 1) <= 1 / d: too little to reach the next whole number.
struct FastDiv {
    uint32_t m, s, d;
    explicit FastDiv(uint32_t by) : s(0), d(by) {
        while (((uint64_t)2 << s) < by) ++s;
        m = (uint32_t)((((uint64_t)1 << (32 + s)) + by - 1) / by);
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const { return __umulhi(x, m) >> s; }
};

constexpr int kTurnBits = 2, kTurnRows = 1 << kTurnBits;
// Where an id's row is: the CTA that owns it and its place there, or no row of the shard. The rows go to the CTAs by
// turns, kTurnRows neighbours at once.
struct Deal {
    int64_t vocab_start;
    int V;
    FastDiv by_ctas;
    __device__ __forceinline__ bool at(int64_t id, uint32_t &cta, uint32_t &bin) const {
        const int64_t local = id - vocab_start;
        const uint32_t group = (uint32_t)local >> kTurnBits, turn = by_ctas.div(group);
        cta = group - turn * by_ctas.d;
        bin = turn << kTurnBits | ((uint32_t)local & (kTurnRows - 1));
        return id >= 0 && (uint32_t)(local >> 32) == 0u && (uint32_t)local < (uint32_t)V;   // no high half, a low one below V
    }
};

// The warps' counters of thread t's column t < width, made offsets: of the column within all that `base` is in front of,
// and within it warp by warp. begin and n: the column's own. By whole CTAs.
struct Column {
    uint32_t begin, n;
};
__device__ __forceinline__ Column column_offsets(uint32_t *counts, int width, uint32_t base, uint32_t *s_sum) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t c[kSortWarps], n = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) c[w] = tid < width ? counts[w * width + tid] : 0u;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n += c[w];
    uint32_t scan = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d) scan += o;
    }
    if (lane == 31) s_sum[warp] = scan;
    __syncthreads();
    const uint32_t sums = s_sum[lane];
    base += __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0u) + scan - n;
    const Column of{base, n};
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        if (tid < width) counts[w * width + tid] = base;
        base += c[w];
    }
    __syncthreads();
    return of;
}

// Many tokens: the ids of each slice of them dealt to their CTAs first, so that a CTA of the sort goes over its own
// tokens alone. dealt[slice][..]: the slice's tokens by CTA and in order, their place at their CTA << 10 | their place in
// the slice; starts[cta][slice]: where those of a CTA begin there (and, one further, end).
constexpr int kSlice = kSortThreads;
static_assert(kSlice <= 1 << 10, "a place's 10 bits");
constexpr int kDealMaxCtas = kSortThreads;
__global__ void __launch_bounds__(kSortThreads)
token_deal_kernel(const int64_t *__restrict__ ids, int64_t N, Deal deal, bool sharded, uint32_t *__restrict__ dealt,
                  uint16_t *__restrict__ starts, int32_t *__restrict__ err) {
    extern __shared__ uint32_t counts[];         // [kSortWarps][CTAs of the sort]
    __shared__ uint32_t s_sum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, width = (int)deal.by_ctas.d;
    for (int i = tid; i < kSortWarps * width; i += kSortThreads) counts[i] = 0u;
    __syncthreads();
    pdl_enter<true>();
    const int64_t slice = blockIdx.x, p = slice * kSlice + tid;
    const int64_t id = p < N ? ids[p] : -1;
    uint32_t cta, bin;
    const bool here = deal.at(id, cta, bin);
    if (id >= 0 && !here && !sharded && err) atomicOr(err, VP_ERRBIT_TARGET_);
    const uint32_t peers = __match_any_sync(0xffffffffu, here ? cta : 0xffffffffu);
    const uint32_t before = __popc(peers & ((1u << lane) - 1u));
    if (here && before == 0) counts[warp * width + cta] = __popc(peers);
    __syncthreads();
    const Column of = column_offsets(counts, width, 0u, s_sum);
    if (tid < width) starts[(int64_t)tid * gridDim.x + slice] = (uint16_t)of.begin;
    if (tid == width - 1) starts[(int64_t)width * gridDim.x + slice] = (uint16_t)(of.begin + of.n);
    if (here) dealt[slice * kSlice + counts[warp * width + cta] + before] = bin << 10 | (uint32_t)tid;
}

// The tokens of the shard, those of one row behind one another in the order of their positions: rows[k] and
// positions[k] of the k-th, spans[v].x .. spans[v].y - 1 those of row v. Rows are dealt to the CTAs, since frequent tokens
// often have neighbouring ids (with a range of ids for a CTA, that of the 500 lowest had 43 % of the 65536 tokens of a
// skewed batch and took 46 us); neighbours written together are a little faster than one row at a time (1 to 3 % of the call).
// A warp places the tokens of the stretch of positions that it has counted, so its counters, made offsets (row by
// row, and warp by warp within a row), put them behind those of earlier stretches. While it counts it notes its own
// tokens; only a warp with more of them than it can note reads its stretch again.
// kDealt: of what token_deal_kernel has left. Otherwise every CTA goes over all ids, and the loop's instructions are what
// that costs (13 of 19 us of 65536 tokens).
template <bool kDealt>
__global__ void __launch_bounds__(kSortThreads)
token_sort_kernel(const int64_t *__restrict__ ids, int64_t N, Deal deal, bool sharded, int bins, int stash_size,
                  const uint32_t *__restrict__ dealt, const uint16_t *__restrict__ starts, int *__restrict__ n_tokens,
                  int2 *__restrict__ spans, int *__restrict__ rows, int *__restrict__ positions,
                  int32_t *__restrict__ err) {
    extern __shared__ uint32_t counts[];         // [kSortWarps][bins], then [kSortWarps][stash_size]
    __shared__ uint32_t s_sum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kSortWarps * bins; i += kSortThreads) counts[i] = 0u;
    __syncthreads();
    pdl_enter<false>();
    const int64_t unit = kDealt ? kSlice : 32, units = (N + unit - 1) / unit;
    const int64_t stretch = (units + kSortWarps - 1) / kSortWarps * unit;
    const int64_t p0 = min(N, warp * stretch), p1 = min(N, p0 + stretch);
    uint32_t *mine = counts + warp * bins, *stash = counts + kSortWarps * bins + warp * stash_size;
    const uint32_t n_stash = (uint32_t)stash_size;
    uint32_t below = 0, noted = 0;               // noted: the same in every lane
    bool wrong = false;
    auto row_of = [](uint32_t bin) {             // of this CTA's
        return ((int64_t)(bin >> kTurnBits) * gridDim.x + blockIdx.x) * kTurnRows + (bin & (kTurnRows - 1));
    };

    // each(which lanes, bin, place in the stretch) of the warp's own tokens in the order of their positions, by whole
    // warps; loads are on their way while those before are looked at
    auto scan_stretch = [&](auto each, bool count) {
        if constexpr (kDealt) {
            const int s0 = (int)min(units, warp * (stretch / kSlice)), s1 = (int)min(units, s0 + stretch / kSlice);
            for (int sb = s0; sb < s1; sb += 32) {
                const int64_t at = (int64_t)blockIdx.x * units + sb + lane;
                const uint32_t begin = sb + lane < s1 ? starts[at] : 0u, end = sb + lane < s1 ? starts[at + units] : 0u;
                if (count) below += begin;
                for (int j = 0; j < min(32, s1 - sb); j += kSortAhead) {
                    uint32_t from[kSortAhead], len[kSortAhead], x[kSortAhead];
#pragma unroll
                    for (int k = 0; k < kSortAhead; ++k) {
                        from[k] = __shfl_sync(0xffffffffu, begin, j + k);
                        len[k] = __shfl_sync(0xffffffffu, end, j + k) - from[k];
                        x[k] = lane < len[k] ? dealt[(int64_t)(sb + j + k) * kSlice + from[k] + lane] : 0u;
                    }
#pragma unroll
                    for (int k = 0; k < kSortAhead; ++k) {
                        const uint32_t *rest = dealt + (int64_t)(sb + j + k) * kSlice + from[k] + lane;
                        const int at_slice = (sb + j + k - s0) * kSlice;
                        auto look = [&](uint32_t i, uint32_t y) {
                            if (i >= len[k]) return;
                            each(__ballot_sync(0xffffffffu, i + lane < len[k]), y >> 10, at_slice + (int)(y & (kSlice - 1)));
                        };
                        look(0, x[k]);
                        for (uint32_t i = 32; i < len[k]; i += 32 * kSortAhead) {      // a frequent token's CTA
                            uint32_t y[kSortAhead];
#pragma unroll
                            for (int m = 0; m < kSortAhead; ++m) y[m] = i + m * 32 + lane < len[k] ? rest[i + m * 32] : 0u;
#pragma unroll
                            for (int m = 0; m < kSortAhead; ++m) look(i + m * 32, y[m]);
                        }
                    }
                }
            }
        } else {
            const int n = (int)(p1 - p0);
            const int64_t *from = ids + p0 + lane;
            int64_t id[kSortAhead], next[kSortAhead];
            auto load = [&](int q) {
#pragma unroll
                for (int k = 0; k < kSortAhead; ++k) next[k] = q + k * 32 + lane < n ? from[q + k * 32] : -1;
            };
            load(0);
            for (int q = 0; q < n; q += 32 * kSortAhead) {
#pragma unroll
                for (int k = 0; k < kSortAhead; ++k) id[k] = next[k];
                load(q + 32 * kSortAhead);
#pragma unroll
                for (int k = 0; k < kSortAhead; ++k) {
                    uint32_t cta, bin;
                    const bool here = deal.at(id[k], cta, bin);
                    if (count) {
                        if (blockIdx.x == 0) wrong |= id[k] >= 0 && !here;
                        if (here && cta < blockIdx.x) ++below;
                    }
                    const uint32_t own = __ballot_sync(0xffffffffu, here && cta == blockIdx.x);
                    if (own) each(own, bin, q + k * 32 + lane);
                }
            }
        }
    };
    scan_stretch(
        [&](uint32_t own, uint32_t bin, int at_stretch) {
            if (own >> lane & 1) {
                atomicAdd(&mine[bin], 1u);
                const uint32_t at = noted + __popc(own & ((1u << lane) - 1u));
                if (at < n_stash) stash[at] = bin << 22 | ((uint32_t)at_stretch & (kStashSpan - 1));
            }
            noted += __popc(own);
        },
        true);
    if (wrong && !sharded && err) atomicOr(err, VP_ERRBIT_TARGET_);
    below = __reduce_add_sync(0xffffffffu, below);
    if (lane == 0) s_sum[warp] = below;
    __syncthreads();
    const uint32_t base = __reduce_add_sync(0xffffffffu, s_sum[lane]);
    __syncthreads();

    // thread t has the CTA's t-th row
    const Column of = column_offsets(counts, bins, base, s_sum);
    if (tid == bins - 1 && blockIdx.x == gridDim.x - 1) *n_tokens = (int)(of.begin + of.n);
    if (tid < bins && row_of((uint32_t)tid) < deal.V) spans[row_of((uint32_t)tid)] = make_int2((int)of.begin, (int)(of.begin + of.n));

    auto place = [&](uint32_t own, uint32_t bin, int at_stretch) {
        const bool is_own = own >> lane & 1;
        const uint32_t peers = __match_any_sync(0xffffffffu, is_own ? bin : 0xffffffffu);
        const uint32_t before = __popc(peers & ((1u << lane) - 1u));
        uint32_t at = 0;
        if (is_own) at = mine[bin] + before;
        __syncwarp();
        if (is_own) {
            if (before == 0) mine[bin] += __popc(peers);
            rows[at] = (int)row_of(bin);
            positions[at] = (int)p0 + at_stretch;
        }
        __syncwarp();
    };
    if (noted <= n_stash && stretch <= (int64_t)kStashSpan) {
        for (uint32_t i = 0; i < noted; i += 32) {
            const uint32_t e = i + lane < noted ? stash[i + lane] : 0u;
            place(__ballot_sync(0xffffffffu, i + lane < noted), e >> 22, (int)(e & (kStashSpan - 1)));
        }
    } else {
        scan_stretch(place, false);
    }
}

constexpr int kGradThreads = 256;
constexpr int kGradMaxWindow = 64;
constexpr int kFillBytes = 256, kFillMaxRows = 1024;     // zeros of a thread, and rows of a CTA, at most

struct TableGrad {
    int64_t N;
    int V, D, window, n_windows, col_blocks;
    Rows dy_rows;
    float scale;
    const int *n_tokens;        // of this shard
    const int2 *spans;          // [V]: where a row's tokens begin and end
    const int *rows, *positions;
    int4 *runs;                 // [n_windows]: the run that goes on behind a window: its row, the window that it begins
                                // in and the one that it ends in (0: none goes on)
    float *partial;             // [n_windows][2][D]: what belongs to a run begun in an earlier window, and
                                // what belongs to one that goes on in later ones
};

// A table row's new value from the sum and, where it is added to, from what the row held.
template <typename TO, bool kVector, bool kAdd>
__device__ __forceinline__ void finish8(TO *dst, int c, int step, int D, float scale, float (&v)[kEmbVec],
                                        const Row8<TO, kVector> &old) {
    float o[kEmbVec];
    if (kAdd) old.get(o);
#pragma unroll
    for (int e = 0; e < kEmbVec; ++e) v[e] = kAdd ? fmaf(v[e], scale, o[e]) : v[e] * scale;
    store8<TO, kVector>(dst, c, step, D, v);
}

template <typename T>
__device__ __forceinline__ void zero_fill(T *p, int64_t n, int tid, int nt) {
    const int64_t head = min(n, (int64_t)((16 - (uintptr_t)p % 16) % 16 / sizeof(T)));
    constexpr int kPer = 16 / sizeof(T);
    const int64_t vecs = (n - head) / kPer, tail = head + vecs * kPer;
    if (tid < head) Elem<T>::store1(p + tid, 0.f);
    for (int64_t i = tid; i < vecs; i += nt) stg_stream(p + head + i * kPer, make_uint4(0, 0, 0, 0));
    if (tid < n - tail) Elem<T>::store1(p + tail + tid, 0.f);
}
// Zeros to the rows v0 .. v1 of a table that no token asks for, runs of them at once.
template <typename T>
__device__ __forceinline__ void fill_unasked(T *dW, int D, int64_t v0, int64_t v1, const bool *asked, int tid, int nt) {
    for (int64_t v = v0; v < v1;) {
        int64_t end = v;
        while (end < v1 && !asked[end - v0]) ++end;
        zero_fill(dW + v * D, (end - v) * D, tid, nt);
        v = end + 1;
    }
}

template <typename TI, typename TO, bool kVector, bool kAdd>
__global__ void __launch_bounds__(kGradThreads)
table_grad_kernel(const TI *__restrict__ dy, const TableGrad a, TO *__restrict__ dW, int fill_rows) {
    __shared__ int s_row[kGradMaxWindow];
    __shared__ int64_t s_off[kGradMaxWindow];
    __shared__ bool s_asked[kFillMaxRows];
    const int tid = threadIdx.x, nt = blockDim.x;
    pdl_enter<false>();
    const int total = *a.n_tokens;
    const int64_t b = blockIdx.x;
    const int64_t n_sum = (int64_t)a.n_windows * a.col_blocks;
    if (b >= n_sum) {
        // zeros for rows that no token asks for
        if constexpr (!kAdd) {
            const int64_t v0 = (b - n_sum) * fill_rows, v1 = min((int64_t)a.V, v0 + fill_rows);
            for (int64_t v = v0 + tid; v < v1; v += nt) s_asked[v - v0] = a.spans[v].x != a.spans[v].y;
            __syncthreads();
            fill_unasked(dW, a.D, v0, v1, s_asked, tid, nt);
        }
        return;
    }
    const int w = (int)(b / a.col_blocks), cb = (int)(b - (int64_t)w * a.col_blocks);
    const int64_t k0 = (int64_t)w * a.window, k1 = min((int64_t)total, k0 + a.window);
    if (cb == 0 && tid == 0) {
        int4 run = make_int4(0, 0, 0, 0);
        if (k1 < total && k0 < k1) {
            const int row = a.rows[k1 - 1];
            const int2 span = a.spans[row];
            if (span.y > k1) run = make_int4(row, span.x / a.window, (span.y - 1) / a.window, 0);
        }
        a.runs[w] = run;
    }
    if (k0 >= k1) return;
    for (int i = tid; i < (int)(k1 - k0); i += nt) {
        s_row[i] = a.rows[k0 + i];
        s_off[i] = a.dy_rows.off(a.positions[k0 + i]);
    }
    __syncthreads();
    const int c = cb * nt * kEmbVec + (kVector ? tid * kEmbVec : tid), step = nt;
    if (c >= a.D) return;
    const int count = (int)(k1 - k0);
    float sum[kEmbVec] = {};
    constexpr int kAhead = 4;
    for (int i = 0; i < count; i += kAhead) {
        // the tokens' rows (the last one again behind the window), and with them what the rows of the table hold
        // whose runs end here
        Row8<TI, kVector> u[kAhead];
        Row8<TO, kVector> old[kAdd ? kAhead : 1];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) u[k].load(dy + s_off[min(i + k, count - 1)], c, step, a.D);
        if constexpr (kAdd) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int at = min(i + k, count - 1);
                if (at + 1 == count || s_row[at + 1] != s_row[at])
                    old[k].load_own(dW + s_row[at] * (int64_t)a.D, c, step, a.D);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i + k >= count) break;
            float v[kEmbVec];
            u[k].get(v);
#pragma unroll
            for (int e = 0; e < kEmbVec; ++e) sum[e] += v[e];
            const int row = s_row[i + k];
            if (i + k + 1 < count && s_row[i + k + 1] == row) continue;
            // the run ends here, or the window does
            const int2 span = a.spans[row];
            const bool begun_before = span.x < k0, goes_on = span.y > k1;
            if (begun_before || goes_on) {
                float *part = a.partial + ((int64_t)w * 2 + (begun_before ? 0 : 1)) * a.D;
                if (kVector) {
                    *reinterpret_cast<float4 *>(part + c) = make_float4(sum[0], sum[1], sum[2], sum[3]);
                    *reinterpret_cast<float4 *>(part + c + 4) = make_float4(sum[4], sum[5], sum[6], sum[7]);
                } else {
                    store8<float, false>(part, c, step, a.D, sum);
                }
            } else {
                finish8<TO, kVector, kAdd>(dW + row * (int64_t)a.D, c, step, a.D, a.scale, sum, old[kAdd ? k : 0]);
            }
#pragma unroll
            for (int e = 0; e < kEmbVec; ++e) sum[e] = 0.f;
        }
    }
}

// Few tokens: one launch. A CTA for each token and 8 columns of each of 64 lanes (32 of a narrow table): where no
// earlier token has the same id, its groups of lanes sum the rows of all that have it, group j those of the j-th,
// (j + groups)-th, .. of them, and their sums are added in order. (One group of 256 lanes took half a microsecond
// a token, since the compiler has no more than two of its rows on their way: 40 us for 55 tokens of one id among 256.)
// More CTAs write zeros, as above.
// Up to how many: of 128 tokens added to 50000 x 2048 bf16, 9 us with ids of their own, 13 with a third of them
// alike, 23 with all alike, against 17 to 18 in three launches; of 256, 11, 19 and 40.
constexpr int kFewTokens = 128;
template <typename TI, typename TO, bool kVector, bool kAdd>
__global__ void __launch_bounds__(kGradThreads)
table_grad_few_kernel(const TI *__restrict__ dy, const TableGrad a, const int64_t *__restrict__ ids, int64_t vocab_start,
                      bool sharded, TO *__restrict__ dW, int32_t *__restrict__ err, int fill_rows, int lanes) {
    __shared__ int s_row[kFewTokens];
    __shared__ int64_t s_off[kFewTokens];        // of the tokens that have the CTA's id, in order
    __shared__ uint32_t s_same[kFewTokens / 32];
    __shared__ bool s_asked[kFillMaxRows];
    __shared__ float s_sum[kGradThreads][kEmbVec + 1];
    const int tid = threadIdx.x, nt = kGradThreads, N = (int)a.N;
    pdl_enter<false>();
    for (int i = tid; i < N; i += nt) {
        const int64_t id = ids[i], local = id - vocab_start;
        const bool here = id >= 0 && local >= 0 && local < a.V;
        s_row[i] = here ? (int)local : -1;
        if (id >= 0 && !here && !sharded && err && blockIdx.x == 0) atomicOr(err, VP_ERRBIT_TARGET_);
    }
    const int64_t b = blockIdx.x, n_sum = (int64_t)N * a.col_blocks;
    if (b >= n_sum) {
        if constexpr (!kAdd) {
            const int64_t v0 = (b - n_sum) * fill_rows, v1 = min((int64_t)a.V, v0 + fill_rows);
            for (int v = tid; v < (int)(v1 - v0); v += nt) s_asked[v] = false;
            __syncthreads();
            for (int i = tid; i < N; i += nt)
                if (s_row[i] >= v0 && s_row[i] < v1) s_asked[s_row[i] - v0] = true;
            __syncthreads();
            fill_unasked(dW, a.D, v0, v1, s_asked, tid, nt);
        }
        return;
    }
    __syncthreads();
    const int i = (int)(b / a.col_blocks), cb = (int)(b - (int64_t)i * a.col_blocks);
    const int row = s_row[i];
    if (row < 0) return;
    // which tokens have this id, a bit each
    for (int k = tid; k < (N + 31) / 32 * 32; k += nt) {         // by whole warps: nt is a multiple of 32
        const uint32_t same = __ballot_sync(0xffffffffu, k < N && s_row[k] == row);
        if (k % 32 == 0) s_same[k / 32] = same;
    }
    __syncthreads();
    int before = 0, count = 0;
    for (int w = 0; w < (N + 31) / 32; ++w) {
        if (w < i / 32) before += __popc(s_same[w]);
        count += __popc(s_same[w]);
    }
    if (before || s_same[i / 32] & ((1u << (i & 31)) - 1u)) return;   // an earlier token's CTA has it
    for (int k = tid; k < N; k += nt)
        if (s_row[k] == row) {
            int at = __popc(s_same[k / 32] & ((1u << (k & 31)) - 1u));
            for (int w = 0; w < k / 32; ++w) at += __popc(s_same[w]);
            s_off[at] = a.dy_rows.off(k);
        }
    __syncthreads();
    const int group = tid / lanes, lane = tid % lanes, groups = nt / lanes;
    const int c = cb * lanes * kEmbVec + (kVector ? lane * kEmbVec : lane), step = lanes;
    const bool inside = c < a.D;
    float sum[kEmbVec] = {};
    Row8<TO, kVector> old;
    TO *dst = dW + row * (int64_t)a.D;
    if (kAdd && inside && group == 0) old.load_own(dst, c, step, a.D);
    constexpr int kAhead = 4;
    for (int k0 = group; inside && k0 < count; k0 += groups * kAhead) {
        Row8<TI, kVector> u[kAhead];                             // the last row again behind the run
#pragma unroll
        for (int k = 0; k < kAhead; ++k) u[k].load(dy + s_off[min(k0 + k * groups, count - 1)], c, step, a.D);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            float v[kEmbVec];
            u[k].get(v);
#pragma unroll
            for (int e = 0; e < kEmbVec; ++e) sum[e] += k0 + k * groups < count ? v[e] : 0.f;
        }
    }
    if (group > 0)
#pragma unroll
        for (int e = 0; e < kEmbVec; ++e) s_sum[tid][e] = sum[e];
    __syncthreads();
    if (group > 0 || !inside) return;
    for (int g = 1; g < min(groups, count); ++g)
#pragma unroll
        for (int e = 0; e < kEmbVec; ++e) sum[e] += s_sum[g * lanes + lane][e];
    finish8<TO, kVector, kAdd>(dst, c, step, a.D, a.scale, sum, old);
}

// The partial sums of a run, by groups of threads, four columns each: group j adds those of its windows w + j,
// w + j + groups, .., then a thread for each column adds the groups'. A run of a few windows is added by the CTAs of its first one, in four
// groups, 512 columns a CTA; a longer one by those of all its windows, in sixteen, 128 columns a CTA (0.3 of 65536
// tokens alike: 10 us; 42 where one window's CTAs added the run).
constexpr int kJoinThreads = 512, kJoinAhead = 4, kJoinFew = 8;
template <typename TO, bool kVector, bool kAdd, int kGroups>
__device__ __forceinline__ void join_run(const TableGrad &a, TO *__restrict__ dW, const int4 &run, int slice, int slices,
                                         DF (*s_sum)[4]) {
    constexpr int kLanes = kJoinThreads / kGroups;
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, w = run.y, until = run.z;
    for (int c0 = slice * kLanes * 4; c0 < a.D; c0 += slices * kLanes * 4) {
        const int c = kVector ? c0 + 4 * lane : c0 + lane, step = kVector ? 1 : kLanes;
        DF sum[4] = {};
        for (int u0 = w + group; u0 <= until; u0 += kGroups * kJoinAhead) {
            float v[kJoinAhead][4];
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const int u = u0 + k * kGroups;
                const float *part = a.partial + ((int64_t)u * 2 + (u == w ? 1 : 0)) * a.D + c;
                if (kVector) {
                    const float4 f = u <= until && c < a.D ? *reinterpret_cast<const float4 *>(part) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[k][0] = f.x; v[k][1] = f.y; v[k][2] = f.z; v[k][3] = f.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[k][e] = u <= until && c + e * step < a.D ? part[e * step] : 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) df_add(sum[e], v[k][e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s_sum[threadIdx.x][e] = sum[e];
        __syncthreads();
        // a thread for each column now
        const int t = threadIdx.x, l = kVector ? t / 4 : t % kLanes, e = kVector ? t % 4 : t / kLanes;
        if (t < kLanes * 4 && c0 + t < a.D) {
            DF total = s_sum[l][e];
#pragma unroll
            for (int j = 1; j < kGroups; ++j) df_add(total, s_sum[j * kLanes + l][e]);
            TO *dst = dW + run.x * (int64_t)a.D + c0 + t;
            // an infinite sum's low part is NaN (inf - inf), a finite one's is finite
            const float s = isfinite(total.hi) ? total.hi + total.lo : total.hi;
            Elem<TO>::store1(dst, kAdd ? fmaf(s, a.scale, (float)*dst) : s * a.scale);
        }
        __syncthreads();
    }
}
template <typename TO, bool kVector, bool kAdd>
__global__ void __launch_bounds__(kJoinThreads, 3)
table_join_kernel(const TableGrad a, TO *__restrict__ dW) {
    __shared__ DF s_sum[kJoinThreads][4];
    pdl_enter<false>();
    const int w = blockIdx.x;
    const int4 run = a.runs[w];
    if (run.z - run.y >= kJoinFew)
        join_run<TO, kVector, kAdd, 16>(a, dW, run, (w - run.y) * gridDim.y + blockIdx.y, (run.z - run.y) * gridDim.y, s_sum);
    else if (run.z && w == run.y)
        join_run<TO, kVector, kAdd, 4>(a, dW, run, blockIdx.y, gridDim.y, s_sum);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
namespace {

int sm_count() {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 1;
}

// Tokens of a window: as many as leave three CTAs for each of GB300's 152 SMs and some (the workspace's size, asked for on
// any host, follows from it), since a window costs up to two partial rows (20000 x 1024
// bf16 into 151936 rows, 64 tokens and 313 CTAs: 81 us, 32 and 625: 72; 8192 x 4096, 32 and 512: 109, 8 and 2048: 111 to 117).
int grad_window(int64_t N, int64_t D) {
    const int64_t col_blocks = (D + kGradThreads * kEmbVec - 1) / (kGradThreads * kEmbVec);
    int w = 8;
    while (w < kGradMaxWindow && N * col_blocks >= (int64_t)w * 2 * 500) w *= 2;
    return w;
}

// From how many tokens on they are dealt first (75968 rows; even ids to 0.3 of one id): of 262144, 10 us for that and 11 to 47
// for the sort, against 58 to 145 by the sort alone; of 65536, 6 and 7 to 15 against 19 to 25; of 16384, 6 and 7 to 10 against
// 9 to 11.
constexpr int64_t kDealTokens = 32768;

struct GradLayout {
    size_t n_tokens, rows, positions, runs, dealt, starts, partial, total;
};
GradLayout grad_layout(int64_t N, int64_t V, int64_t D) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const int64_t windows = (N + grad_window(N, D) - 1) / grad_window(N, D);
    GradLayout L;                                // the rows' spans first
    L.n_tokens = up((size_t)V * sizeof(int2));
    L.rows = L.n_tokens + 256;
    L.positions = L.rows + up((size_t)N * 4);
    L.runs = L.positions + up((size_t)N * 4);
    L.dealt = L.runs + up((size_t)windows * sizeof(int4));
    const size_t slices = N >= kDealTokens ? (size_t)(N + kSlice - 1) / kSlice : 0;
    L.starts = L.dealt + slices * kSlice * 4;
    L.partial = L.starts + up(slices * (kDealMaxCtas + 1) * 2);
    L.total = L.partial + (size_t)windows * 2 * D * 4;
    return L;
}

template <typename TI, typename TO>
cudaError_t embedding_fwd(const EmbeddingArgs &a) {
    const TI *x = static_cast<const TI *>(a.x);
    TO *out = static_cast<TO *>(a.out);
    const bool vector = a.D % kEmbVec == 0 && (uintptr_t)x % 16 == 0 && (uintptr_t)out % 16 == 0 &&
                        a.s_i * sizeof(TI) % 16 == 0;
    const int pieces = (int)((a.D + kEmbPiece - 1) / kEmbPiece);
    const int64_t total = a.N * pieces, ctas = (total + kEmbThreads / 32 - 1) / (kEmbThreads / 32);
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)(ctas < 2147483647 ? ctas : 2147483647)), dim3(kEmbThreads), 0, a.stream,
                          x, a.s_i, (int)a.V, (int)a.D, a.ids, a.vocab_start, a.scale, a.sharded, out, a.err, pieces, total);
    };
    return vector ? go(embedding_fwd_kernel<TI, TO, true>) : go(embedding_fwd_kernel<TI, TO, false>);
}

template <typename TI, typename TO>
cudaError_t embedding_bwd(const EmbeddingArgs &a) {
    const TI *dy = static_cast<const TI *>(a.x);
    TO *dW = static_cast<TO *>(a.out);
    const bool vector = a.D % kEmbVec == 0 && (uintptr_t)dy % 16 == 0 && (uintptr_t)dW % 16 == 0 &&
                        a.s_i * sizeof(TI) % 16 == 0 && a.s_o * sizeof(TI) % 16 == 0;
    const int threads = (int)(a.D >= kGradThreads * kEmbVec ? kGradThreads : ((a.D + kEmbVec - 1) / kEmbVec + 31) / 32 * 32);
    const int64_t row_bytes = a.D * (int64_t)sizeof(TO);
    const int fill_rows = (int)std::clamp<int64_t>((int64_t)kFillBytes * threads / row_bytes, 1, kFillMaxRows);
    const int64_t fill_ctas = a.accumulate ? 0 : (a.V + fill_rows - 1) / fill_rows;
    TableGrad g{};
    g.N = a.N;
    g.V = (int)a.V;
    g.D = (int)a.D;
    g.col_blocks = (int)((a.D + threads * kEmbVec - 1) / (threads * kEmbVec));
    g.dy_rows = Rows{a.R, a.s_o, a.s_i};
    g.scale = a.scale;
    if (a.N <= kFewTokens) {
        const int lanes = a.D > 32 * kEmbVec ? 64 : 32;
        g.col_blocks = (int)((a.D + lanes * kEmbVec - 1) / (lanes * kEmbVec));
        const int rows = (int)std::clamp<int64_t>((int64_t)kFillBytes * kGradThreads / row_bytes, 1, kFillMaxRows);
        const int64_t ctas = a.N * g.col_blocks + (a.accumulate ? 0 : (a.V + rows - 1) / rows);
        if (ctas > 2147483647) return cudaErrorInvalidValue;
        auto few = [&](auto kernel) {
            return launch_pdl(kernel, dim3((unsigned)ctas), dim3(kGradThreads), 0, a.stream, dy, g, a.ids, a.vocab_start,
                              a.sharded, dW, a.err, rows, lanes);
        };
        return vector ? (a.accumulate ? few(table_grad_few_kernel<TI, TO, true, true>) : few(table_grad_few_kernel<TI, TO, true, false>))
                      : (a.accumulate ? few(table_grad_few_kernel<TI, TO, false, true>) : few(table_grad_few_kernel<TI, TO, false, false>));
    }
    const GradLayout L = grad_layout(a.N, a.V, a.D);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    int2 *spans = reinterpret_cast<int2 *>(ws);
    int *n_tokens = reinterpret_cast<int *>(ws + L.n_tokens), *rows = reinterpret_cast<int *>(ws + L.rows),
        *positions = reinterpret_cast<int *>(ws + L.positions);
    // rows of a CTA in the sort: the table over the SMs, within what the counters have room for
    const int sms = sm_count();
    int64_t bins = (a.V + sms - 1) / sms;
    bins = (bins + kTurnRows - 1) / kTurnRows * kTurnRows;
    bins = bins < 32 ? 32 : bins > kSortMaxBins ? kSortMaxBins : bins;
    // the counters' room, asked for once on each device
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t e;
    if (!(attr_done.load() & (1ull << (dev & 63)))) {
        constexpr int most = kSortWarps * (kSortMaxBins + kStash) * 4;
        if ((e = cudaFuncSetAttribute(token_sort_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(token_sort_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(token_deal_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kSortWarps * kDealMaxCtas * 4)) != cudaSuccess)
            return e;
        attr_done.fetch_or(1ull << (dev & 63));
    }
    const unsigned sort_ctas = (unsigned)std::max<int64_t>(2, (a.V + bins - 1) / bins);
    const bool deal_first = a.N >= kDealTokens && sort_ctas <= kDealMaxCtas;
    // a warp notes its whole stretch, where that is short
    const int64_t unit = deal_first ? kSlice : 32, stretch = ((a.N + unit - 1) / unit + kSortWarps - 1) / kSortWarps * unit;
    const int stash = (int)std::min<int64_t>(kStash, stretch);
    const size_t smem = (size_t)kSortWarps * (bins + stash) * 4;
    const Deal deal{a.vocab_start, (int)a.V, FastDiv(sort_ctas)};
    uint32_t *dealt = reinterpret_cast<uint32_t *>(ws + L.dealt);
    uint16_t *starts = reinterpret_cast<uint16_t *>(ws + L.starts);
    auto sort = [&](auto kernel) {
        return launch_pdl(kernel, dim3(sort_ctas), dim3(kSortThreads), smem, a.stream, a.ids, a.N, deal, a.sharded, (int)bins,
                          stash, dealt, starts, n_tokens, spans, rows, positions, a.err);
    };
    if (deal_first) {
        e = launch_pdl(token_deal_kernel, dim3((unsigned)((a.N + kSlice - 1) / kSlice)), dim3(kSortThreads),
                       (size_t)kSortWarps * sort_ctas * 4, a.stream, a.ids, a.N, deal, a.sharded, dealt, starts, a.err);
        if (e == cudaSuccess) e = sort(token_sort_kernel<true>);
    } else {
        e = sort(token_sort_kernel<false>);
    }
    if (e != cudaSuccess) return e;

    g.window = grad_window(a.N, a.D);
    g.n_windows = (int)((a.N + g.window - 1) / g.window);
    g.n_tokens = n_tokens;
    g.spans = spans;
    g.rows = rows;
    g.positions = positions;
    g.runs = reinterpret_cast<int4 *>(ws + L.runs);
    g.partial = reinterpret_cast<float *>(ws + L.partial);
    const int64_t ctas = (int64_t)g.n_windows * g.col_blocks + fill_ctas;
    if (ctas > 2147483647) return cudaErrorInvalidValue;
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)ctas), dim3(threads), 0, a.stream, dy, g, dW, fill_rows);
    };
    e = vector ? (a.accumulate ? go(table_grad_kernel<TI, TO, true, true>) : go(table_grad_kernel<TI, TO, true, false>))
               : (a.accumulate ? go(table_grad_kernel<TI, TO, false, true>) : go(table_grad_kernel<TI, TO, false, false>));
    if (e != cudaSuccess || g.n_windows < 2) return e;
    const int64_t blocks = (a.D + kJoinThreads - 1) / kJoinThreads;
    auto join = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)(g.n_windows - 1), (unsigned)std::min<int64_t>(blocks, 65535)),
                          dim3(kJoinThreads), 0, a.stream, g, dW);
    };
    return vector ? (a.accumulate ? join(table_join_kernel<TO, true, true>) : join(table_join_kernel<TO, true, false>))
                  : (a.accumulate ? join(table_join_kernel<TO, false, true>) : join(table_join_kernel<TO, false, false>));
}

}  // namespace

size_t embedding_bwd_workspace_bytes(int64_t N, int64_t V, int64_t D) {
    return N <= kFewTokens ? 0 : grad_layout(N, V, D).total;
}

cudaError_t launch_embedding_fwd(const EmbeddingArgs &a) {
    if (a.x_bf16)
        return a.out_bf16 ? embedding_fwd<__nv_bfloat16, __nv_bfloat16>(a) : embedding_fwd<__nv_bfloat16, float>(a);
    return a.out_bf16 ? embedding_fwd<float, __nv_bfloat16>(a) : embedding_fwd<float, float>(a);
}

cudaError_t launch_embedding_bwd(const EmbeddingArgs &a) {
    if (a.x_bf16)
        return a.out_bf16 ? embedding_bwd<__nv_bfloat16, __nv_bfloat16>(a) : embedding_bwd<__nv_bfloat16, float>(a);
    return a.out_bf16 ? embedding_bwd<float, __nv_bfloat16>(a) : embedding_bwd<float, float>(a);
}

}  // namespace vp
