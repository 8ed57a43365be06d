// vp_mxfp4.cu -- MXFP4 matrices (OCP Microscaling formats: E2M1 elements, one
// E8M0 scale for each block of 32): quantisation, the values back, and the
// head's product of two such matrices on the block-scaled tensor cores.
//
// Layout of a matrix [rows, D]: include/vp.h. The scale tiles (512 bytes for
// 128 rows x 4 blocks, 16 bytes for each row % 32) are what tcgen05.cp
// 32x128b.warpx4 puts into tensor memory for the block-scaled MMA, so a stage's
// scales are one contiguous bulk copy.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "vp_device.cuh"
#include "vp_gemm_host.cuh"
#include "vp_launch.h"
#include "vp_pair.cuh"
#include "vp_umma.cuh"
#include "vp_waits.h"

namespace vp {

// ---------------------------------------------------------------------------
// Quantisation
// ---------------------------------------------------------------------------
// Eight values to eight E2M1 codes (round to nearest even, saturated), column i
// in bits 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Byte offset of the scale word (4 blocks) of row r in column tile kt of n_kt.
__device__ __forceinline__ int64_t scale_word(int64_t r, int kt, int n_kt) {
    return ((r >> 7) * n_kt + kt) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

constexpr int kQThreads = 128, kQWarps = kQThreads / 32;
constexpr int kQLane = 16;                   // columns of a lane
constexpr int kQChunk = 32 * kQLane;         // columns that a warp reads at once
constexpr int kQChunks = 2;                  // chunks of a warp, all on their way before the first is used

constexpr int kDChunk = 256, kDChunks = 4;   // ... of the way back, whose lanes take 8 columns

// Which rows and chunks a warp works on: groups of chunks, row by row.
struct QuantGrid {
    int64_t rows, groups;                    // groups per row
    unsigned blocks;
    bool ok;
};
static QuantGrid quant_grid(int64_t rows, int64_t D, int of_warp) {
    const int64_t groups = (D + of_warp - 1) / of_warp;
    const int64_t blocks = (rows * groups + kQWarps - 1) / kQWarps;
    return {rows, groups, (unsigned)blocks, blocks <= 0x7fffffff};
}
// (row, first chunk) of this warp; row >= rows: nothing to do
__device__ __forceinline__ int64_t quant_place(int64_t groups, int chunks, int &chunk0) {
    const int64_t unit = (int64_t)blockIdx.x * kQWarps + (threadIdx.x >> 5);
    const int64_t r = unit >> 32 || groups >> 32 ? unit / groups : (int64_t)((uint32_t)unit / (uint32_t)groups);
    chunk0 = (int)(unit - r * groups) * chunks;
    return r;
}

// 32 bytes at an address that is a multiple of 32, read once.
__device__ __forceinline__ void ldg_stream32(const void *p, uint4 &a, uint4 &b) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
}

// The largest |x| of a lane's columns as the bits of an fp32 value; NaN wins.
__device__ __forceinline__ uint32_t lane_amax(const uint4 (&u)[2]) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(u);
    __nv_bfloat162 m = __habs2(p[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(p[i]));
    const uint32_t w = *reinterpret_cast<const uint32_t *>(&m);
    return max(w << 16, w & 0xffff0000u);                  // bit patterns without sign order like the values
}
__device__ __forceinline__ uint32_t lane_amax(const uint4 (&u)[4]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
}

// A lane takes 16 consecutive columns of a chunk: a block is two lanes, its
// maximum a shuffle away. The scale comes from the maximum's exponent bits (E:
// the scale byte is E - 2, at least 0), so x / scale is exact. Rows N .. the next
// multiple of 128 only get their zero scale bytes. Bound by memory: one read of x,
// 17/32 of a byte written per element; 75968 x 4096 bf16 take 124 us, 95% of what a
// copy of as many bytes would. Lanes of 8 columns with 16-byte loads took 157 us (four
// lanes to a block: eight shuffles for 16 columns, here three), a grid that stays on
// the SMs and reads ahead 165.
template <typename T>
__global__ void __launch_bounds__(kQThreads)
mxfp4_quantize_kernel(const T *__restrict__ x, Rows rows, int64_t N, int64_t n_rows, int64_t groups, int D,
                      uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    pdl_enter<true>();
    constexpr int kVecs = kQLane / Elem<T>::kVec;
    const int lane = threadIdx.x & 31, n_kt = (D + 127) / 128;
    int chunk0;
    const int64_t r = quant_place(groups, kQChunks, chunk0);
    if (r >= n_rows) return;
    const T *row = x + (r < N ? (rows.R >= N ? r * rows.s_i : rows.off(r)) : 0);   // no division for one stride
    const uint32_t off = (uint32_t)(uintptr_t)row & 31u;
    uint4 u[kQChunks][kVecs];
#pragma unroll
    for (int k = 0; k < kQChunks; ++k) {
        const int c = (chunk0 + k) * kQChunk + lane * kQLane;   // D is a multiple of 64: whole or absent
#pragma unroll
        for (int i = 0; i < kVecs; ++i) u[k][i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < N && c < D) {
            if (off == 0u) {
#pragma unroll
                for (int i = 0; i < kVecs; i += 2) ldg_stream32(row + c + i * Elem<T>::kVec, u[k][i], u[k][i + 1]);
            } else if (off == 16u) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) u[k][i] = ldg_stream(reinterpret_cast<const uint4 *>(row + c) + i);
            } else {
                T *e = reinterpret_cast<T *>(u[k]);
#pragma unroll
                for (int i = 0; i < kQLane; ++i) e[i] = row[c + i];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kQChunks; ++k) {
        const int chunk = chunk0 + k, c = chunk * kQChunk + lane * kQLane;
        if (chunk * kQChunk >= D) break;                   // uniform in the warp
        const bool valid = r < N && c < D;
        uint32_t amax = lane_amax(u[k]);
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const uint32_t e = amax >> 23;
        const uint32_t byte = e == 255u ? 255u : e > 2u ? e - 2u : 0u;
        if (valid) {
            const float2 inv = f2(__uint_as_float((254u - min(byte, 253u)) << 23));   // 2^(127 - byte)
            uint32_t code[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
#pragma unroll
                for (int i = 0; i < kVecs / 2; ++i) Elem<T>::unpack(u[k][h * (kVecs / 2) + i], v + i * Elem<T>::kVec);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 p = __fmul2_rn(make_float2(v[i], v[i + 1]), inv);
                    v[i] = p.x;
                    v[i + 1] = p.y;
                }
                code[h] = byte == 255u ? 0u : e2m1x8(v);
            }
            *reinterpret_cast<uint2 *>(codes + r * (D / 2) + (c >> 1)) = make_uint2(code[0], code[1]);
        }
        uint32_t word = valid ? byte << (8 * ((lane >> 1) & 3)) : 0u;
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        const int kt = chunk * (kQChunk / 128) + (lane >> 3);
        if ((lane & 7) == 0 && kt < n_kt) *reinterpret_cast<uint32_t *>(scales + scale_word(r, kt, n_kt)) = word;
    }
}

cudaError_t launch_mxfp4_quantize(const Mxfp4QuantArgs &a) {
    const QuantGrid g = quant_grid((a.N + 127) / 128 * 128, a.D, kQChunk * kQChunks);
    if (!g.ok) return cudaErrorInvalidValue;
    const Rows rows{a.R, a.s_o, a.s_i};
    uint8_t *codes = static_cast<uint8_t *>(a.codes), *scales = static_cast<uint8_t *>(a.scales);
    if (a.bf16)
        return launch_pdl(mxfp4_quantize_kernel<__nv_bfloat16>, dim3(g.blocks), dim3(kQThreads), 0, a.stream,
                          static_cast<const __nv_bfloat16 *>(a.x), rows, a.N, g.rows, g.groups, (int)a.D, codes, scales);
    return launch_pdl(mxfp4_quantize_kernel<float>, dim3(g.blocks), dim3(kQThreads), 0, a.stream,
                      static_cast<const float *>(a.x), rows, a.N, g.rows, g.groups, (int)a.D, codes, scales);
}

// Eight codes to their values (the hardware's conversion to fp16, exact).
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// 2^(byte - 127), exact in fp32 (a subnormal for byte 0), NaN for byte 255.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return byte == 255u ? qnan() : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

template <typename T>
__global__ void __launch_bounds__(kQThreads)
mxfp4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t N, int64_t groups,
                        int D, T *__restrict__ out) {
    pdl_enter<true>();
    const int lane = threadIdx.x & 31, n_kt = (D + 127) / 128;
    int chunk0;
    const int64_t r = quant_place(groups, kDChunks, chunk0);
    if (r >= N) return;
    uint32_t w[kDChunks], s[kDChunks];
#pragma unroll
    for (int k = 0; k < kDChunks; ++k) {
        const int c = (chunk0 + k) * kDChunk + lane * 8;
        w[k] = s[k] = 0u;
        if (c < D) {
            w[k] = __ldg(reinterpret_cast<const uint32_t *>(codes + r * (D / 2) + (c >> 1)));
            s[k] = __ldg(scales + scale_word(r, c >> 7, n_kt) + ((c >> 5) & 3));
        }
    }
#pragma unroll
    for (int k = 0; k < kDChunks; ++k) {
        const int c = (chunk0 + k) * kDChunk + lane * 8;
        if (c >= D) break;
        float v[8];
        e2m1x8_values(w[k], v);
        const float scale = e8m0_value(s[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= scale;         // exact: at least 2^-128 or 0
        T *p = out + r * (int64_t)D + c;
#pragma unroll
        for (int i = 0; i < 8 / Elem<T>::kVec; ++i)
            stg_stream(reinterpret_cast<uint4 *>(p) + i, Elem<T>::pack(v + i * Elem<T>::kVec));
    }
}

cudaError_t launch_mxfp4_dequantize(const Mxfp4DequantArgs &a) {
    const QuantGrid g = quant_grid(a.N, a.D, kDChunk * kDChunks);
    if (!g.ok) return cudaErrorInvalidValue;
    const uint8_t *codes = static_cast<const uint8_t *>(a.codes), *scales = static_cast<const uint8_t *>(a.scales);
    if (a.bf16)
        return launch_pdl(mxfp4_dequantize_kernel<__nv_bfloat16>, dim3(g.blocks), dim3(kQThreads), 0, a.stream, codes,
                          scales, a.N, g.groups, (int)a.D, static_cast<__nv_bfloat16 *>(a.out));
    return launch_pdl(mxfp4_dequantize_kernel<float>, dim3(g.blocks), dim3(kQThreads), 0, a.stream, codes, scales, a.N,
                      g.groups, (int)a.D, static_cast<float *>(a.out));
}

// ---------------------------------------------------------------------------
// Product: y[n, v] = sum_k x[n, k] w[v, k]
// ---------------------------------------------------------------------------
// The vocabulary runs along the MMA's rows (operand A, the accumulator's lanes)
// and the tokens along its columns (operand B), so that a single token still reads
// the head at full width and a warp's stores of one token are consecutive. K steps
// of 64 (kind::mxf4, one scale for each 32 columns); a stage holds 256 columns:
// 128-byte rows of both operands in the 128-byte swizzle and two scale tiles for
// each 128 rows. One thread copies a stage's scales to tensor memory (tcgen05.cp,
// executed in order with the MMAs that follow it) and issues its MMAs; every stage
// in flight has scale columns of its own, so a copy never meets an MMA that still
// reads them. (Copying a stage ahead of the MMAs measured 4% slower.)
constexpr int kXM = 128;                     // vocabulary rows of a CTA's tile
constexpr int kXK = 256;                     // columns of a stage
constexpr int kXRow = kXK / 2;               // their bytes in a row
constexpr int kXAStage = kXM * kXRow;       // 16 KB
constexpr int kXSStage = 2 * 512;            // scales of 128 rows
constexpr int kXThreads = 192;               // TMA warp, MMA warp, 4 epilogue warps

constexpr int x_stage_bytes(int nt) { return kXAStage + nt * kXRow + 2 * kXSStage; }
constexpr int x_stages(int nt) { return (200 * 1024) / x_stage_bytes(nt) < 10 ? (200 * 1024) / x_stage_bytes(nt) : 10; }
constexpr int x_smem_bytes(int nt) { return x_stages(nt) * x_stage_bytes(nt) + 1024; }
constexpr uint32_t x_tmem_cols(int nt) {     // two accumulators, 8 + 8 scale columns of each stage
    const int n = 2 * nt + 16 * x_stages(nt);
    return n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512;
}

// Instruction descriptor of kind::mxf4: E2M1 operands, both K-major, E8M0 scales.
__host__ __device__ constexpr uint32_t umma_idesc_mxf4(int M, int N) {
    return (1u << 7)                        // A format: E2M1            [7, 10)
           | (1u << 10)                     // B format: E2M1            [10, 12)
           | ((uint32_t)(N >> 3) << 17)     // N / 8                     [17, 23)
           | (1u << 23)                     // scale format: E8M0        [23]
           | ((uint32_t)(M >> 4) << 24);    // M / 16 (M / 128 at bit 27)
}

// ... with the scales of a K step in byte pair `id` (0 or 2) of their columns.
__device__ __forceinline__ uint32_t idesc_scale_id(uint32_t idesc, uint32_t id) {
    return idesc | (id << 4) | (id << 29);   // B's scale id [4, 6), A's [29, 31)
}

__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// A 512-byte scale tile in shared memory, as 32 rows of 16 bytes: no swizzle,
// groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(const void *smem) {
    return (uint64_t)((smem_u32(smem) >> 4) & 0x3FFFu) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// ... to four tensor-memory columns, repeated in the four quarters of the lanes.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// One lane of a converged warp. Tensor-core and copy instructions take their operands
// from the warp's uniform registers; behind elect.sync the compiler knows that one
// lane is active and moves them there directly, behind `lane == 0` it does not (the
// pair's MMAs alone, 8192 tokens at half their width: 360 us against 714).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// The issuing thread works at the latency of its own instructions, and an MMA of the
// pair takes 128 clocks: descriptors are bases plus multiples of 16 bytes (the
// address field holds them without carry: shared memory ends below 2^18), the
// stage is counted and not divided for, and a whole stage's MMAs are unrolled.
struct StageCount {
    uint32_t st = 0, phase = 0;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++st == n) {
            st = 0;
            phase ^= 1;
        }
    }
};

template <int kNT>
struct Mxfp4Bars {
    uint64_t full[x_stages(kNT)], empty[x_stages(kNT)], acc_full[2], acc_empty[2], done;   // done: every MMA
    uint32_t tmem_base;
};

template <int kNT, typename T>
__global__ void __launch_bounds__(kXThreads, 1)
linear_mxfp4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const uint8_t *__restrict__ w_scales, const uint8_t *__restrict__ x_scales, int N, int V, int D,
                    T *__restrict__ y) {
    constexpr int kStages = x_stages(kNT), kStageBytes = x_stage_bytes(kNT);
    constexpr uint32_t kScaleCol = 2 * kNT;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Mxfp4Bars<kNT> bars;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_vb = (V - 1) / kXM + 1, n_tb = (N - 1) / kNT + 1;   // N and V have up to 31 bits
    const int64_t n_tiles = (int64_t)n_vb * n_tb;
    const int n_k = (D + kXK - 1) / kXK, n_kt = (D + 127) / 128;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars.acc_full[b], 1);
            mbar_init(&bars.acc_empty[b], kXThreads - 64);
        }
        mbar_init(&bars.done, 1);
        fence_mbar_init();
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
    }
    if (warp == 1) tmem_alloc(&bars.tmem_base, x_tmem_cols(kNT));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    pdl_enter<false>();

    if (warp == 0) {
        if (elect_one()) {
            const uint64_t pol_w = l2_policy(n_tb > 1 ? 2 : 1), pol_x = l2_policy(2);
            StageCount at;
            uint32_t fills = 0;
            bool ok = true;
            for (int64_t tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
                const int vb = (int)(tile / n_tb), tb = (int)(tile - (int64_t)vb * n_tb);
                for (int kb = 0; kb < n_k; ++kb, at.next(kStages)) {
                    const uint32_t st = at.st;
                    if (fills >= (uint32_t)kStages && !mbar_wait(&bars.empty[st], at.phase ^ 1)) { ok = false; break; }
                    ++fills;
                    uint8_t *a = smem + st * kStageBytes, *b = a + kXAStage, *sa = b + kNT * kXRow, *sb = sa + kXSStage;
                    const uint32_t sbytes = 512u * (uint32_t)min(2, n_kt - 2 * kb);
                    mbar_arrive_expect_tx(&bars.full[st], kXAStage + kNT * kXRow + 2 * sbytes);
                    tma_load_2d_hint(a, &tm_w, kb * kXRow, vb * kXM, &bars.full[st], pol_w);
                    tma_load_2d_hint(b, &tm_x, kb * kXRow, tb * kNT, &bars.full[st], pol_x);
                    bulk_g2s(sa, w_scales + ((int64_t)vb * n_kt + 2 * kb) * 512, sbytes, &bars.full[st], pol_w);
                    bulk_g2s(sb, x_scales + ((int64_t)(tb * kNT / 128) * n_kt + 2 * kb) * 512, sbytes, &bars.full[st],
                             pol_x);
                }
            }
            // every copy lands before the CTA gives up its shared memory, whoever gave up
            for (uint32_t i = 0; i < (uint32_t)kStages; ++i) {
                const LateStage l = late_stage(i, fills, fills, kStages);
                if (l.owed != kOwedNothing && !mbar_wait(&bars.full[i], l.parity)) { ok = false; break; }
            }
            if (!ok) atomicOr(&g_linear_fault, 1u);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = umma_idesc_mxf4(kXM, kNT);
            const uint64_t a0 = umma_desc_sw128(smem), b0 = umma_desc_sw128(smem + kXAStage),
                           sa0 = scale_desc(smem + kXAStage + kNT * kXRow), sb0 = sa0 + (kXSStage >> 4);
            StageCount at;
            bool ok = true;
            uint32_t j = 0;
            for (int64_t tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x, ++j) {
                const uint32_t buf = j & 1, use_b = j >> 1;
                if (use_b > 0 && !mbar_wait(&bars.acc_empty[buf], (use_b - 1) & 1)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem + buf * kNT;
                for (int kb = 0; kb < n_k; ++kb) {
                    if (!mbar_wait(&bars.full[at.st], at.phase)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t to = at.st * (kStageBytes >> 4);
                    const uint64_t a = a0 + to, b = b0 + to, sa = sa0 + to, sb = sb0 + to;
                    const uint32_t sc = tmem + kScaleCol + at.st * 16;
                    tmem_copy_scales(sc, sa);
                    tmem_copy_scales(sc + 8, sb);
                    if (n_kt - 2 * kb > 1) {
                        tmem_copy_scales(sc + 4, sa + 32);
                        tmem_copy_scales(sc + 12, sb + 32);
                    }
                    const int steps = min(kXK, D - kb * kXK) / 64;
#pragma unroll
                    for (int kk = 0; kk < kXK / 64; ++kk)
                        if (kk < steps)
                            umma_mxf4(d, a + 2 * kk, b + 2 * kk, idesc_scale_id(idesc, (kk & 1) * 2), sc + 4 * (kk >> 1),
                                      sc + 8 + 4 * (kk >> 1), (kb | kk) != 0);
                    umma_commit(&bars.empty[at.st]);
                    at.next(kStages);
                }
                if (!ok) break;                          // a part of a tile is no tile
                umma_commit(&bars.acc_full[buf]);
            }
            umma_commit(&bars.done);                     // tensor memory is given back after the last MMA
            if (!mbar_wait(&bars.done, 0)) ok = false;
            if (!ok) atomicOr(&g_linear_fault, 2u);
        }
    } else {
        const int q = warp & 3;
        uint32_t j = 0;
        bool ok = true;
        for (int64_t tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++j) {
            const int vb = (int)(tile / n_tb), tb = (int)(tile - (int64_t)vb * n_tb);
            const uint32_t buf = j & 1;
            if (ok && !mbar_wait(&bars.acc_full[buf], (j >> 1) & 1)) {
                ok = false;
                atomicOr(&g_linear_fault, 4u);
            }
            tc_fence_after();
            if (__all_sync(0xffffffffu, ok)) {
                const int v = vb * kXM + q * 32 + lane;
                const int64_t t0 = (int64_t)tb * kNT;
#pragma unroll 1
                for (int c = 0; c < kNT && t0 + c < N; c += 16) {
                    float acc[16];
                    tmem_ld16(tmem + buf * kNT + c + ((uint32_t)(q * 32) << 16), acc);
                    T *p = y + (t0 + c) * V + v;
                    if (v < V) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (t0 + c + i < N) Elem<T>::store1(p + (int64_t)i * V, acc[i]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&bars.acc_empty[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, x_tmem_cols(kNT));
}

// ---------------------------------------------------------------------------
// The same product on CTA pairs (tcgen05 cta_group::2), for more tokens than a
// single CTA's tile: a pair computes 256 vocabulary rows x 256 tokens. CTA r holds
// rows 128 r .. of the W tile and of the accumulator, tokens 128 r .. of the x tile
// and the scales of its 128 rows and of all 256 tokens. Per 256 columns of K a CTA
// takes 35 KB for 128 x 256 outputs, half of what a 128 x 128 tile does; that tile
// was bound by this traffic (57 bytes a clock and SM).
//   Tensor memory: the scales of six stages take 144 of the 512 columns, so the two
// accumulators overlap in 144 columns. The epilogue reads these columns into
// registers first and lets the next tile's MMAs begin; the other 112 it reads while
// they run.
// ---------------------------------------------------------------------------
constexpr int kYStages = 6;
constexpr int kYT = 256;                                  // tokens of a tile
constexpr int kYBStage = kYT / 2 * kXRow;                 // 16 KB
constexpr int kYStageBytes = kXAStage + kYBStage + 3 * kXSStage;
constexpr int kYSmemBytes = kYStages * kYStageBytes + 1024;
constexpr uint32_t kYScaleCols = 8 + 16;                  // of a stage: two scale tiles of W, four of x
constexpr uint32_t kYScaleCol = 512 - kYStages * kYScaleCols;
constexpr uint32_t kYAcc1 = kYScaleCol - kYT;             // the second accumulator's first column
constexpr int kYOverlap = kYT - (int)kYAcc1;
static_assert(kYAcc1 == 112 && kYOverlap == 144, "the epilogue's reads are written for these");

struct PairMxfp4Bars {
    uint64_t full[kYStages], empty[kYStages], acc_full[2], shared_free, done;
    uint32_t tmem_base, fills, gave_up;
};

__device__ __forceinline__ void umma_mxf4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// In both CTAs, from the same place of each one's shared memory.
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kXThreads, 1)
linear_mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_xs, int N, int V,
                         int D, T *__restrict__ y) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ PairMxfp4Bars bars;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int n_vp = (V - 1) / (2 * kXM) + 1, n_tb = (N - 1) / kYT + 1;   // N and V have up to 31 bits
    const int64_t n_tiles = (int64_t)n_vp * n_tb, pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    const int n_k = (D + kXK - 1) / kXK, n_kt = (D + 127) / 128;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kYStages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
        }
        mbar_init(&bars.acc_full[0], 1);
        mbar_init(&bars.acc_full[1], 1);
        mbar_init(&bars.shared_free, 2 * (kXThreads - 64));   // the epilogue threads of both CTAs
        mbar_init(&bars.done, 1);
        bars.gave_up = 0u;
        fence_mbar_init();
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_ws);
        prefetch_tensormap(&tm_xs);
    }
    if (warp == 1) tmem_alloc_pair(&bars.tmem_base, 512);
    tc_fence_before();
    cluster_sync();                                      // barriers and tensor memory ready in both CTAs
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    pdl_enter<false>();

    if (warp == 0) {
        // ---------------- TMA producer (both CTAs; all bytes count on the leader's barrier) ----------------
        if (elect_one()) {
            const uint64_t keep = l2_policy(2);
            StageCount at;
            uint32_t fills = 0;
            bool ok = true;
            for (int64_t tile = pair; tile < n_tiles && ok; tile += n_pairs) {
                const int vp = (int)(tile / n_tb), tb = (int)(tile - (int64_t)vp * n_tb);
                const int wb = 2 * vp + (int)rank;
                for (int kb = 0; kb < n_k; ++kb, at.next(kYStages)) {
                    const uint32_t st = at.st;
                    if (fills >= kYStages && !mbar_wait_cluster(&bars.empty[st], at.phase ^ 1)) { ok = false; break; }
                    ++fills;
                    uint8_t *a = smem + st * kYStageBytes, *b = a + kXAStage, *sa = b + kYBStage, *sb = sa + kXSStage;
                    const uint32_t fb = cluster_addr(&bars.full[st], 0);
                    if (rank == 0) mbar_arrive_expect_tx(&bars.full[st], 2 * kYStageBytes);
                    tma_load_2d_pair(a, &tm_w, kb * kXRow, wb * kXM, fb, keep);
                    tma_load_2d_pair(b, &tm_x, kb * kXRow, tb * kYT + (int)rank * kXM, fb, keep);
                    tma_load_2d_pair(sa, &tm_ws, kb * (kXSStage / 4), wb, fb, keep);
                    tma_load_2d_pair(sb, &tm_xs, kb * (kXSStage / 4), 2 * tb, fb, keep);
                    tma_load_2d_pair(sb + kXSStage, &tm_xs, kb * (kXSStage / 4), 2 * tb + 1, fb, keep);
                }
            }
            bars.fills = fills;
            if (!ok || !pair_ring_used<kYStages>(bars, fills)) pair_gives_up(bars, 1u);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader only) ----------------
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = umma_idesc_mxf4(2 * kXM, kYT);
            const uint64_t a0 = umma_desc_sw128(smem), b0 = umma_desc_sw128(smem + kXAStage),
                           sa0 = scale_desc(smem + kXAStage + kYBStage), sb0 = sa0 + (kXSStage >> 4);
            StageCount at;
            bool ok = true;
            uint32_t j = 0;
            for (int64_t tile = pair; tile < n_tiles && ok; tile += n_pairs, ++j) {
                // the columns shared with the tile before it are read (and all of the one before that)
                if (j > 0 && !mbar_wait_cluster(&bars.shared_free, (j - 1) & 1)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem + (j & 1 ? kYAcc1 : 0u);
                for (int kb = 0; kb < n_k; ++kb) {
                    if (!mbar_wait(&bars.full[at.st], at.phase)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t to = at.st * (kYStageBytes >> 4);
                    const uint64_t a = a0 + to, b = b0 + to, sa = sa0 + to, sb = sb0 + to, sb1 = sb + (kXSStage >> 4);
                    const uint32_t sc = tmem + kYScaleCol + at.st * kYScaleCols;
                    tmem_copy_scales_pair(sc, sa);
                    tmem_copy_scales_pair(sc + 8, sb);
                    tmem_copy_scales_pair(sc + 12, sb1);
                    if (n_kt - 2 * kb > 1) {
                        tmem_copy_scales_pair(sc + 4, sa + 32);
                        tmem_copy_scales_pair(sc + 16, sb + 32);
                        tmem_copy_scales_pair(sc + 20, sb1 + 32);
                    }
                    const int steps = min(kXK, D - kb * kXK) / 64;
#pragma unroll
                    for (int kk = 0; kk < kXK / 64; ++kk)
                        if (kk < steps)
                            umma_mxf4_pair(d, a + 2 * kk, b + 2 * kk, idesc_scale_id(idesc, (kk & 1) * 2),
                                           sc + 4 * (kk >> 1), sc + 8 + 8 * (kk >> 1), (kb | kk) != 0);
                    umma_commit_pair(&bars.empty[at.st]);
                    at.next(kYStages);
                }
                if (!ok) break;                          // a part of a tile is no tile
                umma_commit_pair(&bars.acc_full[j & 1]);
            }
            umma_commit_pair_here(&bars.done);           // tensor memory is given back after the last MMA
            if (!mbar_wait(&bars.done, 0)) ok = false;
            if (!ok) pair_gives_up(bars, 2u);
        }
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        const int q = warp & 3;
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        uint32_t j = 0;
        bool ok = true;
        for (int64_t tile = pair; tile < n_tiles; tile += n_pairs, ++j) {
            const int vp = (int)(tile / n_tb), tb = (int)(tile - (int64_t)vp * n_tb);
            const int64_t t0 = (int64_t)tb * kYT, v = (int64_t)(2 * vp + (int)rank) * kXM + q * 32 + lane;
            if (ok && !mbar_wait_cluster(&bars.acc_full[j & 1], (j >> 1) & 1)) {
                ok = false;
                pair_gives_up(bars, 4u);
            }
            tc_fence_after();
            const bool all = __all_sync(0xffffffffu, ok);
            // tokens t0 + c .. of the values acc[0 .. n)
            auto store = [&](int c, const float *acc, auto count) {
                constexpr int n = decltype(count)::value;
                T *p = y + (t0 + c) * V + v;
                if (v < V) {
                    if (t0 + c + n <= N) {
#pragma unroll
                        for (int i = 0; i < n; ++i) Elem<T>::store1(p + (int64_t)i * V, acc[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < n; ++i)
                            if (t0 + c + i < N) Elem<T>::store1(p + (int64_t)i * V, acc[i]);
                    }
                }
            };
            // columns shared with the other accumulator: the first one's last, the second one's first
            const int c0 = j & 1 ? 0 : (int)kYAcc1;
            const uint32_t acc0 = tmem + (j & 1 ? kYAcc1 : 0u) + lanes;
            uint32_t r[kYOverlap];
            if (all) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32_issue(acc0 + c0 + 32 * k, reinterpret_cast<uint32_t(&)[32]>(r[32 * k]));
                tmem_ld16(acc0 + c0 + 128, reinterpret_cast<float *>(r + 128));   // waits for all
            }
            tc_fence_before();
            mbar_arrive_cluster(cluster_addr(&bars.shared_free, 0));
            if (all) store(c0, reinterpret_cast<const float *>(r), std::integral_constant<int, kYOverlap>());
            const int c1 = j & 1 ? kYOverlap : 0;
            if (all) {
#pragma unroll 1
                for (int c = 0; c < (int)kYAcc1; c += 16) {
                    float acc[16];
                    tmem_ld16(acc0 + c1 + c, acc);
                    store(c1 + c, acc, std::integral_constant<int, 16>());
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    pair_ends<kYStages, kYStageBytes>(bars, rank);
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Codes [rows, D / 2] as bytes: boxes of kXRow bytes x box_rows, 128-byte swizzle;
// zeros (the code of 0) past the extents.
static bool make_map_codes(CUtensorMap *map, const void *ptr, int64_t rows, int64_t D, int box_rows) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)(D / 2), (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(D / 2)};
    cuuint32_t box[2] = {(cuuint32_t)kXRow, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as rows of 32-bit words, one row for each 128 rows of the matrix;
// boxes of one row and two tiles. Zeros (2^-127) past the extents.
static bool make_map_scales(CUtensorMap *map, const void *ptr, int64_t rows, int64_t D) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t words = (cuuint64_t)((D + 127) / 128) * 128;
    cuuint64_t dims[2] = {words, (cuuint64_t)((rows + 127) / 128)};
    cuuint64_t strides[1] = {words * 4};
    cuuint32_t box[2] = {(cuuint32_t)(kXSStage / 4), 1u};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sets a kernel's shared memory limit once per device.
template <typename K>
static cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || done.load(std::memory_order_relaxed) >> (dev & 63) & 1u) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
    return e;
}

static int sm_count() {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return std::max(1, sms);
}

template <int kNT, typename T>
static cudaError_t launch_linear_t(const LinearMxfp4Args &a) {
    CUtensorMap tw, tx;
    if (!make_map_codes(&tw, a.w_codes, a.V, a.D, kXM) || !make_map_codes(&tx, a.x_codes, a.N, a.D, kNT))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(linear_mxfp4_kernel<kNT, T>, x_smem_bytes(kNT), done);
    if (e != cudaSuccess) return e;
    const int64_t n_tiles = ((a.V + kXM - 1) / kXM) * ((a.N + kNT - 1) / kNT);
    return launch_pdl(linear_mxfp4_kernel<kNT, T>, dim3((unsigned)std::min<int64_t>(n_tiles, sm_count())),
                      dim3(kXThreads), x_smem_bytes(kNT), a.stream, tw, tx, static_cast<const uint8_t *>(a.w_scales),
                      static_cast<const uint8_t *>(a.x_scales), (int)a.N, (int)a.V, (int)a.D, static_cast<T *>(a.y));
}

template <typename T>
static cudaError_t launch_linear_pair(const LinearMxfp4Args &a) {
    CUtensorMap tw, tx, tws, txs;
    if (!make_map_codes(&tw, a.w_codes, a.V, a.D, kXM) || !make_map_codes(&tx, a.x_codes, a.N, a.D, kXM) ||
        !make_map_scales(&tws, a.w_scales, a.V, a.D) || !make_map_scales(&txs, a.x_scales, a.N, a.D))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(linear_mxfp4_pair_kernel<T>, kYSmemBytes, done);
    if (e != cudaSuccess) return e;
    const int64_t n_tiles = ((a.V + 2 * kXM - 1) / (2 * kXM)) * ((a.N + kYT - 1) / kYT);
    const int64_t pairs = std::max(1, sm_count() / 2);
    return launch_pdl(linear_mxfp4_pair_kernel<T>, dim3((unsigned)(2 * std::min(n_tiles, pairs))), dim3(kXThreads),
                      kYSmemBytes, a.stream, tw, tx, tws, txs, (int)a.N, (int)a.V, (int)a.D, static_cast<T *>(a.y));
}

// Up to 128 tokens one CTA's tile holds them all; more go to the pairs.
template <typename T>
static cudaError_t launch_linear(const LinearMxfp4Args &a) {
    return a.N <= 16 ? launch_linear_t<16, T>(a)
           : a.N <= 32 ? launch_linear_t<32, T>(a)
           : a.N <= 64 ? launch_linear_t<64, T>(a)
           : a.N <= 128 ? launch_linear_t<128, T>(a)
                        : launch_linear_pair<T>(a);
}

cudaError_t launch_linear_mxfp4(const LinearMxfp4Args &a) {
    return a.bf16 ? launch_linear<__nv_bfloat16>(a) : launch_linear<float>(a);
}

cudaError_t read_linear_mxfp4_fault(uint32_t *value, bool clear) { return read_tu_fault(value, clear); }

}  // namespace vp
