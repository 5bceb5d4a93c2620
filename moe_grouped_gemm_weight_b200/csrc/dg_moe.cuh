// dg_moe.cuh -- sm_100a kernels between the routing and the grouped GEMMs:
// the cast of the tokens into the rows of the grouped layout, the weighted sum
// of the experts' rows per token, and its gradient.  All are bound by HBM.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_cast.cuh"
#include "dg_ptx.cuh"

namespace dg {

// 16 bytes that another kernel has just written, not kept in L1.  (Not the
// read-only path: a kernel launched before its predecessor ended must not
// read the predecessor's results through it.)
__device__ __forceinline__ uint4 ld_once_16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Place of row r's scale of K block kb: groups of group_rows rows have blocks
// of their own (masked layout); group_rows == 0: one block for all rows.
__device__ __forceinline__ int64_t scale_at(int64_t r, int kb, int nkb, int stride, int group_rows) {
    if (group_rows == 0) return static_cast<int64_t>(kb) * stride + r;
    const int64_t g = r / group_rows;
    return (g * nkb + kb) * stride + (r - g * group_rows);
}

// ------------------------------------------------------------- dispatch ----

struct DispatchParams {
    uint8_t* Q;            // [rows][K]
    float* sa;
    const uint16_t* X;     // [T][K]
    const int32_t* row_of; // [T][k]
    int T, k, K, nkb;
    int sa_stride, group_rows;
    int64_t rows;
};

// The cast of dg_cast.cuh's cast_1x128_kernel, a token read and cast once and
// written to each of its k rows: half-warp h of a CTA takes a token, NB K
// blocks at a time.  Lane j of the half-warp keeps the token's rows j and
// j + 16 and writes their scales.
template <int NB>
__global__ void __launch_bounds__(kCastThreads)
dispatch_1x128_kernel(const DispatchParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15;
    const int base = threadIdx.x & 16;  // first lane of this half-warp
    const int token_groups = (p.T + kCastRowsPerCta - 1) / kCastRowsPerCta;
    const int kb_groups = (p.nkb + NB - 1) / NB;
    const int64_t items = static_cast<int64_t>(token_groups) * kb_groups;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t t = (it / kb_groups) * kCastRowsPerCta + half;
        const int kb0 = static_cast<int>(it % kb_groups) * NB;
        const bool there = t < p.T;
        const uint16_t* xr = p.X + t * p.K + kb0 * 128 + hl * 8;
        uint4 v[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            v[b] = there && kb0 + b < p.nkb ? ld_once_16(xr + b * 128) : make_uint4(0, 0, 0, 0);
        int row[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = hl + 16 * h;
            row[h] = there && j < p.k ? p.row_of[t * p.k + j] : -1;
            if (row[h] >= p.rows) row[h] = -1;
        }
        uint2 q[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float f[8];
            bf16x8_to_float(v[b], f);
            const float a = fmaxf(half_warp_max(amax8(f)), 1e-4f);
            q[b] = e4m3x8(f, __fdiv_rn(448.f, a));
            const float s = __fdiv_rn(a, 448.f);
            if (kb0 + b < p.nkb) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (row[h] >= 0) p.sa[scale_at(row[h], kb0 + b, p.nkb, p.sa_stride, p.group_rows)] = s;
            }
        }
        for (int j = 0; j < p.k; ++j) {
            const int r = __shfl_sync(0xffffffffu, row[0], base + (j & 15));
            const int r1 = __shfl_sync(0xffffffffu, row[1], base + (j & 15));
            const int to = j < 16 ? r : r1;
            if (to < 0) continue;
            uint8_t* qr = p.Q + static_cast<int64_t>(to) * p.K + kb0 * 128 + hl * 8;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (kb0 + b < p.nkb) *reinterpret_cast<uint2*>(qr + b * 128) = q[b];
        }
    }
}

// -------------------------------------------------------------- combine ----

constexpr int kCombineThreads = 128;
constexpr int kCombineBatch = 8;  // rows in flight per thread

struct CombineParams {
    uint16_t* out;         // [T][N]
    const uint16_t* Y;     // [rows][N]
    const int32_t* row_of; // [T][k]
    const float* w;        // [T][k] or null: all ones
    int T, k, N;
    int64_t rows;
};

// out[t] = sum_j w_j Y[row_j]: one thread per 8 columns of a token, its rows'
// loads in flight together, FP32 sums in slot order.
__global__ void __launch_bounds__(kCombineThreads)
combine_kernel(const CombineParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int chunks = (p.N / 8 + kCombineThreads - 1) / kCombineThreads;
    const int64_t t = blockIdx.x / chunks;
    const int c = (static_cast<int>(blockIdx.x % chunks) * kCombineThreads + static_cast<int>(threadIdx.x)) * 8;
    if (c >= p.N) return;
    float acc[8] = {};
    for (int j0 = 0; j0 < p.k; j0 += kCombineBatch) {
        uint4 v[kCombineBatch];
        float w[kCombineBatch];
#pragma unroll
        for (int i = 0; i < kCombineBatch; ++i) {
            const int j = j0 + i;
            const int row = j < p.k ? p.row_of[t * p.k + j] : -1;
            const bool ok = row >= 0 && row < p.rows;
            v[i] = ok ? ld_once_16(p.Y + static_cast<int64_t>(row) * p.N + c) : make_uint4(0, 0, 0, 0);
            w[i] = !ok ? 0.f : p.w ? p.w[t * p.k + j] : 1.f;
        }
#pragma unroll
        for (int i = 0; i < kCombineBatch; ++i) {
            float f[8];
            bf16x8_to_float(v[i], f);
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[x] = fmaf(w[i], f[x], acc[x]);
        }
    }
    uint4 o;
    o.x = pack_bf16x2(acc[0], acc[1]);
    o.y = pack_bf16x2(acc[2], acc[3]);
    o.z = pack_bf16x2(acc[4], acc[5]);
    o.w = pack_bf16x2(acc[6], acc[7]);
    *reinterpret_cast<uint4*>(p.out + t * p.N + c) = o;
}

// ---------------------------------------------- two casts of one gradient ----

// A CTA of kTileThreads holds a 128 x 128 tile of a gradient in registers:
// half-warp h (0..31) the rows h + 32 i (i < 4), lane hl of it columns
// 8 hl .. 8 hl + 7.  Both casts that a backward pass needs come from the same
// values: a scale per row (1x128, the input gradient's operand) and a scale
// per column (128x1, the weight gradient's, whose K is the rows).
constexpr int kTileThreads = 512;
constexpr int kTileRows = 4;  // rows per thread

struct TileOut {
    uint8_t* Qr;   // [rows][N], scales sr[kb * sr_stride + row]
    float* sr;
    uint8_t* Qc;   // [rows][N], scales sc[(row / 128) * sc_stride + column]
    float* sc;
    int64_t sr_stride, sc_stride;
};

// 1x128: each half-warp has a whole row of the tile.
__device__ __forceinline__ void tile_cast_rows(const TileOut& o, const float (&v)[kTileRows][8], int64_t row0, int N,
                                               int col0) {
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        const int64_t row = row0 + half + 32 * i;
        const float a = fmaxf(half_warp_max(amax8(v[i])), 1e-4f);
        *reinterpret_cast<uint2*>(o.Qr + row * N + col0 + hl * 8) = e4m3x8(v[i], __fdiv_rn(448.f, a));
        if (hl == 0) o.sr[static_cast<int64_t>(col0 / 128) * o.sr_stride + row] = __fdiv_rn(a, 448.f);
    }
}

// 128x1, first half: the warps' column maxima into cm[warp][128].
__device__ __forceinline__ void tile_column_max(const float (&v)[kTileRows][8], float* cm) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        m[x] = 0.f;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) m[x] = fmaxf(m[x], fabsf(v[i][x]));
        m[x] = fmaxf(m[x], __shfl_xor_sync(0xffffffffu, m[x], 16));
    }
    if (lane < 16) {
        float4* to = reinterpret_cast<float4*>(cm + warp * 128 + lane * 8);
        to[0] = make_float4(m[0], m[1], m[2], m[3]);
        to[1] = make_float4(m[4], m[5], m[6], m[7]);
    }
}

// Second half, after a barrier: threads 0..127 join the warps' maxima, write
// the scales and leave 448 / amax in cr[128].
__device__ __forceinline__ void tile_column_scale(const TileOut& o, const float* cm, float* cr, int64_t row0, int col0,
                                                  int tid) {
    float a = cm[tid];
#pragma unroll
    for (int w = 1; w < kTileThreads / 32; ++w) a = fmaxf(a, cm[w * 128 + tid]);
    a = fmaxf(a, 1e-4f);
    cr[tid] = __fdiv_rn(448.f, a);
    o.sc[(row0 / 128) * o.sc_stride + col0 + tid] = __fdiv_rn(a, 448.f);
}

// Third part, after another barrier.
__device__ __forceinline__ void tile_cast_columns(const TileOut& o, const float (&v)[kTileRows][8], const float* cr,
                                                  int64_t row0, int N, int col0) {
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15;
    float r[8];
    *reinterpret_cast<float4*>(r) = *reinterpret_cast<const float4*>(cr + hl * 8);
    *reinterpret_cast<float4*>(r + 4) = *reinterpret_cast<const float4*>(cr + hl * 8 + 4);
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        uint32_t q[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            q[x] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[i][2 * x], r[2 * x]), __fmul_rn(v[i][2 * x + 1], r[2 * x + 1])),
                                            __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2*>(o.Qc + (row0 + half + 32 * i) * N + col0 + hl * 8) =
            make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    }
}

// ----------------------------------------------------- combine, backward ----

struct CombineBwdParams {
    TileOut out;           // of dY [rows][N]
    float* dw;             // [T][k]
    const uint16_t* dout;  // [T][N]
    const uint16_t* Y;     // [rows][N]
    const int32_t* row_of; // [T][k]
    const int32_t* slot_of;// [rows]
    const float* w;        // [T][k]
    int64_t S;             // T * k
    int k, N, nkb;
    int64_t rows;
};

// dY[row] = w dout[t], cast both ways, and dw = <dout[t], Y[row]>.  A cluster
// of CTAs takes a block of 128 rows, each CTA a run of its 128-column tiles;
// the row sums of dw are joined through distributed shared memory in CTA
// order.  Rows without a slot count as zeros; a block without any is left.
__global__ void __launch_bounds__(kTileThreads)
combine_bwd_kernel(const CombineBwdParams p) {
    __shared__ float cm[kTileThreads / 32 * 128];
    __shared__ __align__(16) float cr[128];
    __shared__ float part[128];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, half = tid >> 4, hl = tid & 15;
    const uint32_t rank = cluster_ctarank(), nctas = cluster_nctarank();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / nctas) * 128;

    // Slots that have no row have no gradient.
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kTileThreads + tid; s < p.S;
         s += static_cast<int64_t>(gridDim.x) * kTileThreads) {
        const int r = p.row_of[s];
        if (r < 0 || r >= p.rows) p.dw[s] = 0.f;
    }

    int64_t slot[kTileRows];
    float w[kTileRows], dot[kTileRows];
    bool any = false;
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        const int s = p.slot_of[row0 + half + 32 * i];
        slot[i] = s >= 0 && s < p.S ? s : -1;
        w[i] = slot[i] >= 0 ? p.w[slot[i]] : 0.f;
        dot[i] = 0.f;
        any |= slot[i] >= 0;
    }
    if (!__syncthreads_or(any)) return;  // the same answer in every CTA of the cluster

    const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / nctas);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / nctas);
    for (int kb = kb0; kb < kb1; ++kb) {
        const int col = kb * 128 + hl * 8;
        uint4 g[kTileRows], y[kTileRows];
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            g[i] = y[i] = make_uint4(0, 0, 0, 0);
            if (slot[i] >= 0) {
                g[i] = ld_once_16(p.dout + (slot[i] / p.k) * p.N + col);
                y[i] = ld_once_16(p.Y + (row0 + half + 32 * i) * p.N + col);
            }
        }
        float v[kTileRows][8];
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            float yf[8];
            bf16x8_to_float(g[i], v[i]);
            bf16x8_to_float(y[i], yf);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                dot[i] = fmaf(v[i][x], yf[x], dot[i]);
                v[i][x] = slot[i] >= 0 ? __fmul_rn(v[i][x], w[i]) : 0.f;
            }
        }
        tile_column_max(v, cm);
        tile_cast_rows(p.out, v, row0, p.N, kb * 128);
        __syncthreads();
        if (tid < 128) tile_column_scale(p.out, cm, cr, row0, kb * 128, tid);
        __syncthreads();
        tile_cast_columns(p.out, v, cr, row0, p.N, kb * 128);
    }
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        const float d = half_warp_sum(dot[i]);
        if (hl == 0) part[half + 32 * i] = d;
    }
    __syncwarp();
    cluster_sync();
    if (rank == 0 && tid < 128) {
        const int s = p.slot_of[row0 + tid];
        float d = 0.f;
        for (uint32_t r = 0; r < nctas; ++r) {
            float x;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(dsmem_addr(smem_u32(part + tid), r)) : "memory");
            d += x;
        }
        if (s >= 0 && s < p.S) p.dw[s] = d;
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its sums are being read
}

}  // namespace dg
