// dg_act_bwd.cuh -- sm_100a kernel of the gradient of the GEMM's epilogue: dz = dD
// act'(Z), cast per 1x128 and per 128x1 as the backward GEMMs read it, and its
// column sums, the bias's gradient.  Times are of one B200 in graph replays over
// inputs larger than L2.
#pragma once

#include <stdint.h>

#include "dg_act.cuh"
#include "dg_cast.cuh"
#include "dg_moe.cuh"
#include "dg_ptx.cuh"

namespace dg {

struct ActBwdParams {
    TileOut out;         // Qr [M][N], Qc [128 ceil(M/128)][N]
    float* part;         // [ceil(M/128)][N] column sums of the row blocks, or null
    const uint16_t* dD;  // [M][N]
    const uint16_t* Z;   // [M][N]
    int M, N, nb;        // nb = N / 128
};

constexpr int kActBwdThreads = 256;

// tile_cast_rows of one matrix whose last rows may be missing.
template <int T>
__device__ __forceinline__ void tile_cast_rows_below(const TileOut& o, const F8 (&v)[CastTile<T>::kRows], int64_t row0,
                                                     int64_t rows, int N, int col) {
    constexpr int R = CastTile<T>::kRows;
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15, base = threadIdx.x & 16;
    float a[R];
#pragma unroll
    for (int i = 0; i < R; ++i) a[i] = amax8(v[i]);
    const float s = spread_scale<R>(half_warp_max_spread<R>(a));
    const int64_t mine = row0 + half + CastTile<T>::kStep * (hl - R);
    if (hl >= R && hl < 2 * R && mine < rows) o.sr[static_cast<int64_t>(col >> 7) * o.sr_stride + mine] = s;
    uint8_t* q = o.Qr + (row0 + half) * N + col + hl * 8;
    const int64_t step = static_cast<int64_t>(CastTile<T>::kStep) * N;
#pragma unroll
    for (int i = 0; i < R; ++i, q += step) {
        const float r = __shfl_sync(0xffffffffu, s, base + i);
        if (row0 + half + CastTile<T>::kStep * i < rows) *reinterpret_cast<uint2*>(q) = e4m3x8(v[i], r);
    }
}

// A CTA takes a 128 x 128 tile, thread layout as in dg_moe.cuh's tiles.
template <int ACT>
__global__ void __launch_bounds__(kActBwdThreads, 2)
act_bwd_kernel(const ActBwdParams p) {
    constexpr int T = kActBwdThreads, R = CastTile<T>::kRows;
    __shared__ __align__(16) float cm[CastTile<T>::kWarps * CastTile<T>::kStride];
    __shared__ __align__(16) float cs[CastTile<T>::kWarps * CastTile<T>::kStride];
    __shared__ __align__(16) float cr[128];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, half = tid >> 4, hl = tid & 15;
    const uint32_t rb = blockIdx.x / p.nb;
    const int col = static_cast<int>(blockIdx.x - rb * p.nb) * 128;
    const int64_t row0 = static_cast<int64_t>(rb) * 128;
    const int64_t at = (row0 + half) * p.N + col + hl * 8, step = static_cast<int64_t>(CastTile<T>::kStep) * p.N;
    uint4 d[R], z[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool there = row0 + half + CastTile<T>::kStep * i < p.M;
        d[i] = there ? ld_once_16(p.dD + at + i * step) : make_uint4(0, 0, 0, 0);
        z[i] = there && ACT != kActNone ? ld_once_16(p.Z + at + i * step) : make_uint4(0, 0, 0, 0);
    }
    F8 v[R];
    float2 sum[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) sum[x] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        F8 zz;
        bf16x8_to_f8(d[i], v[i]);
        bf16x8_to_f8(z[i], zz);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (ACT != kActNone) v[i][x] = __fmul2_rn(v[i][x], act_slope2<ACT>(zz[x]));
            sum[x] = __fadd2_rn(sum[x], v[i][x]);
        }
    }
    tile_column_max<T>(v, cm);
    if (p.part != nullptr) {
        // the two half-warps exchange four columns each
        const bool hi = tid & 16;
        float m[8] = {sum[0].x, sum[0].y, sum[1].x, sum[1].y, sum[2].x, sum[2].y, sum[3].x, sum[3].y};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float keep = hi ? m[4 + x] : m[x], send = hi ? m[x] : m[4 + x];
            m[x] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
        }
        *reinterpret_cast<float4*>(cs + (tid >> 5) * CastTile<T>::kStride + hl * 8 + (hi ? 4 : 0)) =
            make_float4(m[0], m[1], m[2], m[3]);
    }
    __syncthreads();
    const int cols[1] = {col};
    tile_column_scale<T>(p.out, cm, cr, row0, cols);
    if (p.part != nullptr && tid < 128) {
        float s = cs[tid];
#pragma unroll
        for (int w = 1; w < CastTile<T>::kWarps; ++w) s += cs[w * CastTile<T>::kStride + tid];
        p.part[static_cast<int64_t>(rb) * p.N + col + tid] = s;
    }
    tile_cast_rows_below<T>(p.out, v, row0, p.M, p.N, col);
    __syncthreads();
    tile_cast_columns<T>(p.out, v, cr, row0, p.N, col);
}

}  // namespace dg
