// dg_ckpt.cuh -- sm_100a kernels of the gated activation with 8-bit
// checkpoints: gate and up are kept for the backward pass as e4m3 codes with a
// scale per 1x128, and the backward pass works from those.  Bound by HBM.
//
//   a = silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g))
//   dg = da u (s + silu (1 - s)),   du = da silu
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "dg_cast.cuh"
#include "dg_moe.cuh"
#include "dg_ptx.cuh"

namespace dg {

// 8 e4m3 codes -> floats (exact).
__device__ __forceinline__ void e4m3x8_to_float(const uint2& c, float (&f)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 x = __half22float2(__half2(h));
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

__device__ __forceinline__ uint2 ld_once_8(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// -------------------------------------------------------------- forward ----

struct SwigluParams {
    uint8_t* Q;                // [rows][F], scales like dg_to_fp8_1x128's
    float* sa;
    uint8_t* C;                // [rows][2F] or null
    float* cs;
    const uint16_t* H;         // [rows][2F]: gate, up
    const int32_t* m_indices;  // [rows] or null; negative: the row is left
    int sa_stride, cs_stride, group_rows;
    int F, nfb;                // nfb = F / 128
    int64_t rows;
};

// Half-warp h of a CTA takes a row, NB pairs of gate and up blocks at a time.
template <int NB>
__global__ void __launch_bounds__(kCastThreads)
swiglu_fp8_kernel(const SwigluParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15;
    const int64_t row_groups = (p.rows + kCastRowsPerCta - 1) / kCastRowsPerCta;
    const int fb_groups = (p.nfb + NB - 1) / NB;
    const int64_t items = row_groups * fb_groups;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t row = (it / fb_groups) * kCastRowsPerCta + half;
        const int fb0 = static_cast<int>(it % fb_groups) * NB;
        const bool there = row < p.rows && (p.m_indices == nullptr || p.m_indices[row] >= 0);
        const uint16_t* hr = p.H + row * 2 * p.F + fb0 * 128 + hl * 8;
        uint4 vg[NB], vu[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const bool ok = there && fb0 + b < p.nfb;
            vg[b] = ok ? ld_once_16(hr + b * 128) : make_uint4(0, 0, 0, 0);
            vu[b] = ok ? ld_once_16(hr + p.F + b * 128) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float g[8], u[8], a[8];
            bf16x8_to_float(vg[b], g);
            bf16x8_to_float(vu[b], u);
#pragma unroll
            for (int x = 0; x < 8; ++x) a[x] = __fdividef(g[x], 1.f + __expf(-g[x])) * u[x];
            // three casts: the scales of a, gate and up (the fourth place is spare)
            float m[4] = {amax8(a), amax8(g), amax8(u), 0.f};
            const float sc = spread_scale<4>(half_warp_max_spread<4>(m));
            const int base = threadIdx.x & 16;
            const float ra = __shfl_sync(0xffffffffu, sc, base), rg = __shfl_sync(0xffffffffu, sc, base + 1);
            const float ru = __shfl_sync(0xffffffffu, sc, base + 2);
            if (!there || fb0 + b >= p.nfb) continue;
            const int fb = fb0 + b;
            *reinterpret_cast<uint2*>(p.Q + row * p.F + fb * 128 + hl * 8) = e4m3x8(a, ra);
            if (hl == 4) p.sa[scale_at(row, fb, p.nfb, p.sa_stride, p.group_rows)] = sc;
            if (p.C != nullptr) {
                uint8_t* cr = p.C + row * 2 * p.F + fb * 128 + hl * 8;
                *reinterpret_cast<uint2*>(cr) = e4m3x8(g, rg);
                *reinterpret_cast<uint2*>(cr + p.F) = e4m3x8(u, ru);
                if (hl == 5 || hl == 6)
                    p.cs[scale_at(row, fb + (hl == 6 ? p.nfb : 0), 2 * p.nfb, p.cs_stride, p.group_rows)] = sc;
            }
        }
    }
}

// ------------------------------------------------------------- backward ----

struct SwigluBwdParams {
    TileOut out;               // of dH [rows][2F]: dg, du
    uint8_t* Qa;               // [rows][F]: a again, per 128x128 block
    float* sb;                 // [F / 128][rows / 128]
    const uint16_t* dA;        // [rows][F]
    const uint8_t* C;          // [rows][2F]
    const float* cs;
    const int32_t* m_indices;  // [rows] or null
    int64_t cs_stride;
    int F, nfb;
    int64_t rows;
};

constexpr int kSwigluBwdThreads = 512;
// A stage of shared memory: each thread's pieces of dA, gate and up, then the
// rows' two scales.
constexpr int kSwigluBwdScales = 128 * 128 * 4;
constexpr int kSwigluBwdStage = kSwigluBwdScales + 128 * 2 * 4;

// A persistent CTA takes 128 x 128 tiles of the expert width, for gate and up:
// thread layout as in dg_moe.cuh's tiles.  dg and silu stay in registers;
// du = da silu and a = silu u are formed where they are used (one product),
// from da and u in shared memory, which keeps the tile within the register
// file.  Two stages: the next tile's bytes arrive during this one's casts, and
// as every thread copies what it will itself use, no barrier guards them.
__global__ void __launch_bounds__(kSwigluBwdThreads)
swiglu_fp8_bwd_kernel(const SwigluBwdParams p) {
    constexpr int T = kSwigluBwdThreads, R = CastTile<T>::kRows;
    static_assert(R == 4 && CastTile<T>::kStep == 32, "a mask of row flags per i");
    extern __shared__ __align__(16) uint8_t stage_smem[];
    __shared__ __align__(16) float cm[2][CastTile<T>::kWarps * CastTile<T>::kStride];
    __shared__ __align__(16) float cr[2][128];
    __shared__ float wm[CastTile<T>::kWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, half = tid >> 4, hl = tid & 15;
    const int64_t tiles = p.rows / 128 * p.nfb;
    const uint32_t stage0 = smem_u32(stage_smem);

    // Row flags of a tile: bit r of mask i is row r + 32 i.
    auto flags = [&](int64_t tile, uint32_t (&mask)[4]) {
        const int64_t row0 = tile / p.nfb * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mask[i] = __ballot_sync(0xffffffffu, p.m_indices == nullptr || p.m_indices[row0 + lane + 32 * i] >= 0);
    };
    auto fetch = [&](int64_t tile, const uint32_t (&mask)[4], int st) {
        const int64_t row0 = tile / p.nfb * 128;
        const int fb = static_cast<int>(tile % p.nfb);
        const int64_t col = fb * 128 + hl * 8;
        const uint32_t at = stage0 + st * kSwigluBwdStage;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t row = row0 + half + 32 * i;
            const bool ok = (mask[i] >> half) & 1u;
            cp_async_16(at + (i * T + tid) * 16, p.dA + row * p.F + col, ok ? 16 : 0);
            cp_async_8(at + R * T * 16 + (2 * i * T + tid) * 8, p.C + row * 2 * p.F + col, ok ? 8 : 0);
            cp_async_8(at + R * T * 16 + ((2 * i + 1) * T + tid) * 8, p.C + row * 2 * p.F + p.F + col, ok ? 8 : 0);
        }
        if (hl < 8) {  // lane i: gate scale of row i, lane 4 + i: up scale
            const int64_t row = row0 + half + 32 * (hl & 3);
            const uint32_t m = (hl & 2) ? (hl & 1 ? mask[3] : mask[2]) : (hl & 1 ? mask[1] : mask[0]);
            cp_async_4(at + kSwigluBwdScales + (half * 8 + hl) * 4,
                       p.cs + static_cast<int64_t>(fb + (hl & 4 ? p.nfb : 0)) * p.cs_stride + row, (m >> half) & 1u ? 4 : 0);
        }
        cp_async_commit();
    };

    int64_t tile = blockIdx.x;
    uint32_t mask[4];
    if (tile < tiles) {
        flags(tile, mask);
        fetch(tile, mask, 0);
    }
    for (int st = 0; tile < tiles; tile += gridDim.x, st ^= 1) {
        const bool live = (mask[0] | mask[1] | mask[2] | mask[3]) != 0;
        if (tile + gridDim.x < tiles) {
            flags(tile + gridDim.x, mask);
            fetch(tile + gridDim.x, mask, st ^ 1);
            cp_async_wait<1>();
        } else {
            cp_async_wait<0>();
        }
        if (!live) continue;  // the same answer in every warp
        __syncwarp();         // the scales were copied by other lanes
        const int64_t rb = tile / p.nfb, row0 = rb * 128;
        const int fb = static_cast<int>(tile % p.nfb);
        const uint32_t at = stage0 + st * kSwigluBwdStage;
        auto piece_da = [&](int i, float (&f)[8]) { bf16x8_to_float(ld_shared_16(at + (i * T + tid) * 16), f); };
        auto piece_c = [&](int i, int up, float (&f)[8]) {
            uint2 c;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(c.x), "=r"(c.y) : "r"(at + R * T * 16 + ((2 * i + up) * T + tid) * 8) : "memory");
            float s;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(at + kSwigluBwdScales + (half * 8 + up * 4 + i) * 4) : "memory");
            e4m3x8_to_float(c, f);
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = __fmul_rn(f[x], s);
        };

        float dg[R][8], silu[R][8];
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float u[8], d[8];
            piece_c(i, 0, silu[i]);
            piece_c(i, 1, u);
            piece_da(i, d);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float g = silu[i][x];
                const float s = __fdividef(1.f, 1.f + __expf(-g));
                silu[i][x] = __fmul_rn(g, s);
                dg[i][x] = d[x] * u[x] * fmaf(silu[i][x], 1.f - s, s);
                am = fmaxf(am, fabsf(__fmul_rn(silu[i][x], u[x])));
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        if (lane == 0) wm[tid >> 5] = am;
        tile_column_max<T>(dg, cm[0]);
        tile_cast_rows<T>(p.out, dg, row0, 2 * p.F, fb * 128);
        {
            float du[R][8];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                piece_da(i, du[i]);
#pragma unroll
                for (int x = 0; x < 8; ++x) du[i][x] = __fmul_rn(du[i][x], silu[i][x]);
            }
            tile_column_max<T>(du, cm[1]);
            tile_cast_rows<T>(p.out, du, row0, 2 * p.F, p.F + fb * 128);
        }
        __syncthreads();
        tile_column_scale<T>(p.out, cm[0], cr[0], row0, fb * 128);
        tile_column_scale<T>(p.out, cm[1], cr[1], row0, p.F + fb * 128);
        am = wm[0];
#pragma unroll
        for (int w = 1; w < CastTile<T>::kWarps; ++w) am = fmaxf(am, wm[w]);
        am = fmaxf(am, 1e-4f);
        const float ra = __fdiv_rn(448.f, am);
        if (tid == 0) p.sb[static_cast<int64_t>(fb) * (p.rows / 128) + rb] = __fdiv_rn(am, 448.f);
        __syncthreads();
        tile_cast_columns<T>(p.out, dg, cr[0], row0, 2 * p.F, fb * 128);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            piece_da(i, dg[i]);
#pragma unroll
            for (int x = 0; x < 8; ++x) dg[i][x] = __fmul_rn(dg[i][x], silu[i][x]);
        }
        tile_cast_columns<T>(p.out, dg, cr[1], row0, 2 * p.F, p.F + fb * 128);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float u[8];
            piece_c(i, 1, u);
#pragma unroll
            for (int x = 0; x < 8; ++x) u[x] = __fmul_rn(silu[i][x], u[x]);
            *reinterpret_cast<uint2*>(p.Qa + (row0 + half + 32 * i) * p.F + fb * 128 + hl * 8) = e4m3x8(u, ra);
        }
    }
}

// --------------------------------------------------------------- recast ----

constexpr int kRecastThreads = 256;

struct RecastParams {
    uint8_t* Qb;               // [rows][K]
    float* sb;                 // [K / 128][rows / 128]
    const uint8_t* Q;          // [rows][K]
    const float* sa;
    const int32_t* m_indices;  // [rows] or null
    int64_t sa_stride;
    int K, nkb;
    int64_t rows;
};

// Largest magnitude among 16 codes, NaN (0x7F) not counted: the 7 low bits of
// an e4m3 code order its magnitudes.
__device__ __forceinline__ uint32_t max_code(const uint4& v) {
    uint32_t m = 0;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t x = w[i] & 0x7F7F7F7Fu;
        x &= ~__vcmpeq4(x, 0x7F7F7F7Fu);
        m = __vmaxu4(m, x);
    }
    m = max(max(m & 255u, (m >> 8) & 255u), max((m >> 16) & 255u, m >> 24));
    return m;
}

// One CTA per 128 x 128 block, 8 threads to a row (16 codes each).  The block's
// maximum comes from the rows' largest codes: code order is magnitude order,
// and rounding code * scale keeps it.
__global__ void __launch_bounds__(kRecastThreads)
recast_128x128_kernel(const RecastParams p) {
    __shared__ float wm[kRecastThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int kb = static_cast<int>(blockIdx.x % p.nkb);
    const int64_t rb = blockIdx.x / p.nkb;
    const int64_t at = (rb * 128 + (tid >> 3)) * p.K + kb * 128 + (tid & 7) * 16;
    uint4 v[4];
    float s[4];
    bool any = false;
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = rb * 128 + (tid >> 3) + 32 * i;
        const bool there = p.m_indices == nullptr || p.m_indices[row] >= 0;
        any |= there;
        v[i] = there ? ld_once_16(p.Q + at + static_cast<int64_t>(32 * i) * p.K) : make_uint4(0, 0, 0, 0);
        s[i] = there ? p.sa[static_cast<int64_t>(kb) * p.sa_stride + row] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(max_code(v[i])), __NV_E4M3);
        a = fmaxf(a, fabsf(__fmul_rn(__half2float(__half(h)), s[i])));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if ((tid & 31) == 0) wm[tid >> 5] = a;
    if (!__syncthreads_or(any)) return;
    a = wm[0];
#pragma unroll
    for (int w = 1; w < kRecastThreads / 32; ++w) a = fmaxf(a, wm[w]);
    a = fmaxf(a, 1e-4f);
    const float r = __fdiv_rn(448.f, a);
    if (tid == 0) p.sb[static_cast<int64_t>(kb) * (p.rows / 128) + rb] = __fdiv_rn(a, 448.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint2 q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[8];
            e4m3x8_to_float(h ? make_uint2(v[i].z, v[i].w) : make_uint2(v[i].x, v[i].y), f);
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = __fmul_rn(f[x], s[i]);
            q[h] = e4m3x8(f, r);
        }
        *reinterpret_cast<uint4*>(p.Qb + at + static_cast<int64_t>(32 * i) * p.K) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
    }
}

}  // namespace dg
