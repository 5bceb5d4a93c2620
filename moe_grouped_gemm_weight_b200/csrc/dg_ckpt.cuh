// dg_ckpt.cuh -- sm_100a kernels of the gated activation with 8-bit
// checkpoints: gate and up are kept for the backward pass as e4m3 codes with a
// scale per 1x128, and the backward pass works from those.  Times are of one
// B200 in graph replays over inputs larger than L2.
//
//   a = silu(g) u,  silu(g) = g s,  s = 1 / (1 + exp(-g))
//   dg = da u (s + silu (1 - s)),   du = da silu
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "dg_act.cuh"
#include "dg_cast.cuh"
#include "dg_moe.cuh"
#include "dg_ptx.cuh"

namespace dg {

// Eight e4m3 codes -> floats (exact).
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3));
}
__device__ __forceinline__ void e4m3x8_to_f8(const uint2& c, F8& f) {
    f[0] = __half22float2(e4m3x2_to_half2(c.x));
    f[1] = __half22float2(e4m3x2_to_half2(c.x >> 16));
    f[2] = __half22float2(e4m3x2_to_half2(c.y));
    f[3] = __half22float2(e4m3x2_to_half2(c.y >> 16));
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
    int rows;
    uint32_t items;            // row groups times pairs of blocks
};

constexpr int kSwigluCtas = 4;  // resident per SM

// Half-warp h of a CTA takes a row, two pairs of gate and up blocks at a time:
// six tiles whose scales are found together (places 3 and 7 of 8 are spare).
// 32768 rows of F = 2048 with the checkpoint: 94 us, 5.1 TB/s, bound by HBM and,
// at 62 % of the issue slots, nearly by instructions; without it 68 us.  512 slots
// in a masked layout of 32 groups of 64 rows, no checkpoint: 4.1 us.
__global__ void __launch_bounds__(kCastThreads, kSwigluCtas)
swiglu_fp8_kernel(const SwigluParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15, base = threadIdx.x & 16;
    const uint32_t fb_groups = (p.nfb + 1) / 2;
    for (uint32_t it = blockIdx.x; it < p.items; it += gridDim.x) {
        const uint32_t rg = it / fb_groups;
        const int row = static_cast<int>(rg) * kCastRowsPerCta + half;
        const int fb0 = static_cast<int>(it - rg * fb_groups) * 2;
        const bool there = row < p.rows && (p.m_indices == nullptr || p.m_indices[row] >= 0);
        if (!__any_sync(0xffffffffu, there)) continue;
        const uint16_t* hr = p.H + static_cast<int64_t>(row) * 2 * p.F + fb0 * 128 + hl * 8;
        uint4 vg[2], vu[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const bool ok = there && fb0 + b < p.nfb;
            vg[b] = ok ? ld_once_16(hr + b * 128) : make_uint4(0, 0, 0, 0);
            vu[b] = ok ? ld_once_16(hr + p.F + b * 128) : make_uint4(0, 0, 0, 0);
        }
        F8 a[2], g[2], u[2];
        float m[8];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            bf16x8_to_f8(vg[b], g[b]);
            bf16x8_to_f8(vu[b], u[b]);
#pragma unroll
            for (int x = 0; x < 4; ++x) a[b][x] = __fmul2_rn(__fmul2_rn(g[b][x], sigmoid2(g[b][x])), u[b][x]);
            m[4 * b] = amax8(a[b]);
            m[4 * b + 1] = amax8(g[b]);
            m[4 * b + 2] = amax8(u[b]);
            m[4 * b + 3] = 0.f;
        }
        const float sc = spread_scale<8>(half_warp_max_spread<8>(m));
        // lane 8 + 4 b + i writes the scale of block b's a, gate or up
        const int b = (hl >> 2) & 1, i = hl & 3;
        if (hl >= 8 && there && fb0 + b < p.nfb && i < 3) {
            if (i == 0)
                p.sa[scale_base(row, p.nfb, p.sa_stride, p.group_rows) + static_cast<int64_t>(fb0 + b) * p.sa_stride] = sc;
            else if (p.C != nullptr)
                p.cs[scale_base(row, 2 * p.nfb, p.cs_stride, p.group_rows) +
                     static_cast<int64_t>(fb0 + b + (i == 2 ? p.nfb : 0)) * p.cs_stride] = sc;
        }
        __syncwarp();
        uint8_t* qr = p.Q + static_cast<int64_t>(row) * p.F + fb0 * 128 + hl * 8;
        uint8_t* cr = p.C + static_cast<int64_t>(row) * 2 * p.F + fb0 * 128 + hl * 8;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float ra = __shfl_sync(0xffffffffu, sc, base + 4 * b), rg = __shfl_sync(0xffffffffu, sc, base + 4 * b + 1);
            const float ru = __shfl_sync(0xffffffffu, sc, base + 4 * b + 2);
            if (there && fb0 + b < p.nfb) {
                *reinterpret_cast<uint2*>(qr + b * 128) = e4m3x8(a[b], ra);
                if (p.C != nullptr) {
                    *reinterpret_cast<uint2*>(cr + b * 128) = e4m3x8(g[b], rg);
                    *reinterpret_cast<uint2*>(cr + p.F + b * 128) = e4m3x8(u[b], ru);
                }
            }
            __syncwarp();
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
    int rows;
    uint32_t tiles;            // row blocks times F blocks
};

constexpr int kSwigluBwdThreads = 512;
// A stage of shared memory: each thread's pieces of dA, gate and up, then the
// rows' two scales.
constexpr int kSwigluBwdScales = 128 * 128 * 4;
constexpr int kSwigluBwdStage = kSwigluBwdScales + 128 * 2 * 4;
constexpr int kSwigluBwdFlags = kSwigluBwdThreads / 32 * 128 * 4;  // behind the stages: each warp's copy of the next tile's row flags

// A persistent CTA takes 128 x 128 tiles of the expert width, for gate and up:
// thread layout as in dg_moe.cuh's tiles.  dg, du and a are formed once and
// stay in registers (96 of 128) for all five casts; row casts and a's fill the
// waits for the column and block maxima.  Two stages: the next tile's bytes
// arrive during this one's casts, and as every thread copies what it will
// itself use, no barrier guards them; the row flags come a tile ahead of the
// rows they decide on.
//
// 32768 rows of F = 2048: 156 us, 4.0 TB/s, bound by instructions (64 % of the
// issue slots with the 16 warps that the registers allow).
__global__ void __launch_bounds__(kSwigluBwdThreads)
swiglu_fp8_bwd_kernel(const SwigluBwdParams p) {
    constexpr int T = kSwigluBwdThreads, R = CastTile<T>::kRows;
    static_assert(R == 4 && CastTile<T>::kMatrices == 2, "row flags and joins below");
    extern __shared__ __align__(16) uint8_t stage_smem[];
    __shared__ __align__(16) float cm[2][CastTile<T>::kWarps * CastTile<T>::kStride];
    __shared__ __align__(16) float cr[2][128];
    __shared__ float wm[CastTile<T>::kWarps];
    __shared__ uint64_t bars[2];
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bars[0], CastTile<T>::kWarps);
        mbar_init(&bars[1], CastTile<T>::kWarps);
        abort_flag = 0;
        fence_mbar_init();
    }
    SplitBarrier maxima{&bars[0], &abort_flag}, joined{&bars[1], &abort_flag};
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, half = tid >> 4, hl = tid & 15;
    const uint32_t stage0 = smem_u32(stage_smem);

    // Tiles in turn: row block rb, F block fb, without a division per step.
    struct At {
        uint32_t rb, fb;
    };
    const uint32_t step_rb = gridDim.x / p.nfb, step_fb = gridDim.x % p.nfb;
    auto advance = [&](At t) {
        t.rb += step_rb;
        t.fb += step_fb;
        if (t.fb >= static_cast<uint32_t>(p.nfb)) {
            t.fb -= p.nfb;
            ++t.rb;
        }
        return t;
    };
    // Row flags of a tile, bit half & 31 of mask i: this thread's row i; `live`: any row.
    const uint32_t flags_at = stage0 + 2 * kSwigluBwdStage + ((tid >> 5) * 128 + lane) * 4;
    auto flags = [&](uint32_t (&mask)[R], bool& live) {
        uint32_t all[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int m = 0;
            if (p.m_indices != nullptr) asm volatile("ld.shared.s32 %0, [%1];" : "=r"(m) : "r"(flags_at + i * 128) : "memory");
            all[i] = __ballot_sync(0xffffffffu, m >= 0);
        }
        live = (all[0] | all[1] | all[2] | all[3]) != 0;
#pragma unroll
        for (int i = 0; i < R; ++i) mask[i] = all[i];
    };
    auto fetch_flags = [&](At t) {
        if (p.m_indices == nullptr || t.rb * 128 >= static_cast<uint32_t>(p.rows)) return;
        const int32_t* m = p.m_indices + static_cast<int64_t>(t.rb) * 128 + lane;
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async_4(flags_at + i * 128, m + 32 * i, 4);
    };
    // A tile's bytes, and the flags of the tile after it, whose own bytes they decide on.
    auto fetch = [&](At t, const uint32_t (&mask)[R], int st) {
        const int64_t row0 = static_cast<int64_t>(t.rb) * 128;
        const int fb = static_cast<int>(t.fb);
        const uint32_t at = stage0 + st * kSwigluBwdStage;
        const int64_t first = (row0 + half) * p.F + fb * 128 + hl * 8, step = static_cast<int64_t>(CastTile<T>::kStep) * p.F;
        const uint16_t* da = p.dA + first;
        const uint8_t* gate = p.C + first + (row0 + half) * p.F;  // rows of C are twice as long
#pragma unroll
        for (int i = 0; i < R; ++i, da += step, gate += 2 * step) {
            const bool ok = (mask[i] >> (half & 31)) & 1u;
            cp_async_16(at + (i * T + tid) * 16, da, ok ? 16 : 0);
            cp_async_8(at + R * T * 16 + (2 * i * T + tid) * 8, gate, ok ? 8 : 0);
            cp_async_8(at + R * T * 16 + ((2 * i + 1) * T + tid) * 8, gate + p.F, ok ? 8 : 0);
        }
        if (hl < 2 * R) {  // lane i: gate scale of row i, lane R + i: up scale
            const int i = hl & (R - 1);
            uint32_t m = mask[0];
#pragma unroll
            for (int x = 1; x < R; ++x) m = i == x ? mask[x] : m;
            cp_async_4(at + kSwigluBwdScales + (half * 2 * R + hl) * 4,
                       p.cs + static_cast<int64_t>(fb + (hl >= R ? p.nfb : 0)) * p.cs_stride + row0 + half + CastTile<T>::kStep * i,
                       (m >> (half & 31)) & 1u ? 4 : 0);
        }
        fetch_flags(advance(t));
        cp_async_commit();
    };

    uint32_t tile = blockIdx.x;
    if (tile >= p.tiles) return;
    uint32_t mask[R];
    bool next_live = false;
    At here{tile / p.nfb, tile % p.nfb};
    fetch_flags(here);
    cp_async_commit();
    cp_async_wait<0>();
    flags(mask, next_live);
    fetch(here, mask, 0);
    for (int st = 0; tile < p.tiles; tile += gridDim.x, st ^= 1) {
        const bool live = next_live;
        cp_async_wait<0>();
        __syncwarp();  // the scales were copied by other lanes
        if (tile + gridDim.x < p.tiles) {
            flags(mask, next_live);
            fetch(advance(here), mask, st ^ 1);
        }
        const int64_t rb = here.rb, row0 = rb * 128;
        const int fb = static_cast<int>(here.fb);
        here = advance(here);
        if (!live) continue;  // the same answer in every warp
        const uint32_t at = stage0 + st * kSwigluBwdStage;
        F8 dh[2][R], act[R];  // d gate and d up; a
        F8(&dg)[R] = dh[0], (&du)[R] = dh[1];
        const int col[2] = {fb * 128, p.F + fb * 128};
        float am = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            uint2 cg, cu;
            float sg, su;
            F8 g, u, d;
            const uint32_t codes = at + R * T * 16 + (2 * i * T + tid) * 8, scale = at + kSwigluBwdScales + (half * 2 * R + i) * 4;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(cg.x), "=r"(cg.y) : "r"(codes) : "memory");
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(cu.x), "=r"(cu.y) : "r"(codes + T * 8) : "memory");
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sg) : "r"(scale) : "memory");
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(su) : "r"(scale + R * 4) : "memory");
            bf16x8_to_f8(ld_shared_16(at + (i * T + tid) * 16), d);
            e4m3x8_to_f8(cg, g);
            e4m3x8_to_f8(cu, u);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                g[x] = __fmul2_rn(g[x], pair(sg));
                u[x] = __fmul2_rn(u[x], pair(su));
                const float2 s = sigmoid2(g[x]);
                const float2 silu = __fmul2_rn(g[x], s);
                const float2 t = __ffma2_rn(silu, __ffma2_rn(s, pair(-1.f), pair(1.f)), s);
                dg[i][x] = __fmul2_rn(__fmul2_rn(d[x], u[x]), t);
                du[i][x] = __fmul2_rn(d[x], silu);
                act[i][x] = __fmul2_rn(silu, u[x]);
                am = amax3(am, act[i][x].x, act[i][x].y);
            }
        }
        tile_column_max<T>(dg, cm[0]);
        tile_column_max<T>(du, cm[1]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        if (lane == 0) wm[tid >> 5] = am;
        maxima.arrive();
        tile_cast_rows<T, 2>(p.out, dh, row0, 2 * p.F, col);
        maxima.wait();
        tile_column_scale<T>(p.out, cm[0], cr[0], row0, col);
        am = wm[lane & (CastTile<T>::kWarps - 1)];
        joined.arrive();
#pragma unroll
        for (int o = CastTile<T>::kWarps / 2; o >= 1; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        am = fmaxf(am, 1e-4f);
        const float ra = __fdiv_rn(448.f, am);
        if (tid == 0) p.sb[static_cast<int64_t>(fb) * (p.rows / 128) + rb] = __fdiv_rn(am, 448.f);
        uint8_t* qa = p.Qa + (row0 + half) * p.F + fb * 128 + hl * 8;
#pragma unroll
        for (int i = 0; i < R; ++i, qa += static_cast<int64_t>(CastTile<T>::kStep) * p.F)
            *reinterpret_cast<uint2*>(qa) = e4m3x8(act[i], ra);
        joined.wait();
        tile_cast_columns<T>(p.out, dg, cr[0], row0, 2 * p.F, col[0]);
        tile_cast_columns<T>(p.out, du, cr[1], row0, 2 * p.F, col[1]);
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
    int rows;
};

// One CTA per 128 x 128 block, 8 threads to a row (16 codes each).  The
// block's maximum comes from the rows' largest codes: rounding code * scale
// keeps their order.  A NaN is no maximum.  6006 rows of 7168: 22.5 us, 3.9
// TB/s, half of the ALU and of the load latency showing in turns (a tile ahead
// by TMA or cp.async took 23.6 and 24.0 us).
__global__ void __launch_bounds__(kRecastThreads)
recast_128x128_kernel(const RecastParams p) {
    __shared__ float wm[kRecastThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const uint32_t rb = blockIdx.x / p.nkb;
    const int kb = static_cast<int>(blockIdx.x - rb * p.nkb);
    const int row0 = static_cast<int>(rb) * 128 + (tid >> 3);
    const int64_t at = static_cast<int64_t>(row0) * p.K + kb * 128 + (tid & 7) * 16, step = 32ll * p.K;
    const float* sa = p.sa + static_cast<int64_t>(kb) * p.sa_stride + row0;
    uint4 v[4];
    float s[4];
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool there = p.m_indices == nullptr || p.m_indices[row0 + 32 * i] >= 0;
        any |= there;
        v[i] = there ? ld_once_16(p.Q + at + i * step) : make_uint4(0, 0, 0, 0);
        s[i] = there ? sa[32 * i] : 0.f;
    }
    __half2 h[4][8];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        __half2 m = __half2(__half(0.f), __half(0.f));
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            h[i][x] = e4m3x2_to_half2(x & 1 ? w[x / 2] >> 16 : w[x / 2]);
            m = __hmax2(m, __habs2(h[i][x]));
        }
        const float2 f = __half22float2(m);
        a = fmaxf(a, fabsf(__fmul_rn(fmaxf(f.x, f.y), s[i])));
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
        for (int o = 0; o < 2; ++o) {
            F8 f;
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = __fmul2_rn(__half22float2(h[i][4 * o + x]), pair(s[i]));
            q[o] = e4m3x8(f, r);
        }
        *reinterpret_cast<uint4*>(p.Qb + at + i * step) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
    }
}

}  // namespace dg
