// dg_norm.cuh -- sm_100a kernels of the norms around a transformer block: the
// block's output is normalised (or not), scaled per column, per token and as a
// whole, and added to the residual stream; the stream's own norm, for the next
// block, comes out of the same pass, as bf16, as the next GEMM's e4m3 operand, or
// both.  Times are of one B200 in graph replays over inputs larger than L2.
//
//   z = c gate[t] w_post y r_y        r_y = 1 / sqrt(mean y^2 + eps), or 1
//   u = x + z
//   h = u r_u w_pre                   r_u = 1 / sqrt(mean u^2 + eps)
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_cast.cuh"
#include "dg_moe.cuh"
#include "dg_ptx.cuh"

namespace dg {

constexpr int kNormMaxColumns = 16384;
constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxParts = 148;  // rows of partial weight gradients, at most

// Eight consecutive values of the residual stream, bf16 or FP32.
__device__ __forceinline__ void load_f8(const uint16_t* p, F8& f) { bf16x8_to_f8(ld_once_16(p), f); }
__device__ __forceinline__ void load_f8(const float* p, F8& f) {
    const uint4 a = ld_once_16(p), b = ld_once_16(p + 4);
    f[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    f[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    f[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
    f[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
}
__device__ __forceinline__ void store_f8(uint16_t* p, const F8& f) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                                              pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ void store_f8(float* p, const F8& f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
// Eight weights of a column run, ones without any.
__device__ __forceinline__ void load_weights(const float* w, int c, F8& f) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(1.f, 1.f);
        return;
    }
    const float4 a = *reinterpret_cast<const float4*>(w + c), b = *reinterpret_cast<const float4*>(w + c + 4);
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ float dot_f8(const F8& a, const F8& b, float s) {
    float2 d = make_float2(s, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __ffma2_rn(a[i], b[i], d);
    return d.x + d.y;
}

// Sums of K values over the CTA, the same in every thread: warps first, then the
// warps' sums in warp order.  `part` holds 32 K floats and is not written again
// before the next but one call's barrier (callers alternate two of them).
template <int K>
__device__ __forceinline__ void cta_sum(float (&v)[K], float* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) part[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = lane < warps ? part[k * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

struct NormParams {
    void* U;               // [T][N] or null
    uint16_t* H;           // [T][N] or null
    uint8_t* Q;            // [T][N] or null, scales like dg_to_fp8_1x128's
    float* sq;
    float* rstd;           // [T][2] or null
    const void* X;         // [T][N] or null: zeros
    const uint16_t* Y;     // [T][N] or null: no block output
    const float* w_post;   // [N] or null
    const float* gate;     // [T] or null
    const float* w_pre;    // [N] or null
    int64_t sq_stride;
    int T, N;
    int post_norm;
    float scale, eps;
};

// One CTA a row at a time; thread i holds the runs of 8 columns i, i + threads,
// ... of it, so a half-warp holds whole 1x128 tiles.
template <typename XT, int CH>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_residual_kernel(const NormParams p) {
    __shared__ float part[4][32];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, runs = p.N / 8;
    const float inv_n = 1.f / static_cast<float>(p.N);
    int turn = 0;
    for (int t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        const int64_t row = static_cast<int64_t>(t) * p.N;
        F8 u[CH], y[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = tid + i * blockDim.x;
#pragma unroll
            for (int x = 0; x < 4; ++x) u[i][x] = y[i][x] = make_float2(0.f, 0.f);
            if (c < runs) {
                if (p.X != nullptr) load_f8(static_cast<const XT*>(p.X) + row + c * 8, u[i]);
                if (p.Y != nullptr) load_f8(p.Y + row + c * 8, y[i]);
            }
        }
        float ry = 1.f;
        if (p.Y != nullptr) {
            if (p.post_norm) {
                float s[1] = {0.f};
#pragma unroll
                for (int i = 0; i < CH; ++i) s[0] = dot_f8(y[i], y[i], s[0]);
                cta_sum<1>(s, part[2 * turn]);
                ry = __frsqrt_rn(fmaf(s[0], inv_n, p.eps));
            }
            float k = p.scale * ry;
            if (p.gate != nullptr) k *= p.gate[t];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = tid + i * blockDim.x;
                if (c >= runs) continue;
                F8 w;
                load_weights(p.w_post, c * 8, w);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    u[i][x] = __ffma2_rn(__fmul2_rn(y[i][x], make_float2(k, k)), w[x], u[i][x]);
            }
        }
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            s[0] = dot_f8(u[i], u[i], s[0]);
            const int c = tid + i * blockDim.x;
            if (p.U != nullptr && c < runs) store_f8(static_cast<XT*>(p.U) + row + c * 8, u[i]);
        }
        cta_sum<1>(s, part[2 * turn + 1]);
        const float ru = __frsqrt_rn(fmaf(s[0], inv_n, p.eps));
        if (p.rstd != nullptr && tid == 0) *reinterpret_cast<float2*>(p.rstd + 2ll * t) = make_float2(ry, ru);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = tid + i * blockDim.x;
            F8 h, w;
            if (c < runs) load_weights(p.w_pre, c * 8, w);
#pragma unroll
            for (int x = 0; x < 4; ++x) h[x] = c < runs ? __fmul2_rn(__fmul2_rn(u[i][x], make_float2(ru, ru)), w[x]) : make_float2(0.f, 0.f);
            if (p.H != nullptr && c < runs) store_f8(p.H + row + c * 8, h);
            if (p.Q != nullptr) {
                float a = amax8(h);
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                a = fmaxf(a, 1e-4f);
                if (c < runs) {
                    *reinterpret_cast<uint2*>(p.Q + row + c * 8) = e4m3x8(h, __fdiv_rn(448.f, a));
                    if ((tid & 15) == 0) p.sq[(c >> 4) * p.sq_stride + t] = __fdiv_rn(a, 448.f);
                }
            }
        }
    }
}

// ------------------------------------------------------------- backward ----

struct NormBwdParams {
    void* dX;              // [T][N] or null
    uint16_t* dY;          // [T][N] or null
    float* dgate;          // [T] or null
    float* part_post;      // [gridDim.x][N] partial sums of the weights' gradients, or null
    float* part_pre;
    const void* dU;        // [T][N] or null: zeros
    const uint16_t* dH;    // [T][N] or null: zeros
    const void* U;         // [T][N]
    const uint16_t* Y;     // [T][N] or null
    const float* rstd;     // [T][2]
    const float* w_post;   // [N] or null
    const float* gate;     // [T] or null
    const float* w_pre;    // [N] or null
    int T, N;
    int post_norm;
    float scale;
};

// With a = u r_u and b = y r_y, both normalised rows:
//   du = dU + r_u (w_pre dH - a mean(a w_pre dH)),  dX = du
//   d  = c gate du:  dw_post += d b,  dw_pre += dH a,  dgate = c sum(du w_post b)
//   dY = r_y (w_post d - b mean(b w_post d)), or w_post d without the norm
// One CTA a row at a time, thread layout as in the forward kernel; the weights'
// gradients of a thread's columns stay in its registers until the last row.
template <typename XT, int CH>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_residual_bwd_kernel(const NormBwdParams p) {
    __shared__ float part[4][32];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, runs = p.N / 8;
    const float inv_n = 1.f / static_cast<float>(p.N);
    F8 dpost[CH], dpre[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) dpost[i][x] = dpre[i][x] = make_float2(0.f, 0.f);
    int turn = 0;
    for (int t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        const int64_t row = static_cast<int64_t>(t) * p.N;
        const float2 r = *reinterpret_cast<const float2*>(p.rstd + 2ll * t);
        const float2 ry = make_float2(r.x, r.x), ru = make_float2(r.y, r.y);
        const float k = p.gate != nullptr ? p.scale * p.gate[t] : p.scale;
        F8 d[CH], a[CH], b[CH], g[CH];
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = tid + i * blockDim.x;
#pragma unroll
            for (int x = 0; x < 4; ++x) d[i][x] = a[i][x] = b[i][x] = g[i][x] = make_float2(0.f, 0.f);
            if (c < runs) {
                if (p.dU != nullptr) load_f8(static_cast<const XT*>(p.dU) + row + c * 8, d[i]);
                if (p.dH != nullptr) load_f8(p.dH + row + c * 8, g[i]);
                load_f8(static_cast<const XT*>(p.U) + row + c * 8, a[i]);
                if (p.Y != nullptr) load_f8(p.Y + row + c * 8, b[i]);
                F8 w;
                load_weights(p.w_pre, c * 8, w);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    a[i][x] = __fmul2_rn(a[i][x], ru);
                    b[i][x] = __fmul2_rn(b[i][x], ry);
                    dpre[i][x] = __ffma2_rn(g[i][x], a[i][x], dpre[i][x]);
                    g[i][x] = __fmul2_rn(g[i][x], w[x]);
                }
                s[0] = dot_f8(a[i], g[i], s[0]);
            }
        }
        cta_sum<1>(s, part[2 * turn]);
        const float mean = s[0] * inv_n;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = tid + i * blockDim.x;
            if (c >= runs) continue;
            F8 w;
            load_weights(p.w_post, c * 8, w);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 in = __ffma2_rn(a[i][x], make_float2(-mean, -mean), g[i][x]);
                d[i][x] = __ffma2_rn(ru, in, d[i][x]);
            }
            if (p.dX != nullptr) store_f8(static_cast<XT*>(p.dX) + row + c * 8, d[i]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                dpost[i][x] = __ffma2_rn(__fmul2_rn(d[i][x], make_float2(k, k)), b[i][x], dpost[i][x]);
                d[i][x] = __fmul2_rn(d[i][x], w[x]);
            }
            s[0] = dot_f8(d[i], b[i], s[0]);
        }
        if (p.Y == nullptr) continue;
        cta_sum<1>(s, part[2 * turn + 1]);
        if (p.dgate != nullptr && tid == 0) p.dgate[t] = p.scale * s[0];
        if (p.dY == nullptr) continue;
        const float sub = p.post_norm ? -s[0] * inv_n : 0.f;
        const float kr = k * r.x;  // r_y is 1 without the norm
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = tid + i * blockDim.x;
            if (c >= runs) continue;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                d[i][x] = __fmul2_rn(__ffma2_rn(b[i][x], make_float2(sub, sub), d[i][x]), make_float2(kr, kr));
            store_f8(p.dY + row + c * 8, d[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = tid + i * blockDim.x;
        if (c >= runs) continue;
        const int64_t at = static_cast<int64_t>(blockIdx.x) * p.N + c * 8;
        if (p.part_post != nullptr) store_f8(p.part_post + at, dpost[i]);
        if (p.part_pre != nullptr) store_f8(p.part_pre + at, dpre[i]);
    }
}

// Sums over the rows of up to two [parts][N] arrays, in row order: the last step
// of the sums over tokens.  A warp takes 32 columns of one array.
struct ColumnSumParams {
    float* out[2];
    const float* in[2];
    int parts, N;
};
constexpr int kColumnSumThreads = 256;

// A CTA takes 32 columns of an array: its 8 warps every eighth row, then the
// warps' sums in order.
__global__ void __launch_bounds__(kColumnSumThreads)
column_sum_kernel(const ColumnSumParams p) {
    __shared__ float part[kColumnSumThreads / 32][32];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    const float* in = p.in[blockIdx.y];
    float* out = p.out[blockIdx.y];
    if (out == nullptr) return;
    float s = 0.f;
    if (c < p.N) {
#pragma unroll 4
        for (int r = warp; r < p.parts; r += kColumnSumThreads / 32) s += in[static_cast<int64_t>(r) * p.N + c];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < p.N) {
#pragma unroll
        for (int w = 1; w < kColumnSumThreads / 32; ++w) s += part[w][lane];
        out[c] = s;
    }
}

}  // namespace dg
