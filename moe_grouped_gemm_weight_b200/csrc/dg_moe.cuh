// dg_moe.cuh -- sm_100a kernels between the routing and the grouped GEMMs:
// the cast of the tokens into the rows of the grouped layout, the weighted sum
// of the experts' rows per token, and its gradient.  Times are of one B200 in
// graph replays over inputs larger than L2.
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

// Eight values as four pairs: products of pairs are one instruction.
using F8 = float2[4];

__device__ __forceinline__ void bf16x8_to_f8(const uint4& v, F8& f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
// max(|a|, |b|, |c|), NaN not counted.
__device__ __forceinline__ float amax3(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float amax8(const F8& f) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = amax3(a, f[i].x, f[i].y);
    return a;
}
__device__ __forceinline__ uint2 pack_e4m3x8(const F8& y) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __nv_cvt_float2_to_fp8x2(y[i], __NV_SATFINITE, __NV_E4M3);
    return make_uint2(__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410));
}
// e4m3x8 of dg_cast.cuh, the same roundings.
__device__ __forceinline__ uint2 e4m3x8(const F8& f, float r) {
    F8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fmul2_rn(f[i], make_float2(r, r));
    return pack_e4m3x8(y);
}

__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Maxima of R values over the 16 lanes of a half-warp, spread: lane hl gets
// that of a[hl % R].  Each step halves the values that a lane carries, so R
// values cost R - 1 + log2(16 / R) exchanges instead of 4 R.
template <int R>
__device__ __forceinline__ float half_warp_max_spread(float (&a)[R]) {
    const int hl = threadIdx.x & 15;
#pragma unroll
    for (int n = R, bit = 1; n > 1; n >>= 1, bit <<= 1) {
        const bool hi = hl & bit;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = hi ? a[2 * i + 1] : a[2 * i], send = hi ? a[2 * i] : a[2 * i + 1];
            a[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, bit));
        }
    }
#pragma unroll
    for (int bit = R; bit < 16; bit <<= 1) a[0] = fmaxf(a[0], __shfl_xor_sync(0xffffffffu, a[0], bit));
    return a[0];
}

// Scales of R tiles (R <= 8) from their spread maxima, one division a lane:
// lane i < R gets 448 / amax of tile i, lane R + i amax / 448 of tile i.
template <int R>
__device__ __forceinline__ float spread_scale(float amax) {
    const bool back = threadIdx.x & R;
    amax = fmaxf(amax, 1e-4f);
    return __fdiv_rn(back ? amax : 448.f, back ? 448.f : amax);
}

// Place of row r's scale of K block 0; block kb lies kb * stride behind it.
// Groups of group_rows rows have scale arrays of their own (masked layout);
// group_rows == 0: one for all rows.
__device__ __forceinline__ int64_t scale_base(int r, int nkb, int stride, int group_rows) {
    if (group_rows == 0) return r;
    const int g = r / group_rows;
    return static_cast<int64_t>(g) * nkb * stride + (r - g * group_rows);
}

// ------------------------------------------------------------- dispatch ----

struct DispatchParams {
    uint8_t* Q;            // [rows][K]
    float* sa;
    const uint16_t* X;     // [T][K]
    const int32_t* row_of; // [T][k]
    int T, k, K, nkb;
    int sa_stride, group_rows;
    int rows;
    int tokens;            // tokens per CTA and step: 1, 2, 4, 8 or 16
    uint32_t items;        // token groups times K block groups
};

// The cast of dg_cast.cuh's cast_1x128_kernel, a token read and cast once and
// written to each of its k rows: a half-warp of a CTA takes NB K blocks of a
// token, as many half-warps side by side as the token has blocks for, so that
// the copies of a row are written in long runs.  Lane j of the half-warp keeps
// the token's rows j and j + 16 and writes their scales.
//
// 4096 tokens of 7168 to 32768 rows: 60 us, 5.0 TB/s.  Bound by the sectors
// written to L2: 7.3 M full ones of codes, and 1.8 M for one 4-byte scale each,
// since a token's rows lie in k segments (49 us without the scales).
template <int NB>
__global__ void __launch_bounds__(kCastThreads)
dispatch_1x128_kernel(const DispatchParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15;
    const int base = threadIdx.x & 16;  // first lane of this half-warp
    const int span = kCastRowsPerCta / p.tokens;  // half-warps side by side on a token
    const uint32_t kb_groups = (p.nkb + NB * span - 1) / (NB * span);
    for (uint32_t it = blockIdx.x; it < p.items; it += gridDim.x) {
        const uint32_t tg = it / kb_groups;
        const int t = static_cast<int>(tg) * p.tokens + half / span;
        const int kb0 = (static_cast<int>(it - tg * kb_groups) * span + half % span) * NB;
        const bool there = t < p.T;
        const uint16_t* xr = p.X + static_cast<int64_t>(t) * p.K + kb0 * 128 + hl * 8;
        uint4 v[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            v[b] = there && kb0 + b < p.nkb ? ld_once_16(xr + b * 128) : make_uint4(0, 0, 0, 0);
        int row[2] = {-1, -1};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = hl + 16 * h;
            if (there && j < p.k) row[h] = p.row_of[static_cast<int64_t>(t) * p.k + j];
            if (row[h] >= p.rows) row[h] = -1;
        }
        F8 f[NB];
        float a[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            bf16x8_to_f8(v[b], f[b]);
            a[b] = amax8(f[b]);
        }
        const float sc = spread_scale<NB>(half_warp_max_spread<NB>(a));
        uint2 q[NB];
        float s[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            q[b] = e4m3x8(f[b], __shfl_sync(0xffffffffu, sc, base + b));
            s[b] = __shfl_sync(0xffffffffu, sc, base + NB + b);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (row[h] < 0) continue;
            float* to = p.sa + scale_base(row[h], p.nkb, p.sa_stride, p.group_rows) + static_cast<int64_t>(kb0) * p.sa_stride;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (kb0 + b < p.nkb) to[static_cast<int64_t>(b) * p.sa_stride] = s[b];
        }
        uint8_t* qc = p.Q + kb0 * 128 + hl * 8;
        __syncwarp();
        for (int j = 0; j < p.k; ++j) {
            const int to = __shfl_sync(0xffffffffu, j < 16 ? row[0] : row[1], base + (j & 15));
            if (to < 0) continue;
            uint8_t* qr = qc + static_cast<int64_t>(to) * p.K;
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
// loads in flight together, FP32 sums in slot order.  Bound by HBM: 4096 tokens
// with 29500 rows of 7168 in 77 us, 6.2 TB/s.
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

// A CTA of T threads holds a 128 x 128 tile of a gradient in registers:
// half-warp h (of T / 16) the rows h + (T / 16) i, lane hl of it columns
// 8 hl .. 8 hl + 7.  Both casts that a backward pass needs come from the same
// values: a scale per row (1x128, the input gradient's operand) and a scale
// per column (128x1, the weight gradient's, whose K is the rows).
template <int T>
struct CastTile {
    static constexpr int kRows = 128 * 16 / T;   // rows per thread
    static constexpr int kStep = T / 16;         // between a thread's rows
    static constexpr int kWarps = T / 32;
    static constexpr int kMatrices = T / 256;    // joined at once, two threads to a column
    static constexpr int kStride = 144;          // of the warps' maxima: the join's reads hit all banks
};

struct TileOut {
    uint8_t* Qr;   // [rows][N], scales sr[kb * sr_stride + row]
    float* sr;
    uint8_t* Qc;   // [rows][N], scales sc[(row / 128) * sc_stride + column]
    float* sc;
    int64_t sr_stride, sc_stride;
};

// 1x128: each half-warp has whole rows of the tile.  M matrices at once (at
// columns col[m] of the output), so that a lane divides once for all their
// scales.
template <int T, int M>
__device__ __forceinline__ void tile_cast_rows(const TileOut& o, const F8 (&v)[M][CastTile<T>::kRows], int64_t row0, int N,
                                               const int (&col)[M]) {
    constexpr int R = CastTile<T>::kRows, A = M * R;
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15, base = threadIdx.x & 16;
    float a[A];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < R; ++i) a[m * R + i] = amax8(v[m][i]);
    const float s = spread_scale<A>(half_warp_max_spread<A>(a));
    if (hl >= A && hl < 2 * A) {
        const int m = (hl - A) / R, i = (hl - A) % R;
        int c = col[0];
#pragma unroll
        for (int x = 1; x < M; ++x) c = m == x ? col[x] : c;
        o.sr[static_cast<int64_t>(c >> 7) * o.sr_stride + row0 + half + CastTile<T>::kStep * i] = s;
    }
    const int64_t step = static_cast<int64_t>(CastTile<T>::kStep) * N;
    uint8_t* row = o.Qr + (row0 + half) * N + hl * 8;
#pragma unroll
    for (int i = 0; i < R; ++i, row += step)
#pragma unroll
        for (int m = 0; m < M; ++m)
            *reinterpret_cast<uint2*>(row + col[m]) = e4m3x8(v[m][i], __shfl_sync(0xffffffffu, s, base + m * R + i));
}

// 128x1, first part: the warps' column maxima into cm[warp][kStride].  The two
// half-warps exchange four columns each.
template <int T>
__device__ __forceinline__ void tile_column_max(const F8 (&v)[CastTile<T>::kRows], float* cm) {
    const int warp = threadIdx.x >> 5, hl = threadIdx.x & 15;
    const bool hi = threadIdx.x & 16;
    float m[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        m[x] = 0.f;
#pragma unroll
        for (int i = 0; i < CastTile<T>::kRows; i += 2)
            m[x] = x & 1 ? amax3(m[x], v[i][x / 2].y, v[i + 1][x / 2].y) : amax3(m[x], v[i][x / 2].x, v[i + 1][x / 2].x);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float keep = hi ? m[4 + x] : m[x], send = hi ? m[x] : m[4 + x];
        m[x] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 16));
    }
    *reinterpret_cast<float4*>(cm + warp * CastTile<T>::kStride + hl * 8 + (hi ? 4 : 0)) = make_float4(m[0], m[1], m[2], m[3]);
}

// Second part, after a barrier: two threads to a column of the T / 256 matrices
// (cm and cr one behind the other) join the warps' maxima; one leaves 448 /
// amax in cr, the other writes the scale.
template <int T>
__device__ __forceinline__ void tile_column_scale(const TileOut& o, const float* cm, float* cr, int64_t row0,
                                                  const int (&col)[CastTile<T>::kMatrices]) {
    const int c = (threadIdx.x >> 1) & 127, m = threadIdx.x >> 8, part = threadIdx.x & 1;
    const float* mine = cm + m * CastTile<T>::kWarps * CastTile<T>::kStride + c;
    float a = 1e-4f;
#pragma unroll
    for (int w = 0; w < CastTile<T>::kWarps; w += 2) a = fmaxf(a, mine[(w + part) * CastTile<T>::kStride]);
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const float s = __fdiv_rn(part ? a : 448.f, part ? 448.f : a);
    if (part) {
        o.sc[(row0 / 128) * o.sc_stride + (CastTile<T>::kMatrices > 1 && m ? col[CastTile<T>::kMatrices - 1] : col[0]) + c] = s;
    } else {
        cr[m * 128 + c] = s;
    }
}

// Third part, after another barrier.
template <int T>
__device__ __forceinline__ void tile_cast_columns(const TileOut& o, const F8 (&v)[CastTile<T>::kRows],
                                                  const float* cr, int64_t row0, int N, int col0) {
    const int half = threadIdx.x >> 4, hl = threadIdx.x & 15;
    const float4 r0 = *reinterpret_cast<const float4*>(cr + hl * 8), r1 = *reinterpret_cast<const float4*>(cr + hl * 8 + 4);
    const F8 r = {make_float2(r0.x, r0.y), make_float2(r0.z, r0.w), make_float2(r1.x, r1.y), make_float2(r1.z, r1.w)};
    uint8_t* q = o.Qc + (row0 + half) * N + col0 + hl * 8;
    const int64_t step = static_cast<int64_t>(CastTile<T>::kStep) * N;
#pragma unroll
    for (int i = 0; i < CastTile<T>::kRows; ++i, q += step) {
        F8 y;
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] = __fmul2_rn(v[i][x], r[x]);
        *reinterpret_cast<uint2*>(q) = pack_e4m3x8(y);
    }
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// A CTA barrier in two halves, so that work between them hides the wait: each
// warp arrives, later each thread waits.  Several in turn order a tile's
// shared values as __syncthreads would.  The wait is bounded like every other.
struct SplitBarrier {
    uint64_t* bar;
    int* abort_flag;
    uint32_t phase = 0;
    __device__ __forceinline__ void arrive() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    }
    __device__ __forceinline__ void wait() {
        mbar_wait(bar, phase, abort_flag);
        phase ^= 1;
    }
};

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

constexpr int kCombineBwdThreads = 256;
constexpr int kCombineBwdStage = 2 * 128 * 128 * 2;  // bytes: a tile of dout and of Y

// dY[row] = w dout[t], cast both ways, and dw = <dout[t], Y[row]>.  A cluster
// of CTAs takes a block of 128 rows, each CTA a run of its 128-column tiles;
// the row sums of dw are joined through distributed shared memory in CTA
// order.  Rows without a slot count as zeros; a block without any is left.
//
// Each thread copies the 16-byte pieces that it will use itself to shared
// memory (cp.async), takes them into registers when they have landed and at
// once asks for the next tile's, so HBM works during the casts and no barrier
// guards the buffer.  Two CTAs of 256 threads an SM: with 512 threads each the
// issue slots fill better (56 against 47 %), but a tile takes a quarter more
// instructions, and the 64 registers spill a little: 217 us.
//
// 32768 rows of 7168: 207 us, 4.9 TB/s (the casts alone 170 us, without loads
// and stores).
__global__ void __launch_bounds__(kCombineBwdThreads, 2)
combine_bwd_kernel(const CombineBwdParams p) {
    constexpr int T = kCombineBwdThreads, R = CastTile<T>::kRows;
    extern __shared__ __align__(16) uint8_t stage_smem[];
    __shared__ __align__(16) float cm[CastTile<T>::kWarps * CastTile<T>::kStride];
    __shared__ __align__(16) float cr[128];
    __shared__ float part[128];
    __shared__ uint64_t bars[2];
    __shared__ int abort_flag;
    const int tid = threadIdx.x, half = tid >> 4, hl = tid & 15;
    if (tid == 0) {
        mbar_init(&bars[0], CastTile<T>::kWarps);
        mbar_init(&bars[1], CastTile<T>::kWarps);
        abort_flag = 0;
        fence_mbar_init();
    }
    SplitBarrier maxima{&bars[0], &abort_flag}, joined{&bars[1], &abort_flag};
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t rank = cluster_ctarank(), nctas = cluster_nctarank();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / nctas) * 128;

    // Slots that have no row have no gradient.
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * T + tid; s < p.S; s += static_cast<int64_t>(gridDim.x) * T) {
        const int r = p.row_of[s];
        if (r < 0 || r >= p.rows) p.dw[s] = 0.f;
    }

    int token[R];  // -1: no slot
    float w[R], dot[R];
    bool any = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int s = p.slot_of[row0 + half + CastTile<T>::kStep * i];
        const bool ok = s >= 0 && s < p.S;
        token[i] = ok ? s / p.k : -1;
        w[i] = ok ? p.w[s] : 0.f;
        dot[i] = 0.f;
        any |= ok;
    }
    if (!__syncthreads_or(any)) return;  // the same answer in every CTA of the cluster

    const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / nctas);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / nctas);
    const uint32_t stage = smem_u32(stage_smem) + tid * 16;
    const uint16_t* y0 = p.Y + (row0 + half) * p.N + hl * 8;
    const int64_t step = static_cast<int64_t>(CastTile<T>::kStep) * p.N;
    auto fetch = [&](int kb) {
        const uint16_t* y = y0 + kb * 128;
        const uint16_t* d = p.dout + kb * 128 + hl * 8;
#pragma unroll
        for (int i = 0; i < R; ++i, y += step) {
            const uint32_t bytes = token[i] >= 0 ? 16 : 0;  // missing rows are zeros
            cp_async_16(stage + 2 * i * T * 16, d + static_cast<int64_t>(max(token[i], 0)) * p.N, bytes);
            cp_async_16(stage + (2 * i + 1) * T * 16, y, bytes);
        }
        cp_async_commit();
    };
    fetch(kb0);
    for (int kb = kb0; kb < kb1; ++kb) {
        cp_async_wait<0>();
        F8 tile[1][R];
        F8(&v)[R] = tile[0];
        const int col[1] = {kb * 128};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            F8 y;
            bf16x8_to_f8(ld_shared_16(stage + 2 * i * T * 16), v[i]);
            bf16x8_to_f8(ld_shared_16(stage + (2 * i + 1) * T * 16), y);
            float2 d = make_float2(dot[i], 0.f);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                d = __ffma2_rn(v[i][x], y[x], d);
                v[i][x] = __fmul2_rn(v[i][x], make_float2(w[i], w[i]));
            }
            dot[i] = d.x + d.y;
        }
        tile_column_max<T>(v, cm);
        maxima.arrive();
        if (kb + 1 < kb1) fetch(kb + 1);
        maxima.wait();
        tile_column_scale<T>(p.out, cm, cr, row0, col);
        joined.arrive();
        tile_cast_rows<T, 1>(p.out, tile, row0, p.N, col);
        joined.wait();
        tile_cast_columns<T>(p.out, v, cr, row0, p.N, kb * 128);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float d = half_warp_sum(dot[i]);
        if (hl == 0) part[half + CastTile<T>::kStep * i] = d;
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
