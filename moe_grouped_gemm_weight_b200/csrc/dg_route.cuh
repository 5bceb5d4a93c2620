// dg_route.cuh -- sm_100a routing kernels: the choice of k experts per token,
// its gradient, and the grouped layout that the choice leads to.
//
// Scores s = softmax(l) or sigmoid(l) over the E logits of a token; choice
// values c = s + bias.  The result is that of exact arithmetic: an order
// decided in FP32 is kept only where neighbours differ by more than FP32 can
// have moved them, else the token is decided again in FP64.
#pragma once

#include <cuda_bf16.h>
#include <float.h>
#include <stdint.h>

#include "dg_ptx.cuh"

namespace dg {

constexpr int kRouteWarps = 8;
// CTAs resident per SM where a lane holds up to `epl` experts.
constexpr int route_ctas(int epl) { return epl <= 8 ? 4 : epl <= 16 ? 2 : 1; }
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 16;       // lanes 0..k hold the k choices and the runner-up
constexpr int kRouteMaxGroups = 32;  // one lane at least per group
constexpr float kRouteEps = 1e-20f;  // added to the sum that renormalised weights are divided by

struct RouteParams {
    const void* logits;  // [T][E]
    const float* bias;   // [E] or null
    int32_t* idx;        // [T][k]
    float* w;            // [T][k]
    int T, E, k;
    int groups, keep, gtop;
    int gsize;            // E / groups
    uint32_t gsize_magic; // e / gsize == (e * gsize_magic) >> 20 for e < 1024
    int flat;             // ceil(E / 32)
    int per;              // experts per lane, at most
    int span, span_shift; // groups with lanes of their own: 1 << span_shift lanes hold the `span` experts of one
    int group_lanes;      // ... there are such
    int vec;              // every lane full, rows and bias 16-byte aligned: wide loads
    int softmax, renorm;
    float scale;

    // The first expert of a lane, and how many it has (none: <= 0).
    template <bool kSpans>
    __device__ __forceinline__ int first_of(int lane) const {
        return kSpans ? (lane >> span_shift) * span + (lane & ((1 << span_shift) - 1)) * per : lane * per;
    }
    template <bool kSpans>
    __device__ __forceinline__ int count_of(int lane) const {
        if (!kSpans) return min(per, E - lane * per);
        return (lane >> span_shift) * span < E ? min(per, span - (lane & ((1 << span_shift) - 1)) * per) : 0;
    }
};

__device__ __forceinline__ float logit_at(const float* p) { return *p; }
__device__ __forceinline__ float logit_at(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

// N consecutive floats with the widest loads (the address is a multiple of the
// load's width).
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&f)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(f + i) = *reinterpret_cast<const float4*>(p + i);
    } else if constexpr (N == 2) {
        *reinterpret_cast<float2*>(f) = *reinterpret_cast<const float2*>(p);
    } else {
        f[0] = *p;
    }
}
// The N logits of a row that a lane holds, as they are in memory: turning bf16
// into floats waits for the load, so it is left to the next token's turn.
template <int N, typename L>
struct RawRow {
    static constexpr bool kPairs = sizeof(L) == 2 && N >= 2;        // wide loads: two to a word
    static constexpr int kChunk = N < 16 / static_cast<int>(sizeof(L)) ? N : 16 / static_cast<int>(sizeof(L));
    uint32_t w[N];

    // Chunks of a wide load's kChunk logits, `step` logits apart.
    __device__ __forceinline__ void load_wide(const L* p, int step) {
        constexpr int kWords = kPairs ? kChunk / 2 : kChunk;
#pragma unroll
        for (int c = 0; c < N / kChunk; ++c) {
            uint32_t* to = w + c * kWords;
            const L* at = p + c * step;
            if constexpr (kWords == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(at);
                to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
            } else if constexpr (kWords == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(at);
                to[0] = v.x, to[1] = v.y;
            } else if constexpr (kPairs) {
                to[0] = *reinterpret_cast<const uint32_t*>(at);
            } else {
                to[0] = bits(at);
            }
        }
    }
    // One by one, -inf where there is none.
    __device__ __forceinline__ void load_one(int i, bool there, const L* p) {
        w[i] = there ? bits(p) : sizeof(L) == 2 ? 0xFF80u : 0xFF800000u;
    }
    __device__ __forceinline__ void get(bool wide, float (&f)[N]) const {
        if constexpr (sizeof(L) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
        } else if (kPairs && wide) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i] << 16);
        }
    }

   private:
    static __device__ __forceinline__ uint32_t bits(const float* p) { return __float_as_uint(*p); }
    static __device__ __forceinline__ uint32_t bits(const uint16_t* p) { return *p; }
};

// Order-preserving integer key of a double: a < b <=> key(a) < key(b); both
// zeros share a key, NaN is above everything, and 0 is left for "none".
__device__ __forceinline__ unsigned long long order_key(double v) {
    if (v != v) return ~0ull;
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
    return (u >> 63) ? ~u : (u | (1ull << 63));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_min(float v) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// Maximum of 64-bit keys: the upper halves, then the lower ones that share it.
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return static_cast<unsigned long long>(hi) << 32 | lo;
}

// For choices, which look again where FP32 cannot tell, and the sum that softmax
// scores are divided by, where a term counts by its share: exp and the sigmoid
// by the special-function unit alone, without the care for subnormal numbers:
// relative error 2^-22 and |x| 2^-24 for the argument's rounding; absolute error
// of the sigmoid below 2^-22.  (The sum by exp_results below: the weights no
// nearer to 64 bits, 16384 x 256 5 % slower.)
__device__ __forceinline__ float exp_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.f + exp_fast(-x)); }
// For results.  Exponentials of N numbers up to zero: 2^t (1 + lo ln 2) with t the
// rounded x log2(e) and lo what the product and the constant's rounding leave of
// it, so the relative error is 5 2^-24 however low x is.  Results below 2^-126 are
// zero (-126 stands for all lower x); a NaN stays one.
template <int N>
__device__ __forceinline__ void exp_results(float (&x)[N]) {
    constexpr float kLog2e = 1.4426950408889634f, kRest = static_cast<float>(1.4426950408889634074 - kLog2e);
    auto pair = [](float v) { return make_float2(v, v); };
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float2 v = make_float2(x[i], i + 1 < N ? x[i + 1] : 0.f);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(v.x) : "f"(-126.f));
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(v.y) : "f"(-126.f));
        float2 e = __fmul2_rn(v, pair(kLog2e));
        const float2 lo = __ffma2_rn(v, pair(kRest), __ffma2_rn(v, pair(kLog2e), make_float2(-e.x, -e.y)));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
        e = __fmul2_rn(e, __ffma2_rn(lo, pair(0.6931471805599453f), pair(1.f)));
        x[i] = e.x;
        if (i + 1 < N) x[i + 1] = e.y;
    }
}
// Relative error a few 2^-24.
__device__ __forceinline__ float sigmoid_f(float x) { return __frcp_rn(1.f + expf(-x)); }

// Signed integers in the order of finite or infinite floats, and back.
__device__ __forceinline__ int ordered_int(float f) {
    const int b = __float_as_int(f);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float ordered_float(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }
constexpr int kNoKey = -0x7FFFFFFF - 1;
constexpr int kLeastKey = static_cast<int>(0x80800000u);  // of the lowest finite float

// The choice in FP64 over the whole row, for a token that FP32 cannot decide
// even in part (a NaN, groups next to one another, a crowd at the border).
// Lane j < k returns the j-th expert, or -1.  Plain rather than fast.
template <int EPL, typename L>
__device__ __noinline__ int choose_exact(const RouteParams& p, const L* row) {
    const int lane = threadIdx.x & 31;
    double c[EPL];
    double m = -INFINITY, z = 1.0;
    if (p.softmax) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane * p.flat + i;
            if (i < p.flat && e < p.E) {
                const double l = logit_at(row + e);
                m = l > m ? l : m;
            }
        }
        for (int o = 16; o >= 1; o >>= 1) {
            const double x = __shfl_xor_sync(0xffffffffu, m, o);
            m = x > m ? x : m;
        }
        z = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane * p.flat + i;
            c[i] = i < p.flat && e < p.E ? exp(static_cast<double>(logit_at(row + e)) - m) : 0.0;
            z += c[i];
        }
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    unsigned long long key[EPL];  // of the choice value, 0: not eligible
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane * p.flat + i;
        key[i] = 0;
        if (i < p.flat && e < p.E) {
            const float l = logit_at(row + e);
            const float b = p.bias ? p.bias[e] : 0.f;
            const double s = p.softmax ? c[i] / z : 1.0 / (1.0 + exp(-static_cast<double>(l)));
            if (l != -INFINITY && b != -INFINITY) key[i] = order_key(s + static_cast<double>(b));
        }
    }
    if (p.groups > 1) {
        unsigned long long mine = 0;
        for (int g = 0; g < p.groups; ++g) {
            // The group's best is left out of the second round, by its index.
            unsigned long long top[2] = {0, 0};
            int taken = -1;
            for (int r = 0; r < p.gtop; ++r) {
                unsigned long long best = 0;
                int at = 0x7FFFFFFF;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane * p.flat + i;
                    const int grp = static_cast<int>((static_cast<uint32_t>(e) * p.gsize_magic) >> 20);
                    if (grp == g && e != taken && key[i] > best) { best = key[i]; at = e; }
                }
                const unsigned long long t = warp_max_u64(best);
                taken = __reduce_min_sync(0xffffffffu, best == t ? at : 0x7FFFFFFF);
                top[r] = t;
            }
            double sum = 0.0;
            for (int r = 0; r < 2; ++r) {
                if (top[r] == 0) continue;
                const unsigned long long u = top[r] >> 63 ? top[r] & ~(1ull << 63) : ~top[r];
                sum += __longlong_as_double(static_cast<long long>(u));
            }
            if (lane == g) mine = top[0] ? order_key(sum) : 0;
        }
        int rank = 0;
        for (int h = 0; h < p.groups; ++h) {
            const unsigned long long o = __shfl_sync(0xffffffffu, mine, h);
            rank += (o > mine || (o == mine && h < lane)) ? 1 : 0;
        }
        const uint32_t kept = __ballot_sync(0xffffffffu, lane < p.groups && mine != 0 && rank < p.keep);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const uint32_t grp = (static_cast<uint32_t>(lane * p.flat + i) * p.gsize_magic) >> 20;
            if (!((kept >> (grp & 31u)) & 1u)) key[i] = 0;
        }
    }
    if (!p.bias) {  // in the order of the logits themselves
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i]) key[i] = order_key(static_cast<double>(logit_at(row + lane * p.flat + i)));
    }
    int my = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) { best = key[i]; at = lane * p.flat + i; }
        const unsigned long long top = warp_max_u64(best);
        if (top == 0) break;
        at = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
        if (lane == j) my = at;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane * p.flat + i == at) key[i] = 0;
    }
    return my;
}

// The groups kept, decided in FP64 where groups have their own lanes: a lane's
// two best experts are e1 and e2 (-1: none; no third is close to them).  Returns
// whether this lane's group is kept.
template <typename L>
__device__ __noinline__ bool keep_groups_exact(const RouteParams& p, const L* row, int e1, int e2) {
    const int lane = threadIdx.x & 31, lanes = 1 << p.span_shift, g = lane >> p.span_shift;
    double m = 0.0, z = 1.0;
    if (p.softmax) {
        m = -INFINITY;
        z = 0.0;
        for (int i = lane; i < p.E; i += 32) m = fmax(m, static_cast<double>(logit_at(row + i)));
        for (int o = 16; o >= 1; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int i = lane; i < p.E; i += 32) z += exp(static_cast<double>(logit_at(row + i)) - m);
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    double v[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = i ? e2 : e1;
        if (e < 0) continue;
        const double l = logit_at(row + e);
        v[i] = (p.softmax ? exp(l - m) / z : 1.0 / (1.0 + exp(-l))) + (p.bias ? static_cast<double>(p.bias[e]) : 0.0);
    }
    double a = fmax(v[0], v[1]), b = fmin(v[0], v[1]);
    for (int o = lanes >> 1; o >= 1; o >>= 1) {
        const double xa = __shfl_xor_sync(0xffffffffu, a, o), xb = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmax(fmax(b, xb), fmin(a, xa));
        a = fmax(a, xa);
    }
    double sum = a + (p.gtop == 2 && b != -INFINITY ? b : 0.0);
    if (g >= p.groups) sum = -INFINITY;
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
        const double o = __shfl_sync(0xffffffffu, sum, h * lanes);
        rank += (o > sum || (o == sum && h < g)) ? 1 : 0;
    }
    return sum != -INFINITY && rank < p.keep;
}

// The order of n <= 32 candidates in FP64: lane j < n holds expert e.  Returns
// the lane's rank.
template <int EPL, typename L>
__device__ __noinline__ int rank_candidates(const RouteParams& p, const L* row, int n, int e) {
    const int lane = threadIdx.x & 31;
    double c = 0.0;
    if (p.softmax) {
        double m = -INFINITY, z = 0.0;
        for (int i = lane; i < p.E; i += 32) m = fmax(m, static_cast<double>(logit_at(row + i)));
        for (int o = 16; o >= 1; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int i = lane; i < p.E; i += 32) z += exp(static_cast<double>(logit_at(row + i)) - m);
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane < n) c = exp(static_cast<double>(logit_at(row + e)) - m) / z;
    } else if (lane < n) {
        c = 1.0 / (1.0 + exp(-static_cast<double>(logit_at(row + e))));
    }
    if (lane < n) c += static_cast<double>(p.bias[e]);
    int rank = 0;
    for (int h = 0; h < n; ++h) {
        const double o = __shfl_sync(0xffffffffu, c, h);
        const int oe = __shfl_sync(0xffffffffu, e, h);
        rank += (o > c || (o == c && oe < e)) ? 1 : 0;
    }
    return rank;
}

// The four largest of a lane's keys in falling order.
struct Top4 {
    int k[4];
    static __device__ __forceinline__ void order(int& a, int& b) {
        const int hi = max(a, b);
        b = min(a, b);
        a = hi;
    }
    template <int N>
    __device__ __forceinline__ void of(const int (&key)[N]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = i < N ? key[i] : kNoKey;
        if (N > 1) order(k[0], k[1]);
        if (N > 2) {
            order(k[2], k[3]);
            order(k[0], k[2]);
            order(k[1], k[3]);
            order(k[1], k[2]);
        }
#pragma unroll
        for (int q = 4; q < N; q += 4) {
            int o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = key[q + i];
            order(o[0], o[1]);
            order(o[2], o[3]);
            order(o[0], o[2]);
            order(o[1], o[3]);
            order(o[1], o[2]);
            // the four largest of both, then in order
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = max(k[i], o[3 - i]);
            order(k[0], k[2]);
            order(k[1], k[3]);
            order(k[0], k[1]);
            order(k[2], k[3]);
        }
    }
};

// Warps take tokens in turn, a token to a warp; the next token's logits are on
// their way meanwhile.  Lane after lane holds consecutive experts, lane i from
// i * per on; kSpans: groups do not end with a lane so, and each starts a lane of
// its own (65536 tokens of 408 experts in 8 groups: 100 us, against 160 with the
// groups read from shared memory, which is left for rows of over 512 experts
// whose lanes would hold more than 32).
//
// The choice works on keys: a value's leading bits in integer order, and in
// its low bits the expert's place (lane, then place in the lane, counted down),
// so that a maximum of keys is a value, its expert and the rule for ties at
// once.  A key costs three instructions, a lane's four largest in order four
// more, and a round of the choice one warp-wide maximum and a shift.  Where
// every chosen key is clearly above the next, the (k+1)-th included, the keys'
// order is the exact one.  Elsewhere the candidates are ordered by their FP32
// values, and by FP64 values where those are not clearly apart.  bf16 logits
// without a bias fit a key whole.
//
// 16384 tokens of 256 float32 logits, 8 groups, bias: 18.7 us on one B200 in
// graph replays (HBM alone 2.6 us), 668 instructions a token at 56 % of the
// issue slots, 20 of them spills (14 loads, 6 stores); 17.0 us without any FP64.
template <int EPL, bool kSpans, typename L>
__global__ void __launch_bounds__(kRouteWarps * 32, route_ctas(EPL))
route_topk_kernel(const RouteParams p) {
    constexpr int kMask = 32 * EPL - 1;  // a key's place bits
    constexpr bool kShort = sizeof(L) == 2;
    // Lanes that would hold more than 32 experts of a group: only rows of over 512 have such.
    const bool group_lanes = kSpans || EPL < 32 || p.group_lanes;
    extern __shared__ float route_smem[];  // groups without lanes of their own: E values per warp
    __shared__ uint16_t cand_smem[kRouteWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool biased = p.bias != nullptr;
    const int lane_bits = (31 - lane) * EPL;
    const int stride = gridDim.x * kRouteWarps;
    int t = blockIdx.x * kRouteWarps + warp;
    if (t >= p.T) return;

    auto load = [&](int token, RawRow<EPL, L>& v) {
        const L* row = static_cast<const L*>(p.logits) + static_cast<int64_t>(token) * p.E;
        if (p.vec) {
            v.load_wide(row + lane * EPL, RawRow<EPL, L>::kChunk);
        } else {
            const int e0 = p.first_of<kSpans>(lane), held = p.count_of<kSpans>(lane);
#pragma unroll
            for (int i = 0; i < EPL; ++i) v.load_one(i, i < held, row + e0 + i);
        }
    };
    float bias[EPL];
    RawRow<EPL, L> fetched;
    load(t, fetched);
    if (biased) {
        if (p.vec) {
            load_floats<EPL>(p.bias + lane * EPL, bias);
        } else {
            const int e0 = p.first_of<kSpans>(lane), held = p.count_of<kSpans>(lane);
#pragma unroll
            for (int i = 0; i < EPL; ++i) bias[i] = i < held ? p.bias[e0 + i] : -INFINITY;
        }
    }

    for (; t < p.T; t += stride) {
        const L* row = static_cast<const L*>(p.logits) + static_cast<int64_t>(t) * p.E;
        float v[EPL];  // logits, then (with a bias) choice values; -inf: not eligible
        fetched.get(p.vec, v);
        if (p.T - t > stride) load(t + stride, fetched);

        float mx = 0.f, rz = 1.f;
        if (p.softmax) {
            float m = v[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
            mx = warp_max(m);
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) z += exp_fast(v[i] - mx);
            rz = 1.f / warp_sum(z);
        }
        // FP32 moves the difference of two choice values by less than 2 slack and 2^-24
        // of each value (adding the bias), that of two sums of two by 4 slack and the
        // like.  A sigmoid moves by 2^-22 (see sigmoid_fast).  A softmax score moves by
        // 6 2^-24 of the largest, rz, for itself (exponential, argument, product).  The
        // sum's error (at most 36 additions, the exponentials' 2^-22, their arguments'
        // 6 2^-24) and the reciprocal's are a factor that all scores of a token share,
        // 47 2^-24 of the difference: 59 2^-24 rz in all, and 118 for the sums, where
        // slack allows 64 and 128.
        const float slack = p.softmax ? rz * 0x1p-19f : 0x1p-22f;
        auto apart_by = [&](float x, float y) {  // more than FP32 can have moved x - y
            return biased ? 2.f * slack + 0x1p-22f * (fabsf(x) + fabsf(y)) : 0.f;
        };
        auto score = [&](float x) { return p.softmax ? exp_fast(x - mx) * rz : sigmoid_fast(x); };

        if (biased) {
            float low = v[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) low = fminf(low, v[i]);
            if (low == -INFINITY) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) v[i] = v[i] == -INFINITY ? -INFINITY : score(v[i]) + bias[i];
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) v[i] = score(v[i]) + bias[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] += 0.f;  // one zero
        }
        // A NaN, or an infinite choice value: to be decided without shortcuts.
        float all = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) all += v[i];
        bool odd = !biased && !p.softmax ? all != all : !(all < INFINITY) || (rz != rz && mx != -INFINITY);
        odd = __any_sync(0xffffffffu, odd);

        bool in = true, sure = !odd;  // in: the lane's experts take part
        if (p.groups > 1 && sure) {
            float a = -INFINITY, b = -INFINITY;  // the two best choice values of the group
            int g, sh;                           // this lane's group, log2 of lanes per group
            // A choice value without a bias is the score of the logit.
            auto choice = [&](float x) { return x == -INFINITY || biased ? x : score(x); };
            if (group_lanes) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    b = fmaxf(b, fminf(a, v[i]));
                    a = fmaxf(a, v[i]);
                }
                a = choice(a);
                b = choice(b);
                sh = p.span_shift;
                g = lane >> sh;
            } else {
                // A power of two of lanes share a group in shared memory.
                float* cs = route_smem + warp * p.E;
                const int e0 = p.first_of<kSpans>(lane), held = p.count_of<kSpans>(lane);
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (i < held) cs[e0 + i] = choice(v[i]);
                __syncwarp();
                sh = 31 - __clz(32 / p.groups);
                g = lane >> sh;
                if (g < p.groups) {
                    const int lanes = 1 << sh;
                    // Each group starts at another place: the same places of groups of 32 share a bank.
                    const int turn = (g << sh) % p.gsize;
                    for (int n = lane & (lanes - 1); n < p.gsize; n += lanes) {
                        const float x = cs[g * p.gsize + (n + turn < p.gsize ? n + turn : n + turn - p.gsize)];
                        b = fmaxf(b, fminf(a, x));
                        a = fmaxf(a, x);
                    }
                }
            }
            for (int o = 1 << sh >> 1; o >= 1; o >>= 1) {
                const float xa = __shfl_xor_sync(0xffffffffu, a, o), xb = __shfl_xor_sync(0xffffffffu, b, o);
                b = fmaxf(fmaxf(b, xb), fminf(a, xa));
                a = fmaxf(a, xa);
            }
            // -inf marks a group without an expert, so a sum below every float (two soft
            // masks of the lowest one) stays at the lowest, level with all such sums.
            float sum = fmaxf(a + (p.gtop == 2 && b != -INFINITY ? b : 0.f), -FLT_MAX);
            if (a == -INFINITY || g >= p.groups) sum = -INFINITY;
            // The best groups, one value (mostly one group) a round.
            bool kept = false;
            float lo = -INFINITY, hi = warp_max(sum);
            int n = 0;
            while (n < p.keep && hi != -INFINITY) {
                lo = hi;
                kept |= sum == hi;
                n = __popc(__ballot_sync(0xffffffffu, kept)) >> sh;
                hi = warp_max(kept ? -INFINITY : sum);
            }
            // Certain when the worst kept group and the best other are clearly apart.
            if (n > p.keep || (hi != -INFINITY && !(lo - hi > 4.f * slack + 0x1p-21f * (fabsf(lo) + fabsf(hi))))) {
                // The lane's two best, if no third can take their place in FP64.
                float b1 = -INFINITY, b2 = -INFINITY, b3 = -INFINITY;
                int e1 = -1, e2 = -1;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const bool first = v[i] > b1, second = v[i] > b2;
                    b3 = fmaxf(b3, fminf(b2, v[i]));
                    e2 = first ? e1 : second ? p.first_of<kSpans>(lane) + i : e2;
                    e1 = first ? p.first_of<kSpans>(lane) + i : e1;
                    b2 = fmaxf(b2, fminf(b1, v[i]));
                    b1 = fmaxf(b1, v[i]);
                }
                const bool two = b3 == -INFINITY || b2 - b3 > apart_by(b2, b3) || (!biased && b2 == b3);
                if (group_lanes && __all_sync(0xffffffffu, two)) kept = keep_groups_exact<L>(p, row, e1, e2);
                else sure = false;
            }
            if (group_lanes) {
                in = kept;
            } else {
                const uint32_t on = __ballot_sync(0xffffffffu, kept);
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const uint32_t grp = (static_cast<uint32_t>(p.first_of<kSpans>(lane) + i) * p.gsize_magic) >> 20;
                    if (!((on >> ((grp << sh) & 31u)) & 1u)) v[i] = -INFINITY;
                }
            }
        }

        int my = -1, slot = lane;
        if (sure) {
            // Keys without the lane's bits, which the lane's own order does not need.
            int key[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = (ordered_int(v[i]) & ~kMask) | (EPL - 1 - i);
            Top4 top;
            top.of(key);
#pragma unroll
            for (int i = 0; i < 4; ++i) top.k[i] = in ? top.k[i] | lane_bits : kNoKey;
            // k rounds, one more for the runner-up.
            int my_key = kNoKey;
            const bool deep = EPL > 4 && top.k[3] >= kLeastKey;  // a fifth key may follow
            for (int j = 0; j <= p.k; ++j) {
                const int best = __reduce_max_sync(0xffffffffu, top.k[0]);
                my_key = lane == j ? best : my_key;
                const bool won = top.k[0] == best;
#pragma unroll
                for (int i = 0; i < 3; ++i) top.k[i] = won ? top.k[i + 1] : top.k[i];
                top.k[3] = won ? kNoKey : top.k[3];
            }
            if (EPL > 4 && __any_sync(0xffffffffu, deep && top.k[0] < kLeastKey)) {
                // A lane gave all four: the rounds again, each looking through the lane's keys.
                int below = 0x7FFFFFFF;
                for (int j = 0; j <= p.k; ++j) {
                    int k1 = kNoKey;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) k1 = max(k1, key[i] < below ? key[i] : kNoKey);
                    k1 = in ? k1 | lane_bits : kNoKey;
                    const int best = __reduce_max_sync(0xffffffffu, k1);
                    my_key = lane == j ? best : my_key;
                    if (k1 == best) below = k1 ^ lane_bits;
                }
            }
            if (my_key >= kLeastKey && lane <= p.k) {
                my = p.first_of<kSpans>(31 - (my_key & kMask) / EPL) + EPL - 1 - (my_key & (EPL - 1));
            }

            if (!kShort || biased) {
                // Every chosen key clearly above the next, whatever its low bits hide?
                const int next = __shfl_down_sync(0xffffffffu, my_key, 1);
                const float x = ordered_float(my_key & ~kMask), y = ordered_float(next | kMask);
                const bool clear = lane >= p.k || next < kLeastKey || x - y > apart_by(x, y);
                if (!__all_sync(0xffffffffu, clear)) {
                    int n = p.k;  // candidates: lane j < n holds one, or none
                    if (!__shfl_sync(0xffffffffu, clear, p.k - 1)) {
                        // All experts that may belong to the k: those not clearly below the k-th.
                        const float last = __shfl_sync(0xffffffffu, x, p.k - 1);
                        const int least = ordered_int(last - apart_by(last, last)) & ~kMask;
                        n = 0;
#pragma unroll
                        for (int i = 0; i < EPL; ++i) {
                            const bool c = in && key[i] >= least && key[i] >= kLeastKey;
                            const uint32_t who = __ballot_sync(0xffffffffu, c);
                            const int at = n + __popc(who & ((1u << lane) - 1u));
                            if (c && at < 32) cand_smem[warp][at] = static_cast<uint16_t>(p.first_of<kSpans>(lane) + i);
                            n += __popc(who);
                        }
                        __syncwarp();
                        my = lane < n && lane < 32 ? cand_smem[warp][lane] : -1;
                        __syncwarp();
                    }
                    if (n > 32) {
                        sure = false;
                    } else {
                        // By FP32 value; equal ones that are so because both logit and bias are, by index.
                        const bool some = lane < n && my >= 0;
                        const float l = some ? logit_at(row + my) : 0.f, b = some && biased ? p.bias[my] : 0.f;
                        const float c = !some ? -INFINITY : biased ? score(l) + b : l;
                        int rank = 0;
                        bool near = false;
                        for (int h = 0; h < n; ++h) {
                            const float o = __shfl_sync(0xffffffffu, c, h);
                            const int oe = __shfl_sync(0xffffffffu, my, h);
                            const float ol = __shfl_sync(0xffffffffu, l, h), ob = __shfl_sync(0xffffffffu, b, h);
                            rank += (o > c || (o == c && oe < my)) ? 1 : 0;
                            near |= some && oe >= 0 && oe != my && !(fabsf(o - c) > apart_by(o, c)) && !(ol == l && ob == b);
                        }
                        if (biased && __any_sync(0xffffffffu, near)) {
                            const int m = __popc(__ballot_sync(0xffffffffu, some));  // lanes 0 .. m - 1
                            rank = rank_candidates<EPL, L>(p, row, m, my);
                        }
                        slot = some ? rank : lane < p.k ? lane : 32;  // lanes behind the last expert keep their place
                    }
                }
            }
        }
        if (!sure) {
            my = choose_exact<EPL, L>(p, row);
            slot = lane;
        }

        const bool chosen = slot < p.k;
        float s = 0.f;
        if (chosen && my >= 0) {
            const float x = logit_at(row + my);
            s = p.softmax ? expf(x - mx) * rz : sigmoid_f(x);
        }
        if (p.renorm) {
            // s / total to an ulp: the unit's reciprocal after one step of Newton's, and what the product leaves.
            const float total = warp_sum(s) + kRouteEps;
            float r = rcp_fast(total);
            r = fmaf(r, fmaf(-total, r, 1.f), r);
            const float q = s * r;
            s = fmaf(fmaf(-total, q, s), r, q);
        }
        if (chosen) {
            const int64_t at = static_cast<int64_t>(t) * p.k + slot;
            p.idx[at] = my;
            p.w[at] = s * p.scale;
        }
    }
}

// ------------------------------------------------------------- gradient ----

struct RouteBwdParams {
    void* dlogits;        // [T][E], the logits' type
    const float* dw;      // [T][k]
    const void* logits;   // [T][E]
    const int32_t* idx;   // [T][k]
    int T, E, k;
    int whole;            // every lane has EPL experts
    int softmax, renorm;
    float scale;
};

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// N <= 4 floats or N <= 8 values of bf16 in one store.
template <int N>
__device__ __forceinline__ void store_chunk(float* p, const float* f) {
    if constexpr (N == 8) {
        store_chunk<4>(p, f);
        store_chunk<4>(p + 4, f + 4);
    } else if constexpr (N == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else {
        *p = f[0];
    }
}
template <int N>
__device__ __forceinline__ void store_chunk(uint16_t* p, const float* f) {
    if constexpr (N >= 2) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        if constexpr (N == 8) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (N == 4) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        }
    } else {
        store_logit(p, f[0]);
    }
}

// w_j = scale s_j (/ S, S = sum_j s_j + eps):  ds_j = scale dw_j, or
// scale/S (dw_j - sum_i dw_i s_i / S).  Sigmoid: dl = ds s (1 - s) at the
// chosen experts, zero elsewhere; softmax: dl_e = s_e (ds_e - sum_j ds_j s_j).
// Warps take tokens in turn; only softmax reads the whole row.  The chosen
// experts' scores come from the row's in shared memory; the row is stored as it
// is without a choice, then the k elements (a row put together in shared memory
// first took 11.7 us below).  What the next token needs is on its way meanwhile.
// kWide: rows are 16-byte aligned and every lane has EPL experts.
// 16384 tokens of 256 float32 logits, softmax: 8.9 us, 3.9 TB/s, bound by
// instructions (HBM alone 5.4 us); 65536 of 1024: 90 us, 6.0 TB/s.  A lane's wide
// chunks lie 32 chunks apart, so that a load takes whole lines: 203 us there with
// 32 logits in a row to a lane, and 568 against 97 us for 1000.
template <int EPL, bool kWide, typename L>
__global__ void __launch_bounds__(kRouteWarps * 32, route_ctas(EPL))
route_topk_bwd_kernel(const RouteBwdParams p) {
    extern __shared__ __align__(16) float route_smem[];  // per warp a row of 32 * EPL; then per warp 16 slots
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Experts of a lane: a wide load's chunk, the next one 32 chunks on; where not
    // all lanes have EPL, every 32nd.
    constexpr int kChunk = RawRow<EPL, L>::kChunk;
    const bool whole = kWide || p.whole;
    const int e0 = whole ? lane * kChunk : lane;
    auto expert = [&](int i) { return e0 + (whole ? i / kChunk * 32 * kChunk + i % kChunk : 32 * i); };
    float* line = route_smem + warp * 32 * EPL;
    float4* slots = reinterpret_cast<float4*>(route_smem + kRouteWarps * 32 * EPL) + warp * kRouteMaxK;
    const int stride = gridDim.x * kRouteWarps;
    int t = blockIdx.x * kRouteWarps + warp;
    if (t >= p.T) return;

    int next_e = -1;
    float next_g = 0.f;
    RawRow<EPL, L> next_d;
    auto load = [&](int token) {
        if (lane < p.k) {
            next_e = p.idx[static_cast<int64_t>(token) * p.k + lane];
            next_g = p.dw[static_cast<int64_t>(token) * p.k + lane];
        }
        if (p.softmax) {
            const L* row = static_cast<const L*>(p.logits) + static_cast<int64_t>(token) * p.E;
            if (kWide) {
                next_d.load_wide(row + e0, 32 * kChunk);
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) next_d.load_one(i, expert(i) < p.E, row + expert(i));
            }
        }
    };
    load(t);
    for (; t < p.T; t += stride) {
        int e = next_e;
        float g = next_g * p.scale, d[EPL];
        if (e < 0 || e >= p.E) {
            e = -1;
            g = 0.f;
        }
        if (p.softmax) next_d.get(kWide, d);
        if (p.T - t > stride) load(t + stride);

        float s = 0.f, not_s = 0.f, rz = 1.f;  // not_s: 1 - s
        if (p.softmax) {
            float m = d[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) m = fmaxf(m, d[i]);
            m = warp_max(m);
            if (m == -INFINITY) m = 0.f;  // every expert masked: no score, no gradient
            float z = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] -= m;
            exp_results<EPL>(d);
#pragma unroll
            for (int i = 0; i < EPL; ++i) z += d[i];
            if (kWide) {
#pragma unroll
                for (int i = 0; i < EPL; i += kChunk) store_chunk<kChunk>(line + e0 + 32 * i, d + i);
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) line[expert(i)] = d[i];
            }
            z = warp_sum(z);
            __syncwarp();
            rz = z > 0.f || z != z ? 1.f / z : 0.f;
            // 1 - s is the other scores' sum: z less the expert's own term cancels for one that
            // has most of z alone, the only one at the maximum.
            float others = 0.f;
            if (z < 2.f) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) others += d[i] == 1.f ? 0.f : d[i];
                others = warp_sum(others);
            }
            if (e >= 0) {
                const float mine = line[e];
                s = mine * rz;
                not_s = (z < 2.f && mine == 1.f ? others : z - mine) * rz;
            }
        } else if (e >= 0) {
            const float x = logit_at(static_cast<const L*>(p.logits) + static_cast<int64_t>(t) * p.E + e);
            // Both of 1 / (1 + e) and e / (1 + e); 1 - s itself cancels (6 % off at x = 16, zero from 17 on).
            const float ex = expf(-fabsf(x)), more = __frcp_rn(1.f + ex), less = ex * more;
            s = x < 0.f ? less : more;
            not_s = x < 0.f ? more : less;
        }
        // The slots among themselves, through shared memory; past k: zeros, expert -1.
        if (lane < kRouteMaxK) slots[lane] = make_float4(g, s, __int_as_float(e), 0.f);
        __syncwarp();
        // g_j - sum_i g_i s_i / S = (sum_i (g_j - g_i) s_i + g_j eps) / S, and
        // g_j - sum_i g_i s_i = g_j (1 - s_j) - sum over the other experts' slots: nothing
        // cancels where one expert has nearly all the weight, or is the only one.
        float diff = 0.f, total = kRouteEps, dot = 0.f, other = 0.f;
        int alike = 0;  // slots with this one's expert
#pragma unroll 1  // unrolled, its loads spill
        for (int j0 = 0; j0 < p.k; j0 += 4) {
            float4 o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = slots[j0 + j];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool same = __float_as_int(o[j].z) == e;
                total += o[j].y;
                dot = fmaf(o[j].x, o[j].y, dot);
                other = fmaf(same ? 0.f : o[j].x, o[j].y, other);
                diff = fmaf(g - o[j].x, o[j].y, diff);
                alike += same ? 1 : 0;
            }
        }
        bool first = e >= 0;
        if (__any_sync(0xffffffffu, first && alike > 1)) {  // an expert's first slot takes the sums, in slot order
            float sum_g = 0.f, sum_d = 0.f;
            for (int j = 0; j < p.k; ++j) {
                const int ej = __shfl_sync(0xffffffffu, e, j);
                const float gj = __shfl_sync(0xffffffffu, g, j), dj = __shfl_sync(0xffffffffu, diff, j);
                sum_g += ej == e ? gj : 0.f;
                sum_d += ej == e ? dj : 0.f;
                first = first && !(ej == e && j < lane);
            }
            g = sum_g;
            diff = sum_d;
        }
        if (p.softmax) g = fmaf(g, not_s, -other);
        if (p.renorm) {
            const float rs = 1.f / total;
            g = fmaf(g, kRouteEps, diff) * rs * rs;
            dot = dot * rs * (kRouteEps * rs);  // sum of the new g s: the differences cancel in pairs
        }
        // The row as it is without a choice, then the chosen experts' values over it.
        L* out = static_cast<L*>(p.dlogits) + static_cast<int64_t>(t) * p.E;
        const float rest = -dot * rz;
        float r[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) r[i] = p.softmax ? rest * d[i] : 0.f;
        if (kWide) {
#pragma unroll
            for (int i = 0; i < EPL; i += kChunk) store_chunk<kChunk>(out + e0 + 32 * i, r + i);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (expert(i) < p.E) store_logit(out + expert(i), r[i]);
        }
        __syncwarp();  // orders the two stores of an element; `line` and `slots` have been read
        if (first) store_logit(out + e, g * (p.softmax ? s : s * not_s));
    }
}

// --------------------------------------------------------------- layout ----

constexpr int kLayoutThreads = 1024;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kLayoutMaxCluster = 8;
constexpr int kLayoutHeld = 4;  // batches of 32 slots that a warp keeps in registers

struct LayoutParams {
    const int32_t* idx;  // [S] chosen experts, -1: none
    int32_t* row_of;     // [S]
    int32_t* m_indices;  // [rows]
    int32_t* slot_of;    // [rows]
    int32_t* offsets;    // [E + 1]
    int32_t* counts;     // [E]
    int64_t S;
    int64_t warp_slots;  // slots per warp, a multiple of 32
    int warps;           // warps of a CTA that have slots
    int E, expert_bits;  // E <= 1 << expert_bits
    int rows;
    int max_rows;        // 0: contiguous segments of whole 128 rows; else rows per group
};

enum LayoutKind : int {
    kLayoutHeldRun = 0,  // a warp's run of slots stays in registers
    kLayoutStaged = 1,   // it is read and ranked again in the second pass
    kLayoutDirect = 2,   // ... and the CTA's slots do not fit in shared memory
};

// A CTA's slots are staged as pairs of 16-bit numbers: place in its run, expert.
constexpr int kLayoutMaxStaged = 65536;

// Shared memory of the layout kernel in ints: counts [warps][E], then [E]
// totals of this CTA, [E + 1] starts, [E] rows held, [E] first rows of this
// CTA's slots, [E] their places among its staged slots, [32] pairs of sums, and
// the staged slots.
__host__ __device__ constexpr int layout_smem_ints(int E, int warps, int staged) {
    return (warps + 5) * E + 2 + 2 * kLayoutWarps + staged;
}

// Stable counting sort of the slots by expert, in one cluster: every warp
// walks a consecutive run of slots; its counts per expert are scanned over the
// warps of a CTA, over the CTAs of the cluster (distributed shared memory) and
// over the experts; a slot's rank among the run's slots of its expert, on top
// of the scanned count, makes its row.  No atomics between warps, so rows
// follow slot order in every launch.  The slots pass through shared memory in
// row order, so that the two arrays by row are written in runs (a 4-byte write
// on its own costs as much as a whole sector).  Bound by latency: a few
// barriers and, in each warp, one dependent step per 32 slots.  In that step the
// lanes of equal expert find one another by a vote per bit of the expert
// (__match_any_sync took 1300 cycles a batch with 32 warps at it).  32768 slots
// over 64 experts: 8.1 us; 512 slots over 32: 3.7 us; 262144 over 256: 40 us.
template <int kKind>
__global__ void __launch_bounds__(kLayoutThreads)
route_layout_kernel(const LayoutParams p) {
    extern __shared__ int layout_smem[];
    int* run = layout_smem;
    int* total = run + p.warps * p.E;  // read by the other CTAs
    int* start = total + p.E;
    int* held = start + p.E + 1;
    uint32_t* base = reinterpret_cast<uint32_t*>(held + p.E);
    int* local_start = held + 2 * p.E;
    unsigned long long* wsum = reinterpret_cast<unsigned long long*>(layout_smem + (((p.warps + 5) * p.E + 2) & ~1));
    uint32_t* staged = reinterpret_cast<uint32_t*>(wsum + kLayoutWarps);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank(), nctas = cluster_nctarank();
    for (int i = tid; i < p.warps * p.E; i += kLayoutThreads) run[i] = 0;
    griddep_wait();
    griddep_launch_dependents();

    const int64_t cta0 = static_cast<int64_t>(rank) * p.warps * p.warp_slots;
    const int64_t s0 = cta0 + warp * p.warp_slots;
    const int64_t end = s0 + p.warp_slots < p.S ? s0 + p.warp_slots : p.S, s1 = warp < p.warps ? end : s0;
    int* mine = run + warp * p.E;
    int idx[kLayoutHeld], local[kLayoutHeld];  // expert (-1: none) and rank in the run
    bool bad = false;
    auto fetch = [&](int64_t at) {
        int x = at < s1 ? p.idx[at] : -1;
        if (x < 0 || x >= p.E) {
            bad |= x != -1;
            x = -1;
        }
        return x;
    };
    // Rank of a batch's slots among the run's so far; the counts move on.
    auto rank_batch = [&](int x) {
        uint32_t same = __ballot_sync(0xffffffffu, x >= 0);
        for (int b = 0; b < p.expert_bits; ++b) {
            const uint32_t ones = __ballot_sync(0xffffffffu, (x >> b) & 1);
            same &= (x >> b) & 1 ? ones : ~ones;
        }
        const int r = x >= 0 ? mine[x] + __popc(same & ((1u << lane) - 1u)) : 0;
        __syncwarp();
        if (x >= 0 && lane == 31 - __clz(same)) mine[x] = r + 1;
        __syncwarp();
        return r;
    };
    if (kKind == kLayoutHeldRun) {
#pragma unroll
        for (int i = 0; i < kLayoutHeld; ++i) idx[i] = fetch(s0 + 32 * i + lane);
    }
    __syncthreads();
    if (kKind == kLayoutHeldRun) {
#pragma unroll
        for (int i = 0; i < kLayoutHeld; ++i) local[i] = s0 + 32 * i < s1 ? rank_batch(idx[i]) : 0;
    } else {
        for (int64_t s = s0 + lane; s < s1; s += 32) {
            const int x = fetch(s);
            if (x >= 0) atomicAdd(mine + x, 1);
        }
    }
    if (bad) atomicOr(&g_dg_error, 32u);
    __syncthreads();
    // Exclusive over this CTA's warps, eight at a time.
    if (tid < p.E) {
        int n = 0;
        for (int w0 = 0; w0 < p.warps; w0 += 8) {
            int x[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) x[w] = w0 + w < p.warps ? run[(w0 + w) * p.E + tid] : 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w0 + w < p.warps) run[(w0 + w) * p.E + tid] = n;
                n += x[w];
            }
        }
        total[tid] = n;
    }
    __syncwarp();
    if (nctas > 1) cluster_sync();
    // Over the CTAs, then over the experts (at most one expert per thread).
    const int e = tid;
    int before = 0, all = 0;
    if (e < p.E) {
        if (nctas > 1) {
#pragma unroll
            for (uint32_t r = 0; r < kLayoutMaxCluster; ++r) {
                if (r >= nctas) break;
                int x;
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(dsmem_addr(smem_u32(total + e), r)) : "memory");
                if (r < rank) before += x;
                all += x;
            }
        } else {
            all = total[e];
        }
    }
    __syncwarp();
    if (nctas > 1) cluster_arrive();  // this thread has read the other CTAs' totals
    const int kept = p.max_rows > 0 ? min(all, p.max_rows) : all;
    const int len = e >= p.E ? 0 : p.max_rows > 0 ? p.max_rows : (all + 127) / 128 * 128;
    // Scanned together: rows of the groups (low half) and this CTA's own slots.
    const uint32_t own = e < p.E ? total[e] : 0;
    unsigned long long incl = static_cast<unsigned long long>(own) << 32 | static_cast<uint32_t>(len);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    {
        // every warp scans the warps' sums for itself
        unsigned long long v = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        const unsigned long long upto = __shfl_sync(0xffffffffu, v, (warp + 31) & 31);
        if (warp) incl += upto;
    }
    const int first = static_cast<int>(static_cast<uint32_t>(incl)) - len;
    if (e < p.E) {
        start[e] = first;
        if (e == p.E - 1) start[p.E] = first + len;
        base[e] = static_cast<uint32_t>(first) + static_cast<uint32_t>(before);
        local_start[e] = static_cast<int>(incl >> 32) - static_cast<int>(own);
        held[e] = kept;
        if (rank == 0) {
            p.offsets[e] = first;
            p.counts[e] = kept;
            if (e == p.E - 1) p.offsets[p.E] = first + len;
        }
    }
    __syncthreads();

    // Places past a masked group's end may pass 31 bits (rows and slots are below that each), 32 never.
    auto row_at = [&](int x, int r) {
        const uint32_t row = base[x] + static_cast<uint32_t>(r);
        return p.max_rows > 0 && row >= static_cast<uint32_t>(start[x] + p.max_rows) ? -1 : static_cast<int>(row);
    };
    auto place = [&](int64_t at, int x, int r) {  // r: rank among the CTA's slots of x
        const int row = x >= 0 ? row_at(x, r) : -1;
        if (at < s1) p.row_of[at] = row;
        if (kKind != kLayoutDirect) {
            if (x >= 0) staged[local_start[x] + r] = static_cast<uint32_t>(at - cta0) << 16 | static_cast<uint32_t>(x);
        } else if (row >= 0) {
            p.m_indices[row] = x;
            p.slot_of[row] = static_cast<int>(at);
        }
    };
    if (kKind == kLayoutHeldRun) {
#pragma unroll
        for (int i = 0; i < kLayoutHeld; ++i)
            if (s0 + 32 * i < s1) place(s0 + 32 * i + lane, idx[i], idx[i] >= 0 ? mine[idx[i]] + local[i] : 0);
    } else {
        for (int64_t s = s0; s < s1; s += 32) {
            const int x = fetch(s + lane);
            place(s + lane, x, rank_batch(x));
        }
    }
    // Rows without a slot: -1 behind each group's last one, and behind the last group.
    const int t0 = static_cast<int>(rank) * kLayoutThreads + tid, nt = static_cast<int>(nctas) * kLayoutThreads;
    auto clear = [&](int r) {
        p.m_indices[r] = -1;
        p.slot_of[r] = -1;
    };
    if (p.max_rows > 0) {
        for (int64_t r = t0; r < p.rows; r += nt) {
            const int g = static_cast<int>(r) / p.max_rows;
            if (static_cast<int>(r) - g * p.max_rows >= held[g]) clear(static_cast<int>(r));
        }
    } else {
        for (int i = t0; i < p.E * 128; i += nt) {  // fewer than 128 rows behind each
            const int g = i >> 7, r = start[g] + held[g] + (i & 127);
            if (r < start[g + 1]) clear(r);
        }
        for (int64_t r = start[p.E] + t0; r < p.rows; r += nt) clear(static_cast<int>(r));
    }
    if (kKind != kLayoutDirect) {
        __syncthreads();
        const int n = local_start[p.E - 1] + total[p.E - 1];
        for (int i = tid; i < n; i += kLayoutThreads) {
            const int x = static_cast<int>(staged[i] & 0xFFFFu), row = row_at(x, i - local_start[x]);
            if (row >= 0) {
                p.m_indices[row] = x;
                p.slot_of[row] = static_cast<int>(cta0 + (staged[i] >> 16));
            }
        }
    }
    __syncwarp();
    if (nctas > 1) cluster_wait();  // no CTA leaves while another may still read its totals
}

}  // namespace dg
