// dg_route.cuh -- sm_100a routing kernels: the choice of k experts per token,
// its gradient, and the grouped layout that the choice leads to.
//
// Scores s = softmax(l) or sigmoid(l) over the E logits of a token; choice
// values c = s + bias.  The result is that of exact arithmetic: an order
// decided in FP32 is kept only where neighbours differ by more than FP32 can
// have moved them, else the token is decided again in FP64.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "dg_ptx.cuh"

namespace dg {

constexpr int kRouteWarps = 8;
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
    int per;              // experts per lane: lane i holds i * per .. i * per + per - 1
    int group_lanes;      // lanes per group where groups are whole lanes (a power of two), else 0
    int vec;              // every lane full, rows and bias 16-byte aligned: wide loads
    int softmax, renorm;
    float scale;
};

__device__ __forceinline__ float logit_at(const float* p) { return *p; }
__device__ __forceinline__ float logit_at(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

// N consecutive logits with the widest loads (the address is a multiple of
// the load's width).
template <int N>
__device__ __forceinline__ void load_logits(const float* p, float (&f)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(f + i) = *reinterpret_cast<const float4*>(p + i);
    } else if constexpr (N == 2) {
        *reinterpret_cast<float2*>(f) = *reinterpret_cast<const float2*>(p);
    } else {
        f[0] = *p;
    }
}
template <int N>
__device__ __forceinline__ void load_logits(const uint16_t* p, float (&f)[N]) {
    if constexpr (N >= 2) {
        uint32_t w[N / 2];
        if constexpr (N >= 8) {
#pragma unroll
            for (int i = 0; i < N / 2; i += 4) *reinterpret_cast<uint4*>(w + i) = *reinterpret_cast<const uint4*>(p + 2 * i);
        } else if constexpr (N == 4) {
            *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        f[0] = logit_at(p);
    }
}

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

// exp and the sigmoid by the special-function unit alone, without the care for
// subnormal numbers: relative error 2^-22 and |x| 2^-24 for the argument's
// rounding; absolute error of the sigmoid below 2^-22.
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
// For results: relative error a few 2^-24.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

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
            const int e = lane * p.per + i;
            if (i < p.per && e < p.E) {
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
            const int e = lane * p.per + i;
            c[i] = i < p.per && e < p.E ? exp(static_cast<double>(logit_at(row + e)) - m) : 0.0;
            z += c[i];
        }
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    unsigned long long key[EPL];  // of the choice value, 0: not eligible
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane * p.per + i;
        key[i] = 0;
        if (i < p.per && e < p.E) {
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
                    const int e = lane * p.per + i;
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
            const uint32_t grp = (static_cast<uint32_t>(lane * p.per + i) * p.gsize_magic) >> 20;
            if (!((kept >> (grp & 31u)) & 1u)) key[i] = 0;
        }
    }
    if (!p.bias) {  // in the order of the logits themselves
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i]) key[i] = order_key(static_cast<double>(logit_at(row + lane * p.per + i)));
    }
    int my = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) { best = key[i]; at = lane * p.per + i; }
        const unsigned long long top = warp_max_u64(best);
        if (top == 0) break;
        at = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
        if (lane == j) my = at;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane * p.per + i == at) key[i] = 0;
    }
    return my;
}

// The groups kept, decided in FP64 where groups are whole lanes: a lane's two
// best experts are e1 and e2 (-1: none; no third is close to them).  Returns
// whether this lane's group is kept.
template <typename L>
__device__ __noinline__ bool keep_groups_exact(const RouteParams& p, const L* row, int e1, int e2) {
    const int lane = threadIdx.x & 31, g = lane / p.group_lanes;
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
    for (int o = p.group_lanes >> 1; o >= 1; o >>= 1) {
        const double xa = __shfl_xor_sync(0xffffffffu, a, o), xb = __shfl_xor_sync(0xffffffffu, b, o);
        b = fmax(fmax(b, xb), fmin(a, xa));
        a = fmax(a, xa);
    }
    double sum = a + (p.gtop == 2 && b != -INFINITY ? b : 0.0);
    if (g >= p.groups) sum = -INFINITY;
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
        const double o = __shfl_sync(0xffffffffu, sum, h * p.group_lanes);
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

// One warp per token, lane i holding the experts i * per ...
//
// The choice works on keys: a value's leading bits in integer order, and in
// its low bits the expert's place (lane, then place in the lane, counted down),
// so that a maximum of keys is a value, its expert and the rule for ties at
// once.  A key costs three instructions, keeping a lane's two largest three
// more, and a round of the choice one warp-wide maximum.  The k experts so
// found are the right set where the (k+1)-th key is clearly below; their order
// is decided by their FP32 values, and by FP64 values where those are not
// clearly apart.  bf16 logits without a bias fit a key whole.
//
// Bound by instructions: 16384 tokens of 256 float32 logits are 2.6 us of HBM.
template <int EPL, typename L>
__global__ void __launch_bounds__(kRouteWarps * 32, EPL <= 8 ? 4 : 1)
route_topk_kernel(const RouteParams p) {
    constexpr int kMask = 32 * EPL - 1;  // a key's place bits
    constexpr bool kShort = sizeof(L) == 2;
    extern __shared__ float route_smem[];  // groups that are not whole lanes: E values per warp
    __shared__ uint16_t cand_smem[kRouteWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (t >= p.T) return;
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    const int e0 = lane * p.per;
    const bool biased = p.bias != nullptr;

    float v[EPL];  // logits, then (with a bias) choice values; -inf: not eligible
    if (p.vec) {
        load_logits<EPL>(row + lane * EPL, v);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = i < p.per && e0 + i < p.E ? logit_at(row + e0 + i) : -INFINITY;
    }
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
    // FP32 moves a choice value by less than `slack` (of the largest score:
    // exponential, sum and reciprocal of a softmax 2^-20, sigmoid_fast 2^-22),
    // and adding the bias by 2^-24 of the value.
    const float slack = p.softmax ? rz * 0x1p-20f : 0x1p-22f;
    auto apart_by = [&](float x, float y) {  // more than FP32 can have moved x - y
        return biased ? 2.f * slack + 0x1p-22f * (fabsf(x) + fabsf(y)) : 0.f;
    };
    auto score = [&](float x) { return p.softmax ? exp_fast(x - mx) * rz : sigmoid_fast(x); };

    if (biased) {
        float b[EPL];
        if (p.vec) {
            load_logits<EPL>(p.bias + lane * EPL, b);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = i < p.per && e0 + i < p.E ? p.bias[e0 + i] : -INFINITY;
        }
        float low = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) low = fminf(low, v[i]);
#pragma unroll
        for (int i = 0; i < EPL; ++i) b[i] += score(v[i]);
        if (low == -INFINITY) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = v[i] == -INFINITY ? -INFINITY : b[i];
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = b[i];
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] += 0.f;  // one zero
    }
    // A NaN, or an infinite choice value: to be decided without shortcuts.
    float all = v[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) all += v[i];
    const bool inf_ok = !biased && !p.softmax;
    bool odd = inf_ok ? all != all : !(all < INFINITY) || (rz != rz && mx != -INFINITY);
    odd = __any_sync(0xffffffffu, odd);

    bool in = true, sure = true;  // in: the lane's experts take part
    if (p.groups > 1 && !odd) {
        float a = -INFINITY, b = -INFINITY;  // the two best choice values of the group
        int g, lanes;                        // this lane's group, lanes per group
        // A choice value without a bias is the score of the logit.
        auto choice = [&](float x) { return x == -INFINITY || biased ? x : score(x); };
        if (p.group_lanes) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                b = fmaxf(b, fminf(a, v[i]));
                a = fmaxf(a, v[i]);
            }
            a = choice(a);
            b = choice(b);
            lanes = p.group_lanes;
            g = lane / lanes;
        } else {
            // A power of two of lanes share a group in shared memory.
            float* cs = route_smem + warp * p.E;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i < p.per && e0 + i < p.E) cs[e0 + i] = choice(v[i]);
            __syncwarp();
            const int sh = 31 - __clz(32 / p.groups);
            g = lane >> sh;
            lanes = 1 << sh;
            if (g < p.groups) {
                const int sub = lane & (lanes - 1);
                // Each group starts at another place: the same places of groups of 32 share a bank.
                const int turn = (g << sh) % p.gsize;
                for (int n = sub; n < p.gsize; n += lanes) {
                    const float x = cs[g * p.gsize + (n + turn < p.gsize ? n + turn : n + turn - p.gsize)];
                    b = fmaxf(b, fminf(a, x));
                    a = fmaxf(a, x);
                }
            }
        }
        for (int o = lanes >> 1; o >= 1; o >>= 1) {
            const float xa = __shfl_xor_sync(0xffffffffu, a, o), xb = __shfl_xor_sync(0xffffffffu, b, o);
            b = fmaxf(fmaxf(b, xb), fminf(a, xa));
            a = fmaxf(a, xa);
        }
        float sum = a + (p.gtop == 2 && b != -INFINITY ? b : 0.f);
        if (g >= p.groups) sum = -INFINITY;
        int rank = 0;
        for (int h = 0; h < p.groups; ++h) {
            const float o = __shfl_sync(0xffffffffu, sum, h * lanes);
            rank += (o > sum || (o == sum && h < g)) ? 1 : 0;
        }
        bool kept = sum != -INFINITY && rank < p.keep;
        // Certain when the worst kept group and the best other are clearly apart.
        const float lo = warp_min(kept ? sum : INFINITY), hi = warp_max(kept ? -INFINITY : sum);
        if (hi != -INFINITY && !(lo - hi > 4.f * slack + 0x1p-21f * (fabsf(lo) + fabsf(hi)))) {
            // The lane's two best, if no third can take their place in FP64.
            float b1 = -INFINITY, b2 = -INFINITY, b3 = -INFINITY;
            int e1 = -1, e2 = -1;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const bool first = v[i] > b1, second = v[i] > b2;
                b3 = fmaxf(b3, fminf(b2, v[i]));
                e2 = first ? e1 : second ? e0 + i : e2;
                e1 = first ? e0 + i : e1;
                b2 = fmaxf(b2, fminf(b1, v[i]));
                b1 = fmaxf(b1, v[i]);
            }
            const bool two = b3 == -INFINITY || b2 - b3 > apart_by(b2, b3) || (!biased && b2 == b3);
            if (p.group_lanes && __all_sync(0xffffffffu, two)) kept = keep_groups_exact<L>(p, row, e1, e2);
            else sure = false;
        }
        if (p.group_lanes) {
            in = kept;
        } else {
            const uint32_t on = __ballot_sync(0xffffffffu, kept);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t grp = (static_cast<uint32_t>(e0 + i) * p.gsize_magic) >> 20;
                if (!((on >> ((grp * lanes) & 31u)) & 1u)) v[i] = -INFINITY;
            }
        }
    }

    int my = -1, slot = lane;
    if (sure && !odd) {
        // Keys: without the lane's bits, which the lane's own order does not need.
        const int lane_bits = (31 - lane) * EPL;
        int key[EPL], k1 = kNoKey, k2 = kNoKey;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            key[i] = (ordered_int(v[i]) & ~kMask) | (EPL - 1 - i);
            k2 = max(k2, min(k1, key[i]));
            k1 = max(k1, key[i]);
        }
        if (in) {
            k1 |= lane_bits;
            k2 |= lane_bits;
        } else {
            k1 = k2 = kNoKey;
        }
        // k rounds, one more for the runner-up.
        int my_key = kNoKey;
        bool two = true;  // k2 is the lane's second largest
        for (int j = 0; j <= p.k; ++j) {
            const int top = __reduce_max_sync(0xffffffffu, k1);
            if (top < kLeastKey) break;
            if (lane == j) my_key = top;
            if (k1 == top) {
                if (two) {
                    k1 = k2;
                    two = false;
                } else {
                    // Look for the largest below it again.
                    const int below = top ^ lane_bits;
                    k1 = kNoKey;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) k1 = max(k1, key[i] < below ? key[i] : kNoKey);
                    k1 |= lane_bits;
                }
            }
        }
        auto expert_of = [&](int k) { return (31 - (k & kMask) / EPL) * p.per + EPL - 1 - (k & (EPL - 1)); };
        if (my_key >= kLeastKey) my = expert_of(my_key);

        if (!kShort || biased) {
            int n = p.k;  // candidates: lane j < n holds one, or none
            bool ranked = true;  // the lanes may not be in order
            const int last = __shfl_sync(0xffffffffu, my_key, p.k - 1), next = __shfl_sync(0xffffffffu, my_key, p.k);
            const float x = ordered_float(last & ~kMask), y = ordered_float(next | kMask);
            if (next >= kLeastKey && !(x - y > apart_by(x, y))) {
                // All experts that may belong to the k: those not clearly below the k-th.
                const int least = ordered_int(x - apart_by(x, x)) & ~kMask;
                n = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const bool c = in && key[i] >= least && key[i] >= kLeastKey;
                    const uint32_t who = __ballot_sync(0xffffffffu, c);
                    const int at = n + __popc(who & ((1u << lane) - 1u));
                    if (c && at < 32) cand_smem[warp][at] = static_cast<uint16_t>(e0 + i);
                    n += __popc(who);
                }
                __syncwarp();
                ranked = false;
                if (n > 32) {
                    sure = false;
                } else {
                    my = lane < n ? cand_smem[warp][lane] : -1;
                }
            }
            // The candidates' values: lane order holds if every one is clearly above the next.
            const bool some = lane < n && my >= 0;
            const float l = some ? logit_at(row + my) : 0.f, b = some && biased ? p.bias[my] : 0.f;
            const float c = !some ? -INFINITY : biased ? score(l) + b : l;
            if (sure) {
                const float below = __shfl_down_sync(0xffffffffu, c, 1);
                const int below_e = __shfl_down_sync(0xffffffffu, my, 1);
                const bool last_one = lane + 1 >= n || below_e < 0 || !some;
                const bool good = last_one || c - below > apart_by(c, below) || (!biased && c == below && my < below_e);
                if (!ranked || !__all_sync(0xffffffffu, good)) {
                    int rank = 0;
                    bool near = false;
                    for (int h = 0; h < n; ++h) {
                        const float o = __shfl_sync(0xffffffffu, c, h);
                        const int oe = __shfl_sync(0xffffffffu, my, h);
                        const float ol = __shfl_sync(0xffffffffu, l, h), ob = __shfl_sync(0xffffffffu, b, h);
                        rank += (o > c || (o == c && oe < my)) ? 1 : 0;
                        // Equal because both logit and bias are: the lower index is right.
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
    if (odd || !sure) {
        my = choose_exact<EPL, L>(p, row);
        slot = lane;
    }

    const bool chosen = slot < p.k;
    float s = 0.f;
    if (chosen && my >= 0) {
        const float x = logit_at(row + my);
        s = p.softmax ? expf(x - mx) * rz : sigmoid_f(x);
    }
    if (p.renorm) s = __fdividef(s, warp_sum(s) + kRouteEps);
    if (chosen) {
        p.idx[t * p.k + slot] = my;
        p.w[t * p.k + slot] = s * p.scale;
    }
}

// ------------------------------------------------------------- gradient ----

struct RouteBwdParams {
    void* dlogits;        // [T][E], the logits' type
    const float* dw;      // [T][k]
    const void* logits;   // [T][E]
    const int32_t* idx;   // [T][k]
    int T, E, k;
    int per;              // experts per lane, as in RouteParams
    int vec;
    int softmax, renorm;
    float scale;
};

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
template <int N>
__device__ __forceinline__ void store_logits(float* p, const float (&f)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    } else if constexpr (N == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else {
        *p = f[0];
    }
}
template <int N>
__device__ __forceinline__ void store_logits(uint16_t* p, const float (&f)[N]) {
    if constexpr (N >= 2) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        if constexpr (N >= 8) {
#pragma unroll
            for (int i = 0; i < N / 2; i += 4) *reinterpret_cast<uint4*>(p + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
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
// One warp per token; only softmax reads the whole row.  The k gradients meet
// their experts through a row of shared memory.
template <int EPL, typename L>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_topk_bwd_kernel(const RouteBwdParams p) {
    extern __shared__ __align__(16) float route_smem[];  // 32 * EPL values per warp
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (t >= p.T) return;
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    L* out = static_cast<L*>(p.dlogits) + t * p.E;
    const int e0 = lane * p.per;

    int e = -1;
    float g = 0.f, x = 0.f;
    if (lane < p.k) {
        e = p.idx[t * p.k + lane];
        if (e < 0 || e >= p.E) e = -1;
        else x = logit_at(row + e);
        g = e < 0 ? 0.f : p.dw[t * p.k + lane] * p.scale;
    }
    float d[EPL];
    float mx = 0.f, rz = 1.f;
    if (p.softmax) {
        if (p.vec) {
            load_logits<EPL>(row + lane * EPL, d);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] = i < p.per && e0 + i < p.E ? logit_at(row + e0 + i) : -INFINITY;
        }
        float m = d[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = fmaxf(m, d[i]);
        mx = warp_max(m);
        if (mx == -INFINITY) mx = 0.f;  // every expert masked: no score, no gradient
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            d[i] = exp_fast(d[i] - mx);
            z += d[i];
        }
        z = warp_sum(z);
        rz = z > 0.f || z != z ? 1.f / z : 0.f;
    }
    float s = 0.f;
    if (e >= 0) s = p.softmax ? expf(x - mx) * rz : sigmoid_f(x);
    if (p.renorm) {
        const float r = 1.f / (warp_sum(s) + kRouteEps);
        const float mean = warp_sum(g * s) * r;
        g = e < 0 ? 0.f : (g - mean) * r;
    }
    float dot = 0.f;
    if (p.softmax) dot = warp_sum(g * s);
    else g *= s * (1.f - s);

    float* line = route_smem + warp * 32 * EPL;
    float r[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) r[i] = 0.f;
    store_logits<EPL>(line + lane * EPL, r);
    // An expert in several slots: its first slot takes the sum, in slot order.
    const uint32_t same = __match_any_sync(0xffffffffu, e >= 0 ? e : -1 - lane);
    if (__any_sync(0xffffffffu, (same & (same - 1u)) != 0)) {
        float sum = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const float gj = __shfl_sync(0xffffffffu, g, j);
            if ((same >> j) & 1u) sum += gj;
        }
        g = sum;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) line[e / p.per * EPL + e % p.per] = g;
    __syncwarp();
    load_logits<EPL>(line + lane * EPL, r);
    if (p.softmax) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) r[i] = (r[i] - dot) * (d[i] * rz);
    }
    if (p.vec) {
        store_logits<EPL>(out + lane * EPL, r);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i < p.per && e0 + i < p.E) store_logit(out + e0 + i, r[i]);
    }
}

// --------------------------------------------------------------- layout ----

constexpr int kLayoutThreads = 1024;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kLayoutMaxCluster = 8;

struct LayoutParams {
    const int32_t* idx;  // [S] chosen experts, -1: none
    int32_t* row_of;     // [S]
    int32_t* m_indices;  // [rows]
    int32_t* slot_of;    // [rows]
    int32_t* offsets;    // [E + 1]
    int32_t* counts;     // [E]
    int64_t S;
    int64_t warp_slots;  // slots per warp, a multiple of 32
    int E;
    int64_t rows;
    int max_rows;        // 0: contiguous segments of whole 128 rows; else rows per group
};

// Stable counting sort of the slots by expert, in one cluster: every warp
// counts a consecutive run of slots per expert; the counts are scanned over
// the warps of a CTA, over the CTAs of the cluster (distributed shared memory)
// and over the experts; then every warp walks its run again and hands out the
// rows.  No atomics between warps, so rows follow slot order in every run.
// Shared memory: layout_smem_ints(E) ints.
__host__ __device__ constexpr int layout_smem_ints(int E) { return (kLayoutWarps + 3) * E + 1 + kLayoutWarps; }

__global__ void __launch_bounds__(kLayoutThreads)
route_layout_kernel(const LayoutParams p) {
    extern __shared__ int layout_smem[];
    int* run = layout_smem;                       // [kLayoutWarps][E]
    int* total = run + kLayoutWarps * p.E;        // [E], read by the other CTAs
    int* start = total + p.E;                     // [E + 1]
    int* held = start + p.E + 1;                  // [E] rows of each group that hold a slot
    int* wsum = held + p.E;                       // [kLayoutWarps]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank(), nctas = cluster_nctarank();
    griddep_wait();
    griddep_launch_dependents();

    for (int i = tid; i < kLayoutWarps * p.E; i += kLayoutThreads) run[i] = 0;
    __syncthreads();
    const int64_t s0 = (static_cast<int64_t>(rank) * kLayoutWarps + warp) * p.warp_slots;
    const int64_t s1 = s0 + p.warp_slots < p.S ? s0 + p.warp_slots : p.S;
    int* mine = run + warp * p.E;
    bool bad = false;
    for (int64_t s = s0 + lane; s < s1; s += 32) {
        const int e = p.idx[s];
        if (e >= 0 && e < p.E) atomicAdd(mine + e, 1);
        else bad |= e != -1;
    }
    if (bad) atomicOr(&g_dg_error, 32u);
    __syncthreads();
    // Exclusive over this CTA's warps.
    for (int e = tid; e < p.E; e += kLayoutThreads) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kLayoutWarps; ++w) {
            const int x = run[w * p.E + e];
            run[w * p.E + e] = n;
            n += x;
        }
        total[e] = n;
    }
    cluster_sync();
    // Over the CTAs, then over the experts (at most one expert per thread).
    const int e = tid;
    int before = 0, all = 0;
    if (e < p.E) {
        for (uint32_t r = 0; r < nctas; ++r) {
            int x;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(dsmem_addr(smem_u32(total + e), r)) : "memory");
            if (r < rank) before += x;
            all += x;
        }
    }
    __syncwarp();
    cluster_arrive();  // this thread has read the other CTAs' totals
    const int kept = p.max_rows > 0 ? min(all, p.max_rows) : all;
    const int len = e >= p.E ? 0 : p.max_rows > 0 ? p.max_rows : (all + 127) / 128 * 128;
    int incl = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        wsum[lane] = v;
    }
    __syncthreads();
    const int first = incl - len + (warp ? wsum[warp - 1] : 0);
    if (e < p.E) {
        start[e] = first;
        if (e == p.E - 1) start[p.E] = first + len;
#pragma unroll 8
        for (int w = 0; w < kLayoutWarps; ++w) run[w * p.E + e] += first + before;
        held[e] = kept;
        if (rank == 0) {
            p.offsets[e] = first;
            p.counts[e] = kept;
            if (e == p.E - 1) p.offsets[p.E] = first + len;
        }
    }
    __syncthreads();

    for (int64_t s = s0; s < s1; s += 32) {
        const int64_t at = s + lane;
        const int x = at < s1 ? p.idx[at] : -1;
        const bool ok = x >= 0 && x < p.E;
        const uint32_t same = __match_any_sync(0xffffffffu, ok ? x : -1);
        int row = -1;
        if (ok) {
            row = mine[x] + __popc(same & ((1u << lane) - 1u));
            if (p.max_rows > 0 && row >= start[x] + p.max_rows) row = -1;
        }
        __syncwarp();
        if (ok && lane == 31 - __clz(same)) mine[x] += __popc(same);
        __syncwarp();
        if (at < s1) p.row_of[at] = row;
        if (row >= 0) {
            p.m_indices[row] = x;
            p.slot_of[row] = static_cast<int>(at);
        }
    }
    // Rows without a slot: -1 behind each group's last one, and behind the last group.
    const int64_t gw = static_cast<int64_t>(rank) * kLayoutWarps + warp, nw = static_cast<int64_t>(nctas) * kLayoutWarps;
    for (int64_t g = gw; g < p.E; g += nw)
        for (int64_t r = start[g] + static_cast<int64_t>(held[g]) + lane; r < start[g + 1]; r += 32) {
            p.m_indices[r] = -1;
            p.slot_of[r] = -1;
        }
    for (int64_t r = start[p.E] + gw * 32 + lane; r < p.rows; r += nw * 32) {
        p.m_indices[r] = -1;
        p.slot_of[r] = -1;
    }
    __syncwarp();
    cluster_wait();  // no CTA leaves while another may still read its totals
}

}  // namespace dg
