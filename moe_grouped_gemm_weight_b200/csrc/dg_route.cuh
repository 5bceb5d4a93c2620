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

// For choosing only: absolute error below 2^-22 (exponential and reciprocal
// good to 2 ulp, one rounding of the sum between).
__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
// For results: relative error a few 2^-24.
__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

// The two largest of a set in the order (value, lower index first).
struct Top2 {
    float v1 = -INFINITY, v2 = -INFINITY;
    int i1 = 0, i2 = 0;
    __device__ __forceinline__ void add(float x, int i) {  // indices come in rising order
        const bool p = x > v1, q = x > v2;
        i2 = p ? i1 : q ? i : i2;
        i1 = p ? i : i1;
        v2 = fmaxf(v2, fminf(v1, x));
        v1 = fmaxf(v1, x);
    }
};

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
    uint32_t ok = 0;  // bit i: the lane's expert i is eligible
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane * p.per + i;
        if (i < p.per && e < p.E) {
            const float l = logit_at(row + e);
            const float b = p.bias ? p.bias[e] : 0.f;
            const double s = p.softmax ? c[i] / z : 1.0 / (1.0 + exp(-static_cast<double>(l)));
            c[i] = s + static_cast<double>(b);
            if (l != -INFINITY && b != -INFINITY) ok |= 1u << i;
        } else {
            c[i] = 0.0;
        }
    }
    if (p.groups > 1) {
        unsigned long long mine = 0;
        for (int g = 0; g < p.groups; ++g) {
            // The group's best is removed for the second round, by its index.
            unsigned long long top[2] = {0, 0};
            int taken = -1;
            for (int r = 0; r < p.gtop; ++r) {
                unsigned long long best = 0;
                int at = 0x7FFFFFFF;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const int e = lane * p.per + i;
                    const unsigned long long x =
                        ((ok >> i) & 1u) && e / p.gsize == g && e != taken ? order_key(c[i]) : 0;
                    if (x > best) { best = x; at = e; }
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
        for (int i = 0; i < EPL; ++i)
            if (!((kept >> (((lane * p.per + i) / p.gsize) & 31)) & 1u)) ok &= ~(1u << i);
    }
    int my = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane * p.per + i;
            if (!((ok >> i) & 1u)) continue;
            const unsigned long long x = order_key(p.bias ? c[i] : static_cast<double>(logit_at(row + e)));
            if (x > best) { best = x; at = e; }
        }
        const unsigned long long top = warp_max_u64(best);
        if (top == 0) break;
        at = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
        if (lane == j) my = at;
        if (at / p.per == lane) ok &= ~(1u << (at - lane * p.per));
    }
    return my;
}

// The order of n <= 32 candidates in FP64: lane j < n holds expert e.  Every
// other expert is known to lie below the k-th of them.  Returns the lane's rank.
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

// One warp per token, lane i holding the experts i * per ..; the order within
// a lane, then over the lanes, is the experts' own, so ties fall to the lowest
// lane.  Each lane keeps the two best of its experts: their sums over a
// group's lanes are the group scores, and the k rounds of a warp-wide maximum
// take from them; a lane that gives both looks through its experts again.
template <int EPL, typename L>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_topk_kernel(const RouteParams p) {
    extern __shared__ float route_smem[];  // groups that are not whole lanes: E values per warp
    __shared__ uint16_t cand_smem[kRouteWarps][32];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (t >= p.T) return;
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    const int e0 = lane * p.per;

    float v[EPL];  // logits, then (with a bias) choice values; -inf: not eligible
    if (p.vec) {
        load_logits<EPL>(row + lane * EPL, v);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = i < p.per && e0 + i < p.E ? logit_at(row + e0 + i) : -INFINITY;
    }
    bool odd = false;  // a NaN somewhere, or an infinite choice value
#pragma unroll
    for (int i = 0; i < EPL; ++i) odd |= v[i] != v[i];

    float mx = 0.f, rz = 1.f;
    if (p.softmax) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
        mx = warp_max(m);
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) z += __expf(v[i] - mx);
        rz = 1.f / warp_sum(z);
        odd |= rz != rz && mx != -INFINITY;  // an infinite logit
    }
    // FP32 moves a choice value by less than `slack` (of the largest score:
    // exponential, sum and reciprocal of a softmax 2^-20, sigmoid_fast 2^-22),
    // and adding the bias by 2^-24 of the value.
    const float slack = p.softmax ? rz * 0x1p-20f : 0x1p-22f;

    if (p.bias != nullptr) {
        float b[EPL];
        if (p.vec) {
            load_logits<EPL>(p.bias + lane * EPL, b);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = i < p.per && e0 + i < p.E ? p.bias[e0 + i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float s = p.softmax ? __expf(v[i] - mx) * rz : sigmoid_fast(v[i]);
            v[i] = v[i] == -INFINITY ? -INFINITY : s + b[i];
            odd |= !(v[i] < INFINITY);
        }
    }
    odd = __any_sync(0xffffffffu, odd);

    Top2 best;
#pragma unroll
    for (int i = 0; i < EPL; ++i) best.add(v[i], i);
    bool in = true, sure = true;  // in: the lane's experts take part
    if (p.groups > 1 && !odd) {
        // A choice value without a bias is the score of the logit.
        auto score = [&](float x) {
            return x == -INFINITY || p.bias != nullptr ? x : p.softmax ? __expf(x - mx) * rz : sigmoid_fast(x);
        };
        float a, b;
        int g, first, stride;  // this lane's group, and the lanes that hold the groups' sums
        if (p.group_lanes) {
            a = score(best.v1);
            b = score(best.v2);
            g = lane / p.group_lanes;
            stride = p.group_lanes;
            first = p.group_lanes;
        } else {
            // 2^sh lanes share a group in shared memory.
            float* cs = route_smem + warp * p.E;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i < p.per && e0 + i < p.E) cs[e0 + i] = score(v[i]);
            __syncwarp();
            const int sh = 31 - __clz(32 / p.groups);
            g = lane >> sh;
            stride = first = 1 << sh;
            a = b = -INFINITY;
            if (g < p.groups) {
                const int sub = lane & (stride - 1);
                // Each group starts at another place: the same places of groups of 32 share a bank.
                const int turn = (g << sh) % p.gsize;
                for (int n = sub; n < p.gsize; n += stride) {
                    const float x = cs[g * p.gsize + (n + turn < p.gsize ? n + turn : n + turn - p.gsize)];
                    b = fmaxf(b, fminf(a, x));
                    a = fmaxf(a, x);
                }
            }
        }
        for (int o = first >> 1; o >= 1; o >>= 1) {
            const float xa = __shfl_xor_sync(0xffffffffu, a, o), xb = __shfl_xor_sync(0xffffffffu, b, o);
            b = fmaxf(fmaxf(b, xb), fminf(a, xa));
            a = fmaxf(a, xa);
        }
        float sum = a + (p.gtop == 2 && b != -INFINITY ? b : 0.f);
        if (g >= p.groups) sum = -INFINITY;
        int rank = 0;
        for (int h = 0; h < p.groups; ++h) {
            const float o = __shfl_sync(0xffffffffu, sum, h * stride);
            rank += (o > sum || (o == sum && h < g)) ? 1 : 0;
        }
        const bool kept = sum != -INFINITY && rank < p.keep;
        // Certain when the worst kept group and the best other are clearly apart.
        const float lo = warp_min(kept ? sum : INFINITY), hi = warp_max(kept ? -INFINITY : sum);
        if (hi != -INFINITY && !(lo - hi > 4.f * slack + 0x1p-21f * (fabsf(lo) + fabsf(hi)))) sure = false;
        if (p.group_lanes) {
            in = kept;
            if (!kept) best = Top2();
        } else {
            const uint32_t lanes = __ballot_sync(0xffffffffu, kept);
            best = Top2();
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t grp = (static_cast<uint32_t>(e0 + i) * p.gsize_magic) >> 20;
                if (!((lanes >> ((grp * stride) & 31u)) & 1u)) v[i] = -INFINITY;
                best.add(v[i], i);
            }
        }
    }

    // k rounds, with a bias one more for the runner-up.
    int my = -1;
    float my_v = -INFINITY;
    bool two = true;  // v2 is the lane's second best
    const int rounds = p.k + (p.bias != nullptr ? 1 : 0);
    for (int j = 0; j < rounds; ++j) {
        const float top = warp_max(best.v1);
        if (top == -INFINITY) break;
        const int wl = __ffs(__ballot_sync(0xffffffffu, best.v1 == top)) - 1;
        const int wi = __shfl_sync(0xffffffffu, best.i1, wl);
        if (lane == j) {
            my = wl * p.per + wi;
            my_v = top;
        }
        if (lane == wl) {
            if (two) {
                best.v1 = best.v2;
                best.i1 = best.i2;
                two = false;
            } else {
                best = Top2();
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    best.add(v[i] < top || (v[i] == top && i > wi) ? v[i] : -INFINITY, i);
                two = true;
            }
        }
    }
    int slot = lane;
    if (p.bias != nullptr && sure && !odd) {
        // Neighbours in the order must be clearly apart, or equal because both
        // logit and bias are (then the lower index is right).
        const int next = __shfl_down_sync(0xffffffffu, my, 1);
        const float next_v = __shfl_down_sync(0xffffffffu, my_v, 1);
        bool apart = true;
        if (lane < p.k && next >= 0)
            apart = my_v - next_v > 2.f * slack + 0x1p-22f * (fabsf(my_v) + fabsf(next_v)) ||
                    (logit_at(row + my) == logit_at(row + next) && p.bias[my] == p.bias[next]);
        if (!__all_sync(0xffffffffu, apart)) {
            // All experts that may belong to the k: those not clearly below the k-th.
            const float last = __shfl_sync(0xffffffffu, my_v, p.k - 1);
            const float floor_v = last - (2.f * slack + 0x1p-21f * fabsf(last));
            int n = 0, e = -1;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const bool c = in && v[i] >= floor_v && v[i] != -INFINITY;
                const uint32_t who = __ballot_sync(0xffffffffu, c);
                const int at = n + __popc(who & ((1u << lane) - 1u));
                if (c && at < 32) cand_smem[warp][at] = static_cast<uint16_t>(e0 + i);
                n += __popc(who);
            }
            __syncwarp();
            if (n <= 32) {
                if (lane < n) e = cand_smem[warp][lane];
                slot = rank_candidates<EPL, L>(p, row, n, e);
                my = e;
                if (lane >= n) slot = 32;
                // Fewer experts than slots: lanes past them fill the rest.
                if (lane >= n && lane < p.k) {
                    my = -1;
                    slot = lane;
                }
            } else {
                sure = false;
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
    if (p.renorm) s = s / (warp_sum(s) + kRouteEps);
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
// One warp per token; only softmax reads the whole row.
template <int EPL, typename L>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_topk_bwd_kernel(const RouteBwdParams p) {
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
        g = p.dw[t * p.k + lane] * p.scale;
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
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            d[i] = mx == -INFINITY ? 0.f : expf(d[i] - mx);  // every expert masked: no score, no gradient
            z += d[i];
        }
        rz = mx == -INFINITY ? 0.f : 1.f / warp_sum(z);
    }
    float s = 0.f;
    if (e >= 0) s = !p.softmax ? sigmoid_f(x) : mx == -INFINITY ? 0.f : expf(x - mx) * rz;
    else g = 0.f;
    if (p.renorm) {
        const float r = 1.f / (warp_sum(s) + kRouteEps);
        const float mean = warp_sum(g * s) * r;  // all lanes take part
        g = e < 0 ? 0.f : (g - mean) * r;
    }
    float dot = 0.f;
    if (p.softmax) {
        dot = warp_sum(g * s);
    } else {
        g *= s * (1.f - s);
    }
    float r[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) r[i] = -dot;
    for (int j = 0; j < p.k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j) - e0;
        const float gj = __shfl_sync(0xffffffffu, g, j);
        // -1 - e0 matches no i in range; another lane's expert neither
#pragma unroll
        for (int i = 0; i < EPL; ++i) r[i] += i == ej && i < p.per ? gj : 0.f;
    }
    if (p.softmax) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) r[i] *= d[i] * rz;
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
