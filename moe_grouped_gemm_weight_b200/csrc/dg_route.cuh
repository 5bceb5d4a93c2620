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
    int softmax, renorm;
    float scale;
};

__device__ __forceinline__ float logit_at(const float* p) { return *p; }
__device__ __forceinline__ float logit_at(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

// Order-preserving integer keys: a < b <=> key(a) < key(b); both zeros share a
// key, NaN is above everything, and 0 is left for "not eligible".
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
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
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const unsigned long long x = __shfl_xor_sync(0xffffffffu, v, o);
        v = x > v ? x : v;
    }
    return v;
}

__device__ __forceinline__ float sigmoid_f(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

// Keep the `keep` best groups: lane g holds group g's key (0: no eligible
// expert).  Ties go to the lower group.  Returns the mask of kept groups.
template <typename Key>
__device__ __forceinline__ uint32_t keep_groups(Key key, int groups, int keep) {
    const int lane = threadIdx.x & 31;
    int rank = 0;
    for (int h = 0; h < groups; ++h) {
        const Key o = __shfl_sync(0xffffffffu, key, h);
        rank += (o > key || (o == key && h < lane)) ? 1 : 0;
    }
    return __ballot_sync(0xffffffffu, lane < groups && key != 0 && rank < keep);
}

// The choice in FP64, for a token whose FP32 order is not certain.  Lane j < k
// returns the j-th expert, or -1.  Plain rather than fast: few tokens need it.
template <int EPL, typename L>
__device__ __noinline__ int choose_exact(const RouteParams& p, const L* row) {
    const int lane = threadIdx.x & 31;
    double c[EPL];
    double m = -INFINITY, z = 1.0;
    if (p.softmax) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane;
            if (e < p.E) {
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
            const int e = i * 32 + lane;
            c[i] = e < p.E ? exp(static_cast<double>(logit_at(row + e)) - m) : 0.0;
            z += c[i];
        }
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    uint32_t ok = 0;  // bit i: expert i * 32 + lane is eligible
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        if (e < p.E) {
            const float l = logit_at(row + e);
            const float b = p.bias ? p.bias[e] : 0.f;
            const double s = p.softmax ? c[i] / z : 1.0 / (1.0 + exp(-static_cast<double>(l)));
            c[i] = s + static_cast<double>(b);
            if (l != -INFINITY && b != -INFINITY) ok |= 1u << i;
        }
    }
    if (p.groups > 1) {
        unsigned long long mine = 0;
        for (int g = 0; g < p.groups; ++g) {
            // The group's two best, by key; sums only where an expert is eligible.
            double a = 0.0, b = 0.0;
            unsigned long long ka = 0, kb = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = i * 32 + lane;
                const unsigned long long x = order_key(c[i]);
                if (((ok >> i) & 1u) && e / p.gsize == g) {
                    if (x > ka) { kb = ka; b = a; ka = x; a = c[i]; }
                    else if (x > kb) { kb = x; b = c[i]; }
                }
            }
            for (int o = 16; o >= 1; o >>= 1) {
                const unsigned long long xa = __shfl_xor_sync(0xffffffffu, ka, o);
                const unsigned long long xb = __shfl_xor_sync(0xffffffffu, kb, o);
                const double ya = __shfl_xor_sync(0xffffffffu, a, o), yb = __shfl_xor_sync(0xffffffffu, b, o);
                if (xa > ka) {
                    if (ka > xb) { kb = ka; b = a; } else { kb = xb; b = yb; }
                    ka = xa; a = ya;
                } else if (xa > kb) {
                    kb = xa; b = ya;
                }
            }
            const double sum = a + (p.gtop == 2 && kb ? b : 0.0);
            if (lane == g) mine = ka ? order_key(sum) : 0;
        }
        const uint32_t kept = keep_groups(mine, p.groups, p.keep);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (!((kept >> ((i * 32 + lane) / p.gsize & 31)) & 1u)) ok &= ~(1u << i);
    }
    int my = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane;
            const unsigned long long x = (ok >> i) & 1u ? order_key(p.bias ? c[i] : static_cast<double>(logit_at(row + e))) : 0;
            if (x > best) { best = x; at = e; }
        }
        const unsigned long long top = warp_max_u64(best);
        if (top == 0) break;
        at = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
        if (lane == j) my = at;
        if ((at & 31) == lane) ok &= ~(1u << (at >> 5));
    }
    return my;
}

// One warp per token; lane holds experts i * 32 + lane.
template <int EPL, typename L>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_topk_kernel(const RouteParams p) {
    extern __shared__ float route_smem[];  // grouped only: E choice values per warp
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
    if (t >= p.T) return;
    const L* row = static_cast<const L*>(p.logits) + t * p.E;

    float l[EPL], c[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        l[i] = e < p.E ? logit_at(row + e) : -INFINITY;
    }
    // Scores.  Without a bias or groups the order is the logits' own, and only
    // the chosen experts' scores are needed.
    float mx = 0.f, rz = 1.f, s_max = 1.f;
    if (p.softmax) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
        mx = warp_max(m);
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            c[i] = expf(l[i] - mx);
            z += c[i];
        }
        rz = 1.f / warp_sum(z);
        s_max = rz;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] *= rz;
    } else if (p.bias != nullptr || p.groups > 1) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = sigmoid_f(l[i]);
    }
    uint32_t key[EPL];
    bool sure = true;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        bool ok = l[i] != -INFINITY && e < p.E;
        if (p.bias != nullptr) {
            const float b = e < p.E ? p.bias[e] : -INFINITY;
            c[i] += b;
            ok = ok && b != -INFINITY;
        }
        key[i] = ok ? order_key(p.bias != nullptr ? c[i] : l[i]) : 0u;
    }
    // FP32 can have moved a choice value by less than 2^-21 of the largest
    // score (exp, sum, reciprocal) and 2^-24 of its own size (adding the bias).
    const float slack = s_max * 0x1p-20f;

    if (p.groups > 1) {
        float* cs = route_smem + warp * p.E;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = i * 32 + lane;
            if (e < p.E) cs[e] = key[i] ? c[i] : -INFINITY;
        }
        __syncwarp();
        // 2^sh lanes share a group: each finds the two best of its share, then
        // the shares are merged.  -inf stands for "none": a choice value of an
        // eligible expert is never -inf.
        const int sh = 31 - __clz(32 / p.groups);
        const int g = lane >> sh, sub = lane & ((1 << sh) - 1);
        float a = -INFINITY, b = -INFINITY;
        bool nan = false;
        if (g < p.groups) {
            // Each group starts at another place: the same places of groups of 32 share a bank.
            const int turn = (g << sh) % p.gsize;
            for (int n = sub; n < p.gsize; n += 1 << sh) {
                const int at = n + turn < p.gsize ? n + turn : n + turn - p.gsize;
                const float x = cs[g * p.gsize + at];
                nan |= x != x;
                b = fmaxf(b, fminf(a, x));
                a = fmaxf(a, x);
            }
        }
        for (int o = (1 << sh) >> 1; o >= 1; o >>= 1) {
            const float xa = __shfl_xor_sync(0xffffffffu, a, o), xb = __shfl_xor_sync(0xffffffffu, b, o);
            nan |= __shfl_xor_sync(0xffffffffu, nan, o);
            b = fmaxf(fmaxf(b, xb), fminf(a, xa));
            a = fmaxf(a, xa);
        }
        const float sum = a + (p.gtop == 2 && b != -INFINITY ? b : 0.f);
        uint32_t gk = nan ? 0xFFFFFFFFu : a == -INFINITY ? 0u : order_key(sum);
        gk = __shfl_sync(0xffffffffu, gk, (lane << sh) & 31);  // lane g holds group g
        if (lane >= p.groups) gk = 0;
        const uint32_t kept = keep_groups(gk, p.groups, p.keep);
        const bool in = (kept >> lane) & 1u;
        // Certain when the worst kept group and the best other are clearly apart.
        const uint32_t lo = __reduce_min_sync(0xffffffffu, in ? gk : 0xFFFFFFFFu);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, in ? 0u : gk);
        if (hi != 0) {
            const float x = key_value(lo), y = key_value(hi);
            if (!(x - y > 2.f * slack + 0x1p-21f * (fabsf(x) + fabsf(y)))) sure = false;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const uint32_t grp = (static_cast<uint32_t>(i * 32 + lane) * p.gsize_magic) >> 20;
            if (!((kept >> (grp & 31u)) & 1u)) key[i] = 0;
        }
    }

    // k rounds of a warp-wide maximum, one more for the runner-up.
    int my = -1;
    uint32_t my_key = 0;
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (key[i] > best) { best = key[i]; at = i * 32 + lane; }
    for (int j = 0; j <= p.k; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0) break;
        const int win = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7FFFFFFF);
        if (lane == j) { my = win; my_key = top; }
        if ((win & 31) == lane) {
            best = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if (i * 32 + lane == win) key[i] = 0;
                if (key[i] > best) { best = key[i]; at = i * 32 + lane; }
            }
        }
    }
    if (p.bias != nullptr) {
        // Neighbours in the order must be clearly apart, or equal because both
        // logit and bias are (then the lower index is right).
        const int next = __shfl_down_sync(0xffffffffu, my, 1);
        const uint32_t next_key = __shfl_down_sync(0xffffffffu, my_key, 1);
        if (lane < p.k && next >= 0) {
            const float x = key_value(my_key), y = key_value(next_key);
            if (!(x - y > 2.f * slack + 0x1p-22f * (fabsf(x) + fabsf(y))) &&
                !(logit_at(row + my) == logit_at(row + next) && p.bias[my] == p.bias[next]))
                sure = false;
        }
    }
    if (!__all_sync(0xffffffffu, sure)) my = choose_exact<EPL, L>(p, row);

    float s = 0.f;
    if (lane < p.k && my >= 0) {
        const float x = logit_at(row + my);
        s = p.softmax ? expf(x - mx) * rz : sigmoid_f(x);
    }
    if (p.renorm) s = s / (warp_sum(lane < p.k ? s : 0.f) + kRouteEps);
    if (lane < p.k) {
        p.idx[t * p.k + lane] = my;
        p.w[t * p.k + lane] = s * p.scale;
    }
}

// ------------------------------------------------------------- gradient ----

struct RouteBwdParams {
    void* dlogits;        // [T][E], the logits' type
    const float* dw;      // [T][k]
    const void* logits;   // [T][E]
    const int32_t* idx;   // [T][k]
    int T, E, k;
    int softmax, renorm;
    float scale;
};

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
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

    int e = -1;
    float g = 0.f;
    if (lane < p.k) {
        e = p.idx[t * p.k + lane];
        if (e < 0 || e >= p.E) e = -1;
        g = p.dw[t * p.k + lane] * p.scale;
    }
    float d[EPL];
    float mx = 0.f, rz = 1.f;
    if (p.softmax) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int x = i * 32 + lane;
            d[i] = x < p.E ? logit_at(row + x) : -INFINITY;
            m = fmaxf(m, d[i]);
        }
        mx = warp_max(m);
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            d[i] = mx == -INFINITY ? 0.f : expf(d[i] - mx);  // every expert masked: no score, no gradient
            z += d[i];
        }
        rz = 1.f / warp_sum(z);
        if (mx == -INFINITY) rz = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] *= rz;
    }
    float s = 0.f;
    if (e >= 0) {
        const float x = logit_at(row + e);
        s = !p.softmax ? sigmoid_f(x) : mx == -INFINITY ? 0.f : expf(x - mx) * rz;
    } else {
        g = 0.f;
    }
    if (p.renorm) {
        const float total = warp_sum(s) + kRouteEps;
        g = (g - warp_sum(g * s) / total) / total;
        if (e < 0) g = 0.f;
    }
    float r[EPL];
    if (p.softmax) {
        const float dot = warp_sum(g * s);
#pragma unroll
        for (int i = 0; i < EPL; ++i) r[i] = -dot;
    } else {
        g *= s * (1.f - s);
#pragma unroll
        for (int i = 0; i < EPL; ++i) r[i] = 0.f;
    }
    for (int j = 0; j < p.k; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, j);
        const float gj = __shfl_sync(0xffffffffu, g, j);
        if (ej >= 0 && (ej & 31) == lane) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == (ej >> 5)) r[i] += gj;
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int x = i * 32 + lane;
        if (x < p.E) store_logit(out + x, p.softmax ? r[i] * d[i] : r[i]);
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
