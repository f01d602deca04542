// Selection of a token's experts from its router scores: softmax, top-k in
// rank order, weighting, and the records of one token, by one warp.
#pragma once

#include "moe_internal.cuh"

#include <math.h>

namespace moe {

struct RouterArgs {
    const void* x;
    const void* W_r;
    const float* b_r;
    const float* lat;
    int32_t* ids;
    float* w;
    float* margin;
    unsigned long long* counters;
    float* Y_zero;
    float* psum;  // [E] sum over tokens of the full-softmax probabilities (nullable)
    int32_t* cand;  // [N, X] rerouting candidates: experts of rank k .. k+X-1 (X > 0 only)
    float* cand_w;  // [N, X] their weights under the layer's normalisation
    int64_t N;
    int d, E, k, norm;
    int X;          // rerouting candidates per token (0: none)
    float theta;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Softmax, top-k in rank order (score descending, ties to the lower expert
// index), weights and records for one token.  The calling warp holds the
// token's scores (bias included) as v[i] = g[lane + 32 i], -inf past E_r.
// ps (shared memory, nullable) accumulates the token's full-softmax
// probabilities per expert, for the mean router probability of the batch.
template <int PER>
__device__ __forceinline__ void select_token(const RouterArgs& a, int64_t t, int lane, float (&v)[PER],
                                             float* ps) {
    const int E = a.E, k = a.k;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !isfinite(v[i])) bad = true;
    }
    // one score that is not finite fails the token: no lane has an expert then
    // (my_e stays -1), whatever its own scores are
    bad = __any_sync(0xffffffffu, bad);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    unsigned taken = 0;
    int my_e = -1;
    float my_g = 0.f, next_g = -INFINITY;
    // ranks 0..k-1 are the chosen experts; rank k gives the margin; ranks
    // k..k+X-1 are the rerouting candidates (lane r holds rank r)
    const int want = k + (a.X > 1 ? a.X : 1);
    const int rounds = want < E ? want : E;
    if (!bad) {
        // order-preserving integer keys (-0 counts as 0), so that the warp's
        // maximum and the lowest index that has it are one instruction each
        auto best = [&](uint32_t& bk, int& be) {
            bk = 0u;
            be = 0x7fffffff;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = lane + 32 * i;
                const uint32_t u = __float_as_uint(v[i] + 0.f);
                const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
                if (!((taken >> i) & 1u) && e < E && key > bk) {
                    bk = key;
                    be = e;
                }
            }
        };
        uint32_t bk;
        int be;
        best(bk, be);
        for (int r = 0; r < rounds; ++r) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
            const int te = (int)__reduce_min_sync(0xffffffffu, bk == top ? (unsigned)be : 0x7fffffffu);
            const uint32_t u = top & 0x80000000u ? top ^ 0x80000000u : ~top;
            const float tv = __uint_as_float(u);
            if (lane == r) {
                my_e = te;
                my_g = tv;
            }
            if (r == k) next_g = tv;
            if ((te & 31) == lane) {
                taken |= 1u << (te >> 5);
                best(bk, be);
            }
        }
    }
    float z = 0.f;
    float ev[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        ev[i] = e < E ? expf(v[i] - m) : 0.f;
        z += ev[i];
    }
    z = warp_sum(z);
    const bool pick = lane < k;
    const float ex = pick && !bad ? expf(my_g - m) : 0.f;
    float wv = 0.f;
    bool active = pick;
    bool lat_bad = false;
    float te = 1.f;
    if (a.norm == MOE_NORM_WLR && pick && !bad) {
        te = a.lat[t * E + my_e];
        lat_bad = !(te > 0.f);  // NaN or non-positive latency
    }
    bad = __any_sync(0xffffffffu, bad || lat_bad);
    const bool is_cand = lane >= k && lane < k + a.X;
    if (bad) {
        if (pick) {
            a.ids[t * k + lane] = -1;
            a.w[t * k + lane] = 0.f;
        }
        if (is_cand) {
            a.cand[t * a.X + (lane - k)] = -1;
            a.cand_w[t * a.X + (lane - k)] = 0.f;
        }
        if (lane == 0) {
            if (a.margin) a.margin[t] = NAN;
            atomicAdd(a.counters + CNT_NONFINITE, 1ull);
        }
        return;
    }
    if (ps) {
        const float iz = 1.f / z;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < E) atomicAdd(&ps[e], ev[i] * iz);
        }
    }
    float sel_sum = 1.f;  // sum of the chosen experts' exp(g - m) (renormalisation)
    if (a.norm == MOE_NORM_FULLPROB) {
        wv = ex / z;
    } else if (a.norm == MOE_NORM_RENORM) {
        sel_sum = warp_sum(ex);
        wv = ex / sel_sum;
    } else {
        const float wlr = (ex / z) / te;  // p_e / t_e (0 when t_e = inf)
        for (;;) {
            const unsigned am = __ballot_sync(0xffffffffu, active);
            if (__popc(am) < 2) break;
            // smallest WLR (on equal WLR the higher expert index) and largest WLR
            float mn = active ? wlr : INFINITY;
            int mne = active ? my_e : -1;
            float mx = active ? wlr : -INFINITY;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float ov = __shfl_xor_sync(0xffffffffu, mn, o);
                const int oe = __shfl_xor_sync(0xffffffffu, mne, o);
                if (ov < mn || (ov == mn && oe > mne)) {
                    mn = ov;
                    mne = oe;
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            const float ratio = mn / (mn + mx);
            if (ratio <= a.theta) {
                if (active && my_e == mne) active = false;
            } else {
                break;
            }
        }
        const float s = warp_sum(active ? ex : 0.f);
        wv = active ? ex / s : 0.f;
        if (active && isinf(te)) wv = 0.f;  // disconnected expert: weight 0
    }
    if (pick) {
        a.ids[t * k + lane] = active ? my_e : -1;
        a.w[t * k + lane] = wv;
    }
    if (is_cand) {
        // the expert of rank `lane`, weighted against the chosen set as the
        // chosen experts are (full probability: p; renormalised: p / sum_S p)
        const bool have = lane < E;
        const float exc = have ? expf(my_g - m) : 0.f;
        a.cand[t * a.X + (lane - k)] = have ? my_e : -1;
        a.cand_w[t * a.X + (lane - k)] = have ? (a.norm == MOE_NORM_FULLPROB ? exc / z : exc / sel_sum) : 0.f;
    }
    const float kth = __shfl_sync(0xffffffffu, my_g, k - 1);
    const float mg = k < E ? kth - next_g : INFINITY;
    if (lane == 0) {
        if (a.margin) a.margin[t] = mg;
        if (mg < kNearTie) atomicAdd(a.counters + CNT_NEAR_TIE, 1ull);
    }
}

}  // namespace moe
