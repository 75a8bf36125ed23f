// Choice of experts and routing weights of one token by one warp, from its fp64
// logits: scores, selection values, groups, top-k.
//
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e - max) / sum exp(l - max)
//   c_e = s_e + b_e                     b only steers the selection
//   G_g = sum of the group_top largest c of group g (E / n_group neighbours)
//   the topk_group groups of largest G, then the k experts of largest c in them;
//   equal values go to the lower group or expert index
//   w_j = scale * s_j [/ sum of the chosen s]
//
// Everything that decides the choice is held in fp64: with a few hundred experts
// two neighbouring c lie within fp32's rounding of each other once in a few
// thousand tokens, so an fp32 choice would depend on the order of the sums.
//
// b_e = -inf masks expert e (as l_e = -inf does): it adds nothing to its group,
// ranks below every unmasked expert and weighs 0.  A NaN c ranks like a masked
// one and keeps its NaN weight.  A token without any finite score gets the first
// experts and weights 0.
#pragma once

#include "common.cuh"

namespace moe {

struct RouteChoice {
    int E, k, sigmoid, n_group, topk_group, group_top, renorm;
    float scale;
    const float* bias;
};

// Order-preserving map of double to uint64; NaN ranks with -inf.  0 is below every value.
__device__ __forceinline__ unsigned long long order_key(double c) {
    if (c != c) c = -INFINITY;
    const unsigned long long b = (unsigned long long)__double_as_longlong(c + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(unsigned long long q) {
    return __longlong_as_double((long long)((q >> 63) ? (q & 0x7fffffffffffffffull) : ~q));
}

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long q) {
    const unsigned hi = unsigned(q >> 32), mh = __reduce_max_sync(0xffffffffu, hi);
    const unsigned lo = hi == mh ? unsigned(q) : 0u;
    return ((unsigned long long)mh << 32) | __reduce_max_sync(0xffffffffu, lo);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// l: the token's E logits, keys: scratch for E keys, both in this warp's shared
// memory (l complete, __syncwarp done).  VPL * 32 >= E.
template <int VPL>
__device__ __forceinline__ void route_choose_warp(const double* l, unsigned long long* keys, const RouteChoice& p,
                                                  int lane, int32_t* idx_out, float* w_out) {
    double mx = 0.0, inv = 1.0;
    if (!p.sigmoid) {
        mx = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 32 * i;
            if (e < p.E) {
                mx = fmax(mx, l[e]);
                nan |= l[e] != l[e];
            }
        }
        mx = key_value(warp_max_key(order_key(mx)));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 32 * i;
            if (e < p.E && l[e] != -INFINITY) sum += exp(l[e] - mx);
        }
        sum = warp_sum(sum);
        inv = 1.0 / sum;
        if (__any_sync(0xffffffffu, nan)) inv = __longlong_as_double(0x7ff8000000000000ll);
    }
    auto score = [&](double v) -> double {
        if (v == -INFINITY) return 0.0;
        return p.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - mx) * inv;
    };
    const unsigned long long masked = order_key(-INFINITY);

    unsigned long long q[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        q[i] = 0;
        if (e < p.E) {
            const float b = p.bias ? __ldg(p.bias + e) : 0.0f;
            q[i] = (b == -INFINITY || l[e] == -INFINITY) ? masked : order_key(score(l[e]) + (double)b);
        }
    }

    if (p.topk_group < p.n_group) {
        // 2^x lanes per group find its two largest keys; then the groups are chosen like experts
        const int gs = p.E / p.n_group;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 32 * i;
            if (e < p.E) keys[e] = q[i];
        }
        __syncwarp();
        int per = 1;
        while (per * 2 * p.n_group <= 32) per *= 2;
        const int g = lane / per, r = lane % per;
        unsigned long long a = 0, b = 0;   // largest, second largest
        if (g < p.n_group) {
            for (int e = g * gs + r; e < (g + 1) * gs; e += per) {
                const unsigned long long v = keys[e];
                if (v > a) { b = a; a = v; } else if (v > b) b = v;
            }
        }
        for (int off = per / 2; off >= 1; off >>= 1) {
            const unsigned long long oa = __shfl_xor_sync(0xffffffffu, a, off);
            const unsigned long long ob = __shfl_xor_sync(0xffffffffu, b, off);
            const unsigned long long lo = a < oa ? a : oa;
            a = a < oa ? oa : a;
            b = b < ob ? ob : b;
            b = b < lo ? lo : b;
        }
        unsigned long long gq = 0;
        if (g < p.n_group && r == 0) {
            double G = key_value(a);
            if (p.group_top == 2 && b > masked) G += key_value(b);
            gq = order_key(G);
        }
        unsigned kept = 0;   // bit g: group g takes part
        for (int j = 0; j < p.topk_group; j++) {
            const unsigned long long best = warp_max_key(gq);
            const int win = __reduce_min_sync(0xffffffffu, gq == best && gq != 0 ? unsigned(g) : 0xffffffffu);
            kept |= 1u << win;
            if (g == win) gq = 0;
        }
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 32 * i;
            if (e < p.E && !((kept >> (e / gs)) & 1u)) q[i] = 0;
        }
    }

    int my_e = 0;
    for (int j = 0; j < p.k; j++) {
        unsigned long long best = 0;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (q[i] > best) { best = q[i]; bi = i; }   // ascending e within the lane: ties keep the lower
        const unsigned long long top = warp_max_key(best);
        const int win = (int)__reduce_min_sync(0xffffffffu, best == top ? unsigned(lane + 32 * bi) : 0xffffffffu);
        if (lane == j) my_e = win;
        if ((win & 31) == lane) {
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (i == (win >> 5)) q[i] = 0;
        }
    }
    double s = 0.0;
    if (lane < p.k) {
        const float b = p.bias ? __ldg(p.bias + my_e) : 0.0f;
        s = b == -INFINITY ? 0.0 : score(l[my_e]);
    }
    if (p.renorm) {
        const double den = warp_sum(s);
        s = den == 0.0 ? 0.0 : s / den;
    }
    if (lane < p.k) {
        idx_out[lane] = my_e;
        w_out[lane] = (float)(s * (double)p.scale);
    }
    __syncwarp();
}

}  // namespace moe
