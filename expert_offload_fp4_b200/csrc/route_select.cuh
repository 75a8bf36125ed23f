// Choice of experts and routing weights of one token by one warp, from its logits:
// scores, selection values, groups, top-k.
//
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e - max) / sum exp(l - max)
//   c_e = s_e + b_e                     b only steers the selection
//   G_g = sum of the group_top largest c of group g (E / n_group neighbours)
//   the topk_group groups of largest G, then the k experts of largest c in them;
//   equal values go to the lower group or expert index
//   w_j = scale * s_j [/ sum of the chosen s]
//
// The choice is the one that fp64 values make: with a few hundred experts two
// neighbouring c lie within fp32's rounding of each other once in a few thousand
// tokens, and an fp32 choice would depend on the order of the sums.  But fp64 scores
// of all experts cost more than all the rest, so the choice is first made in fp32
// (route_fast), with a bound eta on the values' error (eta also covers the error of
// logits that come from the tensor cores), and stands if every distance that decided
// it is above the bounds.  Else (route_attempt) values within their bounds of a
// decision are computed again in fp64, and the choice is repeated until it stands.
//
// b_e = -inf masks expert e (as l_e = -inf does): it adds nothing to its group,
// ranks below every unmasked expert and weighs 0.  A NaN c ranks like a masked
// one and keeps its NaN weight.  A token without any finite score gets the first
// experts and weights 0.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMaxGroups = 32;

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
constexpr unsigned long long kMaskedKey = 0x000fffffffffffffull;   // order_key(-inf)

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

// A warp's scratch for one token, in shared memory: E of each.
struct RouteScratch {
    double* l;                   // logits
    unsigned long long* key;     // order_key of the selection values
    unsigned char* exact;        // 1: that value is the fp64 one
    static __host__ __device__ size_t bytes(int E) { return (size_t(17) * E + 15) / 16 * 16; }
    __device__ RouteScratch(void* p, int E)
        : l(static_cast<double*>(p)), key(reinterpret_cast<unsigned long long*>(l + E)),
          exact(reinterpret_cast<unsigned char*>(key + E)) {}
};

// ---------------------------------------------------------------- fp32 first

__device__ __forceinline__ unsigned order_key32(float c) {
    const unsigned b = __float_as_uint(c + 0.0f);
    return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key32_value(unsigned q) { return __uint_as_float((q >> 31) ? (q & 0x7fffffffu) : ~q); }
constexpr unsigned kMaskedKey32 = 0x007fffffu;   // order_key32(-inf)

// The choice from fp32 logits lf[i] of expert lane + 32 i, each within delta of its logit;
// returns whether it is certain, with my_e the expert of rank `lane`, mx the largest logit.
// sc: scratch of 8 E bytes.
template <int VPL>
__device__ __forceinline__ bool route_fast(const float (&lf)[VPL], const RouteChoice& p, float delta, int lane, void* sc,
                                           float& mx, int& my_e) {
    float* sl = static_cast<float*>(sc);
    unsigned* sk = reinterpret_cast<unsigned*>(sl + p.E);
    bool odd = false;                      // NaN and infinities are left to the 64-bit way
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        if (e >= p.E) continue;
        m = max(m, order_key32(lf[i]));
        odd |= !(lf[i] < INFINITY);
        sl[e] = lf[i];
    }
    mx = key32_value(__reduce_max_sync(0xffffffffu, m));
    if (mx == -INFINITY || delta > 0.05f) odd = true;
    // Without a bias scores order as the logits do: no score is needed for the choice, as long
    // as fp64 scores differ wherever fp32 logits do
    const bool grouped = p.topk_group < p.n_group;
    const bool by_logit = !p.bias && (!grouped || p.group_top == 1) && (!p.sigmoid || mx <= 20.0f);
    float inv = 1.0f;
    if (!p.sigmoid && p.bias) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (lane + 32 * i < p.E) sum += __expf(lf[i] - mx);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        inv = __fdividef(1.0f, sum);
    }
    unsigned q[VPL];
    float cmax = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        q[i] = 0;
        if (e >= p.E) continue;
        float c = lf[i], b = 0.0f;
        if (!by_logit) {
            c = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-lf[i])) : __expf(lf[i] - mx) * inv;
            if (p.bias) {
                b = __ldg(p.bias + e);
                c += b;
            }
            const bool masked = lf[i] == -INFINITY || b == -INFINITY;
            if (masked) c = -INFINITY;
            else odd |= !(fabsf(c) < 1e30f);
            if (!masked) cmax = fmaxf(cmax, fabsf(c));
        }
        q[i] = order_key32(c);
        if (grouped) sk[e] = q[i];
    }
    if (__any_sync(0xffffffffu, odd)) return false;
    // The error of a value: of the logit (|ds/dl| <= 1/4 for a sigmoid), and of the score in
    // fp32 (__expf, sum and quotient: below 2^-21 of the largest score, 2^-18 with a softmax's
    // denominator), and of adding the bias
    float eta;
    if (by_logit) {
        eta = delta;
    } else {
        cmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(cmax)));
        eta = (p.sigmoid ? 0.26f * delta + 0x1p-20f : p.bias ? (2.3f * delta + 0x1p-17f) * inv : 1.1f * delta + 0x1p-19f) +
              cmax * 0x1p-22f;
    }
    __syncwarp();
    if (grouped) {
        // 2^x lanes per group find its two largest; then the groups are chosen like experts
        const int gs = p.E / p.n_group;
        const int sh = 31 - __clz(32 / p.n_group), per = 1 << sh;
        const int g = lane >> sh, r = lane & (per - 1);
        unsigned a = 0, b = 0;
        if (g < p.n_group)
            for (int e = g * gs + r; e < (g + 1) * gs; e += per) {
                const unsigned v = sk[e];
                b = max(b, min(a, v));
                a = max(a, v);
            }
        for (int off = per / 2; off >= 1; off >>= 1) {
            const unsigned oa = __shfl_xor_sync(0xffffffffu, a, off), ob = __shfl_xor_sync(0xffffffffu, b, off);
            b = max(max(b, ob), min(a, oa));
            a = max(a, oa);
        }
        const bool leader = g < p.n_group && r == 0;
        float G = key32_value(a);
        if (p.group_top == 2 && b > kMaskedKey32) G += key32_value(b);
        unsigned left = leader ? order_key32(G) : 0;
        unsigned kept = 0, lowest = 0;   // kept: bit of the leader lane
        for (int j = 0; j < p.topk_group; j++) {
            lowest = __reduce_max_sync(0xffffffffu, left);
            const unsigned win = __ballot_sync(0xffffffffu, left == lowest);
            kept |= win & -win;
            if ((win & -win) >> lane & 1u) left = 0;
        }
        const unsigned next = __reduce_max_sync(0xffffffffu, left);
        // (equal exact logits are a tie, which the lower group has won)
        if (eta > 0.0f && key32_value(lowest) - key32_value(next) <= 2 * p.group_top * eta) return false;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 32 * i;
            if (e < p.E && !((kept >> ((e / gs) << sh)) & 1u)) q[i] = 0;
        }
    }
    // ranks 0 .. k: the last only to compare with
    unsigned my_q = 0, after = 0;
    my_e = 0;
    for (int j = 0; j <= p.k; j++) {
        unsigned best = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++) best = max(best, q[i]);
        const unsigned top = __reduce_max_sync(0xffffffffu, best);
        if (j == p.k) {
            after = top;
            break;
        }
        int at = VPL;
#pragma unroll
        for (int i = VPL - 1; i >= 0; i--) at = q[i] == top ? i : at;
        const unsigned win = __reduce_min_sync(0xffffffffu, at < VPL ? unsigned(lane + 32 * at) : 0xffffffffu);
        if (lane == j) {
            my_e = (int)win;
            my_q = top;
        }
        const int wi = (win & 31) == lane ? int(win >> 5) : -1;
#pragma unroll
        for (int i = 0; i < VPL; i++) q[i] = i == wi ? 0 : q[i];
    }
    // (scores this far down may be equal in fp64)
    if (by_logit && key32_value(__shfl_sync(0xffffffffu, my_q, p.k - 1)) < (p.sigmoid ? -600.0f : mx - 600.0f)) return false;
    if (eta == 0.0f) return true;
    unsigned below = __shfl_down_sync(0xffffffffu, my_q, 1);
    int below_e = __shfl_down_sync(0xffffffffu, my_e, 1);
    if (lane == p.k - 1) {
        below = after;
        below_e = -1;
    }
    bool close = false;
    if (lane < p.k && below != 0 && key32_value(my_q) - key32_value(below) <= 2 * eta)
        // equal exact logits without a bias have equal scores: a tie
        close = !(delta == 0.0f && !p.bias && my_q == below && below_e >= 0 && sl[my_e] == sl[below_e]);
    return !__any_sync(0xffffffffu, close);
}

// ---------------------------------------------------------------- fp64 where it is close

// What the warp knows of the token's softmax (sigmoid: unused).
struct RouteSoftmax {
    double mx = 0.0;     // largest logit
    double inv = 0.0;    // 1 / sum of exp(l - mx), once known in fp64
    bool have_inv = false;
};

__device__ __noinline__ double route_softmax_inv(const double* l, int E, double mx, int lane) {
    double sum = 0.0;
    for (int e = lane; e < E; e += 32)
        if (l[e] != -INFINITY) sum += exp(l[e] - mx);
    return 1.0 / warp_sum(sum);
}

// fp64 score; softmax without its denominator (u = exp(l - mx)).
__device__ __noinline__ double route_score64(double l, int sigmoid, double mx) {
    if (l == -INFINITY) return 0.0;
    return sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - mx);
}

// One attempt at the choice from s.key.  Returns false, with the bits of `mark` set for
// this lane's experts (bit i: expert lane + 32 i) that have to be known exactly first,
// or true with my_e the expert of rank `lane`.
template <int VPL>
__device__ __forceinline__ bool route_attempt(const RouteScratch& s, const RouteChoice& p, double eta, int lane,
                                              unsigned& mark, int& my_e) {
    unsigned long long q[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        q[i] = e < p.E ? s.key[e] : 0;
    }
    mark = 0;
    if (p.topk_group < p.n_group) {
        // 2^x lanes per group find its two largest keys; then the groups are chosen like experts
        const int gs = p.E / p.n_group;
        int per = 1;
        while (per * 2 * p.n_group <= 32) per *= 2;
        const int g = lane / per, r = lane % per;
        unsigned long long a = 0, b = 0;   // largest, second largest
        if (g < p.n_group) {
            for (int e = g * gs + r; e < (g + 1) * gs; e += per) {
                const unsigned long long v = s.key[e];
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
        const bool leader = g < p.n_group && r == 0;
        const bool two = p.group_top == 2 && b > kMaskedKey;
        const double G = two ? key_value(a) + key_value(b) : key_value(a);
        const unsigned long long gq = leader ? order_key(G) : 0;
        unsigned long long left = gq;
        unsigned kept = 0;   // bit g: group g takes part
        unsigned long long lowest = 0;
        for (int j = 0; j < p.topk_group; j++) {
            lowest = warp_max_key(left);
            const int win = (int)__reduce_min_sync(0xffffffffu, left == lowest && left != 0 ? unsigned(g) : 0xffffffffu);
            kept |= 1u << win;
            if (g == win) left = 0;
        }
        const unsigned long long next = warp_max_key(left);
        if (key_value(lowest) - key_value(next) <= 2 * p.group_top * eta) {
            // the last kept group and the first left out are close: which groups are not exact yet?
            const double m = key_value(two ? b : a) - 2 * eta;   // experts below cannot be among the group's best
            bool open = false;
            if (g < p.n_group)
                for (int e = g * gs + r; e < (g + 1) * gs; e += per) open |= !s.exact[e] && key_value(s.key[e]) >= m;
            for (int off = per / 2; off >= 1; off >>= 1) open |= (bool)__shfl_xor_sync(0xffffffffu, (int)open, off);
            const double eg = open ? p.group_top * eta : 0.0;
            const bool in = leader && ((kept >> g) & 1u), out = leader && !((kept >> g) & 1u);
            // (smallest as the largest of the negatives)
            const double low = -key_value(warp_max_key(in ? order_key(-(G - eg)) : 0));
            const double high = key_value(warp_max_key(out ? order_key(G + eg) : 0));
            const bool sel = open && ((in && G - eg <= high) || (out && G + eg >= low));
            const unsigned lanes = __ballot_sync(0xffffffffu, sel);
            if (lanes) {
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const int e = lane + 32 * i, src = e < p.E ? (e / gs) * per : 0;
                    const double mg = __shfl_sync(0xffffffffu, m, src);
                    if (e < p.E && ((lanes >> src) & 1u) && !s.exact[e] && key_value(q[i]) >= mg) mark |= 1u << i;
                }
                return false;
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = lane + 32 * i;
            if (e < p.E && !((kept >> (e / gs)) & 1u)) q[i] = 0;
        }
    }

    unsigned long long my_q = 0;
    my_e = 0;
    for (int j = 0; j < p.k; j++) {
        unsigned long long best = 0;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (q[i] > best) { best = q[i]; bi = i; }   // ascending e within the lane: ties keep the lower
        const unsigned long long top = warp_max_key(best);
        const int win = (int)__reduce_min_sync(0xffffffffu, best == top ? unsigned(lane + 32 * bi) : 0xffffffffu);
        if (lane == j) {
            my_e = win;
            my_q = top;
        }
        const int wi = (win & 31) == lane ? win >> 5 : -1;
#pragma unroll
        for (int i = 0; i < VPL; i++) q[i] = i == wi ? 0 : q[i];
    }

    // Are the ranks safe?  First by plain distances, then by what is known exactly
    const double c = key_value(my_q);
    const double below = __shfl_down_sync(0xffffffffu, c, 1);
    const double last = __shfl_sync(0xffffffffu, c, p.k - 1);
    const unsigned long long near = order_key(last - 2 * eta);
    bool close = lane + 1 < p.k && c - below <= 2 * eta;
#pragma unroll
    for (int i = 0; i < VPL; i++) close |= q[i] != 0 && q[i] >= near;
    if (!__any_sync(0xffffffffu, close)) return true;
    const double my_eta = s.exact[my_e] ? 0.0 : eta;
    unsigned amb = 0;   // ranks to settle
    for (int i = 0; i + 1 < p.k; i++) {
        const double ci = __shfl_sync(0xffffffffu, c, i), m = __shfl_sync(0xffffffffu, my_eta, i) + my_eta;
        const unsigned hit = __ballot_sync(0xffffffffu, lane > i && lane < p.k && m > 0.0 && ci - c <= m);
        if (hit) amb |= hit | (1u << i);
    }
    const double last_eta = __shfl_sync(0xffffffffu, my_eta, p.k - 1);
    bool any = false;
#pragma unroll
    for (int i = 0; i < VPL; i++)
        if (q[i] != 0) {
            const double ei = s.exact[lane + 32 * i] ? 0.0 : eta, m = ei + last_eta;
            if (m > 0.0 && last - key_value(q[i]) <= m) {
                any = true;
                if (ei > 0.0) mark |= 1u << i;
            }
        }
    if (__any_sync(0xffffffffu, any)) amb |= 1u << (p.k - 1);
    for (unsigned r = amb; r; r &= r - 1) {
        const int e = __shfl_sync(0xffffffffu, my_e, __ffs(r) - 1);
        if ((e & 31) == lane && !s.exact[e]) mark |= 1u << (e >> 5);
    }
    return !__any_sync(0xffffffffu, mark != 0);
}

// First selection values, in fp32, from s.l; returns eta.  delta: bound on the error of the
// logits (0: exact).
template <int VPL>
__device__ __forceinline__ double route_first_values(const RouteScratch& s, const RouteChoice& p, double delta, int lane,
                                                     RouteSoftmax& sm) {
    double eta;
    float inv = 1.0f;
    if (p.sigmoid) {
        // |ds/dl| <= 1/4; expf, the sum and the quotient in fp32: below 2^-21 of s <= 1
        eta = 0.26 * delta + 0x1p-20;
    } else {
        unsigned long long m = 0;
        bool nan = false;
        for (int e = lane; e < p.E; e += 32) {
            const unsigned long long v = order_key(s.l[e]);
            m = v > m ? v : m;
            nan |= s.l[e] != s.l[e];
        }
        sm.mx = key_value(warp_max_key(m));
        if (__any_sync(0xffffffffu, nan) || sm.mx == INFINITY) sm.mx = __longlong_as_double(0x7ff8000000000000ll);   // all scores NaN
        // exp(l - mx) <= 1 to 1.1 delta (delta <= 0.05) and fp32's rounding; its argument to
        // |l - mx| 2^-24, which exp's own size makes up for
        eta = 1.1 * delta + 0x1p-19;
        if (p.bias) {
            float sum = 0.0f;
            for (int e = lane; e < p.E; e += 32)
                if (s.l[e] != -INFINITY) sum += __expf((float)(s.l[e] - sm.mx));
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            inv = 1.0f / sum;
            // the denominator errs by as much again; scores are at most inv
            eta = (2.3 * delta + 0x1p-17) * (double)inv;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        if (e >= p.E) continue;
        const double l = s.l[e];
        const float b = p.bias ? __ldg(p.bias + e) : 0.0f;
        unsigned long long q = kMaskedKey;
        bool exact = true;
        if (b != -INFINITY && l != -INFINITY) {
            const float v = p.sigmoid ? 1.0f / (1.0f + __expf(-(float)l)) : __expf((float)(l - sm.mx)) * inv;
            q = order_key((double)v + (double)b);
            exact = v != v;
        }
        s.key[e] = q;
        s.exact[e] = exact;
    }
    __syncwarp();
    return eta;
}

// The fp64 selection value of expert e from s.l[e].
__device__ __forceinline__ void route_make_exact(const RouteScratch& s, const RouteChoice& p, const RouteSoftmax& sm, int e) {
    double v = route_score64(s.l[e], p.sigmoid, sm.mx);
    if (p.bias) v = (p.sigmoid ? v : v * sm.inv) + (double)__ldg(p.bias + e);
    s.key[e] = order_key(v);
    s.exact[e] = 1;
}

// Weights of the chosen experts (my_e: rank `lane`'s, my_l: its logit); inv(): 1 / sum of
// exp(l - mx) over all experts, asked for by the whole warp where the weights need it.
template <class Inv>
__device__ __forceinline__ void route_weights(const RouteChoice& p, double mx, int lane, int my_e, double my_l, Inv inv,
                                              int32_t* idx_out, float* w_out) {
    double v = 0.0;
    if (lane < p.k) {
        const float b = p.bias ? __ldg(p.bias + my_e) : 0.0f;
        v = b == -INFINITY ? 0.0 : route_score64(my_l, p.sigmoid, mx);
    }
    if (p.renorm) {
        const double den = warp_sum(v);
        v = den == 0.0 ? 0.0 : v / den;
    } else if (!p.sigmoid) {
        const double f = inv();
        v = v == 0.0 ? 0.0 : v * f;
    }
    if (lane < p.k) {
        idx_out[lane] = my_e;
        w_out[lane] = (float)(v * (double)p.scale);
    }
}

// The whole choice for logits that are exact (s.l complete, __syncwarp done).
template <int VPL>
__device__ __noinline__ void route_choose_exact(const RouteScratch s, const RouteChoice& p, int lane, int32_t* idx_out,
                                                float* w_out) {
    RouteSoftmax sm;
    const double eta = route_first_values<VPL>(s, p, 0.0, lane, sm);
    unsigned mark;
    int my_e;
    while (!route_attempt<VPL>(s, p, eta, lane, mark, my_e)) {
        if (!p.sigmoid && p.bias && !sm.have_inv) {
            sm.inv = route_softmax_inv(s.l, p.E, sm.mx, lane);
            sm.have_inv = true;
        }
        for (; mark; mark &= mark - 1) route_make_exact(s, p, sm, lane + 32 * (__ffs(mark) - 1));
        __syncwarp();
    }
    route_weights(p, sm.mx, lane, my_e, s.l[my_e],
                  [&]() { return sm.have_inv ? sm.inv : route_softmax_inv(s.l, p.E, sm.mx, lane); }, idx_out, w_out);
    __syncwarp();
}

// Weights after a certain route_fast, whose logits are lf (given as fp64 by l64 where that is more).
template <int VPL, class L64>
__device__ __forceinline__ void route_fast_weights(const float (&lf)[VPL], const RouteChoice& p, float mx, int lane, int my_e,
                                                   L64 l64, int32_t* idx_out, float* w_out) {
    const double m = mx;
    route_weights(p, m, lane, my_e, l64(my_e), [&]() {
        double sum = 0.0;
#pragma unroll 1
        for (int e = lane; e < p.E; e += 32) sum += exp(l64(e) - m);
        return 1.0 / warp_sum(sum);
    }, idx_out, w_out);
}

}  // namespace moe
