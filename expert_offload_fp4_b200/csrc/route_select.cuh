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
// it is above the bounds, eta's or the experts' own (route_groups_clear, route_ranks_clear).  Groups or ranks that are closer are settled by the fp64 values
// of the few experts they hang on (route_settle_groups, then route_fast again with the
// groups given; route_settle).  What is left, such as more than 32 such experts, goes
// through route_attempt: values within their bounds of a decision are computed again in
// fp64, and the choice is repeated until it stands.  (With every close pair of groups
// left to route_attempt, the few tokens that have one were a launch's tail: 2.4 us more for
// 16 tokens of 4096 x 256, 6 for 512.)
//
// b_e = -inf masks expert e (as l_e = -inf does): it adds nothing to its group,
// ranks below every unmasked expert and weighs 0.  A NaN c ranks like a masked
// one and keeps its score's weight (NaN unless only b was).  A token whose experts are
// all masked gets the first ones and weights 0.
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

// A warp's scratch for one token, in shared memory.  fill() the logits and biases of all
// experts before the choice; the fp64 way reuses the fp32 arrays.
struct RouteScratch {
    double* l;                   // logits
    float *l32, *bias;           // in fp32, and the bias (0 without one)
    unsigned* key32;             // order_key32 of the selection values
    unsigned long long* key;     // order_key of the selection values (overlays l32 and key32)
    unsigned char* exact;        // 1: that value is the fp64 one (overlays bias)
    static __host__ __device__ size_t bytes(int E) { return (size_t(20) * E + 15) / 16 * 16; }
    __device__ RouteScratch(void* p, int E)
        : l(static_cast<double*>(p)), l32(reinterpret_cast<float*>(l + E)), bias(l32 + 2 * E),
          key32(reinterpret_cast<unsigned*>(l32 + E)), key(reinterpret_cast<unsigned long long*>(l32)),
          exact(reinterpret_cast<unsigned char*>(bias)) {}
    __device__ __forceinline__ void fill(int e, double v, float v32, float b) const {
        l[e] = v;
        l32[e] = v32;
        bias[e] = b;
    }
};

// ---------------------------------------------------------------- fp32 first

__device__ __forceinline__ unsigned order_key32(float c) {
    const unsigned b = __float_as_uint(c + 0.0f);
    return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key32_value(unsigned q) { return __uint_as_float((q >> 31) ? (q & 0x7fffffffu) : ~q); }
constexpr unsigned kMaskedKey32 = 0x007fffffu;   // order_key32(-inf)

enum RouteStatus {
    kRouteCertain,   // the choice stands
    kRouteClose,     // the groups stand, but some ranks are too close to call: see RouteClose
    kRouteGroups,    // groups are too close to call: see RouteClose
    kRouteOpen       // left to the 64-bit way
};

// The ranks and the experts just below them, one a lane (lanes >= n: none); or, where groups are
// close, the experts that may count in one of those.
struct RouteClose {
    int n = 0, e = 0;
    unsigned kept = 0;   // the groups that are certainly kept, in route_fast's form
    bool want = false;   // its logit has to be known exactly
};

// A warp's best expert by 32-bit keys, taken out of sk; each lane keeps the best of its experts
// lane, lane + 32, ...  (Here and below short loops over shared memory, not unrolled copies over
// registers: a decode step runs this once, at the speed at which it can fetch the instructions;
// 2.0 us against 5.7 for 256 experts.)
struct RouteTop32 {
    unsigned* sk;
    int E, lane, e = 0, e2 = 0;
    unsigned q = 0, q2 = 0;      // the lane's best and second
    bool two = false;            // the second is known
    __device__ __forceinline__ RouteTop32(unsigned* sk_, int E_, int lane_) : sk(sk_), E(E_), lane(lane_) { rescan(); }
    __device__ __forceinline__ void rescan() {
        q = q2 = 0;
#pragma unroll 4
        for (int i = lane; i < E; i += 32) {
            const unsigned v = sk[i];
            if (v > q) {      // ascending e: ties keep the lower
                q2 = q;
                e2 = e;
                q = v;
                e = i;
            } else if (v > q2) {
                q2 = v;
                e2 = i;
            }
        }
        two = true;
    }
    __device__ __forceinline__ unsigned best() const { return __reduce_max_sync(0xffffffffu, q); }
    // the lowest expert whose key is `top`, which no longer takes part
    __device__ __forceinline__ int take(unsigned top) {
        const int win = (int)__reduce_min_sync(0xffffffffu, q == top ? unsigned(e) : 0xffffffffu);
        if (q == top && e == win) {
            sk[win] = 0;
            if (two) {
                q = q2;
                e = e2;
                two = false;
            } else {
                rescan();
            }
        }
        return win;
    }
};

// An expert's own error, which may be far less than the bound for all: a sigmoid's goes with its slope
// s (1 - s) (which changes by less than 6 % within delta <= 0.05), a softmax's with the score (2.3 delta of
// the logits and the denominator, fp32's 2^-17 and that of the argument).  sk: the keys of the values.
struct RouteErrors {
    const float* sl;
    const unsigned* sk;
    float mx, inv, delta, cmax;
    int sigmoid;
    __device__ __forceinline__ float of(int e) const {
        if (sigmoid) {
            const float v = __fdividef(1.0f, 1.0f + __expf(-sl[e]));
            return 1.06f * delta * (v * (1.0f - v)) + 0x1p-20f + cmax * 0x1p-22f;
        }
        const float d = mx - sl[e];
        return (2.3f * delta + 0x1p-17f + d * 0x1p-22f) * __expf(-d) * inv + cmax * 0x1p-22f;
    }
};

// Is the least that a kept group's value can be above the most that any other's can, by the experts' own
// errors?  per lanes a group (r: which), as in route_fast; in: this leader's group is kept.
__device__ __noinline__ bool route_groups_clear(const RouteErrors errors, int gs, bool any, int g, int r, int per, bool leader,
                                                bool in, int group_top) {
    float hi[2] = {-INFINITY, -INFINITY}, lo[2] = {-INFINITY, -INFINITY};   // the two largest of either
    if (any)
        for (int e = g * gs + r; e < (g + 1) * gs; e += per) {
            const unsigned q = errors.sk[e];
            if (q <= kMaskedKey32) continue;
            const float v = key32_value(q), own = errors.of(e);
            hi[1] = fmaxf(hi[1], fminf(hi[0], v + own));
            hi[0] = fmaxf(hi[0], v + own);
            lo[1] = fmaxf(lo[1], fminf(lo[0], v - own));
            lo[0] = fmaxf(lo[0], v - own);
        }
    for (int off = per / 2; off >= 1; off >>= 1) {
        const float h0 = __shfl_xor_sync(0xffffffffu, hi[0], off), h1 = __shfl_xor_sync(0xffffffffu, hi[1], off);
        const float l0 = __shfl_xor_sync(0xffffffffu, lo[0], off), l1 = __shfl_xor_sync(0xffffffffu, lo[1], off);
        hi[1] = fmaxf(fmaxf(hi[1], h1), fminf(hi[0], h0));
        hi[0] = fmaxf(hi[0], h0);
        lo[1] = fmaxf(fmaxf(lo[1], l1), fminf(lo[0], l0));
        lo[0] = fmaxf(lo[0], l0);
    }
    const bool two = group_top == 2 && lo[1] > -INFINITY;
    const unsigned most = __reduce_max_sync(0xffffffffu, leader && !in ? order_key32(two ? hi[0] + hi[1] : hi[0]) : 0u);
    const unsigned least = ~__reduce_max_sync(0xffffffffu, leader && in ? ~order_key32(two ? lo[0] + lo[1] : lo[0]) : 0u);
    return least > most;
}

// Is every rank clear of the next (my_e, my_q: expert and key of rank `lane`), and the last of all that is
// left, by the experts' own errors?
__device__ __noinline__ bool route_ranks_clear(const RouteErrors errors, int E, int k, int lane, int my_e, unsigned my_q, float eta) {
    const float c = key32_value(my_q), own = errors.of(my_e);
    const float next_c = __shfl_down_sync(0xffffffffu, c, 1), next_own = __shfl_down_sync(0xffffffffu, own, 1);
    bool near = lane < k - 1 && c - next_c <= own + next_own;
    const float low = __shfl_sync(0xffffffffu, c - own, k - 1);
    for (int e = lane; e < E; e += 32) {
        const unsigned v = errors.sk[e];
        if (v > kMaskedKey32 && key32_value(v) + eta >= low) near |= key32_value(v) + errors.of(e) >= low;
    }
    return !__any_sync(0xffffffffu, near);
}

// The lanes of a group, which find its largest values together: 2^route_group_shift.
__device__ __forceinline__ int route_group_shift(int n_group) { return 31 - __clz(32 / n_group); }

// The choice from the fp32 logits, each within delta of its logit.  If it is certain, my_e is
// the expert of rank `lane` (masked: chosen for want of others); mx: the largest logit.
// groups: 0, or the groups to keep (bit: each one's first lane).
__device__ __forceinline__ RouteStatus route_fast(const RouteScratch& s, const RouteChoice& p, float delta, int lane,
                                                  unsigned groups, float& mx, int& my_e, bool& masked, RouteClose& close_out) {
    const float* sl = s.l32;
    unsigned* sk = s.key32;
    bool odd = delta > 0.05f;              // also NaN and infinities: left to the 64-bit way
    bool small = false;
    unsigned m = 0;
#pragma unroll 4
    for (int e = lane; e < p.E; e += 32) {
        const float l = sl[e];
        m = max(m, order_key32(l));
        odd |= !(l < INFINITY);
        small |= l != 0.0f && fabsf(l) < 0x1p-18f;
    }
    mx = key32_value(__reduce_max_sync(0xffffffffu, m));
    odd |= mx == -INFINITY;
    // Without a bias scores order as the logits do: no score is needed for the choice, as long as fp64
    // scores differ wherever fp32 logits do.  Two logits have one score if they are within about
    // 2^-52 (2 + e^l) of each other (sigmoid), or 2^-53 of the distance to the largest, or of 1 (softmax);
    // different fp32 values of 2^-18 or more are 2^-42 apart and 2^-24 of themselves, which is above
    // that up to 20 (sigmoid), and for the distances to 600 that are let through below (softmax)
    const bool grouped = p.topk_group < p.n_group;
    const bool by_logit = !p.bias && (!grouped || p.group_top == 1) && (!p.sigmoid || mx <= 20.0f) &&
                          !__any_sync(0xffffffffu, small);
    float inv = 1.0f;
    if (!p.sigmoid && p.bias) {
        float sum = 0.0f;
        for (int e = lane; e < p.E; e += 32) sum += __expf(sl[e] - mx);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        inv = __fdividef(1.0f, sum);
    }
    float cmax = 0.0f;
#pragma unroll 2
    for (int e = lane; e < p.E; e += 32) {
        const float l = sl[e];
        float c = l;
        if (!by_logit) {
            const float b = s.bias[e];
            const float x = __expf(p.sigmoid ? -l : l - mx);
            c = (p.sigmoid ? __fdividef(1.0f, 1.0f + x) : x * inv) + b;
            const bool out = l == -INFINITY || b == -INFINITY;
            odd |= !out && !(fabsf(c) < 1e30f);
            cmax = fmaxf(cmax, out ? 0.0f : fabsf(c));
            if (out) c = -INFINITY;
        }
        sk[e] = order_key32(c);
    }
    if (__any_sync(0xffffffffu, odd)) return kRouteOpen;
    // The error of a value: of the logit (|ds/dl| <= 1/4 for a sigmoid), and of the score in
    // fp32 (__expf, sum and quotient: below 2^-21 of the largest score, 2^-18 with a softmax's
    // denominator), and of adding the bias
    float eta;
    if (by_logit) {
        // (logits that are not exact: with what may make one score of two)
        eta = delta == 0.0f ? 0.0f : delta + (p.sigmoid ? 0x1p-51f * (2.0f + __expf(mx)) : 0x1p-41f);
    } else {
        cmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(cmax)));
        eta = (p.sigmoid ? 0.26f * delta + 0x1p-20f : p.bias ? (2.3f * delta + 0x1p-17f) * inv : 1.1f * delta + 0x1p-19f) +
              cmax * 0x1p-22f;
    }
    const RouteErrors errors{sl, sk, mx, inv, delta, cmax, p.sigmoid};
    const bool sharp = p.sigmoid ? delta > 0.0f && !by_logit : p.bias != nullptr;   // an expert's own error may be less than eta
    __syncwarp();
    if (grouped) {
        // 2^x lanes per group find its two largest; then the groups are chosen like experts
        const int gs = p.E / p.n_group;
        const int sh = route_group_shift(p.n_group), per = 1 << sh;
        const int g = lane >> sh, r = lane & (per - 1);
        unsigned a = 0, b = 0;
        if (g < p.n_group && groups == 0) {
#pragma unroll 2
            for (int e = r; e < gs; e += per) {
                const unsigned v = sk[g * gs + e];
                b = max(b, min(a, v));
                a = max(a, v);
            }
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
#pragma unroll 1
        for (int j = 0; j < p.topk_group; j++) {
            lowest = __reduce_max_sync(0xffffffffu, left);
            const unsigned win = __ballot_sync(0xffffffffu, left == lowest);
            kept |= win & -win;
            if ((win & -win) >> lane & 1u) left = 0;
        }
        const unsigned next = __reduce_max_sync(0xffffffffu, left);
        bool clear = groups != 0 || eta == 0.0f || !(key32_value(lowest) - key32_value(next) <= 2 * p.group_top * eta);
        if (!clear && sharp)
            clear = route_groups_clear(errors, gs, g < p.n_group, g, r, per, leader, (kept >> lane) & 1u, p.group_top);
        if (groups) {
            kept = groups;
        } else if (!clear) {
            // The groups that could change places over the boundary, and their experts that could
            // be among the ones that count
            const float tol = 2 * p.group_top * eta;
            const bool in = (kept >> lane) & 1u;
            const unsigned open = __ballot_sync(0xffffffffu, leader && (in ? G - key32_value(next) <= tol
                                                                           : key32_value(lowest) - G <= tol));
            const float floor = key32_value(p.group_top == 2 && b > kMaskedKey32 ? b : a) - 2 * eta;
            int n = 0;
            for (int i = 0; i < p.E; i += 32) {
                const int at = i + lane, src = at < p.E ? (at / gs) << sh : 0;
                const float low = __shfl_sync(0xffffffffu, floor, src);
                const unsigned v = at < p.E ? sk[at] : 0;
                unsigned h = __ballot_sync(0xffffffffu, ((open >> src) & 1u) && v > kMaskedKey32 && key32_value(v) >= low);
                for (; h; h &= h - 1, n++)
                    if (lane == n) close_out.e = i + __ffs(h) - 1;
            }
            if (n > 32) return kRouteOpen;
            close_out.n = n;
            close_out.kept = kept & ~open;
            close_out.want = lane < n;
            return kRouteGroups;
        }
        // take the other groups out
        if (g < p.n_group && !((kept >> (g << sh)) & 1u))
            for (int e = r; e < gs; e += per) sk[g * gs + e] = 0;
        __syncwarp();
    }
    RouteTop32 top(sk, p.E, lane);
    unsigned my_q = 0;
    my_e = 0;
#pragma unroll 1
    for (int j = 0; j < p.k; j++) {
        const unsigned q = top.best();
        const int win = top.take(q);
        if (lane == j) {
            my_e = win;
            my_q = q;
        }
    }
    masked = my_q == kMaskedKey32;
    const unsigned after = top.best();
    const float last = key32_value(__shfl_sync(0xffffffffu, my_q, p.k - 1));
    // (scores this far down may be equal in fp64)
    if (by_logit && last < (p.sigmoid ? -600.0f : mx - 600.0f)) return kRouteOpen;
    if (eta == 0.0f) return kRouteCertain;
    unsigned below = __shfl_down_sync(0xffffffffu, my_q, 1);
    int below_e = __shfl_down_sync(0xffffffffu, my_e, 1);
    if (lane == p.k - 1) {
        below = after;
        below_e = -1;
    }
    const bool close = lane < p.k && below != 0 && key32_value(my_q) - key32_value(below) <= 2 * eta;
    // (equal exact logits without a bias have equal scores: a tie)
    const bool tie = close && delta == 0.0f && !p.bias && my_q == below && below_e >= 0 && sl[my_e] == sl[below_e];
    if (!__any_sync(0xffffffffu, close && !tie)) return kRouteCertain;
    if (sharp && route_ranks_clear(errors, p.E, p.k, lane, my_e, my_q, eta)) return kRouteCertain;
    const unsigned links = __ballot_sync(0xffffffffu, close);   // bit i: ranks i and i + 1 may change places
    // every rank of a link, and what may come up from below the last rank
    int n = p.k;
    if ((links >> (p.k - 1)) & 1u) {
        const unsigned near = order_key32(last - 2 * eta);
        for (int i = 0; i < p.E; i += 32) {
            const unsigned v = i + lane < p.E ? sk[i + lane] : 0;
            unsigned h = __ballot_sync(0xffffffffu, v != 0 && v >= near);
            for (; h; h &= h - 1, n++)         // one a lane, from lane k on
                if (lane == n) my_e = i + __ffs(h) - 1;
        }
        if (n > 32) return kRouteOpen;
    }
    close_out.n = n;
    close_out.e = my_e;
    close_out.want = lane < p.k ? ((links >> lane) & 1u) || (lane > 0 && ((links >> (lane - 1)) & 1u)) : lane < n;
    return kRouteClose;
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
__device__ __noinline__ bool route_attempt(const RouteScratch s, const RouteChoice& p, double eta, int lane, unsigned& mark,
                                           int& my_e) {
    mark = 0;
    const int gs = p.E / p.n_group;
    unsigned kept = 0xffffffffu;   // bit g: group g takes part
    if (p.topk_group < p.n_group) {
        // 2^x lanes per group find its two largest keys; then the groups are chosen like experts
        const int sh = 31 - __clz(32 / p.n_group), per = 1 << sh;
        const int g = lane >> sh, r = lane & (per - 1);
        unsigned long long a = 0, b = 0;   // largest, second largest
        if (g < p.n_group)
            for (int e = g * gs + r; e < (g + 1) * gs; e += per) {
                const unsigned long long v = s.key[e];
                if (v > a) { b = a; a = v; } else if (v > b) b = v;
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
        unsigned long long left = leader ? order_key(G) : 0, lowest = 0;
        kept = 0;
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
                for (int i = 0; 32 * i < p.E; i++) {
                    const int e = lane + 32 * i, src = e < p.E ? (e / gs) << sh : 0;
                    const double mg = __shfl_sync(0xffffffffu, m, src);
                    if (e < p.E && ((lanes >> src) & 1u) && !s.exact[e] && key_value(s.key[e]) >= mg) mark |= 1u << i;
                }
                return false;
            }
        }
    }

    unsigned part = 0;                   // which of this lane's experts take part, bit i: lane + 32 i
    for (int i = 0; lane + 32 * i < p.E; i++) part |= ((kept >> ((lane + 32 * i) / gs)) & 1u) << i;
    auto left = [&](int i) { return (part >> i) & 1u ? s.key[lane + 32 * i] : 0ull; };
    unsigned long long my_q = 0;
    my_e = 0;
    for (int j = 0; j < p.k; j++) {
        unsigned long long best = 0;
        int bi = 0;
        for (int i = 0; 32 * i < p.E; i++) {
            const unsigned long long v = left(i);
            if (v > best) { best = v; bi = i; }   // ascending e within the lane: ties keep the lower
        }
        const unsigned long long top = warp_max_key(best);
        const int win = (int)__reduce_min_sync(0xffffffffu, best == top ? unsigned(lane + 32 * bi) : 0xffffffffu);
        if (lane == j) {
            my_e = win;
            my_q = top;
        }
        if ((win & 31) == lane) part &= ~(1u << (win >> 5));
    }

    // Are the ranks safe?  First by plain distances, then by what is known exactly
    const double c = key_value(my_q);
    const double below = __shfl_down_sync(0xffffffffu, c, 1);
    const double last = __shfl_sync(0xffffffffu, c, p.k - 1);
    const unsigned long long near = order_key(last - 2 * eta);
    bool close = lane + 1 < p.k && c - below <= 2 * eta;
    for (int i = 0; 32 * i < p.E; i++) {
        const unsigned long long v = left(i);
        close |= v != 0 && v >= near;
    }
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
    for (int i = 0; 32 * i < p.E; i++) {
        const unsigned long long v = left(i);
        if (v == 0) continue;
        const double ei = s.exact[lane + 32 * i] ? 0.0 : eta, m = ei + last_eta;
        if (m > 0.0 && last - key_value(v) <= m) {
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
__device__ __noinline__ double route_first_values(const RouteScratch s, const RouteChoice& p, double delta, int lane,
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
    for (int e = lane; e < p.E; e += 32) {
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

// The true ranks of a close call, whose wanted logits in s.l are exact: the others are far enough
// from any.  Returns the expert of rank `lane`.  inv: 1 / sum of exp(l - mx) with a bias, else 1;
// where inv itself is only known to a relative eps, two wanted experts whose order hangs on it
// clear `sure`.
__device__ __noinline__ int route_settle(const RouteScratch s, const RouteChoice& p, const RouteClose& close, double mx,
                                         double inv, double eps, int lane, bool& sure) {
    double v = -INFINITY, score = 0.0;
    if (lane < close.n && s.l[close.e] != -INFINITY) {
        score = route_score64(s.l[close.e], p.sigmoid, mx) * inv;
        v = score + (p.bias ? (double)__ldg(p.bias + close.e) : 0.0);
    }
    const unsigned long long key = lane < close.n ? order_key(v) : 0;
    int rank = 0;
    for (int j = 0; j < close.n; j++) {
        const unsigned long long kj = __shfl_sync(0xffffffffu, key, j);
        const int ej = __shfl_sync(0xffffffffu, close.e, j);
        rank += kj > key || (kj == key && ej < close.e);
    }
    __syncwarp();
    unsigned* order = s.key32;           // (done with by now) the lane of each rank
    if (lane < close.n) order[rank] = lane;
    __syncwarp();
    const int here = lane < close.n ? (int)order[lane] : 0, next = lane + 1 < close.n ? (int)order[lane + 1] : 0;
    __syncwarp();
    const double dv = __shfl_sync(0xffffffffu, v, here) - __shfl_sync(0xffffffffu, v, next);
    const double ds = __shfl_sync(0xffffffffu, score, here) - __shfl_sync(0xffffffffu, score, next);
    // (both read before the &: a lane may not skip the second exchange)
    const int want_here = __shfl_sync(0xffffffffu, (int)close.want, here);
    const int want_next = __shfl_sync(0xffffffffu, (int)close.want, next);
    sure = !__any_sync(0xffffffffu, lane < p.k && lane + 1 < close.n && (want_here & want_next) && dv <= fabs(ds) * eps && (dv != 0.0 || ds != 0.0));
    return __shfl_sync(0xffffffffu, close.e, here);
}

// The groups to keep where some were close, from the exact logits of the wanted experts; in
// route_fast's form.  inv: as for route_settle.
__device__ __noinline__ unsigned route_settle_groups(const RouteScratch s, const RouteChoice& p, const RouteClose& close, double mx,
                                                     double inv, int lane) {
    const int gs = p.E / p.n_group, g = close.want ? close.e / gs : -1;
    double v = 0.0;
    if (close.want) {
        v = route_score64(s.l[close.e], p.sigmoid, mx) * inv;
        v += p.bias ? (double)__ldg(p.bias + close.e) : 0.0;
    }
    // each group's best (its lane stands for the group) and second best
    int above = 0;
    bool two = false;
    double second = 0.0;
    for (int j = 0; j < close.n; j++) {
        const double vj = __shfl_sync(0xffffffffu, v, j);
        const int gj = __shfl_sync(0xffffffffu, g, j);
        const bool mine = gj == g && j != lane, over = vj > v || (vj == v && j < lane);
        above += mine && over;
        if (mine && !over) {
            second = two ? fmax(second, vj) : vj;
            two = true;
        }
    }
    const int best = close.want && above == 0;
    const double G = p.group_top == 2 && two ? v + second : v;
    // the best of them take the places that are left; equal ones: the lower
    int better = 0;
    for (int j = 0; j < close.n; j++) {
        const double Gj = __shfl_sync(0xffffffffu, G, j);
        const int gj = __shfl_sync(0xffffffffu, g, j);
        const int bj = __shfl_sync(0xffffffffu, best, j);
        better += bj && (Gj > G || (Gj == G && gj < g));
    }
    const bool keep = best && better < p.topk_group - __popc(close.kept);
    return close.kept | __reduce_or_sync(0xffffffffu, keep ? 1u << (g << route_group_shift(p.n_group)) : 0u);
}

// The fp64 selection value of expert e from s.l[e].
__device__ __forceinline__ void route_make_exact(const RouteScratch& s, const RouteChoice& p, const RouteSoftmax& sm, int e) {
    double v = route_score64(s.l[e], p.sigmoid, sm.mx);
    if (p.bias) v = (p.sigmoid ? v : v * sm.inv) + (double)__ldg(p.bias + e);
    s.key[e] = order_key(v);
    s.exact[e] = 1;
}

// Weights of the chosen experts (my_e: rank `lane`'s).
__device__ __noinline__ void route_weights(const RouteScratch s, const RouteChoice& p, double mx, int lane, int my_e, bool masked,
                                           int32_t* idx_out, float* w_out) {
    double v = lane < p.k && !masked ? route_score64(s.l[my_e], p.sigmoid, mx) : 0.0;
    if (p.renorm) {
        const double den = warp_sum(v);
        v = den == 0.0 ? 0.0 : v / den;
    } else if (!p.sigmoid) {
        const double f = route_softmax_inv(s.l, p.E, mx, lane);
        v = v == 0.0 ? 0.0 : v * f;
    }
    if (lane < p.k) {
        idx_out[lane] = my_e;
        w_out[lane] = (float)(v * (double)p.scale);
    }
}

__device__ __forceinline__ bool route_bias_masks(const RouteChoice& p, int e) {
    return p.bias && __ldg(p.bias + e) == -INFINITY;
}

// The whole choice in fp64 for logits that are exact (s.l complete, __syncwarp done).
__device__ __noinline__ void route_choose_exact(const RouteScratch s, const RouteChoice& p, int lane, int32_t* idx_out,
                                                float* w_out) {
    RouteSoftmax sm;
    const double eta = route_first_values(s, p, 0.0, lane, sm);
    unsigned mark;
    int my_e;
    while (!route_attempt(s, p, eta, lane, mark, my_e)) {
        if (!p.sigmoid && p.bias && !sm.have_inv) {
            sm.inv = route_softmax_inv(s.l, p.E, sm.mx, lane);
            sm.have_inv = true;
        }
        for (; mark; mark &= mark - 1) route_make_exact(s, p, sm, lane + 32 * (__ffs(mark) - 1));
        __syncwarp();
    }
    route_weights(s, p, sm.mx, lane, my_e, route_bias_masks(p, my_e), idx_out, w_out);
}

}  // namespace moe
