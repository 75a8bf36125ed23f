// Grouped router: logits x W_r^T, then the choice of route_select.cuh.
//
// Few tokens (a decode step): the logits are fp64 sums of exact products, on the CUDA
// cores.  Two experts a CTA, four warps each, so that the few hundred rows of W_r are
// read by every SM at once; the last CTA of a token tile (a ticket per tile, reset by
// that CTA) makes the choice, one warp a token.
//
// Many tokens (a prompt): fp64 would take 100 times the tensor cores' time.  A tcgen05
// GEMM gives the logits in fp32 together with |x_t| and |W_e|, from which a bound
// delta = kGemmError |x| |W| on a logit's error follows; the choice then computes a
// logit again in fp64, from x and W_r, only where a decision hangs on less than that
// bound allows (a few tokens in a hundred, a few experts each).  So both ways choose
// the same experts.
#include "tcgen05.cuh"
#include "route_select.cuh"

namespace moe {

int make_tmap_2d(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t rows, uint64_t pitch,
                 uint32_t box_bytes, uint32_t box_rows, bool swizzle128);

constexpr int kChooseWarps = 8;          // tokens per CTA of the choosing kernels
constexpr int kSmallTile = 8;            // largest token tile of the fp64 kernel
constexpr int kSmallT = 16;              // most tokens it takes
constexpr size_t kCounterBytes = 256;    // its tickets, at the start of the workspace

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int r = 0; r < 4; r++) {
        v[2 * r] = __uint_as_float(u[r] << 16);
        v[2 * r + 1] = __uint_as_float(u[r] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// One token's choice by a warp from exact logits l64(e); rounded: they are more than fp32 holds.
template <int VPL, class L64>
__device__ __forceinline__ void choose_row(L64 l64, bool rounded, uint8_t* scratch, const RouteChoice& p, int lane,
                                           int32_t* idx_out, float* w_out) {
    float lf[VPL], mx;
    unsigned big = 0;
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = lane + 32 * i;
        lf[i] = e < p.E ? (float)l64(e) : 0.0f;
        big = max(big, __float_as_uint(lf[i]) & 0x7FFFFFFFu);
    }
    // (an infinite or NaN one makes delta so too, and route_fast gives up)
    const float delta = rounded ? __uint_as_float(__reduce_max_sync(0xffffffffu, big)) * 0x1p-23f : 0.0f;
    int my_e;
    if (route_fast<VPL>(lf, p, delta, lane, scratch, mx, my_e)) {
        route_fast_weights<VPL>(lf, p, mx, lane, my_e, l64, idx_out, w_out);
        return;
    }
    const RouteScratch s(scratch, p.E);
    __syncwarp();
    for (int e = lane; e < p.E; e += 32) s.l[e] = l64(e);
    __syncwarp();
    route_choose_exact<VPL>(s, p, lane, idx_out, w_out);
}

// ---------------------------------------------------------------- few tokens

// Sums v[t] over the warp, halving the tokens a lane holds at each step while it can;
// the lanes of group lane / (32 / TT) end with token lane / (32 / TT)'s sum.
template <int TT>
__device__ __forceinline__ double warp_sum_tokens(double (&v)[TT], int lane) {
    int off = 16;
#pragma unroll
    for (int n = TT / 2; n >= 1; n /= 2, off /= 2) {
        const bool up = lane & off;
#pragma unroll
        for (int j = 0; j < n; j++) {
            const double send = up ? v[j] : v[j + n];
            const double keep = up ? v[j + n] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    for (; off >= 1; off /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    return v[0];
}

template <int TT, int VPL>
__global__ void __launch_bounds__(kChooseWarps * 32)
grouped_small_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int T, int H, RouteChoice p,
                     int32_t* __restrict__ idx, float* __restrict__ wout, double* __restrict__ logits,
                     unsigned int* __restrict__ tile_cnt) {
    extern __shared__ __align__(16) uint8_t sm_raw[];
    __shared__ double part[kChooseWarps][TT];
    __shared__ int s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3;
    const int t0 = blockIdx.y * TT, nt = min(TT, T - t0);
    const int e = blockIdx.x * 2 + (warp >> 2);
    const int nch = H / 8;
    pdl_trigger();
    if (e < p.E)
        for (int c = quarter * 32 + lane; c < nch; c += 128) prefetch_l2(wr + size_t(e) * H + c * 8);
    pdl_wait();
    double acc[TT];
#pragma unroll
    for (int t = 0; t < TT; t++) acc[t] = 0.0;
    if (e < p.E) {
        const uint4* wrow = reinterpret_cast<const uint4*>(wr + size_t(e) * H);
        const uint4* xrow = reinterpret_cast<const uint4*>(x + size_t(t0) * H);
        constexpr int U = TT >= 8 ? 1 : 2;   // chunks whose loads are in flight together
#pragma unroll 1
        for (int c0 = quarter * 32 + lane; c0 < nch; c0 += 128 * U) {
            uint4 wq[U], xq[U][TT];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int c = c0 + 128 * u;
                wq[u] = c < nch ? __ldg(wrow + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < TT; t++)
                    xq[u][t] = c < nch && t < nt ? xrow[size_t(t) * nch + c] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                float wf[8];
                unpack8(wq[u], wf);
                double wd[8];
#pragma unroll
                for (int r = 0; r < 8; r++) wd[r] = wf[r];
#pragma unroll
                for (int t = 0; t < TT; t++) {
                    float xf[8];
                    unpack8(xq[u][t], xf);
#pragma unroll
                    for (int r = 0; r < 8; r++) acc[t] = fma((double)xf[r], wd[r], acc[t]);
                }
            }
        }
    }
    const double v = warp_sum_tokens<TT>(acc, lane);
    if (lane % (32 / TT) == 0) part[warp][lane / (32 / TT)] = v;
    __syncthreads();
    if (threadIdx.x < 2 * TT) {
        const int h = threadIdx.x / TT, t = threadIdx.x % TT, ee = blockIdx.x * 2 + h;
        if (ee < p.E && t < nt)
            logits[size_t(t0 + t) * p.E + ee] =
                (part[4 * h][t] + part[4 * h + 1][t]) + (part[4 * h + 2][t] + part[4 * h + 3][t]);
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(tile_cnt + blockIdx.y, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (threadIdx.x == 0) tile_cnt[blockIdx.y] = 0;
    if (warp >= nt) return;
    const double* row = logits + size_t(t0 + warp) * p.E;
    choose_row<VPL>([&](int e) { return __ldcg(row + e); }, true, sm_raw + warp * RouteScratch::bytes(p.E), p, lane,
                    idx + size_t(t0 + warp) * p.k, wout + size_t(t0 + warp) * p.k);
}

// ---------------------------------------------------------------- many tokens: logits

constexpr int kRgStages = 4;
constexpr int kRgThreads = 512;
constexpr int kRgMaxSplit = 16;
constexpr int kRgMaxN = 256;             // experts per CTA
constexpr int kRgTargetCtas = 148;

// A logit's error over |x_t| |W_e|, per element of a CTA's part of H: every MMA step of 16
// elements may cut the accumulator, whose size |x| |W| bounds, by one unit in its 24th bit,
// and as much again in lining up its products: 2^-23 a step, 2^-27 an element.  Measured: 2^-29
// where all products are positive, 2^-33 for normal ones.
constexpr double kGemmError = 0x1p-27;

struct RouteGemmArgs {
    int T, H, E, Ep;          // Ep: row length of the partial logits
    int n_tiles, N, split, Kc;
    float* part;              // [split][T][Ep]
    float* xn;                // [split][T] sums of squares of x
    float* wn;                // [E] sums of squares of W_r
    const uint16_t* wr;
    unsigned long long limit_ns;
};

// One CTA: 128 tokens x N experts over Kc of H.  Warp 0 loads (TMA, 128-byte swizzle),
// warp 1 issues the MMAs, warps 8-15 sum the squares of a share of W_r, warps 4-7 those of
// the x rows as they pass through shared memory, then drain the accumulator.  Waits are
// bounded; where one gives up, the bound on the errors becomes NaN.
__global__ void __launch_bounds__(kRgThreads, 1)
route_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                  const RouteGemmArgs g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kRgStages], empty[kRgStages], accf;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_bad;                // a wait gave up
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b_bytes = g.N * 128, stage = 16384 + b_bytes;
    const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
    const int nt = tile % g.n_tiles, mt = tile / g.n_tiles;
    const int k0 = rank * g.Kc, KT = (min(g.H - k0, g.Kc) + 63) / 64;
    const uint32_t cols = g.N <= 32 ? 32 : g.N <= 64 ? 64 : g.N <= 128 ? 128 : 256;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRgStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1 + 4);
        }
        mbar_init(&accf, 1);
        s_bad = 0;
        fence_mbar_init();
        prefetch_tmap(&map_x);
        prefetch_tmap(&map_w);
    }
    if (warp == 1) tmem_alloc(&tmem_slot, cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t acc = tmem_slot;
    pdl_trigger();
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, ph = 0;
            for (int kt = 0; kt < KT; kt++) {
                if (!mbar_wait(&empty[s], ph ^ 1, g.limit_ns)) s_bad = 1;
                mbar_arrive_expect_tx(&full[s], stage);
                tma_load_2d(sm + s * stage, &map_x, (k0 + kt * 64) * 2, mt * 128, &full[s]);
                tma_load_2d(sm + s * stage + 16384, &map_w, (k0 + kt * 64) * 2, nt * kRgMaxN, &full[s]);
                if (++s == kRgStages) { s = 0; ph ^= 1; }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // D fp32, A and B bf16, K-major, M = 128
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(g.N >> 3) << 17) | (8u << 24);
            int s = 0, ph = 0;
            for (int kt = 0; kt < KT; kt++) {
                if (!mbar_wait(&full[s], ph, g.limit_ns)) s_bad = 1;
                tc_fence_after();
                const uint64_t ad = smem_desc(sm + s * stage, 16, 1024, 2), bd = smem_desc(sm + s * stage + 16384, 16, 1024, 2);
#pragma unroll
                for (int i = 0; i < 4; i++)   // K = 16 elements = 32 bytes per MMA
                    mma_bf16(acc, ad + 2 * i, bd + 2 * i, idesc, (kt > 0 || i > 0) ? 1u : 0u);
                tc_commit(&empty[s]);
                if (++s == kRgStages) { s = 0; ph ^= 1; }
            }
            tc_commit(&accf);
        }
        __syncwarp();
    } else if (warp >= 8) {
        for (int e = blockIdx.x * 8 + warp - 8; e < g.E; e += gridDim.x * 8) {
            const uint4* row = reinterpret_cast<const uint4*>(g.wr + size_t(e) * g.H);
            float sum = 0.0f;
#pragma unroll 8
            for (int c = lane; c < g.H / 8; c += 32) {
                float v[8];
                unpack8(__ldg(row + c), v);
#pragma unroll
                for (int r = 0; r < 8; r++) sum = fmaf(v[r], v[r], sum);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) g.wn[e] = sum;
        }
    } else if (warp >= 4) {
        const int r = threadIdx.x - 128, t = mt * 128 + r;
        float sum = 0.0f;
        int s = 0, ph = 0;
        for (int kt = 0; kt < KT; kt++) {
            if (!mbar_wait(&full[s], ph, g.limit_ns)) s_bad = 1;
            const uint4* row = reinterpret_cast<const uint4*>(sm + s * stage + r * 128);
            if (nt == 0) {
#pragma unroll
                for (int c = 0; c < 8; c++) {
                    float v[8];
                    unpack8(row[(c + r) & 7], v);   // a quarter warp's rows in different banks
#pragma unroll
                    for (int i = 0; i < 8; i++) sum = fmaf(v[i], v[i], sum);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == kRgStages) { s = 0; ph ^= 1; }
        }
        if (!mbar_wait(&accf, 0, g.limit_ns)) s_bad = 1;
        __syncwarp();
        // (a bound of NaN has the choice compute the token's logits in fp64)
        if (t < g.T && (nt == 0 || s_bad)) g.xn[(size_t)rank * g.T + t] = s_bad ? __uint_as_float(0x7FC00000u) : sum;
        tc_fence_after();
        float* dst = g.part + ((size_t)rank * g.T + t) * g.Ep + nt * kRgMaxN;
        const int width = min(g.N, g.Ep - nt * kRgMaxN);
        for (int c = 0; c < width; c += 32) {
            uint32_t v[32];
            tmem_ld_32x32(acc + ((uint32_t)(32 * (warp - 4)) << 16) + c, v);
            if (t < g.T) {
#pragma unroll
                for (int i = 0; i < 32; i += 8)   // whole 32-byte sectors
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c + i), "r"(v[i]),
                                 "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]),
                                 "r"(v[i + 7]) : "memory");
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(acc, cols);
    }
}

// ---------------------------------------------------------------- many tokens: choice

// fp64 dot products of one x row with rows e[0 .. NE) of W_r by a warp.
template <int NE>
__device__ __forceinline__ void exact_logits(const uint16_t* x, const uint16_t* wr, int H, const int (&e)[NE], int lane,
                                             double (&out)[NE]) {
    double acc[NE];
#pragma unroll
    for (int a = 0; a < NE; a++) acc[a] = 0.0;
    constexpr int U = 4;                 // chunks in flight
#pragma unroll 1
    for (int c0 = lane; c0 < H / 8; c0 += 32 * U) {
        uint4 xq[U], wq[U][NE];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = c0 + 32 * u;
            const bool in = c < H / 8;
            xq[u] = in ? __ldg(reinterpret_cast<const uint4*>(x) + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int a = 0; a < NE; a++)
                wq[u][a] = in ? __ldg(reinterpret_cast<const uint4*>(wr + size_t(e[a]) * H) + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            float xf[8];
            unpack8(xq[u], xf);
            double xd[8];
#pragma unroll
            for (int r = 0; r < 8; r++) xd[r] = xf[r];
#pragma unroll
            for (int a = 0; a < NE; a++) {
                float wf[8];
                unpack8(wq[u][a], wf);
#pragma unroll
                for (int r = 0; r < 8; r++) acc[a] = fma(xd[r], (double)wf[r], acc[a]);
            }
        }
    }
#pragma unroll
    for (int a = 0; a < NE; a++) out[a] = warp_sum(acc[a]);
}

// One warp per token.  Logits that have to be known exactly are computed by all warps of
// the CTA together, whichever token they belong to.
template <int VPL>
__global__ void __launch_bounds__(kChooseWarps * 32)
route_gemm_choose_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, RouteGemmArgs g, RouteChoice p,
                         int32_t* __restrict__ idx, float* __restrict__ wout) {
    extern __shared__ __align__(16) uint8_t sm_raw[];
    __shared__ unsigned s_mark[kChooseWarps][32];   // bit i of word j: expert j + 32 i is wanted
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x * kChooseWarps + warp;
    const RouteScratch s(sm_raw + warp * RouteScratch::bytes(p.E), p.E);
    pdl_trigger();
    pdl_wait();
    unsigned mark = 0;
    bool open = false, all = false;      // not chosen yet; every logit is wanted
    RouteSoftmax sm;
    double eta = 0.0;
    if (t < g.T) {
        float lf[VPL], mx, wmax = 0.0f, xn = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; i++) lf[i] = 0.0f;
        for (int c = 0; c < g.split; c++) {
            const float* row = g.part + ((size_t)c * g.T + t) * g.Ep + lane;
            xn += __ldg(g.xn + (size_t)c * g.T + t);
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (lane + 32 * i < p.E) lf[i] += __ldg(row + 32 * i);
        }
        for (int e = lane; e < p.E; e += 32) {
            const float w2 = __ldg(g.wn + e);
            wmax = !(w2 <= wmax) ? w2 : wmax;   // a NaN stays
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, wmax, off);
            wmax = !(o <= wmax) ? o : wmax;
        }
        // (the parts' sum in fp32 adds one rounding each)
        const float delta = (float)(kGemmError * (g.Kc + 8 * g.split) * 1.001 * sqrt((double)xn * (double)wmax));
        int my_e;
        open = true;
        if (!(delta <= 0.05f)) {
            all = true;
        } else if (route_fast<VPL>(lf, p, delta, lane, s.l, mx, my_e)) {
            const float* sl = reinterpret_cast<const float*>(s.l);
            route_fast_weights<VPL>(lf, p, mx, lane, my_e, [&](int e) { return (double)sl[e]; }, idx + size_t(t) * p.k,
                                    wout + size_t(t) * p.k);
            open = false;
        } else if (!p.sigmoid && p.bias) {
            all = true;                  // the denominator hangs on every logit
        } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (lane + 32 * i < p.E) s.l[lane + 32 * i] = lf[i];
            __syncwarp();
            eta = route_first_values<VPL>(s, p, delta, lane, sm);
            if (route_attempt<VPL>(s, p, eta, lane, mark, my_e)) {
                route_weights(p, sm.mx, lane, my_e, s.l[my_e], [&]() { return route_softmax_inv(s.l, p.E, sm.mx, lane); },
                              idx + size_t(t) * p.k, wout + size_t(t) * p.k);
                open = false;
                mark = 0;
            }
        }
        if (all)
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (lane + 32 * i < p.E) mark |= 1u << i;
    }
    while (__syncthreads_or(open)) {
        s_mark[warp][lane] = open ? mark : 0;
        __syncthreads();
        int seen = 0;                    // wanted logits so far: the CTA's warps take them in turn, two at a time
        for (int h = 0; h < kChooseWarps; h++) {
            const unsigned word = s_mark[h][lane];
            int before = __popc(word);   // inclusive prefix sum over the lanes
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off) before += o;
            }
            const int n = __shfl_sync(0xffffffffu, before, 31);
            before -= __popc(word);
            const int th = blockIdx.x * kChooseWarps + h;
            const RouteScratch sh(sm_raw + h * RouteScratch::bytes(p.E), p.E);
            for (int j = 0; j < n; j += 2) {
                if (((seen + j) / 2) % kChooseWarps != warp) continue;
                int e[2];
#pragma unroll
                for (int a = 0; a < 2; a++) {
                    const int m = min(j + a, n - 1);
                    const int src = 31 - __clz(__ballot_sync(0xffffffffu, before <= m && word != 0));
                    unsigned w = __shfl_sync(0xffffffffu, word, src);
                    for (int skip = m - __shfl_sync(0xffffffffu, before, src); skip > 0; skip--) w &= w - 1;
                    e[a] = src + 32 * (__ffs(w) - 1);
                }
                double v[2];
                exact_logits<2>(x + size_t(th) * g.H, wr, g.H, e, lane, v);
                if (lane == 0) {
                    sh.l[e[0]] = v[0];
                    sh.l[e[1]] = v[1];
                }
            }
            seen += (n + 1) / 2 * 2;
        }
        __syncthreads();
        if (open && all) {
            route_choose_exact<VPL>(s, p, lane, idx + size_t(t) * p.k, wout + size_t(t) * p.k);
            open = false;
        } else if (open) {
            for (; mark; mark &= mark - 1) route_make_exact(s, p, sm, lane + 32 * (__ffs(mark) - 1));
            __syncwarp();
            int my_e;
            if (route_attempt<VPL>(s, p, eta, lane, mark, my_e)) {
                route_weights(p, sm.mx, lane, my_e, s.l[my_e], [&]() { return route_softmax_inv(s.l, p.E, sm.mx, lane); },
                              idx + size_t(t) * p.k, wout + size_t(t) * p.k);
                open = false;
            }
        }
    }
}

// ---------------------------------------------------------------- given logits

// One warp per token; logits fp32 or bf16 with row stride ld.
template <int VPL>
__global__ void __launch_bounds__(kChooseWarps * 32)
route_select_kernel(const void* __restrict__ logits, int is_bf16, long long ld, int T, RouteChoice p,
                    int32_t* __restrict__ idx, float* __restrict__ wout) {
    extern __shared__ __align__(16) uint8_t sm_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x * kChooseWarps + warp;
    if (t >= T) return;
    const uint16_t* lh = reinterpret_cast<const uint16_t*>(logits) + t * ld;
    const float* lf = reinterpret_cast<const float*>(logits) + t * ld;
    choose_row<VPL>([&](int e) { return (double)(is_bf16 ? __uint_as_float((uint32_t)lh[e] << 16) : lf[e]); }, false,
                    sm_raw + warp * RouteScratch::bytes(p.E), p, lane, idx + size_t(t) * p.k, wout + size_t(t) * p.k);
}

// ---------------------------------------------------------------- host

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// How many parts of H the CTAs of one tile take: as many as the SMs have room for.
static int route_split(int T, int E) {
    const int tiles = ((T + 127) / 128) * ((E + kRgMaxN - 1) / kRgMaxN);
    return std::max(1, std::min(kRgMaxSplit, kRgTargetCtas / tiles));
}

static int check_choice(const moe_route_choice* c, const float* bias, int T, int E, RouteChoice& p) {
    if (!c) return fail(MOE_EINVAL, "null routing choice");
    if (T <= 0 || E <= 0 || E > kMaxE || c->k <= 0 || c->k > kMaxK)
        return fail(MOE_EINVAL, "grouped route: need T > 0, 0 < E <= 1024, 0 < k <= 32");
    if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
        return fail(MOE_EINVAL, "grouped route: unknown score");
    if (c->n_group <= 0 || c->n_group > kMaxGroups || E % c->n_group)
        return fail(MOE_EINVAL, "grouped route: n_group must divide E and be at most 32");
    if (c->topk_group <= 0 || c->topk_group > c->n_group || c->k > c->topk_group * (E / c->n_group))
        return fail(MOE_EINVAL, "grouped route: need 0 < topk_group <= n_group and k experts in the kept groups");
    if ((c->group_top != 1 && c->group_top != 2) || (c->renormalize != 0 && c->renormalize != 1))
        return fail(MOE_EINVAL, "grouped route: group_top must be 1 or 2, renormalize 0 or 1");
    if (!(c->scale > 0.0f) || c->scale > 3.0e38f) return fail(MOE_EINVAL, "grouped route: scale must be positive and finite");
    p = RouteChoice{E, c->k, c->score == MOE_SCORE_SIGMOID, c->n_group, c->topk_group, c->group_top, c->renormalize,
                    c->scale, bias};
    return MOE_OK;
}

// Raise a kernel's shared-memory limit, once per device.
template <typename Kern>
static cudaError_t raise_smem(Kern kern, int bytes, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

struct RouteCall {
    const uint16_t *x, *wr;
    int T, H;
    RouteChoice p;
    int32_t* idx;
    float* w;
    char* ws;
    cudaStream_t s;
};

template <int TT, int VPL>
static cudaError_t launch_small(const RouteCall& r) {
    auto kern = grouped_small_kernel<TT, VPL>;
    static bool done[64] = {};
    cudaError_t e = raise_smem(kern, (int)(kSmallTile * RouteScratch::bytes(kMaxE)), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((r.p.E + 1) / 2, (r.T + TT - 1) / TT), dim3(kChooseWarps * 32),
                      TT * RouteScratch::bytes(r.p.E), r.s, r.x, r.wr, r.T, r.H, r.p, r.idx, r.w,
                      (double*)(r.ws + kCounterBytes), (unsigned int*)r.ws);
}

template <int VPL>
static int launch_large(const RouteCall& r) {
    const int E = r.p.E;
    RouteGemmArgs g{};
    g.T = r.T; g.H = r.H; g.E = E;
    g.Ep = (E + 31) / 32 * 32;
    g.n_tiles = (E + kRgMaxN - 1) / kRgMaxN;
    g.N = std::min(kRgMaxN, (E + 15) / 16 * 16);
    // at least 256 of H a CTA
    const int want = std::min(route_split(r.T, E), std::max(1, r.H / 256));
    g.Kc = ((r.H + want - 1) / want + 63) / 64 * 64;
    g.split = (r.H + g.Kc - 1) / g.Kc;
    char* at = r.ws + kCounterBytes;
    g.part = (float*)at;
    at += up256(size_t(g.split) * r.T * g.Ep * 4);
    g.xn = (float*)at;
    at += up256(size_t(g.split) * r.T * 4);
    g.wn = (float*)at;
    g.wr = r.wr;
    g.limit_ns = 2000000000ull;
    CUtensorMap mx, mw;
    int rc;
    if ((rc = make_tmap_2d(&mx, r.x, size_t(r.H) * 2, r.T, size_t(r.H) * 2, 128, 128, true))) return rc;
    if ((rc = make_tmap_2d(&mw, r.wr, size_t(r.H) * 2, E, size_t(r.H) * 2, 128, g.N, true))) return rc;
    static bool gdone[64] = {}, cdone[64] = {};
    const int smem = kRgStages * (16384 + g.N * 128) + 1024;
    MOE_CUDA_TRY(raise_smem(route_gemm_kernel, kRgStages * (16384 + kRgMaxN * 128) + 1024, gdone));
    const dim3 grid(((r.T + 127) / 128) * g.n_tiles * g.split);
    MOE_CUDA_TRY(launch_pdl(route_gemm_kernel, grid, dim3(kRgThreads), smem, r.s, mx, mw, g));
    auto kern = route_gemm_choose_kernel<VPL>;
    MOE_CUDA_TRY(raise_smem(kern, (int)(kChooseWarps * RouteScratch::bytes(kMaxE)), cdone));
    MOE_CUDA_TRY(launch_pdl(kern, dim3((r.T + kChooseWarps - 1) / kChooseWarps), dim3(kChooseWarps * 32),
                            kChooseWarps * RouteScratch::bytes(E), r.s, r.x, r.wr, g, r.p, r.idx, r.w));
    return MOE_OK;
}

template <int VPL>
static int launch_grouped(const RouteCall& r) {
    if (r.T > kSmallT) return launch_large<VPL>(r);
    const cudaError_t e = r.T == 1 ? launch_small<1, VPL>(r) : r.T == 2 ? launch_small<2, VPL>(r)
                          : r.T <= 4 ? launch_small<4, VPL>(r) : launch_small<8, VPL>(r);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "grouped router launch");
}

template <int VPL>
static int launch_select(const void* logits, int bf16, long long ld, int T, const RouteChoice& p, int32_t* idx, float* w,
                         cudaStream_t s) {
    auto kern = route_select_kernel<VPL>;
    static bool done[64] = {};
    MOE_CUDA_TRY(raise_smem(kern, (int)(kChooseWarps * RouteScratch::bytes(kMaxE)), done));
    MOE_CUDA_TRY(launch_pdl(kern, dim3((T + kChooseWarps - 1) / kChooseWarps), dim3(kChooseWarps * 32),
                            kChooseWarps * RouteScratch::bytes(p.E), s, logits, bf16, ld, T, p, idx, w));
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_grouped_workspace_bytes(int T, int E) {
    if (T <= 0 || E <= 0 || E > kMaxE) return 0;
    if (T <= kSmallT) return kCounterBytes + up256(size_t(T) * E * sizeof(double));
    const size_t split = route_split(T, E), Ep = (E + 31) / 32 * 32;
    return kCounterBytes + up256(split * T * Ep * 4) + up256(split * T * 4) + up256(size_t(E) * 4);
}

extern "C" int moe_route_grouped(const void* x_bf16, const void* wr_bf16, const float* bias, int T, int H, int E,
                                 const moe_route_choice* choice, int32_t* idx, float* w, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    RouteChoice p;
    const int rc = check_choice(choice, bias, T, E, p);
    if (rc) return rc;
    if (!x_bf16 || !wr_bf16 || !idx || !w) return fail(MOE_EINVAL, "null pointer");
    if (H <= 0 || H % 8) return fail(MOE_EINVAL, "grouped route: H must be a positive multiple of 8");
    if ((reinterpret_cast<uintptr_t>(x_bf16) | reinterpret_cast<uintptr_t>(wr_bf16)) & 15)
        return fail(MOE_EINVAL, "grouped route: x and W_r must be 16-byte aligned");
    if (!workspace || workspace_bytes < moe_route_grouped_workspace_bytes(T, E))
        return fail(MOE_EINVAL, "grouped route: workspace missing or smaller than moe_route_grouped_workspace_bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_EINVAL, "grouped route: workspace must be 256-byte aligned");
    const RouteCall r{(const uint16_t*)x_bf16, (const uint16_t*)wr_bf16, T, H, p, idx, w, (char*)workspace, (cudaStream_t)stream};
    // registers per lane that hold the E selection values
    return E <= 128 ? launch_grouped<4>(r) : E <= 256 ? launch_grouped<8>(r) : launch_grouped<32>(r);
}

extern "C" int moe_route_select(const void* logits, int type, long long ld, const float* bias, int T, int E,
                                const moe_route_choice* choice, int32_t* idx, float* w, void* stream) {
    RouteChoice p;
    const int rc = check_choice(choice, bias, T, E, p);
    if (rc) return rc;
    if (!logits || !idx || !w) return fail(MOE_EINVAL, "null pointer");
    if (type != MOE_BF16 && type != MOE_F32) return fail(MOE_EINVAL, "route select: logits must be bf16 or fp32");
    if (ld < E && T > 1) return fail(MOE_EINVAL, "route select: row stride smaller than E");
    if (reinterpret_cast<uintptr_t>(logits) & (type == MOE_BF16 ? 1 : 3))
        return fail(MOE_EINVAL, "route select: logits not aligned to their type");
    const int bf16 = type == MOE_BF16;
    cudaStream_t s = (cudaStream_t)stream;
    return E <= 128 ? launch_select<4>(logits, bf16, ld, T, p, idx, w, s)
         : E <= 256 ? launch_select<8>(logits, bf16, ld, T, p, idx, w, s)
                    : launch_select<32>(logits, bf16, ld, T, p, idx, w, s);
}
