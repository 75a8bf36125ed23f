// Grouped router: logits x W_r^T, then the choice of route_select.cuh.
//
// Few tokens (a decode step): the logits are fp64 sums of exact products, on the CUDA
// cores.  Two experts a CTA, its eight warps over parts of H, so that the few hundred rows
// of W_r are read by every SM at once; the last CTA of a token tile (a ticket per tile,
// reset by that CTA) makes the choice, one warp a token.  Latency: for one token of 4096 x 256,
// 9.0 us (launch and products 2.7, the rest the choice), which is 2.1 MB at 0.23 TB/s.
//
// Many tokens (a prompt): fp64 would take 100 times the tensor cores' time.  A tcgen05
// GEMM gives the logits in fp32 together with |x_t| and |W_e|, from which a bound on
// a logit's error follows; the choice then computes a logit again in fp64, from x and
// W_r, only where a decision hangs on less than that bound allows (a few tokens in a
// hundred, a few experts each).  So both ways choose the same experts.  8192 tokens of
// 4096 x 256 take 71.5 us: the GEMM 23 (17 GFLOP, 0.75 PFLOP/s; its accumulators are read
// out every 128 of H), the choice the rest (some 2500 instructions a token).  The GEMM's fixed
// cost makes it the slower way up to 32 tokens, whose weights are promised to come from exact
// logits: 24 tokens of 4096 x 256 take 16.0 us in fp64 and 20.6 with it, 32 of 2048 x 128 9.8 and
// 15.0, 32 of 7168 x 256 22.3 and 25.1; 40 tokens 19.2 and 22.1, 11.3 and 15.4, 25.4 and 25.8; 64 of
// 4096 x 256 25.2 and 22.5.
#include "tcgen05.cuh"
#include "route_select.cuh"

#include <atomic>

namespace moe {

int make_tmap_2d(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t rows, uint64_t pitch,
                 uint32_t box_bytes, uint32_t box_rows, bool swizzle128);

constexpr int kChooseWarps = 8;          // warps per CTA of the kernels for few tokens and given logits
constexpr int kGemmTokens = 4;           // tokens, a warp each, per CTA of the choice after the GEMM
constexpr int kSmallTile = 8;            // largest token tile of the fp64 kernel
constexpr int kSmallT = 32;              // most tokens it takes
constexpr size_t kCounterBytes = 256;    // its tickets, at the start of the workspace
constexpr int kMaxRouteSize = 1 << 30;   // largest T and H: twice that, and their rounding up, stay ints

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
template <class L64>
__device__ __forceinline__ void choose_row(L64 l64, bool rounded, uint8_t* scratch, const RouteChoice& p, int lane,
                                           int32_t* idx_out, float* w_out) {
    const RouteScratch s(scratch, p.E);
    unsigned big = 0;
#pragma unroll 4
    for (int e = lane; e < p.E; e += 32) {
        const double l = l64(e);
        s.fill(e, l, (float)l, p.bias ? __ldg(p.bias + e) : 0.0f);
        big = max(big, __float_as_uint((float)l) & 0x7FFFFFFFu);
    }
    __syncwarp();
    // (an infinite or NaN one makes delta so too, and route_fast gives up)
    const float delta = rounded ? __uint_as_float(__reduce_max_sync(0xffffffffu, big)) * 0x1p-23f : 0.0f;
    int my_e;
    float mx;
    bool masked;
    RouteClose close;
    RouteStatus st;
    unsigned groups = 0;
    double inv = 1.0;
    for (int i = 0;; i++) {
        st = route_fast(s, p, delta, lane, groups, mx, my_e, masked, close);
        __syncwarp();
        if (st == kRouteCertain) break;
        if (st == kRouteOpen || i == 2) {
            route_choose_exact(s, p, lane, idx_out, w_out);
            return;
        }
        if (!p.sigmoid && p.bias) inv = route_softmax_inv(s.l, p.E, mx, lane);
        if (st == kRouteClose) break;
        groups = route_settle_groups(s, p, close, mx, inv, lane);
        close = RouteClose();
    }
    if (st == kRouteClose) {
        bool sure;
        my_e = route_settle(s, p, close, mx, inv, 0.0, lane, sure);
        masked = route_bias_masks(p, my_e);
    }
    route_weights(s, p, mx, lane, my_e, masked, idx_out, w_out);
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

// (Two CTAs an SM cover every grid of up to 32 tokens of 256 experts in two rounds, and leave the larger tiles
// the registers they need: without that they spill, and 16 tokens of 4096 x 256 take 15.6 us, not 12.5)
template <int TT>
__global__ void __launch_bounds__(kChooseWarps * 32, TT >= 4 ? 2 : 0)
grouped_small_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int T, int H, RouteChoice p,
                     int32_t* __restrict__ idx, float* __restrict__ wout, double* __restrict__ logits,
                     unsigned int* __restrict__ tile_cnt) {
    extern __shared__ __align__(16) uint8_t sm_raw[];
    __shared__ double part[kChooseWarps][2 * TT];
    __shared__ int s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.y * TT, nt = min(TT, T - t0);
    const int e0 = blockIdx.x * 2, e1 = min(e0 + 1, p.E - 1);
    const int nch = H / 8;
    for (int c = threadIdx.x; c < nch; c += kChooseWarps * 32) {
        prefetch_l2(wr + size_t(e0) * H + c * 8);
        prefetch_l2(wr + size_t(e1) * H + c * 8);
    }
    pdl_wait();
    pdl_trigger();   // (after the wait: a kernel that this lets start may read what earlier ones wrote)
    double acc[2 * TT];
#pragma unroll
    for (int t = 0; t < 2 * TT; t++) acc[t] = 0.0;
    const uint4* w0 = reinterpret_cast<const uint4*>(wr + size_t(e0) * H);
    const uint4* w1 = reinterpret_cast<const uint4*>(wr + size_t(e1) * H);
    const uint4* xrow = reinterpret_cast<const uint4*>(x + size_t(t0) * H);
    constexpr int U = TT >= 8 ? 1 : 2;   // chunks whose loads are in flight together
#pragma unroll 1
    for (int c0 = threadIdx.x; c0 < nch; c0 += kChooseWarps * 32 * U) {
        uint4 wq[U][2], xq[U][TT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int c = c0 + kChooseWarps * 32 * u;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            wq[u][0] = c < nch ? __ldg(w0 + c) : zero;
            wq[u][1] = c < nch ? __ldg(w1 + c) : zero;
#pragma unroll
            for (int t = 0; t < TT; t++) xq[u][t] = c < nch && t < nt ? xrow[size_t(t) * nch + c] : zero;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            double wd[2][8];
#pragma unroll
            for (int a = 0; a < 2; a++) {
                float wf[8];
                unpack8(wq[u][a], wf);
#pragma unroll
                for (int r = 0; r < 8; r++) wd[a][r] = wf[r];
            }
#pragma unroll
            for (int t = 0; t < TT; t++) {
                float xf[8];
                unpack8(xq[u][t], xf);
#pragma unroll
                for (int r = 0; r < 8; r++) {
                    const double xd = xf[r];
                    acc[t] = fma(xd, wd[0][r], acc[t]);
                    acc[TT + t] = fma(xd, wd[1][r], acc[TT + t]);
                }
            }
        }
    }
    const double v = warp_sum_tokens<2 * TT>(acc, lane);
    if (lane % (16 / TT) == 0) part[warp][lane / (16 / TT)] = v;
    __syncthreads();
    if (threadIdx.x < 2 * TT) {
        const int h = threadIdx.x / TT, t = threadIdx.x % TT, ee = e0 + h;
        double sum = 0.0;
        for (int w = 0; w < kChooseWarps; w++) sum += part[w][threadIdx.x];
        if (ee < p.E && t < nt) logits[size_t(t0 + t) * p.E + ee] = sum;
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
    choose_row([&](int e) { return __ldcg(row + e); }, true, sm_raw + warp * RouteScratch::bytes(p.E), p, lane,
                    idx + size_t(t0 + warp) * p.k, wout + size_t(t0 + warp) * p.k);
}

// ---------------------------------------------------------------- many tokens: logits

constexpr int kRgStages = 4;
constexpr int kRgThreads = 384;
constexpr int kRgMaxSplit = 16;
constexpr int kRgMaxN = 256;             // experts per CTA
constexpr int kRgTargetCtas = 148;
constexpr int kRgChunk = 2;              // stages (64 elements each) the tensor core sums by itself

// Error of the tensor core's sums.  What an MMA step does here, seen by sums of powers of two at every
// place: it cuts its 16 products and the accumulator towards zero at the 25th binary place below the
// largest exponent among them, adds them, and cuts the sum to 24 bits.  The largest term loses nothing,
// so step s loses less than 16 2^-25 M_s, M_s its largest product or the accumulator before it, and
// 2^-23 of its sum.  Let q_s be the sum of the sizes of its products, S that of all n steps of a chunk
// (at most the chunk's |x| |W|), V the size of the chunk's sum, as it is read out, and h = (S + V) / 2.
// The accumulator before step s is at most q_1 + .. + q_(s-1), and at most V + q_s + .. + q_n: at most h.
// So all M_s are at most h, but for one whose q_s is above h, and then the others are at most 2 h - q_s:
// their sum is at most n h.  Altogether 2^-25 times 16 n h + 4 (n - 1) h + 4 V, and the chunks' S add up
// to |x| |W| at most.  (One product of 1 before 127 of just under 2^-24 loses 2^-18 of |x| |W|, a
// fifth less than this allows; dense rows 2^-21.9 where all products are positive, 2^-23.6 of random
// sign.)  The chunks are added in fp32 registers: 2^-24 of at most the sum of all V each.
constexpr int kChunkSteps = 4 * kRgChunk;
constexpr double kErrorS = (8 * kChunkSteps + 2 * (kChunkSteps - 1)) * 0x1p-25;
constexpr double kErrorV = kErrorS + 4 * 0x1p-25;

struct RouteGemmArgs {
    int T, H, E, Ep;          // Ep: row length of the partial logits
    int n_tiles, N, split, Kc;
    float* part;              // [split][T][Ep]
    float* xn;                // [split][T] sums of squares of x
    float* xm;                // [split][n_tiles][T] sum over the chunks of a row's largest chunk sum
    float* wn;                // [E] sums of squares of W_r
    const uint16_t* wr;
    unsigned long long limit_ns;
};

// 32 lanes x 16 consecutive fp32 columns; complete after tcgen05.wait::ld.
__device__ __forceinline__ void tmem_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15},"
        " [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void add_f32x2(float& a0, float& a1, float b0, float b1) {
    asm("{ .reg .b64 a, b; mov.b64 a, {%0, %1}; mov.b64 b, {%2, %3}; add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
        : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}

// `bytes` (a multiple of 16) of this CTA's shared memory to global memory, asynchronously.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}

// A row's sum of squares, with what its squares may have lost below the normal range (2^-126 each;
// they are bf16 or fp32) where that is not small beside the sum.  A row of zeros keeps its 0, which
// says that its logits are exact: so the row is looked at, by the whole warp.
__device__ __forceinline__ float with_lost_squares(float sum, const uint4* row, int H, int lane) {
    const float lost = H * 0x1p-126f;
    if (!(sum < lost * 0x1p16f)) return sum;
    uint32_t any = 0;
    for (int c = lane; c < H / 8; c += 32) {
        const uint4 q = __ldg(row + c);
        any |= q.x | q.y | q.z | q.w;
    }
    return __any_sync(0xffffffffu, (any & 0x7FFF7FFFu) != 0) ? sum + lost : sum;
}

// One CTA: 128 tokens x N experts over Kc of H.  Warp 0 loads (TMA, 128-byte swizzle), warp 1
// issues the MMAs into two accumulators in turn, a chunk of K each; warps 4-11 add the chunks up
// in registers (a row and 128 experts a thread), after the sums of squares of a share of W_r;
// warps 2-3 sum the squares of the x rows as they pass through shared memory (two rows a
// thread), apart from the others because a stage is free only when they have read it.  Waits
// are bounded; where one gives up, the bound on the errors becomes NaN.
__global__ void __launch_bounds__(kRgThreads, 1)
route_gemm_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                  const RouteGemmArgs g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kRgStages], empty[kRgStages], accf[2], acce[2];
    __shared__ uint32_t tmem_slot;
    __shared__ unsigned s_max[128];      // the rows' xm (float bits)
    __shared__ float s_sq[128];          // sums of squares of the rows
    __shared__ int s_bad;                // a wait gave up
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b_bytes = g.N * 128, stage = 16384 + b_bytes;
    const int rank = blockIdx.x % g.split, tile = blockIdx.x / g.split;
    const int nt = tile % g.n_tiles, mt = tile / g.n_tiles;
    const int k0 = rank * g.Kc, KT = (min(g.H - k0, g.Kc) + 63) / 64, chunks = (KT + kRgChunk - 1) / kRgChunk;
    const uint32_t cols = g.N <= 16 ? 32 : g.N <= 32 ? 64 : g.N <= 64 ? 128 : g.N <= 128 ? 256 : 512;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRgStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1 + 2);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&accf[i], 1);
            mbar_init(&acce[i], 8);
        }
        s_bad = 0;
        fence_mbar_init();
        prefetch_tmap(&map_x);
        prefetch_tmap(&map_w);
    }
    if (threadIdx.x < 128) s_max[threadIdx.x] = 0;
    if (warp == 1) tmem_alloc(&tmem_slot, cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_slot;
    pdl_wait();
    pdl_trigger();

    // sums of squares of W_r: experts dealt out to the warps w of n a CTA
    auto w_norms = [&](int w, int n) {
        for (int e = blockIdx.x * n + w; e < g.E; e += gridDim.x * n) {
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
            sum = with_lost_squares(sum, row, g.H, lane);
            if (lane == 0) g.wn[e] = sum;
        }
    };

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
            for (int j = 0; j < chunks; j++) {
                if (!mbar_wait(&acce[j & 1], ((j >> 1) & 1) ^ 1, g.limit_ns)) s_bad = 1;
                const uint32_t acc = tbase + (j & 1) * g.N;
                for (int kt = j * kRgChunk; kt < min(KT, (j + 1) * kRgChunk); kt++) {
                    if (!mbar_wait(&full[s], ph, g.limit_ns)) s_bad = 1;
                    tc_fence_after();
                    const uint64_t ad = smem_desc(sm + s * stage, 16, 1024, 2), bd = smem_desc(sm + s * stage + 16384, 16, 1024, 2);
#pragma unroll
                    for (int i = 0; i < 4; i++)   // K = 16 elements = 32 bytes per MMA
                        mma_bf16(acc, ad + 2 * i, bd + 2 * i, idesc, (kt > j * kRgChunk || i > 0) ? 1u : 0u);
                    tc_commit(&empty[s]);
                    if (++s == kRgStages) { s = 0; ph ^= 1; }
                }
                tc_commit(&accf[j & 1]);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        const int r = threadIdx.x - 64;
        float sq[2] = {0.0f, 0.0f};
        int s = 0, ph = 0;
        for (int kt = 0; kt < KT; kt++) {
            if (!mbar_wait(&full[s], ph, g.limit_ns)) s_bad = 1;
            __syncwarp();
            if (nt == 0) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const uint4* row = reinterpret_cast<const uint4*>(sm + s * stage + (r + 64 * h) * 128);
#pragma unroll
                    for (int c = 0; c < 8; c++) {
                        // a quarter warp's rows in different banks; eight squares in bf16, their
                        // sum in fp32: 2^-6 off at most, which the bound allows for
                        const uint4 q = row[(c + r) & 7];
                        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
                        __nv_bfloat162 p = __float2bfloat162_rn(0.0f);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&u[i]);
                            p = __hfma2(v, v, p);
                        }
                        sq[h] += __low2float(p) + __high2float(p);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++s == kRgStages) { s = 0; ph ^= 1; }
        }
        s_sq[r] = sq[0];
        s_sq[r + 64] = sq[1];
        __syncwarp();
        named_sync(1, 320);
    } else {
        const int r = 32 * (warp & 3) + lane, t = mt * 128 + r, half = (warp - 4) >> 2;
        const int width = min(g.N, g.Ep - nt * kRgMaxN) - half * 128;   // columns of this thread
        w_norms(warp - 4, 8);
        __syncwarp();
        float sum[8][16], top = 0.0f;
#pragma unroll
        for (int b = 0; b < 8; b++)
#pragma unroll
            for (int i = 0; i < 16; i++) sum[b][i] = 0.0f;
        for (int j = 0; j < chunks; j++) {
            if (!mbar_wait(&accf[j & 1], (j >> 1) & 1, g.limit_ns)) s_bad = 1;
            __syncwarp();
            tc_fence_after();
            const uint32_t acc = tbase + (j & 1) * g.N + ((uint32_t)(32 * (warp & 3)) << 16) + half * 128;
            float most = 0.0f;
#pragma unroll
            for (int b = 0; b < 8; b++) {
                if (16 * b >= width) break;
                uint32_t v[16];
                tmem_ld_32x16(acc + 16 * b, v);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    add_f32x2(sum[b][i], sum[b][i + 1], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    most = fmaxf(fmaxf(most, fabsf(__uint_as_float(v[i]))), fabsf(__uint_as_float(v[i + 1])));
                }
            }
            top += most;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acce[j & 1]);
        }
        if (width > 0) atomicMax(&s_max[r], __float_as_uint(top));
        __syncwarp();
        named_sync(1, 320);
        if (half == 0 && t < g.T) {
            // (a bound of NaN has the choice compute the token's logits in fp64)
            if (nt == 0) g.xn[(size_t)rank * g.T + t] = s_sq[r];
            g.xm[((size_t)rank * g.n_tiles + nt) * g.T + t] = s_bad ? __uint_as_float(0x7FC00000u) : __uint_as_float(s_max[r]);
        }
        // the stages are free now: a thread's half row goes through shared memory, so that it
        // leaves in one piece (its rows 528 bytes apart: different banks)
        if (width > 0 && t < g.T) {
            float* row = reinterpret_cast<float*>(sm) + (half * 128 + r) * 132;
#pragma unroll
            for (int b = 0; b < 8; b++)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4*>(row + 16 * b + i) =
                        make_float4(sum[b][i], sum[b][i + 1], sum[b][i + 2], sum[b][i + 3]);
            fence_proxy_async_smem();
            bulk_s2g(g.part + ((size_t)rank * g.T + t) * g.Ep + nt * kRgMaxN + half * 128, row, 4 * min(width, 128));
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, cols);
    }
}

// ---------------------------------------------------------------- many tokens: choice

// The larger one; a NaN on either side stays.
__device__ __forceinline__ float max_or_nan(float a, float b) { return b > a || b != b ? b : a; }

// What a warp's token still needs.
enum ChooseMode {
    kDone,
    kRanks,      // exact logits of a few experts, then the order of their ranks
    kGroups,     // exact logits of a few experts, then the groups they decide
    kAttempt,    // exact logits of the marked experts, then another route_attempt
    kAll         // every logit in fp64
};

struct ChooseShared {
    int n[kGemmTokens];                      // wanted logits per token
    int want[kGemmTokens][32];               // their experts (n > 32: all)
    double got[kGemmTokens][32];             // their values
    double part[2][kGemmTokens][4];          // the warps' parts of four dot products
    float w2[kGemmTokens];                   // largest |W_e|^2 each warp saw
};

// The wanted logits of the CTA's tokens in fp64, by all warps: each takes an eighth of H,
// four dot products at a time, U pieces of 8 elements of each on their way together.  Values go to
// got, or to the token's scratch where all are wanted.
template <int U>
__device__ __noinline__ void exact_logits(ChooseShared& sh, uint8_t* scratch, const uint16_t* x, const uint16_t* wr, int H, int E,
                                             int t0, int warp, int lane) {
    int total = 0;
    for (int h = 0; h < kGemmTokens; h++) total += sh.n[h];
    for (int j0 = 0, buf = 0; j0 < total; j0 += 4, buf ^= 1) {
        const uint4 *xr[4], *wrow[4];
#pragma unroll
        for (int a = 0; a < 4; a++) {
            int h = 0, j = min(j0 + a, total - 1);
            while (j >= sh.n[h]) j -= sh.n[h++];
            const int e = sh.n[h] > 32 ? j : sh.want[h][j];
            xr[a] = reinterpret_cast<const uint4*>(x + size_t(t0 + h) * H);
            wrow[a] = reinterpret_cast<const uint4*>(wr + size_t(e) * H);
        }
        double acc[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 1
        for (int c = warp * 32 + lane; c < H / 8; c += 32 * kGemmTokens * U) {
            uint4 xq[U][4], wq[U][4];
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int a = 0; a < 4; a++) {
                    const int at = c + 32 * kGemmTokens * u;
                    const bool in = u == 0 || at < H / 8;
                    xq[u][a] = in ? __ldg(xr[a] + at) : make_uint4(0, 0, 0, 0);
                    wq[u][a] = in ? __ldg(wrow[a] + at) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int a = 0; a < 4; a++) {
                    float xf[8], wf[8];
                    unpack8(xq[u][a], xf);
                    unpack8(wq[u][a], wf);
#pragma unroll
                    for (int r = 0; r < 8; r++) acc[a] = fma((double)xf[r], (double)wf[r], acc[a]);
                }
        }
        const double v = warp_sum_tokens<4>(acc, lane);
        if (lane % 8 == 0) sh.part[buf][warp][lane / 8] = v;
        __syncthreads();
        if (threadIdx.x < 4 && j0 + (int)threadIdx.x < total) {
            double sum = 0.0;
            for (int w = 0; w < kGemmTokens; w++) sum += sh.part[buf][w][threadIdx.x];
            int h = 0, j = j0 + threadIdx.x;
            while (j >= sh.n[h]) j -= sh.n[h++];
            if (sh.n[h] > 32) RouteScratch(scratch + h * RouteScratch::bytes(E), E).l[j] = sum;
            else sh.got[h][j] = sum;
        }
    }
    __syncthreads();
}

// One warp per token.  Five CTAs on an SM leave 96 registers a thread, so that exact_logits has half the
// loads in flight (with as many it spills).  That pays where there are many tokens, most of which need no
// exact logit: 8192 tokens of 4096 x 256 take 71.5 us with five and 73.2 with four, 8192 of 2048 x 128 47.1 and
// 49.3, but 2048 of 2048 x 128 25.5 and 24.4, and 8192 of 4096 x 256 with a softmax and a bias 500 and 388.
template <int kCtas>
__global__ void __launch_bounds__(kGemmTokens * 32, kCtas)
route_gemm_choose_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, RouteGemmArgs g, RouteChoice p,
                         int32_t* __restrict__ idx, float* __restrict__ wout) {
    extern __shared__ __align__(16) uint8_t sm_raw[];
    __shared__ ChooseShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.x * kGemmTokens, t = t0 + warp;
    const RouteScratch s(sm_raw + warp * RouteScratch::bytes(p.E), p.E);
    int32_t* idx_t = idx + size_t(t) * p.k;
    float* w_t = wout + size_t(t) * p.k;
    pdl_wait();
    pdl_trigger();
    int mode = kDone, my_e = 0;
    unsigned mark = 0;
    float delta = 0.0f, mx = 0.0f;
    RouteClose close;
    RouteSoftmax sm;
    double eta = 0.0;
    auto attempt = [&]() {
        if (!route_attempt(s, p, eta, lane, mark, my_e)) {
            mode = __reduce_add_sync(0xffffffffu, __popc(mark)) > 32 ? kAll : kAttempt;
            return;
        }
        route_weights(s, p, sm.mx, lane, my_e, route_bias_masks(p, my_e), idx_t, w_t);
        mode = kDone;
    };
    // the norms and largest sums, on their way while the logits are read
    float w2 = 0.0f, xn = 0.0f, xm = 0.0f;
    for (int e = threadIdx.x; e < p.E; e += kGemmTokens * 32) {
        w2 = max_or_nan(w2, __ldg(g.wn + e));
    }
    if (t < g.T) {
        if (lane < g.split) xn = __ldg(g.xn + (size_t)lane * g.T + t);
        if (lane < g.split)
            for (int i = 0; i < g.n_tiles; i++) xm = max_or_nan(xm, __ldg(g.xm + (size_t)(lane * g.n_tiles + i) * g.T + t));
        auto put = [&](int e, const float (&l)[4]) {
            float bias[4];
#pragma unroll
            for (int i = 0; i < 4; i++) bias[i] = p.bias && e + i < p.E ? __ldg(p.bias + e + i) : 0.0f;
            if (p.E % 4 == 0) {     // four at once: a quarter of the shared-memory conflicts
                *reinterpret_cast<double2*>(s.l + e) = make_double2(l[0], l[1]);
                *reinterpret_cast<double2*>(s.l + e + 2) = make_double2(l[2], l[3]);
                *reinterpret_cast<float4*>(s.l32 + e) = make_float4(l[0], l[1], l[2], l[3]);
                *reinterpret_cast<float4*>(s.bias + e) = make_float4(bias[0], bias[1], bias[2], bias[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (e + i < p.E) s.fill(e + i, l[i], l[i], bias[i]);
            }
        };
        // two times 128 experts, eight parts of each on their way together
#pragma unroll 1
        for (int e = 4 * lane; e < p.E; e += 256) {
            const float* col = g.part + (size_t)t * g.Ep + e;      // (rows are padded to 32)
            const bool two = e + 128 < p.E;
            float l[2][4] = {};
            for (int c0 = 0; c0 < g.split; c0 += 8) {
                float4 v[2][8];
#pragma unroll
                for (int c = 0; c < 8; c++)
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        v[h][c] = c0 + c < g.split && (h == 0 || two)
                                      ? __ldg(reinterpret_cast<const float4*>(col + (size_t)(c0 + c) * g.T * g.Ep + 128 * h))
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < 8; c++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        l[h][0] += v[h][c].x; l[h][1] += v[h][c].y; l[h][2] += v[h][c].z; l[h][3] += v[h][c].w;
                    }
            }
            put(e, l[0]);
            if (two) put(e + 128, l[1]);
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        w2 = max_or_nan(w2, __shfl_xor_sync(0xffffffffu, w2, off));
        xn += __shfl_xor_sync(0xffffffffu, xn, off);
        xm += __shfl_xor_sync(0xffffffffu, xm, off);
    }
    if (lane == 0) sh.w2[warp] = w2;
    __syncthreads();
    bool choose = false;
    unsigned groups = 0;
    if (t < g.T) {
        float wmax = 0.0f;
#pragma unroll
        for (int i = 0; i < kGemmTokens; i++) wmax = max_or_nan(wmax, sh.w2[i]);
        xn = with_lost_squares(xn, reinterpret_cast<const uint4*>(x + size_t(t) * g.H), g.H, lane);
        // (2 % for the norms, which err by 0.4 %, and for the roundings of xm and in these bounds themselves)
        delta = (float)(1.02 * (kErrorS * sqrt((double)xn * (double)wmax) +
                                 (kErrorV + 0x1p-24 * (g.Kc / (64 * kRgChunk) + 1 + g.split)) * (double)xm));
        if (!(delta <= 0.05f)) mode = kAll;
        else choose = true;
    }
    while (true) {
        if (choose) {
            bool masked;
            close = RouteClose();
            const RouteStatus st = route_fast(s, p, delta, lane, groups, mx, my_e, masked, close);
            __syncwarp();
            const bool common = !p.sigmoid && p.bias;     // the denominator hangs on every logit
            if (st == kRouteCertain) {
                route_weights(s, p, mx, lane, my_e, masked, idx_t, w_t);
                mode = kDone;
            } else if (st == kRouteClose) {
                mode = kRanks;
            } else if (common) {
                mode = kAll;
            } else if (st == kRouteGroups) {
                mode = kGroups;
            } else {
                eta = route_first_values(s, p, delta, lane, sm);
                attempt();
            }
            choose = false;
        }
        if (!__syncthreads_or(mode != kDone)) break;
        // publish what is wanted
        int n = mode == kAll ? p.E : 0, at = 0;      // at: this lane's first in the list
        if (mode == kAll && n <= 32) {
            if (lane < n) sh.want[warp][lane] = lane;
        } else if (mode == kRanks || mode == kGroups) {
            const unsigned wants = __ballot_sync(0xffffffffu, close.want);
            n = __popc(wants);
            at = __popc(wants & ((1u << lane) - 1));
            if (close.want) sh.want[warp][at] = close.e;
        } else if (mode == kAttempt) {
            at = __popc(mark);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, at, off);
                if (lane >= off) at += o;
            }
            n = __shfl_sync(0xffffffffu, at, 31);
            at -= __popc(mark);
            int j = at;
            for (unsigned m = mark; m; m &= m - 1) sh.want[warp][j++] = lane + 32 * (__ffs(m) - 1);
        }
        if (lane == 0) sh.n[warp] = n;
        __syncthreads();
        exact_logits<kCtas == 4 ? 2 : 1>(sh, sm_raw, x, wr, g.H, p.E, t0, warp, lane);
        if (mode == kAll) {
            if (n <= 32 && lane < n) s.l[lane] = sh.got[warp][lane];
            __syncwarp();
            route_choose_exact(s, p, lane, idx_t, w_t);
            mode = kDone;
        } else if (mode == kGroups) {
            if (close.want) s.l[close.e] = sh.got[warp][at];
            __syncwarp();
            groups = route_settle_groups(s, p, close, mx, 1.0, lane);
            if (groups != 0) choose = true;
            else mode = kAll;
        } else if (mode == kRanks) {
            if (close.want) s.l[close.e] = sh.got[warp][at];
            __syncwarp();
            // (a softmax's denominator: to the error of its logits)
            const bool common = !p.sigmoid && p.bias;
            bool sure;
            my_e = route_settle(s, p, close, mx, common ? route_softmax_inv(s.l, p.E, mx, lane) : 1.0,
                                common ? 1.1 * delta : 0.0, lane, sure);
            if (sure) route_weights(s, p, mx, lane, my_e, route_bias_masks(p, my_e), idx_t, w_t);
            mode = sure ? kDone : kAll;
        } else if (mode == kAttempt) {
            int j = at;
            for (unsigned m = mark; m; m &= m - 1) {
                const int e = lane + 32 * (__ffs(m) - 1);
                s.l[e] = sh.got[warp][j++];
                route_make_exact(s, p, sm, e);
            }
            __syncwarp();
            attempt();
        }
    }
}

// ---------------------------------------------------------------- given logits

// One warp per token; logits fp32 or bf16 with row stride ld.
__global__ void __launch_bounds__(kChooseWarps * 32)
route_select_kernel(const void* __restrict__ logits, int is_bf16, long long ld, int T, RouteChoice p,
                    int32_t* __restrict__ idx, float* __restrict__ wout) {
    extern __shared__ __align__(16) uint8_t sm_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x * kChooseWarps + warp;
    if (t >= T) return;
    const uint16_t* lh = reinterpret_cast<const uint16_t*>(logits) + t * ld;
    const float* lf = reinterpret_cast<const float*>(logits) + t * ld;
    choose_row([&](int e) { return (double)(is_bf16 ? __uint_as_float((uint32_t)lh[e] << 16) : lf[e]); }, false,
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
    if (T > kMaxRouteSize) return fail(MOE_EINVAL, "grouped route: T must be at most 2^30");
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
static cudaError_t raise_smem(Kern kern, int bytes, std::atomic<bool> (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
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

template <int TT>
static cudaError_t launch_small(const RouteCall& r) {
    auto kern = grouped_small_kernel<TT>;
    static std::atomic<bool> done[64] = {};
    cudaError_t e = raise_smem(kern, (int)(kSmallTile * RouteScratch::bytes(kMaxE)), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((r.p.E + 1) / 2, (r.T + TT - 1) / TT), dim3(kChooseWarps * 32),
                      TT * RouteScratch::bytes(r.p.E), r.s, r.x, r.wr, r.T, r.H, r.p, r.idx, r.w,
                      (double*)(r.ws + kCounterBytes), (unsigned int*)r.ws);
}

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
    g.xm = (float*)at;
    at += up256(size_t(g.split) * g.n_tiles * r.T * 4);
    g.wn = (float*)at;
    g.wr = r.wr;
    g.limit_ns = 2000000000ull;
    CUtensorMap mx, mw;
    int rc;
    if ((rc = make_tmap_2d(&mx, r.x, size_t(r.H) * 2, r.T, size_t(r.H) * 2, 128, 128, true))) return rc;
    if ((rc = make_tmap_2d(&mw, r.wr, size_t(r.H) * 2, E, size_t(r.H) * 2, 128, g.N, true))) return rc;
    static std::atomic<bool> gdone[64] = {}, cdone[2][64] = {};
    // (the sums leave through 2 x 128 half rows of 528 bytes)
    const int smem = std::max(kRgStages * (16384 + g.N * 128), 256 * 528) + 1024;
    MOE_CUDA_TRY(raise_smem(route_gemm_kernel, kRgStages * (16384 + kRgMaxN * 128) + 1024, gdone));
    const dim3 grid(((r.T + 127) / 128) * g.n_tiles * g.split);
    MOE_CUDA_TRY(launch_pdl(route_gemm_kernel, grid, dim3(kRgThreads), smem, r.s, mx, mw, g));
    const int ctas = (r.T + kGemmTokens - 1) / kGemmTokens;
    // more than two rounds of four an SM; a softmax with a bias asks for the most exact logits
    const bool many = ctas > 8 * kRgTargetCtas && (r.p.sigmoid || !r.p.bias);
    auto kern = many ? route_gemm_choose_kernel<5> : route_gemm_choose_kernel<4>;
    MOE_CUDA_TRY(raise_smem(kern, (int)(kGemmTokens * RouteScratch::bytes(kMaxE)), cdone[many]));
    MOE_CUDA_TRY(launch_pdl(kern, dim3(ctas), dim3(kGemmTokens * 32), kGemmTokens * RouteScratch::bytes(E), r.s, r.x, r.wr,
                            g, r.p, r.idx, r.w));
    return MOE_OK;
}

static int launch_grouped(const RouteCall& r) {
    if (r.T > kSmallT) return launch_large(r);
    const cudaError_t e = r.T == 1 ? launch_small<1>(r) : r.T == 2 ? launch_small<2>(r)
                          : r.T <= 4 ? launch_small<4>(r) : launch_small<8>(r);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "grouped router launch");
}

static int launch_select(const void* logits, int bf16, long long ld, int T, const RouteChoice& p, int32_t* idx, float* w,
                         cudaStream_t s) {
    auto kern = route_select_kernel;
    static std::atomic<bool> done[64] = {};
    MOE_CUDA_TRY(raise_smem(kern, (int)(kChooseWarps * RouteScratch::bytes(kMaxE)), done));
    MOE_CUDA_TRY(launch_pdl(kern, dim3((T + kChooseWarps - 1) / kChooseWarps), dim3(kChooseWarps * 32),
                            kChooseWarps * RouteScratch::bytes(p.E), s, logits, bf16, ld, T, p, idx, w));
    return MOE_OK;
}

// Load the kernels now (module loading may wait for the device).
int preload_route_grouped_kernels() {
    cudaFuncAttributes fa;
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, grouped_small_kernel<1>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, grouped_small_kernel<2>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, grouped_small_kernel<4>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, grouped_small_kernel<8>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, route_gemm_kernel));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, route_gemm_choose_kernel<4>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, route_gemm_choose_kernel<5>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, route_select_kernel));
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

// What a call with T tokens uses.
static size_t route_workspace(int T, int E) {
    if (T <= kSmallT) return kCounterBytes + up256(size_t(T) * E * sizeof(double));
    const size_t split = route_split(T, E), Ep = (E + 31) / 32 * 32;
    const size_t tiles = (E + kRgMaxN - 1) / kRgMaxN;
    return kCounterBytes + up256(split * T * Ep * 4) + up256(split * T * 4) + up256(split * tiles * T * 4) + up256(size_t(E) * 4);
}

extern "C" size_t moe_route_grouped_workspace_bytes(int T, int E) {
    if (T <= 0 || T > kMaxRouteSize || E <= 0 || E > kMaxE) return 0;
    // more tiles of tokens have fewer parts: the most of any number of tiles up to T's
    size_t most = route_workspace(T, E);
    for (int t = 128; t < T && t <= 128 * kRgTargetCtas; t += 128) most = std::max(most, route_workspace(t, E));
    return most;
}

extern "C" int moe_route_grouped(const void* x_bf16, const void* wr_bf16, const float* bias, int T, int H, int E,
                                 const moe_route_choice* choice, int32_t* idx, float* w, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    RouteChoice p;
    const int rc = check_choice(choice, bias, T, E, p);
    if (rc) return rc;
    if (!x_bf16 || !wr_bf16 || !idx || !w) return fail(MOE_EINVAL, "null pointer");
    if (H <= 0 || H % 8 || H > kMaxRouteSize)
        return fail(MOE_EINVAL, "grouped route: H must be a positive multiple of 8, at most 2^30");
    if ((reinterpret_cast<uintptr_t>(x_bf16) | reinterpret_cast<uintptr_t>(wr_bf16)) & 15)
        return fail(MOE_EINVAL, "grouped route: x and W_r must be 16-byte aligned");
    if (!workspace || workspace_bytes < route_workspace(T, E))
        return fail(MOE_EINVAL, "grouped route: workspace missing or smaller than moe_route_grouped_workspace_bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MOE_EINVAL, "grouped route: workspace must be 256-byte aligned");
    const RouteCall r{(const uint16_t*)x_bf16, (const uint16_t*)wr_bf16, T, H, p, idx, w, (char*)workspace, (cudaStream_t)stream};
    return launch_grouped(r);
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
    return launch_select(logits, type == MOE_BF16, ld, T, p, idx, w, (cudaStream_t)stream);
}
