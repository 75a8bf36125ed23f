// Grouped router: logits x W_r^T summed in fp64, then the choice of route_select.cuh.
#include "common.cuh"
#include "route_select.cuh"

namespace moe {

constexpr int kGroupedWarps = 4;
constexpr int kGroupedTile = 8;      // largest token tile
constexpr int kMaxGroups = 32;

// Each warp owns EPW experts and a tile of TT tokens; lane j sums the 8-element
// chunks c with c % 32 == j.  Products of two bf16 values are exact in fp64.  The
// last CTA of a token tile (a ticket per tile, reset by that CTA) makes the choice.
template <int EPW, int TT, int VPL>
__global__ void __launch_bounds__(kGroupedWarps * 32)
grouped_router_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ wr, int T, int H, RouteChoice p,
                      int32_t* __restrict__ idx, float* __restrict__ wout, double* __restrict__ logits,
                      unsigned int* __restrict__ tile_cnt) {
    extern __shared__ double sm[];   // [warps][E] logits, [warps][E] keys
    __shared__ int s_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t0 = blockIdx.y * TT, nt = min(TT, T - t0);
    const int e0 = (blockIdx.x * kGroupedWarps + warp) * EPW;
    pdl_trigger();
    pdl_wait();
    double acc[EPW][TT];
#pragma unroll
    for (int a = 0; a < EPW; a++)
#pragma unroll
        for (int t = 0; t < TT; t++) acc[a][t] = 0.0;
    for (int c = lane; c < H / 8; c += 32) {
        double wf[EPW][8];
#pragma unroll
        for (int a = 0; a < EPW; a++) {
            uint4 q = make_uint4(0, 0, 0, 0);
            if (e0 + a < p.E) q = __ldg(reinterpret_cast<const uint4*>(wr + size_t(e0 + a) * H) + c);
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int r = 0; r < 4; r++) {
                wf[a][2 * r] = __uint_as_float(u[r] << 16);
                wf[a][2 * r + 1] = __uint_as_float(u[r] & 0xFFFF0000u);
            }
        }
#pragma unroll
        for (int t = 0; t < TT; t++) {
            if (t >= nt) break;
            const uint4 q = *(reinterpret_cast<const uint4*>(x + size_t(t0 + t) * H) + c);
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const double lo = __uint_as_float(u[r] << 16), hi = __uint_as_float(u[r] & 0xFFFF0000u);
#pragma unroll
                for (int a = 0; a < EPW; a++) {
                    acc[a][t] = fma(lo, wf[a][2 * r], acc[a][t]);
                    acc[a][t] = fma(hi, wf[a][2 * r + 1], acc[a][t]);
                }
            }
        }
    }
#pragma unroll
    for (int a = 0; a < EPW; a++)
#pragma unroll
        for (int t = 0; t < TT; t++) {
            const double v = warp_sum(acc[a][t]);
            if (lane == 0 && e0 + a < p.E && t < nt) logits[size_t(t0 + t) * p.E + e0 + a] = v;
        }
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(tile_cnt + blockIdx.y, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    double* l = sm + warp * p.E;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(sm + (kGroupedWarps + warp) * p.E);
    for (int t = warp; t < nt; t += kGroupedWarps) {
        for (int e = lane; e < p.E; e += 32) l[e] = __ldcg(logits + size_t(t0 + t) * p.E + e);
        __syncwarp();
        route_choose_warp<VPL>(l, keys, p, lane, idx + size_t(t0 + t) * p.k, wout + size_t(t0 + t) * p.k);
    }
    if (threadIdx.x == 0) tile_cnt[blockIdx.y] = 0;
}

// One warp per token; logits fp32 or bf16 with row stride ld.
template <int VPL>
__global__ void __launch_bounds__(kGroupedWarps * 32)
route_select_kernel(const void* __restrict__ logits, int is_bf16, long long ld, int T, RouteChoice p,
                    int32_t* __restrict__ idx, float* __restrict__ wout) {
    extern __shared__ double sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double* l = sm + warp * p.E;
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(sm + (kGroupedWarps + warp) * p.E);
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x * kGroupedWarps + warp;
    if (t >= T) return;
    for (int e = lane; e < p.E; e += 32)
        l[e] = is_bf16 ? (double)__uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(logits)[t * ld + e] << 16)
                       : (double)reinterpret_cast<const float*>(logits)[t * ld + e];
    __syncwarp();
    route_choose_warp<VPL>(l, keys, p, lane, idx + size_t(t) * p.k, wout + size_t(t) * p.k);
}

static size_t round_up256(size_t n) { return (n + 255) / 256 * 256; }
static size_t grouped_logits_bytes(int T, int E) { return round_up256(size_t(T) * E * sizeof(double)); }

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

// VPL registers per lane hold the E selection values
#define MOE_BY_EXPERTS(E, CALL)          \
    ((E) <= 128 ? CALL(4) : (E) <= 256 ? CALL(8) : CALL(32))

static size_t choice_smem(int E) { return size_t(2) * kGroupedWarps * E * sizeof(double); }

template <int EPW, int TT, int VPL>
static cudaError_t launch_grouped(const uint16_t* x, const uint16_t* wr, int T, int H, const RouteChoice& p,
                                  int32_t* idx, float* w, double* logits, unsigned int* cnt, cudaStream_t s) {
    auto kern = grouped_router_kernel<EPW, TT, VPL>;
    const size_t smem = choice_smem(p.E);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)choice_smem(kMaxE));
    if (e != cudaSuccess) return e;
    dim3 grid((p.E + kGroupedWarps * EPW - 1) / (kGroupedWarps * EPW), (T + TT - 1) / TT);
    return launch_pdl(kern, grid, dim3(kGroupedWarps * 32), smem, s, x, wr, T, H, p, idx, w, logits, cnt);
}

template <int VPL>
static cudaError_t grouped_by_tokens(const uint16_t* x, const uint16_t* wr, int T, int H, const RouteChoice& p,
                                     int32_t* idx, float* w, double* logits, unsigned int* cnt, cudaStream_t s) {
    if (T == 1) return launch_grouped<1, 1, VPL>(x, wr, T, H, p, idx, w, logits, cnt, s);
    if (T <= 4) return launch_grouped<1, 4, VPL>(x, wr, T, H, p, idx, w, logits, cnt, s);
    return launch_grouped<2, 8, VPL>(x, wr, T, H, p, idx, w, logits, cnt, s);
}

template <int VPL>
static cudaError_t launch_select(const void* logits, int bf16, long long ld, int T, const RouteChoice& p, int32_t* idx,
                                 float* w, cudaStream_t s) {
    auto kern = route_select_kernel<VPL>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)choice_smem(kMaxE));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((T + kGroupedWarps - 1) / kGroupedWarps), dim3(kGroupedWarps * 32), choice_smem(p.E), s,
                      logits, bf16, ld, T, p, idx, w);
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_grouped_workspace_bytes(int T, int E) {
    if (T <= 0 || E <= 0 || E > kMaxE) return 0;
    return grouped_logits_bytes(T, E) + round_up256(size_t(T) * sizeof(unsigned int));
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
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return fail(MOE_EINVAL, "grouped route: workspace must be 16-byte aligned");
    double* logits = (double*)workspace;
    unsigned int* cnt = (unsigned int*)((char*)workspace + grouped_logits_bytes(T, E));
#define CALL(V) grouped_by_tokens<V>((const uint16_t*)x_bf16, (const uint16_t*)wr_bf16, T, H, p, idx, w, logits, cnt, (cudaStream_t)stream)
    const cudaError_t e = MOE_BY_EXPERTS(E, CALL);
#undef CALL
    if (e != cudaSuccess) return cuda_fail(e, "grouped router launch");
    return MOE_OK;
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
#define CALL(V) launch_select<V>(logits, type == MOE_BF16, ld, T, p, idx, w, (cudaStream_t)stream)
    const cudaError_t e = MOE_BY_EXPERTS(E, CALL);
#undef CALL
    if (e != cudaSuccess) return cuda_fail(e, "route select launch");
    return MOE_OK;
}
