// Products of a few tokens with one 4-bit matrix: y = add + W x, and the gated
// pair h = silu(W_gate x) * (W_up x).
//
// One warp per output row; lane j takes the 32-element chunks c with c % 32 == j
// (16 code bytes), dequantises them and sums its products in fp32.
#include "common.cuh"

namespace moe {

constexpr int kLinWarps = 8;

struct Fp4Mat {
    const uint8_t* codes;
    const uint8_t* scales;
    float ts;
};
struct LinArgs {
    Fp4Mat m[2];
    int N, K, T, x_f32, y_f32;
    const void* x;
    long long ldx;
    const void* add;
    long long ld_add;
    void* y;
    long long ldy;
};

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const float v = m < 2 ? 0.5f * m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return (c & 8u) ? -v : v;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    const uint32_t ex = (b >> 3) & 15u, mn = b & 7u;
    float v = ex ? __uint_as_float(((ex + 120u) << 23) | (mn << 20)) : (float)mn * 0.001953125f;
    if ((b & 0x7fu) == 0x7fu) v = __uint_as_float(0x7fc00000u);
    return (b & 0x80u) ? -v : v;
}
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7fc00000u) : b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u);
}
__device__ __forceinline__ float load_act(const void* p, int f32, long long i) {
    return f32 ? static_cast<const float*>(p)[i]
               : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

template <int FMT, int GATED>
__global__ void __launch_bounds__(kLinWarps * 32) fp4_linear_kernel(const LinArgs a) {
    const int lane = threadIdx.x & 31, n = blockIdx.x * kLinWarps + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (n >= a.N) return;
    constexpr int BS = FMT == MOE_MXFP4 ? 32 : 16;
    for (int t = 0; t < a.T; t++) {
        float acc[2] = {0.0f, 0.0f};
        for (int c = lane; c < a.K / 32; c += 32)
            for (int m = 0; m <= GATED; m++) {
                const uint8_t* cp = a.m[m].codes + (size_t)n * (a.K / 2) + c * 16;
                const uint8_t* sp = a.m[m].scales + (size_t)n * (a.K / BS) + c * (32 / BS);
                for (int b = 0; b < 32 / BS; b++) {
                    float part = 0.0f;
                    for (int i = 0; i < BS / 2; i++) {
                        const uint32_t v = cp[b * (BS / 2) + i];
                        const long long k = c * 32 + b * BS + 2 * i;
                        part = fmaf(e2m1_value(v & 15u), load_act(a.x, a.x_f32, t * a.ldx + k), part);
                        part = fmaf(e2m1_value(v >> 4), load_act(a.x, a.x_f32, t * a.ldx + k + 1), part);
                    }
                    acc[m] = fmaf(part, FMT == MOE_MXFP4 ? e8m0_value(sp[b]) : e4m3_value(sp[b]), acc[m]);
                }
            }
        for (int off = 16; off >= 1; off >>= 1)
            for (int m = 0; m <= GATED; m++) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], off);
        if (lane) continue;
        float v = acc[0] * a.m[0].ts;
        if (GATED) {
            const float u = acc[1] * a.m[1].ts;
            v = v / (1.0f + expf(-v)) * u;
        }
        if (a.add) v += load_act(a.add, a.y_f32, t * a.ld_add + n);
        if (a.y_f32) static_cast<float*>(a.y)[t * a.ldy + n] = v;
        else static_cast<__nv_bfloat16*>(a.y)[t * a.ldy + n] = __float2bfloat16_rn(v);
    }
}

static int check_weight(const moe_fp4_weight* w) {
    if (!w || !w->codes || !w->scales) return fail(MOE_EINVAL, "fp4 weight: null pointer");
    if (w->fmt != MOE_MXFP4 && w->fmt != MOE_NVFP4) return fail(MOE_EINVAL, "fp4 weight: unknown format");
    if (w->N <= 0 || w->K <= 0 || w->K % 32) return fail(MOE_EINVAL, "fp4 weight: need N > 0 and K a positive multiple of 32");
    if (reinterpret_cast<uintptr_t>(w->codes) & 15) return fail(MOE_EINVAL, "fp4 weight: codes must be 16-byte aligned");
    return MOE_OK;
}

static int check_rows(const void* p, int type, long long ld, int width, int T, const char* what) {
    const int size = type == MOE_BF16 ? 2 : 4;
    if (!p) return fail(MOE_EINVAL, std::string("fp4: null ") + what);
    if (type != MOE_BF16 && type != MOE_F32) return fail(MOE_EINVAL, std::string("fp4: bad type of ") + what);
    if (T > 1 && ld < width) return fail(MOE_EINVAL, std::string("fp4: row stride too small for ") + what);
    if (reinterpret_cast<uintptr_t>(p) % size) return fail(MOE_EINVAL, std::string("fp4: not aligned to its type: ") + what);
    return MOE_OK;
}

static int launch(const LinArgs& a, int fmt, int gated, cudaStream_t s) {
    const dim3 grid((a.N + kLinWarps - 1) / kLinWarps), block(kLinWarps * 32);
    cudaError_t e;
    if (fmt == MOE_MXFP4) e = gated ? launch_pdl(fp4_linear_kernel<MOE_MXFP4, 1>, grid, block, 0, s, a)
                                    : launch_pdl(fp4_linear_kernel<MOE_MXFP4, 0>, grid, block, 0, s, a);
    else e = gated ? launch_pdl(fp4_linear_kernel<MOE_NVFP4, 1>, grid, block, 0, s, a)
                   : launch_pdl(fp4_linear_kernel<MOE_NVFP4, 0>, grid, block, 0, s, a);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e, "fp4 linear launch");
}

}  // namespace moe

using namespace moe;

extern "C" int moe_fp4_linear(const moe_fp4_weight* w, const void* x, int x_type, long long ldx, int T, const void* add,
                              long long ld_add, void* y, int y_type, long long ldy, int* status, void* stream) {
    int rc = check_weight(w);
    if (rc) return rc;
    if (T <= 0 || T > kMaxDecodeT) return fail(MOE_EINVAL, "fp4 linear: T must be in [1, 16]");
    if (!status) return fail(MOE_EINVAL, "fp4 linear: null status");
    if ((rc = check_rows(x, x_type, ldx, w->K, T, "x"))) return rc;
    if ((rc = check_rows(y, y_type, ldy, w->N, T, "y"))) return rc;
    if (add && (rc = check_rows(add, y_type, ld_add, w->N, T, "add"))) return rc;
    if ((reinterpret_cast<uintptr_t>(x) & 15) || (T > 1 && (ldx * (x_type == MOE_BF16 ? 2 : 4)) % 16))
        return fail(MOE_EINVAL, "fp4 linear: rows of x must be 16-byte aligned");
    LinArgs a{};
    a.m[0] = Fp4Mat{w->codes, w->scales, w->fmt == MOE_NVFP4 ? w->tensor_scale : 1.0f};
    a.N = w->N; a.K = w->K; a.T = T;
    a.x = x; a.x_f32 = x_type == MOE_F32; a.ldx = ldx;
    a.add = add; a.ld_add = ld_add;
    a.y = y; a.y_f32 = y_type == MOE_F32; a.ldy = ldy;
    return launch(a, w->fmt, 0, (cudaStream_t)stream);
}

extern "C" int moe_fp4_swiglu(const moe_fp4_weight* gate, const moe_fp4_weight* up, const void* x, int x_type,
                              long long ldx, int T, float* h, long long ldh, int* status, void* stream) {
    int rc = check_weight(gate);
    if (rc || (rc = check_weight(up))) return rc;
    if (gate->N != up->N || gate->K != up->K || gate->fmt != up->fmt)
        return fail(MOE_EINVAL, "fp4 swiglu: gate and up must have one shape and format");
    if (T <= 0 || T > kMaxDecodeT) return fail(MOE_EINVAL, "fp4 swiglu: T must be in [1, 16]");
    if (!status) return fail(MOE_EINVAL, "fp4 swiglu: null status");
    if ((rc = check_rows(x, x_type, ldx, gate->K, T, "x"))) return rc;
    if ((rc = check_rows(h, MOE_F32, ldh, gate->N, T, "h"))) return rc;
    if ((reinterpret_cast<uintptr_t>(x) & 15) || (T > 1 && (ldx * (x_type == MOE_BF16 ? 2 : 4)) % 16))
        return fail(MOE_EINVAL, "fp4 swiglu: rows of x must be 16-byte aligned");
    LinArgs a{};
    const bool nv = gate->fmt == MOE_NVFP4;
    a.m[0] = Fp4Mat{gate->codes, gate->scales, nv ? gate->tensor_scale : 1.0f};
    a.m[1] = Fp4Mat{up->codes, up->scales, nv ? up->tensor_scale : 1.0f};
    a.N = gate->N; a.K = gate->K; a.T = T;
    a.x = x; a.x_f32 = x_type == MOE_F32; a.ldx = ldx;
    a.y = h; a.y_f32 = 1; a.ldy = ldh;
    return launch(a, gate->fmt, 1, (cudaStream_t)stream);
}
