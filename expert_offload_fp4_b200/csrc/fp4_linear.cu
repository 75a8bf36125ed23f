// Products of a few tokens with one 4-bit matrix: y = add + W x, and the gated
// pair h = silu(W_gate x) * (W_up x), on the block-scaled FP4 tensor cores.
//
// The tensor core multiplies E2M1 by E2M1 and applies W's block scales itself, so
// the weights go from HBM to shared memory to the MMA untouched, with no
// dequantisation on the way (on the CUDA cores that costs 2-3 instructions a weight
// and keeps them from reading at HBM speed).  What has to become E2M1 is x, and it
// does so without loss: with E the exponent of a token's largest |x| in the CTA's
// share of K, X = rint(x 2^(21 - E)) is a 23-bit integer, and
//     X = sum_d u_d 8^d,  u_d in {-4 .. 3},  d = 0 .. 7
// in balanced octal digits, each of them an E2M1 value.  The 8 digits of a token are
// 8 columns of the MMA's B operand, D_d = W u_d is exact up to fp32 accumulation,
// and  W x = 2^E sum_d 8^(d - 7) D_d.  (bf16 elements down to 2^-14 of the largest
// enter exactly, smaller ones and fp32 elements to 2^-22 of the largest.)  Sixteen
// tokens fill an N = 128 MMA, which still takes a third of the time HBM needs to
// bring its 128 x 64 weights.
//
// A cluster of C CTAs shares the 128 rows of a tile, CTA r taking the r-th part Kc
// of K: with few tiles this spreads a matrix over the SMs, and it keeps the digits
// of a CTA's part of x (4 Kc bytes a token) resident in shared memory for all the
// tiles the cluster works through.  The parts' sums meet in shared memory, row r of
// a tile at the CTA that owns it, and are added in rank order, so the result does
// not depend on timing.  Warp roles:
//   warp 0       TMA producer: a 128-row x 256-element code tile per stage
//   warp 1       MMA issuer (owns the TMEM allocation)
//   warps 1-7    digits of x, first (1-11 where there are many)
//   warps 2-3    exchange buffer -> sum over the cluster -> y, one tile behind the
//                drain, so that neither waits for the other
//   warps 4-7    drain: TMEM -> digit sum -> the owner's exchange buffer
//   warps 8-11   block scales, one row a thread: global memory -> shared memory ->
//                TMEM scale columns (tcgen05.st: four tcgen05.cp a stage took as long
//                as the stage's MMAs)
// The gated form puts 64 gate rows and the same 64 up rows in one tile.
// Bound by HBM for large matrices: 131072 x 4096 NVFP4 takes 51.3 us for one token (5.9 TB/s),
// 62.4 for 16 (their digits take 5 us before the stream starts, then a stage 0.45 us, not
// 0.41); by latency for small ones: 4096 x 4096 6.5 us for one token (1.4 TB/s), 9.5 for 16;
// the gated pair and down of 2048 x 768 10.7 together.
// All waits are bounded; a timeout sets bit 16 of *status and the CTA carries on.
#include "tcgen05.cuh"

#include <mutex>
#include <type_traits>

namespace moe {

int make_tmap_2d(CUtensorMap* map, const void* base, uint64_t row_bytes, uint64_t rows, uint64_t pitch,
                 uint32_t box_bytes, uint32_t box_rows, bool swizzle128);

constexpr int kLinThreads = 384;
constexpr int kLinKT = 256;               // K elements of a stage (128 code bytes a row)
constexpr int kLinMaxStages = 5;
constexpr int kLinMaxCluster = 8;
constexpr int kLinSumThreads = 64;        // warps 2, 3

struct LinMat {
    const uint8_t* scales;
    float ts;
};
struct LinArgs {
    LinMat m[2];
    int N, K, T;
    int Kc;              // K elements per CTA, a multiple of kLinKT
    int C;               // CTAs per cluster
    int stages;
    int tiles;
    int wide_scales;     // scale rows can be read 16 (NVFP4) or 8 (MXFP4) bytes at a time
    uint32_t tmem_cols;
    int tp_inv, r_inv;   // ceil(65536 / x) of Tp and of the output rows per owner, for small quotients
    int x_f32, y_f32;
    const void* x;
    long long ldx;
    const void* add;
    long long ld_add;
    void* y;
    long long ldy;
    int* status;
    unsigned long long limit_ns;
};

// Floats of one row's values in the exchange buffer: its tokens in fours, and four
// more so that the rows of a quarter warp fall into different banks.
__host__ __device__ constexpr int lin_row_words(int Tp) { return (Tp + 3) / 4 * 4 + 4; }

// Shared-memory offsets from the 1024-aligned base.
struct LinSmem {
    int codes, digits, scales, ones, exch, bars, args, total;
    __host__ __device__ LinSmem(int stages, int Tp, int Kc, int C, int gated) {
        codes = 0;
        digits = codes + stages * 16384;
        scales = digits + Tp * 8 * (Kc / 2);
        ones = scales + 4 * 2048;
        exch = ones + 512;
        const int out = gated ? 64 : 128, R = (out + C - 1) / C;
        bars = exch + 2 * 4 * C * (gated ? 2 : 1) * R * lin_row_words(Tp);
        bars = (bars + 15) / 16 * 16;   // (and the arguments after the barriers 8-byte aligned)
        args = bars + (2 * kLinMaxStages + 9) * 8 + 48 * 4 + 16;
        total = args + (int)sizeof(LinArgs);
    }
};

// D[tmem] (+)= A[smem] x B[smem]^T with 32-element E8M0 block scales from TMEM.
__device__ __forceinline__ void mma_mxfp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p; }"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}

// 32 lanes x 8 consecutive fp32 columns; complete after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld_32x8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 lanes x 16 consecutive columns from registers; complete after the wait.
__device__ __forceinline__ void tmem_st_32x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13,"
        " %14, %15};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- cluster

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t smem, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}
// Four floats to a CTA of the cluster; the bytes count on that CTA's barrier `bar`.
__device__ __forceinline__ void st_async_f32x4(uint32_t addr, const float (&v)[4], uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(bar) : "memory");
}
// Without release: it stands for reads whose values were used already, not for writes.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, unsigned long long limit_ns) {
    const unsigned long long t0 = globaltimer();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;"
            " selp.u32 %0, 1, 0, p; }"
            : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
        if (ok) return true;
        if (globaltimer() - t0 > limit_ns) return false;
    }
}

// Bring a tile of global memory towards L2 only: no thread sees the data, so it may
// run before the kernel's wait for its predecessor.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// ---------------------------------------------------------------- x digits

// 8 consecutive elements of x, as they are in memory.
template <int XF32>
struct X8 {
    uint4 q[XF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* x, bool in) {   // zeros if not in
        q[0] = make_uint4(0, 0, 0, 0);
        if (XF32) q[XF32] = q[0];
        if (!in) return;
        q[0] = static_cast<const uint4*>(x)[0];
        if (XF32) q[XF32] = static_cast<const uint4*>(x)[XF32];
    }
    __device__ __forceinline__ void put(uint8_t* p, int lane) const {
        reinterpret_cast<uint4*>(p)[lane] = q[0];
        if (XF32) reinterpret_cast<uint4*>(p)[32 + lane] = q[XF32];
    }
    __device__ __forceinline__ void get(const uint8_t* p, int lane) {
        q[0] = reinterpret_cast<const uint4*>(p)[lane];
        if (XF32) q[XF32] = reinterpret_cast<const uint4*>(p)[32 + lane];
    }
    __device__ __forceinline__ uint32_t bits(int i) const {   // element i as fp32
        const uint4& v = q[XF32 ? i >> 2 : 0];
        const int j = XF32 ? i & 3 : i >> 1;
        const uint32_t w = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
        return XF32 ? w : (i & 1) ? w & 0xFFFF0000u : w << 16;
    }
};

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// X + 4 (8^8 - 1) / 7, whose plain octal digits are u_d + 4, as 8 selector nibbles, the
// lowest digit in the lowest nibble.
__device__ __forceinline__ uint32_t octal_nibbles(uint32_t u) {
    const uint32_t w = u + (u & 0xFFF000u) * 15u;          // 12 bits to the upper half: x + h (2^4 - 1)
    const uint32_t t = w + (w & 0x0FC00FC0u) * 3u;         // 6 bits to the next byte
    return t + (t & 0x38383838u);                          // 3 bits to the next nibble
}

// 8 elements -> for each digit d the 4 bytes (8 codes) of B's row d.
__device__ __forceinline__ void digit_rows(const uint32_t (&X)[8], uint32_t (&row)[8]) {
    // E2M1 codes of -4 -3 -2 -1 | 0 1 2 3, and the same in the high nibble
    constexpr uint32_t la = 0x0A0C0D0Eu, lb = 0x05040200u, ha = la << 4, hb = lb << 4;
    uint32_t p[2][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t s0 = octal_nibbles(X[2 * i]), s1 = octal_nibbles(X[2 * i + 1]);
        p[0][i] = __byte_perm(la, lb, s0) | __byte_perm(ha, hb, s1);
        p[1][i] = __byte_perm(la, lb, s0 >> 16) | __byte_perm(ha, hb, s1 >> 16);
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {   // 4 x 4 byte transpose
        const uint32_t t0 = __byte_perm(p[h][0], p[h][1], 0x5140), t1 = __byte_perm(p[h][2], p[h][3], 0x5140);
        const uint32_t t2 = __byte_perm(p[h][0], p[h][1], 0x7362), t3 = __byte_perm(p[h][2], p[h][3], 0x7362);
        row[4 * h + 0] = __byte_perm(t0, t1, 0x5410);
        row[4 * h + 1] = __byte_perm(t0, t1, 0x7632);
        row[4 * h + 2] = __byte_perm(t2, t3, 0x5410);
        row[4 * h + 3] = __byte_perm(t2, t3, 0x7632);
    }
}

// ---------------------------------------------------------------- block scales

// The scales of one row and stage: 16 bytes (NVFP4) or 8 (MXFP4, in x and y).  p: the
// stage's first scale of the row, n: how many scales the row has from there (0 for
// a row or stage outside).  WIDE: rows are whole stages and aligned to them; else
// bytes, two at a time where the address is even.
template <int FMT, bool WIDE>
__device__ __forceinline__ uint4 load_scales(const uint8_t* p, int n) {
    constexpr int per = FMT == MOE_NVFP4 ? 16 : 8;   // scales per stage
    uint32_t b[4] = {0, 0, 0, 0};
    if (WIDE) {
        if (n > 0) {
            if constexpr (FMT == MOE_NVFP4) return __ldg(reinterpret_cast<const uint4*>(p));
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
            return make_uint4(u.x, u.y, 0, 0);
        }
    } else if ((reinterpret_cast<uintptr_t>(p) & 1) == 0) {
#pragma unroll
        for (int i = 0; i < per / 2; i++)
            if (2 * i + 1 < n) b[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p) + i) << (16 * (i % 2));
            else if (2 * i < n) b[i / 2] |= (uint32_t)__ldg(p + 2 * i) << (16 * (i % 2));
    } else {
#pragma unroll
        for (int i = 0; i < per; i++)
            if (i < n) b[i / 4] |= (uint32_t)__ldg(p + i) << (8 * (i % 4));
    }
    return make_uint4(b[0], b[1], b[2], b[3]);
}

// ---------------------------------------------------------------- kernel

template <int FMT, int GATED, int XF32>
__global__ void __launch_bounds__(kLinThreads, 1)
fp4_linear_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                  const __grid_constant__ LinArgs args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int S = args.stages, C = args.C, T = args.T, Tp = (T + 1) & ~1;
    const LinSmem L(S, Tp, args.Kc, C, GATED);
    // the arguments once more in shared memory: read late for the first time, each line of
    // the constant bank is a miss of several hundred cycles
    const LinArgs& a = *reinterpret_cast<const LinArgs*>(sm + L.args);
    static_assert(sizeof(LinArgs) % 8 == 0 && sizeof(LinArgs) / 4 <= kLinThreads, "");
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L.bars);      // codes landed, scales in TMEM
    uint64_t* empty = full + kLinMaxStages;                         // stage read by its MMAs
    uint64_t* accf = empty + kLinMaxStages;                         // [2] accumulator complete
    uint64_t* acce = accf + 2;                                      // [2] accumulator read
    uint64_t* exf = acce + 2;                                       // [2] exchange buffer complete
    uint64_t* exe = exf + 2;                                        // [2] this CTA's values read by their owners
    uint64_t* bready = exe + 2;                                     // digits of x complete
    uint32_t* xmax = reinterpret_cast<uint32_t*>(bready + 1);       // [16] largest |x| bits, then 2 x [16] 2^E
    float* xscale = reinterpret_cast<float*>(xmax + 16);
    uint32_t* tmem_slot = xmax + 48;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int cl = blockIdx.x / C, ncl = gridDim.x / C;
    const int k0 = rank * args.Kc;
    const int steps = (min(args.K - k0, args.Kc) + 63) / 64;              // 64-element MMA steps of this CTA
    const int KT = (steps + 3) / 4;                                 // stages per tile
    constexpr int TR = GATED ? 64 : 128;                            // rows of each matrix per tile
    // the scale warps help with the digits only where there are many
    const int items = Tp * KT, nprep = items > 21 ? 11 : 7;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; s++) {
            mbar_init(&full[s], 1 + 4);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&accf[i], 1);
            mbar_init(&acce[i], 4);
            mbar_init(&exf[i], C > 1 ? 1 : 4);
            mbar_init(&exe[i], kLinSumThreads / 32 * C);
        }
        mbar_init(bready, nprep);
        fence_mbar_init();
        prefetch_tmap(&map0);
        if (GATED) prefetch_tmap(&map1);
    }
    if (threadIdx.x < sizeof(LinArgs) / 4)
        reinterpret_cast<uint32_t*>(sm + L.args)[threadIdx.x] = reinterpret_cast<const uint32_t*>(&args)[threadIdx.x];
    if (threadIdx.x < 16) xmax[threadIdx.x] = 0;
    if (threadIdx.x >= 64 && threadIdx.x < 64 + 128)
        reinterpret_cast<uint32_t*>(sm + L.ones)[threadIdx.x - 64] = FMT == MOE_NVFP4 ? 0x38383838u : 0x7F7F7F7Fu;
    if (warp == 1) tmem_alloc(tmem_slot, args.tmem_cols);
    fence_proxy_async_smem();   // the scale atom of ones
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (C > 1) cluster_arrive();   // peers may write here once every CTA's barriers are set
    const uint32_t tbase = *tmem_slot;
    const uint32_t sf_base = tbase + 2 * 8 * Tp, sfb = sf_base + 16 * S;
    if (warp == 0 && lane == 0) {
        // the first stages' codes, while the kernel before this one finishes
        int n = 0;
        for (int tile = cl; tile < a.tiles && n < S; tile += ncl)
            for (int kt = 0; kt < KT && n < S; kt++, n++) {
                tma_prefetch_2d(&map0, k0 / 2 + kt * 128, tile * TR);
                if (GATED) tma_prefetch_2d(&map1, k0 / 2 + kt * 128, tile * TR);
            }
    } else if (warp >= 8) {
        const int r = threadIdx.x - 256, which = GATED ? r >> 6 : 0, n = cl * TR + (GATED ? r & 63 : r);
        constexpr int BS = FMT == MOE_NVFP4 ? 16 : 32;
        if (n < a.N)
            for (int o = 0; o < min(a.K - k0, a.Kc) / BS; o += 128)
                prefetch_l2(a.m[which].scales + (size_t)n * (a.K / BS) + k0 / BS + o);
    }
    pdl_wait();
    // The next kernel may launch now.  Not before the wait: the decode FFN reads its bf16 x before it
    // waits for the kernel ahead of it, so that kernel may let it start only when every kernel before
    // is complete.  And not at all where this one's own y could be that x
    if (GATED || a.y_f32) pdl_trigger();

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, ph = 0;
            for (int tile = cl; tile < a.tiles; tile += ncl)
                for (int kt = 0; kt < KT; kt++) {
                    if (!mbar_wait(&empty[s], ph ^ 1, a.limit_ns)) atomicOr(a.status, 1 << 16);
                    mbar_arrive_expect_tx(&full[s], 16384);
                    uint8_t* dst = sm + L.codes + s * 16384;
                    const int c0 = k0 / 2 + kt * 128;
                    tma_load_2d(dst, &map0, c0, tile * TR, &full[s]);
                    if (GATED) tma_load_2d(dst + 8192, &map1, c0, tile * TR, &full[s]);
                    if (++s == S) { s = 0; ph ^= 1; }
                }
        }
        __syncwarp();
    } else {
        // block scales: thread r of warps 8-11 fetches row r's, a few stages ahead
        const int r = threadIdx.x & 127, which_r = GATED ? r >> 6 : 0;
        constexpr int BS = FMT == MOE_NVFP4 ? 16 : 32, per = kLinKT / BS;
        const int pitch = a.K / BS;
        const uint8_t* base = a.m[which_r].scales + k0 / BS;
        const int have = min(a.K - k0, a.Kc) / BS;       // scales of this CTA's part of a row
        const int total = ((a.tiles - cl + ncl - 1) / ncl) * KT;
        int f_it = 0, f_kt = 0, f_n = cl * TR + (GATED ? r & 63 : r);      // the next stage to fetch
        const int N = a.N;
        const bool wide = a.wide_scales;
        auto fetch = [&](auto w) -> uint4 {
            const bool in = f_it < total && f_n < N;
            const int o = f_kt * per;
            const uint4 v = load_scales<FMT, decltype(w)::value>(base + (in ? (size_t)f_n * pitch + o : 0), in ? have - o : 0);
            f_it++;
            if (++f_kt == KT) {
                f_kt = 0;
                f_n += ncl * TR;
            }
            return v;
        };
        uint4 q[4];
        if (warp >= 8 && wide) {
#pragma unroll
            for (int i = 0; i < 4; i++) q[i] = fetch(std::true_type());
        }
        __syncwarp();
        if (warp < 8 || nprep == 11) {
            // digits of x: items are (token, 256 elements), 8 elements per lane.  An item's 1 KiB of
            // digits first holds its elements as loaded; the same warp turns them into digits once
            // the tokens' largest elements are known.  Short loops, not unrolled copies: a CTA runs
            // this once, at the speed at which it can fetch the instructions
            const int pw = warp - 1, tp_inv = a.tp_inv, K = a.K;
            const long long ldx = a.ldx;
            const char* x = static_cast<const char*>(a.x);
            uint8_t* digits = sm + L.digits;                  // item (t, kt) at (kt * Tp + t) KiB
            constexpr int batch = XF32 ? 2 : 4;
            for (int j0 = pw; j0 < items; j0 += batch * nprep) {
                X8<XF32> v[batch];
#pragma unroll
                for (int i = 0; i < batch; i++) {
                    const int j = j0 + i * nprep, kt = (j * tp_inv) >> 16;
                    const int t = j - kt * Tp, k = k0 + kt * kLinKT + lane * 8;
                    v[i].load(x + (t * ldx + k) * (XF32 ? 4 : 2), j < items && t < T && k < K);
                }
#pragma unroll
                for (int i = 0; i < batch; i++) {
                    const int j = j0 + i * nprep;
                    if (j >= items) break;
                    v[i].put(digits + j * 1024, lane);
                    uint32_t mx = 0;
#pragma unroll
                    for (int e = 0; e < 8; e++) mx = max(mx, v[i].bits(e) & 0x7FFFFFFFu);
                    mx = __reduce_max_sync(0xffffffffu, mx);
                    if (lane == 0) atomicMax(&xmax[j - ((j * tp_inv) >> 16) * Tp], mx);
                }
            }
            __syncwarp();
            named_sync(1, nprep * 32);
#pragma unroll 1
            for (int j = pw; j < items; j += nprep) {
                const int t = j - ((j * tp_inv) >> 16) * Tp;
                const uint32_t mx = xmax[t];
                // E: exponent of the largest element (subnormals as they are); 2^(21 - E) in two factors
                const int E = mx == 0 ? 0 : mx < 0x00800000u ? -118 - __clz(mx) : (int)(mx >> 23) - 127;
                const bool finite = mx < 0x7F800000u;
                const int up = 21 - E, h1 = up / 2, d1 = E / 2;
                const float f1 = exp2i(h1), f2 = exp2i(up - h1);
                uint8_t* dst = digits + j * 1024;
                X8<XF32> v;
                v.get(dst, lane);
                // rounded by adding 1.5 2^23, whose bits X then counts from
                uint32_t X[8];
#pragma unroll
                for (int e = 0; e < 8; e++)
                    X[e] = __float_as_uint(fmaf(__uint_as_float(v.bits(e)) * f1, f2, 12582912.0f)) - 0x4B400000u + 0x924924u;
                uint32_t row[8];
                digit_rows(X, row);
                __syncwarp();                                 // all lanes have their elements
                // rows 8 t + d of the K-major operand, 128-byte swizzle: 16-byte chunk c of row d at c ^ d
#pragma unroll
                for (int d = 0; d < 8; d++)
                    *reinterpret_cast<uint32_t*>(dst + d * 128 + (((lane >> 2) ^ d) << 4) + (lane & 3) * 4) = row[d];
                if (j < Tp && lane == 0) {
                    xscale[t] = finite ? exp2i(d1) : __uint_as_float(0x7FC00000u);
                    xscale[16 + t] = exp2i(E - d1);
                }
            }
            // (the MMA thread orders these stores before its reads: a proxy fence here would wait
            // for warps 8-11's loads of scales)
            __syncwarp();
            if (lane == 0) mbar_arrive(bready);
            __syncwarp();
        }
        const int R = (TR + C - 1) / C;                   // output rows per owner
        constexpr int NW = GATED ? 2 : 1;
        const int ldt = lin_row_words(Tp);
        const int buf_words = C * NW * R * ldt;           // [src][which][row - owner * R][t]
        float* exch = reinterpret_cast<float*>(sm + L.exch);
        __syncwarp();

        if (warp >= 8) {
            const uint32_t quarter = (uint32_t)(32 * (warp - 8)) << 16;
            int s = 0, ph = 0;
            auto stages = [&](auto w) {
                using W = decltype(w);
#pragma unroll 1
                for (int it0 = 0; it0 < total; it0 += 4) {
                    // two stages at a time: rows to shared memory, then every warp takes all of them for
                    // its quarter of TMEM's lanes: lane l, column 4 i + j holds step i's scales of row
                    // l + 32 j.  Two buffers, one barrier a pair: a buffer's readers are past the next one
#pragma unroll
                    for (int p = 0; p < 4; p += 2) {
                        const int n = min(2, total - it0 - p);
                        if (n <= 0) break;
                        uint8_t* buf = sm + L.scales + p * 2048;
                        if (!W::value) {
                            q[p] = fetch(w);
                            q[p + 1] = fetch(w);
                        }
                        *reinterpret_cast<uint4*>(buf + 16 * r) = q[p];
                        *reinterpret_cast<uint4*>(buf + 2048 + 16 * r) = q[p + 1];
                        if (W::value) {          // four stages ahead
                            q[p] = fetch(w);
                            q[p + 1] = fetch(w);
                        }
                        __syncwarp();
                        named_sync(2, 128);
                        // everything that can wait first, then the loads and stores of both stages in a row
                        const int s0 = s, s1 = s + 1 == S ? 0 : s + 1;
                        if (!mbar_wait(&empty[s0], ph ^ 1, a.limit_ns) && lane == 0) atomicOr(a.status, 1 << 16);
                        if (++s == S) { s = 0; ph ^= 1; }
                        if (n == 2) {
                            if (!mbar_wait(&empty[s1], ph ^ 1, a.limit_ns) && lane == 0) atomicOr(a.status, 1 << 16);
                            if (++s == S) { s = 0; ph ^= 1; }
                        }
                        __syncwarp();                // the lanes leave the waits one by one
                        tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < n; i++) {
                            uint32_t c[16];
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const uint4 u = *reinterpret_cast<const uint4*>(buf + 2048 * i + 16 * (lane + 32 * j));
                                const bool nv = FMT == MOE_NVFP4;
                                c[j] = nv ? u.x : u.x & 0xFFFFu;
                                c[4 + j] = nv ? u.y : u.x >> 16;
                                c[8 + j] = nv ? u.z : u.y & 0xFFFFu;
                                c[12 + j] = nv ? u.w : u.y >> 16;
                            }
                            tmem_st_32x16(sf_base + 16 * (i == 0 ? s0 : s1) + quarter, c);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane < n) mbar_arrive(&full[lane == 0 ? s0 : s1]);
                        __syncwarp();
                    }
                }
            };
            if (wide) stages(std::true_type());
            else stages(std::false_type());
        } else if (warp == 1) {
            if (lane == 0) {
                if (!mbar_wait(bready, 0, a.limit_ns)) atomicOr(a.status, 1 << 16);
                fence_proxy_async_smem();
                tc_fence_after();
                const uint32_t idesc = idesc_fp4(128, 8 * Tp, FMT == MOE_MXFP4);
                tmem_cp_sf_atom(sfb, smem_desc(sm + L.ones, 16, 128, 0));
                const uint64_t ad0 = smem_desc(sm + L.codes, 16, 1024, 2), bd0 = smem_desc(sm + L.digits, 16, 1024, 2);
                int s = 0, ph = 0, tc = 0;
                for (int tile = cl; tile < a.tiles; tile += ncl, tc++) {
                    const int b = tc & 1;
                    if (!mbar_wait(&acce[b], ((tc >> 1) & 1) ^ 1, a.limit_ns)) atomicOr(a.status, 1 << 16);
                    const uint32_t acc = tbase + b * 8 * Tp;
                    for (int kt = 0; kt < KT; kt++) {
                        if (!mbar_wait(&full[s], ph, a.limit_ns)) atomicOr(a.status, 1 << 16);
                        tc_fence_after();
                        const uint32_t sfa = sf_base + 16 * s;
                        const uint64_t ad = ad0 + s * (16384 >> 4), bd = bd0 + (uint64_t)(kt * Tp * (1024 >> 4));
                        const int ns = steps - 4 * kt;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const uint32_t accum = (kt > 0 || i > 0) ? 1u : 0u;
                            if (i >= ns) break;
                            if (FMT == MOE_NVFP4) mma_nvfp4(acc, ad + 2 * i, bd + 2 * i, idesc, sfa + 4 * i, sfb, accum);
                            else mma_mxfp4(acc, ad + 2 * i, bd + 2 * i, idesc, sfa + 4 * i, sfb, accum);
                        }
                        tc_commit(&empty[s]);
                        if (++s == S) { s = 0; ph ^= 1; }
                    }
                    tc_commit(&accf[b]);
                }
            }
            __syncwarp();
        } else if (warp >= 4) {
            if (!mbar_wait(bready, 0, a.limit_ns) && lane == 0) atomicOr(a.status, 1 << 16);   // xscale
            const int e4 = warp - 4, row = 32 * e4 + lane;
            const int orow = GATED ? row & 63 : row, which = GATED ? row >> 6 : 0;
            const int owner = orow / R;
            const float ts = a.m[which].ts;
            const int at = ((rank * NW + which) * R + orow - owner * R) * ldt;
            const uint32_t dst = map_rank(smem_addr(exch), owner) + 4 * at;
            const uint32_t dst_bar = map_rank(smem_addr(exf), owner);
            __syncwarp();
            if (C > 1) cluster_wait();                        // peers' barriers are set
            int tc = 0;
            for (int tile = cl; tile < a.tiles; tile += ncl, tc++) {
                const int b = tc & 1, ph = (tc >> 1) & 1;
                if (!mbar_wait(&exe[b], ph ^ 1, a.limit_ns) && lane == 0) atomicOr(a.status, 1 << 16);
                if (!mbar_wait(&accf[b], ph, a.limit_ns) && lane == 0) atomicOr(a.status, 1 << 16);
                __syncwarp();
                tc_fence_after();
                const uint32_t acc = tbase + b * 8 * Tp + ((uint32_t)(32 * e4) << 16);
#pragma unroll 1
                for (int t0 = 0; t0 < Tp; t0 += 4) {
                    uint32_t d[4][8];
                    const bool four = Tp - t0 >= 4;
                    tmem_ld_32x8(acc + 8 * t0, d[0]);
                    tmem_ld_32x8(acc + 8 * t0 + 8, d[1]);
                    if (four) {
                        tmem_ld_32x8(acc + 8 * t0 + 16, d[2]);
                        tmem_ld_32x8(acc + 8 * t0 + 24, d[3]);
                    }
                    tmem_ld_wait();
                    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < 4; h++) {
                        if (h >= 2 && !four) break;
                        o[h] = __uint_as_float(d[h][0]);
#pragma unroll
                        for (int g = 1; g < 8; g++) o[h] = fmaf(o[h], 0.125f, __uint_as_float(d[h][g]));
                        o[h] = o[h] * ts * xscale[t0 + h] * xscale[16 + t0 + h];
                    }
                    if (C > 1) st_async_f32x4(dst + 4 * (b * buf_words + t0), o, dst_bar + 8 * b);
                    else *reinterpret_cast<float4*>(exch + b * buf_words + at + t0) = make_float4(o[0], o[1], o[2], o[3]);
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&acce[b]);
                    if (C == 1) mbar_arrive(&exf[b]);
                }
            }
            __syncwarp();
            if (C > 1) cluster_arrive_relaxed();
        } else {
            const int tid = threadIdx.x - 64;
            const uint32_t peer_exe = map_rank(smem_addr(exe), lane < C ? lane : 0);
            const int own0 = rank * R, nown = min(R, TR - own0);
            const int quads = (T + 3) / 4;                    // a thread sums one row of four tokens
            const uint32_t in_bytes = 16 * C * NW * nown * quads;
            const int src_words = NW * R * ldt;
            // (held in registers: the stores below would have them read again each time)
            const int N = a.N, tiles = a.tiles, r_inv = a.r_inv;
            const bool y_f32 = a.y_f32;
            const long long ldy = a.ldy, ld_add = a.ld_add;
            float* const yf = static_cast<float*>(a.y);
            __nv_bfloat16* const yh = static_cast<__nv_bfloat16*>(a.y);
            const float* const addf = static_cast<const float*>(a.add);
            const __nv_bfloat16* const addh = static_cast<const __nv_bfloat16*>(a.add);
            if (C > 1) cluster_wait();
            int tc = 0;
            for (int tile = cl; tile < tiles; tile += ncl, tc++) {
                const int b = tc & 1;
                if (C > 1 && tid == 0) mbar_arrive_expect_tx(&exf[b], in_bytes);
                if (!mbar_wait_cluster(&exf[b], (tc >> 1) & 1, a.limit_ns) && lane == 0) atomicOr(a.status, 1 << 16);
                __syncwarp();
                if (C > 1 && tile + ncl >= tiles) cluster_arrive_relaxed();   // no more access to peers from here
#pragma unroll 1
                for (int j = tid; j < quads * R; j += kLinSumThreads) {
                    const int g = (j * r_inv) >> 16, o = j - g * R, n = tile * TR + own0 + o;
                    if (o >= nown || n >= N) continue;
                    const float* in = exch + b * buf_words + o * ldt + 4 * g;
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
                    for (int c = 0; c < C; c++, in += src_words) {
                        const float4 p = *reinterpret_cast<const float4*>(in);
                        y[0] += p.x; y[1] += p.y; y[2] += p.z; y[3] += p.w;
                        if (GATED) {
                            const float4 q = *reinterpret_cast<const float4*>(in + R * ldt);
                            u[0] += q.x; u[1] += q.y; u[2] += q.z; u[3] += q.w;
                        }
                    }
                    if (GATED) {
#pragma unroll
                        for (int h = 0; h < 4; h++) y[h] = y[h] / (1.0f + expf(-y[h])) * u[h];
                    }
                    const int nt = min(4, T - 4 * g);
                    const long long at = 4 * g * ldy + n;
                    if (addf) {
                        const long long from = 4 * g * ld_add + n;
#pragma unroll
                        for (int h = 0; h < 4; h++)
                            if (h < nt) y[h] += y_f32 ? addf[from + h * ld_add] : __bfloat162float(addh[from + h * ld_add]);
                    }
#pragma unroll
                    for (int h = 0; h < 4; h++)
                        if (h < nt) {
                            if (y_f32) yf[at + h * ldy] = y[h];
                            else yh[at + h * ldy] = __float2bfloat16_rn(y[h]);
                        }
                }
                __syncwarp();
                // the buffer may be written again, if another tile will use it
                if (tile + 2 * ncl < tiles) {
                    if (C > 1) {
                        if (lane < C) mbar_arrive_cluster(peer_exe + 8 * b);
                    } else if (lane == 0) {
                        mbar_arrive(&exe[b]);
                    }
                }
            }
            __syncwarp();
        }
    }
    // No CTA of a cluster ends while a peer may still write to it.  Warps 4-7 arrived after
    // their last store to a peer, warps 2-3 after their last wait
    if (C > 1) {
        __syncwarp();
        if (warp < 2 || warp >= 8) {
            cluster_wait();
            cluster_arrive_relaxed();
        }
        cluster_wait();
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, a.tmem_cols);
    }
}

// ---------------------------------------------------------------- host

static int check_weight(const moe_fp4_weight* w) {
    if (!w || !w->codes || !w->scales) return fail(MOE_EINVAL, "fp4 weight: null pointer");
    if (w->fmt != MOE_MXFP4 && w->fmt != MOE_NVFP4) return fail(MOE_EINVAL, "fp4 weight: unknown format");
    if (w->N <= 0 || w->K <= 0 || w->K % 32) return fail(MOE_EINVAL, "fp4 weight: need N > 0 and K a positive multiple of 32");
    if (w->N > (1 << 30)) return fail(MOE_EINVAL, "fp4 weight: N too large");
    if (reinterpret_cast<uintptr_t>(w->codes) & 15) return fail(MOE_EINVAL, "fp4 weight: codes must be 16-byte aligned");
    return MOE_OK;
}

// The digits of x, 4 bytes an element of a token pair's columns, fill at most 128 KiB of each of a
// cluster's 8 CTAs, and up to a stage of every token more where K does not divide evenly.
static int check_tokens(int T, int K) {
    if (T <= 0 || T > kMaxDecodeT) return fail(MOE_EINVAL, "fp4: T must be in [1, 16]");
    const long long Tp = (T + 1) & ~1;
    if (Tp * ((K + (kLinKT - 1LL)) / kLinKT * kLinKT) > 262144)
        return fail(MOE_EINVAL, "fp4: K too large for this many tokens (K * T, T rounded up to even, at most 262144)");
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

// Do the rows of two matrices share any byte?  (Strides are at least a row's length.)
static bool rows_overlap(const void* a, int a_type, long long lda, int na, const void* b, int b_type, long long ldb, int nb,
                         int T) {
    const int sa = a_type == MOE_BF16 ? 2 : 4, sb = b_type == MOE_BF16 ? 2 : 4;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const uintptr_t wa = uintptr_t(na) * sa, wb = uintptr_t(nb) * sb;
    const uintptr_t pa = uintptr_t(lda) * sa, pb = uintptr_t(ldb) * sb;
    if (a0 + (T - 1) * pa + wa <= b0 || b0 + (T - 1) * pb + wb <= a0) return false;
    for (int i = 0; i < T; i++)
        for (int j = 0; j < T; j++)
            if (a0 + i * pa < b0 + j * pb + wb && b0 + j * pb < a0 + i * pa + wa) return true;
    return false;
}

struct LinDevice {
    int sms = 0;
    int smem = 0;                              // dynamic shared memory a block may take
    int sm_smem = 0, reserved = 0;             // shared memory of an SM, and what each block takes besides
    int clusters[8][kLinMaxCluster + 1] = {};  // co-resident clusters per kernel and cluster size
};

static std::mutex g_lin_mu;   // guards the entries below while they are filled

template <int FMT, int GATED, int XF32>
static int launch_variant(LinArgs& a, const CUtensorMap& m0, const CUtensorMap& m1, LinDevice& d, cudaStream_t s) {
    auto kern = fp4_linear_kernel<FMT, GATED, XF32>;
    const int Tp = (a.T + 1) & ~1, KTall = (a.K + kLinKT - 1) / kLinKT;
    a.tiles = (a.N + (GATED ? 63 : 127)) / (GATED ? 64 : 128);
    int* active = d.clusters[FMT * 4 + GATED * 2 + XF32];
    std::unique_lock<std::mutex> lock(g_lin_mu);
    if (!active[1]) {
        MOE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem));
        for (int C = kLinMaxCluster; C >= 1; C--) {
            cudaLaunchConfig_t lc = {};
            lc.gridDim = dim3(C);
            lc.blockDim = dim3(kLinThreads);
            lc.dynamicSmemBytes = d.smem;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = C;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            lc.attrs = at;
            lc.numAttrs = 1;
            int n = 0;
            MOE_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n, kern, &lc));
            active[C] = n < 1 ? 1 : n;
        }
    }
    lock.unlock();
    // Cluster size: the least of, in twentieths of a stage's 0.4 us, the stages of the busiest
    // CTA, the conversion of its part of x (0.15 a KiB of digits) and the exchange of each tile
    // (0.3).  Measured against the stages alone: 4096 x 4096 for 16 tokens 9.5 us, not 10.9; an
    // exchange of 0.5 has one CTA a tile at 131072 x 4096 for one token: 56.4 us, not 51.3.  Over
    // 200 sizes the choice is 1.1 % above the best C on average, 11 % at most.
    // At most 128 KiB of digits, so that four stages fit beside them; only where no cluster does with
    // that, up to a stage of every token more (140 KiB at most: three stages fit)
    int bestC = 0;
    long long best = 0;
    for (int cap = 128 * 1024; !bestC && cap <= 128 * 1024 + 4 * Tp * kLinKT; cap += 4 * Tp * kLinKT)
        for (int C = 1; C <= kLinMaxCluster && C <= KTall; C++) {
            const int kt = (KTall + C - 1) / C;
            if ((KTall + kt - 1) / kt != C) continue;   // a CTA without work
            if (4 * Tp * kt * kLinKT > cap) continue;
            const int ncl = std::min(a.tiles, active[C]), rounds = (a.tiles + ncl - 1) / ncl;
            const long long cost = 20LL * rounds * kt + 3 * Tp * kt + 6 * rounds;
            if (!bestC || cost < best) { best = cost; bestC = C; }
        }
    if (!bestC) return fail(MOE_EINVAL, "fp4: K too large for this many tokens");
    a.C = bestC;
    const int kt = (KTall + a.C - 1) / a.C;
    a.Kc = kt * kLinKT;
    const int ncl = std::min(a.tiles, active[a.C]);
    const long long total = (long long)((a.tiles + ncl - 1) / ncl) * kt;
    a.stages = (int)std::min<long long>(kLinMaxStages, total);
    while (a.stages > 1 && LinSmem(a.stages, Tp, a.Kc, a.C, GATED).total + 1024 > d.smem) a.stages--;
    int smem = LinSmem(a.stages, Tp, a.Kc, a.C, GATED).total + 1024;
    if (smem > d.smem) return fail(MOE_EINVAL, "fp4: K too large for this many tokens");
    if (a.stages == 1 && total > 1) return fail(MOE_EINVAL, "fp4: K too large for this many tokens");
    const int R = ((GATED ? 64 : 128) + a.C - 1) / a.C;
    a.tp_inv = (65536 + Tp - 1) / Tp;
    a.r_inv = (65536 + R - 1) / R;
    const int cols = 2 * 8 * Tp + 16 * a.stages + 4;
    a.tmem_cols = 32;
    while ((int)a.tmem_cols < cols) a.tmem_cols *= 2;
    // A block takes as large a share of the SM's shared memory as of its 512 TMEM columns, so that
    // blocks which are on an SM together all have their columns: else clusters of two calls
    // (on two streams) could each hold columns that a block of the other waits for
    smem = std::max(smem, (int)((long long)d.sm_smem * a.tmem_cols / 512) - d.reserved);

    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(ncl * a.C);
    lc.blockDim = dim3(kLinThreads);
    lc.dynamicSmemBytes = smem;
    lc.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = a.C;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    lc.attrs = at;
    lc.numAttrs = a.C > 1 ? 2 : 1;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&lc, kern, m0, m1, (const LinArgs)a));
    return MOE_OK;
}

static LinDevice* lin_device(int& rc) {
    static LinDevice devs[64];
    int dev = -1;
    rc = MOE_OK;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) { rc = cuda_fail(e, "cudaGetDevice"); return nullptr; }
    if (dev < 0 || dev >= 64) { rc = fail(MOE_EINVAL, "fp4: device ordinal out of range"); return nullptr; }
    LinDevice& d = devs[dev];
    std::lock_guard<std::mutex> lock(g_lin_mu);
    if (!d.sms) {
        int smem = 0, sms = 0;
        if ((e = cudaDeviceGetAttribute(&d.sm_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&d.reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) {
            rc = cuda_fail(e, "cudaDeviceGetAttribute");
            return nullptr;
        }
        d.smem = smem;
        d.sms = sms;
    }
    return &d;
}

static int launch_linear(LinArgs& a, const moe_fp4_weight* w0, const moe_fp4_weight* w1, cudaStream_t s) {
    int rc;
    LinDevice* d = lin_device(rc);
    if (!d) return rc;
    const int bs = w0->fmt == MOE_NVFP4 ? 16 : 32;
    const moe_fp4_weight* w[2] = {w0, w1};
    CUtensorMap maps[2];
    a.N = w0->N;
    a.K = w0->K;
    a.limit_ns = 2000000000ull;
    uintptr_t low = (uintptr_t)(a.K / bs);
    for (int i = 0; i < (w1 ? 2 : 1); i++) {
        a.m[i] = LinMat{w[i]->scales, w[i]->fmt == MOE_NVFP4 ? w[i]->tensor_scale : 1.0f};
        low |= reinterpret_cast<uintptr_t>(w[i]->scales);
        if ((rc = make_tmap_2d(&maps[i], w[i]->codes, a.K / 2, a.N, a.K / 2, 128, w1 ? 64 : 128, true))) return rc;
    }
    if (!w1) maps[1] = maps[0];
    a.wide_scales = low % (w0->fmt == MOE_NVFP4 ? 16 : 8) == 0;
    const int v = (w0->fmt == MOE_NVFP4 ? 4 : 0) + (w1 ? 2 : 0) + (a.x_f32 ? 1 : 0);
    switch (v) {
        case 0: return launch_variant<MOE_MXFP4, 0, 0>(a, maps[0], maps[1], *d, s);
        case 1: return launch_variant<MOE_MXFP4, 0, 1>(a, maps[0], maps[1], *d, s);
        case 2: return launch_variant<MOE_MXFP4, 1, 0>(a, maps[0], maps[1], *d, s);
        case 3: return launch_variant<MOE_MXFP4, 1, 1>(a, maps[0], maps[1], *d, s);
        case 4: return launch_variant<MOE_NVFP4, 0, 0>(a, maps[0], maps[1], *d, s);
        case 5: return launch_variant<MOE_NVFP4, 0, 1>(a, maps[0], maps[1], *d, s);
        case 6: return launch_variant<MOE_NVFP4, 1, 0>(a, maps[0], maps[1], *d, s);
        default: return launch_variant<MOE_NVFP4, 1, 1>(a, maps[0], maps[1], *d, s);
    }
}

// Load the kernels now (module loading may wait for the device).
int preload_fp4_linear_kernels() {
    cudaFuncAttributes fa;
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_MXFP4, 0, 0>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_MXFP4, 0, 1>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_MXFP4, 1, 0>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_MXFP4, 1, 1>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_NVFP4, 0, 0>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_NVFP4, 0, 1>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_NVFP4, 1, 0>));
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, fp4_linear_kernel<MOE_NVFP4, 1, 1>));
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_fp4_linear(const moe_fp4_weight* w, const void* x, int x_type, long long ldx, int T, const void* add,
                              long long ld_add, void* y, int y_type, long long ldy, int* status, void* stream) {
    int rc = check_weight(w);
    if (rc) return rc;
    if ((rc = check_tokens(T, w->K))) return rc;
    if (!status) return fail(MOE_EINVAL, "fp4 linear: null status");
    if ((rc = check_rows(x, x_type, ldx, w->K, T, "x"))) return rc;
    if ((rc = check_rows(y, y_type, ldy, w->N, T, "y"))) return rc;
    if (add && (rc = check_rows(add, y_type, ld_add, w->N, T, "add"))) return rc;
    if ((reinterpret_cast<uintptr_t>(x) & 15) || (T > 1 && (ldx * (x_type == MOE_BF16 ? 2 : 4)) % 16))
        return fail(MOE_EINVAL, "fp4 linear: rows of x must be 16-byte aligned");
    if (rows_overlap(x, x_type, ldx, w->K, y, y_type, ldy, w->N, T))
        return fail(MOE_EINVAL, "fp4 linear: y overlaps x");
    if (add && !(add == y && (ld_add == ldy || T == 1)) && rows_overlap(add, y_type, ld_add, w->N, y, y_type, ldy, w->N, T))
        return fail(MOE_EINVAL, "fp4 linear: y overlaps add (it may only be add itself)");
    LinArgs a{};
    a.T = T;
    a.x = x; a.x_f32 = x_type == MOE_F32; a.ldx = ldx;
    a.add = add; a.ld_add = ld_add;
    a.y = y; a.y_f32 = y_type == MOE_F32; a.ldy = ldy;
    a.status = status;
    return launch_linear(a, w, nullptr, (cudaStream_t)stream);
}

extern "C" int moe_fp4_swiglu(const moe_fp4_weight* gate, const moe_fp4_weight* up, const void* x, int x_type,
                              long long ldx, int T, float* h, long long ldh, int* status, void* stream) {
    int rc = check_weight(gate);
    if (rc || (rc = check_weight(up))) return rc;
    if (gate->N != up->N || gate->K != up->K || gate->fmt != up->fmt)
        return fail(MOE_EINVAL, "fp4 swiglu: gate and up must have one shape and format");
    if ((rc = check_tokens(T, gate->K))) return rc;
    if (!status) return fail(MOE_EINVAL, "fp4 swiglu: null status");
    if ((rc = check_rows(x, x_type, ldx, gate->K, T, "x"))) return rc;
    if ((rc = check_rows(h, MOE_F32, ldh, gate->N, T, "h"))) return rc;
    if ((reinterpret_cast<uintptr_t>(x) & 15) || (T > 1 && (ldx * (x_type == MOE_BF16 ? 2 : 4)) % 16))
        return fail(MOE_EINVAL, "fp4 swiglu: rows of x must be 16-byte aligned");
    if (rows_overlap(x, x_type, ldx, gate->K, h, MOE_F32, ldh, gate->N, T))
        return fail(MOE_EINVAL, "fp4 swiglu: h overlaps x");
    LinArgs a{};
    a.T = T;
    a.x = x; a.x_f32 = x_type == MOE_F32; a.ldx = ldx;
    a.y = h; a.y_f32 = 1; a.ldy = ldh;
    a.status = status;
    return launch_linear(a, gate, up, (cudaStream_t)stream);
}
