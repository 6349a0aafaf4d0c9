// The router product of dwdp_route_gate: logits = x w^T with the columns of K cut into slices, so that
// every batch fills the chip.  With one slice the logits are written (bias added); with more, each slice's
// partial sums go to part[slice][T][E] and the gate's kernel adds them, in slice order, as it reads them.
//
//   small products  router_few_kernel: 16 x 16 tiles, operands straight from global memory into the matrix
//                   instruction; bound by latency, and by the weights' bytes
//   the others      router_tile_kernel: BM x BN tiles, operands by DMA into an LDS ring; bound by the DMAs
//                   (bf16) or by the matrix cores (fp32)
#include <algorithm>

#include "common.h"
#include "internal.h"
#include "router.h"

namespace dwdp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct RouterArgs {
    const uint8_t* x;
    const uint8_t* w;
    const float* bias;                // or null
    int64_t T;
    int H, E, slices, m_tiles, n_tiles;
    float* out;                       // logits (one slice) or part
};

__device__ __forceinline__ void store_logit(const RouterArgs& a, int slice, int64_t t, int e, float v) {
    if (t >= a.T || e >= a.E) return;
    if (a.slices == 1) a.out[t * a.E + e] = v + (a.bias ? a.bias[e] : 0.0f);
    else a.out[(slice * a.T + t) * a.E + e] = v;
}

// One 16-token x 16-expert tile of one slice; the slice's K steps are split over the workgroup's waves and
// their partial tiles summed through LDS in wave order.  Operand lanes: row (or expert) l % 16 and 16 bytes at
// 16 (l / 16) of the step; a step is 64 bytes of a row.  bf16: one v_mfma_f32_16x16x32_bf16 a step; fp32: four
// v_mfma_f32_16x16x4_f32, each taking one of the four consecutive columns a lane holds, which is the same
// columns on both sides.  Result element r of lane l: token 4 (l / 16) + r, expert l % 16.
//
// Bound by latency: one token of 7168 bf16 columns against 256 experts takes 4.9 us for 3.7 MB of weights, 64
// tokens 6.8 us, of which an empty kernel takes 2.3; eight 64-byte steps of both operands are in flight a wave (four
// were as fast).  Eight waves share a tile's steps: with four, 64 tokens took 0.8 us longer, 16 were no faster.
constexpr int kFewWaves = 8;

template <bool BF16>
__global__ __launch_bounds__(kFewWaves * 64) void router_few_kernel(RouterArgs a) {
    __shared__ float part[kFewWaves][64][5];      // 5: consecutive lanes fall on different banks
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, q = lane >> 4;
    const int n = blockIdx.x % a.n_tiles, ms = blockIdx.x / a.n_tiles, slice = ms % a.slices;
    const int64_t m0 = (int64_t)(ms / a.slices) * 16;
    const int n0 = n * 16;
    const int64_t row_bytes = (int64_t)a.H * (BF16 ? 2 : 4);
    const uint8_t* xr = a.x + min(m0 + l16, a.T - 1) * row_bytes + q * 16;
    const uint8_t* wr = a.w + (int64_t)min(n0 + l16, a.E - 1) * row_bytes + q * 16;
    const int steps = (int)(row_bytes / 64);
    const int s0 = (int)((int64_t)slice * steps / a.slices), ns = (int)((int64_t)(slice + 1) * steps / a.slices) - s0;
    const int sb = s0 + wave * ns / kFewWaves, se = s0 + (wave + 1) * ns / kFewWaves;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int U = 8;                          // steps whose loads are in flight together
    for (int s = sb; s < se; s += U) {
        f32x4 xa[U], wa[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s + u < se) {
                xa[u] = *reinterpret_cast<const f32x4*>(xr + (int64_t)(s + u) * 64);
                wa[u] = *reinterpret_cast<const f32x4*>(wr + (int64_t)(s + u) * 64);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s + u < se) {
                if constexpr (BF16) {
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xa[u]),
                                                                  __builtin_bit_cast(bf16x8, wa[u]), acc, 0, 0, 0);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa[u][c], wa[u][c], acc, 0, 0, 0);
                }
            }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][lane][r] = acc[r];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float s = part[0][lane][r];
#pragma unroll
            for (int w = 1; w < kFewWaves; ++w) s += part[w][lane][r];
            store_logit(a, slice, m0 + q * 4 + r, n0 + l16, s);
        }
    }
}

// 16 bytes per lane from global memory to LDS, lane l at byte 16 l of `lds` (wave-uniform).
__device__ __forceinline__ void dma16(const uint8_t* g, uint8_t* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

__device__ __forceinline__ void ordered_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int PER, int MOST>
__device__ __forceinline__ void wait_steps(int steps) {   // at most `steps` (<= MOST) batches of PER loads outstanding
    if constexpr (MOST == 0) wait_vmcnt<0>();
    else if (steps >= MOST) wait_vmcnt<PER * MOST>();
    else wait_steps<PER, MOST - 1>(steps);
}

// One BM x BN tile of one slice.  WM x WN waves; a K step is 128 bytes of a row (64 bf16 columns, or 32 fp32 ones, of which
// a matrix instruction takes one of the four consecutive that a lane holds, the same on both sides), moved into LDS
// by 1 KB DMA instructions of 8 rows each, into a ring of NS slots with NS - 1 steps in flight.  The slot of step
// k + NS - 1 is the one step k - 1 read, so it is filled after step k's barrier, and its DMAs are issued between
// the step's products: issued in one go they hold up the wave, and with it the products, for as long as the
// address unit takes them.  16-byte chunk c of row r sits in slot c ^ ((r / 2) % 8) of its row, so that 16
// consecutive rows read at one chunk spread over all banks (counted: no bank conflict).
//
// 8192 x 7168 tokens and 256 experts (128 x 256 tiles, 4 slices): 42 us, 709 TFLOP/s; it reads 125 MB from HBM, every
// token once, and 350 MB through the DMAs, which alone take 35 us, and keeps the matrix cores busy for 27% of
// the time.  So what bounds it is the DMAs' way from L2 to LDS, with one workgroup's barrier per step; with the DMAs
// issued together before the products it took 54.7 us.  Not faster: larger tiles for fewer bytes (256 x 128, tokens
// straight into registers: 74.6 us with the gate, against 58.9), smaller ones for two workgroups per compute unit (15%
// slower), four waves of larger tiles (45 and 47 us), 16 waves (the same).  fp32: 8192 x 7168 and 256 experts, 64 x 64 tiles,
// about 250 us, 120 TFLOP/s, three quarters of the fp32 matrix rate of 157.
template <bool BF16, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(WM * WN * 64) void router_tile_kernel(RouterArgs a) {
    constexpr int NW = WM * WN, ROWB = 128, STAGE = (BM + BN) * ROWB, P = NS - 1;
    constexpr int TM = BM / WM, TN = BN / WN, MI = TM / 32, NJ = TN / 32;
    constexpr int PER = (BM + BN) / 8 / NW;       // DMA instructions per wave and step
    static_assert((BM + BN) / 8 % NW == 0 && PER * P < 64, "rows split evenly over the waves");
    static_assert(NS * STAGE <= 163840, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[NS * STAGE];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, l32 = lane & 31, hi = lane >> 5;
    // Workgroup b runs on XCD b % 8.  Each XCD takes a run of consecutive tiles, token tiles innermost, so that
    // the weights it multiplies by (one slice, nearly always) stay in its L2.
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles * a.slices, per_xcd = (tiles + kNumXcd - 1) / kNumXcd;
    const int64_t lin = blockIdx.x % kNumXcd * per_xcd + blockIdx.x / kNumXcd;
    if (blockIdx.x / kNumXcd >= per_xcd || lin >= tiles) return;
    const int m = (int)(lin % a.m_tiles), n = (int)(lin / a.m_tiles % a.n_tiles), slice = (int)(lin / a.m_tiles / a.n_tiles);
    const int64_t m0 = (int64_t)m * BM;
    const int n0 = n * BN;
    const int64_t row_bytes = (int64_t)a.H * (BF16 ? 2 : 4);
    const int steps = (int)(row_bytes / ROWB);
    const int kb = (int)((int64_t)slice * steps / a.slices), KT = (int)((int64_t)(slice + 1) * steps / a.slices) - kb;

    const uint8_t* g[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = (wave * PER + i) * 8 + lane / 8;    // row of the stage: BM token rows, then BN expert rows
        const int c = (lane & 7) ^ ((r >> 1) & 7);
        g[i] = (r < BM ? a.x + min(m0 + r, a.T - 1) * row_bytes : a.w + min(n0 + r - BM, a.E - 1) * row_bytes) +
               (int64_t)kb * ROWB + c * 16;
    }
    auto issue = [&](int kt, int i) {
        dma16(g[i] + (int64_t)kt * ROWB, ring + kt % NS * STAGE + (wave * PER + i) * 1024);
    };
    auto frag = [&](const uint8_t* s, int row, int chunk) {
        return *reinterpret_cast<const f32x4*>(s + row * ROWB + ((chunk ^ ((row >> 1) & 7)) << 4));
    };
    f32x16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    for (int k = 0; k < P && k < KT; ++k)
#pragma unroll
        for (int i = 0; i < PER; ++i) issue(k, i);
    for (int kt = 0; kt < KT; ++kt) {
        // this wave's DMAs of step kt have landed once at most those of the later issued steps are out
        wait_steps<PER, P - 1>(min(P - 1, KT - 1 - kt));
        ordered_barrier();                        // every wave's step kt landed; step kt-1's slot is free
        const uint8_t* A = ring + kt % NS * STAGE;
        const uint8_t* B = A + BM * ROWB;
        const bool more = kt + P < KT;
        f32x4 af[4][MI], bf[4][NJ];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int i = 0; i < MI; ++i) af[s][i] = frag(A, wm * TM + i * 32 + l32, 2 * s + hi);
#pragma unroll
            for (int j = 0; j < NJ; ++j) bf[s][j] = frag(B, wn * TN + j * 32 + l32, 2 * s + hi);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    if constexpr (BF16) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, af[s][i]),
                                                                            __builtin_bit_cast(bf16x8, bf[s][j]),
                                                                            acc[i][j], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(af[s][i][c], bf[s][j][c], acc[i][j], 0, 0, 0);
                    }
                }
            __builtin_amdgcn_sched_barrier(0);
            if (more)
#pragma unroll
                for (int i = PER * s / 4; i < PER * (s + 1) / 4; ++i) issue(kt + P, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        // the fragments are in registers before any wave passes the next barrier
        __builtin_amdgcn_s_waitcnt(0xC07F);       // lgkmcnt(0); vmcnt and expcnt not waited on
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                store_logit(a, slice, m0 + wm * TM + i * 32 + (r >> 2) * 8 + hi * 4 + (r & 3), n0 + wn * TN + j * 32 + l32,
                            acc[i][j][r]);
}

template <bool BF16, int BM, int BN, int WM, int WN, int NS>
void launch_tile(const RouterArgs& a, hipStream_t st) {
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles * a.slices;
    const unsigned grid = (unsigned)((tiles + kNumXcd - 1) / kNumXcd * kNumXcd);
    hipLaunchKernelGGL((router_tile_kernel<BF16, BM, BN, WM, WN, NS>), dim3(grid), dim3(WM * WN * 64), 0, st, a);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Measured, product and gate together in a graph, other inputs in between (us):
//   16 x 16 tiles or 64 x 64: each 16 x 16 tile reads 32 rows, so it is the bytes of a row times the tiles that decide.
//     bf16  0.9 MB (64 tokens x 7168, 256 experts) 12.6 and 14.3, 1.1 MB (80 tokens) 13.6 and 14.9, 1.4 MB (96) 15.5 and
//           14.6, 1.8 MB (1777 x 1984, 60 experts) 15.0 and 12.6
//     fp32  0.9 MB (200 x 1024, 256 experts) 11.9 and 13.6, 1.8 MB (64 x 7168) 17.0 and 29.1, 4.2 MB (512 x 1024, 512
//           experts) 26.3 and 17.8, 235 MB (8192 x 7168, 256 experts) 883 and 279
//   wider tiles, bf16, 7168 columns, 256 experts: 1024 tokens 64 x 64 19.2, 64 x 256 21.7; 2048: 25.4 and 25.8; 4096: 45.6 and
//     36.6; 4096: 64 x 256 36.6, 128 x 256 40.1; 8192: 64.5 and 58.5.  fp32 is bound by its matrix instructions on any tile.
// Slices: as many as give the chip's 256 compute units a tile each (two of the 64 x 64 ones), but few enough that the
// gate's reading of them costs less than they save: for 16 x 16 tiles at most 4 (8: 16 tokens x 5376, 452 experts
// 16.9 against 14.8), of 16 K steps at least; else 8, of 8 K steps at least (4: 567 x 2176, 226 experts 14.9 against 13.5).
RouterPlan plan_router(int64_t T, int H, int E, int dtype) {
    RouterPlan p{};
    const bool bf16 = dtype == DWDP_BF16;
    const int64_t t64 = ceil_div(T, 64), row_bytes = (int64_t)H * (bf16 ? 2 : 4);
    int64_t want = 256;
    // fp32 rows need not be a multiple of the wider tiles' 128-byte K step
    if (ceil_div(T, 16) * ceil_div(E, 16) * row_bytes <= (bf16 ? 5 << 18 : 2 << 20) || row_bytes % 128 != 0) {
        p.bm = p.bn = 16;
    } else if (!bf16 || E <= 64 || t64 * ceil_div(E, 64) <= 128) {
        p.bm = p.bn = 64;
        want = 512;
    } else if (E <= 128) {
        p.bm = 64;
        p.bn = 128;
    } else {
        p.bm = t64 * ceil_div(E, 256) >= 128 ? 128 : 64;
        p.bn = 256;
    }
    const int64_t tiles = ceil_div(T, p.bm) * ceil_div(E, p.bn);
    const int64_t most = p.bm == 16 ? std::min<int64_t>(4, row_bytes / 64 / 16) : std::min<int64_t>(8, row_bytes / 128 / 8);
    // slices * tiles <= want, so the slices' sums are at most want * bm * bn numbers: 32 MiB with the widest tiles
    p.slices = (int)std::max<int64_t>(1, std::min(want / tiles, most));
    return p;
}

bool router_fits(int64_t T, int E, const RouterPlan& p) {
    const int64_t tiles = ceil_div(T, p.bm) * ceil_div(E, p.bn) * p.slices;
    return (tiles + kNumXcd) * 512 <= kMaxLaunchItems;
}

int router_split(const void* x, const void* w, int dtype, const float* bias, int64_t T, int H, int E, const RouterPlan& p,
                 float* logits, float* part, hipStream_t st) {
    RouterArgs a{};
    a.x = static_cast<const uint8_t*>(x);
    a.w = static_cast<const uint8_t*>(w);
    a.bias = bias;
    a.T = T;
    a.H = H;
    a.E = E;
    a.slices = p.slices;
    a.m_tiles = (int)ceil_div(T, p.bm);
    a.n_tiles = (int)ceil_div(E, p.bn);
    a.out = p.slices == 1 ? logits : part;
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles * a.slices;
    if (p.bm == 16) {
        const dim3 grid((unsigned)tiles), block(kFewWaves * 64);
        if (dtype == DWDP_BF16) hipLaunchKernelGGL(router_few_kernel<true>, grid, block, 0, st, a);
        else hipLaunchKernelGGL(router_few_kernel<false>, grid, block, 0, st, a);
    } else if (p.bm == 128) {
        launch_tile<true, 128, 256, 2, 4, 3>(a, st);
    } else if (p.bn == 256) {
        launch_tile<true, 64, 256, 2, 4, 4>(a, st);
    } else if (p.bn == 128) {
        launch_tile<true, 64, 128, 2, 2, 3>(a, st);
    } else if (dtype == DWDP_BF16) {
        launch_tile<true, 64, 64, 2, 2, 4>(a, st);
    } else {
        launch_tile<false, 64, 64, 2, 2, 4>(a, st);
    }
    DWDP_LAUNCHED();
    return DWDP_OK;
}

}  // namespace dwdp
