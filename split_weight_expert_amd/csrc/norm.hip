// Residual addition + RMS norm (dwdp_add_rmsnorm) and the layer boundary (dwdp_combine_add_rmsnorm):
//   z = the row's sum, r = 1 / sqrt(mean(z^2) + eps), n = z r weight
// written as sum_out = z, y = n and / or E4M3 codes of n with one scale per 128 columns.  Everything is
// fp32 until the one rounding of each output.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/dwdp_layer.h"
#include "common.h"
#include "internal.h"

namespace dwdp {
namespace {

constexpr int kMaxK = 64;

struct NormArgs {
    // z's source
    const uint8_t* x;                 // add: [T,H]; combine: y_perm
    const uint8_t* residual;          // or null
    const int32_t* inv_perm;          // combine
    const float* topk_w;
    int k, shared;
    // the rest
    int64_t T;
    int H;
    const uint8_t* weight;            // or null (combine without y and q)
    bool w_bf16;
    float eps;
    uint8_t* sum_out;                 // each or null
    uint8_t* y;
    uint8_t* q;
    float* q_scale;
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// Sum over LANES (16, 32 or 64) lanes, the same in each of them: exchanges inside rows of 16 lanes, then swaps of
// rows and of halves.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
    auto add = [&](uint32_t o) { v += __uint_as_float(o); };
    add(dpp<0xB1>(__float_as_uint(v)));        // lanes 1 apart
    add(dpp<0x4E>(__float_as_uint(v)));        // 2 apart
    add(dpp<0x141>(__float_as_uint(v)));       // mirrored in 8
    add(dpp<0x140>(__float_as_uint(v)));       // mirrored in 16
    if constexpr (LANES >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (LANES == 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return v;
}

// Eight consecutive elements are read and written together.  EVEN: rows of a multiple of 8 elements at 16-byte
// aligned addresses; else addresses are aligned to the element only, which the hardware's 16-byte accesses allow,
// and the last vector of a row has fewer valid elements, taken one by one.
typedef uint32_t raw_even __attribute__((ext_vector_type(4)));
typedef uint32_t raw_odd __attribute__((ext_vector_type(4), aligned(2)));

template <bool BF16>
struct Raw {
    raw_even r[BF16 ? 1 : 2];         // eight elements as they are in memory
};

template <bool BF16, bool EVEN>
__device__ __forceinline__ Raw<BF16> load_raw(const uint8_t* p, int64_t i, int valid = 8) {
    Raw<BF16> x;
    p += i * (BF16 ? 2 : 4);
    if (EVEN) {
        x.r[0] = *reinterpret_cast<const raw_even*>(p);
        if constexpr (!BF16) x.r[1] = *reinterpret_cast<const raw_even*>(p + 16);
    } else if (valid >= 8) {
        x.r[0] = *reinterpret_cast<const raw_odd*>(p);
        if constexpr (!BF16) x.r[1] = *reinterpret_cast<const raw_odd*>(p + 16);
    } else {
        uint32_t e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < 7; ++u)
            if (u < valid) e[u] = BF16 ? reinterpret_cast<const uint16_t*>(p)[u] : reinterpret_cast<const uint32_t*>(p)[u];
        if constexpr (BF16) {
            x.r[0] = raw_even{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
        } else {
            x.r[0] = raw_even{e[0], e[1], e[2], e[3]};
            x.r[1] = raw_even{e[4], e[5], e[6], e[7]};
        }
    }
    return x;
}

// Elements that this launch reads once.
template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_stream(const uint8_t* p) {
    Raw<BF16> x;
    x.r[0] = __builtin_nontemporal_load(reinterpret_cast<const raw_even*>(p));
    if constexpr (!BF16) x.r[1] = __builtin_nontemporal_load(reinterpret_cast<const raw_even*>(p + 16));
    return x;
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16>& x, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
            v[2 * j] = __uint_as_float(x.r[0][j] << 16);
            v[2 * j + 1] = __uint_as_float(x.r[0][j] & 0xffff0000u);
        } else {
            v[j] = __uint_as_float(x.r[0][j]);
            v[4 + j] = __uint_as_float(x.r[1][j]);
        }
    }
}

template <bool BF16, bool EVEN>
__device__ __forceinline__ void store8(uint8_t* p, int64_t i, int valid, const float* v) {
    p += i * (BF16 ? 2 : 4);
    if (EVEN || valid >= 8) {
        using V = typename std::conditional<EVEN, raw_even, raw_odd>::type;
        if constexpr (BF16) {
            *reinterpret_cast<V*>(p) = V{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
        } else {
            *reinterpret_cast<V*>(p) =
                V{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
            *reinterpret_cast<V*>(p + 16) =
                V{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
        }
    } else {
#pragma unroll
        for (int u = 0; u < 7; ++u)
            if (u < valid) {
                if (BF16) reinterpret_cast<uint16_t*>(p)[u] = (uint16_t)bf16x2(v[u], v[u]);
                else reinterpret_cast<float*>(p)[u] = v[u];
            }
    }
}

// Writes one vector of a row: z is its sum, r the row's factor.  With q the 16 lanes of a 128-column group
// call it together.
template <bool BF16, bool EVEN>
__device__ __forceinline__ void finish8(const NormArgs& a, int64_t t, int col, const float* z, float r) {
    const int64_t i = t * a.H + col;
    const int valid = a.H - col;
    if (a.sum_out != nullptr) store8<BF16, EVEN>(a.sum_out, i, valid, z);
    if (a.y == nullptr && a.q == nullptr) return;
    float n[8];
    if (a.w_bf16) unpack<true>(load_raw<true, EVEN>(a.weight, col, valid), n);
    else unpack<false>(load_raw<false, EVEN>(a.weight, col, valid), n);
#pragma unroll
    for (int u = 0; u < 8; ++u) n[u] = z[u] * r * n[u];
    if (a.y != nullptr) store8<BF16, EVEN>(a.y, i, valid, n);
    if constexpr (BF16 && EVEN) {
        if (a.q != nullptr) {
            // the largest magnitude as an integer maximum of the bit patterns, which keeps a NaN
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(n[u]) & 0x7fffffffu);
            m = max(m, dpp<0xB1>(m));
            m = max(m, dpp<0x4E>(m));
            m = max(m, dpp<0x141>(m));
            m = max(m, dpp<0x140>(m));
            // no scale below the smallest normal number: a subnormal one is too coarse to divide by
            const uint32_t sb = max(__float_as_uint(__uint_as_float(m) / 448.0f), 0x00800000u);
            const float s = m == 0 ? 1.0f : __uint_as_float(sb);
            const uint32_t lo = e4m3x4(n[0] / s, n[1] / s, n[2] / s, n[3] / s);
            const uint32_t hi = e4m3x4(n[4] / s, n[5] / s, n[6] / s, n[7] / s);
            *reinterpret_cast<uint2*>(a.q + i) = uint2{lo, hi};
            if ((threadIdx.x & 15) == 0) a.q_scale[i / kFp8Group] = s;
        }
    }
}

// One vector of z = combine + residual, for the two-pass kernel.
template <bool COMBINE, bool BF16, bool EVEN>
__device__ __forceinline__ void load_z(const NormArgs& a, int64_t t, int col, const int32_t* rows, const float* wts,
                                       float* z) {
    const int64_t i = t * a.H + col;
    const int valid = a.H - col;
    float v[8];
    if constexpr (COMBINE) {
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] = 0.0f;
        for (int j = 0; j < a.k + a.shared; ++j) {
            const int64_t row = j < a.k ? (int64_t)rows[j] : a.T * a.k + t;
            if (row < 0) continue;
            const float w = j < a.k ? wts[j] : 1.0f;
            unpack<BF16>(load_raw<BF16, EVEN>(a.x, row * a.H + col), v);
#pragma unroll
            for (int u = 0; u < 8; ++u) z[u] += w * v[u];
        }
    } else {
        unpack<BF16>(load_raw<BF16, EVEN>(a.x, i, valid), z);
    }
    if (a.residual != nullptr) {
        unpack<BF16>(load_raw<BF16, EVEN>(a.residual, i, valid), v);
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] += v[u];
    }
}

// Rows too wide for the registers (above 32768 elements; combine above 16384): one workgroup per row, which reads z
// twice (for the sum of squares, then to write), each element by the same thread, so that outputs may take their
// inputs' place.  Columns are counted without a sign: the step past the last one of a row of nearly 2^31 elements is
// still a number that lies behind the row.  A thread adds H / 2048 vectors: in fp32 the sum of like terms
// was off by 3e-4 at 2^25 elements and by 9% at 2^31.
template <bool COMBINE, bool BF16, bool EVEN>
__global__ __launch_bounds__(256) void norm_two_pass_kernel(NormArgs a) {
    __shared__ int32_t s_row[kMaxK];
    __shared__ float s_w[kMaxK];
    __shared__ float s_part[4];
    const int tid = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        __syncthreads();                               // the previous row's reads of the LDS arrays are done
        if (COMBINE && tid < a.k) {
            const int32_t p = a.inv_perm[t * a.k + tid];
            s_row[tid] = p >= 0 && p < a.T * (a.k + a.shared) ? p : -1;
            s_w[tid] = a.topk_w[t * a.k + tid];
        }
        __syncthreads();
        double sum = 0.0;                              // a vector's squares in fp32, the vectors in fp64
        float z[8];
        for (uint32_t c = tid * 8; c < (uint32_t)a.H; c += 256 * 8) {
            load_z<COMBINE, BF16, EVEN>(a, t, c, s_row, s_w, z);
            float squares = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) squares += z[u] * z[u];
            sum += (double)squares;
        }
        float ss = row_sum<64>((float)sum);
        if ((tid & 63) == 0) s_part[tid >> 6] = ss;
        __syncthreads();
        ss = (s_part[0] + s_part[1]) + (s_part[2] + s_part[3]);
        const float r = 1.0f / sqrtf(ss / (float)a.H + a.eps);
        for (uint32_t c = tid * 8; c < (uint32_t)a.H; c += 256 * 8) {
            load_z<COMBINE, BF16, EVEN>(a, t, c, s_row, s_w, z);
            finish8<BF16, EVEN>(a, t, c, z, r);
        }
    }
}

// ------------------------------------------------------------------------------ rows held in registers
// A thread keeps C vectors of its row (vector c of thread i: c * blockDim.x + i) as fp32 from the one read of
// the inputs to the one write of the outputs.  blockDim.x threads share a row, LANES of them in one wave; rows of
// one wave or less need no LDS and are packed blockDim.y to a workgroup.  Loads past the row's end read its
// last vector instead (combine) or nothing, so that every lane of a wave stays active up to the sum.
//
// Bound by HBM: each input is read and each output written once (counted).  7168-wide bf16 rows, residual, sum, y and
// codes: 16384 rows are 1061 MB in 184 us, 5.8 TB/s; combine of 8192 rows, k = 8 and a shared row, 1470 MB in 271 us,
// 5.4 TB/s (a plain copy reaches 4.9); fp32 rows, sum and y: 4096 tokens 1409 MB in 298 us, 4.7 TB/s.  A few rows are
// bound by latency: one row 3.8 us, of which an empty kernel takes 2.3.  Reading the rows twice (norm_two_pass_kernel) took 241 us and 495 us.
template <bool COMBINE, bool BF16, bool EVEN, int C, int LANES>
__global__ __launch_bounds__(1024) void norm_row_kernel(NormArgs a) {
    static_assert(!COMBINE || EVEN, "combine takes rows of a multiple of 8");
    __shared__ float s_part[16];
    const int tx = threadIdx.x, bx = LANES < 64 ? LANES : blockDim.x, lane = tx & 63;
    const int n_waves = LANES < 64 ? 1 : bx >> 6;
    // a row of whole waves has a number that is the same in all lanes: kept in scalar registers
    const int y = LANES == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.y) : threadIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * blockDim.y + y, stride = (int64_t)gridDim.x * blockDim.y;
    for (int64_t t = t0; t < a.T; t += stride) {
        float z[C][8];
        if constexpr (COMBINE) {
            const int64_t rows = a.T * (a.k + a.shared);
            const int nsrc = a.k + a.shared;
            // rows of a whole wave: lane j holds slot j's row and weight (k <= 64); rows out of range are dropped
            int my_row = -1;
            float my_w = 0.0f;
            if (LANES == 64 && lane < a.k) {
                my_row = a.inv_perm[t * a.k + lane];
                my_w = a.topk_w[t * a.k + lane];
                if (my_row >= rows) my_row = -1;
            }
            const int shared_row = (int)(a.T * a.k + t);
            auto row_of = [&](int j) {
                if (j >= a.k) return shared_row;
                if (LANES == 64) return (int)__builtin_amdgcn_readlane(my_row, j);
                const int r = a.inv_perm[t * a.k + j];
                return r < rows ? r : -1;
            };
            auto weight_of = [&](int j) {
                if (j >= a.k) return 1.0f;
                return LANES == 64 ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_w), j)) : a.topk_w[t * a.k + j];
            };
            // source rows whose loads are in flight together: k = 8 and a shared row are one batch of bf16
            // rows, in the registers of five fp32 ones
            constexpr int B = BF16 ? 10 : 5;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = min((c * bx + tx) * 8, a.H - 8);
#pragma unroll
                for (int u = 0; u < 8; ++u) z[c][u] = 0.0f;
                for (int j0 = 0; j0 < nsrc; j0 += B) {
                    // all loads of the batch first (a dropped slot loads row 0 and is skipped below) ...
                    Raw<BF16> raw[B];
#pragma unroll
                    for (int u = 0; u < B; ++u)
                        if (j0 + u < nsrc) {
                            const int r = row_of(j0 + u);
                            const uint8_t* const base = a.x + (int64_t)(r >= 0 ? r : 0) * a.H * (BF16 ? 2 : 4);
                            raw[u] = load_stream<BF16>(base + (uint32_t)col * (BF16 ? 2u : 4u));
                        }
                    // ... then the sums, in slot order
#pragma unroll
                    for (int u = 0; u < B; ++u) {
                        const int j = j0 + u;
                        if (j >= nsrc || row_of(j) < 0) continue;
                        const float w = weight_of(j);
                        float v[8];
                        unpack<BF16>(raw[u], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[c][i] += w * v[i];
                    }
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (c * bx + tx) * 8;
#pragma unroll
                for (int u = 0; u < 8; ++u) z[c][u] = 0.0f;
                if (col < a.H) unpack<BF16>(load_raw<BF16, EVEN>(a.x, t * a.H + col, a.H - col), z[c]);
            }
        }
        if (a.residual != nullptr) {
            Raw<BF16> res[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (c * bx + tx) * 8;
                if (col < a.H) res[c] = load_raw<BF16, EVEN>(a.residual, t * a.H + col, a.H - col);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float v[8];
                unpack<BF16>(res[c], v);
#pragma unroll
                for (int u = 0; u < 8; ++u) z[c][u] += v[u];
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool in = (c * bx + tx) * 8 < a.H;
#pragma unroll
            for (int u = 0; u < 8; ++u) ss += in ? z[c][u] * z[c][u] : 0.0f;
        }
        ss = row_sum<LANES>(ss);
        if (n_waves > 1) {
            if (lane == 0) s_part[tx >> 6] = ss;
            __syncthreads();
            ss = 0.0f;
            for (int i = 0; i < n_waves; ++i) ss += s_part[i];
            __syncthreads();                          // read before the next row's sums
        }
        const float r = 1.0f / sqrtf(ss / (float)a.H + a.eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * bx + tx) * 8;
            if (col < a.H) finish8<BF16, EVEN>(a, t, col, z[c], r);
        }
    }
}

template <bool COMBINE, bool BF16, bool EVEN, int C, int LANES>
void launch_rows(const NormArgs& a, int threads, hipStream_t st) {
    const int rows = threads <= 64 ? 256 / threads : 1;
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + rows - 1) / rows, kMaxRowGrid);
    hipLaunchKernelGGL((norm_row_kernel<COMBINE, BF16, EVEN, C, LANES>), dim3(grid), dim3(threads, rows), 0, st, a);
}

template <bool COMBINE, bool BF16, bool EVEN>
void launch_typed(const NormArgs& a, hipStream_t st) {
    const int64_t nvec = ((int64_t)a.H + 7) / 8;
    auto threads = [&](int c) { return (int)(((nvec + c - 1) / c + 63) / 64 * 64); };
    // One vector a thread as long as all rows' waves find a place on the chip at once (16 on each of 256 compute
    // units), two beyond: combine of 7168-wide rows, k = 8 and a shared row: 256 tokens 9.6 against 10.6 us,
    // 512 tokens 21.1 against 18.4; 2048-wide: 1024 tokens 10.2 against 11.7, 4096 37.5 against 40.4 (norm alone:
    // 15.4 against 14.7).
    const bool few = a.T * (threads(1) / 64) <= 4096;
    if (nvec <= 16) {
        launch_rows<COMBINE, BF16, EVEN, 1, 16>(a, 16, st);
    } else if (nvec <= 32) {
        launch_rows<COMBINE, BF16, EVEN, 1, 32>(a, 32, st);
    } else if (nvec <= 64 || (few && nvec <= 1024)) {
        launch_rows<COMBINE, BF16, EVEN, 1, 64>(a, threads(1), st);
    } else if (nvec <= 2 * 1024) {
        launch_rows<COMBINE, BF16, EVEN, 2, 64>(a, threads(2), st);
    } else {
        // wider rows: four vectors a thread, unless combine's source rows in flight need the registers
        if constexpr (!COMBINE) {
            if (nvec <= 4 * 1024) return launch_rows<false, BF16, EVEN, 4, 64>(a, threads(4), st);
        }
        const dim3 grid((unsigned)std::min<int64_t>(a.T, kMaxRowGrid));
        hipLaunchKernelGGL((norm_two_pass_kernel<COMBINE, BF16, EVEN>), grid, dim3(256), 0, st, a);
    }
}

// Outputs against every other buffer; sum_out and y may take the place of a row input (x of add, residual).
bool outputs_are_apart(const NormArgs& a, size_t eb, bool combine) {
    const size_t rows = (size_t)a.T * a.H, slots = (size_t)a.T * a.k * 4;
    const Span outs[] = {{a.sum_out, rows * eb}, {a.y, rows * eb}, {a.q, rows}, {a.q_scale, rows / kFp8Group * 4}};
    const Span fixed[] = {{a.weight, (size_t)a.H * (a.w_bf16 ? 2 : 4)}, {a.inv_perm, slots}, {a.topk_w, slots},
                          {combine ? a.x : nullptr, rows * eb * (a.k + a.shared)}};
    if (overlap_any(outs, 4, fixed, 4)) return false;
    const Span in_place[] = {{combine ? nullptr : a.x, rows * eb}, {a.residual, rows * eb}};
    for (int i = 0; i < 4; ++i)
        for (const Span& in : in_place)
            if (overlap(outs[i], in) && !(i < 2 && outs[i].p == in.p)) return false;
    return true;
}

template <bool COMBINE>
int launch_norm(const NormArgs& a, bool bf16, bool even, hipStream_t st) {
    if (even) {
        if (bf16) launch_typed<COMBINE, true, true>(a, st);
        else launch_typed<COMBINE, false, true>(a, st);
    } else if constexpr (!COMBINE) {
        if (bf16) launch_typed<false, true, false>(a, st);
        else launch_typed<false, false, false>(a, st);
    }
    DWDP_LAUNCHED();
    return DWDP_OK;
}

}  // namespace
}  // namespace dwdp

using namespace dwdp;

extern "C" int dwdp_add_rmsnorm(const void* x, const void* residual, int dtype, const void* weight, int w_dtype,
                                float eps, int64_t T, int H, void* sum_out, void* y, void* q, float* q_scale,
                                void* stream) {
    clear_error();
    DWDP_REQUIRE(dtype == DWDP_F32 || dtype == DWDP_BF16, "dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(w_dtype == DWDP_F32 || w_dtype == DWDP_BF16, "w_dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and not negative");
    DWDP_REQUIRE(T >= 0 && T < ((int64_t)1 << 31), "T out of range");
    DWDP_REQUIRE(H > 0, "H must be positive");
    DWDP_REQUIRE((q == nullptr) == (q_scale == nullptr), "q and q_scale are given together");
    if (q != nullptr) DWDP_REQUIRE(dtype == DWDP_BF16 && H % kFp8Group == 0, "q needs DWDP_BF16 and H % 128 == 0");
    if (T == 0) return DWDP_OK;
    DWDP_REQUIRE(x && weight, "x or weight is NULL");
    DWDP_REQUIRE(y || q, "one of y and q must be given");
    DWDP_REQUIRE(sum_out == nullptr || sum_out != y, "sum_out and y are the same buffer");
    const size_t eb = elem_bytes(dtype);
    DWDP_REQUIRE(type_aligned(x, eb) && type_aligned(residual, eb) && type_aligned(sum_out, eb) && type_aligned(y, eb) &&
                     type_aligned(weight, elem_bytes(w_dtype)) && type_aligned(q, 8) && type_aligned(q_scale, 4),
                 "a pointer is not aligned to its element type (q: 8 bytes)");
    const bool even = H % 8 == 0 && aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(sum_out) &&
                     aligned16(y);
    if (q != nullptr) DWDP_REQUIRE(even, "q needs 16-byte aligned x, residual, weight, sum_out and y");
    NormArgs a{};
    a.x = static_cast<const uint8_t*>(x);
    a.residual = static_cast<const uint8_t*>(residual);
    a.T = T;
    a.H = H;
    a.weight = static_cast<const uint8_t*>(weight);
    a.w_bf16 = w_dtype == DWDP_BF16;
    a.eps = eps;
    a.sum_out = static_cast<uint8_t*>(sum_out);
    a.y = static_cast<uint8_t*>(y);
    a.q = static_cast<uint8_t*>(q);
    a.q_scale = q_scale;
    DWDP_REQUIRE(outputs_are_apart(a, eb, false), "an output overlaps another buffer");
    return launch_norm<false>(a, dtype == DWDP_BF16, even, as_stream(stream));
}

extern "C" int dwdp_combine_add_rmsnorm(const void* y_perm, const int32_t* inv_perm, const float* topk_w, int64_t T,
                                        int k, int shared, int H, int dtype, const void* residual, const void* weight,
                                        int w_dtype, float eps, void* sum_out, void* y, void* q, float* q_scale,
                                        void* stream) {
    clear_error();
    DWDP_REQUIRE(dtype == DWDP_F32 || dtype == DWDP_BF16, "dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(w_dtype == DWDP_F32 || w_dtype == DWDP_BF16, "w_dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and not negative");
    DWDP_REQUIRE(k >= 1 && k <= kMaxK, "k must be in [1, 64]");
    DWDP_REQUIRE(shared == 0 || shared == 1, "shared must be 0 or 1");
    DWDP_REQUIRE(T >= 0 && T < ((int64_t)1 << 31) && T * (k + shared) < ((int64_t)1 << 31), "T out of range");
    DWDP_REQUIRE(H > 0 && H % 8 == 0, "H must be a positive multiple of 8");
    DWDP_REQUIRE((q == nullptr) == (q_scale == nullptr), "q and q_scale are given together");
    if (q != nullptr) DWDP_REQUIRE(dtype == DWDP_BF16 && H % kFp8Group == 0, "q needs DWDP_BF16 and H % 128 == 0");
    if (T == 0) return DWDP_OK;
    DWDP_REQUIRE(y_perm && inv_perm && topk_w, "null pointer argument");
    DWDP_REQUIRE(sum_out || y || q, "one of sum_out, y and q must be given");
    DWDP_REQUIRE(weight || (!y && !q), "y and q need weight");
    DWDP_REQUIRE(sum_out == nullptr || sum_out != y, "sum_out and y are the same buffer");
    DWDP_REQUIRE(y_perm != sum_out && y_perm != y && y_perm != q, "y_perm is an output");
    DWDP_REQUIRE(aligned16(y_perm) && aligned16(residual) && aligned16(weight) && aligned16(sum_out) && aligned16(y) &&
                     type_aligned(q, 8) && type_aligned(q_scale, 4) && type_aligned(inv_perm, 4) && type_aligned(topk_w, 4),
                 "y_perm, residual, weight, sum_out and y must be 16-byte aligned (q: 8 bytes)");
    NormArgs a{};
    a.x = static_cast<const uint8_t*>(y_perm);
    a.residual = static_cast<const uint8_t*>(residual);
    a.inv_perm = inv_perm;
    a.topk_w = topk_w;
    a.k = k;
    a.shared = shared;
    a.T = T;
    a.H = H;
    a.weight = static_cast<const uint8_t*>(weight);
    a.w_bf16 = w_dtype == DWDP_BF16;
    a.eps = eps;
    a.sum_out = static_cast<uint8_t*>(sum_out);
    a.y = static_cast<uint8_t*>(y);
    a.q = static_cast<uint8_t*>(q);
    a.q_scale = q_scale;
    DWDP_REQUIRE(outputs_are_apart(a, elem_bytes(dtype), true), "an output overlaps another buffer");
    return launch_norm<true>(a, dtype == DWDP_BF16, true, as_stream(stream));
}
