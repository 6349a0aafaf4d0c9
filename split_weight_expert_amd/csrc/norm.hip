// Residual addition + RMS norm (dwdp_add_rmsnorm) and the layer boundary (dwdp_combine_add_rmsnorm):
//   z = the row's sum, r = 1 / sqrt(mean(z^2) + eps), n = z r weight
// written as sum_out = z, y = n and / or E4M3 codes of n with one scale per 128 columns.  Everything is
// fp32 until the one rounding of each output.
//
// The forms with a branch (dwdp_branch_add_rmsnorm, dwdp_combine_branch_add_rmsnorm) put the block's own norm, gates
// and scales between its output u and the residual,
//   z = residual_scale residual + scale token_gate gate (u / sqrt(mean(u^2) + eps_b) norm),
// and may write int8 codes of n with one scale per row.
#include <algorithm>
#include <cmath>

#include "../../include/dwdp_layer.h"
#include "common.h"
#include "internal.h"
#include "rows.h"

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
    // the block's branch (the kernels' BRANCH forms)
    const uint8_t* norm;              // or null
    const uint8_t* gate;              // or null
    const float* token_gate;          // or null
    bool norm_bf16, gate_bf16, q_int8;
    float norm_eps, scale, residual_scale;
};

// One vector of a per-column array (a norm's weight, a gate).
template <bool EVEN>
__device__ __forceinline__ void load_columns(const uint8_t* p, bool bf16, int col, int valid, float* v) {
    if (bf16) unpack<true>(load_raw<true, EVEN>(p, col, valid), v);
    else unpack<false>(load_raw<false, EVEN>(p, col, valid), v);
}

// What the branch makes of one vector of the block's output, without the residual: r is the factor of its norm, f that
// of the row (scale and token gate).
template <bool EVEN>
__device__ __forceinline__ void branch8(const NormArgs& a, int col, float* z, float r, float f) {
    const int valid = a.H - col;
    float v[8];
    if (a.norm != nullptr) {
        load_columns<EVEN>(a.norm, a.norm_bf16, col, valid, v);
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] = z[u] * r * v[u];
    }
    if (a.gate != nullptr) {
        load_columns<EVEN>(a.gate, a.gate_bf16, col, valid, v);
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] *= v[u];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) z[u] *= f;
}

__device__ __forceinline__ float branch_factor(const NormArgs& a, int64_t t) {
    return a.token_gate != nullptr ? a.scale * a.token_gate[t] : a.scale;
}

// Writes the sum z of one vector of a row and turns it into its norm, which it writes to y; returns the largest
// magnitude's bit pattern.
template <bool BF16, bool EVEN>
__device__ __forceinline__ uint32_t norm8(const NormArgs& a, int64_t t, int col, float* z, float r) {
    const int64_t i = t * a.H + col;
    const int valid = a.H - col;
    if (a.sum_out != nullptr) store8<BF16, EVEN>(a.sum_out, i, valid, z);
    float n[8];
    load_columns<EVEN>(a.weight, a.w_bf16, col, valid, n);
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        z[u] = z[u] * r * n[u];
        m = max(m, __float_as_uint(z[u]) & 0x7fffffffu);
    }
    if (a.y != nullptr) store8<BF16, EVEN>(a.y, i, valid, z);
    return m;
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
    load_columns<EVEN>(a.weight, a.w_bf16, col, valid, n);
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

// One vector of z = combine + residual, for the two-pass kernel; with a branch u alone (RES false), or z.
template <bool COMBINE, bool BRANCH, bool BF16, bool EVEN, bool RES = true>
__device__ __forceinline__ void load_z(const NormArgs& a, int64_t t, int col, const int32_t* rows, const float* wts,
                                       float* z, float r = 1.0f, float f = 1.0f) {
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
    if constexpr (!RES) return;
    if constexpr (BRANCH) branch8<EVEN>(a, col, z, r, f);
    if (a.residual != nullptr) {
        unpack<BF16>(load_raw<BF16, EVEN>(a.residual, i, valid), v);
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] += BRANCH ? a.residual_scale * v[u] : v[u];
    }
}

// Rows too wide for the registers (above 32768 elements; combine above 16384): one workgroup per row, which reads z
// twice (for the sum of squares, then to write), each element by the same thread, so that outputs may take their
// inputs' place.  Columns are counted without a sign: the step past the last one of a row of nearly 2^31 elements is
// still a number that lies behind the row.  A thread adds H / 2048 vectors: in fp32 the sum of like terms
// was off by 3e-4 at 2^25 elements and by 9% at 2^31.  A branch's norm takes one more pass, and so do int8 codes: combine of
// 1024 rows of 20480 bf16, k = 8 and a shared row, 201 us without a branch, 279 with its norm, 368 with codes too; 1024
// dense rows of 40960 85, 102 and 135.
template <bool COMBINE, bool BRANCH, bool BF16, bool EVEN>
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
        // the factor of a norm over the row's vectors as `load` gives them
        auto factor = [&](float eps, auto load) {
            double sum = 0.0;                          // a vector's squares in fp32, the vectors in fp64
            float z[8];
            for (uint32_t c = tid * 8; c < (uint32_t)a.H; c += 256 * 8) {
                load(c, z);
                float squares = 0.0f;
#pragma unroll
                for (int u = 0; u < 8; ++u) squares += z[u] * z[u];
                sum += (double)squares;
            }
            float ss = row_sum<64>((float)sum);
            if ((tid & 63) == 0) s_part[tid >> 6] = ss;
            __syncthreads();
            ss = (s_part[0] + s_part[1]) + (s_part[2] + s_part[3]);
            return 1.0f / sqrtf(ss / (float)a.H + eps);
        };
        float ru = 1.0f, f = 1.0f;
        if constexpr (BRANCH) {
            f = branch_factor(a, t);
            if (a.norm != nullptr) {
                ru = factor(a.norm_eps, [&](uint32_t c, float* z) {
                    load_z<COMBINE, true, BF16, EVEN, false>(a, t, c, s_row, s_w, z);
                });
                __syncthreads();                       // read before the next sums
            }
        }
        auto load = [&](uint32_t c, float* z) { load_z<COMBINE, BRANCH, BF16, EVEN>(a, t, c, s_row, s_w, z, ru, f); };
        const float r = factor(a.eps, load);
        float z[8];
        if constexpr (BRANCH && EVEN) {
            if (a.q_int8) {
                // the inputs may be overwritten only by the last pass
                uint32_t m = 0;
                for (uint32_t c = tid * 8; c < (uint32_t)a.H; c += 256 * 8) {
                    load(c, z);
                    NormArgs none = a;
                    none.sum_out = none.y = nullptr;
                    m = max(m, norm8<BF16, EVEN>(none, t, c, z, r));
                }
                m = row_max<64>(m);
                __syncthreads();
                if ((tid & 63) == 0) s_part[tid >> 6] = __uint_as_float(m);
                __syncthreads();
                for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(s_part[i]));
                const Int8Scale s = int8_scale(m);
                for (uint32_t c = tid * 8; c < (uint32_t)a.H; c += 256 * 8) {
                    load(c, z);
                    norm8<BF16, EVEN>(a, t, c, z, r);
                    *reinterpret_cast<uint2*>(a.q + t * a.H + c) = int8x8<false>(z, s);
                }
                if (tid == 0) a.q_scale[t] = s.scale;
                continue;
            }
        }
        for (uint32_t c = tid * 8; c < (uint32_t)a.H; c += 256 * 8) {
            load(c, z);
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
// With a branch the row is reduced twice (three times with int8 codes) and its columns read two or three more arrays,
// which stay in L2: still one read and one write of each row.  7168-wide bf16, sum and y: 16384 rows of a dense branch 940 MB in
// 180 us, 5.2 TB/s (with int8 codes 1057 MB in 209); combine of 8192, k = 8 and a shared row, with codes, 1470 MB in 279 us,
// 5.3 TB/s; one row 6.7 us, 64 rows 7.3.  Reading the columns ahead of the reductions did not help (7.0 and 7.5).
// Dense branches of four vectors a thread spill 36 bytes a lane (fp32, or bf16 rows that are not EVEN) or 100 (such fp32
// rows): 4096 rows of 20001 bf16 236 us, 176 without a branch.
template <bool COMBINE, bool BRANCH, bool BF16, bool EVEN, int C, int LANES>
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
        auto factor = [&](float eps) {                // of a norm over z
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
                __syncthreads();                      // read before the next sums
            }
            return 1.0f / sqrtf(ss / (float)a.H + eps);
        };
        if (BRANCH || a.residual != nullptr) {
            Raw<BF16> res[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (c * bx + tx) * 8;
                if (BRANCH) res[c] = Raw<BF16>{};
                if (col < a.H && (!BRANCH || a.residual != nullptr))
                    res[c] = load_raw<BF16, EVEN>(a.residual, t * a.H + col, a.H - col);
            }
            if constexpr (BRANCH) {
                const float f = branch_factor(a, t);
                const float ru = a.norm != nullptr ? factor(a.norm_eps) : 1.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int col = (c * bx + tx) * 8;
                    if (col < a.H) branch8<EVEN>(a, col, z[c], ru, f);
                }
            }
            if (!BRANCH || a.residual != nullptr) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float v[8];
                    unpack<BF16>(res[c], v);
#pragma unroll
                    for (int u = 0; u < 8; ++u) z[c][u] += BRANCH ? a.residual_scale * v[u] : v[u];
                }
            }
        }
        const float r = factor(a.eps);
        if constexpr (BRANCH && EVEN) {
            if (a.q_int8) {
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int col = (c * bx + tx) * 8;
                    if (col < a.H) m = max(m, norm8<BF16, EVEN>(a, t, col, z[c], r));
                }
                m = row_max<LANES>(m);
                if (n_waves > 1) {
                    if (lane == 0) s_part[tx >> 6] = __uint_as_float(m);
                    __syncthreads();
                    for (int i = 0; i < n_waves; ++i) m = max(m, __float_as_uint(s_part[i]));
                    __syncthreads();
                }
                const Int8Scale s = int8_scale(m);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int col = (c * bx + tx) * 8;
                    if (col < a.H) *reinterpret_cast<uint2*>(a.q + t * a.H + col) = int8x8<false>(z[c], s);
                }
                if (tx == 0) a.q_scale[t] = s.scale;
                continue;
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * bx + tx) * 8;
            if (col < a.H) finish8<BF16, EVEN>(a, t, col, z[c], r);
        }
    }
}

template <bool COMBINE, bool BRANCH, bool BF16, bool EVEN, int C, int LANES>
void launch_rows(const NormArgs& a, int threads, hipStream_t st) {
    const int rows = threads <= 64 ? 256 / threads : 1;
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + rows - 1) / rows, kMaxRowGrid);
    hipLaunchKernelGGL((norm_row_kernel<COMBINE, BRANCH, BF16, EVEN, C, LANES>), dim3(grid), dim3(threads, rows), 0, st, a);
}

template <bool COMBINE, bool BRANCH, bool BF16, bool EVEN>
void launch_typed(const NormArgs& a, hipStream_t st) {
    const int64_t nvec = ((int64_t)a.H + 7) / 8;
    auto threads = [&](int c) { return (int)(((nvec + c - 1) / c + 63) / 64 * 64); };
    // One vector a thread as long as all rows' waves find a place on the chip at once (16 on each of 256 compute
    // units), two beyond: combine of 7168-wide rows, k = 8 and a shared row: 256 tokens 9.6 against 10.6 us,
    // 512 tokens 21.1 against 18.4; 2048-wide: 1024 tokens 10.2 against 11.7, 4096 37.5 against 40.4 (norm alone:
    // 15.4 against 14.7).
    const bool few = a.T * (threads(1) / 64) <= 4096;
    if (nvec <= 16) {
        launch_rows<COMBINE, BRANCH, BF16, EVEN, 1, 16>(a, 16, st);
    } else if (nvec <= 32) {
        launch_rows<COMBINE, BRANCH, BF16, EVEN, 1, 32>(a, 32, st);
    } else if (nvec <= 64 || (few && nvec <= 1024)) {
        launch_rows<COMBINE, BRANCH, BF16, EVEN, 1, 64>(a, threads(1), st);
    } else if (nvec <= 2 * 1024) {
        launch_rows<COMBINE, BRANCH, BF16, EVEN, 2, 64>(a, threads(2), st);
    } else {
        // wider rows: four vectors a thread, unless combine's source rows in flight need the registers
        if constexpr (!COMBINE) {
            if (nvec <= 4 * 1024) return launch_rows<false, BRANCH, BF16, EVEN, 4, 64>(a, threads(4), st);
        }
        const dim3 grid((unsigned)std::min<int64_t>(a.T, kMaxRowGrid));
        hipLaunchKernelGGL((norm_two_pass_kernel<COMBINE, BRANCH, BF16, EVEN>), grid, dim3(256), 0, st, a);
    }
}

// Outputs against every other buffer; sum_out and y may take the place of a row input (x of add, residual).
bool outputs_are_apart(const NormArgs& a, size_t eb, bool combine) {
    const size_t rows = (size_t)a.T * a.H, slots = (size_t)a.T * a.k * 4;
    const Span outs[] = {{a.sum_out, rows * eb}, {a.y, rows * eb}, {a.q, rows},
                         {a.q_scale, (a.q_int8 ? (size_t)a.T : rows / kFp8Group) * 4}};
    const Span fixed[] = {{a.weight, (size_t)a.H * (a.w_bf16 ? 2 : 4)}, {a.inv_perm, slots}, {a.topk_w, slots},
                          {combine ? a.x : nullptr, rows * eb * (a.k + a.shared)},
                          {a.norm, (size_t)a.H * (a.norm_bf16 ? 2 : 4)}, {a.gate, (size_t)a.H * (a.gate_bf16 ? 2 : 4)},
                          {a.token_gate, (size_t)a.T * 4}};
    if (overlap_any(outs, 4, fixed, 7)) return false;
    const Span in_place[] = {{combine ? nullptr : a.x, rows * eb}, {a.residual, rows * eb}};
    for (int i = 0; i < 4; ++i)
        for (const Span& in : in_place)
            if (overlap(outs[i], in) && !(i < 2 && outs[i].p == in.p)) return false;
    return true;
}

template <bool COMBINE, bool BRANCH = false>
int launch_norm(const NormArgs& a, bool bf16, bool even, hipStream_t st) {
    if (even) {
        if (bf16) launch_typed<COMBINE, BRANCH, true, true>(a, st);
        else launch_typed<COMBINE, BRANCH, false, true>(a, st);
    } else if constexpr (!COMBINE) {
        if (bf16) launch_typed<false, BRANCH, true, false>(a, st);
        else launch_typed<false, BRANCH, false, false>(a, st);
    }
    DWDP_LAUNCHED();
    return DWDP_OK;
}

// The numbers of a branch and of the codes that both calls with one check, and where its arrays are.
int branch_args(const char* fn, const dwdp_branch* b, const float* token_gate, int dtype, int H, const void* q, int q_dtype,
                const float* q_scale, NormArgs* a) {
    auto bad = [&](const char* what) { return fail(DWDP_ERR_INVALID_ARG, std::string(fn) + ": " + what); };
    const dwdp_branch plain{nullptr, nullptr, DWDP_F32, DWDP_F32, 0.0f, 1.0f, 1.0f};
    if (b == nullptr) b = &plain;
    auto known = [](int d) { return d == DWDP_F32 || d == DWDP_BF16; };
    if (!known(b->norm_dtype) || !known(b->gate_dtype)) return bad("the branch's dtypes must be DWDP_F32 or DWDP_BF16");
    if (!std::isfinite(b->eps) || b->eps < 0.0f) return bad("the branch's eps must be finite and not negative");
    if (!std::isfinite(b->scale) || !std::isfinite(b->residual_scale)) return bad("the branch's scales must be finite");
    if ((q == nullptr) != (q_scale == nullptr)) return bad("q and q_scale are given together");
    if (q != nullptr) {
        if (q_dtype != DWDP_FP8_E4M3 && q_dtype != DWDP_INT8) return bad("q_dtype must be DWDP_FP8_E4M3 or DWDP_INT8");
        if (q_dtype == DWDP_FP8_E4M3 && (dtype != DWDP_BF16 || H % kFp8Group != 0))
            return bad("E4M3 codes need DWDP_BF16 and H % 128 == 0");
        if (H % 8 != 0) return bad("int8 codes need H % 8 == 0");
    }
    if (!type_aligned(b->norm, elem_bytes(b->norm_dtype)) || !type_aligned(b->gate, elem_bytes(b->gate_dtype)) ||
        !type_aligned(token_gate, 4))
        return bad("a pointer of the branch is not aligned to its element type");
    a->norm = static_cast<const uint8_t*>(b->norm);
    a->gate = static_cast<const uint8_t*>(b->gate);
    a->token_gate = token_gate;
    a->norm_bf16 = b->norm_dtype == DWDP_BF16;
    a->gate_bf16 = b->gate_dtype == DWDP_BF16;
    a->norm_eps = b->eps;
    a->scale = b->scale;
    a->residual_scale = b->residual_scale;
    a->q_int8 = q != nullptr && q_dtype == DWDP_INT8;
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

extern "C" int dwdp_branch_add_rmsnorm(const void* x, const void* residual, int dtype, const dwdp_branch* branch,
                                       const float* token_gate, const void* weight, int w_dtype, float eps, int64_t T,
                                       int H, void* sum_out, void* y, void* q, int q_dtype, float* q_scale,
                                       void* stream) {
    clear_error();
    DWDP_REQUIRE(dtype == DWDP_F32 || dtype == DWDP_BF16, "dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(w_dtype == DWDP_F32 || w_dtype == DWDP_BF16, "w_dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and not negative");
    DWDP_REQUIRE(T >= 0 && T < ((int64_t)1 << 31), "T out of range");
    DWDP_REQUIRE(H > 0, "H must be positive");
    NormArgs a{};
    const int rc = branch_args(__func__, branch, token_gate, dtype, H, q, q_dtype, q_scale, &a);
    if (rc != DWDP_OK) return rc;
    if (T == 0) return DWDP_OK;
    DWDP_REQUIRE(x != nullptr, "x is NULL");
    DWDP_REQUIRE(sum_out || y || q, "one of sum_out, y and q must be given");
    DWDP_REQUIRE(weight || (!y && !q), "y and q need weight");
    DWDP_REQUIRE(sum_out == nullptr || sum_out != y, "sum_out and y are the same buffer");
    const size_t eb = elem_bytes(dtype);
    DWDP_REQUIRE(type_aligned(x, eb) && type_aligned(residual, eb) && type_aligned(sum_out, eb) && type_aligned(y, eb) &&
                     type_aligned(weight, elem_bytes(w_dtype)) && type_aligned(q, 8) && type_aligned(q_scale, 4),
                 "a pointer is not aligned to its element type (q: 8 bytes)");
    const bool even = H % 8 == 0 && aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(sum_out) &&
                     aligned16(y) && aligned16(a.norm) && aligned16(a.gate);
    if (q != nullptr) DWDP_REQUIRE(even, "q needs 16-byte aligned x, residual, weight, sum_out, y and branch");
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
    return launch_norm<false, true>(a, dtype == DWDP_BF16, even, as_stream(stream));
}

extern "C" int dwdp_combine_branch_add_rmsnorm(const void* y_perm, const int32_t* inv_perm, const float* topk_w,
                                               int64_t T, int k, int shared, int H, int dtype, const void* residual,
                                               const dwdp_branch* branch, const float* token_gate, const void* weight,
                                               int w_dtype, float eps, void* sum_out, void* y, void* q, int q_dtype,
                                               float* q_scale, void* stream) {
    clear_error();
    DWDP_REQUIRE(dtype == DWDP_F32 || dtype == DWDP_BF16, "dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(w_dtype == DWDP_F32 || w_dtype == DWDP_BF16, "w_dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and not negative");
    DWDP_REQUIRE(k >= 1 && k <= kMaxK, "k must be in [1, 64]");
    DWDP_REQUIRE(shared == 0 || shared == 1, "shared must be 0 or 1");
    DWDP_REQUIRE(T >= 0 && T < ((int64_t)1 << 31) && T * (k + shared) < ((int64_t)1 << 31), "T out of range");
    DWDP_REQUIRE(H > 0 && H % 8 == 0, "H must be a positive multiple of 8");
    NormArgs a{};
    const int rc = branch_args(__func__, branch, token_gate, dtype, H, q, q_dtype, q_scale, &a);
    if (rc != DWDP_OK) return rc;
    if (T == 0) return DWDP_OK;
    DWDP_REQUIRE(y_perm && inv_perm && topk_w, "null pointer argument");
    DWDP_REQUIRE(sum_out || y || q, "one of sum_out, y and q must be given");
    DWDP_REQUIRE(weight || (!y && !q), "y and q need weight");
    DWDP_REQUIRE(sum_out == nullptr || sum_out != y, "sum_out and y are the same buffer");
    DWDP_REQUIRE(y_perm != sum_out && y_perm != y && y_perm != q, "y_perm is an output");
    DWDP_REQUIRE(aligned16(y_perm) && aligned16(residual) && aligned16(weight) && aligned16(sum_out) && aligned16(y) &&
                     aligned16(a.norm) && aligned16(a.gate) && type_aligned(q, 8) && type_aligned(q_scale, 4) &&
                     type_aligned(inv_perm, 4) && type_aligned(topk_w, 4),
                 "y_perm, residual, weight, sum_out, y and the branch must be 16-byte aligned (q: 8 bytes)");
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
    return launch_norm<true, true>(a, dtype == DWDP_BF16, true, as_stream(stream));
}
