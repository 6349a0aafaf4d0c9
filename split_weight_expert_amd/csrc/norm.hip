// Residual addition + RMS norm (dwdp_add_rmsnorm) and the layer boundary (dwdp_combine_add_rmsnorm):
//   z = the row's sum, r = 1 / sqrt(mean(z^2) + eps), n = z r weight
// written as sum_out = z, y = n and / or E4M3 codes of n with one scale per 128 columns.  Everything is
// fp32 until the one rounding of each output.
#include <algorithm>
#include <cmath>

#include "../../include/dwdp_layer.h"
#include "common.h"
#include "internal.h"

namespace dwdp {
namespace {

constexpr int kMaxK = 64;
constexpr int kFewRows = 512;
constexpr int kManyC = 2;

typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// VEC consecutive elements (8: 16-byte accesses; 1: element accesses) of a bf16 or fp32 array.
template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const uint8_t* p, int64_t i, float* v) {
    if constexpr (VEC == 1) {
        v[0] = BF16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
    } else if constexpr (BF16) {
        const uint4 r = *reinterpret_cast<const uint4*>(p + i * 2);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p + i * 4);
        const float4 b = *reinterpret_cast<const float4*>(p + i * 4 + 16);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

// 16 bytes that this launch reads once.
__device__ __forceinline__ float4 load_stream(const uint8_t* p) {
    const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    return float4{v[0], v[1], v[2], v[3]};
}

template <bool BF16>
__device__ __forceinline__ void unpack(const float4* raw, float* v) {
    const float f[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
    if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(__float_as_uint(f[j]) << 16);
            v[2 * j + 1] = __uint_as_float(__float_as_uint(f[j]) & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = f[j];
        v[4] = raw[1].x, v[5] = raw[1].y, v[6] = raw[1].z, v[7] = raw[1].w;
    }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(uint8_t* p, int64_t i, const float* v) {
    if constexpr (VEC == 1) {
        if (BF16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)bf16x2(v[0], v[0]);
        else reinterpret_cast<float*>(p)[i] = v[0];
    } else if constexpr (BF16) {
        *reinterpret_cast<uint4*>(p + i * 2) =
            uint4{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
    } else {
        *reinterpret_cast<float4*>(p + i * 4) = float4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<float4*>(p + i * 4 + 16) = float4{v[4], v[5], v[6], v[7]};
    }
}

// z of row t, columns [col, col + VEC)
template <bool COMBINE, bool BF16, int VEC>
__device__ __forceinline__ void load_z(const NormArgs& a, int64_t t, int col, const int32_t* rows, const float* wts,
                                       float* z) {
    const int64_t i = t * a.H + col;
    if constexpr (COMBINE) {
#pragma unroll
        for (int u = 0; u < VEC; ++u) z[u] = 0.0f;
        for (int j = 0; j < a.k + a.shared; ++j) {
            const int64_t row = j < a.k ? (int64_t)rows[j] : a.T * a.k + t;
            if (row < 0) continue;
            const float w = j < a.k ? wts[j] : 1.0f;
            float v[VEC];
            load_vec<BF16, VEC>(a.x, row * a.H + col, v);
#pragma unroll
            for (int u = 0; u < VEC; ++u) z[u] += w * v[u];
        }
    } else {
        load_vec<BF16, VEC>(a.x, i, z);
    }
    if (a.residual != nullptr) {
        float v[VEC];
        load_vec<BF16, VEC>(a.residual, i, v);
#pragma unroll
        for (int u = 0; u < VEC; ++u) z[u] += v[u];
    }
}

// Writes one vector of a row: z is its sum, r the row's factor.  With q the 16 lanes of a 128-column group
// call it together.
template <bool BF16, int VEC>
__device__ __forceinline__ void finish_vec(const NormArgs& a, int64_t t, int col, const float* z, float r) {
    const int64_t i = t * a.H + col;
    if (a.sum_out != nullptr) store_vec<BF16, VEC>(a.sum_out, i, z);
    if (a.y == nullptr && a.q == nullptr) return;
    float w[VEC], n[VEC];
    if (a.w_bf16) load_vec<true, VEC>(a.weight, col, w);
    else load_vec<false, VEC>(a.weight, col, w);
#pragma unroll
    for (int u = 0; u < VEC; ++u) n[u] = z[u] * r * w[u];
    if (a.y != nullptr) store_vec<BF16, VEC>(a.y, i, n);
    if constexpr (BF16 && VEC == 8) {
        if (a.q != nullptr) {
            // the largest magnitude as an integer maximum of the bit patterns, which keeps a NaN
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(n[u]) & 0x7fffffffu);
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 16));
            const float s = m == 0 ? 1.0f : __uint_as_float(m) / 448.0f;
            const uint32_t lo = e4m3x4(n[0] / s, n[1] / s, n[2] / s, n[3] / s);
            const uint32_t hi = e4m3x4(n[4] / s, n[5] / s, n[6] / s, n[7] / s);
            *reinterpret_cast<uint2*>(a.q + i) = uint2{lo, hi};
            if ((threadIdx.x & 15) == 0) a.q_scale[i / kFp8Group] = s;
        }
    }
}

// Any width: one workgroup per row, which reads z twice (for the sum of squares, then to write), each
// element by the same thread, so that outputs may take their inputs' place.
template <bool COMBINE, bool BF16, int VEC>
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
        float ss = 0.0f, z[VEC];
        for (int c = tid * VEC; c < a.H; c += 256 * VEC) {
            load_z<COMBINE, BF16, VEC>(a, t, c, s_row, s_w, z);
#pragma unroll
            for (int u = 0; u < VEC; ++u) ss += z[u] * z[u];
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) ss += __shfl_xor(ss, d);
        if ((tid & 63) == 0) s_part[tid >> 6] = ss;
        __syncthreads();
        ss = (s_part[0] + s_part[1]) + (s_part[2] + s_part[3]);
        const float r = 1.0f / sqrtf(ss / (float)a.H + a.eps);
        for (int c = tid * VEC; c < a.H; c += 256 * VEC) {
            load_z<COMBINE, BF16, VEC>(a, t, c, s_row, s_w, z);
            finish_vec<BF16, VEC>(a, t, c, z, r);
        }
    }
}

// ------------------------------------------------------------------------------ rows held in registers
// A thread keeps C vectors of its row (vector c of thread i: c * blockDim.x + i) as fp32 from the one read of
// the inputs to the one write of the outputs.  blockDim.x threads share a row; rows of one wave need no LDS
// and are packed blockDim.y to a workgroup.  Loads past the row's end read its last vector instead, so that
// every lane of a wave stays active up to the sum (lanes read each other's registers on the way).

// Sum over the wave, the same in every lane: four exchanges inside rows of 16 lanes, then the four rows.
__device__ __forceinline__ float wave_sum(float v) {
#define DWDP_DPP_ADD(ctrl)                                                                                         \
    v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), ctrl, 0xf, 0xf, true))
    DWDP_DPP_ADD(0xB1);        // lanes 1 apart
    DWDP_DPP_ADD(0x4E);        // 2 apart
    DWDP_DPP_ADD(0x141);       // mirrored in 8
    DWDP_DPP_ADD(0x140);       // mirrored in 16
#undef DWDP_DPP_ADD
    const int b = __float_as_int(v);
    return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

template <bool COMBINE, bool BF16, int VEC, int C>
__global__ __launch_bounds__(1024) void norm_row_kernel(NormArgs a) {
    __shared__ float s_part[16];
    const int tx = threadIdx.x, bx = blockDim.x, lane = tx & 63;
    const int n_waves = bx >> 6;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += (int64_t)gridDim.x * blockDim.y) {
        float z[C][VEC];
        if constexpr (COMBINE) {
            // lane j holds slot j's row and weight (k <= 64); rows out of range are dropped
            const int64_t rows = a.T * (a.k + a.shared);
            int my_row = -1;
            float my_w = 0.0f;
            if (lane < a.k) {
                my_row = a.inv_perm[t * a.k + lane];
                my_w = a.topk_w[t * a.k + lane];
                if (my_row >= rows) my_row = -1;
            }
            const int nsrc = a.k + a.shared;
            constexpr int B = BF16 ? 16 : 8;              // source rows whose loads are in flight together
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = min((c * bx + tx) * VEC, a.H - VEC);
#pragma unroll
                for (int u = 0; u < VEC; ++u) z[c][u] = 0.0f;
                for (int j0 = 0; j0 < nsrc; j0 += B) {
                    float4 raw[B][BF16 ? 1 : 2];
#pragma unroll
                    for (int u = 0; u < B; ++u) {
                        const int j = j0 + u;
                        if (j < nsrc) {
                            const int r = j < a.k ? __builtin_amdgcn_readlane(my_row, j) : 0;
                            const int64_t row = j < a.k ? (r >= 0 ? r : 0) : a.T * a.k + t;
                            const uint8_t* p = a.x + (row * a.H + col) * (BF16 ? 2 : 4);
                            raw[u][0] = load_stream(p);
                            if constexpr (!BF16) raw[u][1] = load_stream(p + 16);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < B; ++u) {
                        const int j = j0 + u;
                        if (j >= nsrc || (j < a.k && __builtin_amdgcn_readlane(my_row, j) < 0)) continue;
                        const float w =
                            j < a.k ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(my_w), j)) : 1.0f;
                        float v[8];
                        unpack<BF16>(raw[u], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[c][i] += w * v[i];
                    }
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                load_vec<BF16, VEC>(a.x, t * a.H + min((c * bx + tx) * VEC, a.H - VEC), z[c]);
        }
        if (a.residual != nullptr) {
            float v[C][VEC];
#pragma unroll
            for (int c = 0; c < C; ++c)
                load_vec<BF16, VEC>(a.residual, t * a.H + min((c * bx + tx) * VEC, a.H - VEC), v[c]);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int u = 0; u < VEC; ++u) z[c][u] += v[c][u];
        }
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool in = (c * bx + tx) * VEC < a.H;
#pragma unroll
            for (int u = 0; u < VEC; ++u) ss += in ? z[c][u] * z[c][u] : 0.0f;
        }
        ss = wave_sum(ss);
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
            const int col = (c * bx + tx) * VEC;
            if (col < a.H) finish_vec<BF16, VEC>(a, t, col, z[c], r);
        }
    }
}

template <bool COMBINE, bool BF16, int VEC, int C>
void launch_rows(const NormArgs& a, int threads, hipStream_t st) {
    const int rows = threads == 64 ? 4 : 1;
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + rows - 1) / rows, kMaxRowGrid);
    hipLaunchKernelGGL((norm_row_kernel<COMBINE, BF16, VEC, C>), dim3(grid), dim3(threads, rows), 0, st, a);
}

template <bool COMBINE, bool BF16, int VEC>
void launch_typed(const NormArgs& a, hipStream_t st) {
    // the largest counts that stay in 128 registers (combine: its source rows in flight take the rest)
    constexpr int C1 = VEC == 8 ? kManyC : 4, C2 = COMBINE ? C1 : VEC == 8 ? 4 : 8;
    const int64_t nvec = (a.H + VEC - 1) / VEC;
    auto threads = [&](int c) { return (int)(((nvec + c - 1) / c + 63) / 64 * 64); };
    if (threads(1) <= 64 || (a.T <= kFewRows && threads(1) <= 1024))
        launch_rows<COMBINE, BF16, VEC, 1>(a, threads(1), st);
    else if (threads(C1) <= 1024) launch_rows<COMBINE, BF16, VEC, C1>(a, threads(C1), st);
    else if (C2 != C1 && threads(C2) <= 1024) launch_rows<COMBINE, BF16, VEC, C2>(a, threads(C2), st);
    else {
        const dim3 grid((unsigned)std::min<int64_t>(a.T, kMaxRowGrid));
        hipLaunchKernelGGL((norm_two_pass_kernel<COMBINE, BF16, VEC>), grid, dim3(256), 0, st, a);
    }
}

template <bool COMBINE>
int launch_norm(const NormArgs& a, bool bf16, bool vec, hipStream_t st) {
    if (vec) {
        if (bf16) launch_typed<COMBINE, true, 8>(a, st);
        else launch_typed<COMBINE, false, 8>(a, st);
    } else if constexpr (!COMBINE) {
        if (bf16) launch_typed<false, true, 1>(a, st);
        else launch_typed<false, false, 1>(a, st);
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
    const bool vec = H % 8 == 0 && aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(sum_out) &&
                     aligned16(y);
    if (q != nullptr) DWDP_REQUIRE(vec, "q needs 16-byte aligned x, residual, weight, sum_out and y");
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
    return launch_norm<false>(a, dtype == DWDP_BF16, vec, as_stream(stream));
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
    return launch_norm<true>(a, dtype == DWDP_BF16, true, as_stream(stream));
}
