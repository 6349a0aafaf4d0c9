// Rows as int8 codes with one scale per row (dwdp_quantize_int8; the grouped FFN's A): tokens, or weights by output
// channel.
#include <algorithm>

#include "../../include/dwdp_layer.h"
#include "common.h"
#include "internal.h"
#include "rows.h"

namespace dwdp {
namespace {

struct QuantArgs {
    const uint8_t* x;
    int64_t rows;
    int cols;
    uint8_t* q;
    float* scale;
};

__device__ __forceinline__ uint32_t amax8(const float* v) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(v[u]) & 0x7fffffffu);
    return m;
}

// A thread keeps C vectors of its row (vector c of thread i: c * blockDim.x + i) from the one read of the row to the
// write of its codes; blockDim.x threads share a row, LANES of them in one wave, and rows of a wave or less are packed
// blockDim.y to a workgroup.  Bound by HBM.
template <bool BF16, int C, int LANES>
__global__ __launch_bounds__(1024) void quant_row_kernel(QuantArgs a) {
    __shared__ uint32_t s_part[16];
    const int tx = threadIdx.x, bx = LANES < 64 ? LANES : blockDim.x;
    const int n_waves = LANES < 64 ? 1 : bx >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, stride = (int64_t)gridDim.x * blockDim.y;
    for (int64_t t = t0; t < a.rows; t += stride) {
        float v[C][8];
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * bx + tx) * 8;
#pragma unroll
            for (int u = 0; u < 8; ++u) v[c][u] = 0.0f;
            if (col < a.cols) unpack<BF16>(load_stream<BF16>(a.x + (t * a.cols + col) * (BF16 ? 2 : 4)), v[c]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) m = max(m, amax8(v[c]));
        m = row_max<LANES>(m);
        if (n_waves > 1) {
            if ((tx & 63) == 0) s_part[tx >> 6] = m;
            __syncthreads();
            for (int i = 0; i < n_waves; ++i) m = max(m, s_part[i]);
            __syncthreads();                          // read before the next row's maxima
        }
        const Int8Scale s = int8_scale(m);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * bx + tx) * 8;
            if (col < a.cols) *reinterpret_cast<uint2*>(a.q + t * a.cols + col) = int8x8<true>(v[c], s);
        }
        if (tx == 0) a.scale[t] = s.scale;
    }
}

// Rows too wide for the registers (above 32768 elements), read twice.
template <bool BF16>
__global__ __launch_bounds__(1024) void quant_wide_kernel(QuantArgs a) {
    __shared__ uint32_t s_part[16];
    const int tx = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
        const uint8_t* x = a.x + t * a.cols * (BF16 ? 2 : 4);
        uint32_t m = 0;
        float v[8];
        for (uint32_t c = tx * 8; c < (uint32_t)a.cols; c += 1024 * 8) {
            unpack<BF16>(load_raw<BF16, true>(x, c), v);
            m = max(m, amax8(v));
        }
        m = row_max<64>(m);
        if ((tx & 63) == 0) s_part[tx >> 6] = m;
        __syncthreads();
        for (int i = 0; i < 16; ++i) m = max(m, s_part[i]);
        __syncthreads();
        const Int8Scale s = int8_scale(m);
        for (uint32_t c = tx * 8; c < (uint32_t)a.cols; c += 1024 * 8) {
            unpack<BF16>(load_raw<BF16, true>(x, c), v);
            *reinterpret_cast<uint2*>(a.q + t * a.cols + c) = int8x8<true>(v, s);
        }
        if (tx == 0) a.scale[t] = s.scale;
    }
}

template <bool BF16>
void launch_quant(const QuantArgs& a, hipStream_t st) {
    const int nvec = a.cols / 8;
    auto go = [&](auto kernel, int threads) {
        const int rows = threads <= 64 ? 256 / threads : 1;
        const unsigned grid = (unsigned)std::min<int64_t>((a.rows + rows - 1) / rows, kMaxRowGrid);
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads, rows), 0, st, a);
    };
    auto threads = [&](int c) { return ((nvec + c - 1) / c + 63) / 64 * 64; };
    if (nvec <= 16) go(quant_row_kernel<BF16, 1, 16>, 16);
    else if (nvec <= 32) go(quant_row_kernel<BF16, 1, 32>, 32);
    else if (nvec <= 64) go(quant_row_kernel<BF16, 1, 64>, 64);
    else if (nvec <= 2 * 1024) go(quant_row_kernel<BF16, 2, 64>, threads(2));
    else if (nvec <= 4 * 1024) go(quant_row_kernel<BF16, 4, 64>, threads(4));
    else hipLaunchKernelGGL(quant_wide_kernel<BF16>, dim3((unsigned)std::min<int64_t>(a.rows, kMaxRowGrid)), dim3(1024), 0, st, a);
}

}  // namespace

int quantize_rows_int8(const void* x, int dtype, int64_t rows, int cols, void* q, float* scale, void* stream) {
    QuantArgs a{static_cast<const uint8_t*>(x), rows, cols, static_cast<uint8_t*>(q), scale};
    if (dtype == DWDP_BF16) launch_quant<true>(a, as_stream(stream));
    else launch_quant<false>(a, as_stream(stream));
    DWDP_LAUNCHED();
    return DWDP_OK;
}

}  // namespace dwdp

using namespace dwdp;

extern "C" int dwdp_quantize_int8(const void* x, int dtype, int64_t rows, int cols, void* q, float* scale, void* stream) {
    clear_error();
    DWDP_REQUIRE(dtype == DWDP_F32 || dtype == DWDP_BF16, "dtype must be DWDP_F32 or DWDP_BF16");
    DWDP_REQUIRE(rows >= 0 && rows < ((int64_t)1 << 31), "rows out of range");
    DWDP_REQUIRE(cols > 0 && cols % 8 == 0, "cols must be a positive multiple of 8");
    if (rows == 0) return DWDP_OK;
    DWDP_REQUIRE(x && q && scale, "null pointer argument");
    DWDP_REQUIRE(aligned16(x) && type_aligned(q, 8) && type_aligned(scale, 4),
                 "x must be 16-byte aligned, q 8-byte and scale 4-byte aligned");
    const size_t n = (size_t)rows * cols;
    const Span outs[] = {{q, n}, {scale, (size_t)rows * 4}}, ins[] = {{x, n * elem_bytes(dtype)}};
    DWDP_REQUIRE(!overlap_any(outs, 2, ins, 1), "an output overlaps another buffer");
    return quantize_rows_int8(x, dtype, rows, cols, q, scale, stream);
}
