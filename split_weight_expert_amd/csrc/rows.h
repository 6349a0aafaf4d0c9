// Device helpers of the kernels that keep whole rows in registers (norms, row quantisation): sums and maxima over lanes,
// and vectors of eight elements.
#pragma once

#include <type_traits>

#include "common.h"

namespace dwdp {
namespace {

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

// Largest of LANES (16, 32 or 64) lanes' numbers, the same in each of them.
template <int LANES>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, dpp<0xB1>(v));
    v = max(v, dpp<0x4E>(v));
    v = max(v, dpp<0x141>(v));
    v = max(v, dpp<0x140>(v));
    if constexpr (LANES >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max((uint32_t)r[0], (uint32_t)r[1]);
    }
    if constexpr (LANES == 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max((uint32_t)r[0], (uint32_t)r[1]);
    }
    return v;
}

// int8 codes of a row whose largest magnitude has the bit pattern m (an integer maximum, which keeps a NaN): scale =
// amax / 127, 1 when amax is 0 and no less than the smallest normal number; code = value / scale rounded to nearest
// even.  A row with an infinity or a NaN has the scale NaN and codes 0.
struct Int8Scale {
    float scale, inverse;
};
__device__ __forceinline__ Int8Scale int8_scale(uint32_t m) {
    const float s = m == 0 ? 1.0f : __uint_as_float(max(__float_as_uint(__uint_as_float(m) / 127.0f), 0x00800000u));
    if (m >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.0f};
    return {s, 1.0f / s};
}

// The quotient as IEEE division rounds it, from the scale's rounded reciprocal: one product and one correction by its
// remainder (Markstein's division step) instead of the division's ten instructions.  For scales from 2^-102 on, below which
// the remainder may need bits under fp32's smallest.
__device__ __forceinline__ int int8_code(float v, const Int8Scale& s) {
    const float q = v * s.inverse;
    return (int)rintf(fmaf(fmaf(-q, s.scale, v), s.inverse, q));
}

__device__ __forceinline__ uint2 int8_codes(const float* v, const Int8Scale& s) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < 8; ++u) w[u / 4] |= (uint32_t)(int8_code(v[u], s) & 0xff) << (8 * (u & 3));
    return uint2{w[0], w[1]};
}

// Rows of small scales have the same quotients of values and a scale 2^64 times as large.  APART: in a code path of their
// own, which spares the others the factor but is twice the code.  Quantiser of 16384 x 7168 bf16 64.2 us apart, 65.7 with the
// factor in every row (63.7 without); the norm of one row with codes 5.9 against 5.5.
template <bool APART>
__device__ __forceinline__ uint2 int8x8(const float* v, const Int8Scale& s) {
    if (s.inverse == 0.0f) return uint2{0, 0};
    const bool small = s.inverse > 0x1p100f;
    if (APART && !small) return int8_codes(v, s);
    const float up = small ? 0x1p64f : 1.0f;
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = v[u] * up;
    return int8_codes(x, {s.scale * up, small ? s.inverse * 0x1p-64f : s.inverse});
}

}  // namespace
}  // namespace dwdp
