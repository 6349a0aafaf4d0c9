// A model's gate: scores, balance bias, group limit, top-k and weights of every token, from fp32 logits
// (dwdp_gate_topk) or with the router product before it (dwdp_route_gate).  The definition stands in
// include/dwdp_layer.h.
#include <algorithm>
#include <cmath>

#include "../../include/dwdp_layer.h"
#include "common.h"
#include "gate.h"
#include "internal.h"
#include "router.h"

namespace dwdp {
namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int kNone = 0x7fffffff;     // no expert

struct GateArgs {
    const float* logits;              // [T,E]
    const float* balance;             // [E] or null
    int64_t T;
    int E, k, groups, kept, group_top;
    bool sigmoid, renorm;
    float scale;
    int32_t* idx;
    float* w;
    // with a sliced router product: logits = sum of part[slices][T][E] + bias, written by gate_lanes_kernel
    const float* part;
    const float* bias;                // or null
    int slices;
    float* logits_out;
    // lane layout of gate_lanes_kernel: a group of group_size experts is 2^lane_shift lanes of per_lane experts
    int group_size, lane_shift, per_lane;
    int64_t first;                    // its launch's first token
};

__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ double neg_inf() { return -__builtin_huge_val(); }

// A logit that can be chosen: not NaN and not -inf.
__device__ __forceinline__ bool live_logit(float l) { return l > -__builtin_huge_valf(); }

// One token by one wave, every comparison in fp64.  Lane l holds experts l, l+64, ..; c: LDS, E doubles, then
// groups doubles of this wave.
template <int PL>
__device__ void gate_row_exact(const GateArgs& a, int64_t t, double* c) {
    const int lane = threadIdx.x & 63;
    const int E = a.E;
    const float* row = a.logits + t * E;
    float l[PL];
    double v[PL];
    double m = neg_inf();
#pragma unroll
    for (int s = 0; s < PL; ++s) {
        const int e = lane + 64 * s;
        l[s] = e < E ? row[e] : -__builtin_huge_valf();
        if (live_logit(l[s])) m = fmax(m, (double)l[s]);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmax(m, __shfl_xor(m, d));
    double sum = 0.0;
#pragma unroll
    for (int s = 0; s < PL; ++s) {
        v[s] = 0.0;
        if (live_logit(l[s])) {
            const double x = l[s];
            v[s] = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : (x == m ? 1.0 : exp(x - m));
        }
        sum += v[s];
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    // choices; -inf marks an expert that cannot be chosen
#pragma unroll
    for (int s = 0; s < PL; ++s) {
        const int e = lane + 64 * s;
        if (!a.sigmoid) v[s] /= sum;
        const float b = a.balance != nullptr && e < E ? a.balance[e] : 0.0f;
        v[s] = live_logit(l[s]) && live_logit(b) ? v[s] + (double)b : neg_inf();
    }
    if (a.groups > 1) {
        const int G = a.groups, gs = E / G;
        double* gv = c + E;
#pragma unroll
        for (int s = 0; s < PL; ++s) {
            const int e = lane + 64 * s;
            if (e < E) c[e] = a.balance == nullptr && a.group_top == 1 && v[s] > neg_inf() ? (double)l[s] : v[s];
        }
        wave_lds_sync();
        for (int g = lane; g < G; g += 64) {
            double b1 = neg_inf(), b2 = neg_inf();
            for (int i = 0; i < gs; ++i) {
                const double x = c[g * gs + i];
                if (x > b1) {
                    b2 = b1;
                    b1 = x;
                } else if (x > b2) {
                    b2 = x;
                }
            }
            gv[g] = a.group_top == 2 && b2 > neg_inf() ? b1 + b2 : b1;
        }
        wave_lds_sync();
        // group g stays if fewer than `kept` groups are better, or equal and before it
        for (int g = lane; g < G; g += 64) {
            const double x = gv[g];
            int before = 0;
            for (int h = 0; h < G; ++h) before += gv[h] > x || (gv[h] == x && h < g);
            if (before >= a.kept)
                for (int i = 0; i < gs; ++i) c[g * gs + i] = neg_inf();
        }
        wave_lds_sync();
#pragma unroll
        for (int s = 0; s < PL; ++s) {
            const int e = lane + 64 * s;
            if (e < E && c[e] == neg_inf()) v[s] = neg_inf();
        }
        wave_lds_sync();
    }
    if (a.balance == nullptr) {                   // scores without a bias are ordered as their logits
#pragma unroll
        for (int s = 0; s < PL; ++s)
            if (v[s] > neg_inf()) v[s] = l[s];
    }
    int my_i = kNone;                             // lane j keeps slot j
    for (int j = 0; j < a.k; ++j) {
        double bv = neg_inf();
        int bi = kNone;
#pragma unroll
        for (int s = 0; s < PL; ++s)
            if (v[s] > bv) {
                bv = v[s];
                bi = lane + 64 * s;
            }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            const double ov = __shfl_xor(bv, d);
            const int oi = __shfl_xor(bi, d);
            if (ov > bv || (ov == bv && oi < bi)) {
                bv = ov;
                bi = oi;
            }
        }
        if (lane == j) my_i = bi;
#pragma unroll
        for (int s = 0; s < PL; ++s)
            if (lane + 64 * s == bi) v[s] = neg_inf();
    }
    // weights
    const bool has = my_i != kNone;
    const double x = has ? (double)row[my_i] : 0.0;
    double num;
    if (a.renorm) {
        // shifted by the largest factor, so that the sum cannot vanish: sigmoid(x) = e^min(x,0) / (1 + e^-|x|)
        const double f = a.sigmoid ? fmin(x, 0.0) : x;
        double fm = has ? f : neg_inf();
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) fm = fmax(fm, __shfl_xor(fm, d));
        num = !has ? 0.0 : (f == fm ? 1.0 : exp(f - fm)) / (a.sigmoid ? 1.0 + exp(-fabs(x)) : 1.0);
        double tot = 0.0;
        for (int j = 0; j < a.k; ++j) tot += __shfl(num, j);
        num = has ? num / tot : 0.0;
    } else {
        num = !has ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-x)) : (x == m ? 1.0 : exp(x - m)) / sum;
    }
    if (lane < a.k) {
        a.idx[t * a.k + lane] = has ? my_i : -1;
        a.w[t * a.k + lane] = (float)(num * (double)a.scale);
    }
}

// One wave per token, 4 tokens per workgroup; a bounded grid walks the tokens.  Taken by gates that no lane layout of
// gate_lanes_kernel holds (more than 64 groups, or groups of more than 16 experts a lane).  Bound by fp64 exponentials
// and by the shuffles of the top-k's rounds: 16K tokens, k = 8, sigmoid and bias: 256 experts in 128 groups 85 us, 1000 in 5
// groups 235 (in 8 groups, which gate_lanes_kernel holds, 45); one token of the latter 35 us and 7.
template <int PL>
__global__ __launch_bounds__(256) void gate_exact_kernel(GateArgs a) {
    extern __shared__ double lds[];
    double* c = lds + (threadIdx.x >> 6) * (a.E + a.groups);
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * 4)
        gate_row_exact<PL>(a, t, c);
}

// ------------------------------------------------------------------------------ tokens side by side
// L lanes per token (16: a wave takes four tokens and reductions stay in a row of 16 lanes; or 64), up to PL
// consecutive experts per lane, in expert order.
//
// Keys.  An expert's key is an fp64 number: its choice with the low 10 mantissa bits replaced by the expert's
// number (reversed for positive values), so that keys are unique, the larger key is the better choice, equal
// choices go to the lower expert, and the maximum alone says who won: a round of the top-k is a maximum over
// the token and a comparison per expert, with no search for the winner.  fp64 maxima and comparisons issue at
// the rate of fp32 ones here.
//
// Precision.  Without a balance bias keys are the fp32 logits, exact.  Else they are choices from the
// hardware's fp32 exponential and reciprocal, and every decision on them is checked against the error bounds
// below.  Where the value of a group that is kept and of one that is dropped, each within its own bound, could be the
// other way round, the groups are ranked again by the fp64 choices of their two best; where two consecutive picks
// could, the k picks and the next best, one per lane, by theirs (one token in some hundreds of ordinary logits).
// Where another expert is so close that it could have taken part, gate_row_exact repeats the token.  So the choice is
// the fp64 one in every case.
//
// Error bounds (u = 2^-24).  exp2 and rcp have errors of 2 u, products and sums 1 u.
//   sigmoid: s = 1 / (1 + e), e = exp2(-l log2e): the exponent's error enters e relative by 1.5 |l| u, so s is
//     off by at most s (1 - s) (1.5 |l| + 2) u + 3 s u <= 3.9 u, since s (1 - s) |l| <= 0.23.
//   softmax: n = exp2((l - m) log2e) with x = |l - m|: off by n (2.23 x + 2) u <= 2.1 u, as n = e^-x.  S, the sum of n, is off
//     relative by the mean of that under the softmax, (2.23 ln E + 2) u since the mean of x is at most ln E, and
//     by u for each level of the pairwise sum, log2 E.  With reciprocal and product s = n / S is off by at most
//     (2.1 + 2.23 ln E + 2 + log2 E + 3) u / S: 30 u / S up to 512 experts, 33 u / S up to 1024.
//   the bias' addition adds u |c|.
// Two keys: twice that.  kTol* are those sums rounded up to powers of two.
//   a group's value b1 + b2 is off by twice a score's error, by u (|b1| + |b2|) from the biases and by u |b1 + b2| from
//     its own sum.  Choices of both signs may leave a sum far smaller than they are, so the bound goes by |b1| + |b2|:
//     kTol* + kTolChoice (|b1| + |b2|), of which at least 2 u (|b1| + |b2|) is left for the rounding of value +- bound.
constexpr float kTolSigmoid = 0x1p-21f;       // >= 2 * 3.9 u
constexpr float kTolSoftmax = 0x1p-18f;       // >= 2 * 30 u, times 1 / S
constexpr float kTolSoftmax1024 = 0x1p-17f;   // >= 2 * 33 u, times 1 / S
constexpr float kTolChoice = 0x1p-22f;        // >= 2 u, times the key

constexpr uint32_t kKeyMask = 1023;           // expert numbers: E <= 1024
constexpr uint32_t kGoneHi = 0xfe700000u;     // high word of a key that cannot be (or was) chosen: -2^1000

__device__ __forceinline__ float f_neg_inf() { return -__builtin_huge_valf(); }
__device__ __forceinline__ uint32_t hi32(double v) { return (uint32_t)(__double_as_longlong(v) >> 32); }
__device__ __forceinline__ uint32_t lo32(double v) { return (uint32_t)__double_as_longlong(v); }
__device__ __forceinline__ double from32(uint32_t hi, uint32_t lo) {
    return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}
__device__ __forceinline__ bool gone(double key) { return key < -0x1p999; }

// Maximum of two numbers that are no NaN (the compiler's fmax would first quiet each operand).
__device__ __forceinline__ double max64(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

__device__ __forceinline__ double min64(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// c as the key of expert e.  c: an fp32 number, no NaN (its fp64 form has the low 29 bits free); infinities
// become +-2^1000, beyond every finite one, and -inf is an expert that cannot be chosen.
__device__ __forceinline__ double make_key(float c, int e) {
    const double v = min64(max64((double)c, -0x1p1000), 0x1p1000);
    const uint32_t s = (uint32_t)((int32_t)hi32(v) >> 31);
    return from32(hi32(v), lo32(v) | ((s ^ (uint32_t)~e) & kKeyMask));
}
__device__ __forceinline__ int key_expert(double key) {
    const uint32_t s = (uint32_t)((int32_t)hi32(key) >> 31);
    return (int)((lo32(key) ^ ~s) & kKeyMask);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    return from32((uint32_t)__builtin_amdgcn_update_dpp(0, (int)hi32(v), CTRL, 0xf, 0xf, true),
                  (uint32_t)__builtin_amdgcn_update_dpp(0, (int)lo32(v), CTRL, 0xf, 0xf, true));
}
// This lane's and its partner's number (16 or 32 lanes away), in the order of the lanes.
template <int D>
__device__ __forceinline__ void swap_pair(uint32_t v, uint32_t& a, uint32_t& b) {
    const auto r = D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
}
template <int D, class Op>
__device__ __forceinline__ float with_partner(float v, Op op) {
    uint32_t a, b;
    swap_pair<D>(__float_as_uint(v), a, b);
    return op(__uint_as_float(a), __uint_as_float(b));
}
template <int D, class Op>
__device__ __forceinline__ double with_partner(double v, Op op) {
    uint32_t ah, bh, al, bl;
    swap_pair<D>(hi32(v), ah, bh);
    swap_pair<D>(lo32(v), al, bl);
    return op(from32(ah, al), from32(bh, bl));
}

// Over the L lanes of a token, the same in each of them.
template <int L, class V, class Op>
__device__ __forceinline__ V over_token(V v, Op op) {
    v = op(v, dpp<0xB1>(v));                  // lanes 1 apart
    v = op(v, dpp<0x4E>(v));                  // 2 apart
    v = op(v, dpp<0x141>(v));                 // mirrored in 8
    v = op(v, dpp<0x140>(v));                 // mirrored in 16
    if constexpr (L == 64) v = with_partner<32>(with_partner<16>(v, op), op);
    return v;
}
// Batcher's odd-even merge sort of 16 numbers as its comparators, the larger one to place a.
struct Net16 {
    int n = 0;
    int a[63] = {}, b[63] = {};
    constexpr Net16() {
        for (int p = 1; p < 16; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < 16; j += 2 * k)
                    for (int i = 0; i < k; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            a[n] = i + j;
                            b[n++] = i + j + k;
                        }
    }
};
constexpr Net16 kNet16;

struct MaxF {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct MinF {
    __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct AddF {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct AddD {
    __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};
struct MaxKey {
    __device__ __forceinline__ double operator()(double a, double b) const { return max64(a, b); }
};

// Bound by instruction issue: 16K tokens x 256 experts (sigmoid, bias, 4 of 8 groups, k = 8) are 18 MB, 3.6 us of
// memory traffic, and 1200 vector instructions for each four tokens, 8.0 us if every SIMD issued one every four
// cycles without a pause; 15.4 us measured in a graph, other inputs in between, of which a launch takes 2.3.  Not
// faster: keeping the logits in LDS instead of reading the chosen ones again (2 us more), or taking them from the
// lanes that hold them (0.2 us more at every size).
//
// SORTED: a lane's 16 keys are sorted once (126 maxima and minima), and a round takes the lane's first and moves up the
// others, as far as later rounds can look, in place of 15 maxima and 16 comparisons with their selections.
//
// SLICED: the logits come as a router product's partial sums, and are written on the way; lanes that repeat the last
// token write the same values.  4 slices of 8192 x 256 (34 MB): 17 to 18 us, against 10 us from logits.
template <int L, int PL, bool SLICED, bool SORTED>
__global__ __launch_bounds__(256, 2) void gate_lanes_kernel(GateArgs a) {
    constexpr int TPW = 64 / L;                       // tokens per wave
    constexpr int XPL = L * PL <= 256 ? 4 : PL;       // experts per lane of gate_row_exact (64 lanes)
    extern __shared__ double lds[];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q = lane & (L - 1), tok = lane / L;
    double* xc = lds + wave * (a.E + a.groups);       // only laid out where groups > 1
    const int gs = a.group_size, g = q >> a.lane_shift;
    const int in_group = (q & ((1 << a.lane_shift) - 1)) * a.per_lane;
    const int base = g * gs + in_group;
    const int count = g < a.groups ? max(0, min(a.per_lane, gs - in_group)) : 0;
    const bool biased = a.balance != nullptr;
    const bool pairs = a.groups > 1 && a.group_top == 2;
    const bool need_scores = biased || pairs;         // keys, or groups' values, from inexact scores
    const bool vec = (a.per_lane & 3) == 0 && (gs & 3) == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.balance) |
                       reinterpret_cast<uintptr_t>(a.bias)) & 15) == 0;
    // PL consecutive floats of this lane, -inf behind its count (with vec, counts are multiples of 4 too)
    auto load = [&](const float* p, float* x) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < PL; i += 4) {
                float4 r = float4{f_neg_inf(), f_neg_inf(), f_neg_inf(), f_neg_inf()};
                if (i < count) r = *reinterpret_cast<const float4*>(p + i);
                x[i] = r.x, x[i + 1] = r.y, x[i + 2] = r.z, x[i + 3] = r.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) x[i] = i < count ? p[i] : f_neg_inf();
        }
    };
    constexpr unsigned long long kToken = L == 64 ? ~0ull : (1ull << (L & 63)) - 1;
    // Lanes read each other's logits from memory; with a sliced product this wave has just written them.
    auto logits_written = [&] {
        if constexpr (SLICED) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    };
    // The softmax's denominator and an expert's choice in fp64, for close calls.  m: the largest logit.  The whole
    // wave works on each token that has a lane in `need`, four experts a lane at a time: on the token's own 16 lanes the
    // 16 exponentials of 256 experts, one by one, took 3 us longer (4096 tokens, a softmax with a bias).
    auto softmax_total = [&](unsigned long long need, int64_t t0, float m) {
        double total = 1.0;
        for (int i = 0; i < TPW; ++i) {
            if ((need & (kToken << (i * L))) == 0) continue;
            const float* row = a.logits + min(t0 + i, a.T - 1) * a.E;
            const float mi = __shfl(m, i * L);
            double s = 0.0;
#pragma unroll 1
            for (int e0 = lane; e0 - lane < a.E; e0 += 256) {
                float x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) x[u] = e0 + 64 * u < a.E ? row[e0 + 64 * u] : f_neg_inf();
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const double e = exp(x[u] == mi ? 0.0 : (double)x[u] - (double)mi);
                    s += x[u] > f_neg_inf() ? e : 0.0;
                }
            }
            s = over_token<64>(s, AddD());
            if (tok == i) total = s;
        }
        return total;
    };
    auto choice64 = [&](int64_t t, int e, float m, double total) {
        const float x = a.logits[t * a.E + e];
        const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : (x == m ? 1.0 : exp((double)x - (double)m)) / total;
        return biased ? s + (double)a.balance[e] : s;
    };
    const int64_t t0 = a.first + ((int64_t)blockIdx.x * 4 + wave) * TPW;
    if (t0 < a.T) {
        const int64_t t = min(t0 + tok, a.T - 1);     // lanes behind the last token repeat it and write nothing
        float l[PL], b[PL];
        if constexpr (SLICED) {
            // slices are added in order; four are read together
            const float* p = a.part + t * a.E + base;
            const int64_t stride = a.T * a.E;
#pragma unroll
            for (int i = 0; i < PL; ++i) l[i] = 0.0f;
            for (int s0 = 0; s0 < a.slices; s0 += 4) {
                float more[4][PL];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (s0 + u < a.slices) load(p + (s0 + u) * stride, more[u]);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (s0 + u < a.slices)
#pragma unroll
                        for (int i = 0; i < PL; ++i) l[i] += more[u][i];
            }
            if (a.bias != nullptr) {
                float more[PL];
                load(a.bias + base, more);
#pragma unroll
                for (int i = 0; i < PL; ++i) l[i] += more[i];
            }
            float* out = a.logits_out + t * a.E + base;
            if (vec) {
#pragma unroll
                for (int i = 0; i < PL; i += 4)
                    if (i < count) *reinterpret_cast<float4*>(out + i) = float4{l[i], l[i + 1], l[i + 2], l[i + 3]};
            } else {
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    if (i < count) out[i] = l[i];
            }
        } else {
            load(a.logits + t * a.E + base, l);
        }
        if (biased) load(a.balance + base, b);
        float m = f_neg_inf();
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            // NaN counts as -inf; adding 0 makes -0 into +0.  An expert without a live bias is out, but its logit
            // stays in the softmax.
            l[i] = l[i] > f_neg_inf() ? l[i] + 0.0f : f_neg_inf();
            if (biased) b[i] = l[i] > f_neg_inf() && b[i] > f_neg_inf() ? b[i] : f_neg_inf();
            m = fmaxf(m, l[i]);
        }
        constexpr float kLog2e = 1.44269504088896340736f;
        float sum = 1.0f;                             // the softmax's denominator in units of exp(m)
        float tol = kTolSigmoid;
        float c[PL];                                  // choices; without a bias the logits, or scores for the groups
        if (!a.sigmoid && (need_scores || !a.renorm)) {
            m = over_token<L>(m, MaxF());
            float part[PL];                           // summed pairwise: each addition's error counts log2 PL times
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                c[i] = l[i] == m ? 1.0f : __builtin_amdgcn_exp2f((l[i] - m) * kLog2e);
                c[i] = l[i] > f_neg_inf() ? c[i] : 0.0f;
                part[i] = c[i];
            }
#pragma unroll
            for (int d = PL / 2; d >= 1; d /= 2)
#pragma unroll
                for (int i = 0; i < d; ++i) part[i] += part[i + d];
            sum = over_token<L>(part[0], AddF());
            const float inv = __builtin_amdgcn_rcpf(sum);
            tol = (L * PL <= 512 ? kTolSoftmax : kTolSoftmax1024) * inv;
#pragma unroll
            for (int i = 0; i < PL; ++i) c[i] *= inv;
        } else if (need_scores) {
#pragma unroll
            for (int i = 0; i < PL; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -kLog2e));
        }
        if (biased) {
#pragma unroll
            for (int i = 0; i < PL; ++i) c[i] = b[i] > f_neg_inf() ? c[i] + b[i] : f_neg_inf();
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) c[i] = pairs && l[i] > f_neg_inf() ? c[i] : l[i];
        }
        bool unsure = false, kept = true;
        if (a.groups > 1) {
            float b1 = c[0], b2 = f_neg_inf();
#pragma unroll
            for (int i = 1; i < PL; ++i) {
                b2 = fmaxf(b2, fminf(b1, c[i]));
                b1 = fmaxf(b1, c[i]);
            }
            auto merge = [&](float o1, float o2) {
                b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
                b1 = fmaxf(b1, o1);
            };
            if (a.lane_shift > 0) merge(dpp<0xB1>(b1), dpp<0xB1>(b2));
            if (a.lane_shift > 1) merge(dpp<0x4E>(b1), dpp<0x4E>(b2));
            if (a.lane_shift > 2) merge(dpp<0x141>(b1), dpp<0x141>(b2));
            if (a.lane_shift > 3) merge(dpp<0x140>(b1), dpp<0x140>(b2));
            if constexpr (L == 64) {
                if (a.lane_shift > 4) merge(__shfl_xor(b1, 16), __shfl_xor(b2, 16));
            }
            const float value = pairs && b2 > f_neg_inf() ? b1 + b2 : b1;
            int before = 0;                           // groups ahead of this lane's
            for (int h = 0; h < a.groups; ++h) {
                const float o = __shfl(value, h << a.lane_shift, L);
                before += o > value || (o == value && h < g);
            }
            kept = before < a.kept && g < a.groups;
            // bounds of a group's value, and over the token the lowest of those kept and the highest of those dropped.  An
            // infinite choice is exact, as its sum is; a sum that passes the largest fp32 number has no bound, and a group of no
            // live expert none below.
            const bool alive = b1 > f_neg_inf();
            const float err = b1 == -f_neg_inf() ? 0.0f
                                                 : tol + kTolChoice * (fabsf(b1) + (pairs && b2 > f_neg_inf() ? fabsf(b2) : 0.0f));
            const bool bounded = err < -f_neg_inf();
            const float low = bounded ? value - err : f_neg_inf(), high = bounded ? value + err : -f_neg_inf();
            const float low_kept = need_scores ? over_token<L>(kept ? low : -f_neg_inf(), MinF()) : 0.0f;
            const float high_dropped = need_scores ? over_token<L>(!kept && alive ? high : f_neg_inf(), MaxF()) : 0.0f;
            unsure = need_scores && !(low_kept >= high_dropped);
            const unsigned long long who = __ballot(unsure);
            if (who != 0) {
                logits_written();
                // the same by fp64 values of each group's two best; where a third expert is so near that it may be
                // one of them, in a group whose bounds reach past the border, the token stays unsure
                double k1 = make_key(c[0], base), k2 = from32(kGoneHi, 0);
#pragma unroll
                for (int i = 1; i < PL; ++i) {
                    const double key = make_key(c[i], base + i);
                    k2 = max64(k2, min64(k1, key));
                    k1 = max64(k1, key);
                }
                for (int d = 1; d < 1 << a.lane_shift; d <<= 1) {
                    const double o1 = __shfl_xor(k1, d), o2 = __shfl_xor(k2, d);
                    k2 = max64(min64(k1, o1), max64(k2, o2));
                    k1 = max64(k1, o1);
                }
                const int e1 = gone(k1) ? 0 : key_expert(k1), e2 = gone(k2) ? 0 : key_expert(k2);
                bool third = false;
#pragma unroll
                for (int i = 0; i < PL; ++i)
                    third |= c[i] > f_neg_inf() && base + i != e1 && base + i != e2 && !((pairs ? b2 : b1) - c[i] >= err);
                const double total = a.sigmoid ? 1.0 : softmax_total(who, t0, m);
                const double c1 = gone(k1) ? -__builtin_huge_val() : choice64(t, e1, m, total);
                const double c2 = gone(k2) ? -__builtin_huge_val() : choice64(t, e2, m, total);
                const double v = gone(k2) ? c1 : pairs ? c1 + c2 : fmax(c1, c2);
                int before64 = 0;
                for (int h = 0; h < a.groups; ++h) {
                    const double o = __shfl(v, h << a.lane_shift, L);
                    before64 += o > v || (o == v && h < g);
                }
                // of this token's lanes, all or none are unsure; no other token has a total
                const bool near = kept ? !(low >= high_dropped) : !(low_kept >= high);
                if (unsure) kept = before64 < a.kept && g < a.groups;
                unsure = unsure && third && near;
            }
        }
        double key[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) key[i] = make_key(!kept ? f_neg_inf() : biased ? c[i] : l[i], base + i);
        if constexpr (SORTED) {
#pragma unroll
            for (int u = 0; u < kNet16.n; ++u) {
                const double x = key[kNet16.a[u]], y = key[kNet16.b[u]];
                key[kNet16.a[u]] = max64(x, y);
                key[kNet16.b[u]] = min64(x, y);
            }
        }
        // picks 0 .. k-1, and with inexact keys two more: the next best, a candidate too, and the one behind it
        double picked = from32(kGoneHi, 0), prev = 0.0;   // picked: lane j's is pick j
        bool close = false;
        const int rounds = biased ? a.k + 2 : a.k;
        for (int j = 0; j < rounds; ++j) {
            double top = key[0];
            if constexpr (SORTED) {
                top = over_token<L>(top, MaxKey());
                const bool mine = key[0] == top;
#pragma unroll
                for (int i = 0; i < PL; i += 4)
                    if (i < rounds - 1 - j)           // as deep as later rounds can look
#pragma unroll
                        for (int u = i; u < i + 4; ++u) {
                            const double next = u + 1 < PL ? key[u + 1] : from32(kGoneHi, 0);
                            key[u] = from32(mine ? hi32(next) : hi32(key[u]), mine ? lo32(next) : lo32(key[u]));
                        }
            } else {
#pragma unroll
                for (int i = 1; i < PL; ++i) top = max64(top, key[i]);
                top = over_token<L>(top, MaxKey());
#pragma unroll
                for (int i = 0; i < PL; ++i) key[i] = from32(key[i] == top ? kGoneHi : hi32(key[i]), lo32(key[i]));
            }
            if (biased && j > 0 && j <= a.k) close |= !gone(top) && !(prev - top >= tol + kTolChoice * fabs(prev));
            prev = top;
            if (q == j) picked = top;
        }
        bool has = q < a.k && !gone(picked);
        int my_i = gone(picked) ? 0 : key_expert(picked);
        logits_written();
        const unsigned long long closes = __ballot(close);
        if (closes != 0) {
            // prev is the best expert that is no candidate
            const double total = a.sigmoid ? 1.0 : softmax_total(closes, t0, m);
            const bool cand = q <= a.k && !gone(picked);
            const double c = cand ? choice64(t, my_i, m, total) : -__builtin_huge_val();
            int rank = 0;
            for (int j = 0; j <= a.k; ++j) {
                const double o = __shfl(c, j, L);
                const int oi = __shfl(my_i, j, L);
                rank += o > c || (o == c && oi < my_i && j != q);
            }
            // candidates are ranked 0 .. n-1; each goes to the lane of its rank, every other lane keeps its number
            const int to = cand ? rank : q;
            if (close && cand && rank == a.k - 1) unsure |= !gone(prev) && !(c - prev >= tol + kTolChoice * fabs(prev));
            const int sent = __builtin_amdgcn_ds_permute((to + (lane & ~(L - 1))) * 4, my_i);
            my_i = close ? sent : my_i;
        }
        // weights: lane j of the token has slot j
        const float x = has ? a.logits[t * a.E + my_i] : 0.0f;
        float num = 0.0f;
        if (a.renorm) {
            // shifted by the largest factor, as in gate_row_exact
            const float f = a.sigmoid ? fminf(x, 0.0f) : x;
            const float fm = over_token<L>(has ? f : f_neg_inf(), MaxF());
            num = !has ? 0.0f : (f == fm ? 1.0f : expf(f - fm)) / (a.sigmoid ? 1.0f + expf(-fabsf(x)) : 1.0f);
            const float tot = over_token<L>(num, AddF());
            num = has ? num / tot : 0.0f;
        } else if (has) {
            num = a.sigmoid ? 1.0f / (1.0f + expf(-x)) : (x == m ? 1.0f : expf(x - m)) / sum;
        }
        const unsigned long long redo = __ballot(unsure);
        const bool mine = (redo & (kToken << (lane & ~(L - 1)))) == 0;
        if (q < a.k && t0 + tok < a.T && mine) {
            a.idx[t * a.k + q] = has ? my_i : -1;
            a.w[t * a.k + q] = num * a.scale;
        }
        if (redo != 0) {
            for (int i = 0; i < TPW; ++i)
                if ((redo & (kToken << (i * L))) != 0 && t0 + i < a.T) gate_row_exact<XPL>(a, t0 + i, xc);
        }
    }
}

bool aligned4(const void* a, const void* b, const void* c, const void* d, const void* e = nullptr) {
    return type_aligned(a, 4) && type_aligned(b, 4) && type_aligned(c, 4) && type_aligned(d, 4) && type_aligned(e, 4);
}

GateArgs gate_args(const float* logits, const float* balance, int64_t T, int E, const dwdp_gate& g, int32_t* idx,
                   float* w) {
    GateArgs a{};
    a.logits = logits;
    a.balance = balance;
    a.T = T;
    a.E = E;
    a.k = g.k;
    // a limit that keeps every group is none
    a.groups = g.topk_groups == g.n_groups ? 1 : g.n_groups;
    a.kept = g.topk_groups;
    a.group_top = g.group_top;
    a.sigmoid = g.score == DWDP_SCORE_SIGMOID;
    a.renorm = g.renormalize != 0;
    a.scale = g.scale;
    a.idx = idx;
    a.w = w;
    return a;
}

template <int L, int PL>
bool launch_lanes(GateArgs& a, hipStream_t st) {
    // a group on the fewest lanes (a power of two) that hold it; without groups, the whole token
    const int gs = a.E / a.groups;
    int shift = 0;
    while ((1 << shift) < L && (a.groups == 1 || (gs + (1 << shift) - 1) >> shift > PL)) ++shift;
    int per = (gs + (1 << shift) - 1) >> shift;
    // k picks and the next best, one per lane
    if (per > PL || a.groups << shift > L || a.k >= L) return false;
    if (gs % 4 == 0) per = (per + 3) / 4 * 4;         // 16-byte loads
    a.group_size = gs;
    a.lane_shift = shift;
    a.per_lane = per;
    const size_t lds = a.groups > 1 ? 4 * (size_t)(a.E + a.groups) * sizeof(double) : 0;   // for gate_row_exact
    constexpr int64_t kTokens = 4 * (64 / L);         // per workgroup
    // a launch takes up to kMaxRowGrid workgroups (a loop over tokens in the kernel would keep what is the same
    // for all of them in registers: 200 against 131 when tried)
    //
    // Sorted keys spend fewer instructions over many rounds, but in a longer chain (20 inputs in turn in a graph): 256 experts
    // on 16 lanes, k = 8, sigmoid, bias and groups, 16K tokens 15.4 us sorted and 16.2 not, 4096 tokens 9.0 and 8.9; 1024
    // experts on 64 lanes, 4096 tokens 16.1 and 17.3; 16K tokens with 2 rounds 8.3 and 7.9, 6 rounds 9.4 and 9.8.  So: where a
    // SIMD has more than two waves.
    const int rounds = a.balance != nullptr ? a.k + 2 : a.k;
    const bool sorted = PL == 16 && rounds >= 6 && a.T * L / 64 > 2048;
    for (a.first = 0; a.first < a.T; a.first += kMaxRowGrid * kTokens) {
        const dim3 grid((unsigned)std::min<int64_t>((a.T - a.first + kTokens - 1) / kTokens, kMaxRowGrid));
        auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), lds, st, a); };
        if constexpr (PL == 16) {
            if (sorted) {
                if (a.part != nullptr) launch(gate_lanes_kernel<L, PL, true, true>);
                else launch(gate_lanes_kernel<L, PL, false, true>);
                continue;
            }
        }
        if (a.part != nullptr) launch(gate_lanes_kernel<L, PL, true, false>);
        else launch(gate_lanes_kernel<L, PL, false, false>);
    }
    return true;
}

template <int PL>
void launch_exact(const GateArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)std::min<int64_t>((a.T + 3) / 4, kMaxRowGrid));
    const size_t lds = a.groups > 1 ? 4 * (size_t)(a.E + a.groups) * sizeof(double) : 0;   // at most 64 KB
    hipLaunchKernelGGL(gate_exact_kernel<PL>, grid, dim3(256), lds, st, a);
}

// Whether a lane layout holds the gate: a group on at most 64 / groups lanes, a power of two.
bool lanes_hold(const GateArgs& a) {
    if (a.groups > 64) return false;
    int lanes = 1;
    while (2 * lanes * a.groups <= 64) lanes *= 2;
    return (a.E / a.groups + lanes - 1) / lanes <= 16;
}

int launch_gate(GateArgs a, hipStream_t st) {
    if (lanes_hold(a)) {
        // The narrowest layout that holds it: four tokens to a wave spend fewer instructions on each, 64 lanes on one
        // are done sooner as long as the chip has room for the waves.  16 against 64 lanes, us, 20 inputs in turn in a graph:
        //   4 experts a lane (64 experts, k = 8): 1 token 3.2 and 3.4, 1777 tokens 3.6 and 4.3
        //   8 (128, sigmoid with a bias):         64 tokens 4.5 and 4.4, 1777 5.2 and 5.4, 4096 6.1 and 7.8
        //   16 (256, the same and 4 of 8 groups): 64 tokens 6.7 and 5.2, 2048 8.4 and 7.0, 3500 8.7 and 8.7
        launch_lanes<16, 4>(a, st) || (a.T > 1024 && launch_lanes<16, 8>(a, st)) ||
            (a.T > 2048 && launch_lanes<16, 16>(a, st)) || launch_lanes<64, 4>(a, st) || launch_lanes<64, 8>(a, st) ||
            launch_lanes<64, 16>(a, st);
    } else if (a.E <= 256) {
        launch_exact<4>(a, st);
    } else if (a.E <= 512) {
        launch_exact<8>(a, st);
    } else {
        launch_exact<16>(a, st);
    }
    DWDP_LAUNCHED();
    return DWDP_OK;
}

}  // namespace

int check_gate(const char* fn, const dwdp_gate* g, int E) {
    auto bad = [&](const char* what) { return fail(DWDP_ERR_INVALID_ARG, std::string(fn) + ": " + what); };
    if (g == nullptr) return bad("gate is NULL");
    if (E < 1 || E > kMaxE) return bad("E must be in [1, 1024]");
    if (g->score != DWDP_SCORE_SOFTMAX && g->score != DWDP_SCORE_SIGMOID)
        return bad("score must be DWDP_SCORE_SOFTMAX or DWDP_SCORE_SIGMOID");
    if (g->k < 1 || g->k > E || g->k > kMaxK) return bad("k must be in [1, min(E, 32)]");
    if (g->n_groups < 1 || g->n_groups > E || E % g->n_groups != 0)
        return bad("n_groups must divide E");
    if (g->topk_groups < 1 || g->topk_groups > g->n_groups)
        return bad("topk_groups must be in [1, n_groups]");
    if (g->k > g->topk_groups * (E / g->n_groups))
        return bad("k must be at most the experts of topk_groups groups");
    if (g->group_top != 1 && g->group_top != 2) return bad("group_top must be 1 or 2");
    if (g->renormalize != 0 && g->renormalize != 1)
        return bad("renormalize must be 0 or 1");
    if (!std::isfinite(g->scale)) return bad("scale must be finite");
    return DWDP_OK;
}

}  // namespace dwdp

using namespace dwdp;

extern "C" int dwdp_gate_topk(const float* logits, const float* balance_bias, int64_t T, int E, const dwdp_gate* gate,
                              int32_t* topk_idx, float* topk_w, void* stream) {
    clear_error();
    int rc = check_gate(__func__, gate, E);
    if (rc != DWDP_OK) return rc;
    DWDP_REQUIRE(T >= 0 && T < ((int64_t)1 << 31), "T out of range");
    if (T == 0) return DWDP_OK;
    DWDP_REQUIRE(logits && topk_idx && topk_w, "null pointer argument");
    DWDP_REQUIRE(aligned4(logits, balance_bias, topk_idx, topk_w), "a pointer is not aligned to 4 bytes");
    const size_t chosen = (size_t)T * gate->k * 4;
    const Span outs[] = {{topk_idx, chosen}, {topk_w, chosen}};
    const Span ins[] = {{logits, (size_t)T * E * 4}, {balance_bias, (size_t)E * 4}};
    DWDP_REQUIRE(!overlap_any(outs, 2, ins, 2), "an output overlaps another buffer");
    return launch_gate(gate_args(logits, balance_bias, T, E, *gate, topk_idx, topk_w), as_stream(stream));
}

extern "C" size_t dwdp_route_gate_workspace_bytes(int64_t T, int H, int E, int in_dtype) {
    if (T < 1 || T >= ((int64_t)1 << 31) || E < 1 || E > kMaxE || (in_dtype != DWDP_F32 && in_dtype != DWDP_BF16) ||
        H < 1 || H % (in_dtype == DWDP_BF16 ? 64 : 16) != 0)
        return 0;
    const RouterPlan p = plan_router(T, H, E, in_dtype);
    return p.slices == 1 ? 0 : (size_t)p.slices * T * E * sizeof(float);
}

extern "C" int dwdp_route_gate(const void* x, const void* w_router, int in_dtype, const float* bias,
                               const float* balance_bias, int64_t T, int H, int E, const dwdp_gate* gate,
                               float* logits_out, int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                               void* stream) {
    clear_error();
    DWDP_REQUIRE(in_dtype == DWDP_F32 || in_dtype == DWDP_BF16, "in_dtype must be DWDP_F32 or DWDP_BF16");
    int rc = check_gate(__func__, gate, E);
    if (rc != DWDP_OK) return rc;
    DWDP_REQUIRE(T >= 0 && T < ((int64_t)1 << 31), "T out of range");
    DWDP_REQUIRE(H > 0, "H must be positive");
    if (in_dtype == DWDP_BF16) DWDP_REQUIRE(H % 64 == 0, "bf16 routing needs H % 64 == 0");
    else DWDP_REQUIRE(H % 16 == 0, "f32 routing needs H % 16 == 0");
    if (T == 0) return DWDP_OK;
    DWDP_REQUIRE(x && w_router && logits_out && topk_idx && topk_w, "null pointer argument");
    DWDP_REQUIRE(aligned16(x) && aligned16(w_router), "x and w_router must be 16-byte aligned");
    DWDP_REQUIRE(aligned4(logits_out, balance_bias, topk_idx, topk_w, bias), "a pointer is not aligned to 4 bytes");
    const size_t need = dwdp_route_gate_workspace_bytes(T, H, E, in_dtype);
    if (need != 0) {
        DWDP_REQUIRE(ws != nullptr && aligned16(ws), "ws is NULL or not 16-byte aligned");
        if (ws_bytes < need) return fail(DWDP_ERR_WORKSPACE, "dwdp_route_gate: workspace too small");
    }
    const RouterPlan p = plan_router(T, H, E, in_dtype);
    DWDP_REQUIRE(router_fits(T, E, p), "T too large for one router launch");
    const size_t chosen = (size_t)T * gate->k * 4, row = (size_t)H * elem_bytes(in_dtype);
    const Span outs[] = {{logits_out, (size_t)T * E * 4}, {topk_idx, chosen}, {topk_w, chosen}, {ws, need}};
    const Span ins[] = {{x, T * row}, {w_router, E * row}, {bias, (size_t)E * 4}, {balance_bias, (size_t)E * 4}};
    DWDP_REQUIRE(!overlap_any(outs, 4, ins, 4), "an output or ws overlaps another buffer");
    hipStream_t st = as_stream(stream);
    GateArgs a = gate_args(logits_out, balance_bias, T, E, *gate, topk_idx, topk_w);
    if (p.slices > 1 && lanes_hold(a)) {
        a.part = static_cast<const float*>(ws);
        a.bias = bias;
        a.slices = p.slices;
        a.logits_out = logits_out;
        rc = router_split(x, w_router, in_dtype, bias, T, H, E, p, logits_out, static_cast<float*>(ws), st);
    } else {
        rc = router_split(x, w_router, in_dtype, bias, T, H, E, RouterPlan{p.bm, p.bn, 1}, logits_out, nullptr, st);
    }
    if (rc != DWDP_OK) return rc;
    return launch_gate(a, st);
}
