// A model's gate: scores, balance bias, group limit, top-k and weights of every token, from fp32 logits
// (dwdp_gate_topk) or with the router product before it (dwdp_route_gate).  The definition stands in
// include/dwdp_layer.h.
#include <algorithm>
#include <cmath>

#include "../../include/dwdp_layer.h"
#include "common.h"
#include "internal.h"

namespace dwdp {
int router_logits(const void* x, const void* w_router, int in_dtype, const float* bias, int64_t T, int H, int E,
                  float* logits, hipStream_t st);

namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int kNone = 0x7fffffff;     // no expert

struct GateArgs {
    const float* logits;              // [T,E] (split kernel: written by it, bias included)
    const float* balance;             // [E] or null
    int64_t T;
    int E, k, groups, kept, group_top;
    bool sigmoid, renorm;
    float scale;
    int32_t* idx;
    float* w;
    // lane layout of gate_lanes_kernel: a group is group_lanes lanes (a power of two) of per_lane experts
    int group_lanes, per_lane;
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

// One wave per token, 4 tokens per workgroup; a bounded grid walks the tokens.
template <int PL>
__global__ __launch_bounds__(256) void gate_exact_kernel(GateArgs a) {
    extern __shared__ double lds[];
    double* c = lds + (threadIdx.x >> 6) * (a.E + a.groups);
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * 4)
        gate_row_exact<PL>(a, t, c);
}

// ------------------------------------------------------------------------------ tokens side by side
// L lanes per token (16 of them, so that a wave takes four tokens and reductions stay in a row of 16 lanes;
// or 64), up to PL consecutive experts per lane, in expert order.  Keys are fp32: the logits themselves
// without a balance bias (their order is exact), else score + bias from the hardware exponential and
// reciprocal.  Those carry an error, so every decision taken on them is checked: where two consecutive
// picks, or the last group kept and the first one dropped, are closer than twice the error bound, the wave
// repeats the token in fp64 (gate_row_exact).  The choice therefore is the fp64 one in every case, and one
// token in about a thousand of ordinary logits pays for it.
//
// Error bounds (u = 2^-24).  exp2 and rcp have errors of 2 u, products and sums 1 u.
//   sigmoid: s = 1 / (1 + e), e = exp2(-l log2e): the exponent's error enters e relative by 1.5 |l| u, so s is
//     off by at most s (1 - s) (1.5 |l| + 2) u + 3 s u <= 3.9 u, since s (1 - s) |l| <= 0.23.
//   softmax: f = exp2((l - m) log2e) / S with S >= 1: the numerator is off by at most 3 u, S by 42 u relative
//     (the mean of |l - m| under the softmax is at most ln 1024), so s by at most 51 u / S, as s <= 1 / S.
//   the bias' addition adds u |c|.
// Two keys: twice that.  kTol* below are those sums rounded up to powers of two.
constexpr float kTolSigmoid = 0x1p-20f;       // >= 2 * 3.9 u
constexpr float kTolSoftmax = 0x1p-17f;       // >= 2 * 51 u, times 1 / S
constexpr float kTolChoice = 0x1p-22f;        // >= 2 u, times the key

__device__ __forceinline__ float f_neg_inf() { return -__builtin_huge_valf(); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

struct MaxOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct MinOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct AddOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// Over the L lanes of a token, the same in each of them.
template <int L, class Op>
__device__ __forceinline__ float over_token(float v, Op op) {
    v = op(v, dpp<0xB1>(v));                  // lanes 1 apart
    v = op(v, dpp<0x4E>(v));                  // 2 apart
    v = op(v, dpp<0x141>(v));                 // mirrored in 8
    v = op(v, dpp<0x140>(v));                 // mirrored in 16
    if constexpr (L == 64) {
        const int b = __float_as_int(v);
        v = op(op(__int_as_float(__builtin_amdgcn_readlane(b, 0)), __int_as_float(__builtin_amdgcn_readlane(b, 16))),
               op(__int_as_float(__builtin_amdgcn_readlane(b, 32)), __int_as_float(__builtin_amdgcn_readlane(b, 48))));
    }
    return v;
}

// First lane of this lane's token whose bit is set (its number in the token); none set: 32 or more.
template <int L>
__device__ __forceinline__ int first_lane(unsigned long long b) {
    if constexpr (L == 64) return b == 0 ? 64 : __builtin_ctzll(b);
    const int lane = threadIdx.x & 63;
    const uint32_t half = lane < 32 ? (uint32_t)b : (uint32_t)(b >> 32);
    const uint32_t seg = (half >> (lane & 16)) & 0xffffu;
    return __builtin_ctz(seg | 0x80000000u);
}

template <int L, int PL>
__global__ __launch_bounds__(256) void gate_lanes_kernel(GateArgs a) {
    constexpr int TPW = 64 / L;                       // tokens per wave
    constexpr int XPL = L == 16 ? 4 : PL;             // experts per lane of the fp64 form (64 lanes)
    extern __shared__ double lds[];
    __shared__ int s_slot[4][TPW][L < kMaxK ? L : kMaxK];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q = lane & (L - 1), tok = lane / L;
    double* xc = lds + wave * (a.E + a.groups);       // only laid out where groups > 1
    const int gs = a.E / a.groups, g = q / a.group_lanes;
    const int in_group = (q & (a.group_lanes - 1)) * a.per_lane;
    const int base = g * gs + in_group;
    const int count = g < a.groups ? max(0, min(a.per_lane, gs - in_group)) : 0;
    const bool biased = a.balance != nullptr;
    const bool pairs = a.groups > 1 && a.group_top == 2;
    const bool need_scores = biased || pairs;
    const bool vec = (a.per_lane & 3) == 0 && (gs & 3) == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0;
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * TPW; t0 < a.T; t0 += (int64_t)gridDim.x * 4 * TPW) {
        const int64_t t = min(t0 + tok, a.T - 1);     // lanes behind the last token repeat it and write nothing
        const float* row = a.logits + t * a.E + base;
        float l[PL], v[PL];
        if (vec) {                                    // counts are multiples of 4 too
#pragma unroll
            for (int i = 0; i < PL; i += 4) {
                float4 x = float4{f_neg_inf(), f_neg_inf(), f_neg_inf(), f_neg_inf()};
                if (i < count) x = *reinterpret_cast<const float4*>(row + i);
                l[i] = x.x, l[i + 1] = x.y, l[i + 2] = x.z, l[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) l[i] = i < count ? row[i] : f_neg_inf();
        }
        // NaN counts as -inf; adding 0 makes -0 into +0
        float m = f_neg_inf();
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            l[i] = l[i] > f_neg_inf() ? l[i] + 0.0f : f_neg_inf();
            m = fmaxf(m, l[i]);
        }
        constexpr float kLog2e = 1.44269504088896340736f;
        float sum = 1.0f, tol = kTolSigmoid;
        if (!a.sigmoid && (need_scores || !a.renorm)) {
            m = over_token<L>(m, MaxOp());
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                v[i] = l[i] == m ? 1.0f : __builtin_amdgcn_exp2f((l[i] - m) * kLog2e);
                v[i] = l[i] > f_neg_inf() ? v[i] : 0.0f;
                sum += v[i];
            }
            sum = over_token<L>(sum, AddOp());
            const float inv = __builtin_amdgcn_rcpf(sum);
            tol = kTolSoftmax * inv;
#pragma unroll
            for (int i = 0; i < PL; ++i) v[i] *= inv;
        } else if (need_scores) {
#pragma unroll
            for (int i = 0; i < PL; ++i)
                v[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -kLog2e));
        }
        bool unsure = false;
        if (biased) {
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const float b = i < count ? a.balance[base + i] : f_neg_inf();
                v[i] = l[i] > f_neg_inf() && live_logit(b) ? v[i] + b : f_neg_inf();
            }
        } else {
#pragma unroll
            for (int i = 0; i < PL; ++i) v[i] = pairs && l[i] > f_neg_inf() ? v[i] : l[i];
        }
        if (a.groups > 1) {
            float b1 = f_neg_inf(), b2 = f_neg_inf();
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                b2 = fmaxf(b2, fminf(b1, v[i]));
                b1 = fmaxf(b1, v[i]);
            }
            for (int d = 1; d < a.group_lanes; d <<= 1) {
                const float o1 = __shfl_xor(b1, d), o2 = __shfl_xor(b2, d);
                b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
                b1 = fmaxf(b1, o1);
            }
            const float value = pairs && b2 > f_neg_inf() ? b1 + b2 : b1;
            int before = 0;
            for (int h = 0; h < a.groups; ++h) {
                const float o = __shfl(value, h * a.group_lanes, L);
                before += o > value || (o == value && h < g);
            }
            const bool kept = before < a.kept && g < a.groups;
            if (need_scores) {                        // fp32 scores: is the border wide enough?
                const float lo = over_token<L>(kept ? value : -f_neg_inf(), MinOp());
                const float hi = over_token<L>(!kept && g < a.groups ? value : f_neg_inf(), MaxOp());
                unsure |= hi > f_neg_inf() && !(lo - hi >= 2.0f * tol + 2.0f * kTolChoice * fabsf(lo));
            }
#pragma unroll
            for (int i = 0; i < PL; ++i) v[i] = !kept ? f_neg_inf() : biased ? v[i] : l[i];
        }
        float prev = 0.0f;
        int slots = 0;                                // slots filled
        for (int j = 0; j <= a.k; ++j) {
            if (j == a.k && !biased) break;           // the pick behind the last only matters to the check
            float best = v[0];
#pragma unroll
            for (int i = 1; i < PL; ++i) best = fmaxf(best, v[i]);
            const float top = over_token<L>(best, MaxOp());
            const bool some = top > f_neg_inf();
            if (biased && j > 0)
                unsure |= some && !(prev - top >= tol + kTolChoice * fabsf(prev));
            prev = top;
            if (j == a.k) break;
            bool take = some && first_lane<L>(__ballot(best == top)) == q;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const bool hit = take && v[i] == top;
                v[i] = hit ? f_neg_inf() : v[i];
                if (hit) s_slot[wave][tok][j] = base + i;
                take = take && !hit;
            }
            slots += some;
        }
        wave_lds_sync();
        // weights: lane j of the token has slot j
        const bool has = q < slots;
        const int my_i = has ? s_slot[wave][tok][q] : 0;
        const float x = has ? a.logits[t * a.E + my_i] : 0.0f;
        float num = 0.0f;
        if (a.renorm) {
            const float f = a.sigmoid ? fminf(x, 0.0f) : x;
            const float fm = over_token<L>(has ? f : f_neg_inf(), MaxOp());
            num = !has ? 0.0f : (f == fm ? 1.0f : expf(f - fm)) / (a.sigmoid ? 1.0f + expf(-fabsf(x)) : 1.0f);
            const float tot = over_token<L>(num, AddOp());
            num = has ? num / tot : 0.0f;
        } else if (has) {
            num = a.sigmoid ? 1.0f / (1.0f + expf(-x)) : (x == m ? 1.0f : expf(x - m)) / sum;
        }
        const unsigned long long redo = __ballot(unsure);
        const bool mine = ((redo >> (lane & ~(L - 1))) & 1) == 0;
        if (q < a.k && t0 + tok < a.T && mine) {
            a.idx[t * a.k + q] = has ? my_i : -1;
            a.w[t * a.k + q] = num * a.scale;
        }
        if (redo != 0) {
            for (int i = 0; i < TPW; ++i)
                if (((redo >> (i * L)) & 1) != 0 && t0 + i < a.T) gate_row_exact<XPL>(a, t0 + i, xc);
        }
        wave_lds_sync();                              // s_slot is read before the next token's picks
    }
}

bool aligned4(const void* a, const void* b, const void* c, const void* d, const void* e = nullptr) {
    return type_aligned(a, 4) && type_aligned(b, 4) && type_aligned(c, 4) && type_aligned(d, 4) && type_aligned(e, 4);
}

int check_gate(const char* fn, const dwdp_gate* g, int E) {
    const std::string f = std::string(fn) + ": ";
    if (g == nullptr) return fail(DWDP_ERR_INVALID_ARG, f + "gate is NULL");
    if (E < 1 || E > kMaxE) return fail(DWDP_ERR_INVALID_ARG, f + "E must be in [1, 1024]");
    if (g->score != DWDP_SCORE_SOFTMAX && g->score != DWDP_SCORE_SIGMOID)
        return fail(DWDP_ERR_INVALID_ARG, f + "score must be DWDP_SCORE_SOFTMAX or DWDP_SCORE_SIGMOID");
    if (g->k < 1 || g->k > E || g->k > kMaxK) return fail(DWDP_ERR_INVALID_ARG, f + "k must be in [1, min(E, 32)]");
    if (g->n_groups < 1 || g->n_groups > E || E % g->n_groups != 0)
        return fail(DWDP_ERR_INVALID_ARG, f + "n_groups must divide E");
    if (g->topk_groups < 1 || g->topk_groups > g->n_groups)
        return fail(DWDP_ERR_INVALID_ARG, f + "topk_groups must be in [1, n_groups]");
    if (g->k > g->topk_groups * (E / g->n_groups))
        return fail(DWDP_ERR_INVALID_ARG, f + "k must be at most the experts of topk_groups groups");
    if (g->group_top != 1 && g->group_top != 2) return fail(DWDP_ERR_INVALID_ARG, f + "group_top must be 1 or 2");
    if (g->renormalize != 0 && g->renormalize != 1)
        return fail(DWDP_ERR_INVALID_ARG, f + "renormalize must be 0 or 1");
    if (!std::isfinite(g->scale)) return fail(DWDP_ERR_INVALID_ARG, f + "scale must be finite");
    return DWDP_OK;
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
    int lanes = a.groups == 1 ? L : 1;
    while (lanes < L && (gs + lanes - 1) / lanes > PL) lanes *= 2;
    int per = (gs + lanes - 1) / lanes;
    if (per > PL || lanes * a.groups > L || a.k > L) return false;
    if (gs % 4 == 0) per = (per + 3) / 4 * 4;         // 16-byte loads
    a.group_lanes = lanes;
    a.per_lane = per;
    const int64_t waves = (a.T + 64 / L - 1) / (64 / L);
    const dim3 grid((unsigned)std::min<int64_t>((waves + 3) / 4, kMaxRowGrid));
    const size_t lds = a.groups > 1 ? 4 * (size_t)(a.E + a.groups) * sizeof(double) : 0;   // for gate_row_exact
    hipLaunchKernelGGL((gate_lanes_kernel<L, PL>), grid, dim3(256), lds, st, a);
    return true;
}

template <int PL>
void launch_exact(const GateArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)std::min<int64_t>((a.T + 3) / 4, kMaxRowGrid));
    const size_t lds = a.groups > 1 ? 4 * (size_t)(a.E + a.groups) * sizeof(double) : 0;   // at most 64 KB
    hipLaunchKernelGGL(gate_exact_kernel<PL>, grid, dim3(256), lds, st, a);
}

int launch_gate(GateArgs a, hipStream_t st) {
    // the lane layouts that hold the gate, the narrowest first; else (more groups than lanes) one wave per token
    // in fp64 throughout
    if (!((a.E <= 256 && (launch_lanes<16, 4>(a, st) || launch_lanes<16, 8>(a, st) || launch_lanes<16, 16>(a, st))) ||
          (a.E <= 512 && launch_lanes<64, 8>(a, st)) || launch_lanes<64, 16>(a, st))) {
        if (a.E <= 256) launch_exact<4>(a, st);
        else if (a.E <= 512) launch_exact<8>(a, st);
        else launch_exact<16>(a, st);
    }
    DWDP_LAUNCHED();
    return DWDP_OK;
}

}  // namespace
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
    return launch_gate(gate_args(logits, balance_bias, T, E, *gate, topk_idx, topk_w), as_stream(stream));
}

extern "C" size_t dwdp_route_gate_workspace_bytes(int64_t T, int H, int E, int in_dtype) {
    (void)T, (void)H, (void)E, (void)in_dtype;
    return 0;
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
    hipStream_t st = as_stream(stream);
    rc = router_logits(x, w_router, in_dtype, bias, T, H, E, logits_out, st);
    if (rc != DWDP_OK) return rc;
    return launch_gate(gate_args(logits_out, balance_bias, T, E, *gate, topk_idx, topk_w), st);
}
