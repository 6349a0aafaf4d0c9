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
    const float* logits;
    const float* balance;             // [E] or null
    int64_t T;
    int E, k, groups, kept, group_top;
    bool sigmoid, renorm;
    float scale;
    int32_t* idx;
    float* w;
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

int launch_gate(const GateArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)std::min<int64_t>((a.T + 3) / 4, kMaxRowGrid));
    const size_t lds = a.groups > 1 ? 4 * (size_t)(a.E + a.groups) * sizeof(double) : 0;   // at most 64 KB
    if (a.E <= 64) hipLaunchKernelGGL(gate_exact_kernel<1>, grid, dim3(256), lds, st, a);
    else if (a.E <= 128) hipLaunchKernelGGL(gate_exact_kernel<2>, grid, dim3(256), lds, st, a);
    else if (a.E <= 256) hipLaunchKernelGGL(gate_exact_kernel<4>, grid, dim3(256), lds, st, a);
    else if (a.E <= 512) hipLaunchKernelGGL(gate_exact_kernel<8>, grid, dim3(256), lds, st, a);
    else hipLaunchKernelGGL(gate_exact_kernel<16>, grid, dim3(256), lds, st, a);
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
