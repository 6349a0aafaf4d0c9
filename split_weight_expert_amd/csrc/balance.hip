// The load of a batch's experts as a loss, and the gate's gradient (dwdp_balance_loss, dwdp_gate_backward).  The
// definitions stand in include/dwdp_layer.h.
//
// Both passes cut every sequence into chunks of `chunk` tokens, one workgroup each, from the offsets on the device:
// sequence s starts at chunk offsets[s] / chunk + s, which leaves room for all of its chunks, since
// floor((a + n) / c) + 1 >= floor(a / c) + ceil(n / c).  The loss pass leaves one row of sums per chunk in the
// workspace and a second launch adds a sequence's rows in their order, so no atomic decides a float's bits.
#include <algorithm>

#include "../../include/dwdp_layer.h"
#include "common.h"
#include "gate.h"
#include "internal.h"
#include "rows.h"

namespace dwdp {
namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxSeqs = 1 << 20;
constexpr int kThreads = 512;
constexpr float kNegInf = -__builtin_huge_valf();

struct BalanceArgs {
    const float* logits;              // [T,E]
    const int32_t* idx;               // [T,k]
    int64_t T;
    int E, k, S;
    bool sigmoid;
    const int32_t* offsets;           // [S+1] or null (one sequence)
    int chunk, n_chunks;
    // loss
    float* part_p;                    // [n_chunks][E] sums of p
    int32_t* part_n;                  // [n_chunks][E] counts
    float* part_z;                    // [n_chunks] sums of logsumexp^2
    int32_t* counts;                  // [S][E]; read by the gradient
    float* probs;
    float* balance;
    float* z;                         // or null
    // gradient
    const float* d_w;                 // each or null
    const float* d_balance;
    const float* d_z;
    bool renorm;
    float scale;
    float* d_logits;
};

// First token of sequence s, for s in [0, S].
__device__ __forceinline__ int64_t seq_start(const BalanceArgs& a, int s) {
    if (a.offsets == nullptr) return s == 0 ? 0 : a.T;
    const int64_t o = a.offsets[s];
    return o < 0 ? 0 : o > a.T ? a.T : o;
}

// The gradient covers the tokens of no sequence too: runs 0 .. S+1 are those before the first, the sequences, and
// those behind the last.
__device__ __forceinline__ int64_t run_start(const BalanceArgs& a, int r) {
    return r == 0 ? 0 : r == a.S + 2 ? a.T : seq_start(a, r - 1);
}

template <bool RUNS>
__device__ __forceinline__ int64_t part_start(const BalanceArgs& a, int s) {
    return RUNS ? run_start(a, s) : seq_start(a, s);
}

// The sequence (run) of this workgroup's chunk, and the chunk's tokens [first, last).
template <bool RUNS>
__device__ __forceinline__ int find_chunk(const BalanceArgs& a, int64_t* first, int64_t* last) {
    const int c = blockIdx.x, n = RUNS ? a.S + 2 : a.S;
    int lo = 0, hi = n - 1;
    while (lo < hi) {                          // the last one that starts at or before chunk c
        const int mid = (lo + hi + 1) / 2;
        if (part_start<RUNS>(a, mid) / a.chunk + mid <= c) lo = mid;
        else hi = mid - 1;
    }
    const int64_t start = part_start<RUNS>(a, lo), end = part_start<RUNS>(a, lo + 1);
    *first = start + (c - (start / a.chunk + lo)) * (int64_t)a.chunk;
    *last = min(*first + a.chunk, end);
    return lo;
}

// One token's probabilities, LANES lanes of PL experts each (expert lane + LANES u).
template <int PL, int LANES>
struct TokenProbs {
    float l[PL];          // logits; -inf where an expert takes no part
    float soft[PL];       // softmax(l)
    float p[PL];          // soft, or normalised sigmoids
    float slope[PL];      // 1, or 1 - sigmoid(l)
    float top, inv;       // largest logit; 1 / sum of e^(l - top)
    float lse;            // logsumexp(l), 0 for a token without a live logit
};

// A sigmoid's e^l / (1 + e^l) is e^l to fp32's last bit where every logit is below this, and there the sigmoids'
// shares are a softmax's, whatever underflows.
constexpr float kTiny = -30.0f;

template <int LANES>
__device__ __forceinline__ float row_fmax(float v) {
    // as integers whose order is the floats' (no NaN comes here)
    const uint32_t b = __float_as_uint(v);
    const uint32_t m = row_max<LANES>(b & 0x80000000u ? ~b : b | 0x80000000u);
    return __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
}

__device__ __forceinline__ float exp_from(float l, float top) { return l == top ? 1.0f : __expf(l - top); }

__device__ __forceinline__ void sigmoid_of(float l, float* s, float* one_minus_s) {
    const float e = __expf(-fabsf(l)), r = 1.0f / (1.0f + e);
    *s = l >= 0.0f ? r : e * r;
    *one_minus_s = l >= 0.0f ? e * r : r;
}

template <int PL, int LANES>
__device__ __forceinline__ void token_probs(const BalanceArgs& a, TokenProbs<PL, LANES>& t) {
    float top = kNegInf;
#pragma unroll
    for (int u = 0; u < PL; ++u) top = fmaxf(top, t.l[u]);
    top = row_fmax<LANES>(top);
    t.top = top;
    if (top == kNegInf) {
        t.lse = t.inv = 0.0f;
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            t.soft[u] = t.p[u] = 0.0f;
            t.slope[u] = 1.0f;
        }
        return;
    }
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < PL; ++u) {
        t.soft[u] = t.l[u] == kNegInf ? 0.0f : exp_from(t.l[u], top);
        sum += t.soft[u];
    }
    sum = row_sum<LANES>(sum);
    t.lse = top + __logf(sum);
    t.inv = 1.0f / sum;
#pragma unroll
    for (int u = 0; u < PL; ++u) {
        t.soft[u] *= t.inv;
        t.p[u] = t.soft[u];
        t.slope[u] = 1.0f;
    }
    if (a.sigmoid && top >= kTiny) {
        float total = 0.0f;
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            t.p[u] = 0.0f;
            if (t.l[u] > kNegInf) sigmoid_of(t.l[u], &t.p[u], &t.slope[u]);
            total += t.p[u];
        }
        const float f = 1.0f / row_sum<LANES>(total);
#pragma unroll
        for (int u = 0; u < PL; ++u) t.p[u] *= f;
    }
}

template <int PL, int LANES>
__device__ __forceinline__ void load_logits(const BalanceArgs& a, int64_t tok, int lane, float* l) {
#pragma unroll
    for (int u = 0; u < PL; ++u) {
        const int e = lane + LANES * u;
        const float v = e < a.E ? a.logits[tok * a.E + e] : kNegInf;
        l[u] = v == v ? v : kNegInf;           // NaN
    }
}

// Sums of one chunk: lanes add their experts' probabilities over the tokens, then the token groups meet in LDS.
template <int PL, int LANES>
__global__ __launch_bounds__(kThreads) void balance_chunk_kernel(BalanceArgs a) {
    constexpr int R = kThreads / LANES;        // tokens at a time
    __shared__ float s_p[R * LANES * PL];
    __shared__ float s_z[R];
    __shared__ int s_n[kMaxE];
    int64_t first, last;
    find_chunk<false>(a, &first, &last);
    if (first >= last) return;
    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    for (int e = tid; e < a.E; e += kThreads) s_n[e] = 0;
    __syncthreads();
    for (int64_t i = first * a.k + tid; i < last * a.k; i += kThreads) {
        const int e = a.idx[i];
        if (e >= 0 && e < a.E) atomicAdd(&s_n[e], 1);
    }
    float sum[PL], zsum = 0.0f;
#pragma unroll
    for (int u = 0; u < PL; ++u) sum[u] = 0.0f;
    for (int64_t t = first + group; t < last; t += R) {
        TokenProbs<PL, LANES> tp;
        load_logits<PL, LANES>(a, t, lane, tp.l);
        token_probs(a, tp);
#pragma unroll
        for (int u = 0; u < PL; ++u) sum[u] += tp.p[u];
        zsum += tp.lse * tp.lse;
    }
#pragma unroll
    for (int u = 0; u < PL; ++u) s_p[group * (LANES * PL) + u * LANES + lane] = sum[u];
    if (lane == 0) s_z[group] = zsum;
    __syncthreads();
    const int64_t row = (int64_t)blockIdx.x * a.E;
    for (int e = tid; e < a.E; e += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int g = 0; g < R; ++g) v += s_p[g * (LANES * PL) + e];
        a.part_p[row + e] = v;
        a.part_n[row + e] = s_n[e];
    }
    if (tid == 0) {
        float v = 0.0f;
        for (int g = 0; g < R; ++g) v += s_z[g];
        a.part_z[blockIdx.x] = v;
    }
}

// One sequence: its chunks' rows added in order, `width` experts side by side and 1024 / width rows at a time.
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a, int width) {
    __shared__ double s_p[1024];
    __shared__ float s_b[16];
    __shared__ int s_n[1024];
    const int s = blockIdx.x, tid = threadIdx.x, e = tid % width, part = tid / width, parts = 1024 / width;
    const int64_t start = seq_start(a, s), n = max((int64_t)0, seq_start(a, s + 1) - start);
    const int c0 = (int)(start / a.chunk) + s, nc = (int)((n + a.chunk - 1) / a.chunk);
    double p = 0.0;
    int cnt = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int c = part; c < nc; c += parts) {
            p += a.part_p[(int64_t)(c0 + c) * a.E + e];
            cnt += a.part_n[(int64_t)(c0 + c) * a.E + e];
        }
    }
    s_p[tid] = p;
    s_n[tid] = cnt;
    __syncthreads();
    float b = 0.0f;
    if (part == 0 && e < a.E) {
        for (int i = 1; i < parts; ++i) {
            p += s_p[i * width + e];
            cnt += s_n[i * width + e];
        }
        const float mean = n > 0 ? (float)(p / (double)n) : 0.0f;
        a.counts[(int64_t)s * a.E + e] = cnt;
        a.probs[(int64_t)s * a.E + e] = mean;
        b = n > 0 ? (float)cnt / (float)n * ((float)a.E / (float)a.k) * mean : 0.0f;
    }
    b = row_sum<64>(b);
    if ((tid & 63) == 0) s_b[tid >> 6] = b;
    float z = 0.0f;
    if (a.z != nullptr && tid < 64) {
        double sum = 0.0;
        for (int c = tid; c < nc; c += 64) sum += a.part_z[c0 + c];
        z = row_sum<64>((float)sum);
    }
    __syncthreads();
    if (tid == 0) {
        float v = 0.0f;
        for (int i = 0; i < 16; ++i) v += s_b[i];
        a.balance[s] = v;
        if (a.z != nullptr) a.z[s] = n > 0 ? z / (float)n : 0.0f;
    }
}

// Gradient of one chunk's tokens: LANES lanes hold a token's row from the read of its logits to the write of its
// gradient; lane j < k holds slot j (k <= LANES).
template <int PL, int LANES>
__global__ __launch_bounds__(kThreads) void gate_backward_kernel(BalanceArgs a) {
    constexpr int R = kThreads / LANES;
    int64_t first, last;
    const int run = find_chunk<true>(a, &first, &last);
    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    // what the sequence gives to each of its tokens
    float f[PL], gb = 0.0f, gz = 0.0f;
#pragma unroll
    for (int u = 0; u < PL; ++u) f[u] = 0.0f;
    if (first < last && run >= 1 && run <= a.S) {
        const int s = run - 1;
        const float inv = 1.0f / (float)(seq_start(a, s + 1) - seq_start(a, s));
        if (a.d_balance != nullptr) {
            gb = a.d_balance[s] * inv;
            const float w = inv * ((float)a.E / (float)a.k);
#pragma unroll
            for (int u = 0; u < PL; ++u) {
                const int e = lane + LANES * u;
                if (e < a.E) f[u] = (float)a.counts[(int64_t)s * a.E + e] * w;
            }
        }
        if (a.d_z != nullptr) gz = a.d_z[s] * inv;
    }
    for (int64_t t = first + group; t < last; t += R) {
        TokenProbs<PL, LANES> tp;
        load_logits<PL, LANES>(a, t, lane, tp.l);
        int e_j = -1;
        float l_j = kNegInf, g_j = 0.0f;
        if (a.d_w != nullptr && lane < a.k) {
            e_j = a.idx[t * a.k + lane];
            g_j = a.d_w[t * a.k + lane];
            if (e_j >= 0 && e_j < a.E) l_j = a.logits[t * a.E + e_j];
            if (!(l_j > kNegInf)) {                    // no expert, or one that takes no part
                e_j = -1;
                l_j = kNegInf;
                g_j = 0.0f;
            }
        }
        token_probs(a, tp);
        float d[PL], fp = 0.0f;
#pragma unroll
        for (int u = 0; u < PL; ++u) fp += f[u] * tp.p[u];
        fp = row_sum<LANES>(fp);
        const float gl = gz * 2.0f * tp.lse;
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            d[u] = gb * tp.p[u] * tp.slope[u] * (f[u] - fp);
            if (a.d_z != nullptr) d[u] += gl * tp.soft[u];
            if (tp.l[u] == kNegInf) d[u] = 0.0f;
        }
        if (a.d_w != nullptr) {
            float score = 0.0f, slope = 1.0f;
            if (a.renorm) {
                // shares among the chosen; all of them tiny: those of the limit
                const float top = row_fmax<LANES>(l_j);
                if (l_j > kNegInf) {
                    if (a.sigmoid && top >= kTiny) sigmoid_of(l_j, &score, &slope);
                    else score = exp_from(l_j, top);
                }
                const float sum = row_sum<LANES>(score);
                score = sum > 0.0f ? score / sum : 0.0f;
                g_j -= row_sum<LANES>(g_j * score);
            } else if (l_j > kNegInf) {
                if (a.sigmoid) sigmoid_of(l_j, &score, &slope);
                else score = exp_from(l_j, tp.top) * tp.inv;
            }
            const float d_j = a.scale * g_j * score * slope;
            if (!a.renorm && !a.sigmoid) {
                const float all = row_sum<LANES>(d_j);
#pragma unroll
                for (int u = 0; u < PL; ++u) d[u] -= tp.soft[u] * all;
            }
            for (int j = 0; j < a.k; ++j) {
                const int e = __shfl(e_j, j, LANES);
                const float v = __shfl(d_j, j, LANES);
#pragma unroll
                for (int u = 0; u < PL; ++u)
                    if (e == lane + LANES * u) d[u] += v;
            }
        }
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int e = lane + LANES * u;
            if (e < a.E) a.d_logits[t * a.E + e] = d[u];
        }
    }
}

// Experts a lane: a token takes 16 lanes up to 16 experts, 32 up to 32, a wave beyond.
template <typename F>
void with_layout(int E, F go) {
    if (E <= 16) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
    else if (E <= 32) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{});
    else if (E <= 64) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 64>{});
    else if (E <= 128) go(std::integral_constant<int, 2>{}, std::integral_constant<int, 64>{});
    else if (E <= 256) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 64>{});
    else if (E <= 512) go(std::integral_constant<int, 8>{}, std::integral_constant<int, 64>{});
    else go(std::integral_constant<int, 16>{}, std::integral_constant<int, 64>{});
}

// Tokens of a chunk: about 256 chunks, one a compute unit, of at most 4096 tokens, whose fp32 sums stay short.
int loss_chunk(int64_t T) { return (int)std::min<int64_t>(std::max<int64_t>(8, (T + 255) / 256), 4096); }
int64_t loss_chunks(int64_t T, int S) { return T / loss_chunk(T) + S; }

// Gradient: no sums to leave, so chunks are what a workgroup takes at a time until the launch is large.
int grad_chunk(int64_t T, int E) {
    const int64_t at_once = E <= 16 ? 32 : E <= 32 ? 16 : 8;
    return (int)((T + 65536 * at_once - 1) / (65536 * at_once) * at_once);
}

struct LossWs {
    size_t p, n, z, total;
};
LossWs loss_ws(int64_t T, int E, int S) {
    auto align = [](size_t v) { return (v + 255) & ~(size_t)255; };
    // no fewer than loss_chunks(T, S), and growing with T
    const size_t rows = (size_t)(std::max(std::min<int64_t>(T / 8, 256), T / 4096) + S);
    LossWs w{};
    w.n = align(rows * E * 4);
    w.z = w.n + align(rows * E * 4);
    w.total = w.z + align(rows * 4);
    return w;
}

int check_batch(const char* fn, int64_t T, int E, int k, const int32_t* seq_offsets, int S) {
    auto bad = [&](const char* what) { return fail(DWDP_ERR_INVALID_ARG, std::string(fn) + ": " + what); };
    if (T < 0 || T >= (int64_t)1 << 31 || T * k >= (int64_t)1 << 31) return bad("T out of range");
    if (S < 1 || S > kMaxSeqs) return bad("S must be in [1, 2^20]");
    if (seq_offsets == nullptr && S != 1) return bad("S must be 1 without seq_offsets");
    if (!type_aligned(seq_offsets, 4)) return bad("a pointer is not aligned to 4 bytes");
    return DWDP_OK;
}

}  // namespace
}  // namespace dwdp

using namespace dwdp;

extern "C" size_t dwdp_balance_loss_workspace_bytes(int64_t T, int E, int S) {
    if (T < 0 || T >= (int64_t)1 << 31 || E < 1 || E > kMaxE || S < 1 || S > kMaxSeqs) return 0;
    return loss_ws(T, E, S).total;
}

extern "C" int dwdp_balance_loss(const float* logits, const int32_t* topk_idx, int64_t T, int E, int k, int score,
                                 const int32_t* seq_offsets, int S, int32_t* counts, float* probs, float* balance,
                                 float* z, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    const dwdp_gate g{score, k, 1, 1, 1, 1, 1.0f};
    int rc = check_gate(__func__, &g, E);
    if (rc == DWDP_OK) rc = check_batch(__func__, T, E, k, seq_offsets, S);
    if (rc != DWDP_OK) return rc;
    DWDP_REQUIRE(counts && probs && balance && (T == 0 || (logits && topk_idx)), "null pointer argument");
    DWDP_REQUIRE(type_aligned(logits, 4) && type_aligned(topk_idx, 4) && type_aligned(counts, 4) &&
                     type_aligned(probs, 4) && type_aligned(balance, 4) && type_aligned(z, 4),
                 "a pointer is not aligned to 4 bytes");
    const LossWs w = loss_ws(T, E, S);
    DWDP_REQUIRE(ws != nullptr && aligned16(ws), "ws is NULL or not 16-byte aligned");
    if (ws_bytes < w.total)
        return fail(DWDP_ERR_WORKSPACE, "dwdp_balance_loss: workspace too small (need " + std::to_string(w.total) + ")");
    const size_t se = (size_t)S * E * 4;
    const Span outs[] = {{counts, se}, {probs, se}, {balance, (size_t)S * 4}, {z, (size_t)S * 4}, {ws, w.total}};
    const Span ins[] = {{logits, (size_t)T * E * 4}, {topk_idx, (size_t)T * k * 4},
                        {seq_offsets, ((size_t)S + 1) * 4}};
    DWDP_REQUIRE(!overlap_any(outs, 5, ins, 3), "an output or ws overlaps another buffer");
    BalanceArgs a{};
    a.logits = logits;
    a.idx = topk_idx;
    a.T = T;
    a.E = E;
    a.k = k;
    a.S = S;
    a.sigmoid = score == DWDP_SCORE_SIGMOID;
    a.offsets = seq_offsets;
    a.chunk = loss_chunk(T);
    a.n_chunks = (int)loss_chunks(T, S);
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.part_p = reinterpret_cast<float*>(base + w.p);
    a.part_n = reinterpret_cast<int32_t*>(base + w.n);
    a.part_z = reinterpret_cast<float*>(base + w.z);
    a.counts = counts;
    a.probs = probs;
    a.balance = balance;
    a.z = z;
    hipStream_t st = as_stream(stream);
    if (T > 0) {
        with_layout(E, [&](auto pl, auto lanes) {
            hipLaunchKernelGGL((balance_chunk_kernel<decltype(pl)::value, decltype(lanes)::value>), dim3(a.n_chunks),
                               dim3(kThreads), 0, st, a);
        });
    }
    int width = 64;
    while (width < E) width *= 2;
    hipLaunchKernelGGL(balance_finish_kernel, dim3(S), dim3(1024), 0, st, a, width);
    DWDP_LAUNCHED();
    return DWDP_OK;
}

extern "C" int dwdp_gate_backward(const float* logits, const int32_t* topk_idx, int64_t T, int E, const dwdp_gate* gate,
                                  const float* d_w, const int32_t* seq_offsets, int S, const int32_t* counts,
                                  const float* d_balance, const float* d_z, float* d_logits, void* stream) {
    clear_error();
    int rc = check_gate(__func__, gate, E);
    if (rc == DWDP_OK) rc = check_batch(__func__, T, E, gate->k, seq_offsets, S);
    if (rc != DWDP_OK) return rc;
    if (T == 0) return DWDP_OK;
    DWDP_REQUIRE(d_w || d_balance || d_z, "one of d_w, d_balance and d_z must be given");
    DWDP_REQUIRE(counts || !d_balance, "d_balance needs counts");
    DWDP_REQUIRE(logits && d_logits && (topk_idx || !d_w), "null pointer argument");
    DWDP_REQUIRE(type_aligned(logits, 4) && type_aligned(topk_idx, 4) && type_aligned(d_w, 4) && type_aligned(counts, 4) &&
                     type_aligned(d_balance, 4) && type_aligned(d_z, 4) && type_aligned(d_logits, 4),
                 "a pointer is not aligned to 4 bytes");
    const int k = gate->k;
    const size_t te = (size_t)T * E * 4, tk = (size_t)T * k * 4, s4 = (size_t)S * 4;
    const Span outs[] = {{d_logits, te}};
    const Span ins[] = {{logits, te}, {topk_idx, tk}, {d_w, tk}, {seq_offsets, s4 + 4}, {counts, s4 * E}, {d_balance, s4},
                        {d_z, s4}};
    DWDP_REQUIRE(!overlap_any(outs, 1, ins, 7), "d_logits overlaps another buffer");
    BalanceArgs a{};
    a.logits = logits;
    a.idx = topk_idx;
    a.T = T;
    a.E = E;
    a.k = k;
    a.S = S;
    a.sigmoid = gate->score == DWDP_SCORE_SIGMOID;
    a.offsets = seq_offsets;
    a.chunk = grad_chunk(T, E);
    a.n_chunks = (int)(T / a.chunk + S + 2);
    a.counts = const_cast<int32_t*>(counts);
    a.d_w = d_w;
    a.d_balance = d_balance;
    a.d_z = d_z;
    a.renorm = gate->renormalize != 0;
    a.scale = gate->scale;
    a.d_logits = d_logits;
    hipStream_t st = as_stream(stream);
    with_layout(E, [&](auto pl, auto lanes) {
        hipLaunchKernelGGL((gate_backward_kernel<decltype(pl)::value, decltype(lanes)::value>), dim3(a.n_chunks),
                           dim3(kThreads), 0, st, a);
    });
    DWDP_LAUNCHED();
    return DWDP_OK;
}
