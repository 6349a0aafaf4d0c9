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
constexpr int kThreads = 512;          // of the loss's workgroups
constexpr int kGradThreads = 256;
constexpr int64_t kGradWgs = 1024;
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
    float* part_p;                    // [n_chunks][E rounded up to 4] sums of p
    int32_t* part_n;                  // the same, counts
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
__device__ __forceinline__ uint32_t seq_start(const BalanceArgs& a, int s) {
    if (a.offsets == nullptr) return s == 0 ? 0 : (uint32_t)a.T;
    return (uint32_t)min(max(a.offsets[s], 0), (int)a.T);
}

// The gradient covers the tokens of no sequence too: runs 0 .. S+1 are those before the first, the sequences, and
// those behind the last.
__device__ __forceinline__ uint32_t run_start(const BalanceArgs& a, int r) {
    return r == 0 ? 0 : r == a.S + 2 ? (uint32_t)a.T : seq_start(a, r - 1);
}

template <bool RUNS>
__device__ __forceinline__ uint32_t part_start(const BalanceArgs& a, int s) {
    return RUNS ? run_start(a, s) : seq_start(a, s);
}

// The sequence (run) of this workgroup's chunk, and the chunk's tokens [first, last).
template <bool RUNS>
__device__ __forceinline__ int find_chunk(const BalanceArgs& a, int64_t* first, int64_t* last) {
    constexpr int kWg = RUNS ? kGradThreads : kThreads;
    const int c = blockIdx.x, n = RUNS ? a.S + 2 : a.S;
    const uint32_t chunk = a.chunk;
    // the last one that starts at or before chunk c: every thread asks for its own, which costs one read's latency, or,
    // where there are many, one search
    int lo = 0;
    if (n <= 4 * kWg) {
        for (int s = threadIdx.x; s - (int)threadIdx.x < n; s += kWg) {
            const bool before = s > 0 && s < n && (int)(part_start<RUNS>(a, s) / chunk) + s <= c;
            lo += __syncthreads_count(before);
        }
    } else {
        int hi = n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if ((int)(part_start<RUNS>(a, mid) / chunk) + mid <= c) lo = mid;
            else hi = mid - 1;
        }
    }
    const uint32_t start = part_start<RUNS>(a, lo), end = part_start<RUNS>(a, lo + 1);
    *first = start + (int64_t)(c - ((int)(start / chunk) + lo)) * chunk;
    *last = min(*first + chunk, (int64_t)end);
    return lo;
}

// One token's probabilities, LANES lanes of PL experts each (expert lane + LANES u).
template <int PL, int LANES>
struct TokenProbs {
    float l[PL];          // logits; -inf where an expert takes no part
    float soft[PL];       // softmax(l)
    float p[PL];          // soft, or normalised sigmoids
    float slope[PL];      // 1, or 1 - sigmoid(l)
    float top, inv;       // largest logit; softmax: 1 / sum of e^(l - top)
    float lse;            // logsumexp(l), 0 for a token without a live logit
};

// Orders the LDS accesses of one wave.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A sigmoid's e^l / (1 + e^l) is e^l to fp32's last bit where every logit is below this, and there the sigmoids'
// shares are a softmax's, whatever underflows.
constexpr float kTiny = -30.0f;

// Where all logits are below this, a token's largest (from 0 on) are near enough to 0 for __expf: 10 2^-24 at most.
constexpr float kNear = 8.0f;

template <int LANES>
__device__ __forceinline__ float row_fmax(float v) {
    // as integers whose order is the floats' (no NaN comes here)
    const uint32_t b = __float_as_uint(v);
    const uint32_t m = row_max<LANES>(b & 0x80000000u ? ~b : b | 0x80000000u);
    return __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
}

// Every division is by the hardware reciprocal (1 ulp): the exact one's ten instructions were a third of these kernels.
__device__ __forceinline__ float rcp(float v) { return __builtin_amdgcn_rcpf(v); }

// e^(l - top), where top may be +inf.
__device__ __forceinline__ float exp_from(float l, float top) { return l == top ? 1.0f : __expf(l - top); }

// e^l for l up to 88, to three roundings; 0 where it is below fp32's range, as for -inf.  The rounded exponent of __expf
// loses up to 1.1 |l| 2^-24 more: 5e-6 of a sigmoid's slope and of a softmax's share at l = 80.
__device__ __forceinline__ float exp_of(float l) {
    l = fmaxf(l, -200.0f);
    const float t = l * 1.44269504f;
    const float rest = fmaf(t, 1.90465421e-9f, fmaf(t, -0.693147182f, l));       // l - t ln 2
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, rest, e);
}

// -inf gives 0 and 1, +inf 1 and 0.
__device__ __forceinline__ void sigmoid_of(float l, float* s, float* one_minus_s) {
    const float e = exp_of(-fabsf(l)), r = rcp(1.0f + e), er = e * r;
    *s = l >= 0.0f ? r : er;
    *one_minus_s = l >= 0.0f ? er : r;
}

template <int PL, int LANES>
__device__ __forceinline__ void token_probs(const BalanceArgs& a, TokenProbs<PL, LANES>& t) {
    float top = t.l[0];
#pragma unroll
    for (int u = 1; u < PL; ++u) top = fmaxf(top, t.l[u]);
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
    if (a.sigmoid && top >= 0.0f && top < 80.0f) {
        // x = e^l does for both: x / (1 + x) and x / sum of x; what underflows is below 2^-126 of the sum.  The loss of
        // 65536 x 256, us: 29.0 with __expf for every token, 30.4 with this choice, 33.5 with exp_of for every token.
        float total = 0.0f;
        auto add = [&](auto exp) {
#pragma unroll
            for (int u = 0; u < PL; ++u) {
                const float x = exp(t.l[u]);
                t.slope[u] = rcp(1.0f + x);
                t.p[u] = x * t.slope[u];
                t.soft[u] = x;
                sum += x;
                total += t.p[u];
            }
        };
        if (top < kNear) add([](float l) { return __expf(l); });
        else add([](float l) { return exp_of(l); });
        sum = row_sum<LANES>(sum);
        t.lse = __logf(sum);
        const float inv = rcp(sum), f = rcp(row_sum<LANES>(total));
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            t.soft[u] *= inv;
            t.p[u] *= f;
        }
        return;
    }
    if (top < __builtin_huge_valf()) {
#pragma unroll
        for (int u = 0; u < PL; ++u) sum += t.soft[u] = __expf(t.l[u] - top);      // 0 for -inf
    } else {
#pragma unroll
        for (int u = 0; u < PL; ++u) sum += t.soft[u] = t.l[u] == top ? 1.0f : 0.0f;
    }
    sum = row_sum<LANES>(sum);
    t.lse = top + __logf(sum);
    t.inv = rcp(sum);
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
            sigmoid_of(t.l[u], &t.p[u], &t.slope[u]);
            total += t.p[u];
        }
        const float f = rcp(row_sum<LANES>(total));
#pragma unroll
        for (int u = 0; u < PL; ++u) t.p[u] *= f;
    }
}

// Reads are issued here and looked at in live_logits: a NaN, and what is behind the last expert, takes no part.
template <int PL, int LANES>
__device__ __forceinline__ void live_logits(const BalanceArgs& a, int lane, float* l) {
#pragma unroll
    for (int u = 0; u < PL; ++u) l[u] = lane + LANES * u < a.E ? fmaxf(l[u], kNegInf) : kNegInf;
}

template <int PL, int LANES>
__device__ __forceinline__ void load_logits(const BalanceArgs& a, int64_t tok, int lane, float* l) {
    // the last expert's in the place of those behind it, so that no branch parts the reads
    const float* row = a.logits + tok * a.E;
#pragma unroll
    for (int u = 0; u < PL; ++u) l[u] = row[min(lane + LANES * u, a.E - 1)];
}

// Bound by latency up to some thousand tokens (an empty kernel takes 2.3 us, two of them and their parts' dependent reads
// 7 us), and by vector instructions on the compute units that have a chunk beyond: sigmoids, 256 experts, 65536 tokens are
// 67 MB in 30 us, 132 workgroups whose units' SIMDs are 82% busy, while the others have none (kLossChunks).  16384 tokens
// in four sequences 14.3 us, of which the second launch takes 5.  Before (a wave a token, exact divisions, reads parted by
// branches) 25.9 us.
//
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
    // the first token's reads are on their way while the counts are cleared; the next one's while one is summed
    float next[PL], sum[PL], zsum = 0.0f;
    int e_next = -1;
    auto fetch = [&](int64_t t) {
        if (t >= last) return;
        load_logits<PL, LANES>(a, t, lane, next);
        if (lane < a.k) e_next = a.idx[t * a.k + lane];
    };
    fetch(first + group);
    for (int e = tid; e < kMaxE; e += kThreads) s_n[e] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PL; ++u) sum[u] = 0.0f;
    for (int64_t t = first + group; t < last; t += R) {
        TokenProbs<PL, LANES> tp;
#pragma unroll
        for (int u = 0; u < PL; ++u) tp.l[u] = next[u];
        const int e = e_next;
        fetch(t + R);
        live_logits<PL, LANES>(a, lane, tp.l);
        if (lane < a.k && e >= 0 && e < a.E) atomicAdd(&s_n[e], 1);
        token_probs(a, tp);
#pragma unroll
        for (int u = 0; u < PL; ++u) sum[u] += tp.p[u];
        zsum += tp.lse * tp.lse;
    }
#pragma unroll
    for (int u = 0; u < PL; ++u) s_p[group * (LANES * PL) + u * LANES + lane] = sum[u];
    if (lane == 0) s_z[group] = zsum;
    __syncthreads();
    const int E4 = (a.E + 3) & ~3;
    const int64_t row = (int64_t)blockIdx.x * E4;
    for (int e = tid; e < E4; e += kThreads) {
        float v = 0.0f;
        if (e < LANES * PL) {
#pragma unroll
            for (int g = 0; g < R; ++g) v += s_p[g * (LANES * PL) + e];      // 0 behind the last expert
        }
        a.part_p[row + e] = v;
        a.part_n[row + e] = s_n[e];
    }
    if (tid == 0) {
        float v = 0.0f;
        for (int g = 0; g < R; ++g) v += s_z[g];
        a.part_z[blockIdx.x] = v;
    }
}

// One sequence: its chunks' rows added, four experts a thread, `width` threads side by side and 1024 / width rows at a
// time; the sums of a chunk are fp32, those over chunks fp64.
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceArgs a, int width) {
    __shared__ double s_p[4 * 1024];
    __shared__ int s_n[4 * 1024];
    __shared__ float s_b[16];
    const int s = blockIdx.x, tid = threadIdx.x, col = tid % width, part = tid / width, parts = 1024 / width;
    const int E4 = (a.E + 3) & ~3;
    const uint32_t start = seq_start(a, s), end = seq_start(a, s + 1), n = end > start ? end - start : 0;
    const int64_t c0 = start / (uint32_t)a.chunk + s;
    const int nc = (int)((n + a.chunk - 1) / (uint32_t)a.chunk);
    double p[4] = {0.0, 0.0, 0.0, 0.0};
    int cnt[4] = {0, 0, 0, 0};
    if (4 * col < E4) {
#pragma unroll 4
        for (int c = part; c < nc; c += parts) {
            const int64_t i = (c0 + c) * E4 + 4 * col;
            const float4 v = *reinterpret_cast<const float4*>(a.part_p + i);
            const int4 m = *reinterpret_cast<const int4*>(a.part_n + i);
            p[0] += v.x, p[1] += v.y, p[2] += v.z, p[3] += v.w;
            cnt[0] += m.x, cnt[1] += m.y, cnt[2] += m.z, cnt[3] += m.w;
        }
    }
    float z = 0.0f;
    if (a.z != nullptr && tid < 64) {
        double sum = 0.0;
        for (int c = tid; c < nc; c += 64) sum += a.part_z[c0 + c];
        z = row_sum<64>((float)sum);
    }
    // [part][4 width]
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        s_p[4 * tid + u] = p[u];
        s_n[4 * tid + u] = cnt[u];
    }
    __syncthreads();
    float b = 0.0f;
    if (tid < a.E) {
        double sum = 0.0;
        int m = 0;
        for (int i = 0; i < parts; ++i) {
            sum += s_p[i * 4 * width + tid];
            m += s_n[i * 4 * width + tid];
        }
        const float mean = n > 0 ? (float)(sum / (double)n) : 0.0f;
        a.counts[(int64_t)s * a.E + tid] = m;
        a.probs[(int64_t)s * a.E + tid] = mean;
        b = n > 0 ? (float)m / (float)n * ((float)a.E / (float)a.k) * mean : 0.0f;
    }
    b = row_sum<64>(b);
    if ((tid & 63) == 0) s_b[tid >> 6] = b;
    __syncthreads();
    if (tid == 0) {
        float v = 0.0f;
        for (int i = 0; i < 16; ++i) v += s_b[i];
        a.balance[s] = v;
        if (a.z != nullptr) a.z[s] = n > 0 ? z / (float)n : 0.0f;
    }
}

// Bound by latency, then by vector instructions (SIMDs 89% busy on the whole chip at 65536 tokens): 64 tokens of 256 experts
// 4.8 us, 16384 15.3 us (34.6 MB read and written, 2.3 TB/s), 65536 36 us (138 MB, 3.8 TB/s).
// Before (a workgroup for every eight tokens, k compares for every expert) 16384 took 23.6 us.
//
// Gradient of one chunk's tokens: LANES lanes hold a token's row from the read of its logits to the write of its
// gradient; lane j < k holds slot j (k <= LANES).
template <int PL, int LANES>
__global__ __launch_bounds__(kGradThreads) void gate_backward_kernel(BalanceArgs a) {
    constexpr int R = kGradThreads / LANES;
    __shared__ float s_row[R * LANES * PL];
    int64_t first, last;
    const int run = find_chunk<true>(a, &first, &last);
    const int tid = threadIdx.x, lane = tid % LANES, group = tid / LANES;
    // what the sequence gives to each of its tokens
    float f[PL], gb = 0.0f, gz = 0.0f;
#pragma unroll
    for (int u = 0; u < PL; ++u) f[u] = 0.0f;
    if (first < last && run >= 1 && run <= a.S) {
        const int s = run - 1;
        const float inv = 1.0f / (float)(int)(seq_start(a, s + 1) - seq_start(a, s));
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
    // the next token's reads are on their way while one is computed
    float next[PL], g_next = 0.0f;
    int e_next = -1;
    auto fetch = [&](int64_t t) {
        if (t >= last) return;
        load_logits<PL, LANES>(a, t, lane, next);
        if (a.d_w != nullptr && lane < a.k) {
            e_next = a.idx[t * a.k + lane];
            g_next = a.d_w[t * a.k + lane];
        }
    };
    fetch(first + group);
    for (int64_t t = first + group; t < last; t += R) {
        TokenProbs<PL, LANES> tp;
#pragma unroll
        for (int u = 0; u < PL; ++u) tp.l[u] = next[u];
        int e_j = e_next;
        float l_j = kNegInf, g_j = g_next;
        if (e_j >= 0 && e_j < a.E) l_j = a.logits[t * a.E + e_j];
        fetch(t + R);
        if (!(l_j > kNegInf)) {                        // no expert, or one that takes no part
            e_j = -1;
            l_j = kNegInf;
            g_j = 0.0f;
        }
        live_logits<PL, LANES>(a, lane, tp.l);
        token_probs(a, tp);
        float d[PL], fp = 0.0f;
#pragma unroll
        for (int u = 0; u < PL; ++u) fp += f[u] * tp.p[u];
        fp = row_sum<LANES>(fp);
        const float gl = gz == 0.0f ? 0.0f : gz * 2.0f * tp.lse;      // lse may be infinite where there is no loss
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            d[u] = gb * tp.p[u] * tp.slope[u] * (f[u] - fp);
            if (a.d_z != nullptr) d[u] += gl * tp.soft[u];
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
                score = sum > 0.0f ? score * rcp(sum) : 0.0f;
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
            // to the lanes that hold the experts, through the token's row in LDS, where every slot first leaves its
            // lane: one that finds another there shares its expert, and then the slots are added one by one
            float* const row = s_row + group * (PL * LANES);
            int* const who = reinterpret_cast<int*>(row);
#pragma unroll
            for (int u = 0; u < PL; ++u) row[lane + LANES * u] = 0.0f;
            wave_lds_sync();
            if (e_j >= 0) who[e_j] = lane;
            wave_lds_sync();
            const bool shared = e_j >= 0 && who[e_j] != lane;
            if (__any(shared)) {
                for (int j = 0; j < a.k; ++j) {
                    const int e = __shfl(e_j, j, LANES);
                    const float v = __shfl(d_j, j, LANES);
#pragma unroll
                    for (int u = 0; u < PL; ++u)
                        if (e == lane + LANES * u) d[u] += v;
                }
            } else {
                if (e_j >= 0) row[e_j] = d_j;
                wave_lds_sync();
#pragma unroll
                for (int u = 0; u < PL; ++u) d[u] += row[lane + LANES * u];
            }
            wave_lds_sync();                          // read before the next token's zeros
        }
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int e = lane + LANES * u;
            if (e < a.E) a.d_logits[t * a.E + e] = d[u];
        }
    }
}

// Lanes of a token and experts of a lane: 16 lanes hold up to 256 experts, so that four tokens share a wave's exchanges
// between lanes (the gradient, which keeps six numbers an expert: 8 a lane on up to 64 lanes); a few tokens, and the
// slots of k > 16, take as many lanes as the experts fill.  Loss and gradient, us, narrow against wide, sigmoid:
// 2048 x 256 12.7 + 6.3 against 12.1 + 6.0, 4096 x 256 12.9 + 7.3 against 12.6 + 7.1, 8192 x 256 13.9 + 9.2 against
// 14.2 + 10.3, 16384 x 256 14.1 + 15.3 against 16.5 + 17.4, 16384 x 60 10.2 + 7.3 against 13.4 + 12.7.
bool many_tokens(int64_t T, int k) { return T > 4096 && k <= 16; }

template <typename F>
void with_layout(int E, bool many, bool grad, F go) {
    auto as = [&](auto pl, auto lanes) { go(pl, lanes); };
    using std::integral_constant;
    if (E <= 16) return as(integral_constant<int, 1>{}, integral_constant<int, 16>{});
    if (E > 512) return as(integral_constant<int, 16>{}, integral_constant<int, 64>{});
    if (many) {
        if (E <= 32) as(integral_constant<int, 2>{}, integral_constant<int, 16>{});
        else if (E <= 64) as(integral_constant<int, 4>{}, integral_constant<int, 16>{});
        else if (E <= 128) as(integral_constant<int, 8>{}, integral_constant<int, 16>{});
        else if (grad && E <= 256) as(integral_constant<int, 8>{}, integral_constant<int, 32>{});
        else if (grad) as(integral_constant<int, 8>{}, integral_constant<int, 64>{});
        else if (E <= 256) as(integral_constant<int, 16>{}, integral_constant<int, 16>{});
        else as(integral_constant<int, 16>{}, integral_constant<int, 32>{});
    } else {
        if (E <= 32) as(integral_constant<int, 1>{}, integral_constant<int, 32>{});
        else if (E <= 64) as(integral_constant<int, 1>{}, integral_constant<int, 64>{});
        else if (E <= 128) as(integral_constant<int, 2>{}, integral_constant<int, 64>{});
        else if (E <= 256) as(integral_constant<int, 4>{}, integral_constant<int, 64>{});
        else as(integral_constant<int, 8>{}, integral_constant<int, 64>{});
    }
}

// Tokens that a workgroup of the gradient takes at a time in that layout.
int tokens_at_once(int E, bool many) {
    int n = 0;
    with_layout(E, many, true, [&](auto, auto lanes) { n = kGradThreads / decltype(lanes)::value; });
    return n;
}

// Tokens of a chunk: about 128 chunks, since one workgroup adds all of a sequence's (64, 128 and 256 of them, us: one
// sequence of 4096 x 256 12.6, 11.6, 12.8, of 8192 x 256 13.4, 12.3, 13.9; four of 16384 tokens 18.3, 14.4, 14.3), of at
// most 4096 tokens, whose fp32 sums stay short.
constexpr int64_t kLossChunks = 128;
int loss_chunk(int64_t T) { return (int)std::min<int64_t>(std::max<int64_t>(8, (T + kLossChunks - 1) / kLossChunks), 4096); }
int64_t loss_chunks(int64_t T, int S) { return T / loss_chunk(T) + S; }

// Gradient: no sums to leave, so chunks are what a workgroup takes at a time, or more where the launch has the waves to
// fill the chip all the same.
int grad_chunk(int64_t T, int E, int k) {
    const int64_t at_once = tokens_at_once(E, many_tokens(T, k));
    return (int)(at_once * std::max<int64_t>(1, T / (at_once * kGradWgs)));
}

struct LossWs {
    size_t p, n, z, total;
};
LossWs loss_ws(int64_t T, int E, int S) {
    auto align = [](size_t v) { return (v + 255) & ~(size_t)255; };
    // no fewer than loss_chunks(T, S), and growing with T
    const size_t rows = (size_t)(std::max(std::min<int64_t>(T / 8, kLossChunks), T / 4096) + S);
    LossWs w{};
    const size_t E4 = (size_t)(E + 3) & ~(size_t)3;
    w.n = align(rows * E4 * 4);
    w.z = w.n + align(rows * E4 * 4);
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
        with_layout(E, many_tokens(T, k), false, [&](auto pl, auto lanes) {
            hipLaunchKernelGGL((balance_chunk_kernel<decltype(pl)::value, decltype(lanes)::value>), dim3(a.n_chunks),
                               dim3(kThreads), 0, st, a);
        });
    }
    int width = 16;
    while (4 * width < E) width *= 2;
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
    a.chunk = grad_chunk(T, E, k);
    a.n_chunks = (int)(T / a.chunk + S + 2);
    a.counts = const_cast<int32_t*>(counts);
    a.d_w = d_w;
    a.d_balance = d_balance;
    a.d_z = d_z;
    a.renorm = gate->renormalize != 0;
    a.scale = gate->scale;
    a.d_logits = d_logits;
    hipStream_t st = as_stream(stream);
    with_layout(E, many_tokens(T, k), true, [&](auto pl, auto lanes) {
        hipLaunchKernelGGL((gate_backward_kernel<decltype(pl)::value, decltype(lanes)::value>), dim3(a.n_chunks),
                           dim3(kGradThreads), 0, st, a);
    });
    DWDP_LAUNCHED();
    return DWDP_OK;
}
