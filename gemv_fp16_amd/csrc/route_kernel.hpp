// Routing to experts: scores, the k best, their weights, and the rows sorted by expert.
//
// A wave routes a token: lane l holds the logits of experts VPT * l .. VPT * l +
// VPT - 1, so that the lowest lane and the lowest register among equal keys is the
// lowest expert.  k rounds of a maximum over the lanes (DPP, no LDS) give the
// chosen ones, lane j keeping the j-th.
//
// Keys.  Without a bias, and without sums of two scores in a group's rank, the
// order of the scores is the order of the logits, which are compared as they are.
// Otherwise the keys are score + bias in 64 bits: in 32, an exponential's last bit
// would decide which of two close experts is taken, about once in 10^4 tokens.
//
// The sort is stable and takes no atomics whose order could show: a workgroup
// ranks the entries of its chunk of tokens by expert (per wave, 64 entries at a
// time: the lanes of equal expert by ballots over the expert's bits) and stores the
// chunk's count of each expert; a second launch adds, to each entry's rank, its
// expert's offset and the counts of the chunks before.
#pragma once
#include "wave.hpp"

namespace gf {

constexpr int kRouteMaxExperts = 1024;   // 16 logits a lane
constexpr int kRouteMaxTop = 64;         // lane j holds the j-th choice
constexpr int kRouteMaxGroups = 64;      // lane g ranks group g

struct RouteArgs {
    const void* logits;     // T x E, fp16 or fp32
    const float* bias;      // E, or null
    int* ids;               // T x k
    float* weights;         // T x k
    int T, E, k;
    int sigmoid, renorm;
    int groups, top_groups, group_best;
    float scale;
    // rows sorted by expert; chunk = tokens a workgroup
    int* offsets;           // E + 1, or null: no sort
    int* place;             // T x k
    int* counts;            // chunks x E (two launches), or null (one workgroup)
    int chunk;
};

// ---------------------------------------------------------------------------
// sort by expert
// ---------------------------------------------------------------------------

// Lanes of the wave whose id equals this lane's (all lanes call it; `live` lanes only).
__device__ __forceinline__ uint64_t same_id(int id, bool live, int bits)
{
    uint64_t m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((id >> b) & 1);
        m &= ((id >> b) & 1) ? set : ~set;
    }
    return m;
}

// Exclusive offsets of E counts in LDS, by the first wave; E + 1 entries.
__device__ __forceinline__ void scan_counts(const GF_LDS int* total, GF_LDS int* start, int E)
{
    if (threadIdx.x >= kWave) return;
    const int lane = threadIdx.x;
    int before = 0;
    for (int b = 0; b < E; b += kWave) {
        const int e = b + lane, v = e < E ? total[e] : 0, s = wave_scan(v, lane);
        if (e < E) start[e] = before + s - v;
        before += lane_value(s, kWave - 1);
    }
    if (lane == 0) start[E] = before;
}

// Ranks of n entries by id: place[i] = entries before i of the same id (plus, with
// FINAL, the id's offset among all), -1 where the id is none.  Without FINAL the
// chunk's counts go to `out`, with it the offsets.  cnt: W * E + 2 * E + 1 ints of
// LDS.  The whole workgroup calls it.
template <int W, bool FINAL>
__device__ __forceinline__ void rank_entries(const int* ids, int* place, int n, int E, GF_LDS int* cnt, int* out)
{
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    GF_LDS int* total = cnt + W * E;
    GF_LDS int* start = total + E;
    GF_LDS int* mine = cnt + wave * E;
    for (int i = tid; i < W * E; i += W * kWave) cnt[i] = 0;
    __syncthreads();
    const int seg = ceil_div(ceil_div(n, W), kWave) * kWave;
    const int lo = min(wave * seg, n), hi = min(lo + seg, n);
    for (int i = lo + lane; i < hi; i += kWave) {
        const int id = ids[i];
        if ((unsigned)id < (unsigned)E) __hip_atomic_fetch_add(&mine[id], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    for (int e = tid; e < E; e += W * kWave) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        total[e] = run;
        if (!FINAL) out[e] = run;
    }
    __syncthreads();
    if constexpr (FINAL) {
        scan_counts(total, start, E);
        __syncthreads();
        for (int e = tid; e <= E; e += W * kWave) out[e] = start[e];
    }
    const int bits = 32 - __builtin_clz(E | 1);
    for (int b = lo; b < hi; b += kWave) {
        const int i = b + lane;
        const int id = i < hi ? ids[i] : -1;
        const bool live = (unsigned)id < (unsigned)E;
        const uint64_t same = same_id(id, live, bits);
        const int rank = __builtin_popcountll(same & ((uint64_t(1) << lane) - 1));
        int at = -1;
        if (live) {
            at = mine[id] + rank;
            if (FINAL) at += start[id];
        }
        asm volatile("" ::: "memory");           // every lane has read before the first of each id counts on
        if (live && rank == 0) mine[id] += __builtin_popcountll(same);
        asm volatile("" ::: "memory");
        if (i < hi) place[i] = at;
    }
}

// Ranks alone, for ids that come from elsewhere: chunk entries a workgroup.
template <int W, bool FINAL>
__global__ __launch_bounds__(W * kWave) void rank_kernel(const int* ids, int* place, int n, int E, int chunk, int* out)
{
    extern __shared__ __attribute__((aligned(16))) char smem_raw[];
    const int lo = blockIdx.x * chunk;
    rank_entries<W, FINAL>(ids + lo, place + lo, min(chunk, n - lo), E, (GF_LDS int*)smem_raw,
                           FINAL ? out : out + (size_t)blockIdx.x * E);
}

// The second launch: the entries' offsets and the earlier chunks' counts.
__global__ __launch_bounds__(1024) void place_kernel(const int* ids, int* place, int64_t n, int E, int chunk,
                                                     const int* counts, int chunks, int* offsets)
{
    __shared__ int before[kRouteMaxExperts], total[kRouteMaxExperts], start[kRouteMaxExperts + 1];
    const int tid = threadIdx.x, c = blockIdx.x;
    for (int e = tid; e < E; e += 1024) before[e] = total[e] = 0;
    __syncthreads();
    // `parts` threads an expert, each with every parts-th chunk
    const int width = E <= 1 ? 1 : 1 << (32 - __builtin_clz(E - 1)), parts = 1024 / width;
    const int e = tid % width, part = tid / width;
    if (e < E) {
        int b = 0, t = 0;
#pragma unroll 8
        for (int i = part; i < chunks; i += parts) {
            const int v = counts[(size_t)i * E + e];
            t += v;
            b += i < c ? v : 0;
        }
        atomicAdd(&before[e], b);
        atomicAdd(&total[e], t);
    }
    __syncthreads();
    scan_counts((const GF_LDS int*)total, (GF_LDS int*)start, E);
    __syncthreads();
    if (c == 0)
        for (int i = tid; i <= E; i += 1024) offsets[i] = start[i];
    const int64_t lo = (int64_t)c * chunk, hi = lo + chunk < n ? lo + chunk : n;
    for (int64_t i = lo + tid; i < hi; i += 1024) {
        const int id = ids[i];
        if ((unsigned)id < (unsigned)E) place[i] += start[id] + before[id];
    }
}

// ---------------------------------------------------------------------------
// scores and choice
// ---------------------------------------------------------------------------

template <bool F32>
__device__ __forceinline__ float logit_at(const void* logits, size_t i)
{
    if constexpr (F32) return ((const float*)logits)[i];
    else return (float)((const _Float16*)logits)[i];
}

__device__ __forceinline__ float sigmoid_shifted(float x, float top)
{
    // sigmoid(x) / exp(min(top, 0)): no underflow where top is the largest of the row's choices
    return expf(fminf(x, 0.0f) - fminf(top, 0.0f)) / (1.0f + expf(-fabsf(x)));
}

// The weight of this lane's choice x (lanes without one: live = false); top and
// sum: the softmax's maximum and sum over all experts.
__device__ __forceinline__ float choice_weight(const RouteArgs& a, float x, bool live, float top, float sum)
{
    const float ninf = -__builtin_inff();
    float w;
    if (a.renorm) {
        // shifted by the largest chosen logit: the sum is at least a half
        const float best = wave_max(live ? x : ninf);
        w = live ? (a.sigmoid ? sigmoid_shifted(x, best) : expf(x - best)) : 0.0f;
        w /= wave_sum(w);
    } else {
        w = a.sigmoid ? sigmoid_shifted(x, 0.0f) : expf(x - top) / sum;
    }
    return live ? a.scale * w : 0.0f;
}

// Routes token t; all lanes.  KEY: float (the logits) or double (scores and bias).
// keys: E KEYs of LDS of this wave (where there are groups).
template <int VPT, class KEY, bool F32>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int lane, GF_LDS KEY* keys)
{
    const KEY ninf = -(KEY)__builtin_inf(), inf = (KEY)__builtin_inf();
    constexpr bool WIDE = sizeof(KEY) == 8;
    const int e0 = lane * VPT;
    float x[VPT];
    KEY key[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        x[i] = e0 + i < a.E ? logit_at<F32>(a.logits, (size_t)t * a.E + e0 + i) : -__builtin_inff();

    float top = 0.0f, sum = 1.0f;
    double sum64 = 1.0;
    if (!a.sigmoid && (WIDE || !a.renorm)) {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i) m = fmaxf(m, x[i]);
        top = wave_max(m);
        if constexpr (WIDE) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                key[i] = x[i] == -__builtin_inff() ? 0.0 : exp((double)x[i] - (double)top);
                s += key[i];
            }
            sum64 = wave_sum(s);
            sum = (float)sum64;
        } else {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) s += x[i] == -__builtin_inff() ? 0.0f : expf(x[i] - top);
            sum = wave_sum(s);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (WIDE) {
            double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i])) : key[i] / sum64;
            if (a.bias && e0 + i < a.E) s += (double)a.bias[e0 + i];
            key[i] = x[i] == -__builtin_inff() ? ninf : s;
        } else {
            key[i] = x[i];
        }
        if (key[i] != key[i]) key[i] = inf;
    }

    if (a.groups > 1) {
        // `parts` lanes a group (a power of two) look through its experts' keys
        const int size = a.E / a.groups;
        const int parts = 1 << (31 - __builtin_clz(kWave / a.groups));
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + i < a.E) keys[e0 + i] = key[i];
        asm volatile("" ::: "memory");
        wait_lgkmcnt0();
        const int g = lane / parts, sub = lane % parts;
        KEY first = ninf, second = ninf;
        if (g < a.groups)
            for (int i = sub; i < size; i += parts) {
                const KEY v = keys[g * size + i];
                second = v > first ? first : (v > second ? v : second);
                first = v > first ? v : first;
            }
        for (int d = 1; d < parts; d *= 2) {
            const KEY f = __shfl_xor(first, d), s = __shfl_xor(second, d);
            second = f > first ? (first > s ? first : s) : (second > f ? second : f);
            first = f > first ? f : first;
        }
        KEY mine = first;
        if (a.group_best == 2 && second > ninf) mine += second;
        int rank = 0;
        for (int h = 0; h < a.groups; ++h) {
            const KEY v = lane_value(mine, h * parts);
            rank += v > mine || (v == mine && h < g);
        }
        const uint64_t stay = __ballot(rank < a.top_groups);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + i < a.E && !((stay >> ((e0 + i) / size * parts)) & 1)) key[i] = ninf;
    }

    int id = -1;
    float xs = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        KEY best = key[0];
        int at = 0;
        float bx = x[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i)
            if (key[i] > best) { best = key[i]; at = i; bx = x[i]; }
        const KEY m = wave_max(best);
        if (m == ninf) break;
        const int src = __builtin_ctzll(__ballot(best == m));
        const int which = lane_value(at, src);
        const float cx = lane_value(bx, src);
        if (lane == j) { id = src * VPT + which; xs = cx; }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (lane == src && i == which) key[i] = ninf;
    }
    const float w = choice_weight(a, xs, id >= 0, top, sum);
    if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = id;
        a.weights[(size_t)t * a.k + lane] = w;
    }
}

// chunk tokens a workgroup of W waves, then the chunk's ranks.  FINAL: one
// workgroup does all, the offsets too.
template <int W, int VPT, class KEY, bool F32, bool FINAL>
__global__ __launch_bounds__(W * kWave) void route_kernel(RouteArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char smem_raw[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
    GF_LDS KEY* keys = (GF_LDS KEY*)smem_raw + wave * a.E;
    for (int t = t0 + wave; t < t1; t += W) route_token<VPT, KEY, F32>(a, t, lane, keys);
    if (!a.offsets) return;
    __syncthreads();                              // the ids are written, the keys read
    const size_t at = (size_t)t0 * a.k;
    rank_entries<W, FINAL>(a.ids + at, a.place + at, (t1 - t0) * a.k, a.E, (GF_LDS int*)smem_raw,
                           FINAL ? a.offsets : a.counts + (size_t)blockIdx.x * a.E);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

struct RouteGradArgs {
    const void* logits;
    const int* ids;
    const float* dweights;
    void* dlogits;
    int T, E, k;
    int sigmoid, renorm;
    float scale;
};

// dx of one token a wave.  With p the scores of all experts, r the renormalised
// ones of the chosen, g the weights' gradients times scale:
//   softmax            dx_e = p_e (g_e - sum_j g_j p_j)
//   sigmoid            dx_e = s_e (1 - s_e) g_e
//   softmax, renorm    dx_e = r_e (g_e - sum_j r_j g_j)
//   sigmoid, renorm    dx_e = r_e (1 - s_e) (g_e - sum_j r_j g_j)
// Lane j works out the j-th choice's; the lanes that hold the experts then take it
// over, so that an expert named twice gets both.
template <int VPT, bool F32>
__device__ __forceinline__ void route_grad_token(const RouteGradArgs& a, int t, int lane)
{
    const float ninf = -__builtin_inff();
    const int e0 = lane * VPT;
    const size_t row = (size_t)t * a.E;
    int id = -1;
    float g = 0.0f, xs = ninf;
    if (lane < a.k) {
        id = a.ids[(size_t)t * a.k + lane];
        if ((unsigned)id < (unsigned)a.E) {
            g = a.scale * a.dweights[(size_t)t * a.k + lane];
            xs = logit_at<F32>(a.logits, row + id);
        } else {
            id = -1;
        }
    }
    const bool live = xs != ninf;                 // a NaN is live and shows
    const bool dense = !a.sigmoid && !a.renorm;
    float d = live ? g : 0.0f;
    if (a.renorm) {
        const float best = wave_max(xs);
        float r = live ? (a.sigmoid ? sigmoid_shifted(xs, best) : expf(xs - best)) : 0.0f;
        const float sum = wave_sum(r);
        r = live ? r / sum : 0.0f;
        const float mean = wave_sum(live ? r * g : 0.0f);
        d = live ? r * (g - mean) : 0.0f;
    } else if (a.sigmoid) {
        d *= sigmoid_shifted(xs, 0.0f);
    }
    if (a.sigmoid && live) d *= sigmoid_shifted(-xs, 0.0f);     // 1 - s without cancellation
    float out[VPT] = {};
    for (int j = 0; j < a.k; ++j) {
        const int e = lane_value(id, j) - e0;
        const float v = lane_value(d, j);
#pragma unroll
        for (int i = 0; i < VPT; ++i) out[i] += e == i ? v : 0.0f;
    }
    if (dense) {
        float p[VPT], m = ninf, s = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            p[i] = e0 + i < a.E ? logit_at<F32>(a.logits, row + e0 + i) : ninf;
            m = fmaxf(m, p[i]);
        }
        m = wave_max(m);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            p[i] = p[i] == ninf ? 0.0f : expf(p[i] - m);
            s += p[i];
        }
        s = wave_sum(s);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            p[i] = p[i] == 0.0f ? 0.0f : p[i] / s;
            dot += out[i] * p[i];
        }
        dot = wave_sum(dot);
#pragma unroll
        for (int i = 0; i < VPT; ++i) out[i] = p[i] * (out[i] - dot);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (e0 + i < a.E) {
            if constexpr (F32) ((float*)a.dlogits)[row + e0 + i] = out[i];
            else ((uint16_t*)a.dlogits)[row + e0 + i] = f32_to_f16_bits(out[i]);
        }
}

template <int W, int VPT, bool F32>
__global__ __launch_bounds__(W * kWave) void route_grad_kernel(RouteGradArgs a)
{
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (int t = blockIdx.x * W + wave; t < a.T; t += gridDim.x * W) route_grad_token<VPT, F32>(a, t, lane);
}

}  // namespace gf
