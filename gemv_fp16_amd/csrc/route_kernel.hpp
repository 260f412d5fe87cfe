// Routing to experts: scores, the k best, their weights, and the rows sorted by expert.
//
// A wave routes a token, or, in the common case (QuadRouter), four, one in each row of
// 16 lanes: a lane holds the logits of VPT neighbouring experts, so that the lowest
// lane and register among equal keys is the lowest expert.  k rounds of a maximum over
// the lanes (DPP, no LDS) give the chosen ones, lane j keeping the j-th.  Bound by the
// instructions of those rounds, about 30 to one of a wave's token and 50 to one of four.
//
// Keys.  Without a bias, and without sums of two scores in a group's rank, the
// order of the scores is the order of the logits, which are compared as they are.
// Otherwise the keys are score + bias in 64 bits: in 32, an exponential's last bit
// would decide which of two close experts is taken, about once in 10^4 tokens.  The
// rounds compare them as integers of the same order (32 bits, then where several
// are equal the other 32), which a DPP maximum takes in one instruction.
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
    uint16_t* counts;       // E x stride, one entry a chunk (two launches)
    int chunk, stride;
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
        const int e = b + lane, v = e < E ? total[e] : 0, s = wave_scan(v);
        if (e < E) start[e] = before + s - v;
        before += lane_value(s, kWave - 1);
    }
    if (lane == 0) start[E] = before;
}

// Ranks of n entries by id: place[i] = entries before i of the same id (plus, with
// FINAL, the id's offset among all), -1 where the id is none.  Without FINAL the
// chunk's counts go to counts[e * stride] (n < 2^16), with it the offsets to `offsets`.  cnt:
// W * E + 2 * E + 1 ints of LDS.  The whole workgroup calls it.
template <int W, bool FINAL>
__device__ __forceinline__ void rank_entries(const int* ids, int* place, int n, int E, GF_LDS int* cnt, uint16_t* counts,
                                             int stride, int* offsets)
{
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int seg = ceil_div(ceil_div(n, W), kWave) * kWave;      // entries a wave
    const int waves = n > 0 ? ceil_div(n, seg) : 0;               // that have any
    GF_LDS int* total = cnt + W * E;
    GF_LDS int* start = total + E;
    GF_LDS int* mine = cnt + wave * E;
    for (int i = tid; i < waves * E; i += W * kWave) cnt[i] = 0;
    __syncthreads();
    const int lo = min(wave * seg, n), hi = min(lo + seg, n);
    for (int i = lo + lane; i < hi; i += kWave) {
        const int id = ids[i];
        if ((unsigned)id < (unsigned)E) __hip_atomic_fetch_add(&mine[id], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    for (int e = tid; e < E; e += W * kWave) {
        int run = 0;
        for (int w = 0; w < waves; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        if (FINAL) total[e] = run;
        else counts[(size_t)e * stride] = (uint16_t)run;
    }
    __syncthreads();
    if constexpr (FINAL) {
        scan_counts(total, start, E);
        __syncthreads();
        for (int e = tid; e <= E; e += W * kWave) offsets[e] = start[e];
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
__global__ __launch_bounds__(W * kWave) void rank_kernel(const int* ids, int* place, int n, int E, int chunk,
                                                         uint16_t* counts, int stride, int* offsets)
{
    extern __shared__ __attribute__((aligned(16))) char smem_raw[];
    const int lo = blockIdx.x * chunk;
    rank_entries<W, FINAL>(ids + lo, place + lo, min(chunk, n - lo), E, (GF_LDS int*)smem_raw,
                           FINAL ? nullptr : counts + blockIdx.x, stride, offsets);
}

// The second launch: the entries' offsets and the earlier chunks' counts.  Every
// workgroup adds up all counts for itself, `parts` threads an expert: at 256 chunks of
// 128 experts 64 KB, which costs less than a launch between the two would.
__global__ __launch_bounds__(1024) void place_kernel(const int* ids, int* place, int64_t n, int E, int chunk,
                                                     const uint16_t* counts, int stride, int chunks, int* offsets)
{
    __shared__ int before[kRouteMaxExperts], total[kRouteMaxExperts], start[kRouteMaxExperts + 1];
    const int tid = threadIdx.x, c = blockIdx.x;
    const int64_t lo = (int64_t)c * chunk, hi = lo + chunk < n ? lo + chunk : n;
    const int id0 = lo + tid < hi ? ids[lo + tid] : -1;
    const int at0 = lo + tid < hi ? place[lo + tid] : -1;
    const int width = E <= 16 ? 16 : 1 << (32 - __builtin_clz(E - 1)), parts = 1024 / width;
    const int e = tid / parts, part = tid % parts;
    int b = 0, t = 0;
    if (e < E) {
        const uint16_t* row = counts + (size_t)e * stride;
#pragma unroll 4
        for (int i = part * 8; i < chunks; i += parts * 8) {      // stride: a multiple of 8
            uint16_t v[8];
            __builtin_memcpy(v, row + i, 16);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int x = i + u < chunks ? v[u] : 0;
                t += x;
                b += i + u < c ? x : 0;
            }
        }
    }
    for (int d = 1; d < parts; d *= 2) {
        b += __shfl_xor(b, d);
        t += __shfl_xor(t, d);
    }
    if (e < E && part == 0) {
        before[e] = b;
        total[e] = t;
    }
    __syncthreads();
    scan_counts((const GF_LDS int*)total, (GF_LDS int*)start, E);
    __syncthreads();
    if (c == 0)
        for (int i = tid; i <= E; i += 1024) offsets[i] = start[i];
    if ((unsigned)id0 < (unsigned)E) place[lo + tid] = at0 + start[id0] + before[id0];
    for (int64_t i = lo + tid + 1024; i < hi; i += 1024) {
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

// VPT logits from i on, `left` of them in the row, -infinity past it: one wide load, at
// whatever alignment the row has.
template <int VPT, bool F32>
__device__ __forceinline__ void load_logits(const void* logits, size_t i, int left, float (&x)[VPT])
{
    if (left >= VPT) {
        typename std::conditional<F32, float, _Float16>::type v[VPT];
        __builtin_memcpy(v, (const char*)logits + i * sizeof(v[0]), sizeof(v));
#pragma unroll
        for (int u = 0; u < VPT; ++u) x[u] = (float)v[u];
    } else {
#pragma unroll
        for (int u = 0; u < VPT; ++u) x[u] = u < left ? logit_at<F32>(logits, i + u) : -__builtin_inff();
    }
}

__device__ __forceinline__ float sigmoid_shifted(float x, float top)
{
    // sigmoid(x) / exp(min(top, 0)): no underflow where top is the largest of the row's choices
    return expf(fminf(x, 0.0f) - fminf(top, 0.0f)) / (1.0f + expf(-fabsf(x)));
}

// The weight of this lane's choice x (lanes without one: live = false); top and
// sum: the softmax's maximum and sum over all experts.  most and total reduce over
// the token's lanes.
template <class Most, class Total>
__device__ __forceinline__ float choice_weight(const RouteArgs& a, float x, bool live, float top, float sum, Most most,
                                               Total total)
{
    float w;
    if (a.renorm) {
        // shifted by the largest chosen logit: the sum is at least a half
        const float best = most(live ? x : -__builtin_inff());
        w = live ? (a.sigmoid ? sigmoid_shifted(x, best) : expf(x - best)) : 0.0f;
        w /= total(w);
    } else {
        w = a.sigmoid ? sigmoid_shifted(x, 0.0f) : expf(x - top) / sum;
    }
    return live ? a.scale * w : 0.0f;
}

constexpr int kShut = INT32_MIN;     // the key of an expert that cannot be taken (any more)

// Integers of the order of the floats (no NaN; -0 is the caller's to avoid).
__device__ __forceinline__ int ordered(float v)
{
    const int b = __builtin_bit_cast(int, v);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}

// The logits' own order: NaN as +infinity, -0 as +0, -infinity shut.
__device__ __forceinline__ int logit_key(float x)
{
    const float v = x == x ? x + 0.0f : __builtin_inff();
    return v == -__builtin_inff() ? kShut : ordered(v);
}

// A wave's routing: what stays the same from token to token, and one token's work.
// KEY: float (the logits) or double (scores and bias).
template <int VPT, class KEY, bool F32>
struct TokenRouter {
    static constexpr bool WIDE = sizeof(KEY) == 8;
    const RouteArgs& a;
    const int lane, e0;
    GF_LDS KEY* keys;        // E of them, this wave's, where there are groups
    int size, parts;         // experts a group; lanes that look through one
    int bit[VPT];            // each expert's group as a lane
    double bias[VPT];

    __device__ __forceinline__ TokenRouter(const RouteArgs& a_, int lane_, GF_LDS KEY* keys_)
        : a(a_), lane(lane_), e0(lane_ * VPT), keys(keys_), size(1), parts(1)
    {
        if (a.groups > 1) {
            size = a.E / a.groups;
            parts = 1 << (31 - __builtin_clz(kWave / a.groups));
#pragma unroll
            for (int i = 0; i < VPT; ++i) bit[i] = (e0 + i) / size * parts;
        }
        if (WIDE)
#pragma unroll
            for (int i = 0; i < VPT; ++i) bias[i] = a.bias && e0 + i < a.E ? (double)a.bias[e0 + i] : 0.0;
    }

    __device__ __forceinline__ void load(int t, float (&x)[VPT]) const
    {
        load_logits<VPT, F32>(a.logits, (size_t)t * a.E + e0, a.E - e0, x);
    }

    // Closes the experts outside the best groups.
    __device__ __forceinline__ void keep_groups(KEY (&key)[VPT]) const
    {
        const KEY ninf = -(KEY)__builtin_inf();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + i < a.E) keys[e0 + i] = key[i];
        asm volatile("" ::: "memory");
        wait_lgkmcnt0();
        const int g = lane / parts, sub = lane % parts;
        KEY first = ninf, second = ninf;
        if (g < a.groups)
#pragma unroll 4
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
            if (e0 + i < a.E && !((stay >> bit[i]) & 1)) key[i] = ninf;
        asm volatile("" ::: "memory");
    }

    // Token t of logits x.
    __device__ __forceinline__ void route(int t, const float (&x)[VPT]) const
    {
        const KEY ninf = -(KEY)__builtin_inf(), inf = (KEY)__builtin_inf();
        KEY key[VPT];
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
                const double s = (a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i])) : key[i] / sum64) + bias[i];
                key[i] = x[i] == -__builtin_inff() ? ninf : s;
            } else {
                key[i] = x[i];
            }
            if (key[i] != key[i]) key[i] = inf;
        }
        if (a.groups > 1) keep_groups(key);

        int hi[VPT];
        [[maybe_unused]] uint32_t lo[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if constexpr (WIDE) {
                const uint64_t b = __builtin_bit_cast(uint64_t, key[i]);
                const int sign = (int)(b >> 32) >> 31;
                hi[i] = key[i] == ninf ? kShut : (int)(b >> 32) ^ (sign & 0x7FFFFFFF);
                lo[i] = (uint32_t)b ^ (uint32_t)sign;
            } else {
                hi[i] = logit_key(key[i]);
            }
        }
        int id = -1;
        for (int j = 0; j < a.k; ++j) {
            int best = hi[0];
#pragma unroll
            for (int i = 1; i < VPT; ++i) best = max(best, hi[i]);
            const int m = wave_reduce(best, kShut, [](int p, int q) { return max(p, q); });
            if (m == kShut) break;
            uint64_t at[VPT], any = 0;
            int count = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                at[i] = __ballot(hi[i] == m);
                any |= at[i];
                count += __builtin_popcountll(at[i]);
            }
            if (WIDE && count > 1) {
                uint32_t low = 0;
#pragma unroll
                for (int i = 0; i < VPT; ++i) low = max(low, hi[i] == m ? lo[i] : 0u);
                const uint32_t ml = (uint32_t)wave_reduce((int)low, 0, [](int p, int q) { return (int)max((uint32_t)p, (uint32_t)q); });
                any = 0;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    at[i] = __ballot(hi[i] == m && lo[i] == ml);
                    any |= at[i];
                }
            }
            const int src = __builtin_ctzll(any);
            int which = 0;
#pragma unroll
            for (int i = VPT - 1; i > 0; --i) which = (at[i] >> src) & 1 ? i : which;
            if ((at[0] >> src) & 1) which = 0;
            id = lane == j ? src * VPT + which : id;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (i == which) hi[i] = lane == src ? kShut : hi[i];
        }
        const float xs = id >= 0 ? logit_at<F32>(a.logits, (size_t)t * a.E + id) : 0.0f;
        const float w = choice_weight(a, xs, id >= 0, top, sum, [](float v) { return wave_max(v); },
                                      [](float v) { return wave_sum(v); });
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = id;
            a.weights[(size_t)t * a.k + lane] = w;
        }
    }
};

// Four tokens a wave, lane l of a row of 16 holding experts VPT * l ..: for keys that
// are the logits, without groups, k <= 16 and E <= 256.
template <int VPT, bool F32>
struct QuadRouter {
    const RouteArgs& a;
    const int l, e0;

    __device__ __forceinline__ QuadRouter(const RouteArgs& a_, int lane) : a(a_), l(lane % 16), e0(lane % 16 * VPT) {}

    // Token t of this row, the row's lanes; `in`: there is one.
    __device__ __forceinline__ void route(int t, bool in) const
    {
        const float ninf = -__builtin_inff();
        const size_t row = (size_t)t * a.E;
        float x[VPT];
        load_logits<VPT, F32>(a.logits, row + e0, in ? a.E - e0 : 0, x);
        auto most = [](float v) {
            return row_reduce(v, -__builtin_inff(), [](float p, float q) { return __builtin_fmaxf(p, q); });
        };
        auto total = [](float v) { return row_reduce(v, 0.0f, [](float p, float q) { return p + q; }); };
        float top = 0.0f, sum = 1.0f;
        if (!a.sigmoid && !a.renorm) {
            float m = x[0], s = 0.0f;
#pragma unroll
            for (int i = 1; i < VPT; ++i) m = fmaxf(m, x[i]);
            top = most(m);
#pragma unroll
            for (int i = 0; i < VPT; ++i) s += x[i] == ninf ? 0.0f : expf(x[i] - top);
            sum = total(s);
        }
        int key[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) key[i] = logit_key(x[i]);
        int id = -1;
        for (int j = 0; j < a.k; ++j) {
            int best = key[0];
#pragma unroll
            for (int i = 1; i < VPT; ++i) best = max(best, key[i]);
            const int m = row_reduce(best, kShut, [](int p, int q) { return max(p, q); });
            int e = INT32_MAX;
#pragma unroll
            for (int i = VPT - 1; i >= 0; --i) e = key[i] == m ? e0 + i : e;
            e = row_reduce(e, INT32_MAX, [](int p, int q) { return min(p, q); });
            if (l == j && m != kShut) id = e;
#pragma unroll
            for (int i = 0; i < VPT; ++i) key[i] = e - e0 == i ? kShut : key[i];
        }
        const float xs = id >= 0 ? logit_at<F32>(a.logits, row + id) : 0.0f;
        const float w = choice_weight(a, xs, id >= 0, top, sum, most, total);
        if (in && l < a.k) {
            a.ids[(size_t)t * a.k + l] = id;
            a.weights[(size_t)t * a.k + l] = w;
        }
    }
};

// chunk tokens a workgroup of W waves, then the chunk's ranks.  FINAL: one
// workgroup does all, the offsets too.
// QUAD: four tokens a wave (KEY is float).
template <int W, int VPT, class KEY, bool F32, bool QUAD, bool FINAL>
__global__ __launch_bounds__(W * kWave) void route_kernel(RouteArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char smem_raw[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
    if constexpr (QUAD) {
        const QuadRouter<VPT, F32> router(a, lane);
        for (int t = t0 + 4 * wave; t < t1; t += 4 * W) router.route(t + lane / 16, t + lane / 16 < t1);
    } else {
        GF_LDS KEY* keys = (GF_LDS KEY*)smem_raw + wave * a.E;
        const TokenRouter<VPT, KEY, F32> router(a, lane, keys);
        float x[VPT], next[VPT];
        if (t0 + wave < t1) router.load(t0 + wave, next);
        for (int t = t0 + wave; t < t1; t += W) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) x[i] = next[i];
            if (t + W < t1) router.load(t + W, next);
            router.route(t, x);
        }
    }
    if (!a.offsets) return;
    __syncthreads();                              // the ids are written, the keys read
    const size_t at = (size_t)t0 * a.k;
    rank_entries<W, FINAL>(a.ids + at, a.place + at, (t1 - t0) * a.k, a.E, (GF_LDS int*)smem_raw,
                           FINAL ? nullptr : a.counts + blockIdx.x, a.stride, a.offsets);
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
        load_logits<VPT, F32>(a.logits, row + e0, a.E - e0, p);
#pragma unroll
        for (int i = 0; i < VPT; ++i) m = fmaxf(m, p[i]);
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
    typedef typename std::conditional<F32, float, _Float16>::type T;
    T v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) v[i] = (T)out[i];
    T* dst = (T*)a.dlogits + row + e0;
    if (e0 + VPT <= a.E) {
        __builtin_memcpy(dst, v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + i < a.E) dst[i] = v[i];
    }
}

template <int W, int VPT, bool F32>
__global__ __launch_bounds__(W * kWave) void route_grad_kernel(RouteGradArgs a)
{
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (int t = blockIdx.x * W + wave; t < a.T; t += gridDim.x * W) route_grad_token<VPT, F32>(a, t, lane);
}

}  // namespace gf
