// Routing to experts: argument checks, launch choice and C-ABI entry points.
#include "../../include/gemvfp16.h"
#include "route_kernel.hpp"

namespace gf {
namespace {

constexpr int64_t kRouteMaxElems = (int64_t(1) << 31) - 1;
constexpr int kRouteMaxTokens = 1 << 30;

// One workgroup routes and sorts up to kOneTokens tokens (four times as many where a
// wave takes four), or sorts up to kOneEntries ids, in one launch (64 tokens a wave each
// took 20 us so, 11 in two launches); beyond, many do, and a second launch joins their
// counts (16 bits each: a chunk has fewer than 2^16 entries).  Up to kSmall tokens in
// chunks of one round of four waves, so that they spread over the CUs; beyond, about
// kChunks of them.
constexpr int kOneTokens = 16, kOneEntries = 4096, kChunks = 256, kSmall = 1024;
constexpr int kWaves = 16, kSmallWaves = 4;

// ceil_div of an a that may be next to 2^31.
int ceil_div_large(int a, int b) { return a / b + (a % b != 0); }

// Units (tokens, or entries) a chunk, of n with k entries each.
int chunk_of(int n, int k, int least)
{
    int c = (int)(((int64_t)n + kChunks - 1) / kChunks);
    if (c < least) c = least;
    const int most = 65535 / k;
    return c < most ? c : most;
}

bool off_grid(const void* p, uintptr_t a) { return !p || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int status(hipError_t e) { return e == hipSuccess ? GF_OK : GF_ERR_HIP; }

constexpr int kTokensLeast = 4, kEntriesLeast = 512;   // of a chunk

// Chunks to a row of the counts, which are read eight at a time.
int stride_of(int chunks) { return ceil_div(chunks, 8) * 8; }

// T * k entries in chunks of tokens or of entries: as many of either as there can be.
size_t counts_bytes(int T, int k, int E)
{
    if (T <= kOneTokens && (int64_t)T * k <= kOneEntries) return 0;
    const int by_tokens = k <= kRouteMaxTop ? ceil_div_large(T, chunk_of(T, k, kTokensLeast)) : 0;
    const int by_entries = ceil_div_large(T * k, chunk_of(T * k, 1, kEntriesLeast));
    return (size_t)stride_of(by_tokens > by_entries ? by_tokens : by_entries) * E * sizeof(uint16_t);
}

int check_cfg(const gf_route_cfg* c, int T, int E, int k)
{
    if (!c || T < 0 || E < 1 || k < 1 || k > E) return GF_ERR_INVALID_ARG;
    if (c->score != GF_ROUTE_SOFTMAX && c->score != GF_ROUTE_SIGMOID) return GF_ERR_INVALID_ARG;
    if ((c->renorm != 0 && c->renorm != 1) || !(c->scale == c->scale)) return GF_ERR_INVALID_ARG;
    if (E > kRouteMaxExperts || k > kRouteMaxTop || T > kRouteMaxTokens) return GF_ERR_INVALID_ARG;
    if ((int64_t)T * E > kRouteMaxElems) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

template <int W, bool FINAL, int VPT, class KEY, bool F32, bool QUAD>
hipError_t launch_route(const RouteArgs& a, int grid, hipStream_t stream)
{
    auto kern = route_kernel<W, VPT, KEY, F32, QUAD, FINAL>;
    const int keys = a.groups > 1 ? W * a.E * (int)sizeof(KEY) : 0;
    const int ranks = a.offsets ? ((W + 2) * a.E + 1) * (int)sizeof(int) : 0;
    const int lds = keys > ranks ? keys : ranks;
    if (lds > 64 * 1024) {
        constexpr int most = W * kRouteMaxExperts * 8;
        static_assert(most <= 160 * 1024 && most >= ((W + 2) * kRouteMaxExperts + 1) * 4, "one CU's LDS");
        static std::atomic<uint64_t> opt_in{0};
        const hipError_t e = opt_in_lds((const void*)kern, most, opt_in, stream);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kern, dim3(grid), dim3(W * kWave), lds, stream, a);
    return hipGetLastError();
}

// f(logits a lane, as a constant): the power of two with which `lanes` lanes hold E.
template <class F>
hipError_t by_width(int E, int lanes, F f)
{
    if (E <= lanes) return f(std::integral_constant<int, 1>{});
    if (E <= 2 * lanes) return f(std::integral_constant<int, 2>{});
    if (E <= 4 * lanes) return f(std::integral_constant<int, 4>{});
    if (E <= 8 * lanes) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

template <int W, bool FINAL>
hipError_t launch_route(const RouteArgs& a, bool quad, bool wide, bool f32, int grid, hipStream_t stream)
{
    return by_width(a.E, quad ? 16 : kWave, [&](auto v) {
        constexpr int VPT = decltype(v)::value;
        if constexpr (VPT <= 8 || (W == kWaves && !FINAL))    // past 128 experts for many tokens alone
            if (quad)
                return f32 ? launch_route<W, FINAL, VPT, float, true, true>(a, grid, stream)
                           : launch_route<W, FINAL, VPT, float, false, true>(a, grid, stream);
        if (wide)
            return f32 ? launch_route<W, FINAL, VPT, double, true, false>(a, grid, stream)
                       : launch_route<W, FINAL, VPT, double, false, false>(a, grid, stream);
        return f32 ? launch_route<W, FINAL, VPT, float, true, false>(a, grid, stream)
                   : launch_route<W, FINAL, VPT, float, false, false>(a, grid, stream);
    });
}

hipError_t launch_place(const int* ids, int* place, int64_t n, int E, int chunk, const uint16_t* counts,
                        int chunks, int* offsets, hipStream_t stream)
{
    hipLaunchKernelGGL(place_kernel, dim3(chunks), dim3(1024), 0, stream, ids, place, n, E, chunk, counts,
                       stride_of(chunks), chunks, offsets);
    return hipGetLastError();
}

}  // namespace
}  // namespace gf

using namespace gf;

extern "C" {

size_t route_workspace_bytes(int T, int E, int k)
{
    if (T < 0 || E < 1 || k < 1 || E > kRouteMaxExperts || (int64_t)T * k > kRouteMaxElems) return 0;
    return counts_bytes(T, k, E);
}

int route_topk(const void* logits, int logits_f32, const float* bias, int T, int E, int k, const gf_route_cfg* cfg,
               int* ids, float* weights, int* offsets, int* place, void* workspace, size_t workspace_bytes,
               void* stream)
{
    if (logits_f32 != 0 && logits_f32 != 1) return GF_ERR_INVALID_ARG;
    const int rc = check_cfg(cfg, T, E, k);
    if (rc) return rc;
    if (cfg->groups < 1 || cfg->groups > kRouteMaxGroups || E % cfg->groups != 0) return GF_ERR_INVALID_ARG;
    if (cfg->top_groups < 1 || cfg->top_groups > cfg->groups) return GF_ERR_INVALID_ARG;
    if (cfg->group_best != 1 && cfg->group_best != 2) return GF_ERR_INVALID_ARG;
    if (k > E / cfg->groups * cfg->top_groups) return GF_ERR_INVALID_ARG;
    if (bias && off_grid(bias, 4)) return GF_ERR_INVALID_ARG;
    if (!offsets != !place && T > 0) return GF_ERR_INVALID_ARG;
    if (offsets && off_grid(offsets, 4)) return GF_ERR_INVALID_ARG;
    if (T > 0) {
        if (off_grid(logits, logits_f32 ? 4 : 2) || off_grid(ids, 4) || off_grid(weights, 4)) return GF_ERR_INVALID_ARG;
        if (place && off_grid(place, 4)) return GF_ERR_INVALID_ARG;
    }
    if (offsets && T > kOneTokens && (off_grid(workspace, 4) || workspace_bytes < counts_bytes(T, k, E)))
        return GF_ERR_INVALID_ARG;
    if (T == 0 && !offsets) return GF_OK;

    RouteArgs a;
    a.logits = logits; a.bias = bias; a.ids = ids; a.weights = weights;
    a.T = T; a.E = E; a.k = k;
    a.sigmoid = cfg->score == GF_ROUTE_SIGMOID; a.renorm = cfg->renorm;
    a.groups = cfg->groups; a.top_groups = cfg->top_groups; a.group_best = cfg->group_best;
    a.scale = cfg->scale;
    a.offsets = offsets; a.place = place; a.counts = (uint16_t*)workspace; a.stride = 0;
    const bool wide = bias || (a.groups > 1 && a.group_best == 2);
    // Four tokens a wave past 128 experts (16 logits a lane) where there are many: 8192 tokens
    // of 256 experts 16.2 us against 19.9, 4096 15.4 against 16.2, 2048 15.3 against 15.0, 64
    // 9.8 against 8.8 (but 1024 11.1 against 14.4).
    const bool quad = !wide && a.groups == 1 && k <= 16 && E <= (T < 4096 ? 128 : 256), f32 = logits_f32 != 0;
    hipStream_t s = (hipStream_t)stream;
    if (offsets && T <= (quad ? 4 : 1) * kOneTokens) {
        a.chunk = T;
        return status(launch_route<kWaves, true>(a, quad, wide, f32, 1, s));
    }
    const bool small = T <= kSmall;
    a.chunk = chunk_of(T, k, small && quad ? 4 * kSmallWaves : kTokensLeast);
    const int chunks = ceil_div(T, a.chunk);
    a.stride = stride_of(chunks);
    hipError_t e = small ? launch_route<kSmallWaves, false>(a, quad, wide, f32, chunks, s)
                         : launch_route<kWaves, false>(a, quad, wide, f32, chunks, s);
    if (e == hipSuccess && offsets)
        e = launch_place(ids, place, (int64_t)T * k, E, a.chunk * k, a.counts, chunks, offsets, s);
    return status(e);
}

int route_rows(const int* ids, int T, int k, int E, int* offsets, int* place, void* workspace, size_t workspace_bytes,
               void* stream)
{
    if (T < 0 || k < 1 || E < 1 || E > kRouteMaxExperts) return GF_ERR_INVALID_ARG;
    if (T > kRouteMaxTokens || (int64_t)T * k > kRouteMaxElems) return GF_ERR_INVALID_ARG;
    const int n = T * k;
    if (off_grid(offsets, 4) || (n > 0 && (off_grid(ids, 4) || off_grid(place, 4)))) return GF_ERR_INVALID_ARG;
    const bool one = n <= kOneEntries;
    if (!one && (off_grid(workspace, 4) || workspace_bytes < counts_bytes(T, k, E))) return GF_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    if (one) {
        constexpr int W = kWaves, most = ((W + 2) * kRouteMaxExperts + 1) * 4;
        const int lds = ((W + 2) * E + 1) * 4;
        auto kern = rank_kernel<W, true>;
        if (lds > 64 * 1024) {
            static std::atomic<uint64_t> opt_in{0};
            const hipError_t e = opt_in_lds((const void*)kern, most, opt_in, s);
            if (e != hipSuccess) return GF_ERR_HIP;
        }
        hipLaunchKernelGGL(kern, dim3(1), dim3(W * kWave), lds, s, ids, place, n, E, n, (uint16_t*)nullptr,
                           0, offsets);
        return status(hipGetLastError());
    }
    constexpr int W = 8;
    const int chunk = chunk_of(n, 1, kEntriesLeast), chunks = ceil_div_large(n, chunk);
    auto kern = rank_kernel<W, false>;
    hipLaunchKernelGGL(kern, dim3(chunks), dim3(W * kWave), ((W + 2) * E + 1) * 4, s, ids, place, n, E, chunk,
                       (uint16_t*)workspace, stride_of(chunks), offsets);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = launch_place(ids, place, n, E, chunk, (const uint16_t*)workspace, chunks, offsets, s);
    return status(e);
}

int route_topk_bwd(const void* logits, int logits_f32, const int* ids, const float* dweights, int T, int E, int k,
                   const gf_route_cfg* cfg, void* dlogits, void* stream)
{
    if (logits_f32 != 0 && logits_f32 != 1) return GF_ERR_INVALID_ARG;
    const int rc = check_cfg(cfg, T, E, k);
    if (rc) return rc;
    if (T == 0) return GF_OK;
    const uintptr_t size = logits_f32 ? 4 : 2;
    if (off_grid(logits, size) || off_grid(dlogits, size) || off_grid(ids, 4) || off_grid(dweights, 4))
        return GF_ERR_INVALID_ARG;
    RouteGradArgs a;
    a.logits = logits; a.ids = ids; a.dweights = dweights; a.dlogits = dlogits;
    a.T = T; a.E = E; a.k = k;
    a.sigmoid = cfg->score == GF_ROUTE_SIGMOID; a.renorm = cfg->renorm;
    a.scale = cfg->scale;
    constexpr int W = 4;
    const int grid = ceil_div(T, W) < 65536 ? ceil_div(T, W) : 65536;
    return status(by_width(E, kWave, [&](auto v) {
        constexpr int VPT = decltype(v)::value;
        if (logits_f32)
            hipLaunchKernelGGL((route_grad_kernel<W, VPT, true>), dim3(grid), dim3(W * kWave), 0, (hipStream_t)stream, a);
        else
            hipLaunchKernelGGL((route_grad_kernel<W, VPT, false>), dim3(grid), dim3(W * kWave), 0, (hipStream_t)stream, a);
        return hipGetLastError();
    }));
}

}  // extern "C"
