// Routing to experts: argument checks, launch choice and C-ABI entry points.
#include "../../include/gemvfp16.h"
#include "route_kernel.hpp"

namespace gf {
namespace {

constexpr int64_t kRouteMaxElems = (int64_t(1) << 31) - 1;
constexpr int kRouteMaxTokens = 1 << 30;

// One workgroup routes and sorts up to kOneTokens tokens, or sorts up to
// kOneEntries ids, in one launch; beyond, kMaxChunks workgroups do and a second
// launch joins their counts.
constexpr int kOneTokens = 64, kOneEntries = 4096, kMaxChunks = 256;
constexpr int kOneWaves = 16, kWaves = 8;

bool off_grid(const void* p, uintptr_t a) { return !p || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int status(hipError_t e) { return e == hipSuccess ? GF_OK : GF_ERR_HIP; }

size_t counts_bytes(bool one, int E) { return one ? 0 : (size_t)kMaxChunks * E * sizeof(int); }

int check_cfg(const gf_route_cfg* c, int T, int E, int k)
{
    if (!c || T < 0 || E < 1 || k < 1 || k > E) return GF_ERR_INVALID_ARG;
    if (c->score != GF_ROUTE_SOFTMAX && c->score != GF_ROUTE_SIGMOID) return GF_ERR_INVALID_ARG;
    if ((c->renorm != 0 && c->renorm != 1) || !(c->scale == c->scale)) return GF_ERR_INVALID_ARG;
    if (E > kRouteMaxExperts || k > kRouteMaxTop || T > kRouteMaxTokens) return GF_ERR_INVALID_ARG;
    if ((int64_t)T * E > kRouteMaxElems) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

template <int W, bool FINAL, int VPT, class KEY, bool F32>
hipError_t launch_route(const RouteArgs& a, int grid, hipStream_t stream)
{
    auto kern = route_kernel<W, VPT, KEY, F32, FINAL>;
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

template <int W, bool FINAL, int VPT>
hipError_t launch_route(const RouteArgs& a, bool wide, bool f32, int grid, hipStream_t stream)
{
    if (wide)
        return f32 ? launch_route<W, FINAL, VPT, double, true>(a, grid, stream)
                   : launch_route<W, FINAL, VPT, double, false>(a, grid, stream);
    return f32 ? launch_route<W, FINAL, VPT, float, true>(a, grid, stream)
               : launch_route<W, FINAL, VPT, float, false>(a, grid, stream);
}

// Logits a lane: the power of two that holds E.
template <class F>
hipError_t by_width(int E, F f)
{
    if (E <= 64) return f(std::integral_constant<int, 1>{});
    if (E <= 128) return f(std::integral_constant<int, 2>{});
    if (E <= 256) return f(std::integral_constant<int, 4>{});
    if (E <= 512) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 16>{});
}

// Chunks of n tokens or entries: no more than kMaxChunks, no smaller than `least`.
int chunk_of(int n, int least)
{
    const int c = (int)(((int64_t)n + kMaxChunks - 1) / kMaxChunks);
    return c < least ? least : c;
}

hipError_t launch_place(const int* ids, int* place, int64_t n, int E, int chunk, const int* counts, int chunks,
                        int* offsets, hipStream_t stream)
{
    hipLaunchKernelGGL(place_kernel, dim3(chunks), dim3(1024), 0, stream, ids, place, n, E, chunk, counts, chunks,
                       offsets);
    return hipGetLastError();
}

}  // namespace
}  // namespace gf

using namespace gf;

extern "C" {

size_t route_workspace_bytes(int T, int E, int k)
{
    if (T < 0 || E < 1 || k < 1 || E > kRouteMaxExperts || (int64_t)T * k > kRouteMaxElems) return 0;
    return counts_bytes(T <= kOneTokens && (int64_t)T * k <= kOneEntries, E);
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
    const bool one = T <= kOneTokens;
    if (offsets && !one && (off_grid(workspace, 4) || workspace_bytes < counts_bytes(false, E))) return GF_ERR_INVALID_ARG;
    if (T == 0 && !offsets) return GF_OK;

    RouteArgs a;
    a.logits = logits; a.bias = bias; a.ids = ids; a.weights = weights;
    a.T = T; a.E = E; a.k = k;
    a.sigmoid = cfg->score == GF_ROUTE_SIGMOID; a.renorm = cfg->renorm;
    a.groups = cfg->groups; a.top_groups = cfg->top_groups; a.group_best = cfg->group_best;
    a.scale = cfg->scale;
    a.offsets = offsets; a.place = place; a.counts = (int*)workspace;
    const bool wide = bias || (a.groups > 1 && a.group_best == 2);
    if (one && offsets) {
        a.chunk = T;
        return status(by_width(E, [&](auto v) {
            return launch_route<kOneWaves, true, decltype(v)::value>(a, wide, logits_f32 != 0, 1, (hipStream_t)stream);
        }));
    }
    a.chunk = chunk_of(T, 16);
    const int chunks = ceil_div(T, a.chunk);
    hipError_t e = by_width(E, [&](auto v) {
        return launch_route<kWaves, false, decltype(v)::value>(a, wide, logits_f32 != 0, chunks, (hipStream_t)stream);
    });
    if (e == hipSuccess && offsets)
        e = launch_place(ids, place, (int64_t)T * k, E, a.chunk * k, a.counts, chunks, offsets, (hipStream_t)stream);
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
    if (!one && (off_grid(workspace, 4) || workspace_bytes < counts_bytes(false, E))) return GF_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    if (one) {
        constexpr int W = kOneWaves, most = ((W + 2) * kRouteMaxExperts + 1) * 4;
        const int lds = ((W + 2) * E + 1) * 4;
        auto kern = rank_kernel<W, true>;
        if (lds > 64 * 1024) {
            static std::atomic<uint64_t> opt_in{0};
            const hipError_t e = opt_in_lds((const void*)kern, most, opt_in, s);
            if (e != hipSuccess) return GF_ERR_HIP;
        }
        hipLaunchKernelGGL(kern, dim3(1), dim3(W * kWave), lds, s, ids, place, n, E, n, offsets);
        return status(hipGetLastError());
    }
    constexpr int W = kWaves;
    const int chunk = chunk_of(n, 512), chunks = ceil_div(n, chunk);
    auto kern = rank_kernel<W, false>;
    hipLaunchKernelGGL(kern, dim3(chunks), dim3(W * kWave), ((W + 2) * E + 1) * 4, s, ids, place, n, E, chunk,
                       (int*)workspace);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = launch_place(ids, place, n, E, chunk, (const int*)workspace, chunks, offsets, s);
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
    return status(by_width(E, [&](auto v) {
        constexpr int VPT = decltype(v)::value;
        if (logits_f32)
            hipLaunchKernelGGL((route_grad_kernel<W, VPT, true>), dim3(grid), dim3(W * kWave), 0, (hipStream_t)stream, a);
        else
            hipLaunchKernelGGL((route_grad_kernel<W, VPT, false>), dim3(grid), dim3(W * kWave), 0, (hipStream_t)stream, a);
        return hipGetLastError();
    }));
}

}  // extern "C"
