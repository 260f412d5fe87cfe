// 4-bit weights: launch choice and C-ABI entry points.
#include "../../include/gemvfp16.h"
#include "w4_kernel.hpp"

namespace gf {
namespace {

constexpr int64_t kW4MaxElems = (int64_t(1) << 31) - 1;
constexpr int64_t kW4MaxGrid = (int64_t(1) << 31) - 1;

bool w4_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool w4_bad(const void* p, uintptr_t a) { return !p || !w4_aligned(p, a); }
int w4_status(hipError_t e) { return e == hipSuccess ? GF_OK : GF_ERR_HIP; }

// Sizes and groups of an N x K weight.
int validate_w4(int N, int K, int group)
{
    if (N < 0 || K < 0 || K % 8 != 0 || N > kMaxExtent || K > kMaxExtent) return GF_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return GF_ERR_INVALID_ARG;
    if ((int64_t)N * K > kW4MaxElems) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

int w4_grid(int64_t items)
{
    const int64_t g = (items + 255) / 256;
    return (int)(g < 65536 ? g : 65536);
}

// How rows of K (padded to whole groups of GROUP) are walked, and the grid.
W4Walk w4_walk(int64_t N, int K, int group, int& grid)
{
    W4Walk w;
    w.per_row = ceil_div(K, group) * (group / 8);
    w.rows_at_once = w.per_row >= 256 ? 1 : 256 / w.per_row;
    w.chunks = ceil_div(w.per_row, 256);
    w.rows = N;
    const int64_t iterations = (N + w.rows_at_once - 1) / w.rows_at_once;
    grid = (int)(iterations < 2048 ? iterations : 2048);  // eight workgroups of 256 to a CU
    return w;
}

template <int GROUP, bool ASYM, bool VEC>
hipError_t quantize(const void* W, void* Q, void* S, void* Z, int64_t N, int K, hipStream_t stream)
{
    int grid;
    const W4Walk w = w4_walk(N, K, GROUP, grid);
    auto kern = w.rows_at_once > 1 ? w4_quantize_kernel<GROUP, ASYM, VEC, true> : w4_quantize_kernel<GROUP, ASYM, VEC, false>;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(256), 0, stream, (const uint16_t*)W, (uint32_t*)Q, (uint16_t*)S,
                       (uint8_t*)Z, K, ceil_div(K, GROUP), w);
    return hipGetLastError();
}

template <int GROUP>
hipError_t quantize(const void* W, void* Q, void* S, void* Z, int64_t N, int K, hipStream_t stream)
{
    if (w4_aligned(W, 16))
        return Z ? quantize<GROUP, true, true>(W, Q, S, Z, N, K, stream)
                 : quantize<GROUP, false, true>(W, Q, S, Z, N, K, stream);
    return Z ? quantize<GROUP, true, false>(W, Q, S, Z, N, K, stream)
             : quantize<GROUP, false, false>(W, Q, S, Z, N, K, stream);
}

template <int GROUP, bool VEC>
hipError_t dequantize(const void* Q, const void* S, const void* Z, void* W, int64_t N, int K, hipStream_t stream)
{
    int grid;
    const W4Walk w = w4_walk(N, K, GROUP, grid);
    auto kern = w.rows_at_once > 1 ? w4_dequantize_kernel<GROUP, VEC, true> : w4_dequantize_kernel<GROUP, VEC, false>;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(256), 0, stream, (const uint32_t*)Q, (const uint16_t*)S,
                       (const uint8_t*)Z, (uint16_t*)W, K, ceil_div(K, GROUP), w);
    return hipGetLastError();
}

template <int GROUP>
hipError_t dequantize(const void* Q, const void* S, const void* Z, void* W, int64_t N, int K, hipStream_t stream)
{
    return w4_aligned(W, 16) ? dequantize<GROUP, true>(Q, S, Z, W, N, K, stream)
                             : dequantize<GROUP, false>(Q, S, Z, W, N, K, stream);
}

__global__ void w4_zero_kernel(uint16_t* __restrict__ p, int64_t n)
{
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < n; t += stride) p[t] = 0;
}

template <class Cfg, int GROUP, bool WINDOW, bool GROUPED>
int launch_tile_of(W4Args a, hipStream_t stream)
{
    auto kern = w4_tile_kernel<Cfg, GROUP, WINDOW, GROUPED>;
    static std::atomic<uint64_t> lds_opt_in{0};
    const hipError_t e = opt_in_lds((const void*)kern, Cfg::LDS_BYTES, lds_opt_in, stream);
    if (e != hipSuccess) return GF_ERR_HIP;
    int64_t blocks = ceil_div(a.M, Cfg::BM);
    if (GROUPED) blocks = a.g.T / Cfg::BM + (a.g.E < a.g.T ? a.g.E : a.g.T);
    const int64_t grid = blocks * ceil_div(a.N, Cfg::BN);
    if (grid > kW4MaxGrid) return GF_ERR_INVALID_ARG;
    return w4_status(launch_in_parts(grid, [&](int first, dim3 n) {
        a.g.first = first;
        hipLaunchKernelGGL(kern, n, dim3(Cfg::NT), Cfg::LDS_BYTES, stream, a);
        return hipGetLastError();
    }));
}

template <class Cfg, int GROUP, bool GROUPED>
int launch_tile(const W4Args& a, hipStream_t stream)
{
    if (a.K % 256 == 0)
        return launch_tile_of<Cfg, GROUP, true, GROUPED>(a, stream);
    return launch_tile_of<Cfg, GROUP, false, GROUPED>(a, stream);
}

template <class Cfg, bool GROUPED>
int launch_rows(W4Args a, hipStream_t stream)
{
    auto kern = w4_rows_kernel<Cfg, GROUPED>;
    static_assert(Cfg::LDS_BYTES <= 64 * 1024, "no opt-in for large LDS");
    int64_t blocks = ceil_div(a.M, 16 * Cfg::MB);
    if (GROUPED) blocks = a.g.T / (16 * Cfg::MB) + (a.g.E < a.g.T ? a.g.E : a.g.T);
    const int64_t grid = blocks * ceil_div(a.N, 16 * Cfg::NB);
    if (grid > kW4MaxGrid) return GF_ERR_INVALID_ARG;
    return w4_status(launch_in_parts(grid, [&](int first, dim3 n) {
        a.g.first = first;
        hipLaunchKernelGGL(kern, n, dim3(Cfg::WAVES * 64), Cfg::LDS_BYTES, stream, a);
        return hipGetLastError();
    }));
}

// parts: workgroups that share the row groups of one weight (and 16 MB rows of A),
// at most one each.
template <class Cfg, bool GROUPED>
int launch_band(W4Args a, int ring, int parts, hipStream_t stream)
{
    auto kern = w4_band_kernel<Cfg, GROUPED>;
    static std::atomic<uint64_t> lds_opt_in{0};
    constexpr int kMaxLds = 160 * 1024;
    const hipError_t e = opt_in_lds((const void*)kern, kMaxLds, lds_opt_in, stream);
    if (e != hipSuccess) return GF_ERR_HIP;
    const int red_rows = !GROUPED && a.M < 16 * Cfg::MB ? a.M : 16 * Cfg::MB;
    const int lds = Cfg::WAVES * ring * Cfg::TASK_BYTES + 2 * Cfg::WAVES * red_rows * 64 + (Cfg::XLDS ? a.M * a.K * 2 : 0);
    if (lds > kMaxLds || ring < 1 || ring > Cfg::MAX_RING) return GF_ERR_UNSUPPORTED;
    parts = parts < ceil_div(a.N, 16) ? parts : ceil_div(a.N, 16);
    int64_t grid = Cfg::XLDS ? parts : (int64_t)ceil_div(parts, 8) * 8 * ceil_div(a.M, 16 * Cfg::MB);
    if (GROUPED) grid = (int64_t)parts * (a.g.T / (16 * Cfg::MB) + (a.g.E < a.g.T ? a.g.E : a.g.T));
    if (grid > kW4MaxGrid) return GF_ERR_INVALID_ARG;
    return w4_status(launch_in_parts(grid, [&](int first, dim3 n) {
        a.g.first = first;
        hipLaunchKernelGGL(kern, n, dim3(Cfg::WAVES * 64), lds, stream, a, ring, parts);
        return hipGetLastError();
    }));
}

// The band form's launch.  One weight: two workgroups to a CU, with as much in
// flight as their LDS leaves, where there are row groups for them and the
// registers allow it (not with A in registers); else one with all of it, shared
// among the passes over 16 MB rows of A each.  Grouped: about 256 workgroups in
// all but at least 8 to a pass, two tasks in flight a wave (24 us against 31 with
// twice as many and four, at 24 rows over 16 groups of 4096 x 4096; 15 against 22
// with twice as many at 16 over 8 of 2048 x 8192).
template <class Cfg, bool GROUPED>
int band(const W4Args& a, hipStream_t stream)
{
    if constexpr (GROUPED) {
        const int64_t passes = (a.g.E < a.g.T ? a.g.E : a.g.T) + a.g.T / (16 * Cfg::MB);
        const int want = (int)(256 / passes + 7) / 8 * 8;
        return launch_band<Cfg, true>(a, 2, want < 8 ? 8 : (want > 64 ? 64 : want), stream);
    } else {
        const int passes = ceil_div(a.M, 16 * Cfg::MB), rows = passes > 1 ? 16 * Cfg::MB : a.M;
        const int fixed = 2 * Cfg::WAVES * rows * 64 + (Cfg::XLDS ? a.M * a.K * 2 : 0);
        const int per_task = Cfg::WAVES * Cfg::TASK_BYTES;
        const int groups = ceil_div(a.N, 16);
        const int per_cu = Cfg::XLDS && groups > 256 && fixed + per_task <= 80 * 1024 ? 2 : 1;
        int ring = (160 * 1024 / per_cu - fixed) / per_task;
        // (of each pass, dealt to 8 XCDs)
        const int parts = passes == 1 ? 256 * per_cu : passes <= 32 ? 256 / passes / 8 * 8 : 8;
        const int tasks = ceil_div(groups, parts) * ceil_div(a.K, Cfg::BK * Cfg::WAVES);   // of a wave
        if (ring > Cfg::MAX_RING) ring = Cfg::MAX_RING;
        if (ring > tasks) ring = tasks;
        return launch_band<Cfg, false>(a, ring, parts, stream);
    }
}

// The tile form's launch, timed side by side over sizes (us):
//  * one weight: 256 x 256 where they fill the CUs (129 against 138 for 128 x 256
//    at 2048 x 8192 x 4096), else 128 x 256 with 8 waves from 400 tiles of 128 x
//    128 (70 against 74 and 101 at 1024 x 8192 x 4096), 128 x 128 from 160 (40
//    against 42 at 700 x 4096 x 4096), 64 x 128 from 128 of its own (32 against 38
//    at 300 x 4096 x 4096), else 32 x 128 (77 against 85 at 256 x 2000 x 7072);
//  * grouped, by the mean rows of a group: 32 x 128 up to 48 (24 against 26, and
//    50 in the general form, at 600 rows over 16 groups of 2048 x 2048), 64 x 128 up
//    to 80, each also where the next larger ones are few (72 and 80 against 96 at
//    1284 rows over 2 of 448 x 7072), else 128 x 128 (42 against 47 at
//    1111 over 8 of 2048 x 4096; 256 x 256 wastes the groups' ends: 343 against 314
//    at 8000 over 8 of 4096 x 4096).
template <int GROUP, bool GROUPED>
int tile(const W4Args& a, int64_t rows, hipStream_t stream)
{
    typedef W4TileCfg<1, 1, 1, 4, 5> T32;
    typedef W4TileCfg<2, 1, 1, 4, 4> T64;
    typedef W4TileCfg<4, 1, 1, 4, 4> T128;
    if constexpr (GROUPED) {
        const int used = a.g.E < a.g.T ? a.g.E : a.g.T;
        auto tiles = [&](int bm) { return ((int64_t)(a.g.T / bm) + used) * ceil_div(a.N, 128); };   // at most
        if (rows <= 48 || tiles(64) < 128) return launch_tile<T32, GROUP, true>(a, stream);
        if (rows <= 80 || tiles(128) < 128) return launch_tile<T64, GROUP, true>(a, stream);
        return launch_tile<T128, GROUP, true>(a, stream);
    } else {
        auto tiles = [&](int bm, int bn) { return (int64_t)ceil_div(a.M, bm) * ceil_div(a.N, bn); };
        if (tiles(256, 256) >= 192) return launch_tile<W4TileCfg<4, 2, 2, 4, 4>, GROUP, false>(a, stream);
        if (tiles(128, 128) >= 400) return launch_tile<W4TileCfg<4, 1, 1, 8, 4>, GROUP, false>(a, stream);
        if (tiles(128, 128) >= 160) return launch_tile<T128, GROUP, false>(a, stream);
        if (tiles(64, 128) >= 128) return launch_tile<T64, GROUP, false>(a, stream);
        return launch_tile<T32, GROUP, false>(a, stream);
    }
}

// Which form, by the rows of A (of a group, on average), the blocks of 16 x 16
// entries of C, and by what the operands' sizes and alignment allow.  Timed side
// by side (us):
//  * one weight, up to 64 rows: the band form, in passes of 16 rows of A, or of 32
//    where 16 would make more than two sweeps of the chip (12 against 15 at 24 x
//    11008 x 4096, but 7.3 against 8.4 at 24 x 4096 x 4096).  At 64 x 4096 x 4096 it
//    takes 9.8, the general form 13, tiles 31.  Up to 32768 entries of A in one
//    pass lie in LDS instead (4.8 against 5.7 at 9 x 2048 x 2048).  From 65 rows on,
//    tiles, but for products of few blocks and long K: tiles then leave most of the chip idle
//    through all of K (26 against 6.1 at 100 x 500 x 4096, 30 against 9.8 at 100 x
//    2000 x 4096, 57 against 23 at 512 x 512 x 8192; the general form 29 against 68 at
//    512 x 512 x 7072).  Below K = 2048 they are even.
//  * grouped, the band form up to a mean of 16 rows, and of 32 where K is long (21
//    against 33 at 200 rows over 8 groups of 2048 x 4096; 39 against 24 at 600 over
//    16 of 2048 x 2048), in passes of 32 rows from a mean of 9 on (42 against 55 at
//    150 over 16 of 4096 x 4096); then tiles, but for few blocks.
//    Both band forms end at K = 8192: each wave keeps its part of A, and two blocks of
//    512 k are what its registers hold (16 x 4096 x 14336 in the general form 24, 16 x
//    4096 x 8192 here 8.5; by expert 93 at 24 rows over 8 of 4096 x 14336).
//  * what is left takes the general form, with 16 rows of A by 32 of Q (16 by 16
//    for few rows of both; 32 by 64 for many rows of both where groups of 128
//    leave the registers for it: 23 against 38 at 32 x 16384 x 5000, but 40 against
//    44 the other way round, spilling, with groups of 64).
template <int GROUP, bool GROUPED>
int product(const W4Args& a, hipStream_t stream)
{
    const int64_t rows = GROUPED ? (a.g.T + a.g.E - 1) / a.g.E : a.M;
    const int64_t passes = GROUPED ? a.g.T / 16 + (a.g.E < a.g.T ? a.g.E : a.g.T) : ceil_div(a.M, 16);
    const int64_t blocks = passes * ceil_div(a.N, 16);
    const bool wide = w4_aligned(a.A, 16) && w4_aligned(a.Q, 16) && w4_aligned(a.S, 16) && w4_aligned(a.Z, 8);
    const bool few = blocks <= 2048 && passes <= 64 && a.K >= 2048;
    if (wide && a.K % 512 == 0 && a.K > 0 && a.N >= 16) {
        if constexpr (GROUPED) {
            if ((rows <= 16 || (rows <= 32 && a.K >= 4096) || few) && a.K <= 8192) {
                if (a.K > 4096) return band<W4BandCfg<GROUP, 1, 2>, true>(a, stream);
                if constexpr (GROUP > 32)
                    if (rows > 8) return band<W4BandCfg<GROUP, 2, 1>, true>(a, stream);
                return band<W4BandCfg<GROUP, 1, 1>, true>(a, stream);
            }
        } else {
            if (a.M <= 16 && a.M * a.K <= 32768) return band<W4BandCfg<GROUP, 1, 0>, false>(a, stream);
            if ((a.M <= 64 || few) && a.K <= 8192) {
                if (a.K > 4096) return band<W4BandCfg<GROUP, 1, 2>, false>(a, stream);
                if constexpr (GROUP > 32)                 // (spills with groups of 32)
                    if (a.M > 16 && blocks > 512) return band<W4BandCfg<GROUP, 2, 1>, false>(a, stream);
                return band<W4BandCfg<GROUP, 1, 1>, false>(a, stream);
            }
        }
    }
    if (rows > (GROUPED ? 16 : 64) && !(few && blocks <= 1536) && w4_aligned(a.A, 16) && a.K >= 64)
        return tile<GROUP, GROUPED>(a, rows, stream);
    constexpr int CB = GROUP == 32 ? 2 : 4;
    if constexpr (GROUP == 128)
        if (rows > 16 && a.N >= 8192) return launch_rows<W4RowsCfg<GROUP, 2, 4, 4, 2>, GROUPED>(a, stream);
    return rows > 16 || a.N >= 8192 ? launch_rows<W4RowsCfg<GROUP, 1, 2, 8, CB>, GROUPED>(a, stream)
                                    : launch_rows<W4RowsCfg<GROUP, 1, 1, 8, CB>, GROUPED>(a, stream);
}

template <bool GROUPED>
int product_by_group(const W4Args& a, int group, hipStream_t stream)
{
    switch (group) {
    case 32: return product<32, GROUPED>(a, stream);
    case 64: return product<64, GROUPED>(a, stream);
    default: return product<128, GROUPED>(a, stream);
    }
}

}  // namespace
}  // namespace gf

using namespace gf;

extern "C" {

int w4_quantize_f16(const void* W, void* Q, void* S, void* Z, int N, int K, int group, void* stream)
{
    const int rc = validate_w4(0, K, group);
    if (rc || N < 0) return GF_ERR_INVALID_ARG;
    if (N == 0 || K == 0) return GF_OK;
    if (w4_bad(W, 2) || w4_bad(Q, 4) || w4_bad(S, 2)) return GF_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    switch (group) {
    case 32: return w4_status(quantize<32>(W, Q, S, Z, N, K, s));
    case 64: return w4_status(quantize<64>(W, Q, S, Z, N, K, s));
    default: return w4_status(quantize<128>(W, Q, S, Z, N, K, s));
    }
}

int w4_dequantize_f16(const void* Q, const void* S, const void* Z, void* W, int N, int K, int group, void* stream)
{
    const int rc = validate_w4(0, K, group);
    if (rc || N < 0) return GF_ERR_INVALID_ARG;
    if (N == 0 || K == 0) return GF_OK;
    if (w4_bad(W, 2) || w4_bad(Q, 4) || w4_bad(S, 2)) return GF_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    switch (group) {
    case 32: return w4_status(dequantize<32>(Q, S, Z, W, N, K, s));
    case 64: return w4_status(dequantize<64>(Q, S, Z, W, N, K, s));
    default: return w4_status(dequantize<128>(Q, S, Z, W, N, K, s));
    }
}

int gemm_w4_f16_nt(const void* A, const void* Q, const void* S, const void* Z, void* C, int M, int N, int K,
                   int group, void* stream)
{
    const int rc = validate_w4(N, K, group);
    if (rc) return rc;
    if (M < 0 || M > kMaxExtent || (int64_t)M * K > kW4MaxElems || (int64_t)M * N > kW4MaxElems) return GF_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GF_OK;
    if (w4_bad(C, 2)) return GF_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    if (K == 0) {                                       // the empty sum
        const int64_t mn = (int64_t)M * N;
        hipLaunchKernelGGL(w4_zero_kernel, dim3(w4_grid(mn)), dim3(256), 0, s, (uint16_t*)C, mn);
        return w4_status(hipGetLastError());
    }
    if (w4_bad(A, 2) || w4_bad(Q, 4) || w4_bad(S, 2)) return GF_ERR_INVALID_ARG;
    W4Args a = {(const uint16_t*)A, (const uint32_t*)Q, (const uint16_t*)S, (const uint8_t*)Z, (uint16_t*)C,
                M, N, K, ceil_div(K, group), {nullptr, 0, 0, 0}};
    return product_by_group<false>(a, group, s);
}

int gemv_w4_f16(const void* Q, const void* S, const void* Z, const void* x, void* y, int N, int K, int group,
                void* stream)
{
    return gemm_w4_f16_nt(x, Q, S, Z, y, 1, N, K, group, stream);
}

int gemm_w4_f16_grouped_nt(const void* A, const void* Q, const void* S, const void* Z, void* C,
                           const int* offsets, int T, int E, int N, int K, int group, void* stream)
{
    const int rc = validate_w4(N, K, group);
    if (rc) return rc;
    if (T < 0 || E < 0 || T > kMaxExtent || E > kMaxGroups) return GF_ERR_INVALID_ARG;
    if ((int64_t)T * K > kW4MaxElems || (int64_t)T * N > kW4MaxElems) return GF_ERR_INVALID_ARG;
    if (E > 0 && w4_bad(offsets, 4)) return GF_ERR_INVALID_ARG;
    if (T == 0 || E == 0 || N == 0) return GF_OK;
    if (w4_bad(C, 2)) return GF_ERR_INVALID_ARG;
    // K == 0: the kernel never reads A, Q or S, and stores the empty sums of the groups' rows
    if (K > 0 && (w4_bad(A, 2) || w4_bad(Q, 4) || w4_bad(S, 2))) return GF_ERR_INVALID_ARG;
    W4Args a = {(const uint16_t*)A, (const uint32_t*)Q, (const uint16_t*)S, (const uint8_t*)Z, (uint16_t*)C,
                0, N, K, ceil_div(K, group), {offsets, E, T, 0}};
    return product_by_group<true>(a, group, (hipStream_t)stream);
}

}  // extern "C"
