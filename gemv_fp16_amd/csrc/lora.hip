// Low-rank adapters: argument checks, launch choice and C-ABI entry points.
#include "../../include/gemvfp16.h"
#include "configs.hpp"
#include "lora_kernel.hpp"

namespace gf {
namespace {

constexpr int kMaxRank = 256;
constexpr int kMaxSize = 1 << 30;
constexpr int64_t kMaxElems = (int64_t(1) << 31) - 1;

bool off_grid(const void* p, uintptr_t a) { return !p || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int status(hipError_t e) { return e == hipSuccess ? GF_OK : GF_ERR_HIP; }

// Parts of K that the products by Down are split in, for one CU takes in no more than
// about 40 GB/s: up to 32 rows as many as make 256 workgroups of them (the streaming
// form adds them in LDS, which holds all), beyond as many as make 128 of 16-row blocks,
// but no more than the tiles' epilogue loads at once (100 rows of 8 adapters at 4096 x
// 4096: 35.7 us with 4 parts, 38.4 with one).  Tiles and lora_add_f16 read H, all parts of
// it, again for every 64 columns: 2048 rows of rank 64 took 99 us with 4 parts, 94 with
// one, rank 16 81 and 79.
constexpr int most_floats(int M) { return M <= 16 ? 3840 : 7936; }
int parts_of(int M, int K, int r)
{
    if (M < 1) return 1;
    int s = M <= 32 ? 256 / M : 128 / ceil_div(M, 16);
    const int most = M <= 32 ? kLoraParts : kLoraTileParts;
    if (s > K / 512) s = K / 512;
    if (M <= 32 && s > most_floats(M) / (M * r)) s = most_floats(M) / (M * r);
    return s < 1 ? 1 : (s > most ? most : s);
}

// The form in slices of K: from 3 to 32 rows, of 4 to 8 slices of K, up to 8192 columns;
// 0 elsewhere.  32 rows of 8 adapters, rank 16: 12.5 us at 1024 x 4096 (streaming 19.6),
// 17.2 at 4096 x 4096 (22.1), 25.5 at 8192 x 4096 (26.7), 12.9 at 4096 x 2048 (16.7); but
// 33.4 at 11008 x 4096 (31.0), 11.4 at 4096 x 512 (12.0).  3 rows of one adapter: 9.0 us
// at 1024 x 4096 (13.1), 9.1 at 4096 x 2048 (10.1), 8.5 at 4096 x 1024 (7.9).  16 rows of
// 8192 x 8192, 16 slices: 40.6 (37.5).
constexpr int kSliceColumns = 8192;
int slices_of(int M, int N, int K)
{
    const int s = ceil_div(K, kLoraSlice);
    return M > 2 && M <= 32 && N >= 16 && N <= kSliceColumns && s >= 4 && s <= kLoraSlices ? s : 0;
}

// Floats of n parts of the base, H's parts behind them 16-byte aligned.
size_t base_floats(int n, int M, int N) { return ((size_t)n * M * N + 3) / 4 * 4; }

// Where no fused form fits, the base comes in fp32, some 32 M floats of rows at a time (128
// MB of workspace), in equal shares of whole tiles.  5000 rows of rank 4 at 4096 x 4096: 275
// us, in rounds of 16 M 312; 1000 at 11008 x 4096 166, in rounds of 8 M 240.
int base_rows(int M, int N)
{
    const int64_t rounds = ((int64_t)M * N + (1 << 25) - 1) >> 25;
    const int64_t rows = (M + rounds - 1) / rounds, whole = (rows + 127) / 128 * 128;
    return (int)(whole < M ? whole : M);
}
// Its parts of K: up to 64 rows as many as make 256 tiles of 64 x 64.  64 rows of 24
// adapters at 4096 x 4096: 22.7 us with 4, 39.8 with 1, 28.3 with 2, 31.2 with 8; 32 rows at
// 4096 x 14336 47, 103, 62, 52; but 64 at 11008 x 4096 46 with 1, 42 with 2.
int base_parts(int M, int N, int K)
{
    if (M > 64) return 1;
    int s = 256 / ceil_div(N, 64);
    if (s > K / 512) s = K / 512;
    return s < 1 ? 1 : (s > kLoraBaseParts ? kLoraBaseParts : s);
}
size_t base_need(int M, int N, int K, int r)
{
    return base_floats(base_parts(M, N, K), M, N) + (size_t)parts_of(M, K, r) * M * r;
}
size_t workspace_need(int M, int N, int K, int r)
{
    if (M == 0 || N == 0) return 0;
    const int s = slices_of(M, N, K), p = parts_of(M, K, r);
    size_t need = base_floats(s, M, N) + (size_t)(s > p ? s : p) * M * r;
    const int rows = base_rows(M, N), rest = M % rows;
    const size_t whole = base_need(rows, N, K, r), tail = rest ? base_need(rest, N, K, r) : 0;
    if (need < whole) need = whole;
    return (need < tail ? tail : need) * sizeof(float);
}

int check(const void* A, const int* ids, const void* Down, const void* Up, const float* scales, const void* C, int M,
          int N, int K, int r, int L, const void* workspace, size_t workspace_bytes)
{
    if (M < 0 || N < 0 || K < 0 || L < 0 || r < 1 || r > kMaxRank) return GF_ERR_INVALID_ARG;
    if (M > kMaxSize || N > kMaxSize || K > kMaxSize || L > kMaxSize) return GF_ERR_INVALID_ARG;
    if ((int64_t)M * K > kMaxElems || (int64_t)N * K > kMaxElems || (int64_t)M * N > kMaxElems ||
        (int64_t)r * K > kMaxElems || (int64_t)r * N > kMaxElems || (int64_t)M * r > kMaxElems)
        return GF_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GF_OK;
    if (off_grid(C, 2)) return GF_ERR_INVALID_ARG;
    if (off_grid(ids, 4)) return GF_ERR_INVALID_ARG;
    if (K > 0 && off_grid(A, 2)) return GF_ERR_INVALID_ARG;
    if (L > 0 && (off_grid(Up, 2) || (K > 0 && off_grid(Down, 2)))) return GF_ERR_INVALID_ARG;
    if (scales && off_grid(scales, 4)) return GF_ERR_INVALID_ARG;
    if (off_grid(workspace, 16) || workspace_bytes < workspace_need(M, N, K, r)) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

LoraArgs args(const void* A, const void* B, const int* ids, const void* Down, const void* Up, const float* scales,
              void* C, int M, int N, int K, int r, int L, void* workspace)
{
    LoraArgs a;
    a.A = (const uint16_t*)A; a.B = (const uint16_t*)B; a.ids = ids;
    a.Down = (const uint16_t*)Down; a.Up = (const uint16_t*)Up; a.scales = scales;
    a.C = (uint16_t*)C; a.H = (float*)workspace;
    a.base = nullptr; a.parts = 0;
    a.M = M; a.N = N; a.K = K; a.r = r; a.L = L;
    // the general forms leave K whole, and read H as one part
    const bool split = on16(A) && on16(Down) && K % 8 == 0 && on16(Up) && r % 8 == 0;
    a.S = split ? parts_of(M, K, r) : 1;
    a.part = (int64_t)M * r;
    return a;
}

constexpr int kGrid = 1 << 20;   // workgroups at most (a launch has fewer than 2^32 threads)
int grid_of(int64_t n) { return (int)(n < kGrid ? n : kGrid); }

// H = scale * A . Down^T for every row with an adapter.
int down(const LoraArgs& a, hipStream_t stream)
{
    if (on16(a.A) && on16(a.Down) && a.K % 8 == 0 && a.K > 0) {
        // a block has up to 16 adapters: as many workgroups, in about 512 of them
        const int blocks = ceil_div(a.M, 16);
        int Z = a.M <= 32 ? 16 : 512 / (blocks * a.S);
        if (Z > 16) Z = 16;
        if (Z > a.L) Z = a.L;
        if (Z < 1) Z = 1;
        const dim3 grid(grid_of((int64_t)blocks * Z), a.S);
        return status(a.r <= 16 ? launch_lora_down<LoraDownCfg<8, 1>>(a, grid, Z, stream)
                                : launch_lora_down<LoraDownCfg<8, 2>>(a, grid, Z, stream));
    } else {
        hipLaunchKernelGGL(lora_down_any_kernel, dim3(grid_of(a.M)), dim3(256), 0, stream, a);
    }
    return status(hipGetLastError());
}

// C = base + H . Up^T with BASE, else C += H . Up^T.
template <bool BASE>
int up(const LoraArgs& a, hipStream_t stream)
{
    if (on16(a.Up) && a.r % 8 == 0) {
        const int vec = (reinterpret_cast<uintptr_t>(a.C) & 7) == 0 && a.N % 4 == 0;
        const int64_t items = (int64_t)ceil_div(a.M, 16) * ceil_div(a.N, 16);
        // 64 columns a wave (a quarter of the loads of H, and of the waves), where there are
        // many and an adapter has several rows: 512 rows of 8 adapters at 4096 x 512 8.5 us
        // against 10.5 with 16 columns, 448 11.2 against 10.5; 1024 rows of 128 18.2 against
        // 20.5, of 256 26.1 against 25.8, of 1024 61 against 45.
        const bool wide = items >= 8192 && a.L <= a.M / 8;
        if (wide && a.S <= kLoraTileParts)
            hipLaunchKernelGGL((lora_up_kernel<kLoraTileParts, BASE>), dim3(grid_of((items / 4 + 3) / 4)), dim3(256), 0, stream, a, vec);
        else if (wide)
            hipLaunchKernelGGL((lora_up_kernel<kLoraParts, BASE>), dim3(grid_of((items / 4 + 3) / 4)), dim3(256), 0, stream, a, vec);
        else if (a.r <= 32)
            hipLaunchKernelGGL((lora_up_few_kernel<1, BASE>), dim3((int)(items + 3) / 4), dim3(256), 0, stream, a, vec);
        else if (a.r <= 64)
            hipLaunchKernelGGL((lora_up_few_kernel<2, BASE>), dim3((int)(items + 1) / 2), dim3(256), 0, stream, a, vec);
        else
            hipLaunchKernelGGL((lora_up_few_kernel<4, BASE>), dim3((int)items), dim3(256), 0, stream, a, vec);
    } else {
        hipLaunchKernelGGL(lora_up_any_kernel<BASE>, dim3(grid_of(((int64_t)a.M * a.N + 255) / 256)), dim3(256), 0, stream, a);
    }
    return status(hipGetLastError());
}

// The base as fp32 parts, then the adapters and the one rounding, `rows` rows at a time.
int by_parts(const LoraArgs& all, float* workspace, hipStream_t stream)
{
    const int rows = base_rows(all.M, all.N);
    for (int m = 0; m < all.M; m += rows) {
        const int n = all.M - m < rows ? all.M - m : rows, most = base_parts(n, all.N, all.K);
        LoraArgs a = args(all.A + (size_t)m * all.K, all.B, all.ids + m, all.Down, all.Up, all.scales,
                          all.C + (size_t)m * all.N, n, all.N, all.K, all.r, all.L,
                          workspace + base_floats(most, n, all.N));
        a.base = workspace;
        int rc = gemm_f32_parts(a.A, a.B, workspace, n, a.N, a.K, most, &a.parts, stream);
        if (!rc) rc = down(a, stream);
        if (!rc) rc = up<true>(a, stream);
        if (rc) return rc;
    }
    return GF_OK;
}

// Base and adapters in tiles: default_gemm_cfg's choice among four of its tiles.
template <class Cfg>
int tiles(const LoraArgs& a, int raster, hipStream_t stream)
{
    LoraTileArgs t;
    t.A = a.A; t.B = a.B; t.C = a.C;
    t.M = a.M; t.N = a.N; t.K = a.K;
    t.raster = raster;
    t.low = {a.H, a.ids, a.Up, a.part, a.S, a.r, a.L};
    return status(launch_lora_tile<Cfg>(t, stream));
}

int tiles(const LoraArgs& a, hipStream_t stream)
{
    const int64_t t25612 = (int64_t)ceil_div(a.M, 256) * ceil_div(a.N, 128);
    const int64_t t128 = (int64_t)ceil_div(a.M, 128) * ceil_div(a.N, 128);
    const int64_t t256 = (int64_t)ceil_div(a.M, 256) * ceil_div(a.N, 256);
    if (t256 >= 256 && a.K > 1536) return tiles<GemmCfg<256, 256, 64, 2, 256, 2>>(a, a.K <= 4096 ? 10 : (a.K < 16384 ? 0 : 4), stream);
    if (t25612 >= 256 && a.K >= 2048) return tiles<GemmCfg<256, 128, 64, 3, 256, 2>>(a, t25612 >= 512 ? 10 : 0, stream);
    if (t128 > 256) return tiles<GemmCfg<128, 128, 64, 2, 256, 0>>(a, 0, stream);
    if (t128 >= 128) return tiles<GemmCfg<128, 128, 64, 4, 256, 2>>(a, 0, stream);
    return tiles<GemmCfg<64, 64, 64, 3, 256, 0>>(a, 0, stream);
}

// Base and adapters, B in vectors; GF_ERR_UNSUPPORTED where it does not fit.  Up to 2
// rows (4096 x 4096, rank 16: 10.5 us for one and 14.4 for two, the streaming form
// 15.0 and 15.2; at 4 rows 18.6 against 15.1).  It works out H itself up to 64 ranks in
// all: 10.5 us against 15.1 with a launch for it at one row, 14.4 against 17.0 at two,
// 15.8 against 18.0 at rank 64; at 128 ranks 29 against 19.
constexpr int kVecRows = 2, kVecSelf = 64;

template <int MV, int UNROLL>
int vec(const LoraArgs& a, hipStream_t stream)
{
    constexpr int WAVES = 8;
    const int groups = ceil_div(a.N, WAVES), grid = groups < 256 ? groups : 256, iters = ceil_div(groups, grid);
    const int64_t most = a.M < a.L ? a.M : a.L;          // adapters in use
    const int64_t up_bytes = most * iters * WAVES * a.r * 2, sums = (int64_t)iters * WAVES * MV * 4;
    if (up_bytes > 100 * 1024 || sums > 64 * 1024 || (int64_t)MV * lora_vec_pad(a.K, UNROLL) * 16 > 128 * 1024)
        return GF_ERR_UNSUPPORTED;
    const LoraVecLds at(MV, a.K, a.r, UNROLL, iters * WAVES, (int)most);
    if (at.total > 159 * 1024) return GF_ERR_UNSUPPORTED;
    if (most * a.r <= kVecSelf)
        return status(launch_lora_vec<MV, UNROLL, WAVES, true>(a, grid, iters, (int)most, at.total, stream));
    const int rc = down(a, stream);
    return rc ? rc : status(launch_lora_vec<MV, UNROLL, WAVES, false>(a, grid, iters, (int)most, at.total, stream));
}

// Loads in flight by how they divide a row's: at 4096 x 4096 10.4 us with 8, 10.6 with 4,
// 12.5 with 2; at K = 2048 8.6, 7.2, 7.7; at 1024 7.5, 6.6, 5.8 (but at 11008 25.7, 27.3,
// 30.6).
template <int MV>
int vec(const LoraArgs& a, hipStream_t stream)
{
    if (a.K % 4096 == 0) return vec<MV, 8>(a, stream);
    return a.K >= 2048 ? vec<MV, 4>(a, stream) : vec<MV, 2>(a, stream);
}

// Base and adapters, B streamed once: up to 16 rows of K <= 8192, 32 of K <= 4096
// (a wave holds its part of A in registers).
bool band_takes(int M, int N, int K) { return N >= 16 && ((M <= 16 && K <= 8192) || (M <= 32 && K <= 4096)); }

// Whether the streaming form works out H itself: one adapter of up to 16 ranks (32
// rows at 4096 x 1024: 10.5 us against 12.1 with a launch for it, 16 8.6 against 10.4; at
// 16384 x 2048 and past even; with two blocks of ranks 18.4 against 15.2).
bool band_self(const LoraArgs& a)
{
    const int64_t most = a.M < a.L ? a.M : a.L;
    return most * ceil_div(a.r, 16) <= 1 && a.M * a.r <= most_floats(a.M);
}

template <int MB, int XB>
int band(const LoraArgs& a, hipStream_t stream)
{
    constexpr int RING = MB == 1 ? 4 : 3;
    if constexpr (MB * XB <= 4)                  // Down's ranks in registers beside A
        if (band_self(a)) return status(launch_lora_band<LoraBandCfg<MB, XB, RING>, true>(a, stream));
    const int rc = down(a, stream);
    if (rc) return rc;
    // a smaller ring where H takes its place: 16 rows of rank 248 and 256, 32 of rank 256
    if (LoraBandCfg<MB, XB, RING>::lds_bytes(a.S * a.M * a.r) <= 160 * 1024)
        return status(launch_lora_band<LoraBandCfg<MB, XB, RING>, false>(a, stream));
    return status(launch_lora_band<LoraBandCfg<MB, XB, RING - 1>, false>(a, stream));
}

int band(const LoraArgs& a, hipStream_t stream)
{
    if (a.M > 16) return a.K <= 2048 ? band<2, 2>(a, stream) : band<2, 4>(a, stream);
    if (a.K <= 2048) return band<1, 2>(a, stream);
    return a.K <= 4096 ? band<1, 4>(a, stream) : band<1, 8>(a, stream);
}

}  // namespace
}  // namespace gf

using namespace gf;

extern "C" {

size_t lora_workspace_bytes(int M, int N, int K, int r)
{
    if (M < 0 || N < 0 || K < 0 || r < 1 || r > kMaxRank) return 0;
    return workspace_need(M, N, K, r);
}

int lora_add_f16(const void* A, const int* ids, const void* Down, const void* Up, const float* scales, void* C, int M,
                 int N, int K, int r, int L, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check(A, ids, Down, Up, scales, C, M, N, K, r, L, workspace, workspace_bytes);
    if (rc || M == 0 || N == 0 || L == 0) return rc;
    const LoraArgs a = args(A, nullptr, ids, Down, Up, scales, C, M, N, K, r, L, workspace);
    rc = down(a, (hipStream_t)stream);
    return rc ? rc : up<false>(a, (hipStream_t)stream);
}

int lora_add_f32(const void* A, const int* ids, const void* Down, const void* Up, const float* scales,
                 const float* base, void* C, int M, int N, int K, int r, int L, void* workspace,
                 size_t workspace_bytes, void* stream)
{
    int rc = check(A, ids, Down, Up, scales, C, M, N, K, r, L, workspace, workspace_bytes);
    if (rc || M == 0 || N == 0) return rc;
    if (off_grid(base, 4)) return GF_ERR_INVALID_ARG;
    LoraArgs a = args(A, nullptr, ids, Down, Up, scales, C, M, N, K, r, L, workspace);
    a.base = base;
    a.parts = 1;
    if (L > 0) rc = down(a, (hipStream_t)stream);
    return rc ? rc : up<true>(a, (hipStream_t)stream);
}

int gemm_f16_nt_lora(const void* A, const void* B, const int* ids, const void* Down, const void* Up,
                     const float* scales, void* C, int M, int N, int K, int r, int L, void* workspace,
                     size_t workspace_bytes, void* stream)
{
    int rc = check(A, ids, Down, Up, scales, C, M, N, K, r, L, workspace, workspace_bytes);
    if (rc || M == 0 || N == 0) return rc;
    if (K > 0 && off_grid(B, 2)) return GF_ERR_INVALID_ARG;
    if (L == 0) return gemm_f16_nt(A, B, C, M, N, K, stream);
    const LoraArgs a = args(A, B, ids, Down, Up, scales, C, M, N, K, r, L, workspace);
    const bool al = on16(A) && on16(B) && on16(Down) && on16(Up) && K % 8 == 0 && r % 8 == 0 && K > 0;
    if (al && M <= kVecRows) {
        rc = M == 1 ? vec<1>(a, (hipStream_t)stream) : vec<2>(a, (hipStream_t)stream);
        if (rc != GF_ERR_UNSUPPORTED) return rc;
    }
    const int slices = slices_of(M, N, K);
    if (al && slices > 0) {
        LoraArgs b = a;
        b.S = slices;
        b.H = (float*)workspace + base_floats(slices, M, N);
        return status(M <= 16 ? launch_lora_slices<LoraSliceCfg<1, 8>>(b, (float*)workspace, (hipStream_t)stream)
                              : launch_lora_slices<LoraSliceCfg<2, 6>>(b, (float*)workspace, (hipStream_t)stream));
    }
    if (al && band_takes(M, N, K)) return band(a, (hipStream_t)stream);
    // From 33 to 64 rows the base in parts is ahead of tiles (64 rows of 24 adapters at
    // 4096 x 4096: 22.7 us against 43.0; of 8 at 16384 x 4096 52 against 63, at 11008 x 4096
    // 46 against 44).
    if (al && on16(C) && M > 64) {
        rc = down(a, (hipStream_t)stream);
        return rc ? rc : tiles(a, (hipStream_t)stream);
    }
    return by_parts(a, (float*)workspace, (hipStream_t)stream);
}

}  // extern "C"
