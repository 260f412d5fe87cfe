// Grouped (per expert) products: launch choice and C-ABI entry points.
#include "../../include/gemvfp16.h"
#include "grouped_kernel.hpp"

namespace gf {
namespace {

constexpr int64_t kGroupMaxElems = (int64_t(1) << 31) - 1;
constexpr int64_t kGroupMaxGrid = (int64_t(1) << 31) - 1;

bool g_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// X has rows x K entries in all and Y rows x N; W has N x K in each of E groups
// (W as a whole may pass 2^31: it is addressed group by group).
int validate_groups(const void* offsets, int T, int E, int N, int K)
{
    if (T < 0 || E < 0 || N < 0 || K < 0) return GF_ERR_INVALID_ARG;
    if ((int64_t)T * K > kGroupMaxElems || (int64_t)N * K > kGroupMaxElems || (int64_t)T * N > kGroupMaxElems)
        return GF_ERR_INVALID_ARG;
    if (E > 0 && (!offsets || !g_aligned(offsets, 4))) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

bool bad_ptr(const void* p, uintptr_t a) { return !p || !g_aligned(p, a); }

template <class Cfg>
int run_rows(GroupRowArgs a, bool al, hipStream_t stream)
{
    // Tiles at most: whole ones, and a partial one for every group that can have a row.
    const int64_t blocks = (int64_t)a.g.T / Cfg::BM + (a.g.E < a.g.T ? a.g.E : a.g.T);
    const int64_t grid = blocks * ceil_div(a.N, Cfg::BN);
    if (grid > kGroupMaxGrid) return GF_ERR_INVALID_ARG;
    const hipError_t e = al ? launch_grouped<Cfg, EPI_F16, true>(a, grid, stream)
                            : launch_grouped<Cfg, EPI_F16, false>(a, grid, stream);
    return e == hipSuccess ? GF_OK : GF_ERR_HIP;
}

// LB: 0 for B[e] N x K, 1 for K x N.
template <int LB>
int rows_impl(const void* A, const void* B, void* C, const int* offsets, int T, int E, int N, int K,
              hipStream_t stream)
{
    const int rc = validate_groups(offsets, T, E, N, K);
    if (rc) return rc;
    if (T == 0 || E == 0 || N == 0) return GF_OK;
    if (K > 0 && (bad_ptr(A, 2) || bad_ptr(B, 2))) return GF_ERR_INVALID_ARG;
    if (bad_ptr(C, 2)) return GF_ERR_INVALID_ARG;
    GroupRowArgs a;
    a.A = (const uint16_t*)A;
    a.B = (const uint16_t*)B;
    a.C = C;
    a.M = 0; a.N = N; a.K = K;
    a.g.offsets = offsets; a.g.E = E; a.g.T = T;
    a.c_bytes = 2;
    const bool al = g_aligned(A, 16) && g_aligned(B, 16) && g_aligned(C, 16) && K % 8 == 0 &&
                    (LB == 0 || N % 8 == 0);
    const int64_t mean = (int64_t)T / E;
    if (mean >= 192 && ((int64_t)T / 256) * ceil_div(N, 256) >= 128)
        return run_rows<GemmCfg<256, 256, 64, 2, 256, 2, 0, LB>>(a, al, stream);
    if (mean >= 64) return run_rows<GemmCfg<128, 128, 64, 2, 256, 2, 0, LB>>(a, al, stream);
    return run_rows<GemmCfg<64, 128, 64, 2, 256, 2, 0, LB>>(a, al, stream);
}

template <class Cfg>
int run_depth(GroupDepthArgs a, bool al, bool f32, hipStream_t stream)
{
    const int64_t grid = (int64_t)a.g.E * GroupDepthArgs::run_length<Cfg::BM, Cfg::BN>(a.M, a.N) * 8;
    if (grid > kGroupMaxGrid) return GF_ERR_INVALID_ARG;
    hipError_t e;
    if (f32)
        e = al ? launch_grouped<Cfg, EPI_F32_STORE, true>(a, grid, stream)
               : launch_grouped<Cfg, EPI_F32_STORE, false>(a, grid, stream);
    else
        e = al ? launch_grouped<Cfg, EPI_F16, true>(a, grid, stream)
               : launch_grouped<Cfg, EPI_F16, false>(a, grid, stream);
    return e == hipSuccess ? GF_OK : GF_ERR_HIP;
}

}  // namespace
}  // namespace gf

using namespace gf;

extern "C" {

int gemm_f16_grouped_nt(const void* A, const void* B, void* C, const int* offsets, int T, int E, int N,
                        int K, void* stream)
{
    return rows_impl<0>(A, B, C, offsets, T, E, N, K, (hipStream_t)stream);
}

int gemm_f16_grouped_nn(const void* A, const void* B, void* C, const int* offsets, int T, int E, int N,
                        int K, void* stream)
{
    return rows_impl<1>(A, B, C, offsets, T, E, N, K, (hipStream_t)stream);
}

int gemm_f16_grouped_tn(const void* A, const void* B, void* C, const int* offsets, int T, int E, int M,
                        int N, int c_f32, void* stream)
{
    if (c_f32 != 0 && c_f32 != 1) return GF_ERR_INVALID_ARG;
    const int rc = validate_groups(offsets, T, E, M, N);
    if (rc) return rc;
    if (E == 0 || M == 0 || N == 0) return GF_OK;
    if (T > 0 && (bad_ptr(A, 2) || bad_ptr(B, 2))) return GF_ERR_INVALID_ARG;
    if (bad_ptr(C, c_f32 ? 4 : 2)) return GF_ERR_INVALID_ARG;
    GroupDepthArgs a;
    a.A = (const uint16_t*)A;
    a.B = (const uint16_t*)B;
    a.C = C;
    a.M = M; a.N = N; a.K = 0;
    a.g.offsets = offsets; a.g.E = E; a.g.T = T;
    a.c_bytes = c_f32 ? 4 : 2;
    const bool al = g_aligned(A, 16) && g_aligned(B, 16) && g_aligned(C, 16) && M % 8 == 0 && N % 8 == 0;
    if ((int64_t)E * ceil_div(M, 256) * ceil_div(N, 256) >= 256)
        return run_depth<GemmCfg<256, 256, 64, 2, 256, 2, 1, 1>>(a, al, c_f32 != 0, (hipStream_t)stream);
    return run_depth<GemmCfg<128, 128, 64, 2, 256, 2, 1, 1>>(a, al, c_f32 != 0, (hipStream_t)stream);
}

}  // extern "C"
