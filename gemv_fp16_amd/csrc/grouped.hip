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
    if (T < 0 || E < 0 || N < 0 || K < 0 || E > kMaxGroups) return GF_ERR_INVALID_ARG;
    if (T > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return GF_ERR_INVALID_ARG;
    if ((int64_t)T * K > kGroupMaxElems || (int64_t)N * K > kGroupMaxElems || (int64_t)T * N > kGroupMaxElems)
        return GF_ERR_INVALID_ARG;
    if (E > 0 && (!offsets || !g_aligned(offsets, 4))) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

bool bad_ptr(const void* p, uintptr_t a) { return !p || !g_aligned(p, a); }

// Tiles at most: whole ones, and a partial one for every group that can have a row.
template <class Cfg, class Args>
int64_t most_tiles(const Args& a)
{
    return ((int64_t)a.g.T / Cfg::BM + (a.g.E < a.g.T ? a.g.E : a.g.T)) * ceil_div(a.N, Cfg::BN);
}

template <class Cfg, class Args>
int run_rows(const Args& a, int64_t grid, bool al, hipStream_t stream)
{
    if (grid > kGroupMaxGrid) return GF_ERR_INVALID_ARG;
    const hipError_t e = al ? launch_grouped<Cfg, EPI_F16, true>(a, grid, stream)
                            : launch_grouped<Cfg, EPI_F16, false>(a, grid, stream);
    return e == hipSuccess ? GF_OK : GF_ERR_HIP;
}

template <class Cfg>
int run_rows(const GroupRowArgs& a, bool al, hipStream_t stream)
{
    return run_rows<Cfg>(a, most_tiles<Cfg>(a), al, stream);
}

// 256 x 256 tiles run in rounds of 256, one to a CU; a last round that is at most
// half full costs as much as a full one (8191 rows over 8 groups by 4096: 2.3
// rounds).  So the tiles that fill whole rounds run as one launch and the rest as
// a second one of 128 x 128 tiles, which spread over the chip.  How many there are
// is known on the device only: both launches hold the most there can be, and the
// second one's workgroups end at once where the last round is fuller.  The same
// products in the same order, so the results do not depend on the split.  Where
// there cannot be more than one round, one launch (98 us against 102 at 4096 rows
// over 8 groups of 2048 x 4096).
template <int LB>
int run_rounds(const GroupRowArgs& a, bool al, hipStream_t stream)
{
    typedef GemmCfg<256, 256, 64, 2, 256, 2, 0, LB> Big;
    typedef GemmCfg<128, 128, 64, 4, 256, 2, 0, LB> Small;
    if (most_tiles<Big>(a) <= 256) return run_rows<Big>(a, al, stream);
    GroupRowShare<1> a1;
    GroupRowShare<2> a2;
    static_cast<GemmArgs&>(a1) = a;
    static_cast<GemmArgs&>(a2) = a;
    a1.g = a2.g = a.g;
    const int rc = run_rows<Big>(a1, most_tiles<Big>(a), al, stream);
    return rc ? rc : run_rows<Small>(a2, 4 * 128, al, stream);
}

template <class Cfg>
int run_band(const GroupRowArgs& a, hipStream_t stream)
{
    // Two workgroups to a CU (two tasks in flight a wave), about 256 of them in
    // all but at least 16 a group (most groups of a decode batch have rows, and
    // uneven ones leave a tail).
    const int64_t want = 256 / a.g.E, blocks = ceil_div(a.N, 16);
    int64_t parts = want < 16 ? 16 : (want > 64 ? 64 : want);
    if (parts > blocks) parts = blocks;
    const int64_t grid = (a.g.T / (16 * Cfg::MB) + (a.g.E < a.g.T ? a.g.E : a.g.T)) * parts;
    if (grid > kGroupMaxGrid) return GF_ERR_INVALID_ARG;
    const hipError_t e = launch_group_band<Cfg>(a, 2, (int)parts, grid, stream);
    return e == hipSuccess ? GF_OK : GF_ERR_HIP;
}

// The launch for T rows over E groups, of which only the mean is known.  Timed
// side by side with B rotated through HBM (us):
//  * a handful of rows a group, K-contiguous B: the streaming form, 36 against
//    57 for every tile at T = 48, E = 16, 4096 x 2048; 41 against 59 at T = 16,
//    E = 8, 4096 x 4096; 16 against 20 at T = 18, E = 17, 488 x 2672.  At a mean
//    of 19 the 64 x 64 tile is ahead of it (34 against 39).  It ends at K = 8192,
//    where each wave's part of A fills its registers (16 rows over 8 of 4096 x 14336
//    in the 64 x 64 tile 169, of 14336 x 4096 here 137);
//  * then 64 x 64 up to a mean of 64 (64 against 68 at T = 500, E = 16) and where
//    there are few of 128 x 128 (46 against 74 at T = 1284, E = 2, 448 x 7072; 18
//    against 23 at T = 400, E = 4, 2048 x 2048), 128 x 128 with three stages beyond
//    (45 against 56 at T = 1111, E = 8, 2048 x 4096);
//  * 256 x 256 where the groups fill several of them, they fill the CUs and K is
//    long enough to fill their pipeline (278 against 330 at T = 8191, E = 8, 4096 x
//    4096; 98 against 121 for K x N B at T = 4096, 2048 x 4096; but 50 against 46
//    at T = 5000, E = 16, 4096 x 512);
//  * K x N B (transposing reads, which the one-wave-per-SIMD tiles have): 64 x 128
//    below a mean of 16 (42 against 50 and 58 at T = 48, E = 16, 4096 x 2048), 128 x
//    128 beyond (33 against 37 at T = 500, E = 16, 2048 x 2048);
//  * up to K = 1024, tiles that leave room for two workgroups on a CU, so that one
//    stores while the other multiplies: 128 x 128 with two stages (71 against 84 at
//    T = 5000, E = 16, 4096 x 1024; 43 against 56 at T = 7600, E = 41, K x N of 320
//    x 2784), 64 x 128 for few rows (31 against 40 at T = 306, E = 10, 816 x 6568).
template <int LB>
int rows_dispatch(const GroupRowArgs& a, bool al, hipStream_t stream)
{
    const int64_t mean = (int64_t)a.g.T / a.g.E;
    if constexpr (LB == 0) {
        if (al && mean <= 12 && a.N >= 16 && a.K > 0) {
            if (mean > 4 && a.K <= 4096)
                return a.K <= 2048 ? run_band<GroupBandCfg<2, 2>>(a, stream) : run_band<GroupBandCfg<2, 4>>(a, stream);
            if (a.K <= 2048) return run_band<GroupBandCfg<1, 2>>(a, stream);
            if (a.K <= 4096) return run_band<GroupBandCfg<1, 4>>(a, stream);
            if (a.K <= 8192) return run_band<GroupBandCfg<1, 8>>(a, stream);
        }
    }
    if (mean >= 192 && a.K > 1024 && ((int64_t)a.g.T / 256) * ceil_div(a.N, 256) >= 128)
        return run_rounds<LB>(a, al, stream);
    if constexpr (LB == 0)
        if (mean < 64 || most_tiles<GemmCfg<128, 128, 64, 3, 256, 2, 0, 0>>(a) < 128)
            return run_rows<GemmCfg<64, 64, 64, 3, 256, 0, 0, 0>>(a, al, stream);
    if constexpr (LB == 1)
        if (mean < (a.K > 1024 ? 16 : 64))
            return run_rows<GemmCfg<64, 128, 64, 2, 256, 2, 0, LB>>(a, al, stream);
    if (a.K > 1024) return run_rows<GemmCfg<128, 128, 64, 3, 256, 2, 0, LB>>(a, al, stream);
    return run_rows<GemmCfg<128, 128, 64, 2, 256, 2, 0, LB>>(a, al, stream);
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
    const bool al = g_aligned(A, 16) && g_aligned(B, 16) && g_aligned(C, 16) && K % 8 == 0 &&
                    (LB == 0 || N % 8 == 0);
    return rows_dispatch<LB>(a, al, stream);
}

template <class Cfg>
int run_depth(GroupDepthArgs a, bool al, bool f32, hipStream_t stream)
{
    const int64_t grid = (int64_t)a.g.E * GroupDepthArgs::run_length<Cfg::BM, Cfg::BN>(a.M, a.N) * 8;
    if (grid > kGroupMaxGrid) return GF_ERR_INVALID_ARG;
    hipError_t e;
    if (f32)
        e = al ? launch_grouped<Cfg, EPI_F32_ROWS, true>(a, grid, stream)
               : launch_grouped<Cfg, EPI_F32_ROWS, false>(a, grid, stream);
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
    // Shallow groups are all start and store, which three workgroups on a CU overlap
    // (48 KB of LDS each): 128 x 128 tiles in steps of 32 rows, 56 us against 62 at
    // 2999 rows over 32 groups of 1024 x 2048 (61 in steps of 64, two to a CU), 154
    // against 192 at 600 over 2 of 8192 x 8192.  Deep ones are matrix work: 307
    // against 233 at 8192 over 2 of 4096 x 4096; even at 4096 over 8 (110).
    if ((int64_t)E * ceil_div(M, 256) * ceil_div(N, 256) >= 256 && T / E >= 384)
        return run_depth<GemmCfg<256, 256, 64, 2, 256, 2, 1, 1>>(a, al, c_f32 != 0, (hipStream_t)stream);
    return run_depth<GemmCfg<128, 128, 32, 3, 256, 2, 1, 1>>(a, al, c_f32 != 0, (hipStream_t)stream);
}

}  // extern "C"
