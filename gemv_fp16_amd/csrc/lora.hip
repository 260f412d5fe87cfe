// Low-rank adapters: argument checks, launch choice and C-ABI entry points.
#include "../../include/gemvfp16.h"
#include "lora_kernel.hpp"

namespace gf {
namespace {

constexpr int kMaxRank = 256;
constexpr int kMaxSize = 1 << 30;
constexpr int64_t kMaxElems = (int64_t(1) << 31) - 1;

bool off_grid(const void* p, uintptr_t a) { return !p || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int status(hipError_t e) { return e == hipSuccess ? GF_OK : GF_ERR_HIP; }

size_t workspace_need(int M, int r) { return (size_t)M * r * sizeof(float); }

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
    if (off_grid(workspace, 16) || workspace_bytes < workspace_need(M, r)) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

int add(const LoraArgs& a, hipStream_t stream)
{
    const bool al = on16(a.A) && on16(a.Down) && a.K % 8 == 0;
    const int rows = a.M < (1 << 20) ? a.M : 1 << 20;
    if (al)
        hipLaunchKernelGGL(lora_down_kernel<true>, dim3(rows), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(lora_down_kernel<false>, dim3(rows), dim3(256), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return GF_ERR_HIP;
    const int64_t groups = ((int64_t)a.M * a.N + 255) / 256;
    hipLaunchKernelGGL(lora_up_kernel, dim3((unsigned)(groups < (1 << 20) ? groups : 1 << 20)), dim3(256), 0, stream, a);
    return status(hipGetLastError());
}

}  // namespace
}  // namespace gf

using namespace gf;

extern "C" {

size_t lora_workspace_bytes(int M, int N, int K, int r)
{
    if (M < 0 || N < 0 || K < 0 || r < 1 || r > kMaxRank) return 0;
    return workspace_need(M, r);
}

int lora_add_f16(const void* A, const int* ids, const void* Down, const void* Up, const float* scales, void* C, int M,
                 int N, int K, int r, int L, void* workspace, size_t workspace_bytes, void* stream)
{
    const int rc = check(A, ids, Down, Up, scales, C, M, N, K, r, L, workspace, workspace_bytes);
    if (rc || M == 0 || N == 0 || L == 0) return rc;
    LoraArgs a;
    a.A = (const uint16_t*)A; a.ids = ids; a.Down = (const uint16_t*)Down; a.Up = (const uint16_t*)Up;
    a.scales = scales; a.C = (uint16_t*)C; a.H = (float*)workspace;
    a.M = M; a.N = N; a.K = K; a.r = r; a.L = L;
    return add(a, (hipStream_t)stream);
}

int gemm_f16_nt_lora(const void* A, const void* B, const int* ids, const void* Down, const void* Up,
                     const float* scales, void* C, int M, int N, int K, int r, int L, void* workspace,
                     size_t workspace_bytes, void* stream)
{
    int rc = check(A, ids, Down, Up, scales, C, M, N, K, r, L, workspace, workspace_bytes);
    if (rc || M == 0 || N == 0) return rc;
    rc = gemm_f16_nt(A, B, C, M, N, K, stream);
    if (rc || L == 0) return rc;
    return lora_add_f16(A, ids, Down, Up, scales, C, M, N, K, r, L, workspace, workspace_bytes, stream);
}

}  // extern "C"
