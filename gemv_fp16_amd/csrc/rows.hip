// Rows to experts and back: dispatch, combine and its gradient.
//
// All three are bound by the rows' bytes: each is read once and written once, 16
// bytes a lane, at whatever 2-byte alignment the rows have (the vector loads and
// stores of gfx950 take it).
#include "../../include/gemvfp16.h"
#include "wave.hpp"

namespace gf {
namespace {

constexpr int kMaxTop = 64;          // lane j holds a token's j-th place
constexpr int kMaxSize = 1 << 30;
constexpr int64_t kMaxElems = (int64_t(1) << 31) - 1;
constexpr int kWaves = 4;
constexpr int kGrid = 1 << 20;       // workgroups at most (a launch has fewer than 2^32 threads)

// 8 fp16 at any 2-byte alignment; n < 8 of them at a row's end, zeros for the rest.
__device__ __forceinline__ half8 load8(const uint16_t* p, int n)
{
    half8 v = {};
    if (n >= 8) __builtin_memcpy(&v, p, 16);
    else
        for (int i = 0; i < n; ++i) v[i] = __builtin_bit_cast(_Float16, p[i]);
    return v;
}

__device__ __forceinline__ void store8(uint16_t* p, half8 v, int n)
{
    if (n >= 8) __builtin_memcpy(p, &v, 16);
    else
        for (int i = 0; i < n; ++i) p[i] = __builtin_bit_cast(uint16_t, (_Float16)v[i]);
}

struct MoveArgs {
    const uint16_t* in;        // dispatch: X; combine: C
    const int* place;
    const float* weights;
    uint16_t* out;             // dispatch: A; combine: Y
    int T, k, R, D;
    int pieces;                // 512-wide pieces of a row
};

// A wave moves a 512-wide piece of a token's row to the token's k places.
__global__ __launch_bounds__(kWaves * kWave) void dispatch_kernel(MoveArgs a)
{
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t items = (int64_t)a.T * a.pieces;
    for (int64_t it = (int64_t)blockIdx.x * kWaves + wave; it < items; it += (int64_t)gridDim.x * kWaves) {
        const int t = (int)(it / a.pieces), d = ((int)(it % a.pieces) * kWave + lane) * 8;
        const int at = lane < a.k ? a.place[(size_t)t * a.k + lane] : -1;
        const half8 v = load8(a.in + (size_t)t * a.D + d, a.D - d);
        for (int j = 0; j < a.k; ++j) {
            const int r = lane_value(at, j);
            if ((unsigned)r < (unsigned)a.R) store8(a.out + (size_t)r * a.D + d, v, a.D - d);
        }
    }
}

// A wave sums a 512-wide piece of a token's k rows.
template <bool WEIGHTS>
__global__ __launch_bounds__(kWaves * kWave) void combine_kernel(MoveArgs a)
{
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t items = (int64_t)a.T * a.pieces;
    for (int64_t it = (int64_t)blockIdx.x * kWaves + wave; it < items; it += (int64_t)gridDim.x * kWaves) {
        const int t = (int)(it / a.pieces), d = ((int)(it % a.pieces) * kWave + lane) * 8;
        const int at = lane < a.k ? a.place[(size_t)t * a.k + lane] : -1;
        const float w = WEIGHTS && lane < a.k ? a.weights[(size_t)t * a.k + lane] : 1.0f;
        float acc[8] = {};
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int r = lane_value(at, j);
            if ((unsigned)r >= (unsigned)a.R) continue;
            const float wj = lane_value(w, j);
            const half8 v = load8(a.in + (size_t)r * a.D + d, a.D - d);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = WEIGHTS ? __builtin_fmaf(wj, (float)v[i], acc[i]) : acc[i] + (float)v[i];
        }
        half8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (_Float16)acc[i];
        store8(a.out + (size_t)t * a.D + d, o, a.D - d);
    }
}

struct CombineGradArgs {
    const uint16_t* dY;
    const uint16_t* C;
    const int* place;
    const float* weights;
    uint16_t* dC;
    float* dweights;
    int T, k, R, D;
};

// A workgroup takes a token; its waves share the row's width, and their parts of
// the dot products are added in wave order.
__global__ __launch_bounds__(kWaves * kWave) void combine_grad_kernel(CombineGradArgs a)
{
    __shared__ float parts[kWaves][kMaxTop];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t row = (size_t)t * a.k;
        const int at = lane < a.k ? a.place[row + lane] : -1;
        const float w = lane < a.k ? a.weights[row + lane] : 0.0f;
        float dot = 0.0f;                        // lane j: this wave's part of choice j's
        for (int d0 = wave * kWave * 8; d0 < a.D; d0 += kWaves * kWave * 8) {
            const int d = d0 + lane * 8, n = a.D - d;
            const half8 g = load8(a.dY + (size_t)t * a.D + d, n);
            for (int j = 0; j < a.k; ++j) {
                const int r = lane_value(at, j);
                if ((unsigned)r >= (unsigned)a.R) continue;
                const float wj = lane_value(w, j);
                const half8 c = load8(a.C + (size_t)r * a.D + d, n);
                half8 o;
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i] = (_Float16)(wj * (float)g[i]);
                    s = __builtin_fmaf((float)g[i], (float)c[i], s);
                }
                store8(a.dC + (size_t)r * a.D + d, o, n);
                s = wave_sum(s);
                if (lane == j) dot += s;
            }
        }
        parts[wave][lane] = dot;
        __syncthreads();
        if (wave == 0 && lane < a.k) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) s += parts[v][lane];
            a.dweights[row + lane] = s;
        }
        __syncthreads();
    }
}

bool off_grid(const void* p, uintptr_t a) { return !p || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int check_sizes(int T, int k, int R, int D)
{
    if (T < 0 || R < 0 || D < 0 || k < 1 || k > kMaxTop) return GF_ERR_INVALID_ARG;
    if (T > kMaxSize || R > kMaxSize || D > kMaxSize) return GF_ERR_INVALID_ARG;
    if ((int64_t)T * k > kMaxElems || (int64_t)T * D > kMaxElems || (int64_t)R * D > kMaxElems) return GF_ERR_INVALID_ARG;
    return GF_OK;
}

int status(hipError_t e) { return e == hipSuccess ? GF_OK : GF_ERR_HIP; }

template <class Kernel>
int move(Kernel kern, const void* in, const int* place, const float* weights, void* out, int T, int k, int R, int D,
         hipStream_t stream)
{
    MoveArgs a;
    a.in = (const uint16_t*)in; a.place = place; a.weights = weights; a.out = (uint16_t*)out;
    a.T = T; a.k = k; a.R = R; a.D = D;
    a.pieces = ceil_div(D, 512);
    const int64_t groups = ((int64_t)T * a.pieces + kWaves - 1) / kWaves;
    hipLaunchKernelGGL(kern, dim3((unsigned)(groups < kGrid ? groups : kGrid)), dim3(kWaves * kWave), 0, stream, a);
    return status(hipGetLastError());
}

}  // namespace
}  // namespace gf

using namespace gf;

extern "C" {

int dispatch_f16(const void* X, const int* place, void* A, int T, int k, int R, int D, void* stream)
{
    const int rc = check_sizes(T, k, R, D);
    if (rc) return rc;
    if (T == 0 || D == 0) return GF_OK;
    if (off_grid(X, 2) || off_grid(place, 4) || (R > 0 && off_grid(A, 2))) return GF_ERR_INVALID_ARG;
    if (R == 0) return GF_OK;
    return move(dispatch_kernel, X, place, nullptr, A, T, k, R, D, (hipStream_t)stream);
}

int combine_f16(const void* C, const int* place, const float* weights, void* Y, int T, int k, int R, int D, void* stream)
{
    const int rc = check_sizes(T, k, R, D);
    if (rc) return rc;
    if (T == 0 || D == 0) return GF_OK;
    if (off_grid(Y, 2) || off_grid(place, 4) || (R > 0 && off_grid(C, 2))) return GF_ERR_INVALID_ARG;
    if (weights && off_grid(weights, 4)) return GF_ERR_INVALID_ARG;
    if (weights) return move(combine_kernel<true>, C, place, weights, Y, T, k, R, D, (hipStream_t)stream);
    return move(combine_kernel<false>, C, place, nullptr, Y, T, k, R, D, (hipStream_t)stream);
}

int combine_f16_bwd(const void* dY, const void* C, const int* place, const float* weights, void* dC, float* dweights,
                    int T, int k, int R, int D, void* stream)
{
    const int rc = check_sizes(T, k, R, D);
    if (rc) return rc;
    if (T == 0) return GF_OK;
    if (off_grid(place, 4) || off_grid(weights, 4) || off_grid(dweights, 4)) return GF_ERR_INVALID_ARG;
    if (D > 0 && (off_grid(dY, 2) || (R > 0 && (off_grid(C, 2) || off_grid(dC, 2))))) return GF_ERR_INVALID_ARG;
    CombineGradArgs a;
    a.dY = (const uint16_t*)dY; a.C = (const uint16_t*)C; a.place = place; a.weights = weights;
    a.dC = (uint16_t*)dC; a.dweights = dweights;
    a.T = T; a.k = k; a.R = R; a.D = D;
    hipLaunchKernelGGL(combine_grad_kernel, dim3(T < kGrid ? T : kGrid), dim3(kWaves * kWave), 0, (hipStream_t)stream, a);
    return status(hipGetLastError());
}

}  // extern "C"
