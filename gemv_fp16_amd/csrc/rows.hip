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
constexpr int kTogether = 4;         // rows whose loads are in flight together
constexpr int kGrid = 1 << 20;       // workgroups at most (a launch has fewer than 2^32 threads)

// A lane's 8 fp16 of a row of D: from d on, or, where the row ends within them, its
// last 8 (so every lane that has any moves 8 at a time, some a second time with the
// same result); of a row shorter than 8, those that there are, zeros for the rest.
__device__ __forceinline__ int first_of(int d, int D) { return max(min(d, D - 8), 0); }

__device__ __forceinline__ half8 load8(const uint16_t* p, int D)
{
    half8 v = {};
    if (D >= 8) __builtin_memcpy(&v, p, 16);
    else
        for (int i = 0; i < D; ++i) v[i] = __builtin_bit_cast(_Float16, p[i]);
    return v;
}

__device__ __forceinline__ void store8(uint16_t* p, half8 v, int D)
{
    if (D >= 8) __builtin_memcpy(p, &v, 16);
    else
        for (int i = 0; i < D; ++i) p[i] = __builtin_bit_cast(uint16_t, (_Float16)v[i]);
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
        if (d >= a.D) continue;
        const int f = first_of(d, a.D);
        const half8 v = load8(a.in + (size_t)t * a.D + f, a.D);
        for (int j = 0; j < a.k; ++j) {
            const int r = lane_value(at, j);
            if ((unsigned)r < (unsigned)a.R) store8(a.out + (size_t)r * a.D + f, v, a.D);
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
        if (d >= a.D) continue;
        const int f = first_of(d, a.D);
        float acc[8] = {};
        for (int j0 = 0; j0 < a.k; j0 += kTogether) {
            half8 v[kTogether];
            int r[kTogether];
#pragma unroll
            for (int u = 0; u < kTogether; ++u) {
                r[u] = lane_value(at, min(j0 + u, kMaxTop - 1));
                if ((unsigned)r[u] < (unsigned)a.R) v[u] = load8(a.in + (size_t)r[u] * a.D + f, a.D);
            }
#pragma unroll
            for (int u = 0; u < kTogether; ++u) {
                if ((unsigned)r[u] >= (unsigned)a.R) continue;
                const float wj = lane_value(w, min(j0 + u, kMaxTop - 1));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] = WEIGHTS ? __builtin_fmaf(wj, (float)v[u][i], acc[i]) : acc[i] + (float)v[u][i];
            }
        }
        half8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = (_Float16)acc[i];
        store8(a.out + (size_t)t * a.D + f, o, a.D);
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

// PER waves take a token and share the row's width; their parts of the dot products
// are added in wave order.
template <int PER>
__global__ __launch_bounds__(kWaves * kWave) void combine_grad_kernel(CombineGradArgs a)
{
    __shared__ float parts[kWaves][kMaxTop];
    constexpr int TOKENS = kWaves / PER;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int sub = wave % PER;
    for (int t0 = blockIdx.x * TOKENS; t0 < a.T; t0 += gridDim.x * TOKENS) {
        const int t = t0 + wave / PER;
        const size_t row = (size_t)t * a.k;
        const bool mine = t < a.T && lane < a.k;
        const int at = mine ? a.place[row + lane] : -1;
        const float w = mine ? a.weights[row + lane] : 0.0f;
        float dot = 0.0f;                        // lane j: this wave's part of choice j's
        for (int d0 = sub * kWave * 8; t < a.T && d0 < a.D; d0 += PER * kWave * 8) {
            const int d = d0 + lane * 8, f = first_of(d, a.D);
            const bool in = d < a.D;
            const half8 g = in ? load8(a.dY + (size_t)t * a.D + f, a.D) : half8{};
            for (int j0 = 0; j0 < a.k; j0 += kTogether) {
                half8 c[kTogether];
                int r[kTogether];
#pragma unroll
                for (int u = 0; u < kTogether; ++u) {
                    r[u] = lane_value(at, min(j0 + u, kMaxTop - 1));
                    if (j0 + u >= a.k || (unsigned)r[u] >= (unsigned)a.R) r[u] = -1;
                    c[u] = half8{};
                    if (r[u] >= 0 && in) c[u] = load8(a.C + (size_t)r[u] * a.D + f, a.D);
                }
#pragma unroll
                for (int u = 0; u < kTogether; ++u) {
                    if (r[u] < 0) continue;
                    const float wj = lane_value(w, j0 + u);
                    half8 o;
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[i] = (_Float16)(wj * (float)g[i]);
                        if (f + i >= d) s = __builtin_fmaf((float)g[i], (float)c[u][i], s);   // once where 8 overlap the 8 before
                    }
                    if (in) store8(a.dC + (size_t)r[u] * a.D + f, o, a.D);
                    s = wave_sum(s);
                    if (lane == j0 + u) dot += s;
                }
            }
        }
        if constexpr (PER > 1) {
            parts[wave][lane] = dot;
            __syncthreads();
            if (sub == 0)
#pragma unroll
                for (int v = 1; v < PER; ++v) dot += parts[wave + v][lane];
            __syncthreads();
        }
        if (sub == 0 && mine) a.dweights[row + lane] = dot;
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
    const auto launch = [&](auto per) {
        constexpr int PER = decltype(per)::value;
        const int groups = ceil_div(T, kWaves / PER);
        hipLaunchKernelGGL(combine_grad_kernel<PER>, dim3(groups < kGrid ? groups : kGrid), dim3(kWaves * kWave), 0,
                           (hipStream_t)stream, a);
        return status(hipGetLastError());
    };
    if (D <= 512) return launch(std::integral_constant<int, 1>{});
    if (D <= 1024) return launch(std::integral_constant<int, 2>{});
    return launch(std::integral_constant<int, 4>{});
}

}  // extern "C"
