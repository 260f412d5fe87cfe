// Low-rank adapters: C[m] += scale[a] * (A[m] . Down[a]^T) . Up[a]^T, a = ids[m].
#pragma once
#include "wave.hpp"

namespace gf {

struct LoraArgs {
    const uint16_t* A;       // M x K
    const int* ids;          // M
    const uint16_t* Down;    // L x r x K
    const uint16_t* Up;      // L x N x r
    const float* scales;     // L, or null
    uint16_t* C;             // M x N
    float* H;                // M x r: the scaled products by Down
    int M, N, K, r, L;
};

// H[m][j] for one row m a workgroup; a wave takes every 4th j.
template <bool ALIGNED>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
        const int id = a.ids[m];
        if ((unsigned)id >= (unsigned)a.L) continue;
        const float scale = a.scales ? a.scales[id] : 1.0f;
        const uint16_t* x = a.A + (size_t)m * a.K;
        for (int j = wave; j < a.r; j += 4) {
            const uint16_t* w = a.Down + ((size_t)id * a.r + j) * a.K;
            float s = 0.0f;
            if constexpr (ALIGNED) {
                for (int k = lane * 8; k < a.K; k += kWave * 8) {
                    const half8 u = *(const half8*)(x + k), v = *(const half8*)(w + k);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s = __builtin_fmaf((float)u[i], (float)v[i], s);
                }
            } else {
                for (int k = lane; k < a.K; k += kWave) s = __builtin_fmaf(f16_bits_to_f32(x[k]), f16_bits_to_f32(w[k]), s);
            }
            s = wave_sum(s);
            if (lane == 0) a.H[(size_t)m * a.r + j] = scale * s;
        }
    }
}

// C[m][n] += H[m] . Up[a][n]: a thread an output.
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a)
{
    const int64_t total = (int64_t)a.M * a.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int m = (int)(i / a.N), n = (int)(i % a.N), id = a.ids[m];
        if ((unsigned)id >= (unsigned)a.L) continue;
        const float* h = a.H + (size_t)m * a.r;
        const uint16_t* u = a.Up + ((size_t)id * a.N + n) * a.r;
        float s = f16_bits_to_f32(a.C[i]);
        for (int j = 0; j < a.r; ++j) s = __builtin_fmaf(h[j], f16_bits_to_f32(u[j]), s);
        a.C[i] = f32_to_f16_bits(s);
    }
}

}  // namespace gf
