// 4-bit weights with a scale and a zero point per group of consecutive k.
//
// Codes: word j of a row holds k = 8 j .. 8 j + 7, four bits each, lowest
// first; group g of row n (k = g * group ..) stands for (q - z) * s with
// s = S[n][g] (fp16) and z = Z[n][g] (a byte), or z = 8 without Z.
//
// A code q put in the low bits of an fp16 is the subnormal q * 2^-24, exactly.
// The matrix cores take subnormal operands at full speed and keep them (checked
// on the GPU, for both shapes used here), so unpacking needs no conversion: a
// shift and a mask give two codes per 32-bit register, a packed fp16 subtraction
// gives q - z (exact: small integers times 2^-24), and the products a * (q - z)
// are summed in fp32 within a group.  Each group's sum is then scaled by
// s * 2^24 in fp32, so that the only rounding to fewer bits is that of the
// output: weights are never rounded to fp16.
#pragma once
#include "common.hpp"
#include "grouped_kernel.hpp"

namespace gf {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// quantize and back
// ---------------------------------------------------------------------------

// Reduction over the LANES neighbouring lanes (4, 8 or 16) that share a group.
template <int LANES, class F>
__device__ __forceinline__ float group_reduce(float v, F f)
{
    v = f(v, __shfl_xor(v, 1));
    v = f(v, __shfl_xor(v, 2));
    if constexpr (LANES >= 8) v = f(v, __shfl_xor(v, 4));
    if constexpr (LANES >= 16) v = f(v, __shfl_xor(v, 8));
    return v;
}

// One thread holds 8 consecutive k (a word of codes), GROUP / 8 neighbouring
// lanes one group.  Rows are padded to whole groups in the thread index, so a
// group never straddles two rows; the lanes past K hold zeros, which change
// neither min(0, w), max(0, w) nor max |w|.
//
// The code is the quotient w / s rounded to nearest, ties to even, and has to
// be that of the exact quotient.  w * (1 / s) can fall on the wrong side of a
// tie, so one correction step follows: the residual w - t s is exact in fp32
// (w and s have 11 significant bits), and t + residual / s is the exact
// quotient wherever that is representable, as every tie is; the quotients that
// are not ties lie further from one than the rounding errors here.
template <int GROUP, bool VEC>
__global__ __launch_bounds__(256) void w4_quantize_kernel(const uint16_t* __restrict__ W,
                                                          uint32_t* __restrict__ Q,
                                                          uint16_t* __restrict__ S, uint8_t* __restrict__ Z,
                                                          int K, int G, int64_t items)
{
    constexpr int LANES = GROUP / 8;
    const int per_row = G * LANES;
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t base = (int64_t)blockIdx.x * 256; base < items; base += stride) {
        const int64_t idx = base + threadIdx.x;
        const bool live = idx < items;
        const int64_t row = live ? idx / per_row : 0;
        const int j = live ? (int)(idx - row * per_row) : 0;
        const bool some = live && j * 8 < K;
        uint16_t h[8] = {};
        if (some) {
            const uint16_t* p = W + row * K + (int64_t)j * 8;
            if constexpr (VEC) {
                const u32x4 v = __builtin_nontemporal_load((const u32x4*)p);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = p[i];
            }
        }
        float w[8], lo = 0.0f, hi = 0.0f, inf = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = f16_bits_to_f32(h[i]);
            if ((h[i] & 0x7c00) == 0x7c00) inf = 1.0f;    // an infinity or a NaN
            lo = fminf(lo, w[i]);
            hi = fmaxf(hi, w[i]);
        }
        auto mx = [](float a, float b) { return fmaxf(a, b); };
        auto mn = [](float a, float b) { return fminf(a, b); };
        hi = group_reduce<LANES>(hi, mx);
        lo = group_reduce<LANES>(lo, mn);
        inf = group_reduce<LANES>(inf, mx);
        // (a zero scale is +0, whatever the signs of the zeros it came from)
        const uint16_t sb = f32_to_f16_bits(fabsf(Z ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f));
        const float s = f16_bits_to_f32(sb);
        const bool flat = s == 0.0f || inf != 0.0f;       // all codes are z
        const float r = 1.0f / s;
        float z = 8.0f;
        if (Z) z = flat ? 0.0f : fminf(rintf(-lo / s), 15.0f);
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t0 = w[i] * r;
            const float t = fmaf(fmaf(-t0, s, w[i]), r, t0);
            const float q = flat ? z : fminf(fmaxf(rintf(t) + z, 0.0f), 15.0f);
            word |= (uint32_t)(int)q << (4 * i);
        }
        if (some) __builtin_nontemporal_store(word, Q + row * (K / 8) + j);
        if (live && j % LANES == 0) {
            const int64_t at = row * G + j / LANES;
            S[at] = inf != 0.0f ? (uint16_t)0x7e00 : sb;
            if (Z) Z[at] = (uint8_t)(int)z;
        }
    }
}

// One word of codes per thread.  (q - z) * s has at most 15 significant bits,
// so the fp32 product is exact and the store rounds once.
template <int GROUP, bool VEC>
__global__ __launch_bounds__(256) void w4_dequantize_kernel(const uint32_t* __restrict__ Q,
                                                            const uint16_t* __restrict__ S,
                                                            const uint8_t* __restrict__ Z,
                                                            uint16_t* __restrict__ W, int K, int G,
                                                            int64_t words)
{
    const int per_row = K / 8;
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x; idx < words; idx += stride) {
        const int64_t row = idx / per_row;
        const int j = (int)(idx - row * per_row);
        const uint32_t q = __builtin_nontemporal_load(Q + idx);
        const int64_t at = row * G + j / (GROUP / 8);
        const float s = f16_bits_to_f32(S[at]), z = Z ? (float)Z[at] : 8.0f;
        uint16_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = f32_to_f16_bits(((float)((q >> (4 * i)) & 15u) - z) * s);
        if constexpr (VEC) {
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
            __builtin_nontemporal_store(v, (u32x4*)W + idx);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) W[idx * 8 + i] = h[i];
        }
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

struct W4Args {
    const uint16_t* A;    // M x K (T x K when grouped)
    const uint32_t* Q;    // N x K / 8 (E x N x K / 8)
    const uint16_t* S;    // N x G
    const uint8_t* Z;     // N x G or null
    uint16_t* C;          // M x N
    int M, N, K, G;
    Groups g;             // grouped form: the rows of A and C by group; M unused
};

// Four codes pairs of a word: k = (0, 4), (1, 5), (2, 6), (3, 7) of its eight.
__device__ __forceinline__ half8 w4_unpack(uint32_t w, half2v z)
{
    constexpr uint32_t kMask = 0x000f000fu;
    const half2v a = __builtin_bit_cast(half2v, w & kMask) - z;
    const half2v b = __builtin_bit_cast(half2v, (w >> 4) & kMask) - z;
    const half2v c = __builtin_bit_cast(half2v, (w >> 8) & kMask) - z;
    const half2v d = __builtin_bit_cast(half2v, (w >> 12) & kMask) - z;
    return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight consecutive k of A in the order of w4_unpack.
__device__ __forceinline__ half8 w4_order(u32x4 v)
{
    const half8 h = __builtin_bit_cast(half8, v);
    return __builtin_shufflevector(h, h, 0, 4, 1, 5, 2, 6, 3, 7);
}

// Row-streaming product for few rows of A.  A workgroup owns 16 * NB rows of
// Q and up to 16 * MB rows of A; its waves split K into chunks of 128, each
// wave multiplying 16 x 16 x 32 MFMA steps, and their partial sums are added
// in wave order through LDS (a fixed order: results repeat bit for bit).
// A lane's 16-byte load of Q holds 32 consecutive k of one row.  An MFMA step
// sums over the four lanes of a row, and has to stay within one group: with
// groups of 128 the whole chunk is one group and step i takes word i of each
// lane; with shorter groups the four words of four lanes are exchanged first
// (two rounds of lane swaps), so that step i holds k = 32 i .. 32 i + 31.
// Out of range: rows of Q and A are clamped (the results are not stored), k
// past K multiplies a zeroed A.
template <int GROUP, int MB, int NB, int WAVES, bool QVEC, bool AVEC, bool GROUPED>
__global__ __launch_bounds__(WAVES * 64) void w4_stream_kernel(W4Args a)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int CK = 128;
    constexpr bool SWAP = QVEC && GROUP < 128;
    constexpr bool BY_LANE = QVEC && GROUP == 128;      // step i: word i of each lane
    extern __shared__ __attribute__((aligned(16))) char w4_smem[];
    GF_LDS float* red = (GF_LDS float*)w4_smem;

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, c4 = lane / 16;
    const int tiles_n = ceil_div(a.N, 16 * NB);
    int tm, tn, M = a.M;
    if constexpr (GROUPED) {
        int e, lo, hi, item;
        if (!a.g.template find<16 * MB>(blockIdx.x, tiles_n, e, lo, hi, item)) return;
        M = hi - lo;
        a.A += (size_t)lo * a.K;
        a.C += (size_t)lo * a.N;
        a.Q += (size_t)e * a.N * (a.K / 8);
        a.S += (size_t)e * a.N * a.G;
        if (a.Z) a.Z += (size_t)e * a.N * a.G;
        tm = item % ceil_div(M, 16 * MB);
        tn = item / ceil_div(M, 16 * MB);
    } else {
        tm = blockIdx.x / tiles_n;
        tn = blockIdx.x % tiles_n;
    }
    const int m0 = tm * 16 * MB, n0 = tn * 16 * NB;
    const int K = a.K, nch = ceil_div(K, CK);

    const uint32_t* qrow[NB];
    int srow[NB];
    const uint16_t* arow[MB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int n = min(n0 + 16 * b + r16, a.N - 1);
        qrow[b] = a.Q + (size_t)n * (K / 8);
        srow[b] = n * a.G;
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) arow[b] = a.A + (size_t)min(m0 + 16 * b + r16, M - 1) * K;

    struct Chunk {
        u32x4 q[NB], x[MB][4];
    };
    auto load = [&](int ch, Chunk& c) __attribute__((always_inline)) {
        const int k0 = ch * CK;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if constexpr (QVEC) {
                const int k = min(k0 + 32 * c4, K - 32);
                c.q[b] = __builtin_nontemporal_load((const u32x4*)(qrow[b] + k / 8));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) c.q[b][i] = qrow[b][min(k0 + 32 * i + 8 * c4, K - 8) / 8];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + (BY_LANE ? 32 * c4 + 8 * i : 32 * i + 8 * c4);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                u32x4 v = {0u, 0u, 0u, 0u};
                if (k < K) {
                    if constexpr (AVEC) {
                        v = *(const u32x4*)(arow[b] + k);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = arow[b][k + 2 * e] | ((uint32_t)arow[b][k + 2 * e + 1] << 16);
                    }
                }
                c.x[b][i] = v;
            }
        }
    };

    floatx4 acc[MB][NB] = {};
    constexpr int SPG = GROUP / 32;                     // MFMA steps per group
    auto compute = [&](int ch, Chunk& c) __attribute__((always_inline)) {
        half8 x[MB][4];
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[b][i] = w4_order(c.x[b][i]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            u32x4 q = c.q[nb];
            if constexpr (SWAP) {
                u32x2 p = __builtin_amdgcn_permlane32_swap(q[0], q[2], false, false);
                u32x2 r = __builtin_amdgcn_permlane32_swap(q[1], q[3], false, false);
                u32x2 s = __builtin_amdgcn_permlane16_swap(p[0], r[0], false, false);
                u32x2 t = __builtin_amdgcn_permlane16_swap(p[1], r[1], false, false);
                q = u32x4{s[0], s[1], t[0], t[1]};
            }
#pragma unroll
            for (int g0 = 0; g0 < 4 / SPG; ++g0) {
                const int g = ch * (CK / GROUP) + g0;
                const bool in = g < a.G;
                const int at = srow[nb] + (in ? g : a.G - 1);
                // past the last group: a scale of 0, not another group's (which may be infinite)
                const float s = in ? f16_bits_to_f32(a.S[at]) * 16777216.0f : 0.0f;
                const uint32_t zi = a.Z ? a.Z[at] : 8u;
                const half2v z = __builtin_bit_cast(half2v, zi * 0x00010001u);
                floatx4 part[MB] = {};
#pragma unroll
                for (int i = g0 * SPG; i < (g0 + 1) * SPG; ++i) {
                    const half8 w = w4_unpack(q[i], z);
#pragma unroll
                    for (int b = 0; b < MB; ++b)
                        part[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[b][i], w, part[b], 0, 0, 0);
                }
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[b][nb][i] = fmaf(part[b][i], s, acc[b][nb][i]);
            }
        }
    };

    if (wave < nch) {
        Chunk c0, c1;
        load(wave, c0);
        int ch = wave;
        for (; ch + WAVES < nch; ch += 2 * WAVES) {
            load(ch + WAVES, c1);
            compute(ch, c0);
            if (ch + 2 * WAVES < nch) load(ch + 2 * WAVES, c0);
            compute(ch + WAVES, c1);
        }
        if (ch < nch) compute(ch, c0);
    }

    // ---- the waves' sums, in wave order ----
    constexpr int PER_WAVE = MB * NB * 256;             // floats
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[wave * PER_WAVE + ((b * NB + nb) * 4 + i) * 64 + lane] = acc[b][nb][i];
    __syncthreads();
    for (int t = threadIdx.x; t < PER_WAVE; t += WAVES * 64) {
        const int n = t % (16 * NB), m = t / (16 * NB);            // within the tile
        const int at = (((m / 16) * NB + n / 16) * 4 + m % 4) * 64 + (m % 16) / 4 * 16 + n % 16;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += red[w * PER_WAVE + at];
        if (m0 + m < M && n0 + n < a.N) a.C[(size_t)(m0 + m) * a.N + n0 + n] = f32_to_f16_bits(s);
    }
#endif
}

}  // namespace gf
