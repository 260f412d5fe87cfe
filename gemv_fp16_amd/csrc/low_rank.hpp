// The second half of a low-rank adapter on the matrix cores: H . Up[a]^T for rows
// with different adapters.
//
// H (M x r, fp32: the scaled products by Down) comes as S parts of the contraction,
// added here in order.  The matrix cores take fp16, so each value goes in as two:
// its nearest fp16 and what that leaves, 22 bits together; a value past fp16's
// range becomes an infinity.  A block of rows costs one pass for each adapter that it
// has; where it has several, each one's sums are added to its own rows alone, so that
// an infinity or a NaN in one adapter stays in the rows that have it.
#pragma once
#include "common.hpp"

namespace gf {

struct LowRank {
    const float* H;          // S x M x r
    const int* ids;          // M
    const uint16_t* Up;      // L x N x r
    int64_t part;            // M * r
    int S, r, L;

    // Adapter of row m of M, -1 where there is none (past M: the last row's, so that
    // a block of one adapter stays one).
    __device__ __forceinline__ int adapter(int m, int M) const
    {
        const int id = ids[min(m, M - 1)];
        return (unsigned)id < (unsigned)L ? id : -1;
    }

    static __device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo)
    {
        hi = (_Float16)v;
        const float rest = v - (float)hi;
        lo = rest - rest == 0.0f ? (_Float16)rest : (_Float16)0.0f;   // none beside an infinity or a NaN
    }

    // k .. k + 7 of row m's H as pairs; k + 8 <= r.  SP: parts at most, their loads all
    // in flight together.
    template <int SP>
    __device__ __forceinline__ void pairs(int m, int k, half8& hi, half8& lo) const
    {
        floatx4 a[SP][2];
#pragma unroll
        for (int s = 0; s < SP; ++s) {
            a[s][0] = a[s][1] = floatx4{};
            if (s > 0 && s >= S) continue;
            const float* p = H + s * part + (size_t)m * r + k;
            a[s][0] = *(const floatx4*)p;
            a[s][1] = *(const floatx4*)(p + 4);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = a[0][i / 4][i % 4];
#pragma unroll
            for (int s = 1; s < SP; ++s) v += a[s][i / 4][i % 4];
            _Float16 h, rest;
            split(v, h, rest);
            hi[i] = h;
            lo[i] = rest;
        }
    }

    // The sums of MT rows row0 .. by FN x MT columns col0 .. (zeros for rows without an
    // adapter); r % 8 == 0, Up 16-byte aligned, S <= SP.  Where the rows have several
    // adapters, NA at a time, so that many have their loads in flight together.  All
    // lanes.
    template <class MF, int MT, int KS, int FN, int NA, int SP>
    __device__ __forceinline__ void block(typename MF::acc_t (&sum)[FN], int row0, int col0, int M, int N,
                                          int from = 0, int step = KS) const
    {
        const int lane = threadIdx.x % kWave, l = lane % MT, kq = lane / MT * 8;
        const int id = adapter(row0 + l, M), first = __builtin_amdgcn_readfirstlane(id);
        const uint64_t some = __ballot(id >= 0);
        const bool one = __ballot(id == first) == ~uint64_t(0);
#pragma unroll
        for (int g = 0; g < FN; ++g) sum[g] = typename MF::acc_t{};
        if (one && first >= 0) {
            const uint16_t* up = Up + (size_t)first * N * r;
            for (int k0 = from; k0 < r; k0 += step) {
                const int k = min(k0 + kq, r - 8);
                half8 hi, lo, u[FN];
#pragma unroll
                for (int g = 0; g < FN; ++g) u[g] = *(const half8*)(up + (size_t)min(col0 + g * MT + l, N - 1) * r + k);
                pairs<SP>(min(row0 + l, M - 1), k, hi, lo);
#pragma unroll
                for (int g = 0; g < FN; ++g) {
                    const half8 v = k0 + kq < r ? u[g] : half8{};
                    sum[g] = MF::run(hi, v, sum[g]);
                    sum[g] = MF::run(lo, v, sum[g]);
                }
            }
        } else if (!one) {
#pragma unroll
            for (int g = 0; g < FN; ++g)
                for (int k0 = from; k0 < r; k0 += step) {
                    const int k = min(k0 + kq, r - 8), col = min(col0 + g * MT + l, N - 1);
                    const bool in = k0 + kq < r;
                    half8 hi, lo;
                    pairs<SP>(min(row0 + l, M - 1), k, hi, lo);
                    uint64_t left = some;
                    while (left) {
                        int a[NA];                       // the next adapters of these rows
                        uint64_t rows[NA];               // none past the last
                        half8 u[NA];
#pragma unroll
                        for (int n = 0; n < NA; ++n) {
                            a[n] = left ? __builtin_amdgcn_readlane(id, __builtin_ctzll(left)) : a[0];
                            rows[n] = left & __ballot(id == a[n]);
                            left &= ~rows[n];
                            u[n] = *(const half8*)(Up + ((size_t)a[n] * N + col) * r + k);
                        }
#pragma unroll
                        for (int n = 0; n < NA; ++n) {
                            if (!rows[n]) break;
                            const half8 v = in ? u[n] : half8{};
                            typename MF::acc_t t = {};
                            t = MF::run(hi, v, t);
                            t = MF::run(lo, v, t);
#pragma unroll
                            for (int i = 0; i < MF::NACC; ++i)
                                sum[g][i] += ((uint32_t)rows[n] >> MF::row(i, lane)) & 1 ? t[i] : 0.0f;
                        }
                    }
                }
        }
    }
};

}  // namespace gf
