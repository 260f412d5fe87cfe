// The second half of a low-rank adapter on the matrix cores: H . Up[a]^T for rows
// with different adapters.
//
// H (M x r, fp32: the scaled products by Down) comes as S parts of the contraction,
// added here in order.  The matrix cores take fp16, so each value goes in as two, its
// nearest fp16 and what that leaves, after a power of two that brings the largest of
// the row's ranks in one step to 2^14 .. 2^15, and the step's sums are multiplied by its
// inverse: 22 bits of every value down to 2^-17 of the largest, 2^-39 of the largest
// below, whatever the size of H.  A block of rows costs one pass for each adapter that it
// has; where it has several, each one's sums are added to its own rows alone, so that
// an infinity or a NaN in one adapter stays in the rows that have it.  Infinities come out
// as the formula has them: an infinite value has no second half, a second half does not
// meet Up's infinities (0 times one would be a NaN), and ranks that are not there are 0 on
// both sides.
#pragma once
#include "wave.hpp"

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

    // u with numbers for infinities and NaN: what the second halves are multiplied by.
    static __device__ __forceinline__ half8 finite(half8 u)
    {
        const half8 most = (half8)(_Float16)65504.0f;
        return __builtin_elementwise_min(__builtin_elementwise_max(u, -most), most);
    }

    // The larger of m and |v|; an infinity or a NaN does not count.
    static __device__ __forceinline__ float larger(float m, float v)
    {
        const float f = __builtin_fabsf(v);
        return __builtin_fmaxf(m, f < __builtin_inff() ? f : 0.0f);
    }

    // Powers of two: `up` brings `most`, a finite magnitude, to 2^14 .. 2^15 (or less, from
    // below 2^-112), `down` is its inverse.
    struct Scale {
        float up, down;
        explicit __device__ __forceinline__ Scale(float most)
        {
            const int e = max(__builtin_bit_cast(int, most) >> 23, 15);
            up = __builtin_bit_cast(float, (268 - e) << 23);
            down = __builtin_bit_cast(float, (e - 14) << 23);
        }
    };

    // k .. k + 7 of row m's H as scaled pairs (0 where not `in`), and the scale's inverse;
    // k + 8 <= r.  SP: parts at most, their loads all in flight together.  The row's other
    // ranks of this step are in the lanes MT further.  All lanes.
    template <int MT, int SP>
    __device__ __forceinline__ float pairs(int m, int k, bool in, half8& hi, half8& lo) const
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
        float v[8], most = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = a[0][i / 4][i % 4];
#pragma unroll
            for (int s = 1; s < SP; ++s) v[i] += a[s][i / 4][i % 4];
            v[i] = in ? v[i] : 0.0f;
            most = larger(most, v[i]);
        }
        const Scale scale(rows_max<MT>(most));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            _Float16 h, rest;
            split(v[i] * scale.up, h, rest);
            hi[i] = h;
            lo[i] = rest;
        }
        return scale.down;
    }

    // The values v that the lanes l < MT hold for rows l, beside each row's accumulators: one
    // product with ones (2048 rows at 4096 x 4096, rank 64: 92.5 us; with 16 cross-lane
    // reads a block 95.6, and 89 without any scaling).
    template <class MF>
    static __device__ __forceinline__ typename MF::acc_t beside_rows(float v)
    {
        typename MF::acc_t f = {};
        if constexpr (MF::ROW_IN_LANE) {
            f += v;
        } else {
            static_assert(MF::NACC == 16, "blocks of 32 x 32");
            f = __builtin_amdgcn_mfma_f32_32x32x2f32(threadIdx.x % kWave < 32 ? v : 0.0f, 1.0f, f, 0, 0, 0);
        }
        return f;
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
                const bool in = k0 + kq < r;
                half8 hi, lo, u[FN];
#pragma unroll
                for (int g = 0; g < FN; ++g) u[g] = *(const half8*)(up + (size_t)min(col0 + g * MT + l, N - 1) * r + k);
                const float down = pairs<MT, SP>(min(row0 + l, M - 1), k, in, hi, lo);
                const typename MF::acc_t f = beside_rows<MF>(down);
#pragma unroll
                for (int g = 0; g < FN; ++g) {
                    const half8 v = in ? u[g] : half8{};
                    typename MF::acc_t t = {};
                    t = MF::run(hi, v, t);
                    t = MF::run(lo, finite(v), t);
#pragma unroll
                    for (int i = 0; i < MF::NACC; ++i) sum[g][i] += t[i] * f[i];
                }
            }
        } else if (!one) {
#pragma unroll
            for (int g = 0; g < FN; ++g)
                for (int k0 = from; k0 < r; k0 += step) {
                    const int k = min(k0 + kq, r - 8), col = min(col0 + g * MT + l, N - 1);
                    const bool in = k0 + kq < r;
                    half8 hi, lo;
                    const float down = pairs<MT, SP>(min(row0 + l, M - 1), k, in, hi, lo);
                    const typename MF::acc_t f = beside_rows<MF>(down);
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
                            t = MF::run(lo, finite(v), t);
#pragma unroll
                            for (int i = 0; i < MF::NACC; ++i)
                                sum[g][i] += ((uint32_t)rows[n] >> MF::row(i, lane)) & 1 ? t[i] * f[i] : 0.0f;
                        }
                    }
                }
        }
    }
};

}  // namespace gf
