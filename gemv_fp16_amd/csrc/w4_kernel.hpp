// 4-bit weights with a scale and a zero point per group of consecutive k.
//
// Codes: word j of a row holds k = 8 j .. 8 j + 7, four bits each, lowest
// first; group g of row n (k = g * group ..) stands for (q - z) * s with
// s = S[n][g] (fp16) and z = Z[n][g] (a byte), or z = 8 without Z.
//
// A code q put in the low bits of an fp16 is the subnormal q * 2^-24, exactly.
// The matrix cores take subnormal operands at full speed and keep them (checked
// on the GPU, for both shapes used here), so unpacking needs no conversion:
// masks and byte moves place two codes in a 32-bit register, one packed fp16
// operation gives q - z (exact: small integers times 2^-24), and the products
// a * (q - z) are summed in fp32 within a group.  Each group's sum is then scaled by
// s * 2^24 in fp32, so that the only rounding to fewer bits is that of the
// output.  That is how few rows of A are multiplied; the tiles for many rows round
// each weight to fp16 first (why, and what it buys, stands there).
#pragma once
#include "common.hpp"
#include "gemv_kernel.hpp"
#include "grouped_kernel.hpp"

namespace gf {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// quantize and back
// ---------------------------------------------------------------------------

// Rows are walked by whole workgroups, R rows at a time where they are short and
// in pieces of 256 threads where they are long, grid-stride over the rows: a
// thread's place in its row is found once, without a division per piece.
struct W4Walk {
    int per_row;          // threads a row takes (a multiple of a group's)
    int rows_at_once;     // R = max(1, 256 / per_row)
    int chunks;           // pieces of 256 threads that a row takes (1 if R > 1)
    int64_t rows;
};

// SHORT: several rows at once.  Otherwise the row is the same for the whole
// workgroup, and its addresses are scalars.
template <bool SHORT>
struct W4Place {
    int64_t row0;         // first row of the iteration
    int sub, j, c;        // this thread's row in it; word within the row; piece
    __device__ __forceinline__ W4Place(const W4Walk& w)
    {
        sub = SHORT ? (int)threadIdx.x / w.per_row : 0;
        j = (int)threadIdx.x - sub * w.per_row;
        c = 0;
        row0 = (int64_t)blockIdx.x * (SHORT ? w.rows_at_once : 1);
    }
    __device__ __forceinline__ int64_t row() const { return SHORT ? row0 + sub : row0; }
    __device__ __forceinline__ bool more(const W4Walk& w) const { return row0 < w.rows; }   // uniform
    __device__ __forceinline__ bool live(const W4Walk& w) const
    {
        if constexpr (SHORT) return sub < w.rows_at_once && row0 + sub < w.rows;
        else return row0 < w.rows && j < w.per_row;
    }
    __device__ __forceinline__ void next(const W4Walk& w)
    {
        if constexpr (SHORT) {
            row0 += (int64_t)gridDim.x * w.rows_at_once;
        } else if (++c < w.chunks) {
            j += 256;
        } else {
            j -= (w.chunks - 1) * 256;
            c = 0;
            row0 += gridDim.x;
        }
    }
};

// Maximum of both 16-bit halves over the LANES neighbouring lanes (4, 8 or 16)
// that share a group, in all of them, by lane permutes within a DPP row.
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
template <int CTRL>
__device__ __forceinline__ uint32_t w4_max_step(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, v),
                                                                  __builtin_bit_cast(ushort2v, o)));
}

template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    v = w4_max_step<0xB1>(v);                             // quad_perm [1,0,3,2]
    v = w4_max_step<0x4E>(v);                             // quad_perm [2,3,0,1]
    if constexpr (LANES >= 8) v = w4_max_step<0x141>(v);  // row_half_mirror
    if constexpr (LANES >= 16) v = w4_max_step<0x140>(v); // row_mirror
    return v;
}

// a / b with r = 1 / b to within a rounding: the first quotient's residual is
// exact, and the quotient it corrects is the nearest one (Markstein's method).
__device__ __forceinline__ float w4_quotient(float a, float b, float r)
{
    const float q = a * r;
    return fmaf(fmaf(-q, b, a), r, q);
}

// q = (hi - lo) / 15 in fp32, on the side of a tie between two fp16 scales where
// the exact quotient is.  hi - lo can need more than 24 bits; fp32 loses up to half
// a unit of its last place.  A tie t times 15 is a whole number of these units, so
// unless the rounded difference is 15 t itself, it is a unit away from it at least:
// then exact and rounded difference lie on the same side of 15 t, and the fp32
// quotient, which a 15th of a unit is enough to move, on that side of t.  If it is
// 15 t, q is t, and what the difference lost decides: q moves one fp32 step that
// way.  (Ties have 12 significant bits.  The other numbers that end in 12 zeros are
// fp16 numbers, and round to themselves from a step beside.)
__device__ __forceinline__ float w4_beside_tie(float q, float lost)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, q);
    const uint32_t beside = lost > 0.0f ? b + 1u : b - 1u;
    return __builtin_bit_cast(float, lost != 0.0f && (b & 0xfffu) == 0u ? beside : b);
}

// One thread holds 8 consecutive k (a word of codes), GROUP / 8 neighbouring
// lanes one group.  Rows are padded to whole groups in the thread index, so a
// group never straddles two rows; the lanes past K hold zeros, which change
// neither min(0, w), max(0, w) nor max |w|.
//
// The code is the quotient w / s rounded to nearest, ties to even, and has to
// be that of the exact quotient.  w * (1 / s) can fall on the wrong side of a
// tie, hence the correction: its residual is exact (w and s have 11 significant
// bits), so it gives the exact quotient wherever that is representable, as every
// tie is; the quotients that are not ties lie further from one than fp32 rounds.
// Bound by HBM and the vector ALU alike (2 bytes read and half a byte written
// for about 10 instructions), so the codes are put together as exact fp32
// integers, six to a sum, and the zero point is added to all eight at once.
// 8192 x 8192 in groups of 128 with zero points: 41 us, 4.1 TB/s, the vector ALU
// busy for 74 % of it.
template <int GROUP, bool ASYM, bool VEC, bool SHORT>
__global__ __launch_bounds__(256) void w4_quantize_kernel(const uint16_t* __restrict__ W,
                                                          uint32_t* __restrict__ Q,
                                                          uint16_t* __restrict__ S, uint8_t* __restrict__ Z,
                                                          int K, int G, W4Walk walk)
{
    constexpr int LANES = GROUP / 8;
    typedef W4Place<SHORT> Place;
    auto load = [&](const Place& p) __attribute__((always_inline)) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (p.live(walk) && p.j * 8 < K) {
            const uint16_t* src = W + p.row() * K + p.j * 8;
            if constexpr (VEC) {
                v = __builtin_nontemporal_load((const u32x4*)src);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i / 2] |= (uint32_t)src[i] << (16 * (i % 2));
            }
        }
        return v;
    };
    Place at(walk), ahead(walk);
    u32x4 v = load(at);
    for (; at.more(walk); at = ahead) {                   // the next piece is in flight while one is worked on
        ahead.next(walk);
        const u32x4 following = load(ahead);
        const bool live = at.live(walk), some = live && at.j * 8 < K;
        const int64_t row = at.row();
        const int j = at.j;
        const half8 h = __builtin_bit_cast(half8, v);
        // An infinity or a NaN has all exponent bits set: one more carries into
        // the sign's place.
        uint32_t carry = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) carry |= (v[i] & 0x7c007c00u) + 0x04000400u;
        bool bad = (carry & 0x80008000u) != 0;
        if (__ballot(bad)) bad = group_max<LANES>(bad ? 1u : 0u) != 0;   // rare, and then for the whole wave
        // max(0, w) and max(0, -w) side by side: as 16-bit patterns both are
        // non-negative numbers, which order like whole ones
        const half2v h0 = {h[0], h[1]}, h1 = {h[2], h[3]}, h2 = {h[4], h[5]}, h3 = {h[6], h[7]};
        const half2v top = __builtin_elementwise_max(__builtin_elementwise_max(h0, h1), __builtin_elementwise_max(h2, h3));
        const half2v low = __builtin_elementwise_min(__builtin_elementwise_min(h0, h1), __builtin_elementwise_min(h2, h3));
        const uint32_t t = __builtin_bit_cast(uint32_t, top), n = __builtin_bit_cast(uint32_t, low) ^ 0x80008000u;
        const half2v zero = {(_Float16)0.0f, (_Float16)0.0f};
        const half2v side = __builtin_elementwise_max(
            __builtin_elementwise_max(__builtin_bit_cast(half2v, __builtin_amdgcn_perm(n, t, 0x05040100u)),
                                      __builtin_bit_cast(half2v, __builtin_amdgcn_perm(n, t, 0x07060302u))), zero);
        const uint32_t both = group_max<LANES>(__builtin_bit_cast(uint32_t, side) & 0x7fff7fffu);
        const float hi = f16_bits_to_f32((uint16_t)both), lo = -f16_bits_to_f32((uint16_t)(both >> 16));
        // (a zero scale is +0, whatever the signs of the zeros it came from)
        const float span = ASYM ? hi - lo : __builtin_fmaxf(hi, -lo);
        float quot = w4_quotient(span, ASYM ? 15.0f : 7.0f, ASYM ? 1.0f / 15.0f : 1.0f / 7.0f);
        if constexpr (ASYM) {
            const float big = __builtin_fmaxf(hi, -lo), small = __builtin_fminf(hi, -lo);
            const float lost = small - (span - big);      // hi - lo is span + lost, exactly
            if (__ballot(lost != 0.0f)) quot = w4_beside_tie(quot, lost);   // rare
        }
        const uint16_t sb = f32_to_f16_bits(quot);
        const float s = f16_bits_to_f32(sb);
        const bool flat = s == 0.0f || bad;               // all codes are z
        const float r0 = __builtin_amdgcn_rcpf(flat ? 1.0f : s), r = fmaf(fmaf(-s, r0, 1.0f), r0, r0);
        const float z = !ASYM ? 8.0f : flat ? 0.0f : fminf(rintf(w4_quotient(-lo, s, r)), 15.0f);
        const float least = -z, most = 15.0f - z;
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)                       // the bounds are whole: clamping first is the same
            c[i] = rintf(__builtin_amdgcn_fmed3f(w4_quotient((float)h[i], s, r), least, most));
        // c0 + 16 c1 + .. + 16^5 c5, exact below 2^24
        const float six = fmaf(fmaf(fmaf(fmaf(fmaf(c[5], 16.0f, c[4]), 16.0f, c[3]), 16.0f, c[2]), 16.0f, c[1]), 16.0f, c[0]);
        const float two = fmaf(c[7], 16.0f, c[6]);
        const uint32_t codes = flat ? 0u : (uint32_t)(int)six + ((uint32_t)(int)two << 24);
        if (some) __builtin_nontemporal_store(codes + (uint32_t)(int)z * 0x11111111u, Q + row * (K / 8) + j);
        if (live && j % LANES == 0) {
            const int64_t g = row * G + j / LANES;
            S[g] = bad ? (uint16_t)0x7e00 : sb;
            if (ASYM) Z[g] = (uint8_t)(int)z;
        }
        v = following;
    }
}

// The eight weights (q - z) * s of a word as fp16, in order.  A byte holds an
// even k's code in its low half and the next one's in its high half; with the
// exponent of 1024 put over them they are 1024 + q and 1024 + 16 q, and one
// fused multiply-add brings both to q - z, exactly; the product with s rounds.
// off: w4_offsets(z).
__device__ __forceinline__ half8 w4_weights(uint32_t w, half2v off, half2v s)
{
    const half2v f = {(_Float16)1.0f, (_Float16)0.0625f};
    half2v p[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t u = __builtin_amdgcn_perm(0u, w, 0x0c000c00u + 0x00010001u * (uint32_t)b);
        p[b] = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (u & 0x00f0000fu) | 0x64006400u), f, off) * s;
    }
    return half8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// -1024 - z and -64 - z: steps of 1 and of 1/16 from the bits of -1024 and -64.
__device__ __forceinline__ half2v w4_offsets(uint32_t z)
{
    return __builtin_bit_cast(half2v, 0xd400e400u + (z & 0xffu) * 0x00100001u);
}

__device__ __forceinline__ half2v w4_twice(uint32_t bits)
{
    return __builtin_bit_cast(half2v, (bits & 0xffffu) * 0x00010001u);
}

// One word of codes per thread; bound by HBM's mix of reads and writes.  8192 x 8192
// in groups of 128: 41 us, 4.2 TB/s (a plain copy of this size: 5.1).
template <int GROUP, bool VEC, bool SHORT>
__global__ __launch_bounds__(256) void w4_dequantize_kernel(const uint32_t* __restrict__ Q,
                                                            const uint16_t* __restrict__ S,
                                                            const uint8_t* __restrict__ Z,
                                                            uint16_t* __restrict__ W, int K, int G, W4Walk walk)
{
    typedef W4Place<SHORT> Place;
    struct Word {
        uint32_t q, s, z;
    };
    auto load = [&](const Place& p) __attribute__((always_inline)) {
        Word w = {0u, 0u, 8u};
        if (p.live(walk) && p.j * 8 < K) {
            w.q = __builtin_nontemporal_load(Q + p.row() * (K / 8) + p.j);
            const uint32_t g = (uint32_t)p.j / (GROUP / 8);
            w.s = *(S + p.row() * G + g);
            if (Z) w.z = *(Z + p.row() * G + g);
        }
        return w;
    };
    Place at(walk), ahead(walk);
    Word w0 = load(at);
    ahead.next(walk);
    Word w1 = load(ahead);
    for (; at.more(walk); at.next(walk)) {                // two more words in flight
        ahead.next(walk);
        const Word w2 = load(ahead), w = w0;
        w0 = w1;
        w1 = w2;
        if (!at.live(walk) || at.j * 8 >= K) continue;
        const half8 h = w4_weights(w.q, w4_offsets(w.z), w4_twice(w.s));
        uint16_t* p = W + at.row() * K + at.j * 8;
        // (taken apart as words: a bit cast of one element of h was seen to yield
        // the first one for all eight)
        const u32x4 v = __builtin_bit_cast(u32x4, h);
        if constexpr (VEC) {
            __builtin_nontemporal_store(v, (u32x4*)p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
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
    int f32;              // one weight: whether C is fp32 (its sums before they are rounded)
    Groups g;             // grouped form: the rows of A and C by group, M unused; else only `first`
};

// Entry i of C.
template <bool GROUPED>
__device__ __forceinline__ void w4_store(const W4Args& a, size_t i, float v)
{
    if (!GROUPED && a.f32) ((float*)a.C)[i] = v;
    else a.C[i] = f32_to_f16_bits(v);
}

// The eight q - z of a word, in order, as fp16 subnormals (times 2^-24).  A byte
// holds an even k's code in its low half and the next one's in its high half,
// 16 times too large once masked; the fused multiply-add that subtracts the
// zero point takes that factor out, exactly.  10 instructions for 8 codes (a
// shift and a mask for each pair take 11 and leave k in the order 0, 4, 1, 5,
// .., which A then has to be brought into).  nz: -z in both halves.
__device__ __forceinline__ half8 w4_unpack(uint32_t w, half2v nz)
{
    const uint32_t lo = w & 0x0f0f0f0fu, hi = w & 0xf0f0f0f0u;
    const half2v f = {(_Float16)1.0f, (_Float16)0.0625f};
    half2v p[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint32_t u = __builtin_amdgcn_perm(hi, lo, 0x0c040c00u + 0x00010001u * (uint32_t)b);
        p[b] = __builtin_elementwise_fma(__builtin_bit_cast(half2v, u), f, nz);
    }
    return half8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// -z (a byte) as the subnormal pair that w4_unpack adds.
__device__ __forceinline__ half2v w4_minus(uint32_t z)
{
    return __builtin_bit_cast(half2v, z * 0x00010001u | 0x80008000u);
}

// Word i of the lane with c4 = j to word j of the lane with c4 = i, among the four
// lanes c4 * 16 + r of each r.
__device__ __forceinline__ u32x4 w4_exchange(u32x4 q)
{
    const u32x2 p = __builtin_amdgcn_permlane32_swap(q[0], q[2], false, false);
    const u32x2 r = __builtin_amdgcn_permlane32_swap(q[1], q[3], false, false);
    const u32x2 s = __builtin_amdgcn_permlane16_swap(p[0], r[0], false, false);
    const u32x2 t = __builtin_amdgcn_permlane16_swap(p[1], r[1], false, false);
    return u32x4{s[0], s[1], t[0], t[1]};
}

constexpr float kW4Unit = 16777216.0f;   // 2^24: one code step, as a subnormal, is its reciprocal

// Loads of wider words than their addresses are aligned to (the hardware takes
// any alignment; the compiler has to be told).
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

// N consecutive 32-bit words (N = 1, 2, 4 or 8), or a 16-bit one for N = 0.
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t* v)
{
    if constexpr (N == 0) {
        v[0] = *(const u16_any*)p;
    } else if constexpr (N == 1) {
        v[0] = *(const u32_any*)p;
    } else if constexpr (N == 2) {
        const u32x2 t = *(const u32x2_any*)p;
        v[0] = t[0]; v[1] = t[1];
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) load_words<2>((const u32x2_any*)p + i, v + 2 * i);
    }
}

// The general product for few rows of A: any K (a multiple of 8), N and
// alignment.  A workgroup owns 16 * NB rows of Q and up to 16 * MB rows of A; its
// waves split K, each multiplying 16 x 16 x 32 MFMA steps, and their partial sums
// are added in wave order through LDS (a fixed order: results repeat bit for bit).
// What bounds it is not only the bytes: each row that a load touches is a cache
// line of its own, and a line costs its cycle whether 2 or 64 bytes of it are
// used.  So the waves take K in blocks of CB chunks of 128 (block b goes to wave
// b % WAVES), and load a block's scales and zero points with few instructions;
// the next block is in flight while one is multiplied, and the next chunk of A.
// A lane's 16-byte load of Q holds 32 consecutive k of one row.  An MFMA step
// sums over the four lanes of a row, and has to stay within one group: with
// groups of 128 the whole chunk is one group and step i takes word i of each
// lane; with shorter groups the four words of four lanes are exchanged first
// (two rounds of lane swaps), so that step i holds k = 32 i .. 32 i + 31.
// What is left of K behind the last block goes chunk by chunk, word by word.
// Out of range: rows of Q and A are clamped (the results are not stored), k
// past K multiplies a zeroed A.
// 3 x 10623 x 8632 in groups of 128: 25 us, 1.9 TB/s; the band form below takes 15
// for 3 x 10624 x 8192.
template <int GROUP_, int MB_, int NB_, int WAVES_, int CB_>
struct W4RowsCfg {
    static constexpr int GROUP = GROUP_, MB = MB_, NB = NB_, WAVES = WAVES_, CB = CB_;
    static constexpr int BK = 128 * CB;                  // k per block
    static constexpr int SW = BK / GROUP / 2;            // registers of a block's scales
    static constexpr int ZW = (BK / GROUP + 3) / 4;      // and zero points
    static constexpr int LDS_BYTES = WAVES * MB * NB * 256 * 4;
};

template <class Cfg, bool GROUPED>
__global__ __launch_bounds__(Cfg::WAVES * 64) void w4_rows_kernel(W4Args a)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int GROUP = Cfg::GROUP, MB = Cfg::MB, NB = Cfg::NB, WAVES = Cfg::WAVES, CB = Cfg::CB;
    constexpr int GPB = Cfg::BK / GROUP;                 // groups per block
    extern __shared__ __attribute__((aligned(16))) char w4_smem[];
    GF_LDS float* red = (GF_LDS float*)w4_smem;

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, c4 = lane / 16;
    const int tiles_n = ceil_div(a.N, 16 * NB);
    int tm, tn, M = a.M;
    if constexpr (GROUPED) {
        int e, lo, hi, item;
        if (!a.g.template find<16 * MB>(a.g.workgroup(), tiles_n, e, lo, hi, item)) return;
        M = hi - lo;
        a.A += (size_t)lo * a.K;
        a.C += (size_t)lo * a.N;
        a.Q += (size_t)e * a.N * (a.K / 8);
        a.S += (size_t)e * a.N * a.G;
        if (a.Z) a.Z += (size_t)e * a.N * a.G;
        tm = item % ceil_div(M, 16 * MB);
        tn = item / ceil_div(M, 16 * MB);
    } else {
        const unsigned w = a.g.workgroup();
        tm = w / tiles_n;
        tn = w % tiles_n;
    }
    const int m0 = tm * 16 * MB, n0 = tn * 16 * NB;
    const int K = a.K, nblk = K / Cfg::BK, rest = ceil_div(K - nblk * Cfg::BK, 128);

    const uint32_t* qrow[NB];
    int srow[NB];
    const uint8_t* zsrc = a.Z ? a.Z : (const uint8_t*)a.S;   // without zero points: some bytes to load
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int n = min(n0 + 16 * b + r16, a.N - 1);
        qrow[b] = a.Q + (size_t)n * (K / 8);
        srow[b] = n * a.G;
    }
    struct Block {
        u32x4 q[CB][NB];
        uint32_t s[NB][Cfg::SW], z[NB][Cfg::ZW];
    };
    auto load = [&](int blk, Block& v) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int b = 0; b < NB; ++b) v.q[c][b] = *(const u32x4_any*)(qrow[b] + (blk * CB + c) * 16 + c4 * 4);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            load_words<Cfg::SW>(a.S + srow[b] + blk * GPB, v.s[b]);
            load_words<GPB / 4>(zsrc + srow[b] + blk * GPB, v.z[b]);
        }
    };

    // A: chunk ch's four fragments (step i: word i of each lane's 32 k with
    // groups of 128, else k = 32 i .. 32 i + 31)
    const int koff = GROUP == 128 ? 32 * c4 : 8 * c4;
    constexpr int kstep = GROUP == 128 ? 8 : 32;
    const uint16_t* arow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) arow[b] = a.A + (size_t)min(m0 + 16 * b + r16, M - 1) * K;
    half8 x[MB][4];
    auto load_x = [&](int ch, half8 (&v)[MB][4]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < MB; ++b)
                v[b][i] = __builtin_bit_cast(half8, (u32x4)*(const u32x4_any*)(arow[b] + koff + ch * 128 + kstep * i));
    };

    floatx4 acc[MB][NB] = {};
    constexpr int SPG = GROUP / 32, GPC = 128 / GROUP;   // MFMA steps per group, groups per chunk
    // One group of one column block: steps g0 * SPG .. of a chunk.
    auto group = [&](int nb, int g0, const u32x4& q, float s, half2v nz) __attribute__((always_inline)) {
        floatx4 part[MB] = {};
#pragma unroll
        for (int i = g0 * SPG; i < (g0 + 1) * SPG; ++i) {
            const half8 w = w4_unpack(q[i], nz);
#pragma unroll
            for (int b = 0; b < MB; ++b) part[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[b][i], w, part[b], 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][nb][i] = fmaf(part[b][i], s, acc[b][nb][i]);
    };
    auto multiply = [&](const Block& v, auto c_c) __attribute__((always_inline)) {
        constexpr int c = decltype(c_c)::value;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            u32x4 q = v.q[c][nb];
            if constexpr (GROUP < 128) q = w4_exchange(q);
#pragma unroll
            for (int g0 = 0; g0 < GPC; ++g0) {
                const int g = c * GPC + g0;              // within the block
                const uint16_t sb = (uint16_t)(v.s[nb][g / 2] >> (16 * (g % 2)));
                const half2v nz = w4_minus(a.Z ? (v.z[nb][g / 4] >> (8 * (g % 4))) & 0xffu : 8u);
                group(nb, g0, q, f16_bits_to_f32(sb) * kW4Unit, nz);
            }
            if constexpr (MB > 1) __builtin_amdgcn_sched_barrier(0);   // unpacked operands of one block at a time
        }
    };

    // Blocks are loaded for a clamped number past the wave's last one, so that
    // no load stands under a branch.
    auto block = [&](int blk, const Block& v, int last) __attribute__((always_inline)) {
        static_for<CB>([&](auto c_c) __attribute__((always_inline)) {
            constexpr int c = decltype(c_c)::value;
            half8 next[MB][4];
            load_x(c + 1 < CB ? blk * CB + c + 1 : min(blk + WAVES, last) * CB, next);
            multiply(v, c_c);
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[b][i] = next[b][i];
        });
    };
    if (wave < nblk) {
        const int last = nblk - 1;
        Block v0, v1;
        load(wave, v0);
        load_x(wave * CB, x);
        int blk = wave;
        for (; blk + WAVES <= last; blk += 2 * WAVES) {
            load(blk + WAVES, v1);
            block(blk, v0, last);
            load(min(blk + 2 * WAVES, last), v0);
            block(blk + WAVES, v1, last);
        }
        if (blk <= last) block(blk, v0, last);
    }
    // ---- the chunks behind the last block ----
    for (int i = 0; i < rest; ++i) {
        if ((nblk + i) % WAVES != wave) continue;
        const int ch = nblk * CB + i, k0 = ch * 128 + 8 * c4;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = k0 + 32 * s;
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                u32x4 v = *(const u32x4_any*)(arow[b] + min(k, K - 8));
                x[b][s] = __builtin_bit_cast(half8, k < K ? v : u32x4{0u, 0u, 0u, 0u});
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            u32x4 q;
#pragma unroll
            for (int s = 0; s < 4; ++s) q[s] = qrow[nb][min(k0 + 32 * s, K - 8) / 8];
#pragma unroll
            for (int g0 = 0; g0 < GPC; ++g0) {
                const int g = ch * GPC + g0, at = srow[nb] + min(g, a.G - 1);
                // past the last group: a scale of 0, not another's (which may be infinite)
                const float s = g < a.G ? f16_bits_to_f32(a.S[at]) * kW4Unit : 0.0f;
                group(nb, g0, q, s, w4_minus(a.Z ? a.Z[at] : 8u));
            }
        }
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
    const int rows = min(16 * MB, M - m0);              // no thread for rows past M
    for (int t = threadIdx.x; t < rows * 16 * NB; t += WAVES * 64) {
        const int n = t % (16 * NB), m = t / (16 * NB);            // within the tile
        const int at = (((m / 16) * NB + n / 16) * 4 + m % 4) * 64 + (m % 16) / 4 * 16 + n % 16;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += red[w * PER_WAVE + at];
        if (n0 + n < a.N) w4_store<GROUPED>(a, (size_t)(m0 + m) * a.N + n0 + n, s);
    }
#endif
}

// The same product through LDS: K % 512 == 0, N >= 16 and the alignments above.
// Streaming wants whole cache lines: 33.5 MB of codes read as 16 rows x 64 bytes
// an instruction take 8.7 us, as whole lines (4 rows x 256 bytes) 6.2 us.  MFMA
// operands want the former.  So codes, scales and zero points go to LDS by
// direct loads that read lines, and each wave reads its operands from there: no
// registers are spent on loads in flight, and no wave waits for another's.
// The waves split K; a wave's tasks are its blocks of 512 k of one row group
// after the other (row groups of 16, walked grid-stride), `ring` tasks in flight.
// The last group takes the last 16 rows, some of them a second time, so that no
// address needs a bound.
// A task's buffer: 16 rows of 16 chunks of 16 bytes, chunk c of row n at slot
// c ^ n (so that the 16 rows read together lie in different banks), then the
// scales and zero points as 32-bit words, word j of row n at 16 j + n.
// Each row group ends in one barrier; the sums' slots alternate.
// XB == 0: A is copied to LDS once (chunk c of row m at slot c ^ m % 8);
// otherwise each wave keeps its part of 16 * MB rows of A in registers, XB blocks'
// worth, read through the tasks' buffers in whole lines as well (operands loaded
// from A straight: 18.0 us against 12.8 at 32 x 11008 x 4096, 14.7 against 8.7 at
// 16 x 4096 x 8192).  More rows are further passes, by workgroups of their own;
// grouped, an expert with many rows has many.
// What is left is the vector ALU's work, so it is kept short: a task's addresses
// are one scalar offset, a scale multiplies straight from its half of a word
// (acc is in units of 2^-24 until the end), and a word unpacks in 10
// instructions, or 9 where A's registers hold k in the order 0, 4, 1, 5, ...
template <int GROUP_, int MB_, int XB_>
struct W4BandCfg {
    static constexpr int GROUP = GROUP_, MB = MB_, XB = XB_, WAVES = 8, BK = 512;
    static constexpr bool XLDS = XB == 0;
    static constexpr int SWORDS = BK / GROUP / 2, ZWORDS = BK / GROUP / 4;   // per row
    // direct loads of a task: 4 of codes, then scales and zero points, which
    // share one instruction where 16 rows of both fit its 64 lanes
    static constexpr int SLOADS = GROUP == 128 ? 1 : SWORDS / 4, ZLOADS = GROUP == 128 ? 0 : 1;
    static constexpr int LOADS = 4 + SLOADS + ZLOADS;
    static constexpr int TASK_BYTES = 4096 + (SLOADS + ZLOADS) * 256;
    static constexpr int MAX_RING = 4;
};

// w4_unpack's values in the order 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ half8 w4_unpack_pairs(uint32_t w, half2v nz)
{
    constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;
    const half2v f = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t v = w >> 8;
    const half2v p0 = __builtin_bit_cast(half2v, w & kLo) + nz;
    const half2v p1 = __builtin_elementwise_fma(__builtin_bit_cast(half2v, w & kHi), f, nz);
    const half2v p2 = __builtin_bit_cast(half2v, v & kLo) + nz;
    const half2v p3 = __builtin_elementwise_fma(__builtin_bit_cast(half2v, v & kHi), f, nz);
    return half8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

template <class Cfg, bool GROUPED>
__global__ __launch_bounds__(Cfg::WAVES * 64) void w4_band_kernel(W4Args a, int ring, int parts)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int GROUP = Cfg::GROUP, MB = Cfg::MB, WAVES = Cfg::WAVES, L = Cfg::LOADS;
    constexpr int GPB = Cfg::BK / GROUP;                  // groups per block
    extern __shared__ __attribute__((aligned(1024))) char w4_smem[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, c4 = lane / 16;
    const int N = a.N, K = a.K, G = a.G;

    int part = a.g.workgroup(), M = a.M;
    if constexpr (GROUPED) {
        int e, lo, hi, item;
        if (!a.g.template find<16 * MB>(part, parts, e, lo, hi, item)) return;
        const int passes = ceil_div(hi - lo, 16 * MB);
        part = item / passes;
        const int first = lo + item % passes * 16 * MB;
        M = min(hi - first, 16 * MB);
        a.A += (size_t)first * K;
        a.C += (size_t)first * N;
        a.Q += (size_t)e * N * (K / 8);
        a.S += (size_t)e * N * G;
        if (a.Z) a.Z += (size_t)e * N * G;
    } else if constexpr (!Cfg::XLDS) {
        // passes over the same rows of Q on one XCD, at the same time
        const int passes = ceil_div(M, 16 * MB), x = part / 8;
        part = x / passes * 8 + part % 8;
        if (part >= parts) return;
        const int first = x % passes * 16 * MB;
        M = min(M - first, 16 * MB);
        a.A += (size_t)first * K;
        a.C += ((size_t)first * N) << a.f32;
    }
    const int red_rows = GROUPED ? 16 * MB : min(a.M, 16 * MB);
    GF_LDS char* tasks = (GF_LDS char*)w4_smem + wave * ring * Cfg::TASK_BYTES;
    GF_LDS float* red = (GF_LDS float*)((GF_LDS char*)w4_smem + WAVES * ring * Cfg::TASK_BYTES);
    GF_LDS char* xs = (GF_LDS char*)(red + 2 * WAVES * red_rows * 16);

    const int nblk = K / Cfg::BK;
    const int b0 = wave * nblk / WAVES, nb = (wave + 1) * nblk / WAVES - b0;   // this wave's blocks
    const int groups = ceil_div(N, 16);
    const int ng = (groups - part + parts - 1) / parts;   // row groups of this workgroup

    // ---- per-lane offsets of a task's direct loads, and its operands in LDS ----
    uint32_t qoff[4], qat[4], xat[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + c4;
        qoff[i] = (uint32_t)r * (uint32_t)(K / 2) + (uint32_t)(r16 ^ r) * 16u;
        qat[i] = (uint32_t)(r16 * 256 + (((4 * i + c4) ^ r16) * 16));
    }
    const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
        (void*)a.Q, 0, (int)((uint32_t)N * (uint32_t)(K / 2)), 0x00020000);
    // scales and zero points: this lane's word in each load, at group 0 of row group 0
    const uint8_t* zsrc = a.Z ? a.Z : (const uint8_t*)a.S;
    const char* szp[Cfg::SLOADS + Cfg::ZLOADS];
    int szshift[Cfg::SLOADS + Cfg::ZLOADS];
#pragma unroll
    for (int i = 0; i < Cfg::SLOADS + Cfg::ZLOADS; ++i) {
        const bool scales = GROUP == 128 ? c4 < 2 : i < Cfg::SLOADS;
        szshift[i] = scales ? 1 : 0;
        const int zword = GROUP == 128 ? 0 : min(c4, Cfg::ZWORDS - 1);
        szp[i] = scales ? (const char*)(a.S + (size_t)r16 * G + 8 * i + 2 * c4)
                        : (const char*)(zsrc + (size_t)r16 * G + 4 * zword);
    }

    // ---- A ----
    // Step i of a chunk of 128 k holds word i of each lane's 32 k with groups of
    // 128, else k = 32 i .. 32 i + 31.
    constexpr int xstep = GROUP == 128 ? 1 : 4;
    const int xchunk = GROUP == 128 ? 4 * c4 : c4;
    const int xm = min(r16, M - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        xat[i] = (uint32_t)(xm * K * 2 + ((xchunk + xstep * i) ^ (xm & 7)) * 16 + b0 * (Cfg::BK * 2));
    if constexpr (Cfg::XLDS) {
        const int per = K / 8, n = M * per;               // 16-byte chunks
        for (int t0 = wave * kWave; t0 < n; t0 += WAVES * kWave) {
            const int t = min(t0 + lane, n - 1), m = t / per, j = t - m * per;
            __builtin_amdgcn_global_load_lds((const void*)(a.A + (size_t)m * K + (j ^ (m & 7)) * 8),
                                             (GF_LDS void*)(xs + t0 * 16), 16, 0, 0);
        }
    }

    // ---- direct loads of a task ----
    const int ntasks = ng * nb;
    int ig = part, ib = 0, islot = 0, issued = 0;     // the next task to issue
    auto issue = [&]() __attribute__((always_inline)) {
        GF_LDS char* buf = tasks + islot * Cfg::TASK_BYTES;
        const int n0 = min(ig * 16, N - 16);
        const uint32_t so = (uint32_t)__builtin_amdgcn_readfirstlane(n0 * (K / 2) + (b0 + ib) * (Cfg::BK / 2));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (GF_LDS void*)(buf + i * 1024), 16, qoff[i], so, 0, 2);
        const size_t at = (size_t)n0 * G + (b0 + ib) * GPB;
#pragma unroll
        for (int i = 0; i < Cfg::SLOADS + Cfg::ZLOADS; ++i)
            __builtin_amdgcn_global_load_lds((const void*)(szp[i] + (at << szshift[i])),
                                             (GF_LDS void*)(buf + 4096 + i * 256), 4, 0, 0);
        ++issued;
        if (++ib == nb) { ib = 0; ig += parts; }
        if (++islot == ring) islot = 0;
    };
    // At most `left` younger tasks' loads stay pending.
    auto wait_tasks = [&](int left) __attribute__((always_inline)) {
        left = __builtin_amdgcn_readfirstlane(left);
        if (left >= 3) wait_vmcnt<3 * L>();
        else if (left == 2) wait_vmcnt<2 * L>();
        else if (left == 1) wait_vmcnt<L>();
        else wait_vmcnt<0>();
    };
    int done = 0, slot = 0;
    half8 xreg[Cfg::XLDS ? 1 : Cfg::XB * 16][MB];
    if constexpr (Cfg::XLDS) {
        const int first = min(ring, ntasks);
        for (int i = 0; i < first; ++i) issue();
        if (first >= 4) wait_vmcnt<4 * L>();              // A has landed: only whole tasks are pending
        else wait_tasks(first);
        lds_barrier();
    } else if (nb > 0) {
        // A passes through the tasks' buffers too, 16 rows by 128 k at a time, so
        // that it is read in whole lines; the tasks follow it.
        constexpr int P = Cfg::XB * 4 * MB;
        const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
            (void*)a.A, 0, (int)((uint32_t)M * (uint32_t)K * 2u), 0x00020000);
        uint32_t xoff[MB][4];
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * i + c4;
                xoff[m][i] = (uint32_t)min(16 * m + r, M - 1) * (uint32_t)K * 2u + (uint32_t)(r16 ^ r) * 16u;
            }
        auto issue_x = [&](auto p_c) __attribute__((always_inline)) {
            constexpr int b = decltype(p_c)::value / (4 * MB), c = decltype(p_c)::value / MB % 4,
                          m = decltype(p_c)::value % MB;
            GF_LDS char* buf = tasks + islot * Cfg::TASK_BYTES;
            const uint32_t so = (uint32_t)__builtin_amdgcn_readfirstlane(
                min(b0 + b, nblk - 1) * (Cfg::BK * 2) + c * 256);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (GF_LDS void*)(buf + i * 1024), 16, xoff[m][i], so, 0, 0);
            if (++islot == ring) islot = 0;
        };
        static_for<Cfg::MAX_RING < P ? Cfg::MAX_RING : P>([&](auto p) __attribute__((always_inline)) {
            if (decltype(p)::value < ring) issue_x(p);
        });
        static_for<P>([&](auto p_c) __attribute__((always_inline)) {
            constexpr int p = decltype(p_c)::value, b = p / (4 * MB), c = p / MB % 4, m = p % MB;
            // younger pieces and tasks, of 4 loads at least
            const int left = __builtin_amdgcn_readfirstlane(min(p + ring, P) + issued - p - 1);
            if (left >= 3) wait_vmcnt<12>();
            else if (left == 2) wait_vmcnt<8>();
            else if (left == 1) wait_vmcnt<4>();
            else wait_vmcnt<0>();
            asm volatile("" ::: "memory");
            const GF_LDS char* buf = tasks + slot * Cfg::TASK_BYTES;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const half8 v = *(const GF_LDS half8*)(buf + r16 * 256 + (((xchunk + xstep * i) ^ r16) * 16));
                xreg[b * 16 + c * 4 + i][m] = __builtin_shufflevector(v, v, 0, 4, 1, 5, 2, 6, 3, 7);
            }
            asm volatile("" ::: "memory");
            wait_lgkmcnt0();
            // the freed buffer: the piece after those in flight (rings of 1 to 4),
            // or the next task
            static_for<Cfg::MAX_RING>([&](auto r) __attribute__((always_inline)) {
                constexpr int ahead = decltype(r)::value + 1;
                if (ring == ahead) {
                    if constexpr (p + ahead < P) issue_x(std::integral_constant<int, p + ahead>{});
                    else if (issued < ntasks) issue();
                }
            });
            if (++slot == ring) slot = 0;
        });
    }

    for (int gi = 0; gi < ng; ++gi) {
        floatx4 acc[MB] = {};
        auto block = [&](int b, auto xb_c) __attribute__((always_inline)) {
            constexpr int xb = decltype(xb_c)::value;
            wait_tasks(issued - done - 1);
            asm volatile("" ::: "memory");
            const GF_LDS char* buf = tasks + slot * Cfg::TASK_BYTES;
            const GF_LDS uint32_t* sz = (const GF_LDS uint32_t*)(buf + 4096) + r16;
            uint32_t sw[Cfg::SWORDS], zw[Cfg::ZWORDS];
#pragma unroll
            for (int j = 0; j < Cfg::SWORDS; ++j) sw[j] = sz[16 * j];
#pragma unroll
            for (int j = 0; j < Cfg::ZWORDS; ++j)
                zw[j] = a.Z ? sz[16 * ((GROUP == 128 ? 2 : Cfg::SLOADS * 4) + j)] : 0x08080808u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {             // chunks of 128 k
                u32x4 q = *(const GF_LDS u32x4*)(buf + qat[c]);
                if constexpr (GROUP < 128) q = w4_exchange(q);
                constexpr int SPG = GROUP / 32, GPC = 128 / GROUP;
#pragma unroll
                for (int g0 = 0; g0 < GPC; ++g0) {
                    const int g = c * GPC + g0;       // within the block
                    const _Float16 s = __builtin_bit_cast(_Float16, (uint16_t)(sw[g / 2] >> (16 * (g % 2))));
                    const half2v nz = -__builtin_bit_cast(half2v, __builtin_amdgcn_perm(
                        0u, zw[g / 4], 0x0c000c00u + 0x00010001u * (uint32_t)(g % 4)));
                    floatx4 sum[MB] = {};
#pragma unroll
                    for (int i = g0 * SPG; i < (g0 + 1) * SPG; ++i) {
                        if constexpr (Cfg::XLDS) {
                            const half8 x = *(const GF_LDS half8*)(xs + xat[i] + b * (Cfg::BK * 2) + c * 256);
                            sum[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w4_unpack(q[i], nz), sum[0], 0, 0, 0);
                        } else {
                            const half8 w = w4_unpack_pairs(q[i], nz);
#pragma unroll
                            for (int m = 0; m < MB; ++m)
                                sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xreg[xb * 16 + 4 * c + i][m], w,
                                                                                sum[m], 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < MB; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][i] = fmaf(sum[m][i], (float)s, acc[m][i]);
                }
            }
            asm volatile("" ::: "memory");
            wait_lgkmcnt0();                          // the buffer is read: it may be filled again
            if (issued < ntasks) issue();
            ++done;
            if (++slot == ring) slot = 0;
        };
        if constexpr (Cfg::XLDS) {
            for (int b = 0; b < nb; ++b) block(b, std::integral_constant<int, 0>{});
        } else {
            static_for<Cfg::XB>([&](auto xb) __attribute__((always_inline)) {
                if (decltype(xb)::value < nb) block(decltype(xb)::value, xb);
            });
        }
        // ---- the waves' sums, in wave order ----
        GF_LDS float* mine = red + (gi & 1) * WAVES * red_rows * 16;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * m + 4 * c4 + i;
                if (row < M) mine[(wave * red_rows + row) * 16 + r16] = acc[m][i];
            }
        lds_barrier();
        const int n0 = min((part + gi * parts) * 16, N - 16);
        for (int t = threadIdx.x; t < M * 16; t += WAVES * kWave) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) s += mine[w * red_rows * 16 + t];
            w4_store<GROUPED>(a, (size_t)(t / 16) * N + n0 + t % 16, s * kW4Unit);
        }
    }
    wait_vmcnt<0>();
#endif
}

// ---------------------------------------------------------------------------
// tiles: many rows of A
// ---------------------------------------------------------------------------
//
// A BM x BN tile by WM x WN waves of 32 FM rows by 32 FN columns, over K in
// steps of 64.  Bound by the matrix cores, so here each weight is rounded once
// to fp16, (q - z) * s as w4_dequantize_f16 rounds it, and the products are
// accumulated over all of K in place: the result is that of gemm_f16_nt on the
// dequantized weights.  (Scaling each group's sum in fp32 instead keeps the
// weights exact, but holds a second set of accumulators and passes all of them
// through the vector ALU once per group: built, it ran at 0.6 of this form's
// rate with groups of 128 and 0.3 with groups of 32.)
//  * A goes to LDS by direct loads, STAGES buffers in a ring, rows swizzled as
//    in gemm_kernel.hpp (chunk c of row r at slot c ^ (r / 2 % 8)).
//  * The codes never pass through LDS: a lane loads 16 bytes of its own row of
//    Q and unpacks them in registers as MFMA operands.  Which k an MFMA step
//    holds is free as long as both operands agree: lane half h takes words
//    4 h .. 4 h + 3 of the 64 k, step j word j of them, and A's chunks are read
//    to match.  A lane's 32 k lie in one group whatever its size, so the lane
//    needs one scale and zero point per step.
//  * Under the MFMAs of one unpacked operand the next one is unpacked (16
//    vector instructions for 8 codes, FM MFMAs of 32 cycles each), and under
//    those of a step of 16 k the next step's fragments of A are read.
//  * The barrier of step t stands before its last 16 k: by then every wave has
//    read all of step t's fragments and has waited for its own loads of step
//    t + 1, so the next fragments are read, and the loads of step t + STAGES
//    issued into the freed buffer, under the last MFMAs.  At most the direct
//    loads of STAGES - 2 steps are then pending: a count of those alone, since
//    the compiler may merge or reorder the loads into registers, for which it
//    waits itself.  Loads are issued for every step, also past the last, and
//    from inside the rows: where K ends within a step, what lies past it is
//    cleared once the last step has landed.  No load stands under a branch or
//    goes through the flat path: the compiler would then wait for all of them
//    wherever it needs one.
// 2048 x 8192 x 4096 in groups of 128: 129 us, 1065 TFLOP/s (gemm_f16_nt's tiles
// reach 1280 to 1370 at 8192 x 8192 x 8192).
template <int FM_, int FN_, int WM_, int WN_, int STAGES_>
struct W4TileCfg {
    static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr int WAVES = WM * WN, NT = WAVES * kWave;
    static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN, BK = 64;
    static constexpr int STAGE_BYTES = BM * BK * 2;
    static constexpr int LPS = BM * 8 / NT;              // 16-byte loads of A per thread and step
    static_assert(LPS >= 1 && BM * 8 % NT == 0 && LPS * (STAGES - 2) < 64, "loads per thread");
    static constexpr int EPAD = 8;
    static constexpr int EPI_BYTES = WAVES * 32 * FM * (32 * FN + EPAD) * 2;
    static constexpr int LDS_BYTES = STAGES * STAGE_BYTES > EPI_BYTES ? STAGES * STAGE_BYTES : EPI_BYTES;
    static_assert(LDS_BYTES <= 160 * 1024, "one CU's LDS");
};

// K >= 64, A 16-byte aligned.  WINDOW: K % 256 == 0.  A row of Q, S or Z is a
// line of its own, so what a lane loads from them costs a line whatever its
// width: codes are then loaded two steps at a time and scales and zero points
// four (a window).  Otherwise step by step.
template <class Cfg, int GROUP, bool WINDOW, bool GROUPED>
__global__ __launch_bounds__(Cfg::NT) void w4_tile_kernel(W4Args a)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int FM = Cfg::FM, FN = Cfg::FN, BK = Cfg::BK, S = Cfg::STAGES;
    extern __shared__ __attribute__((aligned(1024))) char w4_smem[];
    GF_LDS char* smem = (GF_LDS char*)w4_smem;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
    const int r32 = lane % 32, h = lane / 32;

    const int tiles_n = ceil_div(a.N, Cfg::BN);
    int tm, tn, M = a.M;
    if constexpr (GROUPED) {
        int e, lo, hi, item;
        if (!a.g.template find<Cfg::BM>(a.g.workgroup(), tiles_n, e, lo, hi, item)) return;
        M = hi - lo;
        a.A += (size_t)lo * a.K;
        a.C += (size_t)lo * a.N;
        a.Q += (size_t)e * a.N * (a.K / 8);
        a.S += (size_t)e * a.N * a.G;
        if (a.Z) a.Z += (size_t)e * a.N * a.G;
        grouped_tile(item, ceil_div(M, Cfg::BM), tiles_n, kGroupPanel, tm, tn);
    } else {
        const int tiles_m = ceil_div(M, Cfg::BM);
        grouped_tile(xcd_remap(a.g.workgroup(), tiles_m * tiles_n), tiles_m, tiles_n, kGroupPanel, tm, tn);
    }
    const int m0 = tm * Cfg::BM, n0 = tn * Cfg::BN;
    const int K = a.K, nk = ceil_div(K, BK);

    // ---- A: byte offset of load r's chunk at k = 0 ----
    uint32_t voff[Cfg::LPS];
#pragma unroll
    for (int r = 0; r < Cfg::LPS; ++r) {
        const int slot = r * Cfg::NT + tid, row = slot / 8, c = (slot % 8) ^ (row / 2 % 8);
        voff[r] = ((uint32_t)min(m0 + row, M - 1) * (uint32_t)K + 8u * c) * 2u;
    }
    // In the last step, chunks past K: the last one inside instead (zeros later).
    const int last_chunks = (K - (nk - 1) * BK) / 8;
    uint32_t back[Cfg::LPS];
#pragma unroll
    for (int r = 0; r < Cfg::LPS; ++r) {
        const int slot = r * Cfg::NT + tid, c = (slot % 8) ^ (slot / 16 % 8);
        back[r] = WINDOW ? 0u : 16u * (uint32_t)max(c - (last_chunks - 1), 0);
    }
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        (void*)a.A, 0, (int)((uint32_t)M * (uint32_t)K * 2u), 0x00020000);
    auto issue_a = [&](int t, int stage_no) __attribute__((always_inline)) {
        GF_LDS char* stage = smem + stage_no * Cfg::STAGE_BYTES;
        const int ts = __builtin_amdgcn_readfirstlane(min(t, nk - 1));
#pragma unroll
        for (int r = 0; r < Cfg::LPS; ++r)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (GF_LDS void*)(stage + (r * Cfg::NT + wave * kWave) * 16), 16,
                WINDOW || ts < nk - 1 ? voff[r] : voff[r] - back[r], (uint32_t)ts * (BK * 2), 0, 0);
    };

    // ---- codes, scale and zero point of the lane's 32 k in each column block ----
    constexpr int D = WINDOW ? 4 : 2;                     // steps unrolled: one window, or the codes' two
    constexpr int SW = WINDOW ? 128 / GROUP : 1, ZW = WINDOW && GROUP == 32 ? 2 : 1;   // registers
    // (without zero points, the bytes of S stand in for the loads' sake)
    const uint8_t* zsrc = a.Z ? a.Z : (const uint8_t*)a.S;
    const uint32_t* qrow[FN];
    int srow[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        const int n = min(n0 + (wn * FN + f) * 32 + r32, a.N - 1);
        qrow[f] = a.Q + (size_t)n * (K / 8);
        srow[f] = n * a.G;
    }
    // Codes of step t in codes[t % D]; scales and zero points of the window, or
    // of step t in place t % D.
    u32x4 codes[D][FN];
    uint32_t sw[WINDOW ? 1 : D][FN][SW], zw[WINDOW ? 1 : D][FN][ZW];
    auto load_codes = [&](int t, auto i_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
        const int kc = min(min(t, nk - 1) * BK + 32 * h, K - 32);
#pragma unroll
        for (int f = 0; f < FN; ++f) codes[i][f] = *(const u32x4_any*)(qrow[f] + kc / 8);
    };
    auto load_scales = [&](int t, auto i_c) __attribute__((always_inline)) {
        constexpr int i = WINDOW ? 0 : decltype(i_c)::value;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            if constexpr (WINDOW) {
                const int at = srow[f] + min(t * BK, K - 4 * BK) / GROUP;
                load_words<SW>(a.S + at, sw[i][f]);
                load_words<GROUP == 128 ? 0 : ZW>(zsrc + at, zw[i][f]);
            } else {
                const int at = srow[f] + min(min(t, nk - 1) * BK + 32 * h, K - 8) / GROUP;
                sw[i][f][0] = a.S[at];
                zw[i][f][0] = zsrc[at];
            }
        }
    };
    // In the last step: how many words of this lane's 32 k lie inside K, and how
    // many words its codes, loaded from inside the row, are ahead of their place.
    const int last_k = (nk - 1) * BK + 32 * h;
    const int last_words = WINDOW ? 4 : max(K - last_k, 0) / 8;
    const int last_ahead = max(last_k - (K - 32), 0) / 8;
    half2v off[FN], sc[FN];
    // Scale and offset of step i of the D unrolled.
    auto scale = [&](auto i_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            uint32_t sb, z;
            if constexpr (!WINDOW) {
                sb = sw[i][f][0];
                z = zw[i][f][0];
            } else if constexpr (GROUP == 32) {
                sb = sw[0][f][i % SW] >> (16 * h);
                z = zw[0][f][i / 2 % ZW] >> (16 * (i % 2) + 8 * h);
            } else {
                constexpr int g = i * BK / GROUP;         // within the window
                sb = sw[0][f][g / 2 % SW] >> (16 * (g % 2));
                z = zw[0][f][0] >> (8 * g);
            }
            sc[f] = w4_twice(sb);
            off[f] = w4_offsets(a.Z ? z : 8u);
        }
    };

    // The operand of column block f for 16 k j of step t, which is step i of the D
    // unrolled.  A word past K stands for zeros: its codes are 0, but 0 - z times a
    // large scale would pass the fp16 range, and infinity times the cleared A is NaN.
    auto operand = [&](int t, auto i_c, auto f_c, auto j_c) __attribute__((always_inline)) {
        constexpr int i = decltype(i_c)::value, f = decltype(f_c)::value, j = decltype(j_c)::value;
        half2v s = sc[f];
        if constexpr (!WINDOW) s = t < nk - 1 || j < last_words ? s : w4_twice(0u);
        return w4_weights(codes[i][f][j], off[f], s);
    };

    // ---- fragments of A ----
    const int abase = (wm * FM * 32 + r32) * (BK * 2), akey = r32 / 2 % 8;
    half8 x[2][FM];
    auto read_x = [&](int stage_no, auto j_c) __attribute__((always_inline)) {
        constexpr int j = decltype(j_c)::value;
        const GF_LDS char* p = smem + stage_no * Cfg::STAGE_BYTES + abase + (((4 * h + j) ^ akey) * 16);
#pragma unroll
        for (int f = 0; f < FM; ++f) x[j & 1][f] = *(const GF_LDS half8*)(p + f * 32 * (BK * 2));
    };

    floatx16 acc[FM][FN] = {};
    half8 b;
    // FM MFMAs with operand b of column block f and fragments x[j & 1], woven
    // with the LDS reads and unpacking the caller has issued before them.
    auto mfmas = [&](auto f_c, auto j_c, half8 op) __attribute__((always_inline)) {
        constexpr int f = decltype(f_c)::value, j = decltype(j_c)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[j & 1][i], op, acc[i][f], 0, 0, 0);
        static_for<FM>([&](auto) __attribute__((always_inline)) {
            __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
            if constexpr (f == 0) __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 20 / FM, 0);         // vector ALU
        });
        __builtin_amdgcn_sched_barrier(0);
    };

    static_for<D>([&](auto p) __attribute__((always_inline)) {
        load_codes(decltype(p)::value, p);
        if constexpr (!WINDOW || decltype(p)::value == 0) load_scales(decltype(p)::value, p);
    });
    asm volatile("" ::: "memory");
#pragma unroll
    for (int t = 0; t < S - 1; ++t) issue_a(t, t);
    asm volatile("" ::: "memory");
    wait_vmcnt<Cfg::LPS * (S - 2)>();
    lds_barrier();                                        // step 0 has landed
    issue_a(S - 1, S - 1);
    read_x(0, std::integral_constant<int, 0>{});
    scale(std::integral_constant<int, 0>{});
    constexpr std::integral_constant<int, 0> zero_c;
    b = operand(0, zero_c, zero_c, zero_c);

    int st = 0;                                           // buffer of step t
    auto step = [&](int t, auto p) __attribute__((always_inline)) {
        constexpr int i = decltype(p)::value, i1 = (i + 1) % D;
        const int st1 = st + 1 == S ? 0 : st + 1;
        static_for<4>([&](auto j_c) __attribute__((always_inline)) {
            constexpr int j = decltype(j_c)::value;
            if constexpr (j == 3) {
                asm volatile("" ::: "memory");
                wait_vmcnt<Cfg::LPS * (S - 2)>();
                lds_barrier();                            // step t + 1 has landed; buffer st is free
                if constexpr (!WINDOW) {
                    if (K % BK != 0 && t == nk - 2) {     // the last step's k past K: zeros on both sides
                        for (int z = tid; z < Cfg::BM * 8; z += Cfg::NT) {
                            const int row = z / 8, c = z % 8;
                            if (c >= last_chunks)
                                *(GF_LDS u32x4*)(smem + st1 * Cfg::STAGE_BYTES + row * (BK * 2) +
                                                 ((c ^ (row / 2 % 8)) * 16)) = u32x4{0u, 0u, 0u, 0u};
                        }
#pragma unroll
                        for (int f = 0; f < FN; ++f) {
                            u32x4 q = codes[i1][f];
                            if (last_ahead & 1) q = u32x4{q[1], q[2], q[3], 0u};
                            if (last_ahead & 2) q = u32x4{q[2], q[3], 0u, 0u};
                            codes[i1][f] = q;
                        }
                        lds_barrier();
                    }
                }
                issue_a(t + S, st);
            }
            static_for<FN>([&](auto f_c) __attribute__((always_inline)) {
                constexpr int f = decltype(f_c)::value;
                if constexpr (f == 0) {
                    if constexpr (j < 3) read_x(st, std::integral_constant<int, j + 1>{});
                    else read_x(st1, std::integral_constant<int, 0>{});
                }
                // the next operand: the next column block's, or the next 16 k's first
                half8 next;
                if constexpr (f + 1 < FN) {
                    next = operand(t, p, std::integral_constant<int, f + 1>{}, j_c);
                } else if constexpr (j < 3) {
                    next = operand(t, p, zero_c, std::integral_constant<int, j + 1>{});
                } else {
                    scale(std::integral_constant<int, i1>{});
                    next = operand(t + 1, std::integral_constant<int, i1>{}, zero_c, zero_c);
                }
                mfmas(f_c, j_c, b);
                b = next;
            });
        });
        if constexpr (!WINDOW) {
            load_codes(t + D, p);
            load_scales(t + D, p);
        } else {
            if constexpr (i % 2 == 1) {                   // a pair of steps done: the pair four steps on
                load_codes(t + 3, std::integral_constant<int, i - 1>{});
                load_codes(t + 4, p);
            }
            if constexpr (i == 2) load_scales(t + 2, p);  // the window's last use was the next step's scale()
        }
        st = st1;
    };
    int t = 0;
    for (; t + D <= nk; t += D)                           // (a window never leaves a rest)
        static_for<D>([&](auto p) __attribute__((always_inline)) { step(t + decltype(p)::value, p); });
    if constexpr (!WINDOW)
        if (t < nk) step(t, std::integral_constant<int, 0>{});
    wait_vmcnt<0>();                                      // no load may land once the epilogue writes LDS

    constexpr int WR = 32 * FM, WC = 32 * FN, LDW = WC + Cfg::EPAD;
    if (!GROUPED && a.f32) {                              // 128 bytes of a row a store
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int fn = 0; fn < FN; ++fn)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = m0 + wm * WR + f * 32 + 8 * (i / 4) + 4 * h + i % 4;
                    const int col = n0 + wn * WC + fn * 32 + r32;
                    if (row < M && col < a.N) ((float*)a.C)[(size_t)row * a.N + col] = acc[f][fn][i];
                }
        return;
    }

    // ---- epilogue: per-wave transpose in LDS, 16-byte stores ----
    lds_barrier();
    GF_LDS uint16_t* reg = (GF_LDS uint16_t*)(smem + wave * (WR * LDW * 2));
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int fn = 0; fn < FN; ++fn)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                reg[(f * 32 + 8 * (i / 4) + 4 * h + i % 4) * LDW + fn * 32 + r32] =
                    f32_to_f16_bits(acc[f][fn][i]);
    asm volatile("" ::: "memory");
    wait_lgkmcnt0();
    constexpr int CPR = WC / 8, ITERS = WR * CPR / kWave;
#pragma unroll
    for (int it = 0; it < ITERS; ++it) {
        const int q = it * kWave + lane, r = q / CPR, cc = q % CPR;
        const u32x4 v = *(const GF_LDS u32x4*)(reg + r * LDW + cc * 8);
        const int row = m0 + wm * WR + r, col = n0 + wn * WC + cc * 8;
        if (row >= M) continue;
        uint16_t* dst = a.C + (size_t)row * a.N + col;
        if (col + 8 <= a.N) {                             // (whatever its alignment)
            __builtin_nontemporal_store(v, (u32x4_any*)dst);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e < a.N) dst[e] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
        }
    }
#endif
}

}  // namespace gf
