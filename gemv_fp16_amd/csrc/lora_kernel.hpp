// Low-rank adapters: C[m] = base + scale[a] * (A[m] . Down[a]^T) . Up[a]^T, a = ids[m].
//
// Two launches: H, the scaled products by Down, in fp32; then the base product with
// H . Up[a]^T added to its accumulators before its one rounding (one or two rows in
// vectors, up to 32 streaming B, beyond the tiles of gemm_kernel.hpp), or, for a base that
// is computed already, that sum alone: onto a base in fp32, which is rounded with it, or
// in place.  From 3 to 32 rows of a narrow B the first launch takes the base's parts as
// well (K in slices), and the second joins all.  Where none of these forms fits, the base
// comes as fp32 parts from gemm_kernel.hpp.  Operands off the 16-byte grid, or K or r that
// are not multiples of 8, take the general forms: an output or a lane at a time.
#pragma once
#include "gemm_kernel.hpp"
#include "gemv_kernel.hpp"
#include "low_rank.hpp"

namespace gf {

constexpr int kLoraParts = 8, kLoraTileParts = 4;   // of K in the products by Down, at most (up to 32 rows; beyond)

struct LoraArgs {
    const uint16_t* A;       // M x K
    const uint16_t* B;       // N x K, or null: the base is there already
    const int* ids;          // M
    const uint16_t* Down;    // L x r x K
    const uint16_t* Up;      // L x N x r
    const float* scales;     // L, or null
    uint16_t* C;             // M x N
    float* H;                // S x M x r
    int64_t part;            // floats of one of the S
    const float* base;       // parts x M x N (BASE forms), else C holds it
    int M, N, K, r, L, S, parts;

    __device__ __forceinline__ LowRank low() const { return {H, ids, Up, part, S, r, L}; }
};

// A uniform value through the scalar cache (read-only while the kernel runs).
template <class T>
__device__ __forceinline__ T scalar_load(const T* p)
{
    return *(const __attribute__((address_space(4))) T*)(uintptr_t)p;
}

// ---------------------------------------------------------------------------
// products by Down
// ---------------------------------------------------------------------------
//
// Workgroup (16-row block and z, s) works for every Z-th of the block's adapters: one
// is read once for each block that has it.  The waves, and S workgroups, split K in
// tasks of 128 k: 16 rows of A and RB times 16 ranks of Down come to LDS by direct
// loads of whole cache lines (chunk c of row n at slot c ^ n, so that the 16 rows read
// together lie in different banks), A's before the ids are known, and meet in MFMAs 16
// x 16 x 32; the results of rows with other adapters are dropped, and the waves' sums
// added in order.  Ranks past 16 * RB: further passes over A.
// Bound by the bytes, and for few rows by the chain of ids, loads and sums.  Loads
// straight to registers, 16 rows of 64 bytes each, came to 2.2 TB/s (8192 rows, rank
// 16, K = 4096: 30 us).
template <int W_, int RB_>
struct LoraDownCfg {
    static constexpr int W = W_, RB = RB_, TILE = 4096, WAVE_BYTES = (1 + RB) * TILE;
    static constexpr int PART_BYTES = W * RB * kWave * 16, LDS_BYTES = W * WAVE_BYTES + PART_BYTES;
    static_assert(LDS_BYTES <= 160 * 1024, "one CU's LDS");
};

template <class Cfg>
__global__ __launch_bounds__(Cfg::W * kWave) void lora_down_kernel(LoraArgs a, int Z)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int W = Cfg::W, RB = Cfg::RB;
    extern __shared__ __attribute__((aligned(1024))) char smem_raw[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, c4 = lane / 16;
    GF_LDS char* tiles = (GF_LDS char*)smem_raw + wave * Cfg::WAVE_BYTES;   // A's, then Down's
    GF_LDS floatx4* parts = (GF_LDS floatx4*)((GF_LDS char*)smem_raw + W * Cfg::WAVE_BYTES);   // [W][RB][64]
    const int tasks = ceil_div(a.K, 128), cut = a.S * W, blocks = ceil_div(a.M, 16);
    const int part = blockIdx.y * W + wave;
    const int t0 = (int)((int64_t)tasks * part / cut), t1 = (int)((int64_t)tasks * (part + 1) / cut);
    // 16 rows first .. (those past `last` are that one) of 128 k from task t
    auto load = [&](const uint16_t* base, int first, int last, int t, GF_LDS char* tile) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * i + c4, k = t * 128 + (r16 ^ row) * 8;
            const void* p = base + (size_t)min(first + row, last) * a.K + k;
            if (k >= a.K) p = (const void*)g_zero16;
            __builtin_amdgcn_global_load_lds(p, (GF_LDS void*)(tile + i * 1024), 16, 0, 0);
        }
    };
    auto frag = [&](const GF_LDS char* tile, int i) __attribute__((always_inline)) {
        return *(const GF_LDS half8*)(tile + r16 * 256 + (((4 * i + c4) ^ r16) * 16));
    };
    for (int w = blockIdx.x; w < blocks * Z; w += gridDim.x) {
        const int block = w % blocks * 16, z = w / blocks;
        const int mine = block + r16 < a.M ? a.ids[block + r16] : -1;
        int held = t0;                           // the task whose rows of A are in LDS
        if (t0 < t1) load(a.A, block, a.M - 1, t0, tiles);
        uint32_t left = (uint32_t)__ballot((unsigned)mine < (unsigned)a.L) & 0xFFFF;
        for (int d = 0; left; ++d) {
            const int id = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
            const uint32_t rows = (uint32_t)__ballot(mine == id) & left;
            left &= ~rows;
            if (d % Z != z) continue;
            const uint16_t* down = a.Down + (size_t)id * a.r * a.K;
            const float scale = a.scales ? scalar_load(a.scales + id) : 1.0f;
            for (int j0 = 0; j0 < a.r; j0 += 16 * RB) {
                floatx4 acc[RB] = {};
                for (int t = t0; t < t1; ++t) {
                    if (t != held) load(a.A, block, a.M - 1, t, tiles);
                    held = t;
#pragma unroll
                    for (int b = 0; b < RB; ++b) load(down, j0 + 16 * b, a.r - 1, t, tiles + (1 + b) * Cfg::TILE);
                    wait_vmcnt<0>();
                    asm volatile("" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const half8 x = frag(tiles, i);
#pragma unroll
                        for (int b = 0; b < RB; ++b)
                            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, frag(tiles + (1 + b) * Cfg::TILE, i), acc[b], 0, 0, 0);
                    }
                    asm volatile("" ::: "memory");
                    wait_lgkmcnt0();             // the tiles are read: they may be filled again
                }
                __syncthreads();                 // the sums of the pass before are read
#pragma unroll
                for (int b = 0; b < RB; ++b) parts[(wave * RB + b) * kWave + lane] = acc[b];
                __syncthreads();
                for (int t = threadIdx.x; t < RB * kWave; t += W * kWave) {
                    const int l = t % kWave, j = j0 + 16 * (t / kWave) + l % 16;
                    floatx4 sum = parts[t];
#pragma unroll
                    for (int v = 1; v < W; ++v) sum += parts[v * RB * kWave + t];
                    // accumulator i of lane l: row 4 * (l / 16) + i, rank l % 16
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 4 * (l / 16) + i;
                        if (j < a.r && ((rows >> row) & 1))
                            a.H[blockIdx.y * a.part + (size_t)(block + row) * a.r + j] = scale * sum[i];
                    }
                }
            }
        }
        wait_vmcnt<0>();                         // rows of A that nobody wanted: the next ones go to their place
    }
#endif
}

template <class Cfg>
hipError_t launch_lora_down(const LoraArgs& a, dim3 grid, int Z, hipStream_t stream)
{
    auto kern = lora_down_kernel<Cfg>;
    static std::atomic<uint64_t> lds_opt_in{0};
    const hipError_t e = opt_in_lds((const void*)kern, Cfg::LDS_BYTES, lds_opt_in, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, grid, dim3(Cfg::W * kWave), Cfg::LDS_BYTES, stream, a, Z);
    return hipGetLastError();
}

// Any alignment, K and r: a workgroup a row, a wave a rank at a time (S == 1).
__global__ __launch_bounds__(256) void lora_down_any_kernel(LoraArgs a)
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
            for (int k = lane; k < a.K; k += kWave) s = __builtin_fmaf(f16_bits_to_f32(x[k]), f16_bits_to_f32(w[k]), s);
            s = wave_sum(s);
            if (lane == 0) a.H[(size_t)m * a.r + j] = scale * s;
        }
    }
}

// ---------------------------------------------------------------------------
// H . Up[a]^T added to C
// ---------------------------------------------------------------------------
//
// The operands are swapped (Up's rows in the place of A's), so that a lane holds four
// neighbouring columns of one row.  C is asked for before the sums are worked out, which
// takes a chain of loads out of it (lora_add_f16, 2048 rows of 8 adapters, rank 64, at
// 4096 x 4096: 35.5 us, rank 16 21; a copy of C takes 6.5, the products by Down 7 to 14).
// What bounds it past rank 16 are H's and Up's bytes through L2.
struct SwappedMfma {
    typedef floatx4 acc_t;
    static constexpr int NACC = 4;
    static constexpr bool ROW_IN_LANE = true;    // all of a lane's accumulators are of one row
    static __device__ __forceinline__ acc_t run(half8 h, half8 u, acc_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(u, h, c, 0, 0, 0);
    }
    static __device__ __forceinline__ int row(int, int lane) { return lane % 16; }
};

// The adapters' sums of a wave's 16 rows and 16 columns, J waves to a block: each has
// 32 ranks in turn, and the first adds what the others found, in order.  True for the
// waves that have the sums.  All of a wave's adapters have their loads in flight: each
// round of them is a chain of 3 us.  (lora_add_f16, 32 rows of 32 adapters, rank 64, at
// 8192 x 4096: 22.2 us, with one wave to a block and 8 adapters at a time 27.0.)
template <int J, int SP>
__device__ __forceinline__ bool lora_join(const LowRank& low, floatx4 (&sum)[1], int row0, int col0, int M, int N)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, j = wave % J;
    low.template block<SwappedMfma, 16, 32, 1, 16, SP>(sum, row0, col0, M, N, 32 * j, 32 * J);
    if constexpr (J > 1) {
        __shared__ floatx4 part[4][kWave];
        part[wave][lane] = sum[0];
        __syncthreads();
        if (j > 0) return false;
#pragma unroll
        for (int i = 1; i < J; ++i) sum[0] += part[wave + i][lane];
    }
    return true;
}

// Parts of a base in fp32, at most.
constexpr int kLoraBaseParts = 8;

// Columns n .. n + 3 of row m of each part (zeros where there are none): all loads in flight.
struct LoraBase {
    floatx4 v[kLoraBaseParts];

    __device__ __forceinline__ void load(const LoraArgs& a, int m, int n)
    {
        const float* p = a.base + (size_t)m * a.N + n;
        const size_t part = (size_t)a.M * a.N;
#pragma unroll
        for (int s = 0; s < kLoraBaseParts; ++s) {
            v[s] = floatx4{};
            if (s >= a.parts) continue;
            if (n + 4 <= a.N) __builtin_memcpy(&v[s], p + s * part, 16);
            else
                for (int i = 0; n + i < a.N; ++i) v[s][i] = p[s * part + i];
        }
    }
    __device__ __forceinline__ floatx4 sum() const   // in order
    {
        floatx4 t = v[0];
#pragma unroll
        for (int s = 1; s < kLoraBaseParts; ++s) t += v[s];
        return t;
    }
};

// 16 rows by 16 columns, J waves each.  BASE: the base's parts and the adapters, rounded
// once, to every row of C; else C, the base, gets the adapters added in its rows that
// have one.
template <int J, bool BASE>
__global__ __launch_bounds__(256) void lora_up_few_kernel(LoraArgs a, int vec)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = threadIdx.x % kWave, r16 = lane % 16, c4 = lane / 16;
    const int across = ceil_div(a.N, 16), items = across * ceil_div(a.M, 16);
    const LowRank low = a.low();
    const int w = __builtin_amdgcn_readfirstlane(min((int)(blockIdx.x * 4 + threadIdx.x / kWave) / J, items - 1));
    const int row0 = w / across * 16, col0 = w % across * 16, m = row0 + r16, n = col0 + 4 * c4;
    uint16_t* c = a.C + (size_t)min(m, a.M - 1) * a.N + n;
    const bool four = vec && n + 4 <= a.N;
    typedef _Float16 half4 __attribute__((ext_vector_type(4)));
    half4 v = {};
    [[maybe_unused]] LoraBase base;
    if constexpr (BASE) {                        // asked for before the sums are worked out
        if (threadIdx.x / kWave % J == 0) base.load(a, min(m, a.M - 1), n);
    } else {
        if (four) v = *(const half4*)c;
    }
    floatx4 sum[1];
    if (!lora_join<J, kLoraParts>(low, sum, row0, col0, a.M, a.N)) return;
    if ((int)(blockIdx.x * 4 + threadIdx.x / kWave) / J >= items || m >= a.M) return;
    if constexpr (BASE) {
        sum[0] = low.adapter(m, a.M) < 0 ? base.sum() : base.sum() + sum[0];
    } else {
        if (low.adapter(m, a.M) < 0) return;
        if (four)
            for (int i = 0; i < 4; ++i) sum[0][i] += (float)v[i];
        else
            for (int i = 0; i < 4; ++i) sum[0][i] += n + i < a.N ? f16_bits_to_f32(c[i]) : 0.0f;
    }
    if (four) {
        half4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (_Float16)sum[0][i];
        *(half4*)c = o;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.N) c[i] = f32_to_f16_bits(sum[0][i]);
    }
#endif
}

// 16 rows by 64 columns a wave, S <= SP; BASE as above, of one part (more are added one
// after the other, each a round of loads).
template <int SP, bool BASE>
__global__ __launch_bounds__(256, SP > 4 ? 3 : 4) void lora_up_kernel(LoraArgs a, int vec)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int NB = 4;
    const int lane = threadIdx.x % kWave, r16 = lane % 16, c4 = lane / 16;
    const int across = ceil_div(a.N, 16 * NB), down = ceil_div(a.M, 16);
    const LowRank low = a.low();
    const int64_t items = (int64_t)across * down;
    for (int64_t w = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; w < items; w += (int64_t)gridDim.x * 4) {
        const int row0 = __builtin_amdgcn_readfirstlane((int)(w / across) * 16);
        const int col0 = __builtin_amdgcn_readfirstlane((int)(w % across) * 16 * NB);
        const int m = row0 + r16;
        typedef _Float16 half4 __attribute__((ext_vector_type(4)));
        typedef typename std::conditional<BASE, floatx4, half4>::type base4;
        base4 v[NB];                             // asked for before the sums are worked out
        const int64_t at = (int64_t)min(m, a.M - 1) * a.N;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int n = col0 + 16 * b + 4 * c4;
            v[b] = base4{};
            if constexpr (BASE) {
                for (int s = 0; s < a.parts; ++s) {
                    const float* p = a.base + (int64_t)s * a.M * a.N + at + n;
                    floatx4 t = {};
                    if (n + 4 <= a.N) __builtin_memcpy(&t, p, 16);
                    else
                        for (int i = 0; n + i < a.N; ++i) t[i] = p[i];
                    v[b] += t;
                }
            } else {
                if (vec && n + 4 <= a.N) v[b] = *(const half4*)(a.C + at + n);
                else
                    for (int i = 0; i < 4; ++i)
                        if (n + i < a.N) v[b][i] = __builtin_bit_cast(_Float16, a.C[at + n + i]);
            }
        }
        floatx4 sum[NB];
        low.template block<SwappedMfma, 16, 32, NB, 2, SP>(sum, row0, col0, a.M, a.N);
        const bool none = low.adapter(m, a.M) < 0;
        if (m >= a.M || (!BASE && none)) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int n = col0 + 16 * b + 4 * c4;
            uint16_t* c = a.C + (size_t)m * a.N + n;
            half4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = (_Float16)((float)v[b][i] + (none ? 0.0f : sum[b][i]));
            if (vec && n + 4 <= a.N) {
                *(half4*)c = o;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.N) c[i] = __builtin_bit_cast(uint16_t, (_Float16)o[i]);
            }
        }
    }
#endif
}

// Any alignment and r: a thread an output (S == 1).
template <bool BASE>
__global__ __launch_bounds__(256) void lora_up_any_kernel(LoraArgs a)
{
    const int64_t total = (int64_t)a.M * a.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int m = (int)(i / a.N), n = (int)(i % a.N), id = a.ids[m];
        const bool some = (unsigned)id < (unsigned)a.L;
        float c = 0.0f;
        if constexpr (BASE) {
            for (int s = 0; s < a.parts; ++s) c += a.base[s * total + i];
        } else {
            if (!some) continue;
            c = f16_bits_to_f32(a.C[i]);
        }
        if (some) {
            const float* h = a.H + (size_t)m * a.r;
            const uint16_t* u = a.Up + ((size_t)id * a.N + n) * a.r;
            float s = 0.0f;
            for (int j = 0; j < a.r; ++j) s = __builtin_fmaf(h[j], f16_bits_to_f32(u[j]), s);
            c += s;
        }
        a.C[i] = f32_to_f16_bits(c);
    }
}

// ---------------------------------------------------------------------------
// base and adapters, tiles
// ---------------------------------------------------------------------------

struct LoraTileArgs : GemmArgs {
    LowRank low;
    static constexpr bool LOW_RANK = true;
};

template <class Cfg>
hipError_t launch_lora_tile(LoraTileArgs a, hipStream_t stream)
{
    auto kern = gemm_nt_kernel<Cfg, EPI_F16, true, LoraTileArgs>;
    static std::atomic<uint64_t> lds_opt_in{0};
    const hipError_t e = opt_in_lds((const void*)kern, Cfg::LDS_BYTES, lds_opt_in, stream);
    if (e != hipSuccess) return e;
    a.slices = 1;
    a.kt_per_slice = ceil_div(a.K, Cfg::BK) + 1;
    const int64_t tiles = (int64_t)ceil_div(a.M, Cfg::BM) * ceil_div(a.N, Cfg::BN);
    hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(Cfg::NT), Cfg::LDS_BYTES, stream, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// base and adapters, one or two rows: B in vectors
// ---------------------------------------------------------------------------
//
// The MFMA operand holds 16 rows of A whatever M is; for a handful of rows B streams
// faster in vectors.  A wave takes a row of B at a time (a workgroup WAVES
// neighbouring ones, then those a grid further), its lanes the 16-byte chunks l, l +
// 64, .., UNROLL of them in flight beside the next step's, against A in LDS (rows past
// M, and chunks past K, zeros).  The rows' sums wait in LDS for H: the Up rows of the
// workgroup's columns come there by direct loads while B streams, and are met at the
// end by a thread an output.
// SELF: no launch before this one: every workgroup works out H itself, the ranks of
// Down as further rows, which come through L2; else H comes in a.S parts.
// K % 8 == 0, r % 8 == 0; A, B, Down and Up 16-byte aligned; M <= MV.
__host__ __device__ constexpr int lora_vec_pad(int K, int unroll) { return ceil_div(K / 8, kWave * unroll) * kWave * unroll; }

struct LoraVecLds {
    int a, h, sums, up, total;
    __host__ __device__ LoraVecLds(int MV, int K, int r, int unroll, int rows, int most)
    {
        a = 0;
        h = a + MV * lora_vec_pad(K, unroll) * 16;
        sums = h + MV * r * 4;
        up = (sums + rows * MV * 4 + 15) / 16 * 16;
        total = up + ceil_div(most * rows * r * 2, 1024) * 1024;   // in whole loads
    }
};

template <int MV, int UNROLL, int WAVES, bool SELF>
__global__ __launch_bounds__(WAVES * kWave) void lora_vec_kernel(LoraArgs a, int iters, int most)
{
#if defined(__HIP_DEVICE_COMPILE__)
    extern __shared__ __attribute__((aligned(1024))) char smem_raw[];
    __shared__ int lead[MV], slot_of[MV];                // adapters in use; which of them a row has
    __shared__ float scale_of[MV];
    constexpr int STEP = kWave * UNROLL;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int M = a.M, N = a.N, K = a.K, r = a.r;
    const int nch = K / 8, spg = ceil_div(nch, STEP), npad = spg * STEP;
    const bool ragged = npad != nch;
    const int rows = iters * WAVES, n0 = blockIdx.x * WAVES, nstep = gridDim.x * WAVES;
    const LoraVecLds at(MV, K, r, UNROLL, rows, most);
    GF_LDS char* smem = (GF_LDS char*)smem_raw;
    GF_LDS half8* as = (GF_LDS half8*)(smem + at.a);     // [MV][npad]
    GF_LDS float* H = (GF_LDS float*)(smem + at.h);      // [MV][r]
    GF_LDS float* sums = (GF_LDS float*)(smem + at.sums);// [rows][MV]
    GF_LDS uint16_t* up = (GF_LDS uint16_t*)(smem + at.up);   // [adapter][rows][r]

    const int mine = n0 + wave < N ? (N - n0 - wave + nstep - 1) / nstep : 0;   // this wave's rows of B
    const int nb = mine * spg;
    auto load_row = [&](const uint16_t* row, int i, half8 (&b)[UNROLL]) __attribute__((always_inline)) {
        const int c0 = (i % spg) * STEP + lane;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) b[u] = *((const half8*)row + min(c0 + u * kWave, nch - 1));
    };
    auto row_of = [&](int i) __attribute__((always_inline)) -> const uint16_t* {
        const int g = i / spg;
        if (!SELF || g < mine) return a.B + (size_t)(n0 + wave + g * nstep) * K;
        const int t = wave + (g - mine) * WAVES;         // a rank of an adapter
        return a.Down + ((size_t)lead[t / r] * r + t % r) * K;
    };
    half8 buf[2][UNROLL];
    if (nb > 0) load_row(a.B + (size_t)(n0 + wave) * K, 0, buf[0]);   // B's bytes are on their way first
    for (int j = threadIdx.x; j < MV * npad; j += WAVES * kWave) {
        const int m = j / npad, c = j - m * npad;
        as[j] = m < M && c < nch ? ((const half8*)a.A)[(size_t)m * nch + c] : half8{};
    }
    int nd = 0;
#pragma unroll
    for (int m = 0; m < MV; ++m) {
        const int id = m < M ? scalar_load(a.ids + min(m, M - 1)) : -1;
        int s = -1;
        if ((unsigned)id < (unsigned)a.L) {
#pragma unroll
            for (int p = 0; p < m; ++p)
                if (s < 0 && p < M && scalar_load(a.ids + p) == id) s = slot_of[p];
            if (s < 0) {
                s = nd++;
                if (threadIdx.x == 0) lead[s] = id;
            }
        }
        // every thread writes the same; a row is looked up again by later ones above
        slot_of[m] = s;
        if ((int)threadIdx.x == m) scale_of[m] = s >= 0 && a.scales ? a.scales[id] : 1.0f;
    }
    if constexpr (!SELF)
        for (int i = threadIdx.x; i < M * r; i += WAVES * kWave) {
            float s = a.H[i];
            for (int p = 1; p < a.S; ++p) s += a.H[p * a.part + i];
            H[i] = s;
        }
    __syncthreads();
    {
        const int per = r / 8, total = nd * rows * per;  // chunks of 8 ranks
        for (int c0 = wave * kWave; c0 < total; c0 += WAVES * kWave) {
            const int c = c0 + lane, row = c / per % rows, d = c / (per * rows);
            const int n = n0 + row % WAVES + row / WAVES * nstep;
            const void* p = (const void*)g_zero16;
            if (c < total && n < N) p = a.Up + ((size_t)lead[d] * N + n) * r + c % per * 8;
            __builtin_amdgcn_global_load_lds(p, (GF_LDS void*)(up + c0 * 8), 16, 0, 0);
        }
    }
    const int ranks = SELF ? nd * r : 0;
    const int ntasks = nb + (wave < ranks ? (ranks - wave + WAVES - 1) / WAVES : 0) * spg;
    if (nb == 0 && ntasks > 0) load_row(row_of(0), 0, buf[0]);

    float acc[MV];
#pragma unroll
    for (int m = 0; m < MV; ++m) acc[m] = 0.0f;
    auto load = [&](int i, half8 (&b)[UNROLL]) __attribute__((always_inline)) { load_row(row_of(i), i, b); };
    auto compute = [&](int i, half8 (&b)[UNROLL]) __attribute__((always_inline)) {
        const int c0 = (i % spg) * STEP + lane;
        if (ragged && i % spg == spg - 1) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if (c0 + u * kWave >= nch) b[u] = half8{};
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int m = 0; m < MV; ++m) acc[m] = dot8(b[u], as[m * npad + c0 + u * kWave], acc[m]);
        if (i % spg == spg - 1) {
            const int g = i / spg;
#pragma unroll
            for (int m = 0; m < MV; ++m) {
                const float s = wave_sum(acc[m]);
                acc[m] = 0.0f;
                if (lane != m) continue;
                if (!SELF || g < mine) {
                    sums[(g * WAVES + wave) * MV + m] = s;
                } else {
                    const int t = wave + (g - mine) * WAVES;
                    if (slot_of[m] == t / r) H[m * r + t % r] = scale_of[m] * s;
                }
            }
        }
    };
    int i = 0;
    for (; i + 2 < ntasks; i += 2) {                     // tasks i + 1 and i + 2 exist
        load(i + 1, buf[1]);
        __builtin_amdgcn_sched_barrier(0);               // the loads leave before the multiply waits
        compute(i, buf[0]);
        load(i + 2, buf[0]);
        __builtin_amdgcn_sched_barrier(0);
        compute(i + 1, buf[1]);
    }
    if (i + 1 < ntasks) {
        load(i + 1, buf[1]);
        compute(i, buf[0]);
        compute(i + 1, buf[1]);
    } else if (i < ntasks) {
        compute(i, buf[0]);
    }
    wait_vmcnt<0>();                                     // this wave's Up rows have landed
    __syncthreads();
    for (int t = threadIdx.x; t < rows * M; t += WAVES * kWave) {
        const int m = t / rows, row = t % rows, n = n0 + row % WAVES + row / WAVES * nstep;
        if (n >= N) continue;
        float s = sums[row * MV + m];
        if (slot_of[m] >= 0) {
            const GF_LDS half8* u = (const GF_LDS half8*)(up + (slot_of[m] * rows + row) * r);
            for (int j = 0; j < r; j += 8) {
                const half8 v = u[j / 8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s = __builtin_fmaf(H[m * r + j + e], (float)v[e], s);
            }
        }
        a.C[(size_t)m * N + n] = f32_to_f16_bits(s);
    }
#endif
}

template <int MV, int UNROLL, int WAVES, bool SELF>
hipError_t launch_lora_vec(const LoraArgs& a, int grid, int iters, int most, int lds, hipStream_t stream)
{
    auto kern = lora_vec_kernel<MV, UNROLL, WAVES, SELF>;
    static std::atomic<uint64_t> lds_opt_in{0};
    const hipError_t e = opt_in_lds((const void*)kern, 159 * 1024, lds_opt_in, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(WAVES * kWave), lds, stream, a, iters, most);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// base and adapters, few rows: stream B
// ---------------------------------------------------------------------------
//
// Bound by B's bytes and those of the adapters in use.  A workgroup (one to a CU)
// walks the 16-row blocks of B grid-stride, its 8 waves split K in tasks of 128 k:
// 16 rows of 256 bytes by direct loads of whole cache lines, RING tasks in flight a
// wave, read from LDS as MFMA operands (chunk c of row n at slot c ^ n: the 16 rows
// read together lie in different banks).  Each wave keeps its part of A in
// registers (XB tasks' worth).  After a row block's K come its adapters' tasks, in
// the same ring so that their bytes stream too: up to four units, each the 16 rows'
// 32 ranks of Up of one adapter, dealt over the waves; H lies in LDS and enters as
// in low_rank.hpp.  The waves' sums are added in wave order.  Every step loads a task,
// past the last one zeros, so that the loads in flight, and each wait, are constant.
//
// SELF: no launch before this one: every workgroup works out H itself, with Down's
// ranks, 16 at a time, in registers beside its first row block's bytes in LDS.  Down
// then comes through L2 to every workgroup, so it is for few adapters of low rank.
// K % 8 == 0, r % 8 == 0, N >= 16; A, B, Down and Up 16-byte aligned; M <= 16 * MB;
// K <= 1024 * XB.
template <int MB_, int XB_, int RING_>
struct LoraBandCfg {
    static constexpr int MB = MB_, XB = XB_, RING = RING_, WAVES = 8, BK = 128, LOADS = 4, TASK_BYTES = 4096;
    static constexpr int ROWS = 16 * MB;
    static constexpr int RED_BYTES = 2 * WAVES * ROWS * 16 * 4;
    // the rings, the waves' sums, the adapters in use and their rows, the largest of H's rows
    // and their scales, H's parts in whole loads
    static constexpr int lds_bytes(int h_floats)
    {
        return WAVES * RING * TASK_BYTES + RED_BYTES + 4 * ROWS * 4 + ceil_div(h_floats * 4, 1024) * 1024;
    }
};

template <class Cfg, bool SELF>
__global__ __launch_bounds__(Cfg::WAVES * 64) void lora_band_kernel(LoraArgs a, int te)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int MB = Cfg::MB, XB = Cfg::XB, RING = Cfg::RING, WAVES = Cfg::WAVES, L = Cfg::LOADS, MR = Cfg::ROWS;
    extern __shared__ __attribute__((aligned(1024))) char smem_raw[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, c4 = lane / 16;
    const int M = a.M, N = a.N, K = a.K, r = a.r;
    GF_LDS char* tasks = (GF_LDS char*)smem_raw + wave * RING * Cfg::TASK_BYTES;
    GF_LDS float* red = (GF_LDS float*)((GF_LDS char*)smem_raw + WAVES * RING * Cfg::TASK_BYTES);
    GF_LDS int* used = (GF_LDS int*)((GF_LDS char*)red + Cfg::RED_BYTES);
    GF_LDS uint32_t* rows_of = (GF_LDS uint32_t*)(used + MR);
    GF_LDS int* most_of = (GF_LDS int*)(rows_of + MR);   // the largest magnitude of each row of H
    GF_LDS float* back = (GF_LDS float*)(most_of + MR);  // what its scaled sums are multiplied by
    GF_LDS float* H = back + MR;                         // S x M x r; then, 4 ranks to 16 bytes, their fp16 pairs

    if (threadIdx.x < MR) most_of[threadIdx.x] = 0;      // (a barrier before the first pack())
    const int nblk = ceil_div(K, Cfg::BK);
    const int b0 = wave * nblk / WAVES, nk = (wave + 1) * nblk / WAVES - b0;   // this wave's tasks of K
    const int blocks = ceil_div(N, 16), part = blockIdx.x, parts = gridDim.x;
    const int nq = (blocks - part + parts - 1) / parts;
    const int id = a.ids[min(lane, M - 1)];

    const int rk = ceil_div(r, 32);              // units of an adapter
    int nd = 0;                                  // adapters in use, in the order of their first rows
    auto find_used = [&]() __attribute__((always_inline)) {   // every wave finds the same
        uint64_t left = __ballot(lane < M && (unsigned)id < (unsigned)a.L);
        while (left) {
            const int v = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
            const uint64_t rows = left & __ballot(id == v);
            left &= ~rows;
            if (lane == 0) {
                used[nd] = v;
                rows_of[nd] = (uint32_t)rows;
            }
            ++nd;
        }
        asm volatile("" ::: "memory");
        wait_lgkmcnt0();
    };

    uint32_t boff[4];                            // direct loads' sources
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + c4;
        boff[i] = (uint32_t)row * (uint32_t)K + (uint32_t)(r16 ^ row) * 8u;
    }
    int iq = 0, ib = 0, islot = 0;               // the next task to issue
    auto next_slot = [&]() __attribute__((always_inline)) {
        if (++islot == RING) islot = 0;
    };
    auto issue_k = [&]() __attribute__((always_inline)) {
        GF_LDS char* buf = tasks + islot * Cfg::TASK_BYTES;
        const int k0 = (b0 + ib) * Cfg::BK;
        const uint16_t* src = a.B + (size_t)min((part + iq * parts) * 16, N - 16) * K + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const void* p = src + boff[i];
            if (k0 + (r16 ^ (4 * i + c4)) * 8 >= K || iq >= nq) p = (const void*)g_zero16;
            __builtin_amdgcn_global_load_lds(p, (GF_LDS void*)(buf + i * 1024), 16, 0, 2);
        }
    };
    auto issue = [&]() __attribute__((always_inline)) {
        if (ib < nk) {
            issue_k();
        } else {
            // unit u: lane l loads chunk l % 4 of row l / 4
            GF_LDS char* buf = tasks + islot * Cfg::TASK_BYTES;
            const int n0 = min((part + iq * parts) * 16, N - 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int u = ((ib - nk) * 4 + i) * WAVES + wave;
                const void* p = (const void*)g_zero16;
                if (u < nd * rk && iq < nq) {
                    const int k = u % rk * 32 + lane % 4 * 8;
                    if (k < r) p = a.Up + ((size_t)used[u / rk] * N + n0 + lane / 4) * r + k;
                }
                __builtin_amdgcn_global_load_lds(p, (GF_LDS void*)(buf + i * 1024), 16, 0, 0);
            }
        }
        if (++ib == nk + te) { ib = 0; ++iq; }
        next_slot();
    };
    if (nk >= RING) {                            // B's bytes are on their way before the ids are looked at
        static_for<RING>([&](auto) __attribute__((always_inline)) { issue_k(); ++ib; next_slot(); });
        find_used();
    } else {
        find_used();
        static_for<RING>([&](auto) __attribute__((always_inline)) { issue(); });
    }
    const int units = nd * rk;

    half8 x[XB * 4][MB];                         // zeros past M, past K, and past this wave's K
#pragma unroll
    for (int b = 0; b < XB * 4; ++b)
#pragma unroll
        for (int m = 0; m < MB; ++m) x[b][m] = half8{};
#pragma unroll
    for (int m = 0; m < MB; ++m)
        if (16 * m + r16 < M) {
            const uint16_t* src = a.A + (size_t)(16 * m + r16) * K;
#pragma unroll
            for (int b = 0; b < XB * 4; ++b) {
                const int k = b0 * Cfg::BK + 32 * b + 8 * c4;
                x[b][m] = *(const half8*)(k < K && b < 4 * nk ? (const void*)(src + k) : (const void*)g_zero16);
            }
        }
    // H's parts to LDS, then each value as a scaled pair of fp16 in its place (low_rank.hpp):
    // the parts' sums and each row's largest, a barrier, the pairs.
    auto pack = [&](int parts) __attribute__((always_inline)) {
        for (int i = threadIdx.x * 4; i < M * r; i += WAVES * kWave * 4) {
            floatx4 v = *(const GF_LDS floatx4*)(H + i);
            for (int p = 1; p < parts; ++p) v += *(const GF_LDS floatx4*)(H + p * M * r + i);
            *(GF_LDS floatx4*)(H + i) = v;
            float most = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) most = LowRank::larger(most, v[e]);
            // magnitudes are ordered as integers, in whichever order they come
            __hip_atomic_fetch_max(&most_of[i / r], __builtin_bit_cast(int, most), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        lds_barrier();
        for (int i = threadIdx.x * 4; i < M * r; i += WAVES * kWave * 4) {
            const floatx4 v = *(const GF_LDS floatx4*)(H + i);
            const int m = i / r;
            const LowRank::Scale scale(__builtin_bit_cast(float, most_of[m]));
            half8 pair;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                _Float16 hi, lo;
                LowRank::split(v[e] * scale.up, hi, lo);
                pair[e] = hi;
                pair[e + 4] = lo;
            }
            *(GF_LDS half8*)(H + i) = pair;
            if (i == m * r) back[m] = scale.down;
        }
        lds_barrier();
    };
    if constexpr (!SELF) {
        const int total = a.S * M * r;                   // a multiple of 4
        for (int i = wave * 256; i < total; i += WAVES * 256) {
            const int at = i + lane * 4, p = at / (M * r);
            const void* src = at < total ? (const void*)(a.H + p * a.part + (at - p * M * r)) : (const void*)g_zero16;
            __builtin_amdgcn_global_load_lds(src, (GF_LDS void*)(H + i), 16, 0, 0);
        }
        wait_vmcnt<0>();
        lds_barrier();
        pack(a.S);
    }

    // SELF: this wave's K of 16 ranks of Down, block q of ranks (the last block of an
    // adapter is its last 16; with r = 8 they are there twice).
    const int rb = ceil_div(r, 16), nh = SELF ? nd * rb : 0;
    auto rank0 = [&](int q) __attribute__((always_inline)) { return max(min(q % rb * 16, r - 16), 0); };
    half8 down[SELF ? XB * 4 : 1];
    auto load_down = [&](int q) __attribute__((always_inline)) {
        const int j = rank0(q) + (r < 16 ? r16 & 7 : r16);
        const uint16_t* src = a.Down + ((size_t)__builtin_amdgcn_readfirstlane(used[q / rb]) * r + j) * K;
#pragma unroll
        for (int b = 0; b < XB * 4; ++b) {
            const int k = b0 * Cfg::BK + 32 * b + 8 * c4;
            down[b] = *(const half8*)(k < K && b < 4 * nk ? (const void*)(src + k) : (const void*)g_zero16);
        }
    };
    if constexpr (SELF)
        if (nh > 0) load_down(0);

    int slot = 0, side = 0;
    // The waves' sums, row by row of 16 columns, handed to f(index, sum).
    auto reduce = [&](const floatx4 (&acc)[MB], auto f) __attribute__((always_inline)) {
        GF_LDS float* mine = red + side * WAVES * MR * 16;
        side ^= 1;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * m + 4 * c4 + i;
                if (row < M) mine[(wave * MR + row) * 16 + r16] = acc[m][i];
            }
        lds_barrier();
        for (int t = threadIdx.x; t < M * 16; t += WAVES * kWave) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) s += mine[w * MR * 16 + t];
            f(t, s);
        }
    };
    for (int q = 0; q < nq; ++q) {
        floatx4 acc[MB] = {};
        auto next = [&]() __attribute__((always_inline)) {
            asm volatile("" ::: "memory");
            wait_lgkmcnt0();                      // the buffer is read: it may be filled again
            issue();
            if (++slot == RING) slot = 0;
        };
        static_for<XB>([&](auto b_c) __attribute__((always_inline)) {
            constexpr int b = decltype(b_c)::value;
            if (b < nk) {
                wait_vmcnt<(RING - 1) * L>();
                asm volatile("" ::: "memory");
                const GF_LDS char* buf = tasks + slot * Cfg::TASK_BYTES;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const half8 w = *(const GF_LDS half8*)(buf + r16 * 256 + (((4 * i + c4) ^ r16) * 16));
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[b * 4 + i][m], w, acc[m], 0, 0, 0);
                }
                next();
            }
        });
        if constexpr (SELF) {
            for (int h = 0; q == 0 && h < nh; ++h) {
                const int ad = __builtin_amdgcn_readfirstlane(used[h / rb]), j0 = rank0(h);
                const uint32_t mask = rows_of[h / rb];
                const float scale = a.scales ? scalar_load(a.scales + ad) : 1.0f;
                floatx4 sum[MB] = {};
#pragma unroll
                for (int b = 0; b < XB * 4; ++b)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[b][m], down[b], sum[m], 0, 0, 0);
                if (h + 1 < nh) load_down(h + 1);
                reduce(sum, [&](int t, float s) {
                    if (((mask >> (t / 16)) & 1) && t % 16 < r) H[t / 16 * r + j0 + t % 16] = scale * s;
                });
            }
            if (q == 0) {
                lds_barrier();                    // H is whole
                pack(1);
            }
        }
        for (int t = 0; t < te; ++t) {
            wait_vmcnt<(RING - 1) * L>();
            asm volatile("" ::: "memory");
            const GF_LDS char* buf = tasks + slot * Cfg::TASK_BYTES;
            for (int i = 0; i < 4; ++i) {
                const int u = (t * 4 + i) * WAVES + wave;
                if (u >= units) break;
                const int k = u % rk * 32 + 8 * c4;
                const uint32_t mask = __builtin_amdgcn_readfirstlane(rows_of[u / rk]);
                const half8 w = *(const GF_LDS half8*)(buf + i * 1024 + r16 * 64 + c4 * 16), w1 = LowRank::finite(w);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    if (((mask >> (16 * m)) & 0xFFFF) == 0) continue;
                    const GF_LDS half8* h = (const GF_LDS half8*)(H + min(16 * m + r16, M - 1) * r + k);
                    half8 p = {}, q = {};
                    if (k < r) {
                        p = h[0];
                        q = h[1];
                    }
                    const floatx4 f = *(const GF_LDS floatx4*)(back + 16 * m + 4 * c4);
                    floatx4 t = {};
                    t = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_shufflevector(p, q, 0, 1, 2, 3, 8, 9, 10, 11), w, t, 0, 0, 0);
                    t = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_shufflevector(p, q, 4, 5, 6, 7, 12, 13, 14, 15), w1, t, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][e] += (mask >> (16 * m + 4 * c4 + e)) & 1 ? t[e] * f[e] : 0.0f;
                }
            }
            next();
        }
        const int n0 = min((part + q * parts) * 16, N - 16);
        reduce(acc, [&](int t, float s) { a.C[(size_t)(t / 16) * N + n0 + t % 16] = f32_to_f16_bits(s); });
    }
    wait_vmcnt<0>();
#endif
}

template <class Cfg, bool SELF>
hipError_t launch_lora_band(const LoraArgs& a, hipStream_t stream)
{
    auto kern = lora_band_kernel<Cfg, SELF>;
    const int most = a.M < a.L ? a.M : a.L;      // adapters in use
    const int te = ceil_div(ceil_div(most * ceil_div(a.r, 32), Cfg::WAVES), 4);
    const int lds = Cfg::lds_bytes((SELF ? 1 : a.S) * a.M * a.r);
    static std::atomic<uint64_t> lds_opt_in{0};
    const hipError_t e = opt_in_lds((const void*)kern, 160 * 1024, lds_opt_in, stream);
    if (e != hipSuccess) return e;
    const int blocks = ceil_div(a.N, 16);
    hipLaunchKernelGGL(kern, dim3(blocks < 256 ? blocks : 256), dim3(Cfg::WAVES * kWave), lds, stream, a, te);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// base and adapters, a decode batch: K in slices
// ---------------------------------------------------------------------------
//
// The streaming form above has every CU read all of A (7 us for 32 rows of 4096, at 40
// GB/s a CU), and the products by Down are a launch of their own.  Here a workgroup has
// one slice of 512 k: its part of A (16 KB for 16 rows) in LDS, its waves taking 16-row
// blocks of B, and 16 ranks of Down at a time like any of them, through a ring of tasks
// as above.  A slice's sums go to memory, part by part; a second launch adds the parts
// and the adapters, and rounds once.  The parts are M / 128 of B's bytes, written and
// read again.  32 rows of 24 adapters at 4096 x 4096, rank 16: 19.2 us, 11.5 of them the
// first launch (2.9 TB/s) and 7 the second, a chain of three loads with 13 adapters
// for 16 rows; the base alone takes 12, the streaming form with the adapters 22.
// K % 8 == 0, r % 8 == 0, N >= 16; A, B, Down and Up 16-byte aligned; M <= 16 * MB.
constexpr int kLoraSlice = 512, kLoraSlices = 8;

template <int MB_, int W_>
struct LoraSliceCfg {
    static constexpr int MB = MB_, W = W_, RING = 2, T = 4, SLICE = kLoraSlice, ROWS = 16 * MB, TASK_BYTES = 4096;
    static constexpr int X_BYTES = ROWS * SLICE * 2, LDS_BYTES = X_BYTES + W * RING * TASK_BYTES;
    static_assert(SLICE == 128 * T);
    static_assert(LDS_BYTES <= 80 * 1024, "two workgroups to a CU");
};

// P: slices x M x N, the base's parts; a.H: slices x M x r, no more slices than
// kLoraSlices.  hb: blocks of ranks there
// can be (the launch takes them first), per: blocks a wave, parts: workgroups a slice.
template <class Cfg>
__global__ __launch_bounds__(Cfg::W * kWave) void lora_slice_kernel(LoraArgs a, float* P, int hb, int per, int parts)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int MB = Cfg::MB, W = Cfg::W, RING = Cfg::RING, T = Cfg::T, L = 4;
    extern __shared__ __attribute__((aligned(1024))) char smem_raw[];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, c4 = lane / 16;
    const int M = a.M, N = a.N, K = a.K, r = a.r;
    const int slice = blockIdx.x / parts, part = blockIdx.x % parts, k0 = slice * Cfg::SLICE;
    GF_LDS char* xs = (GF_LDS char*)smem_raw;                // row m: 64 chunks, c at slot c ^ (m % 16)
    GF_LDS char* tasks = xs + Cfg::X_BYTES + wave * RING * Cfg::TASK_BYTES;
    const int id = a.ids[min(lane, M - 1)];
    for (int m = wave; m < Cfg::ROWS; m += W) {
        const int k = k0 + (lane ^ (m % 16)) * 8;
        const void* p = m < M && k < K ? (const void*)(a.A + (size_t)m * K + k) : (const void*)g_zero16;
        __builtin_amdgcn_global_load_lds(p, (GF_LDS void*)(xs + m * 1024), 16, 0, 0);
    }
    const int rb = ceil_div(r, 16), blocks = hb + ceil_div(N, 16);
    const uint64_t live = __ballot(lane < M && (unsigned)id < (unsigned)a.L);
    // The rows of the d-th adapter in use, 0 past the last.
    auto rows_of = [&](int d) __attribute__((always_inline)) {
        uint64_t left = live, rows = 0;
        for (int i = 0; i <= d && left; ++i) {
            rows = left & __ballot(id == __builtin_amdgcn_readlane(id, __builtin_ctzll(left)));
            left &= ~rows;
            if (i < d) rows = 0;
        }
        return rows;
    };
    auto rank0 = [&](int b) __attribute__((always_inline)) { return max(min(b % rb * 16, r - 16), 0); };
    auto block_of = [&](int i) __attribute__((always_inline)) { return (i * parts + part) * W + wave; };

    const uint16_t* src = nullptr;               // of the block whose tasks are being issued
    int ii = 0, it = 0, islot = 0, wrap = 15;
    auto issue = [&]() __attribute__((always_inline)) {
        if (it == 0) {
            const int b = ii < per ? block_of(ii) : blocks;
            src = nullptr;
            wrap = 15;
            if (b < hb) {
                const uint64_t rows = rows_of(b / rb);
                if (rows) {
                    src = a.Down + ((size_t)__builtin_amdgcn_readlane(id, __builtin_ctzll(rows)) * r + rank0(b)) * K;
                    wrap = r < 16 ? 7 : 15;      // rank 8: its ranks are there twice
                }
            } else if (b < blocks) {
                src = a.B + (size_t)min((b - hb) * 16, N - 16) * K;
            }
        }
        GF_LDS char* buf = tasks + islot * Cfg::TASK_BYTES;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * i + c4, k = k0 + it * 128 + (r16 ^ row) * 8;
            const void* p = src && k < K ? (const void*)(src + (size_t)(row & wrap) * K + k) : (const void*)g_zero16;
            __builtin_amdgcn_global_load_lds(p, (GF_LDS void*)(buf + i * 1024), 16, 0, 2);
        }
        if (++it == T) { it = 0; ++ii; }
        if (++islot == RING) islot = 0;
    };
    static_for<RING>([&](auto) __attribute__((always_inline)) { issue(); });
    wait_vmcnt<RING * L>();                      // this wave's rows of A are there
    lds_barrier();                               // everyone's
    int slot = 0;
    for (int i = 0; i < per; ++i) {
        const int b = block_of(i);
        floatx4 acc[MB] = {};
        static_for<T>([&](auto t_c) __attribute__((always_inline)) {
            constexpr int t = decltype(t_c)::value;
            wait_vmcnt<(RING - 1) * L>();
            asm volatile("" ::: "memory");
            const GF_LDS char* buf = tasks + slot * Cfg::TASK_BYTES;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const half8 w = *(const GF_LDS half8*)(buf + r16 * 256 + (((4 * s + c4) ^ r16) * 16));
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const half8 x = *(const GF_LDS half8*)(xs + (16 * m + r16) * 1024 + (((16 * t + 4 * s + c4) ^ r16) * 16));
                    acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, w, acc[m], 0, 0, 0);
                }
            }
            asm volatile("" ::: "memory");
            wait_lgkmcnt0();                     // the buffer is read: it may be filled again
            issue();
            if (++slot == RING) slot = 0;
        });
        if (b >= blocks) break;
        // accumulator e of lane l: row 4 * (l / 16) + e, column l % 16
        if (b < hb) {
            const uint64_t rows = rows_of(b / rb);
            if (!rows) continue;
            const int ad = __builtin_amdgcn_readlane(id, __builtin_ctzll(rows));
            const float scale = a.scales ? scalar_load(a.scales + ad) : 1.0f;
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 16 * m + 4 * c4 + e;
                    if (((rows >> row) & 1) && r16 < r)
                        a.H[slice * a.part + (size_t)row * r + rank0(b) + r16] = scale * acc[m][e];
                }
        } else {
            float* out = P + ((size_t)slice * M) * N + min((b - hb) * 16, N - 16) + r16;
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 16 * m + 4 * c4 + e;
                    if (row < M) out[(size_t)row * N] = acc[m][e];
                }
        }
    }
    wait_vmcnt<0>();
#endif
}

// C = the parts' sum and the adapters: 16 rows by 16 columns, J waves each.
template <int J>
__global__ __launch_bounds__(256) void lora_finish_kernel(LoraArgs a, const float* P, int vec)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = threadIdx.x % kWave, r16 = lane % 16, c4 = lane / 16;
    const int across = ceil_div(a.N, 16), down = ceil_div(a.M, 16);
    const int nth = (int)(blockIdx.x * 4 + threadIdx.x / kWave) / J;
    const int w = __builtin_amdgcn_readfirstlane(min(nth, across * down - 1));
    const int row0 = w / across * 16, col0 = min(w % across * 16, a.N - 16);
    const int m = row0 + r16;
    const float* p = P + (size_t)min(m, a.M - 1) * a.N + col0 + 4 * c4;
    const size_t part = (size_t)a.M * a.N;
    floatx4 v[kLoraSlices], base = {}, sum[1];   // all parts in flight, added in order
#pragma unroll
    for (int s = 0; s < kLoraSlices; ++s)
        if (threadIdx.x / kWave % J == 0) __builtin_memcpy(&v[s], p + min(s, a.S - 1) * part, 16);
    if (!lora_join<J, kLoraSlices>(a.low(), sum, row0, col0, a.M, a.N)) return;
#pragma unroll
    for (int s = 0; s < kLoraSlices; ++s)
        if (s < a.S) base += v[s];
    if (nth >= across * down || m >= a.M) return;
    uint16_t* c = a.C + (size_t)m * a.N + col0 + 4 * c4;
    typedef _Float16 half4 __attribute__((ext_vector_type(4)));
    half4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (_Float16)(base[i] + sum[0][i]);
    if (vec) {
        *(half4*)c = o;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = __builtin_bit_cast(uint16_t, (_Float16)o[i]);
    }
#endif
}

template <class Cfg>
hipError_t launch_lora_slices(const LoraArgs& a, float* P, hipStream_t stream)
{
    auto kern = lora_slice_kernel<Cfg>;
    static std::atomic<uint64_t> lds_opt_in{0};
    hipError_t e = opt_in_lds((const void*)kern, Cfg::LDS_BYTES, lds_opt_in, stream);
    if (e != hipSuccess) return e;
    const int most = a.M < a.L ? a.M : a.L, hb = most * ceil_div(a.r, 16), blocks = hb + ceil_div(a.N, 16);
    // about two workgroups to a CU, each wave with the same number of blocks
    int per = (int)((int64_t)blocks * a.S / (512 * Cfg::W));
    if (per < 1) per = 1;
    const int parts = ceil_div(blocks, Cfg::W * per);
    hipLaunchKernelGGL(kern, dim3(parts * a.S), dim3(Cfg::W * kWave), Cfg::LDS_BYTES, stream, a, P, hb, per, parts);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int items = ceil_div(a.M, 16) * ceil_div(a.N, 16);
    const int vec = (reinterpret_cast<uintptr_t>(a.C) & 7) == 0 && a.N % 4 == 0;
    if (a.r <= 32)
        hipLaunchKernelGGL(lora_finish_kernel<1>, dim3(ceil_div(items, 4)), dim3(256), 0, stream, a, P, vec);
    else if (a.r <= 64)
        hipLaunchKernelGGL(lora_finish_kernel<2>, dim3(ceil_div(items, 2)), dim3(256), 0, stream, a, P, vec);
    else
        hipLaunchKernelGGL(lora_finish_kernel<4>, dim3(items), dim3(256), 0, stream, a, P, vec);
    return hipGetLastError();
}

}  // namespace gf
