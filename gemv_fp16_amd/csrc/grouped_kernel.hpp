// Products grouped by expert, on the tiles of gemm_kernel.hpp.
//
// The T rows of A are sorted by group: group e owns rows offsets[e] ..
// offsets[e + 1] - 1 (device memory: the router's output never visits the
// host).
//  * By rows (forward product and input gradient): C[r] = A[r] . op(B[e]).
//    The number of tiles is known on the device only, so the launch holds the
//    most there can be (every group may end in a partial tile) and each
//    workgroup finds its group with a wave-wide scan over the groups' tile
//    counts; the workgroups past the last tile end at once.
//  * By depth (weight gradient): C[e] = A_e^T . B_e, the contraction over the
//    group's rows.  The tiles are known on the host, their depth is not.
// The workgroup narrows the operands to its group and runs the ordinary tile:
// rows past the group's end are clamped on load and masked on store, rows past
// the contraction's end read as zeros, and an empty contraction stores zeros.
#pragma once
#include "gemm_kernel.hpp"

namespace gf {

constexpr int kMaxExtent = 1 << 30;    // of each size: the kernels round sizes up in 32 bits
constexpr int kMaxGroups = 1 << 16;    // each workgroup looks through the groups

// A launch has fewer than 2^32 threads: one of 2^32 is refused, a larger one wraps.
// So work runs as launches of at most this many workgroups (of 512 threads or
// fewer), each told the number of its first.  A multiple of 8, so that the mapping
// to the XCDs goes on where the launch before ended.
constexpr int kMaxLaunch = 1 << 22;

template <class Launch>
hipError_t launch_in_parts(int64_t grid, Launch launch)
{
    for (int64_t first = 0; first < grid; first += kMaxLaunch) {
        const int64_t n = grid - first < kMaxLaunch ? grid - first : kMaxLaunch;
        const hipError_t e = launch((int)first, dim3((unsigned)n));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The groups, and what every kernel that walks them shares.
struct Groups {
    const int* offsets;   // E + 1 entries
    int E, T;
    int first;            // number of the launch's first workgroup

    __device__ __forceinline__ int workgroup() const { return first + (int)blockIdx.x; }

    // Rows of group e.  Entries outside 0 .. T and a group whose end comes
    // before its begin (both against the contract) still name no row outside A
    // and C.
    __device__ __forceinline__ void rows(int e, int& lo, int& hi) const
    {
        lo = min(max(offsets[e], 0), T);
        hi = max(min(offsets[e + 1], T), lo);
    }

    // The group and the tile within it of work item w, where a group of n rows
    // has ceil(n / BM) * per_block items; the items are dealt to the XCDs in
    // contiguous runs.  Every lane of the wave must call it; the results are
    // wave-uniform.  Returns false past the last item.
    // SHARE 0: all items.  1: those that fill whole rounds of 256 (all of them
    // where the last round is more than half full).  2: the rest, w / 4 (the
    // caller cuts each in four).
    template <int BM, int SHARE = 0>
    __device__ __forceinline__ bool find(int w, int per_block, int& e, int& lo, int& hi, int& item) const
    {
        const int lane = threadIdx.x % kWave;
        int l = 0, h = 0, total = 0, scan = 0, mine = 0;
        for (int base = 0; base < E; base += kWave) {
            l = h = 0;
            if (base + lane < E) rows(base + lane, l, h);
            mine = ceil_div(h - l, BM) * per_block;
            scan = mine;
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) {
                const int v = __shfl_up(scan, d);
                if (lane >= d) scan += v;
            }
            total += __builtin_amdgcn_readlane(scan, kWave - 1);
        }
        const int whole = total % 256 <= 128 ? total - total % 256 : total;
        int L;
        if constexpr (SHARE == 2) {
            L = whole + w / 4;
            if (L >= total) return false;
        } else {
            const int share = SHARE == 1 ? whole : total;
            if (w >= share) return false;
            L = xcd_remap(w, share);
        }
        int before = 0;
        for (int base = 0;; base += kWave) {
            if (E > kWave) {                       // else the first loop's one pass is still in registers
                l = h = 0;
                if (base + lane < E) rows(base + lane, l, h);
                mine = ceil_div(h - l, BM) * per_block;
                scan = mine;
#pragma unroll
                for (int d = 1; d < kWave; d *= 2) {
                    const int v = __shfl_up(scan, d);
                    if (lane >= d) scan += v;
                }
            }
            const uint64_t past = __ballot(before + scan > L);
            if (past) {
                const int src = __builtin_ctzll(past);
                e = base + src;
                lo = __builtin_amdgcn_readlane(l, src);
                hi = __builtin_amdgcn_readlane(h, src);
                const int n = __builtin_amdgcn_readlane(mine, src);
                item = L - before - (__builtin_amdgcn_readlane(scan, src) - n);
                return item >= 0 && item < n;      // false only where counts of overlapping groups wrapped
            }
            before += __builtin_amdgcn_readlane(scan, kWave - 1);
            if (base + kWave >= E) return false;   // not reached: L < total
        }
    }
};

constexpr int kGroupPanel = 8;   // tile-rows per raster panel within a group

// By rows.  M and C's rows are the group's; A, B, C point at its parts.
// SHARE 1 and 2: the launch in two parts of grouped.hip's run_rounds (1 with the
// whole tiles, 2 with tiles of half their side).
template <int SHARE>
struct GroupRowShare : GemmArgs {
    Groups g;
    static constexpr bool PER_GROUP = true;

    template <int BM, int BN>
    __device__ __forceinline__ bool locate(int& tm, int& tn)
    {
        constexpr int F = SHARE == 2 ? 2 : 1;             // tiles are F * BM x F * BN
        const int tiles_n = ceil_div(N, F * BN);
        int e, lo, hi, item;
        if (!g.find<F * BM, SHARE>(g.workgroup(), tiles_n, e, lo, hi, item)) return false;
        M = hi - lo;
        A += (size_t)lo * K;
        B += (size_t)e * N * K;
        C = (uint16_t*)C + (size_t)lo * N;
        grouped_tile(item, ceil_div(M, F * BM), tiles_n, kGroupPanel, tm, tn);
        if constexpr (SHARE == 2) {
            tm = 2 * tm + (blockIdx.x % 4) / 2;
            tn = 2 * tn + blockIdx.x % 2;
            return tm * BM < M && tn * BN < N;
        }
        return true;
    }
};
typedef GroupRowShare<0> GroupRowArgs;

// By depth.  C is E x M x N; K becomes the group's number of rows.
struct GroupDepthArgs : GemmArgs {
    Groups g;
    int c_bytes;
    static constexpr bool PER_GROUP = true;

    // Each group's tiles are cut into 8 runs, one for each XCD: a group much
    // deeper than the others then keeps all XCDs busy, not one.
    template <int BM, int BN>
    __host__ __device__ static int run_length(int M, int N)
    {
        return ceil_div(ceil_div(M, BM) * ceil_div(N, BN), 8);
    }

    template <int BM, int BN>
    __device__ __forceinline__ bool locate(int& tm, int& tn)
    {
        const int run = run_length<BM, BN>(M, N);
        const unsigned w = g.workgroup();
        const int i = w / 8, e = i / run;
        const int t = (w % 8) * run + i % run;
        const int tiles_m = ceil_div(M, BM), tiles_n = ceil_div(N, BN);
        if (t >= tiles_m * tiles_n) return false;
        int lo, hi;
        g.rows(e, lo, hi);
        K = hi - lo;
        A += (size_t)lo * M;
        B += (size_t)lo * N;
        C = (char*)C + (size_t)e * M * N * c_bytes;
        grouped_tile(t, tiles_m, tiles_n, kGroupPanel, tm, tn);
        return true;
    }
};

template <class Cfg, int EPI, bool ALIGNED, class Args>
hipError_t launch_grouped(Args a, int64_t grid, hipStream_t stream)
{
    auto kern = gemm_nt_kernel<Cfg, EPI, ALIGNED, Args>;
    static std::atomic<uint64_t> lds_opt_in{0};   // devices where the LDS size is opted into
    const hipError_t e = opt_in_lds((const void*)kern, Cfg::LDS_BYTES, lds_opt_in, stream);
    if (e != hipSuccess) return e;
    a.slices = 1;
    a.raster = 0;
    a.kt_per_slice = 1 << 26;                     // one slice: more K tiles than any contraction (2^30) has
    return launch_in_parts(grid, [&](int first, dim3 n) {
        a.g.first = first;
        hipLaunchKernelGGL(kern, n, dim3(Cfg::NT), Cfg::LDS_BYTES, stream, a);
        return hipGetLastError();
    });
}

// ---------------------------------------------------------------------------
// few rows a group: stream the weights
// ---------------------------------------------------------------------------
//
// C[r] = A[r] . B[e]^T where a group has a handful of rows: bound by B's bytes.
// For each 16 * MB rows of A of a group, `parts` workgroups walk the 16-row blocks
// of B[e] grid-stride (the last one is the last 16 rows, some a second time): a
// group with many rows has many workgroups, next to each other so that they share
// B in their L2.  A workgroup's 8 waves split K in tasks of 128 k; a task's 16 rows of
// 256 bytes go to LDS by direct loads of whole cache lines, `ring` tasks in
// flight a wave, and are read from there as MFMA operands (chunk c of row n at
// slot c ^ n: the 16 rows read together lie in different banks).  Each wave keeps
// its part of A in registers (XB tasks' worth), so nothing else is loaded in the
// loop and no wave waits for another's loads.  Each row block ends in one
// barrier; the waves' sums are added in wave order, in slots that alternate.
// k past K: A's registers hold zeros, B's chunks are read from 16 zero bytes.
// K % 8 == 0, N >= 16, A and B 16-byte aligned.
// 16 groups of 4096 x 2048, 48 rows over 14 of them: 36 us, 6.5 TB/s of the 6.6
// that a plain read reaches (tiles: 57 us; what they measured is in grouped.hip).
template <int MB_, int XB_>
struct GroupBandCfg {
    static constexpr int MB = MB_, XB = XB_, WAVES = 8, BK = 128, LOADS = 4, TASK_BYTES = 4096, MAX_RING = 4;
    static constexpr int RED_BYTES = 2 * WAVES * 16 * MB * 16 * 4;
    static constexpr int lds_bytes(int ring) { return WAVES * ring * TASK_BYTES + RED_BYTES; }
};

template <class Cfg>
__global__ __launch_bounds__(Cfg::WAVES * 64) void group_band_kernel(GroupRowArgs a, int ring, int parts)
{
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int MB = Cfg::MB, XB = Cfg::XB, WAVES = Cfg::WAVES, L = Cfg::LOADS, MR = 16 * MB;
    extern __shared__ __attribute__((aligned(1024))) char smem_raw[];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane % 16, c4 = lane / 16;
    const int N = a.N, K = a.K;
    int e, lo, hi, item;
    if (!a.g.template find<MR>(a.g.workgroup(), parts, e, lo, hi, item)) return;
    const int passes = ceil_div(hi - lo, MR), part = item / passes;
    const int begin = lo + item % passes * MR, M = min(hi - begin, MR);
    const uint16_t* A = a.A + (size_t)begin * K;
    const uint16_t* B = a.B + (size_t)e * N * K;
    uint16_t* C = (uint16_t*)a.C + (size_t)begin * N;

    GF_LDS char* tasks = (GF_LDS char*)smem_raw + wave * ring * Cfg::TASK_BYTES;
    GF_LDS float* red = (GF_LDS float*)((GF_LDS char*)smem_raw + WAVES * ring * Cfg::TASK_BYTES);
    const int nblk = ceil_div(K, Cfg::BK);
    const int b0 = wave * nblk / WAVES, nb = (wave + 1) * nblk / WAVES - b0;   // this wave's tasks per row block
    const int blocks = ceil_div(N, 16);
    const int ng = (blocks - part + parts - 1) / parts;
    const int ntasks = ng * nb;

    uint32_t boff[4], bat[4];                             // direct loads' sources; operands' places
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + c4;
        boff[i] = (uint32_t)r * (uint32_t)K + (uint32_t)(r16 ^ r) * 8u;
        bat[i] = (uint32_t)(r16 * 256 + (((4 * i + c4) ^ r16) * 16));
    }
    int ig = part, ib = 0, islot = 0, issued = 0;     // the next task to issue
    auto issue = [&]() __attribute__((always_inline)) {
        GF_LDS char* buf = tasks + islot * Cfg::TASK_BYTES;
        const int k0 = (b0 + ib) * Cfg::BK;
        const uint16_t* src = B + (size_t)min(ig * 16, N - 16) * K + k0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const void* p = src + boff[i];
            if (k0 + Cfg::BK > K && k0 + (r16 ^ (4 * i + c4)) * 8 >= K) p = (const void*)g_zero16;
            __builtin_amdgcn_global_load_lds(p, (GF_LDS void*)(buf + i * 1024), 16, 0, 2);
        }
        ++issued;
        if (++ib == nb) { ib = 0; ig += parts; }
        if (++islot == ring) islot = 0;
    };
    auto wait_tasks = [&](int left) __attribute__((always_inline)) {   // younger tasks that may be pending
        left = __builtin_amdgcn_readfirstlane(left);
        if (left >= 3) wait_vmcnt<3 * L>();
        else if (left == 2) wait_vmcnt<2 * L>();
        else if (left == 1) wait_vmcnt<L>();
        else wait_vmcnt<0>();
    };
    const int first = min(ring, ntasks);
    for (int i = 0; i < first; ++i) issue();
    half8 x[XB * 4][MB];
#pragma unroll
    for (int b = 0; b < XB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const int k = (b0 + b) * Cfg::BK + 32 * i + 8 * c4;
                const half8 v = *(const half8*)(A + (size_t)min(16 * m + r16, M - 1) * K + min(k, K - 8));
                x[b * 4 + i][m] = k < K ? v : half8{};
            }

    int done = 0, slot = 0;
    for (int gi = 0; gi < ng; ++gi) {
        floatx4 acc[MB] = {};
        static_for<XB>([&](auto b_c) __attribute__((always_inline)) {
            constexpr int b = decltype(b_c)::value;
            if (b < nb) {
                wait_tasks(issued - done - 1);
                asm volatile("" ::: "memory");
                const GF_LDS char* buf = tasks + slot * Cfg::TASK_BYTES;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const half8 w = *(const GF_LDS half8*)(buf + bat[i]);
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[b * 4 + i][m], w, acc[m], 0, 0, 0);
                }
                asm volatile("" ::: "memory");
                wait_lgkmcnt0();                      // the buffer is read: it may be filled again
                if (issued < ntasks) issue();
                ++done;
                if (++slot == ring) slot = 0;
            }
        });
        GF_LDS float* mine = red + (gi & 1) * WAVES * MR * 16;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * m + 4 * c4 + i;
                if (row < M) mine[(wave * MR + row) * 16 + r16] = acc[m][i];
            }
        lds_barrier();
        const int n0 = min((part + gi * parts) * 16, N - 16);
        for (int t = threadIdx.x; t < M * 16; t += WAVES * kWave) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) s += mine[w * MR * 16 + t];
            C[(size_t)(t / 16) * N + n0 + t % 16] = f32_to_f16_bits(s);
        }
    }
    wait_vmcnt<0>();
#endif
}

template <class Cfg>
hipError_t launch_group_band(GroupRowArgs a, int ring, int parts, int64_t grid, hipStream_t stream)
{
    auto kern = group_band_kernel<Cfg>;
    static std::atomic<uint64_t> lds_opt_in{0};
    const int lds = Cfg::lds_bytes(ring);
    static_assert(Cfg::lds_bytes(Cfg::MAX_RING) <= 160 * 1024, "one CU's LDS");
    const hipError_t e = opt_in_lds((const void*)kern, Cfg::lds_bytes(Cfg::MAX_RING), lds_opt_in, stream);
    if (e != hipSuccess) return e;
    return launch_in_parts(grid, [&](int first, dim3 n) {
        a.g.first = first;
        hipLaunchKernelGGL(kern, n, dim3(Cfg::WAVES * kWave), lds, stream, a, ring, parts);
        return hipGetLastError();
    });
}

}  // namespace gf
