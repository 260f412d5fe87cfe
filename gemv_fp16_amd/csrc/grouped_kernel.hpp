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

// The groups, and what every kernel that walks them shares.
struct Groups {
    const int* offsets;   // E + 1 entries
    int E, T;

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
    template <int BM>
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
        if (w >= total) return false;
        const int L = xcd_remap(w, total);
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
struct GroupRowArgs : GemmArgs {
    Groups g;
    int c_bytes;          // of one element of C
    static constexpr bool PER_GROUP = true;

    template <int BM, int BN>
    __device__ __forceinline__ bool locate(int& tm, int& tn)
    {
        const int tiles_n = ceil_div(N, BN);
        int e, lo, hi, item;
        if (!g.find<BM>(blockIdx.x, tiles_n, e, lo, hi, item)) return false;
        M = hi - lo;
        A += (size_t)lo * K;
        B += (size_t)e * N * K;
        C = (char*)C + (size_t)lo * N * c_bytes;
        grouped_tile(item, ceil_div(M, BM), tiles_n, kGroupPanel, tm, tn);
        return true;
    }
};

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
        const int i = blockIdx.x / 8, e = i / run;
        const int t = (blockIdx.x % 8) * run + i % run;
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
    a.kt_per_slice = 1 << 24;                     // one slice: more K tiles than any contraction has
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(Cfg::NT), Cfg::LDS_BYTES, stream, a);
    return hipGetLastError();
}

}  // namespace gf
