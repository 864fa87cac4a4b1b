// Row tiles of the grouped products whose workgroups walk items of (m-tile,
// n-block), and the order of those items. Internal to libmoe.so.
#pragma once

#include "ffn_dev.h"

namespace moe {
namespace {

constexpr int kRowPanel = 4;   // m-tiles per item panel

// Sums over a wave by DPP moves: a shuffle through LDS takes some 100 cycles a level, a DPP move under ten.
// wave_scan: inclusive prefix sums; the total is lane 63's.
template <typename T, int kCtrl, int kRows>
__device__ __forceinline__ T dpp_or_zero(T v) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, kRows, 0xf, false));
}
template <typename T>
__device__ __forceinline__ T wave_scan(T v) {
    v += dpp_or_zero<T, 0x111, 0xf>(v);  // row_shr 1, 2, 4, 8: within 16 lanes
    v += dpp_or_zero<T, 0x112, 0xf>(v);
    v += dpp_or_zero<T, 0x114, 0xf>(v);
    v += dpp_or_zero<T, 0x118, 0xf>(v);
    v += dpp_or_zero<T, 0x142, 0xa>(v);  // lane 15 to the next 16, in the second and fourth
    v += dpp_or_zero<T, 0x143, 0xc>(v);  // lane 31 to the upper 32
    return v;
}
template <typename T>
__device__ __forceinline__ T wave_total(T v) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wave_scan(v)), 63));
}

// Tiles and rows of the groups, built by every workgroup once from the
// device-resident offsets: first tile (tile_start) and first row (row0, clamped
// to the buffer) of each group. A group's nt = ceil(m / height) tiles split its
// m rows evenly. Looked up from LDS alone, since every item's start waits for it.
template <int kGroups>
struct RowTiles {
    int tile_start[kGroups + 1];
    int row0[kGroups + 1];
    int sums[3];
};

// first tile of each group for tiles of h rows, and their number; the first wave's work, row0 must be there
template <int kGroups>
__device__ __forceinline__ void number_tiles(RowTiles<kGroups>& tm, int n_groups, int h) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (wave == 0) {  // 64 groups at a time
        int run = 0;
        for (int g0 = 0; g0 < n_groups; g0 += 64) {
            const int g = g0 + lane;
            const int nt = g < n_groups ? max(0, tm.row0[g + 1] - tm.row0[g] + h - 1) / h : 0;
            const int sum = wave_scan(nt);
            if (g < n_groups) tm.tile_start[g] = run + sum - nt;
            run += __builtin_amdgcn_readlane(sum, 63);
        }
        if (lane == 0) tm.tile_start[n_groups] = run;
    }
}

// the same for tiles of at most h rows, from the offsets; all kThreads threads call, returns the number of tiles
template <int kThreads, int kGroups>
__device__ __forceinline__ int even_tiles(RowTiles<kGroups>& tm, const int32_t* __restrict__ offsets, int n_groups,
                                          int max_rows, int h) {
    for (int g = threadIdx.x; g <= n_groups; g += kThreads) tm.row0[g] = clamp_row(offsets[g], max_rows);
    __syncthreads();
    number_tiles(tm, n_groups, h);
    __syncthreads();
    return tm.tile_start[n_groups];
}

// All kThreads threads call (it holds barriers); returns the number of tiles. The height
// is kTile rows, or half or a quarter of it where all items then still run at once: a call so
// small takes as long as its tallest tile (MXFP4, nine groups of 17 rows and one of 203
// at H = 1280, I = 384: gate/up 14.2 us with one tile of 203 rows, 10.0 with four).
template <int kThreads, int kTile, int kGroups>
__device__ __forceinline__ int build_row_tiles(RowTiles<kGroups>& tm, const int32_t* __restrict__ offsets,
                                               int n_groups, int max_rows, int NB) {
    for (int g = threadIdx.x; g <= n_groups; g += kThreads) tm.row0[g] = clamp_row(offsets[g], max_rows);
    __syncthreads();
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int height = kTile >> wave;  // waves 0 to 2 count tiles of the whole, half and a quarter of the height
    auto tiles_of = [&](int g, int h) {
        return g < n_groups ? max(0, tm.row0[g + 1] - tm.row0[g] + h - 1) / h : 0;
    };
    if (wave < 3) {
        int sum = 0;
        for (int g = lane; g < n_groups; g += 64) sum += tiles_of(g, height);
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
        if (lane == 0) tm.sums[wave] = sum;
    }
    __syncthreads();
    const int h = tm.sums[2] <= (int)gridDim.x / NB ? kTile / 4 : tm.sums[1] <= (int)gridDim.x / NB ? kTile / 2 : kTile;
    number_tiles(tm, n_groups, h);
    __syncthreads();
    return tm.tile_start[n_groups];
}

// Item -> tile and n-block, in panels of kRowPanel m-tiles of a group (the last
// one may be shorter): all n-blocks of a panel, its m-tiles fastest, so the
// workgroups of one XCD share both operands' slices of a K step through L2.
template <int kGroups>
__device__ __forceinline__ MTile row_item_at(const RowTiles<kGroups>& tm, int n_groups, int item, int NB, int& nb) {
    const int mt = item / NB;
    int lo = 0, hi = n_groups - 1;  // the group: the last g with tile_start[g] <= mt
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tm.tile_start[mid] <= mt) lo = mid;
        else hi = mid - 1;
    }
    const int t0 = __builtin_amdgcn_readfirstlane(tm.tile_start[lo]);
    const int nt = __builtin_amdgcn_readfirstlane(tm.tile_start[lo + 1]) - t0;
    const int r0 = __builtin_amdgcn_readfirstlane(tm.row0[lo]);
    const int m = __builtin_amdgcn_readfirstlane(tm.row0[lo + 1]) - r0;
    const int local = item - t0 * NB;
    const int pi = local / (kRowPanel * NB);  // never past the last panel
    const int ph = min(kRowPanel, nt - pi * kRowPanel);
    const int idx = local - pi * kRowPanel * NB;
    nb = idx / ph;
    const int i = pi * kRowPanel + idx - nb * ph;
    const int each = m / nt, more = m - each * nt;  // the first `more` tiles hold one row more
    return MTile{__builtin_amdgcn_readfirstlane(lo), r0 + i * each + min(i, more), each + (i < more ? 1 : 0)};
}

// weight row (within the wave's 32) that MFMA row rho reads: lane (l31, hi)
// then holds the D values of 16 consecutive weight rows 16 hi + [0, 16), so
// it writes 16 neighbouring outputs
__device__ __forceinline__ int mx_row_of(int rho) { return 16 * ((rho >> 2) & 1) + 4 * (rho >> 3) + (rho & 3); }

}  // namespace
}  // namespace moe
