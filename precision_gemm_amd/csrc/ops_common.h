// What the kernels of i8gemm.hip and experts.hip share: element types, loads
// of any alignment, and the search of the group a row tile belongs to.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>
#include "sgemm.h"

namespace {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Vectors at any address: one global_load_dwordx4 or store each (the hardware
// takes unaligned addresses, at a lower rate).
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef int i32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef int i32_any __attribute__((aligned(1)));

__device__ __forceinline__ i32x4 load16(const void *p)
{
    return *static_cast<const i32x4_any *>(p);
}

__device__ __forceinline__ void store16(void *p, i32x4 v)
{
    *static_cast<i32x4_any *>(p) = v;
}

__host__ __device__ __forceinline__ int type_bytes(int type)
{
    return type == SGEMM_F32 ? 4 : type == SGEMM_I8 ? 1 : 2;
}

// A group's rows [lo, hi), brought into [0, rows] whatever the device array
// holds.
__device__ __forceinline__ void group_rows(const int *offsets, int g, int rows, int &lo, int &hi)
{
    lo = min(max(offsets[g], 0), rows);
    hi = min(max(offsets[g + 1], lo), rows);
}

// A tile of a grouped product. Row tiles of `bm` rows are counted group by
// group; `pick` is told how many there are and returns the number of the one
// wanted, or -1 for none. Every lane of the wave returns the same group, its
// first row and row count, and the tile's first row within the group; false if
// there is no such tile. A wave's lanes take groups/64 consecutive groups each
// and add up their tiles with a scan over the lanes.
template <typename Pick>
__device__ __forceinline__ bool find_tile(const int *offsets, int groups, int rows, int bm,
                                          Pick pick, int &g_out, int &lo_out, int &n_out,
                                          int &m_out)
{
    const int lane = __lane_id();
    const unsigned per = ((unsigned)groups + 63u) >> 6;
    const int g0 = (int)min(lane * per, (unsigned)groups);
    const int g1 = (int)min(g0 + per, (unsigned)groups);
    int tiles = 0;
    for (int g = g0; g < g1; ++g) {
        int lo, hi;
        group_rows(offsets, g, rows, lo, hi);
        tiles += (hi - lo + bm - 1) / bm;
    }
    int upto = tiles; // tiles of lanes 0..lane
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d)
            upto += v;
    }
    const int slot = pick(__builtin_amdgcn_readlane(upto, 63));
    const int before = upto - tiles;
    const bool mine = slot >= before && slot < upto;
    const unsigned long long who = __ballot(mine);
    if (who == 0)
        return false;
    int g_at = 0, lo_at = 0, n_at = 0, m_at = 0;
    if (mine) {
        int left = slot - before;
        for (int g = g0; g < g1; ++g) {
            int lo, hi;
            group_rows(offsets, g, rows, lo, hi);
            const int t = (hi - lo + bm - 1) / bm;
            if (left < t) {
                g_at = g;
                lo_at = lo;
                n_at = hi - lo;
                m_at = left * bm;
                break;
            }
            left -= t;
        }
    }
    const int src = __builtin_ctzll(who);
    g_out = __builtin_amdgcn_readlane(g_at, src);
    lo_out = __builtin_amdgcn_readlane(lo_at, src);
    n_out = __builtin_amdgcn_readlane(n_at, src);
    m_out = __builtin_amdgcn_readlane(m_at, src);
    return true;
}

// The group that is `nth` by its number of rows, the most first (equal ones in
// their order); at most 64 groups, one a lane.
__device__ __forceinline__ int group_by_size(const int *offsets, int groups, int rows, int nth)
{
    const int lane = __lane_id();
    int lo = 0, hi = -1; // (lanes without a group come last)
    if (lane < groups)
        group_rows(offsets, lane, rows, lo, hi);
    const int own = hi - lo;
    int before = 0;
    for (int i = 0; i < groups; ++i) {
        const int n = __builtin_amdgcn_readlane(own, i);
        before += n > own || (n == own && i < lane);
    }
    return __builtin_ctzll(__ballot(lane < groups && before == nth));
}

// Workgroup -> (row tile, column tile) of `tiles_m` x `tiles_n`, or false for
// one too many: consecutive workgroups go round the 8 XCDs, each of which gets
// a contiguous run of the tiles, ordered in bands of `band` row tiles so that
// the rows and weights in use stay in its L2.
__device__ __forceinline__ bool tile_order(int tiles_m, int tiles_n, int band, int &tm, int &tn)
{
    const int num = tiles_m * tiles_n, pid = blockIdx.x;
    const int xcd = pid & 7, local = pid >> 3, q = num >> 3, r = num & 7;
    if (local >= q + (xcd < r))
        return false;
    const int at = xcd < r ? xcd * (q + 1) + local : r * (q + 1) + (xcd - r) * q + local;
    const int each = band * tiles_n, first = at / each * band;
    const int rows = min(tiles_m - first, band);
    tm = first + at % each % rows;
    tn = at % each / rows;
    return true;
}

// Most row tiles that `groups` groups over `rows` rows can have.
inline long long most_tiles(int rows, int groups, int bm)
{
    return rows / bm + (groups < rows ? groups : rows);
}

// Every workgroup reads all offsets to find its tile, so the groups' part of the
// work grows with their square.
constexpr int kMaxGroups = 65536;

// Row tiles of a band of the tile order: as many as a group has on average.
inline int group_band(long long rows, long long groups, int bm)
{
    const long long each = (rows + groups * (bm / 2)) / (groups * bm);
    return each < 1 ? 1 : each > 8 ? 8 : (int)each;
}

inline long long ceil_div_ll(long long a, long long b) { return (a + b - 1) / b; }

} // namespace
