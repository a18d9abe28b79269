// What the kernels of more than one of the other files share: element types,
// loads of any alignment, the search of the group a row tile belongs to, loads
// straight into LDS, and the rounding to 8 bits.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
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
// and add up their tiles with a scan over the lanes. Sums stop at the most tiles
// that nondecreasing offsets give, so that decreasing ones, whose groups can hold
// all rows each, do not pass what an int holds.
template <typename Pick>
__device__ __forceinline__ bool find_tile(const int *offsets, int groups, int rows, int bm,
                                          Pick pick, int &g_out, int &lo_out, int &n_out,
                                          int &m_out)
{
    const int lane = __lane_id();
    const unsigned per = ((unsigned)groups + 63u) >> 6;
    const int g0 = (int)min(lane * per, (unsigned)groups);
    const int g1 = (int)min(g0 + per, (unsigned)groups);
    const int most = rows / bm + min(groups, rows);
    int tiles = 0;
    for (int g = g0; g < g1; ++g) {
        int lo, hi;
        group_rows(offsets, g, rows, lo, hi);
        tiles = min(tiles + (hi - lo + bm - 1) / bm, most);
    }
    int upto = tiles; // tiles of lanes 0..lane
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d)
            upto = min(upto + v, most);
    }
    const int slot = pick(__builtin_amdgcn_readlane(upto, 63));
    int before = __shfl_up(upto, 1);
    if (lane == 0)
        before = 0;
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

constexpr float kLeastScale = 1.17549435e-38f; // 2^-126

// The integer nearest to x / s (ties to even), |x / s| < 127.5. r, from a
// product with the reciprocal, can be one off next to a tie; d = x - r s is
// exact (for r = 0 it is x, for r = +-1 the subtraction of numbers within a
// factor of two, or, for x just below s / 2, one that rounds to no less than
// s / 2; beyond that a multiple of s's last place below 2^24 of them), and so is
// 2 d, so comparing that with s puts r right. (s / 2 would not be exact: from
// 2^-126 to 2^-125 half of an odd last place is no number.)
__device__ __forceinline__ int quantize_one(float x, float s, float inv)
{
    float r = __builtin_rintf(x * inv);
    const float d = __builtin_fmaf(-r, s, x);
    const float twice = 2.0f * __builtin_fabsf(d);
    const bool odd = ((int)r) & 1;
    if (twice > s || (twice == s && odd))
        r += d > 0.0f ? 1.0f : -1.0f;
    return (int)r;
}

// The 16 bytes of a chunk as floats.
template <typename T>
__device__ __forceinline__ void unpack(i32x4 v, float (&x)[16 / sizeof(T)])
{
    constexpr int VEC = 16 / sizeof(T);
    typedef T tv __attribute__((ext_vector_type(VEC)));
    const tv h = __builtin_bit_cast(tv, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        x[i] = (float)h[i];
}

template <typename F>
__device__ __forceinline__ void with_type(int type, F f)
{
    if (type == SGEMM_F32)
        f(float{});
    else if (type == SGEMM_F16)
        f(_Float16{});
    else
        f(__bf16{});
}

// Four neighbouring outputs at any address.
template <typename T>
__device__ __forceinline__ void store4(T *c, f32x4 x)
{
    typedef T t4 __attribute__((ext_vector_type(4)));
    const t4 h = {(T)x[0], (T)x[1], (T)x[2], (T)x[3]};
    if constexpr (sizeof(T) == 4)
        store16(c, __builtin_bit_cast(i32x4, h));
    else
        *reinterpret_cast<i32x2_any *>(c) = __builtin_bit_cast(i32x2, h);
}

// 16 bytes of a row from its byte k on, zeros from byte K on; nothing outside
// the row's K bytes is read. The chunk that K ends in comes from the row's last
// 16 bytes, moved down.
__device__ __forceinline__ i32x4 row_chunk(const signed char *row, int k, int K)
{
    if (k + 16 <= K)
        return load16(row + k);
    if (k >= K)
        return i32x4{0, 0, 0, 0};
    if (K >= 16) {
        const int n = k + 16 - K; // 1 to 15 bytes down
        i32x4 v = load16(row + K - 16);
        if (n & 4)
            v = i32x4{v[1], v[2], v[3], 0};
        if (n & 8)
            v = i32x4{v[2], v[3], 0, 0};
        return i32x4{(int)__builtin_amdgcn_alignbyte(v[1], v[0], n & 3),
                     (int)__builtin_amdgcn_alignbyte(v[2], v[1], n & 3),
                     (int)__builtin_amdgcn_alignbyte(v[3], v[2], n & 3),
                     (int)__builtin_amdgcn_alignbyte(0, v[3], n & 3)};
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (k + i < K)
            w[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
    return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// The 16 bytes of a row of K 4-bit elements from its byte k on (row_chunk), without
// what the last byte of an odd K holds beyond it. (Whole chunks first: a lane that
// clears has to wait for what it has loaded.)
__device__ __forceinline__ i32x4 mx4_chunk(const signed char *row, int k, int K)
{
    if (k + 16 <= K >> 1)
        return load16(row + k);
    i32x4 v = row_chunk(row, k, (K + 1) >> 1);
    const int last = (K >> 1) - k; // the byte that an odd K ends in
    if ((K & 1) && last >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i == last >> 2)
                v[i] &= ~(0xf0 << (8 * (last & 3)));
    }
    return v;
}

constexpr uint32_t kOutside = 0x80000000u;
constexpr int kMaxTileLd = 1 << 22;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const signed char *base, long long bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<signed char *>(base), (short)0,
                                             (int)(bytes < 0x7fffffff ? bytes : 0x7fffffff),
                                             0x00020000);
}

// vmcnt <= N, lgkmcnt and expcnt as they are.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// All waves meet: N of this wave's memory operations may still be under way,
// its LDS reads are done.
template <int N>
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    wait_loads<N>();
    __builtin_amdgcn_s_waitcnt(0xc07f); // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

inline int current_cus(int *out)
{
    static std::atomic<int> cache[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return (int)e;
    const bool cached = dev >= 0 && dev < 64;
    int cus = cached ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (cus == 0) {
        e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
        if (e != hipSuccess)
            return (int)e;
        if (cached)
            cache[dev].store(cus, std::memory_order_relaxed);
    }
    *out = cus;
    return 0;
}

// Whether a launch holds `tiles` workgroups: fewer than 2^32 work-items.
inline bool fits_launch(double tiles, int threads) { return tiles * threads <= 4294967295.0; }

inline bool c_type_ok(int type) { return type == SGEMM_F32 || type == SGEMM_F16 || type == SGEMM_BF16; }

} // namespace
