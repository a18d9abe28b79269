// 8-bit integer products with a scale for each token and channel, and the row
// quantization that makes their left operand (i8gemm.h), for MI355X (gfx950).

#include "ops_common.h"

#include "i8gemm.h"

#include <type_traits>

namespace {

// ---------------------------------------------------------------------------
// Row quantization
// ---------------------------------------------------------------------------

// NT threads a row (below 256: 256 / NT rows a workgroup), which hold the row
// in registers, CH chunks of 16 bytes each, between its maximum and its
// rounding: one pass over memory. CH = 0: rows of any length, read twice.
// Bound by memory: 16384 x 4092 in fp32 takes 62 us (5.4 TB/s, a large copy's
// rate), 16384 x 4096 in bf16 40 us (5.1); 4 x 4096 takes 3.7 us, a launch and
// one trip to memory. Rows of up to 1 KiB share a wave or a part of one
// (1000000 x 40 fp16: 42 us, 315 with a wave each).
template <typename T, int NT, int CH>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
i8_quantize_kernel(int M, int K, const T *X, int ldx, signed char *Q, int ldq, float *scale)
{
    constexpr int VEC = 16 / sizeof(T);
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, WAVES = NT / 64;
    static_assert(NT <= 64 || ROWS == 1, "a row is a part of a wave, a wave or a workgroup");
    const int t = threadIdx.x % NT;
    const long long m = (long long)blockIdx.x * ROWS + threadIdx.x / NT;
    if (m >= M)
        return; // (all threads of a row, and with NT > 64 never)
    const T *x = X + m * ldx;
    signed char *q = Q + m * ldq;

    // |x| as ordered integers: the largest of them keeps NaN above infinity.
    uint32_t peak = 0;
    auto chunk = [&](int k, float (&f)[VEC]) {
        if (k + VEC <= K) {
            unpack<T>(load16(x + k), f);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                f[i] = k + i < K ? (float)x[k + i] : 0.0f;
        }
    };
    auto take = [&](const float (&f)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            peak = max(peak, __builtin_bit_cast(uint32_t, f[i]) & 0x7fffffffu);
    };
    float held[CH > 0 ? CH : 1][VEC];
    if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            chunk((c * NT + t) * VEC, held[c]);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            take(held[c]);
    } else {
        for (int k = t * VEC; k < K; k += NT * VEC) {
            float f[VEC];
            chunk(k, f);
            take(f);
        }
    }
#pragma unroll
    for (int d = 1; d < (NT < 64 ? NT : 64); d <<= 1)
        peak = max(peak, (uint32_t)__shfl_xor((int)peak, d));
    if constexpr (WAVES > 1) {
        __shared__ uint32_t peaks[WAVES];
        if ((t & 63) == 0)
            peaks[t >> 6] = peak;
        __syncthreads();
        peak = peaks[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
            peak = max(peak, peaks[w]);
    }
    const float top = __builtin_bit_cast(float, peak);
    const bool finite = peak < 0x7f800000u;
    const float s = finite ? __builtin_fmaxf(top / 127.0f, kLeastScale) : top;
    if (t == 0)
        scale[m] = s;
    const float inv = 1.0f / s;

    auto put = [&](int k, const float (&f)[VEC]) {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint32_t b = finite ? (uint32_t)quantize_one(f[i], s, inv) & 0xffu : 0u;
            w[i / 4] = i % 4 == 0 ? b : w[i / 4] | b << (8 * (i % 4));
        }
        if (k + VEC <= K) {
            if constexpr (VEC == 4)
                *reinterpret_cast<i32_any *>(q + k) = (int)w[0];
            else
                *reinterpret_cast<i32x2_any *>(q + k) = i32x2_any{(int)w[0], (int)w[1]};
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (k + i < K)
                    q[k + i] = (signed char)(w[i / 4] >> (8 * (i % 4)));
        }
    };
    if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * NT + t) * VEC;
            if (k < K)
                put(k, held[c]);
        }
    } else {
        for (int k = t * VEC; k < K; k += NT * VEC) {
            float f[VEC];
            chunk(k, f);
            put(k, f);
        }
    }
}

template <typename T>
int launch_quantize(int M, int K, const void *X, int ldx, signed char *Q, int ldq, float *scale,
                    hipStream_t s)
{
    constexpr int VEC = 16 / sizeof(T);
    typedef void (*Fn)(int, int, const T *, int, signed char *, int, float *);
    const long long chunks = ceil_div_ll(K, VEC);
    Fn fn;
    int threads = 256, rows = 1;
    if (chunks <= 8) {
        fn = i8_quantize_kernel<T, 8, 1>;
        rows = 32;
    } else if (chunks <= 16) {
        fn = i8_quantize_kernel<T, 16, 1>;
        rows = 16;
    } else if (chunks <= 32) {
        fn = i8_quantize_kernel<T, 32, 1>;
        rows = 8;
    } else if (chunks <= 64) {
        fn = i8_quantize_kernel<T, 64, 1>;
        rows = 4;
    } else if (chunks <= 256) {
        fn = i8_quantize_kernel<T, 64, 4>;
        rows = 4;
    } else if (chunks <= 512) {
        fn = i8_quantize_kernel<T, 256, 2>;
    } else if (chunks <= 1024) {
        fn = i8_quantize_kernel<T, 256, 4>;
    } else if (chunks <= 2048) {
        fn = i8_quantize_kernel<T, 256, 8>;
    } else if (chunks <= 8192) {
        fn = i8_quantize_kernel<T, 1024, 8>;
        threads = 1024;
    } else {
        fn = i8_quantize_kernel<T, 1024, 0>;
        threads = 1024;
    }
    // A launch holds fewer than 2^32 work-items.
    const long long most = (1 << 21) * (long long)rows;
    for (long long m0 = 0; m0 < M; m0 += most) {
        int n = (int)(M - m0 < most ? M - m0 : most);
        const T *x = static_cast<const T *>(X) + m0 * ldx;
        signed char *q = Q + m0 * ldq;
        float *sc = scale + m0;
        void *args[] = {&n, &K, &x, &ldx, &q, &ldq, &sc};
        const hipError_t e =
            hipLaunchKernel((const void *)fn, dim3((unsigned)ceil_div_ll(n, rows)), dim3(threads),
                            args, 0, s);
        if (e != hipSuccess)
            return (int)e;
    }
    return 0;
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------

struct I8Params {
    const signed char *A, *B;
    const float *sA, *sB, *bias;
    void *C;
    const int *offsets; // grouped calls: row ranges of the groups
    long long strideB;
    int M, N, K;
    int lda, ldb, ldc;
    int type;
    int groups;           // 0: one product
    int tiles_m, tiles_n; // the grid
    int band;             // row tiles of a band of the grid's order
};

// Where a workgroup stands: its group's operands and its rows [m0, M) of
// them, counted from the group's first row.
struct I8Tile {
    const signed char *A, *B;
    const float *sA, *sB, *bias;
    long long row0; // C's row of the group's first row
    int M, m0, n0;
};

template <int BM, int BN>
__device__ __forceinline__ bool i8_tile_of(const I8Params &p, I8Tile &t)
{
    int tm = 0, tn = 0;
    t.A = p.A;
    t.B = p.B;
    t.sA = p.sA;
    t.sB = p.sB;
    t.bias = p.bias;
    t.row0 = 0;
    t.M = p.M;
    if (p.groups == 0) {
        if (!tile_order(p.tiles_m, p.tiles_n, p.band, tm, tn))
            return false;
        t.m0 = tm * BM;
    } else {
        auto pick = [&](int tiles) {
            return tile_order(tiles, p.tiles_n, p.band, tm, tn) ? tm : -1;
        };
        int g, lo;
        if (!find_tile(p.offsets, p.groups, p.M, BM, pick, g, lo, t.M, t.m0))
            return false;
        t.row0 = lo;
        t.A += (long long)lo * p.lda;
        t.sA += lo;
        t.B += g * p.strideB;
        t.sB += (long long)g * p.N;
        if (t.bias)
            t.bias += (long long)g * p.N;
    }
    t.n0 = tn * BN;
    return true;
}

__device__ __forceinline__ void store_c(const I8Params &p, long long at, float v)
{
    with_type(p.type, [&](auto t) { static_cast<decltype(t) *>(p.C)[at] = (decltype(t))v; });
}

// One output: every kernel rounds in this order.
__device__ __forceinline__ float scaled(float acc, float sa, float sb, float bias)
{
    return __builtin_fmaf(acc * sa, sb, bias);
}

// The tile for every alignment: 64 T x 64 T of C by four waves, each one T x T
// accumulators of v_mfma_i32_32x32x32_i8 (lane l supplies 16 bytes of row
// l % 32 from k = 16 (l / 32) on; register v of lane l holds row 8 (v / 4) +
// 4 (l / 32) + v % 4, column l % 32). 64-byte K-steps go through registers to
// LDS, so any alignment and any K will do, and zeros behind K leave the sum as
// it is. LDS rows are 64 bytes, four of them one sweep of the 64 banks, so the
// 16-byte chunk index is XORed with row / 4 for conflict-free reads. Rows
// behind M or N repeat the last one and are not stored.
template <int T>
__global__ void __launch_bounds__(256) i8_tile_kernel(I8Params p)
{
    constexpr int BM = 64 * T, BN = 64 * T, BK = 64;
    __shared__ __attribute__((aligned(16))) signed char lds[2][2][BM * BK];
    I8Tile t;
    if (!i8_tile_of<BM, BN>(p, t))
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = tid >> 2, c = tid & 3;
    const signed char *ra[T], *rb[T];
#pragma unroll
    for (int x = 0; x < T; ++x) {
        ra[x] = t.A + (long long)min(t.m0 + 64 * x + r, t.M - 1) * p.lda;
        rb[x] = t.B + (long long)min(t.n0 + 64 * x + r, p.N - 1) * p.ldb;
    }
    const int at = r * BK + 16 * (c ^ ((r >> 2) & 3)); // (64 rows on: the same chunk)
    const int wm = 32 * T * (wave & 1), wn = 32 * T * (wave >> 1);

    i32x16 acc[T][T] = {};
    const int steps = (p.K + BK - 1) / BK;
    i32x4 va[T] = {}, vb[T] = {};
    auto load = [&](int k) {
#pragma unroll
        for (int x = 0; x < T; ++x) {
            va[x] = row_chunk(ra[x], k + 16 * c, p.K);
            vb[x] = row_chunk(rb[x], k + 16 * c, p.K);
        }
    };
    if (steps > 0)
        load(0);
    for (int s = 0; s < steps; ++s) {
        signed char *la = lds[s & 1][0], *lb = lds[s & 1][1];
#pragma unroll
        for (int x = 0; x < T; ++x) {
            *reinterpret_cast<i32x4 *>(la + at + 64 * BK * x) = va[x];
            *reinterpret_cast<i32x4 *>(lb + at + 64 * BK * x) = vb[x];
        }
        __syncthreads();
        if (s + 1 < steps)
            load((s + 1) * BK);
#pragma unroll
        for (int q = 0; q < BK / 32; ++q) {
            const int o = lane & 31, ch = 16 * ((2 * q + (lane >> 5)) ^ ((o >> 2) & 3));
            i32x4 fa[T], fb[T];
#pragma unroll
            for (int x = 0; x < T; ++x) {
                fa[x] = *reinterpret_cast<const i32x4 *>(la + (wm + 32 * x + o) * BK + ch);
                fb[x] = *reinterpret_cast<const i32x4 *>(lb + (wn + 32 * x + o) * BK + ch);
            }
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < T; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0,
                                                                      0, 0);
        }
        // (The next step writes the other stage, which every wave left before
        // this step's barrier.)
    }
    with_type(p.type, [&](auto type) {
        typedef decltype(type) C;
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int n = t.n0 + wn + 32 * j + (lane & 31);
            if (n >= p.N)
                continue;
            const float sb = t.sB[n], bias = t.bias ? t.bias[n] : 0.0f;
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int m = t.m0 + wm + 32 * i + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
                    if (m < t.M)
                        static_cast<C *>(p.C)[(t.row0 + m) * p.ldc + n] =
                            (C)scaled((float)acc[i][j][v], t.sA[m], sb, bias);
                }
        }
    });
}

// 16 bytes from any address by two aligned loads and a shift, for streams of
// unaligned rows, whose bytes come slowly by unaligned loads. Reads the aligned
// 16 bytes around the first and the last byte.
__device__ __forceinline__ i32x4 load16_shifted(const signed char *p)
{
    const uint32_t s = (uint32_t)(uintptr_t)p & 15u;
    const signed char *q = p - s;
    const i32x4 a = *reinterpret_cast<const i32x4 *>(q);
    const i32x4 b = *reinterpret_cast<const i32x4 *>(q + (s ? 16 : 0));
    int w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    if (s & 4)
#pragma unroll
        for (int i = 0; i < 7; ++i)
            w[i] = w[i + 1];
    if (s & 8)
#pragma unroll
        for (int i = 0; i < 5; ++i)
            w[i] = w[i + 2];
    i32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = (int)__builtin_amdgcn_alignbyte(w[i + 1], w[i], s & 3);
    return r;
}

// ---------------------------------------------------------------------------
// Few rows: the weights' bytes bound the call, so they go from memory straight
// into the matrix instructions' registers, once, and no LDS stage stands
// between. A workgroup owns 16 * NT channels and up to 16 * MT rows; its WAVES
// waves take every WAVES-th block of 64 * U of k, so all of a short K is in
// flight at once, and their exact integer sums are added in LDS.
// v_mfma_i32_16x16x64_i8: lane l supplies 16 bytes of row l % 16 from k =
// 16 (l / 16) on; register v of lane l holds row 4 (l / 16) + v, column l % 16.
// Rows behind the last repeat it and are not stored. ALIGNED: rows start on
// 16-byte boundaries; otherwise load16_shifted, inside the row (256 rows over
// 64 groups, N = 2048: K = 2048 46 us, K = 2047 84, by unaligned loads 141).
// ---------------------------------------------------------------------------
template <int MT, int NT, int WAVES, int U, bool ALIGNED>
__global__ void __launch_bounds__(64 * WAVES) i8_stream_kernel(I8Params p)
{
    constexpr int BM = 16 * MT, BN = 16 * NT;
    __shared__ int sums[WAVES][BM][BN];
    I8Tile t;
    if (!i8_tile_of<BM, BN>(p, t))
        return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, kq = 16 * (lane >> 4);
    const signed char *ra[MT], *rb[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        ra[i] = t.A + (long long)min(t.m0 + 16 * i + r, t.M - 1) * p.lda;
#pragma unroll
    for (int j = 0; j < NT; ++j)
        rb[j] = t.B + (long long)min(t.n0 + 16 * j + r, p.N - 1) * p.ldb;

    i32x4 acc[MT][NT] = {};
    auto products = [&](const i32x4 (&fa)[MT], const i32x4 (&fb)[NT]) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    };
    // A block at a row's end or, unaligned, its start.
    auto edge = [&](int k) {
        for (int q = k; q < p.K && q < k + 64 * U; q += 64) {
            i32x4 fb[NT], fa[MT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fb[j] = row_chunk(rb[j], q + kq, p.K);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                fa[i] = row_chunk(ra[i], q + kq, p.K);
            products(fa, fb);
        }
    };
    auto load = [&](const signed char *x) { return ALIGNED ? load16(x) : load16_shifted(x); };
    int k = wave * 64 * U;
    if (!ALIGNED && wave == 0) {
        edge(0);
        k = WAVES * 64 * U;
    }
    for (; k + 64 * U + (ALIGNED ? 0 : 16) <= p.K; k += WAVES * 64 * U) {
        i32x4 fb[U][NT], fa[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fb[u][j] = load(rb[j] + kq + k + 64 * u);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                fa[u][i] = load(ra[i] + kq + k + 64 * u);
#pragma unroll
        for (int u = 0; u < U; ++u)
            products(fa[u], fb[u]);
    }
    edge(k);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                sums[wave][16 * i + 4 * (lane >> 4) + v][16 * j + r] = acc[i][j][v];
    __syncthreads();
    const int rows = min(BM, t.M - t.m0);
    for (int e = tid; e < rows * BN; e += 64 * WAVES) {
        const int m = e / BN, n = t.n0 + e % BN;
        if (n >= p.N)
            continue;
        int sum = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            sum += sums[w][m][e % BN];
        store_c(p, (t.row0 + t.m0 + m) * p.ldc + n,
                scaled((float)sum, t.sA[t.m0 + m], t.sB[n], t.bias ? t.bias[n] : 0.0f));
    }
}

// ---------------------------------------------------------------------------
// Larger products: BM x BN of C by WAVES_M x WAVES_N waves, K in steps of 128
// bytes that go straight from memory to LDS (buffer_load_dwordx4 ... lds)
// through a ring of STAGES stages. Lane l of a load fills the l-th 16 bytes of
// a 1 KiB block, 8 rows of 128 bytes: whole cache lines, so half the requests
// of 64-byte steps (which measured the same on cached operands, and 577 us
// against 474 on 4096 x 4096 x 32768). LDS rows are 128 bytes, two of them one
// sweep of the 64 banks: the 16-byte chunk index is XORed with row / 2, on the
// memory side, for conflict-free reads. A lane whose chunk lies behind K
// fetches zeros from a 2^31 byte offset, outside the buffer. Loads are issued
// for steps past the last too (of zeros), so that the number in flight is the
// same at every wait. Needs 16-byte-aligned rows, K a multiple of 16 and
// leading dimensions below 2^22 (32-bit offsets within a tile).
//
// What bounds the 256 x 256 tile: power. 8192^3 runs at 2.37 POP/s (465 us; the
// library product of integers alone 470 on the same card; other cards 441 to
// 490), 4096 x 8192 x 4096 takes 126 us (131); the matrix units are busy 55 % of
// the cycles of a clock that stands at 1.8 GHz. Without its loads the loop takes
// 17 % less, without its LDS reads 18 %, and on operands of zeros 30 %. Eight
// waves of 128 x 64 each beat four of 128 x 128 (4001 x 8192 x 4096: 132 us
// against 144), whose outputs leave one wave a SIMD idle.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WAVES_M, int WAVES_N>
struct I8Core {
    static constexpr int BK = 128, KH = BK / 32, NW = WAVES_M * WAVES_N;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 32, TN = WN / 32;
    static constexpr int STAGE = (BM + BN) * BK;
    static constexpr int NA = BM * BK / 1024 / NW, NB = BN * BK / 1024 / NW; // blocks a wave loads
    static_assert(NA >= 1 && NB >= 1, "a wave loads of both operands");
    static constexpr int PATCH = 16 * WN * 4; // bytes of LDS a wave's outputs turn over in

    int lane, wave, wm, wn, chunk, o;
    int at[KH];
    // The operands that loads are issued of.
    const signed char *A, *B;
    long long bytesA, bytesB;
    int K;
    uint32_t offA[NA], offB[NB];
    i32x16 acc[TM][TN];
    i32x4 fa[2][TM], fb[2][TN]; // of k-groups by parity
    // What the outputs of the tile are scaled with: lane l holds the wave's
    // rows l and 64 + l, and the four columns that it stores.
    float sa[(WM + 63) / 64], sb[4], bias[4];

    __device__ __forceinline__ void init()
    {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        // (Waves that share a SIMD, four apart, lie above one another in M.)
        wm = (wave / WAVES_N) * WM;
        wn = (wave % WAVES_N) * WN;
        chunk = 16 * ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
        // This lane's 16 bytes of k-group q (32 bytes of the step) in row 32 i +
        // l % 32 of the wave's part; 32 rows on is a fixed distance.
        o = lane & 31;
#pragma unroll
        for (int q = 0; q < KH; ++q)
            at[q] = o * BK + 16 * ((2 * q + (lane >> 5)) ^ ((o >> 1) & 7));
    }

    __device__ __forceinline__ void operands(const I8Params &p, const I8Tile &t)
    {
        A = t.A + (long long)t.m0 * p.lda;
        B = t.B + (long long)t.n0 * p.ldb;
        bytesA = (long long)(t.M - t.m0 - 1) * p.lda + p.K;
        bytesB = (long long)(p.N - t.n0 - 1) * p.ldb + p.K;
        K = p.K;
        // (Rows behind the last repeat it; they are not stored.)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            offA[i] = (uint32_t)(min(8 * (wave + NW * i) + (lane >> 3), t.M - t.m0 - 1) * p.lda + chunk);
#pragma unroll
        for (int i = 0; i < NB; ++i)
            offB[i] = (uint32_t)(min(8 * (wave + NW * i) + (lane >> 3), p.N - t.n0 - 1) * p.ldb + chunk);
    }

    // The loads of a step into a stage; of zeros for a step past the last.
    __device__ __forceinline__ void issue(int step, signed char *to) const
    {
        typedef __attribute__((address_space(3))) void lds_void;
        const __amdgpu_buffer_rsrc_t rsA = rows_rsrc(A, bytesA), rsB = rows_rsrc(B, bytesB);
        const int k = step * BK;
        const uint32_t off = k + chunk < K ? 0u : kOutside;
#pragma unroll
        for (int i = 0; i < NA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsA, (lds_void *)(to + 1024 * (wave + NW * i)), 16, offA[i] | off, k, 0, 0);
#pragma unroll
        for (int i = 0; i < NB; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsB, (lds_void *)(to + BM * BK + 1024 * (wave + NW * i)), 16, offB[i] | off, k, 0,
                0);
    }

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = i32x16{};
    }

    __device__ __forceinline__ void read(const signed char *stage, int q)
    {
        const signed char *a = stage + wm * BK + at[q], *b = stage + (BM + wn) * BK + at[q];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[q & 1][i] = *reinterpret_cast<const i32x4 *>(a + 32 * BK * i);
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[q & 1][j] = *reinterpret_cast<const i32x4 *>(b + 32 * BK * j);
    }

    __device__ __forceinline__ void products(int q)
    {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[q & 1][i], fb[q & 1][j],
                                                                  acc[i][j], 0, 0, 0);
    }

    // All but the last k-group of the step in `stage` (whose first one is read).
    __device__ __forceinline__ void step_front(const signed char *stage)
    {
#pragma unroll
        for (int q = 0; q + 1 < KH; ++q) {
            read(stage, q + 1);
            products(q);
            __builtin_amdgcn_sched_group_barrier(0x100, TM + TN, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, TM * TN, 0);
        }
    }

    // The last k-group, with the first one of the next step's stage read and
    // the loads of step `ahead` issued under its products.
    __device__ __forceinline__ void step_back(const signed char *next, int ahead, signed char *to)
    {
        read(next, 0);
        issue(ahead, to);
        products(KH - 1);
        constexpr int GAP = TM * TN / (NA + NB) > 0 ? TM * TN / (NA + NB) : 1;
        __builtin_amdgcn_sched_group_barrier(0x100, TM + TN, 0);
#pragma unroll
        for (int i = 0; i < NA + NB; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, GAP, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, TM * TN, 0);
        __builtin_amdgcn_sched_barrier(0);
    }

    __device__ __forceinline__ int column() const { return wn + 4 * (lane % (WN / 4)); }

    __device__ __forceinline__ void load_scales(const I8Params &p, const I8Tile &t)
    {
#pragma unroll
        for (int x = 0; x < (WM + 63) / 64; ++x)
            sa[x] = t.sA[min(t.m0 + wm + 64 * x + lane, t.M - 1)];
        const int n = t.n0 + column();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sb[e] = t.sB[min(n + e, p.N - 1)];
            bias[e] = t.bias ? t.bias[min(n + e, p.N - 1)] : 0.0f;
        }
    }

    // The wave's outputs, 16 rows at a time through a patch of LDS of its own,
    // so that a row's leave as 16-byte (fp32) or 8-byte pieces. Rows 4 apart,
    // which one write instruction holds, are 32 banks apart by the XOR. EDGE:
    // the tile reaches past M or N.
    template <typename T, bool EDGE>
    __device__ __forceinline__ void turn_over(const I8Params &p, const I8Tile &t, float *patch) const
    {
        constexpr int PER = WN / 4, RPI = 64 / PER; // lanes a row, rows a store
        const int r = lane / PER, c = 4 * (lane % PER);
        const int n = t.n0 + wn + c;
        const int left = t.M - (t.m0 + wm); // the wave's rows
        T *out = static_cast<T *>(p.C) + (t.row0 + t.m0 + wm + r) * p.ldc + n;
        const long long step = (long long)RPI * p.ldc;
#pragma unroll
        for (int h = 0; h < 2 * TM; ++h) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const int row = 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    patch[(row * WN + 32 * j + o) ^ (8 * (row & 4))] =
                        (float)acc[h / 2][j][8 * (h & 1) + v];
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += RPI) {
                const int row = r0 + r, m = 16 * h + row;
                f32x4 x = *reinterpret_cast<const f32x4 *>(
                    patch + ((row * WN + c) ^ (8 * (row & 4))));
                const float s = __shfl(sa[(16 * h + r0) / 64], m & 63);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = scaled(x[e], s, sb[e], bias[e]);
                if (!EDGE || (m < left && n + 4 <= p.N)) {
                    store4(out, x);
                } else if (m < left) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < p.N)
                            out[e] = (T)x[e];
                }
                out += step;
            }
            __builtin_amdgcn_wave_barrier();
        }
    }

    __device__ __forceinline__ void outputs(const I8Params &p, const I8Tile &t, float *patch) const
    {
        const bool whole = t.m0 + BM <= t.M && t.n0 + BN <= p.N;
        with_type(p.type, [&](auto type) {
            if (whole)
                turn_over<decltype(type), false>(p, t, patch);
            else
                turn_over<decltype(type), true>(p, t, patch);
        });
    }
};

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES>
__device__ __forceinline__ void i8_large_tile(const I8Params &p, signed char *lds)
{
    typedef I8Core<BM, BN, WAVES_M, WAVES_N> Core;
    constexpr int LOADS = Core::NA + Core::NB;
    static_assert(STAGES >= 2 && (STAGES - 1) * LOADS <= 63, "loads in flight");
    static_assert(Core::NW * Core::PATCH <= STAGES * Core::STAGE, "the patches fit in the stages");

    I8Tile t;
    if (!i8_tile_of<BM, BN>(p, t))
        return;
    Core c;
    c.init();
    c.operands(p, t);

    // Step s in stage s % STAGES: each k-group is read under the products of
    // the one before. Once the last one is read, all meet: the loads of step
    // s + 1 have to be there, those of step s + STAGES take the stage just
    // read, and the first k-group of s + 1 is read under the last products of
    // s. (After the last step this reads zeros.)
    const int steps = (p.K + Core::BK - 1) / Core::BK;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        c.issue(s, lds + s * Core::STAGE);
    meet<(STAGES - 2) * LOADS>();
    c.issue(STAGES - 1, lds + (STAGES - 1) * Core::STAGE);
    int cur = 0;
    if (t.m0 + c.wm < t.M) {
        c.zero();
        c.read(lds, 0);
        for (int s = 0; s < steps; ++s) {
            signed char *stage = lds + cur * Core::STAGE;
            c.step_front(stage);
            meet<(STAGES - 2) * LOADS>();
            cur = cur + 1 == STAGES ? 0 : cur + 1;
            c.step_back(lds + cur * Core::STAGE, s + STAGES, stage);
        }
        c.load_scales(p, t);
    } else {
        // A wave whose rows all lie behind the group's last only loads, and
        // leaves the matrix unit to the other wave of its SIMD.
        for (int s = 0; s < steps; ++s) {
            meet<(STAGES - 2) * LOADS>();
            c.issue(s + STAGES, lds + cur * Core::STAGE);
            cur = cur + 1 == STAGES ? 0 : cur + 1;
        }
    }
    wait_loads<0>();
    __syncthreads();
    if (t.m0 + c.wm < t.M)
        c.outputs(p, t, reinterpret_cast<float *>(lds + c.wave * Core::PATCH));
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES>
__global__ void
__attribute__((amdgpu_flat_work_group_size(64 * WAVES_M * WAVES_N, 64 * WAVES_M * WAVES_N)))
i8_large_kernel(I8Params p)
{
    __shared__ __attribute__((aligned(1024))) signed char lds[STAGES * (BM + BN) * 128];
    i8_large_tile<BM, BN, WAVES_M, WAVES_N, STAGES>(p, lds);
}

typedef void (*I8Fn)(I8Params);

struct I8Variant {
    I8Fn fn;
    int bm, bn, threads;
};

template <int MT, int NT, int WAVES, int U>
I8Variant stream_variant(bool aligned)
{
    return {aligned ? i8_stream_kernel<MT, NT, WAVES, U, true>
                    : i8_stream_kernel<MT, NT, WAVES, U, false>,
            16 * MT, 16 * NT, 64 * WAVES};
}

I8Variant variant_of(int kernel, bool aligned)
{
    switch (kernel) {
    case I8GEMM_KERNEL_S16x16: return stream_variant<1, 1, 8, 2>(aligned);
    case I8GEMM_KERNEL_S16x16_W16: return stream_variant<1, 1, 16, 2>(aligned);
    case I8GEMM_KERNEL_S16x32: return stream_variant<1, 2, 4, 2>(aligned);
    case I8GEMM_KERNEL_S32x16: return stream_variant<2, 1, 8, 2>(aligned);
    case I8GEMM_KERNEL_S32x32: return stream_variant<2, 2, 8, 2>(aligned);
    case I8GEMM_KERNEL_S32x64: return stream_variant<2, 4, 4, 2>(aligned);
    case I8GEMM_KERNEL_T64x64: return {i8_tile_kernel<1>, 64, 64, 256};
    case I8GEMM_KERNEL_T128x128: return {i8_tile_kernel<2>, 128, 128, 256};
    case I8GEMM_KERNEL_L32x64: return {i8_large_kernel<32, 64, 1, 2, 4>, 32, 64, 128};
    case I8GEMM_KERNEL_L64x64_R4: return {i8_large_kernel<64, 64, 2, 2, 4>, 64, 64, 256};
    case I8GEMM_KERNEL_L64x64: return {i8_large_kernel<64, 64, 2, 2, 3>, 64, 64, 256};
    case I8GEMM_KERNEL_L64x128: return {i8_large_kernel<64, 128, 2, 2, 3>, 64, 128, 256};
    case I8GEMM_KERNEL_L128x128: return {i8_large_kernel<128, 128, 2, 4, 4>, 128, 128, 512};
    case I8GEMM_KERNEL_L128x256: return {i8_large_kernel<128, 256, 2, 4, 3>, 128, 256, 512};
    default: return {i8_large_kernel<256, 256, 2, 4, 2>, 256, 256, 512};
    }
}

// The tiles that load straight into LDS, with what they cost on 256 CUs
// (measured, us): `step` for 128 bytes of K of one tile a CU, `fixed` for the
// launch, the first loads and the outputs. `one_round`: only where every CU
// gets at most one tile, as its four stages leave room for few workgroups.
struct I8Large {
    int kernel, bm, bn;
    float step, fixed;
    bool one_round;
};
const I8Large kLarge[] = {
    {I8GEMM_KERNEL_L32x64, 32, 64, 0.22f, 4.0f, false},
    {I8GEMM_KERNEL_L64x64_R4, 64, 64, 0.28f, 4.0f, true},
    {I8GEMM_KERNEL_L64x64, 64, 64, 0.33f, 4.0f, false},
    {I8GEMM_KERNEL_L64x128, 64, 128, 0.45f, 4.5f, false},
    {I8GEMM_KERNEL_L128x128, 128, 128, 0.70f, 5.0f, false},
    {I8GEMM_KERNEL_L128x256, 128, 256, 1.10f, 6.5f, false},
    {I8GEMM_KERNEL_L256x256, 256, 256, 1.85f, 8.0f, false},
};

long long i8_row_tiles(int M, int groups, int bm)
{
    return groups ? most_tiles(M, groups, bm) : ceil_div_ll(M, bm);
}

// The kernel of a call (an i8gemm_kernel), or -22 if the tiles of none fit a
// launch. Those whose tiles do not are passed over. Times below are graph
// replays over weights that no cache holds.
int choose_i8(int M, int N, int K, int groups, bool aligned, bool direct, int cus)
{
    auto takes = [&](int kernel) {
        const I8Variant v = variant_of(kernel, aligned);
        return fits_launch((double)i8_row_tiles(M, groups, v.bm) * (double)ceil_div_ll(N, v.bn),
                           v.threads);
    };
    const long long n16 = ceil_div_ll(N, 16);
    int stream = -1;
    if (groups) {
        // Up to 8 rows a group on average: the weights stream (256 rows over
        // 64 groups, 2048 x 2048: 51 us against 53.5 with the 32 x 64 tile;
        // 512 over 128, 4096 x 1024: 97 against 107; with 16 rows a group 72.5
        // against 55).
        if (M <= 8LL * groups || (!direct && M <= 16LL * groups))
            stream = I8GEMM_KERNEL_S16x32;
    } else if (M <= 16) {
        // One row tile: 16 channels a workgroup, K over 8 waves, or 16 for a
        // token or a few over a deep K (1 x 4096 x 16384: 14.7 us against
        // 16.5; with 16 rows 18.9 against 17.6). With many workgroups, 32
        // channels for as many rows as make A's bytes count (16 x 16384 x 4096:
        // 17.9 us against 19.1; one row 17.0 against 17.1, 28672 channels 26.8
        // against 23.7).
        if (M <= 4)
            stream = K >= 4096 && n16 <= 2LL * cus ? I8GEMM_KERNEL_S16x16_W16
                                                   : I8GEMM_KERNEL_S16x16;
        else
            stream = n16 >= 4LL * cus ? I8GEMM_KERNEL_S16x32 : I8GEMM_KERNEL_S16x16;
    } else {
        // Row tiles of 32 as long as every CU gets one workgroup at most: 16,
        // 32 or 64 channels (64 x 1024 x 4096: 7.9 us, the 32 x 64 tile 10.0;
        // 64 x 4096 x 4096: 10.9 and 11.7; 32 x 16384 x 4096: 20.7 and 28 with
        // the 64 x 64 tile; 128 x 4096 x 4096, two a CU: 17.8 and 11.8).
        const long long m32 = ceil_div_ll(M, 32);
        if (m32 * n16 <= cus)
            stream = I8GEMM_KERNEL_S32x16;
        else if (m32 * ceil_div_ll(N, 32) <= cus)
            stream = I8GEMM_KERNEL_S32x32;
        else if (m32 * ceil_div_ll(N, 64) <= cus && M <= 32)
            stream = I8GEMM_KERNEL_S32x64;
    }
    if (stream >= 0 && takes(stream))
        return stream;
    const double used = groups < M ? groups : M;
    // Row tiles: of groups, every one's own and half a tile more, since only
    // the device knows their rows.
    auto row_tiles = [&](int bm) {
        if (!groups)
            return (double)ceil_div_ll(M, bm);
        const double each = (double)M / groups / bm + 0.5;
        return used * (each > 1.0 ? each : 1.0);
    };
    if (!direct) {
        if (row_tiles(128) * (double)ceil_div_ll(N, 128) < cus && takes(I8GEMM_KERNEL_T64x64))
            return I8GEMM_KERNEL_T64x64;
        return takes(I8GEMM_KERNEL_T128x128) ? I8GEMM_KERNEL_T128x128 : -22;
    }
    int best = -22;
    float least = 0.0f;
    for (const I8Large &l : kLarge) {
        const double tiles = row_tiles(l.bm) * (double)ceil_div_ll(N, l.bn);
        if ((l.one_round && tiles > cus) || !takes(l.kernel))
            continue;
        const float rounds = (float)ceil_div_ll((long long)(tiles + 0.999), cus);
        const float cost = l.fixed + rounds * (float)ceil_div_ll(K, 128) * l.step;
        if (best < 0 || cost < least) {
            best = l.kernel;
            least = cost;
        }
    }
    return best;
}

// (Refused before the device is asked: not even 256 x 256 tiles fit a launch.)
bool too_many_tiles(int M, int N, int groups)
{
    return !fits_launch((double)i8_row_tiles(M, groups, 256) * (double)ceil_div_ll(N, 256), 512);
}

int launch_i8(I8Params p, hipStream_t s)
{
    if (too_many_tiles(p.M, p.N, p.groups))
        return -22;
    int cus = 0;
    const int st = current_cus(&cus);
    if (st != 0)
        return st;
    const bool aligned = (((uintptr_t)p.A | (uintptr_t)p.B) & 15) == 0 && p.lda % 16 == 0 &&
                         p.ldb % 16 == 0 && p.strideB % 16 == 0;
    const bool direct =
        aligned && p.K % 16 == 0 && p.lda < kMaxTileLd && p.ldb < kMaxTileLd && p.K > 0;
    const int kernel = choose_i8(p.M, p.N, p.K, p.groups, aligned, direct, cus);
    if (kernel < 0)
        return kernel;
    const I8Variant v = variant_of(kernel, aligned);
    p.tiles_m = (int)i8_row_tiles(p.M, p.groups, v.bm);
    p.tiles_n = (int)ceil_div_ll(p.N, v.bn);
    p.band = p.groups ? group_band(p.M, p.groups, v.bm) : 8;
    void *args[] = {&p};
    return (int)hipLaunchKernel((const void *)v.fn,
                                dim3((unsigned)((long long)p.tiles_m * p.tiles_n)),
                                dim3(v.threads), args, 0, s);
}

} // namespace

extern "C" int i8_quantize_rows(int M, int K, const void *X, int x_type, int ldx, signed char *Q,
                                int ldq, float *scale, sgemm_stream_t stream)
{
    if (M < 0) return -101;
    if (K < 0 || K > INT32_MAX - 65536) return -102;
    if (!c_type_ok(x_type)) return -104;
    const int row = K > 1 ? K : 1;
    if (ldx < row) return -105;
    if (ldq < row) return -107;
    if (M > 0 && K > 0 && X == nullptr) return -103;
    if (M > 0 && K > 0 && Q == nullptr) return -106;
    if (M > 0 && scale == nullptr) return -108;
    if (M == 0)
        return 0;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (x_type == SGEMM_F32)
        return launch_quantize<float>(M, K, X, ldx, Q, ldq, scale, s);
    if (x_type == SGEMM_F16)
        return launch_quantize<_Float16>(M, K, X, ldx, Q, ldq, scale, s);
    return launch_quantize<__bf16>(M, K, X, ldx, Q, ldq, scale, s);
}

extern "C" int i8gemm(int M, int N, int K, const signed char *A, int lda, const float *scaleA,
                      const signed char *B, int ldb, const float *scaleB, const float *bias,
                      void *C, int c_type, int ldc, sgemm_stream_t stream)
{
    if (M < 0) return -201;
    if (N < 0) return -202;
    if (K < 0 || K > I8GEMM_MAX_K) return -203;
    const int row = K > 1 ? K : 1;
    if (lda < row) return -205;
    if (ldb < row) return -208;
    if (!c_type_ok(c_type)) return -212;
    if (ldc < (N > 1 ? N : 1)) return -213;
    if (M == 0 || N == 0)
        return 0;
    if (K > 0 && A == nullptr) return -204;
    if (scaleA == nullptr) return -206;
    if (K > 0 && B == nullptr) return -207;
    if (scaleB == nullptr) return -209;
    if (C == nullptr) return -211;
    I8Params p{A, B, scaleA, scaleB, bias, C, nullptr, 0, M, N, K, lda, ldb, ldc, c_type, 0, 0, 0, 0};
    return launch_i8(p, static_cast<hipStream_t>(stream));
}

extern "C" int i8gemm_grouped(int M, int N, int K, int groups, const int *offsets,
                              const signed char *A, int lda, const float *scaleA,
                              const signed char *B, int ldb, long long strideB,
                              const float *scaleB, const float *bias, void *C, int c_type, int ldc,
                              sgemm_stream_t stream)
{
    if (M < 0) return -301;
    if (N < 0) return -302;
    if (K < 0 || K > I8GEMM_MAX_K) return -303;
    if (groups < 0 || groups > kMaxGroups) return -304;
    const int row = K > 1 ? K : 1;
    if (lda < row) return -307;
    if (ldb < row) return -310;
    if (strideB < 0) return -311;
    if (!c_type_ok(c_type)) return -315;
    if (ldc < (N > 1 ? N : 1)) return -316;
    if (M == 0 || N == 0 || groups == 0)
        return 0;
    if (offsets == nullptr) return -305;
    if (K > 0 && A == nullptr) return -306;
    if (scaleA == nullptr) return -308;
    if (K > 0 && B == nullptr) return -309;
    if (scaleB == nullptr) return -312;
    if (C == nullptr) return -314;
    I8Params p{A,   B,   scaleA, scaleB, bias,   C,      offsets, strideB, M,
               N,   K,   lda,    ldb,    ldc,    c_type, groups, 0, 0, 0};
    return launch_i8(p, static_cast<hipStream_t>(stream));
}

extern "C" int i8gemm_select_kernel(int M, int N, int K, int groups, int aligned, int num_cus)
{
    if (M < 0) return -201;
    if (N < 0) return -202;
    if (K < 0 || K > I8GEMM_MAX_K) return -203;
    if (groups < 0 || groups > kMaxGroups) return -304;
    if (too_many_tiles(M, N, groups)) return -22;
    return choose_i8(M, N, K, groups, aligned != 0, aligned != 0 && K > 0 && K % 16 == 0,
                     num_cus > 1 ? num_cus : 1);
}
