// Rows in blocks of 4-bit floating point with shared scales, and their products
// (mx4gemm.h), for MI355X (gfx950).

#include "ops_common.h"

#include "mx4gemm.h"

#include <type_traits>

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// Rounding to 4 bits and back. A lane holds 8 neighbouring elements, four lanes
// a block of 32, a wave 512 elements of a row.
// ---------------------------------------------------------------------------

// A lane's eight elements as they lie in memory (WHOLE: the wave's 512 are all
// there, so that no load stands in a branch), zeros behind the row's end.
template <typename T> struct Eight {
    static constexpr int VEC = 16 / (int)sizeof(T), N = 8 / VEC;
    i32x4 raw[N];

    template <bool WHOLE> __device__ __forceinline__ void load(const T *row, int k, int K)
    {
        if (WHOLE || k + 8 <= K) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                raw[i] = load16(row + k + i * VEC);
        } else {
            typedef T tv __attribute__((ext_vector_type(VEC)));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                tv v;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    v[e] = k + i * VEC + e < K ? row[k + i * VEC + e] : (T)0.0f;
                raw[i] = __builtin_bit_cast(i32x4, v);
            }
        }
    }

    __device__ __forceinline__ void floats(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[VEC];
            unpack<T>(raw[i], v);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                f[i * VEC + e] = v[e];
        }
    }
};

// The four bytes of eight elements' codes at q + k / 2, as far as the row goes.
__device__ __forceinline__ void store_codes(unsigned char *q, int k, int K, uint32_t codes)
{
    if (k + 8 <= K) {
        *reinterpret_cast<i32_any *>(q + (k >> 1)) = (int)codes;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + 2 * i < K)
                q[(k >> 1) + i] = (unsigned char)(codes >> (8 * i));
    }
}

// ROWS rows of 512 elements a workgroup, RW a wave, all loaded before the first is
// rounded; the scales leave as neighbouring rows' words. Bound by memory: 16 rows,
// 4 a wave (8192 x 4092 in fp32 33 us, 4.6 TB/s; behind a pass that left its writes
// to go to memory 40, with 32 rows, 8 a wave, 44), few rows one a wave (16 x 4096 in
// bf16 2.4 us, a launch and one trip to memory).
// A block's scale byte is the exponent field of its largest magnitude less 2
// (fields are offset by 127 as the bytes are; subnormal ones have field 0), and
// 2^-e is the number of field 254 - byte, so the quotient is an exact product
// and the conversion's rounding, to nearest with ties to even, the only one.
template <typename T, int ROWS, int RW>
__global__ void __launch_bounds__(64 * ROWS / RW)
mx4_quantize_kernel(int M, int K, const T *X, long long ldx, unsigned char *Q, long long ldq,
                    unsigned char *scale, long long lds)
{
    __shared__ uint32_t bytes[4][ROWS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k = blockIdx.x * 512 + 8 * lane;
    const long long m0 = (long long)blockIdx.y * ROWS;
    Eight<T> held[RW];
    auto load = [&](auto whole) {
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const long long m = m0 + wave * RW + r;
            held[r].template load<decltype(whole)::value>(X + (m < M ? m : M - 1) * ldx, k, K);
        }
    };
    if ((int)blockIdx.x * 512 + 512 <= K)
        load(std::true_type{});
    else
        load(std::false_type{});
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const long long m = m0 + wave * RW + r;
        float f[8];
        held[r].floats(f);
        uint32_t peak = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            peak = max(peak, __builtin_bit_cast(uint32_t, f[i]) & 0x7fffffffu);
        peak = max(peak, (uint32_t)__shfl_xor((int)peak, 1));
        peak = max(peak, (uint32_t)__shfl_xor((int)peak, 2));
        const int field = (int)(peak >> 23);
        const bool finite = field < 255;
        const int byte = finite ? max(field - 2, 0) : 255;
        const float up = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
        uint32_t codes = 0;
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[0] * up, f[1] * up, 1.0f, 0);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[2] * up, f[3] * up, 1.0f, 1);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[4] * up, f[5] * up, 1.0f, 2);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[6] * up, f[7] * up, 1.0f, 3);
        if (m < M && k < K)
            store_codes(Q + m * ldq, k, K, finite ? codes : 0u);
        // Four blocks' bytes in one word; 0 for blocks behind the row's last.
        uint32_t word = (k & ~31) < K ? (uint32_t)byte << (8 * ((lane >> 2) & 3)) : 0u;
        word |= (uint32_t)__shfl_xor((int)word, 4);
        word |= (uint32_t)__shfl_xor((int)word, 8);
        if ((lane & 15) == 0)
            bytes[lane >> 4][wave * RW + r] = word;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 4 * ROWS; i += 64 * ROWS / RW) {
        const int g = blockIdx.x * 4 + i / ROWS;
        const long long m = m0 + i % ROWS;
        if (m < M && g < (K + 127) / 128)
            reinterpret_cast<uint32_t *>(scale)[g * lds + m] = bytes[i / ROWS][i % ROWS];
    }
}

template <typename T>
int launch_mx4_quantize(int M, int K, const void *X, long long ldx, unsigned char *Q, long long ldq,
                        unsigned char *scale, long long lds, hipStream_t s)
{
    const T *x = static_cast<const T *>(X);
    typedef void (*Fn)(int, int, const T *, long long, unsigned char *, long long, unsigned char *,
                       long long);
    const bool few = M <= 64;
    const Fn fn = few ? mx4_quantize_kernel<T, 4, 1> : mx4_quantize_kernel<T, 16, 4>;
    const int rows = few ? 4 : 16;
    const unsigned columns = (unsigned)ceil_div_ll(K, 512);
    // Rows in launches of fewer than 2^32 work-items and 65536 rows of workgroups.
    long long most = (1LL << 23) / columns;
    most = rows * (most < 1 ? 1 : most < 65535 ? most : 65535);
    for (long long m0 = 0; m0 < M; m0 += most) {
        int n = (int)(M - m0 < most ? M - m0 : most);
        const T *xs = x + m0 * ldx;
        unsigned char *q = Q + m0 * ldq, *sc = scale + 4 * m0;
        void *args[] = {&n, &K, &xs, &ldx, &q, &ldq, &sc, &lds};
        const hipError_t e = hipLaunchKernel((const void *)fn,
                                             dim3(columns, (unsigned)ceil_div_ll(n, rows)),
                                             dim3(256), args, 0, s);
        if (e != hipSuccess)
            return (int)e;
    }
    return 0;
}

// The scale of a byte: fields are offset alike, but for the ends.
__device__ __forceinline__ float scale_of(uint32_t byte)
{
    const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23;
    return __builtin_bit_cast(float, bits);
}

// And back: kBackRows rows of 512 elements a wave, with a store of 16 bytes a lane,
// so that neighbouring lanes fill whole lines. Bound by memory: 8192 x 4096 to fp32
// that no cache holds takes 30.5 us (5 TB/s; 41 with two stores of a lane side by
// side), 8192 x 4092, rows off a line, 36 (47). More rows a wave gain nothing there
// and cost the few their latency (16 x 4096 in bf16: 2, 4 and 8 rows 2.4, 2.8, 3.8).
constexpr int kBackRows = 2;

template <typename T>
__global__ void __launch_bounds__(256)
mx4_dequantize_kernel(int M, int K, const unsigned char *Q, long long ldq,
                      const unsigned char *scale, long long lds, T *Y, long long ldy)
{
    constexpr int VEC = 16 / sizeof(T), PARTS = 8 / VEC;
    typedef T tv __attribute__((ext_vector_type(VEC)));
    typedef unsigned short u16_any __attribute__((aligned(1)));
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k0 = blockIdx.x * 512 + VEC * lane;
    const long long m0 = ((long long)blockIdx.y * 4 + wave) * kBackRows;
    uint32_t codes[kBackRows][PARTS], bytes[kBackRows][PARTS];
#pragma unroll
    for (int r = 0; r < kBackRows; ++r)
#pragma unroll
        for (int c = 0; c < PARTS; ++c) {
            const long long m = m0 + r;
            const int k = k0 + c * 64 * VEC;
            codes[r][c] = bytes[r][c] = 0;
            if (m >= M || k >= K)
                continue;
            const unsigned char *q = Q + m * ldq + (k >> 1);
            bytes[r][c] = scale[((k >> 7) * lds + m) * 4 + ((k >> 5) & 3)];
            if (k + VEC <= K) {
                if constexpr (VEC == 4)
                    codes[r][c] = *reinterpret_cast<const u16_any *>(q);
                else
                    codes[r][c] = (uint32_t)*reinterpret_cast<const i32_any *>(q);
            } else {
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i)
                    if (k + 2 * i < K)
                        codes[r][c] |= (uint32_t)q[i] << (8 * i);
            }
        }
#pragma unroll
    for (int r = 0; r < kBackRows; ++r)
#pragma unroll
        for (int c = 0; c < PARTS; ++c) {
            const long long m = m0 + r;
            const int k = k0 + c * 64 * VEC;
            if (m >= M || k >= K)
                continue;
            const float s = scale_of(bytes[r][c]);
            tv v;
            auto pair = [&](f32x2 f, int i) {
                v[i] = (T)f[0];
                v[i + 1] = (T)f[1];
            };
            pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[r][c], s, 0), 0);
            pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[r][c], s, 1), 2);
            if constexpr (VEC == 8) {
                pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[r][c], s, 2), 4);
                pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[r][c], s, 3), 6);
            }
            T *y = Y + m * ldy + k;
            if (k + VEC <= K) {
                store16(y, __builtin_bit_cast(i32x4, v));
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (k + i < K)
                        y[i] = v[i];
            }
        }
}

template <typename T>
int launch_mx4_dequantize(int M, int K, const unsigned char *Q, long long ldq,
                          const unsigned char *scale, long long lds, void *Y, long long ldy,
                          hipStream_t s)
{
    const unsigned columns = (unsigned)ceil_div_ll(K, 512);
    long long most = (1LL << 23) / columns;
    constexpr int rows = 4 * kBackRows; // a workgroup
    most = rows * (most < 1 ? 1 : most < 65535 ? most : 65535);
    for (long long m0 = 0; m0 < M; m0 += most) {
        int n = (int)(M - m0 < most ? M - m0 : most);
        const unsigned char *q = Q + m0 * ldq, *sc = scale + 4 * m0;
        T *y = static_cast<T *>(Y) + m0 * ldy;
        void *args[] = {&n, &K, &q, &ldq, &sc, &lds, &y, &ldy};
        const hipError_t e = hipLaunchKernel((const void *)mx4_dequantize_kernel<T>,
                                             dim3(columns, (unsigned)ceil_div_ll(n, rows)), dim3(256),
                                             args, 0, s);
        if (e != hipSuccess)
            return (int)e;
    }
    return 0;
}

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------

struct Mx4Params {
    const signed char *A, *B;   // elements, two a byte
    const uint32_t *sA, *sB;    // scales, four blocks a word
    const float *bias;
    void *C;
    const int *offsets; // grouped calls: row ranges of the groups
    long long strideB, strideSB; // of sB in words
    int M, N, K;
    int lda, ldb, ldc;
    int ldsa, ldsb;
    int type;
    int groups;           // 0: one product
    int tiles_m, tiles_n; // the grid
    int band;             // row tiles of a band of the grid's order
};

// Where a workgroup stands: its group's operands and its rows [m0, M) of
// them, counted from the group's first row.
struct Mx4Tile {
    const signed char *A, *B;
    const uint32_t *sA, *sB;
    const float *bias;
    long long row0; // C's row of the group's first row
    int M, m0, n0;
};

template <int BM, int BN>
__device__ __forceinline__ bool mx4_tile_of(const Mx4Params &p, Mx4Tile &t)
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
        t.sB += g * p.strideSB;
        if (t.bias)
            t.bias += (long long)g * p.N;
    }
    t.n0 = tn * BN;
    return true;
}

// A block's 16 bytes as the matrix instructions take them (the upper half of
// their operands is for wider elements).
__device__ __forceinline__ i32x8 operand(i32x4 v)
{
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

constexpr int kFp4 = 4; // the instructions' number of the element type

// The bytes of a word of scales that belong to blocks: all but in a row's last.
__device__ __forceinline__ uint32_t scale_mask(int word, int K)
{
    const int blocks = ((K + 31) >> 5) - 4 * word;
    return blocks >= 4 ? 0xffffffffu : blocks <= 0 ? 0u : (1u << (8 * blocks)) - 1;
}

// The tile for every alignment: 64 T x 64 T of C by four waves, each one T x T
// accumulators of v_mfma_scale_f32_32x32x64 (lane l supplies 32 elements, a
// block, of row l % 32 from k = 32 (l / 32) on, and its scale; register v of
// lane l holds row 8 (v / 4) + 4 (l / 32) + v % 4, column l % 32). 64-byte
// K-steps go through registers to LDS, so any alignment and any K will do, and
// zeros behind K leave the sum as it is. LDS rows are 64 bytes, four of them one
// sweep of the 64 banks, so the 16-byte chunk index is XORed with row / 4 for
// conflict-free reads. A step is a word of scales a row, which lanes load for
// themselves, neighbouring rows' side by side. Rows behind M or N repeat the
// last one and are not stored.
template <int T>
__global__ void __launch_bounds__(256) mx4_tile_kernel(Mx4Params p)
{
    constexpr int BM = 64 * T, BN = 64 * T, BK = 64;
    __shared__ __attribute__((aligned(16))) signed char lds[2][2][BM * BK];
    Mx4Tile t;
    if (!mx4_tile_of<BM, BN>(p, t))
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = tid >> 2, c = tid & 3;
    const int o = lane & 31, half = lane >> 5;
    const int wm = 32 * T * (wave & 1), wn = 32 * T * (wave >> 1);
    const signed char *ra[T], *rb[T];
    const uint32_t *pa[T], *pb[T];
#pragma unroll
    for (int x = 0; x < T; ++x) {
        ra[x] = t.A + (long long)min(t.m0 + 64 * x + r, t.M - 1) * p.lda;
        rb[x] = t.B + (long long)min(t.n0 + 64 * x + r, p.N - 1) * p.ldb;
        pa[x] = t.sA + min(t.m0 + wm + 32 * x + o, t.M - 1);
        pb[x] = t.sB + min(t.n0 + wn + 32 * x + o, p.N - 1);
    }
    const int at = r * BK + 16 * (c ^ ((r >> 2) & 3)); // (64 rows on: the same chunk)

    f32x16 acc[T][T] = {};
    const int steps = (p.K + 2 * BK - 1) / (2 * BK);
    i32x4 va[T] = {}, vb[T] = {};
    uint32_t wa[T] = {}, wb[T] = {};
    auto load = [&](int s) {
        const uint32_t mask = scale_mask(s, p.K);
#pragma unroll
        for (int x = 0; x < T; ++x) {
            va[x] = mx4_chunk(ra[x], s * BK + 16 * c, p.K);
            vb[x] = mx4_chunk(rb[x], s * BK + 16 * c, p.K);
            wa[x] = pa[x][(long long)s * p.ldsa] & mask;
            wb[x] = pb[x][(long long)s * p.ldsb] & mask;
        }
    };
    if (steps > 0)
        load(0);
    for (int s = 0; s < steps; ++s) {
        signed char *la = lds[s & 1][0], *lb = lds[s & 1][1];
        int sa[T], sb[T];
#pragma unroll
        for (int x = 0; x < T; ++x) {
            *reinterpret_cast<i32x4 *>(la + at + 64 * BK * x) = va[x];
            *reinterpret_cast<i32x4 *>(lb + at + 64 * BK * x) = vb[x];
            // (Blocks 2 q + half: bytes 0 and 2 of the word from there on.)
            sa[x] = (int)(wa[x] >> (8 * half));
            sb[x] = (int)(wb[x] >> (8 * half));
        }
        __syncthreads();
        if (s + 1 < steps)
            load(s + 1);
        auto group = [&](auto which) {
            constexpr int q = decltype(which)::value;
            const int ch = 16 * ((2 * q + half) ^ ((o >> 2) & 3));
            i32x8 fa[T], fb[T];
#pragma unroll
            for (int x = 0; x < T; ++x) {
                fa[x] = operand(*reinterpret_cast<const i32x4 *>(la + (wm + 32 * x + o) * BK + ch));
                fb[x] = operand(*reinterpret_cast<const i32x4 *>(lb + (wn + 32 * x + o) * BK + ch));
            }
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int j = 0; j < T; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fa[i], fb[j], acc[i][j], kFp4, kFp4, 2 * q, sa[i], 2 * q, sb[j]);
        };
        group(std::integral_constant<int, 0>{});
        group(std::integral_constant<int, 1>{});
        // (The next step writes the other stage, which every wave left before
        // this step's barrier.)
    }
    with_type(p.type, [&](auto type) {
        typedef decltype(type) C;
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const int n = t.n0 + wn + 32 * j + o;
            if (n >= p.N)
                continue;
            const float bias = t.bias ? t.bias[n] : 0.0f;
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int m = t.m0 + wm + 32 * i + 8 * (v >> 2) + 4 * half + (v & 3);
                    if (m < t.M)
                        static_cast<C *>(p.C)[(t.row0 + m) * p.ldc + n] =
                            (C)(acc[i][j][v] + bias);
                }
        }
    });
}

// ---------------------------------------------------------------------------
// Few rows: the weights' bytes bound the call, so they go from memory straight
// into the matrix instructions' registers, once, and no LDS stage stands
// between. A workgroup owns 16 * NT channels and up to 16 * MT rows; its WAVES
// waves take every WAVES-th block of 128 * U of k, so all of a short K is in
// flight at once, and their sums are added in LDS, in the waves' order.
// v_mfma_scale_f32_16x16x128: lane l supplies the block l / 16 of row l % 16 and
// its scale, a byte of the word that the row's four lanes load alike; register v
// of lane l holds row 4 (l / 16) + v, column l % 16. Rows behind the last repeat
// it and are not stored. 1 x 4096 x 4096 takes 4.0 us, 16384 channels 8.8 (4.0 TB/s).
// ---------------------------------------------------------------------------
template <int MT, int NT, int WAVES, int U>
__global__ void __launch_bounds__(64 * WAVES) mx4_stream_kernel(Mx4Params p)
{
    constexpr int BM = 16 * MT, BN = 16 * NT;
    __shared__ float sums[WAVES][BM][BN];
    Mx4Tile t;
    if (!mx4_tile_of<BM, BN>(p, t))
        return;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const signed char *ra[MT], *rb[NT];
    const uint32_t *pa[MT], *pb[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = min(t.m0 + 16 * i + r, t.M - 1);
        ra[i] = t.A + (long long)m * p.lda + 16 * q;
        pa[i] = t.sA + m;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = min(t.n0 + 16 * j + r, p.N - 1);
        rb[j] = t.B + (long long)n * p.ldb + 16 * q;
        pb[j] = t.sB + n;
    }

    f32x4 acc[MT][NT] = {};
    auto products = [&](const i32x4 (&fa)[MT], const uint32_t (&sa)[MT], const i32x4 (&fb)[NT],
                        const uint32_t (&sb)[NT]) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    operand(fa[i]), operand(fb[j]), acc[i][j], kFp4, kFp4, 0,
                    (int)(sa[i] >> (8 * q)), 0, (int)(sb[j] >> (8 * q)));
    };
    const int words = (p.K + 127) >> 7, whole = p.K >> 7; // words of scales; full steps
    int s = wave * U;
    for (; s + U <= whole; s += WAVES * U) {
        i32x4 fb[U][NT], fa[U][MT];
        uint32_t sb[U][NT], sa[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                fb[u][j] = load16(rb[j] + 64LL * (s + u));
                sb[u][j] = pb[j][(long long)(s + u) * p.ldsb];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                fa[u][i] = load16(ra[i] + 64LL * (s + u));
                sa[u][i] = pa[i][(long long)(s + u) * p.ldsa];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            products(fa[u], sa[u], fb[u], sb[u]);
    }
    // The block at the rows' end.
    for (; s < words && s / U % WAVES == wave; ++s) {
        i32x4 fb[NT], fa[MT];
        uint32_t sb[NT], sa[MT];
        const uint32_t mask = scale_mask(s, p.K);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            fb[j] = mx4_chunk(rb[j] - 16 * q, 64 * s + 16 * q, p.K);
            sb[j] = pb[j][(long long)s * p.ldsb] & mask;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            fa[i] = mx4_chunk(ra[i] - 16 * q, 64 * s + 16 * q, p.K);
            sa[i] = pa[i][(long long)s * p.ldsa] & mask;
        }
        products(fa, sa, fb, sb);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                sums[wave][16 * i + 4 * q + v][16 * j + r] = acc[i][j][v];
    __syncthreads();
    const int rows = min(BM, t.M - t.m0);
    for (int e = tid; e < rows * BN; e += 64 * WAVES) {
        const int m = e / BN, n = t.n0 + e % BN;
        if (n >= p.N)
            continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            sum += sums[w][m][e % BN];
        if (t.bias)
            sum += t.bias[n];
        const long long at = (t.row0 + t.m0 + m) * p.ldc + n;
        with_type(p.type, [&](auto type) {
            static_cast<decltype(type) *>(p.C)[at] = (decltype(type))sum;
        });
    }
}

// ---------------------------------------------------------------------------
// Larger products: BM x BN of C by WAVES_M x WAVES_N waves, K in steps of 256
// (128 bytes a row) that go straight from memory to LDS (buffer_load ... lds)
// through a ring of STAGES stages, as the 8-bit product's do. Lane l of a load
// fills the l-th 16 bytes of a 1 KiB block, 8 rows of 128 bytes: whole cache
// lines. LDS rows are 128 bytes, two of them one sweep of the 64 banks: the
// 16-byte chunk index is XORed with row / 2, on the memory side, for
// conflict-free reads. Behind a stage's rows stand their scales, two words a
// row: 64 neighbouring rows' words a load. Lanes of the lower half of a wave
// take the first four chunks of a row's eight and the first word, those of the
// upper half the others, so that the k-group's number is the byte of the word
// that the instruction takes (the order of k within a sum is free). A lane whose
// chunk or word lies behind K fetches zeros from a 2^31 byte offset, outside the
// buffer; the bytes of a row's last word that belong to no block are masked.
// Loads are issued for steps past the last too (of zeros), so that the number in
// flight is the same at every wait. Needs 16-byte-aligned rows, K a multiple of
// 32 and leading dimensions below 2^22 (32-bit offsets within a tile).
//
// 8192^3 runs at 4.2 PFLOP/s (261 us; the library product of such blocks 357),
// 4096 x 8192 x 4096 takes 76 us (101): the matrix units are busy 41 % of the
// cycles of a clock that stands at 1.95 GHz, LDS reads take three quarters of
// those the products do. Four waves of 128 x 128 each, with two thirds of the
// reads but a wave a SIMD, take 277 us.
// ---------------------------------------------------------------------------
template <int BM, int BN, int WAVES_M, int WAVES_N>
struct Mx4Core {
    static constexpr int BK = 128, KH = BK / 32, NW = WAVES_M * WAVES_N; // (bytes of a row)
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 32, TN = WN / 32;
    static constexpr int WORDS = (BM + BN) * BK; // the scales' offset in a stage
    static constexpr int STAGE = WORDS + (BM + BN) * 8;
    static constexpr int NA = BM * BK / 1024 / NW, NB = BN * BK / 1024 / NW; // blocks a wave loads
    // Loads of 64 words: of A's rows' first words, their second ones, B's. Waves
    // beyond the last repeat an earlier load, into the same place.
    static constexpr int SLOADS = (BM + BN) / 32, NS = (SLOADS + NW - 1) / NW;
    static constexpr int LOADS = NA + NB + NS;
    static_assert(NA >= 1 && NB >= 1, "a wave loads of both operands");
    static_assert(STAGE == (BM + BN) * 136, "a row's bytes and its words");
    static_assert(BM % 64 == 0 && BN % 64 == 0, "a load's words belong to one operand");
    static constexpr int PATCH = 16 * WN * 4; // bytes of LDS a wave's outputs turn over in

    int lane, wave, wm, wn, chunk, o, half;
    int at[KH];
    // The operands that loads are issued of.
    const signed char *A, *B;
    const uint32_t *sA, *sB;
    long long bytesA, bytesB;
    int K, words, ldsa, ldsb;
    uint32_t offA[NA], offB[NB], offS[NS];
    f32x16 acc[TM][TN];
    i32x4 fa[2][TM], fb[2][TN]; // of k-groups by parity
    int wa[TM], wb[TN];         // words of scales of the step
    float bias[4];              // of the four columns that the lane stores

    __device__ __forceinline__ void init()
    {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        // (Waves that share a SIMD, four apart, lie above one another in M.)
        wm = (wave / WAVES_N) * WM;
        wn = (wave % WAVES_N) * WN;
        chunk = 16 * ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
        // This lane's 16 bytes of k-group q in row 32 i + l % 32 of the wave's
        // part; 32 rows on is a fixed distance.
        o = lane & 31;
        half = lane >> 5;
#pragma unroll
        for (int q = 0; q < KH; ++q)
            at[q] = o * BK + 16 * ((4 * half + q) ^ ((o >> 1) & 7));
    }

    // Which rows' words load i of this wave holds.
    __device__ __forceinline__ void word_load(int i, bool &ofA, int &second, int &row) const
    {
        int n = (wave + NW * i) % SLOADS;
        ofA = n < BM / 32;
        n -= ofA ? 0 : BM / 32;
        const int each = (ofA ? BM : BN) / 64 > 0 ? (ofA ? BM : BN) / 64 : 1;
        second = n / each;
        row = 64 * (n % each);
    }

    __device__ __forceinline__ void operands(const Mx4Params &p, const Mx4Tile &t)
    {
        const int bytes = p.K / 2;
        A = t.A + (long long)t.m0 * p.lda;
        B = t.B + (long long)t.n0 * p.ldb;
        sA = t.sA + t.m0;
        sB = t.sB + t.n0;
        bytesA = (long long)(t.M - t.m0 - 1) * p.lda + bytes;
        bytesB = (long long)(p.N - t.n0 - 1) * p.ldb + bytes;
        K = bytes;
        words = (p.K + 127) >> 7;
        ldsa = p.ldsa;
        ldsb = p.ldsb;
        // (Rows behind the last repeat it; they are not stored.)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            offA[i] = (uint32_t)(min(8 * (wave + NW * i) + (lane >> 3), t.M - t.m0 - 1) * p.lda + chunk);
#pragma unroll
        for (int i = 0; i < NB; ++i)
            offB[i] = (uint32_t)(min(8 * (wave + NW * i) + (lane >> 3), p.N - t.n0 - 1) * p.ldb + chunk);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            bool ofA;
            int second, row;
            word_load(i, ofA, second, row);
            offS[i] = 4u * (uint32_t)min(row + lane, ofA ? t.M - t.m0 - 1 : p.N - t.n0 - 1);
        }
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
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            bool ofA;
            int second, row;
            word_load(i, ofA, second, row);
            const int word = 2 * step + second;
            // (The word's row of the scales as the base: no offset grows with K.)
            const uint32_t *base = (ofA ? sA : sB) + (long long)min(word, words - 1) * (ofA ? ldsa : ldsb);
            const __amdgpu_buffer_rsrc_t rs =
                rows_rsrc(reinterpret_cast<const signed char *>(base), 1 << 12);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (lds_void *)(to + WORDS + 256 * ((wave + NW * i) % SLOADS)), 4,
                offS[i] | (word < words ? 0u : kOutside), 0, 0, 0);
        }
    }

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = f32x16{};
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

    // The step's words of scales, without the bytes of blocks that are none.
    __device__ __forceinline__ void read_words(const signed char *stage, int step)
    {
        const int left = (K >> 4) - 4 * (2 * step + half); // blocks from the lane's word on
        const int mask = left >= 4 ? -1 : left <= 0 ? 0 : (1 << (8 * left)) - 1;
        const int *w = reinterpret_cast<const int *>(stage + WORDS) + half * BM + wm + o;
#pragma unroll
        for (int i = 0; i < TM; ++i)
            wa[i] = w[32 * i] & mask;
        w = reinterpret_cast<const int *>(stage + WORDS) + 2 * BM + half * BN + wn + o;
#pragma unroll
        for (int j = 0; j < TN; ++j)
            wb[j] = w[32 * j] & mask;
    }

    template <int q> __device__ __forceinline__ void products()
    {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    operand(fa[q & 1][i]), operand(fb[q & 1][j]), acc[i][j], kFp4, kFp4, q, wa[i],
                    q, wb[j]);
    }

    // All but the last k-group of the step in `stage` (whose first one is read).
    __device__ __forceinline__ void step_front(const signed char *stage)
    {
        front<0>(stage);
        front<1>(stage);
        front<2>(stage);
    }

    template <int q> __device__ __forceinline__ void front(const signed char *stage)
    {
        read(stage, q + 1);
        products<q>();
        __builtin_amdgcn_sched_group_barrier(0x100, TM + TN, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, TM * TN, 0);
    }

    // The last k-group, with the first one of the next step's stage read and
    // the loads of step `ahead` issued under its products.
    __device__ __forceinline__ void step_back(const signed char *next, int ahead, signed char *to)
    {
        read(next, 0);
        issue(ahead, to);
        products<KH - 1>();
        constexpr int GAP = TM * TN / LOADS > 0 ? TM * TN / LOADS : 1;
        __builtin_amdgcn_sched_group_barrier(0x100, TM + TN, 0);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, GAP, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, TM * TN, 0);
        __builtin_amdgcn_sched_barrier(0);
    }

    __device__ __forceinline__ void load_bias(const Mx4Params &p, const Mx4Tile &t)
    {
        const int n = t.n0 + wn + 4 * (lane % (WN / 4));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            bias[e] = t.bias ? t.bias[min(n + e, p.N - 1)] : 0.0f;
    }

    // The wave's outputs, 16 rows at a time through a patch of LDS of its own,
    // so that a row's leave as 16-byte (fp32) or 8-byte pieces. Rows 4 apart,
    // which one write instruction holds, are 32 banks apart by the XOR. EDGE:
    // the tile reaches past M or N.
    template <typename T, bool EDGE>
    __device__ __forceinline__ void turn_over(const Mx4Params &p, const Mx4Tile &t, float *patch) const
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
                    patch[(row * WN + 32 * j + o) ^ (8 * (row & 4))] = acc[h / 2][j][8 * (h & 1) + v];
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int r0 = 0; r0 < 16; r0 += RPI) {
                const int row = r0 + r, m = 16 * h + row;
                f32x4 x = *reinterpret_cast<const f32x4 *>(
                    patch + ((row * WN + c) ^ (8 * (row & 4))));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] += bias[e];
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

    __device__ __forceinline__ void outputs(const Mx4Params &p, const Mx4Tile &t, float *patch) const
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
__device__ __forceinline__ void mx4_large_tile(const Mx4Params &p, signed char *lds)
{
    typedef Mx4Core<BM, BN, WAVES_M, WAVES_N> Core;
    constexpr int LOADS = Core::LOADS;
    static_assert(STAGES >= 2 && (STAGES - 1) * LOADS <= 63, "loads in flight");
    static_assert(Core::NW * Core::PATCH <= STAGES * Core::STAGE, "the patches fit in the stages");

    Mx4Tile t;
    if (!mx4_tile_of<BM, BN>(p, t))
        return;
    Core c;
    c.init();
    c.operands(p, t);

    // Step s in stage s % STAGES: each k-group is read under the products of
    // the one before. Once the last one is read, all meet: the loads of step
    // s + 1 have to be there, those of step s + STAGES take the stage just
    // read, and the first k-group of s + 1 is read under the last products of
    // s. (After the last step this reads zeros.)
    const int steps = (c.K + Core::BK - 1) / Core::BK;
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
            c.read_words(stage, s);
            c.step_front(stage);
            meet<(STAGES - 2) * LOADS>();
            cur = cur + 1 == STAGES ? 0 : cur + 1;
            c.step_back(lds + cur * Core::STAGE, s + STAGES, stage);
        }
        c.load_bias(p, t);
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
mx4_large_kernel(Mx4Params p)
{
    __shared__ __attribute__((aligned(1024))) signed char lds[STAGES * (BM + BN) * 136];
    mx4_large_tile<BM, BN, WAVES_M, WAVES_N, STAGES>(p, lds);
}

typedef void (*Mx4Fn)(Mx4Params);

struct Mx4Variant {
    Mx4Fn fn;
    int bm, bn, threads;
};

template <int MT, int NT, int WAVES, int U> Mx4Variant stream_variant()
{
    return {mx4_stream_kernel<MT, NT, WAVES, U>, 16 * MT, 16 * NT, 64 * WAVES};
}

Mx4Variant variant_of(int kernel)
{
    switch (kernel) {
    case MX4GEMM_KERNEL_S16x16: return stream_variant<1, 1, 8, 2>();
    case MX4GEMM_KERNEL_S16x32: return stream_variant<1, 2, 4, 2>();
    case MX4GEMM_KERNEL_S32x16: return stream_variant<2, 1, 8, 2>();
    case MX4GEMM_KERNEL_S32x32: return stream_variant<2, 2, 8, 2>();
    case MX4GEMM_KERNEL_S32x64: return stream_variant<2, 4, 4, 2>();
    case MX4GEMM_KERNEL_T64x64: return {mx4_tile_kernel<1>, 64, 64, 256};
    case MX4GEMM_KERNEL_T128x128: return {mx4_tile_kernel<2>, 128, 128, 256};
    case MX4GEMM_KERNEL_L64x64: return {mx4_large_kernel<64, 64, 2, 2, 3>, 64, 64, 256};
    case MX4GEMM_KERNEL_L64x128: return {mx4_large_kernel<64, 128, 2, 2, 3>, 64, 128, 256};
    case MX4GEMM_KERNEL_L128x128: return {mx4_large_kernel<128, 128, 2, 4, 4>, 128, 128, 512};
    case MX4GEMM_KERNEL_L128x128_R2: return {mx4_large_kernel<128, 128, 2, 4, 2>, 128, 128, 512};
    case MX4GEMM_KERNEL_L128x256: return {mx4_large_kernel<128, 256, 2, 4, 3>, 128, 256, 512};
    default: return {mx4_large_kernel<256, 256, 2, 4, 2>, 256, 256, 512};
    }
}

// The tiles that load straight into LDS, with what they cost on 256 CUs
// (measured, us): a lone tile a CU takes 4.5 and `wait` for 256 of K, its loads'
// way; a CU with tiles enough takes `fixed` and `step` for 256 of K of each. (The
// 128 x 128 tile with two stages of LDS for four has two workgroups a CU, whose
// outputs and first loads run under each other's products: 2048 x 4096 x 4096
// 28 us against 32, a tile a CU, 1024 x 4096 x 4096, 20.4 against 17.7.)
struct Mx4Large {
    int kernel, bm, bn;
    float wait, fixed, step;
};
const Mx4Large kLarge[] = {
    {MX4GEMM_KERNEL_L64x64, 64, 64, 0.32f, 2.2f, 0.15f},
    {MX4GEMM_KERNEL_L64x128, 64, 128, 0.50f, 3.2f, 0.29f},
    {MX4GEMM_KERNEL_L128x128, 128, 128, 0.76f, 4.2f, 0.64f},
    {MX4GEMM_KERNEL_L128x128_R2, 128, 128, 0.99f, 4.0f, 0.52f},
    {MX4GEMM_KERNEL_L128x256, 128, 256, 1.02f, 6.5f, 1.05f},
    {MX4GEMM_KERNEL_L256x256, 256, 256, 1.70f, 10.8f, 1.70f},
};

long long mx4_row_tiles(int M, int groups, int bm)
{
    return groups ? most_tiles(M, groups, bm) : ceil_div_ll(M, bm);
}

// The kernel of a call (an mx4gemm_kernel), or -22 if the tiles of none fit a
// launch. Those whose tiles do not are passed over.
int choose_mx4(int M, int N, int K, int groups, bool direct, int cus)
{
    auto takes = [&](int kernel) {
        const Mx4Variant v = variant_of(kernel);
        return fits_launch((double)mx4_row_tiles(M, groups, v.bm) * (double)ceil_div_ll(N, v.bn),
                           v.threads);
    };
    const long long n16 = ceil_div_ll(N, 16);
    int stream = -1;
    // Times are graph replays over operands that no cache holds.
    if (groups) {
        // Up to 4 rows a group on average the weights stream (256 rows over 64
        // groups, 2048 x 2048: 28.8 us against 29.4 with the 64 x 128 tile; with
        // 8 rows a group 34.6 against 31.6).
        if (M <= 4LL * groups || (!direct && M <= 16LL * groups))
            stream = MX4GEMM_KERNEL_S16x32;
    } else if (M <= 16) {
        // One row tile: 16 channels a workgroup, with many of them 32 (16 x 4096
        // x 4096: 4.8 us against 5.9; 16 x 16384 x 4096: 13.4 against 10.3).
        stream = n16 >= 4LL * cus ? MX4GEMM_KERNEL_S16x32 : MX4GEMM_KERNEL_S16x16;
    } else {
        // Row tiles of 32 as long as every CU gets one workgroup at most (32 x
        // 4096 x 4096: 5.8 us against 7.9 with the 64 x 64 tile, 64 x 4096 x 4096
        // 7.4 and 8.4, 128 x 4096 x 4096, more than one a CU, 11.1 and 8.7).
        const long long m32 = ceil_div_ll(M, 32);
        if (m32 * n16 <= cus)
            stream = MX4GEMM_KERNEL_S32x16;
        else if (m32 * ceil_div_ll(N, 32) <= cus)
            stream = MX4GEMM_KERNEL_S32x32;
        else if (m32 * ceil_div_ll(N, 64) <= cus && M <= 32)
            stream = MX4GEMM_KERNEL_S32x64;
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
        if (row_tiles(128) * (double)ceil_div_ll(N, 128) < cus && takes(MX4GEMM_KERNEL_T64x64))
            return MX4GEMM_KERNEL_T64x64;
        return takes(MX4GEMM_KERNEL_T128x128) ? MX4GEMM_KERNEL_T128x128 : -22;
    }
    int best = -22;
    float least = 0.0f;
    for (const Mx4Large &l : kLarge) {
        const double tiles = row_tiles(l.bm) * (double)ceil_div_ll(N, l.bn);
        if (!takes(l.kernel))
            continue;
        const float rounds = (float)ceil_div_ll((long long)(tiles + 0.999), cus);
        const float steps = (float)ceil_div_ll(K, 256);
        const float lone = 4.5f + steps * l.wait;
        const float busy = 2.5f + rounds * (l.fixed + steps * l.step);
        const float cost = lone > busy ? lone : busy;
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
    return !fits_launch((double)mx4_row_tiles(M, groups, 256) * (double)ceil_div_ll(N, 256), 512);
}

int launch_mx4(Mx4Params p, hipStream_t s)
{
    if (too_many_tiles(p.M, p.N, p.groups))
        return -22;
    int cus = 0;
    const int st = current_cus(&cus);
    if (st != 0)
        return st;
    const bool direct = (((uintptr_t)p.A | (uintptr_t)p.B) & 15) == 0 && p.lda % 16 == 0 &&
                        p.ldb % 16 == 0 && p.strideB % 16 == 0 && p.K % 32 == 0 &&
                        p.lda < kMaxTileLd && p.ldb < kMaxTileLd && p.K > 0;
    const int kernel = choose_mx4(p.M, p.N, p.K, p.groups, direct, cus);
    if (kernel < 0)
        return kernel;
    const Mx4Variant v = variant_of(kernel);
    p.tiles_m = (int)mx4_row_tiles(p.M, p.groups, v.bm);
    p.tiles_n = (int)ceil_div_ll(p.N, v.bn);
    p.band = p.groups ? group_band(p.M, p.groups, v.bm) : 8;
    void *args[] = {&p};
    return (int)hipLaunchKernel((const void *)v.fn,
                                dim3((unsigned)((long long)p.tiles_m * p.tiles_n)),
                                dim3(v.threads), args, 0, s);
}

bool k_ok(int K) { return K >= 0 && K <= INT32_MAX - 65536; }
int row_bytes(int K) { return K > 2 ? (K + 1) / 2 : 1; }
bool words(const void *scale) { return scale != nullptr && ((uintptr_t)scale & 3) == 0; }

} // namespace

extern "C" int mx4_quantize_rows(int M, int K, const void *X, int x_type, int ldx,
                                 unsigned char *Q, int ldq, unsigned char *scale, int lds,
                                 sgemm_stream_t stream)
{
    if (M < 0) return -1301;
    if (!k_ok(K)) return -1302;
    if (!c_type_ok(x_type)) return -1304;
    if (ldx < (K > 1 ? K : 1)) return -1305;
    if (ldq < row_bytes(K)) return -1307;
    if (lds < (M > 1 ? M : 1)) return -1309;
    if (M == 0 || K == 0)
        return 0;
    if (X == nullptr) return -1303;
    if (Q == nullptr) return -1306;
    if (!words(scale)) return -1308;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (x_type == SGEMM_F32)
        return launch_mx4_quantize<float>(M, K, X, ldx, Q, ldq, scale, lds, s);
    if (x_type == SGEMM_F16)
        return launch_mx4_quantize<_Float16>(M, K, X, ldx, Q, ldq, scale, lds, s);
    return launch_mx4_quantize<__bf16>(M, K, X, ldx, Q, ldq, scale, lds, s);
}

extern "C" int mx4_dequantize_rows(int M, int K, const unsigned char *Q, int ldq,
                                   const unsigned char *scale, int lds, void *Y, int y_type,
                                   int ldy, sgemm_stream_t stream)
{
    if (M < 0) return -1401;
    if (!k_ok(K)) return -1402;
    if (ldq < row_bytes(K)) return -1404;
    if (lds < (M > 1 ? M : 1)) return -1406;
    if (!c_type_ok(y_type)) return -1408;
    if (ldy < (K > 1 ? K : 1)) return -1409;
    if (M == 0 || K == 0)
        return 0;
    if (Q == nullptr) return -1403;
    if (!words(scale)) return -1405;
    if (Y == nullptr) return -1407;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (y_type == SGEMM_F32)
        return launch_mx4_dequantize<float>(M, K, Q, ldq, scale, lds, Y, ldy, s);
    if (y_type == SGEMM_F16)
        return launch_mx4_dequantize<_Float16>(M, K, Q, ldq, scale, lds, Y, ldy, s);
    return launch_mx4_dequantize<__bf16>(M, K, Q, ldq, scale, lds, Y, ldy, s);
}

extern "C" int mx4gemm(int M, int N, int K, const unsigned char *A, int lda,
                       const unsigned char *scaleA, int ldsa, const unsigned char *B, int ldb,
                       const unsigned char *scaleB, int ldsb, const float *bias, void *C,
                       int c_type, int ldc, sgemm_stream_t stream)
{
    if (M < 0) return -1501;
    if (N < 0) return -1502;
    if (!k_ok(K)) return -1503;
    if (lda < row_bytes(K)) return -1505;
    if (ldsa < M) return -1507;
    if (ldb < row_bytes(K)) return -1509;
    if (ldsb < N) return -1511;
    if (!c_type_ok(c_type)) return -1514;
    if (ldc < (N > 1 ? N : 1)) return -1515;
    if (M == 0 || N == 0)
        return 0;
    if (K > 0 && A == nullptr) return -1504;
    if (K > 0 && !words(scaleA)) return -1506;
    if (K > 0 && B == nullptr) return -1508;
    if (K > 0 && !words(scaleB)) return -1510;
    if (C == nullptr) return -1513;
    Mx4Params p{};
    p.A = reinterpret_cast<const signed char *>(A);
    p.B = reinterpret_cast<const signed char *>(B);
    p.sA = reinterpret_cast<const uint32_t *>(scaleA);
    p.sB = reinterpret_cast<const uint32_t *>(scaleB);
    p.bias = bias;
    p.C = C;
    p.M = M;
    p.N = N;
    p.K = K;
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = ldc;
    p.ldsa = ldsa;
    p.ldsb = ldsb;
    p.type = c_type;
    return launch_mx4(p, static_cast<hipStream_t>(stream));
}

extern "C" int mx4gemm_grouped(int M, int N, int K, int groups, const int *offsets,
                               const unsigned char *A, int lda, const unsigned char *scaleA,
                               int ldsa, const unsigned char *B, int ldb, long long strideB,
                               const unsigned char *scaleB, int ldsb, long long strideSB,
                               const float *bias, void *C, int c_type, int ldc,
                               sgemm_stream_t stream)
{
    if (M < 0) return -1601;
    if (N < 0) return -1602;
    if (!k_ok(K)) return -1603;
    if (groups < 0 || groups > kMaxGroups) return -1604;
    if (lda < row_bytes(K)) return -1607;
    if (ldsa < M) return -1609;
    if (ldb < row_bytes(K)) return -1611;
    if (strideB < 0) return -1612;
    if (ldsb < N) return -1614;
    if (strideSB < 0 || strideSB % 4 != 0) return -1615;
    if (!c_type_ok(c_type)) return -1618;
    if (ldc < (N > 1 ? N : 1)) return -1619;
    if (M == 0 || N == 0 || groups == 0)
        return 0;
    if (offsets == nullptr) return -1605;
    if (K > 0 && A == nullptr) return -1606;
    if (K > 0 && !words(scaleA)) return -1608;
    if (K > 0 && B == nullptr) return -1610;
    if (K > 0 && !words(scaleB)) return -1613;
    if (C == nullptr) return -1617;
    Mx4Params p{};
    p.A = reinterpret_cast<const signed char *>(A);
    p.B = reinterpret_cast<const signed char *>(B);
    p.sA = reinterpret_cast<const uint32_t *>(scaleA);
    p.sB = reinterpret_cast<const uint32_t *>(scaleB);
    p.bias = bias;
    p.C = C;
    p.offsets = offsets;
    p.strideB = strideB;
    p.strideSB = strideSB / 4;
    p.M = M;
    p.N = N;
    p.K = K;
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = ldc;
    p.ldsa = ldsa;
    p.ldsb = ldsb;
    p.type = c_type;
    p.groups = groups;
    return launch_mx4(p, static_cast<hipStream_t>(stream));
}

extern "C" int mx4gemm_select_kernel(int M, int N, int K, int groups, int aligned, int num_cus)
{
    if (M < 0) return -1501;
    if (N < 0) return -1502;
    if (!k_ok(K)) return -1503;
    if (groups < 0 || groups > kMaxGroups) return -1604;
    if (too_many_tiles(M, N, groups)) return -22;
    return choose_mx4(M, N, K, groups, aligned != 0 && K > 0 && K % 32 == 0,
                      num_cus > 1 ? num_cus : 1);
}
