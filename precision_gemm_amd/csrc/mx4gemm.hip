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

template <typename T>
__device__ __forceinline__ void load8(const T *row, int k, int K, float (&f)[8])
{
    if (k + 8 <= K) {
        constexpr int VEC = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 8; i += VEC) {
            float v[VEC];
            unpack<T>(load16(row + k + i), v);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                f[i + e] = v[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = k + i < K ? (float)row[k + i] : 0.0f;
    }
}

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

// 32 rows (RW of each of the 32 / RW waves) of 512 elements a workgroup, so that
// the scales leave as whole lines of neighbouring rows.
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
    float f[RW][8];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const long long m = m0 + wave * RW + r;
        load8<T>(X + (m < M ? m : M - 1) * ldx, k, K, f[r]);
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const long long m = m0 + wave * RW + r;
        uint32_t peak = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            peak = max(peak, __builtin_bit_cast(uint32_t, f[r][i]) & 0x7fffffffu);
        peak = max(peak, (uint32_t)__shfl_xor((int)peak, 1));
        peak = max(peak, (uint32_t)__shfl_xor((int)peak, 2));
        const int field = (int)(peak >> 23);
        const bool finite = field < 255;
        const int byte = finite ? max(field - 2, 0) : 255;
        const float up = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
        uint32_t codes = 0;
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][0] * up, f[r][1] * up, 1.0f, 0);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][2] * up, f[r][3] * up, 1.0f, 1);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][4] * up, f[r][5] * up, 1.0f, 2);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[r][6] * up, f[r][7] * up, 1.0f, 3);
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
    const Fn fn = few ? mx4_quantize_kernel<T, 4, 1> : mx4_quantize_kernel<T, 32, 8>;
    const int rows = few ? 4 : 32;
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

template <typename T>
__global__ void __launch_bounds__(256)
mx4_dequantize_kernel(int M, int K, const unsigned char *Q, long long ldq,
                      const unsigned char *scale, long long lds, T *Y, long long ldy)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k = blockIdx.x * 512 + 8 * lane;
    if (k >= K)
        return;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const long long m = (long long)blockIdx.y * 8 + 2 * wave + r;
        if (m >= M)
            return;
        const unsigned char *q = Q + m * ldq;
        const float s = scale_of(scale[((k >> 7) * lds + m) * 4 + ((k >> 5) & 3)]);
        uint32_t codes = 0;
        if (k + 8 <= K) {
            codes = (uint32_t)*reinterpret_cast<const i32_any *>(q + (k >> 1));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k + 2 * i < K)
                    codes |= (uint32_t)q[(k >> 1) + i] << (8 * i);
        }
        float f[8];
        auto pair = [&](f32x2 v, int i) {
            f[i] = v[0];
            f[i + 1] = v[1];
        };
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 0), 0);
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 1), 2);
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 2), 4);
        pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 3), 6);
        T *y = Y + m * ldy + k;
        if (k + 8 <= K) {
            store4<T>(y, f32x4{f[0], f[1], f[2], f[3]});
            store4<T>(y + 4, f32x4{f[4], f[5], f[6], f[7]});
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < K)
                    y[i] = (T)f[i];
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
    most = 8 * (most < 1 ? 1 : most < 65535 ? most : 65535);
    for (long long m0 = 0; m0 < M; m0 += most) {
        int n = (int)(M - m0 < most ? M - m0 : most);
        const unsigned char *q = Q + m0 * ldq, *sc = scale + 4 * m0;
        T *y = static_cast<T *>(Y) + m0 * ldy;
        void *args[] = {&n, &K, &q, &ldq, &sc, &lds, &y, &ldy};
        const hipError_t e = hipLaunchKernel((const void *)mx4_dequantize_kernel<T>,
                                             dim3(columns, (unsigned)ceil_div_ll(n, 8)), dim3(256),
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

// The 16 bytes of a row of K elements from its byte k on (row_chunk), without
// what the last byte holds beyond an odd K.
__device__ __forceinline__ i32x4 mx4_chunk(const signed char *row, int k, int K)
{
    i32x4 v = row_chunk(row, k, (K + 1) >> 1);
    const int last = (K >> 1) - k; // the byte that an odd K ends in
    if ((K & 1) && last >= 0 && last < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i == last >> 2)
                v[i] &= ~(0xf0 << (8 * (last & 3)));
    }
    return v;
}

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

typedef void (*Mx4Fn)(Mx4Params);

struct Mx4Variant {
    Mx4Fn fn;
    int bm, bn, threads;
};

long long mx4_row_tiles(int M, int groups, int bm)
{
    return groups ? most_tiles(M, groups, bm) : ceil_div_ll(M, bm);
}

// (Refused before the device is asked: not even the largest tiles fit a launch.)
bool too_many_tiles(int M, int N, int groups)
{
    return !fits_launch((double)mx4_row_tiles(M, groups, 128) * (double)ceil_div_ll(N, 128), 256);
}

int launch_mx4(Mx4Params p, hipStream_t s)
{
    if (too_many_tiles(p.M, p.N, p.groups))
        return -22;
    int cus = 0;
    const int st = current_cus(&cus);
    if (st != 0)
        return st;
    Mx4Variant v = {mx4_tile_kernel<2>, 128, 128, 256};
    if (mx4_row_tiles(p.M, p.groups, 128) * ceil_div_ll(p.N, 128) < cus)
        v = {mx4_tile_kernel<1>, 64, 64, 256};
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
