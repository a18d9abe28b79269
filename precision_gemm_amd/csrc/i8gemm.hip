// 8-bit integer products with a scale for each token and channel, and the row
// quantization that makes their left operand (i8gemm.h), for MI355X (gfx950).

#include "ops_common.h"

#include "i8gemm.h"

#include <type_traits>

namespace {

// ---------------------------------------------------------------------------
// Row quantization
// ---------------------------------------------------------------------------

constexpr float kLeastScale = 1.17549435e-38f; // 2^-126

// The integer nearest to x / s (ties to even), |x / s| < 127.5. r, from a
// product with the reciprocal, can be one off next to a tie; d = x - r s is
// exact (for r = 0 it is x, for r = +-1 the subtraction of numbers within a
// factor of two, beyond that a multiple of s's last place below 2^24 of them),
// so comparing it with s / 2 (exact: s >= 2^-126) puts r right.
__device__ __forceinline__ int quantize_one(float x, float s, float inv)
{
    float r = __builtin_rintf(x * inv);
    const float d = __builtin_fmaf(-r, s, x);
    const float half = 0.5f * s;
    const float a = __builtin_fabsf(d);
    const bool odd = ((int)r) & 1;
    if (a > half || (a == half && odd))
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

// NT threads a row (NT = 64: four rows a workgroup, one a wave), which hold
// the row in registers, CH chunks of 16 bytes each, between its maximum and
// its rounding: one pass over memory. CH = 0: rows of any length, read twice.
template <typename T, int NT, int CH>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
i8_quantize_kernel(int M, int K, const T *X, int ldx, signed char *Q, int ldq, float *scale)
{
    constexpr int VEC = 16 / sizeof(T);
    constexpr int ROWS = NT == 64 ? 4 : 1, WAVES = NT / 64;
    const int t = NT == 64 ? threadIdx.x & 63 : threadIdx.x;
    const long long m = (long long)blockIdx.x * ROWS + (NT == 64 ? threadIdx.x >> 6 : 0);
    if (m >= M)
        return; // (whole waves, and with NT > 64 never)
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
    for (int d = 1; d < 64; d <<= 1)
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
    if (chunks <= 64) {
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
    int groups;  // 0: one product
    int tiles_n; // grid: row tiles x tiles_n
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
__device__ __forceinline__ bool i8_tile_of(const I8Params &p, int slot, int tn, I8Tile &t)
{
    t.n0 = tn * BN;
    t.A = p.A;
    t.B = p.B;
    t.sA = p.sA;
    t.sB = p.sB;
    t.bias = p.bias;
    t.row0 = 0;
    t.M = p.M;
    t.m0 = slot * BM;
    if (p.groups == 0)
        return true;
    int g, lo;
    if (!find_tile(p.offsets, p.groups, p.M, BM, slot, g, lo, t.M, t.m0))
        return false;
    t.row0 = lo;
    t.A += (long long)lo * p.lda;
    t.sA += lo;
    t.B += g * p.strideB;
    t.sB += (long long)g * p.N;
    if (t.bias)
        t.bias += (long long)g * p.N;
    return true;
}

__device__ __forceinline__ void store_c(const I8Params &p, long long at, float v)
{
    if (p.type == SGEMM_F32)
        static_cast<float *>(p.C)[at] = v;
    else if (p.type == SGEMM_F16)
        static_cast<_Float16 *>(p.C)[at] = (_Float16)v;
    else
        static_cast<__bf16 *>(p.C)[at] = (__bf16)v;
}

// 16 bytes of a row from its byte k on, zeros from byte K on; nothing outside
// the row's K bytes is read.
__device__ __forceinline__ i32x4 row_chunk(const signed char *row, int k, int K)
{
    if (k + 16 <= K)
        return load16(row + k);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K)
            w[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
    return i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// The tile for every call: 64 x 64 of C by four waves, each one 32 x 32
// accumulator of v_mfma_i32_32x32x32_i8 (lane l supplies 16 bytes of row
// l % 32 from k = 16 (l / 32) on; register v of lane l holds row 8 (v / 4) +
// 4 (l / 32) + v % 4, column l % 32). 64-byte K-steps go through registers to
// LDS, so any alignment and any K will do, and zeros behind K leave the sum as
// it is. LDS rows are 64 bytes, four of them one sweep of the 64 banks, so the
// 16-byte chunk index is XORed with row / 4 for conflict-free reads. Rows
// behind M or N repeat the last one and are not stored.
__global__ void __launch_bounds__(256) i8_tile_kernel(I8Params p)
{
    constexpr int BM = 64, BN = 64, BK = 64;
    __shared__ __attribute__((aligned(16))) signed char lds[2][2][64 * BK];
    I8Tile t;
    if (!i8_tile_of<BM, BN>(p, blockIdx.x / p.tiles_n, blockIdx.x % p.tiles_n, t))
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = tid >> 2, c = tid & 3;
    const signed char *ra = t.A + (long long)min(t.m0 + r, t.M - 1) * p.lda;
    const signed char *rb = t.B + (long long)min(t.n0 + r, p.N - 1) * p.ldb;
    const int at = r * BK + 16 * (c ^ ((r >> 2) & 3));
    const int wm = 32 * (wave & 1), wn = 32 * (wave >> 1);

    i32x16 acc = {};
    const int steps = (p.K + BK - 1) / BK;
    i32x4 va = {}, vb = {};
    if (steps > 0) {
        va = row_chunk(ra, 16 * c, p.K);
        vb = row_chunk(rb, 16 * c, p.K);
    }
    for (int s = 0; s < steps; ++s) {
        signed char *la = lds[s & 1][0], *lb = lds[s & 1][1];
        *reinterpret_cast<i32x4 *>(la + at) = va;
        *reinterpret_cast<i32x4 *>(lb + at) = vb;
        __syncthreads();
        if (s + 1 < steps) {
            va = row_chunk(ra, (s + 1) * BK + 16 * c, p.K);
            vb = row_chunk(rb, (s + 1) * BK + 16 * c, p.K);
        }
#pragma unroll
        for (int q = 0; q < BK / 32; ++q) {
            const int o = lane & 31, ch = 2 * q + (lane >> 5);
            const i32x4 fa = *reinterpret_cast<const i32x4 *>(
                la + (wm + o) * BK + 16 * (ch ^ (((wm + o) >> 2) & 3)));
            const i32x4 fb = *reinterpret_cast<const i32x4 *>(
                lb + (wn + o) * BK + 16 * (ch ^ (((wn + o) >> 2) & 3)));
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa, fb, acc, 0, 0, 0);
        }
        // (The next step writes the other stage, which every wave left before
        // this step's barrier.)
    }
    const int n = t.n0 + wn + (lane & 31);
    if (n >= p.N)
        return;
    const float sb = t.sB[n], bias = t.bias ? t.bias[n] : 0.0f;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int m = t.m0 + wm + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
        if (m < t.M)
            store_c(p, (t.row0 + m) * p.ldc + n, (float)acc[v] * t.sA[m] * sb + bias);
    }
}

int launch_i8(I8Params p, hipStream_t s)
{
    const long long tiles_m =
        p.groups ? most_tiles(p.M, p.groups, 64) : ceil_div_ll(p.M, 64);
    const long long tiles_n = ceil_div_ll(p.N, 64);
    if (tiles_m * tiles_n > (1 << 23))
        return -22;
    p.tiles_n = (int)tiles_n;
    void *args[] = {&p};
    return (int)hipLaunchKernel((const void *)i8_tile_kernel, dim3((unsigned)(tiles_m * tiles_n)),
                                dim3(256), args, 0, s);
}

bool c_type_ok(int type) { return type == SGEMM_F32 || type == SGEMM_F16 || type == SGEMM_BF16; }

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
    I8Params p{A, B, scaleA, scaleB, bias, C, nullptr, 0, M, N, K, lda, ldb, ldc, c_type, 0, 0};
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
    if (groups < 0) return -304;
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
               N,   K,   lda,    ldb,    ldc,    c_type, groups,  0};
    return launch_i8(p, static_cast<hipStream_t>(stream));
}
