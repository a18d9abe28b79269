// The root-mean-square norm with the residual's addition, in the input's type
// or in 8-bit integers, and its gradients (norm.h), for MI355X (gfx950).

#include "ops_common.h"

#include "norm.h"

#include <type_traits>

namespace {

template <typename T> constexpr int kVec = 16 / (int)sizeof(T); // elements of 16 bytes

// A chunk of 16 bytes of a row as floats, zeros behind its last element.
template <typename T>
__device__ __forceinline__ void load_row(const T *row, int k, int K, float (&f)[kVec<T>])
{
    if (k + kVec<T> <= K) {
        unpack<T>(load16(row + k), f);
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            f[i] = k + i < K ? (float)row[k + i] : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store_row(T *row, int k, int K, const float (&f)[kVec<T>])
{
    typedef T tv __attribute__((ext_vector_type(kVec<T>)));
    tv v;
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
        v[i] = (T)f[i];
    if (k + kVec<T> <= K) {
        store16(row + k, __builtin_bit_cast(i32x4, v));
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (k + i < K)
                row[k + i] = v[i];
    }
}

// The weights of a chunk, as load_row takes its elements.
template <int VEC>
__device__ __forceinline__ void load_weights(const float *w, int k, int K, float (&f)[VEC])
{
    if (k + VEC <= K) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const f32x4 v = __builtin_bit_cast(f32x4, load16(w + k + i));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[i + e] = v[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            f[i] = k + i < K ? w[k + i] : 0.0f;
    }
}

// N values of every thread added over the NT threads of a row, in a fixed order,
// and the largest of their peaks. `shared`: (N + 1) * NT / 64 words where NT > 64,
// which the caller's last row has left.
template <int NT, int N>
__device__ __forceinline__ void over_row(float (&v)[N], uint32_t &peak, uint32_t *shared)
{
#pragma unroll
    for (int d = 1; d < (NT < 64 ? NT : 64); d <<= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor(v[i], d);
        peak = max(peak, (uint32_t)__shfl_xor((int)peak, d));
    }
    if constexpr (NT > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                shared[wave * (N + 1) + i] = __builtin_bit_cast(uint32_t, v[i]);
            shared[wave * (N + 1) + N] = peak;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float f = __uint_as_float(shared[w * (N + 1) + i]);
                v[i] = w == 0 ? f : v[i] + f;
            }
            peak = max(peak, shared[w * (N + 1) + N]);
        }
    }
}

__device__ __forceinline__ float rstd_of(float squares, int K, float eps)
{
    return 1.0f / __builtin_sqrtf(squares / (float)K + eps);
}

struct NormParams {
    const void *X, *R;
    const float *weight;
    void *H, *out;
    float *scale;
    long long ldx, ldr, ldh, ldo;
    int M, K;
    float eps;
};

// NT threads a row (below 256: 256 / NT rows a workgroup), which hold the row's
// h in registers, CH chunks of 16 bytes each, between its sums and its output:
// one pass over memory. CH = 0: rows of any length, read twice (h from H where
// it is kept, which each thread wrote itself). Bound by memory: 16384 x 4096 in
// bf16 to 8 bits takes 92 us (5.1 TB/s, a large copy's rate), 16384 x 2048 in
// bf16 45 us (a part of it cached); 4 x 4096 3.5 us, a launch, one trip to
// memory and one meeting of the row's waves, with the sum and the largest value
// at once.
template <typename T, typename Out, int NT, int CH>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_kernel(NormParams p)
{
    constexpr int VEC = kVec<T>;
    constexpr bool I8 = std::is_same<Out, signed char>::value;
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, WAVES = NT / 64;
    static_assert(NT <= 64 || ROWS == 1, "a row is a part of a wave, a wave or a workgroup");
    __shared__ uint32_t shared[NT > 64 ? 2 * WAVES : 1];
    const int t = threadIdx.x % NT;
    const long long m = (long long)blockIdx.x * ROWS + threadIdx.x / NT;
    if (m >= p.M)
        return; // (all threads of a row, and with NT > 64 never)
    const T *x = static_cast<const T *>(p.X) + m * p.ldx;
    const T *r = p.R ? static_cast<const T *>(p.R) + m * p.ldr : nullptr;
    T *hrow = p.H ? static_cast<T *>(p.H) + m * p.ldh : nullptr;
    Out *out = static_cast<Out *>(p.out) + m * p.ldo;

    auto sum_of = [&](int k, float (&h)[VEC]) {
        load_row<T>(x, k, p.K, h);
        if (r) {
            float f[VEC];
            load_row<T>(r, k, p.K, f);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                h[i] = (float)(T)(h[i] + f[i]);
        }
    };
    float squares[1] = {0.0f};
    uint32_t peak = 0; // of |t| as ordered integers: NaN above infinity
    auto take = [&](int k, const float (&h)[VEC], const float (&w)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            squares[0] = __builtin_fmaf(h[i], h[i], squares[0]);
        if constexpr (I8)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                peak = max(peak, __builtin_bit_cast(uint32_t, h[i] * w[i]) & 0x7fffffffu);
    };
    // The weights are loaded along with the row, one trip to memory, where there
    // are registers for both.
    constexpr bool EARLY = CH > 0 && CH * VEC <= 32;
    float held[CH > 0 ? CH : 1][VEC], weights[EARLY ? CH : 1][VEC];
    if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            sum_of((c * NT + t) * VEC, held[c]);
            if constexpr (EARLY)
                load_weights<VEC>(p.weight, (c * NT + t) * VEC, p.K, weights[c]);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if constexpr (!EARLY && I8)
                load_weights<VEC>(p.weight, (c * NT + t) * VEC, p.K, weights[0]);
            take((c * NT + t) * VEC, held[c], weights[EARLY ? c : 0]);
        }
    } else {
        for (int k = t * VEC; k < p.K; k += NT * VEC) {
            float h[VEC], w[VEC] = {};
            sum_of(k, h);
            if constexpr (I8)
                load_weights<VEC>(p.weight, k, p.K, w);
            if (hrow)
                store_row<T>(hrow, k, p.K, h);
            take(k, h, w);
        }
    }
    over_row<NT, 1>(squares, peak, shared);
    const float rstd = rstd_of(squares[0], p.K, p.eps);
    float s = 0.0f, inv = 0.0f;
    bool finite = true;
    if constexpr (I8) {
        const float top = __builtin_bit_cast(float, peak);
        finite = peak < 0x7f800000u;
        s = finite ? __builtin_fmaxf(top / 127.0f, kLeastScale) : __builtin_nanf("");
        inv = 1.0f / s;
        if (t == 0)
            p.scale[m] = s * rstd;
    }

    auto put = [&](int k, const float (&h)[VEC], const float (&w)[VEC]) {
        if constexpr (I8) {
            uint32_t b[VEC / 4];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const uint32_t q =
                    finite ? (uint32_t)quantize_one(h[i] * w[i], s, inv) & 0xffu : 0u;
                b[i / 4] = i % 4 == 0 ? q : b[i / 4] | q << (8 * (i % 4));
            }
            if (k + VEC <= p.K) {
                if constexpr (VEC == 4)
                    *reinterpret_cast<i32_any *>(out + k) = (int)b[0];
                else
                    *reinterpret_cast<i32x2_any *>(out + k) = i32x2_any{(int)b[0], (int)b[1]};
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (k + i < p.K)
                        out[k + i] = (signed char)(b[i / 4] >> (8 * (i % 4)));
            }
        } else {
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                y[i] = h[i] * w[i] * rstd;
            store_row<T>(out, k, p.K, y);
        }
    };
    if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * NT + t) * VEC;
            if constexpr (!EARLY)
                load_weights<VEC>(p.weight, k, p.K, weights[0]);
            if (k >= p.K)
                continue;
            if (hrow) // (behind the meeting, which would wait for it)
                store_row<T>(hrow, k, p.K, held[c]);
            put(k, held[c], weights[EARLY ? c : 0]);
        }
    } else {
        for (int k = t * VEC; k < p.K; k += NT * VEC) {
            float h[VEC], w[VEC];
            load_weights<VEC>(p.weight, k, p.K, w);
            if (hrow)
                load_row<T>(hrow, k, p.K, h);
            else
                sum_of(k, h);
            put(k, h, w);
        }
    }
}

typedef void (*NormFn)(NormParams);

template <typename T, bool I8>
int launch_norm(NormParams p, hipStream_t s)
{
    typedef typename std::conditional<I8, signed char, T>::type Out;
    const long long chunks = ceil_div_ll(p.K, kVec<T>);
    NormFn fn;
    int threads = 256, rows = 1;
    if (chunks <= 8) {
        fn = norm_kernel<T, Out, 8, 1>;
        rows = 32;
    } else if (chunks <= 16) {
        fn = norm_kernel<T, Out, 16, 1>;
        rows = 16;
    } else if (chunks <= 32) {
        fn = norm_kernel<T, Out, 32, 1>;
        rows = 8;
    } else if (chunks <= 64) {
        fn = norm_kernel<T, Out, 64, 1>;
        rows = 4;
    } else if (chunks <= 256) {
        // (A wave with four chunks a lane: 16384 x 2048 in bf16 62 us against 52,
        // 64 x 2048 7.8 against 4.0.)
        fn = norm_kernel<T, Out, 256, 1>;
    } else if (chunks <= 512 && p.M <= 1024) {
        // Few rows: half the work a thread (4 x 4096 in bf16: 3.9 us against 5.3;
        // 16384 rows 104 against 99).
        fn = norm_kernel<T, Out, 512, 1>;
        threads = 512;
    } else if (chunks <= 512) {
        fn = norm_kernel<T, Out, 256, 2>;
    } else if (chunks <= 1024) {
        // From here on as many threads as leave each two chunks, or more with
        // 1024: a row is one trip to memory, and its arithmetic is short. 16 x 8192
        // in bf16 with int8 out 5.3 us against 7.5 of 256 threads with four, 4096
        // rows 44 against 48; slower at worst for 1024 x 8192 in fp32, 21.3
        // against 19.9.
        fn = norm_kernel<T, Out, 512, 2>;
        threads = 512;
    } else if (chunks <= 2048) {
        // (256 threads with eight: 16 x 14915 in bf16 8.2 us against 15.6,
        // 4096 x 16384 121 against 143.)
        fn = norm_kernel<T, Out, 1024, 2>;
        threads = 1024;
    } else if (chunks <= 4096) {
        // (With eight: 16 x 30000 in bf16 9.4 us against 15.1, 2048 rows 121
        // against 164.)
        fn = norm_kernel<T, Out, 1024, 4>;
        threads = 1024;
    } else if (chunks <= 8192) {
        fn = norm_kernel<T, Out, 1024, 8>;
        threads = 1024;
    } else {
        fn = norm_kernel<T, Out, 1024, 0>;
        threads = 1024;
    }
    // A launch holds fewer than 2^32 work-items.
    const long long most = (1 << 21) * (long long)rows;
    const int M = p.M;
    for (long long m0 = 0; m0 < M; m0 += most) {
        NormParams q = p;
        q.M = (int)(M - m0 < most ? M - m0 : most);
        q.X = static_cast<const T *>(p.X) + m0 * p.ldx;
        q.R = p.R ? static_cast<const T *>(p.R) + m0 * p.ldr : nullptr;
        q.H = p.H ? static_cast<T *>(p.H) + m0 * p.ldh : nullptr;
        q.out = static_cast<Out *>(p.out) + m0 * p.ldo;
        q.scale = I8 ? p.scale + m0 : nullptr;
        void *args[] = {&q};
        const hipError_t e = hipLaunchKernel((const void *)fn,
                                             dim3((unsigned)ceil_div_ll(q.M, rows)), dim3(threads),
                                             args, 0, s);
        if (e != hipSuccess)
            return (int)e;
    }
    return 0;
}

// K == 0: nothing but the scales of empty rows.
__global__ void __launch_bounds__(256) empty_rows_kernel(float *scale, int M)
{
    for (long long m = blockIdx.x * 256LL + threadIdx.x; m < M; m += gridDim.x * 256LL)
        scale[m] = kLeastScale;
}

// ---------------------------------------------------------------------------
// The gradients
// ---------------------------------------------------------------------------

struct GradParams {
    const void *dY, *H, *dH;
    const float *weight;
    void *dX;
    float *partial; // a row of K sums for every row group, or NULL
    long long lddy, ldh, lddh, lddx;
    int M, K;
    float eps;
};

// As norm_kernel, but a row group (NT threads) takes every gridDim.x * ROWS-th
// row, so that it can add up its rows' part of dweight in registers; the second
// kernel adds the groups' sums. Rows come in a fixed order, so do the sums. Bound
// by memory: 16384 x 2048 in bf16 takes 57 us (4.7 TB/s), 500 x 1000 in fp32 8.6,
// of which the second kernel 5.
template <typename T, int NT, int CH>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_grad_kernel(GradParams p)
{
    constexpr int VEC = kVec<T>;
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, WAVES = NT / 64;
    __shared__ uint32_t shared[2][NT > 64 ? 3 * WAVES : 1]; // of rows by parity
    const int t = threadIdx.x % NT;
    const long long group = (long long)blockIdx.x * ROWS + threadIdx.x / NT;
    float w[CH][VEC], dw[CH][VEC] = {};
#pragma unroll
    for (int c = 0; c < CH; ++c)
        load_weights<VEC>(p.weight, (c * NT + t) * VEC, p.K, w[c]);
    int turn = 0;
    for (long long m = group; m < p.M; m += (long long)gridDim.x * ROWS) {
        const T *dy = static_cast<const T *>(p.dY) + m * p.lddy;
        const T *h = static_cast<const T *>(p.H) + m * p.ldh;
        const T *dh = p.dH ? static_cast<const T *>(p.dH) + m * p.lddh : nullptr;
        T *dx = static_cast<T *>(p.dX) + m * p.lddx;
        float g[CH][VEC], x[CH][VEC], d[CH][VEC] = {}, v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            load_row<T>(dy, (c * NT + t) * VEC, p.K, g[c]);
            load_row<T>(h, (c * NT + t) * VEC, p.K, x[c]);
            if (dh)
                load_row<T>(dh, (c * NT + t) * VEC, p.K, d[c]);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[0] = __builtin_fmaf(x[c][i], x[c][i], v[0]);
                v[1] = __builtin_fmaf(w[c][i] * g[c][i], x[c][i], v[1]);
            }
        uint32_t none = 0;
        over_row<NT, 2>(v, none, shared[turn ^= 1]);
        const float rstd = rstd_of(v[0], p.K, p.eps);
        const float along = v[1] / (float)p.K * rstd * rstd;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = (c * NT + t) * VEC;
            if (k >= p.K)
                continue;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                dw[c][i] = __builtin_fmaf(g[c][i], x[c][i] * rstd, dw[c][i]);
                d[c][i] = __builtin_fmaf(rstd, w[c][i] * g[c][i] - x[c][i] * along, d[c][i]);
            }
            store_row<T>(dx, k, p.K, d[c]);
        }
    }
    if (p.partial == nullptr)
        return;
    float *to = p.partial + group * p.K;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int k = (c * NT + t) * VEC + i;
            if (k < p.K)
                to[k] = dw[c][i];
        }
}

// dweight[k] = sum of the row groups' sums: 16 columns a workgroup, the groups
// over 64 threads each (1024 groups of 2048 columns: 4.9 us; 32 columns over 32
// threads 11).
constexpr int kAddThreads = 1024, kAddColumns = 16;

__global__ void __launch_bounds__(kAddThreads)
norm_grad_add_kernel(const float *partial, int groups, int K, float *dweight)
{
    constexpr int PARTS = kAddThreads / kAddColumns;
    __shared__ float part[PARTS][kAddColumns + 1];
    const int c = threadIdx.x % kAddColumns, at = threadIdx.x / kAddColumns;
    const int k = blockIdx.x * kAddColumns + c;
    float sum = 0.0f;
    if (k < K) {
        int g = at;
        for (; g + 3 * PARTS < groups; g += 4 * PARTS) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = partial[(long long)(g + i * PARTS) * K + k];
            sum += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; g < groups; g += PARTS)
            sum += partial[(long long)g * K + k];
    }
    part[at][c] = sum;
    __syncthreads();
    for (int n = PARTS / 2; n > 0; n >>= 1) {
        if (at < n)
            part[at][c] += part[at + n][c];
        __syncthreads();
    }
    if (at == 0 && k < K)
        dweight[k] = part[0][c];
}

typedef void (*GradFn)(GradParams);

struct GradPlan {
    GradFn fn;
    int threads, rows; // a workgroup
    int blocks;
};

static_assert(RMS_NORM_GRAD_MAX_K <= 1024 * 2 * kVec<_Float16> &&
                  RMS_NORM_GRAD_MAX_K <= 1024 * 4 * kVec<float>,
              "the widest kernels hold a row");

template <typename T>
GradPlan grad_plan_of(int M, int K)
{
    const long long chunks = ceil_div_ll(K, kVec<T>);
    GradPlan g;
    if (chunks <= 16)
        g = {norm_grad_kernel<T, 16, 1>, 256, 16, 0};
    else if (chunks <= 64)
        g = {norm_grad_kernel<T, 64, 1>, 256, 4, 0};
    else if (chunks <= 128)
        g = {norm_grad_kernel<T, 64, 2>, 256, 4, 0};
    else if (chunks <= 256)
        g = {norm_grad_kernel<T, 256, 1>, 256, 1, 0};
    else if (chunks <= 512)
        g = {norm_grad_kernel<T, 256, 2>, 256, 1, 0};
    else if (chunks <= 1024)
        g = {norm_grad_kernel<T, 512, 2>, 512, 1, 0};
    else if (chunks <= 2048 || sizeof(T) == 2)
        g = {norm_grad_kernel<T, 1024, 2>, 1024, 1, 0};
    else if constexpr (sizeof(T) == 4)
        g = {norm_grad_kernel<T, 1024, 4>, 1024, 1, 0};
    const long long blocks = ceil_div_ll(M, g.rows);
    g.blocks = (int)(blocks < 1024 ? blocks : 1024);
    return g;
}

GradPlan grad_plan(int M, int K, int type)
{
    return type == SGEMM_F32   ? grad_plan_of<float>(M, K)
           : type == SGEMM_F16 ? grad_plan_of<_Float16>(M, K)
                               : grad_plan_of<__bf16>(M, K);
}

int norm_checks(int base, int M, int K, const void *X, int type, int ldx, const void *R, int ldr,
                const float *weight, float eps, const void *H, int ldh, const void *out, int ldo)
{
    if (M < 0) return -(base + 1);
    if (K < 0 || K > INT32_MAX - 65536) return -(base + 2);
    if (!c_type_ok(type)) return -(base + 4);
    const int row = K > 1 ? K : 1;
    if (ldx < row) return -(base + 5);
    if (R != nullptr && ldr < row) return -(base + 7);
    if (!(eps >= 0.0f)) return -(base + 9);
    if (H != nullptr && ldh < row) return -(base + 11);
    if (ldo < row) return -(base + 13);
    if (M == 0 || K == 0)
        return 0;
    if (X == nullptr) return -(base + 3);
    if (weight == nullptr) return -(base + 8);
    if (out == nullptr) return -(base + 12);
    return 0;
}

} // namespace

extern "C" int rms_norm(int M, int K, const void *X, int type, int ldx, const void *R, int ldr,
                        const float *weight, float eps, void *H, int ldh, void *Y, int ldy,
                        sgemm_stream_t stream)
{
    const int st = norm_checks(1000, M, K, X, type, ldx, R, ldr, weight, eps, H, ldh, Y, ldy);
    if (st != 0 || M == 0 || K == 0)
        return st;
    const NormParams p{X, R, weight, H, Y, nullptr, ldx, ldr, ldh, ldy, M, K, eps};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (type == SGEMM_F32)
        return launch_norm<float, false>(p, s);
    if (type == SGEMM_F16)
        return launch_norm<_Float16, false>(p, s);
    return launch_norm<__bf16, false>(p, s);
}

extern "C" int rms_norm_i8(int M, int K, const void *X, int type, int ldx, const void *R, int ldr,
                           const float *weight, float eps, void *H, int ldh, signed char *Q,
                           int ldq, float *scale, sgemm_stream_t stream)
{
    const int st = norm_checks(1100, M, K, X, type, ldx, R, ldr, weight, eps, H, ldh, Q, ldq);
    if (st != 0 || M == 0)
        return st;
    if (scale == nullptr) return -1114;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) {
        const long long blocks = ceil_div_ll(M, 256);
        void *args[] = {&scale, &M};
        return (int)hipLaunchKernel((const void *)empty_rows_kernel,
                                    dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256),
                                    args, 0, s);
    }
    const NormParams p{X, R, weight, H, Q, scale, ldx, ldr, ldh, ldq, M, K, eps};
    if (type == SGEMM_F32)
        return launch_norm<float, true>(p, s);
    if (type == SGEMM_F16)
        return launch_norm<_Float16, true>(p, s);
    return launch_norm<__bf16, true>(p, s);
}

extern "C" size_t rms_norm_grad_workspace_size(int M, int K, int type)
{
    if (M < 0 || K < 0 || K > RMS_NORM_GRAD_MAX_K || !c_type_ok(type))
        return 0;
    const GradPlan g = grad_plan(M, K, type);
    return (size_t)g.blocks * g.rows * K * sizeof(float);
}

extern "C" int rms_norm_grad(int M, int K, const void *dY, int type, int lddy, const void *H,
                             int ldh, const float *weight, float eps, const void *dH, int lddh,
                             void *dX, int lddx, float *dweight, void *workspace,
                             size_t workspace_bytes, sgemm_stream_t stream)
{
    if (M < 0) return -1201;
    if (K < 0 || K > RMS_NORM_GRAD_MAX_K) return -1202;
    if (!c_type_ok(type)) return -1204;
    const int row = K > 1 ? K : 1;
    if (lddy < row) return -1205;
    if (ldh < row) return -1207;
    if (!(eps >= 0.0f)) return -1209;
    if (dH != nullptr && lddh < row) return -1211;
    if (lddx < row) return -1213;
    if (K == 0 || (M == 0 && dweight == nullptr))
        return 0;
    if (M > 0) {
        if (dY == nullptr) return -1203;
        if (H == nullptr) return -1206;
        if (weight == nullptr) return -1208;
        if (dX == nullptr) return -1212;
    }
    const size_t need = dweight ? rms_norm_grad_workspace_size(M, K, type) : 0;
    if (need > 0 && (workspace == nullptr || ((uintptr_t)workspace & 15))) return -1215;
    if (workspace_bytes < need) return -1216;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const GradPlan g = grad_plan(M, K, type);
    float *partial = dweight ? static_cast<float *>(workspace) : nullptr;
    if (M > 0) {
        GradParams p{dY, H, dH, weight, dX, partial, lddy, ldh, lddh, lddx, M, K, eps};
        void *args[] = {&p};
        const hipError_t e = hipLaunchKernel((const void *)g.fn, dim3((unsigned)g.blocks),
                                             dim3(g.threads), args, 0, s);
        if (e != hipSuccess)
            return (int)e;
    }
    if (dweight == nullptr)
        return 0;
    int groups = g.blocks * g.rows;
    void *args[] = {&partial, &groups, &K, &dweight};
    return (int)hipLaunchKernel((const void *)norm_grad_add_kernel,
                                dim3((unsigned)ceil_div_ll(K, kAddColumns)), dim3(kAddThreads), args, 0, s);
}
