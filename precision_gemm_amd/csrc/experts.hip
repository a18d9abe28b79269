// Tokens sorted by expert and back, with the gradients (experts.h), for MI355X
// (gfx950).

#include "ops_common.h"

#include "experts.h"

#include <type_traits>

namespace {

// ---------------------------------------------------------------------------
// The sort: a stable counting sort of the slots by expert. Slots without an
// expert get the key `experts`, one past the last.
//
// The slots are cut into at most kMaxBlocks consecutive runs, one a workgroup.
// The first kernel counts each run's keys. In the second, a workgroup adds up
// the counts of the runs before its own and of all experts below each, which
// is the row of its first slot with that expert; its waves, each on a
// consecutive part of the run, then number their slots: a slot's row is its
// expert's next row for the wave plus the lanes before it with the same
// expert. Every count is an integer sum, so the order in which workgroups run
// changes nothing.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBlocks = 256;
constexpr int kLeastRun = 2048;  // slots of a run, but for the last
constexpr int kMaxKeys = EXPERT_SORT_MAX_EXPERTS + 1;

struct SortPlan {
    int blocks, run; // runs of `run` slots (a multiple of 64 * kSortWaves)
};

SortPlan sort_plan(long long slots)
{
    const long long unit = 64 * kSortWaves;
    long long run = ceil_div_ll(ceil_div_ll(slots, kMaxBlocks), unit) * unit;
    if (run < kLeastRun)
        run = kLeastRun;
    const long long blocks = slots > 0 ? ceil_div_ll(slots, run) : 1;
    return SortPlan{(int)blocks, (int)run};
}

template <typename Id>
__device__ __forceinline__ int key_of(const Id *ids, long long i, int experts)
{
    const Id v = ids[i];
    return v >= 0 && v < (Id)experts ? (int)v : experts;
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
expert_count_kernel(const Id *ids, int slots, int experts, int run, int *counts)
{
    __shared__ int hist[kMaxKeys];
    const int keys = experts + 1;
    for (int e = threadIdx.x; e < keys; e += kSortThreads)
        hist[e] = 0;
    __syncthreads();
    const long long lo = (long long)blockIdx.x * run;
    const long long hi = lo + run < slots ? lo + run : slots;
    for (long long i = lo + threadIdx.x; i < hi; i += kSortThreads)
        atomicAdd(&hist[key_of(ids, i, experts)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < keys; e += kSortThreads)
        counts[(long long)blockIdx.x * keys + e] = hist[e];
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads)
expert_place_kernel(const Id *ids, int slots, int experts, int run, const int *counts,
                    int *offsets, int *row_of_slot)
{
    __shared__ int next[kSortWaves * kMaxKeys]; // each wave's next row of every key
    __shared__ int total[kMaxKeys];
    __shared__ int wave_sum[kSortWaves];
    const int keys = experts + 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const long long lo = (long long)blockIdx.x * run;
    const long long hi = lo + run < slots ? lo + run : slots;
    const int part = run / kSortWaves; // a multiple of 64
    const long long wlo = lo + (long long)wave * part;
    const long long whi = wlo + part < hi ? wlo + part : hi;

    for (int i = tid; i < kSortWaves * keys; i += kSortThreads)
        next[i] = 0;
    __syncthreads();
    int *mine = next + wave * keys;
    for (long long i = wlo + lane; i < whi; i += 64)
        atomicAdd(&mine[key_of(ids, i, experts)], 1);
    __syncthreads();

    // Each key: all runs' slots, and those of the runs before this one.
    constexpr int PER = (kMaxKeys + kSortThreads - 1) / kSortThreads;
    int before[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = tid + j * kSortThreads;
        int all = 0, bef = 0;
        if (e < keys) {
            if (counts == nullptr) { // a single run: its own counts are all
                for (int w = 0; w < kSortWaves; ++w)
                    all += next[w * keys + e];
            } else {
                for (int b = 0; b < (int)gridDim.x; ++b) {
                    const int n = counts[(long long)b * keys + e];
                    all += n;
                    bef += b < (int)blockIdx.x ? n : 0;
                }
            }
            total[e] = all;
        }
        before[j] = bef;
    }
    __syncthreads();

    // The rows before each key: an exclusive scan of the totals, 512 at a time.
    int carry = 0;
    int start[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = tid + j * kSortThreads;
        const int n = e < keys ? total[e] : 0;
        int upto = n;
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d);
            if (lane >= d)
                upto += v;
        }
        if (lane == 63)
            wave_sum[wave] = upto;
        __syncthreads();
        int base = carry, sum = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            base += w < wave ? wave_sum[w] : 0;
            sum += wave_sum[w];
        }
        start[j] = base + upto - n;
        carry += sum;
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = tid + j * kSortThreads;
        if (e >= keys)
            continue;
        if (blockIdx.x == 0)
            offsets[e] = start[j];
        int at = start[j] + before[j];
        for (int w = 0; w < kSortWaves; ++w) {
            const int n = next[w * keys + e];
            next[w * keys + e] = at;
            at += n;
        }
    }
    __syncthreads();

    int bits = 0;
    while ((1 << bits) < keys)
        ++bits;
    volatile int *rows = mine; // written by one lane, read by all, in this wave's program order
    for (long long i0 = wlo; i0 < whi; i0 += 64) {
        const long long i = i0 + lane;
        const bool in = i < whi;
        const int e = in ? key_of(ids, i, experts) : 0;
        unsigned long long same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const bool one = (e >> b) & 1;
            const unsigned long long set = __ballot(one);
            same &= one ? set : ~set;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        const int first = in ? rows[e] : 0;
        __builtin_amdgcn_wave_barrier();
        if (in) {
            if (rank == 0)
                rows[e] = first + __builtin_popcountll(same);
            row_of_slot[i] = e < experts ? first + rank : -1;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename Id>
int launch_sort(int slots, int experts, const void *ids_, int *offsets, int *row_of_slot,
                int *counts, hipStream_t s)
{
    const Id *ids = static_cast<const Id *>(ids_);
    SortPlan plan = sort_plan(slots);
    if (plan.blocks == 1)
        counts = nullptr;
    if (counts) {
        void *args[] = {&ids, &slots, &experts, &plan.run, &counts};
        const hipError_t e = hipLaunchKernel((const void *)expert_count_kernel<Id>,
                                             dim3(plan.blocks), dim3(kSortThreads), args, 0, s);
        if (e != hipSuccess)
            return (int)e;
    }
    void *args[] = {&ids, &slots, &experts, &plan.run, &counts, &offsets, &row_of_slot};
    return (int)hipLaunchKernel((const void *)expert_place_kernel<Id>, dim3(plan.blocks),
                                dim3(kSortThreads), args, 0, s);
}

// ---------------------------------------------------------------------------
// Rows to and from the sorted order. `lanes` (a power of two up to 256)
// neighbouring threads take one token's row, 16 bytes each at a time, so 256 /
// lanes tokens share a workgroup. Rows need no alignment.
// ---------------------------------------------------------------------------
struct RowParams {
    const char *in;      // X or dout, or Y of the sum
    const char *in2;     // Y of the gradient
    char *out;
    const int *row_of_slot;
    const float *weights;
    float *dweights;
    long long ld_in, ld_in2, ld_out; // bytes
    int tokens, topk, lanes;
    int bytes; // of a row
};

__device__ __forceinline__ bool valid_row(const RowParams &p, int r)
{
    return (unsigned)r < (unsigned)p.tokens * (unsigned)p.topk;
}

template <int ES>
__global__ void __launch_bounds__(256) expert_gather_kernel(RowParams p)
{
    const int lane = threadIdx.x & (p.lanes - 1);
    const long long t = (long long)blockIdx.x * (256 / p.lanes) + threadIdx.x / p.lanes;
    if (t >= p.tokens)
        return;
    const char *x = p.in + t * p.ld_in;
    const int *rows = p.row_of_slot + t * p.topk;
    for (int b = 16 * lane; b < p.bytes; b += 16 * p.lanes) {
        if (b + 16 <= p.bytes) {
            const i32x4 v = load16(x + b);
            for (int j = 0; j < p.topk; ++j) {
                const int r = rows[j];
                if (valid_row(p, r))
                    store16(p.out + r * p.ld_out + b, v);
            }
        } else {
            typedef std::conditional_t<ES == 4, int, std::conditional_t<ES == 2, short, char>> E;
            const int n = (p.bytes - b) / ES;
            for (int j = 0; j < p.topk; ++j) {
                const int r = rows[j];
                if (valid_row(p, r))
                    for (int i = 0; i < n; ++i)
                        reinterpret_cast<E *>(p.out + r * p.ld_out + b)[i] =
                            reinterpret_cast<const E *>(x + b)[i];
            }
        }
    }
}

// 16 bytes of a row from byte b on as floats, zeros behind the row's end.
template <typename T>
__device__ __forceinline__ void load_chunk(const char *row, int b, int bytes,
                                           float (&x)[16 / sizeof(T)])
{
    constexpr int VEC = 16 / sizeof(T);
    if (b + 16 <= bytes) {
        typedef T tv __attribute__((ext_vector_type(VEC)));
        const tv h = __builtin_bit_cast(tv, load16(row + b));
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            x[i] = (float)h[i];
    } else {
        const T *e = reinterpret_cast<const T *>(row + b);
        const int n = (bytes - b) / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            x[i] = i < n ? (float)e[i] : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store_chunk(char *row, int b, int bytes,
                                            const float (&x)[16 / sizeof(T)])
{
    constexpr int VEC = 16 / sizeof(T);
    if (b + 16 <= bytes) {
        typedef T tv __attribute__((ext_vector_type(VEC)));
        tv h;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            h[i] = (T)x[i];
        store16(row + b, __builtin_bit_cast(i32x4, h));
    } else {
        T *e = reinterpret_cast<T *>(row + b);
        const int n = (bytes - b) / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < n)
                e[i] = (T)x[i];
    }
}

template <typename T>
__global__ void __launch_bounds__(256) expert_combine_kernel(RowParams p)
{
    constexpr int VEC = 16 / sizeof(T);
    const int lane = threadIdx.x & (p.lanes - 1);
    const long long t = (long long)blockIdx.x * (256 / p.lanes) + threadIdx.x / p.lanes;
    if (t >= p.tokens)
        return;
    const int *rows = p.row_of_slot + t * p.topk;
    const float *w = p.weights ? p.weights + t * p.topk : nullptr;
    for (int b = 16 * lane; b < p.bytes; b += 16 * p.lanes) {
        float sum[VEC] = {};
        for (int j = 0; j < p.topk; ++j) {
            const int r = rows[j];
            if (!valid_row(p, r))
                continue;
            float y[VEC];
            load_chunk<T>(p.in + r * p.ld_in, b, p.bytes, y);
            const float wj = w ? w[j] : 1.0f;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                sum[i] = __builtin_fmaf(wj, y[i], sum[i]);
        }
        store_chunk<T>(p.out + t * p.ld_out, b, p.bytes, sum);
    }
}

// A token's lanes hold a part of dout's row; each slot's partial dot products
// are added over the lanes by exchanges within a wave and through LDS across
// the waves of a 256-lane token, always in the same order.
template <typename T>
__global__ void __launch_bounds__(256) expert_combine_grad_kernel(RowParams p)
{
    constexpr int VEC = 16 / sizeof(T);
    constexpr int SLOTS = 8; // slots taken together
    __shared__ float part[4][SLOTS];
    const int lane = threadIdx.x & (p.lanes - 1);
    const long long t = (long long)blockIdx.x * (256 / p.lanes) + threadIdx.x / p.lanes;
    const bool live = t < p.tokens; // (all threads reach the barriers)
    const long long at = live ? t * p.topk : 0;
    const char *g = p.in + (live ? t : 0) * p.ld_in;
    for (int j0 = 0; j0 < p.topk; j0 += SLOTS) {
        float dot[SLOTS] = {};
        int r[SLOTS];
        float w[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const bool in = live && j0 + j < p.topk;
            r[j] = in ? p.row_of_slot[at + j0 + j] : -1;
            if (!valid_row(p, r[j]))
                r[j] = -1;
            w[j] = in && p.weights ? p.weights[at + j0 + j] : 1.0f;
        }
        if (live) {
            for (int b = 16 * lane; b < p.bytes; b += 16 * p.lanes) {
                float d[VEC];
                load_chunk<T>(g, b, p.bytes, d);
#pragma unroll
                for (int j = 0; j < SLOTS; ++j) {
                    if (r[j] < 0)
                        continue;
                    float v[VEC];
                    if (p.dweights) {
                        load_chunk<T>(p.in2 + r[j] * p.ld_in2, b, p.bytes, v);
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            dot[j] = __builtin_fmaf(d[i], v[i], dot[j]);
                    }
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        v[i] = w[j] * d[i];
                    store_chunk<T>(p.out + r[j] * p.ld_out, b, p.bytes, v);
                }
            }
        }
        if (!p.dweights)
            continue;
        const int within = p.lanes < 64 ? p.lanes : 64;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
            for (int d = 1; d < within; d <<= 1)
                dot[j] += __shfl_xor(dot[j], d);
        if (p.lanes > 64) {
            __syncthreads();
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int j = 0; j < SLOTS; ++j)
                    part[threadIdx.x >> 6][j] = dot[j];
            __syncthreads();
            const int w0 = (threadIdx.x / p.lanes) * (p.lanes / 64);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                dot[j] = part[w0][j];
                for (int k = 1; k < p.lanes / 64; ++k)
                    dot[j] += part[w0 + k][j];
            }
        }
        if (live && lane == 0)
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
                if (j0 + j < p.topk)
                    p.dweights[at + j0 + j] = r[j] < 0 ? 0.0f : dot[j];
    }
}

int launch_rows(const void *fn, RowParams p, hipStream_t s)
{
    p.lanes = 1;
    while (p.lanes < 256 && 16LL * p.lanes < p.bytes)
        p.lanes *= 2;
    const int per = 256 / p.lanes;
    // A launch holds fewer than 2^32 work-items. A later one starts at the
    // token it is given; the rows it names stay those of all tokens.
    const long long blocks = ceil_div_ll(p.tokens, per);
    if (blocks > (1 << 23))
        return -22;
    void *args[] = {&p};
    return (int)hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(256), args, 0, s);
}

bool float_type(int type) { return type == SGEMM_F32 || type == SGEMM_F16 || type == SGEMM_BF16; }

bool slots_ok(int tokens, int topk)
{
    return tokens >= 0 && (long long)tokens * (topk > 0 ? topk : 1) <= INT32_MAX;
}

} // namespace

extern "C" size_t expert_sort_workspace_size(int tokens, int topk, int experts)
{
    if (topk < 1 || !slots_ok(tokens, topk) || experts < 1 || experts > EXPERT_SORT_MAX_EXPERTS)
        return 0;
    const SortPlan plan = sort_plan((long long)tokens * topk);
    return plan.blocks > 1 ? (size_t)plan.blocks * (experts + 1) * sizeof(int) : 0;
}

extern "C" int expert_sort(int tokens, int topk, int experts, const void *ids, int id_bytes,
                           int *offsets, int *row_of_slot, void *workspace,
                           size_t workspace_bytes, sgemm_stream_t stream)
{
    if (topk < 1) return -402;
    if (!slots_ok(tokens, topk)) return -401;
    if (experts < 1 || experts > EXPERT_SORT_MAX_EXPERTS) return -403;
    if (tokens > 0 && ids == nullptr) return -404;
    if (id_bytes != 4 && id_bytes != 8) return -405;
    if (offsets == nullptr) return -406;
    if (tokens > 0 && row_of_slot == nullptr) return -407;
    const size_t need = expert_sort_workspace_size(tokens, topk, experts);
    if (need > 0 && (workspace == nullptr || ((uintptr_t)workspace & 3))) return -408;
    if (workspace_bytes < need) return -409;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    int *counts = static_cast<int *>(workspace);
    return id_bytes == 4
               ? launch_sort<int>(tokens * topk, experts, ids, offsets, row_of_slot, counts, s)
               : launch_sort<long long>(tokens * topk, experts, ids, offsets, row_of_slot, counts,
                                        s);
}

extern "C" int expert_gather(int tokens, int topk, int cols, const void *X, int type, int ldx,
                             const int *row_of_slot, void *Y, int ldy, sgemm_stream_t stream)
{
    if (topk < 1) return -502;
    if (!slots_ok(tokens, topk)) return -501;
    if (cols < 0) return -503;
    if (!float_type(type) && type != SGEMM_I8) return -505;
    const int row = cols > 1 ? cols : 1;
    if (ldx < row) return -506;
    if (ldy < row) return -509;
    const int es = type_bytes(type);
    if ((long long)cols * es > INT32_MAX - 4096) return -503;
    if (tokens == 0 || cols == 0)
        return 0;
    if (X == nullptr) return -504;
    if (row_of_slot == nullptr) return -507;
    if (Y == nullptr) return -508;
    RowParams p{};
    p.in = static_cast<const char *>(X);
    p.out = static_cast<char *>(Y);
    p.row_of_slot = row_of_slot;
    p.ld_in = (long long)ldx * es;
    p.ld_out = (long long)ldy * es;
    p.tokens = tokens;
    p.topk = topk;
    p.bytes = cols * es;
    const void *fn = es == 4   ? (const void *)expert_gather_kernel<4>
                     : es == 2 ? (const void *)expert_gather_kernel<2>
                               : (const void *)expert_gather_kernel<1>;
    return launch_rows(fn, p, static_cast<hipStream_t>(stream));
}

extern "C" int expert_combine(int tokens, int topk, int cols, const void *Y, int type, int ldy,
                              const int *row_of_slot, const float *weights, void *out, int ldo,
                              sgemm_stream_t stream)
{
    if (topk < 1) return -602;
    if (!slots_ok(tokens, topk)) return -601;
    if (cols < 0) return -603;
    if (!float_type(type)) return -605;
    const int row = cols > 1 ? cols : 1;
    if (ldy < row) return -606;
    if (ldo < row) return -610;
    const int es = type_bytes(type);
    if ((long long)cols * es > INT32_MAX - 4096) return -603;
    if (tokens == 0 || cols == 0)
        return 0;
    if (Y == nullptr) return -604;
    if (row_of_slot == nullptr) return -607;
    if (out == nullptr) return -609;
    RowParams p{};
    p.in = static_cast<const char *>(Y);
    p.out = static_cast<char *>(out);
    p.row_of_slot = row_of_slot;
    p.weights = weights;
    p.ld_in = (long long)ldy * es;
    p.ld_out = (long long)ldo * es;
    p.tokens = tokens;
    p.topk = topk;
    p.bytes = cols * es;
    const void *fn = type == SGEMM_F32   ? (const void *)expert_combine_kernel<float>
                     : type == SGEMM_F16 ? (const void *)expert_combine_kernel<_Float16>
                                         : (const void *)expert_combine_kernel<__bf16>;
    return launch_rows(fn, p, static_cast<hipStream_t>(stream));
}

extern "C" int expert_combine_grad(int tokens, int topk, int cols, const void *dout, int type,
                                   int ldo, const void *Y, int ldy, const int *row_of_slot,
                                   const float *weights, void *dY, int lddy, float *dweights,
                                   sgemm_stream_t stream)
{
    if (topk < 1) return -702;
    if (!slots_ok(tokens, topk)) return -701;
    if (cols < 0) return -703;
    if (!float_type(type)) return -705;
    const int row = cols > 1 ? cols : 1;
    if (ldo < row) return -706;
    if (dweights != nullptr && ldy < row) return -708;
    if (lddy < row) return -712;
    const int es = type_bytes(type);
    if ((long long)cols * es > INT32_MAX - 4096) return -703;
    // (With cols == 0 the sums over no columns are still written.)
    if (tokens == 0 || (cols == 0 && dweights == nullptr))
        return 0;
    if (cols > 0 && dout == nullptr) return -704;
    if (cols > 0 && dweights != nullptr && Y == nullptr) return -707;
    if (row_of_slot == nullptr) return -709;
    if (cols > 0 && dY == nullptr) return -711;
    RowParams p{};
    p.in = static_cast<const char *>(dout);
    p.in2 = static_cast<const char *>(Y);
    p.out = static_cast<char *>(dY);
    p.row_of_slot = row_of_slot;
    p.weights = weights;
    p.dweights = dweights;
    p.ld_in = (long long)ldo * es;
    p.ld_in2 = (long long)ldy * es;
    p.ld_out = (long long)lddy * es;
    p.tokens = tokens;
    p.topk = topk;
    p.bytes = cols * es;
    const void *fn = type == SGEMM_F32   ? (const void *)expert_combine_grad_kernel<float>
                     : type == SGEMM_F16 ? (const void *)expert_combine_grad_kernel<_Float16>
                                         : (const void *)expert_combine_grad_kernel<__bf16>;
    return launch_rows(fn, p, static_cast<hipStream_t>(stream));
}
