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
// The slots are cut into consecutive runs, one a workgroup (sort_plan).
// The first kernel counts each run's keys. In the second, a workgroup adds up
// the counts of the runs before its own and of all experts below each, which
// is the row of its first slot with that expert; its waves, each on a
// consecutive part of the run, then number their slots: a slot's row is its
// expert's next row for the wave plus the lanes before it with the same
// expert. Every count is an integer sum, so the order in which workgroups run
// changes nothing. The sort moves 8 bytes a slot, so latencies bound it: 256
// slots take 4 us, 65536 of 64 experts 8.4 us, 2097152 24 us.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxKeys = EXPERT_SORT_MAX_EXPERTS + 1;

struct SortPlan {
    int blocks, run; // runs of `run` slots (a multiple of 64 * kSortWaves)
};

// Up to 2048 slots are one run and one kernel (2048 slots of 64 experts: 6.3
// us, against 7.5 in two runs and kernels). Beyond, runs of 1024 (16384 slots:
// 8.6 us, of 2048 9.5), longer ones where there would be over 256, or, up to
// 8192, where each workgroup would read over 2^16 counts (1024 experts: 131072
// slots 20 us with 64 runs, 25 with 128; 524288 slots 34 with 64, 43 with 256;
// 2097152 slots 84 with 64, 56 with 256).
SortPlan sort_plan(long long slots, int keys)
{
    const long long unit = 64 * kSortWaves;
    if (slots <= 2048)
        return SortPlan{1, (int)(slots > 0 ? ceil_div_ll(slots, unit) * unit : unit)};
    long long most = (1 << 16) / keys;
    most = most < slots / 8192 ? slots / 8192 : most;
    most = most < 256 ? most : 256;
    long long run = ceil_div_ll(ceil_div_ll(slots, most), unit) * unit;
    if (run < 1024)
        run = 1024;
    return SortPlan{(int)ceil_div_ll(slots, run), (int)run};
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
    __shared__ int total[kMaxKeys], before[kMaxKeys];
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

    // Each key: all runs' slots, and those of the runs before this one. A
    // single run's own counts are all; otherwise the threads share out the runs
    // of the keys, so that all counts are in flight at once.
    if (counts == nullptr) {
        for (int e = tid; e < keys; e += kSortThreads) {
            int all = 0;
            for (int w = 0; w < kSortWaves; ++w)
                all += next[w * keys + e];
            total[e] = all;
            before[e] = 0;
        }
    } else {
        for (int e = tid; e < keys; e += kSortThreads)
            total[e] = before[e] = 0;
        __syncthreads();
        int width = 64; // threads along the keys
        while (width < keys && width < kSortThreads)
            width *= 2;
        for (int e = tid & (width - 1); e < keys; e += width) {
            int all = 0, bef = 0;
#pragma unroll 8
            for (int b = tid / width; b < (int)gridDim.x; b += kSortThreads / width) {
                const int n = counts[(long long)b * keys + e];
                all += n;
                bef += b < (int)blockIdx.x ? n : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&before[e], bef);
        }
    }
    __syncthreads();

    // The rows before each key: an exclusive scan of the totals, 512 at a time.
    constexpr int PER = (kMaxKeys + kSortThreads - 1) / kSortThreads;
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
        int at = start[j] + before[e];
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
    SortPlan plan = sort_plan(slots, experts + 1);
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
// lanes tokens share a workgroup. A row's last 16 bytes are taken as they lie,
// over the chunk before them: what both hold is written twice, the same. (A row
// of fewer bytes goes element by element.) SLOTS slots (a power of two up to 8, as many
// as topk needs) go together, so that their rows are in flight at once. Rows
// need no alignment. With WAVE, a token has whole waves, and its slots' rows
// and weights are scalars. Bound by memory: 16384 tokens x 4 of 2048 bf16 move
// at 5.0 TB/s (gather, 67 us), 5.1 (sum, 65 us) and 4.7 (gradients, 127 us);
// with a slot's row fetched after the one before it the sum took 94 us and the
// gradients of 8192 x 8 slots 131 (114 so).
// ---------------------------------------------------------------------------
struct RowParams {
    const char *in;      // X or dout, or Y of the sum
    const char *in2;     // Y of the gradient
    char *out;
    const int *row_of_slot;
    const float *weights;
    float *dweights;
    long long ld_in, ld_in2, ld_out; // bytes
    int tokens, topk;
    int lanes, log_lanes;
    int bytes; // of a row
};

template <bool WAVE>
__device__ __forceinline__ int token_of(const RowParams &p)
{
    const int in_block = threadIdx.x >> p.log_lanes;
    return blockIdx.x * (256 >> p.log_lanes) +
           (WAVE ? __builtin_amdgcn_readfirstlane(in_block) : in_block);
}

// Through the constant address space a wave's common value is a scalar load
// (no kernel here writes what it reads so).
template <bool WAVE, typename T>
__device__ __forceinline__ T slot_value(const T *x, long long i)
{
    if constexpr (WAVE)
        return ((const __attribute__((address_space(4))) T *)(uintptr_t)x)[i];
    else
        return x[i];
}

// The sorted rows of slots j0.. of the token whose first slot is `at`, -1 for
// none.
template <bool WAVE, int SLOTS>
__device__ __forceinline__ void slot_rows(const RowParams &p, long long at, int j0, int (&r)[SLOTS])
{
    const unsigned all = (unsigned)p.tokens * (unsigned)p.topk;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        // (Behind the last slot: the last one's again, and then -1.)
        r[j] = slot_value<WAVE>(p.row_of_slot, at + min(j0 + j, p.topk - 1));
        r[j] = j0 + j < p.topk && (unsigned)r[j] < all ? r[j] : -1;
    }
}

template <bool WAVE, int SLOTS>
__device__ __forceinline__ void slot_weights(const RowParams &p, long long at, int j0,
                                             float (&w)[SLOTS])
{
#pragma unroll
    for (int j = 0; j < SLOTS; ++j)
        w[j] = 1.0f;
    if (p.weights)
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
            w[j] = slot_value<WAVE>(p.weights, at + min(j0 + j, p.topk - 1));
}

// Where the chunk from byte b on is taken: at the row's end, the last 16 bytes.
__device__ __forceinline__ int chunk_at(const RowParams &p, int b)
{
    return min(b, max(p.bytes - 16, 0));
}

template <int ES, int SLOTS, bool WAVE>
__global__ void __launch_bounds__(256) expert_gather_kernel(RowParams p)
{
    const int lane = threadIdx.x & (p.lanes - 1);
    const int t = token_of<WAVE>(p);
    if (t >= p.tokens)
        return;
    const char *x = p.in + t * p.ld_in;
    const long long at = (long long)t * p.topk;
    for (int b0 = 16 * lane; b0 < p.bytes; b0 += 16 * p.lanes) {
        const int b = chunk_at(p, b0);
        const bool whole = b + 16 <= p.bytes;
        i32x4 v = {};
        if (whole)
            v = load16(x + b);
        for (int j0 = 0; j0 < p.topk; j0 += SLOTS) {
            int r[SLOTS];
            slot_rows<WAVE>(p, at, j0, r);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                if (r[j] < 0)
                    continue;
                char *y = p.out + r[j] * p.ld_out + b;
                if (whole) {
                    store16(y, v);
                } else {
                    typedef std::conditional_t<
                        ES == 4, int, std::conditional_t<ES == 2, short, char>> E;
                    const int n = (p.bytes - b) / ES;
                    for (int i = 0; i < n; ++i)
                        reinterpret_cast<E *>(y)[i] = reinterpret_cast<const E *>(x + b)[i];
                }
            }
        }
    }
}

// 16 bytes of a row from byte b on as floats, zeros behind the row's end.
template <typename T>
__device__ __forceinline__ void load_chunk(const char *row, int b, int bytes,
                                           float (&x)[16 / sizeof(T)])
{
    if (b + 16 <= bytes) {
        unpack<T>(load16(row + b), x);
        return;
    }
    const T *e = reinterpret_cast<const T *>(row + b);
    const int n = (bytes - b) / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i)
        x[i] = i < n ? (float)e[i] : 0.0f;
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

// A chunk of the rows of SLOTS slots. A slot without a row fetches row 0 (which
// there always is); its values are not used.
template <typename T, int SLOTS>
__device__ __forceinline__ void load_slots(const char *y, long long ld, const int (&r)[SLOTS], int b,
                                           int bytes, float (&v)[SLOTS][16 / sizeof(T)])
{
    if (b + 16 <= bytes) {
        i32x4 raw[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
            raw[j] = load16(y + max(r[j], 0) * ld + b);
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
            unpack<T>(raw[j], v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
            load_chunk<T>(y + max(r[j], 0) * ld, b, bytes, v[j]);
    }
}

template <typename T, int SLOTS, bool WAVE>
__global__ void __launch_bounds__(256) expert_combine_kernel(RowParams p)
{
    constexpr int VEC = 16 / sizeof(T);
    const int lane = threadIdx.x & (p.lanes - 1);
    const int t = token_of<WAVE>(p);
    if (t >= p.tokens)
        return;
    const long long at = (long long)t * p.topk;
    for (int b0 = 16 * lane; b0 < p.bytes; b0 += 16 * p.lanes) {
        const int b = chunk_at(p, b0);
        float sum[VEC] = {};
        for (int j0 = 0; j0 < p.topk; j0 += SLOTS) {
            int r[SLOTS];
            float w[SLOTS], y[SLOTS][VEC];
            slot_rows<WAVE>(p, at, j0, r);
            slot_weights<WAVE>(p, at, j0, w);
            load_slots<T>(p.in, p.ld_in, r, b, p.bytes, y);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    sum[i] = r[j] < 0 ? sum[i] : __builtin_fmaf(w[j], y[j][i], sum[i]);
        }
        store_chunk<T>(p.out + t * p.ld_out, b, p.bytes, sum);
    }
}

// A token's lanes hold a part of dout's row; each slot's partial dot products
// are added over the lanes by exchanges within a wave and through LDS across
// the waves of a token, always in the same order.
template <typename T, int SLOTS, bool WAVE>
__global__ void __launch_bounds__(256) expert_combine_grad_kernel(RowParams p)
{
    constexpr int VEC = 16 / sizeof(T);
    __shared__ float part[4][SLOTS];
    const int lane = threadIdx.x & (p.lanes - 1);
    const int token = token_of<WAVE>(p);
    const bool live = token < p.tokens; // (all threads reach the barriers)
    const int t = live ? token : 0;
    const long long at = (long long)t * p.topk;
    const char *g = p.in + t * p.ld_in;
    for (int j0 = 0; j0 < p.topk; j0 += SLOTS) {
        float dot[SLOTS] = {}, w[SLOTS];
        int r[SLOTS];
        slot_rows<WAVE>(p, at, j0, r);
        slot_weights<WAVE>(p, at, j0, w);
        if (live) {
            for (int b0 = 16 * lane; b0 < p.bytes; b0 += 16 * p.lanes) {
                const int b = chunk_at(p, b0);
                const int again = (b0 - b) / (int)sizeof(T); // elements of the chunk before
                float d[VEC];
                if (p.dweights) {
                    float y[SLOTS][VEC];
                    load_slots<T>(p.in2, p.ld_in2, r, b, p.bytes, y);
                    load_chunk<T>(g, b, p.bytes, d);
                    // (The elements of the chunk before are counted there.)
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j)
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            dot[j] = i < again ? dot[j]
                                               : __builtin_fmaf(d[i], y[j][i], dot[j]);
                } else {
                    load_chunk<T>(g, b, p.bytes, d);
                }
#pragma unroll
                for (int j = 0; j < SLOTS; ++j) {
                    if (r[j] < 0)
                        continue;
                    float v[VEC];
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
            const int w0 = (threadIdx.x >> p.log_lanes) * (p.lanes / 64);
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

typedef void (*RowFn)(RowParams);

// A kernel by slots taken together (1, 2, 4, 8) and by WAVE.
struct RowKernels {
    RowFn fn[4][2];
};

#define ROW_KERNELS(kernel, type)                                      \
    RowKernels                                                         \
    {                                                                  \
        {{kernel<type, 1, false>, kernel<type, 1, true>},              \
         {kernel<type, 2, false>, kernel<type, 2, true>},              \
         {kernel<type, 4, false>, kernel<type, 4, true>},              \
         {kernel<type, 8, false>, kernel<type, 8, true>}},             \
    }

int launch_rows(const RowKernels &k, RowParams p, hipStream_t s)
{
    p.lanes = 1;
    while (p.lanes < 256 && 16LL * p.lanes < p.bytes) {
        p.lanes *= 2;
        ++p.log_lanes;
    }
    const long long blocks = ceil_div_ll(p.tokens, 256 / p.lanes);
    if (blocks > (1 << 23)) // a launch holds fewer than 2^32 work-items
        return -22;
    const int slots = p.topk <= 1 ? 0 : p.topk <= 2 ? 1 : p.topk <= 4 ? 2 : 3;
    void *args[] = {&p};
    return (int)hipLaunchKernel((const void *)k.fn[slots][p.lanes >= 64], dim3((unsigned)blocks),
                                dim3(256), args, 0, s);
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
    const SortPlan plan = sort_plan((long long)tokens * topk, experts + 1);
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
    static const RowKernels kernels[] = {ROW_KERNELS(expert_gather_kernel, 4),
                                         ROW_KERNELS(expert_gather_kernel, 2),
                                         ROW_KERNELS(expert_gather_kernel, 1)};
    return launch_rows(kernels[es == 4 ? 0 : es == 2 ? 1 : 2], p, static_cast<hipStream_t>(stream));
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
    static const RowKernels kernels[] = {ROW_KERNELS(expert_combine_kernel, float),
                                         ROW_KERNELS(expert_combine_kernel, _Float16),
                                         ROW_KERNELS(expert_combine_kernel, __bf16)};
    return launch_rows(kernels[type], p, static_cast<hipStream_t>(stream));
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
    static const RowKernels kernels[] = {ROW_KERNELS(expert_combine_grad_kernel, float),
                                         ROW_KERNELS(expert_combine_grad_kernel, _Float16),
                                         ROW_KERNELS(expert_combine_grad_kernel, __bf16)};
    return launch_rows(kernels[type], p, static_cast<hipStream_t>(stream));
}
