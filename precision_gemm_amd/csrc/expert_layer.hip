// A whole layer of experts for a few tokens (expert_layer of experts.h), for
// MI355X (gfx950).

#include "ops_common.h"

#include "experts.h"

#include <cmath>
#include <type_traits>

namespace {

// The work is the weights of the experts that the tokens name, read once: bound
// by memory. So the weights go from memory straight into the matrix
// instructions' registers, 16 rows of them against up to 16 slots (columns) an
// instruction, with K over the waves of a workgroup; what the tokens supply is
// small and comes from the caches. Each workgroup finds its expert and that
// expert's slots from the ids itself, so nothing has to be sorted first.
//
// Weights of 8 bits are exact in bf16, and so are those of 4 bits times their scale,
// from 2^-128 to below 2^128 (the scale bytes 253 and 254 make infinities of some),
// so those products run in bf16 (8-bit weights of fp16 tokens: in fp16) on as many
// terms as the other operand needs to lose nothing: fp16 tokens are two bf16
// numbers, fp32 ones three. The layer's inner values, fp32 in memory, are three
// terms (with fp32 weights fp32 themselves): all 24 bits. Two, 16 bits, would take
// 83 us instead of 86 for the 64 tokens below and 46 instead of 54 for 128 tokens
// through 2 of 8 experts, but what an output's sum cancels would show their
// rounding. The terms are made once a workgroup, as its columns of activations
// are brought to LDS.
//
// 64 tokens through 8 of 128 experts, 2048 x 768, in bf16 with 4-bit weights: 46
// us for W1 (4.2 TB/s), 32 for W2, 5 for the sums; 16 through 4 of 64, 2048 x 1024,
// fp16 with 8-bit weights: 28, 18 and 4.7; one through 8 of 128 in bf16: 13.4 (of
// 50 MB; 6 without the weights' loads), 9 and 4.

struct Mx4 {};
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <typename E> struct FragOf;
template <> struct FragOf<float> { typedef float type; };
template <> struct FragOf<_Float16> { typedef f16x8 type; };
template <> struct FragOf<__bf16> { typedef bf16x8 type; };

__device__ __forceinline__ f32x4 mfma(float a, float b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The upper halves of two numbers' bits: bf16 by truncation.
__device__ __forceinline__ int upper_halves(float lo, float hi)
{
    return (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi),
                                      __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}

// What a number's truncation to bf16 leaves (exact); nothing of an infinity or
// NaN, which that term carries alone.
__device__ __forceinline__ float rest_of(float x)
{
    const uint32_t bits = __builtin_bit_cast(uint32_t, x);
    const float r = x - __builtin_bit_cast(float, bits & 0xffff0000u);
    return (bits & 0x7f800000u) == 0x7f800000u ? 0.0f : r;
}

// Eight numbers as N terms of bf16: each the truncation of what the ones before
// leave, the last one rounded (of three, which hold all 24 bits, it needs none).
template <int N>
__device__ __forceinline__ void split8(float (&f)[8], bf16x8 (&to)[N])
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (n + 1 == N && N > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                to[n][i] = (__bf16)f[i];
        } else {
            i32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = upper_halves(f[2 * i], f[2 * i + 1]);
            to[n] = __builtin_bit_cast(bf16x8, v);
            if (n + 1 < N)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = rest_of(f[i]);
        }
    }
}

__device__ __forceinline__ float mx4_scale(uint32_t byte)
{
    const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23;
    return __builtin_bit_cast(float, bits);
}

// The products of one call: X's and the weights' types, and whether the
// activations are the tokens (UP) or the inner values.
template <typename X, typename W, bool UP> struct Math {
    static constexpr bool F32 = std::is_same<W, float>::value;
    static constexpr bool MX4 = std::is_same<W, Mx4>::value;
    static constexpr bool I8 = std::is_same<W, signed char>::value;
    typedef typename std::conditional<UP, X, float>::type In; // the activations in memory
    typedef typename std::conditional<
        F32, float,
        typename std::conditional<UP && std::is_same<X, _Float16>::value && !MX4, _Float16,
                                  __bf16>::type>::type Elem;
    typedef typename FragOf<Elem>::type Frag;
    static constexpr int EPC = MX4 ? 32 : I8 ? 16 : F32 ? 4 : 8; // elements of 16 bytes of weights
    static constexpr int NM = F32 ? 4 : EPC / 8;                 // instructions of them
    static constexpr bool BF = std::is_same<Elem, __bf16>::value;
    static constexpr int NW = BF && std::is_same<W, _Float16>::value ? 2 : 1; // terms
    static constexpr int NX = !BF                                        ? 1
                              : !UP || std::is_same<X, float>::value     ? 3
                              : std::is_same<X, _Float16>::value         ? 2
                                                                         : 1;
    static constexpr int VEC = 16 / (int)sizeof(Elem); // elements of 16 bytes in LDS

    // Instruction i's operand of a chunk of weights; s: the scale of its block.
    static __device__ __forceinline__ void weights(int i, i32x4 v, float s, Frag (&to)[NW])
    {
        if constexpr (F32) {
            to[0] = __int_as_float(v[i]);
        } else if constexpr (MX4) {
            i32x4 w;
            w[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 0));
            w[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 1));
            w[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 2));
            w[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 3));
            to[0] = __builtin_bit_cast(bf16x8, w);
        } else if constexpr (I8) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = (float)(signed char)(v[2 * i + e / 4] >> (8 * (e % 4)));
            if constexpr (BF) {
                split8<1>(f, to);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    to[0][e] = (_Float16)f[e];
            }
        } else if constexpr (NW == 2) {
            float f[8];
            unpack<_Float16>(v, f);
            split8<2>(f, to);
        } else {
            to[0] = __builtin_bit_cast(Frag, v);
        }
    }

    // VEC neighbouring activations as they lie, and as terms; zeros behind K.
    static constexpr int NR = VEC * (int)sizeof(In) / 16;

    static __device__ __forceinline__ void fetch(const In *row, int k, i32x4 (&to)[NR])
    {
#pragma unroll
        for (int i = 0; i < NR; ++i)
            to[i] = load16(row + k + i * (VEC / NR));
    }

    static __device__ __forceinline__ void fetch_edge(const In *row, int k, int K, i32x4 (&to)[NR])
    {
        typedef In iv __attribute__((ext_vector_type(VEC / NR)));
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            iv v;
#pragma unroll
            for (int e = 0; e < VEC / NR; ++e) {
                const int at = k + i * (VEC / NR) + e;
                v[e] = at < K ? row[at] : (In)0.0f;
            }
            to[i] = __builtin_bit_cast(i32x4, v);
        }
    }

    static __device__ __forceinline__ void terms(const i32x4 (&v)[NR], i32x4 (&to)[NX])
    {
        if constexpr (std::is_same<In, Elem>::value) {
            to[0] = v[0];
        } else {
            float f[VEC];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                float x[VEC / NR];
                unpack<In>(v[i], x);
#pragma unroll
                for (int e = 0; e < VEC / NR; ++e) // (quiet NaNs, whose truncation is one)
                    f[i * (VEC / NR) + e] = __builtin_canonicalizef(x[e]);
            }
            bf16x8 b[NX];
            split8<NX>(f, b);
#pragma unroll
            for (int n = 0; n < NX; ++n)
                to[n] = __builtin_bit_cast(i32x4, b[n]);
        }
    }
};

constexpr int kColumns = 16; // slots that are multiplied at a time: an instruction's columns

// Slots of one expert that a workgroup multiplies: the first kernel finds them and
// leaves them for the second.
struct LayerGroup {
    int e, cols; // e: -1 for none
    int slots[kColumns];
};

struct LayerParams {
    const void *X, *ids;
    const float *mix;
    const void *W1, *W2;
    const void *scale1, *scale2;
    void *out;
    float *inner;    // the inner values, slots x inner_cols
    float *partial;  // W2's products, slots x H
    LayerGroup *groups;
    long long strideW1, strideW2, ldw1, ldw2; // bytes
    long long ldx, ldo;
    int tokens, topk, experts, H, F;
    int inner_cols; // F rounded up to 16 bytes
    int id_bytes;
    int tiles; // row tiles of an expert
    uint32_t inverse; // of topk
    int parts; // waves that share a tile, K over them: 1, 2 or 4
};

constexpr int kLayerWaves = 4;
constexpr int kLayerThreads = 64 * kLayerWaves;
constexpr int kColumnBytes = 28 << 10; // of LDS for the columns of activations

// Quotients of numbers below 2^16 by one of them, from ceil(2^32 / d): the error is
// below n / 2^32 < 1 / d. (0 stands for 2^32, the inverse of 1.)
__host__ __device__ __forceinline__ uint32_t inverse_of(int d)
{
    return d == 1 ? 0u : 0xffffffffu / (uint32_t)d + 1u;
}

__device__ __forceinline__ int divide(int n, uint32_t inverse)
{
    return inverse ? (int)__umulhi((uint32_t)n, inverse) : n;
}

__device__ __forceinline__ int id_of(const LayerParams &p, int slot)
{
    if (p.id_bytes == 4) {
        const int v = static_cast<const int *>(p.ids)[slot];
        return v >= 0 && v < p.experts ? v : -1;
    }
    const long long v = static_cast<const long long *>(p.ids)[slot];
    return v >= 0 && v < p.experts ? (int)v : -1;
}

struct LayerShared {
    int count[EXPERT_LAYER_MAX_EXPERTS]; // slots of each expert
    int slots[kColumns];
    // Columns of activations while they are multiplied, then the waves' sums.
    __attribute__((aligned(16))) signed char columns[kColumnBytes];
};

// The experts that up to 16 slots name, a bit each at its first slot; id: the
// lane's slot's, or -1. Every lane of the wave gets the same.
__device__ __forceinline__ unsigned long long first_slots(const LayerParams &p, int &id)
{
    const int lane = threadIdx.x & 63, slots = p.tokens * p.topk;
    id = id_of(p, min(lane, slots - 1));
    if (lane >= slots)
        id = -1;
    bool first = id >= 0;
    for (int i = 0; i + 1 < slots; ++i) {
        const int other = __builtin_amdgcn_readlane(id, i);
        first = first & !((i < lane) & (other == id));
    }
    return __ballot(first);
}

// The lane of the nth bit.
__device__ __forceinline__ int nth_bit(unsigned long long bits, int nth)
{
    for (; nth > 0; --nth)
        bits &= bits - 1;
    return __builtin_ctzll(bits);
}

// The `nth` group of up to 16 slots with one expert, that expert and the group's
// slots (in sh.slots after the workgroup's next meeting): first each named
// expert's first 16 slots, in the experts' order, then the second 16 of those
// that have as many, and so on. False if there are fewer. Every thread of the
// workgroup takes part.
__device__ __forceinline__ bool find_slots(const LayerParams &p, int nth, LayerShared &sh, int &e,
                                           int &cols)
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int slots = p.tokens * p.topk;
    if (slots <= kColumns) { // (few enough for each wave to find them in its registers)
        int id;
        const unsigned long long experts = first_slots(p, id);
        if (nth >= __popcll(experts))
            return false;
        e = __builtin_amdgcn_readlane(id, nth_bit(experts, nth));
        const unsigned long long mine = __ballot(id == e);
        cols = __popcll(mine);
        if (id == e)
            sh.slots[__popcll(mine & ((1ull << lane) - 1))] = lane;
        return true;
    }
    constexpr int HELD = 8;
    int held[HELD]; // the ids of the first 512 slots, loaded side by side
    auto hold = [&](auto type) {
        typedef decltype(type) Id;
        Id v[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            v[i] = static_cast<const Id *>(p.ids)[min(64 * i + lane, slots - 1)];
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            held[i] = 64 * i + lane < slots && v[i] >= 0 && v[i] < (Id)p.experts ? (int)v[i] : -1;
    };
    if (p.id_bytes == 4)
        hold(int{});
    else
        hold((long long)0);
    for (int i = tid; i < p.experts; i += kLayerThreads)
        sh.count[i] = 0;
    __syncthreads();
    // (Each wave counts its share of every 64 * kLayerWaves slots.)
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (i % kLayerWaves == tid >> 6 && held[i] >= 0)
            atomicAdd(&sh.count[held[i]], 1);
    for (int s = 64 * HELD + tid; s < slots; s += kLayerThreads) {
        const int id = id_of(p, s);
        if (id >= 0)
            atomicAdd(&sh.count[id], 1);
    }
    __syncthreads();
    e = -1;
    int from = 0, total = 0; // the group's first slot among the expert's, and all of those
    for (bool any = true; any && e < 0; from += kColumns) {
        any = false;
        for (int i = 0; i < p.experts; i += 64) {
            const int n = i + lane < p.experts ? sh.count[i + lane] : 0;
            unsigned long long left = __ballot(n > from);
            const int here = __popcll(left);
            any = any || here > 0;
            if (nth < here) {
                for (; nth > 0; --nth)
                    left &= left - 1;
                e = i + __builtin_ctzll(left);
                total = __builtin_amdgcn_readlane(n, __builtin_ctzll(left));
                break;
            }
            nth -= here;
        }
    }
    if (e < 0)
        return false;
    from -= kColumns;
    cols = min(kColumns, total - from);
    int n = -from;
    auto add = [&](int first, int id) {
        const unsigned long long mine = __ballot(id == e);
        const int at = n + __popcll(mine & ((1ull << lane) - 1));
        if (id == e && at >= 0 && at < kColumns)
            sh.slots[at] = first + lane; // (every wave writes the same)
        n += __popcll(mine);
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        if (64 * i < slots)
            add(64 * i, held[i]);
    for (int s = 64 * HELD; s < slots && n < cols; s += 64)
        add(s, s + lane < slots ? id_of(p, s + lane) : -1);
    return true;
}

// Rows of weights as a wave's lanes load them. Where rows start on 16-byte
// boundaries, hold a multiple of 16 bytes and lie within 2^31 bytes of each other
// (`Even`), loads go through a buffer descriptor with 32-bit offsets, one outside
// it for zeros behind a row's end; others (`Ragged`) chunk by chunk at any address.
template <int NT> struct Even {
    __amdgpu_buffer_rsrc_t w[2], sc; // (of W1 the gate's part and the other)
    uint32_t offw[NT], offs[NT];
    int wbytes;
    uint32_t ldsc;
};

template <int NT> struct Ragged {
    const signed char *w[NT];
    const uint32_t *sc[NT];
    int wbytes;
    long long ldsc;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t whole(const void *base)
{
    return rows_rsrc(static_cast<const signed char *>(base), 0x7fffffff);
}

// The products of NT times 16 rows of weights a wave with the workgroup's `cols`
// columns of activations (up to 16; column c is row_of(c) of `in`), as much
// of K at a time as LDS holds of the columns. A step is 4 chunks of 16 bytes of a
// row of weights (lane l: chunk l / 16 of row l % 16); a wave takes the steps
// part, part + parts, ... The first steps' weights are loaded before the columns
// are, and DEPTH steps' loads are under way at once. A column's terms stand one
// behind the other, 16 bytes further in each column than a multiple of 256, so
// that the 16 columns that are read together lie in different banks.
template <typename M, bool UP, int NT, bool EVEN, int WAVES, typename Row, typename Shared>
__device__ __forceinline__ void
products(const typename std::conditional<EVEN, Even<NT>, Ragged<NT>>::type &rows,
         const typename M::In *in, Row row_of, int K, int cols, bool live, int part, int parts,
         Shared &sh, f32x4 (&acc)[NT])
{
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    constexpr int SPAN = 4 * M::EPC;            // elements of a step
    constexpr int ES = (int)sizeof(typename M::Elem);
    constexpr int DEPTH = NT == 1 ? 4 : NT == 2 ? 2 : 1;
    constexpr int HALF = NT > 1 ? NT / 2 : 1;
    struct Step {
        i32x4 w[NT];
        uint32_t word[NT];
    };
    auto load = [&](int s, Step &to) {
        const int c = 4 * s + q;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (EVEN) {
                to.w[t] = __builtin_bit_cast(
                    i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               rows.w[UP ? t / HALF : 0],
                               16 * c < rows.wbytes ? rows.offw[t] + 16u * c : kOutside, 0, 0));
                if constexpr (M::MX4)
                    to.word[t] = __builtin_amdgcn_raw_buffer_load_b32(
                        rows.sc, rows.offs[t] + s * rows.ldsc, 0, 0);
            } else if constexpr (M::MX4) {
                // (An element behind an odd K would meet a zero, but with a large scale
                // as an infinity.)
                to.w[t] = mx4_chunk(rows.w[t], 16 * c, K);
                to.word[t] = rows.sc[t][s * rows.ldsc];
            } else {
                to.w[t] = row_chunk(rows.w[t], 16 * c, rows.wbytes);
            }
        }
    };
    const int room = ((int)sizeof(sh.columns) / cols - 16) / (ES * M::NX) / 128 * 128;
    const int chunk = min(room, (K + 127) / 128 * 128), steps = (K + SPAN - 1) / SPAN;
    const int plane = chunk * ES, column = M::NX * plane + 16;
    for (int k0 = 0; k0 < K; k0 += chunk) {
        const int first = k0 / SPAN, end = live ? min(steps, first + chunk / SPAN) : 0;
        Step ring[DEPTH + 1];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (first + part + d * parts < end)
                load(first + part + d * parts, ring[d]);
        __syncthreads(); // (what stood in LDS has been read)
        const int here = min(chunk, (K - k0 + 127) / 128 * 128);
        // A wave takes every WAVES-th of the columns' pieces of 64 * VEC
        // elements, AT of them at a time.
        constexpr int AT = 4 / M::NR > 0 ? 4 / M::NR : 1, PIECE = 64 * M::VEC;
        const int each = (here + PIECE - 1) / PIECE, pieces = cols * each;
        const uint32_t inverse = inverse_of(each);
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        for (int i = wave; i < pieces; i += AT * WAVES) {
            i32x4 raw[AT][M::NR];
            int c[AT], k[AT];
#pragma unroll
            for (int a = 0; a < AT; ++a) {
                const int at = min(i + a * WAVES, pieces - 1);
                c[a] = divide(at, inverse);
                k[a] = (at - c[a] * each) * PIECE + lane * M::VEC;
            }
            if (k0 + here <= K) { // (K a multiple of 128, or not its end yet)
#pragma unroll
                for (int a = 0; a < AT; ++a)
                    M::fetch(in + row_of(c[a]), k0 + min(k[a], here - M::VEC), raw[a]);
            } else {
#pragma unroll
                for (int a = 0; a < AT; ++a)
                    M::fetch_edge(in + row_of(c[a]), k0 + k[a], K, raw[a]);
            }
#pragma unroll
            for (int a = 0; a < AT; ++a) {
                i32x4 v[M::NX];
                M::terms(raw[a], v);
                if (k[a] < here)
#pragma unroll
                    for (int n = 0; n < M::NX; ++n)
                        *reinterpret_cast<i32x4 *>(sh.columns + c[a] * column + n * plane +
                                                   k[a] * ES) = v[n];
            }
        }
        __syncthreads();
        const signed char *x = sh.columns + min(lane & 15, cols - 1) * column;
        auto multiply = [&](int s, const Step &v) {
            float scale[NT] = {};
            if constexpr (M::MX4)
#pragma unroll
                for (int t = 0; t < NT; ++t) // (Bytes of blocks behind K may hold anything.)
                    scale[t] = mx4_scale(32 * (4 * s + q) < K ? v.word[t] >> (8 * q) & 255u : 0u);
            const int at = ((s - first) * SPAN + q * M::EPC) * ES;
#pragma unroll
            for (int i = 0; i < M::NM; ++i) {
                typename M::Frag fw[NT][M::NW];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    M::weights(i, v.w[t], scale[t], fw[t]);
#pragma unroll
                for (int b = 0; b < M::NX; ++b) {
                    const typename M::Frag fx = *reinterpret_cast<const typename M::Frag *>(
                        x + b * plane + at + (int)sizeof(typename M::Frag) * i);
#pragma unroll
                    for (int a = 0; a < M::NW; ++a)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            acc[t] = mfma(fw[t][a], fx, acc[t]);
                }
            }
        };
        for (int s = first + part; s < end; s += (DEPTH + 1) * parts) {
#pragma unroll
            for (int d = 0; d <= DEPTH; ++d) {
                const int now = s + d * parts, ahead = now + DEPTH * parts;
                if (now >= end)
                    break;
                if (ahead < end)
                    load(ahead, ring[(d + DEPTH) % (DEPTH + 1)]);
                multiply(now, ring[d]);
            }
        }
    }
}

// The waves' sums through LDS: the `parts` waves that share a tile each get the
// subtiles t = part, part + parts, ... of its sum, added in the waves' order;
// alone, a wave has them already.
template <int NT>
__device__ __forceinline__ f32x4 joined(const f32x4 (&acc)[NT], int t, int parts,
                                        const f32x4 (*sums)[NT][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (parts == 1)
        return acc[t];
    const int first = wave & ~(parts - 1);
    f32x4 v = sums[first][t][lane];
    for (int i = 1; i < parts; ++i)
        v += sums[first + i][t][lane];
    return v;
}

template <int NT>
__device__ __forceinline__ void give(const f32x4 (&acc)[NT], int parts, f32x4 (*sums)[NT][64])
{
    if (parts == 1)
        return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads(); // (the columns have been read)
#pragma unroll
    for (int t = 0; t < NT; ++t)
        sums[wave][t][lane] = acc[t];
    __syncthreads();
}

// W1: NT / 2 times 16 rows of the gate and as many of the other part a tile (NT =
// 1: 8 and 8, in one instruction's rows), for up to 16 slots of an expert.
template <typename X, typename W, int NT, bool EVEN>
__global__ void __launch_bounds__(kLayerThreads) layer_up_kernel(LayerParams p)
{
    typedef Math<X, W, true> M;
    constexpr int HALF = NT > 1 ? NT / 2 : 1, ROWS = NT > 1 ? 16 * HALF : 8;
    __shared__ LayerShared sh;
    f32x4(*sums)[NT][64] = reinterpret_cast<f32x4(*)[NT][64]>(sh.columns);
    static_assert(sizeof(f32x4[kLayerWaves][NT][64]) <= kColumnBytes, "the sums fit");
    const int lane = threadIdx.x & 63, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave & (p.parts - 1), each = kLayerWaves / p.parts; // tiles of a workgroup
    const int blocks = (p.tiles + each - 1) / each;
    const int f0 = ((int)(blockIdx.x % blocks) * each + wave / p.parts) * ROWS;
    int e, cols = 0;
    const bool any = find_slots(p, blockIdx.x / blocks, sh, e, cols);
    if (blockIdx.x % blocks == 0 && wave == 0) { // (which wrote all slots itself)
        LayerGroup &to = p.groups[blockIdx.x / blocks];
        if (lane == 0) {
            to.e = any ? e : -1;
            to.cols = cols;
        }
        if (lane < cols)
            to.slots[lane] = sh.slots[lane];
    }
    if (!any)
        return;
    const bool live = f0 < p.F; // (a wave without a tile still meets the others)
    typename std::conditional<EVEN, Even<NT>, Ragged<NT>>::type rows;
    rows.wbytes = M::MX4 ? (p.H + 1) / 2 : p.H * (M::I8 ? 1 : (int)sizeof(X));
    const signed char *w1 = static_cast<const signed char *>(p.W1) + e * p.strideW1;
    const long long ldsc = 2LL * p.F;
    const uint32_t *sc = static_cast<const uint32_t *>(p.scale1) +
                         (M::MX4 ? e * ((p.H + 127LL) / 128) * ldsc : 0);
    const int base = min(f0, p.F - 1);
    if constexpr (EVEN) {
        rows.w[0] = whole(w1 + base * p.ldw1);
        rows.w[1] = whole(w1 + (base + (long long)p.F) * p.ldw1);
        rows.sc = whole(sc);
        rows.ldsc = (uint32_t)ldsc * 4;
    } else {
        rows.ldsc = ldsc;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const bool other = NT > 1 ? t / HALF : r >= 8;
        const int row = min(f0 + 16 * (t % HALF) + (NT > 1 ? r : r & 7), p.F - 1);
        const int at = row + (other ? p.F : 0);
        if constexpr (EVEN) {
            rows.offw[t] = (uint32_t)(((NT > 1 ? row : at) - base) * (int)p.ldw1);
            rows.offs[t] = 4u * at;
        } else {
            rows.w[t] = w1 + at * p.ldw1;
            rows.sc[t] = sc + at;
        }
    }
    f32x4 acc[NT] = {};
    products<M, true, NT, EVEN, kLayerWaves>(
        rows, static_cast<const X *>(p.X),
        [&](int c) { return divide(sh.slots[c], p.inverse) * p.ldx; }, p.H, cols, live, part,
        p.parts, sh, acc);
    give(acc, p.parts, sums);
    if (!live || r >= cols)
        return;
    float *to = p.inner + (long long)sh.slots[r] * p.inner_cols;
#pragma unroll
    for (int t = 0; t < HALF; ++t) {
        if ((t & (p.parts - 1)) != part)
            continue;
        // The lane's four inner values, one behind the other.
        const f32x4 gate = joined(acc, t, p.parts, sums);
        f32x4 up;
        if constexpr (NT > 1) {
            up = joined(acc, HALF + t, p.parts, sums);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                up[v] = __shfl_down(gate[v], 32);
            if (lane >= 32)
                continue;
        }
        const int f = f0 + 16 * t + 4 * (lane >> 4);
        f32x4 a;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            float x0 = gate[v], x1 = up[v];
            if constexpr (M::I8) {
                const float *s = static_cast<const float *>(p.scale1) + 2LL * p.F * e;
                x0 *= s[min(f + v, p.F - 1)];
                x1 *= s[p.F + min(f + v, p.F - 1)];
            }
            a[v] = x0 / (1.0f + expf(-x0)) * x1;
        }
        if (f < p.F) // (a row holds a multiple of four)
            store16(to + f, __builtin_bit_cast(i32x4, a));
    }
}

// W2: NT times 16 rows of it a tile, for up to 16 slots of an expert.
template <typename X, typename W, int NT, bool EVEN>
__global__ void __launch_bounds__(kLayerThreads) layer_down_kernel(LayerParams p)
{
    typedef Math<X, W, false> M;
    __shared__ LayerShared sh;
    f32x4(*sums)[NT][64] = reinterpret_cast<f32x4(*)[NT][64]>(sh.columns);
    const int lane = threadIdx.x & 63, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave & (p.parts - 1), each = kLayerWaves / p.parts;
    const int blocks = (p.tiles + each - 1) / each;
    const int h0 = ((int)(blockIdx.x % blocks) * each + wave / p.parts) * 16 * NT;
    const LayerGroup &group = p.groups[blockIdx.x / blocks];
    const int e = group.e, cols = group.cols;
    if (e < 0)
        return;
    if ((int)threadIdx.x < cols) // (read after the workgroup's next meeting)
        sh.slots[threadIdx.x] = group.slots[threadIdx.x];
    const bool live = h0 < p.H;
    typename std::conditional<EVEN, Even<NT>, Ragged<NT>>::type rows;
    rows.wbytes = M::MX4 ? (p.F + 1) / 2 : p.F * (M::I8 ? 1 : (int)sizeof(X));
    const signed char *w2 = static_cast<const signed char *>(p.W2) + e * p.strideW2;
    const uint32_t *sc = static_cast<const uint32_t *>(p.scale2) +
                         (M::MX4 ? e * ((p.F + 127LL) / 128) * p.H : 0);
    const int base = min(h0, p.H - 1);
    if constexpr (EVEN) {
        rows.w[0] = rows.w[1] = whole(w2 + base * p.ldw2);
        rows.sc = whole(sc);
        rows.ldsc = (uint32_t)p.H * 4;
    } else {
        rows.ldsc = p.H;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int row = min(h0 + 16 * t + r, p.H - 1);
        if constexpr (EVEN) {
            rows.offw[t] = (uint32_t)((row - base) * (int)p.ldw2);
            rows.offs[t] = 4u * row;
        } else {
            rows.w[t] = w2 + row * p.ldw2;
            rows.sc[t] = sc + row;
        }
    }
    f32x4 acc[NT] = {};
    products<M, false, NT, EVEN, kLayerWaves>(
        rows, p.inner, [&](int c) { return (long long)sh.slots[c] * p.inner_cols; }, p.F, cols,
        live, part, p.parts, sh, acc);
    give(acc, p.parts, sums);
    if (!live || r >= cols)
        return;
    float *to = p.partial + (long long)sh.slots[r] * p.H;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if ((t & (p.parts - 1)) != part)
            continue;
        f32x4 y = joined(acc, t, p.parts, sums);
        const int h = h0 + 16 * t + 4 * (lane >> 4);
        if constexpr (M::I8) {
            const float *s = static_cast<const float *>(p.scale2) + (long long)e * p.H;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                y[v] *= s[min(h + v, p.H - 1)];
        }
        if (h + 4 <= p.H) {
            store16(to + h, __builtin_bit_cast(i32x4, y));
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (h + v < p.H)
                    to[h + v] = y[v];
        }
    }
}

// Up to 8 slots: 16 rows of W2 a workgroup with the whole sum over a token's
// slots, so that no partial products are written and read again. A column is a
// slot; each of 8 waves takes an expert, or a part of one's K.
constexpr int kFewSlots = 8;

struct FewShared {
    f32x4 sums[kFewSlots][4][kFewSlots]; // by part of K, four rows and slot
    __attribute__((aligned(16))) signed char columns[56 << 10];
};

template <typename X, typename W>
__global__ void __launch_bounds__(64 * kFewSlots) layer_down_few_kernel(LayerParams p)
{
    typedef Math<X, W, false> M;
    __shared__ FewShared sh;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slots = p.tokens * p.topk, h0 = (int)blockIdx.x * 16;
    int id; // (of the lane's slot, as is its weight)
    const unsigned long long experts = first_slots(p, id);
    const float mix = p.mix ? p.mix[min(lane, slots - 1)] : 1.0f;
    const int named = __popcll(experts);
    int parts = 1; // (no expert may be named at all)
    while (2 * parts * max(named, 1) <= kFewSlots)
        parts *= 2;
    const int nth = wave / parts, part = wave & (parts - 1);
    const bool live = nth < named;
    const int e = live ? __builtin_amdgcn_readlane(id, nth_bit(experts, nth)) : 0;
    const int row = min(h0 + r, p.H - 1);
    Even<1> rows;
    rows.wbytes = M::MX4 ? (p.F + 1) / 2 : p.F * (M::I8 ? 1 : (int)sizeof(X));
    rows.w[0] = rows.w[1] =
        whole(static_cast<const signed char *>(p.W2) + e * p.strideW2 + h0 * p.ldw2);
    rows.sc = whole(static_cast<const uint32_t *>(p.scale2) +
                    (M::MX4 ? e * ((p.F + 127LL) / 128) * p.H : 0));
    rows.ldsc = (uint32_t)p.H * 4;
    rows.offw[0] = (uint32_t)((row - h0) * (int)p.ldw2);
    rows.offs[0] = 4u * row;
    f32x4 acc[1] = {};
    // (Slots without an expert hold no inner values: a column of theirs is some
    // bits that no one uses.)
    products<M, false, 1, true, kFewSlots>(
        rows, p.inner, [&](int c) { return (long long)c * p.inner_cols; }, p.F, slots, live, part,
        parts, sh, acc);
    if (live && __shfl(id, r) == e && r < slots)
        sh.sums[part][q][r] = acc[0];
    __syncthreads();
    // Thread i < 16 * tokens: row i % 16 of token i / 16.
    const int t = min(tid >> 4, p.tokens - 1), h = min(h0 + (tid & 15), p.H - 1);
    float sum = 0.0f;
    for (int j = 0; j < p.topk; ++j) {
        const int slot = t * p.topk + j, expert = __shfl(id, slot);
        const float w = __shfl(mix, slot);
        if (expert < 0)
            continue;
        float y = 0.0f;
        for (int i = 0; i < parts; ++i)
            y += sh.sums[i][(tid & 15) >> 2][slot][tid & 3];
        if constexpr (M::I8)
            y *= static_cast<const float *>(p.scale2)[(long long)expert * p.H + h];
        sum = __builtin_fmaf(w, y, sum);
    }
    if (tid >> 4 < p.tokens && h0 + (tid & 15) < p.H)
        static_cast<X *>(p.out)[t * p.ldo + h] = (X)sum;
}

// out[t] = sum_j mix[t, j] partial[t, j]. (A slot without an expert has no
// products: what is read in their place is not used, so that no read waits for
// the ids.)
template <typename X>
__global__ void __launch_bounds__(256) layer_join_kernel(LayerParams p)
{
    const long long at = blockIdx.x * 256LL + threadIdx.x;
    if (at >= (long long)p.tokens * p.H)
        return;
    const int t = (int)(at / p.H), h = (int)(at - (long long)t * p.H);
    float sum = 0.0f;
    if (p.F > 0) {
        constexpr int AT = 8;
        for (int j0 = 0; j0 < p.topk; j0 += AT) {
            float y[AT], w[AT];
            bool there[AT];
#pragma unroll
            for (int j = 0; j < AT; ++j) {
                const int slot = t * p.topk + min(j0 + j, p.topk - 1);
                y[j] = p.partial[(long long)slot * p.H + h];
                w[j] = p.mix ? p.mix[slot] : 1.0f;
                there[j] = j0 + j < p.topk && id_of(p, slot) >= 0;
            }
#pragma unroll
            for (int j = 0; j < AT; ++j)
                sum = there[j] ? __builtin_fmaf(w[j], y[j], sum) : sum;
        }
    }
    static_cast<X *>(p.out)[t * p.ldo + h] = (X)sum;
}

typedef void (*LayerFn)(LayerParams);

// One of the two kernels: tiles of `rows` rows of `total`, a workgroup's waves
// sharing them, K over them, as far as it takes for enough waves for the card.
struct LayerStep {
    LayerFn fn;
    int tiles, parts;
    long long blocks;
};

LayerStep layer_step(LayerFn fn, int total, int rows, double experts, int most, long long steps)
{
    LayerStep l{fn, (int)ceil_div_ll(total, rows), 1, 0};
    while (l.parts < kLayerWaves && 2 * l.parts <= steps && experts * l.tiles * l.parts < 3000)
        l.parts *= 2;
    l.blocks = most * ceil_div_ll(l.tiles, kLayerWaves / l.parts);
    return l;
}

hipError_t launch_step(const LayerStep &l, LayerParams p, hipStream_t s)
{
    p.tiles = l.tiles;
    p.parts = l.parts;
    void *args[] = {&p};
    return hipLaunchKernel((const void *)l.fn, dim3((unsigned)l.blocks), dim3(kLayerThreads), args,
                           0, s);
}

template <typename X, typename W> int launch_layer(LayerParams p, hipStream_t s)
{
    typedef Math<X, W, true> M;
    const int slots = p.tokens * p.topk;
    // Most groups of up to 16 slots of an expert: every named one may have one that
    // is not full.
    const int named = slots < p.experts ? slots : p.experts;
    const int most = named + (slots - named) / kColumns;
    p.inverse = inverse_of(p.topk);
    if (p.F > 0) {
        // Experts that even choices reach on average.
        const double even_reach = p.experts * (1.0 - std::pow(1.0 - 1.0 / p.experts, slots));
        const double reached = even_reach < 1.0 ? 1.0 : even_reach;
        auto row_bytes = [](long long K) {
            return M::MX4 ? (K + 1) / 2 : M::I8 ? K : K * (long long)sizeof(X);
        };
        auto even = [&](const void *w, long long ld, long long stride, long long K, long long R) {
            return (((uintptr_t)w | ld | stride | row_bytes(K)) & 15) == 0 && ld < 1 << 24 &&
                   (!M::MX4 || (K % 32 == 0 && ceil_div_ll(K, 128) * 4 * R < INT32_MAX));
        };
        const bool even1 = even(p.W1, p.ldw1, p.strideW1, p.H, 2LL * p.F);
        const bool even2 = even(p.W2, p.ldw2, p.strideW2, p.F, p.H);
        const long long steps1 = ceil_div_ll(row_bytes(p.H), 64);
        const long long steps2 = ceil_div_ll(row_bytes(p.F), 64);
        // (Refused before the device is asked: narrower tiles are for fewer of them,
        // too few to be more than a launch holds.)
        const LayerStep least1 = layer_step(nullptr, p.F, even1 ? 32 : 16, reached, most, steps1);
        const LayerStep least2 = layer_step(nullptr, p.H, even2 ? 64 : 32, reached, most, steps2);
        if (!fits_launch((double)least1.blocks, kLayerThreads) ||
            !fits_launch((double)least2.blocks, kLayerThreads))
            return -22;
        int cus = 0;
        const int st = current_cus(&cus);
        if (st != 0)
            return st;
        // Tiles: 64 rows where there are enough of them for the card, 32 or, with a
        // few a CU, 16, where the CUs' shares come out more even (one token through 8
        // experts, 768 x 2048 in bf16: 384 workgroups on 256 CUs take as long as 512
        // would, 16.2 us, 768 of half the rows 13.5); but not of narrow weights, of
        // which the activations' share grows (2 tokens, 2880 x 2880 in 4 bits: 29 us
        // against 34).
        auto tile = [&](bool even, bool narrow, int total, int rows) {
            const double n = reached * ceil_div_ll(total, rows);
            if (!even)
                return 2;
            if (n / 2 * kLayerWaves >= 3000)
                return 4;
            auto rounds = [&](double tiles) { return (double)(long long)(tiles / cus + 0.999); };
            return narrow && !M::MX4 && !M::I8 && n <= 3.0 * cus && rounds(2 * n) < 2 * rounds(n) ? 1
                                                                                              : 2;
        };
        // (The narrowest tile of W1 reaches both its parts by one offset of 32 bits.)
        const int nt1 = tile(even1, (p.F + 64LL) * p.ldw1 < INT32_MAX, p.F, 16);
        const int nt2 = tile(even2, true, p.H, 32);
        constexpr int NARROW = M::MX4 || M::I8 ? 2 : 1; // the narrowest tile
        const LayerFn up = !even1     ? layer_up_kernel<X, W, 2, false>
                           : nt1 == 4 ? layer_up_kernel<X, W, 4, true>
                           : nt1 == 2 ? layer_up_kernel<X, W, 2, true>
                                      : layer_up_kernel<X, W, NARROW, true>;
        const LayerFn down = !even2     ? layer_down_kernel<X, W, 2, false>
                             : nt2 == 4 ? layer_down_kernel<X, W, 4, true>
                             : nt2 == 2 ? layer_down_kernel<X, W, 2, true>
                                        : layer_down_kernel<X, W, NARROW, true>;
        hipError_t e = launch_step(layer_step(up, p.F, 8 * nt1, reached, most, steps1), p, s);
        if (e != hipSuccess)
            return (int)e;
        // The whole sum in 16 rows a workgroup, unless that leaves CUs idle for
        // longer than the partial products' way takes (4 us): a CU draws some 20 KB a
        // us from memory.
        const double drawn = reached * row_bytes(p.F) / 20e3;
        const double tiles = (double)ceil_div_ll(p.H, 16);
        const double whole = (double)ceil_div_ll((long long)tiles, cus) * 16 * drawn;
        if (slots <= kFewSlots && even2 && whole < tiles / cus * 16 * drawn + 4.0) {
            void *args[] = {&p};
            return (int)hipLaunchKernel((const void *)layer_down_few_kernel<X, W>,
                                        dim3((unsigned)ceil_div_ll(p.H, 16)),
                                        dim3(64 * kFewSlots), args, 0, s);
        }
        e = launch_step(layer_step(down, p.H, 16 * nt2, reached, most, steps2), p, s);
        if (e != hipSuccess)
            return (int)e;
    }
    const long long items = (long long)p.tokens * p.H;
    void *args[] = {&p};
    return (int)hipLaunchKernel((const void *)layer_join_kernel<X>,
                                dim3((unsigned)ceil_div_ll(items, 256)), dim3(256), args, 0, s);
}

template <typename X> int launch_layer_of(const LayerParams &p, int w_type, hipStream_t s)
{
    if (w_type == SGEMM_I8)
        return launch_layer<X, signed char>(p, s);
    if (w_type == SGEMM_MX4)
        return launch_layer<X, Mx4>(p, s);
    return launch_layer<X, X>(p, s);
}

constexpr int kMaxWidth = 1 << 20;

bool layer_slots_ok(int tokens, int topk)
{
    return tokens >= 0 && (long long)tokens * (topk > 0 ? topk : 1) <= EXPERT_LAYER_MAX_SLOTS;
}

long long padded_cols(int F) { return ((long long)F + 3) / 4 * 4; }

size_t inner_bytes(long long slots, int F) { return (size_t)slots * padded_cols(F) * sizeof(float); }

// As many groups as slots at most, on a 16-byte boundary behind the inner values,
// then the partial products.
size_t group_bytes(long long slots) { return ((size_t)slots * sizeof(LayerGroup) + 15) / 16 * 16; }

// Bytes of a row of weights; ldw has to reach as far.
long long weight_row(int K, int w_type)
{
    return w_type == SGEMM_MX4 ? ((long long)K + 1) / 2 : K;
}

} // namespace

extern "C" size_t expert_layer_workspace_size(int tokens, int topk, int H, int F, int type)
{
    if (topk < 1 || !layer_slots_ok(tokens, topk) || H < 0 || H > kMaxWidth || F < 0 ||
        F > kMaxWidth || !c_type_ok(type))
        return 0;
    const long long slots = (long long)tokens * topk;
    return inner_bytes(slots, F) + group_bytes(slots) + (size_t)slots * H * sizeof(float);
}

extern "C" int expert_layer(int tokens, int topk, int experts, int H, int F, const void *X,
                            int type, int ldx, const void *ids, int id_bytes,
                            const float *weights, const void *W1, int w_type, int ldw1,
                            long long strideW1, const void *scale1, const void *W2, int ldw2,
                            long long strideW2, const void *scale2, void *out, int ldo,
                            void *workspace, size_t workspace_bytes, sgemm_stream_t stream)
{
    if (topk < 1) return -1702;
    if (!layer_slots_ok(tokens, topk)) return -1701;
    if (experts < 1 || experts > EXPERT_LAYER_MAX_EXPERTS) return -1703;
    if (H < 0 || H > kMaxWidth) return -1704;
    if (F < 0 || F > kMaxWidth) return -1705;
    if (!c_type_ok(type)) return -1707;
    if (w_type != type && w_type != SGEMM_I8 && w_type != SGEMM_MX4) return -1713;
    const int row = H > 1 ? H : 1;
    if (ldx < row) return -1708;
    if (id_bytes != 4 && id_bytes != 8) return -1710;
    const long long row1 = weight_row(H, w_type), row2 = weight_row(F, w_type);
    if (ldw1 < (row1 > 1 ? row1 : 1)) return -1714;
    if (strideW1 < 0) return -1715;
    if (ldw2 < (row2 > 1 ? row2 : 1)) return -1718;
    if (strideW2 < 0) return -1719;
    if (ldo < row) return -1722;
    if (tokens == 0 || H == 0)
        return 0;
    if (X == nullptr) return -1706;
    if (ids == nullptr) return -1709;
    const bool scaled = w_type == SGEMM_I8 || w_type == SGEMM_MX4;
    if (F > 0) {
        if (W1 == nullptr) return -1712;
        if (scaled && (scale1 == nullptr || ((uintptr_t)scale1 & 3))) return -1716;
        if (W2 == nullptr) return -1717;
        if (scaled && (scale2 == nullptr || ((uintptr_t)scale2 & 3))) return -1720;
    }
    if (out == nullptr) return -1721;
    const size_t need = expert_layer_workspace_size(tokens, topk, H, F, type);
    if (workspace == nullptr || ((uintptr_t)workspace & 15)) return -1723;
    if (workspace_bytes < need) return -1724;
    const int es = w_type == SGEMM_I8 || w_type == SGEMM_MX4 ? 1 : type_bytes(w_type);
    LayerParams p{};
    p.X = X;
    p.ids = ids;
    p.mix = weights;
    p.W1 = W1;
    p.W2 = W2;
    p.scale1 = scale1;
    p.scale2 = scale2;
    p.out = out;
    p.inner = static_cast<float *>(workspace);
    const long long slots = (long long)tokens * topk;
    char *at = static_cast<char *>(workspace) + inner_bytes(slots, F);
    p.groups = reinterpret_cast<LayerGroup *>(at);
    p.partial = reinterpret_cast<float *>(at + group_bytes(slots));
    p.strideW1 = strideW1 * es;
    p.strideW2 = strideW2 * es;
    p.ldw1 = (long long)ldw1 * es;
    p.ldw2 = (long long)ldw2 * es;
    p.ldx = ldx;
    p.ldo = ldo;
    p.tokens = tokens;
    p.topk = topk;
    p.experts = experts;
    p.H = H;
    p.F = F;
    p.inner_cols = (int)padded_cols(F);
    p.id_bytes = id_bytes;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (type == SGEMM_F32)
        return launch_layer_of<float>(p, w_type, s);
    if (type == SGEMM_F16)
        return launch_layer_of<_Float16>(p, w_type, s);
    return launch_layer_of<__bf16>(p, w_type, s);
}
