// A whole layer of experts for a few tokens (expert_layer of experts.h), for
// MI355X (gfx950).

#include "ops_common.h"

#include "experts.h"

#include <type_traits>

namespace {

// The work is the weights of the experts that the tokens name, read once: bound
// by memory. So the weights go from memory straight into the matrix
// instructions' registers, 16 rows of them against up to 16 slots (columns) an
// instruction, with K over the waves of a workgroup; what the tokens supply is
// small and comes from the caches. Each workgroup finds its expert and that
// expert's slots from the ids itself, so nothing has to be sorted first.
//
// Weights of 8 and 4 bits and the scales of the latter are exact in bf16, so
// those products run in bf16 (8-bit weights of fp16 tokens: in fp16) on as many
// terms as the other operand needs to lose nothing: fp16 tokens are two bf16
// numbers, fp32 ones three. The layer's inner values, which no one type holds,
// are stored as two (fp32 layers: three), so they lose nothing that out could
// show.

struct Mx4 {};
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

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

// Eight numbers as N terms of bf16, each the truncation of what the ones before
// leave.
template <int N>
__device__ __forceinline__ void split8(float (&f)[8], bf16x8 (&to)[N])
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
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
    typedef typename std::conditional<
        F32, float,
        typename std::conditional<UP && std::is_same<X, _Float16>::value && !MX4, _Float16,
                                  __bf16>::type>::type Elem;
    typedef typename FragOf<Elem>::type Frag;
    static constexpr int EPC = MX4 ? 32 : I8 ? 16 : F32 ? 4 : 8; // elements of 16 bytes of weights
    static constexpr int NM = F32 ? 4 : EPC / 8;                 // instructions of them
    static constexpr bool BF = std::is_same<Elem, __bf16>::value;
    static constexpr int NW = BF && std::is_same<W, _Float16>::value ? 2 : 1; // terms
    static constexpr int NX = !BF                                   ? 1
                              : std::is_same<X, float>::value       ? 3
                              : !UP || std::is_same<X, _Float16>::value ? 2
                                                                    : 1;
    // Loads of 16 bytes of a slot's activations for 16 bytes of weights.
    static constexpr int NL = UP ? EPC * (int)sizeof(X) / 16 : F32 ? 1 : NX * EPC / 8;

    static __device__ __forceinline__ void weights(i32x4 v, uint32_t byte, Frag (&to)[NM][NW])
    {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                to[i][0] = __int_as_float(v[i]);
        } else if constexpr (MX4) {
            const float s = mx4_scale(byte);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                i32x4 w;
                w[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 0));
                w[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 1));
                w[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 2));
                w[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 3));
                to[i][0] = __builtin_bit_cast(bf16x8, w);
            }
        } else if constexpr (I8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = (float)(signed char)(v[2 * i + e / 4] >> (8 * (e % 4)));
                if constexpr (BF) {
                    split8<1>(f, to[i]);
                } else {
                    f16x8 h;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[e] = (_Float16)f[e];
                    to[i][0] = h;
                }
            }
        } else if constexpr (NW == 2) {
            float f[8];
            unpack<_Float16>(v, f);
            split8<2>(f, to[0]);
        } else {
            to[0][0] = __builtin_bit_cast(Frag, v);
        }
    }

    // The activations that belong to a chunk of weights, from their loads.
    static __device__ __forceinline__ void activations(const i32x4 (&v)[NL], Frag (&to)[NM][NX])
    {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                to[i][0] = __int_as_float(v[0][i]);
        } else if constexpr (!UP) {
#pragma unroll
            for (int i = 0; i < NM; ++i)
#pragma unroll
                for (int n = 0; n < NX; ++n)
                    to[i][n] = __builtin_bit_cast(Frag, v[n * NM + i]);
        } else if constexpr (std::is_same<X, Elem>::value) {
#pragma unroll
            for (int i = 0; i < NM; ++i)
                to[i][0] = __builtin_bit_cast(Frag, v[i]);
        } else {
            constexpr int VEC = 16 / sizeof(X);
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; j += VEC) {
                    float x[VEC];
                    unpack<X>(v[(8 * i + j) / VEC], x);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) // (quiet NaNs, whose truncation is one)
                        f[j + e] = __builtin_canonicalizef(x[e]);
                }
                split8<NX>(f, to[i]);
            }
        }
    }
};

struct LayerParams {
    const void *X, *ids;
    const float *mix;
    const void *W1, *W2;
    const void *scale1, *scale2;
    void *out;
    void *inner;     // the inner values: planes of slots x inner_cols
    float *partial;  // W2's products, slots x H
    long long strideW1, strideW2, ldw1, ldw2; // bytes
    long long ldx, ldo;
    int tokens, topk, experts, H, F;
    int inner_cols; // F rounded up to a step of the widest chunks
    int id_bytes;
    int tiles; // row tiles of an expert
};

constexpr int kLayerWaves = 8;
constexpr int kLayerThreads = 64 * kLayerWaves;
constexpr int kTileRows = 32; // rows of weights of a workgroup: two of an instruction's 16

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
    uint32_t named[EXPERT_LAYER_MAX_EXPERTS / 32]; // one bit an expert
    int count;
    unsigned short slots[EXPERT_LAYER_MAX_SLOTS];
    float sums[kLayerWaves][kTileRows][17];
};

// The `nth` expert that some slot names, in the experts' order, and its slots
// (in any order: a slot's results do not depend on its column); false if there
// are fewer. Every thread of the workgroup takes part.
__device__ __forceinline__ bool find_expert(const LayerParams &p, int nth, LayerShared &sh, int &e)
{
    const int tid = threadIdx.x, lane = tid & 63;
    const int slots = p.tokens * p.topk;
    if (tid < EXPERT_LAYER_MAX_EXPERTS / 32)
        sh.named[tid] = 0;
    if (tid == 0)
        sh.count = 0;
    __syncthreads();
    constexpr int PER = EXPERT_LAYER_MAX_SLOTS / kLayerThreads;
    int id[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = tid + i * kLayerThreads;
        id[i] = s < slots ? id_of(p, s) : -1;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (id[i] >= 0)
            atomicOr(&sh.named[id[i] >> 5], 1u << (id[i] & 31));
    __syncthreads();
    const uint32_t word = lane < EXPERT_LAYER_MAX_EXPERTS / 32 ? sh.named[lane] : 0;
    int upto = __popc(word);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d)
            upto += v;
    }
    const int before = upto - __popc(word);
    const unsigned long long who = __ballot(nth >= before && nth < upto);
    if (who == 0)
        return false;
    uint32_t left = word;
    if (nth >= before && nth < upto)
        for (int i = before; i < nth; ++i)
            left &= left - 1;
    const int src = __builtin_ctzll(who);
    e = 32 * src + __builtin_ctz((uint32_t)__builtin_amdgcn_readlane((int)left, src));
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (id[i] == e)
            sh.slots[atomicAdd(&sh.count, 1)] = (unsigned short)(tid + i * kLayerThreads);
    __syncthreads();
    return true;
}

// A wave's part of the products of two times 16 rows of weights with 16 * CG
// columns: steps wave, wave + kLayerWaves, ... of K, a step being 4 chunks of 16
// bytes of a row (lane l: chunk l / 16 of row l % 16; of the activations the same
// elements of column l % 16). cols: bytes of a row of activations (UP), or the
// bytes between their planes.
template <typename M, bool UP, int CG>
__device__ __forceinline__ void products(const signed char *const (&w)[2], int wbytes,
                                         const uint32_t *const (&sc)[2], long long ldsc, int K,
                                         const signed char *const (&x)[CG], long long xbytes,
                                         f32x4 (&acc)[2][CG])
{
    const int lane = threadIdx.x & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int steps = (wbytes + 63) / 64;
    constexpr int XB = UP ? M::NL * 16 : M::F32 ? 16 : M::EPC * 2; // of a chunk, a plane
    auto one = [&](int s, auto load_w, auto load_x) {
        const int c = 4 * s + q;
        i32x4 vw[2], vx[CG][M::NL];
        uint32_t byte[2] = {0, 0};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            vw[t] = load_w(w[t], 16 * c);
            if constexpr (M::MX4)
                byte[t] = sc[t][s * ldsc];
        }
#pragma unroll
        for (int g = 0; g < CG; ++g)
#pragma unroll
            for (int i = 0; i < M::NL; ++i) {
                if constexpr (UP || M::F32)
                    vx[g][i] = load_x(x[g], XB * c + 16 * i);
                else
                    vx[g][i] = load16(x[g] + (i / M::NM) * xbytes + XB * c + 16 * (i % M::NM));
            }
        typename M::Frag fw[2][M::NM][M::NW];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (M::MX4) {
                // (Bytes of blocks behind K may hold anything.)
                const bool there = 32 * c < K;
                byte[t] = there ? byte[t] >> (8 * q) & 255u : 0u;
            }
            M::weights(vw[t], byte[t], fw[t]);
        }
#pragma unroll
        for (int g = 0; g < CG; ++g) {
            typename M::Frag fx[M::NM][M::NX];
            M::activations(vx[g], fx);
#pragma unroll
            for (int i = 0; i < M::NM; ++i)
#pragma unroll
                for (int a = 0; a < M::NW; ++a)
#pragma unroll
                    for (int b = 0; b < M::NX; ++b)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            acc[t][g] = mfma(fw[t][i][a], fx[i][b], acc[t][g]);
        }
    };
    auto whole = [](const signed char *row, int k) { return load16(row + k); };
    auto edge_w = [&](const signed char *row, int k) { return row_chunk(row, k, wbytes); };
    auto edge_x = [&](const signed char *row, int k) {
        return UP ? row_chunk(row, k, (int)xbytes) : load16(row + k);
    };
    const int full = wbytes / 64 - (M::MX4 && K % 128 != 0 && wbytes % 64 == 0 ? 1 : 0);
    int s = wave;
    for (; s < full; s += kLayerWaves)
        one(s, whole, whole);
    for (; s < steps; s += kLayerWaves)
        one(s, edge_w, edge_x);
}

// acc of all waves added, through LDS, in the waves' order: thread i < 512 gets
// row i / 16, column i % 16 of the 32 rows.
__device__ __forceinline__ float join(const f32x4 &a0, const f32x4 &a1, LayerShared &sh)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    __syncthreads(); // (the last sums have been read)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        sh.sums[wave][4 * (lane >> 4) + v][lane & 15] = a0[v];
        sh.sums[wave][16 + 4 * (lane >> 4) + v][lane & 15] = a1[v];
    }
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kLayerWaves; ++w)
        sum += sh.sums[w][tid >> 4][tid & 15];
    return sum;
}

// W1: the gate's and the other 16 rows of 16 inner values, for all slots of an
// expert.
template <typename X, typename W>
__global__ void __launch_bounds__(kLayerThreads) layer_up_kernel(LayerParams p)
{
    typedef Math<X, W, true> M;
    __shared__ LayerShared sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int f0 = (int)(blockIdx.x % p.tiles) * 16;
    int e;
    if (!find_expert(p, blockIdx.x / p.tiles, sh, e))
        return;
    const int n = sh.count;
    const int wbytes = M::MX4 ? (p.H + 1) / 2 : p.H * (M::I8 ? 1 : (int)sizeof(X));
    const signed char *w[2];
    const uint32_t *sc[2] = {nullptr, nullptr};
    const int row = min(f0 + (lane & 15), p.F - 1);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        w[t] = static_cast<const signed char *>(p.W1) + e * p.strideW1 +
               (row + (long long)t * p.F) * p.ldw1;
        if constexpr (M::MX4)
            sc[t] = static_cast<const uint32_t *>(p.scale1) +
                    (long long)e * ((p.H + 127) / 128) * 2 * p.F + row + (long long)t * p.F;
    }
    const int slots = p.tokens * p.topk;
    auto columns = [&](int c0, auto groups) {
        constexpr int CG = decltype(groups)::value;
        const signed char *x[CG];
#pragma unroll
        for (int g = 0; g < CG; ++g) {
            const int slot = sh.slots[min(c0 + 16 * g + (lane & 15), n - 1)];
            x[g] = static_cast<const signed char *>(p.X) + (slot / p.topk) * p.ldx * sizeof(X);
        }
        f32x4 acc[2][CG] = {};
        products<M, true, CG>(w, wbytes, sc, 2LL * p.F, p.H, x, (long long)p.H * sizeof(X), acc);
#pragma unroll
        for (int g = 0; g < CG; ++g) {
            const float mine = join(acc[0][g], acc[1][g], sh);
            // Thread i < 256 holds the gate's row i / 16, thread 256 + i the other's.
            __syncthreads();
            if (tid >= 256)
                sh.sums[0][(tid >> 4) - 16][tid & 15] = mine;
            __syncthreads();
            const int f = f0 + (tid >> 4), c = c0 + 16 * g + (tid & 15);
            if (tid < 256 && c < n) {
                const int slot = sh.slots[c];
                float gate = mine, up = sh.sums[0][tid >> 4][tid & 15], a = 0.0f;
                if (f < p.F) {
                    if constexpr (M::I8) {
                        const float *s = static_cast<const float *>(p.scale1) + 2LL * p.F * e;
                        gate *= s[f];
                        up *= s[p.F + f];
                    }
                    a = gate / (1.0f + expf(-gate)) * up;
                }
                // The last tile fills the columns behind F with zeros.
                const int end = f0 + 16 < p.F ? f0 + 16 : p.inner_cols;
                for (int k = f; k < end; k += 16) {
                    float v = k < p.F ? a : 0.0f;
                    const long long at = (long long)slot * p.inner_cols + k;
                    const long long plane = (long long)slots * p.inner_cols;
                    if constexpr (M::F32) {
                        static_cast<float *>(p.inner)[at] = v;
                    } else {
                        constexpr int N = Math<X, W, false>::NX;
                        uint16_t *to = static_cast<uint16_t *>(p.inner) + at;
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            // Two terms: the second is rounded, to 16 bits in all;
                            // three hold all 24.
                            to[i * plane] = i + 1 < N
                                                ? (uint16_t)(__builtin_bit_cast(uint32_t, v) >> 16)
                                                : __builtin_bit_cast(uint16_t, (__bf16)v);
                            v = rest_of(v);
                        }
                    }
                }
            }
        }
    };
    int c0 = 0;
    for (; n - c0 > 32; c0 += 64)
        columns(c0, std::integral_constant<int, 4>{});
    if (n - c0 > 16)
        columns(c0, std::integral_constant<int, 2>{});
    else if (n - c0 > 0)
        columns(c0, std::integral_constant<int, 1>{});
}

// W2: 32 rows of it for all slots of an expert.
template <typename X, typename W>
__global__ void __launch_bounds__(kLayerThreads) layer_down_kernel(LayerParams p)
{
    typedef Math<X, W, false> M;
    __shared__ LayerShared sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int h0 = (int)(blockIdx.x % p.tiles) * kTileRows;
    int e;
    if (!find_expert(p, blockIdx.x / p.tiles, sh, e))
        return;
    const int n = sh.count;
    const int wbytes = M::MX4 ? (p.F + 1) / 2 : p.F * (M::I8 ? 1 : (int)sizeof(X));
    const signed char *w[2];
    const uint32_t *sc[2] = {nullptr, nullptr};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int row = min(h0 + 16 * t + (lane & 15), p.H - 1);
        w[t] = static_cast<const signed char *>(p.W2) + e * p.strideW2 + row * p.ldw2;
        if constexpr (M::MX4)
            sc[t] = static_cast<const uint32_t *>(p.scale2) +
                    (long long)e * ((p.F + 127) / 128) * p.H + row;
    }
    const int slots = p.tokens * p.topk;
    constexpr int ES = M::F32 ? 4 : 2; // bytes of an inner value's term
    auto columns = [&](int c0, auto groups) {
        constexpr int CG = decltype(groups)::value;
        const signed char *x[CG];
#pragma unroll
        for (int g = 0; g < CG; ++g) {
            const int slot = sh.slots[min(c0 + 16 * g + (lane & 15), n - 1)];
            x[g] = static_cast<const signed char *>(p.inner) +
                   (long long)slot * p.inner_cols * ES;
        }
        f32x4 acc[2][CG] = {};
        products<M, false, CG>(w, wbytes, sc, p.H, p.F, x, (long long)slots * p.inner_cols * ES,
                               acc);
#pragma unroll
        for (int g = 0; g < CG; ++g) {
            float mine = join(acc[0][g], acc[1][g], sh);
            const int h = h0 + (tid >> 4), c = c0 + 16 * g + (tid & 15);
            if (h < p.H && c < n) {
                if constexpr (M::I8)
                    mine *= static_cast<const float *>(p.scale2)[(long long)e * p.H + h];
                p.partial[(long long)sh.slots[c] * p.H + h] = mine;
            }
        }
    };
    int c0 = 0;
    for (; n - c0 > 32; c0 += 64)
        columns(c0, std::integral_constant<int, 4>{});
    if (n - c0 > 16)
        columns(c0, std::integral_constant<int, 2>{});
    else if (n - c0 > 0)
        columns(c0, std::integral_constant<int, 1>{});
}

// out[t] = sum_j mix[t, j] partial[t, j]
template <typename X>
__global__ void __launch_bounds__(256) layer_join_kernel(LayerParams p)
{
    const long long at = blockIdx.x * 256LL + threadIdx.x;
    if (at >= (long long)p.tokens * p.H)
        return;
    const int t = (int)(at / p.H), h = (int)(at % p.H);
    float sum = 0.0f;
    for (int j = 0; j < p.topk; ++j) {
        const int slot = t * p.topk + j;
        if (p.F > 0 && id_of(p, slot) >= 0)
            sum = __builtin_fmaf(p.mix ? p.mix[slot] : 1.0f,
                                 p.partial[(long long)slot * p.H + h], sum);
    }
    static_cast<X *>(p.out)[t * p.ldo + h] = (X)sum;
}

template <typename X, typename W> int launch_layer(LayerParams p, hipStream_t s)
{
    const int slots = p.tokens * p.topk, most = slots < p.experts ? slots : p.experts;
    void *args[] = {&p};
    hipError_t e = hipSuccess;
    if (p.F > 0) {
        p.tiles = (p.F + 15) / 16;
        if (!fits_launch((double)most * p.tiles, kLayerThreads) ||
            !fits_launch((double)most * ((p.H + kTileRows - 1) / kTileRows), kLayerThreads))
            return -22;
        e = hipLaunchKernel((const void *)layer_up_kernel<X, W>, dim3((unsigned)(most * p.tiles)),
                            dim3(kLayerThreads), args, 0, s);
        if (e != hipSuccess)
            return (int)e;
        p.tiles = (p.H + kTileRows - 1) / kTileRows;
        e = hipLaunchKernel((const void *)layer_down_kernel<X, W>,
                            dim3((unsigned)(most * p.tiles)), dim3(kLayerThreads), args, 0, s);
        if (e != hipSuccess)
            return (int)e;
    }
    const long long items = (long long)p.tokens * p.H;
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

long long padded_cols(int F) { return ((long long)F + 127) / 128 * 128; }

// Bytes of the inner values, a multiple of 16 (inner_cols is one of 128).
size_t inner_bytes(long long slots, int F, int type)
{
    return (size_t)slots * padded_cols(F) * (type == SGEMM_F32 ? 6 : 4);
}

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
    return inner_bytes(slots, F, type) + (size_t)slots * H * sizeof(float);
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
    p.inner = workspace;
    p.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                          inner_bytes((long long)tokens * topk, F, type));
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
