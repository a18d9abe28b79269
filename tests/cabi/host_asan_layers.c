/*
 * Host-side checks of the norms, the 4-bit calls and the experts' layer under
 * AddressSanitizer and the undefined-behaviour checks: test infrastructure,
 * built as host_asan.c is. Over many seeded arguments it drives
 *   - the choice of kernel (mx4gemm_select_kernel), checking its range;
 *   - the workspace sizes, checking their bounds;
 *   - argument validation of every call and quick returns, with pointers that
 *     must never be dereferenced.
 * Nothing here reaches a device call. Exit status 0 only if every check passed.
 */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>

#include "experts.h"
#include "mx4gemm.h"
#include "norm.h"

static int failures = 0;

#define CHECK(cond, ...)                      \
    do {                                      \
        if (!(cond)) {                        \
            if (failures < 20) {              \
                fprintf(stderr, __VA_ARGS__); \
                fputc('\n', stderr);          \
            }                                 \
            ++failures;                       \
        }                                     \
    } while (0)

static uint64_t rng_state = 0x9e3779b97f4a7c15ull;
static uint64_t next_u64(void)
{
    rng_state ^= rng_state << 13;
    rng_state ^= rng_state >> 7;
    rng_state ^= rng_state << 17;
    return rng_state;
}

/* A size from a mix of scales: tiny, around the tile sizes, large and close to
   the int range; 0 and negative now and then. */
static int dim(void)
{
    switch (next_u64() % 8) {
    case 0: return (int)(next_u64() % 9);
    case 1: return 1 + (int)(next_u64() % 130);
    case 2: return 1 + (int)(next_u64() % 5000);
    case 3: return 1 + (int)(next_u64() % 70000);
    case 4: return 1 << (next_u64() % 31);
    case 5: return INT_MAX - (int)(next_u64() % 70000);
    case 6: return -(int)(next_u64() % 5);
    default: return 1 + (int)(next_u64() % 0x7ffffffeu);
    }
}

static void choices(int rounds)
{
    for (int i = 0; i < rounds; ++i) {
        const int M = dim(), N = dim(), K = dim(), groups = next_u64() % 2 ? 0 : dim();
        const int k = mx4gemm_select_kernel(M, N, K, groups, (int)(next_u64() & 1),
                                            (int)(next_u64() % 512));
        CHECK(k < MX4GEMM_KERNEL_COUNT && (k >= 0 || k == -22 || k == -1501 || k == -1502 ||
                                           k == -1503 || k == -1604),
              "mx4gemm_select_kernel(%d, %d, %d, %d) = %d", M, N, K, groups, k);
        const int type = (int)(next_u64() % 5);
        const size_t g = rms_norm_grad_workspace_size(M, K, type);
        CHECK(g <= (size_t)16 * 1024 * RMS_NORM_GRAD_MAX_K * sizeof(float),
              "rms_norm_grad_workspace_size(%d, %d, %d) = %zu", M, K, type, g);
        const size_t l = expert_layer_workspace_size(M, N, K, groups, type);
        CHECK(l <= (size_t)EXPERT_LAYER_MAX_SLOTS * (2 << 20) * sizeof(float),
              "expert_layer_workspace_size(%d, %d, %d, %d) = %zu", M, N, K, groups, l);
    }
}

/* Calls whose last check fails whatever came before, so that no valid one
   reaches a launch: some pointer is NULL where it may not be. */
static void refusals(int rounds)
{
    void *wild = (void *)(uintptr_t)0x1000;
    float *f = wild;
    unsigned char *u = wild;
    for (int i = 0; i < rounds; ++i) {
        const int M = dim(), N = dim(), K = dim(), a = dim(), b = dim(), c = dim(), d = dim();
        const int t = (int)(next_u64() % 5), g = dim();
        const long long ll = (long long)next_u64();
        int st[] = {
            rms_norm(M, K, wild, t, a, wild, b, f, 0.0f, wild, c, NULL, d, NULL),
            rms_norm_i8(M, K, wild, t, a, wild, b, f, 0.0f, wild, c, NULL, d, NULL, NULL),
            rms_norm_grad(M, K, wild, t, a, wild, b, f, 0.0f, wild, c, NULL, d, NULL, NULL, 0, NULL),
            mx4_quantize_rows(M, K, wild, t, a, u, b, NULL, c, NULL),
            mx4_dequantize_rows(M, K, u, a, u, b, NULL, t, c, NULL),
            mx4gemm(M, N, K, u, a, u, b, u, c, u, d, NULL, NULL, t, g, NULL),
            mx4gemm_grouped(M, N, K, g, wild, u, a, u, b, u, c, ll, u, d, 4 * (ll / 4), NULL, NULL,
                            t, N, NULL),
            expert_layer(M, N, K, a, b, wild, t, c, wild, 4, NULL, wild, (int)(next_u64() % 6), d,
                         ll, wild, wild, g, ll / 2, wild, wild, a, NULL, (size_t)next_u64(), NULL),
        };
        /* (rms_norm_i8 of empty rows would launch: its scale is missing here.) */
        for (size_t k = 0; k < sizeof st / sizeof *st; ++k) {
            const int base = 1000 + 100 * (int)k;
            CHECK(st[k] == 0 || (st[k] < -base && st[k] > -base - 100), "call %zu gave %d", k, st[k]);
        }
    }
}

int main(void)
{
    choices(200000);
    refusals(200000);
    printf("host checks: %d failures\n", failures);
    return failures != 0;
}
