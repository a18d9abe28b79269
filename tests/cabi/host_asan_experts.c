/*
 * Host-side checks of the expert, grouped and 8-bit calls under
 * AddressSanitizer and the undefined-behaviour checks: test infrastructure,
 * built as host_asan.c is. Over many seeded arguments it drives
 *   - the choices of kernel (i8gemm_select_kernel, sgemm_grouped_select_kernel,
 *     sgemm_grouped_outer_select_kernel), checking their ranges;
 *   - the sort's plan (expert_sort_workspace_size), checking its bounds;
 *   - argument validation of every call, with one argument of a valid call
 *     replaced, and quick returns, with pointers that must never be
 *     dereferenced; every status has a message of its own.
 * Nothing here reaches a device call. Exit status 0 only if every check passed.
 */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "experts.h"
#include "i8gemm.h"

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
   the int range; 0 now and then. */
static int dim(void)
{
    switch (next_u64() % 7) {
    case 0: return (int)(next_u64() % 9);
    case 1: return 1 + (int)(next_u64() % 130);
    case 2: return 1 + (int)(next_u64() % 5000);
    case 3: return 1 + (int)(next_u64() % 70000);
    case 4: return 1 << (next_u64() % 31);
    case 5: return INT_MAX - (int)(next_u64() % 600);
    default: return 1 + (int)(next_u64() % 0x7ffffffeu);
    }
}

static void choices(int rounds)
{
    for (int r = 0; r < rounds; ++r) {
        const int M = dim(), N = dim(), K = dim() % (I8GEMM_MAX_K + 1);
        const int groups = next_u64() % 3 ? (int)(next_u64() % 65537) : 0;
        const int flag = (int)(next_u64() % 2), tB = (int)(next_u64() % 2);
        const int cus = (int)(next_u64() % 1024);
        int k = i8gemm_select_kernel(M, N, K, groups, flag, cus);
        CHECK(k == -22 || (k >= 0 && k < I8GEMM_KERNEL_COUNT),
              "i8gemm_select_kernel(%d, %d, %d, %d, %d, %d) = %d", M, N, K, groups, flag, cus, k);
        k = sgemm_grouped_select_kernel(tB, M, N, groups, flag, cus);
        CHECK(k == -22 || (k >= 0 && k < SGEMM_GROUPED_COUNT),
              "sgemm_grouped_select_kernel(%d, %d, %d, %d, %d, %d) = %d", tB, M, N, groups, flag,
              cus, k);
        const int many = dim();
        k = sgemm_grouped_outer_select_kernel(M, N, many, flag, cus);
        CHECK(k == -22 || (k >= 0 && k < SGEMM_GROUPED_OUTER_COUNT),
              "sgemm_grouped_outer_select_kernel(%d, %d, %d, %d, %d) = %d", M, N, many, flag, cus,
              k);
    }
}

static void sort_plans(int rounds)
{
    for (int r = 0; r < rounds; ++r) {
        const int tokens = dim(), topk = 1 + (int)(next_u64() % 16);
        const int experts = 1 + (int)(next_u64() % EXPERT_SORT_MAX_EXPERTS);
        const size_t need = expert_sort_workspace_size(tokens, topk, experts);
        const size_t a_run = (size_t)(experts + 1) * sizeof(int);
        CHECK(need % a_run == 0 && need <= 256 * a_run, "workspace of %d x %d, %d experts: %zu",
              tokens, topk, experts, need);
        if ((long long)tokens * topk > INT_MAX || (long long)tokens * topk <= 2048)
            CHECK(need == 0, "workspace of %d x %d: %zu", tokens, topk, need);
    }
}

/* Every call takes its integers from v and its pointers from p, in the order
   of its arguments, so that one of them can be replaced. */
enum { MOST = 20 };
typedef struct {
    long long v[MOST];
    void *p[MOST];
} Args;

#define I(i) ((int)a->v[i])
#define P(i) (a->p[i])
static int call_quantize(const Args *a)
{
    return i8_quantize_rows(I(1), I(2), P(3), I(4), I(5), P(6), I(7), P(8), NULL);
}
static int call_i8gemm(const Args *a)
{
    return i8gemm(I(1), I(2), I(3), P(4), I(5), P(6), P(7), I(8), P(9), P(10), P(11), I(12), I(13),
                  NULL);
}
static int call_i8gemm_grouped(const Args *a)
{
    return i8gemm_grouped(I(1), I(2), I(3), I(4), P(5), P(6), I(7), P(8), P(9), I(10), a->v[11],
                          P(12), P(13), P(14), I(15), I(16), NULL);
}
static int call_sort(const Args *a)
{
    return expert_sort(I(1), I(2), I(3), P(4), I(5), P(6), P(7), P(8), (size_t)a->v[9], NULL);
}
static int call_gather(const Args *a)
{
    return expert_gather(I(1), I(2), I(3), P(4), I(5), I(6), P(7), P(8), I(9), NULL);
}
static int call_combine(const Args *a)
{
    return expert_combine(I(1), I(2), I(3), P(4), I(5), I(6), P(7), P(8), P(9), I(10), NULL);
}
static int call_combine_grad(const Args *a)
{
    return expert_combine_grad(I(1), I(2), I(3), P(4), I(5), I(6), P(7), I(8), P(9), P(10), P(11),
                               I(12), P(13), NULL);
}
static int call_grouped(const Args *a)
{
    return sgemm_grouped(I(1), I(2), I(3), I(4), I(5), P(6), 1.0f, P(8), I(9), P(10), I(11),
                         a->v[12], 0.0f, P(14), I(15), NULL);
}
static int call_outer(const Args *a)
{
    return sgemm_grouped_outer(I(1), I(2), I(3), I(4), P(5), 1.0f, P(7), I(8), P(9), I(10), 0.0f,
                               P(12), I(13), a->v[14], NULL);
}
#undef I
#undef P

typedef struct {
    int (*call)(const Args *);
    int base;
    const char *name;
    /* by position: 'n' a size (at least 1), 'l' a leading dimension, 't' a type,
       's' a stride, 'p' a pointer that has to be there, 'o' one that may be
       NULL, 'x' something else, ' ' no argument that is checked */
    const char *kinds;
} Call;

static const Call calls[] = {
    {call_quantize, 100, "i8_quantize_rows", "nnptlplp"},
    {call_i8gemm, 200, "i8gemm", "nnnplpplpoptl"},
    {call_i8gemm_grouped, 300, "i8gemm_grouped", "nnnnpplpplspoptl"},
    {call_sort, 400, "expert_sort", "nnnpxppox"},
    {call_gather, 500, "expert_gather", "nnnptlppl"},
    {call_combine, 600, "expert_combine", "nnnptlpopl"},
    {call_combine_grad, 700, "expert_combine_grad", "nnnptlplpoplo"},
    {call_grouped, 800, "sgemm_grouped", "xnnnnp plpls pl"},
    {call_outer, 900, "sgemm_grouped_outer", "nnnnp plpl pls"},
};

static void arguments(int rounds)
{
    for (int r = 0; r < rounds; ++r)
        for (size_t c = 0; c < sizeof calls / sizeof calls[0]; ++c) {
            const Call *f = &calls[c];
            const int n = (int)strlen(f->kinds);
            Args a;
            memset(&a, 0, sizeof a);
            for (int i = 1; i <= n; ++i) {
                const char k = f->kinds[i - 1];
                a.v[i] = k == 'n'   ? 1 + (long long)(next_u64() % 1000)
                         : k == 'l' ? 1000 + (long long)(next_u64() % 2000)
                         : k == 't' ? (long long)(next_u64() % 3)
                         : k == 's' ? (long long)(next_u64() >> 8)
                                    : 0;
                a.p[i] = (void *)(uintptr_t)(4096 * (1 + next_u64() % 1000));
            }
            if (f->call == call_sort) {
                a.v[5] = next_u64() % 2 ? 4 : 8;
                a.v[9] = 1 << 30;
            }
            /* one argument made invalid: its status, with a message that says so */
            const int at = 1 + (int)(next_u64() % n);
            const char k = f->kinds[at - 1];
            if (k == ' ' || k == 'o')
                continue;
            if (k == 'p')
                a.p[at] = NULL;
            else if (k == 't')
                a.v[at] = next_u64() % 2 ? -1 - (long long)(next_u64() % 1000)
                                         : 4 + (long long)(next_u64() % 1000);
            else if (k == 'l' || (k == 'n' && f->call != call_sort))
                a.v[at] = next_u64() % 2 ? INT_MIN + (long long)(next_u64() % 1000)
                                         : -1 - (long long)(next_u64() % 1000);
            else if (k == 's')
                a.v[at] = next_u64() % 2 ? LLONG_MIN : -1;
            else if (f->call == call_sort && at == 9)
                a.v[1] = 1000, a.v[2] = 100, a.v[9] = 0;
            else
                a.v[at] = next_u64() % 2 ? INT_MIN : -1 - (long long)(next_u64() % 1000);
            const int st = f->call(&a), want = -(f->base + at);
            CHECK(st == want, "%s with argument %d invalid: %d, want %d", f->name, at, st, want);
            const char *m = sgemm_status_string(want);
            CHECK(m != NULL && strncmp(m, f->name, strlen(f->name)) == 0, "%s: message %s", f->name,
                  m ? m : "none");
        }
}

static void quick_returns(void)
{
    /* Nothing to compute: nothing read, whatever the pointers. */
    int *const off = (int *)(uintptr_t)4096;
    float *const P = (float *)(uintptr_t)8192;
    CHECK(i8_quantize_rows(0, 5, NULL, 0, 5, NULL, 5, NULL, NULL) == 0, "no rows to quantize");
    CHECK(i8gemm(0, INT_MAX, 8, NULL, 8, NULL, NULL, 8, NULL, NULL, NULL, 0, INT_MAX, NULL) == 0,
          "i8gemm of no rows");
    CHECK(i8gemm_grouped(5, 5, 8, 0, NULL, NULL, 8, NULL, NULL, 8, 0, NULL, NULL, NULL, 0, 5,
                         NULL) == 0, "i8gemm_grouped of no groups");
    CHECK(expert_gather(0, 3, 5, NULL, 0, 5, NULL, NULL, 5, NULL) == 0, "no tokens");
    CHECK(expert_combine(7, 3, 0, NULL, 0, 1, NULL, NULL, NULL, 1, NULL) == 0, "no columns");
    CHECK(expert_combine_grad(7, 3, 0, NULL, 0, 1, NULL, 1, NULL, NULL, NULL, 1, NULL, NULL) == 0,
          "no columns and no weights");
    CHECK(sgemm_grouped(0, 5, 5, 5, 0, NULL, 1.f, NULL, 5, NULL, 5, 0, 0.f, NULL, 5, NULL) == 0,
          "no groups");
    CHECK(sgemm_grouped(0, 5, 5, 5, 2, off, 0.f, NULL, 5, NULL, 5, 0, 1.f, P, 5, NULL) == 0,
          "alpha 0, beta 1");
    CHECK(sgemm_grouped_outer(5, 5, 0, 2, off, 1.f, NULL, 5, NULL, 5, 1.f, P, 5, 25, NULL) == 0,
          "no rows, beta 1");
    /* More tiles than a launch holds, found before the device is asked. */
    CHECK(i8gemm(INT_MAX, INT_MAX, 8, (void *)P, 8, P, (void *)P, 8, P, NULL, P, 0, INT_MAX,
                 NULL) == -22, "i8gemm of 2^62 outputs");
    CHECK(sgemm_grouped(0, INT_MAX, 2097151, 8, 65536, off, 1.f, P, 8, P, 2097151, 0, 0.f, P,
                        2097151, NULL) == -22, "sgemm_grouped of 2^52 outputs");
    CHECK(sgemm_grouped_outer(2097151, 2097151, 8, INT_MAX, off, 1.f, P, 2097151, P, 2097151, 0.f,
                              P, 2097151, 0, NULL) == -22, "sgemm_grouped_outer of 2^73 outputs");
}

int main(void)
{
    choices(200000);
    sort_plans(200000);
    arguments(20000);
    quick_returns();
    printf("host checks: %d failures\n", failures);
    return failures == 0 ? 0 : 1;
}
