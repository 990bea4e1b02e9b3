/*
 * Drives the host side of liblinear_norm (argument checks, plans, launches) over a large seeded
 * sample of valid and invalid arguments, for a host-only build under AddressSanitizer and
 * UndefinedBehaviorSanitizer (tests/test_linear_norm_sanitizers.py).  There is no GPU and no HIP
 * runtime: the runtime entry points the library imports are defined here; a launch is counted
 * and its grid checked, and nothing runs.  Pointers are fake, never dereferenced.  Prints counts
 * and "ok"; sanitizers abort the process on the first finding.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "linear_norm.h"

typedef struct { unsigned x, y, z; } dim3_t;
char FATBIN_SYM[64];
static long launches = 0;
static dim3_t grid, block;
void **__hipRegisterFatBinary(const void *data) { static void *h; (void)data; return &h; }
void __hipRegisterFunction(void **m, const void *f, char *d, const char *n, unsigned t, void *a,
                           void *b, void *c, void *e, int *w)
{
    (void)m, (void)f, (void)d, (void)n, (void)t, (void)a, (void)b, (void)c, (void)e, (void)w;
}
void __hipUnregisterFatBinary(void **m) { (void)m; }
void __hipRegisterVar(void **m, void *var, char *hv, const char *dv, int ext, size_t size,
                      int constant, int global)
{
    (void)m, (void)var, (void)hv, (void)dv, (void)ext, (void)size, (void)constant, (void)global;
}
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t s, void *q)
{
    (void)s, (void)q;
    grid = g, block = b;
    return 0;
}
int __hipPopCallConfiguration(dim3_t *g, dim3_t *b, size_t *s, void **q)
{
    *g = grid, *b = block, *s = 0, *q = NULL;
    return 0;
}
static int last_error = 0;
int hipLaunchKernel(const void *f, dim3_t g, dim3_t b, void **a, size_t s, void *q)
{
    (void)f, (void)a, (void)s, (void)q;
    ++launches;
    if (g.x < 1 || g.y != 1 || g.z != 1 || b.x < 64 || b.x > 1024 || b.x % 64) {
        printf("bad launch: grid %u %u %u block %u\n", g.x, g.y, g.z, b.x);
        exit(1);
    }
    /* the runtime refuses grids of 2^32 threads */
    last_error = (uint64_t)g.x * b.x >= ((uint64_t)1 << 32);
    return last_error;
}
int hipGetLastError(void) { const int e = last_error; last_error = 0; return e; }

static uint64_t state = 0x9E3779B97F4A7C15ull;
static uint64_t next(void)
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return state;
}
static int64_t pick(const int64_t *v, int n) { return v[next() % (uint64_t)n]; }
/* the first n_valid entries of v are valid values: drawn 15 times in 16 */
static int64_t mostly(const int64_t *v, int n_valid, int n)
{
    return (next() & 15) ? pick(v, n_valid) : pick(v, n);
}

static const int64_t dims[] = {1, 2, 8, 16, 17, 31, 63, 64, 65, 255, 256, 257, 1000, 4093, 4096,
                               4097, 8192, 20000, 0, 1 << 20, ((int64_t)1 << 31) - 1,
                               (int64_t)1 << 31, -1, (int64_t)1 << 62};
static const int64_t pads[] = {0, 0, 0, 1, 3, 8, 64, 16, -1, (int64_t)1 << 40, INT64_MAX / 4};
static int64_t dim(void) { return mostly(dims, 18, 24); }
static int64_t pad(void) { return mostly(pads, 8, 11); }
/* matrix i at its own 2^56 bytes; now and then null, misaligned, or another matrix's */
static void *at(int i)
{
    const uint64_t r = next() % 64;
    if (r == 0) return NULL;
    if (r == 1) return (void *)(uintptr_t)(((uint64_t)(1 + i) << 56) + 1);
    if (r == 2) i = (int)(next() % 8);
    return (void *)(uintptr_t)((uint64_t)(1 + i) << 56);
}
static void *sometimes(int i) { return next() & 1 ? at(i) : NULL; }
static long calls = 0, good = 0;
static void count(int rc)
{
    ++calls;
    if (rc == GEMM_F16F32_OK) ++good;
    if (rc > 0 || rc < -9) {
        printf("unknown code %d\n", rc);
        exit(1);
    }
}

int main(void)
{
    for (long i = 0; i < 300000; ++i) {
        const int64_t m = dim(), n = dim(), k = dim();
        const int cols_a = next() & 1, cols_b = next() & 1, cols_db = next() & 1;
        linear_forward_args f;
        memset(&f, 0, sizeof f);
        f.m = m, f.n = n, f.k = k;
        f.type = (int64_t)(next() % 3);
        if (next() % 32 == 0) f.type = 7;
        f.out_type = f.type == 2 ? (int64_t)(next() & 1) : f.type;
        f.activation = (int64_t)(next() % 5);
        const int64_t unit = f.type == 2 ? 16 : 1;
        f.a = at(0), f.b = at(1), f.out = at(2), f.pre = sometimes(3), f.residual = sometimes(4);
        f.bias = sometimes(5);
        f.a_row = (k + unit - 1) / unit * unit + pad() / unit * unit, f.a_col = 1;
        if (cols_a && f.type != 2) f.a_row = 1, f.a_col = m + pad();
        f.b_row = n + pad(), f.b_col = 1;
        if (cols_b || f.type == 2) f.b_row = 1, f.b_col = (k + unit - 1) / unit * unit + pad() / unit * unit;
        f.out_row = n + pad(), f.pre_row = n + pad(), f.residual_row = n + pad();
        int64_t need = linear_forward_workspace(&f);
        if (need > 0) f.workspace = at(8), f.workspace_bytes = need - (next() % 16 == 0);
        count(linear_forward(&f));

        linear_backward_args w;
        memset(&w, 0, sizeof w);
        w.m = m, w.n = n, w.k = k;
        w.type = (int64_t)(next() & 1);
        w.activation = (int64_t)(next() % 5);
        w.dc = at(0), w.a = at(1), w.b = at(2), w.pre = at(3);
        w.da = sometimes(4), w.db = sometimes(5), w.dbias = sometimes(6);
        w.dc_row = n + pad(), w.pre_row = n + pad(), w.da_row = k + pad();
        w.a_row = cols_a ? 1 : k + pad(), w.a_col = cols_a ? m + pad() : 1;
        w.b_row = cols_b ? 1 : n + pad(), w.b_col = cols_b ? k + pad() : 1;
        w.db_row = cols_db ? 1 : n + pad(), w.db_col = cols_db ? k + pad() : 1;
        need = linear_backward_workspace(&w);
        if (need > 0) w.workspace = at(8), w.workspace_bytes = need - (next() % 16 == 0);
        count(linear_backward(&w));

        rms_norm_forward_args r;
        memset(&r, 0, sizeof r);
        r.rows = m, r.dim = n;
        r.type = (int64_t)(next() & 1);
        r.out_type = next() & 1 ? r.type : 2;
        r.x = at(0), r.weight = at(1), r.y = at(2), r.residual = sometimes(3), r.h = sometimes(4);
        r.rstd = sometimes(5), r.scale = r.out_type == 2 ? at(6) : NULL;
        r.x_row = n + pad(), r.y_row = n + pad(), r.residual_row = n + pad(), r.h_row = n + pad();
        r.eps = next() % 16 ? 1e-5 : -1.0;
        count(rms_norm_forward(&r));

        rms_norm_backward_args q;
        memset(&q, 0, sizeof q);
        q.rows = m, q.dim = n;
        q.type = (int64_t)(next() & 1);
        q.dy = at(0), q.h = at(1), q.weight = at(2), q.rstd = at(3), q.dx = at(4);
        q.dh = sometimes(5), q.dweight = sometimes(6);
        q.dy_row = n + pad(), q.h_row = n + pad(), q.dx_row = n + pad(), q.dh_row = n + pad();
        need = rms_norm_backward_workspace(&q);
        if (need > 0) q.workspace = at(8), q.workspace_bytes = need - (next() % 16 == 0);
        count(rms_norm_backward(&q));
    }
    if (good < calls / 10 || launches < good / 2) {
        printf("sample too weak: %ld calls, %ld good, %ld launches\n", calls, good, launches);
        return 1;
    }
    printf("%ld calls, %ld good, %ld launches: ok\n", calls, good, launches);
    return 0;
}
