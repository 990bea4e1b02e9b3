/*
 * The largest extents that liblinear_norm's host side accepts: every call here has to be launched
 * in grids that the runtime takes, or be refused by a code of its own, never by the runtime
 * (GEMM_F16F32_ERR_HIP).  The stand-ins for the runtime are those of sanitize_linear_norm.c.
 */
#define main sampled_main
#include "sanitize_linear_norm.c"
#undef main

enum { F16 = LINEAR_NORM_F16, E4M3 = LINEAR_NORM_E4M3 };
static const int64_t TOP = ((int64_t)1 << 31) - 1;
static int failures = 0;

static void *matrix(int i) { return (void *)(uintptr_t)((uint64_t)(1 + i) << 56); }

static void expect(const char *what, int64_t m, int64_t n, int64_t k, int rc, int want)
{
    if (rc == want) return;
    printf("%s %lld x %lld x %lld: %d, not %d\n", what, (long long)m, (long long)n, (long long)k,
           rc, want);
    ++failures;
}

/* b_cols: b is stored k-contiguous */
static void forward(int64_t type, int64_t m, int64_t n, int64_t k, int b_cols, int want)
{
    const int64_t row = type == E4M3 ? (k + 15) / 16 * 16 : k;
    linear_forward_args f;
    memset(&f, 0, sizeof f);
    f.m = m, f.n = n, f.k = k, f.type = type, f.out_type = F16;
    f.a = matrix(0), f.a_row = row, f.a_col = 1;
    f.b = matrix(1), f.b_row = b_cols ? 1 : n, f.b_col = b_cols ? row : 1;
    f.out = matrix(2), f.out_row = n;
    const int64_t need = linear_forward_workspace(&f);
    if (need > 0) f.workspace = matrix(8), f.workspace_bytes = need;
    expect("forward", m, n, k, linear_forward(&f), want);
}

static void bias_gradient(int64_t m, int64_t n)
{
    linear_backward_args w;
    memset(&w, 0, sizeof w);
    w.m = m, w.n = n, w.k = 8;
    w.dc = matrix(0), w.dc_row = n, w.dbias = matrix(1);
    w.a = matrix(2), w.a_row = 8, w.a_col = 1, w.b = matrix(3), w.b_row = n, w.b_col = 1;
    const int64_t need = linear_backward_workspace(&w);
    if (need > 0) w.workspace = matrix(8), w.workspace_bytes = need;
    expect("bias gradient", m, n, 8, linear_backward(&w), GEMM_F16F32_OK);
}

static void norms(int64_t rows, int64_t dim)
{
    rms_norm_forward_args r;
    memset(&r, 0, sizeof r);
    r.rows = rows, r.dim = dim;
    r.x = matrix(0), r.weight = matrix(1), r.y = matrix(2);
    r.x_row = r.y_row = dim;
    expect("norm", rows, dim, 0, rms_norm_forward(&r), GEMM_F16F32_OK);
    rms_norm_backward_args q;
    memset(&q, 0, sizeof q);
    q.rows = rows, q.dim = dim;
    q.dy = matrix(0), q.h = matrix(1), q.weight = matrix(2), q.rstd = matrix(3), q.dx = matrix(4);
    q.dy_row = q.h_row = q.dx_row = dim, q.dweight = matrix(5);
    const int64_t need = rms_norm_backward_workspace(&q);
    if (need > 0) q.workspace = matrix(8), q.workspace_bytes = need;
    expect("norm backward", rows, dim, 0, rms_norm_backward(&q), GEMM_F16F32_OK);
}

int main(void)
{
    static const int64_t columns[] = {((int64_t)1 << 26) + 5, ((int64_t)1 << 27) - 16, (int64_t)1 << 27,
                                      ((int64_t)1 << 27) + 16, ((int64_t)1 << 28) + 1,
                                      (int64_t)1 << 29, ((int64_t)1 << 29) + 8, (int64_t)1 << 30,
                                      ((int64_t)1 << 31) - 1};
    static const int64_t depths[] = {1, 7, 8, 15, 16, 100};
    for (unsigned c = 0; c < sizeof columns / sizeof *columns; ++c)
        for (unsigned d = 0; d < sizeof depths / sizeof *depths; ++d)
            for (int64_t m = 1; m <= 16; m += 5) {
                forward(F16, m, columns[c], depths[d], 1, GEMM_F16F32_OK);
                forward(E4M3, m, columns[c], depths[d], 1,
                        columns[c] > TOP - 128 ? GEMM_F16F32_ERR_TOO_LARGE : GEMM_F16F32_OK);
            }
    /* b row-major: a panel's 64 rows pass the 32-bit offsets */
    forward(F16, 1, (int64_t)1 << 28, 8, 0, GEMM_F16F32_OK);
    forward(F16, 1, ((int64_t)1 << 29) + 8, 8, 0, GEMM_F16F32_ERR_TOO_LARGE);
    forward(F16, 17, ((int64_t)1 << 25) + 8, 8, 0, GEMM_F16F32_ERR_TOO_LARGE);
    forward(F16, TOP, 1, 8, 1, GEMM_F16F32_OK);
    forward(F16, TOP, 64, 64, 1, GEMM_F16F32_OK);
    forward(F16, (int64_t)1 << 30, 100, 1, 0, GEMM_F16F32_OK);
    forward(E4M3, TOP - 1000, 16, 16, 1, GEMM_F16F32_OK);
    forward(E4M3, TOP, 16, 16, 1, GEMM_F16F32_ERR_TOO_LARGE);
    forward(F16, 1, 64, TOP, 1, GEMM_F16F32_OK);
    bias_gradient(TOP, 8);
    bias_gradient(8, TOP);
    bias_gradient((int64_t)1 << 27, (int64_t)1 << 27);
    norms(TOP, 1);
    norms(TOP, 8);
    norms(1, TOP);
    norms(3, ((int64_t)1 << 29) + 1);
    if (failures) return 1;
    printf("ok\n");
    return 0;
}
