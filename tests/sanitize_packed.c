/*
 * Drives the host side of the layer norm, the 8-bit rows and the checkpoints in liblinear_norm over a
 * large seeded sample of valid and invalid arguments, and over the largest extents, for a host-only
 * build under AddressSanitizer and UndefinedBehaviorSanitizer (tests/test_packed_sanitizers.py).
 * The stand-ins for the HIP runtime are those of sanitize_linear_norm.c.
 */
#define main sampled_main
#include "sanitize_linear_norm.c"
#undef main

enum { F16 = LINEAR_NORM_F16, BF16 = LINEAR_NORM_BF16, E4M3 = LINEAR_NORM_E4M3, I8 = LINEAR_NORM_I8 };
static const int64_t TOP = ((int64_t)1 << 31) - 1;
static int failures = 0;

static packed8_matrix packed(int i, int64_t dim, int64_t more)
{
    packed8_matrix p;
    p.values = at(i), p.values_row = dim + more;
    p.scale = at(i + 1), p.scale_row = (dim + 31) / 32 + (more > 0 && more < 100 ? more : 0);
    return p;
}
static int64_t out_type(int64_t type)
{
    static const int64_t t[] = {E4M3, I8};
    return next() & 1 ? type : pick(t, 2);
}

static void sample(void)
{
    const int64_t m = dim(), n = dim(), k = dim();
    layer_norm_forward_args r;
    memset(&r, 0, sizeof r);
    r.rows = m, r.dim = n, r.type = (int64_t)(next() & 1), r.out_type = out_type(r.type);
    r.x = at(0), r.weight = at(1), r.y = at(2), r.residual = sometimes(3), r.h = sometimes(4);
    r.rstd = sometimes(5), r.mean = sometimes(6), r.bias = sometimes(7);
    r.scale = r.out_type != r.type ? at(9) : NULL;
    r.x_row = n + pad(), r.y_row = n + pad(), r.residual_row = n + pad(), r.h_row = n + pad();
    r.eps = next() % 16 ? 1e-5 : -1.0;
    count(layer_norm_forward(&r));

    layer_norm_backward_args q;
    memset(&q, 0, sizeof q);
    q.rows = m, q.dim = n, q.type = (int64_t)(next() & 1);
    q.dy = at(0), q.h = at(1), q.weight = at(2), q.rstd = at(3), q.dx = at(4), q.mean = at(7);
    q.dh = sometimes(5), q.dweight = sometimes(6), q.dbias = sometimes(9);
    q.dy_row = n + pad(), q.h_row = n + pad(), q.dx_row = n + pad(), q.dh_row = n + pad();
    int64_t need = layer_norm_backward_workspace(&q);
    if (need > 0) q.workspace = at(8), q.workspace_bytes = need - (next() % 16 == 0);
    count(layer_norm_backward(&q));

    quantize_rows_args z;
    memset(&z, 0, sizeof z);
    z.rows = m, z.dim = n, z.type = (int64_t)(next() & 1), z.out_type = next() & 1 ? E4M3 : I8;
    z.x = at(0), z.values = at(1), z.scale = at(2), z.x_row = n + pad(), z.values_row = n + pad();
    count(quantize_rows(&z));

    pack8_args p;
    memset(&p, 0, sizeof p);
    p.rows = m, p.dim = n, p.type = (int64_t)(next() & 1), p.x = at(0), p.x_row = n + pad();
    p.out = packed(1, n, pad());
    count(pack8(&p));

    unpack8_args u;
    memset(&u, 0, sizeof u);
    u.rows = m, u.dim = n, u.type = (int64_t)(next() & 1), u.activation = (int64_t)(next() % 5);
    u.in = packed(1, n, pad()), u.y = at(0), u.y_row = n + pad();
    count(unpack8(&u));

    linear_forward_args f;
    memset(&f, 0, sizeof f);
    f.m = m, f.n = n, f.k = k;
    f.type = next() & 1 ? I8 : (int64_t)(next() % 3);
    f.out_type = f.type >= E4M3 ? (int64_t)(next() & 1) : f.type;
    f.activation = (int64_t)(next() % 5);
    const int64_t unit = f.type >= E4M3 ? 16 : 1, row = (k + unit - 1) / unit * unit;
    f.a = at(0), f.b = at(1), f.out = at(2), f.residual = sometimes(4), f.bias = sometimes(5);
    f.a_row = row + pad() / unit * unit, f.a_col = 1;
    f.b_row = 1, f.b_col = row + pad() / unit * unit;
    f.out_row = n + pad(), f.residual_row = n + pad();
    packed8_matrix pre = packed(9, n, pad());
    need = linear_forward_packed_workspace(&f, &pre);
    if (need > 0) f.workspace = at(8), f.workspace_bytes = need - (next() % 16 == 0);
    count(linear_forward_packed(&f, &pre));

    linear_backward_args w;
    linear_kept kept;
    memset(&w, 0, sizeof w);
    memset(&kept, 0, sizeof kept);
    w.m = m, w.n = n, w.k = k, w.type = (int64_t)(next() & 1);
    w.activation = (int64_t)(next() % 5);
    w.dc = at(0), w.b = at(2), w.da = sometimes(4), w.db = sometimes(5), w.dbias = sometimes(6);
    w.dc_row = n + pad(), w.pre_row = n + pad(), w.da_row = k + pad();
    w.a_row = k + pad(), w.a_col = 1, w.b_row = 1, w.b_col = k + pad();
    w.db_row = n + pad(), w.db_col = 1;
    if (next() & 1)
        kept.a = packed(9, k, pad()), kept.a_activation = (int64_t)(next() % 5);
    else
        w.a = at(1);
    if (next() & 1) kept.pre = packed(11, n, pad());
    else w.pre = at(3);
    need = linear_backward_packed_workspace(&w, &kept);
    if (need > 0) w.workspace = at(8), w.workspace_bytes = need - (next() % 16 == 0);
    count(linear_backward_packed(&w, &kept));
}

static void *matrix(int i) { return (void *)(uintptr_t)((uint64_t)(1 + i) << 56); }
static void expect(const char *what, int64_t rows, int64_t dim, int rc)
{
    if (rc == GEMM_F16F32_OK) return;
    printf("%s %lld x %lld: %d\n", what, (long long)rows, (long long)dim, rc);
    ++failures;
}
/* every call has to be launched in grids that the runtime takes */
static void largest(int64_t rows, int64_t cols)
{
    layer_norm_forward_args r;
    memset(&r, 0, sizeof r);
    r.rows = rows, r.dim = cols, r.x = matrix(0), r.weight = matrix(1), r.y = matrix(2);
    r.x_row = r.y_row = cols;
    expect("layer norm", rows, cols, layer_norm_forward(&r));
    layer_norm_backward_args q;
    memset(&q, 0, sizeof q);
    q.rows = rows, q.dim = cols, q.dy = matrix(0), q.h = matrix(1), q.weight = matrix(2);
    q.mean = matrix(3), q.rstd = matrix(4), q.dx = matrix(5), q.dweight = matrix(6);
    q.dbias = matrix(7), q.dy_row = q.h_row = q.dx_row = cols;
    q.workspace_bytes = layer_norm_backward_workspace(&q), q.workspace = matrix(8);
    expect("layer norm backward", rows, cols, layer_norm_backward(&q));
    quantize_rows_args z;
    memset(&z, 0, sizeof z);
    z.rows = rows, z.dim = cols, z.out_type = I8, z.x = matrix(0), z.values = matrix(1);
    z.scale = matrix(2), z.x_row = z.values_row = cols;
    expect("quantize", rows, cols, quantize_rows(&z));
    packed8_matrix p = {matrix(1), cols, matrix(2), (cols + 31) / 32};
    pack8_args k = {rows, cols, F16, matrix(0), cols, p, NULL};
    expect("pack", rows, cols, pack8(&k));
    unpack8_args u = {rows, cols, BF16, LINEAR_ACT_GELU, p, matrix(0), cols, NULL};
    expect("unpack", rows, cols, unpack8(&u));
    /* a bias gradient, with an operand restored beside it */
    linear_backward_args w;
    linear_kept kept;
    memset(&w, 0, sizeof w);
    memset(&kept, 0, sizeof kept);
    w.m = rows, w.n = 8, w.k = cols, w.dc = matrix(0), w.dc_row = 8, w.b = matrix(3);
    w.b_row = 8, w.b_col = 1, w.db = matrix(4), w.db_row = 8, w.db_col = 1, w.dbias = matrix(5);
    kept.a = p;
    const int64_t need = linear_backward_packed_workspace(&w, &kept);
    if (need == GEMM_F16F32_ERR_TOO_LARGE) return;   /* a panel's offsets */
    w.workspace = matrix(8), w.workspace_bytes = need;
    expect("backward", rows, cols, linear_backward_packed(&w, &kept));
}

int main(void)
{
    for (long i = 0; i < 100000; ++i) sample();
    if (good < calls / 10 || launches < good / 2) {
        printf("sample too weak: %ld calls, %ld good, %ld launches\n", calls, good, launches);
        return 1;
    }
    static const int64_t sizes[] = {1, 3, 31, 64, 1000, 16384, 16385, (int64_t)1 << 21};
    for (int i = 0; i < 8; ++i) {
        largest(TOP, sizes[i]);
        largest(sizes[i], TOP);
        largest(TOP / sizes[i], sizes[i] + 1);
    }
    if (failures) return 1;
    printf("%ld calls, %ld good, %ld launches: ok\n", calls, good, launches);
    return 0;
}
