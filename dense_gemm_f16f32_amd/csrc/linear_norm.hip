// C-ABI of the linear layer and the root-mean-square norm: argument checks, kernel choice,
// launches.  The declarations and their contracts are in include/linear_norm.h.
#include "linear_norm.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include "linear_launch.hpp"
#include "norm_kernels.hpp"

namespace {

using lk::GemmPlan;
using lk::LinArgs;

constexpr int64_t kMax = (int64_t)1 << 31;
constexpr int64_t kThreads = (int64_t)1 << 32;   // a launch has fewer
constexpr int kCUs = 256;

int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t round_up(int64_t x, int64_t y) { return cdiv(x, y) * y; }

bool is16(int64_t type) { return type == LINEAR_NORM_F16 || type == LINEAR_NORM_BF16; }

// ---- matrices ------------------------------------------------------------------------------
// Bytes from a matrix's first element to one past its last (rows ld apart); saturating.
struct Region {
  const void* p;
  uint64_t n;
};
Region region(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
  if (p == nullptr || rows <= 0 || cols <= 0) return {p, 0};
  const __int128 b = (__int128)elem * ((__int128)(rows - 1) * ld + cols);
  return {p, b > (__int128)UINT64_MAX ? UINT64_MAX : (uint64_t)b};
}
bool overlap(const Region& a, const Region& b) {
  if (a.n == 0 || b.n == 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x >= y ? x - y < b.n : y - x < a.n;
}
// Whether any of the nw written regions meets another of them or any of the nr read ones.
bool conflict(const Region* w, int nw, const Region* r, int nr) {
  for (int i = 0; i < nw; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(w[i], w[j])) return true;
    for (int j = 0; j < nr; ++j)
      if (overlap(w[i], r[j])) return true;
  }
  return false;
}

// A row-major matrix: row stride (of no meaning without a second row) and alignment.
int check_rows(const void* p, int64_t rows, int64_t cols, int64_t* ld, int64_t elem, bool needed) {
  if (rows <= 1 || cols == 0) *ld = cols > 0 ? cols : 1;
  if (rows == 0 || cols == 0) return GEMM_F16F32_OK;
  if (p == nullptr) return needed ? GEMM_F16F32_ERR_NULL : GEMM_F16F32_OK;
  if ((uintptr_t)p % elem) return GEMM_F16F32_ERR_OPTS;
  if (*ld < cols) return GEMM_F16F32_ERR_LD;
  // byte offsets inside the matrix stay below 2^62
  if (*ld > ((int64_t)1 << 60) / rows) return GEMM_F16F32_ERR_TOO_LARGE;
  return GEMM_F16F32_OK;
}

// A product's operand: X rows (of a) or columns (of b), K deep, element (x, k) at
// x * sx + k * sk.  km: k-contiguous, rows of ld; else x-contiguous, k rows of ld.
struct Operand {
  const void* p;
  int64_t ld;
  bool km;
};
int operand(const void* p, int64_t X, int64_t K, int64_t sx, int64_t sk, int64_t type,
            Operand* o) {
  const int64_t elem = type == LINEAR_NORM_E4M3 ? 1 : 2;
  *o = {p, K > 1 ? K : 1, true};
  if (X == 0 || K == 0) return GEMM_F16F32_OK;
  if (p == nullptr) return GEMM_F16F32_ERR_NULL;
  if ((uintptr_t)p % (elem == 1 ? 16 : 2)) return GEMM_F16F32_ERR_OPTS;
  if ((sk == 1 || K == 1) && (X == 1 || sx >= K)) {
    if (X > 1) o->ld = sx;
  } else if (elem == 2 && (sx == 1 || X == 1) && sk >= X) {
    o->ld = sk;
    o->km = false;
  } else {
    return GEMM_F16F32_ERR_LD;
  }
  if (elem == 1) {
    if (X == 1) o->ld = round_up(K, 16);
    if (o->ld % 16) return GEMM_F16F32_ERR_LD;
  }
  if (o->ld > ((int64_t)1 << 60) / (o->km ? X : K)) return GEMM_F16F32_ERR_TOO_LARGE;
  return GEMM_F16F32_OK;
}
Region operand_region(const Operand& o, int64_t X, int64_t K, int64_t type) {
  const int64_t e = type == LINEAR_NORM_E4M3 ? 1 : 2;
  return o.km ? region(o.p, X, K, o.ld, e) : region(o.p, K, X, o.ld, e);
}

// ---- matrix products -------------------------------------------------------------------------
// Sets a plan's split: the tiles from `whole` on in `splits` slices of `depth` panels or units.
void set_split(GemmPlan* g, int64_t whole, int64_t depth, int64_t splits, int64_t block) {
  g->whole = g->programs;
  g->splits = 1;
  g->per_split = (int)depth;
  if (splits < 2 || depth < 2) return;
  const int64_t per = cdiv(depth, splits);
  splits = cdiv(depth, per);   // no slice is empty
  if (splits < 2) return;
  g->whole = whole;
  g->splits = (int)splits;
  g->per_split = (int)per;
  g->w_bytes = (g->programs - whole) * splits * block * 4;
}

// Time of one round of a tile's workgroups in us, fixed + panels * panel, with at most one
// workgroup a CU and with more.  Fitted to bf16 products over M in 32 .. 4096, N in 256 .. 8192
// and K in 256 .. 8192 (an e4m3 panel holds twice the k and takes the same time).  Checked
// against all tiles with 1 .. 16 slices on 81 shapes (bf16 with b in both orders, odd sizes,
// e4m3): the plan chosen is within 5 % of the fastest at 76 and within 12 % at all.
struct TileCost {
  double panel1, fixed1, panel, fixed;
  int per_cu;   // workgroups that a CU holds
};
constexpr TileCost kTileCosts[lk::kTiles] = {
    {1.32, 12.0, 1.32, 12.0, 1}, {0.71, 4.5, 0.85, 8.0, 2}, {0.215, 3.7, 0.37, 4.8, 2}};
double round_cost(const TileCost& c, int64_t workgroups, int64_t panels) {
  if (workgroups <= 0) return 0.0;
  return workgroups <= kCUs ? c.fixed1 + panels * c.panel1 : c.fixed + panels * c.panel;
}

// The path, tile and split of an M x N x K product (M, N > 0).
int plan_gemm(int64_t type, int64_t M, int64_t N, int64_t K, const Operand& a, const Operand& b,
              GemmPlan* g) {
  const int64_t E = type == LINEAR_NORM_E4M3 ? 2 : 1;
  *g = {};
  g->akm = a.km;
  g->bkm = b.km;
  const int64_t panels = cdiv(K, lk::kTileDepth * E);
  // few rows (and where b is row-major, rows that its loads fit into), in a launch's threads
  if (M <= lk::kSkinnyRows && a.km && (b.km || (N >= 4 && K >= 8)) &&
      cdiv(N, 64) * 512 < kThreads) {
    g->path = b.km ? lk::kPathSkinnyK : lk::kPathSkinnyN;
    const int64_t depth = b.km ? panels : cdiv(K, 32);
    // b k-contiguous: a is read once per workgroup, so with many rows the workgroups take more
    // columns, as long as the CUs have one each, if need be in two slices of k.  In us, with the
    // weights partly in the last-level cache / with other weights in between: e4m3, 16 x 16384 x
    // 4096: 16 columns 19.5 / 22.3, 64 columns 14.1 / 17.7; 16 x 8192 x 8192: 16 columns 18.8 /
    // 21.5, 64 in two slices 16.4 / 20.3 (32 columns in one piece, which this rule does not
    // take, 18.2 / 18.7); one row, bf16, 16384 x 4096: 16 columns 24.1 / 28.1, 64 columns 25.0 /
    // 29.7.
    const int64_t wide = cdiv(N, 64);
    g->cols = 64;
    if (b.km && (M <= 8 || K < 16 || (wide < kCUs && (2 * wide < kCUs || depth < 64))))
      g->cols = M > 8 && K >= 16 && 2 * wide >= kCUs ? 32 : 16;
    if (K >= 8 * E && cdiv(N, g->cols) * 512 >= kThreads) g->cols = 64;
    g->programs = cdiv(N, g->cols);
    // Few columns leave CUs idle: slices of k, of 16 units at least, up to a workgroup a CU.
    // Below 64 units the second launch costs more (4 rows, 512 columns, K = 8192 in bf16: 6.8 us
    // in 8 slices, 13.0 in one; 1024 columns, K = 4096 in e4m3: 6.2 in 4, 5.9 in one).
    int64_t z = 1;
    while (depth >= 64 && z < 16 && g->programs * z * 2 <= kCUs && depth / (z * 2) >= 16) z *= 2;
    set_split(g, 0, depth, z, 16 * g->cols);
    g->cost = 4.0 + (double)(N * K * 2 / E) / 4.5e6 + (g->splits > 1 ? 3.0 : 0.0);
  } else {
    g->path = lk::kPathTiles;
    double best = 0.0;
    GemmPlan chosen = *g;
    for (int t = 0; t < lk::kTiles; ++t) {
      const lk::TileShape& s = lk::kTileShapes[t];
      const TileCost& c = kTileCosts[t];
      // short 8-bit sums are taken as f16, which the largest tile does not do
      if (t == lk::kTile256 && type == LINEAR_NORM_E4M3 && K <= lk::kHalvesK) continue;
      // panels' 32-bit offsets
      const int64_t ra = a.km ? s.bm : lk::kTileDepth, rb = b.km ? s.bn : lk::kTileDepth;
      if (ra * (a.ld / E) >= kMax || rb * (b.ld / E) >= kMax) continue;
      const int64_t P = cdiv(M, s.bm) * cdiv(N, s.bn), slots = (int64_t)kCUs * c.per_cu;
      const int64_t rounds = P / slots, rest = P % slots;
      auto consider = [&](int64_t whole, int64_t splits) {
        // full rounds, then the rest in slices; the second launch and the sums' way through
        // memory (mostly through the caches) for a split
        const int64_t per = cdiv(panels, splits), tail = P - whole;
        if ((whole + tail * splits) * 256 >= kThreads) return;
        double cost = (double)(whole / slots) * round_cost(c, slots, panels);
        cost += round_cost(c, tail * splits, per);
        if (splits > 1) cost += 3.0 + (double)(tail * splits) * s.bm * s.bn * 8 / 8.0e6;
        if (best == 0.0 || cost < best) {
          best = cost;
          chosen.tile = t;
          chosen.programs = P;
          chosen.w_bytes = 0;
          set_split(&chosen, whole, panels, splits, (int64_t)s.bm * s.bn);
        }
      };
      consider(rounds * slots, 1);
      for (int64_t z = 2; z <= 16 && rest > 0 && rest * z <= slots && panels >= 4 * z; ++z)
        consider(rounds * slots, z);
    }
    if (best == 0.0) return GEMM_F16F32_ERR_TOO_LARGE;
    *g = chosen;
    g->cost = best;
  }
  return GEMM_F16F32_OK;
}

// A product in one piece, or cut at the last whole 256 x 256 tile of one axis or both, with the
// slivers left of it as products of their own.
struct Part {
  GemmPlan g;
  int64_t m0, n0, M, N;
};
constexpr int kParts = 3;
struct Product {
  Part part[kParts];
  int parts;       // 0: nothing to compute
  int64_t w_bytes; // workspace, shared by the parts
  double cost;
};
int plan_product(int64_t type, int64_t M, int64_t N, int64_t K, const Operand& a,
                 const Operand& b, Product* p) {
  p->part[0] = {{}, 0, 0, M, N};
  p->parts = 1;
  const int rc = plan_gemm(type, M, N, K, a, b, &p->part[0].g);
  if (rc != GEMM_F16F32_OK) return rc;
  p->cost = p->part[0].g.cost;
  // In one piece a sliver costs a whole row of tiles, or a second round of workgroups; cut off, a
  // launch (about 2.5 us) and what its shape takes (4095 x 4097 x 4093: 145 us in one piece, 135
  // in two; 4097 x 4096 x 4096: 132 and 116).
  const int64_t rm = M > 256 ? M % 256 : 0, rn = N > 256 ? N % 256 : 0;
  for (int cut = 1; cut < 4 && p->part[0].g.path == lk::kPathTiles; ++cut) {
    const int64_t cm = cut & 1 ? rm : 0, cn = cut & 2 ? rn : 0;
    if (((cut & 1) && cm == 0) || ((cut & 2) && cn == 0)) continue;
    Product q = {};
    q.part[q.parts++] = {{}, 0, 0, M - cm, N - cn};
    if (cn > 0) q.part[q.parts++] = {{}, 0, N - cn, M, cn};
    if (cm > 0) q.part[q.parts++] = {{}, M - cm, 0, cm, N - cn};
    bool ok = true;
    q.cost = 2.5 * (q.parts - 1);
    for (int i = 0; ok && i < q.parts; ++i) {
      Part& t = q.part[i];
      ok = plan_gemm(type, t.M, t.N, K, a, b, &t.g) == GEMM_F16F32_OK;
      q.cost += t.g.cost;
    }
    if (ok && q.cost < p->cost) *p = q;
  }
  p->w_bytes = 0;
  for (int i = 0; i < p->parts; ++i)
    if (p->part[i].g.w_bytes > p->w_bytes) p->w_bytes = p->part[i].g.w_bytes;
  return GEMM_F16F32_OK;
}

// The kernel arguments of a product, epilogue left empty.
LinArgs product(int64_t type, int64_t K, const Operand& a, const Operand& b) {
  const int64_t E = type == LINEAR_NORM_E4M3 ? 2 : 1;
  LinArgs p = {};
  p.A = (const uint16_t*)a.p;
  p.B = (const uint16_t*)b.p;
  p.lda = a.ld / E;
  p.ldb = b.ld / E;
  p.K = (int32_t)K;
  p.out_type = (int32_t)type;
  return p;
}

// ... those of one part of it.
LinArgs part_args(const LinArgs& whole, const Part& t, void* ws) {
  const GemmPlan& g = t.g;
  LinArgs p = whole;
  if (p.K > 0) {   // else there are no operands
    p.A += g.akm ? t.m0 * p.lda : t.m0;
    p.B += g.bkm ? t.n0 * p.ldb : t.n0;
  }
  p.out += t.m0 * p.ldo + t.n0;
  if (p.pre) p.pre += t.m0 * p.ldp + t.n0;
  if (p.res) p.res += t.m0 * p.ldr + t.n0;
  if (p.bias) p.bias += t.n0;
  if (p.scale_a) p.scale_a += t.m0;
  if (p.scale_b) p.scale_b += t.n0;
  p.M = (int32_t)t.M;
  p.N = (int32_t)t.N;
  const bool tiles = g.path == lk::kPathTiles;
  p.num_pid_m = (int32_t)(tiles ? cdiv(t.M, lk::kTileShapes[g.tile].bm) : 1);
  p.num_pid_n = (int32_t)(g.programs / p.num_pid_m);
  const int group = tiles && g.tile == lk::kTile256 ? 8 : 4;
  p.group_m = p.num_pid_m < group ? p.num_pid_m : group;
  // Tiles that share operands go to one XCD's cache; with one row of tiles they share none of
  // b, and neighbours on different XCDs read it faster (1 x 16384 x 4096: 26.3 against 31.9 us).
  p.xcd_remap = p.num_pid_m > 1;
  p.num_programs = (int32_t)g.programs;
  p.W = (float*)ws;
  p.first_split = (int32_t)g.whole;
  p.splits = g.splits;
  p.per_split = g.per_split;
  return p;
}

int launch(int64_t type, const Product& q, const LinArgs& whole, void* ws, void* stream) {
  const hipStream_t s = (hipStream_t)stream;
  for (int i = 0; i < q.parts; ++i) {
    const LinArgs p = part_args(whole, q.part[i], ws);
    const GemmPlan& g = q.part[i].g;
    const hipError_t e = type == LINEAR_NORM_F16    ? lk::launch_type<lk::kF16>(g, p, s)
                         : type == LINEAR_NORM_BF16 ? lk::launch_type<lk::kBF16>(g, p, s)
                                                    : lk::launch_type<lk::kE4M3>(g, p, s);
    if (e != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  return GEMM_F16F32_OK;
}

int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return GEMM_F16F32_OK;
  return ws == nullptr || have < need || ((uintptr_t)ws & 15) ? GEMM_F16F32_ERR_WORKSPACE
                                                              : GEMM_F16F32_OK;
}

// Partial column sums of `groups` workgroups, in whole blocks of 32 columns.
int64_t partial_bytes(int64_t groups, int64_t cols) { return groups * round_up(cols, 32) * 4; }

bool bad_dim(int64_t d) { return d < 0 || d >= kMax; }

// ---- linear_forward ----------------------------------------------------------------------------
struct ForwardPlan {
  Operand a, b;
  Product q;   // no parts: an empty result
};
int plan_forward(linear_forward_args& x, ForwardPlan* f) {
  *f = {};
  if (bad_dim(x.m) || bad_dim(x.n) || bad_dim(x.k)) return GEMM_F16F32_ERR_DIM;
  if (!is16(x.type) && x.type != LINEAR_NORM_E4M3) return GEMM_F16F32_ERR_OPTS;
  if (!is16(x.out_type) || (is16(x.type) && x.out_type != x.type)) return GEMM_F16F32_ERR_OPTS;
  if (x.activation < LINEAR_ACT_NONE || x.activation > LINEAR_ACT_SILU)
    return GEMM_F16F32_ERR_OPTS;
  if (is16(x.type) && (x.scale_a || x.scale_b)) return GEMM_F16F32_ERR_OPTS;
  if (x.m == 0 || x.n == 0) return GEMM_F16F32_OK;
  int rc = operand(x.a, x.m, x.k, x.a_row, x.a_col, x.type, &f->a);
  if (rc == 0) rc = operand(x.b, x.n, x.k, x.b_col, x.b_row, x.type, &f->b);
  if (rc == 0) rc = check_rows(x.out, x.m, x.n, &x.out_row, 2, true);
  if (rc == 0) rc = check_rows(x.pre, x.m, x.n, &x.pre_row, 2, false);
  if (rc == 0) rc = check_rows(x.residual, x.m, x.n, &x.residual_row, 2, false);
  if (rc != 0) return rc;
  if (((uintptr_t)x.bias & 1) || (((uintptr_t)x.scale_a | (uintptr_t)x.scale_b) & 3))
    return GEMM_F16F32_ERR_OPTS;
  const Region w[] = {region(x.out, x.m, x.n, x.out_row, 2), region(x.pre, x.m, x.n, x.pre_row, 2)};
  const Region r[] = {operand_region(f->a, x.m, x.k, x.type), operand_region(f->b, x.n, x.k, x.type),
                      region(x.bias, 1, x.n, x.n, 2), region(x.scale_a, 1, x.m, x.m, 4),
                      region(x.scale_b, 1, x.n, x.n, 4)};
  if (conflict(w, 2, r, 5)) return GEMM_F16F32_ERR_OVERLAP;
  const Region res = region(x.residual, x.m, x.n, x.residual_row, 2);
  const bool in_place = x.residual == x.out && x.residual_row == x.out_row;
  if (overlap(w[1], res) || (!in_place && overlap(w[0], res))) return GEMM_F16F32_ERR_OVERLAP;
  return plan_product(x.type, x.m, x.n, x.k, f->a, f->b, &f->q);
}

// ---- linear_backward ----------------------------------------------------------------------------
struct BackwardPlan {
  bool dact;                 // the element-wise pass runs
  bool pair;                 // the products and dbias's last step go in one launch
  bool small;                // ... and the element-wise pass as well
  Operand b, a, dt;          // b as da's right operand; a and dpre as db's
  bool db_cols;              // db is column-major: the product is its transpose
  Product qa, qb;            // da's and db's products
  int64_t ldd;               // dpre's row stride
  int row_blocks, rows_per_block;
  int64_t dpre_bytes, part_bytes, w_bytes;
};
int plan_backward(linear_backward_args& x, BackwardPlan* f) {
  *f = {};
  if (bad_dim(x.m) || bad_dim(x.n) || bad_dim(x.k)) return GEMM_F16F32_ERR_DIM;
  if (!is16(x.type)) return GEMM_F16F32_ERR_OPTS;
  if (x.activation < LINEAR_ACT_NONE || x.activation > LINEAR_ACT_SILU)
    return GEMM_F16F32_ERR_OPTS;
  const bool act = x.activation != LINEAR_ACT_NONE;
  int rc = check_rows(x.dc, x.m, x.n, &x.dc_row, 2, true);
  if (rc == 0 && act) rc = check_rows(x.pre, x.m, x.n, &x.pre_row, 2, true);
  if (rc == 0) rc = check_rows(x.da, x.m, x.k, &x.da_row, 2, false);
  if (rc != 0) return rc;
  if ((uintptr_t)x.dbias & 1) return GEMM_F16F32_ERR_OPTS;
  Region ra = {}, rb = {}, rdb = {};
  if (x.da && x.m > 0 && x.k > 0) {
    rc = operand(x.b, x.k, x.n, x.b_row, x.b_col, x.type, &f->b);
    if (rc != 0) return rc;
    rb = operand_region(f->b, x.k, x.n, x.type);
  }
  if (x.db && x.k > 0 && x.n > 0) {
    rc = operand(x.a, x.k, x.m, x.a_col, x.a_row, x.type, &f->a);
    if (rc != 0) return rc;
    ra = operand_region(f->a, x.k, x.m, x.type);
    // db's order: a unit stride along n, or along k
    if ((x.db_col == 1 || x.n == 1) && (x.k == 1 || x.db_row >= x.n)) {
      rc = check_rows(x.db, x.k, x.n, &x.db_row, 2, true);
      rdb = region(x.db, x.k, x.n, x.db_row, 2);
    } else if (x.db_row == 1 || x.k == 1) {
      f->db_cols = true;
      rc = check_rows(x.db, x.n, x.k, &x.db_col, 2, true);
      rdb = region(x.db, x.n, x.k, x.db_col, 2);
    } else {
      rc = GEMM_F16F32_ERR_LD;
    }
    if (rc != 0) return rc;
  }
  const Region w[] = {region(x.da, x.m, x.k, x.da_row, 2), rdb, region(x.dbias, 1, x.n, x.n, 2)};
  const Region r[] = {region(x.dc, x.m, x.n, x.dc_row, 2), ra, rb,
                      region(act ? x.pre : nullptr, x.m, x.n, x.pre_row, 2)};
  if (conflict(w, 3, r, 4)) return GEMM_F16F32_ERR_OVERLAP;

  // the element-wise pass: dpre (rows on 128-byte lines), and blocks of rows for its column sums
  f->dact = x.n > 0 && ((act && x.m > 0) || x.dbias);
  if (f->dact && act) {
    f->ldd = round_up(x.n, 64);
    f->dpre_bytes = round_up(x.m * f->ldd * 2, 256);
  }
  if (f->dact) {
    const int64_t cols = cdiv(x.n, 512);
    // a row a thread, up to 4 workgroups a CU (512^3 f16 with silu: 9.0 us in all; 4 rows: 10.7)
    int64_t blocks = cdiv(x.m, 4);
    const int64_t most = cdiv(4 * kCUs, cols);
    if (blocks > most) blocks = most;
    if (blocks < cdiv(x.m, 1 << 30)) blocks = cdiv(x.m, 1 << 30);   // the kernel's row counter
    if (blocks < 1) blocks = 1;
    f->rows_per_block = (int)round_up(cdiv(x.m, blocks), 4);
    f->row_blocks = x.m > 0 ? (int)cdiv(x.m, f->rows_per_block) : 0;
    if (x.dbias && f->row_blocks != 1) {
      f->part_bytes = round_up(partial_bytes(f->row_blocks, x.n), 256);
    }
  }
  const int64_t ldd = act ? f->ldd : x.dc_row;
  if (x.da && x.m > 0 && x.k > 0) {
    const Operand d = {x.dc, ldd, true};
    rc = plan_product(x.type, x.m, x.k, x.n, d, f->b, &f->qa);
    if (rc != 0) return rc;
    if (f->qa.w_bytes > f->w_bytes) f->w_bytes = f->qa.w_bytes;
  }
  if (x.db && x.k > 0 && x.n > 0) {
    f->dt = {x.dc, ldd, false};
    rc = f->db_cols ? plan_product(x.type, x.n, x.k, x.m, f->dt, f->a, &f->qb)
                    : plan_product(x.type, x.k, x.n, x.m, f->a, f->dt, &f->qb);
    if (rc != 0) return rc;
    if (f->qb.w_bytes > f->w_bytes) f->w_bytes = f->qb.w_bytes;
  }
  // One launch for both products, unsplit, where its estimated time is below theirs and that of
  // the launches saved (about 2 us each).
  if (f->qa.parts > 0 && f->qb.parts > 0 && !f->a.km) {
    const int64_t pa = cdiv(x.m, 64) * cdiv(x.k, 64), pb = cdiv(x.n, 64) * cdiv(x.k, 64);
    const int64_t deep = cdiv(x.m > x.n ? x.m : x.n, lk::kTileDepth);
    const int64_t most = 64, lb = f->b.ld > ldd ? f->b.ld : ldd;
    const bool fits = most * lb < kMax && most * f->a.ld < kMax;
    // as long as its deepest tile, or as all its tiles' work takes
    const TileCost& c = kTileCosts[lk::kTile64];
    const int64_t slots = (int64_t)kCUs * c.per_cu, P = pa + pb;
    const double work = pa * (double)cdiv(x.n, 64) + pb * (double)cdiv(x.m, 64);
    double one = round_cost(c, P < kCUs ? P : kCUs, deep);
    const double all = (c.fixed * P + c.panel * work) / slots;
    if (all > one) one = all;
    const double two = f->qa.cost + f->qb.cost + 2.0 + (f->part_bytes > 0 ? 2.0 : 0.0);
    f->pair = fits && P <= 4 * kCUs && one < two;
    // The element-wise pass as well while a tile's panels are few: its loads go through
    // registers, three panels ahead, and a panel costs about 1.2 us instead of 0.3, for a launch
    // less (f16, silu: 64^3 4.6 us against 8.2 in two launches, 128^3 5.8 and 7.6, 256^3 8.1 and
    // 7.5, 4 x 200 x 300 8.9 and 7.9, 64 x 256 x 3000 8.2 and 7.9, 300^3, past the rule, 11.8 and
    // 9.6).  At four panels only the launch's 3 us of host time speak for it, which a captured
    // graph does not pay.
    f->small = f->pair && deep <= 4 && x.n >= 8 && x.k >= 8;
    if (f->pair) {
      GemmPlan t = {};
      t.path = lk::kPathTiles;
      t.tile = lk::kTile64;
      t.akm = true;
      t.bkm = f->b.km;
      t.programs = t.whole = pa;
      t.splits = 1;
      f->qa.part[0] = {t, 0, 0, x.m, x.k};
      t.akm = t.bkm = false;
      t.programs = t.whole = pb;
      f->qb.part[0] = {t, 0, 0, f->db_cols ? x.n : x.k, f->db_cols ? x.k : x.n};
      f->w_bytes = 0;
      if (f->small) {
        f->dact = false;
        f->dpre_bytes = f->part_bytes = 0;
      }
    }
  }
  return GEMM_F16F32_OK;
}

// ---- norm ----------------------------------------------------------------------------------------
constexpr int64_t kRowsPerLaunch = 1 << 21;   // 2^21 rows of up to 1024 threads

int check_norm(int64_t rows, int64_t dim, int64_t type) {
  if (bad_dim(rows) || dim < 1 || dim >= kMax) return GEMM_F16F32_ERR_DIM;
  return is16(type) ? GEMM_F16F32_OK : GEMM_F16F32_ERR_OPTS;
}

// Waves a row and steps of 512 columns a wave that hold a row of `dim` in registers; C = 0 (long
// rows): none.
template <class F>
void with_row_shape(int64_t dim, F f) {
  if (dim <= 512) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  else if (dim <= 1024) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{});
  else if (dim <= 2048) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
  else if (dim <= 4096) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  else if (dim <= 8192) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
  else if (dim <= 16384) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 16>{}, std::integral_constant<int, 0>{});
}

template <int TY, bool Q8>
void norm_forward(const nk::NormArgs& p, hipStream_t s) {
  with_row_shape(p.dim, [&](auto nw, auto c) {
    hipLaunchKernelGGL((nk::rms_norm_fwd<TY, Q8, nw.value, c.value>), dim3((uint32_t)p.rows),
                       dim3(64 * nw.value), 0, s, p);
  });
}
// The backward pass: as above, but short rows take one wave, four of them a workgroup, and rows
// above 8192 fewer waves of more registers.
constexpr int64_t kShortRow = 1024, kLongRow = 16384;
template <int TY>
void norm_backward(const nk::NormBwdArgs& p, int grid, hipStream_t s) {
#define LN_BACKWARD(NW, C, RW)                                                               \
  hipLaunchKernelGGL((nk::rms_norm_bwd<TY, NW, C, RW>), dim3((uint32_t)grid), dim3(64 * NW * RW), \
                     0, s, p)
  if (p.dim <= 512) LN_BACKWARD(1, 1, 4);
  else if (p.dim <= kShortRow) LN_BACKWARD(1, 2, 4);
  else if (p.dim <= 2048) LN_BACKWARD(4, 1, 1);
  else if (p.dim <= 4096) LN_BACKWARD(4, 2, 1);
  else if (p.dim <= 8192) LN_BACKWARD(8, 2, 1);
  else if (p.dim <= kLongRow) LN_BACKWARD(8, 4, 1);
  else
    hipLaunchKernelGGL((nk::rms_norm_bwd_long<TY, 16>), dim3((uint32_t)grid), dim3(1024), 0, s, p);
#undef LN_BACKWARD
}

// Workgroups of the norm's backward pass, each with partial dweight sums: two a CU keep enough
// loads in flight (8192 x 4096: 45.5 us; four a CU 52.7, their sums being written and read).
// Few rows, 2 for each that a workgroup works on at once, take one workgroup, which writes dweight
// itself: a launch less (1 x 4096: 3.6 us against 5.8, and 3 us of host time; with 8 for each the
// kernel took longer than the launch, 8 x 4096 11.8 us against 6.0).
int backward_groups(int64_t rows, int64_t dim) {
  const int64_t at_once = dim <= kShortRow ? 4 : 1;
  if (dim <= kLongRow && rows <= 2 * at_once) return rows > 0;
  const int64_t n = cdiv(rows, at_once);
  return (int)(n < 2 * kCUs ? n : 2 * kCUs);
}
// Whether dweight needs a second step.
bool backward_sums(int64_t rows, int64_t dim) {
  return dim > kLongRow || backward_groups(rows, dim) != 1;
}

int64_t norm_backward_bytes(const rms_norm_backward_args& x) {
  return x.dweight && backward_sums(x.rows, x.dim)
             ? partial_bytes(backward_groups(x.rows, x.dim), x.dim)
             : 0;
}

template <int TY>
void launch_sum(const float* part, int n, int64_t cols, void* out, hipStream_t s) {
  const int64_t blocks = cdiv(cols, 32), most = kThreads / 256 - 1;
  for (int64_t first = 0; first < blocks; first += most) {
    const int64_t grid = blocks - first < most ? blocks - first : most;
    hipLaunchKernelGGL((nk::sum_partials<TY>), dim3((uint32_t)grid), dim3(256), 0, s, part, n,
                       (int)first, (int)cols, (uint16_t*)out);
  }
}

}  // namespace

extern "C" {

int64_t linear_forward_workspace(const linear_forward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_forward_args x = *args;
  ForwardPlan f;
  const int rc = plan_forward(x, &f);
  return rc != GEMM_F16F32_OK ? rc : f.q.w_bytes;
}

int linear_forward(const linear_forward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_forward_args x = *args;
  ForwardPlan f;
  int rc = plan_forward(x, &f);
  if (rc != GEMM_F16F32_OK || f.q.parts == 0) return rc;
  rc = check_workspace(x.workspace, x.workspace_bytes, f.q.w_bytes);
  if (rc != GEMM_F16F32_OK) return rc;
  if (f.q.w_bytes > 0) {
    const Region w = {x.workspace, (uint64_t)f.q.w_bytes};
    const Region o[] = {region(x.out, x.m, x.n, x.out_row, 2), region(x.pre, x.m, x.n, x.pre_row, 2),
                        region(x.residual, x.m, x.n, x.residual_row, 2),
                        operand_region(f.a, x.m, x.k, x.type), operand_region(f.b, x.n, x.k, x.type),
                        region(x.bias, 1, x.n, x.n, 2), region(x.scale_a, 1, x.m, x.m, 4),
                        region(x.scale_b, 1, x.n, x.n, 4)};
    if (conflict(&w, 1, o, 8)) return GEMM_F16F32_ERR_OVERLAP;
  }
  LinArgs p = product(x.type, x.k, f.a, f.b);
  p.out = (uint16_t*)x.out;
  p.ldo = x.out_row;
  p.pre = (uint16_t*)x.pre;
  p.ldp = x.pre_row;
  p.res = (const uint16_t*)x.residual;
  p.ldr = x.residual_row;
  p.bias = (const uint16_t*)x.bias;
  p.scale_a = x.scale_a;
  p.scale_b = x.scale_b;
  p.act = (int32_t)x.activation;
  p.out_type = (int32_t)x.out_type;
  return launch(x.type, f.q, p, x.workspace, x.stream);
}

int64_t linear_backward_workspace(const linear_backward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_backward_args x = *args;
  BackwardPlan f;
  const int rc = plan_backward(x, &f);
  return rc != GEMM_F16F32_OK ? rc : f.dpre_bytes + f.part_bytes + f.w_bytes;
}

int linear_backward(const linear_backward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_backward_args x = *args;
  BackwardPlan f;
  int rc = plan_backward(x, &f);
  if (rc != GEMM_F16F32_OK) return rc;
  const bool act = x.activation != LINEAR_ACT_NONE;
  const int64_t need = f.dpre_bytes + f.part_bytes + f.w_bytes;
  rc = check_workspace(x.workspace, x.workspace_bytes, need);
  if (rc != GEMM_F16F32_OK) return rc;
  if (need > 0) {
    const Region w = {x.workspace, (uint64_t)need};
    const Region o[] = {region(x.dc, x.m, x.n, x.dc_row, 2),
                        region(act ? x.pre : nullptr, x.m, x.n, x.pre_row, 2),
                        region(x.da, x.m, x.k, x.da_row, 2), region(x.dbias, 1, x.n, x.n, 2),
                        operand_region(f.a, x.k, x.m, x.type), operand_region(f.b, x.k, x.n, x.type),
                        f.db_cols ? region(x.db, x.n, x.k, x.db_col, 2)
                                  : region(x.db, x.k, x.n, x.db_row, 2)};
    if (conflict(&w, 1, o, 7)) return GEMM_F16F32_ERR_OVERLAP;
  }
  const bool bf = x.type == LINEAR_NORM_BF16;
  const hipStream_t s = (hipStream_t)x.stream;
  char* const ws = (char*)x.workspace;
  const void* dpre = x.dc;
  const bool sums = x.dbias != nullptr && f.dact;
  const bool last = sums && f.row_blocks != 1;   // dbias has a second step
  float* const part = last ? (float*)(ws + f.dpre_bytes) : nullptr;
  if (f.dact && f.row_blocks > 0) {
    nk::DactArgs d = {};
    d.dc = (const uint16_t*)x.dc;
    d.dc_row = x.dc_row;
    if (act) {
      d.pre = (const uint16_t*)x.pre;
      d.pre_row = x.pre_row;
      d.dpre = (uint16_t*)ws;
      d.dpre_row = f.ldd;
      dpre = ws;
    }
    d.part = part;
    d.sum = sums && !last ? (uint16_t*)x.dbias : nullptr;
    d.m = (int32_t)x.m;
    d.n = (int32_t)x.n;
    d.act = (int32_t)x.activation;
    d.row_blocks = f.row_blocks;
    d.rows_per_block = f.rows_per_block;
    const dim3 grid((uint32_t)(cdiv(x.n, 512) * f.row_blocks));
    if (bf)
      hipLaunchKernelGGL((nk::lin_dact<lk::kBF16>), grid, dim3(256), 0, s, d);
    else
      hipLaunchKernelGGL((nk::lin_dact<lk::kF16>), grid, dim3(256), 0, s, d);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  if (last && !f.pair) {
    if (bf)
      launch_sum<lk::kBF16>(part, f.row_blocks, x.n, x.dbias, s);
    else
      launch_sum<lk::kF16>(part, f.row_blocks, x.n, x.dbias, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  void* const W = ws ? ws + f.dpre_bytes + f.part_bytes : nullptr;
  LinArgs da = {}, db = {};
  const int64_t ldd = act && !f.small ? f.ldd : x.dc_row;
  if (f.qa.parts > 0) {
    da = product(x.type, x.n, {dpre, ldd, true}, f.b);
    da.out = (uint16_t*)x.da;
    da.ldo = x.da_row;
  }
  if (f.qb.parts > 0) {
    const Operand d = {dpre, ldd, false};
    db = f.db_cols ? product(x.type, x.m, d, f.a) : product(x.type, x.m, f.a, d);
    db.out = (uint16_t*)x.db;
    db.ldo = f.db_cols ? x.db_col : x.db_row;
  }
  if (f.small) {
    const lk::SmallArgs p = {part_args(da, f.qa.part[0], nullptr),
                             part_args(db, f.qb.part[0], nullptr),
                             (const uint16_t*)(act ? x.pre : x.dc), act ? x.pre_row : x.dc_row,
                             (uint16_t*)x.dbias, (int32_t)x.activation};
    const hipError_t e = bf ? lk::launch_small<lk::kBF16>(p, f.b.km, f.db_cols, s)
                            : lk::launch_small<lk::kF16>(p, f.b.km, f.db_cols, s);
    return e == hipSuccess ? GEMM_F16F32_OK : GEMM_F16F32_ERR_HIP;
  }
  if (f.pair) {
    const lk::PairArgs p = {part_args(da, f.qa.part[0], W), part_args(db, f.qb.part[0], W), part,
                            last ? (uint16_t*)x.dbias : nullptr, f.row_blocks, (int32_t)x.n};
    const hipError_t e = bf ? lk::launch_pair<lk::kBF16>(p, f.b.km, s)
                            : lk::launch_pair<lk::kF16>(p, f.b.km, s);
    return e == hipSuccess ? GEMM_F16F32_OK : GEMM_F16F32_ERR_HIP;
  }
  if (f.qa.parts > 0) rc = launch(x.type, f.qa, da, W, x.stream);
  if (rc == GEMM_F16F32_OK && f.qb.parts > 0) rc = launch(x.type, f.qb, db, W, x.stream);
  return rc;
}

int rms_norm_forward(const rms_norm_forward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  rms_norm_forward_args x = *args;
  int rc = check_norm(x.rows, x.dim, x.type);
  if (rc != GEMM_F16F32_OK) return rc;
  const bool q8 = x.out_type == LINEAR_NORM_E4M3;
  if ((!q8 && x.out_type != x.type) || !(x.eps >= 0.0) || (x.scale && !q8))
    return GEMM_F16F32_ERR_OPTS;
  if (x.rows == 0) return GEMM_F16F32_OK;
  rc = check_rows(x.x, x.rows, x.dim, &x.x_row, 2, true);
  if (rc == 0) rc = check_rows(x.residual, x.rows, x.dim, &x.residual_row, 2, false);
  if (rc == 0) rc = check_rows(x.y, x.rows, x.dim, &x.y_row, q8 ? 1 : 2, true);
  if (rc == 0) rc = check_rows(x.h, x.rows, x.dim, &x.h_row, 2, x.residual != nullptr);
  if (rc != 0) return rc;
  if (x.weight == nullptr || (q8 && x.scale == nullptr)) return GEMM_F16F32_ERR_NULL;
  if (((uintptr_t)x.weight & 1) || (((uintptr_t)x.scale | (uintptr_t)x.rstd) & 3))
    return GEMM_F16F32_ERR_OPTS;
  const Region rx = region(x.x, x.rows, x.dim, x.x_row, 2);
  const Region rr = region(x.residual, x.rows, x.dim, x.residual_row, 2);
  const Region rh = region(x.h, x.rows, x.dim, x.h_row, 2);
  const Region w[] = {region(x.y, x.rows, x.dim, x.y_row, q8 ? 1 : 2),
                      region(x.scale, 1, x.rows, x.rows, 4), region(x.rstd, 1, x.rows, x.rows, 4),
                      rh};
  const Region r[] = {rx, rr, region(x.weight, 1, x.dim, x.dim, 2)};
  if (conflict(w, 3, r, 3) || conflict(w, 4, r + 2, 1)) return GEMM_F16F32_ERR_OVERLAP;
  if ((!(x.h == x.x && x.h_row == x.x_row) && overlap(rh, rx)) ||
      (!(x.h == x.residual && x.h_row == x.residual_row) && overlap(rh, rr)))
    return GEMM_F16F32_ERR_OVERLAP;
  const int64_t ys = q8 ? 1 : 2;
  for (int64_t r0 = 0; r0 < x.rows; r0 += kRowsPerLaunch) {
    nk::NormArgs p = {};
    p.x = (const uint16_t*)x.x + r0 * x.x_row;
    p.x_row = x.x_row;
    if (x.residual) p.res = (const uint16_t*)x.residual + r0 * x.residual_row;
    p.res_row = x.residual_row;
    p.weight = (const uint16_t*)x.weight;
    p.y = (char*)x.y + ys * r0 * x.y_row;
    p.y_row = x.y_row;
    if (x.scale) p.scale = x.scale + r0;
    if (x.h) p.h = (uint16_t*)x.h + r0 * x.h_row;
    p.h_row = x.h_row;
    if (x.rstd) p.rstd = x.rstd + r0;
    p.rows = (int32_t)(x.rows - r0 < kRowsPerLaunch ? x.rows - r0 : kRowsPerLaunch);
    p.dim = (int32_t)x.dim;
    p.eps = (float)x.eps;
    p.inv_dim = (float)(1.0 / (double)x.dim);
    const hipStream_t s = (hipStream_t)x.stream;
    if (x.type == LINEAR_NORM_BF16)
      q8 ? norm_forward<lk::kBF16, true>(p, s) : norm_forward<lk::kBF16, false>(p, s);
    else
      q8 ? norm_forward<lk::kF16, true>(p, s) : norm_forward<lk::kF16, false>(p, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  return GEMM_F16F32_OK;
}

int64_t rms_norm_backward_workspace(const rms_norm_backward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  const int rc = check_norm(args->rows, args->dim, args->type);
  return rc != GEMM_F16F32_OK ? rc : norm_backward_bytes(*args);
}

int rms_norm_backward(const rms_norm_backward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  rms_norm_backward_args x = *args;
  int rc = check_norm(x.rows, x.dim, x.type);
  if (rc == 0) rc = check_rows(x.dy, x.rows, x.dim, &x.dy_row, 2, true);
  if (rc == 0) rc = check_rows(x.h, x.rows, x.dim, &x.h_row, 2, true);
  if (rc == 0) rc = check_rows(x.dh, x.rows, x.dim, &x.dh_row, 2, false);
  if (rc == 0) rc = check_rows(x.dx, x.rows, x.dim, &x.dx_row, 2, true);
  if (rc != 0) return rc;
  if (x.rows > 0 && (x.weight == nullptr || x.rstd == nullptr)) return GEMM_F16F32_ERR_NULL;
  if ((((uintptr_t)x.weight | (uintptr_t)x.dweight) & 1) || ((uintptr_t)x.rstd & 3))
    return GEMM_F16F32_ERR_OPTS;
  const int64_t need = norm_backward_bytes(x);
  rc = check_workspace(x.workspace, x.workspace_bytes, need);
  if (rc != GEMM_F16F32_OK) return rc;
  const Region rdx = region(x.dx, x.rows, x.dim, x.dx_row, 2);
  const Region rdy = region(x.dy, x.rows, x.dim, x.dy_row, 2);
  const Region rdh = region(x.dh, x.rows, x.dim, x.dh_row, 2);
  const Region w[] = {region(x.dweight, 1, x.dim, x.dim, 2), {x.workspace, (uint64_t)need}, rdx};
  const Region r[] = {region(x.h, x.rows, x.dim, x.h_row, 2),
                      region(x.weight, 1, x.dim, x.dim, 2), region(x.rstd, 1, x.rows, x.rows, 4),
                      rdy, rdh};
  if (conflict(w, 2, r, 5) || conflict(w, 3, r, 3)) return GEMM_F16F32_ERR_OVERLAP;
  if ((!(x.dx == x.dy && x.dx_row == x.dy_row) && overlap(rdx, rdy)) ||
      (!(x.dx == x.dh && x.dx_row == x.dh_row) && overlap(rdx, rdh)))
    return GEMM_F16F32_ERR_OVERLAP;
  const hipStream_t s = (hipStream_t)x.stream;
  const bool bf = x.type == LINEAR_NORM_BF16;
  const int groups = backward_groups(x.rows, x.dim);
  if (groups > 0) {
    nk::NormBwdArgs p = {};
    p.dy = (const uint16_t*)x.dy;
    p.dy_row = x.dy_row;
    p.h = (const uint16_t*)x.h;
    p.h_row = x.h_row;
    p.weight = (const uint16_t*)x.weight;
    p.rstd = x.rstd;
    p.dh = (const uint16_t*)x.dh;
    p.dh_row = x.dh_row;
    p.dx = (uint16_t*)x.dx;
    p.dx_row = x.dx_row;
    const bool sums = backward_sums(x.rows, x.dim);
    p.part = x.dweight && sums ? (float*)x.workspace : nullptr;
    p.dweight = sums ? nullptr : (uint16_t*)x.dweight;
    p.rows = (int32_t)x.rows;
    p.dim = (int32_t)x.dim;
    p.inv_dim = (float)(1.0 / (double)x.dim);
    bf ? norm_backward<lk::kBF16>(p, groups, s) : norm_backward<lk::kF16>(p, groups, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  if (x.dweight && backward_sums(x.rows, x.dim)) {
    bf ? launch_sum<lk::kBF16>((const float*)x.workspace, groups, x.dim, x.dweight, s)
       : launch_sum<lk::kF16>((const float*)x.workspace, groups, x.dim, x.dweight, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  return GEMM_F16F32_OK;
}

}  // extern "C"
