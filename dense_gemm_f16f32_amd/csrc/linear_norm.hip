// C-ABI of the linear layer, the norms and rows in 8 bits: argument checks, kernel choice,
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
bool is8(int64_t type) { return type == LINEAR_NORM_E4M3 || type == LINEAR_NORM_I8; }

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
  const int64_t elem = is8(type) ? 1 : 2;
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
  const int64_t e = is8(type) ? 1 : 2;
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

// The tile and split of an M x N x K product that are estimated to be the fastest, in at most `slices`
// of k; returns the estimate, or 0 if no tile's panels fit.
double plan_tiles(int64_t type, int64_t M, int64_t N, int64_t K, const Operand& a, const Operand& b,
                  int64_t slices, GemmPlan* g) {
  const int64_t E = is8(type) ? 2 : 1, panels = cdiv(K, lk::kTileDepth * E);
  double best = 0.0;
  GemmPlan chosen = *g;
  chosen.path = lk::kPathTiles;
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
    for (int64_t z = 2; z <= slices && rest > 0 && rest * z <= slots && panels >= 4 * z; ++z)
      consider(rounds * slots, z);
  }
  *g = chosen;
  return best;
}

// A result of at most 16 columns as a pass over a (E: operands' values in a 16-bit slot): whether the
// kernel takes it, and its estimated time.  `odd_a`, `odd_b`: rows off 4-byte boundaries, whose loads
// take longer than their multiplication and than memory (bf16, a's rows / b's / both at odd addresses:
// 64 x 8 x 4096 17.1 / 14.0 / 22.7 us, all even 8.7; 16384 x 1 x 4096 55, even 24).
bool narrow_fits(int64_t E, int64_t M, int64_t N, int64_t K, const Operand& a, const Operand& b) {
  return N <= lk::kSkinnyRows && a.km && b.km && K >= 8 * E && cdiv(M, 16) * 512 < kThreads;
}
double narrow_cost(int64_t E, int64_t M, int64_t N, int64_t K, bool odd_a, bool odd_b) {
  const double mbytes = (double)M * (double)(K * 2 / E) * 1e-6;
  const double deep = (double)K / E * (0.95e-3 + 0.05e-3 * N + (odd_a ? 2.1e-3 : 0.0) +
                                       (odd_b ? 0.15e-3 * N : 0.0));
  const double wide = mbytes * (0.14 + 0.005 * N + (odd_a ? 0.23 : 0.0) + (odd_b ? 0.0145 * N : 0.0));
  return 2.2 + (deep > wide ? deep : wide) + 1.9e-3 * cdiv(M, 16);
}

// The path, tile and split of an M x N x K product (M, N > 0).  `blocks`: the epilogue packs blocks
// of 32 columns, which one workgroup has to hold.
int plan_gemm(int64_t type, int64_t M, int64_t N, int64_t K, const Operand& a, const Operand& b,
              bool blocks, GemmPlan* g) {
  const int64_t E = is8(type) ? 2 : 1;
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
    if (blocks && g->cols == 16) g->cols = 32;
    g->programs = cdiv(N, g->cols);
    // Few columns leave CUs idle: slices of k, of 16 units at least, up to a workgroup a CU.
    // Below 64 units the second launch costs more (4 rows, 512 columns, K = 8192 in bf16: 6.8 us
    // in 8 slices, 13.0 in one; 1024 columns, K = 4096 in e4m3: 6.2 in 4, 5.9 in one).
    int64_t z = 1;
    while (depth >= 64 && z < 16 && g->programs * z * 2 <= kCUs && depth / (z * 2) >= 16) z *= 2;
    set_split(g, 0, depth, z, 16 * g->cols);
    g->cost = 4.0 + (double)(N * K * 2 / E) / 4.5e6 + (g->splits > 1 ? 3.0 : 0.0);
  } else {
    g->cost = plan_tiles(type, M, N, K, a, b, 16, g);
    // At most 16 columns: a pass over a, 16 of its rows a workgroup, in one piece of k, where the
    // estimates say that it is faster than the tiles (whose own leaves out memory's rate: a tile is
    // mostly empty here, and deep or many rows are a pass over a as well).  Few rows of a deep k stay
    // with the tiles and their slices.  In us from memory in a graph, on tiles / so, m x n x k: bf16
    // 64 x 16 x 1024 7.2 / 4.4, 4096 x 1 x 4096 13.8 / 10.5, 16384 x 1 x 16384 121 / 111; int8 256 x 16
    // x 4096 8.2 / 6.8, 4096 x 8 x 16384 22 / 17; and left to the tiles bf16 64 x 16 x 4096 8.9 / 9.9,
    // 32 x 16 x 16384 11.2 / 31, 17 x 1 x 65536 22 / 71, 16384 x 16 x 4096 32 / 39; int8 64 x 8 x 16384
    // 9.5 / 14, 65536 x 16 x 256 10 / 15.  On 772 shapes (3 types, m 17 .. 65536, n 1 .. 16, k 64 ..
    // 65536) the choice takes at most 4 % longer than the tiles (where a is partly in the last-level
    // cache up to 19 %), at most 20 % longer than the faster of the two, and 22 % less in the mean.
    if (narrow_fits(E, M, N, K, a, b)) {
      const bool odd_a = E == 1 && a.ld % 2 != 0, odd_b = E == 1 && N > 1 && b.ld % 2 != 0;
      const double narrow = narrow_cost(E, M, N, K, odd_a, odd_b);
      const double memory = 2.0 + (double)M * (double)(K * 2 / E) / 5.6e6;
      const double tiles = g->cost + 0.8 > memory ? g->cost + 0.8 : memory;
      if (g->cost == 0.0 || narrow < tiles) {
        g->path = lk::kPathSkinnyFlip;
        g->cols = 16;
        g->programs = cdiv(M, 16);
        g->w_bytes = 0;
        set_split(g, 0, panels, 1, 0);
        g->cost = narrow;
      }
    }
    if (g->cost == 0.0) return GEMM_F16F32_ERR_TOO_LARGE;
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
                 const Operand& b, bool blocks, Product* p) {
  p->part[0] = {{}, 0, 0, M, N};
  p->parts = 1;
  const int rc = plan_gemm(type, M, N, K, a, b, blocks, &p->part[0].g);
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
      ok = plan_gemm(type, t.M, t.N, K, a, b, blocks, &t.g) == GEMM_F16F32_OK;
      q.cost += t.g.cost;
    }
    if (ok && q.cost < p->cost) *p = q;
  }
  p->w_bytes = 0;
  for (int i = 0; i < p->parts; ++i)
    if (p->part[i].g.w_bytes > p->w_bytes) p->w_bytes = p->part[i].g.w_bytes;
  // So far everything goes by strides, and with it the workspace.  A pass over a whose rows lie off
  // 4-byte boundaries by their first address alone gives way to tiles that need none (bf16 16384 x 1
  // x 4096 62 us so, 28 on tiles).
  const bool off_a = (uintptr_t)a.p & 2, off_b = (uintptr_t)b.p & 2;
  for (int i = 0; i < p->parts && !is8(type) && (off_a || off_b); ++i) {
    Part& t = p->part[i];
    if (t.g.path != lk::kPathSkinnyFlip) continue;
    const double cost = narrow_cost(1, t.M, t.N, K, off_a || a.ld % 2 != 0, off_b || b.ld % 2 != 0);
    GemmPlan tiles = t.g;
    const double other = plan_tiles(type, t.M, t.N, K, a, b, 1, &tiles);
    if (other > 0.0 && other + 0.8 < cost) t.g = tiles;
  }
  return GEMM_F16F32_OK;
}

// The kernel arguments of a product, epilogue left empty.
LinArgs product(int64_t type, int64_t K, const Operand& a, const Operand& b) {
  const int64_t E = is8(type) ? 2 : 1;
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
  if (p.pre8) {   // n0 is a multiple of 256
    p.pre8 += t.m0 * p.ldp8 + t.n0;
    p.pre8_scale += t.m0 * p.ldps + t.n0 / 32;
  }
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
  p.sum_first = (int32_t)g.grid();
  return p;
}

int launch(int64_t type, const Product& q, const LinArgs& whole, void* ws, void* stream) {
  const hipStream_t s = (hipStream_t)stream;
  for (int i = 0; i < q.parts; ++i) {
    LinArgs p = part_args(whole, q.part[i], ws);
    if (i > 0) p.sum_part = nullptr;   // the first part's launch has done them
    const GemmPlan& g = q.part[i].g;
    const hipError_t e = type == LINEAR_NORM_F16    ? lk::launch_type<lk::kF16>(g, p, s)
                         : type == LINEAR_NORM_BF16 ? lk::launch_type<lk::kBF16>(g, p, s)
                         : type == LINEAR_NORM_I8   ? lk::launch_type<lk::kI8>(g, p, s)
                                                    : lk::launch_type<lk::kE4M3>(g, p, s);
    if (e != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  return GEMM_F16F32_OK;
}

void carry_sums(LinArgs* p, const float* part, int n, int64_t cols, void* out) {
  p->sum_part = part;
  p->sum_n = n;
  p->sum_cols = (int32_t)cols;
  p->sum_out = (uint16_t*)out;
}

int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return GEMM_F16F32_OK;
  return ws == nullptr || have < need || ((uintptr_t)ws & 15) ? GEMM_F16F32_ERR_WORKSPACE
                                                              : GEMM_F16F32_OK;
}

// Partial column sums of `groups` workgroups, in whole blocks of 32 columns.
int64_t partial_bytes(int64_t groups, int64_t cols) { return groups * round_up(cols, 32) * 4; }

bool bad_dim(int64_t d) { return d < 0 || d >= kMax; }

// ---- checkpoints in 8 bits -----------------------------------------------------------------------
constexpr int64_t kBlock = 32;   // values that share a scale
int check_packed(packed8_matrix* p, int64_t rows, int64_t dim) {
  int rc = check_rows(p->values, rows, dim, &p->values_row, 1, true);
  if (rc == 0) rc = check_rows(p->scale, rows, cdiv(dim, kBlock), &p->scale_row, 1, true);
  return rc;
}
Region values_region(const packed8_matrix& p, int64_t rows, int64_t dim) {
  return region(p.values, rows, dim, p.values_row, 1);
}
Region scale_region(const packed8_matrix& p, int64_t rows, int64_t dim) {
  return region(p.scale, rows, cdiv(dim, kBlock), p.scale_row, 1);
}

// ---- linear_forward ----------------------------------------------------------------------------
struct ForwardPlan {
  Operand a, b;
  Product q;   // no parts: an empty result
};
// `pre`: where the value before the activation goes in 8 bits, or null
int plan_forward(linear_forward_args& x, packed8_matrix* pre, ForwardPlan* f) {
  *f = {};
  if (bad_dim(x.m) || bad_dim(x.n) || bad_dim(x.k)) return GEMM_F16F32_ERR_DIM;
  if (!is16(x.type) && !is8(x.type)) return GEMM_F16F32_ERR_OPTS;
  if (!is16(x.out_type) || (is16(x.type) && x.out_type != x.type)) return GEMM_F16F32_ERR_OPTS;
  if (x.activation < LINEAR_ACT_NONE || x.activation > LINEAR_ACT_SILU)
    return GEMM_F16F32_ERR_OPTS;
  if (is16(x.type) && (x.scale_a || x.scale_b)) return GEMM_F16F32_ERR_OPTS;
  if (pre && x.pre) return GEMM_F16F32_ERR_OPTS;
  // sums of products of up to 2^14 in 32-bit integers
  if (x.type == LINEAR_NORM_I8 && x.k >= (1 << 17)) return GEMM_F16F32_ERR_TOO_LARGE;
  if (x.m == 0 || x.n == 0) return GEMM_F16F32_OK;
  int rc = operand(x.a, x.m, x.k, x.a_row, x.a_col, x.type, &f->a);
  if (rc == 0) rc = operand(x.b, x.n, x.k, x.b_col, x.b_row, x.type, &f->b);
  if (rc == 0) rc = check_rows(x.out, x.m, x.n, &x.out_row, 2, true);
  if (rc == 0) rc = check_rows(x.pre, x.m, x.n, &x.pre_row, 2, false);
  if (rc == 0) rc = check_rows(x.residual, x.m, x.n, &x.residual_row, 2, false);
  if (rc == 0 && pre) rc = check_packed(pre, x.m, x.n);
  if (rc != 0) return rc;
  if (((uintptr_t)x.bias & 1) || (((uintptr_t)x.scale_a | (uintptr_t)x.scale_b) & 3))
    return GEMM_F16F32_ERR_OPTS;
  const packed8_matrix none = {}, &p8 = pre ? *pre : none;
  const Region w[] = {region(x.out, x.m, x.n, x.out_row, 2), region(x.pre, x.m, x.n, x.pre_row, 2),
                      values_region(p8, x.m, x.n), scale_region(p8, x.m, x.n)};
  const Region r[] = {operand_region(f->a, x.m, x.k, x.type), operand_region(f->b, x.n, x.k, x.type),
                      region(x.bias, 1, x.n, x.n, 2), region(x.scale_a, 1, x.m, x.m, 4),
                      region(x.scale_b, 1, x.n, x.n, 4)};
  if (conflict(w, 4, r, 5)) return GEMM_F16F32_ERR_OVERLAP;
  const Region res = region(x.residual, x.m, x.n, x.residual_row, 2);
  const bool in_place = x.residual == x.out && x.residual_row == x.out_row;
  if (overlap(w[1], res) || overlap(w[2], res) || overlap(w[3], res) ||
      (!in_place && overlap(w[0], res)))
    return GEMM_F16F32_ERR_OVERLAP;
  return plan_product(x.type, x.m, x.n, x.k, f->a, f->b, pre != nullptr, &f->q);
}

// ---- linear_backward ----------------------------------------------------------------------------
struct BackwardPlan {
  bool dact;                 // the element-wise pass runs
  bool copy;                 // ... and copies dc to aligned rows, for want of an activation
  bool carry;                // dbias's last step goes with the launch of da's product
  bool pair;                 // the products and dbias's last step go in one launch
  bool small;                // ... and the element-wise pass as well
  Operand b, a, dt;          // b as da's right operand; a and dpre as db's
  bool db_cols;              // db is column-major: the product is its transpose
  Product qa, qb;            // da's and db's products
  int64_t ldd;               // dpre's row stride
  int row_blocks, rows_per_block;
  int64_t dpre_bytes, part_bytes, a_bytes, w_bytes;
  int64_t lda;               // row stride of a, restored from 8 bits
  int64_t bytes() const { return dpre_bytes + part_bytes + a_bytes + w_bytes; }
};
// `kept`: what stands in for a and pre, its parts null where they are given in 16 bits; or null
int plan_backward(linear_backward_args& x, linear_kept* kept, BackwardPlan* f) {
  *f = {};
  if (bad_dim(x.m) || bad_dim(x.n) || bad_dim(x.k)) return GEMM_F16F32_ERR_DIM;
  if (!is16(x.type)) return GEMM_F16F32_ERR_OPTS;
  if (x.activation < LINEAR_ACT_NONE || x.activation > LINEAR_ACT_SILU)
    return GEMM_F16F32_ERR_OPTS;
  const bool act = x.activation != LINEAR_ACT_NONE;
  linear_kept none = {};
  linear_kept& k8 = kept ? *kept : none;
  const bool pre8 = act && k8.pre.values, a8 = k8.a.values != nullptr;
  if (k8.a_activation < LINEAR_ACT_NONE || k8.a_activation > LINEAR_ACT_SILU)
    return GEMM_F16F32_ERR_OPTS;
  // an empty a has no address, packed or not
  if ((pre8 && x.pre) || (a8 && x.a) ||
      (!a8 && k8.a_activation != LINEAR_ACT_NONE && x.m > 0 && x.k > 0))
    return GEMM_F16F32_ERR_OPTS;
  int rc = check_rows(x.dc, x.m, x.n, &x.dc_row, 2, true);
  if (rc == 0 && act && !pre8) rc = check_rows(x.pre, x.m, x.n, &x.pre_row, 2, true);
  if (rc == 0 && pre8) rc = check_packed(&k8.pre, x.m, x.n);
  if (rc == 0 && a8) rc = check_packed(&k8.a, x.m, x.k);
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
    if (a8) {   // in the workspace, rows on 128-byte lines
      f->lda = round_up(x.k, 64);
      f->a = {x.dc, f->lda, false};
      f->a_bytes = x.m > 0 ? round_up(x.m * f->lda * 2, 256) : 0;
    } else {
      rc = operand(x.a, x.k, x.m, x.a_col, x.a_row, x.type, &f->a);
      if (rc != 0) return rc;
      ra = operand_region(f->a, x.k, x.m, x.type);
    }
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
                      region(act ? x.pre : nullptr, x.m, x.n, x.pre_row, 2),
                      values_region(k8.a, x.m, x.k), scale_region(k8.a, x.m, x.k),
                      region(pre8 ? k8.pre.values : nullptr, x.m, x.n, k8.pre.values_row, 1),
                      region(pre8 ? k8.pre.scale : nullptr, x.m, cdiv(x.n, kBlock),
                             k8.pre.scale_row, 1)};
  if (conflict(w, 3, r, 8)) return GEMM_F16F32_ERR_OVERLAP;

  // the element-wise pass: dpre (rows on 128-byte lines), and blocks of rows for its column sums
  f->dact = x.n > 0 && ((act && x.m > 0) || x.dbias);
  const bool to_da = x.da && x.m > 0 && x.k > 0, to_db = x.db && x.k > 0 && x.n > 0;
  // Rows of dc that lie off 16-byte boundaries slow the products' loads; where a pass over dc or one
  // beside it runs anyway, and k pays for it, dc is copied as an activation's dpre would be.  (By the
  // stride alone: the workspace's size goes by it, and not by where dc lies.)  In us,
  // both products read in place / copied: m x n x k 2047 x 1025 x 4097 84 / 72, 1000 x 2001 x 999
  // 28 / 27, 4095 x 4097 x 1023 115 / 105, for 2, 2 and 13 of copying.
  f->copy = !act && x.m > 1 && x.n > 0 && to_da && to_db && x.k >= 2048 && (f->dact || a8) &&
            x.dc_row % 8 != 0;
  f->dact |= f->copy;
  if (f->dact && (act || f->copy)) {
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
  const int64_t ldd = act || f->copy ? f->ldd : x.dc_row;
  const void* const dpre = act || f->copy ? nullptr : x.dc;   // null: in the workspace, aligned
  if (to_da) {
    const Operand d = {dpre, ldd, true};
    rc = plan_product(x.type, x.m, x.k, x.n, d, f->b, false, &f->qa);
    if (rc != 0) return rc;
    if (f->qa.w_bytes > f->w_bytes) f->w_bytes = f->qa.w_bytes;
  }
  if (to_db) {
    f->dt = {dpre, ldd, false};
    rc = f->db_cols ? plan_product(x.type, x.n, x.k, x.m, f->dt, f->a, false, &f->qb)
                    : plan_product(x.type, x.k, x.n, x.m, f->a, f->dt, false, &f->qb);
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
    f->small = f->pair && deep <= 4 && x.n >= 8 && x.k >= 8 && !a8 && !pre8;
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
  // Else the bias gradient's last step goes with da's product on tiles.
  f->carry = !f->pair && f->part_bytes > 0 && f->qa.parts > 0 &&
             f->qa.part[0].g.path == lk::kPathTiles &&
             (f->qa.part[0].g.grid() + cdiv(x.n, 32)) * 256 < kThreads;
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

template <int TY, int OUT, bool LN>
void norm_forward(const nk::NormArgs& p, hipStream_t s) {
  with_row_shape(p.dim, [&](auto nw, auto c) {
    hipLaunchKernelGGL((nk::norm_fwd<TY, OUT, LN, nw.value, c.value>), dim3((uint32_t)p.rows),
                       dim3(64 * nw.value), 0, s, p);
  });
}
template <int TY, int OUT>
void quantize(const nk::QuantizeArgs& p, int64_t rows, hipStream_t s) {
  with_row_shape(p.dim, [&](auto nw, auto c) {
    hipLaunchKernelGGL((nk::quantize_rows<TY, OUT, nw.value, c.value>), dim3((uint32_t)rows),
                       dim3(64 * nw.value), 0, s, p);
  });
}
// f(type, form) with a 16-bit type and a form of rows (nk::kOut16, ...) as constants.
template <class F>
void with_types(int64_t type, int64_t out_type, F f) {
  auto with_out = [&](auto ty) {
    if (out_type == LINEAR_NORM_E4M3) f(ty, std::integral_constant<int, nk::kOutE4M3>{});
    else if (out_type == LINEAR_NORM_I8) f(ty, std::integral_constant<int, nk::kOutI8>{});
    else f(ty, std::integral_constant<int, nk::kOut16>{});
  };
  if (type == LINEAR_NORM_BF16) with_out(std::integral_constant<int, lk::kBF16>{});
  else with_out(std::integral_constant<int, lk::kF16>{});
}
// The backward pass: as above, but short rows take one wave, four of them a workgroup, and rows
// above 8192 fewer waves of more registers.
constexpr int64_t kShortRow = 1024, kLongRow = 16384;
// `small`: the column sums in the same launch (layer norm only, up to 8192 columns).
template <int TY, bool LN>
void norm_backward(const nk::NormBwdArgs& p, int grid, bool small, hipStream_t s) {
#define LN_BACKWARD(NW, C, RW)                                                               \
  do {                                                                                       \
    if constexpr (LN && C <= 2) {                                                            \
      if (small) {                                                                           \
        const int columns = (int)cdiv(p.dim, nk::small_columns(512 * NW * C));               \
        hipLaunchKernelGGL((nk::layer_norm_bwd_small<TY, NW, C, RW>),                        \
                           dim3((uint32_t)(grid + columns)), dim3(64 * NW * RW), 0, s, p,    \
                           columns);                                                         \
        break;                                                                               \
      }                                                                                      \
    }                                                                                        \
    hipLaunchKernelGGL((nk::norm_bwd<TY, LN, NW, C, RW>), dim3((uint32_t)grid),              \
                       dim3(64 * NW * RW), 0, s, p);                                         \
  } while (0)
  if (p.dim <= 512) LN_BACKWARD(1, 1, 4);
  else if (p.dim <= kShortRow) LN_BACKWARD(1, 2, 4);
  else if (p.dim <= 2048) LN_BACKWARD(4, 1, 1);
  else if (p.dim <= 4096) LN_BACKWARD(4, 2, 1);
  else if (p.dim <= 8192) LN_BACKWARD(8, 2, 1);
  else if (p.dim <= kLongRow) LN_BACKWARD(8, 4, 1);
  else
    hipLaunchKernelGGL((nk::norm_bwd_long<TY, LN, 16>), dim3((uint32_t)grid), dim3(1024), 0, s, p);
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

// Bytes of one gradient's partial sums, and of all.
int64_t norm_part_bytes(int64_t rows, int64_t dim) {
  return backward_sums(rows, dim) ? partial_bytes(backward_groups(rows, dim), dim) : 0;
}
// Whether the layer norm's column sums go in the launch of dx, from dy and h read a second time: up to
// 1024 rows, whose columns a workgroup takes in one or two steps.  In a graph / launched one by one,
// in two launches and in one: 256 x 1021 7.1 / 9.4 and 4.6 / 5.9 us, 1024 x 512 5.9 / 9.1 and 5.9 /
// 5.7, 1024 x 8192 28.3 / 27.6 and 24.1 / 23.8; past the rule 2048 x 512 7.2 / 8.9 and 12.3 / 12.1.
// dx in dy's memory would be written while the sums still read it.
bool norm_small(const layer_norm_backward_args& x) {
  return x.rows <= 1024 && x.dim <= 8192 && backward_sums(x.rows, x.dim) && x.rows > 0 &&
         x.dx != x.dy;
}
int64_t norm_backward_bytes(const layer_norm_backward_args& x) {
  if (norm_small(x)) return 0;
  return ((x.dweight != nullptr) + (x.dbias != nullptr)) * norm_part_bytes(x.rows, x.dim);
}

// Column sums from their partial sums; `more`: another gradient's, whose partial sums follow, or null
template <int TY>
void launch_sum(const float* part, int n, int64_t cols, void* out, void* more, hipStream_t s) {
  const int64_t blocks = cdiv(cols, 32), all = more ? 2 * blocks : blocks;
  const int64_t most = kThreads / 256 - 1;
  for (int64_t first = 0; first < all; first += most) {
    const int64_t grid = all - first < most ? all - first : most;
    hipLaunchKernelGGL((nk::sum_partials<TY>), dim3((uint32_t)grid), dim3(256), 0, s, part, n,
                       (int)first, (int)cols, (int)blocks, (uint16_t*)out, (uint16_t*)more);
  }
}

int norm_forward_call(layer_norm_forward_args x, bool ln) {
  int rc = check_norm(x.rows, x.dim, x.type);
  if (rc != GEMM_F16F32_OK) return rc;
  const bool q8 = is8(x.out_type);
  if ((!q8 && x.out_type != x.type) || !(x.eps >= 0.0) || (x.scale && !q8))
    return GEMM_F16F32_ERR_OPTS;
  if (x.rows == 0) return GEMM_F16F32_OK;
  rc = check_rows(x.x, x.rows, x.dim, &x.x_row, 2, true);
  if (rc == 0) rc = check_rows(x.residual, x.rows, x.dim, &x.residual_row, 2, false);
  if (rc == 0) rc = check_rows(x.y, x.rows, x.dim, &x.y_row, q8 ? 1 : 2, true);
  if (rc == 0) rc = check_rows(x.h, x.rows, x.dim, &x.h_row, 2, x.residual != nullptr);
  if (rc != 0) return rc;
  if (x.weight == nullptr || (q8 && x.scale == nullptr)) return GEMM_F16F32_ERR_NULL;
  if ((((uintptr_t)x.weight | (uintptr_t)x.bias) & 1) ||
      (((uintptr_t)x.scale | (uintptr_t)x.mean | (uintptr_t)x.rstd) & 3))
    return GEMM_F16F32_ERR_OPTS;
  const Region rx = region(x.x, x.rows, x.dim, x.x_row, 2);
  const Region rr = region(x.residual, x.rows, x.dim, x.residual_row, 2);
  const Region rh = region(x.h, x.rows, x.dim, x.h_row, 2);
  const Region w[] = {region(x.y, x.rows, x.dim, x.y_row, q8 ? 1 : 2),
                      region(x.scale, 1, x.rows, x.rows, 4), region(x.mean, 1, x.rows, x.rows, 4),
                      region(x.rstd, 1, x.rows, x.rows, 4), rh};
  const Region r[] = {rx, rr, region(x.weight, 1, x.dim, x.dim, 2),
                      region(x.bias, 1, x.dim, x.dim, 2)};
  if (conflict(w, 4, r, 4) || conflict(w, 5, r + 2, 2)) return GEMM_F16F32_ERR_OVERLAP;
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
    p.bias = (const uint16_t*)x.bias;
    p.y = (char*)x.y + ys * r0 * x.y_row;
    p.y_row = x.y_row;
    if (x.scale) p.scale = x.scale + r0;
    if (x.h) p.h = (uint16_t*)x.h + r0 * x.h_row;
    p.h_row = x.h_row;
    if (x.mean) p.mean = x.mean + r0;
    if (x.rstd) p.rstd = x.rstd + r0;
    p.rows = (int32_t)(x.rows - r0 < kRowsPerLaunch ? x.rows - r0 : kRowsPerLaunch);
    p.dim = (int32_t)x.dim;
    p.eps = (float)x.eps;
    p.inv_dim = (float)(1.0 / (double)x.dim);
    with_types(x.type, x.out_type, [&](auto ty, auto out) {
      ln ? norm_forward<ty.value, out.value, true>(p, (hipStream_t)x.stream)
         : norm_forward<ty.value, out.value, false>(p, (hipStream_t)x.stream);
    });
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  return GEMM_F16F32_OK;
}

int norm_backward_call(layer_norm_backward_args x, bool ln) {
  int rc = check_norm(x.rows, x.dim, x.type);
  if (rc == 0) rc = check_rows(x.dy, x.rows, x.dim, &x.dy_row, 2, true);
  if (rc == 0) rc = check_rows(x.h, x.rows, x.dim, &x.h_row, 2, true);
  if (rc == 0) rc = check_rows(x.dh, x.rows, x.dim, &x.dh_row, 2, false);
  if (rc == 0) rc = check_rows(x.dx, x.rows, x.dim, &x.dx_row, 2, true);
  if (rc != 0) return rc;
  if (x.rows > 0 && (x.weight == nullptr || x.rstd == nullptr || (ln && x.mean == nullptr)))
    return GEMM_F16F32_ERR_NULL;
  if ((((uintptr_t)x.weight | (uintptr_t)x.dweight | (uintptr_t)x.dbias) & 1) ||
      (((uintptr_t)x.mean | (uintptr_t)x.rstd) & 3))
    return GEMM_F16F32_ERR_OPTS;
  const int64_t need = ln ? norm_backward_bytes(x)
                          : (x.dweight != nullptr) * norm_part_bytes(x.rows, x.dim);
  rc = check_workspace(x.workspace, x.workspace_bytes, need);
  if (rc != GEMM_F16F32_OK) return rc;
  const Region rdx = region(x.dx, x.rows, x.dim, x.dx_row, 2);
  const Region rdy = region(x.dy, x.rows, x.dim, x.dy_row, 2);
  const Region rdh = region(x.dh, x.rows, x.dim, x.dh_row, 2);
  const Region w[] = {region(x.dweight, 1, x.dim, x.dim, 2), region(x.dbias, 1, x.dim, x.dim, 2),
                      {x.workspace, (uint64_t)need}, rdx};
  const Region r[] = {region(x.h, x.rows, x.dim, x.h_row, 2),
                      region(x.weight, 1, x.dim, x.dim, 2), region(x.mean, 1, x.rows, x.rows, 4),
                      region(x.rstd, 1, x.rows, x.rows, 4), rdy, rdh};
  if (conflict(w, 3, r, 6) || conflict(w, 4, r, 4)) return GEMM_F16F32_ERR_OVERLAP;
  if ((!(x.dx == x.dy && x.dx_row == x.dy_row) && overlap(rdx, rdy)) ||
      (!(x.dx == x.dh && x.dx_row == x.dh_row) && overlap(rdx, rdh)))
    return GEMM_F16F32_ERR_OVERLAP;
  const hipStream_t s = (hipStream_t)x.stream;
  const bool bf = x.type == LINEAR_NORM_BF16;
  const int groups = backward_groups(x.rows, x.dim);
  const bool small = ln && (x.dweight || x.dbias) && norm_small(x);
  const bool sums = !small && backward_sums(x.rows, x.dim);
  float* const part = (float*)x.workspace;
  if (groups > 0) {
    nk::NormBwdArgs p = {};
    p.dy = (const uint16_t*)x.dy;
    p.dy_row = x.dy_row;
    p.h = (const uint16_t*)x.h;
    p.h_row = x.h_row;
    p.weight = (const uint16_t*)x.weight;
    p.mean = x.mean;
    p.rstd = x.rstd;
    p.dh = (const uint16_t*)x.dh;
    p.dh_row = x.dh_row;
    p.dx = (uint16_t*)x.dx;
    p.dx_row = x.dx_row;
    if (sums) {   // dweight's, then dbias'
      if (x.dweight) p.part = part;
      if (x.dbias)
        p.part_bias = part + (x.dweight ? norm_part_bytes(x.rows, x.dim) / 4 : 0);
    } else {
      p.dweight = (uint16_t*)x.dweight;
      p.dbias = (uint16_t*)x.dbias;
    }
    p.rows = (int32_t)x.rows;
    p.dim = (int32_t)x.dim;
    p.inv_dim = (float)(1.0 / (double)x.dim);
    if (ln)
      bf ? norm_backward<lk::kBF16, true>(p, groups, small, s)
         : norm_backward<lk::kF16, true>(p, groups, small, s);
    else
      bf ? norm_backward<lk::kBF16, false>(p, groups, false, s)
         : norm_backward<lk::kF16, false>(p, groups, false, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  if ((x.dweight || x.dbias) && sums) {
    void* const first = x.dweight ? x.dweight : x.dbias;
    void* const more = x.dweight ? x.dbias : nullptr;
    bf ? launch_sum<lk::kBF16>(part, groups, x.dim, first, more, s)
       : launch_sum<lk::kF16>(part, groups, x.dim, first, more, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  return GEMM_F16F32_OK;
}

// ---- checkpoints in 8 bits: launches ---------------------------------------------------------
// Pieces of a row's 8-column chunks: a wave's 64, or for shorter rows the next power of two from 4
// (a block of 32 columns stays in 4 lanes of one wave).
nk::PackArgs pack_args(int64_t dim, const packed8_matrix& p) {
  nk::PackArgs a = {};
  const int64_t chunks = cdiv(dim, kBlock) * 4;
  a.lanes = 2;
  while (a.lanes < 6 && ((int64_t)1 << a.lanes) < chunks) ++a.lanes;
  a.segs = (int32_t)cdiv(chunks, (int64_t)1 << a.lanes);
  a.q = (uint8_t*)p.values;
  a.q_row = p.values_row;
  a.scale = (uint8_t*)p.scale;
  a.s_row = p.scale_row;
  a.dim = (int32_t)dim;
  return a;
}
nk::PackArgs unpack_args(int64_t dim, const packed8_matrix& p, int64_t activation, void* y,
                         int64_t y_row) {
  nk::PackArgs a = pack_args(dim, p);
  a.y = (uint16_t*)y;
  a.y_row = y_row;
  a.act = (int32_t)activation;
  return a;
}
// Launches f(args, grid) over all rows, each launch of at most `most` workgroups; `before` more are
// added to the first one's grid.
template <class F>
int pack_launches(nk::PackArgs a, int64_t rows, int64_t before, int64_t most, F f) {
  const int64_t per = (int64_t)4 * nk::kPackRows * (64 >> a.lanes);   // rows a workgroup
  most = (most / a.segs > 0 ? most / a.segs : 1) * per;               // segs is below 2^23
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    a.rows = (int32_t)n;
    f(a, dim3((uint32_t)(before + cdiv(n, per) * a.segs)));
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
    before = 0;
    if (a.x) a.x += n * a.x_row;
    if (a.y) a.y += n * a.y_row;
    a.q += n * a.q_row;
    a.scale += n * a.s_row;
  }
  return GEMM_F16F32_OK;
}
constexpr int64_t kWorkgroups = kThreads / 256 - 1;   // of 256 threads in a launch

void prepare(int64_t type, const nk::DactArgs& d, const nk::PackArgs& u, int64_t before, dim3 grid,
             hipStream_t s) {
  if (type == LINEAR_NORM_BF16)
    hipLaunchKernelGGL((nk::lin_prepare<lk::kBF16>), grid, dim3(256), 0, s, d, u, (int)before);
  else
    hipLaunchKernelGGL((nk::lin_prepare<lk::kF16>), grid, dim3(256), 0, s, d, u, (int)before);
}

}  // namespace

extern "C" {

int64_t linear_forward_packed_workspace(const linear_forward_args* args,
                                        const packed8_matrix* pre) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_forward_args x = *args;
  packed8_matrix p8 = pre ? *pre : packed8_matrix{};
  ForwardPlan f;
  const int rc = plan_forward(x, pre ? &p8 : nullptr, &f);
  return rc != GEMM_F16F32_OK ? rc : f.q.w_bytes;
}
int64_t linear_forward_workspace(const linear_forward_args* args) {
  return linear_forward_packed_workspace(args, nullptr);
}

int linear_forward(const linear_forward_args* args) { return linear_forward_packed(args, nullptr); }

int linear_forward_packed(const linear_forward_args* args, const packed8_matrix* pre) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_forward_args x = *args;
  packed8_matrix p8 = pre ? *pre : packed8_matrix{};
  ForwardPlan f;
  int rc = plan_forward(x, pre ? &p8 : nullptr, &f);
  if (rc != GEMM_F16F32_OK || f.q.parts == 0) return rc;
  rc = check_workspace(x.workspace, x.workspace_bytes, f.q.w_bytes);
  if (rc != GEMM_F16F32_OK) return rc;
  if (f.q.w_bytes > 0) {
    const Region w = {x.workspace, (uint64_t)f.q.w_bytes};
    const Region o[] = {region(x.out, x.m, x.n, x.out_row, 2), region(x.pre, x.m, x.n, x.pre_row, 2),
                        region(x.residual, x.m, x.n, x.residual_row, 2),
                        operand_region(f.a, x.m, x.k, x.type), operand_region(f.b, x.n, x.k, x.type),
                        region(x.bias, 1, x.n, x.n, 2), region(x.scale_a, 1, x.m, x.m, 4),
                        region(x.scale_b, 1, x.n, x.n, 4), values_region(p8, x.m, x.n),
                        scale_region(p8, x.m, x.n)};
    if (conflict(&w, 1, o, 10)) return GEMM_F16F32_ERR_OVERLAP;
  }
  LinArgs p = product(x.type, x.k, f.a, f.b);
  p.out = (uint16_t*)x.out;
  p.ldo = x.out_row;
  p.pre = (uint16_t*)x.pre;
  p.ldp = x.pre_row;
  p.pre8 = (uint8_t*)p8.values;
  p.ldp8 = p8.values_row;
  p.pre8_scale = (uint8_t*)p8.scale;
  p.ldps = p8.scale_row;
  p.res = (const uint16_t*)x.residual;
  p.ldr = x.residual_row;
  p.bias = (const uint16_t*)x.bias;
  p.scale_a = x.scale_a;
  p.scale_b = x.scale_b;
  p.act = (int32_t)x.activation;
  p.out_type = (int32_t)x.out_type;
  return launch(x.type, f.q, p, x.workspace, x.stream);
}

int64_t linear_backward_packed_workspace(const linear_backward_args* args,
                                         const linear_kept* kept) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_backward_args x = *args;
  linear_kept k8 = kept ? *kept : linear_kept{};
  BackwardPlan f;
  const int rc = plan_backward(x, &k8, &f);
  return rc != GEMM_F16F32_OK ? rc : f.bytes();
}
int64_t linear_backward_workspace(const linear_backward_args* args) {
  return linear_backward_packed_workspace(args, nullptr);
}

int linear_backward(const linear_backward_args* args) {
  return linear_backward_packed(args, nullptr);
}

int linear_backward_packed(const linear_backward_args* args, const linear_kept* kept) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  linear_backward_args x = *args;
  linear_kept k8 = kept ? *kept : linear_kept{};
  BackwardPlan f;
  int rc = plan_backward(x, &k8, &f);
  if (rc != GEMM_F16F32_OK) return rc;
  const bool act = x.activation != LINEAR_ACT_NONE;
  const bool pre8 = act && k8.pre.values != nullptr;
  const int64_t need = f.bytes();
  rc = check_workspace(x.workspace, x.workspace_bytes, need);
  if (rc != GEMM_F16F32_OK) return rc;
  if (need > 0) {
    const Region w = {x.workspace, (uint64_t)need};
    const Region o[] = {region(x.dc, x.m, x.n, x.dc_row, 2),
                        region(act ? x.pre : nullptr, x.m, x.n, x.pre_row, 2),
                        region(x.da, x.m, x.k, x.da_row, 2), region(x.dbias, 1, x.n, x.n, 2),
                        f.a_bytes ? Region{} : operand_region(f.a, x.k, x.m, x.type),
                        operand_region(f.b, x.k, x.n, x.type),
                        f.db_cols ? region(x.db, x.n, x.k, x.db_col, 2)
                                  : region(x.db, x.k, x.n, x.db_row, 2),
                        values_region(k8.a, x.m, x.k), scale_region(k8.a, x.m, x.k),
                        region(pre8 ? k8.pre.values : nullptr, x.m, x.n, k8.pre.values_row, 1),
                        region(pre8 ? k8.pre.scale : nullptr, x.m, cdiv(x.n, kBlock),
                               k8.pre.scale_row, 1)};
    if (conflict(&w, 1, o, 11)) return GEMM_F16F32_ERR_OVERLAP;
  }
  const bool bf = x.type == LINEAR_NORM_BF16;
  const hipStream_t s = (hipStream_t)x.stream;
  char* const ws = (char*)x.workspace;
  const void* dpre = x.dc;
  const bool sums = x.dbias != nullptr && f.dact;
  const bool last = sums && f.row_blocks != 1;   // dbias has a second step
  float* const part = last ? (float*)(ws + f.dpre_bytes) : nullptr;
  nk::DactArgs d = {};
  int64_t before = 0;   // workgroups of the element-wise pass
  if (f.dact && f.row_blocks > 0) {
    d.dc = (const uint16_t*)x.dc;
    d.dc_row = x.dc_row;
    if (act) {
      if (pre8) {
        d.pre8 = (const uint8_t*)k8.pre.values;
        d.pre8_row = k8.pre.values_row;
        d.pre8_scale = (const uint8_t*)k8.pre.scale;
        d.ps_row = k8.pre.scale_row;
      } else {
        d.pre = (const uint16_t*)x.pre;
        d.pre_row = x.pre_row;
      }
    }
    if (act || f.copy) {
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
    before = cdiv(x.n, 512) * f.row_blocks;
  }
  // a from 8 bits beside it, as far as one launch's workgroups go
  nk::PackArgs u = {};
  if (f.a_bytes > 0) {
    f.a.p = ws + f.dpre_bytes + f.part_bytes;
    u = unpack_args(x.k, k8.a, k8.a_activation, (void*)f.a.p, f.lda);
    rc = pack_launches(u, x.m, before, kWorkgroups - before, [&](const nk::PackArgs& b, dim3 grid) {
      prepare(x.type, d, b, before, grid, s);
      before = 0;
    });
    if (rc != GEMM_F16F32_OK) return rc;
  }
  if (before > 0) {
    if (d.pre8 || f.copy)
      prepare(x.type, d, u, before, dim3((uint32_t)before), s);
    else if (bf)
      hipLaunchKernelGGL((nk::lin_dact<lk::kBF16>), dim3((uint32_t)before), dim3(256), 0, s, d);
    else
      hipLaunchKernelGGL((nk::lin_dact<lk::kF16>), dim3((uint32_t)before), dim3(256), 0, s, d);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  if (last && !f.pair && !f.carry) {
    if (bf)
      launch_sum<lk::kBF16>(part, f.row_blocks, x.n, x.dbias, nullptr, s);
    else
      launch_sum<lk::kF16>(part, f.row_blocks, x.n, x.dbias, nullptr, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  void* const W = ws ? ws + f.dpre_bytes + f.part_bytes + f.a_bytes : nullptr;
  LinArgs da = {}, db = {};
  const int64_t ldd = (act || f.copy) && !f.small ? f.ldd : x.dc_row;
  if (f.qa.parts > 0) {
    da = product(x.type, x.n, {dpre, ldd, true}, f.b);
    da.out = (uint16_t*)x.da;
    if (f.carry) carry_sums(&da, part, f.row_blocks, x.n, x.dbias);
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
  const rms_norm_forward_args& a = *args;
  layer_norm_forward_args x = {};
  x.rows = a.rows;
  x.dim = a.dim;
  x.type = a.type;
  x.out_type = a.out_type;
  x.x = a.x;
  x.x_row = a.x_row;
  x.residual = a.residual;
  x.residual_row = a.residual_row;
  x.weight = a.weight;
  x.y = a.y;
  x.y_row = a.y_row;
  x.scale = a.scale;
  x.h = a.h;
  x.h_row = a.h_row;
  x.rstd = a.rstd;
  x.eps = a.eps;
  x.stream = a.stream;
  return norm_forward_call(x, false);
}

int layer_norm_forward(const layer_norm_forward_args* args) {
  return args == nullptr ? (int)GEMM_F16F32_ERR_NULL : norm_forward_call(*args, true);
}

int64_t rms_norm_backward_workspace(const rms_norm_backward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  const int rc = check_norm(args->rows, args->dim, args->type);
  return rc != GEMM_F16F32_OK ? rc
                              : (args->dweight != nullptr) * norm_part_bytes(args->rows, args->dim);
}

int rms_norm_backward(const rms_norm_backward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  const rms_norm_backward_args& a = *args;
  layer_norm_backward_args x = {};
  x.rows = a.rows;
  x.dim = a.dim;
  x.type = a.type;
  x.dy = a.dy;
  x.dy_row = a.dy_row;
  x.h = a.h;
  x.h_row = a.h_row;
  x.weight = a.weight;
  x.rstd = a.rstd;
  x.dh = a.dh;
  x.dh_row = a.dh_row;
  x.dx = a.dx;
  x.dx_row = a.dx_row;
  x.dweight = a.dweight;
  x.workspace = a.workspace;
  x.workspace_bytes = a.workspace_bytes;
  x.stream = a.stream;
  return norm_backward_call(x, false);
}

int64_t layer_norm_backward_workspace(const layer_norm_backward_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  const int rc = check_norm(args->rows, args->dim, args->type);
  return rc != GEMM_F16F32_OK ? rc : norm_backward_bytes(*args);
}

int layer_norm_backward(const layer_norm_backward_args* args) {
  return args == nullptr ? (int)GEMM_F16F32_ERR_NULL : norm_backward_call(*args, true);
}

int quantize_rows(const quantize_rows_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  quantize_rows_args x = *args;
  int rc = check_norm(x.rows, x.dim, x.type);
  if (rc != GEMM_F16F32_OK) return rc;
  if (!is8(x.out_type)) return GEMM_F16F32_ERR_OPTS;
  if (x.rows == 0) return GEMM_F16F32_OK;
  rc = check_rows(x.x, x.rows, x.dim, &x.x_row, 2, true);
  if (rc == 0) rc = check_rows(x.values, x.rows, x.dim, &x.values_row, 1, true);
  if (rc != 0) return rc;
  if (x.scale == nullptr) return GEMM_F16F32_ERR_NULL;
  if ((uintptr_t)x.scale & 3) return GEMM_F16F32_ERR_OPTS;
  const Region w[] = {region(x.values, x.rows, x.dim, x.values_row, 1),
                      region(x.scale, 1, x.rows, x.rows, 4)};
  const Region r = region(x.x, x.rows, x.dim, x.x_row, 2);
  if (conflict(w, 2, &r, 1)) return GEMM_F16F32_ERR_OVERLAP;
  for (int64_t r0 = 0; r0 < x.rows; r0 += kRowsPerLaunch) {
    const int64_t n = x.rows - r0 < kRowsPerLaunch ? x.rows - r0 : kRowsPerLaunch;
    nk::QuantizeArgs p = {};
    p.x = (const uint16_t*)x.x + r0 * x.x_row;
    p.x_row = x.x_row;
    p.y = (uint8_t*)x.values + r0 * x.values_row;
    p.y_row = x.values_row;
    p.scale = x.scale + r0;
    p.dim = (int32_t)x.dim;
    const hipStream_t s = (hipStream_t)x.stream;
    const bool bf = x.type == LINEAR_NORM_BF16;
    if (x.out_type == LINEAR_NORM_I8)
      bf ? quantize<lk::kBF16, nk::kOutI8>(p, n, s) : quantize<lk::kF16, nk::kOutI8>(p, n, s);
    else
      bf ? quantize<lk::kBF16, nk::kOutE4M3>(p, n, s) : quantize<lk::kF16, nk::kOutE4M3>(p, n, s);
    if (hipGetLastError() != hipSuccess) return GEMM_F16F32_ERR_HIP;
  }
  return GEMM_F16F32_OK;
}

int pack8(const pack8_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  pack8_args x = *args;
  if (bad_dim(x.rows) || bad_dim(x.dim)) return GEMM_F16F32_ERR_DIM;
  if (!is16(x.type)) return GEMM_F16F32_ERR_OPTS;
  if (x.rows == 0 || x.dim == 0) return GEMM_F16F32_OK;
  int rc = check_rows(x.x, x.rows, x.dim, &x.x_row, 2, true);
  if (rc == 0) rc = check_packed(&x.out, x.rows, x.dim);
  if (rc != 0) return rc;
  const Region w[] = {values_region(x.out, x.rows, x.dim), scale_region(x.out, x.rows, x.dim)};
  const Region r = region(x.x, x.rows, x.dim, x.x_row, 2);
  if (conflict(w, 2, &r, 1)) return GEMM_F16F32_ERR_OVERLAP;
  nk::PackArgs a = pack_args(x.dim, x.out);
  a.x = (const uint16_t*)x.x;
  a.x_row = x.x_row;
  const hipStream_t s = (hipStream_t)x.stream;
  return pack_launches(a, x.rows, 0, kWorkgroups, [&](const nk::PackArgs& b, dim3 grid) {
    if (x.type == LINEAR_NORM_BF16)
      hipLaunchKernelGGL((nk::pack8<lk::kBF16>), grid, dim3(256), 0, s, b);
    else
      hipLaunchKernelGGL((nk::pack8<lk::kF16>), grid, dim3(256), 0, s, b);
  });
}

int unpack8(const unpack8_args* args) {
  if (args == nullptr) return GEMM_F16F32_ERR_NULL;
  unpack8_args x = *args;
  if (bad_dim(x.rows) || bad_dim(x.dim)) return GEMM_F16F32_ERR_DIM;
  if (!is16(x.type) || x.activation < LINEAR_ACT_NONE || x.activation > LINEAR_ACT_SILU)
    return GEMM_F16F32_ERR_OPTS;
  if (x.rows == 0 || x.dim == 0) return GEMM_F16F32_OK;
  int rc = check_packed(&x.in, x.rows, x.dim);
  if (rc == 0) rc = check_rows(x.y, x.rows, x.dim, &x.y_row, 2, true);
  if (rc != 0) return rc;
  const Region w = region(x.y, x.rows, x.dim, x.y_row, 2);
  const Region r[] = {values_region(x.in, x.rows, x.dim), scale_region(x.in, x.rows, x.dim)};
  if (conflict(&w, 1, r, 2)) return GEMM_F16F32_ERR_OVERLAP;
  const nk::PackArgs a = unpack_args(x.dim, x.in, x.activation, x.y, x.y_row);
  const hipStream_t s = (hipStream_t)x.stream;
  return pack_launches(a, x.rows, 0, kWorkgroups, [&](const nk::PackArgs& b, dim3 grid) {
    if (x.type == LINEAR_NORM_BF16)
      hipLaunchKernelGGL((nk::unpack8_rows<lk::kBF16>), grid, dim3(256), 0, s, b);
    else
      hipLaunchKernelGGL((nk::unpack8_rows<lk::kF16>), grid, dim3(256), 0, s, b);
  });
}

}  // extern "C"
