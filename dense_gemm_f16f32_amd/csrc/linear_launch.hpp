// The linear layer's products: how one runs, and its launch.
#pragma once

#include "linear_kernels.hpp"
#include "skinny_kernels.hpp"

namespace lk {

// Tiles of the matrix products: BM x BN, 64 slots deep.
enum { kTile256, kTile128, kTile64, kTiles };
struct TileShape {
  int bm, bn;
};
constexpr TileShape kTileShapes[kTiles] = {{256, 256}, {128, 128}, {64, 64}};
constexpr int kTileDepth = 64;   // slots

enum { kPathTiles, kPathSkinnyK, kPathSkinnyN };
constexpr int kSkinnyRows = 16;   // rows of the skinny kernels' one MFMA block

// How one matrix product runs: `programs` workgroups a pass over the result, of which those from
// `whole` on are split into `splits` slices of `per_split` panels (tiles) or units (skinny) of
// k, with w_bytes of workspace for their sums.
struct GemmPlan {
  int path, tile, cols;   // cols: skinny columns a workgroup
  bool akm, bkm;
  int64_t programs, whole;
  int splits, per_split;
  int64_t w_bytes;
  double cost;            // estimated time in us
  int64_t grid() const { return whole + (programs - whole) * splits; }
};

template <int TY, bool AKM, bool BKM, bool HALVES>
void launch_staged(const GemmPlan& g, const LinArgs& a, dim3 grid, hipStream_t s) {
  // operands of a panel are read as many k steps ahead as a panel of the type has, less one
  constexpr int RD = TY == kE4M3 ? 1 : 3;
  if (g.tile == kTile128)
    hipLaunchKernelGGL((lin_staged<TY, 128, 128, 64, 2, RD, 2, 2, AKM, BKM, HALVES>), grid,
                       dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((lin_staged<TY, 64, 64, 64, 4, RD, 2, 2, AKM, BKM, HALVES>), grid,
                       dim3(256), 0, s, a);
}

template <int TY, bool AKM, bool BKM>
void launch_tile(const GemmPlan& g, const LinArgs& a, dim3 grid, hipStream_t s) {
  if (g.tile == kTile256)
    hipLaunchKernelGGL((lin_ring<TY, AKM, BKM>), grid, dim3(256), 0, s, a);
  else if (TY == kE4M3 && a.K <= kHalvesK)
    launch_staged<TY, AKM, BKM, TY == kE4M3>(g, a, grid, s);
  else
    launch_staged<TY, AKM, BKM, false>(g, a, grid, s);
}

template <int TY, int BM, int BN>
void launch_reduce(const GemmPlan& g, const LinArgs& a, hipStream_t s) {
  constexpr int PER = (BM * BN / 8 + 255) / 256;
  hipLaunchKernelGGL((lin_reduce<TY, BM, BN>), dim3((uint32_t)((g.programs - g.whole) * PER)),
                     dim3(256), 0, s, a);
}

template <int TY>
hipError_t launch_type(const GemmPlan& g, const LinArgs& a, hipStream_t s) {
  const dim3 grid((uint32_t)g.grid());
  if (g.path == kPathSkinnyK) {
    if (a.K < (TY == kE4M3 ? 16 : 8))   // such rows need no more than one wave
      hipLaunchKernelGGL((lin_skinny_k<TY, 1, 1, true>), grid, dim3(64), 0, s, a);
    else if (g.cols == 16)
      hipLaunchKernelGGL((lin_skinny_k<TY, 1, 8, false>), grid, dim3(512), 0, s, a);
    else if (g.cols == 32)
      hipLaunchKernelGGL((lin_skinny_k<TY, 2, 8, false>), grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((lin_skinny_k<TY, 4, 8, false>), grid, dim3(512), 0, s, a);
  } else if (g.path == kPathSkinnyN) {
    if constexpr (TY != kE4M3) {
      hipLaunchKernelGGL((lin_skinny_n<TY, 4, 8>), grid, dim3(512), 0, s, a);
    }
  } else if constexpr (TY == kE4M3) {
    launch_tile<TY, true, true>(g, a, grid, s);
  } else if (g.akm) {
    if (g.bkm)
      launch_tile<TY, true, true>(g, a, grid, s);
    else
      launch_tile<TY, true, false>(g, a, grid, s);
  } else {
    if (g.bkm)
      launch_tile<TY, false, true>(g, a, grid, s);
    else
      launch_tile<TY, false, false>(g, a, grid, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.splits == 1) return e;
  if (g.path != kPathTiles)
    g.cols == 16   ? launch_reduce<TY, 16, 16>(g, a, s)
    : g.cols == 32 ? launch_reduce<TY, 16, 32>(g, a, s)
                   : launch_reduce<TY, 16, 64>(g, a, s);
  else if (g.tile == kTile256)
    launch_reduce<TY, 256, 256>(g, a, s);
  else if (g.tile == kTile128)
    launch_reduce<TY, 128, 128>(g, a, s);
  else
    launch_reduce<TY, 64, 64>(g, a, s);
  return hipGetLastError();
}

template <int TY>
hipError_t launch_pair(const PairArgs& p, bool bkm, hipStream_t s) {
  const dim3 grid((uint32_t)(p.da.num_programs + p.db.num_programs +
                             (p.dbias ? (p.cols + 31) / 32 : 0)));
  if (bkm)
    hipLaunchKernelGGL((lin_pair<TY, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((lin_pair<TY, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <int TY>
hipError_t launch_small(const SmallArgs& p, bool bkm, bool cols, hipStream_t s) {
  const dim3 grid((uint32_t)(p.da.num_programs + p.db.num_programs));
  if (bkm && cols)
    hipLaunchKernelGGL((lin_small_bwd<TY, true, true>), grid, dim3(256), 0, s, p);
  else if (bkm)
    hipLaunchKernelGGL((lin_small_bwd<TY, true, false>), grid, dim3(256), 0, s, p);
  else if (cols)
    hipLaunchKernelGGL((lin_small_bwd<TY, false, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((lin_small_bwd<TY, false, false>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace lk
