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

// How one matrix product runs.
struct GemmPlan {
  int path, tile, cols;   // cols: skinny columns a workgroup
  bool akm, bkm;
  int splits, per_split;  // per_split in panels (tiles) or units (skinny)
  int64_t programs;       // workgroups of one slice
  int64_t ldw, w_bytes;   // split K's partial sums (0: none)
};

template <int TY, bool AKM, bool BKM, bool SPLIT>
void launch_tile(const GemmPlan& g, const LinArgs& a, dim3 grid, hipStream_t s) {
  // operands of a panel are read as many k steps ahead as a panel of the type has, less one
  constexpr int RD = TY == kE4M3 ? 1 : 3;
  switch (g.tile) {
    case kTile256:
      hipLaunchKernelGGL((lin_ring<TY, AKM, BKM, SPLIT>), grid, dim3(256), 0, s, a);
      break;
    case kTile128:
      hipLaunchKernelGGL((lin_staged<TY, 128, 128, 64, 2, RD, 2, 2, AKM, BKM, SPLIT>), grid,
                         dim3(256), 0, s, a);
      break;
    default:
      hipLaunchKernelGGL((lin_staged<TY, 64, 64, 64, 4, RD, 2, 2, AKM, BKM, SPLIT>), grid,
                         dim3(256), 0, s, a);
  }
}

template <int TY, bool AKM, bool BKM>
void launch_layout(const GemmPlan& g, const LinArgs& a, dim3 grid, hipStream_t s) {
  if (g.splits > 1)
    launch_tile<TY, AKM, BKM, true>(g, a, grid, s);
  else
    launch_tile<TY, AKM, BKM, false>(g, a, grid, s);
}

template <int TY>
hipError_t launch_type(const GemmPlan& g, const LinArgs& a, hipStream_t s) {
  const dim3 grid((uint32_t)(g.programs * g.splits));
  if (g.path == kPathSkinnyK) {
    hipLaunchKernelGGL((lin_skinny_k<TY, 8>), grid, dim3(512), 0, s, a);
  } else if (g.path == kPathSkinnyN) {
    if constexpr (TY != kE4M3) {
      if (g.cols == 128)
        hipLaunchKernelGGL((lin_skinny_n<TY, 8, 8>), grid, dim3(512), 0, s, a);
      else
        hipLaunchKernelGGL((lin_skinny_n<TY, 4, 8>), grid, dim3(512), 0, s, a);
    }
  } else if constexpr (TY == kE4M3) {
    launch_layout<TY, true, true>(g, a, grid, s);
  } else if (g.akm) {
    if (g.bkm)
      launch_layout<TY, true, true>(g, a, grid, s);
    else
      launch_layout<TY, true, false>(g, a, grid, s);
  } else {
    if (g.bkm)
      launch_layout<TY, false, true>(g, a, grid, s);
    else
      launch_layout<TY, false, false>(g, a, grid, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.splits == 1) return e;
  const int64_t threads = (int64_t)a.M * (a.ldw / 8);
  hipLaunchKernelGGL((lin_reduce<TY>), dim3((uint32_t)((threads + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace lk
