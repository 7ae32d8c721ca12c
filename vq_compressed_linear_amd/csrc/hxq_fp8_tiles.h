// Which rows a workgroup of a block-scaled product owns: device helpers shared
// by its kernels.
#pragma once

#include "hxq_fp8.h"
#include "hxq_fp8_device.h"

namespace hxq {

struct RowTile {
  int expert;  // 0 for one layer
  int row0;    // first row of y
  int rows;    // rows of the tile; 0: none
};

// First row of expert e, kept within the rows there are, so that offsets that
// break their contract cannot lead out of the tensors.
__device__ __forceinline__ int fp8_offset(const Fp8Args& a, int e) { return min(max(a.offsets[e], 0), a.M); }

// Rows [0, end) belong to some expert.
__device__ __forceinline__ int fp8_rows_end(const Fp8Args& a) { return a.offsets ? fp8_offset(a, a.E) : a.M; }

// Tile t of height tm over the rows: without experts rows t tm .. + tm - 1,
// else the t-th tile when each expert's rows are cut into tiles of their own.
// Found by every wave for itself: the 64 lanes look at 64 experts at a time.
// (Counts are kept below 2^30, past the 2^22 tiles of a launch, so that offsets
// that break their contract cannot overflow them.)
__device__ __forceinline__ RowTile fp8_row_tile(const Fp8Args& a, int t, int tm) {
  if (!a.offsets) return {0, t * tm, min(tm, a.M - t * tm)};
  const int lane = lane_id();
  int before = 0;  // tiles of the experts before this round's
  for (int e0 = 0; e0 < a.E; e0 += kWave) {
    const int e = min(e0 + lane, a.E - 1);
    const int lo = fp8_offset(a, e), hi = fp8_offset(a, e + 1);
    const int rows = e0 + lane < a.E ? max(hi - lo, 0) : 0;
    const int tiles = min((int)(((int64_t)rows + tm - 1) / tm), 1 << 23);
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(incl, d, kWave);
      if (lane >= d) incl += o;
    }
    const uint64_t past = __ballot(before + incl > t);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = before + __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(tiles, l);
      const int r = (t - first) * tm;
      const int n = __builtin_amdgcn_readlane(rows, l) - r;
      return {e0 + l, __builtin_amdgcn_readlane(lo, l) + r, min(n, tm)};
    }
    before = min(before + __builtin_amdgcn_readlane(incl, kWave - 1), 1 << 29);
  }
  return {0, 0, 0};
}

// How many such tiles there are, at most `most`.
__device__ __forceinline__ int fp8_row_tiles(const Fp8Args& a, int tm, int most) {
  int n = 0;
  for (int e = lane_id(); e < a.E; e += kWave) {
    const int rows = max(fp8_offset(a, e + 1) - fp8_offset(a, e), 0);
    n = min(n + min((int)(((int64_t)rows + tm - 1) / tm), most), most);
  }
  return min(wave_sum_dpp_i(n), most);  // most <= 2^22: 64 of them fit
}

// The expert of row m (m < fp8_rows_end): the last e with offset(e) <= m.
__device__ __forceinline__ int fp8_expert_of(const Fp8Args& a, int m) {
  int lo = 0, hi = a.E;  // offset(lo) <= m < offset(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (fp8_offset(a, mid) <= m)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The row of x that row m of y reads; an index out of range reads the nearest row there is.
__device__ __forceinline__ int64_t fp8_x_row(const Fp8Args& a, int m) {
  if (!a.rows) return m;
  const int r = a.rows[m];
  return r < 0 ? 0 : ((int64_t)r < a.Mx ? r : a.Mx - 1);
}

__device__ __forceinline__ void fp8_store(const Fp8Args& a, int64_t at, float v) {
  if (a.y_bf16)
    static_cast<uint16_t*>(a.y)[at] = to_bf16(v);
  else
    static_cast<float*>(a.y)[at] = v;
}

}  // namespace hxq
