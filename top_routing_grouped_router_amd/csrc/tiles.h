// Tile lookup shared by the grouped matrix products: which rows of which expert
// a workgroup's tile covers, from the expert offsets on the device.
#pragma once

#include "common.h"

namespace moe {

constexpr int kXcd = 8;

// Workgroups are dealt to the 8 XCDs in turn: this index gives each XCD a
// contiguous run of tiles, so that tiles that share operands share its L2.
__device__ __forceinline__ int flat_tile() {
  const int per = gridDim.x / kXcd;            // the grid is a multiple of 8
  return (blockIdx.x % kXcd) * per + blockIdx.x / kXcd;
}

// Expert and first row of row tile `tile` (tiles of BM rows; prefix sum of
// per-expert tile counts across wave 0, 4 experts per lane); false when there
// is no such tile
template <int BM>
__device__ inline bool find_row_tile_at(int* scratch, const int32_t* offsets, int E, int tile,
                                        int* e_out, int* m0_out, int* mend_out) {
  int& s_e = scratch[0];
  int& s_m0 = scratch[1];
  int& s_mend = scratch[2];
  if (threadIdx.x == 0) s_e = -1;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    // five independent clamped loads (offsets[E] repeats past the end, so
    // those experts count zero rows): one memory latency, no branches
    int o[5];
#pragma unroll
    for (int s = 0; s < 5; ++s) o[s] = offsets[min(lane * 4 + s, E)];
    int tiles[4], sum = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      tiles[s] = (o[s + 1] - o[s] + BM - 1) / BM;
      sum += tiles[s];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(incl, off, 64);
      if (lane >= off) incl += y;
    }
    const int excl = incl - sum;
    if (tile >= excl && tile < incl) {
      int rem = tile - excl;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (rem >= 0 && rem < tiles[s]) {
          const int e = lane * 4 + s;
          s_e = e;
          s_m0 = o[s] + rem * BM;
          s_mend = o[s + 1];
        }
        rem -= tiles[s];
      }
    }
  }
  __syncthreads();
  *e_out = s_e;
  *m0_out = s_m0;
  *mend_out = s_mend;
  return s_e >= 0;
}

// Work list of a persistent row-mode workgroup.  Row tiles are BM rows of one
// expert (ceil(M_e / BM) per expert, in expert order); item it is (row tile
// it / n_tiles_n, column tile it % n_tiles_n).  The workgroup with remapped
// index flat takes items flat, flat + G, flat + 2 G, ... (G workgroups), so
// each round of G items is one contiguous run, cut into one contiguous slice
// per XCD: a row tile's column tiles share that XCD's L2.
constexpr int kMaxItems = 64;

struct RowSched {
  int32_t pref[257];     // row tiles of the experts before e
  int32_t off[257];      // expert row offsets
  int4 desc[kMaxItems];  // expert, first row, end row of the expert, column tile
};

// Builds the prefix of row tiles per expert (wavefront 0: five independent
// clamped loads per lane, then a lane scan) and the workgroup's item table.
// Returns the number of items (the host sizes the grid so that it is at most
// kMaxItems).
template <int BM, int NT>
__device__ inline int build_row_sched(RowSched& S, const int32_t* offsets, int E, int ntn) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int o[5];
#pragma unroll
    for (int s = 0; s < 5; ++s) o[s] = offsets[min(lane * 4 + s, E)];
    int tiles[4], sum = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      tiles[s] = (o[s + 1] - o[s] + BM - 1) / BM;
      sum += tiles[s];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(incl, off, 64);
      if (lane >= off) incl += y;
    }
    int run = incl - sum;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int e = lane * 4 + s;
      if (e <= E) {
        S.pref[e] = run;
        S.off[e] = o[s];
      }
      run += tiles[s];
    }
    if (lane == 63 && E == 256) {
      S.pref[256] = incl;
      S.off[256] = o[4];
    }
  }
  __syncthreads();
  const int G = gridDim.x, flat = flat_tile();
  const int total = S.pref[E] * ntn;
  const int n = flat < total ? min((total - flat + G - 1) / G, kMaxItems) : 0;
  for (int t = threadIdx.x; t < n; t += NT) {
    const int it = flat + t * G;
    const int rt = it / ntn, nt = it - rt * ntn;
    int lo = 0, hi = E - 1;   // first expert e with pref[e + 1] > rt
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (S.pref[mid + 1] > rt) hi = mid; else lo = mid + 1;
    }
    S.desc[t] = make_int4(lo, S.off[lo] + (rt - S.pref[lo]) * BM, S.off[lo + 1], nt);
  }
  __syncthreads();
  return n;
}

}  // namespace moe
