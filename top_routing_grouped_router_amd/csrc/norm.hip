// The root-mean-square norm in front of the layer, with the residual's addition
// and 8-bit rows for low-precision experts, and its backward pass.
//
//   s = round(x + r);  rstd = 1 / sqrt(mean(s^2) + eps);  y = (s rstd) w
// The norm is taken of s as it is stored (rounded to the act type), so the
// backward pass, which reads s, differentiates what the forward computed.
// Squares are taken and summed in 64 bits, which HBM's time covers (16384 x 2048 bf16
// with 8-bit rows: 50.4 us, as with fp32 squares), y is an fp32 product rounded once to
// the act type, and the 8-bit rows are the roundings of y itself, not of that product:
// near ties it is computed again with what its roundings lost (16384 x 2048 rows: no
// element off instead of 24, for 4% more time, and 9% if every element were computed so).
//   n = s rstd;  g = dy w;  dx = rstd (g - n mean(g n)) + dsum;  dw = sum_t dy n
//
// Every pass is bound by HBM: each tensor is read and written once, with the
// row held in registers between the sum of squares and the scaling.  A short row
// belongs to one wavefront (no barrier, no LDS), a longer one to a workgroup of
// four (fewer bytes per lane, so more rows under way), and rows longer than a
// workgroup's registers are read twice (kWavePieces).
//
// Measured: 16384 x 2048 bf16 with residual, y and 8-bit rows (303 MB) 50.5 us, 6.0
// TB/s (a large copy reaches 5.2); forward and backward there (470 MB) 93 us, of which
// 44, 45 and 4 for the weight gradient's second step; one row of 2048 2.5 us.
#include <algorithm>

#include "mx.h"
#include "two_floats.h"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;

// v plus its value in the neighbouring 16 lanes (ROWS) or the other 32
template <bool ROWS, typename F>
__device__ __forceinline__ F swap_sum(F v) {
  uint32_t a[sizeof(F) / 4], b[sizeof(F) / 4];
  __builtin_memcpy(a, &v, sizeof(F));
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(F) / 4); ++i) {
    const auto t = ROWS ? __builtin_amdgcn_permlane16_swap(a[i], a[i], false, false)
                        : __builtin_amdgcn_permlane32_swap(a[i], a[i], false, false);
    a[i] = t[0];
    b[i] = t[1];
  }
  F x, y;
  __builtin_memcpy(&x, a, sizeof(F));
  __builtin_memcpy(&y, b, sizeof(F));
  return x + y;
}

// the sum over the wavefront, the same in every lane
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
  v += from_lane<kSwap1>(v);
  v += from_lane<kSwap2>(v);
  v += from_lane<kMirror8>(v);
  v += from_lane<kMirror16>(v);
  return swap_sum<false>(swap_sum<true>(v));
}

// the sum over the lanes of the wavefront with the same lane % 4
__device__ __forceinline__ float runs_sum(float v) {
  v += from_lane<kAlong8>(v);
  v += from_lane<kAlong4>(v);
  return swap_sum<false>(swap_sum<true>(v));
}

// sum over the W wavefronts of a row (W = 1: the wavefront's own), the same in
// every lane.  The caller's loop may come here again at once: two barriers.
template <int W, typename F>
__device__ __forceinline__ F row_sum(F v) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    __shared__ F part[W];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w];
    __syncthreads();
  }
  return v;
}

// sum += N squares, in 64 bits: no value of fp32 overflows or vanishes, and what the
// additions lose lies below what rstd's two floats hold
template <int N>
__device__ __forceinline__ double squares(const float* v, double sum) {
#pragma unroll
  for (int i = 0; i < N; ++i) sum = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), sum);
  return sum;
}

// 1 / sqrt(m): the instruction's estimate (about 24 bits) and a step of Newton's
// method, which doubles them
__device__ __forceinline__ Rstd inverse_root(double m) {
  double r = __builtin_amdgcn_rsq(m);
  if (m > 0.0 && m < HUGE_VAL) r = fma(r, 0.5 * fma(-m * r, r, 1.0), r);
  Rstd out;
  out.hi = static_cast<float>(r);
  out.lo = static_cast<float>(r - out.hi);
  return out;
}

// The 8-bit rows are the roundings of y itself.  v = fl(fl(s rstd.hi) w) is within
// 3 * 2^-24 |y| of it, at most 3 of its last places, so only a v that close to a tie
// between elements, or to a scale's limit, can round to another element; these all
// have 19 zero bits behind the first four of the significand.  (Where rstd.lo, or
// what a product of y loses, falls below fp32's range -- rows above 2^100, a y below
// 2^-100 -- an element that close to a tie may be its other neighbour.)
constexpr int kTieShift = 32 - 19;
constexpr uint32_t kTieNear = 4u << kTieShift;   // 4 last places, those bits at the top

struct NormArgs {
  const void* x;
  const void* res;
  const float* weight;
  void* sum;
  void* y;
  uint8_t* q;
  uint8_t* q_scale;
  float* rstd;
  int64_t T;
  int d;
  float eps;
  double inv_d;   // 1 / d
};

// a 16-byte piece: one that is read once goes past the caches' retention (with the
// store of y the same, 62.5 -> 55.7 us at 16384 x 2048 bf16; sum and dx, which the
// next pass reads, are stored as usual)
__device__ __forceinline__ uint4 load16(const void* p, int64_t piece) {
  return ld_nt16(reinterpret_cast<const uint4*>(p) + piece);
}
__device__ __forceinline__ uint4 load16_kept(const void* p, int64_t piece) {
  return reinterpret_cast<const uint4*>(p)[piece];
}

// s of one 16-byte piece, as stored, in fp32; writes it to `sum` if there is one
template <typename T>
__device__ __forceinline__ void piece_sum(const NormArgs& g, int64_t at, uint4 xv, uint4 rv,
                                          float* s) {
  constexpr int N = Act<T>::kPer16B;
  unpack16(xv, s, T{});
  if (g.res) {
    float r[N];
    unpack16(rv, r, T{});
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += r[i];
    const uint4 packed = pack16(s, T{});
    if (g.sum) reinterpret_cast<uint4*>(g.sum)[at] = packed;
    unpack16(packed, s, T{});
  } else if (g.sum) {
    reinterpret_cast<uint4*>(g.sum)[at] = xv;
  }
}

// y of one piece from s: the act row, the 8-bit row and its scales
template <typename T>
__device__ __forceinline__ void piece_out(const NormArgs& g, int64_t row, int p, int per_row,
                                          Rstd rstd, const float* s) {
  constexpr int N = Act<T>::kPer16B;
  constexpr int kLanes = 32 / N;
  float v[N], w[N];
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(w + i) =
      reinterpret_cast<const float4*>(g.weight)[p * (N / 4) + i / 4];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = s[i] * rstd.hi * w[i];
  if (g.y) st_nt16(reinterpret_cast<uint4*>(g.y) + row * per_row + p, pack16(v, T{}));
  if (g.q) {
    uint32_t least = ~0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
      least = min(least, (__float_as_uint(v[i]) << kTieShift) + kTieNear);
    if (least <= 2 * kTieNear) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = scaled_odd(s[i], rstd, w[i]);
    }
    const uint32_t sb = mx_store<kE4M3, N>(v, g.q + (row * per_row + p) * N);
    if (p % kLanes == 0) {
      const int ld = mx_scale_ld(g.d), b = p / kLanes;
      uint8_t* out = g.q_scale + row * ld + b;
      *out = static_cast<uint8_t>(sb);
      if (b == ld - 3 && g.d % 128) out[1] = out[2] = 0;   // the row's padding
    }
  }
}

// W wavefronts per row, NV 16-byte pieces per lane
template <typename T, int W, int NV>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs g) {
  constexpr int N = Act<T>::kPer16B;
  constexpr int L = 64 * W;   // lanes of a row
  constexpr int kRows = kThreads / L;
  const int lane = threadIdx.x % L, per_row = g.d / N;
  // one turn unless the grid limit is passed (whole wavefronts leave, and whole
  // workgroups where they join)
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / L; row < g.T;
       row += static_cast<int64_t>(gridDim.x) * kRows) {
    uint4 xv[NV], rv[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int p = lane + u * L;
      xv[u] = rv[u] = make_uint4(0, 0, 0, 0);
      if (p < per_row) {
        xv[u] = load16(g.x, row * per_row + p);
        if (g.res) rv[u] = load16(g.res, row * per_row + p);
      }
    }
    float s[NV][N];
    double ss = 0.0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int p = lane + u * L;
      if (p < per_row) {
        piece_sum<T>(g, row * per_row + p, xv[u], rv[u], s[u]);
        ss = squares<N>(s[u], ss);
      }
    }
    const Rstd rstd = inverse_root(row_sum<W>(ss) * g.inv_d + g.eps);
    if (g.rstd && lane == 0) g.rstd[row] = rstd.hi;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int p = lane + u * L;
      if (p < per_row) piece_out<T>(g, row, p, per_row, rstd, s[u]);
    }
  }
}

// rows of any length, one workgroup each, read twice (the second time s comes
// from `sum` where it was written, since `sum` may be x or the residual)
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_long_kernel(NormArgs g) {
  constexpr int N = Act<T>::kPer16B;
  const int per_row = g.d / N;
  NormArgs again = g;
  again.sum = nullptr;
  if (g.sum) {
    again.x = g.sum;
    again.res = nullptr;
  }
  for (int64_t row = blockIdx.x; row < g.T; row += gridDim.x) {
    double ss = 0.0;
    for (int p = threadIdx.x; p < per_row; p += kThreads) {
      float s[N];
      const int64_t at = row * per_row + p;
      piece_sum<T>(g, at, load16_kept(g.x, at),
                   g.res ? load16_kept(g.res, at) : make_uint4(0, 0, 0, 0), s);
      ss = squares<N>(s, ss);
    }
    const Rstd rstd = inverse_root(row_sum<kWaves>(ss) * g.inv_d + g.eps);
    if (g.rstd && threadIdx.x == 0) g.rstd[row] = rstd.hi;
    for (int p = threadIdx.x; p < per_row; p += kThreads) {
      float s[N];
      const int64_t at = row * per_row + p;
      piece_sum<T>(again, at, load16_kept(again.x, at),
                   again.res ? load16_kept(again.res, at) : make_uint4(0, 0, 0, 0), s);
      piece_out<T>(g, row, p, per_row, rstd, s);
    }
  }
}

// ---------------------------------------------------------------- backward

struct NormBwdArgs {
  const void* dy;
  const void* s;
  const float* weight;
  const float* rstd;
  const void* dsum;
  void* dx;
  float* part;     // [workgroups, d] weight-gradient partial sums
  int64_t T;
  int64_t chunk;   // rows of a workgroup
  int d;
};

// dx of one piece
template <typename T>
__device__ __forceinline__ void dx_out(const NormBwdArgs& a, int64_t at, float rstd, float c,
                                       const float* gw, const float* n, uint4 dsv) {
  constexpr int N = Act<T>::kPer16B;
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = rstd * (gw[i] - n[i] * c);
  if (a.dsum) {
    float t[N];
    unpack16(dsv, t, T{});
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += t[i];
  }
  reinterpret_cast<uint4*>(a.dx)[at] = pack16(v, T{});
}

// A workgroup takes `chunk` consecutive rows, W wavefronts to a row, and keeps
// the weight gradient of its lanes' columns in registers over all of them; the
// 4 / W row streams are then added in a fixed order.
template <typename T, int W, int NV>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int N = Act<T>::kPer16B;
  constexpr int L = 64 * W, S = kThreads / L;
  const int stream = threadIdx.x / L, lane = threadIdx.x % L, per_row = a.d / N;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t r1 = min(r0 + a.chunk, a.T);
  constexpr bool kKeep = NV <= 4;   // more pieces: the weight is read again (registers)
  float w[NV][N], dw[NV][N];
  auto weights = [&](int u) {
    const int p = lane + u * L;
#pragma unroll
    for (int i = 0; i < N; ++i) w[u][i] = p < per_row ? a.weight[p * N + i] : 0.0f;
  };
#pragma unroll
  for (int u = 0; u < NV; ++u) {
#pragma unroll
    for (int i = 0; i < N; ++i) dw[u][i] = 0.0f;
    if (kKeep) weights(u);
  }
  for (int64_t row = r0 + stream; row < r1; row += S) {
    if (!kKeep) asm volatile("" ::: "memory");   // each row again, not kept
    uint4 dyv[NV], sv[NV], dsv[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int p = lane + u * L;
      dyv[u] = sv[u] = dsv[u] = make_uint4(0, 0, 0, 0);
      if (p < per_row) {
        dyv[u] = load16(a.dy, row * per_row + p);
        sv[u] = load16(a.s, row * per_row + p);
        if (a.dsum) dsv[u] = load16(a.dsum, row * per_row + p);
      }
    }
    const float rstd = a.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float dy[N], s[N];
      unpack16(dyv[u], dy, T{});
      unpack16(sv[u], s, T{});
      if (!kKeep) weights(u);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = s[i] * rstd;
        dot += dy[i] * w[u][i] * n;
        dw[u][i] += dy[i] * n;
      }
    }
    const float c = row_sum<W>(dot) / static_cast<float>(a.d);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int p = lane + u * L;
      if (p >= per_row) continue;
      float gw[N], n[N];
      unpack16(dyv[u], gw, T{});
      unpack16(sv[u], n, T{});
      if (!kKeep) weights(u);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        gw[i] *= w[u][i];
        n[i] *= rstd;
      }
      dx_out<T>(a, row * per_row + p, rstd, c, gw, n, dsv[u]);
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.d;
  __shared__ float lds[S > 1 ? L * NV * N : 1];
  for (int t = 0; t < S; ++t) {
    if (stream == t) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int p = lane + u * L;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (S > 1 && t > 0) dw[u][i] += lds[(u * N + i) * L + lane];
          if (t + 1 < S) lds[(u * N + i) * L + lane] = dw[u][i];
        }
        if (t + 1 == S && p < per_row) {
#pragma unroll
          for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4*>(part + p * N + i) =
                make_float4(dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]);
        }
      }
    }
    if (t + 1 < S) __syncthreads();
  }
}

// dx of rows of any length, one workgroup each, read twice
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_bwd_long_kernel(NormBwdArgs a) {
  constexpr int N = Act<T>::kPer16B;
  const int per_row = a.d / N;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float c = 0.0f;
    for (int turn = 0; turn < 2; ++turn) {
      float dot = 0.0f;
      for (int p = threadIdx.x; p < per_row; p += kThreads) {
        const int64_t at = row * per_row + p;
        float gw[N], n[N];
        unpack16(load16_kept(a.dy, at), gw, T{});
        unpack16(load16_kept(a.s, at), n, T{});
#pragma unroll
        for (int i = 0; i < N; ++i) {
          gw[i] *= a.weight[p * N + i];
          n[i] *= rstd;
          dot += gw[i] * n[i];
        }
        if (turn)
          dx_out<T>(a, at, rstd, c, gw, n,
                    a.dsum ? load16_kept(a.dsum, at) : make_uint4(0, 0, 0, 0));
      }
      if (!turn) c = row_sum<kWaves>(dot) / static_cast<float>(a.d);
    }
  }
}

// the weight gradient's partial sums of long rows: one lane per 16-byte piece
// of the row, over the workgroup's chunk of rows.  Runs before the dx kernel,
// since dx may be written over dy.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_dw_long_kernel(NormBwdArgs a) {
  constexpr int N = Act<T>::kPer16B;
  const int per_row = a.d / N, p = blockIdx.y * kThreads + threadIdx.x;
  if (p >= per_row) return;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t r1 = min(r0 + a.chunk, a.T);
  float dw[N] = {};
  for (int64_t row = r0; row < r1; ++row) {
    const float rstd = a.rstd[row];
    float dy[N], s[N];
    unpack16(load16(a.dy, row * per_row + p), dy, T{});
    unpack16(load16(a.s, row * per_row + p), s, T{});
#pragma unroll
    for (int i = 0; i < N; ++i) dw[i] += dy[i] * (s[i] * rstd);
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.d + p * N;
#pragma unroll
  for (int i = 0; i < N; ++i) part[i] = dw[i];
}

// dweight[c]: the partial sums of 16 columns (four lanes of float4) by 64 runs of
// workgroups, then a tree over the runs: a fixed order
__global__ __launch_bounds__(kThreads) void norm_dw_kernel(const float* part, int parts, int d,
                                                           float* dweight) {
  constexpr int kRuns = 64;
  __shared__ float4 lds[kWaves][4];
  const int c4 = threadIdx.x & 3, run = threadIdx.x >> 2;
  const int col = blockIdx.x * 16 + c4 * 4;   // d is a multiple of 64
  const int len = (parts + kRuns - 1) / kRuns;
  const int b = run * len, e = min(b + len, parts);
  float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
  for (int i = b; i < e; ++i) {
    const float4 t = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(i) * d + col);
    v.x += t.x;
    v.y += t.y;
    v.z += t.z;
    v.w += t.w;
  }
  v.x = runs_sum(v.x);
  v.y = runs_sum(v.y);
  v.z = runs_sum(v.z);
  v.w = runs_sum(v.w);
  if ((threadIdx.x & 63) < 4) lds[threadIdx.x >> 6][c4] = v;
  __syncthreads();
  if (threadIdx.x < 4) {
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      const float4 t = lds[w][c4];
      v.x += t.x;
      v.y += t.y;
      v.z += t.z;
      v.w += t.w;
    }
    *reinterpret_cast<float4*>(dweight + col) = v;
  }
}

// Pieces per lane (a power of two) that hold a row of `pieces` 16-byte pieces
// in `lanes` lanes; 0 if that is more than 8 (registers)
int pieces_per_lane(int pieces, int lanes) {
  for (int nv = 1; nv <= 8; nv *= 2)
    if (pieces <= nv * lanes) return nv;
  return 0;
}

// workgroups for `n` of rows: a launch holds fewer than 2^32 threads
unsigned row_grid(int64_t n) { return static_cast<unsigned>(std::min<int64_t>(n, 1 << 23)); }

// Pieces of a row per lane up to which the row belongs to one wavefront.  us, bf16,
// forward / backward, a wavefront and a workgroup to a row:
//   2 pieces: 16384 x 1024 29.0 / 28.4 and 32.6 / 43.7, 64 x 1024 5.6 / 6.7 and 5.0 / 6.4;
//   4 pieces: 16384 x 2048 55.8 / 53.3 and 50.4 / 57.7, 512 x 2048 7.2 / 8.4 and 5.6 / 8.7,
//   64 x 2048 6.7 / 7.5 and 5.1 / 6.6.
// So the backward pass gives a wavefront 4 pieces too where there are rows enough.
// Rows in registers against rows read twice: 16384 x 4096 99 / 108 and 127 / 163, 8 pieces
// to a lane of a workgroup 16384 x 16384 445 / 495 and 492 / 687.
constexpr int kWavePieces = 2;
constexpr int64_t kWideWaveRows = 512;   // rows from which the backward pass takes 4

template <typename T, int W, int NV>
hipError_t run_norm(const NormArgs& g, hipStream_t s) {
  hipLaunchKernelGGL((norm_kernel<T, W, NV>), dim3(row_grid((g.T * W + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

template <typename T>
hipError_t norm(const NormArgs& g, hipStream_t s) {
  const int pieces = g.d / Act<T>::kPer16B;
  const int one = pieces_per_lane(pieces, 64), four = pieces_per_lane(pieces, 256);
  if (one && one <= kWavePieces)
    return one == 1 ? run_norm<T, 1, 1>(g, s) : run_norm<T, 1, 2>(g, s);
  switch (four) {
    case 1: return run_norm<T, kWaves, 1>(g, s);
    case 2: return run_norm<T, kWaves, 2>(g, s);
    case 4: return run_norm<T, kWaves, 4>(g, s);
    case 8: return run_norm<T, kWaves, 8>(g, s);
  }
  hipLaunchKernelGGL((norm_long_kernel<T>), dim3(row_grid(g.T)), dim3(kThreads), 0, s,
                     g);
  return hipGetLastError();
}

template <typename T, int W, int NV>
hipError_t run_norm_bwd(const NormBwdArgs& a, int parts, hipStream_t s) {
  hipLaunchKernelGGL((norm_bwd_kernel<T, W, NV>), dim3(parts), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_bwd(const NormBwdArgs& a, int parts, hipStream_t s) {
  const int pieces = a.d / Act<T>::kPer16B;
  const int one = pieces_per_lane(pieces, 64), four = pieces_per_lane(pieces, 256);
  if (one && one <= kWavePieces)
    return one == 1 ? run_norm_bwd<T, 1, 1>(a, parts, s) : run_norm_bwd<T, 1, 2>(a, parts, s);
  if (one == 4 && a.T >= kWideWaveRows) return run_norm_bwd<T, 1, 4>(a, parts, s);
  switch (four) {
    case 1: return run_norm_bwd<T, kWaves, 1>(a, parts, s);
    case 2: return run_norm_bwd<T, kWaves, 2>(a, parts, s);
    case 4: return run_norm_bwd<T, kWaves, 4>(a, parts, s);
    case 8: return run_norm_bwd<T, kWaves, 8>(a, parts, s);
  }
  const unsigned cols = static_cast<unsigned>((pieces + kThreads - 1) / kThreads);
  hipLaunchKernelGGL((norm_dw_long_kernel<T>), dim3(parts, cols), dim3(kThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((norm_bwd_long_kernel<T>), dim3(row_grid(a.T)), dim3(kThreads),
                     0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const moe_dims& dm, const void* x, const void* res, const float* weight,
                          float eps, void* sum, void* y, void* q, uint8_t* q_scale, float* rstd,
                          hipStream_t s) {
  if (dm.T == 0) return hipSuccess;
  NormArgs g{x, res, weight, sum, y, static_cast<uint8_t*>(q), q_scale, rstd, dm.T, dm.d, eps,
             1.0 / dm.d};
  return dm.act == MOE_BF16 ? norm<bf16_t>(g, s) : norm<float>(g, s);
}

// Workgroups of the backward pass: two for each of the 256 CUs, at least 4 rows each
// (their weight gradients are read again), of rows that take a whole workgroup at
// least one: 64 rows of 4096 in bf16 10.8 -> 7.5 us; a row each also where there are
// 512 costs 12.0 -> 15.6.  At 16384 x 2048, 256 and 1024 workgroups take as long as 512
// (58, 61 and 58 us, a workgroup to a row), at 16384 x 512 longer (25, 20 and 19).
int rmsnorm_bwd_parts(const moe_dims& dm) {
  const int pieces = dm.d / (dm.act == MOE_BF16 ? 8 : 4);
  const int64_t few = pieces <= 64 * kWavePieces ? 1 : 128;
  return static_cast<int>(
      std::min(std::max((dm.T + 3) / 4, std::min(dm.T, few)), int64_t(512)));
}

hipError_t launch_rmsnorm_bwd(const moe_dims& dm, const void* dy, const void* s_in,
                              const float* weight, const float* rstd, const void* dsum, void* dx,
                              float* dweight, float* ws_part, hipStream_t s) {
  const int parts = rmsnorm_bwd_parts(dm);
  if (parts > 0) {
    const NormBwdArgs a{dy, s_in, weight, rstd, dsum, dx, ws_part, dm.T,
                        (dm.T + parts - 1) / parts, dm.d};
    const hipError_t e =
        dm.act == MOE_BF16 ? norm_bwd<bf16_t>(a, parts, s) : norm_bwd<float>(a, parts, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_dw_kernel, dim3(dm.d / 16), dim3(kThreads), 0, s, ws_part, parts, dm.d,
                     dweight);
  return hipGetLastError();
}

}  // namespace moe
