// The experts for a few tokens, straight from the router's table: products of
// single rows with 4-bit weights (e2m1 in blocks of 32, mx.h), activations in
// the layer's own type.
//
//   y[t] = sum_j gate[t, j] W2[e] (silu(W1[e] x[t]) * (W3[e] x[t])),  e = topk_idx[t, j]
//
// The weights of the chosen experts are read once each and bound the call, so
// nothing is sorted first: a workgroup finds the (token, slot) pairs of its
// expert in the table itself.  The codes become bf16 in registers (one
// conversion per two weights, the block's scale applied by it: a code times a
// power of two is exact in bf16) and go to the matrix cores with up to 16
// tokens as the other operand: the instruction costs the same for one token,
// and sums over k without a reduction across lanes.
//
// A lane loads 16 bytes, one block of 32 codes of its weight row; the j-th
// MFMA of the block takes k = 8 j + [0, 8) of it, so the token operand is read
// at the same k.  fp32 activations are cut into three bf16 terms (8 bits each,
// exactly), h into two in a bf16 layer (it is kept to 16 bits rather than
// rounded to 8 between the two products) and three in an fp32 one; each term
// is one more MFMA on the same weights.
//
// The four wavefronts of a workgroup take a quarter of K each, so that all of
// a workgroup's loads are in flight at once, and are added in a fixed order.
#include <algorithm>

#include "mx.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kRows = 16;      // weight rows of a workgroup, and tokens of an MFMA
constexpr int kChunk = 128;    // k of one load per lane: four lanes of 32 to a row

enum Mode { UP = 0, DOWN = 1 };

struct TokenArgs {
  const void* x;            // UP: [T, d] act
  const int32_t* ids;       // [T, k]
  const float* gate;        // [T, k]
  const uint8_t* w[2];      // UP: W1, W3 [E, f, d / 2]; DOWN: W2 [E, d, f / 2]
  const uint8_t* scale[2];
  bf16_t* h;                // [planes][slots, f]: terms of h
  float* rows;              // [slots, d]: W2 h of each pair
  void* y;                  // [T, d] act
  int64_t T;
  int d, E, f, k, slots;
  int by_slot;              // blockIdx.y: a slot whose expert is new in the table, or an expert
};

// bf16 terms of fp32 values: the upper 8 significant bits each, the remainders
// exact; infinities and NaNs stay in the first term alone
template <int P>
__device__ __forceinline__ void terms(float v, bf16_t* out) {
  uint32_t u = __float_as_uint(v);
  const bool odd = (u & 0x7F800000u) == 0x7F800000u;
  if (odd && (u & 0x007FFFFFu)) u = 0x7FC00000u;
  out[0] = static_cast<bf16_t>(u >> 16);
#pragma unroll
  for (int p = 1; p < P; ++p) {
    v -= __uint_as_float(u & 0xFFFF0000u);
    u = odd ? 0u : __float_as_uint(v);
    out[p] = static_cast<bf16_t>(u >> 16);
  }
}

// terms of eight fp32 values as MFMA operands
template <int P>
__device__ __forceinline__ void terms8(const float* v, bf16x8* out) {
  uint32_t w[P][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bf16_t a[P], b[P];
    terms<P>(v[2 * i], a);
    terms<P>(v[2 * i + 1], b);
#pragma unroll
    for (int p = 0; p < P; ++p)
      w[p][i] = static_cast<uint32_t>(a[p]) | (static_cast<uint32_t>(b[p]) << 16);
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
    out[p] = __builtin_bit_cast(bf16x8, make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]));
}

// eight e2m1 codes with their scale
__device__ __forceinline__ bf16x8 expand(uint32_t codes, float scale) {
  const uint4 v = make_uint4(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3)));
  return __builtin_bit_cast(bf16x8, v);
}

// The table's pairs of this workgroup's expert, in slot order, into `list`;
// returns how many (0: nothing to do here), and the expert.
__device__ __forceinline__ int find_slots(const TokenArgs& g, int* list, int* s_n, int* expert) {
  const int y = blockIdx.y;
  const int e = g.by_slot ? g.ids[y] : y;
  *expert = e;
  if (e < 0 || e >= g.E) return 0;
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int n = 0;
    bool seen = false;   // an earlier slot has this expert and takes it
    for (int base = 0; base < g.slots; base += 64) {
      const int i = base + lane;
      const bool hit = i < g.slots && g.ids[i] == e;
      const uint64_t mask = __ballot(hit);
      if (hit) list[n + __popcll(mask & ((uint64_t(1) << lane) - 1))] = i;
      seen |= __ballot(hit && i < y) != 0;
      n += __popcll(mask);
    }
    if (lane == 0) *s_n = g.by_slot && seen ? 0 : n;
  }
  __syncthreads();
  return *s_n;
}

// 16 weight rows (UP: of W1 and of W3) of one expert times its tokens.
// P: terms of the token operand.
template <typename T, int MODE, int P>
__global__ __launch_bounds__(kThreads) void token_kernel(TokenArgs g) {
  constexpr int NM = MODE == UP ? 2 : 1;
  constexpr int PH = sizeof(T) == 2 ? 2 : 3;   // terms of h
  constexpr int kBatch = P == 1 ? 4 : 2;       // chunks loaded together
  __shared__ int list[MOE_TOKEN_MAX_SLOTS];
  __shared__ int s_n;
  __shared__ float red[kWaves][NM][4][64];
  int e;
  const int n = find_slots(g, list, &s_n, &e);
  if (n == 0) return;
  const int K = MODE == UP ? g.d : g.f, N = MODE == UP ? g.f : g.d;
  const int n0 = blockIdx.x * kRows;           // N is a multiple of 64
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int ld = mx_scale_ld(K);
  const int64_t row = static_cast<int64_t>(e) * N + n0 + r;
  const uint8_t* w[NM];
  const uint8_t* sc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    w[m] = g.w[m] + row * (K / 2) + q * 16;
    sc[m] = g.scale[m] + row * ld;
  }
  const int chunks = (K + kChunk - 1) / kChunk, per = (chunks + kWaves - 1) / kWaves;
  const int c0 = wave * per, c1 = min(c0 + per, chunks);

  for (int t0 = 0; t0 < n; t0 += kRows) {
    const bool there = t0 + r < n;
    const int slot = there ? list[t0 + r] : 0;
    const int64_t token = slot / g.k;
    f32x4 acc[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) acc[m] = f32x4{};
    for (int cb = c0; cb < c1; cb += kBatch) {
      uint4 codes[kBatch][NM];
      uint32_t sw[kBatch][NM];
      uint4 xv[kBatch][4][P];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int c = cb + u, k0 = c * kChunk + q * 32;
        // K may end in half a chunk: its last two lanes of a row hold nothing
        const bool in = c < c1 && k0 < K;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          codes[u][m] = make_uint4(0, 0, 0, 0);
          sw[u][m] = 0;
          if (in) {
            codes[u][m] = *reinterpret_cast<const uint4*>(w[m] + c * (kChunk / 2));
            sw[u][m] = *reinterpret_cast<const uint32_t*>(sc[m] + c * 4);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int p = 0; p < P; ++p) {
            xv[u][j][p] = make_uint4(0, 0, 0, 0);
            if (in && there) {
              if constexpr (MODE == DOWN)
                xv[u][j][p] = *reinterpret_cast<const uint4*>(
                    g.h + (static_cast<int64_t>(p) * g.slots + slot) * K + k0 + 8 * j);
              else if constexpr (P == 1)
                xv[u][j][p] = *reinterpret_cast<const uint4*>(
                    static_cast<const bf16_t*>(g.x) + token * K + k0 + 8 * j);
              else if (p < 2)   // the eight fp32 values, cut below
                xv[u][j][p] = *reinterpret_cast<const uint4*>(
                    static_cast<const float*>(g.x) + token * K + k0 + 8 * j + 4 * p);
            }
          }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float s[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) s[m] = mx_scale((sw[u][m] >> (8 * q)) & 255u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x8 xf[P];
          if constexpr (MODE == UP && P == 3) {
            float v[8];
            unpack16(xv[u][j][0], v, 0.0f);
            unpack16(xv[u][j][1], v + 4, 0.0f);
            terms8<P>(v, xf);
          } else {
#pragma unroll
            for (int p = 0; p < P; ++p) xf[p] = __builtin_bit_cast(bf16x8, xv[u][j][p]);
          }
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            const uint32_t word = j == 0 ? codes[u][m].x : j == 1 ? codes[u][m].y
                                  : j == 2 ? codes[u][m].z : codes[u][m].w;
            const bf16x8 wf = expand(word, s[m]);
#pragma unroll
            for (int p = 0; p < P; ++p)
              acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[p], acc[m], 0, 0, 0);
          }
        }
      }
    }
    // lane (r, q) holds weight rows 4 q + [0, 4) of token r
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave][m][v][lane] = acc[m][v];
    __syncthreads();
    const int c = threadIdx.x & 15, t = threadIdx.x >> 4;
    if (t0 + t < n) {
      float sum[NM];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        sum[m] = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) sum[m] += red[v][m][c & 3][t + 16 * (c >> 2)];
      }
      const int64_t to = list[t0 + t];
      if constexpr (MODE == UP) {
        bf16_t term[PH];
        terms<PH>(silu_f(sum[0]) * sum[1], term);
#pragma unroll
        for (int p = 0; p < PH; ++p)
          g.h[(static_cast<int64_t>(p) * g.slots + to) * N + n0 + c] = term[p];
      } else {
        g.rows[to * N + n0 + c] = sum[0];
      }
    }
    __syncthreads();
  }
}

// y[t] = sum over the slots, in order, of gate * row (pairs without an expert
// have no row)
template <typename T>
__global__ __launch_bounds__(kThreads) void token_combine_kernel(TokenArgs g) {
  const int c = (blockIdx.x * kThreads + threadIdx.x) * 4;
  const int64_t t = blockIdx.y;
  if (c >= g.d) return;
  float v[4] = {};
  for (int j = 0; j < g.k; ++j) {
    const int e = g.ids[t * g.k + j];
    if (e < 0 || e >= g.E) continue;
    const float gate = g.gate[t * g.k + j];
    const float4 row = *reinterpret_cast<const float4*>(g.rows + (t * g.k + j) * g.d + c);
    v[0] += gate * row.x;
    v[1] += gate * row.y;
    v[2] += gate * row.z;
    v[3] += gate * row.w;
  }
  T* y = static_cast<T*>(g.y) + t * g.d + c;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
  else
    *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
}

int h_planes(const moe_dims& dm) { return dm.act == MOE_BF16 ? 2 : 3; }

}  // namespace

size_t token_h_elems(const moe_dims& dm) {
  return static_cast<size_t>(dm.T) * dm.k * dm.f * h_planes(dm);
}
size_t token_row_elems(const moe_dims& dm) { return static_cast<size_t>(dm.T) * dm.k * dm.d; }

hipError_t launch_token_swiglu(const moe_dims& dm, const void* x, const int32_t* idx,
                               const float* gate, const void* w1, const uint8_t* w1_scale,
                               const void* w3, const uint8_t* w3_scale, const void* w2,
                               const uint8_t* w2_scale, void* y, bf16_t* ws_h, float* ws_rows,
                               hipStream_t s) {
  if (dm.T == 0) return hipSuccess;
  TokenArgs g{};
  g.x = x;
  g.ids = idx;
  g.gate = gate;
  g.h = ws_h;
  g.rows = ws_rows;
  g.y = y;
  g.T = dm.T;
  g.d = dm.d;
  g.E = dm.E;
  g.f = dm.f;
  g.k = dm.k;
  g.slots = static_cast<int>(dm.T * dm.k);
  g.by_slot = g.slots <= dm.E;
  g.w[0] = static_cast<const uint8_t*>(w1);
  g.scale[0] = w1_scale;
  g.w[1] = static_cast<const uint8_t*>(w3);
  g.scale[1] = w3_scale;
  const unsigned ny = static_cast<unsigned>(std::min(g.slots, dm.E));
  const dim3 up(dm.f / kRows, ny), down(dm.d / kRows, ny);
  const bool bf = dm.act == MOE_BF16;
  if (bf) hipLaunchKernelGGL((token_kernel<bf16_t, UP, 1>), up, dim3(kThreads), 0, s, g);
  else hipLaunchKernelGGL((token_kernel<float, UP, 3>), up, dim3(kThreads), 0, s, g);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  g.w[0] = static_cast<const uint8_t*>(w2);
  g.scale[0] = w2_scale;
  if (bf) hipLaunchKernelGGL((token_kernel<bf16_t, DOWN, 2>), down, dim3(kThreads), 0, s, g);
  else hipLaunchKernelGGL((token_kernel<float, DOWN, 3>), down, dim3(kThreads), 0, s, g);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 all((dm.d / 4 + kThreads - 1) / kThreads, static_cast<unsigned>(dm.T));
  if (bf) hipLaunchKernelGGL((token_combine_kernel<bf16_t>), all, dim3(kThreads), 0, s, g);
  else hipLaunchKernelGGL((token_combine_kernel<float>), all, dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace moe
