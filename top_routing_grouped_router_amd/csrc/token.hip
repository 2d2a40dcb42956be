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
// exactly), h into two in a bf16 layer (it is rounded to 16 bits rather than to
// 8 between the two products) and three in an fp32 one; each term is one more
// MFMA on the same weights.
//
// A few tokens take two launches, in which each pair reads its expert by itself
// and the second product sums a token's experts (use_direct); more take three, in
// which each expert's weights are read once for all of its tokens (up to 16 at a time).
//
// Measured, d = 2048, 64 experts of 1024, k = 6, bf16: 1 token (20 MB of weights) 13.0 us
// replayed, of which the two kernels 5.5 and 6.2: bound by latency (launch, the id,
// the weights, one after another).  16 tokens (170 MB) 44 us: 22 us for the first
// product (5.0 TB/s, the rate of a copy), 17 for the second (3.4 TB/s: each workgroup's
// 32 KB cost it a search and two batches' latencies), 5 for the combine.  Token
// operands through the caches instead of LDS: 65 us (their loads, a few lanes
// each, were most of the loads issued).
#include <algorithm>
#include <type_traits>

#include "mx.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kRows = 16;      // weight rows of a workgroup, and tokens of an MFMA
constexpr int kChunk = 128;    // k of one load per lane: four lanes of 32 to a row
constexpr int kBatch = 512;    // k of the loads in flight together: four chunks

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
// exact, the last one rounded to nearest even (three terms hold all 24 bits);
// infinities and NaNs stay in the first term alone
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
    if (p == P - 1) u += 0x7FFFu + ((u >> 16) & 1u);
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
    for (int base = 0; base < g.slots; base += 256) {
      int id[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {   // four loads in flight
        const int i = base + 64 * u + lane;
        id[u] = i < g.slots ? g.ids[i] : -1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = base + 64 * u + lane;
        const bool hit = id[u] == e;
        const uint64_t mask = __ballot(hit);
        if (hit) list[n + __popcll(mask & ((uint64_t(1) << lane) - 1))] = i;
        seen |= __ballot(hit && i < y) != 0;
        n += __popcll(mask);
      }
    }
    if (lane == 0) *s_n = g.by_slot && seen ? 0 : n;
  }
  __syncthreads();
  return *s_n;
}

// 16 bytes at a 4-byte boundary
struct __attribute__((packed, aligned(4))) Words4 {
  uint32_t v[4];
};

// The codes and scales of a batch of four chunks of 16 weight rows, NM matrices:
// lane (r, q) holds blocks q of row r.  Everything past K is zero.
template <int NM>
struct Weights {
  uint4 codes[4][NM];
  uint32_t scale[4][NM];

  // w and sc at the lane's row (and its quarter of a chunk)
  __device__ __forceinline__ void load(const uint8_t* const (&w)[NM],
                                       const uint8_t* const (&sc)[NM], int K, int batch) {
    const int q = (threadIdx.x & 63) >> 4, c0 = batch * 4, chunks = (K + kChunk - 1) / kChunk;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // K may end in half a chunk: its last two lanes of a row hold nothing
        codes[u][m] = make_uint4(0, 0, 0, 0);
        if ((c0 + u) * kChunk + q * 32 < K)
          codes[u][m] = *reinterpret_cast<const uint4*>(w[m] + (c0 + u) * (kChunk / 2));
      }
      // the scales of four chunks are one load (a load of them touches as many
      // cache lines as one of weights)
      if (c0 + 4 <= chunks) {
        const Words4 t = *reinterpret_cast<const Words4*>(sc[m] + c0 * 4);
#pragma unroll
        for (int u = 0; u < 4; ++u) scale[u][m] = t.v[u];
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          scale[u][m] =
              c0 + u < chunks ? *reinterpret_cast<const uint32_t*>(sc[m] + (c0 + u) * 4) : 0u;
      }
    }
  }
};

// acc += the batch's weights times the token operand in LDS: term p of lane r's
// token, 16-byte piece i (8 values from k = 8 i of the batch), is at(p, i)
template <int NM, int P, typename At>
__device__ __forceinline__ void multiply(const Weights<NM>& w, f32x4 (&acc)[NM], At at) {
  const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float s[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) s[m] = mx_scale((w.scale[u][m] >> (8 * q)) & 255u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 xf[P];
#pragma unroll
      for (int p = 0; p < P; ++p)
        xf[p] = __builtin_bit_cast(bf16x8, *at(p, 16 * u + 4 * q + j));
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const uint4 c = w.codes[u][m];
        const bf16x8 wf = expand(j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w, s[m]);
#pragma unroll
        for (int p = 0; p < P; ++p)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[p], acc[m], 0, 0, 0);
      }
    }
  }
}

// One 16-byte piece of a token operand, P terms of 8 values from k: x of a bf16
// layer, x of an fp32 layer cut into its terms, or the stored terms of h.  Zeros
// past K (the weights are zero there, but what lies there need not be finite).
template <typename T, int MODE, int P>
struct Piece {
  uint4 v[P < 2 ? 2 : P];

  __device__ __forceinline__ void load(const TokenArgs& g, int64_t slot, int k, int K) {
    if (k >= K) {
#pragma unroll
      for (auto& t : v) t = make_uint4(0, 0, 0, 0);
    } else if constexpr (MODE == DOWN) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        v[p] = *reinterpret_cast<const uint4*>(g.h + (int64_t(p) * g.slots + slot) * K + k);
    } else {
      const T* x = static_cast<const T*>(g.x) + slot / g.k * K + k;
      v[0] = *reinterpret_cast<const uint4*>(x);
      if constexpr (P == 3) v[1] = *reinterpret_cast<const uint4*>(x + 4);
    }
  }
  __device__ __forceinline__ void terms(uint4 (&out)[P]) const {
    if constexpr (MODE == UP && P == 3) {
      float f[8];
      bf16x8 t[P];
      unpack16(v[0], f, 0.0f);
      unpack16(v[1], f + 4, 0.0f);
      terms8<P>(f, t);
#pragma unroll
      for (int p = 0; p < P; ++p) out[p] = __builtin_bit_cast(uint4, t[p]);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p) out[p] = v[p];
    }
  }
};

// terms of the token operands: x of a bf16 layer is one, h two; three in fp32
template <typename T, int MODE>
constexpr int operand_terms() {
  return sizeof(T) == 4 ? 3 : MODE == UP ? 1 : 2;
}

// The rows of one expert's weights (UP: of W1 and of W3) times its tokens: 64
// weight rows per workgroup, 16 per wavefront, all of K; the tokens' operands
// pass through LDS in batches of 512 k, which the four wavefronts share.  Weights
// asked for a whole batch ahead, or before the table is searched, need registers that
// cost more wavefronts than the waits (29 and 30 against 22 us for the first product at
// 16 tokens; 45 us in all).  One turn at a time leaves room for a fourth workgroup on a
// CU, at 49 us (its waits are longer), and 6% less where experts have over 16 tokens.
// The second product of a bf16 layer fits four as it is (126 registers against 132:
// 44.2 us, 118 against 122 at 128 tokens); the others would spill (54).
template <typename T, int MODE>
__global__ __launch_bounds__(kThreads, MODE == DOWN && sizeof(T) == 2 ? 4 : 1) void token_kernel(TokenArgs g) {
  constexpr int NM = MODE == UP ? 2 : 1, P = operand_terms<T, MODE>();
  constexpr int PH = operand_terms<T, DOWN>();
  __shared__ int list[MOE_TOKEN_MAX_SLOTS];
  __shared__ int s_n;
  // 16-byte pieces of token r at piece ^ r: 16 tokens read at one piece hit
  // distinct banks
  __shared__ uint4 xs[P][kRows][kBatch / 8];
  int e;
  const int n = find_slots(g, list, &s_n, &e);
  if (n == 0) return;
  const int K = MODE == UP ? g.d : g.f, N = MODE == UP ? g.f : g.d;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int n0 = (blockIdx.x * kWaves + wave) * kRows;   // N is a multiple of 64
  const int64_t row = static_cast<int64_t>(e) * N + n0 + r, ld = mx_scale_ld(K);
  const uint8_t* w[NM];
  const uint8_t* sc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    w[m] = g.w[m] + row * (K / 2) + q * 16;
    sc[m] = g.scale[m] + row * ld;
  }
  const int batches = (K + kBatch - 1) / kBatch;
  constexpr int kPieces = kBatch / 8;                    // of a token and batch
  constexpr int kEach = kRows * kPieces / kThreads;      // of a lane
  for (int t0 = 0; t0 < n; t0 += kRows) {
    f32x4 acc[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) acc[m] = f32x4{};
    Piece<T, MODE, P> piece[kEach];
    auto load_x = [&](int batch) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int t = t0 + wave + i * kWaves;            // a wavefront per token
        if (t < n) piece[i].load(g, list[t], batch * kBatch + lane * 8, K);
      }
    };
    load_x(0);
    auto turn = [&](int batch) {
      Weights<NM> wt;
      wt.load(w, sc, K, batch);
      __syncthreads();                                   // the last batch has been read
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int t = wave + i * kWaves;
        if (t0 + t < n) {
          uint4 out[P];
          piece[i].terms(out);
#pragma unroll
          for (int p = 0; p < P; ++p) xs[p][t][lane ^ t] = out[p];
        }
      }
      __syncthreads();
      if (batch + 1 < batches) load_x(batch + 1);
      // the columns of tokens past the last take what lies there: a column of the
      // product depends on its own token alone, and they are not stored
      multiply<NM, P>(wt, acc, [&](int p, int i) { return &xs[p][r][i ^ r]; });
    };
    // two turns at once: the second one's weights are asked for during the first
    int batch = 0;
    for (; batch + 1 < batches; batch += 2) {
      turn(batch);
      turn(batch + 1);
    }
    if (batch < batches) turn(batch);
    // lane (r, q) holds weight rows 4 q + [0, 4) of token r
    if (t0 + r < n) {
      const int64_t to = list[t0 + r];
      if constexpr (MODE == UP) {
        bf16_t term[4][PH];
#pragma unroll
        for (int v = 0; v < 4; ++v) terms<PH>(silu_f(acc[0][v]) * acc[1][v], term[v]);
#pragma unroll
        for (int p = 0; p < PH; ++p)
          *reinterpret_cast<uint2*>(g.h + (int64_t(p) * g.slots + to) * N + n0 + 4 * q) =
              make_uint2(term[0][p] | static_cast<uint32_t>(term[1][p]) << 16,
                         term[2][p] | static_cast<uint32_t>(term[3][p]) << 16);
      } else {
        *reinterpret_cast<float4*>(g.rows + to * N + n0 + 4 * q) =
            make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
      }
    }
  }
}

// Very few pairs: a pair's expert is read for it alone (one that two tokens share
// comes from the caches the second time), so nothing is searched for and the
// second product can sum a token's slots itself.  The wavefronts split K; each
// passes its part of the token's operand through LDS of its own.
//
// This wavefront's share `part` of `parts` of K: 16 rows of NM matrices
template <typename T, int MODE, int P, int NM>
__device__ __forceinline__ void direct_rows(const TokenArgs& g, int slot, int e, int n0, int part,
                                            int parts, uint4 (*xs)[kBatch / 8], f32x4 (&acc)[NM]) {
  const int K = MODE == UP ? g.d : g.f, N = MODE == UP ? g.f : g.d;
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(e) * N + n0 + (lane & 15), ld = mx_scale_ld(K);
  const uint8_t* w[NM];
  const uint8_t* sc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    w[m] = g.w[m] + row * (K / 2) + (lane >> 4) * 16;
    sc[m] = g.scale[m] + row * ld;
  }
  const int batches = (K + kBatch - 1) / kBatch;
  for (int batch = part; batch < batches; batch += parts) {
    Weights<NM> wt;
    Piece<T, MODE, P> piece;
    uint4 out[P];
    wt.load(w, sc, K, batch);
    piece.load(g, slot, batch * kBatch + lane * 8, K);
    piece.terms(out);
#pragma unroll
    for (int p = 0; p < P; ++p) xs[p][lane] = out[p];
    multiply<NM, P>(wt, acc, [&](int p, int i) { return &xs[p][i]; });   // one token: 16 like columns
  }
}

// 16 rows of W1 and of W3 times one pair's token
template <typename T>
__global__ __launch_bounds__(kThreads) void token_up_kernel(TokenArgs g) {
  constexpr int P = operand_terms<T, UP>(), PH = operand_terms<T, DOWN>();
  __shared__ uint4 xs[kWaves][P][kBatch / 8];
  __shared__ float part[kWaves][2][kRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int slot = blockIdx.y, n0 = blockIdx.x * kRows;
  const int e = g.ids[slot];
  if (e < 0 || e >= g.E) return;
  f32x4 acc[2] = {};
  direct_rows<T, UP, P, 2>(g, slot, e, n0, wave, kWaves, xs[wave], acc);
  if ((lane & 15) == 0) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][m][(lane >> 4) * 4 + v] = acc[m][v];
  }
  __syncthreads();
  if (threadIdx.x < kRows) {
    float sum[2] = {};
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      sum[0] += part[v][0][threadIdx.x];
      sum[1] += part[v][1][threadIdx.x];
    }
    bf16_t term[PH];
    terms<PH>(silu_f(sum[0]) * sum[1], term);
#pragma unroll
    for (int p = 0; p < PH; ++p)
      g.h[(static_cast<int64_t>(p) * g.slots + slot) * g.f + n0 + threadIdx.x] = term[p];
  }
}

// 16 columns of one token: kw wavefronts along f for each of its k slots
template <typename T>
__global__ __launch_bounds__(1024) void token_down_kernel(TokenArgs g, int kw) {
  constexpr int P = operand_terms<T, DOWN>();
  __shared__ uint4 xs[16][P][kBatch / 8];
  __shared__ float part[16][kRows];   // [slot * kw + share][column]
  __shared__ float s_gate[16];
  __shared__ int s_valid[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.y;
  const int n0 = blockIdx.x * kRows;
  const int slot = static_cast<int>(t) * g.k + wave / kw;
  const int e = g.ids[slot];
  if (lane == 0) {
    s_gate[wave] = g.gate[slot];
    s_valid[wave] = e >= 0 && e < g.E;
  }
  if (e >= 0 && e < g.E) {   // the wavefront's
    f32x4 acc[1] = {};
    direct_rows<T, DOWN, P, 1>(g, slot, e, n0, wave % kw, kw, xs[wave], acc);
    if ((lane & 15) == 0) {
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][(lane >> 4) * 4 + v] = acc[0][v];
    }
  }
  __syncthreads();
  if (threadIdx.x < kRows) {
    float y = 0.0f;
    for (int s = 0; s < g.k; ++s) {
      if (!s_valid[s * kw]) continue;
      float v = 0.0f;
      for (int u = 0; u < kw; ++u) v += part[s * kw + u][threadIdx.x];
      y += s_gate[s * kw] * v;
    }
    static_cast<T*>(g.y)[t * g.d + n0 + threadIdx.x] = Act<T>::from_f32(y);
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
  for (int j0 = 0; j0 < g.k; j0 += 8) {
    int e[8];
    float gate[8];
    float4 row[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {   // eight slots' loads in flight (the last one again past the end)
      const int64_t slot = t * g.k + min(j0 + u, g.k - 1);
      e[u] = g.ids[slot];
      gate[u] = g.gate[slot];
      row[u] = *reinterpret_cast<const float4*>(g.rows + slot * g.d + c);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (j0 + u >= g.k || e[u] < 0 || e[u] >= g.E) continue;   // its row was not written
      v[0] += gate[u] * row[u].x;
      v[1] += gate[u] * row[u].y;
      v[2] += gate[u] * row[u].z;
      v[3] += gate[u] * row[u].w;
    }
  }
  T* y = static_cast<T*>(g.y) + t * g.d + c;
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
  else
    *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
}

template <typename T, int MODE>
hipError_t run_rows(const TokenArgs& g, int N, unsigned ny, hipStream_t s) {
  hipLaunchKernelGGL((token_kernel<T, MODE>), dim3(N / (kRows * kWaves), ny), dim3(kThreads), 0, s,
                     g);
  return hipGetLastError();
}

// Each pair reads its expert by itself: up to 8 tokens, while experts that several pairs
// share are not read too often (what more than one read of them costs grows with d f,
// what two launches and no search save with d).  us of the call, so / with the search
// of the table, replayed: d = 2048, f = 1024, 64 experts, k = 6: 1 token 13.0 / 20.8, 8
// tokens 36.2 / 38.5, 12 tokens 49.5 / 45.0; 4 experts, k = 4: 4 tokens 18.0 / 21.5, 6
// tokens 22.8 / 21.9, 8 tokens 27.7 / 23.0; f = 2048, 8 experts, k = 2: 6 tokens 22.3 /
// 25.3, 8 tokens 27.2 / 25.9; d = 1024, f = 512, 16 experts, k = 16: 2 tokens 14.3 / 16.5,
// 4 tokens 17.6 / 16.7, 8 tokens 26.4 / 18.4; f = 1024, k = 8: 3 tokens 15.6 / 17.4, 4
// tokens 17.1 / 17.9 (searched), 6 tokens 23.4 / 18.6; d = 768, 16 experts of 512, k = 2:
// 8 tokens 10.9 / 14.2, 24 tokens 20.1 / 16.5.
bool use_direct(const moe_dims& dm) {
  const int64_t R = dm.T * dm.k;
  return dm.T <= 8 && (R - std::min<int64_t>(R, dm.E)) * dm.f < 16384;
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
  const bool bf = dm.act == MOE_BF16;
  if (use_direct(dm)) {
    const dim3 up(dm.f / kRows, g.slots);
    if (bf) hipLaunchKernelGGL((token_up_kernel<bf16_t>), up, dim3(kThreads), 0, s, g);
    else hipLaunchKernelGGL((token_up_kernel<float>), up, dim3(kThreads), 0, s, g);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    g.w[0] = static_cast<const uint8_t*>(w2);
    g.scale[0] = w2_scale;
    const int kw = 16 / dm.k;
    const dim3 down(dm.d / kRows, static_cast<unsigned>(dm.T)), block(64 * kw * dm.k);
    if (bf) hipLaunchKernelGGL((token_down_kernel<bf16_t>), down, block, 0, s, g, kw);
    else hipLaunchKernelGGL((token_down_kernel<float>), down, block, 0, s, g, kw);
    return hipGetLastError();
  }
  hipError_t err = bf ? run_rows<bf16_t, UP>(g, dm.f, ny, s) : run_rows<float, UP>(g, dm.f, ny, s);
  if (err != hipSuccess) return err;
  g.w[0] = static_cast<const uint8_t*>(w2);
  g.scale[0] = w2_scale;
  err = bf ? run_rows<bf16_t, DOWN>(g, dm.d, ny, s) : run_rows<float, DOWN>(g, dm.d, ny, s);
  if (err != hipSuccess) return err;
  const dim3 all((dm.d / 4 + kThreads - 1) / kThreads, static_cast<unsigned>(dm.T));
  if (bf) hipLaunchKernelGGL((token_combine_kernel<bf16_t>), all, dim3(kThreads), 0, s, g);
  else hipLaunchKernelGGL((token_combine_kernel<float>), all, dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace moe
