// The experts' products in low precision: rows in 8 bits (e4m3) against weights
// in 4 bits (e2m1), both in blocks of 32 with power-of-two scales (mx.h), for
// prompts: every expert's rows together, of any count.
//
//   UP    a = x W1^T, b = x W3^T, h = silu(a) b, h to 8 bits in the epilogue
//   DOWN  y_perm = h W2^T
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both formats and both scales, so
// nothing is expanded on the way: the tiles stay in 8 and 4 bits in LDS.  With
// one 8-bit operand it runs at the 8-bit rate, twice that of bf16.  On random
// operands from registers the 16x16x128 form reaches 4.2 PFLOP/s and 32x32x64 3.5
// (power: both reach 4.7-5.0 on zeros), so the smaller one is used.
//
//  * Within a block of 32 the instruction aligns the products to the largest and
//    drops what lies below 2^-13 of its power of two; blocks join in fp32.  That is
//    its arithmetic, taken for its rate: products in bf16, exact for these operands,
//    run at half of it.  It moves some h across an e4m3 tie: both products of 16384
//    tokens end 0.00177 from 64-bit sums (in norm, with h's own rounding), fp32
//    sums 0.00166.
//  * The weights are the first MFMA operand, so a lane holds columns of one row;
//    which weight rows its fragments take is chosen so that they lie side by
//    side (frag_col): an h block is four lanes, and outputs go from registers to
//    HBM in 8- and 16-byte pieces.  fp32 a, b and h are rounded once, to e4m3.
//  * An 8-bit operand's lane holds k = 16 q + [0, 16) and 64 + 16 q + [0, 16) of a
//    128-wide step (q = lane / 16), a 4-bit one k = 32 q + [0, 32); the scale of
//    block q comes from lane group q in both.
//  * K steps of 128: a row is 128 bytes of A, 64 of B and one word of scales.
//    A ring of stages is filled by buffer loads straight into LDS; the 16-byte
//    chunks are XOR-swizzled through the loads' global addresses, so that the 16
//    rows of a fragment read at one chunk hit distinct banks.
//  * Rows past the expert's end, columns past the matrix and the half step at
//    the end of a K that is no multiple of 128 read zeros through the buffer
//    bounds; their scales are clamped into range (a scale of row m or column n
//    reaches only outputs of that row or column).
//  * One workgroup computes an output in a fixed k order: the results are
//    bitwise reproducible.
//
// Measured at 98304 rows, d = 2048, 64 experts of 1024 (UP and DOWN together,
// 1.24 TFLOP): one tile per workgroup 709 us; the persistent stream of tiles 650;
// fills spread between the MFMAs instead of all behind the barrier 612; without the
// MFMAs of wavefronts past a tile's rows 608; DOWN by wavefronts of 128 x 128, 577 to
// 592 (by themselves 354 and 232, with fp32 outputs 306).  The MFMAs alone are 257 us at 2.4 GHz and about 300
// at the clock that random data leaves.  What the rest is, by leaving out parts of the
// loop: DOWN's 402 MB of stores cost it 75 us, UP's epilogue (the exponential and
// reciprocal of silu, at a quarter of the vector rate, while the matrix cores idle)
// 45, all fills 20 to 40 a product, barriers 10 to 25.  Two workgroups to a CU with
// 128 x 256 tiles hide the epilogues but fill a third more: 664.  An epilogue spread
// over the next tile's first step, fills sent ahead of the stores, stores past the
// caches' retention and starts staggered over the CUs change nothing or lose.
#include <algorithm>
#include <type_traits>

#include "mx.h"
#include "tiles.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

enum Mode { UP = 0, DOWN = 1 };

constexpr uint32_t kOutOfRange = 0x80000000u;   // above every resource size (< 2^31)
constexpr int kStep = 128;                      // k of a stage

struct MxArgs {
  const uint8_t* a;         // [rows, K] e4m3
  const uint8_t* a_scale;   // [rows, mx_scale_ld(K)]
  const int32_t* x_rows;    // UP: row p of the expert rows is a[x_rows[p]]; NULL: a[p]
  const int32_t* offsets;
  const uint8_t* w0;        // [E, N, K / 2] e2m1: W1 or W2
  const uint8_t* w0_scale;  // [E, N, mx_scale_ld(K)]
  const uint8_t* w1;        // UP: W3
  const uint8_t* w1_scale;
  void* out;                // UP: [R, N] e4m3; DOWN: [R, N] act
  uint8_t* out_scale;       // UP: [R, mx_scale_ld(N)]
  int64_t x_tokens;         // rows of a behind x_rows
  int K, N, E, n_tiles_n;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* base, int nbytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, nbytes, 0x00020000);
}
// Fills of LDS by buffer loads, 16 or 4 bytes a lane, one lane after another from
// `lds`.  In assembly, since the compiler would hold every later LDS read back
// for all of them; the waits are ours (wait_vm).  They return nothing to
// registers.
__device__ __forceinline__ void dma16(i32x4 r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(r) : "m0");
}
__device__ __forceinline__ void dma4(i32x4 r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(r) : "m0");
}
// resource words of [p, p + nbytes), p and nbytes the same in every lane
__device__ __forceinline__ i32x4 words(const uint8_t* p, int nbytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return i32x4{__builtin_amdgcn_readfirstlane(static_cast<int>(v)),
               __builtin_amdgcn_readfirstlane(static_cast<int>((v >> 32) & 0xFFFF)),
               __builtin_amdgcn_readfirstlane(nbytes), 0x00020000};
}
__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p)));
}
// a pointer that is the same in every lane, in scalar registers
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}
// s_waitcnt with vmcnt = N (N < 64: bits 3-0 and 15-14), expcnt and lgkmcnt left free
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// Tile configurations: WM x WN wavefronts of FM x FN fragments of 16 x 16, a ring
// of NST stages, PER_CU workgroups resident on a CU.
template <int FM_, int FN_, int WM_, int WN_, int NST_, int PER_CU_>
struct Tile {
  static constexpr int FM = FM_, FN = FN_, WM = WM_, WN = WN_, NST = NST_, PER_CU = PER_CU_;
  static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int kA = BM * kStep, kB = BN * kStep / 2, kS = (BM + BN) * 4;
  static constexpr int kStage = kA + kB + kS;
  static constexpr int PA = BM / 8 / NW;                        // fills per wavefront and stage:
  static constexpr int PB = BN / 16 / NW;                       // 1 KB of A, of B,
  static constexpr int PS = ((BM + BN) / 64 + NW - 1) / NW;     // and 64 words of scales
  static constexpr int kPer = PA + PB + PS;
  static_assert(BM % (8 * NW) == 0 && BN % (16 * NW) == 0 && (BM + BN) % 64 == 0, "whole fills");
  static_assert(FM % FN == 0, "a ring of FN row fragments");
  static_assert(NST >= 3, "a stage on its way while the next one is waited for");
};
typedef Tile<8, 4, 2, 4, 3, 1> Big;     // 256 x 256, wavefronts of 128 x 64
typedef Tile<8, 8, 2, 2, 3, 1> Wide;    // 256 x 256, wavefronts of 128 x 128
typedef Tile<4, 4, 1, 4, 3, 2> Small;   // 64 x 256

// The accumulators of a row fragment stand in registers here, in order with what is
// volatile around: 256 of them in the accumulation registers, fewer in the others.
template <int FN>
__device__ __forceinline__ void pin(f32x4 (&acc)[FN]) {
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    if constexpr (FN > 4) asm volatile("" : "+a"(acc[j]));
    else asm volatile("" : "+v"(acc[j]));
  }
}

// stores of a wavefront for one tile (store_tile)
template <int MODE, typename C, typename OUT>
constexpr int tile_stores() {
  return MODE == UP ? 2 * C::FM : C::FM * C::FN * static_cast<int>(sizeof(OUT)) / 4;
}

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t r, uint32_t voff, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, static_cast<int>(voff), 0, 0);
}

// largest of a value over the four lanes that share lane % 16
__device__ __forceinline__ uint32_t max_over_groups(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// Which weight row of a wavefront's columns lane r of column fragment j holds: chosen
// so that a lane's outputs of two fragments lie side by side, 8 columns, and those of
// its four lane groups too (UP: two fragments of a and the same of b; DOWN: 64 columns).
__device__ __forceinline__ int frag_col(int r, int j) {
  return 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3);
}
// chunk swizzle of weight row n: distinct for the four runs of a fragment
__device__ __forceinline__ int w_key(int n) { return (n >> 3) & 3; }

// The tile's outputs, from registers: lane (r, q) holds row r of each row
// fragment, and of the wavefront's columns 8 q + [0, 8), DOWN also 32 + 8 q + [0, 8).
// Rows and columns out of range are dropped by the buffer bounds, so every
// wavefront issues the same number of stores, which the fill counts allow for.
template <int MODE, typename C, typename OUT>
__device__ __forceinline__ void store_tile(const MxArgs& g, f32x4 (&acc)[C::FM][C::FN],
                                           int m0, int rows, int n0) {
  constexpr int FN = C::FN;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));   // nothing of this is kept through the K loop
  const int r = lane & 15, q = lane >> 4;
  const int N = g.N;
  const auto out = rsrc(static_cast<uint8_t*>(g.out) + static_cast<int64_t>(m0) * N * sizeof(OUT),
                        static_cast<int>(rows * N * sizeof(OUT)));
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    __builtin_amdgcn_sched_barrier(0);   // one row fragment's temporaries at a time
    pin<FN>(acc[i]);
    const int row = wm * 16 * C::FM + i * 16 + r;
    if constexpr (MODE == UP) {
      static_assert(FN == 4, "a block of h from two fragments of a and two of b");
      float h[8];
      uint32_t amax = 0;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        h[v] = silu_f(acc[i][v / 4][v % 4]) * acc[i][2 + v / 4][v % 4];
        amax = max(amax, abs_bits(h[v]));
      }
      const uint32_t s = mx_scale_byte<kE4M3>(max_over_groups(amax));
      const float inv = mx_inverse(s);
      const u32x2 packed = {pack_e4m3(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv),
                            pack_e4m3(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv)};
      const int n = n0 + wn * 32, ldn = mx_scale_ld(N);
      __builtin_amdgcn_raw_buffer_store_b64(
          packed, out,
          static_cast<int>(row < rows && n < N ? static_cast<uint32_t>(row) * N + n + q * 8
                                               : kOutOfRange), 0, 0);
      // a tile's columns are whole words of scales; columns past N pad the last
      const auto sc = rsrc(g.out_scale + static_cast<int64_t>(m0) * ldn, rows * ldn);
      __builtin_amdgcn_raw_buffer_store_b8(
          static_cast<uint8_t>(n < N ? s : 0), sc,
          static_cast<int>(row < rows && q == 0 && n / 32 < ldn
                               ? static_cast<uint32_t>(row) * ldn + n / 32 : kOutOfRange), 0, 0);
    } else {
#pragma unroll
      for (int b = 0; b < FN / 4; ++b) {   // 64 columns
        const int n = n0 + wn * 16 * FN + 64 * b;
        const uint32_t at = (static_cast<uint32_t>(row) * N + n + q * 8) * sizeof(OUT);
        const bool in = row < rows && n < N;
        const f32x4* a = acc[i] + 4 * b;
        if constexpr (sizeof(OUT) == 2) {
#pragma unroll
          for (int j = 0; j < 4; j += 2)
            store16(out, in ? at + frag_col(0, j) * 2 : kOutOfRange,
                    u32x4{bf16x2_rne(a[j][0], a[j][1]), bf16x2_rne(a[j][2], a[j][3]),
                          bf16x2_rne(a[j + 1][0], a[j + 1][1]),
                          bf16x2_rne(a[j + 1][2], a[j + 1][3])});
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            store16(out, in ? at + frag_col(0, j) * 4 : kOutOfRange,
                    __builtin_bit_cast(u32x4, a[j]));
        }
      }
    }
  }
}

// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, typename F>
__device__ __forceinline__ void for_each_place(F&& f) {
  if constexpr (N > 1) for_each_place<N - 1>(f);
  if constexpr (N > 0) f(std::integral_constant<int, N - 1>{});
}

// Persistent: a workgroup runs its list of tiles (build_row_sched) as one stream
// of K steps, so the fills of a tile's first steps are on their way while the
// last one is multiplied and stored.
template <int MODE, typename C, typename OUT>
__global__ __launch_bounds__(C::NT, (C::PER_CU * C::NW + 3) / 4) void mx_rows_kernel(MxArgs g) {
  constexpr int FM = C::FM, FN = C::FN, NST = C::NST, BM = C::BM, BN = C::BN, NW = C::NW;
  constexpr int kRing = C::kStage * NST;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing];
  __shared__ __attribute__((aligned(16))) int4 s_desc[kMaxItems];
  __shared__ __attribute__((aligned(16))) int32_t s_rows[MODE == UP ? 2 : 1][MODE == UP ? BM : 1];
  static_assert(sizeof(RowSched) <= kRing, "the schedule is built in the ring");
  RowSched& sched = *reinterpret_cast<RowSched*>(lds);
  const int n_items = __builtin_amdgcn_readfirstlane(
      build_row_sched<BM, C::NT>(sched, g.offsets, g.E, g.n_tiles_n));
  if (n_items == 0) return;
  if (threadIdx.x < n_items) s_desc[threadIdx.x] = sched.desc[threadIdx.x];
  __syncthreads();

  const int K = g.K, N = g.N, ldk = mx_scale_ld(K);
  constexpr int kCols = MODE == UP ? BN / 2 : BN;   // output columns of a tile
  const int nk = (K + kStep - 1) / kStep;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool gather = MODE == UP && g.x_rows;
  struct Item {
    int e, m0, rows, n0;
  };
  auto item_at = [&](int it) {
    const int4 d = s_desc[it];
    Item t;
    t.e = __builtin_amdgcn_readfirstlane(d.x);
    t.m0 = __builtin_amdgcn_readfirstlane(d.y);
    t.rows = min(BM, __builtin_amdgcn_readfirstlane(d.z) - t.m0);
    t.n0 = __builtin_amdgcn_readfirstlane(d.w) * kCols;
    return t;
  };
  auto join = [&] {   // every wavefront's reads and waits so far, before what follows
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  // ---- fills: this wavefront's global offsets for the tile being filled
  uint32_t va[C::PA], vb[C::PB], vs[C::PS];
  uint32_t last_a = 0, last_b = 0;   // bit u: past K in a half step
#pragma unroll
  for (int u = 0; u < C::PA; ++u) {
    const int row = (wave * C::PA + u) * 8 + (lane >> 3);
    last_a |= (((lane & 7) ^ ((row >> 1) & 7)) >= 4 ? 1u : 0u) << u;
  }
#pragma unroll
  for (int u = 0; u < C::PB; ++u) {
    const int row = (wave * C::PB + u) * 16 + (lane >> 2);
    last_b |= (((lane & 3) ^ w_key(row)) >= 2 ? 1u : 0u) << u;
  }
  const bool second = MODE == UP && wave * C::PB * 16 >= kCols;   // this wavefront fills W3
  const uint8_t *abase = g.a, *bbase = g.w0, *sbase[C::PS];
  int abytes = 0, bbytes = 0, sbytes[C::PS], sslot[C::PS];
#pragma unroll
  for (int u = 0; u < C::PS; ++u)   // the fills past the last one repeat it
    sslot[u] = min(wave + u * NW, (BM + BN) / 64 - 1);
  int fill_item = 0, fill_kt = 0;
  const uint32_t lds_base = lds_at(lds), rows_base = lds_at(s_rows);
  // the gather table of tile `it` into its half of s_rows
  auto fetch_rows = [&](int it) {
    if constexpr (MODE == UP) {
      if (!gather || it >= n_items) return;
      const Item t = item_at(it);
      for (int p = wave; p < BM / 64; p += NW)
        dma4(words(reinterpret_cast<const uint8_t*>(g.x_rows + t.m0), t.rows * 4),
             rows_base + ((it & 1) * BM + p * 64) * 4, (p * 64 + lane) * 4);
    }
  };
  auto aim = [&](int it) {   // the offsets of tile `it`; its gather table has landed
    const Item t = item_at(it);
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));   // computed here, not kept through the K loop
    auto source = [&](int row) {
      return static_cast<uint32_t>(MODE == UP ? s_rows[it & 1][row] : row);
    };
#pragma unroll
    for (int u = 0; u < C::PA; ++u) {
      const int row = (wave * C::PA + u) * 8 + (lane >> 3);
      const int chunk = (lane & 7) ^ ((row >> 1) & 7);
      const uint32_t from = source(row) * K + chunk * 16;
      va[u] = row < t.rows ? from : kOutOfRange;
    }
#pragma unroll
    for (int u = 0; u < C::PB; ++u) {
      const int row = (wave * C::PB + u) * 16 + (lane >> 2);
      const int chunk = (lane & 3) ^ w_key(row);
      const int n = row & (kCols - 1);
      vb[u] = t.n0 + n < N ? static_cast<uint32_t>(n) * (K / 2) + chunk * 16 : kOutOfRange;
    }
    const int64_t wrow = static_cast<int64_t>(t.e) * N + t.n0;   // first weight row of the tile
    abase = uniform(gather ? g.a : g.a + static_cast<int64_t>(t.m0) * K);
    abytes = static_cast<int>(gather ? g.x_tokens * K : static_cast<int64_t>(t.rows) * K);
    bbase = uniform((second ? g.w1 : g.w0) + wrow * (K / 2));
    bbytes = min(kCols, N - t.n0) * (K / 2);
#pragma unroll
    for (int u = 0; u < C::PS; ++u) {
      const int row = sslot[u] * 64 + lane;
      if (sslot[u] * 64 < BM) {
        sbase[u] = uniform(gather ? g.a_scale : g.a_scale + static_cast<int64_t>(t.m0) * ldk);
        sbytes[u] = static_cast<int>(gather ? g.x_tokens * ldk : static_cast<int64_t>(t.rows) * ldk);
        vs[u] = source(min(row, t.rows - 1)) * ldk;
      } else {
        const int b = row - BM;
        sbase[u] = uniform((sslot[u] * 64 - BM >= kCols ? g.w1_scale : g.w0_scale) + wrow * ldk);
        sbytes[u] = min(kCols, N - t.n0) * ldk;
        vs[u] = static_cast<uint32_t>(min(b & (kCols - 1), N - 1 - t.n0)) * ldk;
      }
    }
  };
  // The u-th fill of the stream's next step, into ring slot `slot`.  The sizes that are
  // left for the step stay positive, as they must (a negative one would be read as about
  // 4 GB, with kOutOfRange inside): a tile has rows, and columns (its column tile is below
  // n_tiles_n, so n0 < N), and kt * kStep < K.
  auto fill = [&](auto which, int slot) {
    constexpr int u = decltype(which)::value;
    const uint32_t st = lds_base + slot * C::kStage;
    const int kt = fill_kt;
    const bool half = (kt + 1) * kStep > K;
    if constexpr (u < C::PA) {
      dma16(words(abase + kt * kStep, abytes - kt * kStep), st + (wave * C::PA + u) * 1024,
            half && ((last_a >> u) & 1) ? kOutOfRange : va[u]);
    } else if constexpr (u < C::PA + C::PB) {
      constexpr int n = u - C::PA;
      dma16(words(bbase + kt * (kStep / 2), bbytes - kt * (kStep / 2)),
            st + C::kA + (wave * C::PB + n) * 1024,
            half && ((last_b >> n) & 1) ? kOutOfRange : vb[n]);
    } else if constexpr (u < C::kPer) {
      constexpr int n = u - C::PA - C::PB;
      dma4(words(sbase[n] + kt * 4, sbytes[n] - kt * 4), st + C::kA + C::kB + sslot[n] * 256,
           vs[n]);
    }
  };
  // To the stream's next step.  A new tile's gather table was fetched a tile ago:
  // with NST steps to a tile it has landed.  Past the last tile the fills go on,
  // out of range (zeros, no memory read), so that the counts below stay right.
  auto advance = [&] {
    if (++fill_kt < nk) return;
    fill_kt = 0;
    if (++fill_item < n_items) {
      if (gather && nk < NST) {
        wait_vm<0>();
        join();
      }
      aim(fill_item);
      fetch_rows(fill_item + 1);
    } else {
#pragma unroll
      for (int u = 0; u < C::PA; ++u) va[u] = kOutOfRange;
#pragma unroll
      for (int u = 0; u < C::PB; ++u) vb[u] = kOutOfRange;
#pragma unroll
      for (int u = 0; u < C::PS; ++u) vs[u] = kOutOfRange;
    }
  };

  // ---- fragments
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int r = lane & 15, q = lane >> 4;
  f32x4 acc[FM][FN];
  constexpr int kFragW = MODE == UP ? FN / 2 : FN;   // column fragments of one matrix
  const int wcol = wn * 16 * kFragW + frag_col(r, 0);
  const uint32_t aoff0 = (wm * 16 * FM + r) * kStep + ((q ^ ((r >> 1) & 7)) * 16);
  const uint32_t aoff1 = (wm * 16 * FM + r) * kStep + (((4 + q) ^ ((r >> 1) & 7)) * 16);
  const uint32_t boff = C::kA + wcol * (kStep / 2) + ((q ^ w_key(wcol)) * 16);
  const uint32_t sxoff = C::kA + C::kB + (wm * 16 * FM + r) * 4;
  const uint32_t swoff = C::kA + C::kB + (BM + wcol) * 4;
  // Row fragments go through a ring of FN, read FN / 2 ahead of their MFMAs; the
  // column fragments of the next step are read beside the last row fragments.
  constexpr int P = FN / 2;   // row fragments behind a step's join
  i32x8 x[FN];
  int sx[FN];
  i32x4 w[FN], w_next[FN];
  int sw[FN], sw_next[FN];
  auto read_x = [&](uint32_t st, int i) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + st + aoff0 + i * 16 * kStep);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + st + aoff1 + i * 16 * kStep);
    x[i % FN] = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    sx[i % FN] = *reinterpret_cast<const int*>(lds + st + sxoff + i * 64);
  };
  auto read_w = [&](uint32_t st) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int row = j < kFragW ? frag_col(0, j) : kCols + frag_col(0, j - kFragW);
      w_next[j] = *reinterpret_cast<const i32x4*>(lds + st + boff + row * (kStep / 2));
      sw_next[j] = *reinterpret_cast<const int*>(lds + st + swoff + row * 4);
    }
  };
  auto take_w = [&] {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      w[j] = w_next[j];
      sw[j] = sw_next[j] >> (8 * q);   // the lane group's block
    }
  };
  auto multiply = [&](int i, auto first, auto reads) {
    const int s = sx[i % FN] >> (8 * q);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const i32x8 wf = {w[j][0], w[j][1], w[j][2], w[j][3], 0, 0, 0, 0};
      const f32x4 c = decltype(first)::value ? f32x4{} : acc[i][j];
      acc[i][j] =
          __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, x[i % FN], c, 4, 0, 0, sw[j], 0, s);
    }
    // keeps the MFMAs where they stand among the reads, waits and barriers (they
    // touch no memory, so the compiler would sink them all behind the branches)
    pin<FN>(acc[i]);
    // the matrix cores first, `reads` LDS reads behind each MFMA
    if constexpr (decltype(reads)::value > 0) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, decltype(reads)::value, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // ---- the stream
  // A step's fills go out a few at a time between its MFMAs (all at once they
  // queue behind each other while the matrix cores idle): the first P behind
  // the join that frees the slot, the others in the next step, before its join.
  constexpr int kEach = (C::kPer + FM - 1) / FM;   // fills of a place
  auto fills = [&](auto place, int slot) {
    constexpr int p = decltype(place)::value;
    fill(std::integral_constant<int, p * kEach>{}, slot);
    if constexpr (kEach > 1) fill(std::integral_constant<int, p * kEach + 1>{}, slot);
    static_assert(kEach <= 2, "fills of a place");
  };
  if constexpr (MODE == UP) {
    if (!gather)
      for (int p = tid; p < 2 * BM; p += C::NT) s_rows[p / BM][p % BM] = p % BM;
    fetch_rows(0);
    wait_vm<0>();
    join();
  }
  aim(0);
  fetch_rows(1);
  for (int s = 0; s < NST - 1; ++s) {
    for_each_place<FM>([&](auto place) { fills(place, s); });
    advance();
  }
  for_each_place<P>([&](auto place) { fills(place, NST - 1); });
  wait_vm<(NST - 2) * C::kPer + std::min(P * kEach, C::kPer)>();   // the first step's
  join();
  read_w(0);
#pragma unroll
  for (int i = 0; i < P; ++i) read_x(0, i);
  take_w();
  int slot = 0, filling = NST - 1;
  // fills and stores newer than the fills that a tile's first step waits for (a
  // larger count than the instruction holds: it waits for a little more)
  constexpr int kStored =
      std::min(63, (NST - 2) * C::kPer + tile_stores<MODE, C, OUT>());
  // One step.  Its last P row fragments run behind the join: by then it has
  // been read by all (their operands are in registers) and the next step has
  // landed for all; the step NST on is filled in its place.  `stored`: the
  // stores of the tile before are newer than the fills that are waited for.
  auto step = [&](auto first, bool stored) {
    const uint32_t st = slot * C::kStage;
    const int next = slot + 1 == NST ? 0 : slot + 1;
    const uint32_t sn = next * C::kStage;
    for_each_place<FM - P>([&](auto place) {
      constexpr int i = decltype(place)::value;
      read_x(st, i + P);
      fills(std::integral_constant<int, i + P>{}, filling);
      multiply(i, first, std::integral_constant<int, 1>{});
    });
    advance();
    if (decltype(first)::value && stored) wait_vm<kStored>();
    else wait_vm<(NST - 2) * C::kPer>();
    join();
    filling = slot;
    read_w(sn);
    for_each_place<P>([&](auto place) {
      constexpr int i = decltype(place)::value;
      // the next step's column fragments behind the first group, its row fragments
      // behind the second (all behind the first where there are two)
      if constexpr (i == (P > 2)) {
#pragma unroll
        for (int u = 0; u < P; ++u) read_x(sn, u);
      }
      fills(place, filling);
      constexpr int kReads = P > 2 ? (i < 2 ? 2 : 0) : (i < 1 ? 4 : 0);
      multiply(FM - P + i, first, std::integral_constant<int, kReads>{});
    });
    take_w();
    slot = next;
  };
  // A step of a tile without rows for this wavefront: its share of the fills (a
  // tile of 128 rows of 256 then costs 4% to 15% less; skipping single row fragments
  // breaks up the reads between the MFMAs and costs full tiles 5%).
  auto pass = [&](bool stored) {
    for_each_place<FM - P>([&](auto place) {
      fills(std::integral_constant<int, decltype(place)::value + P>{}, filling);
    });
    advance();
    if (stored) wait_vm<kStored>();
    else wait_vm<(NST - 2) * C::kPer>();
    join();
    filling = slot;
    for_each_place<P>([&](auto place) { fills(place, filling); });
    slot = slot + 1 == NST ? 0 : slot + 1;
  };
  for (int it = 0; it < n_items; ++it) {
    const Item t = item_at(it);
    if (C::WM > 1 && t.rows <= wm * 16 * FM) {
      for (int kt = 0; kt < nk; ++kt) pass(it > 0 && kt == 0);
      const uint32_t st = slot * C::kStage;
      read_w(st);
#pragma unroll
      for (int i = 0; i < P; ++i) read_x(st, i);
      take_w();
    } else {
      step(std::integral_constant<bool, true>{}, it > 0);
      for (int kt = 1; kt < nk; ++kt) step(std::integral_constant<bool, false>{}, false);
    }
    store_tile<MODE, C, OUT>(g, acc, t.m0, t.rows, t.n0);
  }
  wait_vm<0>();   // no fill may land after the workgroup's end
}

// workgroups that cover any split of the rows over the experts: an expert's last
// tile may be partial, at most one more than the full ones each
template <int MODE, typename C>
int64_t grid_tiles(const moe_dims& dm, int64_t N) {
  constexpr int kCols = MODE == UP ? C::BN / 2 : C::BN;
  const int64_t R = dm.T * dm.k;
  const int64_t row_tiles = R / C::BM + std::min<int64_t>(dm.E, R);
  return (row_tiles * ((N + kCols - 1) / kCols) + kXcd - 1) / kXcd * kXcd;
}

template <int MODE, typename C, typename OUT>
hipError_t run_rows(MxArgs g, const moe_dims& dm, hipStream_t s) {
  constexpr int kCols = MODE == UP ? C::BN / 2 : C::BN;
  g.n_tiles_n = (g.N + kCols - 1) / kCols;
  const int64_t tiles = grid_tiles<MODE, C>(dm, g.N);
  const int64_t grid = std::max(std::min(tiles, int64_t(256 * C::PER_CU)),   // what 256 CUs hold
                                (tiles + kMaxItems * kXcd - 1) / (kMaxItems * kXcd) * kXcd);
  hipLaunchKernelGGL((mx_rows_kernel<MODE, C, OUT>), dim3(static_cast<unsigned>(grid)),
                     dim3(C::NT), 0, s, g);
  return hipGetLastError();
}

// The large tile where the full ones would occupy half of the 256 CUs, the experts
// have half a tile of rows each on average, and the K loop is long enough to hide
// a tile's ends.  Both products, large against small tile, us, at d = 2048, f = 1024:
//   8 experts of 256, 512 and 1024 rows: 49 and 42, 51 and 61, 89 and 92;
//   256 experts of 32, 64, 128 and 256 rows: 253 and 232, 303 and 293, 370 and 417,
//   534 and 683;
// at d = f = 256, 16 experts of 512 and 4096 rows: 25 and 22, 47 and 40.
bool use_big(const moe_dims& dm, int64_t cols, int64_t K) {
  const int64_t R = dm.T * dm.k;
  return R / Big::BM * ((cols + Big::BN - 1) / Big::BN) >= 128 && R >= 128 * dm.E && K >= 512;
}

// The down product's large tile with four wavefronts instead of eight: 40% fewer LDS
// reads for a product, but one wavefront to a SIMD, whose stalls nothing fills.  us at
// d = 2048, four wavefronts and eight: 64 experts of 1536 rows of 1024 233 and 258;
// with the same first product, 8 experts of 2048 and 8192 rows 125 and 123, 384 and
// 397; 256 experts of 256 and 512 rows 530 and 533, 878 and 892; at d = 1024, 32 experts
// of 1024 and 4096 rows of 512 82 and 80, 237 and 246.
bool use_wide(const moe_dims& dm) {
  return dm.T * dm.k / Wide::BM * ((dm.d + Wide::BN - 1) / Wide::BN) >= 2048;
}

template <typename OUT>
hipError_t run_down(const MxArgs& g, const moe_dims& dm, hipStream_t s) {
  if (!use_big(dm, dm.d, dm.f)) return run_rows<DOWN, Small, OUT>(g, dm, s);
  if (use_wide(dm)) return run_rows<DOWN, Wide, OUT>(g, dm, s);
  return run_rows<DOWN, Big, OUT>(g, dm, s);
}

}  // namespace

// A launch holds fewer than 2^32 threads.  The large tile needs the most: up to four
// times as many of the small one share their workgroups by kMaxItems, of half the threads.
bool mx_tiles_ok(const moe_dims& dm) {
  const int64_t limit = (int64_t(1) << 32) / Big::NT;
  return grid_tiles<UP, Big>(dm, dm.f) < limit && grid_tiles<DOWN, Big>(dm, dm.d) < limit;
}

hipError_t launch_up_mx(const moe_dims& dm, const void* xq, const uint8_t* x_scale,
                        const int32_t* x_rows, const int32_t* offsets, const void* w1,
                        const uint8_t* w1_scale, const void* w3, const uint8_t* w3_scale, void* hq,
                        uint8_t* h_scale, hipStream_t s) {
  if (dm.T == 0) return hipSuccess;
  MxArgs g{};
  g.a = static_cast<const uint8_t*>(xq);
  g.a_scale = x_scale;
  g.x_rows = x_rows;
  g.offsets = offsets;
  g.w0 = static_cast<const uint8_t*>(w1);
  g.w0_scale = w1_scale;
  g.w1 = static_cast<const uint8_t*>(w3);
  g.w1_scale = w3_scale;
  g.out = hq;
  g.out_scale = h_scale;
  g.x_tokens = dm.T;
  g.K = dm.d;
  g.N = dm.f;
  g.E = dm.E;
  if (use_big(dm, 2 * static_cast<int64_t>(dm.f), dm.d)) return run_rows<UP, Big, uint8_t>(g, dm, s);
  return run_rows<UP, Small, uint8_t>(g, dm, s);
}

hipError_t launch_down_mx(const moe_dims& dm, const void* hq, const uint8_t* h_scale,
                          const int32_t* offsets, const void* w2, const uint8_t* w2_scale, void* y,
                          hipStream_t s) {
  if (dm.T == 0) return hipSuccess;
  MxArgs g{};
  g.a = static_cast<const uint8_t*>(hq);
  g.a_scale = h_scale;
  g.offsets = offsets;
  g.w0 = static_cast<const uint8_t*>(w2);
  g.w0_scale = w2_scale;
  g.out = y;
  g.K = dm.f;
  g.N = dm.d;
  g.E = dm.E;
  return dm.act == MOE_BF16 ? run_down<bf16_t>(g, dm, s) : run_down<float>(g, dm, s);
}

}  // namespace moe
