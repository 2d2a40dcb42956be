// The experts' products in low precision: rows in 8 bits (e4m3) against weights
// in 4 bits (e2m1), both in blocks of 32 with power-of-two scales (mx.h), for
// prompts: every expert's rows together, of any count.
//
//   UP    a = x W1^T, b = x W3^T, h = silu(a) b, h to 8 bits in the epilogue
//   DOWN  y_perm = h W2^T
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes both formats and both scales, so
// nothing is expanded on the way: the tiles stay in 8 and 4 bits in LDS.  With
// one 8-bit operand it runs at the 8-bit rate, twice that of bf16.
//
//  * The weights are the first MFMA operand, so a lane holds 16 columns of one
//    row: the 32 columns of an h block lie in two lanes, and quantising h costs
//    one exchange between the halves of the wavefront.  fp32 a, b and h are
//    rounded once, to e4m3.
//  * An 8-bit operand's lane holds k = 16 g + [0, 16) and 32 + 16 g + [0, 16) of a
//    64-wide step (g = lane / 32), a 4-bit one k = 32 g + [0, 32); the scale of
//    block g comes from lane group g in both.
//  * K steps of 128: a row is 128 bytes of A, 64 of B and one word of scales.
//    A ring of stages is filled by buffer loads straight into LDS; the 16-byte
//    chunks are XOR-swizzled through the loads' global addresses (A by
//    (row >> 1) & 7, B by (row >> 2) & 3), so that 16 rows read at one chunk
//    hit distinct banks.
//  * Rows past the expert's end, columns past the matrix and the half step at
//    the end of a K that is no multiple of 128 read zeros through the buffer
//    bounds; their scales are clamped into range (a scale of row m or column n
//    reaches only outputs of that row or column).
//  * One workgroup computes an output in a fixed k order: the results are
//    bitwise reproducible.
#include <algorithm>

#include "mx.h"
#include "tiles.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

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
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)lds, 16, static_cast<int>(voff), 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)lds, 4, static_cast<int>(voff), 0, 0, 0);
}
// s_waitcnt with vmcnt = N (N < 64: bits 3-0 and 15-14), expcnt and lgkmcnt left free
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// Tile configurations: WM x WN wavefronts of FM x 2 fragments of 32 x 32.
template <int FM_, int WM_, int WN_, int NST_>
struct Tile {
  static constexpr int FM = FM_, WM = WM_, WN = WN_, NST = NST_;
  static constexpr int BM = 32 * FM * WM, BN = 64 * WN;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int kA = BM * kStep, kB = BN * kStep / 2, kS = (BM + BN) * 4;
  static constexpr int kStage = kA + kB + kS;
  static constexpr int PA = BM / 8 / NW;                        // fills per wavefront and stage:
  static constexpr int PB = BN / 16 / NW;                       // 1 KB of A, of B,
  static constexpr int PS = ((BM + BN) / 64 + NW - 1) / NW;     // and 64 words of scales
  static_assert(BM % (8 * NW) == 0 && BN % (16 * NW) == 0 && (BM + BN) % 64 == 0, "whole fills");
};
typedef Tile<4, 2, 4, 3> Big;     // 256 x 256
typedef Tile<2, 1, 4, 3> Small;   // 64 x 256

// the four runs of 4 columns that a lane holds of a 32-column fragment (columns
// 8 q + 4 g + [0, 4)) to 16 consecutive ones (16 g + [0, 16)): one swap between
// the wavefront's halves per word of each run
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

template <int MODE, typename C, typename OUT>
__global__ __launch_bounds__(C::NT, 1) void mx_rows_kernel(MxArgs g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kStage * C::NST];
  constexpr int FM = C::FM, NST = C::NST, BM = C::BM, BN = C::BN, NW = C::NW;
  const int flat = flat_tile();
  const int row_tile = flat / g.n_tiles_n, nt = flat - row_tile * g.n_tiles_n;
  int e, m0, mend;
  if (!find_row_tile_at<BM>(reinterpret_cast<int*>(lds), g.offsets, g.E, row_tile, &e, &m0, &mend))
    return;
  e = __builtin_amdgcn_readfirstlane(e);
  m0 = __builtin_amdgcn_readfirstlane(m0);
  mend = __builtin_amdgcn_readfirstlane(mend);
  __syncthreads();   // every lane holds them before the first fill lands there
  const int rows = min(BM, mend - m0);
  const int K = g.K, N = g.N, ldk = mx_scale_ld(K);
  constexpr int kCols = MODE == UP ? BN / 2 : BN;   // output columns of the tile
  const int n0 = nt * kCols;
  const int nk = (K + kStep - 1) / kStep;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // ---- fills: global offsets of this wavefront's lanes, and the last step's
  // where K ends in half a step
  uint32_t va[C::PA], vb[C::PB], vs[C::PS];
  uint32_t last_a = 0, last_b = 0;   // bit u: out of range in the half step
#pragma unroll
  for (int u = 0; u < C::PA; ++u) {
    const int row = (wave * C::PA + u) * 8 + (lane >> 3);
    const int chunk = (lane & 7) ^ ((row >> 1) & 7);
    const int src = MODE == UP && g.x_rows ? g.x_rows[min(m0 + row, mend - 1)] : row;
    va[u] = row < rows ? static_cast<uint32_t>(src) * K + chunk * 16 : kOutOfRange;
    last_a |= (chunk >= 4 ? 1u : 0u) << u;
  }
#pragma unroll
  for (int u = 0; u < C::PB; ++u) {
    const int row = (wave * C::PB + u) * 16 + (lane >> 2);
    const int chunk = (lane & 3) ^ ((row >> 2) & 3);
    const int n = row & (kCols - 1);
    vb[u] = n0 + n < N ? static_cast<uint32_t>(n) * (K / 2) + chunk * 16 : kOutOfRange;
    last_b |= (chunk >= 2 ? 1u : 0u) << u;
  }
  const int64_t wrow = static_cast<int64_t>(e) * N + n0;   // first weight row of the tile
  const bool gather = MODE == UP && g.x_rows;
  const uint8_t* abase = gather ? g.a : g.a + static_cast<int64_t>(m0) * K;
  const int abytes = static_cast<int>(gather ? g.x_tokens * K : static_cast<int64_t>(rows) * K);
  const bool second = MODE == UP && wave * C::PB * 16 >= kCols;   // this wavefront fills W3
  const uint8_t* bbase = (second ? g.w1 : g.w0) + wrow * (K / 2);
  const int bbytes = min(kCols, N - n0) * (K / 2);
  const uint8_t* sbase[C::PS];
  int sbytes[C::PS], sslot[C::PS];
#pragma unroll
  for (int u = 0; u < C::PS; ++u) {
    // the fills past the last one repeat it (every wavefront issues as many)
    sslot[u] = min(wave + u * NW, (BM + BN) / 64 - 1);
    const int row = sslot[u] * 64 + lane;
    if (sslot[u] * 64 < BM) {
      const int at = min(m0 + row, mend - 1);
      const int src = gather ? g.x_rows[at] : at - m0;
      sbase[u] = gather ? g.a_scale : g.a_scale + static_cast<int64_t>(m0) * ldk;
      sbytes[u] = static_cast<int>(gather ? g.x_tokens * ldk : static_cast<int64_t>(rows) * ldk);
      vs[u] = static_cast<uint32_t>(src) * ldk;
    } else {
      const int b = row - BM, n = min(b & (kCols - 1), N - 1 - n0);
      sbase[u] = (sslot[u] * 64 - BM >= kCols ? g.w1_scale : g.w0_scale) + wrow * ldk;
      sbytes[u] = min(kCols, N - n0) * ldk;
      vs[u] = static_cast<uint32_t>(n) * ldk;
    }
  }
  auto issue = [&](int kt, int slot) {
    uint8_t* st = lds + slot * C::kStage;
    const bool half = (kt + 1) * kStep > K;
    const auto ra = rsrc(abase + kt * kStep, abytes - kt * kStep);
#pragma unroll
    for (int u = 0; u < C::PA; ++u)
      dma16(ra, st + (wave * C::PA + u) * 1024,
            half && ((last_a >> u) & 1) ? kOutOfRange : va[u]);
    const auto rb = rsrc(bbase + kt * (kStep / 2), bbytes - kt * (kStep / 2));
#pragma unroll
    for (int u = 0; u < C::PB; ++u)
      dma16(rb, st + C::kA + (wave * C::PB + u) * 1024,
            half && ((last_b >> u) & 1) ? kOutOfRange : vb[u]);
#pragma unroll
    for (int u = 0; u < C::PS; ++u)
      dma4(rsrc(sbase[u] + kt * 4, sbytes[u] - kt * 4), st + C::kA + C::kB + sslot[u] * 256, vs[u]);
  };

  // ---- fragments
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int r = lane & 31, gq = lane >> 5;
  f32x16 acc[FM][2];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  uint32_t aoff[4], boff[2];   // byte offsets of the lane's chunks in a stage
#pragma unroll
  for (int c = 0; c < 4; ++c)
    aoff[c] = (wm * 32 * FM + r) * kStep + (((2 * c + gq) ^ ((r >> 1) & 7)) * 16);
#pragma unroll
  for (int c = 0; c < 2; ++c)
    boff[c] = C::kA + (wn * 32 + r) * (kStep / 2) + (((2 * c + gq) ^ ((r >> 2) & 3)) * 16);
  const uint32_t soff = C::kA + C::kB;

#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (s < nk) issue(s, s);
  constexpr int kPer = C::PA + C::PB + C::PS;
  int slot = 0;
  for (int kt = 0; kt < nk; ++kt) {
    // stage kt has landed when at most the fills of the later stages are out
    if (kt + NST - 2 < nk) wait_vm<(NST - 2) * kPer>();
    else wait_vm<0>();
    // landed for all, and stage kt - 1 read by all (its reads are waited for
    // here, wherever the compiler has put the MFMAs that use them)
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (kt + NST - 1 < nk) issue(kt + NST - 1, slot == 0 ? NST - 1 : slot - 1);
    const uint8_t* st = lds + slot * C::kStage;
    int sx[FM], sw[2];
#pragma unroll
    for (int i = 0; i < FM; ++i)
      sx[i] = *reinterpret_cast<const int*>(st + soff + (wm * 32 * FM + i * 32 + r) * 4) >> (8 * gq);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      sw[j] = *reinterpret_cast<const int*>(st + soff + (BM + j * (BN / 2) + wn * 32 + r) * 4) >>
              (8 * gq);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      i32x8 wf[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const i32x4 b =
            *reinterpret_cast<const i32x4*>(st + boff[kk] + j * (BN / 2) * (kStep / 2));
        wf[j] = i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(st + aoff[2 * kk] + i * 32 * kStep);
        const i32x4 hi = *reinterpret_cast<const i32x4*>(st + aoff[2 * kk + 1] + i * 32 * kStep);
        const i32x8 xf = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (kk == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[j], xf, acc[i][j], 4, 0,
                                                                        0, sw[j], 0, sx[i]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[j], xf, acc[i][j], 4, 0,
                                                                        2, sw[j], 2, sx[i]);
        }
      }
    }
    slot = slot + 1 == NST ? 0 : slot + 1;
  }

  // ---- epilogue, from registers: lane (r, gq) holds columns 8 q + 4 gq + [0, 4)
  // of row r of each fragment
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = wm * 32 * FM + i * 32 + r;
    const int64_t m = m0 + row;
    if constexpr (MODE == UP) {
      float h[16];
      uint32_t amax = 0;
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        h[v] = silu_f(acc[i][0][v]) * acc[i][1][v];
        amax = max(amax, abs_bits(h[v]));
      }
      uint32_t other = amax;
      swap_halves(amax, other);
      const uint32_t s = mx_scale_byte<kE4M3>(max(amax, other));
      const float inv = mx_inverse(s);
      uint32_t q[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        q[c] = pack_e4m3(h[4 * c] * inv, h[4 * c + 1] * inv, h[4 * c + 2] * inv,
                         h[4 * c + 3] * inv);
      swap_halves(q[0], q[2]);
      swap_halves(q[1], q[3]);
      const int n = n0 + wn * 32, ldn = mx_scale_ld(N);
      if (row < rows) {
        if (n < N)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.out) + m * N + n + gq * 16) =
              make_uint4(q[0], q[2], q[1], q[3]);
        // a tile's 128 columns are one word of scales; columns past N pad it
        if (gq == 0 && n / 32 < ldn)
          g.out_scale[m * ldn + n / 32] = static_cast<uint8_t>(n < N ? s : 0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = n0 + j * (BN / 2) + wn * 32;
        OUT* out = static_cast<OUT*>(g.out) + m * N + n + gq * 16;
        if constexpr (sizeof(OUT) == 2) {
          uint32_t lo[4], hi[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            lo[c] = bf16x2_rne(acc[i][j][4 * c], acc[i][j][4 * c + 1]);
            hi[c] = bf16x2_rne(acc[i][j][4 * c + 2], acc[i][j][4 * c + 3]);
          }
          swap_halves(lo[0], lo[2]);
          swap_halves(hi[0], hi[2]);
          swap_halves(lo[1], lo[3]);
          swap_halves(hi[1], hi[3]);
          if (row < rows && n < N) {
            reinterpret_cast<uint4*>(out)[0] = make_uint4(lo[0], hi[0], lo[2], hi[2]);
            reinterpret_cast<uint4*>(out)[1] = make_uint4(lo[1], hi[1], lo[3], hi[3]);
          }
        } else {
          uint32_t t[4][4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) t[c][v] = __float_as_uint(acc[i][j][4 * c + v]);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            swap_halves(t[0][v], t[2][v]);
            swap_halves(t[1][v], t[3][v]);
          }
          if (row < rows && n < N) {
            const int order[4] = {0, 2, 1, 3};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              reinterpret_cast<uint4*>(out)[c] =
                  make_uint4(t[order[c]][0], t[order[c]][1], t[order[c]][2], t[order[c]][3]);
          }
        }
      }
    }
  }
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
  hipLaunchKernelGGL((mx_rows_kernel<MODE, C, OUT>), dim3(static_cast<unsigned>(tiles)),
                     dim3(C::NT), 0, s, g);
  return hipGetLastError();
}

// The large tile where there are full ones for most of the 256 CUs; else the
// small one, whose workgroups are four times as many.
bool use_big(const moe_dims& dm, int64_t cols) {
  return dm.T * dm.k / Big::BM * ((cols + Big::BN - 1) / Big::BN) >= 256;
}

}  // namespace

// a launch holds fewer than 2^32 threads (dims this large take the big tile)
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
  if (use_big(dm, 2 * static_cast<int64_t>(dm.f))) return run_rows<UP, Big, uint8_t>(g, dm, s);
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
  const bool big = use_big(dm, dm.d);
  if (dm.act == MOE_BF16)
    return big ? run_rows<DOWN, Big, bf16_t>(g, dm, s) : run_rows<DOWN, Small, bf16_t>(g, dm, s);
  return big ? run_rows<DOWN, Big, float>(g, dm, s) : run_rows<DOWN, Small, float>(g, dm, s);
}

}  // namespace moe
