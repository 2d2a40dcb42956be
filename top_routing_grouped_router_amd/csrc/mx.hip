// Rows to and from the block-scaled formats of mx.h (OCP Microscaling Formats:
// e4m3 and e2m1 elements, one power-of-two scale per 32).
//
// Both directions read and write each value once and are bound by HBM.  A lane
// holds 16 bytes of the act tensor (8 bf16 or 4 fp32 values); a block's largest
// value comes from 4 or 8 neighbouring lanes by vector instructions (from_lane), so
// loads and stores stay coalesced (a lane per block would load at a 64- or 128-byte
// stride).
// Lanes take 4 pieces each, a workgroup apart, to have 4 loads in flight: with 1, 2, 4
// and 8 the quantisation of 134M bf16 values to e2m1 (340 MB) takes 58, 53, 53 and 54
// us (6.4 TB/s), the way back 47, 47, 48 and 49 (7.1 TB/s: codes just written are read
// from the caches; a large copy reaches 5.2).
#include "mx.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;

template <typename T, int FMT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const T* src, uint8_t* q,
                                                               uint8_t* scale, int64_t pieces,
                                                               int cols) {
  constexpr int N = Act<T>::kPer16B;
  constexpr int kLanes = 32 / N;   // lanes of a block
  const int per_row = cols / N, ld = mx_scale_ld(cols);
  const bool whole = cols % 128 == 0;   // no padding: scales lie one after another
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kPieces) + threadIdx.x;
  uint4 raw[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t p = first + u * kThreads;
    raw[u] = p < pieces ? ld_nt16(reinterpret_cast<const uint4*>(src) + p) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t p = first + u * kThreads;
    if (p >= pieces) break;   // whole blocks: a row is a multiple of 64 values
    float v[N];
    unpack16(raw[u], v, T{});
    const uint32_t s =
        mx_store<FMT, N>(v, q + p * (FMT == kE4M3 ? N : N / 2));
    if (p % kLanes == 0) {
      if (whole) {
        scale[p / kLanes] = static_cast<uint8_t>(s);
      } else {
        const int64_t row = p / per_row;
        const int at = static_cast<int>(p - row * per_row) / kLanes;
        scale[row * ld + at] = static_cast<uint8_t>(s);
        if (at == ld - 3) scale[row * ld + at + 1] = scale[row * ld + at + 2] = 0;   // padding
      }
    }
  }
}

template <typename T, int FMT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint8_t* q,
                                                                 const uint8_t* scale, T* dst,
                                                                 int64_t pieces, int cols) {
  constexpr int N = Act<T>::kPer16B;
  constexpr int kLanes = 32 / N;
  const int per_row = cols / N, ld = mx_scale_ld(cols);
  const bool whole = cols % 128 == 0;   // no padding: scales lie one after another
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kPieces) + threadIdx.x;
  uint32_t raw[kPieces][2];
  uint32_t s[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t p = first + u * kThreads;
    raw[u][0] = raw[u][1] = s[u] = 0;
    if (p < pieces) {
      const uint8_t* at = q + p * (FMT == kE4M3 ? N : N / 2);
      if constexpr (FMT == kE4M3 && N == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(at);
        raw[u][0] = w.x;
        raw[u][1] = w.y;
      } else if constexpr (FMT == kE4M3 || N == 8) {
        raw[u][0] = *reinterpret_cast<const uint32_t*>(at);
      } else {
        raw[u][0] = *reinterpret_cast<const uint16_t*>(at);
      }
      const int64_t row = whole ? 0 : p / per_row;
      s[u] = scale[whole ? p / kLanes : row * ld + static_cast<int>(p - row * per_row) / kLanes];
    }
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t p = first + u * kThreads;
    if (p >= pieces) break;
    const float sc = mx_scale(s[u]);
    float v[N];
    f32x2_hw t;
    if constexpr (FMT == kE4M3) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(raw[u][i], sc, false);
        v[4 * i] = t.x;
        v[4 * i + 1] = t.y;
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(raw[u][i], sc, true);
        v[4 * i + 2] = t.x;
        v[4 * i + 3] = t.y;
      }
    } else {
      t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[u][0], sc, 0);
      v[0] = t.x;
      v[1] = t.y;
      t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[u][0], sc, 1);
      v[2] = t.x;
      v[3] = t.y;
      if constexpr (N == 8) {
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[u][0], sc, 2);
        v[4] = t.x;
        v[5] = t.y;
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[u][0], sc, 3);
        v[6] = t.x;
        v[7] = t.y;
      }
    }
    st_nt16(reinterpret_cast<uint4*>(dst) + p, pack16(v, T{}));
  }
}

template <typename T>
hipError_t quantize(int64_t rows, int32_t cols, const void* src, int32_t fmt, void* q,
                    uint8_t* scale, unsigned grid, int64_t pieces, hipStream_t s) {
  const T* in = static_cast<const T*>(src);
  uint8_t* out = static_cast<uint8_t*>(q);
  if (fmt == kE4M3)
    hipLaunchKernelGGL((mx_quantize_kernel<T, kE4M3>), dim3(grid), dim3(kThreads), 0, s, in, out,
                       scale, pieces, cols);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<T, kE2M1>), dim3(grid), dim3(kThreads), 0, s, in, out,
                       scale, pieces, cols);
  return hipGetLastError();
}

template <typename T>
hipError_t dequantize(const void* q, const uint8_t* scale, int32_t cols, int32_t fmt, void* dst,
                      unsigned grid, int64_t pieces, hipStream_t s) {
  const uint8_t* in = static_cast<const uint8_t*>(q);
  T* out = static_cast<T*>(dst);
  if (fmt == kE4M3)
    hipLaunchKernelGGL((mx_dequantize_kernel<T, kE4M3>), dim3(grid), dim3(kThreads), 0, s, in,
                       scale, out, pieces, cols);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<T, kE2M1>), dim3(grid), dim3(kThreads), 0, s, in,
                       scale, out, pieces, cols);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(int64_t rows, int32_t cols, int32_t act, const void* src,
                              int32_t fmt, void* q, uint8_t* scale, hipStream_t s) {
  const int64_t pieces = rows * (cols / (act == MOE_BF16 ? 8 : 4));
  if (pieces == 0) return hipSuccess;
  const unsigned grid =
      static_cast<unsigned>((pieces + kThreads * kPieces - 1) / (kThreads * kPieces));
  return act == MOE_BF16 ? quantize<bf16_t>(rows, cols, src, fmt, q, scale, grid, pieces, s)
                         : quantize<float>(rows, cols, src, fmt, q, scale, grid, pieces, s);
}

hipError_t launch_mx_dequantize(int64_t rows, int32_t cols, int32_t act, const void* q,
                                const uint8_t* scale, int32_t fmt, void* dst, hipStream_t s) {
  const int64_t pieces = rows * (cols / (act == MOE_BF16 ? 8 : 4));
  if (pieces == 0) return hipSuccess;
  const unsigned grid =
      static_cast<unsigned>((pieces + kThreads * kPieces - 1) / (kThreads * kPieces));
  return act == MOE_BF16 ? dequantize<bf16_t>(q, scale, cols, fmt, dst, grid, pieces, s)
                         : dequantize<float>(q, scale, cols, fmt, dst, grid, pieces, s);
}

}  // namespace moe
