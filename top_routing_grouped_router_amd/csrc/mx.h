// Block-scaled 8- and 4-bit numbers (OCP Microscaling formats), shared by the
// quantiser, the norm and the low-precision experts.
//
// 32 consecutive values of a row share a power of two, held as a byte s that
// stands for 2^(s - 127) (255: NaN).  Elements are e4m3 (largest 448) or e2m1
// (largest 6 = 1.5 * 2^2).  The scale is the smallest power of two with
// amax <= largest * 2^(s - 127), so no element saturates; by the bits of amax
// it is the exponent field, one more when the fraction lies above the largest
// element's fraction (448 = 1.75 * 2^8, so fraction bits above 0x600000; 6:
// above 0x400000), less the largest element's exponent (8 or 2), and at least
// 0.  Dividing by a power of two is exact, so each value is rounded once (to
// nearest even, by the conversion instruction).  A block that holds a NaN or
// an infinity gets scale 255: every value of it reads as NaN, which the
// products carry on (a finite stand-in would hide the fault).
#pragma once

#include "common.h"

namespace moe {

enum MxFormat { kE4M3 = MOE_MX_E4M3, kE2M1 = MOE_MX_E2M1 };

// bytes of a scale row: one per 32 values, padded to whole words, so the
// scales of 128 values are one aligned word for the matrix kernels
__host__ __device__ __forceinline__ int mx_scale_ld(int cols) { return (cols + 127) / 128 * 4; }

// |v| as bits: ordered like the values, NaN above infinity
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// v of another lane, by a vector instruction (a shuffle goes through LDS and waits for
// it: the norm of 16384 x 2048 takes 55 us with them, 50.5 so): the neighbour, the
// neighbouring pair, the mirrored lane of 8 and of 16, the lane 4 and 8 along in 16
enum LaneOf {
  kSwap1 = 0xB1, kSwap2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140, kAlong4 = 0x124, kAlong8 = 0x128
};
template <int LANE, typename T>
__device__ __forceinline__ T from_lane(T v) {
  int w[sizeof(T) / 4];
  __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
  for (int& i : w) i = __builtin_amdgcn_update_dpp(0, i, LANE, 0xF, 0xF, true);
  __builtin_memcpy(&v, w, sizeof(T));
  return v;
}

// scale byte of a block with the largest |value| bits `amax`
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  constexpr uint32_t kOver = FMT == kE4M3 ? 0x1FFFFFu : 0x3FFFFFu;
  constexpr int kTop = FMT == kE4M3 ? 8 : 2;
  const int s = max(static_cast<int>((amax + kOver) >> 23) - kTop, 0);
  return amax >= 0x7F800000u ? 255u : static_cast<uint32_t>(s);
}

// 2^(127 - s), what the block's values are multiplied by (NaN for 255)
__device__ __forceinline__ float mx_inverse(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7FC00000u : (254u - s) << 23);
}

// 2^(s - 127): a subnormal for s = 0; 255 gives infinity's bits, which the
// conversion instructions below take as NaN, whatever the element
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __uint_as_float(s ? s << 23 : 0x00400000u);
}

// four values to four e4m3 bytes
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}
// eight values to eight e2m1 codes, the first in the low half byte
__device__ __forceinline__ uint32_t pack_e2m1(const float* v) {
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
}
// four values to four e2m1 codes in the low 16 bits
__device__ __forceinline__ uint32_t pack_e2m1x4(const float* v) {
  const uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], 1.0f, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
}

// Quantise the N values of a lane (N = 8 bf16 or 4 fp32 values: 16 bytes of the
// source), one piece of a block that 32 / N neighbouring lanes hold together
// (all of them or none active): returns the block's scale byte and writes the
// lane's elements (N bytes of e4m3 or N / 2 of e2m1) to `q`.
template <int FMT, int N>
__device__ __forceinline__ uint32_t mx_store(const float (&v)[N], void* q) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) m = max(m, abs_bits(v[i]));
  m = max(m, from_lane<kSwap1>(m));
  m = max(m, from_lane<kSwap2>(m));
  if constexpr (N == 4) m = max(m, from_lane<kMirror8>(m));
  const uint32_t s = mx_scale_byte<FMT>(m);
  const float inv = mx_inverse(s);
  float u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = v[i] * inv;
  if constexpr (FMT == kE4M3) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] = pack_e4m3(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    if constexpr (N == 8) *static_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else *static_cast<uint32_t*>(q) = w[0];
  } else {
    if constexpr (N == 8) *static_cast<uint32_t*>(q) = pack_e2m1(u);
    else *static_cast<uint16_t*>(q) = static_cast<uint16_t>(pack_e2m1x4(u));
  }
  return s;
}

}  // namespace moe
