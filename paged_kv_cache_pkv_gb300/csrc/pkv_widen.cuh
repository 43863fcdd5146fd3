// pkv_widen.cuh -- E4M3 pages widened to bf16 tiles for the tensor cores, shared
// by the kernels that read FP8 pages through tcgen05.
#pragma once

#include <cuda_fp16.h>

#include "pkv_common.cuh"

namespace pkv {

// Four E4M3 codes (lowest byte first) -> two f16x2 (exact: E4M3 is a subset of f16).
__device__ __forceinline__ void e4m3x4_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// f16 pair times a power of two -> bf16 pair (exact for E4M3 values under the
// row scales the FP8 write produces).
__device__ __forceinline__ uint32_t widen_pair(uint32_t h2, float sc) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  return pack_bf16x2(f.x * sc, f.y * sc);
}

// Four E4M3 codes (lowest byte first) times 2^(scale-127) -> four bf16 (two
// pairs, lowest first), integer arithmetic only.  For a code with a nonzero
// exponent field E and mantissa m, the product is 2^(E-7) * (1 + m/8) *
// 2^(scale-127): bf16 exponent field E + scale - 7, mantissa m in its top
// three bits, the sign as is.  `adj` is (scale - 7) << 7 in both halves; it
// is exact for scale in [7, 246] (exponent fields 1..254) and codes with a
// nonzero exponent field (zero and subnormal codes take the f16 route).
__device__ __forceinline__ void widen4_int(uint32_t w, uint32_t adj, uint32_t& lo, uint32_t& hi) {
  const uint32_t p0 = __byte_perm(w, 0u, 0x1404u);  // codes 0, 1 in the high byte of each half
  const uint32_t p1 = __byte_perm(w, 0u, 0x3424u);  // codes 2, 3
  lo = (((p0 >> 4) & 0x07F007F0u) + adj) | (p0 & 0x80008000u);
  hi = (((p1 >> 4) & 0x07F007F0u) + adj) | (p1 & 0x80008000u);
}

// Nonzero when some code of w has a zero exponent field (zero or subnormal).
__device__ __forceinline__ uint32_t zero_field(uint32_t w) {
  const uint32_t t = w & 0x78787878u;
  return (t - 0x01010101u) & ~t & 0x80808080u;
}

// Same through f16 (exact for every finite code and any scale byte).
__device__ __forceinline__ void widen4_f16(uint32_t w, float sc, uint32_t& lo, uint32_t& hi) {
  uint32_t a0, a1;
  e4m3x4_f16x2(w, a0, a1);
  lo = widen_pair(a0, sc);
  hi = widen_pair(a1, sc);
}

// One lane's half row of an FP8 page: codes of dims 64h..64h+63 of row r (the
// staged page as TMA laid it out, 128-byte swizzle) times 2^(scale-127), as
// bf16 into row `drow` of the half-h block of a K/V tile (128-byte swizzle,
// row index = key within the tile, congruent to r mod 8).  The chunk order
// c = cc ^ 4h keeps each quarter-warp's 16-byte stores on distinct banks.
// One branch per lane: the integer route when the scale byte and every code
// allow it (nearly always), else the f16 route.  Words are picked with
// compile-time indices (a select on h), so w[] stays in registers.
__device__ __forceinline__ void widen_row_half(const uint8_t* spage, uint32_t sbyte, uint8_t* drow,
                                               int r, int h) {
  uint32_t w[16];  // codes of dims 64h + 4k .. 64h + 4k + 3
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(spage + r * 128 + (((4 * h + i) ^ (r & 7)) << 4));
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
  uint32_t z = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) z |= zero_field(w[k]);
  if (z == 0u && sbyte >= 7u && sbyte <= 246u) {
    const uint32_t adj = ((sbyte - 7u) << 7) * 0x00010001u;
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) {
      const int c = cc ^ (h << 2);  // dims 8c..8c+7 of the half
      const uint32_t wa = h ? w[2 * (cc ^ 4)] : w[2 * cc];
      const uint32_t wb = h ? w[2 * (cc ^ 4) + 1] : w[2 * cc + 1];
      uint4 o;
      widen4_int(wa, adj, o.x, o.y);
      widen4_int(wb, adj, o.z, o.w);
      *reinterpret_cast<uint4*>(drow + ((c ^ (r & 7)) << 4)) = o;
    }
  } else {
    const float sc = __uint_as_float(sbyte << 23);  // 2^(sbyte-127); byte 0 is never written
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint4 o;
      widen4_f16(w[2 * c], sc, o.x, o.y);
      widen4_f16(w[2 * c + 1], sc, o.z, o.w);
      *reinterpret_cast<uint4*>(drow + ((c ^ (r & 7)) << 4)) = o;
    }
  }
}

}  // namespace pkv
