// The microscaled 4-bit format (OCP MXFP4): blocks of 32 consecutive elements
// share a scale 2^(b - 127) held as one byte b (255 is NaN), each element is a
// 4-bit e2m1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives); element 2i
// sits in the low four bits of byte i.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace ra {

constexpr int kMxBlock = LORA_MX_BLOCK;

// Tiles of an expert's scale bytes (lora_mx_tile_scales): 512 bytes for every
// 128 outputs and 128 elements, an even number of them along the elements.
constexpr int kMxTile = 128, kMxTileBytes = 512;
__host__ __device__ constexpr int mx_tiles_out(int d_out) { return (d_out + kMxTile - 1) / kMxTile; }
__host__ __device__ constexpr int mx_tiles_in(int d_in) { return (d_in + 2 * kMxTile - 1) / (2 * kMxTile) * 2; }

// Eight elements to e2m1 codes, nearest (ties to the even code), magnitudes
// above 6 saturate; element 0 in the lowest four bits.
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight codes (lowest four bits first).
__device__ __forceinline__ void mx_decode8(uint32_t q, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// 2^(b - 127); byte 0 is 2^-127 (subnormal), byte 255 NaN.
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : b == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}

// Scale byte of a block whose largest magnitude has the float bits `amax`:
// floor(log2 amax) - 2 (the format's largest element is 6 = 1.5 * 2^2), held to
// byte 0 at the low end; 255 when the block holds a NaN or an infinity.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int b = (int)(amax >> 23) - 2;
  return b > 0 ? (uint32_t)b : 0u;
}
// 2^(127 - b), the factor that brings a block's elements onto the codes' grid
// (b <= 252: the bytes mx_scale_byte gives a finite block).
__device__ __forceinline__ float mx_inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// A block's quarter: four neighbouring lanes hold its 32 elements, eight each.
// Gives this lane's codes and the block's scale byte. Every lane of the warp
// must call it.
__device__ __forceinline__ uint32_t mx_quantize8(const float (&v)[8], uint32_t &byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);  // NaN sorts above every number
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  byte = mx_scale_byte(m);
  if (byte == 255u) return 0u;
  const float f = mx_inv_scale(byte);
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = v[i] * f;  // a power of two: exact wherever the code is not 0
  return mx_encode8(s);
}

}  // namespace ra
