// mxfp4.cuh — the microscaled 4-bit format shared by the quantizers and the product.
//
// MXFP4: E2M1 elements (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one power-of-two (E8M0)
// scale per 32 elements (low-precision format table).  Codes are packed two to a byte, the
// even element in the low half.  The scale rule is the library's own carried to this
// element: e = the smallest integer with amax <= 6 * 2^e, 0 for an all-zero tile.
//
// Scale bytes are stored as the tensor cores read them, in 512-byte tiles of 128 rows x 4
// scales (128 elements of K): tile (r / 128, c / 4) of row r and scale column c, tiles
// row-major, and inside a tile byte (r % 32) * 16 + (r % 128 / 32) * 4 + c % 4.
#pragma once

#include "common.cuh"

namespace fp8q {

constexpr int kSfTileBytes = 512;

// Byte offset of the four scales of row r, K tile c4 (128 elements); k128 = K / 128.
__device__ __forceinline__ int64_t sf_word_offset(int64_t r, int64_t c4, int64_t k128) {
  return ((r >> 7) * k128 + c4) * kSfTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Scale exponent of a tile from its BF16 amax bit pattern: amax = (1 + m/128) * 2^(E-127),
// 6 = 1.5 * 2^2, so e = E - 129, plus one when m > 64.
__device__ __forceinline__ int mxfp4_tile_exponent(uint32_t amax16) {
  const int e = (int)(amax16 >> 7) - 129 + ((amax16 & 0x7Fu) > 0x40u ? 1 : 0);
  return amax16 == 0u ? 0 : max(e, -127);
}

// Eight bf16 (four words) times s -> eight codes, round to nearest even, element 0 in the
// low nibble.  The product by a power of two is exact except below 2^-126, where E2M1
// rounds to +-0 either way.
__device__ __forceinline__ uint32_t encode8_e2m1(const uint4& v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16) * s;
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * s;
  }
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

}  // namespace fp8q
