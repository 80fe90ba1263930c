// Microscaled 4-bit floating point: formats and sizes shared by the row
// kernels and the grouped product.
//
// Codes are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a
// byte, the even element in the low half.  A block of consecutive elements of
// a row shares one 8-bit scale:
//   MX  32 elements, E8M0 (2^e);      NV  16 elements, E4M3 times 2^scale_exp.
// Scale rows are padded to whole 256-element steps (zero bytes).
#pragma once

#include <stdint.h>

namespace fp4 {

constexpr int kStepElems = 256;  // elements of K per pipeline step: 128 bytes of codes

template <int FMT>
struct Fmt;
template <>
struct Fmt<0> {  // MX
  static constexpr int kBlock = 32;
  static constexpr int kScaleBytes = 8;  // scale bytes of a row per step
  static constexpr uint32_t kScaleBad = 0xFF;
};
template <>
struct Fmt<1> {  // NV
  static constexpr int kBlock = 16;
  static constexpr int kScaleBytes = 16;
  static constexpr uint32_t kScaleBad = 0x7F;
};

// Weight tiles: 256 weight rows (two halves of 128) x 256 elements of K.
constexpr int kHalfRows = 128;
constexpr int kTileCodes = 2 * kHalfRows * 128;
__host__ __device__ constexpr int tile_bytes(int fmt) { return kTileCodes + 2 * kHalfRows * (fmt == 1 ? 16 : 8); }

}  // namespace fp4
