// fp4.cuh -- the FP4 cache format: where a tile keeps its bytes, and the conversions.
//
// A (block, kv head) tile holds BS token rows of D dims, each row D/16 groups of 16
// dims: 16 E2M1 codes and one E4M3 scale sf a group.  An element reads back as
// code * sf * s with the tensor's fp32 scale s.  The tile is the codes (D/2 bytes a
// row, low nibble first), then one scale byte per row and group.
//
// The order of rows and scales is the one the decode kernel's tensor-core fragments
// read without bank conflicts.  Rows come in sub-tiles of 16 tokens; in one, the four
// lanes (t4) of a fragment row group own tokens 4 t4 .. 4 t4 + 3:
//   * code row of token t: (t / 4) ^ (3 if t is odd) + 4 (t % 4).  The V fragments
//     read token 4 t4 + i of all four t4 at once, four rows in a run; the K fragments
//     read tokens 4 k and 4 k + 1 together, rows of different parity (D 128) or in
//     different quarters of 128 bytes (D 64).  At D 128 the 32-byte halves of a row
//     change places where bit 1 of its row number is set, so that the four V rows'
//     32-byte pieces fall on all 32 banks.
//   * K scales: the bytes one lane needs (its groups for tokens t and t + 2) adjacent.
//   * V scales: group-major, the tokens of a group adjacent.
#pragma once

#include "pa_device.cuh"

namespace pa {
namespace fp4 {

__host__ __device__ constexpr int tile_bytes(int D, int BS) { return BS * (D / 2 + D / 16); }

// Byte offset in a tile of byte j (dims 2j, 2j + 1) of token t's row of codes.
template <int D>
__host__ __device__ constexpr int code_at(int t, int j) {
  const int r = t & 15;
  const int row = (t & ~15) + ((r >> 2) ^ ((r & 1) ? 3 : 0)) + 4 * (r & 3);
  return row * (D / 2) + (D == 128 ? (j ^ (((row >> 1) & 1) << 5)) : j);
}
// Byte offset in a tile of the scale of group g of token t, in a K and in a V tile.
template <int D, int BS>
__host__ __device__ constexpr int k_scale_at(int t, int g) {
  constexpr int G = D / 16, GL = G / 4;  // groups of a row, and of a lane of four
  const int r = t & 15;
  return BS * (D / 2) + (t & ~15) * G + (2 * (r >> 2) + (r & 1)) * 2 * G + (g / GL) * 2 * GL + ((r >> 1) & 1) * GL +
         g % GL;
}
template <int D, int BS>
__host__ __device__ constexpr int v_scale_at(int t, int g) {
  return BS * (D / 2) + (t & ~15) * (D / 16) + g * 16 + (t & 15);
}

// Eight codes (nibble i = code i) as four packed fp16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 codes (the low 16 bits) as a packed fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t h;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(two));
  return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight fp32 values to E2M1 codes: nearest, ties to even, at most 6 (a NaN: 6).
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&y)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

}  // namespace fp4
}  // namespace pa
