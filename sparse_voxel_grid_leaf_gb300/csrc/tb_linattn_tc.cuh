// What the two chunk kernels of linear attention share (tb_linattn_chunk.cu,
// tb_linattn_split.cu).
#pragma once

#include "tb_linattn.cuh"
#include "tb_linattn_scan.cuh"
#include "tb_tc.cuh"

namespace tb {

constexpr int kC = 64;       // rows of a chunk
constexpr int kTile = 8192;  // 64 rows x 128 bytes
// decay^32 within 2^50: half of the exponents that 32-bit floats have are left
// to the values.
constexpr float kSteep = 0.34f;

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ float low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ float shared_bf16(uint32_t at) {
  uint16_t bits;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(at));
  return __uint_as_float((uint32_t)bits << 16);
}
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
// What is left of a scale next to a value that is not finite: its sign, or 0 or
// NaN, which make the product NaN.
__device__ __forceinline__ float sign_of(float x) { return x > 0.f ? 1.f : x < 0.f ? -1.f : x; }
// Element x of row r in a tile of 64-element rows.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int r, int x) {
  return tile + r * 128 + (((x >> 3) ^ (r & 7)) << 4) + (x & 7) * 2;
}

}  // namespace tb
