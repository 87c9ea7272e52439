// e4m3.cuh -- conversion of E4M3 tiles into tensor-core operand tiles, shared by the kernels that read
// an 8-bit cache.
#pragma once
#include "ptx.cuh"

namespace sps {

// Four E4M3 codes as two FP16 pairs, or, with BF16, as two BF16 pairs (both exact: NaN codes give NaN).
template <bool BF16>
__device__ __forceinline__ void cvt_e4m3x4(uint32_t w, uint32_t& a, uint32_t& b) {
  a = cvt_e4m3x2((uint16_t)(w & 0xffffu));
  b = cvt_e4m3x2((uint16_t)(w >> 16));
  if (BF16) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(a) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(y.y), "f"(y.x));
  }
}

// 16 consecutive codes of a row, from column 16 i on, into the row of an operand tile: 128 rows of D
// elements in the 128-byte-swizzled layout TMA writes, in column blocks of 64 elements (16 KB each).
template <bool BF16>
__device__ __forceinline__ void e4m3_store16(const uint4& x, uint8_t* dst, int row, int i) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) cvt_e4m3x4<BF16>(w[j], h[2 * j], h[2 * j + 1]);
  uint8_t* d = dst + (i / 4) * 16384;
#pragma unroll
  for (int u = 0; u < 2; ++u)
    *reinterpret_cast<uint4*>(d + sw128_offset(row, 2 * (i % 4) + u)) =
        make_uint4(h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
}

// One tile of codes [128][D] into the operand tile.  Thread t of nt takes whole 16-byte chunks; eight
// threads in a row take the chunks of eight rows, each at a column of its own, which keeps their loads
// and stores on distinct banks (D = 128; two threads share a bank at D = 64).
template <int D, bool BF16>
__device__ __forceinline__ void e4m3_tile_convert(const uint8_t* raw, uint8_t* dst, int t, int nt) {
  constexpr int CPR = D / 16;
#pragma unroll 4
  for (int c = t; c < 128 * CPR; c += nt) {
    const int row = c % 128, i = (c / 128 + row) % CPR;
    e4m3_store16<BF16>(reinterpret_cast<const uint4*>(raw)[row * CPR + i], dst, row, i);
  }
}

// Zeros in place of the rows from `rows` on, each 16 codes' by the thread that converted them.
template <int D>
__device__ __forceinline__ void e4m3_tile_clear(uint8_t* dst, int t, int nt, int rows) {
#pragma unroll 1
  for (int c = t; c < 128 * (D / 16); c += nt) {
    const int row = c % 128, i = (c / 128 + row) % (D / 16);
    if (row >= rows) e4m3_store16<false>(make_uint4(0, 0, 0, 0), dst, row, i);
  }
}

}  // namespace sps
