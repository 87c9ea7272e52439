// nvfp4.cuh -- conversion of NVFP4 tiles into tensor-core operand tiles, shared by the kernels
// that read an NVFP4 cache in their loaders.
#pragma once
#include "ptx.cuh"

namespace sps {

// One NVFP4 tile (codes [128][D/2], then scales [128][D/16], in `raw`) into the operand tile
// `dst`: 128 rows of D elements in the 128-byte-swizzled layout TMA writes, as FP16 products
// code x scale (exact) in column blocks of 64 elements (16 KB each), or, with E4M3OUT, as those
// products rounded to E4M3 (one 128-byte block per row; D = 128).  Thread t of nt converts the
// 16-byte code chunks t, t + nt, ... (32 elements each).
template <int D, bool E4M3OUT>
__device__ __forceinline__ void nvfp4_tile_convert(const uint8_t* raw, uint8_t* dst, int t, int nt) {
  constexpr int CPR = D / 32;  // code chunks per row
  const uint8_t* scl = raw + 128 * D / 2;
  for (int c = t; c < 128 * CPR; c += nt) {
    const int row = c / CPR, i = c % CPR;
    const uint4 cw = reinterpret_cast<const uint4*>(raw)[c];
    const uint32_t sb = *reinterpret_cast<const uint16_t*>(scl + row * (D / 16) + 2 * i);
    const uint32_t s0 = cvt_e4m3x2((uint16_t)((sb & 0xffu) * 0x0101u));  // elements 0..15
    const uint32_t s1 = cvt_e4m3x2((uint16_t)((sb >> 8) * 0x0101u));     // elements 16..31
    const uint32_t w[4] = {cw.x, cw.y, cw.z, cw.w};
    uint32_t h[16];  // h[4 j + b]: elements 8 j + 2 b, +1 of the chunk
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        h[4 * j + b] = hmul2_u32(cvt_e2m1x2((uint16_t)((w[j] >> (8 * b)) & 0xffu)), j < 2 ? s0 : s1);
    if (E4M3OUT) {
      uint32_t e[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        e[u] = (uint32_t)cvt_f16x2_e4m3x2(h[2 * u]) | ((uint32_t)cvt_f16x2_e4m3x2(h[2 * u + 1]) << 16);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<uint4*>(dst + sw128_offset(row, 2 * i + u)) =
            make_uint4(e[4 * u], e[4 * u + 1], e[4 * u + 2], e[4 * u + 3]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = 32 * i + 8 * u;
        *reinterpret_cast<uint4*>(dst + (col / 64) * 16384 + sw128_offset(row, (col % 64) / 8)) =
            make_uint4(h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
      }
    }
  }
}

// The four bytes of w, two E2M1 codes each, as FP16 pairs (exact).
__device__ __forceinline__ void cvt_e2m1x8(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// (One word at a time: with the bytes taken out by shifts the conversion of a tile, which shares its
// SM's issue slots with the softmax, made an attention chunk 8 % slower.)
// The same FP16 products with a thread per row (128 threads): a row's codes and scales in
// registers, then its operand row.  Rows marked empty become zero, whatever their codes and scales
// hold.  A thread starts at a column of its own (row / 2 or row / 4), which keeps a quarter warp's
// loads, and at D = 128 its stores, on distinct banks.
template <int D>
struct Nvfp4Row {
  static constexpr int CPR = D / 32;  // 16-byte code chunks per row
  uint4 cw[CPR];
  uint64_t sc;  // the row's scales, one byte per 16 elements
  __device__ __forceinline__ static int turn(int row) { return CPR == 4 ? row >> 1 : row >> 2; }
  __device__ __forceinline__ void load(const uint8_t* raw, int row, bool empty) {
    const uint4* codes = reinterpret_cast<const uint4*>(raw) + row * CPR;
    if (CPR == 4) sc = *reinterpret_cast<const uint64_t*>(raw + 64 * D + row * 8);
    else sc = *reinterpret_cast<const uint32_t*>(raw + 64 * D + row * 4);
#pragma unroll
    for (int k = 0; k < CPR; ++k) cw[k] = codes[(k + turn(row)) % CPR];
    if (empty) {
      sc = 0;
#pragma unroll
      for (int k = 0; k < CPR; ++k) cw[k] = make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void store(uint8_t* dst, int row) const {
#pragma unroll
    for (int k = 0; k < CPR; ++k) {
      const int i = (k + turn(row)) % CPR;
      // the scales of elements 0..15 and 16..31 of the chunk
      const uint32_t two = cvt_e4m3x2((uint16_t)(sc >> (16 * i)));
      const uint32_t s0 = __byte_perm(two, two, 0x1010), s1 = __byte_perm(two, two, 0x3232);
      const uint32_t w[4] = {cw[k].x, cw[k].y, cw[k].z, cw[k].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t h[4];
        cvt_e2m1x8(w[u], h);
#pragma unroll
        for (int b = 0; b < 4; ++b) h[b] = hmul2_u32(h[b], u < 2 ? s0 : s1);
        const int col = 32 * i + 8 * u;
        *reinterpret_cast<uint4*>(dst + (col / 64) * 16384 + sw128_offset(row, (col % 64) / 8)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
  }
};

}  // namespace sps
