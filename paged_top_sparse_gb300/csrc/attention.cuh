// attention.cuh -- what the full-attention kernels share: row packing, the pieces of a block's run,
// kernel arguments.
#pragma once
#include "ptx.cuh"
#include "sps_internal.h"

namespace sps {
namespace att {

constexpr float kRescale = 8.f;   // log2 of the growth of the maximum that rescales O
constexpr float kF16Bias = 7.f;   // log2 of the factor on FP16 p
constexpr int kMaxCtas = 256;     // blocks (one per SM) that a plan lists work for, at most

// Row packing of a head group.
struct RowPack {
  int HB, TB, blocks;  // heads and tokens per row tile, row-tile head blocks per KV head
  __device__ __host__ explicit RowPack(int hg) {
    HB = hg < 128 ? hg : 128;
    TB = 128 / HB;
    blocks = (hg + HB - 1) / HB;
  }
};

// A run of pages [page0, page1) of one work tile.
struct Piece {
  int req, vg, tok0, ntok;  // tokens tok0 .. of the request (relative), ntok of them
  int page0, page1, pages;  // `pages` of the whole tile
  int q_len, ctx, flat0;    // the request's
  int nt;                   // row tiles with rows
};

// A block's pieces in turn.  The next one is read ahead.
struct PieceList {
  int left, at;
  int4 a, b;  // the next piece
  __device__ __forceinline__ explicit PieceList(const DevPlan& p) {
    const int4* h = reinterpret_cast<const int4*>(p.att_heads + blockIdx.x);
    a = h[0];
    b = h[1];
    const int4 c = h[2];
    left = c.x;
    at = c.y;
  }
  __device__ __forceinline__ bool next(const DevPlan& p, const RowPack& rp, Piece& pc) {
    if (left <= 0) return false;
    pc.req = a.x;
    pc.vg = a.y;
    pc.q_len = b.y;
    pc.ctx = b.z;
    pc.flat0 = b.w;
    pc.tok0 = a.z * 2 * rp.TB;
    pc.ntok = min(2 * rp.TB, pc.q_len - pc.tok0);
    pc.pages = ((pc.ctx + pc.tok0 + pc.ntok - 1) >> 7) + 1;
    pc.page0 = a.w;
    pc.page1 = b.x;
    pc.nt = pc.ntok > rp.TB ? 2 : 1;
    if (--left > 0) {
      const int4* x = reinterpret_cast<const int4*>(p.att_pieces + at++);
      a = __ldg(x);
      b = __ldg(x + 1);
    }
    return true;
  }
};

// Two values rounded to nearest even in 16 bits: P for the second product, or the output.
template <bool F16>
__device__ __forceinline__ uint32_t pack_p(float a, float b) {
  uint32_t r;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// Halves of sdesc_sw128: the low word of a shared address (or of an address in 16-byte units added
// to the one of address 0), and the descriptor of a low word (1024 bytes between 8-row groups).
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t sdesc_hi(uint32_t lo) {
  return (sdesc_sw128(0, 0, 1024) & 0xffffffff00000000ull) | lo;
}
// Warp-level products and exchanges of the single-token kernels.
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, transposed over the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The largest, or the sum, of a row's values over the lanes that share the row.
template <int ROWS, typename Op>
__device__ __forceinline__ float row_reduce(float x, Op op) {
#pragma unroll
  for (int o = ROWS == 16 ? 1 : 4; o < (ROWS == 16 ? 4 : 32); o <<= 1)
    x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

constexpr float kScaleLog2 = 40.f;  // log2 of the range of a V scale, either way

// The power of two 2^k with amax 2^-k in (224, 448] (1 for zero, infinity and NaN).
__device__ __forceinline__ float row_scale(float amax) {
  const uint32_t b = __float_as_uint(amax), e = b >> 23;
  if (e == 0 || e == 255) return 1.f;
  const int k = (int)e - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)max(1, k + 127) << 23);
}

// The log2 of a V scale within its range.
__device__ __forceinline__ float scale_log2(float s) {
  float x;
  asm("lg2.approx.f32 %0, %1;" : "=f"(x) : "f"(s));
  return fminf(fmaxf(x, -kScaleLog2), kScaleLog2);
}

struct AttArgs {
  const uint8_t *q, *kc, *vc, *ks, *vs;  // quantised plans (and Q); E4M3: ks, vs are FP32
  int64_t q_stride;
  const int32_t* page_table;
  uint16_t* out;
  int64_t out_stride;
  float* out_lse;
  float *part, *part_lse;  // [2 att_ctas][slot rows][D], [2 att_ctas][slot rows]
  float c;                 // softmax scale x q_scale x log2 e
  uint64_t skip_wait_ns;   // limit of a wait that follows the block's pieces
};

// Single tokens over an NVFP4 cache (tiles of at most 16 rows): the products' part of launch_attention.
cudaError_t launch_decode_nvfp4(const DevPlan& p, const AttArgs& a, cudaStream_t st);

// The merge of the tiles that the plan cut over blocks, behind any of the products' kernels.
cudaError_t launch_merge(const DevPlan& p, const AttArgs& a, cudaStream_t st);

// The products over an E4M3 cache for tiles of at most 16 rows (single tokens).
cudaError_t launch_decode_e4m3(const DevPlan& p, bool q_e4m3, const AttArgs& a, cudaStream_t st);

// Full attention over an E4M3 cache with a scale for each page and KV head.
cudaError_t launch_attention_e4m3(const DevPlan& p, bool q_e4m3, const AttArgs& a, cudaStream_t st);

}  // namespace att
}  // namespace sps
