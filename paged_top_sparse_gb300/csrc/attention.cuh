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

struct AttArgs {
  const uint8_t *q, *kc, *vc, *ks, *vs;  // NVFP4 plans (and Q's codes)
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

}  // namespace att
}  // namespace sps
