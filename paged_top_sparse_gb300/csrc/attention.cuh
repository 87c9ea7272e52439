// attention.cuh -- what the full-attention kernels share: row packing, the pieces of a block's run,
// kernel arguments.
#pragma once
#include "ptx.cuh"
#include "sps_internal.h"

namespace sps {
namespace att {

constexpr float kRescale = 8.f;   // log2 of the growth of the maximum that rescales O
constexpr float kF16Bias = 7.f;   // log2 of the factor on FP16 p
constexpr int kMaxCtas = 256;

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

// The piece at cursor c of a block whose run ends at e; advances c.  False at the end.  The cursor
// carries its request's numbers, so that a run's first piece needs no further read.
__device__ __forceinline__ bool next_piece(const DevPlan& p, const RowPack& rp, AttCursor& c,
                                           const AttCursor& e, Piece& pc) {
  const int tt = 2 * rp.TB, nv = p.Hkv * rp.blocks;
  for (;;) {
    if (c.req >= p.batch) return false;
    if (c.req == e.req && c.vg == e.vg && c.tile == e.tile && c.page == e.page) return false;
    if (c.q_len > 0) {
      const bool last = c.req == e.req && c.vg == e.vg && c.tile == e.tile;
      pc.req = c.req;
      pc.vg = c.vg;
      pc.q_len = c.q_len;
      pc.ctx = c.ctx;
      pc.flat0 = c.flat0;
      pc.tok0 = c.tile * tt;
      pc.ntok = min(tt, c.q_len - pc.tok0);
      pc.pages = ((pc.ctx + pc.tok0 + pc.ntok - 1) >> 7) + 1;
      pc.page0 = c.page;
      pc.page1 = last ? min(e.page, pc.pages) : pc.pages;
      pc.nt = pc.ntok > rp.TB ? 2 : 1;
      if (last) {
        c = e;
        return pc.page0 < pc.page1;
      }
      c.page = 0;
      if ((c.tile + 1) * tt < c.q_len) {
        ++c.tile;
        return true;
      }
      c.tile = 0;
      if (++c.vg < nv) return true;
      c.vg = 0;
    }
    const bool done = c.q_len > 0;  // a piece was found above
    if (++c.req < p.batch) {
      const ReqInfo* ri = p.reqs + c.req;
      c.q_len = __ldg(&ri->q_len);
      c.ctx = __ldg(&ri->ctx);
      c.flat0 = __ldg(&ri->tok0);
    }
    if (done) return true;
  }
}

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
};

// Single tokens over an NVFP4 cache (tiles of at most 16 rows): the products' part of launch_attention.
cudaError_t launch_decode_nvfp4(const DevPlan& p, const AttArgs& a, cudaStream_t st);

}  // namespace att
}  // namespace sps
