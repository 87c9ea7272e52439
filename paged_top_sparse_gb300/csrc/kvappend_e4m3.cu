// kvappend_e4m3.cu -- the append of new tokens' K/V into a paged cache held in 8 bits: E4M3 codes
// and one FP32 scale for each (page, KV head) of K and of V (sps_kv_append and sps_kv_append_rope on a
// plan with an E4M3 cache).
//
// Mathematics.  y: the key row normalised and rotated in FP32 (rope.cuh), or the value row.  For each
// touched page and head, over the rows that this call adds to it:
//   s_new = 2^k, the smallest power of two with max |y| / s_new <= 448, within [2^-40, 2^40]
//   s = max(s_old, s_new) where the page holds earlier tokens of the request, else s_new
//   code = E4M3(y / s); where s grew, earlier codes become E4M3(code * (s_old / s)).
// A power of two: E4M3 keeps four significant bits over 15 binades whatever the scale, so a finer scale
// would gain nothing; y / s is exact, and a scale that grows moves the exponents of the earlier codes,
// exactly unless they fall below 2^-6.
//
// Layout.  A block takes a touched page (the plan's list) and some of its heads, K or V.  Its rows come into
// shared memory by asynchronous copies (the next head's while this one's codes are made), the page's
// angles are made once for all heads, and each row is worked out twice: for the maximum, then for the
// codes.  D / 8 lanes hold a row, 8 elements (16 bytes) each.
//
// Bound: many tokens, the rows worked out twice: 65536 tokens of 8 heads, 403 MB, take 153 us (2.6 TB/s) with
// the issue slots 68 % and the ALU 45 % busy, so that no unit is full and the waits between a row's steps
// count as well; results kept in registers instead halve the warps on an SM (186 us), and rows unrolled cost
// instruction fetches (349).  Angles read a lane's own pairs in a row put every fourth lane on one bank:
// 332 us against 204.  4096 tokens of 2 heads 8.1 us, a decode step of 64 3.3 (a chain of the list, the
// page table, the rows, the maximum): `sps_kv_append_rope` into a BF16 cache takes 5.3 and 2.3.
#include <algorithm>

#include "rope.cuh"

namespace sps {
namespace {

constexpr int kScaleExp = 40;  // scales lie within 2^-40 .. 2^40

// The smallest power of two s with amax / s <= 448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = max(-kScaleExp, min(kScaleExp, k));
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

// Codes of 8 elements: y / s.  A scale that this file made is a power of two, whose inverse is exact.
__device__ __forceinline__ uint2 codes8(const uint64_t (&y)[4], float s, float inv, bool pow2) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t q = mul_f32x2(y[i], pack_f32x2(inv, inv));
    if (!pow2) {
      float lo, hi;
      unpack_f32x2(y[i], lo, hi);
      q = pack_f32x2(__fdiv_rn(lo, s), __fdiv_rn(hi, s));
    }
    o[i] = f32x2_to_e4m3x2(q);
  }
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// Cosines and sines of a token's pairs where its rows' lanes read them side by side (a lane's own pairs in a
// row of shared memory would put every fourth lane on one bank): 16-byte entry (q, chunk) holds pairs 2 q
// and 2 q + 1 of the chunk, as (cos, cos, sin, sin), or, for adjacent pairs, as (cos, sin, cos, sin).
// Made by the whole block for tokens tok0 .. of cache positions pos0 .. .
template <bool INTER, int THREADS>
__device__ __forceinline__ void chunk_angles(const DevRope& r, const DevPlan& p, int tok0, int pos0, int count,
                                             const uint64_t* turns, float* cs) {
  constexpr int PPC = INTER ? 4 : 8;  // pairs of a chunk
  const int half = r.rot / 2, chunks = half / PPC;
  const int warp = threadIdx.x >> 5;
  for (int j = threadIdx.x & 31; j < half; j += 32) {
    float* e = cs + (j % PPC / 2 * chunks + j / PPC) * 4 + (INTER ? j % 2 * 2 : j % 2);
    const uint64_t turn = turns[j];
    const int32_t* at = r.positions ? r.positions + (int64_t)r.axis[j] * p.T + tok0 : nullptr;
#pragma unroll 4
    for (int i = warp; i < count; i += THREADS / 32) {
      const uint64_t t = (uint64_t)(int64_t)(at ? __ldg(at + i) : pos0 + i) * turn;
      float sn, cn;
      sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &sn, &cn);  // (as token_angles does)
      e[i * r.rot] = cn;
      e[i * r.rot + (INTER ? 1 : 2)] = sn;
    }
  }
}

// A lane's part in its rows: y = (x w) cos + (x_partner w_partner) sin, over the row's root mean square.
template <int D, bool INTER>
struct KeyRows {
  uint64_t w[4], wp[4];  // the weights of its 8 dims and, with the sine's sign, of their partners
  int partner;           // lane of the partner chunk (half-split pairs)
  int entry, chunks;     // its place among the token's entries; -1: the dims are not rotated
  __device__ __forceinline__ void make(const DevRope& r, const float* weight, int lane) {
    const int d0 = lane % (D / 8) * 8, half = r.rot / 2;
    entry = -1;
    chunks = half / (INTER ? 4 : 8);
    partner = lane;
    int p0 = d0;
    if (d0 < r.rot) {
      entry = INTER ? d0 / 8 : d0 % half / 8;
      if (!INTER) {
        partner = d0 < half ? lane + half / 8 : lane - half / 8;
        p0 = d0 < half ? d0 + half : d0 - half;
      }
    }
    float own[8], other[8];
    load_weights(weight, d0, own);
    load_weights(weight, p0, other);
    const float sign = d0 < half ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_f32x2(own[2 * i], own[2 * i + 1]);
      wp[i] = INTER ? pack_f32x2(-own[2 * i + 1], own[2 * i])
                    : pack_f32x2(sign * other[2 * i], sign * other[2 * i + 1]);
    }
  }
  // All 32 lanes call it.
  __device__ __forceinline__ void apply(const uint4& raw, const float4* cs, bool norm, float eps,
                                        uint64_t (&y)[4]) const {
    const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
    uint64_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_f32x2(bf16_lo(x[i]), bf16_hi(x[i]));
    float scale = 1.f;
    if (norm) {
      uint64_t s2 = mul_f32x2(v[0], v[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) s2 = fma_f32x2(v[i], v[i], s2);
      float lo, hi;
      unpack_f32x2(s2, lo, hi);
      float ss = lo + hi;
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      scale = rsqrtf(fmaf(ss, 1.f / D, eps));
    }
    uint64_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (INTER) {
        q[i] = pack_f32x2(bf16_hi(x[i]), bf16_lo(x[i]));
      } else {
        const uint32_t o = __shfl_sync(0xffffffffu, x[i], partner);
        q[i] = pack_f32x2(bf16_lo(o), bf16_hi(o));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul_f32x2(v[i], w[i]);
    if (entry >= 0) {  // (a dim that is not rotated must not meet 0 * infinity)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 t = cs[(INTER ? i / 2 : i) * chunks + entry];
        const float c0 = INTER && i % 2 ? t.z : t.x, c1 = INTER ? c0 : t.y;
        const float s0 = INTER && i % 2 ? t.w : INTER ? t.y : t.z, s1 = INTER ? s0 : t.w;
        v[i] = fma_f32x2(mul_f32x2(q[i], wp[i]), pack_f32x2(s0, s1), mul_f32x2(v[i], pack_f32x2(c0, c1)));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul_f32x2(v[i], pack_f32x2(scale, scale));
  }
};

template <int D, bool INTER, int THREADS, int ROWS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
kv_append_e4m3_kernel(DevPlan p, const __grid_constant__ DevRope r, KvRopeArgs a, int heads) {
  constexpr int RPW = 256 / D, WARPS = THREADS / 32, STEP = WARPS * RPW;
  extern __shared__ __align__(16) uint4 rows_in[];  // [ROWS][D / 8]: the rows, each thread's own chunks
  float4* cs = reinterpret_cast<float4*>(rows_in + ROWS * (D / 8));  // [ROWS][rot / 4], keys with a rotation
  __shared__ uint64_t turns[64];
  __shared__ float red[2][WARPS];
  pdl_wait();
  pdl_trigger();
  const AppUnit u = p.app_units[blockIdx.x];
  if (u.count == 0) return;
  const bool key = blockIdx.z == 0;
  const int phys = __ldg(a.page_table + (int64_t)u.req * p.max_pages + u.page);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / (D / 8), chunk = lane % (D / 8), row0 = warp * RPW + sub;
  const int g0 = blockIdx.y * heads, g1 = min(p.Hkv, g0 + heads);
  const uint16_t* src = key ? a.k : a.v;
  const int64_t stride = key ? a.k_stride : a.v_stride;
  auto load = [&](int g, int i) {  // this lane's chunk of row i, asynchronously
    if (i < u.count)
      async_copy16(smem_u32(rows_in + i * (D / 8) + chunk),
                   src + (u.tok0 + i) * stride + (int64_t)g * D + chunk * 8);
  };
  for (int i = row0; i < u.count; i += STEP) load(g0, i);
  const int entries = r.rot / 4;  // of a token
  KeyRows<D, INTER> rows;
  if (key) rows.make(r, a.k_weight, lane);
  if (key && entries) {
    stage_turns(r, turns);
    chunk_angles<INTER, THREADS>(r, p, u.tok0, u.page * kPage + u.slot0, u.count, turns,
                                 reinterpret_cast<float*>(cs));
    __syncthreads();
  }
  if (phys < 0 || phys >= p.num_phys) {
    if (threadIdx.x == 0) set_status(p.status, DEV_BAD_PAGE);
    async_wait_all();
    return;
  }
  uint8_t* cache = key ? a.kc : a.vc;
  float* scales = reinterpret_cast<float*>(key ? a.ks : a.vs);
  for (int g = g0; g < g1; ++g) {
    const int64_t tile = (int64_t)phys * p.Hkv + g;
    const float s_old = u.slot0 > 0 ? scales[tile] : 0.f;
    float amax = 0.f, s = 0.f, inv = 0.f;
    bool pow2 = true;
    uint8_t* dst = cache + (tile * 128 + u.slot0) * D + chunk * 8;
    async_wait_all();
    // The rows twice, for the maximum and for the codes: kept from one to the other they would take the
    // registers of half the warps, and a copy of the code for every row (read from memory where it runs
    // once: twice the time)
#pragma unroll 1
    for (int phase = 0; phase < 2; ++phase) {
#pragma unroll 1
      for (int i0 = warp * RPW; i0 < u.count; i0 += STEP) {  // (a warp's rows)
        const int i = i0 + sub;
        const uint4 raw = i < u.count ? rows_in[i * (D / 8) + chunk] : make_uint4(0, 0, 0, 0);
        uint64_t y[4];
        if (key) {
          rows.apply(raw, cs + min(i, u.count - 1) * entries, a.k_weight != nullptr, a.eps, y);
        } else {
          const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = pack_f32x2(bf16_lo(x[e]), bf16_hi(x[e]));
        }
        if (phase == 0) {
          // (a row behind the last is zero, or NaN of 0 / 0, which the maximum passes over)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo, hi;
            unpack_f32x2(y[e], lo, hi);
            amax = fmaxf(amax, fmaxf(fabsf(lo), fabsf(hi)));
          }
        } else if (i < u.count) {
          *reinterpret_cast<uint2*>(dst + i * D) = codes8(y, s, inv, pow2);
          if (g + 1 < g1) load(g + 1, i);  // (this thread has just read what lay there)
        }
      }
      if (phase) break;
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
      if (lane == 0) red[g & 1][warp] = amax;
      __syncthreads();
      amax = lane < WARPS ? red[g & 1][lane] : 0.f;
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
      s = fmaxf(s_old, pow2_scale(amax));
      pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
      inv = __frcp_rn(s);
      if (threadIdx.x == 0) scales[tile] = s;
    }
    if (u.slot0 > 0 && s > s_old) {  // the earlier rows follow the scale
      const float f = __fdiv_rn(s_old, s);
      uint2* old = reinterpret_cast<uint2*>(cache + tile * 128 * D);
      for (int i = threadIdx.x; i < u.slot0 * (D / 8); i += THREADS) {
        const uint2 c = old[i];
        const uint32_t w[2] = {c.x, c.y};
        uint32_t o[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t x = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) x |= f32_to_e4m3(e4m3_to_f32((w[e] >> (8 * b)) & 0xffu) * f) << (8 * b);
          o[e] = x;
        }
        old[i] = make_uint2(o[0], o[1]);
      }
    }
  }
}

// (page, head) tiles of K and V.
inline int64_t tiles(const DevPlan& p) { return 2ll * p.num_app_units * p.Hkv; }

template <int D, bool INTER, int THREADS, int ROWS>
cudaError_t run(const DevPlan& p, const DevRope& r, const KvRopeArgs& a, cudaStream_t st) {
  auto kern = kv_append_e4m3_kernel<D, INTER, THREADS, ROWS>;  // ROWS: of a page, at most
  const int smem = ROWS * (D * 2 + r.rot * 4);
  if (smem > 32 * 1024) {
    // the room of the largest rotation, whatever this one is: the limit is the kernel's, and another thread
    // may be between its own setting and its launch
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         ROWS * (D * 2 + D * 4));
    if (e != cudaSuccess) return e;
  }
  // heads a block: one, until the blocks fill the GPU several times; then a page's angles serve more
  const int64_t want = 4ll * num_sms();
  const int heads = (int)std::min<int64_t>(p.Hkv, std::max<int64_t>(1, tiles(p) / want));
  const dim3 grid((unsigned)p.num_app_units, (unsigned)((p.Hkv + heads - 1) / heads), 2);
  if (grid.y > 65535) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_pdl(kern, grid, dim3(THREADS), (size_t)smem, st, p, r, a, heads);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool INTER>
cudaError_t run_rows(const DevPlan& p, const DevRope& r, const KvRopeArgs& a, cudaStream_t st) {
  // Batches of few new tokens a request (a decode step) take small blocks; where the blocks find a place at
  // once, large ones, which are done sooner, else two to an SM.  (512 / 1024 threads: 4096 tokens of 2 heads,
  // 160 tiles, 11.5 / 8.1 us; 5.6K tokens of 8 heads, D 64, 752 tiles, 12.4 / 16.4; 65536 tokens of 8 heads
  // 153 / 195.)
  if (p.app_max_rows <= 8) return run<D, INTER, 128, 8>(p, r, a, st);
  if (tiles(p) <= 2ll * num_sms()) return run<D, INTER, 1024, 128>(p, r, a, st);
  return run<D, INTER, 512, 128>(p, r, a, st);
}

}  // namespace

cudaError_t launch_kv_append_e4m3(const DevPlan& p, const DevRope& r, const KvRopeArgs& a,
                                  bool interleaved, cudaStream_t st) {
  if (p.D == 128) return interleaved ? run_rows<128, true>(p, r, a, st) : run_rows<128, false>(p, r, a, st);
  return interleaved ? run_rows<64, true>(p, r, a, st) : run_rows<64, false>(p, r, a, st);
}

}  // namespace sps
