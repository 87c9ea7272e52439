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
// Layout.  A block takes a touched page (the plan's list) and some of its heads, K or V: D / 8 lanes
// hold a row, 8 elements (16 bytes) each, and the page's rows stay in registers between the maximum and
// the codes, so each is read once.
#include <algorithm>

#include "rope.cuh"

namespace sps {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
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

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads)
kv_append_e4m3_kernel(DevPlan p, const __grid_constant__ DevRope r, KvRopeArgs a, int heads) {
  constexpr int RPW = 256 / D, STEP = kWarps * RPW, PASSES = 128 / STEP;
  extern __shared__ __align__(16) float2 cs[];  // [rows][rot / 2], keys with a rotation
  __shared__ uint64_t turns[64];
  __shared__ float red[2][kWarps];
  pdl_wait();
  pdl_trigger();
  const AppUnit u = p.app_units[blockIdx.x];
  if (u.count == 0) return;
  const bool key = blockIdx.z == 0;
  const int phys = __ldg(a.page_table + (int64_t)u.req * p.max_pages + u.page);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (phys < 0 || phys >= p.num_phys) {
    if (threadIdx.x == 0) set_status(p.status, DEV_BAD_PAGE);
    return;
  }
  const int half = r.rot / 2;
  if (key && half) {
    stage_turns(r, turns);
    for (int i = warp; i < u.count; i += kWarps)
      token_angles(r, p, u.tok0 + i, turns, cs + i * half, lane);
    __syncthreads();
  }
  const int sub = lane / (D / 8), chunk = lane % (D / 8), row0 = warp * RPW + sub;
  const uint16_t* src = (key ? a.k : a.v) + chunk * 8;
  const int64_t stride = key ? a.k_stride : a.v_stride;
  uint8_t* cache = key ? a.kc : a.vc;
  float* scales = reinterpret_cast<float*>(key ? a.ks : a.vs);
  const int h1 = min(p.Hkv, (int)(blockIdx.y + 1) * heads);
  for (int g = blockIdx.y * heads; g < h1; ++g) {
    const int64_t tile = (int64_t)phys * p.Hkv + g;
    const float s_old = u.slot0 > 0 ? scales[tile] : 0.f;
    uint64_t y[PASSES][4];
    uint4 raw[PASSES];
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      const int i = k * STEP + row0;
      raw[k] = i < u.count ? *reinterpret_cast<const uint4*>(src + (u.tok0 + i) * stride + (int64_t)g * D)
                           : make_uint4(0, 0, 0, 0);
    }
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      if (k * STEP + warp * RPW >= u.count) {  // (the whole warp)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[k][e] = 0;
        continue;
      }
      if (key) {
        Rotation<D, INTER> rt;
        rt.make(r, a.k_weight, cs + min(k * STEP + row0, u.count - 1) * half, lane);
        rt.apply(raw[k], a.k_weight != nullptr, a.eps, 1.f, y[k]);
      } else {
        const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) y[k][e] = pack_f32x2(bf16_lo(x[e]), bf16_hi(x[e]));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo, hi;
        unpack_f32x2(y[k][e], lo, hi);
        amax = fmaxf(amax, fmaxf(fabsf(lo), fabsf(hi)));
      }
    }
    // (a row behind the last repeats nothing: its raw bits are zero, so is its result)
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if (lane == 0) red[g & 1][warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, red[g & 1][w]);
    const float s = fmaxf(s_old, pow2_scale(amax));
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
    const float inv = __frcp_rn(s);
    if (threadIdx.x == 0) scales[tile] = s;
    uint8_t* dst = cache + (tile * 128 + u.slot0) * D + chunk * 8;
#pragma unroll
    for (int k = 0; k < PASSES; ++k) {
      const int i = k * STEP + row0;
      if (i < u.count) *reinterpret_cast<uint2*>(dst + i * D) = codes8(y[k], s, inv, pow2);
    }
    if (u.slot0 > 0 && s > s_old) {  // the earlier rows follow the scale
      const float f = __fdiv_rn(s_old, s);
      uint2* old = reinterpret_cast<uint2*>(cache + tile * 128 * D);
      for (int i = threadIdx.x; i < u.slot0 * (D / 8); i += kThreads) {
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

template <int D, bool INTER>
cudaError_t run(const DevPlan& p, const DevRope& r, const KvRopeArgs& a, cudaStream_t st) {
  auto kern = kv_append_e4m3_kernel<D, INTER>;
  const int smem = 128 * (r.rot / 2) * (int)sizeof(float2);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
  if (e != cudaSuccess) return e;
  // heads a block: one, until the blocks fill the GPU several times; then a page's angles serve more
  const int64_t blocks = 2ll * p.num_app_units * p.Hkv, want = 8ll * num_sms();
  const int heads = (int)std::min<int64_t>(p.Hkv, std::max<int64_t>(1, blocks / want));
  const dim3 grid((unsigned)p.num_app_units, (unsigned)((p.Hkv + heads - 1) / heads), 2);
  if (grid.y > 65535) return cudaErrorInvalidConfiguration;
  e = launch_pdl(kern, grid, dim3(kThreads), (size_t)smem, st, p, r, a, heads);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append_e4m3(const DevPlan& p, const DevRope& r, const KvRopeArgs& a,
                                  bool interleaved, cudaStream_t st) {
  if (p.D == 128) return interleaved ? run<128, true>(p, r, a, st) : run<128, false>(p, r, a, st);
  return interleaved ? run<64, true>(p, r, a, st) : run<64, false>(p, r, a, st);
}

}  // namespace sps
