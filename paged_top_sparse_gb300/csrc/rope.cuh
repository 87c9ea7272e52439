// rope.cuh -- the rotation's device code, shared by the kernels that rotate rows (rope.cu,
// kvappend_e4m3.cu).
#pragma once
#include "ptx.cuh"
#include "sps_internal.h"

namespace sps {

// 2^64 / (2 pi), rounded down: one radian as a fraction of a turn.
constexpr uint64_t kTurn = 2935890503282001226ull;

// inv_freq (radians per position) as a fraction of a turn in units of 2^-64, modulo a turn.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t b = __float_as_uint(f);
  const int e = (b >> 23) & 0xff;
  const uint64_t m = e ? ((b & 0x7fffffu) | 0x800000u) : (b & 0x7fffffu);  // |f| = m 2^(e - 150)
  const int s = 150 - (e ? e : 1);
  const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
  uint64_t r;
  if (s >= 128) r = 0;
  else if (s >= 64) r = hi >> (s - 64);
  else if (s > 0) r = (lo >> s) | (hi << (64 - s));
  else r = s > -64 ? lo << -s : 0;
  return (b >> 31) ? 0 - r : r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// The pairs' frequencies as turn fractions, made once per block.
__device__ __forceinline__ void stage_turns(const DevRope& r, uint64_t* turns) {
  if ((int)threadIdx.x < r.rot / 2) turns[threadIdx.x] = turn_fraction(__ldg(r.inv_freq + threadIdx.x));
  __syncthreads();
}

// Cosine and sine of every pair of a token, by the whole warp.
__device__ __forceinline__ void token_angles(const DevRope& r, const DevPlan& p, int tok,
                                             const uint64_t* turns, float2* cs, int lane) {
  for (int j = lane; j < r.rot / 2; j += 32) {
    const int pos = r.positions ? __ldg(r.positions + (int64_t)r.axis[j] * p.T + tok)
                                : __ldg(p.tok_pos + tok);
    const uint64_t a = (uint64_t)(int64_t)pos * turns[j];
    // a half turn is 2^31 units of the top word: the argument of sin(pi x)
    sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &cs[j].y, &cs[j].x);
  }
  __syncwarp();
}

__device__ __forceinline__ void load_weights(const float* w, int d, float (&o)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 1.f;
  if (w) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4*>(o + 4 * i) = __ldg(reinterpret_cast<const float4*>(w + d) + i);
  }
}

// What a lane needs to rotate its chunk of 8 elements of any row of the token:
// y = x A + x_partner B, packed in pairs.
template <int D, bool INTER>
struct Rotation {
  uint64_t A[4], B[4];
  bool on;      // the chunk lies inside the rotated dims
  int partner;  // lane that holds the partner elements (half-split pairs)
  __device__ __forceinline__ void make(const DevRope& r, const float* w, const float2* cs, int lane) {
    const int chunk = lane % (D / 8), half = r.rot / 2, d0 = chunk * 8;
    on = d0 < r.rot;
    partner = lane;
    int p0 = d0;  // the partner elements' first dim
    if (!INTER && on) {
      partner = d0 < half ? lane + half / 8 : lane - half / 8;
      p0 = d0 < half ? d0 + half : d0 - half;
    }
    float own[8], other[8], t[16], a[8], b[8];  // t: cosine and sine of the chunk's pairs in turn
    load_weights(w, d0, own);
    if (INTER) {
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = own[e ^ 1];
    } else {
      load_weights(w, p0, other);
    }
    constexpr int NP = INTER ? 4 : 8;  // pairs of a chunk
    if (on) {
      const float4* c4 = reinterpret_cast<const float4*>(cs + (INTER ? d0 / 2 : min(d0, p0)));
#pragma unroll
      for (int i = 0; i < NP / 2; ++i) *reinterpret_cast<float4*>(t + 4 * i) = c4[i];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = INTER ? e / 2 : e;
      const bool first = INTER ? e % 2 == 0 : d0 < half;
      a[e] = on ? own[e] * t[2 * j] : own[e];
      b[e] = on ? other[e] * (first ? -t[2 * j + 1] : t[2 * j + 1]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      A[i] = pack_f32x2(a[2 * i], a[2 * i + 1]);
      B[i] = pack_f32x2(b[2 * i], b[2 * i + 1]);
    }
  }
  // This lane's chunk `raw` of a row, normalised (where `norm`), rotated and times `sign`; all 32
  // lanes call it.
  __device__ __forceinline__ void apply(const uint4& raw, bool norm, float eps, float sign,
                                        uint64_t (&y)[4]) const {
    const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
    uint64_t v[4];
    float scale = sign;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_f32x2(bf16_lo(x[i]), bf16_hi(x[i]));
    if (norm) {
      uint64_t s2 = mul_f32x2(v[0], v[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) s2 = fma_f32x2(v[i], v[i], s2);
      float lo, hi;
      unpack_f32x2(s2, lo, hi);
      float ss = lo + hi;
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      scale *= rsqrtf(fmaf(ss, 1.f / D, eps));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint64_t q;
      if (INTER) {
        q = pack_f32x2(bf16_hi(x[i]), bf16_lo(x[i]));
      } else {
        const uint32_t o = __shfl_sync(0xffffffffu, x[i], partner);
        q = pack_f32x2(bf16_lo(o), bf16_hi(o));
      }
      y[i] = mul_f32x2(v[i], A[i]);
      if (on) y[i] = fma_f32x2(q, B[i], y[i]);  // (a dim behind R must not meet 0 * infinity)
      y[i] = mul_f32x2(y[i], pack_f32x2(scale, scale));
    }
  }
};

}  // namespace sps
