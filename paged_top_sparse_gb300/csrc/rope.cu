// rope.cu -- the norm and rotation of queries and keys, alone (sps_qk_norm_rope) and on the way
// into the paged cache (sps_kv_append_rope).
//
// Mathematics, per (token, head) row x of D elements, in FP32 with one rounding at the end:
//   n_d = x_d * w_d / sqrt(mean_d x_d^2 + eps)            (n = x where there is no weight)
//   (y_a, y_b) = (n_a cos - n_b sin, n_b cos + n_a sin)   for the pair (a, b) of index j < R/2,
//   (a, b) = (j, j + R/2) or (2j, 2j + 1), angle = position[axis_j] * inv_freq[j]; y_d = n_d for
//   d >= R.
// The angle of a far position does not fit FP32 (a position of 2^20 leaves 2^-4 of a radian), so
// it is kept as a 64-bit fraction of a turn: F = inv_freq / 2 pi in 2^-64 turns, and position * F
// modulo 2^64 is the angle modulo a whole turn, without a reduction; its top 32 bits go to
// sincospi.  F is off by at most two units for inv_freq <= 1, so the angle by 2^-31 turns for any
// 32-bit position.
//
// Layout: D / 8 lanes hold a row, 8 elements (16 bytes) each; a warp takes one token and walks
// its rows, 32 * 8 / D at a time, so a token's angles are made once for all its heads.  Row sums
// and the partner halves of a rotation travel by shuffles.
#include <algorithm>
#include <cstring>

#include "ptx.cuh"
#include "sps_internal.h"

namespace sps {
namespace {

constexpr int kWarps = 4;  // per block

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
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// This lane's share of a token's rotation: cosines and sines of its 8 elements (half-split pairs:
// the sine carries the sign of its half; interleaved: entry 2 i serves the pair 2 i, 2 i + 1).
template <int D, bool INTER>
struct Rotation {
  float c[8], s[8];
  bool on;       // this chunk lies inside the rotated dims
  int partner;   // lane that holds the other elements of this chunk's pairs
  __device__ void make(const DevRope& r, const DevPlan& p, int tok, int lane) {
    constexpr int L = D / 8;
    const int chunk = lane % L, half = r.rot / 2;
    on = chunk * 8 < r.rot;
    partner = lane;
    if (!INTER && on) partner = chunk * 8 < half ? lane + half / 8 : lane - half / 8;
    if (!on) return;
#pragma unroll
    for (int e = 0; e < 8; e += INTER ? 2 : 1) {
      const int d = chunk * 8 + e;
      const int j = INTER ? d / 2 : (d < half ? d : d - half);
      const int pos = r.positions ? __ldg(r.positions + (int64_t)r.axis[j] * p.T + tok)
                                  : __ldg(p.tok_pos + tok);
      const uint64_t a = (uint64_t)(int64_t)pos * turn_fraction(__ldg(r.inv_freq + j));
      // a half turn is 2^31 units of the top word: the argument of sin(pi x)
      sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &s[e], &c[e]);
      if (!INTER && d < half) s[e] = -s[e];
    }
  }
};

// Norm (where `norm`) and rotation (where `rotate`) of this lane's chunk of a row, `w` its weights
// in shared memory (ones without a norm); all 32 lanes call it, whatever their flags.
template <int D, bool INTER>
__device__ __forceinline__ void norm_rotate(const uint4& raw, const float* w, bool norm, float eps,
                                            const Rotation<D, INTER>& rt, bool rotate, int lane,
                                            float (&y)[8]) {
  constexpr int L = D / 8;
  const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
  float inv = 1.f;
  if (__any_sync(0xffffffffu, norm)) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ss = fmaf(bf16_lo(x[i]), bf16_lo(x[i]), ss);
      ss = fmaf(bf16_hi(x[i]), bf16_hi(x[i]), ss);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (norm) inv = rsqrtf(fmaf(ss, 1.f / D, eps));
  }
  auto scaled = [&](const uint32_t (&v)[4], int chunk, float (&o)[8]) {
    const float4 w0 = *reinterpret_cast<const float4*>(w + chunk * 8);
    const float4 w1 = *reinterpret_cast<const float4*>(w + chunk * 8 + 4);
    const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = bf16_lo(v[i]) * inv * ww[2 * i];
      o[2 * i + 1] = bf16_hi(v[i]) * inv * ww[2 * i + 1];
    }
  };
  scaled(x, lane % L, y);
  if (INTER) {
    if (rotate && rt.on) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float a = y[e], b = y[e + 1];
        y[e] = a * rt.c[e] - b * rt.s[e];
        y[e + 1] = b * rt.c[e] + a * rt.s[e];
      }
    }
  } else {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], rt.partner);
    if (rotate && rt.on) {
      float q[8];
      scaled(o, rt.partner % L, q);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * rt.c[e] + q[e] * rt.s[e];
    }
  }
}

// The block's copy of a weight in shared memory: ones where there is no norm.
template <int D>
__device__ __forceinline__ void stage_weight(const float* w, float* sm) {
  for (int i = threadIdx.x; i < D; i += blockDim.x) sm[i] = w ? __ldg(w + i) : 1.f;
}

// One warp: one token, some of its rows: the H query rows, then the G key rows.
template <int D, bool INTER, bool E4M3OUT>
__global__ void __launch_bounds__(kWarps * 32)
qk_norm_rope_kernel(DevPlan p, DevRope r, QkRopeArgs a) {
  constexpr int L = D / 8, RPW = 32 / L;
  __shared__ __align__(16) float sw[2][D];
  pdl_wait();
  pdl_trigger();
  stage_weight<D>(a.q_weight, sw[0]);
  stage_weight<D>(a.k_weight, sw[1]);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int tok = (int)(w / a.splits), part = (int)(w % a.splits);
  if (tok >= p.T) return;
  const int rows = p.H + (a.k ? p.Hkv : 0);
  const int r0 = part * a.rows_per_warp, r1 = min(rows, r0 + a.rows_per_warp);
  if (r0 >= r1) return;
  const int sub = lane / L, chunk = lane % L;
  auto src_of = [&](int row) {
    return row < p.H ? a.q + tok * a.q_stride + (int64_t)row * D
                     : a.k + tok * a.k_stride + (int64_t)(row - p.H) * D;
  };
  // the next rows are in flight while the angles are made and the present ones are rotated
  uint4 nxt = make_uint4(0, 0, 0, 0);
  if (r0 + sub < r1) nxt = *reinterpret_cast<const uint4*>(src_of(r0 + sub) + chunk * 8);
  Rotation<D, INTER> rt;
  rt.make(r, p, tok, lane);
  for (int base = r0; base < r1; base += RPW) {
    const int row = base + sub;
    const uint4 raw = nxt;
    if (row + RPW < r1) nxt = *reinterpret_cast<const uint4*>(src_of(row + RPW) + chunk * 8);
    float y[8];
    const bool is_q = row < p.H;
    norm_rotate<D, INTER>(raw, sw[is_q ? 0 : 1], (is_q ? a.q_weight : a.k_weight) != nullptr, a.eps,
                          rt, true, lane, y);
    if (row >= r1) continue;
    if (E4M3OUT && is_q) {
      uint32_t o[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        o[h] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[h] |= f32_to_e4m3(__fdiv_rn(y[4 * h + e], a.q_scale)) << (8 * e);
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.q_out) + tok * a.q_out_stride +
                                (int64_t)row * D + chunk * 8) = make_uint2(o[0], o[1]);
    } else {
      uint16_t* dst = is_q ? static_cast<uint16_t*>(a.q_out) + tok * a.q_out_stride + (int64_t)row * D
                           : a.k_out + tok * a.k_out_stride + (int64_t)(row - p.H) * D;
      *reinterpret_cast<uint4*>(dst + chunk * 8) =
          make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                     pack_bf16(y[6], y[7]));
    }
  }
}

// One warp: one token, some of its 2 G rows (the G key rows, then the G value rows).
template <int D, bool INTER, bool NVFP4>
__global__ void __launch_bounds__(kWarps * 32)
kv_append_rope_kernel(DevPlan p, DevRope r, KvRopeArgs a) {
  constexpr int L = D / 8, RPW = 32 / L;
  __shared__ __align__(16) float sw[D];
  pdl_wait();
  pdl_trigger();
  stage_weight<D>(a.k_weight, sw);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int tok = (int)(w / a.splits), part = (int)(w % a.splits);
  if (tok >= p.T) return;
  const int G = p.Hkv, rows = 2 * G;
  const int r0 = part * a.rows_per_warp, r1 = min(rows, r0 + a.rows_per_warp);
  if (r0 >= r1) return;
  const int t = __ldg(p.tok_pos + tok), req = __ldg(p.tok_req + tok);
  const int phys = __ldg(a.page_table + (int64_t)req * p.max_pages + (t >> 7));
  const int sub = lane / L, chunk = lane % L;
  auto load = [&](int row) {
    const uint16_t* s = row < G ? a.k + tok * a.k_stride + (int64_t)row * D
                                : a.v + tok * a.v_stride + (int64_t)(row - G) * D;
    return *reinterpret_cast<const uint4*>(s + chunk * 8);
  };
  uint4 nxt = make_uint4(0, 0, 0, 0);
  if (r0 + sub < r1) nxt = load(r0 + sub);
  Rotation<D, INTER> rt;
  if (r0 < G) rt.make(r, p, tok, lane);
  else rt.on = false, rt.partner = lane;
  if (phys < 0 || phys >= p.num_phys) {
    if (lane == 0) set_status(p.status, DEV_BAD_PAGE);
    return;
  }
  for (int base = r0; base < r1; base += RPW) {
    const int row = base + sub;
    const bool is_k = row < G;
    const uint4 raw = nxt;
    if (row + RPW < r1) nxt = load(row + RPW);
    float y[8];
    if (__any_sync(0xffffffffu, is_k))
      norm_rotate<D, INTER>(raw, sw, a.k_weight != nullptr, a.eps, rt, is_k, lane, y);
    if (!is_k) {  // a value row as it is
      const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf16_lo(x[i]);
        y[2 * i + 1] = bf16_hi(x[i]);
      }
    }
    const int64_t slot = ((int64_t)phys * G + (is_k ? row : row - G)) * 128 + (t & 127);
    if (!NVFP4) {
      if (row < r1)
        *reinterpret_cast<uint4*>((is_k ? a.kc : a.vc) + (slot * D + chunk * 8) * 2) =
            is_k ? make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                              pack_bf16(y[6], y[7]))
                 : raw;
      continue;
    }
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // 16 elements: two lanes
    if (row >= r1) continue;
    const uint32_t scode = f32_to_e4m3(__fdiv_rn(amax, 6.0f));
    const float sv = e4m3_to_f32(scode);
    uint32_t packed = 0;
    if (sv != 0.f) {
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        packed |= f32x2_to_e2m1x2(__fdiv_rn(y[e], sv), __fdiv_rn(y[e + 1], sv)) << (4 * e);
    }
    *reinterpret_cast<uint32_t*>((is_k ? a.kc : a.vc) + slot * (D / 2) + chunk * 4) = packed;
    if (chunk % 2 == 0) (is_k ? a.ks : a.vs)[slot * (D / 16) + chunk / 2] = (uint8_t)scode;
  }
}

// Rows a warp walks: all of a token's where that gives every SM 32 warps, else fewer, so that a
// batch of few tokens still spreads over the GPU (a decode step of 64 tokens: a warp per pass).
int split_rows(int64_t tokens, int rows, int rpw, int* splits) {
  const int passes = (rows + rpw - 1) / rpw;
  const int64_t want = 32LL * num_sms();
  const int64_t s = std::min<int64_t>(passes, std::max<int64_t>(1, (want + tokens - 1) / tokens));
  const int per = (int)((passes + s - 1) / s);
  *splits = (passes + per - 1) / per;
  return per * rpw;
}

template <typename K, typename A>
cudaError_t launch_rows(K kern, const DevPlan& p, const DevRope& r, A a, int rows, int rpw,
                        cudaStream_t st) {
  a.rows_per_warp = split_rows(p.T, rows, rpw, &a.splits);
  const int64_t blocks = ((int64_t)p.T * a.splits + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kWarps * 32), 0, st, p, r, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const DevPlan& p, const DevRope& r, const QkRopeArgs& a,
                                bool interleaved, bool e4m3, cudaStream_t st) {
  const int rows = p.H + (a.k ? p.Hkv : 0);
#define SPS_QK(DD, II, EE) \
  return launch_rows(qk_norm_rope_kernel<DD, II, EE>, p, r, a, rows, 256 / DD, st)
  if (p.D == 128) {
    if (interleaved) { if (e4m3) SPS_QK(128, true, true); else SPS_QK(128, true, false); }
    else { if (e4m3) SPS_QK(128, false, true); else SPS_QK(128, false, false); }
  } else {
    if (interleaved) { if (e4m3) SPS_QK(64, true, true); else SPS_QK(64, true, false); }
    else { if (e4m3) SPS_QK(64, false, true); else SPS_QK(64, false, false); }
  }
#undef SPS_QK
}

cudaError_t launch_kv_append_rope(const DevPlan& p, const DevRope& r, const KvRopeArgs& a,
                                  bool interleaved, bool nvfp4, cudaStream_t st) {
  const int rows = 2 * p.Hkv;
#define SPS_KV(DD, II, NN) \
  return launch_rows(kv_append_rope_kernel<DD, II, NN>, p, r, a, rows, 256 / DD, st)
  if (p.D == 128) {
    if (interleaved) { if (nvfp4) SPS_KV(128, true, true); else SPS_KV(128, true, false); }
    else { if (nvfp4) SPS_KV(128, false, true); else SPS_KV(128, false, false); }
  } else {
    if (interleaved) { if (nvfp4) SPS_KV(64, true, true); else SPS_KV(64, true, false); }
    else { if (nvfp4) SPS_KV(64, false, true); else SPS_KV(64, false, false); }
  }
#undef SPS_KV
}

}  // namespace sps
