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
// modulo 2^64 is the angle modulo a whole turn, without a reduction; its top 32 bits, rounded to FP32
// (2^-26 turns), go to sincospi.  F is off by at most |inv_freq| + 1 units (2^64 / 2 pi and the shift
// are cut off), so for inv_freq <= 1 the angle by 2^-32 turns at any 32-bit position.
//
// Layout: D / 8 lanes hold a row, 8 elements (16 bytes) each; a warp takes one token and walks its
// rows, 32 * 8 / D at a time, two such passes in flight.  Its lanes make the token's angles once
// (two pairs each) and hand them round through shared memory; weight, cosine and sine become two
// coefficients per element, so a row costs y = (x A + x_partner B) / rms.  Row sums and the partner
// halves travel by shuffles.
//
// Bound: memory for many tokens.  8192 tokens x 34 rows x 128 (143 MB): 28.6 us, 5.0 TB/s, 0.73
// of a plain copy; the rest is the start and end of a launch of 20 us of work (32768 tokens x 40
// rows: 111 us, 6.0 TB/s, 0.89) and the angles in front of a token's rows.  With the angles and
// coefficients made per row group instead of per token an earlier form took 41.7 us.  5.6K tokens x 28
// rows to E4M3 on three axes: 22.2 us, 0.53 of a copy (more arithmetic for fewer bytes).  64 tokens
// (1.1 MB): 2.8 us, a launch and a chain of three dependent reads.  Append: 65536 tokens of 8 heads
// (537 MB) into a BF16 cache 104 us, 5.2 TB/s; into an NVFP4 cache 147 us, the divisions of its rule.
// More passes in flight cost resident warps, larger blocks leave more of them idle at the end: 8192
// tokens four passes 29.9 us, eight 33.9, blocks of 8 warps 34.2; E4M3 26.4, 29.3 and 25.0.
#include <algorithm>
#include <cstring>

#include "rope.cuh"

namespace sps {
namespace {

constexpr int kWarps = 4;  // per block

// A warp's rows [r0, r1) of one kind, kInFlight passes at a time; the next ones are loaded before the
// present ones' arithmetic, the first ones when the walk is made (ahead of the token's angles).
constexpr int kInFlight = 2;
template <int D, typename Load>
struct RowWalk {
  static constexpr int RPW = 256 / D;
  Load load;
  int r0, r1, sub;
  uint4 raw[kInFlight];
  __device__ __forceinline__ RowWalk(Load f, int b, int e, int s) : load(f), r0(b), r1(e), sub(s) {
    fetch(r0, raw);
  }
  __device__ __forceinline__ void fetch(int base, uint4 (&x)[kInFlight]) const {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int row = base + k * RPW + sub;
      x[k] = row < r1 ? load(row) : make_uint4(0, 0, 0, 0);
    }
  }
  template <typename Body>
  __device__ __forceinline__ void run(Body body) {
    for (int base = r0; base < r1; base += kInFlight * RPW) {
      uint4 next[kInFlight];
      fetch(base + kInFlight * RPW, next);
#pragma unroll
      for (int k = 0; k < kInFlight; ++k)
        if (base + k * RPW < r1) body(base + k * RPW + sub, raw[k]);
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) raw[k] = next[k];
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  float a, b;
  unpack_f32x2(v, a, b);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// E4M3 codes of -y / s, the quotient rounded to FP32 first as sps_quantize_e4m3 does it (it decides
// the codes next to a border).
//
// A division costs ten instructions an element (5.6K tokens x 28 rows: 28.5 us, and 20.3 by a product
// with the rounded 1 / s alone), so a quotient is made of products, in pairs (P. Markstein, IBM J.
// Res. Dev. 34, 1990): q = y (hi + lo), hi + lo = 1 / s to 2^-47, is off by little more than half a unit
// in the last place; the remainder q s - y of such a q is exact, and q - (q s - y) r with r = 1 / s
// rounded to nearest is the rounded quotient.  hi is rounded towards zero, so that lo has its sign: with
// y negated in advance a zero then keeps its own.  Where a product is infinite there is no remainder,
// and where s is so small or large that remainders or r lose bits the host passes NaN for r: these take
// the division.
__device__ __forceinline__ void e4m3_codes(const uint64_t (&y)[4], const DevQuot& d, uint32_t (&o)[2]) {
  const uint64_t s2 = pack_f32x2(d.s, d.s), nr = pack_f32x2(-d.r, -d.r);
  const uint64_t nhi = pack_f32x2(-d.hi, -d.hi), nlo = pack_f32x2(-d.lo, -d.lo);
  uint64_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = fma_f32x2(y[i], nhi, mul_f32x2(y[i], nlo));
    q[i] = fma_f32x2(fma_f32x2(q[i], s2, y[i]), nr, q[i]);
  }
  float lo, hi;
  unpack_f32x2(add_f32x2(add_f32x2(q[0], q[1]), add_f32x2(q[2], q[3])), lo, hi);
  if (!(fabsf(lo + hi) <= 3.4e38f)) {  // an infinity became NaN (or large quotients' sum overflowed)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack_f32x2(y[i], lo, hi);
      q[i] = pack_f32x2(__fdiv_rn(-lo, d.s), __fdiv_rn(-hi, d.s));
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) o[h] = f32x2_to_e4m3x2(q[2 * h]) | (f32x2_to_e4m3x2(q[2 * h + 1]) << 16);
}

// The rows [r0, r1) of one kind that warp `part` of a token walks; `at` counts the passes of the
// kinds before it.
template <int D>
__device__ __forceinline__ void my_rows(int part, int per, int rows, int& at, int& r0, int& r1) {
  constexpr int RPW = 256 / D;
  const int passes = (rows + RPW - 1) / RPW;
  const int b = max(0, part * per - at), e = min(passes, (part + 1) * per - at);
  at += passes;
  r0 = b * RPW;
  r1 = b < e ? min(rows, e * RPW) : r0;
}

// One warp: one token, some of its rows: the H query rows, then the G key rows.
template <int D, bool INTER, bool E4M3OUT>
__global__ void __launch_bounds__(kWarps * 32)
qk_norm_rope_kernel(DevPlan p, const __grid_constant__ DevRope r, QkRopeArgs a) {
  __shared__ uint64_t turns[64];
  __shared__ __align__(16) float2 cs[kWarps][64];
  pdl_wait();
  pdl_trigger();
  stage_turns(r, turns);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int tok = (int)(w / a.splits), part = (int)(w % a.splits);
  if (tok >= p.T) return;
  const int sub = lane / (D / 8), chunk = lane % (D / 8);
  int at = 0, q0, q1, k0, k1;
  my_rows<D>(part, a.passes, p.H, at, q0, q1);
  my_rows<D>(part, a.passes, a.k ? p.Hkv : 0, at, k0, k1);
  const uint16_t* qsrc = a.q + tok * a.q_stride + chunk * 8;
  const uint16_t* ksrc = a.k + tok * a.k_stride + chunk * 8;
  auto qload = [&](int row) { return *reinterpret_cast<const uint4*>(qsrc + (int64_t)row * D); };
  auto kload = [&](int row) { return *reinterpret_cast<const uint4*>(ksrc + (int64_t)row * D); };
  RowWalk<D, decltype(qload)> qw(qload, q0, q1, sub);
  token_angles(r, p, tok, turns, cs[warp], lane);
  Rotation<D, INTER> rt;
  uint64_t y[4];
  if (q0 < q1) {
    rt.make(r, a.q_weight, cs[warp], lane);
    uint8_t* dst = static_cast<uint8_t*>(a.q_out) +
                   (tok * a.q_out_stride + chunk * 8) * (E4M3OUT ? 1 : 2);
    qw.run([&](int row, const uint4& raw) {
      rt.apply(raw, a.q_weight != nullptr, a.eps, E4M3OUT ? -1.f : 1.f, y);
      if (row >= q1) return;
      if (E4M3OUT) {
        uint32_t o[2];
        e4m3_codes(y, a.q_scale, o);
        *reinterpret_cast<uint2*>(dst + (int64_t)row * D) = make_uint2(o[0], o[1]);
      } else {
        *reinterpret_cast<uint4*>(dst + (int64_t)row * D * 2) =
            make_uint4(pack_bf16(y[0]), pack_bf16(y[1]), pack_bf16(y[2]), pack_bf16(y[3]));
      }
    });
  }
  if (k0 < k1) {
    RowWalk<D, decltype(kload)> kw(kload, k0, k1, sub);
    rt.make(r, a.k_weight, cs[warp], lane);
    uint16_t* dst = a.k_out + tok * a.k_out_stride + chunk * 8;
    kw.run([&](int row, const uint4& raw) {
      rt.apply(raw, a.k_weight != nullptr, a.eps, 1.f, y);
      if (row < k1)
        *reinterpret_cast<uint4*>(dst + (int64_t)row * D) =
            make_uint4(pack_bf16(y[0]), pack_bf16(y[1]), pack_bf16(y[2]), pack_bf16(y[3]));
    });
  }
}

// 16 elements (two lanes' chunks) as NVFP4: codes of this lane's 8, and the block's scale.  The
// rule is sps_kv_append's, divisions included.
__device__ __forceinline__ uint32_t nvfp4_codes(const float (&y)[8], uint32_t& scode) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  scode = f32_to_e4m3(__fdiv_rn(amax, 6.0f));
  const float sv = e4m3_to_f32(scode);
  uint32_t packed = 0;
  if (sv != 0.f) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      packed |= f32x2_to_e2m1x2(__fdiv_rn(y[e], sv), __fdiv_rn(y[e + 1], sv)) << (4 * e);
  }
  return packed;
}

// One warp: one token, some of its 2 G rows: the G key rows, then the G value rows.
template <int D, bool INTER, bool NVFP4>
__global__ void __launch_bounds__(kWarps * 32)
kv_append_rope_kernel(DevPlan p, const __grid_constant__ DevRope r, KvRopeArgs a) {
  __shared__ uint64_t turns[64];
  __shared__ __align__(16) float2 cs[kWarps][64];
  pdl_wait();
  pdl_trigger();
  stage_turns(r, turns);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int tok = (int)(w / a.splits), part = (int)(w % a.splits);
  if (tok >= p.T) return;
  const int G = p.Hkv, sub = lane / (D / 8), chunk = lane % (D / 8);
  const int t = __ldg(p.tok_pos + tok), req = __ldg(p.tok_req + tok);
  const int phys = __ldg(a.page_table + (int64_t)req * p.max_pages + (t >> 7));
  int at = 0, k0, k1, v0, v1;
  my_rows<D>(part, a.passes, G, at, k0, k1);
  my_rows<D>(part, a.passes, G, at, v0, v1);
  const uint16_t* ksrc = a.k + tok * a.k_stride + chunk * 8;
  const uint16_t* vsrc = a.v + tok * a.v_stride + chunk * 8;
  auto kload = [&](int row) { return *reinterpret_cast<const uint4*>(ksrc + (int64_t)row * D); };
  auto vload = [&](int row) { return *reinterpret_cast<const uint4*>(vsrc + (int64_t)row * D); };
  RowWalk<D, decltype(kload)> kw(kload, k0, k1, sub);
  Rotation<D, INTER> rt;
  if (k0 < k1) {
    token_angles(r, p, tok, turns, cs[warp], lane);
    rt.make(r, a.k_weight, cs[warp], lane);
  }
  if (phys < 0 || phys >= p.num_phys) {
    if (lane == 0) set_status(p.status, DEV_BAD_PAGE);
    return;
  }
  const int64_t slot0 = (int64_t)phys * G * 128 + (t & 127);  // slot of head g: + 128 g
  auto quantised = [&](int row, const float (&y)[8], uint8_t* codes, uint8_t* scales, bool live) {
    uint32_t scode;
    const uint32_t packed = nvfp4_codes(y, scode);
    if (!live) return;
    const int64_t slot = slot0 + 128 * row;
    *reinterpret_cast<uint32_t*>(codes + slot * (D / 2) + chunk * 4) = packed;
    if (chunk % 2 == 0) scales[slot * (D / 16) + chunk / 2] = (uint8_t)scode;
  };
  kw.run([&](int row, const uint4& raw) {
    uint64_t y[4];
    rt.apply(raw, a.k_weight != nullptr, a.eps, 1.f, y);
    if (NVFP4) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack_f32x2(y[i], f[2 * i], f[2 * i + 1]);
      quantised(row, f, a.kc, a.ks, row < k1);
    } else if (row < k1) {
      *reinterpret_cast<uint4*>(a.kc + ((slot0 + 128 * row) * D + chunk * 8) * 2) =
          make_uint4(pack_bf16(y[0]), pack_bf16(y[1]), pack_bf16(y[2]), pack_bf16(y[3]));
    }
  });
  RowWalk<D, decltype(vload)> vw(vload, v0, v1, sub);
  vw.run([&](int row, const uint4& raw) {  // value rows as they are
    if (NVFP4) {
      const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(x[i]);
        f[2 * i + 1] = bf16_hi(x[i]);
      }
      quantised(row, f, a.vc, a.vs, row < v1);
    } else if (row < v1) {
      *reinterpret_cast<uint4*>(a.vc + ((slot0 + 128 * row) * D + chunk * 8) * 2) = raw;
    }
  });
}

// Passes a warp walks: all of a token's where that gives every SM 24 warps, else fewer, so that a
// batch of few tokens still spreads over the GPU (a decode step of 64 tokens: a warp per pass).
// From 20 to 32 warps measures the same; 64 as the target splits tokens that need not be, 31.0
// against 28.6 us for 8192 tokens, since each part makes the token's angles again.
template <typename K, typename A>
cudaError_t launch_rows(K kern, const DevPlan& p, const DevRope& r, A a, int passes,
                        cudaStream_t st) {
  const int64_t want = 24LL * num_sms();
  const int64_t s = std::min<int64_t>(passes, std::max<int64_t>(1, (want + p.T - 1) / p.T));
  a.passes = (int)((passes + s - 1) / s);
  a.splits = (passes + a.passes - 1) / a.passes;
  const int64_t blocks = ((int64_t)p.T * a.splits + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)blocks), dim3(kWarps * 32), 0, st, p, r, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const DevPlan& p, const DevRope& r, const QkRopeArgs& a,
                                bool interleaved, bool e4m3, cudaStream_t st) {
  const int rpw = 256 / p.D;
  const int passes = (p.H + rpw - 1) / rpw + (a.k ? (p.Hkv + rpw - 1) / rpw : 0);
#define SPS_QK(DD, II, EE) \
  return launch_rows(qk_norm_rope_kernel<DD, II, EE>, p, r, a, passes, st)
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
  const int rpw = 256 / p.D, passes = 2 * ((p.Hkv + rpw - 1) / rpw);
#define SPS_KV(DD, II, NN) \
  return launch_rows(kv_append_rope_kernel<DD, II, NN>, p, r, a, passes, st)
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
