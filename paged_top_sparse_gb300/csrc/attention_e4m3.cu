// attention_e4m3.cu -- full causal attention over a paged cache held in 8 bits (E4M3 codes, one FP32
// scale for each page and KV head): out_r = sum_j p_j vs_j v_j / sum_j p_j with
// p_j = 2^(c ks_j q_r . k_j - m), c = scale * q_scale * log2 e, and the log-sum-exp.
//
// The plain form: a warp per (token, head) row walks its request's keys four at a time, a lane holding
// D / 32 dims of q and of the output, with a running maximum and sum in FP32.
#include "attention.cuh"

namespace sps {
namespace att {
namespace {

constexpr int kWarps = 8;

// D / 32 consecutive codes at p as FP32.
template <int E>
__device__ __forceinline__ void load_codes(const uint8_t* p, float (&o)[E]) {
  uint32_t w = E == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = e4m3_to_f32((w >> (8 * e)) & 0xffu);
}

template <int D, bool QE4M3>
__global__ void __launch_bounds__(kWarps * 32)
attention_e4m3_kernel(DevPlan p, AttArgs a) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= (int64_t)p.T * p.H) return;
  const int tok = (int)(row / p.H), head = (int)(row % p.H), g = head / p.Hg;
  const int pos = __ldg(p.tok_pos + tok), req = __ldg(p.tok_req + tok);
  const float* ks = reinterpret_cast<const float*>(a.ks);
  const float* vs = reinterpret_cast<const float*>(a.vs);
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  const int64_t at = tok * a.q_stride + (int64_t)head * D + lane * E;
  if (QE4M3) {
    load_codes<E>(a.q + at, q);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = bf16_to_f32(reinterpret_cast<const uint16_t*>(a.q)[at + e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int page = 0; page <= pos >> 7; ++page) {
    const int phys = __ldg(a.page_table + (int64_t)req * p.max_pages + page);
    if (phys < 0 || phys >= p.num_phys) {
      if (lane == 0) set_status(p.status, DEV_BAD_PAGE);
      return;
    }
    const int64_t tile = (int64_t)phys * p.Hkv + g;
    const float ck = a.c * ks[tile], vscale = vs[tile];
    const int n = min(128, pos - page * 128 + 1);
    for (int j0 = 0; j0 < n; j0 += 4) {
      float s[4], v[4][E];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = 0.f;
        if (j0 + j < n) {
          float k[E];
          load_codes<E>(a.kc + (tile * 128 + j0 + j) * D + lane * E, k);
          load_codes<E>(a.vc + (tile * 128 + j0 + j) * D + lane * E, v[j]);
#pragma unroll
          for (int e = 0; e < E; ++e) s[j] += q[e] * k[e];
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
      float mx = m;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = j0 + j < n ? s[j] * ck : -INFINITY;
        mx = fmaxf(mx, s[j]);
      }
      const float f = exp2f(m - mx);
      m = mx;
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j < n) {
          const float x = exp2f(s[j] - m);
          l += x;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += x * vscale * v[j][e];
        }
    }
  }
  uint16_t* out = a.out + tok * a.out_stride + (int64_t)head * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(out + e) = pack_p<false>(acc[e] / l, acc[e + 1] / l);
  if (lane == 0 && a.out_lse) a.out_lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool QE4M3>
cudaError_t run(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  const int64_t blocks = ((int64_t)p.T * p.H + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_pdl(attention_e4m3_kernel<D, QE4M3>, dim3((unsigned)blocks),
                             dim3(kWarps * 32), 0, st, p, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_e4m3(const DevPlan& p, bool q_e4m3, const AttArgs& a, cudaStream_t st) {
  if (p.D == 128) return q_e4m3 ? run<128, true>(p, a, st) : run<128, false>(p, a, st);
  return q_e4m3 ? run<64, true>(p, a, st) : run<64, false>(p, a, st);
}

}  // namespace att
}  // namespace sps
