// attention_decode.cu -- full attention of tiles of at most 16 rows (single tokens of a head group)
// over an NVFP4 cache.
//
// The tcgen05 kernel (attention.cu) brings NVFP4 tiles to the tensor core through shared memory: per
// page of 128 keys its FP16 operand tiles cost 64 KB written and 96 KB read, 1560 cycles at 128 bytes
// a cycle, where the page's 18 KB arrive from HBM in about 840.  With 16 rows the products are small
// (1 MFLOP a page), so here the codes go from shared memory to registers once, become FP16 fragments
// there, and feed the warp-level tensor instruction (mma.sync m16n8k16, FP32 accumulation);
// nothing is written back.  64 tokens after 32K (H 32 / H_kv 2, D 128): 278 us there, 159 here;
// one token after 8K 15 and 9.5.
//
// Bound: the SM's issue slots and its warp-level products.  A 32-key chunk costs its warp about
// 64 products, 128 conversions and 128 multiplications by block scales, some 1250 cycles of one
// scheduler, and a page gives each of the four schedulers one chunk: 1400 cycles a page measured,
// 3.8 TB/s (copying the same pages and doing nothing takes 103 us).  Twelve product warps (161
// us), copies issued by the last warp to leave a stage (161) and pages fetched into L2 ahead
// (181) were no faster.
//
// Mathematics as in attention.cu: p = 2^((s - m) c + 7) with a lazily raised reference m, l and O in
// FP32, P rounded to FP16.
//
// One persistent CTA per SM: two warps copy pages (codes and scales of K and V, 18 KB) into a
// ring (one would take as long to issue a page's copies as a page may last); the others take the
// pages' 32-key chunks in turn (32 keys share a load of the Q fragments: 159 us, 16-key chunks
// 184), each with a running (m, l, O) of its own, merged through shared memory at the end of a
// piece.
//
// Fragments.  Lane (g, t) = (lane / 4, lane % 4).  The order of the contracted dims is free, so a
// lane reads whole words of a key (its dims (D / 4) t ..), and the pairs of a B register are the two
// codes of a byte.  For P V the pairs run along keys: the nibbles of two keys' words are interleaved.
// O's dims are ordered so that a lane's B columns are one run of D / 8 dims of a key, under one scale.
#include "attention.cuh"
#include "nvfp4.cuh"

namespace sps {
namespace att {
namespace {

constexpr int kMmaWarps = 8;
constexpr int kChunks = 4;                        // 32-key chunks of a page
constexpr int kPageStep = kMmaWarps / kChunks;    // a warp takes a chunk of every kPageStep-th page
static_assert(kMmaWarps % kChunks == 0, "a warp keeps its place in the page");
constexpr int kCopyWarps = 2;  // a warp copies every kCopyWarps-th page (D 64: one 120 us, two 103)
constexpr int kDecThreads = 32 * (kMmaWarps + kCopyWarps);

template <int D>
struct DecSmem {
  static constexpr int CODES = 64 * D, SCALES = 8 * D;  // of a 128-key tile
  static constexpr int PAGE = 2 * (CODES + SCALES);     // K codes, K scales, V codes, V scales
  static constexpr int S0 = (227 * 1024 - kMmaWarps * 16 * (D * 4 + 8) - D * 32 - 512) / PAGE;
  // A multiple of kPageStep: a warp then finds in a stage, each time round, the page after one that
  // it took itself, so that the phase it waits for is never more than one ahead of the barrier's (a
  // parity wait two phases ahead passes at once).  Between pieces the warps meet.
  static constexpr int STAGES = (S0 > 12 ? 12 : S0) / 4 * 4;
  static_assert(4 % kPageStep == 0 && 4 % kCopyWarps == 0 && STAGES >= 8, "a warp's own stages");
  uint8_t page[STAGES][PAGE];
  float o[kMmaWarps][16][D];
  float2 stat[kMmaWarps][16];  // (m, l)
  uint4 qf[D / 16][32];        // Q fragments, k-step by lane
  uint64_t full[STAGES], empty[STAGES], meet;
  int abort_flag;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, 1) decode_nvfp4_kernel(DevPlan p, AttArgs a) {
  using Smem = DecSmem<D>;
  constexpr int S = Smem::STAGES, WORDS = D / 32;  // WORDS: 8-code words of a key in a lane
  constexpr int NT = D / 8;                        // column tiles of O
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int32_t* status = p.status;
  volatile int* abort_flag = &sm.abort_flag;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), kChunks);
    }
    mbar_init(smem_u32(&sm.meet), kMmaWarps);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();  // from here on: what earlier kernels wrote
  const RowPack rp(p.Hg);
  PieceList work(p);
  Piece pc;

  if (warp >= kMmaWarps) {
    // ------------------------------------------------ copies
    uint32_t page_it = 0;  // pages before the piece
    bool ok = true;
    while (ok && work.next(p, rp, pc)) {
      const int n = pc.page1 - pc.page0;
      const int32_t* pages = a.page_table + (int64_t)pc.req * p.max_pages + pc.page0;
      // this warp's pages of the piece: s0, s0 + kCopyWarps, ...; a lane holds every one's tile
      const int s0 = (int)((warp - kMmaWarps + kCopyWarps - page_it % kCopyWarps) % kCopyWarps);
      auto load_ids = [&](int k) {  // physical tiles of its pages k + lane
        const int s = s0 + (k + lane) * kCopyWarps;
        int id = 0;
        if (s < n) {
          id = __ldg(pages + s);
          if (id < 0 || id >= p.num_phys) {
            set_status(status, DEV_BAD_PAGE);
            id = 0;
          }
        }
        return id * p.Hkv + pc.vg;
      };
      int ids = load_ids(0), next_ids = 0;
      for (int s = s0, k = 0; s < n && ok; s += kCopyWarps, ++k) {
        if (k > 0 && (k & 31) == 0) ids = next_ids;
        if ((k & 31) == 8) next_ids = load_ids(k + 24);
        const int64_t tile = __shfl_sync(0xffffffffu, ids, k & 31);
        const uint32_t it = page_it + s, st = it % S;
        if (lane == 0) {
          ok = mbar_wait(smem_u32(&sm.empty[st]), ((it / S) & 1) ^ 1, abort_flag, status);
          if (ok) {
            const uint32_t f = smem_u32(&sm.full[st]), d = smem_u32(sm.page[st]);
            mbar_expect_tx(f, Smem::PAGE);
            bulk_load(d, a.kc + tile * Smem::CODES, Smem::CODES, f);
            bulk_load(d + Smem::CODES, a.ks + tile * Smem::SCALES, Smem::SCALES, f);
            bulk_load(d + Smem::PAGE / 2, a.vc + tile * Smem::CODES, Smem::CODES, f);
            bulk_load(d + Smem::PAGE / 2 + Smem::CODES, a.vs + tile * Smem::SCALES, Smem::SCALES, f);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      page_it += n;
    }
  } else {
    // ------------------------------------------------ products: chunks of 32 keys
    const int g = lane / 4, t = lane % 4;
    const float c = a.c;
    bool ok = true;
    uint32_t met = 0, page_it = 0;  // meetings, pages before the piece
    auto meet = [&]() {             // the product warps (a bounded wait, unlike a block barrier)
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.meet));
      return mbar_wait(smem_u32(&sm.meet), met++ & 1, abort_flag, status);
    };
    while (ok && work.next(p, rp, pc)) {
      const int n = pc.page1 - pc.page0, kv_len = pc.ctx + pc.q_len;
      int pos[2];  // of rows g and g + 8
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = (g + 8 * h) / rp.HB;
        pos[h] = tok < pc.q_len && tok < rp.TB ? pc.ctx + tok : 0x3fffffff;
      }
      // Q fragments, a k-step per warp: (row g, row g + 8) x columns 2 t and 2 t + 8, which are the
      // lane's dims 4 k .. 4 k + 3
      for (int k = warp; k < D / 16; k += kMmaWarps) {
        uint32_t f[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = g + 8 * h, tok = r / rp.HB, hd = r % rp.HB;
          uint32_t x = 0;
          if (tok < pc.q_len && tok < rp.TB)
            x = __ldg(reinterpret_cast<const uint32_t*>(
                a.q + (int64_t)(pc.flat0 + tok) * a.q_stride +
                (int64_t)(pc.vg * p.Hg + hd) * D + t * (D / 4) + 4 * k));
          f[h] = cvt_e4m3x2((uint16_t)x);
          f[2 + h] = cvt_e4m3x2((uint16_t)(x >> 16));
        }
        sm.qf[k][lane] = make_uint4(f[0], f[1], f[2], f[3]);
      }
      if (!meet()) break;
      const int first_pos = pc.ctx;  // the smallest position of the tile
      float o[NT][4], m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      bool first = true;
      for (int ch = warp; ch < kChunks * n; ch += kMmaWarps) {
        const uint32_t it = page_it + ch / kChunks, stg = it % S;
        if (!mbar_wait(smem_u32(&sm.full[stg]), (it / S) & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        const int kb = 32 * (ch % kChunks);
        const uint8_t* kp = sm.page[stg];
        const uint8_t* vp = kp + Smem::PAGE / 2;
        const int key0 = (pc.page0 + ch / kChunks) * 128 + kb;  // the chunk's first key
        // S = Q K^T for keys kb + 8 u + (column)
        float s[4][4];
        uint32_t kw[4][WORDS], ks[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = kb + 8 * u + g;
          if (D == 128) {
            *reinterpret_cast<uint4*>(kw[u]) = *reinterpret_cast<const uint4*>(kp + key * 64 + t * 16);
            ks[u] = *reinterpret_cast<const uint16_t*>(kp + Smem::CODES + key * 8 + t * 2);
          } else {
            *reinterpret_cast<uint2*>(kw[u]) = *reinterpret_cast<const uint2*>(kp + key * 32 + t * 8);
            ks[u] = kp[Smem::CODES + key * 4 + t];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) ks[u] = cvt_e4m3x2((uint16_t)ks[u]);
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {  // 8 dims of a lane: two k-steps of 4
          const uint4 q0 = sm.qf[2 * w][lane], q1 = sm.qf[2 * w + 1][lane];
          const uint32_t qa[4] = {q0.x, q0.y, q0.z, q0.w}, qb[4] = {q1.x, q1.y, q1.z, q1.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t f = __byte_perm(ks[u], ks[u], w < 2 ? 0x1010 : 0x3232);
            uint32_t x[4];
            cvt_e2m1x8(kw[u][w], x);
            mma_16816(s[u], qa, hmul2_u32(x[0], f), hmul2_u32(x[1], f));
            mma_16816(s[u], qb, hmul2_u32(x[2], f), hmul2_u32(x[3], f));
          }
        }
        if (key0 + 31 > first_pos) {  // some key lies behind some row
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + 8 * u + 2 * t + (e & 1) > pos[e / 2]) s[u][e] = -INFINITY;
        }
        // the reference maximum: raised for the warp's rows together when some score asks for it
        float mb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mb[h] = fmaxf(fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1])),
                        fmaxf(fmaxf(s[2][2 * h], s[2][2 * h + 1]), fmaxf(s[3][2 * h], s[3][2 * h + 1])));
        if (__any_sync(0xffffffffu, first || (mb[0] - m[0]) * c > kRescale ||
                                        (mb[1] - m[1]) * c > kRescale)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = mb[h];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            if (x == -INFINITY) x = first ? 0.f : m[h];
            const bool raise = first || x > m[h];
            const float f = raise && !first ? fast_exp2((m[h] - x) * c) : 1.f;
            if (raise) m[h] = x;
            l[h] *= f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              o[i][2 * h] *= f;
              o[i][2 * h + 1] *= f;
            }
          }
        }
        first = false;
        uint32_t pf[2][4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float off = kF16Bias - m[h] * c;
            const float x = fast_exp2(fmaf(s[u][2 * h], c, off));
            const float y = fast_exp2(fmaf(s[u][2 * h + 1], c, off));
            l[h] += x + y;
            pf[u / 2][2 * (u % 2) + h] = pack_p<true>(x, y);
          }
        // O += P V, 16 keys at a time: keys 2 t, 2 t + 1 (first half of the contraction) and
        // 8 + 2 t, + 1; dims (D / 8) g .. of each
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t v[4][D / 64], vs[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = kb + 16 * y + 2 * t + (k & 1) + 8 * (k >> 1);
            if (D == 128) {
              *reinterpret_cast<uint2*>(v[k]) = *reinterpret_cast<const uint2*>(vp + key * 64 + g * 8);
              vs[k] = vp[Smem::CODES + key * 8 + g];
            } else {
              v[k][0] = *reinterpret_cast<const uint32_t*>(vp + key * 32 + g * 4);
              vs[k] = vp[Smem::CODES + key * 4 + g / 2];
            }
          }
          if (key0 + 31 >= kv_len) {  // slots behind the request's last token: zero, never NaN
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + 16 * y + 2 * t + (k & 1) + 8 * (k >> 1) >= kv_len) {
                vs[k] = 0;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) v[k][i] = 0;
              }
          }
          if (y == 1) {  // the codes are in registers: the stage may be refilled
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.empty[stg]));
          }
          const uint32_t sa = cvt_e4m3x2((uint16_t)(vs[0] | (vs[1] << 8)));
          const uint32_t sb = cvt_e4m3x2((uint16_t)(vs[2] | (vs[3] << 8)));
#pragma unroll
          for (int i = 0; i < D / 64; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // even and odd dims of 8
              constexpr uint32_t LO = 0x0F0F0F0Fu;
              const uint32_t a0 = h ? v[0][i] >> 4 : v[0][i], a1 = h ? v[1][i] : v[1][i] << 4;
              const uint32_t b0 = h ? v[2][i] >> 4 : v[2][i], b1 = h ? v[3][i] : v[3][i] << 4;
              uint32_t xa[4], xb[4];
              cvt_e2m1x8((a0 & LO) | (a1 & ~LO), xa);
              cvt_e2m1x8((b0 & LO) | (b1 & ~LO), xb);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_16816(o[8 * i + 2 * k + h], pf[y], hmul2_u32(xa[k], sa), hmul2_u32(xb[k], sb));
            }
        }
      }
      page_it += n;
      if (!ok) break;
      // the warps' results meet in shared memory.  Column tile i, column q of a tile is dim
      // (D / 8) q + i: lane (g, t) holds dims (D / 4) t + i and (D / 4) t + D / 8 + i
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) sm.stat[warp][g + 8 * h] = make_float2(m[h], l[h]);
        float* row = sm.o[warp][g + 8 * h] + t * (D / 4);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < NT; i += 4)
            *reinterpret_cast<float4*>(row + e * (D / 8) + i) = make_float4(
                o[i][2 * h + e], o[i + 1][2 * h + e], o[i + 2][2 * h + e], o[i + 3][2 * h + e]);
      }
      if (!meet()) break;
      if (tid < 256) {
        const int r = tid / 16, q = tid % 16;  // row, and its dims (D / 16) q ..
        const int tok = r / rp.HB, hd = r % rp.HB;
        float mx = -INFINITY, sum = 0.f, f[kMmaWarps], acc[D / 16];
#pragma unroll
        for (int k = 0; k < kMmaWarps; ++k) {
          const float2 x = sm.stat[k][r];
          f[k] = x.x;
          if (x.y > 0.f) mx = fmaxf(mx, x.x);
        }
#pragma unroll
        for (int k = 0; k < kMmaWarps; ++k) {
          const float lk = sm.stat[k][r].y;
          f[k] = lk > 0.f ? fast_exp2((f[k] - mx) * c) : 0.f;
          sum += lk * f[k];
        }
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[e] = 0.f;
#pragma unroll
        for (int k = 0; k < kMmaWarps; ++k)
          if (f[k] != 0.f) {
#pragma unroll
            for (int e = 0; e < D / 16; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(&sm.o[k][r][q * (D / 16) + e]);
              acc[e] += f[k] * x.x;
              acc[e + 1] += f[k] * x.y;
              acc[e + 2] += f[k] * x.z;
              acc[e + 3] += f[k] * x.w;
            }
          }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        if (tok < pc.q_len && tok < rp.TB) {
          const float lse =
              sum > 0.f ? (mx * c - kF16Bias + log2f(sum)) * 0.6931471805599453f : -INFINITY;
          const int64_t flat = pc.flat0 + tok;
          const int head = pc.vg * p.Hg + hd;
          if (pc.page0 == 0 && pc.page1 == pc.pages) {
            if (q == 0 && a.out_lse) a.out_lse[flat * p.H + head] = lse;
            uint32_t w[D / 32];
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
              w[e] = pack_p<false>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
            uint16_t* out = a.out + flat * a.out_stride + (int64_t)head * D + q * (D / 16);
            if (D == 128) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<uint4*>(w);
            else *reinterpret_cast<uint2*>(out) = *reinterpret_cast<uint2*>(w);
          } else {
            const int64_t srow =
                (2 * (int64_t)blockIdx.x + (pc.page0 > 0 ? 0 : 1)) * p.att_slot_rows + r;
            if (q == 0) a.part_lse[srow] = lse;
#pragma unroll
            for (int e = 0; e < D / 16; e += 4)
              *reinterpret_cast<float4*>(a.part + srow * D + q * (D / 16) + e) = make_float4(
                  acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
          }
        }
      }
      if (!meet()) break;  // the areas may be written again
    }
  }
  settle_after_abort(abort_flag);
}

template <int D>
cudaError_t run_decode(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  const int smem = (int)sizeof(DecSmem<D>);
  static_assert(sizeof(DecSmem<D>) <= 227 * 1024, "shared memory");
  auto kern = decode_nvfp4_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.att_ctas), dim3(kDecThreads), smem, st, p, a);
}

}  // namespace

cudaError_t launch_decode_nvfp4(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  return p.D == 128 ? run_decode<128>(p, a, st) : run_decode<64>(p, a, st);
}

}  // namespace att
}  // namespace sps
