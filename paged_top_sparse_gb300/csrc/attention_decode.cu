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
// Bound: the warps' own chains of conversion and product.  A 32-key chunk costs its warp about 64
// products, 128 conversions and 128 multiplications by block scales, a page gives each of the four
// schedulers one chunk, and two or three warps a scheduler hide only part of each other's waits: 64
// tokens after 32K read 4.0 TB/s with issue slots 45 %, the tensor pipe 40 % and DRAM 51 % busy
// (copying the same pages and doing nothing takes 103 us).  Copies issued by the last warp to leave a
// stage (161 us) and pages fetched into L2 ahead (181) were no faster.
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
// Tiles of at most 8 rows (groups of up to 8 heads) turn both products round, K Q^T and V^T P^T: the
// keys, then the dims, are the instruction's 16 rows and the query rows its 8 columns, so half as
// many products do, P crossing the warp as transposed 8 x 8 tiles.  The converted registers are the
// same.  64 tokens after 32K, H 32: H_kv 8 564 -> 452 us, H_kv 4 290 -> 233 (with 8 warps).
#include "attention.cuh"
#include "nvfp4.cuh"

namespace sps {
namespace att {
namespace {

constexpr int kChunks = 4;     // 32-key chunks of a page
constexpr int kCopyWarps = 2;  // a warp copies every kCopyWarps-th page (D 64: one 120 us, two 103)
// Product warps: 12 where 128 registers (four warps a scheduler) hold the accumulators, else 8.
// 64 tokens after 32K: 8 rows, D 128, H_kv 8 457 us with 8 and 412 with 12; D 64 306 and 266; 16
// rows, D 64 103 and 90, D 128 158 and 161.  (A context of a few pages loses 0.5 us of 9 by them.)
template <int D, int ROWS>
constexpr int kWarps = D * ROWS <= 1024 ? 12 : 8;

template <int D, int ROWS>
struct DecSmem {
  static constexpr int WARPS = kWarps<D, ROWS>;
  static constexpr int STEP = WARPS / kChunks;  // a warp takes a chunk of every STEP-th page
  static_assert(WARPS % kChunks == 0, "a warp keeps its place in the page");
  static constexpr int UNIT = STEP % kCopyWarps ? STEP * kCopyWarps : STEP;
  static constexpr int CODES = 64 * D, SCALES = 8 * D;  // of a 128-key tile
  static constexpr int PAGE = 2 * (CODES + SCALES);     // K codes, K scales, V codes, V scales
  static constexpr int S0 = (227 * 1024 - WARPS * ROWS * (D * 4 + 8) - D * 32 - 512) / PAGE;
  // A multiple of STEP and kCopyWarps: a warp then finds in a stage, each time round, the page after
  // one that it took itself, so that the phase it waits for is never more than one ahead of the
  // barrier's (a parity wait two phases ahead passes at once).  Between pieces the warps meet.
  static constexpr int STAGES = (S0 > 12 ? 12 : S0) / UNIT * UNIT;
  static_assert(UNIT % STEP == 0 && UNIT % kCopyWarps == 0 && STAGES >= 6, "stages");
  uint8_t page[STAGES][PAGE];
  float o[WARPS][ROWS][D];
  float2 stat[WARPS][ROWS];  // (m, l)
  uint4 qf[D / 16][32];        // Q fragments, k-step by lane
  uint64_t full[STAGES], empty[STAGES], meet;
  int abort_flag;
};

template <int D, int ROWS>
__global__ void __launch_bounds__(32 * (kWarps<D, ROWS> + kCopyWarps), 1)
decode_nvfp4_kernel(DevPlan p, AttArgs a) {
  using Smem = DecSmem<D, ROWS>;
  constexpr int WARPS = Smem::WARPS;
  constexpr bool FLIP = ROWS == 8;  // keys, and then dims, as the products' 16 rows
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
    mbar_init(smem_u32(&sm.meet), WARPS);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();  // from here on: what earlier kernels wrote
  const RowPack rp(p.Hg);
  PieceList work(p);
  Piece pc;

  if (warp >= WARPS) {
    // ------------------------------------------------ copies
    uint32_t page_it = 0;  // pages before the piece
    bool ok = true;
    while (ok && work.next(p, rp, pc)) {
      const int n = pc.page1 - pc.page0;
      const int32_t* pages = a.page_table + (int64_t)pc.req * p.max_pages + pc.page0;
      // this warp's pages of the piece: s0, s0 + kCopyWarps, ...; a lane holds every one's tile
      const int s0 = (int)((warp - WARPS + kCopyWarps - page_it % kCopyWarps) % kCopyWarps);
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
      int pos[2];  // of this lane's two rows of the scores
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = (FLIP ? 2 * t + h : g + 8 * h) / rp.HB;
        pos[h] = tok < pc.q_len && tok < rp.TB ? pc.ctx + tok : 0x3fffffff;
      }
      // Q fragments, a k-step per warp: (row g, row g + 8) x columns 2 t and 2 t + 8, which are the
      // lane's dims 4 k .. 4 k + 3
      for (int k = warp; k < D / 16; k += WARPS) {
        uint32_t f[4] = {};
#pragma unroll
        for (int h = 0; h < (FLIP ? 1 : 2); ++h) {
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
      // o: column tile i of 8 dims x rows (g, g + 8), or two of them as the rows of one product
      float o[FLIP ? NT / 2 : NT][4], m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < (FLIP ? NT / 2 : NT); ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      bool first = true;
      for (int ch = warp; ch < kChunks * n; ch += WARPS) {
        const uint32_t it = page_it + ch / kChunks, stg = it % S;
        if (!mbar_wait(smem_u32(&sm.full[stg]), (it / S) & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        const int kb = 32 * (ch % kChunks);
        const uint8_t* kp = sm.page[stg];
        const uint8_t* vp = kp + Smem::PAGE / 2;
        const int key0 = (pc.page0 + ch / kChunks) * 128 + kb;  // the chunk's first key
        // S = Q K^T for keys kb + 8 u + (column), in s[u]; or K Q^T, keys kb + 8 u + (row) of
        // u = 0, 1 in s[0] and u = 2, 3 in s[1]
        float s[FLIP ? 2 : 4][4];
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
          if (!FLIP || u < 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u % (FLIP ? 2 : 4)][e] = 0.f;
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) ks[u] = cvt_e4m3x2((uint16_t)ks[u]);
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {  // 8 dims of a lane: two k-steps of 4
          const uint4 q0 = sm.qf[2 * w][lane], q1 = sm.qf[2 * w + 1][lane];
          const uint32_t qa[4] = {q0.x, q0.y, q0.z, q0.w}, qb[4] = {q1.x, q1.y, q1.z, q1.w};
          uint32_t x[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t f = __byte_perm(ks[u], ks[u], w < 2 ? 0x1010 : 0x3232);
            cvt_e2m1x8(kw[u][w], x[u]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[u][k] = hmul2_u32(x[u][k], f);
            if (!FLIP) {
              mma_16816(s[u % (FLIP ? 2 : 4)], qa, x[u][0], x[u][1]);
              mma_16816(s[u % (FLIP ? 2 : 4)], qb, x[u][2], x[u][3]);
            } else if (u % 2) {  // 16 keys
              const uint32_t ka[4] = {x[u - 1][0], x[u][0], x[u - 1][1], x[u][1]};
              const uint32_t kb2[4] = {x[u - 1][2], x[u][2], x[u - 1][3], x[u][3]};
              mma_16816(s[u / 2], ka, qa[0], qa[2]);
              mma_16816(s[u / 2], kb2, qb[0], qb[2]);
            }
          }
        }
        // the score of key 8 u + .. in row h of this lane: two of them (z) of a key pair, or one
        auto score = [&](int u, int h, int z) -> float& {
          return FLIP ? s[u / 2 % 2][2 * (u % 2) + h] : s[u % (FLIP ? 2 : 4)][2 * h + z];
        };
        constexpr int NZ = FLIP ? 1 : 2;
        if (key0 + 31 > first_pos) {  // some key lies behind some row
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int z = 0; z < NZ; ++z)
                if (key0 + 8 * u + (FLIP ? g : 2 * t + z) > pos[h]) score(u, h, z) = -INFINITY;
        }
        // the reference maximum: raised for the warp's rows together when some score asks for it
        float mb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mb[h] = fmaxf(fmaxf(fmaxf(score(0, h, 0), score(0, h, NZ - 1)),
                              fmaxf(score(1, h, 0), score(1, h, NZ - 1))),
                        fmaxf(fmaxf(score(2, h, 0), score(2, h, NZ - 1)),
                              fmaxf(score(3, h, 0), score(3, h, NZ - 1))));
        if (__any_sync(0xffffffffu, first || (mb[0] - m[0]) * c > kRescale ||
                                        (mb[1] - m[1]) * c > kRescale)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = row_reduce<ROWS>(mb[h], [](float y, float z) { return fmaxf(y, z); });
            if (x == -INFINITY) x = first ? 0.f : m[h];
            const bool raise = first || x > m[h];
            const float f = raise && !first ? fast_exp2((m[h] - x) * c) : 1.f;
            if (raise) m[h] = x;
            l[h] *= f;
#pragma unroll
            for (int i = 0; i < (FLIP ? NT / 2 : NT); ++i) {
              o[i][FLIP ? h : 2 * h] *= f;
              o[i][FLIP ? 2 + h : 2 * h + 1] *= f;
            }
          }
        }
        first = false;
        // P: rows (g, g + 8) x key pairs, or (FLIP) key pairs x row g, from key g x rows (2 t, 2 t + 1)
        uint32_t pf[2][4];
        const float off[2] = {kF16Bias - m[0] * c, kF16Bias - m[1] * c};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (FLIP) {
            const float x = fast_exp2(fmaf(score(u, 0, 0), c, off[0]));
            const float y = fast_exp2(fmaf(score(u, 1, 0), c, off[1]));
            l[0] += x;
            l[1] += y;
            pf[u / 2][u % 2] = transpose_8x8(pack_p<true>(x, y));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = fast_exp2(fmaf(score(u, h, 0), c, off[h]));
              const float y = fast_exp2(fmaf(score(u, h, 1), c, off[h]));
              l[h] += x + y;
              pf[u / 2][2 * (u % 2) + h] = pack_p<true>(x, y);
            }
          }
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
              for (int k = 0; k < 4; ++k) {
                xa[k] = hmul2_u32(xa[k], sa);
                xb[k] = hmul2_u32(xb[k], sb);
                if (!FLIP) {
                  mma_16816(o[(8 * i + 2 * k + h) % (FLIP ? NT / 2 : NT)], pf[y], xa[k], xb[k]);
                } else if (k % 2) {  // column tiles 8 i + 2 (k - 1) + h and 8 i + 2 k + h
                  const uint32_t va[4] = {xa[k - 1], xa[k], xb[k - 1], xb[k]};
                  mma_16816(o[4 * i + 2 * h + k / 2], va, pf[y][0], pf[y][1]);
                }
              }
            }
        }
      }
      page_it += n;
      if (!ok) break;
      // the warps' results meet in shared memory.  Column tile i, column q of a tile is dim
      // (D / 8) q + i: lane (g, t) holds dims (D / 4) t + i and (D / 4) t + D / 8 + i of its rows, or
      // (FLIP) dims (D / 8) g + i
      auto dim_of = [&](int i, int h, int e) {
        const int k = i / 2 % 4;
        return FLIP ? o[(4 * (i / 8) + 2 * (i % 2) + k / 2) % (NT / 2)][2 * (k % 2) + h]
                    : o[i % (FLIP ? NT / 2 : NT)][2 * h + e];
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = FLIP ? 2 * t + h : g + 8 * h;
        l[h] = row_reduce<ROWS>(l[h], [](float y, float z) { return y + z; });
        if ((FLIP ? g : t) == 0) sm.stat[warp][r] = make_float2(m[h], l[h]);
        float* row = sm.o[warp][r] + (FLIP ? g * (D / 8) : t * (D / 4));
#pragma unroll
        for (int e = 0; e < (FLIP ? 1 : 2); ++e)
#pragma unroll
          for (int i = 0; i < NT; i += 4)
            *reinterpret_cast<float4*>(row + e * (D / 8) + i) =
                make_float4(dim_of(i, h, e), dim_of(i + 1, h, e), dim_of(i + 2, h, e),
                            dim_of(i + 3, h, e));
      }
      if (!meet()) break;
      if (tid < 16 * ROWS) {
        const int r = tid / 16, q = tid % 16;  // row, and its dims (D / 16) q ..
        const int tok = r / rp.HB, hd = r % rp.HB;
        float mx = -INFINITY, sum = 0.f, f[WARPS], acc[D / 16];
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
          const float2 x = sm.stat[k][r];
          f[k] = x.x;
          if (x.y != 0.f) mx = fmaxf(mx, x.x);  // (0: nothing seen; a NaN is no such row)
        }
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
          const float lk = sm.stat[k][r].y;
          f[k] = lk != 0.f ? fast_exp2((f[k] - mx) * c) : 0.f;
          sum += lk * f[k];
        }
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[e] = 0.f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k)
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
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        if (tok < pc.q_len && tok < rp.TB) {
          const float lse =
              sum != 0.f ? (mx * c - kF16Bias + log2f(sum)) * 0.6931471805599453f : -INFINITY;
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

template <int D, int ROWS>
cudaError_t run_decode(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  const int smem = (int)sizeof(DecSmem<D, ROWS>);
  static_assert(sizeof(DecSmem<D, ROWS>) <= 227 * 1024, "shared memory");
  auto kern = decode_nvfp4_kernel<D, ROWS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.att_ctas), dim3(32 * (kWarps<D, ROWS> + kCopyWarps)), smem, st, p,
                    a);
}

}  // namespace

cudaError_t launch_decode_nvfp4(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  if (p.att_slot_rows <= 8)
    return p.D == 128 ? run_decode<128, 8>(p, a, st) : run_decode<64, 8>(p, a, st);
  return p.D == 128 ? run_decode<128, 16>(p, a, st) : run_decode<64, 16>(p, a, st);
}

}  // namespace att
}  // namespace sps
