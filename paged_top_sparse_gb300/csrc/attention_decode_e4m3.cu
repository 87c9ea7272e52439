// attention_decode_e4m3.cu -- full attention of tiles of at most 16 rows (single tokens of a head group)
// over an E4M3 cache with a scale for each page and KV head.
//
// The tcgen05 kernel (attention_e4m3.cu) moves about 180 KB through shared memory for a page whose 32 KB
// arrive from HBM in 1400 cycles.  As for an NVFP4 cache (attention_decode.cu) the products of 16 rows
// are small, so the codes go from shared memory to registers once, become FP16 fragments there, and feed
// the warp-level tensor instruction (mma.sync m16n8k16, FP32 accumulation).
//
// Bound: HBM.  64 tokens after 32K, H 32 / H_kv 2, D 128 (1.08 GB): 176 us, of which 161 are the read at the
// rate of a plain copy and most of the rest start, fill and merge (204 in the tcgen05 kernel); H_kv 4 311 us,
// 6.9 TB/s; D 64 99 us; one token after 128K 17 us.  A second copy warp and ring stages of 64 keys
// measured the same.
//
// Mathematics as in attention_e4m3.cu: the scale of a page's keys multiplies its scores' factor, that of its
// values, 2^e, the exponent; the reference m follows both; l takes p' 2^-e.  A BF16 query row becomes
// FP16 after division by a power of two (its largest element then lies in (224, 448]: exact but for
// elements 2^-22 of it and less, which are off by 2^-33 of it at most).
//
// One persistent CTA per SM: a warp copies pages (K and V codes, by TMA with the swizzle that keeps the
// fragment reads below on distinct banks) into a ring; the others take the pages' 32-key chunks in turn,
// each with a running (m, l, O) of its own, merged through shared memory at the end of a piece.
//
// Fragments.  Lane (g, t) = (lane / 4, lane % 4).  For Q K^T a lane reads D / 4 dims of a key, a word of
// four codes to a k-step; for P V the pairs of a B register run along keys, so the bytes of two keys'
// words are interleaved, and O's dims are ordered so that a lane's columns are one run of D / 8 dims.
// Tiles of at most 8 rows turn both products round (K Q^T and V^T P^T), half as many products.
#include <cstring>

#include "attention.cuh"
#include "e4m3.cuh"

namespace sps {
namespace att {
namespace {

constexpr int kChunks = 4;     // 32-key chunks of a page
constexpr int kWarps = 8;      // product warps (D 64: 12 measured 101 us for 64 tokens after 32K, 8 99)

template <int D, int ROWS>
struct DecSmem {
  static constexpr int WARPS = kWarps;
  static constexpr int STEP = WARPS / kChunks;  // a warp takes a chunk of every STEP-th page
  static constexpr int TILE = 128 * D;    // codes of K, or of V
  static constexpr int PAGE = 2 * TILE;
  static constexpr int S0 = (227 * 1024 - WARPS * ROWS * (D * 4 + 8) - D * 32 - 1024) / PAGE;
  // A multiple of STEP: a warp then finds in a stage, each time round, the page after
  // one that it took itself, so that the phase it waits for is never more than one ahead of the
  // barrier's.  Between pieces the warps meet.
  static constexpr int STAGES = (S0 > 9 ? 9 : S0) / STEP * STEP;
  static_assert(WARPS % kChunks == 0 && STAGES >= 4, "stages");
  uint8_t page[STAGES][PAGE];
  float o[WARPS][ROWS][D];
  float2 stat[WARPS][ROWS];  // (m, l)
  uint4 qf[D / 16][32];      // Q fragments, k-step by lane
  float q_mul[16];           // the power of two that a row was divided by
  uint64_t full[STAGES], empty[STAGES], meet;
  int abort_flag;
};

// Byte of 16-byte chunk c of row r of a tile of D-byte rows, as TMA writes it.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
  return D == 128 ? sw128_offset(r, c) : r * 64u + (((c ^ (r >> 1)) & 3u) << 4);
}

template <int D, int ROWS, bool QB>
__global__ void __launch_bounds__(32 * (kWarps + 1), 1)
decode_e4m3_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   DevPlan p, AttArgs a) {
  using Smem = DecSmem<D, ROWS>;
  constexpr int WARPS = Smem::WARPS;
  constexpr bool FLIP = ROWS == 8;  // keys, and then dims, as the products' 16 rows
  constexpr int S = Smem::STAGES, TILE = Smem::TILE;
  constexpr int KW = D / 16;  // 4-code words of a key in a lane
  constexpr int VW = D / 32;  // 4-code words of a value row in a lane
  constexpr int NT = D / 8;   // column tiles of O
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int32_t* status = p.status;
  volatile int* abort_flag = &sm.abort_flag;
  if (smem_u32(smem_raw) & 1023) {  // the swizzled tiles need it; dynamic shared memory has it
    if (tid == 0) set_status(status, DEV_OVERFLOW);
    return;
  }
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
      auto load_ids = [&](int k) {  // physical tiles of pages k + lane
        int id = 0;
        if (k + lane < n) {
          id = __ldg(pages + k + lane);
          if (id < 0 || id >= p.num_phys) {
            set_status(status, DEV_BAD_PAGE);
            id = 0;
          }
        }
        return id * p.Hkv + pc.vg;
      };
      int ids = load_ids(0), next_ids = 0;
      for (int s = 0; s < n && ok; ++s) {
        if (s > 0 && (s & 31) == 0) ids = next_ids;
        if ((s & 31) == 8) next_ids = load_ids(s + 24);
        const int tile = __shfl_sync(0xffffffffu, ids, s & 31);
        const uint32_t it = page_it + s, st = it % S;
        if (lane == 0) {
          ok = mbar_wait(smem_u32(&sm.empty[st]), ((it / S) & 1) ^ 1, abort_flag, status);
          if (ok) {
            const uint32_t f = smem_u32(&sm.full[st]), d = smem_u32(sm.page[st]);
            mbar_expect_tx(f, Smem::PAGE);
            tma_load_2d(d, &tmK, 0, tile * 128, f);
            tma_load_2d(d + TILE, &tmV, 0, tile * 128, f);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      page_it += n;
    }
  } else {
    // ------------------------------------------------ products: chunks of 32 keys
    const int g = lane / 4, t = lane % 4;
    const float* kscale = reinterpret_cast<const float*>(a.ks);
    const float* vscale = reinterpret_cast<const float*>(a.vs);
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
      // the scales of this warp's pages, a chunk ahead (their place, two)
      const int32_t* pages = a.page_table + (int64_t)pc.req * p.max_pages + pc.page0;
      auto tile_of = [&](int ch) {
        const int id = ch < kChunks * n ? __ldg(pages + ch / kChunks) : 0;
        return (int64_t)(id < 0 || id >= p.num_phys ? 0 : id) * p.Hkv + pc.vg;
      };
      int64_t tile1 = tile_of(warp);
      float ks1 = __ldg(kscale + tile1), vs1 = __ldg(vscale + tile1);
      tile1 = tile_of(warp + WARPS);
      // Q fragments, a row per warp, four dims a lane: (row g, row g + 8) x columns 2 t and 2 t + 8 of a
      // k-step are the lane's dims 4 k .. 4 k + 3
      for (int r = warp; r < ROWS; r += WARPS) {
        const int tok = r / rp.HB, hd = r % rp.HB;
        const bool live = tok < pc.q_len && tok < rp.TB && lane < D / 4;
        const int64_t at = (int64_t)(pc.flat0 + tok) * a.q_stride + (int64_t)(pc.vg * p.Hg + hd) * D + 4 * lane;
        uint32_t f0 = 0, f1 = 0;
        if (QB) {
          uint2 x = make_uint2(0, 0);
          if (live) x = __ldg(reinterpret_cast<const uint2*>(a.q + 2 * at));
          const float f[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                              __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u)};
          float amax = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // (a row with an infinity becomes NaN, as in attention_e4m3.cu)
          const float s = row_scale(amax), inv = isinf(amax) ? __uint_as_float(0x7fc00000u) : 1.f / s;
          f0 = pack_p<true>(f[0] * inv, f[1] * inv);
          f1 = pack_p<true>(f[2] * inv, f[3] * inv);
          if (lane == 0) sm.q_mul[r] = s;
        } else {
          uint32_t x = 0;
          if (live) x = __ldg(reinterpret_cast<const uint32_t*>(a.q + at));
          f0 = cvt_e4m3x2((uint16_t)(x & 0xffffu));
          f1 = cvt_e4m3x2((uint16_t)(x >> 16));
        }
        if (lane < D / 4) {
          uint32_t* cell = reinterpret_cast<uint32_t*>(&sm.qf[lane % KW][(r % 8) * 4 + lane / KW]);
          cell[r / 8] = f0;
          cell[2 + r / 8] = f1;
        }
      }
      if (!meet()) break;
      float c[2] = {a.c, a.c};
      if (QB) {
#pragma unroll
        for (int h = 0; h < 2; ++h) c[h] *= sm.q_mul[(FLIP ? 2 * t + h : g + 8 * h) % ROWS];
      }
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
        // (a factor of zero would make NaN of a masked score's infinity)
        const float ck[2] = {fmaxf(c[0] * ks1, 1.18e-38f), fmaxf(c[1] * ks1, 1.18e-38f)};
        const float e2 = scale_log2(vs1);
        ks1 = __ldg(kscale + tile1);
        vs1 = __ldg(vscale + tile1);
        tile1 = tile_of(ch + 2 * WARPS);
        if (!mbar_wait(smem_u32(&sm.full[stg]), (it / S) & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        const int kb = 32 * (ch % kChunks);
        const uint8_t* kp = sm.page[stg];
        const uint8_t* vp = kp + TILE;
        const int key0 = (pc.page0 + ch / kChunks) * 128 + kb;  // the chunk's first key
        // S = Q K^T for keys kb + 8 u + (column), in s[u]; or K Q^T, keys kb + 8 u + (row) of
        // u = 0, 1 in s[0] and u = 2, 3 in s[1]
        float s[FLIP ? 2 : 4][4];
#pragma unroll
        for (int u = 0; u < (FLIP ? 2 : 4); ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
#pragma unroll
        for (int w0 = 0; w0 < KW; w0 += 4) {  // 16 dims of a lane: four k-steps
          uint4 kw[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            kw[u] = *reinterpret_cast<const uint4*>(kp + chunk_at<D>(kb + 8 * u + g, t * (KW / 4) + w0 / 4));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 q = sm.qf[w0 + k][lane];
            const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
            uint32_t x[4][2];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t w = k == 0 ? kw[u].x : k == 1 ? kw[u].y : k == 2 ? kw[u].z : kw[u].w;
              cvt_e4m3x4<false>(w, x[u][0], x[u][1]);
              if (!FLIP) {
                mma_16816(s[u % (FLIP ? 2 : 4)], qa, x[u][0], x[u][1]);
              } else if (u % 2) {  // 16 keys
                const uint32_t ka[4] = {x[u - 1][0], x[u][0], x[u - 1][1], x[u][1]};
                mma_16816(s[u / 2], ka, qa[0], qa[2]);
              }
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
        // the reference: raised for the warp's rows together when some score asks for it
        float mb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mb[h] = fmaf(fmaxf(fmaxf(fmaxf(score(0, h, 0), score(0, h, NZ - 1)),
                                   fmaxf(score(1, h, 0), score(1, h, NZ - 1))),
                             fmaxf(fmaxf(score(2, h, 0), score(2, h, NZ - 1)),
                                   fmaxf(score(3, h, 0), score(3, h, NZ - 1)))),
                       ck[h], e2);
        if (__any_sync(0xffffffffu, first || mb[0] - m[0] > kRescale || mb[1] - m[1] > kRescale)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = row_reduce<ROWS>(mb[h], [](float y, float z) { return fmaxf(y, z); });
            if (x == -INFINITY) x = first ? 0.f : m[h];
            const bool raise = first || x > m[h];
            const float f = raise && !first ? fast_exp2(m[h] - x) : 1.f;
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
        const float off[2] = {e2 + kF16Bias - m[0], e2 + kF16Bias - m[1]};
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (FLIP) {
            const float x = fast_exp2(fmaf(score(u, 0, 0), ck[0], off[0]));
            const float y = fast_exp2(fmaf(score(u, 1, 0), ck[1], off[1]));
            sum[0] += x;
            sum[1] += y;
            pf[u / 2][u % 2] = transpose_8x8(pack_p<true>(x, y));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = fast_exp2(fmaf(score(u, h, 0), ck[h], off[h]));
              const float y = fast_exp2(fmaf(score(u, h, 1), ck[h], off[h]));
              sum[h] += x + y;
              pf[u / 2][2 * (u % 2) + h] = pack_p<true>(x, y);
            }
          }
        }
        const float back = fast_exp2(-e2);
        l[0] = fmaf(sum[0], back, l[0]);
        l[1] = fmaf(sum[1], back, l[1]);
        // O += P V, 16 keys at a time: keys 2 t, 2 t + 1 (first half of the contraction) and
        // 8 + 2 t, + 1; dims (D / 8) g .. of each
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t v[4][VW];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = kb + 16 * y + 2 * t + (k & 1) + 8 * (k >> 1);
            if (D == 128)
              *reinterpret_cast<uint4*>(v[k]) = *reinterpret_cast<const uint4*>(vp + chunk_at<D>(key, g));
            else
              *reinterpret_cast<uint2*>(v[k]) =
                  *reinterpret_cast<const uint2*>(vp + chunk_at<D>(key, g / 2) + (g & 1) * 8);
          }
          if (key0 + 31 >= kv_len) {  // slots behind the request's last token: zero, never NaN
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (key0 + 16 * y + 2 * t + (k & 1) + 8 * (k >> 1) >= kv_len) {
#pragma unroll
                for (int i = 0; i < VW; ++i) v[k][i] = 0;
              }
          }
          if (y == 1) {  // the codes are in registers: the stage may be refilled
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.empty[stg]));
          }
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            uint32_t xa[4], xb[4];  // dims 4 i .. 4 i + 3: keys (2 t, 2 t + 1), and 8 behind them
            cvt_e4m3x4<false>(__byte_perm(v[0][i], v[1][i], 0x5140), xa[0], xa[1]);
            cvt_e4m3x4<false>(__byte_perm(v[0][i], v[1][i], 0x7362), xa[2], xa[3]);
            cvt_e4m3x4<false>(__byte_perm(v[2][i], v[3][i], 0x5140), xb[0], xb[1]);
            cvt_e4m3x4<false>(__byte_perm(v[2][i], v[3][i], 0x7362), xb[2], xb[3]);
            if (!FLIP) {
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_16816(o[(4 * i + j) % (FLIP ? NT / 2 : NT)], pf[y], xa[j], xb[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {  // column tiles 4 i + 2 j and 4 i + 2 j + 1
                const uint32_t va[4] = {xa[2 * j], xa[2 * j + 1], xb[2 * j], xb[2 * j + 1]};
                mma_16816(o[(2 * i + j) % (FLIP ? NT / 2 : NT)], va, pf[y][0], pf[y][1]);
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
        return FLIP ? o[i / 2 % (FLIP ? NT / 2 : NT)][2 * (i % 2) + h]
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
          f[k] = lk != 0.f ? fast_exp2(f[k] - mx) : 0.f;
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
          const float lse = sum != 0.f ? (mx - kF16Bias + log2f(sum)) * 0.6931471805599453f : -INFINITY;
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

template <int D, int ROWS, bool QB>
cudaError_t run_decode(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  alignas(64) CUtensorMap tmK, tmV;
  const uint64_t rows = (uint64_t)p.num_phys * p.Hkv * 128;
  if (!encode_tmap_2d_bytes(&tmK, a.kc, D, rows, D, D, 128) ||
      !encode_tmap_2d_bytes(&tmV, a.vc, D, rows, D, D, 128))
    return cudaErrorInvalidValue;
  const int smem = (int)sizeof(DecSmem<D, ROWS>);
  static_assert(sizeof(DecSmem<D, ROWS>) <= 227 * 1024, "shared memory");
  auto kern = decode_e4m3_kernel<D, ROWS, QB>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.att_ctas), dim3(32 * (kWarps + 1)), smem, st, tmK, tmV, p, a);
}

template <int D, int ROWS>
cudaError_t run_rows(const DevPlan& p, bool q_e4m3, const AttArgs& a, cudaStream_t st) {
  return q_e4m3 ? run_decode<D, ROWS, false>(p, a, st) : run_decode<D, ROWS, true>(p, a, st);
}

}  // namespace

cudaError_t launch_decode_e4m3(const DevPlan& p, bool q_e4m3, const AttArgs& a, cudaStream_t st) {
  if (p.att_slot_rows <= 8)
    return p.D == 128 ? run_rows<128, 8>(p, q_e4m3, a, st) : run_rows<64, 8>(p, q_e4m3, a, st);
  return p.D == 128 ? run_rows<128, 16>(p, q_e4m3, a, st) : run_rows<64, 16>(p, q_e4m3, a, st);
}

}  // namespace att
}  // namespace sps
