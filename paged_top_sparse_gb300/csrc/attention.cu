// attention.cu -- full causal attention of a batch of new tokens (chunks and single tokens mixed)
// over the paged K/V cache: out_r = sum_j softmax_j(scale q_r . k_j) v_j over the keys j <= t of the
// row's request, and the log-sum-exp.
//
// Mathematics.  One pass over a row's pages keeps a reference maximum m, l = sum_j p_j and
// O = sum_j p_j v_j with p_j = 2^((s_j - m) c), c = scale * q_scale * log2 e, all in FP32.  The
// reference follows the running maximum lazily: O and l are rescaled only when the maximum has
// grown by more than 2^8, so p stays at or below 2^8 and the tensor-memory round trip of O is rare.
// P is rounded to the 16-bit type of V for the second product (BF16, or FP16 over an NVFP4 cache,
// whose exact products FP16 holds); l sums the unrounded p.  FP16's narrow range is centred by a
// factor 2^7 on p (largest 2^15, smallest normal 2^-14), which cancels in O / l.
//
// Rows.  The heads of one KV head's group share its keys, so a row tile packs TB tokens x HB heads
// (HB = min(H / H_kv, 128), TB = 128 / HB) into the 128 rows of a tcgen05 accumulator; a work tile
// is two of them (256 rows), fed by the same K and V tiles.
//
// Work.  The plan lists each SM's pieces (runs of pages of a work tile): whole tiles shared out by
// size where there are many, else the (tile, page) pairs in order cut into equal runs, so that
// prompts, chunks and a single token after a long context all fill the GPU.  A tile cut over blocks
// is merged from its pieces' partial results by a second small kernel.  (Merged by the last block
// to arrive instead, every block would pay a fence and an atomic round trip: slower throughout.)
//
// Bound, prompts and chunks: the tensor core and the shared memory that feeds it.  A page of a
// work tile is 2048 cycles of products; Q K^T reads 64 KB of operands per row tile (512 cycles at
// 128 bytes a cycle, as long as its products), so copies into the ring and P's way through the
// softmax show, and a page takes about 1.6 us (3000 cycles).  BF16, D 128, H 32 / H_kv 2: an
// 8192-token prompt 365 us (1.51 PFLOP/s, 0.77 of a large library product at boost clocks, 0.86
// of its sustained rate), 8 x 512 after 32K 1.39 ms (1.61).  Single tokens: the cache's bytes; 64
// after 32K (2.16 GB) 320 us, 6.75 TB/s. An NVFP4 cache adds the conversion of each tile in the
// same SM's issue slots: four chunks of 200 to 700 after 2K to 9K 139 us (0.99 PFLOP/s), 64 x 3
// tokens after 32K 229 us.
//
// One persistent CTA per SM (512-column TMEM: S0 S1 O0 O1, 128 columns each):
//   warp 0     page-table reads and the copies: Q tiles and the K, V tiles of a page into a ring
//              (BF16: TMA with the 128-byte swizzle; NVFP4: codes and scales by bulk copies);
//   warp 1     one thread issues every MMA: S_t = Q_t K^T, and O_t += P_t V with P in TMEM over S_t.
//              With two row tiles their chains alternate, so one tile's products run under the
//              other's softmax; with one row tile its pages alternate between the two chains
//              (S0 O0 the even, S1 O1 the odd ones) and the epilogue merges O0 and O1;
//   warp 2     rows of the last page behind the request's last token are zeroed in the V tile (an
//              unwritten slot may hold NaN, and 0 * NaN would reach every row);
//   warps 4-7, 8-11   softmax and epilogue of row tile 0 / 1, a thread per row;
//   warps 12-15 (NVFP4)  conversion of E4M3 Q and NVFP4 K, V into FP16 operand tiles.
#include <cuda_bf16.h>

#include <atomic>
#include <cstring>

#include "attention.cuh"
#include "nvfp4.cuh"

namespace sps {
using namespace att;
namespace {

// SINGLE: every work tile of the batch has one row tile (decode steps); the second Q tile's room
// goes to the rings.
template <int D, bool QUANT, bool SINGLE>
struct AttSmem {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int RAWB = 128 * D / 2 + 128 * D / 16;  // NVFP4 codes and scales of a tile
  static constexpr int QT = SINGLE ? 1 : 2;
  static constexpr int kBudget = 227 * 1024 - 1536;  // less the barriers and row statistics
  // BF16: as many K/V stages as fit beside the epilogue's staging (32 rows x 128 bytes a warp).
  // NVFP4: four, so that a step's K and V never wait for the products of the step before; the raw
  // ring takes the rest, and the epilogue stages in the Q tile that its products have done with.
  static constexpr int STG = QUANT ? 0 : 8;
  static constexpr int S0 = QUANT ? 4 : (kBudget - QT * TILE - STG * 4096) / TILE;
  static constexpr int STAGES = S0 > 8 ? 8 : S0;
  static constexpr int RS0 = QUANT ? (kBudget - (QT + STAGES) * TILE) / RAWB : 1;
  static constexpr int RS = RS0 > 10 ? 10 : RS0;
  static_assert(STAGES >= 4 && (!QUANT || RS >= 2), "shared memory");
  uint8_t q[QT][TILE];
  uint8_t kv[STAGES][TILE];
  uint8_t stage[QUANT ? 1 : 8][QUANT ? 16 : 4096];
  alignas(16) uint8_t raw[RS][QUANT ? RAWB : 16];
  uint64_t q_full[2], q_empty[2], kv_full[STAGES], kv_empty[STAGES], raw_full[RS], raw_empty[RS];
  uint64_t s_full[2], p_half[2], p_full[2];  // p_half: P of the first 64 keys
  uint64_t o_done[2];                        // the piece's last P V product into O_t
  uint64_t o_free[2], stat_full, tail_go, tail_done, done;
  float2 stat[128];  // (m, l) of the odd pages' rows
  uint32_t tmem_base;
  uint32_t progress;  // pieces begun, by the MMA warp
  int abort_flag;
};

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// Halves of sdesc_sw128: the low word of a shared address (or of an address in 16-byte units added
// to the one of address 0), and the descriptor of a low word (1024 bytes between 8-row groups).
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t sdesc_hi(uint32_t lo) {
  return (sdesc_sw128(0, 0, 1024) & 0xffffffff00000000ull) | lo;
}
// Scratch slot of piece i of a cut tile: a block's first piece goes to slot 2 block when it begins
// inside its tile, its last piece to slot 2 block + 1 when it begins its tile.
__device__ __forceinline__ int64_t piece_slot(const AttMerge& mg, int i) {
  return i == 0 ? 2 * mg.cta0 + 1 : 2 * (mg.cta0 + i);
}

template <int D, bool QUANT, bool SINGLE>
__global__ void __launch_bounds__(QUANT ? 512 : 384, 1)
attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, DevPlan p, AttArgs a) {
  using Smem = AttSmem<D, QUANT, SINGLE>;
  constexpr int TILE = Smem::TILE, S = Smem::STAGES, RS = Smem::RS, DB = D / 64;
  constexpr uint32_t IDESC_QK = idesc_mma(!QUANT, !QUANT, 128, 128, false, false);
  constexpr uint32_t IDESC_PV = idesc_mma(!QUANT, !QUANT, 128, D, false, true);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int32_t* status = p.status;
  const RowPack rp(p.Hg);

  if (smem_u32(smem_raw) & 1023) {  // the swizzled tiles need it; dynamic shared memory has it
    if (tid == 0) set_status(status, DEV_OVERFLOW);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), QUANT ? 4 : 1);
      mbar_init(smem_u32(&sm.q_empty[i]), QUANT ? 4 : 1);  // the epilogue's warps, or the MMA
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.p_half[i]), 4);
      mbar_init(smem_u32(&sm.p_full[i]), 4);
      mbar_init(smem_u32(&sm.o_done[i]), 1);
      mbar_init(smem_u32(&sm.o_free[i]), 4);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&sm.kv_full[i]), QUANT ? 4 : 1);
      mbar_init(smem_u32(&sm.kv_empty[i]), 1);
    }
    for (int i = 0; i < RS; ++i) {
      mbar_init(smem_u32(&sm.raw_full[i]), 1);
      mbar_init(smem_u32(&sm.raw_empty[i]), 4);
    }
    mbar_init(smem_u32(&sm.stat_full), 4);
    mbar_init(smem_u32(&sm.tail_go), 1);
    mbar_init(smem_u32(&sm.tail_done), 1);
    mbar_init(smem_u32(&sm.done), 1);
    sm.progress = 0;
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // from here on: what earlier kernels wrote.  (No early launch of the next kernel: waiting blocks
  // of the merge kernel measured 2 us slower on small batches, 13 us on an 8192-token prompt.)
  pdl_wait();
  const uint32_t tmem = sm.tmem_base;  // S0 S1 at columns 0, 128; O0 O1 at 256, 384
  volatile int* abort_flag = &sm.abort_flag;
  // Two roles skip pieces that are not theirs (the second softmax warpgroup those of one page and
  // one row tile, warp 2 those without a tail), so one wait of theirs may last as long as a block's
  // other pieces: its deadline follows the pieces.
  volatile uint32_t* progress = &sm.progress;
  PieceList work(p);
  Piece pc;

  if (warp < 4) {
    if (QUANT) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ------------------------------------------------ copies
      uint32_t it = 0, qc0 = 0, qc1 = 0;
      bool ok = true;
      while (ok && work.next(p, rp, pc)) {
        const int g = pc.vg / rp.blocks, h0 = g * p.Hg + (pc.vg % rp.blocks) * 128;
        // K runs a page ahead of V: K_0, K_1, V_0, K_2, V_1, ...
        const int n = pc.page1 - pc.page0;
        const int32_t* pages = a.page_table + (int64_t)pc.req * p.max_pages + pc.page0;
        auto load_ids = [&](int first) {  // physical pages of the lanes' pages first + lane
          int id = 0;
          if (first + lane < n) {
            id = __ldg(pages + first + lane);
            if (id < 0 || id >= p.num_phys) {
              set_status(status, DEV_BAD_PAGE);
              id = 0;
            }
          }
          return id * p.Hkv + g;
        };
        int ids = load_ids(0), next_ids = 0, k_tile = 0;
        for (int s = 0; s <= n && ok; ++s) {
          const int at = s & 31, v_tile = k_tile;
          if (s > 0 && at == 0) ids = next_ids;
          if (at == 8) next_ids = load_ids(s - 8 + 32);
          k_tile = __shfl_sync(0xffffffffu, ids, at);
          if (QUANT) {
            // the copies in flight hold too few bytes to cover the memory's latency: pages go to
            // L2 kAhead steps before their copy (at the start all of the first ones at once, but
            // for those whose copies come right behind: fetched twice they cost 64 x 3 tokens
            // after 32K 225 -> 243 us; without any such start 247)
            constexpr int kAhead = 8, kDirect = 2;
            const int f = s == 0 ? lane : s + kAhead;
            const int src = f & 31;
            const int t = s == 0 ? ids
                                 : __shfl_sync(0xffffffffu, f / 32 == s / 32 ? ids : next_ids, src);
            if (f < n && (s == 0 ? lane > kDirect && lane <= kAhead : lane < 4)) {
              if (s == 0 || lane == 0) bulk_prefetch_l2(a.kc + (int64_t)t * (64 * D), 64 * D);
              if (s == 0 || lane == 1) bulk_prefetch_l2(a.vc + (int64_t)t * (64 * D), 64 * D);
              if (s == 0 || lane == 2) bulk_prefetch_l2(a.ks + (int64_t)t * (8 * D), 8 * D);
              if (s == 0 || lane == 3) bulk_prefetch_l2(a.vs + (int64_t)t * (8 * D), 8 * D);
            }
          }
          if (lane == 0) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              if (kv ? s == 0 : s == n) continue;  // no V before, no K behind
              const int tile = kv ? v_tile : k_tile;
              if (QUANT) {
                const uint32_t r = it % RS, f = smem_u32(&sm.raw_full[r]), d = smem_u32(sm.raw[r]);
                ok = mbar_wait(smem_u32(&sm.raw_empty[r]), ((it / RS) & 1) ^ 1, abort_flag, status);
                if (!ok) break;
                mbar_expect_tx(f, Smem::RAWB);
                bulk_load(d, (kv ? a.vc : a.kc) + (int64_t)tile * (64 * D), 64 * D, f);
                bulk_load(d + 64 * D, (kv ? a.vs : a.ks) + (int64_t)tile * (8 * D), 8 * D, f);
                ++it;
                continue;
              }
              const uint32_t sg = it % S, f = smem_u32(&sm.kv_full[sg]);
              ok = mbar_wait(smem_u32(&sm.kv_empty[sg]), ((it / S) & 1) ^ 1, abort_flag, status);
              if (!ok) break;
              mbar_expect_tx(f, TILE);
              for (int db = 0; db < DB; ++db)
                tma_load_2d(smem_u32(sm.kv[sg]) + db * 16384, kv ? &tmV : &tmK, db * 64, tile * 128,
                            f);
              ++it;
              if (s == 0) {  // Q behind the first K tile
                for (int t = 0; t < (SINGLE ? 1 : pc.nt) && ok; ++t) {
                  uint32_t& qc = t ? qc1 : qc0;
                  ok = mbar_wait(smem_u32(&sm.q_empty[t]), (qc & 1) ^ 1, abort_flag, status);
                  if (!ok) break;
                  ++qc;
                  const uint32_t fq = smem_u32(&sm.q_full[t]);
                  mbar_expect_tx(fq, DB * rp.HB * rp.TB * 128);
                  for (int db = 0; db < DB; ++db)
                    tma_load_3d(smem_u32(sm.q[t]) + db * 16384, &tmQ, db * 64, h0,
                                pc.flat0 + pc.tok0 + t * rp.TB, fq);
                }
                if (!ok) break;
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer
      // The warp runs the loop as one and an elected lane issues.  Descriptors are a constant high
      // word and a low word that grows by the operand's offset.
      const bool leader = elect_one();
      const uint32_t q_lo = sdesc_lo(smem_u32(sm.q[0]), 16), kv_lo = smem_u32(sm.kv[0]) >> 4;
      uint32_t st = 0, ph = 0;  // ring stage and phase of the next K or V tile
      uint32_t qc0 = 0, qc1 = 0, sc[2] = {0, 0}, oc[2] = {0, 0}, tc = 0;
      bool ok = true;
      auto wait = [&](uint64_t& bar, uint32_t parity) {
        if (ok) ok = mbar_wait(smem_u32(&bar), parity, abort_flag, status);
      };
      struct Tile {
        uint32_t stage, phase;
      };
      auto take = [&]() {
        const Tile x{st, ph};
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
        return x;
      };
      auto commit = [&](uint64_t& bar) {
        if (leader) mma_commit(smem_u32(&bar));
      };
      // S_t = Q_q K^T
      auto issue_s = [&](int t, int q, const Tile& k) {
        tc_fence_after();
        const uint32_t qa = q_lo + q * (TILE >> 4),
                       ka = sdesc_lo(0, 16) + kv_lo + k.stage * (TILE >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
            mma_f16_ss(tmem + t * 128, sdesc_hi(qa + off), sdesc_hi(ka + off), IDESC_QK, kk > 0);
          }
        }
        commit(sm.s_full[t]);
      };
      // O_t (+)= P_t V in two halves of 64 keys, the first as soon as its P is there
      auto issue_pv = [&](int t, const Tile& v, bool first, bool last, bool tail) {
        const uint32_t va = sdesc_lo(0, 16384) + kv_lo + v.stage * (TILE >> 4);
        auto half = [&](int h) {
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
              mma_f16_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8,
                         sdesc_hi(va + kk * (2048 >> 4)), IDESC_PV, kk > 0 || !first);
          }
        };
        wait(sm.p_half[t], sc[t] & 1);
        if (first) {
          wait(sm.o_free[t], (oc[t] & 1) ^ 1);
          ++oc[t];
        }
        if (tail) {
          wait(sm.tail_done, tc & 1);
          ++tc;
        }
        if (!ok) return;
        half(0);
        wait(sm.p_full[t], sc[t] & 1);
        ++sc[t];
        if (!ok) return;
        half(1);
        if (last) commit(sm.o_done[t]);
      };
      uint32_t begun = 0;
      while (ok && work.next(p, rp, pc)) {
        if (leader) *progress = ++begun;
        const int n = pc.page1 - pc.page0;
        // rows of the last page behind the request's last token
        const bool tail = !QUANT && pc.page1 * 128 > pc.ctx + pc.q_len;
        {
          const Tile k = take();
          wait(sm.kv_full[k.stage], k.phase);
          wait(sm.q_full[0], qc0 & 1);
          ++qc0;
          if (!ok) break;
          issue_s(0, 0, k);
          if (!QUANT && n == 1) commit(sm.q_empty[0]);
          if (!SINGLE && pc.nt == 2) {
            wait(sm.q_full[1], qc1 & 1);
            ++qc1;
            if (!ok) break;
            issue_s(1, 1, k);
            if (!QUANT && n == 1) commit(sm.q_empty[1]);
          }
          commit(sm.kv_empty[k.stage]);
        }
        if (!SINGLE && pc.nt == 2) {
          for (int j = 0; j < n; ++j) {
            const bool more = j + 1 < n;
            Tile k{};
            if (more) k = take();
            const Tile v = take();
            wait(sm.kv_full[v.stage], v.phase);
            // (converted tiles are there long before; a copied K tile may land later than its V)
            if (QUANT && more) wait(sm.kv_full[k.stage], k.phase);
            if (tail && !more && ok && leader) mbar_arrive(smem_u32(&sm.tail_go));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (ok) issue_pv(t, v, j == 0, !more, t == 0 && tail && !more);
              if (ok && more) {
                if (!QUANT && t == 0) wait(sm.kv_full[k.stage], k.phase);
                if (ok) issue_s(t, t, k);
                if (!QUANT && ok && j + 2 == n) commit(sm.q_empty[t]);
              }
            }
            if (!ok) break;
            commit(sm.kv_empty[v.stage]);
            if (more) commit(sm.kv_empty[k.stage]);
          }
        } else {
          auto next_s = [&](int i, int t) {  // S of page i
            const Tile k = take();
            wait(sm.kv_full[k.stage], k.phase);
            if (!ok) return;
            issue_s(t, 0, k);
            commit(sm.kv_empty[k.stage]);
            if (!QUANT && i + 1 == n) commit(sm.q_empty[0]);
          };
          auto page = [&](int j, int t) {
            const Tile v = take();
            wait(sm.kv_full[v.stage], v.phase);
            const bool z = tail && j + 1 == n;
            if (z && ok && leader) mbar_arrive(smem_u32(&sm.tail_go));
            if (ok) issue_pv(t, v, j < 2, j + 2 >= n, z);
            if (!ok) return;
            commit(sm.kv_empty[v.stage]);
            if (j + 2 < n) next_s(j + 2, t);
          };
          if (n > 1) next_s(1, 1);
          for (int j = 0; j < n && ok; j += 2) {
            page(j, 0);
            if (j + 1 < n && ok) page(j + 1, 1);
          }
        }
      }
      commit(sm.done);
      mbar_wait(smem_u32(&sm.done), 0, nullptr, status);
    } else if (warp == 2 && !QUANT) {
      // ------------------------------------------------ zero V rows of the request's unwritten slots
      uint32_t it = 0, tc = 0;
      while (work.next(p, rp, pc)) {
        const int n = pc.page1 - pc.page0, kv_len = pc.ctx + pc.q_len;
        if (pc.page1 * 128 > kv_len) {
          if (!mbar_wait_beside(smem_u32(&sm.tail_go), tc & 1, abort_flag, status, progress,
                                a.skip_wait_ns))
            break;
          ++tc;
          const int r0 = kv_len - (pc.page1 - 1) * 128;  // rows r0 .. 127
          uint8_t* v = sm.kv[(it + 2 * n - 1) % S];
          for (int db = 0; db < DB; ++db)
            for (int i = r0 * 8 + lane; i < 1024; i += 32)
              *reinterpret_cast<uint4*>(v + db * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.tail_done));
        }
        it += 2 * n;
      }
    }
  } else if (warp < 12) {
    if (QUANT) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------ softmax and epilogue of row tile w
    // (registers: with 168 of NVFP4's 512 x 128 a row's scores spill; 176 hold them, 3 to 5 %)
    const int w = warp >= 8, quarter = warp % 4, row = quarter * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t obase = tmem + lane_addr + 256 + w * 128;
    const float c = a.c, bias = QUANT ? kF16Bias : 0.f;
    const int ti = row / rp.HB, hh = row % rp.HB;
    uint32_t su = 0, od = 0, sx = 0;  // uses of S_w, pieces in O_w, statistics received
    bool ok = true;
    while (ok && work.next(p, rp, pc)) {
      // with one row tile, this warpgroup takes the pages of its parity
      const bool split = SINGLE || pc.nt == 1;
      const int np = pc.page1 - pc.page0, n = split ? (np + 1 - w) / 2 : np;
      if (n == 0) continue;
      const int tok = pc.tok0 + (split ? 0 : w * rp.TB) + ti;
      const int hg = (pc.vg % rp.blocks) * 128 + hh;  // head within the KV head's group
      const bool valid = ti < rp.TB && tok < pc.q_len && hg < p.Hg;
      const int pos = pc.ctx + tok;
      const bool active = __any_sync(0xffffffffu, valid);
      float m = 0.f;
      uint64_t lsum[2] = {0, 0};
      for (int j = 0; j < n; ++j) {
        const int page = pc.page0 + (split ? 2 * j + w : j);
        const int nvis = valid ? pos - page * 128 + 1 : 128;
        const bool masked = __any_sync(0xffffffffu, nvis < 128);
        if (!mbar_wait_beside(smem_u32(&sm.s_full[w]), su & 1, abort_flag, status, progress,
                              a.skip_wait_ns)) {
          ok = false;
          break;
        }
        ++su;  // (a commit covers what its thread issued before: the last product into O_w too)
        const uint32_t bar_half = smem_u32(&sm.p_half[w]), bar_full = smem_u32(&sm.p_full[w]);
        bool half_sent = false;
        if (active) {
          tc_fence_after();
          const uint32_t sbase = tmem + lane_addr + w * 128;
          uint32_t v[4][32];
          float red[4];
          const uint64_t c2 = pack_f32x2(c, c);
          auto exps = [&](int cc, uint32_t* pk) {  // P of the keys 32 cc .. 32 cc + 31
            const uint64_t off2 = pack_f32x2(bias - m * c, bias - m * c);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x, y;
              unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[cc][e]), __uint_as_float(v[cc][e + 1])),
                               c2, off2), x, y);
              x = fast_exp2(x);
              y = fast_exp2(y);
              lsum[(e >> 1) & 1] = add_f32x2(lsum[(e >> 1) & 1], pack_f32x2(x, y));
              pk[e / 2] = pack_p<QUANT>(x, y);
            }
          };
          // The usual page (`fast`): the reference maximum holds, so the first half's exponentials
          // run under the second half's load.  The first page, a masked one, or one whose maximum
          // asks for a rescale loads the whole row first.  (One copy of each part: code that a
          // block runs once is fetched at a memory latency.)
          bool fast = j > 0 && !masked;
          uint32_t pk[32];
          for (;;) {
            if (fast) {
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) red[cc] = tmem_ld32_max(sbase + cc * 32, v[cc]);
              tmem_ld_wait();
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) {
                reg_fence(v[cc]);
                reg_fence1(red[cc]);
              }
#pragma unroll
              for (int cc = 2; cc < 4; ++cc) red[cc] = tmem_ld32_max(sbase + cc * 32, v[cc]);
            } else {
              for (bool again = true; again;) {
                again = false;
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) red[cc] = tmem_ld32_max(sbase + cc * 32, v[cc]);
                tmem_ld_wait();
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                  reg_fence(v[cc]);
                  reg_fence1(red[cc]);
                }
                float mb = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
                if (masked) {
                  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                  for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                      if (cc * 32 + i >= nvis) v[cc][i] = 0xff800000u;  // -inf
                      mx[i % 4] = fmaxf(mx[i % 4], __uint_as_float(v[cc][i]));
                    }
                  mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                }
                const bool need = j > 0 && (mb - m) * c > kRescale;
                if (j == 0) {
                  m = mb == -INFINITY ? 0.f : mb;  // a row that sees nothing here keeps p = 0
                } else if (__any_sync(0xffffffffu, need)) {
                  const float f = need ? fast_exp2((m - mb) * c) : 1.f;
                  if (need) m = mb;
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float x, y;
                    unpack_f32x2(lsum[h], x, y);
                    lsum[h] = pack_f32x2(x * f, y * f);
                  }
#pragma unroll 1
                  for (int cc = 0; cc < D / 32; ++cc) {
                    tmem_ld32(obase + cc * 32, v[0]);
                    tmem_ld_wait();
                    reg_fence(v[0]);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                      v[0][i] = __float_as_uint(__uint_as_float(v[0][i]) * f);
                    tmem_st32(obase + cc * 32, v[0]);
                  }
                  tmem_st_wait();
                  again = true;
                }
              }
            }
            const uint64_t keep0 = lsum[0], keep1 = lsum[1];
            exps(0, pk);
            exps(1, pk + 16);
            if (!fast) break;
            tmem_ld_wait();
#pragma unroll
            for (int cc = 2; cc < 4; ++cc) {
              reg_fence(v[cc]);
              reg_fence1(red[cc]);
            }
            const float mb = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
            if (!__any_sync(0xffffffffu, (mb - m) * c > kRescale)) break;
            lsum[0] = keep0;
            lsum[1] = keep1;
            fast = false;
          }
          tmem_st32(sbase, pk);
          uint32_t pk2[32];
          exps(2, pk2);  // under the store
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_half);  // the products of the first 64 keys may begin
          half_sent = true;
          exps(3, pk2 + 16);
          tmem_st32(sbase + 32, pk2);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!half_sent) mbar_arrive(bar_half);
          mbar_arrive(bar_full);
        }
      }
      if (!ok) break;
      if (!mbar_wait(smem_u32(&sm.o_done[w]), od & 1, abort_flag, status)) break;
      ++od;
      float l;
      {
        float x, y, z, t;
        unpack_f32x2(lsum[0], x, y);
        unpack_f32x2(lsum[1], z, t);
        l = (x + y) + (z + t);
      }
      if (split && w == 1) {  // the odd pages' statistics; warpgroup 0 reads O_1 itself
        sm.stat[row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.stat_full));
        continue;
      }
      const bool two = split && np > 1;
      float f0 = 1.f, f1 = 0.f;
      if (two) {
        if (!mbar_wait(smem_u32(&sm.stat_full), sx & 1, abort_flag, status)) break;
        ++sx;
        const float2 o = sm.stat[row];
        if (o.y > 0.f) {  // (0: the row sees nothing in the odd pages)
          const float mm = l > 0.f ? fmaxf(m, o.x) : o.x;
          f0 = l > 0.f ? fast_exp2((m - mm) * c) : 0.f;
          f1 = fast_exp2((o.x - mm) * c);
          l = l * f0 + o.y * f1;
          m = mm;
        }
      }
      if (active) {
        tc_fence_after();
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float lse = l > 0.f ? (m * c - bias + log2f(l)) * 0.6931471805599453f : -INFINITY;
        f0 *= inv;
        f1 *= inv;
        const bool whole = pc.page0 == 0 && pc.page1 == pc.pages;
        const int64_t slot = 2 * blockIdx.x + (pc.page0 > 0 ? 0 : 1);
        const int64_t srow = slot * p.att_slot_rows + w * 128 + row;  // (split: w = 0)
        const int64_t flat = pc.flat0 + tok;
        const int head = (pc.vg / rp.blocks) * p.Hg + hg;
        if (valid) {
          if (!whole) a.part_lse[srow] = lse;
          else if (a.out_lse) a.out_lse[flat * p.H + head] = lse;
        }
        // a thread holds a row; the warp turns 128 bytes of each of its 32 rows at a time in its
        // staging area, so that eight lanes write 128 contiguous bytes of a row (a thread writing
        // its own row would cost a memory transaction per 16 bytes)
        uint8_t* stg = QUANT ? sm.q[SINGLE ? 0 : w] + quarter * (TILE / 4) : sm.stage[warp - 4];
        const uint32_t vrows = __ballot_sync(0xffffffffu, valid);
        const int64_t obyte = whole ? (flat * a.out_stride + (int64_t)head * D) * 2 : srow * D * 4;
        uint8_t* const base = whole ? reinterpret_cast<uint8_t*>(a.out)
                                    : reinterpret_cast<uint8_t*>(a.part);
        auto flush = [&](int piece) {  // 128-byte piece `piece` of every row
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + lane / 8;
            const uint4 x = *reinterpret_cast<const uint4*>(stg + sw128_offset(r, lane % 8));
            const int64_t at = __shfl_sync(0xffffffffu, obyte, r);
            if (vrows >> r & 1)
              *reinterpret_cast<uint4*>(base + at + piece * 128 + (lane % 8) * 16) = x;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t v[32];
          tmem_ld32(obase + cc * 32, v);
          if (two) {
            uint32_t x[32];
            tmem_ld32(obase + 128 + cc * 32, x);
            tmem_ld_wait();
            reg_fence(v);
            reg_fence(x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = __float_as_uint(__uint_as_float(v[i]) * f0 + __uint_as_float(x[i]) * f1);
          } else {
            tmem_ld_wait();
            reg_fence(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f0);
          }
          if (cc == D / 32 - 1) {  // O is read: the next work tile's products may begin
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(smem_u32(&sm.o_free[w]));
              if (two) mbar_arrive(smem_u32(&sm.o_free[1]));
            }
          }
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[k] = pack_p<false>(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
              *reinterpret_cast<uint4*>(stg + sw128_offset(lane, (cc & 1) * 4 + i / 8)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (cc & 1) flush(cc / 2);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(stg + sw128_offset(lane, i / 4)) =
                  make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            flush(cc);
          }
        }
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.o_free[w]));
          if (two) mbar_arrive(smem_u32(&sm.o_free[1]));
        }
      }
      if (QUANT && lane == 0) mbar_arrive(smem_u32(&sm.q_empty[w]));  // staging and Q tile are free
    }
  } else {
    if (QUANT) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    // ------------------------------------------------ operand conversion (NVFP4 plans)
    const int ct = tid - 384;
    uint32_t it = 0, qc0 = 0, qc1 = 0;
    bool ok = QUANT;
    while (ok && work.next(p, rp, pc)) {
      const int h0 = (pc.vg % rp.blocks) * 128;
      const int n = pc.page1 - pc.page0;
      for (int i = 0; i < 2 * n; ++i, ++it) {  // K_0, K_1, V_0, K_2, V_1, ...
        const uint32_t r = it % RS, sg = it % S;
        const bool is_v = i > 0 && (i % 2 == 0 || i == 2 * n - 1);
        const int page = pc.page0 + (i == 2 * n - 1 ? n - 1 : i / 2 - 1);  // (of a V tile)
        if (!mbar_wait(smem_u32(&sm.raw_full[r]), (it / RS) & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        Nvfp4Row<D> x;
        // V rows behind the request's last token become zero, whatever the slots hold
        x.load(sm.raw[r], ct, is_v && pc.ctx + pc.q_len <= page * 128 + ct);
        if (!mbar_wait(smem_u32(&sm.kv_empty[sg]), ((it / S) & 1) ^ 1, abort_flag, status)) {
          ok = false;
          break;
        }
        x.store(sm.kv[sg], ct);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.kv_full[sg]));
          mbar_arrive(smem_u32(&sm.raw_empty[r]));
        }
        // E4M3 Q rows, exactly, into the FP16 operand tiles, behind the first K tile (behind as many
        // tiles as the ring holds measured the same)
        for (int t = 0; i == 0 && t < (SINGLE ? 1 : pc.nt) && ok; ++t) {
          // this thread's 16-byte chunks of the tile, all on the way at once (one after another
          // they took 5400 cycles of a piece's start)
          constexpr int QCH = D / 16;
          uint4 qx[QCH];
#pragma unroll
          for (int k = 0; k < QCH; ++k) {
            const int ch = ct + 128 * k, row = ch / QCH, col = ch % QCH;
            const int tok = pc.tok0 + t * rp.TB + row / rp.HB, hg = h0 + row % rp.HB;
            qx[k] = make_uint4(0, 0, 0, 0);
            if (row < rp.HB * rp.TB && tok < pc.q_len && hg < p.Hg)
              qx[k] = __ldg(reinterpret_cast<const uint4*>(
                  a.q + (pc.flat0 + tok) * a.q_stride +
                  (int64_t)((pc.vg / rp.blocks) * p.Hg + hg) * D + col * 16));
          }
          uint32_t& qc = t ? qc1 : qc0;
          ok = mbar_wait(smem_u32(&sm.q_empty[t]), (qc & 1) ^ 1, abort_flag, status);
          if (!ok) break;
          ++qc;
#pragma unroll
          for (int k = 0; k < QCH; ++k) {
            const int ch = ct + 128 * k, row = ch / QCH, col = ch % QCH;
            const uint32_t wd[4] = {qx[k].x, qx[k].y, qx[k].z, qx[k].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e] = cvt_e4m3x2((uint16_t)(wd[e / 2] >> (16 * (e & 1))));
            uint8_t* d = sm.q[t] + (col / 4) * 16384;
            *reinterpret_cast<uint4*>(d + sw128_offset(row, 2 * (col % 4))) =
                make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(d + sw128_offset(row, 2 * (col % 4) + 1)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[t]));
        }
        if (!ok) break;
      }
    }
  }
  settle_after_abort(abort_flag);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merge of the tiles cut over several blocks: out = sum_i w_i O_i / sum_i w_i with
// w_i = exp(lse_i - max lse); a piece in which the row sees no key (lse = -inf) is never read.
struct MergeRow {
  bool live;
  int64_t flat;
  int head;
};
__device__ __forceinline__ MergeRow merge_row(const DevPlan& p, const RowPack& rp,
                                              const AttMerge& mg, int lr) {
  const int row = lr % 128, ti = row / rp.HB, hg = (mg.vg % rp.blocks) * 128 + row % rp.HB;
  const int tok = mg.tile * 2 * rp.TB + (lr / 128) * rp.TB + ti;
  return {lr < p.att_slot_rows && ti < rp.TB && tok < mg.q_len && hg < p.Hg,
          (int64_t)mg.flat0 + tok, (mg.vg / rp.blocks) * p.Hg + hg};
}
template <int D>
__device__ __forceinline__ void merge_store(const DevPlan& p, const AttArgs& a, const MergeRow& r,
                                            int lane, const float (&acc)[D / 32], float inv) {
  uint16_t* out = a.out + r.flat * a.out_stride + (int64_t)r.head * D + lane * (D / 32);
  if (D == 128)
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack_p<false>(acc[0] * inv, acc[1] * inv),
                   pack_p<false>(acc[D / 32 - 2] * inv, acc[D / 32 - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(out) = pack_p<false>(acc[0] * inv, acc[1] * inv);
}
// Tiles of many rows (few pieces each): a warp takes 8 rows, a lane the weight of one of four
// pieces of one of them, so that a warp has up to 32 rows of partial results on the way.
constexpr int kMergeRows = 8;
template <int D>
__global__ void __launch_bounds__(256)
attention_merge_rows_kernel(DevPlan p, AttArgs a) {
  pdl_wait();
  pdl_trigger();
  const AttMerge mg = p.att_merges[blockIdx.x];
  if (mg.req < 0) return;
  const RowPack rp(p.Hg);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int lr0 = (blockIdx.y * 8 + warp) * kMergeRows;
  const int np = mg.cta1 - mg.cta0 + 1;
  const int k = lane % kMergeRows, ii = lane / kMergeRows;  // this lane's row and piece (mod 4)
  const MergeRow mine = merge_row(p, rp, mg, lr0 + k);
  const uint32_t live = __ballot_sync(0xffffffffu, mine.live);
  if (!live) return;
  auto lse_of = [&](int i) {
    return mine.live && i < np
               ? a.part_lse[piece_slot(mg, i) * p.att_slot_rows + lr0 + k]
               : -INFINITY;
  };
  // rows of a group of pieces that are on the way together
  constexpr int E = D / 32, kGroup = 2;
  float x[kGroup][kMergeRows][E];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        const float* src =
            a.part + (piece_slot(mg, i0 + j) * p.att_slot_rows + lr0 + r) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) x[j][r][e] = 0.f;
        if (i0 + j < np && (live >> r & 1)) {
          if (E == 4) *reinterpret_cast<float4*>(x[j][r]) = *reinterpret_cast<const float4*>(src);
          else *reinterpret_cast<float2*>(x[j][r]) = *reinterpret_cast<const float2*>(src);
        }
      }
  };
  float l[4], mx = -INFINITY;  // the first 16 pieces' statistics, and their rows, at once
#pragma unroll
  for (int c = 0; c < 4; ++c) l[c] = lse_of(4 * c + ii);
  fetch(0);
#pragma unroll
  for (int c = 0; c < 4; ++c) mx = fmaxf(mx, l[c]);
  for (int c = 16; c < np; c += 4) mx = fmaxf(mx, lse_of(c + ii));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
  float sum = 0.f, acc[kMergeRows][E] = {};
  for (int c = 0; c < np; c += 4) {
    const float lc = c == 0 ? l[0] : c == 4 ? l[1] : c == 8 ? l[2] : c == 12 ? l[3] : lse_of(c + ii);
    const float wt = lc == -INFINITY ? 0.f : __expf(lc - mx);
    sum += wt;
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += kGroup) {
#pragma unroll
      for (int j = 0; j < kGroup; ++j)
#pragma unroll
        for (int r = 0; r < kMergeRows; ++r) {
          const float w = __shfl_sync(0xffffffffu, wt, (j0 + j) * kMergeRows + r);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (w != 0.f) acc[r][e] += w * x[j][r][e];
        }
      if (c + j0 + kGroup < np) fetch(c + j0 + kGroup);
    }
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
  if (ii == 0 && mine.live && a.out_lse)
    a.out_lse[mine.flat * p.H + mine.head] = sum > 0.f ? mx + logf(sum) : -INFINITY;
#pragma unroll
  for (int r = 0; r < kMergeRows; ++r) {
    const float s = __shfl_sync(0xffffffffu, sum, r);
    if (live >> r & 1)
      merge_store<D>(p, a, merge_row(p, rp, mg, lr0 + r), lane, acc[r],
                     s > 0.f ? 1.f / s : 0.f);
  }
}

// Tiles of few rows (a single token's may be cut over every SM): a block per row, its warps share
// the pieces; one warp would walk 76 of them at a memory latency each.
template <int D>
__global__ void __launch_bounds__(256)
attention_merge_pieces_kernel(DevPlan p, AttArgs a) {
  constexpr int E = D / 32;  // elements per lane
  __shared__ float wts[kMaxCtas];
  __shared__ float sums[8][32 * E];
  // The entry is the plan's: the products' kernel lets nothing begin before its blocks end, and
  // they began after the upload.  (One token after 8K 10.3 -> 10.1 us, 32 after 1K 36.4 -> 35.6.)
  const AttMerge mg = p.att_merges[blockIdx.x];
  const RowPack rp(p.Hg);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, lr = blockIdx.y;
  const MergeRow row = merge_row(p, rp, mg, lr);
  pdl_wait();
  pdl_trigger();
  if (mg.req < 0) return;
  if (!row.live) return;  // the whole block
  const int np = mg.cta1 - mg.cta0 + 1;
  // this warp's first pieces are on the way while the weights are found
  constexpr int kAhead = 8;
  float x[kAhead][E];
  auto fetch = [&](int i, float (&o)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (i < np) {
      const float* src = a.part + (piece_slot(mg, i) * p.att_slot_rows + lr) * D + lane * E;
      if (E == 4) *reinterpret_cast<float4*>(o) = *reinterpret_cast<const float4*>(src);
      else *reinterpret_cast<float2*>(o) = *reinterpret_cast<const float2*>(src);
    }
  };
  // every warp finds the weights (the same values); the first one keeps them
  float mx = -INFINITY, l[kMaxCtas / 32];
#pragma unroll
  for (int k = 0; k < kMaxCtas / 32; ++k) {
    const int i = lane + 32 * k;
    l[k] = i < np ? a.part_lse[piece_slot(mg, i) * p.att_slot_rows + lr] : -INFINITY;
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) fetch(warp + 8 * k, x[k]);
#pragma unroll
  for (int k = 0; k < kMaxCtas / 32; ++k) mx = fmaxf(mx, l[k]);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kMaxCtas / 32; ++k) {
    const float wt = l[k] == -INFINITY ? 0.f : __expf(l[k] - mx);
    if (warp == 0 && lane + 32 * k < np) wts[lane + 32 * k] = wt;
    sum += wt;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  float acc[E] = {};
  for (int i0 = warp; i0 < np; i0 += 8 * kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + 8 * k;
      const float wt = i < np ? wts[i] : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (wt != 0.f) acc[e] += wt * x[k][e];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(i0 + 8 * (kAhead + k), x[k]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[e];
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int e = 0; e < E; ++e)
    for (int k = 1; k < 8; ++k) acc[e] += sums[k][lane * E + e];
  merge_store<D>(p, a, row, lane, acc, sum > 0.f ? 1.f / sum : 0.f);
  if (lane == 0 && a.out_lse)
    a.out_lse[row.flat * p.H + row.head] = sum > 0.f ? mx + logf(sum) : -INFINITY;
}

template <int D>
cudaError_t run_merge(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  // att_merge_cap bounds the cut tiles of any plan of these q_lens.  An eager call of a plan without
  // a cut tile needs no merge; a captured one keeps it, since it may be replayed over another plan's
  // metadata (same q_lens, other contexts).
  int merges = p.att_merge_cap;
  if (p.att_num_merges == 0 && merges > 0) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(st, &cap);
    if (e != cudaSuccess) return e;
    if (cap == cudaStreamCaptureStatusNone) merges = 0;
  }
  cudaError_t e = cudaSuccess;
  if (merges > 0) {
    if (p.att_slot_rows <= 32)
      e = launch_pdl(attention_merge_pieces_kernel<D>, dim3(merges, p.att_slot_rows), dim3(256), 0,
                     st, p, a);
    else
      e = launch_pdl(attention_merge_rows_kernel<D>,
                     dim3(merges, (p.att_slot_rows + 8 * kMergeRows - 1) / (8 * kMergeRows)),
                     dim3(256), 0, st, p, a);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, bool QUANT, bool SINGLE>
cudaError_t run_attention(const DevPlan& p, const AttArgs& a, const void* q, const void* kc,
                          const void* vc, cudaStream_t st) {
  alignas(64) CUtensorMap tmQ, tmK, tmV;
  memset(&tmQ, 0, sizeof tmQ);
  memset(&tmK, 0, sizeof tmK);
  memset(&tmV, 0, sizeof tmV);
  const RowPack rp(p.Hg);
  if (!QUANT) {
    const uint64_t rows = (uint64_t)p.num_phys * p.Hkv * 128;
    if (!encode_tmap_3d(&tmQ, 0, const_cast<void*>(q), D, p.H, p.T, (uint64_t)D * 2,
                        (uint64_t)a.q_stride * 2, 64, rp.HB, rp.TB, true) ||
        !encode_tmap_2d(&tmK, 0, const_cast<void*>(kc), D, rows, (uint64_t)D * 2, 64, 128, true) ||
        !encode_tmap_2d(&tmV, 0, const_cast<void*>(vc), D, rows, (uint64_t)D * 2, 64, 128, true))
      return cudaErrorInvalidValue;
  }
  if (QUANT && SINGLE && p.att_slot_rows <= 16) {
    cudaError_t e = launch_decode_nvfp4(p, a, st);
    return e != cudaSuccess ? e : run_merge<D>(p, a, st);
  }
  const int smem = (int)sizeof(AttSmem<D, QUANT, SINGLE>);
  static_assert(sizeof(AttSmem<D, QUANT, SINGLE>) <= 227 * 1024, "shared memory");
  auto kern = attention_kernel<D, QUANT, SINGLE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(p.att_ctas), dim3(QUANT ? 512 : 384), smem, st, tmQ, tmK, tmV, p, a);
  if (e != cudaSuccess) return e;
  return run_merge<D>(p, a, st);
}

std::atomic<uint64_t> g_skip_wait_ns{kWaitLimitNs};

}  // namespace

// Limit of the waits that follow the block's pieces, for a test of them (0: the library's).
extern "C" void sps_internal_attention_wait(int64_t limit_ns) {
  g_skip_wait_ns = limit_ns > 0 ? (uint64_t)limit_ns : kWaitLimitNs;
}

cudaError_t launch_attention(const DevPlan& p, bool quant, const void* q, int64_t q_stride,
                             float q_scale, const void* kc, const void* vc, const void* ks,
                             const void* vs, const int32_t* page_table, void* out,
                             int64_t out_stride, float* out_lse, void* scratch, cudaStream_t st) {
  if (p.att_ctas < 1 || p.att_ctas > kMaxCtas) return cudaErrorInvalidConfiguration;
  AttArgs a{};
  a.q = static_cast<const uint8_t*>(q);
  a.kc = static_cast<const uint8_t*>(kc);
  a.vc = static_cast<const uint8_t*>(vc);
  a.ks = static_cast<const uint8_t*>(ks);
  a.vs = static_cast<const uint8_t*>(vs);
  a.q_stride = q_stride;
  a.page_table = page_table;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.out_lse = out_lse;
  a.part = static_cast<float*>(scratch);
  a.part_lse = a.part + 2ll * p.att_ctas * p.att_slot_rows * p.D;
  a.c = attention_factor(p.sm_scale, q_scale);
  a.skip_wait_ns = g_skip_wait_ns.load(std::memory_order_relaxed);
  const RowPack rp(p.Hg);
  const bool single = p.att_slot_rows <= rp.TB * rp.HB;
#define SPS_ATT(DD, QQ) \
  return single ? run_attention<DD, QQ, true>(p, a, q, kc, vc, st) \
                : run_attention<DD, QQ, false>(p, a, q, kc, vc, st)
  if (p.D == 128) {
    if (quant) SPS_ATT(128, true);
    SPS_ATT(128, false);
  }
  if (quant) SPS_ATT(64, true);
  SPS_ATT(64, false);
#undef SPS_ATT
}

}  // namespace sps
