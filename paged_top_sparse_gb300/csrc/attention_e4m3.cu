// attention_e4m3.cu -- full causal attention over a paged cache held in 8 bits (E4M3 codes, one FP32
// scale for each page and KV head): out_r = sum_j p_j vs_j v_j / sum_j p_j with
// p_j = 2^(c ks_j q_r . k_j - max), c = scale * q_scale * log2 e, and the log-sum-exp.
//
// Mathematics.  As in attention.cu: one pass over a row's pages with a lazily raised reference m, l and O
// in FP32.  The scale of a page's keys multiplies its scores' factor.  The scale of its values, 2^e, goes
// into the exponent, p' = 2^(c ks s + e - m), where m follows the largest c ks s + e: so P, rounded to FP16
// for the second product, is largest where p times the value's size is, and pages whose values are
// smaller by any factor cost no precision where they matter.  The row's sum takes p' 2^-e.  e is kept
// within 2^-40 .. 2^40 (sps_kv_append's range), so that FP32 holds the sum whatever the order of the pages.
//
// The first product runs on the FP8 tensor core straight from the cache's codes: E4M3 queries as they are;
// a BF16 query row, scaled by a power of two to at most 448, as the sum of two E4M3 rows (8 significant
// bits are 4 + 4: exact for elements down to 2^-10 of the row's largest, off by 2^-17 of that below), two
// products into one accumulator, which cost what one BF16 product does.  So K is copied by TMA into its
// operand tile and never converted.  V is converted to FP16 (exactly) by four warps, since P needs more
// than E4M3's four bits.
//
// Work, rows and merge are attention.cu's (256-row work tiles, the plan's pieces).
//
// Bound, prompts and chunks: the chain of a row tile, its softmax and its own products (256 or 512 cycles of
// Q K^T, 512 of P V) with the hand-offs between, beside the other tile's; then the power limit.  No unit is
// full: at D 128 the tensor pipe is 72 % busy (64 % with E4M3 queries) and the issue slots 44 %, at D 64 the
// issue slots 46 %, exp2 and the tensor pipe 42 %.  H 32 / H_kv 2, an 8192-token prompt: 334 us with BF16
// queries and 281 with E4M3 ones (1.65 and 1.95 PFLOP/s), D 64 279 and 265, where pages are alike; where
// keys and values differ in size from page to page, by up to 3 and 16, 347 and 293 (294 and 279), by 4 and 8
// 371 and 318 (298 and 283): a page above the reference takes the rolled code and rescales O.
// 8 x 512 after 32K 1166 and 1023 us in short runs (1.90 and 2.17 PFLOP/s), 1205 to 1240 and 1026 to 1060 in
// long ones, under the power limit.  Few rows: the cache's bytes, 64 x 3 tokens after 32K 178 us (6.0 TB/s).
//
// What a role executes per page is laid out by two measurements (the prompt, pages of one scale).  The four roles
// of a scheduler share little code, and what they go through together does not fit next to the scheduler: with
// every inner loop unrolled the prompt took 531 us in place of 390, and a second copy of the MMA steps 7 % more.
// And a jump costs about a hundred cycles of fetching: products in loops of one instruction took 480 us where
// straight lines took 313.  So the page that is the rule, in the MMA's loop and in the softmax's, is a straight
// line; every other page (first, masked, last, one that asks for a rescale) goes through rolled code beside it.
// The straight lines took the prompt from 358 to 333 us (BF16 queries) and from 313 to 283.  Half a page at a
// time, so that products and exponentials of one tile overlap, doubles the hand-offs and the reads of Q (509 and
// 406).
//
// One persistent CTA per SM (512-column TMEM: S0 S1 O0 O1, 128 columns each):
//   warp 0     page-table reads and the copies: K tiles by TMA (128-byte or, D = 64, 64-byte swizzle) into
//              one ring, V's codes by bulk copies into another;
//   warp 1     one thread issues every MMA, as in attention.cu: two row tiles' chains alternate, or with one
//              row tile its even and odd pages;
//   warps 4-7, 8-11   softmax and epilogue of row tile 0 / 1, a thread per row;
//   warps 12-15  Q tiles (with the row scales), as soon as the piece before has used them last, and V into
//              FP16 operand tiles, a thread per row.
#include <cstring>

#include "attention.cuh"
#include "e4m3.cuh"

namespace sps {
namespace att {
namespace {

// QB: BF16 queries, two E4M3 planes.  SINGLE: every work tile of the batch has one row tile.
template <int D, bool QB, bool SINGLE>
struct E4Smem {
  static constexpr int TK = 128 * D, TV = 128 * D * 2;  // bytes of a K (or raw V) and of an FP16 V tile
  static constexpr int QT = SINGLE ? 1 : 2;
  static constexpr int QPLANES = QB ? 2 : 1;
  static constexpr int TQ = QPLANES * TK;
  static constexpr int kBudget = 224 * 1024;  // 227 KB less the barriers and statistics
  static constexpr int VS = 2;
  static constexpr int S0 = (kBudget - QT * TQ - VS * TV) / (2 * TK);
  static constexpr int S = S0 > 8 ? 8 : S0;  // stages of the K ring and of the raw V ring
  static_assert(S >= 3, "shared memory");
  uint8_t q[QT][TQ];
  uint8_t k[S][TK];
  uint8_t v[VS][TV];
  uint8_t raw[S][TK];
  uint64_t q_full[2], q_empty[2], k_full[S], k_empty[S], raw_full[S], raw_empty[S], v_full[VS], v_empty[VS];
  uint64_t s_full[2], p_half[2], p_full[2];  // p_half: P of the first 64 keys
  uint64_t o_done[2];                        // the piece's last P V product into O_t
  uint64_t o_free[2], q_seen[2], stat_full, done;  // q_seen: the row scales, by warpgroup
  float2 stat[128];      // (m, l) of the odd pages' rows
  float2 scale[64];      // of a page: K's, and V's as a power of two; a ring over the block's pages
  // BF16 queries: the power of two that a row was divided by (its exponent field), by piece parity
  uint8_t q_exp[2][2][128];
  uint32_t tmem_base;
  uint32_t progress;  // pieces begun, by the MMA warp
  int abort_flag;
};

// Registers of a thread by role: of the copies and the MMA, the softmax, and the tiles' filling.  The block is
// launched with 512 x 128 of them.  D 64, BF16 queries: 283 us, with 88 + 168 + 88 292 (the filling spills); the
// other forms are within 1 % with any split of the kind.
template <bool QB>
struct E4Regs {
  static constexpr int kIssue = 80, kSoftmax = QB ? 168 : 176, kFill = QB ? 96 : 80;
  static_assert(kIssue + 2 * kSoftmax + kFill == 4 * 128, "registers");
};
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The wait for a barrier that has usually been reached, or is within a first try's patience: what follows
// it stays next to what goes before.
__device__ __forceinline__ bool wait_soon(uint64_t& bar, uint32_t parity, volatile int* abort, int32_t* status) {
  if (__builtin_expect(mbar_try_wait(smem_u32(&bar), parity), 1)) return true;
  return mbar_wait(smem_u32(&bar), parity, abort, status);
}

// Byte of 16-byte chunk c of row r of a tile of D-byte rows, as TMA writes it and the tensor core reads it.
template <int D>
__device__ __forceinline__ uint32_t row_offset(uint32_t r, uint32_t c) {
  return D == 128 ? sw128_offset(r, c) : r * 64u + (((c ^ (r >> 1)) & 3u) << 4);
}
// Descriptor of a K-major tile of D-byte rows from its low word.
template <int D>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t lo) {
  constexpr uint64_t sw64 = ((uint64_t)(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
  return D == 128 ? sdesc_hi(lo) : sw64 | lo;
}

// Eight lanes' rows of eight 16-byte chunks each, transposed: lane l gets chunk l of the eight rows.
__device__ __forceinline__ void transpose_chunks(uint32_t (&x)[32], int lane) {
#pragma unroll
  for (int m = 4; m; m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i & m) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t &lo = x[4 * i + e], &hi = x[4 * (i | m) + e];
        const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? lo : hi, m);
        if (up) lo = y;
        else hi = y;
      }
    }
  }
}

template <int D, bool QB, bool SINGLE>
__global__ void __launch_bounds__(512, 1)
attention_e4m3_kernel(const __grid_constant__ CUtensorMap tmK, DevPlan p, AttArgs a) {
  using Smem = E4Smem<D, QB, SINGLE>;
  constexpr int TK = Smem::TK, TV = Smem::TV, TQ = Smem::TQ, S = Smem::S, VS = Smem::VS;
  constexpr uint32_t IDESC_QK = idesc_mma(false, false, 128, 128, false, false);
  constexpr uint32_t IDESC_PV = idesc_mma(false, false, 128, D, false, true);
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
      mbar_init(smem_u32(&sm.q_full[i]), 4);
      mbar_init(smem_u32(&sm.q_empty[i]), 1);
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.p_half[i]), 4);
      mbar_init(smem_u32(&sm.p_full[i]), 4);
      mbar_init(smem_u32(&sm.o_done[i]), 1);
      mbar_init(smem_u32(&sm.o_free[i]), 4);
      mbar_init(smem_u32(&sm.q_seen[i]), 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&sm.k_full[i]), 1);
      mbar_init(smem_u32(&sm.k_empty[i]), 1);
      mbar_init(smem_u32(&sm.raw_full[i]), 1);
      mbar_init(smem_u32(&sm.raw_empty[i]), 4);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(smem_u32(&sm.v_full[i]), 4);
      mbar_init(smem_u32(&sm.v_empty[i]), 1);
    }
    mbar_init(smem_u32(&sm.stat_full), 4);
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
  pdl_wait();  // from here on: what earlier kernels wrote
  const uint32_t tmem = sm.tmem_base;  // S0 S1 at columns 0, 128; O0 O1 at 256, 384
  volatile int* abort_flag = &sm.abort_flag;
  // The second softmax warpgroup skips pieces of one page and one row tile, so one wait of its may last as
  // long as a block's other pieces: its deadline follows the pieces.
  volatile uint32_t* progress = &sm.progress;
  PieceList work(p);
  Piece pc;

  using Regs = E4Regs<QB>;
  if (warp < 4) {
    reg_dec<Regs::kIssue>();
    if (warp == 0) {
      // ------------------------------------------------ copies
      const float* kscale = reinterpret_cast<const float*>(a.ks);
      const float* vscale = reinterpret_cast<const float*>(a.vs);
      uint32_t it = 0;  // tiles copied before this piece
      bool ok = true;
      while (ok && work.next(p, rp, pc)) {
        const int g = pc.vg / rp.blocks;
        // K runs a page ahead of V: K_0, K_1, V_0, K_2, V_1, ...
        const int n = pc.page1 - pc.page0;
        float ks, vs;
        const int32_t* pages = a.page_table + (int64_t)pc.req * p.max_pages + pc.page0;
        auto load_ids = [&](int first) {  // tiles of the lanes' pages first + lane, and their scales
          int id = 0;
          if (first + lane < n) {
            id = __ldg(pages + first + lane);
            if (id < 0 || id >= p.num_phys) {
              set_status(status, DEV_BAD_PAGE);
              id = 0;
            }
          }
          id = id * p.Hkv + g;
          ks = __ldg(kscale + id);
          vs = __ldg(vscale + id);
          return id;
        };
        // A page's scales reach the softmax by way of its K tile's barrier and the MMA thread.  (They are at
        // most 32 + S + 2 pages old when the ring comes round: S of a page waits for P of an earlier one.)
        auto send_scales = [&](int first) {
          sm.scale[(it + first + lane) & 63] = make_float2(ks, scale_log2(vs));
          __syncwarp();
        };
        int ids = load_ids(0), next_ids = 0, k_tile = 0;
        send_scales(0);
        for (int s = 0; s <= n && ok; ++s) {
          const int at = s & 31, v_tile = k_tile;
          if (s > 0 && at == 0) {
            ids = next_ids;
            send_scales(s);
          }
          if (at == 8) next_ids = load_ids(s - 8 + 32);
          k_tile = __shfl_sync(0xffffffffu, ids, at);
          if (lane == 0) {
            if (s < n) {
              const uint32_t sg = (it + s) % S, f = smem_u32(&sm.k_full[sg]);
              ok = mbar_wait(smem_u32(&sm.k_empty[sg]), (((it + s) / S) & 1) ^ 1, abort_flag, status);
              if (ok) {
                mbar_expect_tx(f, TK);
                tma_load_2d(smem_u32(sm.k[sg]), &tmK, 0, k_tile * 128, f);
              }
            }
            if (ok && s > 0) {
              const uint32_t i = it + s - 1, sg = i % S, f = smem_u32(&sm.raw_full[sg]);
              ok = mbar_wait(smem_u32(&sm.raw_empty[sg]), ((i / S) & 1) ^ 1, abort_flag, status);
              if (ok) {
                mbar_expect_tx(f, TK);
                bulk_load(smem_u32(sm.raw[sg]), a.vc + (int64_t)v_tile * TK, TK, f);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        it += n;
      }
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer
      // One thread alone runs the loop: descriptors and barrier addresses pass through registers that the
      // warp's lanes share, so lanes that came apart at a wait must not run beside the one that issues (as
      // a whole warp with an elected lane, D = 64 read wrong scores and lost arrivals).  Descriptors are
      // a constant high word and a low word that grows by the operand's offset.
      if (elect_one()) {
        const uint32_t q_lo = sdesc_lo(smem_u32(sm.q[0]), 16), k_lo = sdesc_lo(smem_u32(sm.k[0]), 16),
                       v_lo = sdesc_lo(smem_u32(sm.v[0]), 16384);
        uint32_t qc = 0, sc = 0, oc = 0;  // a phase bit for each tile
        bool ok = true;
        auto wait = [&](uint64_t& bar, uint32_t parity) {
          if (ok) ok = mbar_wait(smem_u32(&bar), parity, abort_flag, status);
        };
        auto soon = [&](uint64_t& bar, uint32_t parity) { return ok = wait_soon(bar, parity, abort_flag, status); };
        struct Ring {
          uint32_t stage, phase;
          __device__ __forceinline__ Ring take(uint32_t n) {
            const Ring x = *this;
            if (++stage == n) {
              stage = 0;
              phase ^= 1;
            }
            return x;
          }
        };
        Ring kr{0, 0}, vr{0, 0};
        auto commit = [&](uint64_t& bar) {
          mma_commit(smem_u32(&bar));
        };
        // S_t = Q K^T from the operands' descriptors
        auto mma_s = [&](int t, uint32_t tm, uint32_t qa, uint32_t ka) {
#pragma unroll
          for (int pl = 0; pl < Smem::QPLANES; ++pl)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              mma_f8_ss(tm + t * 128, sdesc_rows<D>(qa + ((pl * TK + kk * 32) >> 4)),
                        sdesc_rows<D>(ka + (kk * 32 >> 4)), IDESC_QK, pl + kk > 0);
        };
        // O_t (+)= P_t V for half a page's keys
        auto pv_half = [&](int t, int h, uint32_t tm, uint32_t va, bool add) {
          tc_fence_after();
#pragma unroll
          for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
            mma_f16_ts(tm + 256 + t * 128, tm + t * 128 + kk * 8, sdesc_hi(va + kk * (2048 >> 4)), IDESC_PV,
                       kk > 0 || add);
        };
        auto issue_s = [&](int t, int q, const Ring& k) {
          tc_fence_after();
          uint32_t qa = q_lo + q * (TQ >> 4), ka = k_lo + k.stage * (TK >> 4);
          asm volatile("" : "+r"(qa), "+r"(ka));  // (sums made here, not kept from outside the loops)
          mma_s(t, tmem, qa, ka);
          commit(sm.s_full[t]);
        };
        // P V in two halves, the first as soon as its P is there
        auto issue_pv = [&](int t, const Ring& v, bool first, bool last) {
          uint32_t va = v_lo + v.stage * (TV >> 4);
          asm volatile("" : "+r"(va));
          wait(sm.p_half[t], sc >> t & 1);
          if (first) {
            wait(sm.o_free[t], (oc >> t & 1) ^ 1);
            oc ^= 1u << t;
          }
          if (!ok) return;
          pv_half(t, 0, tmem, va, !first);
          wait(sm.p_full[t], sc >> t & 1);
          sc ^= 1u << t;
          if (!ok) return;
          pv_half(t, 1, tmem, va, true);
          if (last) commit(sm.o_done[t]);
        };
        uint32_t begun = 0;
        while (ok && work.next(p, rp, pc)) {
          *progress = ++begun;
          const int n = pc.page1 - pc.page0;
          // Steps: P V of a page and row tile (or chain), then S of the page that follows it there; two
          // steps of S alone in front.
          const bool split = SINGLE || pc.nt == 1;
          const int steps = split ? n : 2 * n;
          Ring k{0, 0}, v{0, 0};
#pragma unroll 1
          for (int i = -2; i < steps && ok; ++i) {
            // The steps between, in a straight line
            if (i == 2 && (SINGLE || !split)) {
#pragma unroll 1
              for (; ok && i + (SINGLE ? 3 : 2) < steps; i += 2) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  if (SINGLE || t == 0) {
                    v = vr.take(VS);
                    if (!soon(sm.v_full[v.stage], v.phase)) break;
                  }
                  uint32_t va = v_lo + v.stage * (TV >> 4), qa = q_lo + (SINGLE ? 0 : t) * (TQ >> 4), tm = tmem;
                  asm volatile("" : "+r"(va), "+r"(qa), "+r"(tm));  // (sums made here)
                  if (!soon(sm.p_half[t], sc >> t & 1)) break;
                  pv_half(t, 0, tm, va, true);
                  if (!soon(sm.p_full[t], sc >> t & 1)) break;
                  pv_half(t, 1, tm, va, true);
                  if (SINGLE || t == 0) {
                    k = kr.take(S);
                    if (!soon(sm.k_full[k.stage], k.phase)) break;
                  }
                  uint32_t ka = k_lo + k.stage * (TK >> 4);
                  asm volatile("" : "+r"(ka));
                  mma_s(t, tm, qa, ka);
                  commit(sm.s_full[t]);
                  if (SINGLE || t == 1) {
                    commit(sm.v_empty[v.stage]);
                    commit(sm.k_empty[k.stage]);
                  }
                  if (i + 2 + (SINGLE ? t + 1 : 2) == steps) commit(sm.q_empty[SINGLE ? 0 : t]);
                }
                if (!ok) break;
                sc ^= 3;
              }
              if (!ok) break;
            }
            const int t = i & 1, pv = split ? i : i >> 1, sn = split ? i + 2 : pv + 1;
            const bool one = split || t == 0, both = split || t == 1;  // begins, ends with a K or V tile
            if (i >= 0) {
              if (one) {
                v = vr.take(VS);
                wait(sm.v_full[v.stage], v.phase);
              }
              if (ok) issue_pv(t, v, split ? pv < 2 : pv == 0, split ? pv + 2 >= n : pv + 1 == n);
              if (!ok) break;
              if (both) commit(sm.v_empty[v.stage]);
            }
            if (sn < n) {
              const int q = split ? 0 : t;
              if (one) {
                k = kr.take(S);
                wait(sm.k_full[k.stage], k.phase);
              }
              if (i < 0 && (i == -2 || !split)) {
                wait(sm.q_full[q], qc >> q & 1);
                qc ^= 1u << q;
                // (a warpgroup that skips pieces could not follow q_full's phases)
                if (QB && ok) {
                  mbar_arrive(smem_u32(&sm.q_seen[q]));
                  if (split && n > 1) mbar_arrive(smem_u32(&sm.q_seen[1]));
                }
              }
              if (!ok) break;
              issue_s(t, q, k);
              if (both) commit(sm.k_empty[k.stage]);
              if (sn + 1 == n) commit(sm.q_empty[q]);
            }
          }
        }
        commit(sm.done);
        mbar_wait(smem_u32(&sm.done), 0, nullptr, status);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    reg_inc<Regs::kSoftmax>();
    // ------------------------------------------------ softmax and epilogue of row tile w
    const int w = warp >= 8, quarter = warp % 4, row = quarter * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t obase = tmem + lane_addr + 256 + w * 128;
    // The registers of this loop are a page's scores: what else lives through it is kept to little.  A
    // piece is read from the list where it is needed (again for the epilogue), and phases share a word.
    constexpr uint32_t kS = 1, kO = 2, kStat = 4, kQ = 8;  // uses of S_w, pieces in O_w, statistics, pieces
    uint32_t phase = kQ;
    auto is = [&](uint32_t bit) { return phase & bit ? 1u : 0u; };
    const int pieces = p.att_heads[blockIdx.x].count, list = p.att_heads[blockIdx.x].next - 1;
    struct Place {  // of this thread's row in a piece
      int tok, hg;
      bool split, valid;
    };
    auto read_piece = [&](int i, Piece& x) {
      asm volatile("" : "+r"(i));  // (a second reading is one)
      const AttPiece* at = i ? p.att_pieces + list + i : &p.att_heads[blockIdx.x].first;
      const int4 a0 = __ldg(reinterpret_cast<const int4*>(at)), b0 = __ldg(reinterpret_cast<const int4*>(at) + 1);
      x.req = a0.x;
      x.vg = a0.y;
      x.q_len = b0.y;
      x.ctx = b0.z;
      x.flat0 = b0.w;
      x.tok0 = a0.z * 2 * rp.TB;
      x.ntok = min(2 * rp.TB, x.q_len - x.tok0);
      x.pages = ((x.ctx + x.tok0 + x.ntok - 1) >> 7) + 1;
      x.page0 = a0.w;
      x.page1 = b0.x;
      x.nt = x.ntok > rp.TB ? 2 : 1;
      Place r;
      r.split = SINGLE || x.nt == 1;
      r.tok = x.tok0 + (r.split ? 0 : w * rp.TB) + row / rp.HB;
      r.hg = (x.vg % rp.blocks) * 128 + row % rp.HB;  // head within the KV head's group
      r.valid = row / rp.HB < rp.TB && r.tok < x.q_len && r.hg < p.Hg;
      return r;
    };
    bool ok = true;
    uint32_t next_at = 0;  // the block's pages before the next piece
    for (int i = 0; i < pieces && ok; ++i) {
      phase ^= kQ;
      bool split, active;
      int n, step, vis;  // vis: keys of the page that the row sees (128 and more: all)
      uint32_t at = next_at;
      float c = a.c;
      {
        const Place r = read_piece(i, pc);
        // with one row tile, this warpgroup takes the pages of its parity
        split = r.split;
        n = pc.page1 - pc.page0;
        next_at += n;
        step = split ? 2 : 1;
        if (split) n = (n + 1 - w) / 2;
        if (n == 0) continue;
        const int skip = split ? w : 0;
        at += skip;
        active = __any_sync(0xffffffffu, r.valid);
        vis = r.valid ? pc.ctx + r.tok + 1 - (pc.page0 + skip) * 128 : 0x40000000;
        if (QB) {
          if (!mbar_wait_beside(smem_u32(&sm.q_seen[w]), is(kO), abort_flag, status, progress,
                                a.skip_wait_ns))
            break;
          c = r.valid ? c * __uint_as_float((uint32_t)sm.q_exp[is(kQ)][split ? 0 : w][row] << 23) : 0.f;
        }
      }
      float m = 0.f, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int nvis = vis;
        vis -= step * 128;
        const bool masked = __any_sync(0xffffffffu, nvis < 128);
        if (__builtin_expect(!mbar_try_wait(smem_u32(&sm.s_full[w]), is(kS)), 0)) {
          if (!mbar_wait_beside(smem_u32(&sm.s_full[w]), is(kS), abort_flag, status, progress,
                                a.skip_wait_ns)) {
            ok = false;
            break;
          }
        }
        phase ^= kS;  // (a commit covers what its thread issued before: the last product into O_w too)
        const uint32_t bar_half = smem_u32(&sm.p_half[w]), bar_full = smem_u32(&sm.p_full[w]);
        const float2 sc = sm.scale[at & 63];
        at += step;
        // (a factor of zero would make NaN of a masked score's infinity)
        const float ck = fmaxf(c * sc.x, 1.18e-38f), e = sc.y;
        const uint32_t sbase = tmem + lane_addr + w * 128;
        auto exps = [&](const uint32_t (&v)[32], uint32_t* pk, uint64_t (&lsum)[2]) {  // P of 32 keys
          const float off = e + kF16Bias - m;
          const uint64_t c2 = pack_f32x2(ck, ck), off2 = pack_f32x2(off, off);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x, y;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2, off2), x, y);
            x = fast_exp2(x);
            y = fast_exp2(y);
            lsum[(i >> 1) & 1] = add_f32x2(lsum[(i >> 1) & 1], pack_f32x2(x, y));
            pk[i / 2] = pack_p<true>(x, y);
          }
        };
        auto add_l = [&](const uint64_t (&lsum)[2]) {
          float x, y, z, t;
          unpack_f32x2(lsum[0], x, y);
          unpack_f32x2(lsum[1], z, t);
          l = fmaf((x + y) + (z + t), fast_exp2(-e), l);
        };
        tc_fence_after();
        // The usual page, a straight line: the reference holds, so the first half's exponentials run under the
        // second half's load.
        bool usual = j > 0 && !masked && active;
        if (__builtin_expect(usual, 1)) {
          uint32_t v[4][32], pk[32];
          float red[4];
          uint64_t lsum[2] = {0, 0};
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
          exps(v[0], pk, lsum);
          exps(v[1], pk + 16, lsum);
          tmem_ld_wait();
#pragma unroll
          for (int cc = 2; cc < 4; ++cc) {
            reg_fence(v[cc]);
            reg_fence1(red[cc]);
          }
          const float mb = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
          usual = !__any_sync(0xffffffffu, fmaf(mb, ck, e) - m > kRescale);
          if (__builtin_expect(usual, 1)) {
            tmem_st32(sbase, pk);
            uint32_t pk2[32];
            exps(v[2], pk2, lsum);  // under the store
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_half);  // the products of the first 64 keys may begin
            tmem_st16(sbase + 32, *reinterpret_cast<uint32_t(*)[16]>(pk2));
            exps(v[3], pk2 + 16, lsum);
            tmem_st16(sbase + 48, *reinterpret_cast<uint32_t(*)[16]>(pk2 + 16));
            add_l(lsum);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_full);
          }
        }
        if (__builtin_expect(!usual, 0)) {
          // The first page, a masked one, or one whose maximum asks for a rescale: the whole row's maximum
          // first.  The second half is read for it, then the first, which becomes P, and the second again.
          if (active) {
            uint32_t v[2][32], pk[32];
            float mb = -INFINITY;
            uint64_t lsum[2] = {0, 0};
#pragma unroll 1
            for (int s = 0; s < 3; ++s) {
              const int h = s == 1 ? 0 : 1;
              float red[2];
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) red[cc] = tmem_ld32_max(sbase + h * 64 + cc * 32, v[cc]);
              tmem_ld_wait();
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) {
                reg_fence(v[cc]);
                reg_fence1(red[cc]);
              }
              if (masked) {
                const int left = nvis - h * 64;
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    if (cc * 32 + i >= left) v[cc][i] = 0xff800000u;  // -inf
                    mx[i % 4] = fmaxf(mx[i % 4], __uint_as_float(v[cc][i]));
                  }
                red[0] = fmaxf(mx[0], mx[1]);
                red[1] = fmaxf(mx[2], mx[3]);
              }
              if (s < 2) mb = fmaxf(mb, fmaxf(red[0], red[1]));
              if (s == 0) continue;
              if (s == 1) {
                mb = fmaf(mb, ck, e);
                const bool need = j > 0 && mb - m > kRescale;
                if (j == 0) {
                  m = mb == -INFINITY ? 0.f : mb;  // a row that sees nothing here keeps p = 0
                } else if (__any_sync(0xffffffffu, need)) {
                  const float f = need ? fast_exp2(m - mb) : 1.f;
                  if (need) m = mb;
                  l *= f;
#pragma unroll 1
                  for (int d = 0; d < D / 32; ++d) {
                    tmem_ld32(obase + d * 32, pk);
                    tmem_ld_wait();
                    reg_fence(pk);
#pragma unroll
                    for (int i = 0; i < 32; ++i) pk[i] = __float_as_uint(__uint_as_float(pk[i]) * f);
                    tmem_st32(obase + d * 32, pk);
                  }
                  tmem_st_wait();
                }
              }
              exps(v[0], pk, lsum);
              exps(v[1], pk + 16, lsum);
              tmem_st32(sbase + h * 32, pk);  // (over scores that have been read)
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(h ? bar_full : bar_half);
            }
            add_l(lsum);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar_half);
              mbar_arrive(bar_full);
            }
          }
        }
      }
      if (!ok) break;
      if (!mbar_wait(smem_u32(&sm.o_done[w]), is(kO), abort_flag, status)) break;
      phase ^= kO;
      if (split && w == 1) {  // the odd pages' statistics; warpgroup 0 reads O_1 itself
        sm.stat[row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.stat_full));
        continue;
      }
      const Place r = read_piece(i, pc);
      const bool two = split && pc.page1 - pc.page0 > 1;
      float f0 = 1.f, f1 = 0.f;
      if (two) {
        if (!mbar_wait(smem_u32(&sm.stat_full), is(kStat), abort_flag, status)) break;
        phase ^= kStat;
        const float2 o = sm.stat[row];
        if (o.y != 0.f) {  // (0: the row sees nothing in the odd pages; a NaN is no such row)
          const float mm = l != 0.f ? fmaxf(m, o.x) : o.x;
          f0 = l != 0.f ? fast_exp2(m - mm) : 0.f;
          f1 = fast_exp2(o.x - mm);
          l = l * f0 + o.y * f1;
          m = mm;
        }
      }
      if (active) {
        tc_fence_after();
        const float inv = l != 0.f ? 1.f / l : 0.f;
        const float lse = l != 0.f ? (m - kF16Bias + log2f(l)) * 0.6931471805599453f : -INFINITY;
        f0 *= inv;
        f1 *= inv;
        const bool whole = pc.page0 == 0 && pc.page1 == pc.pages;
        const int64_t slot = 2 * blockIdx.x + (pc.page0 > 0 ? 0 : 1);
        const int64_t srow = slot * p.att_slot_rows + w * 128 + row;  // (split: w = 0)
        const int64_t flat = pc.flat0 + r.tok;
        const int head = (pc.vg / rp.blocks) * p.Hg + r.hg;
        if (r.valid) {
          if (!whole) a.part_lse[srow] = lse;
          else if (a.out_lse) a.out_lse[flat * p.H + head] = lse;
        }
        // a thread holds a row; eight lanes exchange the 16-byte chunks of 128 bytes of their rows, so that
        // they then write 128 contiguous bytes of a row together (a thread writing its own row would
        // cost a memory transaction per 16 bytes)
        const uint32_t vrows = __ballot_sync(0xffffffffu, r.valid);
        const int64_t obyte = whole ? (flat * a.out_stride + (int64_t)head * D) * 2 : srow * D * 4;
        uint8_t* const base = whole ? reinterpret_cast<uint8_t*>(a.out)
                                    : reinterpret_cast<uint8_t*>(a.part);
        auto flush = [&](uint32_t (&x)[32], int piece) {  // 128-byte piece `piece` of every row
          transpose_chunks(x, lane);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (lane & 24) + i;
            const int64_t at = __shfl_sync(0xffffffffu, obyte, r);
            if (vrows >> r & 1)
              *reinterpret_cast<uint4*>(base + at + piece * 128 + (lane & 7) * 16) =
                  make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        };
        auto load = [&](int cc, uint32_t (&v)[32]) {  // the row's dims 32 cc .. 32 cc + 31
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
        };
        if (whole) {
#pragma unroll 1
          for (int h = 0; h < D / 64; ++h) {
            uint32_t o[32];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t v[32];
              load(2 * h + u, v);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[16 * u + i] = pack_p<false>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            }
            flush(o, h);
          }
        } else {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t v[32];
            load(cc, v);
            flush(v, cc);
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
    }
  } else {
    reg_dec<Regs::kFill>();
    // ------------------------------------------------ Q tiles, and V into FP16 operand tiles
    const int ct = tid - 384;
    uint32_t it = 0, qc0 = 0, qc1 = 0, parity = 1;
    bool ok = true;
    while (ok && work.next(p, rp, pc)) {
      const int h0 = (pc.vg % rp.blocks) * 128, g = pc.vg / rp.blocks;
      const int n = pc.page1 - pc.page0;
      parity ^= 1;
      for (int t = 0; t < (SINGLE ? 1 : pc.nt) && ok; ++t) {  // Q, a row a thread
        uint32_t& qc = t ? qc1 : qc0;
        const int tok = pc.tok0 + t * rp.TB + ct / rp.HB, hg = h0 + ct % rp.HB;
        const bool valid = ct < rp.TB * rp.HB && tok < pc.q_len && hg < p.Hg;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((pc.flat0 + tok) * a.q_stride + (int64_t)(g * p.Hg + hg) * D) * (QB ? 2 : 1));
        constexpr int CH = QB ? D / 8 : D / 16, XN = QB ? 4 : CH;  // 16-byte chunks, and on the way together
        uint4 x[XN];
        auto fetch = [&](int b) {
#pragma unroll
          for (int k = 0; k < XN; ++k) x[k] = valid ? __ldg(src + b + k) : make_uint4(0, 0, 0, 0);
        };
        float inv = 1.f, mul = 1.f;
        if (QB) {
          uint32_t mx = 0;  // bits of a non-negative float order like the float
#pragma unroll 1
          for (int b = CH - XN; b >= 0; b -= XN) {
            fetch(b);
#pragma unroll
            for (int k = 0; k < XN; ++k) {
              const uint32_t wd[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) mx = max(mx, max((wd[i] & 0x7fffu) << 16, wd[i] & 0x7fff0000u));
            }
          }
          mul = row_scale(__uint_as_float(mx));
          // (an infinity has no E4M3 code: its row becomes NaN, which it would be at the end)
          inv = mx < 0x7f800000u ? 1.f / mul : __uint_as_float(0x7fc00000u);
        } else {
          fetch(0);
        }
        ok = mbar_wait(smem_u32(&sm.q_empty[t]), (qc & 1) ^ 1, abort_flag, status);
        if (!ok) break;
        ++qc;
        if (QB) {
          sm.q_exp[parity][t][ct] = (uint8_t)(__float_as_uint(mul) >> 23);
#pragma unroll 1
          for (int b = 0; b < CH; b += XN) {
            if (b > 0) fetch(b);
#pragma unroll
            for (int k = 0; k < XN; k += 2) {
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4& y = x[k + i / 4];
                const uint32_t wd = i % 4 == 0 ? y.x : i % 4 == 1 ? y.y : i % 4 == 2 ? y.z : y.w;
                const uint64_t f = mul_f32x2(pack_f32x2(__uint_as_float(wd << 16),
                                                        __uint_as_float(wd & 0xffff0000u)),
                                             pack_f32x2(inv, inv));
                const uint32_t h = f32x2_to_e4m3x2(f), h2 = cvt_e4m3x2((uint16_t)h);
                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                const uint32_t d = f32x2_to_e4m3x2(add_f32x2(f, pack_f32x2(-back.x, -back.y)));
                hi[i / 2] = i % 2 ? hi[i / 2] | (h << 16) : h;
                lo[i / 2] = i % 2 ? lo[i / 2] | (d << 16) : d;
              }
              uint8_t* dst = sm.q[t] + row_offset<D>(ct, (b + k) / 2);
              *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(dst + TK) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < XN; ++k) *reinterpret_cast<uint4*>(sm.q[t] + row_offset<D>(ct, k)) = x[k];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[t]));
      }
      for (int j = 0; j < n && ok; ++j, ++it) {
        const uint32_t r = it % S, sg = it % VS;
        constexpr int CPR = D / 16;
        if (!wait_soon(sm.raw_full[r], (it / S) & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        uint4 x[CPR];
        const uint4* codes = reinterpret_cast<const uint4*>(sm.raw[r]) + ct * CPR;
        const int turn = CPR == 8 ? ct : ct >> 1;  // (a column of its own: distinct banks)
#pragma unroll
        for (int k = 0; k < CPR; ++k) x[k] = codes[(k + turn) % CPR];
        // rows behind the request's last token become zero, whatever the slots hold
        if (pc.ctx + pc.q_len <= (pc.page0 + j) * 128 + ct) {
#pragma unroll
          for (int k = 0; k < CPR; ++k) x[k] = make_uint4(0, 0, 0, 0);
        }
        if (!wait_soon(sm.v_empty[sg], ((it / VS) & 1) ^ 1, abort_flag, status)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int k = 0; k < CPR; ++k) e4m3_store16<false>(x[k], sm.v[sg], ct, (k + turn) % CPR);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sm.v_full[sg]));
          mbar_arrive(smem_u32(&sm.raw_empty[r]));
        }
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

template <int D, bool QB, bool SINGLE>
cudaError_t run(const DevPlan& p, const AttArgs& a, cudaStream_t st) {
  alignas(64) CUtensorMap tmK;
  memset(&tmK, 0, sizeof tmK);
  const uint64_t rows = (uint64_t)p.num_phys * p.Hkv * 128;
  if (!encode_tmap_2d_bytes(&tmK, a.kc, D, rows, D, D, 128)) return cudaErrorInvalidValue;
  const int smem = (int)sizeof(E4Smem<D, QB, SINGLE>);
  static_assert(sizeof(E4Smem<D, QB, SINGLE>) <= 227 * 1024, "shared memory");
  auto kern = attention_e4m3_kernel<D, QB, SINGLE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(p.att_ctas), dim3(512), smem, st, tmK, p, a);
  if (e != cudaSuccess) return e;
  return launch_merge(p, a, st);
}

}  // namespace

cudaError_t launch_attention_e4m3(const DevPlan& p, bool q_e4m3, const AttArgs& a, cudaStream_t st) {
  if (p.att_slot_rows <= 16) {
    cudaError_t e = launch_decode_e4m3(p, q_e4m3, a, st);
    return e != cudaSuccess ? e : launch_merge(p, a, st);
  }
  const RowPack rp(p.Hg);
  const bool single = p.att_slot_rows <= rp.TB * rp.HB;
#define SPS_E4(DD, QQ) return single ? run<DD, QQ, true>(p, a, st) : run<DD, QQ, false>(p, a, st)
  if (p.D == 128) {
    if (q_e4m3) SPS_E4(128, false);
    SPS_E4(128, true);
  }
  if (q_e4m3) SPS_E4(64, false);
  SPS_E4(64, true);
#undef SPS_E4
}

}  // namespace att
}  // namespace sps
