// host.cpp -- C ABI of libsps: problem validation, the plan (per-token metadata, indexer work
// list, workspace layout), the metadata upload (through a page-locked staging ring), and the
// argument checks in front of every kernel launch.  No device memory is ever allocated here.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>
#include <numeric>
#include <string>
#include <vector>

#include "sps_internal.h"

using namespace sps;

namespace {

thread_local std::string g_err;

sps_status fail(sps_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

sps_status cuda_fail(cudaError_t e, const char* what) {
  return fail(SPS_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Page-locked staging for the plan-metadata uploads.  The bytes are written into a mapped
// page-locked ring and a copy kernel on the caller's stream reads them from there: a copy from
// pageable memory makes the GPU wait while the driver stages it, and a DMA on the copy engine
// queues behind the caller's own transfers on other streams (for instance the next batch's
// inputs).  One ring per process, allocated on first use (by the calls that may allocate) and
// never freed; a region is reused only after the event recorded behind its copy has completed.
// Uploads that do not fit, uploads into a stream being captured into a graph (the graph must
// keep reading the plan's own copy), a failed page-locked allocation or mapping, or a call
// that may not allocate while the ring does not exist yet copy from pageable memory instead.
class StagingRing {
 public:
  cudaError_t upload(void* dst, const void* src, size_t n, cudaStream_t s, bool may_alloc) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
      (void)cudaGetLastError();
      return cudaMemcpyAsync(dst, src, n, cudaMemcpyHostToDevice, s);
    }
    std::lock_guard<std::mutex> lock(mu_);
    if (!buf_ && !failed_ && may_alloc) {
      if (cudaHostAlloc(reinterpret_cast<void**>(&buf_), kBytes,
                        cudaHostAllocPortable | cudaHostAllocMapped) != cudaSuccess) {
        buf_ = nullptr;
        failed_ = true;
        (void)cudaGetLastError();
      } else if (cudaHostGetDevicePointer(reinterpret_cast<void**>(&dbuf_), buf_, 0) !=
                 cudaSuccess) {
        dbuf_ = nullptr;  // not mapped: DMA from the ring instead
        (void)cudaGetLastError();
      }
    }
    if (!buf_ || n > kBytes / 2) return cudaMemcpyAsync(dst, src, n, cudaMemcpyHostToDevice, s);
    size_t off = head_;
    if (off + n > kBytes) off = 0;
    // wait for the copies still reading [off, off + n)
    while (!live_.empty() && overlaps(live_.front(), off, off + n)) {
      cudaError_t e = cudaEventSynchronize(live_.front().ev);
      free_ev_.push_back(live_.front().ev);
      live_.erase(live_.begin());
      if (e != cudaSuccess) return e;
    }
    memcpy(buf_ + off, src, n);
    cudaError_t e = (dbuf_ && aligned(dst, 16))
                        ? launch_staged_copy(dbuf_ + off, dst, n, s)
                        : cudaMemcpyAsync(dst, buf_ + off, n, cudaMemcpyHostToDevice, s);
    if (e != cudaSuccess) return e;
    cudaEvent_t ev;
    if (!free_ev_.empty()) {
      ev = free_ev_.back();
      free_ev_.pop_back();
    } else if ((e = cudaEventCreateWithFlags(&ev, cudaEventDisableTiming)) != cudaSuccess) {
      return cudaStreamSynchronize(s);  // no event: the region is safe once the copy is done
    }
    if ((e = cudaEventRecord(ev, s)) != cudaSuccess) {
      cudaEventDestroy(ev);
      return cudaStreamSynchronize(s);
    }
    live_.push_back({off, off + n, ev});
    head_ = (size_t)align_up((int64_t)(off + n), 256);
    return cudaSuccess;
  }

 private:
  struct Live {
    size_t begin, end;
    cudaEvent_t ev;
  };
  static bool overlaps(const Live& l, size_t b, size_t e) { return l.begin < e && b < l.end; }
  static constexpr size_t kBytes = 16u << 20;
  std::mutex mu_;
  uint8_t* buf_ = nullptr;   // host address of the ring
  uint8_t* dbuf_ = nullptr;  // its device address (NULL: not mapped)
  bool failed_ = false;
  size_t head_ = 0;
  std::vector<Live> live_;  // in ring order
  std::vector<cudaEvent_t> free_ev_;
};
StagingRing g_staging;

}  // namespace

struct sps_plan {
  sps_problem pb;                 // copy (host arrays below)
  std::vector<int32_t> q_lens, ctx_lens;
  std::vector<ReqInfo> reqs;
  std::vector<int32_t> page_req;  // [total_pages]
  std::vector<IdxTask> idx_tasks;
  int64_t T = 0, R = 0, num_buckets = 0, max_entries = 0, max_fwd_tasks = 0;
  int64_t total_pages = 0, num_chunks = 0, inv_blocks = 0;
  // workspace layout (bytes)
  int64_t off_status = 0, off_counters = 0, off_tok_pos = 0, off_tok_req = 0, off_reqs = 0,
          off_page_req = 0, off_idx_tasks = 0, off_chunk_offsets = 0, off_bucket_totals = 0,
          off_range_sums = 0,
          off_qconv = -1, off_kconv = -1,
          off_bucket_offsets = 0, off_entries = 0, off_fwd_tasks = 0, off_topk_lists = -1,
          off_topk_meta = -1, off_topk_gmax = -1,
          ws_bytes = 0;
  // the part the forward uses: [fwd_base, fwd_base + fwd_ws_bytes), the no-allocation forward's need
  int64_t fwd_base = 0, fwd_ws_bytes = 0;
  int32_t topk_nseg = 1, topk_segg = 0;
  int32_t fwd_prefetch = 0;
  // full attention (attention.cu): the blocks' work, the tiles cut over blocks
  std::vector<AttHead> att_heads;
  std::vector<AttPiece> att_pieces;
  std::vector<AttMerge> att_merges;
  int32_t att_ctas = 0, att_slot_rows = 0, att_num_merges = 0, att_merge_cap = 0;
  int64_t off_att_heads = 0, off_att_pieces = 0, off_att_merges = 0;
  int64_t att_tiles = 0;
  int64_t upload_bytes = 0;  // [0, upload_bytes) of the workspace comes from `blob`
  std::vector<uint8_t> blob;
};

namespace {

sps_status validate_problem(const sps_problem* p) {
  if (!p) return fail(SPS_EINVAL, "problem is NULL");
  if (p->batch < 1) return fail(SPS_EINVAL, "batch must be >= 1 (got %d)", p->batch);
  if (!p->q_lens || !p->ctx_lens) return fail(SPS_EINVAL, "q_lens/ctx_lens must be host arrays");
  if (p->page_size != kPage) return fail(SPS_EUNSUPPORTED, "page_size must be 128");
  if (p->head_dim != 64 && p->head_dim != 128)
    return fail(SPS_EUNSUPPORTED, "head_dim must be 64 or 128 (got %d)", p->head_dim);
  if (p->num_q_heads < 1 || p->num_kv_heads < 1 || p->num_q_heads % p->num_kv_heads)
    return fail(SPS_EINVAL, "num_q_heads (%d) must be a positive multiple of num_kv_heads (%d)",
                p->num_q_heads, p->num_kv_heads);
  if (p->top_k < 1 || p->top_k > kMaxTopK)
    return fail(SPS_EINVAL, "top_k must be in [1, %d] (got %d)", kMaxTopK, p->top_k);
  if (p->num_phys_pages < 1) return fail(SPS_EINVAL, "num_phys_pages must be >= 1");
  if (!(p->softmax_scale > 0.f) || !std::isfinite(p->softmax_scale))
    return fail(SPS_EINVAL, "softmax_scale must be finite and > 0");
  bool attn_ok = (p->q_dtype == SPS_BF16 && p->kv_dtype == SPS_BF16) ||
                 (p->q_dtype == SPS_E4M3 && p->kv_dtype == SPS_NVFP4);
  if (!attn_ok) return fail(SPS_EUNSUPPORTED, "attention dtypes must be BF16/BF16 or E4M3/NVFP4");
  bool idx_ok = (p->idx_q_dtype == SPS_BF16 && p->idx_k_dtype == SPS_BF16) ||
                (p->idx_q_dtype == SPS_E4M3 && p->idx_k_dtype == SPS_E4M3) ||
                (p->idx_q_dtype == SPS_E4M3 && p->idx_k_dtype == SPS_NVFP4);
  if (!idx_ok)
    return fail(SPS_EUNSUPPORTED, "indexer dtypes must be BF16/BF16, E4M3/E4M3 or E4M3/NVFP4");
  if (p->idx_q_dtype == SPS_E4M3 && p->idx_k_dtype == SPS_E4M3 && p->head_dim != 128)
    return fail(SPS_EUNSUPPORTED, "the E4M3 x E4M3 indexer needs head_dim 128");
  int64_t T = 0;
  for (int b = 0; b < p->batch; ++b) {
    if (p->q_lens[b] < 0 || p->ctx_lens[b] < 0)
      return fail(SPS_EINVAL, "request %d: negative q_len/ctx_len", b);
    int64_t last = (int64_t)p->ctx_lens[b] + p->q_lens[b] - 1;
    if (last >= (int64_t)1 << 24) return fail(SPS_EINVAL, "request %d: sequence too long", b);
    int64_t np = p->q_lens[b] > 0 ? last / kPage + 1 : 0;
    if (np > p->max_pages_per_req)
      return fail(SPS_EINVAL, "request %d needs %lld pages > max_pages_per_req %d", b,
                  (long long)np, p->max_pages_per_req);
    T += p->q_lens[b];
  }
  if (T < 1) return fail(SPS_EINVAL, "the batch has no query tokens");
  int64_t R = T * p->num_q_heads;
  if (R * p->top_k >= ((int64_t)1 << 31) || R * p->head_dim >= ((int64_t)1 << 40))
    return fail(SPS_EUNSUPPORTED, "batch too large (rows x top_k must stay below 2^31)");
  const int page_cap = p->top_k <= 16 ? kMaxPagesPerReq : kMaxPagesWideK;
  if (p->max_pages_per_req > page_cap)
    return fail(SPS_EUNSUPPORTED,
                "max_pages_per_req above %d (%dK tokens of context per request) is not supported "
                "with top_k %d",
                page_cap, page_cap * kPage / 1024, p->top_k);
  return SPS_OK;
}

// Indexer work list: tiles of <= 128 tokens x (1 or 2 heads of one KV group) against page
// chunks; the chunk starts at 128 pages and halves (down to 8) until there are enough items
// for a few waves.  Items are ordered by decreasing page count (largest first), then by
// their natural order, so a static round-robin over CTAs balances well.
void build_indexer_tasks(sps_plan* pl) {
  const sps_problem& p = pl->pb;
  const int Hg = p.num_q_heads / p.num_kv_heads;
  const int nh = (Hg % 2 == 0) ? 2 : 1;
  const int64_t target = 4LL * std::max(1, num_sms());
  // items and their page counts at a chunk size, found without listing them
  auto count = [&](int chunk, std::vector<int64_t>& by_pages) {
    by_pages.assign(chunk + 1, 0);
    int64_t n = 0;
    for (const ReqInfo& ri : pl->reqs)
      for (int i0 = 0; i0 < ri.q_len; i0 += kPage) {
        const int pages = (ri.ctx + std::min(i0 + kPage, ri.q_len) - 1) / kPage + 1;
        by_pages[chunk] += pages / chunk;
        if (pages % chunk) ++by_pages[pages % chunk];
        n += (pages + chunk - 1) / chunk;
      }
    const int64_t heads = (int64_t)p.num_kv_heads * (Hg / nh);
    for (int64_t& x : by_pages) x *= heads;
    return n * heads;
  };
  int chunk = 128;
  std::vector<int64_t> at;
  int64_t total = count(chunk, at);
  while (total < target && chunk > 8) total = count(chunk /= 2, at);
  // each page count's place in the list, the largest first
  int64_t next = 0;
  for (int n = chunk; n >= 1; --n) {
    const int64_t c = at[n];
    at[n] = next;
    next += c;
  }
  pl->idx_tasks.resize(total);
  for (int b = 0; b < p.batch; ++b) {
    const ReqInfo& ri = pl->reqs[b];
    for (int i0 = 0; i0 < ri.q_len; i0 += kPage) {
      const int ntok = std::min(kPage, ri.q_len - i0);
      const int o_last = (ri.ctx + i0 + ntok - 1) / kPage;
      for (int g = 0; g < p.num_kv_heads; ++g)
        for (int hl = 0; hl < Hg; hl += nh)
          for (int pb = 0; pb <= o_last; pb += chunk) {
            IdxTask t;
            t.req = b;
            t.g = g;
            t.h0 = g * Hg + hl;
            t.nh = nh;
            t.tok0 = ri.tok0 + i0;
            t.ntok = ntok;
            t.page_begin = pb;
            t.page_end = std::min(o_last + 1, pb + chunk);
            pl->idx_tasks[at[t.page_end - pb]++] = t;
          }
    }
  }
}

// Work split of the full attention: tiles (two row tiles of 128 / HB tokens x HB heads of a KV head's
// group, over the pages their last token sees) and pieces of tiles, listed for one block per SM.
//
// Costs are in pages (about 1.6 us): a piece's pages plus kAttTileCost for its fill, drain and
// epilogue.  A cut tile's partial rows are written and merged by a second kernel, which is estimated
// too; of the splits made, the one with the smallest estimate is kept.
// A left-over piece has at least kAttMinPiece pages (32 tokens after 1K: 3 cost 36.0 us, 5 34.4; 8
// cost four chunks after 2K to 9K 3 % more), and a tile cost of 1 or 3 measured slower or the same.
constexpr int kAttTileCost = 2, kAttMinPiece = 5;

struct AttTile {
  int32_t req, vg, tile, pages;
};

// The tiles, and the cost in front of each: `at` has one entry more.
struct AttTiles {
  std::vector<AttTile> list;
  std::vector<int64_t> at;
  int max_pages = 0;
};

// What a split costs: its longest block, and its cut tiles' pieces to merge.  One unit for kernels whose
// page takes 0.7 us (single tokens over NVFP4) to 1.6 us (two row tiles): a rule of thumb.  Measured,
// us, with the merge left out and with it doubled (H / H_kv 32 / 8, 32 / 2, 4 / 2 and 32 / 4):
//   few rows   32 tokens after 1K 32.8 (38.0, 32.8), 64 after 2K over NVFP4 16.0 (28.1, 16.0), 20 after
//              5K 74.2 (70.0, 74.3); one token after 8K or 128K the same
//   many rows  a 512-token prompt 12.7 (14.5, 12.7), five ragged requests D 64 14.1 (14.1, 18.5), D 128
//              21.0 (18.8, 21.0), four chunks over NVFP4 165 (171, 165)
double split_estimate(int64_t longest, int64_t pieces, bool few_rows) {
  const double merge = few_rows ? 6 + 0.01 * pieces : 2.5 + 0.05 * pieces;
  return (double)longest + (pieces ? merge : 0);
}

// A block's begin (or cut): a tile and a page of it.
struct AttPos {
  int32_t tile, page;
};

// The (tile, page) pairs in order, cut into runs of equal cost.  A cut at most `snap` pages from a
// tile's border moves onto the nearer one.  (Measured on H 32 / H_kv 8, D 128: 32 single tokens after
// 1K cost 42 us with snap 5 and 49 with 1, a 512-token prompt 15 and 20; one token after 8K, where
// every cut counts, 17 and 14.)
// `cuts` are the equal runs' begins, a page below the cost of a tile's start counted as its page 0;
// `begins` are the blocks' begins after the snap.
struct AttRuns {
  std::vector<AttPos> begins;
  int64_t longest = 0, pieces = 0;
};
std::vector<AttPos> equal_cuts(const AttTiles& t, int ctas) {
  const int64_t total = t.at.back(), n = std::min<int64_t>(ctas, total);
  std::vector<AttPos> cuts(n);
  size_t k = 0;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t bound = i * total / n;
    // (a cut is usually a few tiles behind the one before, or many)
    if (bound >= t.at[k + 1]) k = std::upper_bound(t.at.begin() + k + 1, t.at.end(), bound) - t.at.begin() - 1;
    cuts[i] = AttPos{(int32_t)k, (int32_t)std::max<int64_t>(0, bound - t.at[k] - kAttTileCost)};
  }
  return cuts;
}
void split_runs(const AttTiles& t, const std::vector<AttPos>& cuts, int snap, AttRuns& out) {
  out.begins.clear();
  out.longest = out.pieces = 0;
  out.begins.push_back(AttPos{0, 0});
  int64_t from = 0;  // cost in front of the present block
  auto begin = [&](int32_t tile, int32_t page) {
    const AttPos& l = out.begins.back();
    if (tile < l.tile || (tile == l.tile && page <= l.page)) return;
    const int64_t border = t.at[tile] + page;
    out.longest = std::max(out.longest, border + (page ? kAttTileCost : 0) - from);
    out.pieces += page == 0 ? 0 : l.tile == tile && l.page ? 1 : 2;  // the piece in front, and the rest
    from = border;
    out.begins.push_back(AttPos{tile, page});
  };
  for (const AttPos& c : cuts) {
    const int n = t.list[c.tile].pages;
    const bool front = c.page <= n - c.page;
    if (c.page == 0 || (front && c.page <= snap)) begin(c.tile, 0);
    else if (front || n - c.page > snap) begin(c.tile, c.page);
    else if (c.tile + 1 < (int32_t)t.list.size()) begin(c.tile + 1, 0);
  }
  out.longest = std::max(out.longest, t.at.back() - from);
}

// Whole tiles, the largest first, each to the block with the least work as long as that stays within
// an equal share; the tiles left over are cut to fill the blocks up.  Blocks that work at the same
// time then read the same keys: 8 x 512 tokens after 32K reads 270 MB of keys and values that
// consecutive runs, each block at another place, would stream past the L2 again and again.
// (Loads only grow, so the least loaded block is found by walking a list of blocks per load.)
struct AttShares {
  std::vector<int32_t> order;             // tiles by falling pages
  std::vector<int32_t> at_load, peer;     // blocks of a load, linked
  std::vector<int32_t> first, last, next; // a block's tiles, linked
  std::vector<int32_t> rest;
  int64_t share = 0, low = 0, longest = 0, pieces = 0;

  void sort(const AttTiles& t) {
    std::vector<int32_t> from(t.max_pages + 2, 0);
    for (const AttTile& x : t.list) ++from[t.max_pages - x.pages + 1];
    for (int i = 0; i <= t.max_pages; ++i) from[i + 1] += from[i];
    order.resize(t.list.size());
    for (size_t k = 0; k < t.list.size(); ++k)
      order[from[t.max_pages - t.list[k].pages]++] = (int32_t)k;
  }
  // The whole tiles' places, and what is left over.
  void place(const AttTiles& t, int64_t s, int ctas) {
    share = s;
    at_load.assign(share + 1, -1);
    peer.resize(ctas);
    first.assign(ctas, -1);
    last.assign(ctas, -1);
    next.assign(t.list.size(), -1);
    rest.clear();
    for (int i = ctas - 1; i >= 0; --i) {
      peer[i] = at_load[0];
      at_load[0] = i;
    }
    low = 0;
    for (int32_t k : order) {
      while (at_load[low] < 0) ++low;
      const int64_t load = low + t.list[k].pages + kAttTileCost;
      if (load > share) {
        rest.push_back(k);
        continue;
      }
      const int32_t c = at_load[low];
      at_load[low] = peer[c];
      peer[c] = at_load[load];
      at_load[load] = c;
      (first[c] < 0 ? first[c] : next[last[c]]) = k;
      last[c] = k;
    }
  }
  // The blocks in turn, the ones with the most room first, filled up with the left-over tiles:
  // block() at each, run(tile, page0, page1) for its pieces.  False: some do not fit.
  template <typename Block, typename Run>
  bool fill(const AttTiles& t, Block block, Run run) {
    longest = pieces = 0;
    size_t j = 0;
    int page = 0;
    for (int64_t l = low; l <= share; ++l)
      for (int32_t c = at_load[l]; c >= 0; c = peer[c]) {
        block(c);
        int64_t room = share - l;
        while (j < rest.size() && room >= kAttTileCost + kAttMinPiece) {
          const int n = t.list[rest[j]].pages;
          int to = (int)std::min<int64_t>(n, page + room - kAttTileCost);
          if (n - to < kAttMinPiece) to = n;
          run(rest[j], page, to);
          pieces += page > 0 || to < n;
          room -= to - page + kAttTileCost;
          page = to;
          if (to < n) break;
          ++j;
          page = 0;
        }
        longest = std::max(longest, share - room);
      }
    return j == rest.size();
  }
};

void build_attention_work(sps_plan* pl) {
  const sps_problem& p = pl->pb;
  const int hg = p.num_q_heads / p.num_kv_heads, HB = std::min(hg, 128), TB = 128 / HB;
  const int nv = p.num_kv_heads * ((hg + HB - 1) / HB), tt = 2 * TB;
  AttTiles tiles;
  int64_t count = 0;
  int max_q = 0;
  for (const ReqInfo& ri : pl->reqs) {
    count += (int64_t)nv * ((ri.q_len + tt - 1) / tt);
    max_q = std::max(max_q, ri.q_len);
  }
  tiles.list.resize(count);
  tiles.at.resize(count + 1);
  int64_t k = 0, at = 0;
  for (int b = 0; b < p.batch; ++b) {
    const ReqInfo& ri = pl->reqs[b];
    for (int v = 0; v < nv; ++v)
      for (int t = 0; t * tt < ri.q_len; ++t) {
        const int n = (ri.ctx + std::min((t + 1) * tt, ri.q_len) - 1) / kPage + 1;
        tiles.list[k] = AttTile{b, v, t, n};
        tiles.at[k++] = at;
        at += n + kAttTileCost;
        tiles.max_pages = std::max(tiles.max_pages, n);
      }
  }
  tiles.at[k] = at;
  const int64_t total = at;
  const int ctas = std::min(std::max(1, num_sms()), 256);
  pl->att_ctas = ctas;
  pl->att_tiles = count;
  pl->att_slot_rows = max_q > TB ? 256 : max_q * HB;
  pl->att_merge_cap = (int32_t)std::min<int64_t>(ctas - 1, count);

  // the splits' estimates: runs by snap, or shares of a size at which the left-over tiles fit
  const bool few_rows = pl->att_slot_rows <= 32;
  const std::vector<AttPos> cuts = equal_cuts(tiles, ctas);
  AttRuns runs, trial;
  double best = 0;
  for (int s : {1, 2, 4, 8, 1 << 20}) {
    split_runs(tiles, cuts, s, trial);
    const double x = split_estimate(trial.longest, trial.pieces, few_rows);
    if (s == 1 || x < best) {
      best = x;
      std::swap(runs, trial);
    }
    if (count >= 8 * ctas) break;
  }
  AttShares shares;
  bool shared = false;
  if (count > ctas) {
    shares.sort(tiles);
    for (int64_t x = (total + ctas - 1) / ctas + kAttTileCost; (double)x < best && x < 1 << 20;
         x += std::max<int64_t>(1, x / 64)) {
      shares.place(tiles, x, ctas);
      if (!shares.fill(tiles, [](int) {}, [](int, int, int) {})) continue;
      shared = split_estimate(shares.longest, shares.pieces, few_rows) < best;
      break;
    }
  }

  pl->att_heads.assign(ctas, AttHead{});
  pl->att_merges.assign(ctas, AttMerge{-1, 0, 0, 0, 0, 0, 0, 0});
  pl->att_pieces.resize(count + 2 * ctas);  // (the blob's room)
  AttPiece* next = pl->att_pieces.data();
  int merges = 0, cta = -1;
  auto run = [&](int tile, int page0, int page1) {  // a piece more of block `cta`
    const AttTile& t = tiles.list[tile];
    const ReqInfo& ri = pl->reqs[t.req];
    AttHead& h = pl->att_heads[cta];
    AttPiece* x = &h.first;
    if (h.count++ == 0) h.next = (int32_t)(next - pl->att_pieces.data());
    else x = next++;
    *x = AttPiece{t.req, t.vg, t.tile, page0, page1, ri.q_len, ri.ctx, ri.tok0};
    if (page0 == 0 && page1 < t.pages)
      pl->att_merges[merges++] = AttMerge{t.req, t.vg, t.tile, cta, cta, ri.q_len, ri.tok0, 0};
    else if (page0 > 0)
      pl->att_merges[merges - 1].cta1 = cta;
  };
  if (shared) {
    shares.fill(
        tiles,
        [&](int c) {
          ++cta;
          for (int32_t i = shares.first[c]; i >= 0; i = shares.next[i]) run(i, 0, tiles.list[i].pages);
        },
        run);
  } else {
    for (size_t i = 0; i < runs.begins.size(); ++i) {
      ++cta;
      const bool end = i + 1 == runs.begins.size();
      const AttPos to = end ? AttPos{(int32_t)count, 0} : runs.begins[i + 1];
      for (AttPos x = runs.begins[i]; x.tile < to.tile; x = AttPos{x.tile + 1, 0})
        run(x.tile, x.page, tiles.list[x.tile].pages);
      if (to.page) {
        const AttPos& x = runs.begins[i];
        run(to.tile, x.tile == to.tile ? x.page : 0, to.page);
      }
    }
  }
  pl->att_num_merges = merges;
}

// Fills the plan of a valid problem (throws std::bad_alloc).
void make_plan(const sps_problem& problem, sps_plan* pl) {
  pl->pb = problem;
  const sps_problem& p = pl->pb;
  pl->q_lens.assign(problem.q_lens, problem.q_lens + p.batch);
  pl->ctx_lens.assign(problem.ctx_lens, problem.ctx_lens + p.batch);
  pl->pb.q_lens = pl->q_lens.data();
  pl->pb.ctx_lens = pl->ctx_lens.data();
  const int Hg = p.num_q_heads / p.num_kv_heads;

  // per-request info, per-token metadata
  const size_t num_tokens = std::accumulate(pl->q_lens.begin(), pl->q_lens.end(), (size_t)0);
  std::vector<int32_t> tok_pos(num_tokens), tok_req(num_tokens);
  pl->reqs.reserve(p.batch);
  int32_t tok = 0, page_base = 0;
  for (int b = 0; b < p.batch; ++b) {
    ReqInfo ri{};
    ri.tok0 = tok;
    ri.q_len = pl->q_lens[b];
    ri.ctx = pl->ctx_lens[b];
    ri.npages = ri.q_len > 0 ? (ri.ctx + ri.q_len - 1) / kPage + 1 : 0;
    ri.page_base = page_base;
    ri.words = (int32_t)((int64_t(ri.q_len) * Hg + 31) / 32);
    ri.ch_per_bucket = (ri.words + kChunkWords - 1) / kChunkWords;
    ri.blk_base = (int32_t)pl->inv_blocks;
    pl->inv_blocks += (int64_t)p.num_kv_heads * ri.ch_per_bucket;
    ri.ch_base = (int32_t)pl->num_chunks;
    pl->num_chunks += (int64_t)ri.npages * p.num_kv_heads * ri.ch_per_bucket;
    std::iota(tok_pos.begin() + tok, tok_pos.begin() + tok + ri.q_len, ri.ctx);
    std::fill_n(tok_req.begin() + tok, ri.q_len, b);
    pl->page_req.insert(pl->page_req.end(), ri.npages, b);
    page_base += ri.npages;
    tok += ri.q_len;
    pl->reqs.push_back(ri);
  }
  pl->T = tok;
  pl->R = (int64_t)tok * p.num_q_heads;
  pl->total_pages = page_base;
  pl->num_buckets = (int64_t)page_base * p.num_kv_heads;
  pl->max_entries = pl->R * p.top_k;
  const int64_t per_task = (int64_t)kFwdTaskGroups * 128;
  pl->max_fwd_tasks = pl->max_entries / per_task + pl->num_buckets + 1;
  build_indexer_tasks(pl);
  build_attention_work(pl);

  // workspace layout
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    int64_t o = off;
    off = align_up(off + std::max<int64_t>(bytes, 4), 256);
    return o;
  };
  // the full attention's tables, in front: the no-allocation forward leaves them out.  (Their sizes
  // and those up to off_page_req follow from q_lens and the heads alone: a plan with other contexts
  // has the same layout up to there.)
  pl->off_att_heads = take(sizeof(AttHead) * pl->att_heads.size());
  pl->off_att_merges = take(sizeof(AttMerge) * pl->att_merges.size());
  pl->off_att_pieces = take(sizeof(AttPiece) * (pl->att_tiles + 2 * pl->att_ctas));
  pl->fwd_base = off;
  pl->off_status = take(4);
  pl->off_counters = take(16 * 4);
  pl->off_tok_pos = take(4 * pl->T);
  pl->off_tok_req = take(4 * pl->T);
  pl->off_reqs = take(sizeof(ReqInfo) * p.batch);
  pl->off_page_req = take(4 * std::max<int64_t>(1, pl->total_pages));
  pl->off_idx_tasks = take(sizeof(IdxTask) * std::max<size_t>(1, pl->idx_tasks.size()));
  int64_t upload_end = off;
  pl->off_chunk_offsets = take(4 * (pl->num_chunks + 1));
  pl->off_bucket_totals = take(4 * pl->num_buckets);
  // per block of the single-launch inversion, or of the multi-kernel one's scan: its range's
  // entries and work items
  pl->off_range_sums = take(8 * std::max<int64_t>(
      {int64_t(1), pl->inv_blocks, (pl->num_buckets + kInvScanBuckets - 1) / kInvScanBuckets}));
  pl->off_bucket_offsets = take(4 * (pl->num_buckets + 1));
  pl->off_entries = take(8 * std::max<int64_t>(1, pl->max_entries));
  pl->off_fwd_tasks = take(sizeof(FwdTask) * pl->max_fwd_tasks);
  // FP16 staging of quantised inputs for the tensor-core paths: an exact FP16 copy of E4M3 Q;
  // an indexer over NVFP4 keys also takes FP16 copies of the key tiles of the pages the batch
  // sees (every one of them is read by the indexer), so the workspace grows with the batch,
  // not with the physical pool.  The forward dequantises NVFP4 K/V inside its loader, and
  // E4M3 x E4M3 indexing runs on the FP8 tensor core directly; neither needs a copy.
  const bool idx_fp16 = p.idx_k_dtype == SPS_NVFP4;
  if (p.q_dtype == SPS_E4M3 || (idx_fp16 && p.idx_q_dtype == SPS_E4M3))
    pl->off_qconv = take(2 * pl->R * p.head_dim);
  if (idx_fp16)
    pl->off_kconv = take(2 * std::max<int64_t>(1, pl->total_pages) * p.num_kv_heads * kPage *
                         p.head_dim);
  pl->fwd_ws_bytes = off - pl->fwd_base;
  // at most 128 entries per bucket on average: most work items are a single group
  pl->fwd_prefetch = pl->max_entries <= 128 * std::max<int64_t>(1, pl->num_buckets) ? 1 : 0;
  // Top-k with top_k <= 16 runs a thread per row, so long rows of a small batch leave few
  // warps, each walking hundreds of 16-page groups one after another.  From 64 groups on, pass
  // 1 is split into segments of at least 32 groups, enough of them for ~24 warps per SM of a
  // 152-SM GPU; each segment's 16 largest scores go to this area and merge per row, and the
  // largest score of each 16-page group lets pass 2 read only the groups that can hold a
  // chosen page.
  const int64_t groups = (p.max_pages_per_req + 15) / 16;
  if (p.top_k > 1 && p.top_k <= 16 && groups >= 64) {
    const int64_t warps = (pl->R + 31) / 32, target = 24 * 152;
    const int64_t nseg = std::min<int64_t>(groups / 32, (target + warps - 1) / warps);
    if (nseg >= 2) {
      pl->topk_nseg = (int32_t)nseg;
      pl->topk_segg = (int32_t)((groups + nseg - 1) / nseg);
      pl->off_topk_lists = take(4 * 16 * pl->R * nseg);
      pl->off_topk_meta = take(4 * 3 * pl->R);
      pl->off_topk_gmax = take(4 * groups * pl->R);
    }
  }
  pl->ws_bytes = off;

  // the host image of [0, upload_end): the metadata, the status word and counters (zero)
  pl->upload_bytes = upload_end;
  pl->blob.assign(pl->upload_bytes, 0);
  auto put = [&](int64_t o, const void* src, size_t n) {
    if (n) memcpy(pl->blob.data() + o, src, n);
  };
  put(pl->off_tok_pos, tok_pos.data(), 4 * tok_pos.size());
  put(pl->off_tok_req, tok_req.data(), 4 * tok_req.size());
  put(pl->off_reqs, pl->reqs.data(), sizeof(ReqInfo) * pl->reqs.size());
  put(pl->off_att_heads, pl->att_heads.data(), sizeof(AttHead) * pl->att_heads.size());
  put(pl->off_att_pieces, pl->att_pieces.data(), sizeof(AttPiece) * pl->att_pieces.size());
  put(pl->off_att_merges, pl->att_merges.data(), sizeof(AttMerge) * pl->att_merges.size());
  put(pl->off_page_req, pl->page_req.data(), 4 * pl->page_req.size());
  put(pl->off_idx_tasks, pl->idx_tasks.data(), sizeof(IdxTask) * pl->idx_tasks.size());
}

}  // namespace

extern "C" {

const char* sps_last_error(void) { return g_err.c_str(); }

sps_status sparse_prefill_plan(const sps_problem* problem, sps_plan** out,
                               size_t* workspace_bytes) {
  if (!out || !workspace_bytes) return fail(SPS_EINVAL, "plan/workspace_bytes out-pointers NULL");
  *out = nullptr;
  sps_status st = validate_problem(problem);
  if (st != SPS_OK) return st;
  try {
    std::unique_ptr<sps_plan> pl(new sps_plan());
    make_plan(*problem, pl.get());
    *workspace_bytes = (size_t)pl->ws_bytes;
    *out = pl.release();
    return SPS_OK;
  } catch (const std::bad_alloc&) {
    return fail(SPS_EINVAL, "out of host memory");
  }
}

void sps_plan_destroy(sps_plan* plan) { delete plan; }

sps_status sps_plan_get_info(const sps_plan* pl, sps_plan_info* info) {
  if (!pl || !info) return fail(SPS_EINVAL, "plan/info NULL");
  info->num_tokens = pl->T;
  info->num_rows = pl->R;
  info->num_buckets = pl->num_buckets;
  info->max_entries = pl->max_entries;
  info->indexer_tasks = (int64_t)pl->idx_tasks.size();
  info->max_fwd_tasks = pl->max_fwd_tasks;
  info->workspace_bytes = pl->ws_bytes;
  info->off_status = pl->off_status;
  info->off_tok_pos = pl->off_tok_pos;
  info->off_tok_req = pl->off_tok_req;
  info->off_bucket_offsets = pl->off_bucket_offsets;
  info->off_entries = pl->off_entries;
  info->off_fwd_task_count = pl->off_counters + 2 * 4;
  return SPS_OK;
}

}  // extern "C"

namespace {

DevPlan make_dev_plan(const sps_plan* pl, void* ws) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  const sps_problem& p = pl->pb;
  DevPlan d{};
  d.batch = p.batch;
  d.T = (int32_t)pl->T;
  d.H = p.num_q_heads;
  d.Hkv = p.num_kv_heads;
  d.Hg = p.num_q_heads / p.num_kv_heads;
  d.D = p.head_dim;
  d.K = p.top_k;
  d.max_pages = p.max_pages_per_req;
  d.num_phys = p.num_phys_pages;
  d.num_buckets = (int32_t)pl->num_buckets;
  d.max_entries = (int32_t)pl->max_entries;
  d.max_fwd_tasks = (int32_t)pl->max_fwd_tasks;
  d.n_idx_tasks = (int32_t)pl->idx_tasks.size();
  d.total_pages = (int32_t)pl->total_pages;
  d.inv_blocks = (int32_t)pl->inv_blocks;
  d.sm_scale = p.softmax_scale;
  d.status = reinterpret_cast<int32_t*>(base + pl->off_status);
  d.counters = reinterpret_cast<int32_t*>(base + pl->off_counters);
  d.tok_pos = reinterpret_cast<const int32_t*>(base + pl->off_tok_pos);
  d.tok_req = reinterpret_cast<const int32_t*>(base + pl->off_tok_req);
  d.reqs = reinterpret_cast<const ReqInfo*>(base + pl->off_reqs);
  d.page_req = reinterpret_cast<const int32_t*>(base + pl->off_page_req);
  d.idx_tasks = reinterpret_cast<const IdxTask*>(base + pl->off_idx_tasks);
  d.num_chunks = (int32_t)pl->num_chunks;
  d.chunk_offsets = reinterpret_cast<int32_t*>(base + pl->off_chunk_offsets);
  d.bucket_offsets = reinterpret_cast<int32_t*>(base + pl->off_bucket_offsets);
  d.bucket_totals = reinterpret_cast<int32_t*>(base + pl->off_bucket_totals);
  d.range_sums = reinterpret_cast<int32_t*>(base + pl->off_range_sums);
  d.entries = reinterpret_cast<int2*>(base + pl->off_entries);
  d.fwd_tasks = reinterpret_cast<FwdTask*>(base + pl->off_fwd_tasks);
  d.qconv = pl->off_qconv >= 0 ? base + pl->off_qconv : nullptr;
  d.kconv = pl->off_kconv >= 0 ? base + pl->off_kconv : nullptr;
  d.topk_lists = pl->off_topk_lists >= 0 ? reinterpret_cast<float*>(base + pl->off_topk_lists)
                                         : nullptr;
  d.topk_meta = pl->off_topk_meta >= 0 ? reinterpret_cast<int32_t*>(base + pl->off_topk_meta)
                                       : nullptr;
  d.topk_gmax = pl->off_topk_gmax >= 0 ? reinterpret_cast<float*>(base + pl->off_topk_gmax)
                                       : nullptr;
  d.topk_nseg = pl->topk_nseg;
  d.fwd_prefetch = pl->fwd_prefetch;
  d.topk_segg = pl->topk_segg;
  d.att_heads = reinterpret_cast<const AttHead*>(base + pl->off_att_heads);
  d.att_pieces = reinterpret_cast<const AttPiece*>(base + pl->off_att_pieces);
  d.att_merges = reinterpret_cast<const AttMerge*>(base + pl->off_att_merges);
  d.att_ctas = pl->att_ctas;
  d.att_slot_rows = pl->att_slot_rows;
  d.att_num_merges = pl->att_num_merges;
  d.att_merge_cap = pl->att_merge_cap;
  return d;
}

sps_status check_plan_ws(const sps_plan* pl, const void* ws) {
  if (!pl) return fail(SPS_EINVAL, "plan is NULL");
  if (!ws) return fail(SPS_EINVAL, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(SPS_EINVAL, "workspace must be 256-byte aligned");
  return SPS_OK;
}

sps_status launched(cudaError_t e, const char* what) {
  if (e == cudaErrorNotSupported)
    return fail(SPS_EUNSUPPORTED, "%s: not implemented for this dtype combination / head_dim",
                what);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return SPS_OK;
}

}  // namespace

extern "C" {

sps_status sps_plan_upload(const sps_plan* pl, void* ws, size_t ws_bytes, sps_stream_t stream) {
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  if ((int64_t)ws_bytes < pl->ws_bytes)
    return fail(SPS_ENOSPACE, "workspace of %zu bytes < %lld required", ws_bytes,
                (long long)pl->ws_bytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  // one copy: the plan metadata, the zeroed status word and counters
  cudaError_t e = g_staging.upload(base, pl->blob.data(), pl->upload_bytes, s, true);
  if (e != cudaSuccess) return cuda_fail(e, "plan upload");
  return SPS_OK;
}

sps_status indexer_scores(const sps_plan* pl, const void* q_idx, float q_scale,
                          const void* k_idx_cache, const void* k_idx_scales, float k_scale,
                          const int32_t* page_table, float* scores, int64_t score_pitch,
                          void* ws, sps_stream_t stream) {
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  const sps_problem& p = pl->pb;
  if (!q_idx || !k_idx_cache || !page_table || !scores)
    return fail(SPS_EINVAL, "indexer_scores: NULL input/output pointer");
  if (p.idx_k_dtype == SPS_NVFP4 && !k_idx_scales)
    return fail(SPS_EINVAL, "indexer_scores: NVFP4 keys need k_idx_scales");
  if (score_pitch < p.max_pages_per_req)
    return fail(SPS_EINVAL, "score_pitch %lld < max_pages_per_req %d", (long long)score_pitch,
                p.max_pages_per_req);
  if (!aligned(q_idx, 16) || !aligned(k_idx_cache, 16) || (k_idx_scales && !aligned(k_idx_scales, 16)))
    return fail(SPS_EINVAL, "indexer_scores: q/k buffers must be 16-byte aligned");
  if (!aligned(scores, 4)) return fail(SPS_EINVAL, "scores must be 4-byte aligned");
  if (!std::isfinite(q_scale) || !std::isfinite(k_scale))
    return fail(SPS_EINVAL, "indexer_scores: scales must be finite");
  DevPlan d = make_dev_plan(pl, ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(launch_indexer(d, p.idx_q_dtype, p.idx_k_dtype, q_idx, q_scale, k_idx_cache,
                                 k_idx_scales, k_scale, page_table, scores, score_pitch, s),
                  "indexer launch");
}

sps_status topk_select(const sps_plan* pl, const float* scores, int64_t score_pitch,
                       int32_t* idx, void* ws, sps_stream_t stream) {
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  if (!scores || !idx) return fail(SPS_EINVAL, "topk_select: NULL scores/idx");
  if (score_pitch < pl->pb.max_pages_per_req)
    return fail(SPS_EINVAL, "score_pitch %lld < max_pages_per_req %d", (long long)score_pitch,
                pl->pb.max_pages_per_req);
  if (!aligned(scores, 4) || !aligned(idx, 4)) return fail(SPS_EINVAL, "misaligned scores/idx");
  DevPlan d = make_dev_plan(pl, ws);
  return launched(launch_topk(d, scores, score_pitch, idx, reinterpret_cast<cudaStream_t>(stream)),
                  "top-k launch");
}

namespace {

// The forward with FP32, BF16 or FP16 partials, or the FP8-QK route: the same checks and
// launches.
enum class FwdKind { kFP32, kBF16Partials, kF16Partials, kFP8QK };
sps_status fwd_common(const sps_plan* pl, const void* q, float q_scale, const void* k_cache,
                      const void* v_cache, const void* k_scales, const void* v_scales,
                      const int32_t* page_table, const int32_t* idx, void* partial,
                      int64_t split_stride, float* lse, int64_t lse_split_stride, void* ws,
                      sps_stream_t stream, FwdKind kind) {
  const bool p16 = kind == FwdKind::kBF16Partials || kind == FwdKind::kF16Partials;
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  const sps_problem& p = pl->pb;
  if (!q || !k_cache || !v_cache || !page_table || !idx || !partial || !lse)
    return fail(SPS_EINVAL, "sparse_prefill_fwd: NULL input/output pointer");
  if (p.kv_dtype == SPS_NVFP4 && (!k_scales || !v_scales))
    return fail(SPS_EINVAL, "sparse_prefill_fwd: NVFP4 K/V need k_scales and v_scales");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      (k_scales && !aligned(k_scales, 16)) || (v_scales && !aligned(v_scales, 16)))
    return fail(SPS_EINVAL, "sparse_prefill_fwd: q/k/v buffers must be 16-byte aligned");
  if (!aligned(partial, 16)) return fail(SPS_EINVAL, "partial must be 16-byte aligned");
  const int64_t qa = p16 ? 8 : 4;  // elements per 16 bytes
  if (split_stride < pl->R * p.head_dim || split_stride % qa)
    return fail(SPS_EINVAL, "split_stride must be >= rows*head_dim and a multiple of %lld",
                (long long)qa);
  if (lse_split_stride < pl->R) return fail(SPS_EINVAL, "lse_split_stride must be >= rows");
  if (!std::isfinite(q_scale)) return fail(SPS_EINVAL, "q_scale must be finite");
  if (kind == FwdKind::kFP8QK &&
      (p.q_dtype != SPS_E4M3 || p.kv_dtype != SPS_NVFP4 || p.head_dim != 128))
    return fail(SPS_EUNSUPPORTED, "sparse_prefill_fwd_fp8qk: needs E4M3 Q, NVFP4 K/V, D = 128");
  DevPlan d = make_dev_plan(pl, ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // no counter needs clearing here: the inversion writes the task count, and its grid barrier
  // returns to zero when it completes (the plan upload clears it first)
  cudaError_t e = launch_inversion(d, idx, lse, lse_split_stride, s);
  if (e != cudaSuccess) return cuda_fail(e, "inversion launch");
  if (kind == FwdKind::kFP8QK)
    return launched(launch_forward_fp8qk(d, p.q_dtype, p.kv_dtype, q, q_scale, k_cache, v_cache,
                                         k_scales, v_scales, page_table,
                                         static_cast<float*>(partial), split_stride, lse,
                                         lse_split_stride, s),
                    "forward launch");
  if (kind == FwdKind::kBF16Partials)
    return launched(launch_forward_bf16p(d, p.q_dtype, p.kv_dtype, q, q_scale, k_cache, v_cache,
                                         k_scales, v_scales, page_table, partial, split_stride,
                                         lse, lse_split_stride, s),
                    "forward launch");
  if (kind == FwdKind::kF16Partials)
    return launched(launch_forward_f16p(d, p.q_dtype, p.kv_dtype, q, q_scale, k_cache, v_cache,
                                        k_scales, v_scales, page_table, partial, split_stride,
                                        lse, lse_split_stride, s),
                    "forward launch");
  return launched(launch_forward(d, p.q_dtype, p.kv_dtype, q, q_scale, k_cache, v_cache, k_scales,
                                 v_scales, page_table, static_cast<float*>(partial),
                                 split_stride, lse, lse_split_stride, s),
                  "forward launch");
}

sps_status combine_common(int64_t rows, int32_t splits, int32_t head_dim, const void* partial,
                          int64_t split_stride, const float* lse, int64_t lse_split_stride,
                          void* out_bf16, int64_t out_row_stride, float* out_lse,
                          int32_t* dev_status, sps_stream_t stream, int ptype) {
  const bool p16 = ptype != 0;  // 0: FP32, 1: BF16, 2: FP16 partials
  if (rows < 0) return fail(SPS_EINVAL, "rows must be >= 0");
  if (splits < 1 || splits > kMaxTopK) return fail(SPS_EINVAL, "splits must be in [1, 64]");
  if (head_dim != 64 && head_dim != 128) return fail(SPS_EUNSUPPORTED, "head_dim must be 64 or 128");
  if (rows == 0) return SPS_OK;
  if (!partial || !lse || !out_bf16) return fail(SPS_EINVAL, "partial_combine: NULL pointer");
  if (!aligned(partial, 16) || !aligned(out_bf16, 16) || !aligned(lse, 4))
    return fail(SPS_EINVAL, "partial/out must be 16-byte aligned, lse 4-byte aligned");
  const int64_t qa = p16 ? 8 : 4;  // elements per 16 bytes
  if (split_stride % qa || split_stride < rows * head_dim)
    return fail(SPS_EINVAL, "split_stride must be a multiple of %lld and >= rows*head_dim",
                (long long)qa);
  if (lse_split_stride < rows) return fail(SPS_EINVAL, "lse_split_stride must be >= rows");
  if (out_row_stride < head_dim || out_row_stride % 8)
    return fail(SPS_EINVAL, "out_row_stride must be >= head_dim and a multiple of 8");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (ptype == 1)
    return launched(launch_combine_bf16p(rows, splits, head_dim, partial, split_stride, lse,
                                         lse_split_stride, out_bf16, out_row_stride, out_lse,
                                         dev_status, s),
                    "combine launch");
  if (ptype == 2)
    return launched(launch_combine_f16p(rows, splits, head_dim, partial, split_stride, lse,
                                        lse_split_stride, out_bf16, out_row_stride, out_lse,
                                        dev_status, s),
                    "combine launch");
  return launched(launch_combine(rows, splits, head_dim, static_cast<const float*>(partial),
                                 split_stride, lse, lse_split_stride, out_bf16, out_row_stride,
                                 out_lse, dev_status, s),
                  "combine launch");
}

}  // namespace

sps_status sparse_prefill_fwd(const sps_plan* pl, const void* q, float q_scale,
                              const void* k_cache, const void* v_cache, const void* k_scales,
                              const void* v_scales, const int32_t* page_table,
                              const int32_t* idx, float* partial, int64_t split_stride,
                              float* lse, int64_t lse_split_stride, void* ws,
                              sps_stream_t stream) {
  return fwd_common(pl, q, q_scale, k_cache, v_cache, k_scales, v_scales, page_table, idx,
                    partial, split_stride, lse, lse_split_stride, ws, stream, FwdKind::kFP32);
}

sps_status sparse_prefill_fwd_fp8qk(const sps_plan* pl, const void* q, float q_scale,
                                    const void* k_cache, const void* v_cache,
                                    const void* k_scales, const void* v_scales,
                                    const int32_t* page_table, const int32_t* idx, float* partial,
                                    int64_t split_stride, float* lse, int64_t lse_split_stride,
                                    void* ws, sps_stream_t stream) {
  return fwd_common(pl, q, q_scale, k_cache, v_cache, k_scales, v_scales, page_table, idx,
                    partial, split_stride, lse, lse_split_stride, ws, stream, FwdKind::kFP8QK);
}

sps_status sparse_prefill_fwd_bf16(const sps_plan* pl, const void* q, float q_scale,
                                   const void* k_cache, const void* v_cache,
                                   const void* k_scales, const void* v_scales,
                                   const int32_t* page_table, const int32_t* idx,
                                   void* partial_bf16, int64_t split_stride, float* lse,
                                   int64_t lse_split_stride, void* ws, sps_stream_t stream) {
  return fwd_common(pl, q, q_scale, k_cache, v_cache, k_scales, v_scales, page_table, idx,
                    partial_bf16, split_stride, lse, lse_split_stride, ws, stream,
                    FwdKind::kBF16Partials);
}

sps_status partial_combine(int64_t rows, int32_t splits, int32_t head_dim, const float* partial,
                           int64_t split_stride, const float* lse, int64_t lse_split_stride,
                           void* out_bf16, int64_t out_row_stride, float* out_lse,
                           int32_t* dev_status, sps_stream_t stream) {
  return combine_common(rows, splits, head_dim, partial, split_stride, lse, lse_split_stride,
                        out_bf16, out_row_stride, out_lse, dev_status, stream, 0);
}

sps_status partial_combine_bf16(int64_t rows, int32_t splits, int32_t head_dim,
                                const void* partial_bf16, int64_t split_stride, const float* lse,
                                int64_t lse_split_stride, void* out_bf16, int64_t out_row_stride,
                                float* out_lse, int32_t* dev_status, sps_stream_t stream) {
  return combine_common(rows, splits, head_dim, partial_bf16, split_stride, lse,
                        lse_split_stride, out_bf16, out_row_stride, out_lse, dev_status, stream,
                        1);
}

sps_status sparse_prefill_fwd_f16(const sps_plan* pl, const void* q, float q_scale,
                                  const void* k_cache, const void* v_cache, const void* k_scales,
                                  const void* v_scales, const int32_t* page_table,
                                  const int32_t* idx, void* partial_f16, int64_t split_stride,
                                  float* lse, int64_t lse_split_stride, void* ws,
                                  sps_stream_t stream) {
  return fwd_common(pl, q, q_scale, k_cache, v_cache, k_scales, v_scales, page_table, idx,
                    partial_f16, split_stride, lse, lse_split_stride, ws, stream,
                    FwdKind::kF16Partials);
}

sps_status partial_combine_f16(int64_t rows, int32_t splits, int32_t head_dim,
                               const void* partial_f16, int64_t split_stride, const float* lse,
                               int64_t lse_split_stride, void* out_bf16, int64_t out_row_stride,
                               float* out_lse, int32_t* dev_status, sps_stream_t stream) {
  return combine_common(rows, splits, head_dim, partial_f16, split_stride, lse, lse_split_stride,
                        out_bf16, out_row_stride, out_lse, dev_status, stream, 2);
}

sps_status sps_kv_append(const sps_plan* pl, const void* k_new, const void* v_new,
                         const int32_t* page_table, void* k_cache, void* v_cache, void* k_scales,
                         void* v_scales, void* ws, sps_stream_t stream) {
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  const sps_problem& p = pl->pb;
  const bool nvfp4 = p.kv_dtype == SPS_NVFP4;
  if (p.kv_dtype != SPS_BF16 && !nvfp4)
    return fail(SPS_EUNSUPPORTED, "sps_kv_append: the cache must be BF16 or NVFP4");
  if (!k_new || !v_new || !page_table || !k_cache || !v_cache)
    return fail(SPS_EINVAL, "sps_kv_append: NULL pointer");
  if (nvfp4 && (!k_scales || !v_scales))
    return fail(SPS_EINVAL, "sps_kv_append: an NVFP4 cache needs k_scales and v_scales");
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(page_table, 4))
    return fail(SPS_EINVAL, "sps_kv_append: buffers must be 16-byte aligned");
  DevPlan d = make_dev_plan(pl, ws);
  return launched(launch_kv_append(d, nvfp4, k_new, v_new, page_table, k_cache, v_cache, k_scales,
                                   v_scales, reinterpret_cast<cudaStream_t>(stream)),
                  "kv append launch");
}

namespace {

// A caller's rotation checked and copied for the kernels; rope NULL: none.
sps_status make_rope(const sps_rope* rope, int head_dim, const char* who, DevRope* out) {
  *out = DevRope{};
  if (!rope) return SPS_OK;
  const int r = rope->rotary_dim;
  if (r < 0 || r > head_dim)
    return fail(SPS_EINVAL, "%s: rotary_dim %d outside [0, head_dim]", who, r);
  if (r % 16) return fail(SPS_EUNSUPPORTED, "%s: rotary_dim must be a multiple of 16", who);
  if (rope->num_axes < 1 || rope->num_axes > 4)
    return fail(SPS_EINVAL, "%s: num_axes must be in [1, 4] (got %d)", who, rope->num_axes);
  if (r == 0) return SPS_OK;
  if (!rope->inv_freq || !aligned(rope->inv_freq, 4) ||
      (rope->positions && !aligned(rope->positions, 4)))
    return fail(SPS_EINVAL, "%s: inv_freq must be given, it and positions 4-byte aligned", who);
  for (int j = 0; j < r / 2; ++j)
    if (rope->pair_axis[j] >= rope->num_axes)
      return fail(SPS_EINVAL, "%s: pair_axis[%d] = %d outside [0, num_axes)", who, j,
                  rope->pair_axis[j]);
  out->inv_freq = rope->inv_freq;
  out->positions = rope->positions;
  out->rot = r;
  memcpy(out->axis, rope->pair_axis, sizeof out->axis);
  return SPS_OK;
}

DevQuot make_quot(float s) {
  DevQuot d{s, NAN, 0.f, 0.f};
  if (!(s >= 0x1p-90f && s <= 0x1p90f)) return d;  // the kernel divides
  const double inv = 1.0 / s;
  d.r = 1.f / s;
  d.hi = (float)inv;
  if ((double)d.hi > inv) d.hi = std::nextafterf(d.hi, 0.f);
  d.lo = (float)(inv - d.hi);
  return d;
}

bool rows_ok(const void* x, int64_t stride, int64_t row_elems, int64_t multiple) {
  return x && aligned(x, 16) && stride >= row_elems && stride % multiple == 0;
}

}  // namespace

sps_status sps_qk_norm_rope(const sps_plan* pl, const void* q, int64_t q_stride, const void* k,
                            int64_t k_stride, const float* q_weight, const float* k_weight,
                            float eps, const sps_rope* rope, void* q_out, int64_t q_out_stride,
                            sps_dtype q_out_dtype, float q_scale, void* k_out,
                            int64_t k_out_stride, void* ws, sps_stream_t stream) {
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  const sps_problem& p = pl->pb;
  const bool e4m3 = q_out_dtype == SPS_E4M3;
  if (!e4m3 && q_out_dtype != SPS_BF16)
    return fail(SPS_EUNSUPPORTED, "sps_qk_norm_rope: q_out must be BF16 or E4M3");
  if (!k != !k_out) return fail(SPS_EINVAL, "sps_qk_norm_rope: k and k_out go together");
  const int64_t qn = (int64_t)p.num_q_heads * p.head_dim, kn = (int64_t)p.num_kv_heads * p.head_dim;
  if (!rows_ok(q, q_stride, qn, 8) || !rows_ok(q_out, q_out_stride, qn, e4m3 ? 16 : 8) ||
      (k && (!rows_ok(k, k_stride, kn, 8) || !rows_ok(k_out, k_out_stride, kn, 8))))
    return fail(SPS_EINVAL,
                "sps_qk_norm_rope: buffers must be non-NULL and 16-byte aligned, token strides "
                "multiples of 16 bytes and at least a token's rows");
  // in place, each row lies on itself; else a warp's rows would lie on rows that others still read
  if ((q_out == q && (e4m3 || q_out_stride != q_stride)) ||
      (k && k_out == k && k_out_stride != k_stride))
    return fail(SPS_EINVAL, "sps_qk_norm_rope: an output in place is BF16 and has the input's stride");
  if ((q_weight && !aligned(q_weight, 16)) || (k_weight && !aligned(k_weight, 16)))
    return fail(SPS_EINVAL, "sps_qk_norm_rope: weights must be 16-byte aligned");
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return fail(SPS_EINVAL, "sps_qk_norm_rope: eps must be finite and >= 0");
  if (e4m3 && (!(q_scale > 0.f) || !std::isfinite(q_scale) || !std::isfinite(1.f / q_scale)))
    return fail(SPS_EINVAL, "sps_qk_norm_rope: q_scale and its inverse must be finite and > 0");
  DevRope r;
  st = make_rope(rope, p.head_dim, "sps_qk_norm_rope", &r);
  if (st != SPS_OK) return st;
  QkRopeArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.q_out = q_out;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.eps = eps;
  a.q_scale = make_quot(q_scale);
  return launched(launch_qk_norm_rope(make_dev_plan(pl, ws), r, a, rope && rope->interleaved, e4m3,
                                      reinterpret_cast<cudaStream_t>(stream)),
                  "q/k norm and rotation launch");
}

sps_status sps_kv_append_rope(const sps_plan* pl, const void* k_new, int64_t k_stride,
                              const void* v_new, int64_t v_stride, const float* k_weight,
                              float eps, const sps_rope* rope, const int32_t* page_table,
                              void* k_cache, void* v_cache, void* k_scales, void* v_scales,
                              void* ws, sps_stream_t stream) {
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  const sps_problem& p = pl->pb;
  const bool nvfp4 = p.kv_dtype == SPS_NVFP4;
  if (p.kv_dtype != SPS_BF16 && !nvfp4)
    return fail(SPS_EUNSUPPORTED, "sps_kv_append_rope: the cache must be BF16 or NVFP4");
  if (!page_table || !k_cache || !v_cache || (nvfp4 && (!k_scales || !v_scales)))
    return fail(SPS_EINVAL, "sps_kv_append_rope: NULL pointer (an NVFP4 cache needs its scales)");
  const int64_t kn = (int64_t)p.num_kv_heads * p.head_dim;
  if (!rows_ok(k_new, k_stride, kn, 8) || !rows_ok(v_new, v_stride, kn, 8))
    return fail(SPS_EINVAL,
                "sps_kv_append_rope: k_new/v_new must be non-NULL and 16-byte aligned, token "
                "strides multiples of 8 and at least num_kv_heads * head_dim");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(page_table, 4) ||
      (k_weight && !aligned(k_weight, 16)))
    return fail(SPS_EINVAL, "sps_kv_append_rope: misaligned cache, page table or weight");
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return fail(SPS_EINVAL, "sps_kv_append_rope: eps must be finite and >= 0");
  DevRope r;
  st = make_rope(rope, p.head_dim, "sps_kv_append_rope", &r);
  if (st != SPS_OK) return st;
  KvRopeArgs a{};
  a.k = static_cast<const uint16_t*>(k_new);
  a.v = static_cast<const uint16_t*>(v_new);
  a.k_weight = k_weight;
  a.page_table = page_table;
  a.kc = static_cast<uint8_t*>(k_cache);
  a.vc = static_cast<uint8_t*>(v_cache);
  a.ks = static_cast<uint8_t*>(k_scales);
  a.vs = static_cast<uint8_t*>(v_scales);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.eps = eps;
  return launched(launch_kv_append_rope(make_dev_plan(pl, ws), r, a, rope && rope->interleaved,
                                        nvfp4, reinterpret_cast<cudaStream_t>(stream)),
                  "kv append with rotation launch");
}

sps_status paged_attention_scratch(const sps_plan* pl, size_t* bytes) {
  if (!pl || !bytes) return fail(SPS_EINVAL, "paged_attention_scratch: plan/scratch_bytes NULL");
  *bytes = (size_t)align_up(2ll * pl->att_ctas * pl->att_slot_rows * (pl->pb.head_dim + 1) * 4, 256);
  return SPS_OK;
}

sps_status paged_attention_fwd(const sps_plan* pl, const void* q, int64_t q_stride, float q_scale,
                               const void* k_cache, const void* v_cache, const void* k_scales,
                               const void* v_scales, const int32_t* page_table, void* out_bf16,
                               int64_t out_stride, float* out_lse, void* scratch,
                               size_t scratch_bytes, void* ws, sps_stream_t stream) {
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  const sps_problem& p = pl->pb;
  const bool quant = p.kv_dtype == SPS_NVFP4;
  const int64_t n = (int64_t)p.num_q_heads * p.head_dim;
  if (!rows_ok(q, q_stride, n, quant ? 16 : 8) || !rows_ok(out_bf16, out_stride, n, 8))
    return fail(SPS_EINVAL,
                "paged_attention_fwd: q and out must be non-NULL and 16-byte aligned, token "
                "strides multiples of 16 bytes and at least num_q_heads * head_dim");
  if (!k_cache || !v_cache || !page_table || (quant && (!k_scales || !v_scales)))
    return fail(SPS_EINVAL, "paged_attention_fwd: NULL pointer (an NVFP4 cache needs its scales)");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || (quant && (!aligned(k_scales, 16) ||
      !aligned(v_scales, 16))) || !aligned(page_table, 4) || (out_lse && !aligned(out_lse, 4)))
    return fail(SPS_EINVAL, "paged_attention_fwd: caches must be 16-byte, page_table and out_lse "
                            "4-byte aligned");
  if (!(q_scale > 0.f) || !std::isfinite(q_scale))
    return fail(SPS_EINVAL, "paged_attention_fwd: q_scale must be finite and > 0");
  const float c = attention_factor(p.softmax_scale, q_scale);
  if (!(c > 0.f) || !std::isfinite(c))
    return fail(SPS_EINVAL, "paged_attention_fwd: softmax_scale x q_scale must stay within FP32");
  size_t need = 0;
  paged_attention_scratch(pl, &need);
  if (!scratch || !aligned(scratch, 256))
    return fail(SPS_EINVAL, "paged_attention_fwd: scratch must be non-NULL and 256-byte aligned");
  if (scratch_bytes < need)
    return fail(SPS_ENOSPACE, "paged_attention_fwd: scratch of %zu bytes < %zu required",
                scratch_bytes, need);
  if ((int64_t)p.num_phys_pages * p.num_kv_heads > 0x7fffffff / kPage)
    return fail(SPS_EUNSUPPORTED, "paged_attention_fwd: num_phys_pages x num_kv_heads must stay "
                                  "below 2^24");
  return launched(launch_attention(make_dev_plan(pl, ws), quant, q, q_stride, q_scale, k_cache,
                                   v_cache, k_scales, v_scales, page_table, out_bf16, out_stride,
                                   out_lse, scratch, reinterpret_cast<cudaStream_t>(stream)),
                  "paged attention launch");
}

sps_status sps_quantize_e4m3(const void* x_bf16, int64_t n, float scale, void* codes,
                             sps_stream_t stream) {
  if (n < 0 || n % 16) return fail(SPS_EINVAL, "sps_quantize_e4m3: n must be a multiple of 16");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return fail(SPS_EINVAL, "sps_quantize_e4m3: scale must be finite and > 0");
  if (n == 0) return SPS_OK;
  if (!x_bf16 || !codes || !aligned(x_bf16, 16) || !aligned(codes, 16))
    return fail(SPS_EINVAL, "sps_quantize_e4m3: buffers must be non-NULL and 16-byte aligned");
  return launched(launch_quantize_e4m3(x_bf16, n, scale, codes,
                                       reinterpret_cast<cudaStream_t>(stream)),
                  "quantize launch");
}

sps_status sps_absmax_bf16(const void* x_bf16, int64_t n, float* absmax, sps_stream_t stream) {
  if (n < 0 || n % 16) return fail(SPS_EINVAL, "sps_absmax_bf16: n must be a multiple of 16");
  if (!absmax || !aligned(absmax, 4)) return fail(SPS_EINVAL, "sps_absmax_bf16: bad output");
  if (n > 0 && (!x_bf16 || !aligned(x_bf16, 16)))
    return fail(SPS_EINVAL, "sps_absmax_bf16: input must be non-NULL and 16-byte aligned");
  return launched(launch_absmax_bf16(x_bf16, n, absmax, reinterpret_cast<cudaStream_t>(stream)),
                  "absmax launch");
}

sps_status sps_dequantize(sps_dtype in_dtype, const void* in, const void* scales, int64_t n,
                          void* out_f16, sps_stream_t stream) {
  if (in_dtype != SPS_E4M3 && in_dtype != SPS_NVFP4)
    return fail(SPS_EUNSUPPORTED, "sps_dequantize: input must be E4M3 or NVFP4");
  if (n < 0 || n % 16) return fail(SPS_EINVAL, "sps_dequantize: n must be a multiple of 16");
  if (n == 0) return SPS_OK;
  if (!in || !out_f16 || (in_dtype == SPS_NVFP4 && !scales))
    return fail(SPS_EINVAL, "sps_dequantize: NULL pointer");
  if (!aligned(in, in_dtype == SPS_E4M3 ? 16 : 8) || !aligned(out_f16, 16))
    return fail(SPS_EINVAL, "sps_dequantize: input must be %d-byte and output 16-byte aligned",
                in_dtype == SPS_E4M3 ? 16 : 8);
  return launched(launch_dequant(in_dtype, in, scales, n, out_f16,
                                 reinterpret_cast<cudaStream_t>(stream)),
                  "dequant launch");
}

sps_status sps_check_wait_timeout(int64_t limit_ns, int32_t* dev_status, sps_stream_t stream) {
  if (!dev_status || !aligned(dev_status, 4))
    return fail(SPS_EINVAL, "sps_check_wait_timeout: dev_status must be a device int32");
  if (limit_ns < 1000000 || limit_ns > 10000000000LL)
    return fail(SPS_EINVAL, "sps_check_wait_timeout: limit_ns must be in [1e6, 1e10]");
  return launched(launch_wait_timeout(dev_status, limit_ns, reinterpret_cast<cudaStream_t>(stream)),
                  "wait-timeout check launch");
}

sps_status sps_check_barrier_timeout(int64_t limit_ns, uint32_t* dev_barrier,
                                     int32_t* dev_status, sps_stream_t stream) {
  if (!dev_status || !aligned(dev_status, 4) || !dev_barrier || !aligned(dev_barrier, 4))
    return fail(SPS_EINVAL, "sps_check_barrier_timeout: dev_barrier/dev_status must be device words");
  if (limit_ns < 1000000 || limit_ns > 10000000000LL)
    return fail(SPS_EINVAL, "sps_check_barrier_timeout: limit_ns must be in [1e6, 1e10]");
  return launched(launch_barrier_timeout(dev_barrier, dev_status, limit_ns,
                                         reinterpret_cast<cudaStream_t>(stream)),
                  "barrier timeout check launch");
}

sps_status sps_read_device_status(const sps_plan* pl, const void* ws, int32_t* code) {
  if (!code) return fail(SPS_EINVAL, "code is NULL");
  sps_status st = check_plan_ws(pl, ws);
  if (st != SPS_OK) return st;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  e = cudaMemcpy(code, static_cast<const uint8_t*>(ws) + pl->off_status, 4,
                 cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(status)");
  if (*code != 0) return fail(SPS_EDEVICE, "device status %d", *code);
  return SPS_OK;
}

}  // extern "C"

// ------------------------------------------------------------------ driver helpers
namespace sps {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
void load_encode() {
  cudaDriverEntryPointQueryResult q;
  void* fn = nullptr;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}
CUtensorMapDataType tm_type(int code) {
  switch (code) {
    case 0: return CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    case 1: return CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    default: return CU_TENSOR_MAP_DATA_TYPE_UINT8;
  }
}
int tm_size(int code) { return code <= 1 ? 2 : 1; }
}  // namespace

bool encode_tmap_2d(void* map, int dtype_code, void* base, uint64_t inner, uint64_t outer,
                    uint64_t outer_stride_bytes, uint32_t box_inner, uint32_t box_outer,
                    bool swizzle128) {
  std::call_once(g_encode_once, load_encode);
  if (!g_encode) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {outer_stride_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t es[2] = {1, 1};
  (void)tm_size;
  return g_encode(reinterpret_cast<CUtensorMap*>(map), tm_type(dtype_code), 2, base, dims,
                  strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tmap_3d(void* map, int dtype_code, void* base, uint64_t d0, uint64_t d1,
                    uint64_t d2, uint64_t s1_bytes, uint64_t s2_bytes, uint32_t b0, uint32_t b1,
                    uint32_t b2, bool swizzle128) {
  std::call_once(g_encode_once, load_encode);
  if (!g_encode) return false;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {s1_bytes, s2_bytes};
  cuuint32_t box[3] = {b0, b1, b2};
  cuuint32_t es[3] = {1, 1, 1};
  return g_encode(reinterpret_cast<CUtensorMap*>(map), tm_type(dtype_code), 3, base, dims,
                  strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tmap_2d_f32_sw64(void* map, const void* base, uint64_t inner, uint64_t outer,
                             uint64_t outer_stride_bytes, uint32_t box_inner,
                             uint32_t box_outer) {
  std::call_once(g_encode_once, load_encode);
  if (!g_encode) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {outer_stride_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t es[2] = {1, 1};
  return g_encode(reinterpret_cast<CUtensorMap*>(map), CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int num_sms() {
  static int n = -1;
  if (n < 0) {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
      n = v;
    else
      n = 152;  // planning without a device: the GB300 SM count
  }
  return n;
}

}  // namespace sps

// ------------------------------------------------------------------ scratch-array forward
// Used by sparse_prefill_fwd_noalloc (noalloc.cu), which owns the scratch array: the same
// checks and launches as sparse_prefill_fwd, with the plan's metadata copied into the given
// scratch area first (the caller has no workspace to upload into).
sps_status sps_internal_cuda_fail(cudaError_t e, const char* what) { return cuda_fail(e, what); }

sps_status sps_internal_fwd_noalloc(const sps_plan* pl, const void* q, float q_scale,
                                    const void* k_cache, const void* v_cache, const void* k_scales,
                                    const void* v_scales, const int32_t* page_table,
                                    const int32_t* idx, float* partial, int64_t split_stride,
                                    float* lse, int64_t lse_split_stride, void* scratch,
                                    size_t scratch_bytes, int32_t* dev_status,
                                    sps_stream_t stream) {
  if (!pl) return fail(SPS_EINVAL, "plan is NULL");
  const sps_problem& p = pl->pb;
  if (!q || !k_cache || !v_cache || !page_table || !idx || !partial || !lse)
    return fail(SPS_EINVAL, "sparse_prefill_fwd_noalloc: NULL input/output pointer");
  if (p.kv_dtype == SPS_NVFP4 && (!k_scales || !v_scales))
    return fail(SPS_EINVAL, "sparse_prefill_fwd_noalloc: NVFP4 K/V need k_scales and v_scales");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      (k_scales && !aligned(k_scales, 16)) || (v_scales && !aligned(v_scales, 16)))
    return fail(SPS_EINVAL, "sparse_prefill_fwd_noalloc: q/k/v buffers must be 16-byte aligned");
  if (!aligned(partial, 16)) return fail(SPS_EINVAL, "partial must be 16-byte aligned");
  if (split_stride < pl->R * p.head_dim || split_stride % 4)
    return fail(SPS_EINVAL, "split_stride must be >= rows*head_dim and a multiple of 4");
  if (lse_split_stride < pl->R) return fail(SPS_EINVAL, "lse_split_stride must be >= rows");
  if (!std::isfinite(q_scale)) return fail(SPS_EINVAL, "q_scale must be finite");
  if (dev_status && !aligned(dev_status, 4)) return fail(SPS_EINVAL, "dev_status misaligned");
  if ((int64_t)scratch_bytes < pl->fwd_ws_bytes)
    return fail(SPS_ENOSPACE,
                "sparse_prefill_fwd_noalloc: this batch needs %lld bytes of scratch, the built-in "
                "array holds %zu; split the batch or use sparse_prefill_fwd with a workspace",
                (long long)pl->fwd_ws_bytes, scratch_bytes);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // the array keeps the previous call's contents: one copy zeroes the status word and
  // counters and writes this plan's metadata over the old one
  cudaError_t e = g_staging.upload(scratch, pl->blob.data() + pl->fwd_base,
                                   pl->upload_bytes - pl->fwd_base, s, false);
  if (e != cudaSuccess) return cuda_fail(e, "plan metadata -> scratch");
  // (offsets count from the workspace's start, fwd_base bytes in front of the array)
  DevPlan d = make_dev_plan(pl, reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(scratch) -
                                                        (uintptr_t)pl->fwd_base));
  if (dev_status) d.status = dev_status;
  e = launch_inversion(d, idx, lse, lse_split_stride, s);
  if (e != cudaSuccess) return cuda_fail(e, "inversion launch");
  return launched(launch_forward(d, p.q_dtype, p.kv_dtype, q, q_scale, k_cache, v_cache,
                                 k_scales, v_scales, page_table, partial, split_stride, lse,
                                 lse_split_stride, s),
                  "forward launch");
}

// The full attention's tables as they are uploaded, for the tests of the work split: their start, and
// in `info` the offsets of heads, pieces, merges and of what follows them, the blocks, the rows of a
// slot, the cut tiles and their cap.
extern "C" const uint8_t* sps_internal_attention_tables(const sps_plan* pl, int64_t* info) {
  const int64_t v[8] = {pl->off_att_heads, pl->off_att_pieces,    pl->off_att_merges,
                        pl->fwd_base,      pl->att_ctas,          pl->att_slot_rows,
                        pl->att_num_merges, pl->att_merge_cap};
  memcpy(info, v, sizeof v);
  return pl->blob.data();
}
