// pagetable.cu -- page tables and slot maps from request lengths on the device (sps_page_tables).
//
// Request b holds pages for its ctx tokens; its q new ones need ceil((ctx + q) / 128) - ceil(ctx / 128)
// more, taken from the list of free pages in request order.  With the running sums of q and of the pages
// taken, every table entry, slot and position follows by itself.
//
// One launch: each block makes both running sums of the whole batch in shared memory (a few requests a
// thread) and finds a token's request in them by bisection; so no block waits for another.  The list's
// counter is read by every block and advanced by the last one to have read it, which a ticket beside it
// shows; results do not depend on the order.
//
// It writes 12 bytes for each of max_tokens and reads 8 bytes for each request in every block.  At the sizes
// of a step that is little (64 single tokens 4 KB, 64K tokens of 256 requests 0.8 MB), so it is bound by one
// pass of latency: the counter, the lengths, two scans, the bisections (8 steps for 256 requests).  64
// requests of one token take 2.8 us on the GPU, 256 requests of 64K tokens together 4.5 us.  A launch for
// the sums and one for the maps would take two such passes.  A thread's lengths lie in a row, so a large
// batch costs each block strided reads: 1000 requests of one token 4.0 us, 4096 10.4, 16384 53.
#include <algorithm>

#include "ptx.cuh"
#include "sps_internal.h"

namespace sps {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }

// The last entry of the ascending a[0 .. n] that is <= x (a[0] = 0 <= x < a[n]).
__device__ __forceinline__ int find(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_tables_kernel(PageTableArgs a) {
  extern __shared__ int32_t sums[];  // tokens before each request, then pages taken before it
  int32_t *tok = sums, *take = sums + a.batch + 1;
  __shared__ long long part[2][kThreads / 32];
  __shared__ int head, bad;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    bad = 0;
    head = *(volatile int32_t*)a.free_state;
    // every block has read the counter before the last one moves it on
    __threadfence();
    if (atomicAdd(a.free_state + 1, 1) != (int)gridDim.x - 1) bad = -1;
  }
  __syncthreads();
  const bool last = bad == 0;
  __syncthreads();
  if (tid == 0) bad = 0;
  // this thread's requests in a row, and their sums
  const int per = (a.batch + kThreads - 1) / kThreads, b0 = min(a.batch, tid * per),
            b1 = min(a.batch, b0 + per);
  const int64_t room = (int64_t)a.max_pages * kPage;
  long long q_sum = 0, t_sum = 0;
  bool wrong = false;
  for (int b = b0; b < b1; ++b) {
    const int q = __ldg(a.q_lens + b), c = __ldg(a.ctx_lens + b);
    if (q < 0 || c < 0 || (int64_t)q + c > room) {
      wrong = true;
      continue;
    }
    q_sum += q;
    t_sum += pages_of(q + c) - pages_of(c);
  }
  long long q_at = q_sum, t_at = t_sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, q_at, o), y = __shfl_up_sync(0xffffffffu, t_at, o);
    if (lane >= o) {
      q_at += x;
      t_at += y;
    }
  }
  if (lane == 31) {
    part[0][warp] = q_at;
    part[1][warp] = t_at;
  }
  __syncthreads();
  if (wrong) bad = DEV_BAD_LENGTH;
  long long q_all = 0, t_all = 0;
  q_at -= q_sum;
  t_at -= t_sum;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      q_at += part[0][w];
      t_at += part[1][w];
    }
    q_all += part[0][w];
    t_all += part[1][w];
  }
  __syncthreads();
  int code = bad;
  if (!code && q_all > (a.slots || a.positions ? a.max_tokens : 0x7fffffffLL)) code = DEV_BAD_LENGTH;
  if (!code && (head < 0 || head + t_all > a.num_free)) code = DEV_NO_PAGES;
  const int64_t first = (int64_t)blockIdx.x * kThreads + tid, step = (int64_t)gridDim.x * kThreads;
  if (code) {  // nothing is taken
    if (tid == 0 && last) {
      set_status(a.status, code);
      a.free_state[1] = 0;
    }
    for (int64_t t = first; (a.slots || a.positions) && t < a.max_tokens; t += step) {
      if (a.slots) a.slots[t] = -1;
      if (a.positions) a.positions[t] = 0;
    }
    for (int64_t b = first; a.starts && b <= a.batch; b += step) a.starts[b] = 0;
    return;
  }
  for (int b = b0; b < b1; ++b) {
    const int q = __ldg(a.q_lens + b), c = __ldg(a.ctx_lens + b);
    tok[b] = (int)q_at;
    take[b] = (int)t_at;
    q_at += q;
    t_at += pages_of(q + c) - pages_of(c);
  }
  const int T = (int)q_all, taken = (int)t_all;
  if (tid == 0) {
    tok[a.batch] = T;
    take[a.batch] = taken;
    if (last) {
      a.free_state[0] = head + taken;
      a.free_state[1] = 0;
    }
  }
  __syncthreads();
  for (int64_t b = first; a.starts && b <= a.batch; b += step) a.starts[b] = tok[b];
  const int32_t* list = a.free_pages + head;
  for (int64_t i = first; i < taken; i += step) {
    const int b = find(take, a.batch, (int)i);
    a.page_table[(int64_t)b * a.max_pages + pages_of(__ldg(a.ctx_lens + b)) + (int)i - take[b]] =
        __ldg(list + i);
  }
  if (!a.slots && !a.positions) return;
  for (int64_t t = first; t < a.max_tokens; t += step) {
    int64_t slot = -1;
    int pos = 0;
    if (t < T) {
      const int b = find(tok, a.batch, (int)t), c = __ldg(a.ctx_lens + b);
      pos = c + (int)t - tok[b];
      const int page = pos / kPage, have = pages_of(c);
      // (a page that the request held, or one that this call takes: no read of another thread's write)
      const int phys = page < have ? a.page_table[(int64_t)b * a.max_pages + page]
                                   : __ldg(list + take[b] + page - have);
      if (phys >= 0) slot = (int64_t)phys * kPage + pos % kPage;
    }
    if (a.slots) a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
}

}  // namespace

cudaError_t launch_page_tables(const PageTableArgs& a, cudaStream_t st) {
  const size_t smem = 8 * ((size_t)a.batch + 1);
  if (smem > 32 * 1024) {  // (48 KB without asking, less what the kernel declares itself)
    cudaError_t e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         8 * (kMaxTableBatch + 1));
    if (e != cudaSuccess) return e;
  }
  const int64_t work = std::max<int64_t>(a.max_tokens, a.batch);
  const unsigned grid = (unsigned)std::min<int64_t>((work + kThreads - 1) / kThreads, num_sms());
  cudaError_t e = launch_pdl(page_tables_kernel, dim3(std::max(1u, grid)), dim3(kThreads), smem, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sps
