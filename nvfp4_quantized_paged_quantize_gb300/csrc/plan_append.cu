// plan_append.cu -- where a step's new tokens go: page-table entries off a stack
// of free pages, cache slots, positions and workspace rows, from the requests'
// lengths (nvfp4kv_plan_append), so that a captured step needs no host in it.
//
// Request b has c_b cached tokens and n_b new ones; it needs
// ceil((c_b + n_b) / 16) - ceil(c_b / 16) more pages.  Three prefix sums over the
// requests (pages, tokens, workspace rows) place everything else: token i of
// request b is new token sum(n before b) + i, at position c_b + i, and the k-th
// page needed is the k-th from the top of the stack.
//
// Every CTA does the sums for itself (batch is small beside the tokens), the first one
// writes what there is per request, and the tokens are spread over all threads, each
// finding its request by bisection of the token sums in shared memory.  Where the
// lengths or the free count are updated in place, the CTAs are one cluster, with a
// barrier between reading and writing them.
// Bound by latency: a launch, the loads of the lengths, the sums, and for each token
// two dependent loads and its stores.  256 requests of one token each 3.1 us, 16 of
// 820 to 2048 2.9, in a captured graph (one block of 1024 threads with 64-bit sums:
// 6.9 and, in a cluster of eight, 8.9: the instructions of its SM).
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kPlanMaxCluster = 8;  // the portable limit

template <int kThreads>
struct PlanShared {
  int32_t cached[kThreads];  // c_b
  int32_t token[kThreads];   // new tokens before request b
  int32_t page[kThreads];    // new pages before request b
  long long row[kThreads];   // workspace rows before request b
  uint32_t sum_pages[32], sum_tokens[32];  // of the warps
  long long sum_cached[32];
  uint32_t total_tokens, total_pages;  // of the requests served
};

// Sums of pages and tokens stop at 2^31 - 1, more than any limit (checked on the host):
// what follows a request that does not fit is of no account.
constexpr uint32_t kEnough = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t add_up(uint32_t a, uint32_t b) { return min(a + b, kEnough); }

// kThreads requests per round.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs p, int ctas, bool in_place) {
  __shared__ PlanShared<kThreads> s;
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x;
  after_earlier_kernels();
  int free_count = *p.free_count;
  if (free_count < 0 || free_count > p.free_capacity) {
    if (rank == 0 && tid == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    free_count = free_count < 0 ? 0 : p.free_capacity;
  }
  const int room = p.max_pages * kPage;
  uint32_t pages0 = 0, tokens0 = 0;  // of the requests of earlier rounds
  long long cached0 = 0;
  int placed = 0, used = 0;          // tokens and pages of the requests served so far
  if (rank == 0 && tid == 0) {
    if (p.cu_q) p.cu_q[0] = 0;
    if (p.cu_prefix) p.cu_prefix[0] = 0;
  }
  for (int base = 0; base < p.batch; base += kThreads) {
    const int b = base + tid;
    const bool real = b < p.batch;
    int cached = 0, fresh = 0;
    if (real) {
      cached = p.cached_lens[b];
      fresh = p.new_lens[b];
      const bool bad = cached < 0 || cached > room || fresh < 0 || fresh > room - min(max(cached, 0), room);
      if (bad && rank == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
      cached = min(max(cached, 0), room);
      fresh = min(max(fresh, 0), room - cached);
    }
    const int have = (cached + kPage - 1) / kPage, need = (cached + fresh + kPage - 1) / kPage - have;
    uint32_t pages = (uint32_t)need, tokens = (uint32_t)fresh;
    long long sum = cached;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t up_pages = __shfl_up_sync(0xFFFFFFFFu, pages, off), up_tokens = __shfl_up_sync(0xFFFFFFFFu, tokens, off);
      const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, off);
      if (lane >= off) {
        pages = add_up(pages, up_pages);
        tokens = add_up(tokens, up_tokens);
        sum += up;
      }
    }
    if (lane == 31) {
      s.sum_pages[warp] = pages;
      s.sum_tokens[warp] = tokens;
      s.sum_cached[warp] = sum;
    }
    if (tid == 0) {
      s.total_tokens = placed;
      s.total_pages = used;
    }
    __syncthreads();
    // lane = warp: the sums up to each warp, the last one's the round's
    uint32_t all_pages = lane < kWarps ? s.sum_pages[lane] : 0, all_tokens = lane < kWarps ? s.sum_tokens[lane] : 0;
    long long all_cached = lane < kWarps ? s.sum_cached[lane] : 0;
    if (lane == 0) {
      all_pages = add_up(all_pages, pages0);
      all_tokens = add_up(all_tokens, tokens0);
      all_cached += cached0;
    }
#pragma unroll
    for (int off = 1; off < kWarps; off <<= 1) {
      const uint32_t up_pages = __shfl_up_sync(0xFFFFFFFFu, all_pages, off), up_tokens = __shfl_up_sync(0xFFFFFFFFu, all_tokens, off);
      const long long up = __shfl_up_sync(0xFFFFFFFFu, all_cached, off);
      if (lane >= off) {
        all_pages = add_up(all_pages, up_pages);
        all_tokens = add_up(all_tokens, up_tokens);
        all_cached += up;
      }
    }
    const int last = warp > 0 ? warp - 1 : 0;
    const uint32_t warp_pages = __shfl_sync(0xFFFFFFFFu, all_pages, last), warp_tokens = __shfl_sync(0xFFFFFFFFu, all_tokens, last);
    const long long warp_cached = __shfl_sync(0xFFFFFFFFu, all_cached, last);
    const uint32_t pages_to = add_up(warp > 0 ? warp_pages : pages0, pages);
    const uint32_t tokens_to = add_up(warp > 0 ? warp_tokens : tokens0, tokens);
    const long long cached_to = (warp > 0 ? warp_cached : cached0) + sum;
    pages0 = __shfl_sync(0xFFFFFFFFu, all_pages, kWarps - 1);
    tokens0 = __shfl_sync(0xFFFFFFFFu, all_tokens, kWarps - 1);
    cached0 = __shfl_sync(0xFFFFFFFFu, all_cached, kWarps - 1);
    // requests are served in order until one does not fit; the sums only grow
    const bool served = real && pages_to <= (uint32_t)free_count && tokens_to <= (uint32_t)p.max_tokens;
    if (!served && real && fresh > 0 && rank == 0) flag_error(p.status, NVFP4KV_DEVERR_POOL);
    const uint32_t most_tokens = __reduce_max_sync(0xFFFFFFFFu, served ? tokens_to : 0u);
    const uint32_t most_pages = __reduce_max_sync(0xFFFFFFFFu, served ? pages_to : 0u);
    if (lane == 0) {
      atomicMax(&s.total_tokens, most_tokens);
      atomicMax(&s.total_pages, most_pages);
    }
    __syncthreads();
    const int first = placed;
    placed = (int)s.total_tokens;
    used = (int)s.total_pages;
    const int tokens_before = served ? (int)tokens_to - fresh : placed;
    s.cached[tid] = cached;
    s.token[tid] = real ? tokens_before : placed;
    s.page[tid] = served ? (int)pages_to - need : used;
    s.row[tid] = cached_to - cached + tokens_before;
    __syncthreads();
    if (in_place && ctas > 1) cluster_sync();  // every CTA has read the lengths and the count
    if (rank == 0 && real) {
      const int now = served ? fresh : 0;
      p.seq_lens[b] = cached + now;
      if (p.cu_q) p.cu_q[b + 1] = tokens_before + now;
      if (p.cu_prefix) p.cu_prefix[b + 1] = cached_to + tokens_before + now;
    }
    const int rows = min(kThreads, p.batch - base);
    for (int t = first + rank * kThreads + tid; t < placed; t += ctas * kThreads) {
      // the token's request: the last one with token[] <= t
      int lo = 0, hi = rows;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.token[mid] <= t) lo = mid; else hi = mid;
      }
      const int have_t = (s.cached[lo] + kPage - 1) / kPage;
      const int pos = s.cached[lo] + (t - s.token[lo]), page = pos / kPage;
      int32_t* const entry = p.page_table + (long long)(base + lo) * p.max_pages + page;
      int id;
      if (page >= have_t) {
        id = p.free_pages[free_count - 1 - (s.page[lo] + page - have_t)];
        if (pos % kPage == 0) *entry = id;  // a new page's first token is always among the new ones
      } else {
        id = *entry;
      }
      const bool valid = id >= 0 && id < p.num_pages;
      if (!valid) flag_error(p.status, NVFP4KV_DEVERR_PAGE);
      p.slot_mapping[t] = valid ? (long long)id * kPage + pos % kPage : -1;
      if (p.positions) p.positions[t] = pos;
      if (p.ws_rows) p.ws_rows[t] = s.row[lo] + pos;
    }
    __syncthreads();
  }
  // what is left of the arrays: tokens that the append skips
  for (long long t = placed + (long long)rank * kThreads + tid; t < p.max_tokens; t += (long long)ctas * kThreads) {
    p.slot_mapping[t] = -1;
    if (p.positions) p.positions[t] = 0;
    if (p.ws_rows) p.ws_rows[t] = -1;
  }
  if (rank == 0 && tid == 0) *p.free_left = free_count - used;
}

}  // namespace

cudaError_t launch_plan_append(const PlanArgs& args, cudaStream_t stream) {
  // few requests: small blocks, whose barriers cost less (256 requests of one token 3.1 us, with
  // 1024 threads 3.6, 16 of up to 2048 2.9 and 3.8; but 300, two rounds of small blocks, 4.8 and 3.9)
  const bool small = args.batch <= 256;
  const int threads = small ? 256 : 1024;
  const bool in_place = args.seq_lens == args.cached_lens || args.free_left == args.free_count;
  // (16 requests of up to 2048 tokens over 128 blocks 2.9 us, over 8 8.9)
  const int64_t want = (args.max_tokens + threads - 1) / threads, most = in_place ? kPlanMaxCluster : 128;
  const int ctas = (int)(want < 1 ? 1 : want < most ? want : most);
  return launch_overlapped(small ? plan_kernel<256> : plan_kernel<1024>, ctas, threads, 0, in_place ? ctas : 1, stream,
                           args, ctas, in_place);
}

}  // namespace nvfp4kv
