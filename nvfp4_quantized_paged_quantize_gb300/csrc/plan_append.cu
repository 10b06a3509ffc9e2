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
// One cluster.  Every CTA does the sums for itself (batch is small beside the
// tokens), the first one writes what there is per request, and the tokens are
// spread over all threads, each finding its request by bisection of the token
// sums in shared memory.  A cluster barrier between reading the lengths and
// writing the new ones lets them be the same memory, and the free count too.
// Bound by latency: a launch, the loads of the lengths, the sums, and for each
// token one dependent load and its stores.
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMaxCluster = 8;  // the portable limit

struct PlanShared {
  int32_t cached[kPlanThreads];   // c_b
  int32_t token[kPlanThreads];    // new tokens before request b
  int32_t page[kPlanThreads];     // new pages before request b
  long long row[kPlanThreads];    // workspace rows before request b
  long long sums[kPlanWarps][3];
  int32_t total_tokens, total_pages;  // of the requests served
};

__device__ __forceinline__ long long shfl_up_ll(long long v, int by) { return __shfl_up_sync(0xFFFFFFFFu, v, by); }

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs p, int ctas) {
  __shared__ PlanShared s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x;  // one cluster is the whole grid
  int free_count = *p.free_count;
  if (free_count < 0 || free_count > p.free_capacity) {
    if (rank == 0 && tid == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    free_count = free_count < 0 ? 0 : p.free_capacity;
  }
  const int room = p.max_pages * kPage;
  long long pages0 = 0, tokens0 = 0, cached0 = 0;  // of the requests of earlier rounds
  int placed = 0, used = 0;                        // tokens and pages of the requests served so far
  if (rank == 0 && tid == 0) {
    if (p.cu_q) p.cu_q[0] = 0;
    if (p.cu_prefix) p.cu_prefix[0] = 0;
  }
  for (int base = 0; base < p.batch; base += kPlanThreads) {
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
    long long v[3] = {need, fresh, cached};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const long long up = shfl_up_ll(v[k], off);
        if (lane >= off) v[k] += up;
      }
    }
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < 3; ++k) s.sums[warp][k] = v[k];
    }
    if (tid == 0) {
      s.total_tokens = placed;
      s.total_pages = used;
    }
    __syncthreads();
    long long before[3] = {pages0, tokens0, cached0}, all[3] = {pages0, tokens0, cached0};
    for (int w = 0; w < kPlanWarps; ++w) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const long long n = s.sums[w][k];
        if (w < warp) before[k] += n;
        all[k] += n;
      }
    }
    pages0 = all[0], tokens0 = all[1], cached0 = all[2];
    const long long pages_to = before[0] + v[0], tokens_to = before[1] + v[1], cached_to = before[2] + v[2];
    // requests are served in order until one does not fit; the sums only grow
    const bool served = real && pages_to <= free_count && tokens_to <= p.max_tokens;
    if (served) {
      atomicMax(&s.total_tokens, (int)tokens_to);
      atomicMax(&s.total_pages, (int)pages_to);
    } else if (real && fresh > 0 && rank == 0) {
      flag_error(p.status, NVFP4KV_DEVERR_POOL);
    }
    __syncthreads();
    const int first = placed;
    placed = s.total_tokens;
    used = s.total_pages;
    const int tokens_before = served ? (int)tokens_to - fresh : placed;
    s.cached[tid] = cached;
    s.token[tid] = real ? tokens_before : placed;
    s.page[tid] = served ? (int)pages_to - need : used;
    s.row[tid] = cached_to - cached + tokens_before;
    __syncthreads();
    if (ctas > 1) cluster_sync();  // every CTA has read the lengths: seq_lens may be cached_lens
    if (rank == 0 && real) {
      const int now = served ? fresh : 0;
      p.seq_lens[b] = cached + now;
      if (p.cu_q) p.cu_q[b + 1] = tokens_before + now;
      if (p.cu_prefix) p.cu_prefix[b + 1] = cached_to + tokens_before + now;
    }
    const int rows = min(kPlanThreads, p.batch - base);
    for (int t = first + rank * kPlanThreads + tid; t < placed; t += ctas * kPlanThreads) {
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
  for (long long t = placed + (long long)rank * kPlanThreads + tid; t < p.max_tokens; t += (long long)ctas * kPlanThreads) {
    p.slot_mapping[t] = -1;
    if (p.positions) p.positions[t] = 0;
    if (p.ws_rows) p.ws_rows[t] = -1;
  }
  if (rank == 0 && tid == 0) *p.free_left = free_count - used;
}

}  // namespace

cudaError_t launch_plan_append(const PlanArgs& args, cudaStream_t stream) {
  int ctas = 1;
  while (ctas < kPlanMaxCluster && args.max_tokens > (long long)ctas * kPlanThreads) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, args, ctas);
}

}  // namespace nvfp4kv
