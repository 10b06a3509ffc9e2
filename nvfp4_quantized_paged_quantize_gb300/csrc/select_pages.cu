// select_pages.cu -- the pages that a sparse decode reads: of every (sequence, KV
// head) the first, the latest, and those between with the largest scores
// (nvfp4kv_select_pages), in page order.
//
// One CTA per pair.  A radix selection over the scores' bits as ordered integers
// finds the smallest kept key, eight bits at a time; equal keys go to the lower
// page: with n above the threshold and e equal to it before a page, the page
// lands at place n + min(e, equal ones still wanted).
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kSpThreads = 512;
constexpr int kSpWarps = kSpThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;

// An unsigned integer that orders like the float: +-0 equal, NaN on top.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSpThreads) select_kernel(const SelectArgs p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];
  __shared__ uint32_t counts[kSpWarps][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long pair = blockIdx.x;
  const int b = (int)(pair / p.hkv);
  const int L = __ldg(p.seq_lens + b);
  long long pages = ((long long)L + kPage - 1) / kPage;
  if (L < 0 || pages > p.score_stride) {
    if (tid == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    pages = L < 0 ? 0 : p.score_stride;
  }
  const int n = (int)pages;
  const float* scores = p.scores + pair * p.score_stride;
  int32_t* selected = p.selected + pair * p.budget;
  if (n <= p.budget) {
    for (int i = tid; i < p.budget; i += kSpThreads) selected[i] = i < n ? i : -1;
    return;
  }
  // n > budget >= first + recent: the middle is not empty
  const int middle = n - p.first - p.recent, want = p.budget - p.first - p.recent;
  for (int i = tid; i < p.first; i += kSpThreads) selected[i] = i;
  for (int i = tid; i < p.recent; i += kSpThreads) selected[p.budget - p.recent + i] = n - p.recent + i;
  if (want == 0) return;
  const float* mine = scores + p.first;
  uint32_t prefix = 0, left = (uint32_t)want;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < middle; i += kSpThreads) {
      const uint32_t k = order_key(mine[i]);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // this lane's eight bins from the top down
      uint32_t sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += hist[255 - 8 * lane - j];
      uint32_t incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(kAll, incl, off);
        if (lane >= off) incl += v;
      }
      uint32_t above = incl - sum;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t c = hist[255 - 8 * lane - j];
        if (above < left && above + c >= left) {
          found[0] = 255 - 8 * lane - j;
          found[1] = above;
        }
        above += c;
      }
    }
    __syncthreads();
    prefix = prefix << 8 | found[0];
    left -= found[1];
    __syncthreads();
  }
  // prefix is the smallest kept key; `left` of the pages equal to it stay
  uint32_t g0 = 0, e0 = 0;
  for (int base = 0; base < middle; base += kSpThreads) {
    const int i = base + tid;
    const uint32_t k = i < middle ? order_key(mine[i]) : 0;
    const uint32_t bg = __ballot_sync(kAll, i < middle && k > prefix), be = __ballot_sync(kAll, i < middle && k == prefix);
    if (lane == 0) {
      counts[warp][0] = __popc(bg);
      counts[warp][1] = __popc(be);
    }
    __syncthreads();
    uint32_t g = g0, e = e0;
    for (int w = 0; w < kSpWarps; ++w) {
      if (w < warp) {
        g += counts[w][0];
        e += counts[w][1];
      }
      g0 += counts[w][0];
      e0 += counts[w][1];
    }
    const uint32_t below = (1u << lane) - 1;
    g += __popc(bg & below);
    e += __popc(be & below);
    if (i < middle && (k > prefix || (k == prefix && e < left))) selected[p.first + (int)(g + min(e, left))] = p.first + i;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_select_pages(const SelectArgs& args, cudaStream_t stream) {
  select_kernel<<<(unsigned)((int64_t)args.batch * args.hkv), kSpThreads, 0, stream>>>(args);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
