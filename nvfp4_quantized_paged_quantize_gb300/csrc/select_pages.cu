// select_pages.cu -- the pages that a sparse decode reads: of every (sequence, KV
// head) the first, the latest, and those between with the largest scores
// (nvfp4kv_select_pages), in page order.
//
// One CTA per pair; each thread keeps its pages' scores in registers, as integers
// that order like the floats.  The smallest kept key is found by a histogram of
// 2048 equal parts of the keys' range (not of all keys: scores of one pair share
// their upper bits), then of the part that holds it, until that part's keys all
// stay, are all equal, or are few enough (32) for a warp to rank.  Equal keys go to
// the lower page: with n keys above the threshold and e equal to it before a page,
// the page lands at place n + min(e, equal ones still wanted), so one ordered count
// over the warps, which hold consecutive pages, gives every destination.
// Bound by latency: the loads, then some seven block barriers.
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kBins = 2048;
constexpr int kFew = 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr uint32_t kKeyNone = 0;  // no float's key: below that of -inf

// An unsigned integer that orders like the float: +-0 equal, NaN on top.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <int kThreads>
struct SelectShared {
  uint32_t hist[kBins];
  uint32_t warp_sum[kThreads / 32], warp_min[kThreads / 32], warp_max[kThreads / 32];
  uint2 warp_count[kThreads / 32];  // a warp's keys above and equal to the threshold
  uint32_t bin, above, in_bin;      // the threshold's part, the keys above it, the keys in it
  uint32_t few[kFew], few_count;
};

// kRows: keys of a thread in registers.  A warp holds consecutive pages, `rows` to a
// lane; kMore: there may be more than kRows, read again at every use.
template <int kThreads, int kRows, bool kMore>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ SelectShared<kThreads> s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long pair = blockIdx.x;
  const int L = __ldg(p.seq_lens + (int)(pair / p.hkv));
  long long pages = ((long long)L + kPage - 1) / kPage;
  if (L < 0 || pages > p.score_stride) {
    if (tid == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    pages = L < 0 ? 0 : p.score_stride;
  }
  const int n = (int)pages;
  int32_t* selected = p.selected + pair * p.budget;
  if (n <= p.budget) {
    for (int i = tid; i < p.budget; i += kThreads) selected[i] = i < n ? i : -1;
    return;
  }
  // n > budget >= first + recent: the middle is not empty
  const int middle = n - p.first - p.recent, want = p.budget - p.first - p.recent;
  const float* mine = p.scores + pair * p.score_stride + p.first;
  const int rows = (middle + kThreads - 1) / kThreads;  // warp w: pages [32 rows w, 32 rows (w + 1)) of the middle
  const int at0 = warp * rows * 32 + lane;
  uint32_t key[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int i = at0 + 32 * j;
    key[j] = j < rows && i < middle ? order_key(__ldg(mine + i)) : kKeyNone;
  }
  auto key_at = [&](int j) {  // rows past the registers
    const int i = at0 + 32 * j;
    return i < middle ? order_key(__ldg(mine + i)) : kKeyNone;
  };
  auto each = [&](auto f) {  // every key of the thread, in page order over the warp
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (j < rows) f(j, key[j]);
    if constexpr (kMore)
      for (int j = kRows; j < rows; ++j) f(j, key_at(j));
  };
  for (int i = tid; i < p.first; i += kThreads) selected[i] = i;
  for (int i = tid; i < p.recent; i += kThreads) selected[p.budget - p.recent + i] = n - p.recent + i;
  if (want == 0) return;

  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  each([&](int, uint32_t k) {
    if (k != kKeyNone) {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  });
  lo = __reduce_min_sync(kAll, lo);
  hi = __reduce_max_sync(kAll, hi);
  if (lane == 0) {
    s.warp_min[warp] = lo;
    s.warp_max[warp] = hi;
  }
  if (tid == 0) s.few_count = 0;
#pragma unroll
  for (int i = 0; i < kBins / kThreads; ++i) s.hist[tid + i * kThreads] = 0;
  __syncthreads();
  lo = __reduce_min_sync(kAll, s.warp_min[lane % kWarps]);
  hi = __reduce_max_sync(kAll, s.warp_max[lane % kWarps]);

  // the threshold lies among the keys lo + [0, width), of which the `left` largest stay
  uint32_t left = (uint32_t)want, width = 0xFFFFFFFFu, cut;
  int shift = max(0, 32 - __clz(hi - lo) - 11);  // (hi - lo) >> shift < 2048
  while (true) {
    each([&](int, uint32_t k) {
      if (k != kKeyNone && k - lo < width) atomicAdd(&s.hist[(k - lo) >> shift], 1u);
    });
    __syncthreads();
    constexpr int kPer = kBins / kThreads;
    // this thread's parts, from the top down
    uint32_t c[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int bin = kBins - 1 - (kPer * tid + j);
      sum += c[j] = s.hist[bin];
      s.hist[bin] = 0;
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t v = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t above = incl - sum + __reduce_add_sync(kAll, lane < warp ? s.warp_sum[lane % kWarps] : 0u);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (above < left && above + c[j] >= left) {  // exactly one part
        s.bin = kBins - 1 - (kPer * tid + j);
        s.above = above;
        s.in_bin = c[j];
      }
      above += c[j];
    }
    __syncthreads();
    lo += s.bin << shift;
    left -= s.above;
    const uint32_t count = s.in_bin;
    if (shift == 0) {  // one key
      cut = lo;
      break;
    }
    if (count == left) {  // the whole part stays
      cut = lo - 1;
      left = 0;
      break;
    }
    width = 1u << shift;
    if (count <= kFew) {
      each([&](int, uint32_t k) {
        if (k != kKeyNone && k - lo < width) s.few[atomicAdd(&s.few_count, 1u)] = k;
      });
      __syncthreads();
      // every warp ranks them: the cut has fewer than `left` keys above it, and with its equals at least that
      const uint32_t k = lane < count ? s.few[lane] : kKeyNone;
      uint32_t greater = 0, equal = 0;
      for (uint32_t r = 0; r < count; ++r) {
        const uint32_t other = __shfl_sync(kAll, k, r);
        greater += other > k;
        equal += other == k;
      }
      const uint32_t is = __ballot_sync(kAll, lane < count && greater < left && greater + equal >= left);
      const int who = __ffs(is) - 1;
      cut = __shfl_sync(kAll, k, who);
      left -= __shfl_sync(kAll, greater, who);
      break;
    }
    shift = max(0, shift - 11);
  }

  // keys above the cut stay, and the first `left` equal to it
  uint32_t gt = 0, eq = 0;
  each([&](int, uint32_t k) {
    gt += k > cut;
    eq += k == cut;
  });
  gt = __reduce_add_sync(kAll, gt);
  eq = __reduce_add_sync(kAll, eq);
  if (lane == 0) s.warp_count[warp] = make_uint2(gt, eq);
  __syncthreads();
  const uint2 counted = s.warp_count[lane % kWarps];
  uint32_t g = __reduce_add_sync(kAll, lane < warp ? counted.x : 0u), e = __reduce_add_sync(kAll, lane < warp ? counted.y : 0u);
  const uint32_t below = (1u << lane) - 1;
  each([&](int j, uint32_t k) {
    const uint32_t bg = __ballot_sync(kAll, k > cut), be = __ballot_sync(kAll, k == cut);
    const uint32_t before = e + __popc(be & below);
    if (k > cut || (k == cut && before < left))
      selected[p.first + (int)(g + __popc(bg & below) + min(before, left))] = p.first + at0 + 32 * j;
    g += __popc(bg);
    e += __popc(be);
  });
}

}  // namespace

cudaError_t launch_select_pages(const SelectArgs& args, cudaStream_t stream) {
  const unsigned pairs = (unsigned)((int64_t)args.batch * args.hkv);
  // the lengths are on the device, so the shape goes by the pages that the scores have room for
  const int64_t most = args.score_stride;
  if (most <= 256 * 8)
    select_kernel<256, 8, false><<<pairs, 256, 0, stream>>>(args);
  else if (most <= 1024 * 16)
    select_kernel<1024, 16, false><<<pairs, 1024, 0, stream>>>(args);
  else
    select_kernel<1024, 16, true><<<pairs, 1024, 0, stream>>>(args);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
