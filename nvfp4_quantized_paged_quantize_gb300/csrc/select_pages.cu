// select_pages.cu -- the pages that a sparse decode reads: of every (sequence, KV
// head) the first, the latest, and those between with the largest scores
// (nvfp4kv_select_pages), in page order.
//
// One CTA per pair, or a cluster where there are many pages; each thread keeps its pages' scores in registers.  The smallest
// kept one is found by a histogram of equal parts of the scores' range (1024 or 2048),
// whose part with the threshold mostly has few enough to rank one by one.  Else,
// and where the range is not finite, by histograms of the scores as integers that
// order like the floats (keys), of equal parts of what is left each time.
// (Parts of the integers' range from the start are too wide wherever scores lie on both
// sides of zero: half of the integers are smaller than 1 in size.)  Equal keys go to
// the lower page: with n keys above the threshold and e equal to it before a page,
// the page lands at place n + min(e, equal ones still wanted), so one ordered count
// over the warps, which hold consecutive pages, gives every destination.
// Bound by the instructions of one SM and the latency of its steps: the loads, then
// six block barriers (figures: launch_select_pages).
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kFew = 256;
constexpr int kMaxCtas = 8;  // of a cluster, the portable limit
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr uint32_t kKeyNone = 0;  // no float's key: below that of -inf
constexpr float kLeastRange = 1e-30f;  // of the scores, for parts of it

// An unsigned integer that orders like the float: +-0 equal, NaN on top.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// (in order with its like; the compiler spread plain loads: 0.3 us)
__device__ __forceinline__ float load_score(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

template <int kThreads, int kBins>
struct SelectShared {
  uint32_t hist[kBins];
  uint32_t warp_sum[kThreads / 32], warp_min[kThreads / 32], warp_max[kThreads / 32];
  uint2 warp_count[kThreads / 32];  // a warp's keys above and equal to the threshold
  uint32_t bin, above, in_bin;      // the threshold's part, the keys above it, the keys in it
  uint32_t few[kFew], few_count;
  uint32_t all_few[kFew];  // of a cluster's CTAs
  uint32_t cta_min, cta_max;  // of a cluster's CTA
  uint2 cta_count;
};

// kRows: scores of a thread in registers.  A warp holds consecutive pages, `rows` to a
// lane; kMore: there may be more than kRows, read again at every use.  kCluster: a cluster
// of `ctas` CTAs per pair, each with consecutive pages; every CTA adds up all parts of the
// histograms and finds the same cut.
template <int kThreads, int kBins, int kRows, bool kMore, bool kCluster, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) select_kernel(const SelectArgs p, int ctas) {
  constexpr int kWarps = kThreads / 32;
  __shared__ SelectShared<kThreads, kBins> s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long pair = kCluster ? blockIdx.x / ctas : blockIdx.x;
  const int cta = kCluster ? blockIdx.x % ctas : 0;
  after_earlier_kernels();
  const int L = p.seq_lens[(int)(pair / p.hkv)];
  long long pages = ((long long)L + kPage - 1) / kPage;
  if (L < 0 || pages > p.score_stride) {
    if (tid == 0 && cta == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    pages = L < 0 ? 0 : p.score_stride;
  }
  const int n = (int)pages;
  int32_t* selected = p.selected + pair * p.budget;
  auto meet = [] {  // of the cluster's threads
    __syncwarp();
    cluster_sync();
  };
  const int all_threads = kCluster ? ctas * kThreads : kThreads, all_tid = cta * kThreads + tid;
  if (n <= p.budget) {
    for (int i = all_tid; i < p.budget; i += all_threads) selected[i] = i < n ? i : -1;
    return;
  }
  // n > budget >= first + recent: the middle is not empty
  const int middle = n - p.first - p.recent, want = p.budget - p.first - p.recent;
  const float* mine = p.scores + pair * p.score_stride + p.first;
  // warp w of all: pages [32 rows w, 32 rows (w + 1)) of the middle
  const int rows = (middle + all_threads - 1) / all_threads;
  const int at0 = (all_tid >> 5) * rows * 32 + lane;
  const int own = min(max((middle - at0 + 31) / 32, 0), rows);  // scores of this thread
  float x[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) x[j] = j < own ? load_score(mine + at0 + 32 * j) : 0.0f;
  auto each = [&](auto f) {  // every score of the thread
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (j < own) f(x[j]);
    if constexpr (kMore)
      for (int j = kRows; j < own; ++j) f(mine[at0 + 32 * j]);
  };
  for (int i = all_tid; i < p.first; i += all_threads) selected[i] = i;
  for (int i = all_tid; i < p.recent; i += all_threads) selected[p.budget - p.recent + i] = n - p.recent + i;
  if (want == 0) return;

  // the smallest and the largest key of the scores that `of` picks, over the block; every
  // thread calls it, after the last use of the warps' words
  uint32_t lo, hi;
  auto bounds = [&](auto of) {
    lo = 0xFFFFFFFFu;
    hi = 0;
    each([&](float v) {
      if (!of(v)) return;
      const uint32_t k = order_key(v);
      lo = min(lo, k);
      hi = max(hi, k);
    });
    lo = __reduce_min_sync(kAll, lo);
    hi = __reduce_max_sync(kAll, hi);
    if (lane == 0) {
      s.warp_min[warp] = lo;
      s.warp_max[warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(kAll, s.warp_min[lane % kWarps]);
    hi = __reduce_max_sync(kAll, s.warp_max[lane % kWarps]);
    if constexpr (kCluster) {
      if (tid == 0) {
        s.cta_min = lo;
        s.cta_max = hi;
      }
      meet();
      lo = __reduce_min_sync(kAll, ld_cluster(&s.cta_min, lane % ctas));
      hi = __reduce_max_sync(kAll, ld_cluster(&s.cta_max, lane % ctas));
    }
  };
  if (tid == 0) s.few_count = 0;
#pragma unroll
  for (int i = 0; i < kBins / kThreads; ++i) s.hist[tid + i * kThreads] = 0;
  bounds([](float) { return true; });

  // the threshold lies among the keys lo + [0, width), of which the `left` largest stay
  uint32_t left = (uint32_t)want, width = 0xFFFFFFFFu, cut = 0;
  int shift = 0;
  // the largest part, and what a count found: the threshold's part, the keys in it
  uint32_t bin = 0, count = 0;
  // counts the scores by their parts `of` (kBins for none), finds the threshold's
  auto find = [&](auto of) {
    each([&](float v) {
      const uint32_t at = of(v);
      if (at < kBins) atomicAdd(&s.hist[at], 1u);
    });
    if constexpr (kCluster) meet(); else __syncthreads();
    constexpr int kPer = kBins / kThreads;
    // this thread's parts, from the top down
    uint32_t c[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = kBins - 1 - (kPer * tid + j);
      if constexpr (kCluster) {
        c[j] = 0;
#pragma unroll
        for (int r = 0; r < kMaxCtas; ++r)
          if (r < ctas) c[j] += ld_cluster(&s.hist[i], r);
      } else {
        c[j] = s.hist[i];
        s.hist[i] = 0;
      }
      sum += c[j];
    }
    if constexpr (kCluster) {
      meet();  // every CTA has read them
#pragma unroll
      for (int j = 0; j < kPer; ++j) s.hist[kBins - 1 - (kPer * tid + j)] = 0;
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
    bin = s.bin;
    count = s.in_bin;
    left -= s.above;
  };
  // the cut among the `count` <= kFew scores that `of` picks, ranked by every warp (up to 32)
  // or by the block: it has fewer than `left` keys above it, and with its equals at least that
  auto rank = [&](auto of) {
    each([&](float v) {
      if (!of(v)) return;
      const uint32_t at = atomicAdd(&s.few_count, 1u);
      if (at < kFew) s.few[at] = order_key(v);  // (always, unless the scores change meanwhile)
    });
    const uint32_t* few = s.few;
    if constexpr (kCluster) {
      meet();
      // the CTAs' keys one after the other
      uint32_t before = 0, here = 0;
      int from = 0;
      for (; from < ctas; before += here, ++from) {
        here = ld_cluster(&s.few_count, from);
        if (tid < before + here) break;
      }
      if (from < ctas && tid < kFew) s.all_few[tid] = ld_cluster(&s.few[tid - before], from);
      few = s.all_few;
    }
    __syncthreads();
    if (count <= 32) {
      const uint32_t k = lane < count ? few[lane] : kKeyNone;
      uint32_t greater = 0, equal = 0;
      for (uint32_t r = 0; r < count; ++r) {
        const uint32_t other = __shfl_sync(kAll, k, r);
        greater += other > k;
        equal += other == k;
      }
      const int who = __ffs(__ballot_sync(kAll, lane < count && greater < left && greater + equal >= left)) - 1;
      cut = __shfl_sync(kAll, k, who);
      left -= __shfl_sync(kAll, greater, who);
    } else {
      if (tid < count) {
        const uint32_t k = few[tid];
        uint32_t greater = 0, equal = 0;
        for (uint32_t r = 0; r < count; ++r) {
          const uint32_t other = few[r];
          greater += other > k;
          equal += other == k;
        }
        if (greater < left && greater + equal >= left) {  // equal keys: the same words
          s.bin = k;
          s.above = greater;
        }
      }
      __syncthreads();
      cut = s.bin;
      left -= s.above;
    }
  };
  bool found = false;
  const float low = key_score(lo), range = key_score(hi) - low;
  if (range >= kLeastRange && range < INFINITY) {  // (not with an infinity or a NaN at either end)
    const float scale = (float)(kBins - 1) / range;
    // rounding keeps the order: a larger score is in no lower part
    auto part = [&](float v) { return min((uint32_t)((v - low) * scale), (uint32_t)kBins - 1); };
    find(part);
    const uint32_t chosen = bin;
    if (count <= kFew) {
      rank([&](float v) { return part(v) == chosen; });
      found = true;
    } else {
      bounds([&](float v) { return part(v) == chosen; });
      width = hi - lo + 1;
    }
  }
  constexpr int kBits = kBins == 2048 ? 11 : 10;
  static_assert(kBins == 1 << kBits, "a part is a bit field of the keys");
  if (!found) shift = max(0, 32 - __clz(hi - lo) - kBits);  // (hi - lo) >> shift < kBins
  while (!found) {
    find([&](float v) {
      const uint32_t k = order_key(v);
      return k - lo < width ? (k - lo) >> shift : (uint32_t)kBins;
    });
    lo += bin << shift;
    found = true;
    width = min(1u << shift, hi - lo + 1);  // the last piece ends with the part: keys behind it are counted already
    if (shift == 0) {  // one key
      cut = lo;
    } else if (count == left) {  // the whole part stays
      cut = lo - 1;
      left = 0;
    } else if (count <= kFew) {
      rank([&](float v) { return order_key(v) - lo < width; });
    } else {
      shift = max(0, shift - kBits);
      found = false;
    }
  }

  // keys above the cut stay, and the first `left` equal to it: by rows of the warp, then
  // by warps
  uint32_t above[kRows], equal[kRows], g = 0, e = 0;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const uint32_t k = j < own ? order_key(x[j]) : kKeyNone;
    above[j] = __ballot_sync(kAll, k > cut);
    equal[j] = __ballot_sync(kAll, k == cut);
    g += __popc(above[j]);
    e += __popc(equal[j]);
  }
  auto more = [&](int j, uint32_t& a, uint32_t& q) {  // a row past the registers
    const uint32_t k = j < own ? order_key(mine[at0 + 32 * j]) : kKeyNone;
    a = __ballot_sync(kAll, k > cut);
    q = __ballot_sync(kAll, k == cut);
  };
  if constexpr (kMore)
    for (int j = kRows; j < rows; ++j) {
      uint32_t a, q;
      more(j, a, q);
      g += __popc(a);
      e += __popc(q);
    }
  if (lane == 0) s.warp_count[warp] = make_uint2(g, e);
  __syncthreads();
  const uint2 counted = s.warp_count[lane % kWarps], counted_last = s.warp_count[kWarps - 1];
  g = __reduce_add_sync(kAll, lane < warp ? counted.x : 0u);
  e = __reduce_add_sync(kAll, lane < warp ? counted.y : 0u);
  if constexpr (kCluster) {
    if (warp == kWarps - 1 && lane == 0) s.cta_count = make_uint2(g + counted_last.x, e + counted_last.y);
    meet();
    const bool earlier = lane < cta;
    g += __reduce_add_sync(kAll, earlier ? ld_cluster(&s.cta_count.x, lane) : 0u);
    e += __reduce_add_sync(kAll, earlier ? ld_cluster(&s.cta_count.y, lane) : 0u);
  }
  const uint32_t below = (1u << lane) - 1;
  auto put = [&](int j, uint32_t a, uint32_t q) {
    const uint32_t before = e + __popc(q & below);
    if ((a >> lane & 1) || ((q >> lane & 1) && before < left))
      selected[p.first + (int)(g + __popc(a & below) + min(before, left))] = p.first + at0 + 32 * j;
    g += __popc(a);
    e += __popc(q);
  };
#pragma unroll
  for (int j = 0; j < kRows; ++j)
    if (j < rows) put(j, above[j], equal[j]);
  if constexpr (kMore)
    for (int j = kRows; j < rows; ++j) {
      uint32_t a, q;
      more(j, a, q);
      put(j, a, q);
    }
  if constexpr (kCluster) meet();  // no CTA leaves while another may still read its words
}

}  // namespace

cudaError_t launch_select_pages(const SelectArgs& args, int num_sms, cudaStream_t stream) {
  const int64_t pairs = (int64_t)args.batch * args.hkv;
  // The lengths are on the device, so the shape goes by the pages that the scores have room
  // for.  256 threads, 1024 with 9 scores each and 1024 with 16, in a captured graph: 768
  // pairs of 500 pages 6.8, 25 and 34 us, of 2000 8.9, 27 and 36, 32 pairs of 2000 4.5, 5.5
  // and 7.1, of 8187 -, 7.4 and 9.4.
  const int64_t most = args.score_stride;
  if (most <= 256 * 8)
    return launch_overlapped(select_kernel<256, 1024, 8, false, false, 6>, pairs, 256, 0, 1, stream, args, 1);
  // More than a CTA keeps in registers, where SMs would stay empty: clusters with 4096 pages
  // or more to a CTA.  With them and without (scores past the registers read again at every
  // use): 8 pairs of 62500 pages 18 and 40 us, of 125000 20 and 88, 32 of 31250 14 and 20;
  // but 32 of 15625 11.5 and 10.9, six barriers of a cluster.
  int ctas = 1;
  while (most > 1024 * 16 && ctas < kMaxCtas && pairs * 2 * ctas <= num_sms && most >= 2 * ctas * 4096) ctas *= 2;
  if (ctas > 1 && most <= (int64_t)ctas * 1024 * 9)
    return launch_overlapped(select_kernel<1024, 2048, 9, false, true, 1>, pairs * ctas, 1024, 0, ctas, stream, args, ctas);
  if (ctas > 1)
    return launch_overlapped(select_kernel<1024, 2048, 16, true, true, 1>, pairs * ctas, 1024, 0, ctas, stream, args, ctas);
  if (most <= 1024 * 9)
    return launch_overlapped(select_kernel<1024, 2048, 9, false, false, 1>, pairs, 1024, 0, 1, stream, args, 1);
  return launch_overlapped(select_kernel<1024, 2048, 16, true, false, 1>, pairs, 1024, 0, 1, stream, args, 1);
}

}  // namespace nvfp4kv
