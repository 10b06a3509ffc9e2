// evict.cu -- cache eviction by accumulated attention weight: keep the first
// and the most recent tokens and, of those between, the ones with the largest
// sums, packed in order into other pages (nvfp4kv_evict).
//
// select_kernel: a cluster of 1 to 8 CTAs per (sequence, KV head).  Each CTA
//   reads its share of the middle tokens' sums once into shared memory, as
//   integers that order like the floats.  A radix selection finds the smallest
//   kept key: three passes over shared memory (11, 11 and 10 bits), each a
//   histogram of its own tokens whose bins that are not empty every CTA adds to
//   the first CTA's totals (distributed shared memory; few bins hold anything),
//   which finds the threshold's bin and tells the others.  Equal keys go to the
//   lower index: with g tokens above and e tokens equal to the threshold before
//   it, a kept token lands at place g + min(e, equal ones still wanted), so one
//   ordered count over the cluster gives every destination and the list comes out
//   in token order.
//   Bytes: 4 read per token, 8 written per kept token.  Bound by the latency of
//   its passes: 18 us for 256 pairs of 8193 tokens (8.4 MB read), 31 us for 32
//   pairs of 100K to 131K (14.8 MB), cold.
// pack_kernel: one warp per destination page-head, launched as the programmatic
//   dependent of the first.  It gathers 16 tokens' K rows and scales, their
//   nibbles of V's token-pair bytes and their V scale bytes, all loads in
//   flight together, and writes the page-head whole.  HBM-bound: 144 bytes in
//   and out per kept token, plus what the 32-byte sectors drag along (a V byte
//   holds two tokens, a V scale sector the scales of two blocks).  2048 of 8193
//   tokens kept, 256 pairs: 45 us, 147.8 MB read and 39.4 MB written back to DRAM.
//   With the packing in the selection's launch (a cluster packs its own pair) the
//   whole eviction took 73 us instead of 69: fewer warps gather at a time.
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;           // 11 bits
constexpr int kPasses = 3;            // of 11, 11 and 10 bits
constexpr int kSpan = 128;            // tokens a warp takes at a time, four per lane
constexpr int kKeyCap = 20 * 1024;    // keys a CTA holds: with the histograms two CTAs fit an SM
static_assert(kKeyCap % (kSpan * kSelectWarps) == 0, "the keys are padded to whole spans of every warp");
constexpr int kMaxCluster = 8;        // the portable limit
static_assert(kMaxCluster * kSelectThreads == 4096, "the largest budget of nvfp4kv_evict allows for this stride");
constexpr int kPackWarps = 8;

struct EvictParams {
  uint8_t* pages;
  int32_t num_pages;
  int32_t hkv;
  const int32_t* page_table;
  int32_t max_pages;
  const int32_t* seq_lens;
  const float* weights;
  long long weight_stride;
  int32_t budget, first, recent;
  const int32_t* dst_table;
  int32_t dst_max_pages;
  int32_t dst_pages;      // pages of `budget` tokens
  long long page_heads;   // batch * hkv * dst_pages
  int32_t* kept;
  float* kept_weights;    // or null
  long long kept_stride;
  int32_t* new_lens;      // or null
  int32_t* status;
};

// A sequence's tokens: its length, cut to what the page table and the sums
// cover (flagged by the select kernel).
__device__ __forceinline__ int seq_tokens(const EvictParams& p, int b, bool flag) {
  int L = __ldg(p.seq_lens + b);
  const long long cover = (long long)p.max_pages * kPage;
  const int lmax = (int)(cover < p.weight_stride ? cover : p.weight_stride);
  if (L < 0 || L > lmax) {
    if (flag) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    L = L < 0 ? 0 : lmax;
  }
  return L;
}

// An unsigned integer that orders like the float: +-0 equal, NaN on top.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr uint32_t kKeyNone = 0;  // no float's key: below that of -inf

// Store to, add to, the same shared-memory word in another CTA of the cluster.
__device__ __forceinline__ void st_cluster(uint32_t* local, uint32_t rank, uint32_t n) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(n) : "memory");
}
__device__ __forceinline__ void add_cluster(uint32_t* local, uint32_t rank, uint32_t n) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(n) : "memory");
}

struct SelectShared {
  alignas(16) uint32_t total[kPasses][kBins];  // over the cluster
  alignas(16) uint32_t own[kBins];             // this CTA's, where the cluster has others
  uint32_t warp_sum[kSelectWarps];
  uint32_t found_bin[kPasses], found_above[kPasses];  // the threshold's bin, and how many keys lie in bins above it
  uint32_t warp_count[kSelectWarps][2];  // tokens above / equal to the threshold
  uint32_t cta_gt, cta_eq;
};

// kFits: every CTA's share of the tokens fits its shared memory (else what does
// not is read again in each pass).
template <bool kFits>
__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const EvictParams p, int cluster) {
  extern __shared__ __align__(16) uint32_t keys[];  // kKeyCap
  __shared__ SelectShared s;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pair = blockIdx.x / cluster, rank = blockIdx.x - pair * cluster;
  const int b = pair / p.hkv;
  const int L = seq_tokens(p, b, tid == 0 && rank == 0 && pair % p.hkv == 0);
  const int n = L < p.budget ? L : p.budget;
  const float* w = p.weights + (long long)pair * p.weight_stride;
  int32_t* kept = p.kept + (long long)pair * p.budget;
  float* kw = p.kept_weights ? p.kept_weights + (long long)pair * p.kept_stride : nullptr;
  const int part = rank * kSelectThreads + tid, parts = cluster * kSelectThreads;
  for (int i = n + part; i < p.budget; i += parts) {
    kept[i] = -1;
    if (kw) kw[i] = 0.0f;
  }
  if (L <= p.budget) {
    for (int i = part; i < L; i += parts) {
      kept[i] = i;
      if (kw) kw[i] = __ldg(w + i);
    }
    return;
  }
  const int middle = L - p.first - p.recent, want = n - p.first - p.recent;  // 0 <= want < middle
  // the tokens that stay in any case
  auto keep_ends = [&]() {
    for (int i = part; i < p.first + p.recent; i += parts) {
      const int place = i < p.first ? i : n - p.first - p.recent + i;
      const int token = i < p.first ? i : L - p.first - p.recent + i;
      kept[place] = token;
      if (kw) kw[place] = __ldg(w + token);
    }
  };
  if (want == 0) {
    keep_ends();
    return;
  }

  // this CTA's share of the middle tokens, as keys
  const int t0 = p.first + (int)((long long)middle * rank / cluster);
  const int count = p.first + (int)((long long)middle * (rank + 1) / cluster) - t0;
  const float* mine = w + t0;
  constexpr int kBatch = 16;  // loads in flight per thread
  float x[kBatch];
  auto fetch = [&](int b0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = b0 + j * kSelectThreads;
      x[j] = i < count ? __ldg(mine + i) : 0.0f;
    }
  };
  fetch(tid);
  constexpr int kPer = kBins / kSelectThreads;
  static_assert(kPer == 4, "a thread's bins are one 16-byte word");
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass)
    *reinterpret_cast<uint4*>(&s.total[pass][kPer * tid]) = make_uint4(0u, 0u, 0u, 0u);
  *reinterpret_cast<uint4*>(&s.own[kPer * tid]) = make_uint4(0u, 0u, 0u, 0u);
  // spans of the CTA's tokens; a warp's are contiguous: [i0, i1)
  const int spans = (count + kSpan - 1) / kSpan, warp_spans = (spans + kSelectWarps - 1) / kSelectWarps;
  const int i0 = warp * warp_spans * kSpan, i1 = i0 + warp_spans * kSpan;
  // the keys of the CTA's tokens i .. i + 3 (i a multiple of 4)
  auto keys_at = [&](int i) {
    if (kFits || i < kKeyCap) return *reinterpret_cast<const uint4*>(keys + i);
    uint4 k;
    k.x = i < count ? order_key(__ldg(mine + i)) : kKeyNone;
    k.y = i + 1 < count ? order_key(__ldg(mine + i + 1)) : kKeyNone;
    k.z = i + 2 < count ? order_key(__ldg(mine + i + 2)) : kKeyNone;
    k.w = i + 3 < count ? order_key(__ldg(mine + i + 3)) : kKeyNone;
    return k;
  };
  const int padded = min(warp_spans * kSelectWarps * kSpan, kKeyCap);
  for (int i = count + tid; i < padded; i += kSelectThreads) keys[i] = kKeyNone;
  keep_ends();
  // every CTA's totals are zero before any CTA adds to them
  __syncthreads();
  if (cluster > 1) cluster_sync();
  for (int b0 = tid; b0 < count; b0 += kBatch * kSelectThreads) {
    if (b0 != tid) fetch(b0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = b0 + j * kSelectThreads;
      if (i < count) {
        const uint32_t k = order_key(x[j]);
        if (kFits || i < kKeyCap) keys[i] = k;
        atomicAdd(&(cluster > 1 ? s.own : s.total[0])[k >> 21], 1u);
      }
    }
  }

  uint32_t prefix = 0, left = (uint32_t)want;  // the threshold's bits so far; keys still to be found among those that share them
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    constexpr int kShift[kPasses] = {21, 10, 0};
    const int shift = kShift[pass], bits = pass == kPasses - 1 ? 10 : 11;
    uint32_t* const hist = cluster > 1 ? s.own : s.total[pass];
    if (pass > 0) {
      const int above = kShift[pass > 0 ? pass - 1 : 0];
      for (int i = i0 + 4 * lane; i < i1; i += kSpan) {
        const uint4 k4 = keys_at(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t k = j == 0 ? k4.x : j == 1 ? k4.y : j == 2 ? k4.z : k4.w;
          if ((k >> above) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
        }
      }
    }
    __syncthreads();
    if (cluster > 1) {
      uint4* const at = reinterpret_cast<uint4*>(&s.own[kPer * tid]);
      const uint4 mine4 = *at;
      *at = make_uint4(0u, 0u, 0u, 0u);
      const uint32_t n[kPer] = {mine4.x, mine4.y, mine4.z, mine4.w};
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (n[j] != 0)
          add_cluster(&s.total[pass][kPer * tid + j], 0, n[j]);
      __syncwarp();
      cluster_sync();
    }
    if (rank == 0) {
      // this thread's four bins, from the top down
      const uint4 c = *reinterpret_cast<const uint4*>(&s.total[pass][kBins - kPer * (tid + 1)]);
      const uint32_t bin[kPer] = {c.w, c.z, c.y, c.x};
      const uint32_t sum = (c.x + c.y) + (c.z + c.w);
      uint32_t incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += v;
      }
      if (lane == 31) s.warp_sum[warp] = incl;
      __syncthreads();
      uint32_t before = incl - sum;
      for (int k = 0; k < warp; ++k) before += s.warp_sum[k];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (before < left && before + bin[j] >= left) {  // exactly one bin of the whole histogram
          const uint32_t found = kBins - 1 - (tid * kPer + j);
          s.found_bin[pass] = found;
          s.found_above[pass] = before;
          for (int r = 1; r < cluster; ++r) {
            st_cluster(&s.found_bin[pass], r, found);
            st_cluster(&s.found_above[pass], r, before);
          }
        }
        before += bin[j];
      }
    }
    __syncthreads();
    if (cluster > 1) cluster_sync();
    prefix = (prefix << bits) | s.found_bin[pass];
    left -= s.found_above[pass];
  }
  // prefix is the smallest kept key; `left` of the tokens equal to it stay

  // ordered counts: a warp's contiguous tokens, then the warps, then the CTAs
  auto count4 = [&](const uint4& k, uint32_t& gt, uint32_t& eq) {
    gt += (uint32_t)(k.x > prefix) + (uint32_t)(k.y > prefix) + (uint32_t)(k.z > prefix) + (uint32_t)(k.w > prefix);
    eq += (uint32_t)(k.x == prefix) + (uint32_t)(k.y == prefix) + (uint32_t)(k.z == prefix) + (uint32_t)(k.w == prefix);
  };
  uint32_t gt = 0, eq = 0;
  for (int i = i0 + 4 * lane; i < i1; i += kSpan) count4(keys_at(i), gt, eq);
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  if (lane == 0) {
    s.warp_count[warp][0] = gt;
    s.warp_count[warp][1] = eq;
  }
  __syncthreads();
  uint32_t g0 = 0, e0 = 0, gall = 0, eall = 0, gcta = 0, ecta = 0;  // before: the warp (in its CTA), all of the CTA, the CTA
  for (int k = 0; k < kSelectWarps; ++k) {
    if (k == warp) g0 = gall, e0 = eall;
    gall += s.warp_count[k][0];
    eall += s.warp_count[k][1];
  }
  if (cluster > 1) {
    if (tid == 0) {
      s.cta_gt = gall;
      s.cta_eq = eall;
    }
    __syncwarp();
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      gcta += ld_cluster(&s.cta_gt, r);
      ecta += ld_cluster(&s.cta_eq, r);
    }
    g0 += gcta;
    e0 += ecta;
  }
  const uint32_t below = (1u << lane) - 1;
  for (int i = i0 + 4 * lane; i < i1; i += kSpan) {
    const uint4 k4 = keys_at(i);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    uint32_t bg[4], be[4];  // token j of each lane: above, equal
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bg[j] = __ballot_sync(0xFFFFFFFFu, k[j] > prefix);
      be[j] = __ballot_sync(0xFFFFFFFFu, k[j] == prefix);
    }
    // what lies before the lane's first token: tokens run over j, then over lanes
    uint32_t g = g0 + __popc(bg[0] & below) + __popc(bg[1] & below) + __popc(bg[2] & below) + __popc(bg[3] & below);
    uint32_t e = e0;
    const bool ties = (be[0] | be[1] | be[2] | be[3]) != 0;
    if (ties) e += __popc(be[0] & below) + __popc(be[1] & below) + __popc(be[2] & below) + __popc(be[3] & below);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool up = k[j] > prefix, tie = ties && k[j] == prefix;
      if (up || (tie && e < left)) {
        kept[p.first + (int)(g + min(e, left))] = t0 + i + j;
      }
      g += up;
      e += tie;
    }
    g0 += __popc(bg[0]) + __popc(bg[1]) + __popc(bg[2]) + __popc(bg[3]);
    if (ties) e0 += __popc(be[0]) + __popc(be[1]) + __popc(be[2]) + __popc(be[3]);
  }
  if (kw) {
    // the sums of what this CTA kept: [first_place, last_place) of the list
    __syncthreads();
    const int first_place = p.first + (int)(gcta + min(ecta, left));
    const int last_place = p.first + (int)(gcta + gall + min(ecta + eall, left));
    for (int i = first_place + tid; i < last_place; i += kSelectThreads) kw[i] = __ldg(w + kept[i]);
  }
  __syncwarp();
  if (cluster > 1) cluster_sync();  // no CTA leaves while another may still read its counts
}

// Bytes 0-15 of a V pair row -> the token's codes in the low nibbles (odd
// tokens lie in the high ones).
__device__ __forceinline__ uint32_t v_codes(uint32_t w, bool odd) { return (odd ? w >> 4 : w) & 0x0F0F0F0Fu; }

__global__ void __launch_bounds__(kPackWarps * 32) pack_kernel(const EvictParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long at = (long long)blockIdx.x * kPackWarps + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (at >= p.page_heads) return;
  const int pair = (int)(at / p.dst_pages), page = (int)(at - (long long)pair * p.dst_pages);
  const int b = pair / p.hkv, h = pair - b * p.hkv;
  // min(min(L, budget), budget) is min(L, budget): new_lens may be seq_lens itself
  const int L = seq_tokens(p, b, false), n = L < p.budget ? L : p.budget;
  if (h == 0 && page == 0 && lane == 0 && p.new_lens) p.new_lens[b] = n;
  if (page * kPage >= n) return;
  const int dst_id = __ldg(p.dst_table + (long long)b * p.dst_max_pages + page);
  if (dst_id < 0 || dst_id >= p.num_pages) {
    if (lane == 0) flag_error(p.status, NVFP4KV_DEVERR_PAGE);
    return;
  }
  // lane r (and r + 16): where token r's page-head lies (-1: zeros) and its row there
  long long base = -1;
  int row = 0;
  const int slot = page * kPage + (lane & 15);
  if (slot < n) {
    const int token = __ldcg(p.kept + (long long)pair * p.budget + slot);
    const int id = __ldg(p.page_table + (long long)b * p.max_pages + token / kPage);
    row = token % kPage;
    if (id >= 0 && id < p.num_pages)
      base = ((long long)id * p.hkv + h) * kPageHeadBytes;
    else
      flag_error(p.status, NVFP4KV_DEVERR_PAGE);
  }
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto load16 = [&](long long from, int offset) {
    return from < 0 ? zero : __ldg(reinterpret_cast<const uint4*>(p.pages + from + offset));
  };
  // K rows: token 8 i + lane / 4, 16 bytes each
  uint4 k[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 8 * i + (lane >> 2);
    const long long from = __shfl_sync(0xFFFFFFFFu, base, r);
    const int src = __shfl_sync(0xFFFFFFFFu, row, r);
    k[i] = load16(from, kOffKData + src * kRowBytes + 16 * (lane & 3));
  }
  // K scales: lane r < 16, 8 bytes
  uint2 ks = make_uint2(0u, 0u);
  if (lane < 16 && base >= 0) ks = __ldg(reinterpret_cast<const uint2*>(p.pages + base + k_scale_offset(row, 0)));
  // V pairs: pair 4 i + lane / 8, 16 dimensions each, of both tokens
  uint4 v[2][2];
  bool odd[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = 2 * (4 * i + (lane >> 3)) + j;
      const long long from = __shfl_sync(0xFFFFFFFFu, base, r);
      const int src = __shfl_sync(0xFFFFFFFFu, row, r);
      odd[i][j] = src & 1;
      v[i][j] = load16(from, kOffVData + (src >> 1) * kVPairBytes + 16 * (lane & 7));
    }
  // V scales: block lane / 4 of tokens 4 (lane % 4) .. + 3
  uint32_t vs = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 4 * (lane & 3) + j;
    const long long from = __shfl_sync(0xFFFFFFFFu, base, r);
    const int src = __shfl_sync(0xFFFFFFFFu, row, r);
    if (from >= 0) vs |= (uint32_t)__ldg(p.pages + from + v_scale_offset(src, lane >> 2)) << (8 * j);
  }
  uint8_t* dst = p.pages + ((long long)dst_id * p.hkv + h) * kPageHeadBytes;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    reinterpret_cast<uint4*>(dst + kOffKData)[32 * i + lane] = k[i];
    uint4 o;
    o.x = v_codes(v[i][0].x, odd[i][0]) | (v_codes(v[i][1].x, odd[i][1]) << 4);
    o.y = v_codes(v[i][0].y, odd[i][0]) | (v_codes(v[i][1].y, odd[i][1]) << 4);
    o.z = v_codes(v[i][0].z, odd[i][0]) | (v_codes(v[i][1].z, odd[i][1]) << 4);
    o.w = v_codes(v[i][0].w, odd[i][0]) | (v_codes(v[i][1].w, odd[i][1]) << 4);
    reinterpret_cast<uint4*>(dst + kOffVData)[32 * i + lane] = o;
  }
  if (lane < 16) reinterpret_cast<uint2*>(dst + kOffKScale)[lane] = ks;
  reinterpret_cast<uint32_t*>(dst + kOffVScale)[lane] = vs;
}

}  // namespace

cudaError_t launch_evict(const nvfp4kv_cache& c, const int32_t* page_table, int32_t max_pages,
                         const int32_t* seq_lens, int32_t batch, const float* weights, int64_t weight_stride,
                         int32_t budget, int32_t first, int32_t recent, const int32_t* dst_table,
                         int32_t dst_max_pages, int32_t* kept, float* kept_weights, int64_t kept_stride,
                         int32_t* new_lens, int32_t* device_status, int num_sms, cudaStream_t stream) {
  EvictParams p;
  p.pages = c.pages;
  p.num_pages = (int32_t)c.num_pages;
  p.hkv = c.num_kv_heads;
  p.page_table = page_table;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.weights = weights;
  p.weight_stride = weight_stride;
  p.budget = budget;
  p.first = first;
  p.recent = recent;
  p.dst_table = dst_table;
  p.dst_max_pages = dst_max_pages;
  p.dst_pages = (int32_t)(((int64_t)budget + kPage - 1) / kPage);
  const int64_t pairs = (int64_t)batch * c.num_kv_heads;
  p.page_heads = pairs * p.dst_pages;
  p.kept = kept;
  p.kept_weights = kept_weights;
  p.kept_stride = kept_stride;
  p.new_lens = new_lens;
  p.status = device_status;
  static PerDeviceOnce attr_once;
  cudaError_t e = attr_once.run([] {
    const cudaError_t a =
        cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCap * 4);
    if (a != cudaSuccess) return a;
    return cudaFuncSetAttribute(select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCap * 4);
  });
  if (e != cudaSuccess) return e;
  // as many CTAs per pair as its keys need to fit shared memory, and more while
  // SMs would stay empty and a CTA keeps 2048 tokens or more.  The lengths are on
  // the device, so the rule goes by what the page table and the sums have room
  // for, and room to spare costs time: the whole call for 256 pairs of 8193 tokens
  // takes 73 us with room for 8208 tokens, 86, 104 and 148 with room for 32768,
  // 65536 and 131072.  Selection, with just the room it needs, with 1,
  // 2, 4, 8 CTAs a pair: 32 pairs of 16384 tokens 14.9, 12.9, 11.5 (taken), 13.2
  // us; 256 pairs of 8193 16.0 (taken), 27.6, 47.7, 93.7; 32 pairs of 131072 163,
  // 102, 57 (keys read again in each pass), 26.0 (taken)
  const int64_t most = weight_stride < (int64_t)max_pages * kPage ? weight_stride : (int64_t)max_pages * kPage;
  int cluster = 1;
  while (cluster < kMaxCluster && (most > (int64_t)cluster * kKeyCap ||
                                   (pairs * cluster * 2 <= 2 * num_sms && most > (int64_t)cluster * 4096)))
    cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * cluster));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = (size_t)kKeyCap * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, most <= (int64_t)cluster * kKeyCap ? select_kernel<true> : select_kernel<false>, p,
                         cluster);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((p.page_heads + kPackWarps - 1) / kPackWarps));
  cfg.blockDim = dim3(kPackWarps * 32);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, pack_kernel, p);
}

}  // namespace nvfp4kv
