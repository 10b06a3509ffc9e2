// evict.cu -- cache eviction by accumulated attention weight: keep the first
// and the most recent tokens and, of those between, the ones with the largest
// sums, packed in order into other pages (nvfp4kv_evict).
//
// select_kernel: a cluster of 1 to 8 CTAs per (sequence, KV head).  Each CTA
//   reads its share of the middle tokens' sums once into shared memory, as
//   integers that order like the floats.  A radix selection finds the smallest
//   kept key: three passes over shared memory (11, 11 and 10 bits), each a
//   histogram whose bins are summed over the cluster through distributed
//   shared memory.  Equal keys go to the lower index: with g tokens above and
//   e tokens equal to the threshold before it, a kept token lands at place
//   g + min(e, equal ones still wanted), so one ordered count over the cluster
//   gives every destination and the list comes out in token order.
//   Bytes: 4 read per token, 8 written per kept token; a few microseconds of
//   latency per pass otherwise.
// pack_kernel: one warp per destination page-head, launched as the programmatic
//   dependent of the first.  It gathers 16 tokens' K rows and scales, their
//   nibbles of V's token-pair bytes and their V scale bytes, all loads in
//   flight together, and writes the page-head whole.  HBM-bound: 144 bytes in
//   and out per kept token, plus what the 32-byte sectors drag along (a V byte
//   holds two tokens, a V scale sector the scales of two blocks).
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;           // 11 bits
constexpr int kPasses = 3;            // of 11, 11 and 10 bits
constexpr int kKeyCap = 20 * 1024;    // keys a CTA holds: with the histograms two CTAs fit an SM
constexpr int kMaxCluster = 8;        // the portable limit
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

// The word at this address of the same shared-memory variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* local, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

struct SelectShared {
  uint32_t hist[kPasses][kBins];
  uint32_t warp_sum[kSelectWarps];
  uint32_t found_bin, found_above;       // the threshold's bin, and how many keys lie in bins above it
  uint32_t warp_gt[kSelectWarps], warp_eq[kSelectWarps];
  uint32_t cta_gt, cta_eq;
};

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
  auto keep = [&](int place, int token) {
    kept[place] = token;
    if (kw) kw[place] = __ldg(w + token);
  };
  const int part = rank * kSelectThreads + tid, parts = cluster * kSelectThreads;
  for (int i = n + part; i < p.budget; i += parts) {
    kept[i] = -1;
    if (kw) kw[i] = 0.0f;
  }
  if (L <= p.budget) {
    for (int i = part; i < L; i += parts) keep(i, i);
    return;
  }
  for (int i = part; i < p.first; i += parts) keep(i, i);
  for (int i = part; i < p.recent; i += parts) keep(n - p.recent + i, L - p.recent + i);
  const int middle = L - p.first - p.recent, want = n - p.first - p.recent;  // 0 <= want < middle
  if (want == 0) return;

  // this CTA's share of the middle tokens, as keys
  const int t0 = p.first + (int)((long long)middle * rank / cluster);
  const int count = p.first + (int)((long long)middle * (rank + 1) / cluster) - t0;
  const float* mine = w + t0;
  for (int i = tid; i < kPasses * kBins; i += kSelectThreads) (&s.hist[0][0])[i] = 0;
  __syncthreads();
  // the key of the CTA's token i (those past the shared memory's room are read again in each pass)
  auto key_at = [&](int i) { return i < kKeyCap ? keys[i] : order_key(__ldg(mine + i)); };
  for (int i = tid; i < count; i += kSelectThreads) {
    const uint32_t k = order_key(__ldg(mine + i));
    if (i < kKeyCap) keys[i] = k;
    atomicAdd(&s.hist[0][k >> 21], 1u);
  }

  uint32_t prefix = 0, left = (uint32_t)want;  // the threshold's bits so far; keys still to be found among those that share them
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    constexpr int kShift[kPasses] = {21, 10, 0};
    const int shift = kShift[pass], bits = pass == kPasses - 1 ? 10 : 11;
    if (pass > 0) {
      const int above = kShift[pass > 0 ? pass - 1 : 0];
      for (int i = tid; i < count; i += kSelectThreads) {
        const uint32_t k = key_at(i);
        if ((k >> above) == prefix) atomicAdd(&s.hist[pass][(k >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    __syncthreads();
    if (cluster > 1) cluster_sync();
    // this thread's four bins, from the top down, over the cluster
    constexpr int kPer = kBins / kSelectThreads;
    uint32_t bin[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t* at = &s.hist[pass][kBins - 1 - (tid * kPer + j)];
      uint32_t c = 0;
      if (cluster > 1) {
        for (int r = 0; r < cluster; ++r) c += ld_cluster(at, r);
      } else {
        c = *at;
      }
      bin[j] = c;
      sum += c;
    }
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
        s.found_bin = kBins - 1 - (tid * kPer + j);
        s.found_above = before;
      }
      before += bin[j];
    }
    __syncthreads();
    prefix = (prefix << bits) | s.found_bin;
    left -= s.found_above;
    __syncthreads();
  }
  // prefix is the smallest kept key; `left` of the tokens equal to it stay

  // ordered counts: a warp's contiguous tokens, then the warps, then the CTAs
  const int span = ((count + kSelectWarps - 1) / kSelectWarps + 31) & ~31;
  const int i0 = min(warp * span, count), i1 = min(i0 + span, count);
  uint32_t gt = 0, eq = 0;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key_at(i + lane) : 0;
    gt += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < i1 && k > prefix));
    eq += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < i1 && k == prefix));
  }
  if (lane == 0) {
    s.warp_gt[warp] = gt;
    s.warp_eq[warp] = eq;
  }
  __syncthreads();
  uint32_t g0 = 0, e0 = 0, gall = 0, eall = 0;
  for (int k = 0; k < kSelectWarps; ++k) {
    if (k == warp) g0 = gall, e0 = eall;
    gall += s.warp_gt[k];
    eall += s.warp_eq[k];
  }
  if (cluster > 1) {
    if (tid == 0) {
      s.cta_gt = gall;
      s.cta_eq = eall;
    }
    __syncwarp();
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      g0 += ld_cluster(&s.cta_gt, r);
      e0 += ld_cluster(&s.cta_eq, r);
    }
  }
  const uint32_t below = (1u << lane) - 1;
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const uint32_t k = in ? key_at(i + lane) : 0;
    const uint32_t bg = __ballot_sync(0xFFFFFFFFu, in && k > prefix);
    const uint32_t be = __ballot_sync(0xFFFFFFFFu, in && k == prefix);
    const uint32_t e = e0 + __popc(be & below), g = g0 + __popc(bg & below);
    if (in && (k > prefix || (k == prefix && e < left))) keep(p.first + (int)(g + min(e, left)), t0 + i + lane);
    g0 += __popc(bg);
    e0 += __popc(be);
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
    return cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCap * 4);
  });
  if (e != cudaSuccess) return e;
  // as many CTAs per pair as its keys need to fit shared memory, and more while
  // SMs would stay empty and a CTA keeps 2048 tokens or more
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
  e = cudaLaunchKernelEx(&cfg, select_kernel, p, cluster);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((p.page_heads + kPackWarps - 1) / kPackWarps));
  cfg.blockDim = dim3(kPackWarps * 32);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, pack_kernel, p);
}

}  // namespace nvfp4kv
