// page_digest.cu -- bounds of every page's keys (nvfp4kv_page_digest), and from
// them an upper bound of every page's scores (nvfp4kv_page_scores), so that a
// decode can leave out the pages that cannot matter much to it.
//
// With hi_d and lo_d the largest and smallest of the keys' dimension d in a page,
// each token's score obeys
//   q . k = sum_d q_d k_d <= sum_d max(q_d hi_d, q_d lo_d) = q+ . hi + q- . lo
// (q+ = max(q, 0), q- = min(q, 0)): one product of twice the length.  A digest
// keeps hi and lo in E4M3, rounded outwards so that the bound holds, times one
// power of two per page-head that puts the largest into [128, 256).
//
// Both kernels cut the flattened list of their items evenly, over all warps (digests)
// or blocks (scores).
#include <climits>

#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kDgThreads = 256;
constexpr int kDgWarps = kDgThreads / 32;
constexpr int kDigestCtasPerSm = 4, kScoreCtasPerSm = 2;  // the grids are what fits at once
constexpr uint32_t kAll = 0xFFFFFFFFu;

constexpr int kOffScale = 2 * kHeadDim;  // behind hi and lo
constexpr int kDigestBytes = NVFP4KV_DIGEST_BYTES;
static_assert(kDigestBytes == kOffScale + 16, "a digest's tail keeps the next one 16-byte aligned");

// A sequence's tokens, cut to what the page table covers (flagged on request).
__device__ __forceinline__ int seq_tokens(const DigestArgs& p, int b, bool flag) {
  int L = p.seq_lens[b];
  const int lmax = p.max_pages * kPage;
  if (L < 0 || L > lmax) {
    if (flag) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    L = L < 0 ? 0 : lmax;
  }
  return L;
}

// Where a share [begin, end) of the flattened items starts: in sequence b,
// whose first item is `first`.
struct Share {
  int begin, end;
  int b, first;
};

struct ShareShared {
  int sums[kDgWarps + 1];
  int begin[kDgWarps + 1];  // the block's shares
  int b[kDgWarps], first[kDgWarps];
};

// The block's share number `mine`, of `shares`; items of sequence b: count(b).  Every
// thread of the block's kThreads calls this.
template <int kThreads, class Count>
__device__ __forceinline__ Share split(ShareShared& s, int batch, int shares, int mine, Count count) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // one pass over the sequences for the total, and (again, unless they were few
  // enough to stay in a register) one to find the shares' starts
  int kept = 0, local = 0;
  for (int b = tid; b < batch; b += kThreads) local += kept = count(b);
  int sum = __reduce_add_sync(kAll, local);
  if (lane == 0) s.sums[warp] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) total += s.sums[w];
  if (tid <= shares)
    s.begin[tid] = (int)(total * ((long long)blockIdx.x * shares + tid) / ((long long)gridDim.x * shares));
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const int b = base + tid;
    const int n = batch <= kThreads ? kept : b < batch ? count(b) : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) s.sums[warp] = incl;
    __syncthreads();
    int first = carry + incl - n, all = carry;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) first += s.sums[w];
      all += s.sums[w];
    }
    if (n > 0) {
      for (int w = 0; w < shares; ++w) {
        const int at = s.begin[w];
        if (at >= first && at - first < n) {
          s.b[w] = b;
          s.first[w] = first;
        }
      }
    }
    carry = all;
    __syncthreads();
  }
  Share r;
  r.begin = s.begin[mine];
  r.end = s.begin[mine + 1];
  r.b = s.b[mine];
  r.first = s.first[mine];
  return r;
}

// ---------------------------------------------------------------------------
// digests
// ---------------------------------------------------------------------------

union H2 {
  uint32_t u;
  __half2 h;
};
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  H2 x, y, r;
  x.u = a, y.u = b;
  r.h = __hmax2(x.h, y.h);
  return r.u;
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
  H2 x, y, r;
  x.u = a, y.u = b;
  r.h = __hmin2(x.h, y.h);
  return r.u;
}
// a * (the low or the high half of s, in both halves): the broadcast is left to the
// multiply's operand selection
template <bool kHi>
__device__ __forceinline__ uint32_t hmul2_bcast(uint32_t a, uint32_t s) {
  H2 x, y, r;
  x.u = a, y.u = s;
  r.h = __hmul2(x.h, kHi ? __high2half2(y.h) : __low2half2(y.h));
  return r.u;
}
__device__ __forceinline__ uint32_t hneg2(uint32_t a) { return a ^ 0x80008000u; }
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// A warp's ring: page-heads' keys and scales as stored, 1152 bytes a stage.
constexpr int kDgStages = 3;
constexpr int kDgStageBytes = kPageDataBytes + kPageScaleBytes;
static_assert(kOffKScale == kPageDataBytes, "the keys' scales follow the keys");

// Starts the copy of a page-head's keys and scales (nothing if it is not there) into a
// stage; both addresses are the lane's, 16 bytes from one lane to the next.
__device__ __forceinline__ void fetch_keys(uint32_t stage, const uint8_t* src, bool there, int lane) {
  if (there) {
    asm volatile(
        "{\n .reg .pred p;\n"
        " setp.lt.u32 p, %2, 8;\n"
        " cp.async.cg.shared.global [%0], [%1], 16;\n"
        " cp.async.cg.shared.global [%0+512], [%1+512], 16;\n"
        " @p cp.async.cg.shared.global [%0+1024], [%1+1024], 16;\n"
        "}\n" ::"r"(stage), "l"(src), "r"((uint32_t)lane)
        : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// v (below 256 in size) rounded up to an E4M3 value: to a whole number of its
// binade's steps, 2^-9 below 2^-6.
__device__ __forceinline__ float up_to_step(float v) {
  const uint32_t ex = max(__float_as_uint(v) >> 23 & 0xFFu, 127u - 6u);
  const float step = __uint_as_float((ex - 3u) << 23), steps = __uint_as_float((254u + 3u - ex) << 23);
  return ceilf(v * steps) * step;
}

// A page-head's digest from a warp's keys.  Every value e2m1 * e4m3 has at most six
// significant bits and is 0 or at least 2^-10 in size: exact in f16.  The lanes of
// the odd rows hold all values negated (their scales' signs are flipped), so that
// after one exchange the even ones hold hi, the odd ones -lo, and both round up.
// A lane has dimensions 8 dg .. 8 dg + 7 of every other row; kFull: the page is (else
// rows past its `valid` ones read row 0 instead, which changes no bound).
template <bool kFull>
__device__ __forceinline__ void write_digest(const uint8_t* keys, int valid, uint8_t* d, int lane) {
  const int dg = lane & 15, rh = lane >> 4;
  const uint8_t* const data = keys + 4 * dg;
  const uint8_t* const scales = keys + kOffKScale + (dg >> 1);
  auto row_at = [&](int r) { return kFull || 2 * r + rh < valid ? 2 * r + rh : 0; };
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    // the scales of rows r and r + 1 together
    const uint32_t sc = e4m3x2_to_f16x2(scales[row_at(r & 6) * kRowScales] +
                                        scales[row_at((r & 6) + 1) * kRowScales] * 0x100u + (rh ? 0x8080u : 0u));
    const uint32_t k = *reinterpret_cast<const uint32_t*>(data + row_at(r) * kRowBytes);
    auto scaled = [&](uint32_t v) { return (r & 1) ? hmul2_bcast<true>(v, sc) : hmul2_bcast<false>(v, sc); };
    const uint32_t v[4] = {scaled(e2m1x2_to_f16x2<0>(k)), scaled(e2m1x2_to_f16x2<1>(k)),
                           scaled(e2m1x2_to_f16x2<2>(k)), scaled(e2m1x2_to_f16x2<3>(k))};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = r == 0 ? v[j] : hmax2(hi[j], v[j]);
      lo[j] = r == 0 ? v[j] : hmin2(lo[j], v[j]);
    }
  }
  uint32_t x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = hmax2(hi[j], hneg2(__shfl_xor_sync(kAll, lo[j], 16)));
  // the largest of them all is max(|hi|, |lo|) >= 0 (negative zeros count as below 0)
  const uint32_t t2 = hmax2(hmax2(x[0], x[1]), hmax2(x[2], x[3]));
  const int most = __reduce_max_sync(kAll, max((int)(int16_t)(t2 & 0xFFFFu), (int)t2 >> 16));
  // 2^e with most / 2^e in [128, 256), from f16's exponent field (a normal number)
  const int field = most > 0 ? most >> 10 : 15 + 7;
  const int down = 15 + 7 - field;  // -e, in [-4, 17]: one or two factors that f16 holds
  const int first = min(down, 15), second = down - first;
  const uint32_t f1 = (uint32_t)(15 + first) << 10, f2 = (uint32_t)(15 + second) << 10;
  uint32_t code[4];
  uint32_t small = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t t = hfma2(hmul2(x[j], f1 | f1 << 16), f2 | f2 << 16, 0u);  // + 0: no negative zeros
    H2 u, lim;
    u.u = t;
    lim.u = 0x24002400u;  // 2^-6
    small |= __hlt2_mask(__habs2(u.h), lim.h) & t;  // 0 < |t| < 2^-6: steps that are coarser than the binade's
    // E4M3 drops seven of f16's ten mantissa bits; a negative value's magnitude is cut off
    uint32_t negative;  // each half all ones where its sign is set (prmt copying bytes 1 and 3's signs)
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(negative) : "r"(t));
    const uint32_t up = (t + (0x007F007Fu & ~negative)) & 0xFF80FF80u;
    code[j] = e4m3x2_from_f16x2(hfma2(up, rh ? 0xBC00BC00u : 0x3C003C00u, 0u));  // times the lane's sign
    x[j] = t;
  }
  if (__any_sync(kAll, small != 0)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      H2 u;
      u.u = x[j];
      const float a = up_to_step(__low2float(u.h)), b = up_to_step(__high2float(u.h));
      code[j] = e4m3x2_from_f32((rh ? -a : a) + 0.0f, (rh ? -b : b) + 0.0f);
    }
  }
  reinterpret_cast<uint2*>(d)[lane] = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
  if (lane == 0)
    *reinterpret_cast<uint4*>(d + kOffScale) = make_uint4((uint32_t)(127 - down) << 23, 0u, 0u, 0u);  // 2^e; 1 without any
}

// A warp takes one page-head at a time; the keys of the next kDgStages - 1 are on
// their way meanwhile.  1152 bytes in (whole lines) and 272 out per page-head.  Bound by
// the integer pipe (76 % busy), which converts the codes and takes the bounds: 28.8
// thousand pages of 8 heads 76 us, 4.3 TB/s (without the ring 99; with each item's
// address worked out from its head and page 82); 32 pages 3.1.
__global__ void __launch_bounds__(kDgThreads, kDigestCtasPerSm) digest_kernel(const DigestArgs p) {
  __shared__ ShareShared s;
  __shared__ __align__(128) uint8_t rings[kDgWarps][kDgStages * kDgStageBytes];
  const int lane = threadIdx.x & 31;
  after_earlier_kernels();
  auto from_page = [&](int b) { return p.first_tokens ? max(p.first_tokens[b], 0) / kPage : 0; };
  const Share w = split<kDgThreads>(s, p.batch, kDgWarps, (int)(threadIdx.x >> 5), [&](int b) {
    const int L = seq_tokens(p, b, blockIdx.x == 0);
    return max((L + kPage - 1) / kPage - from_page(b), 0) * p.hkv;
  });
  if (w.begin >= w.end) return;
  // the next item to fetch: a head of page `page` of sequence b, which has `end` pages
  int b = w.b, L = seq_tokens(p, b, false), page = from_page(b), end = (L + kPage - 1) / kPage;
  const int i = w.begin - w.first;
  page += i / p.hkv - 1;
  int heads = 0, skip = i % p.hkv;  // heads left of the page; heads of the first page that are another warp's
  int row = 0, valid = 0;           // its row of the pool (below 0: the page is not there), its tokens
  const uint8_t* src = nullptr;
  int left = w.end - w.begin;
  const uint8_t* const ring = rings[threadIdx.x >> 5];
  const uint32_t ring_u32 = smem_u32(ring) + 16 * lane;
  // starts the next item's copy; returns its row of the pool (below 0 for none) and its valid tokens
  auto fetch = [&](int stage) -> int2 {
    if (left == 0) {
      fetch_keys(0, nullptr, false, lane);
      return make_int2(-1, 0);
    }
    --left;
    if (heads == 0) {
      ++page;
      while (page >= end) {  // the next sequence that has any
        ++b;
        L = seq_tokens(p, b, false);
        page = from_page(b);
        end = (L + kPage - 1) / kPage;
      }
      const int id = p.page_table[(long long)b * p.max_pages + page];
      const bool there = id >= 0 && id < p.num_pages;
      if (!there && lane == 0) flag_error(p.status, NVFP4KV_DEVERR_PAGE);
      heads = p.hkv - skip;
      row = there ? id * p.hkv + skip : INT_MIN;
      src = p.pages + (long long)max(row, 0) * kPageHeadBytes + 16 * lane;
      valid = min(L - page * kPage, kPage);
      skip = 0;
    }
    fetch_keys(ring_u32 + stage * kDgStageBytes, src, row >= 0, lane);
    const int2 r = make_int2(row, valid);
    --heads;
    ++row;
    src += kPageHeadBytes;
    return r;
  };
  static_assert(kDgStages == 3, "waits for all but the two latest copies");
  int2 item[kDgStages];
  item[0] = fetch(0);
  item[1] = fetch(1);
  int to_do = w.end - w.begin;
  while (true) {
#pragma unroll
    for (int stage = 0; stage < kDgStages; ++stage) {
      item[(stage + 2) % kDgStages] = fetch((stage + 2) % kDgStages);
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      __syncwarp();
      if (item[stage].x >= 0) {
        uint8_t* const d = p.digest + (long long)item[stage].x * kDigestBytes;
        const uint8_t* const keys = ring + stage * kDgStageBytes;
        if (item[stage].y == kPage)
          write_digest<true>(keys, kPage, d, lane);
        else
          write_digest<false>(keys, item[stage].y, d, lane);
      }
      __syncwarp();  // the stage may be filled again
      if (--to_do == 0) break;
    }
    if (to_do == 0) break;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------------------
// scores
// ---------------------------------------------------------------------------

constexpr int kTile = 16;  // pages of one KV head per step: the rows of an MMA

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The queries of a pair as B fragments, and the powers of two that their heads' products
// are multiplied with.  Lane (g, t) holds head g's dimensions 16 t .. 16 t + 15 and
// 64 + 16 t ..: the order in which a digest's 16-byte pieces bring them.
struct Queries {
  uint32_t pos[8][2], neg[8][2];
  float down0, down1;  // heads 2 t, 2 t + 1
};

__device__ __forceinline__ void load_queries(const ScoreArgs& p, int pair, int lane, Queries& q) {
  const int g = lane >> 2, t = lane & 3;
  float v[32];
  if (g < p.group) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + ((long long)pair * p.group + g) * kHeadDim);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 w = src[8 * (j >> 1) + 2 * t + (j & 1)];
      v[8 * j + 0] = bf16_to_f32(w.x & 0xFFFFu); v[8 * j + 1] = bf16_to_f32(w.x >> 16);
      v[8 * j + 2] = bf16_to_f32(w.y & 0xFFFFu); v[8 * j + 3] = bf16_to_f32(w.y >> 16);
      v[8 * j + 4] = bf16_to_f32(w.z & 0xFFFFu); v[8 * j + 5] = bf16_to_f32(w.z >> 16);
      v[8 * j + 6] = bf16_to_f32(w.w & 0xFFFFu); v[8 * j + 7] = bf16_to_f32(w.w >> 16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
  }
  // times a power of two that puts the head's largest into [2^14, 2^15), so that
  // f16 holds them (as in the decode); the products stay below 2^31
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(v[j]));
  amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
  const F16Range r = f16_range(amax);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = v[4 * i] * r.up, b = v[4 * i + 1] * r.up, c = v[4 * i + 2] * r.up, d = v[4 * i + 3] * r.up;
    q.pos[i][0] = pack_f16x2(fmaxf(a, 0.0f), fmaxf(b, 0.0f));
    q.pos[i][1] = pack_f16x2(fmaxf(c, 0.0f), fmaxf(d, 0.0f));
    q.neg[i][0] = pack_f16x2(fminf(a, 0.0f), fminf(b, 0.0f));
    q.neg[i][1] = pack_f16x2(fminf(c, 0.0f), fminf(d, 0.0f));
  }
  q.down0 = __shfl_sync(kAll, r.down, 8 * t);
  q.down1 = __shfl_sync(kAll, r.down, 8 * t + 4);
}

// How a block goes through a sequence's pages: `together` KV heads at once, one per
// warp, of `streams` tiles of 16 consecutive pages, in `rounds` over all heads.  A
// page's digests of those heads are one run of memory, copied as such to every
// `stride` bytes of a stage (64 more than a multiple of 128: the 16-byte reads of eight
// lanes, two pages' 64 bytes each, then meet no bank twice).
struct ScorePlan {
  int together, streams, rounds, pages, stride;
};

__host__ __device__ inline ScorePlan score_plan(int hkv) {
  ScorePlan k;
  k.together = hkv < kDgWarps ? hkv : kDgWarps;
  k.streams = kDgWarps / k.together;
  k.rounds = (hkv + k.together - 1) / k.together;
  k.pages = kTile * k.streams;
  k.stride = (k.together * kDigestBytes + 63) / 128 * 128 + 64;
  return k;
}

constexpr int kUnit = 8;  // shares are cut at multiples of so many pages: whole sectors of scores and ids
constexpr int kScStages = 2;
// the most that score_plan asks for: one head, 128 pages of 320 bytes
constexpr int kScStageBytes = 128 * 320;

// A block takes an equal share of all pages, in items of up to 16 to 128 consecutive ones
// of one sequence and up to eight KV heads; a warp (but the last) one of the heads and 16
// of the pages, the rows of an MMA whose eight columns are the query heads.  Lane (g, t)
// reads 16-byte pieces t and 4 + t of hi and of lo of pages g and g + 8.  The last warp
// starts the copies, one per page (2176 bytes with eight heads), into a stage as soon as the
// others have left it.  28.8 thousand pages of 8 heads 15.3 us (15.9 with a barrier of all warps
// per item, 19.8 so with items of half the pages; some 18 with each row fetched by
// itself), 16.4 thousand 10.4 (10.7 with shares of whole items): some 5 us for the launch,
// the shares and the first page, then the pages at 6 TB/s.
constexpr int kScThreads = kDgThreads + 32;

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__global__ void __launch_bounds__(kScThreads, kScoreCtasPerSm) scores_kernel(const ScoreArgs p) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ ShareShared s;
  __shared__ __align__(8) uint64_t bars[2 * kScStages];
  __shared__ uint32_t s_there[kScStages][4];  // a stage's pages that are there, bit by bit
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const DigestArgs& d = p.d;
  const ScorePlan k = score_plan(d.hkv);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kScStages, st0 = smem_u32(stages);
  if (tid == 0) {
    for (int i = 0; i < kScStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, kDgWarps);
    }
    fence_mbar_init();
  }
  after_earlier_kernels();
  auto pages_of = [&](int b, bool flag) {
    int n = (seq_tokens(d, b, flag) + kPage - 1) / kPage;
    if (n > p.score_stride) {
      if (flag) flag_error(d.status, NVFP4KV_DEVERR_LENGTH);
      n = (int)p.score_stride;
    }
    return n;
  };
  auto units_of = [&](int pages) { return (pages + kUnit - 1) / kUnit; };
  const Share w =
      split<kScThreads>(s, d.batch, 1, 0, [&](int b) { return units_of(pages_of(b, blockIdx.x == 0)) * k.rounds; });
  if (w.begin >= w.end) return;
  // a walk over the share: from page `page` of the `pages` of sequence b, heads from together *
  // round on, `left` units to go
  struct Walk {
    int b, round, page, pages, left;
  };
  auto item_pages = [&](const Walk& x) { return min(min(k.pages, x.pages - x.page), x.left * kUnit); };
  auto advance = [&](Walk& x) {
    const int n = item_pages(x);
    x.page += n;
    x.left -= units_of(n);
    if (x.left == 0 || x.page < x.pages) return;
    x.page = 0;
    if (++x.round < k.rounds) return;
    x.round = 0;
    do {  // the next sequence that has any
      if (++x.b >= d.batch) {
        x.left = 0;
        return;
      }
      x.pages = pages_of(x.b, false);
    } while (x.pages == 0);
  };
  Walk at;
  at.b = w.b;
  at.pages = pages_of(w.b, false);
  at.round = (w.begin - w.first) / units_of(at.pages);
  at.page = (w.begin - w.first - at.round * units_of(at.pages)) * kUnit;
  at.left = w.end - w.begin;

  if (warp == kDgWarps) {
    // the copies: lane = page of the item modulo 32; the ids of an item are read while the one before it is copied
    constexpr int kMost = 128 / 32;
    int ids[kMost];
    auto read_ids = [&](const Walk& x) {
      const int item = item_pages(x);
#pragma unroll
      for (int c = 0; c < kMost; ++c) {
        const int in = 32 * c + lane;
        ids[c] = -1;
        if (in < item) {
          ids[c] = d.page_table[(long long)x.b * d.max_pages + x.page + in];
          if (ids[c] < 0 || ids[c] >= d.num_pages) {
            flag_error(d.status, NVFP4KV_DEVERR_PAGE);
            ids[c] = -1;
          }
        }
      }
    };
    read_ids(at);
    for (int n = 0; at.left > 0; ++n) {
      const int stage = n % kScStages, head = at.round * k.together;
      const uint32_t bytes = (uint32_t)(min(k.together, d.hkv - head) * kDigestBytes);
      int now[kMost];
      uint32_t there[kMost], count = 0;
#pragma unroll
      for (int c = 0; c < kMost; ++c) {
        now[c] = ids[c];
        there[c] = __ballot_sync(kAll, ids[c] >= 0);
        count += __popc(there[c]);
      }
      advance(at);
      read_ids(at);
      if (n >= kScStages && !mbar_wait(empty + 8 * stage, (uint32_t)(n / kScStages - 1) & 1u) && lane == 0)
        flag_error(d.status, kDevErrTimeout);
      if (lane == 0) {
#pragma unroll
        for (int c = 0; c < kMost; ++c) s_there[stage][c] = there[c];
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full + 8 * stage), "r"(bytes * count)
                     : "memory");
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < kMost; ++c) {
        if (now[c] < 0) continue;
        const uint8_t* src = d.digest + ((long long)now[c] * d.hkv + head) * kDigestBytes;
        asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         st0 + stage * kScStageBytes + (32 * c + lane) * k.stride),
                     "l"(src), "r"(bytes), "r"(full + 8 * stage)
                     : "memory");
      }
    }
    return;
  }

  const int stream = warp / k.together, mine = warp - stream * k.together;
  Queries q;
  int loaded = -1;
  for (int n = 0; at.left > 0; ++n) {
    const int stage = n % kScStages, head = at.round * k.together + mine, pair = at.b * d.hkv + head;
    const int mine_pages = item_pages(at) - stream * kTile;  // of the item, from the warp's first on
    const bool live = stream < k.streams && head < d.hkv && mine_pages > 0;
    if (live && pair != loaded) {
      load_queries(p, pair, lane, q);
      loaded = pair;
    }
    // (a wait that gives up: the outputs are not valid, every access stays in bounds)
    if (!mbar_wait(full + 8 * stage, (uint32_t)(n / kScStages) & 1u) && lane == 0) flag_error(d.status, kDevErrTimeout);
    if (live) {
      const uint32_t there = s_there[stage][stream >> 1] >> (kTile * (stream & 1));
      const uint8_t* const rows = stages + stage * kScStageBytes + stream * kTile * k.stride + mine * kDigestBytes;
      const uint8_t* const r0 = rows + g * k.stride + 16 * t;
      const uint8_t* const r1 = r0 + 8 * k.stride;
      float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 x0 = *reinterpret_cast<const uint4*>(r0 + 64 * j), x1 = *reinterpret_cast<const uint4*>(r1 + 64 * j);
        const uint32_t a[4] = {x0.x, x0.y, x0.z, x0.w}, e[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t* f = (j & 2) ? q.neg[4 * (j & 1) + m] : q.pos[4 * (j & 1) + m];
          mma16816(c, e4m3x2_to_f16x2(a[m] & 0xFFFFu), e4m3x2_to_f16x2(e[m] & 0xFFFFu), e4m3x2_to_f16x2(a[m] >> 16),
                   e4m3x2_to_f16x2(e[m] >> 16), f[0], f[1]);
        }
      }
      const float u0 = *reinterpret_cast<const float*>(rows + g * k.stride + kOffScale);
      const float u1 = *reinterpret_cast<const float*>(rows + (g + 8) * k.stride + kOffScale);
      __syncwarp();
      if (lane == 0) arrive(empty + 8 * stage);
      // A sum times its page's unit, the scale, and its head's power of two, in this order: sums in
      // units lie within 2^-50 .. 2^36, so that no step leaves fp32's normal numbers before the score does.
      // The largest over the group's heads, 2 t and 2 t + 1 in this lane.
      const bool first = 2 * t < p.group, second = 2 * t + 1 < p.group;
      const float c00 = first ? c[0] * u0 * p.score_scale * q.down0 : -INFINITY;
      const float c01 = second ? c[1] * u0 * p.score_scale * q.down1 : -INFINITY;
      const float c10 = first ? c[2] * u1 * p.score_scale * q.down0 : -INFINITY;
      const float c11 = second ? c[3] * u1 * p.score_scale * q.down1 : -INFINITY;
      float m0 = fmaxf(c00, c01), m1 = fmaxf(c10, c11);
#pragma unroll
      for (int off = 1; off < 4; off <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(kAll, m0, off));
        m1 = fmaxf(m1, __shfl_xor_sync(kAll, m1, off));
      }
      const int r = g + 8 * t;  // lanes t = 0 and 1 write pages g and g + 8
      if (t < 2 && r < mine_pages)
        p.scores[(long long)pair * p.score_stride + at.page + stream * kTile + r] = (there >> r & 1) ? (t ? m1 : m0) : -INFINITY;
    } else if (lane == 0) {
      arrive(empty + 8 * stage);
    }
    advance(at);
  }
}

}  // namespace

cudaError_t launch_page_digest(const DigestArgs& args, int num_sms, cudaStream_t stream) {
  const int64_t need = ((int64_t)args.batch * args.max_pages * args.hkv + kDgWarps - 1) / kDgWarps;
  const int64_t fit = (int64_t)num_sms * kDigestCtasPerSm;
  return launch_overlapped(digest_kernel, need < fit ? need : fit, kDgThreads, 0, 1, stream, args);
}

cudaError_t launch_page_scores(const ScoreArgs& args, int num_sms, cudaStream_t stream) {
  static PerDeviceOnce attr_once;
  const cudaError_t e = attr_once.run([] {
    return cudaFuncSetAttribute(scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kScStages * kScStageBytes);
  });
  if (e != cudaSuccess) return e;
  const ScorePlan k = score_plan(args.d.hkv);
  const int64_t items = args.d.batch * (((int64_t)args.d.max_pages + k.pages - 1) / k.pages) * k.rounds;
  const int64_t fit = (int64_t)num_sms * kScoreCtasPerSm;
  return launch_overlapped(scores_kernel, items < fit ? items : fit, kScThreads, kScStages * kScStageBytes, 1, stream,
                           args);
}

}  // namespace nvfp4kv
