// decode_attention.cu -- paged GQA decode attention over the NVFP4 cache with
// the dequantisation inside the kernel ("nvfp4-kv-cache-memory-wall", section
// 3, item 3: decode dequantises in registers with no separate pass, because
// decode is bound by the KV read; a round trip through memory would read and
// write the whole cache once more).
//
// Work partition (split-K, balanced): the flattened list of (sequence, KV
// head, page) items -- "page-heads" -- is cut into gridDim.x contiguous ranges
// whose sizes differ by at most one, one per CTA, and each CTA range into kNW
// such ranges, one per warp.
// A warp streams its pages through a private ring of kStages shared-memory
// stages.  A page-head is 2304 contiguous bytes of the pool (K data, K scales,
// V data, V scales); all 32 lanes copy it into a stage as it is, in 16-byte
// cp.async pieces, completion counted on one mbarrier per stage.  For each
// page it
//   1. converts K's E2M1 pairs to f16x2 with cvt.rn.f16x2.e2m1x2, multiplies
//      by the E4M3 block scale (exact in f16), and computes S^T = Khat q^T for
//      the 16 tokens x G query heads with mma.sync m16n8k16 (f16 in, f32 acc);
//      two pages of the same pair are taken per step (32 tokens);
//   2. runs the online softmax in base 2 (scores scaled by softmax_scale *
//      log2(e) * g_K, folded into one FMA per score); the running max is only
//      raised when a score exceeds it by more than 8, so the rescale of the
//      accumulators is rare;
//   3. transposes P (f16) with movmatrix and accumulates O^T += Vhat^T P^T,
//      Vhat^T converted straight from V's token-pair bytes (each byte one
//      dimension of two tokens) and scaled per token.
// A (sequence, KV head) pair that lies inside one warp range is finished by
// that warp.  A piece of a pair cut by a warp boundary is written to the
// workspace as a record (unnormalised O, running max m, sum l) and the warp
// is done: no CTA-wide barrier or merge sits at the end of the decode, where
// it would wait on the slowest warp and run cold code under full memory load.
// combine_kernel, launched right behind the decode as a programmatic
// dependent, merges each cut pair's records (the flash-decoding combine); it
// finds them from the split itself, which it rederives from the lengths while
// the decode still runs.
//
// The scored decode (template argument M, 0 for the plain one) is the same two
// kernels with the scores of step 2 capped (tanh on the FMA pipe, two scores per
// instruction) and biased before the maximum, bf16 outputs and the log-sum-exp.
// Decode kernel of 32 x 8193 tokens, 64 / 8 heads: 56.1 us, biased 60.1, capped
// 60.3.  A window changes only which pages are items: those of the sinks and of
// the window, so it costs what it reads (14.7 us under one of 1024).
// With accumulated weights the scores are also written out (fp32, 512 bytes per
// 2304-byte page-head) for weights_kernel, which adds every token's weight to
// its running sum once the log-sum-exps are there: 65.6 us and 16.5 us for the
// weights.  Writing and reading them moves 1024 bytes per page-head; working the
// scores out again would read K's 1152 and repeat the products.
//
// Exactness: e2m1 * E4M3 has at most 6 significant bits in [2^-10, 2688], so
// Khat and Vhat are exact in f16.  q is bf16; it is multiplied by a power of
// two per head so its largest element sits in [2^14, 2^15) before rounding to
// f16, and the factor is folded back into the score scale.
#include <cfloat>
#include <cstdint>

#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"
#include "scoring.cuh"

namespace nvfp4kv {
namespace {

#ifndef NVFP4KV_DECODE_WARPS
#define NVFP4KV_DECODE_WARPS 4
#endif
#ifndef NVFP4KV_DECODE_STAGES
#define NVFP4KV_DECODE_STAGES 4
#endif
#ifndef NVFP4KV_DECODE_CTAS_PER_SM
#define NVFP4KV_DECODE_CTAS_PER_SM 3
#endif
#ifndef NVFP4KV_DECODE_QK_CHAINS
#define NVFP4KV_DECODE_QK_CHAINS 1  // independent QK accumulator chains per page (1 or 2)
#endif
constexpr int kNW = NVFP4KV_DECODE_WARPS;              // warps per CTA (each streams its own pages)
constexpr int kStages = NVFP4KV_DECODE_STAGES;         // ring stages per warp (2 pages in compute)
constexpr int kCtasPerSm = NVFP4KV_DECODE_CTAS_PER_SM; // resident CTAs per SM the launch is sized for
constexpr int kGMax = 8;        // query heads per KV head (one MMA n-tile)
constexpr float kLazy = 8.0f;   // running-max slack (log2 units): P <= 2^8 in f16

// Cache formats the decode reads: NVFP4; NVFP4 of Hadamard-rotated rows (q is
// rotated on the way in and the output rotated back, both exact orthonormal
// transforms); MXFP4 (blocks of 32 with E8M0 scales, 4 per row).
enum : int { kFmtNvfp4 = 0, kFmtHadamard = 1, kFmtMxfp4 = 2 };

// Scored decode (nvfp4kv_decode_attention_scored / _weights): bit flags of the
// kernels' second template argument; 0 is the plain decode.
enum : int {
  kScored = 1,   // bf16 output, log-sum-exp, a window with sinks (both run-time: they touch no inner loop)
  kCapped = 2,   // scores through cap * tanh(s / cap)
  kBiased = 4,   // minus slope * distance
  kStored = 8,   // the scores of every visited token are kept for weights_kernel
  kSelected = 16 // only the pages that a list names are items (nvfp4kv_decode_attention_selected)
};

// stage layout: the page-head as stored (K data | K scales | V data | V scales)
constexpr int kOffKD = kOffKData;
__host__ __device__ constexpr int ph_bytes(int F) { return F == kFmtMxfp4 ? kMxPageHeadBytes : kPageHeadBytes; }
__host__ __device__ constexpr int off_vd(int F) { return F == kFmtMxfp4 ? kMxOffVData : kOffVData; }
__host__ __device__ constexpr int off_ks(int F) { return F == kFmtMxfp4 ? kMxOffKScale : kOffKScale; }
__host__ __device__ constexpr int off_vs(int F) { return F == kFmtMxfp4 ? kMxOffVScale : kOffVScale; }
constexpr int kStageBytes = kPageHeadBytes;  // stage stride: the larger page-head (2304)

// a (partial) result record: O[kGMax][128] unnormalised, m[kGMax] (base 2), l[kGMax]
constexpr int kRecFloats = kGMax * kHeadDim + 2 * kGMax;
constexpr int kOffM = kGMax * kHeadDim;
constexpr int kOffL = kGMax * kHeadDim + kGMax;

constexpr int kRingBytes = kNW * kStages * kStageBytes;
constexpr int kBarBytes = kNW * kStages * 8;
constexpr int kSmemBytes = kRingBytes + kBarBytes;

struct DecodeParams {
  const uint8_t* pages;  // [num_pages][hkv][kPageHeadBytes]
  int32_t num_pages;
  int32_t hkv;
  const uint16_t* q;
  float* out;
  const int32_t* page_table;
  int32_t max_pages;
  const int32_t* seq_lens;
  int32_t batch;
  int32_t hq;
  int32_t group;
  float score_scale;  // softmax_scale * log2(e) * g_K
  float v_gscale;     // g_V
  float* part;        // [2 * num_ctas * kNW] records: warp w's first (2w) and last (2w + 1) cut piece
  int32_t* status;
  int32_t* cu_pages;  // [batch + 1], written by CTA 0: pages of the sequences before each, then of all
  int32_t ncta;       // CTAs of the decode grid (its split, rederived by the combine)
  int32_t comb_heads; // query heads per combine block
  // scored decode only
  float cap_scale;       // kCapped: softmax_scale * g_K / cap (score_scale is then cap * log2(e))
  int32_t window;        // a query sees the last `window` tokens (0: all of them)
  int32_t sinks;         // and the first `sinks`
  const float* slopes;   // [hq], kBiased
  uint16_t* out16;       // bf16 output
  float* lse;            // natural log-sum-exp [batch][hq], or null
  float* lse2;           // kStored: base-2 log-sum-exp [batch][hq]
  float* scores;         // kStored: base-2 scores [items][16 tokens][score_heads]
  int32_t score_heads;   // 2, 4 or 8: the group rounded up
  long long score_items; // page-heads that `scores` has room for
  float* weights;        // [batch][hkv][weight_stride]
  long long weight_stride;
  float decay;
  const int32_t* selected;  // kSelected: [batch][hkv][budget] pages of the sequence, below 0 for none
  int32_t budget;
};

// ---------------------------------------------------------------------------
// small helpers
// ---------------------------------------------------------------------------

// (kFresh: from a kernel that overlaps the one ahead of it; see after_earlier_kernels)
template <bool kFresh = false>
__device__ __forceinline__ int clamp_len(const DecodeParams& p, int b) {
  int L = kFresh ? p.seq_lens[b] : __ldg(p.seq_lens + b);
  const int lmax = p.max_pages * kPage;
  if (L < 0 || L > lmax) {
    flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    L = L < 0 ? 0 : lmax;
  }
  return L;
}

// The pages of a sequence of L tokens that hold visible ones.  Without a
// window: all of them.  With one: the pages of the first `sinks` tokens and
// those from the window's first token on, the pages between left out (their
// page-table entries are not read).
struct VisiblePages {
  int count;   // pages visited
  int lead;    // the first `lead` of them are pages 0 .. lead - 1 ...
  int skip;    // ... and the others come this many pages later than their index
};

template <int M>
__device__ __forceinline__ VisiblePages visible_pages(const DecodeParams& p, int L) {
  VisiblePages v;
  v.count = (L + kPage - 1) / kPage;
  v.lead = v.count;
  v.skip = 0;
  if constexpr ((M & kSelected) != 0) {
    // as many items as the list has places for the sequence's pages
    v.lead = v.count = min(v.count, p.budget);
  } else if constexpr (M != 0) {
    if (p.window > 0 && L > p.window) {
      const int first = (L - p.window) / kPage;  // page of the window's first token
      v.lead = min(first, p.sinks / kPage + (p.sinks % kPage != 0));
      v.skip = first - v.lead;
      v.count -= v.skip;
    }
  }
  return v;
}

template <int M>
__device__ __forceinline__ int pages_of(const DecodeParams& p, int b) {
  return visible_pages<M>(p, clamp_len(p, b)).count;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero accumulator: d = a * b (the first MMA of a chain).
__device__ __forceinline__ void mma16816_zero(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t dup_lo(uint32_t h2) { return __byte_perm(h2, 0, 0x1010); }

// a * (the low or the high half of s, in both halves): the broadcast is left to
// the multiply's operand selection
union H2U {
  uint32_t u;
  __half2 h;
};
template <bool kHi>
__device__ __forceinline__ uint32_t hmul2_bcast(uint32_t a, uint32_t s) {
  H2U x, y, r;
  x.u = a;
  y.u = s;
  r.h = __hmul2(x.h, kHi ? __high2half2(y.h) : __low2half2(y.h));
  return r.u;
}

template <int K>
__device__ __forceinline__ uint32_t cvt_sel(uint32_t w) { return e2m1x2_to_f16x2<K>(w); }

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Balanced partition of W page-heads over N CTAs: the first W % N CTAs take
// W / N + 1, the rest W / N.  (Weighting CTAs by their launch order on an SM,
// whose warp scheduler favours older CTAs by about 5%, balanced the CTAs'
// finish times but did not shorten the launch: the slowest warps are spread
// over all SMs.)
__device__ __forceinline__ long long cta_start(long long c, long long W, long long N) {
  // W < 2^31 (checked on the host): 32-bit division
  const int q = (int)W / (int)N, rem = (int)W - q * (int)N;
  return c * q + (c < rem ? c : rem);
}

// Where each item of a 32-item chunk of a warp's range lives (one per lane).
struct ItemMap {
  int row;     // the page id as loaded; after resolve_chunk the physical row pid * hkv + h, or -1
  int h;       // KV head
  int pair;    // b * hkv + h, -1 past the warp's range
  int page;    // page index within the sequence
  int np;      // pages of the pair
  int lastnv;  // valid tokens in the pair's last page (1..16); kSelected: in this page (0: the list names none)
  int nv;      // after resolve_chunk: valid tokens of the item's page (0 for an invalid id or past the range)
  int hole;    // scored: rows [hole & 255, hole >> 8) of the page are out of sight (0: none)
  int dist;    // scored: the position of the page's first token minus the query's
};

// The sequence a chunk walk starts from: its index, its first page (in units
// of pages of all earlier sequences) and its clamped length.
struct SeqCursor {
  int b;
  int cu;
  int L;
};

// Map items [i0, i0 + 32) of the warp range starting at wr0 (n items) to pages
// and start the page-table loads; resolve_chunk turns the loaded ids into rows
// later, so the load latency is hidden behind the pages already staged.
// `sc` is a sequence whose first page-head is <= the chunk's first item; on
// return it is the sequence of the chunk's last valid item.
template <int M>
__device__ __forceinline__ ItemMap map_chunk(const DecodeParams& p, long long wr0, int i0, int n, SeqCursor& sc,
                                             int lane) {
  ItemMap m;
  m.row = -1;
  m.h = 0;
  m.pair = -1;
  m.page = 0;
  m.np = 1;
  m.lastnv = kPage;
  m.nv = 0;
  m.hole = 0;
  m.dist = 0;
  const int i = i0 + lane;
  int b = sc.b, cu = sc.cu, L = sc.L;
  if (i < n) {
    const long long r = wr0 + i;
    VisiblePages v = visible_pages<M>(p, L);
    while (r >= (long long)(cu + v.count) * p.hkv) {
      cu += v.count;
      ++b;
      L = clamp_len(p, b);
      v = visible_pages<M>(p, L);
    }
    const int np = v.count;
    const int local = (int)(r - (long long)cu * p.hkv);
    const int h = local / np;
    const int page = local - h * np;
    m.h = h;
    m.pair = b * p.hkv + h;
    m.page = page;
    m.np = np;
    m.lastnv = L - (np + v.skip - 1) * kPage;
    int at = page < v.lead ? page : page + v.skip;  // the page within the sequence
    if constexpr ((M & kSelected) != 0) {
      at = __ldg(p.selected + (long long)m.pair * p.budget + page);
      const bool named = at >= 0 && at < (L + kPage - 1) / kPage;
      if (at >= 0 && !named) flag_error(p.status, NVFP4KV_DEVERR_PAGE);
      at = named ? at : 0;
      m.lastnv = named ? min(L - at * kPage, kPage) : 0;
    } else if constexpr (M != 0) {
      const int t0 = at * kPage;
      m.dist = t0 - (L - 1);
      if (p.window > 0 && L > p.window) {
        const int lo = min(max(p.sinks - t0, 0), kPage), hi = min(max(L - p.window - t0, 0), kPage);
        if (lo < hi) m.hole = lo | (hi << 8);
      }
    }
    m.row = __ldg(p.page_table + (long long)b * p.max_pages + at);
  }
  const int last = min(31, n - 1 - i0);
  sc.b = __shfl_sync(0xFFFFFFFFu, b, last);
  sc.cu = __shfl_sync(0xFFFFFFFFu, cu, last);
  sc.L = __shfl_sync(0xFFFFFFFFu, L, last);
  return m;
}

// Turn the loaded page ids of a chunk map into physical rows (-1 for an id out
// of range, which is flagged); returns the valid-page bits (bit l: lane l).
template <int M>
__device__ __forceinline__ uint32_t resolve_chunk(const DecodeParams& p, ItemMap& m) {
  const bool real = m.pair >= 0 && ((M & kSelected) == 0 || m.lastnv > 0);
  const bool valid = real && m.row >= 0 && m.row < p.num_pages;
  if (real && !valid) flag_error(p.status, NVFP4KV_DEVERR_PAGE);
  m.row = valid ? m.row * p.hkv + m.h : -1;
  m.nv = valid ? ((M & kSelected) != 0 || m.page == m.np - 1 ? m.lastnv : kPage) : 0;
  return __ballot_sync(0xFFFFFFFFu, valid);
}

// cp.async staging: lane l copies the 16-byte pieces l, l + 32, ... of the
// page-head (NVFP4: lanes 0-15 five of the 144, the others four; MXFP4: lanes
// 0-7 five of the 136), then arrives (no-increment) on the stage's mbarrier,
// which expects 32 arrivals.  The lane's source base and shared-memory offset
// are set up once.
struct LaneCopy {
  const uint8_t* src;  // pages + 16 * lane
  uint32_t off;        // 16 * lane
  bool fifth;          // a fifth piece at 16 * (lane + 128)
  uint64_t policy;     // kStored: the L2 policy of the copies: first to go, so that more of the
                       // kept scores are still there for weights_kernel (19.0 -> 16.8 us)
};

template <int F>
__device__ __forceinline__ LaneCopy lane_copy(const DecodeParams& p, int lane) {
  LaneCopy c;
  c.src = p.pages + 16 * lane;
  c.off = 16u * lane;
  c.fifth = lane + 128 < ph_bytes(F) / 16;
  c.policy = 0;
  return c;
}

// Wait, warp-wide, for a ring stage: one try_wait per lane and a vote when
// the data is there (the usual case); otherwise all lanes retry together
// until the phase completes or about a second has passed (returns false).
__device__ __forceinline__ bool stage_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
      : "=r"(done) : "r"(bar), "r"(parity), "r"(1000000u) : "memory");
  if (__all_sync(0xFFFFFFFFu, done)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(done) : "r"(bar), "r"(parity), "r"(1000000u) : "memory");
    if (__all_sync(0xFFFFFFFFu, done)) return true;
    if (__shfl_sync(0xFFFFFFFFu, global_timer_ns() - t0 > 1000000000ull ? 1 : 0, 0)) return false;
  }
}

// An item of a warp's range as the loop uses it: the byte offset of its
// page-head in the pool and its valid tokens (0: nothing to copy or attend).
// Scored: bits 8 and up of nv hold ItemMap::hole, so a page seen whole is
// still nv == 16.
struct alignas(16) ItemEntry {
  long long off;
  int nv;
  int dist;  // ItemMap::dist
};

// cp.async staging of one page-head at byte offset `off` of the pool: lane l
// copies the 16-byte pieces l, l + 32, ... (NVFP4: lanes 0-15 five of the 144,
// the others four; MXFP4: lanes 0-7 five of the 136), predicated, none when nv
// is 0, then arrives (no-increment) on the stage's mbarrier, which expects 32
// arrivals; it fires once all of the lane's earlier copies have landed, so a
// stage's barrier covers every stage issued before it as well.
template <int F, int M>
__device__ __forceinline__ void issue_page_off(const LaneCopy& c, long long off, int nv, uint32_t st, uint32_t bar) {
  const uint8_t* src = c.src + off;
  const uint32_t dst = st + c.off;
  const uint32_t v5 = (nv > 0 && c.fifth) ? 1u : 0u;
  if constexpr ((M & kStored) != 0) {
    asm volatile(
        "{\n .reg .pred p, q;\n"
        " setp.gt.s32 p, %2, 0;\n"
        " setp.ne.u32 q, %3, 0;\n"
        " @p cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %5;\n"
        " @p cp.async.cg.shared.global.L2::cache_hint [%0+512], [%1+512], 16, %5;\n"
        " @p cp.async.cg.shared.global.L2::cache_hint [%0+1024], [%1+1024], 16, %5;\n"
        " @p cp.async.cg.shared.global.L2::cache_hint [%0+1536], [%1+1536], 16, %5;\n"
        " @q cp.async.cg.shared.global.L2::cache_hint [%0+2048], [%1+2048], 16, %5;\n"
        " cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%4];\n"
        "}\n" ::"r"(dst), "l"(src), "r"(nv), "r"(v5), "r"(bar), "l"(c.policy)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p, q;\n"
        " setp.gt.s32 p, %2, 0;\n"
        " setp.ne.u32 q, %3, 0;\n"
        " @p cp.async.cg.shared.global [%0], [%1], 16;\n"
        " @p cp.async.cg.shared.global [%0+512], [%1+512], 16;\n"
        " @p cp.async.cg.shared.global [%0+1024], [%1+1024], 16;\n"
        " @p cp.async.cg.shared.global [%0+1536], [%1+1536], 16;\n"
        " @q cp.async.cg.shared.global [%0+2048], [%1+2048], 16;\n"
        " cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%4];\n"
        "}\n" ::"r"(dst), "l"(src), "r"(nv), "r"(v5), "r"(bar)
        : "memory");
  }
}

// Two NVFP4 page-heads (288 pieces of 16 bytes: 9 per lane), into stages a and
// b: lane l copies pieces l + 32 k of the pair of page-heads, i.e. a's pieces
// l, l + 32, l + 64, l + 96, then a's l + 128 (l < 16) or b's l - 16 (l >= 16),
// then b's l + 16, l + 48, l + 80, l + 112; then arrives on both barriers.
// Nothing is copied for an entry with no valid tokens (a bad page id).
template <int M>
__device__ __forceinline__ void issue_two_off(const LaneCopy& c, const ItemEntry& a, const ItemEntry& b,
                                              uint32_t sta, uint32_t stb, uint32_t bara, uint32_t barb,
                                              bool lo) {
  const uint8_t* srca = c.src + a.off;
  const uint8_t* srcb = c.src + b.off;
  const uint32_t dsta = sta + c.off, dstb = stb + c.off;
  const uint32_t dst4 = lo ? dsta + 2048 : dstb - 256;
  const uint8_t* src4 = lo ? srca + 2048 : srcb - 256;
  const int n4 = lo ? a.nv : b.nv;
  if constexpr ((M & kStored) != 0) {
    asm volatile(
        "{\n .reg .pred pa, pb, p4;\n"
        " setp.gt.s32 pa, %4, 0;\n"
        " setp.gt.s32 pb, %5, 0;\n"
        " setp.gt.s32 p4, %6, 0;\n"
        " @pa cp.async.cg.shared.global.L2::cache_hint [%0], [%2], 16, %11;\n"
        " @pa cp.async.cg.shared.global.L2::cache_hint [%0+512], [%2+512], 16, %11;\n"
        " @pa cp.async.cg.shared.global.L2::cache_hint [%0+1024], [%2+1024], 16, %11;\n"
        " @pa cp.async.cg.shared.global.L2::cache_hint [%0+1536], [%2+1536], 16, %11;\n"
        " @p4 cp.async.cg.shared.global.L2::cache_hint [%7], [%8], 16, %11;\n"
        " @pb cp.async.cg.shared.global.L2::cache_hint [%1+256], [%3+256], 16, %11;\n"
        " @pb cp.async.cg.shared.global.L2::cache_hint [%1+768], [%3+768], 16, %11;\n"
        " @pb cp.async.cg.shared.global.L2::cache_hint [%1+1280], [%3+1280], 16, %11;\n"
        " @pb cp.async.cg.shared.global.L2::cache_hint [%1+1792], [%3+1792], 16, %11;\n"
        " cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%9];\n"
        " cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%10];\n"
        "}\n" ::"r"(dsta), "r"(dstb), "l"(srca), "l"(srcb), "r"(a.nv), "r"(b.nv), "r"(n4), "r"(dst4), "l"(src4),
        "r"(bara), "r"(barb), "l"(c.policy)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred pa, pb, p4;\n"
        " setp.gt.s32 pa, %4, 0;\n"
        " setp.gt.s32 pb, %5, 0;\n"
        " setp.gt.s32 p4, %6, 0;\n"
        " @pa cp.async.cg.shared.global [%0], [%2], 16;\n"
        " @pa cp.async.cg.shared.global [%0+512], [%2+512], 16;\n"
        " @pa cp.async.cg.shared.global [%0+1024], [%2+1024], 16;\n"
        " @pa cp.async.cg.shared.global [%0+1536], [%2+1536], 16;\n"
        " @p4 cp.async.cg.shared.global [%7], [%8], 16;\n"
        " @pb cp.async.cg.shared.global [%1+256], [%3+256], 16;\n"
        " @pb cp.async.cg.shared.global [%1+768], [%3+768], 16;\n"
        " @pb cp.async.cg.shared.global [%1+1280], [%3+1280], 16;\n"
        " @pb cp.async.cg.shared.global [%1+1792], [%3+1792], 16;\n"
        " cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%9];\n"
        " cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%10];\n"
        "}\n" ::"r"(dsta), "r"(dstb), "l"(srca), "l"(srcb), "r"(a.nv), "r"(b.nv), "r"(n4), "r"(dst4), "l"(src4),
        "r"(bara), "r"(barb)
        : "memory");
  }
}

// Per-warp attention state of the current pair.
struct WarpState {
  float o[8][4];    // O^T tiles: tile i rows d = 16g+2i (c0,c1) and 16g+2i+1 (c2,c3), cols heads 2t,2t+1
  uint32_t qf[8][2];  // q B-fragments: tile i holds q[head g][32t+4i .. 32t+4i+3]
  float m0, m1;     // running max (base 2) of heads 2t, 2t+1
  float l0, l1;     // this lane's partial sums of P over its tokens
  float c0, c1;     // score multipliers of heads 2t, 2t+1
  float x0, x1;     // kCapped: multipliers of the scores inside the tanh (c0, c1 come after it)
  float b0, b1;     // kBiased: base-2 bias per token of distance
};

// Orthonormal Walsh-Hadamard transform (Sylvester order) of the 128 values of
// a row held by a group of lanes: each lane holds N consecutive values (index
// bits below log2 N); passes across lanes pair the lane with lane ^ x for
// each lane mask x in `xs` (index bits above, lowest first), the lower lane
// keeping a + b and the upper a - b.  Then one product with RN(1 / sqrt(128)).
template <int N, int NX>
__device__ __forceinline__ void hadamard_lanes(float (&v)[N], const int (&xs)[NX], int lane) {
#pragma unroll
  for (int h = 1; h < N; h *= 2)
#pragma unroll
    for (int i = 0; i < N; i += 2 * h)
#pragma unroll
      for (int j = i; j < i + h; ++j) {
        const float a = v[j], b = v[j + h];
        v[j] = a + b;
        v[j + h] = a - b;
      }
#pragma unroll
  for (int k = 0; k < NX; ++k) {
    const bool upper = (lane & xs[k]) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, v[i], xs[k]);
      v[i] = upper ? o - v[i] : v[i] + o;
    }
  }
  const float c = 0x1.6a09e6p-4f;  // RN(1 / sqrt(128))
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] *= c;
}

// 2^d as an f16 for an integer d <= 0 (0 below f16's range): the relative
// weight of an MXFP4 block whose E8M0 exponent is d below the page's largest.
__device__ __forceinline__ uint32_t exp2_f16_bits(int d) {
  if (d >= -14) return (uint32_t)(d + 15) << 10;   // normal
  if (d >= -24) return 1u << (d + 24);             // subnormal
  return 0u;
}

// 2^e as an fp32 for an E8M0 exponent e in [-127, 127].
__device__ __forceinline__ float exp2_f32(int e) {
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(0x00400000u);
}

// The bf16 q elements lane (g, t) needs for pair b * hkv + h: head h * G + g,
// elements 32t .. 32t + 31 (zeros for g >= G).  Query heads of pair P start at
// row P * G of q, since hq = hkv * G.
struct QRaw {
  uint4 w[4];
};

template <bool kFresh = false>
__device__ __forceinline__ QRaw fetch_q(const DecodeParams& p, int pair, int g, int t) {
  QRaw r;
  if (g < p.group) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + ((long long)pair * p.group + g) * kHeadDim + 32 * t);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = kFresh ? src[j] : __ldg(src + j);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[j] = make_uint4(0u, 0u, 0u, 0u);
  }
  return r;
}

// Turn fetched q into B-fragments with a per-head power-of-two prescale and
// reset the pair's softmax state.
template <int F, int M>
__device__ __forceinline__ void load_q(const DecodeParams& p, const QRaw& raw, WarpState& s, int pair, int g, int t) {
  float qv[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 w = raw.w[j];
    qv[8 * j + 0] = bf16_to_f32(w.x & 0xFFFFu); qv[8 * j + 1] = bf16_to_f32(w.x >> 16);
    qv[8 * j + 2] = bf16_to_f32(w.y & 0xFFFFu); qv[8 * j + 3] = bf16_to_f32(w.y >> 16);
    qv[8 * j + 4] = bf16_to_f32(w.z & 0xFFFFu); qv[8 * j + 5] = bf16_to_f32(w.z >> 16);
    qv[8 * j + 6] = bf16_to_f32(w.w & 0xFFFFu); qv[8 * j + 7] = bf16_to_f32(w.w >> 16);
  }
  if constexpr (F == kFmtHadamard) {
    // the cache holds NVFP4 of H k for each key k: q . k = (H q) . (H k), so q
    // is rotated once here (lane t holds elements 32t .. 32t + 31: passes 1-16
    // inside the lane, 32 and 64 across lanes t ^ 1 and t ^ 2)
    const int xs[2] = {1, 2};
    hadamard_lanes<32, 2>(qv, xs, (g << 2) | t);
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(qv[j]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  const F16Range r = f16_range(amax);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s.qf[i][0] = pack_f16x2(qv[4 * i] * r.up, qv[4 * i + 1] * r.up);
    s.qf[i][1] = pack_f16x2(qv[4 * i + 2] * r.up, qv[4 * i + 3] * r.up);
  }
  const float c = fminf(p.score_scale * r.down, FLT_MAX);  // score multiplier of head g; finite: it may meet a zero
  if constexpr ((M & kCapped) != 0) {
    // finite: it may meet a zero (and anything else it makes far larger than 1 either way)
    const float x = fminf(p.cap_scale * r.down, FLT_MAX);
    s.x0 = __shfl_sync(0xFFFFFFFFu, x, (2 * t) * 4);
    s.x1 = __shfl_sync(0xFFFFFFFFu, x, (2 * t + 1) * 4);
    s.c0 = s.c1 = p.score_scale;
  } else {
    s.c0 = __shfl_sync(0xFFFFFFFFu, c, (2 * t) * 4);
    s.c1 = __shfl_sync(0xFFFFFFFFu, c, (2 * t + 1) * 4);
  }
  if constexpr ((M & kBiased) != 0) {
    const float* sl = p.slopes + (long long)(pair % p.hkv) * p.group;
    s.b0 = 2 * t < p.group ? base2_slope(__ldg(sl + 2 * t)) : 0.0f;
    s.b1 = 2 * t + 1 < p.group ? base2_slope(__ldg(sl + 2 * t + 1)) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s.o[i][j] = 0.0f;
  s.m0 = s.m1 = -INFINITY;
  s.l0 = s.l1 = 0.0f;
}

__device__ __forceinline__ bool in_hole(int hole, int row) { return row >= (hole & 255) && row < (hole >> 8); }

// Sixteen fp32 -> bf16 (round to nearest even) at a 16-byte boundary.
__device__ __forceinline__ void store_bf16x16(uint16_t* dst, const float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    reinterpret_cast<uint4*>(dst)[j] =
        make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                   pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
}

// The log-sum-exp of one (sequence, query head) from its base-2 running max
// and sum; -inf when nothing was visible.
template <int M>
__device__ __forceinline__ void store_lse(const DecodeParams& p, long long row, float m, float l) {
  const float v = l > 0.0f ? m + log2f(l) : -INFINITY;
  if (p.lse != nullptr) p.lse[row] = v * kLn2;
  if constexpr ((M & kStored) != 0) p.lse2[row] = v;
}

// Keep a page's base-2 scores (masked ones are -inf): [16 tokens][score_heads]
// floats, the lane's heads 2t and 2t + 1 of tokens g and g + 8; the warp's
// stores of eight heads cover 512 contiguous bytes.
__device__ __forceinline__ void store_scores(const DecodeParams& p, float* dst, const float (&S)[4], float c0,
                                             float c1, int g, int t) {
  if (dst != nullptr && 2 * t < p.score_heads) {
    *reinterpret_cast<float2*>(dst + g * p.score_heads + 2 * t) = make_float2(S[0] * c0, S[1] * c1);
    *reinterpret_cast<float2*>(dst + (g + 8) * p.score_heads + 2 * t) = make_float2(S[2] * c0, S[3] * c1);
  }
}

// Phase 1 of a step: S^T = Khat q^T for NP pages (16 tokens x G heads each),
// one accumulator chain per page (or two, tiles 0-3 and 4-7, with
// NVFP4KV_DECODE_QK_CHAINS 2: shorter chains, four more adds per page).
// MXFP4 pages carry their scales relative to the page's largest exponent (per
// K and per V, so every product stays inside f16): kx[k] = 2^(K's largest)
// multiplies the page's scores, ve[k] (V's largest) enters the softmax exponent.
struct PageExp {
  float kx;  // 2^ek
  int ve;    // ev
};

template <int NP, int F>
__device__ __forceinline__ void qk_phase(const uint8_t* const (&stage)[NP], const int (&nvalid)[NP],
                                         const WarpState& s, float (&sc)[NP][2][4], PageExp (&pe)[NP], int g,
                                         int t) {
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const uint8_t* kd = stage[k] + kOffKD;
    const uint8_t* ks = stage[k] + off_ks(F);
    const uint4 ka = *reinterpret_cast<const uint4*>(kd + g * kRowBytes + 16 * t);
    const uint4 kb = *reinterpret_cast<const uint4*>(kd + (g + 8) * kRowBytes + 16 * t);
    uint32_t sa, sb;  // f16x2: the scales of blocks 2t (low half) and 2t + 1 (high half) of rows g, g + 8
    if constexpr (F == kFmtMxfp4) {
      // the lane's 32 values of rows g and g + 8 are one block (t); the 64 K
      // scale bytes of the page are read once over the warp, as are V's
      // (rows at or past the page's valid tokens hold other data: they count as 0)
      const int nv = nvalid[k];
      const int ea = g < nv ? ks[g * kMxRowScales + t] : 0, eb = g + 8 < nv ? ks[(g + 8) * kMxRowScales + t] : 0;
      int ek = max(ea, eb);
      const uint8_t* vsc = stage[k] + off_vs(F) + (g >> 1) * kPage;
      int ev = max(max(2 * t < nv ? vsc[2 * t] : 0, 2 * t + 1 < nv ? vsc[2 * t + 1] : 0),
                   max(2 * t + 8 < nv ? vsc[2 * t + 8] : 0, 2 * t + 9 < nv ? vsc[2 * t + 9] : 0));
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        ek = max(ek, __shfl_xor_sync(0xFFFFFFFFu, ek, off));
        ev = max(ev, __shfl_xor_sync(0xFFFFFFFFu, ev, off));
      }
      pe[k].kx = exp2_f32(ek - 127);
      pe[k].ve = ev - 127;
      sa = dup_lo(exp2_f16_bits(ea - ek));
      sb = dup_lo(exp2_f16_bits(eb - ek));
    } else {
      sa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + g * kRowScales + 2 * t));
      sb = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + (g + 8) * kRowScales + 2 * t));
      pe[k].kx = 1.0f;
      pe[k].ve = 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t wa = word_of(ka, i >> 1), wb = word_of(kb, i >> 1);
      uint32_t a0, a1, a2, a3;
      if (i & 1) {
        a0 = cvt_sel<2>(wa); a1 = cvt_sel<2>(wb); a2 = cvt_sel<3>(wa); a3 = cvt_sel<3>(wb);
      } else {
        a0 = cvt_sel<0>(wa); a1 = cvt_sel<0>(wb); a2 = cvt_sel<1>(wa); a3 = cvt_sel<1>(wb);
      }
      if (i < 4) {
        a0 = hmul2_bcast<false>(a0, sa); a2 = hmul2_bcast<false>(a2, sa);
        a1 = hmul2_bcast<false>(a1, sb); a3 = hmul2_bcast<false>(a3, sb);
      } else {
        a0 = hmul2_bcast<true>(a0, sa); a2 = hmul2_bcast<true>(a2, sa);
        a1 = hmul2_bcast<true>(a1, sb); a3 = hmul2_bcast<true>(a3, sb);
      }
      // chain c = i / 4 (two chains) or 0: its first MMA starts from zero
      const int c = NVFP4KV_DECODE_QK_CHAINS == 2 ? (i >> 2) : 0;
      if (i == 0 || (NVFP4KV_DECODE_QK_CHAINS == 2 && i == 4))
        mma16816_zero(sc[k][c], a0, a1, a2, a3, s.qf[i][0], s.qf[i][1]);
      else
        mma16816(sc[k][c], a0, a1, a2, a3, s.qf[i][0], s.qf[i][1]);
    }
  }

}

// Phase 2: online softmax (base 2) over the NP pages' scores, one running-max
// check for all of them; returns P^T as mma B fragments (k = tokens, n = heads).
// Scored: S becomes the score in units of c0 / c1 -- the product itself, its
// tanh, or (with a bias) the base-2 score, c0 = c1 = 1 from there on.
template <int NP, bool kFull, int F, int M>
__device__ __forceinline__ void softmax_phase(const DecodeParams& p, const float (&sc)[NP][2][4],
                                              const PageExp (&pe)[NP], const int (&nvalid)[NP],
                                              const int (&hole)[NP], const int (&dist)[NP], float* (&keep)[NP],
                                              WarpState& s, uint32_t (&pb)[NP][2], int g, int t) {
  // raw scores; the running max is kept in scaled (base-2) units: max(S c) = c max(S), c > 0.
  // MXFP4: page k's weights carry 2^ve[k] (its V exponent), folded into the
  // exponent so that P stays within f16; the sums l take it out again.
  float S[NP][4];
  float mx0 = -INFINITY, mx1 = -INFINITY;
  const float c0 = (M & kBiased) != 0 ? 1.0f : s.c0, c1 = (M & kBiased) != 0 ? 1.0f : s.c1;
  if constexpr ((M & kCapped) != 0) {
    float2 x[2 * NP];
#pragma unroll
    for (int k = 0; k < NP; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[2 * k + j].x = (NVFP4KV_DECODE_QK_CHAINS == 2 ? sc[k][0][2 * j] + sc[k][1][2 * j] : sc[k][0][2 * j]) * s.x0;
        x[2 * k + j].y =
            (NVFP4KV_DECODE_QK_CHAINS == 2 ? sc[k][0][2 * j + 1] + sc[k][1][2 * j + 1] : sc[k][0][2 * j + 1]) * s.x1;
      }
    tanh_warp(x);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      S[k][0] = x[2 * k].x;
      S[k][1] = x[2 * k].y;
      S[k][2] = x[2 * k + 1].x;
      S[k][3] = x[2 * k + 1].y;
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    if constexpr ((M & kCapped) == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) S[k][j] = NVFP4KV_DECODE_QK_CHAINS == 2 ? sc[k][0][j] + sc[k][1][j] : sc[k][0][j];
    }
    if constexpr ((M & kBiased) != 0) {
      // tokens g and g + 8 of the page lie dist + g and dist + g + 8 (<= 0) from the query
      const float d0 = (float)(dist[k] + g), d1 = (float)(dist[k] + g + 8);
      S[k][0] = fmaf(S[k][0], s.c0, s.b0 * d0);
      S[k][1] = fmaf(S[k][1], s.c1, s.b1 * d0);
      S[k][2] = fmaf(S[k][2], s.c0, s.b0 * d1);
      S[k][3] = fmaf(S[k][3], s.c1, s.b1 * d1);
    }
    if constexpr (F == kFmtMxfp4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) S[k][j] *= pe[k].kx;
    }
    if (!kFull && nvalid[k] < kPage) {
      if (g >= nvalid[k]) S[k][0] = S[k][1] = -INFINITY;
      if (g + 8 >= nvalid[k]) S[k][2] = S[k][3] = -INFINITY;
    }
    if constexpr (M != 0) {
      if (!kFull && hole[k]) {  // between the sinks and the window
        if (in_hole(hole[k], g)) S[k][0] = S[k][1] = -INFINITY;
        if (in_hole(hole[k], g + 8)) S[k][2] = S[k][3] = -INFINITY;
      }
    }
    if constexpr ((M & kStored) != 0) store_scores(p, keep[k], S[k], c0, c1, g, t);
    float a0 = fmaxf(S[k][0], S[k][2]) * c0, a1 = fmaxf(S[k][1], S[k][3]) * c1;
    if constexpr (F == kFmtMxfp4) {
      a0 += (float)pe[k].ve;
      a1 += (float)pe[k].ve;
    }
    mx0 = fmaxf(mx0, a0);
    mx1 = fmaxf(mx1, a1);
  }
  const bool need = (mx0 > s.m0 + kLazy) || (mx1 > s.m1 + kLazy);
  if (__any_sync(0xFFFFFFFFu, need)) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, off));
    }
    const float n0 = fmaxf(s.m0, mx0), n1 = fmaxf(s.m1, mx1);
    float f0 = ex2(s.m0 - n0), f1 = ex2(s.m1 - n1);
    if constexpr ((M & kBiased) != 0) {
      // a head that has seen nothing yet (a bias of -inf) while another's maximum moves
      f0 = n0 == -INFINITY ? 1.0f : f0;
      f1 = n1 == -INFINITY ? 1.0f : f1;
    }
    s.l0 *= f0;
    s.l1 *= f1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s.o[i][0] *= f0; s.o[i][1] *= f1; s.o[i][2] *= f0; s.o[i][3] *= f1;
    }
    s.m0 = n0;
    s.m1 = n1;
  }
  const float nm0 = -s.m0, nm1 = -s.m1;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    float o0 = nm0, o1 = nm1;
    if constexpr (F == kFmtMxfp4) {
      o0 += (float)pe[k].ve;
      o1 += (float)pe[k].ve;
    }
    float p0, p1, p2, p3;
    if constexpr (M != 0 && (!kFull || (M & kBiased) != 0)) {
      // nothing may have shown yet (rows in the hole, a bias of -inf): a maximum
      // of -inf gives zeros
      o0 = s.m0 == -INFINITY ? -INFINITY : o0;
      o1 = s.m1 == -INFINITY ? -INFINITY : o1;
    }
    p0 = ex2(fmaf(S[k][0], c0, o0)), p1 = ex2(fmaf(S[k][1], c1, o1));
    p2 = ex2(fmaf(S[k][2], c0, o0)), p3 = ex2(fmaf(S[k][3], c1, o1));
    if constexpr (F == kFmtMxfp4) {
      const float un = exp2_f32(-pe[k].ve);  // 2^-ve: the sum counts the plain weights
      s.l0 += (p0 + p2) * un;
      s.l1 += (p1 + p3) * un;
    } else {
      s.l0 += p0 + p2;
      s.l1 += p1 + p3;
    }
    // P^T (tokens x heads) in the accumulator layout -> B fragments (k = tokens, n = heads)
    pb[k][0] = movmatrix_trans(pack_f16x2(p0, p1));
    pb[k][1] = movmatrix_trans(pack_f16x2(p2, p3));
  }
}

// Phase 3: O^T += Vhat^T P^T for the NP pages.
template <int NP, bool kFull, int F, int M>
__device__ __forceinline__ void pv_phase(const uint8_t* const (&stage)[NP], const int (&nvalid)[NP],
                                         const int (&hole)[NP], const PageExp (&pe)[NP],
                                         const uint32_t (&pb)[NP][2], WarpState& s, int g, int t) {
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const uint8_t* vd = stage[k] + off_vd(F);
    const uint8_t* vs = stage[k] + off_vs(F);
    const int t0 = 2 * t, t1 = 2 * t + 1, t8 = 2 * t + 8, t9 = 2 * t + 9;
    uint32_t sv01, sv89;  // (token 2t, token 2t+1) and (2t+8, 2t+9) scales of the lane's block, f16x2
    if constexpr (F == kFmtMxfp4) {
      // the lane's 16 values are in block g / 2; its E8M0 exponents relative to the page's largest
      const uint8_t* b = vs + (g >> 1) * kPage;
      const bool full = kFull || nvalid[k] >= kPage;
      const int ve = pe[k].ve + 127;
      const uint32_t e0 = (full || t0 < nvalid[k]) ? exp2_f16_bits(b[t0] - ve) : 0u;
      const uint32_t e1 = (full || t1 < nvalid[k]) ? exp2_f16_bits(b[t1] - ve) : 0u;
      const uint32_t e8 = (full || t8 < nvalid[k]) ? exp2_f16_bits(b[t8] - ve) : 0u;
      const uint32_t e9 = (full || t9 < nvalid[k]) ? exp2_f16_bits(b[t9] - ve) : 0u;
      sv01 = e0 | (e1 << 16);
      sv89 = e8 | (e9 << 16);
    } else {
      // V scales are block-major: block g's scales of tokens (2t, 2t+1) and (2t+8, 2t+9) are adjacent pairs
      uint32_t p01 = *reinterpret_cast<const uint16_t*>(vs + g * kPage + t0);
      uint32_t p89 = *reinterpret_cast<const uint16_t*>(vs + g * kPage + t8);
      if (!kFull && nvalid[k] < kPage) {  // tokens past the end: scale 0 keeps unwritten bytes out of the sum
        if (t0 >= nvalid[k]) p01 &= 0xFF00u;
        if (t1 >= nvalid[k]) p01 &= 0x00FFu;
        if (t8 >= nvalid[k]) p89 &= 0xFF00u;
        if (t9 >= nvalid[k]) p89 &= 0x00FFu;
      }
      if constexpr (M != 0) {
        if (!kFull && hole[k]) {
          if (in_hole(hole[k], t0)) p01 &= 0xFF00u;
          if (in_hole(hole[k], t1)) p01 &= 0x00FFu;
          if (in_hole(hole[k], t8)) p89 &= 0xFF00u;
          if (in_hole(hole[k], t9)) p89 &= 0x00FFu;
        }
      }
      sv01 = e4m3x2_to_f16x2(p01);
      sv89 = e4m3x2_to_f16x2(p89);
    }
    // V data by token pair: pair t holds tokens (2t, 2t+1), pair t + 4 tokens
    // (2t+8, 2t+9); bytes 16g .. 16g + 15 of a pair row are dimensions 16g ..
    // 16g + 15, each byte the two tokens' codes of one dimension: one E2M1
    // conversion gives an A-operand register (k = the two tokens) as it is
    const uint4 w01 = *reinterpret_cast<const uint4*>(vd + t * kVPairBytes + 16 * g);
    const uint4 w89 = *reinterpret_cast<const uint4*>(vd + (t + 4) * kVPairBytes + 16 * g);
    const uint32_t pb0 = pb[k][0], pb1 = pb[k][1];
    // tile I: rows g and g + 8 are dimensions 16g + 2I and 16g + 2I + 1, bytes
    // 2I and 2I + 1 of the lane's 16
#define NVFP4KV_PV_TILE(I, W01, W89, K0, K1)                                    \
  {                                                                             \
    const uint32_t a0 = hmul2(cvt_sel<K0>(W01), sv01);                          \
    const uint32_t a1 = hmul2(cvt_sel<K1>(W01), sv01);                          \
    const uint32_t a2 = hmul2(cvt_sel<K0>(W89), sv89);                          \
    const uint32_t a3 = hmul2(cvt_sel<K1>(W89), sv89);                          \
    mma16816(s.o[I], a0, a1, a2, a3, pb0, pb1);                                 \
  }
    NVFP4KV_PV_TILE(0, w01.x, w89.x, 0, 1)
    NVFP4KV_PV_TILE(1, w01.x, w89.x, 2, 3)
    NVFP4KV_PV_TILE(2, w01.y, w89.y, 0, 1)
    NVFP4KV_PV_TILE(3, w01.y, w89.y, 2, 3)
    NVFP4KV_PV_TILE(4, w01.z, w89.z, 0, 1)
    NVFP4KV_PV_TILE(5, w01.z, w89.z, 2, 3)
    NVFP4KV_PV_TILE(6, w01.w, w89.w, 0, 1)
    NVFP4KV_PV_TILE(7, w01.w, w89.w, 2, 3)
#undef NVFP4KV_PV_TILE
  }
}

// NP pages of one KV head (16 tokens each, nvalid[k] of them valid) from ring
// stages, folded into the warp's running softmax state with one max update.
// kFull: every page has all 16 tokens (no masking code).
template <int NP, bool kFull, int F, int M>
__device__ __forceinline__ void process_pages(const DecodeParams& p, const uint8_t* const (&stage)[NP],
                                              const int (&nv)[NP], const int (&dist)[NP], float* (&keep)[NP],
                                              WarpState& s, int g, int t) {
  float sc[NP][2][4];
  uint32_t pb[NP][2];
  PageExp pe[NP];
  int nvalid[NP], hole[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    nvalid[k] = M != 0 ? nv[k] & 255 : nv[k];
    hole[k] = M != 0 ? nv[k] >> 8 : 0;
  }
  qk_phase<NP, F>(stage, nvalid, s, sc, pe, g, t);
  softmax_phase<NP, kFull, F, M>(p, sc, pe, nvalid, hole, dist, keep, s, pb, g, t);
  pv_phase<NP, kFull, F, M>(stage, nvalid, hole, pe, pb, s, g, t);
}

// Finish a warp's piece of a pair: total l over the lanes, then either write
// the final output (complete pair) or store the piece's record at `slot`.
template <int F, int M>
__device__ __forceinline__ void finish_piece(const DecodeParams& p, WarpState& s, int pair, bool complete,
                                             float* slot, int g, int t) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    s.l0 += __shfl_xor_sync(0xFFFFFFFFu, s.l0, off);
    s.l1 += __shfl_xor_sync(0xFFFFFFFFu, s.l1, off);
  }
  const int h0 = 2 * t, h1 = 2 * t + 1;
  if (complete) {
    const int b = pair / p.hkv, h = pair - (pair / p.hkv) * p.hkv;
    const long long row0 = (long long)b * p.hq + (long long)h * p.group;
    const float r0 = s.l0 > 0.0f ? p.v_gscale / s.l0 : 0.0f;
    const float r1 = s.l1 > 0.0f ? p.v_gscale / s.l1 : 0.0f;
    // the lane's values of heads 2t and 2t + 1: d = 16 g + k, k = 0 .. 15
    float v0[16], v1[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v0[2 * i] = s.o[i][0] * r0; v0[2 * i + 1] = s.o[i][2] * r0;
      v1[2 * i] = s.o[i][1] * r1; v1[2 * i + 1] = s.o[i][3] * r1;
    }
    if constexpr (F == kFmtHadamard) {
      // rotate the output back (d bits 0-3 in the lane, 4-6 across lanes g: lane ^ 4, 8, 16)
      const int xs[3] = {4, 8, 16};
      hadamard_lanes<16, 3>(v0, xs, (g << 2) | t);
      hadamard_lanes<16, 3>(v1, xs, (g << 2) | t);
    }
    if constexpr (M != 0) {
      if (h0 < p.group) store_bf16x16(p.out16 + (row0 + h0) * kHeadDim + 16 * g, v0);
      if (h1 < p.group) store_bf16x16(p.out16 + (row0 + h1) * kHeadDim + 16 * g, v1);
      if (g == 0 && h0 < p.group) store_lse<M>(p, row0 + h0, s.m0, s.l0);
      if (g == 0 && h1 < p.group) store_lse<M>(p, row0 + h1, s.m1, s.l1);
    } else {
      float* base = p.out + row0 * kHeadDim;
      if (h0 < p.group) {
        float4* dst = reinterpret_cast<float4*>(base + h0 * kHeadDim + 16 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = make_float4(v0[4 * j], v0[4 * j + 1], v0[4 * j + 2], v0[4 * j + 3]);
      }
      if (h1 < p.group) {
        float4* dst = reinterpret_cast<float4*>(base + h1 * kHeadDim + 16 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = make_float4(v1[4 * j], v1[4 * j + 1], v1[4 * j + 2], v1[4 * j + 3]);
      }
    }
  } else {
    float4* d0 = reinterpret_cast<float4*>(slot + h0 * kHeadDim + 16 * g);
    float4* d1 = reinterpret_cast<float4*>(slot + h1 * kHeadDim + 16 * g);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d0[j] = make_float4(s.o[2 * j][0], s.o[2 * j][2], s.o[2 * j + 1][0], s.o[2 * j + 1][2]);
      d1[j] = make_float4(s.o[2 * j][1], s.o[2 * j][3], s.o[2 * j + 1][1], s.o[2 * j + 1][3]);
    }
    if (g == 0) {
      slot[kOffM + h0] = s.m0;
      slot[kOffM + h1] = s.m1;
      slot[kOffL + h0] = s.l0;
      slot[kOffL + h1] = s.l1;
    }
  }
}

__device__ __forceinline__ long long block_sum_ll(long long v, long long* red, int warp, int lane) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kNW; ++w) total += red[w];
  __syncthreads();
  return total;
}

// The output rows of an empty sequence: zeros (and a log-sum-exp of -inf).
template <int M>
__device__ __forceinline__ void zero_sequence(const DecodeParams& p, int b) {
  if constexpr (M != 0) {
    uint4* o = reinterpret_cast<uint4*>(p.out16 + (long long)b * p.hq * kHeadDim);
    for (int j = 0; j < p.hq * kHeadDim / 8; ++j) o[j] = make_uint4(0u, 0u, 0u, 0u);
    for (int j = 0; j < p.hq; ++j) store_lse<M>(p, (long long)b * p.hq + j, 0.0f, 0.0f);
  } else {
    float4* o = reinterpret_cast<float4*>(p.out + (long long)b * p.hq * kHeadDim);
    for (int j = 0; j < p.hq * kHeadDim / 4; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

template <int F, int M>
__global__ void __launch_bounds__(kNW * 32, kCtasPerSm) decode_kernel(const DecodeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRingBytes);
  __shared__ long long red[kNW];
  __shared__ int wstart_b[kNW], wstart_cu[kNW];
  // per warp: (page-head row, valid tokens) of items [32 chunk, 32 chunk + 64),
  // item k at k % 64, written as each 32-item chunk map is resolved
  __shared__ ItemEntry s_items[kNW][64];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  // the combine kernel may be scheduled now: its blocks take SMs as decode CTAs
  // retire and wait (griddepcontrol.wait) for the whole decode grid
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- prologue: total work, zero outputs of empty sequences -------------------
  {
    // bring q and the page table into L2 early (each CTA a slice, 128-byte
    // lines): the first chunk maps and later pieces then find them there
    // instead of queueing behind the KV stream
    const long long step = (long long)gridDim.x * blockDim.x, first = (long long)blockIdx.x * blockDim.x + tid;
    const long long qlines = ((long long)p.batch * p.hq * kHeadDim * 2 + 127) / 128;
    for (long long l = first; l < qlines; l += step)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(p.q) + 128 * l));
    const long long plines = ((long long)p.batch * p.max_pages * 4 + 127) / 128;
    for (long long l = first; l < plines; l += step)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(p.page_table) + 128 * l));
  }
  long long W = 0;
  long long r0 = 0, r1 = 0;
  const long long N = gridDim.x;
  if (p.batch <= kNW * 32) {
    // one pass: every sequence's length is read once, by thread b
    const int b = tid;
    int np = 0;
    if (b < p.batch) {
      const int L = clamp_len(p, b);
      np = visible_pages<M>(p, L).count;
      if (L == 0 && (b % (int)gridDim.x) == (int)blockIdx.x) zero_sequence<M>(p, b);
    }
    int incl = np;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      if (w < warp) before += red[w];
      total += red[w];
    }
    W = total * p.hkv;
    if (W == 0) {
      if ((M & kStored) != 0 && blockIdx.x == 0 && tid == 0) p.cu_pages[p.batch] = 0;
      asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows waits for this grid, not for an append ahead
      return;
    }
    r0 = cta_start(blockIdx.x, W, N);
    r1 = cta_start((long long)blockIdx.x + 1, W, N);
    const int excl = (int)before + incl - np;
    if (blockIdx.x == 0 && b < p.batch) p.cu_pages[b] = excl;
    if (blockIdx.x == 0 && tid == 0) p.cu_pages[p.batch] = (int)total;
    if (np > 0) {
      for (int w2 = 0; w2 < kNW; ++w2) {
        const long long ws = r0 + (r1 - r0) * w2 / kNW, we = r0 + (r1 - r0) * (w2 + 1) / kNW;
        if (ws < we && ws >= (long long)excl * p.hkv && ws < (long long)(excl + np) * p.hkv) {
          wstart_b[w2] = b;
          wstart_cu[w2] = excl;
        }
      }
    }
    __syncthreads();
  } else {
    long long pages_local = 0;
    for (int b = tid; b < p.batch; b += kNW * 32) {
      const int L = clamp_len(p, b);
      pages_local += visible_pages<M>(p, L).count;
      if (L == 0 && (b % (int)gridDim.x) == (int)blockIdx.x) zero_sequence<M>(p, b);
    }
    W = block_sum_ll(pages_local, red, warp, lane) * p.hkv;
    if (W == 0) {
      if ((M & kStored) != 0 && blockIdx.x == 0 && tid == 0) p.cu_pages[p.batch] = 0;
      asm volatile("griddepcontrol.wait;" ::: "memory");  // what follows waits for this grid, not for an append ahead
      return;
    }
    r0 = cta_start(blockIdx.x, W, N);
    r1 = cta_start((long long)blockIdx.x + 1, W, N);

    // locate the sequence holding each warp's first page-head
    int carry = 0;
    for (int base = 0; base < p.batch; base += kNW * 32) {
      const int b = base + tid;
      const int np = b < p.batch ? pages_of<M>(p, b) : 0;
      int incl = np;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += v;
      }
      if (lane == 31) red[warp] = incl;
      __syncthreads();
      int before = carry, chunk = 0;
#pragma unroll
      for (int w = 0; w < kNW; ++w) {
        if (w < warp) before += (int)red[w];
        chunk += (int)red[w];
      }
      const int excl = before + incl - np;
      if (blockIdx.x == 0 && b < p.batch) p.cu_pages[b] = excl;
      if (np > 0) {
        for (int w2 = 0; w2 < kNW; ++w2) {
          const long long ws = r0 + (r1 - r0) * w2 / kNW, we = r0 + (r1 - r0) * (w2 + 1) / kNW;
          if (ws < we && ws >= (long long)excl * p.hkv && ws < (long long)(excl + np) * p.hkv) {
            wstart_b[w2] = b;
            wstart_cu[w2] = excl;
          }
        }
      }
      carry += chunk;
      __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) p.cu_pages[p.batch] = carry;
  }

  // ---- per-warp streaming over its page-heads ----------------------------------
  const long long wr0 = r0 + (r1 - r0) * warp / kNW;
  const long long wr1 = r0 + (r1 - r0) * (warp + 1) / kNW;
  const int n = (int)(wr1 - wr0);
  uint8_t* wring = ring + warp * kStages * kStageBytes;
  const uint32_t wbar = smem_u32(bars + warp * kStages);
  const long long gwarp = (long long)blockIdx.x * kNW + warp;  // global warp index

  if (n == 0 && lane < kGMax) {
    // a warp with no items lies between the pieces of a cut pair when a CTA's
    // range is shorter than kNW: its first record is marked empty (m = -inf),
    // which the combine skips
    p.part[2 * gwarp * kRecFloats + kOffM + lane] = -INFINITY;
  }
  if (n > 0) {
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) mbar_init(wbar + 8 * s, 32);
      fence_mbar_init();
    }
    __syncwarp();
    SeqCursor seq;
    seq.b = wstart_b[warp];
    seq.cu = wstart_cu[warp];
    seq.L = clamp_len(p, seq.b);
    ItemMap cur = map_chunk<M>(p, wr0, 0, n, seq, lane);
    // the first piece's q goes out before the ring prefill, so it does not
    // queue behind the pages
    const int pair_first = __shfl_sync(0xFFFFFFFFu, cur.pair, 0);
    const QRaw q_first = fetch_q(p, pair_first, g, t);
    ItemMap nxt = cur;
    bool nres = true;  // nxt has been resolved (or is not used)
    if (n > 32) {
      nxt = map_chunk<M>(p, wr0, 32, n, seq, lane);
      nres = false;
    }
    ItemEntry* const tab = s_items[warp];
    // an item's entry: computed by its lane once per chunk, used by the loop
    auto entry_of = [&](const ItemMap& m) {
      ItemEntry e;
      e.off = m.row < 0 ? 0 : (long long)m.row * ph_bytes(F);
      e.nv = M != 0 && m.nv > 0 ? m.nv | (m.hole << 8) : m.nv;
      e.dist = M != 0 ? m.dist : 0;
      return e;
    };
    resolve_chunk<M>(p, cur);
    tab[lane] = entry_of(cur);
    __syncwarp();

    // Launched right behind the append of the same decode step
    // (nvfp4kv_append_decode_attention), this grid ran everything above while
    // the append was still writing the new tokens' pages: wait for it before
    // the first page is read.  Without a prerequisite grid this returns at once.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // producer: prefill the ring (all within the first chunk: kStages < 32)
    const int pre = n < kStages ? n : kStages;
    LaneCopy lc = lane_copy<F>(p, lane);
    if constexpr ((M & kStored) != 0)
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(lc.policy));
    const uint32_t wring_u32 = smem_u32(wring);
    for (int j = 0; j < pre; ++j) {
      issue_page_off<F, M>(lc, tab[j].off, tab[j].nv, wring_u32 + j * kStageBytes, wbar + 8 * j);
    }
    int issued = pre;
    int chunk = 0;   // the chunk `cur` maps
    int st = 0;      // ring stage of the next item
    uint32_t ph = 0; // its mbarrier phase parity
    WarpState s;
    load_q<F, M>(p, q_first, s, pair_first, g, t);  // the first piece's q, fetched before the prefill
    int nseg = 0;
    int i = 0;
    // where the scores of the warp's item k are kept (null: no room for this batch)
    auto score_row = [&](int k) -> float* {
      return W <= p.score_items ? p.scores + (wr0 + k) * (long long)(kPage * p.score_heads) : nullptr;
    };
    // resolve the next chunk's map into the item table
#define NVFP4KV_RESOLVE_NXT()                                          \
  {                                                                     \
    resolve_chunk<M>(p, nxt);                                           \
    tab[(32 * (chunk + 1) + lane) & 63] = entry_of(nxt);                \
    __syncwarp();                                                       \
  }
    // the chunk maps hold items [32 chunk, 32 chunk + 64): move them up to item k
#define NVFP4KV_ADVANCE_TO(k)                                   \
  while (((k) >> 5) != chunk) {                                 \
    if (!nres) NVFP4KV_RESOLVE_NXT();                           \
    cur = nxt;                                                  \
    ++chunk;                                                    \
    nres = true;                                                \
    if ((chunk + 1) * 32 < n) {                                 \
      nxt = map_chunk<M>(p, wr0, (chunk + 1) * 32, n, seq, lane); \
      nres = false;                                             \
    }                                                           \
  }
    while (i < n) {
      // ---- one piece: items [i, iend) of one (sequence, KV head) pair -------------
      NVFP4KV_ADVANCE_TO(i)
      const int li = i & 31;
      const int pair = __shfl_sync(0xFFFFFFFFu, cur.pair, li);
      const int page0 = __shfl_sync(0xFFFFFFFFu, cur.page, li);
      const int np = __shfl_sync(0xFFFFFFFFu, cur.np, li);
      const int iend = min(n, i + (np - page0));
      ++nseg;
      if (nseg > 1) load_q<F, M>(p, fetch_q(p, pair, g, t), s, pair, g, t);
      int j = i;
      // the next item at which the chunk maps need work: the next chunk's start,
      // or half way through this chunk while the next one's rows are unresolved
#define NVFP4KV_NEXT_EVENT() (nres ? 32 * (chunk + 1) : min(32 * (chunk + 1), 32 * chunk + 16))
      int ev = NVFP4KV_NEXT_EVENT();
      // two pages per step
      for (; j + 1 < iend; j += 2) {
        if (j >= ev) {
          NVFP4KV_ADVANCE_TO(j)
          // the next chunk's rows are first needed at item 32 chunk + 32 - kStages - 1;
          // resolving them half way through the chunk leaves their loads time to land
          if (!nres && (j & 31) >= 16) {
            NVFP4KV_RESOLVE_NXT();
            nres = true;
          }
          ev = NVFP4KV_NEXT_EVENT();
        }
        const int st1 = st + 1 == kStages ? 0 : st + 1;
        const uint32_t ph1 = st1 == 0 ? ph ^ 1u : ph;
        // The second stage's barrier fires only after each lane's earlier copies
        // (those of the first stage) have landed too, so one wait covers both.
        if (!stage_wait(wbar + 8 * st1, ph1)) goto timed_out;
        {
          const int nv0 = tab[j & 63].nv, nv1 = tab[(j + 1) & 63].nv;
          const uint8_t* const stg[2] = {wring + st * kStageBytes, wring + st1 * kStageBytes};
          const int nvs[2] = {nv0, nv1};
          int dist[2] = {0, 0};
          float* keep[2] = {nullptr, nullptr};
          if constexpr ((M & kBiased) != 0) {
            dist[0] = tab[j & 63].dist;
            dist[1] = tab[(j + 1) & 63].dist;
          }
          if constexpr ((M & kStored) != 0) {
            keep[0] = score_row(j);
            keep[1] = score_row(j + 1);
          }
          if (M != 0 ? nv0 == kPage && nv1 == kPage : (nv0 & nv1) == kPage)
            process_pages<2, true, F, M>(p, stg, nvs, dist, keep, s, g, t);
          else if ((nv0 | nv1) || (M & kStored) != 0)  // scores are kept of pages with a bad id, too (-inf)
            process_pages<2, false, F, M>(p, stg, nvs, dist, keep, s, g, t);
          __syncwarp();
          // refill the freed stages with items j + kStages and j + 1 + kStages
          const int ja = j + kStages, jb = ja + 1;
          if (jb < n) {
            const ItemEntry ea = tab[ja & 63], eb = tab[jb & 63];
            if constexpr (F == kFmtMxfp4) {
              issue_page_off<F, M>(lc, ea.off, ea.nv, wring_u32 + st * kStageBytes, wbar + 8 * st);
              issue_page_off<F, M>(lc, eb.off, eb.nv, wring_u32 + st1 * kStageBytes, wbar + 8 * st1);
            } else {
              issue_two_off<M>(lc, ea, eb, wring_u32 + st * kStageBytes, wring_u32 + st1 * kStageBytes,
                            wbar + 8 * st, wbar + 8 * st1, lane < 16);
            }
            issued = jb + 1;
          } else if (ja < n) {
            issue_page_off<F, M>(lc, tab[ja & 63].off, tab[ja & 63].nv, wring_u32 + st * kStageBytes, wbar + 8 * st);
            issued = ja + 1;
          }
        }
        st = st1 + 1 == kStages ? 0 : st1 + 1;
        ph = st == 0 ? ph1 ^ 1u : ph1;
      }
      if (j < iend) {
        // the piece's last page on its own
        NVFP4KV_ADVANCE_TO(j)
        if (!nres && (j & 31) >= 16) {
          NVFP4KV_RESOLVE_NXT();
          nres = true;
        }
        if (!stage_wait(wbar + 8 * st, ph)) goto timed_out;
        {
          const int nv0 = tab[j & 63].nv;
          const uint8_t* const stg[2] = {wring + st * kStageBytes, wring + st * kStageBytes};
          const int nvs[2] = {nv0, 0};
          int dist[2] = {0, 0};
          float* keep[2] = {nullptr, nullptr};
          if constexpr ((M & kBiased) != 0) dist[0] = tab[j & 63].dist;
          if constexpr ((M & kStored) != 0) keep[0] = score_row(j);
          if (nv0 || (M & kStored) != 0) process_pages<2, false, F, M>(p, stg, nvs, dist, keep, s, g, t);
          __syncwarp();
          const int ja = j + kStages;
          if (ja < n) {
            issue_page_off<F, M>(lc, tab[ja & 63].off, tab[ja & 63].nv, wring_u32 + st * kStageBytes, wbar + 8 * st);
            issued = ja + 1;
          }
        }
        st = st + 1 == kStages ? 0 : st + 1;
        ph = st == 0 ? ph ^ 1u : ph;
        ++j;
      }
#undef NVFP4KV_NEXT_EVENT
#undef NVFP4KV_ADVANCE_TO
#undef NVFP4KV_RESOLVE_NXT
      __syncwarp();
      // a piece that ends before the warp range does is complete unless it is the
      // first; a cut piece becomes record 2 gwarp (the warp's first piece) or
      // 2 gwarp + 1 (its last piece), merged later by combine_kernel
      const int last_page = page0 + (iend - i) - 1;
      const bool complete = page0 == 0 && last_page == np - 1;
      const int slot = (iend == n && nseg > 1) ? 1 : 0;
      finish_piece<F, M>(p, s, pair, complete, p.part + (2 * gwarp + slot) * kRecFloats, g, t);
      i = iend;
    }
    return;
  timed_out:
    // a wait gave up: flag it, wait (bounded) for every copy still in flight so
    // that none lands after the warp has gone, and leave; the call's outputs
    // are then unspecified, but every access stays in bounds
    if (lane == 0) flag_error(p.status, kDevErrTimeout);
    for (int jj = issued - kStages; jj < issued; ++jj) {
      if (jj < 0) continue;
      mbar_wait(wbar + 8 * (jj % kStages), (uint32_t)((jj / kStages) & 1));
    }
  }
}

// Merge the records of every pair the warp ranges cut: block = (pair, a chunk
// of its query heads), warp = (query head, record group), thread = 4 columns.
// Group k of a head takes records k, k + groups, ... with an online rescale,
// then group 0 merges the groups' partial results.  Launched as a
// programmatic dependent of decode_kernel: griddepcontrol.wait returns once
// the decode grid has finished and its writes are visible; what comes before
// it reads only the call's inputs.
constexpr int kCombineMaxGroups = 16;

__device__ __forceinline__ void online_merge(float& M, float& L, float4& acc, float m, float l, float4 v) {
  if (m == -INFINITY) {  // an empty record: only its m was written, the rest is whatever the scratch held
    l = 0.0f;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float Mn = fmaxf(M, m);
  const float a = M == -INFINITY ? 0.0f : ex2(M - Mn);
  const float b = m == -INFINITY ? 0.0f : ex2(m - Mn);
  L = L * a + l * b;
  acc.x = acc.x * a + v.x * b;
  acc.y = acc.y * a + v.y * b;
  acc.z = acc.z * a + v.z * b;
  acc.w = acc.w * a + v.w * b;
  M = Mn;
}

// The split's arithmetic in 32 bits, for W < 2^31 page-heads (the combine's use).
__device__ __forceinline__ int cta_start32(int c, int W, int N) {
  const int q = W / N, rem = W - q * N;
  return c * q + (c < rem ? c : rem);
}
__device__ __forceinline__ int warp_of_item32(int r, int W, int N) {
  const int q = W / N, rem = W - q * N, big = rem * (q + 1);
  const int c = r < big ? r / (q + 1) : rem + (r - big) / q;
  const int r0 = cta_start32(c, W, N), len = cta_start32(c + 1, W, N) - r0;
  return c * kNW + (int)(((long long)(r - r0 + 1) * kNW - 1) / len);
}

// A sequence's length as the decode clamps it (without flagging: the decode does).
__device__ __forceinline__ int clamped_len(const DecodeParams& p, int b) {
  const int L = __ldg(p.seq_lens + b), lmax = p.max_pages * kPage;
  return L < 0 ? 0 : (L > lmax ? lmax : L);
}

// Block = (pair, chunk of its query heads); warp = (head, record group).
constexpr int kCombineMaxWarps = 32;
constexpr int kCombineScanMax = 1024;  // batches up to this size: the combine sums the lengths itself

template <int F, int M>
__global__ void __launch_bounds__(kCombineMaxWarps * 32) combine_kernel(const DecodeParams p) {
  __shared__ float s_m[kCombineMaxWarps][32], s_l[kCombineMaxWarps][32];
  __shared__ float4 s_o[kCombineMaxWarps][32];
  __shared__ int s_info[3];  // first record, first warp, record count (0: nothing to merge)
  const int pair = blockIdx.x;
  const int b = pair / p.hkv, hh = pair - b * p.hkv;
  const int warp = threadIdx.x >> 5, col = threadIdx.x & 31;
  const int hb = p.comb_heads;                 // query heads per block
  const int groups = (blockDim.x >> 5) / hb;   // record groups per head
  const int hl = warp % hb, grp = warp / hb;
  const int head = blockIdx.y * hb + hl;
  // Where the pair lies in the decode's split, worked out by warp 0 in 32-bit
  // arithmetic (page-head indices stay below 2^31): the pages of the sequences
  // before b and of all sequences, then the warps holding the pair's first and
  // last page-heads.  For up to kCombineScanMax sequences the pages come from
  // the lengths, inputs of the call, so this runs while the decode is still
  // streaming; for more, from the prefix the decode's CTA 0 wrote (after the
  // wait), which keeps the work per block independent of the batch.
  const bool scan = p.batch <= kCombineScanMax;
  if (warp == 0) {
    int before = 0, total = 0;
    if (scan) {
      for (int i = col; i < p.batch; i += 32) {
        const int npi = visible_pages<M>(p, clamped_len(p, i)).count;
        total += npi;
        before += i < b ? npi : 0;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        total += __shfl_xor_sync(0xFFFFFFFFu, total, off);
        before += __shfl_xor_sync(0xFFFFFFFFu, before, off);
      }
    }
    if (col == 0) {
      const int np = visible_pages<M>(p, clamped_len(p, b)).count;
      int rec0 = 0, wf = 0, cnt = 0;
      if (np > 0) {
        if (!scan) {
          asm volatile("griddepcontrol.wait;" ::: "memory");
          before = __ldcg(p.cu_pages + b);
          total = __ldcg(p.cu_pages + p.batch);
        }
        const int W = total * p.hkv, N = p.ncta;
        const int P0 = before * p.hkv + hh * np;  // the pair's first page-head
        wf = warp_of_item32(P0, W, N);
        const int wl = warp_of_item32(P0 + np - 1, W, N);
        if (wl != wf) {
          // the first piece is warp wf's last piece (record 2 wf + 1), or its
          // only one when the pair starts wf's range (record 2 wf); every later
          // warp up to wl holds one piece as its first (record 2 w)
          const int cf = wf / kNW, r0c = cta_start32(cf, W, N), r1c = cta_start32(cf + 1, W, N);
          const int wr0 = r0c + (int)((long long)(r1c - r0c) * (wf - cf * kNW) / kNW);
          rec0 = 2 * wf + (P0 > wr0 ? 1 : 0);
          cnt = wl - wf + 1;
        }
      }
      s_info[0] = rec0;
      s_info[1] = wf;
      s_info[2] = cnt;
    }
  }
  __syncthreads();
  const int rec0 = s_info[0], wf = s_info[1], cnt = s_info[2];
  // The first block also with nothing to merge: what is launched behind the combine
  // (launch_overlapped, the accumulated weights) waits for the combine alone, which
  // therefore must not end before the decode.  (Where all blocks wait, those that the
  // GPU does not hold at once start after it: 256 sequences of a page 14.5 us, so 13.8.)
  if (cnt > 0 || (blockIdx.x | blockIdx.y) == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (cnt == 0) return;  // an empty sequence (the decode wrote its zeros) or one warp held the whole pair
  // warp (head, grp) merges the head's records grp, grp + groups, ...: four at
  // a time, all loads issued before any is used (a warp of the decode with no
  // items marked its record m = -inf)
  float mrun = -INFINITY, L = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (head < p.group) {
    for (int c0 = grp; c0 < cnt; c0 += 4 * groups) {
      float m[4], l[4];
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + i * groups;
        m[i] = -INFINITY;
        l[i] = 0.0f;
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < cnt) {
          const float* r = p.part + (c == 0 ? (long long)rec0 : 2LL * (wf + c)) * kRecFloats;
          m[i] = __ldcg(r + kOffM + head);
          l[i] = __ldcg(r + kOffL + head);
          v[i] = __ldcg(reinterpret_cast<const float4*>(r + head * kHeadDim) + col);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) online_merge(mrun, L, acc, m[i], l[i], v[i]);
    }
  }
  s_m[warp][col] = mrun;
  s_l[warp][col] = L;
  s_o[warp][col] = acc;
  __syncthreads();
  if (grp != 0 || head >= p.group) return;
  for (int k = 1; k < groups; ++k) {
    const int w2 = k * hb + hl;
    online_merge(mrun, L, acc, s_m[w2][col], s_l[w2][col], s_o[w2][col]);
  }
  const float sc = L > 0.0f ? p.v_gscale / L : 0.0f;
  float v[4] = {acc.x * sc, acc.y * sc, acc.z * sc, acc.w * sc};
  if constexpr (F == kFmtHadamard) {
    // rotate the merged output back (d bits 0-1 in the thread, 2-6 across the warp's 32 columns)
    const int xs[5] = {1, 2, 4, 8, 16};
    hadamard_lanes<4, 5>(v, xs, col);
  }
  const long long row = (long long)pair * p.group + head;
  if constexpr (M != 0) {
    reinterpret_cast<uint2*>(p.out16 + row * kHeadDim)[col] =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    if (col == 0) store_lse<M>(p, row, mrun, L);
  } else {
    reinterpret_cast<float4*>(p.out + row * kHeadDim)[col] = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// The decode over listed pages where one wave of CTAs holds it: a cluster of `splits`
// CTAs per (sequence, KV head) pair, each CTA an equal part of the pair's list, each
// warp an eighth of that, with the ring and the phases of decode_kernel.  The warps'
// results meet in shared memory and the CTAs' in that of the cluster (each CTA
// finishes every splits-th head, which the others store in its memory), so there are no records in global memory, no second
// kernel and no scan over the batch: what is left of them is some 6 us, beside 11 of
// decode_kernel and its combine, and the pages come at 5.7 TB/s and more.  Captured,
// 64 / 8 heads, here and there: 32 x 8193 tokens, 8 pages a head 6.3 and 11.3 us, 64
// 12.2 and 17.1, 256 32.4 and 35.8, 512 58.4 and 59.9; 37 x 8193, 512 58.9 and 66.5;
// 4 x 131073, 64 7.7, 1024 20.9 and 23.2, 4096 59.5 and 59.0.  Past one wave the even cut
// wins (96 sequences, 64 pages 37.8 and 32.9), and where the clusters leave SMs empty
// and lists are long: 1 x 131073, 256 pages 7.1 and 14.6, 1024 13.5 and 15.7, 2048 22.5 and 20.8.
// (Cutting several pairs of a cluster evenly over its warps, and 4 warps with three
// CTAs an SM, were both a tenth slower; the merge of cut pairs is what cost the first.)
constexpr int kSW = 8, kSelCtas = 2;  // warps of a CTA, CTAs of an SM
constexpr int kMaxSplits = 8;  // the portable cluster
// in shared memory: the warps' rings (and records), their barriers, the parts of the heads
// that this CTA finishes, from every CTA of the cluster
constexpr int kSelRingBytes = kSW * kStages * kStageBytes;
constexpr int kOffParts = kSelRingBytes + (kSW * kStages * 8 + 127) / 128 * 128;
constexpr int kPartFloats = kHeadDim + 4;
constexpr int kSelSmemBytes = kOffParts + (kGMax + kMaxSplits - 1) * kPartFloats * 4;
static_assert(kRecFloats * 4 <= kStages * kStageBytes, "a warp's record fits its ring");
static_assert(kSW >= kGMax && kSW <= 8 && kMaxSplits <= 8 && kHeadDim == 32 * 4, "a warp finishes a head of eight parts at most");

// The address of this shared memory in another CTA of the cluster; a store there.
__device__ __forceinline__ uint32_t map_cluster(const float* local, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  return at;
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t at, const float4& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
// The two halves of a barrier of the cluster's threads that orders no memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

__global__ void __launch_bounds__(kSW * 32, kSelCtas) selected_kernel(const DecodeParams p, int splits) {
  constexpr int F = kFmtNvfp4, M = kScored;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ItemEntry s_items[kSW][64];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int pair = blockIdx.x / splits, rank = blockIdx.x - pair * splits;
  const int b = pair / p.hkv, h = pair - b * p.hkv;
  if (splits > 1) cluster_arrive();
  after_earlier_kernels();
  const QRaw q = fetch_q<true>(p, pair, g, t);
  // the warp's part [w0, w0 + n) of a list of `listed` entries
  int w0, n;
  auto part = [&](int listed) {
    const int c0 = (int)((long long)listed * rank / splits), c1 = (int)((long long)listed * (rank + 1) / splits);
    w0 = c0 + (c1 - c0) * warp / kSW;
    n = c0 + (c1 - c0) * (warp + 1) / kSW - w0;
  };
  // the lane's entry of the part's 32-entry chunk k
  const int32_t* const list = p.selected + (long long)pair * p.budget;
  auto entry = [&](int k) { return 32 * k + lane < n ? list[w0 + 32 * k + lane] : -1; };
  // the first entries are read before the length is there, as if the list were full
  const int full = min(p.max_pages, p.budget);
  part(full);
  int sel0 = entry(0);
  const int L = clamp_len<true>(p, b), pages = (L + kPage - 1) / kPage, listed = min(pages, p.budget);
  if (listed != full) {
    part(listed);
    sel0 = entry(0);
  }
  const int32_t* const table = p.page_table + (long long)b * p.max_pages;
  uint8_t* const ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_u32 = smem_u32(ring);
  const uint32_t bar = smem_u32(smem + kSelRingBytes) + 8 * warp * kStages;
  ItemEntry* const tab = s_items[warp];

  // an entry's page id, and what the loop uses of it
  auto page_id = [&](int sel) {
    if (sel >= pages) flag_error(p.status, NVFP4KV_DEVERR_PAGE);
    return sel >= 0 && sel < pages ? table[sel] : -1;
  };
  auto put = [&](int k, int sel, int id) {
    const bool named = sel >= 0 && sel < pages, valid = named && id >= 0 && id < p.num_pages;
    if (named && !valid) flag_error(p.status, NVFP4KV_DEVERR_PAGE);
    ItemEntry e;
    e.off = valid ? ((long long)id * p.hkv + h) * kPageHeadBytes : 0;
    e.nv = valid ? min(L - sel * kPage, kPage) : 0;
    e.dist = 0;
    tab[(32 * k + lane) & 63] = e;
    __syncwarp();
  };

  WarpState s;
  if (n == 0) load_q<F, M>(p, q, s, pair, g, t);
  if (n > 0) {
    int sel1 = entry(1), sel2 = entry(2);  // of the next chunk and the one after it
    const int id0 = page_id(sel0);
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) mbar_init(bar + 8 * i, 32);
      fence_mbar_init();
    }
    __syncwarp();
    put(0, sel0, id0);
    int id1 = page_id(sel1);
    int chunk = 0;
    const LaneCopy lc = lane_copy<F>(p, lane);
    int issued = 0;
    auto issue = [&](int i) {
      const int st = i % kStages;
      issue_page_off<F, M>(lc, tab[i & 63].off, tab[i & 63].nv, ring_u32 + st * kStageBytes, bar + 8 * st);
      issued = i + 1;
    };
    for (int i = 0; i < min(n, kStages); ++i) issue(i);
    load_q<F, M>(p, q, s, pair, g, t);
    bool alive = true;
    for (int j = 0; j < n && alive; j += 2) {
      if ((j & 31) == 16 && 32 * (chunk + 1) < n) {
        // half way through the chunk: the next one's entries, and the loads of those behind it
        put(chunk + 1, sel1, id1);
        sel1 = sel2;
        id1 = page_id(sel1);
        sel2 = entry(chunk + 3);
        ++chunk;
      }
      const bool two = j + 1 < n;
      const int st0 = j % kStages, st1 = (j + 1) % kStages, last = two ? j + 1 : j;
      // a stage's barrier fires only after the lanes' earlier copies have landed too
      if (!stage_wait(bar + 8 * (last % kStages), (uint32_t)(last / kStages) & 1u)) {
        alive = false;
        break;
      }
      const int nv0 = tab[j & 63].nv, nv1 = two ? tab[(j + 1) & 63].nv : 0;
      const uint8_t* const stg[2] = {ring + st0 * kStageBytes, ring + (two ? st1 : st0) * kStageBytes};
      const int nvs[2] = {nv0, nv1}, dist[2] = {0, 0};
      float* keep[2] = {nullptr, nullptr};
      if (nv0 == kPage && nv1 == kPage)
        process_pages<2, true, F, M>(p, stg, nvs, dist, keep, s, g, t);
      else if (nv0 | nv1)
        process_pages<2, false, F, M>(p, stg, nvs, dist, keep, s, g, t);
      __syncwarp();
      const int ja = j + kStages, jb = ja + 1;
      if (jb < n) {
        issue_two_off<M>(lc, tab[ja & 63], tab[jb & 63], ring_u32 + st0 * kStageBytes, ring_u32 + st1 * kStageBytes,
                         bar + 8 * st0, bar + 8 * st1, lane < 16);
        issued = jb + 1;
      } else if (ja < n) {
        issue(ja);
      }
    }
    if (!alive) {
      // a wait gave up: flag it and let (bounded) every copy in flight land before the ring is used again
      if (lane == 0) flag_error(p.status, kDevErrTimeout);
      for (int i = max(issued - kStages, 0); i < issued; ++i) mbar_wait(bar + 8 * (i % kStages), (uint32_t)(i / kStages) & 1u);
    }
  }
  __syncwarp();
  // the warps' records, each in its own ring
  finish_piece<F, M>(p, s, pair, false, reinterpret_cast<float*>(ring), g, t);
  __syncthreads();
  // warp = head, lane = four dimensions: the head's parts, lane k < parts holding part
  // k's maximum and sum, o4(k) its four values
  auto merge = [&](int parts, float m, float l, auto o4, float& top, float& sum, float4& o) {
    top = lane < parts ? m : -INFINITY;
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    const float w = lane < parts && m != -INFINITY ? ex2(m - top) : 0.0f;
    sum = lane < parts ? w * l : 0.0f;
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    top = __shfl_sync(0xFFFFFFFFu, top, 0);
    sum = __shfl_sync(0xFFFFFFFFu, sum, 0);
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= parts) break;
      const float4 v = o4(k);
      const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
      o.x = fmaf(wk, v.x, o.x);
      o.y = fmaf(wk, v.y, o.y);
      o.z = fmaf(wk, v.z, o.z);
      o.w = fmaf(wk, v.w, o.w);
    }
  };
  auto put_out = [&](int head, float m, float l, const float4& o) {
    const long long row = (long long)pair * p.group + head;
    const float r = l > 0.0f ? p.v_gscale / l : 0.0f;
    reinterpret_cast<uint2*>(p.out16 + row * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(o.x * r, o.y * r), pack_bf16x2(o.z * r, o.w * r));
    if (lane == 0) store_lse<M>(p, row, m, l);
  };
  float* const parts = reinterpret_cast<float*>(smem + kOffParts);
  if (warp < p.group) {
    // part k: warp k's record
    auto rec = [&](int k) { return reinterpret_cast<const float*>(smem + k * kStages * kStageBytes); };
    const int k = lane < kSW ? lane : 0;
    float m, l;
    float4 o;
    merge(kSW, rec(k)[kOffM + warp], rec(k)[kOffL + warp],
          [&](int i) { return reinterpret_cast<const float4*>(rec(i) + warp * kHeadDim)[lane]; }, m, l, o);
    if (splits == 1) {
      put_out(warp, m, l, o);
    } else {
      // to the CTA that finishes the head
      cluster_wait();  // every CTA has started
      const uint32_t to = map_cluster(parts + (warp / splits * splits + rank) * kPartFloats, warp % splits);
      st_cluster_f32x4(to + 16 * lane, o);
      if (lane == 0) st_cluster_f32x4(to + 4 * kHeadDim, make_float4(m, l, 0.0f, 0.0f));
    }
  } else if (splits > 1) {
    cluster_wait();
  }
  if (splits > 1) {
    __syncwarp();
    cluster_sync();
    // part k: CTA k's; every splits-th head to a CTA
    const int head = rank + splits * warp;
    if (head < p.group) {
      const float* const mine = parts + warp * splits * kPartFloats;
      const int k = lane < splits ? lane : 0;
      float m, l;
      float4 o;
      merge(splits, mine[k * kPartFloats + kHeadDim], mine[k * kPartFloats + kHeadDim + 1],
            [&](int i) { return reinterpret_cast<const float4*>(mine + i * kPartFloats)[lane]; }, m, l, o);
      put_out(head, m, l, o);
    }
  }
}

// Accumulated attention weights: w[b][h][t] <- decay * w + sum over the KV
// head's query heads of 2^(score - lse), from the scores the decode kept and
// the pairs' log-sum-exps (base 2).  Memory-bound: per page-head 512 bytes of
// scores (G = 8) and 64 bytes of sums in and out, 84 MB in 16.8 us for 32 x 8193
// tokens and 8 KV heads (0.75 of the measured copy rate).  A warp takes a contiguous
// range of the decode's page-heads, as the scores lie, in runs of one pair's
// consecutive pages; lane = (token, half of the heads), several pages' loads in
// flight.  Launched behind the combine as its programmatic dependent.
constexpr int kWeightWarps = 8;      // per block
constexpr int kWeightBlocksPerSm = 6;
constexpr int kWeightUnroll = 4;

// kHalf query heads' scores of one token.
template <int kHalf>
__device__ __forceinline__ void load_scores(const float* src, float (&x)[kHalf]) {
  if constexpr (kHalf == 4) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(src));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else if constexpr (kHalf == 2) {
    const float2 v = __ldcs(reinterpret_cast<const float2*>(src));
    x[0] = v.x, x[1] = v.y;
  } else {
    x[0] = __ldcs(src);
  }
}

template <int kHalf>  // query heads per lane
__global__ void __launch_bounds__(kWeightWarps * 32) weights_kernel(const DecodeParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int token = lane >> 1, half = lane & 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long W = (long long)__ldcg(p.cu_pages + p.batch) * p.hkv;
  if (W > p.score_items) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    return;
  }
  const long long nwarps = (long long)gridDim.x * kWeightWarps, w = (long long)blockIdx.x * kWeightWarps + warp;
  const long long r1 = W * (w + 1) / nwarps;
  long long r = W * w / nwarps;
  if (r >= r1) return;
  // the sequence of page-head r: the last one whose first page-head is <= r (a
  // 32-way search of the page prefix)
  int b = 0;
  for (int hi = p.batch; hi - b > 1;) {
    const int step = (hi - b + 31) / 32, at = b + lane * step;
    const bool before = at < hi && (long long)__ldcg(p.cu_pages + at) * p.hkv <= r;
    b += (__popc(__ballot_sync(0xFFFFFFFFu, before)) - 1) * step;  // lane 0's always is
    hi = min(hi, b + step);
  }
  int L = clamped_len(p, b);
  VisiblePages v = visible_pages<kScored>(p, L);
  const int in = (int)(r - (long long)__ldcg(p.cu_pages + b) * p.hkv);
  int h = in / v.count, local = in - h * v.count;  // KV head, index among the pair's visited pages
  while (true) {
    // one run: pages [local, local + run) of the pair, consecutive in the sequence
    const long long pair = (long long)b * p.hkv + h;
    const int stop = (int)min((long long)(local < v.lead ? v.lead : v.count), local + (r1 - r));
    float lse[kHalf];  // +inf where nothing was visible or there is no such head
#pragma unroll
    for (int k = 0; k < kHalf; ++k) {
      const int head = half * kHalf + k;
      const float x = head < p.group ? __ldcg(p.lse2 + pair * p.group + head) : -INFINITY;
      lse[k] = x == -INFINITY ? INFINITY : x;
    }
    float* const sums = p.weights + pair * p.weight_stride;
    const int page = local < v.lead ? local : local + v.skip;  // the run's first page in the sequence
    const int limit = (int)min((long long)L, p.weight_stride);
    if (limit < L && (page + stop - local) * kPage > limit) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
    const float* src = p.scores + (r * (2 * kPage) + lane) * kHalf;
    int t = page * kPage + token;  // the lane's token
    for (int k = local; k < stop; k += kWeightUnroll) {
      float x[kWeightUnroll][kHalf], old[kWeightUnroll];
#pragma unroll
      for (int j = 0; j < kWeightUnroll; ++j) {
        old[j] = 0.0f;
        if (k + j < stop) {
          load_scores<kHalf>(src + j * (2 * kPage * kHalf), x[j]);
          if (half == 0 && t + j * kPage < limit && p.decay != 0.0f) old[j] = sums[t + j * kPage];
        } else {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) x[j][i] = -INFINITY;
        }
      }
#pragma unroll
      for (int j = 0; j < kWeightUnroll; ++j) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) sum += ex2(x[j][i] - lse[i]);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        if (half == 0 && k + j < stop && t + j * kPage < limit) sums[t + j * kPage] = fmaf(p.decay, old[j], sum);
      }
      src += kWeightUnroll * 2 * kPage * kHalf;
      t += kWeightUnroll * kPage;
    }
    if (v.skip > 0 && p.decay != 1.0f) {
      // the pages out of sight decay as well: to each page seen an equal share of them
      const long long f0 = (v.lead + (long long)v.skip * local / v.count) * kPage;
      const long long f1 = min((v.lead + (long long)v.skip * stop / v.count) * kPage, (long long)limit);
      for (long long f = f0 + lane; f < f1; f += 32) sums[f] = p.decay == 0.0f ? 0.0f : p.decay * sums[f];
    }
    r += stop - local;
    if (r >= r1) return;
    local = stop;
    if (local == v.count) {  // the next pair
      local = 0;
      if (++h == p.hkv) {
        h = 0;
        do L = clamped_len(p, ++b);
        while (L == 0);
        v = visible_pages<kScored>(p, L);
      }
    }
  }
}

}  // namespace

int decode_num_ctas(int num_sms) { return num_sms * kCtasPerSm; }

size_t decode_workspace_bytes(int num_sms, int32_t batch, int32_t num_kv_heads) {
  size_t rec = 2 * (size_t)decode_num_ctas(num_sms) * kNW * kRecFloats * sizeof(float);
  (void)num_kv_heads;
  rec = (rec + 255) / 256 * 256;
  return rec + ((size_t)batch + 1) * sizeof(int32_t);
}

size_t decode_workspace_bound(int num_sms, int32_t batch, int32_t num_q_heads) {
  return decode_workspace_bytes(num_sms, batch, num_q_heads);
}

namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Query heads of a group as the kept scores are laid out.
int score_heads_of(int group) { return group <= 2 ? 2 : group <= 4 ? 4 : 8; }

}  // namespace

size_t decode_weights_workspace_bytes(int num_sms, int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                      int64_t max_total_pages) {
  const size_t lse = up256((size_t)batch * num_q_heads * sizeof(float));
  const size_t row = (size_t)kPage * score_heads_of(num_q_heads / num_kv_heads) * sizeof(float);
  return up256(decode_workspace_bytes(num_sms, batch, num_kv_heads)) + lse +
         (size_t)max_total_pages * num_kv_heads * row;
}

namespace {

template <int F>
DecodeParams decode_params(const nvfp4kv_cache& c, const uint16_t* q, const int32_t* page_table, int32_t max_pages,
                           const int32_t* seq_lens, int32_t batch, int32_t num_q_heads, float softmax_scale,
                           void* workspace, int32_t* device_status, int num_sms) {
  DecodeParams p = {};
  p.pages = c.pages;
  p.num_pages = (int32_t)c.num_pages;
  p.hkv = c.num_kv_heads;
  p.q = q;
  p.page_table = page_table;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.batch = batch;
  p.hq = num_q_heads;
  p.group = num_q_heads / c.num_kv_heads;
  // MXFP4 has no global scales: its blocks carry power-of-two scales alone
  const float gk = F == kFmtMxfp4 ? 1.0f : c.k_global_scale, gv = F == kFmtMxfp4 ? 1.0f : c.v_global_scale;
  p.score_scale = softmax_scale * 1.4426950408889634f * gk;
  p.v_gscale = gv;
  p.ncta = decode_num_ctas(num_sms);
  p.part = static_cast<float*>(workspace);
  p.cu_pages = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) +
                                          up256(2 * (size_t)p.ncta * kNW * kRecFloats * sizeof(float)));
  p.status = device_status;
  return p;
}

// A launch that may start before the kernel ahead of it on the stream has
// finished (a programmatic dependent).
template <class K>
cudaError_t launch_dependent(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             const DecodeParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The decode and its combine.
template <int F, int M>
cudaError_t enqueue_decode(DecodeParams p, cudaStream_t stream, bool after_kernel) {
  // the shared-memory limit is an attribute of the function on each device
  static PerDeviceOnce attr_once;
  const cudaError_t ae = attr_once.run([] {
    return cudaFuncSetAttribute(decode_kernel<F, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (ae != cudaSuccess) return ae;
  const int num_ctas = p.ncta;
  cudaError_t e;
  if (after_kernel) {
    // a programmatic dependent of the kernel before it on the stream
    e = launch_dependent(decode_kernel<F, M>, dim3((unsigned)num_ctas), kNW * 32, kSmemBytes, stream, p);
  } else {
    decode_kernel<F, M><<<num_ctas, kNW * 32, kSmemBytes, stream>>>(p);
    e = cudaGetLastError();
  }
  const size_t pairs = (size_t)p.batch * (size_t)p.hkv;
  if (e != cudaSuccess || pairs == 0) return e;
  // the combine, as a programmatic dependent of the decode on the same stream
  // records per cut pair are about (warps / pairs) when the sequences are
  // alike: a record group per four to eight of them, up to 16 groups per head,
  // and as many of the pair's query heads per block as fit 32 warps
  const long long per_pair = (2LL * num_ctas * kNW) / (long long)pairs;
  int groups = 1;
  while (groups < kCombineMaxGroups && groups * 8 < per_pair) groups *= 2;
  const int hb = p.group < kCombineMaxWarps / groups ? p.group : kCombineMaxWarps / groups;
  p.comb_heads = hb;
  return launch_dependent(combine_kernel<F, M>, dim3((unsigned)pairs, (unsigned)((p.group + hb - 1) / hb)),
                          32 * hb * groups, 0, stream, p);
}

template <int F>
cudaError_t launch_decode_fmt(const nvfp4kv_cache& c, const uint16_t* q, float* out, const int32_t* page_table,
                              int32_t max_pages, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                              float softmax_scale, void* workspace, int32_t* device_status, int num_sms,
                              cudaStream_t stream, bool after_kernel) {
  DecodeParams p = decode_params<F>(c, q, page_table, max_pages, seq_lens, batch, num_q_heads, softmax_scale,
                                    workspace, device_status, num_sms);
  p.out = out;
  return enqueue_decode<F, 0>(p, stream, after_kernel);
}

template <int M>
cudaError_t enqueue_scored(const DecodeParams& p, cudaStream_t stream) {
  return enqueue_decode<kFmtNvfp4, M>(p, stream, false);
}

}  // namespace

cudaError_t launch_decode_scored(const nvfp4kv_cache& c, const uint16_t* q, uint16_t* out, float* lse,
                                 const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                                 int32_t batch, int32_t num_q_heads, float softmax_scale,
                                 const nvfp4kv_scoring& sc, const DecodeWeights* weights, void* workspace,
                                 int32_t* device_status, int num_sms, cudaStream_t stream) {
  DecodeParams p = decode_params<kFmtNvfp4>(c, q, page_table, max_pages, seq_lens, batch, num_q_heads,
                                            softmax_scale, workspace, device_status, num_sms);
  p.out16 = out;
  p.lse = lse;
  p.window = sc.window;
  p.sinks = sc.sinks;
  p.slopes = sc.slopes;
  int m = kScored;
  if (sc.softcap > 0.0f) {
    m |= kCapped;
    const double inner = (double)softmax_scale * (double)c.k_global_scale / (double)sc.softcap;
    p.cap_scale = (float)(inner < FLT_MAX ? inner : FLT_MAX);
    p.score_scale = (float)((double)sc.softcap * 1.4426950408889634);
  }
  if (sc.slopes != nullptr) m |= kBiased;
  if (weights == nullptr) {
    switch (m) {
      case kScored: return enqueue_scored<kScored>(p, stream);
      case kScored | kCapped: return enqueue_scored<kScored | kCapped>(p, stream);
      case kScored | kBiased: return enqueue_scored<kScored | kBiased>(p, stream);
      default: return enqueue_scored<kScored | kCapped | kBiased>(p, stream);
    }
  }
  uint8_t* at = static_cast<uint8_t*>(workspace) + up256(decode_workspace_bytes(num_sms, batch, p.hkv));
  p.lse2 = reinterpret_cast<float*>(at);
  p.scores = reinterpret_cast<float*>(at + up256((size_t)batch * num_q_heads * sizeof(float)));
  p.score_heads = score_heads_of(p.group);
  p.score_items = weights->max_total_pages * p.hkv;
  p.weights = weights->sums;
  p.weight_stride = weights->stride;
  p.decay = weights->decay;
  cudaError_t e;
  switch (m) {
    case kScored: e = enqueue_scored<kScored | kStored>(p, stream); break;
    case kScored | kCapped: e = enqueue_scored<kScored | kStored | kCapped>(p, stream); break;
    case kScored | kBiased: e = enqueue_scored<kScored | kStored | kBiased>(p, stream); break;
    default: e = enqueue_scored<kScored | kStored | kCapped | kBiased>(p, stream); break;
  }
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(num_sms * kWeightBlocksPerSm));
  auto kernel = p.score_heads == 8 ? weights_kernel<4> : p.score_heads == 4 ? weights_kernel<2> : weights_kernel<1>;
  return launch_dependent(kernel, grid, kWeightWarps * 32, 0, stream, p);
}

cudaError_t launch_decode_selected(const nvfp4kv_cache& c, const uint16_t* q, uint16_t* out, float* lse,
                                   const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                                   int32_t batch, int32_t num_q_heads, float softmax_scale, const int32_t* selected,
                                   int32_t budget, void* workspace, int32_t* device_status, int num_sms,
                                   cudaStream_t stream) {
  DecodeParams p = decode_params<kFmtNvfp4>(c, q, page_table, max_pages, seq_lens, batch, num_q_heads,
                                            softmax_scale, workspace, device_status, num_sms);
  p.out16 = out;
  p.lse = lse;
  p.selected = selected;
  p.budget = budget;
  // as many CTAs per pair (up to the largest cluster) as one wave holds
  const int64_t pairs = (int64_t)batch * p.hkv, slots = (int64_t)num_sms * kSelCtas;
  int splits = 1;
  while (splits < kMaxSplits && pairs * (splits + 1) <= slots) ++splits;
  // past one wave, or with more than 512 pages to a CTA (in proportion fewer where
  // SMs stay empty), the even cut over the whole device (both sides: selected_kernel)
  const int64_t ctas = pairs * splits, listed = budget < max_pages ? budget : max_pages;
  if (ctas > slots || listed * num_sms > 512 * splits * (ctas < num_sms ? ctas : num_sms))
    return enqueue_scored<kScored | kSelected>(p, stream);
  static PerDeviceOnce attr_once;
  const cudaError_t e = attr_once.run([] {
    return cudaFuncSetAttribute(selected_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmemBytes);
  });
  if (e != cudaSuccess) return e;
  return launch_overlapped(selected_kernel, ctas, kSW * 32, kSelSmemBytes, splits, stream, p, splits);
}

cudaError_t launch_decode(const nvfp4kv_cache& c, const uint16_t* q, float* out, const int32_t* page_table,
                          int32_t max_pages, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                          float softmax_scale, void* workspace, int32_t* device_status, int num_sms,
                          cudaStream_t stream, bool after_kernel) {
  return launch_decode_fmt<kFmtNvfp4>(c, q, out, page_table, max_pages, seq_lens, batch, num_q_heads, softmax_scale,
                                      workspace, device_status, num_sms, stream, after_kernel);
}

cudaError_t launch_decode_variant(int variant, const nvfp4kv_cache& c, const uint16_t* q, float* out,
                                  const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                                  int32_t batch, int32_t num_q_heads, float softmax_scale, void* workspace,
                                  int32_t* device_status, int num_sms, cudaStream_t stream) {
  if (variant == NVFP4KV_VARIANT_HADAMARD)
    return launch_decode_fmt<kFmtHadamard>(c, q, out, page_table, max_pages, seq_lens, batch, num_q_heads,
                                           softmax_scale, workspace, device_status, num_sms, stream, false);
  if (variant == NVFP4KV_VARIANT_MXFP4)
    return launch_decode_fmt<kFmtMxfp4>(c, q, out, page_table, max_pages, seq_lens, batch, num_q_heads,
                                        softmax_scale, workspace, device_status, num_sms, stream, false);
  // stochastic rounding writes the plain NVFP4 format
  return launch_decode_fmt<kFmtNvfp4>(c, q, out, page_table, max_pages, seq_lens, batch, num_q_heads, softmax_scale,
                                      workspace, device_status, num_sms, stream, false);
}

}  // namespace nvfp4kv
