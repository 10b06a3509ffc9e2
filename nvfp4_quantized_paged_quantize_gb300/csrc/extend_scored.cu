// extend_scored.cu -- extend attention over the FP8 workspace with scored
// attention: a tanh cap, a distance bias, a window with sinks, prefix and
// document masks, bf16 output and the log-sum-exp
// (nvfp4kv_extend_attention_scored).
//
// A CTA owns 256 query rows of one (sequence, KV head): two tiles of 128 rows
// (128 / G tokens x the G query heads of the KV head), so each K/V tile feeds
// 256 rows.  16 warps:
//   - Warps 0-3 and 4-7, a softmax group per row tile: one query row per
//     thread (TMEM lane = row).  They write the row of Q (f16) into shared
//     memory, then per key tile read the S row for its maximum.  A tile with
//     nothing masked, no bias and no score near its cap is left as it is; any
//     other is capped, biased and masked in the same pass and put back.  They run
//     the lazy base-2 online softmax (the running max moves only when it grows by
//     2^8, and O is then rescaled in TMEM), read the row once more for the
//     exponentials (and the cap, where the first pass left it), and write P (f16)
//     over the S columns just read.  At the end: O * s_ws(V) / l -> bf16.
//   - Warps 8-11 load the key tiles of the workspace (K and V alternately, one
//     of each in flight in registers), convert E4M3 -> f16 (exact) and store
//     them as B operands (K K-major, V MN-major) in a ring of five 32 KB slots.
//   - Warp 12 issues S_t = Q_t K^T (both operands in shared memory) and O_t +=
//     P_t V (P in TMEM), t = 0, 1, f32 accumulators; the whole warp runs the loop
//     and one lane's instructions take effect.  The order PV_0, S_0, PV_1, S_1 lets one group's softmax run while the tensor
//     core works for the other; MMAs execute in issue order, so S_t(i + 1) may
//     overwrite the columns that P_t(i) was read from, and the completion of
//     S_t(i + 1) implies that of PV_t(i).
// Registers: the softmax groups take what the loaders and the MMA group give
// back (setmaxnreg).  Nothing may spill: with 224 KB of shared memory in use there
// is next to no L1 left, and a spilled word comes back from L2 after some 400
// cycles.
// TMEM (512 columns): S_0 0-127, S_1 128-255 (P_t in the first 64 of S_t),
// O_0 256-383, O_1 384-511.
// What bounds it: the chain softmax -> P V -> S of a tile, which the other tile's
// hides in part, then the FMA pipe where scores are capped.  16384 + 2048 tokens,
// 64 / 8 heads: 1.27 ms capped, 0.99 ms plain (0.48 and 0.61 of the measured bf16
// rate; nvfp4kv_extend_attention, without any scoring, 1.49 ms), 1.43 ms biased
// (every tile is put back), 0.11 ms under a window of 1024.
// Key tiles that no query of the CTA sees are skipped, and workspace rows that
// none sees are zeros in shared memory, not read.  Every wait is bounded: a stalled pipeline flags
// NVFP4KV_DEVERR_TIMEOUT and drains its MMAs before the TMEM is freed.
#include "extend_tiles.cuh"
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"
#include "scoring.cuh"
#include "tcgen05.cuh"

namespace nvfp4kv {
namespace {

// the kernel's template argument
enum : int {
  kCapped = 1,  // scores through cap * tanh(s / cap)
  kBiased = 2   // minus slope * distance
};

enum : int { kFar, kNear, kAny };  // the cap's forms

constexpr int kTileM = 128;    // query rows per tile (TMEM lanes); a CTA takes two
constexpr int kTileN = 128;    // keys per K/V tile
constexpr int kRows = 2 * kTileM;
constexpr int kSoftmaxWarps = 8, kLoadWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kLoadWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;  // 512: the MMA warp's group is whole for setmaxnreg
constexpr uint32_t kTileBytes = kTileN * kHeadDim * 2;  // one f16 tile (of Q, K or V), 32 KB
constexpr uint32_t kSlotBytes = kTileBytes;
constexpr int kSlots = 5;                               // K/V ring
constexpr uint32_t kSmemBytes = 2 * kTileBytes + kSlots * kSlotBytes;  // 224 KB: one CTA per SM
constexpr uint32_t kTmemCols = 512, kTmemO = 256;
constexpr float kLazy = 8.0f;
constexpr uint64_t kWaitNs = 1000000000ull;
// registers: 512 threads are launched with 128 each, 65536 in all
constexpr int kSoftmaxRegs = 192, kLoadRegs = 104, kMmaRegs = 24;
static_assert(256 * kSoftmaxRegs + 128 * kLoadRegs + 128 * kMmaRegs <= 512 * 128, "register split");

struct ScoredParams {
  const uint16_t* q;
  const int64_t* cu_q;
  const uint8_t* ws_k;
  const uint8_t* ws_v;
  const int64_t* cu_prefix;
  const int32_t* prefix_lens;
  int32_t hq, hkv, group, log2_group;
  int32_t max_q_len;
  int64_t total_rows;
  float unit;                // base-2 score per unit of q . k (not capped)
  float out_scale;           // v_ws_scale
  CapPoly cap;               // capped: q . k -> base-2 score
  int32_t window, sinks;     // 0: no window
  const float* slopes;       // [hq], biased
  const int32_t* full_lens;  // [batch] or null
  const int32_t* doc_starts; // [total_q] or null
  uint16_t* out;
  float* lse;                // or null
  int32_t* status;
};

struct Barriers {
  uint64_t q_full;         // 8: the softmax warps
  uint64_t full[kSlots];   // 4: the load warps
  uint64_t empty[kSlots];  // 1: an MMA commit
  uint64_t s_full[2];      // 1: an MMA commit
  uint64_t p_full[2];      // 4: the group's softmax warps
  uint64_t drain;
};

// Tiles of Q, K and V in shared memory, in the 128-byte swizzle: atoms of 8 rows
// (queries or keys) x 64 head dims, the 16-byte chunk c (8 head dims) of row r
// stored at c ^ r; the row groups of one half of the head dims follow one another.
// For Q and K (contracted over head dims) this is the K-major form, for V (over
// keys) the MN-major one.
constexpr uint32_t kHalfD = kTileBytes / 2, kSBO8 = 1024;  // next 64 head dims, next 8 keys
__device__ __forceinline__ uint32_t tile_off(int row, int chunk) {  // chunk 0 .. 15
  return (uint32_t)(chunk >> 3) * kHalfD + (uint32_t)row * 128 + (((uint32_t)chunk ^ (uint32_t)row) & 7) * 16;
}

// Positions within a sequence are 32-bit: prefix and chunk together stay below
// 2^31 - 2^8 (a longer sequence is cut, and flagged).
constexpr int kMaxKeys = INT32_MAX - 255;

// The keys one query sees: low <= j < end, and (with a window) j >= near or
// j < sink_end.
struct KeyRange {
  int low, end, near, sink_end;
};

// The query at position pos of a sequence of `keys` tokens, whose first `full`
// positions every query sees and whose document starts at doc.
__device__ __forceinline__ KeyRange key_range(const ScoredParams& p, int keys, int pos, int full, int doc) {
  KeyRange r;
  r.low = min(max(doc, 0), keys);
  r.end = max(pos + 1, min(full, keys));
  r.near = r.low;
  r.sink_end = r.low;
  if (p.window > 0) {
    r.near = max(r.low, pos - p.window + 1);
    r.sink_end = r.low + min(p.sinks, keys - r.low);
  }
  return r;
}

// The first n of 32 bits.
__device__ __forceinline__ uint32_t first_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Of keys at .. at + 31, those outside the range (bit c: key at + c).
__device__ __forceinline__ uint32_t hidden_bits(const KeyRange& r, int at) {
  return ~first_bits(r.end - at) |
         (first_bits(r.near - at) & ~(first_bits(r.sink_end - at) & ~first_bits(r.low - at)));
}

// What the CTA's queries see, as the warps share it.  Without documents one
// range holds what any of them sees (their windows follow one another); with
// documents each query has its own, as the sinks of two documents may lie far
// apart and no query sees what is between them.
struct Sight {
  KeyRange all;             // without documents
  int ranges;               // 1, or one per query
  int keys, full;           // the sequence's tokens, the positions that every query sees
  int first_pos;            // of the queries
  int row_low, row_high;    // keys outside have no row in the workspace
  int steps;                // documents with sinks: the tiles to visit
  int32_t doc[kRows];       // document starts of the queries
};

// (Loops over the ranges are not unrolled: 20 KB more code cost a first call 4 us.)
__device__ __forceinline__ KeyRange sight_range(const ScoredParams& p, const Sight& s, int k) {
  return p.doc_starts != nullptr ? key_range(p, s.keys, s.first_pos + k, s.full, s.doc[k]) : s.all;
}

// The tiles [first, last] that hold a range's sinks (none: last is -1).
struct Tiles {
  int first, last;
};
__device__ __forceinline__ Tiles sink_tiles(const KeyRange& r) {
  const int stop = min(r.sink_end, r.end);
  Tiles t;
  t.first = r.low / kTileN;
  t.last = stop > r.low ? (stop - 1) / kTileN : -1;
  return t;
}

// The key tiles to visit: all from near_tile on (where the nearest key of any
// query's window or document lies), and before it those that hold a sink.
struct Visit {
  int steps;      // one at least
  int near_tile;
  int lead;       // without documents: tiles [0, lead) hold the sinks
};

__device__ __forceinline__ bool document_sinks(const ScoredParams& p) {
  return p.doc_starts != nullptr && p.window > 0 && p.sinks > 0;
}

// The first tile to visit from `from` on; warp-uniform.
__device__ __forceinline__ int next_tile(const ScoredParams& p, const Visit& v, const Sight& s, int from, int lane) {
  if (from >= v.near_tile) return from;
  if (!document_sinks(p)) return from < v.lead ? from : v.near_tile;
  int t = v.near_tile;
#pragma unroll 1
  for (int k = lane; k < s.ranges; k += 32) {
    const Tiles sinks = sink_tiles(sight_range(p, s, k));
    if (sinks.last >= from) t = min(t, max(from, sinks.first));
  }
  return __reduce_min_sync(0xFFFFFFFFu, t);
}

// For the queries of tokens [t0, t1] of a chunk behind a prefix of P tokens
// (every warp for itself; v.steps without the tiles of documents' sinks).  One
// warp keeps the document starts.
__device__ __forceinline__ Visit plan_visit(const ScoredParams& p, int64_t q0, int P, int keys, int t0, int t1,
                                            int full, KeyRange& all, int32_t* keep, int lane) {
  Visit v;
  v.lead = 0;
  int last;
  if (p.doc_starts == nullptr) {
    all = key_range(p, keys, P + t1, full, 0);
    all.near = key_range(p, keys, P + t0, full, 0).near;
    last = (all.end - 1) / kTileN;
    v.near_tile = all.near / kTileN;
    v.lead = min(sink_tiles(all).last + 1, v.near_tile);
  } else {
    int first = INT32_MAX;
    last = 0;
#pragma unroll 1
    for (int t = t0 + lane; t <= t1; t += 32) {
      const int doc = __ldg(p.doc_starts + q0 + t);
      if (keep != nullptr) keep[t - t0] = doc;
      const KeyRange r = key_range(p, keys, P + t, full, doc);
      if (r.low < r.end) {  // (else the query sees nothing)
        first = min(first, r.near);
        last = max(last, r.end - 1);
      }
    }
    last = __reduce_max_sync(0xFFFFFFFFu, last) / kTileN;
    v.near_tile = min(__reduce_min_sync(0xFFFFFFFFu, first) / kTileN, last);
  }
  v.steps = v.lead + last - v.near_tile + 1;
  return v;
}

// How many tiles before near_tile hold a document's sinks (one warp's work):
// run after run of tiles [t, stop] that sinks cover without a gap.
__device__ __forceinline__ int count_sink_tiles(const ScoredParams& p, const Visit& v, const Sight& s, int lane) {
  int count = 0;
  for (int t = next_tile(p, v, s, 0, lane); t < v.near_tile;) {
    int stop = t;
    while (true) {
      int reach = stop;
#pragma unroll 1
      for (int k = lane; k < s.ranges; k += 32) {
        const Tiles sinks = sink_tiles(sight_range(p, s, k));
        if (sinks.first <= stop + 1) reach = max(reach, sinks.last);
      }
      reach = min(__reduce_max_sync(0xFFFFFFFFu, reach), v.near_tile - 1);
      if (reach == stop) break;
      stop = reach;
    }
    count += stop - t + 1;
    t = next_tile(p, v, s, stop + 1, lane);
  }
  return count;
}

template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ uint32_t try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
      : "=r"(done) : "r"(bar), "r"(parity), "r"(1000000u) : "memory");
  return done;
}

// Wait for a phase with one outcome for the whole warp; false after about kWaitNs.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xFFFFFFFFu, try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (__all_sync(0xFFFFFFFFu, try_wait(bar, parity))) return true;
    if (__shfl_sync(0xFFFFFFFFu, global_timer_ns() - t0 > kWaitNs ? 1 : 0, 0)) return false;
  }
}

__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int M>
__global__ void __launch_bounds__(kThreads, 1) extend_scored_kernel(const ScoredParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Barriers bars;
  __shared__ uint32_t s_tmem;
  __shared__ Sight sight;

  // the broadcast tells the compiler that a warp's lanes take the same role
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int b = blockIdx.y, hk = blockIdx.z;
  const int tile_tokens = kTileM >> p.log2_group;

  // the sequence: chunk length C, prefix P, first workspace row
  const int64_t q0 = __ldg(p.cu_q + b);
  const int64_t chunk = __ldg(p.cu_q + b + 1) - q0;
  const int C = (int)min(max(chunk, (int64_t)0), (int64_t)min(p.max_q_len, kMaxKeys));
  const int prefix = __ldg(p.prefix_lens + b);
  const int P = min(max(prefix, 0), kMaxKeys - C);
  if ((C != chunk || P != prefix) && threadIdx.x == 0 && blockIdx.x == 0) flag_error(p.status, NVFP4KV_DEVERR_LENGTH);
  // the latest (longest) row blocks first
  const int64_t first_token = (int64_t)(gridDim.x - 1 - blockIdx.x) * 2 * tile_tokens;
  if (first_token >= C) return;  // no query
  const int t0 = (int)first_token, t1 = min(t0 + 2 * tile_tokens, C) - 1;
  const int keys = P + C;
  const int full = p.full_lens != nullptr ? __ldg(p.full_lens + b) : 0;

  const uint32_t sQ = smem_u32(smem), sRing = sQ + 2 * kTileBytes;
  const uint32_t b_q = smem_u32(&bars.q_full), b_full = smem_u32(&bars.full[0]), b_empty = smem_u32(&bars.empty[0]);
  const uint32_t b_s = smem_u32(&bars.s_full[0]), b_p = smem_u32(&bars.p_full[0]);  // [2], 8 bytes apart
  const uint32_t b_drain = smem_u32(&bars.drain);
  if (threadIdx.x == 0) {
    mbar_init(b_q, kSoftmaxWarps);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(b_full + 8 * s, kLoadWarps);
      mbar_init(b_empty + 8 * s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(b_s + 8 * t, 1);
      mbar_init(b_p + 8 * t, kSoftmaxWarps / 2);
    }
    mbar_init(b_drain, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc1::tmem_alloc(smem_u32(&s_tmem), kTmemCols);
  // bring the CTA's query rows (one 256-byte row per softmax thread) closer
  // while the rest is set up
  if (threadIdx.x < kRows) {
    const int64_t t = t0 + (threadIdx.x >> p.log2_group);
    if (t <= t1) {
      const uint16_t* q = p.q + ((q0 + t) * p.hq + hk * p.group + (threadIdx.x & (p.group - 1))) * kHeadDim;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
    }
  }
  KeyRange all = {};
  const bool keeps = warp == kMmaWarp + 1;
  const int64_t row0 = __ldg(p.cu_prefix + b);
  Visit v = plan_visit(p, q0, P, keys, t0, t1, full, all, keeps ? sight.doc : nullptr, lane);
  if (keeps) {
    if (lane == 0) {
      auto clamp_key = [](int64_t j) { return (int)(j < 0 ? 0 : (j > INT32_MAX ? INT32_MAX : j)); };
      sight.all = all;
      sight.ranges = p.doc_starts != nullptr ? t1 - t0 + 1 : 1;
      sight.keys = keys;
      sight.full = full;
      sight.first_pos = P + t0;
      sight.row_low = clamp_key(-row0);
      sight.row_high = clamp_key(p.total_rows - row0);
    }
    __syncwarp();
    if (document_sinks(p)) {
      const int sinks = count_sink_tiles(p, v, sight, lane);
      if (lane == 0) sight.steps = v.steps + sinks;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
  if (document_sinks(p)) v.steps = __shfl_sync(0xFFFFFFFFu, sight.steps, 0);
  const int G = p.group;

  if (warp >= kMmaWarp) {
    fewer_registers<kMmaRegs>();
    if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issue
      // The whole warp runs this loop (so that addresses and descriptors live in
      // uniform registers) and one lane's instructions take effect.
      constexpr uint32_t id_qk = tc::idesc_f16_f32(kTileM, kTileN, false, false);
      constexpr uint32_t id_pv = tc::idesc_f16_f32(kTileM, kHeadDim, false, true);
      const uint32_t lead = lane == 0;
      // shared-memory descriptors are a constant plus the address in their low word
      const uint64_t desc = tc::smem_desc_swizzle128(0, kHalfD, kSBO8);
      // the ring's items are K of step 0, V of step 0, K of step 1, ...: `at` is
      // the slot of the item in use, `round` the parity of its phase
      const int items = 2 * v.steps;
      int item = 0, at = 0;
      uint32_t round = 0;
      auto ready = [&]() { return warp_wait(b_full + 8 * at, round); };
      auto done = [&]() {  // free the slot for a later item, if there is one, and step on
        if (item + kSlots < items) tc1::commit(b_empty + 8 * at, lead);
        ++item;
        if (++at == kSlots) {
          at = 0;
          round ^= 1;
        }
      };
      auto scores = [&](int t, int slot) {  // S_t = Q_t K^T
        uint32_t q = (sQ + t * kTileBytes) >> 4, k = (sRing + slot * kSlotBytes) >> 4;
        asm volatile("" : "+r"(q));  // not worth 16 registers across the loop
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          // 16 head dims are 32 bytes of a row
          tc1::mma_f16(tmem + t * kTileN, desc | (q + (kk >> 2) * (kHalfD >> 4) + (kk & 3) * 2),
                       desc | (k + (kk >> 2) * (kHalfD >> 4) + (kk & 3) * 2), id_qk, kk > 0, lead);
        tc1::commit(b_s + 8 * t, lead);
      };
      bool ok = warp_wait(b_q, 0) && ready();
      if (ok) {
        tc::fence_after_sync();
        scores(0, 0);
        scores(1, 0);
        done();
      }
      for (int i = 0; i < v.steps && ok; ++i) {
        const bool more = i + 1 < v.steps;
        const int v_at = at, k_at = at + 1 == kSlots ? 0 : at + 1;  // V of this step, K of the next
        if (!(ok = ready())) break;
        if (more && !(ok = warp_wait(b_full + 8 * k_at, k_at == 0 ? round ^ 1 : round))) break;
        // PV_0, S_0 of the next step, PV_1, S_1 of the next step
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (!(ok = warp_wait(b_p + 8 * t, i & 1))) break;
          tc::fence_after_sync();
          const uint32_t vv = (sRing + v_at * kSlotBytes) >> 4;
#pragma unroll
          for (int kk = 0; kk < kTileN / 16; ++kk)
            tc1::mma_f16_tmem_a(tmem + kTmemO + t * kHeadDim, tmem + t * kTileN + kk * 8,
                                desc | (vv + kk * (2 * kSBO8 >> 4)), id_pv, (i > 0 || kk > 0) ? 1u : 0u, lead);
          if (t == 1) done();  // V
          if (more)
            scores(t, k_at);
          else
            tc1::commit(b_s + 8 * t, lead);  // O_t is complete
          if (t == 1 && more) done();  // K
        }
      }
      if (!ok && lane == 0) flag_error(p.status, NVFP4KV_DEVERR_TIMEOUT);
      // nothing this warp issued may still be running when the TMEM is freed
      tc1::commit(b_drain, lead);
      warp_wait(b_drain, 0);
    }
  } else if (warp >= kSoftmaxWarps) {
    // ------------------------------------------------------------ loaders
    fewer_registers<kLoadRegs>();
    // lane parts of a tile: key 32 lw + 4 g + lane / 8 (g < 8), its 16 bytes (head
    // dims) 16 (lane % 8): whole 128-byte rows per load
    const int lw = warp - kSoftmaxWarps, part = lane & 7;
    uint4 xk[8], xv[8];
    // this thread's first byte of key 0 in a workspace, and the bytes from key to key
    const int64_t key_bytes = (int64_t)p.hkv * kHeadDim;
    const int64_t key0 = (row0 * p.hkv + hk) * kHeadDim + part * 16;
    // Keys [whole_low, whole_high) are seen and have their rows, so that few tiles
    // take the long way.  With documents: what the query with the most near keys
    // sees, found while the first tile is on its way.
    int whole_low = max(all.near, sight.row_low), whole_high = min(all.end, sight.row_high);
    // of the warp's keys of a tile, those that some query sees and whose rows the workspace has
    auto rows_to_load = [&](int tile) {
      if (tile * kTileN >= whole_low && (tile + 1) * kTileN <= whole_high) return ~0u;
      const int at = tile * kTileN + 32 * lw;
      uint32_t seen = 0;
#pragma unroll 1
      for (int k = lane; k < sight.ranges; k += 32) seen |= ~hidden_bits(sight_range(p, sight, k), at);
      return __reduce_or_sync(0xFFFFFFFFu, seen) & first_bits(sight.row_high - at) & ~first_bits(sight.row_low - at);
    };
    int tile = next_tile(p, v, sight, 0, lane);
    uint32_t rows = rows_to_load(tile);
    auto load = [&](const uint8_t* ws, uint4 (&x)[8]) {
      const uint8_t* src = ws + (key0 + (tile * kTileN + lw * 32 + (lane >> 3)) * key_bytes);
      if (rows == ~0u) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          x[g] = __ldg(reinterpret_cast<const uint4*>(src));
          src += 4 * key_bytes;
        }
      } else {
        const uint32_t mine = rows >> (lane >> 3);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          x[g] = (mine >> (4 * g) & 1) ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
          src += 4 * key_bytes;
        }
      }
    };
    load(p.ws_k, xk);
    load(p.ws_v, xv);
    {
      KeyRange most = {0, 0, 0, 0};
      bool missing = false;
#pragma unroll 1
      for (int k = lane; k < sight.ranges; k += 32) {
        const KeyRange r = sight_range(p, sight, k);
        if (r.low >= r.end) continue;
        if (r.end - r.near > most.end - most.near) most = r;
        missing |= (r.sink_end > r.low ? r.low : r.near) < sight.row_low || r.end > sight.row_high;
      }
      if (missing) flag_error(p.status, NVFP4KV_DEVERR_ROW);
      if (p.doc_starts != nullptr) {
        const int keys_of = most.end - most.near, top = __reduce_max_sync(0xFFFFFFFFu, keys_of);
        const int of = __ffs(__ballot_sync(0xFFFFFFFFu, keys_of == top)) - 1;
        whole_low = __shfl_sync(0xFFFFFFFFu, most.near, of);
        whole_high = min(whole_low + top, sight.row_high);
        whole_low = max(whole_low, sight.row_low);
      }
    }
    bool ok = true;
    int s = 0;            // the ring slot
    uint32_t round = 1;   // the parity of its last release; its first use waits for none
    bool reuse = false;
    for (int i = 0; i < v.steps && ok; ++i) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {  // K, then V
        if (reuse && !warp_wait(b_empty + 8 * s, round)) {
          ok = false;
          break;
        }
        const uint32_t at = sRing + s * kSlotBytes;
        // a lane's 16 values are chunks 2 part and 2 part + 1; the upper four lanes
        // of a row store theirs the other way round, so that a row's eight lanes
        // hit eight banks
        const int first = part >> 2;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int key = lw * 32 + 4 * g + (lane >> 3);
          const uint4 x = w == 0 ? xk[g] : xv[g];
          const uint4 lo = e4m3x8_to_f16x8(x.x, x.y), hi = e4m3x8_to_f16x8(x.z, x.w);
          st_shared_v4(at + tile_off(key, 2 * part + first), first ? hi : lo);
          st_shared_v4(at + tile_off(key, 2 * part + 1 - first), first ? lo : hi);
        }
        tc::fence_smem_to_async();
        __syncwarp();
        if (lane == 0) arrive(b_full + 8 * s);
        if (++s == kSlots) {
          s = 0;
          round ^= 1;
          reuse = true;
        }
        if (i + 1 < v.steps) {
          if (w == 0) {
            tile = next_tile(p, v, sight, tile + 1, lane);
            rows = rows_to_load(tile);
            load(p.ws_k, xk);
          } else {
            load(p.ws_v, xv);
          }
        }
      }
    }
    if (!ok) flag_error(p.status, NVFP4KV_DEVERR_TIMEOUT);
  } else {
    // ------------------------------------------------------------ softmax rows
    more_registers<kSoftmaxRegs>();
    const int tile = warp >> 2, r = threadIdx.x & (kTileM - 1);  // the row tile, the row (TMEM lane)
    const int t = t0 + tile * tile_tokens + (r >> p.log2_group);
    const bool live = t <= t1;
    const int pos = P + t;
    const int head = hk * G + (r & (G - 1));
    {
      // the warp's 32 rows of Q, two whole rows per load
      const uint32_t dst = sQ + tile * kTileBytes;
#pragma unroll 8
      for (int i = 0; i < 16; ++i) {
        const int r2 = 32 * (warp & 3) + 2 * i + (lane >> 4);
        const int t2 = t0 + tile * tile_tokens + (r2 >> p.log2_group);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (t2 <= t1)
          x = __ldg(reinterpret_cast<const uint4*>(p.q + ((q0 + t2) * p.hq + hk * G + (r2 & (G - 1))) * kHeadDim) +
                    (lane & 15));
        st_shared_v4(dst + tile_off(r2, lane & 15), bf16x8_to_f16x8(x));
      }
      tc::fence_smem_to_async();
      __syncwarp();
      if (lane == 0) arrive(b_q);
    }
    KeyRange kr = key_range(p, keys, pos, full, p.doc_starts != nullptr && live ? __ldg(p.doc_starts + q0 + t) : 0);
    if (!live) kr.end = 0;  // a row past the chunk sees nothing
    const float slope = (M & kBiased) != 0 ? base2_slope(__ldg(p.slopes + head)) : 0.0f;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_s = t_lane + tile * kTileN, t_o = t_lane + kTmemO + tile * kHeadDim;
    const uint32_t bar_s = b_s + 8 * tile, bar_p = b_p + 8 * tile;
    float m = -INFINITY;
    float2 l[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    bool ok = true;
    int key_tile = -1;
    for (int i = 0; i < v.steps; ++i) {
      key_tile = next_tile(p, v, sight, key_tile + 1, lane);
      if (!warp_wait(bar_s, i & 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const int kbase = key_tile * kTileN;
      // keys c of [low, sink) and [near, end) of this tile are visible to the row
      const int end = kr.end - kbase, low = kr.low - kbase, sink = kr.sink_end - kbase, near = kr.near - kbase;
      const bool masked = end < kTileN || (near > 0 && (low > 0 || sink < kTileN));
      const bool any_masked = __any_sync(0xFFFFFFFFu, masked);
      // All visible, no bias, and no score beyond 0.6 of its cap: the row's maximum is
      // that of the products (the cap keeps the order), and the cap is left to the
      // second pass, where the FMA pipe works beside the special-function unit.
      bool direct = false;
      int form = kAny;        // the cap's
      uint32_t gone = 0;      // bit k: none of the warp's rows sees keys 32 k .. 32 k + 31
      float top = -INFINITY;  // the row's maximum in base 2
      if constexpr ((M & kBiased) == 0) {
        if (!any_masked) {
          uint32_t w[kTileN];
          tc::tmem_ld128(t_s, w);
          float hi[4], lo[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) hi[c] = lo[c] = __uint_as_float(w[c]);
#pragma unroll
          for (int c = 4; c < kTileN; c += 2) {
            const float a = __uint_as_float(w[c]), b = __uint_as_float(w[c + 1]);
            hi[c >> 1 & 3] = max3(hi[c >> 1 & 3], a, b);
            if constexpr (M == kCapped) lo[c >> 1 & 3] = min3(lo[c >> 1 & 3], a, b);
          }
          const float h = fmaxf(max3(hi[0], hi[1], hi[2]), hi[3]);
          if constexpr (M == kCapped) {
            const float l0 = fminf(min3(lo[0], lo[1], lo[2]), lo[3]);
            form = __all_sync(0xFFFFFFFFu, h <= p.cap.far && l0 >= -p.cap.far)     ? kFar
                   : __all_sync(0xFFFFFFFFu, h <= p.cap.near && l0 >= -p.cap.near) ? kNear
                                                                                    : kAny;
            const float2 zero = both(0.0f);
            top = (form == kFar ? cap_far(both(h), p.cap, zero) : cap_near(both(h), p.cap, zero)).x;
          } else {
            top = h * p.unit;  // (the unit is positive)
          }
          direct = M == 0 || form != kAny;
        }
      }
      if (!direct) {
        // cap, bias and mask the scores where they lie, 32 at a time, leaving out
        // the chunks that none of the warp's rows sees
        float mr[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int at = 0; at < kTileN; at += 32) {
          uint32_t hidden = 0;  // bit c: key at + c
          if (any_masked) {
            hidden = hidden_bits(kr, kbase + at);
            if (__all_sync(0xFFFFFFFFu, hidden == ~0u)) {
              gone |= 1u << (at / 32);
              continue;
            }
          }
          uint32_t w[32];
          tc::tmem_ld32(t_s + at, w);
          float2(&x)[16] = *reinterpret_cast<float2(*)[16]>(&w[0]);
          if constexpr ((M & kCapped) != 0) cap_scores(x, p.cap);
          if constexpr ((M & kBiased) != 0) {
            const float d0 = (float)(pos - kbase - at);
            const float unit = (M & kCapped) != 0 ? 1.0f : p.unit;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              x[c].x = fmaf(-slope, fabsf(d0 - (float)(2 * c)), x[c].x * unit);
              x[c].y = fmaf(-slope, fabsf(d0 - (float)(2 * c + 1)), x[c].y * unit);
            }
          }
          if (__any_sync(0xFFFFFFFFu, hidden != 0)) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (hidden >> c & 1) w[c] = 0xFF800000u;  // -inf
          }
          tc::tmem_st32_async(t_s + at, w);
#pragma unroll
          for (int c = 0; c < 16; ++c) mr[c & 3] = max3(mr[c & 3], x[c].x, x[c].y);
        }
        tc::tmem_wait_st();  // they are read again below
        top = fmaxf(fmaxf(mr[0], mr[1]), fmaxf(mr[2], mr[3])) * (M == 0 ? p.unit : 1.0f);
      }
      const bool grow = top > m + kLazy;  // false while nothing is visible (top = -inf)
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float alpha = grow ? ex2(m - top) : 1.0f;  // 0 on the first visible tile (m = -inf)
        if (grow) m = top;
        l[0] = mul2(l[0], both(alpha));
        l[1] = mul2(l[1], both(alpha));
        if (i > 0) {
          // S of this step is complete, so P V of the last one is: O is at rest
#pragma unroll 1
          for (int k = 0; k < kHeadDim / 16; ++k) {
            uint32_t o[16];
            tc::tmem_ld16(t_o + 16 * k, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tc::tmem_st16_async(t_o + 16 * k, o);
          }
        }
      }
      // p = 2^(x - m); masked scores are -inf and give 0, and so does every
      // score of a row that has seen nothing yet (m = -inf).  The scores are read
      // again, 32 at a time with the next 32 on their way: without a whole row in
      // registers the compiler keeps 16 pairs in flight instead of two or three.
      const float off = m > -INFINITY ? -m : -INFINITY;
      auto weights = [&](auto exponent) {
        uint32_t y[2][32], ph[2][16];
        auto chunk = [&](const uint32_t (&x)[32], uint32_t (&out)[16]) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float2 e = exponent(make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])));
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            out[c] = f16x2_bits(e.x, e.y);
            l[c & 1] = add2(l[c & 1], e);
          }
        };
        // P (two keys per column) goes over S columns already read: the A operand
        // of P V
        if (!any_masked) {
          // a chunk is stored one round late, under the next one's arithmetic
          tc::tmem_ld32_async(t_s, y[0]);
#pragma unroll
          for (int c4 = 0; c4 < kTileN / 32; ++c4) {
            tc::tmem_wait_ld(y[c4 & 1]);
            if (c4 + 1 < kTileN / 32) tc::tmem_ld32_async(t_s + 32 * (c4 + 1), y[(c4 + 1) & 1]);
            chunk(y[c4 & 1], ph[c4 & 1]);
            if (c4 > 0) tc::tmem_st16_async(t_s + 16 * (c4 - 1), ph[(c4 - 1) & 1]);
          }
          tc::tmem_st16_async(t_s + kTileN / 2 - 16, ph[1]);
        } else {  // (an edge tile: in a loop, which costs less to fetch than it loses)
#pragma unroll 1
          for (int at = 0; at < kTileN; at += 32) {
            if (gone >> (at / 32) & 1) {
#pragma unroll
              for (int c = 0; c < 16; ++c) ph[0][c] = 0;
            } else {
              tc::tmem_ld32(t_s + at, y[0]);
              chunk(y[0], ph[0]);
            }
            tc::tmem_st16_async(t_s + at / 2, ph[0]);
          }
        }
      };
      if constexpr (M == 0)
        weights([&](float2 s) { return fma2(s, both(p.unit), both(off)); });
      else if (M != kCapped || !direct)
        weights([&](float2 s) { return add2(s, both(off)); });
      else if (form == kFar)
        weights([&](float2 s) { return cap_far(s, p.cap, both(off)); });
      else
        weights([&](float2 s) { return cap_near(s, p.cap, both(off)); });
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(bar_p);
    }
    if (ok && warp_wait(bar_s, v.steps & 1)) {
      tc::fence_after_sync();
      const float sum = (l[0].x + l[1].x) + (l[0].y + l[1].y);
      const float inv = sum > 0.0f ? p.out_scale / sum : 0.0f;
      // (worked out again rather than kept over the loop)
      const int64_t row = (__ldg(p.cu_q + b) + (live ? pos - P : 0)) * p.hq + hk * G + (r & (G - 1));
      uint4* dst = reinterpret_cast<uint4*>(p.out + row * kHeadDim);
      if (live && p.lse != nullptr) p.lse[row] = sum > 0.0f ? (m + log2f(sum)) * kLn2 : -INFINITY;
#pragma unroll
      for (int c4 = 0; c4 < kHeadDim / 32; ++c4) {
        uint32_t w[32];
        tc::tmem_ld32(t_o + c4 * 32, w);
        if (live) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = pack_bf16x2(__uint_as_float(w[8 * j + 2 * k]) * inv, __uint_as_float(w[8 * j + 2 * k + 1]) * inv);
            dst[c4 * 4 + j] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    } else {
      flag_error(p.status, NVFP4KV_DEVERR_TIMEOUT);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc1::tmem_dealloc(tmem, kTmemCols);
}

template <int M>
cudaError_t enqueue(const ScoredParams& p, int32_t batch, cudaStream_t stream) {
  // the shared-memory limit is an attribute of the function on each device
  static PerDeviceOnce attr_once;
  const cudaError_t attr = attr_once.run([] {
    return cudaFuncSetAttribute(extend_scored_kernel<M>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  });
  if (attr != cudaSuccess) return attr;
  const int64_t blocks = ((int64_t)p.max_q_len * p.group + kRows - 1) / kRows;
  const dim3 grid((unsigned)blocks, (unsigned)batch, (unsigned)p.hkv);
  extend_scored_kernel<M><<<grid, kThreads, kSmemBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend_scored(const uint16_t* q, const int64_t* cu_q, int32_t max_q_len, const uint8_t* ws_k,
                                 const uint8_t* ws_v, const int64_t* cu_prefix, const int32_t* prefix_lens,
                                 int32_t batch, int64_t total_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                 float k_ws_scale, float v_ws_scale, float softmax_scale, const nvfp4kv_scoring& sc,
                                 const int32_t* full_lens, const int32_t* doc_starts, uint16_t* out, float* lse,
                                 int32_t* device_status, cudaStream_t stream) {
  ScoredParams p = {};
  p.q = q;
  p.cu_q = cu_q;
  p.ws_k = ws_k;
  p.ws_v = ws_v;
  p.cu_prefix = cu_prefix;
  p.prefix_lens = prefix_lens;
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.group = num_q_heads / num_kv_heads;
  while ((1 << p.log2_group) < p.group) ++p.log2_group;
  p.max_q_len = max_q_len;
  p.total_rows = total_rows;
  const double scale = (double)softmax_scale * (double)k_ws_scale;
  p.unit = (float)(scale * 1.4426950408889634);
  p.out_scale = v_ws_scale;
  if (sc.softcap > 0.0f) p.cap = cap_poly(scale / (double)sc.softcap, (double)sc.softcap * 1.4426950408889634);
  p.window = sc.window;
  p.sinks = sc.sinks;
  p.slopes = sc.slopes;
  p.full_lens = full_lens;
  p.doc_starts = doc_starts;
  p.out = out;
  p.lse = lse;
  p.status = device_status;
  if (sc.softcap > 0.0f)
    return sc.slopes ? enqueue<kCapped | kBiased>(p, batch, stream) : enqueue<kCapped>(p, batch, stream);
  return sc.slopes ? enqueue<kBiased>(p, batch, stream) : enqueue<0>(p, batch, stream);
}

}  // namespace nvfp4kv
