// norm_rope_append.cu -- the norms of queries and keys for each head, the
// position rotation, and the quantised append of the keys and values, in one
// pass over the projection's output (nvfp4kv_norm_rope_append; the append is
// "nvfp4-kv-cache-memory-wall", section 3, flow 1: new K/V are quantised on the
// way into the cache).
//
// Every row is 128 values of one (token, head).  For queries and keys
//   r = 1 / sqrt(sum(x^2) / 128 + eps),   y = (x r) w,
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the pairs (a, b)
// and y rounded to bf16; each step one rounded binary32 operation, the sum a
// tree of neighbours (x_0^2 + x_1^2) + (x_2^2 + x_3^2) ..., so the bytes of the
// cache are determined.  Queries are stored; keys, and values as they come, go
// through the blocks of quantize_append.cu to their slot.
//
// Eight lanes hold a row, 16 consecutive values each: a quantisation block, and
// with half-split pairs the partner's values lie one to four lanes away.  A warp
// takes four rows at a time and walks the flattened (token, head) list of its share,
// so that a token's cosines and sines, 128 bytes a lane, stay in registers over its
// heads.  Values go by token pairs, two groups of lanes to a unit, because a byte of
// V data holds two tokens.  Rows come through a ring of kStages stages of shared
// memory per warp (cp.async, no barrier but the warp's own), which keeps 64 KB in
// flight on an SM at two CTAs; products two to an instruction.
// HBM-bound on long inputs: 512 bytes per query row, 256 + 72 (+ 128 with the
// workspace) per key or value row, and the cosines once per token.
#include "fp8_quotient.cuh"
#include "nvfp4_block.cuh"
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;
constexpr int kNrCtasPerSm = 2;
constexpr int kStages = 4;            // rows in flight per 8-lane group
constexpr int kStageBytes = 4 * 256;  // four rows
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct NormRopeParams {
  NormRopeArgs a;
  WsScales ws;
  int32_t q_steps, k_steps, v_steps;  // of four rows each
};

// The steps [begin, end) of one kind that a warp takes: an equal share of them, or,
// where all kinds' steps together are no more than the warps, at most one, of one
// kind alone (`before`: the steps of the kinds before this one).
struct Steps {
  int begin, end;
};

__device__ __forceinline__ Steps share(const NormRopeParams& p, int steps, int before) {
  const int warp = (int)blockIdx.x * kNrWarps + (threadIdx.x >> 5), warps = (int)gridDim.x * kNrWarps;
  if ((long long)p.q_steps + p.k_steps + p.v_steps <= warps) {
    const int at = warp - before;
    return at >= 0 && at < steps ? Steps{at, at + 1} : Steps{0, 0};
  }
  return Steps{(int)((long long)steps * warp / warps), (int)((long long)steps * (warp + 1) / warps)};
}

// Where an 8-lane group is in a flattened list of `heads` per major index (a token,
// or a pair of tokens).
struct Walk {
  int major, head;
  __device__ __forceinline__ void start(long long at, int heads) {
    major = (int)(at / heads);
    head = (int)(at - (long long)major * heads);
  }
  __device__ __forceinline__ void skip(int by, int heads) {
    head += by;
    while (head >= heads) {
      head -= heads;
      ++major;
    }
  }
};

// One row's 16 values of a lane, as stored.
struct Row {
  uint4 a, b;
};

// A row's 16-byte piece q lies at piece_at(q) of its 256 bytes of a stage: the
// lanes of a group write pieces s and 8 + s (whole sectors of the row) and read 2 s
// and 2 s + 1, both without bank conflicts.
__device__ __forceinline__ int piece_at(int q) { return 16 * ((q & 1) ? 8 + ((q >> 1) ^ 4) : q >> 1); }

// Starts the copy of the group's row (nothing for a null one) into a stage.
__device__ __forceinline__ void fetch_row(uint32_t stage, const uint16_t* row, int lane) {
  const int sub = lane & 7;
  if (row != nullptr) {
    const uint32_t dst = stage + (lane >> 3) * 256;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(row) + 16 * sub;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + piece_at(sub)), "l"(src) : "memory");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + piece_at(8 + sub)), "l"(src + 128) : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// The oldest stage's row, once its copy (kStages - 1 later ones may be under way) has landed.
__device__ __forceinline__ Row take_row(const uint8_t* stage, int lane) {
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  __syncwarp();
  const uint8_t* r = stage + (lane >> 3) * 256;
  const int sub = lane & 7;
  Row x;
  x.a = *reinterpret_cast<const uint4*>(r + piece_at(2 * sub));
  x.b = *reinterpret_cast<const uint4*>(r + piece_at(2 * sub + 1));
  __syncwarp();  // the stage may be filled again
  return x;
}

// Two products per instruction.  Sums of products stay scalar: __fadd_rn is never
// merged with the products before it, where add.rn.f32x2 was (one query value in 50000 a
// bit off).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

__device__ __forceinline__ void unpack(const uint4& x, float2* f) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// The lane's cosines and signed sines of one token: value i of the lane turns as
// y_i cos_i + partner_i sin_i.
struct Turn {
  float2 cos[8], sin[8];
  bool on;  // the lane's values take part in the rotation
};

template <bool kInterleaved>
__device__ __forceinline__ void load_turn(const NormRopeArgs& p, int token, int sub, Turn& t) {
  const int pos = __ldg(p.positions + token);
  t.on = 16 * sub < p.rot;
  if (pos < 0 || pos >= p.max_position) {
    flag_error(p.status, NVFP4KV_DEVERR_POSITION);
    t.on = false;
  }
  if (!t.on) return;
  const int half = p.rot >> 1;
  const float* row = p.cos_sin + (long long)pos * p.rot;
  if constexpr (kInterleaved) {
    // pairs (2 i, 2 i + 1): angles 8 sub .. 8 sub + 7
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + 8 * sub) + j);
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + 8 * sub) + j);
      const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.cos[4 * j + i] = make_float2(cs[i], cs[i]);
        t.sin[4 * j + i] = make_float2(-sn[i], sn[i]);
      }
    }
  } else {
    // pairs (i, i + half): the first half's lanes hold a, the second's b
    const bool second = 16 * sub >= half;
    const int at = 16 * sub - (second ? half : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + at) + j);
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + at) + j);
      t.cos[2 * j] = make_float2(c.x, c.y);
      t.cos[2 * j + 1] = make_float2(c.z, c.w);
      t.sin[2 * j] = second ? make_float2(s.x, s.y) : make_float2(-s.x, -s.y);
      t.sin[2 * j + 1] = second ? make_float2(s.z, s.w) : make_float2(-s.z, -s.w);
    }
  }
}

// y = (x r) w over the eight lanes of a row.
__device__ __forceinline__ void normalise(float2 (&f)[8], const float2 (&w)[8], float eps) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 sq = mul2(f[i], f[i]);
    s[i] = __fadd_rn(sq.x, sq.y);
  }
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = __fadd_rn(s[2 * i], s[2 * i + 1]);
  float sum = s[0];
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, x));
  const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / kHeadDim), eps)));
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = mul2(mul2(f[i], make_float2(r, r)), w[i]);
}

template <bool kInterleaved>
__device__ __forceinline__ void rotate(float2 (&f)[8], const Turn& t, int lane, int rot) {
  if constexpr (kInterleaved) {
    if (t.on) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = add2(mul2(f[i], t.cos[i]), mul2(make_float2(f[i].y, f[i].x), t.sin[i]));
    }
  } else {
    const int sub = lane & 7, by = rot >> 5;  // lanes of half the rotated values
    const int from = sub < by ? lane + by : sub < 2 * by ? lane - by : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 o = make_float2(__shfl_sync(kAll, f[i].x, from), __shfl_sync(kAll, f[i].y, from));
      if (t.on) f[i] = add2(mul2(f[i], t.cos[i]), mul2(o, t.sin[i]));
    }
  }
}

// The lane's 16 bf16 values as 16 E4M3 bytes of workspace row `row`.
__device__ __forceinline__ void store_ws(const NormRopeParams& p, bool v, long long row, int head, int sub,
                                         const uint32_t (&w)[8]) {
  if (row < 0) return;
  if (row >= p.a.ws_total_rows) {
    flag_error(p.a.status, NVFP4KV_DEVERR_ROW);
    return;
  }
  const float s = v ? p.ws.sv : p.ws.sk, rs = v ? p.ws.rsv : p.ws.rsk;
  const bool fast = v ? p.ws.sv_fast : p.ws.sk_fast;
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    e[i] = e4m3x2_from_quotients(bf16_to_f32(w[i] & 0xFFFFu), bf16_to_f32(w[i] >> 16), s, rs, fast, p.ws.unit);
  uint8_t* ws = v ? p.a.ws_v : p.a.ws_k;
  reinterpret_cast<uint4*>(ws + (row * p.a.hkv + head) * kHeadDim)[sub] =
      make_uint4(e[0] | (e[1] << 16), e[2] | (e[3] << 16), e[4] | (e[5] << 16), e[6] | (e[7] << 16));
}

// The slot's page-head, null for padding and for a slot past the pool (flagged).
__device__ __forceinline__ uint8_t* page_head(const NormRopeArgs& p, long long slot, int head) {
  if (slot < 0) return nullptr;
  if (slot >= p.capacity) {
    flag_error(p.status, NVFP4KV_DEVERR_SLOT);
    return nullptr;
  }
  return p.pages + ((slot >> 4) * p.hkv + head) * kPageHeadBytes;
}

__device__ __forceinline__ void unpack_words(const uint32_t (&w)[8], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  }
}

// The warp's steps of the queries or of the keys.
template <bool kInterleaved, bool kKeys>
__device__ __forceinline__ void turn_rows(const NormRopeParams& p, Steps st, uint8_t* ring, int lane) {
  if (st.begin >= st.end) return;
  const NormRopeArgs& a = p.a;
  const int sub = lane & 7, heads = kKeys ? a.hkv : a.hq;
  const uint16_t* src = kKeys ? a.k : a.q;
  const long long stride = kKeys ? a.k_stride : a.q_stride;
  const uint16_t* weight = kKeys ? a.k_weight : a.q_weight;
  float2 w[8];
  if (weight) {
    unpack(__ldg(reinterpret_cast<const uint4*>(weight) + 2 * sub), w);
    unpack(__ldg(reinterpret_cast<const uint4*>(weight) + 2 * sub + 1), w + 4);
  }
  Walk at, ahead;
  at.start(4LL * st.begin + (lane >> 3), heads);
  ahead = at;
  int fetched = st.begin;  // the step that the next fetch is of
  const uint32_t ring_u32 = smem_u32(ring);
  auto fetch = [&](int stage) {
    const bool live = fetched < st.end && ahead.major < a.ntok;
    fetch_row(ring_u32 + stage * kStageBytes, live ? src + ahead.major * stride + ahead.head * kHeadDim : nullptr, lane);
    ahead.skip(4, heads);
    ++fetched;
  };
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) fetch(j);
  GlobalScale gs;
  if constexpr (kKeys) gs = global_scale(a.gk);
  Turn turn;
  turn.on = false;
  int turned = -1;  // the token that `turn` is of
  int stage = 0;
  for (int step = st.begin; step < st.end; ++step) {
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    const int tok = at.major, h = at.head;
    const bool live = tok < a.ntok;
    at.skip(4, heads);
    if (live && a.rot > 0 && tok != turned) {
      load_turn<kInterleaved>(a, tok, sub, turn);
      turned = tok;
    }
    const Row row = take_row(ring + stage * kStageBytes, lane);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float2 f[8];
    unpack(row.a, f);
    unpack(row.b, f + 4);
    if (weight) normalise(f, w, a.eps);
    if (a.rot > 0) rotate<kInterleaved>(f, turn, lane, a.rot);
    uint32_t y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = pack_bf16x2(f[k].x, f[k].y);
    if (!live) continue;
    if constexpr (kKeys) {
      if (a.ws_rows) store_ws(p, false, __ldg(a.ws_rows + tok), h, sub, y);
      const long long slot = __ldg(a.slots + tok);
      uint8_t* ph = page_head(a, slot, h);
      if (ph) {
        float x[16];
        unpack_words(y, x);
        const BlockCodes c = quantize_block(x, gs);
        const int rin = (int)(slot & (kPage - 1));
        reinterpret_cast<uint2*>(ph + kOffKData + rin * kRowBytes)[sub] = make_uint2(c.lo, c.hi);
        ph[k_scale_offset(rin, sub)] = (uint8_t)c.sb;
      }
    } else {
      uint4* dst = reinterpret_cast<uint4*>(a.q_out + tok * a.q_out_stride + h * kHeadDim) + 2 * sub;
      dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
      dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// The warp's steps of the values: two units of a token pair and a head each, two
// 8-lane groups to a unit.
__device__ __forceinline__ void value_rows(const NormRopeParams& p, Steps st, uint8_t* ring, int lane) {
  if (st.begin >= st.end) return;
  const NormRopeArgs& a = p.a;
  const int sub = lane & 7, which = (lane >> 3) & 1;
  const GlobalScale gs = global_scale(a.gv);
  Walk at, ahead;
  at.start(2LL * st.begin + (lane >> 4), a.hkv);
  ahead = at;
  int fetched = st.begin;
  const uint32_t ring_u32 = smem_u32(ring);
  auto fetch = [&](int stage) {
    const int tok = 2 * ahead.major + which;
    const bool live = fetched < st.end && ahead.major < (a.ntok + 1) >> 1 && tok < a.ntok;
    fetch_row(ring_u32 + stage * kStageBytes, live ? a.v + tok * a.v_stride + ahead.head * kHeadDim : nullptr, lane);
    ahead.skip(2, a.hkv);
    ++fetched;
  };
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) fetch(j);
  int stage = 0;
  for (int step = st.begin; step < st.end; ++step) {
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    const int tok = 2 * at.major + which, h = at.head;
    const bool live = at.major < (a.ntok + 1) >> 1 && tok < a.ntok;
    at.skip(2, a.hkv);
    const long long slot = live ? __ldg(a.slots + tok) : -1;
    const long long mate = live && (tok ^ 1) < a.ntok ? __ldg(a.slots + (tok ^ 1)) : -1;
    const Row row = take_row(ring + stage * kStageBytes, lane);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const uint32_t y[8] = {row.a.x, row.a.y, row.a.z, row.a.w, row.b.x, row.b.y, row.b.z, row.b.w};
    float f[16];
    unpack_words(y, f);
    const BlockCodes c = quantize_block(f, gs);
    // the pair's other token (lane ^ 8 holds the same block of it)
    const uint32_t plo = __shfl_xor_sync(kAll, c.lo, 8), phi = __shfl_xor_sync(kAll, c.hi, 8);
    if (!live) continue;
    if (a.ws_rows) store_ws(p, true, __ldg(a.ws_rows + tok), h, sub, y);
    uint8_t* ph = page_head(a, slot, h);
    if (!ph) continue;
    const int rin = (int)(slot & (kPage - 1));
    const long long even = which ? mate : slot, odd = which ? slot : mate;
    if ((even & 1) == 0 && odd == even + 1) {
      if (which == 0) v_store_block_pair(ph + kOffVData, rin >> 1, sub, c.lo, c.hi, plo, phi);
    } else {
      v_store_block_one(ph + kOffVData, rin, sub, c.lo, c.hi);
    }
    ph[v_scale_offset(rin, sub)] = (uint8_t)c.sb;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads, kNrCtasPerSm) norm_rope_kernel(const NormRopeParams p) {
  __shared__ __align__(128) uint8_t rings[kNrWarps][kStages * kStageBytes];
  const int lane = threadIdx.x & 31;
  uint8_t* ring = rings[threadIdx.x >> 5];
  turn_rows<kInterleaved, true>(p, share(p, p.k_steps, 0), ring, lane);
  value_rows(p, share(p, p.v_steps, p.k_steps), ring, lane);
  turn_rows<kInterleaved, false>(p, share(p, p.q_steps, p.k_steps + p.v_steps), ring, lane);
}

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeArgs& args, float k_ws_scale, float v_ws_scale, int num_sms,
                                    cudaStream_t stream) {
  NormRopeParams p;
  p.a = args;
  p.ws = ws_scales(k_ws_scale, v_ws_scale);
  auto steps = [](int64_t n, int per) { return (int32_t)((n + per - 1) / per); };
  p.q_steps = steps((int64_t)args.ntok * args.hq, 4);
  p.k_steps = steps((int64_t)args.ntok * args.hkv, 4);
  p.v_steps = steps((int64_t)((args.ntok + 1) / 2) * args.hkv, 2);
  const int64_t all = (int64_t)p.q_steps + p.k_steps + p.v_steps, fit = (int64_t)num_sms * kNrCtasPerSm;
  const int64_t need = (all + kNrWarps - 1) / kNrWarps;
  const unsigned blocks = (unsigned)(need < fit ? need : fit);
  if (args.interleaved)
    norm_rope_kernel<true><<<blocks, kNrThreads, 0, stream>>>(p);
  else
    norm_rope_kernel<false><<<blocks, kNrThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
