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
// Eight lanes hold a row: lane s has values 8 s .. 8 s + 7 and 64 + 8 s .., so that
// its loads and stores are whole sectors, the partners of a rotation of all 128
// values (in either order of pairs) are in one lane, and a quantisation block in
// two neighbours.  A step is four heads of one token, all queries or all keys (the
// last one of either may have fewer), and a warp walks its share of the list of every
// token's steps: what a step does is the same over the warp, a token's cosines and
// sines stay in registers over its steps, and every warp has its part of the keys'
// arithmetic and of the queries' bytes.  Values go by two heads of a token pair,
// because a byte of V data holds two tokens.
// Rows come through a ring of kStages stages of shared memory per warp (cp.async; a
// lane reads what it copied itself, so without any barrier), which keeps 96 KB in
// flight on an SM at three CTAs; products two to an instruction.
// HBM-bound on long inputs: 512 bytes per query row, 256 + 72 (+ 128 with the
// workspace) per key or value row, and the cosines once per token.  12.7 thousand tokens
// of 64 / 8 heads with workspace rows take 91 us, 5.6 TB/s (a warp per row with a piece
// of four values to a lane: 154; lists of rows of mixed kinds: 107); 32 tokens 3.1.
#include "fp8_quotient.cuh"
#include "nvfp4_block.cuh"
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_launch.h"

namespace nvfp4kv {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;
constexpr int kStages = 4;            // rows in flight per 8-lane group
constexpr int kStageBytes = 4 * 256;  // four rows
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct NormRopeParams {
  NormRopeArgs a;
  WsScales ws;
  int32_t q_steps, k_steps;  // of one token
  int32_t v_steps;           // of one token pair
  int32_t t_all, v_all;      // of all tokens, of all pairs
};

// The steps [begin, end) of one kind that a warp takes: an equal share of them, or,
// where both kinds' steps together are no more than the warps, at most one, of one
// kind alone (`before`: the steps of the kind before this one).
struct Steps {
  int begin, end;
};

__device__ __forceinline__ Steps share(const NormRopeParams& p, int warp_in_block, int steps, int before) {
  const int warp = (int)blockIdx.x * kNrWarps + warp_in_block, warps = (int)gridDim.x * kNrWarps;
  if ((long long)p.t_all + p.v_all <= warps) {
    const int at = warp - before;
    return at >= 0 && at < steps ? Steps{at, at + 1} : Steps{0, 0};
  }
  return Steps{(int)((long long)steps * warp / warps), (int)((long long)steps * (warp + 1) / warps)};
}

// Starts the copy of the lane's two pieces of a row (none if it is not live) into a
// stage: [half][lane][16 bytes].
__device__ __forceinline__ void fetch_row(uint32_t stage, const uint16_t* row, bool live) {
  asm volatile(
      "{\n .reg .pred p;\n"
      " setp.ne.u32 p, %2, 0;\n"
      " @p cp.async.cg.shared.global [%0], [%1], 16;\n"
      " @p cp.async.cg.shared.global [%0+512], [%1+128], 16;\n"
      " cp.async.commit_group;\n"
      "}\n" ::"r"(stage), "l"(row), "r"((uint32_t)live)
      : "memory");
}

// The lane's values of the oldest stage's row, as stored, once its copy (kStages - 1
// later ones may be under way) has landed: words 0-3 values 8 s .., 4-7 64 + 8 s ...
__device__ __forceinline__ void take_row(const uint8_t* stage, uint32_t (&w)[8]) {
  asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  const uint4 a = *reinterpret_cast<const uint4*>(stage), b = *reinterpret_cast<const uint4*>(stage + 512);
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// Two products per instruction.  Sums of products stay scalar: __fadd_rn is never
// merged with the products before it, where add.rn.f32x2 was (one query value in
// 50000 a bit off).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 shfl2(float2 a, int from) {
  return make_float2(__shfl_sync(kAll, a.x, from), __shfl_sync(kAll, a.y, from));
}

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// How the pairs of a rotation lie over the lanes.
enum Rotation : int {
  kNone,         // no rotation
  kWhole,        // halves, all 128 values: (8 s + i, 64 + 8 s + i), one lane's two pieces
  kFirst,        // halves of the first 32 or 64 values: the first pieces of lanes s and s ^ (rotary_dim / 16)
  kThreeQuarters,// halves of the first 96: pieces of different lanes and places
  kInterleaved   // (2 i, 2 i + 1)
};

// CTAs of an SM: three at 80 registers, two where the pieces of a pair need more.
__host__ __device__ constexpr int ctas_per_sm(int R) { return R == kThreeQuarters ? 2 : 3; }

// The lane's cosines and sines of one token: value i of piece h turns as
// y_i cos[h]_i + partner_i sin[h]_i, the sine's sign taken in.  kWhole: both pieces
// have the angles of cos[0], sin[0].
struct Turn {
  float2 cos[2][4], sin[2][4];
  bool on[2];  // the piece takes part
};

__device__ __forceinline__ void load4x2(const float* src, float2 (&d)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(src), b = reinterpret_cast<const float4*>(src)[1];
  d[0] = make_float2(a.x, a.y), d[1] = make_float2(a.z, a.w), d[2] = make_float2(b.x, b.y), d[3] = make_float2(b.z, b.w);
}

template <int R>
__device__ __forceinline__ void load_turn(const NormRopeArgs& p, int token, int sub, Turn& t) {
  const int pos = p.positions[token];
  const bool good = pos >= 0 && pos < p.max_position;
  if (!good) flag_error(p.status, NVFP4KV_DEVERR_POSITION);
  const int half = p.rot >> 1;
  const float* row = p.cos_sin + (long long)(good ? pos : 0) * p.rot;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = 64 * h + 8 * sub;  // the piece's first value
    t.on[h] = good && d < p.rot;
    if (!t.on[h]) continue;
    if constexpr (R == kInterleaved) {
      const float4 c = *reinterpret_cast<const float4*>(row + d / 2);
      const float4 s = *reinterpret_cast<const float4*>(row + half + d / 2);
      const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.cos[h][i] = make_float2(cs[i], cs[i]);
        t.sin[h][i] = make_float2(-sn[i], sn[i]);
      }
    } else if (R != kWhole || h == 0) {
      const bool second = d >= half;
      const int at = d - (second ? half : 0);
      load4x2(row + at, t.cos[h]);
      load4x2(row + half + at, t.sin[h]);
      if (R != kWhole && !second) {
#pragma unroll
        for (int i = 0; i < 4; ++i) t.sin[h][i] = neg2(t.sin[h][i]);
      }
    }
  }
}

// The norms' weights in fp32, those of the queries and of the keys: [tensor][piece]
// [half of the piece][lane of the group][4], so that a group's reads have no bank
// conflicts.  Ones without a weight.
using Weights = float4[2][2][2][8];

__device__ __forceinline__ void load_weights(const NormRopeArgs& a, Weights& w) {
  if (threadIdx.x < 2 * 2 * 2 * 8) {
    const int s = threadIdx.x & 7, half = threadIdx.x >> 3 & 1, h = threadIdx.x >> 4 & 1, keys = threadIdx.x >> 5;
    const uint16_t* src = keys ? a.k_weight : a.q_weight;
    float4 v = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (src) {
      const uint2 x = *reinterpret_cast<const uint2*>(src + 64 * h + 8 * s + 4 * half);
      const float2 lo = unpack2(x.x), hi = unpack2(x.y);
      v = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    w[keys][h][half][s] = v;
  }
}

// y = (x r) w over the eight lanes of a row; a row that is not `normed` has r and
// weights of 1, which change nothing.
__device__ __forceinline__ void normalise(float2 (&f)[8], const Weights& w, int keys, int sub, bool normed, float eps) {
  float sum[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 sq = mul2(f[4 * h + i], f[4 * h + i]);
      s[i] = __fadd_rn(sq.x, sq.y);
    }
    sum[h] = __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) sum[h] = __fadd_rn(sum[h], __shfl_xor_sync(kAll, sum[h], x));
  }
  float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(__fadd_rn(sum[0], sum[1]), 1.0f / kHeadDim), eps)));
  r = normed ? r : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = w[keys][i >> 1][i & 1][sub];
    f[2 * i] = mul2(mul2(f[2 * i], make_float2(r, r)), make_float2(v.x, v.y));
    f[2 * i + 1] = mul2(mul2(f[2 * i + 1], make_float2(r, r)), make_float2(v.z, v.w));
  }
}

__device__ __forceinline__ void turn4(float2* f, const float2 (&o)[4], const float2 (&cos)[4], const float2 (&sin)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = add2(mul2(f[i], cos[i]), mul2(o[i], sin[i]));
}

template <int R>
__device__ __forceinline__ void rotate(float2 (&f)[8], const Turn& t, int lane, int rot) {
  const int sub = lane & 7;
  if constexpr (R == kWhole) {
    if (t.on[0]) {  // (on[1] is the same)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = f[i], b = f[4 + i];
        f[i] = add2(mul2(a, t.cos[0][i]), neg2(mul2(b, t.sin[0][i])));
        f[4 + i] = add2(mul2(b, t.cos[0][i]), mul2(a, t.sin[0][i]));
      }
    }
  } else if constexpr (R == kFirst) {
    float2 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = shfl2(f[i], lane ^ (rot >> 4));
    if (t.on[0]) turn4(f, o, t.cos[0], t.sin[0]);
  } else if constexpr (R == kThreeQuarters) {
    // 48 apart: first pieces of lanes 0, 1 and 6, 7; first pieces of lanes 2 .. 5 and second ones of 0 .. 3
    float2 far[4], low[4], high[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      far[i] = shfl2(f[i], sub < 2 ? lane + 6 : sub > 5 ? lane - 6 : lane);
      low[i] = shfl2(f[i], sub < 4 ? lane + 2 : lane);       // for the second pieces of lanes 0 .. 3
      high[i] = shfl2(f[4 + i], sub >= 2 ? lane - 2 : lane);  // for the first pieces of lanes 2 .. 5
      if (sub >= 2 && sub <= 5) far[i] = high[i];
    }
    if (t.on[0]) turn4(f, far, t.cos[0], t.sin[0]);
    if (t.on[1]) turn4(f + 4, low, t.cos[1], t.sin[1]);
  } else if constexpr (R == kInterleaved) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!t.on[h]) continue;
      float2 o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = make_float2(f[4 * h + i].y, f[4 * h + i].x);
      turn4(f + 4 * h, o, t.cos[h], t.sin[h]);
    }
  }
}

// The lane's 16 bf16 values as E4M3 bytes of workspace row `row`.
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
  uint2* dst = reinterpret_cast<uint2*>((v ? p.a.ws_v : p.a.ws_k) + (row * p.a.hkv + head) * kHeadDim) + sub;
  dst[0] = make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
  dst[8] = make_uint2(e[4] | (e[5] << 16), e[6] | (e[7] << 16));
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

// The codes and scales of the lane's two half blocks: piece h is half of block
// sub / 2 + 4 h, whose other half the neighbour lane has.  Every lane calls this.
struct HalfBlocks {
  uint32_t codes[2], sb[2];
};
__device__ __forceinline__ HalfBlocks quantize_halves(const uint32_t (&w)[8], const GlobalScale& gs) {
  HalfBlocks q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2(w[4 * h + i]);
      f[2 * i] = x.x, f[2 * i + 1] = x.y;
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
    amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
    const BlockScale b = block_scale<true>(amax, gs);
    uint32_t c[1];
    block_codes<true>(f, amax, b, c);
    q.codes[h] = c[0];
    q.sb[h] = b.sb;
  }
  return q;
}

// The warp's steps of the queries and keys.
template <int R>
__device__ __forceinline__ void turn_rows(const NormRopeParams& p, Steps st, uint8_t* ring, const Weights& weights, int lane) {
  if (st.begin >= st.end) return;
  const NormRopeArgs& a = p.a;
  const int sub = lane & 7, group = lane >> 3, steps = p.q_steps + p.k_steps;
  const bool norms = a.q_weight || a.k_weight;
  // the lane's first value of head 4 j + group of a token, j counting its steps
  auto row_of = [&](int token, int j) {
    return (j < p.q_steps ? a.q + token * a.q_stride + 4 * j * kHeadDim
                          : a.k + token * a.k_stride + 4 * (j - p.q_steps) * kHeadDim) + group * kHeadDim + 8 * sub;
  };
  auto live_at = [&](int j) { return j < p.q_steps ? 4 * j + group < a.hq : 4 * (j - p.q_steps) + group < a.hkv; };
  int token = st.begin / steps, j = st.begin - token * steps;
  // the fetches run kStages - 1 steps ahead
  int left = st.end - st.begin, next_token = token, next_j = j;
  const uint16_t* next = row_of(token, j);
  const uint32_t ring_u32 = smem_u32(ring) + 16 * lane;
  auto fetch = [&](int stage) {
    fetch_row(ring_u32 + stage * kStageBytes, next, left > 0 && live_at(next_j));
    --left;
    next += 4 * kHeadDim;
    ++next_j;
    if (next_j == p.q_steps || next_j == steps) {
      if (next_j == steps) {
        next_j = 0;
        ++next_token;
      }
      next = row_of(next_token, next_j);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  const GlobalScale gs = global_scale(a.gk);
  Turn turn;
  turn.on[0] = turn.on[1] = false;
  bool entered = false;  // `turn`, `slot`, `ws_row` and `dst` are of this token
  long long slot = -1, ws_row = -1;
  uint16_t* dst = nullptr;  // where the queries' next step goes
  int stage = 0;
  for (int step = st.begin; step < st.end; ++step) {
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    if (!entered) {
      slot = a.slots[token];
      if (a.ws_rows) ws_row = a.ws_rows[token];
      if constexpr (R != kNone) load_turn<R>(a, token, sub, turn);
      dst = a.q_out + token * a.q_out_stride + (4 * j + group) * kHeadDim + 8 * sub;
      entered = true;
    }
    const bool key = j >= p.q_steps, live = live_at(j);
    const int h = 4 * (j - p.q_steps) + group;
    uint32_t y[8];
    take_row(ring + stage * kStageBytes + 16 * lane, y);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float2 f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = unpack2(y[i]);
    if (norms) normalise(f, weights, key, sub, (key ? a.k_weight : a.q_weight) != nullptr, a.eps);
    rotate<R>(f, turn, lane, a.rot);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = pack_bf16x2(f[i].x, f[i].y);
    const long long s = slot, ws = ws_row;
    if (++j == steps) {
      j = 0;
      ++token;
      entered = false;
    }
    if (!key) {
      if (live) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(dst + 64) = make_uint4(y[4], y[5], y[6], y[7]);
      }
      dst += 4 * kHeadDim;
      continue;
    }
    const HalfBlocks q = quantize_halves(y, gs);
    if (!live) continue;
    if (a.ws_rows) store_ws(p, false, ws, h, sub, y);
    uint8_t* ph = page_head(a, s, h);
    if (!ph) continue;
    const int rin = (int)(s & (kPage - 1));
    uint32_t* d = reinterpret_cast<uint32_t*>(ph + kOffKData + rin * kRowBytes) + sub;
    d[0] = q.codes[0];
    d[8] = q.codes[1];
    // lane 2 i: block i, lane 2 i + 1: block 4 + i
    ph[k_scale_offset(rin, (sub >> 1) + 4 * (sub & 1))] = (uint8_t)((sub & 1) ? q.sb[1] : q.sb[0]);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The warp's steps of the values: two heads of a token pair, two 8-lane groups to
// each.
__device__ __forceinline__ void value_rows(const NormRopeParams& p, Steps st, uint8_t* ring, int lane) {
  if (st.begin >= st.end) return;
  const NormRopeArgs& a = p.a;
  const int sub = lane & 7, which = (lane >> 3) & 1, group = lane >> 4;
  const GlobalScale gs = global_scale(a.gv);
  int pair = st.begin / p.v_steps, j = st.begin - pair * p.v_steps;
  int left = st.end - st.begin, next_pair = pair, next_j = j;
  const uint32_t ring_u32 = smem_u32(ring) + 16 * lane;
  auto fetch = [&](int stage) {
    const long long tok = 2LL * next_pair + which;
    const int h = 2 * next_j + group;
    fetch_row(ring_u32 + stage * kStageBytes, a.v + tok * a.v_stride + h * kHeadDim + 8 * sub,
              left > 0 && tok < a.ntok && h < a.hkv);
    --left;
    if (++next_j == p.v_steps) {
      next_j = 0;
      ++next_pair;
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);
  int stage = 0;
  for (int step = st.begin; step < st.end; ++step) {
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    const int tok = 2 * pair + which, h = 2 * j + group;
    const bool live = tok < a.ntok && h < a.hkv;
    if (++j == p.v_steps) {
      j = 0;
      ++pair;
    }
    const long long slot = live ? a.slots[tok] : -1;
    const long long mate = live && (tok ^ 1) < a.ntok ? a.slots[tok ^ 1] : -1;
    const long long ws_row = live && a.ws_rows ? a.ws_rows[tok] : -1;
    uint32_t y[8];
    take_row(ring + stage * kStageBytes + 16 * lane, y);
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const HalfBlocks q = quantize_halves(y, gs);
    // the pair's other token (lane ^ 8 holds the same values of it)
    const uint32_t o0 = __shfl_xor_sync(kAll, q.codes[0], 8), o1 = __shfl_xor_sync(kAll, q.codes[1], 8);
    if (!live) continue;
    if (a.ws_rows) store_ws(p, true, ws_row, h, sub, y);
    uint8_t* ph = page_head(a, slot, h);
    if (!ph) continue;
    const int rin = (int)(slot & (kPage - 1));
    const long long even = which ? mate : slot, odd = which ? slot : mate;
    uint8_t* const d = ph + kOffVData + (rin >> 1) * kVPairBytes + 8 * sub;
    if ((even & 1) == 0 && odd == even + 1) {
      // a lane of either token writes one of the two pieces of both
      *reinterpret_cast<uint2*>(d + 64 * which) = which ? v_pair_bytes(o1, q.codes[1]) : v_pair_bytes(q.codes[0], o0);
    } else {
      v_store_half_one(d, rin & 1, q.codes[0]);
      v_store_half_one(d + 64, rin & 1, q.codes[1]);
    }
    ph[v_scale_offset(rin, (sub >> 1) + 4 * (sub & 1))] = (uint8_t)((sub & 1) ? q.sb[1] : q.sb[0]);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int R>
__global__ void __launch_bounds__(kNrThreads, ctas_per_sm(R)) norm_rope_kernel(const NormRopeParams p) {
  __shared__ __align__(128) uint8_t rings[kNrWarps][kStages * kStageBytes];
  __shared__ Weights weights;
  after_earlier_kernels();
  load_weights(p.a, weights);
  __syncthreads();
  // (broadcast: the compiler then keeps what follows from it in uniform registers)
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kAll, (int)(threadIdx.x >> 5), 0);
  uint8_t* ring = rings[warp];
  value_rows(p, share(p, warp, p.v_all, 0), ring, lane);
  turn_rows<R>(p, share(p, warp, p.t_all, p.v_all), ring, weights, lane);
}

template <int R>
cudaError_t launch(const NormRopeParams& p, int num_sms, cudaStream_t stream) {
  const int64_t steps = (int64_t)p.t_all + p.v_all, fit = (int64_t)num_sms * ctas_per_sm(R);
  const int64_t need = (steps + kNrWarps - 1) / kNrWarps;
  return launch_overlapped(norm_rope_kernel<R>, need < fit ? need : fit, kNrThreads, 0, 1, stream, p);
}

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeArgs& args, float k_ws_scale, float v_ws_scale, int num_sms,
                                    cudaStream_t stream) {
  NormRopeParams p;
  p.a = args;
  p.ws = ws_scales(k_ws_scale, v_ws_scale);
  p.q_steps = (args.hq + 3) / 4;
  p.k_steps = (args.hkv + 3) / 4;
  p.v_steps = (args.hkv + 1) / 2;
  p.t_all = args.ntok * (p.q_steps + p.k_steps);  // (below 2^31: ntok times the more of hq and hkv is)
  p.v_all = (args.ntok + 1) / 2 * p.v_steps;
  switch (args.rot == 0 ? kNone : args.interleaved ? kInterleaved : args.rot == kHeadDim ? kWhole
          : args.rot == 96 ? kThreeQuarters : kFirst) {
    case kNone: return launch<kNone>(p, num_sms, stream);
    case kWhole: return launch<kWhole>(p, num_sms, stream);
    case kFirst: return launch<kFirst>(p, num_sms, stream);
    case kThreeQuarters: return launch<kThreeQuarters>(p, num_sms, stream);
    default: return launch<kInterleaved>(p, num_sms, stream);
  }
}

}  // namespace nvfp4kv
