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
// with half-split pairs the partner's values lie one to four lanes away.  An
// 8-lane group takes up to kRows rows that follow one another in the flattened
// (token, head) list, so that a token's cosines and sines, 128 bytes a lane,
// stay in registers over its heads.  Values go by token pairs, two groups to a
// unit, because a byte of V data holds two tokens.
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
constexpr int kMaxRows = 4;  // rows of an 8-lane group
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct NormRopeParams {
  NormRopeArgs a;
  WsScales ws;
  int32_t rows;                          // rows of a group
  int32_t q_chunks, k_chunks, v_chunks;  // warps of each kind
};

// One row's 16 values of a lane, as stored.
struct Row {
  uint4 a, b;
};

__device__ __forceinline__ Row load_row(const uint16_t* base, long long stride, int token, int head, int sub) {
  const uint4* s = reinterpret_cast<const uint4*>(base + token * stride + head * kHeadDim) + 2 * sub;
  return Row{s[0], s[1]};  // not the read-only path: the queries may be normed in place
}

// The lane's cosines and signed sines of one token: value i of the lane turns as
// y_i cos_i + partner_i sin_i.
struct Turn {
  float cos[16], sin[16];
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
        t.cos[8 * j + 2 * i] = t.cos[8 * j + 2 * i + 1] = cs[i];
        t.sin[8 * j + 2 * i] = -sn[i];
        t.sin[8 * j + 2 * i + 1] = sn[i];
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
      t.cos[4 * j] = c.x, t.cos[4 * j + 1] = c.y, t.cos[4 * j + 2] = c.z, t.cos[4 * j + 3] = c.w;
      t.sin[4 * j] = second ? s.x : -s.x;
      t.sin[4 * j + 1] = second ? s.y : -s.y;
      t.sin[4 * j + 2] = second ? s.z : -s.z;
      t.sin[4 * j + 3] = second ? s.w : -s.w;
    }
  }
}

// y = (x r) w over the eight lanes of a row.
__device__ __forceinline__ void normalise(float (&f)[16], const uint4 (&w)[2], float eps) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = __fadd_rn(__fmul_rn(f[2 * i], f[2 * i]), __fmul_rn(f[2 * i + 1], f[2 * i + 1]));
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = __fadd_rn(s[2 * i], s[2 * i + 1]);
  float sum = s[0];
#pragma unroll
  for (int x = 1; x < 8; x <<= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, x));
  const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / kHeadDim), eps)));
  float wf[16];
  unpack_bf16x8(w[0], wf);
  unpack_bf16x8(w[1], wf + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __fmul_rn(__fmul_rn(f[i], r), wf[i]);
}

template <bool kInterleaved>
__device__ __forceinline__ void rotate(float (&f)[16], const Turn& t, int lane, int rot) {
  if constexpr (kInterleaved) {
    if (t.on) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float a = f[i], b = f[i + 1];
        f[i] = __fadd_rn(__fmul_rn(a, t.cos[i]), __fmul_rn(b, t.sin[i]));
        f[i + 1] = __fadd_rn(__fmul_rn(b, t.cos[i + 1]), __fmul_rn(a, t.sin[i + 1]));
      }
    }
  } else {
    const int sub = lane & 7, by = rot >> 5;  // lanes of half the rotated values
    const int from = sub < by ? lane + by : sub < 2 * by ? lane - by : lane;
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __shfl_sync(kAll, f[i], from);
    if (t.on) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = __fadd_rn(__fmul_rn(f[i], t.cos[i]), __fmul_rn(o[i], t.sin[i]));
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

// Rows [chunk * 4 rows, + 4 rows) of the flattened (token, head) list of the
// queries or the keys, `rows` to each 8-lane group.
template <bool kInterleaved, bool kKeys>
__device__ __forceinline__ void turn_rows(const NormRopeParams& p, int chunk, int lane) {
  const NormRopeArgs& a = p.a;
  const int sub = lane & 7, heads = kKeys ? a.hkv : a.hq;
  const uint16_t* src = kKeys ? a.k : a.q;
  const long long stride = kKeys ? a.k_stride : a.q_stride;
  const long long total = (long long)a.ntok * heads;
  const long long r0 = ((long long)chunk * 4 + (lane >> 3)) * p.rows;
  const uint16_t* weight = kKeys ? a.k_weight : a.q_weight;
  uint4 w[2];
  if (weight) {
    w[0] = __ldg(reinterpret_cast<const uint4*>(weight) + 2 * sub);
    w[1] = __ldg(reinterpret_cast<const uint4*>(weight) + 2 * sub + 1);
  }
  int token = (int)(r0 / heads), head = (int)(r0 - (long long)token * heads);
  Row next = {};
  if (r0 < total) next = load_row(src, stride, token, head, sub);
  GlobalScale gs;
  if constexpr (kKeys) gs = global_scale(a.gk);
  Turn turn;
  turn.on = false;
  int turned = -1;  // the token that `turn` is of
  for (int i = 0; i < p.rows; ++i) {
    const bool live = r0 + i < total;
    const int tok = token, h = head;
    const Row row = next;
    if (++head == heads) {
      head = 0;
      ++token;
    }
    if (i + 1 < p.rows && r0 + i + 1 < total) next = load_row(src, stride, token, head, sub);
    if (live && a.rot > 0 && tok != turned) {
      load_turn<kInterleaved>(a, tok, sub, turn);
      turned = tok;
    }
    float f[16];
    unpack_bf16x8(row.a, f);
    unpack_bf16x8(row.b, f + 8);
    if (weight) normalise(f, w, a.eps);
    if (a.rot > 0) rotate<kInterleaved>(f, turn, lane, a.rot);
    uint32_t y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
    if (!live) continue;
    if constexpr (kKeys) {
      if (a.ws_rows) store_ws(p, false, __ldg(a.ws_rows + tok), h, sub, y);
      const long long slot = __ldg(a.slots + tok);
      uint8_t* ph = page_head(a, slot, h);
      if (ph) {
        unpack_words(y, f);
        const BlockCodes c = quantize_block(f, gs);
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
}

// Values: units of a token pair and a head, two 8-lane groups to each, `rows`
// units to a pair of groups.
__device__ __forceinline__ void value_rows(const NormRopeParams& p, int chunk, int lane) {
  const NormRopeArgs& a = p.a;
  const int sub = lane & 7, which = (lane >> 3) & 1;
  const long long units = (long long)((a.ntok + 1) >> 1) * a.hkv;
  const long long u0 = ((long long)chunk * 2 + (lane >> 4)) * p.rows;
  const GlobalScale gs = global_scale(a.gv);
  int pair = (int)(u0 / a.hkv), head = (int)(u0 - (long long)pair * a.hkv);
  Row next = {};
  if (u0 < units && 2 * pair + which < a.ntok) next = load_row(a.v, a.v_stride, 2 * pair + which, head, sub);
  for (int i = 0; i < p.rows; ++i) {
    const int tok = 2 * pair + which, h = head;
    const bool live = u0 + i < units && tok < a.ntok;
    const Row row = next;
    if (++head == a.hkv) {
      head = 0;
      ++pair;
    }
    if (i + 1 < p.rows && u0 + i + 1 < units && 2 * pair + which < a.ntok)
      next = load_row(a.v, a.v_stride, 2 * pair + which, head, sub);
    const uint32_t y[8] = {row.a.x, row.a.y, row.a.z, row.a.w, row.b.x, row.b.y, row.b.z, row.b.w};
    float f[16];
    unpack_words(y, f);
    const BlockCodes c = quantize_block(f, gs);
    // the pair's other token (lane ^ 8 holds the same block of it)
    const uint32_t plo = __shfl_xor_sync(kAll, c.lo, 8), phi = __shfl_xor_sync(kAll, c.hi, 8);
    const long long slot = live ? __ldg(a.slots + tok) : -1;
    const long long mate = live && (tok ^ 1) < a.ntok ? __ldg(a.slots + (tok ^ 1)) : -1;
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
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
  const int lane = threadIdx.x & 31;
  int w = (int)blockIdx.x * kNrWarps + (threadIdx.x >> 5);
  // warp-uniform kinds: keys, values, then the queries
  if (w < p.k_chunks) {
    turn_rows<kInterleaved, true>(p, w, lane);
  } else if ((w -= p.k_chunks) < p.v_chunks) {
    value_rows(p, w, lane);
  } else if ((w -= p.v_chunks) < p.q_chunks) {
    turn_rows<kInterleaved, false>(p, w, lane);
  }
}

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeArgs& args, float k_ws_scale, float v_ws_scale, int num_sms,
                                    cudaStream_t stream) {
  NormRopeParams p;
  p.a = args;
  p.ws = ws_scales(k_ws_scale, v_ws_scale);
  const int64_t q_rows = (int64_t)args.ntok * args.hq, k_rows = (int64_t)args.ntok * args.hkv;
  const int64_t v_units = (int64_t)((args.ntok + 1) / 2) * args.hkv;
  // more rows to a group once every SM has 16 warps without them
  const int64_t warps = (q_rows + k_rows + 2 * v_units) / 4;
  p.rows = 1;
  while (p.rows < kMaxRows && warps / (2 * p.rows) >= (int64_t)num_sms * 16) p.rows *= 2;
  auto chunks = [&](int64_t n, int per) { return (int32_t)((n + per * p.rows - 1) / (per * p.rows)); };
  p.q_chunks = chunks(q_rows, 4);
  p.k_chunks = chunks(k_rows, 4);
  p.v_chunks = chunks(v_units, 2);
  const int64_t all = (int64_t)p.q_chunks + p.k_chunks + p.v_chunks;
  const unsigned blocks = (unsigned)((all + kNrWarps - 1) / kNrWarps);
  if (args.interleaved)
    norm_rope_kernel<true><<<blocks, kNrThreads, 0, stream>>>(p);
  else
    norm_rope_kernel<false><<<blocks, kNrThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace nvfp4kv
