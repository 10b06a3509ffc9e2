// api.cu -- the C ABI of libnvfp4kv.so (declared in include/nvfp4kv.h): host
// validation, size queries and kernel launches.  Nothing here allocates device
// memory or synchronises; every launch goes to the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "nvfp4kv.h"
#include "nvfp4kv_launch.h"

namespace {

constexpr int kHeadDim = 128;

constexpr int kPageSize = 16;
constexpr int kMaxDevices = 64;
std::atomic<int> g_num_sms[kMaxDevices];  // 0 = not queried yet

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool positive_finite(float x) { return std::isfinite(x) && x > 0.0f; }

// SM count of the current device (cached; the query is a host call).
int current_num_sms(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4KV_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices) {
    int cached = g_num_sms[dev].load(std::memory_order_relaxed);
    if (cached > 0) {
      *num_sms = cached;
      return NVFP4KV_OK;
    }
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return NVFP4KV_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices) g_num_sms[dev].store(n, std::memory_order_relaxed);
  *num_sms = n;
  return NVFP4KV_OK;
}

// Shape and pointer checks common to every call that reads or writes the pool.
int check_cache(const nvfp4kv_cache* c) {
  if (c == nullptr) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (c->head_dim != kHeadDim || c->page_size != kPageSize) return NVFP4KV_ERR_UNSUPPORTED;
  if (c->num_pages <= 0 || c->num_kv_heads <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  // row indices (page * heads + head) * page_size stay below 2^31
  if (c->num_pages * (int64_t)c->num_kv_heads * kPageSize >= (int64_t(1) << 31))
    return NVFP4KV_ERR_UNSUPPORTED;
  if (!c->pages || !aligned(c->pages, 16)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!positive_finite(c->k_global_scale) || !positive_finite(c->v_global_scale))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  return NVFP4KV_OK;
}

// the last CUDA error a call of this thread returned NVFP4KV_ERR_CUDA for
thread_local cudaError_t last_cuda_error = cudaSuccess;

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return NVFP4KV_OK;
  last_cuda_error = e;
  return NVFP4KV_ERR_CUDA;
}

}  // namespace

extern "C" {

int nvfp4kv_cache_bytes(int64_t num_pages, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                        size_t* pool_bytes) {
  if (pool_bytes == nullptr) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_pages <= 0 || num_kv_heads <= 0 || head_dim <= 0 || page_size <= 0 || head_dim % 16 != 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  // rows of K (and of V), each head_dim / 2 data bytes and head_dim / 16 scale bytes
  const int64_t row_bytes = 2 * (int64_t)(head_dim / 2 + head_dim / 16);
  if (num_pages > INT64_MAX / num_kv_heads / page_size / row_bytes) return NVFP4KV_ERR_UNSUPPORTED;
  *pool_bytes = (size_t)(num_pages * num_kv_heads * (int64_t)page_size * row_bytes);
  return NVFP4KV_OK;
}

// Host checks of quantize-append arguments (nothing is enqueued).
static int check_append(const nvfp4kv_cache* cache, const void* k, const void* v, const int64_t* slot_mapping,
                        int64_t num_tokens, int32_t* device_status) {
  int st = check_cache(cache);
  if (st != NVFP4KV_OK) return st;
  if (num_tokens < 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return NVFP4KV_OK;
  if (num_tokens * (int64_t)cache->num_kv_heads >= (int64_t(1) << 31)) return NVFP4KV_ERR_UNSUPPORTED;
  if (!k || !v || !slot_mapping) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_mapping, 8)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (device_status && !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  return NVFP4KV_OK;
}

int nvfp4kv_quantize_append(const nvfp4kv_cache* cache, const void* k, const void* v,
                            const int64_t* slot_mapping, int64_t num_tokens, int32_t* device_status,
                            nvfp4kv_stream_t stream) {
  int st = check_append(cache, k, v, slot_mapping, num_tokens, device_status);
  if (st != NVFP4KV_OK || num_tokens == 0) return st;
  int nsm = 0;
  if ((st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_quantize_append(
      *cache, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), slot_mapping, num_tokens,
      device_status, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_quantize_append_fp8(const nvfp4kv_cache* cache, const void* k, const void* v,
                                const int64_t* slot_mapping, int64_t num_tokens, const int64_t* ws_rows,
                                int64_t total_rows, float k_ws_scale, float v_ws_scale, uint8_t* ws_k,
                                uint8_t* ws_v, int32_t* device_status, nvfp4kv_stream_t stream) {
  int st = check_append(cache, k, v, slot_mapping, num_tokens, device_status);
  if (st != NVFP4KV_OK) return st;
  if (total_rows < 0 || !std::isfinite(k_ws_scale) || !std::isfinite(v_ws_scale) || k_ws_scale <= 0.0f ||
      v_ws_scale <= 0.0f)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return NVFP4KV_OK;
  if (!ws_rows || !ws_k || !ws_v || !aligned(ws_rows, 8) || !aligned(ws_k, 16) || !aligned(ws_v, 16))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  if ((st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_quantize_append_fp8(
      *cache, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), slot_mapping, num_tokens, ws_rows,
      total_rows, k_ws_scale, v_ws_scale, ws_k, ws_v, device_status, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_quantize_append_variant(int variant, const nvfp4kv_cache* cache, const void* k, const void* v,
                                    const int64_t* slot_mapping, int64_t num_tokens, const uint8_t* rand_k,
                                    const uint8_t* rand_v, int32_t* device_status, nvfp4kv_stream_t stream) {
  if (variant != NVFP4KV_VARIANT_SR && variant != NVFP4KV_VARIANT_HADAMARD && variant != NVFP4KV_VARIANT_MXFP4)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  const int st = check_append(cache, k, v, slot_mapping, num_tokens, device_status);
  if (st != NVFP4KV_OK || num_tokens == 0) return st;
  if (variant == NVFP4KV_VARIANT_SR && (!rand_k || !rand_v || !aligned(rand_k, 16) || !aligned(rand_v, 16)))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  return cuda_status(nvfp4kv::launch_quantize_variant(variant, *cache, static_cast<const uint16_t*>(k),
                                                      static_cast<const uint16_t*>(v), slot_mapping, num_tokens,
                                                      rand_k, rand_v, device_status,
                                                      reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_decode_workspace_size(const nvfp4kv_cache* cache, int32_t batch, int32_t num_q_heads,
                                  size_t* bytes) {
  if (bytes == nullptr || cache == nullptr) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (cache->num_kv_heads <= 0 || batch < 0 || num_q_heads <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  int st = current_num_sms(&nsm);
  if (st != NVFP4KV_OK) return st;
  *bytes = nvfp4kv::decode_workspace_bytes(nsm, batch, cache->num_kv_heads);
  return NVFP4KV_OK;
}

size_t nvfp4kv_decode_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t max_seq_len, int32_t num_sms) {
  (void)max_seq_len;  // the split is over pages of all sequences together: lengths do not size it
  if (batch < 0 || num_q_heads <= 0 || num_sms <= 0) return 0;
  // the KV-head count divides num_q_heads (num_q_heads = G * num_kv_heads)
  return nvfp4kv::decode_workspace_bound(num_sms, batch, num_q_heads);
}

// Host checks of decode arguments (nothing is enqueued); *nsm gets the
// current device's SM count when batch > 0.
static int check_decode(const nvfp4kv_cache* cache, const void* q, float* out, const int32_t* page_table,
                        int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                        float softmax_scale, void* workspace, size_t workspace_bytes, int32_t* device_status,
                        int* nsm) {
  int st = check_cache(cache);
  if (st != NVFP4KV_OK) return st;
  if (batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_q_heads % cache->num_kv_heads != 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  const int group = num_q_heads / cache->num_kv_heads;
  if (group > 8) return NVFP4KV_ERR_UNSUPPORTED;
  if (!positive_finite(softmax_scale)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  // global page-head indices (sequence pages times KV heads) stay below 2^31
  if ((int64_t)batch * max_pages_per_seq * cache->num_kv_heads >= (int64_t(1) << 31) ||
      (int64_t)max_pages_per_seq * kPageSize >= (int64_t(1) << 31))
    return NVFP4KV_ERR_UNSUPPORTED;
  if (!q || !out || !page_table || !seq_lens) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (device_status && !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if ((st = current_num_sms(nsm)) != NVFP4KV_OK) return st;
  const size_t need = nvfp4kv::decode_workspace_bytes(*nsm, batch, cache->num_kv_heads);
  if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256)) return NVFP4KV_ERR_WORKSPACE;
  return NVFP4KV_OK;
}

int nvfp4kv_decode_attention(const nvfp4kv_cache* cache, const void* q, float* out,
                             const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
                             int32_t batch, int32_t num_q_heads, float softmax_scale, void* workspace,
                             size_t workspace_bytes, int32_t* device_status, nvfp4kv_stream_t stream) {
  int nsm = 0;
  const int st = check_decode(cache, q, out, page_table, max_pages_per_seq, seq_lens, batch, num_q_heads,
                              softmax_scale, workspace, workspace_bytes, device_status, &nsm);
  if (st != NVFP4KV_OK || batch == 0) return st;
  return cuda_status(nvfp4kv::launch_decode(*cache, static_cast<const uint16_t*>(q), out, page_table,
                                            max_pages_per_seq, seq_lens, batch, num_q_heads, softmax_scale,
                                            workspace, device_status, nsm,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_decode_attention_variant(int variant, const nvfp4kv_cache* cache, const void* q, float* out,
                                     const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
                                     int32_t batch, int32_t num_q_heads, float softmax_scale, void* workspace,
                                     size_t workspace_bytes, int32_t* device_status, nvfp4kv_stream_t stream) {
  if (variant != NVFP4KV_VARIANT_SR && variant != NVFP4KV_VARIANT_HADAMARD && variant != NVFP4KV_VARIANT_MXFP4)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  const int st = check_decode(cache, q, out, page_table, max_pages_per_seq, seq_lens, batch, num_q_heads,
                              softmax_scale, workspace, workspace_bytes, device_status, &nsm);
  if (st != NVFP4KV_OK || batch == 0) return st;
  return cuda_status(nvfp4kv::launch_decode_variant(variant, *cache, static_cast<const uint16_t*>(q), out, page_table,
                                                    max_pages_per_seq, seq_lens, batch, num_q_heads, softmax_scale,
                                                    workspace, device_status, nsm,
                                                    reinterpret_cast<cudaStream_t>(stream)));
}

// Host checks of a scoring (nullptr: none); *sc gets its value.
static int check_scoring(const nvfp4kv_scoring* scoring, nvfp4kv_scoring* sc) {
  *sc = nvfp4kv_scoring{0.0f, 0, 0, nullptr};
  if (scoring == nullptr) return NVFP4KV_OK;
  *sc = *scoring;
  if (sc->softcap != 0.0f && !(sc->softcap >= 0x1p-20f && sc->softcap <= 0x1p+20f))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (sc->window < 0 || sc->sinks < 0 || !aligned(sc->slopes, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  return NVFP4KV_OK;
}

int nvfp4kv_decode_attention_scored(const nvfp4kv_cache* cache, const void* q, void* out, float* lse,
                                    const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
                                    int32_t batch, int32_t num_q_heads, float softmax_scale,
                                    const nvfp4kv_scoring* scoring, void* workspace, size_t workspace_bytes,
                                    int32_t* device_status, nvfp4kv_stream_t stream) {
  nvfp4kv_scoring sc;
  int st = check_scoring(scoring, &sc);
  if (st != NVFP4KV_OK) return st;
  int nsm = 0;
  st = check_decode(cache, q, static_cast<float*>(out), page_table, max_pages_per_seq, seq_lens, batch, num_q_heads,
                    softmax_scale, workspace, workspace_bytes, device_status, &nsm);
  if (st != NVFP4KV_OK) return st;
  if (!aligned(lse, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  return cuda_status(nvfp4kv::launch_decode_scored(*cache, static_cast<const uint16_t*>(q),
                                                   static_cast<uint16_t*>(out), lse, page_table, max_pages_per_seq,
                                                   seq_lens, batch, num_q_heads, softmax_scale, sc, nullptr, workspace,
                                                   device_status, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

// Checks of the sizes that the weights' workspace depends on, and its bytes.
static int weights_workspace(const nvfp4kv_cache* cache, int32_t batch, int32_t num_q_heads, int64_t max_total_pages,
                             int nsm, size_t* bytes) {
  if (cache == nullptr || cache->num_kv_heads <= 0 || batch < 0 || num_q_heads <= 0 || max_total_pages < 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_q_heads % cache->num_kv_heads != 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_q_heads / cache->num_kv_heads > 8) return NVFP4KV_ERR_UNSUPPORTED;
  // page-heads of a batch stay below 2^31 (so the size below does not overflow)
  if (max_total_pages > (int64_t(1) << 31) / cache->num_kv_heads) return NVFP4KV_ERR_UNSUPPORTED;
  *bytes = nvfp4kv::decode_weights_workspace_bytes(nsm, batch, num_q_heads, cache->num_kv_heads, max_total_pages);
  return NVFP4KV_OK;
}

int nvfp4kv_decode_weights_workspace_size(const nvfp4kv_cache* cache, int32_t batch, int32_t num_q_heads,
                                          int64_t max_total_pages, size_t* bytes) {
  if (bytes == nullptr) return NVFP4KV_ERR_INVALID_ARGUMENT;
  size_t n = 0;
  int st = weights_workspace(cache, batch, num_q_heads, max_total_pages, 1, &n);  // the checks, before any CUDA call
  int nsm = 0;
  if (st != NVFP4KV_OK || (st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  return weights_workspace(cache, batch, num_q_heads, max_total_pages, nsm, bytes);
}

int nvfp4kv_decode_attention_weights(const nvfp4kv_cache* cache, const void* q, void* out, float* lse,
                                     const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
                                     int32_t batch, int32_t num_q_heads, float softmax_scale,
                                     const nvfp4kv_scoring* scoring, float* weights, int64_t weight_stride,
                                     float decay, int64_t max_total_pages, void* workspace, size_t workspace_bytes,
                                     int32_t* device_status, nvfp4kv_stream_t stream) {
  nvfp4kv_scoring sc;
  int st = check_scoring(scoring, &sc);
  if (st != NVFP4KV_OK) return st;
  if (weight_stride <= 0 || !std::isfinite(decay) || decay < 0.0f || max_total_pages < 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  st = check_decode(cache, q, static_cast<float*>(out), page_table, max_pages_per_seq, seq_lens, batch, num_q_heads,
                    softmax_scale, workspace, workspace_bytes, device_status, &nsm);
  if (st != NVFP4KV_OK) return st;
  if (!aligned(lse, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  if (weights == nullptr || !aligned(weights, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (weight_stride > (int64_t(1) << 40)) return NVFP4KV_ERR_UNSUPPORTED;
  size_t need = 0;
  if ((st = weights_workspace(cache, batch, num_q_heads, max_total_pages, nsm, &need)) != NVFP4KV_OK) return st;
  if (workspace_bytes < need) return NVFP4KV_ERR_WORKSPACE;
  const nvfp4kv::DecodeWeights w = {weights, weight_stride, decay, max_total_pages};
  return cuda_status(nvfp4kv::launch_decode_scored(*cache, static_cast<const uint16_t*>(q),
                                                   static_cast<uint16_t*>(out), lse, page_table, max_pages_per_seq,
                                                   seq_lens, batch, num_q_heads, softmax_scale, sc, &w, workspace,
                                                   device_status, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_append_decode_attention(const nvfp4kv_cache* cache, const void* k, const void* v,
                                    const int64_t* slot_mapping, int64_t num_tokens, const void* q, float* out,
                                    const int32_t* page_table, int32_t max_pages_per_seq,
                                    const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                                    float softmax_scale, void* workspace, size_t workspace_bytes,
                                    int32_t* device_status, nvfp4kv_stream_t stream) {
  int st = check_append(cache, k, v, slot_mapping, num_tokens, device_status);
  if (st != NVFP4KV_OK) return st;
  int nsm = 0;
  st = check_decode(cache, q, out, page_table, max_pages_per_seq, seq_lens, batch, num_q_heads, softmax_scale,
                    workspace, workspace_bytes, device_status, &nsm);
  if (st != NVFP4KV_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (num_tokens > 0) {
    int asm_ = nsm;
    if (asm_ == 0 && (st = current_num_sms(&asm_)) != NVFP4KV_OK) return st;
    st = cuda_status(nvfp4kv::launch_quantize_append(*cache, static_cast<const uint16_t*>(k),
                                                     static_cast<const uint16_t*>(v), slot_mapping, num_tokens,
                                                     device_status, asm_, s));
    if (st != NVFP4KV_OK) return st;
  }
  if (batch == 0) return NVFP4KV_OK;
  return cuda_status(nvfp4kv::launch_decode(*cache, static_cast<const uint16_t*>(q), out, page_table,
                                            max_pages_per_seq, seq_lens, batch, num_q_heads, softmax_scale,
                                            workspace, device_status, nsm, s, num_tokens > 0));
}

int nvfp4kv_bf16_to_fp8_workspace(const void* k_bf16, const void* v_bf16, const int64_t* ws_rows,
                                   int64_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                                   int64_t total_rows, float k_ws_scale, float v_ws_scale, uint8_t* ws_k,
                                   uint8_t* ws_v, int32_t* device_status, nvfp4kv_stream_t stream) {
  if (num_tokens < 0 || num_kv_heads <= 0 || total_rows < 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (head_dim != 128) return NVFP4KV_ERR_UNSUPPORTED;
  if (!std::isfinite(k_ws_scale) || !std::isfinite(v_ws_scale) || k_ws_scale <= 0.0f || v_ws_scale <= 0.0f)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (device_status && !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return NVFP4KV_OK;
  if (!k_bf16 || !v_bf16 || !ws_rows || !ws_k || !ws_v) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(ws_rows, 8) || !aligned(ws_k, 16) ||
      !aligned(ws_v, 16))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_tokens > (INT64_MAX / 2) / ((int64_t)num_kv_heads * 16)) return NVFP4KV_ERR_UNSUPPORTED;
  int nsm = 0;
  const int st = current_num_sms(&nsm);
  if (st != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_chunk_to_ws(static_cast<const uint16_t*>(k_bf16),
                                                 static_cast<const uint16_t*>(v_bf16), ws_rows, num_tokens,
                                                 num_kv_heads, total_rows, k_ws_scale, v_ws_scale, ws_k, ws_v,
                                                 device_status, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

// Host checks of extend arguments (nothing is enqueued); out is fp32 or bf16.
static int check_extend(const void* q_bf16, const int64_t* cu_q, int32_t max_q_len, const uint8_t* ws_k,
                        const uint8_t* ws_v, const int64_t* cu_prefix, const int32_t* prefix_lens, int32_t batch,
                        int64_t total_rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                        float k_ws_scale, float v_ws_scale, float softmax_scale, const void* out,
                        const int32_t* device_status) {
  if (batch < 0 || max_q_len < 0 || total_rows < 0 || num_q_heads <= 0 || num_kv_heads <= 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_q_heads % num_kv_heads != 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  const int32_t group = num_q_heads / num_kv_heads;
  if (head_dim != 128 || group > 128 || (group & (group - 1)) != 0 || batch > 65535 || num_kv_heads > 65535)
    return NVFP4KV_ERR_UNSUPPORTED;
  for (float sc : {k_ws_scale, v_ws_scale, softmax_scale})
    if (!std::isfinite(sc) || sc <= 0.0f) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (device_status && !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0 || max_q_len == 0) return NVFP4KV_OK;
  if (!q_bf16 || !cu_q || !ws_k || !ws_v || !cu_prefix || !prefix_lens || !out)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!aligned(q_bf16, 16) || !aligned(out, 16) || !aligned(ws_k, 16) || !aligned(ws_v, 16) || !aligned(cu_q, 8) ||
      !aligned(cu_prefix, 8) || !aligned(prefix_lens, 4))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if ((int64_t)max_q_len * group > (int64_t)INT32_MAX) return NVFP4KV_ERR_UNSUPPORTED;
  return NVFP4KV_OK;
}

int nvfp4kv_extend_attention(const void* q_bf16, const int64_t* cu_q, int32_t max_q_len, const uint8_t* ws_k,
                             const uint8_t* ws_v, const int64_t* cu_prefix, const int32_t* prefix_lens,
                             int32_t batch, int64_t total_rows, int32_t num_q_heads, int32_t num_kv_heads,
                             int32_t head_dim, float k_ws_scale, float v_ws_scale, float softmax_scale,
                             float* out, int32_t* device_status, nvfp4kv_stream_t stream) {
  const int st = check_extend(q_bf16, cu_q, max_q_len, ws_k, ws_v, cu_prefix, prefix_lens, batch, total_rows,
                              num_q_heads, num_kv_heads, head_dim, k_ws_scale, v_ws_scale, softmax_scale, out,
                              device_status);
  if (st != NVFP4KV_OK || batch == 0 || max_q_len == 0) return st;
  return cuda_status(nvfp4kv::launch_extend_attention(
      static_cast<const uint16_t*>(q_bf16), cu_q, max_q_len, ws_k, ws_v, cu_prefix, prefix_lens, batch,
      total_rows, num_q_heads, num_kv_heads, k_ws_scale, v_ws_scale, softmax_scale, out, device_status,
      reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_extend_attention_scored(const void* q_bf16, const int64_t* cu_q, int32_t max_q_len, const uint8_t* ws_k,
                                    const uint8_t* ws_v, const int64_t* cu_prefix, const int32_t* prefix_lens,
                                    int32_t batch, int64_t total_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t head_dim, float k_ws_scale, float v_ws_scale, float softmax_scale,
                                    const nvfp4kv_scoring* scoring, const int32_t* full_lens,
                                    const int32_t* doc_starts, void* out, float* lse, int32_t* device_status,
                                    nvfp4kv_stream_t stream) {
  nvfp4kv_scoring sc;
  int st = check_scoring(scoring, &sc);
  if (st != NVFP4KV_OK) return st;
  st = check_extend(q_bf16, cu_q, max_q_len, ws_k, ws_v, cu_prefix, prefix_lens, batch, total_rows, num_q_heads,
                    num_kv_heads, head_dim, k_ws_scale, v_ws_scale, softmax_scale, out, device_status);
  if (st != NVFP4KV_OK) return st;
  if (!aligned(full_lens, 4) || !aligned(doc_starts, 4) || !aligned(lse, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0 || max_q_len == 0) return NVFP4KV_OK;
  return cuda_status(nvfp4kv::launch_extend_scored(
      static_cast<const uint16_t*>(q_bf16), cu_q, max_q_len, ws_k, ws_v, cu_prefix, prefix_lens, batch, total_rows,
      num_q_heads, num_kv_heads, k_ws_scale, v_ws_scale, softmax_scale, sc, full_lens, doc_starts,
      static_cast<uint16_t*>(out), lse, device_status, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_evict(const nvfp4kv_cache* cache, const int32_t* page_table, int32_t max_pages_per_seq,
                  const int32_t* seq_lens, int32_t batch, const float* weights, int64_t weight_stride,
                  int32_t budget, int32_t first, int32_t recent, const int32_t* dst_page_table,
                  int32_t dst_max_pages_per_seq, int32_t* kept, float* kept_weights, int64_t kept_stride,
                  int32_t* new_lens, int32_t* device_status, nvfp4kv_stream_t stream) {
  int st = check_cache(cache);
  if (st != NVFP4KV_OK) return st;
  if (batch < 0 || max_pages_per_seq <= 0 || weight_stride <= 0 || dst_max_pages_per_seq <= 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (budget <= 0 || first < 0 || recent < 0 || (int64_t)first + recent > budget) return NVFP4KV_ERR_INVALID_ARGUMENT;
  const int64_t dst_pages = ((int64_t)budget + kPageSize - 1) / kPageSize;
  if (dst_max_pages_per_seq < dst_pages || (kept_weights && kept_stride < budget)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  const int64_t pairs = (int64_t)batch * cache->num_kv_heads;
  if ((int64_t)max_pages_per_seq * kPageSize >= (int64_t(1) << 31) || weight_stride > (int64_t(1) << 40) ||
      kept_stride > (int64_t(1) << 40) || pairs >= (int64_t(1) << 27) || pairs * dst_pages >= (int64_t(1) << 31))
    return NVFP4KV_ERR_UNSUPPORTED;
  // the selection's loops over a list of `budget` step by up to 4096 (8 CTAs of 512 threads) in 32 bits
  if (budget > INT32_MAX - 4095) return NVFP4KV_ERR_UNSUPPORTED;
  if (!page_table || !seq_lens || !weights || !dst_page_table || !kept) return NVFP4KV_ERR_INVALID_ARGUMENT;
  for (const void* ptr : {(const void*)page_table, (const void*)seq_lens, (const void*)weights,
                          (const void*)dst_page_table, (const void*)kept, (const void*)kept_weights,
                          (const void*)new_lens, (const void*)device_status})
    if (!aligned(ptr, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  // packing in place, or sums on top of those still being read, would go wrong silently
  const float* const weights_end = weights + pairs * weight_stride;
  const float* const kept_end = kept_weights ? kept_weights + pairs * kept_stride : kept_weights;
  if (dst_page_table == page_table || (kept_weights && kept_weights < weights_end && weights < kept_end))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  // new_lens may be seq_lens (min(min(L, budget), budget) = min(L, budget)), but at an offset one
  // sequence's new length would be another's old one
  if (new_lens && new_lens != seq_lens && new_lens < seq_lens + batch && seq_lens < new_lens + batch)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  if ((st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_evict(*cache, page_table, max_pages_per_seq, seq_lens, batch, weights,
                                           weight_stride, budget, first, recent, dst_page_table,
                                           dst_max_pages_per_seq, kept, kept_weights, kept_stride, new_lens,
                                           device_status, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------------------
// a step's plan, its normed and rotated append, and the pages that its decode reads
// ---------------------------------------------------------------------------

// Whether the n elements of two arrays share memory other than by being the same array.
static bool overlap_at_offset(const int32_t* a, const int32_t* b, int64_t n) {
  return a != b && a < b + n && b < a + n;
}

int nvfp4kv_plan_append(int32_t* page_table, int32_t max_pages_per_seq, const int32_t* cached_lens,
                        const int32_t* new_lens, int32_t batch, const int32_t* free_pages, int32_t free_capacity,
                        const int32_t* free_count, int64_t num_pages, int64_t max_tokens, int32_t* seq_lens,
                        int64_t* slot_mapping, int32_t* positions, int64_t* cu_q, int64_t* ws_rows,
                        int64_t* cu_prefix, int32_t* free_left, int32_t* device_status, nvfp4kv_stream_t stream) {
  if (batch < 0 || max_pages_per_seq <= 0 || free_capacity < 0 || num_pages <= 0 || max_tokens < 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if ((int64_t)max_pages_per_seq * kPageSize >= (int64_t(1) << 31) || max_tokens >= (int64_t(1) << 31) - (1 << 18) ||
      num_pages >= (int64_t(1) << 31) / kPageSize || batch >= (1 << 30) || free_capacity > (1 << 30))
    return NVFP4KV_ERR_UNSUPPORTED;
  if (!free_count || !free_left || (free_capacity > 0 && !free_pages) || (max_tokens > 0 && !slot_mapping))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch > 0 && (!page_table || !cached_lens || !new_lens || !seq_lens)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  for (const void* ptr : {(const void*)page_table, (const void*)cached_lens, (const void*)new_lens,
                          (const void*)free_pages, (const void*)free_count, (const void*)seq_lens,
                          (const void*)positions, (const void*)free_left, (const void*)device_status})
    if (!aligned(ptr, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  for (const void* ptr : {(const void*)slot_mapping, (const void*)cu_q, (const void*)ws_rows, (const void*)cu_prefix})
    if (!aligned(ptr, 8)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  // the lengths may be updated in place, but not at an offset
  if (overlap_at_offset(seq_lens, cached_lens, batch) || (batch > 0 && seq_lens == new_lens) ||
      overlap_at_offset(seq_lens, new_lens, batch))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  const nvfp4kv::PlanArgs a = {page_table, max_pages_per_seq, cached_lens, new_lens,  batch,  free_pages,
                               free_capacity, free_count,     num_pages,   max_tokens, seq_lens, slot_mapping,
                               positions,  cu_q,              ws_rows,     cu_prefix, free_left, device_status};
  return cuda_status(nvfp4kv::launch_plan_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_norm_rope_append(const nvfp4kv_cache* cache, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride, int32_t num_q_heads,
                             int64_t num_tokens, const int64_t* slot_mapping, const int32_t* positions,
                             const float* cos_sin, int32_t max_position, const nvfp4kv_norm_rope* how, void* q_out,
                             int64_t q_out_stride, const int64_t* ws_rows, int64_t total_rows, float k_ws_scale,
                             float v_ws_scale, uint8_t* ws_k, uint8_t* ws_v, int32_t* device_status,
                             nvfp4kv_stream_t stream) {
  int st = check_cache(cache);
  if (st != NVFP4KV_OK) return st;
  if (how == nullptr || num_tokens < 0 || num_q_heads <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (how->rotary_dim < 0 || how->rotary_dim > kHeadDim || how->rotary_dim % 32 != 0) return NVFP4KV_ERR_UNSUPPORTED;
  if (!aligned(how->q_weight, 16) || !aligned(how->k_weight, 16)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if ((how->q_weight || how->k_weight) && !positive_finite(how->eps)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (how->rotary_dim > 0 && max_position <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  // rows of one token do not run into the next token's, and start on 16 bytes
  const int64_t q_row = (int64_t)num_q_heads * kHeadDim, kv_row = (int64_t)cache->num_kv_heads * kHeadDim;
  if (q_stride < q_row || q_out_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride % 8 != 0 ||
      q_out_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (ws_rows &&
      (total_rows < 0 || !positive_finite(k_ws_scale) || !positive_finite(v_ws_scale)))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (device_status && !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return NVFP4KV_OK;
  const int64_t most = int64_t(1) << 40;
  if (num_q_heads > (1 << 20) || cache->num_kv_heads > (1 << 20) || num_tokens >= (int64_t(1) << 30) ||
      num_tokens >= (int64_t(1) << 31) / (num_q_heads > cache->num_kv_heads ? num_q_heads : cache->num_kv_heads) ||
      q_stride > most || q_out_stride > most || k_stride > most || v_stride > most || total_rows > most)
    return NVFP4KV_ERR_UNSUPPORTED;
  // byte offsets of the last tokens' rows fit 62 bits
  const int64_t longest = std::max(std::max(q_stride, q_out_stride), std::max(k_stride, v_stride));
  if (longest > (int64_t(1) << 60) / num_tokens) return NVFP4KV_ERR_UNSUPPORTED;
  if (!q || !k || !v || !slot_mapping || !q_out || (how->rotary_dim > 0 && (!positions || !cos_sin)))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(cos_sin, 16) ||
      !aligned(slot_mapping, 8) || !aligned(positions, 4))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (ws_rows && (!ws_k || !ws_v || !aligned(ws_rows, 8) || !aligned(ws_k, 16) || !aligned(ws_v, 16)))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  // normed queries may replace their inputs, not lie across them
  const uint16_t *q0 = static_cast<const uint16_t*>(q), *o0 = static_cast<const uint16_t*>(q_out);
  if (q_out == q ? q_out_stride != q_stride
                 : o0 < q0 + (num_tokens - 1) * q_stride + q_row && q0 < o0 + (num_tokens - 1) * q_out_stride + q_row)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  if ((st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  nvfp4kv::NormRopeArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_out_stride = q_out_stride;
  a.q_weight = static_cast<const uint16_t*>(how->q_weight);
  a.k_weight = static_cast<const uint16_t*>(how->k_weight);
  a.eps = how->eps;
  a.cos_sin = cos_sin;
  a.rot = how->rotary_dim;
  a.max_position = max_position;
  a.interleaved = how->interleaved != 0;
  a.positions = positions;
  a.slots = slot_mapping;
  a.ntok = (int32_t)num_tokens;
  a.hq = num_q_heads;
  a.hkv = cache->num_kv_heads;
  a.capacity = cache->num_pages * (int64_t)kPageSize;
  a.pages = cache->pages;
  a.gk = cache->k_global_scale;
  a.gv = cache->v_global_scale;
  a.ws_rows = ws_rows;
  a.ws_total_rows = total_rows;
  a.ws_k = ws_k;
  a.ws_v = ws_v;
  a.status = device_status;
  return cuda_status(nvfp4kv::launch_norm_rope_append(a, ws_rows ? k_ws_scale : 1.0f, ws_rows ? v_ws_scale : 1.0f, nsm,
                                                      reinterpret_cast<cudaStream_t>(stream)));
}

// Host checks of what the digest and the page scores share (nothing is enqueued).
static int check_digest(const nvfp4kv_cache* cache, const int32_t* page_table, int32_t max_pages_per_seq,
                        const int32_t* seq_lens, int32_t batch, const uint8_t* digest, const int32_t* device_status) {
  const int st = check_cache(cache);
  if (st != NVFP4KV_OK) return st;
  if (batch < 0 || max_pages_per_seq <= 0 || !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  if ((int64_t)batch * max_pages_per_seq * cache->num_kv_heads >= (int64_t(1) << 31) ||
      (int64_t)max_pages_per_seq * kPageSize >= (int64_t(1) << 31))
    return NVFP4KV_ERR_UNSUPPORTED;
  if (!page_table || !seq_lens || !digest) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(digest, 16)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  return NVFP4KV_OK;
}

static nvfp4kv::DigestArgs digest_args(const nvfp4kv_cache& c, const int32_t* page_table, int32_t max_pages_per_seq,
                                       const int32_t* seq_lens, const int32_t* first_tokens, int32_t batch,
                                       uint8_t* digest, int32_t* device_status) {
  return nvfp4kv::DigestArgs{c.pages,  (int32_t)c.num_pages, c.num_kv_heads, page_table, max_pages_per_seq,
                             seq_lens, first_tokens,         batch,          digest,     device_status};
}

int nvfp4kv_page_digest(const nvfp4kv_cache* cache, const int32_t* page_table, int32_t max_pages_per_seq,
                        const int32_t* seq_lens, const int32_t* first_tokens, int32_t batch, uint8_t* digest,
                        int32_t* device_status, nvfp4kv_stream_t stream) {
  int st = check_digest(cache, page_table, max_pages_per_seq, seq_lens, batch, digest, device_status);
  if (st != NVFP4KV_OK) return st;
  if (!aligned(first_tokens, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  int nsm = 0;
  if ((st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_page_digest(
      digest_args(*cache, page_table, max_pages_per_seq, seq_lens, first_tokens, batch, digest, device_status), nsm,
      reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_page_scores(const nvfp4kv_cache* cache, const uint8_t* digest, const void* q, const int32_t* page_table,
                        int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                        float softmax_scale, float* scores, int64_t score_stride, int32_t* device_status,
                        nvfp4kv_stream_t stream) {
  int st = check_digest(cache, page_table, max_pages_per_seq, seq_lens, batch, digest, device_status);
  if (st != NVFP4KV_OK) return st;
  if (num_q_heads <= 0 || num_q_heads % cache->num_kv_heads != 0 || score_stride <= 0)
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (num_q_heads / cache->num_kv_heads > 8) return NVFP4KV_ERR_UNSUPPORTED;
  if (!positive_finite(softmax_scale)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  if (score_stride > (int64_t(1) << 40)) return NVFP4KV_ERR_UNSUPPORTED;
  if (!q || !scores || !aligned(q, 16) || !aligned(scores, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  if ((st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  const nvfp4kv::ScoreArgs a = {
      digest_args(*cache, page_table, max_pages_per_seq, seq_lens, nullptr, batch, const_cast<uint8_t*>(digest),
                  device_status),
      static_cast<const uint16_t*>(q), num_q_heads / cache->num_kv_heads, softmax_scale * cache->k_global_scale, scores,
      score_stride};
  return cuda_status(nvfp4kv::launch_page_scores(a, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_select_pages(const float* scores, int64_t score_stride, const int32_t* seq_lens, int32_t batch,
                         int32_t num_kv_heads, int32_t budget, int32_t first, int32_t recent, int32_t* selected,
                         int32_t* device_status, nvfp4kv_stream_t stream) {
  if (batch < 0 || num_kv_heads <= 0 || score_stride <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (budget <= 0 || first < 0 || recent < 0 || (int64_t)first + recent > budget) return NVFP4KV_ERR_INVALID_ARGUMENT;
  // pages of a sequence fit 27 bits, as its tokens fit 31
  if (budget > (1 << 27) || (int64_t)batch * num_kv_heads >= (int64_t(1) << 27) || score_stride > (int64_t(1) << 40))
    return NVFP4KV_ERR_UNSUPPORTED;
  if (!aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  if (!scores || !seq_lens || !selected || !aligned(scores, 4) || !aligned(seq_lens, 4) || !aligned(selected, 4))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  const nvfp4kv::SelectArgs a = {scores, score_stride, seq_lens, batch, num_kv_heads, budget, first, recent, selected,
                                 device_status};
  int nsm = 0;
  const int st = current_num_sms(&nsm);
  if (st != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_select_pages(a, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_decode_attention_selected(const nvfp4kv_cache* cache, const void* q, void* out, float* lse,
                                      const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
                                      int32_t batch, int32_t num_q_heads, float softmax_scale,
                                      const int32_t* selected, int32_t budget, void* workspace,
                                      size_t workspace_bytes, int32_t* device_status, nvfp4kv_stream_t stream) {
  int nsm = 0;
  int st = check_decode(cache, q, static_cast<float*>(out), page_table, max_pages_per_seq, seq_lens, batch,
                        num_q_heads, softmax_scale, workspace, workspace_bytes, device_status, &nsm);
  if (st != NVFP4KV_OK) return st;
  if (budget <= 0 || !aligned(lse, 4) || !aligned(selected, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0) return NVFP4KV_OK;
  if (!selected) return NVFP4KV_ERR_INVALID_ARGUMENT;
  return cuda_status(nvfp4kv::launch_decode_selected(
      *cache, static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), lse, page_table, max_pages_per_seq,
      seq_lens, batch, num_q_heads, softmax_scale, selected, budget, workspace, device_status, nsm,
      reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_tensor_amax(const void* x_bf16, int64_t n, float* amax, int accumulate,
                        nvfp4kv_stream_t stream) {
  if (n < 0 || amax == nullptr || !aligned(amax, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (n > 0 && (x_bf16 == nullptr || !aligned(x_bf16, 16))) return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  const int st = current_num_sms(&nsm);
  if (st != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_tensor_amax(static_cast<const uint16_t*>(x_bf16), n, amax, accumulate != 0,
                                                 nsm, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_calibrated_global_scale(float amax, float* g) {
  if (g == nullptr || !std::isfinite(amax) || amax < 0.0f) return NVFP4KV_ERR_INVALID_ARGUMENT;
  *g = amax == 0.0f ? 1.0f : amax / (6.0f * 448.0f);  // one binary32 division
  return NVFP4KV_OK;
}

int nvfp4kv_dequant_to_fp8_workspace(const nvfp4kv_cache* cache, const int32_t* page_table,
                                     int32_t max_pages_per_seq, const int32_t* prefix_lens,
                                     const int64_t* cu_prefix, int32_t batch, int64_t total_rows,
                                     float k_ws_scale, float v_ws_scale, uint8_t* ws_k, uint8_t* ws_v,
                                     int32_t* device_status, nvfp4kv_stream_t stream) {
  int st = check_cache(cache);
  if (st != NVFP4KV_OK) return st;
  if (batch < 0 || total_rows < 0 || max_pages_per_seq <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!positive_finite(k_ws_scale) || !positive_finite(v_ws_scale)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch == 0 || total_rows == 0) return NVFP4KV_OK;
  if ((int64_t)max_pages_per_seq * kPageSize >= (int64_t(1) << 31)) return NVFP4KV_ERR_UNSUPPORTED;
  if (total_rows * cache->num_kv_heads >= (int64_t(1) << 40)) return NVFP4KV_ERR_UNSUPPORTED;
  if (!page_table || !prefix_lens || !cu_prefix || !ws_k || !ws_v) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (!aligned(page_table, 4) || !aligned(prefix_lens, 4) || !aligned(cu_prefix, 8) || !aligned(ws_k, 16) ||
      !aligned(ws_v, 16))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (device_status && !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  return cuda_status(nvfp4kv::launch_dequant_fp8(*cache, page_table, max_pages_per_seq, prefix_lens, cu_prefix,
                                                 batch, total_rows, k_ws_scale, v_ws_scale, ws_k, ws_v,
                                                 device_status, reinterpret_cast<cudaStream_t>(stream)));
}

int nvfp4kv_stream_probe(const nvfp4kv_cache* cache, const int32_t* page_table, int32_t max_pages_per_seq,
                         const int32_t* seq_lens, int32_t batch, int mode, uint32_t* sink, int32_t* device_status,
                         nvfp4kv_stream_t stream) {
  int st = check_cache(cache);
  if (st != NVFP4KV_OK) return st;
  if (mode != NVFP4KV_PROBE_DECODE_PATTERN && mode != NVFP4KV_PROBE_WHOLE_PAGES) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (batch < 0 || max_pages_per_seq <= 0) return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (mode == NVFP4KV_PROBE_WHOLE_PAGES && cache->num_kv_heads > 16) return NVFP4KV_ERR_UNSUPPORTED;
  if (batch == 0) return NVFP4KV_OK;
  if ((int64_t)batch * max_pages_per_seq * cache->num_kv_heads >= (int64_t(1) << 31) ||
      (int64_t)max_pages_per_seq * kPageSize >= (int64_t(1) << 31))
    return NVFP4KV_ERR_UNSUPPORTED;
  if (!page_table || !seq_lens || !sink || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(sink, 4))
    return NVFP4KV_ERR_INVALID_ARGUMENT;
  if (device_status && !aligned(device_status, 4)) return NVFP4KV_ERR_INVALID_ARGUMENT;
  int nsm = 0;
  if ((st = current_num_sms(&nsm)) != NVFP4KV_OK) return st;
  return cuda_status(nvfp4kv::launch_stream_probe(*cache, page_table, max_pages_per_seq, seq_lens, batch, mode,
                                                  sink, device_status, nsm, reinterpret_cast<cudaStream_t>(stream)));
}

const char* nvfp4kv_last_cuda_error(void) {
  return last_cuda_error == cudaSuccess ? "no CUDA error" : cudaGetErrorString(last_cuda_error);
}

const char* nvfp4kv_status_string(int status) {
  switch (status) {
    case NVFP4KV_OK: return "ok";
    case NVFP4KV_ERR_INVALID_ARGUMENT: return "invalid argument";
    case NVFP4KV_ERR_UNSUPPORTED: return "unsupported configuration";
    case NVFP4KV_ERR_CUDA: return "CUDA error (see cudaGetLastError)";
    case NVFP4KV_ERR_WORKSPACE: return "workspace null, too small or misaligned";
    default: return "unknown status";
  }
}

}  // extern "C"
