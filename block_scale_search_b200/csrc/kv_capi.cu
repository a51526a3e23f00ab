// kv_capi.cu -- the extern "C" entry points of the NVFP4 K/V cache.  As
// everywhere: arguments are checked on the host before anything is enqueued,
// and no C++ exception leaves.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <vector>

#include "kv_cache.cuh"
#include "nvtx_range.cuh"

namespace nvfp4 {
int record_cuda_status(cudaError_t e);
unsigned int kv_stalls(bool reset, cudaError_t* e);
bool kv_wait_limit(long long cycles, cudaError_t* e);
}  // namespace nvfp4

namespace {

constexpr int64_t kIntMax = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxStride = int64_t{1} << 40;  // guards index arithmetic
constexpr int64_t kMaxPageStride = (int64_t{1} << 32) - 16;

// SM count of the current device, cached per device ordinal (0 on failure).
int sm_count() {
  static std::atomic<int> cache[128];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 128 && (n = cache[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 128) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_cache(const nvfp4_kv_cache* c) {
  if (c == nullptr || c->k_codes == nullptr || c->k_scales == nullptr || c->v_codes == nullptr ||
      c->v_scales == nullptr || c->k_S == nullptr || c->v_S == nullptr)
    return NVFP4_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1)
    return NVFP4_ERR_INVALID_ARG;
  if (c->num_pages > kIntMax || c->page_size < 16 || c->page_size > 65536 ||
      (c->page_size & (c->page_size - 1)) != 0 || c->kv_heads > 1024 || c->head_dim % 16 != 0 ||
      c->head_dim > 1024)
    return NVFP4_ERR_SHAPE;
  const int64_t rows = static_cast<int64_t>(c->kv_heads) * c->page_size;
  if (c->code_page_stride < rows * c->head_dim / 2 || c->scale_page_stride < rows * c->head_dim / 16 ||
      c->code_page_stride > kMaxPageStride || c->scale_page_stride > kMaxPageStride)
    return NVFP4_ERR_SHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
      !aligned(c->v_scales, 16) || c->code_page_stride % 16 != 0 || c->scale_page_stride % 16 != 0 ||
      !aligned(c->k_S, 4) || !aligned(c->v_S, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// Strides (elements of `size` bytes) of rows [tokens][heads][dim].
int check_rows(const void* p, int64_t token_stride, int64_t head_stride, int size) {
  if (token_stride < 0 || head_stride < 0) return NVFP4_ERR_INVALID_ARG;
  if (token_stride > kMaxStride || head_stride > kMaxStride) return NVFP4_ERR_SHAPE;
  if (!aligned(p, 16) || token_stride * size % 16 != 0 || head_stride * size % 16 != 0)
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int check_attention_sizes(int64_t batch, int64_t max_q, int64_t max_kv, int q_heads, int kv_heads,
                          int head_dim) {
  if (batch < 0 || max_q < 0 || max_kv < 0 || q_heads < 1 || kv_heads < 1) return NVFP4_ERR_INVALID_ARG;
  if (batch > 65535 || max_kv > kIntMax - 65536 || q_heads > 1024 || q_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128) || max_q > kIntMax / q_heads - 1024)
    return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_kv_append(const nvfp4_kv_cache* cache, const void* K, const void* V, int type,
                    int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                    int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                    int* status, void* stream) {
  NVFP4_RANGE("nvfp4_kv_append");
  int st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  if (type < NVFP4_TYPE_BF16 || type > NVFP4_TYPE_FP32 || tokens < 0) return NVFP4_ERR_INVALID_ARG;
  if (tokens > 0 && (K == nullptr || V == nullptr || slots == nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (tokens > kMaxStride) return NVFP4_ERR_SHAPE;
  const int size = type == NVFP4_TYPE_FP32 ? 4 : 2;
  if ((st = check_rows(K, k_token_stride, k_head_stride, size)) != NVFP4_OK) return st;
  if ((st = check_rows(V, v_token_stride, v_head_stride, size)) != NVFP4_OK) return st;
  if (!aligned(slots, 8) || !aligned(status, 4)) return NVFP4_ERR_ALIGN;
  if (tokens == 0 && status == nullptr) return NVFP4_OK;
  const int sms = sm_count();
  if (sms <= 0) return nvfp4::record_cuda_status(cudaErrorNoDevice);
  return nvfp4::record_cuda_status(nvfp4::launch_kv_append(
      *cache, nvfp4::KvRows{K, k_token_stride, k_head_stride},
      nvfp4::KvRows{V, v_token_stride, v_head_stride}, type, tokens, slots, status, sms,
      static_cast<cudaStream_t>(stream)));
}

int nvfp4_kv_read(const nvfp4_kv_cache* cache, const int64_t* slots, int64_t tokens, int type,
                  void* K, void* V, void* stream) {
  NVFP4_RANGE("nvfp4_kv_read");
  const int st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  if (type < NVFP4_TYPE_BF16 || type > NVFP4_TYPE_FP32 || tokens < 0) return NVFP4_ERR_INVALID_ARG;
  if (tokens > 0 && (K == nullptr || V == nullptr || slots == nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (tokens > kMaxStride) return NVFP4_ERR_SHAPE;
  if (!aligned(K, 32) || !aligned(V, 32) || !aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  if (tokens == 0) return NVFP4_OK;
  const int sms = sm_count();
  if (sms <= 0) return nvfp4::record_cuda_status(cudaErrorNoDevice);
  return nvfp4::record_cuda_status(nvfp4::launch_kv_read(*cache, tokens, slots, type, K, V, sms,
                                                         static_cast<cudaStream_t>(stream)));
}

int nvfp4_kv_copy_pages(const nvfp4_kv_cache* cache, int64_t layers, int64_t code_layer_stride,
                        int64_t scale_layer_stride, const int32_t* src, const int32_t* dst,
                        int64_t n, void* stream) {
  NVFP4_RANGE("nvfp4_kv_copy_pages");
  const int st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  if (layers < 0 || n < 0 || (n > 0 && (src == nullptr || dst == nullptr))) return NVFP4_ERR_INVALID_ARG;
  if (layers > 65535) return NVFP4_ERR_SHAPE;
  if (layers > 1) {
    if (code_layer_stride < 0 || scale_layer_stride < 0) return NVFP4_ERR_INVALID_ARG;
    if (code_layer_stride > kMaxStride || scale_layer_stride > kMaxStride) return NVFP4_ERR_SHAPE;
    if (code_layer_stride % 16 != 0 || scale_layer_stride % 16 != 0) return NVFP4_ERR_ALIGN;
  }
  if (n == 0 || layers == 0) return NVFP4_OK;
  for (int64_t i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= cache->num_pages || dst[i] < 0 || dst[i] >= cache->num_pages)
      return NVFP4_ERR_INVALID_ARG;
  try {
    // the pages written, in order: none twice, and none among those read
    std::vector<int32_t> out(dst, dst + n);
    std::sort(out.begin(), out.end());
    if (std::adjacent_find(out.begin(), out.end()) != out.end()) return NVFP4_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i)
      if (std::binary_search(out.begin(), out.end(), src[i])) return NVFP4_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return NVFP4_ERR_WORKSPACE;
  } catch (...) {
    return NVFP4_ERR_INVALID_ARG;
  }
  return nvfp4::record_cuda_status(nvfp4::launch_kv_copy_pages(
      *cache, layers, layers > 1 ? code_layer_stride : 0, layers > 1 ? scale_layer_stride : 0, src,
      dst, n, static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_kv_attention_workspace_size(int64_t batch, int64_t max_q, int64_t max_kv, int q_heads,
                                         int kv_heads, int head_dim) {
  if (check_attention_sizes(batch, max_q, max_kv, q_heads, kv_heads, head_dim) != NVFP4_OK) return 0;
  const int sms = sm_count();
  if (sms <= 0) return 0;
  return nvfp4::kv_attention_workspace_bytes(batch, max_q, max_kv, q_heads, kv_heads, head_dim, sms);
}

int nvfp4_kv_attention(const nvfp4_kv_cache* cache, const void* Q, int type, int q_heads,
                       int64_t total_q, int64_t q_token_stride, int64_t q_head_stride,
                       const int32_t* q_offsets, const int32_t* kv_lengths, const int32_t* table,
                       int64_t table_stride, int64_t batch, int64_t max_q, int64_t max_kv,
                       float sm_scale, int causal, int64_t window, void* out,
                       int64_t o_token_stride, int64_t o_head_stride, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream) {
  NVFP4_RANGE("nvfp4_kv_attention");
  int st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  if ((type != NVFP4_TYPE_BF16 && type != NVFP4_TYPE_FP16) || total_q < 0 || table_stride < 0 ||
      (causal != 0 && causal != 1) || window < 0 || (window > 0 && causal == 0) ||
      !std::isfinite(sm_scale))
    return NVFP4_ERR_INVALID_ARG;
  if ((st = check_attention_sizes(batch, max_q, max_kv, q_heads, cache->kv_heads, cache->head_dim)) != NVFP4_OK)
    return st;
  if (total_q > kIntMax || table_stride > kMaxStride ||
      max_kv > table_stride * static_cast<int64_t>(cache->page_size))
    return NVFP4_ERR_SHAPE;
  const bool empty = batch == 0 || total_q == 0 || max_q == 0;
  if (!empty && (Q == nullptr || out == nullptr || q_offsets == nullptr || kv_lengths == nullptr ||
                 (table == nullptr && max_kv > 0)))
    return NVFP4_ERR_INVALID_ARG;
  if ((st = check_rows(Q, q_token_stride, q_head_stride, 2)) != NVFP4_OK) return st;
  if ((st = check_rows(out, o_token_stride, o_head_stride, 2)) != NVFP4_OK) return st;
  if (!aligned(lse, 4) || !aligned(q_offsets, 4) || !aligned(kv_lengths, 4) || !aligned(table, 4))
    return NVFP4_ERR_ALIGN;
  if (empty) return NVFP4_OK;
  if (workspace == nullptr) return NVFP4_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
  const int sms = sm_count();
  if (sms <= 0) return nvfp4::record_cuda_status(cudaErrorNoDevice);
  const size_t need =
      nvfp4::kv_attention_workspace_bytes(batch, max_q, max_kv, q_heads, cache->kv_heads, cache->head_dim, sms);
  if (need == 0) return NVFP4_ERR_SHAPE;
  if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
  nvfp4::KvAttention a{};
  a.c = *cache;
  a.Q = Q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.out = out;
  a.o_token_stride = o_token_stride;
  a.o_head_stride = o_head_stride;
  a.lse = lse;
  a.q_offsets = q_offsets;
  a.kv_lengths = kv_lengths;
  a.table = table;
  a.table_stride = table_stride;
  a.type = type;
  a.q_heads = q_heads;
  a.batch = static_cast<int>(batch);
  a.total_q = static_cast<int>(total_q);
  a.max_q = static_cast<int>(max_q);
  a.max_kv = static_cast<int>(max_kv);
  a.causal = causal;
  // no sequence is longer than max_kv: a window past it hides nothing
  a.window = window > max_kv ? 0 : static_cast<int>(window);
  a.scale = sm_scale;
  return nvfp4::record_cuda_status(
      nvfp4::launch_kv_attention(a, workspace, sms, static_cast<cudaStream_t>(stream)));
}

int nvfp4_debug_kv_stalls(unsigned int* count, int reset) {
  if (count == nullptr || (reset != 0 && reset != 1)) return NVFP4_ERR_INVALID_ARG;
  cudaError_t e = cudaSuccess;
  *count = nvfp4::kv_stalls(reset != 0, &e);
  return nvfp4::record_cuda_status(e);
}

int nvfp4_debug_kv_wait_limit(int64_t cycles) {
  cudaError_t e = cudaSuccess;
  if (cycles < 0 || !nvfp4::kv_wait_limit(cycles, &e)) return NVFP4_ERR_INVALID_ARG;
  return nvfp4::record_cuda_status(e);
}

}  // extern "C"
