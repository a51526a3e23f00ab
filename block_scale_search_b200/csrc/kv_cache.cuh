// kv_cache.cuh -- the paged NVFP4 key/value cache: launch functions and the
// helpers that its kernels share.
//
// Layout of one tensor (K or V) of one layer: pages of `page` tokens,
//   codes  [page id][KV head][row][dim / 2]    page stride given in bytes
//   scales [page id][KV head][row][dim / 16]   page stride given in bytes
// so that 16 rows of one head are one contiguous piece of 8 * dim code bytes
// and one of dim scale bytes: what the attention kernels copy at a time.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "checks.cuh"
#include "nvfp4hs.h"

namespace nvfp4 {

// Where a check of the checked build failed (checks.cuh): every global address
// of the cache's kernels goes through checked() or checked_at().
enum KvCheckSite : int {
  kSiteKvRowsIn = 64, kSiteKvRowsOut, kSiteKvSlots, kSiteKvStatus, kSiteKvCodes, kSiteKvScales, kSiteKvS,
  kSiteKvOffsets, kSiteKvTable, kSiteKvLse, kSiteKvPartial, kSiteKvCut, kSiteKvSplit
};

// Bytes of one layer's codes and scales, from the first page to the last one's end.
__device__ __forceinline__ int64_t codes_extent(const nvfp4_kv_cache& c) {
  return (c.num_pages - 1) * c.code_page_stride + static_cast<int64_t>(c.kv_heads) * c.page_size * (c.head_dim / 2);
}
__device__ __forceinline__ int64_t scales_extent(const nvfp4_kv_cache& c) {
  return (c.num_pages - 1) * c.scale_page_stride + static_cast<int64_t>(c.kv_heads) * c.page_size * (c.head_dim / 16);
}
// Bytes of strided rows [tokens][heads][dim] of elements of `size` bytes.
__device__ __forceinline__ int64_t rows_extent(int64_t tokens, int64_t token_stride, int heads, int64_t head_stride,
                                               int dim, int size) {
  return ((tokens - 1) * token_stride + (heads - 1) * head_stride + dim) * size;
}
// checked() of a T at `at` + kSkip, for addresses kept as integers: what to use as `at`.
template <typename T, int kSkip = 0>
__device__ __forceinline__ uint64_t checked_at(uint64_t at, const void* base, int64_t bytes, int site) {
#ifdef NVFP4HS_CHECKS
  return reinterpret_cast<uint64_t>(checked(reinterpret_cast<const T*>(at + kSkip), base, bytes, site)) - kSkip;
#else
  return at;
#endif
}

// A row's element type of the calls that take several.
enum : int { kBf16 = NVFP4_TYPE_BF16, kFp16 = NVFP4_TYPE_FP16, kFp32 = NVFP4_TYPE_FP32 };

struct KvRows {  // strided rows [token][head][dim] of K or V, strides in elements
  const void* p;
  int64_t token_stride, head_stride;
};

// The eight E2M1 values of a word as four f16x2, byte i's low nibble in the
// low half of r[i].
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  asm("{ .reg .b8 a, b, c, d;\n"
      "mov.b32 {a, b, c, d}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

cudaError_t launch_kv_append(const nvfp4_kv_cache& c, const KvRows& K, const KvRows& V, int type,
                             int64_t tokens, const int64_t* slots, int* status, int num_sms,
                             cudaStream_t stream);
cudaError_t launch_kv_read(const nvfp4_kv_cache& c, int64_t tokens, const int64_t* slots, int type,
                           void* K, void* V, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_copy_pages(const nvfp4_kv_cache& c, int64_t layers,
                                 int64_t code_layer_stride, int64_t scale_layer_stride,
                                 const int* src, const int* dst, int64_t n, cudaStream_t stream);

// One attention call, checked by the entry point.
struct KvAttention {
  nvfp4_kv_cache c;
  const void* Q;
  int64_t q_token_stride, q_head_stride;
  void* out;
  int64_t o_token_stride, o_head_stride;
  float* lse;  // [total_q][q_heads] or NULL
  const int* q_offsets;
  const int* kv_lengths;
  const int* table;
  int64_t table_stride;
  int type, q_heads, batch, total_q, max_q, max_kv, causal, window;
  float scale;
};

// 0 for a call whose bounds allow more work than the kernels can count.
size_t kv_attention_workspace_bytes(int64_t batch, int64_t max_q, int64_t max_kv, int q_heads,
                                    int kv_heads, int head_dim, int num_sms);
cudaError_t launch_kv_attention(const KvAttention& a, void* workspace, int num_sms,
                                cudaStream_t stream);

}  // namespace nvfp4
