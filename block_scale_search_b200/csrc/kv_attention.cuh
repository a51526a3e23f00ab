// kv_attention.cuh -- what the two attention kernels over the NVFP4 cache share:
// a call's parameters, number conversions, the mask, and the results' rounding.
#pragma once

#include <atomic>

#include "kv_cache.cuh"
#include "nvfp4_device.cuh"

namespace nvfp4 {

// Probabilities P = 2^(score - m), all factors in base 2, go to FP16 for the
// tensor cores.  m is set 2^7 below the largest score so far and moves when a
// score makes P pass 2^15 (of FP16's 65504): the largest P is 2^7 to 2^15, so
// that FP16 keeps its 11 bits down to 2^-21 of the largest weight and half a
// step of 2^-32 below.  (With m at the largest score 131071 tokens 24 bits below
// one whose V is 0, spread by a third of a bit, came out 1% off, 82% at 25.5
// bits; so they are 2^-17 off.)
constexpr float kAim = 7.0f, kTop = 15.0f;
// m for the largest score, x f: not above its exact value - kAim, so that P is
// at least 2^7 there, and at most 2^15 below 2^25, where FP32 steps are 4 or
// less.  Rows whose scores may lie further out (|q| is below 2^16, |k| at most
// 6 * 448) have their exponents held at kTop: tokens with the largest score then
// have equal weights and the others theirs, to what FP32 knows of such scores.
// Holding takes an instruction a score, so the loops exist with and without it
// (a branch in one loop: the chunk case 520 us, so 508; 48 sequences of up to
// 8192 tokens 57.1 and 57.0).
__device__ __forceinline__ float m_for(float x, float f) { return __fadd_rd(__fmul_rd(x, f), -kAim); }
template <int D>
__device__ __forceinline__ bool may_pass_top(float f) { return !(f < 0x1p25f / (D * 65536.0f * 2688.0f)); }
__device__ __forceinline__ float held(float y) {
  float r;  // (a NaN stays)
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(y), "f"(kTop));
  return r;
}

struct Params {
  KvAttention a;
  int group, page_shift;
  float scale_log2;
  float* partial;  // [CTA][2][R * D] sums, then [CTA][2][R * 2] maximum and sum
  float* partial_ml;
  int ctas;
  int4* cut;       // [CTA]: sequence, item, first CTA and number of pieces (0: none) of a cut item; or NULL
  int rows_limit;  // kv_rows_kernel serves sequences with at most so many query rows for a KV head
  int row_blocks, splits;  // of kv_prompt_kernel
  float* split_o;          // [item][split][256][D] sums, and their maxima and sums
  float2* split_ml;
};

// Raises a kernel's limit of dynamic shared memory, once per device.
struct SmemOptIn {
  std::atomic<uint64_t> done{0};  // bit d: set on device d
  cudaError_t set(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};

// Prompts (kv_prompt.cu): how a call's items (256 query rows of a sequence and
// KV head) are laid over CTAs, and the launch.
struct PromptPlan {
  int64_t row_blocks, items;
  int splits;
};
PromptPlan prompt_plan(int64_t batch, int64_t rows, int64_t max_kv, int kv_heads, int num_sms);
size_t prompt_workspace_bytes(const PromptPlan& plan, int head_dim);
cudaError_t launch_kv_prompt(Params& p, const PromptPlan& plan, void* workspace, cudaStream_t stream);

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float to_f32(uint16_t v, int type) {
  return type == kBf16 ? __uint_as_float(static_cast<uint32_t>(v) << 16)
                       : __half2float(__ushort_as_half(v));
}

// Scaling of a query row whose largest magnitude is mx: the row goes to FP16
// times `shrink`, a power of two that puts its maximum into [2^15, 2^16), the
// top of FP16's range.  So rows of FP16 stay exact (shrink >= 1), and of a row
// of BF16 all elements down to 2^-32 of the largest do; smaller ones are rounded
// to steps of at most 2^-39 of it.  (Rows below 2^-111 lie lower in FP16: shrink
// is at most 2^126, a finite number.)  A row that holds Inf goes all to NaN: its
// scores could all be -inf, which stands for hidden ones.  `factor` turns a dot
// product into a score in base 2.  It is kept above 0 (a negative one turns the
// row's sign), so that it keeps the order of scores and a hidden score's -inf.
__device__ __forceinline__ void row_scale(float mx, float scale, float& shrink, float& factor) {
  const uint32_t e = min(max(__float_as_uint(mx) >> 23, 16u), 254u);
  shrink = __uint_as_float((269u - e) << 23);
  factor = __uint_as_float((e - 15u) << 23) * scale;
  if (factor < 0.0f) factor = -factor, shrink = -shrink;
  if (factor < 0x1p-120f) factor = 0x1p-120f;
  if (mx == INFINITY) shrink = __uint_as_float(0x7FC00000u);
}

// One sequence: its first query row, new tokens and cached tokens, whatever the
// device arrays hold brought into the call's bounds.
struct Span {
  int q0, lq, lk;
};
__device__ __forceinline__ Span span_of(const Params& p, int b) {
  Span s;
  auto offset = [&](int i) {
    return *checked(p.a.q_offsets + i, p.a.q_offsets, (static_cast<int64_t>(p.a.batch) + 1) * 4, kSiteKvOffsets);
  };
  const int lo = offset(b), hi = offset(b + 1);
  s.q0 = min(max(lo, 0), p.a.total_q);
  s.lq = min(min(max(hi, s.q0), p.a.total_q) - s.q0, p.a.max_q);
  s.lk = min(max(*checked(p.a.kv_lengths + b, p.a.kv_lengths, static_cast<int64_t>(p.a.batch) * 4, kSiteKvOffsets), 0),
             p.a.max_kv);
  return s;
}

// Entry i of a sequence's row of the page table.
__device__ __forceinline__ int table_entry(const Params& p, const int* row, int i) {
  const int64_t pages = (static_cast<int64_t>(p.a.max_kv) + p.a.c.page_size - 1) / p.a.c.page_size;
  return *checked(row + i, p.a.table, ((p.a.batch - 1) * p.a.table_stride + pages) * 4, kSiteKvTable);
}
// 8 elements of a query row, from its element d on.
__device__ __forceinline__ uint4 query_piece(const Params& p, const uint16_t* at) {
  return *checked(reinterpret_cast<const uint4*>(at), p.a.Q,
                  rows_extent(p.a.total_q, p.a.q_token_stride, p.a.q_heads, p.a.q_head_stride, p.a.c.head_dim, 2),
                  kSiteKvRowsIn);
}
__device__ __forceinline__ float head_S(const Params& p, const float* S, int h) {
  return *checked(S + h, S, p.a.c.kv_heads * 4, kSiteKvS);
}

// Tokens [lo, hi) that row `row` of a sequence (query row / G, head h G + row % G)
// may see; none behind its last row.
__device__ __forceinline__ void visible(const Params& p, const Span& s, int row, int& lo, int& hi) {
  if (row >= s.lq * p.group) {
    lo = hi = 0;
    return;
  }
  const int pos = s.lk - s.lq + row / p.group;
  hi = p.a.causal ? min(s.lk, pos + 1) : s.lk;
  lo = p.a.window > 0 ? max(0, pos - p.a.window + 1) : 0;
}

__device__ __forceinline__ void write_row(const Params& p, const Span& s, int h, int row, int d, float4 v,
                                          float inv) {
  const int64_t t = s.q0 + row / p.group;
  const int64_t head = h * p.group + row % p.group;
  uint16_t* o = static_cast<uint16_t*>(p.a.out) + t * p.a.o_token_stride + head * p.a.o_head_stride + d;
  uint2 w;
  if (p.a.type == kBf16) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y * inv), "f"(v.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w * inv), "f"(v.z * inv));
  } else {
    w.x = pack_f16x2(v.x * inv, v.y * inv);
    w.y = pack_f16x2(v.z * inv, v.w * inv);
  }
  *checked(reinterpret_cast<uint2*>(o), p.a.out,
           rows_extent(p.a.total_q, p.a.o_token_stride, p.a.q_heads, p.a.o_head_stride, p.a.c.head_dim, 2), kSiteKvRowsOut) = w;
}

__device__ __forceinline__ void write_lse(const Params& p, const Span& s, int h, int row, float m, float l) {
  if (p.a.lse == nullptr) return;
  const int64_t t = s.q0 + row / p.group;
  *checked(p.a.lse + t * p.a.q_heads + h * p.group + row % p.group, p.a.lse,
           static_cast<int64_t>(p.a.total_q) * p.a.q_heads * 4, kSiteKvLse) =
      l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

}  // namespace nvfp4
