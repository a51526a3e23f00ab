// kv_cache.cu -- writing, reading and copying the paged NVFP4 K/V cache.
//
// Append reads 2 (or 4) bytes an element and writes 0.5625, read the reverse,
// copy moves bytes.  Measured with 8 heads of 128: append of 16001 tokens of 16
// bits 21 us (4.0 TB/s; 220 instructions a group of 16 keep the schedulers 63%
// busy beside it, neither is full: a warp's loads and its arithmetic take
// turns) and of 32 bits 25 us (5.9 TB/s), read of 100003 tokens to FP16 88 us
// (6.0 TB/s), copy of 511 pages in 16 layers 99 us (6.1 TB/s).  The last two are
// bound by HBM.  A page and layer is copied by one CTA, for caches of small pages
// and many layers: one page of 256 tokens in one layer takes 8 us, of 4096 101.
#include <type_traits>

#include <cuda_bf16.h>

#include "kv_cache.cuh"
#include "nvfp4_device.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ append

// One group of 16 as floats, and the bit pattern of its largest magnitude
// (magnitudes of one IEEE type order as their bit patterns do).
template <int kType>
__device__ __forceinline__ bool load_group(const void* p, float (&x)[16], float& amax) {
  uint32_t m = 0;
  if constexpr (kType == kFp32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = ld_stream_v4(static_cast<const float*>(p) + 4 * i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[4 * i + j] = __uint_as_float(w[j]);
        m = max(m, w[j] & 0x7FFFFFFFu);
      }
    }
    amax = __uint_as_float(m);
    return m < 0x7F800000u;
  } else {
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = ld_stream_v4(static_cast<const uint16_t*>(p) + 8 * i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m2 = __vmaxu2(m2, w[j] & 0x7FFF7FFFu);
        if constexpr (kType == kBf16) {
          x[8 * i + 2 * j] = bf16_lo(w[j]);
          x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          x[8 * i + 2 * j] = f.x;
          x[8 * i + 2 * j + 1] = f.y;
        }
      }
    }
    m = max(m2 & 0xFFFFu, m2 >> 16);
    if constexpr (kType == kBf16) {
      amax = __uint_as_float(m << 16);
      return m < 0x7F80u;
    } else {
      amax = __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
      return m < 0x7C00u;
    }
  }
}

// E2M1 code of |x| at scale v * S, decided on the exact products: |x| passes
// the midpoint t = m v S of a pair of neighbours if |x| > t, or at a tie where
// the upper one is the even code.  m v has at most 8 bits, so t is one product
// of two FP32 numbers; as |x| is an FP32 number too, |x| > t is |x| > t rounded
// down, and |x| >= t is |x| >= t rounded up.
__device__ __noinline__ uint32_t e2m1_exact(float a, float v, float S) {
  uint32_t k = 0;
  k += a > __fmul_rd(0.25f * v, S);
  k += a >= __fmul_ru(0.75f * v, S);
  k += a > __fmul_rd(1.25f * v, S);
  k += a >= __fmul_ru(1.75f * v, S);
  k += a > __fmul_rd(2.5f * v, S);
  k += a >= __fmul_ru(3.5f * v, S);
  k += a > __fmul_rd(5.0f * v, S);
  return k;
}

// Eight floats to E2M1 nibbles, round-to-nearest-even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8_rne(f32x2_t a, f32x2_t b, f32x2_t c, f32x2_t d) {
  float f[8];
  f2_unpack(a, f[0], f[1]);
  f2_unpack(b, f[2], f[3]);
  f2_unpack(c, f[4], f[5]);
  f2_unpack(d, f[6], f[7]);
  uint32_t r;
  asm("{ .reg .b8 p, q, r, s;\n"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n"
      "mov.b32 %0, {p, q, r, s}; }"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// A head's S, 1 / (6 S), and whether S is far enough from the ends of the FP32
// range for products with that to be within rounding of the quotients.
struct HeadScale {
  float S, inv6;
  bool plain;
};
__device__ __forceinline__ HeadScale head_scale(float S) {
  return {S, __fdividef(1.0f, 6.0f * S), S > 0x1p-100f && S < 0x1p100f};
}

// Codes of one group (element i in nibble i) and its scale byte.  A zero
// magnitude is stored without a sign.
__device__ __forceinline__ void quantize_group(const float (&x)[16], float amax, const HeadScale& hs,
                                               uint32_t (&codes)[2], uint32_t& scale) {
  const float S = hs.S;
  // The scale code of fl32(fl32(a / 6) / S): as below, from a quotient taken
  // too small and too large; the divisions themselves where the two differ.
  const float u = amax * hs.inv6;
  uint32_t two;
  asm("{ .reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %1, %2; cvt.u32.u16 %0, t; }"
      : "=r"(two) : "f"(u * (1.0f + 0x1p-20f)), "f"(u * (1.0f - 0x1p-20f)));
  int b = two & 0xFF;
  if (b != static_cast<int>(two >> 8) || !hs.plain || !(u > 0x1p-100f && u < 0x1p100f))
    b = e4m3_code_rne_sat(__fdiv_rn(__fdiv_rn(amax, 6.0f), S));
  b = amax == 0.0f ? 0 : clamp_code(b);
  scale = b;
  codes[0] = codes[1] = 0;
  if (b == 0) return;
  const float v = e4m3_value(b);
  const float vs = v * S;
  // Fast path: the hardware's E2M1 conversion of x / (v S) taken a little too
  // small and a little too large (by 2^-20 to 2^-19; the reciprocal and the
  // products are within 2^-21).  Rounding is monotone, so where both give the
  // same codes they are those of the exact quotient; otherwise some element is
  // next to a midpoint, and the group's decisions are taken exactly.
  const float inv = __fdividef(1.0f, vs);
  const f32x2_t lo = f2_pack(inv * (1.0f - 0x1.8p-20f), inv * (1.0f - 0x1.8p-20f));
  const f32x2_t hi = f2_pack(inv * (1.0f + 0x1.8p-20f), inv * (1.0f + 0x1.8p-20f));
  uint32_t other[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    codes[i] = e2m1x8_rne(f2_mul(f2_pack(x[8 * i], x[8 * i + 1]), lo), f2_mul(f2_pack(x[8 * i + 2], x[8 * i + 3]), lo),
                          f2_mul(f2_pack(x[8 * i + 4], x[8 * i + 5]), lo), f2_mul(f2_pack(x[8 * i + 6], x[8 * i + 7]), lo));
    other[i] = e2m1x8_rne(f2_mul(f2_pack(x[8 * i], x[8 * i + 1]), hi), f2_mul(f2_pack(x[8 * i + 2], x[8 * i + 3]), hi),
                          f2_mul(f2_pack(x[8 * i + 4], x[8 * i + 5]), hi), f2_mul(f2_pack(x[8 * i + 6], x[8 * i + 7]), hi));
  }
  if (codes[0] != other[0] || codes[1] != other[1] || !(vs > 0x1p-100f && vs < 0x1p100f)) {
    codes[0] = codes[1] = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t k = e2m1_exact(fabsf(x[i]), v, S) | (x[i] < 0.0f ? 8u : 0u);
      codes[i >> 3] |= k << (4 * (i & 7));
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // -0 becomes +0: keep a sign bit only beside a nonzero magnitude
    const uint32_t nz = (codes[i] & 0x77777777u) + 0x77777777u;
    codes[i] &= nz | 0x77777777u;
  }
}

// How tokens and groups of 16 (those of K, then of V) are laid over a CTA: a
// thread keeps its group's column and takes every (grid * per_pass)-th token,
// so that divisions are made once.  Rows with more groups than a CTA has
// threads are taken in several rounds of columns.
struct Columns {
  uint32_t per_token;  // groups of a token, K and V
  uint32_t per_pass;   // tokens a CTA takes side by side
  int page_shift;
};

// Calls body(token, isv, head, group) for this thread's groups, kUnroll tokens
// at a time (token < 0: nothing to do).
template <int kUnroll, typename Body>
__device__ __forceinline__ void for_groups(const nvfp4_kv_cache& c, const Columns& m, int64_t tokens, Body body) {
  const uint32_t gd = c.head_dim / 16, gt = m.per_token / 2;
  const uint32_t tl = m.per_pass > 1 ? threadIdx.x / m.per_token : 0u;
  if (tl >= m.per_pass) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * m.per_pass;
  for (uint32_t col = threadIdx.x - tl * m.per_token; col < m.per_token; col += kThreads) {
    const bool isv = col >= gt;
    const uint32_t r = isv ? col - gt : col, h = r / gd, g = r - h * gd;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * m.per_pass + tl; t < tokens; t += kUnroll * step) {
      int64_t ts[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) ts[i] = t + i * step < tokens ? t + i * step : -1;
      body(ts, isv, h, g);
    }
    if (m.per_pass > 1) break;
  }
}

// Byte offsets of a group of the row at `slot` in a codes and in a scales
// array; false for a slot that is not in the cache.
__device__ __forceinline__ bool locate(const nvfp4_kv_cache& c, int page_shift, int64_t slot, uint32_t h, uint32_t g,
                                       int64_t& codes, int64_t& scales) {
  if (slot < 0 || (slot >> page_shift) >= c.num_pages) return false;
  const uint64_t page = static_cast<uint64_t>(slot >> page_shift);
  const uint32_t row = static_cast<uint32_t>(slot) & ((1u << page_shift) - 1);
  const uint32_t gd = c.head_dim / 16;
  const uint64_t in_page = (static_cast<uint64_t>(h) << page_shift) + row;
  codes = static_cast<int64_t>(page * static_cast<uint32_t>(c.code_page_stride) + in_page * (8 * gd) + 8 * g);
  scales = static_cast<int64_t>(page * static_cast<uint32_t>(c.scale_page_stride) + in_page * gd + g);
  return true;
}

// Tokens whose loads are in flight per thread, and resident CTAs an SM, which
// are as many as are launched (two waves of 4 with 4 tokens: 100003 tokens read
// in 96 us, one wave 93, 3 with 8 tokens 88, 2 with 16 88 but 500 tokens 3.5
// instead of 2.7; append of 16001 with 4 tokens and 2 CTAs 1 us more).
constexpr int kAppendUnroll = 2, kReadUnroll = 8;
constexpr int kAppendCtas = 4, kReadCtas = 3;

// Bytes of a group, for the checks of its address.
template <int kBytes>
struct Group {
  char bytes[kBytes];
};

template <int kType>
__global__ void __launch_bounds__(kThreads, kAppendCtas)
kv_append_kernel(nvfp4_kv_cache c, KvRows K, KvRows V, Columns m, int64_t tokens,
                 const int64_t* __restrict__ slots, int* __restrict__ status) {
  for_groups<kAppendUnroll>(c, m, tokens, [&](const int64_t(&ts)[kAppendUnroll], bool isv, uint32_t h, uint32_t g) {
    const KvRows& X = isv ? V : K;
    const float* const all_S = isv ? c.v_S : c.k_S;
    const HeadScale S = head_scale(*checked(all_S + h, all_S, c.kv_heads * 4, kSiteKvS));
    uint8_t* const codes_out = isv ? c.v_codes : c.k_codes;
    uint8_t* const scales_out = isv ? c.v_scales : c.k_scales;
    int64_t slot[kAppendUnroll];
    float x[kAppendUnroll][16], amax[kAppendUnroll];
    bool finite[kAppendUnroll];
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i) {
      slot[i] = ts[i] >= 0 ? *checked(slots + ts[i], slots, tokens * 8, kSiteKvSlots) : -1;
      const int64_t at = (ts[i] < 0 ? 0 : ts[i]) * X.token_stride + h * X.head_stride + 16 * g;
      constexpr int kSize = kType == kFp32 ? 4 : 2;
      const int64_t bytes = rows_extent(tokens, X.token_stride, c.kv_heads, X.head_stride, c.head_dim, kSize);
      finite[i] = load_group<kType>(
          checked(reinterpret_cast<const Group<16 * kSize>*>(static_cast<const char*>(X.p) + at * kSize), X.p, bytes,
                  kSiteKvRowsIn),
          x[i], amax[i]);
    }
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i) {
      int64_t co, so;
      if (!locate(c, m.page_shift, slot[i], h, g, co, so)) continue;
      uint32_t codes[2] = {0u, 0u}, scale = 0x7F;
      if (finite[i])
        quantize_group(x[i], amax[i], S, codes, scale);
      else if (status)
        *checked(status, status, 4, kSiteKvStatus) = NVFP4_ERR_NONFINITE;
      *checked(reinterpret_cast<uint2*>(codes_out + co), codes_out, codes_extent(c), kSiteKvCodes) =
          make_uint2(codes[0], codes[1]);
      *checked(scales_out + so, scales_out, scales_extent(c), kSiteKvScales) = static_cast<uint8_t>(scale);
    }
  });
}

// -------------------------------------------------------------------- read

// (evict first: what is read back is written once, and should not push the
// cache's pages out of L2; append of 16001 tokens and their read back 47 -> 44 us)
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <int kType>
__global__ void __launch_bounds__(kThreads, kReadCtas)
kv_read_kernel(nvfp4_kv_cache c, Columns m, int64_t tokens, const int64_t* __restrict__ slots, void* __restrict__ K,
               void* __restrict__ V) {
  constexpr int kSize = kType == kFp32 ? 4 : 2;
  for_groups<kReadUnroll>(c, m, tokens, [&](const int64_t(&ts)[kReadUnroll], bool isv, uint32_t h, uint32_t g) {
    const float* const all_S = isv ? c.v_S : c.k_S;
    const float S = *checked(all_S + h, all_S, c.kv_heads * 4, kSiteKvS);
    const uint8_t* const codes_in = isv ? c.v_codes : c.k_codes;
    const uint8_t* const scales_in = isv ? c.v_scales : c.k_scales;
    int64_t slot[kReadUnroll];
    uint2 w[kReadUnroll];
    uint32_t sc[kReadUnroll];
#pragma unroll
    for (int i = 0; i < kReadUnroll; ++i) slot[i] = ts[i] >= 0 ? *checked(slots + ts[i], slots, tokens * 8, kSiteKvSlots) : -1;
#pragma unroll
    for (int i = 0; i < kReadUnroll; ++i) {
      int64_t co, so;
      w[i] = make_uint2(0u, 0u);
      sc[i] = 0;
      if (locate(c, m.page_shift, slot[i], h, g, co, so)) {
        w[i] = *checked(reinterpret_cast<const uint2*>(codes_in + co), codes_in, codes_extent(c), kSiteKvCodes);
        sc[i] = *checked(scales_in + so, scales_in, scales_extent(c), kSiteKvScales);
      }
    }
#pragma unroll
    for (int i = 0; i < kReadUnroll; ++i) {
      if (ts[i] < 0) continue;
      uint32_t hh;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hh) : "h"(static_cast<uint16_t>(sc[i] | (sc[i] << 8))));
      char* const rows = static_cast<char*>(isv ? V : K);
      char* const out = reinterpret_cast<char*>(
          checked(reinterpret_cast<Group<16 * kSize>*>(rows + ((ts[i] * c.kv_heads + h) * c.head_dim + 16 * g) * kSize),
                  rows, tokens * c.kv_heads * c.head_dim * kSize, kSiteKvRowsOut));
      uint32_t r[16];
      const uint32_t words[2] = {w[i].x, w[i].y};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t e[4];
        e2m1x8_to_f16x2(words[u], e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // code * scale is exact in FP16 (6 bits)
          const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&e[j]), *reinterpret_cast<const __half2*>(&hh));
          const float2 f = __half22float2(v);
          const float a = f.x * S, z = f.y * S;
          if constexpr (kType == kFp32) {
            r[8 * u + 2 * j] = __float_as_uint(a);
            r[8 * u + 2 * j + 1] = __float_as_uint(z);
          } else if constexpr (kType == kBf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(a, z);
            r[4 * u + j] = *reinterpret_cast<const uint32_t*>(&b);
          } else {
            const __half2 b = __floats2half2_rn(a, z);
            r[4 * u + j] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
      }
      const uint32_t lo[8] = {r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7]};
      store32(out, lo);
      if constexpr (kType == kFp32) {
        const uint32_t hi[8] = {r[8], r[9], r[10], r[11], r[12], r[13], r[14], r[15]};
        store32(out + 32, hi);
      }
    }
  });
}

// -------------------------------------------------------------------- copy

// Pairs travel in the kernel's parameters: no staging copy, nothing to keep
// alive after the call, and a captured launch replays with its own pairs.
template <int kPairs>
struct PagePairs {
  int2 p[kPairs];
};

template <int kPairs>
__global__ void __launch_bounds__(kThreads)
kv_copy_kernel(nvfp4_kv_cache c, int64_t code_layer_stride, int64_t scale_layer_stride, int n,
               const __grid_constant__ PagePairs<kPairs> pairs) {
  const int64_t layer = blockIdx.y;
  const int64_t rows = static_cast<int64_t>(c.kv_heads) * c.page_size;
  const int64_t cv = rows * c.head_dim / 32, sv = rows * c.head_dim / 256;  // 16-byte vectors
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t src = pairs.p[i].x, dst = pairs.p[i].y;
    auto move = [&](uint8_t* all, int64_t layer_stride, int64_t page_stride, int64_t vecs, int site) {
      uint8_t* const base = all + layer * layer_stride;
      const int64_t bytes = site == kSiteKvCodes ? codes_extent(c) : scales_extent(c);
      const uint4* const s = reinterpret_cast<const uint4*>(base + src * page_stride);
      uint4* const d = reinterpret_cast<uint4*>(base + dst * page_stride);
      auto in_base = [&](auto* p) { return checked(p, base, bytes, site); };
      int64_t v = threadIdx.x;
      for (; v + 3 * kThreads < vecs; v += 4 * kThreads) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = ld_stream_v4(in_base(s + v + u * kThreads));
#pragma unroll
        for (int u = 0; u < 4; ++u) *in_base(d + v + u * kThreads) = x[u];
      }
      for (; v < vecs; v += kThreads) *in_base(d + v) = ld_stream_v4(in_base(s + v));
    };
    move(c.k_codes, code_layer_stride, c.code_page_stride, cv, kSiteKvCodes);
    move(c.v_codes, code_layer_stride, c.code_page_stride, cv, kSiteKvCodes);
    move(c.k_scales, scale_layer_stride, c.scale_page_stride, sv, kSiteKvScales);
    move(c.v_scales, scale_layer_stride, c.scale_page_stride, sv, kSiteKvScales);
  }
}

template <int kPairs>
cudaError_t copy_chunk(const nvfp4_kv_cache& c, int64_t layers, int64_t cls, int64_t sls,
                       const int* src, const int* dst, int n, cudaStream_t stream) {
  PagePairs<kPairs> pp;
  for (int i = 0; i < n; ++i) pp.p[i] = make_int2(src[i], dst[i]);
  for (int i = n; i < kPairs; ++i) pp.p[i] = make_int2(0, 0);
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(layers));
  kv_copy_kernel<kPairs><<<grid, kThreads, 0, stream>>>(c, cls, sls, n, pp);
  return cudaGetLastError();
}

struct TokenGrid {
  Columns m;
  unsigned blocks;
};
// One wave of resident CTAs at most.
TokenGrid token_grid(const nvfp4_kv_cache& c, int64_t tokens, int num_sms, int ctas_per_sm) {
  TokenGrid g{};
  g.m.per_token = 2u * c.kv_heads * (c.head_dim / 16);
  g.m.per_pass = g.m.per_token <= kThreads ? kThreads / g.m.per_token : 1;
  while ((1 << g.m.page_shift) < c.page_size) ++g.m.page_shift;
  int64_t blocks = (tokens + g.m.per_pass - 1) / g.m.per_pass;
  const int64_t wave = static_cast<int64_t>(num_sms) * ctas_per_sm;
  if (blocks > wave) blocks = wave;
  g.blocks = static_cast<unsigned>(blocks);
  return g;
}

}  // namespace

cudaError_t launch_kv_append(const nvfp4_kv_cache& c, const KvRows& K, const KvRows& V, int type,
                             int64_t tokens, const int64_t* slots, int* status, int num_sms,
                             cudaStream_t stream) {
  if (status) {
    const cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int), stream);  // NVFP4_OK
    if (e != cudaSuccess) return e;
  }
  if (tokens == 0) return cudaSuccess;
  const TokenGrid g = token_grid(c, tokens, num_sms, kAppendCtas);
  auto launch = [&](auto t) {
    kv_append_kernel<decltype(t)::value><<<g.blocks, kThreads, 0, stream>>>(c, K, V, g.m, tokens, slots, status);
  };
  if (type == kBf16) launch(std::integral_constant<int, kBf16>{});
  else if (type == kFp16) launch(std::integral_constant<int, kFp16>{});
  else launch(std::integral_constant<int, kFp32>{});
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const nvfp4_kv_cache& c, int64_t tokens, const int64_t* slots, int type,
                           void* K, void* V, int num_sms, cudaStream_t stream) {
  if (tokens == 0) return cudaSuccess;
  const TokenGrid g = token_grid(c, tokens, num_sms, kReadCtas);
  auto launch = [&](auto t) {
    kv_read_kernel<decltype(t)::value><<<g.blocks, kThreads, 0, stream>>>(c, g.m, tokens, slots, K, V);
  };
  if (type == kBf16) launch(std::integral_constant<int, kBf16>{});
  else if (type == kFp16) launch(std::integral_constant<int, kFp16>{});
  else launch(std::integral_constant<int, kFp32>{});
  return cudaGetLastError();
}

cudaError_t launch_kv_copy_pages(const nvfp4_kv_cache& c, int64_t layers,
                                 int64_t code_layer_stride, int64_t scale_layer_stride,
                                 const int* src, const int* dst, int64_t n, cudaStream_t stream) {
  if (layers == 0) return cudaSuccess;
  constexpr int kSmall = 64, kLarge = 1024;  // 0.5 and 8 KB of parameters
  for (int64_t i = 0; i < n;) {
    const int64_t left = n - i;
    const int m = static_cast<int>(left < kLarge ? left : kLarge);
    const cudaError_t e =
        m <= kSmall ? copy_chunk<kSmall>(c, layers, code_layer_stride, scale_layer_stride, src + i, dst + i, m, stream)
                    : copy_chunk<kLarge>(c, layers, code_layer_stride, scale_layer_stride, src + i, dst + i, m, stream);
    if (e != cudaSuccess) return e;
    i += m;
  }
  return cudaSuccess;
}

}  // namespace nvfp4
