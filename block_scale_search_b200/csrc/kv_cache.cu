// kv_cache.cu -- writing, reading and copying the paged NVFP4 K/V cache.
//
// All three are bound by HBM: append reads 2 (or 4) bytes an element and
// writes 0.5625, read the reverse, copy moves bytes.
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

// Codes of one group (element i in nibble i) and its scale byte.  A zero
// magnitude is stored without a sign.
__device__ __forceinline__ void quantize_group(const float (&x)[16], float amax, float S,
                                               uint32_t (&codes)[2], uint32_t& scale) {
  const int b = amax == 0.0f ? 0 : clamp_code(e4m3_code_rne_sat(__fdiv_rn(__fdiv_rn(amax, 6.0f), S)));
  scale = b;
  codes[0] = codes[1] = 0;
  if (b == 0) return;
  const float v = e4m3_value(b);
  const float vs = v * S;
  // Fast path: y = x / (v S) within 2^-21, rounded by the hardware's E2M1
  // conversion.  Its decision is the exact one unless y lies within 2^-20 of a
  // midpoint; every midpoint is a float whose low 21 bits are 0, so the test
  // is on those bits (it also sends 0 and grid values to the exact path).
  uint32_t near = 0xFFFFFFFFu;
  const float inv = __fdividef(1.0f, vs);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y0 = x[2 * i] * inv, y1 = x[2 * i + 1] * inv;
    near = min(near, min((__float_as_uint(y0) + 8u) & 0x1FFFFFu, (__float_as_uint(y1) + 8u) & 0x1FFFFFu));
    codes[i >> 2] |= e2m1x2_rne(y0, y1) << (8 * (i & 3));
  }
  if (near <= 16u || !(vs > 0x1p-100f && vs < 0x1p100f)) {
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

template <int kType>
__global__ void __launch_bounds__(kThreads)
kv_append_kernel(nvfp4_kv_cache c, KvRows K, KvRows V, int64_t tokens, int tile,
                 const int64_t* __restrict__ slots, int* __restrict__ status) {
  const uint32_t gd = c.head_dim / 16, gt = gd * c.kv_heads, unit = 2 * gt;
  const int64_t page = c.page_size, nslots = c.num_pages * page;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile; t0 < tokens;
       t0 += static_cast<int64_t>(gridDim.x) * tile) {
    const int64_t left = tokens - t0;
    const uint32_t n = static_cast<uint32_t>(left < tile ? left : tile) * unit;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t tl = i / unit;
      uint32_t r = i - tl * unit;
      const bool isv = r >= gt;
      if (isv) r -= gt;
      const uint32_t h = r / gd, g = r - h * gd;
      const int64_t t = t0 + tl;
      const int64_t slot = slots[t];
      if (slot < 0 || slot >= nslots) continue;
      const KvRows& X = isv ? V : K;
      const int64_t at = t * X.token_stride + h * X.head_stride + 16 * g;
      float x[16], amax;
      const bool finite = load_group<kType>(
          static_cast<const char*>(X.p) + at * (kType == kFp32 ? 4 : 2), x, amax);
      uint32_t codes[2] = {0u, 0u}, scale = 0x7F;
      if (finite)
        quantize_group(x, amax, (isv ? c.v_S : c.k_S)[h], codes, scale);
      else if (status)
        *status = NVFP4_ERR_NONFINITE;
      const int64_t p = slot / page, row = slot - p * page;
      const int64_t in_page = h * page + row;
      uint8_t* cd = (isv ? c.v_codes : c.k_codes) + p * c.code_page_stride + in_page * (gd * 8) + g * 8;
      uint8_t* sc = (isv ? c.v_scales : c.k_scales) + p * c.scale_page_stride + in_page * gd + g;
      *reinterpret_cast<uint2*>(cd) = make_uint2(codes[0], codes[1]);
      *sc = static_cast<uint8_t>(scale);
    }
  }
}

// -------------------------------------------------------------------- read

// Value of any scale byte (0x7F and the negative codes' NaN give NaN).
__device__ __forceinline__ float scale_value(uint32_t byte) {
  uint32_t hh;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hh) : "h"(static_cast<uint16_t>(byte)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(hh & 0xFFFFu)));
}

template <int kType>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(nvfp4_kv_cache c, int64_t tokens, int tile, const int64_t* __restrict__ slots,
               void* __restrict__ K, void* __restrict__ V) {
  // one thread writes half a group: 8 elements, one 16- or 32-byte store
  const uint32_t gd = c.head_dim / 16, ht = 2 * gd * c.kv_heads, unit = 2 * ht;
  const int64_t page = c.page_size, nslots = c.num_pages * page;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile; t0 < tokens;
       t0 += static_cast<int64_t>(gridDim.x) * tile) {
    const int64_t left = tokens - t0;
    const uint32_t n = static_cast<uint32_t>(left < tile ? left : tile) * unit;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t tl = i / unit;
      uint32_t r = i - tl * unit;
      const bool isv = r >= ht;
      if (isv) r -= ht;
      const uint32_t h = r / (2 * gd), e = r - h * (2 * gd);  // e: half-group of the row
      const int64_t t = t0 + tl;
      const int64_t slot = slots[t];
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (slot >= 0 && slot < nslots) {
        const int64_t p = slot / page, row = slot - p * page;
        const int64_t in_page = h * page + row;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(
            (isv ? c.v_codes : c.k_codes) + p * c.code_page_stride + in_page * (gd * 8) + e * 4);
        const float v = scale_value((isv ? c.v_scales : c.k_scales)[p * c.scale_page_stride + in_page * gd + e / 2]);
        const float S = (isv ? c.v_S : c.k_S)[h];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t hh = e2m1x2_to_f16x2((w >> (8 * j)) & 0xFFu);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh));
          y[2 * j] = (f.x * v) * S;  // the first product is exact (6 bits)
          y[2 * j + 1] = (f.y * v) * S;
        }
      }
      const int64_t at = (t * c.kv_heads + h) * c.head_dim + 8 * e;
      void* out = isv ? V : K;
      if constexpr (kType == kFp32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(static_cast<float*>(out) + at),
                     "r"(__float_as_uint(y[0])), "r"(__float_as_uint(y[1])), "r"(__float_as_uint(y[2])),
                     "r"(__float_as_uint(y[3])), "r"(__float_as_uint(y[4])), "r"(__float_as_uint(y[5])),
                     "r"(__float_as_uint(y[6])), "r"(__float_as_uint(y[7])) : "memory");
      } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (kType == kBf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
            o[j] = *reinterpret_cast<const uint32_t*>(&b);
          } else {
            const __half2 b = __floats2half2_rn(y[2 * j], y[2 * j + 1]);
            o[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
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
    auto move = [&](uint8_t* base, int64_t layer_stride, int64_t page_stride, int64_t vecs) {
      const uint4* s = reinterpret_cast<const uint4*>(base + layer * layer_stride + src * page_stride);
      uint4* d = reinterpret_cast<uint4*>(base + layer * layer_stride + dst * page_stride);
      int64_t v = threadIdx.x;
      for (; v + 3 * kThreads < vecs; v += 4 * kThreads) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = ld_stream_v4(s + v + u * kThreads);
#pragma unroll
        for (int u = 0; u < 4; ++u) d[v + u * kThreads] = x[u];
      }
      for (; v < vecs; v += kThreads) d[v] = ld_stream_v4(s + v);
    };
    move(c.k_codes, code_layer_stride, c.code_page_stride, cv);
    move(c.v_codes, code_layer_stride, c.code_page_stride, cv);
    move(c.k_scales, scale_layer_stride, c.scale_page_stride, sv);
    move(c.v_scales, scale_layer_stride, c.scale_page_stride, sv);
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

// Tokens that one CTA takes at a time, and the grid: enough CTAs to fill the
// GPU once where there are tokens for it, each with about two units a thread.
struct TokenGrid {
  int tile;
  unsigned blocks;
};
TokenGrid token_grid(int64_t tokens, int64_t units_per_token, int num_sms) {
  int64_t tile = 2 * kThreads / units_per_token;
  if (tile < 1) tile = 1;
  int64_t blocks = (tokens + tile - 1) / tile;
  const int64_t cap = static_cast<int64_t>(num_sms) * 32;
  if (blocks > cap) blocks = cap;
  return {static_cast<int>(tile), static_cast<unsigned>(blocks)};
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
  const TokenGrid g = token_grid(tokens, int64_t{2} * c.kv_heads * c.head_dim / 16, num_sms);
  auto launch = [&](auto t) {
    kv_append_kernel<decltype(t)::value><<<g.blocks, kThreads, 0, stream>>>(c, K, V, tokens, g.tile, slots, status);
  };
  if (type == kBf16) launch(std::integral_constant<int, kBf16>{});
  else if (type == kFp16) launch(std::integral_constant<int, kFp16>{});
  else launch(std::integral_constant<int, kFp32>{});
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const nvfp4_kv_cache& c, int64_t tokens, const int64_t* slots, int type,
                           void* K, void* V, int num_sms, cudaStream_t stream) {
  if (tokens == 0) return cudaSuccess;
  const TokenGrid g = token_grid(tokens, int64_t{2} * c.kv_heads * c.head_dim / 8, num_sms);
  auto launch = [&](auto t) {
    kv_read_kernel<decltype(t)::value><<<g.blocks, kThreads, 0, stream>>>(c, tokens, g.tile, slots, K, V);
  };
  if (type == kBf16) launch(std::integral_constant<int, kBf16>{});
  else if (type == kFp16) launch(std::integral_constant<int, kFp16>{});
  else launch(std::integral_constant<int, kFp32>{});
  return cudaGetLastError();
}

cudaError_t launch_kv_copy_pages(const nvfp4_kv_cache& c, int64_t layers,
                                 int64_t code_layer_stride, int64_t scale_layer_stride,
                                 const int* src, const int* dst, int64_t n, int num_sms,
                                 cudaStream_t stream) {
  (void)num_sms;
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
