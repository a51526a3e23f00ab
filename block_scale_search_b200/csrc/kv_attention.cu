// kv_attention.cu -- attention over the paged NVFP4 cache.
//
// For query i of a sequence with Lq new and Lk cached tokens (the new ones
// included) and query head q over KV head h = q / G:
//   x_j = scale * Q . K_j,  j visible: j < Lk, causal: j <= p = Lk - Lq + i,
//                                      window w > 0: j > p - w
//   out = sum_j e^(x_j - m) V_j / sum_j e^(x_j - m),   lse = log sum_j e^x_j
// (no visible j: out = 0, lse = -inf).
//
// kv_rows_kernel: up to 8 NT query rows against one KV head, what decoding and
// drafting ask for.  Bound by HBM (1.125 bytes per cached element, K and V)
// with the 4-bit decode next, so the tensor work is arranged for few
// instructions per cached element:
//   - mma.sync m16n8k16 with the cache as the 16-row operand and the query
//     rows as the 8 columns: S^T = K Q^T and O^T = V^T P^T.  A decoded pair of
//     values goes straight into an operand register; nothing passes through
//     shared memory twice.  Eight shared heads fill the columns exactly.
//     (tcgen05 takes its operands from shared memory, 128 rows at a time: the
//     decoded tile would be written and read again, for 8 useful rows.)
//   - the product's inner index may run in any order.  For S^T lane (g, l)
//     takes the d of its own 16-byte piece of a K row; for O^T lane g owns
//     head_dim / 8 consecutive d, and the k index runs over tokens.
//   - a value is code * scale, exact in FP16 (6 bits); S is applied to the
//     scores and to the result.  Q goes to FP16 after an exact power-of-two
//     scaling per row, P in (0, 2^8] is rounded to FP16 (2^-11 relative, below
//     the rounding of a 16-bit result); sums and the running maximum are FP32.
//   - the running maximum moves only when a score passes it by 2^8 (P stays
//     in FP16 range until then): one vote per tile in place of a reduction.
//
// Work split: the tiles (16 tokens) of all (sequence, row block, KV head)
// items form one line; each CTA takes an equal piece of it, cutting items
// where it must, so ragged batches and single long sequences fill the GPU
// alike.  A CTA's warps take tiles in turn, each with its own ring of bulk
// copies (16 rows of a page are contiguous).  An item inside one CTA is
// finished there; of a cut item each CTA leaves a partial result (at most its
// first and its last item), which kv_join_kernel adds up.
#include <type_traits>

#include "kv_cache.cuh"
#include "nvfp4_device.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;    // tokens
constexpr int kStages = 4;   // tiles in flight per warp
constexpr float kSlack = 8.0f;  // log2 by which a score may pass the running maximum

struct Params {
  KvAttention a;
  int group, page_shift;
  float scale_log2;
  float* partial;  // [CTA][2][R * D] sums, then [CTA][2][R * 2] maximum and sum
  float* partial_ml;
  int ctas;
};

__device__ unsigned int g_stalls;  // waits given up (never, unless a copy is lost)

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity) {
  uint32_t done = 0;
  for (int i = 0; i < (1 << 22); ++i) {
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return;
  }
  atomicAdd(&g_stalls, 1u);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// What the schedule knows of one sequence.
struct Seq {
  int q0, lq, lk;     // first query row, new tokens, cached tokens
  int t0, tiles;      // first tile that a query sees, tiles per item (at least 1)
  int blocks;         // row blocks
};

template <int R>
__device__ __forceinline__ Seq sequence(const Params& p, int b) {
  Seq s;
  const int lo = p.a.q_offsets[b], hi = p.a.q_offsets[b + 1];
  s.q0 = min(max(lo, 0), p.a.total_q);
  s.lq = min(min(max(hi, s.q0), p.a.total_q) - s.q0, p.a.max_q);
  s.lk = min(max(p.a.kv_lengths[b], 0), p.a.max_kv);
  const int first = p.a.window > 0 ? max(0, s.lk - s.lq - p.a.window + 1) : 0;
  s.t0 = first / kTile;
  s.tiles = max(1, (s.lk + kTile - 1) / kTile - s.t0);
  s.blocks = (s.lq * p.group + R - 1) / R;
  return s;
}

template <int R>
__device__ __forceinline__ long long seq_tiles(const Params& p, int b) {
  const Seq s = sequence<R>(p, b);
  return static_cast<long long>(s.blocks) * p.a.c.kv_heads * s.tiles;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum of seq_tiles over b < n, by the whole CTA (every thread gets it).
template <int R>
__device__ __forceinline__ long long tiles_before(const Params& p, int n, long long* red) {
  long long v = 0;
  for (int b = threadIdx.x; b < n; b += kThreads) v += seq_tiles<R>(p, b);
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += red[w];
  return v;
}

// Tiles per CTA: an equal share, but no less than two tiles a warp.
__device__ __forceinline__ long long tiles_per_cta(long long total, int ctas) {
  const long long share = (total + ctas - 1) / ctas;
  return share > 2 * kWarps ? share : 2 * kWarps;
}

// A row r of a block of a sequence: query r / G, head h G + r % G.
__device__ __forceinline__ void visible(const Params& p, const Seq& s, int row, int& lo, int& hi) {
  if (row >= s.lq * p.group) {
    lo = hi = 0;
    return;
  }
  const int pos = s.lk - s.lq + row / p.group;
  hi = p.a.causal ? min(s.lk, pos + 1) : s.lk;
  lo = p.a.window > 0 ? max(0, pos - p.a.window + 1) : 0;
}

__device__ __forceinline__ void write_row(const Params& p, const Seq& s, int h, int row, int d, float4 v,
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
  *reinterpret_cast<uint2*>(o) = w;
}

__device__ __forceinline__ void write_lse(const Params& p, const Seq& s, int h, int row, float m, float l) {
  if (p.a.lse == nullptr) return;
  const int64_t t = s.q0 + row / p.group;
  p.a.lse[t * p.a.q_heads + h * p.group + row % p.group] =
      l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : (NT == 2 ? 3 : 2))
kv_rows_kernel(const __grid_constant__ Params p) {
  constexpr int R = 8 * NT;
  constexpr int KW = D / 32;            // K words (8 values) per lane and row
  constexpr int VW = D / 64;            // V words per lane and token
  constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16;
  constexpr int kStageBytes = 2 * (kCodes + kScales);
  extern __shared__ __align__(128) uint8_t smem[];
  // [warp][stage] tiles, then the join area [warp][R][D] and its maxima and
  // sums [warp][R][2], then the barriers
  float* const join_o = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes);
  float* const join_ml = join_o + kWarps * R * D;
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ long long red[kWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, l4 = lane & 3;
  const nvfp4_kv_cache& c = p.a.c;
  uint8_t* const ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_u = smem_u32(ring), bar_u = smem_u32(&bars[warp][0]);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(bar_u + 8 * s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  // this CTA's piece of the line of tiles
  const long long total = tiles_before<R>(p, p.a.batch, red);
  const long long per = tiles_per_cta(total, p.ctas);
  long long cur = per * blockIdx.x;
  const long long end = min(total, cur + per);
  if (cur >= end) return;
  // the sequence that holds tile `cur`
  int b = 0;
  long long base = 0;
  {
    // every warp scans 32 sequences at a time
    for (;; b += 32) {
      if (b >= p.a.batch) return;
      const int bb = b + lane;
      const long long n = bb < p.a.batch ? seq_tiles<R>(p, bb) : 0;
      long long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += up;
      }
      const unsigned past = __ballot_sync(0xFFFFFFFFu, base + inc > cur);
      if (past) {
        const int f = __ffs(past) - 1;
        base += __shfl_sync(0xFFFFFFFFu, inc - n, f);
        b += f;
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
  }

  uint32_t fill = 0, use = 0;  // tiles this warp has requested and consumed, over all items
  while (cur < end) {
    const Seq s = sequence<R>(p, b);
    const long long in_seq = cur - base;
    const int item = static_cast<int>(in_seq / s.tiles);
    const int ts = static_cast<int>(in_seq - static_cast<long long>(item) * s.tiles);
    const int h = item % c.kv_heads, r0 = item / c.kv_heads * R;
    const int te = static_cast<int>(min(static_cast<long long>(s.tiles), ts + (end - cur)));
    const int mine = te - ts > warp ? (te - ts - warp + kWarps - 1) / kWarps : 0;

    // ---- bulk copies of this warp's k-th tile of the item
    const int64_t head_codes = static_cast<int64_t>(h) * c.page_size * (D / 2);
    const int64_t head_scales = static_cast<int64_t>(h) * c.page_size * (D / 16);
    const int* const row_table = p.a.table + b * p.a.table_stride;
    auto page_at = [&](int k) {  // page id of tile k, or -1
      const int tok = (s.t0 + ts + warp + k * kWarps) * kTile;
      if (k >= mine || tok >= s.lk) return -1;
      const int id = row_table[tok >> p.page_shift];
      return id >= 0 && id < c.num_pages ? id : -1;
    };
    int ids = page_at(lane), ids_base = 0;  // lane i: page of tile ids_base + i
    uint32_t live_mask = 0;                 // bit (tile % 32): the tile's page exists
    int requested = 0;
    auto request = [&]() {
      if (requested >= mine) return;
      if (requested == ids_base + 32) {
        ids_base += 32;
        ids = page_at(ids_base + lane);
      }
      const int id = __shfl_sync(0xFFFFFFFFu, ids, requested - ids_base);
      const uint32_t st = fill % kStages;
      const uint32_t bit = 1u << (requested & 31);
      if (id >= 0) {
        live_mask |= bit;
        if (lane == 0) mbar_expect(bar_u + 8 * st, kStageBytes);
        __syncwarp();
        if (lane < 4) {
          const int row = ((s.t0 + ts + warp + requested * kWarps) * kTile) & (c.page_size - 1);
          const bool isv = lane & 2;
          const uint8_t* src;
          uint32_t dst = ring_u + st * kStageBytes + (isv ? kCodes + kScales : 0);
          uint32_t bytes;
          if (lane & 1) {
            src = (isv ? c.v_scales : c.k_scales) + id * c.scale_page_stride + head_scales + row * (D / 16);
            dst += kCodes;
            bytes = kScales;
          } else {
            src = (isv ? c.v_codes : c.k_codes) + id * c.code_page_stride + head_codes + row * (D / 2);
            bytes = kCodes;
          }
          bulk_load(dst, src, bytes, bar_u + 8 * st);
        }
      } else {
        live_mask &= ~bit;
        if (lane == 0)  // nothing to copy: complete the phase
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar_u + 8 * st) : "memory");
      }
      ++requested;
      ++fill;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) request();

    // ---- query rows: lane (g, l4) holds d [l4 D/4, (l4+1) D/4) of row g of
    // every 8-row tile, in FP16 after scaling the row's maximum to [1, 2)
    uint32_t q[NT][KW * 4];
    float f[NT][2];              // factor of the scores of columns 2 l4, 2 l4 + 1
    int vlo[NT][2], vhi[NT][2];  // visible tokens of those columns
    int all_lo = 0, all_hi = 0x7FFFFFFF;  // tokens that every row sees
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = r0 + 8 * n + g;
      const bool have = row < s.lq * p.group;
      float y[KW * 8];
      float mx = 0.0f;
      if (have) {
        const uint16_t* src = static_cast<const uint16_t*>(p.a.Q) +
                              (s.q0 + row / p.group) * p.a.q_token_stride +
                              (h * p.group + row % p.group) * p.a.q_head_stride + l4 * (D / 4);
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[8 * i + 2 * j] = to_f32(w[j] & 0xFFFFu, p.a.type);
            y[8 * i + 2 * j + 1] = to_f32(w[j] >> 16, p.a.type);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < KW * 8; ++i) y[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < KW * 8; ++i) mx = fmaxf(mx, fabsf(y[i]));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      // power of two at or below the maximum, kept where its reciprocal is a
      // normal number; Inf and NaN stay what they are in FP16
      const uint32_t e = min(max(__float_as_uint(mx) >> 23, 1u), 253u);
      const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
      for (int i = 0; i < KW * 4; ++i) q[n][i] = pack_f16x2(y[2 * i] * down, y[2 * i + 1] * down);
      const float fs = up * p.scale_log2 * c.k_S[h];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f[n][k] = __shfl_sync(0xFFFFFFFFu, fs, (2 * l4 + k) * 4);
        visible(p, s, r0 + 8 * n + 2 * l4 + k, vlo[n][k], vhi[n][k]);
        if (r0 + 8 * n + 2 * l4 + k < s.lq * p.group) {
          all_lo = max(all_lo, vlo[n][k]);
          all_hi = min(all_hi, vhi[n][k]);
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      all_lo = max(all_lo, __shfl_xor_sync(0xFFFFFFFFu, all_lo, o));
      all_hi = min(all_hi, __shfl_xor_sync(0xFFFFFFFFu, all_hi, o));
    }

    float o[NT][VW * 4][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.0f;

    // S^T row r holds token r ^ (r >> 1 & 1): neighbouring rows and the
    // tokens of one V load then differ in parity, which halves the bank
    // conflicts of 64-byte rows
    auto tok = [](int r) { return r ^ ((r >> 1) & 1); };

    for (int k = 0; k < mine; ++k) {
      request();
      const uint32_t st = use % kStages;
      mbar_wait(bar_u + 8 * st, (use / kStages) & 1);
      ++use;
      const uint8_t* const kc = ring + st * kStageBytes;
      const uint8_t* const ks = kc + kCodes;
      const uint8_t* const vc = ks + kScales;
      const uint8_t* const vs = vc + kCodes;
      const int tb = (s.t0 + ts + warp + k * kWarps) * kTile;  // first token
      const bool live = (live_mask >> (k & 31)) & 1;
      if (live) {
        // ---- S^T
        float x[NT][4] = {};
        uint32_t kw[2][KW];
        uint32_t ksc[2];  // two scales (D = 64: one, twice)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = tok(g) + 8 * j;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(kc + t * 64 + l4 * 16);
            kw[j][0] = v.x, kw[j][1] = v.y, kw[j][2] = v.z, kw[j][3] = v.w;
            ksc[j] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + t * 8 + l4 * 2));
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(kc + t * 32 + l4 * 8);
            kw[j][0] = v.x, kw[j][1] = v.y;
            ksc[j] = e4m3x2_to_f16x2(ks[t * 4 + l4]);
          }
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          // block of word w: two words a block
          const uint32_t sel = w < 2 ? 0x1010 : 0x3232;
          const uint32_t s0 = __byte_perm(ksc[0], 0, sel), s1 = __byte_perm(ksc[1], 0, sel);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t a[4];
            a[0] = mul_f16x2(e2m1x2_to_f16x2((kw[0][w] >> (16 * j)) & 0xFFu), s0);
            a[1] = mul_f16x2(e2m1x2_to_f16x2((kw[1][w] >> (16 * j)) & 0xFFu), s1);
            a[2] = mul_f16x2(e2m1x2_to_f16x2((kw[0][w] >> (16 * j + 8)) & 0xFFu), s0);
            a[3] = mul_f16x2(e2m1x2_to_f16x2((kw[1][w] >> (16 * j + 8)) & 0xFFu), s1);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(x[n], a, q[n][4 * w + 2 * j], q[n][4 * w + 2 * j + 1]);
          }
        }
        const bool edge = tb < all_lo || tb + kTile > all_hi;
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y = x[n][i] * f[n][i & 1];
            if (edge) {
              const int t = tb + tok(g) + (i & 2) * 4;
              if (t < vlo[n][i & 1] || t >= vhi[n][i & 1]) y = -INFINITY;
            }
            x[n][i] = y;
            over |= y > m[n][i & 1] + kSlack;
          }
        }
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float t = fmaxf(x[n][i], x[n][i + 2]);
              t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
              t = fmaxf(t, m[n][i]);
              const float r = t == m[n][i] ? 1.0f : exp2_approx(m[n][i] - t);
              m[n][i] = t;
              l[n][i] *= r;
#pragma unroll
              for (int u = 0; u < VW * 4; ++u) o[n][u][i] *= r, o[n][u][i + 2] *= r;
            }
          }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float mm = m[n][i & 1];
            x[n][i] = exp2_approx(x[n][i] - (mm == -INFINITY ? 0.0f : mm));
            l[n][i & 1] += x[n][i];
          }
          pb[n][0] = transpose8x8(pack_f16x2(x[n][0], x[n][1]));
          pb[n][1] = transpose8x8(pack_f16x2(x[n][2], x[n][3]));
        }
        // ---- O^T: tokens of the k index 2 l4, 2 l4 + 1, 2 l4 + 8, 2 l4 + 9
        const int ta = tok(2 * l4), tc = tok(2 * l4 + 1);
        uint32_t vw[4][VW], vsc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = (j & 1 ? tc : ta) + (j & 2) * 4;
          if constexpr (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(vc + t * 64 + g * 8);
            vw[j][0] = v.x, vw[j][1] = v.y;
            vsc[j] = vs[t * 8 + g];
          } else {
            vw[j][0] = *reinterpret_cast<const uint32_t*>(vc + t * 32 + g * 4);
            vsc[j] = vs[t * 4 + (g >> 1)];
          }
        }
        uint32_t nan_tokens = 0;  // bit j: vsc[j] is NaN and its token is hidden from some row
        if (edge) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = tb + (j & 1 ? tc : ta) + (j & 2) * 4;
            if ((vsc[j] & 0x7Fu) == 0x7Fu) {
              // 0 * NaN would reach rows that do not see the token: take it
              // out of the product and give it to the rows that do (below)
              if (t < s.lk) nan_tokens |= 1u << j;
              vsc[j] = 0;
            }
          }
        }
        const uint32_t sab = e4m3x2_to_f16x2(vsc[0] | (vsc[1] << 8));
        const uint32_t scd = e4m3x2_to_f16x2(vsc[2] | (vsc[3] << 8));
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          constexpr uint32_t kLow = 0x0F0F0F0Fu;
          const uint32_t lo_ab = (vw[0][w] & kLow) | ((vw[1][w] << 4) & ~kLow);
          const uint32_t hi_ab = ((vw[0][w] >> 4) & kLow) | (vw[1][w] & ~kLow);
          const uint32_t lo_cd = (vw[2][w] & kLow) | ((vw[3][w] << 4) & ~kLow);
          const uint32_t hi_cd = ((vw[2][w] >> 4) & kLow) | (vw[3][w] & ~kLow);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t a[4];
            a[0] = mul_f16x2(e2m1x2_to_f16x2((lo_ab >> (8 * u)) & 0xFFu), sab);
            a[1] = mul_f16x2(e2m1x2_to_f16x2((hi_ab >> (8 * u)) & 0xFFu), sab);
            a[2] = mul_f16x2(e2m1x2_to_f16x2((lo_cd >> (8 * u)) & 0xFFu), scd);
            a[3] = mul_f16x2(e2m1x2_to_f16x2((hi_cd >> (8 * u)) & 0xFFu), scd);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(o[n][4 * w + u], a, pb[n][0], pb[n][1]);
          }
        }
        if (edge && __any_sync(0xFFFFFFFFu, nan_tokens != 0)) {
          // the NaN tokens of lane g's own elements, gathered over l4
#pragma unroll
          for (int src = 0; src < 4; ++src) {
            const uint32_t bits = __shfl_sync(0xFFFFFFFFu, nan_tokens, (lane & ~3) | src);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (!((bits >> j) & 1)) continue;
              const int t = tb + tok(2 * src + (j & 1)) + (j & 2) * 4;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (t >= vlo[n][i] && t < vhi[n][i]) {
#pragma unroll
                    for (int u = 0; u < VW * 4; ++u)
                      o[n][u][i] = o[n][u][i + 2] = __uint_as_float(0x7FC00000u);
                  }
            }
          }
        }
      }
      __syncwarp();  // the stage may be written again
    }

    // ---- join the warps
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t = l[n][i];
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 4);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 8);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 16);
        const int col = 8 * n + 2 * l4 + i;
        if (g == 0) {
          join_ml[(warp * R + col) * 2] = m[n][i];
          join_ml[(warp * R + col) * 2 + 1] = t;
        }
        float* dst = join_o + (warp * R + col) * D + g * (D / 8);
#pragma unroll
        for (int u = 0; u < VW * 4; u += 2)
          *reinterpret_cast<float4*>(dst + 2 * u) =
              make_float4(o[n][u][i], o[n][u][i + 2], o[n][u + 1][i], o[n][u + 1][i + 2]);
      }
    }
    __syncthreads();
    const bool whole = ts == 0 && te == s.tiles;
    const int slot = ts == 0 ? 1 : 0;  // of a cut item: 0 where an earlier CTA has its start
    const float vS = c.v_S[h];
    const int rows = min(R, s.lq * p.group - r0);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, join_ml[(w * R + row) * 2]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = join_ml[(w * R + row) * 2];
        const float z = mw == mm ? 1.0f : exp2_approx(mw - mm);
        const float4 v = *reinterpret_cast<const float4*>(join_o + (w * R + row) * D + d);
        ll += z * join_ml[(w * R + row) * 2 + 1];
        acc.x += z * v.x, acc.y += z * v.y, acc.z += z * v.z, acc.w += z * v.w;
      }
      if (whole) {
        write_row(p, s, h, r0 + row, d, acc, ll == 0.0f ? 0.0f : vS / ll);
        if (d == 0) write_lse(p, s, h, r0 + row, mm, ll);
      } else {
        const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * R + row;
        *reinterpret_cast<float4*>(p.partial + at * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(p.partial_ml + at * 2) = make_float2(mm, ll);
      }
    }
    __syncthreads();

    // ---- next item
    cur += te - ts;
    if (cur < end) {
      long long n = seq_tiles<R>(p, b);
      while (cur >= base + n) {  // also steps over sequences without new tokens
        base += n;
        if (++b >= p.a.batch) return;
        n = seq_tiles<R>(p, b);
      }
    }
  }
}

// One CTA per row of an item: adds up the partial results of an item that was
// cut, in the order of its CTAs.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(const __grid_constant__ Params p, int blocks) {
  constexpr int R = 8 * NT;
  __shared__ long long red[kWarps];
  const int b = blockIdx.y;
  const Seq s = sequence<R>(p, b);
  const int row = blockIdx.x % R, item = blockIdx.x / R;
  const int h = item % p.a.c.kv_heads, rb = item / p.a.c.kv_heads;
  if (rb >= s.blocks || rb * R + row >= s.lq * p.group) return;
  const long long base = tiles_before<R>(p, b, red);
  const long long total = tiles_before<R>(p, p.a.batch, red);
  const long long per = tiles_per_cta(total, p.ctas);
  const long long first = base + static_cast<long long>(item) * s.tiles, last = first + s.tiles - 1;
  const long long c0 = first / per, c1 = last / per;
  if (c0 == c1) return;
  auto at = [&](long long cta) {
    const int slot = cta * per <= first ? 1 : 0;
    return (cta * 2 + slot) * R + row;
  };
  // maximum and sum over the pieces
  __shared__ float sm[kWarps], sl[kWarps];
  float m = -INFINITY;
  for (long long cta = c0 + threadIdx.x; cta <= c1; cta += kThreads) m = fmaxf(m, p.partial_ml[at(cta) * 2]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
  __syncthreads();
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float l = 0.0f;
  for (long long cta = c0 + threadIdx.x; cta <= c1; cta += kThreads) {
    const float2 ml = *reinterpret_cast<const float2*>(p.partial_ml + at(cta) * 2);
    l += ml.y * (ml.x == m ? 1.0f : exp2_approx(ml.x - m));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  if ((threadIdx.x & 31) == 0) sl[threadIdx.x >> 5] = l;
  __syncthreads();
  l = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  // lane i of warp w: 4 elements of every kWarps-th piece
  __shared__ float4 acc_s[kWarps][D / 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < D / 4) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long cta = c0 + warp; cta <= c1; cta += kWarps) {
      const float mw = p.partial_ml[at(cta) * 2];
      const float z = mw == m ? 1.0f : exp2_approx(mw - m);
      const float4 v = *reinterpret_cast<const float4*>(p.partial + at(cta) * D + 4 * lane);
      acc.x += z * v.x, acc.y += z * v.y, acc.z += z * v.z, acc.w += z * v.w;
    }
    acc_s[warp][lane] = acc;
  }
  __syncthreads();
  if (threadIdx.x < D / 4) {
    float4 acc = acc_s[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = acc_s[w][threadIdx.x];
      acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
    write_row(p, s, h, rb * R + row, 4 * threadIdx.x, acc, l == 0.0f ? 0.0f : p.a.c.v_S[h] / l);
    if (threadIdx.x == 0) write_lse(p, s, h, rb * R + row, m, l);
  }
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Rows per item: the fewest 8-row tiles that hold all rows of a sequence.
int row_tiles(int64_t max_q, int q_heads, int kv_heads) {
  const int64_t rows = max_q * (q_heads / kv_heads);
  return rows <= 8 ? 1 : (rows <= 16 ? 2 : 4);
}

int ctas_per_sm(int nt) { return nt == 1 ? 4 : (nt == 2 ? 3 : 2); }

int row_ctas(int64_t batch, int64_t max_q, int64_t max_kv, int q_heads, int kv_heads, int nt, int num_sms) {
  const int64_t blocks = (max_q * (q_heads / kv_heads) + 8 * nt - 1) / (8 * nt);
  const double tiles = static_cast<double>(batch) * blocks * kv_heads *
                       static_cast<double>((max_kv + kTile - 1) / kTile + 1);
  const int64_t wave = static_cast<int64_t>(num_sms) * ctas_per_sm(nt);
  const double want = tiles / (2 * kWarps) + 1.0;
  return static_cast<int>(want < static_cast<double>(wave) ? static_cast<int64_t>(want) : wave);
}

template <int D, int NT>
cudaError_t run_rows(Params& p, cudaStream_t stream) {
  constexpr int R = 8 * NT;
  constexpr int kStageBytes = 2 * kTile * (D / 2 + D / 16);
  constexpr int smem = kWarps * (kStages * kStageBytes + R * (D + 2) * 4);
  const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&kv_rows_kernel<D, NT>),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  p.partial_ml = p.partial + static_cast<int64_t>(p.ctas) * 2 * R * D;
  kv_rows_kernel<D, NT><<<p.ctas, kThreads, smem, stream>>>(p);
  cudaError_t r = cudaGetLastError();
  if (r != cudaSuccess) return r;
  const int blocks = (p.a.max_q * p.group + R - 1) / R;
  const dim3 grid(static_cast<unsigned>(blocks) * p.a.c.kv_heads * R, static_cast<unsigned>(p.a.batch));
  kv_join_kernel<D, NT><<<grid, kThreads, 0, stream>>>(p, blocks);
  return cudaGetLastError();
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t batch, int64_t max_q, int64_t max_kv, int q_heads,
                                    int kv_heads, int head_dim, int num_sms) {
  const int nt = row_tiles(max_q, q_heads, kv_heads);
  const int ctas = row_ctas(batch, max_q, max_kv, q_heads, kv_heads, nt, num_sms);
  return static_cast<size_t>(ctas) * 2 * 8 * nt * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention(const KvAttention& a, void* workspace, int num_sms, cudaStream_t stream) {
  if (a.batch == 0 || a.total_q == 0) return cudaSuccess;
  Params p{};
  p.a = a;
  p.group = a.q_heads / a.c.kv_heads;
  p.page_shift = log2_of(a.c.page_size);
  p.scale_log2 = a.scale * 1.44269504088896341f;
  p.partial = static_cast<float*>(workspace);
  const int nt = row_tiles(a.max_q, a.q_heads, a.c.kv_heads);
  p.ctas = row_ctas(a.batch, a.max_q, a.max_kv, a.q_heads, a.c.kv_heads, nt, num_sms);
  if (a.c.head_dim == 128) {
    if (nt == 1) return run_rows<128, 1>(p, stream);
    if (nt == 2) return run_rows<128, 2>(p, stream);
    return run_rows<128, 4>(p, stream);
  }
  if (nt == 1) return run_rows<64, 1>(p, stream);
  if (nt == 2) return run_rows<64, 2>(p, stream);
  return run_rows<64, 4>(p, stream);
}

unsigned int kv_stalls(bool reset, cudaError_t* e) {
  unsigned int n = 0;
  *e = cudaMemcpyFromSymbol(&n, g_stalls, sizeof(n));
  if (*e == cudaSuccess && reset) {
    const unsigned int z = 0;
    *e = cudaMemcpyToSymbol(g_stalls, &z, sizeof(z));
  }
  return n;
}

}  // namespace nvfp4
