// kv_attention.cu -- attention over the paged NVFP4 cache.
//
// For query i of a sequence with Lq new and Lk cached tokens (the new ones
// included) and query head q over KV head h = q / G:
//   x_j = scale * Q . K_j,  j visible: j < Lk, causal: j <= p = Lk - Lq + i,
//                                      window w > 0: j > p - w
//   out = sum_j e^(x_j - m) V_j / sum_j e^(x_j - m),   lse = log sum_j e^x_j
// (no visible j: out = 0, lse = -inf).
//
// kv_rows_kernel: few query rows against one KV head, what decoding and
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
//     scores and to the result.  Q goes to FP16 after a power-of-two scaling
//     per row (exact but for what lies 2^32 below a row's largest), and so does
//     P, scaled so that the largest is 2^7 to 2^15 (2^-11 relative, below the
//     rounding of a 16-bit result); sums and the running maximum are FP32.
//   - the running maximum moves only when a score passes it by 2^8 (P stays
//     in FP16 range until then): one vote per tile in place of a reduction.
// A tile of 32 tokens takes 640 instructions at head_dim 128 with 8 rows, 140
// of them conversions, 128 products with scales and 32 MMAs (2, 2 and 8.5
// cycles of a scheduler each), against 745 cycles of a scheduler's share of
// HBM; in the loop it takes about 870, that is 5.9 TB/s, also where the cache
// lies in L2: what bounds it is instructions.  Over a whole call 4.3 TB/s (48
// sequences of up to 8192 tokens, 64 / 8 heads of 128: 57.0 us) and 4.8 TB/s
// (two of 131072: 63.2 us) remain: a CTA takes about 6 us until its first tile
// is there (lengths, page ids and tiles are three trips to memory one after
// another) and 2 us to join its warps, the cut items 3 to 5 us.
//
// Work split: the tiles (32 tokens) of all (sequence, row block, KV head)
// items form one line; each CTA takes an equal piece of it, cutting items
// where it must, so ragged batches and single long sequences fill the GPU
// alike.  A CTA's warps take tiles in turn, each with its own ring of
// asynchronous copies (16 rows of a page are contiguous).  An item inside one
// CTA is finished there; of a cut item each CTA leaves a partial result (at
// most its first and its last item), which kv_join_kernel adds up.
#include <type_traits>

#include "kv_attention.cuh"

namespace nvfp4 {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32;    // tokens a warp takes at a time, in two halves of 16
constexpr int kHalf = kTile / 2;
constexpr int kStages = 2;   // tiles of a warp's ring (and the code below counts on 2)
// What starting and finishing an item costs a CTA, in tiles: its page ids and
// queries arrive in two trips to memory, its warps meet twice at the end.
constexpr int kItemCost = 10;
// Query rows of a sequence and KV head up to which this kernel serves it, in
// blocks of 32; kv_prompt_kernel takes those with more.  Measured on 64 / 8
// heads, 1 to 64 sequences of 500 to 32000 tokens: 32 rows take 12 to 157 us
// here and 19 to 261 us there at head_dim 128, 64 rows (two blocks, the cache
// decoded twice) 13 to 294 and 19 to 264; at head_dim 64, where a step of the
// other kernel costs nearly as much, 64 rows take 10 to 178 and 17 to 223.
constexpr int64_t rows_limit(int head_dim) { return head_dim == 64 ? 64 : 32; }

// Resident CTAs the kernel is built for (its registers and shared memory).  More
// warps are worth a few spilled registers: 16 rows at head_dim 128 take 102 us
// with 4 CTAs and 180 bytes of spills, 105 with 3 and none (64 sequences of up
// to 8000 tokens); with 5 and 550 bytes 153.
__host__ __device__ constexpr int ctas_per_sm(int D, int nt) {
  return nt == 1 ? 5 : (nt == 2 ? 4 : (D == 64 ? 3 : 2));
}

// Shared memory: the rings [warp][stage] and the queries' operands [8-row
// tile][word][lane] of 16 bytes; once an item's tiles are used up, the join
// area, sums [warp][R][D] and maxima and sums [warp][R][2], lies over both.
__host__ __device__ constexpr int ring_bytes(int D) { return kWarps * kStages * 2 * kTile * (D / 2 + D / 16); }
__host__ __device__ constexpr int rows_smem(int D, int NT) {
  const int use = ring_bytes(D) + NT * (D / 32) * 512, join = kWarps * 8 * NT * (D + 2) * 4;
  return use > join ? use : join;
}

// 16 bytes to shared memory, or 16 zeros where `bytes` is 0.
template <int kDst, int kSrc>
__device__ __forceinline__ void copy16(uint32_t dst, uint64_t src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(kDst),
               "n"(kSrc)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// a where `mask` is 1 and b where it is 0, in one instruction (the compiler
// rewrites the C expression with shifts into two)
__device__ __forceinline__ uint32_t merge(uint32_t a, uint32_t b, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(a), "r"(b), "r"(mask));
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
// What the schedule knows of one sequence.
struct Seq : Span {
  int t0, tiles;      // first tile that a query sees, tiles per item (at least 1)
  int span;           // units of an item on the line of work: kItemCost, then its tiles
  int blocks;         // row blocks (0: no rows, or the other kernel's)
};

template <int R>
__device__ __forceinline__ Seq sequence(const Params& p, int b) {
  Seq s;
  static_cast<Span&>(s) = span_of(p, b);
  const int first = p.a.window > 0 ? max(0, s.lk - s.lq - p.a.window + 1) : 0;
  s.t0 = first / kTile;
  s.tiles = max(1, (s.lk + kTile - 1) / kTile - s.t0);
  s.span = s.tiles + kItemCost;
  const int rows = s.lq * p.group;
  s.blocks = rows > p.rows_limit ? 0 : (rows + R - 1) / R;
  return s;
}

// (The host refuses calls whose bounds allow 2^31 units: a 64-bit division here
// is a call, for which the whole kernel would save registers to memory.)
template <int R>
__device__ __forceinline__ int seq_units(const Params& p, int b) {
  const Seq s = sequence<R>(p, b);
  return s.blocks * p.a.c.kv_heads * s.span;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// Sum of seq_units over all sequences, by the whole CTA (every thread gets it).
template <int R>
__device__ __forceinline__ int all_units(const Params& p, int* red) {
  int v = 0;
  for (int b = threadIdx.x; b < p.a.batch; b += kThreads) v += seq_units<R>(p, b);
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += red[w];
  return v;
}

// Sums of seq_units over the sequences before n (x) and over all (y), by a CTA
// of kW warps (every thread gets them).  red: 2 kW.
template <int R, int kW>
__device__ __forceinline__ int2 units_before(const Params& p, int n, int* red) {
  int x = 0, y = 0;
  for (int b = threadIdx.x; b < p.a.batch; b += 32 * kW) {
    const int u = seq_units<R>(p, b);
    y += u;
    if (b < n) x += u;
  }
  x = warp_sum(x);
  y = warp_sum(y);
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = x;
    red[kW + (threadIdx.x >> 5)] = y;
  }
  __syncthreads();
  int2 r = {0, 0};
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    r.x += red[w];
    r.y += red[kW + w];
  }
  return r;
}

// Units per CTA: an equal share, but no less than a tile a warp.
__device__ __forceinline__ int units_per_cta(int total, int ctas) { return max((total + ctas - 1) / ctas, kWarps); }

// Where a CTA lists its cut item, and a row's partial sums from element d on,
// and maximum and sum (R rows an item, two items a CTA).
__device__ __forceinline__ int4* cut_at(const Params& p, unsigned int cta) {
  return checked(p.cut + cta, p.cut, static_cast<int64_t>(p.ctas) * 16, kSiteKvCut);
}
template <int D, int R>
__device__ __forceinline__ float4* partial_at(const Params& p, int64_t row, int d) {
  return checked(reinterpret_cast<float4*>(p.partial + row * D + d), p.partial, static_cast<int64_t>(p.ctas) * 2 * R * D * 4,
                 kSiteKvPartial);
}
template <int R>
__device__ __forceinline__ float2* partial_ml_at(const Params& p, int64_t row) {
  return checked(reinterpret_cast<float2*>(p.partial_ml + row * 2), p.partial_ml, static_cast<int64_t>(p.ctas) * 2 * R * 8,
                 kSiteKvPartial);
}

// Of a query row of the item: factor of its scores (base 2), visible tokens.
struct RowInfo {
  float f;
  int lo, hi;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT))
kv_rows_kernel(const __grid_constant__ Params p) {
  constexpr int R = 8 * NT;
  constexpr int KW = D / 32;            // K words (8 values) per lane and row
  constexpr int VW = D / 64;            // V words per lane and token
  constexpr int kCodes = kHalf * D / 2, kScales = kHalf * D / 16;  // of one half, K or V
  constexpr int kHalfBytes = 2 * (kCodes + kScales);
  constexpr int kStageBytes = 2 * kHalfBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  float* const join_o = reinterpret_cast<float*>(smem);
  float* const join_ml = join_o + kWarps * R * D;
  __shared__ int red[kWarps];
  __shared__ RowInfo row_info[R];

  // warp: from lane 0, so that the compiler takes it, and branches on it, as
  // uniform.  lane: by a shuffle, or it would be read anew, with all that
  // follows from it, in every tile (11 instructions).
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int lane = __shfl_sync(0xFFFFFFFFu, threadIdx.x & 31, threadIdx.x & 31);
  const int g = lane >> 2, l4 = lane & 3;
  const nvfp4_kv_cache& c = p.a.c;
  uint8_t* const ring = smem + warp * kStages * kStageBytes;
  constexpr int kRing = ring_bytes(D);
  uint4* const q_all = reinterpret_cast<uint4*>(smem + kRing);
  const uint4* const q = q_all + lane;
  const uint32_t ring_u = smem_u32(ring);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // kv_join_kernel may be set up meanwhile

  // this CTA's piece of the line of work, and the sequence that holds its start
  __shared__ int start_b;
  __shared__ int start_base;
  int b = 0;
  int base = 0, cur, end;  // base: first unit of sequence b
  __shared__ int share;  // units per CTA, for the list of cut items
  if (p.cut != nullptr && threadIdx.x == 0) *cut_at(p, blockIdx.x) = make_int4(0, 0, 0, 0);
  if (p.a.batch <= kThreads) {   // a sequence a thread: one look at the lengths
    const int n = threadIdx.x < p.a.batch ? seq_units<R>(p, threadIdx.x) : 0;
    int inc = warp_scan(n, lane);
    if (lane == 31) red[warp] = inc;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) inc += red[w];
      total += red[w];
    }
    const int per = units_per_cta(total, p.ctas);
    cur = per * blockIdx.x;
    end = min(total, cur + per);
    if (threadIdx.x == 0) share = per;
    if (inc - n <= cur && cur < inc) {
      start_b = threadIdx.x;
      start_base = inc - n;
    }
    __syncthreads();
    if (cur >= end) return;
    b = start_b;
    base = start_base;
  } else {
    const int total = all_units<R>(p, red);
    const int per = units_per_cta(total, p.ctas);
    cur = per * blockIdx.x;
    end = min(total, cur + per);
    if (threadIdx.x == 0) share = per;  // (only that thread reads it)
    if (cur >= end) return;
    for (;; b += 32) {  // every warp scans 32 sequences at a time
      if (b >= p.a.batch) return;
      const int bb = b + lane;
      const int n = bb < p.a.batch ? seq_units<R>(p, bb) : 0;
      const int inc = warp_scan(n, lane);
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

  while (cur < end) {
    const Seq s = sequence<R>(p, b);
    const int in_seq = cur - base;
    const int item = in_seq / s.span, us = in_seq - item * s.span, ue = min(s.span, us + (end - cur));
    const int ts = max(0, us - kItemCost), te = max(0, ue - kItemCost);  // this CTA's tiles of the item
    const int h = item % c.kv_heads, r0 = item / c.kv_heads * R;
    auto next_item = [&]() {  // false at the end of the batch
      cur += ue - us;
      if (cur >= end) return true;
      int n = seq_units<R>(p, b);
      while (cur >= base + n) {  // also steps over sequences without new tokens
        base += n;
        if (++b >= p.a.batch) return false;
        n = seq_units<R>(p, b);
      }
      return true;
    };
    if (ts >= te) {  // the piece ends before the item's first tile
      if (!next_item()) return;
      continue;
    }
    const int mine = te - ts > warp ? (te - ts - warp + kWarps - 1) / kWarps : 0;

    // ---- copies of this warp's k-th tile of the item
    const int64_t head_codes = static_cast<int64_t>(h) * c.page_size * (D / 2);
    const int64_t head_scales = static_cast<int64_t>(h) * c.page_size * (D / 16);
    const int* const row_table = p.a.table + b * p.a.table_stride;
    auto page_at = [&](int k, int half) {  // the table's entry for half a tile, or -1
      const int tok = (s.t0 + ts + warp + k * kWarps) * kTile + half * kHalf;
      if (k >= mine || tok >= s.lk) return -1;
      return table_entry(p, row_table, tok >> p.page_shift);  // (looked at when it is used: a look waits for the load)
    };
    // Lane i + 16 h keeps half h of tile i of the 16 that are next: its page, and
    // from its first use on where its rows lie from a head's in page 0 on
    // (worked out by a lane a half and not by all lanes for each tile: 13
    // instructions a tile less).
    int id = page_at(lane & 15, lane >> 4);
    uint64_t code_off = 0, scale_off = 0;
    uint32_t bad = 0;        // bit i + 16 h: no page there (zeros are written)
    uint32_t none_next = 0;  // of the tile requested last: bit h, no page
    int requested = 0;
    // The queries' loads go out before the tiles': behind them they would wait
    // for the whole GPU's first requests to be served.  A thread takes 8
    // elements (piece `qp` of a row) of NT rows.
    constexpr int kRowPieces = D / 8, kPass = kThreads / kRowPieces;  // rows of a pass
    const int qp = threadIdx.x % kRowPieces, qr = threadIdx.x / kRowPieces;
    constexpr int kPasses = (R + kPass - 1) / kPass;
    uint4 qv[kPasses];
#pragma unroll
    for (int n = 0; n < kPasses; ++n) {
      const int row = r0 + qr + n * kPass;
      qv[n] = make_uint4(0u, 0u, 0u, 0u);
      if (qr + n * kPass < R && row < s.lq * p.group) {
        const int qi = row / p.group, gi = row - qi * p.group;
        qv[n] = query_piece(p, static_cast<const uint16_t*>(p.a.Q) + (s.q0 + qi) * p.a.q_token_stride +
                                   (h * p.group + gi) * p.a.q_head_stride + 8 * qp);
      }
    }
    const float kS = head_S(p, c.k_S, h);

    // scale bytes: lanes 8 i .. 8 i + 7 (D = 64: 4 i .. 4 i + 3) copy those of
    // K (i < 2) or V of half i % 2
    constexpr int kScaleLanes = kScales / 16;
    const int sc_part = lane / kScaleLanes;
    const uint64_t sc_src = reinterpret_cast<uint64_t>((sc_part & 2 ? c.v_scales : c.k_scales) + head_scales) +
                            lane % kScaleLanes * 16;
    const uint32_t sc_dst = ring_u + (sc_part & 1) * kHalfBytes + (sc_part & 2 ? kCodes + kScales : 0) + kCodes +
                            lane % kScaleLanes * 16;
    const uint64_t k_src = reinterpret_cast<uint64_t>(c.k_codes + head_codes) + lane * 16;
    const uint64_t v_src = reinterpret_cast<uint64_t>(c.v_codes + head_codes) + lane * 16;
    const uint32_t code_dst = ring_u + lane * 16;
    int fill = 0;  // ring position of the next request, in bytes
    auto request = [&]() {
      if (requested < mine) {
        const int at = requested & 15;
        if (at == 0) {
          if (requested > 0) id = page_at(requested + (lane & 15), lane >> 4);
          const bool ok = id >= 0 && id < c.num_pages;
          bad = __ballot_sync(0xFFFFFFFFu, !ok);
          const uint32_t page = ok ? id : 0;
          const uint32_t row = ((s.t0 + ts + warp + (requested + (lane & 15)) * kWarps) * kTile + (lane >> 4) * kHalf) &
                               (c.page_size - 1);
          // page strides are below 2^32 bytes: one 32 x 32 -> 64 multiply-add
          code_off = static_cast<uint64_t>(page) * static_cast<uint32_t>(c.code_page_stride) + row * (D / 2);
          scale_off = static_cast<uint64_t>(page) * static_cast<uint32_t>(c.scale_page_stride) + row * (D / 16);
        }
        const uint64_t off0 = __shfl_sync(0xFFFFFFFFu, code_off, at), off1 = __shfl_sync(0xFFFFFFFFu, code_off, at + 16);
        const uint64_t sc_off = __shfl_sync(0xFFFFFFFFu, scale_off, at + 16 * (sc_part & 1));
        const uint32_t no0 = (bad >> at) & 1u, no1 = (bad >> (at + 16)) & 1u;
        none_next = no0 + 2 * no1;
        const int n0 = 16 - 16 * no0, n1 = 16 - 16 * no1;
        const uint32_t dst = code_dst + fill;
        auto k_at = [&](auto skip, uint64_t off) {
          return checked_at<uint4, decltype(skip)::value>(k_src + off, c.k_codes, codes_extent(c), kSiteKvCodes);
        };
        auto v_at = [&](auto skip, uint64_t off) {
          return checked_at<uint4, decltype(skip)::value>(v_src + off, c.v_codes, codes_extent(c), kSiteKvCodes);
        };
        constexpr std::integral_constant<int, 0> first{};
        copy16<0, 0>(dst, k_at(first, off0), n0);
        copy16<kCodes + kScales, 0>(dst, v_at(first, off0), n0);
        copy16<kHalfBytes, 0>(dst, k_at(first, off1), n1);
        copy16<kHalfBytes + kCodes + kScales, 0>(dst, v_at(first, off1), n1);
        if constexpr (kCodes == 1024) {
          constexpr std::integral_constant<int, 512> second{};
          copy16<512, 512>(dst, k_at(second, off0), n0);
          copy16<512 + kCodes + kScales, 512>(dst, v_at(second, off0), n0);
          copy16<512 + kHalfBytes, 512>(dst, k_at(second, off1), n1);
          copy16<512 + kHalfBytes + kCodes + kScales, 512>(dst, v_at(second, off1), n1);
        }
        if (kScaleLanes == 8 || sc_part < 4) copy16<0, 0>(sc_dst + fill,
                                                            checked_at<uint4>(sc_src + sc_off, sc_part & 2 ? c.v_scales : c.k_scales,
                                                                              scales_extent(c), kSiteKvScales),
                                                            sc_part & 1 ? n1 : n0);
        ++requested;
        fill = kStageBytes - fill;
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) request();

    // ---- query rows in FP16, scaled, as the lanes
    // of every warp will read them: lane (g, l4) has d [l4 D/4, (l4+1) D/4) of
    // row g of an 8-row tile, word w of it at [tile][w][lane]
#pragma unroll
    for (int n = 0; n < kPasses; ++n) {
      const int r = qr + n * kPass;
      const uint32_t w[4] = {qv[n].x, qv[n].y, qv[n].z, qv[n].w};
      float y[8], mx = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[2 * j] = to_f32(w[j] & 0xFFFFu, p.a.type);
        y[2 * j + 1] = to_f32(w[j] >> 16, p.a.type);
        mx = fmaxf(mx, fmaxf(fabsf(y[2 * j]), fabsf(y[2 * j + 1])));
      }
#pragma unroll
      for (int off = 1; off < kRowPieces; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
      float shrink, fs;
      row_scale(mx, p.scale_log2 * kS, shrink, fs);
      if (r < R) {
        q_all[((r >> 3) * KW + qp % KW) * 32 + (r & 7) * 4 + qp / KW] =
            make_uint4(pack_f16x2(y[0] * shrink, y[1] * shrink), pack_f16x2(y[2] * shrink, y[3] * shrink),
                       pack_f16x2(y[4] * shrink, y[5] * shrink), pack_f16x2(y[6] * shrink, y[7] * shrink));
        if (qp == 0) {
          RowInfo info;
          info.f = fs;
          visible(p, s, r0 + r, info.lo, info.hi);
          row_info[r] = info;
        }
      }
    }
    __syncthreads();
    float f[NT][2];              // factor of the scores of columns 2 l4, 2 l4 + 1
    int vlo[NT][2], vhi[NT][2];  // visible tokens of those columns
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const RowInfo info = row_info[8 * n + 2 * l4 + k];
        f[n][k] = info.f;
        vlo[n][k] = info.lo;
        vhi[n][k] = info.hi;
      }
    // tokens that every row sees: a row's bounds grow with its position
    const int all_lo = __shfl_sync(0xFFFFFFFFu, row_info[min(R, s.lq * p.group - r0) - 1].lo, 0);
    const int all_hi = __shfl_sync(0xFFFFFFFFu, row_info[0].hi, 0);

    float o[NT][VW * 4][4] = {};
    // what is added to a score (-m; 0 while nothing was seen), the value that the
    // sum may not pass (-inf until then, so that the first score passes it), and
    // this lane's share of the sum of P.  (Compared is what the exponentials
    // get, the same fma: a score and m round apart where they are large.)
    float down[NT][2] = {}, limit[NT][2], l[NT][2] = {};
#pragma unroll
    for (int n = 0; n < NT; ++n) limit[n][0] = limit[n][1] = -INFINITY;
    auto at_m = [&](int n, int i) { return limit[n][i] == -INFINITY ? -INFINITY : -down[n][i]; };

    // S^T row r holds token r ^ (r >> 1 & 1): neighbouring rows and the
    // tokens of one V load then differ in parity, which halves the bank
    // conflicts of 64-byte rows
    auto tok = [](int r) { return r ^ ((r >> 1) & 1); };

    int use = 0;  // ring position of the tile in use, in bytes
    auto walk = [&](auto hold) {
      for (int k = 0; k < mine; ++k) {
        const uint32_t none = none_next;
        request();
        copy_wait<kStages - 1>();
        __syncwarp();
        const uint8_t* const stage = ring + use;
        use = kStageBytes - use;
        const int tb = (s.t0 + ts + warp + k * kWarps) * kTile;  // first token
        const bool edge = tb < all_lo || tb + kTile > all_hi || none != 0;
        // ---- S^T
        float x[NT][2][4] = {};
        uint32_t kw[2][2][KW];
        uint32_t ksc[2][2];  // two scales (D = 64: one, and a zero)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* const kc = stage + half * kHalfBytes;
          const uint8_t* const ks = kc + kCodes;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int t = tok(g) + 8 * j;
            uint32_t(&k4)[KW] = kw[half][j];
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(kc + t * 64 + l4 * 16);
              k4[0] = v.x, k4[1] = v.y, k4[2] = v.z, k4[3] = v.w;
              ksc[half][j] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(ks + t * 8 + l4 * 2));
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(kc + t * 32 + l4 * 8);
              k4[0] = v.x, k4[1] = v.y;
              ksc[half][j] = e4m3x2_to_f16x2(ks[t * 4 + l4]);
            }
          }
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          uint4 qw[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) qw[n] = q[(n * KW + w) * 32];
          const uint32_t sel = w < 2 ? 0x1010 : 0x3232;  // block of word w: two words a block
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t s0 = __byte_perm(ksc[half][0], 0, sel), s1 = __byte_perm(ksc[half][1], 0, sel);
            uint32_t e0[4], e1[4];
            e2m1x8_to_f16x2(kw[half][0][w], e0);
            e2m1x8_to_f16x2(kw[half][1][w], e1);
            const uint32_t a[4] = {mul_f16x2(e0[0], s0), mul_f16x2(e1[0], s1), mul_f16x2(e0[1], s0), mul_f16x2(e1[1], s1)};
            const uint32_t b[4] = {mul_f16x2(e0[2], s0), mul_f16x2(e1[2], s1), mul_f16x2(e0[3], s0), mul_f16x2(e1[3], s1)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma(x[n][half], a, qw[n].x, qw[n].y);
              mma(x[n][half], b, qw[n].z, qw[n].w);
            }
          }
        }
        if (edge) {
          __syncwarp();  // keeps this a branch
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int t = tb + (i >> 2) * kHalf + tok(g) + (i & 2) * 4;
              if (t < vlo[n][i & 1] || t >= vhi[n][i & 1] || ((none >> (i >> 2)) & 1)) x[n][i >> 2][i & 3] = -INFINITY;
            }
        }
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            over |= fmaf(fmaxf(fmaxf(x[n][0][i], x[n][0][i + 2]), fmaxf(x[n][1][i], x[n][1][i + 2])), f[n][i],
                         down[n][i]) > limit[n][i];
        }
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float t = m_for(fmaxf(fmaxf(x[n][0][i], x[n][0][i + 2]), fmaxf(x[n][1][i], x[n][1][i + 2])), f[n][i]);
              t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
              const float m = at_m(n, i);
              t = fmaxf(t, m);
              const float r = t == m ? 1.0f : exp2_approx(m - t);
              if (t != -INFINITY) down[n][i] = -t, limit[n][i] = kTop;
              l[n][i] *= r;
#pragma unroll
              for (int u = 0; u < VW * 4; ++u) o[n][u][i] *= r, o[n][u][i + 2] *= r;
            }
          }
        }
        uint32_t pb[NT][2][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float y = fmaf(x[n][half][i], f[n][i & 1], down[n][i & 1]);
              x[n][half][i] = exp2_approx(decltype(hold)::value ? held(y) : y);
            }
            l[n][0] += x[n][half][0] + x[n][half][2];
            l[n][1] += x[n][half][1] + x[n][half][3];
            pb[n][half][0] = transpose8x8(pack_f16x2(x[n][half][0], x[n][half][1]));
            pb[n][half][1] = transpose8x8(pack_f16x2(x[n][half][2], x[n][half][3]));
          }
        }
        // ---- O^T: tokens of the k index 2 l4, 2 l4 + 1, 2 l4 + 8, 2 l4 + 9
        const int ta = tok(2 * l4), tc = tok(2 * l4 + 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* const vc = stage + half * kHalfBytes + kCodes + kScales;
          const uint8_t* const vs = vc + kCodes;
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
          uint32_t nan_tokens = 0;  // bit j: vsc[j] is NaN and its token may be hidden from some row
          if (edge) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int t = tb + half * kHalf + (j & 1 ? tc : ta) + (j & 2) * 4;
              const bool gone = t >= s.lk || ((none >> half) & 1);
              if (gone || (vsc[j] & 0x7Fu) == 0x7Fu) {
                // 0 * NaN would reach rows that do not see the token: take it
                // out of the product and give it to the rows that do (below)
                if (!gone) nan_tokens |= 1u << j;
                vsc[j] = 0;
              }
            }
          }
          const uint32_t sab = e4m3x2_to_f16x2(vsc[0] | (vsc[1] << 8));
          const uint32_t scd = e4m3x2_to_f16x2(vsc[2] | (vsc[3] << 8));
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            constexpr uint32_t kLow = 0x0F0F0F0Fu;
            uint32_t lo_ab[4], hi_ab[4], lo_cd[4], hi_cd[4];
            e2m1x8_to_f16x2(merge(vw[0][w], vw[1][w] << 4, kLow), lo_ab);
            e2m1x8_to_f16x2(merge(vw[0][w] >> 4, vw[1][w], kLow), hi_ab);
            e2m1x8_to_f16x2(merge(vw[2][w], vw[3][w] << 4, kLow), lo_cd);
            e2m1x8_to_f16x2(merge(vw[2][w] >> 4, vw[3][w], kLow), hi_cd);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t a[4] = {mul_f16x2(lo_ab[u], sab), mul_f16x2(hi_ab[u], sab),
                                     mul_f16x2(lo_cd[u], scd), mul_f16x2(hi_cd[u], scd)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma(o[n][4 * w + u], a, pb[n][half][0], pb[n][half][1]);
            }
          }
          if (edge && __any_sync(0xFFFFFFFFu, nan_tokens != 0)) {
            // the NaN tokens of lane g's own elements, gathered over l4
#pragma unroll 1
            for (int src = 0; src < 4; ++src) {
              const uint32_t bits = __shfl_sync(0xFFFFFFFFu, nan_tokens, (lane & ~3) | src);
#pragma unroll 1
              for (int j = 0; j < 4; ++j) {
                if (!((bits >> j) & 1)) continue;
                const int t = tb + half * kHalf + tok(2 * src + (j & 1)) + (j & 2) * 4;
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
    };
    bool far = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) far |= may_pass_top<D>(f[n][0]) || may_pass_top<D>(f[n][1]);
    if (__any_sync(0xFFFFFFFFu, far))
      walk(std::true_type{});
    else
      walk(std::false_type{});

    // ---- join the warps (their areas lie over all rings)
    __syncthreads();
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
          join_ml[(warp * R + col) * 2] = at_m(n, i);
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
    if (p.cut != nullptr && ts == 0 && !whole && threadIdx.x == 0) {
      // at most one item is cut behind its first tile in this CTA
      // its last tile is tiles - te - 1 units behind this CTA's end
      *cut_at(p, blockIdx.x) = make_int4(b, item, blockIdx.x, (s.tiles - te - 1) / share + 2);
    }
    const float vS = head_S(p, c.v_S, h);
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
        *partial_at<D, R>(p, at, d) = acc;
        if (d == 0) *partial_ml_at<R>(p, at) = make_float2(mm, ll);
      }
    }
    __syncthreads();

    if (!next_item()) return;
  }
}

// A CTA for RC rows of an item (8, or 1 where there are few items): adds up the
// partial results of an item that was cut, in an order that depends on their
// number alone.  The items are all of the call's, whose pieces each CTA works
// out while kv_rows_kernel still runs, or (kList) those that it listed as cut.
// D / 4 lanes take 4 elements each of the rows of a piece, the CTA's 8 warps
// every kStripes-th piece.
constexpr int kJoinWarps = 8;

template <int D, int NT, int RC, bool kList>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(const __grid_constant__ Params p) {
  constexpr int R = 8 * NT;
  constexpr int kLanes = D / 4, kStripes = kJoinWarps * 32 / kLanes;
  __shared__ float2 ml_s[kJoinWarps][RC];
  __shared__ float4 acc_s[kStripes][RC][kLanes];
  const int r0 = blockIdx.x % (R / RC) * RC;
  // Every CTA waits for kv_rows_kernel before it ends, also where it has
  // nothing to add up: what follows on the stream waits for this kernel only.
  auto rows_done = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  Span s;
  int b, item, c0, pieces;
  if constexpr (kList) {
    rows_done();
    const int4 cut = *cut_at(p, blockIdx.x / (R / RC));
    if (cut.w == 0) return;
    b = cut.x, item = cut.y, c0 = cut.z, pieces = cut.w;
    s = span_of(p, b);
  } else {
    __shared__ int red[2 * kJoinWarps];
    b = blockIdx.y;
    item = blockIdx.x / (R / RC);
    const Seq seq = sequence<R>(p, b);
    s = seq;
    if (item >= seq.blocks * p.a.c.kv_heads) return rows_done();
    const int2 units = units_before<R, kJoinWarps>(p, b, red);
    const int per = units_per_cta(units.y, p.ctas);
    const int first = units.x + item * seq.span + kItemCost;
    c0 = first / per;
    pieces = (first + seq.tiles - 1) / per - c0 + 1;
    rows_done();
    if (pieces == 1) return;
  }
  const int h = item % p.a.c.kv_heads, rb = item / p.a.c.kv_heads;
  const int rows = min(RC, s.lq * p.group - rb * R - r0);
  if (rows <= 0) return;
  // first of the RC rows of a piece; the one that holds the item's start lies in slot 1
  auto at = [&](int piece) { return ((static_cast<long long>(c0) + piece) * 2 + (piece == 0 ? 1 : 0)) * R + r0; };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // maximum m and sum l of row lane % RC: over pieces, lanes, warps
  auto add = [](float& m, float& l, float m2, float l2) {
    const float top = fmaxf(m, m2);
    l = l * (m == top ? 1.0f : exp2_approx(m - top)) + l2 * (m2 == top ? 1.0f : exp2_approx(m2 - top));
    m = top;
  };
  float m = -INFINITY, l = 0.0f;
  for (int i = threadIdx.x / RC; i < pieces; i += 32 * kJoinWarps / RC) {
    const float2 ml = *partial_ml_at<R>(p, at(i) + threadIdx.x % RC);
    add(m, l, ml.x, ml.y);
  }
#pragma unroll
  for (int o = RC; o < 32; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, o), l2 = __shfl_xor_sync(0xFFFFFFFFu, l, o);
    add(m, l, m2, l2);
  }
  if (lane < RC) ml_s[warp][lane] = make_float2(m, l);
  __syncthreads();
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) add(m, l, ml_s[w][lane % RC].x, ml_s[w][lane % RC].y);

  const int el = threadIdx.x % kLanes, stripe = threadIdx.x / kLanes;
  float4 acc[RC] = {};
#pragma unroll 4
  for (int i0 = 0; i0 < pieces; i0 += kStripes) {  // (whole warps stay together for the shuffles)
    const int i = i0 + stripe;
    const bool have = i < pieces;
    const long long row0 = at(have ? i : 0);
    // weight of row lane % RC of this lane's piece (D = 64: a warp has two)
    const float mi = partial_ml_at<R>(p, row0 + lane % RC)->x;
    const float z = !have ? 0.0f : (mi == m ? 1.0f : exp2_approx(mi - m));
#pragma unroll
    for (int r = 0; r < RC; ++r) {
      const float zr = __shfl_sync(0xFFFFFFFFu, z, (lane / kLanes * kLanes + r) & 31);
      if (have) {
        const float4 v = *partial_at<D, R>(p, row0 + r, 4 * el);
        acc[r].x += zr * v.x, acc[r].y += zr * v.y, acc[r].z += zr * v.z, acc[r].w += zr * v.w;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RC; ++r) acc_s[stripe][r][el] = acc[r];
  __syncthreads();
  const float vS = head_S(p, p.a.c.v_S, h);
  // (RC kLanes is a multiple of 32 or less than a warp's worth: warp 0 alone)
  for (int i = threadIdx.x; i < (RC * kLanes + 31) / 32 * 32; i += 32 * kJoinWarps) {
    const int r = i / kLanes, e = i % kLanes;
    const float mr = __shfl_sync(0xFFFFFFFFu, m, r % RC), lr = __shfl_sync(0xFFFFFFFFu, l, r % RC);
    if (r >= rows) continue;
    float4 a = acc_s[0][r][e];
#pragma unroll
    for (int w = 1; w < kStripes; ++w) {
      const float4 v = acc_s[w][r][e];
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    write_row(p, s, h, rb * R + r0 + r, 4 * e, a, lr == 0.0f ? 0.0f : vS / lr);
    if (e == 0) write_lse(p, s, h, rb * R + r0 + r, mr, lr);
  }
}

// Rows per item: the fewest 8-row tiles that hold all rows of a sequence.
int row_tiles(int64_t rows) { return rows <= 8 ? 1 : (rows <= 16 ? 2 : 4); }

// How a call is served: sequences of at most `limit` query rows for a KV head
// by kv_rows_kernel, the others by kv_prompt_kernel.
struct Plan {
  int64_t rows;   // most rows that kv_rows_kernel gets of a sequence
  int nt, ctas;   // its 8-row tiles and CTAs
  int items;      // its items of a sequence, at most
  enum { kByRow, kByTile, kListed } join;
  int limit;
  bool prompt;
  int num_sms;
  PromptPlan prompts;
  size_t rows_bytes, prompt_bytes;  // of the workspace
  bool fits;      // the work can be counted in 32 bits
};

Plan plan_of(int64_t batch, int64_t max_q, int64_t max_kv, int q_heads, int kv_heads, int head_dim, int num_sms) {
  Plan p{};
  p.num_sms = num_sms;
  const int64_t rows = max_q * (q_heads / kv_heads);
  const int64_t limit = rows_limit(head_dim);
  p.prompt = rows > limit;
  p.limit = static_cast<int>(limit);
  p.rows = p.prompt ? limit : rows;
  p.nt = row_tiles(p.rows);
  p.items = static_cast<int>((p.rows + 8 * p.nt - 1) / (8 * p.nt)) * kv_heads;
  // Joining: 8 rows a CTA read a piece's rows together; where that leaves SMs
  // without a CTA, a row a CTA shortens the walk over the pieces (two sequences
  // of 131072 tokens, 16 items of 47 pieces: 72 us with 8 rows a CTA, 67 with
  // 1; 48 of 8192: 60 us with 8, 64 with 1).  Where items are many, looking at
  // all lengths in every CTA costs more than a list of the cut ones (8 KV heads
  // of 128, sequences of up to 1000 tokens, without and with the list: 24
  // sequences 16.3 and 16.7 us, 48 21.3 and 21.7, 64, which are 512 CTAs, 27.0
  // and 25.0, 256 74.2 and 67.7; of up to 8000: 24 41.0 and 41.6, 64 94.1 and 91.3).
  const int64_t join_ctas = static_cast<int64_t>(p.items) * batch * p.nt;
  p.join = join_ctas < num_sms ? Plan::kByRow : (join_ctas < 512 ? Plan::kByTile : Plan::kListed);
  const double tiles = static_cast<double>(batch) * p.items * static_cast<double>((max_kv + kTile - 1) / kTile + 1 + kItemCost);
  p.fits = tiles < 0x7FF00000;
  const int64_t wave = static_cast<int64_t>(num_sms) * ctas_per_sm(head_dim, p.nt);
  const double want = tiles / kWarps + 1.0;
  p.ctas = static_cast<int>(want < static_cast<double>(wave) ? static_cast<int64_t>(want) : wave);
  p.rows_bytes = (static_cast<size_t>(p.ctas) * 2 * 8 * p.nt * (head_dim + 2) * sizeof(float) +
                  static_cast<size_t>(p.ctas) * sizeof(int4) + 255) / 256 * 256;
  if (p.prompt) {
    p.prompts = prompt_plan(batch, rows, max_kv, kv_heads, num_sms);
    p.prompt_bytes = prompt_workspace_bytes(p.prompts, head_dim);
    p.fits = p.fits && p.prompts.items * p.prompts.splits <= 0x7FFFFFFF;  // the grid
  }
  return p;
}

template <int D, int NT>
cudaError_t run_rows(Params& p, const Plan& plan, cudaStream_t stream) {
  constexpr int R = 8 * NT;
  constexpr int smem = rows_smem(D, NT);
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.set(reinterpret_cast<const void*>(&kv_rows_kernel<D, NT>), smem);
  if (e != cudaSuccess) return e;
  p.partial_ml = p.partial + static_cast<int64_t>(p.ctas) * 2 * R * D;
  p.cut = plan.join == Plan::kListed ? reinterpret_cast<int4*>(p.partial_ml + static_cast<int64_t>(p.ctas) * 2 * R * 2) : nullptr;
  kv_rows_kernel<D, NT><<<p.ctas, kThreads, smem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the joining kernel is launched while the first still runs (programmatic
  // dependent launch) and waits for its end on the device
  cudaLaunchConfig_t cfg{};
  if (plan.join == Plan::kListed)
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas) * NT);
  else
    cfg.gridDim = dim3(static_cast<unsigned>(plan.items * (plan.join == Plan::kByRow ? R : NT)), static_cast<unsigned>(p.a.batch));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const Params& args = p;
  if (plan.join == Plan::kByRow) return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NT, 1, false>, args);
  if (plan.join == Plan::kByTile) return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NT, 8, false>, args);
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, NT, 8, true>, args);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t batch, int64_t max_q, int64_t max_kv, int q_heads,
                                    int kv_heads, int head_dim, int num_sms) {
  const Plan p = plan_of(batch, max_q, max_kv, q_heads, kv_heads, head_dim, num_sms);
  return p.fits ? p.rows_bytes + p.prompt_bytes : 0;
}

cudaError_t launch_kv_attention(const KvAttention& a, void* workspace, int num_sms, cudaStream_t stream) {
  if (a.batch == 0 || a.total_q == 0) return cudaSuccess;
  const Plan plan = plan_of(a.batch, a.max_q, a.max_kv, a.q_heads, a.c.kv_heads, a.c.head_dim, num_sms);
  Params p{};
  p.a = a;
  p.group = a.q_heads / a.c.kv_heads;
  while ((1 << p.page_shift) < a.c.page_size) ++p.page_shift;
  p.scale_log2 = a.scale * 1.44269504088896341f;
  p.partial = static_cast<float*>(workspace);
  p.ctas = plan.ctas;
  p.rows_limit = plan.limit;
  if (plan.prompt) {
    const cudaError_t e = launch_kv_prompt(p, plan.prompts, static_cast<char*>(workspace) + plan.rows_bytes, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.c.head_dim == 128) {
    if (plan.nt == 1) return run_rows<128, 1>(p, plan, stream);
    if (plan.nt == 2) return run_rows<128, 2>(p, plan, stream);
    return run_rows<128, 4>(p, plan, stream);
  }
  if (plan.nt == 1) return run_rows<64, 1>(p, plan, stream);
  if (plan.nt == 2) return run_rows<64, 2>(p, plan, stream);
  return run_rows<64, 4>(p, plan, stream);
}

}  // namespace nvfp4
