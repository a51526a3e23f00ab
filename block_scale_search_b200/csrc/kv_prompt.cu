// kv_prompt.cu -- attention of many query rows over the paged NVFP4 cache
// (prompts and prompt chunks), on the tcgen05 tensor cores.
//
// One CTA takes 256 query rows (two tiles of 128) of one sequence and KV head
// and walks the cached tokens 128 at a time:
//   S = Q K^T     Q, K in shared memory (FP16), S in TMEM (FP32)
//   P = e^(S - m) S from TMEM to registers and back as FP16 over S's columns
//   O += P V      P from TMEM, V in shared memory, O in TMEM (FP32)
// At head_dim 128 a step of 256 x 128 scores is 2048 cycles of MMA at the
// nominal rate, and 2048 cycles of ex2 at 16 a clock, so all else has to run
// beside them:
//   warps 0-3, 4-7   softmax of tile 0 and of tile 1, a thread a row
//   warps 8-11       decode K and V: packed rows, which arrive by cp.async two
//                    half steps ahead, to FP16 rows, two stages each
//   warp 12          issues the MMAs: P V of one tile and then Q K^T of its
//                    next step, in turn with the other tile, so that one
//                    tile's MMAs run while the other's softmax does
// Registers move from the last two groups of warps to the softmax, whose
// threads hold a row's 128 scores at once.  A step takes 3400 cycles: a tile's
// softmax 2400 (1900 of them in the exponentials, which both tiles share) and
// then its MMAs 1024 before its next scores are there.  Measured: 4 chunks of
// 2048 tokens over up to 8192, 32 / 8 heads of 128, 508 us in short bursts or
// 1.03 PFLOP/s (62% of the measured GEMM rate), 565 us back to back under the
// power cap; 8000 tokens at once 1.06.  At head_dim 64 the MMAs halve and the
// softmax does not: 8000 tokens at once 394 us for half the work that takes 498
// at 128.
// The cache is decoded once per CTA: 256 rows share it.  A decoded value (code
// times scale) is exact in FP16; Q's rows are scaled by powers of two and P is
// rounded as in kv_attention.cu, and the running maximum moves by the same
// rule, which leaves O alone in almost every step.
//
// K and V rows lie alike: 128-byte rows of 64 elements with the 128-byte
// swizzle, halves of a row 16 KB apart.  K is the K-major operand of S; of
// P V, whose inner index are the tokens, the same rows are the MN-major one.
#include <type_traits>

#include "kv_attention.cuh"

namespace nvfp4 {

namespace {

constexpr int kTokens = 128;                // of a step
constexpr int kTileRows = 128;
constexpr int kRows = 2 * kTileRows;        // of a CTA
constexpr int kPromptWarps = 16;
constexpr int kPromptThreads = 32 * kPromptWarps;
constexpr int kHalfTile = kTokens * 128;    // bytes: 128 rows of 64 elements

__device__ unsigned int g_stalls;           // waits given up
// Cycles after which a wait is given up, every how many tries (a power of two)
// it looks at the clock, and the instruction that tries: try_wait may hold the
// warp a while.  Tests of the checked build set the limit, to 0 too.
#ifdef NVFP4HS_CHECKS
__device__ long long g_wait_limit = 1ll << 32;
constexpr uint32_t kLookEvery = 1;
#define NVFP4_MBAR_TRY "mbarrier.test_wait"
#else
constexpr long long g_wait_limit = 1ll << 32;
constexpr uint32_t kLookEvery = 256;
#define NVFP4_MBAR_TRY "mbarrier.try_wait"
#endif

// Shared memory from a 1024-byte boundary: Q of both tiles, two stages of K,
// two of V, and three slots of packed rows (K or V of a step).
template <int D>
struct Layout {
  static constexpr int kTile = kHalfTile * (D / 64);
  static constexpr int kSlot = kTokens * (D / 2) + kTokens * (D / 32) * 4;
  static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile, kPacked = 6 * kTile;
  static constexpr int kBytes = kPacked + 3 * kSlot;
};

enum Bar : int {
  kQFull = 0,             // +t: Q of tile t is written
  kKFull = 2, kKEmpty = 4,  // +stage
  kVFull = 6, kVEmpty = 8,
  kSFull = 10,            // +t: S of tile t (and all earlier P V) is done
  kPFull = 12,            // +2 t + half: that half of P's columns of tile t is written
  kOFull = 16,            // +t: the last P V of tile t is done
  kScan = 18,             // all V scales were seen
  kBars = 19
};

struct Shared {
  uint64_t bar[kBars];
  uint32_t tmem;
  int gave_up;   // a wait was given up: no further one waits
  int nan_v;     // some visible V scale is NaN
};

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; " NVFP4_MBAR_TRY ".parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}
// Waits for a phase, for about two seconds at most: a wait given up is counted
// and ends all later ones of the CTA, which then runs to its end and leaves NaN.
template <int kSleep>
__device__ __forceinline__ void mbar_wait_slow(Shared* sh, uint32_t bar, uint32_t parity) {
  long long t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if constexpr (kSleep > 0) __nanosleep(kSleep);
    if (mbar_try(bar, parity)) return;
    if ((n & (kLookEvery - 1)) != 0) continue;
    if (*reinterpret_cast<volatile int*>(&sh->gave_up)) return;
    if (t0 == 0) t0 = clock64();
    if (clock64() - t0 > g_wait_limit) {
      atomicAdd(&g_stalls, 1u);
      *reinterpret_cast<volatile int*>(&sh->gave_up) = 1;
      __threadfence_block();  // before what this warp makes of the unfinished phase
      return;
    }
  }
}
// kSleep: ns between tries, which leaves issue slots to the warps that work.
constexpr int kSoftmaxSleep = 20, kDecodeSleep = 100;
// Waits for MMAs in flight before TMEM is given back, also after a wait was
// given up (then for a tenth of a second at most).
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity) && clock64() - t0 < (1ll << 28)) {
  }
}
template <int kSleep = 0>
__device__ __forceinline__ void mbar_wait(Shared* sh, uint32_t bar, uint32_t parity) {
  if (!mbar_try(bar, parity)) mbar_wait_slow<kSleep>(sh, bar, parity);
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// True in one lane of a converged warp, in a way that the compiler knows to be
// one lane (a comparison of the lane's number makes it serialise every MMA,
// whose operands are warp-uniform: 147 cycles each instead of 64).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(one));
  return one != 0;
}

// Operand descriptor: 128-byte swizzle, groups of 8 rows 1024 bytes apart;
// `lead` is the distance of 64-element halves (used by the MN-major operand).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
// FP16 operands, FP32 sums, 128 rows, n columns; b_mn: B's outer index is contiguous.
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(add ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(add ? 1 : 0)
      : "memory");
}

#define NVFP4_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define NVFP4_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : NVFP4_R8(r, 0), NVFP4_R8(r, 8), NVFP4_R8(r, 16), NVFP4_R8(r, 24) : "r"(addr));
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : NVFP4_R8(r, 0), NVFP4_R8(r, 8) : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::NVFP4_I8(
          r, 0),
      NVFP4_I8(r, 8), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#undef NVFP4_R8
#undef NVFP4_I8

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Every how many pairs of exponentials one is computed by exp2_poly2.
constexpr int kPolyEvery = 4;

// 2^x of two numbers on the FMA pipe, beside the ex2 unit's 16 a clock.
// x = n + r with n whole and |r| <= 1/2: adding 1.5 * 2^23 rounds to n and
// leaves it in the low bits.  2^r by a quartic (least squares of the relative
// error, reweighted until it was even: 2.6e-6), n into the exponent.  Below
// -126 the result stays at 2^-126.
__device__ __forceinline__ void exp2_poly2(f32x2_t x, float& a, float& z) {
  f2_unpack(x, a, z);
  x = f2_pack(fmaxf(a, -126.0f), fmaxf(z, -126.0f));
  const f32x2_t t = f2_add(x, f2_pack(12582912.0f, 12582912.0f));
  const f32x2_t n = f2_add(t, f2_pack(-12582912.0f, -12582912.0f));
  const f32x2_t r = f2_fma(n, f2_pack(-1.0f, -1.0f), x);
  f32x2_t y = f2_fma(r, f2_pack(0.00957010128f, 0.00957010128f), f2_pack(0.0559178603f, 0.0559178603f));
  y = f2_fma(y, r, f2_pack(0.240247448f, 0.240247448f));
  y = f2_fma(y, r, f2_pack(0.693121815f, 0.693121815f));
  y = f2_fma(y, r, f2_pack(0.999999261f, 0.999999261f));
  float ta, tz, ya, yz;
  f2_unpack(t, ta, tz);
  f2_unpack(y, ya, yz);
  a = __uint_as_float((__float_as_uint(ta) << 23) + __float_as_uint(ya));
  z = __uint_as_float((__float_as_uint(tz) << 23) + __float_as_uint(yz));
}

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, uint64_t src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Byte offset of 16-byte piece `piece` (of D / 8) of row `row` of a tile.
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return (piece >> 3) * kHalfTile + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// A row's sums of one split from element d on, and its maximum and sum.
__device__ __forceinline__ int64_t split_rows(const Params& p) {
  return static_cast<int64_t>(p.row_blocks) * p.a.batch * p.a.c.kv_heads * p.splits * kRows;
}
template <int D>
__device__ __forceinline__ float4* split_o_at(const Params& p, int64_t row, int d) {
  return checked(reinterpret_cast<float4*>(p.split_o + row * D + d), p.split_o, split_rows(p) * D * 4, kSiteKvSplit);
}
__device__ __forceinline__ float2* split_ml_at(const Params& p, int64_t row) {
  return checked(p.split_ml + row, p.split_ml, split_rows(p) * 8, kSiteKvSplit);
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1) kv_prompt_kernel(const __grid_constant__ Params p) {
  using L = Layout<D>;
  extern __shared__ uint8_t dynamic[];
  __shared__ Shared sh;
  uint8_t* const smem = dynamic + ((1024 - (smem_u32(dynamic) & 1023)) & 1023);
  const uint32_t smem_a = smem_u32(smem);
  const nvfp4_kv_cache& c = p.a.c;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  // the longest items (a sequence's last rows) first, their splits side by side
  const int per_block = p.a.batch * c.kv_heads;
  const int item = static_cast<int>(blockIdx.x) / p.splits, split = static_cast<int>(blockIdx.x) % p.splits;
  const int rb = p.row_blocks - 1 - item / per_block;
  const int bh = item % per_block;
  const int b = bh / c.kv_heads, h = bh % c.kv_heads;
  const Span s = span_of(p, b);
  const int rows = s.lq * p.group, r0 = rb * kRows;
  if (rows <= p.rows_limit || r0 >= rows) return;  // the other kernel's, or no rows

  // tokens that some row sees, and the steps over them
  int lo, hi, unused;
  visible(p, s, r0, lo, unused);
  visible(p, s, min(r0 + kRows, rows) - 1, unused, hi);
  const int all_first = lo / kTokens;
  const int all_steps = hi > lo ? (hi + kTokens - 1) / kTokens - all_first : 0;
  // and this CTA's part of them
  const int begin = static_cast<int>(static_cast<int64_t>(all_steps) * split / p.splits);
  const int first = all_first + begin;
  const int steps = static_cast<int>(static_cast<int64_t>(all_steps) * (split + 1) / p.splits) - begin;

  // steps [from(t), to(t)) of them in which tile t sees a token: with a window
  // or causally the other steps are the other tile's only
  int tile_from[2], tile_to[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int a = r0 + t * kTileRows, z = min(a + kTileRows, rows) - 1;
    int t_lo, t_hi, other;
    visible(p, s, a, t_lo, other);
    visible(p, s, z, other, t_hi);
    const bool some = a <= z && t_hi > t_lo;
    tile_from[t] = some ? min(max(t_lo / kTokens - first, 0), steps) : 0;
    tile_to[t] = some ? min(max((t_hi + kTokens - 1) / kTokens - first, tile_from[t]), steps) : 0;
  }
  auto bar = [&](int i) { return smem_u32(&sh.bar[i]); };
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(kQFull + t), 128);
      mbar_init(bar(kKFull + t), 128);
      mbar_init(bar(kKEmpty + t), 1);
      mbar_init(bar(kVFull + t), 128);
      mbar_init(bar(kVEmpty + t), 1);
      mbar_init(bar(kSFull + t), 1);
      mbar_init(bar(kPFull + 2 * t), 128);
      mbar_init(bar(kPFull + 2 * t + 1), 128);
      mbar_init(bar(kOFull + t), 1);
    }
    mbar_init(bar(kScan), 128);
    sh.gave_up = 0;
    sh.nan_v = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {  // all of TMEM: one CTA an SM
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // columns: S (P over its first half) of tile t at 128 t, O at 256 + D t

  // 128 registers a thread at launch; 128 * (2 * 184 + 96 + 48) are all of them
  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int t = warp >> 2, row = r0 + t * kTileRows + (threadIdx.x & 127);
    const bool have = row < rows;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 (warp % 4)
    const uint32_t s_col = tmem + lane_base + 128 * t, o_col = tmem + lane_base + 256 + D * t;
    float f;  // factor of the row's scores, base 2
    {
      const uint16_t* src = static_cast<const uint16_t*>(p.a.Q) +
                            (s.q0 + (have ? row : r0) / p.group) * p.a.q_token_stride +
                            static_cast<int64_t>(h * p.group + (have ? row : r0) % p.group) * p.a.q_head_stride;
      uint4 v[D / 8];
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        v[i] = have ? query_piece(p, src + 8 * i) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mx = fmaxf(mx, fmaxf(fabsf(to_f32(w[j] & 0xFFFFu, p.a.type)), fabsf(to_f32(w[j] >> 16, p.a.type))));
      }
      float shrink;
      row_scale(mx, p.scale_log2 * head_S(p, c.k_S, h), shrink, f);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = pack_f16x2(to_f32(w[j] & 0xFFFFu, p.a.type) * shrink, to_f32(w[j] >> 16, p.a.type) * shrink);
        *reinterpret_cast<uint4*>(smem + L::kQ + t * L::kTile + tile_at(threadIdx.x & 127, i)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_async();
      mbar_arrive(bar(kQFull + t));
    }
    int vlo, vhi;
    visible(p, s, row, vlo, vhi);
    // tokens that all rows of the tile see
    int all_lo, all_hi, x0, x1;
    visible(p, s, min(r0 + t * kTileRows, rows - 1), x0, all_hi);
    visible(p, s, min(r0 + (t + 1) * kTileRows, rows) - 1, all_lo, x1);
    const int* const row_table = p.a.table + b * p.a.table_stride;
    // lane i < 8: the table's entry for tokens 16 i .. of a step (0 if none is
    // needed), loaded a step before it is looked at
    auto page_of = [&](int i) {
      const int tok = (first + i) * kTokens + 16 * lane;
      return lane < 8 && i < steps && tok < s.lk ? table_entry(p, row_table, tok >> p.page_shift) : 0;
    };
    int page = 0;
    // what is added to a score (-m; 0 while nothing was seen), what the sum may
    // not pass, and the sum of P, as in kv_rows_kernel
    float down = 0.0f, limit = -INFINITY, l = 0.0f;
    auto at_m = [&] { return limit == -INFINITY ? -INFINITY : -down; };
    const int from = t ? tile_from[1] : tile_from[0], to = t ? tile_to[1] : tile_to[0];
    page = page_of(from);
    auto walk = [&](auto hold) {
      for (int i = from; i < to; ++i) {
        const uint32_t parity = (i - from) & 1;
        const int tb = (first + i) * kTokens;
        const uint32_t dead = __ballot_sync(0xFFFFFFFFu, page < 0 || page >= c.num_pages);
        page = page_of(i + 1);
        const bool edge = tb < all_lo || tb + kTokens > all_hi || dead != 0;
        mbar_wait<kSoftmaxSleep>(&sh, bar(kSFull + t), parity);
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_load32(s_col + 32 * q, x[q]);
        tmem_wait_load();
        if (edge) {  // hidden scores become -inf
          __syncwarp();  // keeps this a branch
          // tokens [a, z) of the step are visible but for those of dead pages
          const int a = min(max(vlo - tb, 0), kTokens), z = min(max(vhi - tb, 0), kTokens);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // bit j: column 32 q + j is visible
            const int from = min(max(a - 32 * q, 0), 32), to = min(max(z - 32 * q, 0), 32);
            uint32_t vis = static_cast<uint32_t>((uint64_t{1} << to) - (uint64_t{1} << from));
            if (to <= from) vis = 0;
            if ((dead >> (2 * q)) & 1) vis &= 0xFFFF0000u;
            if ((dead >> (2 * q + 1)) & 1) vis &= 0x0000FFFFu;
#pragma unroll
            for (int j = 0; j < 32; ++j) x[q][j] = (vis >> j) & 1 ? x[q][j] : 0xFF800000u;
          }
        }
        // a NaN score has to reach m: not every exponential below would keep it
        float m4[4];  // chains short enough to overlap
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float a = __uint_as_float(x[q][0]), z = __uint_as_float(x[q][1]);
#pragma unroll
          for (int j = 2; j < 32; j += 4) {
            a = max3_nan(a, __uint_as_float(x[q][j]), __uint_as_float(x[q][j + 1]));
            if (j + 3 < 32) z = max3_nan(z, __uint_as_float(x[q][j + 2]), __uint_as_float(x[q][j + 3]));
          }
          m4[q] = max3_nan(a, z, z);
        }
        const float mx = max3_nan(max3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]);
        if (__any_sync(0xFFFFFFFFu, !(fmaf(mx, f, down) <= limit))) {
          // (inf - inf below would be NaN, which the polynomial does not keep)
          const float m = at_m(), next = m_for(mx, f);
          float top = max3_nan(m, next, next);
          if (top == INFINITY) top = __uint_as_float(0x7FC00000u);
          const float r = top == m ? 1.0f : exp2_approx(m - top);
          if (top != -INFINITY) down = -top, limit = kTop;
          l *= r;
          if (i > from) {
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_load16(o_col + 16 * q, o);
              tmem_wait_load();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * r);
              tmem_store16(o_col + 16 * q, o);
            }
          }
        }
        const f32x2_t f2 = f2_pack(f, f), d2 = f2_pack(down, down);
        f32x2_t sum[4] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            f32x2_t y = f2_fma(f2_pack(__uint_as_float(x[q][2 * j]), __uint_as_float(x[q][2 * j + 1])), f2, d2);
            float a, z;
            if constexpr (decltype(hold)::value) {
              f2_unpack(y, a, z);
              y = f2_pack(held(a), held(z));
            }
            if (j % kPolyEvery == kPolyEvery - 1) {
              exp2_poly2(y, a, z);
            } else {
              f2_unpack(y, a, z);
              a = exp2_approx(a);
              z = exp2_approx(z);
            }
            sum[j & 3] = f2_add(sum[j & 3], f2_pack(a, z));
            o[j] = pack_f16x2(a, z);
          }
          tmem_store16(s_col + 16 * q, o);  // over scores that are in registers
          if (q == 1) {  // P V may begin
            tmem_wait_store();
            tc_fence_before();
            mbar_arrive(bar(kPFull + 2 * t));
          }
        }
        {
          float a, z;
          f2_unpack(f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3])), a, z);
          l += a + z;
        }
        tmem_wait_store();
        tc_fence_before();
        mbar_arrive(bar(kPFull + 2 * t + 1));
      }
    };
    if (__any_sync(0xFFFFFFFFu, may_pass_top<D>(f)))
      walk(std::true_type{});
    else
      walk(std::false_type{});
    // -------------------------------------------------------------- result
    if (to > from) {
      mbar_wait(&sh, bar(kOFull + t), 0);
      tc_fence_after();
      mbar_wait(&sh, bar(kScan), 0);
    }
    uint32_t nan_blocks = 0;  // bit i: a visible V of elements 16 i .. is NaN
    if (*reinterpret_cast<volatile int*>(&sh.nan_v) && have) {
      const int tk1 = min(vhi, (first + steps) * kTokens);
      for (int tk = max(vlo, first * kTokens); tk < tk1; ++tk) {
        const int id = table_entry(p, row_table, tk >> p.page_shift);
        if (id < 0 || id >= c.num_pages) continue;
        const uint8_t* sc = c.v_scales + id * c.scale_page_stride +
                            (static_cast<int64_t>(h) * c.page_size + (tk & (c.page_size - 1))) * (D / 16);
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t code = *checked(sc + i, c.v_scales, scales_extent(c), kSiteKvScales);
          nan_blocks |= (code & 0x7Fu) == 0x7Fu ? 1u << i : 0u;
        }
      }
    }
    float m = at_m();
    // No number of an unfinished phase leaves the CTA as a result.
    if (*reinterpret_cast<volatile int*>(&sh.gave_up)) m = l = __uint_as_float(0x7FC00000u);
    if (m == -INFINITY) l = 0.0f;  // saw no token (the sum may hold some 2^-126)
    const float inv = l == 0.0f ? 0.0f : head_S(p, c.v_S, h) / l;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + t) * kTileRows + (threadIdx.x & 127);
    if (p.splits > 1 && have) {
      // (a NaN maximum goes into the sum: the joining maximum passes over it)
      *split_ml_at(p, at) = m != m ? make_float2(0.0f, m) : make_float2(m, l);
    }
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
      uint32_t x[32];
      if (to > from) {
        tmem_load32(o_col + 32 * q, x);
        tmem_wait_load();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = 0;
      }
      if (have) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if ((nan_blocks >> (2 * q + j / 16)) & 1) x[j] = 0x7FC00000u;
        if (p.splits > 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *split_o_at<D>(p, at, 32 * q + 4 * j) =
                make_float4(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1]),
                            __uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            write_row(p, s, h, row, 32 * q + 4 * j,
                      make_float4(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1]),
                                  __uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])),
                      inv);
        }
      }
    }
    if (have && p.splits == 1) write_lse(p, s, h, row, m, l);
    tc_fence_before();
  } else if (warp < 12) {
    // ------------------------------------------------------------- decode
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    // A tile is 128 rows of D / 2 code bytes; a thread takes 16 bytes (32
    // elements) of D / 32 rows, of K and of V.  Lanes 2 i and 2 i + 1 take
    // neighbouring parts of row i of the warp's 16: loads are whole sectors,
    // and eight lanes' stores cover all banks.
    constexpr int kPieces = D / 32;
    const int th = threadIdx.x - 256, wg_warp = warp - 8;
    const int part = D == 128 ? (th & 1) + 2 * (wg_warp & 1) : th & 1;
    const int tr = D == 128 ? ((th >> 1) & 15) + 16 * (wg_warp >> 1) : th >> 1;  // row tr + j 128 / kPieces
    const int* const row_table = p.a.table + b * p.a.table_stride;
    const int64_t head_codes = static_cast<int64_t>(h) * c.page_size * (D / 2) + part * 16;
    // (a row's scales are copied four at a time)
    const int64_t head_scales = static_cast<int64_t>(h) * c.page_size * (D / 16) + (part >> 1) * 4;
    const uint32_t code_page = static_cast<uint32_t>(c.code_page_stride);
    const uint32_t scale_page = static_cast<uint32_t>(c.scale_page_stride);
    const uint64_t k_codes = reinterpret_cast<uint64_t>(c.k_codes + head_codes);
    const uint64_t v_codes = reinterpret_cast<uint64_t>(c.v_codes + head_codes);
    const uint64_t k_scales = reinterpret_cast<uint64_t>(c.k_scales + head_scales);
    const uint64_t v_scales = reinterpret_cast<uint64_t>(c.v_scales + head_scales);
    // A thread copies what it will decode, so nobody else waits for it:
    // codes at slot + (j 128 + th) 16, scales behind them at (j 128 + th) 4.
    const uint32_t packed = smem_a + L::kPacked;
    auto page_of = [&](int i) {  // lane l < 8: the table's entry for tokens 16 l .. of step i, or -1
      const int tok = (first + i) * kTokens + 16 * lane;
      return lane < 8 && i < steps && tok < s.lk ? table_entry(p, row_table, tok >> p.page_shift) : -1;
    };
    // starts the copy of K or V of step i, whose pages are `ids`, to a slot;
    // returns bit j: the row of piece j is a cached token (the others are any
    // row, to be given scale 0)
    auto request = [&](int i, int ids, bool isv, uint32_t slot) {
      const uint64_t codes = isv ? v_codes : k_codes, scales = isv ? v_scales : k_scales;
      uint32_t there = 0;
      if (i < steps) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const int row = tr + j * (kTokens / kPieces), tok = (first + i) * kTokens + row;
          const int id = __shfl_sync(0xFFFFFFFFu, ids, row >> 4);
          const bool ok = id >= 0 && id < c.num_pages && tok < s.lk;
          const uint64_t page = static_cast<uint32_t>(ok ? id : 0);
          const uint32_t in_page = tok & (c.page_size - 1);
          there |= ok ? 1u << j : 0u;
          copy_async<16>(packed + slot + (j * 128 + th) * 16,
                         checked_at<uint4>(codes + page * code_page + in_page * (D / 2), isv ? c.v_codes : c.k_codes,
                                           codes_extent(c), kSiteKvCodes));
          copy_async<4>(packed + slot + kTokens * (D / 2) + (j * 128 + th) * 4,
                        checked_at<uint32_t>(scales + page * scale_page + in_page * (D / 16),
                                             isv ? c.v_scales : c.k_scales, scales_extent(c), kSiteKvScales));
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return there;
    };
    uint32_t at[4];  // of a row's four pieces in a tile; rows are 8 k apart, so the swizzle stays
#pragma unroll
    for (int u = 0; u < 4; ++u) at[u] = tile_at(tr, part * 4 + u);
    // decodes a slot's rows into a tile, once the tile's last use is over
    bool nan_v = false;
    auto decode = [&](uint32_t slot, uint32_t there, bool isv, int bar_empty, uint32_t parity, uint8_t* tile) {
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      const uint8_t* const from = smem + L::kPacked + slot;
      uint4 w[kPieces];
      uint32_t sc[kPieces], odd = 0;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        w[j] = *reinterpret_cast<const uint4*>(from + (j * 128 + th) * 16);
        sc[j] = *reinterpret_cast<const uint32_t*>(from + kTokens * (D / 2) + (j * 128 + th) * 4);
        if (part & 1) sc[j] >>= 16;
        sc[j] = (there >> j) & 1 ? sc[j] & 0xFFFFu : 0u;
        odd |= ((sc[j] & 0x7F7Fu) + 0x0101u) & 0x8080u;
      }
      if (isv && odd) {
        // 0 * NaN would reach rows that do not see the token: NaN is taken out
        // of the product, and the rows that see it look for it at the end
        nan_v = true;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          if ((sc[j] & 0x7Fu) == 0x7Fu) sc[j] &= 0xFF00u;
          if ((sc[j] & 0x7F00u) == 0x7F00u) sc[j] &= 0x00FFu;
        }
      }
      mbar_wait<kDecodeSleep>(&sh, bar(bar_empty), parity);
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const uint32_t two = e4m3x2_to_f16x2(sc[j]);
        const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
        const uint32_t wv[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t e[4];
          e2m1x8_to_f16x2(wv[u], e);
          const uint32_t sx = u < 2 ? s0 : s1;
          *reinterpret_cast<uint4*>(tile + at[u] + j * (kTokens / kPieces) * 128) =
              make_uint4(mul_f16x2(e[0], sx), mul_f16x2(e[1], sx), mul_f16x2(e[2], sx), mul_f16x2(e[3], sx));
        }
      }
      fence_async();
    };
    int ids = page_of(0);
    uint32_t there = request(0, ids, false, 0);
    request(0, ids, true, L::kSlot);
    ids = page_of(1);
    uint32_t slot = 0;  // of K of step i; V's is the next, and the one after is free
    auto after = [](uint32_t sl) { return sl == 2 * L::kSlot ? 0u : sl + L::kSlot; };
    for (int i = 0; i < steps; ++i) {
      const int st = i & 1;
      const uint32_t parity = ((i >> 1) & 1) ^ 1, v_slot = after(slot), free_slot = after(v_slot);
      const int ids_after = page_of(i + 2);
      const uint32_t next_there = request(i + 1, ids, false, free_slot);
      decode(slot, there, false, kKEmpty + st, parity, smem + L::kK + st * L::kTile);
      mbar_arrive(bar(kKFull + st));
      request(i + 1, ids, true, slot);
      decode(v_slot, there, true, kVEmpty + st, parity, smem + L::kV + st * L::kTile);
      mbar_arrive(bar(kVFull + st));
      ids = ids_after;
      there = next_there;
      slot = free_slot;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (nan_v) *reinterpret_cast<volatile int*>(&sh.nan_v) = 1;
    mbar_arrive(bar(kScan));
  } else {
    // ---------------------------------------------------------------- MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 12 && steps > 0) {
      constexpr uint32_t kQk = mma_desc(kTokens, false), kPv = mma_desc(D, true);
      const uint64_t q_desc = smem_desc(smem_a + L::kQ, 16), k_desc = smem_desc(smem_a + L::kK, 16),
                     v_desc = smem_desc(smem_a + L::kV, kHalfTile);
      constexpr uint64_t kTileStep = L::kTile >> 4;  // in a descriptor's address units
      auto qk = [&](int t, int st) {
        const uint64_t a = q_desc + t * kTileStep, k0 = k_desc + st * kTileStep;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t at = ((k >> 2) * kHalfTile + (k & 3) * 32) >> 4;
          mma_ss(tmem + 128 * t, a + at, k0 + at, kQk, k > 0);
        }
        tc_commit(bar(kSFull + t));
      };
      auto pv = [&](int t, int st, int k0, int k1, bool add) {
        const uint64_t v0 = v_desc + st * kTileStep;
#pragma unroll
        for (int k = k0; k < k1; ++k)
          mma_ts(tmem + 256 + D * t, tmem + 128 * t + 8 * k, v0 + k * (2048 >> 4), kPv, add || k > 0);
      };
      auto active = [&](int t, int i) {
        return t ? i >= tile_from[1] && i < tile_to[1] : i >= tile_from[0] && i < tile_to[0];
      };
      mbar_wait(&sh, bar(kKFull), 0);
      mbar_wait(&sh, bar(kQFull), 0);
      mbar_wait(&sh, bar(kQFull + 1), 0);
      tc_fence_after();
      if (elect_one()) {
        for (int t = 0; t < 2; ++t)
          if (active(t, 0)) qk(t, 0);
        tc_commit(bar(kKEmpty));
      }
      __syncwarp();
      // One warp issues for both tiles, in turn: with a warp each their MMAs
      // mix and both tiles wait for both (631 us instead of 502 for 4 x 2048
      // rows over 8192).
      for (int i = 0; i < steps; ++i) {
        const int st = i & 1, nst = st ^ 1;
        const bool more = i + 1 < steps;
        mbar_wait(&sh, bar(kVFull + st), (i >> 1) & 1);
        if (more) mbar_wait(&sh, bar(kKFull + nst), ((i + 1) >> 1) & 1);
        tc_fence_after();
        for (int t = 0; t < 2; ++t) {
          const bool now = active(t, i), next = more && active(t, i + 1);
          const int from = t ? tile_from[1] : tile_from[0];
          if (now) {
            const uint32_t parity = (i - from) & 1;
            mbar_wait(&sh, bar(kPFull + 2 * t), parity);
            tc_fence_after();
            if (elect_one()) pv(t, st, 0, kTokens / 32, i > from);
            __syncwarp();
            mbar_wait(&sh, bar(kPFull + 2 * t + 1), parity);
            tc_fence_after();
          }
          if (elect_one()) {
            if (now) pv(t, st, kTokens / 32, kTokens / 16, true);
            if (now && !next) tc_commit(bar(kOFull + t));
            if (next) qk(t, nst);
            // (not behind the last step: no one waits for those, and an arrival
            // could then come after the CTA's end)
            if (t == 1 && more) {
              tc_commit(bar(kVEmpty + st));
              tc_commit(bar(kKEmpty + nst));
            }
          }
          __syncwarp();
        }
      }
      // nothing of this CTA's is in flight when it ends
      for (int t = 0; t < 2; ++t) {
        if (t ? tile_to[1] > tile_from[1] : tile_to[0] > tile_from[0]) {
          mbar_wait(&sh, bar(kOFull + t), 0);
          mbar_drain(bar(kOFull + t), 0);
        }
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Adds up the splits of an item: a warp a row, at most 32 splits.
constexpr int kJoinRows = 8;

template <int D>
__global__ void __launch_bounds__(32 * kJoinRows) kv_prompt_join_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = D / 4;  // of a row; D = 64: half warps take every other split
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x, in_item = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
  const int per_block = p.a.batch * p.a.c.kv_heads;
  const int rb = p.row_blocks - 1 - item / per_block, bh = item % per_block;
  const int b = bh / p.a.c.kv_heads, h = bh % p.a.c.kv_heads;
  const Span s = span_of(p, b);
  const int rows = s.lq * p.group, row = rb * kRows + in_item;
  if (rows <= p.rows_limit || row >= rows) return;
  auto at = [&](int split) { return (static_cast<int64_t>(item) * p.splits + split) * kRows + in_item; };
  const float2 ml = lane < p.splits ? *split_ml_at(p, at(lane)) : make_float2(-INFINITY, 0.0f);
  float m = ml.x;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  // splits that saw no token are left out, but none whose weight is 0 in 32
  // bits: 0 times the NaN of a V that the row sees is NaN
  const uint32_t saw = __ballot_sync(0xFFFFFFFFu, ml.x != -INFINITY);
  const float z = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - m);
  float l = z * ml.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  const int el = lane % kLanes, half = lane / kLanes;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i0 = 0; i0 < p.splits; i0 += 32 / kLanes) {
    const int i = i0 + half;
    const float zi = __shfl_sync(0xFFFFFFFFu, z, i & 31);
    if (i < p.splits && (saw >> i) & 1) {
      const float4 v = *split_o_at<D>(p, at(i), 4 * el);
      acc.x += zi * v.x, acc.y += zi * v.y, acc.z += zi * v.z, acc.w += zi * v.w;
    }
  }
  if constexpr (kLanes == 16) {
    acc.x += __shfl_xor_sync(0xFFFFFFFFu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xFFFFFFFFu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xFFFFFFFFu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xFFFFFFFFu, acc.w, 16);
  }
  if (half == 0) write_row(p, s, h, row, 4 * el, acc, l == 0.0f ? 0.0f : head_S(p, p.a.c.v_S, h) / l);
  if (lane == 0) write_lse(p, s, h, row, m, l);
}

template <int D>
cudaError_t run_prompt(const Params& p, cudaStream_t stream) {
  constexpr int smem = Layout<D>::kBytes + 1024;
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in.set(reinterpret_cast<const void*>(&kv_prompt_kernel<D>), smem);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(p.row_blocks) * p.a.batch * p.a.c.kv_heads;
  kv_prompt_kernel<D><<<static_cast<unsigned>(items * p.splits), kPromptThreads, smem, stream>>>(p);
  const cudaError_t r = cudaGetLastError();
  if (r != cudaSuccess || p.splits == 1) return r;
  kv_prompt_join_kernel<D><<<dim3(static_cast<unsigned>(items), kRows / kJoinRows), 32 * kJoinRows, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Splits of an item's steps: where a call has fewer items than SMs, each is
// given to several CTAs.  The number with the shortest estimate, in steps of
// 256 rows by 128 tokens (1.7 us at head_dim 128): every wave of CTAs takes its
// share of steps and about 4 more to start and finish; partial results cost
// about 2 a wave's worth of them, and the joining kernel 3.  One sequence of 64
// new tokens over 32000, 64 / 8 heads of 128, takes 75 us so and 428 unsplit.
// The host knows bounds alone, so items are max_q rows of every sequence: those
// that turn out empty still cost about half a microsecond of an SM each, and
// count as items here (255 single tokens over 4000 beside a chunk of 2048, 32 / 8
// heads, 1117 us, apart 223 and 114; 63 beside that one sequence 602, apart 68
// and 75).
PromptPlan prompt_plan(int64_t batch, int64_t rows, int64_t max_kv, int kv_heads, int num_sms) {
  PromptPlan best{};
  best.row_blocks = (rows + kRows - 1) / kRows;
  best.items = best.row_blocks * batch * kv_heads;
  best.splits = 1;
  const int64_t steps = (max_kv + kTokens - 1) / kTokens;
  double least = 0.0;
  for (int n = 1; n <= 32 && (n == 1 || (best.items * n <= 4 * num_sms && steps >= 2 * n)); ++n) {
    const double waves = static_cast<double>((best.items * n + num_sms - 1) / num_sms);
    double cost = waves * (static_cast<double>((steps + n - 1) / n) + 4.0);
    if (n > 1) cost += 3.0 + 2.0 * static_cast<double>(best.items * n) / num_sms;
    if (n == 1 || cost < least) {
      least = cost;
      best.splits = n;
    }
  }
  return best;
}

size_t prompt_workspace_bytes(const PromptPlan& plan, int head_dim) {
  return plan.splits == 1 ? 0 : static_cast<size_t>(plan.items) * plan.splits * kRows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_prompt(Params& p, const PromptPlan& plan, void* workspace, cudaStream_t stream) {
  p.row_blocks = static_cast<int>(plan.row_blocks);
  p.splits = plan.splits;
  p.split_o = static_cast<float*>(workspace);
  p.split_ml = reinterpret_cast<float2*>(p.split_o + plan.items * plan.splits * kRows * p.a.c.head_dim);
  return p.a.c.head_dim == 128 ? run_prompt<128>(p, stream) : run_prompt<64>(p, stream);
}

// False where the limit is built in.
bool kv_wait_limit(long long cycles, cudaError_t* e) {
#ifdef NVFP4HS_CHECKS
  *e = cudaMemcpyToSymbol(g_wait_limit, &cycles, sizeof(cycles));
  return true;
#else
  (void)cycles;
  *e = cudaSuccess;
  return false;
#endif
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
