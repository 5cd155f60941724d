// The cache attention for many rows of one sequence and key/value head
// (prompt chunks, drafted tokens): the mathematics of attn_x8.cuh with both
// products on the 5th-generation tensor cores, rows on the MMA's M side (up to
// two tiles of 128 per CTA, each row one TMEM lane and one softmax thread).
//
//  S[128 x 64] = Q K^T, kind::f8f6f4: K straight from the cache's image (it is
//    the 128-byte, for D = 64 the 64-byte, swizzled operand), q as hi + lo of
//    two E4M3 values after a power-of-two scale per row: bf16 has 8 significant
//    bits, hi takes 4 and the remainder fits lo's, exactly down to 2^-10 of the
//    row's largest value and within 2^-18 of it below.
//  O[128 x D] += P V, kind::f16: P in f16, written over its scores in TMEM
//    (the A operand); V converted to f16 (exact) into a shared tile once per
//    page for both row tiles. O stays in TMEM for the whole item.
//  The weights are held relative to a reference per row, p = 2^7 exp(s - ref),
//    ref the maximum of the row's first page: while later maxima stay within
//    2^8 of it nothing is rescaled; beyond that, the row's O and sum are scaled
//    down once (its thread reads and writes its TMEM lane). f16 holds 2^15, and
//    11 bits down to 2^-21 of the reference.
//  The page's value scale goes into P relative to one that each row keeps: that
//    of the last page that was louder, or more than 2^8 quieter, than the one
//    before it; O is scaled to it in the same way, down or up, as far as fp32
//    holds the sum so far. P's halvings are exact while f16 holds the bits: a
//    weight on a page 2^-k as loud (k <= 8) keeps 11 bits down to 2^(k - 21) of
//    the reference. Pages of which a row sees nothing, or gives all tokens less
//    weight than f16 holds, do not count: a scale there touches no row.
//
// Masked tokens: scores are replaced; a value byte that is NaN becomes 0 in the
// shared tile, and the rows that see its token are made NaN (in all dims) at the
// item's end, so an unwritten or masked place touches nobody.
//
// Bound by the tensor cores' operand reads. Per page and tile of D = 128 the
// scores are 8 products of 64 x 32 and the values 4 of 128 x 16; with two
// issuers one of the first takes 61 cycles (its 6 KB of shared-memory operands
// at about 100 bytes a cycle; 33 by the peak rate) and one of the second 70:
// 770 cycles, the softmax about 1000 beside it. mma.sync on the same work takes
// 142 cycles for every 8 rows and converts K and V once per 16 rows: 238 us
// where this takes 54 (48 query tokens over 32k, 8 heads with 5 query heads
// each), 66 where it takes 36 (6 sequences of 8 tokens over 3k to 8k). Of the
// 54 us about 28 are the pages (27 a CTA, 2050 cycles each), 3.5 the start, 5
// more pass to the first scores, 4 are the output, the rest the join of 19 parts.
//
// Row groups of more than 128 rows fill both tiles, and every page goes to both.
// Smaller ones have one tile of rows: its two softmax groups take the pages in
// turn, each with sums of its own that are joined at the item's end (the
// softmax is the longer part of a page).
//
// Warps: 0 and 1 issue the MMAs of the two tiles, 2 fills the ring of page
// slots (issuing a page's copy takes its thread ~670 cycles), 3 converts the
// values, 4-7 and 8-11 are the softmax groups. (More warps would leave 128
// registers a thread instead of 168: the softmax spills, and the little L1
// beside the shared memory does not hold the spills.)
#pragma once

#include "attn_x8.cuh"

namespace moe {
namespace attn {

constexpr float kLog2PWide = 7.0f;
constexpr float kUnPWide = 0x1p-15f;  // of O read out: P's scale, and the headroom, which fp32 has not for the largest values
constexpr float kHeadroom = 8.0f;  // how far above the reference a row's scores may rise (log2)
constexpr float kNothing = 33.0f;  // below the reference by more: weights under 2^(7 - 33), 0 in f16
constexpr int kQuieter = 8;        // value codes by which P is scaled down before O is scaled up instead
// Pages that some rows of a group see whole or in part and others do not: its
// positions span at most 255 tokens, so causality cuts 5 pages, the window's
// start 5 and the sinks' end one.
constexpr int kNanPages = 11;

template <int D>
struct WideCfg {
  static constexpr int kThreads = 384;
  static constexpr int kConverters = 1;  // warp 3
  static constexpr int kV16Bufs = 3;
  static constexpr int kRows = 256;
  static constexpr uint32_t kHalf = kPageTokens * D;
  static constexpr uint32_t kPage = 2 * kHalf;
  static constexpr uint32_t kQTile = 128 * D;            // one E4M3 tile of 128 rows
  static constexpr uint32_t kV16 = D * kPageTokens * 2;  // f16 values of a page
  static constexpr int kSlots = 98304 / kPage;           // 6 (D = 128), 12 (D = 64)
  static constexpr uint32_t kOffQ = 0;                   // [tile][hi, lo]
  static constexpr uint32_t kOffPages = kOffQ + 4 * kQTile;
  static constexpr uint32_t kOffV16 = kOffPages + kSlots * kPage;
  static constexpr uint32_t kOffBar = kOffV16 + kV16Bufs * kV16;
  static constexpr uint32_t kOffMisc = kOffBar + 512;
  static constexpr uint32_t kOffXchg = kOffMisc + 768;   // [128 rows] {ref, sum, value scale, -}
  // [segment & 1][256 rows] raw score -> log2 units (keys' scale apart). Two
  // buffers: a segment's rows may be made while a softmax warp has yet to read
  // its factor of the one before (q_free follows the score products alone), but
  // not before every softmax warp made the rows of that one, which it does
  // behind its read of the factor two before.
  static constexpr uint32_t kOffFactor = kOffXchg + 2048;
  static constexpr uint32_t kSmem = kOffFactor + 2048 + 1024;  // slack for aligning the base to 1024
  static_assert(kSmem <= 232448, "shared memory");
};

// ---------------------------------------------------------------- tcgen05 forms
// Has the phase of that parity completed? (does not wait)
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes)
      : "r"(bar), "r"(parity)
      : "memory");
  return yes != 0;
}

// D[128 x N] (+)= A . B^T over K = 32 E4M3 values, both from shared memory.
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// D[128 x N] (+)= A . B^T over K = 16 f16 values, A from TMEM.
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Instruction descriptor: fp32 accumulators, A and B K-major of format 0 (E4M3
// for kind::f8f6f4, f16 for kind::f16), M = 128.
__host__ __device__ constexpr uint32_t idesc_dense(uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// K-major operand tile of 64-byte rows (64-byte swizzle, 8-row atoms of 512 B).
__device__ __forceinline__ uint64_t sdesc_k64_sw64(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(4) << 61);
}

template <int D>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr) {
  return D == 64 ? sdesc_k64_sw64(saddr) : ptx::sdesc_k128_sw128(saddr);
}

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two f16 values as two E4M3 bytes (to nearest even, NaN stays) and back.
__device__ __forceinline__ uint32_t f16x2_e4m3(uint32_t x) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ __half2 e4m3x2_f16(uint32_t x) {
  uint32_t y;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(static_cast<uint16_t>(x)));
  return *reinterpret_cast<const __half2*>(&y);
}

// The tokens t0 .. t0 + 63 that a row at position `at` sees, as bits.
__device__ __forceinline__ unsigned long long seen_tokens(const AttnX8Params& p, int t0, int at) {
  const auto below = [&](int t) {  // the tokens before t
    const int n = t - t0;
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
  };
  unsigned long long m = below(at + 1);
  if (p.window > 0) m &= ~below(at - p.window + 1) | below(p.sinks);
  return m;
}

// A page's values from E4M3 to the f16 operand tile, by one warp. kNan: NaN
// bytes become 0, and the tokens of this lane's are returned.
template <int D, bool kNan>
__device__ __forceinline__ unsigned long long values_to_f16(const uint8_t* src, uint8_t* dst, int lane) {
  unsigned long long tokens = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < 4; c0 += 2) {  // 16 tokens of D dims, two at a time
    uint32_t x[2][D / 32][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int d = lane + 32 * i;
        const uint4 w = *reinterpret_cast<const uint4*>(src + d * kPageTokens + (((c0 + h) ^ ((d >> 1) & 3)) << 4));
        x[h][i][0] = w.x;
        x[h][i][1] = w.y;
        x[h][i][2] = w.z;
        x[h][i][3] = w.w;
      }
    if (kNan) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t hits = 0;  // 0x80 in the bytes whose low 7 bits are all set
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t hit = ((x[h][i][k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            x[h][i][k] &= ~((hit >> 7) * 0xFFu);
            hits |= hit;
          }
          // word k: tokens 2 k, 2 k + 1, 2 k + 8, 2 k + 9 of the chunk
          const unsigned long long bits =
              ((hits >> 7) & 1u) | ((hits >> 14) & 2u) | ((hits >> 15) & 0x100u) | ((hits >> 22) & 0x200u);
          tokens |= bits << ((c0 + h) * 16 + 2 * k);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int d = lane + 32 * i, c = c0 + h;
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) e4m3x4_f16(x[h][i][k], lo[k], hi[k]);
        uint8_t* row = dst + d * 128;
        *reinterpret_cast<uint4*>(row + (((2 * c) ^ (d & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (d & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
  }
  return tokens;
}

// Barriers (8 bytes each, from kOffBar). Every waiter of a barrier either waits
// for each of its phases in turn or is known to come no more than one phase
// late: the page c of a tile uses buffer c % 2, and scores of page c are only
// issued when the value product of page c - 2 is done, so whoever has seen the
// scores of page c may wait for the product of page c - 1 or c.
struct WideBars {
  uint64_t full[12];       // page slot: the copy
  uint64_t empty[12];      // page slot: both MMA warps (scores done) and the converters
  uint64_t v16_full[3];    // f16 values: the converters
  uint64_t v16_empty[3];   // both MMA warps (products done)
  uint64_t q_full;         // the rows' operands: softmax and converter warps
  uint64_t q_free;         // ... have been used: both MMA warps (scores done)
  uint64_t s_full[2][2];   // [tile][buffer] scores (commit)
  uint64_t p_full[2][2];   // [tile][buffer] weights: 4 warps
  uint64_t pv_done[2][2];  // [tile][buffer] a page's value product (commit, and the issuer's list)
  uint64_t o_free[2];      // [tile] O read out: 4 warps
  uint64_t b_done;         // tile 1's part of shared rows is complete: its 4 warps
  uint64_t x_free;         // ... and has been taken: tile 0's 4 warps
  uint64_t drain[2];       // the MMA threads' last commits
};
static_assert(sizeof(WideBars) <= 512, "barrier area");

struct WideMisc {
  Shared shared[2];
  Walk walk;  // the CTA's run, found by warp 0
  int per, parts, work;
  uint32_t tmem;
  int abort;
  int id[12];                        // [slot] the page, or -1
  unsigned long long nan_tokens[3];  // [buffer] tokens with a NaN value byte
  // [tile] this item part's cut pages with NaN values: page index and tokens
  int nan_count[2];
  int nan_page[2][kNanPages];
  unsigned long long nan_list[2][kNanPages];
};
static_assert(sizeof(WideMisc) <= 768, "misc area");

template <int D>
__global__ void __launch_bounds__(WideCfg<D>::kThreads, 1) attn_wide_kernel(const AttnX8Params p) {
  using C = WideCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - (ptx::smem_u32(smem_raw) & 1023)) % 1024;
  const uint32_t sbase = ptx::smem_u32(smem);
  WideBars* bars = reinterpret_cast<WideBars*>(smem + C::kOffBar);
  WideMisc* misc = reinterpret_cast<WideMisc*>(smem + C::kOffMisc);
  volatile int* abort = &misc->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      ptx::mbar_init(bar(bars->full[i]), 1);
      ptx::mbar_init(bar(bars->empty[i]), 2 + C::kConverters);
    }
    for (int i = 0; i < C::kV16Bufs; ++i) {
      ptx::mbar_init(bar(bars->v16_full[i]), C::kConverters);
      ptx::mbar_init(bar(bars->v16_empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) {
        ptx::mbar_init(bar(bars->s_full[i][j]), 1);
        ptx::mbar_init(bar(bars->p_full[i][j]), 4);
        ptx::mbar_init(bar(bars->pv_done[i][j]), 2);
      }
      ptx::mbar_init(bar(bars->o_free[i]), 4);
      ptx::mbar_init(bar(bars->drain[i]), 1);
      misc->shared[i].c1 = -1;
    }
    ptx::mbar_init(bar(bars->q_full), 8 + C::kConverters);
    ptx::mbar_init(bar(bars->q_free), 2);
    ptx::mbar_init(bar(bars->b_done), 4);
    ptx::mbar_init(bar(bars->x_free), 4);
    ptx::fence_mbar_init();
    misc->abort = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(&misc->tmem), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc->tmem;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  if (warp == 0) {
    Walk w;
    int per, parts;
    const bool work = find_run<C::kRows, 1>(p, 2, lane, warp, w, per, parts);
    if (lane == 0) {
      misc->walk = w;
      misc->per = per;
      misc->parts = parts;
      misc->work = work;
    }
  }
  __syncthreads();
  Walk walk = misc->walk;
  const int per = misc->per, parts = misc->parts;
  const bool work = misc->work != 0;
  bool ok = true;  // (per warp; in the MMA warps, of the thread that issues)
  // a wait by all lanes; on a failure the CTA's roles give up one after another
  const auto wait = [&](uint64_t& b, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_wait(bar(b), parity & 1, abort))) return true;
    if (p.status) atomicOr(p.status, kKvErrTimeout);
    return false;
  };
  // the segment's row tiles
  const auto tiles_of = [&](const Walk& k) { return k.s.n * p.group - k.group * C::kRows > 128 ? 2 : 1; };
  // The rows' operands of a segment, by the softmax and converter warps: hi and
  // lo E4M3 parts of q 2^a, the largest value of a row in [128, 256), in the
  // MMA's layout, and the rows' factors. Four lanes take a row, 8 dims at a
  // time (what a row needs once is shared by 32 of its values: with 16 lanes a
  // row this took 5.6 us for 240 rows, now 3.1). hi is x rounded to 4 significant
  // bits and lo the rest, off by at most 2^-10; the f16 between is exact for all
  // that neither rounds away. A row with an infinity or NaN becomes NaN.
  const auto make_rows = [&](const Walk& k, int who, int seg) {
    if (seg > 0 && !wait(bars->q_free, seg - 1)) return false;
    constexpr int kPer = 8, kChunks = D / 32, kMakers = 8 + C::kConverters, kBatch = 2;
    const int sub = lane >> 2, l4 = lane & 3;
    const int rows = k.s.n * p.group, row0 = k.group * C::kRows, count = min(rows - row0, C::kRows);
    float* factors = reinterpret_cast<float*>(smem + C::kOffFactor) + (seg & 1) * C::kRows;
    const __nv_bfloat16* base = p.q + k.s.q0 * p.ldq + static_cast<long long>(k.head * p.group) * D + l4 * 8;
    for (int i0 = who * kPer; i0 < count; i0 += kBatch * kMakers * kPer) {
      uint4 v[kBatch][kChunks];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int lr = i0 + i * kMakers * kPer + sub;
        const int rr = row0 + min(lr, count - 1), token = by_group(p, rr);
        const __nv_bfloat16* src = base + token * p.ldq + (rr - token * p.group) * D;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) v[i][c] = __ldg(reinterpret_cast<const uint4*>(src + c * 32));
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (i0 + i * kMakers * kPer >= count) break;
        const int lr = i0 + i * kMakers * kPer + sub;
        // the largest magnitude as bf16 bits
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i][c].x & 0x7FFF7FFFu, v[i][c].y & 0x7FFF7FFFu),
                                       __vmaxu2(v[i][c].z & 0x7FFF7FFFu, v[i][c].w & 0x7FFF7FFFu)));
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = static_cast<int>(max(top >> 16, top & 0xFFFFu) >> 7);
        const int a = top != 0 ? min(134 - e, 126) : 0;
        const float mul = __uint_as_float(e == 255 ? 0x7FC00000u : static_cast<uint32_t>(127 + a) << 23);
        const int row = lr & 127, turn = D >= 128 ? (row & 7) : ((row >> 1) & 3);
        uint8_t* dst = smem + C::kOffQ + 2 * (lr >> 7) * C::kQTile + row * D + (l4 & 1) * 8;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const uint32_t w[4] = {v[i][c].x, v[i][c].y, v[i][c].z, v[i][c].w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t x = pack_f16(__uint_as_float(w[j] << 16) * mul, __uint_as_float(w[j] & 0xFFFF0000u) * mul);
            hi[j] = f16x2_e4m3(x);
            const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&x), e4m3x2_f16(hi[j]));
            lo[j] = f16x2_e4m3(*reinterpret_cast<const uint32_t*>(&rest));
          }
          if (lr < count) {
            uint8_t* at = dst + (((2 * c + (l4 >> 1)) ^ turn) << 4);
            *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(at + C::kQTile) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          }
        }
        if (l4 == 0 && lr < count) factors[lr] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (elect_one()) ptx::mbar_arrive(bar(bars->q_full));
    return true;
  };

  if (work && warp < 2) {
    // ------------------------------------------------------------ MMA issuer of tile t
    // One thread. It goes through every page twice, for the scores (up to two
    // pages of its own ahead) and for the value products, and issues whichever
    // is ready, value products first; pages of the other tile alone it only
    // releases.
    const int t = warp;
    if (elect_one()) {
      const auto wait1 = [&](uint64_t& b, uint32_t parity) {
        if (mbar_wait(bar(b), parity & 1, abort)) return true;
        if (p.status) atomicOr(p.status, kKvErrTimeout);
        return false;
      };
      const auto ready = [&](uint64_t& b, uint32_t parity) { return mbar_test(bar(b), parity & 1); };
      const uint32_t tile = tmem + t * 256;
      int slot = 0, vb = 0, seg = 0;
      uint32_t slot_phase = 0, v_phase = 0;
      int c_s = 0, c_v = 0;  // own pages: scores issued, value products issued
      Walk k = walk;
      while (ok && next_segment<C::kRows>(p, k)) {
        const bool split = tiles_of(k) == 1;
        const int pages = k.last - k.first;
        const uint32_t qb = sbase + C::kOffQ + (split ? 0 : 2 * t * C::kQTile);
        ok = wait1(bars->q_full, seg);
        ptx::tc_fence_after();
        bool first = true;     // no value product in this segment yet
        int si = 0, vi = 0;    // pages whose scores, whose value products are issued (or the other tile's)
        uint32_t polls = 0;
        long long since = 0;
        while (ok && (vi < pages || si < pages)) {
          bool moved = false;
          if (vi < pages && ready(bars->v16_full[vb], v_phase)) {
            const bool own = !split || (vi & 1) == t;
            bool taken = !own;
            if (own && ready(bars->p_full[t][c_v & 1], c_v >> 1)) {
              if (first) {
                if (seg > 0 && !wait1(bars->o_free[t], seg - 1)) {
                  ok = false;
                  break;
                }
                misc->nan_count[t] = 0;
              }
              const unsigned long long nan = misc->nan_tokens[vb];
              if (nan != 0) {
                const int at = misc->nan_count[t];
                misc->nan_page[t][at] = k.first + vi;
                misc->nan_list[t][at] = nan;
                misc->nan_count[t] = at + 1;
              }
              ptx::tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kPageTokens / 16; ++kk)
                tc_mma_f16_ta(tile + 128, tile + (c_v & 1) * 64 + 8 * kk,
                              ptx::sdesc_k128_sw128(sbase + C::kOffV16 + vb * C::kV16 + 32 * kk), idesc_dense(D),
                              !first || kk != 0);
              ptx::tc_commit(bar(bars->pv_done[t][c_v & 1]));
              ptx::mbar_arrive(bar(bars->pv_done[t][c_v & 1]));
              ptx::tc_commit(bar(bars->v16_empty[vb]));
              ++c_v;
              first = false;
              taken = true;
            } else if (!own) {
              ptx::mbar_arrive(bar(bars->v16_empty[vb]));
            }
            if (taken) {
              moved = true;
              ++vi;
              if (++vb == C::kV16Bufs) {
                vb = 0;
                v_phase ^= 1;
              }
            }
          }
          if (si < pages && ready(bars->full[slot], slot_phase)) {
            const bool own = !split || (si & 1) == t;
            // (the weights that lie where the scores go were read)
            const bool room = c_s < 2 || (c_s < c_v + 2 && ready(bars->pv_done[t][c_s & 1], (c_s - 2) >> 1));
            if (own && room) {
              ptx::tc_fence_after();
              const uint32_t kb = sbase + C::kOffPages + slot * C::kPage;
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  tc_mma_f8(tile + (c_s & 1) * 64, sdesc_rows<D>(qb + h * C::kQTile + 32 * kk),
                            sdesc_rows<D>(kb + 32 * kk), idesc_dense(kPageTokens), h != 0 || kk != 0);
              ptx::tc_commit(bar(bars->s_full[t][c_s & 1]));
              ptx::tc_commit(bar(bars->empty[slot]));
              ++c_s;
            } else if (!own) {
              ptx::mbar_arrive(bar(bars->empty[slot]));
            }
            if (!own || room) {
              ++si;
              if (si == pages) ptx::tc_commit(bar(bars->q_free));
              if (++slot == C::kSlots) {
                slot = 0;
                slot_phase ^= 1;
              }
              moved = true;
            }
          }
          if (moved) {
            polls = 0;
          } else if (++polls == 1) {
            since = clock64();
          } else if ((polls & 63) == 0) {
            if (*abort || clock64() - since > kWaitClocks) {
              *abort = 1;
              if (p.status) atomicOr(p.status, kKvErrTimeout);
              ok = false;
              break;
            }
          }
        }
        if (ok && first && seg > 0) ok = wait1(bars->o_free[t], seg - 1);  // (every phase is waited for)
        ++seg;
      }
      // everything this thread issued has completed once drain fires
      ptx::tc_commit(bar(bars->drain[t]));
      const uint64_t t0 = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(bar(bars->drain[t]), 0) && ptx::globaltimer_ns() - t0 < kWaitLimitNs) {
      }
    }
    __syncwarp();
  } else if (work && warp == 2) {
    // ------------------------------------------------------------ page slots
    int n = 0, slot = 0, round = 0;
    while (ok && next_segment<C::kRows>(p, walk)) {
      int ids = -1;
      for (int j = walk.first; j < walk.last; ++j) {
        const int k = (j - walk.first) & 31;
        if (k == 0) {  // the next 32 page ids, one per lane
          ids = -1;
          if (j + lane < walk.last && walk.s.kv > 0) {
            const int t = j + lane;
            const int index = t < walk.s.sink_pages ? t : walk.s.lo + (t - walk.s.sink_pages);
            ids = __ldg(p.page_table + static_cast<size_t>(walk.b) * p.max_pages + index);
            if (ids < 0 || ids >= p.pages) {
              ids = -1;
              if (p.status) atomicOr(p.status, kKvErrPage);
            }
          }
        }
        const int id = __shfl_sync(0xffffffffu, ids, k);
        if (round > 0 && !wait(bars->empty[slot], round - 1)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          misc->id[slot] = id;
          if (id < 0) {  // stale bytes: every row masks the page
            ptx::mbar_arrive(bar(bars->full[slot]));
          } else {
            ptx::mbar_arrive_expect_tx(bar(bars->full[slot]), C::kPage);
            ptx::bulk_load(sbase + C::kOffPages + slot * C::kPage,
                           p.blocks + (static_cast<size_t>(id) * p.kv_heads + walk.head) * C::kPage, C::kPage,
                           bar(bars->full[slot]));
          }
        }
        __syncwarp();
        ++n;
        if (++slot == C::kSlots) {
          slot = 0;
          ++round;
        }
      }
    }
    // the copies in flight land before the CTA's shared memory goes (in a run
    // without errors all of them are consumed)
    for (int i = 0; i < C::kSlots && i < n; ++i) {
      const int fills = (n - i + C::kSlots - 1) / C::kSlots;
      const uint64_t t0 = ptx::globaltimer_ns();
      while (!ptx::mbar_try_wait(bar(bars->full[i]), (fills - 1) & 1) &&
             ptx::globaltimer_ns() - t0 < kWaitLimitNs / 8) {
      }
    }
  } else if (work && warp == 3) {
    // ------------------------------------------------------------ values to f16
    int slot = 0, vb = 0, round = 0;
    uint32_t phase = 0;
    for (int seg = 0; ok && next_segment<C::kRows>(p, walk); ++seg) {
      ok = make_rows(walk, 8, seg);
      const int row0 = walk.group * C::kRows, rows = walk.s.n * p.group;
      const int pos_lo = walk.s.kv - walk.s.n + by_group(p, row0);
      const int pos_hi = walk.s.kv - walk.s.n + by_group(p, min(row0 + C::kRows, rows) - 1);
      for (int j = walk.first; j < walk.last && ok; ++j) {
        if (!wait(bars->full[slot], phase) || (round > 0 && !wait(bars->v16_empty[vb], round - 1))) {
          ok = false;
          break;
        }
        const uint8_t* src = smem + C::kOffPages + slot * C::kPage + C::kHalf;
        uint8_t* dst = smem + C::kOffV16 + vb * C::kV16;
        // A NaN goes the way of any value on pages that every row sees whole.
        // On others its byte becomes 0 and its token is noted.
        const int t0 = (j < walk.s.sink_pages ? j : walk.s.lo + (j - walk.s.sink_pages)) * kPageTokens;
        const int id = misc->id[slot];
        unsigned long long tokens = 0;
        const int kind = id < 0 ? 0 : page_kind(p, t0, t0 + kPageTokens - 1, pos_lo, pos_hi);
        if (kind == 1) {
          values_to_f16<D, false>(src, dst, lane);
        } else {
          tokens = values_to_f16<D, true>(src, dst, lane);
          const unsigned lo = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(tokens));
          const unsigned hi = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(tokens >> 32));
          tokens = kind == 0 ? 0 : (static_cast<unsigned long long>(hi) << 32) | lo;
        }
        if (lane == 0) misc->nan_tokens[vb] = tokens;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
          ptx::mbar_arrive(bar(bars->empty[slot]));
          ptx::mbar_arrive(bar(bars->v16_full[vb]));
        }
        if (++slot == C::kSlots) {
          slot = 0;
          phase ^= 1;
        }
        if (++vb == C::kV16Bufs) {
          vb = 0;
          ++round;
        }
      }
    }
  } else if (work && warp >= 4) {
    // ------------------------------------------------------------ softmax: a row per thread
    const int t = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t mine = tmem + t * 256 + lanes, o_cols = mine + 128;
    float4* xchg = reinterpret_cast<float4*>(smem + C::kOffXchg);
    int c = 0;       // pages of this tile
    int splits = 0;  // segments that both tiles shared
    for (int seg = 0; ok && next_segment<C::kRows>(p, walk); ++seg) {
      const Seq s = walk.s;
      const int pages = walk.last - walk.first;
      const bool split = tiles_of(walk) == 1;
      const int rows = s.n * p.group, row0 = walk.group * C::kRows;
      const int lr = (split ? 0 : t * 128) + quarter * 32 + lane;  // row in the group
      const int r = row0 + lr;
      const int pos = s.kv - s.n + by_group(p, min(r, rows - 1));  // rows past the last repeat it
      const int pos_lo = __shfl_sync(0xffffffffu, pos, 0), pos_hi = __shfl_sync(0xffffffffu, pos, 31);
      const bool idle = r - lane >= rows;  // no row of this warp

      // the ids and then the codes of the next 32 pages, one per lane
      const auto page_id = [&](int j) {
        if (j >= walk.last || s.kv == 0) return -1;
        const int index = j < s.sink_pages ? j : s.lo + (j - s.sink_pages);
        return __ldg(p.page_table + static_cast<size_t>(walk.b) * p.max_pages + index);
      };
      const auto page_codes = [&](int id) {
        if (id < 0 || id >= p.pages) return -1;
        return static_cast<int>(__ldg(reinterpret_cast<const unsigned short*>(p.codes) +
                                      static_cast<size_t>(id) * p.kv_heads + walk.head));
      };
      const int id32 = page_id(walk.first + lane);
      if (!make_rows(walk, warp - 4, seg)) {
        ok = false;
        break;
      }
      int codes32 = page_codes(id32);
      if (!wait(bars->q_full, seg)) {
        ok = false;
        break;
      }
      const float factor =
          r < rows ? reinterpret_cast<const float*>(smem + C::kOffFactor)[(seg & 1) * C::kRows + lr] : 0.0f;

      float ref = -INFINITY, l = 0.0f;
      int vref = -1;      // the value code that the row's P and O are relative to (-1: O is 0)
      float most = 0.0f;  // a bound: |O| <= 448 most
      int own = 0;        // pages of this segment taken
      for (int i = 0; i < pages; ++i) {
        if (i > 0 && (i & 31) == 0) codes32 = page_codes(page_id(walk.first + i + lane));
        if (split && (i & 1) != t) continue;
        const int codes = __shfl_sync(0xffffffffu, codes32, i & 31);
        const int j = walk.first + i;
        const int t0 = (j < s.sink_pages ? j : s.lo + (j - s.sink_pages)) * kPageTokens;
        const int kind = codes < 0 || idle ? 0 : page_kind(p, t0, t0 + kPageTokens - 1, pos_lo, pos_hi);
        if (!wait(bars->s_full[t][c & 1], c >> 1)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t s_cols = mine + (c & 1) * 64;
        uint32_t pk[32];
        if (kind == 0) {
#pragma unroll
          for (int k = 0; k < 32; ++k) pk[k] = 0;
        } else {
          uint32_t sc[64];
          tmem_ld_x32(s_cols, sc);
          tmem_ld_x32(s_cols + 32, sc + 32);
          ptx::tmem_wait_ld();
          if (kind == 2) {
            const unsigned long long seen = seen_tokens(p, t0, pos);
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (!((seen >> k) & 1)) sc[k] = 0xFF800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 64; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(sc[k]));
          const float f = fmaxf(factor * e8m0_value(codes & 0xFF), FLT_MIN);  // (never 0: masked scores are -inf)
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
          const int vc = codes >> 8;
          const bool rise = ref != -INFINITY && top > ref + kHeadroom;
          const bool counts = top > fmaxf(ref - kNothing, -FLT_MAX);
          const bool turn = counts && vref >= 0 && (vc > vref || vc < vref - kQuieter);
          if (counts && vref < 0) vref = vc;
          if (__any_sync(0xffffffffu, rise || turn)) {
            // scale O (stable: the last own page's product is done, this one's
            // not begun) and the sum down to the new reference, O to the new
            // value scale (up by what keeps 448 most below 2^111)
            const float w = rise ? ex2(ref - top) : 1.0f;
            int to = vref;
            if (turn) {
              const int room = 228 - static_cast<int>(__float_as_uint(most * w) >> 23);
              to = vc > vref ? vc : max(vc, vref - max(room, 0));
            }
            // (in two factors: 2^(vref - to) may pass fp32's exponents)
            const int by = min(max(vref - to, -126), 126);
            const float w0 = w * __uint_as_float(static_cast<uint32_t>(127 + by) << 23);
            const float w1 = __uint_as_float(static_cast<uint32_t>(max(127 + vref - to - by, 0)) << 23);
            if (own > 0) {
              if (!wait(bars->pv_done[t][(c - 1) & 1], (c - 1) >> 1)) {
                ok = false;
                break;
              }
              ptx::tc_fence_after();
#pragma unroll 1
              for (int d = 0; d < D; d += 32) {
                uint32_t x[32];
                tmem_ld_x32(o_cols + d, x);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * w0 * w1);
                tmem_st_x16(o_cols + d, x);
                tmem_st_x16(o_cols + d + 16, x + 16);
              }
              tmem_wait_st();
            }
            l *= w;
            most = most * w0 * w1;
            if (rise) ref = top;
            vref = to;
          }
          if (ref == -INFINITY) ref = top;  // the row's first visible tokens
          const float shift = kLog2PWide - (ref == -INFINITY ? 0.0f : ref);
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float a = ex2(fmaf(__uint_as_float(sc[2 * k]), f, shift));
            const float b = ex2(fmaf(__uint_as_float(sc[2 * k + 1]), f, shift));
            sum[(2 * k) & 3] += a;
            sum[(2 * k + 1) & 3] += b;
            pk[k] = pack_f16(a, b);
          }
          const float page = (sum[0] + sum[1]) + (sum[2] + sum[3]);
          l += page;
          const float dv = counts && vc != vref ? ex2(static_cast<float>(vc - vref)) : 1.0f;
          most = fmaf(page, dv, most);
          if (dv != 1.0f) {
            const __half2 dv2 = __float2half2_rn(dv);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&pk[k]), dv2);
              pk[k] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
        }
        tmem_st_x16(s_cols, pk);
        tmem_st_x16(s_cols + 16, pk + 16);
        tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(bar(bars->p_full[t][c & 1]));
        ++c;
        ++own;
      }
      if (!ok) break;

      // ---- the part's rows: NaN values seen, the two groups of shared rows
      // joined, then finished or to the workspace
      if (own > 0) {
        if (!wait(bars->pv_done[t][(c - 1) & 1], (c - 1) >> 1)) {
          ok = false;
          break;
        }
        const int nans = misc->nan_count[t];
#pragma unroll 1
        for (int k = 0; k < nans; ++k) {
          const int j = misc->nan_page[t][k];
          const int t0 = (j < s.sink_pages ? j : s.lo + (j - s.sink_pages)) * kPageTokens;
          if (misc->nan_list[t][k] & seen_tokens(p, t0, pos)) l = __int_as_float(0x7FC00000);
        }
      }
      const float vscale = vref < 0 ? 0.0f : e8m0_value(vref) * kUnPWide;
      const bool whole = walk.first == 0 && walk.last == s.pages;
      if (split && t == 1) {
        // tile 0's threads read this one's O and finish the rows
        if (splits > 0 && !wait(bars->x_free, splits - 1)) {
          ok = false;
          break;
        }
        xchg[quarter * 32 + lane] = make_float4(ref, l, vscale, 0.0f);
        ptx::tc_fence_before();
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(bar(bars->b_done));
        ++splits;
        continue;
      }
      float wa = vscale, wb = 0.0f;
      if (split) {
        if (!wait(bars->b_done, splits)) {
          ok = false;
          break;
        }
        const float4 x = xchg[quarter * 32 + lane];
        const float high = fmaxf(ref, x.x), use = high == -INFINITY ? 0.0f : high;
        const float ka = ex2(ref - use), kb = ex2(x.x - use);
        l = l * ka + x.y * kb;
        wa = vscale * ka;
        wb = x.z * kb;
        ref = high;
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(bar(bars->x_free));
        ++splits;
      }
      const bool both = split && pages > 1;  // (of one page tile 1 has no part)
      ptx::tc_fence_after();
      int c0 = 0, c1 = 0;
      if (!whole) item_ctas(walk.item_start, s.pages, per, parts, c0, c1);
      const int part_slot = static_cast<int>(blockIdx.x) == c0;
      float* part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + part_slot) * C::kRows * (D + 2);
      if (!whole && tid == 128) {
        Shared& x = misc->shared[part_slot];
        x.c0 = c0;
        x.c1 = c1;
        x.q0 = s.q0;
        x.rows = rows;
        x.head = walk.head;
        x.row0 = row0;
      }
      const int token = by_group(p, r);
      const size_t at_out = static_cast<size_t>(s.q0 + token) * (p.kv_heads * p.group) +
                            walk.head * p.group + r - token * p.group;
      // (behind the value scale: the two together may leave fp32's exponents)
      const float inv = l == 0.0f ? 0.0f : __frcp_rn(l) * (1.0f / kUnPWide);
#pragma unroll 2
      for (int d = 0; d < D; d += 16) {
        float x[16], y[16];
        ptx::tmem_ld_32x32b_x16(o_cols + d, x);
        if (both) ptx::tmem_ld_32x32b_x16(o_cols + 256 + d, y);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          x[k] *= wa;
          if (both) x[k] = fmaf(y[k], wb, x[k]);
        }
        if (r < rows) {
          if (whole) {
            __align__(16) __nv_bfloat162 z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] = __floats2bfloat162_rn(x[2 * k] * inv, x[2 * k + 1] * inv);
            uint4* dst = reinterpret_cast<uint4*>(p.out + at_out * D + d);
            dst[0] = reinterpret_cast<const uint4*>(z)[0];
            dst[1] = reinterpret_cast<const uint4*>(z)[1];
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<float4*>(part)[(d / 4 + k) * C::kRows + lr] =
                  make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
        }
      }
      if (whole && r < rows && p.lse)
        p.lse[at_out] = l == 0.0f ? -INFINITY : (ref + log2f(l) - kLog2PWide) * 0.69314718055994531f;
      if (!whole && r < rows)
        *reinterpret_cast<float2*>(part + static_cast<size_t>(C::kRows) * D + 2 * lr) = make_float2(ref, l);
      ptx::tc_fence_before();
      __syncwarp();
      if (elect_one()) {
        ptx::mbar_arrive(bar(bars->o_free[t]));
        if (split) ptx::mbar_arrive(bar(bars->o_free[1]));
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (tid == 0) static_cast<Shared*>(p.records)[blockIdx.x] = misc->shared[1];
}

// The rows of items that several CTAs share, joined with the whole GPU behind
// the kernel above (in it, the few CTAs that arrive last would take longer for
// up to 256 rows than all the rest: 110 of 207 us for 240 rows in 19 parts; here
// 9 us by itself, 14 with one group of threads and a grid of blocks by CTA).
// A part holds four dims of all rows after another, then each row's
// {reference, sum}. A unit is kJoinRows rows of an item: four dims of a row per
// thread, neighbouring lanes on neighbouring rows, the item's parts in turn to
// kJoinGroups groups of threads whose sums are joined through shared memory (the
// order of the sums depends on nothing but the parts' number). The blocks take
// units in turn.
constexpr int kJoinThreads = 512, kJoinGroups = 2, kJoinBatch = 5, kJoinBlocks = 2;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_wide_join_kernel(const AttnX8Params p) {
  const int ctas = gridDim.x / kJoinBlocks;  // of the kernel above
  constexpr int kRows = WideCfg<D>::kRows, kMembers = kJoinThreads / kJoinGroups;
  constexpr int kJoinRows = kMembers / (D / 4);
  __shared__ int warp_units[kJoinThreads / 32];
  __shared__ int4 found;  // {record, first row, -, -}
  __shared__ float4 sums[kJoinGroups - 1][kMembers];
  __shared__ float2 tops[kJoinGroups - 1][kMembers];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = tid / kMembers, member = tid % kMembers;
  const int d4 = member / kJoinRows;
  const Shared* records = static_cast<const Shared*>(p.records);
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // where the units of record `tid` begin
  int mine = 0;
  if (tid < ctas && __ldcg(&records[tid].c1) >= 0)
    mine = (min(__ldcg(&records[tid].rows) - __ldcg(&records[tid].row0), kRows) + kJoinRows - 1) / kJoinRows;
  int end = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end += x;
  }
  if (lane == 31) warp_units[warp] = end;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    if (w < warp) end += warp_units[w];
    total += warp_units[w];
  }
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    if (u >= end - mine && u < end) found = make_int4(tid, (u - (end - mine)) * kJoinRows, 0, 0);
    __syncthreads();
    const Shared x = records[found.x];
    const int lr = found.y + member % kJoinRows;
    const bool real = x.row0 + lr < x.rows && lr < kRows;
    float top = -INFINITY, den = 0.0f;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (real) {
      const auto partial = [&](int c) {
        return p.part + (static_cast<size_t>(c) * 2 + (c == x.c0)) * kRows * (D + 2);
      };
      for (int cb = x.c0 + group; cb <= x.c1; cb += kJoinBatch * kJoinGroups) {  // a batch's loads in flight
        float4 y[kJoinBatch];
        float2 t[kJoinBatch];
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) {
          if (cb + k * kJoinGroups > x.c1) break;
          const float* src = partial(cb + k * kJoinGroups);
          y[k] = __ldcg(reinterpret_cast<const float4*>(src) + (d4 * kRows + lr));
          t[k] = __ldcg(reinterpret_cast<const float2*>(src + kRows * D) + lr);
        }
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) {
          if (cb + k * kJoinGroups > x.c1) break;
          const float high = fmaxf(top, t[k].x), use = high == -INFINITY ? 0.0f : high;
          const float keep = ex2(top - use), w = ex2(t[k].x - use);
          top = high;
          den = fmaf(t[k].y, w, den * keep);
          sum.x = fmaf(y[k].x, w, sum.x * keep);
          sum.y = fmaf(y[k].y, w, sum.y * keep);
          sum.z = fmaf(y[k].z, w, sum.z * keep);
          sum.w = fmaf(y[k].w, w, sum.w * keep);
        }
      }
    }
    if (group > 0) {
      sums[group - 1][member] = sum;
      tops[group - 1][member] = make_float2(top, den);
    }
    __syncthreads();
    if (group == 0 && real) {
#pragma unroll
      for (int k = 0; k < kJoinGroups - 1; ++k) {
        const float4 y = sums[k][member];
        const float2 t = tops[k][member];
        const float high = fmaxf(top, t.x), use = high == -INFINITY ? 0.0f : high;
        const float keep = ex2(top - use), w = ex2(t.x - use);
        top = high;
        den = fmaf(t.y, w, den * keep);
        sum.x = fmaf(y.x, w, sum.x * keep);
        sum.y = fmaf(y.y, w, sum.y * keep);
        sum.z = fmaf(y.z, w, sum.z * keep);
        sum.w = fmaf(y.w, w, sum.w * keep);
      }
      store_row<D>(p, x.q0, x.head, x.row0 + lr, d4, sum, top, den, kLog2PWide, 1.0f / kUnPWide);
    }
  }
}

template <int D>
cudaError_t launch_wide(const AttnX8Params& p, int device, int grid, cudaStream_t s) {
  using C = WideCfg<D>;
  static std::atomic<unsigned long long> raised{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (device > 63 || !(raised.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  const cudaError_t e = launch_pdl(attn_wide_kernel<D>, dim3(grid), dim3(C::kThreads), C::kSmem, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_wide_join_kernel<D>, dim3(kJoinBlocks * grid), dim3(kJoinThreads), 0, s, p);
}

}  // namespace attn
}  // namespace moe
