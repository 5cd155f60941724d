// Attention of a step's query rows over the 8-bit paged cache (kv_x8.cuh).
//
// A sequence with kv tokens in the cache has n query rows; row i sits at
// position pos = kv - n + i and sees the tokens j <= pos with j > pos - window
// (window > 0) or j < sinks. Per row: s_j = scale q.k_j, m = max s,
// out = sum exp(s_j - m) v_j / l with l = sum exp(s_j - m), lse = m + ln l.
//
// Work. An item is (sequence, key/value head, row group): up to kRows query
// rows (query token x head of the group) that read the same pages. The items'
// visible pages are cut into runs, one per CTA (one CTA per SM): where the
// items fit the grid and are about equally long, each is cut into equal parts;
// else all of them form one list that is cut into equal runs, so that ragged
// batches balance and a run can hold the end of one item, whole ones and the
// start of another. A CTA whose run covers part of an item writes its partial
// rows (m, l, unnormalised out) to the workspace; the last of the item's CTAs
// to arrive (a ticket) joins them in CTA order, so results do not depend on
// the arrival order. No CTA waits for another.
//
// In a CTA, teams of kRW warps take the run's pages in turn. Each team has its
// own ring of page slots (key and value image, one contiguous bulk copy) that
// its first warp refills; the copies run ahead across items. The warps of a
// team share its pages, each on kNT tiles of 8 rows.
//
// Mathematics of a page (64 tokens) in a warp, rows on the MMA's N side so
// that 8 rows fill a tile (swap-AB, as the expert kernel), f16 MMAs
// (m16n8k16) with fp32 sums throughout:
//  S^T[64 x 8] = K Q^T. E4M3 is a subset of f16, so K converts exactly; q is
//    held in f16 after a power-of-two scale per row that puts its largest
//    value in [2^14, 2^15): bf16's 8 significant bits fit f16's 11, exactly
//    down to 2^-28 of the row's largest value and to 2^-39 of it below.
//    (mma.sync on E4M3 operands would spare the conversion, but converts
//    inside: 0.16 of depth 32 per cycle and SM with operands that change,
//    where f16 issues 0.39 of depth 16.)
//  the softmax in fp32, with the running maximum per row and warp;
//  O^T[D x 8] += V^T P^T, V converted exactly, P in f16 scaled by 2^14: 11
//    significant bits down to 2^-28 of the row's largest weight, so the tail
//    of a long context is kept. (E4M3 weights would lose what lies 2^-18 below
//    the largest.) The value transposed in the cache is the MMA's A operand as
//    it lies; P^T gets from the accumulators' layout to the B operand's by
//    movmatrix.
//  A page's product starts from zero and joins the running sum as
//    O = O * alpha + acc * 2^(code - 127 - 14): one FMA per value does the
//    softmax's rescaling, the page's own value scale and P's.
//
// Masked tokens never touch a row, whatever their bytes: scores are replaced
// (not added to), and on pages where some row's mask cuts, the product runs
// once per query token of the tile with the other tokens' value bytes zeroed,
// so that a NaN in an unwritten or masked place stays there.
//
// Bound by HBM while a warp's work on a page (about 700 instructions per tile of
// 8 rows) stays below its six-fold share of the page's copy time. 8 heads of
// 128, 5 query heads each: 48 sequences of up to 16k tokens 131 us (6.3 TB/s,
// 93 % of a plain copy's rate), up to 4k 41 us (72 %), one of 131k 48 us (82 %),
// 16 windows of 4k 25 us (72 %). What is left is about 10 us a call: the start (3),
// an item's end and the next one's rows (1.5 to 2 each, covered by the copies
// that run ahead), the teams' and CTAs' joins (3 to 5). 16 rows: 77 us where 8
// take 64 (48 sequences over 3.5k tokens): two warps then convert each page.
//
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "internal.cuh"
#include "kv_x8.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {
namespace attn {

constexpr float kLog2P = 14.0f;  // P and its sum are held times 2^14
constexpr float kUnP = 0x1p-14f;  // O is not: it has fp32's whole range for values as large as bf16's

template <int D, int NT, int RW>
struct Cfg {
  // Two slots a team at least, 255 registers a thread (8 warps), and room for
  // the teams' join: of 12 pages of 16 KB (D = 128) two for each of six warps or
  // three for each of four teams of two (16 rows: 77 us, by six such warps 97; 48
  // sequences over 3.5k tokens, 8 heads); of 24 pages of 8 KB (D = 64) three for
  // each of eight warps (8 rows: 37 us, with six 42, with twelve 38); of the 32 KB
  // pages of D = 256 six for three teams of one warp or two of two (16 rows: 102
  // us, three of two 109), four for two teams of three.
  static constexpr int kWarps = D == 256 ? (RW == 1 ? 3 : RW == 2 ? 4 : 6) : D == 64 || RW == 2 ? 8 : 6;
  static constexpr uint32_t kRingBytes = D == 256 && RW == 3 ? 131072 : 196608;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTeams = kWarps / RW;
  static constexpr int kRows = 8 * NT * RW;              // rows of a row group
  static constexpr uint32_t kHalf = kPageTokens * D;     // bytes of an image
  static constexpr uint32_t kPage = 2 * kHalf;
  static constexpr int kSlots = kRingBytes / kPage;      // all teams'
  static constexpr int kTeamSlots = kSlots / kTeams;
  static constexpr uint32_t kOffMerge = kRingBytes;      // [warp][8 rows][D] fp32
  static constexpr uint32_t kOffMl = kOffMerge + kWarps * 8 * D * 4;  // [warp][NT][8] x {m, l}
  static constexpr uint32_t kOffBar = kOffMl + kWarps * NT * 8 * 8;
  static constexpr uint32_t kOffMeta = kOffBar + kSlots * 16;
  static constexpr uint32_t kOffMisc = kOffMeta + (kSlots * 4 + 15) / 16 * 16;
  static constexpr uint32_t kSmem = kOffMisc + 256;
  static_assert(kWarps % RW == 0 && kTeamSlots >= 2, "ring");
  static_assert(kSmem <= 232448, "shared memory");
};

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four E4M3 bytes -> two f16 pairs (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

using ptx::elect_one;
using ptx::kWaitClocks;

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return ptx::mbar_wait_clocks(bar, parity, abort);
}

// ---------------------------------------------------------------- work list
// A CTA's start and end are chains of scalar code that nothing overlaps, so
// the divisions in them are short ones.
//
// x / group: exact while x * group < 2^32 (the host checks it)
__device__ __forceinline__ int by_group(const AttnX8Params& p, int x) {
  return p.group == 1 ? x : static_cast<int>(__umulhi(static_cast<unsigned>(x), p.group_magic));
}

// a / b for 0 <= a, 0 < b: the fp32 quotient is off by at most one below 2^22
__device__ __forceinline__ int div_pos(int a, int b) {
  if (a >= (1 << 22) || b >= (1 << 22)) return a / b;
  int n = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  const int r = a - n * b;
  n += r >= b ? 1 : 0;
  n -= r < 0 ? 1 : 0;
  return n;
}

// One sequence's rows and visible pages.
struct Seq {
  int q0, n, kv;      // first query token, query tokens, tokens in the cache
  int sink_pages, lo; // visible: pages [0, sink_pages) and [lo, ceil(kv / 64))
  int pages;          // their number (at least 1 where there are rows)
  int groups;         // row groups per head
};

template <int kRows>
__device__ __forceinline__ Seq load_seq(const AttnX8Params& p, int b) {
  Seq s;
  const int len = __ldg(p.kv_len + b);
  if (p.cu_q) {
    const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1);
    s.q0 = min(max(c0, 0), p.tokens);
    s.n = min(max(c1, s.q0), p.tokens) - s.q0;
  } else {
    s.q0 = b;
    s.n = 1;
  }
  s.kv = min(max(len, 0), p.max_kv);
  const int hi = (s.kv + kPageTokens - 1) / kPageTokens;
  s.lo = 0;
  s.sink_pages = 0;
  if (p.window > 0) {
    s.lo = max(s.kv - s.n - p.window + 1, 0) / kPageTokens;
    s.sink_pages = min((min(p.sinks, s.kv) + kPageTokens - 1) / kPageTokens, s.lo);
  }
  s.pages = s.n > 0 ? max(s.sink_pages + hi - s.lo, 1) : 0;
  s.groups = (s.n * p.group + kRows - 1) / kRows;
  return s;
}

// List positions of one item: kItemCost for its start and end (they cost about
// as much as that many pages), then its pages.
__device__ __forceinline__ int item_size(const Seq& s) { return s.pages + kItemCost; }

// A walk over a run [w, end) of the work list, segment by segment: the run's
// part of one item's pages.
struct Walk {
  int w, end, base;  // base: list position of the sequence's first item
  int b;
  Seq s;
  // the current segment
  int head, group, first, last;  // pages [first, last) of the item's
  int item_start;                // list position of the item
};

template <int kRows>
__device__ __forceinline__ bool next_segment(const AttnX8Params& p, Walk& k) {
  while (k.w < k.end) {
    int size = item_size(k.s) * k.s.groups * p.kv_heads;
    while (k.w >= k.base + size) {
      if (++k.b >= p.seqs) return false;  // (not reached: the run ends inside the list)
      k.base += size;
      k.s = load_seq<kRows>(p, k.b);
      size = item_size(k.s) * k.s.groups * p.kv_heads;
    }
    const int local = k.w - k.base;
    const int item = div_pos(local, item_size(k.s));
    k.head = k.s.groups == 1 ? item : div_pos(item, k.s.groups);
    k.group = item - k.head * k.s.groups;
    k.item_start = k.base + item * item_size(k.s);
    const int stop = min(k.item_start + item_size(k.s), k.end);
    k.first = max(k.w - k.item_start - kItemCost, 0);
    k.last = stop - k.item_start - kItemCost;
    k.w = stop;
    if (k.last > k.first) return true;
  }
  return false;
}

// This CTA's run of the work list, found by every warp for itself, 32 sequences
// at a time (nothing to wait for but the lengths): once over them for the
// list's length, once more (the first 32 from registers) to the run's start.
// False: nothing to do (the same in every warp). `teams`: pages that a CTA works on at once. parts: CTAs per
// item (aligned runs), or 0 and then per: list positions per run. kUneven: how
// much longer than others a run may be, in eighths (bandwidth goes where pages
// are left, the time of products does not).
template <int kRows, int kUneven>
__device__ __forceinline__ bool find_run(const AttnX8Params& p, int teams, int lane, int warp, Walk& walk,
                                         int& per, int& parts) {
  parts = 0;
  int total = 0, items = 0, longest = 0;
  bool odd_len = false, falls = false;
  Seq head = {};  // of sequence `lane`, which the search below begins with
  for (int b = lane; b < p.seqs; b += 32) {
    const Seq s = load_seq<kRows>(p, b);
    if (b == lane) head = s;
    odd_len |= __ldg(p.kv_len + b) != s.kv;
    const int n = s.groups * p.kv_heads;
    total += item_size(s) * n;
    items += n;
    longest = max(longest, s.pages);
    falls |= p.cu_q != nullptr && __ldg(p.cu_q + b) > __ldg(p.cu_q + b + 1);
  }
  // Starts that do not ascend: rows of two sequences could be the same, and the
  // list longer than 32 bits count.
  const bool disorder = __any_sync(0xffffffffu, falls);
  odd_len |= disorder;
  if (odd_len && blockIdx.x == 0 && warp == 0 && p.status) atomicOr(p.status, kKvErrLength);
  total = __reduce_add_sync(0xffffffffu, total);
  items = __reduce_add_sync(0xffffffffu, items);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (items == 0 || disorder) return false;
  const int cta = blockIdx.x, grid = gridDim.x;
  per = div_pos(total + grid - 1, grid);
  // Aligned: every item in `parts` equal parts, when that makes no run longer
  // than an equal share of the pages by more than kUneven eighths, each part
  // at least two pages per team (shorter ones save less than the join costs).
  if (items <= grid) {
    const int share = div_pos(total - items * kItemCost, grid);
    const int k = max(min(div_pos(grid, items), longest / (2 * teams)), 1);
    if (div_pos(longest + k - 1, k) <= max(share + share * kUneven / 8, 2 * teams)) parts = k;
  }
  // list: no run shorter than one page per team while items have as many
  if (parts == 0) per = max(per, min(teams, div_pos(total, items)));
  const int at = parts ? div_pos(cta, parts) : min(per * cta, total);  // item, or list position
  if (at >= (parts ? items : total)) return false;
  int base = 0, seen = 0;  // list position and units before the current 32 sequences
  for (int b0 = 0;; b0 += 32) {
    Seq s = head;
    if (b0 > 0) {
      s = {};
      if (b0 + lane < p.seqs) s = load_seq<kRows>(p, b0 + lane);
    }
    const int n = s.groups * p.kv_heads, size = item_size(s) * n, step = parts ? n : size;
    if (b0 + 32 < p.seqs) {
      const int all = __reduce_add_sync(0xffffffffu, step);
      if (at >= seen + all) {
        seen += all;
        base += __reduce_add_sync(0xffffffffu, size);
        continue;
      }
    }
    int upto = step, pos = size;  // inclusive sums over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o), v = __shfl_up_sync(0xffffffffu, pos, o);
      if (lane >= o) {
        upto += u;
        pos += v;
      }
    }
    const int who = __ffs(__ballot_sync(0xffffffffu, at < seen + upto)) - 1;  // (there is one)
    walk.b = b0 + who;
    walk.base = base + __shfl_sync(0xffffffffu, pos - size, who);
    seen += __shfl_sync(0xffffffffu, upto - step, who);
    walk.s.q0 = __shfl_sync(0xffffffffu, s.q0, who);
    walk.s.n = __shfl_sync(0xffffffffu, s.n, who);
    walk.s.kv = __shfl_sync(0xffffffffu, s.kv, who);
    walk.s.sink_pages = __shfl_sync(0xffffffffu, s.sink_pages, who);
    walk.s.lo = __shfl_sync(0xffffffffu, s.lo, who);
    walk.s.pages = __shfl_sync(0xffffffffu, s.pages, who);
    walk.s.groups = __shfl_sync(0xffffffffu, s.groups, who);
    break;
  }
  if (parts) {
    const int len = div_pos(walk.s.pages + parts - 1, parts);
    const int first = (cta - at * parts) * len;
    if (first >= walk.s.pages) return false;
    walk.w = walk.base + (at - seen) * item_size(walk.s) + kItemCost + first;
    walk.end = walk.w + min(len, walk.s.pages - first);
  } else {
    walk.w = at;
    walk.end = at + min(per, total - at);
  }
  return true;
}

// The first and last CTA of an item of which this CTA has a part.
__device__ __forceinline__ void item_ctas(int item_start, int pages, int per, int parts, int& c0, int& c1) {
  if (parts) {
    c0 = div_pos(blockIdx.x, parts) * parts;
    const int len = div_pos(pages + parts - 1, parts);
    c1 = c0 + div_pos(pages + len - 1, len) - 1;
  } else {
    c0 = div_pos(item_start + kItemCost, per);
    c1 = div_pos(item_start + kItemCost + pages - 1, per);
  }
}

// A segment whose item other CTAs share, joined at the CTA's end.
struct Shared {
  int c0, c1;  // the item's CTAs (c1 < 0: no such segment)
  int q0, rows, head, row0;
  int last;    // this CTA arrived last
  int pad;
};

// Does a row at position `at` see a token?
__device__ __forceinline__ bool sees(const AttnX8Params& p, int token, int at) {
  return token <= at && (p.window == 0 || token > at - p.window || token < p.sinks);
}

// What rows at positions lo .. hi see of tokens t0 .. t1: 0 nothing, 1 all of
// it every one, 2 otherwise.
__device__ __forceinline__ int page_kind(const AttnX8Params& p, int t0, int t1, int lo, int hi) {
  if (t1 <= lo && (p.window == 0 || t0 > hi - p.window || t1 < p.sinks)) return 1;
  if (t0 > hi || (p.window > 0 && t1 <= lo - p.window && t0 >= p.sinks)) return 0;
  return 2;
}

// Four dims of a finished row: sum / den, and with the first ones the lse;
// both are relative to `top` (log2 units), den is held times 2^log2_scale and
// `ratio` times as large as sum.
template <int D>
__device__ __forceinline__ void store_row(const AttnX8Params& p, int q0, int head, int r, int d4, const float4& sum,
                                          float top, float den, float log2_scale, float ratio) {
  const int token = by_group(p, r);
  const size_t at = static_cast<size_t>(q0 + token) * (p.kv_heads * p.group) + head * p.group + r - token * p.group;
  const float inv = den == 0.0f ? 0.0f : __frcp_rn(den) * ratio;
  __align__(8) __nv_bfloat162 y[2] = {__floats2bfloat162_rn(sum.x * inv, sum.y * inv),
                                      __floats2bfloat162_rn(sum.z * inv, sum.w * inv)};
  *reinterpret_cast<uint2*>(p.out + at * D + d4 * 4) = *reinterpret_cast<const uint2*>(y);
  if (d4 == 0 && p.lse)
    p.lse[at] = den == 0.0f ? -INFINITY : (top + log2f(den) - log2_scale) * 0.69314718055994531f;
}

// The CTA's end: items of several CTAs (a run has at most two). The last CTA
// to arrive joins their partial rows, in the order of the CTAs: each warp the
// parts c0 + w, c0 + w + kWarps, ... of 256 x 4 dims at a time, then the warps'
// sums through shared memory (`space`, 256 x kWarps x 24 bytes that nothing
// uses any more). All threads call this after a barrier behind their partial
// rows.
template <int D, int kRows, int kWarps>
__device__ __forceinline__ void join_shared(const AttnX8Params& p, Shared* shared, uint8_t* space, int tid,
                                            float log2_scale, float ratio) {
  if (shared[0].c1 < 0 && shared[1].c1 < 0) return;  // (the same in every thread)
  if (tid < 2) {
    Shared& x = shared[tid];
    x.last = 0;
    if (x.c1 >= 0) {
      // releases the CTA's partial rows (the barrier before orders them) and
      // acquires those of the CTAs that came earlier
      int done;
      asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(done) : "l"(p.tickets + x.c0) : "memory");
      if (done == x.c1 - x.c0) {
        p.tickets[x.c0] = 0;
        x.last = 1;
      }
    }
  }
  __syncthreads();
  constexpr int kUnits = 256, kPer = kUnits / 32;  // units of 4 dims, per lane
  float4* sums = reinterpret_cast<float4*>(space);                      // [warp][kUnits]
  float2* mls = reinterpret_cast<float2*>(sums + kWarps * kUnits);
  const int warp = tid >> 5, lane = tid & 31;
  for (int i = 0; i < 2; ++i) {
    const Shared x = shared[i];
    if (x.c1 < 0 || !x.last) continue;
    const int count = min(kRows, x.rows - x.row0) * (D / 4);
    for (int u0 = 0; u0 < count; u0 += kUnits) {
      float4 sum[kPer];
      float top[kPer], den[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        sum[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        top[k] = -INFINITY;
        den[k] = 0.0f;
      }
#pragma unroll 2
      for (int c = x.c0 + warp; c <= x.c1; c += kWarps) {
        const float* part = p.part + (static_cast<size_t>(c) * 2 + (c == x.c0)) * kRows * (D + 2);
        float4 y[kPer];
        float2 t[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int u = min(u0 + lane + 32 * k, count - 1);
          y[k] = __ldcg(reinterpret_cast<const float4*>(part) + u);
          t[k] = __ldcg(reinterpret_cast<const float2*>(part + kRows * D) + u / (D / 4));
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const float high = fmaxf(top[k], t[k].x), use = high == -INFINITY ? 0.0f : high;
          const float keep = ex2(top[k] - use), w = ex2(t[k].x - use);
          top[k] = high;
          den[k] = den[k] * keep + t[k].y * w;
          sum[k].x = sum[k].x * keep + y[k].x * w;
          sum[k].y = sum[k].y * keep + y[k].y * w;
          sum[k].z = sum[k].z * keep + y[k].z * w;
          sum[k].w = sum[k].w * keep + y[k].w * w;
        }
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        sums[warp * kUnits + lane + 32 * k] = sum[k];
        mls[warp * kUnits + lane + 32 * k] = make_float2(top[k], den[k]);
      }
      __syncthreads();
#pragma unroll 1
      for (int u = tid; u < kUnits && u0 + u < count; u += 32 * kWarps) {
        float high = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) high = fmaxf(high, mls[w * kUnits + u].x);
        const float use = high == -INFINITY ? 0.0f : high;
        float all = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = sums[w * kUnits + u];
          const float2 t = mls[w * kUnits + u];
          const float k = ex2(t.x - use);
          all = fmaf(t.y, k, all);
          o.x = fmaf(y.x, k, o.x);
          o.y = fmaf(y.y, k, o.y);
          o.z = fmaf(y.z, k, o.z);
          o.w = fmaf(y.w, k, o.w);
        }
        store_row<D>(p, x.q0, x.head, x.row0 + (u0 + u) / (D / 4), (u0 + u) % (D / 4), o, high, all, log2_scale,
                     ratio);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- the kernel
template <int D, int NT, int RW>
__global__ void __launch_bounds__(Cfg<D, NT, RW>::kThreads, 1)
    attn_x8_kernel(const AttnX8Params p) {
  using C = Cfg<D, NT, RW>;
  constexpr int kKC = D / 16;  // 16-dim chunks (depth steps of the score product)
  constexpr int kDT = D / 16;  // dim tiles of the value product
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  int* meta = reinterpret_cast<int*>(smem + C::kOffMeta);
  Shared* shared = reinterpret_cast<Shared*>(smem + C::kOffMisc);  // [2] by partial slot
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 64);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int team = warp / RW, rw = warp % RW;
  const int g = lane >> 2, q = lane & 3;

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      ptx::mbar_init(sbase + C::kOffBar + i * 16, 1);
      ptx::mbar_init(sbase + C::kOffBar + i * 16 + 8, RW);
    }
    ptx::fence_mbar_init();
    *abort_flag = 0;
    shared[0].c1 = shared[1].c1 = -1;
  }
  __syncthreads();
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // ---- this CTA's run
  Walk walk;
  int per, parts;
  if (!find_run<C::kRows, 3>(p, C::kTeams, lane, warp, walk, per, parts)) return;  // the whole CTA

  // ---- the query rows of a segment, raw: 4 dims of each 16 per thread
  uint2 raw[NT][kKC];
  const auto load_rows = [&](const Walk& k) {
    const int rows = k.s.n * p.group;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = k.group * C::kRows + (rw * NT + nt) * 8 + g;
      const int token = by_group(p, r);
      const __nv_bfloat16* qr = p.q + (k.s.q0 + token) * p.ldq +
                                static_cast<long long>(k.head * p.group + r - token * p.group) * D;
#pragma unroll
      for (int c = 0; c < kKC; ++c) {
        raw[nt][c] = make_uint2(0, 0);
        if (r < rows) raw[nt][c] = __ldg(reinterpret_cast<const uint2*>(qr + 16 * c + 4 * q));
      }
    }
  };

  // ---- the ring's filler: the team's first warp walks the same run ahead
  const int slot0 = team * C::kTeamSlots;
  const auto full = [&](int slot) { return sbase + C::kOffBar + (slot0 + slot) * 16; };
  const auto empty = [&](int slot) { return sbase + C::kOffBar + (slot0 + slot) * 16 + 8; };
  Walk ahead = walk;
  bool ahead_on = true;
  int ahead_page = 0;         // next page of the segment for this team
  int ahead_at = 32;          // lane that holds it among the fetched ids
  int ids = -1;
  int filled = 0;             // pages issued
  ahead.last = 0;
  int fill_slot = 0;
  uint32_t fill_phase = 0;    // parity of the slot's last release
  bool dead = false;          // a wait gave up: no more copies

  const auto fill = [&]() {  // issues the next page, all lanes of the warp together
    if (!ahead_on || dead) return;
    while (ahead_page >= ahead.last) {
      if (!next_segment<C::kRows>(p, ahead)) {
        ahead_on = false;
        return;
      }
      ahead_page = ahead.first + team;
      ahead_at = 32;
    }
    if (ahead_at == 32) {  // the next 32 page ids, one per lane
      const int j = ahead_page + lane * C::kTeams;
      ids = -1;
      if (j < ahead.last && ahead.s.kv > 0) {
        const int index = j < ahead.s.sink_pages ? j : ahead.s.lo + (j - ahead.s.sink_pages);
        ids = __ldg(p.page_table + static_cast<size_t>(ahead.b) * p.max_pages + index);
        if (ids < 0 || ids >= p.pages) {
          ids = -1;
          if (p.status) atomicOr(p.status, kKvErrPage);
        }
      }
      ahead_at = 0;
    }
    const int id = __shfl_sync(0xffffffffu, ids, ahead_at);
    if (RW > 1 && filled >= C::kTeamSlots) {
      if (!__all_sync(0xffffffffu, mbar_wait(empty(fill_slot), fill_phase, abort_flag))) {
        dead = true;
        if (p.status) atomicOr(p.status, kKvErrTimeout);
        return;
      }
    }
    if (elect_one()) {
      const uint32_t bar = full(fill_slot);
      meta[slot0 + fill_slot] = id;
      if (id < 0) {
        ptx::mbar_arrive(bar);
      } else {
        ptx::mbar_arrive_expect_tx(bar, C::kPage);
        ptx::bulk_load(sbase + (slot0 + fill_slot) * C::kPage,
                       p.blocks + (static_cast<size_t>(id) * p.kv_heads + ahead.head) * C::kPage, C::kPage, bar);
      }
    }
    __syncwarp();
    ++filled;
    if (++fill_slot == C::kTeamSlots) {
      fill_slot = 0;
      if (filled > C::kTeamSlots) fill_phase ^= 1;
    }
    ahead_page += C::kTeams;
    ++ahead_at;
  };

  bool more = next_segment<C::kRows>(p, walk);
  if (more) load_rows(walk);
  if (rw == 0)
    for (int i = 0; i < (RW > 1 ? C::kTeamSlots - 1 : C::kTeamSlots); ++i) fill();

  // ---- consume
  int use_slot = 0;
  uint32_t use_phase = 0;
  const auto wait_full = [&]() {
    if (!__all_sync(0xffffffffu, mbar_wait(full(use_slot), use_phase, abort_flag))) {
      dead = true;
      if (p.status) atomicOr(p.status, kKvErrTimeout);
      return -1;
    }
    return meta[slot0 + use_slot];
  };
  const auto release = [&]() {  // this warp is done with the page
    __syncwarp();
    if (RW > 1 && lane == 0) ptx::mbar_arrive(empty(use_slot));
    if (++use_slot == C::kTeamSlots) {
      use_slot = 0;
      use_phase ^= 1;
    }
    if (rw == 0) fill();
  };

  // matrix-load rows of this lane: 8 rows x {16-byte chunk} per quarter warp
  const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mchunk = lane >> 4;
  const int kswz = D >= 128 ? (lane & 7) : ((lane & 7) >> 1);
  const int vswz = (lane & 7) >> 1;

  while (more) {
    const Seq s = walk.s;
    const int rows = s.n * p.group;  // of the head
    const int row0 = walk.group * C::kRows + rw * NT * 8;
    const int first = walk.first, last = walk.last, head = walk.head, item_start = walk.item_start;
    const int group0 = walk.group * C::kRows;

    // ---- the rows: Q in f16, positions, factors
    uint32_t qf[NT][kKC][2];
    float factor[NT][2];   // raw score -> log2 units, rows 2q and 2q + 1
    int pos[NT][2];
    int pos_lo[NT], pos_hi[NT];
    float m[NT][2], l[NT][2];
    float o[NT][kDT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float amax = 0.0f;
#pragma unroll
      for (int c = 0; c < kKC; ++c) {
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[nt][c].x << 16)),
                                 fabsf(__uint_as_float(raw[nt][c].x & 0xFFFF0000u))));
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[nt][c].y << 16)),
                                 fabsf(__uint_as_float(raw[nt][c].y & 0xFFFF0000u))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // the row times 2^a, its largest value in [2^14, 2^15)
      const int e = static_cast<int>(__float_as_uint(amax) >> 23);
      const int a = amax > 0.0f ? min(141 - e, 126) : 0;
      const float mul = __uint_as_float(static_cast<uint32_t>(127 + a) << 23);
      const float f = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
#pragma unroll
      for (int c = 0; c < kKC; ++c) {
        const uint2 w = raw[nt][c];
        qf[nt][c][0] = pack_f16(__uint_as_float(w.x << 16) * mul, __uint_as_float(w.x & 0xFFFF0000u) * mul);
        qf[nt][c][1] = pack_f16(__uint_as_float(w.y << 16) * mul, __uint_as_float(w.y & 0xFFFF0000u) * mul);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        factor[nt][c] = __shfl_sync(0xffffffffu, f, (2 * q + c) * 4);
        const int rc = min(row0 + nt * 8 + 2 * q + c, rows - 1);  // rows past the last see what it sees
        pos[nt][c] = s.kv - s.n + by_group(p, rc);
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.0f;
      }
      pos_lo[nt] = s.kv - s.n + by_group(p, min(row0 + nt * 8, rows - 1));
      pos_hi[nt] = s.kv - s.n + by_group(p, min(row0 + nt * 8 + 7, rows - 1));
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][d][j] = 0.0f;
    }

    for (int j = first + team; j < last; j += C::kTeams) {
      const int index = j < s.sink_pages ? j : s.lo + (j - s.sink_pages);
      const int t0 = index * kPageTokens, t1 = t0 + kPageTokens - 1;
      int kind[NT];
      bool any = false, cut = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        kind[nt] = row0 + nt * 8 >= rows ? 0 : page_kind(p, t0, t1, pos_lo[nt], pos_hi[nt]);
        any |= kind[nt] != 0;
        cut |= kind[nt] == 2;
      }
      const int id = wait_full();
      if (any && id >= 0) {  // (a page id out of range is skipped)
        // the page's codes: needed after the score product, under which they arrive
        const int page_codes = __ldg(reinterpret_cast<const unsigned short*>(p.codes) +
                                     static_cast<size_t>(id) * p.kv_heads + head);
        const uint32_t kb = sbase + (slot0 + use_slot) * C::kPage, vb = kb + C::kHalf;
        float sc[NT][4][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[nt][mt][i] = 0.0f;
        // four token tiles side by side: independent chains hide the MMA's latency
#pragma unroll
        for (int k = 0; k < kKC / 2; ++k) {
          uint32_t w[4][4];
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
            ldsm_x4(kb + (mt * 16 + mrow) * D + (((2 * k + mchunk) ^ kswz) << 4), w[mt]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              uint32_t a[4];
              e4m3x4_f16(w[mt][2 * h], a[0], a[2]);
              e4m3x4_f16(w[mt][2 * h + 1], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(sc[nt][mt], a, qf[nt][2 * k + h][0], qf[nt][2 * k + h][1]);
            }
        }

        // ---- softmax of the page
        const float kscale = e8m0_value(page_codes & 0xFF), vscale = e8m0_value(page_codes >> 8) * kUnP;
        uint32_t pf[NT][4][2];
        float alpha[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (kind[nt] == 2) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!sees(p, t0 + mt * 16 + g + (i >> 1) * 8, pos[nt][i & 1]))
                  sc[nt][mt][i] = -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(sc[nt][0][c], sc[nt][0][c + 2]);
#pragma unroll
            for (int mt = 1; mt < 4; ++mt) mx = fmaxf(mx, fmaxf(sc[nt][mt][c], sc[nt][mt][c + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float f = fmaxf(factor[nt][c] * kscale, FLT_MIN);  // (never 0: masked scores are -inf)
            const float top = kind[nt] == 0 ? m[nt][c] : fmaxf(m[nt][c], mx * f);
            const float use = top == -INFINITY ? 0.0f : top;
            alpha[nt][c] = ex2(m[nt][c] - use);
            m[nt][c] = top;
            float sum = 0.0f;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
              sc[nt][mt][c] = ex2(fmaf(sc[nt][mt][c], f, kLog2P - use));
              sc[nt][mt][c + 2] = ex2(fmaf(sc[nt][mt][c + 2], f, kLog2P - use));
              sum += sc[nt][mt][c] + sc[nt][mt][c + 2];
            }
            if (kind[nt] != 0) l[nt][c] = l[nt][c] * alpha[nt][c] + sum;
          }
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            pf[nt][mt][0] = movm(pack_f16(sc[nt][mt][0], sc[nt][mt][1]));
            pf[nt][mt][1] = movm(pack_f16(sc[nt][mt][2], sc[nt][mt][3]));
          }
        }

        if (!cut) {
          constexpr int kG = 4;  // dim tiles side by side
#pragma unroll
          for (int d0 = 0; d0 < kDT; d0 += kG) {
            float acc[kG][NT][4];
#pragma unroll
            for (int dd = 0; dd < kG; ++dd)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[dd][nt][i] = 0.0f;
#pragma unroll
            for (int cp = 0; cp < 2; ++cp) {
              uint32_t w[kG][4];
#pragma unroll
              for (int dd = 0; dd < kG; ++dd)
                ldsm_x4(vb + ((d0 + dd) * 16 + mrow) * kPageTokens + (((2 * cp + mchunk) ^ vswz) << 4), w[dd]);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int dd = 0; dd < kG; ++dd) {
                  uint32_t a[4];
                  e4m3x4_f16(w[dd][2 * h], a[0], a[2]);
                  e4m3x4_f16(w[dd][2 * h + 1], a[1], a[3]);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    mma_f16(acc[dd][nt], a, pf[nt][2 * cp + h][0], pf[nt][2 * cp + h][1]);
                }
            }
#pragma unroll
            for (int dd = 0; dd < kG; ++dd)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                if (kind[nt] != 0)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    o[nt][d0 + dd][i] = fmaf(o[nt][d0 + dd][i], alpha[nt][i & 1], acc[dd][nt][i] * vscale);
          }
        } else {
          // some row's mask cuts this page: per query token of the tile, the
          // tokens it does not see have their value bytes zeroed, and only
          // its rows take the sum
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (kind[nt] == 0) continue;
            for (int at = pos_lo[nt]; at <= pos_hi[nt]; ++at) {
              uint32_t keep[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int t = t0 + c * 16 + 2 * q;
                keep[c] = (sees(p, t, at) ? 0x000000FFu : 0u) | (sees(p, t + 1, at) ? 0x0000FF00u : 0u) |
                          (sees(p, t + 8, at) ? 0x00FF0000u : 0u) | (sees(p, t + 9, at) ? 0xFF000000u : 0u);
              }
              const bool mine[2] = {pos[nt][0] == at, pos[nt][1] == at};
#pragma unroll
              for (int d = 0; d < kDT; ++d) {
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int cp = 0; cp < 2; ++cp) {
                  uint32_t w[4], a0[4], a1[4];
                  ldsm_x4(vb + (d * 16 + mrow) * kPageTokens + (((2 * cp + mchunk) ^ vswz) << 4), w);
                  e4m3x4_f16(w[0] & keep[2 * cp], a0[0], a0[2]);
                  e4m3x4_f16(w[1] & keep[2 * cp], a0[1], a0[3]);
                  e4m3x4_f16(w[2] & keep[2 * cp + 1], a1[0], a1[2]);
                  e4m3x4_f16(w[3] & keep[2 * cp + 1], a1[1], a1[3]);
                  mma_f16(acc, a0, pf[nt][2 * cp][0], pf[nt][2 * cp][1]);
                  mma_f16(acc, a1, pf[nt][2 * cp + 1][0], pf[nt][2 * cp + 1][1]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (mine[i & 1])
                    o[nt][d][i] = fmaf(o[nt][d][i], alpha[nt][i & 1], acc[i] * vscale);
              }
            }
          }
        }
      }
      release();
    }

    // the next segment's rows are on their way while this one is joined
    const bool whole = first == 0 && last == s.pages;
    more = next_segment<C::kRows>(p, walk);
    if (more) load_rows(walk);

    // ---- the segment's rows: join the teams, then write them out or to the workspace
    int c0 = 0, c1 = 0;
    if (!whole) item_ctas(item_start, s.pages, per, parts, c0, c1);
    const int part_slot = static_cast<int>(blockIdx.x) == c0;
    float* part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + part_slot) * C::kRows * (D + 2);
    if (!whole && tid == 0) {
      Shared& x = shared[part_slot];
      x.c0 = c0;
      x.c1 = c1;
      x.q0 = s.q0;
      x.rows = rows;
      x.head = head;
      x.row0 = group0;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float t = l[nt][c];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        l[nt][c] = t;
        if (g == 0) ml[(warp * NT + nt) * 8 + 2 * q + c] = make_float2(m[nt][c], t);
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // this warp's rows, relative to the teams' common maximum
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < C::kTeams; ++t)
          top = fmaxf(top, ml[((t * RW + rw) * NT + nt) * 8 + 2 * q + c].x);
        const float w = top == -INFINITY ? 0.0f : ex2(m[nt][c] - top);
        const int row = 2 * q + c;
#pragma unroll
        for (int d = 0; d < kDT; ++d)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            merge[(warp * 8 + row) * D + ((d * 16 + h * 8 + g) ^ (q << 3))] = o[nt][d][2 * h + c] * w;
      }
      __syncthreads();
      // 4 dims a thread, teams in order
      for (int i = tid; i < RW * 8 * (D / 4); i += C::kThreads) {
        const int d4 = i % (D / 4), row = (i / (D / 4)) % 8, w = i / (D / 4) / 8;
        const int r = group0 + (w * NT + nt) * 8 + row;
        if (r >= rows) continue;
        const int at = (d4 * 4) ^ ((row >> 1) << 3);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float top = -INFINITY, den = 0.0f;
#pragma unroll
        for (int t = 0; t < C::kTeams; ++t)
          top = fmaxf(top, ml[((t * RW + w) * NT + nt) * 8 + row].x);
#pragma unroll
        for (int t = 0; t < C::kTeams; ++t) {
          const float4 x = *reinterpret_cast<const float4*>(merge + ((t * RW + w) * 8 + row) * D + at);
          sum.x += x.x;
          sum.y += x.y;
          sum.z += x.z;
          sum.w += x.w;
          const float2 t_ml = ml[((t * RW + w) * NT + nt) * 8 + row];
          den += top == -INFINITY ? 0.0f : t_ml.y * ex2(t_ml.x - top);
        }
        if (whole) {
          store_row<D>(p, s.q0, head, r, d4, sum, top, den, kLog2P, 1.0f / kUnP);
        } else {
          const int lr = (w * NT + nt) * 8 + row;
          *reinterpret_cast<float4*>(part + static_cast<size_t>(lr) * D + d4 * 4) = sum;
          if (d4 == 0)
            *reinterpret_cast<float2*>(part + static_cast<size_t>(C::kRows) * D + 2 * lr) = make_float2(top, den);
        }
      }
      __syncthreads();
    }
  }

  join_shared<D, C::kRows, C::kWarps>(p, shared, smem, tid, kLog2P, 1.0f / kUnP);

  // Every copy issued has been waited for, as each page of the run is
  // consumed. After a wait that gave up, the copies in flight get their time
  // before the CTA's shared memory goes.
  if (dead && rw == 0 && lane == 0) {
    for (int i = 0; i < C::kTeamSlots; ++i) {
      const int fills = (filled - i + C::kTeamSlots - 1) / C::kTeamSlots;
      const uint64_t t0 = ptx::globaltimer_ns();
      while (fills > 0 && !ptx::mbar_try_wait(full(i), (fills - 1) & 1) &&
             ptx::globaltimer_ns() - t0 < kWaitLimitNs / 8) {
      }
    }
  }
}

template <int D, int NT, int RW>
cudaError_t launch(const AttnX8Params& p, int device, int grid, cudaStream_t s) {
  using C = Cfg<D, NT, RW>;
  // the kernel's shared-memory limit, raised once per device
  static std::atomic<unsigned long long> raised{0};
  const unsigned long long bit = 1ull << (device & 63);
  if (device > 63 || !(raised.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_x8_kernel<D, NT, RW>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_pdl(attn_x8_kernel<D, NT, RW>, dim3(grid), dim3(C::kThreads), C::kSmem, s, p);
}

}  // namespace attn
}  // namespace moe
