// Attention of a step's query rows over the 8-bit paged cache (kv_x8.cuh).
//
// A sequence with kv tokens in the cache has n query rows; row i sits at
// position pos = kv - n + i and sees the tokens j <= pos with j > pos - window
// (window > 0) or j < sinks. Per row: s_j = scale q.k_j, m = max s,
// out = sum exp(s_j - m) v_j / l with l = sum exp(s_j - m), lse = m + ln l.
//
// Work. An item is (sequence, key/value head, row group): up to kRows query
// rows (query token x head of the group) that read the same pages. All items'
// visible pages form one list, cut into equal runs, one per CTA (one CTA per
// SM): ragged batches balance by themselves and one long sequence spreads over
// the whole GPU. A CTA whose run covers part of an item writes its partial
// rows (m, l, unnormalised out) to the workspace; the last of the item's CTAs
// to arrive (a ticket) joins them in CTA order, so results do not depend on
// the arrival order. No CTA waits for another.
//
// In a CTA, teams of kRW warps take the run's pages in turn. Each team has its
// own ring of half pages (a key or a value image each, one contiguous bulk
// copy) that its first warp refills; the copies run ahead across items. The
// warps of a team share its pages, each on kNT tiles of 8 rows.
//
// Mathematics of a page (64 tokens) in a warp, rows on the MMA's N side so
// that 8 rows fill a tile (swap-AB, as the expert kernel):
//  S^T[64 x 8] = K Q^T on E4M3 MMAs (m16n8k32): K straight from the cache, and
//    each q as a sum hi + lo of two E4M3 values after a power-of-two scale per
//    row. A bf16 value has 8 significant bits, hi takes 4 and the remainder
//    fits lo's, so the sum is exact for values down to 2^-10 of the row's
//    largest and within 2^-18 of it below: nothing bf16 held is lost. mma.sync
//    issues an E4M3 product of twice the depth at twice the rate of an f16
//    one (measured: 0.91 against 0.49 per ns and SM), and K needs no
//    conversion.
//  the softmax in fp32, with the running maximum per row and warp;
//  O^T[D x 8] += V^T P^T on f16 MMAs (m16n8k16): V converted exactly (E4M3 is
//    a subset of f16), P in f16 scaled by 2^14: 11 significant bits down to
//    2^-28 of the row's largest weight, so the tail of a long context is
//    kept. (E4M3 weights would lose what lies 2^-18 below the largest.) The
//    value transposed in the cache is the MMA's A operand as it lies; P^T gets
//    from the accumulators' layout to the B operand's by movmatrix.
//  A page's product starts from zero and joins the running sum as
//    O = O * alpha + acc * 2^(code - 127): one FMA per value does both the
//    softmax's rescaling and the page's own value scale.
//
// Masked tokens never touch a row, whatever their bytes: scores are replaced
// (not added to), and on pages where some row's mask cuts, the product runs
// once per query token of the tile with the other tokens' value bytes zeroed,
// so that a NaN in an unwritten or masked place stays there.
//
// Bound by memory while rows are few: 64 tokens x 8 rows at D = 128 cost about
// 370 warp instructions, where HBM delivers one page per SM in ~712 cycles.
// From about 7 tiles of rows on the tensor and issue slots bind.
#pragma once

#include <cuda_fp16.h>

#include "internal.cuh"
#include "kv_x8.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {
namespace attn {

constexpr uint32_t kRingBytes = 196608;
constexpr float kLog2P = 14.0f;  // P is held times 2^14

template <int D, int NT, int RW>
struct Cfg {
  static constexpr int kWarps = D == 256 ? 4 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTeams = kWarps / RW;
  static constexpr int kRows = 8 * NT * RW;              // rows of a row group
  static constexpr uint32_t kHalf = kPageTokens * D;     // bytes of an image
  static constexpr int kSlots = kRingBytes / kHalf;      // all teams'
  static constexpr int kTeamSlots = kSlots / kTeams;
  static constexpr uint32_t kOffRing = 0;
  static constexpr uint32_t kOffMerge = kRingBytes;      // [warp][8 rows][D] fp32
  static constexpr uint32_t kOffMl = kOffMerge + kWarps * 8 * D * 4;  // [warp][NT][8] x {m, l}
  static constexpr uint32_t kOffBar = kOffMl + kWarps * NT * 8 * 8;
  static constexpr uint32_t kOffMeta = kOffBar + kSlots * 16;
  static constexpr uint32_t kOffMisc = kOffMeta + kSlots * 4;
  static constexpr uint32_t kSmem = kOffMisc + 256;
  static_assert(kWarps % RW == 0 && kTeamSlots >= 3, "ring");
  static_assert(kSmem <= 232448, "shared memory");
};

// ---------------------------------------------------------------- instructions
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_e4m3(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// ---------------------------------------------------------------- work list
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
  if (p.cu_q) {
    s.q0 = min(max(__ldg(p.cu_q + b), 0), p.tokens);
    s.n = min(max(__ldg(p.cu_q + b + 1), s.q0), p.tokens) - s.q0;
  } else {
    s.q0 = b;
    s.n = 1;
  }
  s.kv = static_cast<int>(min(static_cast<long long>(max(__ldg(p.kv_len + b), 0)),
                              static_cast<long long>(p.max_pages) * kPageTokens));
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

// A walk over a run [w, end) of the work list, segment by segment: the run's
// part of one item.
struct Walk {
  long long w, end, base;  // base: list position of the sequence's first item
  int b;
  Seq s;
  // the current segment
  int head, group, first, last;  // pages [first, last) of the item's
  long long item_start;          // list position of the item's first page
};

template <int kRows>
__device__ __forceinline__ bool next_segment(const AttnX8Params& p, Walk& k) {
  if (k.w >= k.end) return false;
  long long size = static_cast<long long>(k.s.pages) * k.s.groups * p.kv_heads;
  while (k.w >= k.base + size) {
    if (++k.b >= p.seqs) return false;  // (not reached: the run ends inside the list)
    k.base += size;
    k.s = load_seq<kRows>(p, k.b);
    size = static_cast<long long>(k.s.pages) * k.s.groups * p.kv_heads;
  }
  const long long local = k.w - k.base;
  const int item = static_cast<int>(local / k.s.pages);
  k.head = item / k.s.groups;
  k.group = item % k.s.groups;
  k.first = static_cast<int>(local % k.s.pages);
  k.item_start = k.w - k.first;
  k.last = static_cast<int>(min(static_cast<long long>(k.s.pages), k.first + (k.end - k.w)));
  k.w += k.last - k.first;
  return true;
}

// ---------------------------------------------------------------- the kernel
template <int D, int NT, int RW>
__global__ void __launch_bounds__(Cfg<D, NT, RW>::kThreads, 1)
    attn_x8_kernel(const AttnX8Params p) {
  using C = Cfg<D, NT, RW>;
  constexpr int kKS = D / 32;  // depth steps of the score product
  constexpr int kDT = D / 16;  // dim tiles of the value product
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  int* meta = reinterpret_cast<int*>(smem + C::kOffMeta);
  long long* misc = reinterpret_cast<long long*>(smem + C::kOffMisc);  // [0..15] scan, [16..] results
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 24);
  int* last_flag = reinterpret_cast<int*>(misc + 25);

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
  }
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // ---- this CTA's run: thread t sums a stretch of sequences, a block scan
  // gives the list's length and the run's first sequence
  Walk walk;
  long long per;
  {
    const int chunk = (p.seqs + C::kThreads - 1) / C::kThreads;
    const int b0 = min(tid * chunk, p.seqs), b1 = min(b0 + chunk, p.seqs);
    long long sum = 0, items = 0;
    bool odd_len = false;
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq<C::kRows>(p, b);
      odd_len |= __ldg(p.kv_len + b) != s.kv;
      sum += static_cast<long long>(s.pages) * s.groups * p.kv_heads;
      items += static_cast<long long>(s.groups) * p.kv_heads;
    }
    if (odd_len && blockIdx.x == 0 && p.status) atomicOr(p.status, kKvErrLength);
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
      items += __shfl_xor_sync(0xffffffffu, items, o);
    }
    if (lane == 31) misc[warp] = inc;
    if (lane == 0) misc[8 + warp] = items;
    __syncthreads();
    long long before = 0, total = 0, all_items = 0;
#pragma unroll
    for (int i = 0; i < C::kWarps; ++i) {
      if (i < warp) before += misc[i];
      total += misc[i];
      all_items += misc[8 + i];
    }
    // pages per CTA: an equal share, but no less than one per team while an
    // item has as many (a shorter run saves no time and adds partial rows)
    per = (total + gridDim.x - 1) / gridDim.x;
    if (all_items > 0) per = max(per, min(static_cast<long long>(C::kTeams), total / all_items));
    walk.w = min(per * blockIdx.x, total);
    walk.end = min(walk.w + per, total);
    if (walk.w >= walk.end) return;  // uniform
    const long long from = before + inc - sum;
    if (walk.w >= from && walk.w < from + sum) {  // one thread
      long long base = from;
      int b = b0;
      for (;; ++b) {
        const Seq s = load_seq<C::kRows>(p, b);
        const long long size = static_cast<long long>(s.pages) * s.groups * p.kv_heads;
        if (walk.w < base + size || b + 1 >= b1) break;
        base += size;
      }
      misc[16] = base;
      misc[17] = b;
    }
    __syncthreads();
    walk.base = misc[16];
    walk.b = static_cast<int>(misc[17]);
    walk.s = load_seq<C::kRows>(p, walk.b);
  }

  // ---- the ring's filler: the team's first warp walks the same run ahead
  const int slot0 = team * C::kTeamSlots;
  const auto full = [&](int slot) { return sbase + C::kOffBar + (slot0 + slot) * 16; };
  const auto empty = [&](int slot) { return sbase + C::kOffBar + (slot0 + slot) * 16 + 8; };
  Walk ahead = walk;
  bool ahead_on = true;
  int ahead_page = 0;         // next page of the segment for this team
  int ahead_half = 0;
  int ahead_at = 32;          // lane that holds it among the fetched ids
  int ids = -1, ids_codes = 0;
  int filled = 0;             // halves issued
  ahead.last = 0;
  int fill_slot = 0;
  uint32_t fill_phase = 0;    // parity of the slot's last release
  bool dead = false;          // a wait gave up: no more copies

  const auto fill = [&]() {  // issues the next half, all lanes of the warp together
    if (!ahead_on || dead) return;
    if (ahead_half == 0) {
      while (ahead_page >= ahead.last) {
        if (!next_segment<C::kRows>(p, ahead)) {
          ahead_on = false;
          return;
        }
        ahead_page = ahead.first + team;
        ahead_at = 32;
      }
      if (ahead_at == 32) {  // the next 32 page ids and codes, one per lane
        const int j = ahead_page + lane * C::kTeams;
        ids = -1;
        ids_codes = 0;
        if (j < ahead.last && ahead.s.kv > 0) {
          const int index = j < ahead.s.sink_pages ? j : ahead.s.lo + (j - ahead.s.sink_pages);
          ids = __ldg(p.page_table + static_cast<size_t>(ahead.b) * p.max_pages + index);
          if (ids < 0 || ids >= p.pages) {
            ids = -1;
            if (p.status) atomicOr(p.status, kKvErrPage);
          } else {
            ids_codes = __ldg(reinterpret_cast<const unsigned short*>(p.codes) +
                              static_cast<size_t>(ids) * p.kv_heads + ahead.head);
          }
        }
        ahead_at = 0;
      }
    }
    const int id = __shfl_sync(0xffffffffu, ids, ahead_at);
    const int cc = __shfl_sync(0xffffffffu, ids_codes, ahead_at);
    if (RW > 1 && filled >= C::kTeamSlots) {
      if (!__all_sync(0xffffffffu, ptx::mbar_wait(empty(fill_slot), fill_phase, abort_flag, kWaitLimitNs))) {
        dead = true;
        if (p.status) atomicOr(p.status, kKvErrTimeout);
        return;
      }
    }
    if (lane == 0) {
      meta[slot0 + fill_slot] = id < 0 ? -1 : cc;
      if (id < 0) {
        ptx::mbar_arrive(full(fill_slot));
      } else {
        ptx::mbar_arrive_expect_tx(full(fill_slot), C::kHalf);
        const size_t owner = (static_cast<size_t>(id) * p.kv_heads + ahead.head) * 2 + ahead_half;
        ptx::bulk_load(sbase + C::kOffRing + (slot0 + fill_slot) * C::kHalf,
                       p.blocks + owner * C::kHalf, C::kHalf, full(fill_slot));
      }
    }
    __syncwarp();
    ++filled;
    if (++fill_slot == C::kTeamSlots) {
      fill_slot = 0;
      if (filled > C::kTeamSlots) fill_phase ^= 1;
    }
    ahead_half ^= 1;
    if (ahead_half == 0) {
      ahead_page += C::kTeams;
      ++ahead_at;
    }
  };
  if (rw == 0)
    for (int i = 0; i < (RW > 1 ? C::kTeamSlots - 1 : C::kTeamSlots); ++i) fill();

  // ---- consume
  int use_slot = 0;
  uint32_t use_phase = 0;
  const auto wait_full = [&]() {
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(full(use_slot), use_phase, abort_flag, kWaitLimitNs))) {
      dead = true;
      if (p.status) atomicOr(p.status, kKvErrTimeout);
      return -1;
    }
    return meta[slot0 + use_slot];
  };
  const auto release = [&]() {  // this warp is done with the half
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

  while (next_segment<C::kRows>(p, walk)) {
    const Seq s = walk.s;
    const int rows = s.n * p.group;  // of the head
    const int row0 = walk.group * C::kRows + rw * NT * 8;

    // ---- the rows: Q as hi + lo E4M3 operands, positions, factors
    uint32_t qf[NT][kKS][4];
    float factor[NT][2];   // raw score -> log2 units, rows 2q and 2q + 1
    int pos[NT][2];
    int pos_lo[NT], pos_hi[NT];
    float m[NT][2], l[NT][2];
    float o[NT][kDT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      float v[kKS][8];
      float amax = 0.0f;
      const bool in = r < rows;
      const __nv_bfloat16* qr =
          p.q + (s.q0 + (in ? r / p.group : 0)) * p.ldq +
          static_cast<long long>(walk.head * p.group + (in ? r % p.group : 0)) * D;
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint2 w = make_uint2(0, 0);
          if (in) w = __ldg(reinterpret_cast<const uint2*>(qr + 32 * k + 16 * h + 4 * q));
          v[k][4 * h] = __uint_as_float(w.x << 16);
          v[k][4 * h + 1] = __uint_as_float(w.x & 0xFFFF0000u);
          v[k][4 * h + 2] = __uint_as_float(w.y << 16);
          v[k][4 * h + 3] = __uint_as_float(w.y & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[k][j]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // the row times 2^a, its largest value in [128, 256)
      const int e = static_cast<int>(__float_as_uint(amax) >> 23);
      const int a = amax > 0.0f ? min(134 - e, 126) : 0;
      const float mul = __uint_as_float(static_cast<uint32_t>(127 + a) << 23);
      const float f = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t hi = 0, lo = 0;
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const float x0 = v[k][4 * h + j] * mul, x1 = v[k][4 * h + j + 1] * mul;
            const uint32_t t = e4m3x2(x0, x1);
            uint32_t h16;
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
                : "=r"(h16)
                : "r"(t));
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h16));
            hi |= t << (8 * j);
            lo |= static_cast<uint32_t>(e4m3x2(x0 - back.x, x1 - back.y)) << (8 * j);
          }
          qf[nt][k][h] = hi;
          qf[nt][k][2 + h] = lo;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        factor[nt][c] = __shfl_sync(0xffffffffu, f, (2 * q + c) * 4);
        const int rc = min(row0 + nt * 8 + 2 * q + c, rows - 1);  // rows past the last see what it sees
        pos[nt][c] = s.kv - s.n + rc / p.group;
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.0f;
      }
      pos_lo[nt] = s.kv - s.n + min(row0 + nt * 8, rows - 1) / p.group;
      pos_hi[nt] = s.kv - s.n + min(row0 + nt * 8 + 7, rows - 1) / p.group;
#pragma unroll
      for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][d][j] = 0.0f;
    }
    const bool idle = row0 >= rows;  // this warp has no rows in the segment

    const auto sees = [&](int token, int at) {
      return token <= at && (p.window == 0 || token > at - p.window || token < p.sinks);
    };

    for (int j = walk.first + team; j < walk.last; j += C::kTeams) {
      const int index = j < s.sink_pages ? j : s.lo + (j - s.sink_pages);
      const int t0 = index * kPageTokens, t1 = t0 + kPageTokens - 1;
      // 0: no row of the tile sees any of the page, 1: every row sees all of it, 2: mixed
      int kind[NT];
      bool any = false, cut = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        kind[nt] = 2;
        if (t1 <= pos_lo[nt] && (p.window == 0 || t0 > pos_hi[nt] - p.window || t1 < p.sinks))
          kind[nt] = 1;
        else if (t0 > pos_hi[nt] ||
                 (p.window > 0 && t1 <= pos_lo[nt] - p.window && t0 >= p.sinks))
          kind[nt] = 0;
        if (idle || row0 + nt * 8 >= rows) kind[nt] = 0;
        any |= kind[nt] != 0;
        cut |= kind[nt] == 2;
      }
      const int mt_k = wait_full();
      const bool on = any && mt_k >= 0;  // (a page id out of range is skipped)
      float sc[NT][4][4];
      if (on) {
        const uint32_t kb = sbase + C::kOffRing + (slot0 + use_slot) * C::kHalf;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[nt][mt][i] = 0.0f;
#pragma unroll
          for (int k = 0; k < kKS; ++k) {
            uint32_t a[4];
            ldsm_x4(kb + (mt * 16 + mrow) * D + (((2 * k + mchunk) ^ kswz) << 4), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_e4m3(sc[nt][mt], a, qf[nt][k][0], qf[nt][k][1]);
              mma_e4m3(sc[nt][mt], a, qf[nt][k][2], qf[nt][k][3]);
            }
          }
        }
      }
      release();

      // ---- softmax of the page
      uint32_t pf[NT][4][2];
      float alpha[NT][2];
      if (on) {
        const float kscale = e8m0_value(mt_k & 0xFF);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (kind[nt] == 2) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!sees(t0 + mt * 16 + g + (i >> 1) * 8, pos[nt][i & 1]))
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
            const float f = factor[nt][c] * kscale;
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
      }

      const int mt_v = wait_full();
      if (on && mt_v >= 0) {
        const uint32_t vb = sbase + C::kOffRing + (slot0 + use_slot) * C::kHalf;
        const float vscale = e8m0_value(mt_v >> 8);
        if (!cut) {
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
#pragma unroll
            for (int cp = 0; cp < 2; ++cp) {
              uint32_t w[4], a0[4], a1[4];
              ldsm_x4(vb + (d * 16 + mrow) * kPageTokens + (((2 * cp + mchunk) ^ vswz) << 4), w);
              e4m3x4_f16(w[0], a0[0], a0[2]);
              e4m3x4_f16(w[1], a0[1], a0[3]);
              e4m3x4_f16(w[2], a1[0], a1[2]);
              e4m3x4_f16(w[3], a1[1], a1[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(acc[nt], a0, pf[nt][2 * cp][0], pf[nt][2 * cp][1]);
                mma_f16(acc[nt], a1, pf[nt][2 * cp + 1][0], pf[nt][2 * cp + 1][1]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (kind[nt] != 0)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  o[nt][d][i] = fmaf(o[nt][d][i], alpha[nt][i & 1], acc[nt][i] * vscale);
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
                keep[c] = (sees(t, at) ? 0x000000FFu : 0u) | (sees(t + 1, at) ? 0x0000FF00u : 0u) |
                          (sees(t + 8, at) ? 0x00FF0000u : 0u) | (sees(t + 9, at) ? 0xFF000000u : 0u);
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

    // ---- the segment's rows: join the teams, then write them out or to the workspace
    const bool whole = walk.first == 0 && walk.last == s.pages;
    const long long c0 = walk.item_start / per;
    const int part_slot = static_cast<int>(blockIdx.x == c0);
    float* part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + part_slot) * C::kRows * (D + 2);
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
        const int r = walk.group * C::kRows + (w * NT + nt) * 8 + row;
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
          const int token = s.q0 + r / p.group, head = walk.head * p.group + r % p.group;
          const size_t at_out = static_cast<size_t>(token) * (p.kv_heads * p.group) + head;
          const float inv = den == 0.0f ? 0.0f : 1.0f / den;
          __align__(8) __nv_bfloat162 y[2] = {__floats2bfloat162_rn(sum.x * inv, sum.y * inv),
                                              __floats2bfloat162_rn(sum.z * inv, sum.w * inv)};
          *reinterpret_cast<uint2*>(p.out + at_out * D + d4 * 4) = *reinterpret_cast<const uint2*>(y);
          if (d4 == 0 && p.lse)
            p.lse[at_out] = den == 0.0f ? -INFINITY : (top + log2f(den) - kLog2P) * 0.69314718055994531f;
        } else {
          const int lr = (w * NT + nt) * 8 + row;
          *reinterpret_cast<float4*>(part + static_cast<size_t>(lr) * D + d4 * 4) = sum;
          if (d4 == 0)
            *reinterpret_cast<float2*>(part + static_cast<size_t>(C::kRows) * D + 2 * lr) = make_float2(top, den);
        }
      }
      __syncthreads();
    }
    if (whole) continue;

    // ---- an item of several CTAs: the last to arrive joins their partial rows
    const long long item_end = walk.item_start + s.pages;
    const int c1 = static_cast<int>((item_end - 1) / per);
    if (tid == 0) {
      __threadfence();
      const int done = atomicAdd(p.tickets + c0, 1);
      const int last = done == c1 - static_cast<int>(c0);
      if (last) {
        p.tickets[c0] = 0;
        __threadfence();
      }
      *last_flag = last;
    }
    __syncthreads();
    if (*last_flag) {
      for (int lr = warp; lr < C::kRows; lr += C::kWarps) {
        const int r = walk.group * C::kRows + lr;
        if (r >= rows) break;
        const auto partial = [&](int c) {
          return p.part + (static_cast<size_t>(c) * 2 + (c == c0)) * C::kRows * (D + 2);
        };
        float top = -INFINITY;
        for (int c = static_cast<int>(c0) + lane; c <= c1; c += 32)
          top = fmaxf(top, __ldcg(partial(c) + C::kRows * D + 2 * lr));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        float den = 0.0f;
        float sum[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) sum[i] = 0.0f;
        for (int cb = static_cast<int>(c0); cb <= c1; cb += 32) {
          float w = 0.0f, lw = 0.0f;
          if (cb + lane <= c1) {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(partial(cb + lane) + C::kRows * D) + lr);
            w = top == -INFINITY ? 0.0f : ex2(x.x - top);
            lw = x.y * w;
          }
          const int count = min(32, c1 - cb + 1);
#pragma unroll 4
          for (int k = 0; k < count; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            den += __shfl_sync(0xffffffffu, lw, k);
            const float* src = partial(cb + k) + static_cast<size_t>(lr) * D + lane * (D / 32);
#pragma unroll
            for (int i = 0; i < D / 32; i += 2) {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(src + i));
              sum[i] = fmaf(x.x, wk, sum[i]);
              sum[i + 1] = fmaf(x.y, wk, sum[i + 1]);
            }
          }
        }
        const int token = s.q0 + r / p.group, head = walk.head * p.group + r % p.group;
        const size_t at_out = static_cast<size_t>(token) * (p.kv_heads * p.group) + head;
        const float inv = den == 0.0f ? 0.0f : 1.0f / den;
#pragma unroll
        for (int i = 0; i < D / 32; i += 2)
          *reinterpret_cast<__nv_bfloat162*>(p.out + at_out * D + lane * (D / 32) + i) =
              __floats2bfloat162_rn(sum[i] * inv, sum[i + 1] * inv);
        if (lane == 0 && p.lse)
          p.lse[at_out] = den == 0.0f ? -INFINITY : (top + log2f(den) - kLog2P) * 0.69314718055994531f;
      }
    }
  }

  // Every copy issued has been waited for, as each half of the run is
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
cudaError_t launch(const AttnX8Params& p, int grid, cudaStream_t s) {
  using C = Cfg<D, NT, RW>;
  const cudaError_t e = cudaFuncSetAttribute(attn_x8_kernel<D, NT, RW>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_x8_kernel<D, NT, RW>, dim3(grid), dim3(C::kThreads), C::kSmem, s, p);
}

}  // namespace attn
}  // namespace moe
