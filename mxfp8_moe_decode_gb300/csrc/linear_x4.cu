// Products with 4-bit weights: out[m, n] = bf16(sum_k x[m, k] w[n, k]) for MXFP4
// rows w (E2M1 with one E8M0 code per 32 columns) and rows x in MXFP8 or bf16.
//
// Both operands go to the block-scaled tensor cores as they are (tcgen05
// kind::mxf8f6f4, E2M1 against E4M3): products and their scales are exact, sums
// fp32. bf16 rows become two MXFP8 rows first: with the group's code c, hi =
// E4M3(x 2^(127 - c)) and lo = E4M3(16 (x 2^(127 - c) - hi)) under the code c - 4.
// bf16 has 8 significant bits, hi takes 4 and the rest, at most half a step of
// hi, fits lo's 4 while x 2^(127 - c) is at least 2^-6, E4M3's smallest normal
// value: exact down to 2^-13 of the group's largest value, which lies above 224.
// Below, lo's steps are 2^-13: off by half of one, 2^-21 of the largest, at most.
//
// Swap-AB: 128 weight rows are the MMA's M and up to 192 token rows its N, so
// few tokens still fill the tensor cores' lanes, and the weights stream once
// for up to 192 rows.
//
// A persistent CTA an SM, its warps by role around one ring of K blocks (128
// columns): one thread copies weights (a 4-bit tensor copy that spreads the
// codes as the tensor cores read them) and rows; warps gather the scale codes
// from global memory into the images that tcgen05.cp takes; one or two threads
// issue copies of scales and products; four warps take the sums out of TMEM.
// Where a call has fewer tiles than SMs, a cluster shares a tile's K and sums
// its parts in an exchange over distributed shared memory, in the order of the
// ranks. choose_shape weighs tile heights and shares.
//
// What bounds it, and what it takes (graph replays of calls back to back, weights
// from HBM; one by one from Python 0.3 to 0.6 us more):
//  7 rows, 5120 -> 129281 columns (352 MB): the weights' stream, 55 us (6.4 TB/s)
//  48 rows, 5120 -> 27648: 18.1 us, of which the stream is 11; the rest is the
//    start, a CTA's last tile and the exchange
//  1 row, 5120 -> 7168: 7.6 us. The stream is 2.9; 1.7 are a launch's, 1.1 the
//    first codes and weights, 1.3 the exchange and the end, and a K block takes
//    some 100 to 170 ns however few columns it has: one thread issues at most a
//    block in 300, two half of that, four (a ring of 8 slots) no better
//  4000 rows, 5120 -> 7168: 104 us in a short burst (2070 MHz, 2830 TFLOP/s), 112 to
//    116 in a long run, which the power cap slows (1680 to 1970 MHz, 2530 to 2630);
//    bf16 rows (two products) 199 and 214. The tensor cores work 64 % of the time (two
//    accumulators of 192 columns fill TMEM, so one thread issues), shared memory 62 %
// Slower: weights by plain loads through registers (7 rows above: 133 us) or by
// cp.async and warps that spread the codes (91 to 107; shared memory's port);
// pairs of CTAs that share the rows' copies by multicast (no change); tiles of 160
// rows at most (4000 rows above, then 117 us: 141); the whole warp in the
// issuing loop, fences with the writers, 4 blocks' scales at once (none faster).
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "internal.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kTileN = 128;      // weight rows of a tile (MMA M)
constexpr int kMaxRows = 192;    // token rows of a tile (MMA N): two accumulators and the scales fit TMEM
constexpr int kMaxTasks = 1 << 30;
constexpr int kMaxSlots = 12;
constexpr int kMaxCluster = 8;
constexpr int kStep = 2;         // a CTA's share of K begins at a multiple of so many K blocks (of 128)
constexpr int kGroup = 4;        // K blocks whose scale codes are loaded at once: 16 bytes of a row
// Warps by role. Several warps that take the ring's blocks in turn (issuers,
// rows' codes) are an even number no larger than the slots', which is even too:
// a warp's blocks then have one issuer, which frees them in order, and it has
// seen its last one freed, less than a round before. (A warp that had missed a
// phase of a slot could take its parity for the one it waits for.)
// The rows' codes come last, as many warps as the launch has left.
constexpr int kIssuer = 4, kCodesW = 6, kCopy = 8, kRowsX = 9;  // (epilogue: 0-3)
constexpr int threads_of(bool raw) { return 32 * (kRowsX + (raw ? 8 : 4)); }  // at most
constexpr uint32_t kABytes = kTileN * 128;
constexpr uint32_t kImg = 512;   // scale image of 128 rows and one K block
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSmemMax = 227 * 1024;

struct LinearParams {
  CUtensorMap tm_x;      // the rows' parts: [K / 128][part][M][128]; bf16 rows (kRaw): [K / 64][M][128 bytes]
  CUtensorMap tm_w;      // the weights: [K / 128][N][128 of 4 bits], a box one K block of a tile
  const uint8_t* wc;     // [N][K / 32]
  const uint8_t* xc[2];  // [M][K / 32]
  __nv_bfloat16* out;
  long long ldo;
  int* status;
  int M, N, K;
  int nt;                // token rows of a tile (a multiple of 16, stacked of 8)
  int tiles_m, tasks;
  int parts;             // 1 (MXFP8 rows) or 2 (bf16 rows as hi and lo)
  int stacked;           // two parts as columns of one product (few rows), else as two products
  int cols;              // columns of a product (MMA N): nt, stacked 2 nt
  int slots;             // of the ring: a K block's weights, rows and scale images each
  int code_warps;        // warps that make the weights' scale images (1 or 2)
  int issuers;           // 1 or 2, each with its own accumulators
  int accs;              // of an issuer: 2 in turn, or 1 where a CTA has one tile only
  int turns;             // one product: warps that take its rows' codes in turn (1, 2 or 4)
  int split;             // CTAs (a cluster) that share a tile's K
  int early;             // the kernel before made the rows' parts: weights may be read while it runs
  uint32_t off_b, slot_b, off_img, slot_img, off_xchg, off_bar;
};

struct Bars {
  uint64_t full[kMaxSlots];   // a K block's weights, rows and images are there
  uint64_t raw[kMaxSlots];    // its bf16 rows are there
  uint64_t empty[kMaxSlots];  // its MMAs have read them
  uint64_t tfull[2], tempty[2];
  uint64_t efree;             // every CTA of the cluster has its exchange buffer free
  uint64_t efull;             // this CTA's exchange buffer is full
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

using ptx::elect_one;
using ptx::mbar_wait_clocks;

// What a CTA goes through: its cluster's tiles, and of each the same K blocks
// (its share of K, from an even one on).
struct Work {
  int first, step;  // tiles
  int rank;
  int nk, k0, k1;
};

__device__ __forceinline__ Work work_of(const LinearParams& p) {
  Work w;
  const int S = p.split;
  w.first = static_cast<int>(blockIdx.x) / S;
  w.step = static_cast<int>(gridDim.x) / S;
  w.rank = static_cast<int>(blockIdx.x) - w.first * S;
  w.nk = p.K / 128;
  const int steps = (w.nk + kStep - 1) / kStep;
  w.k0 = kStep * (steps * w.rank / S);
  w.k1 = min(kStep * (steps * (w.rank + 1) / S), w.nk);
  return w;
}

__device__ __forceinline__ int tile_n(const LinearParams& p, int t) { return t / p.tiles_m * kTileN; }
__device__ __forceinline__ int tile_m(const LinearParams& p, int t) { return t % p.tiles_m * p.nt; }

// A place in the ring, and the parity of its present phase.
struct Slot {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n, uint32_t by) {
    at += by;
    if (at >= n) {
      at -= n;
      phase ^= 1;
    }
  }
};

// 4 K blocks' codes of one row (word j: the block 4 g + j), as 16 bytes where a
// row's codes are 16-byte aligned; the 128 bytes around them come to L2 too.
__device__ __forceinline__ uint4 load_codes(const uint8_t* row, int g, int nk, bool wide) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (wide) {
    asm volatile("ld.global.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(reinterpret_cast<const uint4*>(row) + g));
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + kGroup * g;
    const int n = nk - kGroup * g;
    v.x = __ldg(w);
    if (n > 1) v.y = __ldg(w + 1);
    if (n > 2) v.z = __ldg(w + 2);
    if (n > 3) v.w = __ldg(w + 3);
  }
  return v;
}

template <int kImages>
struct Codes {
  uint4 v[kImages][4];
};

template <int kImages>
__device__ __forceinline__ void load_group(const LinearParams& p, const Work& w, int part, bool wide, int t, int g,
                                           Codes<kImages>& c) {
  const int lane = threadIdx.x & 31;
  const int r0 = tile_m(p, t), rows = min(p.M - r0, p.nt);
  const long long pitch = p.K / 32;
#pragma unroll
  for (int i = 0; i < kImages; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      int r = 128 * i + 32 * q + lane;
      const uint8_t* from = p.xc[part];
      if (p.stacked && r >= p.nt) {  // lo behind hi
        r -= p.nt;
        from = p.xc[1];
      }
      c.v[i][q] = make_uint4(0, 0, 0, 0);
      if (r < rows) c.v[i][q] = load_codes(from + (r0 + r) * pitch, g, w.nk, wide);
    }
}

__device__ __forceinline__ uint32_t word(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// A K block's scale image as tcgen05.cp reads it: lane i's 16 bytes hold the 4
// codes each of the rows i, 32 + i, 64 + i, 96 + i.
__device__ __forceinline__ void store_image(uint8_t* img, const uint4 (&v)[4], int j) {
  *reinterpret_cast<uint4*>(img) = make_uint4(word(v[0], j), word(v[1], j), word(v[2], j), word(v[3], j));
}

// The weights' scale images by one warp, or by two that take the groups of 4 K
// blocks in turn (code_warps_of says when); the next group's codes are on their
// way meanwhile.
__device__ __forceinline__ void weight_codes(const LinearParams& p, const Work& w, Bars* bars, uint8_t* smem, int turn) {
  const int lane = threadIdx.x & 31, turns = p.code_warps;
  volatile int* abort = &bars->abort;
  const bool wide = p.K % 512 == 0 && (reinterpret_cast<uintptr_t>(p.wc) & 15) == 0;
  const long long pitch = p.K / 32;
  const int g0 = w.k0 / kGroup, g1 = (w.k1 + kGroup - 1) / kGroup;
  int t = w.first, g = g0;  // of the group to load next
  const auto fetch = [&](uint4 (&v)[4]) {
    const int n0 = tile_n(p, t);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = make_uint4(0, 0, 0, 0);
      const int n = n0 + 32 * q + lane;
      if (n < p.N) v[q] = load_codes(p.wc + n * pitch, g, w.nk, wide);
    }
  };
  const auto advance = [&](int n) {
    for (g += n; g >= g1; g -= g1 - g0) t += w.step;
  };
  uint4 next[4];
  advance(turn);
  if (!p.early) ptx::griddep_wait();
  if (t < p.tasks) fetch(next);
  Slot slot;
  uint8_t* base = smem + p.off_img + lane * 16;
  const uint32_t empty0 = ptx::smem_u32(bars->empty), full0 = ptx::smem_u32(bars->full), R = p.slots;
  int at = turn;  // of this warp's next group in the present tile
  for (int u = w.first; u < p.tasks; u += w.step) {
    int k = w.k0;
    for (; at < g1 - g0; at += turns) {
      const int begin = max(w.k0, (g0 + at) * kGroup), end = min(w.k1, (g0 + at + 1) * kGroup);
      if (begin > k) slot.next(R, begin - k);  // (at most a group's: the other warp's)
      uint4 now[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) now[q] = next[q];
      advance(turns);
      if (t < p.tasks) fetch(next);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const int kj = (g0 + at) * kGroup + j;
        if (kj < begin || kj >= end) continue;
        if (!__all_sync(0xffffffffu, mbar_wait_clocks(empty0 + slot.at * 8, slot.phase ^ 1, abort))) return;
        store_image(base + slot.at * p.slot_img, now, j);
        __syncwarp();
        if (elect_one()) ptx::mbar_arrive(full0 + slot.at * 8);
        slot.next(R, 1);
      }
      k = end;
    }
    if (w.k1 > k) slot.next(R, w.k1 - k);
    at -= g1 - g0;
  }
}

// The scale images of a product's rows, of the part `part`, by one warp, or by
// `turns` in turn, this one `turn`. Codes are loaded 4 K blocks at a time, one
// such group ahead.
template <int kImages>
__device__ __forceinline__ void row_codes(const LinearParams& p, const Work& w, Bars* bars, uint8_t* smem, int part,
                                          int turn, int turns) {
  const int lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  const bool wide = p.K % 512 == 0 && (reinterpret_cast<uintptr_t>(p.xc[part]) & 15) == 0;  // (the workspace's are aligned)
  uint8_t* base = smem + p.off_img + (1 + part * kImages) * kImg + lane * 16;
  const int g0 = w.k0 / kGroup;
  ptx::griddep_wait();
  Codes<kImages> next;  // (of two images' rows only the present group is held)
  if (kImages == 1 && w.first < p.tasks) load_group<kImages>(p, w, part, wide, w.first, g0, next);
  Slot slot;
  slot.at = turn;
  const uint32_t empty0 = ptx::smem_u32(bars->empty), full0 = ptx::smem_u32(bars->full), R = p.slots;
  int k = w.k0 + turn;  // this warp's next block in the present tile
  int next_t = w.first, next_g = g0;
  for (int t = w.first; t < p.tasks; t += w.step) {
    Codes<kImages> now;
    for (int have = -1; k < w.k1; k += turns, slot.next(R, turns)) {
      if (k / kGroup != have) {
        have = k / kGroup;
        if (kImages == 1 && next_t == t && next_g == have)
          now = next;
        else  // (not guessed: the other warp had all the blocks in between)
          load_group<kImages>(p, w, part, wide, t, have, now);
        if (kImages == 1) {
          next_t = (have + 1) * kGroup < w.k1 ? t : t + w.step;
          next_g = next_t == t ? have + 1 : g0;
          if (next_t < p.tasks) load_group<kImages>(p, w, part, wide, next_t, next_g, next);
        }
      }
      const int j = k % kGroup;
      if (!__all_sync(0xffffffffu, mbar_wait_clocks(empty0 + slot.at * 8, slot.phase ^ 1, abort))) return;
      uint8_t* dst = base + slot.at * p.slot_img;
#pragma unroll
      for (int m = 0; m < kImages; ++m) store_image(dst + m * kImg, now.v[m], j);
      __syncwarp();
      if (elect_one()) ptx::mbar_arrive(full0 + slot.at * 8);
    }
    k += w.k0 - w.k1;
  }
}

// A K block's bf16 rows in a slot, in place, to its hi and lo rows, and their
// images. The copy brings every row as two halves of 64 columns, hi's bytes of a
// row come where the first half was, lo's where the second was: 8 rows a step,
// a lane a row's 32 columns of one code.
__device__ __forceinline__ void split_block(uint8_t* b, uint8_t* img, int nt, int rows, int first) {
  const int lane = threadIdx.x & 31, r = lane & 7, g = lane >> 3;  // (so 8 lanes' chunks lie in 8 columns of banks)
  for (int row = first + r; row < rows + r; row += 16) {
    const uint8_t* from = b + ((g >> 1) * nt + row) * 128;
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 u = *reinterpret_cast<const uint4*>(from + (((g & 1) * 4 + j) ^ r) * 16);
      w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
    }
    __syncwarp();
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
    if (__any_sync(0xffffffffu, max(top >> 16, top & 0xFFFFu) >= 0x7F80u)) {  // values that are not finite: NaN, and not looked at
      top = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t m = w[j] & 0x7FFF7FFFu, finite = __vcmpltu2(m, 0x7F807F80u);
        top = __vmaxu2(top, m & finite);
        w[j] = (w[j] & finite) | (0x7FFF7FFFu & ~finite);
      }
    }
    // (rows past the last, zeros, some code: the division by 448 is slow at the smallest values)
    const int code = mx_code(row < rows ? __uint_as_float(max(top >> 16, top & 0xFFFFu) << 16) : 1.0f), low = max(code - 4, 0);
    const float mul = mx_mul(code);
    const __half2 up = __float2half2_rn(static_cast<float>(1 << (code - low)));
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t h2[2], l2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = w[2 * j + i];
        // (f16 holds what the two parts can: 448 and below, in steps of 2^-24)
        const __half2 v = __floats2half2_rn(__uint_as_float(x << 16) * mul, __uint_as_float(x & 0xFFFF0000u) * mul);
        const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
        const __half2 rest = __hmul2(__hsub2(v, __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3))), up);
        h2[i] = h;
        l2[i] = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(rest), __NV_SATFINITE, __NV_E4M3);
      }
      hi[j] = h2[0] | (h2[1] << 16);
      lo[j] = l2[0] | (l2[1] << 16);
    }
    uint8_t* to = b + row * 128;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = ((2 * g + i) ^ r) * 16;
      *reinterpret_cast<uint4*>(to + at) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
      *reinterpret_cast<uint4*>(to + nt * 128 + at) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
    }
    const int c = nt + row;
    img[(row & 31) * 16 + (row >> 5) * 4 + g] = static_cast<uint8_t>(code);
    img[(c & 31) * 16 + (c >> 5) * 4 + g] = static_cast<uint8_t>(low);
  }
}

// The bf16 rows' warps, which take the blocks in turn.
__device__ __forceinline__ void split_rows(const LinearParams& p, const Work& w, Bars* bars, uint8_t* smem, int who) {
  const int turn = who >> 1;
  volatile int* abort = &bars->abort;
  const uint32_t empty0 = ptx::smem_u32(bars->empty), full0 = ptx::smem_u32(bars->full), raw0 = ptx::smem_u32(bars->raw),
                 R = p.slots;
  Slot slot;
  slot.at = turn;
  int k = w.k0 + turn;
  for (int t = w.first; t < p.tasks; t += w.step) {
    const int rows = min(p.M - tile_m(p, t), p.nt);
    for (; k < w.k1; k += p.turns, slot.next(R, p.turns)) {
      // (the slot is free, so its copy before has come: the other phase of that parity cannot be taken for this one)
      const bool ok = mbar_wait_clocks(empty0 + slot.at * 8, slot.phase ^ 1, abort) &&
                      mbar_wait_clocks(raw0 + slot.at * 8, slot.phase, abort);
      if (!__all_sync(0xffffffffu, ok)) return;
      split_block(smem + p.off_b + slot.at * p.slot_b, smem + p.off_img + slot.at * p.slot_img + kImg, p.nt, rows, 8 * (who & 1));
      __syncwarp();
      if (elect_one()) ptx::mbar_arrive(full0 + slot.at * 8);
    }
    k += w.k0 - w.k1;
  }
}

// What the loops of single threads go by is fixed when the kernel is compiled:
// kRaw: the copies bring bf16 rows, and the kernel takes them apart itself (a
//   switch in the loops: 7 rows, 129281 columns 64 us in place of 57);
// kProducts of a K block, kHimg scale images of a product's columns (values read
//   from the parameters: 1 row 7.9 us in place of 7.7, 4000 rows 110 in place of 102).
template <bool kRaw, int kProducts, int kHimg>
__global__ void __launch_bounds__(threads_of(kRaw), 1) linear_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - (ptx::smem_u32(smem_raw) & 1023)) % 1024;
  const uint32_t sbase = ptx::smem_u32(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + p.off_bar);
  volatile int* abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
  const int S = p.split;
  const Work w = work_of(p);

  if (warp == 0) {
    if (lane < kMaxSlots) {
      ptx::mbar_init(bar(bars->full[lane]), 2 + (kRaw ? 2 : kProducts));  // the copies, the weights' images, each product's rows'
      if (kRaw) ptx::mbar_init(bar(bars->raw[lane]), 1);
      ptx::mbar_init(bar(bars->empty[lane]), 1);
    } else if (lane >= 16 && lane < 18) {
      ptx::mbar_init(bar(bars->tfull[lane - 16]), p.issuers);
      ptx::mbar_init(bar(bars->tempty[lane - 16]), 4);
    } else if (lane == 18) {
      ptx::mbar_init(bar(bars->efree), 4 * S);
    } else if (lane == 19) {
      ptx::mbar_init(bar(bars->efull), 1);
    } else if (lane == 20) {
      ptx::mbar_init(bar(bars->drain), p.issuers);
    } else if (lane == 21) {
      bars->abort = 0;
    }
    ptx::fence_mbar_init();
  } else if (warp == kIssuer) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem), kTmemCols);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  } else if (warp == kCopy && elect_one()) {
    ptx::prefetch_tmap(&p.tm_w);
    ptx::prefetch_tmap(&p.tm_x);
  }
  __syncwarp();
  __syncthreads();
  ptx::tc_fence_after();
  if (S > 1) {  // the others' barriers are there
    ptx::cluster_arrive();
    ptx::cluster_wait();
  }
  if (warp == 0) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
  }

  bool arrived = false;
  // (what reads the kernel before's results waits for it in its own branch)
  if (warp >= kCodesW && warp < kCodesW + p.code_warps) {
    weight_codes(p, w, bars, smem, warp - kCodesW);
  } else if (warp >= kRowsX) {
    const int who = warp - kRowsX, part = kProducts > 1 ? who : 0;
    const int turn = kProducts > 1 ? 0 : who, turns = kProducts > 1 ? 1 : p.turns;
    if (kRaw)
      split_rows(p, w, bars, smem, who);
    else if (kHimg == 1)
      row_codes<1>(p, w, bars, smem, part, turn, turns);
    else
      row_codes<2>(p, w, bars, smem, part, turn, turns);
  } else if (warp == kCopy) {
    // ------------------------------------------------------------ copies
    // A 4-bit box spreads its codes as the tensor cores read E2M1 rows: 16 (8
    // bytes) in a unit of 16 bytes, whose other half is not looked at. One
    // thread keeps the ring full (3, 4 or 5 warps in turn: no faster).
    if (elect_one()) {
      const uint64_t keep = ptx::policy_evict_last();
      const uint64_t policy = p.tiles_m > 1 ? ptx::policy_evict_normal() : ptx::policy_evict_first();
      const uint32_t empty0 = bar(bars->empty[0]), full0 = bar(bars->full[0]), raw0 = bar(bars->raw[0]), R = p.slots;
      Slot slot;
      int k = w.k0;
      const auto copy_w = [&](int n0, int at) {
        ptx::mbar_arrive_expect_tx(full0 + slot.at * 8, kABytes / 2 + (kRaw ? 0 : p.slot_b));  // (a 4-bit box counts its global bytes)
        ptx::tma_load_3d(sbase + slot.at * kABytes, &p.tm_w, 0, n0, at, full0 + slot.at * 8, policy);
      };
      const auto copy_x = [&](int m0, int at) {
        if (kRaw) {
          ptx::mbar_arrive_expect_tx(raw0 + slot.at * 8, p.slot_b);
          ptx::tma_load_3d(sbase + p.off_b + slot.at * p.slot_b, &p.tm_x, 0, m0, 2 * at, raw0 + slot.at * 8, keep);
          return;
        }
        ptx::tma_load_4d(sbase + p.off_b + slot.at * p.slot_b, &p.tm_x, 0, m0, 0, at, full0 + slot.at * 8, keep);
      };
      bool ok = true;
      if (w.first < p.tasks) {  // the ring's first round, all its slots empty
        const int n0 = tile_n(p, w.first), m0 = tile_m(p, w.first), end = min(w.k1, w.k0 + static_cast<int>(R));
        if (!p.early) ptx::griddep_wait();
        for (int at = k; at < end; ++at, ++slot.at) copy_w(n0, at);
        if (p.early) ptx::griddep_wait();
        slot.at = 0;
        for (; k < end; ++k, slot.next(R, 1)) copy_x(m0, k);
      }
      for (int t = w.first; ok && t < p.tasks; t += w.step) {
        const int n0 = tile_n(p, t), m0 = tile_m(p, t);
        for (; k < w.k1; ++k, slot.next(R, 1)) {
          if (!mbar_wait_clocks(empty0 + slot.at * 8, slot.phase ^ 1, abort)) {
            ok = false;
            break;
          }
          copy_w(n0, k);
          copy_x(m0, k);
        }
        k = w.k0;
      }
    }
    __syncwarp();
  } else if (warp >= kIssuer && warp < kIssuer + p.issuers) {
    // ------------------------------------------------------------ MMA issuers
    if (elect_one()) {
      const uint32_t me = warp - kIssuer, tmem = bars->tmem;
      // A K block's scale columns in TMEM, by its slot: 4 of the weights, then 4
      // kHimg of each product's rows. (The products take them from a column that
      // is a multiple of 4 only.)
      const uint32_t sfx = 4 * kHimg, sf_slot = 4 + kProducts * sfx;
      const uint32_t sf0 = tmem + p.accs * p.issuers * p.cols;
      const uint32_t part_units = static_cast<uint32_t>(p.nt) * 8u;  // of 16 bytes, as descriptors count
      const uint32_t idesc = ptx::idesc_mxf8(p.cols, 0, ptx::kFmtE2M1), idesc_k = ptx::idesc_mxf8(0, 1, 0) - ptx::idesc_mxf8(0, 0, 0);
      const uint64_t a0 = ptx::sdesc_k128_sw128(sbase), b0 = ptx::sdesc_k128_sw128(sbase + p.off_b),
                     i0 = ptx::sdesc_rows16(sbase + p.off_img);
      const uint32_t empty0 = bar(bars->empty[0]), full0 = bar(bars->full[0]), R = p.slots, turns = p.issuers;
      const uint32_t slot_b = p.slot_b >> 4, slot_img = p.slot_img >> 4;
      uint32_t acc = 0, acc_phase = 1;
      Slot slot;
      slot.at = me;
      int k = w.k0 + static_cast<int>(me);  // this issuer's next block in the present tile
      bool ok = true;
      for (int t = w.first; ok && t < p.tasks; t += w.step) {
        if (!mbar_wait_clocks(bar(bars->tempty[acc]), acc_phase, abort)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + (acc * p.issuers + me) * p.cols;
        uint32_t some = 0;
        for (; k < w.k1; k += turns, slot.next(R, turns)) {
          if (!mbar_wait_clocks(full0 + slot.at * 8, slot.phase, abort)) {
            ok = false;
            break;
          }
          // The images that other warps wrote, to the tensor cores' view of
          // shared memory.
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_after();
          const uint64_t a = a0 + slot.at * (kABytes >> 4), img = i0 + slot.at * slot_img;
          uint64_t b = b0 + slot.at * slot_b;
          const uint32_t sfa = sf0 + slot.at * sf_slot;
          ptx::tc_cp_32x128b_x4(sfa, img);
#pragma unroll
          for (int h = 0; h < kProducts; ++h, b += part_units) {
            const uint32_t sx = sfa + 4 + h * sfx;
#pragma unroll
            for (int i = 0; i < kHimg; ++i)
              ptx::tc_cp_32x128b_x4(sx + 4 * i, img + (1 + h * kHimg + i) * (kImg >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              ptx::tc_mma_mxf8(d, a + 2 * kk, b + 2 * kk, idesc + kk * idesc_k, sfa, sx, some);
              some = 1;
            }
          }
          ptx::tc_commit(empty0 + slot.at * 8);
        }
        if (ok) ptx::tc_commit(bar(bars->tfull[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
        k += w.k0 - w.k1;
      }
      // everything this thread issued has completed once drain fires
      ptx::tc_commit(bar(bars->drain));
      int never = 0;
      mbar_wait_clocks(bar(bars->drain), 0, &never);
    }
    __syncwarp();
  } else if (warp < kIssuer) {
    // ------------------------------------------------------------ epilogue
    // Warp q holds the tile's weight rows 32 q .. 32 q + 31, one a lane.
    // A warp whose wait ran out goes on to the next tile's barrier, where all
    // four give up together.
    const auto all_ok = [](bool ok) {
      uint32_t all;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(all)
          : "r"(static_cast<uint32_t>(ok))
          : "memory");
      return all != 0;
    };
    const uint32_t lanes = bars->tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const int per = (p.nt / 4 + S - 1) / S;  // groups of 4 columns that a CTA of the cluster sums
    const uint32_t xchg = sbase + p.off_xchg + tid * 16;
    const bool over = p.off_xchg == 0;
    int lt = 0;
    bool ok = true;
    for (int t = w.first; t < p.tasks; t += w.step, ++lt) {
      const int n = tile_n(p, t) + tid, m0 = tile_m(p, t);
      const int cols = min(p.nt, p.M - m0);
      const int acc = lt & 1;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_clocks(bar(bars->tfull[acc]), (lt >> 1) & 1, abort));
      if (S > 1 ? !all_ok(ok) : !ok) break;
      ptx::tc_fence_after();
      // the issuers' accumulators (one, if the tile had a single K block: its issuer's)
      const uint32_t d0 = lanes + acc * p.issuers * p.cols;
      const bool two = p.issuers > 1 && w.k1 - w.k0 > 1;
      const uint32_t d = d0 + (p.issuers > 1 && !two ? (lt & 1) * p.cols : 0);
      const int sums = (two ? 2 : 1) * (p.stacked ? 2 : 1), apart = p.stacked ? p.nt : p.cols;
      const auto load = [&](int c0, float* v) {  // the issuers' sums, and hi's and lo's, in this order
        ptx::tmem_ld_32x32b_x16(d + c0, v);
        ptx::tmem_wait_ld();
        for (int i = 1; i < sums; ++i) {  // (all four at once: 128 registers, and 1 us slower)
          float u[16];
          ptx::tmem_ld_32x32b_x16(d + i * apart + c0, u);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += u[j];
        }
      };
      __nv_bfloat16* out = p.out + static_cast<long long>(m0) * p.ldo + n;
      if (S == 1) {
        for (int c0 = 0; c0 < cols; c0 += 16) {
          float v[16];
          load(c0, v);
          if (n < p.N) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + j < cols) out[(c0 + j) * p.ldo] = __float2bfloat16_rn(v[j]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars->tempty[acc]));
        continue;
      }
      // Columns 4 c .. 4 c + 3 of the tile are summed by the CTA c % S: every CTA
      // sends its parts of the columns to their CTAs, and adds up those it gets
      // in the order of the ranks. Its warps say when the buffer is free: over
      // the ring, when all MMAs are done; else when the last tile's sums are read.
      if (over && lane < S) ptx::mbar_arrive_cluster(ptx::cluster_addr(bar(bars->efree), lane));
      if (over || lt > 0) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar(bars->efree), (over ? 0 : lt - 1) & 1, abort));
        if (!ok) continue;
      }
      const int groups = (cols + 3) / 4, own = groups > w.rank ? (groups - w.rank + S - 1) / S : 0;
      if (tid == 0) ptx::mbar_arrive_expect_tx(bar(bars->efull), static_cast<uint32_t>(own * S) * 2048u);
      int owner = 0;
      uint32_t at = xchg + w.rank * per * 2048;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        load(c0, v);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          if (c0 + j < cols) {
            ptx::st_async_v4(ptx::cluster_addr(at, owner), v[j], v[j + 1], v[j + 2], v[j + 3],
                             ptx::cluster_addr(bar(bars->efull), owner));
            if (++owner == S) {
              owner = 0;
              at += 2048;
            }
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(bars->tempty[acc]));
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar(bars->efull), lt & 1, abort));
      if (!ok) continue;
      if (t + w.step >= p.tasks) {  // all is sent and all has come
        ptx::cluster_arrive();
        arrived = true;
      }
      if (n < p.N) {
        const float4* part = reinterpret_cast<const float4*>(smem + p.off_xchg) + tid;
        for (int c = 4 * w.rank; c < cols; c += 4 * S, part += 128) {
          float4 sum = part[0];
          for (int r = 1; r < S; ++r) {
            const float4 u = part[r * per * 128];
            sum.x += u.x;
            sum.y += u.y;
            sum.z += u.z;
            sum.w += u.w;
          }
          __nv_bfloat16* o = out + c * p.ldo;
          o[0] = __float2bfloat16_rn(sum.x);
          if (c + 1 < cols) o[p.ldo] = __float2bfloat16_rn(sum.y);
          if (c + 2 < cols) o[2 * p.ldo] = __float2bfloat16_rn(sum.z);
          if (c + 3 < cols) o[3 * p.ldo] = __float2bfloat16_rn(sum.w);
        }
      }
      if (!over && t + w.step < p.tasks) {
        __syncwarp();
        if (lane < S) ptx::mbar_arrive_cluster(ptx::cluster_addr(bar(bars->efree), lane));
      }
    }
  }

  // ------------------------------------------------------------ teardown
  // In a cluster nobody ends before all others have sent what they send.
  if (S > 1 && !arrived) ptx::cluster_arrive();
  ptx::tc_fence_before();
  __syncthreads();
  if (*abort) {
    if (tid == 0) {
      if (p.status) atomicOr(p.status, MOE_LINEAR_STATUS_TIMEOUT);
      // copies still under way land before the shared memory goes (in a run
      // without errors all of them are consumed)
      const long long t0 = clock64();
      while (clock64() - t0 < ptx::kWaitClocks / 100) {
      }
    }
    __syncthreads();
  }
  if (warp == kIssuer) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(bars->tmem, kTmemCols);
  }
  if (S > 1) ptx::cluster_wait();
}

// ---------------------------------------------------------------- bf16 rows as two MXFP8 rows
struct SplitParams {
  const __nv_bfloat16* x;
  long long ldx;
  uint8_t* x8[2];  // [M][K]
  uint8_t* xc[2];  // [M][K / 32]
  long long octets;
  int K;
};

// Four lanes share a group of 32 columns. A value that is not finite makes its
// row NaN (the E4M3 NaN in hi), as it makes the sum not finite; it does not touch the scale.
__global__ void __launch_bounds__(256) split_kernel(const SplitParams p) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const long long o = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (o >= p.octets) return;  // (whole groups: K is a multiple of 32)
  const int row_octets = p.K >> 3;
  const long long m = o / row_octets;
  const int c = static_cast<int>(o - m * row_octets);
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p.x + m * p.ldx) + c);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float v[8], amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(v[j]);
    amax = fmaxf(amax, a <= FLT_MAX ? a : 0.0f);
  }
  const unsigned mask = 0xFu << (threadIdx.x & 28);
  amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 2));
  const int code = mx_code(amax), low = max(code - 4, 0);
  const float mul = mx_mul(code), up = static_cast<float>(1 << (code - low));
  uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float a = fabsf(v[j]) <= FLT_MAX ? v[j] * mul : __uint_as_float(0x7FC00000u);
    const float b = fabsf(v[j + 1]) <= FLT_MAX ? v[j + 1] * mul : __uint_as_float(0x7FC00000u);
    const uint32_t h = e4m3x2(a, b);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h), __NV_E4M3)));
    hi[j >> 2] |= h << (8 * (j & 3));
    lo[j >> 2] |= static_cast<uint32_t>(e4m3x2((a - f.x) * up, (b - f.y) * up)) << (8 * (j & 3));
  }
  reinterpret_cast<uint2*>(p.x8[0])[o] = make_uint2(hi[0], hi[1]);
  reinterpret_cast<uint2*>(p.x8[1])[o] = make_uint2(lo[0], lo[1]);
  if ((o & 3) == 0) {
    p.xc[0][o >> 2] = static_cast<uint8_t>(code);
    p.xc[1][o >> 2] = static_cast<uint8_t>(low);
  }
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

// Two warps may make the weights' scale images in turn, by groups of 4 K blocks,
// where for each block that one of them waits for it has waited for one of the
// same issuer's (an even number of blocks before) less than a round, `slots`
// blocks, ago. Between a warp's groups lie 4 blocks at most: its last group's
// last two are 5 and 6 before, or where that one has a single block (a tile's
// last, 4 i + 1 blocks of K) that is 5 before and the one of the same issuer 10.
int code_warps_of(int slots, int nk) { return slots >= 10 || (slots >= 6 && nk % 4 != 1) ? 2 : 1; }

using Kernel = void (*)(LinearParams);
constexpr Kernel kKernels[] = {linear_kernel<false, 1, 1>, linear_kernel<false, 1, 2>, linear_kernel<false, 2, 1>,
                               linear_kernel<false, 2, 2>, linear_kernel<true, 1, 1>};
constexpr int kRawKernel = 4;

int round_up(int v, int to) { return (v + to - 1) / to * to; }

// How many clusters of each size the device holds at once (looked up once per device).
int max_clusters(int device, int split) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];
  if (device < 0 || device >= kDevices) return 0;
  int n = known[device][split].load(std::memory_order_relaxed);
  if (n > 0) return n;
  for (const Kernel k : kKernels)
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(threads_of(true));
  cfg.dynamicSmemBytes = kSmemMax;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kKernels[kRawKernel], &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[device][split].store(n, std::memory_order_relaxed);
  return n;
}

// How a product is laid out over the GPU, and what that takes.
struct Shape {
  int nt, tiles_m;  // token rows of a tile, and such tiles
  int64_t tasks;
  bool stacked;
  int cols, products, himg;
  int split, clusters;
  bool over;  // the exchange buffer lies over the ring (one tile a cluster)
  uint32_t xchg;
  int accs, issuers, slots;
  bool raw;  // the kernel takes the bf16 rows apart itself
  int64_t ns;  // estimate, without what all shapes have alike
};

// The shape for tiles of up to nt token rows and K shared by `split` CTAs, of
// which the device holds `clusters` clusters; false where it does not work.
bool shape_of(int M, int N, int K, int parts, int nt, int split, int clusters, Shape& s) {
  s.tiles_m = (M + nt - 1) / nt;
  const int per_tile = (M + s.tiles_m - 1) / s.tiles_m;
  // Few rows' hi and lo are columns of one product (one of 32 to 64 columns takes
  // the time of one of 16), more rows' two that share the weights and their scales.
  s.stacked = parts == 2 && per_tile <= 64;
  s.nt = round_up(per_tile, s.stacked ? 8 : 16);
  s.products = s.stacked ? 1 : parts;
  s.cols = s.stacked ? 2 * s.nt : s.nt;
  s.himg = s.cols > 128 ? 2 : 1;
  s.tasks = static_cast<int64_t>((N + kTileN - 1) / kTileN) * s.tiles_m;
  s.split = split;
  s.clusters = clusters;
  if (s.tasks > kMaxTasks || (split > 1 && s.tasks > clusters && s.nt > 64)) return false;
  s.over = split > 1 && s.nt > 64;
  s.xchg = split > 1 ? static_cast<uint32_t>(round_up(s.nt / 4, split)) * 2048u : 0;
  s.accs = s.tasks > clusters ? 2 : 1;
  // Two issuers where their accumulators and a ring of 4 slots (all even, see
  // above) fit: 300 MXFP8 rows of 5120 to 7168 columns, 160 a tile: 16.4 us with
  // two, 20.3 with one; bf16 rows alike, on a ring of 2 slots in place of 3, 33.1 and 28.7.
  const uint32_t room = kSmemMax - 1024 - static_cast<uint32_t>(sizeof(Bars)) - 64 - (s.over ? 0 : s.xchg);
  const uint32_t slot = kABytes + parts * s.nt * 128u + (1 + s.products * s.himg) * kImg;
  for (s.issuers = 2;; s.issuers = 1) {
    const int tmem = static_cast<int>(kTmemCols) - s.accs * s.issuers * s.cols;
    s.slots = std::min({static_cast<int>(room / slot), tmem / (4 + 4 * s.products * s.himg), kMaxSlots});
    if (s.slots >= 4 || s.issuers == 1) break;
  }
  if (s.slots > 3) s.slots &= ~1;
  // The estimate: a K block's time (a line through measured ones of 48 to 384
  // columns; one issuer takes 340 ns and more, with two products 500), what a
  // tile's columns cost at its end, and what it costs to share K: an exchange,
  // behind which a CTA's next tile hides from some 4 us on. (48 rows, 5120
  // columns to 27648, three tiles a pair: 18.3 us, with whole tiles 19.5; to 7168,
  // one tile a pair 9.4, two tiles five CTAs 10.9.)
  int64_t block = 110 + 5 * s.products * s.cols / 4;
  if (s.issuers == 1) block = std::max<int64_t>(block, 180 + 160 * s.products);
  const int steps = (K / 128 + kStep - 1) / kStep;
  const int64_t tiles = (s.tasks + clusters - 1) / clusters, tile = (steps + split - 1) / split * kStep * block + 10 * s.nt;
  // A kernel in front that takes bf16 rows apart costs some 1.5 us; the warps that
  // do it here, 8 rows of a K block a step, are the slower the more rows a CTA
  // goes through. To 5120 columns from 5120 (14 blocks a CTA): 1 row 8.1 us here,
  // 8.8 with a kernel in front, 16 rows (224) 8.7 and 9.4, 24 (336) 10.2 and 9.8,
  // 48 12.9 and 10.9; 16 rows of 2048 to 2048 (64) 4.8 and 6.6, 16 rows of 5120 to
  // 7168 (320) 9.8 and 10.3, 17 rows of 1024 to 60000 (768) 15.5 and 13.2.
  s.raw = s.stacked && tiles * ((steps + split - 1) / split) * kStep * s.nt <= 320;
  s.ns = split == 1 ? tiles * tile : (tiles - 1) * std::max<int64_t>(tile, 4000) + tile + 1500 + 5 * s.nt;
  return true;
}

// The shape of the smallest estimate. (5120 columns to 7168, MXFP8: 400 rows in
// five tiles of 80 rows 20.2 us, in three of 144 as few as can be 32.1; 192 rows
// of 2048 to 2048 in six tiles of 32 7.2, in one with K shared by four CTAs 8.9.)
bool choose_shape(int M, int N, int K, int parts, int device, Shape& best) {
  const int steps = (K / 128 + kStep - 1) / kStep;
  bool any = false;
  for (int nt = kMaxRows, tiles = 0; nt > 0; nt -= 16) {
    if ((M + nt - 1) / nt == tiles) continue;  // (the last one's tiles, as even as they get)
    tiles = (M + nt - 1) / nt;
    for (int split = 1; split <= std::min(kMaxCluster, steps); ++split) {
      Shape s;
      const int clusters = max_clusters(device, split);
      if (clusters == 0 || !shape_of(M, N, K, parts, nt, split, clusters, s)) continue;
      if (!any || s.ns < best.ns) best = s;
      any = true;
    }
  }
  return any;
}

int weight_code_warps(const Shape& s, int K) { return code_warps_of(s.slots, K / 128); }

// Warps that take the blocks' rows' codes (s.raw: pairs of warps, their bf16 rows)
// in turn; of two products, one each. Four where a CTA has whole tiles to stream:
// 129281 columns of 5120, 7 rows 56 us, with two 59.
int row_turns(const Shape& s) {
  return s.slots % 2 ? 1 : (s.slots >= 6 && s.split == 1) || (s.raw && s.slots >= 4) ? 4 : 2;
}

// One part's codes in the workspace.
size_t split_codes(int M, int K) { return (static_cast<size_t>(M) * K / 32 + 15) / 16 * 16; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_linear_x4_workspace_bytes(int M, int K, int x_format) {
  return x_format == MOE_LINEAR_BF16 && M > 0 && K > 0
             ? 2 * (static_cast<size_t>(M) * K + moe::split_codes(M, K))
             : 0;
}

extern "C" int moe_linear_x4_shape(int M, int N, int K, int x_format, moe_linear_shape* shape) {
  using namespace moe;
  if (M < 1 || M > (1 << 20) || N < 1 || N > (1 << 24)) return MOE_ERR_RANGE;
  if (K < 128 || K % 128 || K > (1 << 16)) return MOE_ERR_UNSUPPORTED;
  if (!shape || (x_format != MOE_LINEAR_BF16 && x_format != MOE_LINEAR_MXFP8)) return MOE_ERR_ARG;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  Shape s;
  if (!choose_shape(M, N, K, x_format == MOE_LINEAR_BF16 ? 2 : 1, device, s)) return MOE_ERR_CUDA;
  *shape = {s.nt,       static_cast<int>(s.tasks), s.split, s.clusters, s.products, s.himg, s.stacked, s.raw, s.over,
            s.issuers,  s.slots,                   weight_code_warps(s, K),         s.products > 1 ? 1 : row_turns(s)};
  return MOE_OK;
}

extern "C" int moe_linear_x4(const void* x, int64_t ldx, const uint8_t* x_codes, int M, const uint8_t* w,
                             const uint8_t* w_codes, int N, int K, void* out, int64_t ldo, void* workspace,
                             size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace moe;
  if (M < 0 || M > (1 << 20) || N < 0 || N > (1 << 24)) return MOE_ERR_RANGE;
  if (K < 128 || K % 128 || K > (1 << 16)) return MOE_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MOE_OK;
  if (!x || !w || !w_codes || !out) return MOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w, 32) || !aligned(w_codes, 4) || !aligned(out, 2) || !aligned(x_codes, 4) ||
      !aligned(status, 4) || !aligned(workspace, 16) || ldx % (x_codes ? 16 : 8))
    return MOE_ERR_ALIGN;
  if (ldx < K || ldo < N || out == x) return MOE_ERR_ARG;
  const size_t need = moe_linear_x4_workspace_bytes(M, K, x_codes ? MOE_LINEAR_MXFP8 : MOE_LINEAR_BF16);
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_ARG;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);

  LinearParams p = {};
  p.wc = w_codes;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.status = status;
  p.M = M;
  p.N = N;
  p.K = K;
  p.parts = x_codes ? 1 : 2;
  Shape shape;
  if (!choose_shape(M, N, K, p.parts, device, shape)) return MOE_ERR_CUDA;
  const int products = shape.products, split = shape.split;
  const int clusters = static_cast<int>(std::min<int64_t>(shape.clusters, shape.tasks));
  p.tiles_m = shape.tiles_m;
  p.nt = shape.nt;
  p.tasks = static_cast<int>(shape.tasks);
  p.stacked = shape.stacked;
  p.cols = shape.cols;
  p.issuers = shape.issuers;
  p.accs = shape.accs;
  p.slots = shape.slots;
  p.split = split;
  p.slot_b = p.parts * p.nt * 128u;
  p.slot_img = (1 + products * shape.himg) * kImg;
  p.code_warps = weight_code_warps(shape, K);
  p.turns = row_turns(shape);
  p.off_b = p.slots * kABytes;
  p.off_img = p.off_b + p.slots * p.slot_b;
  // (a ring has 3 slots at least, more than the 100 KB that an exchange buffer over it takes at most)
  p.off_xchg = shape.over ? 0 : p.off_img + p.slots * p.slot_img;
  p.off_bar = p.off_img + p.slots * p.slot_img + (shape.over ? 0 : shape.xchg);

  p.early = !x_codes && !shape.raw;
  const uint8_t* rows = static_cast<const uint8_t*>(x);
  int64_t row_bytes = ldx;
  p.xc[0] = x_codes;
  if (p.early) {
    SplitParams q;
    q.x = static_cast<const __nv_bfloat16*>(x);
    q.ldx = ldx;
    q.K = K;
    q.octets = static_cast<long long>(M) * (K / 8);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    q.x8[0] = ws;
    q.x8[1] = ws + static_cast<size_t>(M) * K;
    q.xc[0] = ws + 2 * static_cast<size_t>(M) * K;
    q.xc[1] = q.xc[0] + split_codes(M, K);
    for (int h = 0; h < 2; ++h) p.xc[h] = q.xc[h];
    rows = ws;
    row_bytes = K;
    const cudaError_t e = launch_pdl(split_kernel, dim3(static_cast<unsigned>((q.octets + 255) / 256)), dim3(256), 0, st, q);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
  }
  if (!encode_blocks(&p.tm_w, w, true, K, N, K / 2, 0, 0, kTileN, 1)) return MOE_ERR_CUDA;
  const bool encoded =
      shape.raw ? encode_blocks(&p.tm_x, x, false, 2 * static_cast<uint64_t>(K), M, 2 * ldx, 0, 0, p.nt, 2)
            : encode_blocks(&p.tm_x, rows, false, K, M, row_bytes, p.parts, static_cast<uint64_t>(M) * K, p.nt, p.parts);
  if (!encoded) return MOE_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * split));
  cfg.blockDim = dim3(32u * (kRowsX + (products > 1 ? products : shape.raw ? 2 * p.turns : p.turns)));
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  cfg.dynamicSmemBytes = p.off_bar + sizeof(Bars) + 1024;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kKernels[shape.raw ? kRawKernel : 2 * (products - 1) + shape.himg - 1], p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
