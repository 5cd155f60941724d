// Products with 4-bit weights: out[m, n] = bf16(sum_k x[m, k] w[n, k]) for MXFP4
// rows w (E2M1 with one E8M0 code per 32 columns) and rows x in MXFP8 or bf16.
//
// Both operands go to the block-scaled tensor cores as they are (tcgen05
// kind::mxf8f6f4, E2M1 against E4M3): products and their scales are exact, sums
// fp32. bf16 rows become two MXFP8 rows first: with the group's code c, hi =
// E4M3(x 2^(127 - c)) and lo = E4M3(16 (x 2^(127 - c) - hi)) under the code c - 4.
// bf16 has 8 significant bits, hi takes 4 and the rest, at most half a step of
// hi, fits lo's 4: exact down to 2^-14 of the group's largest value, and off by
// at most 2^-21 of that below (E4M3's subnormals).
//
// Swap-AB: 128 weight rows are the MMA's M and up to 192 token rows its N, so
// few tokens still fill the tensor cores' lanes, and the weights stream once
// for up to 192 rows.
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
constexpr int kMaxStages = 16;
constexpr int kMaxCluster = 8;
constexpr int kAProducers = 4;   // warps that issue the weights' copies
constexpr int kBProducers = 3;   // warps that issue the rows' copies
// warps: 0-3 epilogue, 4 MMA issuer, 5-7 scale images (weights, rows, rows' second part), 8.. producers
constexpr int kWarps = 8 + kAProducers + kBProducers;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kABytes = kTileN * 128;
constexpr uint32_t kImg = 512;   // scale image of 128 rows and one K block of 128
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSmemMax = 227 * 1024;

struct LinearParams {
  CUtensorMap tm_w, tm_x[2];
  const uint8_t* wc;     // [N][K / 32]
  const uint8_t* xc[2];  // [M][K / 32]
  __nv_bfloat16* out;
  long long ldo;
  int* status;
  int M, N, K;
  int nt;                // token rows of a tile (a multiple of 16)
  int tiles_m, tasks;
  int parts;             // 1 (MXFP8 rows) or 2 (bf16 rows as hi and lo)
  int blocks;            // K blocks of a stage (1 or 2)
  int stages;            // ring slots
  int split;             // CTAs (a cluster) that share a tile's K
  uint32_t slot_bytes, off_img, slot_img, off_xchg, off_bar;
};

struct Bars {
  uint64_t full[kMaxStages];   // weights, rows and scale images are there
  uint64_t empty[kMaxStages];  // the stage's MMAs have read them
  uint64_t tfull[2], tempty[2];
  uint64_t xfree;              // every CTA of the cluster has its exchange buffer free
  uint64_t xfull;              // this CTA's exchange buffer is full
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

using ptx::elect_one;
using ptx::mbar_wait_clocks;

// 4 K blocks' codes of one row (word j: the block 4 g + j), as 16 bytes where a
// row's codes are 16-byte aligned.
__device__ __forceinline__ uint4 load_codes(const uint8_t* row, int g, int nk, bool wide) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (wide) {
    v = __ldg(reinterpret_cast<const uint4*>(row) + g);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + 4 * g;
    const int n = nk - 4 * g;
    v.x = __ldg(w);
    if (n > 1) v.y = __ldg(w + 1);
    if (n > 2) v.z = __ldg(w + 2);
    if (n > 3) v.w = __ldg(w + 3);
  }
  return v;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - (ptx::smem_u32(smem_raw) & 1023)) % 1024;
  Bars* bars = reinterpret_cast<Bars*>(smem + p.off_bar);
  volatile int* abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const auto bar = [](uint64_t& b) { return ptx::smem_u32(&b); };
  const int S = p.split, R = p.stages;
  const int rank = S > 1 ? static_cast<int>(blockIdx.x) % S : 0;
  const int cluster = static_cast<int>(blockIdx.x) / S, clusters = static_cast<int>(gridDim.x) / S;
  const int nk = p.K / 128, steps = (nk + p.blocks - 1) / p.blocks;
  const int s0 = steps * rank / S, s1 = steps * (rank + 1) / S;  // this CTA's stages of a tile
  const int himg = p.nt > 128 ? 2 : 1;                           // scale images of a rows' part

  if (tid == 0) {
    for (int i = 0; i < R; ++i) {
      ptx::mbar_init(bar(bars->full[i]), 2 + 2 * p.parts);  // copies and images of the weights and each part
      ptx::mbar_init(bar(bars->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(bars->tfull[i]), 1);
      ptx::mbar_init(bar(bars->tempty[i]), 4);
    }
    ptx::mbar_init(bar(bars->xfree), S);
    ptx::mbar_init(bar(bars->xfull), 4 * S);
    ptx::mbar_init(bar(bars->drain), 1);
    bars->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tm_w);
    ptx::prefetch_tmap(&p.tm_x[0]);
    if (p.parts > 1) ptx::prefetch_tmap(&p.tm_x[1]);
  }
  if (warp == 4) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem), kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (S > 1) ptx::cluster_sync();  // the others' barriers are initialised
  const uint32_t tmem = bars->tmem;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  if (warp >= 8) {
    // ------------------------------------------------------------ producers
    // The stages go to the warps of a kind in turn, to no more warps than the
    // ring has slots: the slots are freed in order, and a warp has seen that of
    // its last stage, at most R stages ago, free, so none comes two phases late
    // to a slot (and takes its parity for the one it wants).
    const bool is_a = warp < 8 + kAProducers;
    const int who = is_a ? warp - 8 : warp - 8 - kAProducers, of = min(is_a ? kAProducers : kBProducers, R);
    if (who < of && elect_one()) {
      const uint64_t policy = is_a ? ptx::policy_evict_first() : ptx::policy_evict_last();
      const uint32_t part_bytes = static_cast<uint32_t>(p.nt) * 128u * p.blocks;
      // (a 4-bit box counts its global bytes, half of what it fills)
      const uint32_t bytes = is_a ? kABytes / 2 * p.blocks : part_bytes;
      int it = 0;
      bool ok = true;
      for (int t = cluster; ok && t < p.tasks; t += clusters) {
        const int n0 = t / p.tiles_m * kTileN, m0 = t % p.tiles_m * p.nt;
        for (int s = s0; s < s1; ++s, ++it) {
          if (it % of != who) continue;
          const int slot = it % R;
          if (!mbar_wait_clocks(bar(bars->empty[slot]), ((it / R) & 1) ^ 1, abort)) {
            ok = false;
            break;
          }
          const uint32_t full = bar(bars->full[slot]);
          const uint32_t dst = ptx::smem_u32(smem) + slot * p.slot_bytes;
          if (is_a) {
            ptx::mbar_arrive_expect_tx(full, bytes);
            ptx::tma_load_3d(dst, &p.tm_w, 0, n0, s * p.blocks, full, policy);
          } else {
            for (int h = 0; h < p.parts; ++h) {
              ptx::mbar_arrive_expect_tx(full, bytes);
              ptx::tma_load_3d(dst + p.blocks * kABytes + h * part_bytes, &p.tm_x[h], 0, m0, s * p.blocks, full,
                               policy);
            }
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      const uint32_t sf0 = tmem + 2 * p.nt, sf_slot = p.blocks * (4 + 4 * p.parts * himg);
      const uint32_t part_bytes = static_cast<uint32_t>(p.nt) * 128u * p.blocks;
      uint32_t idesc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) idesc[k] = ptx::idesc_mxf8(p.nt, k, ptx::kFmtE2M1);
      int slot = 0, round = 0, lt = 0;
      bool ok = true;
      for (int t = cluster; ok && t < p.tasks; t += clusters, ++lt) {
        const int acc = lt & 1;
        if (!mbar_wait_clocks(bar(bars->tempty[acc]), ((lt >> 1) & 1) ^ 1, abort)) break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + acc * p.nt;
        uint32_t some = 0;
        for (int s = s0; s < s1; ++s) {
          if (!mbar_wait_clocks(bar(bars->full[slot]), round & 1, abort)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a = ptx::smem_u32(smem) + slot * p.slot_bytes;
          const uint32_t b = a + p.blocks * kABytes;
          uint32_t img = ptx::smem_u32(smem) + p.off_img + slot * p.slot_img;
          uint32_t sf = sf0 + slot * sf_slot;
          for (int k = 0; k < p.blocks; ++k) {
            ptx::tc_cp_32x128b_x4(sf, ptx::sdesc_rows16(img));
            for (int h = 0; h < p.parts * himg; ++h)
              ptx::tc_cp_32x128b_x4(sf + 4 + 4 * h, ptx::sdesc_rows16(img + (1 + h) * kImg));
            for (int h = 0; h < p.parts; ++h) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                ptx::tc_mma_mxf8(d, ptx::sdesc_k128_sw128(a + k * kABytes + 32 * kk),
                                 ptx::sdesc_k128_sw128(b + h * part_bytes + k * p.nt * 128 + 32 * kk), idesc[kk], sf,
                                 sf + 4 + 4 * h * himg, some);
                some = 1;
              }
            }
            sf += 4 + 4 * p.parts * himg;
            img += (1 + p.parts * himg) * kImg;
          }
          ptx::tc_commit(bar(bars->empty[slot]));
          if (++slot == R) {
            slot = 0;
            ++round;
          }
        }
        if (ok) ptx::tc_commit(bar(bars->tfull[acc]));
      }
      // everything this thread issued has completed once drain fires
      ptx::tc_commit(bar(bars->drain));
      int never = 0;
      mbar_wait_clocks(bar(bars->drain), 0, &never);
    }
    __syncwarp();
  } else if (warp >= 5) {
    // ------------------------------------------------------------ scale images
    // Image of a K block: lane i's 16 bytes hold the 4 codes of the rows i, 32 +
    // i, 64 + i, 96 + i. Codes are loaded 4 K blocks at a time, one such group
    // ahead.
    const int part = warp - 6;  // -1: the weights
    if (part < p.parts) {
      const uint8_t* codes = part < 0 ? p.wc : p.xc[part];
      const int count = part < 0 ? p.N : p.M, images = part < 0 ? 1 : himg, pitch = p.K / 32;
      const int tile = part < 0 ? kTileN : p.nt;
      const bool wide = pitch % 16 == 0 && (reinterpret_cast<uintptr_t>(codes) & 15) == 0;
      const uint32_t off = part < 0 ? 0 : (1 + part * himg) * kImg;
      int slot = 0, round = 0;
      bool ok = true;
      for (int t = cluster; ok && t < p.tasks; t += clusters) {
        const int r0 = part < 0 ? t / p.tiles_m * kTileN : t % p.tiles_m * p.nt;
        const auto fetch = [&](uint4 (&v)[2][4], int g) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int r = 128 * i + 32 * c + lane;
              v[i][c] = make_uint4(0, 0, 0, 0);
              if (i < images && r < tile && r0 + r < count && 4 * g < nk)
                v[i][c] = load_codes(codes + static_cast<long long>(r0 + r) * pitch, g, nk, wide);
            }
        };
        uint4 cur[2][4], nxt[2][4];
        fetch(nxt, s0 * p.blocks / 4);
        for (int s = s0; s < s1; ++s) {
          const int k0 = s * p.blocks;
          if (s == s0 || k0 % 4 == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int c = 0; c < 4; ++c) cur[i][c] = nxt[i][c];
            fetch(nxt, k0 / 4 + 1);
          }
          if (!__all_sync(0xffffffffu, mbar_wait_clocks(bar(bars->empty[slot]), (round & 1) ^ 1, abort))) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + p.off_img + slot * p.slot_img + off + lane * 16;
          for (int k = 0; k < p.blocks; ++k) {
            const int j = (k0 + k) & 3;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (i < images)
                *reinterpret_cast<uint4*>(dst + i * kImg) =
                    make_uint4(word(cur[i][0], j), word(cur[i][1], j), word(cur[i][2], j), word(cur[i][3], j));
            dst += (1 + p.parts * himg) * kImg;
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (elect_one()) ptx::mbar_arrive(bar(bars->full[slot]));
          if (++slot == R) {
            slot = 0;
            ++round;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Warp q holds the tile's weight rows 32 q .. 32 q + 31, one a lane.
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
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
    int lt = 0;
    bool ok = true;
    for (int t = cluster; t < p.tasks; t += clusters, ++lt) {
      const int n = t / p.tiles_m * kTileN + tid, m0 = t % p.tiles_m * p.nt;
      const int cols = min(p.nt, p.M - m0);
      const int acc = lt & 1;
      ok = ok && __all_sync(0xffffffffu, mbar_wait_clocks(bar(bars->tfull[acc]), (lt >> 1) & 1, abort));
      if (S > 1 ? !all_ok(ok) : !ok) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem + lanes + acc * p.nt;
      __nv_bfloat16* out = p.out + static_cast<long long>(m0) * p.ldo + n;
      if (S == 1) {
        for (int c0 = 0; c0 < cols; c0 += 16) {
          float v[16];
          ptx::tmem_ld_32x32b_x16(d + c0, v);
          ptx::tmem_wait_ld();
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
      // The tile's column j is summed by the CTA j % S. Every CTA says that its
      // buffer is free (its last tile's sums are read; where the buffer lies
      // over the ring, all MMAs are done too), sends its parts of the columns to
      // their CTAs, and adds up those it gets in the order of the ranks.
      if (tid < S) ptx::mbar_arrive_cluster(ptx::cluster_addr(bar(bars->xfree), tid));
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar(bars->xfree), lt & 1, abort));
      if (!ok) continue;
      const int per = (p.nt + S - 1) / S;
      const uint32_t xchg = ptx::smem_u32(smem) + p.off_xchg;
      for (int c0 = 0; c0 < cols; c0 += 16) {
        float v[16];
        ptx::tmem_ld_32x32b_x16(d + c0, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int c = c0 + j;
          if (c < cols)
            ptx::st_cluster_f32(ptx::cluster_addr(xchg + ((rank * per + c / S) * 128 + tid) * 4, c % S), v[j]);
        }
      }
      ptx::tc_fence_before();
      ptx::fence_cluster();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(bars->tempty[acc]));
      if (lane < S) ptx::mbar_arrive_cluster(ptx::cluster_addr(bar(bars->xfull), lane));
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_cluster(bar(bars->xfull), lt & 1, abort));
      if (!ok) continue;
      const float* part = reinterpret_cast<const float*>(smem + p.off_xchg) + tid;
      if (n < p.N) {
        for (int i = 0; i * S + rank < cols; ++i) {
          float sum = part[i * 128];
          for (int r = 1; r < S; ++r) sum += part[(r * per + i) * 128];
          out[(i * S + rank) * p.ldo] = __float2bfloat16_rn(sum);
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  ptx::tc_fence_before();
  __syncthreads();
  if (*abort && tid == 0) {
    if (p.status) atomicOr(p.status, MOE_LINEAR_STATUS_TIMEOUT);
    // copies still under way land before the shared memory goes (in a run
    // without errors all of them are consumed)
    const long long t0 = clock64();
    while (clock64() - t0 < ptx::kWaitClocks / 100) {
    }
  }
  __syncthreads();
  if (warp == 4) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (S > 1) ptx::cluster_sync();  // nobody writes here any more
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

int round16(int v) { return (v + 15) / 16 * 16; }

// How many clusters of each size the device holds at once (looked up once per device).
int max_clusters(int device, int split) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];
  if (device < 0 || device >= kDevices) return 0;
  int n = known[device][split].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaFuncSetAttribute(linear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemMax;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, linear_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[device][split].store(n, std::memory_order_relaxed);
  return n;
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
  if (ldx < K || ldo < N) return MOE_ERR_ARG;
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
  p.tiles_m = (M + kMaxRows - 1) / kMaxRows;
  p.nt = round16((M + p.tiles_m - 1) / p.tiles_m);
  const int64_t tasks = static_cast<int64_t>((N + kTileN - 1) / kTileN) * p.tiles_m;
  if (tasks > 0x3FFFFFFF) return MOE_ERR_UNSUPPORTED;
  p.tasks = static_cast<int>(tasks);
  p.blocks = p.nt * p.parts <= 32 ? 2 : 1;
  const int steps = (K / 128 + p.blocks - 1) / p.blocks;

  // CTAs that share a tile's K: as many as the device holds at once over all
  // tiles, while each has some stages to itself; shares of one task a cluster
  // only, or with an exchange buffer beside the ring.
  int split = 1, clusters = max_clusters(device, 1);
  if (clusters == 0) return MOE_ERR_CUDA;
  const auto cost = [&](int s, int c) { return (tasks + c - 1) / c * ((steps + s - 1) / s + (s > 1 ? 4 : 2)); };
  int64_t best = cost(1, clusters);
  for (int s = 2; s <= kMaxCluster && s <= steps; ++s) {
    const int c = max_clusters(device, s);
    if (c == 0 || (tasks > c && p.nt > 64)) continue;
    if (cost(s, c) < best) {
      best = cost(s, c);
      split = s;
      clusters = c;
    }
  }
  p.split = split;
  clusters = static_cast<int>(std::min<int64_t>(clusters, tasks));
  const int himg = p.nt > 128 ? 2 : 1;
  p.slot_bytes = p.blocks * (kABytes + p.parts * p.nt * 128u);
  p.slot_img = p.blocks * (1 + p.parts * himg) * kImg;
  const uint32_t xchg = split > 1 ? static_cast<uint32_t>((p.nt + split - 1) / split * split) * 512u : 0;
  const bool over = tasks <= clusters;  // the exchange buffer lies over the ring
  const uint32_t room = kSmemMax - 1024 - static_cast<uint32_t>(sizeof(Bars)) - 64 - (over ? 0 : xchg);
  const uint32_t by_smem = room / (p.slot_bytes + p.slot_img);
  const uint32_t by_tmem = (kTmemCols - 2 * p.nt) / (p.blocks * (4 + 4 * p.parts * himg));
  p.stages = static_cast<int>(std::min<uint32_t>({by_smem, by_tmem, kMaxStages}));
  p.off_img = p.stages * p.slot_bytes;
  p.off_xchg = over ? 0 : p.off_img + p.stages * p.slot_img;
  p.off_bar = p.off_img + p.stages * p.slot_img + (over ? 0 : xchg);
  if (over && xchg > p.off_bar) return MOE_ERR_UNSUPPORTED;

  const uint8_t* xs[2] = {static_cast<const uint8_t*>(x), nullptr};
  int64_t row_bytes = ldx;
  p.xc[0] = x_codes;
  if (!x_codes) {
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
    for (int h = 0; h < 2; ++h) {
      xs[h] = q.x8[h];
      p.xc[h] = q.xc[h];
    }
    row_bytes = K;
    const cudaError_t e = launch_pdl(split_kernel, dim3(static_cast<unsigned>((q.octets + 255) / 256)), dim3(256), 0, st, q);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
  }
  if (!encode_blocks(&p.tm_w, w, true, K, N, K / 2, kTileN, p.blocks)) return MOE_ERR_CUDA;
  for (int h = 0; h < p.parts; ++h)
    if (!encode_blocks(&p.tm_x[h], xs[h], false, K, M, row_bytes, p.nt, p.blocks)) return MOE_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemMax;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_kernel, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
