// The norms around a block, with its gate and the residual's scale, of any
// number of bf16 token rows:
//   b   = (x * rx) * post_w,  rx = (mean(x^2) + eps)^(-1/2)     (no post_w: b = x)
//   res = bf16(res_scale * residual + block_scale * (gate * b)) (no gate: 1)
//   y   = (res * r) * norm_w, r = (mean(res^2) + eps)^(-1/2)
//   MXFP8 of the fp32 y (E4M3 bytes + one E8M0 code per 32 columns), and
//   optionally bf16(y).
// Everything is fp32 up to the one rounding of res, which the next norm reads:
// it is the row every other reader of the residual stream sees. Both sums of
// squares have the seam's fixed order (seam.cuh), so y and its bytes equal
// moe_attn_seam_x8 of res bit for bit, whatever the number of rows.
//
// Bound by memory: 4 H bytes in (6 H with a gate per row) and 3.03 H (5.03 H
// with normed) out per row. One CTA of 128 threads per row, thread i holding
// the octets i, i + 128, ... of the row as packed bf16 (4 registers an octet)
// from the loads, all issued before the first use, to the stores: a row is read
// once, and the two sums cost two exchanges of four floats.
// 12000 rows of 5120: with a gate per row 91 us (556 MB, 6.1 TB/s, 91 % of a copy's
// rate), without 74, with normed beside the gate 107. Arithmetic is in fp32 pairs, and
// what scales a row is one factor (before: 104 us, bound by instructions). 48 rows 3.0
// to 3.3 us in graph replays: a launch and one row's chain of loads, two exchanges and
// stores; by single calls from Python, which allocate three or four outputs, 14 to 16. Six CTAs an SM
// where a thread has 4 or 5 octets: 93.4 us without (79 registers hold the rows of
// 5120; of wider ones they would not).
#include "f32x2.cuh"
#include "internal.cuh"
#include "ptx.cuh"
#include "seam.cuh"

namespace moe {
namespace {

constexpr int kThreads = kSeamOwners;

struct NormAddNormParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;
  const __nv_bfloat16* gate;    // or null
  const __nv_bfloat16* post_w;  // or null
  const __nv_bfloat16* norm_w;
  __nv_bfloat16* res_out;
  uint8_t* x8;
  uint8_t* x8c;
  __nv_bfloat16* normed;        // or null
  long long ldx, ldr, ldg;      // elements between rows (ldg 0: one gate row for all)
  int H;
  float eps, res_scale, block_scale;
};

// kOct octets a thread (H <= 1024 kOct); kFew: the weights are loaded with the
// rows, before the sums that they wait for otherwise (launch says when)
template <int kOct, bool kFew>
__global__ void __launch_bounds__(kThreads, !kFew && (kOct == 4 || kOct == 5) ? 6 : 1) norm_add_norm_kernel(const NormAddNormParams p) {
  const size_t t = blockIdx.x;
  const int H = p.H;
  const int noct = H >> 3;
  const int tid = threadIdx.x;
  __shared__ float red[2][kThreads / 32];
  ptx::griddep_wait();  // any input may come from the previous kernel on the stream
  ptx::griddep_launch_dependents();
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + t * p.ldx);
  const uint4* rr = reinterpret_cast<const uint4*>(p.residual + t * p.ldr);
  const uint4* gr = reinterpret_cast<const uint4*>(p.gate + t * p.ldg);
  const uint4* pr = reinterpret_cast<const uint4*>(p.post_w);
  const uint4* wr = reinterpret_cast<const uint4*>(p.norm_w);
  const bool gated = p.gate != nullptr, post = p.post_w != nullptr;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 s[kOct], b[kOct], g[kOct];
#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const int o = tid + i * kThreads;
    const bool in = o < noct;
    b[i] = in ? __ldcs(xr + o) : zero;
    s[i] = in ? __ldcs(rr + o) : zero;
    g[i] = in && gated ? (p.ldg ? __ldcs(gr + o) : __ldg(gr + o)) : zero;
  }
  uint4 pw[kFew ? kOct : 1], nw[kFew ? kOct : 1];
  if (kFew) {
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      const int o = tid + i * kThreads;
      pw[i] = o < noct && post ? __ldg(pr + o) : zero;
      nw[i] = o < noct ? __ldg(wr + o) : zero;
    }
  }
  float rx = p.block_scale;
  if (post) {
    Pair q0 = pair(0.0f, 0.0f), q1 = q0;
#pragma unroll
    for (int i = 0; i < kOct; ++i) {  // (octets past the row are zeros)
      const Pair a = pair(b[i].x), c = pair(b[i].y), d = pair(b[i].z), e = pair(b[i].w);
      q0 = fma(d, d, fma(a, a, q0));
      q1 = fma(e, e, fma(c, c, q1));
    }
    const float2 u = floats(q0), v = floats(q1);
    const float ss = seam_warp_sum((u.x + u.y) + (v.x + v.y));
    if ((tid & 31) == 0) red[0][tid >> 5] = ss;
    __syncthreads();
    const float tot = (red[0][0] + red[0][1]) + (red[0][2] + red[0][3]);
    rx *= __frsqrt_rn(tot / static_cast<float>(H) + p.eps);
  }
  // block_scale * rx, one factor
  const Pair f = pair(rx, rx), rs = pair(p.res_scale, p.res_scale);
  float ss = 0.0f;
  uint4* ro = reinterpret_cast<uint4*>(p.res_out + t * H);
#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const int o = tid + i * kThreads;
    if (o < noct) {
      const uint4 m = kFew ? pw[kFew ? i : 0] : post ? __ldg(pr + o) : zero;
      const uint32_t xs[4] = {b[i].x, b[i].y, b[i].z, b[i].w}, ms[4] = {m.x, m.y, m.z, m.w},
                     gs[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
      uint32_t r[4] = {s[i].x, s[i].y, s[i].z, s[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        Pair v = mul(pair(xs[j]), f);
        if (post) v = mul(v, pair(ms[j]));
        if (gated) v = mul(v, pair(gs[j]));
        const float2 n = floats(fma(rs, pair(r[j]), v));
        const __nv_bfloat162 h = __floats2bfloat162_rn(n.x, n.y);
        r[j] = *reinterpret_cast<const uint32_t*>(&h);
        const float2 k = floats(pair(r[j]));  // (the seam's order)
        ss = fmaf(k.x, k.x, ss);
        ss = fmaf(k.y, k.y, ss);
      }
      s[i] = make_uint4(r[0], r[1], r[2], r[3]);
      ro[o] = s[i];
    }
  }
  ss = seam_warp_sum(ss);
  if ((tid & 31) == 0) red[1][tid >> 5] = ss;
  __syncthreads();
  const float r = seam_scale(red[1], H, p.eps);
  const Pair r2 = pair(r, r);

#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const int o = tid + i * kThreads;
    if (i * kThreads >= noct) break;  // uniform across the CTA
    const bool in = o < noct;
    const uint4 w = kFew ? nw[kFew ? i : 0] : in ? __ldg(wr + o) : zero;
    const uint32_t vs[4] = {s[i].x, s[i].y, s[i].z, s[i].w}, ws[4] = {w.x, w.y, w.z, w.w};
    Pair y[4];
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = mul(mul(pair(vs[j]), r2), pair(ws[j]));
      const float2 u = floats(y[j]);
      amax = fmaxf(amax, fmaxf(fabsf(u.x), fabsf(u.y)));
    }
    // the 32-group's amax over its four lanes
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int code = mx_code(amax);
    const float up = mx_mul(code);
    const Pair mm = pair(up, up);
    if (in) {
      // (the conversion saturates; finite values are at most 448 here)
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = floats(mul(y[j], mm));
        q[j] = e4m3x2(u.x, u.y);
      }
      reinterpret_cast<uint2*>(p.x8 + t * H)[o] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      if ((o & 3) == 0) p.x8c[t * (H >> 5) + (o >> 2)] = static_cast<uint8_t>(code);
      if (p.normed) {
        __align__(16) __nv_bfloat162 n[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = floats(y[j]);
          n[j] = __floats2bfloat162_rn(u.x, u.y);
        }
        reinterpret_cast<uint4*>(p.normed + t * H)[o] = *reinterpret_cast<const uint4*>(n);
      }
    }
  }
}

// Rows for which the SMs have room at once: a call lasts one row's chain (5120
// columns: 48 rows 3.3 us in place of 4.7, 600 rows 6.9 in place of 8.6). Of more,
// more CTAs an SM hide it, whose registers hold no weights (600 rows of 8192: 13.9
// us, with the weights first 14.7).
template <int kOct>
cudaError_t launch(const NormAddNormParams& p, int M, cudaStream_t s) {
  return launch_pdl(M <= 152 * (kOct > 5 ? 2 : 4) ? norm_add_norm_kernel<kOct, true> : norm_add_norm_kernel<kOct, false>, dim3(M), dim3(kThreads), 0, s, p);
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

}  // namespace
}  // namespace moe

extern "C" int moe_norm_add_norm_x8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                    const void* gate, int64_t ldg, const void* post_w,
                                    const void* norm_w, int M, int hidden, float res_scale,
                                    float block_scale, float eps, void* res_out, uint8_t* x8,
                                    uint8_t* x8_codes, void* normed, void* stream) {
  using namespace moe;
  if (M < 0) return MOE_ERR_RANGE;
  if (hidden % 32 || hidden < 32 || hidden > 8 * kSeamOwners * kSeamMaxOct)
    return MOE_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f)) return MOE_ERR_ARG;
  // (a difference of itself is 0 for finite numbers only)
  if (res_scale - res_scale != 0.0f || block_scale - block_scale != 0.0f) return MOE_ERR_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !residual || !norm_w || !res_out || !x8 || !x8_codes) return MOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gate, 16) || !aligned(post_w, 16) ||
      !aligned(norm_w, 16) || !aligned(res_out, 16) || !aligned(x8, 16) || !aligned(normed, 16))
    return MOE_ERR_ALIGN;
  if (ldx < hidden || ldr < hidden || (gate && ldg != 0 && ldg < hidden)) return MOE_ERR_ARG;
  if (ldx % 8 || ldr % 8 || (gate && ldg % 8)) return MOE_ERR_ALIGN;
  // in place only where the rows coincide
  if ((res_out == residual && ldr != hidden) || (res_out == x && ldx != hidden)) return MOE_ERR_ARG;
  NormAddNormParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.gate = static_cast<const __nv_bfloat16*>(gate);
  p.post_w = static_cast<const __nv_bfloat16*>(post_w);
  p.norm_w = static_cast<const __nv_bfloat16*>(norm_w);
  p.res_out = static_cast<__nv_bfloat16*>(res_out);
  p.x8 = x8;
  p.x8c = x8_codes;
  p.normed = static_cast<__nv_bfloat16*>(normed);
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldg = gate ? ldg : 0;
  p.H = hidden;
  p.eps = eps;
  p.res_scale = res_scale;
  p.block_scale = block_scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch ((hidden / 8 + kThreads - 1) / kThreads) {
    case 1: e = launch<1>(p, M, st); break;
    case 2: e = launch<2>(p, M, st); break;
    case 3: e = launch<3>(p, M, st); break;
    case 4: e = launch<4>(p, M, st); break;
    case 5: e = launch<5>(p, M, st); break;
    case 6: e = launch<6>(p, M, st); break;
    case 7: e = launch<7>(p, M, st); break;
    default: e = launch<8>(p, M, st); break;
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
