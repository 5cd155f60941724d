// Residual addition + RMSNorm + MXFP8 of any number of bf16 token rows:
//   res = bf16(x + residual),  y = (res * r) * w with r = (mean(res^2) + eps)^(-1/2),
//   MXFP8 of the fp32 y (E4M3 bytes + one E8M0 code per 32 columns), and
//   optionally bf16(y).
// The norm reads the rounded sum, the row the next layer and every other
// reader of the residual stream sees; the sum itself is exact to that one
// rounding (fp32 holds the sum of two bf16 values wherever it can reach a
// bf16 rounding border). Norm and quantisation are the attention seam's
// ("vllm.models.deepseek_v41.amd.mono.layer", store_x8), in its fixed order
// of the sum of squares (see seam.cuh), so the bytes equal moe_attn_seam_x8 of
// res bit for bit, whatever the number of rows.
//
// Bound by memory: 4 H bytes in and 3.03 H (5.03 H with normed) out per row.
// One CTA of 128 threads per row, thread i holding the octets i, i + 128, ...
// of the row in registers between the two passes (as the packed bf16 sum: 4
// registers an octet), so a row is read once; all its loads are issued before
// the first use, and up to 16 rows are in flight on an SM.
// 16384 rows of 5120: 90 us, 6.5 TB/s, 96 % of the rate of a plain copy on the
// same GPU; 1 to 48 rows: 3.1 us, the length of one row's chain (load, sum of
// squares, maxima, store) and the launch.
#include "internal.cuh"
#include "ptx.cuh"
#include "seam.cuh"

namespace moe {
namespace {

constexpr int kThreads = kSeamOwners;

struct AddNormParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;
  const __nv_bfloat16* norm_w;
  __nv_bfloat16* res_out;
  uint8_t* x8;
  uint8_t* x8c;
  __nv_bfloat16* normed;  // or null
  long long ldx, ldr;     // elements between rows
  int H;
  float eps;
};

__device__ __forceinline__ uint4 add_octet(const uint4& a, const uint4& b) {
  float x[8], y[8];
  unpack_bf16x8(a, x);
  unpack_bf16x8(b, y);
  __align__(16) __nv_bfloat162 s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    s[j] = __floats2bfloat162_rn(x[2 * j] + y[2 * j], x[2 * j + 1] + y[2 * j + 1]);
  return *reinterpret_cast<const uint4*>(s);
}

// kOct octets a thread (H <= 1024 kOct)
template <int kOct>
__global__ void __launch_bounds__(kThreads) add_norm_kernel(const AddNormParams p) {
  const size_t t = blockIdx.x;
  const int H = p.H;
  const int noct = H >> 3;
  const int tid = threadIdx.x;
  const uint4* wr = reinterpret_cast<const uint4*>(p.norm_w);
  ptx::griddep_wait();  // any input may come from the previous kernel on the stream
  ptx::griddep_launch_dependents();
  const uint4* xr = reinterpret_cast<const uint4*>(p.x + t * p.ldx);
  const uint4* rr = reinterpret_cast<const uint4*>(p.residual + t * p.ldr);
  uint4 s[kOct], b[kOct];
#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const int o = tid + i * kThreads;
    const bool in = o < noct;
    s[i] = in ? __ldcs(xr + o) : make_uint4(0, 0, 0, 0);
    b[i] = in ? __ldcs(rr + o) : make_uint4(0, 0, 0, 0);
  }
  float ss = 0.0f;
  uint4* ro = reinterpret_cast<uint4*>(p.res_out + t * H);
#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const int o = tid + i * kThreads;
    if (o < noct) {
      s[i] = add_octet(s[i], b[i]);
      ro[o] = s[i];
      float v[8];
      unpack_bf16x8(s[i], v);
      ss = seam_sumsq_octet(v, ss);
    }
  }
  ss = seam_warp_sum(ss);
  __shared__ float red[kThreads / 32];
  if ((tid & 31) == 0) red[tid >> 5] = ss;
  __syncthreads();
  const float r = seam_scale(red, H, p.eps);

#pragma unroll
  for (int i = 0; i < kOct; ++i) {
    const int o = tid + i * kThreads;
    if (i * kThreads >= noct) break;  // uniform across the CTA
    const bool in = o < noct;
    float v[8], w[8], y[8];
    unpack_bf16x8(s[i], v);
    unpack_bf16x8(in ? __ldg(wr + o) : make_uint4(0, 0, 0, 0), w);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      y[j] = (v[j] * r) * w[j];
      amax = fmaxf(amax, fabsf(y[j]));
    }
    // the 32-group's amax over its four lanes
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int code = mx_code(amax);
    const float mul = mx_mul(code);
    if (in) {
      uint2 q;
      q.x = static_cast<uint32_t>(e4m3x2(clamp_e4m3(y[0] * mul), clamp_e4m3(y[1] * mul))) |
            (static_cast<uint32_t>(e4m3x2(clamp_e4m3(y[2] * mul), clamp_e4m3(y[3] * mul))) << 16);
      q.y = static_cast<uint32_t>(e4m3x2(clamp_e4m3(y[4] * mul), clamp_e4m3(y[5] * mul))) |
            (static_cast<uint32_t>(e4m3x2(clamp_e4m3(y[6] * mul), clamp_e4m3(y[7] * mul))) << 16);
      reinterpret_cast<uint2*>(p.x8 + t * H)[o] = q;
      if ((o & 3) == 0) p.x8c[t * (H >> 5) + (o >> 2)] = static_cast<uint8_t>(code);
      if (p.normed) {
        __align__(16) __nv_bfloat162 n[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) n[j] = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
        reinterpret_cast<uint4*>(p.normed + t * H)[o] = *reinterpret_cast<const uint4*>(n);
      }
    }
  }
}

template <int kOct>
cudaError_t launch(const AddNormParams& p, int M, cudaStream_t s) {
  return launch_pdl(add_norm_kernel<kOct>, dim3(M), dim3(kThreads), 0, s, p);
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

}  // namespace
}  // namespace moe

extern "C" int moe_add_norm_x8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                               const void* norm_w, int M, int hidden, float eps, void* res_out,
                               uint8_t* x8, uint8_t* x8_codes, void* normed, void* stream) {
  using namespace moe;
  if (M < 0) return MOE_ERR_RANGE;
  if (hidden % 32 || hidden < 32 || hidden > 8 * kSeamOwners * kSeamMaxOct)
    return MOE_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f)) return MOE_ERR_ARG;
  if (M == 0) return MOE_OK;
  if (!x || !residual || !norm_w || !res_out || !x8 || !x8_codes) return MOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(norm_w, 16) || !aligned(res_out, 16) ||
      !aligned(x8, 16) || (normed && !aligned(normed, 16)))
    return MOE_ERR_ALIGN;
  if (ldx < hidden || ldr < hidden) return MOE_ERR_ARG;
  if (ldx % 8 || ldr % 8) return MOE_ERR_ALIGN;
  // in place only where the rows coincide
  if ((res_out == residual && ldr != hidden) || (res_out == x && ldx != hidden)) return MOE_ERR_ARG;
  AddNormParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.norm_w = static_cast<const __nv_bfloat16*>(norm_w);
  p.res_out = static_cast<__nv_bfloat16*>(res_out);
  p.x8 = x8;
  p.x8c = x8_codes;
  p.normed = static_cast<__nv_bfloat16*>(normed);
  p.ldx = ldx;
  p.ldr = ldr;
  p.H = hidden;
  p.eps = eps;
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
