// Products with 4-bit weights: out[m, n] = sum_k x[m, k] w[n, k] for MXFP4 rows
// w (E2M1 with one E8M0 code per 32 columns) and rows x in MXFP8 or bf16.
//
// One warp per output column and 8 rows: a lane takes every 32nd group of 32
// columns, products and sums in fp32.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "internal.cuh"
#include "kv_x8.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 8;

struct LinearParams {
  const uint8_t* x;   // bf16 or E4M3 rows
  const uint8_t* xc;  // [M][K / 32], or null: bf16
  const uint8_t* w;
  const uint8_t* wc;
  __nv_bfloat16* out;
  long long ldx, ldo;  // bytes between rows of x, elements between rows of out
  int M, N, K;
};

__global__ void __launch_bounds__(kThreads) linear_kernel(const LinearParams p) {
  const int lane = threadIdx.x & 31;
  const long long n = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (n >= p.N) return;
  const long long m0 = static_cast<long long>(blockIdx.y) * kRows;
  const int rows = min(kRows, static_cast<int>(p.M - m0));
  const int groups = p.K / 32;
  float acc[kRows] = {};
  for (int g = lane; g < groups; g += 32) {
    const uint4 q = *reinterpret_cast<const uint4*>(p.w + n * (p.K / 2) + g * 16);
    const uint32_t words[4] = {q.x, q.y, q.z, q.w};
    float w[32];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(words[j / 4] >> (8 * (j % 4))), __NV_E2M1);
      const float2 f = __half22float2(__half2(h));
      w[2 * j] = f.x;
      w[2 * j + 1] = f.y;
    }
    const float ws = e8m0_value(p.wc[n * groups + g]);
    for (int r = 0; r < kRows; ++r) {
      if (r >= rows) break;
      const uint8_t* row = p.x + (m0 + r) * p.ldx;
      float s = 0.0f;
      if (p.xc) {
        for (int j = 0; j < 32; j += 2) {
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(*reinterpret_cast<const uint16_t*>(row + g * 32 + j), __NV_E4M3);
          const float2 f = __half22float2(__half2(h));
          s = fmaf(f.x, w[j], s);
          s = fmaf(f.y, w[j + 1], s);
        }
        s *= e8m0_value(p.xc[(m0 + r) * groups + g]);
      } else {
        const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(row) + g * 32;
        for (int j = 0; j < 32; ++j) s = fmaf(__bfloat162float(b[j]), w[j], s);
      }
      acc[r] = fmaf(s, ws, acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float a = acc[r];
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0 && r < rows) p.out[(m0 + r) * p.ldo + n] = __float2bfloat16_rn(a);
  }
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_linear_x4_workspace_bytes(int M, int K, int x_format) { return 0; }

extern "C" int moe_linear_x4(const void* x, int64_t ldx, const uint8_t* x_codes, int M, const uint8_t* w,
                             const uint8_t* w_codes, int N, int K, void* out, int64_t ldo, void* workspace,
                             size_t workspace_bytes, int32_t* status, void* stream) {
  using namespace moe;
  if (M < 0 || M > (1 << 20) || N < 0 || N > (1 << 24)) return MOE_ERR_RANGE;
  if (K < 128 || K % 128 || K > (1 << 16)) return MOE_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MOE_OK;
  if (!x || !w || !w_codes || !out) return MOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w, 32) || !aligned(w_codes, 4) || !aligned(out, 2) || !aligned(x_codes, 4) ||
      !aligned(status, 4) || ldx % (x_codes ? 16 : 8))
    return MOE_ERR_ALIGN;
  if (ldx < K || ldo < N) return MOE_ERR_ARG;
  LinearParams p;
  p.x = static_cast<const uint8_t*>(x);
  p.xc = x_codes;
  p.w = w;
  p.wc = w_codes;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldx = ldx * (x_codes ? 1 : 2);
  p.ldo = ldo;
  p.M = M;
  p.N = N;
  p.K = K;
  const dim3 grid((N + 3) / 4, (M + kRows - 1) / kRows);
  const cudaError_t e = launch_pdl(linear_kernel, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
