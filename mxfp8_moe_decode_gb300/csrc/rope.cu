// Rotary positions of any number of bf16 token rows (rope.cuh has the
// mathematics): rows of `heads` heads of `dim` values, turned in place or into
// rows of their own.
//
// Bound by memory, 2 bytes in and 2 out per value. A thread has one item of a
// head (two 16-byte chunks that hold 8 pairs) and takes the same item of
// several heads, so its 8 sines and cosines serve all of them (rope::head_groups).
// 8000 tokens of 40 heads of 128, 64 dims of them in neighbours: 26.2 to 27 us (164 MB,
// 6.1 to 6.3 TB/s, 91 to 94 % of a copy's rate); one token 1.5 us in graph replays, a
// launch (by single calls from Python 4 to 4.6).
#include "internal.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

struct RopeParams {
  rope::Spec spec;
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  const int* positions;
  long long ldx, ldo;
  long long tokens;
  int heads, dim, groups;
};

__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  const int items = p.dim >> 4;
  const long long u = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const unsigned per = static_cast<unsigned>(items * p.groups);
  const long long token = u / per;
  if (token >= p.tokens) return;
  const unsigned rest = static_cast<unsigned>(u - token * per);
  rope::Heads h;
  h.x = reinterpret_cast<const uint4*>(p.x + token * p.ldx);
  h.out = reinterpret_cast<uint4*>(p.out + token * p.ldo);
  h.heads = p.heads;
  h.chunks = p.dim >> 3;
  rope::turn_heads(p.spec, h, __ldg(p.positions + token), rest % items, rest / items, p.groups);
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

}  // namespace
}  // namespace moe

extern "C" int moe_rope(const moe_rope_spec* spec, const void* x, int64_t ldx, int tokens, int heads,
                        int head_dim, const int32_t* positions, void* out, int64_t ldo, void* stream) {
  using namespace moe;
  if (!spec) return MOE_ERR_ARG;
  if (tokens < 0 || tokens > (1 << 24)) return MOE_ERR_RANGE;
  if (head_dim < 16 || head_dim > 1024 || head_dim % 16 || heads < 1 || heads > 4096)
    return MOE_ERR_UNSUPPORTED;
  const int rc = rope::check(spec->freqs, spec->first, spec->rot, head_dim, spec->scale);
  if (rc != MOE_OK) return rc;
  if (tokens == 0) return MOE_OK;
  if (!x || !out || !positions) return MOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(positions, 4) || ldx % 8 || ldo % 8)
    return MOE_ERR_ALIGN;
  const int64_t width = static_cast<int64_t>(heads) * head_dim;
  if (ldx < width || ldo < width || (x == out && ldx != ldo)) return MOE_ERR_ARG;
  RopeParams p;
  p.spec = {spec->freqs, spec->first, spec->rot, spec->interleaved != 0, spec->scale};
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.positions = positions;
  p.ldx = ldx;
  p.ldo = ldo;
  p.tokens = tokens;
  p.heads = heads;
  p.dim = head_dim;
  p.groups = rope::head_groups(tokens, heads, head_dim, false);
  // (at most 2^24 tokens * 4096 heads * 64 items / 128 threads: below 2^35; what does not fit a grid is refused)
  const int64_t ctas = (static_cast<int64_t>(tokens) * p.groups * (head_dim / 16) + kThreads - 1) / kThreads;
  if (ctas > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  const cudaError_t e = launch_pdl(rope_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0,
                                   static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
