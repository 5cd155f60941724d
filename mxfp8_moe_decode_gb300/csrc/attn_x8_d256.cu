// The cache attention (attn_x8.cuh) for heads of 256: one tile of 8 rows per
// warp (its running sum alone takes 64 registers a thread), four warps.
#include "attn_x8.cuh"

namespace moe {

cudaError_t launch_attn_x8_d256(const AttnX8Params& p, int rows, int grid, cudaStream_t s) {
  if (attn_x8_group_rows(256, rows) == 8) return attn::launch<256, 1, 1>(p, grid, s);
  return attn::launch<256, 1, 4>(p, grid, s);
}

}  // namespace moe
