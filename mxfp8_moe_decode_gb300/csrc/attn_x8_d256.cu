// The cache attention (attn_x8.cuh) for heads of 256: one tile of 8 rows per
// warp (its running sum alone takes 64 registers a thread).
#include "attn_x8.cuh"

namespace moe {

cudaError_t launch_attn_x8_d256(const AttnX8Params& p, int rows, int device, int grid, cudaStream_t s) {
  switch (attn_x8_group_rows(256, rows)) {
    case 8: return attn::launch<256, 1, 1>(p, device, grid, s);
    case 16: return attn::launch<256, 1, 2>(p, device, grid, s);
    default: return attn::launch<256, 1, 3>(p, device, grid, s);
  }
}

}  // namespace moe
