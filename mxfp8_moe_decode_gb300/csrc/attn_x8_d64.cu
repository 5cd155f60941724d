// The cache attention for heads of 64: up to 16 rows of a sequence and
// key/value head in attn_x8.cuh's kernel, more in attn_wide.cuh's.
#include "attn_wide.cuh"

namespace moe {

cudaError_t launch_attn_x8_d64(const AttnX8Params& p, int rows, int device, int grid, cudaStream_t s) {
  switch (attn_x8_group_rows(64, rows)) {
    case 8: return attn::launch<64, 1, 1>(p, device, grid, s);
    case 16: return attn::launch<64, 2, 1>(p, device, grid, s);
    default: return attn::launch_wide<64>(p, device, grid, s);
  }
}

}  // namespace moe
