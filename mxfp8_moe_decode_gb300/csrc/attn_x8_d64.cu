// The cache attention (attn_x8.cuh) for heads of 64.
#include "attn_x8.cuh"

namespace moe {

cudaError_t launch_attn_x8_d64(const AttnX8Params& p, int rows, int grid, cudaStream_t s) {
  switch (attn_x8_group_rows(64, rows)) {
    case 8: return attn::launch<64, 1, 1>(p, grid, s);
    case 16: return attn::launch<64, 2, 1>(p, grid, s);
    case 64: return attn::launch<64, 2, 4>(p, grid, s);
    default: return attn::launch<64, 2, 8>(p, grid, s);
  }
}

}  // namespace moe
