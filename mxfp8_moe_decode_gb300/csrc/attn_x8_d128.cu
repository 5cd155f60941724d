// The cache attention (attn_x8.cuh) for heads of 128.
#include "attn_x8.cuh"

namespace moe {

cudaError_t launch_attn_x8_d128(const AttnX8Params& p, int rows, int grid, cudaStream_t s) {
  switch (attn_x8_group_rows(128, rows)) {
    case 8: return attn::launch<128, 1, 1>(p, grid, s);
    case 16: return attn::launch<128, 2, 1>(p, grid, s);
    case 64: return attn::launch<128, 2, 4>(p, grid, s);
    default: return attn::launch<128, 2, 8>(p, grid, s);
  }
}

}  // namespace moe
