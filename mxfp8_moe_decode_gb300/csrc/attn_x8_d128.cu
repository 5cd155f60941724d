// The cache attention for heads of 128: up to 16 rows of a sequence and
// key/value head in attn_x8.cuh's kernel, more in attn_wide.cuh's.
#include "attn_wide.cuh"

namespace moe {

cudaError_t launch_attn_x8_d128(const AttnX8Params& p, int rows, int device, int grid, cudaStream_t s) {
  switch (attn_x8_group_rows(128, rows)) {
    case 8: return attn::launch<128, 1, 1>(p, device, grid, s);
    case 16: return attn::launch<128, 1, 2>(p, device, grid, s);
    default: return attn::launch_wide<128>(p, device, grid, s);
  }
}

}  // namespace moe
