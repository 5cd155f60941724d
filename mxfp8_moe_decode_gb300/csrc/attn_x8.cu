// Host side of the cache attention: argument checks, the choice of the kernel
// variant, and the workspace's layout (tickets, records, then two partial
// blocks per CTA).
#include <cmath>

#include "internal.cuh"
#include "kv_x8.cuh"

namespace moe {

// Rows of a row group for `rows` query rows of one sequence and key/value head.
// Up to 8: a warp per page, one tile of rows (attn_x8.cuh). Up to 16: two warps
// that share the pages (D = 128; 48 sequences over 3.5k tokens, 8 heads: 77 us,
// two tiles on one warp 94) or two tiles on one warp (D = 64: 49 us, two warps
// 52 to 58). Beyond: the tcgen05 kernel's two tiles of 128 (32 rows over 12 such
// sequences: 43 us, two tiles on each of two warps 55; for 16 rows it takes
// 132). Heads of 256, whose key rows are not an operand tile of it, have pages
// shared by two or three warps: a group of 16 rows takes 51 us where one of 24
// takes 64 (12 sequences), so the split of less work in that ratio is chosen.
int attn_x8_group_rows(int head_dim, int rows) {
  if (rows <= 8) return 8;
  if (head_dim == 256) return 4 * ((rows + 15ll) / 16) <= 5 * ((rows + 23ll) / 24) ? 16 : 24;
  return rows <= 16 ? 16 : 256;
}

namespace {

constexpr int kMaxGrid = 384;
constexpr size_t kTicketBytes = 4096;               // 4 bytes a CTA
constexpr size_t kHeadBytes = kTicketBytes + 12288;  // and 32 bytes a CTA of records

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

size_t workspace_bytes(int grid, int head_dim, int rows) {
  return kHeadBytes + static_cast<size_t>(grid) * 2 * attn_x8_group_rows(head_dim, rows) *
                            (head_dim + 2) * sizeof(float);
}

}  // namespace
}  // namespace moe

extern "C" int moe_attn_x8(const moe_kv_cache* cache, const moe_kv_seqs* seqs, const void* q,
                           int64_t ldq, int q_heads, float scale, int window, int sinks, void* out,
                           float* lse, void* workspace, size_t workspace_size, int32_t* status,
                           void* stream) {
  using namespace moe;
  const int rc = kv_check(cache, seqs);
  if (rc != MOE_OK) return rc;
  if (q_heads < 1 || q_heads % cache->kv_heads) return MOE_ERR_ARG;
  const int group = q_heads / cache->kv_heads;
  if (group > 256) return MOE_ERR_UNSUPPORTED;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.0f) || std::isinf(scale_log2) || window < 0 || sinks < 0) return MOE_ERR_ARG;
  if (seqs->max_q < 1) return MOE_ERR_ARG;
  if (seqs->tokens == 0) return MOE_OK;
  if (!q || !out || !workspace) return MOE_ERR_ARG;
  if (!aligned(q, 16) || ldq % 8 || !aligned(out, 16) || !aligned(workspace, 16) ||
      (lse && !aligned(lse, 4)) || (status && !aligned(status, 4)))
    return MOE_ERR_ALIGN;
  if (ldq < static_cast<int64_t>(q_heads) * cache->head_dim) return MOE_ERR_ARG;
  const int max_q = seqs->cu_q ? (seqs->max_q < seqs->tokens ? seqs->max_q : seqs->tokens) : 1;
  const int rows = max_q > (1 << 20) / group ? 1 << 20 : max_q * group;
  // Rows, the list of pages and its cut into equal runs (rounded up: at most a
  // position a CTA more) are counted in 32 bits, whatever the lengths on the device.
  if (static_cast<long long>(seqs->tokens) * group * group > UINT32_MAX) return MOE_ERR_UNSUPPORTED;
  const long long groups =
      static_cast<long long>(seqs->tokens) * group / attn_x8_group_rows(cache->head_dim, rows) + seqs->seqs;
  if (groups * cache->kv_heads > (INT32_MAX - kMaxGrid) / (static_cast<long long>(seqs->max_pages) + kItemCost))
    return MOE_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  const int grid = sms < kMaxGrid ? sms : kMaxGrid;
  if (workspace_size < workspace_bytes(grid, cache->head_dim, rows)) return MOE_ERR_ARG;
  AttnX8Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.blocks = cache->blocks;
  p.codes = cache->codes;
  p.page_table = seqs->page_table;
  p.kv_len = seqs->lens;
  p.cu_q = seqs->cu_q;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.tickets = static_cast<int*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeadBytes);
  p.records = static_cast<uint8_t*>(workspace) + kTicketBytes;
  p.status = status;
  p.tokens = seqs->tokens;
  p.seqs = seqs->seqs;
  p.max_pages = seqs->max_pages;
  p.pages = cache->pages;
  p.kv_heads = cache->kv_heads;
  p.group = group;
  p.group_magic = static_cast<unsigned>((1ull << 32) / static_cast<unsigned>(group) + 1);
  p.max_kv = seqs->max_pages * kPageTokens;
  // A window as long as the longest sequence hides nothing, and one below that
  // keeps position - window in 32 bits for rows before the first token too.
  p.window = window < p.max_kv ? window : 0;
  p.sinks = sinks;
  p.scale_log2 = scale_log2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (cache->head_dim) {
    case 64: e = launch_attn_x8_d64(p, rows, dev, grid, st); break;
    case 128: e = launch_attn_x8_d128(p, rows, dev, grid, st); break;
    default: e = launch_attn_x8_d256(p, rows, dev, grid, st); break;
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
