// The 8-bit paged key/value cache: the layout of a page's images, its scale
// codes, and the parameter blocks of the kernels that write and read it.
//
// A page holds kPageTokens tokens. Per page and head the cache keeps 2 x
// (64 * D) bytes, first the image of the keys and then that of the values
// (E4M3), and two E8M0 codes: a byte b under code c stands for
// e4m3(b) * 2^(c - 127). The images are what the tensor-core kernel reads from
// shared memory, so one contiguous bulk copy stages each and eight rows of a
// matrix load touch eight different 16-byte columns of the banks:
//  keys    one row of D bytes per token; its 16-byte chunk c sits at chunk
//          c ^ s(token), s(t) = t % 8 (rows of 128 bytes and more) or
//          (t / 2) % 4 (rows of 64 bytes);
//  values  transposed, one row of 64 bytes per dim: the tokens' axis is the
//          one the product with the softmax weights contracts. The chunk of
//          tokens 16 c .. 16 c + 15 sits at chunk c ^ ((dim / 2) % 4), and in
//          it word i holds the tokens 2 i, 2 i + 1, 2 i + 8, 2 i + 9: the four
//          a thread of a 16-wide MMA step owns.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/moe_decode.h"

namespace moe {

constexpr int kPageTokens = MOE_KV_PAGE_TOKENS;
constexpr int kItemCost = 10;  // pages that an item of the attention's work list counts for beside its own
static_assert(kPageTokens == 64, "the images' chunk permutations are written for 64 tokens");

// error bits in the status word of the cache kernels
constexpr int kKvErrTimeout = MOE_KV_STATUS_TIMEOUT;
constexpr int kKvErrPage = MOE_KV_STATUS_PAGE;
constexpr int kKvErrLength = MOE_KV_STATUS_LENGTH;

template <int D>
__host__ __device__ __forceinline__ int key_swizzle(int token) {
  return D >= 128 ? (token & 7) : ((token >> 1) & 3);
}

// Byte of (token, dim) in a page's key image.
template <int D>
__host__ __device__ __forceinline__ int key_byte(int token, int dim) {
  return token * D + (((dim >> 4) ^ key_swizzle<D>(token)) << 4) + (dim & 15);
}

// Byte of a token inside its 16-token chunk of a value row.
__host__ __device__ __forceinline__ int value_slot(int j) {
  return ((j & 7) >> 1) * 4 + (j >> 3) * 2 + (j & 1);
}

// Byte of (token, dim) in a page's value image.
__host__ __device__ __forceinline__ int value_byte(int token, int dim) {
  return dim * kPageTokens + (((token >> 4) ^ ((dim >> 1) & 3)) << 4) + value_slot(token & 15);
}

// 2^(code - 127) as fp32 (code 0 is the subnormal 2^-127).
__device__ __forceinline__ float e8m0_value(int code) {
  return __uint_as_float(code == 0 ? 0x00400000u : static_cast<uint32_t>(code) << 23);
}

// Argument checks shared by the cache's entry points.
inline int kv_check(const moe_kv_cache* c, const moe_kv_seqs* s) {
  if (!c || !s) return MOE_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
  if (c->kv_heads < 1 || c->kv_heads > 1024) return MOE_ERR_UNSUPPORTED;
  if (c->pages < 1 || s->max_pages < 1 || s->max_pages > (1 << 24)) return MOE_ERR_ARG;
  if (s->seqs < 0 || s->seqs > (1 << 20) || s->tokens < 0 || s->tokens > (1 << 24))
    return MOE_ERR_RANGE;
  if (!s->cu_q && s->tokens != s->seqs) return MOE_ERR_ARG;
  if (s->tokens > 0 && s->seqs == 0) return MOE_ERR_ARG;
  if (s->tokens == 0) return MOE_OK;
  if (!c->blocks || !c->codes || !s->page_table || !s->lens) return MOE_ERR_ARG;
  const auto off = [](const void* q, uintptr_t a) { return reinterpret_cast<uintptr_t>(q) & (a - 1); };
  if (off(c->blocks, 16) || off(c->codes, 2) || off(s->page_table, 4) || off(s->lens, 4) ||
      off(s->cu_q, 4))
    return MOE_ERR_ALIGN;
  return MOE_OK;
}

struct KvAppendParams {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long ldk, ldv;      // elements between tokens
  uint8_t* blocks;         // [pages][kv_heads][2][64 * D]
  uint8_t* codes;          // [pages][kv_heads][2]
  const int* page_table;   // [seqs][max_pages]
  const int* start;        // [seqs] tokens a sequence had
  const int* cu_q;         // [seqs + 1] or null: one new token a sequence
  int* status;             // or null
  int tokens, seqs, max_pages, pages, kv_heads;
};

struct AttnX8Params {
  const __nv_bfloat16* q;
  long long ldq;           // elements between tokens
  const uint8_t* blocks;
  const uint8_t* codes;
  const int* page_table;
  const int* kv_len;       // [seqs] tokens in the cache, the new ones included
  const int* cu_q;         // [seqs + 1] or null: one query token a sequence
  __nv_bfloat16* out;      // [tokens][q_heads][D]
  float* lse;              // [tokens][q_heads] or null
  float* part;             // workspace: partial rows of items that several CTAs share
  int* tickets;            // workspace: [grid] CTAs of a shared item that are done (0 between calls)
  void* records;           // workspace: [grid] the shared item that starts in a CTA (attn_wide.cuh)
  int* status;             // or null
  int tokens, seqs, max_pages, pages, kv_heads, group;
  unsigned group_magic;    // floor(2^32 / group) + 1 (unused for a group of 1)
  int max_kv;              // 64 * max_pages, the longest a sequence can be
  int window, sinks;
  float scale_log2;        // scale * log2(e)
};

// one instantiation per head dim (their own translation units); `rows`: the
// largest number of query rows of one sequence and key/value head
cudaError_t launch_attn_x8_d64(const AttnX8Params& p, int rows, int device, int grid,
                               cudaStream_t s);
cudaError_t launch_attn_x8_d128(const AttnX8Params& p, int rows, int device, int grid,
                               cudaStream_t s);
cudaError_t launch_attn_x8_d256(const AttnX8Params& p, int rows, int device, int grid,
                               cudaStream_t s);
// rows of one row group for that many query rows
int attn_x8_group_rows(int head_dim, int rows);

}  // namespace moe
