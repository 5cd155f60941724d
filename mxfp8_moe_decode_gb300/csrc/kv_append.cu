// Append of new keys and values to the 8-bit paged cache (kv_x8.cuh).
//
// Per page that new tokens fall into, per head, for keys and values apart:
//   code' = max(code of the page's earlier tokens, mx_code(amax of the new ones))
// (a page that starts with a new token has no earlier ones), the new values
// become E4M3_RNE(x * 2^(127 - code')), and where code' grew the earlier
// bytes are rounded again under it. Scales are powers of two, so a byte moves
// exactly unless it falls into E4M3's subnormals. The amax is that of the
// finite values: an infinite one is stored as +-448 under the code, a NaN as
// NaN, and neither touches the scale of its neighbours.
//
// Bound by memory for prompts (2 bytes read, 1 written per value) and by
// latency for a decode step. One CTA owns one (page, head, keys or values):
// no two CTAs write the same bytes, nothing is atomic. The pages are found
// without a scan: sequence b gets the slots cu_q[b] / 64 + 2 b .. , which are
// at least as many as the pages its tokens can touch, and a CTA whose slot has
// none leaves (all do where the rows' starts do not ascend). Keys are rows;
// values go through shared memory (16 tokens x 4 dims per thread, transposed
// with byte permutes) so that whole 16-byte chunks are stored.
// 8 heads of 128: two prompts of 4100 tokens 10.8 us (50 MB, 4.7 TB/s: 2100 CTAs
// are 1.7 times what the SMs hold, and each is a chain of page lookup, loads,
// maximum and stores; more resident CTAs by fewer registers took 15 to 18 us);
// 48 sequences of one token 3.6 us, one such chain. The values' CTAs, which do
// more, come first in the grid (the keys' first: 11.4 us).
//
// With rotary positions (kRope, rope.cuh) the keys' CTAs turn what they loaded
// and round it to bf16 before anything looks at it, so the cache gets the bytes
// it would get from keys that another kernel had turned. A thread loads both
// values of its pairs (chunks that neighbour lanes exchanged: 40.9 us in place
// of 38.5 below). Further CTAs of the same grid turn the queries, spread evenly
// among these: one launch for q, k and v, and the queries' stream fills the waits
// of the append's chains.
// 40 query heads of 128 over 8: two prompts of 4100 tokens 38.5 us (214 MB, 5.6
// TB/s; 32 at the copy's rate, 48 with the queries' CTAs behind the append's),
// bound by instructions: every key/value head's CTA makes the sines and cosines
// of its tokens. 48 sequences of one token 4.3 to 4.6 us in
// graph replays (by single calls from Python 11). By fewer registers 6 or 7 CTAs
// an SM in place of 5: 38.5 and 38.9, 4 x 128 tokens 9.0 in place of 8.5.
#include "internal.cuh"
#include "kv_x8.cuh"
#include "mx.cuh"
#include "ptx.cuh"
#include "rope.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kByteTokens = 8;  // this many new tokens or fewer: values are stored byte by byte

// Four E4M3 bytes times 2^-shift, rounded again.
__device__ __forceinline__ uint32_t requant4(uint32_t w, float mul) {
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (8 * j)) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    out |= static_cast<uint32_t>(e4m3x2(f.x * mul, f.y * mul)) << (8 * j);
  }
  return out;
}

__device__ __forceinline__ uint4 requant16(const uint4& v, float mul) {
  return make_uint4(requant4(v.x, mul), requant4(v.y, mul), requant4(v.z, mul),
                    requant4(v.w, mul));
}

// Largest magnitudes among 8 bf16 values, as two bf16 bit patterns; kFinite:
// infinities and NaN left out.
template <bool kFinite>
__device__ __forceinline__ uint32_t amax_bits(const uint4& v, uint32_t a) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t m = w[j] & 0x7FFF7FFFu;
    if (kFinite) m &= __vcmpltu2(m, 0x7F807F80u);
    a = __vmaxu2(a, m);
  }
  return a;
}

// 8 values times a power of two -> E4M3: exact in bf16 but for underflow, which
// lies far below E4M3's smallest value; saturating, so that +-inf becomes
// +-448, and NaN stays.
__device__ __forceinline__ uint2 quant8(const uint4& v, __nv_bfloat162 mul) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __bfloat1622float2(__hmul2(h[j], mul));
    b[j] = e4m3x2(f.x, f.y);
  }
  return make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
}

// The CTA's largest bf16 bit pattern.
__device__ __forceinline__ uint32_t cta_max(uint32_t a, uint32_t* red) {
  a = __reduce_max_sync(0xffffffffu, max(a >> 16, a & 0xFFFFu));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = max(a, red[i]);
  return a;
}

struct RopeAppendParams : KvAppendParams {
  rope::Spec spec;
  const int* positions;     // [tokens] or null: the tokens' places in the cache
  const __nv_bfloat16* q;
  __nv_bfloat16* q_out;
  long long ldq, ldqo;      // elements between tokens
  int q_heads, q_groups;    // threads (times D / 16) that share a token's heads
  unsigned slots;           // page slots
  unsigned q_share;         // the queries' part of the CTAs, in units of 2^-32, rounded up
};

// The keys that this thread loaded, turned: item j's two chunks of the tokens
// tid / kItems, + kThreads / kItems, ... of the CTA's (rope::item_chunks: both
// values of its pairs are here). One item's code, gone through in a loop that
// moves the chunks on by two (all of a thread's chunks unrolled, in an earlier
// form: 36 KB of code, 52 us where the loop took 42).
template <int D, int kMax>
__device__ __forceinline__ void turn_keys(const RopeAppendParams& p, uint4 (&v)[kMax], int count, int first_row,
                                          int first_pos) {
  constexpr int kItems = D / 16, kTokens = kThreads / kItems;
  const int j = threadIdx.x % kItems;
  if (16 * j >= p.spec.rot) return;  // (the item's dims do not turn)
  const ulonglong2* f = reinterpret_cast<const ulonglong2*>(p.spec.freqs + rope::kPairs * j);
  const auto turn_one = [&](uint4& a, uint4& b, int row) {
    const int pos = p.positions ? __ldg(p.positions + first_row + row) : first_pos + row;
    Pair c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 g = __ldg(f + i);
      rope::turn(pos, g.x, g.y, p.spec.scale, c[i], s[i]);
    }
    if (p.spec.interleaved) {
      rope::turn_neighbours(a, c, s);
      rope::turn_neighbours(b, c + 2, s + 2);
    } else {
      rope::turn_halves(a, b, c, s);
    }
  };
#pragma unroll 1
  for (int i = 0, row = threadIdx.x / kItems; i < kMax / 2; ++i, row += kTokens) {
    uint4 x = v[0], y = v[1];
    if (row < count) turn_one(x, y, row);
#pragma unroll
    for (int k = 0; k + 2 < kMax; ++k) v[k] = v[k + 2];
    v[kMax - 2] = x;
    v[kMax - 1] = y;
  }
}

// The CTA `block` of those that turn the queries. A row's sequence (its place
// in the cache is its position) is found as the append finds a slot's, from
// the CTA's first row on by halving.
template <int D>
__device__ __forceinline__ void turn_queries(const RopeAppendParams& p, unsigned block) {
  constexpr int kItems = D / 16;
  const unsigned per = kItems * p.q_groups;
  const long long u = static_cast<long long>(block) * kThreads + threadIdx.x;
  const int t0 = static_cast<int>(static_cast<long long>(block) * kThreads / per);
  const int token = static_cast<int>(u / per);
  const unsigned rest = static_cast<unsigned>(u - static_cast<long long>(token) * per);
  int b = token, c0 = token;
  if (p.cu_q) {
    int below = 0;
    bool falls = false;
#pragma unroll 1
    for (int i0 = 0; i0 < p.seqs; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      const int c = i < p.seqs ? p.cu_q[i] : 0;
      falls |= i < p.seqs && c > p.cu_q[i + 1];
      below += __syncthreads_count(i < p.seqs && c <= t0);
    }
    if (__syncthreads_or(falls)) return;  // (the append's CTAs say so)
    if (token >= p.tokens) return;
    if (token > t0) {
      int hi = p.seqs;  // the starts before `below` are <= token, those from hi on are not
      while (below < hi) {
        const int mid = (below + hi) >> 1;
        if (p.cu_q[mid] <= token)
          below = mid + 1;
        else
          hi = mid;
      }
    }
    b = below - 1;
    if (b < 0 || token >= p.cu_q[b + 1]) return;  // a row of no sequence
    c0 = max(p.cu_q[b], 0);
  } else if (token >= p.tokens) {
    return;
  }
  const int start = p.start[b];
  if (start < 0 || start > (1 << 30)) return;
  const int pos = p.positions ? __ldg(p.positions + token) : start + (token - c0);
  rope::Heads h;
  h.x = reinterpret_cast<const uint4*>(p.q + token * p.ldq);
  h.out = reinterpret_cast<uint4*>(p.q_out + token * p.ldqo);
  h.heads = p.q_heads;
  h.chunks = D / 8;
  rope::turn_heads(p.spec, h, pos, rest % kItems, rest / kItems, p.q_groups);
}

template <int D, typename Params>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const Params p) {
  constexpr bool kRope = !std::is_same<Params, KvAppendParams>::value;
  constexpr int kRowChunks = D / 8;                                // 16-byte chunks of a token
  constexpr int kMax = kPageTokens * kRowChunks / kThreads;        // chunks a thread holds
  constexpr int kPitch = D + 4;                                    // staged token row, bytes
  __shared__ __align__(16) uint8_t stage[kPageTokens * kPitch];
  __shared__ uint32_t red[2][kThreads / 32];
  const int tid = threadIdx.x;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  int slot_index, head, kv;
  if constexpr (kRope) {
    // One row of CTAs, the queries' spread evenly among the append's: CTA b is
    // the queries' where b q_share passes a whole number.
    const unsigned q = __umulhi(blockIdx.x, p.q_share);
    if (__umulhi(blockIdx.x + 1, p.q_share) != q) {
      turn_queries<D>(p, q);
      return;
    }
    const unsigned mine = blockIdx.x - q;
    slot_index = mine % p.slots;
    const int rest = mine / p.slots;
    head = rest % p.kv_heads;
    kv = 1 - rest / p.kv_heads;
  } else {
    slot_index = blockIdx.x;
    head = blockIdx.y;
    kv = 1 - blockIdx.z;
  }

  // the slot's sequence and page
  int b, c0, n, page_index;
  if (p.cu_q == nullptr) {
    b = slot_index;
    c0 = b;
    n = 1;
    page_index = p.start[b] / kPageTokens;
  } else {
    const long long slot = slot_index;
    int below = 0;
    bool falls = false;
#pragma unroll 1  // (unrolled, the code of one token a sequence grew too: 3.8 us)
    for (int i0 = 0; i0 < p.seqs; i0 += kThreads) {
      const int i = i0 + tid;
      if (i < p.seqs) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.start + i));  // read next
      const int c = i < p.seqs ? p.cu_q[i] : 0;
      falls |= i < p.seqs && c > p.cu_q[i + 1];
      const bool le = i < p.seqs &&
                      static_cast<long long>(min(max(c, 0), p.tokens) / kPageTokens) + 2ll * i <= slot;
      below += __syncthreads_count(le);
    }
    if (__syncthreads_or(falls)) {  // starts that do not ascend
      if (tid == 0 && slot_index == 0 && p.status) atomicOr(p.status, kKvErrLength);
      return;
    }
    b = max(below - 1, 0);
    c0 = min(max(p.cu_q[b], 0), p.tokens);
    n = min(max(p.cu_q[b + 1], c0), p.tokens) - c0;
    page_index = p.start[b] / kPageTokens +
                 static_cast<int>(slot - c0 / kPageTokens - 2ll * b);
  }
  const int start = p.start[b];
  if (n == 0) return;
  if (start < 0 || start > (1 << 30)) {
    if (tid == 0 && p.status) atomicOr(p.status, kKvErrLength);
    return;
  }
  const int base = page_index * kPageTokens;
  const int t0 = max(start, base), t1 = min(start + n, base + kPageTokens);
  if (t1 <= t0) return;
  const int off = t0 - base;  // the page's earlier tokens
  const int count = t1 - t0;
  const long long ld = kv ? p.ldv : p.ldk;
  const __nv_bfloat16* src = (kv ? p.v : p.k) + (c0 + (t0 - start)) * ld + static_cast<long long>(head) * D;

  // the values are on their way while the page is looked up
  uint4 v[kMax];
  // keys that are to be turned: chunk i is the first or second of an item's of the token `key_token(i)`
  constexpr int kItems = D / 16;
  int chunk[2] = {0, 0};
  const auto key_token = [tid](int i) { return tid / kItems + (i >> 1) * (kThreads / kItems); };
  const bool turned = kRope && kv == 0;
  if constexpr (kRope) {
    if (turned) {
      rope::item_chunks(p.spec, tid % kItems, chunk[0], chunk[1]);
#pragma unroll
      for (int i = 0; i < kMax; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (key_token(i) < count)
          v[i] = __ldcs(reinterpret_cast<const uint4*>(src + key_token(i) * ld) + chunk[i & 1]);
      }
      turn_keys<D>(p, v, count, c0 + (t0 - start), t0);
    }
  }
  if (!turned) {
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int c = tid + i * kThreads;
      v[i] = make_uint4(0, 0, 0, 0);
      if (c < count * kRowChunks)
        v[i] = __ldcs(reinterpret_cast<const uint4*>(src + (c / kRowChunks) * ld) + c % kRowChunks);
    }
  }
  int page = -1;
  if (page_index < p.max_pages)
    page = __ldg(p.page_table + static_cast<size_t>(b) * p.max_pages + page_index);
  if (page < 0 || page >= p.pages) {
    if (tid == 0 && p.status) atomicOr(p.status, page_index < p.max_pages ? kKvErrPage : kKvErrLength);
    return;
  }
  const size_t owner = (static_cast<size_t>(page) * p.kv_heads + head) * 2 + kv;
  uint8_t* img = p.blocks + owner * (static_cast<size_t>(kPageTokens) * D);
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kMax; ++i) a = amax_bits<false>(v[i], a);
  const int had = off > 0 ? min(static_cast<int>(p.codes[owner]), 254) : 0;
  a = cta_max(a, red[0]);
  if (a >= 0x7F80u) {  // (uniform) a value that is not finite: once more without those
    a = 0;
#pragma unroll
    for (int i = 0; i < kMax; ++i) a = amax_bits<true>(v[i], a);
    a = cta_max(a, red[1]);
  }
  const int code = max(had, mx_code(__uint_as_float(a << 16)));
  if (off > 0 && code > had) {
    // every byte is below 2^-10 from a shift of 19 on and rounds to zero, so
    // a larger shift gives the same bytes
    const float mul = mx_mul(127 + min(code - had, 40));
    if (kv == 0) {
      uint4* row = reinterpret_cast<uint4*>(img);
      for (int i = tid; i < off * (D / 16); i += kThreads) row[i] = requant16(row[i], mul);
    } else {
      // whole chunks: bytes past the earlier tokens are new ones (stored
      // below) or never read
      uint4* chunk = reinterpret_cast<uint4*>(img);
      for (int i = tid; i < D * 4; i += kThreads)
        if (((i & 3) ^ ((i >> 3) & 3)) * 16 < off) chunk[i] = requant16(chunk[i], mul);
    }
  }
  if (tid == 0) p.codes[owner] = static_cast<uint8_t>(code);
  const __nv_bfloat162 mul = __float2bfloat162_rn(mx_mul(code));
  if (turned) {
#pragma unroll
    for (int i = 0; i < kMax; ++i)
      if (key_token(i) < count)
        *reinterpret_cast<uint2*>(img + key_byte<D>(off + key_token(i), chunk[i & 1] * 8)) = quant8(v[i], mul);
    return;
  }
  if (kv == 0) {
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int c = tid + i * kThreads;
      if (c < count * kRowChunks)
        *reinterpret_cast<uint2*>(img + key_byte<D>(off + c / kRowChunks, (c % kRowChunks) * 8)) =
            quant8(v[i], mul);
    }
    return;
  }
  __syncthreads();  // the requantised chunks before the new bytes in them
  if (count <= kByteTokens) {
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int c = tid + i * kThreads;
      if (c >= count * kRowChunks) break;
      const uint2 q = quant8(v[i], mul);
      const int t = off + c / kRowChunks, d = (c % kRowChunks) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        img[value_byte(t, d + j)] = static_cast<uint8_t>((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kMax; ++i) {
    const int c = tid + i * kThreads;
    if (c >= count * kRowChunks) break;
    const uint2 q = quant8(v[i], mul);
    uint32_t* d = reinterpret_cast<uint32_t*>(stage + (off + c / kRowChunks) * kPitch + (c % kRowChunks) * 8);
    d[0] = q.x;
    d[1] = q.y;
  }
  __syncthreads();
  // unit = (16-token chunk, 4 dims): 16 words in, four 16-byte chunks out; four
  // neighbouring lanes store a whole row (the chunks of one number: 0.5 us more)
  for (int u = tid; u < 4 * (D / 4); u += kThreads) {
    const int ch = u & 3, d0 = (u >> 2) * 4;
    const int lo = ch * 16, hi = lo + 16;
    if (hi <= off || lo >= off + count) continue;
    const bool whole = lo >= off && hi <= off + count;
    uint32_t o[4][4];  // [dim][word]
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = lo + 2 * w + (j & 1) + (j >> 1) * 8;
        x[j] = t >= off && t < off + count ? *reinterpret_cast<const uint32_t*>(stage + t * kPitch + d0) : 0u;
      }
      const uint32_t a01 = __byte_perm(x[0], x[1], 0x5140), b01 = __byte_perm(x[0], x[1], 0x7362);
      const uint32_t a23 = __byte_perm(x[2], x[3], 0x5140), b23 = __byte_perm(x[2], x[3], 0x7362);
      o[0][w] = __byte_perm(a01, a23, 0x5410);
      o[1][w] = __byte_perm(a01, a23, 0x7632);
      o[2][w] = __byte_perm(b01, b23, 0x5410);
      o[3][w] = __byte_perm(b01, b23, 0x7632);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint8_t* dst = img + (d0 + j) * kPageTokens + ((ch ^ (((d0 + j) >> 1) & 3)) << 4);
      if (whole) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int t = lo + 2 * (k >> 2) + (k & 1) + ((k >> 1) & 1) * 8;
          if (t >= off && t < off + count) dst[k] = static_cast<uint8_t>(o[j][k >> 2] >> (8 * (k & 3)));
        }
      }
    }
  }
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; }

}  // namespace
}  // namespace moe

namespace moe {
namespace {

// The checks and parameters that both entry points share; rows > 0 after MOE_OK.
int append_params(const moe_kv_cache* cache, const moe_kv_seqs* seqs, const void* k, int64_t ldk, const void* v,
                  int64_t ldv, int32_t* status, KvAppendParams& p) {
  if (!k || !v) return MOE_ERR_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || ldk % 8 || ldv % 8 || (status && !aligned(status, 4)))
    return MOE_ERR_ALIGN;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  if (ldk < width || ldv < width) return MOE_ERR_ARG;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.ldk = ldk;
  p.ldv = ldv;
  p.blocks = cache->blocks;
  p.codes = cache->codes;
  p.page_table = seqs->page_table;
  p.start = seqs->lens;
  p.cu_q = seqs->cu_q;
  p.status = status;
  p.tokens = seqs->tokens;
  p.seqs = seqs->seqs;
  p.max_pages = seqs->max_pages;
  p.pages = cache->pages;
  p.kv_heads = cache->kv_heads;
  return MOE_OK;
}

unsigned slots_of(const KvAppendParams& p) {
  return p.cu_q ? static_cast<unsigned>(p.tokens / kPageTokens + 2 * p.seqs) : static_cast<unsigned>(p.seqs);
}

template <typename Params>
int launch_append(const Params& p, int head_dim, dim3 grid, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (head_dim) {
    case 64: e = launch_pdl(kv_append_kernel<64, Params>, grid, dim3(kThreads), 0, st, p); break;
    case 128: e = launch_pdl(kv_append_kernel<128, Params>, grid, dim3(kThreads), 0, st, p); break;
    default: e = launch_pdl(kv_append_kernel<256, Params>, grid, dim3(kThreads), 0, st, p); break;
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_kv_append_x8(const moe_kv_cache* cache, const moe_kv_seqs* seqs, const void* k,
                                int64_t ldk, const void* v, int64_t ldv, int32_t* status,
                                void* stream) {
  using namespace moe;
  int rc = kv_check(cache, seqs);
  if (rc != MOE_OK) return rc;
  if (seqs->tokens == 0) return MOE_OK;
  KvAppendParams p;
  rc = append_params(cache, seqs, k, ldk, v, ldv, status, p);
  if (rc != MOE_OK) return rc;
  return launch_append(p, cache->head_dim, dim3(slots_of(p), cache->kv_heads, 2), stream);
}

extern "C" int moe_rope_kv_append_x8(const moe_kv_cache* cache, const moe_kv_seqs* seqs,
                                     const moe_rope_spec* spec, const int32_t* positions, const void* q,
                                     int64_t ldq, int q_heads, void* q_out, int64_t ldqo, const void* k,
                                     int64_t ldk, const void* v, int64_t ldv, int32_t* status,
                                     void* stream) {
  using namespace moe;
  int rc = kv_check(cache, seqs);
  if (rc != MOE_OK) return rc;
  if (!spec) return MOE_ERR_ARG;
  rc = rope::check(spec->freqs, spec->first, spec->rot, cache->head_dim, spec->scale);
  if (rc != MOE_OK) return rc;
  if (q_heads < 1 || q_heads > 4096) return MOE_ERR_UNSUPPORTED;
  if (seqs->tokens == 0) return MOE_OK;
  RopeAppendParams p;
  rc = append_params(cache, seqs, k, ldk, v, ldv, status, p);
  if (rc != MOE_OK) return rc;
  if (!q || !q_out) return MOE_ERR_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(positions, 4) || ldq % 8 || ldqo % 8) return MOE_ERR_ALIGN;
  const int64_t width = static_cast<int64_t>(q_heads) * cache->head_dim;
  if (ldq < width || ldqo < width || (q == q_out && ldq != ldqo)) return MOE_ERR_ARG;
  p.spec = {spec->freqs, spec->first, spec->rot, spec->interleaved != 0, spec->scale};
  p.positions = positions;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.ldq = ldq;
  p.ldqo = ldqo;
  p.q_heads = q_heads;
  p.q_groups = rope::head_groups(p.tokens, q_heads, cache->head_dim, true);
  p.slots = slots_of(p);
  const int64_t ctas = static_cast<int64_t>(p.slots) * cache->kv_heads * 2;
  const int64_t q_ctas =
      (static_cast<int64_t>(p.tokens) * p.q_groups * (cache->head_dim / 16) + kThreads - 1) / kThreads;
  if (ctas + q_ctas > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  // (ceil(q 2^32 / all): all times it passes q, not q + 1, whole numbers, as all < 2^32; q < all)
  p.q_share = static_cast<unsigned>(((static_cast<uint64_t>(q_ctas) << 32) + (ctas + q_ctas) - 1) / (ctas + q_ctas));
  return launch_append(p, cache->head_dim, dim3(static_cast<unsigned>(ctas + q_ctas)), stream);
}
