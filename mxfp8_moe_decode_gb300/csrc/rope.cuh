// Rotary positions. Pair i of a head's rotated dims turns by the angle
//   a = pos * f_i  (in turns),   (u, v) -> scale * (u cos a - v sin a, v cos a + u sin a),
// with f_i a 64-bit fixed-point number of 2^-64 turns per position. The product
// with a 32-bit position, modulo 2^64, is the angle without its whole turns,
// exactly: no position is too far for it (fp32 products of positions and
// frequencies are off by 0.004 turns at a position of 131072). Of the angle
// the upper 32 bits are kept (to nearest: off by 2^-33 turns, 7e-10 radians).
//
// Sine and cosine: the turn is cut to the nearest quarter, the rest within an
// eighth of a turn (pi / 4) by their Taylor series: sine up to x^9, cosine up to
// x^8 (the terms left out are below 2e-9 and 3e-8), in fp32.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "f32x2.cuh"

namespace moe {
namespace rope {

constexpr int kPairs = 8;  // pairs that a thread turns together

struct Spec {
  const uint64_t* freqs;  // [rot / 2]
  int first, rot;         // the rotated dims first .. first + rot - 1 (multiples of 8 and 16)
  int interleaved;        // pairs (2 i, 2 i + 1) of them, else (i, i + rot / 2)
  float scale;
};

// cos and sin (times scale) of pos * f0 and pos * f1 turns.
__device__ __forceinline__ void turn(int pos, uint64_t f0, uint64_t f1, float scale, Pair& c, Pair& s) {
  const auto phase = [pos](uint64_t f) {
    return static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(pos)) * f + 0x80000000ull) >> 32);
  };
  const uint32_t a0 = phase(f0), a1 = phase(f1);
  const uint32_t q0 = (a0 + 0x20000000u) >> 30, q1 = (a1 + 0x20000000u) >> 30;  // the nearest quarters
  const auto number = [](float v) { return pair(v, v); };
  const Pair x = mul(pair(static_cast<float>(static_cast<int32_t>(a0 - (q0 << 30))),
                          static_cast<float>(static_cast<int32_t>(a1 - (q1 << 30)))),
                     number(0x1.921fb6p-30f));  // 2 pi 2^-32
  const Pair z = mul(x, x);
  Pair sn = fma(z, number(1.0f / 362880.0f), number(-1.0f / 5040.0f));
  sn = fma(z, sn, number(1.0f / 120.0f));
  sn = fma(z, sn, number(-1.0f / 6.0f));
  sn = mul(fma(mul(z, x), sn, x), number(scale));
  Pair cs = fma(z, number(1.0f / 40320.0f), number(-1.0f / 720.0f));
  cs = fma(z, cs, number(1.0f / 24.0f));
  cs = fma(z, cs, number(-0.5f));
  cs = mul(fma(z, cs, number(1.0f)), number(scale));
  // a quarter turn: (cos, sin) -> (-sin, cos)
  const float2 u = floats(cs), v = floats(sn);
  const auto sign = [](float w, uint32_t flip) { return __uint_as_float(__float_as_uint(w) ^ (flip << 31)); };
  c = pair(sign(q0 & 1 ? v.x : u.x, (q0 + 1) >> 1), sign(q1 & 1 ? v.y : u.y, (q1 + 1) >> 1));
  s = pair(sign(q0 & 1 ? u.x : v.x, q0 >> 1), sign(q1 & 1 ? u.y : v.y, q1 >> 1));
}

__device__ __forceinline__ uint32_t rounded(Pair a) {
  const float2 f = floats(a);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pairs (u, v), turned: u cos - v sin and v cos + u sin. (One order of
// operations wherever a pair is turned, so every kernel gives the same bits.)
__device__ __forceinline__ Pair first_of(Pair u, Pair v, Pair c, Pair s) { return fma(u, c, mul(v, negated(s))); }
__device__ __forceinline__ Pair second_of(Pair u, Pair v, Pair c, Pair s) { return fma(v, c, mul(u, s)); }

// 8 pairs whose first values are in a, second ones in b.
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const Pair* c, const Pair* s) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  uint32_t* y = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Pair u = pair(x[j]), v = pair(y[j]);
    x[j] = rounded(first_of(u, v, c[j], s[j]));
    y[j] = rounded(second_of(u, v, c[j], s[j]));
  }
}

// 4 pairs of neighbours.
__device__ __forceinline__ void turn_neighbours(uint4& a, const Pair* c, const Pair* s) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 p = floats(pair(x[2 * j])), q = floats(pair(x[2 * j + 1]));
    const Pair u = pair(p.x, q.x), v = pair(p.y, q.y);
    const float2 m = floats(first_of(u, v, c[j], s[j])), n = floats(second_of(u, v, c[j], s[j]));
    x[2 * j] = rounded(pair(m.x, n.x));
    x[2 * j + 1] = rounded(pair(m.y, n.y));
  }
}

// A head of 16-byte chunks is cut into dim / 16 items of two chunks: first the
// rot / 16 that hold 8 pairs each, then the dims that do not turn. Returns
// whether item j turns (its pairs are 8 j .. 8 j + 7).
__device__ __forceinline__ bool item_chunks(const Spec& r, int j, int& c0, int& c1) {
  const int f = r.first >> 3, half = r.rot >> 4;
  if (j < half) {
    c0 = f + (r.interleaved ? 2 * j : j);
    c1 = f + (r.interleaved ? 2 * j + 1 : j + half);
    return true;
  }
  const int u = 2 * (j - half);
  c0 = u < f ? u : u + 2 * half;
  c1 = u + 1 < f ? u + 1 : u + 1 + 2 * half;
  return false;
}

// The same item j of the heads h0, h0 + step, ... of one token.
struct Heads {
  const uint4* x;  // the token's rows, 16-byte chunks
  uint4* out;
  int heads, chunks;  // chunks of a head
};

__device__ __forceinline__ void turn_heads(const Spec& r, const Heads& t, int pos, int j, int h0, int step) {
  int c0, c1;
  const bool turns = item_chunks(r, j, c0, c1);
  constexpr int kAhead = 4;  // heads whose loads are under way together
  Pair c[kPairs / 2], s[kPairs / 2];
  bool have = false;
  for (int h = h0; h < t.heads; h += kAhead * step) {
    uint4 a[kAhead], b[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int hi = h + i * step;
      if (hi < t.heads) {
        a[i] = __ldcs(t.x + hi * t.chunks + c0);
        b[i] = __ldcs(t.x + hi * t.chunks + c1);
      }
    }
    if (turns && !have) {  // (under the loads)
#pragma unroll
      for (int i = 0; i < kPairs; i += 2) {
        const ulonglong2 f = __ldg(reinterpret_cast<const ulonglong2*>(r.freqs + kPairs * j + i));
        turn(pos, f.x, f.y, r.scale, c[i / 2], s[i / 2]);
      }
      have = true;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int hi = h + i * step;
      if (hi >= t.heads) break;
      if (turns) {
        if (r.interleaved) {
          turn_neighbours(a[i], c, s);
          turn_neighbours(b[i], c + 2, s + 2);
        } else {
          turn_halves(a[i], b[i], c, s);
        }
      }
      t.out[hi * t.chunks + c0] = a[i];
      t.out[hi * t.chunks + c1] = b[i];
    }
  }
}

// Threads that share a token's heads. A thread's sines and cosines serve its
// heads, but a small call lasts as long as one thread's chain. 40 heads of 128,
// with 1, 4, 8 and 16 heads a thread (us):
//   alone: 48 tokens (15000 items of 16 dims) 1.8, 2.0, 2.6, 3.6; 300: 2.9, 2.7, 3.5,
//     5.3; 1000: 7.5, 5.4, 6.0, 7.2; 2000: 12.6, 8.6, 8.4, 9.6; 8000: 46.9, 26.5, 26.5, 27.4
//   with the append, whose own chains are longer: 48 tokens 4.8, 4.6, 4.5, 5.3; 512:
//     10.4, 9.1, 8.7, 8.5; 2000: 24.0, 16.9, 15.9, 14.7; 8200: 76.9, 45.3, 41.8, 40.9
inline int head_groups(int64_t tokens, int heads, int dim, bool with_append) {
  const int64_t items = tokens * heads * (dim / 16);
  const int each = with_append ? (items <= 152 * 1024 ? 8 : 16) : items <= 152 * 256 ? 1 : items <= 152 * 3000 ? 4 : 8;
  return (heads + each - 1) / each;
}

// Argument checks shared by the entry points.
inline int check(const uint64_t* freqs, int first, int rot, int head_dim, float scale) {
  if (rot < 16 || rot % 16 || first < 0 || first % 8 || first + static_cast<int64_t>(rot) > head_dim)
    return MOE_ERR_UNSUPPORTED;
  if (scale - scale != 0.0f) return MOE_ERR_ARG;
  if (!freqs) return MOE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(freqs) & 15) return MOE_ERR_ALIGN;
  return MOE_OK;
}

}  // namespace rope
}  // namespace moe
