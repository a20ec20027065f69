// dropout.cuh -- which elements of the softmax a call with dropout keeps.
//
// Element (b, h, i, j) is kept where an 8-bit number u(b, h, i, j) is at least
// T = round(256 p).  The numbers come from Philox4x32 ("Parallel random numbers: as
// easy as 1, 2, 3", Salmon et al. 2011) with seven rounds, the fewest that the
// paper finds to pass every test of BigCrush (ten, its default, would cost 40 % more of
// the integer work that bounds these kernels' dropout).  A group of 32 keys of a
// row has eight words, from the counters (i, 2 g, bh, offset) and (i, 2 g + 1, bh, offset),
// g = j / 32: bit j % 32 of word k is bit k of u.  So u >= T for a whole group is
// eight bitwise majorities -- from the lowest bit on, at_least = T's bit is set ?
// u & at_least : u | at_least -- and a group's verdict is one word, whoever asks for it:
// the forward's thread has a row, the backward's a key.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

// A number that is the same in all lanes, as the warp's (the reduction's result is one register a warp).
__device__ __forceinline__ uint32_t warp_number(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

struct DropKey {
  uint32_t seed0 = 0, seed1 = 0, offset = 0;
  __device__ __forceinline__ DropKey(const DropParams& p, bool on) {
    if (!on) return;
    const unsigned long long seed = p.rng[0];
    seed0 = (uint32_t)seed;
    seed1 = (uint32_t)(seed >> 32);
    offset = (uint32_t)p.rng[1];
  }
  // The same in what the compiler can tell to be one number a warp: round keys and the rounds that
  // no lane's own numbers have entered are then kept and computed once a warp.
  __device__ __forceinline__ void uniform() {
    seed0 = warp_number(seed0);
    seed1 = warp_number(seed1);
    offset = warp_number(offset);
  }
};

// Words of the groups g0 .. g0 + G - 1 of row i and head bh: bit k for key 32 g + k, 1: kept.
// The 2 G counters go through the rounds side by side and share what they have in common.
template <int G>
__device__ __forceinline__ void keep_words(uint32_t (&keep)[G], uint32_t i, uint32_t bh, uint32_t g0, const DropKey& key,
                                           const DropParams& p) {
  uint32_t c[2 * G][4];
#pragma unroll
  for (int n = 0; n < 2 * G; ++n) {
    c[n][0] = i;
    c[n][1] = 2 * g0 + n;
    c[n][2] = bh;
    c[n][3] = key.offset;
  }
  uint32_t k0 = key.seed0, k1 = key.seed1;
#pragma unroll
  for (int r = 0; r < 7; ++r) {
#pragma unroll
    for (int n = 0; n < 2 * G; ++n) {
      const uint64_t a = (uint64_t)c[n][0] * 0xD2511F53u, b = (uint64_t)c[n][2] * 0xCD9E8D57u;
      c[n][0] = (uint32_t)(b >> 32) ^ c[n][1] ^ k0;
      c[n][1] = (uint32_t)b;
      c[n][2] = (uint32_t)(a >> 32) ^ c[n][3] ^ k1;
      c[n][3] = (uint32_t)a;
    }
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint32_t m = 0xffffffffu;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t u = c[2 * g + k / 4][k % 4], n = p.not_t[k];
      m = (u & m) | (n & (u | m));
    }
    keep[g] = m;
  }
}

// All ones in the halves of a packed pair that bits c and c + 1 (c even) keep.
__device__ __forceinline__ uint32_t pair_mask(uint32_t keep, int c) {
  const uint32_t a = keep << (7 - c % 8), b = keep << (6 - c % 8);  // the bits, each at the top of byte c / 8
  const uint32_t k = c / 8;
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"((8 | k) * 0x11 | (12 | k) * 0x1100));
  return r;
}

// Transpose of a 32 x 32 bit matrix, a row a lane: bit k of lane l to bit l of lane k.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    // Lanes without bit s keep the columns without it, and get the others from what the
    // lane with it has there; and the other way round.
    const uint32_t low = s == 16 ? 0x0000ffffu : s == 8 ? 0x00ff00ffu : s == 4 ? 0x0f0f0f0fu : s == 2 ? 0x33333333u : 0x55555555u;
    const bool upper = lane & s;
    const uint32_t own = upper ? ~low : low;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, s);
    x = (x & own) | (__funnelshift_l(y, y, upper ? 32 - s : s) & ~own);
  }
  return x;
}

}  // namespace attn
