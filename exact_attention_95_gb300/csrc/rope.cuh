// rope.cuh -- rotary positions: the angle of a position, and the rotation of
// rows of bf16 or fp32 elements.
//
// Pair i of a row's first `rot` elements (x1, x2) turns by angle a_i = 2 pi * frac(pos * f_i):
//   y1 = A (x1 cos a_i - x2 sin a_i),   y2 = A (x2 cos a_i + x1 sin a_i),
// with A the amplitude; its gradient turns the other way.  Pairs are (i, i + rot / 2), or
// (2 i, 2 i + 1) interleaved.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

// cos and sin of 2 pi * pos * freq / 2^64.  Frequencies are fractions of a turn in
// units of 2^-64, so the product keeps the fraction of a turn exactly
// for every 32-bit position (a 32-bit float angle is off by 0.01 rad at 131072).
// The nearest quarter turn is taken off in whole numbers; the rest, within
// pi / 4, goes through Taylor's series up to x^9 and x^8 (cut off below 3e-8).
// About 20 instructions.  Off by less than 3 * 2^-24, in units of 2^-24: the angle has the
// product's cut at 2^-32 of a turn (0.03) and a rounding each of the conversion, the constant and their
// product (3 x, which moves cos and sin by x sin x and x cos x, below 0.56, times 3: 1.67);
// cos then its last sum's (0.5), z's (z / 2, 0.31), the inner terms' (0.07) and the rest of the series
// (0.41), sin its last sum's (0.5), the inner terms' (0.33) and the rest (0.03).
__device__ __forceinline__ void cos_sin(uint32_t pos, uint64_t freq, float& c, float& s) {
  const uint32_t t = __umulhi(pos, (uint32_t)freq) + pos * (uint32_t)(freq >> 32);  // of pos * freq, the upper half
  const uint32_t q = (t + 0x20000000u) >> 30;
  const float x = (float)(int)(t - (q << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = x * x;
  const float sx = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
  const float cx = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320, -1.f / 720), 1.f / 24), -0.5f), 1.f);
  c = (q & 1) ? sx : cx;
  s = (q & 1) ? cx : sx;
  if ((q + 1) & 2) c = -c;
  if (q & 2) s = -s;
}

// Rows' elements, eight at a time.
template <class T>
struct Eight;
template <>
struct Eight<uint16_t> {  // bf16
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    v = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

constexpr int kRopeThreads = 256;
// Tokens of a CTA: a thread has 16 elements of a row (eight pairs).
constexpr int rope_tokens(int d) { return kRopeThreads / (d / 16); }

// Rotates `heads` heads from head `h0` on of a group of rope_tokens(D) tokens.
//
// HBM bound: every element is read and written once.  A thread computes the
// eight angles of its pairs of one token once and takes all the CTA's heads
// through them, a batch of heads' loads ahead of their use.  Measured (rope_kernel): 8192
// tokens of 64 heads of 128, bf16, out of a packed projection 42.5 us, 6.3 TB/s, 94 % of the
// measured copy rate; 64 tokens of 40 heads 2.4 us, a launch and two dependent
// reads.  The 16 elements are
// two pieces of eight: i.. and rot / 2 + i.. where halves pair, 16 adjacent
// ones otherwise, so accesses are of 16 bytes and pairs never leave a thread.  A warp's accesses lie side by
// side only in bf16 where whole rows' halves pair; elsewhere each is 16 bytes of 32, in fp32 16 of 64
// where 16 elements are adjacent.  L2 then has up to twice as many sectors to write for the same bytes,
// DRAM no more than the bytes.  8192 tokens of 64 heads of 128: bf16 interleaved 44 us, 48 of 128
// elements turned 43 (either way), fp32 85, interleaved 92.6 (87 % of the copy rate), 48 turned 90 to 92;
// of 64: bf16 25 (79 to 82 %), fp32 45, interleaved 50.  3003 tokens of 20 heads of 64 in fp32 (30 MB), where half a
// head turns 7.8 to 8.0 us, where all of it does in halves 6.6.
template <class T, int D, bool INTER>
__device__ __forceinline__ void rope_block(const RopeParams& p, int group, int h0, int heads) {
  constexpr int UNITS = D / 16;
  constexpr int BATCH = sizeof(T) == 2 ? 4 : 2;  // heads in flight
  const int unit = threadIdx.x % UNITS;
  const unsigned row = (unsigned)group * rope_tokens(D) + threadIdx.x / UNITS;  // below 2^31 + 64
  if (row >= (unsigned)p.B * (unsigned)p.N) return;
  const long long b = p.B == 1 ? 0 : row / (unsigned)p.N, n = row - b * p.N;
  const bool halves = !INTER && unit < p.rot / 16;
  const int at = halves ? 8 * unit : 16 * unit, to = halves ? p.rot / 2 + 8 * unit : 16 * unit + 8;
  const int end = min(h0 + heads, p.Hq + p.Hkv);
  // Queries' heads come before the keys'; both sides' pointers step from head to head.
  auto in = [&](int h) -> const T* {
    const bool is_q = h < p.Hq;
    const RopeRows& r = is_q ? p.q : p.k;
    return static_cast<const T*>(r.in) + b * r.in_batch + (is_q ? h : h - p.Hq) * r.in_head + n * r.in_token;
  };
  auto out = [&](int h) -> T* {
    const bool is_q = h < p.Hq;
    const RopeRows& r = is_q ? p.q : p.k;
    return static_cast<T*>(r.out) + b * r.out_batch + (is_q ? h : h - p.Hq) * r.out_head + n * r.out_token;
  };
  const T* src = in(h0);
  T* dst = out(h0);
  Eight<T> x[BATCH][2];
  auto read = [&](int h) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (h + k < end) {
        x[k][0].load(src + at);
        x[k][1].load(src + to);
        src = h + k + 1 == p.Hq ? in(p.Hq) : src + (h + k < p.Hq ? p.q.in_head : p.k.in_head);
      }
  };
  read(h0);  // (on their way while the angles are computed)
  const int pos = p.positions ? p.positions[b * p.pos_batch + n] : (int)n;
  // A token with a negative position has none: it is copied.
  const bool turns = unit < p.rot / 16 && pos >= 0;
  float c[8], s[8];
  if (turns) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      cos_sin(pos, p.freqs[8 * unit + k], c[k], s[k]);
      c[k] *= p.amplitude;
      s[k] *= p.sine;
    }
  }
  for (int h = h0; h < end; h += BATCH) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (h + k < end) {
        if (turns) {
          float u[8], v[8], y[8], z[8];
          x[k][0].get(u);
          x[k][1].get(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (INTER) {  // pair i is elements 2 i and 2 i + 1 of the sixteen
              const float x1 = i < 4 ? u[(2 * i) & 7] : v[(2 * i) & 7], x2 = i < 4 ? u[(2 * i + 1) & 7] : v[(2 * i + 1) & 7];
              const float y1 = fmaf(x1, c[i], -(x2 * s[i])), y2 = fmaf(x2, c[i], x1 * s[i]);
              (i < 4 ? y : z)[(2 * i) & 7] = y1;
              (i < 4 ? y : z)[(2 * i + 1) & 7] = y2;
            } else {
              y[i] = fmaf(u[i], c[i], -(v[i] * s[i]));
              z[i] = fmaf(v[i], c[i], u[i] * s[i]);
            }
          }
          x[k][0].set(y);
          x[k][1].set(z);
        }
        if (dcheck(h + k < p.Hq + p.Hkv && to + 8 <= D && n < p.N, p.status)) {
          x[k][0].store(dst + at);
          x[k][1].store(dst + to);
        }
        dst = h + k + 1 == p.Hq ? out(p.Hq) : dst + (h + k < p.Hq ? p.q.out_head : p.k.out_head);
      }
    read(h + BATCH);
  }
}

}  // namespace attn
