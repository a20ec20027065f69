// paged_append_rope.cu -- the quantizing append to a paged 8-bit cache with rotary
// positions applied on the way, and the queries of the same tokens rotated beside
// (paged_cache.cu has the append's rules, rope.cuh the rotation's).
#include <algorithm>

#include "launch.cuh"
#include "paged_append.cuh"
#include "rope.cuh"

namespace attn {
namespace {

// Scale and codes are those of the rotated numbers, held in fp32 and rounded once
// (V's, which do not turn, are exact in it).  Infinities and NaNs turn as fp32
// arithmetic has it: the pair gets an infinity or a NaN.
//
// A thread has 16 elements of a row, its unit, as in rope_block(): pairs never
// leave it.  A run is held by the D / 16 threads of one row for up to kGroupRun tokens, by
// a warp for up to kWarpRun, else by the CTA, as in the append without
// positions, all by one copy of the code.
//
// Measured, 8 kv and 32 query heads, d = 128: 64 requests of one token 4.4 us where no page's scale
// grows, and with a page whose scale grows at its last row 17 us (64 tokens a page) or 30 (128), however many
// they are: finish_run() takes the rows before the new one in turns of this run's eight threads, each a
// trip to memory and back (without positions sixteen threads, 9 and 15 us of 2.7); 25157 tokens of nine
// prompts 103 us, 5.5 TB/s, 82 % of the measured copy rate (the append alone 33 us, the
// queries alone 65).  What holds it: the keys' angles (27 instructions an angle, 14 us) and the waits of
// a run's chain (slots, rows, largest element, codes) with three CTAs of 80 registers an
// SM; two CTAs 113 us, four 109, 512 threads of 64 registers 129 (spilling).  Angles of a CTA's
// tokens in shared memory, read by four heads, took fewer instructions and 112 us: the table leaves
// two CTAs an SM.
constexpr int kPer = 4;  // rows of a thread

// want for the largest finite |x|, given as fp32 bits.
__device__ __forceinline__ float power_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);
  int k = e - 127 - ((amax_bits & 0x7fffff) <= 0x600000 ? 8 : 7);  // 448 = 1.75 * 2^8
  if (k < -126 || e == 0) k = -126;
  return __int_as_float((k + 127) << 23);
}
__device__ __noinline__ uint2 encode8_div(float4 a, float4 b, float s) {
  return make_uint2(pack_e4m3x4(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s), __fdiv_rn(a.z, s), __fdiv_rn(a.w, s)),
                    pack_e4m3x4(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s), __fdiv_rn(b.z, s), __fdiv_rn(b.w, s)));
}
__device__ __forceinline__ uint2 encode8(const float* y, float inv, float s) {
  if (inv > 0.f) {
    float q[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) f2unpack(fmul2(f2pack(y[2 * k], y[2 * k + 1]), f2pack(inv, inv)), q[2 * k], q[2 * k + 1]);
    return make_uint2(pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7]));
  }
  return encode8_div(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7]), s);
}

// What a thread reads of a run: kPer rows of its unit, their positions, the scale.
struct Held {
  Eight<uint16_t> a[kPer], b[kPer];
  int pos[kPer];  // -1: not rotated
  float old;
};

template <int D, bool INTER>
struct Unit {
  const uint64_t* freqs;  // of this unit's eight pairs, in shared memory
  float amplitude;
  int at, to;             // first elements of its two pieces of eight
  bool turns;
  __device__ __forceinline__ Unit(const RopeParams& q, const uint64_t* shared, int unit) {
    turns = unit < q.rot / 16;
    const bool halves = !INTER && turns;
    at = halves ? 8 * unit : 16 * unit;
    to = halves ? q.rot / 2 + 8 * unit : 16 * unit + 8;
    freqs = shared + 8 * unit;
    amplitude = q.amplitude;
  }
  // Reads rows row0, row0 + step, .. of a run.
  __device__ __forceinline__ void read(const Run<D>& r, const int* pos, int row0, int step, Held& x) const {
    x.old = *r.scale;
    const uint16_t* src = r.src + row0 * r.ld;
    const long long far = step * r.ld;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int row = row0 + step * j;
      x.a[j].v = x.b[j].v = make_uint4(0, 0, 0, 0);
      x.pos[j] = -1;
      if (row < r.n) {
        x.a[j].v = __ldg(reinterpret_cast<const uint4*>(src + at));
        x.b[j].v = __ldg(reinterpret_cast<const uint4*>(src + to));
        if (pos && turns) x.pos[j] = __ldg(pos + row);
      }
      src += far;
    }
  }
  // Rotates and quantizes what was read; fold(v, keep) is the largest v of the run's threads
  // (keep, where that is a finite number above zero), id and count this thread's place among them.
  template <class Fold>
  __device__ __forceinline__ void write(const Run<D>& r, int row0, int step, int id, int count, const Held& x, Fold fold) const {
    float y[kPer][16];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      float u[8], v[8];
      x.a[j].get(u);
      x.b[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[j][i] = u[i];
        y[j][8 + i] = v[i];
      }
      if (x.pos[j] >= 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float c, s;
          cos_sin(x.pos[j], freqs[k], c, s);
          c *= amplitude;
          s *= amplitude;
          float &x1 = y[j][INTER ? 2 * k : k], &x2 = y[j][INTER ? 2 * k + 1 : 8 + k];
          const float y1 = fmaf(x1, c, -(x2 * s)), y2 = fmaf(x2, c, x1 * s);
          x1 = y1;
          x2 = y2;
        }
      }
    }
    float m = 0.f;  // (a maximum with a NaN is the other number)
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(y[j][i]));
    uint32_t amax = fold(__float_as_uint(m), 0);
    m = 0.f;
    if (amax >= 0x7f800000u) {  // an infinity among them: the largest of the others
#pragma unroll
      for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (fabsf(y[j][i]) < INFINITY) m = fmaxf(m, fabsf(y[j][i]));
    }
    amax = fold(__float_as_uint(m), amax);
    const float want = power_scale(amax);
    const float s = r.off > 0 ? fmaxf(x.old, want) : want;
    const float inv = exact_inverse(s);
    uint8_t* dst = r.dst + (r.off + row0) * D;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (row0 + step * j < r.n) {
        *reinterpret_cast<uint2*>(dst + at) = encode8(&y[j][0], inv, s);
        *reinterpret_cast<uint2*>(dst + to) = encode8(&y[j][8], inv, s);
      }
      dst += step * D;
    }
    finish_run<D>(r, id, count, x.old, s);
  }
};

// A CTA's part of the append: tokens [bx * chunk, ..), pairs [by * pairs, ..).
template <int D, bool INTER>
__device__ __forceinline__ void append_chunk(const KvAppendParams& p, const RopeParams& q, int chunk, int pairs, int bx, int by) {
  constexpr int UNITS = D / 16;
  static_assert(kGroupRun <= kPer && kWarpRun * UNITS <= 32 * kPer && kMaxPage * UNITS <= kAppThreads * kPer, "rows of a thread");
  constexpr int kWarps = kAppThreads / 32;
  __shared__ RunTable runs;
  __shared__ uint32_t s_red[kWarps];
  __shared__ uint64_t s_freqs[D / 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long t0 = (long long)bx * chunk;
  const int pair0 = by * pairs, npairs = min(pairs, 2 * p.Hkv - pair0);
  if (tid < q.rot / 2) s_freqs[tid] = q.freqs[tid];
  bool any_group, any_warp, any_cta;
  const int nruns = find_runs(p, chunk, bx, runs, any_group, any_warp, any_cta);
  const int tasks = nruns * npairs;
  const Unit<D, INTER> unit(q, s_freqs, tid % UNITS);
  auto task_run = [&](int task, int lo, int hi, const int*& pos) -> Run<D> {  // n = 0 unless lo < tokens <= hi
    const int k = min(task, tasks - 1) / npairs, pair = min(task, tasks - 1) - k * npairs;
    const int n = runs.len[k];
    pos = pair0 + pair < p.Hkv ? q.positions + t0 + runs.first[k] : nullptr;
    return run_of<D>(p, t0 + runs.first[k], runs.slot[k], task < tasks && n > lo && n <= hi ? n : 0, pair0 + pair);
  };
  // Short, middling and long runs, one after the other in the same code (three copies of
  // it are fetched for longer than a decoding step takes): held by UNITS threads, a
  // warp or the CTA.
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    if (!(kind == 0 ? any_group : kind == 1 ? any_warp : any_cta)) continue;
    const int lo = kind == 0 ? 0 : kind == 1 ? kGroupRun : kWarpRun;
    const int hi = kind == 0 ? kGroupRun : kind == 1 ? kWarpRun : kMaxPage;
    const int count = kind == 0 ? UNITS : kind == 1 ? 32 : kAppThreads;  // threads of a run
    const int id = tid & (count - 1), row0 = id / UNITS, step = count / UNITS;
#pragma unroll 1
    for (int base = 0; base < tasks; base += kAppThreads / count) {
      const int* pos;  // of K's rows
      const Run<D> r = task_run(base + tid / count, lo, hi, pos);
      if (kind == 2 ? r.n == 0 : __all_sync(0xffffffffu, r.n == 0)) continue;  // (the whole warp or CTA)
      Held x;
      unit.read(r, pos, row0, step, x);
      unit.write(r, row0, step, id, count, x, [&](uint32_t v, uint32_t keep) {
        // A kind's threads all come here, with the same `keep` in a run.
        uint32_t most = v;
        if (kind == 0) {
#pragma unroll
          for (int o = 1; o < UNITS; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        } else if (!(keep && keep < 0x7f800000u)) {
          most = __reduce_max_sync(0xffffffffu, v);
          if (kind == 2) {
            __syncthreads();  // the last use of s_red is over
            if (lane == 0) s_red[warp] = most;
            __syncthreads();
            most = __reduce_max_sync(0xffffffffu, s_red[lane & (kWarps - 1)]);
          }
        }
        return keep && keep < 0x7f800000u ? keep : most;
      });
    }
  }
}

// `appends` CTAs append, the others rotate the queries; the two kinds are spread evenly
// over the grid, as the one is held by its arithmetic and the other by memory.
struct Grid {
  int chunk, pairs, chunks;  // of an append: tokens and pairs of a CTA, CTAs along the tokens
  int q_groups, q_heads;     // of the queries: CTAs along the tokens, heads of a CTA
  int appends;
};
template <int D, bool INTER>
__global__ void __launch_bounds__(kAppThreads, 3)
    kv_append_rope_kernel(const KvAppendParams p, const RopeParams q, const Grid g) {
  static_assert(kAppThreads == kRopeThreads, "one block size for both kinds of CTA");
  griddep_wait();
  const int i = (int)((uint64_t)blockIdx.x * g.appends / gridDim.x);  // appends among the CTAs before this one
  if (i == (int)((uint64_t)(blockIdx.x + 1) * g.appends / gridDim.x)) {
    const int k = blockIdx.x - i;
    rope_block<uint16_t, D, INTER>(q, k % g.q_groups, k / g.q_groups * g.q_heads, g.q_heads);
  } else {
    append_chunk<D, INTER>(p, q, g.chunk, g.pairs, i % g.chunks, i / g.chunks);
  }
}

template <int D, bool INTER>
cudaError_t launch(const KvAppendParams& p, const RopeParams& q, int sms, cudaStream_t stream) {
  const bool few = p.T <= kFewTokens;
  const long long q_groups = (p.T + rope_tokens(D) - 1) / rope_tokens(D);
  Grid g;
  g.chunk = few ? 8 : kMaxChunk;
  g.pairs = few ? kAppThreads / (D / 16) / 8 : 2;
  g.q_heads = rope_heads(q_groups, q.Hq, 8LL * sms);
  const long long chunks = (p.T + g.chunk - 1) / g.chunk, appends = chunks * ((2 * p.Hkv + g.pairs - 1) / g.pairs);
  const long long all = appends + q_groups * ((q.Hq + g.q_heads - 1) / g.q_heads);
  if (all >= 0x7fffffffLL) return cudaErrorNotSupported;
  g.chunks = (int)chunks;
  g.q_groups = (int)q_groups;
  g.appends = (int)appends;
  return launch_behind(kv_append_rope_kernel<D, INTER>, dim3((unsigned)all), kAppThreads, stream, 0, p, q, g);
}

}  // namespace

cudaError_t launch_kv_append_rope(int d, const KvAppendParams& p, const RopeParams& q, int interleaved, int sms,
                                  cudaStream_t stream) {
  if (d == 128) return interleaved ? launch<128, true>(p, q, sms, stream) : launch<128, false>(p, q, sms, stream);
  return interleaved ? launch<64, true>(p, q, sms, stream) : launch<64, false>(p, q, sms, stream);
}

}  // namespace attn
