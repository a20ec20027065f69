// paged_append.cuh -- what the two appends to a paged 8-bit cache share: how the
// tokens of a chunk fall into runs, a run's place, and its scale.
#pragma once

#include "kernels.h"
#include "ptx.cuh"

namespace attn {

constexpr int kAppThreads = 256;
constexpr int kGroupRun = 4;
constexpr int kWarpRun = 16;
constexpr int kMaxPage = 128;
constexpr int kFewTokens = 1024;
constexpr int kMaxChunk = 64;

// 1 / s for a power of two in [2^-126, 2^126], else 0.
__device__ __forceinline__ float exact_inverse(float s) {
  const uint32_t b = __float_as_uint(s);
  return (b & 0x807fffffu) == 0 && b >= 0x00800000u && b <= 0x7e800000u ? __uint_as_float(0x7f000000u - b) : 0.f;
}
// Sixteen codes times r, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float r) {
  float x[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(c >> (16 * k))));
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(x[2 * k]), "=f"(x[2 * k + 1])
        : "r"(h));
  }
  return pack_e4m3x4(x[0] * r, x[1] * r, x[2] * r, x[3] * r);
}

// A (run, pair)'s rows: where they come from and go to.
template <int D>
struct Run {
  const uint16_t* src;  // the first row's element 0
  long long ld;
  uint8_t* dst;  // the page's row 0
  float* scale;
  int off, n;
};
template <int D>
__device__ __forceinline__ Run<D> run_of(const KvAppendParams& p, long long t, long long slot, int n, int pair) {
  const bool is_v = pair >= p.Hkv;
  const int h = is_v ? pair - p.Hkv : pair;
  const long long place = (slot >> p.page_log2) * p.Hkv + h;
  Run<D> r;
  r.ld = is_v ? p.v_stride : p.k_stride;
  r.src = (is_v ? p.V : p.K) + t * r.ld + h * D;
  r.dst = (is_v ? p.v_pages : p.k_pages) + (place << p.page_log2) * D;
  r.scale = (is_v ? p.v_scale : p.k_scale) + place;
  r.off = (int)(slot & ((1 << p.page_log2) - 1));
  // The rows [t, t + n) and [off, off + n) are within the call's tokens and the page.
  r.n = n == 0 || dcheck(pair < 2 * p.Hkv && t >= 0 && t + n <= p.T && slot >= 0 && (slot >> p.page_log2) < p.num_pages &&
                             r.off + n <= 1 << p.page_log2,
                         p.status)
            ? n
            : 0;
  return r;
}

// The end of a run: rows [0, off) at the new scale s where it is larger, and the scale.  (By the run's
// threads, 16 bytes each at a time: for a run of few threads a chain of up to 127 reads and writes.)
template <int D>
__device__ __forceinline__ void finish_run(const Run<D>& r, int id, int count, float old, float s) {
  if (r.n > 0 && r.off > 0 && s > old) {
    // Rows [0, off) at the larger scale.
    const float ratio = __fdiv_rn(old, s);
    for (int u = id; u < r.off * (D / 16); u += count) {
      uint4* q = reinterpret_cast<uint4*>(r.dst) + u;
      uint4 c = *q;
      c.x = rescale4(c.x, ratio);
      c.y = rescale4(c.y, ratio);
      c.z = rescale4(c.z, ratio);
      c.w = rescale4(c.w, ratio);
      *q = c;
    }
  }
  // Every lane's read of the scale comes before this: of a warp's by the barrier, of a
  // CTA's by those of fold() (a shuffle or a vote orders no memory).
  __syncwarp();
  if (id == 0 && r.n > 0) *r.scale = s;
}

// The runs that begin in a chunk of tokens.
struct RunTable {
  uint32_t cont[(kMaxChunk + kMaxPage) / 32 + 1];  // bit i: token i goes on with token i - 1's run
  uint32_t lead[kMaxChunk / 32];                   // bit i: a run begins at token i
  long long slot[kMaxChunk];                       // of each run: its first slot,
  uint16_t first[kMaxChunk], len[kMaxChunk];       // first token, tokens
};
// Fills `s` for tokens [bx * chunk, ..); returns how many runs there are, and whether some
// have up to kGroupRun tokens, up to kWarpRun, or more.  For a CTA of kAppThreads.
__device__ __forceinline__ int find_runs(const KvAppendParams& p, int chunk, int bx, RunTable& s, bool& any_group,
                                         bool& any_warp, bool& any_cta) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.page_log2;
  const long long t0 = (long long)bx * chunk;
  const long long limit = (long long)p.num_pages << p.page_log2;
  // The chunk's slots and those a run of it may reach.
  const int span = (int)min((long long)(chunk + P), p.T - t0);
  const int words = (chunk + P + 31) / 32;
  long long slot = -1;  // of token t0 + tid (chunk <= kAppThreads)
  bool lead = false;
  for (int i = tid; i < words * 32; i += kAppThreads) {
    const long long at = i < span ? p.slots[t0 + i] : -1;
    const long long before = i < span && t0 + i > 0 ? p.slots[t0 + i - 1] : -1;
    const bool valid = at >= 0 && at < limit;
    const bool cont = valid && before >= 0 && at == before + 1 && (at & (P - 1)) != 0;
    const uint32_t cm = __ballot_sync(0xffffffffu, cont);
    const bool ld = valid && !cont && i < chunk;
    const uint32_t lm = __ballot_sync(0xffffffffu, ld);
    if (i == tid) {
      slot = at;
      lead = ld;
    }
    if (lane == 0) {
      s.cont[i >> 5] = cm;
      if (i < kMaxChunk) s.lead[i >> 5] = lm;
    }
  }
  if (tid == 0) s.cont[words] = 0;
  __syncthreads();
  int nruns = 0, len = 0;
  for (int wd = 0; wd < (chunk + 31) / 32; ++wd) nruns += __popc(s.lead[wd]);
  if (lead) {
    int k = __popc(s.lead[warp] & ((1u << lane) - 1));
    for (int wd = 0; wd < warp; ++wd) k += __popc(s.lead[wd]);
    // Tokens of the run: ones of s.cont behind its first.
    int j = tid + 1;
    len = 1;
    for (;;) {
      const int room = 32 - (j & 31);
      const uint32_t rest = ~(s.cont[j >> 5] >> (j & 31));  // bits shifted in from above end the run
      const int take = rest ? min(__ffs((int)rest) - 1, room) : room;
      len += take;
      if (take < room || (j >> 5) + 1 >= words) break;
      j += take;
    }
    s.slot[k] = slot;
    s.first[k] = (uint16_t)tid;
    s.len[k] = (uint16_t)len;
  }
  any_group = __syncthreads_or(len > 0 && len <= kGroupRun);
  any_warp = __syncthreads_or(len > kGroupRun && len <= kWarpRun);
  any_cta = __syncthreads_or(len > kWarpRun);
  return nruns;
}

}  // namespace attn
