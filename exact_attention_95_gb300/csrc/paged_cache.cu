// paged_cache.cu -- a paged 8-bit key/value cache: the tables of a step built
// from the requests' lengths, and the append that quantizes new keys and
// values into their pages.  (paged_fwd.cu has the attention over the cache.)
//
// Cache: K and V pages of P tokens, [num_pages, Hkv, P, d] e4m3 codes with one
// fp32 scale for each (page, kv head).
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

// ------------------------------------------------------------------ tables
// Request r holds c_r tokens and is to take a_r more.  It needs
//   need_r = ceil((c_r + a_r) / P) - ceil(c_r / P)
// pages, handed out of the free list in request order: the inclusive prefix
// sum N_r of the needs says which.  Token t of the flattened new tokens
// belongs to the first request whose inclusive prefix sum of a_r exceeds t.
//
// Latency bound (a few KB in and out).  One launch: every CTA scans all
// requests itself, a block of `blockDim` at a time, both prefix sums in one
// pass, and then writes its share of the block's tokens and table entries,
// found by binary search in the block's sums in shared memory; a second
// launch, or a wait between CTAs, would cost more than the repeated scan.
// Measured, one step in a captured graph: 8 requests 2.3 us, 777 with up
// to 200 new tokens each 4.6 us, 64 prompts of up to 8192 tokens 3.4 us.
// Sums saturate at kCap (associative for non-negative terms), above every
// limit they are compared with.
constexpr unsigned kCap = 0x7fffffffu;
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kCap); }

constexpr int kTabThreads = 1024;

__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const KvTablesParams p) {
  __shared__ unsigned s_tok[kTabThreads], s_need[kTabThreads];  // inclusive sums
  __shared__ int s_cached[kTabThreads];
  __shared__ uint8_t s_served[kTabThreads];
  __shared__ unsigned w_tok[32], w_need[32];
  __shared__ unsigned s_taken, s_refused;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthr = blockDim.x, nwarp = nthr >> 5;
  const int P = 1 << p.page_log2;
  const unsigned T = (unsigned)p.T, F = (unsigned)p.n_free;
  if (tid == 0) s_taken = s_refused = 0;
  griddep_launch_dependents();
  griddep_wait();
  unsigned tok0 = 0, need0 = 0;  // sums over the blocks before this one
  for (int base = 0; base < p.R; base += nthr) {
    const int r = base + tid;
    int c = 0, a = 0;
    if (r < p.R) {
      c = max(p.cached[r], 0);
      a = max(p.added[r], 0);
    }
    const long long end = (long long)c + a;
    const int have = (int)(((long long)c + P - 1) >> p.page_log2);
    const long long full = (end + P - 1) >> p.page_log2;
    const bool wide = full <= p.max_pages;
    unsigned tok = min((unsigned)a, T + 1);
    unsigned need = r < p.R && wide ? (unsigned)(full - have) : 0u;
    const unsigned mine = need;
    // Inclusive sums over the block.
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, tok, o), y = __shfl_up_sync(0xffffffffu, need, o);
      if (lane >= o) {
        tok = sat_add(tok, x);
        need = sat_add(need, y);
      }
    }
    if (lane == 31) {
      w_tok[warp] = tok;
      w_need[warp] = need;
    }
    __syncthreads();
    if (warp == 0) {
      unsigned x = lane < nwarp ? w_tok[lane] : 0, y = lane < nwarp ? w_need[lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
          x = sat_add(x, u);
          y = sat_add(y, v);
        }
      }
      w_tok[lane] = x;
      w_need[lane] = y;
    }
    __syncthreads();
    tok = sat_add(sat_add(tok, tok0), warp ? w_tok[warp - 1] : 0u);
    need = sat_add(sat_add(need, need0), warp ? w_need[warp - 1] : 0u);
    const bool served = r < p.R && wide && tok <= T && (mine == 0 || need <= F);
    s_tok[tid] = tok;
    s_need[tid] = need;
    s_cached[tid] = c;
    s_served[tid] = served;
    if (r < p.R && (base / nthr) % gridDim.x == blockIdx.x) {
      p.kv_lens[r] = served ? (int)end : c;
      p.cu_tokens[r + 1] = (int)min(tok, T);
      if (r == 0) p.cu_tokens[0] = 0;
    }
    if (blockIdx.x == 0) {
      if (served && mine > 0) atomicMax(&s_taken, need);
      if (r < p.R && !served) atomicAdd(&s_refused, 1u);
    }
    __syncthreads();
    const int n = min(nthr, p.R - base);
    const unsigned tok1 = s_tok[n - 1], need1 = s_need[n - 1];
    // First entry of the block whose sum exceeds x.
    auto owner = [&](const unsigned* sums, unsigned x) {
      int lo = 0, hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] > x) hi = mid;
        else lo = mid + 1;
      }
      return lo;
    };
    const unsigned first = blockIdx.x * nthr + tid, step = gridDim.x * nthr;
    for (unsigned long long t = (unsigned long long)tok0 + first; t < min(tok1, T); t += step) {
      const int i = owner(s_tok, (unsigned)t);
      const unsigned start = i ? s_tok[i - 1] : tok0;
      long long slot = -1;
      int pos = -1;
      if (s_served[i]) {
        const int ci = s_cached[i];
        pos = ci + (int)((unsigned)t - start);
        const int pg = pos >> p.page_log2;
        const int held = (int)(((long long)ci + P - 1) >> p.page_log2);
        const unsigned f0 = i ? s_need[i - 1] : need0;
        if (!dcheck(base + i < p.R && pg < p.max_pages && (pg < held || f0 + (pg - held) < F), p.status)) continue;
        const int id = pg >= held ? p.free_pages[f0 + (pg - held)]
                                  : p.block_table[(size_t)(base + i) * p.max_pages + pg];
        slot = (long long)id * P + (pos & (P - 1));
      }
      if (!dcheck(t < T, p.status)) continue;
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
    for (unsigned long long x = (unsigned long long)need0 + first; x < min(need1, F); x += step) {
      const int i = owner(s_need, (unsigned)x);
      if (!s_served[i]) continue;
      const int held = (int)(((long long)s_cached[i] + P - 1) >> p.page_log2);
      const unsigned f0 = i ? s_need[i - 1] : need0;
      const unsigned col = held + ((unsigned)x - f0);
      if (!dcheck(base + i < p.R && col < (unsigned)p.max_pages && x < F, p.status)) continue;
      p.block_table[(size_t)(base + i) * p.max_pages + col] = p.free_pages[x];
    }
    tok0 = tok1;
    need0 = need1;
    __syncthreads();
  }
  // Places behind the last token.
  for (unsigned long long t = (unsigned long long)min(tok0, T) + blockIdx.x * nthr + tid; t < T; t += gridDim.x * nthr) {
    p.slots[t] = -1;
    p.positions[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.taken[0] = (int)s_taken;
    p.taken[1] = (int)s_refused;
  }
}

// ------------------------------------------------------------------ append
// The tokens of one page in the call form a run: consecutive tokens with
// consecutive slots.  For a run and a kv head, with off the first slot's
// offset in its page, x the new rows and s the page's scale:
//   want = the smallest 2^k (k >= -126) with max |x| <= 448 * 2^k (finite x),
//   s'   = off > 0 ? max(s, want) : want,
//   rows [0, off): code' = e4m3(code * s / s') where s' > s,
//   new rows:      code  = e4m3(x / s').
// A power of two keeps e4m3's relative precision for any max |x| (the format
// floats), and re-scaling then only shifts exponents: a code rounded again is
// one that becomes subnormal.
//
// HBM bound where there are many tokens: 2 bytes read and 1 written per
// element.  One read of the new rows: what holds a run's rows in registers is
// the D / 8 lanes of one row for up to kGroupRun tokens (a decoding step: four
// runs or two to a warp), the warp for up to kWarpRun, else the CTA.  A CTA
// looks at `chunk` tokens and `pairs` of the 2 * Hkv (K or V, head) pairs.
// Measured: 64 requests of one token, 8 kv heads, d = 128: 2.5 us, 500 requests,
// 16 kv heads, d = 64: 3.7 us (launch, then the slots, then rows and scales,
// which this code asks for behind the slots though a row's place does not depend
// on its slot, then the page where its scale grows); nine prompts of up to 4096 tokens 34 us, 4.5 TB/s, where the
// integer pipe is 54 % busy (maxima, packing) and each CTA's first reads are
// waited for.  Reading the next run while this one is written, prefetching the
// chunk's rows to L2 while its slots are read, and neighbouring CTAs for the
// heads of one chunk were no faster.
constexpr int kAppThreads = 256;
constexpr int kGroupRun = 4;
constexpr int kWarpRun = 16;
constexpr int kMaxPage = 128;
constexpr int kFewTokens = 1024;
constexpr int kMaxChunk = 64;

// want for the largest |x| given as bf16 bits (below the infinity's).
__device__ __forceinline__ float power_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 7);  // biased exponent
  int k = e - 127 - ((amax_bits & 0x7f) <= 0x60 ? 8 : 7);  // 448 = 1.75 * 2^8
  if (k < -126 || e == 0) k = -126;
  return __int_as_float((k + 127) << 23);
}
// Elementwise larger |x| of packed bf16 pairs, as bits.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
// The same without infinities and NaNs.
__device__ __forceinline__ uint32_t finite_max2(uint32_t m, uint32_t w) {
  uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  if (lo >= 0x7f80u) lo = 0;
  if (hi >= 0x7f80u) hi = 0;
  return __vmaxu2(m, lo | (hi << 16));
}
__device__ __forceinline__ uint32_t fold_max(uint32_t m) { return max(m & 0xffffu, m >> 16); }

// Eight bf16 -> eight codes, times inv.
__device__ __forceinline__ uint2 encode8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t i2 = f2pack(inv, inv);
  float x[8];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    f2unpack(fmul2(f2pack(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)), i2), x[2 * k], x[2 * k + 1]);
  return make_uint2(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]));
}
// The same by division, for a scale that is no power of two.
__device__ __noinline__ uint2 encode8_div(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __fdiv_rn(__uint_as_float(w[k] << 16), s);
    x[2 * k + 1] = __fdiv_rn(__uint_as_float(w[k] & 0xffff0000u), s);
  }
  return make_uint2(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]));
}
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

// Quantizes a run with `count` lanes (this one is `id`) that hold PER pieces
// of its rows each; fold(x) is the largest of their values x.
template <int D, int PER, class Fold>
__device__ __forceinline__ void append_run(const Run<D>& r, int id, int count, Fold fold) {
  constexpr int CH = D / 8;  // 16-byte pieces of a row
  uint4 v[PER];
  uint32_t m = 0;
  const float old = *r.scale;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int u = id + count * j, row = u / CH, col = u % CH;
    v[j] = make_uint4(0, 0, 0, 0);
    if (row < r.n) v[j] = __ldg(reinterpret_cast<const uint4*>(r.src + row * r.ld) + col);
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) m = abs_max2(abs_max2(abs_max2(abs_max2(m, v[j].x), v[j].y), v[j].z), v[j].w);
  uint32_t amax = fold(fold_max(m), 0);
  // An infinity or NaN among them: the largest of the others.
  m = 0;
  if (amax >= 0x7f80u) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      m = finite_max2(finite_max2(finite_max2(finite_max2(m, v[j].x), v[j].y), v[j].z), v[j].w);
  }
  amax = fold(fold_max(m), amax);
  const float want = power_scale(amax);
  const float s = r.off > 0 ? fmaxf(old, want) : want;
  const float inv = exact_inverse(s);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int u = id + count * j, row = u / CH, col = u % CH;
    if (row < r.n)
      *(reinterpret_cast<uint2*>(r.dst + (r.off + row) * D) + col) = inv > 0.f ? encode8(v[j], inv) : encode8_div(v[j], s);
  }
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

template <int D>
__global__ void __launch_bounds__(kAppThreads, 4) kv_append_kernel(const KvAppendParams p, int chunk, int pairs) {
  constexpr int CH = D / 8;                            // lanes of a row
  constexpr int WPER = kWarpRun * CH / 32;             // pieces a lane holds, run of a warp
  constexpr int CPER = kMaxPage * CH / kAppThreads;    // pieces a thread holds, run of the CTA
  constexpr int kWarps = kAppThreads / 32;
  __shared__ uint32_t s_cont[(kMaxChunk + kMaxPage) / 32 + 1];  // bit i: token i goes on with token i - 1's run
  __shared__ uint32_t s_lead[kMaxChunk / 32];                   // bit i: a run begins at token i
  __shared__ long long s_slot[kMaxChunk];                       // of each run: its first slot,
  __shared__ uint16_t s_first[kMaxChunk], s_len[kMaxChunk];     // first token, tokens
  __shared__ uint32_t s_red[kWarps];
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.page_log2;
  const long long t0 = (long long)blockIdx.x * chunk;
  const long long limit = (long long)p.num_pages << p.page_log2;
  const int pair0 = blockIdx.y * pairs, npairs = min(pairs, 2 * p.Hkv - pair0);
  // The chunk's slots and those a run of it may reach.
  const int span = (int)min((long long)(chunk + P), p.T - t0);
  const int words = (chunk + P + 31) / 32;
  long long slot = -1;  // of token t0 + tid (chunk <= kAppThreads)
  bool lead = false;
  for (int i = tid; i < words * 32; i += kAppThreads) {
    const long long s = i < span ? p.slots[t0 + i] : -1;
    const long long before = i < span && t0 + i > 0 ? p.slots[t0 + i - 1] : -1;
    const bool valid = s >= 0 && s < limit;
    const bool cont = valid && before >= 0 && s == before + 1 && (s & (P - 1)) != 0;
    const uint32_t cm = __ballot_sync(0xffffffffu, cont);
    const bool ld = valid && !cont && i < chunk;
    const uint32_t lm = __ballot_sync(0xffffffffu, ld);
    if (i == tid) {
      slot = s;
      lead = ld;
    }
    if (lane == 0) {
      s_cont[i >> 5] = cm;
      if (i < kMaxChunk) s_lead[i >> 5] = lm;
    }
  }
  if (tid == 0) s_cont[words] = 0;
  __syncthreads();
  int nruns = 0, len = 0;
  for (int wd = 0; wd < (chunk + 31) / 32; ++wd) nruns += __popc(s_lead[wd]);
  if (lead) {
    int k = __popc(s_lead[warp] & ((1u << lane) - 1));
    for (int wd = 0; wd < warp; ++wd) k += __popc(s_lead[wd]);
    // Tokens of the run: ones of s_cont behind its first.
    int j = tid + 1;
    len = 1;
    for (;;) {
      const int room = 32 - (j & 31);
      const uint32_t rest = ~(s_cont[j >> 5] >> (j & 31));  // bits shifted in from above end the run
      const int take = rest ? min(__ffs((int)rest) - 1, room) : room;
      len += take;
      if (take < room || (j >> 5) + 1 >= words) break;
      j += take;
    }
    s_slot[k] = slot;
    s_first[k] = (uint16_t)tid;
    s_len[k] = (uint16_t)len;
  }
  const bool any_group = __syncthreads_or(len > 0 && len <= kGroupRun);
  const bool any_warp = __syncthreads_or(len > kGroupRun && len <= kWarpRun);
  const bool any_cta = __syncthreads_or(len > kWarpRun);
  const int tasks = nruns * npairs;
  auto task_run = [&](int task, int lo, int hi) -> Run<D> {  // n = 0 unless lo < tokens <= hi
    const int k = min(task, tasks - 1) / npairs, pair = min(task, tasks - 1) - k * npairs;
    const int n = s_len[k];
    return run_of<D>(p, t0 + s_first[k], s_slot[k], task < tasks && n > lo && n <= hi ? n : 0, pair0 + pair);
  };
  // (No early start of the next kernel: its CTAs would crowd on the SMs that have
  // fewer of these.  Two appends of 2000 tokens in a row 9.7 us each, with it 13.5.)
  if (any_group) {
    constexpr int GROUPS = kAppThreads / CH;
    for (int base = 0; base < tasks; base += GROUPS) {
      const Run<D> r = task_run(base + tid / CH, 0, kGroupRun);
      append_run<D, kGroupRun>(r, tid % CH, CH, [&](uint32_t x, uint32_t keep) {
#pragma unroll
        for (int o = 1; o < CH; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        return keep && keep < 0x7f80u ? keep : x;
      });
    }
  }
  if (any_warp)
    for (int task = warp; task < tasks; task += kWarps) {
      const Run<D> r = task_run(task, kGroupRun, kWarpRun);
      if (r.n)
        append_run<D, WPER>(r, lane, 32, [&](uint32_t x, uint32_t keep) {
          return keep && keep < 0x7f80u ? keep : __reduce_max_sync(0xffffffffu, x);
        });
    }
  if (any_cta)
    for (int task = 0; task < tasks; ++task) {
      const Run<D> r = task_run(task, kWarpRun, kMaxPage);
      if (r.n)
        append_run<D, CPER>(r, tid, kAppThreads, [&](uint32_t x, uint32_t keep) {
          if (keep && keep < 0x7f80u) return keep;
          x = __reduce_max_sync(0xffffffffu, x);
          __syncthreads();  // the last use of s_red is over
          if (lane == 0) s_red[warp] = x;
          __syncthreads();
          return __reduce_max_sync(0xffffffffu, s_red[lane & (kWarps - 1)]);
        });
    }
}

// Launches a kernel that may start while the one before it in the stream ends
// (it waits for that one before it reads anything).
template <class... P, class... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesParams& p, int sms, cudaStream_t stream) {
  // Threads for the requests' scan in few blocks, and a CTA for every block of
  // tokens, up to 1024 threads an SM (64 prompts of up to 8192 tokens, CTAs of
  // 256 an SM: one 4.7 us, four 3.4, eight 4.4).
  const int thr = p.R <= 256 ? 256 : kTabThreads;
  const int most = sms * (kTabThreads / thr);
  const int grid = (int)std::max(1LL, std::min((long long)most, ((long long)p.T + thr - 1) / thr));
  return launch_behind(kv_tables_kernel, grid, thr, stream, p);
}

cudaError_t launch_kv_append(int d, const KvAppendParams& p, int sms, cudaStream_t stream) {
  // Up to kFewTokens tokens: eight, and as many pairs as give every group of
  // lanes a run of one token; more: 64 and two pairs.  Measured on both sides
  // of the border, 16 pairs, d = 128, us, the few tokens' way first: 500 tokens
  // of a prompt 6.0 / 4.2, of 500 requests (32 pairs, d = 64) 4.0 / 5.1; 2000
  // tokens 10.4 / 6.8 and 10.5 / 10.0.  128 tokens and one pair against 64 and
  // two: 25000 tokens of five prompts 32.9 / 32.3, 8000 requests 25.8 / 24.3.
  const int chunk = p.T <= kFewTokens ? 8 : kMaxChunk;
  const int pairs = p.T <= kFewTokens ? kAppThreads / (d / 8) / 8 : 2;
  const long long chunks = (p.T + chunk - 1) / chunk;
  const dim3 grid((unsigned)chunks, (unsigned)((2 * p.Hkv + pairs - 1) / pairs));
  return d == 128 ? launch_behind(kv_append_kernel<128>, grid, kAppThreads, stream, p, chunk, pairs)
                  : launch_behind(kv_append_kernel<64>, grid, kAppThreads, stream, p, chunk, pairs);
}

}  // namespace attn
