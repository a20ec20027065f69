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
        const int id = pg >= held ? p.free_pages[f0 + (pg - held)]
                                  : p.block_table[(size_t)(base + i) * p.max_pages + pg];
        slot = (long long)id * P + (pos & (P - 1));
      }
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
    for (unsigned long long x = (unsigned long long)need0 + first; x < min(need1, F); x += step) {
      const int i = owner(s_need, (unsigned)x);
      if (!s_served[i]) continue;
      const int held = (int)(((long long)s_cached[i] + P - 1) >> p.page_log2);
      const unsigned f0 = i ? s_need[i - 1] : need0;
      p.block_table[(size_t)(base + i) * p.max_pages + held + ((unsigned)x - f0)] = p.free_pages[x];
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
// HBM bound: 2 bytes read and 1 written per element.  One read of the new
// rows: a run of up to kWarpRun tokens is held in a warp's registers (8
// 16-byte loads a lane at d = 128), a longer one in the CTA's.
constexpr int kAppThreads = 256;
constexpr int kWarpRun = 16;
constexpr int kMaxPage = 128;
constexpr int kMaxChunk = 128;

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

// Eight bf16 -> eight codes at scale s (inv = 1 / s when s is a power of two, else 0).
__device__ __forceinline__ uint2 encode8(const uint4& v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = inv > 0.f ? x[k] * inv : __fdiv_rn(x[k], s);
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

template <int D>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const KvAppendParams p, int chunk) {
  constexpr int CH = D / 8;                            // 16-byte pieces of a row
  constexpr int WPER = kWarpRun * CH / 32;             // pieces a lane holds, run of a warp
  constexpr int CPER = kMaxPage * CH / kAppThreads;    // pieces a thread holds, run of the CTA
  __shared__ long long s_slot[kMaxChunk + kMaxPage];
  __shared__ uint32_t s_cont[(kMaxChunk + kMaxPage) / 32 + 1];  // bit i: token i goes on with token i - 1's run
  __shared__ uint32_t s_lead[kMaxChunk / 32];                   // bit i: a run begins at token i
  __shared__ uint32_t s_red[kAppThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const uint16_t* X = is_v ? p.V : p.K;
  const long long ld = is_v ? p.v_stride : p.k_stride;
  uint8_t* pages = is_v ? p.v_pages : p.k_pages;
  float* scales = is_v ? p.v_scale : p.k_scale;
  const int P = 1 << p.page_log2;
  const long long t0 = (long long)blockIdx.x * chunk;
  const long long limit = (long long)p.num_pages << p.page_log2;
  // The chunk's slots and those a run of it may reach.
  const int span = (int)min((long long)(chunk + P), p.T - t0);
  const int words = (chunk + P + 31) / 32;
  for (int i = tid; i < words * 32; i += kAppThreads) {
    const long long s = i < span ? p.slots[t0 + i] : -1;
    const long long before = i < span && t0 + i > 0 ? p.slots[t0 + i - 1] : -1;
    const bool valid = s >= 0 && s < limit;
    const bool cont = valid && before >= 0 && s == before + 1 && (s & (P - 1)) != 0;
    if (i < chunk + P) s_slot[i] = s;
    const uint32_t cm = __ballot_sync(0xffffffffu, cont);
    const uint32_t lm = __ballot_sync(0xffffffffu, valid && !cont && i < chunk);
    if (lane == 0) {
      s_cont[i >> 5] = cm;
      if (i < kMaxChunk) s_lead[i >> 5] = lm;
    }
  }
  if (tid == 0) s_cont[words] = 0;
  __syncthreads();
  // Tokens of the run that begins at i.
  auto run_len = [&](int i) {
    int n = 1, j = i + 1;
    for (;;) {
      const uint32_t rest = ~(s_cont[j >> 5] >> (j & 31));
      const int ones = __ffs((int)rest) - 1;  // bits shifted in from above read as the run's end
      const int room = 32 - (j & 31);
      const int take = ones < 0 ? room : min(ones, room);
      n += take;
      if (take < room || (j >> 5) + 1 >= words) return n;
      j += take;
    }
  };
  // Rows [0, off) of the page at the larger scale, by `count` threads.
  auto rescale = [&](uint8_t* dst, int off, float r, int id, int count) {
    for (int u = id; u < off * (D / 16); u += count) {
      uint4* q = reinterpret_cast<uint4*>(dst) + u;
      uint4 v = *q;
      v.x = rescale4(v.x, r);
      v.y = rescale4(v.y, r);
      v.z = rescale4(v.z, r);
      v.w = rescale4(v.w, r);
      *q = v;
    }
  };
  int k = 0;
  for (int wd = 0; wd < (chunk + 31) / 32; ++wd) {
    for (uint32_t lead = s_lead[wd]; lead; lead &= lead - 1) {
      const int i = wd * 32 + __ffs((int)lead) - 1;
      const int n = run_len(i);
      if (n > kWarpRun || (k++ & (kAppThreads / 32 - 1)) != warp) continue;
      const long long slot = s_slot[i];
      const long long page = slot >> p.page_log2;
      const int off = (int)(slot & (P - 1));
      float* sp = scales + page * p.Hkv + h;
      const float old = *sp;
      uint4 v[WPER];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < WPER; ++j) {
        const int u = lane + 32 * j, row = u / CH, col = u % CH;
        v[j] = make_uint4(0, 0, 0, 0);
        if (row < n) v[j] = __ldg(reinterpret_cast<const uint4*>(X + (t0 + i + row) * ld + (long long)h * D) + col);
        m = abs_max2(abs_max2(abs_max2(abs_max2(m, v[j].x), v[j].y), v[j].z), v[j].w);
      }
      uint32_t amax = __reduce_max_sync(0xffffffffu, fold_max(m));
      if (amax >= 0x7f80u) {
        m = 0;
#pragma unroll
        for (int j = 0; j < WPER; ++j)
          m = finite_max2(finite_max2(finite_max2(finite_max2(m, v[j].x), v[j].y), v[j].z), v[j].w);
        amax = __reduce_max_sync(0xffffffffu, fold_max(m));
      }
      const float want = power_scale(amax);
      const float s = off > 0 ? fmaxf(old, want) : want;
      const float inv = exact_inverse(s);
      uint8_t* dst = pages + ((page * p.Hkv + h) << p.page_log2) * D;
#pragma unroll
      for (int j = 0; j < WPER; ++j) {
        const int u = lane + 32 * j, row = u / CH, col = u % CH;
        if (row < n) *(reinterpret_cast<uint2*>(dst + (off + row) * D) + col) = encode8(v[j], s, inv);
      }
      if (off > 0 && s > old) rescale(dst, off, __fdiv_rn(old, s), lane, 32);
      __syncwarp();
      if (lane == 0) *sp = s;
    }
  }
  // Longer runs, by the whole CTA.
  for (int wd = 0; wd < (chunk + 31) / 32; ++wd) {
    for (uint32_t lead = s_lead[wd]; lead; lead &= lead - 1) {
      const int i = wd * 32 + __ffs((int)lead) - 1;
      const int n = run_len(i);
      if (n <= kWarpRun) continue;
      const long long slot = s_slot[i];
      const long long page = slot >> p.page_log2;
      const int off = (int)(slot & (P - 1));
      float* sp = scales + page * p.Hkv + h;
      const float old = *sp;
      uint4 v[CPER];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < CPER; ++j) {
        const int u = tid + kAppThreads * j, row = u / CH, col = u % CH;
        v[j] = make_uint4(0, 0, 0, 0);
        if (row < n) v[j] = __ldg(reinterpret_cast<const uint4*>(X + (t0 + i + row) * ld + (long long)h * D) + col);
        m = abs_max2(abs_max2(abs_max2(abs_max2(m, v[j].x), v[j].y), v[j].z), v[j].w);
      }
      auto block_max = [&](uint32_t x) {
        x = __reduce_max_sync(0xffffffffu, fold_max(x));
        __syncthreads();  // readers of the last use are done, and every thread has read *sp
        if (lane == 0) s_red[warp] = x;
        __syncthreads();
        return __reduce_max_sync(0xffffffffu, s_red[lane & (kAppThreads / 32 - 1)]);
      };
      uint32_t amax = block_max(m);
      if (amax >= 0x7f80u) {
        m = 0;
#pragma unroll
        for (int j = 0; j < CPER; ++j)
          m = finite_max2(finite_max2(finite_max2(finite_max2(m, v[j].x), v[j].y), v[j].z), v[j].w);
        amax = block_max(m);
      }
      const float want = power_scale(amax);
      const float s = off > 0 ? fmaxf(old, want) : want;
      const float inv = exact_inverse(s);
      uint8_t* dst = pages + ((page * p.Hkv + h) << p.page_log2) * D;
#pragma unroll
      for (int j = 0; j < CPER; ++j) {
        const int u = tid + kAppThreads * j, row = u / CH, col = u % CH;
        if (row < n) *(reinterpret_cast<uint2*>(dst + (off + row) * D) + col) = encode8(v[j], s, inv);
      }
      if (off > 0 && s > old) rescale(dst, off, __fdiv_rn(old, s), tid, kAppThreads);
      if (tid == 0) *sp = s;
    }
  }
}

}  // namespace

cudaError_t launch_kv_tables(const KvTablesParams& p, int sms, cudaStream_t stream) {
  // Enough threads for the requests' scan (a warp to the whole block), and a
  // CTA for every block of tokens, up to one per SM.
  const int thr = p.R <= 256 ? 256 : kTabThreads;
  const int grid = (int)std::max(1LL, std::min((long long)sms, ((long long)p.T + thr - 1) / thr));
  kv_tables_kernel<<<grid, thr, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_append(int d, const KvAppendParams& p, int sms, cudaStream_t stream) {
  // Tokens a CTA looks at: as many as leave four CTAs per SM, 8 (one a warp) to 128.
  int chunk = kMaxChunk;
  while (chunk > 8 && (p.T + chunk - 1) / chunk * p.Hkv * 2 < 4LL * sms) chunk /= 2;
  const dim3 grid((unsigned)((p.T + chunk - 1) / chunk), (unsigned)p.Hkv, 2);
  if (d == 128) kv_append_kernel<128><<<grid, kAppThreads, 0, stream>>>(p, chunk);
  else kv_append_kernel<64><<<grid, kAppThreads, 0, stream>>>(p, chunk);
  return cudaGetLastError();
}

}  // namespace attn
