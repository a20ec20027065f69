// paged_fwd.cu -- attention over a paged 8-bit key/value cache, for ragged
// batches of requests with few query rows per kv head (decoding).
//
//   s_ij = scale * ks(j) * <q_i, Kc_j>,  O_i = sum_j softmax_j(s_i) vs(j) Vc_j
//
// with Kc, Vc the e4m3 codes and ks(j), vs(j) the scales of key j's page.
//
// HBM bound: two bytes per key, kv head and column against 4 * G products.
// All products run in f16 with fp32 sums: an e4m3 code is an f16 number
// exactly, and so is a bf16 query times a power of two of its row (elements
// below 2^-29 of the row's largest lose bits).  The weights are rounded to
// f16, relative to the largest V scale seen, times 2^14: 2^-11 relative for
// every weight down to 2^-28 of the row's largest, which a long tail behind
// one dominant key needs (an 8-bit weight, even as a sum of two, would lose
// it).  mma.sync m16n8k16 rather than tcgen05: a 16-row tile of queries
// against codes that have to be widened in registers anyway leaves the tensor
// pipe mostly idle at HBM speed, and no accumulator leaves the registers.
//
// Work: a tile of 16 query rows (token-major, the G heads of a kv head of one
// token side by side) against the keys of its request, 128 keys to a unit.
// The units of all (request, kv head, row tile) items, in one line, are cut
// into equal ranges, one per CTA; an item cut between CTAs leaves partial
// (m, l, O) in the workspace for the merge kernel.  Every CTA finds its range
// from the lengths on the device; nothing is planned on the host.
//
// A CTA: eight warps that each take 16 keys of a unit, with their own running
// maximum, sum and accumulators, merged at the item's end; one producer warp
// that walks the block table and loads whole (page, head) boxes by TMA.
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kRows = 16;          // query rows of a tile
constexpr int kUnit = 128;         // keys of a unit
constexpr int kWarps = 8;          // consumer warps, 16 keys of a unit each
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxGroups = 512;    // 32 requests each
constexpr float kPScale = 16384.f;

// What a stage holds, written by the producer.
struct StageMeta {
  int flags;      // kBegin, kEnd, kStop
  int key0;       // first key
  int len;        // keys of the request
  int start, n;   // the request's query rows: tokens [start, start + n)
  int tile, h;    // row tile, kv head
  int slot;       // where the item's result goes: -1 output, else partial slot of this worker
  float ks[8], vs[8];  // scales of the unit's pages
  int pages;      // bit i: page i of the unit was loaded
  int pad[3];
};
enum : int { kBegin = 1, kEnd = 2, kStop = 4 };

template <int D>
struct PC {
  static constexpr int STAGES = D == 128 ? 4 : 8;
  static constexpr int KBYTES = kUnit * D;
  static constexpr int SBYTES = 2 * KBYTES;
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_O = STAGES * SBYTES;                   // [warps][16][D] fp32
  static constexpr int OFF_ML = OFF_O + kWarps * kRows * D * 4;   // [warps][16][2] fp32
  static constexpr int OFF_META = OFF_ML + kWarps * kRows * 8;
  static constexpr int OFF_SUMS = OFF_META + STAGES * (int)sizeof(StageMeta);  // [kMaxGroups] int64
  static constexpr int OFF_BAR = OFF_SUMS + kMaxGroups * 8;
  static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_WRITTEN = 2 * STAGES, B_READ = 2 * STAGES + 1;
  static constexpr int OFF_ABORT = OFF_BAR + (2 * STAGES + 2) * 8;
  static constexpr int SMEM = OFF_ABORT + 8 + 1024;
};
static_assert(PC<128>::SMEM <= 232448 && PC<64>::SMEM <= 232448, "shared memory");

__device__ __forceinline__ uint32_t widen(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// The request's query rows and keys, clipped to the arrays.
struct Req {
  int start, n, len;
  long long units;
};
__device__ __forceinline__ Req load_req(const PagedFwdParams& p, int r) {
  Req q{0, 0, 0, 0};
  if (r < p.R) {
    const int a = min(max(p.cu_q[r], 0), p.T), b = min(max(p.cu_q[r + 1], 0), p.T);
    q.start = a;
    q.n = max(b - a, 0);
    q.len = max(p.kv_lens[r], 0);
    const long long room = (long long)p.max_pages << p.page_log2;
    if (q.len > room) {
      q.len = (int)room;
      atomicCAS(p.status, kDevOk, kDevBounds);
    }
    const long long tiles = ((long long)q.n * p.G + kRows - 1) / kRows;
    q.units = tiles * p.Hkv * max(1, (q.len + kUnit - 1) / kUnit);
  }
  return q;
}

// Key index within eight that column n of a product stands for.  The order is
// free; these make the 16-byte (8-byte) shared-memory reads of a swizzled
// page free of bank conflicts.
template <int D>
__device__ __forceinline__ int key_of(int n) {
  return D == 128 ? (n >> 1) | ((n & 1) << 2) : n ^ ((n >> 1) & 1);
}
// Address of 16-byte piece `c` of row `row` in a swizzled page tile.
template <int D>
__device__ __forceinline__ uint32_t piece(uint32_t base, int row, int c) {
  return D == 128 ? base + row * 128 + ((c ^ (row & 7)) << 4) : base + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PagedFwdParams p) {
  using C = PC<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  StageMeta* metas = reinterpret_cast<StageMeta*>(smem + C::OFF_META);
  long long* sums = reinterpret_cast<long long*>(smem + C::OFF_SUMS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar(C::B_FULL + s), 1);
      mbar_init(bar(C::B_EMPTY + s), kWarps);
    }
    mbar_init(bar(C::B_WRITTEN), kWarps);
    mbar_init(bar(C::B_READ), kWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Units of every 32 requests.
  const int groups = (p.R + 31) >> 5;
  for (int g = warp; g < groups; g += kWarps + 1) {
    long long u = load_req(p, g * 32 + lane).units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    if (lane == 0) sums[g] = u;
  }
  __syncthreads();
  const WaitCtx wc{abort_flag, p.status, p.wait_limit_ns};

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    long long total = 0;
    for (int g = lane; g < groups; g += 32) total += sums[g];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const long long per = (total + gridDim.x - 1) / gridDim.x;
    const long long begin = min(total, per * blockIdx.x);
    const long long end = min(total, begin + per);
    int merge_parts = 0, merge_start = 0, merge_n = 0, merge_tile = 0, merge_h = 0;
    const int npg = kUnit >> p.page_log2;  // pages of a unit
    int it = 0;                            // stages filled
    bool ok = true;
    // Take a stage: returns its index once the consumers have left it.
    auto take = [&]() -> int {
      const int s = it % C::STAGES;
      if (it >= C::STAGES) ok = mbar_wait_warp(bar(C::B_EMPTY + s), ((it / C::STAGES) & 1) ^ 1, wc);
      return s;
    };
    if (begin < end) {
      // The group, then the request, that holds unit `begin`.
      long long before = 0;
      int g = 0;
      while (g + 1 < groups && before + sums[g] <= begin) before += sums[g++];
      Req rq = load_req(p, g * 32 + lane);
      long long incl = rq.units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      incl += before;
      int l = __ffs(__ballot_sync(0xffffffffu, incl > begin)) - 1;
      long long off = begin - (__shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, rq.units, l));
      long long pos = begin;
      while (pos < end && ok) {
        const int r = g * 32 + l;
        const int start = __shfl_sync(0xffffffffu, rq.start, l), n = __shfl_sync(0xffffffffu, rq.n, l);
        const int len = __shfl_sync(0xffffffffu, rq.len, l);
        const long long units = __shfl_sync(0xffffffffu, rq.units, l);
        const int kt = max(1, (len + kUnit - 1) / kUnit);
        const int tiles = (int)(((long long)n * p.G + kRows - 1) / kRows);
        const int* row = p.block_table + (size_t)r * p.max_pages;
        long long item = off / kt;
        int k0 = (int)(off - item * kt);
        for (; off < units && pos < end && ok; ++item) {
          const int h = (int)(item / tiles), tile = (int)(item - (long long)h * tiles);
          const int k1 = (int)min((long long)kt, k0 + (end - pos));
          const int slot = k0 == 0 && k1 == kt ? -1 : k0 == 0 ? 1 : 0;
          if (slot == 1) {
            const long long last = pos + kt - 1;  // the item's last unit
            merge_parts = (int)(last / per - blockIdx.x) + 1;
            merge_start = start;
            merge_n = n;
            merge_tile = tile;
            merge_h = h;
          }
          // Keys that some row of the tile may see.
          int seen = len;
          if (p.causal) {
            const int last_tok = (min(n * (long long)p.G, (long long)(tile + 1) * kRows) - 1) / p.G;
            seen = max(0, min(len, len - n + last_tok + 1));
          }
          const int ke = min(k1, max(k0 + 1, (seen + kUnit - 1) / kUnit));
          int id = -1;
          float ks = 0.f, vs = 0.f;
          for (int k = k0; k < ke; ++k) {
            // Page ids and scales, 32 pages at a time (lane i: page i of the batch).
            const int in_batch = ((k - k0) * npg) & 31;
            if (in_batch == 0) {
              const int pg = k * npg + lane;
              id = -1;
              if (((long long)pg << p.page_log2) < seen) {
                id = row[pg];
                if (id < 0 || id >= p.num_pages) {
                  id = -1;
                  atomicCAS(p.status, kDevOk, kDevBounds);
                } else {
                  ks = p.k_scale[(size_t)id * p.Hkv + h];
                  vs = p.v_scale[(size_t)id * p.Hkv + h];
                }
              }
            }
            const int s = take();
            if (!ok) break;
            StageMeta* m = metas + s;
            const int my = __shfl_sync(0xffffffffu, id, in_batch + (lane & 7));
            const float mk = __shfl_sync(0xffffffffu, ks, in_batch + (lane & 7));
            const float mv = __shfl_sync(0xffffffffu, vs, in_batch + (lane & 7));
            const bool load = lane < npg && my >= 0;
            const uint32_t mask = __ballot_sync(0xffffffffu, load);
            if (lane < 8) {
              m->ks[lane] = mk;
              m->vs[lane] = mv;
            }
            if (lane == 0) {
              m->flags = (k == k0 ? kBegin : 0) | (k + 1 == ke ? kEnd : 0);
              m->key0 = k * kUnit;
              m->len = len;
              m->start = start;
              m->n = n;
              m->tile = tile;
              m->h = h;
              m->slot = slot;
              m->pages = (int)mask;
            }
            __syncwarp();
            const uint32_t page_bytes = (uint32_t)D << p.page_log2;
            if (lane == 0) mbar_arrive_expect_tx(bar(C::B_FULL + s), 2 * page_bytes * __popc(mask));
            __syncwarp();
            if (load) {
              const uint32_t dst = sb + C::OFF_RING + s * C::SBYTES + lane * page_bytes;
              const long long plane = (long long)my * p.Hkv + h;
              tma_load_3d(dst, &tmK, bar(C::B_FULL + s), 0, 0, (int)plane);
              tma_load_3d(dst + C::KBYTES, &tmV, bar(C::B_FULL + s), 0, 0, (int)plane);
            }
            ++it;
          }
          pos += k1 - k0;
          off += k1 - k0;
          k0 = 0;
        }
        // The next request that has units.
        if (pos < end && ok) {
          off = 0;
          uint32_t more = __ballot_sync(0xffffffffu, rq.units > 0) & ~(0xffffffffu >> (31 - l));
          while (!more && g + 1 < groups) {
            ++g;
            rq = load_req(p, g * 32 + lane);
            more = __ballot_sync(0xffffffffu, rq.units > 0);
          }
          if (!more) break;
          l = __ffs(more) - 1;
        }
      }
    }
    if (lane == 0) {
      int* d = p.desc + blockIdx.x * 8;
      d[0] = merge_parts;
      d[1] = merge_start;
      d[2] = merge_n;
      d[3] = merge_tile;
      d[4] = merge_h;
    }
    if (ok) {
      const int s = take();
      if (ok) {
        if (lane == 0) {
          metas[s].flags = kStop;
          mbar_arrive(bar(C::B_FULL + s));
        }
      }
    }
    // Copies in flight land before the CTA leaves (the consumers have waited
    // for all of them unless a wait gave up).
    if (!ok)
      for (int k = max(0, it - C::STAGES); k < it; ++k)
        mbar_wait_drain_warp(bar(C::B_FULL + k % C::STAGES), (k / C::STAGES) & 1, wc);
    griddep_launch_dependents();
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  const int ko = key_of<D>(g);                       // this lane's key as a column
  const int kv0 = key_of<D>(2 * c), kv1 = key_of<D>(2 * c + 1);  // its keys as rows of V
  const int cg = D == 128 ? (g >> 1) | ((g & 1) << 2) : g >> 1;  // its 16-byte piece of a V row
  constexpr int QI = D / 64;   // 64-column parts of the contraction over d
  constexpr int NT = D / 8;    // 8-column tiles of O
  uint32_t qa[QI][4][4];
  float o[NT][4];
  float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f, f0 = 0.f, f1 = 0.f, vref = 0.f;
  int lim0 = 0, lim1 = 0, lim_all = 0, lim_any = 0;
  int ends = 0;  // items finished
  for (int it = 0;; ++it) {
    const int s = it % C::STAGES;
    if (!mbar_wait_warp(bar(C::B_FULL + s), (it / C::STAGES) & 1, wc)) break;
    const StageMeta* mt = metas + s;
    const int flags = mt->flags;
    if (flags & kStop) break;
    const int start = mt->start, n = mt->n, tile = mt->tile, h = mt->h, len = mt->len, slot = mt->slot;
    const int rows = (int)min((long long)kRows, (long long)n * p.G - (long long)tile * kRows);
    if (flags & kBegin) {
      // Queries, as f16 after a power of two of the row; limits of the rows' keys.
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = g + 8 * half;
        const int rho = tile * kRows + min(i, rows - 1);
        const int tok = rho / p.G;
        const uint4* src = reinterpret_cast<const uint4*>(p.Q + (long long)(start + tok) * p.q_stride +
                                                          (long long)(h * p.G + rho - tok * p.G) * D);
        uint4 w[QI][2];
        uint32_t am = 0;
#pragma unroll
        for (int q = 0; q < QI; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            w[q][e] = __ldg(src + (64 * q + 16 * c) / 8 + e);
            const uint32_t ws[4] = {w[q][e].x, w[q][e].y, w[q][e].z, w[q][e].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t lo = ws[x] & 0x7fffu, hi = (ws[x] >> 16) & 0x7fffu;
              am = max(am, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            }
          }
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // 2^-e with the row's largest at 2^14 (its exponent's floor); e within what fp32 can undo.
        const int e = min(max((int)(am >> 7) - 127, -100), 126) - 14;
        const float up = __int_as_float((127 - e) << 23);
        const float f = __int_as_float((127 + e) << 23) * p.scale_log2;
#pragma unroll
        for (int q = 0; q < QI; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = w[q][j >> 1];
            const uint32_t a = (j & 1) ? v.z : v.x, b = (j & 1) ? v.w : v.y;
            qa[q][j][half] = pack_f16(__uint_as_float(a << 16) * up, __uint_as_float(a & 0xffff0000u) * up);
            qa[q][j][2 + half] = pack_f16(__uint_as_float(b << 16) * up, __uint_as_float(b & 0xffff0000u) * up);
          }
        const int lim = p.causal ? max(0, min(len, len - n + tok + 1)) : len;
        if (half == 0) {
          f0 = f;
          lim0 = lim;
        } else {
          f1 = f;
          lim1 = lim;
        }
      }
      const int first_tok = tile * kRows / p.G, last_tok = (tile * kRows + rows - 1) / p.G;
      lim_all = p.causal ? max(0, min(len, len - n + first_tok + 1)) : len;
      lim_any = p.causal ? max(0, min(len, len - n + last_tok + 1)) : len;
      m0 = m1 = -INFINITY;
      l0 = l1 = vref = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    }
    const int key0 = mt->key0 + 16 * warp;
    const int pg = (16 * warp) >> p.page_log2;
    if (key0 < lim_any && ((mt->pages >> pg) & 1)) {
      const uint32_t kb = sb + C::OFF_RING + s * C::SBYTES, vb = kb + C::KBYTES;
      const float ks = mt->ks[pg], vs = mt->vs[pg];
      float acc[2][4] = {};
#pragma unroll
      for (int q = 0; q < QI; ++q)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint4 w = lds_u4(piece<D>(kb, 16 * warp + 8 * u + ko, c + 4 * q));
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16(acc[u], qa[q][j], widen(ws[j] & 0xffffu), widen(ws[j] >> 16));
        }
      // Columns 2c and 2c + 1 of the two products: keys kv0, kv1 (+ 8).
      const float c0 = f0 * ks, c1 = f1 * ks;
      float x0[4] = {acc[0][0] * c0, acc[0][1] * c0, acc[1][0] * c0, acc[1][1] * c0};
      float x1[4] = {acc[0][2] * c1, acc[0][3] * c1, acc[1][2] * c1, acc[1][3] * c1};
      if (key0 + 16 > lim_all) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + 8 * (e >> 1) + ((e & 1) ? kv1 : kv0);
          if (key >= lim0) x0[e] = -INFINITY;
          if (key >= lim1) x1[e] = -INFINITY;
        }
      }
      float mx0 = fmaxf(fmaxf(x0[0], x0[1]), fmaxf(x0[2], x0[3]));
      float mx1 = fmaxf(fmaxf(x1[0], x1[1]), fmaxf(x1[2], x1[3]));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1) || vs > vref) {
        const float vnew = fmaxf(vref, vs);
        const float rv = vref > 0.f ? __fdiv_rn(vref, vnew) : 0.f;
        const float a0 = n0 > m0 ? ex2(m0 - n0) : 1.f, a1 = n1 > m1 ? ex2(m1 - n1) : 1.f;
        l0 *= a0;
        l1 *= a1;
        const float b0 = a0 * rv, b1 = a1 * rv;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][0] *= b0;
          o[j][1] *= b0;
          o[j][2] *= b1;
          o[j][3] *= b1;
        }
        m0 = n0;
        m1 = n1;
        vref = vnew;
      }
      const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
      const float rr = vref > 0.f ? __fdiv_rn(vs, vref) * kPScale : vs;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x0[e] = ex2(x0[e] - u0);
        x1[e] = ex2(x1[e] - u1);
      }
      l0 += (x0[0] + x0[1]) + (x0[2] + x0[3]);
      l1 += (x1[0] + x1[1]) + (x1[2] + x1[3]);
      uint32_t pa[4];
      pa[0] = pack_f16(x0[0] * rr, x0[1] * rr);
      pa[1] = pack_f16(x1[0] * rr, x1[1] * rr);
      pa[2] = pack_f16(x0[2] * rr, x0[3] * rr);
      pa[3] = pack_f16(x1[2] * rr, x1[3] * rr);
      const int vrow = 16 * warp;
      uint32_t w[4][D / 32];  // four V rows' piece: keys kv0, kv1, kv0 + 8, kv1 + 8
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int rr_ = vrow + 8 * (e >> 1) + ((e & 1) ? kv1 : kv0);
        if constexpr (D == 128) {
          const uint4 v = lds_u4(piece<D>(vb, rr_, cg));
          w[e][0] = v.x;
          w[e][1] = v.y;
          w[e][2] = v.z;
          w[e][3] = v.w;
        } else {
          const uint2 v = lds_u2(piece<D>(vb, rr_, cg) + 8 * (g & 1));
          w[e][0] = v.x;
          w[e][1] = v.y;
        }
      }
      if (key0 + 16 > len) {  // rows behind the request's last key hold anything, a NaN too
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + 8 * (e >> 1) + ((e & 1) ? kv1 : kv0) >= len)
#pragma unroll
            for (int x = 0; x < D / 32; ++x) w[e][x] = 0;
      }
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint32_t a01 = __byte_perm(w[0][x], w[1][x], 0x5140), a23 = __byte_perm(w[0][x], w[1][x], 0x7362);
        const uint32_t b01 = __byte_perm(w[2][x], w[3][x], 0x5140), b23 = __byte_perm(w[2][x], w[3][x], 0x7362);
        mma_f16(o[4 * x + 0], pa, widen(a01 & 0xffffu), widen(b01 & 0xffffu));
        mma_f16(o[4 * x + 1], pa, widen(a01 >> 16), widen(b01 >> 16));
        mma_f16(o[4 * x + 2], pa, widen(a23 & 0xffffu), widen(b23 & 0xffffu));
        mma_f16(o[4 * x + 3], pa, widen(a23 >> 16), widen(b23 >> 16));
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_EMPTY + s));
    if (!(flags & kEnd)) continue;

    // The item's end: the eight warps' sums meet in shared memory.
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    if (c == 0) {
      ml[warp * kRows + g] = make_float2(m0, l0);
      ml[warp * kRows + g + 8] = make_float2(m1, l1);
    }
    float4* so = reinterpret_cast<float4*>(smem + C::OFF_O);
    const float back = vref * (1.f / kPScale);
    // Column 2c of tile j is column 16c + j of the row (d = 128; column 2c + 1:
    // 64 + 16c + j), or 16c + j and 16c + 8 + j (d = 64): a lane holds runs of
    // 16 columns.  16-byte pieces are exchanged within a run so that the
    // lanes of a store meet no bank twice.
    auto at = [&](int w_, int row, int q4) {
      const int run = q4 >> 2, x = (q4 & 3) ^ (((run >> 1) & 1) | ((row & 1) << 1));
      return (w_ * kRows + row) * (D / 4) + run * 4 + x;
    };
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = g + 8 * half;
      if constexpr (D == 128) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            so[at(warp, row, (c + 4 * e) * 4 + x)] =
                make_float4(o[4 * x][2 * half + e] * back, o[4 * x + 1][2 * half + e] * back,
                            o[4 * x + 2][2 * half + e] * back, o[4 * x + 3][2 * half + e] * back);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            so[at(warp, row, c * 4 + 2 * e + x)] =
                make_float4(o[4 * x][2 * half + e] * back, o[4 * x + 1][2 * half + e] * back,
                            o[4 * x + 2][2 * half + e] * back, o[4 * x + 3][2 * half + e] * back);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_WRITTEN));
    if (!mbar_wait_warp(bar(C::B_WRITTEN), ends & 1, wc)) break;
    for (int x = threadIdx.x; x < rows * (D / 4); x += 32 * kWarps) {
      const int row = x / (D / 4), q4 = x % (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w_ = 0; w_ < kWarps; ++w_) M = fmaxf(M, ml[w_ * kRows + row].x);
      const float ref = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w_ = 0; w_ < kWarps; ++w_) {
        const float2 st = ml[w_ * kRows + row];
        const float wgt = ex2(st.x - ref);
        const float4 v = so[at(w_, row, q4)];
        L += wgt * st.y;
        sum.x += wgt * v.x;
        sum.y += wgt * v.y;
        sum.z += wgt * v.z;
        sum.w += wgt * v.w;
      }
      if (slot >= 0) {
        const size_t base = (size_t)(blockIdx.x * 2 + slot) * kRows + row;
        *reinterpret_cast<float4*>(p.part_o + base * D + q4 * 4) = sum;
        if (q4 == 0) *reinterpret_cast<float2*>(p.part_ml + base * 2) = make_float2(M, L);
      } else {
        const int rho = tile * kRows + row, tok = rho / p.G;
        const size_t orow = (size_t)(start + tok) * p.Hq + h * p.G + (rho - tok * p.G);
        const float inv = L > 0.f ? __fdiv_rn(1.f, L) : L == 0.f ? 0.f : L;  // NaN stays
        if (p.out_f32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.O) + orow * D + q4 * 4) =
              make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + orow * D + q4 * 4) =
              make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
        if (q4 == 0) p.LSE[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_READ));
    if (!mbar_wait_warp(bar(C::B_READ), ends & 1, wc)) break;
    ++ends;
  }
}

// Merge of the items cut between workers: worker w's descriptor names the
// item that begins in its range and goes on in the next parts - 1 workers'.
// A warp per row, four rows to a CTA.
template <int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedFwdParams p) {
  griddep_wait();
  const int w = blockIdx.x;
  const int* d = p.desc + w * 8;
  const int parts = d[0];
  if (parts < 2) return;
  const int start = d[1], n = d[2], tile = d[3], h = d[4];
  const int lane = threadIdx.x & 31, row = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (row >= (long long)n * p.G - (long long)tile * kRows) return;
  auto part = [&](int s) -> size_t { return (size_t)(s == 0 ? 2 * w + 1 : 2 * (w + s)) * kRows + row; };
  constexpr int V = D / 32;  // columns of a lane
  float M = -INFINITY;
  for (int s = lane; s < parts; s += 32) M = fmaxf(M, p.part_ml[part(s) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, acc[V] = {};
  for (int s0 = 0; s0 < parts; s0 += 32) {
    float wl = 0.f;
    if (s0 + lane < parts) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + part(s0 + lane) * 2);
      wl = ex2(ml.x - ref);
      L += wl * ml.y;
    }
    const int cnt = min(32, parts - s0);
#pragma unroll 4
    for (int s = 0; s < cnt; ++s) {
      const float wgt = __shfl_sync(0xffffffffu, wl, s);
      const float* src = p.part_o + part(s0 + s) * D + lane * V;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += wgt * src[v];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const int rho = tile * kRows + row, tok = rho / p.G;
  const size_t orow = (size_t)(start + tok) * p.Hq + h * p.G + (rho - tok * p.G);
  const float inv = L > 0.f ? __fdiv_rn(1.f, L) : L == 0.f ? 0.f : L;
#pragma unroll
  for (int v = 0; v < V; v += 2) {
    if (p.out_f32) {
      float* dst = static_cast<float*>(p.O) + orow * D + lane * V + v;
      dst[0] = acc[v] * inv;
      dst[1] = acc[v + 1] * inv;
    } else {
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.O) + orow * D + lane * V + v) =
          pack_bf16(acc[v] * inv, acc[v + 1] * inv);
    }
  }
  if (lane == 0) p.LSE[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int D>
cudaError_t launch_paged(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedFwdParams& p, int workers,
                         cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(fwd_paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PC<D>::SMEM);
  if (e != cudaSuccess) return e;
  fwd_paged_kernel<D><<<workers, kThreads, PC<D>::SMEM, stream>>>(tmK, tmV, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)workers, kRows / 4);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D>, p);
}

size_t part_o_bytes(int d, int sms) { return (size_t)sms * 2 * kRows * d * 4; }
size_t part_ml_bytes(int sms) { return ((size_t)sms * 2 * kRows * 8 + 255) / 256 * 256; }

}  // namespace

size_t paged_fwd_workspace_bytes(int d, int sms) {
  return part_o_bytes(d, sms) + part_ml_bytes(sms) + ((size_t)sms * 32 + 255) / 256 * 256;
}

cudaError_t launch_fwd_paged(int d, const CUtensorMap& tmK, const CUtensorMap& tmV, PagedFwdParams& p, void* workspace,
                             int sms, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + part_o_bytes(d, sms));
  p.desc = reinterpret_cast<int*>(ws + part_o_bytes(d, sms) + part_ml_bytes(sms));
  return d == 128 ? launch_paged<128>(tmK, tmV, p, sms, stream) : launch_paged<64>(tmK, tmV, p, sms, stream);
}

}  // namespace attn
