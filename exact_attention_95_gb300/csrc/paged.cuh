// paged.cuh -- what the two kernels of attention over a paged cache share
// (paged_fwd.cu: few query rows of a kv head; paged_wide.cu: many): the
// division of a ragged batch between the CTAs, and the merge of items that
// were cut.
//
// An item is a tile of ROWS query rows of a request and kv head (rows
// token-major, the G heads of a token side by side) against the keys of the
// request, kUnit keys to a unit.  The units of all items, in one line, are cut
// into equal ranges, one for each CTA (worker), which finds its own from the
// lengths on the device; nothing is planned on the host.  Equal ranges keep
// every SM's memory traffic the same whatever the lengths are.
#pragma once

#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace paged {

constexpr int kUnit = 128;       // keys of a unit

// Bounded wait of a whole warp, with one result.  As short as it can be: it is
// written out at some twenty places, and a kernel's warps wait for instructions
// where there are more than 128 KB of them (three prompt chunks 562 us with
// mbar_wait's form, 447 with this; 440 with a count of tries, which is no limit
// in time).  The clock is read behind a try that failed (one gives up its issue
// slots for about a microsecond), its low half only: a limit is below 2^32 ns.
// A wait that runs out sets the CTA's abort flag, which ends the others and is
// reported at the kernel's end.
struct Waits {
  volatile int* abort_flag;
  uint32_t limit_ns;
};
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Waits& w) {
  uint32_t t0 = 0;
  for (uint32_t first = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); first = 0) {
    const uint32_t now = globaltimer_low_ns();
    if (first) t0 = now;
    if (__any_sync(0xffffffffu, *w.abort_flag != 0 || now - t0 > w.limit_ns)) {
      *w.abort_flag = 1;
      return false;
    }
  }
  return true;
}

constexpr int kMaxGroups = 512;  // 32 requests each

// An item, or the part of it that a worker has.
struct alignas(16) Item {
  int start, n, len;  // the request's query rows, tokens [start, start + n), and its keys
  int req;            // the request
  int tile, h;        // row tile, kv head
  int k0, count;      // the units' numbers in the item: first and how many; count < 0: no more items
  int slot;           // where the result goes: -1 output, else partial slot of this worker
};

// The request's query rows and keys, clipped to the arrays, and its units
// (none where its rows are not this launch's: p.rows_min < n * G <= p.rows_max).
struct Req {
  int start, n, len;
  long long units;
};
// SPLIT: an item counts as that many units, whatever its keys are (below).
template <int ROWS, int SPLIT = 0>
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
    const int rows = q.n * p.G;
    if (rows > p.rows_min && rows <= p.rows_max)
      q.units = (long long)((rows + ROWS - 1) / ROWS) * p.Hkv * (SPLIT ? SPLIT : max(1, (q.len + kUnit - 1) / kUnit));
  }
  return q;
}

// Units of every 32 requests, by `warps` warps; synchronise before reading.
// (Of a single group walk_range sums them itself.)
template <int ROWS, int SPLIT = 0>
__device__ __forceinline__ void sum_units(const PagedFwdParams& p, long long* sums, int warp, int warps, int lane) {
  if (p.R <= 32) return;
#pragma unroll 1
  for (int g = warp; g < (p.R + 31) >> 5; g += warps) {
    long long u = load_req<ROWS, SPLIT>(p, g * 32 + lane).units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    if (lane == 0) sums[g] = u;
  }
}

// Keys that a query token may see.
__device__ __forceinline__ int key_limit(const PagedFwdParams& p, int len, int n, int tok) {
  return p.causal ? max(0, min(len, len - n + tok + 1)) : len;
}

// a / b for non-negative a and b > 0; units rarely need more than 32 bits.
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Up to 32 pages of an item: the units whose page ids and scales a warp holds
// at once (lane i: page i).
struct Batch {
  int k, units;  // first unit and how many
  bool opens;    // the item's first batch
};

// This worker's range, item by item and batch by batch (a whole warp, every
// lane with the same state).  SPLIT: each item has that many workers, the CTAs
// of a cluster, and each worker an equal part of its units, which may be none;
// the grid has a cluster for every item.
template <int ROWS, int SPLIT = 0>
struct Walker {
  const PagedFwdParams& p;
  const long long* sums;
  int lane;
  int groups, g, l;        // request: group of 32, lane
  Req rq;                  // lane's request of the group
  long long pos, end, per; // units: next, end of the range, of a worker
  long long off, units;    // of the request: next unit, all
  Item im;                 // current item
  int seen, ke;            // keys its rows see, end of its units
  int kt, tiles, item;     // units of an item, tiles of the request, next item
  int k;                   // next unit of the item
  bool opened;             // the current item's first batch has been given
  int merge_parts = 0, merge_start = 0, merge_n = 0, merge_tile = 0, merge_h = 0;

  __device__ __forceinline__ Walker(const PagedFwdParams& p_, const long long* sums_, int lane_)
      : p(p_), sums(sums_), lane(lane_) {
    groups = (p.R + 31) >> 5;
    rq = load_req<ROWS, SPLIT>(p, lane);
    long long total = 0;
    if (groups == 1) total = rq.units;
    else
  #pragma unroll 1
      for (int i = lane; i < groups; i += 32) total += sums[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    per = SPLIT ? 1 : divide(total + gridDim.x - 1, gridDim.x);
    pos = min(total, per * blockIdx.x);
    end = min(total, pos + per);
    g = l = k = ke = 0;
    off = units = 0;
    opened = true;
    if (pos >= end) return;
    // The group, then the request, that holds unit `pos`.
    long long before = 0;
#pragma unroll 1
    while (g + 1 < groups && before + sums[g] <= pos) before += sums[g++];
    if (g > 0) rq = load_req<ROWS, SPLIT>(p, g * 32 + lane);
    long long incl = rq.units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    incl += before;
    l = __ffs(__ballot_sync(0xffffffffu, incl > pos)) - 1;
    open_request();
    off = pos - (__shfl_sync(0xffffffffu, incl, l) - units);
    item = (int)divide(off, kt);
    im.k0 = (int)(off - (long long)item * kt);
    open_item();
  }
  __device__ __forceinline__ void open_request() {
    im.req = g * 32 + l;
    im.start = __shfl_sync(0xffffffffu, rq.start, l);
    im.n = __shfl_sync(0xffffffffu, rq.n, l);
    im.len = __shfl_sync(0xffffffffu, rq.len, l);
    units = __shfl_sync(0xffffffffu, rq.units, l);
    kt = SPLIT ? SPLIT : max(1, (im.len + kUnit - 1) / kUnit);
    tiles = (im.n * p.G + ROWS - 1) / ROWS;
    off = 0;
    item = 0;
    im.k0 = 0;
  }
  __device__ __forceinline__ void open_item() {
    im.h = item / tiles;
    // First and last tiles in turn: under the causal mask a tile's share of its
    // kt units grows with its place, and a worker's range then holds early and
    // late ones alike.
    const int at = item - im.h * tiles;
    im.tile = (at & 1) ? tiles - 1 - (at >> 1) : at >> 1;
    int k0 = im.k0, k1 = (int)min((long long)kt, k0 + (end - pos));
    pos += k1 - k0;
    off += k1 - k0;
    if constexpr (SPLIT > 0) {
      const long long all = (im.len + kUnit - 1) / kUnit;
      im.k0 = k0 = (int)(all * k0 / SPLIT);
      k1 = (int)(all * k1 / SPLIT);
    }
    im.slot = k0 == 0 && k1 == kt ? -1 : k0 == 0 ? 1 : 0;
    if (SPLIT == 0 && im.slot == 1) {
      const long long last = pos - (k1 - k0) + kt - 1;  // the item's last unit
      merge_parts = (int)divide(last, per) - (int)blockIdx.x + 1;
      merge_start = im.start;
      merge_n = im.n;
      merge_tile = im.tile;
      merge_h = im.h;
    }
    seen = key_limit(p, im.len, im.n, (min(im.n * p.G, (im.tile + 1) * ROWS) - 1) / p.G);
    ke = max(k0, min(k1, (seen + kUnit - 1) / kUnit));
    im.count = ke - k0;
    k = k0;
    opened = false;
  }
  // The next batch, or false at the range's end.  `im` and `seen` are its item's.
  __device__ __forceinline__ bool next(Batch& b) {
    if (opened && k >= ke) {
      if (pos >= end) return false;
      if (off >= units) {
        // The next request that has units.
        uint32_t more = __ballot_sync(0xffffffffu, rq.units > 0) & ~(0xffffffffu >> (31 - l));
#pragma unroll 1
        while (!more && g + 1 < groups) {
          ++g;
          rq = load_req<ROWS, SPLIT>(p, g * 32 + lane);
          more = __ballot_sync(0xffffffffu, rq.units > 0);
        }
        if (!more) return false;
        l = __ffs(more) - 1;
        open_request();
      } else {
        ++item;
        im.k0 = 0;
      }
      open_item();
    }
    b.opens = !opened;
    opened = true;
    b.k = k;
    b.units = min(ke - k, 32 >> (7 - p.page_log2));
    k += b.units;
    return true;
  }
  // Whether the lane has a page of a batch of the current item, and its id.
  __device__ __forceinline__ bool page_id(const Batch& b, int& id) const {
    const int pg = (b.k << (7 - p.page_log2)) + lane;
    if (pg >= ((b.k + b.units) << (7 - p.page_log2)) || ((long long)pg << p.page_log2) >= seen) return false;
    id = p.block_table[(size_t)im.req * p.max_pages + pg];
    return true;
  }
  __device__ __forceinline__ void write_descriptor() const {
    if (lane == 0) {
      int* d = p.desc + blockIdx.x * 8;
      d[0] = merge_parts;
      d[1] = merge_start;
      d[2] = merge_n;
      d[3] = merge_tile;
      d[4] = merge_h;
    }
  }
};
static_assert(kUnit == 128, "units are 2^7 keys");

// Walks this worker's range (a whole warp): item_fn(Item) announces an item,
// unit_fn(kv head, lane's page id or negative, its K and V scale, place of the
// unit's first page among the lanes) loads the next unit.  Both return false
// to stop; then so does this.  Page ids are read two batches ahead and scales
// one, so that neither latency is waited for but at the start; an item is
// announced as soon as its first ids are on their way (up to two items before
// its units are loaded: the announcements' ring has to hold four).
template <int ROWS, int SPLIT = 0, class ItemFn, class UnitFn>
__device__ __forceinline__ bool walk_range(const PagedFwdParams& p, const long long* sums, int lane, ItemFn item_fn,
                                           UnitFn unit_fn) {
  Walker<ROWS, SPLIT> w(p, sums, lane);
  struct Held {
    int units = 0;  // 0: none, or an item without units
    int id = -1, h = 0;
    float ks = 1.f, vs = 0.f;
    bool any = false, page = false;
  };
  bool ok = true;
  auto take = [&]() -> Held {
    Held x;
    Batch b;
    x.any = ok && w.next(b);
    if (x.any) {
      x.units = b.units;
      x.h = w.im.h;
      x.page = w.page_id(b, x.id);
      if (b.opens) ok = item_fn(w.im);
    }
    return x;
  };
  auto scales = [&](Held& x) {
    if (!x.page) return;
    if (x.id < 0 || x.id >= p.num_pages) {
      x.id = -1;
      atomicCAS(p.status, kDevOk, kDevBounds);
    } else {
      x.ks = p.k_scale[(size_t)x.id * p.Hkv + x.h];
      x.vs = p.v_scale[(size_t)x.id * p.Hkv + x.h];
    }
  };
  const int npg_log2 = 7 - p.page_log2;
  // (One place for each step: the code of a walk is long, and instructions are
  // fetched too.)
  Held cur, nxt;
#pragma unroll 1
  for (;;) {
    scales(nxt);
    const Held then = take();
#pragma unroll 1
    for (int j = 0; j < cur.units && ok; ++j) ok = unit_fn(cur.h, cur.id, cur.ks, cur.vs, j << npg_log2);
    if (!ok || !(nxt.any || then.any)) break;
    cur = nxt;
    nxt = then;
  }
  if (SPLIT == 0) w.write_descriptor();
  return ok;
}

// Two e4m3 codes as two f16 numbers (exact).
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
// Address of 16-byte piece `c` of row `row` of a code tile (rows of D bytes, swizzled).
template <int D>
__device__ __forceinline__ uint32_t piece(uint32_t base, int row, int c) {
  return D == 128 ? base + row * 128 + ((c ^ (row & 7)) << 4) : base + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

// Bytes 0xff where four codes hold a NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t c) { return __vcmpeq4(c & 0x7f7f7f7fu, 0x7f7f7f7fu); }
// A NaN in V at a key that some rows of a tile see and others do not (a drafted
// token behind them, say) would reach all of them: 0 * NaN is one.  The kernels
// take such codes for 0 and note it; at the item's end every row looks up the
// codes of the keys that it does see.  Four codes of key `key` from column c on:
__device__ __forceinline__ uint32_t v_codes(const uint8_t* v_pages, const int* block_table, int num_pages, int page_log2,
                                         int Hkv, int D, size_t row0, int key, int h, int c) {
  const int id = block_table[row0 + (key >> page_log2)];
  if (id < 0 || id >= num_pages) return 0;
  const size_t row = (((size_t)id * Hkv + h) << page_log2) + (key & ((1 << page_log2) - 1));
  return *reinterpret_cast<const uint32_t*>(v_pages + row * D + c);
}

// Row `row` of a tile in the output arrays.
__device__ __forceinline__ size_t output_row(const PagedFwdParams& p, int start, int h, int rho) {
  const int tok = rho / p.G;
  return (size_t)(start + tok) * p.Hq + h * p.G + (rho - tok * p.G);
}

// Debug builds' checks of a copy's coordinate, of a row of the outputs and of a row
// of a worker's partial sums (tiles of `rows` rows).
__device__ __forceinline__ bool plane_ok(const PagedFwdParams& p, int plane) {
  return dcheck(plane >= 0 && plane < p.num_pages * p.Hkv, p.status);
}
__device__ __forceinline__ bool output_ok(const PagedFwdParams& p, size_t orow) {
  return dcheck(orow < (size_t)p.T * p.Hq, p.status);
}
__device__ __forceinline__ bool part_ok(const PagedFwdParams& p, size_t prow, int rows) {
  return dcheck(prow < (size_t)gridDim.x * 2 * rows, p.status);
}

// 1 / l for the output: 0 for a row without keys, NaN stays.
__device__ __forceinline__ float output_factor(float l) { return l > 0.f ? __fdiv_rn(1.f, l) : l == 0.f ? 0.f : l; }
// ln of the sum of a row with maximum m (log2 units).
__device__ __forceinline__ float output_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Launch attribute: may start while the kernel before it in the stream ends.
__host__ inline void overlap_with_previous(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& at) {
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
}

// Launches a kernel of `workers` CTAs with `smem` bytes of dynamic shared
// memory, behind whatever is in the stream (it waits for that kernel before it
// reads anything), in clusters of `cluster` CTAs.  ID tells the kernels of one signature apart: the attribute
// is set once on a device.
template <int ID, class Kernel>
cudaError_t launch_workers(Kernel kern, int threads, int smem, const CUtensorMap& tmK, const CUtensorMap& tmV,
                           const PagedFwdParams& p, int workers, cudaStream_t stream, int cluster = 1) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)workers);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2] = {};
  overlap_with_previous(cfg, at[0]);
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  if (cluster > 1) cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, tmK, tmV, p);
}

}  // namespace paged
}  // namespace attn
