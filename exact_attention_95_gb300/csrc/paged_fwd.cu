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
// below 2^-31 of the row's largest lose bits).  The weights are rounded to
// f16, relative to the largest V scale seen, times 2^14: 2^-11 relative for
// every weight down to 2^-28 of the row's largest, which a long tail behind
// one dominant key needs (an 8-bit weight, even as a sum of two, would lose
// it).  mma.sync m16n8k16 rather than tcgen05: a tile of eight query
// rows against codes that have to be widened in registers anyway leaves the tensor
// pipe mostly idle at HBM speed, and no accumulator leaves the registers.
//
// A CTA: a producer warp that walks its range and loads whole (page, head)
// boxes by TMA into a ring of units, and four consumer warps, 32 keys of a unit
// each.  Every warp keeps its own running maximum, sum and accumulators of the
// item; they meet in shared memory at the item's end.
//
// SPLIT: a small decoding step gives every item a cluster of SPLIT CTAs, each an
// equal part of its keys.  Their sums meet through distributed shared memory
// instead of through the workspace and a second launch.
//
// Measured (whole calls, 8 kv heads, d = 128, a token a request): 64 requests of
// up to 8192 keys 121 us, 6.2 TB/s; one of 131072 keys 51 us, 5.3 TB/s; four of
// up to 700 keys 7.4 us in clusters (start, lengths, page ids, codes, the meeting:
// each waits for the one before; 9.4 us with the merge's launch).  33 requests of
// up to 3001 keys, 16 kv heads, d = 64: 33 us, 4.3 TB/s.  16 requests of up to
// 5000 keys with six tokens of four heads each, two tiles of 16 rows: 54 us, bound
// by the latencies of a tile's own instructions.  Dropped: a tile of 24 rows, whose sums leave no
// registers for the queries (16 requests of 4096 keys, 24 rows: 71 us against
// 64 by two tiles of 16); three CTAs to an SM for 16 rows too, with the queries
// in shared memory and K's and V's tiles in one ring (49 us against 45 at 16
// rows, 127 against 121 for the 64 requests above: the ring's hand-offs double).
#include "paged.cuh"

namespace attn {
namespace {

using namespace paged;

constexpr int kItems = 4;          // items announced ahead
constexpr float kPScale = 16384.f;

// What a unit's stage holds besides the codes.
struct UnitMeta {
  float ks[8], vs[8];  // scales of its pages
  int pages;           // bit i: page i was loaded
  int pad[3];
};

// NB: eight-row blocks of a tile.  Three CTAs to an SM for one block, two, with
// a third more registers, for two: they share nothing, so one's waits (the
// ends of items, page ids, query rows) are the others' time.
template <int D, int NB>
struct PC {
  static constexpr int ROWS = 8 * NB;
  static constexpr int CTAS = NB == 1 ? 3 : 2;
  static constexpr int WARPS = 4;      // consumer warps, 32 keys of a unit each
  static constexpr int HALF = 2;       // warps whose sums the exchange buffer holds
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr int KBYTES = kUnit * D;
  static constexpr int SBYTES = 2 * KBYTES;
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_O = STAGES * SBYTES;                   // [HALF][ROWS][D] fp32
  static constexpr int OFF_SUMS = OFF_O;                          // [kMaxGroups] int64, until the first item
  static constexpr int OFF_ML = OFF_O + HALF * ROWS * D * 4;      // [2][HALF][ROWS][2] fp32
  static constexpr int OFF_ITEM = OFF_ML + 2 * HALF * ROWS * 8;
  static constexpr int OFF_META = OFF_ITEM + kItems * (int)sizeof(Item);
  static constexpr int OFF_BAR = OFF_META + STAGES * (int)sizeof(UnitMeta);
  static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_IFULL = 2 * STAGES, B_IEMPTY = B_IFULL + kItems;
  static constexpr int B_GIVEN = B_IEMPTY + kItems, B_WRITTEN = B_GIVEN + 1, B_READ = B_GIVEN + 2;
  static constexpr int OFF_NAN = OFF_BAR + (B_READ + 1) * 8;  // [kItems]: number + 1 of an item with a NaN put aside
  static constexpr int OFF_ABORT = OFF_NAN + kItems * 4;
  static constexpr int SMEM = OFF_ABORT + 8 + 1024;
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory");
  static_assert(WARPS == 2 * HALF, "half of the warps hand over to the others");
  static_assert(kMaxGroups * 8 <= HALF * ROWS * D * 4, "the sums fit the exchange buffer");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit elements, two of a row in a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Key index within eight that column n of a product stands for.  The order is
// free; these make the 16-byte (8-byte) shared-memory reads of a swizzled
// page free of bank conflicts.
template <int D>
__device__ __forceinline__ int key_of(int n) {
  return D == 128 ? (n >> 1) | ((n & 1) << 2) : n ^ ((n >> 1) & 1);
}
// Piece q4 (four columns) of an output row: its sum, maximum and weights' sum.
template <int D>
__device__ __forceinline__ void put_piece(const PagedFwdParams& p, size_t orow, int q4, float4 sum, float M, float L) {
  const float inv = output_factor(L);
  if (!output_ok(p, orow)) return;
  if (p.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.O) + orow * D + q4 * 4) =
        make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + orow * D + q4 * 4) =
        make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
  if (q4 == 0) p.LSE[orow] = output_lse(M, L);
}

// All threads of the cluster's CTAs; what they wrote before is seen after.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Shared memory of the cluster's CTA r at this CTA's address a.
__device__ __forceinline__ uint32_t peer(uint32_t a, int r) {
  uint32_t x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(a), "r"(r));
  return x;
}
__device__ __forceinline__ uint4 peer_u4(uint32_t a, int r) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(peer(a, r)));
  return v;
}
__device__ __forceinline__ uint2 peer_u2(uint32_t a, int r) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(peer(a, r)));
  return v;
}

template <int D, int NB, int SPLIT>
__global__ void __launch_bounds__(PC<D, NB>::THREADS, PC<D, NB>::CTAS)
    fwd_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PagedFwdParams p) {
  using C = PC<D, NB>;
  constexpr int kRows = C::ROWS, kWarps = C::WARPS, kHalf = C::HALF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  volatile int* nans = reinterpret_cast<volatile int*>(smem + C::OFF_NAN);
  UnitMeta* metas = reinterpret_cast<UnitMeta*>(smem + C::OFF_META);
  Item* items = reinterpret_cast<Item*>(smem + C::OFF_ITEM);
  long long* sums = reinterpret_cast<long long*>(smem + C::OFF_SUMS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar(C::B_FULL + s), 1);
      mbar_init(bar(C::B_EMPTY + s), kWarps);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(C::B_IFULL + i), 1);
      mbar_init(bar(C::B_IEMPTY + i), kWarps);
    }
    mbar_init(bar(C::B_GIVEN), kWarps - kHalf);
    mbar_init(bar(C::B_WRITTEN), kHalf);
    mbar_init(bar(C::B_READ), kHalf);
    *abort_flag = 0;
    for (int i = 0; i < kItems; ++i) nans[i] = 0;
    fence_mbar_init();
  }
  if (!p.behind) griddep_wait();  // the lengths, pages and queries of the kernel before
  sum_units<kRows, SPLIT>(p, sums, warp, kWarps + 1, lane);
  __syncthreads();
  const Waits wc{abort_flag, (uint32_t)p.wait_limit_ns};

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int npg = kUnit >> p.page_log2;  // pages of a unit
    const uint32_t page_bytes = (uint32_t)D << p.page_log2;
    int it = 0, stage = 0, turn = 0;  // units loaded; place and round of the next in the ring
    int items_out = 0;  // items announced
    auto announce = [&](const Item& im) -> bool {
      const int i = items_out % kItems;
      if (items_out >= kItems && !wait_bar(bar(C::B_IEMPTY + i), ((items_out / kItems) & 1) ^ 1, wc)) return false;
      if (lane == 0) {
        items[i] = im;
        mbar_arrive(bar(C::B_IFULL + i));
      }
      // The item's query rows, on their way to L1 before the warps ask for them.
      constexpr int LINES = D * 2 / 128;  // of a row
      const int rows = min(kRows, im.n * p.G - im.tile * kRows);
#pragma unroll 1
      for (int x = lane; x < rows * LINES; x += 32) {
        const int rho = im.tile * kRows + x / LINES, tok = rho / p.G;
        const uint16_t* q = p.Q + (long long)(im.start + tok) * p.q_stride +
                            (long long)(im.h * p.G + rho - tok * p.G) * D + x % LINES * 64;
        asm volatile("prefetch.global.L1 [%0];" ::"l"(q));
      }
      __syncwarp();
      ++items_out;
      return true;
    };
    bool ok = walk_range<kRows, SPLIT>(
        p, sums, lane, announce, [&](int h, int id, float ks, float vs, int in_batch) -> bool {
          const int s = stage;
          if (it >= C::STAGES && !wait_bar(bar(C::B_EMPTY + s), turn ^ 1, wc)) return false;
          const int my = __shfl_sync(0xffffffffu, id, in_batch + (lane & 7));
          const bool load = lane < npg && my >= 0;
          const uint32_t mask = __ballot_sync(0xffffffffu, load);
          // The copies are issued first: the barrier's phase cannot end before
          // the arrival below, which waits for the scales.
          if (load) {
            const uint32_t dst = sb + C::OFF_RING + s * C::SBYTES + lane * page_bytes;
            const int plane = my * p.Hkv + h;
            if (plane_ok(p, plane)) {
              tma_load_3d(dst, &tmK, bar(C::B_FULL + s), 0, 0, plane);
              tma_load_3d(dst + C::KBYTES, &tmV, bar(C::B_FULL + s), 0, 0, plane);
            }
          }
          UnitMeta* m = metas + s;
          const float mk = __shfl_sync(0xffffffffu, ks, in_batch + (lane & 7));
          const float mv = __shfl_sync(0xffffffffu, vs, in_batch + (lane & 7));
          if (lane < 8) {
            m->ks[lane] = mk;
            m->vs[lane] = mv;
          }
          if (lane == 0) m->pages = (int)mask;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(bar(C::B_FULL + s), 2 * page_bytes * __popc(mask));
          ++it;
          if (++stage == C::STAGES) {
            stage = 0;
            turn ^= 1;
          }
          return true;
        });
    if (ok) {
      Item im{};  // (no rows)
      im.count = -1;
      ok = announce(im);
    }
    // Copies in flight land before the CTA leaves (the consumers have waited
    // for all of them unless a wait gave up).
    if (!ok) {
      const WaitCtx drain{abort_flag, p.status, p.wait_limit_ns};
#pragma unroll 1
      for (int k = max(0, it - C::STAGES); k < it; ++k)
        mbar_wait_drain_warp(bar(C::B_FULL + k % C::STAGES), (k / C::STAGES) & 1, drain);
    }
    if (*abort_flag && lane == 0) atomicCAS(p.status, kDevOk, kDevTimeout);
    griddep_launch_dependents();
    // Behind the wide kernel: this one's completion stands for both.
    if (p.behind) griddep_wait();
    if constexpr (SPLIT > 0) {
      cluster_meet();
      cluster_meet();
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  const int part = 32 * warp;   // its keys in a unit
  const int ko = key_of<D>(g);  // its key as a row of the first product (and 8 more)
  const int kv0 = key_of<D>(2 * c), kv1 = key_of<D>(2 * c + 1);  // its keys as a column of the second
  const int cg = D == 128 ? (g >> 1) | ((g & 1) << 2) : g >> 1;  // its 16-byte piece of a V row
  constexpr int QI = D / 64;   // 64-column parts of the contraction over d
  constexpr int MT = D / 16;   // 16-column tiles of O
  uint32_t qb[NB][QI][4][2];
  float o[NB][MT][4];
  // Of each block rows 2c and 2c + 1: running maximum, sum, factor of the products, limit of the keys.
  float m[NB][2], l[NB][2], f[NB][2], vref = 0.f;
  int lim[NB][2], lim_all = 0, lim_any = 0;
  // Places of its pieces in a unit's K and V: rows 8 further on are 8 * D bytes
  // on; the other half of a row's pieces (d = 128) is 64 bytes away, by the
  // swizzle in the direction that flips bit 6.
  const uint32_t koff = piece<D>(0, part + ko, c);
  const uint32_t voff0 = piece<D>(0, part + kv0, cg) + (D == 64 ? 8 * (g & 1) : 0);
  const uint32_t voff1 = piece<D>(0, part + kv1, cg) + (D == 64 ? 8 * (g & 1) : 0);
  int stage = 0, turn = 0;  // place and round of the next unit in the ring
  auto consume = [&]() {
#pragma unroll 1
    for (int i = 0;; ++i) {
      if (!wait_bar(bar(C::B_IFULL + i % kItems), (i / kItems) & 1, wc)) return;
      const Item* im = items + i % kItems;
      const int count = im->count;
      if (count < 0) return;
      const int tile = im->tile, h = im->h, len = im->len, n = im->n, start = im->start;
      const int rows = min(kRows, n * p.G - tile * kRows);
      // Queries (row g of a block), as f16 after a power of two of the row; limits of the rows' keys.
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int rho = tile * kRows + min(8 * b + g, rows - 1);
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
            for (int x = 0; x < 4; ++x) am = __vmaxu2(am, ws[x] & 0x7fff7fffu);
          }
        am = max(am & 0xffffu, am >> 16);
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        // 2^-e takes the row's largest to [2^14, 2^15); e within what fp32 can undo.
        const int e = min(max((int)(am >> 7) - 127, -100), 126) - 14;
        // An infinity or NaN in the row: NaN for all of it, so that every logit is one (an
        // infinity times codes of one sign would give -inf alone, a masked key's).
        const float up = am >= 0x7f80u ? NAN : __int_as_float((127 - e) << 23);
        const float fr = __int_as_float((127 + e) << 23) * p.scale_log2;
#pragma unroll
        for (int q = 0; q < QI; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = w[q][j >> 1];
            const uint32_t x = (j & 1) ? v.z : v.x, y = (j & 1) ? v.w : v.y;
            qb[b][q][j][0] = pack_f16(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
            qb[b][q][j][1] = pack_f16(__uint_as_float(y << 16) * up, __uint_as_float(y & 0xffff0000u) * up);
          }
        const int lr = key_limit(p, len, n, tok);
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          f[b][e2] = __shfl_sync(0xffffffffu, fr, 8 * c + 4 * e2);
          lim[b][e2] = __shfl_sync(0xffffffffu, lr, 8 * c + 4 * e2);
          m[b][e2] = -INFINITY;
          l[b][e2] = 0.f;
        }
        if (b == 0) lim_all = __shfl_sync(0xffffffffu, lr, 0);        // the first token's
        if (b == NB - 1) lim_any = __shfl_sync(0xffffffffu, lr, 28);  // the last one's
#pragma unroll
        for (int j = 0; j < MT; ++j) o[b][j][0] = o[b][j][1] = o[b][j][2] = o[b][j][3] = 0.f;
      }
      vref = 0.f;
      int key0 = im->k0 * kUnit + part;
#pragma unroll 1
      for (int u = 0; u < count; ++u, key0 += kUnit) {
        const int s = stage;
        if (!wait_bar(bar(C::B_FULL + s), turn, wc)) return;
        const UnitMeta* mt = metas + s;
        const int pa = part >> p.page_log2, pb = (part + 16) >> p.page_log2;  // pages of its two 16 keys
        const bool la = (mt->pages >> pa) & 1, lb = (mt->pages >> pb) & 1;
        if (key0 < lim_any && (la || lb)) {
          const uint32_t kb = sb + C::OFF_RING + s * C::SBYTES, vb = kb + C::KBYTES;
          // S^T = K Q^T: twice 16 keys by 8 rows of a block.
          float acc[NB][2][4] = {};
#pragma unroll
          for (int q = 0; q < QI; ++q) {
            const uint32_t ka = (kb + koff) ^ (64 * q);
            const uint4 w0 = lds_u4(ka), w1 = lds_u4(ka + 8 * D), w2 = lds_u4(ka + 16 * D), w3 = lds_u4(ka + 24 * D);
            const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
            const uint32_t x2[4] = {w2.x, w2.y, w2.z, w2.w}, x3[4] = {w3.x, w3.y, w3.z, w3.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a0[4] = {widen(x0[j]), widen(x1[j]), widen(x0[j] >> 16), widen(x1[j] >> 16)};
              const uint32_t a1[4] = {widen(x2[j]), widen(x3[j]), widen(x2[j] >> 16), widen(x3[j] >> 16)};
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                mma_f16(acc[b][0], a0, qb[b][q][j][0], qb[b][q][j][1]);
                mma_f16(acc[b][1], a1, qb[b][q][j][0], qb[b][q][j][1]);
              }
            }
          }
          // Keys ko, ko + 8 (and 16 on) of rows 2c, 2c + 1.
          const float vsa = mt->vs[pa], vsb = mt->vs[pb];
          const float ksa = mt->ks[pa], ksb = mt->ks[pb];
          const bool edge = key0 + 32 > lim_all || !la || !lb;
          const float vsm = fmaxf(la ? vsa : 0.f, lb ? vsb : 0.f);
          const float vnew = fmaxf(vref, vsm);
          const float rv = vnew > vref && vref > 0.f ? __fdiv_rn(vref, vnew) : vnew > vref ? 0.f : 1.f;
          vref = vnew;
          const float rra = vsa == vref ? kPScale : vref > 0.f ? __fdiv_rn(vsa, vref) * kPScale : vsa;
          const float rrb = vsb == vref ? kPScale : vref > 0.f ? __fdiv_rn(vsb, vref) * kPScale : vsb;
          uint32_t pt[NB][4];  // P^T with row g and the keys of a column pair in a lane
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float ca0 = f[b][0] * ksa, ca1 = f[b][1] * ksa, cb0 = f[b][0] * ksb, cb1 = f[b][1] * ksb;
            if (edge) {
              // A factor that underflowed must not meet the infinities (any sum times 1e-37 is 0 as well).
              ca0 = fmaxf(ca0, 1e-37f);
              ca1 = fmaxf(ca1, 1e-37f);
              cb0 = fmaxf(cb0, 1e-37f);
              cb1 = fmaxf(cb1, 1e-37f);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (key0 + 8 * (e >> 1) + ko >= lim[b][e & 1] || !(e < 4 ? la : lb)) acc[b][e >> 2][e & 3] = -INFINITY;
            }
            float mx0 = fmaxf(fmaxf(acc[b][0][0], acc[b][0][2]) * ca0, fmaxf(acc[b][1][0], acc[b][1][2]) * cb0);
            float mx1 = fmaxf(fmaxf(acc[b][0][1], acc[b][0][3]) * ca1, fmaxf(acc[b][1][1], acc[b][1][3]) * cb1);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
              mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
            }
            if (__any_sync(0xffffffffu, mx0 > m[b][0] || mx1 > m[b][1]) || rv != 1.f) {
              const float n0 = fmaxf(m[b][0], mx0), n1 = fmaxf(m[b][1], mx1);
              const float a0 = n0 > m[b][0] ? ex2(m[b][0] - n0) : 1.f, a1 = n1 > m[b][1] ? ex2(m[b][1] - n1) : 1.f;
              l[b][0] *= a0;
              l[b][1] *= a1;
              const float b0 = a0 * rv, b1 = a1 * rv;
#pragma unroll
              for (int j = 0; j < MT; ++j) {
                o[b][j][0] *= b0;
                o[b][j][1] *= b1;
                o[b][j][2] *= b0;
                o[b][j][3] *= b1;
              }
              m[b][0] = n0;
              m[b][1] = n1;
            }
            const float u0 = m[b][0] == -INFINITY ? 0.f : m[b][0], u1 = m[b][1] == -INFINITY ? 0.f : m[b][1];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float rr = e ? rrb : rra, c0 = e ? cb0 : ca0, c1 = e ? cb1 : ca1;
              const float x0 = ex2(fmaf(acc[b][e][0], c0, -u0)), x1 = ex2(fmaf(acc[b][e][1], c1, -u1));
              const float x2 = ex2(fmaf(acc[b][e][2], c0, -u0)), x3 = ex2(fmaf(acc[b][e][3], c1, -u1));
              l[b][0] += x0 + x2;
              l[b][1] += x1 + x3;
              pt[b][2 * e] = transpose8(pack_f16(x0 * rr, x1 * rr));
              pt[b][2 * e + 1] = transpose8(pack_f16(x2 * rr, x3 * rr));
            }
          }
          // O^T += V^T P^T: row g of tile t is column 16 cg + 2t (d = 64: 8g + 2t), row g + 8 the one after.
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[4][D / 32];  // four V rows' piece: keys kv0, kv1, kv0 + 8, kv1 + 8
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t va = vb + ((e & 1) ? voff1 : voff0) + (16 * hf + 8 * (e >> 1)) * D;
              if constexpr (D == 128) {
                const uint4 v = lds_u4(va);
                w[e][0] = v.x;
                w[e][1] = v.y;
                w[e][2] = v.z;
                w[e][3] = v.w;
              } else {
                const uint2 v = lds_u2(va);
                w[e][0] = v.x;
                w[e][1] = v.y;
              }
            }
            if (edge) {  // V rows that no row of the tile sees hold anything, a NaN too
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + 16 * hf + 8 * (e >> 1) + ((e & 1) ? kv1 : kv0);
                const bool seen = key < lim_any && (hf ? lb : la);
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {
                  const uint32_t bad = seen && key >= lim_all ? nan_codes(w[e][y]) : 0u;
                  if (bad) nans[i % kItems] = i + 1;
                  w[e][y] = seen ? w[e][y] & ~bad : 0u;
                }
              }
            }
#pragma unroll
            for (int y = 0; y < D / 32; ++y) {
              const uint32_t a01 = __byte_perm(w[0][y], w[1][y], 0x5140), a23 = __byte_perm(w[0][y], w[1][y], 0x7362);
              const uint32_t b01 = __byte_perm(w[2][y], w[3][y], 0x5140), b23 = __byte_perm(w[2][y], w[3][y], 0x7362);
              const uint32_t t0[4] = {widen(a01), widen(a01 >> 16), widen(b01), widen(b01 >> 16)};
              const uint32_t t1[4] = {widen(a23), widen(a23 >> 16), widen(b23), widen(b23 >> 16)};
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                mma_f16(o[b][2 * y], t0, pt[b][2 * hf], pt[b][2 * hf + 1]);
                mma_f16(o[b][2 * y + 1], t1, pt[b][2 * hf], pt[b][2 * hf + 1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_EMPTY + s));
        if (++stage == C::STAGES) {
          stage = 0;
          turn ^= 1;
        }
      }

      // The item's end: the warps' sums meet in shared memory.
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
      float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
      float4* so = reinterpret_cast<float4*>(smem + C::OFF_O);
      const float back = vref * (1.f / kPScale);
      // Place of 16-byte piece q4 of a row: exchanged with its neighbours so that
      // the eight lanes of a store (four rows, two pieces) meet no bank twice.
      auto at = [&](int w_, int row, int q4) {
        const int c2 = (row >> 1) & 3;
        const int x = D == 128 ? c2 | ((q4 >> 4) << 2) : (c2 & 1) | ((c2 >> 1) << 2);
        return (w_ * kRows + row) * (D / 4) + (q4 ^ x);
      };
      // The last item's sums have been read.
      if (i > 0 && !wait_bar(bar(C::B_READ), (i - 1) & 1, wc)) return;
      if (warp >= kHalf) {
        // Hand over to warp - kHalf, lane by lane.
        float4* to = so + (warp - kHalf) * kRows * (D / 4) + lane;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < MT; ++j)
            to[32 * (b * MT + j)] =
                make_float4(o[b][j][0] * back, o[b][j][1] * back, o[b][j][2] * back, o[b][j][3] * back);
        if (g == 0)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              ml[(warp - kHalf) * kRows + 8 * b + 2 * c + e] = make_float2(m[b][e], l[b][e]);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(C::B_GIVEN));
          mbar_arrive(bar(C::B_IEMPTY + i % kItems));
        }
        continue;
      }
      const int slot = im->slot;
      if (!wait_bar(bar(C::B_GIVEN), i & 1, wc)) return;
      const float4* from = so + warp * kRows * (D / 4) + lane;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float wa[2], wb[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 gv = ml[warp * kRows + 8 * b + 2 * c + e];
          const float mn = fmaxf(m[b][e], gv.x), r = mn == -INFINITY ? 0.f : mn;
          const float x = ex2(m[b][e] - r);
          wb[e] = ex2(gv.x - r);
          wa[e] = back * x;
          l[b][e] = l[b][e] * x + gv.y * wb[e];
          m[b][e] = mn;
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const float4 v = from[32 * (b * MT + j)];
          o[b][j][0] = fmaf(o[b][j][0], wa[0], v.x * wb[0]);
          o[b][j][1] = fmaf(o[b][j][1], wa[1], v.y * wb[1]);
          o[b][j][2] = fmaf(o[b][j][2], wa[0], v.z * wb[0]);
          o[b][j][3] = fmaf(o[b][j][3], wa[1], v.w * wb[1]);
        }
      }
      __syncwarp();
      ml += kHalf * kRows;
      if (g == 0)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) ml[warp * kRows + 8 * b + 2 * c + e] = make_float2(m[b][e], l[b][e]);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < MT / 2; ++x)
            so[at(warp, 8 * b + 2 * c + e, (D == 128 ? 4 * cg : 2 * g) + x)] =
                make_float4(o[b][2 * x][e], o[b][2 * x][2 + e], o[b][2 * x + 1][e], o[b][2 * x + 1][2 + e]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_WRITTEN));
      if (!wait_bar(bar(C::B_WRITTEN), i & 1, wc)) return;
#pragma unroll 1
      for (int x = threadIdx.x; x < rows * (D / 4); x += 32 * kHalf) {
        const int row = x / (D / 4), q4 = x % (D / 4);
        float M = -INFINITY;
#pragma unroll 4
        for (int w_ = 0; w_ < kHalf; ++w_) M = fmaxf(M, ml[w_ * kRows + row].x);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w_ = 0; w_ < kHalf; ++w_) {
          const float2 st = ml[w_ * kRows + row];
          const float wgt = ex2(st.x - ref);
          const float4 v = so[at(w_, row, q4)];
          L += wgt * st.y;
          sum.x += wgt * v.x;
          sum.y += wgt * v.y;
          sum.z += wgt * v.z;
          sum.w += wgt * v.w;
        }
        if (nans[i % kItems] == i + 1) {
          const int tok = (tile * kRows + row) / p.G;
          const int from = max(im->k0 * kUnit, lim_all), to = min((im->k0 + count) * kUnit, key_limit(p, len, n, tok));
#pragma unroll 1
          for (int key = from; key < to; ++key) {
            const uint32_t bad = nan_codes(v_codes(p.v_pages, p.block_table, p.num_pages, p.page_log2, p.Hkv, D,
                                                   (size_t)im->req * p.max_pages, key, h, q4 * 4));
            if (bad & 0xffu) sum.x = NAN;
            if (bad & 0xff00u) sum.y = NAN;
            if (bad & 0xff0000u) sum.z = NAN;
            if (bad & 0xff000000u) sum.w = NAN;
          }
        }
        if constexpr (SPLIT > 0) {
          // For the cluster: where this thread has read its own piece, and where the statistics handed over were.
          so[at(0, row, q4)] = sum;
          if (q4 == 0) ml[row - kHalf * kRows] = make_float2(M, L);
        } else if (slot >= 0) {
          const size_t base = (size_t)(blockIdx.x * 2 + slot) * kRows + row;
          if (!part_ok(p, base, kRows)) continue;
          *reinterpret_cast<float4*>(p.part_o + base * D + q4 * 4) = sum;
          if (q4 == 0) *reinterpret_cast<float2*>(p.part_ml + base * 2) = make_float2(M, L);
        } else {
          put_piece<D>(p, output_row(p, start, h, tile * kRows + row), q4, sum, M, L);
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::B_READ));
        mbar_arrive(bar(C::B_IEMPTY + i % kItems));
      }
    }
  };
  consume();
  // A wait that gave up.
  if (*abort_flag && lane == 0) atomicCAS(p.status, kDevOk, kDevTimeout);
  if constexpr (SPLIT > 0) {
    // The item's parts, from the shared memory of the cluster's CTAs: each
    // joins every SPLIT-th 32 pieces.  Without an item there is none in all of them.
    __syncwarp();
    cluster_meet();
    const Item* im = items;  // (the first announcement)
    if (warp == 0 && im->count >= 0) {
      const int tile = im->tile, h = im->h, start = im->start, rows = min(kRows, im->n * p.G - tile * kRows);
#pragma unroll 1
      for (int x = 32 * (int)cluster_rank() + lane; x < rows * (D / 4); x += 32 * SPLIT) {
        const int row = x / (D / 4), q4 = x % (D / 4);
        const int c2 = (row >> 1) & 3, sw = D == 128 ? c2 | ((q4 >> 4) << 2) : (c2 & 1) | ((c2 >> 1) << 2);
        float2 st[SPLIT];
        float4 v[SPLIT];
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
          const uint4 a = peer_u4(sb + C::OFF_O + (row * (D / 4) + (q4 ^ sw)) * 16, r);
          const uint2 b = peer_u2(sb + C::OFF_ML + row * 8, r);
          v[r] = make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w));
          st[r] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
        }
        float M = st[0].x;
#pragma unroll
        for (int r = 1; r < SPLIT; ++r) M = fmaxf(M, st[r].x);
        const float ref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < SPLIT; ++r) {
          const float wgt = ex2(st[r].x - ref);
          L += wgt * st[r].y;
          sum.x += wgt * v[r].x;
          sum.y += wgt * v[r].y;
          sum.z += wgt * v[r].z;
          sum.w += wgt * v[r].w;
        }
        put_piece<D>(p, output_row(p, start, h, tile * kRows + row), q4, sum, M, L);
      }
    }
    __syncwarp();
    cluster_meet();
  }
}

}  // namespace

namespace {

template <int D, int NB, int SPLIT = 0>
cudaError_t launch_narrow(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedFwdParams& p, int workers,
                          cudaStream_t stream) {
  using C = PC<D, NB>;
  static_assert(C::CTAS == paged_ctas(C::ROWS), "workers of an SM");
  return launch_workers<D * 64 + NB * 16 + SPLIT>(fwd_paged_kernel<D, NB, SPLIT>, C::THREADS, C::SMEM, tmK, tmV, p,
                                                       workers, stream, SPLIT ? SPLIT : 1);
}

}  // namespace

cudaError_t launch_paged_narrow(int d, int rows, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                const PagedFwdParams& p, int workers, int split, cudaStream_t stream) {
  if (split == 8)
    return d == 128 ? launch_narrow<128, 1, 8>(tmK, tmV, p, workers, stream)
                    : launch_narrow<64, 1, 8>(tmK, tmV, p, workers, stream);
  if (split == 4)
    return d == 128 ? launch_narrow<128, 1, 4>(tmK, tmV, p, workers, stream)
                    : launch_narrow<64, 1, 4>(tmK, tmV, p, workers, stream);
  if (rows == 8)
    return d == 128 ? launch_narrow<128, 1>(tmK, tmV, p, workers, stream)
                    : launch_narrow<64, 1>(tmK, tmV, p, workers, stream);
  return d == 128 ? launch_narrow<128, 2>(tmK, tmV, p, workers, stream)
                  : launch_narrow<64, 2>(tmK, tmV, p, workers, stream);
}

}  // namespace attn
