// paged_wide.cu -- attention over a paged 8-bit key/value cache for requests
// with many query rows of a kv head: prompt chunks, verification of drafted
// tokens, large groups.  The same function as paged_fwd.cu computes.
//
// Tensor bound: per unit of 128 keys and 128-row tile, S = Q K^T and O += P V
// are two 128 x 128 x d products of 512 clocks each at d = 128.  Both run on
// tcgen05 with the codes as they come or exactly widened:
//   S: K's e4m3 codes straight from the page boxes against Q as the sum of
//      two e4m3 numbers, hi = e4m3(q / s), lo = e4m3(q / s - hi) with s a power
//      of two of the row (kind::f8f6f4, twice the rate, two products: the
//      time of one 16-bit product and no widening of K).  bf16 has 8
//      significant bits, hi and lo four each.  With the row's largest element
//      scaled to (224, 448] the sum is exact for elements from 2^-2 on, 2^-9.8 of
//      the largest, and off by at most 2^-10 below, 2^-17.8 of it.
//   P V: P in f16 from TMEM, V's codes widened to f16 in shared memory (kind::f16).
//      P is not split into 8-bit terms: below 2^-18 of the row's largest
//      weight they hold nothing, and the tail behind one dominant key is lost.
//
// Two row tiles (256 rows) to an item share every unit.  Roles (16 warps):
//   warp 0       producer: walks the range, loads page boxes (TMA).
//   warps 1, 2   MMA issuers of row tile 0 and 1 (as in fwd_persist.cu).
//   warp 3       idle.
//   warps 4-7    widen V: 8-bit tile -> f16 tile, 64-column blocks.
//   warps 8-11, 12-15  softmax and epilogue of tile 0, 1; a thread is a row.
// TMEM (512 columns): S [0, 128) shared by the tiles in turn, P_t 64 columns
// each, O_t d columns each.  A tile without rows takes part in every hand-off
// and skips the work.
//
// Measured: three requests with chunks of up to 1000 tokens against up to 16384
// keys, 32 query and 8 kv heads, d = 128: 440 us, 1200 TFLOPS (63 % of a plain
// bf16 product's rate); the tensor pipe is busy 56 % of the time, the softmax
// warps issue the rest.  Dropped: the tiles with an S buffer each, or a unit to
// each tile in turn where an item has up to 128 rows (477 to 635 us).
#include "paged.cuh"

namespace attn {
namespace {

using namespace paged;

constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128;
constexpr int kRegsLow = 72;    // producer and issuers
constexpr int kRegsWiden = 56;
constexpr int kRegsHigh = 192;  // softmax
static_assert(128 * (kRegsLow + kRegsWiden) + 256 * kRegsHigh <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr int kBM = 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kMetas = 8;       // units whose scales are kept
constexpr int kItems = 4;       // items announced ahead
// P is 2^9 times the weight relative to 2^m, and m moves when the row's
// maximum exceeds it by more than 2^6: P <= 2^15 fits f16, and weights down to
// 2^-23 of 2^m are normal numbers.
constexpr float kShift = 9.f;
constexpr float kThreshold = 6.f;
constexpr float kLowRatio = -60.f;  // log2 of the smallest V scale ratio that is told from zero

struct UnitMeta {
  float ks[8];  // for every 16 keys: K scale of their page
  float lv[8];  // log2 of its V scale, -infinity where the page was not loaded
  int pages;    // bit i: page i was loaded
  int pad[3];
};

template <int D>
struct WC {
  static constexpr int KS = D == 128 ? 3 : 6;   // K tiles
  static constexpr int VS = D == 128 ? 3 : 6;   // V code tiles
  static constexpr int WS = 2;                  // widened V tiles
  static constexpr int T8 = kUnit * D;          // bytes of a code tile
  static constexpr int T16 = 2 * T8;
  static constexpr int OFF_Q = 0;               // per row tile: hi, lo
  static constexpr int OFF_K = 4 * T8;
  static constexpr int OFF_V = OFF_K + KS * T8;
  static constexpr int OFF_W = OFF_V + VS * T8;
  static constexpr int OFF_SUMS = OFF_W;        // until the first item
  static constexpr int OFF_ITEM = OFF_W + WS * T16;
  static constexpr int OFF_META = OFF_ITEM + kItems * (int)sizeof(Item);
  static constexpr int OFF_BAR = OFF_META + kMetas * (int)sizeof(UnitMeta);
  static constexpr int B_KFULL = 0;
  static constexpr int B_KEMPTY = B_KFULL + KS;
  static constexpr int B_VFULL = B_KEMPTY + KS;
  static constexpr int B_VEMPTY = B_VFULL + VS;
  static constexpr int B_WFULL = B_VEMPTY + VS;
  static constexpr int B_WEMPTY = B_WFULL + WS;
  static constexpr int B_MFULL = B_WEMPTY + WS;
  static constexpr int B_MEMPTY = B_MFULL + kMetas;
  static constexpr int B_IFULL = B_MEMPTY + kMetas;
  static constexpr int B_IEMPTY = B_IFULL + kItems;
  static constexpr int B_QFULL = B_IEMPTY + kItems;  // 2
  static constexpr int B_SFULL = B_QFULL + 2;        // 2
  static constexpr int B_SREAD = B_SFULL + 2;        // 2
  static constexpr int B_PFULL = B_SREAD + 2;        // 2
  static constexpr int B_ODONE = B_PFULL + 2;        // 2
  static constexpr int B_DRAIN = B_ODONE + 2;        // 2
  static constexpr int OFF_NAN = OFF_BAR + (B_DRAIN + 2) * 8;  // [kItems]: number + 1 of an item with a NaN put aside
  static constexpr int OFF_TMEMSLOT = OFF_NAN + kItems * 4;
  static constexpr int OFF_ABORT = OFF_TMEMSLOT + 4;
  static constexpr int SMEM = OFF_ABORT + 4 + 1024;
  static constexpr uint32_t IDESC_S = idesc_e4m3(kBM, kUnit);
  // f16 A and B (format 0), fp32 sums, B as V's rows (MN-major).
  static constexpr uint32_t IDESC_O = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
  static constexpr uint32_t TM_S = 0, TM_P = 128, TM_O = 256;
};
static_assert(WC<128>::SMEM <= 232448 && WC<64>::SMEM <= 232448, "shared memory");
static_assert(kMaxGroups * 8 <= WC<64>::WS * WC<64>::T16, "the sums fit the widened tiles");

// Descriptor of a K-major tile of D-byte rows: 128-byte or 64-byte swizzle, groups of eight rows 8 * D bytes apart.
template <int D>
__device__ __forceinline__ uint64_t code_desc(uint32_t addr) {
  if constexpr (D == 128) return sdesc_sw128(addr, 16, 1024);
  // Layout code 4: 64-byte swizzle.
  return (sdesc_sw128(addr, 16, 512) & ~(uint64_t(7) << 61)) | (uint64_t(4) << 61);
}
// The four e4m3 values of packed codes.
__device__ __forceinline__ void values4(uint32_t c, float (&x)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(x[2 * k]), "=f"(x[2 * k + 1])
        : "r"(widen(c >> (16 * k))));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_paged_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const PagedFwdParams p) {
  using C = WC<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::OFF_BAR + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEMSLOT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
  volatile int* nans = reinterpret_cast<volatile int*>(smem + C::OFF_NAN);
  UnitMeta* metas = reinterpret_cast<UnitMeta*>(smem + C::OFF_META);
  Item* items = reinterpret_cast<Item*>(smem + C::OFF_ITEM);
  long long* sums = reinterpret_cast<long long*>(smem + C::OFF_SUMS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();  // the lengths, pages and queries of the kernel before
  // A batch without such requests costs a look at their row counts.
  bool any = false;
  for (int r = threadIdx.x; r < p.R; r += kThreads) any |= load_req<kPagedWideRows>(p, r).units > 0;
  if (!__syncthreads_or(any)) {
    if (threadIdx.x == 0) p.desc[blockIdx.x * 8] = 0;  // nothing to merge
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::KS; ++s) {
      mbar_init(bar(C::B_KFULL + s), 1);
      mbar_init(bar(C::B_KEMPTY + s), 2);  // both tiles' products
    }
    for (int s = 0; s < C::VS; ++s) {
      mbar_init(bar(C::B_VFULL + s), 1);
      mbar_init(bar(C::B_VEMPTY + s), 4);  // widening warps
    }
    for (int s = 0; s < C::WS; ++s) {
      mbar_init(bar(C::B_WFULL + s), 4);
      mbar_init(bar(C::B_WEMPTY + s), 2);
    }
    for (int s = 0; s < kMetas; ++s) {
      mbar_init(bar(C::B_MFULL + s), 1);
      mbar_init(bar(C::B_MEMPTY + s), 12);  // softmax and widening warps
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(bar(C::B_IFULL + s), 1);
      mbar_init(bar(C::B_IEMPTY + s), 14);  // all but the producer and the idle warp
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(C::B_QFULL + t), 4);
      mbar_init(bar(C::B_SFULL + t), 1);
      mbar_init(bar(C::B_SREAD + t), 4);
      mbar_init(bar(C::B_PFULL + t), 4);
      mbar_init(bar(C::B_ODONE + t), 1);
      mbar_init(bar(C::B_DRAIN + t), 1);
    }
    *abort_flag = 0;
    for (int i = 0; i < kItems; ++i) nans[i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  sum_units<kPagedWideRows>(p, sums, warp, kThreads / 32, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Waits wc{abort_flag, (uint32_t)p.wait_limit_ns};
  const WaitCtx drain{abort_flag, p.status, p.wait_limit_ns};
  // Item i, for a consumer warp.
  auto wait_item = [&](int i) -> bool { return wait_bar(bar(C::B_IFULL + i % kItems), (i / kItems) & 1, wc); };
  auto release_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_IEMPTY + i % kItems));
  };
  auto release = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };

  if (warp < 4) {
    regs_dec<kRegsLow>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
      const int npg = kUnit >> p.page_log2;
      const uint32_t page_bytes = (uint32_t)D << p.page_log2;
      int u = 0;          // units loaded
      int items_out = 0;  // items announced
      auto reuse = [&](int b, int n, int ring) -> bool {  // wait until place n % ring is free again
        return n < ring || wait_bar(bar(b + n % ring), ((n / ring) & 1) ^ 1, wc);
      };
      auto announce = [&](const Item& im) -> bool {
        if (!reuse(C::B_IEMPTY, items_out, kItems)) return false;
        if (lane == 0) {
          items[items_out % kItems] = im;
          mbar_arrive(bar(C::B_IFULL + items_out % kItems));
        }
        __syncwarp();
        ++items_out;
        return true;
      };
      bool ok = walk_range<kPagedWideRows>(
          p, sums, lane, announce, [&](int h, int id, float ks, float vs, int in_batch) -> bool {
            const int my = __shfl_sync(0xffffffffu, id, in_batch + (lane & 7));
            const bool load = lane < npg && my >= 0;
            const uint32_t mask = __ballot_sync(0xffffffffu, load);
            const uint32_t bytes = page_bytes * __popc(mask);
            const int plane = my * p.Hkv + h;
            if (!reuse(C::B_KEMPTY, u, C::KS)) return false;
            const int sk = u % C::KS;
            if (load && plane_ok(p, plane))
              tma_load_3d(sb + C::OFF_K + sk * C::T8 + lane * page_bytes, &tmK, bar(C::B_KFULL + sk), 0, 0, plane);
            if (lane == 0) mbar_arrive_expect_tx(bar(C::B_KFULL + sk), bytes);
            if (!reuse(C::B_MEMPTY, u, kMetas)) return false;
            UnitMeta* m = metas + u % kMetas;
            const int seg = ((lane & 7) * 16) >> p.page_log2;
            const float mk = __shfl_sync(0xffffffffu, ks, in_batch + seg);
            const float mv = __shfl_sync(0xffffffffu, vs, in_batch + seg);
            if (lane < 8) {
              m->ks[lane] = mk;
              m->lv[lane] = lg2(mv);
            }
            if (lane == 0) m->pages = (int)mask;
            release(C::B_MFULL + u % kMetas);
            if (!reuse(C::B_VEMPTY, u, C::VS)) return false;
            const int sv = u % C::VS;
            if (load && plane_ok(p, plane))
              tma_load_3d(sb + C::OFF_V + sv * C::T8 + lane * page_bytes, &tmV, bar(C::B_VFULL + sv), 0, 0, plane);
            if (lane == 0) mbar_arrive_expect_tx(bar(C::B_VFULL + sv), bytes);
            ++u;
            return true;
          });
      if (ok) {
        Item im{};
        im.count = -1;
        announce(im);
      }
      // Copies in flight land before the CTA leaves: those of the units loaded
      // whole, and K's of one whose loading was given up.
      for (int k = max(0, u - C::KS); k < u; ++k) mbar_wait_drain_warp(bar(C::B_KFULL + k % C::KS), (k / C::KS) & 1, drain);
      for (int k = max(0, u - C::VS); k < u; ++k) mbar_wait_drain_warp(bar(C::B_VFULL + k % C::VS), (k / C::VS) & 1, drain);
      if (!ok) mbar_wait_drain_warp(bar(C::B_KFULL + u % C::KS), (u / C::KS) & 1, drain);
      griddep_launch_dependents();
    } else if (warp < 3) {
      // ---------------------------------------------------------- MMA issuers
      const int t = warp - 1;
      int u0 = 0;  // units before the item
      int qn = 0;  // items with units
      int ns = 0;  // S products of this tile issued
      int pf = 0;  // P_t hand-offs waited for
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (!wait_item(i)) break;
        const Item* im = items + i % kItems;
        const int n = im->count;
        const bool live = im->n * p.G - im->tile * kPagedWideRows > t * kBM;
        release_item(i);
        if (n < 0) break;
        if (n == 0) continue;
        auto wait_ring = [&](int b, int k, int ring) -> bool {
          if (!wait_bar(bar(b + k % ring), (k / ring) & 1, wc)) return false;
          tc_fence_after();
          return true;
        };
        // The S buffer is free for this tile's next S once the other tile has
        // read the S issued before it (S_0(j), S_1(j), S_0(j + 1), ...).
        auto wait_sbuf = [&]() -> bool {
          if (t == 0 && ns == 0) return true;
          const int phase = t == 0 ? ns - 1 : ns;
          if (!wait_bar(bar(C::B_SREAD + (t ^ 1)), phase & 1, wc)) return false;
          tc_fence_after();
          return true;
        };
        auto issue_s = [&](int j) {
          const int s = (u0 + j) % C::KS;
          if (live) {
            uint64_t qd = code_desc<D>(sb + C::OFF_Q + t * 2 * C::T8);
            asm volatile("" : "+l"(qd));
            const uint64_t kd = code_desc<D>(sb + C::OFF_K + s * C::T8);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_ss_f8_warp(tmem + C::TM_S, qd + ((part * C::T8 + kk * 32) >> 4), kd + (kk * 32 >> 4), C::IDESC_S,
                               part + kk > 0 ? 1u : 0u);
          }
          tc_commit_warp(bar(C::B_SFULL + t));
          tc_commit_warp(bar(C::B_KEMPTY + s));
          ++ns;
        };
        auto issue_pv = [&](int j) {
          const int s = (u0 + j) % C::WS;
          if (live) {
            const uint64_t vd = sdesc_sw128(sb + C::OFF_W + s * C::T16, 16384, 1024);
#pragma unroll
            for (int kk = 0; kk < kUnit / 16; ++kk)
              mma_ts_warp(tmem + C::TM_O + t * D, tmem + C::TM_P + t * 64 + kk * 8, vd + (kk * 2048 >> 4), C::IDESC_O,
                          (kk > 0 || j > 0) ? 1u : 0u);
          }
          tc_commit_warp(bar(C::B_ODONE + t));
          tc_commit_warp(bar(C::B_WEMPTY + s));
        };
        ok = wait_sbuf() && wait_bar(bar(C::B_QFULL + t), qn & 1, wc) && wait_ring(C::B_KFULL, u0, C::KS);
        if (ok) issue_s(0);
        for (int j = 0; j < n && ok; ++j) {
          if (j + 1 < n) {
            ok = wait_sbuf() && wait_ring(C::B_KFULL, u0 + j + 1, C::KS);
            if (!ok) break;
            issue_s(j + 1);
          }
          ok = wait_ring(C::B_WFULL, u0 + j, C::WS) && wait_bar(bar(C::B_PFULL + t), pf & 1, wc);
          if (!ok) break;
          ++pf;
          tc_fence_after();
          issue_pv(j);
        }
        u0 += n;
        ++qn;
      }
      // All products of this warp complete before TMEM is released.
      tc_commit_warp(bar(C::B_DRAIN + t));
      mbar_wait_drain_warp(bar(C::B_DRAIN + t), 0, drain);
    }
  } else if (warp < 8) {
    regs_dec<kRegsWiden>();
    // ---------------------------------------------------------- widening of V
    const int wl = threadIdx.x - 128;
    int u = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!wait_item(i)) break;
      const Item* im = items + i % kItems;
      const int n = im->count, k0 = im->k0;
      // Keys behind the last one that a row of the tile sees hold anything, a NaN code too.
      const int seen =
          key_limit(p, im->len, im->n, (min(im->n * p.G, (im->tile + 1) * kPagedWideRows) - 1) / p.G);
      const int seen_all = key_limit(p, im->len, im->n, im->tile * kPagedWideRows / p.G);  // by its first row
      release_item(i);
      if (n < 0) break;
      for (int j = 0; j < n; ++j, ++u) {
        const int sv = u % C::VS, sw = u % C::WS;
        if (!wait_bar(bar(C::B_MFULL + u % kMetas), (u / kMetas) & 1, wc) ||
            !wait_bar(bar(C::B_VFULL + sv), (u / C::VS) & 1, wc) ||
            (u >= C::WS && !wait_bar(bar(C::B_WEMPTY + sw), ((u / C::WS) & 1) ^ 1, wc))) {
          ok = false;
          break;
        }
        const uint32_t pages = (uint32_t)metas[u % kMetas].pages;
        const int valid = min(kUnit, seen - (k0 + j) * kUnit);
        const int all = seen_all - (k0 + j) * kUnit;
        const bool whole = all >= kUnit && pages == (1u << (kUnit >> p.page_log2)) - 1;
        constexpr int PC = D / 16;  // pieces of a row
        const uint32_t src = sb + C::OFF_V + sv * C::T8, dst = sb + C::OFF_W + sw * C::T16;
        // Piece x of this thread, widened.
        auto put = [&](int x, const uint4& v) {
          const int e = wl + 128 * x, row = e / PC, pc = e % PC;
          const uint32_t base = dst + (pc >> 2) * 16384 + row * 128;
          const int c0 = 2 * (pc & 3);
          // The two halves in an order that keeps the eight lanes of a row off each other's banks.
          const int flip = pc >> 2;
          const uint32_t first[2] = {flip ? v.z : v.x, flip ? v.w : v.y}, second[2] = {flip ? v.x : v.z, flip ? v.y : v.w};
          sts_u4(base + (((c0 + flip) ^ (row & 7)) << 4), widen(first[0]), widen(first[0] >> 16), widen(first[1]),
                 widen(first[1] >> 16));
          sts_u4(base + (((c0 + 1 - flip) ^ (row & 7)) << 4), widen(second[0]), widen(second[0] >> 16),
                 widen(second[1]), widen(second[1] >> 16));
        };
        constexpr int NX = kUnit * PC / 128;  // pieces of a thread
        if (whole) {
#pragma unroll 1
          for (int x0 = 0; x0 < NX; x0 += 4) {
            uint4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int e = wl + 128 * (x0 + x);
              v[x] = lds_u4(piece<D>(src, e / PC, e % PC));
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) put(x0 + x, v[x]);
          }
        } else {
#pragma unroll 1
          for (int x = 0; x < NX; ++x) {
            const int e = wl + 128 * x, row = e / PC;
            uint4 v = lds_u4(piece<D>(src, row, e % PC));
            if (row >= valid || !((pages >> (row >> p.page_log2)) & 1)) {
              v = make_uint4(0, 0, 0, 0);
            } else if (row >= all) {  // some rows do not see it
              const uint32_t b0 = nan_codes(v.x), b1 = nan_codes(v.y), b2 = nan_codes(v.z), b3 = nan_codes(v.w);
              if (b0 | b1 | b2 | b3) nans[i % kItems] = i + 1;
              v = make_uint4(v.x & ~b0, v.y & ~b1, v.z & ~b2, v.w & ~b3);
            }
            put(x, v);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(C::B_WFULL + sw));
          mbar_arrive(bar(C::B_VEMPTY + sv));
          mbar_arrive(bar(C::B_MEMPTY + u % kMetas));
        }
      }
    }
  } else {
    regs_inc<kRegsHigh>();
    // ---------------------------------------------------------- softmax + epilogue
    const int t = (warp - 8) >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t s_t = tmem + lane_off + C::TM_S;
    const uint32_t p_t = tmem + lane_off + C::TM_P + t * 64;
    const uint32_t o_t = tmem + lane_off + C::TM_O + t * D;
    const uint32_t q_hi = sb + C::OFF_Q + t * 2 * C::T8, q_lo = q_hi + C::T8;
    int u = 0;   // units
    int sg = 0;  // S tiles completed (one per unit; ODONE likewise)
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!wait_item(i)) break;
      const Item* im = items + i % kItems;
      const int n = im->count;
      if (n < 0) break;
      const int rho = im->tile * kPagedWideRows + t * kBM + row;
      const int last = im->n * p.G - 1;  // last row of the request
      // A warp without rows takes part in the hand-offs only.
      const bool live = rho - lane <= last;
      const int tok = min(rho, last) / p.G;
      const int lim = key_limit(p, im->len, im->n, tok);
      const int lim_all = __shfl_sync(0xffffffffu, lim, 0);  // the warp's first row's
      float f = 0.f;
      if (n > 0) {
        if (live) {
          // This thread's row of Q as hi + lo.  The products that read the
          // tile's last Q have completed: their S tiles were waited for.
          const uint4* src = reinterpret_cast<const uint4*>(
              p.Q + (long long)(im->start + tok) * p.q_stride +
              (long long)(im->h * p.G + min(rho, last) - tok * p.G) * D);
          uint32_t am = 0;
          uint4 qr[D / 8];  // one wait for all of them
#pragma unroll
          for (int x = 0; x < D / 8; ++x) qr[x] = __ldg(src + x);
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            const uint32_t w[4] = {qr[x].x, qr[x].y, qr[x].z, qr[x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) am = __vmaxu2(am, w[y] & 0x7fff7fffu);
          }
          am = max(am & 0xffffu, am >> 16);
          // 2^k with the row's largest in (224, 448].
          int k = (int)(am >> 7) - 127 - ((am & 0x7f) <= 0x60 ? 8 : 7);
          k = min(max(k, -110), 118);
          // An infinity or NaN in the row: NaN codes for all of it.  Its logits are NaN
          // then, but for those of masked keys (a row that sees none stays empty).
          const float down = am >= 0x7f80u ? NAN : __int_as_float((127 - k) << 23);
          f = __int_as_float((127 + k) << 23) * p.scale_log2;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint4 v = qr[2 * x + y];
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const float a0 = __uint_as_float(w[2 * z] << 16) * down, a1 = __uint_as_float(w[2 * z] & 0xffff0000u) * down;
                const float a2 = __uint_as_float(w[2 * z + 1] << 16) * down;
                const float a3 = __uint_as_float(w[2 * z + 1] & 0xffff0000u) * down;
                const uint32_t h4 = pack_e4m3x4(a0, a1, a2, a3);
                float r[4];
                values4(h4, r);
                hi[2 * y + z] = h4;
                lo[2 * y + z] = pack_e4m3x4(a0 - r[0], a1 - r[1], a2 - r[2], a3 - r[3]);
              }
            }
            sts_u4(piece<D>(q_hi, row, x), hi[0], hi[1], hi[2], hi[3]);
            sts_u4(piece<D>(q_lo, row, x), lo[0], lo[1], lo[2], lo[3]);
          }
          fence_async_smem();
        }
        release(C::B_QFULL + t);
      }
      float m = -INFINITY, l = 0.f;
      float lvref = -1e30f;  // log2 of the largest V scale seen
      for (int j = 0; j < n; ++j, ++u) {
        const int key0 = (im->k0 + j) * kUnit;
        if (!wait_bar(bar(C::B_MFULL + u % kMetas), (u / kMetas) & 1, wc) ||
            !wait_bar(bar(C::B_SFULL + t), sg & 1, wc)) {
          ok = false;
          break;
        }
        ++sg;
        tc_fence_after();
        // The hand-off of S(j) back, of the scales, and of P(j) once P(j - 1) has been used.
        if (!live) {
          tc_fence_before();
          release(C::B_SREAD + t);
          if (lane == 0) mbar_arrive(bar(C::B_MEMPTY + u % kMetas));
          if (j > 0 && !wait_bar(bar(C::B_ODONE + t), sg & 1, wc)) {
            ok = false;
            break;
          }
          release(C::B_PFULL + t);
          continue;
        }
        const UnitMeta* mt = metas + u % kMetas;
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_t + c * 32, sr[c]);
        tmem_ld_wait(sr[0]);
        reg_fence32(sr[1]);
        reg_fence32(sr[2]);
        reg_fence32(sr[3]);
        tc_fence_before();
        release(C::B_SREAD + t);
        float alpha = 1.f;
        bool move = false;
        uint32_t wv[2][32];
        {
          const uint32_t pages = (uint32_t)mt->pages;
          if (key0 + kUnit > lim_all || pages != (1u << (kUnit >> p.page_log2)) - 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (key0 + c * 32 + x >= lim || !((pages >> ((c * 32 + (x & 16)) >> p.page_log2)) & 1))
                  sr[c][x] = __float_as_uint(-INFINITY);
          }
          float cf[8], lv[8];
#pragma unroll
          for (int x = 0; x < 8; x += 4) {
            const float4 a = *reinterpret_cast<const float4*>(mt->ks + x);
            const float4 b = *reinterpret_cast<const float4*>(mt->lv + x);
            cf[x] = f * a.x, cf[x + 1] = f * a.y, cf[x + 2] = f * a.z, cf[x + 3] = f * a.w;
            lv[x] = b.x, lv[x + 1] = b.y, lv[x + 2] = b.z, lv[x + 3] = b.w;
          }
          // Largest logit and V scale of the unit; 16 keys are of one page.  A
          // factor that underflowed must not meet an infinity (a sum times
          // 1e-37 is 0 as well); a NaN stays.
          float mx = -INFINITY, lvm = -INFINITY;
#pragma unroll
          for (int sgm = 0; sgm < 8; ++sgm) {
            const int c = sgm >> 1, x0 = 16 * (sgm & 1);
            if (cf[sgm] < 1e-37f) cf[sgm] = 1e-37f;
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int x = 0; x < 8; x += 2) {
              a = fmax3(a, __uint_as_float(sr[c][x0 + x]), __uint_as_float(sr[c][x0 + x + 1]));
              b = fmax3(b, __uint_as_float(sr[c][x0 + 8 + x]), __uint_as_float(sr[c][x0 + 9 + x]));
            }
            mx = fmaxf(mx, fmaxf(a, b) * cf[sgm]);
            lvm = fmaxf(lvm, lv[sgm]);
          }
          move = mx > m + kThreshold || lvm > lvref;
          if (move) {
            const float mn = fmaxf(m, mx), ln = fmaxf(lvref, lvm);
            alpha = ex2(m - mn);
            if (mn == -INFINITY) alpha = 1.f;
            l *= alpha;
            alpha *= ex2(lvref - ln);
            m = mn;
            lvref = ln;
          }
          const float m_use = m == -INFINITY ? 0.f : m;
          float lsum = 0.f;
#pragma unroll
          for (int sgm = 0; sgm < 8; ++sgm) {
            const int c = sgm >> 1, x0 = 16 * (sgm & 1);
            const float ratio = fmaxf(lv[sgm] - lvref, kLowRatio) + kShift;
            const uint64_t c2 = f2pack(cf[sgm], cf[sgm]), off2 = f2pack(ratio - m_use, ratio - m_use);
            uint64_t rs = 0, rs1 = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              float y0, y1;
              f2unpack(ffma2(f2pack(__uint_as_float(sr[c][x0 + 2 * x]), __uint_as_float(sr[c][x0 + 2 * x + 1])), c2, off2),
                       y0, y1);
              const float p0 = ex2(y0), p1 = ex2(y1);
              if (x & 1) rs1 = fadd2(rs1, f2pack(p0, p1));
              else rs = fadd2(rs, f2pack(p0, p1));
              wv[c >> 1][(c & 1) * 16 + (x0 >> 1) + x] = pack_f16(p0, p1);
            }
            float a0, a1;
            f2unpack(fadd2(rs, rs1), a0, a1);
            lsum = fmaf(a0 + a1, ex2(-ratio), lsum);
          }
          l += lsum;
        }
        release(C::B_MEMPTY + u % kMetas);
        if (j > 0) {
          // The item's last P_t V has completed: it read the P_t written below, and O_t may be scaled.
          if (!wait_bar(bar(C::B_ODONE + t), sg & 1, wc)) {  // phase sg - 2
            ok = false;
            break;
          }
          tc_fence_after();
          if (__any_sync(0xffffffffu, move)) {
            // 32 columns at a time: P_t's 64 registers are live here.
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_t + c * 32, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tmem_st32(o_t + c * 32, o);
            }
          }
        }
        tmem_st32(p_t, wv[0]);
        tmem_st32(p_t + 32, wv[1]);
        tmem_st_wait();
        tc_fence_before();
        release(C::B_PFULL + t);
      }
      if (!ok) break;
      if (n > 0) {
        if (!wait_bar(bar(C::B_ODONE + t), (sg - 1) & 1, wc)) break;
        tc_fence_after();
      }
      if (live) {
        // O = sums * part * mul.  (In one factor the smallest V scales would be lost:
        // 2^-126 * 2^-9 / l is subnormal.)
        const size_t orow = output_row(p, im->start, im->h, min(rho, last));
        const float part = (im->slot < 0 ? output_factor(l) : 1.f) * (1.f / (1 << (int)kShift));
        const float mul = n > 0 ? ex2(lvref) : 0.f;
        const size_t prow = (size_t)(blockIdx.x * 2 + max(im->slot, 0)) * kPagedWideRows + t * kBM + row;
        const bool valid = rho <= last && output_ok(p, orow) && part_ok(p, prow, kPagedWideRows);
        // bf16 rows go through the warp's quarter of the Q tile (whose products have completed).
        const uint32_t stage = q_hi + quad * 32 * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(o_t + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * part);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0u;
          }
          if (im->slot >= 0 || p.out_f32) {
            if (valid) {
              float4* dst = reinterpret_cast<float4*>(im->slot >= 0 ? p.part_o + prow * D + c * 32
                                                                    : static_cast<float*>(p.O) + orow * D + c * 32);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                dst[x] = make_float4(__uint_as_float(o[4 * x]) * mul, __uint_as_float(o[4 * x + 1]) * mul,
                                     __uint_as_float(o[4 * x + 2]) * mul, __uint_as_float(o[4 * x + 3]) * mul);
            }
          } else if constexpr (D == 128) {
            epi_stage32(stage, lane, c, o, mul);
            if (c & 1) {
              __syncwarp();
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int r = 4 * x + (lane >> 3), k = lane & 7;
                const uint4 v = lds_u4(stage + r * 128 + ((k ^ (r & 7)) << 4));
                const size_t to = __shfl_sync(0xffffffffu, (unsigned long long)orow, r);
                if (rho - lane + r <= last && output_ok(p, to))
                  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + to * D + (c >> 1) * 64 + k * 8) = v;
              }
              __syncwarp();
            }
          } else if (valid) {
            // d = 64: a row's 64 bytes at a time, as it stands.
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + orow * D + c * 32);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              dst[x] = make_uint4(pack_bf16(__uint_as_float(o[8 * x]) * mul, __uint_as_float(o[8 * x + 1]) * mul),
                                  pack_bf16(__uint_as_float(o[8 * x + 2]) * mul, __uint_as_float(o[8 * x + 3]) * mul),
                                  pack_bf16(__uint_as_float(o[8 * x + 4]) * mul, __uint_as_float(o[8 * x + 5]) * mul),
                                  pack_bf16(__uint_as_float(o[8 * x + 6]) * mul, __uint_as_float(o[8 * x + 7]) * mul));
          }
        }
        __syncwarp();
        if (n > 0 && nans[i % kItems] == i + 1 && valid) {
          // Over what the warp has stored.
          const int from = max(im->k0 * kUnit, key_limit(p, im->len, im->n, im->tile * kPagedWideRows / p.G));
          const int to = min((im->k0 + n) * kUnit, lim);
#pragma unroll 1
          for (int key = from; key < to; ++key)
#pragma unroll 1
            for (int c = 0; c < D; ++c) {
              if (!(nan_codes(v_codes(p.v_pages, p.block_table, p.num_pages, p.page_log2, p.Hkv, D,
                                      (size_t)im->req * p.max_pages, key, im->h, c & ~3)) >> (8 * (c & 3)) & 0xffu))
                continue;
              if (im->slot >= 0) p.part_o[prow * D + c] = NAN;
              else if (p.out_f32) static_cast<float*>(p.O)[orow * D + c] = NAN;
              else static_cast<uint16_t*>(p.O)[orow * D + c] = 0x7fc0;
            }
        }
        if (valid) {
          if (im->slot >= 0) *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m, l);
          else p.LSE[orow] = output_lse(m, l);
        }
      }
      release_item(i);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicCAS(p.status, kDevOk, kDevTimeout);
}

template <int D>
cudaError_t launch_wide(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedFwdParams& p, int workers,
                        cudaStream_t stream) {
  // The register split draws on what the launch allocates: it has to be kLaunchRegs a thread.
  static std::atomic<int> known{-1};  // one per instantiation
  int regs = known.load(std::memory_order_relaxed);
  if (regs < 0) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, fwd_paged_wide_kernel<D>);
    if (e != cudaSuccess) return e;
    known.store(regs = fa.numRegs, std::memory_order_relaxed);
  }
  if (regs != kLaunchRegs) return cudaErrorInvalidKernelImage;
  return launch_workers<D>(fwd_paged_wide_kernel<D>, kThreads, WC<D>::SMEM, tmK, tmV, p, workers, stream);
}

}  // namespace

cudaError_t launch_paged_wide(int d, const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedFwdParams& p,
                              int workers, cudaStream_t stream) {
  return d == 128 ? launch_wide<128>(tmK, tmV, p, workers, stream) : launch_wide<64>(tmK, tmV, p, workers, stream);
}

}  // namespace attn
