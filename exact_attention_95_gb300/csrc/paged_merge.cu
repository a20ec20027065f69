// paged_merge.cu -- merge of the partial results of attention over a paged
// cache: the items that were cut between workers (paged.cuh).
//
// Worker w's descriptor names the item that begins in its range and goes on in
// the next parts - 1 workers': with M = max_s m_s,
//   l = sum_s 2^{m_s - M} l_s,  O = sum_s 2^{m_s - M} O_s / l.
// Latency bound: launched so that its start overlaps the kernel's end.  Of an
// item in many parts (a long context cut over all workers has dozens) a CTA
// takes a row at a time, its eight warps the parts in turn; else a warp does.
// Measured by leaving it out: 4 us of a call of 121 (64 requests of up to 8192
// keys), 5 of 51 (one of 131072 keys).  Joining the parts in the main kernel, by
// the last of an item's workers, would take counters that are zero at every
// call's start, which a caller's workspace is not; clusters do without (small
// steps, paged_fwd.cu).
#include "paged.cuh"

namespace attn {
namespace {

using namespace paged;

constexpr int kMergeWarps = 8;
constexpr int kTallRows = 128;  // tiles of so many rows keep the warps busy without sharing one

struct MergeSet {
  const float* part_o;
  const float* part_ml;
  const int* desc;
  int rows, workers, ctas;  // of a tile; of the launch; of a worker, here
};
struct MergeParams {
  MergeSet set[2];
  PagedFwdParams p;
};

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const MergeParams q) {
  constexpr int V = D / 32;  // columns of a lane
  __shared__ float s_acc[kMergeWarps][D], s_l[kMergeWarps], s_m[kMergeWarps];
  griddep_launch_dependents();  // the next call's start overlaps this end
  griddep_wait();
  const bool second = (int)blockIdx.x >= q.set[0].workers * q.set[0].ctas;
  const MergeSet& t = q.set[second];
  const PagedFwdParams& p = q.p;
  const int cta = blockIdx.x - (second ? q.set[0].workers * q.set[0].ctas : 0);
  const int w = cta / t.ctas, slice = cta - w * t.ctas;
  const int* d = t.desc + w * 8;
  const int parts = d[0];
  if (parts < 2) return;
  const int start = d[1], n = d[2], tile = d[3], h = d[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = min(t.rows, n * p.G - tile * t.rows);
  // Warps that share a row, and this one's number among them.
  const int team = parts > 2 * kMergeWarps && t.rows < kTallRows ? kMergeWarps : 1, mate = warp % team;
  const int step = t.ctas * (kMergeWarps / team);  // rows at once
  const int rounds = (rows + step - 1) / step;
  for (int i = 0; i < rounds; ++i) {
    const int row = i * step + slice * (kMergeWarps / team) + warp / team;
    if (row >= rows) break;  // (a whole team)
    auto part = [&](int s) -> size_t { return (size_t)(s == 0 ? 2 * w + 1 : 2 * (w + s)) * t.rows + row; };
    // One pass with a running maximum: a part's statistics and sums are one
    // load's wait, four parts at a time.
    float M = -INFINITY, L = 0.f, acc[V] = {};
    for (int s0 = mate; s0 < parts; s0 += 4 * team) {
      float2 ml[4];
      float o[4][V];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int s = s0 + k * team;
        ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) o[k][v] = 0.f;
        if (s < parts) {
          ml[k] = *reinterpret_cast<const float2*>(t.part_ml + part(s) * 2);
          const float* src = t.part_o + part(s) * D + lane * V;
          if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            o[k][0] = x.x, o[k][1] = x.y, o[k][2] = x.z, o[k][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            o[k][0] = x.x, o[k][1] = x.y;
          }
        }
      }
      const float mn = fmaxf(fmaxf(fmaxf(M, ml[0].x), fmaxf(ml[1].x, ml[2].x)), ml[3].x);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float old = ex2(M - ref);
      L *= old;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= old;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float wgt = ex2(ml[k].x - ref);
        L += wgt * ml[k].y;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += wgt * o[k][v];
      }
      M = mn;
    }
    const size_t orow = output_row(p, start, h, tile * t.rows + row);
    const bool in = output_ok(p, orow);
    // Columns c, c + 1 of the row.
    auto put = [&](int c, float x, float y, float inv) {
      if (!in) return;
      if (p.out_f32)
        *reinterpret_cast<float2*>(static_cast<float*>(p.O) + orow * D + c) = make_float2(x * inv, y * inv);
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.O) + orow * D + c) = pack_bf16(x * inv, y * inv);
    };
    if (team == 1) {
#pragma unroll
      for (int v = 0; v < V; v += 2) put(lane * V + v, acc[v], acc[v + 1], output_factor(L));
      if (lane == 0 && in) p.LSE[orow] = output_lse(M, L);
      continue;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
    if (lane == 0) {
      s_l[warp] = L;
      s_m[warp] = M;
    }
    __syncthreads();
    if (threadIdx.x < D / 2) {
      const int c = 2 * threadIdx.x;
      float x = 0.f, y = 0.f;
      M = s_m[0];
#pragma unroll
      for (int j = 1; j < kMergeWarps; ++j) M = fmaxf(M, s_m[j]);
      const float ref = M == -INFINITY ? 0.f : M;
      L = 0.f;
#pragma unroll
      for (int j = 0; j < kMergeWarps; ++j) {
        const float wgt = ex2(s_m[j] - ref);
        x += wgt * s_acc[j][c];
        y += wgt * s_acc[j][c + 1];
        L += wgt * s_l[j];
      }
      put(c, x, y, output_factor(L));
      if (c == 0 && in) p.LSE[orow] = output_lse(M, L);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_paged_merge(int d, const PagedFwdParams& p, int rows, int workers, const PagedFwdParams* p2,
                               int rows2, int workers2, cudaStream_t stream) {
  MergeParams q{};
  q.p = p;
  cudaLaunchConfig_t cfg{};
  // Four CTAs to a worker where items are in many parts (a decoding step with
  // fewer than an eighth as many items as workers), else one: a pass of its warps
  // covers the tile.  Measured, four against one (whole calls, 8 kv heads,
  // d = 128): one request of 131072 keys 51.1 / 56.3 us; the other way 64 requests
  // of up to 8192 keys 124.4 / 122.9 us.  Sixteen for tall tiles, against
  // eight: a chunk of 100 tokens against 4000 keys 31.2 / 37.0 us, of 50 against
  // 20000 (32 kv heads) 71.3 / 70.3.
  const bool few = (long long)p.R * p.Hkv * 8 <= workers;
  const int tall = 16;
  q.set[0] = {p.part_o, p.part_ml, p.desc, rows, workers, rows >= kTallRows ? tall : few ? 4 : 1};
  if (p2) q.set[1] = {p2->part_o, p2->part_ml, p2->desc, rows2, workers2, tall};
  cfg.gridDim = dim3((unsigned)(workers * q.set[0].ctas + workers2 * q.set[1].ctas));
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  overlap_with_previous(cfg, at);
  return d == 128 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<128>, q)
                  : cudaLaunchKernelEx(&cfg, paged_merge_kernel<64>, q);
}

}  // namespace attn
