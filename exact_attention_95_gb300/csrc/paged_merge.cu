// paged_merge.cu -- merge of the partial results of attention over a paged
// cache: the items that were cut between workers (paged.cuh).
//
// Worker w's descriptor names the item that begins in its range and goes on in
// the next parts - 1 workers': with M = max_s m_s,
//   l = sum_s 2^{m_s - M} l_s,  O = sum_s 2^{m_s - M} O_s / l.
// Latency bound: launched so that its start overlaps the kernel's end.  A warp
// per row, kMergeCtas CTAs of four warps to an item.
#include <algorithm>

#include "paged.cuh"

namespace attn {
namespace {

using namespace paged;

constexpr int kMergeCtas = 8;

struct MergeSet {
  const float* part_o;
  const float* part_ml;
  const int* desc;
  int rows;
};
struct MergeParams {
  MergeSet set[2];
  PagedFwdParams p;
};

template <int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(const MergeParams q) {
  griddep_wait();
  const MergeSet& t = q.set[blockIdx.z];
  const PagedFwdParams& p = q.p;
  const int w = blockIdx.x;
  const int* d = t.desc + w * 8;
  const int parts = d[0];
  if (parts < 2) return;
  const int start = d[1], n = d[2], tile = d[3], h = d[4];
  const int lane = threadIdx.x & 31;
  const int rows = min(t.rows, n * p.G - tile * t.rows);
  for (int row = blockIdx.y * 4 + (threadIdx.x >> 5); row < rows; row += 4 * gridDim.y) {
    auto part = [&](int s) -> size_t { return (size_t)(s == 0 ? 2 * w + 1 : 2 * (w + s)) * t.rows + row; };
    constexpr int V = D / 32;  // columns of a lane
    float M = -INFINITY;
    for (int s = lane; s < parts; s += 32) M = fmaxf(M, t.part_ml[part(s) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[V] = {};
    for (int s0 = 0; s0 < parts; s0 += 32) {
      float wl = 0.f;
      if (s0 + lane < parts) {
        const float2 ml = *reinterpret_cast<const float2*>(t.part_ml + part(s0 + lane) * 2);
        wl = ex2(ml.x - ref);
        L += wl * ml.y;
      }
      const int cnt = min(32, parts - s0);
#pragma unroll 4
      for (int s = 0; s < cnt; ++s) {
        const float wgt = __shfl_sync(0xffffffffu, wl, s);
        const float* src = t.part_o + part(s0 + s) * D + lane * V;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += wgt * src[v];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const size_t orow = output_row(p, start, h, tile * t.rows + row);
    const float inv = output_factor(L);
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
    if (lane == 0) p.LSE[orow] = output_lse(M, L);
  }
}

}  // namespace

cudaError_t launch_paged_merge(int d, const PagedFwdParams& p, int rows, const PagedFwdParams* p2, int rows2,
                               int workers, cudaStream_t stream) {
  MergeParams q{};
  q.p = p;
  q.set[0] = {p.part_o, p.part_ml, p.desc, rows};
  if (p2) q.set[1] = {p2->part_o, p2->part_ml, p2->desc, rows2};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)workers, (unsigned)std::min(std::max(rows, p2 ? rows2 : 0) / 4, kMergeCtas), p2 ? 2u : 1u);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  overlap_with_previous(cfg, at);
  return d == 128 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<128>, q)
                  : cudaLaunchKernelEx(&cfg, paged_merge_kernel<64>, q);
}

}  // namespace attn
