// rope.cu -- rotary positions of queries and keys, and their gradient (rope.cuh
// has the mathematics).
#include <algorithm>

#include "launch.cuh"
#include "rope.cuh"

namespace attn {
namespace {

template <class T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeParams p, int heads) {
  griddep_wait();
  rope_block<T, D, INTER>(p, blockIdx.x, blockIdx.y * heads, heads);
}

template <class T, int D>
cudaError_t launch(const RopeParams& p, int interleaved, int sms, cudaStream_t stream) {
  const long long groups = ((long long)p.B * p.N + rope_tokens(D) - 1) / rope_tokens(D);
  const int heads = rope_heads(groups, p.Hq + p.Hkv, 16LL * sms);
  const dim3 grid((unsigned)groups, (unsigned)((p.Hq + p.Hkv + heads - 1) / heads));
  return interleaved ? launch_behind(rope_kernel<T, D, true>, grid, kRopeThreads, stream, 0, p, heads)
                     : launch_behind(rope_kernel<T, D, false>, grid, kRopeThreads, stream, 0, p, heads);
}

}  // namespace

// Heads of a CTA: as many as leave about `ctas` CTAs, spread evenly.  Measured with 8192
// tokens of 64 heads, CTAs an SM: 4 45.6 us, 8 44.0, 16 42.1, 24 42.2, 48 48.9.
int rope_heads(long long groups, int all, long long ctas) {
  const long long want = std::min<long long>(all, std::max(1LL, groups * all / ctas));
  const long long parts = (all + want - 1) / want;
  return (int)((all + parts - 1) / parts);
}

cudaError_t launch_rope(int d, int f32, const RopeParams& p, int interleaved, int sms, cudaStream_t stream) {
  if (d == 128)
    return f32 ? launch<float, 128>(p, interleaved, sms, stream) : launch<uint16_t, 128>(p, interleaved, sms, stream);
  return f32 ? launch<float, 64>(p, interleaved, sms, stream) : launch<uint16_t, 64>(p, interleaved, sms, stream);
}

}  // namespace attn
