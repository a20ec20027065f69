// rope.cu -- rotary positions of queries and keys, and their gradient (rope.cuh
// has the mathematics).
#include <algorithm>

#include "launch.cuh"
#include "rope.cuh"

namespace attn {
namespace {

template <class T, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int heads) {
  griddep_wait();
  rope_block<T, D, INTER>(p, blockIdx.x, blockIdx.y * heads, heads);
}

template <class T, int D>
cudaError_t launch(const RopeParams& p, int interleaved, int sms, cudaStream_t stream) {
  const long long groups = ((long long)p.B * p.N + rope_tokens(D) - 1) / rope_tokens(D);
  const int heads = rope_heads(groups, p.Hq + p.Hkv, sms);
  const dim3 grid((unsigned)groups, (unsigned)((p.Hq + p.Hkv + heads - 1) / heads));
  return interleaved ? launch_behind(rope_kernel<T, D, true>, grid, kRopeThreads, stream, p, heads)
                     : launch_behind(rope_kernel<T, D, false>, grid, kRopeThreads, stream, p, heads);
}

}  // namespace

// Heads of a CTA: as many as leave eight CTAs for every SM, in fours.
int rope_heads(long long groups, int all, int sms) {
  const long long want = groups * all / (8LL * sms);
  return want < 2 ? 1 : (int)std::min<long long>(all, want < 4 ? want : want / 4 * 4);
}

cudaError_t launch_rope(int d, int f32, const RopeParams& p, int interleaved, int sms, cudaStream_t stream) {
  if (d == 128)
    return f32 ? launch<float, 128>(p, interleaved, sms, stream) : launch<uint16_t, 128>(p, interleaved, sms, stream);
  return f32 ? launch<float, 64>(p, interleaved, sms, stream) : launch<uint16_t, 64>(p, interleaved, sms, stream);
}

}  // namespace attn
