// rope_api.cu -- entry points of the rotary positions declared in
// include/attn.h: frequencies, argument checks, launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "checks.h"
#include "kernels.h"
#include "ptx.cuh"

namespace {

using attn::aligned;
using attn::Rows;

Rows rows_of(const attn_rows& r, int B, int H, int N, int d, int size) {
  return Rows(r.data, B, H, N, r.batch, r.head, r.token, d, size);
}
attn::RopeRows both(const Rows& in, const Rows& out) {
  return {in.p,         in.stride[0],  in.stride[1],  in.stride[2], const_cast<void*>(out.p),
          out.stride[0], out.stride[1], out.stride[2]};
}

attn_status run(const attn_rows* Q, const attn_rows* K, const attn_rows* Qo, const attn_rows* Ko,
                const int32_t* positions, long long positions_batch, const uint64_t* freqs, int rot, int interleaved,
                float amplitude, float direction, int B, int Hq, int Hkv, int N, int d, attn_dtype dtype, void* stream) {
  if (!Q || !Qo || !freqs || (K == nullptr) != (Ko == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || N < 0 || d < 1 || rot < 1 || Hkv < (K ? 1 : 0)) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_BF16 && dtype != ATTN_F32) return ATTN_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || !std::isfinite(amplitude) || !(amplitude > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (rot > d || positions_batch < 0 || !aligned(positions, 4) || !aligned(freqs, 8)) return ATTN_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || rot % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  const int heads = K ? Hkv : 0, size = dtype == ATTN_F32 ? 4 : 2;
  // Tokens and heads are grid dimensions, the latter in single ones at most.
  if ((long long)B * N > 0x7fffffffLL || (long long)Hq + heads > 65535) return ATTN_ERR_UNSUPPORTED;
  if (N == 0) return ATTN_OK;
  const Rows q = rows_of(*Q, B, Hq, N, d, size), qo = rows_of(*Qo, B, Hq, N, d, size);
  const Rows k = rows_of(K ? *K : *Q, B, K ? Hkv : Hq, N, d, size), ko = rows_of(K ? *Ko : *Qo, B, K ? Hkv : Hq, N, d, size);
  for (const Rows* r : {&q, &qo, &k, &ko})
    if (!r->p || !aligned(r->p, 16) || !r->strides_ok()) return ATTN_ERR_INVALID_ARG;
  if (!qo.distinct() || !ko.distinct()) return ATTN_ERR_INVALID_ARG;
  // An output may be its own input; over anything else of the call it may not lie.
  if (!(qo.same(q) || apart(qo, q))) return ATTN_ERR_INVALID_ARG;
  if (K && (!(ko.same(k) || apart(ko, k)) || !apart(qo, k) || !apart(ko, q) || !apart(qo, ko))) return ATTN_ERR_INVALID_ARG;
  const attn::Span small[] = {{positions, positions ? ((size_t)(B - 1) * (size_t)positions_batch + (size_t)N) * 4 : 0},
                              {freqs, (size_t)rot * 4}};
  for (const attn::Span& s : small)
    if (overlap(s, qo.span()) || overlap(s, ko.span())) return ATTN_ERR_INVALID_ARG;
  attn::RopeParams p{};
  p.q = both(q, qo);
  p.k = both(k, ko);
  p.positions = positions;
  p.pos_batch = positions_batch;
  p.freqs = freqs;
  p.amplitude = amplitude;
  p.sine = direction * amplitude;
  p.rot = rot;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = heads;
  if (attn::kDebugChecks && !(p.status = attn::device_status_word())) return ATTN_ERR_CUDA;
  const int sms = attn::device_sms();
  cudaError_t e = attn::launch_rope(d, dtype == ATTN_F32, p, interleaved, sms > 0 ? sms : 152, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status attn_rope_freqs(uint64_t* freqs, double* amplitude, int rot, double base, attn_rope_scaling scaling,
                            double factor, double original_len, double low, double high) {
  if (!freqs || !amplitude || rot < 1 || !std::isfinite(base) || !(base > 1.0)) return ATTN_ERR_INVALID_ARG;
  if (scaling != ATTN_ROPE_NONE && scaling != ATTN_ROPE_LINEAR && scaling != ATTN_ROPE_BASE && scaling != ATTN_ROPE_PARTS)
    return ATTN_ERR_INVALID_ARG;
  if (rot % 2 != 0 || rot > 1024) return ATTN_ERR_UNSUPPORTED;
  if (scaling != ATTN_ROPE_NONE && (!std::isfinite(factor) || !(factor >= 1.0))) return ATTN_ERR_INVALID_ARG;
  if (scaling == ATTN_ROPE_BASE && rot == 2) return ATTN_ERR_INVALID_ARG;  // a single pair has no base
  if (scaling == ATTN_ROPE_PARTS && (!std::isfinite(original_len) || !(original_len > 0.0) || !std::isfinite(low) ||
                                     !std::isfinite(high) || !(low >= 0.0) || !(high > low)))
    return ATTN_ERR_INVALID_ARG;
  if (scaling == ATTN_ROPE_BASE) base *= std::pow(factor, (double)rot / (rot - 2));
  const double turn = 6.283185307179586476925286766559;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot) / turn;
    if (scaling == ATTN_ROPE_LINEAR) f /= factor;
    if (scaling == ATTN_ROPE_PARTS) {
      const double keep = std::min(1.0, std::max(0.0, (f * original_len - low) / (high - low)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    freqs[i] = (uint64_t)std::llround(std::ldexp(f, 64));  // f < 1 / (2 pi): below 2^62
  }
  *amplitude = scaling == ATTN_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return ATTN_OK;
}

attn_status attn_rope(const attn_rows* Q, const attn_rows* K, const attn_rows* Q_out, const attn_rows* K_out,
                      const int32_t* positions, long long positions_batch, const uint64_t* freqs, int rot,
                      int interleaved, float amplitude, int B, int Hq, int Hkv, int N, int d, attn_dtype dtype,
                      void* stream) {
  return run(Q, K, Q_out, K_out, positions, positions_batch, freqs, rot, interleaved, amplitude, 1.f, B, Hq, Hkv, N, d,
             dtype, stream);
}

attn_status attn_rope_bwd(const attn_rows* dQ, const attn_rows* dK, const attn_rows* dQ_out, const attn_rows* dK_out,
                          const int32_t* positions, long long positions_batch, const uint64_t* freqs, int rot,
                          int interleaved, float amplitude, int B, int Hq, int Hkv, int N, int d, attn_dtype dtype,
                          void* stream) {
  return run(dQ, dK, dQ_out, dK_out, positions, positions_batch, freqs, rot, interleaved, amplitude, -1.f, B, Hq, Hkv, N,
             d, dtype, stream);
}

}  // extern "C"
