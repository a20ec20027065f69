// paged_api.cu -- entry points of the paged 8-bit key/value cache declared in
// include/attn.h: argument checks, tensor maps, launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "checks.h"
#include "kernels.h"
#include "paged.cuh"

namespace {

using attn::aligned;
using attn::any_overlap;
using attn::Span;

// log2 of a supported page size, else -1.
int page_log2(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
  }
  return -1;
}

constexpr unsigned long long kMostWaitNs = 4000000000ull;  // the paged kernels' waits count 32 bits of nanoseconds
constexpr int kMaxRequests = 16384;  // the attention's table of sums holds as many

// Checks shared by the calls that take pages.
attn_status check_cache(const void* kp, const float* ks, const void* vp, const float* vs, int Hkv, int d,
                        int num_pages, int page_size) {
  if (!kp || !ks || !vp || !vs) return ATTN_ERR_INVALID_ARG;
  if (!aligned(kp, 16) || !aligned(vp, 16) || !aligned(ks, 4) || !aligned(vs, 4)) return ATTN_ERR_INVALID_ARG;
  if (Hkv < 1 || d < 1 || num_pages < 1 || page_size < 1) return ATTN_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || page_log2(page_size) < 0) return ATTN_ERR_UNSUPPORTED;
  // K's and V's heads are a grid dimension, (page, head) a 31-bit tensor coordinate.
  if (Hkv > 32767 || (long long)num_pages * Hkv > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Tokens of `heads` rows of d elements, `stride` elements apart.
bool token_stride_ok(long long stride, long long heads, int d) { return stride >= heads * d && stride % 8 == 0; }

// Which kernels a call runs, by T, R and G: the host does not know the requests'
// rows.  A decoding step (T <= R: on average a token a request at most) with
// groups of up to eight heads runs the eight-row kernel alone, whatever the
// requests' rows are: mostly a launch for wider ones would find nothing to do.
// Where it would, a tall request among idle ones is slow: 128 tokens against
// 4000 keys, 32/8 heads, d = 128, 60.5 us in 256 slots and 35.0 in 101 (500 keys:
// 21.7 and 27.1).  Groups above eight heads always take the other way: 64
// requests of 4096 keys with 16 heads a kv head 115 us (81 by their bytes), four
// of 700 keys 14.8.  Any other call runs the 16-row kernel for the requests with
// up to kNarrowMost query rows of a kv head and the 256-row kernel for the
// rest.  Measured with 16 requests of 4096 keys, 8 kv heads, d = 128: 32 rows
// 66 us by two tiles of 16 and 69 us by a tile of 256, 48 rows 94 and 70 us.
// A single request runs one of the two only: the wide one if T has more rows than
// that, even if the request turns out to have fewer.
constexpr int kNarrowMost = 32;
bool runs_wide(int R, int T, int G) { return T > R || G > 8; }
// CTAs of a cluster for every item of a decoding step, whose sums then meet in
// shared memory, or 0: the workers' equal ranges and the merge.  Items are tiles
// of eight rows, and no more than T * Hkv of them as G <= 8.  Clusters where all
// are resident at once (from 7/8 of the workers on they are not: GPCs leave
// holes) and where the table is too narrow for a CTA to get more than eight
// units (its width is all that the host knows of the lengths: four requests of
// 700 keys 7.4 us, with a table of 32768 keys a request 10.1).  Measured against the ranges, us, 8 kv heads, d = 128, requests of 700 /
// 4096 / 8192 keys each: clusters of 8, two requests 7.1 / 9.7 / 13.8 against
// 9.8 / 13.2 / 15.0, six 7.8 / 12.1 / 20.0 against 10.3 / 14.8 / 23.9, one of
// 16384 keys (beyond the rule) 19.0 against 15.8; clusters of 4, twelve 9.5 / 19.8 / - against
// 11.1 / 23.5; fourteen (448 CTAs) 15.4 / 34.3 against 11.3 / 26.5.
int split_of(int T, int Hkv, long long keys, int workers) {
  for (int s = 8; s >= 4; s /= 2)
    if ((long long)T * Hkv * s * 7 <= 6LL * workers && keys <= 1024 * s) return s;
  return 0;
}
// Workspace: partial sums (O, then maxima and sums, then merge descriptors) of
// every worker, two slots each.
int workers_of(int rows, int sms) { return sms * attn::paged_ctas(rows); }
size_t part_o_bytes(int rows, int d, int sms) { return (size_t)workers_of(rows, sms) * 2 * rows * d * 4; }
size_t part_ml_bytes(int rows, int sms) { return (size_t)workers_of(rows, sms) * 2 * rows * 8; }
size_t part_bytes(int rows, int d, int sms) {
  return part_o_bytes(rows, d, sms) + part_ml_bytes(rows, sms) +
         ((size_t)workers_of(rows, sms) * 32 + 255) / 256 * 256;
}
size_t workspace_bytes_for(bool wide, int d, int sms) {
  return wide ? part_bytes(16, d, sms) + part_bytes(attn::kPagedWideRows, d, sms) : part_bytes(8, d, sms);
}
// The partial sums of tiles of `rows` rows at `ws`.
void place(attn::PagedFwdParams& p, uint8_t* ws, int rows, int d, int sms) {
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + part_o_bytes(rows, d, sms));
  p.desc = reinterpret_cast<int*>(ws + part_o_bytes(rows, d, sms) + part_ml_bytes(rows, sms));
}

// Diagnostic: one warp waits, as the paged kernels do, on an mbarrier that is never completed.
__global__ void selftest_paged_wait_kernel(int* status, uint32_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    attn::mbar_init(attn::smem_u32(&bar), 1);
    abort_flag = 0;
    attn::fence_mbar_init();
  }
  __syncthreads();
  const attn::paged::Waits w{&abort_flag, limit_ns};
  const bool got = attn::paged::wait_bar(attn::smem_u32(&bar), 0, w);
  if (!got && threadIdx.x == 0 && *w.abort_flag) atomicCAS(status, attn::kDevOk, attn::kDevTimeout);
}

int sms_or_default() {
  const int n = attn::device_sms();
  return n > 0 ? n : 152;
}

// Checks of an append and its parameters (T may be 0: K, V and slots are then not read).
attn_status append_params(const void* K, long long k_stride, const void* V, long long v_stride, const int64_t* slots,
                          void* k_pages, float* k_scale, void* v_pages, float* v_scale, int T, int Hkv, int d,
                          int num_pages, int page_size, attn::KvAppendParams& p) {
  attn_status st = check_cache(k_pages, k_scale, v_pages, v_scale, Hkv, d, num_pages, page_size);
  if (st != ATTN_OK) return st;
  if (T < 0) return ATTN_ERR_INVALID_ARG;
  if (T == 0) return ATTN_OK;
  if (!K || !V || !slots) return ATTN_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 8)) return ATTN_ERR_INVALID_ARG;
  if (!token_stride_ok(k_stride, Hkv, d) || !token_stride_ok(v_stride, Hkv, d)) return ATTN_ERR_INVALID_ARG;
  // No updated array may be another array of the call.
  const size_t codes = (size_t)num_pages * Hkv * page_size * d, scales = (size_t)num_pages * Hkv * 4;
  const Span all[] = {{k_pages, codes}, {v_pages, codes}, {k_scale, scales}, {v_scale, scales}, {slots, (size_t)T * 8},
                      {K, ((size_t)(T - 1) * k_stride + (size_t)Hkv * d) * 2},
                      {V, ((size_t)(T - 1) * v_stride + (size_t)Hkv * d) * 2}};
  if (any_overlap(all, 4, 7)) return ATTN_ERR_INVALID_ARG;
  p.K = static_cast<const uint16_t*>(K);
  p.V = static_cast<const uint16_t*>(V);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = reinterpret_cast<const long long*>(slots);
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  if (attn::kDebugChecks && !(p.status = attn::device_status_word())) return ATTN_ERR_CUDA;
  p.T = T;
  p.Hkv = Hkv;
  p.num_pages = num_pages;
  p.page_log2 = page_log2(page_size);
  return ATTN_OK;
}

}  // namespace

extern "C" {

attn_status attn_kv_tables(const int32_t* cached, const int32_t* added, const int32_t* free_pages, int n_free,
                           int32_t* block_table, int max_pages, int page_size, int32_t* kv_lens,
                           int32_t* cu_tokens, int64_t* slots, int32_t* positions, int32_t* taken, int R, int T,
                           void* stream) {
  if (!cached || !added || !block_table || !kv_lens || !cu_tokens || !taken) return ATTN_ERR_INVALID_ARG;
  if (R < 1 || T < 0 || n_free < 0 || max_pages < 1 || page_size < 1) return ATTN_ERR_INVALID_ARG;
  if ((n_free > 0 && !free_pages) || (T > 0 && (!slots || !positions))) return ATTN_ERR_INVALID_ARG;
  const void* words[] = {cached, added, free_pages, block_table, kv_lens, cu_tokens, positions, taken};
  for (const void* q : words)
    if (!aligned(q, 4)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return ATTN_ERR_INVALID_ARG;
  const int pl = page_log2(page_size);
  if (pl < 0 || (long long)max_pages * page_size > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  // The kernel's sums saturate at 2^31 - 1, which has to exceed both limits.
  if (T >= 0x7fffffff || n_free >= 0x7fffffff) return ATTN_ERR_UNSUPPORTED;
  // Every CTA reads all lengths and the table while others write: no output may be an input or another output.
  const Span all[] = {{kv_lens, (size_t)R * 4}, {cu_tokens, (size_t)R * 4 + 4}, {slots, (size_t)T * 8},
                      {positions, (size_t)T * 4}, {taken, 8}, {block_table, (size_t)R * max_pages * 4},
                      {cached, (size_t)R * 4}, {added, (size_t)R * 4}, {free_pages, (size_t)n_free * 4}};
  if (any_overlap(all, 6, 9)) return ATTN_ERR_INVALID_ARG;
  attn::KvTablesParams p{};
  p.cached = cached;
  p.added = added;
  p.free_pages = free_pages;
  p.block_table = block_table;
  p.kv_lens = kv_lens;
  p.cu_tokens = cu_tokens;
  p.slots = reinterpret_cast<long long*>(slots);
  p.positions = positions;
  p.taken = taken;
  if (attn::kDebugChecks && !(p.status = attn::device_status_word())) return ATTN_ERR_CUDA;
  p.R = R;
  p.n_free = n_free;
  p.max_pages = max_pages;
  p.page_log2 = pl;
  p.T = T;
  cudaError_t e = attn::launch_kv_tables(p, sms_or_default(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_kv_append_fp8(const void* K, long long k_stride, const void* V, long long v_stride,
                               const int64_t* slots, void* k_pages, float* k_scale, void* v_pages, float* v_scale,
                               int T, int Hkv, int d, int num_pages, int page_size, void* stream) {
  attn::KvAppendParams p{};
  attn_status st = append_params(K, k_stride, V, v_stride, slots, k_pages, k_scale, v_pages, v_scale, T, Hkv, d, num_pages,
                                 page_size, p);
  if (st != ATTN_OK || T == 0) return st;
  cudaError_t e = attn::launch_kv_append(d, p, sms_or_default(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_kv_append_rope_fp8(const void* Q, long long q_stride, const void* K, long long k_stride, const void* V,
                                    long long v_stride, const int32_t* positions, const int64_t* slots,
                                    const uint64_t* freqs, int rot, int interleaved, float amplitude, void* Q_out,
                                    long long q_out_stride, void* k_pages, float* k_scale, void* v_pages, float* v_scale,
                                    int T, int Hq, int Hkv, int d, int num_pages, int page_size, void* stream) {
  attn::KvAppendParams p{};
  attn_status st = append_params(K, k_stride, V, v_stride, slots, k_pages, k_scale, v_pages, v_scale, T, Hkv, d, num_pages,
                                 page_size, p);
  if (st != ATTN_OK) return st;
  if (Hq < 1 || rot < 1 || rot > d || (interleaved != 0 && interleaved != 1) || !std::isfinite(amplitude) || !(amplitude > 0.f))
    return ATTN_ERR_INVALID_ARG;
  if (rot % 16 != 0 || Hq > 65535) return ATTN_ERR_UNSUPPORTED;
  if (T == 0) return ATTN_OK;
  if (!Q || !Q_out || !positions || !freqs) return ATTN_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(Q_out, 16) || !aligned(positions, 4) || !aligned(freqs, 8)) return ATTN_ERR_INVALID_ARG;
  if (!token_stride_ok(q_stride, Hq, d) || !token_stride_ok(q_out_stride, Hq, d)) return ATTN_ERR_INVALID_ARG;
  // Q_out may be Q, or lie between K's and V's rows in a packed projection; what is
  // written may be no other array of the call.
  const attn::Rows q(Q, 1, Hq, T, 0, d, q_stride, d, 2), qo(Q_out, 1, Hq, T, 0, d, q_out_stride, d, 2);
  const attn::Rows k(K, 1, Hkv, T, 0, d, k_stride, d, 2), v(V, 1, Hkv, T, 0, d, v_stride, d, 2);
  if (!(qo.same(q) || apart(qo, q)) || !apart(qo, k) || !apart(qo, v)) return ATTN_ERR_INVALID_ARG;
  const size_t codes = (size_t)num_pages * Hkv * page_size * d, scales = (size_t)num_pages * Hkv * 4;
  const Span written[] = {qo.span(), {k_pages, codes}, {v_pages, codes}, {k_scale, scales}, {v_scale, scales}};
  const Span read[] = {{positions, (size_t)T * 4}, {freqs, (size_t)rot * 4}};
  for (int i = 0; i < 5; ++i) {
    if (overlap(written[i], read[0]) || overlap(written[i], read[1])) return ATTN_ERR_INVALID_ARG;
    if (i > 0 && (overlap(written[i], qo.span()) || overlap(written[i], q.span()))) return ATTN_ERR_INVALID_ARG;
  }
  if (overlap({slots, (size_t)T * 8}, qo.span())) return ATTN_ERR_INVALID_ARG;
  attn::RopeParams r{};
  r.q = {Q, 0, d, q_stride, Q_out, 0, d, q_out_stride};
  r.positions = positions;
  r.freqs = freqs;
  r.amplitude = r.sine = amplitude;
  r.rot = rot;
  r.B = 1;
  r.N = T;
  r.Hq = Hq;
  r.status = p.status;
  cudaError_t e = attn::launch_kv_append_rope(d, p, r, interleaved, sms_or_default(), static_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return ATTN_ERR_UNSUPPORTED;
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_fwd_paged_workspace_size(int R, int T, int Hq, int Hkv, int d) {
  if (R < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
  return workspace_bytes_for(runs_wide(R, T, Hq / Hkv), d, sms_or_default());
}

attn_status attn_fwd_paged_fp8(const void* Q, long long q_stride, const void* k_pages, const float* k_scale,
                               const void* v_pages, const float* v_scale, const int32_t* block_table,
                               const int32_t* cu_q, const int32_t* kv_lens, void* O, float* LSE, int R, int T, int Hq,
                               int Hkv, int d, int num_pages, int page_size, int max_pages, float scale, int causal,
                               attn_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  attn_status st = check_cache(k_pages, k_scale, v_pages, v_scale, Hkv, d, num_pages, page_size);
  if (st != ATTN_OK) return st;
  if (!block_table || !cu_q || !kv_lens) return ATTN_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4)) return ATTN_ERR_INVALID_ARG;
  if (out_dtype != ATTN_BF16 && out_dtype != ATTN_F32) return ATTN_ERR_INVALID_ARG;
  if (R < 1 || T < 0 || Hq < 1 || Hq % Hkv != 0 || max_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f) || (causal != 0 && causal != 1)) return ATTN_ERR_INVALID_ARG;
  if (T == 0) return ATTN_OK;
  if (!Q || !O || !LSE || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4) || !aligned(workspace, 256)) return ATTN_ERR_INVALID_ARG;
  if (!token_stride_ok(q_stride, Hq, d)) return ATTN_ERR_INVALID_ARG;
  if (R > kMaxRequests || (long long)T * Hq > 0x7fffff00LL || (long long)max_pages * page_size > 0x7fffff00LL)
    return ATTN_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  const bool wide = runs_wide(R, T, G);
  const size_t need = workspace_bytes_for(wide, d, sms_or_default());
  if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
  // What is written may be no other array of the call: others still read.
  const size_t codes = (size_t)num_pages * Hkv * page_size * d, scales = (size_t)num_pages * Hkv * 4;
  const Span all[] = {{O, (size_t)T * Hq * d * (out_dtype == ATTN_F32 ? 4 : 2)}, {LSE, (size_t)T * Hq * 4},
                      {workspace, need}, {Q, ((size_t)(T - 1) * q_stride + (size_t)Hq * d) * 2}, {k_pages, codes},
                      {v_pages, codes}, {k_scale, scales}, {v_scale, scales},
                      {block_table, (size_t)R * max_pages * 4}, {cu_q, (size_t)R * 4 + 4}, {kv_lens, (size_t)R * 4}};
  if (any_overlap(all, 3, 11)) return ATTN_ERR_INVALID_ARG;
  const int sms = attn::device_sms();
  int* status = attn::device_status_word();
  if (sms < 1 || !status) return ATTN_ERR_CUDA;
  CUtensorMap tk, tv;
  const long long planes = (long long)num_pages * Hkv;
  if (!attn::make_page_map(&tk, k_pages, planes, page_size, d) ||
      !attn::make_page_map(&tv, v_pages, planes, page_size, d))
    return ATTN_ERR_CUDA;
  attn::PagedFwdParams p{};
  p.Q = static_cast<const uint16_t*>(Q);
  p.q_stride = q_stride;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.v_pages = static_cast<const uint8_t*>(v_pages);
  p.block_table = block_table;
  p.cu_q = cu_q;
  p.kv_lens = kv_lens;
  p.O = O;
  p.LSE = LSE;
  p.status = status;
  p.R = R;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.num_pages = num_pages;
  p.page_log2 = page_log2(page_size);
  p.max_pages = max_pages;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = causal;
  p.out_f32 = out_dtype == ATTN_F32;
  p.wait_limit_ns = std::min(attn::device_wait_limit(), kMostWaitNs);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int rows = wide ? 16 : 8;
  const bool big = wide && (long long)T * G > kNarrowMost, small = !wide || (G <= kNarrowMost && !(big && R == 1));
  attn::PagedFwdParams pw = p;
  place(p, ws, rows, d, sms);
  p.behind = big;
  p.rows_min = 0;
  p.rows_max = wide ? kNarrowMost : 0x7fffffff;
  place(pw, ws + part_bytes(rows, d, sms), attn::kPagedWideRows, d, sms);
  pw.rows_min = small ? kNarrowMost : 0;
  pw.rows_max = 0x7fffffff;
  cudaError_t e = cudaSuccess;
  const int wide_rows = attn::kPagedWideRows, w1 = workers_of(rows, sms), w2 = workers_of(wide_rows, sms);
  const int split = wide ? 0 : split_of(T, Hkv, (long long)max_pages * page_size, w1);
  if (split) {
    e = attn::launch_paged_narrow(d, rows, tk, tv, p, T * Hkv * split, split, cs);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }
  if (big) e = attn::launch_paged_wide(d, tk, tv, pw, w2, cs);
  if (e == cudaSuccess && small) e = attn::launch_paged_narrow(d, rows, tk, tv, p, w1, 0, cs);
  if (e == cudaSuccess)
    e = small ? attn::launch_paged_merge(d, p, rows, w1, big ? &pw : nullptr, wide_rows, big ? w2 : 0, cs)
              : attn::launch_paged_merge(d, pw, wide_rows, w2, nullptr, 0, 0, cs);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_selftest_paged_wait_timeout(unsigned long long limit_ns, void* stream) {
  if (limit_ns == 0 || limit_ns > 1000000000ull) return ATTN_ERR_INVALID_ARG;
  int* status = attn::device_status_word();
  if (!status) return ATTN_ERR_CUDA;
  selftest_paged_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(status, (uint32_t)limit_ns);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
