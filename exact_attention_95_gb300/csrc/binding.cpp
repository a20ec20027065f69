// binding.cpp -- the Python calls of the paged 8-bit cache, of rotary positions and of
// attention with dropout without Python's share of the work.
//
// A decoding step makes these calls once a layer around kernels of a few
// microseconds; checks, allocations and pointer passing in Python take three
// times as long as the kernels.  The functions below take the arguments of the
// package's functions of the same names, positionally.  They return the
// outputs, the library's status as an int where a call fails, or None where an
// argument is not as it has to be (or a stream is named): the package's own
// checks then word the error.  Without the module (a host that cannot build it, one
// built for another Python or PyTorch) the package's own checks make the calls.
// The library is reached through the addresses that bind() is given, so whichever
// build of it is loaded is used.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <exception>

#include "../../include/attn.h"

namespace {

decltype(&attn_kv_tables) g_tables = nullptr;
decltype(&attn_kv_append_fp8) g_append = nullptr;
decltype(&attn_fwd_paged_fp8) g_fwd = nullptr;
decltype(&attn_fwd_paged_workspace_size) g_workspace = nullptr;
decltype(&attn_rope) g_rope[2] = {nullptr, nullptr};  // forward, gradient
decltype(&attn_kv_append_rope_fp8) g_append_rope = nullptr;
decltype(&attn_fwd_dropout) g_fwd_dropout = nullptr;
decltype(&attn_bwd_dropout) g_bwd_dropout = nullptr;
decltype(&attn_bwd_dropout_workspace_size) g_bwd_workspace = nullptr;

// The tensor of an argument, or null.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A contiguous CUDA tensor of this type, shape and device.
bool is(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  return t && t->scalar_type() == type && t->device() == device && t->sizes() == shape && t->is_contiguous();
}
// A bf16 [T, heads, d] tensor whose tokens may be apart: elements between tokens, or -1.
long long token_stride(const at::Tensor* t, int64_t heads, int64_t d, at::Device device) {
  if (!t || t->scalar_type() != at::kBFloat16 || t->device() != device || t->dim() != 3 || t->size(1) != heads ||
      t->size(2) != d)
    return -1;
  const int64_t apart = t->size(0) > 1 ? t->stride(0) : heads * d;
  if (t->stride(2) != 1 || (heads > 1 && t->stride(1) != d) || apart < heads * d || apart % 8) return -1;
  return apart;
}
bool small_int(PyObject* o, long long lo, long long hi, int& out) {
  if (!PyLong_Check(o)) return false;
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (overflow || v < lo || v > hi) return false;
  out = (int)v;
  return true;
}
bool fits(int64_t v) { return v >= 0 && v <= 0x7fffffff; }

// New device memory on the current device and stream, from torch's allocator.
// Called directly: the dispatcher's code on the way to an at::empty, cold after
// a kernel launch, takes longer than the allocation.
at::Storage memory(size_t bytes) {
  c10::Allocator* from = c10::cuda::CUDACachingAllocator::get();
  return at::Storage(c10::make_intrusive<c10::StorageImpl>(c10::StorageImpl::use_byte_size_t(), bytes,
                                                           from->allocate(bytes), from, /*resizable=*/true));
}
// A contiguous tensor of this type and shape in it, from element `first` (of this type) on.
at::Tensor part_of(at::Storage s, at::ScalarType type, int64_t first, at::IntArrayRef shape) {
  at::Tensor v = at::detail::make_tensor<c10::TensorImpl>(std::move(s), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                          c10::scalarTypeToTypeMeta(type));
  v.unsafeGetTensorImpl()->set_storage_offset(first);
  v.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return v;
}
// A tensor with a storage of its own.
at::Tensor fresh(at::ScalarType type, at::IntArrayRef shape) {
  size_t bytes = c10::elementSize(type);
  for (const int64_t n : shape) bytes *= (size_t)n;
  return part_of(memory(bytes), type, 0, shape);
}
// An output: the caller's if it is as it has to be, a new one for None (`device` is the current one).
bool output(PyObject* o, at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, at::Device device) {
  if (o == Py_None) {
    t = fresh(type, shape);
    return true;
  }
  const at::Tensor* given = tensor(o);
  if (!is(given, type, shape, device)) return false;
  t = *given;
  return true;
}
// Sets the device, where it is another one, for as long as this lives.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(at::Device d) {
    if (c10::cuda::current_device() != d.index()) guard.set_device(d);
  }
};
PyObject* wrap(PyObject* given, at::Tensor& t) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(std::move(t));
}

// Pages and scales of a cache.
struct Cache {
  const at::Tensor *kp, *ks, *vp, *vs;
  int64_t num_pages, Hkv, page, d;
  bool read(PyObject* const* a, at::Device device) {
    kp = tensor(a[0]);
    ks = tensor(a[1]);
    vp = tensor(a[2]);
    vs = tensor(a[3]);
    if (!kp || kp->dim() != 4) return false;
    num_pages = kp->size(0);
    Hkv = kp->size(1);
    page = kp->size(2);
    d = kp->size(3);
    return fits(num_pages) && fits(Hkv) && fits(page) && fits(d) && is(kp, at::kByte, kp->sizes(), device) &&
           is(vp, at::kByte, kp->sizes(), device) && is(ks, at::kFloat, {num_pages, Hkv}, device) &&
           is(vs, at::kFloat, {num_pages, Hkv}, device);
  }
};

// The call on the device's current stream, without Python's lock (it throws nothing).
template <class F>
int without_lock(at::Device device, F call) {
  void* const stream = (void*)c10::cuda::getCurrentCUDAStream(device.index()).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = call(stream);
  Py_END_ALLOW_THREADS;
  return rc;
}
// A tuple of new references.
template <class... P>
PyObject* tuple(P*... items) {
  PyObject* t = PyTuple_New(sizeof...(P));
  Py_ssize_t i = 0;
  if (t) (PyTuple_SET_ITEM(t, i++, items), ...);
  return t;
}

// What PyTorch throws is raised as its own calls raise it (an allocation that fails is
// torch.OutOfMemoryError).
#define ATTN_GUARD(...)                                             \
  try {                                                             \
    __VA_ARGS__                                                     \
  } catch (const std::exception&) {                                 \
    torch::translate_exception_to_python(std::current_exception()); \
    return nullptr;                                                 \
  }

// cached, added, free_pages, block_table, page_size, T, kv_lens, cu_tokens, slots, positions, taken
PyObject* kv_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  ATTN_GUARD(
    if (n != 11) Py_RETURN_NONE;
    const at::Tensor *cached = tensor(a[0]), *added = tensor(a[1]), *free_pages = tensor(a[2]), *table = tensor(a[3]);
    int page = 0, T = 0;
    if (!cached || !cached->is_cuda() || !table || table->dim() != 2 || !free_pages || free_pages->dim() != 1 ||
        !small_int(a[4], 0, 0x7fffffff, page) || !small_int(a[5], 0, 0x7fffffff, T))
      Py_RETURN_NONE;
    const at::Device dev = cached->device();
    const int64_t R = table->size(0), width = table->size(1), F = free_pages->size(0);
    if (!fits(R) || !fits(width) || !fits(F) || !is(cached, at::kInt, {R}, dev) || !is(added, at::kInt, {R}, dev) ||
        !is(free_pages, at::kInt, {F}, dev) || !is(table, at::kInt, {R, width}, dev))
      Py_RETURN_NONE;
    const OnDevice on(dev);
    at::Tensor lens, cu, slots, positions, taken;
    if (a[6] == Py_None && a[7] == Py_None && a[10] == Py_None) {
      // The small ones in one allocation: each takes 0.35 us of a call.  (The arrays of
      // the tokens have their own: who keeps `taken` keeps no megabytes.)
      const at::Storage small = memory(4 * (size_t)(2 * R + 3));
      lens = part_of(small, at::kInt, 0, {R});
      cu = part_of(small, at::kInt, R, {R + 1});
      taken = part_of(small, at::kInt, 2 * R + 1, {2});
    } else if (!output(a[6], lens, at::kInt, {R}, dev) || !output(a[7], cu, at::kInt, {R + 1}, dev) ||
               !output(a[10], taken, at::kInt, {2}, dev)) {
      Py_RETURN_NONE;
    }
    if (!output(a[8], slots, at::kLong, {T}, dev) || !output(a[9], positions, at::kInt, {T}, dev)) Py_RETURN_NONE;
    const int rc = without_lock(dev, [&](void* stream) {
      return g_tables((const int32_t*)cached->data_ptr(), (const int32_t*)added->data_ptr(),
                      (const int32_t*)free_pages->data_ptr(), (int)F, (int32_t*)table->data_ptr(), (int)width, page,
                      (int32_t*)lens.data_ptr(), (int32_t*)cu.data_ptr(), (int64_t*)slots.data_ptr(),
                      (int32_t*)positions.data_ptr(), (int32_t*)taken.data_ptr(), (int)R, T, stream);
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    return tuple(wrap(a[6], lens), wrap(a[7], cu), wrap(a[8], slots), wrap(a[9], positions), wrap(a[10], taken));)
}

// K, V, slots, k_pages, k_scale, v_pages, v_scale
PyObject* kv_append_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  ATTN_GUARD(
    if (n != 7) Py_RETURN_NONE;
    const at::Tensor *K = tensor(a[0]), *V = tensor(a[1]), *slots = tensor(a[2]);
    Cache c;
    if (!K || !K->is_cuda() || !c.read(a + 3, K->device())) Py_RETURN_NONE;
    const at::Device dev = K->device();
    const long long ks = token_stride(K, c.Hkv, c.d, dev), vs = token_stride(V, c.Hkv, c.d, dev);
    if (ks < 0 || vs < 0 || K->size(0) != V->size(0) || !fits(K->size(0)) || !is(slots, at::kLong, {K->size(0)}, dev))
      Py_RETURN_NONE;
    const OnDevice on(dev);
    const int rc = without_lock(dev, [&](void* stream) {
      return g_append(K->data_ptr(), ks, V->data_ptr(), vs, (const int64_t*)slots->data_ptr(), c.kp->data_ptr(),
                      (float*)c.ks->data_ptr(), c.vp->data_ptr(), (float*)c.vs->data_ptr(), (int)K->size(0), (int)c.Hkv,
                      (int)c.d, (int)c.num_pages, (int)c.page, stream);
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    return PyTuple_Pack(4, a[3], a[4], a[5], a[6]);)
}

// The softmax scale: a number, or None for 1 / sqrt(d); false with Python's error set.
bool scale_of(PyObject* o, int64_t d, double& scale) {
  scale = o == Py_None ? 1.0 / std::sqrt((double)d) : PyFloat_AsDouble(o);
  return o == Py_None || !PyErr_Occurred();
}

// Q, k_pages, k_scale, v_pages, v_scale, block_table, cu_q, kv_lens, scale, causal, fp32 output, O, LSE, workspace
PyObject* fwd_paged_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  ATTN_GUARD(
    if (n != 14) Py_RETURN_NONE;
    const at::Tensor *Q = tensor(a[0]), *table = tensor(a[5]), *cu = tensor(a[6]), *lens = tensor(a[7]);
    Cache c;
    if (!Q || !Q->is_cuda() || Q->dim() != 3 || !table || table->dim() != 2 || !c.read(a + 1, Q->device()))
      Py_RETURN_NONE;
    const at::Device dev = Q->device();
    const int64_t T = Q->size(0), Hq = Q->size(1), R = table->size(0), width = table->size(1);
    const long long stride = token_stride(Q, Hq, c.d, dev);
    if (stride < 0 || !fits(T) || !fits(Hq) || !fits(R) || !fits(width) || !is(table, at::kInt, {R, width}, dev) ||
        !is(cu, at::kInt, {R + 1}, dev) || !is(lens, at::kInt, {R}, dev))
      Py_RETURN_NONE;
    double scale = 0;
    if (!scale_of(a[8], c.d, scale)) return nullptr;
    const int causal = PyObject_IsTrue(a[9]), f32 = PyObject_IsTrue(a[10]);
    if (causal < 0 || f32 < 0) return nullptr;
    const OnDevice on(dev);
    at::Tensor O, LSE;
    if (!output(a[11], O, f32 ? at::kFloat : at::kBFloat16, {T, Hq, c.d}, dev) ||
        !output(a[12], LSE, at::kFloat, {T, Hq}, dev))
      Py_RETURN_NONE;
    const size_t need = g_workspace((int)R, (int)T, (int)Hq, (int)c.Hkv, (int)c.d);
    c10::DataPtr own;  // freed at the end of this call, for later work of the same stream
    void* ws = nullptr;
    if (a[13] == Py_None) {
      own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
      ws = own.get();
    } else {
      const at::Tensor* given = tensor(a[13]);
      if (!given || !is(given, at::kByte, given->sizes(), dev) || (size_t)given->numel() < need) Py_RETURN_NONE;
      ws = given->data_ptr();
    }
    const int rc = without_lock(dev, [&](void* stream) {
      return g_fwd(Q->data_ptr(), stride, c.kp->data_ptr(), (const float*)c.ks->data_ptr(), c.vp->data_ptr(),
                   (const float*)c.vs->data_ptr(), (const int32_t*)table->data_ptr(), (const int32_t*)cu->data_ptr(),
                   (const int32_t*)lens->data_ptr(), O.data_ptr(), (float*)LSE.data_ptr(), (int)R, (int)T, (int)Hq,
                   (int)c.Hkv, (int)c.d, (int)c.num_pages, (int)c.page, (int)width, (float)scale, causal,
                   f32 ? ATTN_F32 : ATTN_BF16, ws, need, stream);
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    return tuple(wrap(a[11], O), wrap(a[12], LSE));)
}

// Rows of a [T, H, d] or [B, H, N, d] tensor.
bool rows_of(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, at::Device device, attn_rows& r) {
  if (!t || t->scalar_type() != type || t->device() != device || t->sizes() != shape) return false;
  const int64_t k = t->dim();
  if (t->size(k - 1) > 1 && t->stride(k - 1) != 1) return false;
  r.data = t->data_ptr();
  r.batch = k == 4 ? t->stride(0) : 0;
  r.head = t->stride(1);
  r.token = k == 4 ? t->stride(2) : t->stride(0);
  return true;
}
// An output of such rows: the caller's, or a new contiguous one for None.
bool rows_out(PyObject* o, at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, at::Device device, attn_rows& r) {
  if (o == Py_None)
    t = fresh(type, shape);
  else if (const at::Tensor* given = tensor(o))
    t = *given;
  else
    return false;
  return rows_of(&t, type, shape, device, r);
}
bool float_of(PyObject* o, float& v) {
  if (!PyFloat_Check(o)) return false;
  v = (float)PyFloat_AS_DOUBLE(o);
  return true;
}

// gradient, Q, K, freqs, positions, interleaved, amplitude, Q_out, K_out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  ATTN_GUARD(
    if (n != 9) Py_RETURN_NONE;
    const at::Tensor *Q = tensor(a[1]), *K = tensor(a[2]), *freqs = tensor(a[3]), *pos = tensor(a[4]);
    if (!Q || !Q->is_cuda() || (Q->dim() != 3 && Q->dim() != 4) || Q->numel() == 0 || (!K && (a[2] != Py_None || a[8] != Py_None)) ||
        (K && K->dim() != Q->dim()) || (!pos && a[4] != Py_None))
      Py_RETURN_NONE;
    const at::Device dev = Q->device();
    const at::ScalarType type = Q->scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) Py_RETURN_NONE;
    const bool tokens = Q->dim() == 3;
    const int64_t B = tokens ? 1 : Q->size(0), N = Q->size(tokens ? 0 : 2), Hq = Q->size(1), d = Q->size(tokens ? 2 : 3);
    const int64_t Hkv = K ? K->size(1) : 0;
    float amplitude = 1;
    attn_rows q, k{}, qo, ko{};
    const int64_t three[3] = {N, Hkv, d}, four[4] = {B, Hkv, N, d};
    const at::IntArrayRef k_shape = tokens ? at::IntArrayRef(three, 3) : at::IntArrayRef(four, 4);
    if (!fits(B) || !fits(N) || !fits(Hq) || !fits(Hkv) || !fits(d) || (K && Hkv == 0) || !float_of(a[6], amplitude) ||
        !rows_of(Q, type, Q->sizes(), dev, q) || (K && !rows_of(K, type, k_shape, dev, k)) || !freqs ||
        freqs->dim() != 1 || freqs->size(0) < 1 || 2 * freqs->size(0) > d || !is(freqs, at::kLong, freqs->sizes(), dev))
      Py_RETURN_NONE;
    long long pos_batch = 0;
    if (pos) {
      if (!tokens && pos->dim() == 2 ? !is(pos, at::kInt, {B, N}, dev) : !is(pos, at::kInt, {N}, dev)) Py_RETURN_NONE;
      pos_batch = pos->dim() == 2 ? N : 0;
    }
    const int gradient = PyObject_IsTrue(a[0]), pairs = PyObject_IsTrue(a[5]);
    if (gradient < 0 || pairs < 0) return nullptr;
    const OnDevice on(dev);
    at::Tensor Qo, Ko;
    if (!rows_out(a[7], Qo, type, Q->sizes(), dev, qo) || (K && !rows_out(a[8], Ko, type, k_shape, dev, ko))) Py_RETURN_NONE;
    const int rc = without_lock(dev, [&](void* stream) {
      return g_rope[gradient](&q, K ? &k : nullptr, &qo, K ? &ko : nullptr, pos ? (const int32_t*)pos->data_ptr() : nullptr,
                              pos_batch, (const uint64_t*)freqs->data_ptr(), (int)(2 * freqs->size(0)), pairs, amplitude,
                              (int)B, (int)Hq, (int)Hkv, (int)N, (int)d, type == at::kFloat ? ATTN_F32 : ATTN_BF16, stream);
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    if (!K) {
      Py_INCREF(Py_None);
      return tuple(wrap(a[7], Qo), Py_None);
    }
    return tuple(wrap(a[7], Qo), wrap(a[8], Ko));)
}

// Q, K, V, positions, slots, freqs, k_pages, k_scale, v_pages, v_scale, interleaved, amplitude, Q_out
PyObject* kv_append_rope_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  ATTN_GUARD(
    if (n != 13) Py_RETURN_NONE;
    const at::Tensor *Q = tensor(a[0]), *K = tensor(a[1]), *V = tensor(a[2]), *pos = tensor(a[3]), *slots = tensor(a[4]);
    const at::Tensor* freqs = tensor(a[5]);
    Cache c;
    float amplitude = 1;
    if (!Q || Q->dim() != 3 || !K || !K->is_cuda() || !c.read(a + 6, K->device()) || !float_of(a[11], amplitude))
      Py_RETURN_NONE;
    const at::Device dev = K->device();
    const int64_t T = K->size(0), Hq = Q->size(1);
    const long long qs = token_stride(Q, Hq, c.d, dev), ks = token_stride(K, c.Hkv, c.d, dev), vs = token_stride(V, c.Hkv, c.d, dev);
    if (qs < 0 || ks < 0 || vs < 0 || Q->size(0) != T || V->size(0) != T || !fits(T) || !fits(Hq) ||
        !is(slots, at::kLong, {T}, dev) || !is(pos, at::kInt, {T}, dev) || !freqs || freqs->dim() != 1 ||
        freqs->size(0) < 1 || 2 * freqs->size(0) > c.d || !is(freqs, at::kLong, freqs->sizes(), dev))
      Py_RETURN_NONE;
    const int pairs = PyObject_IsTrue(a[10]);
    if (pairs < 0) return nullptr;
    const OnDevice on(dev);
    at::Tensor Qo;
    if (a[12] == Py_None)
      Qo = fresh(at::kBFloat16, {T, Hq, c.d});
    else if (const at::Tensor* given = tensor(a[12]))
      Qo = *given;
    else
      Py_RETURN_NONE;
    const long long qos = token_stride(&Qo, Hq, c.d, dev);
    if (qos < 0 || Qo.size(0) != T) Py_RETURN_NONE;
    const int rc = without_lock(dev, [&](void* stream) {
      return g_append_rope(Q->data_ptr(), qs, K->data_ptr(), ks, V->data_ptr(), vs, (const int32_t*)pos->data_ptr(),
                           (const int64_t*)slots->data_ptr(), (const uint64_t*)freqs->data_ptr(),
                           (int)(2 * freqs->size(0)), pairs, amplitude, Qo.data_ptr(), qos, c.kp->data_ptr(),
                           (float*)c.ks->data_ptr(), c.vp->data_ptr(), (float*)c.vs->data_ptr(), (int)T, (int)Hq,
                           (int)c.Hkv, (int)c.d, (int)c.num_pages, (int)c.page, stream);
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    return wrap(a[12], Qo);)
}

// Sizes of Q [B, Hq, N, d] and K [B, Hkv, N, d].
struct Heads {
  int64_t B, Hq, Hkv, N, d;
  at::Device dev = at::kCPU;
  // Q, K and V (bf16, contiguous) and the generator's state.
  bool read(const at::Tensor* Q, const at::Tensor* K, const at::Tensor* V, const at::Tensor* rng) {
    if (!Q || !Q->is_cuda() || Q->dim() != 4 || !K || K->dim() != 4) return false;
    B = Q->size(0);
    Hq = Q->size(1);
    N = Q->size(2);
    d = Q->size(3);
    Hkv = K->size(1);
    dev = Q->device();
    return fits(B) && fits(Hq) && fits(Hkv) && fits(N) && fits(d) && q(Q) && kv(K) && kv(V) && is(rng, at::kLong, {2}, dev);
  }
  bool q(const at::Tensor* t) const { return is(t, at::kBFloat16, {B, Hq, N, d}, dev); }
  bool kv(const at::Tensor* t) const { return is(t, at::kBFloat16, {B, Hkv, N, d}, dev); }
};

// Q, K, V, p, rng, scale, causal, fp32 output, O, LSE
PyObject* fwd_dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  ATTN_GUARD(
    if (n != 10) Py_RETURN_NONE;
    const at::Tensor *Q = tensor(a[0]), *K = tensor(a[1]), *V = tensor(a[2]), *rng = tensor(a[4]);
    Heads s;
    float p = 0;
    double scale = 0;
    if (!s.read(Q, K, V, rng) || !float_of(a[3], p)) Py_RETURN_NONE;
    if (!scale_of(a[5], s.d, scale)) return nullptr;
    const int causal = PyObject_IsTrue(a[6]), f32 = PyObject_IsTrue(a[7]);
    if (causal < 0 || f32 < 0) return nullptr;
    const OnDevice on(s.dev);
    at::Tensor O, LSE;
    if (!output(a[8], O, f32 ? at::kFloat : at::kBFloat16, Q->sizes(), s.dev) ||
        !output(a[9], LSE, at::kFloat, {s.B, s.Hq, s.N}, s.dev))
      Py_RETURN_NONE;
    const int rc = without_lock(s.dev, [&](void* stream) {
      return g_fwd_dropout(Q->data_ptr(), K->data_ptr(), V->data_ptr(), O.data_ptr(), (float*)LSE.data_ptr(), (int)s.B,
                           (int)s.Hq, (int)s.Hkv, (int)s.N, (int)s.d, (float)scale, causal, p,
                           (const uint64_t*)rng->data_ptr(), f32 ? ATTN_F32 : ATTN_BF16, stream);
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    return tuple(wrap(a[8], O), wrap(a[9], LSE));)
}

// Q, K, V, O, dO, LSE, p, rng, scale, causal, dQ, dK, dV, workspace
PyObject* bwd_dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  ATTN_GUARD(
    if (n != 14) Py_RETURN_NONE;
    const at::Tensor *Q = tensor(a[0]), *K = tensor(a[1]), *V = tensor(a[2]), *O = tensor(a[3]), *dO = tensor(a[4]);
    const at::Tensor *LSE = tensor(a[5]), *rng = tensor(a[7]);
    Heads s;
    float p = 0;
    double scale = 0;
    if (!s.read(Q, K, V, rng) || !s.q(O) || !s.q(dO) || !is(LSE, at::kFloat, {s.B, s.Hq, s.N}, s.dev) ||
        !float_of(a[6], p))
      Py_RETURN_NONE;
    if (!scale_of(a[8], s.d, scale)) return nullptr;
    const int causal = PyObject_IsTrue(a[9]);
    if (causal < 0) return nullptr;
    const OnDevice on(s.dev);
    at::Tensor dQ, dK, dV;
    if (!output(a[10], dQ, at::kBFloat16, Q->sizes(), s.dev) || !output(a[11], dK, at::kBFloat16, K->sizes(), s.dev) ||
        !output(a[12], dV, at::kBFloat16, K->sizes(), s.dev))
      Py_RETURN_NONE;
    // (0 for sizes that the library refuses: with some workspace it says why.)
    const size_t bytes = std::max<size_t>(g_bwd_workspace((int)s.B, (int)s.Hq, (int)s.Hkv, (int)s.N, (int)s.d, causal), 1);
    c10::DataPtr own;  // freed at the end of this call, for later work of the same stream
    void* ws = nullptr;
    if (a[13] == Py_None) {
      own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
      ws = own.get();
    } else {
      const at::Tensor* given = tensor(a[13]);
      if (!given || !is(given, at::kByte, given->sizes(), s.dev) || (size_t)given->numel() < bytes) Py_RETURN_NONE;
      ws = given->data_ptr();
    }
    const int rc = without_lock(s.dev, [&](void* stream) {
      return g_bwd_dropout(Q->data_ptr(), K->data_ptr(), V->data_ptr(), O->data_ptr(), dO->data_ptr(),
                           (const float*)LSE->data_ptr(), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), (int)s.B, (int)s.Hq,
                           (int)s.Hkv, (int)s.N, (int)s.d, (float)scale, causal, p, (const uint64_t*)rng->data_ptr(), ws,
                           bytes, stream);
    });
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    return tuple(wrap(a[10], dQ), wrap(a[11], dK), wrap(a[12], dV));)
}

// bind(addresses of attn_kv_tables, attn_kv_append_fp8, attn_fwd_paged_fp8, attn_fwd_paged_workspace_size, attn_rope,
// attn_rope_bwd, attn_kv_append_rope_fp8, attn_fwd_dropout, attn_bwd_dropout, attn_bwd_dropout_workspace_size)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kAddresses = 10;
  if (n != kAddresses) {
    PyErr_SetString(PyExc_TypeError, "bind takes ten addresses");
    return nullptr;
  }
  void* p[kAddresses];
  for (int i = 0; i < kAddresses; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_tables = reinterpret_cast<decltype(g_tables)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_fwd = reinterpret_cast<decltype(g_fwd)>(p[2]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[3]);
  g_rope[0] = reinterpret_cast<decltype(&attn_rope)>(p[4]);
  g_rope[1] = reinterpret_cast<decltype(&attn_rope)>(p[5]);
  g_append_rope = reinterpret_cast<decltype(g_append_rope)>(p[6]);
  g_fwd_dropout = reinterpret_cast<decltype(g_fwd_dropout)>(p[7]);
  g_bwd_dropout = reinterpret_cast<decltype(g_bwd_dropout)>(p[8]);
  g_bwd_workspace = reinterpret_cast<decltype(g_bwd_workspace)>(p[9]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void*)F, METH_FASTCALL, ""};
}
PyMethodDef g_methods[] = {method<kv_tables>("kv_tables"), method<kv_append_fp8>("kv_append_fp8"),
                           method<fwd_paged_fp8>("fwd_paged_fp8"), method<rope>("rope"),
                           method<kv_append_rope_fp8>("kv_append_rope_fp8"), method<fwd_dropout>("fwd_dropout"),
                           method<bwd_dropout>("bwd_dropout"), method<bind>("bind"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
