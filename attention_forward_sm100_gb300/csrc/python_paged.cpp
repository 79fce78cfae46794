// Python side of the paged-cache operators (attn_paged.h): argument checks,
// output and workspace allocation, and the call into the library. Compiled
// code instead of ctypes because a decoding step is a few microseconds of GPU
// work: with the checks in Python one paged_forward call cost 28 us of host
// time on GB300's CPU, an append 15 us.
//
// Functions take positional arguments (paged.py has the public signatures and
// their documentation) and return the outputs, or the library's status as an
// int if the call was refused there. Bad arguments raise ValueError before
// anything is allocated or enqueued.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cuda_runtime_api.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <stdexcept>
#include <string>

#include "../../include/attn_paged.h"
#include "paged_host.h"

namespace {

struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};

void need(bool ok, const char* message) {
  if (!ok) throw BadArgument(message);
}
void need_f(bool ok, const char* format, ...) {
  if (ok) return;
  char text[256];
  va_list ap;
  va_start(ap, format);
  vsnprintf(text, sizeof(text), format, ap);
  va_end(ap);
  throw BadArgument(text);
}

// A tensor argument, or nothing for None.
struct Arg {
  const char* name;
  const at::Tensor* t;
  explicit operator bool() const { return t != nullptr; }
  const at::Tensor* operator->() const { return t; }
  void* ptr() const { return t != nullptr ? t->data_ptr() : nullptr; }
};

Arg tensor_or_none(const char* name, PyObject* o) {
  if (o == Py_None) return {name, nullptr};
  if (!THPVariable_Check(o)) {
    need_f(false, "%s must be a tensor", name);
  }
  return {name, &THPVariable_Unpack(o)};
}
Arg tensor(const char* name, PyObject* o) {
  const Arg a = tensor_or_none(name, o);
  need_f(bool(a), "%s must be a tensor", name);
  return a;
}
int64_t integer(const char* name, PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    need_f(false, "%s must be an integer", name);
  }
  return v;
}

// Uninitialised memory from torch's allocator (not through the dispatcher).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, c10::DeviceIndex device) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, c10::Device(c10::kCUDA, device), c10::nullopt));
}

bool is(const Arg& a, at::ScalarType t) { return a->scalar_type() == t; }

// Element stride of dimension i; 0 where the dimension has size 1 (its stride says nothing).
int64_t stride(const Arg& a, int64_t i) { return a->size(i) == 1 ? 0 : a->stride(i); }

int32_t int32(const char* what, int64_t v) {
  need_f(v >= 0 && v <= 0x7fffffffll, "%s does not fit 32 bits", what);
  return static_cast<int32_t>(v);
}

void check_int32(const Arg& a, int64_t n) {
  need_f(is(a, at::kInt) && a->is_contiguous(), "%s must be a contiguous int32 tensor", a.name);
  need_f(a->dim() == 1 && a->size(0) == n, "%s must have %lld entries", a.name, (long long)n);
}

attn_kv_cache check_cache(const Arg& k, const Arg& v, const Arg& table, const Arg& k_scale, const Arg& v_scale) {
  need(k->dim() == 4 && k->sizes() == v->sizes(), "k_cache and v_cache must be [pages, page_size, Hkv, D] of one shape");
  need(is(k, at::kBFloat16) || is(k, at::kFloat8_e4m3fn), "unsupported cache dtype (bf16 or float8_e4m3fn)");
  need(k->scalar_type() == v->scalar_type(), "k_cache and v_cache must have one dtype");
  need(k->stride(3) == 1 && v->stride(3) == 1, "the cache's depth must be contiguous");
  need(table->dim() == 2 && is(table, at::kInt), "block_table must be an int32 [B, max_pages] tensor");
  need(table->size(1) <= 1 || table->stride(1) == 1, "the rows of block_table must be contiguous");
  attn_kv_cache c = {};
  const bool fp8 = is(k, at::kFloat8_e4m3fn);
  c.num_pages = int32("pages", k->size(0));
  c.page_size = int32("page_size", k->size(1));
  c.num_heads_kv = int32("Hkv", k->size(2));
  c.head_dim = int32("D", k->size(3));
  for (const Arg* s : {&k_scale, &v_scale}) {
    if (!fp8) {
      need(!*s, "a bf16 cache takes no scales");
      continue;
    }
    need_f(bool(*s), "an e4m3 cache needs %s", s->name);
    need_f(is(*s, at::kFloat) && (*s)->is_contiguous() && (*s)->dim() == 3 && (*s)->size(0) == c.num_pages &&
               (*s)->size(1) == c.num_heads_kv && (*s)->size(2) == c.page_size,
           "%s must be a contiguous fp32 [pages, Hkv, page_size] tensor", s->name);
  }
  c.k = k.ptr();
  c.v = v.ptr();
  c.k_scale = static_cast<float*>(k_scale.ptr());
  c.v_scale = static_cast<float*>(v_scale.ptr());
  c.block_table = static_cast<const int32_t*>(table.ptr());
  for (int i = 0; i < 3; ++i) {
    c.k_stride[i] = stride(k, i);
    c.v_stride[i] = stride(v, i);
  }
  c.table_stride = stride(table, 0);
  c.dtype = fp8 ? ATTN_DTYPE_FP8_E4M3 : ATTN_DTYPE_BF16;
  c.max_pages = int32("max_pages", table->size(1));
  c.batch = int32("B", table->size(0));
  return c;
}

// The device all of them are on.
template <size_t N>
c10::DeviceIndex check_device(const std::array<Arg, N>& args) {
  int device = -1;
  for (const Arg& a : args) {
    if (!a) continue;
    need_f(a->is_cuda(), "%s must be a CUDA tensor (this library has no CPU path)", a.name);
    const int i = a->get_device();
    need_f(device < 0 || i == device, "%s is on another device than the other tensors", a.name);
    device = i;
  }
  return static_cast<c10::DeviceIndex>(device);
}

void check_workspace(const Arg& ws) {
  need_f(!ws || (ws->is_contiguous() && ws->nbytes() >= ATTN_FWD_WORKSPACE_BYTES),
         "workspace must be contiguous and hold at least %d bytes", ATTN_FWD_WORKSPACE_BYTES);
}

// One buffer per device and stream, for calls that bring none (never freed: at
// the process's end the driver may be gone before this map).
using Buffers = std::map<std::pair<int, cudaStream_t>, at::Tensor>;
Buffers& buffers() {
  static Buffers* b = new Buffers;
  return *b;
}

void enqueued(cudaError_t e) {
  if (e != cudaSuccess) throw std::runtime_error(std::string("workspace: ") + cudaGetErrorString(e));
}

// Bytes of a stream's buffer at most: the partial results of any call (80 MB on
// 152 SMs) fit. What needs more, the bf16 copy of long e4m3 sequences (up to 1 GiB),
// takes memory of torch's allocator for the one call.
constexpr int64_t kKeptBytes = 128ll << 20;

// Workspace of a call on `stream` (current, as is `device`): the stream's own
// buffer, which grows with need, so calls on different streams never share one.
// A captured call gets its own from the graph's memory, so that graphs do
// not share one either.
struct Workspace {
  at::Tensor memory;    // its head, and all of it unless that would be more than is kept
  at::Tensor scratch;   // else the rest, for this call

  void take(c10::DeviceIndex device, cudaStream_t stream, int64_t bytes) {
    const int64_t zeroed = ATTN_PAGED_ZEROED_BYTES;
    auto zero_filled = [&](int64_t n) {
      const at::Tensor t = fresh({n}, at::kByte, device);
      enqueued(cudaMemsetAsync(t.data_ptr(), 0, zeroed, stream));
      return t;
    };
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
      memory = zero_filled(bytes);
      return;
    }
    at::Tensor& kept = buffers()[{device, stream}];
    const int64_t keep = bytes <= kKeptBytes ? bytes : zeroed;
    if (!kept.defined()) {
      kept = zero_filled(keep);
    } else if (kept.numel() < keep) {
      const at::Tensor grown = fresh({keep}, at::kByte, device);
      // an error that nobody has read yet moves with it
      enqueued(cudaMemcpyAsync(grown.data_ptr(), kept.data_ptr(), zeroed, cudaMemcpyDeviceToDevice, stream));
      kept = grown;
    }
    memory = kept;
    if (bytes > kKeptBytes) scratch = fresh({bytes - zeroed}, at::kByte, device);
  }
};

PyObject* status(attn_status st) { return PyLong_FromLong(st); }

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

#define PAGED_BEGIN \
  HANDLE_TH_ERRORS  \
  try {
#define PAGED_END                                      \
  }                                                    \
  catch (const BadArgument& e) {                       \
    PyErr_SetString(PyExc_ValueError, e.what());       \
    return nullptr;                                    \
  }                                                    \
  END_HANDLE_TH_ERRORS

bool arity(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
  return false;
}

// (k, v, k_cache, v_cache, block_table, seqlens_k, k_scale, v_scale, cu_seqlens_q, workspace)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 10)) return nullptr;
  PAGED_BEGIN
  const Arg k = tensor("k", a[0]), v = tensor("v", a[1]), kc = tensor("k_cache", a[2]), vc = tensor("v_cache", a[3]),
            table = tensor("block_table", a[4]), lens = tensor("seqlens_k", a[5]),
            ks = tensor_or_none("k_scale", a[6]), vs = tensor_or_none("v_scale", a[7]),
            cu = tensor_or_none("cu_seqlens_q", a[8]), ws = tensor_or_none("workspace", a[9]);
  attn_cache_append_params p = {};
  p.cache = check_cache(kc, vc, table, ks, vs);
  const int lead = cu ? 1 : 2;
  need(is(k, at::kBFloat16) && is(v, at::kBFloat16), "new keys and values must be bf16");
  need(k->dim() == lead + 2 && k->sizes() == v->sizes(),
       "k and v must be [B, Sq, Hkv, D], or [T, Hkv, D] with cu_seqlens_q, of one shape");
  need(k->size(lead) == p.cache.num_heads_kv && k->size(lead + 1) == p.cache.head_dim,
       "k and v must have the cache's heads and depth");
  need(k->stride(lead + 1) == 1 && v->stride(lead + 1) == 1, "the depth of k and v must be contiguous");
  check_int32(lens, p.cache.batch);
  if (cu) {
    check_int32(cu, p.cache.batch + 1ll);
    p.total_q = int32("T", k->size(0));
  } else {
    need(k->size(0) == p.cache.batch, "k and block_table batch sizes differ");
    p.seqlen_q = int32("Sq", k->size(1));
  }
  for (int i = 0; i <= lead; ++i) {
    p.k_stride[i + 2 - lead] = stride(k, i);
    p.v_stride[i + 2 - lead] = stride(v, i);
  }
  check_workspace(ws);
  const c10::DeviceIndex device = check_device(std::array<Arg, 10>{k, v, kc, vc, table, lens, ks, vs, cu, ws});
  const c10::cuda::CUDAGuard guard(device);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(device).stream();
  Workspace own;
  if (!ws) own.take(device, stream, ATTN_PAGED_ZEROED_BYTES);
  p.k = k.ptr();
  p.v = v.ptr();
  p.seqlens_k = static_cast<const int32_t*>(lens.ptr());
  p.cu_seqlens_q = static_cast<const int32_t*>(cu.ptr());
  p.workspace = ws ? ws.ptr() : own.memory.data_ptr();
  return status(attn_cache_append(&p, stream));
  PAGED_END
}

// (k_cache, v_cache, block_table, cu_seqlens_k, total_k, k_scale, v_scale, out_k, out_v, workspace)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 10)) return nullptr;
  PAGED_BEGIN
  const Arg kc = tensor("k_cache", a[0]), vc = tensor("v_cache", a[1]), table = tensor("block_table", a[2]),
            cu = tensor("cu_seqlens_k", a[3]), ks = tensor_or_none("k_scale", a[5]),
            vs = tensor_or_none("v_scale", a[6]), ok = tensor_or_none("out_k", a[7]),
            ov = tensor_or_none("out_v", a[8]), ws = tensor_or_none("workspace", a[9]);
  attn_cache_read_params p = {};
  p.cache = check_cache(kc, vc, table, ks, vs);
  const int64_t heads = p.cache.num_heads_kv, dim = p.cache.head_dim;
  check_int32(cu, p.cache.batch + 1ll);
  need(bool(ok) == bool(ov), "out_k and out_v go together");
  int64_t total = -1;
  if (a[4] != Py_None) {
    total = integer("total_k", a[4]);
    need(total >= 0, "total_k must not be negative");
  }
  if (!ok) {
    need(total >= 0, "total_k (the rows to allocate) or out_k and out_v are needed");
  } else {
    const int64_t rows = ok->dim() ? ok->size(0) : 0;
    need(total < 0 || total == rows, "total_k differs from the rows of out_k");
    total = rows;
    for (const Arg* o : {&ok, &ov})
      need_f(is(*o, at::kBFloat16) && (*o)->dim() == 3 && (*o)->size(0) == rows && (*o)->size(1) == heads &&
                 (*o)->size(2) == dim && (*o)->stride(2) == 1,
             "%s must be a bf16 [Tk, Hkv, D] tensor with contiguous depth", o->name);
  }
  p.total_k = int32("total_k", total);
  check_workspace(ws);
  const c10::DeviceIndex device = check_device(std::array<Arg, 9>{kc, vc, table, cu, ks, vs, ok, ov, ws});
  const c10::cuda::CUDAGuard guard(device);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(device).stream();
  at::Tensor fresh_k, fresh_v;
  Workspace own;
  if (!ok) {
    fresh_k = fresh({total, heads, dim}, at::kBFloat16, device);
    fresh_v = fresh({total, heads, dim}, at::kBFloat16, device);
  }
  const Arg k = {"out_k", ok ? ok.t : &fresh_k}, v = {"out_v", ov ? ov.t : &fresh_v};
  if (!ws) own.take(device, stream, ATTN_PAGED_ZEROED_BYTES);
  p.k = k.ptr();
  p.v = v.ptr();
  for (int i = 0; i < 2; ++i) {
    p.k_stride[i] = stride(k, i);
    p.v_stride[i] = stride(v, i);
  }
  p.cu_seqlens_k = static_cast<const int32_t*>(cu.ptr());
  p.workspace = ws ? ws.ptr() : own.memory.data_ptr();
  const attn_status st = attn_cache_read(&p, stream);
  if (st != ATTN_OK) return status(st);
  PyObject* r = PyTuple_New(2);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, ok ? same(a[7]) : THPVariable_Wrap(std::move(fresh_k)));
  PyTuple_SET_ITEM(r, 1, ov ? same(a[8]) : THPVariable_Wrap(std::move(fresh_v)));
  return r;
  PAGED_END
}

// (q, k_cache, v_cache, block_table, seqlens_k, causal, softmax_scale, k_scale, v_scale, cu_seqlens_q, max_seqlen_q,
//  max_seqlen_k, out, lse, return_lse, workspace)
PyObject* paged_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 16)) return nullptr;
  PAGED_BEGIN
  const Arg q = tensor("q", a[0]), kc = tensor("k_cache", a[1]), vc = tensor("v_cache", a[2]),
            table = tensor("block_table", a[3]), lens = tensor("seqlens_k", a[4]),
            ks = tensor_or_none("k_scale", a[7]), vs = tensor_or_none("v_scale", a[8]),
            cu = tensor_or_none("cu_seqlens_q", a[9]), out = tensor_or_none("out", a[12]),
            lse = tensor_or_none("lse", a[13]), ws = tensor_or_none("workspace", a[15]);
  attn_paged_params p = {};
  p.cache = check_cache(kc, vc, table, ks, vs);
  const int lead = cu ? 1 : 2;
  need(is(q, at::kBFloat16), "q must be bf16");
  need(q->dim() == lead + 2, "q must be [B, Sq, Hq, D], or [T, Hq, D] with cu_seqlens_q");
  need(q->size(lead + 1) == p.cache.head_dim, "q and the cache have different depths");
  need(q->stride(lead + 1) == 1, "the depth of q must be contiguous");
  check_int32(lens, p.cache.batch);
  const int64_t hq = q->size(lead);
  std::array<int64_t, 3> lse_shape = {p.cache.batch, hq, 0};
  if (cu) {
    check_int32(cu, p.cache.batch + 1ll);
    need(a[10] != Py_None, "packed q needs max_seqlen_q");
    const int64_t most = integer("max_seqlen_q", a[10]);
    need(most >= 0, "max_seqlen_q must not be negative");
    p.total_q = int32("T", q->size(0));
    p.seqlen_q = static_cast<int32_t>(std::min<int64_t>(most, p.total_q));
    lse_shape = {hq, p.total_q, 0};
  } else {
    need(q->size(0) == p.cache.batch, "q and block_table batch sizes differ");
    p.seqlen_q = int32("Sq", q->size(1));
    lse_shape[2] = p.seqlen_q;
  }
  const at::IntArrayRef lse_sizes(lse_shape.data(), cu ? 2 : 3);
  int64_t most_k = (int64_t)p.cache.max_pages * p.cache.page_size;
  if (a[11] != Py_None) {
    const int64_t bound = integer("max_seqlen_k", a[11]);
    need(bound >= 0, "max_seqlen_k must not be negative");
    most_k = std::min(most_k, bound);
  }
  p.seqlen_k = int32("max_pages * page_size", most_k);
  need(!out || (is(out, at::kBFloat16) && out->sizes() == q->sizes() && out->stride(lead + 1) == 1),
       "out must be a bf16 tensor of q's shape with contiguous depth");
  need(!lse || (is(lse, at::kFloat) && lse->sizes() == lse_sizes && lse->is_contiguous()),
       "lse must be a contiguous fp32 tensor of shape [B, Hq, Sq], or [Hq, T] with cu_seqlens_q");
  double scale = 1.0 / std::sqrt((double)(p.cache.head_dim > 0 ? p.cache.head_dim : 1));
  if (a[6] != Py_None) {
    scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  const int causal = PyObject_IsTrue(a[5]), want_lse = PyObject_IsTrue(a[14]);
  if (causal < 0 || want_lse < 0) return nullptr;
  check_workspace(ws);
  const c10::DeviceIndex device = check_device(std::array<Arg, 11>{q, kc, vc, table, lens, ks, vs, cu, out, lse, ws});
  const c10::cuda::CUDAGuard guard(device);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(device).stream();
  at::Tensor fresh_o, fresh_l;
  Workspace own;
  if (!out) fresh_o = fresh(q->sizes(), at::kBFloat16, device);
  if (!lse && want_lse) fresh_l = fresh(lse_sizes, at::kFloat, device);
  const Arg o = {"out", out ? out.t : &fresh_o};
  p.q = q.ptr();
  p.o = o.ptr();
  p.lse = lse ? static_cast<float*>(lse.ptr()) : (want_lse ? fresh_l.data_ptr<float>() : nullptr);
  p.seqlens_k = static_cast<const int32_t*>(lens.ptr());
  p.cu_seqlens_q = static_cast<const int32_t*>(cu.ptr());
  for (int i = 0; i <= lead; ++i) {
    p.q_stride[i + 2 - lead] = stride(q, i);
    p.o_stride[i + 2 - lead] = stride(o, i);
  }
  p.num_heads_q = int32("Hq", hq);
  p.causal = causal;
  p.softmax_scale = static_cast<float>(scale);
  if (ws) {
    p.workspace = ws.ptr();
    p.workspace_bytes = ws->nbytes();
  } else {
    own.take(device, stream, (int64_t)attn_paged_workspace_bytes(&p));
    p.workspace = own.memory.data_ptr();
    p.workspace_bytes = own.memory.nbytes();
  }
  const attn_status st = own.scratch.defined()
                             ? af::paged_fwd(&p, own.scratch.data_ptr(), own.scratch.nbytes(), stream)
                             : attn_paged_fwd(&p, stream);
  if (st != ATTN_OK) return status(st);
  PyObject* r = PyTuple_New(2);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, out ? same(a[12]) : THPVariable_Wrap(std::move(fresh_o)));
  PyTuple_SET_ITEM(r, 1, lse ? same(a[13]) : (want_lse ? THPVariable_Wrap(std::move(fresh_l)) : same(Py_None)));
  return r;
  PAGED_END
}

// (device index, stream handle): address of that stream's buffer, 0 if there is none.
PyObject* workspace_address(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!arity(n, 2)) return nullptr;
  PAGED_BEGIN
  const auto it = buffers().find({(int)integer("device", a[0]),
                                  reinterpret_cast<cudaStream_t>(static_cast<intptr_t>(integer("stream", a[1])))});
  return PyLong_FromVoidPtr(it == buffers().end() || !it->second.defined() ? nullptr : it->second.data_ptr());
  PAGED_END
}

#define FAST(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FAST(cache_append), FAST(cache_read), FAST(paged_forward), FAST(workspace_address),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_native() { return PyModule_Create(&module); }
