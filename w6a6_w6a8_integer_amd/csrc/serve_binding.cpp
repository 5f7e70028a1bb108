// serve_binding.cpp -- the Python side of the decoding-step calls that run once a layer
// and step (all of serve.py's but pack_w4): the argument checks,
// output allocation and C call of serve.py's functions without the interpreter between
// them.  A step's smallest calls take 4 to 10 us on the GPU; checked in Python they took
// 11 to 22 us of the host's time, here 5 to 11.
//
// The C functions are those of the library that the package has loaded: bind() takes
// their addresses.  Every other function takes all of its arguments by position (serve.py
// has the signatures and their documentation), raises TypeError or ValueError before the C
// ABI sees a pointer, and FlexqError for a status it returns.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>
#include <utility>

#include "../../include/flexq_serve.h"

namespace {

using at::Tensor;

struct {
  decltype(&flexq_gemv_w4) gemv_w4;
  decltype(&flexq_gemv_w4_workspace_bytes) gemv_w4_workspace_bytes;
  decltype(&flexq_block_tables) block_tables;
  decltype(&flexq_kv_cache_write) kv_cache_write;
  decltype(&flexq_tree_attention) tree_attention;
  decltype(&flexq_tree_attention_workspace_bytes) tree_attention_workspace_bytes;
  decltype(&flexq_kv4_cache_write) kv4_cache_write;
  decltype(&flexq_kv4_cache_read) kv4_cache_read;
  decltype(&flexq_kv4_attention) kv4_attention;
  decltype(&flexq_kv4_attention_workspace_bytes) kv4_attention_workspace_bytes;
  decltype(&flexq_lora_add) lora_add;
  decltype(&flexq_lora_add_workspace_bytes) lora_add_workspace_bytes;
} library;

// A refused argument, on its way to the interpreter.
struct Refusal {
  PyObject* type;
  std::string text;
};

template <class... Parts>
[[noreturn]] void refuse(PyObject* type, const Parts&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw Refusal{type, s.str()};
}

template <class... Parts>
void value_check(bool ok, const Parts&... parts) {
  if (!ok) refuse(PyExc_ValueError, parts...);
}

std::string shape_text(at::IntArrayRef shape) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < shape.size(); ++i) s << (i ? ", " : "") << shape[i];
  s << (shape.size() == 1 ? ",)" : ")");
  return s.str();
}

std::string dtype_text(at::ScalarType t) {
  PyObject* o = reinterpret_cast<PyObject*>(torch::getTHPDtype(t));
  PyObject* r = PyObject_Str(o);
  std::string s = r ? PyUnicode_AsUTF8(r) : "?";
  Py_XDECREF(r);
  return s;
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    refuse(PyExc_TypeError, name, " must be a torch.Tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

void dtype_check(const Tensor& t, at::ScalarType dtype, const char* name) {
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, name, " must be ", dtype_text(dtype), ", got ",
           dtype_text(t.scalar_type()));
}

void dims_check(const Tensor& t, int64_t dims, const char* name) {
  value_check(t.dim() == dims, name, " must be ", dims, "-D, got shape ", shape_text(t.sizes()));
}

// type, exact shape and contiguity
const Tensor& exact(const Tensor& t, at::ScalarType dtype, const char* name,
                    at::IntArrayRef shape) {
  dtype_check(t, dtype, name);
  value_check(t.sizes() == shape, name, " must have shape ", shape_text(shape), ", got ",
              shape_text(t.sizes()));
  value_check(t.is_contiguous(), name, " must be contiguous");
  return t;
}

// a flat buffer of at least `bytes`
const Tensor& flat(const Tensor& t, at::ScalarType dtype, const char* name, int64_t bytes) {
  dims_check(t, 1, name);
  dtype_check(t, dtype, name);
  const int64_t has = t.numel() * (int64_t)t.element_size();
  value_check(has >= bytes, name, " holds ", has, " bytes; at least ", bytes, " are needed");
  value_check(t.is_contiguous(), name, " must be contiguous");
  return t;
}

// the last dimension contiguous, the others as they are
const Tensor& rows(const Tensor& t, at::ScalarType dtype, const char* name, int64_t dims) {
  dtype_check(t, dtype, name);
  dims_check(t, dims, name);
  value_check(t.size(-1) <= 1 || t.stride(-1) == 1, name,
              " must be contiguous along its last dimension");
  return t;
}

int32_t half_type(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kHalf) return FLEXQ_FP16;
  if (t.scalar_type() == at::kBFloat16) return FLEXQ_BF16;
  refuse(PyExc_TypeError, name, " must be float16 or bfloat16, got ",
         dtype_text(t.scalar_type()));
}

// no tensor that autograd would ask for a gradient of
void no_grad_check(const Tensor& t, const char* name) {
  value_check(!t.defined() || !t.requires_grad() || !c10::GradMode::is_enabled(), name,
              " requires grad, and there is no backward pass: call it under torch.no_grad()");
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, name, " must be an integer, got ", Py_TYPE(o)->tp_name);
  }
  return v;
}

// Every argument on one GPU.
class OneGpu {
 public:
  void add(const Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(PyExc_TypeError, name, " must be a CUDA (HIP) tensor");
    if (!device_) {
      device_ = t.device();
    } else if (t.device() != *device_) {
      refuse(PyExc_ValueError, name, " is on ", t.device().str(), ", the other arguments on ",
             device_->str());
    }
  }
  c10::DeviceIndex index() const { return device_->index(); }

 private:
  std::optional<at::Device> device_;
};

// That GPU current while the call is made.
class Current {
 public:
  explicit Current(c10::DeviceIndex index) : before_(c10::hip::current_device()) {
    if (index != before_) c10::hip::set_device(index);
  }
  ~Current() {
    if (c10::hip::current_device() != before_) c10::hip::set_device(before_);
  }

 private:
  c10::DeviceIndex before_;
};

void* stream_of(c10::DeviceIndex index) {
  return c10::hip::getCurrentHIPStream(index).stream();
}

PyObject* raise_status(flexq_status status, const char* name) {
  PyObject* package = PyImport_ImportModule("w6a6_w6a8_integer_amd");
  PyObject* type = package ? PyObject_GetAttrString(package, "FlexqError") : nullptr;
  PyObject* error = type ? PyObject_CallFunction(type, "is", (int)status, name) : nullptr;
  if (error) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(package);
  return nullptr;
}

const void* data(const Tensor& t) { return t.const_data_ptr(); }

Tensor make(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(like.device()));
}

// [pages][Hkv][page_size/16][D][16] and the keys that go with it
struct Cache {
  int64_t pages, heads, width;
  int32_t page_size;
};

Cache cache_of(const Tensor& k, const Tensor& v, at::ScalarType dtype) {
  value_check(v.dim() == 5, "v_cache must be a 5-D tensor [pages][Hkv][page_size/16][D][16]");
  const int64_t blocks = v.size(2), D = v.size(3);
  const bool page = blocks == 1 || blocks == 2 || blocks == 4 || blocks == 8 || blocks == 16;
  const bool width = D == 64 || D == 96 || D == 128 || D == 256;
  value_check(page && width && v.size(4) == 16,
              "v_cache must be [pages][Hkv][page_size/16][D][16] with page_size one of (16, 32, "
              "64, 128, 256) and D one of (64, 96, 128, 256), got ",
              shape_text(v.sizes()));
  exact(v, dtype, "v_cache", v.sizes());
  exact(k, dtype, "k_cache", {v.size(0), v.size(1), blocks, D / 32, 16, 32});
  return {v.size(0), v.size(1), D, (int32_t)(16 * blocks)};
}

bool given(PyObject* o) { return o != Py_None; }

PyObject* gemv_w4(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  const int32_t type = half_type(x, "x");
  rows(x, x.scalar_type(), "x", 2);
  const int64_t M = x.size(0), K = x.size(1), N = integer(a[3], "N");
  value_check(K > 0 && K % 128 == 0, "gemv_w4: K = ", K, " must be a positive multiple of 128");
  value_check(N >= 0 && N % 16 == 0, "N = ", N, " must be a non-negative multiple of 16");
  const Tensor& s = tensor(a[2], "s_w");
  value_check(s.dim() == 2, "s_w must be a 2-D tensor [K/group][N]");
  const int64_t G = s.size(0);
  value_check(G > 0 && K % G == 0, "s_w must have K / group rows for K = ", K, ", got ", G);
  const int64_t group = K / G;
  value_check(group == 32 || group == 64 || group == 128, "group = ", group,
              " must be 32, 64 or 128");
  exact(s, at::kHalf, "s_w", {G, N});
  const Tensor& w = flat(tensor(a[1], "w4"), at::kInt, "w4", N * K / 2);
  OneGpu gpu;
  Tensor y, ws;
  if (given(a[4])) y = exact(tensor(a[4], "y"), x.scalar_type(), "y", {M, N});
  const int64_t need = (int64_t)library.gemv_w4_workspace_bytes(M, N, K);
  if (given(a[5])) ws = flat(tensor(a[5], "workspace"), at::kByte, "workspace", need);
  gpu.add(x, "x");
  gpu.add(w, "w4");
  gpu.add(s, "s_w");
  if (!y.defined()) y = make({M, N}, x.scalar_type(), x);
  gpu.add(y, "y");
  if (!ws.defined() && need > 0) ws = make({need}, at::kByte, x);
  if (ws.defined()) gpu.add(ws, "workspace");
  Current current(gpu.index());
  const flexq_status status = library.gemv_w4(
      (const uint16_t*)data(x), type, x.stride(0), (const uint32_t*)data(w),
      (const uint16_t*)data(s), M, N, K, (int32_t)group,
      ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? ws.numel() : 0,
      (uint16_t*)y.mutable_data_ptr(), stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_gemv_w4");
  return THPVariable_Wrap(y);
}

PyObject* block_tables(PyObject* const* a) {
  const Tensor& table = tensor(a[3], "block_table");
  dims_check(table, 2, "block_table");
  exact(table, at::kInt, "block_table", table.sizes());
  const int64_t B = table.size(0), max_blocks = table.size(1);
  const Tensor& ctx = exact(tensor(a[0], "ctx_lens"), at::kInt, "ctx_lens", {B});
  const Tensor& add = exact(tensor(a[1], "new_lens"), at::kInt, "new_lens", {B});
  const Tensor& pages = flat(tensor(a[2], "free_pages"), at::kInt, "free_pages", 0);
  const int64_t page_size = integer(a[4], "page_size"), most = integer(a[5], "max_tokens");
  value_check(most >= 0, "max_tokens = ", most, " must not be negative");
  value_check(page_size == (int32_t)page_size, "page_size = ", page_size, " is out of range");
  OneGpu gpu;
  Tensor head, slots, cu, counts;
  if (given(a[6])) head = exact(tensor(a[6], "free_head"), at::kInt, "free_head", {1});
  if (given(a[7])) slots = exact(tensor(a[7], "slot_map"), at::kInt, "slot_map", {most});
  if (given(a[8])) cu = exact(tensor(a[8], "cu_new"), at::kInt, "cu_new", {B + 1});
  if (given(a[9])) counts = exact(tensor(a[9], "counts"), at::kInt, "counts", {3});
  gpu.add(table, "block_table");
  gpu.add(ctx, "ctx_lens");
  gpu.add(add, "new_lens");
  gpu.add(pages, "free_pages");
  if (head.defined()) gpu.add(head, "free_head");
  if (!slots.defined()) slots = make({most}, at::kInt, table);
  if (!cu.defined()) cu = make({B + 1}, at::kInt, table);
  if (!counts.defined()) counts = make({3}, at::kInt, table);
  gpu.add(slots, "slot_map");
  gpu.add(cu, "cu_new");
  gpu.add(counts, "counts");
  Current current(gpu.index());
  const flexq_status status = library.block_tables(
      (const int32_t*)data(ctx), (const int32_t*)data(add), B, (const int32_t*)data(pages),
      pages.numel(), head.defined() ? (const int32_t*)data(head) : nullptr, (int32_t)page_size,
      (int32_t*)table.mutable_data_ptr(), max_blocks, most, (int32_t*)slots.mutable_data_ptr(),
      (int32_t*)cu.mutable_data_ptr(), (int32_t*)counts.mutable_data_ptr(),
      stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_block_tables");
  PyObject* out = PyTuple_New(3);
  if (!out) return nullptr;
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(slots));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(cu));
  PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(counts));
  return out;
}

PyObject* kv_cache_write(PyObject* const* a) {
  const Tensor& k = tensor(a[0], "k");
  const Tensor& v = tensor(a[1], "v");
  half_type(k, "k");
  const at::ScalarType dtype = k.scalar_type();
  rows(k, dtype, "k", 3);
  const Tensor &kc = tensor(a[3], "k_cache"), &vc = tensor(a[4], "v_cache");
  const Cache cache = cache_of(kc, vc, dtype);
  const int64_t T = k.size(0);
  const int64_t shape[3] = {T, cache.heads, cache.width};
  value_check(k.sizes() == at::IntArrayRef(shape), "k must have shape ", shape_text(shape),
              ", got ", shape_text(k.sizes()));
  rows(v, dtype, "v", 3);
  value_check(v.sizes() == k.sizes(), "v must have shape ", shape_text(shape), ", got ",
              shape_text(v.sizes()));
  const Tensor& slots = exact(tensor(a[2], "slot_map"), at::kInt, "slot_map", {T});
  OneGpu gpu;
  gpu.add(k, "k");
  gpu.add(v, "v");
  gpu.add(slots, "slot_map");
  gpu.add(kc, "k_cache");
  gpu.add(vc, "v_cache");
  Current current(gpu.index());
  const flexq_status status = library.kv_cache_write(
      (const uint16_t*)data(k), k.stride(0), k.stride(1), (const uint16_t*)data(v), v.stride(0),
      v.stride(1), (const int32_t*)data(slots), T, cache.heads, cache.width, cache.pages,
      cache.page_size, (uint16_t*)kc.mutable_data_ptr(), (uint16_t*)vc.mutable_data_ptr(),
      stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_kv_cache_write");
  Py_RETURN_NONE;
}

// The arguments that the attention calls share, checked but for the cache's own: q, the block
// table and lengths, the masks and the outputs.
struct Attention {
  Tensor q, table, ctx, cu, mask, out, lse, ws;
  int32_t type;
  at::ScalarType dtype;
  int64_t T, H, D, B, max_blocks, max_new, words = 0;
  double scale;
  bool want_lse;

  Attention(PyObject* query, PyObject* block_table, PyObject* ctx_lens, PyObject* cu_new,
            PyObject* tree_mask, PyObject* scale_or_none, PyObject* most_new, PyObject* out_or_none,
            PyObject* lse_or_none, PyObject* return_lse, const Cache& cache) {
    q = tensor(query, "q");
    type = half_type(q, "q");
    dtype = q.scalar_type();
    rows(q, dtype, "q", 3);
    T = q.size(0), H = q.size(1), D = q.size(2);
    value_check(cache.width == D && cache.heads > 0 && H > 0 && H % cache.heads == 0, "q [", T, "][",
                H, "][", D, "] does not fit a cache of ", cache.heads, " heads of ", cache.width);
    table = tensor(block_table, "block_table");
    dims_check(table, 2, "block_table");
    exact(table, at::kInt, "block_table", table.sizes());
    B = table.size(0), max_blocks = table.size(1);
    ctx = exact(tensor(ctx_lens, "ctx_lens"), at::kInt, "ctx_lens", {B});
    cu = exact(tensor(cu_new, "cu_new"), at::kInt, "cu_new", {B + 1});
    max_new = given(most_new) ? integer(most_new, "max_new") : T;
    if (given(tree_mask)) {
      mask = tensor(tree_mask, "tree_mask");
      dims_check(mask, 2, "tree_mask");
      words = mask.size(1);
      exact(mask, at::kInt, "tree_mask", {T, words});
      // a mask's bits are as many as one request's tokens may be
      if (!given(most_new)) max_new = std::min(T, 32 * words);
      value_check(max_new <= 32 * words, "tree_mask has ", 32 * words, " bits a token; max_new = ",
                  max_new);
    }
    scale = 1.0 / std::sqrt((double)D);
    if (given(scale_or_none)) {
      scale = PyFloat_AsDouble(scale_or_none);
      if (scale == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(PyExc_TypeError, "scale must be a number, got ", Py_TYPE(scale_or_none)->tp_name);
      }
    }
    if (given(out_or_none)) out = exact(tensor(out_or_none, "out"), dtype, "out", {T, H, D});
    if (given(lse_or_none)) lse = exact(tensor(lse_or_none, "lse"), at::kFloat, "lse", {T, H});
    const int truth = PyObject_IsTrue(return_lse);
    if (truth < 0) {
      PyErr_Clear();
      refuse(PyExc_TypeError, "return_lse has no truth value");
    }
    want_lse = truth != 0;
  }

  // Every tensor on one GPU; outputs and the workspace made where the caller brings none.
  void place(OneGpu& gpu, std::initializer_list<std::pair<const Tensor*, const char*>> cache,
             PyObject* workspace, int64_t need) {
    if (given(workspace)) ws = flat(tensor(workspace, "workspace"), at::kByte, "workspace", need);
    gpu.add(q, "q");
    for (const auto& c : cache) gpu.add(*c.first, c.second);
    gpu.add(table, "block_table");
    gpu.add(ctx, "ctx_lens");
    gpu.add(cu, "cu_new");
    if (mask.defined()) gpu.add(mask, "tree_mask");
    if (!out.defined()) out = make({T, H, D}, dtype, q);
    gpu.add(out, "out");
    if (!lse.defined() && want_lse) lse = make({T, H}, at::kFloat, q);
    if (lse.defined()) gpu.add(lse, "lse");
    if (!ws.defined()) ws = make({std::max<int64_t>(16, need)}, at::kByte, q);
    gpu.add(ws, "workspace");
  }

  const int32_t* mask_data() const { return mask.defined() ? (const int32_t*)data(mask) : nullptr; }
  float* lse_data() const { return lse.defined() ? (float*)lse.mutable_data_ptr() : nullptr; }

  PyObject* result() const {
    if (!lse.defined()) return THPVariable_Wrap(out);
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(lse));
    return both;
  }
};

PyObject* tree_attention(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  half_type(q, "q");
  rows(q, q.scalar_type(), "q", 3);
  const Tensor &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
  const Cache cache = cache_of(kc, vc, q.scalar_type());
  Attention t(a[0], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], cache);
  OneGpu gpu;
  t.place(gpu, {{&kc, "k_cache"}, {&vc, "v_cache"}}, a[12],
          (int64_t)library.tree_attention_workspace_bytes(t.B, t.max_new, t.H, cache.heads, t.D));
  Current current(gpu.index());
  const flexq_status status = library.tree_attention(
      (const uint16_t*)data(q), t.type, q.stride(0), q.stride(1), (const uint16_t*)data(kc),
      (const uint16_t*)data(vc), cache.pages, cache.page_size, (const int32_t*)data(t.table),
      t.max_blocks, (const int32_t*)data(t.ctx), (const int32_t*)data(t.cu), t.B, t.T, t.max_new,
      t.H, cache.heads, t.D, t.mask_data(), t.words, (float)t.scale, t.ws.mutable_data_ptr(),
      t.ws.numel(), (uint16_t*)t.out.mutable_data_ptr(), t.lse_data(), stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_tree_attention");
  return t.result();
}

// codes [pages][Hkv][page_size/16][16][D/8] and [..][2][D/2][2], scales [..][4][16]
Cache kv4_cache_of(const Tensor& k, const Tensor& v, const Tensor& s) {
  value_check(k.dim() == 5, "k_codes must be a 5-D tensor [pages][Hkv][page_size/16][16][D/8]");
  const int64_t blocks = k.size(2), D = 8 * k.size(4);
  const bool page = blocks == 1 || blocks == 2 || blocks == 4 || blocks == 8 || blocks == 16;
  const bool width = D == 64 || D == 96 || D == 128 || D == 256;
  value_check(page && width && k.size(3) == 16,
              "k_codes must be [pages][Hkv][page_size/16][16][D/8] with page_size one of (16, 32, "
              "64, 128, 256) and D one of (64, 96, 128, 256), got ",
              shape_text(k.sizes()));
  exact(k, at::kInt, "k_codes", k.sizes());
  exact(v, at::kInt, "v_codes", {k.size(0), k.size(1), blocks, 2, D / 2, 2});
  exact(s, at::kHalf, "scales", {k.size(0), k.size(1), blocks, 4, 16});
  return {k.size(0), k.size(1), D, (int32_t)(16 * blocks)};
}

PyObject* kv4_cache_write(PyObject* const* a) {
  const Tensor& k = tensor(a[0], "k");
  const Tensor& v = tensor(a[1], "v");
  const int32_t type = half_type(k, "k");
  const at::ScalarType dtype = k.scalar_type();
  rows(k, dtype, "k", 3);
  const Tensor &kc = tensor(a[3], "k_codes"), &vc = tensor(a[4], "v_codes");
  const Tensor& sc = tensor(a[5], "scales");
  const Cache cache = kv4_cache_of(kc, vc, sc);
  const int64_t T = k.size(0);
  const int64_t shape[3] = {T, cache.heads, cache.width};
  value_check(k.sizes() == at::IntArrayRef(shape), "k must have shape ", shape_text(shape),
              ", got ", shape_text(k.sizes()));
  rows(v, dtype, "v", 3);
  value_check(v.sizes() == k.sizes(), "v must have shape ", shape_text(shape), ", got ",
              shape_text(v.sizes()));
  const Tensor& slots = exact(tensor(a[2], "slot_map"), at::kInt, "slot_map", {T});
  OneGpu gpu;
  gpu.add(k, "k");
  gpu.add(v, "v");
  gpu.add(slots, "slot_map");
  gpu.add(kc, "k_codes");
  gpu.add(vc, "v_codes");
  gpu.add(sc, "scales");
  Current current(gpu.index());
  const flexq_status status = library.kv4_cache_write(
      (const uint16_t*)data(k), k.stride(0), k.stride(1), (const uint16_t*)data(v), v.stride(0),
      v.stride(1), type, (const int32_t*)data(slots), T, cache.heads, cache.width, cache.pages,
      cache.page_size, (uint32_t*)kc.mutable_data_ptr(), (uint32_t*)vc.mutable_data_ptr(),
      (uint16_t*)sc.mutable_data_ptr(), stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_kv4_cache_write");
  Py_RETURN_NONE;
}

PyObject* kv4_cache_read(PyObject* const* a) {
  const Tensor &kc = tensor(a[1], "k_codes"), &vc = tensor(a[2], "v_codes");
  const Tensor& sc = tensor(a[3], "scales");
  const Cache cache = kv4_cache_of(kc, vc, sc);
  const Tensor& slots = tensor(a[0], "slot_map");
  dims_check(slots, 1, "slot_map");
  exact(slots, at::kInt, "slot_map", slots.sizes());
  const int64_t T = slots.size(0);
  value_check(THPDtype_Check(a[4]), "dtype must be torch.float16 or torch.bfloat16");
  const at::ScalarType dtype = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
  value_check(dtype == at::kHalf || dtype == at::kBFloat16,
              "dtype must be torch.float16 or torch.bfloat16, got ", dtype_text(dtype));
  const int64_t shape[3] = {T, cache.heads, cache.width};
  OneGpu gpu;
  Tensor k, v;
  if (given(a[5])) k = exact(tensor(a[5], "k"), dtype, "k", shape);
  if (given(a[6])) v = exact(tensor(a[6], "v"), dtype, "v", shape);
  gpu.add(slots, "slot_map");
  gpu.add(kc, "k_codes");
  gpu.add(vc, "v_codes");
  gpu.add(sc, "scales");
  if (!k.defined()) k = make(shape, dtype, slots);
  if (!v.defined()) v = make(shape, dtype, slots);
  gpu.add(k, "k");
  gpu.add(v, "v");
  Current current(gpu.index());
  const flexq_status status = library.kv4_cache_read(
      (const uint32_t*)data(kc), (const uint32_t*)data(vc), (const uint16_t*)data(sc),
      (const int32_t*)data(slots), T, cache.heads, cache.width, cache.pages, cache.page_size,
      dtype == at::kHalf ? FLEXQ_FP16 : FLEXQ_BF16, (uint16_t*)k.mutable_data_ptr(),
      (uint16_t*)v.mutable_data_ptr(), stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_kv4_cache_read");
  PyObject* both = PyTuple_New(2);
  if (!both) return nullptr;
  PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(k));
  PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(v));
  return both;
}

PyObject* kv4_attention(PyObject* const* a) {
  const Tensor &kc = tensor(a[1], "k_codes"), &vc = tensor(a[2], "v_codes");
  const Tensor& sc = tensor(a[3], "scales");
  const Cache cache = kv4_cache_of(kc, vc, sc);
  Attention t(a[0], a[4], a[5], a[6], a[7], a[8], a[9], a[12], a[13], a[14], cache);
  // (none is 0 in C)
  const int64_t window = given(a[10]) ? integer(a[10], "window") : 0;
  value_check(!given(a[10]) || window > 0, "window = ", window, " must be positive, or None");
  const int64_t sinks = integer(a[11], "sinks");
  value_check(sinks >= 0, "sinks = ", sinks, " must not be negative");
  OneGpu gpu;
  t.place(gpu, {{&kc, "k_codes"}, {&vc, "v_codes"}, {&sc, "scales"}}, a[15],
          (int64_t)library.kv4_attention_workspace_bytes(t.B, t.max_new, t.H, cache.heads, t.D));
  Current current(gpu.index());
  const flexq_status status = library.kv4_attention(
      (const uint16_t*)data(t.q), t.type, t.q.stride(0), t.q.stride(1), (const uint32_t*)data(kc),
      (const uint32_t*)data(vc), (const uint16_t*)data(sc), cache.pages, cache.page_size,
      (const int32_t*)data(t.table), t.max_blocks, (const int32_t*)data(t.ctx),
      (const int32_t*)data(t.cu), t.B, t.T, t.max_new, t.H, cache.heads, t.D, t.mask_data(),
      t.words, window, sinks, (float)t.scale, t.ws.mutable_data_ptr(), t.ws.numel(),
      (uint16_t*)t.out.mutable_data_ptr(), t.lse_data(), stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_kv4_attention");
  return t.result();
}

PyObject* lora_add(PyObject* const* p) {
  const Tensor& x = tensor(p[0], "x");
  const int32_t type = half_type(x, "x");
  const at::ScalarType dtype = x.scalar_type();
  rows(x, dtype, "x", 2);
  const int64_t T = x.size(0), K = x.size(1);
  const Tensor& y = rows(tensor(p[1], "y"), dtype, "y", 2);
  value_check(y.size(0) == T, "y must have ", T, " rows, got shape ", shape_text(y.sizes()));
  const int64_t N = y.size(1);
  value_check(K > 0 && K % 128 == 0, "lora_add: K = ", K, " must be a positive multiple of 128");
  value_check(N % 16 == 0, "N = ", N, " must be a multiple of 16");
  const Tensor& adapters = exact(tensor(p[2], "adapters"), at::kInt, "adapters", {T});
  const Tensor& a = tensor(p[3], "a");
  dims_check(a, 3, "a");
  const int64_t L = a.size(0), R = a.size(1);
  value_check(R > 0 && R % 8 == 0 && R <= 256, "a has rank ", R,
              ", which must be a multiple of 8 up to 256");
  exact(a, dtype, "a", {L, R, K});
  const Tensor& b = exact(tensor(p[4], "b"), dtype, "b", {L, N, R});
  Tensor ranks, scales, out = y, ws;
  if (given(p[5])) ranks = exact(tensor(p[5], "ranks"), at::kInt, "ranks", {L});
  if (given(p[6])) scales = exact(tensor(p[6], "scales"), at::kFloat, "scales", {L});
  if (given(p[7])) {
    out = rows(tensor(p[7], "out"), dtype, "out", 2);
    value_check(out.sizes() == y.sizes(), "out must have shape ", shape_text(y.sizes()), ", got ",
                shape_text(out.sizes()));
  }
  no_grad_check(x, "x");
  no_grad_check(y, "y");
  no_grad_check(a, "a");
  no_grad_check(b, "b");
  no_grad_check(scales, "scales");
  no_grad_check(out, "out");
  OneGpu gpu;
  gpu.add(x, "x");
  gpu.add(y, "y");
  gpu.add(adapters, "adapters");
  gpu.add(a, "a");
  gpu.add(b, "b");
  if (ranks.defined()) gpu.add(ranks, "ranks");
  if (scales.defined()) gpu.add(scales, "scales");
  gpu.add(out, "out");
  const int64_t need = (int64_t)library.lora_add_workspace_bytes(T, N, K, R, L);
  if (given(p[8]))
    ws = flat(tensor(p[8], "workspace"), at::kByte, "workspace", need);
  else if (need > 0)
    ws = make({need}, at::kByte, x);
  if (ws.defined()) gpu.add(ws, "workspace");
  Current current(gpu.index());
  const flexq_status status = library.lora_add(
      (const uint16_t*)data(x), type, x.stride(0), (const uint16_t*)data(y), y.stride(0),
      (const int32_t*)data(adapters), (const uint16_t*)data(a), (const uint16_t*)data(b),
      ranks.defined() ? (const int32_t*)data(ranks) : nullptr,
      scales.defined() ? (const float*)data(scales) : nullptr, T, N, K, R, L,
      ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? ws.numel() : 0,
      (uint16_t*)out.mutable_data_ptr(), out.stride(0), stream_of(gpu.index()));
  if (status != FLEXQ_SUCCESS) return raise_status(status, "flexq_lora_add");
  return THPVariable_Wrap(out);
}

template <class F>
void take(F& to, PyObject* address) {
  to = reinterpret_cast<F>(PyLong_AsVoidPtr(address));
}

PyObject* bind(PyObject* const* a) {
  take(library.gemv_w4, a[0]);
  take(library.gemv_w4_workspace_bytes, a[1]);
  take(library.block_tables, a[2]);
  take(library.kv_cache_write, a[3]);
  take(library.tree_attention, a[4]);
  take(library.tree_attention_workspace_bytes, a[5]);
  take(library.kv4_cache_write, a[6]);
  take(library.kv4_cache_read, a[7]);
  take(library.kv4_attention, a[8]);
  take(library.kv4_attention_workspace_bytes, a[9]);
  take(library.lora_add, a[10]);
  take(library.lora_add_workspace_bytes, a[11]);
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

// Entry from the interpreter: the argument count, and every exception turned into Python's.
template <PyObject* (*call)(PyObject* const*), int count>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "%d arguments are taken, got %zd", count, n);
    return nullptr;
  }
  try {
    return call(args);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*call)(PyObject* const*), int count>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<call, count>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<bind, 12>("bind"), method<gemv_w4, 6>("gemv_w4"), method<block_tables, 10>("block_tables"),
    method<kv_cache_write, 5>("kv_cache_write"), method<tree_attention, 13>("tree_attention"),
    method<kv4_cache_write, 6>("kv4_cache_write"), method<kv4_cache_read, 7>("kv4_cache_read"),
    method<kv4_attention, 16>("kv4_attention"), method<lora_add, 9>("lora_add"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", nullptr, -1, methods,
                      nullptr,               nullptr,   nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) { return PyModule_Create(&module); }
