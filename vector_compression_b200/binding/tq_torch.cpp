// The paged cache's and the norm + rotation's entry points on torch tensors:
// checks of the arguments, memory for outputs and workspaces, the current
// stream and device.  Everything else is libtq's.  In C++ because these calls
// run once per layer and step: from Python the checks and the conversion of 20
// to 25 arguments took longer than the kernels of a small step.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <tuple>

#include "../../include/tq.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

// Raises the package's TQError for a status that is not TQ_OK.
void check(const char* fn, tq_status status) {
  if (status == TQ_OK) return;
  const py::object error = py::module_::import("vector_compression_b200._lib").attr("TQError");
  const py::object e = error(fn, (int)status);
  PyErr_SetObject(error.ptr(), e.ptr());
  throw py::error_already_set();
}

// A size as the library takes it.
int count(const char* what, int64_t n) {
  if (n > 0x7fffffff) refuse(std::string(what) + " is too large");
  return (int)n;
}

const Tensor* opt(const Maybe& t) { return t ? &*t : nullptr; }
void* ptr(const Tensor& t) { return t.data_ptr(); }

// The CUDA device that every given tensor is on.
c10::Device device_of(std::initializer_list<const Tensor*> ts) {
  const Tensor* first = nullptr;
  for (const Tensor* t : ts) {
    if (!t) continue;
    if (!t->is_cuda()) refuse("a CUDA device is needed");
    if (first && t->device() != first->device()) refuse("the tensors are on different devices");
    if (!first) first = t;
  }
  return first->device();
}

// The device made current, and its current stream.
struct Here {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Here(c10::Device d) : guard(d), stream(c10::cuda::getCurrentCUDAStream(d.index()).stream()) {}
};

tq_dtype dtype_of(const char* name, const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return TQ_F32;
    case at::kHalf: return TQ_F16;
    case at::kBFloat16: return TQ_BF16;
    default: refuse(std::string(name) + " must be float32, float16 or bfloat16");
  }
}

void* whole(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
    refuse(std::string(name) + " must be contiguous " + c10::toString(type) + " of shape " + c10::str(shape));
  return t.data_ptr();
}
template <typename T>
T* whole(const char* name, const Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
  return static_cast<T*>(whole(name, t, type, shape));
}

// The first byte of a workspace, whose bytes lie together (an expanded or strided view holds fewer than it counts).
void* together(const Tensor& ws) {
  if (!ws.is_contiguous()) refuse("ws must be contiguous");
  return ws.data_ptr();
}

int64_t rows_of(const char* name, const Tensor& t) {
  if (t.dim() != 1) refuse(std::string(name) + " must have one dimension");
  return t.size(0);
}

// A [n, heads, d] tensor whose last dimension is contiguous.
struct Heads {
  void* p;
  int64_t token, head;
  Heads(const char* name, const Tensor& x, int64_t n, int64_t heads, int64_t d, at::ScalarType type) {
    if (x.dim() != 3 || x.scalar_type() != type || x.size(0) != n || x.size(1) != heads || x.size(2) != d)
      refuse(std::string(name) + " must be " + c10::toString(type) + " [" + std::to_string(n) + ", " +
             std::to_string(heads) + ", " + std::to_string(d) + "]");
    if (x.stride(2) != 1 && d > 1 && n * heads) refuse("the last dimension of " + std::string(name) + " must be contiguous");
    p = x.data_ptr();
    token = x.stride(0);
    head = x.stride(1);
  }
};

std::tuple<Tensor, Maybe> qk_norm_rope(uintptr_t rope, const Tensor& q, const Maybe& k, const Maybe& pos, const Maybe& wq,
                                       const Maybe& wk, double eps, Maybe q_out, Maybe k_out) {
  if (q.dim() != 3) refuse("q must have three dimensions");
  const int64_t n = q.size(0), Hq = count("the number of heads", q.size(1)), d = count("the size of a head", q.size(2));
  const at::ScalarType type = q.scalar_type();
  const tq_dtype dt = dtype_of("q", q);
  const Here here(device_of({&q, opt(k), opt(pos), opt(wq), opt(wk), opt(q_out), opt(k_out)}));
  if (rope && !pos) refuse("a rotation needs positions");
  const Heads qi("q", q, n, Hq, d, type);
  if (!q_out) q_out = at::empty(q.sizes(), q.options());
  const Heads qo("q_out", *q_out, n, Hq, d, type);
  int64_t Hkv = 0;
  Heads ki = qi, ko = qo;
  if (k) {
    if (k->dim() != 3) refuse("k must have three dimensions");
    Hkv = count("the number of heads", k->size(1));
    ki = Heads("k", *k, n, Hkv, d, type);
    if (!k_out) k_out = at::empty(k->sizes(), k->options());
    ko = Heads("k_out", *k_out, n, Hkv, d, type);
  }
  const int64_t* p = pos ? whole<int64_t>("pos", *pos, at::kLong, {n}) : nullptr;
  const void* w0 = wq ? whole("wq", *wq, type, {d}) : nullptr;
  const void* w1 = wk ? whole("wk", *wk, type, {d}) : nullptr;
  tq_status s;
  {
    py::gil_scoped_release go;
    s = tq_qk_norm_rope(reinterpret_cast<const tq_rope*>(rope), dt, n, (int)d, (int)Hq, qi.p, qi.token, qi.head,
                        (int)Hkv, k ? ki.p : nullptr, ki.token, ki.head, p, w0, w1, (float)eps, qo.p, qo.token, qo.head,
                        k ? ko.p : nullptr, ko.token, ko.head, here.stream);
  }
  check("tq_qk_norm_rope", s);
  return {*q_out, k ? k_out : std::nullopt};
}

// What the calls need of a cache's description.
struct Paged {
  uintptr_t handle;
  int64_t page_words, hkv, d, key_words, sign_words, value_words;
  bool half_rnorm;
  const tq_paged* get() const { return reinterpret_cast<const tq_paged*>(handle); }
  uint32_t* pool(const Tensor& t) const {
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(1) != page_words || !t.is_contiguous())
      refuse("pool must be contiguous int32 [n_pages, " + std::to_string(page_words) + "]");
    return static_cast<uint32_t*>(t.data_ptr());
  }
};

// A page table: rows contiguous, any stride between them.
struct Table {
  int32_t* p;
  int64_t ld;
  int width;
  Table(const char* name, const Tensor& t, int64_t B) {
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != B)
      refuse(std::string(name) + " must be int32 [" + std::to_string(B) + ", max_pages]");
    width = count("the number of pages of a sequence", t.size(1));
    if (B && ((t.stride(1) != 1 && width > 1) || (B > 1 && t.stride(0) < width)))
      refuse("the rows of " + std::string(name) + " must be contiguous and apart");
    p = static_cast<int32_t*>(t.data_ptr());
    ld = std::max<int64_t>(t.stride(0), width);
  }
};

template <typename T>
T* encoded(const char* name, const Tensor& t, at::ScalarType type, int64_t n) {
  if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous())
    refuse(std::string(name) + " must be " + std::to_string(n) + " contiguous " + c10::toString(type));
  return static_cast<T*>(t.data_ptr());
}

void paged_append(const Paged& pg, const Tensor& pool, int layer, const Tensor& kcodes, const Tensor& ksigns,
                  const Tensor& knorms, const Tensor& krnorms, const Tensor& vcodes, const Tensor& vnorms,
                  const Tensor& start, const Tensor& tables, const Maybe& cu) {
  const int64_t B = count("the number of sequences", rows_of("start", start)), rows = knorms.numel(), n_tok = rows / pg.hkv;
  if (rows != n_tok * pg.hkv) refuse(std::to_string(rows) + " rows are no multiple of " + std::to_string(pg.hkv) + " heads");
  if (!cu && n_tok != B) refuse(std::to_string(n_tok) + " tokens for " + std::to_string(B) + " sequences need cu");
  const Here here(device_of({&pool, &kcodes, &ksigns, &knorms, &krnorms, &vcodes, &vnorms, &start, &tables, opt(cu)}));
  const Table t("tables", tables, B);
  uint32_t* const to = pg.pool(pool);
  const auto* c = encoded<uint32_t>("key codes", kcodes, at::kInt, rows * pg.key_words);
  const auto* s = encoded<uint32_t>("key signs", ksigns, at::kInt, rows * pg.sign_words);
  const auto* kn = encoded<float>("key norms", knorms, at::kFloat, rows);
  const auto* kr = encoded<float>("residual norms", krnorms, pg.half_rnorm ? at::kHalf : at::kFloat, rows);
  const auto* v = encoded<uint32_t>("value codes", vcodes, at::kInt, rows * pg.value_words);
  const auto* vn = encoded<float>("value norms", vnorms, at::kFloat, rows);
  const int32_t* cp = cu ? whole<int32_t>("cu", *cu, at::kInt, {B + 1}) : nullptr;
  const int32_t* sp = whole<int32_t>("start", start, at::kInt, {B});
  tq_status e;
  {
    py::gil_scoped_release go;
    e = tq_paged_append(pg.get(), to, pool.size(0), layer, c, s, kn, kr, v, vn, n_tok, (int)B, cp, sp, t.p, t.ld, t.width,
                        here.stream);
  }
  check("tq_paged_append", e);
}

std::tuple<Tensor, Maybe> paged_attention(const Paged& pg, Tensor q, const Tensor& pool, int layer, const Tensor& lens,
                                          const Tensor& tables, double scale, Maybe out, Maybe lse, Maybe ws, bool want_lse) {
  if (q.dim() != 3 || q.size(2) != pg.d) refuse("q must be [B, Hq, " + std::to_string(pg.d) + "]");
  const int64_t B = count("the number of sequences", q.size(0)), Hq = count("the number of heads", q.size(1)), d = q.size(2);
  const tq_dtype dt = dtype_of("q", q);
  const Here here(device_of({&q, &pool, &lens, &tables, opt(out), opt(lse), opt(ws)}));
  if (q.numel() && (q.stride(2) != 1 || q.stride(1) != d || (B > 1 && q.stride(0) < Hq * d))) q = q.contiguous();
  if (!out) out = at::empty(q.sizes(), q.options());
  if (!lse && want_lse) lse = at::empty({B, Hq}, q.options().dtype(at::kFloat));
  if (!ws) {
    size_t bytes = 0;
    check("tq_paged_attention_workspace_size", tq_paged_attention_workspace_size(pg.get(), (int)B, (int)Hq, &bytes));
    if (bytes) ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
  }
  const Table t("tables", tables, B);
  const uint32_t* from = pg.pool(pool);
  const int32_t* n = whole<int32_t>("lens", lens, at::kInt, {B});
  void* o = whole("out", *out, q.scalar_type(), {B, Hq, d});
  float* l = lse ? whole<float>("lse", *lse, at::kFloat, {B, Hq}) : nullptr;
  void* const w = ws ? together(*ws) : nullptr;
  tq_status e;
  {
    py::gil_scoped_release go;
    e = tq_paged_attention(pg.get(), ptr(q), dt, std::max(q.stride(0), Hq * d), (int)B, (int)Hq, from, pool.size(0), layer,
                           n, t.p, t.ld, t.width, (float)scale, o, l, w, ws ? ws->nbytes() : 0, here.stream);
  }
  check("tq_paged_attention", e);
  return {*out, want_lse ? lse : std::nullopt};
}

void paged_fork(const Paged& pg, const Tensor& pool, const Tensor& tables, const Tensor& lens, const Tensor& parents,
                const Tensor& children, const Tensor& fresh) {
  const int64_t B = count("the number of sequences", rows_of("lens", lens)), n = count("the number of forks", rows_of("parents", parents));
  const Here here(device_of({&pool, &tables, &lens, &parents, &children, &fresh}));
  const Table t("tables", tables, B);
  uint32_t* const p = pg.pool(pool);
  int32_t* const l = whole<int32_t>("lens", lens, at::kInt, {B});
  const int32_t* a = whole<int32_t>("parents", parents, at::kInt, {n});
  const int32_t* c = whole<int32_t>("children", children, at::kInt, {n});
  const int32_t* f = whole<int32_t>("fresh", fresh, at::kInt, {n});
  tq_status e;
  {
    py::gil_scoped_release go;
    e = tq_paged_fork(pg.get(), p, pool.size(0), t.p, t.ld, t.width, l, (int)B, a, c, f, (int)n, here.stream);
  }
  check("tq_paged_fork", e);
}

Tensor paged_compact(const Paged& pg, const Tensor& pool, const Tensor& tables, const Tensor& lens, Maybe tables_out,
                     Maybe n_used, Maybe ws) {
  const int64_t B = count("the number of sequences", rows_of("lens", lens));
  const Here here(device_of({&pool, &tables, &lens, opt(tables_out), opt(n_used), opt(ws)}));
  if (!tables_out) tables_out = tables;
  else if (tables_out->sizes() != tables.sizes() || tables_out->strides() != tables.strides())
    refuse("tables_out must have the shape and strides of tables");
  if (!n_used) n_used = at::empty({1}, tables.options().dtype(at::kInt));
  uint32_t* const p = pg.pool(pool);
  if (!ws) {
    size_t bytes = 0;
    check("tq_paged_compact_workspace_size", tq_paged_compact_workspace_size(pool.size(0), &bytes));
    ws = at::empty({(int64_t)bytes}, tables.options().dtype(at::kByte));
  }
  const Table t("tables", tables, B), to("tables_out", *tables_out, B);
  const int32_t* l = whole<int32_t>("lens", lens, at::kInt, {B});
  int32_t* const u = whole<int32_t>("n_used", *n_used, at::kInt, {1});
  void* const w = together(*ws);
  tq_status e;
  {
    py::gil_scoped_release go;
    e = tq_paged_compact(pg.get(), p, pool.size(0), t.p, to.p, t.ld, t.width, l, (int)B, u, w, ws->nbytes(),
                         here.stream);
  }
  check("tq_paged_compact", e);
  return *n_used;
}

}  // namespace

PYBIND11_MODULE(_torch_binding, m) {
  py::class_<Paged>(m, "Paged")
      .def(py::init([](uintptr_t handle, int64_t page_words, int64_t hkv, int64_t d, int64_t key_words, int64_t sign_words,
                       int64_t value_words, bool half_rnorm) {
        return Paged{handle, page_words, hkv, d, key_words, sign_words, value_words, half_rnorm};
      }))
      .def_readwrite("handle", &Paged::handle);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("paged_append", &paged_append);
  m.def("paged_attention", &paged_attention);
  m.def("paged_fork", &paged_fork);
  m.def("paged_compact", &paged_compact);
}
