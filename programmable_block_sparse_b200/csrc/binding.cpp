// Python binding of the calls that are made once a layer and token: query / key
// preparation, cache appends and attention over an e4m3 cache.  It does what
// the ctypes functions of __init__.py do for the other entry points -- tensors
// become pointers, sizes and strides, specification dicts become the C structs,
// missing outputs and workspaces are allocated -- but in C++, because a Python
// function that packs those structs takes longer than the smallest of these
// kernels runs (a preparation of 32 tokens: 16 us a call from Python, 7.5 from
// here, 3.7 on the device).
// Tensors whose extent the library cannot know are checked here.
#include <ATen/cuda/CUDAContext.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/extension.h>

#include <string>

#include "flexattn.h"

namespace py = pybind11;
using at::Tensor;

namespace {

[[noreturn]] void raise(int status, const std::string& message) {
  py::object cls = py::module_::import("programmable_block_sparse_b200").attr("FlexAttnError");
  py::object err = cls(status, message);
  PyErr_SetObject(cls.ptr(), err.ptr());
  throw py::error_already_set();
}
void check(int status) {
  if (status != FA_OK) raise(status, flexattn_last_error());
}

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16:
      return FA_DTYPE_BF16;
    case at::kFloat:
      return FA_DTYPE_F32;
    case at::kFloat8_e4m3fn:
      return FA_DTYPE_E4M3;
    default:
      return -1;
  }
}
std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// The device of a call: its first tensor's, which has to be a CUDA device.
c10::Device cuda_device(const Tensor& t, const char* name) {
  if (dtype_code(t.scalar_type()) < 0) raise(FA_ERR_DTYPE, std::string(name) + ": unsupported dtype " + toString(t.scalar_type()));
  if (!t.is_cuda()) raise(FA_ERR_PARAM, std::string(name) + " is on " + t.device().str() + ", expected a CUDA device");
  return t.device();
}

fa_tensor view(const Tensor& t, const char* name, c10::Device dev) {
  const int code = dtype_code(t.scalar_type());
  if (code < 0) raise(FA_ERR_DTYPE, std::string(name) + ": unsupported dtype " + toString(t.scalar_type()));
  if (t.dim() != 4) raise(FA_ERR_SHAPE, std::string(name) + ": expected a 4-D tensor, got shape " + text(t.sizes()));
  if (t.device() != dev) raise(FA_ERR_PARAM, std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  fa_tensor s;
  s.data = t.data_ptr();
  s.dtype = code;
  s.reserved = 0;
  for (int i = 0; i < 4; ++i) {
    s.size[i] = t.size(i);
    s.stride[i] = t.stride(i);
  }
  return s;
}

// Address of a contiguous tensor of a given type and shape (the library reads
// it without knowing its extent).
void* array(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  if (t.scalar_type() != type)
    raise(FA_ERR_DTYPE, std::string(name) + ": expected " + toString(type) + ", got " + toString(t.scalar_type()));
  if (t.sizes() != shape) raise(FA_ERR_SHAPE, std::string(name) + ": expected shape " + text(shape) + ", got " + text(t.sizes()));
  if (t.device() != dev) raise(FA_ERR_PARAM, std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  if (!t.is_contiguous()) raise(FA_ERR_ALIGN, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

// Entries of a specification dict: a borrowed reference, or null where the key
// is absent or its value is None.
PyObject* entry(const py::handle& spec, const char* key) {
  if (!PyDict_Check(spec.ptr())) raise(FA_ERR_PARAM, std::string("expected a dict with ") + key);
  PyObject* v = PyDict_GetItemString(spec.ptr(), key);
  return v == nullptr || v == Py_None ? nullptr : v;
}
Tensor tensor(PyObject* v, const char* name) {
  if (!THPVariable_Check(v)) raise(FA_ERR_PARAM, std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(v);
}
Tensor required(const py::handle& spec, const char* key) {
  PyObject* v = entry(spec, key);
  if (!v) raise(FA_ERR_NULL, std::string(key) + " is missing");
  return tensor(v, key);
}
int64_t integer(PyObject* v) { return v ? py::handle(v).cast<int64_t>() : 0; }
bool given(const py::object& o) { return !o.is_none(); }

const fa_head_norm* norm_of(const py::object& spec, const char* name, int64_t D, c10::Device dev, fa_head_norm* n) {
  if (!given(spec)) return nullptr;
  PyObject *w = entry(spec, "weight"), *eps = entry(spec, "eps");
  n->weight = nullptr;
  n->weight_dtype = FA_DTYPE_F32;
  n->eps = eps ? py::handle(eps).cast<float>() : 1e-6f;
  if (w) {
    const Tensor t = tensor(w, name);
    n->weight = array(t, name, t.scalar_type(), {D}, dev);
    n->weight_dtype = dtype_code(t.scalar_type());
  }
  return n;
}

const fa_rope* rope_of(const py::object& spec, int64_t B, int64_t N, c10::Device dev, fa_rope* r) {
  if (!given(spec)) return nullptr;
  const Tensor f = required(spec, "inv_freq");
  const int64_t half = f.numel();
  *r = fa_rope{};
  r->inv_freq = static_cast<const float*>(array(f, "inv_freq", at::kFloat, {half}, dev));
  r->rot_dim = static_cast<int32_t>(2 * half);
  PyObject* next = entry(spec, "interleaved");
  r->interleaved = next && PyObject_IsTrue(next) ? 1 : 0;
  if (PyObject* p = entry(spec, "pos")) {
    const Tensor pos = tensor(p, "rope pos");
    const int64_t rows = pos.dim() == 2 ? pos.size(0) : 1;
    if (rows != 1 && rows != B)
      raise(FA_ERR_BATCH, "rope pos: " + std::to_string(rows) + " rows, expected 1 or " + std::to_string(B));
    r->pos = static_cast<const int32_t*>(pos.dim() == 2 ? array(pos, "rope pos", at::kInt, {rows, N}, dev)
                                                        : array(pos, "rope pos", at::kInt, {N}, dev));
    r->pos_batch = static_cast<int32_t>(rows);
  }
  return r;
}

// A call's device and stream, current for as long as this lives: a stream that
// the caller names is also the one that new outputs and workspaces belong to, so
// that a workspace freed on return is not handed to other work before the
// kernels on that stream are done with it.
class Launch {
 public:
  Launch(c10::Device dev, const py::object& stream) : guard_(dev) {
    if (!given(stream)) return;
    const py::object handle = PyLong_Check(stream.ptr()) ? stream : py::object(stream.attr("cuda_stream"));
    const auto raw = reinterpret_cast<cudaStream_t>(handle.cast<uintptr_t>());
    on_.reset_stream(raw ? at::cuda::getStreamFromExternal(raw, dev.index())
                         : at::cuda::getDefaultCUDAStream(dev.index()));
  }
  void* stream(c10::Device dev) const { return at::cuda::getCurrentCUDAStream(dev.index()).stream(); }

 private:
  c10::cuda::CUDAGuard guard_;
  c10::cuda::OptionalCUDAStreamGuard on_;
};

// A workspace that the caller gave: contiguous, on the call's device.
Tensor workspace_of(const py::object& o, c10::Device dev) {
  Tensor t = tensor(o.ptr(), "workspace");
  if (t.device() != dev) raise(FA_ERR_PARAM, "workspace is on " + t.device().str() + ", expected " + dev.str());
  if (!t.is_contiguous()) raise(FA_ERR_ALIGN, "workspace must be contiguous");
  return t;
}

Tensor like(const Tensor& x, at::ScalarType type) { return at::empty(x.sizes(), x.options().dtype(type)); }

// An optional tensor argument.
struct Given {
  Tensor t;
  fa_tensor s;
  bool on = false;
  void take(const py::object& o, const char* name, c10::Device dev) {
    if (!given(o)) return;
    t = tensor(o.ptr(), name);
    s = view(t, name, dev);
    on = true;
  }
  void take_or_new(const py::object& o, const Tensor& as, at::ScalarType type, const char* name, c10::Device dev) {
    t = given(o) ? tensor(o.ptr(), name) : like(as, type);
    s = view(t, name, dev);
    on = true;
  }
  const fa_tensor* ptr() const { return on ? &s : nullptr; }
  py::object object() const { return on ? py::cast(t) : py::none(); }
};

py::tuple qk_norm_rope(const py::object& q, const py::object& k, const py::object& q_norm, const py::object& k_norm,
                       const py::object& rope, const py::object& q_out, const py::object& k_out,
                       const py::object& stream) {
  if (!given(q) && !given(k)) raise(FA_ERR_NULL, "q and k are both None");
  const Tensor x = given(q) ? tensor(q.ptr(), "q") : tensor(k.ptr(), "k");
  const c10::Device dev = cuda_device(x, given(q) ? "q" : "k");
  const Launch launch(dev, stream);
  Given in[2], out[2];
  in[0].take(q, "q", dev);
  in[1].take(k, "k", dev);
  if (in[0].on) out[0].take_or_new(q_out, in[0].t, in[0].t.scalar_type(), "q_out", dev);
  if (in[1].on) out[1].take_or_new(k_out, in[1].t, in[1].t.scalar_type(), "k_out", dev);
  if (x.dim() != 4) raise(FA_ERR_SHAPE, "expected 4-D tensors");
  fa_head_norm qn, kn;
  fa_rope rp;
  const fa_head_norm* pq = norm_of(q_norm, "q_norm weight", x.size(3), dev, &qn);
  const fa_head_norm* pk = norm_of(k_norm, "k_norm weight", x.size(3), dev, &kn);
  const fa_rope* pr = rope_of(rope, x.size(0), x.size(2), dev, &rp);
  void* st = launch.stream(dev);
  int status;
  {
    py::gil_scoped_release nogil;
    status = flexattn_qk_norm_rope(in[0].ptr(), in[1].ptr(), out[0].ptr(), out[1].ptr(), pq, pk, pr, st);
  }
  check(status);
  return py::make_tuple(given(q) ? out[0].object() : q_out, given(k) ? out[1].object() : k_out);
}

py::tuple qk_norm_rope_backward(const py::object& q, const py::object& k, const py::object& dq_out,
                                const py::object& dk_out, const py::object& q_norm, const py::object& k_norm,
                                const py::object& rope, const py::object& dq, const py::object& dk,
                                const py::object& grad_dtype, bool weight_grads, const py::object& workspace,
                                const py::object& stream) {
  if (!given(dq_out) && !given(dk_out)) raise(FA_ERR_NULL, "dq_out and dk_out are both None");
  const Tensor g = given(dq_out) ? tensor(dq_out.ptr(), "dq_out") : tensor(dk_out.ptr(), "dk_out");
  const c10::Device dev = cuda_device(g, given(dq_out) ? "dq_out" : "dk_out");
  const Launch launch(dev, stream);
  if (g.dim() != 4) raise(FA_ERR_SHAPE, "expected 4-D tensors");
  const int64_t D = g.size(3);
  const py::object *xs[2] = {&q, &k}, *dys[2] = {&dq_out, &dk_out}, *dxs[2] = {&dq, &dk}, *norms[2] = {&q_norm, &k_norm};
  const char *xn[2] = {"q", "k"}, *dyn[2] = {"dq_out", "dk_out"}, *dxn[2] = {"dq", "dk"};
  Given x[2], dy[2], dx[2];
  Tensor dw[2];
  bool sums = false;
  for (int i = 0; i < 2; ++i) {
    if (given(*norms[i])) x[i].take(*xs[i], xn[i], dev);
    dy[i].take(*dys[i], dyn[i], dev);
    if (!dy[i].on) continue;
    const at::ScalarType type = given(grad_dtype) ? grad_dtype.cast<at::ScalarType>() : dy[i].t.scalar_type();
    dx[i].take_or_new(*dxs[i], dy[i].t, type, dxn[i], dev);
    if (weight_grads && given(*norms[i])) {
      dw[i] = at::empty({D}, g.options().dtype(at::kFloat));
      sums = true;
    }
  }
  Tensor ws;
  size_t bytes = 0;
  if (given(workspace)) {
    ws = workspace_of(workspace, dev);
    bytes = ws.nbytes();
  } else if (sums) {
    check(flexattn_qk_norm_rope_backward_workspace_size(static_cast<int32_t>(D), 1, &bytes));
    ws = at::empty({static_cast<int64_t>(bytes)}, g.options().dtype(at::kByte));
  }
  fa_head_norm qn, kn;
  fa_rope rp;
  const fa_head_norm* pq = norm_of(q_norm, "q_norm weight", D, dev, &qn);
  const fa_head_norm* pk = norm_of(k_norm, "k_norm weight", D, dev, &kn);
  const fa_rope* pr = rope_of(rope, g.size(0), g.size(2), dev, &rp);
  void* st = launch.stream(dev);
  float* pw[2];
  for (int i = 0; i < 2; ++i) pw[i] = dw[i].defined() ? dw[i].data_ptr<float>() : nullptr;
  void* pws = ws.defined() ? ws.data_ptr() : nullptr;
  int status;
  {
    py::gil_scoped_release nogil;
    status = flexattn_qk_norm_rope_backward(x[0].ptr(), x[1].ptr(), dy[0].ptr(), dy[1].ptr(), dx[0].ptr(), dx[1].ptr(),
                                            pw[0], pw[1], pq, pk, pr, pws, bytes, st);
  }
  check(status);
  auto grad = [&](int i) { return dw[i].defined() ? py::cast(dw[i]) : py::object(py::none()); };
  return py::make_tuple(dy[0].on ? dx[0].object() : dq, dy[1].on ? dx[1].object() : dk, grad(0), grad(1));
}

// Shape of a pool's scales.
std::array<int64_t, 3> scale_shape(const fa_tensor& pool, int64_t block) {
  return {pool.size[0], pool.size[1], block > 0 ? (pool.size[2] + block - 1) / block : 0};
}

py::object cache_append(const Tensor& k, const Tensor& v, const py::dict& cache, const py::object& k_norm,
                        const py::object& rope, const py::object& q, const py::object& q_norm, const py::object& q_out,
                        const py::object& stream) {
  const c10::Device dev = cuda_device(k, "k");
  const Launch launch(dev, stream);
  const fa_tensor ks = view(k, "k", dev), vs = view(v, "v", dev);
  const int64_t B = k.size(0), N = k.size(2), E = k.size(3);
  const Tensor kp = required(cache, "k"), vp = required(cache, "v");
  fa_kv_cache c{};
  c.k = view(kp, "cache k", dev);
  c.v = view(vp, "cache v", dev);
  c.cache_len = static_cast<const int32_t*>(array(required(cache, "cache_len"), "cache_len", at::kInt, {B}, dev));
  if (PyObject* o = entry(cache, "new_len"))
    c.new_len = static_cast<const int32_t*>(array(tensor(o, "new_len"), "new_len", at::kInt, {B}, dev));
  if (PyObject* o = entry(cache, "page_table")) {
    const Tensor t = tensor(o, "page_table");
    const int64_t pages = t.dim() ? t.size(-1) : 0;
    c.page_table = static_cast<const int32_t*>(array(t, "page_table", at::kInt, {B, pages}, dev));
    c.pages_per_seq = static_cast<int32_t>(pages);
  }
  PyObject *sk = entry(cache, "k_scale"), *sv = entry(cache, "v_scale");
  if (sk || sv) {
    c.scale_block = static_cast<int32_t>(integer(entry(cache, "scale_block")));
    if (sk) c.k_scale = static_cast<float*>(array(tensor(sk, "k_scale"), "k_scale", at::kFloat, scale_shape(c.k, c.scale_block), dev));
    if (sv) c.v_scale = static_cast<float*>(array(tensor(sv, "v_scale"), "v_scale", at::kFloat, scale_shape(c.v, c.scale_block), dev));
  }
  Given in, out;
  in.take(q, "q", dev);
  if (in.on) out.take_or_new(q_out, in.t, in.t.scalar_type(), "q_out", dev);
  fa_head_norm qn, kn;
  fa_rope rp;
  const fa_head_norm* pk = norm_of(k_norm, "k_norm weight", E, dev, &kn);
  const fa_head_norm* pq = norm_of(q_norm, "q_norm weight", E, dev, &qn);
  const fa_rope* pr = rope_of(rope, B, N, dev, &rp);
  void* st = launch.stream(dev);
  int status;
  {
    py::gil_scoped_release nogil;
    status = flexattn_cache_append(&ks, &vs, &c, pk, pr, in.ptr(), out.ptr(), pq, st);
  }
  check(status);
  return in.on ? out.object() : q_out;
}

// k, v, their scales and page table, as both calls below take them.
struct Fp8Args {
  c10::Device dev;
  fa_tensor q, k, v;
  fa_kv_quant quant{};
  fa_block_mask bm{};
  fa_forward_options opt{};
  Fp8Args(const Tensor& qt, const Tensor& kt, const Tensor& vt, const py::object& mask, const py::dict& spec,
          const py::object& paged)
      : dev(cuda_device(qt, "q")), q(view(qt, "q", dev)), k(view(kt, "k", dev)), v(view(vt, "v", dev)) {
    quant.scale_block = static_cast<int32_t>(integer(entry(spec, "scale_block")));
    quant.k_scale = static_cast<const float*>(
        array(required(spec, "k_scale"), "k_scale", at::kFloat, scale_shape(k, quant.scale_block), dev));
    quant.v_scale = static_cast<const float*>(
        array(required(spec, "v_scale"), "v_scale", at::kFloat, scale_shape(v, quant.scale_block), dev));
    auto number = [&](const char* n) { return mask.attr(n).cast<int32_t>(); };
    bm.B = number("B");
    bm.H = number("H");
    bm.L = number("L");
    bm.S = number("S");
    bm.BM = number("BM");
    bm.BN = number("BN");
    bm.Mb = number("Mb");
    bm.Nb = number("Nb");
    auto list = [&](const char* n, bool indices) {
      const Tensor t = tensor(py::object(mask.attr(n)).ptr(), n);
      const int64_t B = bm.B, H = bm.H, M = bm.Mb, Nn = bm.Nb;
      return static_cast<int32_t*>(indices ? array(t, n, at::kInt, {B, H, M, Nn}, dev) : array(t, n, at::kInt, {B, H, M}, dev));
    };
    bm.kv_num_blocks = list("kv_num_blocks", false);
    bm.kv_indices = list("kv_indices", true);
    bm.full_kv_num_blocks = list("full_kv_num_blocks", false);
    bm.full_kv_indices = list("full_kv_indices", true);
    if (given(paged)) {
      const Tensor t = required(paged, "page_table");
      const int64_t pages = t.dim() ? t.size(-1) : 0;
      opt.page_table = static_cast<const int32_t*>(array(t, "page_table", at::kInt, {qt.size(0), pages}, dev));
      opt.page_size = static_cast<int32_t>(integer(entry(paged, "page_size")));
      opt.pages_per_seq = static_cast<int32_t>(pages);
    }
  }
};

size_t forward_fp8_workspace_size(const Tensor& q, const Tensor& k, const Tensor& v, const py::object& block_mask,
                                  const py::dict& quant, int split_kv, const py::object& paged) {
  const Fp8Args a(q, k, v, block_mask, quant, paged);
  const c10::cuda::CUDAGuard guard(a.dev);
  size_t n = 0;
  check(flexattn_forward_fp8_workspace_size(&a.q, &a.k, &a.v, &a.quant, &a.bm, split_kv, &a.opt, &n));
  return n;
}

// score_mod and mask_mod: addresses of the structs that __init__.py made.
py::tuple forward_fp8(const Tensor& q, const Tensor& k, const Tensor& v, const py::object& block_mask,
                      const py::dict& quant, uintptr_t score_mod, uintptr_t mask_mod, double scale, bool enable_gqa,
                      const py::object& out, const py::object& lse, int split_kv, const py::object& workspace,
                      const py::object& stream, const py::object& out_dtype, const py::object& max_scores,
                      bool rows_safe, int64_t wait_cycles, const py::object& paged) {
  Fp8Args a(q, k, v, block_mask, quant, paged);
  const Launch launch(a.dev, stream);
  const int64_t B = q.size(0), Hq = q.size(1), L = q.size(2), Ev = v.size(3);
  const at::ScalarType type = given(out_dtype) ? out_dtype.cast<at::ScalarType>() : q.scalar_type();
  const Tensor o = given(out) ? tensor(out.ptr(), "out") : at::empty({B, Hq, L, Ev}, q.options().dtype(type));
  const fa_tensor os = view(o, "out", a.dev);
  // True: a new fp32 (B, Hq, L) tensor; a tensor: that one; None or False: none
  auto rows = [&](const py::object& arg, const char* name) {
    if (!given(arg) || arg.ptr() == Py_False) return Tensor();
    if (arg.ptr() == Py_True) return at::empty({B, Hq, L}, q.options().dtype(at::kFloat));
    Tensor t = tensor(arg.ptr(), name);
    array(t, name, at::kFloat, {B, Hq, L}, a.dev);
    return t;
  };
  const Tensor tl = rows(lse, "lse"), tm = rows(max_scores, "max_scores");
  a.opt.max_scores = tm.defined() ? tm.data_ptr<float>() : nullptr;
  a.opt.wait_cycles = wait_cycles;
  a.opt.flags = rows_safe ? FA_FLAG_ROWS_GUARANTEED_SAFE : 0;
  Tensor ws;
  size_t bytes = 0;
  if (given(workspace)) {
    ws = workspace_of(workspace, a.dev);
    bytes = ws.nbytes();
  } else {
    check(flexattn_forward_fp8_workspace_size(&a.q, &a.k, &a.v, &a.quant, &a.bm, split_kv, &a.opt, &bytes));
    if (bytes) ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
  }
  void* st = launch.stream(a.dev);
  float* pl = tl.defined() ? tl.data_ptr<float>() : nullptr;
  void* pws = ws.defined() ? ws.data_ptr() : nullptr;
  int status;
  {
    py::gil_scoped_release nogil;
    status = flexattn_forward_fp8(&a.q, &a.k, &a.v, &a.quant, &os, pl, static_cast<float>(scale), enable_gqa ? 1 : 0,
                                  reinterpret_cast<const fa_score_mod*>(score_mod),
                                  reinterpret_cast<const fa_mask_mod*>(mask_mod), &a.bm, split_kv, &a.opt, pws, bytes, st);
  }
  check(status);
  const py::object rl = tl.defined() ? py::cast(tl) : py::object(py::none());
  if (tm.defined()) return py::make_tuple(o, rl, tm);
  return py::make_tuple(o, rl);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_backward", &qk_norm_rope_backward);
  m.def("cache_append", &cache_append);
  m.def("forward_fp8_workspace_size", &forward_fp8_workspace_size);
  m.def("forward_fp8", &forward_fp8);
}
