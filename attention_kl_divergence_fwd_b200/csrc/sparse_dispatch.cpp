// sparse_dispatch.cpp - PyTorch side of the block-sparse attention calls (sparse.py).
//
// A single-token call takes 6 to 10 us on the GPU and a short training step 90 us: the same argument
// checks, allocations and autograd bookkeeping in Python cost more than the kernels (mass of one
// token 11.4 us against 8.4 with this module, its selection 10.5 against 8.2, a training step of
// 1337 tokens 148 against 100). This module checks tensors, allocates outputs and workspace on the
// current stream, calls the C entry points (whose addresses sparse.py hands over once, so that
// there is one instance of the library) and is the autograd node of sparse_attention.
#include <torch/extension.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/functions/basic_ops.h>

#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <limits>
#include <string>
#include <tuple>

#include "streamkl.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

// The C entry points.
decltype(&streamkl_block_mass) f_mass = nullptr;
decltype(&streamkl_block_mass_workspace) f_mass_ws = nullptr;
decltype(&streamkl_block_select) f_select = nullptr;
decltype(&streamkl_sparse_attn_workspace) f_attn_ws = nullptr;
decltype(&streamkl_sparse_attn_fwd) f_fwd = nullptr;
decltype(&streamkl_sparse_attn_bwd) f_bwd = nullptr;
decltype(&streamkl_status_string) f_string = nullptr;
decltype(&streamkl_device_status) f_device_status = nullptr;

template <typename F>
void set(F& f, uintptr_t address) {
  f = reinterpret_cast<F>(address);
}

void bind(const std::vector<uintptr_t>& a) {
  TORCH_CHECK(a.size() == 8, "eight entry points");
  set(f_mass, a[0]);
  set(f_mass_ws, a[1]);
  set(f_select, a[2]);
  set(f_attn_ws, a[3]);
  set(f_fwd, a[4]);
  set(f_bwd, a[5]);
  set(f_string, a[6]);
  set(f_device_status, a[7]);
}

// StreamKLError, the Python class (kept for the life of the process).
PyObject* error_class = nullptr;

// Raises a failure status as StreamKLError: out of a call from Python, or out of the backward on one
// of autograd's threads, which do not hold the interpreter and hand the error to their caller.
void check(int status, const char* where) {
  if (status == 0) return;
  TORCH_CHECK(error_class != nullptr, where, ": ", f_string(static_cast<streamkl_status>(status)));
  const bool from_python = PyGILState_Check();
  py::gil_scoped_acquire gil;
  py::object error = py::reinterpret_borrow<py::object>(error_class)(status, py::str(where));
  PyErr_SetObject(error_class, error.ptr());
  if (from_python) throw py::error_already_set();
  python_error e;
  e.persist();
  throw e;
}

void want(const char* name, const Tensor& t, at::ScalarType type, const at::Device& dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.device() == dev && t.is_contiguous(), name,
                    " must be a contiguous ", type, " tensor on ", dev);
}

void want_shape(const char* name, const Tensor& t, at::IntArrayRef shape) {
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
}

// Neither the forward nor the backward has a derivative in forward mode: a tangent would be lost.
void refuse_tangent(const Tensor& t, const char* name) {
  if (!c10::AutogradState::get_tls_state().get_fw_grad_mode()) return;
  TORCH_CHECK_NOT_IMPLEMENTED(!t._fw_grad(0).defined(), "sparse_attention: ", name,
                              " carries a forward-mode tangent; only reverse-mode gradients are "
                              "implemented");
}

int narrow(int64_t n) {
  TORCH_CHECK_VALUE(n <= std::numeric_limits<int>::max() && n >= std::numeric_limits<int>::min(),
                    n, " is out of range");
  return static_cast<int>(n);
}

// Sizes of q [B,H,N_Q,d] and k [B,H_kv,N_K,d].
struct Sizes {
  int B, H, Hkv, nq, nk, d;
};

Sizes qk_sizes(const Tensor& q, const Tensor& k) {
  TORCH_CHECK_VALUE(q.is_cuda(), "q must be on a CUDA device");
  want("q", q, at::kBFloat16, q.device());
  want("k", k, at::kBFloat16, q.device());
  TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4 && q.size(0) == k.size(0) && q.size(3) == k.size(3),
                    "q and k must be [B, heads, N, d] with one B and d");
  return {narrow(q.size(0)), narrow(q.size(1)), narrow(k.size(1)),
          narrow(q.size(2)), narrow(k.size(2)), narrow(q.size(3))};
}

const int* lens_ptr(const OptTensor& lens, const Tensor& like, int64_t B) {
  if (!lens) return nullptr;
  want("seqlens_k", *lens, at::kInt, like.device());
  want_shape("seqlens_k", *lens, {B});
  return lens->const_data_ptr<int>();
}

// Workspace sizes that the library gives; -1: sizes that it rejects.
long long accepted(long long bytes, const char* where) {
  if (bytes < 0) check(STREAMKL_ERR_UNSUPPORTED, where);
  return bytes;
}

Tensor scratch(long long bytes, const Tensor& like) {
  return bytes ? at::empty({bytes}, like.options().dtype(at::kByte)) : Tensor();
}

// Gives up the interpreter lock while it lives, where the caller holds it (autograd's threads do
// not): allocations, launches and the wait of a status check may take long or depend on work that
// another Python thread of the process has yet to queue.
class WithoutPython {
 public:
  WithoutPython() {
    if (PyGILState_Check()) release_.emplace();
  }

 private:
  std::optional<py::gil_scoped_release> release_;
};

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

cudaStream_t stream_of(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}

// t as the library takes it: contiguous and at a multiple of 16 bytes, a copy where it is not (a view
// may begin anywhere in its storage).
Tensor laid_out(const Tensor& t) {
  const bool contiguous = t.is_contiguous();
  if (contiguous && reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0) return t;
  const WithoutPython free;
  return contiguous ? t.clone(at::MemoryFormat::Contiguous) : t.contiguous();
}

// The device's status once the stream of t is done, if asked for.
int device_status(bool on, const Tensor& t) { return on ? f_device_status(stream_of(t)) : 0; }

Tensor block_mass(const Tensor& q_in, const Tensor& k_in, double scale, bool causal,
                  const OptTensor& lse_in, const OptTensor& lens, bool check_status) {
  const Tensor q = laid_out(q_in), k = laid_out(k_in);
  const OptTensor lse = lse_in ? OptTensor(laid_out(*lse_in)) : std::nullopt;
  const Sizes s = qk_sizes(q, k);
  const int* n = lens_ptr(lens, q, s.B);
  if (lse) {
    want("lse", *lse, at::kFloat, q.device());
    want_shape("lse", *lse, {s.B, s.H, s.nq});
  }
  const c10::cuda::CUDAGuard guard(q.device());
  const long long bytes =
      lse ? 0 : accepted(f_mass_ws(s.B, s.H, s.Hkv, s.nq, s.nk, s.d), "block_mass");
  Tensor mass;
  int status;
  {
    const WithoutPython free;
    const Tensor ws = scratch(bytes, q);
    mass = at::empty({s.B, s.Hkv, s.nq, (s.nk + 63ll) / 64}, q.options().dtype(at::kFloat));
    status = f_mass(q.const_data_ptr(), k.const_data_ptr(), n, s.B, s.H, s.Hkv, s.nq, s.nk, s.d,
                    static_cast<float>(scale), causal, lse ? lse->const_data_ptr<float>() : nullptr,
                    ptr(ws), bytes, mass.data_ptr<float>(), stream_of(q));
    if (status == 0) status = device_status(check_status, q);
  }
  check(status, "block_mass");
  return mass;
}

Tensor select_blocks(const Tensor& mass_in, int64_t n_k, int64_t topk, bool causal, int64_t n_first,
                     int64_t n_last, const OptTensor& lens, bool check_status) {
  const Tensor mass = laid_out(mass_in);
  TORCH_CHECK_VALUE(mass.dim() == 4, "mass must be [B, H_sel, N_Q, NB]");
  TORCH_CHECK_VALUE(n_k >= 0 && (n_k + 63) / 64 == mass.size(3), "mass has ", mass.size(3),
                    " blocks, n_k = ", n_k, " keys make ", (n_k + 63) / 64);
  TORCH_CHECK_VALUE(mass.is_cuda(), "mass must be on a CUDA device");
  want("mass", mass, at::kFloat, mass.device());
  const int* n = lens_ptr(lens, mass, mass.size(0));
  const int B = narrow(mass.size(0)), Hsel = narrow(mass.size(1)), nq = narrow(mass.size(2)),
            nk = narrow(n_k), k = narrow(topk), first = narrow(n_first), last = narrow(n_last);
  const c10::cuda::CUDAGuard guard(mass.device());
  Tensor idx;
  int status;
  {
    const WithoutPython free;
    idx = at::empty({B, Hsel, nq, k > 0 ? k : 0}, mass.options().dtype(at::kInt));
    status = f_select(mass.const_data_ptr<float>(), n, B, Hsel, nq, nk, causal, k, first, last,
                      idx.data_ptr<int>(), stream_of(mass));
    if (status == 0) status = device_status(check_status, mass);
  }
  check(status, "select_blocks");
  return idx;
}

std::tuple<Tensor, Tensor> attn_fwd(const Tensor& q, const Tensor& k, const Tensor& v,
                                    const Tensor& idx, const OptTensor& lens, double scale,
                                    bool causal, bool with_lse, bool check_status) {
  const Sizes s = qk_sizes(q, k);
  want("v", v, at::kBFloat16, q.device());
  want_shape("v", v, k.sizes());
  want("block_idx", idx, at::kInt, q.device());
  TORCH_CHECK_VALUE(idx.dim() == 4, "block_idx must be [B, H_sel, N_Q, topk]");
  want_shape("block_idx", idx, {s.B, idx.size(1), s.nq, idx.size(3)});
  const int Hsel = narrow(idx.size(1)), topk = narrow(idx.size(3));
  const int* n = lens_ptr(lens, q, s.B);
  const c10::cuda::CUDAGuard guard(q.device());
  const long long bytes =
      accepted(f_attn_ws(s.B, s.H, s.Hkv, Hsel, s.nq, s.nk, s.d, topk, 0), "sparse_attention");
  Tensor out, lse;
  int status;
  {
    const WithoutPython free;
    out = at::empty_like(q);
    if (with_lse) lse = at::empty({s.B, s.H, s.nq}, q.options().dtype(at::kFloat));
    const Tensor ws = scratch(bytes, q);
    status = f_fwd(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(),
                   idx.const_data_ptr<int>(), n, s.B, s.H, s.Hkv, Hsel, s.nq, s.nk, s.d, topk,
                   static_cast<float>(scale), causal, ptr(ws), bytes, out.data_ptr(),
                   with_lse ? lse.data_ptr<float>() : nullptr, stream_of(q));
    if (status == 0) status = device_status(check_status, q);
  }
  check(status, "sparse_attention forward");
  return {out, lse};
}

bool capturing() {
  return c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None;
}

// A gradient goes on to the stream on which the function that made the tensor ran, or, for a leaf, on
// which the oldest graph that still holds it began. A backward captured meanwhile would make that
// stream wait for the capture, which for the default stream CUDA takes as an error on a thread of
// autograd's, and the process ends. So leaves of such a graph are refused while capturing;
// other tensors are noted (the text for a refusal is returned), because a captured forward alone
// is sound: their backward is refused.
std::string check_capture(const Tensor& t, const char* name) {
  if (!t.requires_grad()) return {};
  const auto node = t.is_leaf() ? torch::autograd::impl::try_get_grad_accumulator(t)
                                : torch::autograd::impl::gradient_edge(t).function;
  if (node == nullptr) return {};
  const auto stream = node->stream();
  if (!stream ||
      c10::cuda::CUDAStream(*stream) != c10::cuda::getDefaultCUDAStream(t.device().index()))
    return {};
  const std::string part = std::string("sparse_attention: ") + name +
                           " is part of a graph made on the default stream; release that graph "
                           "(or pass " + name + ".detach().requires_grad_()) ";
  TORCH_CHECK(!t.is_leaf(), part, "before capturing a CUDA graph");
  return part;
}

// Attention over selected blocks as an autograd node; gradients flow to q, k and v.
struct SparseAttention : torch::autograd::Function<SparseAttention> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& q,
                                                const Tensor& k, const Tensor& v, const Tensor& idx,
                                                const OptTensor& lens, double scale, bool causal,
                                                bool check_status, const std::string& eager) {
    at::AutoDispatchBelowADInplaceOrView below;
    auto [out, lse] = attn_fwd(q, k, v, idx, lens, scale, causal, true, check_status);
    ctx->save_for_backward({q, k, v, out, lse, idx, lens ? *lens : Tensor()});
    ctx->saved_data["scale"] = scale;
    ctx->saved_data["causal"] = causal;
    ctx->saved_data["check"] = check_status;
    if (!eager.empty()) ctx->saved_data["eager"] = eager;
    ctx->mark_non_differentiable({lse});
    ctx->set_materialize_grads(false);
    return {out, lse};
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx,
                                                 torch::autograd::variable_list grads) {
    torch::autograd::variable_list none(9);
    if (!grads[0].defined()) return none;
    refuse_tangent(grads[0], "dout");
    const auto eager = ctx->saved_data.find("eager");
    TORCH_CHECK(eager == ctx->saved_data.end() || !capturing(), eager->second.toStringRef(),
                "before capturing its backward");
    const auto saved = ctx->get_saved_variables();
    const Tensor &q = saved[0], &k = saved[1], &v = saved[2], &out = saved[3], &lse = saved[4],
                 &idx = saved[5];
    const OptTensor lens = saved[6].defined() ? OptTensor(saved[6]) : std::nullopt;
    const c10::cuda::CUDAGuard guard(q.device());
    const Sizes s = qk_sizes(q, k);
    const int Hsel = narrow(idx.size(1)), topk = narrow(idx.size(3));
    const int* n = lens_ptr(lens, q, s.B);
    const long long bytes = accepted(f_attn_ws(s.B, s.H, s.Hkv, Hsel, s.nq, s.nk, s.d, topk, 1),
                                     "sparse_attention backward");
    Tensor dq, dk, dv;
    int status;
    {
      const WithoutPython free;
      const Tensor dout = laid_out(grads[0].to(at::kBFloat16));
      dq = at::empty_like(q);
      dk = at::empty_like(k);
      dv = at::empty_like(v);
      const Tensor ws = scratch(bytes, q);
      status = f_bwd(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), out.const_data_ptr(),
                     lse.const_data_ptr<float>(), dout.const_data_ptr(), idx.const_data_ptr<int>(), n,
                     s.B, s.H, s.Hkv, Hsel, s.nq, s.nk, s.d, topk,
                     static_cast<float>(ctx->saved_data["scale"].toDouble()),
                     ctx->saved_data["causal"].toBool(), ptr(ws), bytes, dq.data_ptr(), dk.data_ptr(),
                     dv.data_ptr(), stream_of(q));
      if (status == 0) status = device_status(ctx->saved_data["check"].toBool(), q);
    }
    check(status, "sparse_attention backward");
    torch::autograd::variable_list d{dq, dk, dv};
    if (at::GradMode::is_enabled()) {  // create_graph: an error for whoever differentiates these
      for (Tensor& t : d) t.set_requires_grad(true);
      d = torch::autograd::DelayedError("sparse_attention is differentiable once", 3).apply(std::move(d));
    }
    std::copy(d.begin(), d.end(), none.begin());
    return none;
  }
};

std::tuple<Tensor, Tensor> sparse_attention(const Tensor& q, const Tensor& k, const Tensor& v,
                                            const Tensor& idx, const OptTensor& lens, double scale,
                                            bool causal, bool with_lse, bool check_status) {
  refuse_tangent(q, "q");
  refuse_tangent(k, "k");
  refuse_tangent(v, "v");
  const Tensor qc = laid_out(q), kc = laid_out(k), vc = laid_out(v), ic = laid_out(idx);
  if (at::GradMode::is_enabled() && (q.requires_grad() || k.requires_grad() || v.requires_grad())) {
    const c10::OptionalDeviceGuard guard(q.device());
    std::string eager;
    if (q.is_cuda() && capturing())
      for (const std::string& e : {check_capture(q, "q"), check_capture(k, "k"), check_capture(v, "v")})
        if (eager.empty()) eager = e;
    auto r = SparseAttention::apply(qc, kc, vc, ic, lens, scale, causal, check_status, eager);
    return {r[0], r[1]};
  }
  return attn_fwd(qc, kc, vc, ic, lens, scale, causal, with_lse, check_status);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.attr("built_for") = BUILT_FOR;  // sparse.py looks for this text in the file
  m.def("bind", &bind);
  m.def("block_mass", &block_mass);
  m.def("select_blocks", &select_blocks);
  m.def("sparse_attention", &sparse_attention);
  m.def("raise_as", [](py::object error) { error_class = error.release().ptr(); });
  m.def("check", [](int status, const std::string& where) { check(status, where.c_str()); });
}
