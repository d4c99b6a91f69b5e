// Torch binding of the language-model operators: checks of tensors, output
// and scratch allocation on the current stream, and the call of the C entry
// (include/okls.h).  It computes nothing.  A call costs a few microseconds of
// host time, where the same in Python cost 15 to 25 (one token's norm: 20).
//
// Wrong tensors raise ValueError; what the C entry refuses raises OklsError.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <atomic>
#include <optional>
#include <tuple>

#include "../../include/okls.h"

namespace {

namespace py = pybind11;
using at::Tensor;
typedef std::optional<Tensor> Maybe;

constexpr int64_t kGroup = 128;

PyObject* g_okls_error = nullptr;  // _lib.OklsError

#define REFUSE(cond, ...) TORCH_CHECK_VALUE(!(cond), "okls.lm: ", __VA_ARGS__)

void check(okls_status s) {
  if (s == OKLS_OK) return;
  py::object args = py::make_tuple(static_cast<int>(s), std::string(okls_last_error()));
  PyErr_SetObject(g_okls_error, args.ptr());
  throw py::error_already_set();
}

int float_code(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return OKLS_F32;
  if (t == at::kBFloat16) return OKLS_BF16;
  REFUSE(true, name, " must be fp32 or bf16, not ", t);
  return -1;
}

// A tensor as rows x columns with a row pitch, without a copy.
struct Mat {
  void* p;
  int64_t rows, cols, ld;
};

Mat matrix(const Tensor& t, const char* name) {
  REFUSE(!t.is_cuda(), name, " must be on a CUDA device");
  const int64_t d = t.dim();
  REFUSE(d == 0, name, " needs at least one dimension");
  const int64_t cols = t.size(d - 1);
  int64_t rows = 1;
  for (int64_t i = 0; i + 1 < d; ++i) rows *= t.size(i);
  Mat m = {t.data_ptr(), rows, cols, cols};
  if (t.numel() == 0 || t.is_contiguous()) return m;
  REFUSE(cols > 1 && t.stride(d - 1) != 1, "the last dimension of ", name, " must be contiguous");
  // the leading dimensions fold when each steps over the ones after it
  int64_t step = -1, span = 0;
  for (int64_t i = d - 2; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (step < 0) {
      step = span = t.stride(i);
    } else {
      REFUSE(t.stride(i) != span, "the leading dimensions of ", name, " do not fold into rows without a copy");
    }
    span *= t.size(i);
  }
  if (step >= 0) m.ld = step;
  return m;
}

Mat plain_matrix(const Tensor& t, const char* name, int64_t rows, int64_t cols) {
  REFUSE(t.dim() != 2 || t.size(0) != rows || t.size(1) != cols, name, " must be a matrix of shape (", rows, ", ", cols, ")");
  return matrix(t, name);
}

const void* vector(const Tensor& t, const char* name, int64_t count) {
  REFUSE(!t.is_cuda(), name, " must be on a CUDA device");
  REFUSE(!t.is_contiguous(), name, " must be contiguous");
  REFUSE(t.numel() != count, name, " must hold ", count, " values, not ", t.numel());
  return t.data_ptr();
}

float* floats(const Tensor& t, const char* name, int64_t count) {
  REFUSE(t.scalar_type() != at::kFloat, name, " must be fp32, not ", t.scalar_type());
  return static_cast<float*>(const_cast<void*>(vector(t, name, count)));
}

int ids_code(const Tensor& t, int64_t count) {
  REFUSE(t.scalar_type() != at::kInt && t.scalar_type() != at::kLong, "ids must be int32 or int64, not ", t.scalar_type());
  vector(t, "ids", count);
  return t.scalar_type() == at::kLong;
}

void same_device(const Tensor& a, const Tensor& b) {
  REFUSE(a.device() != b.device(), "tensors on ", a.device(), " and ", b.device());
}
void same_device(const Tensor& a, const Maybe& b) {
  if (b) same_device(a, *b);
}

// A tensor of the caller that a call writes over.  Autograd learns of the write
// from the tensor's version, by which a backward that saved the tensor finds
// out; it cannot learn of a new value of a tensor that requires a gradient.
void writable(const Tensor& t, const char* name) {
  REFUSE(at::GradMode::is_enabled() && t.requires_grad(), name,
         " requires a gradient, which a write in place would not have: detach it, or call under no_grad");
  REFUSE(t.is_inference() && !c10::InferenceMode::is_enabled(), name, " is an inference tensor, written outside inference mode");
}
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Current device and stream of a call; scratch and outputs come from it.
struct Call {
  c10::cuda::CUDAGuard guard;
  at::TensorOptions opt;
  explicit Call(const Tensor& t) : guard(t.device()), opt(t.options().requires_grad(false)) {}
  void* stream() const { return c10::cuda::getCurrentCUDAStream().stream(); }
  // (straight to the allocator: through the dispatcher a call of five outputs takes 2 us longer)
  Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, opt.device(), std::nullopt);
  }
  Tensor workspace(size_t bytes) const {
    return bytes ? at::empty({static_cast<int64_t>(bytes)}, opt.dtype(at::kByte)) : Tensor();
  }
};

void* ptr_of(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The library's status word of a device, by its address.
uint32_t* status_word(int64_t device) {
  static std::atomic<uint32_t*> words[64] = {};
  REFUSE(device < 0 || device >= 64, "device index ", device);
  uint32_t* w = words[device].load();
  if (!w) {
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
    check(okls_status_word(&w));
    words[device].store(w);
  }
  return w;
}
uint32_t* status_of(const Tensor& t) { return status_word(t.device().index()); }

// ---------------------------------------------------------------- embedding
Tensor embedding(const Tensor& weight, const Tensor& ids, double scale, std::optional<at::ScalarType> out_dtype) {
  REFUSE(weight.dim() != 2, "weight must be vocab x dim");
  const Mat w = matrix(weight, "weight");
  const int dt = float_code(weight.scalar_type(), "weight"), i64 = ids_code(ids, ids.numel());
  const at::ScalarType ot = out_dtype.value_or(weight.scalar_type());
  const int od = float_code(ot, "the output type");
  same_device(weight, ids);
  Call c(weight);
  std::vector<int64_t> shape = ids.sizes().vec();
  shape.push_back(w.cols);
  Tensor out = c.empty(shape, ot);
  check(okls_embedding(w.p, dt, w.ld, w.rows, w.cols, ids.data_ptr(), i64, ids.numel(), static_cast<float>(scale),
                       out.data_ptr(), od, w.cols, status_of(weight), c.stream()));
  return out;
}

Tensor embedding_grad(const Tensor& dy, const Tensor& ids, int64_t vocab, double scale, const Maybe& base, Maybe out,
                      at::ScalarType dtype) {
  const Mat d = matrix(dy, "dy");
  const int dt = float_code(dy.scalar_type(), "dy"), i64 = ids_code(ids, d.rows);
  Mat b = {}, o = {};
  if (base) b = plain_matrix(*base, "base", vocab, d.cols);
  const bool given = out.has_value();
  if (given) o = plain_matrix(*out, "out", vocab, d.cols), writable(*out, "out");
  REFUSE(base && out && base->scalar_type() != out->scalar_type(), "base and out must have one type");
  same_device(dy, ids);
  same_device(dy, base);
  same_device(dy, out);
  Call c(dy);
  if (!out) {
    out = c.empty({vocab < 0 ? 0 : vocab, d.cols}, base ? base->scalar_type() : dtype);
    o = {out->data_ptr(), vocab, d.cols, d.cols};
  }
  const int od = float_code(out->scalar_type(), "the output type");
  size_t need = 0;
  check(okls_embedding_grad_workspace_bytes(d.rows, vocab, d.cols, &need));
  Tensor ws = c.workspace(need);
  check(okls_embedding_grad(d.p, dt, d.ld, ids.data_ptr(), i64, d.rows, vocab, d.cols, static_cast<float>(scale), b.p, b.ld,
                            o.p, od, o.ld, ptr_of(ws), need, status_of(dy), c.stream()));
  if (given) written(*out);
  return *out;
}

// -------------------------------------------------------------------- 8 bits
// Rows start at multiples of 128 bytes (the product's copies need 16); the
// scales lie group by group, so that neighbouring rows' scales are neighbours.
std::tuple<Tensor, Tensor> fp8_empty(const Call& c, int64_t rows, int64_t cols, bool square) {
  const int64_t groups = (cols + kGroup - 1) / kGroup, lines = square ? (rows + kGroup - 1) / kGroup : rows;
  const int64_t lp = std::max<int64_t>((lines + 3) / 4 * 4, 1);
  return {at::empty_strided({rows, cols}, {std::max<int64_t>(groups, 1) * kGroup, 1}, c.opt.dtype(at::kFloat8_e4m3fn)),
          at::empty_strided({lines, groups}, {1, lp}, c.opt.dtype(at::kFloat))};
}

std::tuple<Tensor, Tensor, Tensor, Tensor> fp8_quantize(const Tensor& x, bool square, bool plain, bool transposed) {
  const Mat m = matrix(x, "x");
  const int dt = float_code(x.scalar_type(), "x");
  Call c(x);
  Tensor q, s, qt, st;
  if (plain) std::tie(q, s) = fp8_empty(c, m.rows, m.cols, square);
  if (transposed) std::tie(qt, st) = fp8_empty(c, m.cols, m.rows, square);
  check(okls_fp8_quantize(m.p, dt, m.ld, m.rows, m.cols, square ? OKLS_FP8_SQUARE : OKLS_FP8_ROW, ptr_of(q),
                          plain ? q.stride(0) : 0, plain ? s.data_ptr<float>() : nullptr, plain ? s.stride(0) : 0,
                          plain ? s.stride(1) : 0, ptr_of(qt), transposed ? qt.stride(0) : 0,
                          transposed ? st.data_ptr<float>() : nullptr, transposed ? st.stride(0) : 0,
                          transposed ? st.stride(1) : 0, c.stream()));
  return {q, s, qt, st};
}

// The kernels read one scale for each 128 x 1 or 128 x 128 of the codes, so
// the fields of an Fp8Tensor, which a caller can assign, are checked here again.
void check_fp8(const Tensor& q, const Tensor& s, bool square, const char* name) {
  REFUSE(!q.is_cuda(), "tensors must be on a CUDA device");
  REFUSE(q.dim() != 2 || q.scalar_type() != at::kFloat8_e4m3fn, name, " must be a matrix of float8_e4m3fn");
  REFUSE(q.numel() != 0 && q.size(1) > 1 && q.stride(1) != 1, "the last dimension of ", name, " must be contiguous");
  const int64_t lines = square ? (q.size(0) + kGroup - 1) / kGroup : q.size(0), groups = (q.size(1) + kGroup - 1) / kGroup;
  REFUSE(s.dim() != 2 || s.scalar_type() != at::kFloat || s.size(0) != lines || s.size(1) != groups, "the scale of ", name,
         " must be fp32 of shape (", lines, ", ", groups, ")");
  same_device(q, s);
}

Tensor fp8_matmul(const Tensor& a, const Tensor& as, const Tensor& b, const Tensor& bs, bool b_square, Maybe out,
                  at::ScalarType out_dtype, bool accumulate) {
  check_fp8(a, as, false, "the first factor");
  check_fp8(b, bs, b_square, "the second factor");
  const int64_t m = a.size(0), k = a.size(1), n = b.size(0);
  REFUSE(b.size(1) != k, "sums of length ", k, " and ", b.size(1));
  REFUSE(accumulate && !out, "accumulate needs out");
  same_device(a, b);
  same_device(a, out);
  Mat o = {};
  const bool given = out.has_value();
  if (given) o = plain_matrix(*out, "out", m, n), writable(*out, "out");
  Call c(a);
  if (!out) {
    out = c.empty({m, n}, out_dtype);
    o = {out->data_ptr(), m, n, n};
  }
  const int od = float_code(out->scalar_type(), "the output type");
  check(okls_fp8_matmul(a.data_ptr(), a.stride(0), as.data_ptr<float>(), as.stride(0), as.stride(1), b.data_ptr(), b.stride(0),
                        bs.data_ptr<float>(), bs.stride(0), bs.stride(1), b_square ? OKLS_FP8_SQUARE : OKLS_FP8_ROW, m, n, k,
                        o.p, od, o.ld, accumulate, status_of(a), c.stream()));
  if (given) written(*out);
  return *out;
}

// --------------------------------------------------------------------- norm
std::tuple<Tensor, Maybe, Tensor, Tensor> rms_norm(const Tensor& x, const Tensor& weight, const Maybe& residual, double eps,
                                                   std::optional<at::ScalarType> out_dtype, bool inplace) {
  const Mat m = matrix(x, "x");
  const int dt = float_code(x.scalar_type(), "x"), wd = float_code(weight.scalar_type(), "weight");
  const void* w = vector(weight, "weight", m.cols);
  const at::ScalarType ot = out_dtype.value_or(x.scalar_type());
  const bool fp8 = ot == at::kFloat8_e4m3fn;
  const int od = fp8 ? static_cast<int>(OKLS_E4M3) : float_code(ot, "the output type");
  same_device(x, weight);
  same_device(x, residual);
  Mat r = {};
  if (residual) {
    REFUSE(residual->sizes() != x.sizes(), "residual has shape ", residual->sizes(), ", not ", x.sizes());
    REFUSE(residual->scalar_type() != x.scalar_type(), "residual is ", residual->scalar_type(), ", not ", x.scalar_type());
    r = matrix(*residual, "residual");
    if (inplace) writable(*residual, "residual");
  }
  Call c(x);
  Tensor total = x, rstd = c.empty({m.rows}, at::kFloat), y, ys;
  Mat s = {};
  if (residual) {
    total = inplace ? *residual : c.empty(x.sizes(), x.scalar_type());
    s = inplace ? r : Mat{total.data_ptr(), m.rows, m.cols, m.cols};
  }
  if (fp8)
    std::tie(y, ys) = fp8_empty(c, m.rows, m.cols, false);
  else
    y = c.empty(x.sizes(), ot);
  check(okls_rms_norm(m.p, dt, m.ld, r.p, r.ld, w, wd, m.rows, m.cols, static_cast<float>(eps), y.data_ptr(), od,
                      fp8 ? y.stride(0) : m.cols, fp8 ? ys.data_ptr<float>() : nullptr, fp8 ? ys.stride(0) : 0,
                      fp8 ? ys.stride(1) : 0, s.p, s.ld, rstd.data_ptr<float>(), c.stream()));
  if (residual && inplace) written(total);
  return {y, fp8 ? Maybe(ys) : std::nullopt, total, rstd};
}

std::tuple<Tensor, Maybe> rms_norm_grad(const Tensor& dy, const Tensor& s, const Tensor& weight, const Tensor& rstd,
                                        const Maybe& dresidual, bool need_dweight) {
  REFUSE(dy.sizes() != s.sizes(), "dy has shape ", dy.sizes(), ", not ", s.sizes());
  const Mat g = matrix(dy, "dy"), m = matrix(s, "s");
  const int gd = float_code(dy.scalar_type(), "dy"), sd = float_code(s.scalar_type(), "s");
  const int wd = float_code(weight.scalar_type(), "weight");
  const void* w = vector(weight, "weight", m.cols);
  const float* rs = floats(rstd, "rstd", m.rows);
  same_device(s, dy);
  same_device(s, weight);
  same_device(s, rstd);
  same_device(s, dresidual);
  Mat e = {};
  if (dresidual) {
    REFUSE(dresidual->sizes() != s.sizes() || dresidual->scalar_type() != s.scalar_type(),
           "dresidual must have the shape and type of s");
    e = matrix(*dresidual, "dresidual");
  }
  Call c(s);
  Tensor ds = c.empty(s.sizes(), s.scalar_type()), dw;
  size_t need = 0;
  if (need_dweight) {
    dw = c.empty({m.cols}, at::kFloat);
    check(okls_rms_norm_grad_workspace_bytes(m.rows, m.cols, &need));
  }
  Tensor ws = c.workspace(need);
  check(okls_rms_norm_grad(g.p, gd, g.ld, m.p, sd, m.ld, w, wd, rs, e.p, e.ld, m.rows, m.cols, ds.data_ptr(), m.cols,
                           need_dweight ? dw.data_ptr<float>() : nullptr, ptr_of(ws), need, c.stream()));
  return {ds, need_dweight ? Maybe(dw) : std::nullopt};
}

// --------------------------------------------------------- log probabilities
std::tuple<Tensor, Tensor, Tensor, Maybe, Maybe, Tensor> token_logprobs(const Tensor& logits, const Tensor& ids,
                                                                        int64_t top_k, double scale) {
  const Mat z = matrix(logits, "logits");
  const int dt = float_code(logits.scalar_type(), "logits"), i64 = ids_code(ids, z.rows);
  same_device(logits, ids);
  Call c(logits);
  const at::IntArrayRef lead = logits.sizes().slice(0, logits.dim() - 1);
  Tensor logp = c.empty(lead, at::kFloat), entropy = c.empty(lead, at::kFloat), lse = c.empty(lead, at::kFloat);
  Tensor rest = c.empty(lead, at::kFloat);
  Maybe top_ids, top_logp;
  if (top_k > 0) {
    std::vector<int64_t> shape = lead.vec();
    shape.push_back(top_k);
    top_ids = c.empty(shape, at::kInt);
    top_logp = c.empty(shape, at::kFloat);
  }
  check(okls_token_logprobs_rest(z.p, dt, z.ld, ids.data_ptr(), i64, z.rows, z.cols, static_cast<float>(scale),
                                 static_cast<int32_t>(std::max<int64_t>(-1, std::min<int64_t>(top_k, 64))),
                                 logp.data_ptr<float>(), entropy.data_ptr<float>(), lse.data_ptr<float>(),
                                 rest.data_ptr<float>(), top_ids ? top_ids->data_ptr<int32_t>() : nullptr,
                                 top_logp ? top_logp->data_ptr<float>() : nullptr, status_of(logits), c.stream()));
  return {logp, entropy, lse, top_ids, top_logp, rest};
}

Tensor token_logprobs_grad(const Tensor& logits, const Tensor& ids, const Tensor& lse, const Maybe& rest,
                           const Maybe& entropy, const Tensor& dlogp, const Maybe& dentropy, double scale, bool inplace) {
  const Mat z = matrix(logits, "logits");
  const int dt = float_code(logits.scalar_type(), "logits"), i64 = ids_code(ids, z.rows);
  const float* l = floats(lse, "lse", z.rows);
  const float* g = floats(dlogp, "dlogp", z.rows);
  const float* lr = rest ? floats(*rest, "lse_rest", z.rows) : nullptr;
  const float *h = nullptr, *e = nullptr;
  if (dentropy) {
    REFUSE(!entropy, "dentropy needs the entropy");
    h = floats(*dentropy, "dentropy", z.rows);
    e = floats(*entropy, "entropy", z.rows);
  }
  same_device(logits, ids);
  same_device(logits, lse);
  same_device(logits, rest);
  same_device(logits, dlogp);
  same_device(logits, dentropy);
  if (dentropy) same_device(logits, entropy);
  if (inplace) writable(logits, "logits");
  Call c(logits);
  Tensor d = inplace ? logits : c.empty(logits.sizes(), logits.scalar_type());
  check(okls_token_logprobs_grad_rest(z.p, dt, z.ld, ids.data_ptr(), i64, z.rows, z.cols, static_cast<float>(scale), l, lr,
                                      e, g, h, d.data_ptr(), inplace ? z.ld : z.cols, c.stream()));
  if (inplace) written(logits);
  return d;
}

}  // namespace

PYBIND11_MODULE(_lm_native, m) {
  py::object error = py::module_::import("kronecker_factored_second_gb300._lib").attr("OklsError");
  g_okls_error = error.release().ptr();
  m.def("status_word", [](int64_t device) { return reinterpret_cast<uintptr_t>(status_word(device)); });
  m.def("embedding", &embedding);
  m.def("embedding_grad", &embedding_grad);
  m.def("rms_norm", &rms_norm);
  m.def("rms_norm_grad", &rms_norm_grad);
  m.def("fp8_quantize", &fp8_quantize);
  m.def("fp8_matmul", &fp8_matmul);
  m.def("token_logprobs", &token_logprobs);
  m.def("token_logprobs_grad", &token_logprobs_grad);
}
