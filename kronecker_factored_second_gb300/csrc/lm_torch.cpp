// Torch binding of the language-model operators and of the AdamW step: checks
// of tensors, output and scratch allocation on the current stream, and the call
// of the C entry (include/okls.h).  It computes nothing.  A call costs a few microseconds of
// host time, where the same in Python cost 15 to 25 (one token's norm: 20).
//
// Wrong tensors raise ValueError; what the C entry refuses raises OklsError.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <limits>
#include <optional>
#include <tuple>
#include <vector>

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

// -------------------------------------------------------------------- AdamW
// The tensors of a list or tuple.
class TensorList {
 public:
  TensorList(const py::object& o, const char* name) : name_(name) {
    PyObject* fast = PySequence_Fast(o.ptr(), name);
    if (!fast) throw py::error_already_set();
    seq_ = py::reinterpret_steal<py::object>(fast);
  }
  int64_t size() const { return PySequence_Fast_GET_SIZE(seq_.ptr()); }
  const Tensor& operator[](int64_t i) const {
    PyObject* o = PySequence_Fast_GET_ITEM(seq_.ptr(), i);
    REFUSE(!THPVariable_Check(o), name_, " must hold tensors");
    return THPVariable_Unpack(o);
  }

 private:
  const char* name_;
  py::object seq_;
};

// Memory of a step, [begin, end) of each tensor: what it writes, kind after kind, and the gradients, which it
// only reads (and which may be one and the same).
typedef std::pair<uintptr_t, uintptr_t> Range;

void refuse_overlaps(std::vector<Range>* kinds, int count, const std::vector<Range>& grads) {
  // usual are a few buffers, each of which its tensors go through upwards
  bool plain = true;
  std::vector<Range> all;
  Range hull[5];
  int used = 0;
  for (int k = 0; k < count && plain; ++k) {
    const std::vector<Range>& r = kinds[k];
    for (size_t i = 1; i < r.size(); ++i) plain = plain && r[i - 1].second <= r[i].first;
    if (r.empty()) continue;
    const Range h = {r.front().first, r.back().second};
    for (int i = 0; i < used; ++i) plain = plain && (h.second <= hull[i].first || hull[i].second <= h.first);
    hull[used++] = h;
  }
  if (!plain) {
    for (int k = 0; k < count; ++k) all.insert(all.end(), kinds[k].begin(), kinds[k].end());
    std::sort(all.begin(), all.end());
    for (size_t i = 1; i < all.size(); ++i)
      REFUSE(all[i].first < all[i - 1].second, "a parameter or a state appears twice, or two of them overlap");
    kinds = &all, count = 1;
  }
  Range read = {UINTPTR_MAX, 0};
  for (const Range& g : grads) read = {std::min(read.first, g.first), std::max(read.second, g.second)};
  for (int k = 0; k < count; ++k) {
    const std::vector<Range>& r = kinds[k];
    if (r.empty() || read.second <= r.front().first || r.back().second <= read.first) continue;
    for (const Range& g : grads) {
      // the first tensor that ends behind the gradient's begin
      const auto at = std::upper_bound(r.begin(), r.end(), g.first, [](uintptr_t p, const Range& t) { return p < t.second; });
      REFUSE(at != r.end() && at->first < g.second, "a gradient overlaps a parameter or a state");
    }
  }
}

// A tensor of a step, as the kernels see it: `count` elements in a row.
void* flat(const Tensor& t, const char* name, c10::Device device, int64_t count, std::vector<Range>& ranges, bool writes = true) {
  const c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  REFUSE(!impl->is_cuda(), name, " must be on a CUDA device");
  REFUSE(impl->device() != device, "tensors on ", device, " and ", impl->device());
  REFUSE(!impl->is_contiguous(), name, " must be contiguous");
  REFUSE(impl->numel() != count, name, " must hold ", count, " values, not ", impl->numel());
  REFUSE(count > (int64_t(1) << 33), name, " must hold 2^33 values at most, not ", count);
  void* p = const_cast<void*>(impl->data());
  REFUSE((reinterpret_cast<uintptr_t>(p) & (impl->itemsize() - 1)) != 0, name, " is not aligned to its elements");
  if (writes && t.is_inference()) writable(t, name);
  if (count) ranges.emplace_back(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + count * impl->itemsize());
  return p;
}

void adamw_step(const py::object& params, const py::object& grads, const py::object& avgs, const py::object& sqs,
                const py::object& avg_scales, const py::object& sq_scales, const py::object& step, const py::object& lr,
                double beta1, double beta2, double eps, double weight_decay, uint64_t seed) {
  c10::AutoGradMode no_grad(false);  // an optimizer's step: leaves are written
  const TensorList P(params, "params"), G(grads, "grads"), M(avgs, "exp_avgs"), V(sqs, "exp_avg_sqs");
  const int64_t num = P.size();
  REFUSE(G.size() != num || M.size() != num || V.size() != num, "params, grads, exp_avgs and exp_avg_sqs must be as many");
  REFUSE(avg_scales.is_none() != sq_scales.is_none(), "avg_scales and sq_scales go together");
  const bool bits8 = !avg_scales.is_none();
  std::optional<TensorList> MS, VS;
  if (bits8) {
    MS.emplace(avg_scales, "avg_scales"), VS.emplace(sq_scales, "sq_scales");
    REFUSE(MS->size() != num || VS->size() != num, "avg_scales and sq_scales must be as many as params");
  }
  okls_adamw_config cfg = {0.0, beta1, beta2, eps, weight_decay, seed};
  const bool counted = THPVariable_Check(step.ptr()), lr_given = THPVariable_Check(lr.ptr());
  const float* lr_dev = nullptr;
  int64_t number = 0;
  int64_t* step_dev = nullptr;
  if (lr_given) {
    const Tensor& t = THPVariable_Unpack(lr.ptr());
    REFUSE(!counted, "a learning rate on the device needs the step's number there, too");
    lr_dev = floats(t, "lr", 1);
  } else {
    cfg.lr = lr.cast<double>();
  }
  if (counted) {
    const Tensor& t = THPVariable_Unpack(step.ptr());
    REFUSE(t.scalar_type() != at::kLong, "step must be int64, not ", t.scalar_type());
    step_dev = static_cast<int64_t*>(const_cast<void*>(vector(t, "step", 1)));
    writable(t, "step");
  } else {
    number = step.cast<int64_t>();
  }
  if (num == 0 && !counted) return;
  const Tensor& first = counted ? THPVariable_Unpack(step.ptr()) : P[0];
  REFUSE(!first.is_cuda(), "tensors must be on a CUDA device");
  if (lr_given) same_device(first, THPVariable_Unpack(lr.ptr()));

  // one call of the C entry for each pair of types
  std::vector<okls_adamw_tensor> lists[4];
  std::vector<Range> ranges[5];
  std::vector<Range> read;
  for (auto& r : ranges) r.reserve(num);
  read.reserve(num);
  const c10::Device device = first.device();
  for (auto& l : lists) l.reserve(lists == &l ? num : 0);
  for (int64_t i = 0; i < num; ++i) {
    const Tensor &p = P[i], &g = G[i], &m = M[i], &v = V[i];
    const int64_t n = p.numel();
    okls_adamw_tensor e = {};
    const int pd = float_code(p.scalar_type(), "a parameter"), gd = float_code(g.scalar_type(), "a gradient");
    const at::ScalarType sd = bits8 ? at::kFloat8_e4m3fn : at::kFloat;
    REFUSE(m.scalar_type() != sd || v.scalar_type() != sd, "exp_avgs and exp_avg_sqs must be ", sd,
           bits8 ? " where scales are given" : "");
    e.param = flat(p, "a parameter", device, n, ranges[0]);
    e.grad = flat(g, "a gradient", device, n, read, false);
    e.exp_avg = flat(m, "exp_avg", device, n, ranges[1]);
    e.exp_avg_sq = flat(v, "exp_avg_sq", device, n, ranges[2]);
    if (bits8) {
      const Tensor &ms = (*MS)[i], &vs = (*VS)[i];
      REFUSE(ms.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat, "scales must be fp32");
      const int64_t groups = (n + kGroup - 1) / kGroup;
      e.avg_scale = static_cast<float*>(flat(ms, "avg_scale", device, groups, ranges[3]));
      e.sq_scale = static_cast<float*>(flat(vs, "sq_scale", device, groups, ranges[4]));
    }
    e.count = n, e.id = static_cast<int32_t>(i);
    lists[2 * pd + gd].push_back(e);
  }
  refuse_overlaps(ranges, 5, read);

  Call c(first);
  Tensor scalars;
  if (counted) {
    scalars = c.workspace(OKLS_ADAMW_SCALARS_BYTES);
  } else {
    REFUSE(c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None,
           "a captured step needs its number on the device (step as a tensor), or every replay would be the same step");
  }
  // the settings, too, are checked before anything is written
  for (int k = 0; k < 4; ++k) {
    if (lists[k].empty() && k > 0) continue;
    check(okls_adamw_step(nullptr, 0, k / 2, k % 2, bits8 ? OKLS_E4M3 : OKLS_F32, &cfg, counted ? 1 : number, ptr_of(scalars),
                          c.stream()));
  }
  if (counted) {
    check(okls_adamw_clock(&cfg, lr_dev, step_dev, scalars.data_ptr(), c.stream()));
    written(first);
  }
  for (int k = 0; k < 4; ++k) {
    if (lists[k].empty()) continue;
    check(okls_adamw_step(lists[k].data(), static_cast<int64_t>(lists[k].size()), k / 2, k % 2, bits8 ? OKLS_E4M3 : OKLS_F32,
                          &cfg, counted ? 1 : number, ptr_of(scalars), c.stream()));
  }
  for (int64_t i = 0; i < num; ++i) {
    written(P[i]), written(M[i]), written(V[i]);
    if (bits8) written((*MS)[i]), written((*VS)[i]);
  }
}

// -------------------------------------------------------------------- 4 bits
// bf16 values laid group by group, so that neighbouring rows' are neighbours.
Tensor group_values(const Call& c, int64_t rows, int64_t groups) {
  return at::empty_strided({rows, groups}, {1, std::max<int64_t>((rows + 7) / 8 * 8, 1)}, c.opt.dtype(at::kBFloat16));
}

void check_group(int64_t group) {
  REFUSE(group != 32 && group != 64 && (group < 128 || group % 128 != 0), "group must be 32, 64 or a multiple of 128, not ", group);
}

std::tuple<Tensor, Tensor, Maybe> int4_quantize(const Tensor& x, int64_t group, bool symmetric) {
  REFUSE(x.dim() != 2, "a weight is a matrix");
  const Mat m = matrix(x, "x");
  const int dt = float_code(x.scalar_type(), "x");
  check_group(group);
  Call c(x);
  const int64_t groups = (m.cols + group - 1) / group, pitch = std::max<int64_t>((m.cols + 127) / 128, 1) * 64;
  Tensor q = at::empty_strided({m.rows, (m.cols + 1) / 2}, {pitch, 1}, c.opt.dtype(at::kByte));
  Tensor s = group_values(c, m.rows, groups), z;
  if (!symmetric) z = group_values(c, m.rows, groups);
  check(okls_int4_quantize(m.p, dt, m.ld, m.rows, m.cols, group, q.data_ptr(), pitch, s.data_ptr(), s.stride(0), s.stride(1),
                           ptr_of(z), symmetric ? 0 : z.stride(0), symmetric ? 0 : z.stride(1), c.stream()));
  return {q, s, symmetric ? std::nullopt : Maybe(z)};
}

Tensor int4_matmul(const Tensor& x, const Tensor& codes, const Tensor& scale, const Maybe& zero, int64_t cols, int64_t group,
                   Maybe out, std::optional<at::ScalarType> out_dtype, bool accumulate) {
  const Mat m = matrix(x, "x");
  const int dt = float_code(x.scalar_type(), "x");
  // (the fields of an Int4Tensor can be assigned)
  check_group(group);
  REFUSE(!codes.is_cuda(), "the weight must be on a CUDA device");
  REFUSE(cols < 0 || codes.dim() != 2 || codes.scalar_type() != at::kByte || codes.size(1) != (cols + 1) / 2,
         "codes must be a matrix of uint8 with ", (cols + 1) / 2, " columns");
  REFUSE(codes.numel() != 0 && codes.size(1) > 1 && codes.stride(1) != 1, "the last dimension of codes must be contiguous");
  const int64_t n = codes.size(0), groups = (cols + group - 1) / group;
  const auto check_values = [&](const Tensor& t, const char* name) {
    REFUSE(t.dim() != 2 || t.scalar_type() != at::kBFloat16 || t.size(0) != n || t.size(1) != groups, name,
           " must be bf16 of shape (", n, ", ", groups, ")");
    same_device(x, t);
  };
  check_values(scale, "scale");
  if (zero) check_values(*zero, "zero");
  REFUSE(m.cols != cols, "sums of length ", m.cols, " and ", cols);
  REFUSE(accumulate && !out, "accumulate needs out");
  same_device(x, codes);
  same_device(x, out);
  Mat o = {};
  const bool given = out.has_value();
  if (given) {
    o = plain_matrix(*out, "out", m.rows, n), writable(*out, "out");
  }
  Call c(x);
  if (!out) {
    std::vector<int64_t> shape = x.sizes().vec();
    shape.back() = n;
    out = c.empty(shape, out_dtype.value_or(x.scalar_type()));
    o = {out->data_ptr(), m.rows, n, n};
  }
  const int od = float_code(out->scalar_type(), "the output type");
  check(okls_int4_matmul(m.p, dt, m.ld, codes.data_ptr(), codes.stride(0), scale.data_ptr(), scale.stride(0), scale.stride(1),
                         zero ? zero->data_ptr() : nullptr, zero ? zero->stride(0) : 0, zero ? zero->stride(1) : 0, group,
                         m.rows, n, cols, o.p, od, o.ld, accumulate, c.stream()));
  if (given) written(*out);
  return *out;
}

// ------------------------------------------------------------------ sampling
// A setting of `sample`: None, a number for all rows, or a value for each row.
template <class N>
void setting(const py::object& o, const char* name, at::ScalarType type, const Tensor& logits, int64_t rows, N& all, const N*& dev) {
  if (o.is_none()) return;
  if (!THPVariable_Check(o.ptr())) {
    all = static_cast<N>(o.cast<double>());
    return;
  }
  const Tensor& t = THPVariable_Unpack(o.ptr());
  REFUSE(t.scalar_type() != type, name, " must be ", type, ", not ", t.scalar_type());
  dev = static_cast<const N*>(vector(t, name, rows));
  same_device(logits, t);
}

std::tuple<Tensor, Tensor> sample(const Tensor& logits, const Tensor& u, const py::object& temperature, const py::object& top_k,
                                  const py::object& top_p, const py::object& min_p) {
  const Mat z = matrix(logits, "logits");
  const int dt = float_code(logits.scalar_type(), "logits");
  const float* r = floats(u, "u", z.rows);
  same_device(logits, u);
  okls_sample_settings s = {nullptr, nullptr, nullptr, nullptr, 1.0f, 0, 1.0f, 0.0f};
  double k = 0.0;
  const double* unused = nullptr;
  setting(temperature, "temperature", at::kFloat, logits, z.rows, s.temperature, s.temperature_dev);
  if (!top_k.is_none() && THPVariable_Check(top_k.ptr()))
    setting(top_k, "top_k", at::kInt, logits, z.rows, s.top_k, s.top_k_dev);
  else
    setting(top_k, "top_k", at::kInt, logits, z.rows, k, unused);
  setting(top_p, "top_p", at::kFloat, logits, z.rows, s.top_p, s.top_p_dev);
  setting(min_p, "min_p", at::kFloat, logits, z.rows, s.min_p, s.min_p_dev);
  REFUSE(!(s.temperature >= 0.0f), "temperature must not be negative");
  REFUSE(std::isnan(s.top_p) || std::isnan(s.min_p) || std::isnan(k) || k != std::floor(k), "top_k must be a whole number, top_p and min_p numbers");
  if (!s.top_k_dev) s.top_k = static_cast<int32_t>(std::max(-1.0, std::min(k, 2147483647.0)));
  Call c(logits);
  const at::IntArrayRef lead = logits.sizes().slice(0, logits.dim() - 1);
  Tensor ids = c.empty(lead, at::kInt), logp = c.empty(lead, at::kFloat);
  check(okls_sample(z.p, dt, z.ld, z.rows, z.cols, r, &s, ids.data_ptr<int32_t>(), logp.data_ptr<float>(), c.stream()));
  return {ids, logp};
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
  m.def("adamw_step", &adamw_step);
  m.def("int4_quantize", &int4_quantize);
  m.def("int4_matmul", &int4_matmul);
  m.def("sample", &sample);
}
