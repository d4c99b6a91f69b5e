// C ABI of the language-model operators: argument checks and launches (see
// include/okls.h for the contract).
#include <string.h>

#include <atomic>
#include <cmath>
#include <utility>

#include "okls_host.h"
#include "okls_internal.h"
#include "okls_lm.h"

using namespace okls;

namespace {

typedef long long ll;

okls_status bad(const char* op, const char* what) { return host_fail(OKLS_ERR_INVALID_ARG, "%s: %s", op, what); }

bool float_dtype(int32_t d) { return d == OKLS_F32 || d == OKLS_BF16; }
int elem_size(int32_t d) { return d == OKLS_F32 ? 4 : d == OKLS_BF16 ? 2 : 1; }

// A matrix argument: not null, aligned to its element, pitch at least cols.
okls_status check_mat(const char* op, const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld,
                      int elem) {
  if (rows < 0 || cols < 0) return host_fail(OKLS_ERR_INVALID_ARG, "%s: negative size of %s", op, name);
  if (rows == 0 || cols == 0) return OKLS_OK;
  if (!p) return host_fail(OKLS_ERR_INVALID_ARG, "%s: %s is NULL", op, name);
  if (reinterpret_cast<uintptr_t>(p) % elem != 0)
    return host_fail(OKLS_ERR_INVALID_ARG, "%s: %s is not aligned to its %d-byte elements", op, name, elem);
  if (rows > 1 && ld < cols)
    return host_fail(OKLS_ERR_INVALID_ARG, "%s: row pitch %lld of %s is below its %lld columns", op,
                     static_cast<ll>(ld), name, static_cast<ll>(cols));
  if (ld > (int64_t(1) << 40) / rows)
    return host_fail(OKLS_ERR_INVALID_ARG, "%s: row pitch %lld of %s is too large", op, static_cast<ll>(ld), name);
  return OKLS_OK;
}

// A row of elements whose size is a power of two: the checks of many tensors take no division.
inline okls_status check_row(const char* op, const char* name, const void* p, int elem) {
  if (p && (reinterpret_cast<uintptr_t>(p) & (elem - 1)) == 0) return OKLS_OK;
  return check_mat(op, name, p, 1, 1, 1, elem);
}

// A vector of 4-byte elements that may be absent.
okls_status check_vec(const char* op, const char* name, const void* p) {
  if (reinterpret_cast<uintptr_t>(p) % 4 == 0) return OKLS_OK;
  return host_fail(OKLS_ERR_INVALID_ARG, "%s: %s is not aligned to its 4-byte elements", op, name);
}

#define LM_TRY(call)                   \
  do {                                 \
    const okls_status s_ = (call);     \
    if (s_ != OKLS_OK) return s_;      \
  } while (0)

okls_status launched(const char* op, cudaError_t e) {
  if (e == cudaSuccess) return OKLS_OK;
  return host_fail(OKLS_ERR_CUDA, "%s: %s", op, cudaGetErrorString(e));
}

okls_status check_ids(const char* op, const void* ids, int32_t ids_i64, int64_t count) {
  if (ids_i64 != 0 && ids_i64 != 1) return bad(op, "ids_i64 must be 0 or 1");
  return check_mat(op, "ids", ids, 1, count, count, ids_i64 ? 8 : 4);
}

okls_status check_status(const char* op, const uint32_t* status_dev) {
  if (!status_dev) return bad(op, "status_dev is NULL");
  return check_vec(op, "status_dev", status_dev);
}

okls_status check_workspace(const char* op, const void* ws, size_t have, size_t need) {
  if (need == 0) return OKLS_OK;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return bad(op, "workspace must be 256-byte aligned");
  if (have < need)
    return host_fail(OKLS_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", op, have, need);
  return OKLS_OK;
}

// The library's own status word (okls_status_word).
__device__ uint32_t g_status;

// Words that status reads take their bits through: calls at the same time use
// words of their own.
constexpr uint32_t kTaken = 256;
__device__ uint32_t g_taken[kTaken];

// Reads and clears in one step: bits that a launch on another stream raises
// meanwhile are read now or stay for the next read.
__global__ void k_status_take(uint32_t* status, uint32_t* taken) { *taken = atomicExch(status, 0u); }

// Runs of `width` bytes, `pitch` apart in the order of their addresses.
struct Runs {
  uintptr_t p;
  int64_t count, width, pitch;
};
Runs runs_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem) {
  return {reinterpret_cast<uintptr_t>(p), rows, cols * elem, ld * elem};
}
// Values of `elem` bytes with a pitch in both directions: runs along the one whose
// neighbours are neighbours, or all that lies between the first and the last.
Runs runs_of_values(const void* p, int64_t rows, int64_t cols, int64_t ld_row, int64_t ld_col, int elem) {
  if ((ld_col == 1 || cols == 1) && (ld_row >= cols || rows == 1)) return runs_of(p, rows, cols, ld_row, elem);
  if ((ld_row == 1 || rows == 1) && (ld_col >= rows || cols == 1)) return runs_of(p, cols, rows, ld_col, elem);
  return runs_of(p, 1, (rows - 1) * ld_row + (cols - 1) * ld_col + 1, 0, elem);
}

// Whether two sets of runs have a byte in common.
bool share_memory(Runs a, Runs b) {
  if (!a.p || !b.p || a.count <= 0 || b.count <= 0 || a.width <= 0 || b.width <= 0) return false;
  if (b.p < a.p) std::swap(a, b);
  if (a.p + (a.count - 1) * a.pitch + a.width <= b.p) return false;
  if (a.count > 1 && b.count > 1 && a.pitch == b.pitch) {
    const int64_t off = static_cast<int64_t>(b.p - a.p) % a.pitch;
    return off < a.width || off + b.width > a.pitch;
  }
  const auto next = [](const Runs& r, int64_t i, uintptr_t to) {  // the last run that begins at or before `to`, if that is behind run i
    const int64_t at = r.count > 1 ? static_cast<int64_t>(to - r.p) / r.pitch : i + 1;
    return at > i ? at : i + 1;
  };
  for (int64_t i = 0, j = 0; i < a.count && j < b.count;) {
    const uintptr_t pa = a.p + i * a.pitch, pb = b.p + j * b.pitch;
    if (pa + a.width <= pb)
      i = next(a, i, pb);
    else if (pb + b.width <= pa)
      j = next(b, j, pa);
    else
      return true;
  }
  return false;
}

constexpr int64_t kMaxSide = (int64_t(1) << 31) - 2;
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

}  // namespace

extern "C" {

okls_status okls_status_word(uint32_t** status_dev) {
  if (!status_dev) return bad("okls_status_word", "status_dev is NULL");
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  void* p = nullptr;
  const cudaError_t e = cudaGetSymbolAddress(&p, g_status);
  if (e == cudaSuccess) *status_dev = static_cast<uint32_t*>(p);
  return launched("okls_status_word", e);
}

okls_status okls_status_word_read(uint32_t* status_dev, void* stream, uint32_t* dev_status) {
  LM_TRY(check_status("okls_status_word_read", status_dev));
  static std::atomic<uint32_t> next{0};
  uint32_t v = 0;
  void* words = nullptr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaGetSymbolAddress(&words, g_taken);
  if (e == cudaSuccess) {
    uint32_t* taken = static_cast<uint32_t*>(words) + next.fetch_add(1) % kTaken;
    k_status_take<<<1, 1, 0, st>>>(status_dev, taken);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyAsync(&v, taken, sizeof(v), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e != cudaSuccess) return launched("okls_status_word_read", e);
  if (dev_status) *dev_status = v;
  if (v & OKLS_DEV_TIMEOUT) return host_fail(OKLS_ERR_TIMEOUT, "a bounded device wait expired");
  if (v & OKLS_DEV_BAD_TOKEN) return host_fail(OKLS_ERR_INVALID_ARG, "a token id is at or past the vocabulary");
  return OKLS_OK;
}

// ------------------------------------------------------------- embedding
okls_status okls_embedding(const void* weight, int32_t weight_dtype, int64_t ldw, int64_t vocab, int64_t dim,
                           const void* ids, int32_t ids_i64, int64_t tokens, float scale, void* out,
                           int32_t out_dtype, int64_t ldo, uint32_t* status_dev, void* stream) {
  const char* op = "okls_embedding";
  if (!float_dtype(weight_dtype) || !float_dtype(out_dtype)) return bad(op, "dtypes must be fp32 or bf16");
  if (vocab < 1 || dim < 1 || tokens < 0) return bad(op, "vocab and dim must be positive, tokens non-negative");
  if (vocab > kMaxSide || dim > kMaxSide || tokens > kMaxSide) return bad(op, "sizes must be below 2^31");
  LM_TRY(check_status(op, status_dev));
  LM_TRY(check_mat(op, "weight", weight, vocab, dim, ldw, elem_size(weight_dtype)));
  LM_TRY(check_ids(op, ids, ids_i64, tokens));
  LM_TRY(check_mat(op, "out", out, tokens, dim, ldo, elem_size(out_dtype)));
  if (lm_div_up(dim, 1024) > 8 * kMaxGrid / (tokens > 0 ? tokens : 1))
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: tokens x dim is too large for one launch", op);
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  EmbedArgs A = {weight, ldw, vocab, dim, ids, ids_i64, tokens, scale, out, out_dtype, ldo, status_dev};
  return launched(op, launch_embedding(A, weight_dtype, static_cast<cudaStream_t>(stream)));
}

static okls_status check_grad_sizes(const char* op, int64_t tokens, int64_t vocab, int64_t dim) {
  if (vocab < 1 || dim < 1 || tokens < 0) return bad(op, "vocab and dim must be positive, tokens non-negative");
  if (vocab > kMaxSide || dim > kMaxSide || tokens > kMaxSide) return bad(op, "sizes must be below 2^31");
  // one CTA per row and slice of 2048 columns
  if (lm_div_up(dim, 2048) > kMaxGrid / vocab || dim > 65535 * int64_t(128))
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: vocab x dim is too large for one launch", op);
  if (tokens > 0 && lm_div_up(dim, 2048) > kMaxGrid / tokens)
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: tokens x dim is too large for one launch", op);
  return OKLS_OK;
}

okls_status okls_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim, size_t* workspace_bytes) {
  const char* op = "okls_embedding_grad_workspace_bytes";
  if (!workspace_bytes) return bad(op, "workspace_bytes is NULL");
  LM_TRY(check_grad_sizes(op, tokens, vocab, dim));
  *workspace_bytes = embedding_grad_workspace(tokens, vocab, dim);
  return OKLS_OK;
}

okls_status okls_embedding_grad(const void* dy, int32_t dy_dtype, int64_t lddy, const void* ids, int32_t ids_i64,
                                int64_t tokens, int64_t vocab, int64_t dim, float scale, const void* base,
                                int64_t ldbase, void* out, int32_t out_dtype, int64_t ldo, void* workspace,
                                size_t workspace_bytes, uint32_t* status_dev, void* stream) {
  const char* op = "okls_embedding_grad";
  if (!float_dtype(dy_dtype) || !float_dtype(out_dtype)) return bad(op, "dtypes must be fp32 or bf16");
  LM_TRY(check_grad_sizes(op, tokens, vocab, dim));
  LM_TRY(check_status(op, status_dev));
  LM_TRY(check_mat(op, "dy", dy, tokens, dim, lddy, elem_size(dy_dtype)));
  LM_TRY(check_ids(op, ids, ids_i64, tokens));
  LM_TRY(check_mat(op, "out", out, vocab, dim, ldo, elem_size(out_dtype)));
  if (base) LM_TRY(check_mat(op, "base", base, vocab, dim, ldbase, elem_size(out_dtype)));
  if (base == out && ldbase != ldo) return bad(op, "base is out but has another row pitch");
  LM_TRY(check_workspace(op, workspace, workspace_bytes, embedding_grad_workspace(tokens, vocab, dim)));
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  EmbedGradArgs A = {dy, lddy, ids, ids_i64, tokens, vocab, dim, scale, base, ldbase, out, ldo, status_dev};
  return launched(op, launch_embedding_grad(A, dy_dtype, out_dtype, workspace, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ norm
okls_status okls_rms_norm(const void* x, int32_t dtype, int64_t ldx, const void* residual, int64_t ldr,
                          const void* weight, int32_t weight_dtype, int64_t rows, int64_t dim, float eps, void* out,
                          int32_t out_dtype, int64_t ldo, float* out_scale, int64_t lds_row, int64_t lds_group,
                          void* res_out, int64_t ldro, float* rstd, void* stream) {
  const char* op = "okls_rms_norm";
  if (!float_dtype(dtype) || !float_dtype(weight_dtype)) return bad(op, "input dtypes must be fp32 or bf16");
  if (!float_dtype(out_dtype) && out_dtype != OKLS_E4M3) return bad(op, "out_dtype must be fp32, bf16 or e4m3");
  if (rows < 0 || rows > kMaxGrid || dim < 1) return bad(op, "rows must be in [0, 2^31), dim positive");
  if (dim > kNormMaxDim)
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: dim %lld is above %d", op, static_cast<ll>(dim), kNormMaxDim);
  if (!(eps >= 0.0f) || std::isinf(eps)) return bad(op, "eps must be finite and non-negative");
  LM_TRY(check_mat(op, "x", x, rows, dim, ldx, elem_size(dtype)));
  LM_TRY(check_mat(op, "weight", weight, 1, dim, dim, elem_size(weight_dtype)));
  LM_TRY(check_mat(op, "out", out, rows, dim, ldo, elem_size(out_dtype)));
  if ((residual == nullptr) != (res_out == nullptr) && rows > 0)
    return bad(op, "residual and res_out go together");
  if (residual) {
    LM_TRY(check_mat(op, "residual", residual, rows, dim, ldr, elem_size(dtype)));
    LM_TRY(check_mat(op, "res_out", res_out, rows, dim, ldro, elem_size(dtype)));
  }
  if ((out_dtype == OKLS_E4M3) != (out_scale != nullptr) && rows > 0)
    return bad(op, "out_scale belongs to an e4m3 output, and to no other");
  if (out_scale && (lds_row < 0 || lds_group < 0)) return bad(op, "negative scale pitch");
  LM_TRY(check_vec(op, "out_scale", out_scale));
  LM_TRY(check_vec(op, "rstd", rstd));
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  NormArgs A = {x,   ldx,       residual, ldr,       weight,  weight_dtype, rows,    static_cast<int32_t>(dim), eps,
                out, out_dtype, ldo,      out_scale, lds_row, lds_group,    res_out, ldro,                      rstd};
  return launched(op, launch_rms_norm(A, dtype, sms, static_cast<cudaStream_t>(stream)));
}

okls_status okls_rms_norm_grad_workspace_bytes(int64_t rows, int64_t dim, size_t* workspace_bytes) {
  const char* op = "okls_rms_norm_grad_workspace_bytes";
  if (!workspace_bytes) return bad(op, "workspace_bytes is NULL");
  if (rows < 0 || dim < 1) return bad(op, "rows must be non-negative, dim positive");
  if (dim > kNormMaxDim)
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: dim %lld is above %d", op, static_cast<ll>(dim), kNormMaxDim);
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  *workspace_bytes = rms_norm_grad_workspace(rows, dim, sms);
  return OKLS_OK;
}

okls_status okls_rms_norm_grad(const void* dy, int32_t dy_dtype, int64_t lddy, const void* s, int32_t s_dtype,
                               int64_t lds, const void* weight, int32_t weight_dtype, const float* rstd,
                               const void* dres, int64_t lddres, int64_t rows, int64_t dim, void* ds, int64_t ldds,
                               float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const char* op = "okls_rms_norm_grad";
  if (!float_dtype(dy_dtype) || !float_dtype(s_dtype) || !float_dtype(weight_dtype))
    return bad(op, "dtypes must be fp32 or bf16");
  if (rows < 0 || dim < 1) return bad(op, "rows must be non-negative, dim positive");
  if (dim > kNormMaxDim)
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: dim %lld is above %d", op, static_cast<ll>(dim), kNormMaxDim);
  LM_TRY(check_mat(op, "dy", dy, rows, dim, lddy, elem_size(dy_dtype)));
  LM_TRY(check_mat(op, "s", s, rows, dim, lds, elem_size(s_dtype)));
  LM_TRY(check_mat(op, "weight", weight, 1, dim, dim, elem_size(weight_dtype)));
  LM_TRY(check_mat(op, "rstd", rstd, 1, rows, rows, 4));
  LM_TRY(check_mat(op, "ds", ds, rows, dim, ldds, elem_size(s_dtype)));
  if (dres) LM_TRY(check_mat(op, "dres", dres, rows, dim, lddres, elem_size(s_dtype)));
  if (dweight) LM_TRY(check_mat(op, "dweight", dweight, 1, dim, dim, 4));
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  if (dweight) LM_TRY(check_workspace(op, workspace, workspace_bytes, rms_norm_grad_workspace(rows, dim, sms)));
  NormGradArgs A = {dy,   dy_dtype, lddy, s,    lds,  weight, weight_dtype,
                    rstd, dres,     lddres, rows, static_cast<int32_t>(dim), ds, ldds,
                    dweight ? static_cast<float*>(workspace) : nullptr};
  return launched(op, launch_rms_norm_grad(A, s_dtype, dweight, sms, static_cast<cudaStream_t>(stream)));
}

// -------------------------------------------------------------- quantise
okls_status okls_fp8_quantize(const void* x, int32_t dtype, int64_t ldx, int64_t rows, int64_t cols, int32_t block,
                              void* q, int64_t ldq, float* scale, int64_t lds_row, int64_t lds_group, void* qt,
                              int64_t ldqt, float* scale_t, int64_t ldst_row, int64_t ldst_group, void* stream) {
  const char* op = "okls_fp8_quantize";
  if (!float_dtype(dtype)) return bad(op, "dtype must be fp32 or bf16");
  if (block != OKLS_FP8_ROW && block != OKLS_FP8_SQUARE) return bad(op, "block must be OKLS_FP8_ROW or OKLS_FP8_SQUARE");
  if (rows > kMaxSide || cols > kMaxSide) return bad(op, "sizes must be below 2^31");
  LM_TRY(check_mat(op, "x", x, rows, cols, ldx, elem_size(dtype)));
  const bool some = rows > 0 && cols > 0;
  if (some && !q && !qt) return bad(op, "q and qt are both NULL");
  if ((q == nullptr) != (scale == nullptr) && some) return bad(op, "q and scale go together");
  if ((qt == nullptr) != (scale_t == nullptr) && some) return bad(op, "qt and scale_t go together");
  if (q) LM_TRY(check_mat(op, "q", q, rows, cols, ldq, 1));
  if (qt) LM_TRY(check_mat(op, "qt", qt, cols, rows, ldqt, 1));
  if (lds_row < 0 || lds_group < 0 || ldst_row < 0 || ldst_group < 0) return bad(op, "negative scale pitch");
  LM_TRY(check_vec(op, "scale", scale));
  LM_TRY(check_vec(op, "scale_t", scale_t));
  if (lm_div_up(rows, kFp8Group) > 65535)
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: more than 65535 blocks of 128 rows", op);
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  QuantArgs A = {x,     ldx,     rows,      cols, static_cast<uint8_t*>(q), ldq, scale, lds_row, lds_group,
                 static_cast<uint8_t*>(qt), ldqt, scale_t, ldst_row, ldst_group};
  return launched(op, launch_fp8_quantize(A, dtype, block == OKLS_FP8_SQUARE, static_cast<cudaStream_t>(stream)));
}

// --------------------------------------------------------------- product
static okls_status check_product(const char* op, int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 0) return bad(op, "negative size");
  if (m > kMaxSide || n > kMaxSide || k > kMaxSide) return bad(op, "sizes must be below 2^31");
  if (lm_div_up(m, 128) > kMaxGrid / (lm_div_up(n, 64) > 0 ? lm_div_up(n, 64) : 1))
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: m x n is too large for one launch", op);
  return OKLS_OK;
}

// 2-D map of an e4m3 matrix: boxes of 128 columns x box_rows rows in 128-byte
// swizzled rows; what lies outside the matrix arrives as zeros.
static okls_status fp8_map(const char* op, CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld,
                           int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = host_encode_fn();
  if (!fn) return host_fail(OKLS_ERR_NO_DEVICE, "%s: cuTensorMapEncodeTiled unavailable", op);
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols > 0 ? cols : 1), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: cuTensorMapEncodeTiled failed (%d) rows=%lld cols=%lld ld=%lld", op,
                     static_cast<int>(r), static_cast<ll>(rows), static_cast<ll>(cols), static_cast<ll>(ld));
  return OKLS_OK;
}

okls_status okls_fp8_matmul(const void* a, int64_t lda, const float* a_scale, int64_t lda_row, int64_t lda_group,
                            const void* b, int64_t ldb, const float* b_scale, int64_t ldb_row, int64_t ldb_group,
                            int32_t b_block, int64_t m, int64_t n, int64_t k, void* out, int32_t out_dtype,
                            int64_t ldo, int32_t accumulate, uint32_t* status_dev, void* stream) {
  const char* op = "okls_fp8_matmul";
  if (!float_dtype(out_dtype)) return bad(op, "out_dtype must be fp32 or bf16");
  if (b_block != OKLS_FP8_ROW && b_block != OKLS_FP8_SQUARE)
    return bad(op, "b_block must be OKLS_FP8_ROW or OKLS_FP8_SQUARE");
  if (accumulate != 0 && accumulate != 1) return bad(op, "accumulate must be 0 or 1");
  LM_TRY(check_product(op, m, n, k));
  LM_TRY(check_status(op, status_dev));
  LM_TRY(check_mat(op, "a", a, m, k, lda, 1));
  LM_TRY(check_mat(op, "b", b, n, k, ldb, 1));
  LM_TRY(check_mat(op, "out", out, m, n, ldo, elem_size(out_dtype)));
  if (m == 0 || n == 0) return OKLS_OK;
  if (k > 0 && (!a_scale || !b_scale)) return bad(op, "a scale is NULL");
  LM_TRY(check_vec(op, "a_scale", a_scale));
  LM_TRY(check_vec(op, "b_scale", b_scale));
  if (lda_row < 0 || lda_group < 0 || ldb_row < 0 || ldb_group < 0) return bad(op, "negative scale pitch");
  if (k > 0 && (reinterpret_cast<uintptr_t>(a) % 16 || reinterpret_cast<uintptr_t>(b) % 16 ||
                (m > 1 && lda % 16) || (n > 1 && ldb % 16)))
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: a and b need 16-byte aligned rows (lda %lld, ldb %lld)", op,
                     static_cast<ll>(lda), static_cast<ll>(ldb));
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  if (k == 0) {
    // an empty sum: zeros, or nothing to add
    if (accumulate) return OKLS_OK;
    return launched(op, cudaMemset2DAsync(out, static_cast<size_t>(ldo) * elem_size(out_dtype), 0,
                                          static_cast<size_t>(n) * elem_size(out_dtype), static_cast<size_t>(m),
                                          static_cast<cudaStream_t>(stream)));
  }
  const Fp8Plan P = fp8_plan(m, n, b_block == OKLS_FP8_SQUARE, sms);
  Fp8GemmArgs A;
  memset(&A, 0, sizeof(A));
  // a single row's pitch is not used, but the map wants a multiple of 16
  if (m == 1) lda = lm_div_up(k, 16) * 16;
  if (n == 1) ldb = lm_div_up(k, 16) * 16;
  if (!P.skinny) {
    LM_TRY(fp8_map(op, &A.amap, a, m, k, lda, P.box_a));
    LM_TRY(fp8_map(op, &A.bmap, b, n, k, ldb, P.box_b));
  }
  // whole boxes of a bf16 output leave through the copy engine
  if (P.pair && out_dtype == OKLS_BF16 && !accumulate && reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo % 8 == 0) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = host_encode_fn();
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(m)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ldo) * 2};
    cuuint32_t box[2] = {64, 32}, step[2] = {1, 1};
    // (an output the map cannot describe is stored by the threads)
    A.tma_out = fn(&A.omap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  A.a = static_cast<const uint8_t*>(a), A.b = static_cast<const uint8_t*>(b);
  A.lda = lda, A.ldb = ldb;
  A.a_scale = a_scale, A.lda_row = lda_row, A.lda_group = lda_group;
  A.b_scale = b_scale, A.ldb_row = ldb_row, A.ldb_group = ldb_group;
  A.b_square = b_block == OKLS_FP8_SQUARE;
  A.m = static_cast<int32_t>(m), A.n = static_cast<int32_t>(n), A.k = static_cast<int32_t>(k);
  A.out = out, A.out_dtype = out_dtype, A.ldo = ldo, A.accumulate = accumulate;
  A.status = status_dev;
  return launched(op, launch_fp8_gemm(A, P, sms, static_cast<cudaStream_t>(stream)));
}

// ----------------------------------------------------- log probabilities
okls_status okls_token_logprobs_rest(const void* logits, int32_t dtype, int64_t ldl, const void* ids, int32_t ids_i64,
                                     int64_t rows, int64_t vocab, float scale, int32_t top_k, float* logp,
                                     float* entropy, float* lse, float* lse_rest, int32_t* top_ids, float* top_logp,
                                     uint32_t* status_dev, void* stream) {
  const char* op = "okls_token_logprobs";
  if (!float_dtype(dtype)) return bad(op, "dtype must be fp32 or bf16");
  if (rows < 0 || vocab < 1 || vocab > kMaxSide) return bad(op, "rows must be non-negative, vocab in [1, 2^31)");
  if (rows > kMaxGrid / 8) return bad(op, "rows must be below 2^28");
  if (!(scale > 0.0f) || std::isinf(scale)) return bad(op, "scale must be positive and finite");
  if (top_k < 0 || top_k > 32 || top_k > vocab) return bad(op, "top_k must be in [0, min(vocab, 32)]");
  LM_TRY(check_status(op, status_dev));
  LM_TRY(check_mat(op, "logits", logits, rows, vocab, ldl, elem_size(dtype)));
  if (logp) LM_TRY(check_ids(op, ids, ids_i64, rows));
  if (top_k > 0 && rows > 0 && (!top_ids || !top_logp)) return bad(op, "top_ids and top_logp are needed for top_k > 0");
  LM_TRY(check_vec(op, "logp", logp));
  LM_TRY(check_vec(op, "entropy", entropy));
  LM_TRY(check_vec(op, "lse", lse));
  LM_TRY(check_vec(op, "lse_rest", lse_rest));
  LM_TRY(check_vec(op, "top_ids", top_ids));
  LM_TRY(check_vec(op, "top_logp", top_logp));
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  ScoreArgs A = {logits, ldl, ids, ids_i64, rows, vocab, scale, top_k, logp, entropy, lse, lse_rest, top_ids, top_logp, status_dev};
  return launched(op, launch_token_logprobs(A, dtype, sms, static_cast<cudaStream_t>(stream)));
}

okls_status okls_token_logprobs(const void* logits, int32_t dtype, int64_t ldl, const void* ids, int32_t ids_i64,
                                int64_t rows, int64_t vocab, float scale, int32_t top_k, float* logp, float* entropy,
                                float* lse, int32_t* top_ids, float* top_logp, uint32_t* status_dev, void* stream) {
  return okls_token_logprobs_rest(logits, dtype, ldl, ids, ids_i64, rows, vocab, scale, top_k, logp, entropy, lse, nullptr,
                                  top_ids, top_logp, status_dev, stream);
}

okls_status okls_token_logprobs_grad_rest(const void* logits, int32_t dtype, int64_t ldl, const void* ids,
                                          int32_t ids_i64, int64_t rows, int64_t vocab, float scale, const float* lse,
                                          const float* lse_rest, const float* entropy, const float* dlogp,
                                          const float* dentropy, void* dlogits, int64_t ldd, void* stream) {
  const char* op = "okls_token_logprobs_grad";
  if (!float_dtype(dtype)) return bad(op, "dtype must be fp32 or bf16");
  if (rows < 0 || vocab < 1 || vocab > kMaxSide) return bad(op, "rows must be non-negative, vocab in [1, 2^31)");
  if (!(scale > 0.0f) || std::isinf(scale)) return bad(op, "scale must be positive and finite");
  LM_TRY(check_mat(op, "logits", logits, rows, vocab, ldl, elem_size(dtype)));
  LM_TRY(check_mat(op, "dlogits", dlogits, rows, vocab, ldd, elem_size(dtype)));
  LM_TRY(check_ids(op, ids, ids_i64, rows));
  LM_TRY(check_mat(op, "lse", lse, 1, rows, rows, 4));
  LM_TRY(check_mat(op, "dlogp", dlogp, 1, rows, rows, 4));
  if (dentropy && !entropy) return bad(op, "dentropy needs entropy");
  LM_TRY(check_vec(op, "lse_rest", lse_rest));
  LM_TRY(check_vec(op, "entropy", entropy));
  LM_TRY(check_vec(op, "dentropy", dentropy));
  if (lm_div_up(vocab, 8192) > kMaxGrid / (rows > 0 ? rows : 1))
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: rows x vocab is too large for one launch", op);
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  ScoreGradArgs A = {logits, ldl, ids, ids_i64, rows, vocab, scale, lse, lse_rest, entropy, dlogp, dentropy, dlogits, ldd};
  return launched(op, launch_token_logprobs_grad(A, dtype, static_cast<cudaStream_t>(stream)));
}

okls_status okls_token_logprobs_grad(const void* logits, int32_t dtype, int64_t ldl, const void* ids, int32_t ids_i64,
                                     int64_t rows, int64_t vocab, float scale, const float* lse, const float* entropy,
                                     const float* dlogp, const float* dentropy, void* dlogits, int64_t ldd,
                                     void* stream) {
  return okls_token_logprobs_grad_rest(logits, dtype, ldl, ids, ids_i64, rows, vocab, scale, lse, nullptr, entropy, dlogp,
                                       dentropy, dlogits, ldd, stream);
}

// ----------------------------------------------------------------- AdamW
static_assert(sizeof(AdamwScalars) <= OKLS_ADAMW_SCALARS_BYTES, "okls.h holds the size");

static okls_status check_adamw(const char* op, const okls_adamw_config* c) {
  if (!c) return bad(op, "config is NULL");
  if (!(c->lr >= 0.0) || std::isinf(c->lr)) return bad(op, "lr must be finite and non-negative");
  if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0)) return bad(op, "betas must be in [0, 1)");
  if (!(c->eps >= 0.0) || std::isinf(c->eps)) return bad(op, "eps must be finite and non-negative");
  if (!(c->weight_decay >= 0.0) || std::isinf(c->weight_decay)) return bad(op, "weight_decay must be finite and non-negative");
  return OKLS_OK;
}

static AdamwHyper adamw_hyper(const okls_adamw_config* c) {
  return {c->lr, c->beta1, c->beta2, c->eps, c->weight_decay, c->seed};
}

okls_status okls_adamw_clock(const okls_adamw_config* config, const float* lr_dev, int64_t* step_dev, void* scalars_dev,
                             void* stream) {
  const char* op = "okls_adamw_clock";
  LM_TRY(check_adamw(op, config));
  LM_TRY(check_vec(op, "lr_dev", lr_dev));
  LM_TRY(check_mat(op, "step_dev", step_dev, 1, 1, 1, 8));
  LM_TRY(check_mat(op, "scalars_dev", scalars_dev, 1, 1, 1, 16));
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  return launched(op, launch_adamw_clock(adamw_hyper(config), lr_dev, step_dev, static_cast<AdamwScalars*>(scalars_dev),
                                         static_cast<cudaStream_t>(stream)));
}

okls_status okls_adamw_step(const okls_adamw_tensor* tensors, int64_t num, int32_t param_dtype, int32_t grad_dtype,
                            int32_t state_dtype, const okls_adamw_config* config, int64_t step, const void* scalars_dev,
                            void* stream) {
  const char* op = "okls_adamw_step";
  if (!float_dtype(param_dtype) || !float_dtype(grad_dtype)) return bad(op, "param and grad dtypes must be fp32 or bf16");
  if (state_dtype != OKLS_F32 && state_dtype != OKLS_E4M3) return bad(op, "state_dtype must be fp32 or e4m3");
  LM_TRY(check_adamw(op, config));
  if (num < 0 || (num > 0 && !tensors)) return bad(op, "tensors is NULL or num negative");
  if (!scalars_dev && step < 1) return bad(op, "step counts from 1");
  LM_TRY(check_mat(op, "scalars_dev", scalars_dev ? scalars_dev : tensors, 1, scalars_dev ? 1 : 0, 1, 16));
  const bool bits8 = state_dtype == OKLS_E4M3;
  const int se = bits8 ? 1 : 4;
  bool some = false;
  for (int64_t i = 0; i < num; ++i) {  // all of them, before the first launch
    const okls_adamw_tensor& t = tensors[i];
    if (t.count < 0 || t.count > (int64_t(1) << 33)) return bad(op, "a tensor's count must be in [0, 2^33]");
    if (t.count == 0) continue;
    LM_TRY(check_row(op, "param", t.param, elem_size(param_dtype)));
    LM_TRY(check_row(op, "grad", t.grad, elem_size(grad_dtype)));
    LM_TRY(check_row(op, "exp_avg", t.exp_avg, se));
    LM_TRY(check_row(op, "exp_avg_sq", t.exp_avg_sq, se));
    if (bits8) {
      LM_TRY(check_row(op, "avg_scale", t.avg_scale, 4));
      LM_TRY(check_row(op, "sq_scale", t.sq_scale, 4));
    }
    some = true;
  }
  if (!some) return OKLS_OK;
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  const AdamwScalars s = adamw_scalars(adamw_hyper(config), scalars_dev ? 1 : step);
  AdamwEntry e[kAdamwTable];
  for (int64_t i = 0; i < num;) {
    int k = 0;
    for (; i < num && k < kAdamwTable; ++i) {
      const okls_adamw_tensor& t = tensors[i];
      if (t.count != 0) e[k++] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.avg_scale, t.sq_scale, t.count, t.id};
    }
    if (k == 0) break;
    LM_TRY(launched(op, launch_adamw(e, k, param_dtype, grad_dtype, bits8, s, static_cast<const AdamwScalars*>(scalars_dev),
                                     static_cast<cudaStream_t>(stream))));
  }
  return OKLS_OK;
}

// ---------------------------------------------------------------- 4 bits
// Sizes and the vectors of a group's bf16 scales and zero points.
static okls_status check_int4(const char* op, int64_t rows, int64_t cols, int64_t group, const void* scale, int64_t lds_row,
                              int64_t lds_group, const void* zero, int64_t ldz_row, int64_t ldz_group) {
  if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide) return bad(op, "sizes must be in [0, 2^31)");
  if (group != 32 && group != 64 && (group < 128 || group % 128 != 0 || group > kMaxSide))
    return bad(op, "group must be 32, 64 or a multiple of 128");
  LM_TRY(check_mat(op, "scale", scale, 1, rows > 0 && cols > 0, 1, 2));
  if (zero) LM_TRY(check_mat(op, "zero", zero, 1, 1, 1, 2));
  if (lds_row < 0 || lds_group < 0 || ldz_row < 0 || ldz_group < 0) return bad(op, "negative scale pitch");
  return OKLS_OK;
}

okls_status okls_int4_quantize(const void* x, int32_t dtype, int64_t ldx, int64_t rows, int64_t cols, int64_t group,
                               void* codes, int64_t ldq, void* scale, int64_t lds_row, int64_t lds_group, void* zero,
                               int64_t ldz_row, int64_t ldz_group, void* stream) {
  const char* op = "okls_int4_quantize";
  if (!float_dtype(dtype)) return bad(op, "dtype must be fp32 or bf16");
  LM_TRY(check_int4(op, rows, cols, group, scale, lds_row, lds_group, zero, ldz_row, ldz_group));
  LM_TRY(check_mat(op, "x", x, rows, cols, ldx, elem_size(dtype)));
  LM_TRY(check_mat(op, "codes", codes, rows, lm_div_up(cols, 2), ldq, 1));
  if (rows == 0 || cols == 0) return OKLS_OK;
  if (lm_div_up(cols, group) > kMaxGrid / rows) return host_fail(OKLS_ERR_UNSUPPORTED, "%s: too many groups for one launch", op);
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  Int4QuantArgs A = {x,     ldx,       rows, cols,    group,    static_cast<uint8_t*>(codes), ldq, scale, lds_row,
                     lds_group, zero, ldz_row, ldz_group};
  return launched(op, launch_int4_quantize(A, dtype, static_cast<cudaStream_t>(stream)));
}

okls_status okls_int4_matmul(const void* x, int32_t x_dtype, int64_t ldx, const void* codes, int64_t ldq, const void* scale,
                             int64_t lds_row, int64_t lds_group, const void* zero, int64_t ldz_row, int64_t ldz_group,
                             int64_t group, int64_t rows, int64_t n, int64_t k, void* out, int32_t out_dtype, int64_t ldo,
                             int32_t accumulate, void* stream) {
  const char* op = "okls_int4_matmul";
  if (!float_dtype(x_dtype) || !float_dtype(out_dtype)) return bad(op, "dtypes must be fp32 or bf16");
  if (accumulate != 0 && accumulate != 1) return bad(op, "accumulate must be 0 or 1");
  if (rows < 0 || rows > kMaxSide) return bad(op, "sizes must be in [0, 2^31)");
  LM_TRY(check_int4(op, n, k, group, scale, lds_row, lds_group, zero, ldz_row, ldz_group));
  LM_TRY(check_mat(op, "x", x, rows, k, ldx, elem_size(x_dtype)));
  LM_TRY(check_mat(op, "codes", codes, n, lm_div_up(k, 2), ldq, 1));
  LM_TRY(check_mat(op, "out", out, rows, n, ldo, elem_size(out_dtype)));
  if (rows == 0 || n == 0) return OKLS_OK;
  if (k > 0 && (reinterpret_cast<uintptr_t>(codes) % 16 || (n > 1 && ldq % 16)))
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: codes need 16-byte aligned rows (ldq %lld)", op, static_cast<ll>(ldq));
  if (rows > 65535 * int64_t(8)) return host_fail(OKLS_ERR_UNSUPPORTED, "%s: more than 524280 rows", op);
  // (blocks store out while others still read)
  const Runs out_runs = runs_of(out, rows, n, ldo, elem_size(out_dtype));
  const int64_t groups = lm_div_up(k, group);
  if (share_memory(out_runs, runs_of(x, rows, k, ldx, elem_size(x_dtype)))) return bad(op, "out must not share memory with x");
  if (share_memory(out_runs, runs_of(codes, n, lm_div_up(k, 2), ldq, 1)) ||
      (k > 0 && (share_memory(out_runs, runs_of_values(scale, n, groups, lds_row, lds_group, 2)) ||
                 share_memory(out_runs, runs_of_values(zero, n, groups, ldz_row, ldz_group, 2)))))
    return bad(op, "out must not share memory with the weight");
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  if (k == 0) {
    // an empty sum: zeros, or nothing to add
    if (accumulate) return OKLS_OK;
    return launched(op, cudaMemset2DAsync(out, static_cast<size_t>(ldo) * elem_size(out_dtype), 0,
                                          static_cast<size_t>(n) * elem_size(out_dtype), static_cast<size_t>(rows),
                                          static_cast<cudaStream_t>(stream)));
  }
  Int4Args A = {static_cast<const uint8_t*>(codes), ldq, scale, lds_row, lds_group, zero, ldz_row, ldz_group, group, x, ldx,
                reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rows <= 1 || ldx * elem_size(x_dtype) % 16 == 0),
                rows, n, k, out, out_dtype, ldo, accumulate};
  return launched(op, launch_int4_matmul(A, x_dtype, sms, static_cast<cudaStream_t>(stream)));
}

// -------------------------------------------------------------- sampling
okls_status okls_sample(const void* logits, int32_t dtype, int64_t ldl, int64_t rows, int64_t vocab, const float* u,
                        const okls_sample_settings* settings, int32_t* ids, float* logp, void* stream) {
  const char* op = "okls_sample";
  if (!float_dtype(dtype)) return bad(op, "dtype must be fp32 or bf16");
  if (rows < 0 || rows > kMaxSide || vocab < 1) return bad(op, "rows must be in [0, 2^31), vocab positive");
  if (vocab > kSampleMaxVocab)
    return host_fail(OKLS_ERR_UNSUPPORTED, "%s: vocab %lld is above %lld", op, static_cast<ll>(vocab), static_cast<ll>(kSampleMaxVocab));
  if (!settings) return bad(op, "settings is NULL");
  LM_TRY(check_mat(op, "logits", logits, rows, vocab, ldl, elem_size(dtype)));
  LM_TRY(check_mat(op, "u", u, 1, rows, rows, 4));
  LM_TRY(check_mat(op, "ids", ids, 1, rows, rows, 4));
  LM_TRY(check_mat(op, "logp", logp, 1, rows, rows, 4));
  const okls_sample_settings& s = *settings;
  LM_TRY(check_vec(op, "temperature", s.temperature_dev));
  LM_TRY(check_vec(op, "top_k", s.top_k_dev));
  LM_TRY(check_vec(op, "top_p", s.top_p_dev));
  LM_TRY(check_vec(op, "min_p", s.min_p_dev));
  if (rows == 0) return OKLS_OK;
  int sms = 0;
  LM_TRY(host_device_sms(&sms));
  SampleArgs A = {logits, ldl, rows, vocab, u, s.temperature_dev, s.top_k_dev, s.top_p_dev, s.min_p_dev, s.temperature,
                  s.top_k, s.top_p, s.min_p, ids, logp, 0};
  return launched(op, launch_sample(A, dtype, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
