// Launch interface of the language-model operators (token embedding, RMS
// norm, 8-bit quantisation and product, token log probabilities, AdamW step,
// 4-bit product, sampling).  The entry file validates; these functions pick
// the launch shape.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace okls {

constexpr uint32_t kStBadToken = 0x10u;  // mirror of OKLS_DEV_BAD_TOKEN

constexpr int kDtF32 = 0, kDtBf16 = 1, kDtE4m3 = 2;  // mirror of okls_dtype

constexpr int kFp8Group = 128;          // values that share a scale
constexpr float kFp8Max = 448.0f;       // largest e4m3 value
constexpr float kFp8AmaxFloor = 7.888609052210118e-31f;  // 2^-100

__host__ __device__ inline int64_t lm_div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ------------------------------------------------------------- embedding
struct EmbedArgs {
  const void* weight;
  int64_t ldw, vocab, dim;
  const void* ids;
  int32_t ids_i64;
  int64_t tokens;
  float scale;
  void* out;
  int32_t out_dtype;
  int64_t ldo;
  uint32_t* status;
};
cudaError_t launch_embedding(const EmbedArgs& A, int weight_dtype, cudaStream_t st);

struct EmbedGradArgs {
  const void* dy;
  int64_t lddy;
  const void* ids;
  int32_t ids_i64;
  int64_t tokens, vocab, dim;
  float scale;
  const void* base;
  int64_t ldbase;
  void* out;
  int64_t ldo;
  uint32_t* status;
};
size_t embedding_grad_workspace(int64_t tokens, int64_t vocab, int64_t dim);
cudaError_t launch_embedding_grad(const EmbedGradArgs& A, int dy_dtype, int out_dtype, void* workspace,
                                  cudaStream_t st);

// ------------------------------------------------------------------ norm
struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  int32_t weight_dtype;
  int64_t rows;
  int32_t dim;
  float eps;
  void* out;
  int32_t out_dtype;
  int64_t ldo;
  float* out_scale;
  int64_t lds_row, lds_group;
  void* res_out;
  int64_t ldro;
  float* rstd;
};
cudaError_t launch_rms_norm(const NormArgs& A, int dtype, int num_sms, cudaStream_t st);

struct NormGradArgs {
  const void* dy;
  int32_t dy_dtype;
  int64_t lddy;
  const void* s;
  int64_t lds;
  const void* weight;
  int32_t weight_dtype;
  const float* rstd;
  const void* dres;
  int64_t lddres;
  int64_t rows;
  int32_t dim;
  void* ds;
  int64_t ldds;
  float* part;  // [CTAs][dim] partial sums of dweight, or null
};
constexpr int kNormMaxDim = 32768;
size_t rms_norm_grad_workspace(int64_t rows, int64_t dim, int num_sms);
cudaError_t launch_rms_norm_grad(const NormGradArgs& A, int s_dtype, float* dweight, int num_sms, cudaStream_t st);

// -------------------------------------------------------------- quantise
struct QuantArgs {
  const void* x;
  int64_t ldx, rows, cols;
  uint8_t* q;
  int64_t ldq;
  float* scale;
  int64_t lds_row, lds_group;
  uint8_t* qt;
  int64_t ldqt;
  float* scale_t;
  int64_t ldst_row, ldst_group;
};
cudaError_t launch_fp8_quantize(const QuantArgs& A, int dtype, int square, cudaStream_t st);

// --------------------------------------------------------------- product
struct Fp8GemmArgs {
  CUtensorMap amap, bmap;  // codes: boxes of 128 columns
  CUtensorMap omap;        // a bf16 output: boxes of 64 columns x 32 rows (tma_out)
  const uint8_t* a;
  const uint8_t* b;
  int64_t lda, ldb;
  const float* a_scale;
  int64_t lda_row, lda_group;
  const float* b_scale;
  int64_t ldb_row, ldb_group;
  int32_t b_square;
  int32_t m, n, k;
  void* out;
  int32_t out_dtype;
  int64_t ldo;
  int32_t accumulate;
  int32_t tma_out;
  uint32_t* status;
};
// What a product of this size runs as.
struct Fp8Plan {
  bool skinny;  // a few tokens
  bool pair;    // CTA pairs
  int box_a, box_b;
};
Fp8Plan fp8_plan(int64_t m, int64_t n, bool b_square, int num_sms);
cudaError_t launch_fp8_gemm(const Fp8GemmArgs& A, const Fp8Plan& P, int num_sms, cudaStream_t st);

// ----------------------------------------------------- log probabilities
struct ScoreArgs {
  const void* logits;
  int64_t ldl;
  const void* ids;
  int32_t ids_i64;
  int64_t rows, vocab;
  float scale;
  int32_t top_k;
  float* logp;
  float* entropy;
  float* lse;
  float* lse_rest;
  int32_t* top_ids;
  float* top_logp;
  uint32_t* status;
};
cudaError_t launch_token_logprobs(const ScoreArgs& A, int dtype, int num_sms, cudaStream_t st);

struct ScoreGradArgs {
  const void* logits;
  int64_t ldl;
  const void* ids;
  int32_t ids_i64;
  int64_t rows, vocab;
  float scale;
  const float* lse;
  const float* lse_rest;
  const float* entropy;
  const float* dlogp;
  const float* dentropy;
  void* dlogits;
  int64_t ldd;
};
cudaError_t launch_token_logprobs_grad(const ScoreGradArgs& A, int dtype, cudaStream_t st);

// ----------------------------------------------------------------- AdamW
struct AdamwEntry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;  // scales of 8-bit moments
  float* vs;
  int64_t count;
  int32_t id;  // the tensor's number, for its random numbers
};
constexpr int kAdamwTable = 400;  // tensors in one launch: 27 of the 32 KB that parameters may take

struct AdamwHyper {
  double lr, beta1, beta2, eps, weight_decay;
  uint64_t seed;
};
// What the kernels use of the hyperparameters and the step's number.
struct AdamwScalars {
  float beta1, rest1, beta2, rest2;  // rest = 1 - beta
  float rate;                        // lr / (1 - beta1^t)
  float root;                        // 1 / sqrt(1 - beta2^t)
  float eps, decay;                  // lr * weight_decay
  uint32_t key, low;                 // words of seed + t * 0x9E3779B97F4A7C15
};
__host__ __device__ inline AdamwScalars adamw_scalars(const AdamwHyper& h, int64_t t) {
  AdamwScalars s;
  s.beta1 = static_cast<float>(h.beta1), s.rest1 = static_cast<float>(1.0 - h.beta1);
  s.beta2 = static_cast<float>(h.beta2), s.rest2 = static_cast<float>(1.0 - h.beta2);
  s.rate = static_cast<float>(h.lr / (1.0 - pow(h.beta1, static_cast<double>(t))));
  s.root = static_cast<float>(1.0 / sqrt(1.0 - pow(h.beta2, static_cast<double>(t))));
  s.eps = static_cast<float>(h.eps), s.decay = static_cast<float>(h.lr * h.weight_decay);
  const uint64_t w = h.seed + static_cast<uint64_t>(t) * 0x9E3779B97F4A7C15ull;
  s.key = static_cast<uint32_t>(w >> 32), s.low = static_cast<uint32_t>(w);
  return s;
}
cudaError_t launch_adamw(const AdamwEntry* e, int num, int param_dtype, int grad_dtype, bool bits8,
                         const AdamwScalars& s, const AdamwScalars* s_dev, cudaStream_t st);
cudaError_t launch_adamw_clock(const AdamwHyper& h, const float* lr_dev, int64_t* step_dev, AdamwScalars* out,
                               cudaStream_t st);

// ---------------------------------------------------------------- 4 bits
struct Int4Args {
  const uint8_t* codes;  // n x ceil(k / 2), the even column in the low half
  int64_t ldq;
  const void* scale;  // bf16
  int64_t lds_row, lds_group;
  const void* zero;  // bf16, or null for 8
  int64_t ldz_row, ldz_group;
  int64_t group;
  const void* x;
  int64_t ldx;
  int32_t x_vec;  // x's rows start on 16-byte boundaries
  int64_t rows, n, k;
  void* out;
  int32_t out_dtype;
  int64_t ldy;
  int32_t accumulate;
};
cudaError_t launch_int4_matmul(const Int4Args& A, int x_dtype, int num_sms, cudaStream_t st);

struct Int4QuantArgs {
  const void* x;
  int64_t ldx, rows, cols, group;
  uint8_t* codes;
  int64_t ldq;
  void* scale;
  int64_t lds_row, lds_group;
  void* zero;
  int64_t ldz_row, ldz_group;
};
cudaError_t launch_int4_quantize(const Int4QuantArgs& A, int dtype, cudaStream_t st);

// -------------------------------------------------------------- sampling
constexpr float kSampleColdest = 9.5367431640625e-07f;  // 2^-20: a lower temperature takes the best token
constexpr int64_t kSampleMaxVocab = int64_t(1) << 20;
struct SampleArgs {
  const void* logits;
  int64_t ldl, rows, vocab;
  const float* u;
  // settings: for each row, or one for all
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  float temperature_all;
  int32_t top_k_all;
  float top_p_all, min_p_all;
  int32_t* ids;
  float* logp;
  int32_t shift;  // log2 of the vocabulary, rounded up, at least 1 (the launch fills it in)
};
cudaError_t launch_sample(const SampleArgs& A, int dtype, int num_sms, cudaStream_t st);

}  // namespace okls
