// Launch interface of the language-model operators (token embedding, RMS
// norm, 8-bit quantisation and product, token log probabilities).  The entry
// file validates; these functions pick the launch shape.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
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

}  // namespace okls
