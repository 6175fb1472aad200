// bi_quant.h -- host-side interfaces of the 8-bit operators: quantisation in
// blocks (bi_quant.cu), the block-scaled matrix product (bi_mm8.cu); and of
// token sampling (bi_sample.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "../../include/bi.h"

namespace bi {

// Sets the thread's last-error message and returns st (bi_abi.cu).
bi_status abi_finish(bi_status st, const std::string& why);

// q = e4m3(x / scale), a scale for each block of rows x 128.
struct QuantParams {
  const void* x;    // [M][K], row stride ld_x elements
  uint8_t* q;       // [M][K], row stride ld_q
  float* scales;    // [ceil(M / rows)][ceil(K / 128)], strides s_m, s_k
  int64_t ld_x, ld_q, s_m, s_k;
  int32_t M, K, kb; // kb = ceil(K / 128)
  int32_t rows;     // 1 or 128
  int32_t kind;     // 0 bf16, 1 fp16, 2 fp32
  int32_t vec;      // 16-byte reads, 8-byte writes
};
bi_status launch_quantize(const QuantParams& p, cudaStream_t stream, std::string* why);

// c[m,n] = sum over blocks of 128 of K: a_scales[m,kb] b_scales[kb,n/128] (a b of the block), + bias[n].
struct ScaledProblem {
  const void* a;  // [M][K] e4m3, row stride lda bytes
  const void* b;  // b[k][n] at n * ldb + k
  int64_t lda, ldb;
  const float *sa, *sb;  // element (m, kb) at m * sa_m + kb * sa_k; (kb, n / 128) at kb * sb_k + nb * sb_n
  int64_t sa_m, sa_k, sb_k, sb_n;
  void* c;
  int64_t ldc;
  int c_kind;  // 0 bf16, 1 fp16, 2 fp32
  const void* bias;
  int64_t bias_stride;
  int bias_kind;  // 0 none, 1 bf16, 2 fp32, 3 fp16
  int64_t M, N, K;
  int vec_store;
};
bi_status launch_scaled_gemm(const ScaledProblem& g, cudaStream_t stream, std::string* why);

// One token of each row of logits.
struct SampleParams {
  const void* x;             // [R][N], row stride ld_x elements
  const float* u;            // [R]
  const float* temperature;  // [R] or null
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  void* tokens;              // [R] int32 or int64
  int64_t R, ld_x;
  int32_t N, x_kind, tok64;
  unsigned int* status_word;
};
constexpr int64_t kMaxVocab = 327680;  // an eighth of a row in fp32 fits the shared memory beside the rest
bi_status launch_sample(SampleParams& p, cudaStream_t stream, std::string* why);

}  // namespace bi
