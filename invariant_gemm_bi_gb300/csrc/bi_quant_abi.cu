// bi_quant_abi.cu -- C ABI of quantisation in blocks, the block-scaled matrix
// product and token sampling: argument validation (all of it before any launch)
// and operand layouts.
#include <cstring>
#include <string>

#include "bi_check.h"
#include "bi_launch.h"
#include "bi_quant.h"

using namespace bi;

namespace {

int64_t blocks_of(int64_t n, int64_t size) { return (n + size - 1) / size; }

// scales must have the extents a x b
void scale_shape(Check& c, const bi_tensor* t, int64_t a, int64_t b, const char* reason) {
  c.that(!c.ok() || (t->shape[0] == a && t->shape[1] == b), BI_ERR_SHAPE_MISMATCH, reason);
}

// Rows of bytes that a tensor map takes: 16-byte base and row stride.
void rows_of_bytes(Check& c, const bi_tensor* t, int row, const char* name) {
  c.that(on(t->ptr, 16) && (t->shape[row] <= 1 || t->stride[row] % 16 == 0), BI_ERR_UNSUPPORTED_LAYOUT,
         "base must be 16-byte aligned and rows multiples of 16 bytes apart", name);
  c.that(t->shape[row] <= 1 || (t->stride[row] > 0 && t->stride[row] < (int64_t)1 << 40), BI_ERR_UNSUPPORTED_LAYOUT,
         "the row stride is out of range", name);
}

}  // namespace

extern "C" bi_status bi_quantize_blocks(const bi_tensor* x, int32_t block_rows, const bi_tensor* q,
                                        const bi_tensor* scales, bi_stream stream) {
  Check c;
  c.tensor(x, "x", 2, false);
  c.operand(q, "q", 2, Check::kE4m3, true);
  c.operand(scales, "scales", 2, Check::kScale, false);
  c.that(block_rows == 1 || block_rows == 128, BI_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t M = x->shape[0], K = x->shape[1], kb = blocks_of(K, 128), mb = blocks_of(M, block_rows);
  c.that(q->shape[0] == M && q->shape[1] == K, BI_ERR_SHAPE_MISMATCH, "q must have x's shape");
  scale_shape(c, scales, mb, kb, "scales must be [ceil(M / block_rows), ceil(K / 128)]");
  c.that(M * kb <= INT32_MAX, BI_ERR_INVALID_ARG, "too many blocks");
  c.distinct(q, "q");
  c.distinct(scales, "scales");
  c.apart(q, x, "bi_quantize_blocks");
  c.apart(scales, x, "bi_quantize_blocks");
  c.apart(scales, q, "bi_quantize_blocks");
  if (!c.ok() || M == 0 || K == 0) return abi_finish(c.st, c.why);
  QuantParams p;
  memset(&p, 0, sizeof(p));
  p.x = x->ptr, p.q = static_cast<uint8_t*>(q->ptr), p.scales = static_cast<float*>(scales->ptr);
  p.ld_x = stride_or(x, 0, 0), p.ld_q = stride_or(q, 0, 0);
  p.s_m = stride_or(scales, 0, 0), p.s_k = stride_or(scales, 1, 0);
  p.M = (int32_t)M, p.K = (int32_t)K, p.kb = (int32_t)kb, p.rows = block_rows, p.kind = kind_of(x->dtype);
  p.vec = rows_on_16(x) && on(q->ptr, 8) && p.ld_q % 8 == 0;
  c.st = launch_quantize(p, (cudaStream_t)stream, &c.why);
  return abi_finish(c.st, c.why);
}

extern "C" bi_status bi_mm_blockscaled(const bi_tensor* a, const bi_tensor* a_scales, const bi_tensor* b,
                                       const bi_tensor* b_scales, const bi_tensor* bias, const bi_tensor* c_out,
                                       bi_stream stream) {
  Check c;
  c.operand(a, "a", 2, Check::kE4m3, true);
  c.operand(a_scales, "a_scales", 2, Check::kScale, false);
  c.operand(b, "b", 2, Check::kE4m3, false);
  c.operand(b_scales, "b_scales", 2, Check::kScale, false);
  c.tensor(c_out, "c", 2, false);
  if (bias) c.operand(bias, "bias", 1, Check::kFloat, false);
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t M = a->shape[0], K = a->shape[1], N = b->shape[1], kb = blocks_of(K, 128);
  c.that(b->shape[0] == K, BI_ERR_SHAPE_MISMATCH, "a and b have different inner dimensions");
  c.that(K <= 1 || b->stride[0] == 1, BI_ERR_UNSUPPORTED_LAYOUT, "b: unit stride on K required (the weight as [N, K], transposed)");
  scale_shape(c, a_scales, M, kb, "a_scales must be [M, ceil(K / 128)]");
  scale_shape(c, b_scales, kb, blocks_of(N, 128), "b_scales must be [ceil(K / 128), ceil(N / 128)]");
  c.that(c_out->shape[0] == M && c_out->shape[1] == N, BI_ERR_SHAPE_MISMATCH, "c must be [M, N]");
  c.that(!bias || bias->shape[0] == N, BI_ERR_SHAPE_MISMATCH, "bias must be [N]");
  c.that(M <= 1 << 30 && N <= 1 << 30 && K <= 1 << 30, BI_ERR_INVALID_ARG, "an extent is out of range");
  c.distinct(c_out, "c");
  const bi_tensor* in[5] = {a, a_scales, b, b_scales, bias};
  for (int i = 0; i < 5; ++i) c.apart(c_out, in[i], "bi_mm_blockscaled");
  if (!c.ok() || M == 0 || N == 0) return abi_finish(c.st, c.why);
  const int esz = bytes_of(c_out->dtype);
  const int64_t ldc = stride_or(c_out, 0, N);
  const int bias_kind = !bias ? 0 : bias->dtype == BI_BF16 ? 1 : bias->dtype == BI_F32 ? 2 : 3;
  const bool vec_store = on(c_out->ptr, 16) && (ldc * esz) % 16 == 0;
  if (K == 0) {  // an empty sum: the bias, or zeros
    GemmProblem g;
    memset(&g, 0, sizeof(g));
    g.L = 1, g.M = M, g.N = N, g.alpha = 1.0f;
    g.c = c_out->ptr, g.ldc = ldc, g.out_f32 = c_out->dtype == BI_F32, g.out_f16 = c_out->dtype == BI_F16;
    g.bias = bias ? bias->ptr : nullptr, g.bias_kind = bias_kind, g.bias_stride = bias ? stride_or(bias, 0, 0) : 0;
    g.vec_store = vec_store;
    c.st = launch_fill_bias(g, (cudaStream_t)stream, &c.why);
    return abi_finish(c.st, c.why);
  }
  rows_of_bytes(c, a, 0, "a");
  rows_of_bytes(c, b, 1, "b");
  if (!c.ok()) return abi_finish(c.st, c.why);
  ScaledProblem g;
  memset(&g, 0, sizeof(g));
  g.a = a->ptr, g.b = b->ptr;
  g.lda = stride_or(a, 0, (int64_t)round_up_u64((uint64_t)K, 16));
  g.ldb = stride_or(b, 1, (int64_t)round_up_u64((uint64_t)K, 16));
  g.sa = static_cast<const float*>(a_scales->ptr), g.sb = static_cast<const float*>(b_scales->ptr);
  g.sa_m = stride_or(a_scales, 0, 0), g.sa_k = stride_or(a_scales, 1, 0);
  g.sb_k = stride_or(b_scales, 0, 0), g.sb_n = stride_or(b_scales, 1, 0);
  g.c = c_out->ptr, g.ldc = ldc, g.c_kind = kind_of(c_out->dtype);
  g.bias = bias ? bias->ptr : nullptr, g.bias_kind = bias_kind, g.bias_stride = bias ? stride_or(bias, 0, 0) : 0;
  g.M = M, g.N = N, g.K = K, g.vec_store = vec_store;
  c.st = launch_scaled_gemm(g, (cudaStream_t)stream, &c.why);
  return abi_finish(c.st, c.why);
}

extern "C" bi_status bi_sample_tokens(const bi_tensor* logits, const bi_tensor* uniforms, const bi_tensor* temperature,
                                      const bi_tensor* top_k, const bi_tensor* top_p, const bi_tensor* min_p,
                                      const bi_tensor* tokens, bi_stream stream) {
  Check c;
  c.tensor(logits, "logits", 2, false);
  c.tensor(tokens, "tokens", 1, true);
  if (!c.ok()) return abi_finish(c.st, c.why);
  const int64_t R = logits->shape[0], N = logits->shape[1];
  c.that(tokens->shape[0] == R, BI_ERR_SHAPE_MISMATCH, "tokens must be [R]");
  c.operand(uniforms, "uniforms", 1, Check::kScale, true);
  if (temperature) c.operand(temperature, "temperature", 1, Check::kScale, true);
  if (top_k) c.tensor(top_k, "top_k", 1, true);
  if (top_p) c.operand(top_p, "top_p", 1, Check::kScale, true);
  if (min_p) c.operand(min_p, "min_p", 1, Check::kScale, true);
  if (!c.ok()) return abi_finish(c.st, c.why);
  c.that(!top_k || top_k->dtype == BI_I32, BI_ERR_UNSUPPORTED_DTYPE, "top_k: int32 is needed");
  const bi_tensor* in[6] = {uniforms, temperature, top_k, top_p, min_p, logits};
  for (int i = 0; i < 5; ++i)
    c.that(!in[i] || in[i]->shape[0] == R, BI_ERR_SHAPE_MISMATCH, "uniforms and each row's settings must be [R]");
  c.that(N <= kMaxVocab, BI_ERR_INVALID_ARG, "rows longer than 327680 elements are not supported");
  c.that(N >= 1 || R == 0, BI_ERR_INVALID_ARG, "a row needs at least one logit");
  c.that(R <= 1 << 27, BI_ERR_INVALID_ARG, "too many rows");
  for (int i = 0; i < 6; ++i) c.apart(tokens, in[i], "bi_sample_tokens");
  if (!c.ok() || R == 0) return abi_finish(c.st, c.why);
  auto f32 = [](const bi_tensor* t) { return t ? static_cast<const float*>(t->ptr) : nullptr; };
  SampleParams p;
  memset(&p, 0, sizeof(p));
  p.x = logits->ptr, p.u = f32(uniforms), p.temperature = f32(temperature), p.top_p = f32(top_p), p.min_p = f32(min_p);
  p.top_k = top_k ? static_cast<const int32_t*>(top_k->ptr) : nullptr;
  p.tokens = tokens->ptr, p.tok64 = tokens->dtype == BI_I64;
  p.R = R, p.ld_x = R > 1 ? logits->stride[0] : 0, p.N = (int32_t)N, p.x_kind = kind_of(logits->dtype);
  c.st = launch_sample(p, (cudaStream_t)stream, &c.why);
  return abi_finish(c.st, c.why);
}
