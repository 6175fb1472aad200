// bi_serve.h -- host-side interfaces of the serving operators around the paged
// key-value cache: page planning (bi_plan.cu), rotary positions and cache
// writes (bi_rope.cu), single-token attention over the cache
// (bi_paged_attn.cu) and token log probabilities (bi_logprobs.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "../../include/bi.h"

namespace bi {

// Sets the thread's last-error message and returns st (bi_abi.cu).
bi_status abi_finish(bi_status st, const std::string& why);

// Block tables and slot maps from request lengths.
struct PlanParams {
  const int32_t* ctx;   // [B] tokens already cached
  const int32_t* add;   // [B] tokens to add
  const int32_t* pool;  // [F] free pages in the order they are handed out
  int32_t* table;       // [B][W], row stride ld_table
  int64_t ld_table;
  int32_t* seq_lens;    // [B]
  int32_t* offsets;     // [B + 1]
  int32_t* positions;   // [T]
  int64_t* slots;       // [T]
  int32_t* totals;      // [2]: pages wanted, tokens
  int32_t B, W, F, T, ps;
};
bi_status launch_plan(const PlanParams& p, cudaStream_t stream, std::string* why);

// One [tokens][heads][D] operand: element (t, h, d) at ptr + t*t_stride + h*h_stride + d.
struct HeadView {
  const void* ptr;
  int64_t t_stride, h_stride;
};
// A paged cache: element (page, row, h, d) at ptr + page*page + row*row + h*head + d.
struct PageView {
  void* ptr;
  int64_t page, row, head;
};

// Rotary positions: q rotated to q_out and, when hkv > 0, k rotated and v
// copied to the cache slots of their tokens.
struct RopeParams {
  uint64_t phase[BI_ROPE_MAX_PAIRS];  // 2^64 * turns per position of pair i (mod 2^64)
  float magnitude;
  int32_t half;         // rotated pairs (0: none)
  int32_t interleaved;
  int32_t transpose;    // rotate by -angle
  HeadView q, k, v;
  void* q_out;
  int64_t qo_t, qo_h;
  PageView kc, vc;
  PageView ks, vs;      // scales of a cache in 8 bits: fp32, element (page, row, h)
  const void* positions;  // [T] int32 or int64
  int32_t pos64;
  const int64_t* slots;   // [T]; negative: not stored
  int64_t num_slots;      // pages * page size
  int32_t T, hq, hkv, D, ps;
  int32_t q_kind, qo_kind, kv_kind, c_kind;  // 0 bf16, 1 fp16, 2 fp32, 3 e4m3 (caches)
  int32_t vec;          // 16-byte units: every row, stride and the rotary split are aligned
  unsigned int* status_word;
};
bi_status launch_rope(const RopeParams& p, cudaStream_t stream, std::string* why);

// Rows of a cache in 8 bits, as numbers again (bi_cache8.cu).
struct LoadParams {
  PageView kc, vc, ks, vs;
  void *k, *v;            // [T][H][D] of `kind`
  int64_t k_t, k_h, v_t, v_h;
  const int64_t* slots;   // [T]; negative: a row of zeros
  int64_t num_slots;
  int32_t T, H, D, ps;
  int32_t kind;           // 0 bf16, 1 fp16, 2 fp32
  int32_t vec;            // 16-byte units
  unsigned int* status_word;
};
bi_status launch_paged_load(LoadParams& p, cudaStream_t stream, std::string* why);

// Attention of one token per request over the paged cache.
struct PagedAttnParams {
  const void* q;  // [B][Hq][D]
  int64_t q_b, q_h;
  const void* k;  // element (page, row, h, d) at page*k_page + row*k_row + h*k_head + d
  const void* v;
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;
  PageView ks, vs;       // scales of caches in 8 bits
  const int32_t* table;  // [B][W], row stride ld_table
  int64_t ld_table;
  const int32_t* lens;   // [B]
  void* o;               // [B][Hq][D]
  int64_t o_b, o_h;
  float* ws_o;           // partial results [B][max_splits][Hq][D]
  float* ws_ml;          // and their maxima and sums [B][max_splits][Hq][2]
  int32_t B, Hq, Hkv, D, W, ps, P;
  int32_t group;         // query heads per key-value head
  int32_t head_tiles;    // tiles of query heads per key-value head
  int32_t max_splits;
  int32_t cap;           // keys a table row can name: min(W * ps, INT32_MAX)
  int32_t ps_shift;      // log2(ps), or -1 when ps is no power of two
  int32_t in_f16, out_kind;  // q's type; the caches have it too, or
  int32_t e4m3;              // are in 8 bits with scales
  float score_log2;      // scale * log2(e), rounded once to fp32
  unsigned int* status_word;
};
// The most pieces of a key range, over all lengths up to cap.
int32_t paged_max_splits(int64_t cap, bool e4m3);
bi_status launch_paged_attention(PagedAttnParams& p, cudaStream_t stream, std::string* why);

// Log probabilities of given tokens, entropies and the best alternatives.
struct LogprobParams {
  const void* x;       // [R][N], row stride ld_x elements, unit column stride
  const void* tokens;  // [R] int32 or int64
  float* lp;           // [R]
  float* entropy;      // [R] or null
  float* top_lp;       // [R][K] contiguous or null
  int32_t* top_ids;    // [R][K]
  int64_t R, N, ld_x;
  int32_t K, tok64, x_kind;
  int32_t cl;  // CTAs a row (set by the launcher)
};
bi_status launch_logprobs(const LogprobParams& p, cudaStream_t stream, std::string* why);

}  // namespace bi
