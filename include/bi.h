/*
 * bi.h -- C ABI of the batch-invariant bf16 contraction library (GB300, sm_103a).
 *
 * Every output element's reduction over K runs in one fixed order: K blocks
 * of 64 in ascending order, each block as four 16-wide tensor-core steps, an
 * fp32 accumulator that starts from zero, then one epilogue.  The tile shape,
 * the K order and the epilogue never depend on M, on the batch count, on the
 * number of SMs or on which SM computes a tile; there is no split-K and no
 * atomic accumulation.  Consequently:
 *
 *   INVARIANCE CONTRACT.  For fixed operation, dtypes, K, N (and, for bmm /
 *   conv, the per-element shapes) and fixed operand layouts, output row m of
 *   mm/addmm depends only on row m of A (and on B, bias): its bits are the
 *   same for every M >= 1 and on every run.  The same holds per batch element
 *   for bmm, per sample for conv2d_patch and per row for softmax_lastdim.
 *
 * Sources of the operations (page title, section):
 *   mm, addmm  "Unmasking the True Culprit: Why Temperature=0 Doesn't Mean
 *              Deterministic LLM Inference", sections "The Data-Parallel
 *              Strategy" and "Implementation Analysis: The matmul_persistent
 *              Function" (fixed tiles per dtype, one CTA owns the whole K
 *              reduction of a tile, K tiles in fixed order, optional bias);
 *              "Batch-Invariant VLAs", section "Thinky's Ops were not enough"
 *              (aten::mm / aten::addmm replacements).
 *   bmm        "Batch-Invariant Kernel Design: Conv2d and Attention BMM",
 *              section "Kernel 2: Attention BMM" (rank-3 [B*H, T, D]
 *              operands, each batch element its own base pointers and the
 *              same ordered reduction over K).
 *   conv2d_patch  same page, section "Kernel 1: Conv2d", and "Batch-Invariant
 *              VLAs", section "Replacing nn.Conv2d" (per-sample unfold times
 *              the flattened filter, plus bias).
 *   softmax_lastdim  "ai-infra handbook: deterministic inference", section on
 *              making normalisation and softmax batch-independent (each row
 *              reduced by one block in a fixed order).
 *
 * General conventions (all entry points):
 *   - All tensor pointers are DEVICE pointers on the current CUDA device.
 *     The caller allocates and owns every buffer, outputs included; the
 *     library allocates no device memory.
 *   - Calls are asynchronous: they validate, enqueue kernels on `stream`
 *     (a cudaStream_t; NULL = legacy default stream) and return.
 *   - Argument, shape, dtype and layout errors are returned BEFORE any
 *     launch; outputs are then untouched.  bi_last_error_message() gives
 *     a one-line reason (thread-local).
 *   - Strides are in ELEMENTS.  Operands are read through TMA, so a matrix
 *     operand needs a unit stride on one of its two matrix dimensions, a
 *     16-byte-aligned base and 16-byte-multiple other strides; anything else
 *     returns BI_ERR_UNSUPPORTED_LAYOUT (there is no fallback path).
 *   - Device-side failures (a bounded wait that ran out) do not hang or trap:
 *     the kernel records a code and exits; bi_device_status() reports it.
 */
#ifndef BI_H_
#define BI_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* bi_stream;

typedef enum {
  BI_BF16 = 0,
  BI_F16 = 1,
  BI_F32 = 2,
  BI_I32 = 3, /* index operands of the serving operations only */
  BI_I64 = 4
} bi_dtype;

typedef enum {
  BI_OK = 0,
  BI_ERR_INVALID_ARG = 1,        /* null pointer, bad rank, negative size ... */
  BI_ERR_SHAPE_MISMATCH = 2,     /* operand extents do not agree */
  BI_ERR_UNSUPPORTED_DTYPE = 3,  /* a dtype this operation does not take */
  BI_ERR_UNSUPPORTED_LAYOUT = 4, /* strides / alignment TMA cannot read */
  BI_ERR_CUDA = 5,               /* a CUDA runtime or driver call failed */
  BI_ERR_TIMEOUT = 6,            /* a device-side bounded wait ran out */
  BI_ERR_NO_DEVICE = 7           /* no usable sm_100-family device */
} bi_status;

/* A strided view of device memory.  shape/stride entries past ndim are ignored. */
typedef struct {
  void* ptr;          /* device address of element [0,...,0]; NULL = absent */
  int32_t ndim;       /* 1..4 */
  int32_t dtype;      /* a bi_dtype value */
  int64_t shape[4];
  int64_t stride[4];  /* in elements */
} bi_tensor;

/*
 * c[m,n] = sum_k a[m,k] * b[k,n]
 *   a: [M,K] bf16 or fp16, unit stride on K (row-major activations).
 *   b: [K,N] of the same type as a, unit stride on N (row-major weight) or on
 *      K (a transposed view of an [N,K] weight, as torch.nn.functional.linear
 *      stores it).  Mixed bf16 / fp16 operands return BI_ERR_UNSUPPORTED_DTYPE.
 *   c: [M,N] fp32, bf16 or fp16, unit stride on N; written, never read.
 *   M, N, K >= 1.  The fp32 accumulator is rounded once to c's dtype (RNE).
 *   fp16 inputs run the same tile and K order as bf16 inputs (the tensor
 *   core's f16 kind, one format for both operands).
 */
bi_status bi_mm(const bi_tensor* a, const bi_tensor* b, const bi_tensor* c, bi_stream stream);

/*
 * c[m,n] = (sum_k a[m,k] * b[k,n]) + bias[n]   (alpha = beta = 1)
 *   bias: [N] bf16, fp16 or fp32, any stride; added to the fp32 accumulator
 *   after the full K reduction, then one rounding to c's dtype.  Operand
 *   types and layouts as bi_mm.
 */
bi_status bi_addmm(const bi_tensor* bias, const bi_tensor* a, const bi_tensor* b,
                   const bi_tensor* c, bi_stream stream);

/*
 * c[l,m,n] = alpha * sum_k a[l,m,k] * b[l,k,n]   for l in [0, L)
 *   a: [L,M,K] bf16 or fp16, unit stride on K;  b: [L,K,N] of the same type,
 *   unit stride on N or on K (so Q @ K^T passes K^T as a stride view);
 *   c: [L,M,N] fp32, bf16 or fp16, unit stride on N.  The fp32 accumulator is
 *   multiplied by alpha (fp32), then rounded once.  Each l is an independent
 *   product.
 */
bi_status bi_bmm(const bi_tensor* a, const bi_tensor* b, const bi_tensor* c, float alpha,
                 bi_stream stream);

/*
 * y = conv2d(x, w, bias), non-transposed, cross-correlation (as nn.Conv2d):
 *   y[b,co,oh,ow] = bias[co] + sum_{ci,kh,kw} x[b, g*Cig+ci, oh*sh-ph+kh*dh, ow*sw-pw+kw*dw]
 *                                             * w[co, ci, kh, kw]
 *   with g = co / (Co/groups), out-of-image positions reading zero, and the
 *   reduction index k = (ci*KH + kh)*KW + kw (the unfold order) ascending.
 *   x: [B,C,H,W] bf16 contiguous;  w: [Co,C/groups,KH,KW] bf16 contiguous;
 *   bias: [Co] bf16 or fp32, or NULL / ptr == NULL for none;
 *   y: [B,Co,Ho,Wo] bf16 or fp32 contiguous, Ho = (H+2ph-dh(KH-1)-1)/sh+1.
 *   stride, padding, dilation: {h, w}.  Each sample is computed as its own
 *   implicit-im2col product (the patch gather happens in shared memory).
 *   Non-overlapping patches -- stride = (KH, KW), padding 0, dilation 1, one
 *   group, KW even and <= 16, W a multiple of 8 and <= 256, W/KW <= 128, x
 *   16-byte and w 4-byte aligned -- run the patch kernel of
 *   bi_conv2d_patch_packed straight from w (its filter stages are built from
 *   w in shared memory; nothing is allocated) and give its bits: each
 *   tensor-core K = 16 step is one kernel row (ci, kh), kw padded with exact
 *   zeros.  Every other geometry sums k in steps of 16 of the unfold order.
 *   Which of the two runs is a function of the geometry and of the two
 *   pointers' alignment, never of B (a batch slice of an aligned x stays
 *   aligned); the two groupings agree within rounding, not bit for bit.
 */
bi_status bi_conv2d_patch(const bi_tensor* x, const bi_tensor* w, const bi_tensor* bias,
                          const bi_tensor* y, const int32_t stride[2], const int32_t padding[2],
                          const int32_t dilation[2], int32_t groups, bi_stream stream);

/*
 * Packed patch-embedding filter, for bi_conv2d_patch_packed.  The filter
 * w[Co][C][KH][KW] of a non-overlapping patch convolution stored as a
 * row-major [Co][Kp] bf16 matrix with reduction index
 *   kp = (ci*KHp + kh)*16 + kw,   KHp = KH rounded up to a multiple of 4,
 * i.e. every kernel row (ci, kh) padded to 16 slots and every channel to a
 * multiple of 4 kernel rows; slots with kh >= KH or kw >= KW hold zero.
 * Packing is a data-layout service for the same convolution, not one of the
 * pages' operations.
 */
typedef struct {
  void* ptr;              /* device buffer holding the packed filter (caller-owned) */
  int64_t bytes;          /* its size in bytes */
  int64_t Co, C, KH, KW;  /* shape of the filter it was packed from */
  int64_t Kp;             /* row length C * KHp * 16 */
} bi_conv_packed_weight;

/* Bytes of the packed form of a [Co,C,KH,KW] filter (0 if KW > 16 or empty). */
int64_t bi_conv_packed_weight_bytes(int64_t Co, int64_t C, int64_t KH, int64_t KW);

/*
 * Packs w ([Co,C,KH,KW] bf16 contiguous, KW <= 16) into dst (device, 16-byte
 * aligned, dst_bytes >= bi_conv_packed_weight_bytes(...)); fills *out.
 * Asynchronous on `stream`.
 */
bi_status bi_conv_pack_weight(const bi_tensor* w, void* dst, int64_t dst_bytes,
                              bi_conv_packed_weight* out, bi_stream stream);

/*
 * y = conv2d(x, w, bias, stride = (KH, KW), padding 0, dilation 1, groups 1)
 * -- the patch embedding of "Batch-Invariant VLAs", section "Replacing
 * nn.Conv2d" -- with w given packed:
 *   y[b,co,oh,ow] = bias[co] + sum_{ci,kh,kw} x[b, ci, oh*KH+kh, ow*KW+kw] * w[co,ci,kh,kw]
 * The reduction runs over the packed index kp in ascending order; each
 * tensor-core K = 16 step is one kernel row (ci, kh) (its zero slots add
 * exact zeros; image pixels outside a position's own window are never read
 * into it).  Per output element this is a fixed order, the same for every
 * batch size, and the same as bi_conv2d_patch's for the geometries that
 * bi_conv2d_patch runs on the patch kernel (bit for bit).
 *   x: [B,C,H,W] bf16 contiguous, 16-byte aligned, W a multiple of 8 and
 *      <= 256;  y: [B,Co,H/KH,W/KW] bf16 or fp32 contiguous, W/KW <= 128;
 *   bias: [Co] bf16 or fp32, or NULL / ptr == NULL.  Image rows or columns
 *   past the last whole patch are ignored (as the size formula does).
 */
bi_status bi_conv2d_patch_packed(const bi_tensor* x, const bi_conv_packed_weight* w,
                                 const bi_tensor* bias, const bi_tensor* y, bi_stream stream);

/*
 * p[r,:] = softmax(s[r,:]) over the last dimension, per row r:
 *   mx = max_j s[r,j];  e_j = expf(s[r,j] - mx);  p[r,j] = e_j * RN(1 / sum_j e_j),
 *   sums in fp32 in a fixed order set by the element index only (4-element
 *   groups g, lane g mod 32 of one warp, then a fixed butterfly).
 *   s: [R,N] fp32, unit stride on N;  p: [R,N] bf16 or fp32, unit stride on N.
 */
bi_status bi_softmax_lastdim(const bi_tensor* s, const bi_tensor* p, bi_stream stream);

/*
 * Fused attention, per head l and query row i:
 *   o[l,i,:] = sum_j softmax_j(scale * q[l,i,:] . k[l,j,:]) v[l,j,:]
 * in one kernel, the scores and probabilities never written to memory
 * ("ai-infra handbook: deterministic inference", section on fixed splitting:
 * attention's key range is not split by load -- here not split at all -- and
 * a query row's result does not depend on how queries are chunked).  Per
 * query row: key blocks of 128 in ascending order; scores from a fixed
 * sequence of tensor-core steps over the head dimension (fp32); t = RN(s * c)
 * with c = RN(scale * log2 e); a running maximum m, replaced only when a block
 * raises it by more than 8; p = 2^(t - m) (the SFU's approximation);
 * l = RN(l * 2^(m_old - m_new)) + sum p (keys ascending); O accumulated in
 * fp32 from bf16(p) v in key order (rescaled with m); o = RN(O * RN(1/l)),
 * rounded once to o's type.  None of it depends on L, Tq, the tile a row
 * falls in or the SM count: a head alone gives the bits it gives in any
 * batch, and a query row the bits it gives among any other query rows.
 *   q: [L,Tq,D], k and v: [L,Tk,D], bf16, unit stride on the head
 *   dimension, 16-byte aligned bases, row and batch strides multiples of 16
 *   bytes;  o: [L,Tq,D] fp32 or bf16 (same layout rules);  scale finite.
 *   Head dimension D = 64, 128 or 256 (BI_ERR_INVALID_ARG otherwise); Tk >= 1
 *   (BI_ERR_INVALID_ARG otherwise); L == 0 or Tq == 0 launches nothing.
 *   Non-causal, no mask.
 */
bi_status bi_attention(const bi_tensor* q, const bi_tensor* k, const bi_tensor* v, float scale,
                       const bi_tensor* o, bi_stream stream);

/*
 * Long key ranges.  When Tk > 2048 the key range is split into fixed
 * 2048-key pieces ("ai-infra handbook: deterministic inference", section on
 * fixed splitting: a split by a fixed length, never by load, keeps attention
 * batch-invariant -- the split depends on Tk only).  Each (head, 128 query
 * rows, split) is one work unit of the kernel above, which writes its partial
 * O (relative to its own running maximum m_s) and (m_s, l_s) to a workspace;
 * a merge kernel then forms, per row, M = max_s m_s, w_s = 2^(m_s - M),
 * l = sum_s RN(w_s l_s), O = sum_s RN(w_s O_s) (splits in ascending order)
 * and o = RN(O * RN(1 / l)).  Tk <= 2048 is not split and needs no
 * workspace; bi_attention refuses a longer key range (BI_ERR_INVALID_ARG).
 *
 * Bytes of workspace bi_attention_ws needs for [L, Tq] queries against Tk
 * keys of head dimension D: 0 when Tk <= 2048 (or any argument is out of
 * range), else ceil(Tk / 2048) * L * Tq * (D + 2) * 4.
 */
int64_t bi_attention_workspace_bytes(int64_t L, int64_t Tq, int64_t Tk, int64_t D);

/*
 * bi_attention with a caller-owned device workspace (16-byte aligned, at
 * least bi_attention_workspace_bytes(L, Tq, Tk, D) bytes; may be NULL when that
 * is 0).  The workspace is scratch: its contents on entry do not matter and
 * on return are unspecified; it must not be used by other work on the device
 * while the call's kernels run (stream order).  Results for Tk <= 2048 are
 * those of bi_attention, bit for bit.
 */
bi_status bi_attention_ws(const bi_tensor* q, const bi_tensor* k, const bi_tensor* v, float scale,
                          const bi_tensor* o, void* workspace, int64_t workspace_bytes, bi_stream stream);

/*
 * bi_attention_ws without a caller workspace: a split key range uses a
 * scratch area the library keeps in static device memory (64 MiB per device,
 * 256-byte aligned, allocated when the library's module is loaded on the
 * device).  A problem whose workspace would not fit returns
 * BI_ERR_INVALID_ARG before any launch (use bi_attention_ws).  The scratch is
 * shared by every call on the device, so calls must not overlap: issue them
 * on one stream or order them.  Results are those of bi_attention_ws, bit
 * for bit.  The scratch's device address is looked up (cudaGetSymbolAddress)
 * on the first call on each device and again whenever that device's CUDA
 * context has been replaced (after cudaDeviceReset); that first call should
 * come before any stream capture.  No call allocates or frees device memory.
 * The pages have no counterpart of this entry point: it packages the same
 * operation for callers that cannot allocate device memory -- a serving
 * engine whose allocator reserves all device memory up front and gives no
 * library a way around it, or code that may not call cudaMalloc / cudaFree
 * because those synchronise the device.
 */
bi_status bi_attention_noalloc(const bi_tensor* q, const bi_tensor* k, const bi_tensor* v, float scale,
                               const bi_tensor* o, bi_stream stream);

/*
 * Row reductions over the last dimension -- the normalisation, log-softmax
 * and mean operations that "Unmasking the True Culprit: Why Temperature=0
 * Doesn't Mean Deterministic LLM Inference" (section "Beyond Matrix
 * Multiplication: Other Critical Operations") and "Batch-Invariant VLAs"
 * (aten::mean.dim) say must reduce each row in one fixed order.  A row of N
 * elements is reduced by a team of T threads, T chosen from N and the input
 * type alone: the first of 32, 64, 256, 1024 with N <= 4*G*T, G = 16 for
 * 16-bit inputs and 8 for fp32.  The row is cut into groups of 4 consecutive
 * elements; thread t adds the elements of groups t, t+T, t+2T, ... in
 * ascending index order in fp32, each warp combines its 32 partials by a
 * fixed xor butterfly, and the warp partials are added in warp order.  Rows
 * longer than 4096*G elements are split, by N alone, over a cluster of
 * cl = ceil(N / (4096*G)) <= 8 CTAs of 1024 threads: CTA r reduces the r-th
 * of cl equal contiguous slices of the row's groups as above, and the cl
 * slice totals are added in rank order.  The order therefore depends on N,
 * the input type and the element index only -- not on how many rows are
 * reduced together, on where the row sits in memory (aligned rows are loaded
 * 4 elements at a time, others one at a time, with the same arithmetic) or
 * on the launch.  Each add, multiply, divide and square root is one
 * separately rounded fp32 operation; the output is rounded once to its type.
 *
 * All three: x (or s): [R,N] bf16, fp16 or fp32 with a unit stride on N,
 * aligned to its element size, N <= 2^24; outputs of any of the three types.
 * Asynchronous on `stream`; R == 0 (or N == 0 for the first two) launches
 * nothing.  Shape, layout or type errors are returned before any launch.
 */

/*
 * y[r,j] = RN(RN(x[r,j] * inv) * weight[j]),
 *   inv = RN(1 / RN(sqrt(RN(RN(sum_j x[r,j]^2) / N) + eps))),
 * the multiply by weight left out when weight is NULL (or weight->ptr is
 * NULL).  weight: [N] of any of the three types, any stride; y: [R,N], unit
 * stride on N; eps finite and >= 0 (BI_ERR_INVALID_ARG otherwise).
 */
bi_status bi_rmsnorm_lastdim(const bi_tensor* x, const bi_tensor* weight, float eps,
                             const bi_tensor* y, bi_stream stream);

/*
 * y[r,j] = RN(RN(s[r,j] - mx) - lse),  mx = max_j s[r,j],
 *   lse = logf(sum_j expf(RN(s[r,j] - mx))).
 * y: [R,N], unit stride on N.  For 1024-thread teams, when the rows' clusters
 * are more than the GPU runs at once with each thread holding its groups in
 * registers, each pass reloads them instead (two CTAs per SM); the order
 * above, and so every bit, is the same either way.
 */
bi_status bi_log_softmax_lastdim(const bi_tensor* s, const bi_tensor* y, bi_stream stream);

/*
 * y[r] = RN(RN(sum_j x[r,j]) / N).  y: [R], any stride.  N == 0 with R > 0
 * is BI_ERR_INVALID_ARG (the mean of an empty row).
 */
bi_status bi_mean_lastdim(const bi_tensor* x, const bi_tensor* y, bi_stream stream);

/*
 * Packed weights -- for products whose B operand is a fixed weight streamed
 * from HBM many times (decode-sized M).  Packing stores B as the exact
 * sequence of 128-byte-swizzled 64 x 64 shared-memory tile images the kernel
 * would otherwise assemble with strided TMA loads, ordered [k block][64-column
 * chunk] and zero-padded to whole output tiles, so one pipeline stage of B is
 * one contiguous range moved by a single bulk copy.  The tensor core reads the
 * same shared-memory bytes either way: results with a packed weight are bit
 * identical to results with the plain weight.  Packing is not one of the
 * pages' operations; it is a data-layout service for the same product.
 */
typedef struct {
  void* ptr;        /* device buffer holding the packed form (caller-owned) */
  int64_t bytes;    /* its size in bytes */
  int64_t K, N;     /* logical shape of the packed [K, N] weight */
  int32_t layout;   /* 1: images of a row-major [K,N] weight, 2: of a [N,K] (transposed view) */
  int32_t tile_n;   /* output-tile width the packing was made for (must match the library) */
  int32_t dtype;    /* element type of the weight: BI_BF16 or BI_F16 */
} bi_packed_weight;

/* Bytes needed to pack a [K, N] bf16 weight (0 for an empty one). */
int64_t bi_packed_weight_bytes(int64_t K, int64_t N);

/*
 * Packs b ([K,N] bf16 or fp16 on the device, unit stride on N or on K, 16-byte aligned
 * base and 16-byte multiple other stride) into dst (device, 16-byte aligned,
 * dst_bytes >= bi_packed_weight_bytes(K, N)); fills *out.  Asynchronous on
 * `stream`; dst must not be used before the packing has run.
 */
bi_status bi_pack_weight(const bi_tensor* b, void* dst, int64_t dst_bytes, bi_packed_weight* out,
                         bi_stream stream);

/*
 * c[m,n] = sum_k a[m,k] * B[k,n] (+ bias[n] when bias is non-NULL with a
 * non-NULL ptr), B given in packed form.  a: [M,K] of the packed weight's
 * type, as in bi_mm; c: [M,N] fp32, bf16 or fp16; bias: [N] bf16, fp16 or
 * fp32.  Same arithmetic, same bits as bi_mm / bi_addmm on the unpacked weight.
 */
bi_status bi_addmm_packed(const bi_tensor* bias, const bi_tensor* a, const bi_packed_weight* b,
                          const bi_tensor* c, bi_stream stream);

/*
 * Serving operations around a paged key-value cache.
 *
 * One layer's cache is two tensors k_cache and v_cache [P, page_size, Hkv, D]
 * of P pages.  Request b's j-th token lies in page page_table[b, j / page_size],
 * row j % page_size; its "slot" is page * page_size + row.  One decode step is
 * bi_paged_plan (once), then per layer bi_paged_store and bi_paged_attention,
 * then bi_token_logprobs on the logits.  Each is one launch (the attention two
 * for wide tables and large batches), allocates nothing and reads lengths and
 * tables on the device, so a step can be captured into a CUDA graph and
 * replayed as the batch grows within the captured extents; graphs whose
 * replays may overlap need workspaces of their own.
 *
 * Invariance: a request's rows depend on that request alone -- not on the
 * batch, on which pages hold its tokens or on the page size.
 *
 * Index operands are int32 or int64 tensors as each entry states, contiguous.
 * A slot, page or length that the cache or the table does not have is found on
 * the device: nothing is read or written through it, and bi_device_status
 * reports BI_ERR_INVALID_ARG.  No output may overlap an input or another
 * output in memory unless the entry says so (BI_ERR_INVALID_ARG).
 */

/*
 * Block tables and slot maps from request lengths.
 *   context_lens [B], new_lens [B] int32: tokens already cached, tokens to add
 *     (negative ones count as 0); B <= 2^22;
 *   page_table [B, W] int32, unit stride on W, updated: the first
 *     ceil(context / page_size) entries of a row are its pages;
 *   free_pages [F] int32: pages handed out in this order.
 * Requests take ceil((context+new) / page_size) - ceil(context / page_size)
 * pages each, in request order, appended to their rows; other entries are not
 * written.  Outputs:
 *   seq_lens [B] int32 = context + new;
 *   token_offsets [B+1] int32: first token of each request, then their number;
 *   positions [T] int32, slots [T] int64: of the new tokens, request after
 *     request; entries past the last token get position 0 and slot -1;
 *   totals [2] int32: pages wanted, tokens.
 * totals[0] > F says that the pool was too small: entries past it are -1, and
 * so are the slots of tokens on such pages or past the table's last column.
 * totals[1] > T says that T was too small: the tokens past it are left out.
 * Sums past 2^31 - 1 are given as 2^31 - 1.  Calling again with the same
 * operands writes the same values.
 */
bi_status bi_paged_plan(const bi_tensor* context_lens, const bi_tensor* new_lens,
                        const bi_tensor* page_table, const bi_tensor* free_pages, int32_t page_size,
                        const bi_tensor* seq_lens, const bi_tensor* token_offsets,
                        const bi_tensor* positions, const bi_tensor* slots, const bi_tensor* totals,
                        bi_stream stream);

/*
 * Rotary positions.  Pair i of a head at position n is turned by n * f_i:
 *   y1 = a (x1 cos - x2 sin),  y2 = a (x1 sin + x2 cos),   i < rotary_dim / 2,
 * with (x1, x2) the elements (i, i + rotary_dim/2) of the head, or (2i, 2i+1)
 * when interleaved; elements from rotary_dim on are copied.  a = magnitude.
 * A configuration is host memory that a program fills once; calls copy it.
 * Frequencies are doubles.  n * f_i is taken modulo one turn in 64-bit
 * integers, f_i / (2 pi) rounded to 2^-64 once: the reduced angle is off by |n|
 * 2^-65 turns at most (1.9e-7 radians times |n| / 2^40) and its rounding to fp32.
 */
#define BI_ROPE_MAX_PAIRS 128

typedef enum {
  BI_ROPE_PLAIN = 0,       /* f_i = base^(-2i / rotary_dim) */
  BI_ROPE_LINEAR = 1,      /* f_i / factor */
  BI_ROPE_BASE = 2,        /* base * factor^(R / (R - 2)) in base's place, R = rotary_dim > 2 */
  BI_ROPE_RAMP_TURNS = 3,  /* f_i (g + (1 - g) / factor), g = clamp((r - low) / (high - low), 0, 1),
                              r = original_length f_i / (2 pi): turns over the original length */
  BI_ROPE_RAMP_INDEX = 4   /* the same with g = 1 - clamp((i - i_high) / (i_low - i_high), 0, 1),
                              i_high = max(floor(idx(high)), 0), i_low = min(ceil(idx(low)), R - 1),
                              idx(r) = R ln(original_length / (2 pi r)) / (2 ln base) */
} bi_rope_scaling_kind;

typedef struct {
  int32_t kind;            /* a bi_rope_scaling_kind */
  int32_t reserved;        /* 0 */
  double factor;           /* > 0 */
  double original_length;  /* > 0, the two ramps */
  double low, high;        /* 0 < low < high in turns, the two ramps */
} bi_rope_scaling;

typedef struct {
  int32_t rotary_dim;                /* even, 2 .. 2 * BI_ROPE_MAX_PAIRS */
  int32_t interleaved;               /* 0 or 1 */
  float magnitude;                   /* a */
  int32_t reserved;
  uint64_t phase[BI_ROPE_MAX_PAIRS]; /* 2^64 * (f_i / (2 pi) mod 1) */
} bi_rope_config;

/* Fills *out; scaling may be NULL (plain).  base > 1; magnitude finite.  Host only. */
bi_status bi_rope_init(bi_rope_config* out, int32_t rotary_dim, int32_t interleaved, double base,
                       const bi_rope_scaling* scaling, double magnitude);
/* The same with the rotary_dim / 2 angular frequencies given (below 2^53 in magnitude). */
bi_status bi_rope_init_frequencies(bi_rope_config* out, int32_t rotary_dim, int32_t interleaved,
                                   const double* frequencies, double magnitude);

/*
 * y = rotate(x):  x, y [T,H,D] bf16, fp16 or fp32 (each its own type), unit
 * stride on D; positions [T] int32 or int64, of any value; rotary_dim <= D <=
 * 1024.  transpose != 0 applies the transposed map (angles negated, the
 * magnitude kept): the gradient with respect to x of bi_rope.  Arithmetic in
 * fp32, one rounding to y's type.  y may be x itself (same pointer, strides
 * and type); other overlaps are refused.  Rows and heads that are multiples of
 * 16 bytes, with rotary_dim / 2 a multiple of 8 and D - rotary_dim of 16, run
 * a wider kernel with the same bits.
 */
bi_status bi_rope(const bi_rope_config* config, const bi_tensor* x, const bi_tensor* positions,
                  int32_t transpose, const bi_tensor* y, bi_stream stream);

/*
 * Writes a step's keys and values into the cache: for every token t with
 * slots[t] >= 0, k_cache[slot] = rotate(k[t]) and v_cache[slot] = v[t]; and,
 * when q is given, q_out[t] = rotate(q[t]) for every t (stored or not).
 *   config NULL: nothing is rotated, q and positions must be absent;
 *   positions [T] int32 or int64; slots [T] int64, negative: not stored;
 *   k, v [T,Hkv,D] of one type, q [T,Hq,D]; q_out [T,Hq,D] of any of the three
 *   types (may be q itself, as in bi_rope); k_cache, v_cache
 *   [P,page_size,Hkv,D] of one type, bf16, fp16 or fp32; unit strides on D;
 *   P * page_size < 2^31.
 * Slots must be distinct: a row that two tokens name holds parts of either, and
 * which is not specified.  Cache rows that no token names are left as they were.
 */
bi_status bi_paged_store(const bi_rope_config* config, const bi_tensor* positions,
                         const bi_tensor* slots, const bi_tensor* q, const bi_tensor* q_out,
                         const bi_tensor* k, const bi_tensor* v, const bi_tensor* k_cache,
                         const bi_tensor* v_cache, bi_stream stream);

/*
 * Attention of one new token per request over its cached keys and values:
 *   o[b,h,:] = sum_j softmax_j(scale * q[b,h,:] . k_j) v_j,  j < seq_lens[b],
 * k_j and v_j the cache rows of token j for key-value head h / (Hq / Hkv).
 *   q [B,Hq,D] bf16 or fp16; k_cache, v_cache [P,page_size,Hkv,D] of q's type;
 *   o [B,Hq,D] fp32, bf16 or fp16;  Hkv divides Hq;  D = 64, 128 or 256;
 *   page_table [B,W] int32, unit stride on W; seq_lens [B] int32; any
 *   page_size >= 1 with P * page_size < 2^31 and W * page_size <= 2^30; B <= 2^22.
 *   q, caches and o: unit stride on D, 16-byte aligned, other strides
 *   multiples of 16 bytes.  scale and scale * log2(e) finite.
 * A request of length <= 0 gives zeros (the new token itself is normally in
 * the cache by then).  A length past W * page_size counts as W * page_size,
 * keys on a page outside [0, P) as absent; both are reported.  Rows past a
 * request's length are never read.  Among a request's own keys, one with score
 * -inf weighs nothing (all of them: zeros); a NaN or a score of +inf makes its
 * heads NaN; a NaN value makes its dimension of them NaN, an infinite value
 * makes it infinite or NaN.
 *
 * Order: a request of n keys is cut into pieces of s keys, s = 256 up to n =
 * 2048, beyond that 512 * 2^k, k the least with n <= 128 s -- a rule on its own
 * length.  In a piece, warp w of W takes the tiles w, w + W, ... in order with a
 * running maximum (tiles of 32 keys, 16 at D = 256; W = 4, or 8 at D = 256 and,
 * for more than 8 query heads a key-value head, at D = 128); p = 2^(t - m), t = RN(score * RN(scale
 * log2 e)).  Warp w + W/2 is joined into warp w, then warps 1, 2, ... into
 * warp 0, groups of 16 pieces in piece order, then the groups in order, all in
 * fp32.  Sums are of the unrounded p; the product with v takes p as the
 * sum of three bf16 or of two fp16 (of 2^15 p: what is below 2^-40 of a warp's
 * largest p is not in o).  A 16-bit o is the fp32 o rounded once.
 *
 * workspace: caller-owned, 16-byte aligned, at least
 * bi_paged_attention_workspace_bytes(B, Hq, D, W * page_size) bytes -- 0 when
 * W * page_size <= 256, else B * Hq * n * (D + 2) * 4, n the most pieces of a
 * request: with L = W * page_size, ceil(L / 256) up to L = 2048, beyond that
 * ceil(L / 512), but at least 8 and at most 128.  Scratch, as in bi_attention_ws.
 * What the table can name decides this size and the form of the launch, not the
 * lengths, which the host does not know: one launch while L <= 4096 and all
 * pieces of the batch run at once, else two.  A table kept for 131072 keys makes
 * one request of 1021 keys take 10.7 us in place of 7.6 on the device, and asks
 * for 2.1 MB of workspace for it (256 requests of 32 heads of 128: 545 MB).
 */
int64_t bi_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t D, int64_t max_len);
bi_status bi_paged_attention(const bi_tensor* q, const bi_tensor* k_cache, const bi_tensor* v_cache,
                             const bi_tensor* page_table, const bi_tensor* seq_lens, float scale,
                             const bi_tensor* o, void* workspace, int64_t workspace_bytes,
                             bi_stream stream);

/*
 * Log probabilities of given tokens, entropies and the best alternatives of
 * each row of logits [R,N] (bf16, fp16 or fp32, unit stride on N, N <= 2^24):
 *   logprobs[r] = RN(RN(x[r,tok] - M) - lse), M the row's maximum and lse =
 *     ln sum_j e^(x_j - M); tokens [R] int32 or int64; a token outside [0, N)
 *     has probability zero: -inf;
 *   entropy[r] = -sum_j p_j ln p_j, forbidden tokens (-inf) adding 0;
 *   top_ids[r,:K] the K tokens of the largest logits, largest first, the lower
 *     index first among equals (a NaN counts as larger than any number);
 *     top_logprobs[r,:] their log probabilities.
 * logprobs, entropy fp32 [R]; top_ids int32 and top_logprobs fp32 [R,K], all
 * contiguous; entropy may be NULL; top_ids and top_logprobs are given together
 * or not at all, K <= 64 and K <= N.  A row that holds a NaN or +inf, or
 * nothing but -inf, has NaN log probabilities and entropy (the ids stand, and a
 * token outside [0, N) has -inf there too).
 *
 * Order: 256 threads; slices of 16 KB of the row, of which thread t has the
 * 16-byte units t, t + 256, t + 512, t + 768, reduced relative to their own
 * maximum (sums of 2^(x log2 e - m), one fused multiply-add and the SFU's 2^x);
 * with s slices, groups of ceil(s / 8) are joined in slice order, then the
 * groups, then the lanes, then the warps by fixed trees -- by N and the type
 * alone, whatever the number of rows and the rows' alignment.  One pass: the
 * log probabilities agree with bi_log_softmax_lastdim's, which takes its sum in
 * another order and from expf, within rounding, not bit for bit.
 */
bi_status bi_token_logprobs(const bi_tensor* logits, const bi_tensor* tokens,
                            const bi_tensor* logprobs, const bi_tensor* entropy,
                            const bi_tensor* top_logprobs, const bi_tensor* top_ids,
                            bi_stream stream);

/*
 * Synchronises `stream`, then returns and clears the device-side status word
 * of the current device: BI_OK, BI_ERR_TIMEOUT when a kernel's bounded wait
 * ran out since the last call, or BI_ERR_INVALID_ARG when a serving operation
 * met a slot, page or length that does not exist (detail in
 * bi_last_error_message()).
 */
bi_status bi_device_status(bi_stream stream);

/*
 * Test hook for the failure path: launches one block that waits, with a
 * limit of `limit_ns` nanoseconds (1 ms .. 2 s), on a barrier that nothing
 * ever signals.  The wait runs out, the kernel records BI_ERR_TIMEOUT and
 * exits normally; the next bi_device_status() returns it.
 */
bi_status bi_debug_expire_wait(uint64_t limit_ns, bi_stream stream);

/* Static, human-readable name of a status code. */
const char* bi_status_string(bi_status status);

/* Reason for the last non-OK status returned on this thread ("" if none). */
const char* bi_last_error_message(void);

/* ABI version of this header (incremented on any signature change). */
int32_t bi_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BI_H_ */
