// bi_logprobs.cu -- log probabilities of given tokens, entropies and the K
// best alternatives of each row of logits:
//   lp = RN(RN(x_tok - mx) - lse),  lse = logf(S),  S = sum expf(RN(x_j - mx)),
//   H  = lse - (sum e_j (x_j - mx)) / S.
// mx and S are taken in the order of the invariant row reductions
// (bi_rows.cuh), so lp is bit for bit the element that bi_log_softmax_lastdim
// gives, without its R x N output being written.
//
// Alternatives.  The selection is exact, so it is free to use any order.  The
// maxima of 128 groups of a CTA's threads come with the maximum; the K-th
// largest of them, tau, is a lower bound of the K-th largest logit (K distinct
// elements reach it) and a close one: K of 128 groups are reached by about
// 128 ln(128 / (128 - K)) elements, 22 for K = 20.  Elements >= tau are
// collected and ranked by counting.  A CTA whose candidates overflow their
// buffer (rows with thousands of equal entries, such as all but a few tokens
// forbidden) and rows with NaNs extract one element a round instead.
//
// Bound: the row is read once; for 16-bit logits the conversions,
// exponentials and sums of an element cost about as much issue time as its
// two bytes cost bandwidth.
#include "bi_rows.cuh"
#include "bi_serve.h"

namespace bi {
namespace {

constexpr int kMaxTop = 64;
constexpr int kGroups = 128;     // groups of threads whose maxima bound the K-th largest
constexpr int kBuffer = 1024;    // candidates of a CTA

struct Cand {
  float v;
  int32_t j;
};

// Total order of the alternatives as an integer: NaN above every number, -0
// equal to +0, and the lower index above the higher one among equals.
__device__ __forceinline__ uint64_t order_key(float v, int j) {
  uint32_t b = __float_as_uint(v + 0.0f);
  b = v != v ? 0xffffffffu : (b >> 31 ? ~b : b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint32_t)(~j);
}

struct TopShared {
  float group[kGroups];
  Cand cand[kBuffer];
  Cand top[kMaxTop];  // the CTA's best K, best first
  uint64_t best[32];
  float tau;
  int count;
};

// f(value, index) over the thread's elements of the chunk.
template <int T, int X, int GN, typename F>
__device__ __forceinline__ void chunk_visit_at(const RowChunk<X, GN>& ch, int N, F&& f) {
#pragma unroll
  for (int k = 0; k < GN; ++k) {
    const int n = chunk_n<T, X>(ch, k, N);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) f(word_val<X>(ch.w[k], i), 4 * (ch.g0 + k * T) + i);
  }
}

// The CTA's best K of the elements that visit(f(value, index)) walks over, in
// sm.top; lm: the thread's maximum; plain: no NaN among them.  At least K
// elements in the CTA.  Every thread calls it.
template <int NT, typename V>
__device__ __forceinline__ void select_top(TopShared& sm, float lm, bool plain, int K, V&& visit) {
  constexpr int L = NT / kGroups;  // lanes of a group
  const int tid = threadIdx.x;
  float gm = lm;
#pragma unroll
  for (int x = 1; x < L; x <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, x));
  if (tid % L == 0) sm.group[tid / L] = gm;
  if (tid == 0) sm.count = 0;
  __syncthreads();
  if (tid < kGroups) {
    const float v = sm.group[tid];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < kGroups; ++i) {
      const float o = sm.group[i];
      rank += o > v || (o == v && i < tid);
    }
    if (rank == K - 1) sm.tau = v;
  }
  __syncthreads();
  if (plain) {
    const float tau = sm.tau;
    if (lm >= tau) {
      visit([&](float v, int j) {
        if (v >= tau) {
          const int at = atomicAdd(&sm.count, 1);  // the order of the buffer does not matter
          if (at < kBuffer) sm.cand[at] = {v, j};
        }
      });
    }
    __syncthreads();
    const int n = sm.count;
    if (n <= kBuffer) {
      for (int c = tid; c < n; c += NT) {
        const Cand x = sm.cand[c];
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          const Cand o = sm.cand[i];
          rank += o.v > x.v || (o.v == x.v && o.j < x.j);
        }
        if (rank < K) sm.top[rank] = x;
      }
      __syncthreads();
      return;
    }
  }
  // one element a round: the largest below the last one
  uint64_t last = ~0ull;
  bool first = true;
  for (int r = 0; r < K; ++r) {
    uint64_t best = 0;
    float bv = 0.0f;
    visit([&](float v, int j) {
      const uint64_t k = order_key(v, j);
      if ((first || k < last) && k > best) best = k, bv = v;
    });
    uint64_t all = best;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, all, x);
      all = o > all ? o : all;
    }
    __syncthreads();
    if ((tid & 31) == 0) sm.best[tid >> 5] = all;
    __syncthreads();
    all = sm.best[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) all = sm.best[w] > all ? sm.best[w] : all;
    if (best == all) sm.top[r] = {bv, (int32_t)~(uint32_t)all};
    last = all;
    first = false;
  }
  __syncthreads();
}

// Row r's token, and its log probability.
__device__ __forceinline__ float token_logprob(const LogprobParams& p, const void* x, int64_t r, float m, float lse) {
  const int64_t tok = p.tok64 ? __ldg(static_cast<const long long*>(p.tokens) + r)
                              : (int64_t)__ldg(static_cast<const int*>(p.tokens) + r);
  if (tok < 0 || tok >= p.N) return -INFINITY;
  return __fsub_rn(__fsub_rn(row_load(x, p.x_kind, tok), m), lse);
}

// e = expf(x - m) and its share of the entropy's sum; a zero e adds zero.
__device__ __forceinline__ void add_exp(float v, float m, float& s, float& h) {
  const float z = __fsub_rn(v, m), e = expf(z);
  s = __fadd_rn(s, e);
  h = fmaf(e, fmaxf(z, -1e4f), h);  // expf is 0 well above -1e4
}

// Rows of up to 4 G 256 elements: one block of 256 threads a row, its first T
// threads forming the row's team.
template <int T, int X>
__global__ void __launch_bounds__(256) logprobs_small_kernel(const LogprobParams p) {
  __shared__ TopShared sm;
  __shared__ float red[3][8];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, N = (int)p.N;
  const char* x = static_cast<const char*>(p.x) + row * p.ld_x * Elem<X>::kBytes;
  const bool vec = aligned4(x, Elem<X>::kBytes);
  const RowSpan span = row_span(N, 1, 0);
  RowChunk<X> ch;
  float lm = -INFINITY;
  if (tid < T) {
    load_chunk<T, X>(x, vec, N, span, tid, 0, ch);
    chunk_visit<T, X>(ch, N, [&](float v) { lm = fmaxf(lm, v); });
  }
  float m = rows_warp_max(lm);
  if ((tid & 31) == 0) red[0][tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w) m = fmaxf(m, red[0][w]);
  float s = 0.0f, h = 0.0f;
  if (tid < T) chunk_visit<T, X>(ch, N, [&](float v) { add_exp(v, m, s, h); });
  s = rows_warp_sum(s), h = rows_warp_sum(h);
  if ((tid & 31) == 0) red[1][tid >> 5] = s, red[2][tid >> 5] = h;
  __syncthreads();
  s = red[1][0], h = red[2][0];
#pragma unroll
  for (int w = 1; w < T / 32; ++w) s = __fadd_rn(s, red[1][w]), h = __fadd_rn(h, red[2][w]);
  const float lse = logf(s);
  if (tid == 0) {
    p.lp[row] = token_logprob(p, x, row, m, lse);
    if (p.entropy) p.entropy[row] = lse - __fdiv_rn(h, s);
  }
  if (p.K == 0) return;
  const bool plain = s == s;
  if constexpr (T == 256) {
    select_top<256>(sm, lm, plain, p.K, [&](auto&& f) { chunk_visit_at<T, X>(ch, N, f); });
  } else {
    // a small team's row again, spread over the whole block
    float bm = -INFINITY;
    for (int j = tid; j < N; j += 256) bm = fmaxf(bm, row_load(x, X, j));
    select_top<256>(sm, bm, plain, p.K, [&](auto&& f) {
      for (int j = tid; j < N; j += 256) f(row_load(x, X, j), j);
    });
  }
  if (tid < p.K) {
    const Cand c = sm.top[tid];
    p.top_ids[row * p.K + tid] = c.j;
    p.top_lp[row * p.K + tid] = __fsub_rn(__fsub_rn(c.v, m), lse);
  }
}

// Longer rows: a team of 1024 threads, or a cluster of cl such teams, each
// with a contiguous slice of the row.
template <int X>
__global__ void __launch_bounds__(1024, 1) logprobs_kernel(const LogprobParams p) {
  constexpr int T = 1024;
  __shared__ TopShared sm;
  __shared__ float red[32];
  __shared__ float cx[2];
  const int tid = threadIdx.x, N = (int)p.N, cl = p.cl;
  const int64_t row = blockIdx.x / cl;
  const int rank = (int)(blockIdx.x % cl);
  const char* x = static_cast<const char*>(p.x) + row * p.ld_x * Elem<X>::kBytes;
  const bool vec = aligned4(x, Elem<X>::kBytes);
  const RowSpan span = row_span(N, cl, rank);
  const int nch = row_chunks<T, X>(span);
  int slot = 0;
  RowChunk<X> ch;
  float lm = -INFINITY;
  for (int c = 0; c < nch; ++c) {
    load_chunk<T, X>(x, vec, N, span, tid, c, ch);
    chunk_visit<T, X>(ch, N, [&](float v) { lm = fmaxf(lm, v); });
  }
  float m = team_max<T>(lm, red);
  if (cl > 1) m = cluster_combine<true>(m, cx, cl, slot);
  float s = 0.0f, h = 0.0f;
  for (int c = 0; c < nch; ++c) {
    if (nch > 1) load_chunk<T, X>(x, vec, N, span, tid, c, ch);
    chunk_visit<T, X>(ch, N, [&](float v) { add_exp(v, m, s, h); });
  }
  s = team_sum<T>(s, red);
  if (cl > 1) s = cluster_combine<false>(s, cx, cl, slot);
  h = team_sum<T>(h, red);
  if (cl > 1) h = cluster_combine<false>(h, cx, cl, slot);
  const float lse = logf(s);
  if (tid == 0 && rank == 0) {
    p.lp[row] = token_logprob(p, x, row, m, lse);
    if (p.entropy) p.entropy[row] = lse - __fdiv_rn(h, s);
  }
  if (p.K > 0) {
    select_top<T>(sm, lm, s == s, p.K, [&](auto&& f) {
      for (int c = 0; c < nch; ++c) {
        if (nch > 1) load_chunk<T, X>(x, vec, N, span, tid, c, ch);
        chunk_visit_at<T, X>(ch, N, f);
      }
    });
    if (cl > 1) {
      // rank 0 ranks the CTAs' lists; its own candidates are done with
      cluster_sync_all();
      if (rank == 0) {
        const int n = cl * p.K;
        if (tid < n) {
          const uint32_t a = cluster_map_shared(smem_u32(&sm.top[tid % p.K]), (uint32_t)(tid / p.K));
          Cand c;
          c.v = ld_shared_cluster_f32(a);
          c.j = (int32_t)__float_as_uint(ld_shared_cluster_f32(a + 4));
          sm.cand[tid] = c;
        }
        __syncthreads();
        if (tid < n) {
          const Cand c = sm.cand[tid];
          const uint64_t key = order_key(c.v, c.j);
          int at = 0;
          for (int i = 0; i < n; ++i) at += order_key(sm.cand[i].v, sm.cand[i].j) > key;
          if (at < p.K) {
            p.top_ids[row * p.K + at] = c.j;
            p.top_lp[row * p.K + at] = __fsub_rn(__fsub_rn(c.v, m), lse);
          }
        }
      }
    } else if (tid < p.K) {
      const Cand c = sm.top[tid];
      p.top_ids[row * p.K + tid] = c.j;
      p.top_lp[row * p.K + tid] = __fsub_rn(__fsub_rn(c.v, m), lse);
    }
  }
  if (cl > 1) cluster_sync_all();  // no CTA leaves while a peer may read its totals or list
}

template <int X>
void launch_x(int T, const LogprobParams& p, cudaStream_t stream) {
  const unsigned rows = (unsigned)p.R;
  if (T == 32) {
    logprobs_small_kernel<32, X><<<rows, 256, 0, stream>>>(p);
  } else if (T == 64) {
    logprobs_small_kernel<64, X><<<rows, 256, 0, stream>>>(p);
  } else if (T == 256) {
    logprobs_small_kernel<256, X><<<rows, 256, 0, stream>>>(p);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * (unsigned)p.cl);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, logprobs_kernel<X>, p);
  }
}

}  // namespace

bi_status launch_logprobs(const LogprobParams& p_in, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  LogprobParams p = p_in;
  const int T = row_team_size(p.N, p.x_kind);
  p.cl = T == 1024 ? row_cluster_size(p.N, p.x_kind) : 1;
  if (p.R * p.cl > INT32_MAX) {
    *why = "too many rows";
    return BI_ERR_INVALID_ARG;
  }
  if (p.x_kind == 2)
    launch_x<2>(T, p, stream);
  else if (p.x_kind == 1)
    launch_x<1>(T, p, stream);
  else
    launch_x<0>(T, p, stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("token log probabilities launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
