// bi_logprobs.cu -- log probabilities of given tokens, entropies and the K
// best alternatives of each row of logits, in one pass over the row.
//
// With L = log2 e and a reference m' = RN(m L), t_j = RN(x_j L - m') is one
// fused multiply-add (the product is exact inside it), e_j = 2^t_j the SFU's
// approximation, and
//   S = sum e_j,  H = sum e_j t_j
// are kept relative to a running maximum: going from m' to M' = m' + d turns
// them into 2^-d S and 2^-d (H - d S).  Then, with M the row's maximum,
//   log-sum = ln S + ln 2 (M' - M L)        (what RN(M L) left out, one fma)
//   lp      = (x_tok - M) - log-sum,   entropy = ln S - ln 2 H / S.
// 2048 rows of 128256 bf16 logits (525 MB, 77 us at the copy rate) take 87 us,
// 9.6 instructions an element.  Two passes with expf
// over differences, which would give the log-softmax entry's own bits, cost 21
// and took 229 us in the best of three layouts (a row in the registers of a
// cluster 334 us, streamed twice 229 us).  8 fp32 rows with 20 alternatives
// take 6.9 us.
//
// Order.  256 threads; a thread's chunk of a slice is four 16-byte units, 256
// units apart (32 elements of 16 bits or 16 of fp32; a slice is 16 KB), reduced
// relative to its own maximum.  The slices are split, by N alone, into at most
// eight equal groups; a thread joins the slices of a group in order, then the
// groups in order; then the 32 lanes of a warp by a fixed tree, then the eight
// warps by another.  Rows in hundreds are taken a CTA each; for fewer the
// groups are spread over a cluster of 2, 4 or 8 CTAs, whose threads hand their
// groups' states to the first CTA's through distributed shared memory.  The
// joins are the same, so the bits are.
//
// Loads.  Every thread copies its own chunks into a shared-memory ring of its
// own, half a slice a stage, by 16-byte asynchronous copies, and the ring runs
// on from row to row: no barrier and no producer, 128 KB an SM in flight.  Rows
// that are not on 16-byte boundaries are copied from the boundary before, and a
// thread puts its units together from its own and the next lane's, by a shift
// that is the row's (N = 128257 110 us, 128258 107; words loaded straight into
// registers 177 and 113; rows of less than a slice are slower for it, 20000 of
// 1001 123 us against 113).
//
// Alternatives.  The selection is exact, so it is free to use any order.  The
// K-th largest, tau, of the maxima of 2 K or more groups of threads is a lower
// bound of the K-th largest logit (K distinct elements reach it) and a close
// one: K of 2 K groups are reached by about 1.4 K elements.  The chunks whose
// maximum reaches tau are read again (out of L2), all at once, and the elements
// that do are ranked by counting.  (A thread reading its own chunks again, one
// latency after the other: 19 us in place of 7 for the 8 rows.)  Rows with more
// than 512 such elements (ties) and rows with NaNs extract one element a round
// instead.  Where fewer than K groups have an allowed token, tau is -inf and
// the whole row is read again, an element a thread: right, and slow (10 tokens
// allowed, K = 20: 8 bf16 rows 38 us in place of 7.5, 2048 rows 334 of 95).
#include "bi_rows.cuh"
#include "bi_serve.h"

namespace bi {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnits = 4;        // 16-byte units of a thread in a slice
constexpr int kHalf = kUnits / 2;  // units of a ring stage
constexpr int kStages = 5;
constexpr int kGroups = 8;       // groups of slices
constexpr int kMaxTop = 64;
constexpr int kMaxima = 128;     // thread groups whose maxima bound the K-th largest
constexpr int kBuffer = 512;     // candidates
constexpr int kHits = 1024;      // chunks that hold candidates
constexpr float kL = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int X>
struct Slice {
  static constexpr int E = 16 / Elem<X>::kBytes;        // elements of a unit
  static constexpr int kSlice = kThreads * kUnits * E;  // 8192 or 4096
};
// How a row of N elements is cut: a function of N and the type alone.
struct Cut {
  int slices, per_group, groups;
};
__host__ __device__ inline Cut cut_row(int64_t N, int slice) {
  Cut c;
  c.slices = (int)((N + slice - 1) / slice);
  c.per_group = (c.slices + kGroups - 1) / kGroups;
  c.groups = (c.slices + c.per_group - 1) / c.per_group;
  return c;
}

struct Cand {
  float v;
  int32_t j;
};
// m: m', the reference in base-2 units; S and H relative to it.
struct State {
  float m, S, H;
};
constexpr float kNone = -3e38f;  // the reference of nothing

__device__ __forceinline__ State join(const State& a, const State& b) {
  const float m = fmaxf(a.m, b.m);
  // below -150 the factor is 0 all the same
  const float da = fmaxf(a.m - m, -150.0f), db = fmaxf(b.m - m, -150.0f);
  const float fa = ex2_approx(da), fb = ex2_approx(db);
  return {m, fmaf(fb, b.S, __fmul_rn(fa, a.S)), fmaf(fb, fmaf(db, b.S, b.H), __fmul_rn(fa, fmaf(da, a.S, a.H)))};
}
__device__ __forceinline__ State shuffle_down(const State& s, int x) {
  return {__shfl_down_sync(0xffffffffu, s.m, x), __shfl_down_sync(0xffffffffu, s.S, x),
          __shfl_down_sync(0xffffffffu, s.H, x)};
}

struct Shared {
  unsigned char ring[kStages][(kThreads + kWarps) * kHalf * 16];
  float best[kGroups][kThreads];  // the threads' maxima in each group of slices
  __align__(16) float group[kMaxima];
  Cand cand[kBuffer];
  uint16_t hit[kHits];  // thread + kThreads * group
  uint64_t round[kWarps];
  State warp[kWarps];
  float max[kWarps];
  float tau, M, lse;
  int count, hits, kind;  // kind of row: kUsual, ...
};
enum : int { kUsual = 0, kNaN = 1, kUnusual = 2 };
// The first CTA of a cluster also takes the groups' states.
struct SharedCluster {
  Shared s;
  float4 state[kGroups][kThreads];
};

// A reference is a rounded product, so the largest t of a chunk is what the
// rounding left out: up to 2^-24 |m'|, no longer a small number when m' is not.
// Hence references are held above a floor, whose chunks (of masked entries)
// weigh nothing in a usual row; rows whose maximum is not clear of the floor,
// or as large, are summed by the definition.  16-bit entries are held above it
// themselves, so that -inf has a finite t: within a usual row e is 0 there, and
// e t with it.
template <int X>
struct Floor {  // -2^21; fp16's lowest number
  static constexpr float v = X == 1 ? -65504.0f : -2097152.0f;
};
template <int X>
__device__ __forceinline__ bool usual(float m) { return m > (X == 1 ? -6e4f : -1048576.0f) && m < 1048576.0f; }
// Larger of two 16-bit pairs, a NaN giving way to a number.
template <int X>
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (X == 1)
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The same, a NaN staying one.
template <int X>
__device__ __forceinline__ uint32_t max16x2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (X == 1)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A thread's chunk of 16 words: its state and its maximum.  Entries at -inf
// (e = 0) add 0 to H: those of 16 bits by their floor, half an instruction an
// element (an instruction to hold t itself: 3 us more); an fp32 t is held above
// -200 there.
template <int X>
__device__ __forceinline__ State reduce_chunk(const uint32_t (&w)[4 * kUnits], float& best) {
  constexpr int NW = 4 * kUnits;
  float m;
  if constexpr (X == 2) {
    m = __uint_as_float(w[0]);
#pragma unroll
    for (int i = 1; i < NW; ++i) m = fmaxf(m, __uint_as_float(w[i]));
  } else {
    uint32_t m2 = w[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) m2 = max16x2<X>(m2, w[i]);
    m = fmaxf(half_bits_to_float(m2 & 0xffffu, X), half_bits_to_float(m2 >> 16, X));
  }
  best = m;
  const float r = __fmul_rn(fmaxf(m, Floor<X>::v), kL);
  const uint64_t l2 = pack2(kL, kL), r2 = pack2(-r, -r);
  uint64_t S2 = pack2(0.0f, 0.0f), H2 = S2;
#pragma unroll
  for (int i = 0; i < NW; i += X == 2 ? 2 : 1) {
    uint64_t v;
    if constexpr (X == 2) {
      v = pack2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
    } else {
      const uint32_t f = max16x2_nan<X>(w[i], X == 1 ? 0xfbfffbffu : 0xca00ca00u);  // the floor, twice
      v = pack2(half_bits_to_float(f & 0xffffu, X), half_bits_to_float(f >> 16, X));
    }
    const uint64_t t = fma2(v, l2, r2);
    float t0, t1;
    unpack2(t, t0, t1);
    const uint64_t e = pack2(ex2_approx(t0), ex2_approx(t1));
    S2 = add2(S2, e);
    H2 = fma2(e, X == 2 ? pack2(fmaxf(t0, -200.0f), fmaxf(t1, -200.0f)) : t, H2);
  }
  float s0, s1, h0, h1;
  unpack2(S2, s0, s1);
  unpack2(H2, h0, h1);
  return {r, __fadd_rn(s0, s1), __fadd_rn(h0, h1)};
}

// Elements j0 .. of the row as a unit's four words, whatever the row's
// alignment; only what lies inside the row is read.
template <int X>
__device__ __forceinline__ void load_unit_any(const char* x, int j0, int N, uint32_t* w) {
  constexpr int E = Slice<X>::E;
  if constexpr (X == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = j0 + i < N ? __ldg(reinterpret_cast<const uint32_t*>(x) + j0 + i) : 0u;
  } else {
    const char* a = x + (int64_t)j0 * 2;
    if (reinterpret_cast<uintptr_t>(a) % 4 == 0 && j0 + E <= N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(a) + i);
    } else if (reinterpret_cast<uintptr_t>(a) % 4 != 0 && j0 > 0 && j0 + E < N) {
      uint32_t q[5];  // the words from the element before to the element after
#pragma unroll
      for (int i = 0; i < 5; ++i) q[i] = __ldg(reinterpret_cast<const uint32_t*>(a - 2) + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __byte_perm(q[i], q[i + 1], 0x5432);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t h[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          h[k] = j0 + 2 * i + k < N ? __ldg(reinterpret_cast<const unsigned short*>(a) + 2 * i + k) : 0u;
        w[i] = h[0] | (h[1] << 16);
      }
    }
  }
}
// Replaces the elements past the row's end by -inf.
template <int X>
__device__ __forceinline__ void pad_unit(uint32_t* w, int j0, int N) {
  constexpr int E = Slice<X>::E;
  if (j0 + E <= N) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (X == 2) {
      if (j0 + i >= N) w[i] = 0xff800000u;
    } else {
      constexpr uint32_t low = X == 1 ? 0xfc00u : 0xff80u;
      if (j0 + 2 * i >= N) w[i] = (w[i] & 0xffff0000u) | low;
      if (j0 + 2 * i + 1 >= N) w[i] = (w[i] & 0xffffu) | (low << 16);
    }
  }
}

// Total order of the alternatives as an integer: NaN above every number, -0
// equal to +0, and the lower index above the higher one among equals.
__device__ __forceinline__ uint64_t order_key(float v, int j) {
  uint32_t b = __float_as_uint(v + 0.0f);
  b = v != v ? 0xffffffffu : (b >> 31 ? ~b : b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint32_t)(~j);
}

__device__ __forceinline__ void add_candidate(Shared& sm, float y, int j) {
  // of the entries at -inf the first 2 kMaxTop are enough: fewer than kMaxTop of
  // those are not at -inf, or K better elements exist
  if (!(y > -INFINITY || j < 2 * kMaxTop)) return;
  const int at = atomicAdd(&sm.count, 1);  // the order of the buffer does not matter
  if (at < kBuffer) sm.cand[at] = {y, j};
}
// Collects the elements that reach tau, by the whole CTA: the chunks (of a
// thread in a group of slices) whose maximum does are listed, then their units
// are read again, a unit a thread, so that one load's latency covers them all.
template <int X>
__device__ __forceinline__ void collect(Shared& sm, const char* x, int N, const Cut& cut, bool aligned) {
  constexpr int E = Slice<X>::E;
  const int tid = threadIdx.x;
  const float tau = sm.tau;
  for (int g = 0; g < cut.groups; ++g) {
    if (sm.best[g][tid] < tau) continue;
    const int at = atomicAdd(&sm.hits, 1);
    if (at < kHits) sm.hit[at] = (uint16_t)(g * kThreads + tid);
  }
  __syncthreads();
  const int hits = sm.hits;
  if (hits > kHits) {  // nearly all: the row in order
    for (int j = tid; j < N; j += kThreads) {
      const float y = row_load(x, X, j);
      if (y >= tau) add_candidate(sm, y, j);
    }
    return;
  }
  const int units = cut.per_group * kUnits;  // of a chunk
  for (int i = tid; i < hits * units; i += kThreads) {
    const int h = i / units, r = i - h * units, who = sm.hit[h];
    const int s = who / kThreads * cut.per_group + r / kUnits;
    const int j0 = s * Slice<X>::kSlice + ((r % kUnits) * kThreads + who % kThreads) * E;
    if (j0 >= N) continue;
    uint32_t w[4];
    if (aligned && j0 + E <= N) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)j0 * Elem<X>::kBytes));
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
      load_unit_any<X>(x, j0, N, w);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float y =
          X == 2 ? __uint_as_float(w[k & 3]) : half_bits_to_float((w[k >> 1 & 3] >> (16 * (k & 1))) & 0xffffu, X);
      if (y >= tau && j0 + k < N) add_candidate(sm, y, j0 + k);
    }
  }
}

// The best K one element a round, the largest below the last one: put(rank,
// element).  Every thread calls it.
template <int X, typename P>
__device__ __forceinline__ void extract_top(Shared& sm, const char* x, int N, int K, P&& put) {
  const int tid = threadIdx.x;
  uint64_t last = ~0ull;
  for (int r = 0; r < K; ++r) {
    uint64_t mine = 0;
    float mv = 0.0f;
    for (int j = tid; j < N; j += kThreads) {
      const float y = row_load(x, X, j);
      const uint64_t k = order_key(y, j);
      if ((r == 0 || k < last) && k > mine) mine = k, mv = y;
    }
    uint64_t top = mine;
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, top, y);
      top = o > top ? o : top;
    }
    __syncthreads();
    if ((tid & 31) == 0) sm.round[tid >> 5] = top;
    __syncthreads();
    top = sm.round[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = sm.round[w] > top ? sm.round[w] : top;
    if (mine == top) put(r, Cand{mv, (int32_t)~(uint32_t)top});
    last = top;
  }
}

// The same sums from the definition, for rows whose maximum is out of the
// ordinary (all entries masked by low numbers, or enormous ones): expf
// over differences, thread t over elements t, t + 256, ..., warps in order.
template <int X>
__device__ __forceinline__ void sums_by_definition(Shared& sm, const char* x, int N, float M, float& S, float& H) {
  const int tid = threadIdx.x;
  float s = 0.0f, h = 0.0f;
  for (int j = tid; j < N; j += kThreads) {
    const float z = row_load(x, X, j) - M, e = expf(z);
    s += e;
    h = fmaf(e, fmaxf(z, -1e4f), h);
  }
  s = rows_warp_sum(s), h = rows_warp_sum(h);
  __syncthreads();
  if ((tid & 31) == 0) sm.warp[tid >> 5] = {0.0f, s, h};
  __syncthreads();
  S = sm.warp[0].S, H = sm.warp[0].H;
  for (int w = 1; w < kWarps; ++w) S = __fadd_rn(S, sm.warp[w].S), H = __fadd_rn(H, sm.warp[w].H);
  __syncthreads();  // read before the next row's states are written there
}

// A row's results from the threads' states, by the whole CTA; thread 0 brings
// the token and its logit.  Four barriers; what a barrier of the next row
// protects is not protected again.
template <int X>
__device__ __forceinline__ void finish_row(const LogprobParams& p, Shared& sm, int64_t row, const char* x, int N,
                                           const Cut& cut, State st, float best, int64_t tok, float xt, bool aligned) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = p.K;
#pragma unroll
  for (int y = 16; y > 0; y >>= 1) st = join(st, shuffle_down(st, y));
  // maxima of groups of neighbouring lanes, at least 2 K of them, and the warp's
  const int groups = K <= 8 ? 16 : K <= 16 ? 32 : K <= 32 ? 64 : kMaxima, lanes = kThreads / groups;
  float v = best, gm = best;
#pragma unroll
  for (int y = 1; y < 32; y <<= 1) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, y));
    if (2 * y <= lanes) gm = v;
  }
  if (tid % lanes == 0) sm.group[tid / lanes] = gm;
  if (lane == 0) sm.warp[warp] = st, sm.max[warp] = v;
  __syncthreads();
  if (warp == 0) {
    State all = lane < kWarps ? sm.warp[lane] : State{kNone, 0.0f, 0.0f};
    const float M = rows_warp_max(lane < kWarps ? sm.max[lane] : -INFINITY);
#pragma unroll
    for (int y = kWarps / 2; y > 0; y >>= 1) all = join(all, shuffle_down(all, y));
    if (lane == 0) {
      const bool u = usual<X>(M);
      const float ln_s = logf(all.S), lse = fmaf(kLn2, fmaf(-M, kL, all.m), ln_s);
      sm.M = M, sm.lse = lse;
      sm.count = 0, sm.hits = 0;
      sm.kind = !u ? kUnusual : all.S != all.S ? kNaN : kUsual;
      if (u) {
        p.lp[row] = tok >= 0 && tok < p.N ? __fsub_rn(__fsub_rn(xt, M), lse) : -INFINITY;
        if (p.entropy) p.entropy[row] = fmaf(-kLn2, __fdiv_rn(all.H, all.S), ln_s);
      }
    }
  } else if (tid - 32 < groups) {
    // the K-th largest of the groups' maxima
    const int i = tid - 32;
    const float g = sm.group[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < groups; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(&sm.group[j]);
      rank += (o.x > g || (o.x == g && j < i)) + (o.y > g || (o.y == g && j + 1 < i)) +
              (o.z > g || (o.z == g && j + 2 < i)) + (o.w > g || (o.w == g && j + 3 < i));
    }
    if (rank == K - 1) sm.tau = g;
  }
  __syncthreads();
  const float M = sm.M;
  float lse = sm.lse;
  int kind = sm.kind;
  if (kind == kUnusual) {
    float S, H;
    sums_by_definition<X>(sm, x, N, M, S, H);
    lse = logf(S);
    if (S != S) kind = kNaN;
    if (tid == 0) {
      p.lp[row] = tok >= 0 && tok < p.N ? __fsub_rn(__fsub_rn(xt, M), lse) : -INFINITY;
      if (p.entropy) p.entropy[row] = lse - __fdiv_rn(H, S);
    }
  }
  if (K == 0) return;
  auto put = [&](int r, const Cand& c) {
    p.top_ids[row * K + r] = c.j;
    p.top_lp[row * K + r] = __fsub_rn(__fsub_rn(c.v, M), lse);
  };
  if (kind != kNaN) collect<X>(sm, x, N, cut, aligned);
  __syncthreads();
  const int n = sm.count;
  if (kind != kNaN && n <= kBuffer) {
    for (int c = tid; c < n; c += kThreads) {
      const Cand y = sm.cand[c];
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const Cand o = sm.cand[i];
        rank += o.v > y.v || (o.v == y.v && o.j < y.j);
      }
      if (rank < K) put(rank, y);
    }
  } else {
    extract_top<X>(sm, x, N, K, put);
  }
}

__device__ __forceinline__ void copy_unit(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of a unit, then zeros.
__device__ __forceinline__ void copy_unit(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}

// A thread's half slice out of a stage whose units start 2 K bytes before the
// row's: each is the end of the thread's and the start of the next one's.
template <int K, int kPitch>
__device__ __forceinline__ void read_shifted(uint32_t src, uint32_t* w) {
#pragma unroll
  for (int u = 0; u < kHalf; ++u, src += kPitch, w += 4) {
    const uint4 a = ld_shared_v4(src), b = K ? ld_shared_v4(src + 16) : a;
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = K & 1 ? __byte_perm(v[i + K / 2], v[(i + K / 2 + 1) & 7], 0x5432) : v[i + K / 2];
  }
}
template <int X, int kPitch>
__device__ __forceinline__ void read_half(uint32_t src, int k, uint32_t* w) {
  switch (k) {
    case 0: return read_shifted<0, kPitch>(src, w);
    case 2: return read_shifted<2, kPitch>(src, w);
    case 4: return read_shifted<4, kPitch>(src, w);
    case 6: return read_shifted<6, kPitch>(src, w);
  }
  if constexpr (X != 2) {
    switch (k) {
      case 1: return read_shifted<1, kPitch>(src, w);
      case 3: return read_shifted<3, kPitch>(src, w);
      case 5: return read_shifted<5, kPitch>(src, w);
      case 7: return read_shifted<7, kPitch>(src, w);
    }
  }
}

// CL: rows are spread over clusters of p.cl CTAs, a row each; otherwise a
// persistent grid takes a row a CTA.  ALIGNED: rows on 16-byte boundaries.
template <int X, bool ALIGNED, bool CL>
__global__ void __launch_bounds__(kThreads, CL ? 2 : 4) logprobs_kernel(const LogprobParams p) {
  constexpr int E = Slice<X>::E, kSlice = Slice<X>::kSlice;
  extern __shared__ __align__(128) unsigned char dyn[];
  Shared& sm = *reinterpret_cast<Shared*>(dyn);
  const int tid = threadIdx.x, N = (int)p.N;
  const Cut cut = cut_row(N, kSlice);
  const int cl = CL ? p.cl : 1, rank = CL ? (int)(blockIdx.x % cl) : 0;
  const int64_t step = CL ? p.R : gridDim.x;  // a cluster has one row
  const int64_t first = CL ? blockIdx.x / cl : blockIdx.x;
  const int groups_here = (cut.groups + cl - 1) / cl;
  const int g_beg = min(cut.groups, rank * groups_here), g_end = min(cut.groups, g_beg + groups_here);
  const int s_beg = min(cut.slices, g_beg * cut.per_group), s_end = min(cut.slices, g_end * cut.per_group);
  const char* base = static_cast<const char*>(p.x);
  const int64_t ld = p.ld_x * Elem<X>::kBytes;

  // the thread's place in a stage, and the half slice to request next.  Rows off
  // 16-byte boundaries are copied from the boundary before: `off` bytes earlier,
  // a warp's 33rd unit by its last lane, and a first unit that would start
  // before the row not at all.
  constexpr int kPitch = (ALIGNED ? kThreads : kThreads + kWarps) * 16;  // of a unit in a stage
  constexpr uint32_t kStage = kHalf * kPitch;
  constexpr int kHalfBytes = kThreads * kHalf * 16;  // of the row, a half slice
  constexpr int kFull = (kHalf - 1) * kThreads * 16 + (ALIGNED ? 16 : 32);
  const uint32_t mine = smem_u32(sm.ring[0]) + (ALIGNED ? tid : tid + (tid >> 5)) * 16;
  const int halves = 2 * (s_end - s_beg);
  const bool last = !ALIGNED && (tid & 31) == 31;
  bool head = false;  // the thread's next unit starts before the row
  int64_t prow = first;
  int phalf = 0, stage = 0, left;
  const char* pa;
  auto start_row = [&]() {
    const char* x = base + prow * ld;
    const int off = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(x) & 15);
    pa = x - off + (int64_t)s_beg * kSlice * Elem<X>::kBytes + tid * 16;
    left = (N - s_beg * kSlice) * Elem<X>::kBytes - tid * 16 + off;  // bytes from pa to the row's end; below 2^27
    if (!ALIGNED) head = tid == 0 && s_beg == 0 && off != 0;
  };
  start_row();
  uint32_t pdst = mine;
  auto request = [&]() {
    if (prow < p.R && halves > 0) {
      if (left >= kFull && !head) {
#pragma unroll
        for (int u = 0; u < kHalf; ++u) {
          copy_unit(pdst + u * kPitch, pa + u * (kThreads * 16));
          if (last) copy_unit(pdst + u * kPitch + 16, pa + u * (kThreads * 16) + 16);
        }
      } else {
        // (what is not copied is past the row's end, and replaced)
#pragma unroll
        for (int u = 0; u < kHalf; ++u) {
          const int have = left - u * (kThreads * 16);
          if (have > 0 && !(u == 0 && head)) copy_unit(pdst + u * kPitch, pa + u * (kThreads * 16), min(16, have));
          if (last && have > 16) copy_unit(pdst + u * kPitch + 16, pa + u * (kThreads * 16) + 16, min(16, have - 16));
        }
        head = false;
      }
      pa += kHalfBytes, left -= kHalfBytes;
      if (++phalf == halves) {
        phalf = 0, prow += step;
        if constexpr (ALIGNED)
          pa += step * ld - (int64_t)halves * kHalfBytes, left += halves * kHalfBytes;
        else
          start_row();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    pdst = pdst == mine + (kStages - 1) * kStage ? mine : pdst + kStage;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) request();
  if constexpr (CL) cluster_sync_all();  // the first CTA's shared memory is there

  for (int64_t row = first; row < p.R; row += step) {
    const char* x = base + row * ld;
    const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15);
    int64_t tok = -1;  // its logit, requested early
    float xt = 0.0f;
    if (tid == 0 && rank == 0) {
      tok = p.tok64 ? __ldg(static_cast<const long long*>(p.tokens) + row)
                    : (int64_t)__ldg(static_cast<const int*>(p.tokens) + row);
      if (tok >= 0 && tok < p.N) xt = row_load(x, X, tok);
    }
    State total = {kNone, 0.0f, 0.0f};
    float best = -INFINITY;
    for (int g = g_beg; g < g_end; ++g) {
      State st = {kNone, 0.0f, 0.0f};
      float gbest = -INFINITY;
      for (int s = g * cut.per_group; s < min(cut.slices, (g + 1) * cut.per_group); ++s) {
        const int j0 = s * kSlice + tid * E;
        uint32_t w[4 * kUnits];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
          if constexpr (ALIGNED) {
#pragma unroll
            for (int u = 0; u < kHalf; ++u) {
              const uint4 q = ld_shared_v4(mine + stage * kStage + u * kPitch);
              const int i = 4 * (half * kHalf + u);
              w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
            }
          } else {
            __syncwarp();  // the next lane's units are here, and the stage before this one is read
            read_half<X, kPitch>(mine + stage * kStage, off >> 1, w + 4 * kHalf * half);
          }
          stage = stage + 1 == kStages ? 0 : stage + 1;
          request();  // into the stage read before this one
        }
        if (!ALIGNED && j0 == 0 && off != 0) load_unit_any<X>(x, 0, N, w);
        if ((s + 1) * kSlice > N) {
          if (j0 >= N) continue;  // nothing of this slice is this thread's
#pragma unroll
          for (int u = 0; u < kUnits; ++u) pad_unit<X>(w + 4 * u, j0 + u * kThreads * E, N);
        }
        float b;
        st = join(st, reduce_chunk<X>(w, b));
        gbest = fmaxf(gbest, b);
      }
      if constexpr (CL) {
        const uint32_t to = smem_u32(&reinterpret_cast<SharedCluster*>(dyn)->state[g][tid]);
        st_cluster_v4(cluster_map_shared(to, 0), st.m, st.S, st.H, gbest);
      } else {
        total = join(total, st);
        sm.best[g][tid] = gbest;
        best = fmaxf(best, gbest);
      }
    }
    if constexpr (CL) {
      cluster_sync_all();  // all groups' states are with the first CTA
      if (rank != 0) return;
      for (int g = 0; g < cut.groups; ++g) {
        const float4 q = reinterpret_cast<SharedCluster*>(dyn)->state[g][tid];
        total = join(total, {q.x, q.y, q.z});
        sm.best[g][tid] = q.w;
        best = fmaxf(best, q.w);
      }
    }
    finish_row<X>(p, sm, row, x, N, cut, total, best, tok, xt, ALIGNED);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int X, bool ALIGNED>
cudaError_t launch(const LogprobParams& p_in, int num_sms, cudaStream_t stream) {
  LogprobParams p = p_in;
  const Cut cut = cut_row(p.N, Slice<X>::kSlice);
  // Clusters while their CTAs fit the SMs, two each.
  p.cl = 1;
  while (2 * p.cl <= cut.groups && p.R * 2 * p.cl <= 2 * num_sms) p.cl *= 2;
  constexpr int kSlot = 44 + (ALIGNED ? 0 : 6) + 2 * X;
  const bool clusters = p.cl > 1;
  const void* fn = clusters ? reinterpret_cast<const void*>(&logprobs_kernel<X, ALIGNED, true>)
                            : reinterpret_cast<const void*>(&logprobs_kernel<X, ALIGNED, false>);
  const int bytes = clusters ? (int)sizeof(SharedCluster) : (int)sizeof(Shared);
  static_assert(2 * (sizeof(SharedCluster) + 1024) <= 228 * 1024 && 4 * (sizeof(Shared) + 1024) <= 228 * 1024,
                "shared memory of an SM");
  cudaError_t e = set_smem_once(fn, bytes, kSlot + clusters);
  if (e != cudaSuccess) return e;
  if (!clusters) {
    const unsigned grid = (unsigned)std::min<int64_t>(p.R, 4 * (int64_t)num_sms);
    logprobs_kernel<X, ALIGNED, false><<<grid, kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.R * p.cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<X, ALIGNED, true>, p);
}

}  // namespace

bi_status launch_logprobs(const LogprobParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  const int esz = p.x_kind == 2 ? 4 : 2;
  const bool aligned = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ld_x * esz % 16 == 0;
  cudaError_t e;
  if (p.x_kind == 2)
    e = aligned ? launch<2, true>(p, dev.num_sms, stream) : launch<2, false>(p, dev.num_sms, stream);
  else if (p.x_kind == 1)
    e = aligned ? launch<1, true>(p, dev.num_sms, stream) : launch<1, false>(p, dev.num_sms, stream);
  else
    e = aligned ? launch<0, true>(p, dev.num_sms, stream) : launch<0, false>(p, dev.num_sms, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    *why = std::string("token log probabilities launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
