// bi_sample.cu -- one token of each row of logits, drawn by a given number u of
// [0, 1): with z_j = x_j / temperature, the filters keep a prefix of the tokens
// in the order of their logits (largest first, the lower index first among
// equals) --
//   top-k   the first k,
//   top-p   of those the shortest prefix with sum e^z_j >= top_p * all of it,
//   min-p   the tokens with e^(z_j - max z) >= min_p
// -- and the token is the first in index order at which the running sum of the
// kept e^z_j exceeds u times all of it.
//
// Exact sums.  A token is right or wrong, and a running sum in fp32 is off by
// 2^-24 of the sum at each of N places at which a token ends, so that one row
// in a few hundred would get a neighbour of its token.  A weight is therefore
// e^(z - max z) as a 64-bit integer, good to about 2^-33 of itself, and sums of
// integers do not depend on their order: not on the split of a row, not on the
// atomics that count, not on the batch.
//   e^(z - max) = 2^-y, y = (max - x) log2(e) / T in pairs of fp32 (difference
//   and product with their exact errors); y = k / 256 + r; the table's
//   2^(-(k mod 256) / 256) to 2^-41, times a polynomial of r ln 2 < 2^-9.5, whose
//   fp32 roundings are 2^-24 of it; shifted by k / 256.
// The unit is 2^-sh of the largest weight, sh = 62 - ceil(log2 N), at most 46.
//
// Work.  A row is a cluster's, a slice of it a CTA's, held in shared memory from
// the only read of it on.  Prefixes are found by counting: 2048 bins of y (of
// the bits of x, below) with the number and the weight of their elements, the
// weight as three sums of 16 bits in 32; the CTAs add up a share of the bins
// each; the bin where the k-th element, or the given weight, is reached is
// narrowed to its largest and smallest element, and binned again by their bits
// until it is one value, of which the first t by index are kept.  The draw sums
// the kept elements by warps' segments in index order, then looks into one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
#include "bi_quant.h"

namespace bi {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCl = 8;
constexpr float kRange = 62.0f;              // y from here on: weight 0
constexpr float kBinsPerBit = kBins / 64.0f;  // kRange of them end below kBins

// 2^40 2^(-j / 256), by repeated multiplication: off by 256 roundings of 2^-53 at
// most, and half a unit of the integer.
struct Powers {
  uint64_t v[256];
};
constexpr Powers powers() {
  Powers p = {};
  double x = 1099511627776.0;
  for (int j = 0; j < 256; ++j) {
    p.v[j] = (uint64_t)(x + 0.5);
    x *= 0.99729605608547012625;  // 2^(-1 / 256)
  }
  return p;
}
__device__ const Powers kPowers = powers();

struct Shared {
  uint64_t table[256];  // 2^40 2^(-j / 256)
  float tablef[256];    // 2^40 2^(-j / 256) again
  uint32_t n[kBins], w0[kBins], w1[kBins], w2[kBins];
  // written by every CTA of the cluster
  uint64_t seg_w[kMaxCl * kWarps];
  uint32_t seg_n[kMaxCl * kWarps];
  uint32_t top[kMaxCl], bad[kMaxCl], lo[kMaxCl], hi[kMaxCl];
  uint64_t part_w[kMaxCl];
  uint32_t part_n[kMaxCl];
  uint64_t found_w;
  uint32_t found_n, found_bin, found_count;
  // this CTA's own
  uint64_t warp_w[kWarps];
  uint32_t warp_n[kWarps], warp_m[kWarps];
  float ch, cl, floor;
  int32_t k;
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_map_shared(addr, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map_shared(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(const void* p, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_map_shared(smem_u32(p), rank)), "l"(v) : "memory");
}

// Bits whose order as unsigned integers is the numbers'; zeros of either sign alike.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

template <int KIND>
__device__ __forceinline__ float element(const unsigned char* s, int i) {
  if constexpr (KIND == 2) return reinterpret_cast<const float*>(s)[i];
  if constexpr (KIND == 1) return __half2float(reinterpret_cast<const __half*>(s)[i]);
  return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(s)[i] << 16);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  return v;
}

template <int KIND>
struct Row {
  Shared& sm;
  const unsigned char* x;  // the slice
  int count, first;        // its elements, and the row's index of the first
  int cl, rank, sh;
  float top, ch, lo;       // the row's maximum; log2(e) / T in two parts
  int warp, lane;

  __device__ __forceinline__ float at(int i) const { return element<KIND>(x, i); }
  // this warp's part of the slice
  __device__ __forceinline__ int seg_len() const { return ((count + kWarps - 1) / kWarps + 31) & ~31; }

  // y of an element, without its low part: never smaller for a smaller x
  __device__ __forceinline__ float bits_below(float v) const { return __fmul_rn(__fsub_rn(top, v), ch); }

  __device__ __forceinline__ uint64_t weight(float v) const {
    const float d = __fsub_rn(top, v), p = __fmul_rn(d, ch);
    if (!(p < kRange)) return 0;
    // what the difference's rounding left out (Knuth's two-sum), and the product's
    const float t = __fsub_rn(d, top), dl = __fsub_rn(__fsub_rn(top, __fsub_rn(d, t)), __fadd_rn(v, t));
    float e = __fmaf_rn(d, ch, -p);
    e = __fmaf_rn(d, lo, e);
    e = __fmaf_rn(dl, ch, e);
    const int k = __float2int_rn(p * 256.0f);
    const float r = __fadd_rn(__fmaf_rn(__int2float_rn(k), -1.0f / 256.0f, p), e);
    const float a = r * -0.693147180559945f;
    const float g = a * fmaf(a, fmaf(a, fmaf(a, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), 1.0f);
    const int j = k & 255, i = k >> 8;
    uint64_t w = sm.table[j] + (int64_t)__float2int_rn(g * sm.tablef[j]);
    w <<= sh - 40;
    return (w + (((uint64_t)1 << i) >> 1)) >> i;
  }

  // --- exchanges: one value of this CTA to all, then a barrier of the cluster
  template <class F>
  __device__ __forceinline__ void to_all(F store) const {
    if ((int)threadIdx.x < cl) store(threadIdx.x);
  }
  __device__ __forceinline__ uint32_t block_max(uint32_t v) const {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) sm.warp_m[warp] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < kWarps ? sm.warp_m[lane] : 0u);
  }

  __device__ __forceinline__ void clear_bins() const {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sm.n[i] = sm.w0[i] = sm.w1[i] = sm.w2[i] = 0;
    __syncthreads();
  }
  __device__ __forceinline__ void into_bin(int b, float v, bool weigh) const {
    atomicAdd(&sm.n[b], 1u);
    if (weigh) {
      const uint64_t w = weight(v);
      atomicAdd(&sm.w0[b], (uint32_t)w & 0xffffu);
      atomicAdd(&sm.w1[b], (uint32_t)(w >> 16) & 0xffffu);
      atomicAdd(&sm.w2[b], (uint32_t)(w >> 32));
    }
  }

  // The bin where the running count (or weight) over all CTAs' bins reaches what
  // is left of the target: its number and count; n and w get what lies before
  // it.  False if the bins hold less (then the same in every CTA).
  __device__ __forceinline__ bool find_bin(bool by_weight, uint64_t target, uint32_t& n, uint64_t& w, int& bin,
                                           uint32_t& in_bin) const {
    cluster_sync_all();  // every CTA's bins are counted
    const int per = kBins / cl, each = max(1, per / kThreads), mine = threadIdx.x * each;
    uint32_t bn[kBins / kThreads], sn = 0;
    uint64_t bw[kBins / kThreads], sw = 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      bn[i] = 0, bw[i] = 0;
      if (i < each && mine + i < per) {
        const int b = rank * per + mine + i;
        for (int r = 0; r < cl; ++r) {
          bn[i] += ld_cluster_u32(smem_u32(&sm.n[b]), r);
          bw[i] += (uint64_t)ld_cluster_u32(smem_u32(&sm.w0[b]), r) + ((uint64_t)ld_cluster_u32(smem_u32(&sm.w1[b]), r) << 16) +
                   ((uint64_t)ld_cluster_u32(smem_u32(&sm.w2[b]), r) << 32);
        }
      }
      sn += bn[i], sw += bw[i];
    }
    // running sums over the threads
    uint32_t cn = sn;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, cn, d);
      if (lane >= d) cn += y;
    }
    uint64_t cw = warp_scan(sw, lane);
    if (lane == 31) sm.warp_n[warp] = cn, sm.warp_w[warp] = cw;
    __syncthreads();
    uint32_t all_n = 0;
    uint64_t all_w = 0;
    for (int i = 0; i < kWarps; ++i) {
      if (i == warp) cn += all_n, cw += all_w;
      all_n += sm.warp_n[i], all_w += sm.warp_w[i];
    }
    to_all([&](int r) {
      st_cluster_u32(&sm.part_n[rank], r, all_n);
      st_cluster_u64(&sm.part_w[rank], r, all_w);
    });
    cluster_sync_all();
    uint64_t sum_n = n, sum_w = w;
    for (int r = 0; r < cl; ++r) {
      if (r == rank) cn += (uint32_t)sum_n, cw += sum_w;
      sum_n += sm.part_n[r], sum_w += sm.part_w[r];
    }
    if ((by_weight ? sum_w : sum_n) < target) return false;
    cn -= sn, cw -= sw;  // before this thread's
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      const uint64_t from = by_weight ? cw : cn, to = by_weight ? cw + bw[i] : cn + bn[i];
      if (from < target && to >= target)
        for (int r = 0; r < cl; ++r) {
          st_cluster_u32(&sm.found_bin, r, (uint32_t)(rank * per + mine + i));
          st_cluster_u32(&sm.found_count, r, bn[i]);
          st_cluster_u32(&sm.found_n, r, cn);
          st_cluster_u64(&sm.found_w, r, cw);
        }
      cn += bn[i], cw += bw[i];
    }
    cluster_sync_all();
    bin = (int)sm.found_bin, in_bin = sm.found_count;
    n = sm.found_n, w = sm.found_w;
    return true;
  }

  // Largest and smallest key of the elements that `in` holds for.
  template <class F>
  __device__ __forceinline__ void range_of(F in, uint32_t& kmin, uint32_t& kmax) const {
    uint32_t hi = 0, lo_inv = 0;
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const float v = at(i);
      const uint32_t k = key_of(v);
      if (in(v, k)) hi = max(hi, k), lo_inv = max(lo_inv, ~k);
    }
    hi = block_max(hi);
    lo_inv = block_max(lo_inv);
    to_all([&](int r) {
      st_cluster_u32(&sm.hi[rank], r, hi);
      st_cluster_u32(&sm.lo[rank], r, lo_inv);
    });
    cluster_sync_all();
    hi = lo_inv = 0;
    for (int r = 0; r < cl; ++r) hi = max(hi, sm.hi[r]), lo_inv = max(lo_inv, sm.lo[r]);
    kmax = hi, kmin = ~lo_inv;
  }

  // The shortest prefix that holds `target` elements (of weight above 0), or the
  // weight `target`: all above the value, and its first `ties`.  sum: the
  // prefix's weight, if `weigh`.  False if there is less.
  __device__ __forceinline__ bool prefix(bool by_weight, bool weigh, uint64_t target, float& value, uint32_t& ties,
                                         uint64_t& sum) const {
    uint32_t n = 0, in_bin;
    uint64_t w = 0;
    int bin;
    clear_bins();
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const float v = at(i), y = bits_below(v);
      if (y < kRange) into_bin((int)(y * kBinsPerBit), v, weigh);
    }
    if (!find_bin(by_weight, target, n, w, bin, in_bin)) return false;
    uint32_t kmin, kmax;
    range_of([&](float v, uint32_t) { const float y = bits_below(v); return y < kRange && (int)(y * kBinsPerBit) == bin; },
             kmin, kmax);
    while (kmin != kmax) {
      const int bits = 32 - __clz(kmax - kmin), shift = max(0, bits - 11);
      clear_bins();
      for (int i = threadIdx.x; i < count; i += kThreads) {
        const float v = at(i);
        const uint32_t k = key_of(v);
        if (k >= kmin && k <= kmax) into_bin((int)((kmax - k) >> shift), v, weigh);
      }
      find_bin(by_weight, target, n, w, bin, in_bin);  // (there is one: the bin before held it)
      const uint32_t hi = kmax - ((uint32_t)bin << shift);
      if (shift == 0) {
        kmin = kmax = hi;
      } else {
        const uint32_t width = (1u << shift) - 1, low = hi - kmin > width ? hi - width : kmin;
        range_of([&](float, uint32_t k) { return k >= low && k <= hi; }, kmin, kmax);
      }
    }
    value = of_key(kmax);
    const uint64_t each = weigh ? weight(value) : 0;
    ties = (uint32_t)(by_weight ? (target - w + each - 1) / each : target - n);
    sum = w + ties * each;
    return true;
  }
};

template <int KIND>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p, int cl, int slice, int sh) {
  constexpr int E = KIND == 2 ? 4 : 2;
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared& sm = *reinterpret_cast<Shared*>(dyn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x / (unsigned)cl;
  const int rank = (int)(blockIdx.x % (unsigned)cl), first = min(p.N, rank * slice), count = min(p.N - first, slice);

  // --- the slice, at its address's place in a 16-byte unit
  const unsigned char* src = static_cast<const unsigned char*>(p.x) + (r * p.ld_x + first) * E;
  const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15), end = off + count * E;
  unsigned char* data = dyn + (sizeof(Shared) + 15) / 16 * 16;
  float top = -INFINITY;
  bool bad = false;
  auto look = [&](float v) { top = fmaxf(top, v), bad |= !(v < INFINITY); };
  constexpr int U = 8;
  for (int u0 = threadIdx.x; 16 * u0 < end; u0 += U * kThreads) {
    uint4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = 16 * (u0 + i * kThreads);
      if (at >= off && at + 16 <= end) v[i] = __ldcs(reinterpret_cast<const uint4*>(src - off + at));
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = 16 * (u0 + i * kThreads);
      if (at >= off && at + 16 <= end) {
        *reinterpret_cast<uint4*>(data + at) = v[i];
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (KIND == 2) {
            look(__uint_as_float(w[j]));
          } else if constexpr (KIND == 1) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            look(f.x), look(f.y);
          } else {
            look(__uint_as_float(w[j] << 16)), look(__uint_as_float(w[j] & 0xffff0000u));
          }
        }
      } else {
        for (int b = max(at, off); b < min(at + 16, end); b += E) {  // the ends of a row off 16 bytes
          if constexpr (E == 4)
            *reinterpret_cast<uint32_t*>(data + b) = *reinterpret_cast<const uint32_t*>(src - off + b);
          else
            *reinterpret_cast<uint16_t*>(data + b) = *reinterpret_cast<const uint16_t*>(src - off + b);
          look(element<KIND>(data + b, 0));
        }
      }
    }
  }
  // --- the row's settings, once a CTA
  if (threadIdx.x < 256) {
    const uint64_t t = kPowers.v[threadIdx.x];
    sm.table[threadIdx.x] = t;
    sm.tablef[threadIdx.x] = (float)t;
  }
  Row<KIND> row{sm, data + off, count, first, cl, rank, sh, 0.0f, 0.0f, 0.0f, warp, lane};
  {
    const uint32_t k = row.block_max(key_of(top)), b = row.block_max(bad ? 1u : 0u);
    row.to_all([&](int to) {
      st_cluster_u32(&sm.top[rank], to, k);
      st_cluster_u32(&sm.bad[rank], to, b);
    });
  }
  cluster_sync_all();
  uint32_t key = 0, spoiled = 0;
  for (int i = 0; i < cl; ++i) key = max(key, sm.top[i]), spoiled |= sm.bad[i];
  top = of_key(key);
  const float u = __ldg(p.u + r), t_in = p.temperature ? __ldg(p.temperature + r) : 1.0f;
  const float top_p = p.top_p ? __ldg(p.top_p + r) : 1.0f, min_p = p.min_p ? __ldg(p.min_p + r) : 0.0f;
  int top_k = p.top_k ? __ldg(p.top_k + r) : 0;
  const bool settings = u >= 0.0f && u < 1.0f && t_in >= 0.0f && t_in <= 1048576.0f && top_p == top_p && min_p == min_p;
  if (!settings || spoiled || top == -INFINITY) {  // the same in every CTA of the cluster
    if (rank == 0 && threadIdx.x == 0) {
      if (!settings) record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSiteSample));
      if (p.tok64)
        static_cast<long long*>(p.tokens)[r] = -1;
      else
        static_cast<int*>(p.tokens)[r] = -1;
    }
    return;
  }
  // Temperatures below 2^-20 take the most likely token: the first of the largest.
  const bool greedy = t_in < 9.5367431640625e-7f || top_k == 1 || top_p <= 0.0f;
  if (threadIdx.x == 0) {
    const double T = greedy ? 1.0 : (double)t_in, c = 1.4426950408889634074 / T;
    sm.ch = (float)c;
    sm.cl = (float)(c - (double)sm.ch);
    float f = -INFINITY;  // the smallest logit that min_p keeps
    if (min_p > 0.0f) {
      const double d = min_p >= 1.0f ? (double)top : (double)top + T * log((double)min_p);
      f = __double2float_ru(d);
    }
    sm.floor = f;
  }
  __syncthreads();
  row.top = top, row.ch = sm.ch, row.lo = sm.cl;
  float cut = sm.floor;
  uint32_t ties = 0xffffffffu;
  if (greedy) {
    cut = top, ties = 1;
  } else {
    const bool by_k = top_k > 0 && top_k < p.N, by_p = top_p < 1.0f;
    float v;
    uint32_t n;
    uint64_t sum = 0;
    bool some = false;
    if (by_k) {
      some = row.prefix(false, by_p, (uint64_t)top_k, v, n, sum);
      if (some && v >= cut) {
        ties = v > cut || n < ties ? n : ties;
        cut = v;
      }
    }
    if (by_p) {
      if (!some) {  // all of the row
        uint64_t s = 0;
        for (int i = threadIdx.x; i < count; i += kThreads) s += row.weight(row.at(i));
        s = warp_sum(s);
        if (lane == 0) sm.warp_w[warp] = s;
        __syncthreads();
        s = 0;
        for (int i = 0; i < kWarps; ++i) s += sm.warp_w[i];
        row.to_all([&](int to) { st_cluster_u64(&sm.part_w[rank], to, s); });
        cluster_sync_all();
        for (int i = 0; i < cl; ++i) sum += sm.part_w[i];
        cluster_sync_all();  // read by all before it is written again
      }
      const uint64_t want = min(sum, max((uint64_t)1, (uint64_t)ceil((double)top_p * (double)sum)));
      if (row.prefix(true, true, want, v, n, sum) && v >= cut) {
        ties = v > cut || n < ties ? n : ties;
        cut = v;
      }
    }
  }

  // --- the draw: sums of the kept elements by segments, in index order
  const int len = row.seg_len();
  auto sum_of = [&](int from, int to, uint64_t& w, uint32_t& n) {  // weight above the cut, elements at it
    w = 0, n = 0;
    for (int i = from + lane; i < to; i += 32) {
      const float v = row.at(i);
      if (v > cut)
        w += row.weight(v);
      else if (v == cut)
        ++n;
    }
    w = warp_sum(w);
    n = __reduce_add_sync(0xffffffffu, n);
  };
  {
    const int from = min(count, warp * len), to = min(count, from + len);
    uint64_t w;
    uint32_t n;
    sum_of(from, to, w, n);
    if (lane < cl) {
      st_cluster_u64(&sm.seg_w[rank * kWarps + warp], lane, w);
      st_cluster_u32(&sm.seg_n[rank * kWarps + warp], lane, n);
    }
  }
  cluster_sync_all();
  const uint64_t each = cut > -INFINITY ? row.weight(cut) : 0;
  uint64_t all = 0;
  uint32_t seen = 0;  // elements at the cut so far
  for (int s = 0; s < cl * kWarps; ++s) {
    const uint32_t n = min(sm.seg_n[s], ties - seen);
    all += sm.seg_w[s] + n * each;
    seen += n;
  }
  const uint64_t want = min(all - 1, (uint64_t)((double)u * (double)all));
  uint64_t run = 0;
  int seg = 0;
  seen = 0;
  for (;; ++seg) {
    const uint32_t n = min(sm.seg_n[seg], ties - seen);
    const uint64_t w = sm.seg_w[seg] + n * each;
    if (run + w > want || seg + 1 == cl * kWarps) break;
    run += w, seen += n;
  }
  if (seg / kWarps != rank) return;  // no CTA reads another's memory from here on
  // the segment's parts, a warp each
  const int from = min(count, (seg % kWarps) * len), to = min(count, from + len);
  const int part = ((to - from + kWarps - 1) / kWarps + 31) & ~31;
  const int a = min(to, from + warp * part), b = min(to, a + part);
  uint64_t w;
  uint32_t n;
  sum_of(a, b, w, n);
  __syncthreads();
  if (lane == 0) sm.warp_w[warp] = w, sm.warp_n[warp] = n;
  __syncthreads();
  for (int i = 0; i < warp; ++i) {
    const uint32_t k = min(sm.warp_n[i], ties - seen);
    run += sm.warp_w[i] + k * each, seen += k;
  }
  if (run > want || run + w + min(n, ties - seen) * each <= want) return;  // another warp's
  for (int i = a; i < b; i += 32) {
    const float v = i + lane < b ? row.at(i + lane) : -INFINITY;
    const bool tie = i + lane < b && v == cut;
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    uint64_t m = 0;
    if (v > cut) m = row.weight(v);
    if (tie && (uint32_t)__popc(tied & ((1u << lane) - 1)) < ties - seen) m = each;
    const uint64_t upto = run + warp_scan(m, lane);
    const uint32_t over = __ballot_sync(0xffffffffu, upto > want);
    if (over) {
      if (lane == __ffs(over) - 1) {
        const int64_t token = first + i + lane;
        if (p.tok64)
          static_cast<long long*>(p.tokens)[r] = token;
        else
          static_cast<int*>(p.tokens)[r] = (int)token;
      }
      return;
    }
    run = __shfl_sync(0xffffffffu, upto, 31);
    seen += min((uint32_t)__popc(tied), ties - seen);
  }
}

template <int KIND>
cudaError_t launch(const SampleParams& p, cudaStream_t stream) {
  constexpr int E = KIND == 2 ? 4 : 2;
  constexpr int kHead = (sizeof(Shared) + 15) / 16 * 16 + 16;
  constexpr int kMost = kHead + (int)(kMaxVocab / kMaxCl) * E;
  static_assert(kMost <= 232448, "shared memory of a CTA");
  static_assert(kMaxVocab / kMaxCl <= 65536, "three 16-bit sums of a slice fit 32 bits");
  // Slices of at most 16384 elements while a cluster of eight has them.
  int cl = 1;
  while (cl < kMaxCl && p.N > 16384 * cl) cl *= 2;
  const int slice = ((p.N + cl - 1) / cl + 7) / 8 * 8;  // (16 bytes keep their place)
  int bits = 0;
  while ((1 << bits) < p.N) ++bits;
  const void* fn = reinterpret_cast<const void*>(&sample_kernel<KIND>);
  cudaError_t e = set_smem_once(fn, kMost, 130 + KIND);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.R * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kHead + slice * E;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<KIND>, p, cl, slice, std::min(46, 62 - bits));
}

}  // namespace

bi_status launch_sample(SampleParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  p.status_word = dev.status_word;
  const cudaError_t e = p.x_kind == 2 ? launch<2>(p, stream) : p.x_kind == 1 ? launch<1>(p, stream) : launch<0>(p, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    *why = std::string("sampling launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
