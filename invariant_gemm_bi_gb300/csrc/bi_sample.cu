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
//   e^(z - max) = 2^-y, y = Y - x c, c = log2(e) / T in two fp32, Y = max c cut to
//   a multiple of 1/256 (every weight of a row then has the same factor 2^(Y - max c)
//   too much).  The product with its exact error; y = k / 256 - f, f below 2^-8, from
//   differences that fp32 has exactly; the table's 2^(-(k mod 256) / 256) to 2^-41,
//   times a polynomial of f ln 2, whose fp32 roundings are 2^-24 of it; shifted by k /
//   256.  Rows whose largest |max c| is 8000 or more take the difference first.
// The unit is 2^-40 of the largest weight.
//
// Work.  A row is a cluster's, a slice of it a CTA's, held in shared memory from
// the only read of it on.  Prefixes are found by counting, once for both limits:
//   fp32 and fp16  2048 bins of y, each with the number and the weight of its
//     elements (the weight as three sums of 16 bits in 32).  The elements of the
//     bin where a limit is reached, a few hundred as a rule, are gathered by every
//     CTA and sorted; more than 512 are binned again by their bits until one value
//     or few elements are left.  Where all that is kept is among 512 elements, the
//     first CTA does the rest from a list of those.
//   bf16  a bin for each number of 2^-8 .. 2^6 of either sign: counts alone, whose
//     weights come from a table of the row's (3584 weights in place of a row's
//     128256), and a bin that is reached is a value already.  Numbers nearer to
//     zero share a bin and are weighed one by one; rows with others go the way of
//     fp32.
// The CTAs add up a share of the bins each.  The draw sums the kept elements by
// warps' segments in index order, then looks into one.
//
// What bounds it: 256 bf16 rows of 128256 with top-p 0.95 take 108 us (9.7 at the
// copy rate; 20 MB of 66 in flight at a time, three and a half rounds of CTAs, two an
// SM).  Of a round's 50000 cycles the reads take 10000, counting 15000 (atomics on
// shared memory, 3.5 lanes to a bank), the rest are the row's own chain: maximum,
// table, three exchanges of the cluster, the draw.  8 fp32 rows take
// 40 us with top-p alone, 21 without limits: the chain, and counting in four sums.
// All kernels spill at 64 registers, two CTAs of 512 threads or one of 1024 an SM: what a
// thread knows of the bins, kept over both searches, most in bf16 (730 bytes stored).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
#include "bi_quant.h"

namespace bi {
namespace {

constexpr int kMaxWarps = 32;
constexpr int kBins = 2048;
constexpr int kMaxCl = 8;
constexpr float kRange = 62.0f;               // y from here on: weight 0
constexpr float kMagic = 12582912.0f;         // 1.5 * 2^23: added, it leaves an integer in the low bits
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

constexpr int kList = 512;  // elements that are sorted

// Shared memory that other CTAs of the cluster write or read, and the barrier of the
// cluster between a word's last use and its next one.  ("Searches" are calls of
// find_bin; a scan, scan_bins, has a barrier before it reads and one after.)
//   top              written once, behind the start-up barrier.
//   lo, hi           range_of: read behind its barrier; written by the next range_of
//                    of a limit behind the scan's barriers between them, by the other
//                    limit's behind its search's.
//   part_n, part_w   scan_bins: read behind its second barrier; written again behind
//                    the next scan's first.
//   found_*          find_bin: read behind its barrier.  The same limit's next search
//                    comes behind range_of's barrier (within_bin's loop) or a scan's
//                    (bf16 rows that go on without their table).  Between a search by
//                    count and one by weight there need not be any: two sets.
//   listed           reset by the first CTA before a search's barrier, added to behind
//                    it; the list before was closed by gather's barrier.
//   list             gather: read behind its barrier by its own CTA; written again
//                    behind the next search's, which every CTA reaches when it has read.
//   sum_w, sum_n     written once, in the draw; read behind its barrier.
//   n, w0-w2, n16, middle_w  read by scans, between their two barriers; cleared, counted
//                    again or used as `mine` behind the second.
// Behind the last barrier of a row's path no CTA reads or writes another's memory, so
// each leaves when it is done.

// bf16: numbers of exponents -8 .. 5, in the order of their values: the positive
// ones, what lies between, the negative ones.
constexpr int kBase16 = (127 - 8) << 7, kSpan16 = 14 << 7, kMiddle16 = kSpan16, kBins16 = 2 * kSpan16 + 1;
__device__ __forceinline__ int bin16(uint32_t bits) {  // -1: outside
  const int t = (int)(bits & 0x7fffu) - kBase16;
  if (t < 0) return kMiddle16;
  if (t >= kSpan16) return -1;
  return bits & 0x8000u ? kMiddle16 + 1 + t : kSpan16 - 1 - t;
}
__device__ __forceinline__ float value16(int bin) {  // (not of the middle)
  const uint32_t bits = bin < kMiddle16 ? kBase16 + kSpan16 - 1 - bin : (0x8000u | (kBase16 + bin - kMiddle16 - 1));
  return __uint_as_float(bits << 16);
}

template <int KIND>
struct Shared {
  uint64_t table[256];  // 2^40 2^(-j / 256)
  // written by every CTA of the cluster
  uint32_t top[kMaxCl], lo[kMaxCl], hi[kMaxCl];
  uint64_t part_w[kMaxCl], sum_w[kMaxCl];
  uint32_t part_n[kMaxCl], sum_n[kMaxCl];
  uint64_t found_w[2];  // [0]: where a count is reached, [1]: where a weight is
  uint32_t found_n[2], found_bin[2], found_count[2];
  uint32_t listed;  // the first CTA's counts for all
  uint32_t mine_n, mine_at;
  uint64_t list[kList];
  // this CTA's own
  uint64_t warp_w[kMaxWarps], middle_w, cut_w;
  uint32_t warp_n[kMaxWarps], warp_m[kMaxWarps], cut_key, cut_n;
  float ch, cl, floor;
  // bins: number, and weight in three parts; or for bf16 the number, and the table of weights
  union {
    struct {
      uint32_t n[kBins], w0[kBins], w1[kBins], w2[kBins];
    };
    uint64_t mine[kList];
    struct {
      uint64_t weight16[KIND == 0 ? kBins16 : 1];
      uint32_t n16[KIND == 0 ? kBins16 / 2 + 1 : 1];  // two bins a word: a slice has fewer than 2^16 elements
    };
  };
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_map_shared(addr, rank)));
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

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  return v;
}

// T threads.  KIND 0: bf16, 1: fp16, 2: fp32.
template <int KIND, int T>
struct Row {
  static constexpr int kWarps = T / 32;
  static constexpr int kEach = ((KIND == 0 ? kBins16 : kBins) + T - 1) / T;  // bins of a thread, at most

  Shared<KIND>& sm;
  const unsigned char* x;  // the slice
  int count, first;        // its elements, and the row's index of the first
  int cl, rank;
  float top, ch, lo;       // the row's maximum; log2(e) / T in two parts
  float start;             // 256 Y + 1.5 * 2^23, or 0 for rows that take the difference first
  float least;             // x c from here on: weight 0
  int warp, lane;

  __device__ __forceinline__ float at(int i) const { return element<KIND>(x, i); }
  // this warp's part of the slice
  __device__ __forceinline__ int seg_len() const { return ((count + kWarps - 1) / kWarps + 31) & ~31; }

  // y of an element, without its low part: never smaller for a smaller x
  __device__ __forceinline__ float bits_below(float v) const { return __fmul_rn(__fsub_rn(top, v), ch); }

  // Settings that a row's weights go by, from its maximum and log2(e) / T.
  __device__ __forceinline__ void set(float max, float hi, float low) {
    top = max, ch = hi, lo = low;
    const float y = __fmul_rn(top, ch);
    const float m = __fmaf_rn(y, 256.0f, kMagic);
    start = fabsf(y) < 8000.0f ? m : 0.0f;
    least = __fsub_rn(y, kRange);
  }
  __device__ __forceinline__ uint64_t weight(float v) const {
    float f, m;
    if (start != 0.0f) {
      const float p = __fmul_rn(v, ch);
      if (!(p > least)) return 0;
      float e = __fmaf_rn(v, ch, -p);
      e = __fmaf_rn(v, lo, e);
      m = __fmaf_rn(p, -256.0f, start);  // kMagic + k + what p is of it: the low bits are k's
      f = __fadd_rn(__fmaf_rn(__fsub_rn(m, start), 1.0f / 256.0f, p), e);
    } else {
      const float d = __fsub_rn(top, v), p = __fmul_rn(d, ch);
      if (!(p < kRange)) return 0;
      // what the difference's rounding left out (Knuth's two-sum), and the product's
      const float t = __fsub_rn(d, top), dl = __fsub_rn(__fsub_rn(top, __fsub_rn(d, t)), __fadd_rn(v, t));
      float e = __fmaf_rn(d, ch, -p);
      e = __fmaf_rn(d, lo, e);
      e = __fmaf_rn(dl, ch, e);
      m = __fmaf_rn(p, 256.0f, kMagic);
      f = -__fadd_rn(__fmaf_rn(__fsub_rn(m, kMagic), -1.0f / 256.0f, p), e);
    }
    const int k = __float_as_int(m) & 0x3fffff;
    const float a = f * 0.693147180559945f;
    const float g = a * fmaf(a, fmaf(a, 1.0f / 6.0f, 0.5f), 1.0f);
    const int j = k & 255, i = k >> 8;
    const uint64_t t = sm.table[j];
    // (g times it: its upper 32 of 41 bits do, from a register and not a second table)
    const uint64_t w = t + (int64_t)__float2int_rn(g * (__uint2float_rn((uint32_t)(t >> 9)) * 512.0f));
    return (w + (((uint64_t)1 << i) >> 1)) >> i;
  }
  // The same from the row's table where there is one.
  __device__ __forceinline__ uint64_t weight_at(int i, float v, bool tabled) const {
    if constexpr (KIND == 0) {
      if (tabled) {
        const int b = bin16(__float_as_uint(v) >> 16);
        if (b < 0) return 0;
        if (b != kMiddle16) return sm.weight16[b];
      }
    }
    return weight(v);
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

  // --- bins of y or of bits
  __device__ __forceinline__ void clear_bins() const {
    for (int i = threadIdx.x; i < kBins; i += T) sm.n[i] = sm.w0[i] = sm.w1[i] = sm.w2[i] = 0;
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

  // What a thread knows of the cluster's bins: its own ones', and before them.
  struct Scan {
    uint32_t bn[kEach], cn, all_n;
    uint64_t bw[kEach], cw, all_w;
    int base, each;  // its first bin, and how many
  };
  // Adds every CTA's bins up, a share a CTA, starting from (n, w).
  // (Shares, and a thread's bins where it has several, are of whole words of n16.)
  template <class F>
  __device__ __forceinline__ void scan_bins(int bins, uint32_t n, uint64_t w, Scan& s, F fetch) const {
    cluster_sync_all();  // every CTA's bins are counted
    const int per = ((bins + cl - 1) / cl + 1) & ~1, end = min(bins, (rank + 1) * per);
    s.each = (per + T - 1) / T;
    if (s.each > 1) s.each += s.each & 1;
    s.base = rank * per + (int)threadIdx.x * s.each;
    uint32_t sn = 0;
    uint64_t sw = 0;
    static_assert(kEach % 2 == 0, "bins of a thread");
#pragma unroll
    for (int i = 0; i < kEach; i += 2) {
      s.bn[i] = s.bn[i + 1] = 0, s.bw[i] = s.bw[i + 1] = 0;
      if (i < s.each && s.base + i < end)
        fetch(s.base + i, s.each > 1 && s.base + i + 1 < end, s.bn[i], s.bw[i], s.bn[i + 1], s.bw[i + 1]);
      sn += s.bn[i] + s.bn[i + 1], sw += s.bw[i] + s.bw[i + 1];
    }
    uint32_t cn = warp_scan(sn, lane);
    uint64_t cw = warp_scan(sw, lane);
    if (lane == 31) sm.warp_n[warp] = cn, sm.warp_w[warp] = cw;
    __syncthreads();
    uint32_t all_n = lane < kWarps ? sm.warp_n[lane] : 0;
    uint64_t all_w = lane < kWarps ? sm.warp_w[lane] : 0;
    all_n = warp_scan(all_n, lane), all_w = warp_scan(all_w, lane);
    const uint32_t before_n = __shfl_sync(0xffffffffu, all_n, max(warp - 1, 0));
    const uint64_t before_w = __shfl_sync(0xffffffffu, all_w, max(warp - 1, 0));
    if (warp > 0) cn += before_n, cw += before_w;
    all_n = __shfl_sync(0xffffffffu, all_n, 31), all_w = __shfl_sync(0xffffffffu, all_w, 31);
    to_all([&](int r) {
      st_cluster_u32(&sm.part_n[rank], r, all_n);
      st_cluster_u64(&sm.part_w[rank], r, all_w);
    });
    cluster_sync_all();
    for (int r = 0; r < cl; ++r) {
      if (r == rank) s.cn = cn - sn + n, s.cw = cw - sw + w;
      n += sm.part_n[r], w += sm.part_w[r];
    }
    s.all_n = n, s.all_w = w;
  }
  __device__ __forceinline__ void scan_bins(uint32_t n, uint64_t w, bool weigh, Scan& s) const {
    auto fetch = [&](int b, uint32_t& bn, uint64_t& bw) {
#pragma unroll
      for (int r0 = 0; r0 < kMaxCl; r0 += 4) {
        if (r0 >= cl) break;
        uint32_t v[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // requested together
          const uint32_t from = (uint32_t)min(r0 + r, cl - 1);
          v[r][0] = ld_cluster_u32(smem_u32(&sm.n[b]), from);
          if (weigh) {
            v[r][1] = ld_cluster_u32(smem_u32(&sm.w0[b]), from);
            v[r][2] = ld_cluster_u32(smem_u32(&sm.w1[b]), from);
            v[r][3] = ld_cluster_u32(smem_u32(&sm.w2[b]), from);
          }
        }
        // (A CTA that there is not adds zeros.  With an exit from the loop in their place the
        // bf16 kernels came out of the compiler without the lower words of some of the sums.)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint64_t there = r0 + r < cl ? 1 : 0;
          bn += (uint32_t)there * v[r][0];
          if (weigh) bw += there * ((uint64_t)v[r][1] + ((uint64_t)v[r][2] << 16) + ((uint64_t)v[r][3] << 32));
        }
      }
    };
    scan_bins(kBins, n, w, s, [&](int b, bool two, uint32_t& bn, uint64_t& bw, uint32_t& bn1, uint64_t& bw1) {
      fetch(b, bn, bw);
      if (two) fetch(b + 1, bn1, bw1);
    });
  }
  // The bin where the running count, or weight, reaches the target: its number and
  // count; n and w get what lies before it.  False if all of them hold less (the
  // same in every CTA).  A search by weight may follow one by count at once, with
  // warps that have yet to read the first one's answer: each has words of its own.
  __device__ __forceinline__ bool find_bin(const Scan& s, bool by_weight, uint64_t target, uint32_t& n, uint64_t& w, int& bin,
                                           uint32_t& in_bin) const {
    if ((by_weight ? s.all_w : (uint64_t)s.all_n) < target) return false;
    uint32_t cn = s.cn, hit_n = 0, hit_count = 0;
    uint64_t cw = s.cw, hit_w = 0;
    int hit = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const uint64_t from = by_weight ? cw : cn, to = by_weight ? cw + s.bw[i] : cn + s.bn[i];
      if (i < s.each && from < target && to >= target) hit = s.base + i, hit_n = cn, hit_count = s.bn[i], hit_w = cw;
      cn += s.bn[i], cw += s.bw[i];
    }
    const uint32_t who = __ballot_sync(0xffffffffu, hit >= 0);
    if (who) {  // its warp tells the cluster, a CTA a lane
      const int from = __ffs(who) - 1;
      hit = __shfl_sync(0xffffffffu, hit, from);
      hit_n = __shfl_sync(0xffffffffu, hit_n, from);
      hit_count = __shfl_sync(0xffffffffu, hit_count, from);
      hit_w = __shfl_sync(0xffffffffu, hit_w, from);
      if (lane < cl) {
        st_cluster_u32(&sm.found_bin[by_weight], lane, (uint32_t)hit);
        st_cluster_u32(&sm.found_count[by_weight], lane, hit_count);
        st_cluster_u32(&sm.found_n[by_weight], lane, hit_n);
        st_cluster_u64(&sm.found_w[by_weight], lane, hit_w);
      }
    }
    if (threadIdx.x == 0) sm.listed = sm.mine_n = 0;
    cluster_sync_all();
    bin = (int)sm.found_bin[by_weight], in_bin = sm.found_count[by_weight];
    n = sm.found_n[by_weight], w = sm.found_w[by_weight];
    return true;
  }

  // Largest and smallest key of the elements that `in` holds for.
  template <class F>
  __device__ __forceinline__ void range_of(F in, uint32_t& kmin, uint32_t& kmax) const {
    uint32_t hi = 0, lo_inv = 0;
    for (int i = threadIdx.x; i < count; i += T) {
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

  // Gathers the elements that `in` holds for, at most kList of them, into the lists of
  // the first `to` CTAs: (key, ~index).  First into a list of the CTA's own, in the
  // place of the bins, which nobody reads any more: a place in the cluster's list is
  // asked for once (by every warp with a hit, 334 elements took 9800 cycles).
  template <class F>
  __device__ __forceinline__ void gather(F in, int to) const {
    constexpr int U = 4;
    for (int i0 = warp * 32; i0 < count; i0 += U * T) {
      float v[U];
      bool hit[U], some = false;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * T + lane;
        v[j] = i < count ? at(i) : 0.0f;
        hit[j] = i < count && in(v[j], key_of(v[j]));
        some |= hit[j];
      }
      if (!__any_sync(0xffffffffu, some)) continue;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t hits = __ballot_sync(0xffffffffu, hit[j]);
        if (!hits) continue;
        uint32_t at0 = 0;
        if (lane == 0) at0 = atomicAdd(&sm.mine_n, (uint32_t)__popc(hits));
        at0 = __shfl_sync(0xffffffffu, at0, 0) + __popc(hits & ((1u << lane) - 1));
        if (hit[j] && at0 < (uint32_t)kList)
          sm.mine[at0] = (uint64_t)key_of(v[j]) << 32 | (0xffffffffu - (uint32_t)(first + i0 + j * T + lane));
      }
    }
    __syncthreads();
    const uint32_t have = min(sm.mine_n, (uint32_t)kList);
    if (threadIdx.x == 0 && have > 0)
      asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                   : "=r"(sm.mine_at)
                   : "r"(cluster_map_shared(smem_u32(&sm.listed), 0)), "r"(have)
                   : "memory");
    __syncthreads();
    for (int r = 0; r < to; ++r)
      for (uint32_t i = threadIdx.x; i < have; i += T)
        if (sm.mine_at + i < (uint32_t)kList) st_cluster_u64(&sm.list[sm.mine_at + i], r, sm.mine[i]);
    cluster_sync_all();
  }
  // Sorts the list (no two alike, none 0), largest first, an element a thread: 32 a
  // warp by exchanges, then each to its place, which is the number of larger ones in
  // every run.  (By exchanges through shared memory alone, 334 elements took 13600
  // cycles.)  A barrier before and after.
  __device__ __forceinline__ void sort_list(uint32_t size) const {
    const int runs = ((int)size + 31) / 32;
    uint64_t x = threadIdx.x < size ? sm.list[threadIdx.x] : 0;
    if (warp < runs) {
#pragma unroll
      for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int j = k / 2; j > 0; j /= 2) {
          const uint64_t y = __shfl_xor_sync(0xffffffffu, x, j);
          const bool larger = ((lane & k) == 0) == ((lane & j) == 0);  // this lane keeps the larger one
          x = (x > y) == larger ? x : y;
        }
      sm.list[threadIdx.x] = x;  // (where this warp has read)
    }
    __syncthreads();
    int place = lane;
    if (warp < runs) {
#pragma unroll 4
      for (int r = 0; r < runs; ++r) {
        const uint64_t* run = sm.list + 32 * r;
        int n = 0;
#pragma unroll
        for (int step = 16; step > 0; step /= 2)
          if (run[n + step - 1] > x) n += step;
        if (run[n] > x) ++n;
        place += r == warp ? 0 : n;
      }
    }
    __syncthreads();
    if (x != 0) sm.list[place] = x;
    __syncthreads();
  }
  // Running sum over the list's elements, a thread each (one barrier).
  __device__ __forceinline__ uint64_t list_scan(uint64_t own) const {
    uint64_t upto = warp_scan(own, lane);
    if (lane == 31) sm.warp_w[warp] = upto;
    __syncthreads();
    for (int k = 0; k < min(warp, kList / 32); ++k) upto += sm.warp_w[k];
    return upto;
  }

  // Where in a bin of at most kList elements, which `in` holds for, the target is
  // reached: every CTA gathers and sorts them, by value and then by index.
  template <class F>
  __device__ __forceinline__ void within_list(F in, uint32_t size, bool by_weight, bool weigh, uint64_t target, uint32_t n,
                                              uint64_t w, float& value, uint32_t& ties, uint64_t& sum) const {
    gather(in, cl);
    sort_list(size);
    const int i = threadIdx.x;
    const bool there = i < (int)size;
    const uint64_t e = there ? sm.list[i] : 0;
    const uint32_t key = (uint32_t)(e >> 32);
    const uint64_t own = there && weigh ? weight(of_key(key)) : 0;
    const uint64_t upto = list_scan(own) + w;
    const uint64_t to = by_weight ? upto : (uint64_t)n + i + 1, from = by_weight ? upto - own : (uint64_t)n + i;
    if (there && from < target && to >= target) {
      int same = i;  // the first element of its value
      while (same > 0 && (uint32_t)(sm.list[same - 1] >> 32) == key) --same;
      sm.cut_key = key, sm.cut_n = i - same + 1, sm.cut_w = upto;
    }
    __syncthreads();
    value = of_key(sm.cut_key), ties = sm.cut_n, sum = sm.cut_w;
  }

  // The whole draw from at most kList elements, those of the bins up to `bin`, one of
  // which holds the last one kept: the first CTA gathers and sorts them and finds both
  // limits there (top-p's of `sum`, or of the first `limit` if that is 0), then sorts
  // them by index.  A row of 128256 fp32 with k = 50 and p = 0.9 takes 27 us this way;
  // with a list for each limit and the draw over the slices it took 50.
  __device__ __forceinline__ int draw_from_list(int bin, uint32_t size, uint32_t limit, bool by_p, float top_p, uint64_t sum,
                                                float u) const {
    gather([&](float v, uint32_t) {
      const float y = bits_below(v);
      return y < kRange && (int)(y * kBinsPerBit) <= bin;
    }, 1);
    if (rank != 0) return -1;
    sort_list(size);
    const int i = threadIdx.x;
    const bool there = i < (int)size;
    const uint64_t e = there ? sm.list[i] : 0;
    const float v = of_key((uint32_t)(e >> 32));
    const uint64_t own = there ? weight(v) : 0, upto = list_scan(own);
    if (i + 1 == (int)min(limit, size)) sm.cut_w = upto;
    __syncthreads();
    if (sum == 0) sum = sm.cut_w;
    const bool kept = there && (uint32_t)i < limit && v >= sm.floor && (!by_p || upto - own < share(top_p, sum));
    // by index from here on, the weight in the low bits
    constexpr int kBits = 41;
    static_assert(kMaxVocab < 1 << (62 - kBits), "index and weight in a word");
    if (there) sm.list[i] = (uint64_t)((1u << (62 - kBits)) - 1 - (0xffffffffu - (uint32_t)e)) << kBits | (kept ? own : 0);
    __syncthreads();
    sort_list(size);
    const uint64_t x = there ? sm.list[i] : 0, w = x & (((uint64_t)1 << kBits) - 1), run = list_scan(w);
    if (i == kList - 1) sm.cut_w = run;
    __syncthreads();
    const uint64_t all = sm.cut_w, want = min(all - 1, (uint64_t)((double)u * (double)all));
    return there && run - w <= want && run > want ? (int)((1u << (62 - kBits)) - 1 - (uint32_t)(x >> kBits)) : -1;
  }
  // What top-p keeps of a sum.
  __device__ __forceinline__ uint64_t share(float top_p, uint64_t sum) const {
    return min(sum, max((uint64_t)1, (uint64_t)ceil((double)top_p * (double)sum)));
  }

  // Where in a bin the target is reached: everything above `value`, and its first
  // `ties`; sum: the weight of that, if `weigh`.
  __device__ __forceinline__ void within_bin(int bin, uint32_t in_bin, bool by_weight, bool weigh, uint64_t target, uint32_t n,
                                             uint64_t w, float& value, uint32_t& ties, uint64_t& sum) const {
    auto in_y = [&](float v, uint32_t) {
      const float y = bits_below(v);
      return y < kRange && (int)(y * kBinsPerBit) == bin;
    };
    if (in_bin <= kList) return within_list(in_y, in_bin, by_weight, weigh, target, n, w, value, ties, sum);
    uint32_t kmin, kmax;
    range_of(in_y, kmin, kmax);
    while (kmin != kmax) {
      const int bits = 32 - __clz(kmax - kmin), shift = max(0, bits - 11);
      clear_bins();
      for (int i = threadIdx.x; i < count; i += T) {
        const float v = at(i);
        const uint32_t k = key_of(v);
        if (k >= kmin && k <= kmax) into_bin((int)((kmax - k) >> shift), v, weigh);
      }
      Scan s;
      scan_bins(n, w, weigh, s);
      find_bin(s, by_weight, target, n, w, bin, in_bin);  // (there is one: the bin before held it)
      const uint32_t hi = kmax - ((uint32_t)bin << shift);
      const uint32_t width = (1u << shift) - 1, low = hi - kmin > width ? hi - width : kmin;
      auto in_keys = [&](float, uint32_t k) { return k >= low && k <= hi; };
      if (shift > 0 && in_bin <= kList) return within_list(in_keys, in_bin, by_weight, weigh, target, n, w, value, ties, sum);
      if (shift == 0)
        kmin = kmax = hi;
      else
        range_of(in_keys, kmin, kmax);
    }
    value = of_key(kmax);
    const uint64_t each = weigh ? weight(value) : 0;
    ties = (uint32_t)(by_weight ? (target - w + each - 1) / each : target - n);
    sum = w + ties * each;
  }
};

template <int KIND, int T>
__global__ void __launch_bounds__(T, 1024 / T) sample_kernel(const SampleParams p, int cl, int slice) {
  constexpr int E = KIND == 2 ? 4 : 2, kWarps = T / 32;
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared<KIND>& sm = *reinterpret_cast<Shared<KIND>*>(dyn);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x / (unsigned)cl;
  const int rank = (int)(blockIdx.x % (unsigned)cl), first = min(p.N, rank * slice), count = min(p.N - first, slice);

  cluster_arrive_relaxed();  // waited for before another CTA's shared memory is written

  // --- the row's settings
  const float u = __ldg(p.u + r), t_in = p.temperature ? __ldg(p.temperature + r) : 1.0f;
  const float top_p = p.top_p ? __ldg(p.top_p + r) : 1.0f, min_p = p.min_p ? __ldg(p.min_p + r) : 0.0f;
  const int top_k = p.top_k ? __ldg(p.top_k + r) : 0;
  const bool settings = u >= 0.0f && u < 1.0f && t_in >= 0.0f && t_in <= 1048576.0f && top_p == top_p && min_p == min_p;
  // Temperatures below 2^-20 take the most likely token: the first of the largest.
  const bool greedy = t_in < 9.5367431640625e-7f || top_k == 1 || top_p <= 0.0f;
  const bool by_k = !greedy && top_k > 0 && top_k < p.N, by_p = !greedy && top_p < 1.0f;

  // --- the slice, at its address's place in a 16-byte unit
  const unsigned char* src = static_cast<const unsigned char*>(p.x) + (r * p.ld_x + first) * E;
  const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15), end = off + count * E;
  unsigned char* data = dyn + (sizeof(Shared<KIND>) + 15) / 16 * 16;
  float top = -INFINITY;
  bool bad = false;
  auto look = [&](float v) { top = fmaxf(top, v), bad |= !(v < INFINITY); };
  constexpr int U = 8;
  for (int u0 = threadIdx.x; 16 * u0 < end; u0 += U * T) {
    uint4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = 16 * (u0 + i * T);
      if (at >= off && at + 16 <= end) v[i] = __ldcs(reinterpret_cast<const uint4*>(src - off + at));
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int at = 16 * (u0 + i * T);
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
  for (int i = threadIdx.x; i < 256; i += T) {
    const uint64_t t = kPowers.v[i];
    sm.table[i] = t;
  }
  if constexpr (KIND == 0) {
    if (by_k || by_p) {
      for (int i = threadIdx.x; i < kBins16 / 2 + 1; i += T) sm.n16[i] = 0;
      if (threadIdx.x == 0) sm.middle_w = 0;
    }
  } else if (by_k || by_p) {
    for (int i = threadIdx.x; i < kBins; i += T) sm.n[i] = sm.w0[i] = sm.w1[i] = sm.w2[i] = 0;
  }
  double below = 0.0;  // how far below the largest logit min_p reaches
  if (threadIdx.x == T - 1) {
    const double temp = greedy ? 1.0 : (double)t_in, c = 1.4426950408889634074 / temp;
    sm.ch = (float)c;
    sm.cl = (float)(c - (double)sm.ch);
    if (min_p > 0.0f && min_p < 1.0f) below = temp * log((double)min_p);
  }
  Row<KIND, T> row{sm, data + off, count, first, cl, rank, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, warp, lane};
  {
    const uint32_t k = row.block_max(bad ? 0xffffffffu : key_of(top));  // above any number's
    cluster_wait();
    row.to_all([&](int to) { st_cluster_u32(&sm.top[rank], to, k); });
  }
  cluster_sync_all();
  uint32_t key = 0;
  for (int i = 0; i < cl; ++i) key = max(key, sm.top[i]);
  top = of_key(key);
  if (!settings || key == 0xffffffffu || top == -INFINITY) {  // the same in every CTA of the cluster
    if (rank == 0 && threadIdx.x == 0) {
      if (!settings) record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSiteSample));
      if (p.tok64)
        static_cast<long long*>(p.tokens)[r] = -1;
      else
        static_cast<int*>(p.tokens)[r] = -1;
    }
    return;
  }
  if (threadIdx.x == T - 1)  // the smallest logit that min_p keeps
    sm.floor = min_p > 0.0f ? __double2float_ru((double)top + below) : -INFINITY;
  row.set(top, sm.ch, sm.cl);

  // --- bf16: the row's weights by value, if its numbers that have any are in the bins
  bool tabled = false;
  if constexpr (KIND == 0) {
    const float far = top - kRange / row.ch;  // (what rounding leaves out there weighs nothing)
    tabled = !greedy && top < 64.0f && far > -64.0f;
    if (tabled) {
      for (int b = threadIdx.x; b < kBins16; b += T) {
        const float v = value16(b);
        sm.weight16[b] = b == kMiddle16 || v > top ? 0 : row.weight(v);
      }
    }
  }
  __syncthreads();

  float cut = sm.floor;
  uint32_t ties = 0xffffffffu;
  auto lower = [&](float v, uint32_t n) {  // what is kept is what both limits keep
    if (v < cut) return;
    ties = v > cut || n < ties ? n : ties;
    cut = v;
  };
  if (greedy) {
    cut = top, ties = 1;
  } else if (by_k || by_p) {
    typename Row<KIND, T>::Scan s;
    float v;
    uint32_t n = 0, m, in_bin;
    uint64_t w = 0, sum = 0;
    int bin;
    bool done = false;
    auto store = [&](int token) {  // of the one thread that has it
      if (token < 0) return;
      if (p.tok64)
        static_cast<long long*>(p.tokens)[r] = token;
      else
        static_cast<int*>(p.tokens)[r] = token;
    };
    if constexpr (KIND == 0) {
      if (tabled) {
        uint64_t mine = 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < count; i += T) {
          const uint32_t bits = reinterpret_cast<const uint16_t*>(row.x)[i];
          const int b = bin16(bits);
          if (b >= 0) atomicAdd(&sm.n16[b >> 1], b & 1 ? 65536u : 1u);  // (others have no weight)
          if (b == kMiddle16) mine += row.weight(__uint_as_float(bits << 16));
        }
        if (__any_sync(0xffffffffu, mine != 0)) {
          mine = warp_sum(mine);
          if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sm.middle_w), (unsigned long long)mine);
        }
        auto weigh = [&](int b, uint32_t n) -> uint64_t {
          if (b != kMiddle16) return n * sm.weight16[b];
          uint64_t w = 0;
          const uint32_t a = smem_u32(&sm.middle_w);
          for (int c = 0; c < cl; ++c) w += (uint64_t)ld_cluster_u32(a, c) | (uint64_t)ld_cluster_u32(a + 4, c) << 32;
          return w;
        };
        row.scan_bins(kBins16, 0, 0, s, [&](int b, bool two, uint32_t& bn, uint64_t& bw, uint32_t& bn1, uint64_t& bw1) {
          uint32_t lo = 0, hi = 0;
#pragma unroll
          for (int c0 = 0; c0 < kMaxCl; c0 += 4) {
            if (c0 >= cl) break;
            uint32_t v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = ld_cluster_u32(smem_u32(&sm.n16[b >> 1]), (uint32_t)min(c0 + c, cl - 1));
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c0 + c < cl) lo += v[c] & 0xffffu, hi += v[c] >> 16;
          }
          bn = b & 1 ? hi : lo, bw = weigh(b, bn);
          if (two) bn1 = hi, bw1 = weigh(b + 1, hi);
        });
        done = true;
        const uint64_t all = s.all_w;
        sum = all;
        if (by_k && row.find_bin(s, false, (uint64_t)top_k, n, w, bin, in_bin)) {
          if (bin == kMiddle16) {
            done = false;
          } else {
            m = (uint32_t)top_k - n;
            sum = w + m * sm.weight16[bin];
            if (sm.weight16[bin] > 0) lower(value16(bin), m);
          }
        }
        if (done && by_p) {
          const uint64_t want = row.share(top_p, sum);
          if (row.find_bin(s, true, want, n, w, bin, in_bin)) {
            if (bin == kMiddle16) {
              done = false;
            } else {
              const uint64_t each = sm.weight16[bin];
              lower(value16(bin), (uint32_t)((want - w + each - 1) / each));
            }
          }
        }
        if (!done) {
          cut = sm.floor, ties = 0xffffffffu;
          tabled = false;
          cluster_sync_all();  // every CTA has read the others' counts
        }
      }
      if (!done) row.clear_bins();
    }
    if (!done) {
#pragma unroll 2
      for (int i = threadIdx.x; i < count; i += T) {
        const float x = row.at(i), y = row.bits_below(x);
        if (y < kRange) row.into_bin((int)(y * kBinsPerBit), x, by_p);
      }
      row.scan_bins(0, 0, by_p, s);
      sum = s.all_w;
      if (by_k && row.find_bin(s, false, (uint64_t)top_k, n, w, bin, in_bin)) {
        if (n + in_bin <= kList) return store(row.draw_from_list(bin, n + in_bin, (uint32_t)top_k, by_p, top_p, 0, u));
        row.within_bin(bin, in_bin, false, by_p, (uint64_t)top_k, n, w, v, m, sum);
        lower(v, m);
      }
      if (by_p) {
        const uint64_t want = row.share(top_p, sum);
        if (row.find_bin(s, true, want, n, w, bin, in_bin)) {
          if (n + in_bin <= kList) return store(row.draw_from_list(bin, n + in_bin, 0xffffffffu, true, top_p, sum, u));
          row.within_bin(bin, in_bin, true, true, want, n, w, v, m, sum);
          lower(v, m);
        }
      }
    }
  }

  // --- the draw: sums of the kept elements by segments, in index order
  const int len = row.seg_len();
  auto sum_of = [&](int from, int to, uint64_t& w, uint32_t& n) {  // weight above the cut, elements at it
    w = 0, n = 0;
#pragma unroll 4
    for (int i = from + lane; i < to; i += 32) {
      const float v = row.at(i);
      if (v > cut)
        w += row.weight_at(i, v, tabled);
      else if (v == cut)
        ++n;
    }
    w = warp_sum(w);
    n = __reduce_add_sync(0xffffffffu, n);
  };
  auto sum_segments = [&] {
    const int from = min(count, warp * len), to = min(count, from + len);
    uint64_t w;
    uint32_t n;
    sum_of(from, to, w, n);
    if (lane == 0) sm.warp_w[warp] = w, sm.warp_n[warp] = n;
    __syncthreads();
  };
  // Where the row's values are counted, a CTA's sum follows from its counts, unless
  // the cut is among the numbers near zero; only the CTA that has the token then goes
  // over its elements (256 rows: 108 us against 112).
  const bool counted = KIND == 0 && tabled && (by_k || by_p) && !(fabsf(cut) < 0.00390625f);
  {
    if constexpr (KIND == 0) {
      if (counted) {
        uint64_t w = 0;
        uint32_t n = 0;
        for (int b = threadIdx.x; b < kBins16; b += T) {
          const uint32_t own = b & 1 ? sm.n16[b >> 1] >> 16 : sm.n16[b >> 1] & 0xffffu;
          const float v = b == kMiddle16 ? 0.0f : value16(b);
          if (v > cut)
            w += b == kMiddle16 ? sm.middle_w : own * sm.weight16[b];
          else if (v == cut)
            n += own;
        }
        w = warp_sum(w), n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) sm.warp_w[warp] = w, sm.warp_n[warp] = n;
        __syncthreads();
      }
    }
    if (!counted) sum_segments();
    if (warp == 0) {
      const uint64_t mw = lane < kWarps ? sm.warp_w[lane] : 0;
      const uint64_t all_w = warp_sum(mw);
      const uint32_t all_n = __reduce_add_sync(0xffffffffu, lane < kWarps ? sm.warp_n[lane] : 0u);
      if (lane < cl) {
        st_cluster_u64(&sm.sum_w[rank], lane, all_w);
        st_cluster_u32(&sm.sum_n[rank], lane, all_n);
      }
    }
  }
  cluster_sync_all();
  const uint64_t each = cut > -INFINITY ? row.weight(cut) : 0;
  uint64_t all = 0;
  uint32_t seen = 0;  // elements at the cut so far, which are kept in index order
  for (int c = 0; c < cl; ++c) {
    const uint32_t n = min(sm.sum_n[c], ties - seen);
    all += sm.sum_w[c] + n * each, seen += n;
  }
  const uint64_t want = min(all - 1, (uint64_t)((double)u * (double)all));
  uint64_t run = 0;
  seen = 0;
  for (int c = 0; c < rank; ++c) {
    const uint32_t n = min(sm.sum_n[c], ties - seen);
    run += sm.sum_w[c] + n * each, seen += n;
  }
  const uint64_t upto_cta = run + sm.sum_w[rank] + min(sm.sum_n[rank], ties - seen) * each;
  if (run > want || upto_cta <= want) return;  // another CTA's (none reads another's memory from here on)
  if (counted) sum_segments();
  // its segments, a lane each
  int seg;
  {
    const uint32_t n = lane < kWarps ? sm.warp_n[lane] : 0;
    const uint32_t n_before = min(ties - seen, warp_scan(n, lane) - n), kept = min(n, ties - seen - n_before);
    const uint64_t w = (lane < kWarps ? sm.warp_w[lane] : 0) + kept * each, upto = run + warp_scan(w, lane);
    seg = __ffs(__ballot_sync(0xffffffffu, upto > want)) - 1;
    run = __shfl_sync(0xffffffffu, upto - w, seg);
    seen += __shfl_sync(0xffffffffu, n_before, seg);
  }
  // the segment's parts, a warp each
  const int from = min(count, seg * len), to = min(count, from + len);
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
    const uint32_t tied_lanes = __ballot_sync(0xffffffffu, tie);
    uint64_t m = 0;
    if (v > cut) m = row.weight_at(i + lane, v, tabled);
    if (tie && (uint32_t)__popc(tied_lanes & ((1u << lane) - 1)) < ties - seen) m = each;
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
    seen += min((uint32_t)__popc(tied_lanes), ties - seen);
  }
}

template <int KIND, int T>
cudaError_t launch(const SampleParams& p, int cl, cudaStream_t stream) {
  constexpr int E = KIND == 2 ? 4 : 2;
  constexpr int kHead = (sizeof(Shared<KIND>) + 15) / 16 * 16 + 16;
  constexpr int kMost = kHead + (int)(kMaxVocab / kMaxCl) * E;
  static_assert(kMost <= 232448, "shared memory of a CTA");
  static_assert(kMaxVocab / kMaxCl < 65536, "sums of 16 bits of a slice's weights fit 32");
  static_assert(kMaxVocab <= 1 << 22, "sums of a row's weights fit 63 bits");
  const int slice = ((p.N + cl - 1) / cl + 7) / 8 * 8;  // (16 bytes keep their place)
  const void* fn = reinterpret_cast<const void*>(&sample_kernel<KIND, T>);
  cudaError_t e = set_smem_once(fn, kMost, (T == 1024 ? 133 : 130) + KIND);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.R * cl));
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = kHead + slice * E;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<KIND, T>, p, cl, slice);
}

template <int KIND>
cudaError_t launch(const SampleParams& p, int num_sms, cudaStream_t stream) {
  // Slices of at most 16384 elements while a cluster of eight has them; in 16 bits
  // 32768 for batches that fill the GPU in any case, two CTAs an SM: half of what
  // each does whatever its slice is (256 bf16 rows of 128256 with top-p: 121 us
  // against 158).  An SM to each CTA, when there are so few: twice the threads,
  // half the time of a pass.
  auto clusters = [&](int slice) {
    int cl = 1;
    while (cl < kMaxCl && p.N > slice * cl) cl *= 2;
    return cl;
  };
  int cl = clusters(16384);
  if (p.R * cl <= num_sms) return launch<KIND, 1024>(p, cl, stream);
  if (KIND != 2 && p.R * cl > 2 * (int64_t)num_sms) cl = clusters(32768);
  return launch<KIND, 512>(p, cl, stream);
}

}  // namespace

bi_status launch_sample(SampleParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  p.status_word = dev.status_word;
  const cudaError_t e = p.x_kind == 2   ? launch<2>(p, dev.num_sms, stream)
                        : p.x_kind == 1 ? launch<1>(p, dev.num_sms, stream)
                                        : launch<0>(p, dev.num_sms, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    *why = std::string("sampling launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
