// bi_paged_attn.cu -- attention of one new token per request over a paged
// key-value cache, query heads grouped over key-value heads:
//   o[b,h,:] = sum_j softmax_j(scale q[b,h,:] . k[b,j,h/G,:]) v[b,j,h/G,:],  j < len_b.
//
// What bounds it.  Every key and value is used by the G query heads of one
// group only, 4 G flops an element, so the call is bound by reading the cache
// once; the kernel's job is to keep enough of those reads in flight.
//
// Split.  A request's keys are cut into pieces by a rule on its own length
// alone (paged_split_len), so its bits depend neither on the batch nor on the
// grid.  A unit of work is (request, piece, key-value head, tile of 8 NT of
// its query heads); a persistent grid takes units in order, key-value heads
// fastest, since the heads of one cached token lie side by side in memory.
// The units of a ragged batch are counted in the kernel by prefix sums of the
// requests' piece counts, so there is no block without work and the host needs
// no lengths.
//
// Tile.  The eight warps of a CTA take 16-key tiles of the unit in turn and
// never meet before its end.  Both products run on mma.sync m16n8k16 with the
// long side on M: S^T = K Q^T (16 keys x 8 heads) and O^T += V^T P^T (16
// dimensions x 8 heads).  With one token a head there are 8 rows to a product,
// which a 128-row tcgen05 tile would waste 15/16 of, and the tensor work is a
// third of the load time even so.  Operands go from global memory straight to
// the registers that the product wants them in, 16 bytes a lane: the order of
// the head dimension inside a dot product is free, so lane (g, c) = (lane / 4,
// lane % 4) takes dimensions 32 j + 8 c .. + 7 of keys g and g + 8, four lanes
// covering 64 contiguous bytes; and V^T's fragments want pairs of neighbouring
// keys at one dimension, so lane (g, c) takes dimensions 64 i + 8 g .. + 7 of
// keys 2c, 2c+1, 2c+8, 2c+9 (eight lanes cover 128 bytes) and joins the pairs
// with byte permutes.  P^T's fragment is S^T's transposed in 8 x 8 blocks
// (movmatrix).  No shared memory, no barrier and no copy stage in the loop:
// the next tile's keys are requested before this tile's softmax, its values
// before its scores, so a warp always has 16 keys or values in flight.
//
// Arithmetic, per query head: t = RN(s c) with c = RN(scale log2 e); a running
// maximum m per warp over its tiles; p = 2^(t - m) (the SFU's approximation);
// l sums the unrounded p in fp32; the value product takes p in the cache's
// 16-bit type, the tensor core's operand type: for a 16-bit result one
// rounding of p (the weights are positive, so the result is off by at most
// half a step of the averaged |v|, like its own rounding), for an fp32 result
// p as the sum of two such numbers, 16 or more bits.  O in fp32.  Warps are
// joined in warp order, pieces in piece order: O = sum_w 2^(m_w - M) O_w.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
#include "bi_serve.h"

namespace bi {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;           // keys per warp and step
constexpr int kMinSplit = 256;      // keys of a piece at least
constexpr int kManySplits = 128;    // pieces of a request at most

__host__ __device__ inline int32_t paged_split_len(int64_t len) {
  int64_t s = kMinSplit;
  while (len > kManySplits * s) s *= 2;
  return (int32_t)s;
}
__host__ __device__ inline int32_t split_count(int64_t len) {
  const int32_t s = paged_split_len(len);
  return len <= 0 ? 1 : (int32_t)((len + s - 1) / s);  // an empty request is one unit that writes zeros
}

template <int F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <int F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <int F16>
__device__ __forceinline__ float low16(uint32_t v) {
  if constexpr (F16) return __low2float(*reinterpret_cast<const __half2*>(&v));
  return __uint_as_float(v << 16);
}
template <int F16>
__device__ __forceinline__ float high16(uint32_t v) {
  if constexpr (F16) return __high2float(*reinterpret_cast<const __half2*>(&v));
  return __uint_as_float(v & 0xffff0000u);
}
// 16 bytes of the cache: read once, so kept out of L1.
__device__ __forceinline__ uint4 load_cache(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ void store_out(void* o, int kind, int64_t i, const float (&f)[4]) {
  if (kind == 2) {
    *reinterpret_cast<float4*>(static_cast<float*>(o) + i) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    const uint2 w = kind == 1 ? make_uint2(pack16<1>(f[0], f[1]), pack16<1>(f[2], f[3]))
                              : make_uint2(pack16<0>(f[0], f[1]), pack16<0>(f[2], f[3]));
    *reinterpret_cast<uint2*>(static_cast<unsigned short*>(o) + i) = w;
  }
}

// Keys of request b: its length, at most what its table row can name.
__device__ __forceinline__ int request_len(const PagedAttnParams& p, int b) {
  const int n = __ldg(p.lens + b);
  if (n > p.cap) record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedPage));
  return max(0, min(n, p.cap));
}

constexpr int kNoKey = -1;

// Cache slot (page * ps + row) of key j of a request with table row `tab`;
// kNoKey past its end or on a page that does not exist.
__device__ __forceinline__ int key_slot(const PagedAttnParams& p, const int32_t* tab, int j, int end) {
  if (j >= end) return kNoKey;
  const uint32_t col = (uint32_t)j / (uint32_t)p.ps;
  const int page = __ldg(tab + col);
  if (page < 0 || page >= p.P) {
    record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedPage));
    return kNoKey;
  }
  return page * p.ps + (int)((uint32_t)j - col * (uint32_t)p.ps);
}

template <int F16, int D, int NT>
struct Shared {
  float o[kWarps][8 * NT][D];
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
  int32_t start[kThreads + 1];  // units of the requests before thread i's
  int32_t warp_sum[kWarps];
};

// PS: 16-bit pieces of p in the value product, 2 for an fp32 result.
template <int F16, int D, int NT, int PS>
__global__ void __launch_bounds__(kThreads, D == 64 ? 3 : (D == 128 && NT == 1 ? 2 : 1))
    paged_attn_kernel(const PagedAttnParams p) {
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared<F16, D, NT>& sm = *reinterpret_cast<Shared<F16, D, NT>*>(dyn);
  constexpr int KJ = D / 32, VI = D / 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;

  // units before each thread's requests
  const int per = (p.B + kThreads - 1) / kThreads;
  {
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int n = 0;
    for (int b = b0; b < b1; ++b) n += split_count(request_len(p, b));
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) sm.warp_sum[warp] = sum;
    __syncthreads();
    for (int i = 0; i < warp; ++i) sum += sm.warp_sum[i];
    sm.start[threadIdx.x] = sum - n;
    if (threadIdx.x == kThreads - 1) sm.start[kThreads] = sum;
    __syncthreads();
  }
  const int inner = p.Hkv * p.head_tiles;
  const int64_t units = (int64_t)sm.start[kThreads] * inner;

  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int ss = (int)(unit / inner), hk = (int)(unit % inner);
    const int kvh = hk / p.head_tiles, h0 = (hk % p.head_tiles) * 8 * NT;
    int lo = 0, hi = min(kThreads, (p.B + per - 1) / per);
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sm.start[mid] <= ss)
        lo = mid;
      else
        hi = mid;
    }
    int b = lo * per, at = sm.start[lo], len = request_len(p, b);
    while (ss >= at + split_count(len)) at += split_count(len), len = request_len(p, ++b);
    const int piece = ss - at, pieces = split_count(len);
    const int k0 = piece * paged_split_len(len), k1 = min(len, k0 + paged_split_len(len));
    const int32_t* tab = p.table + b * p.ld_table;
    const int heads = min(8 * NT, p.group - h0);  // query heads of this unit
    const int head = kvh * p.group + h0;

    // Q^T fragments: head g of tile n, dimensions 32 j + 8 c .. + 7
    uint4 q[NT][KJ];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < KJ; ++j)
        q[n][j] = 8 * n + g < heads
                      ? __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(p.q) + b * p.q_b +
                                                             (head + 8 * n + g) * p.q_h + 32 * j + 8 * c))
                      : make_uint4(0, 0, 0, 0);

    float o[VI][4][NT][4] = {};
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.0f;

    const unsigned short* kb = static_cast<const unsigned short*>(p.k) + kvh * p.k_head + 8 * c;
    const unsigned short* vb = static_cast<const unsigned short*>(p.v) + kvh * p.v_head + 8 * g;
    // A step of the loop is one tile of 16 keys; `slot` holds, in lanes 0..15
    // (and again in 16..31), the cache slots of the tile's keys.
    auto load_keys = [&](int slot, uint4 (&k)[2][KJ]) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int s = __shfl_sync(0xffffffffu, slot, g + 8 * r);
        const uint32_t page = (uint32_t)s / (uint32_t)p.ps, row = (uint32_t)s % (uint32_t)p.ps;
        const unsigned short* a = kb + page * p.k_page + row * p.k_row;
#pragma unroll
        for (int j = 0; j < KJ; ++j) k[r][j] = s >= 0 ? load_cache(a + 32 * j) : make_uint4(0, 0, 0, 0);
      }
    };
    int slot = key_slot(p, tab, k0 + warp * kTile + (lane & 15), k1);
    uint4 k[2][KJ];
    load_keys(slot, k);
    for (int key = k0 + warp * kTile; key < k1; key += kWarps * kTile) {
      // values of this tile: keys 2c, 2c+1, 2c+8, 2c+9
      uint4 v[4][VI];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int s = __shfl_sync(0xffffffffu, slot, 2 * c + (r & 1) + 8 * (r >> 1));
        const uint32_t page = (uint32_t)s / (uint32_t)p.ps, row = (uint32_t)s % (uint32_t)p.ps;
        const unsigned short* a = vb + page * p.v_page + row * p.v_row;
#pragma unroll
        for (int i = 0; i < VI; ++i) v[r][i] = s >= 0 ? load_cache(a + 64 * i) : make_uint4(0, 0, 0, 0);
      }
      const uint32_t live = __ballot_sync(0xffffffffu, slot >= 0);
      const int next = key_slot(p, tab, key + kWarps * kTile + (lane & 15), k1);
      // scores of keys g (elements 0, 1) and g + 8 (2, 3) for heads 2c, 2c + 1
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          mma16816<F16>(s[n], k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y, q[n][j].x, q[n][j].y);
          mma16816<F16>(s[n], k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w, q[n][j].z, q[n][j].w);
        }
      }
      load_keys(next, k);
      slot = next;
      uint32_t pf[NT][PS][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[i] = (live >> (g + 8 * (i >> 1))) & 1 ? __fmul_rn(s[n][i], p.score_log2) : -INFINITY;
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = fmaxf(t[h], t[2 + h]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          mx = fmaxf(mx, m[n][h]);
          const float ref = mx == -INFINITY ? 0.0f : mx;  // no key yet: every p is 0
          alpha[h] = ex2_approx(m[n][h] - ref);
          m[n][h] = mx;
          t[h] = ex2_approx(t[h] - ref);
          t[2 + h] = ex2_approx(t[2 + h] - ref);
          l[n][h] = fmaf(l[n][h], alpha[h], t[h] + t[2 + h]);
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < VI; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              o[i][w][n][0] *= alpha[0], o[i][w][n][1] *= alpha[1];
              o[i][w][n][2] *= alpha[0], o[i][w][n][3] *= alpha[1];
            }
        }
#pragma unroll
        for (int x = 0; x < PS; ++x) {
          const uint32_t lo = pack16<F16>(t[0], t[1]), hi = pack16<F16>(t[2], t[3]);
          pf[n][x][0] = transpose8x8(lo);
          pf[n][x][1] = transpose8x8(hi);
          if (x + 1 < PS) {
            t[0] -= low16<F16>(lo), t[1] -= high16<F16>(lo);
            t[2] -= low16<F16>(hi), t[3] -= high16<F16>(hi);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // rows g: dimension 64 i + 8 g + 2 w; rows g + 8: the one after it
          const uint32_t x0 = word(v[0][i], w), x1 = word(v[1][i], w), x2 = word(v[2][i], w), x3 = word(v[3][i], w);
          const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
          const uint32_t a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < PS; ++x) mma16816<F16>(o[i][w][n], a0, a1, a2, a3, pf[n][x][0], pf[n][x][1]);
        }
    }

    // join the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], x);
        const int hh = 8 * n + 2 * c + h;
        if (g == 0) sm.m[warp][hh] = m[n][h], sm.l[warp][hh] = l[n][h];
        if (hh < heads) {
#pragma unroll
          for (int i = 0; i < VI; ++i) {
            float4* dst = reinterpret_cast<float4*>(&sm.o[warp][hh][64 * i + 8 * g]);
            dst[0] = make_float4(o[i][0][n][h], o[i][0][n][2 + h], o[i][1][n][h], o[i][1][n][2 + h]);
            dst[1] = make_float4(o[i][2][n][h], o[i][2][n][2 + h], o[i][3][n][h], o[i][3][n][2 + h]);
          }
        }
      }
    __syncthreads();
    for (int e = threadIdx.x; e < heads * (D / 4); e += kThreads) {
      const int h = e / (D / 4), d = (e % (D / 4)) * 4;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][h]);
      const float ref = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f, a[4] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(sm.m[w][h] - ref);
        const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][h][d]);
        sum = fmaf(f, sm.l[w][h], sum);
        a[0] = fmaf(f, x.x, a[0]), a[1] = fmaf(f, x.y, a[1]), a[2] = fmaf(f, x.z, a[2]), a[3] = fmaf(f, x.w, a[3]);
      }
      if (pieces == 1) {
        const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum);  // no key: zeros
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = __fmul_rn(a[i], inv);
        store_out(p.o, p.out_kind, b * p.o_b + (head + h) * p.o_h + d, a);
      } else {
        const int64_t row = ((int64_t)b * p.max_splits + piece) * p.Hq + head + h;
        *reinterpret_cast<float4*>(p.ws_o + row * D + d) = make_float4(a[0], a[1], a[2], a[3]);
        if (d == 0) p.ws_ml[2 * row] = mx, p.ws_ml[2 * row + 1] = sum;
      }
    }
    __syncthreads();
  }
}

// Joins the pieces of one (request, query head): M = max m_s, then sums of
// 2^(m_s - M) (l_s, O_s), warp w over pieces w, w + 8, ... in ascending order,
// the warps in warp order.  A request of one piece has its result already.
template <int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const PagedAttnParams p) {
  constexpr int V = D / 32;  // dimensions of a lane: 2, 4 or 8
  __shared__ float so[kWarps][D];
  __shared__ float sl[kWarps];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = split_count(request_len(p, b));
  if (n == 1) return;
  const int64_t row0 = (int64_t)b * p.max_splits * p.Hq + h;
  float mx = -INFINITY;
  for (int s = lane; s < n; s += 32) mx = fmaxf(mx, p.ws_ml[2 * (row0 + (int64_t)s * p.Hq)]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
  const float ref = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f, a[V] = {};
#pragma unroll 4
  for (int s = warp; s < n; s += kWarps) {
    const int64_t row = row0 + (int64_t)s * p.Hq;
    const float f = ex2_approx(p.ws_ml[2 * row] - ref);
    sum = fmaf(f, p.ws_ml[2 * row + 1], sum);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 x = *reinterpret_cast<const float2*>(p.ws_o + row * D + 64 * (i / 2) + 2 * lane);
      a[i] = fmaf(f, x.x, a[i]), a[i + 1] = fmaf(f, x.y, a[i + 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < V; i += 2) *reinterpret_cast<float2*>(&so[warp][64 * (i / 2) + 2 * lane]) = make_float2(a[i], a[i + 1]);
  if (lane == 0) sl[warp] = sum;
  __syncthreads();
  if (threadIdx.x < D / 4) {
    const int d = 4 * threadIdx.x;
    float l = 0.0f, r[4] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      l += sl[w];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] += so[w][d + i];
    }
    const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __fmul_rn(r[i], inv);
    store_out(p.o, p.out_kind, b * p.o_b + h * p.o_h + d, r);
  }
}

template <int F16, int D, int NT, int PS>
cudaError_t launch(PagedAttnParams& p, int num_sms, cudaStream_t stream) {
  constexpr int kBytes = sizeof(Shared<F16, D, NT>);
  constexpr int kPerSm = D == 64 ? 3 : (D == 128 && NT == 1 ? 2 : 1);
  // one slot per instance: 20 of them, from 24 on
  constexpr int kSlot = 24 + (D == 256 ? 16 + 2 * F16 + (PS - 1) : (D == 128 ? 8 : 0) + 4 * F16 + 2 * (NT - 1) + (PS - 1));
  static_assert(kSlot < 48, "set_smem_once's table");
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(&paged_attn_kernel<F16, D, NT, PS>), kBytes, kSlot);
  if (e != cudaSuccess) return e;
  p.head_tiles = (p.group + 8 * NT - 1) / (8 * NT);
  const int64_t most = (int64_t)p.B * p.max_splits * p.Hkv * p.head_tiles;
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)num_sms * kPerSm);
  paged_attn_kernel<F16, D, NT, PS><<<grid, kThreads, kBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int F16, int D, int NT>
cudaError_t launch_out(PagedAttnParams& p, int num_sms, cudaStream_t stream) {
  return p.out_kind == 2 ? launch<F16, D, NT, 2>(p, num_sms, stream) : launch<F16, D, NT, 1>(p, num_sms, stream);
}

template <int F16>
cudaError_t launch_dim(PagedAttnParams& p, int num_sms, cudaStream_t stream) {
  // more than eight query heads a key-value head: 16 a unit, except at
  // D = 256, where two tiles' accumulators would not fit the registers
  const bool wide = p.group > 8;
  if (p.D == 64) return wide ? launch_out<F16, 64, 2>(p, num_sms, stream) : launch_out<F16, 64, 1>(p, num_sms, stream);
  if (p.D == 128) return wide ? launch_out<F16, 128, 2>(p, num_sms, stream) : launch_out<F16, 128, 1>(p, num_sms, stream);
  return launch_out<F16, 256, 1>(p, num_sms, stream);
}

}  // namespace

int32_t paged_splits(int64_t len) { return split_count(len); }
int32_t paged_max_splits(int64_t cap) {
  return cap >= (int64_t)kManySplits * kMinSplit ? kManySplits : split_count(cap);
}

bi_status launch_paged_attention(PagedAttnParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  p.status_word = dev.status_word;
  cudaError_t e = p.in_f16 ? launch_dim<1>(p, dev.num_sms, stream) : launch_dim<0>(p, dev.num_sms, stream);
  if (e == cudaSuccess && p.max_splits > 1) {
    const unsigned rows = (unsigned)((int64_t)p.B * p.Hq);
    if (p.D == 64)
      paged_join_kernel<64><<<rows, kThreads, 0, stream>>>(p);
    else if (p.D == 128)
      paged_join_kernel<128><<<rows, kThreads, 0, stream>>>(p);
    else
      paged_join_kernel<256><<<rows, kThreads, 0, stream>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    *why = std::string("paged attention launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
