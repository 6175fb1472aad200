// bi_quant.cu -- quantisation of a matrix in blocks: q = e4m3(x / s), one scale
// s = 2^e for each block of 1 x 128 (rows of activations) or 128 x 128
// (weights).  Every element is read once and written once as a byte: the call
// is bound by memory, small ones by one load's latency and the launch.
//
// A half-warp takes a row's 128 elements of a block, eight a lane (16 bytes of
// a 16-bit type), and holds them in registers between the two steps: their
// largest magnitude -- as bits, whose order is the numbers', a NaN above all --
// then the rounding of each.  A 128 x 128 block is a block of 512 threads, four
// rows a half-warp, the maximum joined through shared memory.
//
// Measured: a weight of 14336 x 4096 bf16, 176 MB in and out, 29.4-30.2 us, 5.9 TB/s (0.87
// of the copy rate; what is left is the barrier between a block's reads and its
// writes: 256 threads of eight rows, three blocks an SM, 32.0 us, four 30.6 but fp32
// 29.8 for 24.1; 1024 threads 37.8).  Rows of 16 x 4096 take 1.6 us, of 8192 x 4096 23.2:
// 4.4 TB/s, by issue (71 % of the cycles).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_e4m3.cuh"
#include "bi_launch.h"
#include "bi_quant.h"

namespace bi {
namespace {

constexpr int kThreads = 256, kTileThreads = 512;

// Eight elements of a row from column k on as they lie in memory, zeros past K.
template <int KIND>
struct Oct {
  uint4 w[KIND == 2 ? 2 : 1];

  __device__ __forceinline__ void load(const QuantParams& p, int64_t row, int k, bool there) {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (KIND == 2) w[1] = w[0];
    if (!there || k >= p.K) return;
    if (p.vec && k + 8 <= p.K) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(p.x) + (row * p.ld_x + k) * (KIND == 2 ? 4 : 2));
      w[0] = __ldcs(s);
      if constexpr (KIND == 2) w[1] = __ldcs(s + 1);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = 0;
        if (k + i < p.K) {
          if constexpr (KIND == 2)
            e[i] = static_cast<const uint32_t*>(p.x)[row * p.ld_x + k + i];
          else
            e[i] = static_cast<const uint16_t*>(p.x)[row * p.ld_x + k + i];
        }
      }
      if constexpr (KIND == 2) {
        w[0] = make_uint4(e[0], e[1], e[2], e[3]);
        w[1] = make_uint4(e[4], e[5], e[6], e[7]);
      } else {
        w[0] = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
      }
    }
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[KIND == 2].x, w[KIND == 2].y, w[KIND == 2].z, w[KIND == 2].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (KIND == 2)
        f[i] = __uint_as_float(v[i]);
      else if constexpr (KIND == 1)
        f[i] = __half2float(__ushort_as_half((unsigned short)(v[i >> 1] >> (16 * (i & 1)))));
      else
        f[i] = __uint_as_float(i & 1 ? v[i >> 1] & 0xffff0000u : v[i >> 1] << 16);
    }
  }
  __device__ __forceinline__ uint32_t size() const {
    float f[8];
    values(f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void store(const QuantParams& p, int64_t row, int k, float inv, bool there) const {
    if (!there || k >= p.K) return;
    float f[8];
    values(f);
    const uint32_t lo = to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    const uint32_t hi = to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    uint8_t* o = p.q + row * p.ld_q + k;
    if (p.vec && k + 8 <= p.K) {
      *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < p.K) o[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
  }
};

__device__ __forceinline__ uint32_t max_of_16(uint32_t m) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// Blocks of 1 x 128: U of them a half-warp, neighbouring ones neighbouring half-warps'.
template <int KIND, int U>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantParams p) {
  const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const uint32_t all = (uint32_t)p.M * (uint32_t)p.kb;
  Oct<KIND> x[U];
  uint32_t row[U], col[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t b = (blockIdx.x * U + i) * (kThreads / 16) + half;
    row[i] = b / (uint32_t)p.kb, col[i] = b - row[i] * (uint32_t)p.kb;
    x[i].load(p, row[i], (int)col[i] * 128 + lane * 8, b < all);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const bool there = (blockIdx.x * U + i) * (kThreads / 16) + half < all;
    const float scale = block_scale(max_of_16(x[i].size()));
    x[i].store(p, row[i], (int)col[i] * 128 + lane * 8, inverse_scale(scale), there);
    if (lane == 0 && there) p.scales[row[i] * p.s_m + col[i] * p.s_k] = scale;
  }
}

// Blocks of 128 x 128.
template <int KIND>
__global__ void __launch_bounds__(kTileThreads, 3) quantize_tiles_kernel(const QuantParams p) {
  constexpr int U = 128 / (kTileThreads / 16);
  __shared__ uint32_t part[kTileThreads / 32];
  const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const uint32_t mb = blockIdx.x / (uint32_t)p.kb, kb = blockIdx.x - mb * (uint32_t)p.kb;
  const int k = (int)kb * 128 + lane * 8;
  Oct<KIND> x[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t row = (int64_t)mb * 128 + i * (kTileThreads / 16) + half;
    x[i].load(p, row, k, row < p.M);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) m = max(m, x[i].size());
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileThreads / 32; ++i) m = max(m, part[i]);
  const float scale = block_scale(m), inv = inverse_scale(scale);
  if (threadIdx.x == 0) p.scales[mb * p.s_m + kb * p.s_k] = scale;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t row = (int64_t)mb * 128 + i * (kTileThreads / 16) + half;
    x[i].store(p, row, k, inv, row < p.M);
  }
}

template <int KIND>
void launch_kind(const QuantParams& p, int num_sms, cudaStream_t stream) {
  if (p.rows == 128) {
    const int64_t tiles = ((int64_t)p.M + 127) / 128 * p.kb;
    quantize_tiles_kernel<KIND><<<(unsigned)tiles, kTileThreads, 0, stream>>>(p);
    return;
  }
  const int64_t blocks = (int64_t)p.M * p.kb, group = kThreads / 16;
  // four blocks of 128 a half-warp, all requested at once, when there are many (rows of 4096,
  // measured side by side: 8191 of them 21.8 us against 22.6, 2400 8.0 against 7.8, 600 3.8
  // against 3.3)
  if (blocks >= 32 * group * num_sms)
    quantize_rows_kernel<KIND, 4><<<(unsigned)((blocks + 4 * group - 1) / (4 * group)), kThreads, 0, stream>>>(p);
  else
    quantize_rows_kernel<KIND, 1><<<(unsigned)((blocks + group - 1) / group), kThreads, 0, stream>>>(p);
}

}  // namespace

bi_status launch_quantize(const QuantParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  if (p.kind == 2)
    launch_kind<2>(p, dev.num_sms, stream);
  else if (p.kind == 1)
    launch_kind<1>(p, dev.num_sms, stream);
  else
    launch_kind<0>(p, dev.num_sms, stream);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("quantisation launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
