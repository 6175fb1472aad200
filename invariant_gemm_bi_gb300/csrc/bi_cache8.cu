// bi_cache8.cu -- reading rows of a paged cache in 8 bits back as numbers:
//   k[t, h, :] = k_cache[slots[t]][h, :] * k_scales[slots[t]][h],  v likewise.
//
// Every byte is read once and every result written once: the call is bound by
// memory.  A thread takes 16 elements of one head (16 bytes in, 32 out in 16
// bits); neighbouring threads take neighbouring units of a token, whose heads
// lie side by side in the cache, and each thread four units, keys and values
// of two tokens, whose loads are all requested before the first is used.
//
// Products are rounded to fp32, where those with a power of two for a scale (the
// library's own) are exact, then to a result of 16 bits.  With any other scale that
// is a second rounding: about one result in 2^17 of bf16, one in 2^14 of fp16, is
// put on the other side of a tie.
//
// Measured: 131071 tokens of 8 heads of 128 into bf16, 815 MB in and out, 132 us,
// 6.2 TB/s (0.91 of the copy rate); 1021 tokens 3.5 us, three dependent loads
// (slot, row, store) and the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_e4m3.cuh"
#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
#include "bi_serve.h"

namespace bi {
namespace {

// Element (0) of head h of the row at `slot`, and its scale; null for a slot that there is not.
__device__ __forceinline__ const uint8_t* row_of(const LoadParams& p, bool v, int64_t slot, int h, float* scale) {
  if (slot >= p.num_slots) record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedSlot));
  if (slot < 0 || slot >= p.num_slots) return nullptr;
  const uint32_t page = (uint32_t)slot / (uint32_t)p.ps, row = (uint32_t)slot - page * (uint32_t)p.ps;
  const PageView& s = v ? p.vs : p.ks;
  const PageView& c = v ? p.vc : p.kc;
  *scale = __ldg(static_cast<const float*>(s.ptr) + page * s.page + row * s.row + h * s.head);
  return static_cast<const uint8_t*>(c.ptr) + page * c.page + row * c.row + h * c.head;
}

template <int KIND>
__device__ __forceinline__ uint32_t pair_of(uint32_t e4m3x2, float scale) {
  const float2 f = e4m3x2_to_float2(e4m3x2);
  if constexpr (KIND == 1) {
    const __half2 h = __floats2half2_rn(f.x * scale, f.y * scale);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

constexpr int kThreads = 256;
constexpr int kTokens = 2;  // tokens a thread takes, with keys and values

template <int KIND>
__global__ void __launch_bounds__(kThreads) load_kernel(const LoadParams p) {
  const uint32_t per = p.D / 16, line = p.H * per;  // units of a head, of a token
  const uint32_t pairs = ((uint32_t)p.T + kTokens - 1) / kTokens;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= (int64_t)pairs * line) return;
  const uint32_t group = (uint32_t)(id / line), u = (uint32_t)(id - (int64_t)group * line);
  const int h = (int)(u / per), d = (int)(u - h * per) * 16;
  uint4 x[kTokens][2];
  float scale[kTokens][2];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int64_t t = (int64_t)group * kTokens + i;
    const int64_t slot = t < p.T ? __ldg(p.slots + t) : -1;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      scale[i][v] = 0.0f;
      const uint8_t* src = row_of(p, v != 0, slot, h, &scale[i][v]);
      x[i][v] = src ? __ldcs(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int64_t t = (int64_t)group * kTokens + i;
    if (t >= p.T) break;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int64_t at = v ? t * p.v_t + h * p.v_h + d : t * p.k_t + h * p.k_h + d;
      void* o = v ? p.v : p.k;
      const uint32_t w[4] = {x[i][v].x, x[i][v].y, x[i][v].z, x[i][v].w};
      const float s = scale[i][v];
      if constexpr (KIND == 2) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(o) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = e4m3x2_to_float2(w[j] & 0xffffu), b = e4m3x2_to_float2(w[j] >> 16);
          __stcs(dst + j, make_float4(a.x * s, a.y * s, b.x * s, b.y * s));
        }
      } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(o) + at);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          __stcs(dst + j, make_uint4(pair_of<KIND>(w[2 * j] & 0xffffu, s), pair_of<KIND>(w[2 * j] >> 16, s),
                                     pair_of<KIND>(w[2 * j + 1] & 0xffffu, s), pair_of<KIND>(w[2 * j + 1] >> 16, s)));
      }
    }
  }
}

// Any alignment: a warp a token's head, an element a lane.
__global__ void __launch_bounds__(kThreads) load_any_kernel(const LoadParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t all = (int64_t)p.T * p.H * 2;
  for (int64_t id = (int64_t)blockIdx.x * (kThreads / 32) + warp; id < all; id += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t t = id / (2 * p.H);
    const int r = (int)(id - t * (2 * p.H)), h = r >> 1;
    const bool v = r & 1;
    float scale = 0.0f;
    const uint8_t* src = row_of(p, v, __ldg(p.slots + t), h, &scale);
    const int64_t at = v ? t * p.v_t + h * p.v_h : t * p.k_t + h * p.k_h;
    void* o = v ? p.v : p.k;
    for (int d = lane; d < p.D; d += 32) {
      const float f = src ? e4m3x2_to_float2(src[d]).x * scale : 0.0f;
      if (p.kind == 2)
        static_cast<float*>(o)[at + d] = f;
      else if (p.kind == 1)
        static_cast<__half*>(o)[at + d] = __float2half_rn(f);
      else
        static_cast<__nv_bfloat16*>(o)[at + d] = __float2bfloat16_rn(f);
    }
  }
}

}  // namespace

bi_status launch_paged_load(LoadParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  p.status_word = dev.status_word;
  if (p.vec) {
    const int64_t threads = ((int64_t)p.T + kTokens - 1) / kTokens * p.H * (p.D / 16);
    const unsigned grid = (unsigned)((threads + kThreads - 1) / kThreads);
    if (p.kind == 2)
      load_kernel<2><<<grid, kThreads, 0, stream>>>(p);
    else if (p.kind == 1)
      load_kernel<1><<<grid, kThreads, 0, stream>>>(p);
    else
      load_kernel<0><<<grid, kThreads, 0, stream>>>(p);
  } else {
    const int64_t warps = (int64_t)p.T * p.H * 2;
    load_any_kernel<<<(unsigned)std::min<int64_t>((warps + 7) / 8, 1 << 20), kThreads, 0, stream>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("paged load launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
