// bi_rope.cu -- rotary positions, and the paged-cache write that goes with
// them: pair (x1, x2) of a head at position n is turned by n f_i,
//   y1 = a (x1 cos - x2 sin),  y2 = a (x1 sin + x2 cos),
// the transposed map (sin negated) being its gradient.
//
// Angles.  An fp32 product n * f_i loses the angle at far positions (at
// n = 10^6 it is off by up to 0.03 rad), and fp64 is slow on this chip.  The
// frequency is held as a 64-bit binary fraction of a turn, so the integer
// product phase * n mod 2^64 is the angle modulo one turn, off by at most
// n 2^-65 turns; its top 32 bits, signed, scale to half turns in [-1, 1) and
// sincospif needs no further reduction.  What remains is that number's
// rounding to fp32: under 1.2e-7 rad.
//
// Work.  A thread owns one unit of a token's head -- 8 pairs (two 16-byte
// pieces of 16-bit data) or 16 elements of the unrotated tail -- computes its
// 8 sines and cosines once and then walks over heads h0, h0 + step, ...,
// kBatch of them loaded together, so the trigonometry is paid once for all of
// a thread's heads and no shared memory or barrier is needed.  Operands whose
// rows or split are not 16-byte aligned take units of one pair with the same
// arithmetic, so the bits do not depend on the layout.  The kernel reads and
// writes every element once: it is bound by memory bandwidth, small calls by
// one load's latency plus the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_launch.h"
#include "bi_ptx.cuh"
#include "bi_serve.h"

namespace bi {
namespace {

constexpr int kAny = -1;  // element kind read from the parameters

__device__ __forceinline__ float half_to_f(uint32_t h, int kind) {
  return kind == 1 ? __half2float(__ushort_as_half((unsigned short)h)) : __uint_as_float(h << 16);
}
__device__ __forceinline__ uint32_t f_to_half(float v, int kind) {
  return kind == 1 ? (uint32_t)__half_as_ushort(__float2half_rn(v))
                   : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ int elem_bytes(int kind) { return kind == 2 ? 4 : 2; }

// Eight consecutive elements (16-byte aligned) as raw words: 4 or 8 of them.
struct Oct {
  uint4 a, b;
};
__device__ __forceinline__ Oct load_oct(const void* p, int kind) {
  Oct o;
  o.a = *reinterpret_cast<const uint4*>(p);
  if (kind == 2) o.b = *(reinterpret_cast<const uint4*>(p) + 1);
  return o;
}
__device__ __forceinline__ void unpack_oct(const Oct& o, int kind, float (&f)[8]) {
  const uint32_t w[8] = {o.a.x, o.a.y, o.a.z, o.a.w, o.b.x, o.b.y, o.b.z, o.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = kind == 2 ? __uint_as_float(w[i]) : half_to_f((w[i >> 1] >> (16 * (i & 1))) & 0xffffu, kind);
}
__device__ __forceinline__ void store_oct(void* p, int kind, const float (&f)[8]) {
  if (kind == 2) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f_to_half(f[2 * i], kind) | (f_to_half(f[2 * i + 1], kind) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ float load_one(const void* p, int kind) {
  return kind == 2 ? *reinterpret_cast<const float*>(p) : half_to_f(*reinterpret_cast<const unsigned short*>(p), kind);
}
__device__ __forceinline__ void store_one(void* p, int kind, float v) {
  if (kind == 2)
    *reinterpret_cast<float*>(p) = v;
  else
    *reinterpret_cast<unsigned short*>(p) = (unsigned short)f_to_half(v, kind);
}

// a cos and a sin of position n's angle for pair i.
__device__ __forceinline__ void turn(const RopeParams& p, int64_t n, int i, float& c, float& s) {
  const uint64_t t = p.phase[i] * (uint64_t)n;
  sincospif(__fmul_rn((float)(int32_t)(t >> 32), 4.656612873077393e-10f /* 2^-31 */), &s, &c);
  c = __fmul_rn(c, p.magnitude);
  s = __fmul_rn(p.transpose ? -s : s, p.magnitude);
}
// One rotated pair: a product rounded, then one fused multiply-add.
__device__ __forceinline__ void rotate(float& x1, float& x2, float c, float s) {
  const float y1 = __fmaf_rn(x1, c, -__fmul_rn(x2, s));
  x2 = __fmaf_rn(x2, c, __fmul_rn(x1, s));
  x1 = y1;
}

// Where head slot h of token t (q heads, then k heads, then v heads) is read
// and written; dst is null for a token that is not stored.
struct Place {
  const char* src;
  char* dst;
  int in, out;  // element kinds
  bool rotated;
};
template <int QK, int QO, int KV, int CK>
__device__ __forceinline__ Place place(const RopeParams& p, int64_t t, int h, int64_t slot) {
  Place r;
  if (h < p.hq) {
    r.in = QK == kAny ? p.q_kind : QK;
    r.out = QO == kAny ? p.qo_kind : QO;
    r.src = static_cast<const char*>(p.q.ptr) + (t * p.q.t_stride + h * p.q.h_stride) * elem_bytes(r.in);
    r.dst = static_cast<char*>(p.q_out) + (t * p.qo_t + h * p.qo_h) * elem_bytes(r.out);
    r.rotated = true;
    return r;
  }
  h -= p.hq;
  const bool is_k = h < p.hkv;
  if (!is_k) h -= p.hkv;
  const HeadView& x = is_k ? p.k : p.v;
  const PageView& c = is_k ? p.kc : p.vc;
  r.in = KV == kAny ? p.kv_kind : KV;
  r.out = CK == kAny ? p.c_kind : CK;
  r.src = static_cast<const char*>(x.ptr) + (t * x.t_stride + h * x.h_stride) * elem_bytes(r.in);
  const uint32_t page = (uint32_t)slot / (uint32_t)p.ps, row = (uint32_t)slot % (uint32_t)p.ps;
  r.dst = slot < 0 ? nullptr
                   : static_cast<char*>(c.ptr) + (page * c.page + row * c.row + h * c.head) * elem_bytes(r.out);
  r.rotated = is_k;
  return r;
}

// Aligned operands.  Units of a head: half/8 of pairs, then (D - 2 half)/16
// of unrotated elements.  Thread index: unit fastest, then head group, then
// token; group g walks heads g, g + groups, ...
template <int QK, int QO, int KV, int CK, int kBatch>
__global__ void __launch_bounds__(256) rope_vec_kernel(const __grid_constant__ RopeParams p, int units, int groups) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int u = (int)(id % units);
  const int64_t tg = id / units;
  const int g = (int)(tg % groups);
  const int64_t t = tg / groups;
  if (t >= p.T) return;
  const int pair_units = p.half >> 3;
  const bool tail = u >= pair_units;
  // the unit's two pieces of eight elements
  int e0, e1;
  if (tail)
    e0 = 2 * p.half + 16 * (u - pair_units), e1 = e0 + 8;
  else if (p.interleaved)
    e0 = 16 * u, e1 = e0 + 8;
  else
    e0 = 8 * u, e1 = p.half + 8 * u;
  int64_t slot = -1;
  if (p.hkv) {
    slot = __ldg(p.slots + t);
    if (slot >= p.num_slots) {
      record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedSlot));
      slot = -1;
    }
  }
  float c[8], s[8];
  if (!tail && p.half) {
    const int64_t n = p.pos64 ? __ldg(static_cast<const long long*>(p.positions) + t)
                              : (int64_t)__ldg(static_cast<const int*>(p.positions) + t);
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(p, n, 8 * u + i, c[i], s[i]);
  }
  const int heads = p.hq + 2 * p.hkv;
  for (int h0 = g; h0 < heads; h0 += groups * kBatch) {
    Place at[kBatch];
    Oct a[kBatch], b[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * groups;
      at[j].dst = nullptr;
      if (h < heads) at[j] = place<QK, QO, KV, CK>(p, t, h, slot);
      if (at[j].dst) {
        a[j] = load_oct(at[j].src + e0 * elem_bytes(at[j].in), at[j].in);
        b[j] = load_oct(at[j].src + e1 * elem_bytes(at[j].in), at[j].in);
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (!at[j].dst) continue;
      float x[8], y[8];
      unpack_oct(a[j], at[j].in, x);
      unpack_oct(b[j], at[j].in, y);
      if (!tail && at[j].rotated) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) rotate(x[2 * i], x[2 * i + 1], c[i], s[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) rotate(y[2 * i], y[2 * i + 1], c[4 + i], s[4 + i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) rotate(x[i], y[i], c[i], s[i]);
        }
      }
      store_oct(at[j].dst + e0 * elem_bytes(at[j].out), at[j].out, x);
      store_oct(at[j].dst + e1 * elem_bytes(at[j].out), at[j].out, y);
    }
  }
}

// Any alignment: units of one pair, then of one unrotated element.
__global__ void __launch_bounds__(256) rope_any_kernel(const __grid_constant__ RopeParams p, int units) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int u = (int)(id % units);
  const int64_t t = id / units;
  if (t >= p.T) return;
  const bool tail = u >= p.half;
  int e0, e1;
  if (tail)
    e0 = p.half + u, e1 = -1;
  else if (p.interleaved)
    e0 = 2 * u, e1 = e0 + 1;
  else
    e0 = u, e1 = p.half + u;
  int64_t slot = -1;
  if (p.hkv) {
    slot = __ldg(p.slots + t);
    if (slot >= p.num_slots) {
      record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedSlot));
      slot = -1;
    }
  }
  float c = 1.0f, s = 0.0f;
  if (!tail) {
    const int64_t n = p.pos64 ? __ldg(static_cast<const long long*>(p.positions) + t)
                              : (int64_t)__ldg(static_cast<const int*>(p.positions) + t);
    turn(p, n, u, c, s);
  }
  const int heads = p.hq + 2 * p.hkv;
  for (int h = 0; h < heads; ++h) {
    const Place at = place<kAny, kAny, kAny, kAny>(p, t, h, slot);
    if (!at.dst) continue;
    const int ie = elem_bytes(at.in), oe = elem_bytes(at.out);
    float x = load_one(at.src + e0 * ie, at.in), y = 0.0f;
    if (!tail) {
      y = load_one(at.src + e1 * ie, at.in);
      if (at.rotated) rotate(x, y, c, s);
    }
    store_one(at.dst + e0 * oe, at.out, x);
    if (!tail) store_one(at.dst + e1 * oe, at.out, y);
  }
}

template <int QK, int QO, int KV, int CK>
void launch_vec(const RopeParams& p, int num_sms, cudaStream_t stream) {
  const int units = p.half / 8 + (p.D - 2 * p.half) / 16, heads = p.hq + 2 * p.hkv;
  // Four heads a thread once that still leaves two full waves of threads,
  // else one (a latency-bound call wants every load in flight at once).
  const int64_t all = (int64_t)p.T * units * heads;
  const bool batch = all >= 4ll * 2 * num_sms * 2048;
  const int groups = batch ? (heads + 7) / 8 : heads;
  const unsigned grid = (unsigned)(((int64_t)p.T * units * groups + 255) / 256);
  if (batch)
    rope_vec_kernel<QK, QO, KV, CK, 4><<<grid, 256, 0, stream>>>(p, units, groups);
  else
    rope_vec_kernel<QK, QO, KV, CK, 1><<<grid, 256, 0, stream>>>(p, units, groups);
}

}  // namespace

bi_status launch_rope(const RopeParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  RopeParams q = p;
  q.status_word = dev.status_word;
  const int kq = p.hq ? p.q_kind : p.kv_kind, ko = p.hq ? p.qo_kind : p.c_kind;
  const int kk = p.hkv ? p.kv_kind : kq, kc = p.hkv ? p.c_kind : ko;
  if (!p.vec) {
    const int units = p.D - p.half;
    const int64_t grid = ((int64_t)p.T * units + 255) / 256;
    rope_any_kernel<<<(unsigned)grid, 256, 0, stream>>>(q, units);
  } else if (kq == 0 && ko == 0 && kk == 0 && kc == 0) {
    launch_vec<0, 0, 0, 0>(q, dev.num_sms, stream);
  } else if (kq == 1 && ko == 1 && kk == 1 && kc == 1) {
    launch_vec<1, 1, 1, 1>(q, dev.num_sms, stream);
  } else {
    launch_vec<kAny, kAny, kAny, kAny>(q, dev.num_sms, stream);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("rotary launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
