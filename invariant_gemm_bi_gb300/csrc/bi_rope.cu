// bi_rope.cu -- rotary positions, and the paged-cache write that goes with
// them: pair (x1, x2) of a head at position n is turned by n f_i,
//   y1 = a (x1 cos - x2 sin),  y2 = a (x1 sin + x2 cos),
// the transposed map (sin negated) being its gradient.
//
// Angles.  An fp32 product n * f_i loses the angle at far positions (at
// n = 10^6 it is off by up to 0.03 rad), and fp64 is slow on this chip.  The
// frequency is held as a 64-bit binary fraction of a turn, so the integer
// product phase * n mod 2^64 is the angle modulo one turn, off by at most
// n 2^-65 turns; signed, it is rounded to fp32 once and scales to half turns in
// [-1, 1], so sincospif needs no further reduction.  That rounding is relative:
// 2^-24 of the reduced angle, under 1.0e-7 rad, and a slow pair's small angle
// keeps all its digits (the top 32 bits alone would be off by 1.5e-9 rad, to
// one side, 7e-4 of an angle of 2e-6).  Positions n and -n are mirror images.
//
// Work.  A block takes a few tokens and all heads (a part of the heads when
// there are few tokens).  Its threads compute each sine and cosine of its
// tokens once, into shared memory, while the data are already on their way: a
// warp takes a head at a time, and a lane one unit of a token's head -- two
// pieces of eight elements, of the first and the second half of the rotated
// part (their 8 pairs in either layout) or of the unrotated tail -- so
// neighbouring lanes move neighbouring 16 bytes.  Each lane copies its units to
// places of its own in shared memory, six heads ahead, by asynchronous copies:
// no registers and no barrier, and its 8 sines and cosines stay in registers
// over its heads.  (8191 tokens of 32 + 8 + 8 heads of 128, 201 MB: loads into
// registers, eight heads a thread, 47 us; this way 38 us.  16383 tokens of 32
// heads, 268 MB: 52 and 40 us, 6.64 TB/s.  The 8191 are 2048 blocks, 3.37 waves
// of four an SM, each with the position's, then the slot's latency at its start.
// Types other than bf16 or fp16 throughout take rings twice as large, two
// blocks an SM: 8191 x 32 x 128 fp32 73 us, 1.8 times its bytes.)  Operands
// whose rows or split are not 16-byte aligned take units of one pair with the
// same arithmetic, so the bits do not depend on the layout; heads one after the
// other, 8191 x 32 x 96 bf16 with 24 rotated 77 us, 5.2 times its bytes.  The
// kernel reads and writes every element once: it is bound by memory bandwidth,
// small calls by one load's latency plus the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
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
// two elements, one conversion
__device__ __forceinline__ uint32_t f2_to_half2(float a, float b, int kind) {
  if (kind == 1) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ int elem_bytes(int kind) { return kind == 2 ? 4 : 2; }

// Eight consecutive elements from their raw words: 4 or 8 of them.
__device__ __forceinline__ void unpack_oct(const uint4& lo, const uint4& hi, int kind, float (&f)[8]) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = kind == 2 ? __uint_as_float(w[i]) : half_to_f((w[i >> 1] >> (16 * (i & 1))) & 0xffffu, kind);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void store_oct(void* p, int kind, const float (&f)[8]) {
  if (kind == 2) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f2_to_half2(f[2 * i], f[2 * i + 1], kind);
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
  sincospif(__fmul_rn(__ll2float_rn((long long)t), 1.0842021724855044e-19f /* 2^-63 */), &s, &c);
  c = __fmul_rn(c, p.magnitude);
  s = __fmul_rn(p.transpose ? -s : s, p.magnitude);
}
// One rotated pair: a product rounded, then one fused multiply-add.
__device__ __forceinline__ void rotate(float& x1, float& x2, float c, float s) {
  const float y1 = __fmaf_rn(x1, c, -__fmul_rn(x2, s));
  x2 = __fmaf_rn(x2, c, __fmul_rn(x1, s));
  x1 = y1;
}

// The cache slot of token t: negative when it is not stored.
__device__ __forceinline__ int64_t token_slot(const RopeParams& p, int64_t t) {
  int64_t slot = __ldg(p.slots + t);
  if (slot >= p.num_slots) {
    record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedSlot));
    slot = -1;
  }
  return slot;
}
__device__ __forceinline__ int64_t token_position(const RopeParams& p, int64_t t) {
  return p.pos64 ? __ldg(static_cast<const long long*>(p.positions) + t)
                 : (int64_t)__ldg(static_cast<const int*>(p.positions) + t);
}

// Element 0 of head 0 of a token in each operand; kd and vd are null for a
// token that is not stored.
struct TokenPlace {
  const char *q, *k, *v;
  char *qd, *kd, *vd;
};
__device__ __forceinline__ TokenPlace token_place(const RopeParams& p, int64_t t, int64_t slot) {
  TokenPlace a;
  a.q = static_cast<const char*>(p.q.ptr) + t * p.q.t_stride * elem_bytes(p.q_kind);
  a.qd = static_cast<char*>(p.q_out) + t * p.qo_t * elem_bytes(p.qo_kind);
  a.k = static_cast<const char*>(p.k.ptr) + t * p.k.t_stride * elem_bytes(p.kv_kind);
  a.v = static_cast<const char*>(p.v.ptr) + t * p.v.t_stride * elem_bytes(p.kv_kind);
  a.kd = a.vd = nullptr;
  if (slot >= 0) {
    const uint32_t page = (uint32_t)slot / (uint32_t)p.ps, row = (uint32_t)slot - page * (uint32_t)p.ps;
    a.kd = static_cast<char*>(p.kc.ptr) + (page * p.kc.page + row * p.kc.row) * elem_bytes(p.c_kind);
    a.vd = static_cast<char*>(p.vc.ptr) + (page * p.vc.page + row * p.vc.row) * elem_bytes(p.c_kind);
  }
  return a;
}
// Head slot h: q heads, then k heads, then v heads.
__device__ __forceinline__ const char* source(const RopeParams& p, const TokenPlace& a, int h, int kq, int kk) {
  if (h < p.hq) return a.q + h * p.q.h_stride * elem_bytes(kq);
  h -= p.hq;
  if (h < p.hkv) return a.k + h * p.k.h_stride * elem_bytes(kk);
  return a.v + (h - p.hkv) * p.v.h_stride * elem_bytes(kk);
}
// Where it is written; null for a token that is not stored.
__device__ __forceinline__ char* target(const RopeParams& p, const TokenPlace& a, int h, int ko, int kc) {
  if (h < p.hq) return a.qd + h * p.qo_h * elem_bytes(ko);
  h -= p.hq;
  if (h < p.hkv) return a.kd ? a.kd + h * p.kc.head * elem_bytes(kc) : nullptr;
  return a.vd ? a.vd + (h - p.hkv) * p.vc.head * elem_bytes(kc) : nullptr;
}

// Aligned operands.  A head has half/8 units of pairs and (D - 2 half)/16 of
// tail; block (x, y, z) takes tokens x * tokens .., heads y * heads .. and
// units z * 32 ...  kSlots: heads that a lane requests ahead.
constexpr int kMaxTokens = 32;
template <int QK, int QO, int KV, int CK, int kSlots>
__global__ void __launch_bounds__(256, QK == kAny ? 2 : 4)
    rope_vec_kernel(const __grid_constant__ RopeParams p, int units, int tokens, int heads) {
  constexpr int kPieces = QK == kAny ? 4 : 2;  // 16-byte pieces of a unit: fp32 has two an octet
  extern __shared__ __align__(16) unsigned char dyn[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kq = QK == kAny ? p.q_kind : QK, ko = QO == kAny ? p.qo_kind : QO;
  const int kk = KV == kAny ? p.kv_kind : KV, kc = CK == kAny ? p.c_kind : CK;
  const uint32_t mine = smem_u32(dyn) + tid * 16;
  float2* turns = reinterpret_cast<float2*>(dyn + kSlots * kPieces * 256 * 16);  // [tokens][half]
  const int in_block = min(units, 32);  // units of a token in this block
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int tok = lane / in_block, u = blockIdx.z * 32 + lane % in_block;
  const int64_t t = t0 + tok;
  const bool live = tok < tokens && t < p.T && u < units;
  const int pair_units = p.half >> 3;
  const bool tail = u >= pair_units;
  // the unit's two pieces of eight elements
  const int e0 = tail ? 2 * p.half + 8 * (u - pair_units) : 8 * u;
  const int e1 = e0 + (tail ? (p.D - 2 * p.half) / 2 : p.half);
  TokenPlace at = token_place(p, live ? t : t0, -1);
  const int h_end = min(p.hq + 2 * p.hkv, (int)(blockIdx.y + 1) * heads);
  auto request = [&](int h, int slot) {
    if (live && h < h_end) {
      const int kind = h < p.hq ? kq : kk;
      const char* x = source(p, at, h, kq, kk);
      const uint32_t dst = mine + slot * (kPieces * 256 * 16);
      copy16(dst, x + e0 * elem_bytes(kind));
      copy16(dst + 256 * 16, x + e1 * elem_bytes(kind));
      if (kPieces == 4 && kind == 2) {
        copy16(dst + 2 * 256 * 16, x + e0 * 4 + 16);
        copy16(dst + 3 * 256 * 16, x + e1 * 4 + 16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int h = blockIdx.y * heads + warp;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) request(h + 8 * i, i);
  // the sines and cosines of the block's tokens, and where its tokens go
  float c[8], s[8];
  if (p.half) {
    const int n = (int)min((int64_t)tokens, p.T - t0) * p.half;
    for (int i = tid; i < n; i += 256) {
      const int k = i / p.half, pair = i - k * p.half;
      turn(p, token_position(p, t0 + k), pair, turns[i].x, turns[i].y);
    }
    __syncthreads();
    if (live && !tail) {
      // half layout: pairs 8u ..; interleaved: those of the two pieces
      const float2* f = turns + tok * p.half + (p.interleaved ? 4 * u : 8 * u);
      const float2* f2 = p.interleaved ? f + p.half / 2 : f + 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = f[i].x, s[i] = f[i].y;
        c[4 + i] = f2[i].x, s[4 + i] = f2[i].y;
      }
    }
  }
  if (live && p.hkv) at = token_place(p, t, token_slot(p, t));
  int slot = 0;
  for (; h < h_end; h += 8) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    char* o = live ? target(p, at, h, ko, kc) : nullptr;
    if (o) {
      const int in = h < p.hq ? kq : kk, out = h < p.hq ? ko : kc;
      const uint32_t src = mine + slot * (kPieces * 256 * 16);
      float x[8], y[8];
      const uint4 none = make_uint4(0, 0, 0, 0);
      const bool wide = kPieces == 4 && in == 2;
      unpack_oct(ld_shared_v4(src), wide ? ld_shared_v4(src + 2 * 256 * 16) : none, in, x);
      unpack_oct(ld_shared_v4(src + 256 * 16), wide ? ld_shared_v4(src + 3 * 256 * 16) : none, in, y);
      if (!tail && h < p.hq + p.hkv && p.half) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            rotate(x[2 * i], x[2 * i + 1], c[i], s[i]);
            rotate(y[2 * i], y[2 * i + 1], c[4 + i], s[4 + i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) rotate(x[i], y[i], c[i], s[i]);
        }
      }
      store_oct(o + e0 * elem_bytes(out), out, x);
      store_oct(o + e1 * elem_bytes(out), out, y);
    }
    request(h + 8 * kSlots, slot);  // the slot just read, by this lane
    slot = slot + 1 == kSlots ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
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
  const TokenPlace at = token_place(p, t, p.hkv ? token_slot(p, t) : -1);
  float c = 1.0f, s = 0.0f;
  if (!tail) {
    turn(p, token_position(p, t), u, c, s);
  }
  const int heads = p.hq + 2 * p.hkv;
  for (int h = 0; h < heads; ++h) {
    char* o = target(p, at, h, p.qo_kind, p.c_kind);
    if (!o) continue;
    const char* i = source(p, at, h, p.q_kind, p.kv_kind);
    const int in = h < p.hq ? p.q_kind : p.kv_kind, out = h < p.hq ? p.qo_kind : p.c_kind;
    const int ie = elem_bytes(in), oe = elem_bytes(out);
    float x = load_one(i + e0 * ie, in), y = 0.0f;
    if (!tail) {
      y = load_one(i + e1 * ie, in);
      if (h < p.hq + p.hkv) rotate(x, y, c, s);
    }
    store_one(o + e0 * oe, out, x);
    if (!tail) store_one(o + e1 * oe, out, y);
  }
}

template <int QK, int QO, int KV, int CK>
cudaError_t launch_vec(const RopeParams& p, int num_sms, cudaStream_t stream) {
  const int units = p.half / 8 + (p.D - 2 * p.half) / 16, heads = p.hq + 2 * p.hkv;
  const int tokens = std::min(kMaxTokens, std::max(1, 32 / units));
  const int64_t blocks = ((int64_t)p.T + tokens - 1) / tokens;
  const unsigned z = (unsigned)((units + 31) / 32);
  const size_t turns = sizeof(float2) * tokens * p.half;
  constexpr size_t kSlot = (QK == kAny ? 4 : 2) * 256 * 16;
  // All heads a block, six a warp requested ahead, once that fills the GPU
  // twice; below, a head a warp (a latency-bound call wants every load in
  // flight at once).
  if (blocks * z >= 4 * (int64_t)num_sms || heads > 8 * 65535) {
    constexpr size_t kRing = 6 * kSlot;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(&rope_vec_kernel<QK, QO, KV, CK, 6>),
                                  (int)(kRing + sizeof(float2) * kMaxTokens * BI_ROPE_MAX_PAIRS), 56 + QK + 1);
    if (e != cudaSuccess) return e;
    rope_vec_kernel<QK, QO, KV, CK, 6>
        <<<dim3((unsigned)blocks, 1, z), 256, kRing + turns, stream>>>(p, units, tokens, heads);
  } else {
    const unsigned y = (unsigned)((heads + 7) / 8);
    rope_vec_kernel<QK, QO, KV, CK, 1><<<dim3((unsigned)blocks, y, z), 256, kSlot + turns, stream>>>(p, units, tokens, 8);
  }
  return cudaGetLastError();
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
  cudaError_t e;
  if (!p.vec) {
    const int units = p.D - p.half;
    const int64_t grid = ((int64_t)p.T * units + 255) / 256;
    rope_any_kernel<<<(unsigned)grid, 256, 0, stream>>>(q, units);
    e = cudaGetLastError();
  } else if (kq == 0 && ko == 0 && kk == 0 && kc == 0) {
    e = launch_vec<0, 0, 0, 0>(q, dev.num_sms, stream);
  } else if (kq == 1 && ko == 1 && kk == 1 && kc == 1) {
    e = launch_vec<1, 1, 1, 1>(q, dev.num_sms, stream);
  } else {
    e = launch_vec<kAny, kAny, kAny, kAny>(q, dev.num_sms, stream);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    *why = std::string("rotary launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
