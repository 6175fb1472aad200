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
// places of its own in shared memory, three heads ahead, by asynchronous copies:
// no registers and no barrier, and its 8 sines and cosines stay in registers
// over its heads.  (8191 tokens of 32 + 8 + 8 heads of 128, 201 MB: loads into
// registers, eight heads a thread, 47 us; this way 36 us, six heads ahead 38.
// 16383 tokens of 32 heads, 268 MB: 52 and 41 us, 6.5 TB/s.  The 8191 are 2048
// blocks, 3.37 waves of four an SM, each with the position's, then the slot's
// latency at its start.  Types other than bf16 or fp16 throughout take rings twice
// as large: 8191 x 32 x 128 fp32 60 us, 1.5 times its bytes; two blocks an SM and
// six heads ahead 73.)  Operands
// whose rows or split are not 16-byte aligned take units of one pair with the
// same arithmetic, so the bits do not depend on the layout; heads one after the
// other, 8191 x 32 x 96 bf16 with 24 rotated 77 us, 5.2 times its bytes.  The
// kernel reads and writes every element once: it is bound by memory bandwidth,
// small calls by one load's latency plus the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_e4m3.cuh"
#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
#include "bi_serve.h"

namespace bi {
namespace {

constexpr int kAny = -1;  // element kind read from the parameters
constexpr int kE4m3 = 3;  // a cache in 8 bits, with scales

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
__device__ __forceinline__ int elem_bytes(int kind) { return kind == 2 ? 4 : kind == kE4m3 ? 1 : 2; }

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

// Sine and cosine of t 2^-64 turns, off by at most 0.71 and 0.62 of a last place.
// The nearest whole number of quarter turns is taken off in integers; what is left,
// theta in [-pi/4, pi/4], is the sum of two fp32, and the polynomials (the series to
// theta^9 and theta^10, whose next terms are below 2^-28 of the result) only give what
// is added, in the one last rounding, to theta or to 1 - theta^2 / 2:
//   sin = h + (l (1 - z/2) + h z S(z)),   cos = (1 - z/2) + (z^2 C(z) - h l),   z = h^2,
// with what 1 - z/2 and z leave out.  (Of 3 million results one in 65 is not the
// nearest fp32.)
__device__ __forceinline__ void sine_cosine(int64_t t, float& s, float& c) {
  const uint64_t quarters = ((uint64_t)t + (1ull << 61)) >> 62;
  const int64_t r = (int64_t)((uint64_t)t - (quarters << 62));
  const float a = __ll2float_rn(r), rest = __ll2float_rn(r - __float2ll_rz(a));
  constexpr float kUnit = 3.4061215800865545e-19f;  // 2 pi 2^-64, and what fp32 leaves out
  constexpr float kUnitLow = (float)(3.4061215800865545e-19 - (double)kUnit);
  const float h = __fmul_rn(a, kUnit);
  const float l = __fmaf_rn(rest, kUnit, __fmaf_rn(a, kUnitLow, __fmaf_rn(a, kUnit, -h)));
  const float z = __fmul_rn(h, h), half = __fmul_rn(0.5f, z);
  float u = __fmaf_rn(z, 1.0f / 362880, -1.0f / 5040);
  u = __fmaf_rn(z, u, 1.0f / 120);
  u = __fmaf_rn(z, u, -1.0f / 6);
  const float sine = __fadd_rn(h, __fmaf_rn(__fmul_rn(h, z), u, __fmaf_rn(l, -half, l)));
  float v = __fmaf_rn(z, -1.0f / 3628800, 1.0f / 40320);
  v = __fmaf_rn(z, v, -1.0f / 720);
  v = __fmaf_rn(z, v, 1.0f / 24);
  const float w = __fsub_rn(1.0f, half);
  float d = __fmaf_rn(__fmul_rn(z, z), v, __fsub_rn(__fsub_rn(1.0f, w), half));
  d = __fmaf_rn(h, -l, d);
  d = __fmaf_rn(-0.5f, __fmaf_rn(h, h, -z), d);
  const float cosine = __fadd_rn(w, d);
  s = quarters & 1 ? cosine : sine;
  c = quarters & 1 ? sine : cosine;
  if (quarters & 2) s = -s;
  if ((quarters + 1) & 2) c = -c;
}

// a cos and a sin of position n's angle for pair i.  FINE (caches in 8 bits): by
// sine_cosine.  An element next to a border of two e4m3 numbers is put on one side or
// the other, a sixteenth of it apart, by errors of any size: sines of the angle
// rounded to fp32, off by a last place or two, put two to four times as many on the
// wrong side as sines rounded once.
template <bool FINE = false>
__device__ __forceinline__ void turn(const RopeParams& p, int64_t n, int i, float& c, float& s) {
  const uint64_t t = p.phase[i] * (uint64_t)n;
  if constexpr (FINE)
    sine_cosine((int64_t)t, s, c);
  else
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
  float *ks, *vs;  // scales of a cache in 8 bits
};
__device__ __forceinline__ TokenPlace token_place(const RopeParams& p, int64_t t, int64_t slot) {
  TokenPlace a;
  a.q = static_cast<const char*>(p.q.ptr) + t * p.q.t_stride * elem_bytes(p.q_kind);
  a.qd = static_cast<char*>(p.q_out) + t * p.qo_t * elem_bytes(p.qo_kind);
  a.k = static_cast<const char*>(p.k.ptr) + t * p.k.t_stride * elem_bytes(p.kv_kind);
  a.v = static_cast<const char*>(p.v.ptr) + t * p.v.t_stride * elem_bytes(p.kv_kind);
  a.kd = a.vd = nullptr;
  a.ks = a.vs = nullptr;
  if (slot >= 0) {
    const uint32_t page = (uint32_t)slot / (uint32_t)p.ps, row = (uint32_t)slot - page * (uint32_t)p.ps;
    a.kd = static_cast<char*>(p.kc.ptr) + (page * p.kc.page + row * p.kc.row) * elem_bytes(p.c_kind);
    a.vd = static_cast<char*>(p.vc.ptr) + (page * p.vc.page + row * p.vc.row) * elem_bytes(p.c_kind);
    if (p.ks.ptr) {
      a.ks = static_cast<float*>(p.ks.ptr) + page * p.ks.page + row * p.ks.row;
      a.vs = static_cast<float*>(p.vs.ptr) + page * p.vs.page + row * p.vs.row;
    }
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

// A cache in 8 bits.  The size of a head, from which its scale follows, is the
// largest |a| (|x1| + |x2|) of its rotated pairs and |x| of its other elements:
// no angle takes an element past it, so a key's scale does not depend on its
// position, is known before the angles are, and is the same from one sum of two
// numbers a pair whatever computes it (the largest rotated element, rounded one
// way or the other next to 448 2^e, would decide a whole head's scale).  It is
// up to twice the largest element: at most one binade at the small end.
//
// Measured: 8191 tokens of 32 + 8 + 8 heads of 128, bf16, 185 MB, 40.8 us, 4.5 TB/s: by
// issue (57 %, 285 instructions a warp and unit) and by waves (2048 blocks are 3.37
// of 608); fp32 85 us (105 with two blocks an SM); 64 tokens 3.8 us.  Six heads ahead
// 44.8 us, two 41.6; half the heads a block 51.6 (each block has its sines to compute).
// These instances spill 28 to 52 bytes at 64 registers, the 16-bit ones none.
__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t pair_size(float x1, float x2, float magnitude) {
  return size_bits(__fmul_rn(__fadd_rn(fabsf(x1), fabsf(x2)), magnitude));
}
__device__ __forceinline__ uint2 quantize_oct(const float (&x)[8], float inv) {
  return make_uint2(to_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                    to_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}
__device__ __forceinline__ float* scale_target(const RopeParams& p, const TokenPlace& a, int h) {
  h -= p.hq;
  return h < p.hkv ? a.ks + h * p.ks.head : a.vs + (h - p.hkv) * p.vs.head;
}

// Aligned operands.  A head has half/8 units of pairs and (D - 2 half)/16 of
// tail; block (x, y, z) takes tokens x * tokens .., heads y * heads .. and
// units z * 32 ...  kSlots: heads that a lane requests ahead.
constexpr int kMaxTokens = 32;
template <int QK, int QO, int KV, int CK, int kSlots>
__global__ void __launch_bounds__(256, 4)
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
      turn<CK == kE4m3>(p, token_position(p, t0 + k), pair, turns[i].x, turns[i].y);
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
  const float mag = fabsf(p.magnitude);
  int slot = 0;
  for (; h < h_end; h += 8) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    char* o = live ? target(p, at, h, ko, kc) : nullptr;
    uint32_t size = 0;  // of the unit's part of a cached head
    float x[8], y[8];
    if (o) {
      const int in = h < p.hq ? kq : kk, out = h < p.hq ? ko : kc;
      const uint32_t src = mine + slot * (kPieces * 256 * 16);
      const uint4 none = make_uint4(0, 0, 0, 0);
      const bool wide = kPieces == 4 && in == 2;
      unpack_oct(ld_shared_v4(src), wide ? ld_shared_v4(src + 2 * 256 * 16) : none, in, x);
      unpack_oct(ld_shared_v4(src + 256 * 16), wide ? ld_shared_v4(src + 3 * 256 * 16) : none, in, y);
      if constexpr (CK == kE4m3) {
        if (h >= p.hq) {
          if (tail || h >= p.hq + p.hkv || !p.half) {
#pragma unroll
            for (int i = 0; i < 8; ++i) size = max(size, max(size_bits(x[i]), size_bits(y[i])));
          } else if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              size = max(size, max(pair_size(x[i], x[i + 1], mag), pair_size(y[i], y[i + 1], mag)));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) size = max(size, pair_size(x[i], y[i], mag));
          }
        }
      }
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
      if (CK != kE4m3 || h < p.hq) {
        store_oct(o + e0 * elem_bytes(out), out, x);
        store_oct(o + e1 * elem_bytes(out), out, y);
      }
    }
    if constexpr (CK == kE4m3) {
      if (h >= p.hq) {  // the units of a head are neighbouring lanes, a power of two of them
        for (int d = units >> 1; d > 0; d >>= 1) size = max(size, __shfl_xor_sync(0xffffffffu, size, d));
        if (o) {
          const float scale = block_scale(size), inv = inverse_scale(scale);
          *reinterpret_cast<uint2*>(o + e0) = quantize_oct(x, inv);
          *reinterpret_cast<uint2*>(o + e1) = quantize_oct(y, inv);
          if (u == 0) *scale_target(p, at, h) = scale;
        }
      }
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

// A cache in 8 bits at any alignment and head dimension: a warp a token's head,
// which it reads twice, for the size and for the values.
__global__ void __launch_bounds__(256) rope_quantize_any_kernel(const __grid_constant__ RopeParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, heads = p.hq + 2 * p.hkv;
  const float mag = fabsf(p.magnitude);
  const int64_t all = (int64_t)p.T * heads;
  for (int64_t id = (int64_t)blockIdx.x * 8 + warp; id < all; id += (int64_t)gridDim.x * 8) {
    const int64_t t = id / heads;
    const int h = (int)(id - t * heads);
    const TokenPlace at = token_place(p, t, token_slot(p, t));
    char* o = target(p, at, h, p.qo_kind, kE4m3);
    if (!o) continue;
    const char* src = source(p, at, h, p.q_kind, p.kv_kind);
    const bool query = h < p.hq, turned = h < p.hq + p.hkv;
    const int in = query ? p.q_kind : p.kv_kind, ie = elem_bytes(in);
    const int half = turned ? p.half : 0, units = p.D - half;  // pairs, then single elements
    auto places = [&](int u, int& e0, int& e1) {
      if (u >= half)
        e0 = half + u, e1 = -1;
      else if (p.interleaved)
        e0 = 2 * u, e1 = e0 + 1;
      else
        e0 = u, e1 = half + u;
    };
    float scale = 1.0f;
    if (!query) {
      uint32_t size = 0;
      for (int u = lane; u < units; u += 32) {
        int e0, e1;
        places(u, e0, e1);
        const float x = load_one(src + e0 * ie, in);
        size = max(size, e1 < 0 ? size_bits(x) : pair_size(x, load_one(src + e1 * ie, in), mag));
      }
      scale = block_scale(__reduce_max_sync(0xffffffffu, size));
      if (lane == 0) *scale_target(p, at, h) = scale;
    }
    const float inv = inverse_scale(scale);
    const int64_t n = half ? token_position(p, t) : 0;
    for (int u = lane; u < units; u += 32) {
      int e0, e1;
      places(u, e0, e1);
      float x = load_one(src + e0 * ie, in), y = 0.0f;
      if (e1 >= 0) {
        float c, s;
        turn<true>(p, n, u, c, s);
        y = load_one(src + e1 * ie, in);
        rotate(x, y, c, s);
      }
      if (query) {
        const int oe = elem_bytes(p.qo_kind);
        store_one(o + e0 * oe, p.qo_kind, x);
        if (e1 >= 0) store_one(o + e1 * oe, p.qo_kind, y);
      } else {
        const uint32_t b = to_e4m3x2(x * inv, y * inv);
        o[e0] = (char)b;
        if (e1 >= 0) o[e1] = (char)(b >> 8);
      }
    }
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
  // All heads a block, three a warp requested ahead, once that fills the GPU
  // twice; below, a head a warp (a latency-bound call wants every load in
  // flight at once).
  if (blocks * z >= 4 * (int64_t)num_sms || heads > 8 * 65535) {
    constexpr size_t kRing = 3 * kSlot;
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(&rope_vec_kernel<QK, QO, KV, CK, 3>),
                                  (int)(kRing + sizeof(float2) * kMaxTokens * BI_ROPE_MAX_PAIRS),
                                  (CK == kE4m3 ? 96 : 56) + QK + 1);
    if (e != cudaSuccess) return e;
    rope_vec_kernel<QK, QO, KV, CK, 3>
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
  if (kc == kE4m3) {
    if (!p.vec) {
      const int64_t warps = (int64_t)p.T * (p.hq + 2 * p.hkv);
      rope_quantize_any_kernel<<<(unsigned)std::min<int64_t>((warps + 7) / 8, 1 << 20), 256, 0, stream>>>(q);
      e = cudaGetLastError();
    } else if (kq == 0 && (ko == 0 || !p.hq) && kk == 0) {
      e = launch_vec<0, 0, 0, kE4m3>(q, dev.num_sms, stream);
    } else if (kq == 1 && (ko == 1 || !p.hq) && kk == 1) {
      e = launch_vec<1, 1, 1, kE4m3>(q, dev.num_sms, stream);
    } else {
      e = launch_vec<kAny, kAny, kAny, kE4m3>(q, dev.num_sms, stream);
    }
  } else if (!p.vec) {
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
