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
// Tile.  The warps of a CTA take tiles of 32 keys (16 at D = 256) of the unit
// in turn and never wait for one another before its end.  Both products run on
// mma.sync m16n8k16 with the long side on M: S^T = K Q^T (16 keys x 8 heads)
// and O^T += V^T P^T (16 dimensions x 8 heads).  With one token a head there
// are at most G rows to a product, which a 128-row tcgen05 tile would waste
// 15/16 of, and the tensor pipe is a sixth busy as it is.
//
// Feeding it.  Each warp owns a ring of three shared-memory slots, keys and
// values of a tile taking one each, filled by 16-byte asynchronous copies: two
// slots are always in flight while the third is worked on (128 KB an SM), the
// pages of a tile are looked up one tile before its copies are issued, and the
// pipeline runs on from unit to unit.  The order of the head dimension inside
// a dot product is free, so keys need no layout: lane (g, c) = (lane / 4,
// lane % 4) copies chunks of 8 dimensions c, c + 4, ... of keys g, g + 8, ...
// (64 contiguous bytes a key and instruction) to places of its own and reads
// them back as the fragments they are.  Values are wanted as V^T, pairs of
// neighbouring keys at one dimension: rows with their chunks permuted by the
// key, read by transposing ldmatrix.  P^T's fragment is S^T's transposed in
// 8 x 8 blocks (movmatrix).
//
// Steps, measured on 64 requests of 0 .. 8192 keys, 32 heads over 8, D = 128
// (956 MB; 141 us at the copy rate of 6.79 TB/s): fragments loaded straight
// into registers, 16 warps an SM, 250 us (each unit's first loads exposed);
// shared-memory rings across units, 16-key tiles, 204 us (bound by issue, 512
// instructions a tile and warp); 32-key tiles with transposing reads 164 us,
// longer pieces 160 us, 5.97 TB/s, near the memory's rate (161 with p in three
// pieces, below).
//
// Caches in 8 bits (template kCache8): half the bytes and the same work a key, so
// that issue weighs twice as much.  A slot is a tile of keys of D bytes, three of
// them a warp, 12 warps an SM at D = 128; chunks of 16 dimensions are read back and
// brought to fp16 in registers, two e4m3 a conversion, for the same mma.sync; values
// are read by transposing pairs of dimensions and sorted by byte permutes.  The batch
// above, 493 MB: 109 us, 4.5 TB/s (72.7 us at the copy rate; 40 x 8192 keys 144 us,
// 4.8 TB/s): 127 of those 144 us are the copies alone, 128 bytes a key and head, and
// the join and the launch take 8; issue is 51 % busy, tensor pipes 20 %.  16 warps an
// SM of 16-key tiles 139 us, 8 warps with six slots 133, four slots 123, tiles of 64
// keys 129 (the kept one 120 at that time), one running maximum for weights and sums
// in place of two 115.
//
// Arithmetic, per query head: t = RN(s c) with c = RN(scale log2 e); a running
// maximum m per warp over its tiles; p = 2^(t - m) (the SFU's approximation);
// l sums the unrounded p in fp32; the value product takes p in the cache's
// 16-bit type, the tensor core's operand type, as a sum of such numbers: three
// of bf16 (24 bits) or two of fp16 (22 bits).  One alone, rounded, would be off
// as much as a 16-bit result's own rounding; two of bf16 turn the rounding of
// one result in 500 (against an fp32 evaluation; three: one in 2000).  A piece
// more costs 0.2 % (160.1 us and 160.5 for the batch above; the request of 1021
// keys 6.9 us and 7.1).  A result of 16 bits is the fp32 result rounded once.
// fp16 ends at 2^-24, so there p is carried times 2^15 (and the final division
// takes it off): a weight is then cut at 2^-40 of the largest beside it and not
// at 2^-25, where a long cache's many small ones would be missing in O and yet
// counted in l.  O in fp32: n 2^15 times the largest value at most, 2^61.
// Warps are joined in a fixed tree, pieces in fixed groups in piece order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_e4m3.cuh"
#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
#include "bi_serve.h"

namespace bi {
namespace {

// A piece has 256 keys up to 2048, a cluster's worth of them: 512 would leave a
// short cache to few SMs (one request of 1021 keys, then joined by a second
// launch, 12.3 us against 9.9).  Longer requests have at least 512: fewer
// results to hand over and to join (the batch above 160 us against 164, 32 x
// 4096 keys of 16 ungrouped heads 96 against 98, one request of 4096 keys, all
// in a cluster then, 10.5 against 11.4; one of 8192 is left to fewer SMs, 14.0
// against 12.8).  At most 128 pieces: 256 made 131071 keys at D = 256 wait
// longer for the join than the evener split saved (97.7 us against 97.1).  In 8
// bits what a unit costs beside its keys (820 instructions a warp; 90 a tile of 32
// keys at four tiles a unit) weighs twice as much, and pieces of long requests have
// at least 1024; yet short ones make the units of a batch evener.  The length from
// which on they do, 4096, 8192, 16384 or 32768, by 28 batches of 1 to 128 requests of
// 4096 to 65536 keys, alike or ragged, D = 64, 128 and 256, groups of 1 to 16: on
// average 2.6, 5.1, 2.6 and 2.3 % above each batch's best, at worst 17, 20, 15 and 8 %.
// (us, by the length: 64 ragged up to 8192 keys 129, 120, 120, 121; 40 x 8192 137, 144,
// 143, 143; 24 ragged up to 24000 136, 148, 140, 142; 30 x 10000 137, 136, 141, 141; 64
// ragged up to 30000, 8 heads over 2, 115, 115, 125, 121; 32 ragged up to 12000 at D =
// 256 115, 135, 113, 113.)
constexpr int kMinSplit = 256;
constexpr int kMaxCluster = 8;
constexpr int kManySplits = 128;
constexpr int kLongPieces = 64 * kMinSplit;

__host__ __device__ inline int32_t paged_split_len(int64_t len, bool e4m3) {
  int64_t s = len <= kMaxCluster * kMinSplit ? kMinSplit : (e4m3 && len > kLongPieces ? 4 : 2) * kMinSplit;
  while (len > kManySplits * s) s *= 2;
  return (int32_t)s;
}
__host__ __device__ inline int32_t split_count(int64_t len, bool e4m3) {
  const int32_t s = paged_split_len(len, e4m3);
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
// Kinds of cache: bf16 and fp16 as q, or e4m3 with scales.
constexpr int kCache16 = 1, kCache8 = 2;  // fp16, e4m3
// What a weight is multiplied by before it is cut into 16-bit numbers, and what
// takes it off the joined result.  (In 8 bits weights go up to 2.)
template <int C>
struct Up {
  static constexpr float v = C == kCache8 ? 16384.0f : C == kCache16 ? 32768.0f : 1.0f;
  static constexpr float back = 1.0f / v;
};
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
__device__ __forceinline__ void store_one(void* o, int kind, int64_t i, float v) {
  if (kind == 2)
    static_cast<float*>(o)[i] = v;
  else if (kind == 1)
    static_cast<__half*>(o)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(v);
}
// Keys of request b: its length, at most what its table row can name.
__device__ __forceinline__ int request_len(const PagedAttnParams& p, int b) {
  const int n = __ldg(p.lens + b);
  if (n > p.cap) record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedPage));
  return max(0, min(n, p.cap));
}

// Units of a CTA, held by the lanes of a warp 32 at a time: lane i knows unit
// base + i.
struct Window {
  int64_t base;
  int b, hk, piece, len;  // request, head tile, piece, the request's keys
};
struct Unit {
  int b, hk, piece, len, k0, k1;
};

template <int C, int D, int NT>
struct Shape {
  static constexpr int HT = 8 * NT;                          // query heads of a unit

  static constexpr bool kBig = C != kCache8 && (D == 256 || (D == 128 && NT == 2));
  static constexpr int W = kBig ? 8 : 4;                     // warps of a CTA
  static constexpr int kCtas = C == kCache8 ? (D == 64 && NT == 1 ? 4 : NT == 1 && D == 128 ? 3 : 2)
                               : kBig       ? 1
                                            : (D == 64 ? (NT == 1 ? 4 : 3) : 2);  // CTAs of an SM
  static constexpr int E = C == kCache8 ? 1 : 2;             // bytes of an element
  static constexpr int KT = D == 256 ? 1 : 2;                // 16-key groups of a tile
  static constexpr int kTile = 16 * KT;                      // keys of a tile
  static constexpr int kStep = W * kTile;
  static constexpr int KJ = D * E / 64;                      // 16-byte chunks of a lane in a key row
  static constexpr int kSlotBytes = kTile * D * E;           // a tile's keys, or its values
  static constexpr int kRow = D + 4;                         // padded row of the join: no bank conflicts
  struct Shared {
    unsigned char ring[W][3][kSlotBytes];
    float o[W / 2][HT][kRow];
    float m[W / 2][HT], l[W / 2][HT];
    int32_t start[32 * W + 1];  // pieces of the requests before thread i's
    int32_t warp_sum[W];
  };
};

// 16 bytes from global to shared memory, or 16 zero bytes; read once: not kept in L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 read_chunk(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// Four 8 x 8 blocks of 16-bit values, each transposed on the way.
__device__ __forceinline__ uint4 read_transposed(uint32_t a) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
// A load that stays where it is written, a tile before its use.
__device__ __forceinline__ float load_now(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void barrier_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}
// The join's barriers: upper warps' results written; the rest's written; all read.
constexpr uint32_t kBarUpper = 1, kBarLower = 2, kBarRead = 3;

// ONE: a cluster has one (request, head tile), a CTA each of its pieces, and
// joins them itself.
template <int C, int D, int NT, bool ONE>
__global__ void __launch_bounds__(32 * Shape<C, D, NT>::W, Shape<C, D, NT>::kCtas)
    paged_attn_kernel(const PagedAttnParams p) {
  using Sh = Shape<C, D, NT>;
  constexpr int HT = Sh::HT;
  constexpr bool Q8 = C == kCache8;
  constexpr int F16 = C != 0;  // the tensor cores' operand type
  extern __shared__ __align__(1024) unsigned char dyn[];
  typename Sh::Shared& sm = *reinterpret_cast<typename Sh::Shared*>(dyn);
  constexpr int W = Sh::W, H = W / 2, kThreads = 32 * W, KT = Sh::KT, KJ = Sh::KJ, MT = D / 16;
  constexpr int PS = F16 ? 2 : 3;  // 16-bit pieces of p in the value product
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;

  const int inner = p.Hkv * p.head_tiles;
  const int per = (p.B + kThreads - 1) / kThreads;
  int64_t all = 0, units = 1;  // units of the grid and of this CTA
  if constexpr (!ONE) {
    // pieces before each thread's requests
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int n = 0;
    for (int b = b0; b < b1; ++b) n += split_count(request_len(p, b), Q8);
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
    all = (int64_t)sm.start[kThreads] * inner;
    // this CTA's: blockIdx.x, blockIdx.x + gridDim.x, ...
    units = all > blockIdx.x ? (all - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    if (units == 0) return;
  }

  // The CTA's i-th unit; `w` is refilled, a unit a lane, when i leaves it.
  auto unit_at = [&](int64_t i, Window& w) {
    Unit u;
    if constexpr (ONE) {
      const int id = (int)blockIdx.x / p.max_splits;
      u.b = id / inner, u.hk = id - u.b * inner, u.piece = (int)blockIdx.x % p.max_splits;
      u.len = request_len(p, u.b);
      const int n = paged_split_len(u.len, Q8);
      u.k0 = u.piece * n, u.k1 = min(u.len, u.k0 + n);  // below k0 for a piece that the request has not
      return u;
    }
    if (i >= w.base + 32) {
      w.base = i;
      const int64_t id = blockIdx.x + (i + lane) * gridDim.x;
      w.b = w.hk = w.piece = w.len = 0;
      if (id < all) {
        const int ss = (int)(id / inner);
        w.hk = (int)(id - (int64_t)ss * inner);
        int lo = 0, hi = min(kThreads, (p.B + per - 1) / per);
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (sm.start[mid] <= ss)
            lo = mid;
          else
            hi = mid;
        }
        int at = sm.start[lo];
        w.b = lo * per;
        w.len = request_len(p, w.b);
        while (ss >= at + split_count(w.len, Q8)) at += split_count(w.len, Q8), w.len = request_len(p, ++w.b);
        w.piece = ss - at;
      }
      __syncwarp();
    }
    const int src = (int)(i - w.base);
    u.b = __shfl_sync(0xffffffffu, w.b, src);
    u.hk = __shfl_sync(0xffffffffu, w.hk, src);
    u.piece = __shfl_sync(0xffffffffu, w.piece, src);
    u.len = __shfl_sync(0xffffffffu, w.len, src);
    const int n = paged_split_len(u.len, Q8);
    u.k0 = u.piece * n, u.k1 = min(u.len, u.k0 + n);
    return u;
  };

  // Producer: requests the tile after the one worked on, across units; the
  // tile's page numbers are looked up one tile earlier still.
  Window pw = {-64, 0, 0, 0, 0}, cw = {-64, 0, 0, 0, 0};
  int64_t pi = -1;               // the unit of the tile to request next
  int pkey = 0, pend = 0;        // its first key, and the unit's last
  const int32_t* ptab = nullptr; // the request's page table row
  const unsigned char *kb = nullptr, *vb = nullptr;  // the unit's head, at this lane's chunk
  const float *ksb = nullptr, *vsb = nullptr;        // and its scales
  int page = -1, row = 0;        // of key pkey + lane % kTile; page -1: none
  auto advance = [&]() {         // to the warp's next tile
    pkey += Sh::kStep;
    while (pi < units && pkey >= pend) {
      if (++pi >= units) break;
      const Unit u = unit_at(pi, pw);
      const int kvh = u.hk / p.head_tiles;
      pkey = u.k0 + warp * Sh::kTile, pend = u.k1;
      ptab = p.table + u.b * p.ld_table;
      kb = static_cast<const unsigned char*>(p.k) + kvh * p.k_head * Sh::E + 16 * (Q8 ? lane % (D / 16) : c);
      vb = static_cast<const unsigned char*>(p.v) + kvh * p.v_head * Sh::E + 16 * (Q8 ? lane % (D / 16) : c);
      if constexpr (Q8) {
        ksb = static_cast<const float*>(p.ks.ptr) + kvh * p.ks.head;
        vsb = static_cast<const float*>(p.vs.ptr) + kvh * p.vs.head;
      }
    }
    page = -1;
    const int j = pkey + (lane & (Sh::kTile - 1));
    if (pi < units && j < pend) {
      const uint32_t col = p.ps_shift >= 0 ? (uint32_t)j >> p.ps_shift : (uint32_t)j / (uint32_t)p.ps;
      row = (int)((uint32_t)j - col * (uint32_t)p.ps);
      page = __ldg(ptab + col);
      if (page < 0) page = -2;
    }
  };
  const uint32_t ring = smem_u32(sm.ring[warp][0]);
  uint32_t live_next = 0;  // mask of the requested tile's keys
  int64_t vo = 0;          // byte offset of the lane's key in the value cache
  float ks_next = 0.0f, vs_next = 0.0f;  // in 8 bits: its scales
  // In 8 bits a key's row goes to as many lanes as it has chunks, whole lines of
  // memory to a request; where it lands is the same.
  constexpr int kRowLanes = Q8 ? D / 16 : 4, kRowKeys = 32 / kRowLanes;
  [[maybe_unused]] const int chunk = lane % kRowLanes, rkey = lane / kRowLanes;
  // Keys: lane (g, c) takes chunks c, c + 4, ... of keys g, g + 8, ... to a place of its own.
  auto request_keys = [&](int slot) {
    const bool there = page >= 0 && page < p.P;
    if (!there && page != -1) record_failure(p.status_word, status_code(BI_ERR_INVALID_ARG, kSitePagedPage));
    live_next = __ballot_sync(0xffffffffu, there);
    const int64_t ko = there ? (page * p.k_page + row * p.k_row) * Sh::E : 0;
    vo = there ? (page * p.v_page + row * p.v_row) * Sh::E : 0;
    if constexpr (Q8) {
      ks_next = vs_next = 0.0f;
      if (there) {
        ks_next = load_now(ksb + page * p.ks.page + row * p.ks.row);
        vs_next = load_now(vsb + page * p.vs.page + row * p.vs.row);
      }
    }
    if (pi < units) {
      if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < Sh::kTile / kRowKeys; ++i) {
          const int key = kRowKeys * i + rkey;
          const unsigned char* a = kb + __shfl_sync(0xffffffffu, ko, key);
          copy16(ring + slot * Sh::kSlotBytes + (((key >> 3) * KJ + (chunk >> 2)) * 32 + (key & 7) * 4 + (chunk & 3)) * 16, a,
                 (live_next >> key) & 1);
        }
      } else {
        uint32_t dst = ring + slot * Sh::kSlotBytes + lane * 16;
#pragma unroll
        for (int r = 0; r < 2 * KT; ++r) {
          const unsigned char* a = kb + __shfl_sync(0xffffffffu, ko, 8 * r + g);
          const bool ok = (live_next >> (8 * r + g)) & 1;
#pragma unroll
          for (int j = 0; j < KJ; ++j, dst += 512) copy16(dst, a + 64 * j, ok);
        }
      }
    }
    copies_commit();
  };
  // Values: the same chunks, to rows whose chunks are permuted by their key so
  // that the transposing reads of eight keys meet no bank twice.
  auto request_values = [&](int slot) {
    if (pi < units) {
      if constexpr (Q8) {
        // (rows of 64 bytes: two keys to a line of all banks, the chunk permuted by the pair)
#pragma unroll
        for (int i = 0; i < Sh::kTile / kRowKeys; ++i) {
          const int key = kRowKeys * i + rkey;
          const unsigned char* a = vb + __shfl_sync(0xffffffffu, vo, key);
          copy16(ring + slot * Sh::kSlotBytes + key * D + (chunk ^ (D == 64 ? (key >> 1) & 3 : key & 7)) * 16, a,
                 (live_next >> key) & 1);
        }
      } else {
        const uint32_t dst = ring + slot * Sh::kSlotBytes + g * (2 * D) + ((c ^ g) & 3) * 16 + (g >> 2) * 64;
#pragma unroll
        for (int r = 0; r < 2 * KT; ++r) {
          const unsigned char* a = vb + __shfl_sync(0xffffffffu, vo, 8 * r + g);
          const bool ok = (live_next >> (8 * r + g)) & 1;
#pragma unroll
          for (int j = 0; j < KJ; ++j) copy16((dst + r * 16 * D) ^ (j * 64), a + 64 * j, ok);
        }
      }
    }
    copies_commit();
  };
  // Q^T fragments: head g of tile n, dimensions 32 j + 8 c .. + 7; with caches in
  // 8 bits chunks of 16 dimensions, 64 (j / 2) + 16 c + 8 (j % 2) .. + 7
  constexpr int QJ = D / 32;
  uint4 q[NT][QJ], qn[NT][QJ];  // (qn, the next unit's, in 16 bits: 8 have 16 warps an SM to wait beside)
  float qs[NT][2];  // in 8 bits: a score's factor for heads 2c, 2c + 1
  auto load_queries = [&](const Unit& u, bool now) {
    const int kvh = u.hk / p.head_tiles, h0 = (u.hk - kvh * p.head_tiles) * HT;
    const unsigned short* qb =
        static_cast<const unsigned short*>(p.q) + u.b * p.q_b + (kvh * p.group + h0 + g) * p.q_h + (Q8 ? 16 : 8) * c;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < QJ; ++j) {
        const unsigned short* a = qb + 8 * n * p.q_h + (Q8 ? 64 * (j / 2) + 8 * (j % 2) : 32 * j);
        const bool there = h0 + 8 * n + g < p.group;
        if (Q8 && !now) {
          if (there && j % 2 == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
        } else {
          qn[n][j] = there ? __ldg(reinterpret_cast<const uint4*>(a)) : make_uint4(0, 0, 0, 0);
        }
      }
  };
  // With caches in 8 bits, whose numbers are fp16 to the tensor cores, so is q,
  // brought to a largest element of 2^13 .. 2^14 a head by a power of two: exact
  // but for elements below 2^-27 of the largest, which are off by 2^-39 of it at
  // most.  A head that holds a NaN or an infinity gets a NaN for its factor.
  auto take_queries = [&]() {
    if constexpr (!Q8) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < QJ; ++j) q[n][j] = qn[n][j];
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        auto both = [&](uint32_t w, float& lo, float& hi) {
          lo = p.in_f16 ? low16<1>(w) : low16<0>(w);
          hi = p.in_f16 ? high16<1>(w) : high16<0>(w);
        };
        // magnitudes of 16-bit numbers are ordered as their bits are, a NaN's above all
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < QJ; ++j) {
          const uint32_t w[4] = {qn[n][j].x, qn[n][j].y, qn[n][j].z, qn[n][j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) most = __vmaxu2(most, w[i] & 0x7fff7fffu);
        }
        most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
        most = max(most & 0xffffu, most >> 16);
        float lo, hi;
        both(most, lo, hi);
        const uint32_t top = __float_as_uint(lo);
        const int e = max(min((int)(top >> 23) - 127, 127), -100) - 13;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
        auto scaled = [&](uint32_t w) {
          float lo, hi;
          both(w, lo, hi);
          return pack16<1>(lo * down, hi * down);
        };
#pragma unroll
        for (int j = 0; j < QJ; ++j)
          q[n][j] = make_uint4(scaled(qn[n][j].x), scaled(qn[n][j].y), scaled(qn[n][j].z), scaled(qn[n][j].w));
        float f = __fmul_rn(__uint_as_float((uint32_t)(127 + e) << 23), p.score_log2);
        if (top >= 0x7f800000u) f = __uint_as_float(0x7fffffffu);
#pragma unroll
        for (int h = 0; h < 2; ++h) qs[n][h] = __shfl_sync(0xffffffffu, f, (2 * c + h) * 4);
      }
    }
  };
  // where this lane's row of a transposing read starts: blocks (keys 0-7, dims
  // 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15); the chunk is permuted by the key
  // (in 8 bits a transposed element is two dimensions of a key: blocks (keys 0-7,
  // dims 0-15), (8-15, 0-15), (0-7, 16-31), (8-15, 16-31))
  const uint32_t vrow = ((lane & 7) + ((lane >> (Q8 ? 3 : 4)) & 1) * 8) * (D * Sh::E);
  const uint32_t vchunk = (lane >> (Q8 ? 4 : 3)) & 1, vkey = Q8 && D == 64 ? (lane >> 1) & 3 : lane & 7;
  // the dimensions of the accumulators' rows g and g + 8 of 16-dimension block i
  auto dim = [&](int i, int x) { return Q8 ? 16 * i + 2 * g + x : 16 * i + 8 * x + g; };

  Unit u = unit_at(0, cw);
  load_queries(u, false);
  advance();
  request_keys(0);
  request_values(1);
  advance();
  int sk = 0;  // slot of the tile's keys; its values are in the slot after it
  for (int64_t ui = 0; ui < units; ++ui) {
    if constexpr (Q8) load_queries(u, true);
    take_queries();
    const Unit next = unit_at(min(ui + 1, units - 1), cw);
    load_queries(next, false);
    float o[MT][NT][4] = {};
    float m[NT][2], l[NT][2];  // (in 8 bits m is of t + log2 of a value's scale)
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.0f;
    for (int key = u.k0 + warp * Sh::kTile; key < u.k1; key += Sh::kStep) {
      const int sv = sk == 2 ? 0 : sk + 1, sn = sk == 0 ? 2 : sk - 1;
      copies_wait<1>();  // this tile's keys are here
      __syncwarp();      // and every lane is done with the last tile's values
      const uint32_t live = live_next;
      // in 8 bits: scales of keys 8 r + g, the values' as 2^vlog * vfrac; vsum = 2^-vlog
      float ks[2 * KT], vlog[2 * KT], vfrac[2 * KT], vsum[2 * KT];
      if constexpr (Q8) {
        // below 2^-96 (zero, and what is not a number) vfrac takes the rest: sums of up
        // to 2^30 keys stay in fp32; from 2^126 on, whose inverse fp32 has not, vfrac is
        // infinite
        const uint32_t bits = __float_as_uint(vs_next), e = (bits >> 23) & 255u;
        const bool plain = e >= 127 - 96 && e < 127 + 126;
        const float lg = plain ? (float)((int)e - 127) : (bits << 1) == 0 ? -20.0f : -96.0f;
        const float fr = plain ? __uint_as_float((bits & 0x807fffffu) | 0x3f800000u) : vs_next * 79228162514264337593543950336.0f;
#pragma unroll
        for (int r = 0; r < 2 * KT; ++r) {
          ks[r] = __shfl_sync(0xffffffffu, ks_next, 8 * r + g);
          vlog[r] = __shfl_sync(0xffffffffu, lg, 8 * r + g);
          vfrac[r] = __shfl_sync(0xffffffffu, fr, 8 * r + g);
          vsum[r] = ex2_approx(-vlog[r]);  // (a power of two: exact)
        }
      }
      request_keys(sn);
      // scores of keys g (elements 0, 1) and g + 8 (2, 3) for heads 2c, 2c + 1
      float s[KT][NT][4] = {};
      {
        const uint32_t src = ring + sk * Sh::kSlotBytes + lane * 16;
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const uint4 k0 = read_chunk(src + (2 * t * KJ + j) * 512), k1 = read_chunk(src + ((2 * t + 1) * KJ + j) * 512);
            if constexpr (!Q8) {
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16816<F16>(s[t][n], k0.x, k1.x, k0.y, k1.y, q[n][j].x, q[n][j].y);
                mma16816<F16>(s[t][n], k0.z, k1.z, k0.w, k1.w, q[n][j].z, q[n][j].w);
              }
            } else {
              auto step = [&](uint32_t w0, uint32_t w1, int h, bool upper) {  // four dimensions of a lane
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_half2s(w0, a0, a2);
                e4m3x4_to_half2s(w1, a1, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  const uint4& b = q[n][2 * j + h];
                  mma16816<F16>(s[t][n], a0, a1, a2, a3, upper ? b.z : b.x, upper ? b.w : b.y);
                }
              };
              step(k0.x, k1.x, 0, false), step(k0.y, k1.y, 0, true);
              step(k0.z, k1.z, 1, false), step(k0.w, k1.w, 1, true);
            }
          }
      }
      uint32_t pf[KT][NT][PS][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[t][n][e] = Q8 ? __fadd_rn(__fmul_rn(__fmul_rn(s[t][n][e], ks[2 * t + (e >> 1)]), qs[n][e & 1]), vlog[2 * t + (e >> 1)])
                            : __fmul_rn(s[t][n][e], p.score_log2);
        if (live != (Sh::kTile == 32 ? 0xffffffffu : live | 0xffffu)) {
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((live >> (16 * t + g + 8 * (e >> 1))) & 1)) s[t][n][e] = -INFINITY;
        }
        float mx[2] = {m[n][0], m[n][1]};
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e & 1] = fmaxf(mx[e & 1], s[t][n][e]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1)
#pragma unroll
          for (int h = 0; h < 2; ++h) mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], x));
        if (__any_sync(0xffffffffu, mx[0] != m[n][0] || mx[1] != m[n][1])) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float alpha = mx[h] == -INFINITY ? 0.0f : ex2_approx(m[n][h] - mx[h]);
            m[n][h] = mx[h];
            l[n][h] = __fmul_rn(l[n][h], alpha);
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][n][h] *= alpha, o[i][n][2 + h] *= alpha;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ref = mx[h] == -INFINITY ? 0.0f : mx[h];  // no key yet: every p is 0
          float sum = 0.0f;
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int e = h; e < 4; e += 2) {
              s[t][n][e] = ex2_approx(__fsub_rn(s[t][n][e], ref));
              if constexpr (Q8) {  // e^score for the sum, e^score times the value's scale for the product
                sum = __fmaf_rn(s[t][n][e], vsum[2 * t + (e >> 1)], sum);
                s[t][n][e] = __fmul_rn(s[t][n][e], vfrac[2 * t + (e >> 1)]);
              } else {
                sum += s[t][n][e];
              }
            }
          l[n][h] += sum;
        }
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int x = 0; x < PS; ++x) {
            float(&e)[4] = s[t][n];
            if (F16 && x == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] *= Up<C>::v;
            }
            const uint32_t lo = pack16<F16>(e[0], e[1]), hi = pack16<F16>(e[2], e[3]);
            pf[t][n][x][0] = transpose8x8(lo);
            pf[t][n][x][1] = transpose8x8(hi);
            if (x + 1 < PS) {
              e[0] -= low16<F16>(lo), e[1] -= high16<F16>(lo);
              e[2] -= low16<F16>(hi), e[3] -= high16<F16>(hi);
            }
          }
      }
      copies_wait<1>();  // this tile's values are here
      __syncwarp();      // for every lane, and every lane is done with its keys
      request_values(sk);
      advance();
      const uint32_t src = ring + sv * Sh::kSlotBytes + vrow;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; Q8 && i < MT; i += 2) {
          // of a key two neighbouring dimensions: bytes (k, d) (k, d + 1) (k + 1, d) (k + 1, d + 1)
          const uint4 a = read_transposed(src + t * (16 * D) + (((i + vchunk) ^ vkey) * 16));
          auto step = [&](uint32_t k0, uint32_t k8, int i) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_half2s(__byte_perm(k0, 0, 0x3120), a0, a1);
            e4m3x4_to_half2s(__byte_perm(k8, 0, 0x3120), a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int x = 0; x < PS; ++x) mma16816<F16>(o[i][n], a0, a1, a2, a3, pf[t][n][x][0], pf[t][n][x][1]);
          };
          step(a.x, a.y, i), step(a.z, a.w, i + 1);
        }
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; !Q8 && i < MT; ++i) {
          // rows g: dimension 16 i + g; rows g + 8: 16 i + 8 + g
          const uint4 a = read_transposed(src + t * (32 * D) + (((2 * i + vchunk) ^ vkey) * 16));
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < PS; ++x)
              mma16816<F16>(o[i][n], a.x, a.y, a.z, a.w, pf[t][n][x][0], pf[t][n][x][1]);
        }
      sk = sn;
    }

    // Join: warp w + H into warp w, then warps 1 .. H - 1 into warp 0, through
    // shared memory; a warp that has handed its result over goes on to the
    // next unit.
    const int kvh = u.hk / p.head_tiles, h0 = (u.hk - kvh * p.head_tiles) * HT;
    const int head = kvh * p.group + h0, heads = min(HT, p.group - h0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], x);
    auto hand_over = [&](int to) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int hh = 8 * n + 2 * c + h;
          if (g == 0) sm.m[to][hh] = m[n][h], sm.l[to][hh] = l[n][h];
          if (hh < heads) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              sm.o[to][hh][dim(i, 0)] = o[i][n][h];
              sm.o[to][hh][dim(i, 1)] = o[i][n][2 + h];
            }
          }
        }
    };
    auto take_over = [&](int from) {  // m = max; l, O = f (l, O) + f' (l', O')
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int hh = 8 * n + 2 * c + h;
          const float m2 = sm.m[from][hh], mx = fmaxf(m[n][h], m2), ref = mx == -INFINITY ? 0.0f : mx;
          const float f = ex2_approx(m[n][h] - ref), f2 = ex2_approx(m2 - ref);
          m[n][h] = mx;
          l[n][h] = fmaf(f2, sm.l[from][hh], __fmul_rn(f, l[n][h]));
          if (hh < heads) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][n][h] = fmaf(f2, sm.o[from][hh][dim(i, 0)], __fmul_rn(f, o[i][n][h]));
              o[i][n][2 + h] = fmaf(f2, sm.o[from][hh][dim(i, 1)], __fmul_rn(f, o[i][n][2 + h]));
            }
          }
        }
    };
    if (warp >= H) {
      if (ui > 0) named_barrier(kBarRead, 32 * (H + 1));  // warp 0 has read the last unit's
      hand_over(warp - H);
      barrier_arrive(kBarUpper, kThreads);
    } else {
      named_barrier(kBarUpper, kThreads);
      take_over(warp);
      if (warp > 0) {
        __syncwarp();     // every lane has read the maxima and sums that some lanes replace now
        hand_over(warp);  // where this warp alone has just read
        barrier_arrive(kBarLower, 32 * H);
      } else {
        named_barrier(kBarLower, 32 * H);
#pragma unroll
        for (int w = 1; w < H; ++w) take_over(w);
        if (ui + 1 < units) barrier_arrive(kBarRead, 32 * (H + 1));
        if constexpr (ONE) {
          hand_over(0);  // for the cluster's first CTA, where this warp alone has read
          continue;
        }
        const int pieces = split_count(u.len, Q8);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int hh = 8 * n + 2 * c + h;
            if (hh >= heads) continue;
            if (pieces == 1) {
              const float inv = l[n][h] == 0.0f ? 0.0f : __frcp_rn(l[n][h]) * Up<C>::back;  // no key: zeros
              const int64_t at = u.b * p.o_b + (head + hh) * p.o_h;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                // + 0: a negative zero becomes the positive one that a join makes of it
                store_one(p.o, p.out_kind, at + dim(i, 0), __fmul_rn(__fadd_rn(o[i][n][h], 0.0f), inv));
                store_one(p.o, p.out_kind, at + dim(i, 1), __fmul_rn(__fadd_rn(o[i][n][2 + h], 0.0f), inv));
              }
            } else {
              const int64_t part = ((int64_t)u.b * p.max_splits + u.piece) * p.Hq + head + hh;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                p.ws_o[part * D + dim(i, 0)] = o[i][n][h];
                p.ws_o[part * D + dim(i, 1)] = o[i][n][2 + h];
              }
              if (g == 0) p.ws_ml[2 * part] = m[n][h], p.ws_ml[2 * part + 1] = l[n][h];
            }
          }
      }
    }
    u = next;
  }
  copies_wait<0>();
  if constexpr (ONE) {
    // The first CTA joins the cluster's pieces as paged_join_kernel does a
    // group of them (a piece that the request has not adds zeros).
    cluster_sync_all();
    if (cluster_ctarank() == 0) {
      const int kvh = u.hk / p.head_tiles, h0 = (u.hk - kvh * p.head_tiles) * HT;
      const int head = kvh * p.group + h0, heads = min(HT, p.group - h0);
      for (int e = threadIdx.x; e < heads * (D / 4); e += kThreads) {
        const int h = e / (D / 4), d = (e % (D / 4)) * 4;
        const uint32_t am = smem_u32(&sm.m[0][h]), al = smem_u32(&sm.l[0][h]), ao = smem_u32(&sm.o[0][h][d]);
        float m[kMaxCluster], l[kMaxCluster], o[kMaxCluster][4];
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r >= p.max_splits) break;
          m[r] = ld_shared_cluster_f32(cluster_map_shared(am, (uint32_t)r));
          l[r] = ld_shared_cluster_f32(cluster_map_shared(al, (uint32_t)r));
          const uint32_t x = cluster_map_shared(ao, (uint32_t)r);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[r][i] = ld_shared_cluster_f32(x + 4 * i);
          mx = fmaxf(mx, m[r]);
        }
        const float ref = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f, a[4] = {};
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r >= p.max_splits) break;
          const float f = ex2_approx(m[r] - ref);
          sum = fmaf(f, l[r], sum);
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = fmaf(f, o[r][i], a[i]);
        }
        const float inv = sum == 0.0f ? 0.0f : __frcp_rn(sum) * Up<C>::back;  // no key: zeros
        const int64_t at = u.b * p.o_b + (head + h) * p.o_h + d;
#pragma unroll
        for (int i = 0; i < 4; ++i) store_one(p.o, p.out_kind, at + i, __fmul_rn(a[i], inv));
      }
    }
    cluster_sync_all();  // no CTA leaves while the first may read its results
  }
}

// Joins the pieces of each (request, query head): groups of 16 pieces, each
// summed in piece order relative to the group's maximum, then the groups in
// order.  Lanes hold two neighbouring dimensions of each 64.
constexpr int kJoinGroup = 16;
constexpr int kJoinGroups = kManySplits / kJoinGroup;  // at most
constexpr int kJoinWarps = 8;

// Below this many rows a row is joined by a block a 64 dimensions (four
// requests of 131071 keys: 97 us against 112 with a warp a row), from it on by
// a warp (2048 rows of up to 32 pieces: 164 us against 170).
constexpr int64_t kFewRows = 1024;

template <int V>
struct Part {
  float m, l, o[V][2];
};
// One group, by one warp, 64 V dimensions from d0 on; its loads are requested
// eight pieces at a time before the first is used.
template <int V>
__device__ __forceinline__ Part<V> join_group(const PagedAttnParams& p, int64_t row0, int n, int group, int d0, int lane) {
  const int s0 = group * kJoinGroup, mine = min(kJoinGroup, n - s0);
  float2 ml = make_float2(-INFINITY, 0.0f);
  if (lane < mine) ml = *reinterpret_cast<const float2*>(p.ws_ml + 2 * (row0 + (int64_t)(s0 + lane) * p.Hq));
  const float* o = p.ws_o + (row0 + (int64_t)s0 * p.Hq) * p.D + d0 + 2 * lane;
  const int64_t step = (int64_t)p.Hq * p.D;
  Part<V> r = {};
  float f = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinGroup; i += 8) {
    if (i >= mine) break;
    float2 x[8][V];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v)
        x[k][v] = i + k < mine ? *reinterpret_cast<const float2*>(o + (i + k) * step + 64 * v) : make_float2(0.0f, 0.0f);
    if (i == 0) {
      r.m = ml.x;
#pragma unroll
      for (int y = 8; y > 0; y >>= 1) r.m = fmaxf(r.m, __shfl_xor_sync(0xffffffffu, r.m, y));
      r.m = __shfl_sync(0xffffffffu, r.m, 0);
      f = ex2_approx(ml.x - (r.m == -INFINITY ? 0.0f : r.m));
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i + k >= mine) break;
      const float w = __shfl_sync(0xffffffffu, f, i + k), wl = __shfl_sync(0xffffffffu, ml.y, i + k);
      r.l = fmaf(w, wl, r.l);
#pragma unroll
      for (int v = 0; v < V; ++v) r.o[v][0] = fmaf(w, x[k][v].x, r.o[v][0]), r.o[v][1] = fmaf(w, x[k][v].y, r.o[v][1]);
    }
  }
  return r;
}
template <int V>
__device__ __forceinline__ void join_into(Part<V>& r, float m, float l, const float (&o)[V][2]) {
  const float top = fmaxf(r.m, m), ref = top == -INFINITY ? 0.0f : top;
  const float f = ex2_approx(r.m - ref), f2 = ex2_approx(m - ref);
  r.m = top;
  r.l = fmaf(f2, l, __fmul_rn(f, r.l));
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 2; ++e) r.o[v][e] = fmaf(f2, o[v][e], __fmul_rn(f, r.o[v][e]));
}

// kSplit: a block joins 64 dimensions of one row, a warp a group; otherwise a
// warp joins a whole row (V = D / 64), eight rows a block.  The same bits.
template <int V, bool kSplit>
__global__ void __launch_bounds__(32 * kJoinWarps) paged_join_kernel(const PagedAttnParams p) {
  __shared__ float2 so[kSplit ? kJoinGroups : 1][32];
  __shared__ float sm[kJoinGroups], sl[kJoinGroups];
  static_assert(!kSplit || V == 1, "64 dimensions a block");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slices = kSplit ? p.D / 64 : 1;
  const int64_t bh = kSplit ? blockIdx.x / slices : (int64_t)blockIdx.x * kJoinWarps + warp;
  if (bh >= (int64_t)p.B * p.Hq) return;
  const int d0 = kSplit ? (int)(blockIdx.x % slices) * 64 : 0;
  const int b = (int)(bh / p.Hq), h = (int)(bh % p.Hq);
  const int n = split_count(request_len(p, b), p.e4m3 != 0), groups = (n + kJoinGroup - 1) / kJoinGroup;
  if (n == 1) return;  // written by its only piece
  const int64_t row0 = (int64_t)b * p.max_splits * p.Hq + h;
  Part<V> r = {};
  r.m = -INFINITY;
  if constexpr (kSplit) {
    for (int g = warp; g < groups; g += kJoinWarps) {
      const Part<V> x = join_group<V>(p, row0, n, g, d0, lane);
      so[g][lane] = make_float2(x.o[0][0], x.o[0][1]);
      if (lane == 0) sm[g] = x.m, sl[g] = x.l;
    }
    __syncthreads();
    if (warp > 0) return;
    for (int g = 0; g < groups; ++g) {
      const float o[1][2] = {{so[g][lane].x, so[g][lane].y}};
      join_into<1>(r, sm[g], sl[g], o);
    }
  } else {
    for (int g = 0; g < groups; ++g) {
      const Part<V> x = join_group<V>(p, row0, n, g, d0, lane);
      join_into<V>(r, x.m, x.l, x.o);
    }
  }
  const float inv = r.l == 0.0f ? 0.0f : __frcp_rn(r.l) * (p.e4m3 ? Up<kCache8>::back : p.in_f16 ? Up<kCache16>::back : Up<0>::back);
  const int64_t at = b * p.o_b + h * p.o_h + d0 + 2 * lane;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float y0 = __fmul_rn(r.o[v][0], inv), y1 = __fmul_rn(r.o[v][1], inv);
    if (p.out_kind == 2)
      *reinterpret_cast<float2*>(static_cast<float*>(p.o) + at + 64 * v) = make_float2(y0, y1);
    else
      *reinterpret_cast<uint32_t*>(static_cast<unsigned short*>(p.o) + at + 64 * v) =
          p.out_kind == 1 ? pack16<1>(y0, y1) : pack16<0>(y0, y1);
  }
}

// *joined: whether the launch leaves nothing to join.
template <int C, int D, int NT>
cudaError_t launch(PagedAttnParams& p, int num_sms, bool* joined, cudaStream_t stream) {
  using Sh = Shape<C, D, NT>;
  constexpr int kBytes = sizeof(typename Sh::Shared);
  static_assert(kBytes <= 227 * 1024 && Sh::kCtas * (kBytes + 1024) <= 228 * 1024, "shared memory of an SM");
  // one slot per instance, from 24 on (ONE: from 64 on), for caches in 8 bits from 115 on (120)
  constexpr int kSlot = C == kCache8 ? 115 + (D == 256 ? 4 : (D == 128 ? 2 : 0) + NT - 1)
                                     : 24 + (D == 256 ? 8 + C : (D == 128 ? 4 : 0) + 2 * C + NT - 1);
  constexpr int kOneSlot = C == kCache8 ? kSlot + 5 : kSlot + 40;
  p.head_tiles = (p.group + Sh::HT - 1) / Sh::HT;
  const int64_t most = (int64_t)p.B * p.max_splits * p.Hkv * p.head_tiles;
  // Tables of at most 4096 keys whose units all run at once: a CTA a unit and a
  // cluster a request's head tile, joined in place -- one launch, and no search
  // for the units (one request of 1021 keys 7.6 us; with a table for 131072, and
  // so the other way, 10.7).  The host knows the table's width and not the
  // lengths.  The bits are the same.
  const bool one = p.max_splits <= kMaxCluster && most <= (int64_t)num_sms * Sh::kCtas;
  *joined = p.max_splits == 1 || one;
  if (one) {
    cudaError_t e = set_smem_once(reinterpret_cast<const void*>(&paged_attn_kernel<C, D, NT, true>), kBytes, kOneSlot);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)most);
    cfg.blockDim = dim3(32 * Sh::W);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.max_splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attn_kernel<C, D, NT, true>, p);
  }
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(&paged_attn_kernel<C, D, NT, false>), kBytes, kSlot);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)num_sms * Sh::kCtas);
  paged_attn_kernel<C, D, NT, false><<<grid, 32 * Sh::W, kBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int C>
cudaError_t launch_dim(PagedAttnParams& p, int num_sms, bool* joined, cudaStream_t stream) {
  // more than eight query heads a key-value head: 16 a unit, except at
  // D = 256, where two tiles' accumulators would not fit the registers
  const bool wide = p.group > 8;
  if (p.D == 64) return wide ? launch<C, 64, 2>(p, num_sms, joined, stream) : launch<C, 64, 1>(p, num_sms, joined, stream);
  if (p.D == 128) return wide ? launch<C, 128, 2>(p, num_sms, joined, stream) : launch<C, 128, 1>(p, num_sms, joined, stream);
  return launch<C, 256, 1>(p, num_sms, joined, stream);
}

}  // namespace

int32_t paged_max_splits(int64_t cap, bool e4m3) {
  if (cap <= kMaxCluster * kMinSplit) return split_count(cap, e4m3);
  if (cap >= (int64_t)kManySplits * (e4m3 ? 4 : 2) * kMinSplit) return kManySplits;
  // or a request of 2048 keys, or one of kLongPieces where pieces get longer there
  return std::max(split_count(cap, e4m3), e4m3 && cap > kLongPieces ? split_count(kLongPieces, true) : (int32_t)kMaxCluster);
}

bi_status launch_paged_attention(PagedAttnParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  p.status_word = dev.status_word;
  bool joined = false;
  cudaError_t e = p.e4m3     ? launch_dim<kCache8>(p, dev.num_sms, &joined, stream)
                  : p.in_f16 ? launch_dim<1>(p, dev.num_sms, &joined, stream)
                             : launch_dim<0>(p, dev.num_sms, &joined, stream);
  if (e == cudaSuccess && !joined) {
    const int64_t rows = (int64_t)p.B * p.Hq;
    constexpr int kT = 32 * kJoinWarps;
    if (rows < kFewRows) {
      paged_join_kernel<1, true><<<(unsigned)(rows * (p.D / 64)), kT, 0, stream>>>(p);
    } else {
      const unsigned grid = (unsigned)((rows + kJoinWarps - 1) / kJoinWarps);
      if (p.D == 64)
        paged_join_kernel<1, false><<<grid, kT, 0, stream>>>(p);
      else if (p.D == 128)
        paged_join_kernel<2, false><<<grid, kT, 0, stream>>>(p);
      else
        paged_join_kernel<4, false><<<grid, kT, 0, stream>>>(p);
    }
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    *why = std::string("paged attention launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
