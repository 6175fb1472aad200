// bi_mm8.cu -- matrix product of e4m3 operands with a scale for each block of
// 128 of the reduction:
//   c[m,n] = sum_kb sa[m,kb] sb[kb,n/128] sum_{k in block kb} a[m,k] b[k,n]  (+ bias[n]).
//
// The scales are powers of two, so the tensor core can apply them as it
// multiplies (tcgen05.mma, kind::mxf8f6f4, one 8-bit exponent for each row and 32
// steps of K, here the same for the four steps of a block): accumulators run on
// over blocks.  (With scales applied to each block's accumulator in registers,
// 128 x 128 fp32 of TMEM a warp to read, scale and add every 512 cycles of MMAs,
// the 8192 x 4096 x 14336 product took 554 us: bound by the latency of that
// chain, 1400 cycles a block.)
//   D = the products of a segment of 16 blocks (K = 2048), 64 steps of K = 32 in
//       ascending order, fp32 in TMEM, the first one overwriting;
//   acc = the segments' sums, added in order in fp32.
// One order for every element, whatever the tile it is computed in.  Segments
// bound how long a sum stays in the tensor core, whose adds may truncate.
//
// Pairs of CTAs (cta_group::2), tiles of 256 rows x BN columns:
//   warp 0       producer: A (128 x 128 bytes) and this CTA's half of B's
//                columns of a K block by TMA into a ring of stages (128-byte
//                swizzle), as in the 16-bit product
//   warp 1       TMEM allocation; in the even CTA the issuer of the MMAs
//   warps 4-11   scales, two sets for every other group of four blocks: a warp
//                loads 32 rows' ahead, turns them into exponents, and the four of
//                a set write them all to TMEM, once for each quadrant of lanes,
//                which is a warp's
//   warps 12-19  sums: a warp has 32 rows and half of the tile's columns, BN / 2
//                fp32 registers a thread; it adds a segment's accumulator and
//                frees it (there are two), then bias, rounding and the store.
//
// At decode sizes the weight's bytes set the pace: BN is then narrower, so that
// there are pairs enough, and A stages of at most 32 rows leave room for more of
// B in flight (the tensor core reads 128 rows either way; rows past M are never
// stored): 16 x 14336 x 4096 15.4 us against 19.5, 16 x 4096 x 4096 9.5 against 13.7.
//
// Measured (M x N x K, bf16 results): 8192 x 14336 x 4096 308 us alone, 3.1 PFLOP/s,
// 342-354 in a long run under the power limit; 4096^3 50 us, 2.75 PFLOP/s; 2048 x 4096 x
// 4096 32 us; 300 x 14336 x 4096 23.7 us; 16 x 14336 x 4096 15.4 us, 3.8 TB/s: start
// (TMEM, barriers, a cluster's exchange, 3 us), the copies, the last segment's sums.
// Large ones are bound by the tensor cores and their power: a block's four MMAs take 400
// cycles at the 16-bit product's measured rate doubled, and the issuer 225; 4096^3 (352
// tiles on 76 pairs, 4.6 rounds) keeps the pipe 66 % busy.  One set of scale warps was
// waited for; stages of two blocks at full A leave too few of them; exponents written a
// stage at a time cost the issuer a wait each.
#include <cuda.h>
#include <cuda_runtime.h>

#include "bi_common.h"
#include "bi_launch.h"
#include "bi_ptx_ext.cuh"
#include "bi_quant.h"
#include "bi_roles.cuh"

namespace bi {
namespace {

constexpr int kBK8 = 128;     // K of a block and a stage: one 128-byte swizzle row
constexpr int kUmmaK8 = 32;   // K of a tcgen05.mma of 8-bit operands
constexpr int kSegmentBlocks = 16;  // K blocks of a segment: K = 2048
constexpr int kScaleWarps = 4, kScaleSets = 2, kSumWarps = 8, kParts = 2;
constexpr int kFirstScale = 4, kFirstSum = kFirstScale + kScaleWarps * kScaleSets;  // warps
constexpr int kThreads = 32 * (kFirstSum + kSumWarps);
constexpr int kGroup = 4;  // K blocks whose scales are loaded and written at once
constexpr int kStoreBytes = 2048;  // a sum warp's 32 x 32 results of 16 bits on their way out

struct ScaledParams {
  CUtensorMap tma_a;  // [M][K] bytes, box {128, 128 (32 for M <= 32)}
  CUtensorMap tma_b;  // [N][K] bytes, box {128, BN / 2}
  CUtensorMap tma_c;  // [M][N], box {32, 32}, if use_tma_store
  const float *sa, *sb;
  int64_t sa_m, sa_k, sb_k, sb_n;
  OutDesc out;
  int32_t M, N, m_tiles, n_tiles, k_blocks, num_tiles, use_tma_store;
  unsigned int* status_word;
  uint64_t wait_limit_ns;
};

template <int BN, int A_ROWS>
struct Layout8 {
  static constexpr int PART = BN / kParts;  // columns of a sum warp
  // K blocks of a stage of copies.  One: the ring comes free in small pieces, and
  // more of it is in flight.  Two where a block's copies take less than the 225
  // cycles that a stage costs the issuer.
  static constexpr int BLOCKS = A_ROWS == kBM ? 1 : 2;
  static constexpr int SLOTS = BN > 128 ? 2 : 4;  // groups of exponents in TMEM
  static constexpr int A_BYTES = A_ROWS * kBK8;          // a block
  static constexpr int B_BYTES = BN / 2 * kBK8;          // this CTA's half of the tile's columns
  static constexpr int STAGE_BYTES = BLOCKS * (A_BYTES + B_BYTES);
  static constexpr int ACC = 2;
  // exponents of a block in TMEM, a 32-bit column for each 32 rows of A and of B
  static constexpr int SFA_COLS = 4, SFB_COLS = BN > 128 ? 8 : 4, SF_COLS = SFA_COLS + SFB_COLS;
  static constexpr int BAR_BYTES = 1024;
  static constexpr int EXCHANGE_BYTES = kScaleSets * 2 * kBM * 4;  // exponents on their way between the scale warps
  static constexpr int STAGING_BYTES = A_ROWS == kBM ? kSumWarps * kStoreBytes : 0;
  static constexpr int MAX_DYN = 232448;
  static constexpr int FIT = (MAX_DYN - 1024 - BAR_BYTES - EXCHANGE_BYTES - STAGING_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 16 ? 16 : FIT;
  static constexpr int DYN_BYTES = 1024 + STAGES * STAGE_BYTES + BAR_BYTES + EXCHANGE_BYTES + STAGING_BYTES;
  static constexpr int A_OVERREAD = (kBM - A_ROWS) * kBK8;  // the tensor core reads 128 A rows from a block's base
  static_assert(STAGES >= 3, "pipeline depth");
  static_assert(ACC * BN + SLOTS * kGroup * SF_COLS <= 512, "accumulators and exponents fit TMEM");
  static_assert(SLOTS % kScaleSets == 0, "a slot is always the same warps', who see each of its phases");
  static_assert(8 * (2 * STAGES + 2 * ACC + 2 * SLOTS + 1) + 8 <= BAR_BYTES, "barriers fit their block");
  static_assert(kGroup % BLOCKS == 0 && kSegmentBlocks % kGroup == 0, "stages in groups in segments");
  static_assert(A_OVERREAD <= STAGES * BLOCKS * B_BYTES, "A over-read stays inside the B stages");
  static_assert(DYN_BYTES > 116 * 1024, "one CTA per SM: TMEM is allocated whole");
  static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "stages hold whole swizzle atoms");
};

// CTA pair, kind::mxf8f6f4: D (+)= (A 2^(ea - 127)) (B 2^(eb - 127)), as umma_bf16_pair; the exponents
// of A's rows in each CTA's TMEM, of all of B's columns in both.
__device__ __forceinline__ void umma_mx_pair(uint32_t tmem_d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t tmem_sfa, uint32_t tmem_sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
          tmem_d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(tmem_sfa), "r"(tmem_sfb), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of it: e4m3 A and B (0), both K-major, exponents as UE8M0 (bit 23), in byte 0 of their words.
constexpr uint32_t idesc_mx(uint32_t m, uint32_t n) { return ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24); }

__device__ __forceinline__ void tmem_store_4cols(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// One lane of a converged warp, known as such to the compiler: a branch on lane ==
// 0 makes it move every descriptor through per-thread code (four MMAs 280 cycles
// to issue, this way 65).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// A load that stays where it is written, ahead of the waits before its use.
__device__ __forceinline__ float load_now(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
// The exponent byte of a scale 2^(e - 127); anything else is a NaN to the tensor core.
__device__ __forceinline__ uint32_t exponent_byte(float scale) {
  const uint32_t b = __float_as_uint(scale);
  return (b & 0x807fffffu) == 0 && b != 0 ? b >> 23 : 255u;
}

// A warp's 32 x 32 results at (m0, n0), a row a lane, into rows that 16-byte stores do
// not fit: through the warp's buffer, so that it writes a row at a time (fp32: half of
// two).  5157 x 694 x 369 takes 13 us this way; with a row of its own a lane, 2 bytes a
// sector, a call took 44.
__device__ __forceinline__ void store_32_rows(const OutDesc& o, uint8_t* buf, int m0, int n0, int lane, const float (&f)[32]) {
  const uint32_t to = smem_u32(buf);
  if (!o.out_f32) {
    __syncwarp();
    stage_32(o, to, lane, f);
    __syncwarp();
    uint16_t* c = static_cast<uint16_t*>(o.c) + (int64_t)m0 * o.ldc + n0 + lane;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      const uint16_t v = *reinterpret_cast<const uint16_t*>(buf + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2);
      if (m0 + i < o.M && n0 + lane < o.N) c[i * o.ldc] = v;
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __syncwarp();
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        const int i = 16 * h + 4 * cc;
        st_shared_v4(to + lane * 64 + ((cc ^ ((lane >> 1) & 3)) << 4), __float_as_uint(f[i]), __float_as_uint(f[i + 1]),
                     __float_as_uint(f[i + 2]), __float_as_uint(f[i + 3]));
      }
      __syncwarp();
      const int col = lane & 15, n = n0 + 16 * h + col;
#pragma unroll 8
      for (int i = lane >> 4; i < 32; i += 2) {
        const float v = *reinterpret_cast<const float*>(buf + i * 64 + (((col >> 2) ^ ((i >> 1) & 3)) << 4) + (col & 3) * 4);
        if (m0 + i < o.M && n < o.N) static_cast<float*>(o.c)[(int64_t)(m0 + i) * o.ldc + n] = v;
      }
    }
  }
}

template <int BN, int A_ROWS, bool STREAM_B>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    scaled_gemm_kernel(const __grid_constant__ ScaledParams p) {
  using Lay = Layout8<BN, A_ROWS>;
  constexpr int PART = Lay::PART, ACC = Lay::ACC;
  constexpr uint16_t kBoth = 3;
  const uint32_t crank = cluster_ctarank();
  const int stride = gridDim.x >> 1, first_tile = blockIdx.x >> 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sA = base, sB = base + Lay::STAGES * Lay::BLOCKS * Lay::A_BYTES;
  const uint32_t staging0 = sB + Lay::STAGES * Lay::BLOCKS * Lay::B_BYTES;
  uint32_t* exchange = reinterpret_cast<uint32_t*>(smem + (staging0 + Lay::STAGING_BYTES - base));
  PipeBars bars;
  bars.full0 = staging0 + Lay::STAGING_BYTES + Lay::EXCHANGE_BYTES;
  bars.empty0 = bars.full0 + 8 * Lay::STAGES;
  bars.tfull0 = bars.empty0 + 8 * Lay::STAGES;
  bars.tempty0 = bars.tfull0 + 8 * ACC;
  bars.drain = bars.tempty0 + 8 * ACC;
  const uint32_t sfull0 = bars.drain + 8, sempty0 = sfull0 + 8 * Lay::SLOTS;  // of the groups of exponents
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (sempty0 + 8 * Lay::SLOTS - base));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = (p.k_blocks + Lay::BLOCKS - 1) / Lay::BLOCKS;  // of a tile
  const int groups = (p.k_blocks + kGroup - 1) / kGroup;

  if (threadIdx.x == 0) {
    // Even CTA: a stage is full when the copies of both CTAs have landed, a group
    // of exponents when a set of scale warps in each has written them; an
    // accumulator is free when the sum warps of both have read it.
    for (int s = 0; s < Lay::STAGES; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    for (int g = 0; g < Lay::SLOTS; ++g) {
      mbar_init(sfull0 + 8 * g, 2 * kScaleWarps);
      mbar_init(sempty0 + 8 * g, 1);
    }
    for (int b = 0; b < ACC; ++b) {
      mbar_init(bars.tfull(b), 1);
      mbar_init(bars.tempty(b), 2 * kSumWarps);
    }
    mbar_init(bars.drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tma_a);
    tma_prefetch_desc(&p.tma_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t sf_base = tmem_base + ACC * BN;  // exponents of block j of slot g: sf_base + (g * kGroup + j) * SF_COLS
  cluster_arrive_relaxed();
  cluster_wait();  // both CTAs' barriers are initialised
  const WaitCtl wc{abort_flag, p.status_word, p.wait_limit_ns};

  // 256 x 152 + 384 x 56 <= 640 x 96
  if (warp < kFirstSum) {
    setmaxnreg_dec<56>();
    if (warp == 0 && elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < p.num_tiles; tile += stride) {
        const TileCoord tc = decode_tile(tile, p.m_tiles, p.n_tiles);
        const int mb = 2 * tc.mb + (int)crank;
        const bool a_live = mb * kBM < p.M, peer_live = (mb + 1) * kBM < p.M;  // (peer_live: even CTA)
        const int n0 = tc.nb * BN + (int)crank * (BN / 2);
        for (int st = 0; st < stages; ++st, ++it) {
          const uint32_t s = it % Lay::STAGES, r = it / Lay::STAGES;
          if (r > 0 && !mbar_wait_bounded(bars.empty(s), (r - 1) & 1, wc.abort, wc.status_word, wc.limit_ns,
                                          status_code(6, kSiteProducerEmpty))) {
            ok = false;
            break;
          }
          if (crank == 0)
            mbar_arrive_expect_tx(bars.full(s), Lay::BLOCKS * (2 * Lay::B_BYTES + Lay::A_BYTES * (peer_live ? 2 : 1)));
          const uint32_t fb = cluster_map_shared(bars.full(s), 0);
#pragma unroll
          for (int j = 0; j < Lay::BLOCKS; ++j) {  // (a block past K is all zeros)
            const int k = (st * Lay::BLOCKS + j) * kBK8;
            const uint32_t at = s * Lay::BLOCKS + j;
            if (STREAM_B) {  // B is used by one or two pairs, A by every column tile
              tma_load_3d_pair_hint(sB + at * Lay::B_BYTES, &p.tma_b, fb, k, n0, 0, l2_policy_evict_first());
              if (a_live)
                tma_load_3d_pair_hint(sA + at * Lay::A_BYTES, &p.tma_a, fb, k, mb * kBM, 0, l2_policy_evict_last());
            } else {
              tma_load_3d_pair(sB + at * Lay::B_BYTES, &p.tma_b, fb, k, n0, 0);
              if (a_live) tma_load_3d_pair(sA + at * Lay::A_BYTES, &p.tma_a, fb, k, mb * kBM, 0);
            }
          }
        }
      }
      // every fill of the ring has been consumed before this CTA may leave
      const uint32_t first = it > (uint32_t)Lay::STAGES ? it - Lay::STAGES : 0u;
      for (uint32_t j = first; j < it; ++j)
        if (!mbar_wait_bounded(bars.empty(j % Lay::STAGES), (j / Lay::STAGES) & 1, nullptr, wc.status_word, wc.limit_ns,
                               status_code(6, kSiteDrain)))
          break;
    } else if (warp == 1 && crank == 0 && elect_one()) {
      constexpr uint32_t kIdesc = idesc_mx(2 * kBM, BN);
      uint32_t it = 0, seg = 0, grp = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < p.num_tiles; tile += stride) {
        for (int st = 0; st < stages; ++st, ++it) {
          const int kb = st * Lay::BLOCKS;
          const bool opens = kb % kSegmentBlocks == 0;
          const uint32_t buf = seg % ACC, use = seg / ACC, s = it % Lay::STAGES, slot = grp % Lay::SLOTS;
          if (opens && use > 0 &&
              !mbar_wait_bounded<true>(bars.tempty(buf), (use - 1) & 1, wc.abort, wc.status_word, wc.limit_ns,
                                       status_code(6, kSiteMmaTmemEmpty))) {
            ok = false;
            break;
          }
          // (Exponents, some of them the other CTA's: cluster scope.  Copies: CTA scope,
          // their bytes are counted here when they have landed; the cluster's would cost
          // 150 cycles more a wait.)
          if ((kb % kGroup == 0 && !mbar_wait_bounded<true>(sfull0 + 8 * slot, (grp / Lay::SLOTS) & 1, wc.abort,
                                                            wc.status_word, wc.limit_ns, status_code(6, kSiteMmaFull))) ||
              !mbar_wait_bounded(bars.full(s), (it / Lay::STAGES) & 1, wc.abort, wc.status_word, wc.limit_ns,
                                 status_code(6, kSiteMmaFull))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
#pragma unroll
          for (int j = 0; j < Lay::BLOCKS; ++j) {
            const uint32_t at = s * Lay::BLOCKS + j;
            const uint64_t a = smem_desc_sw128(sA + at * Lay::A_BYTES, 16, 1024);
            const uint64_t b = smem_desc_sw128(sB + at * Lay::B_BYTES, 16, 1024);
            const uint32_t sf = sf_base + (slot * kGroup + (uint32_t)(kb + j) % kGroup) * Lay::SF_COLS;
#pragma unroll
            for (int k = 0; k < kBK8 / kUmmaK8; ++k)  // (the address is the low bits, in 16-byte units)
              umma_mx_pair(tmem_base + buf * BN, a + 2 * k, b + 2 * k, kIdesc, sf, sf + Lay::SFA_COLS,
                           opens && j == 0 && k == 0 ? 0u : 1u);
          }
          umma_commit_pair(bars.empty(s), kBoth);
          const int next = kb + Lay::BLOCKS;
          if (next % kGroup == 0 || st + 1 == stages) {
            umma_commit_pair(sempty0 + 8 * slot, kBoth);
            ++grp;
          }
          if (next % kSegmentBlocks == 0 || st + 1 == stages) {
            umma_commit_pair(bars.tfull(buf), kBoth);
            ++seg;
          }
        }
      }
      umma_commit_pair(bars.drain, 1);
      mbar_wait_bounded(bars.drain, 0, nullptr, wc.status_word, wc.limit_ns, status_code(6, kSiteDrain));
    } else if (warp >= kFirstScale) {
      const int q = warp & 3, set = (warp - kFirstScale) >> 2;  // the set takes every other group
      uint32_t first = 0, turn = 0;                             // groups of the tiles before; exchanges
      // A warp whose wait has run out goes on to the set's next exchange, by which all
      // four leave: none waits there for one that has left.
      bool ok = true, leave = false;
      for (int tile = first_tile; !leave && tile < p.num_tiles; tile += stride, first += groups) {
        const TileCoord tc = decode_tile(tile, p.m_tiles, p.n_tiles);
        const int m0 = (2 * tc.mb + (int)crank) * kBM, n0 = tc.nb * BN;
        // A: this lane's row, 32 q + lane (short A has the first quadrant's only);
        // B: lanes 0-3 the tile's first block of columns, lanes 4-7 its second
        const float* sa = p.sa + (int64_t)min(m0 + (A_ROWS == kBM ? 32 * q : 0) + lane, p.M - 1) * p.sa_m;
        const float* sb = p.sb + (int64_t)min(n0 / 128 + ((lane >> 2) & 1), (p.N - 1) / 128) * p.sb_n;
        float a[kGroup], b;
        auto request = [&](int g) {  // (a block past K: any)
#pragma unroll
          for (int j = 0; j < kGroup; ++j) a[j] = load_now(sa + min(g * kGroup + j, p.k_blocks - 1) * p.sa_k);
          b = load_now(sb + min(g * kGroup + (lane & 3), p.k_blocks - 1) * p.sb_k);
        };
        const int g0 = (set + kScaleSets - (int)(first % kScaleSets)) % kScaleSets;
        request(g0);
        for (int g = g0; g < groups; g += kScaleSets, ++turn) {
          const uint32_t mine = exponent_byte(a[0]) | exponent_byte(a[1]) << 8 | exponent_byte(a[2]) << 16 | exponent_byte(a[3]) << 24;
          const uint32_t col = exponent_byte(b);
          request(g + kScaleSets);
          uint32_t rows[4] = {mine, mine, mine, mine};
          if constexpr (A_ROWS == kBM) {
            uint32_t* x = exchange + (2 * set + (turn & 1)) * kBM;  // (a warp is at most one turn ahead)
            x[32 * q + lane] = mine;
            if (!named_barrier_and(1 + set, 32 * kScaleWarps, ok)) {
              leave = true;
              break;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) rows[c] = x[32 * c + lane];
          }
          const uint32_t slot = (first + g) % Lay::SLOTS, use = (first + g) / Lay::SLOTS;
          const bool got = use == 0 || mbar_wait_bounded(sempty0 + 8 * slot, (use - 1) & 1, wc.abort, wc.status_word,
                                                         wc.limit_ns, status_code(6, kSiteProducerEmpty));
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            if constexpr (A_ROWS == kBM) continue;
            leave = true;
            break;
          }
          tc_fence_after_sync();
          const uint32_t to = sf_base + slot * kGroup * Lay::SF_COLS + ((uint32_t)(q * 32) << 16);
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            const uint32_t pick = j * 0x1111u;  // a byte four times
            tmem_store_4cols(to + j * Lay::SF_COLS, __byte_perm(rows[0], 0, pick), __byte_perm(rows[1], 0, pick),
                             __byte_perm(rows[2], 0, pick), __byte_perm(rows[3], 0, pick));
            // 32 columns of the tile lie in one block of 128
            const uint32_t lo = __shfl_sync(0xffffffffu, col, j) * 0x01010101u, hi = __shfl_sync(0xffffffffu, col, 4 + j) * 0x01010101u;
            uint32_t w[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) w[c] = (n0 + 32 * c) / 128 == n0 / 128 ? lo : hi;
            tmem_store_4cols(to + j * Lay::SF_COLS + Lay::SFA_COLS, w[0], w[1], w[2], w[3]);
            if (Lay::SFB_COLS > 4) tmem_store_4cols(to + j * Lay::SF_COLS + Lay::SFA_COLS + 4, w[4], w[5], w[6], w[7]);
          }
          // (the issuer, in the even CTA, has the pair's MMAs read both CTAs' exponents:
          // stores, fence, arrival and its wait are ordered as mbar_arrive_remote says)
          tmem_store_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if (crank != 0)
              mbar_arrive_remote(sfull0 + 8 * slot, 0);
            else
              mbar_arrive(sfull0 + 8 * slot);
          }
        }
      }
    }
    __syncwarp();
  } else {
    setmaxnreg_inc<152>();
    const int q = warp & 3, part = (warp - kFirstSum) >> 2;
    OutDesc o = p.out;
    o.tma_c = (Lay::STAGING_BYTES > 0 && p.use_tma_store) ? &p.tma_c : nullptr;  // 16 bits
    const uint32_t sbuf = staging0 + (warp - kFirstSum) * kStoreBytes;
    uint32_t seg = 0;
    bool ok = true;
    for (int tile = first_tile; ok && tile < p.num_tiles; tile += stride) {
      const TileCoord tc = decode_tile(tile, p.m_tiles, p.n_tiles);
      const int m0 = (2 * tc.mb + (int)crank) * kBM + q * 32, n0 = tc.nb * BN + part * PART;
      const int n_left = p.N - n0;
      const bool live = m0 < p.M && n_left > 0;  // any output here
      TileBias<PART> tb;
      if (live) load_tile_bias<PART>(o, 0, m0 + lane, n0, lane, tb);
      float acc[PART];
#pragma unroll
      for (int i = 0; i < PART; ++i) acc[i] = 0.0f;
      for (int st = 0; st < stages; st += kSegmentBlocks / Lay::BLOCKS, ++seg) {
        const uint32_t buf = seg % ACC;
        const bool got = mbar_wait_bounded(bars.tfull(buf), (seg / ACC) & 1, wc.abort, wc.status_word, wc.limit_ns,
                                           status_code(6, kSiteEpilogueTmemFull));
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t src = tmem_base + ((uint32_t)(q * 32) << 16) + buf * BN + part * PART;
        if (live) {
#pragma unroll
          for (int j = 0; j < PART / 32; ++j) {
            uint32_t v[32];
            tmem_load_32cols(src + j * 32, v);
            tmem_load_wait(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[32 * j + i] = __fadd_rn(acc[32 * j + i], __uint_as_float(v[i]));
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (crank != 0)
            mbar_arrive_remote(bars.tempty(buf), 0);
          else
            mbar_arrive(bars.tempty(buf));
        }
      }
      if (!ok) break;
      if (!live) continue;
#pragma unroll
      for (int j = 0; j < PART / 32; ++j) {
        if (32 * j >= n_left) break;
        uint32_t v[32];
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(acc[32 * j + i]);
        epilogue_math<PART>(o, j, tb, v, f);
        if (o.tma_c && m0 + 32 <= p.M) {
          if (lane == 0) bulk_wait_read_all();  // the chunk before has left the buffer
          __syncwarp();
          stage_32(o, sbuf, lane, f);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(o.tma_c, sbuf, n0 + 32 * j, m0, 0);
            bulk_commit();
          }
        } else if (Lay::STAGING_BYTES > 0 && !o.vec_store) {
          store_32_rows(o, smem + (sbuf - base), m0, n0 + 32 * j, lane, f);
        } else {
          store_32_direct(o, 0, m0 + lane, n0 + 32 * j, true, f);
        }
      }
    }
    if (o.tma_c && lane == 0) bulk_wait_read_all();
    __syncwarp();
  }

  // Neither CTA leaves while the other may still signal it or use its TMEM.
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

bool encode_bytes(CUtensorMap* map, const void* ptr, int64_t rows, int64_t K, int64_t ld, uint32_t box_rows,
                  std::string* why) {
  const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)rows, 1};
  const cuuint64_t strides[2] = {(cuuint64_t)ld, round_up_u64((uint64_t)ld * (uint64_t)rows, 16)};
  const cuuint32_t box[3] = {kBK8, box_rows, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, const_cast<void*>(ptr), 3, dims,
                      strides, box, why);
}

// Kernel slots from 104 on, one an instance.
template <int BN, int A_ROWS, bool STREAM_B>
cudaError_t launch_variant(ScaledParams& p, cudaStream_t stream, int slot) {
  using Lay = Layout8<BN, A_ROWS>;
  const void* fn = reinterpret_cast<const void*>(&scaled_gemm_kernel<BN, A_ROWS, STREAM_B>);
  cudaError_t e = set_smem_once(fn, Lay::DYN_BYTES, slot);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  e = pair_capacity(fn, kThreads, Lay::DYN_BYTES, slot, &pairs);
  if (e != cudaSuccess) return e;
  const int grid = 2 * std::min(p.num_tiles, pairs);
  scaled_gemm_kernel<BN, A_ROWS, STREAM_B><<<grid, kThreads, Lay::DYN_BYTES, stream>>>(p);
  return cudaGetLastError();
}

template <int BN>
cudaError_t launch_width(ScaledParams& p, cudaStream_t stream) {
  constexpr int kSlot = 104 + (BN == 192 ? 0 : BN == 128 ? 3 : 6);
  if (p.M <= kShortARows) return launch_variant<BN, kShortARows, true>(p, stream, kSlot);
  // (hints to L2: 300 x 14336 x 4096 23.7 us against 24.0, 16 rows of it 15.4 against
  // 15.9; from three row tiles on no difference, and B is better left where it is)
  return p.m_tiles <= 2 ? launch_variant<BN, kBM, true>(p, stream, kSlot + 1)
                        : launch_variant<BN, kBM, false>(p, stream, kSlot + 2);
}

}  // namespace

bi_status launch_scaled_gemm(const ScaledProblem& g, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  ScaledParams p;
  memset(&p, 0, sizeof(p));
  p.M = (int32_t)g.M, p.N = (int32_t)g.N;
  p.m_tiles = (int32_t)((g.M + 2 * kBM - 1) / (2 * kBM));
  p.k_blocks = (int32_t)((g.K + kBK8 - 1) / kBK8);
  // The width whose rounds of tiles take least: a K block takes a pair a time of
  // about BN + 128 columns' (short A: BN + 64); the wider one among equals.  (192, 128,
  // 64 columns: 16 x 14336 x 4096 15.4, 17.1, 19.8 us; 16 x 4096 x 14336 28.7, 22.4,
  // 21.5; 300 x 4096 x 4096 14.2, 13.1, 19.4; 4096^3 50, 59, 108.)
  const int64_t pairs = dev.num_sms / 2;
  auto tiles = [&](int64_t bn) { return (int64_t)p.m_tiles * ((g.N + bn - 1) / bn); };
  const int64_t each = g.M <= kShortARows ? 64 : 128;
  auto cost = [&](int64_t bn) { return (tiles(bn) + pairs - 1) / pairs * (bn + each); };
  int bn = 192;
  for (int w : {128, 64})
    if (cost(w) < cost(bn)) bn = w;
  if (tiles(bn) > INT32_MAX) {
    *why = "tile count exceeds 2^31";
    return BI_ERR_INVALID_ARG;
  }
  p.n_tiles = (int32_t)((g.N + bn - 1) / bn);
  p.num_tiles = p.m_tiles * p.n_tiles;
  if (!encode_bytes(&p.tma_a, g.a, g.M, g.K, g.lda, g.M <= kShortARows ? kShortARows : kBM, why) ||
      !encode_bytes(&p.tma_b, g.b, g.N, g.K, g.ldb, (uint32_t)bn / 2, why))
    return BI_ERR_CUDA;
  p.sa = g.sa, p.sb = g.sb;
  p.sa_m = g.sa_m, p.sa_k = g.sa_k, p.sb_k = g.sb_k, p.sb_n = g.sb_n;
  OutDesc& o = p.out;
  o.c = g.c, o.ldc = g.ldc;
  o.bias = g.bias, o.bias_stride = g.bias_stride, o.bias_kind = g.bias_kind;
  o.alpha = 1.0f, o.M = p.M, o.N = p.N;
  o.out_f32 = g.c_kind == 2, o.out_f16 = g.c_kind == 1;
  o.vec_store = g.vec_store;
  o.bias_groups = 1, o.tile_rows = kBM;
  p.use_tma_store = !o.out_f32 && encode_output_map(&p.tma_c, g.c, false, o.out_f16 != 0, 1, g.M, g.N, g.ldc, 0) ? 1 : 0;
  p.status_word = dev.status_word;
  p.wait_limit_ns = kWaitLimitNs;
  const cudaError_t e = bn == 192 ? launch_width<192>(p, stream) : bn == 128 ? launch_width<128>(p, stream) : launch_width<64>(p, stream);
  if (e != cudaSuccess) {
    *why = std::string("block-scaled product launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
