// bi_mm8.cu -- matrix product of e4m3 operands with a scale for each block of
// 128 of the reduction:
//   c[m,n] = sum_kb sa[m,kb] sb[kb,n/128] sum_{k in block kb} a[m,k] b[k,n]  (+ bias[n]).
//
// The scales change every 128 steps of K, so a tensor-core accumulator can run
// over one block only; what the blocks leave is scaled and summed in registers:
//   D = sum of the block's products (four tcgen05.mma steps of K = 32, fp32 in
//       TMEM, the first one overwriting),
//   acc = fma(D, RN(sa sb), acc), block after block, from zero.
// One order for every element, whatever the tile it is computed in.
//
// Pairs of CTAs (cta_group::2), tiles of 256 rows x BN columns:
//   warp 0       producer: A (128 x 128 bytes) and this CTA's half of B's
//                columns of each K block by TMA into a ring of stages (128-byte
//                swizzle), as in the 16-bit product
//   warp 1       TMEM allocation; in the even CTA the issuer of the MMAs, a
//                K block to one of the ACC = 512 / BN accumulators, in turn
//   warps 4-11   the sums: warp w has rows 32 (w % 4) .. + 31 and half of the
//                tile's columns, BN / 2 fp32 registers a thread.  It reads a
//                block's accumulator, frees it for the issuer at once and adds;
//                after the last block bias, rounding and the store.
// A block's MMAs take 4 x 128 cycles of a pair at BN = 256; reading 128 x 256
// fp32 of TMEM a SM takes half of that, the sums (two a fused multiply-add
// instruction) a quarter, so the tensor cores set the pace.
//
// At decode sizes the weight's bytes do: BN is then narrower, so that there are
// pairs enough, and the A stages of at most 32 rows leave room for more of B in
// flight (the tensor core reads 128 rows either way; rows past M are never
// stored).
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
constexpr int kThreads = 384;
constexpr int kSumWarps = 8;
constexpr int kGroup = 4;  // K blocks whose scales a thread holds
constexpr uint32_t kSumRegs = 232, kOtherRegs = 40;  // 256 x 232 + 128 x 40 = 384 x 168

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
  static constexpr int A_BYTES = A_ROWS * kBK8;
  static constexpr int B_BYTES = BN / 2 * kBK8;  // this CTA's half of the tile's columns
  static constexpr int ACC = 512 / BN > 8 ? 8 : 512 / BN;
  static constexpr int BAR_BYTES = 1024;
  static constexpr int STAGING_BYTES = A_ROWS == kBM ? kSumWarps * 2 * kStageOutBytes : 0;
  static constexpr int MAX_DYN = 232448;
  static constexpr int FIT = (MAX_DYN - 1024 - BAR_BYTES - STAGING_BYTES) / (A_BYTES + B_BYTES);
  static constexpr int STAGES = FIT > 24 ? 24 : FIT;
  static constexpr int DYN_BYTES = 1024 + STAGES * (A_BYTES + B_BYTES) + BAR_BYTES + STAGING_BYTES;
  // the tensor core reads up to 128 A rows from a stage's base
  static constexpr int A_OVERREAD = (kBM - A_ROWS) * kBK8;
  static_assert(STAGES >= 3, "pipeline depth");
  static_assert(8 * (2 * STAGES + 2 * ACC + 1) + 8 <= BAR_BYTES, "barriers fit their block");
  static_assert(A_OVERREAD <= STAGES * B_BYTES, "A over-read stays inside the B stages");
  static_assert(DYN_BYTES > 116 * 1024, "one CTA per SM: TMEM is allocated whole");
  static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "stages hold whole swizzle atoms");
};

// CTA pair, kind::f8f6f4: as umma_bf16_pair with 8-bit operands.
__device__ __forceinline__ void umma_e4m3_pair(uint32_t tmem_d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (0), both K-major.
constexpr uint32_t idesc_e4m3(uint32_t m, uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24); }

// (d0, d1) * s + (a0, a1), two fused multiply-adds of one instruction.
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t d0, uint32_t d1, float s) {
  asm("{\n\t.reg .b64 d, s, a;\n\t"
      "mov.b64 d, {%2, %3};\n\t"
      "mov.b64 s, {%4, %4};\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "fma.rn.f32x2 a, d, s, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "r"(d0), "r"(d1), "f"(s));
}

template <int BN, int A_ROWS, bool STREAM_B>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    scaled_gemm_kernel(const __grid_constant__ ScaledParams p) {
  using Lay = Layout8<BN, A_ROWS>;
  constexpr int HALF = BN / 2, ACC = Lay::ACC;
  constexpr uint16_t kBoth = 3;
  const uint32_t crank = cluster_ctarank();
  const int stride = gridDim.x >> 1, first_tile = blockIdx.x >> 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sA = base, sB = base + Lay::STAGES * Lay::A_BYTES;
  const uint32_t staging0 = sB + Lay::STAGES * Lay::B_BYTES;
  const uint32_t bar0 = staging0 + Lay::STAGING_BYTES;
  PipeBars bars;
  bars.full0 = bar0;
  bars.empty0 = bar0 + 8 * Lay::STAGES;
  bars.tfull0 = bars.empty0 + 8 * Lay::STAGES;
  bars.tempty0 = bars.tfull0 + 8 * ACC;
  bars.drain = bars.tempty0 + 8 * ACC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bars.drain + 8 - base));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Lay::STAGES; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    for (int b = 0; b < ACC; ++b) {
      mbar_init(bars.tfull(b), 1);
      mbar_init(bars.tempty(b), 2 * kSumWarps);  // the sum warps of both CTAs
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
  cluster_arrive_relaxed();
  cluster_wait();  // both CTAs' barriers are initialised
  const WaitCtl wc{abort_flag, p.status_word, p.wait_limit_ns};

  if (warp < 4) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == 0 && lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < p.num_tiles; tile += stride) {
        const TileCoord tc = decode_tile(tile, p.m_tiles, p.n_tiles);
        const int mb = 2 * tc.mb + (int)crank;
        const bool a_live = mb * kBM < p.M, peer_live = (mb + 1) * kBM < p.M;  // (peer_live: even CTA)
        const int n0 = tc.nb * BN + (int)crank * HALF;
        for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
          const uint32_t s = it % Lay::STAGES, r = it / Lay::STAGES;
          if (r > 0 && !mbar_wait_bounded(bars.empty(s), (r - 1) & 1, wc.abort, wc.status_word, wc.limit_ns,
                                          status_code(6, kSiteProducerEmpty))) {
            ok = false;
            break;
          }
          if (crank == 0)
            mbar_arrive_expect_tx(bars.full(s), 2 * Lay::B_BYTES + Lay::A_BYTES * (peer_live ? 2 : 1));
          const uint32_t fb = cluster_map_shared(bars.full(s), 0);
          if (STREAM_B) {  // B is used by one or two pairs, A by every column tile
            tma_load_3d_pair_hint(sB + s * Lay::B_BYTES, &p.tma_b, fb, kb * kBK8, n0, 0, l2_policy_evict_first());
            if (a_live)
              tma_load_3d_pair_hint(sA + s * Lay::A_BYTES, &p.tma_a, fb, kb * kBK8, mb * kBM, 0, l2_policy_evict_last());
          } else {
            tma_load_3d_pair(sB + s * Lay::B_BYTES, &p.tma_b, fb, kb * kBK8, n0, 0);
            if (a_live) tma_load_3d_pair(sA + s * Lay::A_BYTES, &p.tma_a, fb, kb * kBK8, mb * kBM, 0);
          }
        }
      }
      // every fill of the ring has been consumed before this CTA may leave
      const uint32_t first = it > (uint32_t)Lay::STAGES ? it - Lay::STAGES : 0u;
      for (uint32_t j = first; j < it; ++j)
        if (!mbar_wait_bounded(bars.empty(j % Lay::STAGES), (j / Lay::STAGES) & 1, nullptr, wc.status_word, wc.limit_ns,
                               status_code(6, kSiteDrain)))
          break;
    } else if (warp == 1 && lane == 0 && crank == 0) {
      constexpr uint32_t kIdesc = idesc_e4m3(2 * kBM, BN);
      uint32_t it = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < p.num_tiles; tile += stride) {
        for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
          const uint32_t buf = it % ACC, use = it / ACC, s = it % Lay::STAGES;
          if (use > 0 && !mbar_wait_bounded<true>(bars.tempty(buf), (use - 1) & 1, wc.abort, wc.status_word, wc.limit_ns,
                                                  status_code(6, kSiteMmaTmemEmpty))) {
            ok = false;
            break;
          }
          if (!mbar_wait_bounded<true>(bars.full(s), (it / Lay::STAGES) & 1, wc.abort, wc.status_word, wc.limit_ns,
                                       status_code(6, kSiteMmaFull))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a = sA + s * Lay::A_BYTES, b = sB + s * Lay::B_BYTES;
#pragma unroll
          for (int k = 0; k < kBK8 / kUmmaK8; ++k)
            umma_e4m3_pair(tmem_base + buf * BN, smem_desc_sw128(a + k * 32, 16, 1024),
                           smem_desc_sw128(b + k * 32, 16, 1024), kIdesc, k != 0 ? 1u : 0u);
          umma_commit_pair(bars.empty(s), kBoth);
          umma_commit_pair(bars.tfull(buf), kBoth);
        }
      }
      umma_commit_pair(bars.drain, 1);
      mbar_wait_bounded(bars.drain, 0, nullptr, wc.status_word, wc.limit_ns, status_code(6, kSiteDrain));
    }
    __syncwarp();
  } else {
    setmaxnreg_inc<kSumRegs>();
    const int q = warp & 3, half = (warp - 4) >> 2;
    OutDesc o = p.out;
    o.tma_c = (Lay::STAGING_BYTES > 0 && p.use_tma_store) ? &p.tma_c : nullptr;
    const uint32_t staging = staging0 + (warp - 4) * 2 * kStageOutBytes;
    uint32_t it = 0, chunk = 0;
    bool ok = true;
    for (int tile = first_tile; ok && tile < p.num_tiles; tile += stride) {
      TileCoord tc = decode_tile(tile, p.m_tiles, p.n_tiles);
      tc.mb = 2 * tc.mb + (int)crank;
      tc.nb = 2 * tc.nb + half;  // in units of HALF columns
      const int m0 = tc.mb * kBM + q * 32, n0 = tc.nb * HALF;
      const int n_left = p.N - n0;
      const bool live = m0 < p.M && n_left > 0;  // any output here
      TileBias<HALF> tb;
      if (live) load_tile_bias<HALF>(o, 0, m0 + lane, n0, lane, tb);
      const float* sa = p.sa + (int64_t)min(m0 + lane, p.M - 1) * p.sa_m;
      const float* sb = p.sb + (int64_t)(min(n0, p.N - 1) / 128) * p.sb_n;
      // The scales of kGroup blocks are loaded while the group before is summed: a
      // product with one just requested would hold the warp for its latency.
      float sa_next[kGroup], sb_next[kGroup];
      auto request_scales = [&](int kb0) {
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
          const bool there = live && kb0 + j < p.k_blocks;
          sa_next[j] = there ? __ldg(sa + (kb0 + j) * p.sa_k) : 0.0f;
          sb_next[j] = there ? __ldg(sb + (kb0 + j) * p.sb_k) : 0.0f;
        }
      };
      request_scales(0);
      float acc[HALF];
#pragma unroll
      for (int i = 0; i < HALF; ++i) acc[i] = 0.0f;
      for (int kb0 = 0; ok && kb0 < p.k_blocks; kb0 += kGroup) {
        float scale[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j) scale[j] = __fmul_rn(sa_next[j], sb_next[j]);
        request_scales(kb0 + kGroup);
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
          if (kb0 + g >= p.k_blocks) break;
          const uint32_t buf = it % ACC, use = it / ACC;
          const float s = scale[g];
          ++it;
          const bool got = mbar_wait_bounded(bars.tfull(buf), use & 1, wc.abort, wc.status_word, wc.limit_ns,
                                             status_code(6, kSiteEpilogueTmemFull));
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t src = tmem_base + ((uint32_t)(q * 32) << 16) + buf * BN + half * HALF;
          uint32_t va[32], vb[32];
          if (live) tmem_load_32cols(src, va);
#pragma unroll
          for (int j = 0; j < HALF / 32; ++j) {
            uint32_t(&v)[32] = j & 1 ? vb : va;
            uint32_t(&w)[32] = j & 1 ? va : vb;
            if (live) {
              tmem_load_wait(v);
              if (j + 1 < HALF / 32) tmem_load_32cols(src + (j + 1) * 32, w);
            }
            if (j + 1 == HALF / 32) {  // all of it is in registers: the accumulator is free
              tc_fence_before_sync();
              __syncwarp();
              if (lane == 0) {
                if (crank != 0)
                  mbar_arrive_remote(bars.tempty(buf), 0);
                else
                  mbar_arrive(bars.tempty(buf));
              }
            }
            if (live) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) fma2(acc[32 * j + i], acc[32 * j + i + 1], v[i], v[i + 1], s);
            }
          }
        }
      }
      if (!ok) break;
      if (live) {
#pragma unroll
        for (int j = 0; j < HALF / 32; ++j) {
          if (32 * j < n_left) {
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(acc[32 * j + i]);
            epilogue_chunk<HALF>(o, j, tb, v, tc, m0, lane, true, staging, chunk);
          }
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
  constexpr int kSlot = 104 + (BN == 256 ? 0 : BN == 128 ? 3 : 6);
  if (p.M <= kShortARows) return launch_variant<BN, kShortARows, true>(p, stream, kSlot);
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
  // The widest tile that still gives every pair of SMs one.
  const int64_t pairs = dev.num_sms / 2;
  auto tiles = [&](int64_t bn) { return (int64_t)p.m_tiles * ((g.N + bn - 1) / bn); };
  const int bn = tiles(256) >= pairs ? 256 : tiles(128) >= pairs ? 128 : 64;
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
  p.use_tma_store = encode_output_map(&p.tma_c, g.c, o.out_f32 != 0, o.out_f16 != 0, 1, g.M, g.N, g.ldc, 0) ? 1 : 0;
  p.status_word = dev.status_word;
  p.wait_limit_ns = kWaitLimitNs;
  const cudaError_t e = bn == 256 ? launch_width<256>(p, stream) : bn == 128 ? launch_width<128>(p, stream) : launch_width<64>(p, stream);
  if (e != cudaSuccess) {
    *why = std::string("block-scaled product launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
