// bi_plan.cu -- block tables and slot maps of a paged key-value cache, built
// on the GPU from request lengths.
//
// Request b holds ceil(ctx_b / ps) pages and needs ceil((ctx_b + add_b) / ps);
// the difference is taken from the pool in request order, so request b's
// first new page is pool[start_b] with start the exclusive prefix sum of the
// differences, and token t of request b (t counted from the exclusive prefix
// sum of add) sits at position ctx_b + t - offset_b.
//
// One launch, no scratch and no atomics: every block computes the prefix sums
// of the whole batch for itself (8 bytes a request, out of L2) and then takes
// its share of the tokens and of the new pages, each found in the prefix sums
// by a binary search.  The work is a few bytes a token, so what bounds the
// call is its chain of dependent loads: lengths -> prefix sums -> page -> slot.
#include "bi_launch.h"
#include "bi_serve.h"

namespace bi {
namespace {

__device__ __forceinline__ int32_t sat32(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int32_t)v; }

// ceil(n / ps) in 32 bits
__device__ __forceinline__ int64_t pages_of(uint32_t n, uint32_t ps) { return n ? (int64_t)((n - 1) / ps) + 1 : 0; }

struct Req {
  int64_t ctx, add, held, take;
};
// A request's lengths (negative ones count as zero) and pages.
__device__ __forceinline__ Req load_req(const PlanParams& p, int b) {
  Req r;
  r.ctx = max(0, __ldg(p.ctx + b));
  r.add = max(0, __ldg(p.add + b));
  r.held = pages_of((uint32_t)r.ctx, (uint32_t)p.ps);
  r.take = pages_of((uint32_t)(r.ctx + r.add), (uint32_t)p.ps) - r.held;  // the sum fits 32 bits unsigned
  return r;
}

// Inclusive block scan of (a, b) over NT threads; sh: 2 * NT / 32 values.
template <int NT>
__device__ __forceinline__ void block_scan(int64_t& a, int64_t& b, int64_t* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += x, b += y;
  }
  if (lane == 31) sh[w] = a, sh[NT / 32 + w] = b;
  __syncthreads();
  for (int i = 0; i < w; ++i) a += sh[i], b += sh[NT / 32 + i];
}

// Last index i in [0, n) with at[i] <= v (at ascending, at[0] == 0).
template <typename I>
__device__ __forceinline__ int find_last(const I* at, int n, I v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Thread i of a block owns the requests [i * per, (i + 1) * per): their sums
// are what the searches run over; with more requests than threads the rest of
// the way to a request is walked.
template <int NT>
__global__ void __launch_bounds__(NT) plan_kernel(const PlanParams p) {
  __shared__ int64_t sh[2 * NT / 32];
  __shared__ int32_t tok_at[NT];
  __shared__ int64_t page_at[NT];
  const int per = (p.B + NT - 1) / NT;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  int64_t tok = 0, pages = 0;
  for (int b = b0; b < b1; ++b) {
    const Req r = load_req(p, b);
    tok += r.add, pages += r.take;
  }
  const int64_t own_tok = tok, own_pages = pages;
  block_scan<NT>(tok, pages, sh);
  tok_at[threadIdx.x] = sat32(tok - own_tok);
  page_at[threadIdx.x] = pages - own_pages;
  int64_t all_tok = 0, all_pages = 0;
  for (int i = 0; i < NT / 32; ++i) all_tok += sh[i], all_pages += sh[NT / 32 + i];
  __syncthreads();
  if (blockIdx.x == 0) {
    int64_t at = tok - own_tok;
    for (int b = b0; b < b1; ++b) {
      const Req r = load_req(p, b);
      p.offsets[b] = sat32(at);
      p.seq_lens[b] = sat32(r.ctx + r.add);
      at += r.add;
    }
    if (threadIdx.x == 0) {
      p.offsets[p.B] = sat32(all_tok);
      p.totals[0] = sat32(all_pages);
      p.totals[1] = sat32(all_tok);
    }
  }
  const int used = (p.B + per - 1) / max(per, 1);  // threads that own requests
  const int32_t first = (int32_t)(blockIdx.x * NT + threadIdx.x), step = (int32_t)(gridDim.x * NT);
  // new pages; those past a row's last column (lengths that no table can hold)
  // are stepped over a request at a time
  for (int64_t e = first; e < all_pages; e += step) {
    const int i = find_last(page_at, used, e);
    int64_t at = page_at[i];
    int b = i * per;
    Req r = load_req(p, b);
    while (e >= at + r.take) at += r.take, r = load_req(p, ++b);
    const int64_t col = r.held + (e - at);
    if (col < p.W)
      p.table[b * p.ld_table + col] = e < p.F ? __ldg(p.pool + e) : -1;
    else
      e += (at + r.take - 1 - e) / step * step;
  }
  // tokens
  for (int64_t t = first; t < p.T; t += step) {
    if (t >= all_tok) {
      p.positions[t] = 0;
      p.slots[t] = -1;
      continue;
    }
    const int i = find_last(tok_at, used, (int32_t)t);
    int64_t at = tok_at[i], pg = page_at[i];
    int b = i * per;
    Req r = load_req(p, b);
    while (t >= at + r.add) at += r.add, pg += r.take, r = load_req(p, ++b);
    const int64_t pos = r.ctx + (t - at);
    const uint32_t col = (uint32_t)pos / (uint32_t)p.ps, row = (uint32_t)pos % (uint32_t)p.ps;
    int32_t page = -1;
    if (col < (uint32_t)p.W) {
      if (col < r.held) {
        page = p.table[b * p.ld_table + col];  // only columns from `held` on are written by this launch
      } else {
        const int64_t e = pg + (col - r.held);
        if (e < p.F) page = __ldg(p.pool + e);
      }
    }
    p.positions[t] = sat32(pos);
    p.slots[t] = page < 0 ? -1 : (int64_t)page * p.ps + row;
  }
}

}  // namespace

bi_status launch_plan(const PlanParams& p, cudaStream_t stream, std::string* why) {
  DeviceInfo dev;
  const bi_status st = current_device_info(&dev, why);
  if (st != BI_OK) return st;
  // 256 threads own a batch of up to 256 requests one each; larger batches
  // take 1024.  Two tokens a thread, at most two blocks per SM.
  const int nt = p.B <= 256 ? 256 : 1024;
  const int64_t want = std::max<int64_t>(1, ((int64_t)p.T + 2 * nt - 1) / (2 * nt));
  const unsigned grid = (unsigned)std::min<int64_t>(want, 2 * (int64_t)dev.num_sms);
  if (nt == 256)
    plan_kernel<256><<<grid, 256, 0, stream>>>(p);
  else
    plan_kernel<1024><<<grid, 1024, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *why = std::string("page plan launch: ") + cudaGetErrorString(e);
    return BI_ERR_CUDA;
  }
  return BI_OK;
}

}  // namespace bi
