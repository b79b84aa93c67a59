// One serving step's maps, built on the device from the requests' lengths: which pool row each request has,
// where its tokens lie in the packed batch, and each packed token's request and place.
//
// The maps are those of the sequential rule (requests in order; a request without a row takes the lowest
// free one; tokens are handed out until the budget is used up), computed in parallel:
//   rows    a bitmap of the rows in use; the i-th request that wants a row has the i-th free one (if there are
//           that many), found by a search over the running counts of free rows of the bitmap's words
//   tokens  a running sum of the lengths, cut off at the budget.  Once the budget is used up nothing after it has
//           tokens, so no row has to be given back for want of tokens
// Two launches (one CTA for the requests, then one thread a token of the budget), bound by their latency.
#include "gla_delta.cuh"
#include "gla_once.cuh"

namespace gla {
namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;

// Exclusive running sum over the block's threads, and the total.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long run = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, run, off);
    if (lane >= off) run += up;
  }
  if (lane == 31) warp_sums[warp] = run;
  __syncthreads();
  if (warp == 0) {
    long long w = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += up;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[WARPS - 1];
  const long long before = (warp ? warp_sums[warp - 1] : 0) + run - x;
  __syncthreads();
  return before;
}

struct Request {
  int want;   // tokens it would have
  int held;   // its row, -1: none
  bool keeps, asks;
};
__device__ __forceinline__ Request request_at(const int32_t* new_len, const int32_t* held, int n, int rows, int budget) {
  Request r;
  const int len = new_len[n], h = held[n];
  r.held = h >= 0 && h < rows ? h : -1;
  r.keeps = len >= 0 && r.held >= 0;
  r.asks = len > 0 && h == -1;
  r.want = r.asks || (r.keeps && len > 0) ? min(len, budget) : 0;
  return r;
}

__global__ void __launch_bounds__(THREADS, 1)
slot_plan_kernel(const int32_t* __restrict__ new_len, const int32_t* __restrict__ held, int N, int rows, int budget,
                 int32_t* __restrict__ cu, int32_t* __restrict__ slot, int32_t* __restrict__ start, int32_t* __restrict__ row,
                 unsigned* err) {
  extern __shared__ uint32_t sm[];
  __shared__ long long sums[WARPS];
  const int tid = threadIdx.x, words = (rows + 31) / 32;
  uint32_t* const used = sm;           // bit set: the row is held
  uint32_t* const before = sm + words; // free rows of the words before
  for (int w = tid; w < words; w += THREADS) used[w] = w == words - 1 && rows % 32 ? ~0u << (rows % 32) : 0u;
  __syncthreads();
  // each thread has consecutive requests
  const int per = (N + THREADS - 1) / THREADS, n0 = min(N, tid * per), n1 = min(N, n0 + per);
  long long asks = 0, total;
  for (int n = n0; n < n1; ++n) {
    const Request r = request_at(new_len, held, n, rows, budget);
    asks += r.asks;
    if (r.held < 0 && held[n] != -1) raise_error(err, ERR_SHAPE);
    if (r.keeps) {
      const uint32_t bit = 1u << (r.held & 31);
      if (atomicOr(&used[r.held >> 5], bit) & bit) raise_error(err, ERR_SHAPE);  // two requests with one row
    }
  }
  long long rank = block_scan(asks, sums, total);  // (its first barrier also ends the bitmap's updates)
  const int wper = (words + THREADS - 1) / THREADS, w0 = min(words, tid * wper), w1 = min(words, w0 + wper);
  long long free_rows = 0, all_free;
  for (int w = w0; w < w1; ++w) free_rows += __popc(~used[w]);
  long long run = block_scan(free_rows, sums, all_free);
  for (int w = w0; w < w1; ++w) {
    before[w] = (uint32_t)run;
    run += __popc(~used[w]);
  }
  long long tokens = 0, rk = rank;
  for (int n = n0; n < n1; ++n) {
    const Request r = request_at(new_len, held, n, rows, budget);
    if (r.asks ? rk++ < all_free : r.keeps) tokens += r.want;
  }
  long long end = block_scan(tokens, sums, total);  // (and `before` is complete)
  rk = rank;
  for (int n = n0; n < n1; ++n) {
    const Request r = request_at(new_len, held, n, rows, budget);
    const long long i = rk;
    rk += r.asks;
    const long long begin = min(end, (long long)budget);
    if (r.asks ? i < all_free : r.keeps) end += r.want;
    const bool got = min(end, (long long)budget) > begin;
    int mine = r.keeps ? r.held : -1;
    if (r.asks && got) {
      int lo = 0, hi = words - 1;  // the last word with before <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (before[mid] <= (uint32_t)i) lo = mid; else hi = mid - 1;
      }
      uint32_t bits = ~used[lo];
      for (uint32_t skip = (uint32_t)i - before[lo]; skip > 0; --skip) bits &= bits - 1;
      mine = 32 * lo + __ffs((int)bits) - 1;
    }
    cu[n] = (int)begin;
    row[n] = mine;
    slot[n] = got ? mine : -1;
    start[n] = got && r.keeps ? r.held : -1;
    if (n == N - 1) cu[N] = (int)min(end, (long long)budget);
  }
  if (N == 0 && tid == 0) cu[0] = 0;
}

__global__ void __launch_bounds__(256)
slot_plan_tokens_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ seen, int N, int budget,
                        int32_t* __restrict__ token_seq, int32_t* __restrict__ token_pos) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= budget) return;
  int seq = -1, pos = -1;
  if (t < cu[N]) {
    int lo = 0, hi = N - 1;  // the first request whose end is behind t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    seq = lo;
    pos = (seen ? seen[lo] : 0) + t - cu[lo];
  }
  token_seq[t] = seq;
  token_pos[t] = pos;
}

}  // namespace

int slot_plan_smem(int rows) { return ((rows + 31) / 32) * 8; }

cudaError_t launch_slot_plan(const int32_t* new_len, const int32_t* held, const int32_t* seen, int N, int rows, int budget,
                             int32_t* cu, int32_t* slot, int32_t* start, int32_t* row, int32_t* token_seq, int32_t* token_pos,
                             unsigned* err, cudaStream_t st) {
  static OncePerDevice<CudaDeviceApi> once;
  const cudaError_t e = once([] {
    return cudaFuncSetAttribute(slot_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, slot_plan_smem(1 << 19));
  });
  if (e != cudaSuccess) return e;
  slot_plan_kernel<<<1, THREADS, slot_plan_smem(rows), st>>>(new_len, held, N, rows, budget, cu, slot, start, row, err);
  if (budget > 0 && token_seq)
    slot_plan_tokens_kernel<<<(budget + 255) / 256, 256, 0, st>>>(cu, seen, N, budget, token_seq, token_pos);
  return cudaGetLastError();
}

}  // namespace gla
