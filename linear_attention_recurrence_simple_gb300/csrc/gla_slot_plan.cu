// One serving step's maps, built on the device from the requests' lengths: which pool row each request has,
// where its tokens lie in the packed batch, and each packed token's request and place.
//
// The maps are those of the sequential rule (requests in order; a request without a row takes the lowest
// free one; tokens are handed out until the budget is used up), computed in parallel:
//   rows    a bitmap of the rows in use; the i-th request that wants a row has the i-th free one (if there are
//           that many), found by a search over the running counts of free rows of the bitmap's words
//   tokens  a running sum of the lengths, cut off at the budget.  Once the budget is used up nothing after it has
//           tokens, so no row has to be given back for want of tokens
// One launch: every CTA computes the whole plan (a few microseconds, bound by latency: another launch, or a wait for another
// CTA, would cost as much) and writes its share of the tokens' places from the offsets in its shared memory; the first
// one writes the requests' maps.  Batches whose offsets do not fit there have a second launch for the tokens.
// 48 requests and 2,048 tokens take 8 us, 5,000 requests and 65,536 tokens 18 (of a call's 24 to 32 with its binding); as two
// launches 34.
#include "gla_delta.cuh"
#include "gla_once.cuh"

namespace gla {
namespace {

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int KEEP = 8;             // requests that a thread keeps in registers
constexpr int TOKENS = 4 * THREADS; // tokens of a CTA, at least
constexpr int SMEM_MAX = 200 * 1024;

// Exclusive running sum over the block's threads, and the total.  `warp_sums` is used once.
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
  long long w = warp_sums[lane];  // (every warp sums all of them)
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += up;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp ? before : 0) + run - x;
}

struct Request {
  int want;  // tokens it would have
  int held;  // its row, -1: none; -2: one that there is not
  __device__ __forceinline__ bool has() const { return held >= 0; }
  bool keeps, asks;
};
__device__ __forceinline__ Request request_of(int len, int h, int rows, int budget) {
  Request r;
  r.held = h >= -1 && h < rows ? h : -2;
  r.keeps = len >= 0 && r.has();
  r.asks = len > 0 && h == -1;
  r.want = r.asks || (r.keeps && len > 0) ? min(len, budget) : 0;
  return r;
}

__device__ __forceinline__ void token_place(const int32_t* cu, const int32_t* seen, int N, int budget, int t, int32_t* token_seq,
                                            int32_t* token_pos, unsigned* err) {
  int seq = -1, pos = -1;
  if (!GLA_IN_BOUNDS(t >= 0 && t < budget, err)) return;
  if (t < cu[N]) {
    int lo = 0, hi = N - 1;  // the first request whose end is behind t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (cu[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    if (!GLA_IN_BOUNDS(N > 0 && lo >= 0 && lo < N && t >= cu[lo] && t < cu[lo + 1], err)) return;
    seq = lo;
    pos = (seen ? seen[lo] : 0) + t - cu[lo];
  }
  token_seq[t] = seq;
  token_pos[t] = pos;
}

// `ends`: the offsets are kept in shared memory and this CTA's tokens are written from there.
// held and row may be the same array (no __restrict__): a thread reads a request's held, the last time too, before it writes
// that request's row.
__global__ void __launch_bounds__(THREADS, 1)
slot_plan_kernel(const int32_t* __restrict__ new_len, const int32_t* held, const int32_t* __restrict__ seen, int N,
                 int rows, int budget, int32_t* __restrict__ cu, int32_t* __restrict__ slot, int32_t* __restrict__ start,
                 int32_t* row, int32_t* __restrict__ token_seq, int32_t* __restrict__ token_pos, bool ends, unsigned* err) {
  extern __shared__ uint32_t sm[];
  __shared__ long long sums[2][WARPS];
  const int tid = threadIdx.x, words = (rows + 31) / 32;
  const bool writes = blockIdx.x == 0;
  uint32_t* const used = sm;            // bit set: the row is held
  uint32_t* const before = sm + words;  // free rows of the words before
  int32_t* const s_cu = reinterpret_cast<int32_t*>(before + words);
  // each thread has consecutive requests, the first KEEP of them in registers
  const int per = (N + THREADS - 1) / THREADS, n0 = min(N, tid * per), count = min(N, n0 + per) - n0;
  int len[KEEP], has[KEEP];
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    len[i] = i < count ? new_len[n0 + i] : 0;
    has[i] = i < count ? held[n0 + i] : -1;
  }
  for (int w = tid; w < words; w += THREADS) used[w] = w == words - 1 && rows % 32 ? ~0u << (rows % 32) : 0u;
  __syncthreads();
  // f(i, request) for this thread's requests, in order
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (i < count) f(n0 + i, request_of(len[i], has[i], rows, budget));
    for (int i = KEEP; i < count; ++i) f(n0 + i, request_of(new_len[n0 + i], held[n0 + i], rows, budget));
  };
  long long asks = 0;
  each([&](int, const Request& r) {
    asks += r.asks;
    if (r.held == -2 && writes) raise_error(err, ERR_SHAPE);
    if (r.keeps) {
      const uint32_t bit = 1u << (r.held & 31);
      if ((atomicOr(&used[r.held >> 5], bit) & bit) && writes) raise_error(err, ERR_SHAPE);  // two requests with one row
    }
  });
  __syncthreads();
  const int wper = (words + THREADS - 1) / THREADS, w0 = min(words, tid * wper), w1 = min(words, w0 + wper);
  long long free_rows = 0, total;
  for (int w = w0; w < w1; ++w) free_rows += __popc(~used[w]);
  // both counts are below 2^21: one scan
  const long long at = block_scan(asks << 32 | free_rows, sums[0], total);
  const int all_free = (int)(uint32_t)total;
  const int rank = (int)(at >> 32);
  uint32_t run = (uint32_t)at;
  for (int w = w0; w < w1; ++w) {
    before[w] = run;
    run += __popc(~used[w]);
  }
  long long tokens = 0;
  int rk = rank;
  each([&](int, const Request& r) {
    if (r.asks ? rk < all_free : r.keeps) tokens += r.want;
    rk += r.asks;
  });
  long long end = block_scan(tokens, sums[1], total);  // (its barrier also completes `before`)
  const int handed = (int)min(total, (long long)budget);
  rk = rank;
  each([&](int n, const Request& r) {
    const int i = rk;
    rk += r.asks;
    const int begin = (int)min(end, (long long)budget);
    if (r.asks ? i < all_free : r.keeps) end += r.want;
    const bool got = min(end, (long long)budget) > begin;
    if (ends) s_cu[n] = begin;
    if (!writes) return;
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
      if (!GLA_IN_BOUNDS(lo >= 0 && lo < words && bits != 0 && mine < rows, err)) mine = -1;
    }
    cu[n] = begin;
    row[n] = mine;
    slot[n] = got ? mine : -1;
    start[n] = got && r.keeps ? r.held : -1;
  });
  if (tid == 0) {
    if (ends) s_cu[N] = handed;
    if (writes) cu[N] = handed;
  }
  if (!ends) return;
  __syncthreads();
  for (int t = blockIdx.x * THREADS + tid; t < budget; t += gridDim.x * THREADS)  // (below 2^31: GLA_PLAN_MAX_BUDGET)
    token_place(s_cu, seen, N, budget, t, token_seq, token_pos, err);
}

__global__ void __launch_bounds__(256)
slot_plan_tokens_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ seen, int N, int budget,
                        int32_t* __restrict__ token_seq, int32_t* __restrict__ token_pos, unsigned* err) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t < budget) token_place(cu, seen, N, budget, t, token_seq, token_pos, err);
}

}  // namespace

cudaError_t launch_slot_plan(const int32_t* new_len, const int32_t* held, const int32_t* seen, int N, int rows, int budget,
                             int32_t* cu, int32_t* slot, int32_t* start, int32_t* row, int32_t* token_seq, int32_t* token_pos,
                             unsigned* err, cudaStream_t st) {
  static OncePerDevice<CudaDeviceApi> once;
  const cudaError_t e = once([] { return cudaFuncSetAttribute(slot_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX); });
  if (e != cudaSuccess) return e;
  const bool tokens = budget > 0 && token_seq;
  const int maps = ((rows + 31) / 32) * 8, with_ends = maps + (N + 1) * 4;  // (maps: 128 KB at most)
  const bool ends = tokens && with_ends <= SMEM_MAX;
  // Where row is held, a CTA that runs late must not find what the first one wrote: one CTA.
  const unsigned ctas = ends && row != held ? (unsigned)min(64, (budget + TOKENS - 1) / TOKENS) : 1u;
  slot_plan_kernel<<<ctas, THREADS, ends ? with_ends : maps, st>>>(new_len, held, seen, N, rows, budget, cu, slot, start, row, token_seq,
                                                                   token_pos, ends, err);
  if (tokens && !ends) slot_plan_tokens_kernel<<<(budget + 255) / 256, 256, 0, st>>>(cu, seen, N, budget, token_seq, token_pos, err);
  return cudaGetLastError();
}

}  // namespace gla
