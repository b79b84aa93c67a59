// The gated delta rule: what its kernels share (arguments, chunk places, decays of a chunk).
//
// Per head, with a decay a_t = exp(g_t) and a strength beta_t of every token's own,
//     S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t x_t,   x_t = v_t - a_t S_{t-1}^T k_t,   o_t = S_t^T (scale q_t).
// For a chunk of C tokens, S0 the state before it, G_i = g_1 + .. + g_i, B = diag(beta):
//     D_ij = exp(G_i - G_j) for j <= i, else 0,   P = QK^T . D,   M = KK^T . D without its diagonal
//     R = V - diag(e^G) K S0,   (1 + M B) X = R,   U = B X
//     O = s (diag(e^G) Q S0 + P U),   S1 = e^(G_C) S0 + (diag(e^(G_C - G)) K)^T U
// The inverse is kept as Z = (1 + M B)^-1 M, strictly lower triangular: X = R - Z B R, so that the large part
// of X is R itself, and its transpose serves the backward, dR = B (dU - Z^T B dU), without a division by beta.
// Decays enter as exp of a difference of sums, never as e^G_i times e^-G_j: g = -inf (a reset) and long runs of
// strong decay neither overflow nor lose what is left after them.
#pragma once

#include "gla_common.cuh"

namespace gla {

constexpr int DC = 64;  // tokens of a chunk

struct DeltaArgs {
  const void *q, *k, *v, *g, *beta;
  const void* dO;            // backward
  const float* h0;           // may be null: zeros
  const int32_t* h0_row;     // row of h0 that each sequence starts from (-1: zeros), or null: row n
  int h0_rows;
  const float* dhT;          // backward; may be null
  void* o;                   // forward
  float* hT;                 // forward; may be null
  const int32_t* hT_row;     // row of hT that each sequence's final state goes to (-1: none), or null: row n
  int hT_rows;
  void *dq, *dk, *dv, *dg, *dbeta;  // backward
  float* dh0;                       // backward; may be null
  const int32_t* cu_seqlens;        // null: fixed length T
  float scale;
  int n_seq;
  int T;                     // per-sequence length (fixed) or packed total
  int H;
  int slots;                 // chunk places of the call (see chunk_of_slot)
  unsigned* err;
  unsigned long long wait_ns;
  uint8_t* ws;               // workspace
  int32_t* order;            // sequences from the longest on (tensor-core kernels, packed calls), or null
};

// Places for the chunks of a call: sequence n's begin at base(n) = begin / C + n, which leaves room for
// every sequence's ragged last chunk without anything to be summed up (base(n + 1) - base(n) is at least its
// number of chunks); some places stay empty.
__host__ __device__ inline long long delta_slots(int n_seq, int T, bool packed) {
  return packed ? (long long)T / DC + n_seq : (long long)n_seq * (((long long)T + DC - 1) / DC);
}

struct DeltaSeq {
  long long begin;
  int len;
  int slot0;  // place of its first chunk
};
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaArgs& a, int n) {
  DeltaSeq s;
  if (a.cu_seqlens) {
    const long long b = a.cu_seqlens[n], e = a.cu_seqlens[n + 1];
    s.begin = min(max(b, 0ll), (long long)a.T);
    const long long end = min(max(e, s.begin), (long long)a.T);
    if (s.begin != b || end != e) raise_error(a.err, ERR_SHAPE);
    s.len = (int)(end - s.begin);
    s.slot0 = (int)(s.begin / DC) + n;
  } else {
    s.begin = (long long)n * a.T;
    s.len = a.T;
    s.slot0 = n * ((a.T + DC - 1) / DC);
  }
  if (!GLA_IN_BOUNDS(s.len == 0 || (s.begin >= 0 && s.begin + s.len <= (a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T) &&
                                    s.slot0 >= 0 && s.slot0 + (s.len + DC - 1) / DC <= a.slots), a.err))
    s.len = 0;
  return s;
}
// The sequence of a scan's rank-th unit.
__device__ __forceinline__ int delta_unit(const DeltaArgs& a, int rank) {
  int n = a.order && GLA_IN_BOUNDS(rank < a.n_seq, a.err) ? a.order[rank] : rank;
  if (!GLA_IN_BOUNDS(n >= 0 && n < a.n_seq, a.err)) n = 0;
  return n;
}

// The chunk at a place: its first token and its tokens (0: the place is empty).  Whole warps.
struct DeltaChunk {
  long long t0;
  int len;
};
__device__ __forceinline__ DeltaChunk chunk_of_slot(const DeltaArgs& a, int slot) {
  int n;
  if (a.cu_seqlens) {
    // the last sequence with slot0 <= slot: 32 candidates a look
    const int lane = threadIdx.x & 31;
    int lo = 0, step = 1;
    while ((long long)32 * step < a.n_seq) step *= 32;
    for (;; step /= 32) {
      const long long at = lo + (long long)lane * step;
      bool below = false;
      if (at < a.n_seq) below = min(max(a.cu_seqlens[at], 0), a.T) / DC + (int)at <= slot;
      const unsigned v = __ballot_sync(0xffffffffu, below);  // (a run of ones: slot0 grows with n)
      lo += max(__popc(v) - 1, 0) * step;
      if (step == 1) break;
    }
    n = min(lo, a.n_seq - 1);
  } else {
    n = slot / ((a.T + DC - 1) / DC);
  }
  const DeltaSeq s = delta_seq(a, n);
  const long long off = (long long)(slot - s.slot0) * DC;
  DeltaChunk c;
  c.t0 = s.begin + off;
  c.len = off < 0 || off >= s.len ? 0 : (int)min((long long)DC, s.len - off);
  if (!GLA_IN_BOUNDS(c.len == 0 || (c.t0 >= 0 && c.t0 + c.len <= (a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T)), a.err))
    c.len = 0;
  return c;
}

// A call's kernels follow each other without the gap of a launch: CTAs of the next one take the places that the last CTAs
// of this one leave, and wait for its end (and so for all before it) before they read anything (backward, fp32, 2 x 150
// tokens x 4 heads: 129 -> 123 us; bf16, 40 packed sequences x 16 heads: 570 -> 558 us; a call for the next kernel at
// the start of a CTA is slower, 132 and 561 us: what comes early takes room from what runs).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Row of a [rows, H, 96, 192] array that sequence n has: -1 where it has none.
__device__ __forceinline__ int delta_row(const int32_t* row, int rows, int n, unsigned* err) {
  if (!row) return n;
  const int r = row[n];
  if (r >= 0 && r < rows) return r;
  if (r != -1) raise_error(err, ERR_SHAPE);
  return -1;
}

// Packed rows of no sequence (in front of the first offset, behind the last): nothing depends on them, so their gradients
// are zero.  Place p has rows 64 p .. of the packed array (there are at least as many places as that takes).  Whole CTA.
template <class T>
__device__ __noinline__ void zero_spare_rows(const DeltaArgs& a, int place, int h) {
  if (!a.cu_seqlens) return;
  const int first = min(max(a.cu_seqlens[0], 0), a.T), last = min(max(a.cu_seqlens[a.n_seq], 0), a.T);
  const long long t0 = (long long)place * DC, t1 = min(t0 + DC, (long long)a.T);
  if (t0 >= first && t1 <= last) return;
  const int lane = threadIdx.x & 31;
  constexpr int KV = DK * (int)sizeof(T) / 16, VV = DV * (int)sizeof(T) / 16;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (long long t = t0 + threadIdx.x / 32; t < t1; t += blockDim.x / 32) {
    if (t >= first && t < last) continue;
    const long long row = t * a.H + h;
    if (!GLA_IN_BOUNDS(row >= 0 && row < (long long)a.T * a.H, a.err)) continue;
    for (int e = lane; e < VV; e += 32) {
      if (e < KV) reinterpret_cast<uint4*>((T*)a.dq + row * DK)[e] = reinterpret_cast<uint4*>((T*)a.dk + row * DK)[e] = zero;
      reinterpret_cast<uint4*>((T*)a.dv + row * DV)[e] = zero;
    }
    if (lane == 0) ((T*)a.dg)[row] = ((T*)a.dbeta)[row] = from_f<T>(0.f);
  }
}

// Running sums of a chunk's log decays, each as two fp32 (hi + lo): a difference of two of them keeps 24 bits
// of what is left between them, whatever was decayed before.  Summed as whole numbers of 2^-40 (fp64 adds are slow
// here), so that a sum is off by 64 2^-41 at most.  Whole warp; x0, x1 are the log decays of tokens 2 lane and
// 2 lane + 1.  Values below -120 count as -120: exp of it is zero in fp32.
constexpr float LOG_FLOOR = -120.f;
constexpr float LOG_CEIL = 16384.f;  // (exp of it is an infinity; the sums stay within 63 bits)
template <bool BASE2 = false>  // sums of the logs to base 2
__device__ __forceinline__ long long delta_fixed(float x) {
  const float one = 1099511627776.f;  // 2^40
  x = fminf(fmaxf(x, LOG_FLOOR), LOG_CEIL);
  if (!BASE2) return __float2ll_rn(x * one);
  const float hi = x * 1.44269502f, lo = fmaf(x, 1.92596303e-8f, fmaf(x, 1.44269502f, -hi));  // log2(e) in two
  return __float2ll_rn(hi * one) + __float2ll_rn(lo * one);
}
__device__ __forceinline__ float2 delta_two(long long x, float bad) {
  const float hi = __ll2float_rn(x);
  const float lo = __ll2float_rn(x - __float2ll_rn(hi));
  return make_float2(fmaf(hi, 9.094947017729282e-13f, bad), lo * 9.094947017729282e-13f);
}
template <bool BASE2 = false>
__device__ __forceinline__ void delta_sums(float x0, float x1, float2& s0, float2& s1) {
  const long long d0 = delta_fixed<BASE2>(x0), d1 = delta_fixed<BASE2>(x1);
  // NaN from a token on where it is NaN, or +inf
  const float bad0 = x0 > LOG_FLOOR ? 0.f * x0 : x0 <= LOG_FLOOR ? 0.f : x0, bad1 = x1 > LOG_FLOOR ? 0.f * x1 : x1 <= LOG_FLOOR ? 0.f : x1;
  long long run = d0 + d1;
  float bad = bad0 + bad1;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, run, off);
    const float b = __shfl_up_sync(0xffffffffu, bad, off);
    if ((int)(threadIdx.x & 31) >= off) {
      run += up;
      bad += b;
    }
  }
  const float before = __shfl_up_sync(0xffffffffu, bad, 1);
  s0 = delta_two(run - d1, ((threadIdx.x & 31) ? before : 0.f) + bad0);
  s1 = delta_two(run, bad);
}
// exp(G_i - G_j)
__device__ __forceinline__ float delta_decay(float2 gi, float2 gj) { return expf((gi.x - gj.x) + (gi.y - gj.y)); }
__device__ __forceinline__ float delta_decay0(float2 gi) { return expf(gi.x + gi.y); }

int current_device_state(unsigned** err, unsigned long long* wait_ns);
cudaError_t launch_delta_simt_fwd(const DeltaArgs& a, cudaStream_t stream);
cudaError_t launch_delta_simt_bwd(const DeltaArgs& a, cudaStream_t stream);
cudaError_t launch_delta_tc_fwd(DeltaArgs a, cudaStream_t stream);
cudaError_t launch_delta_tc_bwd(DeltaArgs a, cudaStream_t stream);
size_t delta_tc_ws_bytes(int n_seq, long long slots, long long tokens, int H, bool bwd);
size_t delta_simt_ws_bytes(long long slots, long long tokens, int H, bool bwd);

}  // namespace gla
