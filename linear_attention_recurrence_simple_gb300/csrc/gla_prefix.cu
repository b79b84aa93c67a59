// Sequences that continue a shared prefix.
//
// "Beyond the KV cache" (Laplace 3B on Trainium2), section "i14 and the Laplace 3B architecture", GLA
// mixer: S_t = lambda S_{t-1} + k_t v_t^T, o_t = S_t^T (scale q_t).  The recurrence is linear in its
// initial state, so a prefix that many sequences share enters each of them only through one state
// S_p = S after the prefix, computed once; sequence n with the L tokens (k_j, v_j) after it has
//     o = scale (lambda^(L+1) S_p^T q + sum_j lambda^(L-j) (q . k_j) v_j + (q . k) v)
// at its next token (q, k, v).  A decode step over states of their own streams 147 KB (read and
// write) per (sequence, head); this form reads every shared state once for all its sequences and
// 576 bytes (bf16) or 297 (MXFP8) per tail token.
#include <algorithm>
#include <atomic>

#include "gla_tail.cuh"

namespace gla {

int current_device_state(unsigned** err, unsigned long long* wait_ns);
int check_chunk_sizes(int n_seq, int T, int H, int dk, int dv, int dtype, const int32_t* cu_seqlens, long long* tokens);
cudaError_t launch_lpt_order(const int32_t* cu_seqlens, int n_seq, int32_t* order, cudaStream_t stream);
cudaError_t launch_simt_fwd(const ChunkArgs& a, cudaStream_t stream);
cudaError_t launch_simt_bwd(int dtype_f32, const ChunkArgs& a, cudaStream_t stream);
cudaError_t launch_tc_fwd(const ChunkArgs& a, cudaStream_t stream);
cudaError_t launch_tc_bwd(const ChunkArgs& a, float* acc_q, float* acc_k, cudaStream_t stream);
size_t tc_bwd_acc_bytes(long long T_total, int H);

namespace {

// ---- fp32 calls -------------------------------------------------------------------------------
// All arithmetic in fp32 on the CUDA cores.  One CTA per (tile of up to 4 consecutive sequences, head), 192
// threads.  Shared states: a thread owns a column and reads it once for the run of sequences that
// continue it.  Tails, 32 tokens at a time: thread (j, p) = (tid / 6, tid % 6) takes piece p of key j
// (16 values, against the same 16 of q in registers), the six partial products of a token meet in
// shared memory; thread (r, p) = (tid / 12, tid % 12) adds piece p of the values of tokens r and r + 16, loaded
// before the keys are waited for, into 16 sums of its own; the 16 threads of a piece meet once per
// sequence.  A block's scale multiplies the piece's sum (keys) or the weight (values), once for 16 codes; where
// scale, query or weight is so large that this could pass fp32's range, or that code x scale is an infinity, it
// multiplies the codes.  fp32 tails are bound by HBM, MXFP8 ones by the latency of a chunk's loads, which go out
// once the chunk before is used (issue slots 52 % busy, HBM at 35 %): 1,000 x 16 heads, 143 tokens on average, 497 us
// (fp32, 0.81 of the measured copy bandwidth) and 273 us (MXFP8).
constexpr int DEC_THREADS = DV;
constexpr int DEC_TOK = 32;
constexpr int DEC_TILE = 4;
// Scales of 2^65 and more (the code of an infinity stands under 2^120): the element is formed before it is
// multiplied with anything.
constexpr uint32_t WIDE_SCALE = 192;
constexpr float WIDE_FACTOR = 1.152921504606846976e18f;  // 2^60: neither codes x query nor weight x scale passes fp32's range below it
static_assert(DEC_TOK * 6 == DEC_THREADS && 16 * 12 == DEC_THREADS, "pieces of a chunk");

// A 16-value piece as it is stored: fp32, or codes and their block's scale byte.
template <bool MX, int D>
struct TailPiece {
  uint4 w[MX ? 1 : 4];
  uint32_t s;
  __device__ __forceinline__ void load(const void* base, const uint8_t* scales, long long token, int p, bool live) {
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + token * (MX ? D : 4 * D)) + (MX ? 1 : 4) * p;
#pragma unroll
    for (int i = 0; i < (MX ? 1 : 4); ++i) w[i] = live ? from[i] : make_uint4(0u, 0u, 0u, 0u);
    s = MX && live ? scales[token * (D / 32) + (p >> 1)] : 127u;
  }
  // f(e, value without the scale) for the 16 elements
  template <class F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int i = 0; i < (MX ? 1 : 4); ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (MX) {
          const float2 a = e4m3x2_to_f2(v[j] & 0xFFFFu), b = e4m3x2_to_f2(v[j] >> 16);
          f(4 * j, a.x);
          f(4 * j + 1, a.y);
          f(4 * j + 2, b.x);
          f(4 * j + 3, b.y);
        } else {
          f(4 * i + j, __uint_as_float(v[j]));
        }
      }
    }
  }
  __device__ __forceinline__ float scale() const { return MX ? e8m0_to_f(s) : 1.f; }
};

template <bool MX>
__global__ void __launch_bounds__(DEC_THREADS, MX ? 4 : 3)
prefix_decode_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                     const float* __restrict__ log_lambda, float scale, const float* __restrict__ pool, int pool_rows,
                     const int32_t* __restrict__ prefix_row, TailArgs t, float* __restrict__ o, int N, int H, int tile_seqs,
                     unsigned* err) {
  __shared__ __align__(16) float sq[DEC_TILE][DK];
  __shared__ float sw[DEC_TOK][6];
  __shared__ __align__(16) float sp[16][DV];
  __shared__ float s_self[DEC_TILE];
  __shared__ int s_row[DEC_TILE], s_len[DEC_TILE];
  __shared__ long long s_tok0[DEC_TILE];
  const int h = (int)(blockIdx.x % (unsigned)H), n0 = (int)(blockIdx.x / (unsigned)H) * tile_seqs;
  const int cnt = min(tile_seqs, N - n0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < cnt) {
    int row = prefix_row[n0 + tid], L;
    const long long tok0 = tail_token0(t, n0 + tid, H, h, 1, L, err);
    if (row < 0 || row >= pool_rows) {
      raise_error(err, ERR_SHAPE);
      row = -1;
    }
    if (row >= 0 && tok0 >= 0 && !(tail_in_bounds(t, H, tok0, L + 1, err) && state_in_bounds(row, pool_rows, h, H, err) &&
                                   GLA_IN_BOUNDS(n0 + tid < N, err)))
      row = -1;
    s_row[tid] = tok0 < 0 ? -1 : row;  // -1: the sequence is skipped
    s_len[tid] = L;
    s_tok0[tid] = tok0;
  }
  for (int e = tid; e < cnt * DK; e += DEC_THREADS) sq[e / DK][e % DK] = q[((long long)(n0 + e / DK) * H + h) * DK + e % DK];
  __syncthreads();
  const float ll = log_lambda[h];
  // the new tokens: q . k (warps 0 .. 3, one sequence each), and their places in the tails
  if (warp < cnt && s_row[warp] >= 0) {
    const long long nh = (long long)(n0 + warp) * H + h, at = s_tok0[warp] + s_len[warp];
    float d = 0.f;
#pragma unroll
    for (int e = lane; e < DK; e += 32) d = fmaf(sq[warp][e], k[nh * DK + e], d);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (lane == 0) s_self[warp] = d;
    float x[16] = {};
    if (lane < DK / 16) load16(k + nh * DK + 16 * lane, x);
    tail_store16<float, MX, DK>(t.k, t.ks, at, lane, x, lane < DK / 16);
    if (lane < DV / 16) load16(v + nh * DV + 16 * lane, x);
    tail_store16<float, MX, DV>(t.v, t.vs, at, lane, x, lane < DV / 16);
  }
  float acc[DEC_TILE] = {};
  for (int r0 = 0; r0 < cnt;) {
    const int row = s_row[r0];
    int r1 = r0 + 1;
    while (r1 < cnt && s_row[r1] == row) ++r1;
    if (row >= 0) {  // only this run's sequences: a state's infinities and NaN stay with its own
      const float* S = pool + ((long long)row * H + h) * (DK * DV) + tid;
#pragma unroll 8
      for (int a = 0; a < DK; ++a) {
        const float x = S[a * DV];
#pragma unroll
        for (int i = 0; i < DEC_TILE; ++i)
          if (i >= r0 && i < r1) acc[i] = fmaf(sq[i][a], x, acc[i]);
      }
    }
    r0 = r1;
  }
  const int kj = tid / 6, kp = tid % 6, vr = tid / 12, vp = tid % 12;
#pragma unroll
  for (int i = 0; i < DEC_TILE; ++i) {
    if (i >= cnt || s_row[i] < 0) continue;
    const int L = s_len[i];
    const long long tok0 = s_tok0[i];
    float qv[16], sum[16];
    load16(&sq[i][16 * kp], qv);
    bool wide_q = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) wide_q = wide_q || !(fabsf(qv[e]) < WIDE_FACTOR);
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] = 0.f;
    for (int j0 = 0; j0 < L; j0 += DEC_TOK) {
      TailPiece<MX, DV> x[2];
      TailPiece<MX, DK> y;
      y.load(t.k, t.ks, tok0 + j0 + kj, kp, j0 + kj < L);
#pragma unroll
      for (int u = 0; u < 2; ++u) x[u].load(t.v, t.vs, tok0 + j0 + vr + 16 * u, vp, j0 + vr + 16 * u < L);
      float d = 0.f;
      if (MX && (wide_q || y.s >= WIDE_SCALE)) {
        y.each([&](int e, float c) { d = fmaf(c * y.scale(), qv[e], d); });
      } else {
        y.each([&](int e, float c) { d = fmaf(c, qv[e], d); });
        d *= y.scale();
      }
      __syncthreads();  // the weights of the chunk before have been used
      sw[kj][kp] = d;
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int jj = vr + 16 * u, j = j0 + jj;
        if (j < L) {
          float w = (((sw[jj][0] + sw[jj][1]) + (sw[jj][2] + sw[jj][3])) + (sw[jj][4] + sw[jj][5])) * decay_pow(ll, L - j);
          if (MX && (x[u].s >= WIDE_SCALE || !(fabsf(w) < WIDE_FACTOR))) {
            x[u].each([&](int e, float c) { sum[e] = fmaf(w, c * x[u].scale(), sum[e]); });
          } else {
            w *= x[u].scale();
            x[u].each([&](int e, float c) { sum[e] = fmaf(w, c, sum[e]); });
          }
        }
      }
    }
    store16(&sp[vr][16 * vp], sum);
    __syncthreads();
    float tail_sum = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) tail_sum += sp[r][tid];
    const long long at = ((long long)(n0 + i) * H + h) * DV + tid;
    o[at] = scale * fmaf(s_self[i], v[at], fmaf(decay_pow(ll, L + 1), acc[i], tail_sum));
    __syncthreads();  // the sums are free again
  }
}

// ---- bf16 calls: tiles of sequences, tensor cores ----------------------------------------------
// One CTA per (tile of up to 16 consecutive sequences, head).
//   Shared states: for every run of equal prefix rows in the tile, [16 x 96] q times [96 x 192] S with
//     mma.m16n8k16 (bf16, fp32 sums), S split into hi + lo bf16 as it is read (16 significant bits; a
//     single bf16 would put 2^-8 into every term).  A warp owns 48 columns; the S fragments go from
//     global memory (L2 for all but one tile) to registers, nothing is staged.
//   Tails: chunks of 16 or 32 tokens, in order, of all the tile's sequences form one list that is cut evenly
//     over the warps, so one long tail among short ones, or a tile of one sequence, still feeds
//     all of them.  A warp streams its chunks through a stage of its own in shared memory (bulk
//     copies: the tokens of a (row, head) are contiguous) and multiplies on the tensor cores:
//       weights   K [16 tokens x 96] times q (one column of N = 8 used): exact products.  E4M3 codes
//                 widen exactly to f16; q is brought to f16 by a power of two (its 8 bits fit down to
//                 2^-27 of the largest).  Block scales enter in fp32, per 32 columns.
//       output    V^T [16 columns x 16 tokens] times w [16 tokens x 8].  bf16 tails: w's even columns
//                 hold the high bf16 of the weight, the odd ones the low one (their sums meet in one
//                 thread).  MXFP8: column b holds w_j 2^(e_jb), the weight times the scale of column
//                 block b, so that the codes enter unscaled (exact in f16); its high and low f16 go
//                 in turn.  Each column is kept in f16's range by a power of two of its own, raised
//                 (and the sums rescaled) when a weight outgrows it.  A pair has 16 bits of a weight
//                 down to 2^-19 of that power.
//       A chunk with weights below that (the block's largest element may be zero in a column whose sum is made
//       of the others), with a scale of 2^65 or more (an infinity is code 448 under 2^120) or with weights that could
//       leave fp32's range under their scales, and a sequence whose q does not fit, go through the CUDA cores
//       instead: elements code x scale in fp32, products and sums in fp32 (far_sums).  That takes four times as
//       long (1,280 x 16 with such a scale in every chunk: 740 us), but of normally distributed keys and values
//       about one chunk in ten thousand calls for it.
//     The warp that has a sequence's first chunk adds to the tile's sums directly; the others that share it
//     keep their parts, which meet in warp order.
// mma.sync rather than tcgen05: a sequence brings one query row, so a 128-row tile would stand empty, and
// the codes are widened in registers either way.  Bound by latency: 16 warps per SM (accumulators and stages
// leave no room for more) hide that of about 870 warp instructions per 32 MXFP8 tokens only in part, with the
// issue slots half busy and HBM at 56 %: 1,280 x 16 heads, 143 tokens on average, MXFP8, 195 us (0.70 of the
// measured copy bandwidth on its 921 MB; rows in no order, so that a tile reads a state for every sequence:
// 355 us); 333 x 7, 146 tokens, bf16, 49 us (0.62).
constexpr int TILE_MAX = 16;
constexpr int PD_WARPS = 4, PD_THREADS = 32 * PD_WARPS;

// A warp's stage: one chunk, 32 tokens of MXFP8 or 16 of bf16 (9.5 and 9.2 KB: four CTAs per SM).  Keys
// and values have a barrier each, so that the next chunk's keys land while this one's values are used.
template <bool MX>
struct PdStage {
  static constexpr int TOK = MX ? 32 : 16, SUB = TOK / 16;  // tokens; 16-token steps of the MMAs
  static constexpr uint32_t K_ROW = MX ? DK : 2 * DK, V_ROW = MX ? DV : 2 * DV;  // bytes of a token
  static constexpr uint32_t K = 0, V = K + TOK * K_ROW, KS = V + TOK * V_ROW, VS = KS + (MX ? TOK * 3 : 0);
  static constexpr uint32_t BYTES = VS + (MX ? TOK * 6 : 0);
};
template <bool MX>
struct PdSmem {
  static constexpr uint32_t O = PD_WARPS * PdStage<MX>::BYTES;  // [16][192] sums
  static constexpr uint32_t PART = O + TILE_MAX * DV * 4;                        // [warps][192], a warp's part of a sequence that another begins
  static constexpr uint32_t Q = PART + PD_WARPS * DV * 4;                        // [16][96] bf16
  static constexpr uint32_t BAR = Q + TILE_MAX * DK * 2;
  static constexpr uint32_t BYTES = BAR + PD_WARPS * 2 * 8;
};

template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, float c0, float c1, float c2, float c3) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
template <bool F16>
__device__ __forceinline__ void mma16_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  mma16<F16>(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_h(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// (x, y) as hi + lo bf16 pairs.
__device__ __forceinline__ void split_bf(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf(x, y);
  lo = pack_bf(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
}
__device__ __forceinline__ void split_h(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_h(x - f.x, y - f.y);
}
// Two E4M3 codes to an f16 pair (exact; a NaN code stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
// Two E8M0 scale bytes to a bf16 pair, 2^(b - 127) (exact; 255: NaN).
__device__ __forceinline__ uint32_t e8m0x2_to_bf2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
constexpr int WIDE_SUM = 100;  // the MMAs take weights under their scales of up to 2^100, and 2^100 times a run's first
__device__ __forceinline__ int exponent_of(float x) { return (int)((__float_as_uint(x) >> 23) & 0xFFu) - 127; }
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }
// Weights whose bits - 1 are below this are less than 2^-19 of the power of two e (but not zero).
__device__ __forceinline__ uint32_t weak_below(int e) { return __float_as_uint(pow2i(e - 19)) - 1u; }
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// The first n bytes of a word (n <= 0: none).
__device__ __forceinline__ uint32_t cut_bytes(uint32_t x, int n) { return n >= 4 ? x : n <= 0 ? 0u : x & ((1u << (8 * n)) - 1u); }

struct Sums8 {
  float v[8];
};
// An MXFP8 chunk's share of the output in fp32 (whole warp): tokens tok .. tok + m - 1, of ages `age` and less, keys
// from where they stand (the stage may hold the next chunk's), values from the stage.  Lane (g, tq < 3) has
// columns 64 tq + 8 g .. + 7.  Kept out of the kernel's loop, whose registers it would take.
__device__ __noinline__ Sums8 far_sums(const TailArgs& t, long long tok, int m, float ll, int age, const __nv_bfloat16* q,
                                          const uint8_t* v, const uint8_t* vs) {
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  float w = 0.f;  // lane j: token j's weight
  if (lane < m) {
    const uint8_t* k = static_cast<const uint8_t*>(t.k) + (tok + lane) * DK;
    const uint8_t* ks = t.ks + (tok + lane) * (DK / 32);
#pragma unroll 1
    for (int e = 0; e < DK; e += 4) {
      const float s = e8m0_to_f(ks[e >> 5]);
      const uint32_t x = *reinterpret_cast<const uint32_t*>(k + e);
      const uint2 y = *reinterpret_cast<const uint2*>(q + e);
      const float2 c0 = e4m3x2_to_f2(x & 0xFFFFu), c1 = e4m3x2_to_f2(x >> 16);
      w = fmaf(c0.x * s, __uint_as_float(y.x << 16), w);
      w = fmaf(c0.y * s, __uint_as_float(y.x & 0xFFFF0000u), w);
      w = fmaf(c1.x * s, __uint_as_float(y.y << 16), w);
      w = fmaf(c1.y * s, __uint_as_float(y.y & 0xFFFF0000u), w);
    }
    w *= decay_pow(ll, age - lane);
  }
  Sums8 r = {};
#pragma unroll 1
  for (int j = 0; j < m; ++j) {
    const float wj = __shfl_sync(0xffffffffu, w, j);
    if (tq < 3) {
      const float s = e8m0_to_f(vs[6 * j + 2 * tq + (g >> 2)]);
      const uint2 x = *reinterpret_cast<const uint2*>(v + j * DV + 64 * tq + 8 * g);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 c = e4m3x2_to_f2((e < 2 ? x.x : x.y) >> (16 * (e & 1)) & 0xFFFFu);
        r.v[2 * e] = fmaf(wj, c.x * s, r.v[2 * e]);
        r.v[2 * e + 1] = fmaf(wj, c.y * s, r.v[2 * e + 1]);
      }
    }
  }
  return r;
}

template <bool MX>
__global__ void __launch_bounds__(PD_THREADS, 4)
prefix_decode_tile_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
                          const __nv_bfloat16* __restrict__ v, const float* __restrict__ log_lambda, float scale,
                          const float* __restrict__ pool, int pool_rows, const int32_t* __restrict__ prefix_row, TailArgs t,
                          __nv_bfloat16* __restrict__ o, int N, int H, int tile_seqs, unsigned* err,
                          unsigned long long wait_ns) {
  using ST = PdStage<MX>;
  using SM = PdSmem<MX>;
  using BF = __nv_bfloat16;
  extern __shared__ __align__(128) uint8_t pd_smem[];
  __shared__ int s_row[TILE_MAX], s_len[TILE_MAX], s_cu[TILE_MAX + 1], s_part[PD_WARPS];  // s_part: sequences of the warps' parts, -1: none
  __shared__ long long s_tok0[TILE_MAX];
  __shared__ float s_self[TILE_MAX];
  __shared__ int s_abort;
  float* sO = reinterpret_cast<float*>(pd_smem + SM::O);
  float* sPart = reinterpret_cast<float*>(pd_smem + SM::PART);
  BF* sQ = reinterpret_cast<BF*>(pd_smem + SM::Q);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(pd_smem + SM::BAR) + warp * 2;  // keys, values
  const int h = (int)(blockIdx.x % (unsigned)H), n0 = (int)(blockIdx.x / (unsigned)H) * tile_seqs;
  const int cnt = min(tile_seqs, N - n0);
  // Loads that need no index go out before anything is waited for: q, and the new tokens (eight lanes a
  // sequence for its key, sixteen for its value).
  const int ik = warp + PD_WARPS * (lane >> 3), pk = lane & 7, pv = lane & 15;
  auto iv = [&](int u) { return warp + PD_WARPS * (2 * u + (lane >> 4)); };
  uint4 rq[2], nk[2], nv[2][2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = tid + u * PD_THREADS;
    if (e < cnt * (DK / 8))
      rq[u] = *reinterpret_cast<const uint4*>(q + ((long long)(n0 + e / (DK / 8)) * H + h) * DK + 8 * (e % (DK / 8)));
    nk[u] = nv[u][0] = nv[u][1] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (ik < cnt && pk < DK / 16) {
    const uint4* from = reinterpret_cast<const uint4*>(k + ((long long)(n0 + ik) * H + h) * DK + 16 * pk);
    nk[0] = from[0];
    nk[1] = from[1];
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (iv(u) < cnt && pv < DV / 16) {
      const uint4* from = reinterpret_cast<const uint4*>(v + ((long long)(n0 + iv(u)) * H + h) * DV + 16 * pv);
      nv[u][0] = from[0];
      nv[u][1] = from[1];
    }
  const float ll = log_lambda[h];
  if (warp == 0) {
    int row = -1, L = -1;
    long long tok0 = -1;
    if (lane < cnt) {
      row = prefix_row[n0 + lane];
      tok0 = tail_token0(t, n0 + lane, H, h, 1, L, err);
      if (row < 0 || row >= pool_rows) {
        raise_error(err, ERR_SHAPE);
        row = -1;
      }
      if (tok0 < 0) row = -1;  // row -1: the sequence is skipped
      if (row >= 0 && !(tail_in_bounds(t, H, tok0, L + 1, err) && state_in_bounds(row, pool_rows, h, H, err) &&
                        GLA_IN_BOUNDS(n0 + lane < N, err)))
        row = -1;
    }
    int chunks = row >= 0 ? (L + ST::TOK - 1) / ST::TOK : 0;
    if (lane < TILE_MAX) {
      s_row[lane] = row;
      s_len[lane] = L;
      s_tok0[lane] = tok0;
    }
#pragma unroll
    for (int d = 1; d < TILE_MAX; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, chunks, d);
      if (lane >= d) chunks += up;
    }
    if (lane < TILE_MAX) s_cu[lane + 1] = chunks;
    if (lane == 0) {
      s_cu[0] = 0;
      s_abort = 0;
    }
  }
  if (lane == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    s_part[warp] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (tid + u * PD_THREADS < cnt * (DK / 8)) reinterpret_cast<uint4*>(sQ)[tid + u * PD_THREADS] = rq[u];
  for (int e = tid; e < cnt * (DV / 4); e += PD_THREADS) reinterpret_cast<float4*>(sO)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int e = tid; e < PD_WARPS * (DV / 4); e += PD_THREADS) reinterpret_cast<float4*>(sPart)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();

  // ---- this warp's chunks [c0, c1) of the tile's list; its first loads
  const long long total = s_cu[TILE_MAX];
  const int c0 = (int)(total * warp / PD_WARPS), c1 = (int)(total * (warp + 1) / PD_WARPS);
  uint8_t* const st = pd_smem + (size_t)warp * ST::BYTES;
  const uint32_t st32 = smem_u32(st);
  // The next chunk to load (whole warp; lane 0 issues the copies).
  int next = c0, next_seq = 0, next_m = 0, loads_k = 0, loads_v = 0;
  long long next_tok = 0;
  auto load_keys = [&]() {
    while (next >= s_cu[next_seq + 1]) ++next_seq;
    const int j0 = (next - s_cu[next_seq]) * ST::TOK;
    next_m = min(ST::TOK, s_len[next_seq] - j0);
    next_tok = s_tok0[next_seq] + j0;
    ++next;
    ++loads_k;
    // (what the scales' last 16 bytes hold besides lies in the same row: cap is a multiple of 16)
    const bool in = tail_in_bounds(t, H, next_tok, next_m, err) && GLA_IN_BOUNDS(next_m > 0, err);
    if (!in) next_m = 0;
    const uint32_t bytes = (uint32_t)next_m * ST::K_ROW, ks = MX ? (uint32_t)(3 * next_m + 15) / 16 * 16 : 0;
    if (lane == 0) {
      mbar_expect_tx(&full[0], bytes + ks);
      if (in) bulk_copy(st32 + ST::K, static_cast<const uint8_t*>(t.k) + next_tok * ST::K_ROW, bytes, &full[0]);
      if (MX && in) bulk_copy(st32 + ST::KS, t.ks + next_tok * (DK / 32), ks, &full[0]);
    }
  };
  auto load_values = [&]() {  // of the chunk whose keys were loaded last
    ++loads_v;
    const uint32_t bytes = (uint32_t)next_m * ST::V_ROW, vs = MX ? (uint32_t)(6 * next_m + 15) / 16 * 16 : 0;
    if (lane == 0) {
      mbar_expect_tx(&full[1], bytes + vs);
      const bool in = GLA_IN_BOUNDS(next_m > 0, err);
      if (in) bulk_copy(st32 + ST::V, static_cast<const uint8_t*>(t.v) + next_tok * ST::V_ROW, bytes, &full[1]);
      if (MX && in) bulk_copy(st32 + ST::VS, t.vs + next_tok * (DV / 32), vs, &full[1]);
    }
  };
  auto release = [&](int m) {  // a chunk's values are read (the zeros behind its m tokens were written through the generic proxy)
    if (m < ST::TOK) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (loads_v < loads_k) load_values();
  };
  if (c0 < c1) {
    load_keys();
    load_values();
  }

  // The shared states' lines into L2 (a tile that meets a state first would wait for DRAM row by row).
  for (int r0 = 0; r0 < cnt; ++r0) {
    const int row = s_row[r0];
    if (row < 0 || (r0 > 0 && s_row[r0 - 1] == row)) continue;
    const char* S = reinterpret_cast<const char*>(pool + ((long long)row * H + h) * (DK * DV));
    for (int e = tid; e < DK * DV * 4 / 128; e += PD_THREADS) asm volatile("prefetch.global.L2 [%0];" ::"l"(S + 128 * e));
  }

  // ---- the new tokens: q . k, and their places in the tails
  {
    float x[16], d = 0.f;
    const bool live = ik < cnt && s_row[ik] >= 0 && pk < DK / 16;
    load16(reinterpret_cast<const BF*>(nk), x);
    if (live) {
      float z[16];
      load16(sQ + ik * DK + 16 * pk, z);
#pragma unroll
      for (int e = 0; e < 16; ++e) d = fmaf(x[e], z[e], d);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (live && pk == 0) s_self[ik] = d;
    tail_store16<BF, MX, DK>(t.k, t.ks, live ? s_tok0[ik] + s_len[ik] : 0, pk, x, live);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = iv(u);
      const bool lv = i < cnt && s_row[i] >= 0 && pv < DV / 16;
      load16(reinterpret_cast<const BF*>(nv[u]), x);
      tail_store16<BF, MX, DV>(t.v, t.vs, lv ? s_tok0[i] + s_len[i] : 0, pv, x, lv);
    }
  }

  // The shared states' part first in one half of the CTAs and last in the other: its latencies then fall
  // into the others' streams.
  // (the hash mixes both halves on every SM: CTAs i, i + 152, ... tend to share one)
  const int late = (int)((blockIdx.x ^ (blockIdx.x >> 3)) & 1u);
  bool ok = true;
  for (int step = 0; step < 2; ++step) {
   if (step == late) {
    // ---- the shared states
    // q fragments; K step s of thread tq: columns 16 s + 4 tq .. + 3 (the same order as S's rows)
    uint2 qa[6], qb[6];
    const BF* q0 = sQ + g * DK + 4 * tq;
    const BF* q1 = q0 + 8 * DK;
#pragma unroll
    for (int s = 0; s < 6; ++s) {
      qa[s] = g < cnt ? *reinterpret_cast<const uint2*>(q0 + 16 * s) : make_uint2(0u, 0u);
      qb[s] = g + 8 < cnt ? *reinterpret_cast<const uint2*>(q1 + 16 * s) : make_uint2(0u, 0u);
    }
    const float f0 = g < cnt && s_row[g] >= 0 ? decay_pow(ll, s_len[g] + 1) : 0.f;
    const float f1 = g + 8 < cnt && s_row[g + 8] >= 0 ? decay_pow(ll, s_len[g + 8] + 1) : 0.f;
    for (int r0 = 0; r0 < cnt;) {
      const int row = s_row[r0];
      int r1 = r0 + 1;
      while (r1 < cnt && s_row[r1] == row) ++r1;
      if (row >= 0) {
        float d[6][4] = {};
        const float* S = pool + ((long long)row * H + h) * (DK * DV) + 48 * warp;
#pragma unroll
        for (int s = 0; s < 6; ++s) {
          float4 x[4];
          float2 y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* p = S + (16 * s + 4 * tq + e) * DV;
            x[e] = *reinterpret_cast<const float4*>(p + 4 * g);
            y[e] = *reinterpret_cast<const float2*>(p + 32 + 2 * g);
          }
          auto col = [&](float (&dd)[4], float v0, float v1, float v2, float v3) {
            uint32_t h0, l0, h1, l1;
            split_bf(v0, v1, h0, l0);
            split_bf(v2, v3, h1, l1);
            mma16_add<false>(dd, qa[s].x, qb[s].x, qa[s].y, qb[s].y, h0, h1);
            mma16_add<false>(dd, qa[s].x, qb[s].x, qa[s].y, qb[s].y, l0, l1);
          };
          col(d[0], x[0].x, x[1].x, x[2].x, x[3].x);
          col(d[1], x[0].y, x[1].y, x[2].y, x[3].y);
          col(d[2], x[0].z, x[1].z, x[2].z, x[3].z);
          col(d[3], x[0].w, x[1].w, x[2].w, x[3].w);
          col(d[4], y[0].x, y[1].x, y[2].x, y[3].x);
          col(d[5], y[0].y, y[1].y, y[2].y, y[3].y);
        }
        // only this run's rows: a state's infinities and NaN stay with its own sequences
#pragma unroll
        for (int j = 0; j < 6; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = g + 8 * (e >> 1), nn = 2 * tq + (e & 1);
            const int c = 48 * warp + (j < 4 ? 4 * nn + j : 32 + 2 * nn + (j - 4));
            if (r >= r0 && r < r1) sO[r * DV + c] += d[j][e] * (e >> 1 ? f1 : f0);
          }
      }
      r0 = r1;
    }
   } else {
  // ---- the tails
  int seq = 0;
  for (int c = c0; c < c1 && ok;) {
    while (c >= s_cu[seq + 1]) ++seq;
    const int first = s_cu[seq], last = min(s_cu[seq + 1], c1), L = s_len[seq];
    float* const dst = first >= c0 ? sO + seq * DV : sPart + warp * DV;
    if (first < c0 && lane == 0) s_part[warp] = seq;
    bool wide_q = false;  // q's magnitude calls for weights in fp32 throughout
    // q as the B operand: one column (n = 0, the lanes with g = 0); block b, K step u of thread tq:
    // columns 32 b + 8 tq + 4 u .. + 3
    uint32_t qf[3][4];
    float qn = 1.f;  // what the weights are to be multiplied with
    {
      const BF* qr = sQ + seq * DK + 8 * tq;
#pragma unroll
      for (int b = 0; b < 3; ++b) {
        const uint4 u = *reinterpret_cast<const uint4*>(qr + 32 * b);
        qf[b][0] = u.x;
        qf[b][1] = u.y;
        qf[b][2] = u.z;
        qf[b][3] = u.w;
      }
      if (MX) {
        float m = 0.f;
        uint32_t low = ~0u;  // the smallest but zero (bits - 1)
#pragma unroll
        for (int b = 0; b < 3; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = qf[b][e] << 16 & 0x7FFFFFFFu, y = qf[b][e] & 0x7FFF0000u;
            m = fmaxf(m, fmaxf(__uint_as_float(x), __uint_as_float(y)));
            low = min(low, min(x - 1u, y - 1u));
          }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e2 = max(exponent_of(m), -100) - 10;  // the largest comes to [2^10, 2^11)
        wide_q = (m > 0.f && (e2 > 50 || e2 < -50)) || __any_sync(0xffffffffu, low < __float_as_uint(pow2i(e2 - 17)) - 1u);
        const float inv = pow2i(-e2);
        qn = pow2i(e2);
#pragma unroll
        for (int b = 0; b < 3; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            qf[b][e] = pack_h(__uint_as_float(qf[b][e] << 16) * inv, __uint_as_float(qf[b][e] & 0xFFFF0000u) * inv);
      }
#pragma unroll
      for (int b = 0; b < 3; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[b][e] = g == 0 ? qf[b][e] : 0u;
    }
    while (c < last && ok) {  // runs of chunks that the MMAs take, each ended by a far chunk or the last
    bool far_chunk = false;
    float acc[12][4];  // 16 columns each: see the flush below
#pragma unroll
    for (int i = 0; i < 12; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
    int E = -1000;  // (MXFP8) exponent of the power of two of column g of w
    for (; c < last; ++c) {
      const uint32_t phase = (uint32_t)(c - c0) & 1u;
      const int j0 = (c - first) * ST::TOK, m = min(ST::TOK, L - j0);
      ok = __all_sync(0xffffffffu, mbar_wait_at(&full[0], phase, wait_ns, &s_abort, 0, warp == 1 ? c - c0 : -1));
      if (!ok) break;
      // weights: token 16 u + g in lanes tq = 0, sc[u][0]; token 16 u + g + 8, sc[u][1]
      float sc[ST::SUB][2];
#pragma unroll
      for (int u = 0; u < ST::SUB; ++u) {
        const uint8_t* kr = st + ST::K + (uint32_t)(16 * u + g) * ST::K_ROW + (MX ? 8 : 16) * tq;
        float d[3][4];
#pragma unroll
        for (int b = 0; b < 3; ++b) {
          if constexpr (MX) {
            const uint2 x = *reinterpret_cast<const uint2*>(kr + 32 * b), y = *reinterpret_cast<const uint2*>(kr + 8 * DK + 32 * b);
            mma16<true>(d[b], e4m3x2_to_h2(x.x & 0xFFFFu), e4m3x2_to_h2(y.x & 0xFFFFu), e4m3x2_to_h2(x.x >> 16),
                        e4m3x2_to_h2(y.x >> 16), qf[b][0], qf[b][1], 0.f, 0.f, 0.f, 0.f);
            mma16_add<true>(d[b], e4m3x2_to_h2(x.y & 0xFFFFu), e4m3x2_to_h2(y.y & 0xFFFFu), e4m3x2_to_h2(x.y >> 16),
                            e4m3x2_to_h2(y.y >> 16), qf[b][2], qf[b][3]);
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(kr + 64 * b), y = *reinterpret_cast<const uint4*>(kr + 8 * ST::K_ROW + 64 * b);
            mma16<false>(d[b], x.x, y.x, x.y, y.y, qf[b][0], qf[b][1], 0.f, 0.f, 0.f, 0.f);
            mma16_add<false>(d[b], x.z, y.z, x.w, y.w, qf[b][2], qf[b][3]);
          }
        }
        if constexpr (MX) {  // the block scales of the two tokens' keys
          const uint8_t* kp = st + ST::KS + 3 * (16 * u + g);
          const uint32_t u0 = e8m0x2_to_bf2(kp[0] | (uint32_t)kp[1] << 8), u1 = e8m0x2_to_bf2(kp[24] | (uint32_t)kp[25] << 8),
                         u2 = e8m0x2_to_bf2(kp[2] | (uint32_t)kp[26] << 8);
          sc[u][0] = fmaf(d[2][0], __uint_as_float(u2 << 16),
                          fmaf(d[1][0], __uint_as_float(u0 & 0xFFFF0000u), d[0][0] * __uint_as_float(u0 << 16)));
          sc[u][1] = fmaf(d[2][2], __uint_as_float(u2 & 0xFFFF0000u),
                          fmaf(d[1][2], __uint_as_float(u1 & 0xFFFF0000u), d[0][2] * __uint_as_float(u1 << 16)));
        } else {
          sc[u][0] = d[0][0] + d[1][0] + d[2][0];
          sc[u][1] = d[0][2] + d[1][2] + d[2][2];
        }
      }
      uint32_t far = wide_q;  // (MXFP8) not zero in some lane: the chunk goes through the CUDA cores
      if constexpr (MX) {     // the scales' bytes, four a lane: 2^65 and more have their two top bits set
        uint32_t x = lane < DK / 32 * ST::TOK / 4 ? reinterpret_cast<const uint32_t*>(st + ST::KS)[lane] : 0u;
        if (m < ST::TOK) x = cut_bytes(x, 3 * m - 4 * lane);
        far |= x & (x << 1) & 0x80808080u;
      }
      __syncwarp();
      if (next < c1) load_keys();  // the keys are read
      // lane j takes token j's weight (bf16: lanes 16 .. 31 repeat)
      float w = 0.f;
#pragma unroll
      for (int u = 0; u < ST::SUB; ++u) {
        const float lo = __shfl_sync(0xffffffffu, sc[u][0], (lane & 7) * 4), hi = __shfl_sync(0xffffffffu, sc[u][1], (lane & 7) * 4);
        if (ST::SUB == 1 || (lane >> 4) == u) w = lane & 8 ? hi : lo;
      }
      const int jl = lane & (ST::TOK - 1);
      w = jl < m ? w * qn * decay_pow(ll, L - j0 - jl) : 0.f;
      float wt[ST::SUB][4];  // tokens 16 u + tq + 4 i
#pragma unroll
      for (int u = 0; u < ST::SUB; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) wt[u][i] = __shfl_sync(0xffffffffu, w, 16 * u + tq + 4 * i);

      ok = __all_sync(0xffffffffu, mbar_wait_at(&full[1], phase, wait_ns, &s_abort, 1, warp == 1 ? c - c0 : -1));
      if (!ok) break;
      if (m < ST::TOK) {
        // rows past the tail's end hold another chunk's values or nothing: zero, so that their
        // zero weights give zero
        for (uint32_t e = lane; e < (uint32_t)(ST::TOK - m) * ST::V_ROW / 16; e += 32)
          *reinterpret_cast<uint4*>(st + ST::V + (uint32_t)m * ST::V_ROW + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      if constexpr (MX) {
        float mx = 0.f;
        uint32_t low = ~0u;  // the smallest but zero (bits - 1)
#pragma unroll
        for (int u = 0; u < ST::SUB; ++u) {
          const uint8_t* vp = st + ST::VS + 6 * (16 * u + tq) + min(g, DV / 32 - 1);
          const uint32_t u0 = e8m0x2_to_bf2(vp[0] | (uint32_t)vp[24] << 8), u1 = e8m0x2_to_bf2(vp[48] | (uint32_t)vp[72] << 8);
          const float vs[4] = {__uint_as_float(u0 << 16), __uint_as_float(u0 & 0xFFFF0000u), __uint_as_float(u1 << 16),
                               __uint_as_float(u1 & 0xFFFF0000u)};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            wt[u][i] = g < DV / 32 && 16 * u + tq + 4 * i < m ? wt[u][i] * vs[i] : 0.f;  // (past the end: maybe NaN)
            mx = fmaxf(mx, fabsf(wt[u][i]));
            low = min(low, (__float_as_uint(wt[u][i]) & 0x7FFFFFFFu) - 1u);
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int need = mx > 0.f ? max(exponent_of(mx), -115) : -1000;
        uint2 x = lane < DV / 32 * ST::TOK / 8 ? reinterpret_cast<const uint2*>(st + ST::VS)[lane] : make_uint2(0u, 0u);
        if (m < ST::TOK) x = make_uint2(cut_bytes(x.x, 6 * m - 8 * lane), cut_bytes(x.y, 6 * m - 8 * lane - 4));
        far |= ((x.x & (x.x << 1)) | (x.y & (x.y << 1))) & 0x80808080u;
        const bool grow = need > E + 4;
        if (__any_sync(0xffffffffu, far != 0u || grow || low < weak_below(E))) {
          far_chunk = __any_sync(0xffffffffu, far != 0u || need > min(E == -1000 ? 0 : E, 0) + WIDE_SUM ||
                                                  low < weak_below(grow ? need : E));
          if (far_chunk) break;
          const float f = !grow ? 1.f : (E < -126 ? 0.f : pow2i(E - need));
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * tq), f1 = __shfl_sync(0xffffffffu, f, 8 * tq + 4);
#pragma unroll
          for (int i = 0; i < 12; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] *= (e & 1) ? f1 : f0;
          if (grow) E = need;
        }
      }
      const float up = MX ? pow2i(10 - E) : 1.f;
#pragma unroll
      for (int u = 0; u < ST::SUB; ++u) {
        uint32_t h0, h1, l0, l1;
        const uint8_t* vr = st + ST::V + (uint32_t)(16 * u + tq) * ST::V_ROW + (MX ? 8 : 16) * g;
        if constexpr (MX) {
          split_h(wt[u][0] * up, wt[u][1] * up, h0, l0);
          split_h(wt[u][2] * up, wt[u][3] * up, h1, l1);
#pragma unroll
          for (int B = 0; B < 3; ++B) {
            uint2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint2*>(vr + 4 * i * DV + 64 * B);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {  // columns 64 B + 8 g + 2 jj (row g) and the next (row g + 8)
              const uint32_t sel = jj & 1 ? 0x7362 : 0x5140;
              const uint32_t p = __byte_perm(jj & 2 ? x[0].y : x[0].x, jj & 2 ? x[1].y : x[1].x, sel);
              const uint32_t r = __byte_perm(jj & 2 ? x[2].y : x[2].x, jj & 2 ? x[3].y : x[3].x, sel);
              const uint32_t a0 = e4m3x2_to_h2(p & 0xFFFFu), a1 = e4m3x2_to_h2(p >> 16), a2 = e4m3x2_to_h2(r & 0xFFFFu),
                             a3 = e4m3x2_to_h2(r >> 16);
              mma16_add<true>(acc[4 * B + jj], a0, a1, a2, a3, h0, h1);
              mma16_add<true>(acc[4 * B + jj], a0, a1, a2, a3, l0, l1);
            }
          }
        } else {
          split_bf(wt[u][0], wt[u][1], h0, l0);
          split_bf(wt[u][2], wt[u][3], h1, l1);
          const uint32_t b0 = g & 1 ? l0 : h0, b1 = g & 1 ? l1 : h1;
#pragma unroll
          for (int B = 0; B < 3; ++B) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(vr + 4 * i * ST::V_ROW + 128 * B);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const uint32_t x0 = jj == 0 ? x[0].x : jj == 1 ? x[0].y : jj == 2 ? x[0].z : x[0].w;
              const uint32_t x1 = jj == 0 ? x[1].x : jj == 1 ? x[1].y : jj == 2 ? x[1].z : x[1].w;
              const uint32_t x2 = jj == 0 ? x[2].x : jj == 1 ? x[2].y : jj == 2 ? x[2].z : x[2].w;
              const uint32_t x3 = jj == 0 ? x[3].x : jj == 1 ? x[3].y : jj == 2 ? x[3].z : x[3].w;
              mma16_add<false>(acc[4 * B + jj], __byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x7632),
                               __byte_perm(x2, x3, 0x5410), __byte_perm(x2, x3, 0x7632), b0, b1);
            }
          }
        }
      }
      release(m);
    }
    if (!ok) break;
    // the run's sums: thread (g, tq < 3) holds columns 64 tq + 8 g .. + 7
    const float back = MX ? pow2i(__shfl_sync(0xffffffffu, E, 4 * ((2 * tq + (g >> 2)) & 7)) - 10) : 1.f;
    float y[8];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x = 0.f;
#pragma unroll
        for (int B = 0; B < 3; ++B) {
          const float(&a)[4] = acc[4 * B + jj];
          // MXFP8: the column's block is 2 B + (g >> 2), column tq = B of the product, its first or
          // second element; bf16: the high and the low part
          const float z = MX ? (g >> 2 ? a[2 * u + 1] : a[2 * u]) * back : a[2 * u] + a[2 * u + 1];
          x = tq == B ? z : x;
        }
        y[2 * jj + u] = x;
      }
    if (tq < 3) {
      float4* p = reinterpret_cast<float4*>(dst + 64 * tq + 8 * g);
      const float4 a = p[0], b = p[1];
      p[0] = make_float4(y[0] + a.x, y[1] + a.y, y[2] + a.z, y[3] + a.w);
      p[1] = make_float4(y[4] + b.x, y[5] + b.y, y[6] + b.z, y[7] + b.w);
    }
    if constexpr (MX) {
      if (far_chunk) {
        const int j0 = (c - first) * ST::TOK, m = min(ST::TOK, L - j0);
        const Sums8 z = far_sums(t, s_tok0[seq] + j0, m, ll, L - j0, sQ + seq * DK, st + ST::V, st + ST::VS);
        if (tq < 3) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[64 * tq + 8 * g + e] += z.v[e];
        }
        release(m);
        ++c;
      }
    }
    }
  }
   }
   __syncthreads();
  }
  if (!ok) {
    // a wait gave up: no copy into this CTA's shared memory may be in flight when it exits
    if (lane == 0) {
      if (loads_k) mbar_wait_drain(&full[0], (uint32_t)(loads_k - 1) & 1u, 1000000000ull, err);
      if (loads_v) mbar_wait_drain(&full[1], (uint32_t)(loads_v - 1) & 1u, 1000000000ull, err);
      raise_error(err, ERR_TIMEOUT);
    }
  }
  __syncthreads();
  if (s_abort) return;
  // ---- shared parts in warp order, the new tokens (their values on the way meanwhile), and out
  uint4 ov[3];
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    const int e = tid + u * PD_THREADS;
    if (e < cnt * (DV / 8))
      ov[u] = *reinterpret_cast<const uint4*>(v + ((long long)(n0 + e / (DV / 8)) * H + h) * DV + 8 * (e % (DV / 8)));
  }
  for (int col = tid; col < DV; col += PD_THREADS)
#pragma unroll
    for (int p = 0; p < PD_WARPS; ++p)
      if (s_part[p] >= 0) sO[s_part[p] * DV + col] += sPart[p * DV + col];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    const int e = tid + u * PD_THREADS, i = e / (DV / 8), c = 8 * (e % (DV / 8));
    if (e >= cnt * (DV / 8) || s_row[i] < 0 || !GLA_IN_BOUNDS(n0 + i < N && h < H, err)) continue;
    const float g8 = s_self[i];
    const float4 x = *reinterpret_cast<const float4*>(sO + i * DV + c), y = *reinterpret_cast<const float4*>(sO + i * DV + c + 4);
    const uint32_t w[4] = {ov[u].x, ov[u].y, ov[u].z, ov[u].w};
    const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t r[4];
#pragma unroll
    for (int k2 = 0; k2 < 4; ++k2)
      r[k2] = pack_bf(scale * fmaf(g8, __uint_as_float(w[k2] << 16), z[2 * k2]),
                      scale * fmaf(g8, __uint_as_float(w[k2] & 0xFFFF0000u), z[2 * k2 + 1]));
    *reinterpret_cast<uint4*>(o + ((long long)(n0 + i) * H + h) * DV + c) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// Sequences of a tile.  A tile costs its sequences and about four more (its indexes, its pass over the
// states, its output), four CTAs run on an SM, and the last round of CTAs takes as long as any: the
// size with the least rounds x (sequences + 4).  Measured over sizes 2 .. 16, this picks the best or
// comes within 4 %:  1,280 x 16 heads MXFP8: 12 (190 us; 16: 199, 8: 200);  1,000 x 16: 14 (152; 16:
// 164);  800 x 16 bf16: 11 (111; 16: 138);  333 x 7 bf16: 4 (49; 16: 67);  100 x 16 MXFP8: 3 (28; 16: 44).
int decode_tile(int N, int H, int sms) {
  int best = 1;
  long long least = 0;
  for (int ts = 1; ts <= TILE_MAX; ++ts) {
    const long long ctas = (long long)((N + ts - 1) / ts) * H, rounds = (ctas + 4ll * sms - 1) / (4ll * sms);
    const long long cost = rounds * (ts + 4);
    if (ts == 1 || cost < least) {
      least = cost;
      best = ts;
    }
  }
  return best;
}

template <bool MX>
cudaError_t launch_decode_tile(const void* q, const void* k, const void* v, const float* log_lambda, float scale,
                               const float* pool, int pool_rows, const int32_t* prefix_row, const TailArgs& t, void* o,
                               int N, int H, unsigned* err, unsigned long long wait_ns, cudaStream_t s) {
  static std::atomic<int> sms_of[64];  // per device: its SM count, once the kernel's shared memory is allowed
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < 64 ? sms_of[dev].load() : 0;
  if (sms == 0) {
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(prefix_decode_tile_kernel<MX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)PdSmem<MX>::BYTES)) != cudaSuccess)
      return e;
    if (dev < 64) sms_of[dev].store(sms);
  }
  const int ts = decode_tile(N, H, sms);
  const unsigned blocks = (unsigned)((N + ts - 1) / ts) * (unsigned)H;
  using BF = __nv_bfloat16;
  prefix_decode_tile_kernel<MX><<<blocks, PD_THREADS, PdSmem<MX>::BYTES, s>>>(
      (const BF*)q, (const BF*)k, (const BF*)v, log_lambda, scale, pool, pool_rows, prefix_row, t, (BF*)o, N, H, ts, err,
      wait_ns);
  return cudaGetLastError();
}

// dpool[p] = sum of dh0[n] over the sequences n that started from row p, in the order of n (so the
// result does not depend on the schedule); zeros for a row that none started from.
// Bound by reading the per-sequence gradients once: 75 MB for 64 sequences x 16 heads, 15 us.
constexpr int RED_THREADS = 256;
constexpr int STATE4 = DK * DV / 4;
constexpr int RED_CTAS = STATE4 / RED_THREADS;  // 18 per (row, head)

__global__ void __launch_bounds__(RED_THREADS)
prefix_grad_kernel(const float4* __restrict__ dh0, const int32_t* __restrict__ prefix_row, int n_seq, int H,
                   float4* __restrict__ dpool, int pool_rows, [[maybe_unused]] unsigned* err) {
  __shared__ int s_n[RED_THREADS];
  __shared__ int s_warp[RED_THREADS / 32];
  const int part = (int)(blockIdx.x % RED_CTAS);
  const unsigned ph = blockIdx.x / RED_CTAS;
  const int p = (int)(ph / (unsigned)H), h = (int)(ph % (unsigned)H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int e = part * RED_THREADS + tid;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int n0 = 0; n0 < n_seq; n0 += RED_THREADS) {
    // the sequences of row p among these, packed in order
    const bool mine = n0 + tid < n_seq && prefix_row[n0 + tid] == p;
    const unsigned vote = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) s_warp[warp] = __popc(vote);
    __syncthreads();
    int before = 0, count = 0;
#pragma unroll
    for (int w = 0; w < RED_THREADS / 32; ++w) {
      before += w < warp ? s_warp[w] : 0;
      count += s_warp[w];
    }
    if (mine) s_n[before + __popc(vote & ((1u << lane) - 1u))] = n0 + tid;
    __syncthreads();
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      if (!state_in_bounds(s_n[i], n_seq, h, H, err)) continue;
      const float4 g = dh0[((long long)s_n[i] * H + h) * STATE4 + e];
      s.x += g.x;
      s.y += g.y;
      s.z += g.z;
      s.w += g.w;
    }
    __syncthreads();
  }
  if (state_in_bounds(p, pool_rows, h, H, err)) dpool[((long long)p * H + h) * STATE4 + e] = s;
}

bool aligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
int to_status(cudaError_t e) { return e == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH; }

}  // namespace
}  // namespace gla

extern "C" {

int gla_prefix_decode_step(const void* q, const void* k, const void* v, const float* log_lambda, float scale,
                           const float* pool, int pool_rows, const int32_t* prefix_row, const gla_tail* tail,
                           const int32_t* tail_slot, const int32_t* tail_len, void* o, int N, int H, int dk, int dv,
                           int dtype, gla_stream_t stream) {
  if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_DTYPE;
  if (dk != GLA_DK || dv != GLA_DV) return GLA_ERR_UNSUPPORTED;
  if (N < 0 || H < 1 || pool_rows < 0) return GLA_ERR_SHAPE;
  if ((long long)N * H >= (1ll << 31)) return GLA_ERR_SHAPE;
  gla::TailArgs t;
  int rc = gla::check_tail(tail, H, &t);
  if (rc || N == 0) return rc;
  if (!q || !k || !v || !log_lambda || !pool || !prefix_row || !tail_len || !o) return GLA_ERR_NULL;
  if (!tail_slot && tail->rows < N) return GLA_ERR_SHAPE;
  for (const void* p : {q, k, v, (const void*)o, (const void*)pool, (const void*)log_lambda})
    if (!gla::aligned(p, 16)) return GLA_ERR_ALIGN;
  for (const int32_t* p : {prefix_row, tail_slot, tail_len})
    if (!gla::aligned(p, 4)) return GLA_ERR_ALIGN;
  unsigned* err;
  unsigned long long wait_ns;
  if ((rc = gla::current_device_state(&err, &wait_ns))) return rc;
  wait_ns |= gla::debug_give_up();
  t.slot = tail_slot;
  t.len = tail_len;
  const bool mx = tail->format == GLA_TAIL_MXFP8;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == GLA_F32) {
    // four sequences a CTA once that leaves two CTAs for every SM (152); fewer spread one by one
    const int ts = (long long)((N + gla::DEC_TILE - 1) / gla::DEC_TILE) * H >= 2 * 152 ? gla::DEC_TILE : 1;
    const unsigned blocks = (unsigned)((N + ts - 1) / ts) * (unsigned)H;
    auto run = [&](auto kernel) {
      kernel<<<blocks, gla::DEC_THREADS, 0, s>>>((const float*)q, (const float*)k, (const float*)v, log_lambda, scale, pool,
                                                 pool_rows, prefix_row, t, (float*)o, N, H, ts, err);
    };
    if (mx) run(gla::prefix_decode_kernel<true>);
    else run(gla::prefix_decode_kernel<false>);
    return gla::to_status(cudaGetLastError());
  }
  return gla::to_status(mx ? gla::launch_decode_tile<true>(q, k, v, log_lambda, scale, pool, pool_rows, prefix_row, t, o,
                                                           N, H, err, wait_ns, s)
                           : gla::launch_decode_tile<false>(q, k, v, log_lambda, scale, pool, pool_rows, prefix_row, t, o,
                                                            N, H, err, wait_ns, s));
}

size_t gla_prefix_bwd_workspace_bytes(int n_seq, int T, int H, int dtype) {
  if (n_seq < 0 || T < 0 || H < 1 || (dtype != GLA_BF16 && dtype != GLA_F32)) return 0;
  const size_t states = (size_t)n_seq * (size_t)H * (GLA_DK * GLA_DV * sizeof(float));
  return (gla_bwd_workspace_bytes(n_seq, T, H, 1, dtype) + 255) / 256 * 256 + states;
}

int gla_prefix_fwd(const void* q, const void* k, const void* v, const float* log_lambda, const float* pool,
                   int pool_rows, const int32_t* prefix_row, float scale, void* o, float* hT,
                   const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv, int dtype, void* workspace,
                   size_t ws_bytes, gla_stream_t stream) {
  long long tokens = 0;
  int rc = gla::check_chunk_sizes(n_seq, T, H, dk, dv, dtype, cu_seqlens, &tokens);
  if (rc) return rc;
  if (pool_rows < 0) return GLA_ERR_SHAPE;
  if (n_seq == 0) return GLA_OK;
  if (!cu_seqlens || !log_lambda || !pool || !prefix_row) return GLA_ERR_NULL;
  if (!gla::aligned(cu_seqlens, 4) || !gla::aligned(prefix_row, 4)) return GLA_ERR_ALIGN;
  if (T > 0 && (!q || !k || !v || !o)) return GLA_ERR_NULL;
  for (const void* p : {q, k, v, (const void*)o, (const void*)pool, (const void*)hT, (const void*)log_lambda})
    if (!gla::aligned(p, 16)) return GLA_ERR_ALIGN;
  if (!workspace || ws_bytes < gla_workspace_bytes(n_seq, H)) return GLA_ERR_WORKSPACE;
  if (!gla::aligned(workspace, 16)) return GLA_ERR_ALIGN;
  gla::ChunkArgs a = {};
  if ((rc = gla::current_device_state(&a.err, &a.wait_ns))) return rc;
  a.q = q;
  a.k = k;
  a.v = v;
  a.log_lambda = log_lambda;
  a.h0 = pool;
  a.h0_row = prefix_row;
  a.h0_rows = pool_rows;
  a.o = o;
  a.hT = hT;
  a.cu_seqlens = cu_seqlens;
  a.scale = scale;
  a.n_seq = n_seq;
  a.T = T;
  a.H = H;
  cudaStream_t s = (cudaStream_t)stream;
  int32_t* order = (int32_t*)((char*)workspace + 256);
  if (gla::launch_lpt_order(cu_seqlens, n_seq, order, s) != cudaSuccess) return GLA_ERR_LAUNCH;
  a.order = order;
  return gla::to_status(dtype == GLA_F32 ? gla::launch_simt_fwd(a, s) : gla::launch_tc_fwd(a, s));
}

int gla_prefix_bwd(const void* q, const void* k, const void* v, const float* log_lambda, const float* pool,
                   int pool_rows, const int32_t* prefix_row, float scale, const void* dO, const float* dhT, void* dq,
                   void* dk, void* dv, float* dpool, const int32_t* cu_seqlens, int n_seq, int T, int H, int dk_size,
                   int dv_size, int dtype, void* workspace, size_t ws_bytes, gla_stream_t stream) {
  long long tokens = 0;
  int rc = gla::check_chunk_sizes(n_seq, T, H, dk_size, dv_size, dtype, cu_seqlens, &tokens);
  if (rc) return rc;
  if (pool_rows < 0) return GLA_ERR_SHAPE;
  if ((long long)pool_rows * H * gla::RED_CTAS >= (1ll << 31)) return GLA_ERR_SHAPE;
  if (n_seq > 0) {
    if (!cu_seqlens || !log_lambda || !pool || !prefix_row) return GLA_ERR_NULL;
    if (!gla::aligned(prefix_row, 4)) return GLA_ERR_ALIGN;
    if (T > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv)) return GLA_ERR_NULL;
    for (const void* p : {q, k, v, dO, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)pool,
                          (const void*)dhT, (const void*)log_lambda})
      if (!gla::aligned(p, 16)) return GLA_ERR_ALIGN;
    if (!workspace || ws_bytes < gla_prefix_bwd_workspace_bytes(n_seq, T, H, dtype)) return GLA_ERR_WORKSPACE;
    if (!gla::aligned(workspace, 16)) return GLA_ERR_ALIGN;
  }
  if (!gla::aligned(dpool, 16)) return GLA_ERR_ALIGN;
  const bool reduce = dpool && pool_rows > 0;
  if (n_seq == 0 && !reduce) return GLA_OK;
  gla::ChunkArgs a = {};
  if ((rc = gla::current_device_state(&a.err, &a.wait_ns))) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  float* dh0 = nullptr;
  if (n_seq > 0) {
    char* ws = (char*)workspace;
    dh0 = (float*)(ws + (gla_bwd_workspace_bytes(n_seq, T, H, 1, dtype) + 255) / 256 * 256);
    a.q = q;
    a.k = k;
    a.v = v;
    a.dO = dO;
    a.log_lambda = log_lambda;
    a.h0 = pool;
    a.h0_row = prefix_row;
    a.h0_rows = pool_rows;
    a.dhT = dhT;
    a.o = dq;
    a.dk = dk;
    a.dv = dv;
    a.hT = reduce ? dh0 : nullptr;
    a.cu_seqlens = cu_seqlens;
    a.scale = scale;
    a.n_seq = n_seq;
    a.T = T;
    a.H = H;
    int32_t* order = (int32_t*)(ws + 256);
    if (gla::launch_lpt_order(cu_seqlens, n_seq, order, s) != cudaSuccess) return GLA_ERR_LAUNCH;
    a.order = order;
    cudaError_t e;
    if (dtype == GLA_F32) {
      e = gla::launch_simt_bwd(1, a, s);
    } else {
      const size_t head = gla_workspace_bytes(n_seq, H);
      const size_t acc = (gla::tc_bwd_acc_bytes(tokens, H) + 255) / 256 * 256;
      e = gla::launch_tc_bwd(a, (float*)(ws + head), (float*)(ws + head + acc), s);
    }
    if (e != cudaSuccess) return GLA_ERR_LAUNCH;
  }
  if (reduce) {
    gla::prefix_grad_kernel<<<(unsigned)pool_rows * (unsigned)H * gla::RED_CTAS, gla::RED_THREADS, 0, s>>>(
        (const float4*)dh0, prefix_row, n_seq, H, (float4*)dpool, pool_rows, a.err);
    return gla::to_status(cudaGetLastError());
  }
  return GLA_OK;
}

}  // extern "C"
