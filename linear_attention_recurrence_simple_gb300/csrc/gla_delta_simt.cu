// The gated delta rule in fp32 on the CUDA cores (the all-fp32 mode).
//
// Four kernels, see gla_delta.cuh for the formulas:
//   prep    one CTA a (chunk, head): decays, P, M and the triangular system's Z
//   scan    one CTA a (sequence, head, 32 columns of d_v): the chunks in order; columns of S never meet, so the
//           tiles are independent.  In the backward it keeps each chunk's S0 and X instead of writing o
//   rscan   the same in reverse for dS; writes dv, dS1 of every chunk and its columns' part of dbeta
//   grads   one CTA a (chunk, head): dq, dk, dg, and dbeta's parts summed in tile order
// The operands of a product stand in shared memory with an odd row stride; every thread has a small tile of the
// result in registers.  Bound by shared-memory loads (about 0.7 a multiply-add).
#include "gla_delta.cuh"
#include "gla_once.cuh"

namespace gla {
namespace {

constexpr int SB = 32;             // columns of d_v a scan CTA has
constexpr int SNB = DV / SB;       // 6
constexpr int THREADS = 256;
constexpr int KS = DK + 1, CS = DC + 1, BS = SB + 1;  // row strides in shared memory
constexpr int ZS = DC + 4;         // the solve reads rows in vectors of four

// Workspace of a (chunk place, head), in floats.
constexpr long long WS_Z = 0, WS_P = WS_Z + DC * DC, WS_GT = WS_P + DC * DC, WS_FWD = WS_GT + 5 * DC;
constexpr long long WS_S0 = WS_FWD, WS_X = WS_S0 + DK * DV, WS_DS = WS_X + DC * DV, WS_BWD = WS_DS + DK * DV;
enum { GT_HI = 0, GT_LO = DC, GT_F = 2 * DC, GT_E = 3 * DC, GT_B = 4 * DC };  // sums, e^G, e^(G_C - G), beta

template <bool BWD>
__device__ __forceinline__ float* ws_of(const DeltaArgs& a, int slot, int h) {
  return reinterpret_cast<float*>(a.ws) + ((long long)slot * a.H + h) * (BWD ? WS_BWD : WS_FWD);
}
// rows [0, C) of a [tokens, H, D] tensor, columns [c0, c0 + W), zeros from row `len` on
template <int W, int STRIDE, class T>
__device__ __forceinline__ void load_rows(float* dst, const T* src, long long t0, int len, int H, int h, int D, int c0) {
  for (int e = threadIdx.x; e < DC * W; e += THREADS) {
    const int i = e / W, c = e % W;
    dst[i * STRIDE + c] = i < len ? to_f(src[((t0 + i) * H + h) * D + c0 + c]) : 0.f;
  }
}
// acc[r][c] += sum_k A(k, row r) B(k, column c): rows i0 + r * IS, columns j0 + c * JS
template <int NR, int NC, int K, class FA, class FB>
__device__ __forceinline__ void gemm(float (&acc)[NR][NC], FA fa, FB fb) {
#pragma unroll 4
  for (int k = 0; k < K; ++k) {
    float x[NR], y[NC];
#pragma unroll
    for (int r = 0; r < NR; ++r) x[r] = fa(k, r);
#pragma unroll
    for (int c = 0; c < NC; ++c) y[c] = fb(k, c);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[r][c] = fmaf(x[r], y[c], acc[r][c]);
  }
}

// ---- prep -------------------------------------------------------------------------------------
template <class T, bool BWD>
__global__ void __launch_bounds__(THREADS) delta_prep_simt_kernel(const DeltaArgs a) {
  extern __shared__ float sm[];
  float* const sk = sm;                // [64][97], then M and M B [64][68]
  float* const sq = sk + DC * KS;
  __shared__ float2 sg[DC];
  __shared__ float sb[DC];
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) return;
  float* const ws = ws_of<BWD>(a, slot, h);
  load_rows<DK, KS>(sk, (const T*)a.k, ch.t0, ch.len, a.H, h, DK, 0);
  load_rows<DK, KS>(sq, (const T*)a.q, ch.t0, ch.len, a.H, h, DK, 0);
  if (tid < 32) {
    const T* g = (const T*)a.g + ch.t0 * a.H + h;
    const T* b = (const T*)a.beta + ch.t0 * a.H + h;
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * tid + e;
      x[e] = i < ch.len ? to_f(g[(long long)i * a.H]) : 0.f;
      sb[i] = i < ch.len ? to_f(b[(long long)i * a.H]) : 0.f;
    }
    float2 s0, s1;
    delta_sums(x[0], x[1], s0, s1);
    sg[2 * tid] = s0;
    sg[2 * tid + 1] = s1;
  }
  __syncthreads();
  if (tid < DC) {
    ws[WS_GT + GT_HI + tid] = sg[tid].x;
    ws[WS_GT + GT_LO + tid] = sg[tid].y;
    ws[WS_GT + GT_F + tid] = delta_decay0(sg[tid]);
    ws[WS_GT + GT_E + tid] = delta_decay(sg[DC - 1], sg[tid]);
    ws[WS_GT + GT_B + tid] = sb[tid];
  }
  const int ti = tid / 16, tj = tid % 16;
  float kk[4][4] = {}, qk[4][4] = {};
  gemm<4, 4, DK>(kk, [&](int x, int r) { return sk[(ti + 16 * r) * KS + x]; }, [&](int x, int c) { return sk[(tj + 16 * c) * KS + x]; });
  gemm<4, 4, DK>(qk, [&](int x, int r) { return sq[(ti + 16 * r) * KS + x]; }, [&](int x, int c) { return sk[(tj + 16 * c) * KS + x]; });
  __syncthreads();
  float* const m = sm;
  float* const mb = sm + DC * ZS;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int i = ti + 16 * r, j = tj + 16 * c;
      const float d = j <= i ? delta_decay(sg[i], sg[j]) : 0.f;
      ws[WS_P + i * DC + j] = j <= i ? d * qk[r][c] : 0.f;
      const float x = j < i ? d * kk[r][c] : 0.f;
      m[i * ZS + j] = x;
      mb[i * ZS + j] = x * sb[j];
    }
  __syncthreads();
  if (tid < DC) {
    float z[DC];
    delta_solve_column<ZS>(m, mb, tid, z);
#pragma unroll
    for (int i = 0; i < DC; ++i) ws[WS_Z + i * DC + tid] = z[i];
  }
}

// ---- forward scan ---------------------------------------------------------------------------
constexpr int SCAN_FLOATS = DK * BS + 2 * DC * KS + 2 * DC * CS + 2 * DC * BS + 3 * DC;

template <class T, bool BWD>
__global__ void __launch_bounds__(THREADS) delta_scan_simt_kernel(const DeltaArgs a) {
  extern __shared__ float sm[];
  float* const S = sm;                 // [96][33]
  float* const sk = S + DK * BS;       // [64][97]
  float* const sq = sk + DC * KS;
  float* const sz = sq + DC * KS;      // [64][65]
  float* const sp = sz + DC * CS;
  float* const sr = sp + DC * CS;      // [64][33]: B R
  float* const su = sr + DC * BS;      // [64][33]: U
  float* const sf = su + DC * BS;      // e^G, e^(G_C - G), beta
  const int tile = blockIdx.x % SNB, nh = blockIdx.x / SNB, h = nh % a.H, n = nh / a.H, tid = threadIdx.x;
  const int c0 = tile * SB;
  const DeltaSeq s = delta_seq(a, n);
  const int from = a.h0 ? delta_row(a.h0_row, a.h0_rows, n, a.err) : -1;
  for (int e = tid; e < DK * SB; e += THREADS)
    S[e / SB * BS + e % SB] = from >= 0 ? a.h0[(((long long)from * a.H + h) * DK + e / SB) * DV + c0 + e % SB] : 0.f;
  const int ti = tid / 16, tj = tid % 16;  // rows ti + 16 r, columns tj + 16 c
  for (int c = 0; c * DC < s.len; ++c) {
    const int len = min(DC, s.len - c * DC);
    const long long t0 = s.begin + (long long)c * DC;
    float* const ws = ws_of<BWD>(a, s.slot0 + c, h);
    __syncthreads();
    load_rows<DK, KS>(sk, (const T*)a.k, t0, len, a.H, h, DK, 0);
    if (!BWD) load_rows<DK, KS>(sq, (const T*)a.q, t0, len, a.H, h, DK, 0);
    for (int e = tid; e < DC * DC; e += THREADS) {
      sz[e / DC * CS + e % DC] = ws[WS_Z + e];
      if (!BWD) sp[e / DC * CS + e % DC] = ws[WS_P + e];
    }
    if (tid < 3 * DC) sf[tid] = ws[WS_GT + GT_F + tid];
    if (BWD)
      for (int e = tid; e < DK * SB; e += THREADS) ws[WS_S0 + e / SB * DV + c0 + e % SB] = S[e / SB * BS + e % SB];
    __syncthreads();
    float ks[4][2] = {}, qs[4][2] = {}, r[4][2];
    gemm<4, 2, DK>(ks, [&](int x, int i) { return sk[(ti + 16 * i) * KS + x]; }, [&](int x, int j) { return S[x * BS + tj + 16 * j]; });
    if (!BWD)
      gemm<4, 2, DK>(qs, [&](int x, int i) { return sq[(ti + 16 * i) * KS + x]; }, [&](int x, int j) { return S[x * BS + tj + 16 * j]; });
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = ti + 16 * i, col = tj + 16 * j;
        const float v = row < len ? to_f(((const T*)a.v)[((t0 + row) * a.H + h) * DV + c0 + col]) : 0.f;
        r[i][j] = fmaf(-sf[row], ks[i][j], v);
        sr[row * BS + col] = sf[2 * DC + row] * r[i][j];
      }
    __syncthreads();
    float zr[4][2] = {};
    gemm<4, 2, DC>(zr, [&](int x, int i) { return sz[(ti + 16 * i) * CS + x]; }, [&](int x, int j) { return sr[x * BS + tj + 16 * j]; });
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = ti + 16 * i, col = tj + 16 * j;
        const float x = r[i][j] - zr[i][j];
        su[row * BS + col] = sf[2 * DC + row] * x;
        if (BWD) ws[WS_X + row * DV + c0 + col] = x;
      }
    __syncthreads();
    if (!BWD) {
      float pu[4][2] = {};
      gemm<4, 2, DC>(pu, [&](int x, int i) { return sp[(ti + 16 * i) * CS + x]; }, [&](int x, int j) { return su[x * BS + tj + 16 * j]; });
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = ti + 16 * i, col = tj + 16 * j;
          if (row < len)
            ((T*)a.o)[((t0 + row) * a.H + h) * DV + c0 + col] = from_f<T>(a.scale * fmaf(sf[row], qs[i][j], pu[i][j]));
        }
    }
    float ds[6][2] = {};
    gemm<6, 2, DC>(ds, [&](int x, int i) { return sk[x * KS + ti + 16 * i] * sf[DC + x]; }, [&](int x, int j) { return su[x * BS + tj + 16 * j]; });
    const float last = sf[DC - 1];
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float* const at = S + (ti + 16 * i) * BS + tj + 16 * j;  // (this thread's own, and nothing reads S here)
        *at = fmaf(last, *at, ds[i][j]);
      }
  }
  __syncthreads();
  if (!BWD && a.hT) {
    const int to = delta_row(a.hT_row, a.hT_rows, n, a.err);
    if (to >= 0)
      for (int e = tid; e < DK * SB; e += THREADS)
        a.hT[(((long long)to * a.H + h) * DK + e / SB) * DV + c0 + e % SB] = S[e / SB * BS + e % SB];
  }
}

// ---- reverse scan ---------------------------------------------------------------------------
// (the same shared memory as the scan: dO in the place of U, and the part of dbeta behind the decays)
template <class T>
__global__ void __launch_bounds__(THREADS) delta_rscan_simt_kernel(const DeltaArgs a, float* dbeta_part) {
  extern __shared__ float sm[];
  float* const S = sm;  // dS
  float* const sk = S + DK * BS;
  float* const sq = sk + DC * KS;
  float* const sz = sq + DC * KS;
  float* const sp = sz + DC * CS;
  float* const sw = sp + DC * CS;   // B dU, then -e^G dR
  float* const sd = sw + DC * BS;   // dO
  float* const sf = sd + DC * BS;
  const int tile = blockIdx.x % SNB, nh = blockIdx.x / SNB, h = nh % a.H, n = nh / a.H, tid = threadIdx.x;
  const int c0 = tile * SB;
  const DeltaSeq s = delta_seq(a, n);
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  for (int e = tid; e < DK * SB; e += THREADS)
    S[e / SB * BS + e % SB] = a.dhT ? a.dhT[(((long long)n * a.H + h) * DK + e / SB) * DV + c0 + e % SB] : 0.f;
  const int ti = tid / 16, tj = tid % 16;
  for (int c = (s.len + DC - 1) / DC - 1; c >= 0; --c) {
    const int len = min(DC, s.len - c * DC);
    const long long t0 = s.begin + (long long)c * DC;
    float* const ws = ws_of<true>(a, s.slot0 + c, h);
    __syncthreads();
    load_rows<DK, KS>(sk, (const T*)a.k, t0, len, a.H, h, DK, 0);
    load_rows<DK, KS>(sq, (const T*)a.q, t0, len, a.H, h, DK, 0);
    load_rows<SB, BS>(sd, (const T*)a.dO, t0, len, a.H, h, DV, c0);
    for (int e = tid; e < DC * DC; e += THREADS) {
      sz[e / DC * CS + e % DC] = ws[WS_Z + e];
      sp[e / DC * CS + e % DC] = ws[WS_P + e];
    }
    if (tid < 3 * DC) sf[tid] = ws[WS_GT + GT_F + tid];
    for (int e = tid; e < DK * SB; e += THREADS) ws[WS_DS + e / SB * DV + c0 + e % SB] = S[e / SB * BS + e % SB];
    __syncthreads();
    float kd[4][2] = {}, pd[4][2] = {}, du[4][2];
    gemm<4, 2, DK>(kd, [&](int x, int i) { return sk[(ti + 16 * i) * KS + x]; }, [&](int x, int j) { return S[x * BS + tj + 16 * j]; });
    gemm<4, 2, DC>(pd, [&](int x, int i) { return sp[x * CS + ti + 16 * i]; }, [&](int x, int j) { return sd[x * BS + tj + 16 * j]; });
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = ti + 16 * i;
        du[i][j] = fmaf(sf[DC + row], kd[i][j], a.scale * pd[i][j]);
        sw[row * BS + tj + 16 * j] = sf[2 * DC + row] * du[i][j];
      }
    __syncthreads();
    float zw[4][2] = {}, part[4] = {};
    gemm<4, 2, DC>(zw, [&](int x, int i) { return sz[x * CS + ti + 16 * i]; }, [&](int x, int j) { return sw[x * BS + tj + 16 * j]; });
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = ti + 16 * i;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = tj + 16 * j;
        const float dut = du[i][j] - zw[i][j], dr = sf[2 * DC + row] * dut;
        part[i] = fmaf(dut, ws[WS_X + row * DV + c0 + col], part[i]);
        if (row < len) ((T*)a.dv)[((t0 + row) * a.H + h) * DV + c0 + col] = from_f<T>(dr);
        sw[row * BS + col] = -sf[row] * dr;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) part[i] += __shfl_xor_sync(0xffffffffu, part[i], off);
      if (tj == 0 && row < len) dbeta_part[((long long)tile * tokens + t0 + row) * a.H + h] = part[i];
    }
    __syncthreads();
    float ds[6][2] = {};
    gemm<6, 2, DC>(ds, [&](int x, int i) { return sq[x * KS + ti + 16 * i] * (a.scale * sf[x]); }, [&](int x, int j) { return sd[x * BS + tj + 16 * j]; });
    gemm<6, 2, DC>(ds, [&](int x, int i) { return sk[x * KS + ti + 16 * i]; }, [&](int x, int j) { return sw[x * BS + tj + 16 * j]; });
    const float last = sf[DC - 1];
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float* const at = S + (ti + 16 * i) * BS + tj + 16 * j;
        *at = fmaf(last, *at, ds[i][j]);
      }
  }
  __syncthreads();
  if (a.dh0)
    for (int e = tid; e < DK * SB; e += THREADS)
      a.dh0[(((long long)n * a.H + h) * DK + e / SB) * DV + c0 + e % SB] = S[e / SB * BS + e % SB];
}

// ---- gradients of the chunk ------------------------------------------------------------------
constexpr int GRAD_FLOATS = 2 * DC * KS + 3 * DC * BS + 2 * DK * BS + 2 * DC;
static_assert(2 * DC * CS <= 3 * DC * BS + 2 * DK * BS, "the masked products take the pieces' place");

template <class T>
__global__ void __launch_bounds__(THREADS) delta_grads_simt_kernel(const DeltaArgs a, const float* dbeta_part) {
  extern __shared__ float sm[];
  float* const sk = sm;
  float* const sq = sk + DC * KS;
  float* const sdo = sq + DC * KS;       // [64][33] dO, dR, U
  float* const sdr = sdo + DC * BS;
  float* const su = sdr + DC * BS;
  float* const ss = su + DC * BS;        // [96][33] S0, dS1
  float* const sd = ss + DK * BS;
  float* const sdg = sd + DK * BS;       // [64] dG
  __shared__ float red[THREADS / 32];
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) return;
  const float* const ws = ws_of<true>(a, slot, h);
  const float* const gt = ws + WS_GT;
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  load_rows<DK, KS>(sk, (const T*)a.k, ch.t0, ch.len, a.H, h, DK, 0);
  load_rows<DK, KS>(sq, (const T*)a.q, ch.t0, ch.len, a.H, h, DK, 0);
  const int ti = tid / 16, tj = tid % 16;
  float dp[4][4] = {}, dm[4][4] = {}, dqi[4][6] = {}, dkr[4][6] = {}, dks[4][6] = {}, frob = 0.f;
  for (int c0 = 0; c0 < DV; c0 += SB) {
    __syncthreads();
    load_rows<SB, BS>(sdo, (const T*)a.dO, ch.t0, ch.len, a.H, h, DV, c0);
    load_rows<SB, BS>(sdr, (const T*)a.dv, ch.t0, ch.len, a.H, h, DV, c0);
    for (int e = tid; e < DC * SB; e += THREADS) {
      const int i = e / SB;
      su[i * BS + e % SB] = i < ch.len ? gt[GT_B + i] * ws[WS_X + i * DV + c0 + e % SB] : 0.f;
    }
    for (int e = tid; e < DK * SB; e += THREADS) {
      const float x = ws[WS_S0 + e / SB * DV + c0 + e % SB], y = ws[WS_DS + e / SB * DV + c0 + e % SB];
      ss[e / SB * BS + e % SB] = x;
      sd[e / SB * BS + e % SB] = y;
      frob = fmaf(x, y, frob);
    }
    __syncthreads();
    gemm<4, 4, SB>(dp, [&](int x, int i) { return sdo[(ti + 16 * i) * BS + x]; }, [&](int x, int j) { return su[(tj + 16 * j) * BS + x]; });
    gemm<4, 4, SB>(dm, [&](int x, int i) { return sdr[(ti + 16 * i) * BS + x]; }, [&](int x, int j) { return su[(tj + 16 * j) * BS + x]; });
    gemm<4, 6, SB>(dqi, [&](int x, int i) { return sdo[(ti + 16 * i) * BS + x]; }, [&](int x, int j) { return ss[(tj + 16 * j) * BS + x]; });
    gemm<4, 6, SB>(dkr, [&](int x, int i) { return sdr[(ti + 16 * i) * BS + x]; }, [&](int x, int j) { return ss[(tj + 16 * j) * BS + x]; });
    gemm<4, 6, SB>(dks, [&](int x, int i) { return su[(ti + 16 * i) * BS + x]; }, [&](int x, int j) { return sd[(tj + 16 * j) * BS + x]; });
  }
  __syncthreads();
  float* const es = sdo;              // [64][65] Es, F
  float* const fm = sdo + DC * CS;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int i = ti + 16 * r, j = tj + 16 * c;
      const float d = j <= i ? delta_decay(make_float2(gt[GT_HI + i], gt[GT_LO + i]), make_float2(gt[GT_HI + j], gt[GT_LO + j])) : 0.f;
      es[i * CS + j] = j <= i ? a.scale * d * dp[r][c] : 0.f;
      fm[i * CS + j] = j < i ? -d * dm[r][c] : 0.f;
    }
  __syncthreads();
  float q1[4][6] = {}, k1[4][6] = {}, k2[4][6] = {};  // Es K;  Es^T Q + F^T K;  F K
  gemm<4, 6, DC>(q1, [&](int x, int i) { return es[(ti + 16 * i) * CS + x]; }, [&](int x, int j) { return sk[x * KS + tj + 16 * j]; });
  gemm<4, 6, DC>(k1, [&](int x, int i) { return es[x * CS + ti + 16 * i]; }, [&](int x, int j) { return sq[x * KS + tj + 16 * j]; });
  gemm<4, 6, DC>(k1, [&](int x, int i) { return fm[x * CS + ti + 16 * i]; }, [&](int x, int j) { return sk[x * KS + tj + 16 * j]; });
  gemm<4, 6, DC>(k2, [&](int x, int i) { return fm[(ti + 16 * i) * CS + x]; }, [&](int x, int j) { return sk[x * KS + tj + 16 * j]; });
  float at_end = 0.f;  // sum_j k_j . (e^(G_C - G_j) dS1 u_j), this thread's part
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = ti + 16 * r;
    const float f = gt[GT_F + i], e = gt[GT_E + i];
    float dg = 0.f;
#pragma unroll
    for (int c = 0; c < 6; ++c) {
      const int x = tj + 16 * c;
      const float q = sq[i * KS + x], k = sk[i * KS + x];
      const float dq = fmaf(a.scale * f, dqi[r][c], q1[r][c]);
      const float minus = fmaf(e, dks[r][c], k1[r][c]), plus = fmaf(-f, dkr[r][c], k2[r][c]);
      at_end = fmaf(k, e * dks[r][c], at_end);
      dg = fmaf(q, dq, fmaf(k, plus - minus, dg));
      if (i < ch.len) {
        ((T*)a.dq)[((ch.t0 + i) * a.H + h) * DK + x] = from_f<T>(dq);
        ((T*)a.dk)[((ch.t0 + i) * a.H + h) * DK + x] = from_f<T>(minus + plus);
      }
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) dg += __shfl_xor_sync(0xffffffffu, dg, off);
    if (tj == 0) sdg[i] = dg;
  }
  at_end = fmaf(gt[GT_F + DC - 1], frob, at_end);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) at_end += __shfl_xor_sync(0xffffffffu, at_end, off);
  if ((tid & 31) == 0) red[tid / 32] = at_end;
  __syncthreads();
  if (tid < 32) {  // dg_t = the sum of dG_i over i >= t, and of what hangs on G_C
    float end = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) end += red[w];
    const float hi = sdg[2 * tid + 1];
    float run = sdg[2 * tid] + hi;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float up = __shfl_down_sync(0xffffffffu, run, off);
      if (tid + off < 32) run += up;
    }
    const float pair = run - (sdg[2 * tid] + hi);  // behind this pair
    sdg[2 * tid] = run + end;
    sdg[2 * tid + 1] = pair + hi + end;
  }
  __syncthreads();
  if (tid < ch.len) {
    float b = 0.f;
#pragma unroll
    for (int t = 0; t < SNB; ++t) b += dbeta_part[((long long)t * tokens + ch.t0 + tid) * a.H + h];
    ((T*)a.dg)[(ch.t0 + tid) * a.H + h] = from_f<T>(sdg[tid]);
    ((T*)a.dbeta)[(ch.t0 + tid) * a.H + h] = from_f<T>(b);
  }
}

constexpr int PREP_BYTES = 2 * DC * KS * 4, SCAN_BYTES = SCAN_FLOATS * 4, GRAD_BYTES = GRAD_FLOATS * 4;
static_assert(2 * DC * ZS <= 2 * DC * KS, "M and M B take the place of K and Q");

template <class F>
cudaError_t allow(F* f, int bytes) {
  return cudaFuncSetAttribute((const void*)f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <class T>
cudaError_t allow_all() {
  static OncePerDevice<CudaDeviceApi> once;
  return once([] {
    for (cudaError_t e : {allow(delta_prep_simt_kernel<T, false>, PREP_BYTES), allow(delta_prep_simt_kernel<T, true>, PREP_BYTES),
                          allow(delta_scan_simt_kernel<T, false>, SCAN_BYTES), allow(delta_scan_simt_kernel<T, true>, SCAN_BYTES),
                          allow(delta_rscan_simt_kernel<T>, SCAN_BYTES), allow(delta_grads_simt_kernel<T>, GRAD_BYTES)})
      if (e != cudaSuccess) return e;
    return cudaSuccess;
  });
}

}  // namespace

size_t delta_simt_ws_bytes(long long slots, long long tokens, int H, bool bwd) {
  return (size_t)slots * H * (bwd ? WS_BWD : WS_FWD) * 4 + (bwd ? (size_t)SNB * tokens * H * 4 : 0);
}

template <class T>
static cudaError_t simt_fwd(const DeltaArgs& a, cudaStream_t st) {
  cudaError_t e = allow_all<T>();
  if (e != cudaSuccess) return e;
  if (a.slots > 0) delta_prep_simt_kernel<T, false><<<(unsigned)a.slots * a.H, THREADS, PREP_BYTES, st>>>(a);
  delta_scan_simt_kernel<T, false><<<(unsigned)a.n_seq * a.H * SNB, THREADS, SCAN_BYTES, st>>>(a);
  return cudaGetLastError();
}
template <class T>
static cudaError_t simt_bwd(const DeltaArgs& a, cudaStream_t st) {
  cudaError_t e = allow_all<T>();
  if (e != cudaSuccess) return e;
  float* part = reinterpret_cast<float*>(a.ws) + (long long)a.slots * a.H * WS_BWD;
  const unsigned chunks = (unsigned)a.slots * a.H, units = (unsigned)a.n_seq * a.H * SNB;
  if (a.slots > 0) {
    delta_prep_simt_kernel<T, true><<<chunks, THREADS, PREP_BYTES, st>>>(a);
    delta_scan_simt_kernel<T, true><<<units, THREADS, SCAN_BYTES, st>>>(a);
  }
  delta_rscan_simt_kernel<T><<<units, THREADS, SCAN_BYTES, st>>>(a, part);
  if (a.slots > 0) delta_grads_simt_kernel<T><<<chunks, THREADS, GRAD_BYTES, st>>>(a, part);
  return cudaGetLastError();
}

cudaError_t launch_delta_simt_fwd(const DeltaArgs& a, cudaStream_t st) { return simt_fwd<float>(a, st); }
cudaError_t launch_delta_simt_bwd(const DeltaArgs& a, cudaStream_t st) { return simt_bwd<float>(a, st); }

}  // namespace gla
