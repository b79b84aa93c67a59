// The gated delta rule in fp32 (the all-fp32 mode).
//
// Four kernels, see gla_delta.cuh for the formulas:
//   prep    one CTA a (chunk, head): decays, P, M and the triangular system's Z
//   scan    one CTA a (sequence, head, 32 columns of d_v): the chunks in order; columns of S never meet, so the
//           tiles are independent.  In the backward it keeps each chunk's S0 and X instead of writing o
//   rscan   the same in reverse for dS; writes dv, dS1 of every chunk and its columns' part of dbeta
//   grads   two CTAs a (chunk, head): dq, dk, dg, and dbeta's parts summed in tile order
// States, sums and everything between products are fp32.  The products are three of tf32 each (mma.sync): an operand keeps 22
// bits, sums are of 16 terms in the tensor cores, which cut them off, and of those in fp32: 1.8e-7 of the norm from the exact
// result, against 2.4e-7 with FMAs throughout and 1.5e-6 with the tensor cores' sums over all terms.  With FMAs the reads
// from shared memory were the bound (a 4 x 2 tile of a thread takes six vectors for 32 FMAs): 2 sequences of up to 150 tokens x
// 4 heads, scan 24 -> 22 us, rscan 36 -> 33, grads 49 -> 30; backward 117 -> 95 (with what came after, prep 13, scan 21, rscan
// 31, grads 30; 90).
// Operands stand in shared memory with the summed index contiguous (where both ways are needed, twice).  A chunk's loads go
// out together, in vectors, while the chunk before it is computed.  Bound by latency: eight warps an SM, and short calls have
// few CTAs.
#include "gla_delta.cuh"
#include "gla_once.cuh"

namespace gla {
namespace {

constexpr int SB = 32;             // columns of d_v a scan CTA has
constexpr int SNB = DV / SB;       // 6
constexpr int THREADS = 256;
constexpr int KS = DK + 16, CS = DC + 16, BS = SB + 16;  // row strides in shared memory: 16 mod 32 words

// Workspace of a (chunk place, head), in floats.
constexpr long long WS_Z = 0, WS_P = WS_Z + DC * DC, WS_GT = WS_P + DC * DC, WS_FWD = WS_GT + 5 * DC;
constexpr long long WS_S0 = WS_FWD, WS_X = WS_S0 + DK * DV, WS_DS = WS_X + DC * DV, WS_BWD = WS_DS + DK * DV;
enum { GT_HI = 0, GT_LO = DC, GT_F = 2 * DC, GT_E = 3 * DC, GT_B = 4 * DC };  // sums, e^G, e^(G_C - G), beta

template <bool BWD>
__device__ __forceinline__ float* ws_of(const DeltaArgs& a, int slot, int h) {
  return reinterpret_cast<float*>(a.ws) + ((long long)slot * a.H + h) * (BWD ? WS_BWD : WS_FWD);
}
// N vectors of four, this thread's x-th being vector tid + x * THREADS of the source: loaded together, then placed, with
// other work between the two where there is some.
template <int N>
struct Held {
  static constexpr int PER = (N + THREADS - 1) / THREADS;
  float4 v[PER];
  template <class G>
  __device__ __forceinline__ void fetch(G get) {
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int e = threadIdx.x + x * THREADS;
      v[x] = N % THREADS == 0 || e < N ? get(e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  template <class P>
  __device__ __forceinline__ void place(P put) const {
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const int e = threadIdx.x + x * THREADS;
      if (N % THREADS == 0 || e < N) put(e, v[x]);
    }
  }
};
__device__ __forceinline__ void put_row(float* at, float4 v) { *reinterpret_cast<float4*>(at) = v; }
template <int STRIDE>
__device__ __forceinline__ void put_column(float* at, float4 v) {
  at[0] = v.x;
  at[STRIDE] = v.y;
  at[2 * STRIDE] = v.z;
  at[3 * STRIDE] = v.w;
}
// Vector e of rows of W floats: a warp has 8 rows x 64 bytes, so that columns, too, go to shared memory without conflicts (a
// row after the other, its stores have 12 of 32 lanes on a bank).
template <int W>
struct At {
  int row, col;
  __device__ __forceinline__ explicit At(int e) {
    const int tile = e / 32, lane = e % 32;
    row = 8 * (tile / (W / 16)) + lane / 4;
    col = 16 * (tile % (W / 16)) + 4 * (lane % 4);
  }
};
// Rows [0, C) of a [tokens, H, D] tensor, columns [c0, c0 + W), zeros from row `len` on.
template <int W>
struct Rows : Held<DC * W / 4> {
  __device__ __forceinline__ void fetch(const void* src, long long t0, int len, int H, int h, int D, int c0) {
    Held<DC * W / 4>::fetch([&](int e) {
      const At<W> at(e);
      return at.row < len ? *reinterpret_cast<const float4*>((const float*)src + ((t0 + at.row) * H + h) * D + c0 + at.col)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    });
  }
  template <class P>
  __device__ __forceinline__ void place(P put) const {
    Held<DC * W / 4>::place([&](int e, float4 v) {
      const At<W> at(e);
      put(at.row, at.col, v);
    });
  }
};
// Rows [0, R) x W floats, row stride LD, of the workspace.
template <int R, int W, int LD>
struct Block : Held<R * W / 4> {
  __device__ __forceinline__ void fetch(const float* src) {
    Held<R * W / 4>::fetch([&](int e) {
      const At<W> at(e);
      return *reinterpret_cast<const float4*>(src + at.row * LD + at.col);
    });
  }
  template <class P>
  __device__ __forceinline__ void place(P put) const {
    Held<R * W / 4>::place([&](int e, float4 v) {
      const At<W> at(e);
      put(at.row, at.col, v);
    });
  }
};
template <int R, int W, int LD, class P>
__device__ __forceinline__ void load_block(const float* src, P put) {
  Block<R, W, LD> b;
  b.fetch(src);
  b.place(put);
}
// A fp32 value as two of tf32, 11 bits each: the first rounded, the second cut off by the products, 2^-22 of it left out.
// (In whole numbers: the conversion instruction has a quarter of their rate.  Of a NaN the second is one.)
__device__ __forceinline__ void two(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// acc += sum_k A[row * AS + k] B[col * BS + k] over the warp's MB blocks of 16 rows from `a` on and NT of 8 columns from `b` on,
// each product in three of tf32.  acc[m][n][e]: row 16 m + lane / 4 + 8 (e / 2), column 8 n + 2 (lane % 4) + e % 2.
// A lane reads four of k at once: its elements 4 t .. 4 t + 3 stand for the products' k = t and t + 4, twice.
template <int MB, int NT, int K, int AS, int BS, int UNROLL = 2>
__device__ __forceinline__ void gemm(float (&acc)[MB][NT][4], const float* a, const float* b) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  a += g * AS + 4 * t;
  b += g * BS + 4 * t;
#pragma unroll UNROLL
  for (int k = 0; k < K; k += 16) {
    float4 x[MB][2], y[NT];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      x[m][0] = *reinterpret_cast<const float4*>(a + 16 * m * AS + k);
      x[m][1] = *reinterpret_cast<const float4*>(a + (16 * m + 8) * AS + k);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) y[n] = *reinterpret_cast<const float4*>(b + 8 * n * BS + k);
    float part[MB][NT][4] = {}, small[MB][NT][4] = {};  // (the tensor cores' sums are cut off, not rounded: short ones, added up in fp32)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t ah[MB][4], al[MB][4], bh[NT][2], bl[NT][2];
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          two(half ? x[m][r].z : x[m][r].x, ah[m][r], al[m][r]);
          two(half ? x[m][r].w : x[m][r].y, ah[m][2 + r], al[m][2 + r]);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        two(half ? y[n].z : y[n].x, bh[n][0], bl[n][0]);
        two(half ? y[n].w : y[n].y, bh[n][1], bl[n][1]);
      }
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(small[m][n], al[m], bh[n]);
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(small[m][n], ah[m], bl[n]);
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma(part[m][n], ah[m], bh[n]);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][n][e] += part[m][n][e] + small[m][n][e];
  }
}
// This thread's rows and columns of such a product whose warps stand in rows of `across`, each with 16 MB rows and 8 NT columns.
template <int MB, int NT>
struct Mine {
  int warp_row, warp_col, g, t;
  __device__ __forceinline__ explicit Mine(int across) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    warp_row = warp / across * 16 * MB;
    warp_col = warp % across * 8 * NT;
    g = lane / 4;
    t = lane % 4;
  }
  __device__ __forceinline__ int row(int m, int e) const { return warp_row + 16 * m + g + 8 * (e / 2); }
  __device__ __forceinline__ int col(int n, int e) const { return warp_col + 8 * n + 2 * t + e % 2; }
};

// ---- prep -------------------------------------------------------------------------------------
constexpr int PREP_FLOATS = 2 * DC * KS + 2 * DC * CS;

template <bool BWD>
__global__ void __launch_bounds__(THREADS) delta_prep_simt_kernel(const DeltaArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* const sk = sm;             // [DC][KS]
  float* const sq = sk + DC * KS;
  float* const m = sq + DC * KS;    // [DC][CS]: M and M B
  float* const mb = m + DC * CS;
  __shared__ float2 sg[DC];
  __shared__ float sb[DC];
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) return;
  float* const ws = ws_of<BWD>(a, slot, h);
  if (tid < 32) {
    const float* g = (const float*)a.g + ch.t0 * a.H + h;
    const float* b = (const float*)a.beta + ch.t0 * a.H + h;
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * tid + e;
      x[e] = i < ch.len ? g[(long long)i * a.H] : 0.f;
      sb[i] = i < ch.len ? b[(long long)i * a.H] : 0.f;
    }
    float2 s0, s1;
    delta_sums(x[0], x[1], s0, s1);
    sg[2 * tid] = s0;
    sg[2 * tid + 1] = s1;
  }
  Rows<DK> k, q;
  k.fetch(a.k, ch.t0, ch.len, a.H, h, DK, 0);
  q.fetch(a.q, ch.t0, ch.len, a.H, h, DK, 0);
  k.place([&](int i, int c, float4 v) { put_row(sk + i * KS + c, v); });
  q.place([&](int i, int c, float4 v) { put_row(sq + i * KS + c, v); });
  __syncthreads();
  if (tid < DC) {
    ws[WS_GT + GT_HI + tid] = sg[tid].x;
    ws[WS_GT + GT_LO + tid] = sg[tid].y;
    ws[WS_GT + GT_F + tid] = delta_decay0(sg[tid]);
    ws[WS_GT + GT_E + tid] = delta_decay(sg[DC - 1], sg[tid]);
    ws[WS_GT + GT_B + tid] = sb[tid];
  }
  const Mine<1, 4> my(2);
  float kk[1][4][4] = {}, qk[1][4][4] = {};
  gemm<1, 4, DK, KS, KS, 1>(kk, sk + my.warp_row * KS, sk + my.warp_col * KS);
  gemm<1, 4, DK, KS, KS, 1>(qk, sq + my.warp_row * KS, sk + my.warp_col * KS);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = my.row(0, e), j = my.col(c, e);
      const float d = j <= i ? delta_decay(sg[i], sg[j]) : 0.f;
      ws[WS_P + i * DC + j] = j <= i ? d * qk[0][c][e] : 0.f;
      const float x = j < i ? d * kk[0][c][e] : 0.f;
      m[i * CS + j] = x;
      mb[i * CS + j] = x * sb[j];
    }
  __syncthreads();
  if (tid < DC) {
    // Z = (1 + M B)^-1 M by forward substitution, a thread a column, 16 rows at a time: z_i = M_ic - sum_{j < i} (M B)_ij z_j.
    // (Loops over the blocks: written out, the code takes longer to be fetched than to run: prep 17 us instead of 13.)
    float* const z = sq;  // [DC][DC], Q is done with
#pragma unroll 1
    for (int b = 0; b < DC; b += 16) {
      float y[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) y[r] = m[(b + r) * CS + tid];
#pragma unroll 1
      for (int j = 0; j < b; j += 4) {
        const float z0 = z[j * DC + tid], z1 = z[(j + 1) * DC + tid], z2 = z[(j + 2) * DC + tid], z3 = z[(j + 3) * DC + tid];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(mb + (b + r) * CS + j);
          y[r] = fmaf(-w.w, z3, fmaf(-w.z, z2, fmaf(-w.y, z1, fmaf(-w.x, z0, y[r]))));
        }
      }
#pragma unroll
      for (int r = 1; r < 16; ++r)
#pragma unroll
        for (int j = 0; j < r; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(mb + (b + r) * CS + b + j);
          y[r] = fmaf(-w.x, y[j], y[r]);
          if (j + 1 < r) y[r] = fmaf(-w.y, y[j + 1], y[r]);
          if (j + 2 < r) y[r] = fmaf(-w.z, y[j + 2], y[r]);
          if (j + 3 < r) y[r] = fmaf(-w.w, y[j + 3], y[r]);
        }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        z[(b + r) * DC + tid] = y[r];
        ws[WS_Z + (b + r) * DC + tid] = y[r];
      }
    }
  }
}

// The state's columns (as rows of S) to rows of DV: a warp has four rows x 32 bytes, as a compromise between both sides' orders.
__device__ __forceinline__ void store_state(const float* S, float* to) {
  for (int e = threadIdx.x; e < DK * SB; e += THREADS) {
    const int c = e / 32 % 4 * 8 + e % 8, x = e / 128 * 4 + e % 32 / 8;
    to[x * DV + c] = S[c * KS + x];
  }
}

// ---- forward scan ---------------------------------------------------------------------------
constexpr int SCAN_FLOATS = SB * KS + 2 * DC * KS + DK * CS + 2 * DC * CS + 2 * SB * CS + 3 * DC;

template <bool BWD>
__global__ void __launch_bounds__(THREADS) delta_scan_simt_kernel(const DeltaArgs a) {
  wait_for_previous();
  extern __shared__ __align__(16) float sm[];
  float* const S = sm;                 // [SB][KS]: columns of the state
  float* const sk = S + SB * KS;       // [DC][KS]
  float* const sq = sk + DC * KS;
  float* const st = sq + DC * KS;      // [DK][CS]: K^T
  float* const sz = st + DK * CS;      // [DC][CS]
  float* const sp = sz + DC * CS;
  float* const sr = sp + DC * CS;      // [SB][CS]: columns of B R, then of e^(G_C - G) U
  float* const su = sr + SB * CS;      // [SB][CS]: columns of U
  float* const sf = su + SB * CS;      // e^G, e^(G_C - G), beta
  const int tile = blockIdx.x % SNB, nh = blockIdx.x / SNB, h = nh % a.H, n = delta_unit(a, nh / a.H), tid = threadIdx.x;
  const int c0 = tile * SB;
  const DeltaSeq s = delta_seq(a, n);
  const int from = a.h0 ? delta_row(a.h0_row, a.h0_rows, n, a.err) : -1;
  if (from >= 0)
    load_block<DK, SB, DV>(a.h0 + ((long long)from * a.H + h) * (DK * DV) + c0, [&](int x, int c, float4 v) { put_column<KS>(S + c * KS + x, v); });
  else
    for (int e = tid; e < SB * KS; e += THREADS) S[e] = 0.f;
  const Mine<1, 2> my(2);  // of [64][32]
  const Mine<3, 1> dk(4);  // of [96][32]
  // A chunk's inputs, fetched while the one before is computed.
  Rows<DK> k, q;
  Block<DC, DC, DC> z, p;
  float v[2][4], f = 0.f;
  auto fetch = [&](int c) {
    const int len = min(DC, s.len - c * DC);
    const long long t0 = s.begin + (long long)c * DC;
    const float* const ws = ws_of<BWD>(a, s.slot0 + c, h);
    k.fetch(a.k, t0, len, a.H, h, DK, 0);
    if (!BWD) q.fetch(a.q, t0, len, a.H, h, DK, 0);
    z.fetch(ws + WS_Z);
    if (!BWD) p.fetch(ws + WS_P);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        float2 x = make_float2(0.f, 0.f);
        if (my.row(0, e) < len) x = *reinterpret_cast<const float2*>((const float*)a.v + ((t0 + my.row(0, e)) * a.H + h) * DV + c0 + my.col(n, e));
        v[n][e] = x.x;
        v[n][e + 1] = x.y;
      }
    if (tid < 3 * DC) f = ws[WS_GT + GT_F + tid];
  };
  if (s.len > 0) fetch(0);
  for (int c = 0; c * DC < s.len; ++c) {
    const int len = min(DC, s.len - c * DC);
    const long long t0 = s.begin + (long long)c * DC;
    float* const ws = ws_of<BWD>(a, s.slot0 + c, h);
    __syncthreads();
    if (tid < 3 * DC) sf[tid] = f;
    k.place([&](int i, int x, float4 y) {
      put_row(sk + i * KS + x, y);
      put_column<CS>(st + x * CS + i, y);
    });
    if (!BWD) q.place([&](int i, int x, float4 y) { put_row(sq + i * KS + x, y); });
    z.place([&](int i, int j, float4 y) { put_row(sz + i * CS + j, y); });
    if (!BWD) p.place([&](int i, int j, float4 y) { put_row(sp + i * CS + j, y); });
    float r[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) r[n][e] = v[n][e];
    __syncthreads();
    if ((c + 1) * DC < s.len) fetch(c + 1);
    if (BWD)
      store_state(S, ws + WS_S0 + c0);
    float ks[1][2][4] = {}, qs[1][2][4] = {};
    gemm<1, 2, DK, KS, KS>(ks, sk + my.warp_row * KS, S + my.warp_col * KS);
    if (!BWD) gemm<1, 2, DK, KS, KS>(qs, sq + my.warp_row * KS, S + my.warp_col * KS);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = my.row(0, e);
        r[n][e] = fmaf(-sf[row], ks[0][n][e], r[n][e]);
        sr[my.col(n, e) * CS + row] = sf[2 * DC + row] * r[n][e];
      }
    __syncthreads();
    float zr[1][2][4] = {};
    gemm<1, 2, DC, CS, CS>(zr, sz + my.warp_row * CS, sr + my.warp_col * CS);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = my.row(0, e), col = my.col(n, e);
        const float x = r[n][e] - zr[0][n][e];
        su[col * CS + row] = sf[2 * DC + row] * x;
        if (BWD) ws[WS_X + row * DV + c0 + col] = x;
      }
    __syncthreads();
    if (!BWD) {
      float pu[1][2][4] = {};
      gemm<1, 2, DC, CS, CS>(pu, sp + my.warp_row * CS, su + my.warp_col * CS);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = my.row(0, e);
          if (row < len) ((float*)a.o)[((t0 + row) * a.H + h) * DV + c0 + my.col(n, e)] = a.scale * fmaf(sf[row], qs[0][n][e], pu[0][n][e]);
        }
    }
    // e^(G_C - G) goes to U, which nothing else reads any more
    for (int e = tid; e < SB * DC; e += THREADS) sr[e / DC * CS + e % DC] = sf[DC + e % DC] * su[e / DC * CS + e % DC];
    __syncthreads();
    float ds[3][1][4] = {};
    gemm<3, 1, DC, CS, CS>(ds, st + dk.warp_row * CS, sr + dk.warp_col * CS);
    const float last = sf[DC - 1];
#pragma unroll
    for (int m = 0; m < 3; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float* const at = S + dk.col(0, e) * KS + dk.row(m, e);  // (this thread's own, and nothing reads S here)
        *at = fmaf(last, *at, ds[m][0][e]);
      }
  }
  __syncthreads();
  if (!BWD && a.hT) {
    const int to = delta_row(a.hT_row, a.hT_rows, n, a.err);
    if (to >= 0)
      store_state(S, a.hT + ((long long)to * a.H + h) * (DK * DV) + c0);
  }
}

// ---- reverse scan ---------------------------------------------------------------------------
constexpr int RSCAN_FLOATS = SB * KS + DC * KS + 2 * DK * CS + 2 * DC * CS + 3 * SB * CS + 3 * DC;

__global__ void __launch_bounds__(THREADS) delta_rscan_simt_kernel(const DeltaArgs a, float* dbeta_part) {
  wait_for_previous();
  extern __shared__ __align__(16) float sm[];
  float* const S = sm;              // [SB][KS]: columns of dS
  float* const sk = S + SB * KS;    // [DC][KS]
  float* const skt = sk + DC * KS;  // [DK][CS]: K^T, Q^T
  float* const sqt = skt + DK * CS;
  float* const szt = sqt + DK * CS; // [DC][CS]: Z^T, P^T
  float* const spt = szt + DC * CS;
  float* const sw = spt + DC * CS;  // [SB][CS]: columns of B dU, of -e^G dR
  float* const sn = sw + SB * CS;
  float* const sd = sn + SB * CS;   // [SB][CS]: columns of dO, then weighted with s e^G
  float* const sf = sd + SB * CS;
  const int tile = blockIdx.x % SNB, nh = blockIdx.x / SNB, h = nh % a.H, n = delta_unit(a, nh / a.H), tid = threadIdx.x;
  const int c0 = tile * SB;
  const DeltaSeq s = delta_seq(a, n);
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  if (a.dhT)
    load_block<DK, SB, DV>(a.dhT + ((long long)n * a.H + h) * (DK * DV) + c0, [&](int x, int c, float4 v) { put_column<KS>(S + c * KS + x, v); });
  else
    for (int e = tid; e < SB * KS; e += THREADS) S[e] = 0.f;
  const Mine<1, 2> my(2);  // of [64][32]
  const Mine<3, 1> dk(4);  // of [96][32]
  // A chunk's inputs, fetched while the one before is computed.
  Rows<DK> k, q;
  Rows<SB> d;
  Block<DC, DC, DC> z, p;
  float xs[2][4], f = 0.f;
  auto fetch = [&](int c) {
    const int len = min(DC, s.len - c * DC);
    const long long t0 = s.begin + (long long)c * DC;
    const float* const ws = ws_of<true>(a, s.slot0 + c, h);
    k.fetch(a.k, t0, len, a.H, h, DK, 0);
    q.fetch(a.q, t0, len, a.H, h, DK, 0);
    d.fetch(a.dO, t0, len, a.H, h, DV, c0);
    z.fetch(ws + WS_Z);
    p.fetch(ws + WS_P);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(ws + WS_X + my.row(0, e) * DV + c0 + my.col(n, e));
        xs[n][e] = x.x;
        xs[n][e + 1] = x.y;
      }
    if (tid < 3 * DC) f = ws[WS_GT + GT_F + tid];
  };
  const int nc = (s.len + DC - 1) / DC;
  if (nc > 0) fetch(nc - 1);
  for (int c = nc - 1; c >= 0; --c) {
    const int len = min(DC, s.len - c * DC);
    const long long t0 = s.begin + (long long)c * DC;
    float* const ws = ws_of<true>(a, s.slot0 + c, h);
    __syncthreads();
    if (tid < 3 * DC) sf[tid] = f;
    k.place([&](int i, int e, float4 y) {
      put_row(sk + i * KS + e, y);
      put_column<CS>(skt + e * CS + i, y);
    });
    q.place([&](int i, int e, float4 y) { put_column<CS>(sqt + e * CS + i, y); });
    d.place([&](int i, int e, float4 y) { put_column<CS>(sd + e * CS + i, y); });
    z.place([&](int i, int j, float4 y) { put_column<CS>(szt + j * CS + i, y); });
    p.place([&](int i, int j, float4 y) { put_column<CS>(spt + j * CS + i, y); });
    float x[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] = xs[n][e];
    __syncthreads();
    if (c > 0) fetch(c - 1);
    store_state(S, ws + WS_DS + c0);
    float kd[1][2][4] = {}, pd[1][2][4] = {}, du[2][4];
    gemm<1, 2, DK, KS, KS>(kd, sk + my.warp_row * KS, S + my.warp_col * KS);
    gemm<1, 2, DC, CS, CS>(pd, spt + my.warp_row * CS, sd + my.warp_col * CS);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = my.row(0, e);
        du[n][e] = fmaf(sf[DC + row], kd[0][n][e], a.scale * pd[0][n][e]);
        sw[my.col(n, e) * CS + row] = sf[2 * DC + row] * du[n][e];
      }
    __syncthreads();
    float zw[1][2][4] = {}, part[2] = {};
    gemm<1, 2, DC, CS, CS>(zw, szt + my.warp_row * CS, sw + my.warp_col * CS);
    for (int e = tid; e < SB * DC; e += THREADS) sd[e / DC * CS + e % DC] *= a.scale * sf[e % DC];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = my.row(0, e), col = my.col(n, e);
        const float dut = du[n][e] - zw[0][n][e], dr = sf[2 * DC + row] * dut;
        part[e / 2] = fmaf(dut, x[n][e], part[e / 2]);
        if (row < len) ((float*)a.dv)[((t0 + row) * a.H + h) * DV + c0 + col] = dr;
        sn[col * CS + row] = -sf[row] * dr;
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      part[i] += __shfl_xor_sync(0xffffffffu, part[i], 1);
      part[i] += __shfl_xor_sync(0xffffffffu, part[i], 2);
      const int row = my.row(0, 2 * i);
      if (my.t == 0 && row < len) dbeta_part[((long long)(2 * tile + (my.warp_col > 0)) * tokens + t0 + row) * a.H + h] = part[i];
    }
    __syncthreads();
    float ds[3][1][4] = {};
    gemm<3, 1, DC, CS, CS>(ds, sqt + dk.warp_row * CS, sd + dk.warp_col * CS);
    gemm<3, 1, DC, CS, CS>(ds, skt + dk.warp_row * CS, sn + dk.warp_col * CS);
    const float last = sf[DC - 1];
#pragma unroll
    for (int m = 0; m < 3; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float* const at = S + dk.col(0, e) * KS + dk.row(m, e);
        *at = fmaf(last, *at, ds[m][0][e]);
      }
  }
  __syncthreads();
  if (a.dh0)
    store_state(S, a.dh0 + ((long long)n * a.H + h) * (DK * DV) + c0);
}

// ---- gradients of the chunk ------------------------------------------------------------------
// A cluster of two CTAs a (chunk, head), each with 32 rows of Es and Fm, which both need whole and write to each other,
// and with 48 columns of d_k: short calls have few chunks (one CTA took 1.4 times as long).  Pieces of 32 columns
// of d_v: dO, dR, U [DC][BS], S0, dS1 [HK][BS], the next piece's loads in flight; then Es, Fm and their transposes
// [DC][CS] in their place.  K and Q [DC][HS], K^T and Q^T [HK][CS].
constexpr int HK = DK / 2, HS = HK + 4;
constexpr int PIECES = 3 * DC * BS + 2 * HK * BS, GRAD_FLOATS = 2 * DC * HS + 2 * HK * CS + (PIECES > 4 * DC * CS ? PIECES : 4 * DC * CS) + 4 * DC + 8;

__device__ __forceinline__ uint32_t peer_of(const float* at, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(at)), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void put_peer(uint32_t at, float v) { asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory"); }

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS) delta_grads_simt_kernel(const DeltaArgs a, const float* dbeta_part) {
  wait_for_previous();
  extern __shared__ __align__(16) float sm[];
  float* const sk = sm;
  float* const sq = sk + DC * HS;
  float* const skt = sq + DC * HS;
  float* const sqt = skt + HK * CS;
  float* const sdo = sqt + HK * CS;
  float* const sdr = sdo + DC * BS;
  float* const su = sdr + DC * BS;
  float* const ss = su + DC * BS;
  float* const sd = ss + HK * BS;
  float* const sdg = sm + GRAD_FLOATS - 4 * DC - 8;  // [4][64] dG of two CTAs' columns, by halves; [2] what hangs on G_C
  __shared__ float red[THREADS / 32];
  const int unit = blockIdx.x / 2, rank = blockIdx.x % 2, slot = unit / a.H, h = unit % a.H, tid = threadIdx.x, x0 = rank * HK;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) {  // (both)
    if (rank == 0) zero_spare_rows<float>(a, slot, h);
    return;
  }
  const float* const ws = ws_of<true>(a, slot, h);
  const float* const gt = ws + WS_GT;
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  Rows<HK> k, q;
  Rows<SB> pdo, pdr;
  Block<DC, SB, DV> px;
  Block<HK, SB, DV> ps, pd;
  auto fetch = [&](int c0) {
    pdo.fetch(a.dO, ch.t0, ch.len, a.H, h, DV, c0);
    pdr.fetch(a.dv, ch.t0, ch.len, a.H, h, DV, c0);
    px.fetch(ws + WS_X + c0);
    ps.fetch(ws + WS_S0 + x0 * DV + c0);
    pd.fetch(ws + WS_DS + x0 * DV + c0);
  };
  k.fetch(a.k, ch.t0, ch.len, a.H, h, DK, x0);
  q.fetch(a.q, ch.t0, ch.len, a.H, h, DK, x0);
  fetch(0);
  k.place([&](int i, int c, float4 v) {
    put_row(sk + i * HS + c, v);
    put_column<CS>(skt + c * CS + i, v);
  });
  q.place([&](int i, int c, float4 v) {
    put_row(sq + i * HS + c, v);
    put_column<CS>(sqt + c * CS + i, v);
  });
  const Mine<1, 2> pair(4);  // of [32][64]: rows i0 .. of Es and Fm
  const Mine<1, 3> my(2);    // of [64][48]
  const int i0 = rank * (DC / 2);
  float dp[1][2][4] = {}, dm[1][2][4] = {}, dqi[1][3][4] = {}, dkr[1][3][4] = {}, dks[1][3][4] = {}, frob = 0.f;
  for (int c0 = 0; c0 < DV; c0 += SB) {
    __syncthreads();
    pdo.place([&](int i, int c, float4 v) { put_row(sdo + i * BS + c, v); });
    pdr.place([&](int i, int c, float4 v) { put_row(sdr + i * BS + c, v); });
    px.place([&](int i, int c, float4 v) {
      const float b = gt[GT_B + i];
      put_row(su + i * BS + c, make_float4(b * v.x, b * v.y, b * v.z, b * v.w));
    });
    ps.place([&](int x, int c, float4 v) { put_row(ss + x * BS + c, v); });
    pd.place([&](int x, int c, float4 v) { put_row(sd + x * BS + c, v); });
    __syncthreads();
    if (c0 + SB < DV) fetch(c0 + SB);
    for (int e = tid; e < HK * SB; e += THREADS) frob = fmaf(ss[e / SB * BS + e % SB], sd[e / SB * BS + e % SB], frob);
    gemm<1, 2, SB, BS, BS>(dp, sdo + (i0 + pair.warp_row) * BS, su + pair.warp_col * BS);
    gemm<1, 2, SB, BS, BS>(dm, sdr + (i0 + pair.warp_row) * BS, su + pair.warp_col * BS);
    gemm<1, 3, SB, BS, BS>(dqi, sdo + my.warp_row * BS, ss + my.warp_col * BS);
    gemm<1, 3, SB, BS, BS>(dkr, sdr + my.warp_row * BS, ss + my.warp_col * BS);
    gemm<1, 3, SB, BS, BS>(dks, su + my.warp_row * BS, sd + my.warp_col * BS);
  }
  cluster_sync();  // (neither reads its pieces any more)
  float* const es = sdo;              // [DC][CS] Es, Fm, and their transposes
  float* const fm = es + DC * CS;
  float* const est = fm + DC * CS;
  float* const fmt = est + DC * CS;
  const uint32_t peer = peer_of(es, rank ^ 1);
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int i = i0 + pair.row(0, c), j = pair.col(n, c);
      const float d = j <= i ? delta_decay(make_float2(gt[GT_HI + i], gt[GT_LO + i]), make_float2(gt[GT_HI + j], gt[GT_LO + j])) : 0.f;
      const float e = j <= i ? a.scale * d * dp[0][n][c] : 0.f, f = j < i ? -d * dm[0][n][c] : 0.f;
      const int at = i * CS + j, att = 2 * DC * CS + j * CS + i;
      es[at] = es[att] = e;
      fm[at] = fm[att] = f;
      put_peer(peer + 4 * at, e);
      put_peer(peer + 4 * att, e);
      put_peer(peer + 4 * (DC * CS + at), f);
      put_peer(peer + 4 * (DC * CS + att), f);
    }
  cluster_sync();
  float q1[1][3][4] = {}, k1[1][3][4] = {}, k2[1][3][4] = {};  // Es K;  Es^T Q + Fm^T K;  Fm K
  gemm<1, 3, DC, CS, CS>(q1, es + my.warp_row * CS, skt + my.warp_col * CS);
  gemm<1, 3, DC, CS, CS>(k1, est + my.warp_row * CS, sqt + my.warp_col * CS);
  gemm<1, 3, DC, CS, CS>(k1, fmt + my.warp_row * CS, skt + my.warp_col * CS);
  gemm<1, 3, DC, CS, CS>(k2, fm + my.warp_row * CS, skt + my.warp_col * CS);
  const uint32_t first = peer_of(sdg, 0);
  float at_end = 0.f;  // sum_j k_j . (e^(G_C - G_j) dS1 u_j), this thread's part
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = my.row(0, 2 * r);
    const float f = gt[GT_F + i], e = gt[GT_E + i];
    float dg = 0.f;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      float dq[2], dk[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = 2 * r + x, col = my.col(n, c);
        const float q = sq[i * HS + col], k = sk[i * HS + col];
        dq[x] = fmaf(a.scale * f, dqi[0][n][c], q1[0][n][c]);
        const float minus = fmaf(e, dks[0][n][c], k1[0][n][c]), plus = fmaf(-f, dkr[0][n][c], k2[0][n][c]);
        dk[x] = minus + plus;
        at_end = fmaf(k, e * dks[0][n][c], at_end);
        dg = fmaf(q, dq[x], fmaf(k, plus - minus, dg));
      }
      if (i < ch.len) {
        const long long at = ((ch.t0 + i) * a.H + h) * DK + x0 + my.col(n, 0);
        *reinterpret_cast<float2*>((float*)a.dq + at) = make_float2(dq[0], dq[1]);
        *reinterpret_cast<float2*>((float*)a.dk + at) = make_float2(dk[0], dk[1]);
      }
    }
    dg += __shfl_xor_sync(0xffffffffu, dg, 1);
    dg += __shfl_xor_sync(0xffffffffu, dg, 2);
    if (my.t == 0) put_peer(first + 4 * ((2 * rank + (my.warp_col > 0)) * DC + i), dg);
  }
  at_end = fmaf(gt[GT_F + DC - 1], frob, at_end);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) at_end += __shfl_xor_sync(0xffffffffu, at_end, off);
  if ((tid & 31) == 0) red[tid / 32] = at_end;
  __syncthreads();
  if (tid == 0) {
    float end = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) end += red[w];
    put_peer(first + 4 * (4 * DC + rank), end);
  }
  cluster_sync();  // (after it the second CTA touches only its own memory)
  if (rank == 0 && tid < 32) {  // dg_t = the sum of dG_i over i >= t, and of what hangs on G_C
    const float end = sdg[4 * DC] + sdg[4 * DC + 1];
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      lo += sdg[x * DC + 2 * tid];
      hi += sdg[x * DC + 2 * tid + 1];
    }
    float run = lo + hi;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float up = __shfl_down_sync(0xffffffffu, run, off);
      if (tid + off < 32) run += up;
    }
    const float behind = run - (lo + hi);
    float* const dst = (float*)a.dg + ch.t0 * a.H + h;
    if (2 * tid < ch.len) dst[(long long)(2 * tid) * a.H] = run + end;
    if (2 * tid + 1 < ch.len) dst[(long long)(2 * tid + 1) * a.H] = behind + hi + end;
  } else if (rank == 1 && tid < ch.len) {
    const long long t = ch.t0 + tid;
    float b = 0.f;
#pragma unroll
    for (int x = 0; x < 2 * SNB; ++x) b += dbeta_part[((long long)x * tokens + t) * a.H + h];
    ((float*)a.dbeta)[t * a.H + h] = b;
  }
  if (rank == 0) zero_spare_rows<float>(a, slot, h);
}

constexpr int PREP_BYTES = PREP_FLOATS * 4, SCAN_BYTES = SCAN_FLOATS * 4, RSCAN_BYTES = RSCAN_FLOATS * 4, GRAD_BYTES = GRAD_FLOATS * 4;
static_assert(SCAN_BYTES <= 232448 && RSCAN_BYTES <= 232448 && GRAD_BYTES <= 232000, "shared memory");

template <class F>
cudaError_t allow(F* f, int bytes) {
  return cudaFuncSetAttribute((const void*)f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
cudaError_t allow_all() {
  static OncePerDevice<CudaDeviceApi> once;
  return once([] {
    for (cudaError_t e : {allow(delta_prep_simt_kernel<false>, PREP_BYTES), allow(delta_prep_simt_kernel<true>, PREP_BYTES),
                          allow(delta_scan_simt_kernel<false>, SCAN_BYTES), allow(delta_scan_simt_kernel<true>, SCAN_BYTES),
                          allow(delta_rscan_simt_kernel, RSCAN_BYTES), allow(delta_grads_simt_kernel, GRAD_BYTES)})
      if (e != cudaSuccess) return e;
    return cudaSuccess;
  });
}

}  // namespace

size_t delta_simt_ws_bytes(long long slots, long long tokens, int H, bool bwd) {
  return (size_t)slots * H * (bwd ? WS_BWD : WS_FWD) * 4 + (bwd ? (size_t)2 * SNB * tokens * H * 4 : 0);
}

cudaError_t launch_delta_simt_fwd(const DeltaArgs& a, cudaStream_t st) {
  const cudaError_t e = allow_all();
  if (e != cudaSuccess) return e;
  if (a.slots > 0) delta_prep_simt_kernel<false><<<(unsigned)a.slots * a.H, THREADS, PREP_BYTES, st>>>(a);
  const cudaError_t scan = launch_behind(delta_scan_simt_kernel<false>, (unsigned)a.n_seq * a.H * SNB, THREADS, SCAN_BYTES, st, a);
  return scan != cudaSuccess ? scan : cudaGetLastError();
}
cudaError_t launch_delta_simt_bwd(const DeltaArgs& a, cudaStream_t st) {
  const cudaError_t e = allow_all();
  if (e != cudaSuccess) return e;
  float* part = reinterpret_cast<float*>(a.ws) + (long long)a.slots * a.H * WS_BWD;
  const unsigned chunks = (unsigned)a.slots * a.H, units = (unsigned)a.n_seq * a.H * SNB;
  if (a.slots > 0) {
    delta_prep_simt_kernel<true><<<chunks, THREADS, PREP_BYTES, st>>>(a);
    const cudaError_t scan = launch_behind(delta_scan_simt_kernel<true>, units, THREADS, SCAN_BYTES, st, a);
    if (scan != cudaSuccess) return scan;
  }
  cudaError_t last = launch_behind(delta_rscan_simt_kernel, units, THREADS, RSCAN_BYTES, st, a, part);
  if (a.slots > 0 && last == cudaSuccess) last = launch_behind(delta_grads_simt_kernel, 2 * chunks, THREADS, GRAD_BYTES, st, a, part);
  return last != cudaSuccess ? last : cudaGetLastError();
}

}  // namespace gla
