// The gated delta rule on the 5th-generation tensor cores (bf16 calls).  Formulas: gla_delta.cuh.
//
//   prep    one CTA a (chunk, head): KK^T and QK^T on the tensor cores, the decays, and the triangular system, solved
//           once for everything that it multiplies: rows y with y (1 + B M) = r by back substitution, one thread a
//           row, in fp32.  With r the rows of P and of (diag(e^(G_C - G)) K)^T it gives P^ and K^, and the chunk is
//               O = s (diag(e^G) Q S0 + P^ B R),   S1 = e^(G_C) S0 + K^ B R,   R = V - diag(e^G) K S0:
//           U is never formed, and two dependent products are left between a state and the next instead of three.
//   scan    one CTA a (sequence, head, 64 columns of d_v), chunks in order: [K; Q] S0 (one M = 128 product), then
//           K^ B R and P^ B R.  Tiles of d_v are independent.
// What carries the state is held in two bf16 (hi + lo: 16 bits): S, B R and K^; [hi | lo] stand beside each other
// as N = 128 columns of one product.  P^ and the outputs are one bf16.
#include "gla_delta.cuh"
#include "gla_once.cuh"
#include "gla_tc.cuh"

namespace gla {
namespace {

// ---- shared pieces --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 widen2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// (x, y) as two bf16 pairs, hi + lo
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = bf2(x, y);
  const float2 h = widen2(hi);
  lo = bf2(x - h.x, y - h.y);
}
__device__ __forceinline__ float2 fmadd2(float2 a, float2 b, float2 c) {
  uint64_t r, x, y, z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// 16 columns at each of two tensor-memory addresses of this thread's lane.
__device__ __forceinline__ void tm_ld16x2(uint32_t ta, uint32_t tb, uint32_t (&r)[32]) {
#define R4(b) "=r"(r[b]), "=r"(r[b + 1]), "=r"(r[b + 2]), "=r"(r[b + 3])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : R4(0), R4(4), R4(8), R4(12), R4(16), R4(20), R4(24), R4(28)
      : "r"(ta), "r"(tb)
      : "memory");
#undef R4
}
template <int COLS>
__device__ __forceinline__ void tm_alloc(uint32_t* slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(COLS));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS>
__device__ __forceinline__ void tm_free(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(COLS));
}
// Place of 16-byte piece c of row r in a tile of 128-byte rows (swizzle over 8 rows), of 64-byte rows (over 4 pairs).
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
__device__ __forceinline__ uint32_t sw64(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

constexpr unsigned long long DRAIN_NS = 1000000000ull;

// ---- workspace of a (chunk place, head), in bytes --------------------------------------------
// K^ hi and lo: 96 rows (d_k) x 64 tokens; P^: 64 rows x 64 tokens; as the swizzled tiles that the scan copies.
constexpr uint32_t W_KD = 0, W_PH = 24576, W_OP = 32768;  // (one copy of W_OP bytes)
constexpr uint32_t W_GT = 32768;                          // e^G, beta: fp32 [64] each
constexpr uint32_t W_FWD = W_GT + 512;

// ---- prep -------------------------------------------------------------------------------------
// 160 threads: warps 0-3 take the products' 128 rows (K's, then Q's) out of tensor memory; warps 2 and 3 then solve
// for the rows of P^, warps 0, 1 and 4 for those of K^.
constexpr int MSTR = DC + 4;
struct PrepSmem {
  static constexpr uint32_t P0 = 0, P1 = 16384, M = 24576, G = M + DC * MSTR * 4, B = G + DC * 8, BAR = B + DC * 4, BYTES = BAR + 32;
};

// Rows y of y (1 + BM) = r, last element first: y_m is final once the later ones are; each takes its multiple of row
// m of BM off the elements before it.
__device__ __forceinline__ void solve_row(const float* bm, float2 (&r)[DC / 2]) {
#pragma unroll
  for (int m = DC - 1; m > 0; --m) {
    const float y = -((m & 1) ? r[m / 2].y : r[m / 2].x);
    const float2 yy = make_float2(y, y);
#pragma unroll
    for (int j = 0; j < m; j += 4) {  // (BM is zero from the diagonal on)
      const float4 w = *reinterpret_cast<const float4*>(bm + m * MSTR + j);
      r[j / 2] = fmadd2(yy, make_float2(w.x, w.y), r[j / 2]);
      if (j + 2 < m) r[j / 2 + 1] = fmadd2(yy, make_float2(w.z, w.w), r[j / 2 + 1]);
    }
  }
}

__global__ void __launch_bounds__(160, 3) delta_prep_kernel(const DeltaArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  float* const bm = reinterpret_cast<float*>(sm + PrepSmem::M);
  float2* const sg = reinterpret_cast<float2*>(sm + PrepSmem::G);  // sums of log2 decays
  float* const sbeta = reinterpret_cast<float*>(sm + PrepSmem::B);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + PrepSmem::BAR);
  uint32_t* const slot_tm = reinterpret_cast<uint32_t*>(sm + PrepSmem::BAR + 8);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + PrepSmem::BAR + 12);
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x, warp = tid >> 5;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) return;
  uint8_t* const ws = a.ws + ((long long)slot * a.H + h) * W_FWD;
  for (int e = tid; e < 128 * 12; e += 160) {
    const int r = e / 12, c = e % 12, t = r & 63;
    const __nv_bfloat16* src = (const __nv_bfloat16*)(r < 64 ? a.k : a.q) + ((ch.t0 + (t < ch.len ? t : 0)) * a.H + h) * DK + 8 * c;
    cp16(sb + (c < 8 ? PrepSmem::P0 + sw128(r, c) : PrepSmem::P1 + sw64(r, c - 8)), src, t < ch.len);
  }
  cp_commit();
  if (warp == 4) tm_alloc<64>(slot_tm);
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    const __nv_bfloat16* g = (const __nv_bfloat16*)a.g + ch.t0 * a.H + h;
    const __nv_bfloat16* b = (const __nv_bfloat16*)a.beta + ch.t0 * a.H + h;
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * (tid & 31) + e;
      x[e] = i < ch.len ? to_f(g[(long long)i * a.H]) : 0.f;
      sbeta[i] = i < ch.len ? to_f(b[(long long)i * a.H]) : 0.f;
    }
    float2 s0, s1;
    delta_sums<true>(x[0], x[1], s0, s1);
    sg[2 * (tid & 31)] = s0;
    sg[2 * (tid & 31) + 1] = s1;
  }
  cp_wait_all();
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot_tm;
  if (tid == 0) {
    const SDesc d0 = sdesc(sb + PrepSmem::P0, 16, 1024, LAYOUT_SW128), d1 = sdesc(sb + PrepSmem::P1, 16, 512, LAYOUT_SW64);
#pragma unroll
    for (int kk = 0; kk < 6; ++kk) {
      const SDesc d = kk < 4 ? d0 + kk * 32u : d1 + (kk - 4) * 32u;
      umma(tmem, d, d, idesc_bf16(128, 64, 0, 0), kk > 0);
    }
    umma_commit(bar);
  }
  float2 r[DC / 2];
  const int i = tid & 63;
  bool ok = true;
  if (warp < 4) {
    ok = mbar_wait(bar, 0, a.wait_ns, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      tc_fence_after();
      const bool is_k = warp < 2;
      const float2 gi = sg[i];
      const float bi = sbeta[i];
      const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t d[32];
        tmem_ld32(lane_addr + half * 32u, d);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = half * 32 + j + e;
            const float2 gj = sg[col];
            const float w = exp2_fast((gi.x - gj.x) + (gi.y - gj.y)) * __uint_as_float(d[j + e]);
            x[e] = (is_k ? col < i : col <= i) ? w : 0.f;
          }
          r[(half * 32 + j) / 2] = make_float2(x[0], x[1]);
          r[(half * 32 + j) / 2 + 1] = make_float2(x[2], x[3]);
          if (is_k)
            *reinterpret_cast<float4*>(bm + i * MSTR + half * 32 + j) = make_float4(bi * x[0], bi * x[1], bi * x[2], bi * x[3]);
        }
      }
    }
  }
  tc_fence_before();
  const bool gone = __syncthreads_or(!ok);
  if (warp == 4) {
    if (gone) mbar_wait_drain(bar, 0, DRAIN_NS, a.err);
    __syncwarp();
    tc_fence_after();
    tm_free<64>(tmem);
  }
  if (gone) {
    if (tid == 0) raise_error(a.err, ERR_TIMEOUT);
    return;
  }
  if (tid < 64) {
    float* const gt = reinterpret_cast<float*>(ws + W_GT);
    gt[tid] = exp2_fast(sg[tid].x + sg[tid].y);
    gt[DC + tid] = sbeta[tid];
  }
  const bool is_p = warp == 2 || warp == 3;
  const int row = is_p ? i : warp == 4 ? 64 + (tid & 31) : tid;  // row of P^, or of K^ (d_k)
  if (!is_p) {
    const float2 last = sg[DC - 1];
#pragma unroll
    for (int j = 0; j < DC; j += 2) {
      float x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = row < 64 ? PrepSmem::P0 + sw128(j + e, row >> 3) + (row & 7) * 2
                                     : PrepSmem::P1 + sw64(j + e, (row - 64) >> 3) + (row & 7) * 2;
        const float2 gj = sg[j + e];
        x[e] = exp2_fast((last.x - gj.x) + (last.y - gj.y)) * __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + at));
      }
      r[j / 2] = make_float2(x[0], x[1]);
    }
  }
  solve_row(bm, r);
  uint8_t* const out = ws + (is_p ? W_PH : W_KD) + row * 128;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(r[4 * c + e].x, r[4 * c + e].y, hi[e], lo[e]);
    const uint32_t at = (uint32_t)((c ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(out + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (!is_p) *reinterpret_cast<uint4*>(out + 12288 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ---- scan -----------------------------------------------------------------------------------
// 256 threads: warp w has lanes 32 (w % 4) .. of the products' rows and columns 32 (w / 4) .. of the tile's 64.
// Rows of [K; Q] S: 0-63 K's, 64-127 Q's; rows of K^ B R: 0-95 the state's; rows of P^ B R: 64-127.  A thread keeps
// its 32 columns of a state row in fp32 registers.  Tensor memory (256 columns, 2 CTAs an SM): [K; Q] S and then
// P^ B R in 0-127, K^ B R in 128-255, each as [hi | lo].
constexpr int TN = 64, NTILE = DV / TN, SCAN_THREADS = 256;
struct ScanSmem {
  static constexpr uint32_t KQ0 = 0, KQ1 = 16384, OP = 24576, S = OP + W_OP, BR = S + 24576, BAR = BR + 16384, BYTES = BAR + 64;
};
enum { SB_A = 0, SB_C, SB_O, SB_OP, SB_DRAIN, SB_N };

__global__ void __launch_bounds__(SCAN_THREADS, 2) delta_scan_kernel(const DeltaArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + ScanSmem::BAR);
  uint32_t* const slot_tm = reinterpret_cast<uint32_t*>(sm + ScanSmem::BAR + 8 * SB_N);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + ScanSmem::BAR + 8 * SB_N + 4);
  const int tile = blockIdx.x % NTILE, nh = blockIdx.x / NTILE, h = nh % a.H, n = nh / a.H;
  const int tid = threadIdx.x, warp = tid >> 5, q = warp & 3, half = warp >> 2;
  const int row = (tid & 31) + 32 * q;  // lane of the products
  const int tok = row & 63;
  const int col0 = tile * TN + 32 * half;
  const bool k_row = q < 2, s_row = q < 3;
  const DeltaSeq s = delta_seq(a, n);
  const int nc = (s.len + DC - 1) / DC;
  const int from = a.h0 ? delta_row(a.h0_row, a.h0_rows, n, a.err) : -1;

  auto load_kq = [&](int c) {
    const int len = min(DC, s.len - c * DC);
    const long long t0 = s.begin + (long long)c * DC;
#pragma unroll
    for (int x = 0; x < 6; ++x) {
      const int e = tid + SCAN_THREADS * x, r = e / 12, p = e % 12, t = r & 63;
      const __nv_bfloat16* src = (const __nv_bfloat16*)(r < 64 ? a.k : a.q) + ((t0 + (t < len ? t : 0)) * a.H + h) * DK + 8 * p;
      cp16(sb + (p < 8 ? ScanSmem::KQ0 + sw128(r, p) : ScanSmem::KQ1 + sw64(r, p - 8)), src, t < len);
    }
    cp_commit();
  };
  auto ws_of = [&](int c) { return a.ws + ((long long)(s.slot0 + c) * a.H + h) * W_FWD; };
  int ops = 0;
  auto load_op = [&](int c) {  // one thread
    ++ops;
    mbar_expect_tx(&bar[SB_OP], W_OP);
    bulk_load(sb + ScanSmem::OP, ws_of(c), W_OP, &bar[SB_OP]);
  };
  uint4 vv[4];
  float f_row = 0.f, b_row = 0.f, f_last = 0.f;
  auto load_rows = [&](int c) {  // this thread's value and decays
    const int len = min(DC, s.len - c * DC);
    const float* gt = reinterpret_cast<const float*>(ws_of(c) + W_GT);
    f_row = gt[tok];
    b_row = gt[DC + tok];
    f_last = gt[DC - 1];
    if (k_row) {
      const uint4* src = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.v + ((s.begin + (long long)c * DC + tok) * a.H + h) * DV + col0);
#pragma unroll
      for (int x = 0; x < 4; ++x) vv[x] = tok < len ? src[x] : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  float S[32];
#pragma unroll
  for (int x = 0; x < 32; ++x) S[x] = 0.f;
  if (s_row && from >= 0) {
    const float4* src = reinterpret_cast<const float4*>(a.h0 + (((long long)from * a.H + h) * DK + row) * DV + col0);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 w = src[x];
      S[4 * x] = w.x;
      S[4 * x + 1] = w.y;
      S[4 * x + 2] = w.z;
      S[4 * x + 3] = w.w;
    }
  }
  auto put_state = [&] {  // hi and lo of the state row, the next product's operand
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(S[8 * c + 2 * e], S[8 * c + 2 * e + 1], hi[e], lo[e]);
      const uint32_t at = sb + ScanSmem::S + sw128(row, 4 * half + c);
      st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(at + 12288, lo[0], lo[1], lo[2], lo[3]);
    }
  };
  if (nc > 0) {
    if (warp == 0) tm_alloc<256>(slot_tm);
    if (tid == 0) {
      for (int x = 0; x < SB_N; ++x) mbar_init(&bar[x], 1);
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      fence_async_smem();
      load_op(0);
    }
    load_kq(0);
    load_rows(0);
    if (s_row) put_state();
    cp_wait_all();
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot_tm;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + 32u * half;
    bool ok = true;
    int c = 0;
    for (; c < nc; ++c) {
      const uint32_t ph = c & 1;
      if (tid == 0) {
        const SDesc d0 = sdesc(sb + ScanSmem::KQ0, 16, 1024, LAYOUT_SW128), d1 = sdesc(sb + ScanSmem::KQ1, 16, 512, LAYOUT_SW64);
        const SDesc ds = sdesc(sb + ScanSmem::S, 12288, 1024, LAYOUT_SW128);
#pragma unroll
        for (int kk = 0; kk < 6; ++kk)
          umma(tmem, kk < 4 ? d0 + kk * 32u : d1 + (kk - 4) * 32u, ds + kk * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
        umma_commit(&bar[SB_A]);
      }
      __syncwarp();
      ok = mbar_wait(&bar[SB_A], ph, a.wait_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      float qs[32];
      if (ok) {
        tc_fence_after();
        if (c + 1 < nc) load_kq(c + 1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t d[32];
          tm_ld16x2(lane_addr + 16 * x, lane_addr + 64 + 16 * x, d);
          if (k_row) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint4 v4 = vv[2 * x + e / 4];
              const float2 v = widen2(e % 4 == 0 ? v4.x : e % 4 == 1 ? v4.y : e % 4 == 2 ? v4.z : v4.w);
              const float r0 = fmaf(-f_row, __uint_as_float(d[2 * e]) + __uint_as_float(d[16 + 2 * e]), v.x);
              const float r1 = fmaf(-f_row, __uint_as_float(d[2 * e + 1]) + __uint_as_float(d[17 + 2 * e]), v.y);
              split2(b_row * r0, b_row * r1, hi[e], lo[e]);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t at = sb + ScanSmem::BR + sw128(tok, 4 * half + 2 * x + p);
              st_shared_v4(at, hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
              st_shared_v4(at + 8192, lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) qs[16 * x + e] = f_row * (__uint_as_float(d[e]) + __uint_as_float(d[16 + e]));
          }
        }
      }
      const float last = f_last;
      if (c + 1 < nc) load_rows(c + 1);
      fence_async_smem();
      tc_fence_before();
      if (__syncthreads_or(!ok)) break;
      if (tid == 0) {
        if (mbar_wait(&bar[SB_OP], ph, a.wait_ns, abort_flag)) {
          tc_fence_after();
          const SDesc dk = sdesc(sb + ScanSmem::OP + W_KD, 16, 1024, LAYOUT_SW128);
          const SDesc dp = sdesc(sb + ScanSmem::OP + W_PH - 8192, 16, 1024, LAYOUT_SW128);  // P^ in rows 64-127
          const SDesc db = sdesc(sb + ScanSmem::BR, 8192, 1024, LAYOUT_SW128);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma(tmem + 128, dk + (kk >> 2) * 12288u + (kk & 3) * 32u, db + (kk & 3) * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
          umma_commit(&bar[SB_C]);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma(tmem, dp + kk * 32u, db + kk * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
          umma_commit(&bar[SB_O]);
        }
      }
      __syncwarp();
      ok = mbar_wait(&bar[SB_C], ph, a.wait_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && s_row) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t d[32];
          tm_ld16x2(lane_addr + 128 + 16 * x, lane_addr + 192 + 16 * x, d);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            S[16 * x + e] = fmaf(last, S[16 * x + e], __uint_as_float(d[e]) + __uint_as_float(d[16 + e]));
        }
        if (c + 1 < nc) put_state();
      }
      ok = ok && mbar_wait(&bar[SB_O], ph, a.wait_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        if (tid == 0 && c + 1 < nc) load_op(c + 1);
        tc_fence_after();
        if (!k_row) {
          const long long t = s.begin + (long long)c * DC + tok;
          uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + (t * a.H + h) * DV + col0);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t d[32], w[8];
            tm_ld16x2(lane_addr + 16 * x, lane_addr + 64 + 16 * x, d);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[e] = bf2(a.scale * (qs[16 * x + 2 * e] + (__uint_as_float(d[2 * e]) + __uint_as_float(d[16 + 2 * e]))),
                         a.scale * (qs[16 * x + 2 * e + 1] + (__uint_as_float(d[2 * e + 1]) + __uint_as_float(d[17 + 2 * e]))));
            if (tok < s.len - c * DC) {
              dst[2 * x] = make_uint4(w[0], w[1], w[2], w[3]);
              dst[2 * x + 1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      cp_wait_all();
      fence_async_smem();
      tc_fence_before();
      if (__syncthreads_or(!ok)) break;
      tc_fence_after();
    }
    cp_wait_all();
    const bool gone = c < nc;
    if (gone && tid == 0) {
      raise_error(a.err, ERR_TIMEOUT);
      // what this thread has issued ends before its memory is given up: its MMAs and its last copy (the ones before
      // have been waited for)
      umma_commit(&bar[SB_DRAIN]);
      mbar_wait_drain(&bar[SB_DRAIN], 0, DRAIN_NS, a.err);
      mbar_wait_drain(&bar[SB_OP], (ops - 1) & 1, DRAIN_NS, a.err);
    }
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
      tm_free<256>(tmem);
    }
    if (gone) return;
  }
  if (a.hT && s_row) {
    const int to = delta_row(a.hT_row, a.hT_rows, n, a.err);
    if (to >= 0) {
      float4* dst = reinterpret_cast<float4*>(a.hT + (((long long)to * a.H + h) * DK + row) * DV + col0);
#pragma unroll
      for (int x = 0; x < 8; ++x) dst[x] = make_float4(S[4 * x], S[4 * x + 1], S[4 * x + 2], S[4 * x + 3]);
    }
  }
}

}  // namespace

size_t delta_tc_ws_bytes(long long slots, int H) { return (size_t)slots * H * W_FWD; }

cudaError_t launch_delta_tc_fwd(const DeltaArgs& a, cudaStream_t st) {
  static OncePerDevice<CudaDeviceApi> once;
  cudaError_t e = once([] {
    const cudaError_t x = cudaFuncSetAttribute(delta_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepSmem::BYTES);
    return x != cudaSuccess ? x : cudaFuncSetAttribute(delta_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ScanSmem::BYTES);
  });
  if (e != cudaSuccess) return e;
  if (a.slots > 0) delta_prep_kernel<<<(unsigned)a.slots * a.H, 160, PrepSmem::BYTES, st>>>(a);
  delta_scan_kernel<<<(unsigned)a.n_seq * a.H * NTILE, SCAN_THREADS, ScanSmem::BYTES, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gla
