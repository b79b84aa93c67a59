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
#include <cuda.h>
#include <string.h>

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
__device__ __forceinline__ float2 fsub2(float2 a, float2 b) { return fmadd2(make_float2(-1.f, -1.f), b, a); }
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  uint64_t r, x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t r, x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// columns 2 e and 2 e + 1 of a product that stands as [hi | lo], the halves added
__device__ __forceinline__ float2 halves(const uint32_t (&d)[32], int e) {
  return fadd2(make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])),
               make_float2(__uint_as_float(d[16 + 2 * e]), __uint_as_float(d[17 + 2 * e])));
}
// A pair as two bf16 pairs, hi + lo.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = bf2(x.x, x.y);
  const float2 r = fsub2(x, widen2(hi));
  lo = bf2(r.x, r.y);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A box of a [tokens, H, d] tensor into shared memory, and back.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int h, int t) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(h), "r"(t), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void box_prefetch(const CUtensorMap* map, int x, int h, int t) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"((uint64_t)map), "r"(x), "r"(h), "r"(t)
               : "memory");
}
__device__ __forceinline__ void box_store(const CUtensorMap* map, uint32_t src, int x, int h, int t) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"((uint64_t)map), "r"(x),
               "r"(h), "r"(t), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
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

// Tensor maps of a call.  K and Q: a chunk's 64 rows in two boxes, columns 0-63 (128-byte rows) and 64-95 (64-byte
// rows).  V: 64 rows x 64 columns.  O: 32 rows x 32 columns, one a warp.
struct DeltaMaps {
  CUtensorMap k0, k1, q0, q1, v, o;
};
__device__ __forceinline__ void load_kq(const DeltaMaps& m, uint32_t p0, uint32_t p1, uint64_t* bar, int h, int t) {
  mbar_expect_tx(bar, 24576);
  box_load(p0, &m.k0, bar, 0, h, t);
  box_load(p0 + 8192, &m.q0, bar, 0, h, t);
  box_load(p1, &m.k1, bar, 64, h, t);
  box_load(p1 + 4096, &m.q1, bar, 64, h, t);
}

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

__global__ void __launch_bounds__(160, 3) delta_prep_kernel(const __grid_constant__ DeltaMaps maps, const DeltaArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  float* const bm = reinterpret_cast<float*>(sm + PrepSmem::M);
  float2* const sg = reinterpret_cast<float2*>(sm + PrepSmem::G);  // sums of log2 decays
  float* const sbeta = reinterpret_cast<float*>(sm + PrepSmem::B);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + PrepSmem::BAR);
  uint32_t* const slot_tm = reinterpret_cast<uint32_t*>(sm + PrepSmem::BAR + 16);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + PrepSmem::BAR + 20);
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x, warp = tid >> 5;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) return;
  uint8_t* const ws = a.ws + ((long long)slot * a.H + h) * W_FWD;
  if (warp == 4) tm_alloc<64>(slot_tm);
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 1, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    load_kq(maps, sb + PrepSmem::P0, sb + PrepSmem::P1, bar + 1, h, (int)ch.t0);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot_tm;
  // (all threads: each reads K's columns later)
  bool ok = mbar_wait(bar + 1, 0, a.wait_ns, abort_flag);
  if (tid == 0 && ok) {
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
  __syncwarp();
  if (warp < 4) {
    ok = ok && mbar_wait(bar, 0, a.wait_ns, abort_flag);
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
            x[e] = (is_k ? col < i : col <= i) && i < ch.len ? w : 0.f;
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
    if (gone) {  // (nothing is left in flight: the copy, and the product, if it was issued)
      mbar_wait_drain(bar + 1, 0, DRAIN_NS, a.err);
      mbar_wait_drain(bar, 0, DRAIN_NS, a.err);
    }
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
        const float k = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(sm + at));
        x[e] = j + e < ch.len ? exp2_fast((last.x - gj.x) + (last.y - gj.y)) * k : 0.f;
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
    for (int e = 0; e < 4; ++e) split2(r[4 * c + e], hi[e], lo[e]);
    const uint32_t at = (uint32_t)((c ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(out + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (!is_p) *reinterpret_cast<uint4*>(out + 12288 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ---- scan -----------------------------------------------------------------------------------
// 256 threads: warp w has lanes 32 (w % 4) .. of the products' rows and columns 32 (w / 4) .. of the tile's 64.
// Rows of [K; Q] S: 0-63 K's (warps of w % 4 < 2), 64-127 Q's; rows of K^ B R: 0-95 the state's; rows of P^ B R:
// 64-127.  A thread keeps its 32 columns of a state row in fp32 registers.  Tensor memory: two places of 128
// columns ([hi | lo]), 2 CTAs an SM.  A chunk's [K; Q] S and, once that is in registers, its P^ B R have the one, its
// K^ B R the other; the next chunk has them the other way round, so that only the state's way (product, residual,
// product, state) is waited for and the outputs are written while the next chunk's first product runs.
// Warps 3 and 7, which have no state rows, have the issuing threads: of the copies and of the products.
constexpr int TN = 64, NTILE = DV / TN, SCAN_THREADS = 256, ISSUER = 224, LOADER = 96;
struct ScanSmem {
  static constexpr uint32_t KQ0 = 0, KQ1 = 16384, OP = 24576, S = OP + W_OP, BR = S + 24576, V = BR + 16384, OUT = V + 8192,
                            GT = OUT + 8192, BAR = GT + 512, BYTES = BAR + 96;
  static_assert(BYTES <= 115712, "two CTAs an SM");
};
enum { SB_A = 0, SB_C, SB_O, SB_KQ, SB_V, SB_KD, SB_PH, SB_DRAIN, SB_N };

__global__ void __launch_bounds__(SCAN_THREADS, 2) delta_scan_kernel(const __grid_constant__ DeltaMaps maps, const DeltaArgs a) {
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
  const bool k_row = q < 2, s_row = q < 3, issuer = tid == ISSUER, loader = tid == LOADER;
  const DeltaSeq s = delta_seq(a, n);
  const int nc = (s.len + DC - 1) / DC;
  const int from = a.h0 ? delta_row(a.h0_row, a.h0_rows, n, a.err) : -1;

  auto ws_of = [&](int c) { return a.ws + ((long long)(s.slot0 + c) * a.H + h) * W_FWD; };
  // (the loader) a chunk's operands, each as soon as the chunk before is done with their place
  int loads[4] = {};
  auto load_rows = [&](int c) {
    ++loads[0];
    load_kq(maps, sb + ScanSmem::KQ0, sb + ScanSmem::KQ1, &bar[SB_KQ], h, (int)(s.begin + (long long)c * DC));
  };
  auto load_v = [&](int c) {
    ++loads[1];
    mbar_expect_tx(&bar[SB_V], 8192 + 512);
    box_load(sb + ScanSmem::V, &maps.v, &bar[SB_V], tile * TN, h, (int)(s.begin + (long long)c * DC));
    bulk_load(sb + ScanSmem::GT, ws_of(c) + W_GT, 512, &bar[SB_V]);
  };
  auto load_kd = [&](int c) {
    ++loads[2];
    mbar_expect_tx(&bar[SB_KD], W_PH);
    bulk_load(sb + ScanSmem::OP + W_KD, ws_of(c) + W_KD, W_PH, &bar[SB_KD]);
  };
  auto load_ph = [&](int c) {
    ++loads[3];
    mbar_expect_tx(&bar[SB_PH], W_OP - W_PH);
    bulk_load(sb + ScanSmem::OP + W_PH, ws_of(c) + W_PH, W_OP - W_PH, &bar[SB_PH]);
  };
  // What chunk c will load, into L2.
  auto prefetch = [&](int c) {
    const int t = (int)(s.begin + (long long)c * DC);
    box_prefetch(&maps.k0, 0, h, t);
    box_prefetch(&maps.q0, 0, h, t);
    box_prefetch(&maps.k1, 64, h, t);
    box_prefetch(&maps.q1, 64, h, t);
    box_prefetch(&maps.v, tile * TN, h, t);
    bulk_prefetch(ws_of(c), W_FWD);
  };

  float2 S[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) S[x] = both(0.f);
  if (s_row && from >= 0) {
    const float4* src = reinterpret_cast<const float4*>(a.h0 + (((long long)from * a.H + h) * DK + row) * DV + col0);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 w = src[x];
      S[2 * x] = make_float2(w.x, w.y);
      S[2 * x + 1] = make_float2(w.z, w.w);
    }
  }
  auto put_state = [&](int x) {  // hi and lo of 16 columns of the state row, the next product's operand
#pragma unroll
    for (int c = 2 * x; c < 2 * x + 2; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2(S[4 * c + e], hi[e], lo[e]);
      const uint32_t at = sb + ScanSmem::S + sw128(row, 4 * half + c);
      st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
      st_shared_v4(at + 12288, lo[0], lo[1], lo[2], lo[3]);
    }
  };
  if (nc > 0) {
    if (warp == 0) tm_alloc<256>(slot_tm);
    if (loader) {
      for (int x = 0; x < SB_N; ++x) mbar_init(&bar[x], 1);
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      fence_async_smem();
      load_rows(0);
      load_v(0);
      load_kd(0);
      load_ph(0);
      if (nc > 1) prefetch(1);
    }
    if (s_row) {
      put_state(0);
      put_state(1);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    const uint32_t tmem = *slot_tm;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    float2 qs[16];
    bool ok = true;
    // The outputs of chunk c (Q's warps), from the place that its first product had.
    const uint32_t stage = sb + ScanSmem::OUT + 2048u * ((q & 1) + 2 * half);  // this warp's 32 rows x 32 columns
    auto outputs = [&](int c) {
      ok = mbar_wait(&bar[SB_O], c & 1, a.wait_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (loader && c + 1 < nc) load_ph(c + 1);
      tc_fence_after();
      const uint32_t from_tm = tmem + lanes + (c & 1) * 128u + 32u * half;
      const int left = s.len - c * DC;
      const long long t0 = s.begin + (long long)c * DC;
      if ((tid & 31) == 0) stores_read();
      __syncwarp();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t d[32], w[8];
        tm_ld16x2(from_tm + 16 * x, from_tm + 64 + 16 * x, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 y = fmul2(both(a.scale), fadd2(qs[8 * x + e], halves(d, e)));
          w[e] = bf2(y.x, y.y);
        }
        if (left >= DC) {
          st_shared_v4(stage + sw64(tid & 31, 2 * x), w[0], w[1], w[2], w[3]);
          st_shared_v4(stage + sw64(tid & 31, 2 * x + 1), w[4], w[5], w[6], w[7]);
        } else if (tok < left) {  // a sequence's last rows: no box is written past them
          uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + ((t0 + tok) * a.H + h) * DV + col0);
          dst[2 * x] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[2 * x + 1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (left >= DC) {
        fence_async_smem();
        __syncwarp();
        if ((tid & 31) == 0) box_store(&maps.o, stage, col0, h, (int)(t0 + 32 * (q & 1)));
      }
    };
    int c = 0;
    for (; c < nc; ++c) {
      const uint32_t ph = c & 1, at_a = tmem + ph * 128u, at_c = tmem + (ph ^ 1) * 128u;
      if (issuer && mbar_wait(&bar[SB_KQ], ph, a.wait_ns, abort_flag)) {
        tc_fence_after();
        const SDesc d0 = sdesc(sb + ScanSmem::KQ0, 16, 1024, LAYOUT_SW128), d1 = sdesc(sb + ScanSmem::KQ1, 16, 512, LAYOUT_SW64);
        const SDesc ds = sdesc(sb + ScanSmem::S, 12288, 1024, LAYOUT_SW128);
#pragma unroll
        for (int kk = 0; kk < 6; ++kk)
          umma(at_a, kk < 4 ? d0 + kk * 32u : d1 + (kk - 4) * 32u, ds + kk * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
        umma_commit(&bar[SB_A]);
      }
      __syncwarp();
      ok = true;
      if (!k_row && c > 0) outputs(c - 1);
      ok = ok && mbar_wait(&bar[SB_V], ph, a.wait_ns, abort_flag) && mbar_wait(&bar[SB_A], ph, a.wait_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      float last = 0.f;
      if (ok) {
        if (loader && c + 1 < nc) load_rows(c + 1);
        tc_fence_after();
        const float* gt = reinterpret_cast<const float*>(sm + ScanSmem::GT);
        const float f_row = gt[tok], b_row = gt[DC + tok];
        const bool live = tok < s.len - c * DC;  // (rows behind the last hold the next sequence's)
        last = gt[DC - 1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t d[32];
          tm_ld16x2(at_a + lanes + 32 * half + 16 * x, at_a + lanes + 64 + 32 * half + 16 * x, d);
          if (k_row) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t piece = sw128(tok, 4 * half + 2 * x + p);
              const uint4 v4 = ld_shared_v4(sb + ScanSmem::V + piece);
              const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 r = fmul2(both(b_row), fmadd2(both(-f_row), halves(d, 4 * p + e), widen2(vw[e])));
                split2(live ? r : both(0.f), hi[e], lo[e]);
              }
              st_shared_v4(sb + ScanSmem::BR + piece, hi[0], hi[1], hi[2], hi[3]);
              st_shared_v4(sb + ScanSmem::BR + 8192 + piece, lo[0], lo[1], lo[2], lo[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) qs[8 * x + e] = fmul2(both(f_row), halves(d, e));
          }
        }
      }
      fence_async_smem();
      tc_fence_before();
      if (__syncthreads_or(!ok)) break;
      if (issuer) {
        tc_fence_after();
        const SDesc dk = sdesc(sb + ScanSmem::OP + W_KD, 16, 1024, LAYOUT_SW128);
        const SDesc dp = sdesc(sb + ScanSmem::OP + W_PH - 8192, 16, 1024, LAYOUT_SW128);  // P^ in rows 64-127
        const SDesc db = sdesc(sb + ScanSmem::BR, 8192, 1024, LAYOUT_SW128);
        if (mbar_wait(&bar[SB_KD], ph, a.wait_ns, abort_flag)) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma(at_c, dk + (kk >> 2) * 12288u + (kk & 3) * 32u, db + (kk & 3) * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
          umma_commit(&bar[SB_C]);
        }
        if (mbar_wait(&bar[SB_PH], ph, a.wait_ns, abort_flag)) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma(at_a, dp + kk * 32u, db + kk * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
          umma_commit(&bar[SB_O]);
        }
      }
      __syncwarp();
      if (loader && c + 1 < nc) load_v(c + 1);
      if (loader && c + 2 < nc) prefetch(c + 2);
      ok = mbar_wait(&bar[SB_C], ph, a.wait_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && loader && c + 1 < nc) load_kd(c + 1);
      if (ok && s_row) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t d[32];
          tm_ld16x2(at_c + lanes + 32 * half + 16 * x, at_c + lanes + 64 + 32 * half + 16 * x, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) S[8 * x + e] = fmadd2(both(last), S[8 * x + e], halves(d, e));
          if (c + 1 < nc) put_state(x);
        }
      }
      fence_async_smem();
      tc_fence_before();
      if (__syncthreads_or(!ok)) break;
    }
    bool gone = c < nc;
    ok = true;
    if (!gone && !k_row) outputs(nc - 1);
    if (!k_row && (tid & 31) == 0) stores_read();
    tc_fence_before();
    gone = __syncthreads_or(gone || !ok);
    if (gone) {
      // What was issued ends before its memory is given up: the products, and the last copy of each kind (the ones
      // before have been waited for).
      if (issuer) {
        raise_error(a.err, ERR_TIMEOUT);
        umma_commit(&bar[SB_DRAIN]);
        mbar_wait_drain(&bar[SB_DRAIN], 0, DRAIN_NS, a.err);
      }
      if (loader)
        for (int x = 0; x < 4; ++x) mbar_wait_drain(&bar[SB_KQ + x], (loads[x] - 1) & 1, DRAIN_NS, a.err);
      __syncthreads();
    }
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
      for (int x = 0; x < 8; ++x) dst[x] = make_float4(S[2 * x].x, S[2 * x].y, S[2 * x + 1].x, S[2 * x + 1].y);
    }
  }
}

}  // namespace

size_t delta_tc_ws_bytes(long long slots, int H) { return (size_t)slots * H * W_FWD; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// A [tokens, H, d] bf16 tensor in boxes of `cols` columns (64: 128-byte swizzle, 32: 64-byte) x one head x `rows` tokens.
static bool box_map(CUtensorMap* m, const void* base, int d, int H, long long tokens, int cols, int rows) {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess;
    return found ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2};
  const cuuint32_t box[3] = {(cuuint32_t)cols, 1, (cuuint32_t)rows}, step[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_delta_tc_fwd(const DeltaArgs& a, cudaStream_t st) {
  static OncePerDevice<CudaDeviceApi> once;
  cudaError_t e = once([] {
    const cudaError_t x = cudaFuncSetAttribute(delta_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PrepSmem::BYTES);
    return x != cudaSuccess ? x : cudaFuncSetAttribute(delta_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ScanSmem::BYTES);
  });
  if (e != cudaSuccess) return e;
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  DeltaMaps m;
  memset(&m, 0, sizeof(m));
  if (tokens > 0 && !(box_map(&m.k0, a.k, DK, a.H, tokens, 64, DC) && box_map(&m.k1, a.k, DK, a.H, tokens, 32, DC) &&
                      box_map(&m.q0, a.q, DK, a.H, tokens, 64, DC) && box_map(&m.q1, a.q, DK, a.H, tokens, 32, DC) &&
                      box_map(&m.v, a.v, DV, a.H, tokens, 64, DC) && box_map(&m.o, a.o, DV, a.H, tokens, 32, 32)))
    return cudaErrorInvalidValue;
  if (a.slots > 0) delta_prep_kernel<<<(unsigned)a.slots * a.H, 160, PrepSmem::BYTES, st>>>(m, a);
  delta_scan_kernel<<<(unsigned)a.n_seq * a.H * NTILE, SCAN_THREADS, ScanSmem::BYTES, st>>>(m, a);
  return cudaGetLastError();
}

}  // namespace gla
