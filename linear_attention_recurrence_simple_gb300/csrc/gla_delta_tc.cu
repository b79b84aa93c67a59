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
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
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
// One CTA of 4 warps a (chunk, head), all products on mma.sync (m16n8k16): the blocks are 16 wide and each step
// of the substitution waits for the one before, and accumulators are the next product's A operand as they stand.
//   1  warp w: rows 16 w .. of Q K^T (P, kept in registers), and K K^T's blocks that (B M)'s column block 3 - w needs:
//      off the diagonal as B operands (hi + lo) in shared memory, on it in fp32
//   2  the diagonal blocks' inverses (1 + B M_bb)^-1 by substitution, one thread a row, fp32
//   3  slabs of 16 rows y of y (1 + B M) = r, block by block from the last: Y_b = (R_b - sum_c Y_c BM_cb) W_b, each
//      product hi hi + hi lo + lo hi; a slab's rows leave through shared memory as one contiguous copy
// fp32 sums; what is carried from block to block has 16 bits.
constexpr int PREP_THREADS = 128;
struct PrepSmem {
  static constexpr uint32_t P0 = 0, P1 = 16384, STAGE = 24576, DM = STAGE, FRAG = STAGE + 4 * 4096, G = FRAG + 10 * 1024, B = G + DC * 8,
                            BAR = B + DC * 4, BYTES = BAR + 16;
};
static_assert(4 * 16 * 20 * 4 <= 4 * 4096, "the diagonal blocks take the stages' place");

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Piece c (8 columns) of row r of K or Q.
__device__ __forceinline__ uint32_t kq_at(uint32_t sb, bool is_q, int r, int c) {
  return sb + (c < 8 ? PrepSmem::P0 + (is_q ? 8192u : 0u) + sw128(r, c) : PrepSmem::P1 + (is_q ? 4096u : 0u) + sw64(r, c - 8));
}
// 16 x 16 block of X Y^T, rows r0 .. of X and n0 .. of Y: two accumulators of 8 columns.
__device__ __forceinline__ void block_dot(float (&d)[2][4], uint32_t sb, bool x_is_q, int r0, int n0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) d[0][i] = d[1][i] = 0.f;
#pragma unroll
  for (int ks = 0; ks < 6; ++ks) {
    uint32_t x[4], y[4];
    ldsm4(x, kq_at(sb, x_is_q, r0 + (lane & 15), 2 * ks + (lane >> 4)));
    ldsm4(y, kq_at(sb, false, n0 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
    mma(d[0], x, y[0], y[1]);
    mma(d[1], x, y[2], y[3]);
  }
}
// Accumulators of 16 columns as an A operand, hi and lo.
__device__ __forceinline__ void to_operand(const float (&x)[2][4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(make_float2(x[i >> 1][2 * (i & 1)], x[i >> 1][2 * (i & 1) + 1]), hi[i], lo[i]);
}
// d += (hi + lo) times a 16 x 16 block of B operands, hi and lo
__device__ __forceinline__ void block_mul(float (&d)[2][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], const uint8_t* frag) {
  const uint4 h = *reinterpret_cast<const uint4*>(frag + 16 * (threadIdx.x & 31)), l = *reinterpret_cast<const uint4*>(frag + 512 + 16 * (threadIdx.x & 31));
  mma(d[0], lo, h.x, h.y);
  mma(d[1], lo, h.z, h.w);
  mma(d[0], hi, l.x, l.y);
  mma(d[1], hi, l.z, l.w);
  mma(d[0], hi, h.x, h.y);
  mma(d[1], hi, h.z, h.w);
}
// Places of the B operands: -(B M) block (c, b), c > b, and the inverse of diagonal block b.
__device__ __forceinline__ constexpr int frag_off(int c, int b) { return c * (c - 1) / 2 + b; }
__device__ __forceinline__ constexpr int frag_diag(int b) { return 6 + b; }

// A slab's rows, blocks `top` .. 0 (the ones above are zero in r): solved, and copied out (128-byte rows; with
// `lo_out` what the rounding to bf16 leaves, too).
__device__ __forceinline__ void solve_slab(float (&r)[4][2][4], int top, const uint8_t* frags, uint8_t* sm, uint8_t* hi_out, uint8_t* lo_out) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* const stage = sm + PrepSmem::STAGE + 4096 * (threadIdx.x >> 5);
  uint32_t hi[4][4], lo[4][4];
#pragma unroll
  for (int b = 3; b >= 0; --b) {
    if (b <= top) {
#pragma unroll
      for (int c = 3; c > b; --c)
        if (c <= top) block_mul(r[b], hi[c], lo[c], frags + 1024 * frag_off(c, b));
      to_operand(r[b], hi[b], lo[b]);
      float y[2][4] = {};
      block_mul(y, hi[b], lo[b], frags + 1024 * frag_diag(b));
      to_operand(y, hi[b], lo[b]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) hi[b][i] = lo[b][i] = 0u;
    }
  }
  if (lane == 0) stores_read();
  __syncwarp();
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows g, g + 8; columns 16 b + 2 t, and 8 on
      const uint32_t at = sw128(g + 8 * (i & 1), 2 * b + (i >> 1)) + 4 * t;
      *reinterpret_cast<uint32_t*>(stage + at) = hi[b][i];
      *reinterpret_cast<uint32_t*>(stage + 2048 + at) = lo[b][i];
    }
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    bulk_store(hi_out, smem_u32(stage), 2048);
    if (lo_out) bulk_store(lo_out, smem_u32(stage + 2048), 2048);
    stores_commit();
  }
}
// Rows a0 .. of (diag(w) K)^T, w a token's weight.
template <class W>
__device__ __forceinline__ void transposed_slab(float (&r)[4][2][4], const uint32_t (&raw)[4][4], int len, W weight) {
  const int t = threadIdx.x & 3;
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = 16 * b + 8 * n + 2 * t;
      const float w0 = weight(j), w1 = weight(j + 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = widen2(raw[b][2 * n + i]);
        r[b][n][2 * i] = j < len ? w0 * x.x : 0.f;
        r[b][n][2 * i + 1] = j + 1 < len ? w1 * x.y : 0.f;
      }
    }
}
__device__ __forceinline__ void load_transposed(uint32_t (&raw)[4][4], uint32_t sb, bool is_q, int a0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < 4; ++b) ldsm4t(raw[b], kq_at(sb, is_q, 16 * b + 8 * (lane >> 4) + (lane & 7), a0 / 8 + ((lane >> 3) & 1)));
}

__global__ void __launch_bounds__(PREP_THREADS, 4) delta_prep_kernel(const __grid_constant__ DeltaMaps maps, const DeltaArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  float* const dm = reinterpret_cast<float*>(sm + PrepSmem::DM);   // [4][16][20]: diagonal blocks of B M
  uint8_t* const frags = sm + PrepSmem::FRAG;
  float2* const sg = reinterpret_cast<float2*>(sm + PrepSmem::G);  // sums of log2 decays
  float* const sbeta = reinterpret_cast<float*>(sm + PrepSmem::B);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + PrepSmem::BAR);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + PrepSmem::BAR + 8);
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) return;
  uint8_t* const ws = a.ws + ((long long)slot * a.H + h) * W_FWD;
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    load_kq(maps, sb + PrepSmem::P0, sb + PrepSmem::P1, bar, h, (int)ch.t0);
  }
  if (warp == 1) {
    const __nv_bfloat16* gp = (const __nv_bfloat16*)a.g + ch.t0 * a.H + h;
    const __nv_bfloat16* bp = (const __nv_bfloat16*)a.beta + ch.t0 * a.H + h;
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      x[e] = i < ch.len ? to_f(gp[(long long)i * a.H]) : 0.f;
      sbeta[i] = i < ch.len ? to_f(bp[(long long)i * a.H]) : 0.f;
    }
    float2 s0, s1;
    delta_sums<true>(x[0], x[1], s0, s1);
    sg[2 * lane] = s0;
    sg[2 * lane + 1] = s1;
  }
  __syncthreads();
  bool ok = mbar_wait(bar, 0, a.wait_ns, abort_flag);
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      raise_error(a.err, ERR_TIMEOUT);
      mbar_wait_drain(bar, 0, DRAIN_NS, a.err);
    }
    return;
  }
  auto decay = [&](int i, int j) {  // of token j's part in token i
    const float2 x = sg[i], y = sg[j];
    return exp2_fast((x.x - y.x) + (x.y - y.y));
  };
  // 1: P's rows (those behind the last token may hold another sequence's)
  float r[4][2][4];
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (b <= warp) {
      block_dot(r[b], sb, true, 16 * warp, 16 * b);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * warp + g + 8 * (e >> 1), j = 16 * b + 8 * n + 2 * t + (e & 1);
          r[b][n][e] = j <= i && i < ch.len ? decay(i, j) * r[b][n][e] : 0.f;
        }
    }
#pragma unroll
  for (int jb = 0; jb < 4; ++jb) {
    const int mb = 3 - warp;
    if (jb > mb) continue;
    float x[2][4];  // rows j, columns m
    block_dot(x, sb, false, 16 * jb, 16 * mb);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 16 * jb + g + 8 * (e >> 1), m = 16 * mb + 8 * n + 2 * t + (e & 1);
        x[n][e] = j < m && m < ch.len ? -sbeta[m] * (decay(m, j) * x[n][e]) : 0.f;
        if (jb == mb) dm[(mb * 16 + (m & 15)) * 20 + (j & 15)] = x[n][e];
      }
    if (jb != mb) {  // rows of x are the operand's columns
      uint32_t hi[4], lo[4];
      to_operand(x, hi, lo);
      uint8_t* const f = frags + 1024 * frag_off(mb, jb) + 16 * lane;
      *reinterpret_cast<uint4*>(f) = make_uint4(hi[0], hi[2], hi[1], hi[3]);
      *reinterpret_cast<uint4*>(f + 512) = make_uint4(lo[0], lo[2], lo[1], lo[3]);
    }
  }
  __syncthreads();
  // 2: warp b, lane i < 16: row i of the inverse of diagonal block b
  if (lane < 16) {
    float y[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = j == lane ? 1.f : 0.f;
#pragma unroll
    for (int m = 15; m > 0; --m)
#pragma unroll
      for (int j = 0; j < m; ++j) y[j] = fmaf(y[m], dm[(warp * 16 + m) * 20 + j], y[j]);
    __nv_bfloat16* const f = reinterpret_cast<__nv_bfloat16*>(frags + 1024 * frag_diag(warp));
#pragma unroll
    for (int j = 0; j < 16; ++j) {  // operand element (k = lane, n = j)
      const int at = (((j & 7) * 4 + ((lane & 7) >> 1)) * 4 + (j >> 3) * 2 + (lane >> 3)) * 2 + (lane & 1);
      const __nv_bfloat16 x = __float2bfloat16_rn(y[j]);
      f[at] = x;
      f[256 + at] = __float2bfloat16_rn(y[j] - __bfloat162float(x));
    }
  }
  if (tid < DC) {
    float* const gt = reinterpret_cast<float*>(ws + W_GT);
    gt[tid] = exp2_fast(sg[tid].x + sg[tid].y);
    gt[DC + tid] = sbeta[tid];
  }
  __syncthreads();
  // 3: the rows of P^, then those of K^: two slabs for the warps with short rows of P, one for the others
  solve_slab(r, warp, frags, sm, ws + W_PH + 2048 * warp, nullptr);
  const int slab0 = warp < 2 ? 2 * warp : 2 + warp, slabs = warp < 2 ? 2 : 1;
  for (int x = slab0; x < slab0 + slabs; ++x) {
    uint32_t raw[4][4];
    load_transposed(raw, sb, false, 16 * x);
    transposed_slab(r, raw, ch.len, [&](int j) { return decay(DC - 1, j); });
    solve_slab(r, 3, frags, sm, ws + W_KD + 2048 * x, ws + W_KD + 12288 + 2048 * x);
  }
  if (lane == 0) stores_read();
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
  if (a.slots > 0) delta_prep_kernel<<<(unsigned)a.slots * a.H, PREP_THREADS, PrepSmem::BYTES, st>>>(m, a);
  delta_scan_kernel<<<(unsigned)a.n_seq * a.H * NTILE, SCAN_THREADS, ScanSmem::BYTES, st>>>(m, a);
  return cudaGetLastError();
}

}  // namespace gla
