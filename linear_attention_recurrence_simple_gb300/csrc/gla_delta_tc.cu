// The gated delta rule on the 5th-generation tensor cores (bf16 calls).  Formulas: gla_delta.cuh.
//
//   prep    one CTA a (chunk, head): K K^T and Q K^T, the decays, and the triangular system, solved once for everything
//           that it multiplies: rows y with y (1 + B M) = r, 16 x 16 blocks by back substitution.  With r the rows of P
//           and of (diag(e^(G_C - G)) K)^T it gives P^ and K^, and the chunk is
//               O = s (diag(e^G) Q S0 + P^ B R),   S1 = e^(G_C) S0 + K^ B R,   R = V - diag(e^G) K S0:
//           U is never formed, and two dependent products are left between a state and the next instead of three.
//           Backward: also Z, P, Q~ = s (diag(e^G) Q)^T and K~ = -(diag(e^G) K)^T (1 + B M^T)^-1.
//   scan    one CTA a (sequence, head, 64 columns of d_v), chunks in order: [K; Q] S0 (one M = 128 product), then
//           K^ B R and P^ B R.  Tiles of d_v are independent.  Backward: the same pass, which keeps each chunk's S0 and X
//   rscan   the same from the last chunk on: dU = s P^T dO + E K dS1, w = B dU, dS0 = e^(G_C) dS1 + Q~ dO + K~ w; writes
//           dv, every chunk's dS1 and its columns' part of dbeta
//   grads   one CTA a (chunk, head): dq, dk, dg, and dbeta's parts summed in tile order
// States are fp32; what carries them from chunk to chunk enters the products as two halves, [hi | lo] beside each other as N = 128
// columns.  K^, B R and K~, w are two fp16 (22 bits), as are prep's operands; beside operands that are exact in bf16, Q~ is
// three bf16 (24 bits) and S, dS and P two (16 bits).  For fp16's range keys are brought to a length of 1/2 to 1, and residuals
// scaled by a bound (see prep and the scan).  P^ and Z are one fp16.  X, Es and Fm, which nearly every gradient goes through,
// are two bf16; S0 and dS1 for the gradients one.  hT and dh0 are 0.2 to 0.9e-6 of the norm from the exact ones (with two bf16
// throughout 4.4 and 3.1e-6), o and dbeta 1.7e-3, their own rounding (2.1 and 2.3e-3), dq and dk 2.0e-3 and dg 2.4e-3 (with X,
// Es and Fm in one bf16 3.0e-3).  What that costs: forward of 8 x 2,048 x 16 221 -> 256 us, backward 675 -> 771.
// What the chunk's length costs: longer chunks halve the scans' steps, but prep and grads grow with its square; 64 tokens
// are also the 128 rows of [K; Q] and the 128 bytes of a swizzled row.
#include <cuda.h>
#include <cuda_fp16.h>
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
__device__ __forceinline__ float2 pair(const uint32_t (&d)[32], int e) { return make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])); }
// columns 2 e and 2 e + 1 of a product that stands as [hi | lo], the halves added.  (Beside each other: a product's A operand is read
// once for both, and that reading is what bounds these products; both into the same 64 columns, one after the other, the
// scans take 60 us more.)
__device__ __forceinline__ float2 halves(const uint32_t (&d)[32], int e) {
  return fadd2(pair(d, e), make_float2(__uint_as_float(d[16 + 2 * e]), __uint_as_float(d[17 + 2 * e])));
}
// A pair as two bf16 pairs, hi + lo.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = bf2(x.x, x.y);
  const float2 r = fsub2(x, widen2(hi));
  lo = bf2(r.x, r.y);
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// The same in fp16: 22 bits, for values that a power of two has brought into its range.
__device__ __forceinline__ uint32_t hf2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void split2h(float2 x, uint32_t& hi, uint32_t& lo) {
  // (cut off, not rounded: the first then needs no conversion back, and the second keeps 11 bits of what is left)
  const float2 h = make_float2(__uint_as_float(__float_as_uint(x.x) & 0xFFFFE000u), __uint_as_float(__float_as_uint(x.y) & 0xFFFFE000u));
  const float2 r = fsub2(x, h);
  hi = hf2(h.x, h.y);
  lo = hf2(r.x, r.y);
}
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) { return idesc_bf16(M, N, a_mn, b_mn) & ~(1u << 7 | 1u << 10); }
// The power of two that brings `top` to 2^T .. 2^(T + 1), and its inverse.  (Of values below 2^-112 or so, and of zero, one that
// brings them less far: both stay normal numbers.)
template <int T>
__device__ __forceinline__ float2 pow2_to(float top) {
  const int e = min(max((int)(__float_as_uint(top) >> 23), T + 1), 254);
  return make_float2(__uint_as_float((uint32_t)(254 + T - e) << 23), __uint_as_float((uint32_t)(e - T) << 23));
}
__device__ __forceinline__ float finite_size(float x) { return fabsf(x) < __int_as_float(0x7f800000) ? fabsf(x) : 0.f; }
// The largest magnitude of a thread's values (a NaN does not count), and of a warp's.
__device__ __forceinline__ float most_of(const float2 (&x)[16]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) m = fmaxf(m, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
  return m;
}
__device__ __forceinline__ float warp_most(float m) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))); }
__device__ __forceinline__ float most_of4(const float* m) {
  const float4 x = *reinterpret_cast<const float4*>(m);
  return fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
}
// The largest finite magnitude in the first rows of a tile of 64 x 64 bf16 in 128-byte rows, by a whole warp.
__device__ __forceinline__ float most_of_tile(uint32_t tile, int rows) {
  const int lane = threadIdx.x & 31;
  __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 4
  for (int e = lane; e < 8 * rows; e += 32) {
    const uint4 x = ld_shared_v4(tile + 16 * e);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __nv_bfloat162 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    m = __hmax2(m, __hmax2(__hmax2(y[0], y[1]), __hmax2(y[2], y[3])));
  }
  float top = fmaxf(__low2float(m), __high2float(m));
  if (!(top < __int_as_float(0x7f800000))) {
    top = 0.f;
#pragma unroll 1
    for (int e = lane; e < 8 * rows; e += 32) {
      const uint4 x = ld_shared_v4(tile + 16 * e);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(finite_size(__uint_as_float(w[i] << 16)), finite_size(__uint_as_float(w[i] & 0xFFFF0000u))));
    }
  }
  return warp_most(top);
}
// (a power of two for the smallest residuals, times a large weight)
__device__ __forceinline__ float no_more(float x) { return fminf(fmaxf(x, -3e38f), 3e38f); }
// pow2_to for a bound that need not be a number: then nothing is.
template <int T>
__device__ __forceinline__ float2 pow2_of_bound(float bound) {
  const float2 p = pow2_to<T>(bound);
  return bound < __int_as_float(0x7f800000) ? p : both(__int_as_float(0x7fc00000));
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
// 16 columns of this thread's lane.
__device__ __forceinline__ void tm_ld16(uint32_t ta, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(ta)
      : "memory");
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

// Who waits, for gla_debug_give_up: the role is 0 for the thread of the copies, 1 for that of the products, 2 for the warps
// with rows; the chunk is the kernel, the barrier and the phase in one number (phases past 31 are not told apart: -1).
enum { IN_PREP = 0, IN_SCAN, IN_RSCAN, IN_GRADS };
__device__ __forceinline__ constexpr int wait_code(int kernel, int bar, int k) { return k < 32 ? kernel << 10 | bar << 5 | k : -1; }
// mbar_wait_at with a look first: try_wait takes its time even where the phase has ended.  (For a thread that mostly finds
// it ended: the reverse scan's issuer, 228 -> 213 us; the scans, whose two CTAs share an SM, lose 3 % to 10 % by it.)
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, unsigned long long limit_ns, volatile int* abort, int role, int code) {
  if constexpr (kDebugBounds) return mbar_wait_at(bar, parity, limit_ns, abort, role, code);
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0 || mbar_wait_at(bar, parity, limit_ns, abort, role, code);
}

constexpr unsigned long long DRAIN_NS = 1000000000ull;

// Tensor maps of a call.  K and Q: a chunk's 64 rows in two boxes, columns 0-63 (128-byte rows) and 64-95 (64-byte
// rows).  V: 64 rows x 64 columns.  O: 32 rows x 32 columns, one a warp.
// (backward) dO: 64 rows x 64 columns; K and Q in two boxes of 64 columns (96 on: zeros); dv as dO; X (hi and lo), S0 and
// dS1 of the workspace: 128 or 96 rows x 64 columns of a (chunk place, head).
struct DeltaMaps {
  CUtensorMap k0, k1, q0, q1, v, o;
  CUtensorMap dO, dv, x, s0, ds;
  CUtensorMap dvo, xo, xlo;  // (to write: 32 rows x 32 columns, one a warp)
  CUtensorMap xsd;      // X, S0 and dS1, half of their rows: 160 rows x 64 columns
  CUtensorMap dqo, dko; // (to write: 32 rows x 48 columns)
};
__device__ __forceinline__ void load_kq(const DeltaMaps& m, uint32_t p0, uint32_t p1, uint64_t* bar, int h, int t) {
  mbar_expect_tx(bar, 24576);
  box_load(p0, &m.k0, bar, 0, h, t);
  box_load(p0 + 8192, &m.q0, bar, 0, h, t);
  box_load(p1, &m.k1, bar, 64, h, t);
  box_load(p1 + 4096, &m.q1, bar, 64, h, t);
}

// ---- workspace of a (chunk place, head), in bytes --------------------------------------------
// Operands as the swizzled tiles that the scans copy, 128-byte rows of 64 tokens, fp16: K^ hi and lo (96 rows, d_k), P^ or
// (backward) Z (64 rows), all of keys of length 1/2 to 1 (see prep).  Then in fp32: e^G; beta times the power of two of
// the key's length; numbers (below); (backward) the powers; beta; e^(G_C - G) (64 each); the sums of the logs to base 2.
constexpr uint32_t W_KD = 0, W_PH = 24576, W_OP = 32768, W_GT = W_OP;
enum { GT_F = 0, GT_BC = DC, GT_SC = 2 * DC, GT_C = GT_SC + 16, GT_B = GT_C + DC, GT_E = GT_B + DC, GT_SUM = GT_E + DC, GT_ALL = GT_SUM + 2 * DC };  // in floats
// Numbers: what the products of P^'s rows (16 each) and of K~ are to be multiplied with; and what bounds what the scans bring to
// fp16, |S| the length of a state's column, v and d the largest of V and dO:
//     |c beta R| <= CB v + UB |S|,  |c beta dU| <= UE |dS1| + UP d,  |dS0| <= LG (e^(G_C) |dS1| + WQ d)
// and for |S1| (with x = beta |k|^2, e = v - k . S, a write turns |S|^2 to |S|^2 + 2 beta v e - beta (2 - x) e^2, which is
// |S|^2 + beta v^2 / (2 - x) at most: a state's length grows with the root of the tokens)
//     |S1| <= LG sqrt(e^(2 G_C) |S|^2 + A v^2)  (A >= 0),  or, where an x is near 2, LG (e^(G_C) |S| - A v)
enum { SC_PH = 0, SC_KR = 4, SC_CB, SC_UB, SC_LG, SC_A, SC_UE, SC_UP, SC_WQ };
constexpr uint32_t GT_SCAN = 4 * GT_C, GT_STATES = 4 * GT_B, GT_RSCAN = 4 * GT_SUM;  // what the scans read of it, in bytes
constexpr float OP_SCALE = 64.f;  // K^ and Z, which are 1 at most (but where a recurrence grows), stand times this
constexpr float ROOT_DK = 10.f;  // the length of a column of 96 over its largest, and some
constexpr uint32_t W_FWD = W_GT + GT_SCAN;
// Backward: K~ = -(diag(e^G) K)^T (1 + B M^T)^-1 in fp16, hi and lo; Q~ = s (diag(e^G) Q)^T in three bf16, P in two; then what the
// scans leave for the gradients, bf16 rows of 192: X hi and lo (64 each), S0 and dS1 (96), one 320-row tile.
constexpr uint32_t W_KR = W_GT + 2048, W_QT = W_KR + 24576, W_P = W_QT + 36864, W_X = W_P + 16384, W_XL = W_X + DC * DV * 2,
                   W_S0 = W_XL + DC * DV * 2, W_DS = W_S0 + DK * DV * 2, W_BWD = W_DS + DK * DV * 2;
static_assert(W_FWD % 16 == 0 && W_BWD % 256 == 0 && 4 * GT_ALL <= 2048 && GT_RSCAN % 16 == 0 && (4 * GT_B) % 16 == 0 && W_KR % 16 == 0 && W_X % 32 == 0, "copies and tensor maps");

// ---- prep -------------------------------------------------------------------------------------
// One CTA of 4 warps a (chunk, head), all products on mma.sync (m16n8k16): the blocks are 16 wide and each step
// of the substitution waits for the one before, and accumulators are the next product's A operand as they stand.
//   1  warp w: rows 16 w .. of Q K^T (P, kept in registers), and K K^T's blocks that (B M)'s column block 3 - w needs:
//      off the diagonal as B operands (hi + lo) in shared memory, on it in fp32
//   2  the diagonal blocks' inverses (1 + B M_bb)^-1 by substitution, one thread a row, fp32
//   3  slabs of 16 rows y of y (1 + B M) = r, block by block from the last: R'_b = R_b - sum_c Y_c BM_cb,
//      Y_b = R'_b + R'_b (W_b - 1), each product hi hi + hi lo + lo hi
// fp32 sums; operands are two fp16 (22 bits).  For its range keys are brought to a length of 1/2 to 1 by powers of two c_j, exactly:
// with k = c k', k u^T = k' (c u)^T, where c u = (c beta) x, so that K^, P^ and Z come out as those of k', and the scans weigh
// their residuals with c beta instead of beta; the system is (1 + C B M C^-1), whose entries are below 4 where beta |k|^2 <= 2.
// Bound by the latency of its chain (loads, products, a substitution of 16 steps, four of blocks) at 16 (backward 12) warps
// an SM, held there by 128 (168) registers and 56 (66) KB: 8 sequences of 2,048 tokens x 16 heads, 4,096 CTAs, 77 us
// (153), of which the bytes written take 20 (76); with operands of two bf16 and Q~ in two 69 (127).  With the products on
// tcgen05 and one thread a row of the substitution 137.
constexpr int PREP_THREADS = 128;
struct PrepSmem {
  static constexpr uint32_t P0 = 0, P1 = 16384, STAGE = 24576, DM = STAGE, G = STAGE + 4 * 4096, B = G + DC * 8, F = B + DC * 4, E = F + DC * 4,
                            CF = E + DC * 4, RF = CF + DC * 4, BAR = RF + 3 * DC * 4, PM = BAR + 16, C = BAR + 256, IC = C + DC * 4, BC = IC + DC * 4,
                            LG = BC + DC * 4, NK = LG + DC * 4, EK = NK + DC * 4, FK = EK + DC * 4, FRAG = FK + DC * 4;
  static constexpr uint32_t bytes(bool bwd) { return FRAG + (bwd ? 20 : 10) * 1024; }
};
constexpr int DM_FLOATS = 4 * 16 * 20;
static_assert(2 * DM_FLOATS * 4 <= 4 * 4096 && PrepSmem::FRAG % 16 == 0, "the diagonal blocks take the stages' place");

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Piece c (8 columns) of row r of K or Q.
__device__ __forceinline__ uint32_t kq_at(uint32_t sb, bool is_q, int r, int c) {
  return sb + (c < 8 ? PrepSmem::P0 + (is_q ? 8192u : 0u) + sw128(r, c) : PrepSmem::P1 + (is_q ? 4096u : 0u) + sw64(r, c - 8));
}
// 16 x 16 block of X Y^T, rows r0 .. of X and n0 .. of Y (K or Q): two accumulators of 8 columns.
__device__ __forceinline__ void block_dot(float (&d)[2][4], uint32_t sb, bool x_is_q, int r0, int n0, bool y_is_q = false) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) d[0][i] = d[1][i] = 0.f;
#pragma unroll
  for (int ks = 0; ks < 6; ++ks) {
    uint32_t x[4], y[4];
    ldsm4(x, kq_at(sb, x_is_q, r0 + (lane & 15), 2 * ks + (lane >> 4)));
    ldsm4(y, kq_at(sb, y_is_q, n0 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
    mma(d[0], x, y[0], y[1]);
    mma(d[1], x, y[2], y[3]);
  }
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Accumulators of 16 columns as an A operand, hi and lo, in fp16 or (BF) bf16.
template <bool BF = false>
__device__ __forceinline__ void to_operand(const float (&x)[2][4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = make_float2(x[i >> 1][2 * (i & 1)], x[i >> 1][2 * (i & 1) + 1]);
    if (BF) split2(y, hi[i], lo[i]);
    else split2h(y, hi[i], lo[i]);
  }
}
// r += (hi + lo) times a 16 x 16 block of B operands, hi (h) and lo (l).  (The tensor cores cut sums off: on r, which is larger than
// what comes to it, hT would be 0.8e-6 of the norm off instead of 0.6.)
__device__ __forceinline__ void block_mul(float (&r)[2][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], uint4 h, uint4 l) {
  float d[2][4] = {};
  mma_f16(d[0], lo, h.x, h.y);
  mma_f16(d[1], lo, h.z, h.w);
  mma_f16(d[0], hi, l.x, l.y);
  mma_f16(d[1], hi, l.z, l.w);
  mma_f16(d[0], hi, h.x, h.y);
  mma_f16(d[1], hi, h.z, h.w);
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i >> 2][i & 3] += d[i >> 2][i & 3];
}
// Places of the B operands: -(B M) block (c, b), c > b, and the inverse of diagonal block b without its ones; from 10 on the
// same of (B M^T): block (b, c), b < c, and the inverse.
__device__ __forceinline__ constexpr int frag_off(int c, int b) { return c * (c - 1) / 2 + b; }
__device__ __forceinline__ constexpr int frag_diag(int b) { return 6 + b; }

struct Slab {  // 16 rows x 64 columns as A operands, hi and lo
  uint32_t hi[4][4], lo[4][4];
};
// Rows r, of which blocks up to `top` are not zero, times (1 + B M)^-1, or (UP) (1 + B M^T)^-1 (top = 3).  N slabs at
// a time: they share the operands' loads, and each waits less on its own products.
template <bool UP, int N>
__device__ __forceinline__ void solve_slabs(float (&r)[N][4][2][4], const int (&top)[N], const uint8_t* frags, Slab (&s)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int step = 0; step < 4; ++step) {
    const int b = UP ? step : 3 - step;
#pragma unroll
    for (int before = 0; before < step; ++before) {
      const int c = UP ? before : 3 - before;
      const int id = UP ? 10 + frag_off(b, c) : frag_off(c, b);
      const uint8_t* f = frags + 1024 * id + 16 * lane;
      const uint4 h = *reinterpret_cast<const uint4*>(f), l = *reinterpret_cast<const uint4*>(f + 512);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c <= top[i]) block_mul(r[i][b], s[i].hi[c], s[i].lo[c], h, l);
    }
    const int id = (UP ? 10 : 0) + frag_diag(b);
    const uint8_t* f = frags + 1024 * id + 16 * lane;
    const uint4 h = *reinterpret_cast<const uint4*>(f), l = *reinterpret_cast<const uint4*>(f + 512);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (b <= top[i]) {
        to_operand(r[i][b], s[i].hi[b], s[i].lo[b]);
        block_mul(r[i][b], s[i].hi[b], s[i].lo[b], h, l);
        to_operand(r[i][b], s[i].hi[b], s[i].lo[b]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i].hi[b][e] = s[i].lo[b][e] = 0u;
      }
    }
  }
}
// The largest of a slab's values.
__device__ __forceinline__ float most_of_slab(const float (&r)[4][2][4]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) m = fmaxf(m, finite_size(r[e >> 3][(e >> 2) & 1][e & 3]));
  return warp_most(m);
}
// A slab's rows, copied out: 128-byte rows, with `lo_out` what the rounding of the first leaves, too.
__device__ __forceinline__ void store_slab(const Slab& s, uint8_t* sm, uint8_t* hi_out, uint8_t* lo_out) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* const stage = sm + PrepSmem::STAGE + 4096 * (threadIdx.x >> 5);
  if (lane == 0) stores_read();
  __syncwarp();
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows g, g + 8; columns 16 b + 2 t, and 8 on
      const uint32_t at = sw128(g + 8 * (i & 1), 2 * b + (i >> 1)) + 4 * t;
      *reinterpret_cast<uint32_t*>(stage + at) = s.hi[b][i];
      *reinterpret_cast<uint32_t*>(stage + 2048 + at) = s.lo[b][i];
    }
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    bulk_store(hi_out, smem_u32(stage), 2048);
    if (lo_out) bulk_store(lo_out, smem_u32(stage + 2048), 2048);
    stores_commit();
  }
}
// Rows a0 .. of (diag(w) K)^T, w the tokens' weights, times `sign`.
__device__ __forceinline__ void transposed_slab(float (&r)[4][2][4], uint32_t sb, bool is_q, int a0, const float* w, float sign) {
  const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    uint32_t raw[4];
    ldsm4t(raw, kq_at(sb, is_q, 16 * b + 8 * (lane >> 4) + (lane & 7), a0 / 8 + ((lane >> 3) & 1)));
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float2 ww = fmul2(both(sign), *reinterpret_cast<const float2*>(w + 16 * b + 8 * n + 2 * t));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = fmul2(ww, widen2(raw[2 * n + i]));
        r[b][n][2 * i] = x.x;
        r[b][n][2 * i + 1] = x.y;
      }
    }
  }
}

template <bool BWD>
__global__ void __launch_bounds__(PREP_THREADS, BWD ? 3 : 4) delta_prep_kernel(const __grid_constant__ DeltaMaps maps, const DeltaArgs a, int ahead) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  float* const dm = reinterpret_cast<float*>(sm + PrepSmem::DM);   // [4][16][20]: diagonal blocks of -B M, and of -B M^T
  uint8_t* const frags = sm + PrepSmem::FRAG;
  float* const pm = reinterpret_cast<float*>(sm + PrepSmem::PM);  // [4] (backward) the largest |q|^2 of 16
  // the powers of two of the keys' lengths, their inverses; c beta; the weights of K^'s and K~'s right-hand sides
  float* const sc = reinterpret_cast<float*>(sm + PrepSmem::C);
  float* const sic = reinterpret_cast<float*>(sm + PrepSmem::IC);
  float* const sbc = reinterpret_cast<float*>(sm + PrepSmem::BC);
  float* const slg = reinterpret_cast<float*>(sm + PrepSmem::LG);  // what a token lets the state grow by, to base 2: 0 in use
  float* const snk = reinterpret_cast<float*>(sm + PrepSmem::NK);  // |k|^2
  float* const sek = reinterpret_cast<float*>(sm + PrepSmem::EK);
  float* const sfk = reinterpret_cast<float*>(sm + PrepSmem::FK);
  float2* const sg = reinterpret_cast<float2*>(sm + PrepSmem::G);  // sums of log2 decays
  float* const sbeta = reinterpret_cast<float*>(sm + PrepSmem::B);
  // e^G, e^(G_C - G); and the decays between blocks in two factors that are both at most 1: from token j to the end of its
  // block, and from there (end of block 0, 1, 2) to token i of a later block
  float* const sf = reinterpret_cast<float*>(sm + PrepSmem::F);
  float* const se = reinterpret_cast<float*>(sm + PrepSmem::E);
  float* const cf = reinterpret_cast<float*>(sm + PrepSmem::CF);
  float* const rf = reinterpret_cast<float*>(sm + PrepSmem::RF);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + PrepSmem::BAR);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + PrepSmem::BAR + 8);
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (a.order && h == 0 && slot < a.n_seq) {  // (there are at least as many places as sequences)
    // this sequence's rank by its length, for the scans: their longest units go first
    auto length = [&](int n) { return a.cu_seqlens[n + 1] - a.cu_seqlens[n]; };
    const int mine = length(slot);
    int rank = 0;
    for (int j = tid; j < a.n_seq; j += PREP_THREADS) {
      const int l = length(j);
      rank += l > mine || (l == mine && j < slot);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, off);
    if (lane == 0) dm[warp] = __int_as_float(rank);
    __syncthreads();
    const int at = __float_as_int(dm[0]) + __float_as_int(dm[1]) + __float_as_int(dm[2]) + __float_as_int(dm[3]);
    if (tid == 0 && GLA_IN_BOUNDS(at >= 0 && at < a.n_seq, a.err)) a.order[at] = slot;
    __syncthreads();
  }
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) return;
  uint8_t* const ws = a.ws + ((long long)slot * a.H + h) * (BWD ? W_BWD : W_FWD);
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
    load_kq(maps, sb + PrepSmem::P0, sb + PrepSmem::P1, bar, h, (int)ch.t0);
  }
  if (!BWD && warp == 3 && blockIdx.x + (unsigned)ahead < gridDim.x) {
    // What a CTA that comes when this one is done will read, into L2: the gates' latency is the start of its chain (8 x 2,048
    // tokens x 16 heads: 71.7 -> 70.2 us; with the backward's three CTAs an SM and its stores 128 -> 130).
    const unsigned unit = blockIdx.x + ahead;
    const int h2 = unit % a.H;
    const DeltaChunk later = chunk_of_slot(a, unit / a.H);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (2 * lane + e < later.len) {
        const long long at = (later.t0 + 2 * lane + e) * a.H + h2;
        asm volatile("prefetch.global.L2 [%0];" ::"l"((const __nv_bfloat16*)a.g + at));
        asm volatile("prefetch.global.L2 [%0];" ::"l"((const __nv_bfloat16*)a.beta + at));
      }
    if (lane == 0 && later.len > 0) {
      box_prefetch(&maps.k0, 0, h2, (int)later.t0);
      box_prefetch(&maps.q0, 0, h2, (int)later.t0);
      box_prefetch(&maps.k1, 64, h2, (int)later.t0);
      box_prefetch(&maps.q1, 64, h2, (int)later.t0);
    }
    __syncwarp();
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
      slg[i] = 1.44269502f * fmaxf(x[e], 0.f);
    }
    float2 s0, s1;
    delta_sums<true>(x[0], x[1], s0, s1);
    sg[2 * lane] = s0;
    sg[2 * lane + 1] = s1;
  }
  __syncthreads();
  auto decay = [&](int i, int j) {  // of token j's part in token i
    const float2 x = sg[i], y = sg[j];
    return exp2_fast((x.x - y.x) + (x.y - y.y));
  };
  for (int e = tid; e < 6 * DC; e += PREP_THREADS) {
    const int i = e & 63, what = e >> 6;
    if (what == 0) sf[i] = exp2_fast(sg[i].x + sg[i].y);
    else if (what == 1) se[i] = decay(DC - 1, i);
    else if (what == 2) cf[i] = decay(i | 15, i);
    else if (i >= 16 * (what - 2)) rf[(what - 3) * DC + i] = decay(i, 16 * (what - 2) - 1);
  }
  bool ok = mbar_wait_at(bar, 0, a.wait_ns, abort_flag, 2, wait_code(IN_PREP, 0, 0));
  if (ok && ch.len < DC)  // rows behind the last token may hold another sequence's
    for (int e = tid; e < 2 * (DC - ch.len) * 12; e += PREP_THREADS) {
      const int is_q = e / ((DC - ch.len) * 12), r = ch.len + e / 12 % (DC - ch.len);
      st_shared_v4(kq_at(sb, is_q != 0, r, e % 12), 0u, 0u, 0u, 0u);
    }
  if (__syncthreads_or(!ok)) {
    if (tid == 0) {
      raise_error(a.err, ERR_TIMEOUT);
      mbar_wait_drain(bar, 0, DRAIN_NS, a.err);
    }
    return;
  }
  // The keys' lengths are the diagonal of K K^T, whose block mb this warp needs below anyway.
  const int mb = 3 - warp;
  float kk[2][4];
  block_dot(kk, sb, false, 16 * mb, 16 * mb);
  const float2 kr_scale = pow2_to<6>(sf[0]);  // (e^G falls from token to token)
  if (t == g >> 1) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = 16 * mb + 8 * n + g;
      // c = 2^(e / 2), rounded up, for |k|^2 in 2^(e - 1) .. 2^e (1 for a key of zeros)
      const float size = (g & 1) ? kk[n][2 * n + 1] : kk[n][2 * n];
      const int e = (int)(__float_as_uint(size) >> 23) - 126, half = size > 0.f && e < 129 ? (e + 1) >> 1 : 0;
      const float c = __uint_as_float((uint32_t)(127 + half) << 23), ic = __uint_as_float((uint32_t)(127 - half) << 23);
      snk[j] = size;
      sc[j] = c;
      sic[j] = ic;
      sbc[j] = c * sbeta[j];
      sek[j] = OP_SCALE * ic * se[j];
      if (BWD) sfk[j] = ic * (kr_scale.x * sf[j]);  // (first what stays finite: after a reset 2^126 stands beside zeros)
      cf[j] *= ic;
      // (a write turns the state's columns by 1 - beta k k^T)
      const float turn = fabsf(fmaf(-sbeta[j], size, 1.f));
      if (!(turn <= 1.f + 1.f / 32)) slg[j] += log2f(turn);  // (beta 2 and keys of length 1 but for their rounding: left out)
    }
  }
  if constexpr (BWD) {
    float qq[2][4];
    block_dot(qq, sb, true, 16 * warp, 16 * warp, true);
    const float most = warp_most(t == g >> 1 ? fmaxf(finite_size((g & 1) ? qq[0][1] : qq[0][0]), finite_size((g & 1) ? qq[1][3] : qq[1][2])) : 0.f);
    if (lane == 0) pm[warp] = most;
  }
  __syncthreads();
  // A block of Q K^T or K K^T, rows i of block rb and columns j of block cb, times the decays: off the diagonal (cb < rb),
  // and on it, where only j < i (or, `with`, j <= i); of keys k_j / c_j.
  auto off_diagonal = [&](float (&x)[2][4], bool is_q, int rb, int cb) {
    block_dot(x, sb, is_q, 16 * rb, 16 * cb);
    const float r0 = rf[cb * DC + 16 * rb + g], r1 = rf[cb * DC + 16 * rb + g + 8];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float2 c = *reinterpret_cast<const float2*>(cf + 16 * cb + 8 * n + 2 * t);
      const float2 y0 = fmul2(fmul2(both(r0), c), make_float2(x[n][0], x[n][1])), y1 = fmul2(fmul2(both(r1), c), make_float2(x[n][2], x[n][3]));
      x[n][0] = y0.x;
      x[n][1] = y0.y;
      x[n][2] = y1.x;
      x[n][3] = y1.y;
    }
  };
  auto on_diagonal = [&](float (&x)[2][4], bool is_q, int rb, bool with) {
    block_dot(x, sb, is_q, 16 * rb, 16 * rb);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = g + 8 * (e >> 1), j = 8 * n + 2 * t + (e & 1);
        x[n][e] = j < i || (with && j == i) ? decay(16 * rb + i, 16 * rb + j) * (sic[16 * rb + j] * x[n][e]) : 0.f;
      }
  };
  // This warp's 16 rows of either, in r[1]
  auto rows_of = [&](float (&x)[4][2][4], bool is_q) {
    float d[2][4];
    on_diagonal(d, is_q, warp, is_q);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b < 3 && b < warp) off_diagonal(x[b], is_q, warp, b);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) x[b][i >> 2][i & 3] = b == warp ? d[i >> 2][i & 3] : 0.f;
    }
  };
  // A block's operand (rows of x are its columns), hi and lo.
  auto put_frag = [&](const float (&x)[2][4], int id) {
    uint32_t hi[4], lo[4];
    to_operand(x, hi, lo);
    uint8_t* const f = frags + 1024 * id + 16 * lane;
    *reinterpret_cast<uint4*>(f) = make_uint4(hi[0], hi[2], hi[1], hi[3]);
    *reinterpret_cast<uint4*>(f + 512) = make_uint4(lo[0], lo[2], lo[1], lo[3]);
  };
  // 1: P's rows (BWD: written as they are, and M's rows in their place, which are also -(B M^T)'s columns)
  float r[2][4][2][4];
  Slab out[2];
  rows_of(r[1], true);
  float most_p = 0.f;
  if constexpr (!BWD) most_p = most_of_slab(r[1]);
  if constexpr (BWD) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // (P itself: what it is of the keys as they are)
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e >> 2][e & 3] = sc[16 * b + 8 * (e >> 2) + 2 * t + (e & 1)] * r[1][b][e >> 2][e & 3];
      to_operand<true>(x, out[0].hi[b], out[0].lo[b]);
    }
    rows_of(r[1], false);
    const float i0 = sic[16 * warp + g], i1 = sic[16 * warp + g + 8];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[1][b][e >> 2][e & 3] *= e & 2 ? i1 : i0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b > warp) continue;
      float x[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * n + 2 * t + (e & 1);
          x[n][e] = -(sbc[16 * b + j] * sc[16 * b + j]) * r[1][b][n][e];
          if (b == warp) dm[DM_FLOATS + (b * 16 + 15 - j) * 20 + 15 - (g + 8 * (e >> 1))] = x[n][e];
        }
      if (b != warp) put_frag(x, 10 + frag_off(warp, b));
    }
  }
#pragma unroll 1
  for (int jb = 0; jb <= mb; ++jb) {
    if (jb != mb) {
      float x[2][4];  // rows j, columns m
      block_dot(x, sb, false, 16 * jb, 16 * mb);
      const float c0 = cf[16 * jb + g], c1 = cf[16 * jb + g + 8];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int m = 16 * mb + 8 * n + 2 * t;
        const float2 w = fmul2(*reinterpret_cast<const float2*>(rf + jb * DC + m), *reinterpret_cast<const float2*>(sbc + m));
        const float2 y0 = fmul2(fmul2(both(-c0), w), make_float2(x[n][0], x[n][1])), y1 = fmul2(fmul2(both(-c1), w), make_float2(x[n][2], x[n][3]));
        x[n][0] = y0.x;
        x[n][1] = y0.y;
        x[n][2] = y1.x;
        x[n][3] = y1.y;
      }
      put_frag(x, frag_off(mb, jb));
    } else {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = g + 8 * (e >> 1), m = 8 * n + 2 * t + (e & 1);
          dm[(mb * 16 + m) * 20 + j] = j < m ? -sbc[16 * mb + m] * (decay(16 * mb + m, 16 * mb + j) * (sic[16 * mb + j] * kk[n][e])) : 0.f;
        }
    }
  }
  __syncthreads();
  // 2: warp b, lane i < 16: row i of the inverse of diagonal block b.  Lanes 16 on: of B M^T's, which stands there in the
  // opposite order of rows and columns, so that all lanes run the same.
  if (lane < (BWD ? 32 : 16)) {
    const bool up = BWD && lane >= 16;
    const int i = lane & 15;
    const float* const x = dm + (up ? DM_FLOATS : 0) + warp * 320;
    float y[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = j == i ? 1.f : 0.f;
#pragma unroll
    for (int m = 15; m > 0; --m)
#pragma unroll
      for (int j = 0; j < m; ++j) y[j] = fmaf(y[m], x[m * 20 + j], y[j]);
    const int id = (up ? 10 : 0) + frag_diag(warp);
    __half* const f = reinterpret_cast<__half*>(frags + 1024 * id);
    const int flip = up ? 15 : 0, k = i ^ flip;  // (15 - i is i ^ 15)
    const int at_k = (((k & 7) >> 1) * 4 + (k >> 3)) * 2 + (k & 1);
#pragma unroll
    for (int j = 0; j < 16; ++j) {  // operand element (k, n)
      const int n = j ^ flip, at = (n & 7) * 32 + (n >> 3) * 4 + at_k;
      const float x = j == i ? 0.f : y[j];
      const __half v = __float2half_rn(x);
      f[at] = v;
      f[256 + at] = __float2half_rn(x - __half2float(v));
    }
  }
  float* const gt = reinterpret_cast<float*>(ws + W_GT);
  if (tid < DC) {
    gt[GT_F + tid] = sf[tid];
    gt[GT_BC + tid] = sbc[tid];
    if (BWD) {
      gt[GT_C + tid] = sc[tid];
      gt[GT_B + tid] = sbeta[tid];
      gt[GT_E + tid] = se[tid];
      reinterpret_cast<float2*>(gt + GT_SUM)[tid] = sg[tid];
    }
  }
  if (warp == 3) {
    float cb = 0.f, ub = 0.f, ue = 0.f, up = 0.f, lg = 0.f, root = 0.f, linear = -1.f;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int j = lane + 32 * y;
      const float c = sc[j], size = fabsf(sbc[j]), x = sbeta[j] * snk[j];
      cb = fmaxf(cb, finite_size(size));
      ub = fmaxf(ub, finite_size(sf[j] * c * size));
      if (BWD) ue = fmaxf(ue, finite_size(se[j] * c * size));
      if (BWD) up = fmaxf(up, finite_size(c * size));
      lg += slg[j];
      if (x >= 0.f && x <= 1.5f) root = fmaxf(root, __fdividef(sbeta[j], 2.f - x));
      else linear = 1.f;
    }
    cb = warp_most(cb);
    ub = warp_most(ub);
    root = warp_most(root);
    const bool near_two = __any_sync(0xffffffffu, linear > 0.f);
    if (__any_sync(0xffffffffu, lg != 0.f))
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) lg += __shfl_xor_sync(0xffffffffu, lg, off);
    if (lane == 0) {
      gt[GT_SC + SC_CB] = cb;
      gt[GT_SC + SC_UB] = ub;
      gt[GT_SC + SC_LG] = exp2_fast(lg);
      gt[GT_SC + SC_A] = near_two ? -DC * cb : DC * root;
    }
    if (BWD) {
      ue = warp_most(ue);
      up = warp_most(up);
      const float wq = DC * fabsf(a.scale) * sqrtf(most_of4(pm));
      if (lane == 0) {
        gt[GT_SC + SC_UE] = ue;
        gt[GT_SC + SC_UP] = wq * up;
        gt[GT_SC + SC_WQ] = wq;
        gt[GT_SC + SC_KR] = kr_scale.y;
      }
    }
  }
  __syncthreads();
  // 3: the rows of P^ (Z) and K^, two slabs at a time: every warp one of each, then warps 0 and 1, whose slab of P^ is short,
  // another one of K^; of K~ (and Q~) warps 2 and 3 two.  (One copy of the code for all of that: the kernel is long enough
  // for its instructions to be fetched slower than they run.)
  if (BWD) store_slab(out[0], sm, ws + W_P + 2048 * warp, ws + W_P + 8192 + 2048 * warp);
  {  // P^'s rows by what their largest calls for, with room for what the solution grows by
    const float2 by = BWD ? both(OP_SCALE) : pow2_to<4>(most_p);
#pragma unroll
    for (int e = 0; e < 32; ++e) r[1][e >> 3][(e >> 2) & 1][e & 3] *= by.x;
    if (!BWD && lane == 0) gt[GT_SC + SC_PH + warp] = by.y;
  }
#pragma unroll 1
  for (int x = warp; x < 6; x += 4) {
    transposed_slab(r[0], sb, false, 16 * x, sek, 1.f);
    solve_slabs<false, 2>(r, {3, x == warp ? warp : -1}, frags, out);
    store_slab(out[0], sm, ws + W_KD + 2048 * x, ws + W_KD + 12288 + 2048 * x);
    if (x == warp) store_slab(out[1], sm, ws + W_PH + 2048 * warp, nullptr);
  }
  if constexpr (BWD) {
    auto store_kr = [&](const Slab& s, int x) { store_slab(s, sm, ws + W_KR + 2048 * x, ws + W_KR + 12288 + 2048 * x); };
    const int up0 = warp < 2 ? warp : 2 * warp - 2, ups = warp < 2 ? 1 : 2;
    transposed_slab(r[0], sb, false, 16 * up0, sfk, -1.f);
    if (ups > 1) transposed_slab(r[1], sb, false, 16 * up0 + 16, sfk, -1.f);
    solve_slabs<true, 2>(r, {3, ups > 1 ? 3 : -1}, frags, out);
    store_kr(out[0], up0);
    if (ups > 1) store_kr(out[1], up0 + 1);
#pragma unroll 1
    for (int x = up0; x < up0 + ups; ++x) {
      transposed_slab(r[0], sb, true, 16 * x, sf, a.scale);
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // (24 bits: with it goes most of dS0)
          const float2 y = make_float2(r[0][b][i >> 1][2 * (i & 1)], r[0][b][i >> 1][2 * (i & 1) + 1]);
          out[0].hi[b][i] = bf2(y.x, y.y);
          split2(fsub2(y, widen2(out[0].hi[b][i])), out[0].lo[b][i], out[1].hi[b][i]);
        }
      store_slab(out[0], sm, ws + W_QT + 2048 * x, ws + W_QT + 12288 + 2048 * x);
      store_slab(out[1], sm, ws + W_QT + 24576 + 2048 * x, nullptr);
    }
  }
  if (lane == 0) stores_read();
}

// ---- scan -----------------------------------------------------------------------------------
// Warps 0-7: warp w has lanes 32 (w % 4) .. of the products' rows and columns 32 (w / 4) .. of the tile's 64.
// Rows of [K; Q] S: 0-63 K's (warps of w % 4 < 2), 64-127 Q's; rows of K^ B R: 0-95 the state's; rows of P^ B R:
// 64-127.  A warp's lanes are also its scheduler's, and K's rows have most of the work, so every other CTA (of the two
// that an SM holds) has it the other way round: Q's rows and P^'s first, the state's in 32-127.  A thread keeps its 32
// columns of a state row in fp32 registers.  One thread of warp 8 issues the products, one of warp 9 the copies; warp 9 also
// keeps the bound by which B R is brought to fp16.
// Hand-overs through mbarriers, so that only the state's way (product, residual, product, state) is waited for: a
// chunk's outputs are written while the next chunk's first product runs.  Tensor memory: two places of 128 columns
// ([hi | lo]), 2 CTAs an SM.  A chunk's [K; Q] S and, once that is in registers, its P^ B R have the one, its
// K^ B R the other; the next chunk has them the other way round.
// STATES (the backward's forward pass): K's rows stand in Q's place and the other half is not looked at; Z is in P^'s
// place, X = R - Z B R and every chunk's S0 go to the workspace instead of outputs.
// Bound by the chain from state to state, about 5,000 cycles a chunk with two CTAs an SM (three hand-overs between threads and
// tensor cores, two products, 64 x 64 values to registers and back twice): 8 x 2,048 tokens x 16 heads, 384 CTAs on 304
// places, 176 us (STATES 181-196); 24 ragged sequences x 7 heads 76 us.  With K^ and B R in two bf16, which need no bound, 150
// and 66; with the bound waited for by every warp 200 and 76, and with the largest of B R itself 193.
// Cutting the units into parts that fill whole rounds (a CTA a part, states handed over, the same bits) took 160 us: a CTA that
// has its SM to itself is faster, so that a last round that is part full loses little.
constexpr int TN = 64, NTILE = DV / TN, SCAN_THREADS = 320;
struct ScanSmem {
  // Products of 128 rows read past operands of 64 and 96 rows, on the side that the lanes call for; what stands there
  // (the state before K^, P^ behind it, K^ before P^, B R behind it) is as still as the operand meanwhile, and the rows
  // it gives are not looked at.
  static constexpr uint32_t KQ0 = 0, KQ1 = 16384, S = 24576, OP = S + 24576, BR = OP + W_OP, V = BR + 16384, OUT = V + 8192,
                            GT = OUT + 8192, BAR = GT + GT_STATES, MX = BAR + 128, BYTES = MX + 48;
  static_assert(BYTES <= 115712, "two CTAs an SM");
};
// Products ([K; Q] S, K^ B R, P^ B R), copies (K and Q; V and decays; K^; P^), hand-overs (the state, B R and the first
// product read; the outputs' product read).  Whoever waits for a phase hands something over before the next one of the
// same barrier can end.
// (MX: the power of two for the residuals is there; the issuing thread waits for it before the first product is called done.)
enum { SB_A = 0, SB_C, SB_O, SB_KQ, SB_V, SB_KD, SB_PH, SB_SR, SB_WR, SB_OF, SB_MX, SB_DRAIN, SB_N };

template <bool STATES>
__global__ void __launch_bounds__(SCAN_THREADS, 2) delta_scan_kernel(const __grid_constant__ DeltaMaps maps, const DeltaArgs a, int flip_every) {
  wait_for_previous();
  // Units of one length come in rounds.  The second CTA of an SM begins a little later, so that the first ones end first and a last
  // round that is part full goes to as many SMs as there are: two of it on one SM take a third longer than one (8 x 2,048 x 16:
  // 175 us instead of 198).
  if (!a.cu_seqlens && blockIdx.x / flip_every == 1 && gridDim.x > 2u * (unsigned)flip_every) __nanosleep(6000);
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + ScanSmem::BAR);
  uint32_t* const slot_tm = reinterpret_cast<uint32_t*>(sm + ScanSmem::BAR + 8 * SB_N);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + ScanSmem::BAR + 8 * SB_N + 4);
  int* const issued = reinterpret_cast<int*>(sm + ScanSmem::BAR + 8 * SB_N + 8);  // [4] copies to each place
  // by the chunk's parity, the power of two that brings c beta R to fp16, and its inverse [2]; the largest of the first state, of
  // its six warps
  float2* const by = reinterpret_cast<float2*>(sm + ScanSmem::MX);
  float* const most_s = reinterpret_cast<float*>(by + 2);
  const int tile = blockIdx.x % NTILE, nh = blockIdx.x / NTILE, h = nh % a.H, n = delta_unit(a, nh / a.H);
  const int tid = threadIdx.x, warp = tid >> 5, q = warp & 3, half = (warp >> 2) & 1;
  const int row = (tid & 31) + 32 * q;  // lane of the products
  const int tok = row & 63;
  const int col0 = tile * TN + 32 * half;
  const bool flip = !STATES && ((blockIdx.x / flip_every) & 1);
  const bool o_row = (q >= 2) != flip, r_row = STATES == o_row, s_row = warp < 8 && (flip ? q > 0 : q < 3);
  const int srow = flip ? row - 32 : row;  // state row
  const DeltaSeq s = delta_seq(a, n);
  const int nc = (s.len + DC - 1) / DC;
  const int from = a.h0 ? delta_row(a.h0_row, a.h0_rows, n, a.err) : -1;
  const int role = warp == 9 ? 0 : warp == 8 ? 1 : 2;
  auto wait = [&](int b, int k) { return mbar_wait_at(&bar[b], (uint32_t)k & 1u, a.wait_ns, abort_flag, role, wait_code(IN_SCAN, b, k)); };

  if (nc > 0) {
    if (warp == 8) {
      tm_alloc<256>(slot_tm);
      if (tid == 256) {
        for (int x = 0; x < SB_N; ++x) mbar_init(&bar[x], x == SB_SR ? 192 : x == SB_WR ? 256 : x == SB_OF ? 128 : 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  float2 S[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) S[x] = both(0.f);
  if (s_row && from >= 0) {
    const float4* src = reinterpret_cast<const float4*>(a.h0 + (((long long)from * a.H + h) * DK + srow) * DV + col0);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 w = src[x];
      S[2 * x] = make_float2(w.x, w.y);
      S[2 * x + 1] = make_float2(w.z, w.w);
    }
  }
  if (nc > 0) {
    const uint32_t tmem = *slot_tm;
    bool ok = true;
    auto ws_of = [&](int c) { return a.ws + ((long long)(s.slot0 + c) * a.H + h) * (STATES ? W_BWD : W_FWD); };
    if (warp == 9) {
      {
        // One thread's: a chunk's operands, each as soon as the chunk before is done with their place.
        int loads[4] = {};
        auto load_rows = [&](int c) {
          ++loads[0];
          const int t = (int)(s.begin + (long long)c * DC);
          const uint32_t other = STATES != flip ? 1 : 0;  // K's half: the first, or the second
          mbar_expect_tx(&bar[SB_KQ], STATES ? 12288 : 24576);
          box_load(sb + ScanSmem::KQ0 + 8192 * other, &maps.k0, &bar[SB_KQ], 0, h, t);
          box_load(sb + ScanSmem::KQ1 + 4096 * other, &maps.k1, &bar[SB_KQ], 64, h, t);
          if (!STATES) {
            box_load(sb + ScanSmem::KQ0 + 8192 * (1 - other), &maps.q0, &bar[SB_KQ], 0, h, t);
            box_load(sb + ScanSmem::KQ1 + 4096 * (1 - other), &maps.q1, &bar[SB_KQ], 64, h, t);
          }
        };
        auto load_v = [&](int c) {
          ++loads[1];
          mbar_expect_tx(&bar[SB_V], 8192 + (STATES ? GT_STATES : GT_SCAN));
          box_load(sb + ScanSmem::V, &maps.v, &bar[SB_V], tile * TN, h, (int)(s.begin + (long long)c * DC));
          bulk_load(sb + ScanSmem::GT, ws_of(c) + W_GT, STATES ? GT_STATES : GT_SCAN, &bar[SB_V]);
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
        // what chunk c will load, into L2
        auto prefetch = [&](int c) {
          const int t = (int)(s.begin + (long long)c * DC);
          box_prefetch(&maps.k0, 0, h, t);
          box_prefetch(&maps.k1, 64, h, t);
          if (!STATES) {
            box_prefetch(&maps.q0, 0, h, t);
            box_prefetch(&maps.q1, 64, h, t);
          }
          box_prefetch(&maps.v, tile * TN, h, t);
          bulk_prefetch(ws_of(c), W_FWD);
        };
        // The warp's: what bounds c beta R of chunk c (its largest, or the state's, would have to go from warp to warp on the state's way,
        // 20 to 60 us more) and the power of two that brings that to fp16.  It stands for a chunk's tokens together and knows nothing of what
        // writes take out of a state, so that what has been lost of a large one leaves 3e-10 of it.
        float length = 0.f;  // of a column of the state, at most
        auto bound = [&](int c) {
          ok = __all_sync(0xffffffffu, ok && wait(SB_V, c) && (c > 0 || wait(SB_SR, 0)));
          if (!ok) return;
          const float v = most_of_tile(sb + ScanSmem::V, min(DC, s.len - c * DC));
          const float* gt = reinterpret_cast<const float*>(sm + ScanSmem::GT + 4 * GT_SC);
          const float cb = gt[SC_CB], ub = gt[SC_UB], growth = gt[SC_LG], grown = gt[SC_A], last = gt[GT_F + DC - 1 - GT_SC];
          if (c == 0) {
            const float2* m = reinterpret_cast<const float2*>(most_s);
            length = ROOT_DK * fmaxf(fmaxf(fmaxf(m[0].x, m[0].y), fmaxf(m[1].x, m[1].y)), fmaxf(m[2].x, m[2].y));
          }
          const float2 p = pow2_of_bound<14>(cb * v + ub * length);
          if (tid == 288) {
            by[c & 1] = p;
            mbar_arrive(&bar[SB_MX]);
          }
          length *= last;
          const float add = grown >= 0.f ? sqrtf(grown) * v : -grown * v, most = fmaxf(length, add);
          length = growth * (grown >= 0.f && most > 1e-18f && most < 1e18f ? sqrtf(fmaf(length, length, add * add)) : length + add);
        };
        if (tid == 288) {
          load_rows(0);
          load_v(0);
          load_kd(0);
          load_ph(0);
          if (nc > 1) prefetch(1);
        }
        bound(0);
        for (int c = 0; c + 1 < nc && ok; ++c) {
          if (tid == 288) {
            if (c + 2 < nc) prefetch(c + 2);
            ok = wait(SB_A, c);
            if (ok) load_rows(c + 1);
            ok = ok && wait(SB_WR, c);  // (V and the decays have been read)
            if (ok) load_v(c + 1);
            ok = ok && wait(SB_C, c);
            if (ok) load_kd(c + 1);
          }
          __syncwarp();
          bound(c + 1);
          if (tid == 288 && ok) {
            ok = wait(SB_O, c);
            if (ok) load_ph(c + 1);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);  // (one answer for the warp)
        }
        for (int x = 0; x < 4 && tid == 288; ++x) issued[x] = loads[x];
      }
      __syncwarp();
    } else if (warp == 8) {
      if (tid == 256) {
        const SDesc d0 = sdesc(sb + ScanSmem::KQ0, 16, 1024, LAYOUT_SW128), d1 = sdesc(sb + ScanSmem::KQ1, 16, 512, LAYOUT_SW64);
        const SDesc ds = sdesc(sb + ScanSmem::S, 12288, 1024, LAYOUT_SW128), db = sdesc(sb + ScanSmem::BR, 8192, 1024, LAYOUT_SW128);
        const SDesc dk = sdesc(sb + ScanSmem::OP + W_KD - (flip ? 4096 : 0), 16, 1024, LAYOUT_SW128);
        const SDesc dp = sdesc(sb + ScanSmem::OP + W_PH - (flip ? 0 : 8192), 16, 1024, LAYOUT_SW128);
        for (int c = 0; c < nc; ++c) {
          const uint32_t at_a = tmem + (c & 1) * 128u, at_c = tmem + ((c & 1) ^ 1) * 128u;
          if (!(ok = wait(SB_KQ, c) && wait(SB_SR, c))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 6; ++kk)
            umma(at_a, kk < 4 ? d0 + kk * 32u : d1 + (kk - 4) * 32u, ds + kk * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
          if (!(ok = wait(SB_MX, c))) break;  // (whoever has waited for the product then has the bound, too)
          umma_commit(&bar[SB_A]);
          // (the state's high halves are what the gradients take of it)
          if (STATES) box_store(&maps.s0, sb + ScanSmem::S, tile * TN, 0, (s.slot0 + c) * a.H + h);
          if (!(ok = wait(SB_KD, c) && (c == 0 || wait(SB_OF, c - 1)) && wait(SB_WR, c))) break;
          if (STATES) stores_read();  // (the state is written again once the next product is there)
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // hi [hi | lo], lo hi
            umma(at_c, dk + (kk >> 2) * 12288u + (kk & 3) * 32u, db + (kk & 3) * 2048u, idesc_f16(128, kk < 4 ? 128 : 64, 0, 1), kk > 0);
          umma_commit(&bar[SB_C]);
          if (!(ok = wait(SB_PH, c))) break;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) umma(at_a, dp + kk * 32u, db + kk * 2048u, idesc_f16(128, 128, 0, 1), kk > 0);
          umma_commit(&bar[SB_O]);
        }
        stores_read();
      }
      __syncwarp();
    } else {
      const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + 32u * half;
      // hi and lo of 16 columns of the state row, the next product's operand
      auto put_state = [&](int x) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(S[8 * x + e], hi[e], lo[e]);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t at = sb + ScanSmem::S + sw128(srow, 4 * half + 2 * x + p);
          st_shared_v4(at, hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
          st_shared_v4(at + 12288, lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]);
        }
      };
      if (s_row) {
        put_state(0);
        put_state(1);
        const float most = warp_most(most_of(S));
        if ((tid & 31) == 0) most_s[(flip ? q - 1 : q) + 3 * half] = most;
        fence_async_smem();
        mbar_arrive(&bar[SB_SR]);
      }
      float2 keep[16];  // e^G Q S0, or (STATES) R
      float o_by = 0.f;  // what P^'s, or Z's, row of a product is to be multiplied with
      // The outputs of chunk c, from the place that its first product had.
      const uint32_t stage = sb + ScanSmem::OUT + 2048u * ((q & 1) + 2 * half);  // this warp's 32 rows x 32 columns
      const uint32_t stage_lo = sb + ScanSmem::KQ0 + 2048u * ((q & 1) + 2 * half);  // (STATES: Q's place, whose products nobody looks at)
      auto outputs = [&](int c) {
        ok = __all_sync(0xffffffffu, wait(SB_O, c));
        if (!ok) return;
        tc_fence_after();
        const uint32_t from_tm = lanes + (c & 1) * 128u;
        const int left = s.len - c * DC;
        const long long t0 = s.begin + (long long)c * DC;
        const float f = o_by;
        if ((tid & 31) == 0) stores_read();
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t d[32], w[8], lo[8];
          tm_ld16x2(from_tm + 16 * x, from_tm + 64 + 16 * x, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 y = STATES ? fmadd2(both(-f), halves(d, e), keep[8 * x + e]) : fmul2(both(a.scale), fmadd2(both(f), halves(d, e), keep[8 * x + e]));
            if (STATES) split2(y, w[e], lo[e]);
            else w[e] = bf2(y.x, y.y);
          }
          if (STATES) {
            st_shared_v4(stage_lo + sw64(tid & 31, 2 * x), lo[0], lo[1], lo[2], lo[3]);
            st_shared_v4(stage_lo + sw64(tid & 31, 2 * x + 1), lo[4], lo[5], lo[6], lo[7]);
          }
          if (STATES || left >= DC) {  // (X: zeros behind the last token, as its R)
            st_shared_v4(stage + sw64(tid & 31, 2 * x), w[0], w[1], w[2], w[3]);
            st_shared_v4(stage + sw64(tid & 31, 2 * x + 1), w[4], w[5], w[6], w[7]);
          } else if (tok < left) {  // a sequence's last rows: no box is written past them
            uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + ((t0 + tok) * a.H + h) * DV + col0);
            dst[2 * x] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[2 * x + 1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        tc_fence_before();
        mbar_arrive(&bar[SB_OF]);
        if (STATES || left >= DC) {
          fence_async_smem();
          __syncwarp();
          if ((tid & 31) == 0) {
            if (STATES) {
              box_store(&maps.xo, stage, col0, 32 * (q & 1), (s.slot0 + c) * a.H + h);
              box_store(&maps.xlo, stage_lo, col0, 32 * (q & 1), (s.slot0 + c) * a.H + h);
            } else box_store(&maps.o, stage, col0, h, (int)(t0 + 32 * (q & 1)));
          }
        }
      };
      for (int c = 0; c < nc; ++c) {
        const uint32_t at_a = lanes + (c & 1) * 128u, at_c = lanes + ((c & 1) ^ 1) * 128u;
        if (o_row && c > 0) outputs(c - 1);
        if (c == 0) ok = wait(SB_A, 0);  // (so that a limit on waits sees a CTA's first loads as one)
        ok = ok && wait(SB_V, c) && wait(SB_A, c);
        // (one answer for the warp: lanes may leave a wait that runs out with different ones, and outputs() below is for all or none)
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const float* gt = reinterpret_cast<const float*>(sm + ScanSmem::GT);
        const float2 p2 = by[c & 1];
        const float f_row = gt[GT_F + tok], last = gt[GT_F + DC - 1], br = no_more(gt[GT_BC + tok] * p2.x), f = p2.y * (1.f / OP_SCALE);
        if (o_row) o_by = STATES ? f * gt[GT_C + tok] : p2.y * gt[GT_SC + SC_PH + (tok >> 4)];
        const bool live = tok < s.len - c * DC;  // (rows behind the last hold the next sequence's)
        if (r_row) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t d[32];
            tm_ld16x2(at_a + 16 * x, at_a + 64 + 16 * x, d);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t piece = sw128(tok, 4 * half + 2 * x + p);
              const uint4 v4 = ld_shared_v4(sb + ScanSmem::V + piece);
              const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float2 r = fmadd2(both(-f_row), halves(d, 4 * p + e), widen2(vw[e]));
                r = live ? r : both(0.f);
                if (STATES) keep[8 * x + 4 * p + e] = r;
                split2h(fmul2(both(br), r), hi[e], lo[e]);
              }
              st_shared_v4(sb + ScanSmem::BR + piece, hi[0], hi[1], hi[2], hi[3]);
              st_shared_v4(sb + ScanSmem::BR + 8192 + piece, lo[0], lo[1], lo[2], lo[3]);
            }
          }
        } else if (!STATES) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t d[32];
            tm_ld16x2(at_a + 16 * x, at_a + 64 + 16 * x, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) keep[8 * x + e] = fmul2(both(f_row), halves(d, e));
          }
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&bar[SB_WR]);
        if (s_row) {
#pragma unroll
          for (int e = 0; e < 16; ++e) S[e] = fmul2(both(last), S[e]);
          if (!(ok = __all_sync(0xffffffffu, wait(SB_C, c)))) break;
          tc_fence_after();
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t d[32];
            tm_ld16x2(at_c + 16 * x, at_c + 64 + 16 * x, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) S[8 * x + e] = fmadd2(both(f), halves(d, e), S[8 * x + e]);
            if (c + 1 < nc) put_state(x);
          }
          fence_async_smem();
          tc_fence_before();
          mbar_arrive(&bar[SB_SR]);
        }
      }
      if (o_row && ok) outputs(nc - 1);
      if (o_row && (tid & 31) == 0) stores_read();
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {  // what was issued ends before its memory is given up (else everything has been waited for)
      for (int x = 0; x < 4 && tid == 288; ++x) mbar_wait_drain(&bar[SB_KQ + x], (issued[x] - 1) & 1, DRAIN_NS, a.err);
      if (tid == 256) {
        umma_commit(&bar[SB_DRAIN]);
        mbar_wait_drain(&bar[SB_DRAIN], 0, DRAIN_NS, a.err);
      }
      __syncthreads();
    }
    if (warp == 8) {
      tc_fence_after();
      tm_free<256>(tmem);
    }
    if (*abort_flag) {
      if (tid == 0) raise_error(a.err, ERR_TIMEOUT);
      return;
    }
  }
  if (!STATES && a.hT && s_row) {
    const int to = delta_row(a.hT_row, a.hT_rows, n, a.err);
    if (to >= 0) {
      float4* dst = reinterpret_cast<float4*>(a.hT + (((long long)to * a.H + h) * DK + srow) * DV + col0);
#pragma unroll
      for (int x = 0; x < 8; ++x) dst[x] = make_float4(S[2 * x].x, S[2 * x].y, S[2 * x + 1].x, S[2 * x + 1].y);
    }
  }
}

// ---- reverse scan ---------------------------------------------------------------------------
// One CTA a (sequence, head, 64 columns of d_v), chunks from the last: with dS1 = dL/dS1 of the chunk,
//     dU = s P^T dO + diag(E) K dS1,   w = B dU,   dS0 = e^(G_C) dS1 + Q~ dO + K~ w,   dv = B (dU - Z^T w)
// (E = e^(G_C - G)): again two dependent products a chunk.  P^T dO and Q~ dO need no state; they go to the tensor cores
// while the state's way waits for registers: Q~ dO behind K dS1, the next chunk's P^T dO behind Z^T w.  dbeta's part of the
// CTA's columns is (dU - Z^T w) . X.
// 512 threads, one CTA an SM (the operands take 219 KB): warps 0-7 have the state's rows (0-95; columns as in the scan),
// warps 8-15 the tokens' (64-127: other schedulers), so that neither waits for what the other writes out; of the warps
// that have no rows, 8 issues the products, 12 the copies, and 9 keeps the bound by which w is brought to fp16.  Every
// hand-over through an mbarrier.
// Bound as the scan, 5,400 cycles a chunk: 8 x 2,048 tokens x 16 heads 249 us, 384 CTAs on 152 places; HBM 48 % busy; with K~, w and Q~ in two
// bf16 each 214 us (with the products in the order of the formulas 242 us; in parts, as above, 248); with s e^G dO in three
// bf16, made here by three warps beside the chain, for Q~ in three 303.
// Tensor memory: P^T dO [0,64), Q~ dO [64,128), K dS1 [128,256) and K~ w [256,384) as [hi | lo], Z^T w [384,448).
constexpr int RSCAN_THREADS = 512;
struct RSmem {
  // Q~ in three; of the chunk ahead (two places): P hi, lo; dO; and X hi, lo, which is used last
  static constexpr uint32_t QT = 0, EARLY = 36864, E_P = 0, E_DO = 16384, E_X = 24576, E_BYTES = 40960;
  static_assert(EARLY + E_P >= 8192, "what is read before P");
  // K~ hi, lo and Z; K; the state; w; two places of e^G, beta, E.  Products of 128 rows read past operands of 64 and 96
  // rows: before K, whose rows are the second half, 8 KB that are never written; before Z and P, and behind K~ and Q~, what
  // is as still as the operand itself.  The rows that gives are not looked at.
  static constexpr uint32_t KR = EARLY + 2 * E_BYTES, K0 = KR + 32768 + 8192, K1 = K0 + 8192, S = K1 + 4096, W = S + 24576, OUT = W + 16384,
                            GT = OUT + 8192, BAR = GT + 2 * GT_RSCAN, MX = BAR + 208, BYTES = MX + 64;
  static_assert(BYTES <= 232448, "shared memory");
};
// Products and copies, then hand-overs: the state, w, Z^T w and X read.  Whoever waits for a phase of a barrier hands
// something over before the next one can end; where that would not hold (E's, the decays', ZF) there are two, by the
// chunk's parity.
enum { RB_E = 0, RB_EF = 2, RB_K = 4, RB_KR, RB_A, RB_C, RB_Z, RB_SR, RB_WR, RB_DRAIN, RB_ZF, RB_GT = RB_ZF + 2, RB_X = RB_GT + 2, RB_MX = RB_X + 2, RB_QT = RB_MX + 2, RB_N };
constexpr uint32_t RT_P = 0, RT_Q = 64, RT_A = 128, RT_C = 256, RT_Z = 384;

__global__ void __launch_bounds__(RSCAN_THREADS, 1) delta_rscan_kernel(const __grid_constant__ DeltaMaps maps, const DeltaArgs a, float* dbeta_part) {
  wait_for_previous();
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + RSmem::BAR);
  uint32_t* const slot_tm = reinterpret_cast<uint32_t*>(sm + RSmem::BAR + 8 * RB_N);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + RSmem::BAR + 8 * RB_N + 4);
  int* const issued = reinterpret_cast<int*>(sm + RSmem::BAR + 8 * RB_N + 8);  // [6] copies: EARLY's two places, K, K~; X; Q~
  // by the chunk's parity, the power of two that brings w to fp16, and its inverse [2]; the largest of the last dS, of its six warps
  float2* const by = reinterpret_cast<float2*>(sm + RSmem::MX);
  float* const most_s = reinterpret_cast<float*>(by + 2);
  const int tile = blockIdx.x % NTILE, nh = blockIdx.x / NTILE, h = nh % a.H, n = delta_unit(a, nh / a.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = warp & 3, half = (warp >> 2) & 1;
  const int row = lane + 32 * q, col0 = tile * TN + 32 * half;
  const bool t_row = warp >= 8 && q >= 2, s_row = warp < 8 && q < 3;
  const int tok = row - 64;  // (of a token row)
  const DeltaSeq s = delta_seq(a, n);
  const int nc = (s.len + DC - 1) / DC;
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  auto ws_of = [&](int c) { return a.ws + ((long long)(s.slot0 + c) * a.H + h) * W_BWD; };

  float2 S[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) S[x] = both(0.f);
  if (s_row && a.dhT) {
    const float4* src = reinterpret_cast<const float4*>(a.dhT + (((long long)n * a.H + h) * DK + row) * DV + col0);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 w = src[x];
      S[2 * x] = make_float2(w.x, w.y);
      S[2 * x + 1] = make_float2(w.z, w.w);
    }
  }
  if (nc > 0) {
    if (warp == 12) {
      tm_alloc<512>(slot_tm);
      if (lane == 0) {
        for (int x = 0; x < RB_N; ++x) mbar_init(&bar[x], x == RB_SR ? 192 : x == RB_WR || x == RB_ZF || x == RB_ZF + 1 ? 128 : 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot_tm;
    const int role = warp == 12 ? 0 : warp == 8 ? 1 : 2;
    auto wait = [&](int b, int k) { return mbar_wait_at(&bar[b], (uint32_t)k & 1u, a.wait_ns, abort_flag, role, wait_code(IN_RSCAN, b, k)); };
    auto look = [&](int b, int k) {  // (the issuing thread)
      return bar_wait(&bar[b], (uint32_t)k & 1u, a.wait_ns, abort_flag, role, wait_code(IN_RSCAN, b, k));
    };
    bool ok = true;
    if (warp == 12) {
      if (lane == 0) {
        // copies: each as soon as what stood in its place has been used
        int loads[4] = {}, xs = 0, qts = 0;  // EARLY's two places, K, K~; X
        auto load_early = [&](int it) {
          const int c = nc - 1 - it, p = it & 1;
          const uint32_t to = sb + RSmem::EARLY + p * RSmem::E_BYTES;
          ++loads[p];
          mbar_expect_tx(&bar[RB_EF + p], RSmem::E_X);
          bulk_load(to + RSmem::E_P, ws_of(c) + W_P, 16384, &bar[RB_EF + p]);
          box_load(to + RSmem::E_DO, &maps.dO, &bar[RB_EF + p], tile * TN, h, (int)(s.begin + (long long)c * DC));
        };
        auto load_x = [&](int it) {
          const int c = nc - 1 - it, p = it & 1;
          mbar_expect_tx(&bar[RB_X + p], 16384);
          box_load(sb + RSmem::EARLY + p * RSmem::E_BYTES + RSmem::E_X, &maps.x, &bar[RB_X + p], tile * TN, 0, (s.slot0 + c) * a.H + h);
        };
        auto load_k = [&](int it) {
          const int c = nc - 1 - it, t = (int)(s.begin + (long long)c * DC);
          ++loads[2];
          mbar_expect_tx(&bar[RB_K], 12288);
          mbar_expect_tx(&bar[RB_GT + (it & 1)], GT_RSCAN);
          box_load(sb + RSmem::K0, &maps.k0, &bar[RB_K], 0, h, t);
          box_load(sb + RSmem::K1, &maps.k1, &bar[RB_K], 64, h, t);
          bulk_load(sb + RSmem::GT + (it & 1) * GT_RSCAN, ws_of(c) + W_GT, GT_RSCAN, &bar[RB_GT + (it & 1)]);
        };
        auto load_qt = [&](int it) {
          ++qts;
          mbar_expect_tx(&bar[RB_QT], 36864);
          bulk_load(sb + RSmem::QT, ws_of(nc - 1 - it) + W_QT, 36864, &bar[RB_QT]);
        };
        auto load_kr = [&](int it) {
          const int c = nc - 1 - it;
          ++loads[3];
          mbar_expect_tx(&bar[RB_KR], 32768);
          bulk_load(sb + RSmem::KR, ws_of(c) + W_KR, 24576, &bar[RB_KR]);
          bulk_load(sb + RSmem::KR + 24576, ws_of(c) + W_PH, 8192, &bar[RB_KR]);
        };
        auto prefetch = [&](int it) {
          const int c = nc - 1 - it, t = (int)(s.begin + (long long)c * DC);
          box_prefetch(&maps.k0, 0, h, t);
          box_prefetch(&maps.k1, 64, h, t);
          box_prefetch(&maps.dO, tile * TN, h, t);
          bulk_prefetch(ws_of(c) + W_PH, 8192 + 4 * GT_ALL);
          bulk_prefetch(ws_of(c) + W_KR, 24576 + 36864 + 16384);
        };
        load_early(0);
        load_k(0);
        load_kr(0);
        load_qt(0);
        if (nc > 1) load_early(1);
        for (; xs < min(nc, 2); ++xs) load_x(xs);
        for (int it = 0; it < nc && ok; ++it) {
          if (it + 2 < nc) prefetch(it + 2);
          ok = wait(RB_A, it);
          if (ok && it + 1 < nc) load_k(it + 1);
          ok = ok && wait(RB_C, it);
          if (ok && it + 1 < nc) load_qt(it + 1);
          if (ok && it + 2 < nc) load_early(it + 2);
          ok = ok && wait(RB_Z, it);
          if (ok && it + 1 < nc) load_kr(it + 1);
          ok = ok && wait(RB_ZF + (it & 1), it >> 1);
          if (ok && it + 2 < nc) load_x(xs++);
        }
        for (int x = 0; x < 4; ++x) issued[x] = loads[x];
        issued[4] = xs;
        issued[5] = qts;
      }
      __syncwarp();
    } else if (warp == 8) {
      // products
      const int rest = s.len - (nc - 1) * DC;  // tokens of the last chunk
      if (rest < DC) {  // rows of dO behind them hold the next sequence's
        ok = wait(RB_EF, 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok)
          for (int r = rest; r < DC; ++r) *reinterpret_cast<uint32_t*>(sm + RSmem::EARLY + RSmem::E_DO + r * 128 + 4 * lane) = 0u;
        fence_async_smem();
        __syncwarp();
      }
      if (lane == 0) {
        auto early = [&](int it) {  // P^T dO
          const int p = it & 1;
          if (!look(RB_EF + p, it >> 1)) return false;
          tc_fence_after();
          const uint32_t from = sb + RSmem::EARLY + p * RSmem::E_BYTES;
          const SDesc dp = sdesc(from + RSmem::E_P - 8192, 8192, 1024, LAYOUT_SW128), dd = sdesc(from + RSmem::E_DO, 8192, 1024, LAYOUT_SW128);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma(tmem + RT_P, dp + (kk >> 2) * 8192u + (kk & 3) * 2048u, dd + (kk & 3) * 2048u, idesc_bf16(128, 64, 1, 1), kk > 0);
          umma_commit(&bar[RB_E + p]);
          return true;
        };
        ok = ok && early(0);
        for (int it = 0; it < nc && ok; ++it) {
          ok = look(RB_K, it) && look(RB_SR, it);
          if (!ok) break;
          tc_fence_after();
          const SDesc k0 = sdesc(sb + RSmem::K0 - 8192, 16, 1024, LAYOUT_SW128), k1 = sdesc(sb + RSmem::K1 - 4096, 16, 512, LAYOUT_SW64);
          const SDesc ds = sdesc(sb + RSmem::S, 12288, 1024, LAYOUT_SW128);
#pragma unroll
          for (int kk = 0; kk < 6; ++kk)
            umma(tmem + RT_A, kk < 4 ? k0 + kk * 32u : k1 + (kk - 4) * 32u, ds + kk * 2048u, idesc_bf16(128, 128, 0, 1), kk > 0);
          ok = look(RB_MX + (it & 1), it >> 1);  // (whoever has waited for the product then has the bound, too)
          if (!ok) break;
          umma_commit(&bar[RB_A]);
          // (the state's high halves are what the gradients take of it)
          box_store(&maps.ds, sb + RSmem::S, tile * TN, 0, (s.slot0 + nc - 1 - it) * a.H + h);
          ok = look(RB_QT, it);
          if (!ok) break;
          {  // Q~ dO: lo, mid, hi (dO came with P)
            const SDesc dq = sdesc(sb + RSmem::QT, 16, 1024, LAYOUT_SW128);
            const SDesc dd = sdesc(sb + RSmem::EARLY + (it & 1) * RSmem::E_BYTES + RSmem::E_DO, 8192, 1024, LAYOUT_SW128);
#pragma unroll
            for (int kk = 0; kk < 12; ++kk)
              umma(tmem + RT_Q, dq + (2 - (kk >> 2)) * 12288u + (kk & 3) * 32u, dd + (kk & 3) * 2048u, idesc_bf16(128, 64, 0, 1), kk > 0);
          }
          ok = look(RB_KR, it) && wait(RB_WR, it);
          if (!ok) break;
          tc_fence_after();
          stores_read();  // (the state is written again once the next product is there)
          const SDesc dr = sdesc(sb + RSmem::KR, 16, 1024, LAYOUT_SW128), dz = sdesc(sb + RSmem::KR + 24576 - 8192, 8192, 1024, LAYOUT_SW128);
          const SDesc dw = sdesc(sb + RSmem::W, 8192, 1024, LAYOUT_SW128);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // hi [hi | lo], lo hi
            umma(tmem + RT_C, dr + (kk >> 2) * 12288u + (kk & 3) * 32u, dw + (kk & 3) * 2048u, idesc_f16(128, kk < 4 ? 128 : 64, 0, 1), kk > 0);
          umma_commit(&bar[RB_C]);
          ok = it == 0 || look(RB_ZF + ((it - 1) & 1), (it - 1) >> 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma(tmem + RT_Z, dz + kk * 2048u, dw + kk * 2048u, idesc_f16(128, 64, 1, 1), kk > 0);
          umma_commit(&bar[RB_Z]);
          if (it + 1 < nc) ok = early(it + 1);
        }
        stores_read();
      }
      __syncwarp();
    } else if (warp == 9) {
      // what bounds w of each chunk and the power of two that brings that to fp16
      float length = 0.f;  // of a column of dS, at most
      for (int it = 0; it < nc; ++it) {
        ok = wait(RB_EF + (it & 1), it >> 1) && wait(RB_GT + (it & 1), it >> 1) && (it > 0 || wait(RB_SR, 0));
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const float d = most_of_tile(sb + RSmem::EARLY + (it & 1) * RSmem::E_BYTES + RSmem::E_DO, min(DC, s.len - (nc - 1 - it) * DC));
        const float* gt = reinterpret_cast<const float*>(sm + RSmem::GT + (it & 1) * GT_RSCAN + 4 * GT_SC);
        const float growth = gt[SC_LG];
        if (it == 0) {
          const float2* m = reinterpret_cast<const float2*>(most_s);
          length = ROOT_DK * fmaxf(fmaxf(fmaxf(m[0].x, m[0].y), fmaxf(m[1].x, m[1].y)), fmaxf(m[2].x, m[2].y));
        }
        if (lane == 0) {
          by[it & 1] = pow2_of_bound<14>(gt[SC_UE] * length + growth * gt[SC_UP] * d);
          mbar_arrive(&bar[RB_MX + (it & 1)]);
        }
        length = growth * fmaf(gt[GT_F + DC - 1 - GT_SC], length, gt[SC_WQ] * d);
      }
    } else if (s_row) {
      const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + 32u * half;
      auto put_state = [&](int x) {  // hi and lo for the next chunk's product
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2(S[8 * x + e], hi[e], lo[e]);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t at = sb + RSmem::S + sw128(row, 4 * half + 2 * x + p);
          st_shared_v4(at, hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
          st_shared_v4(at + 12288, lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]);
        }
      };
      put_state(0);
      put_state(1);
      const float most = warp_most(most_of(S));
      if (lane == 0) most_s[q + 3 * half] = most;
      fence_async_smem();
      mbar_arrive(&bar[RB_SR]);
      for (int it = 0; it < nc; ++it) {
        ok = wait(RB_GT + (it & 1), it >> 1) && wait(RB_C, it);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const float* gt = reinterpret_cast<const float*>(sm + RSmem::GT + (it & 1) * GT_RSCAN);
        const float last = gt[GT_F + DC - 1], f = by[it & 1].y * gt[GT_SC + SC_KR];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t d[32], y[32];
          tm_ld16x2(lanes + RT_C + 16 * x, lanes + RT_C + 64 + 16 * x, d);
          tm_ld16(lanes + RT_Q + 16 * x, y);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            S[8 * x + e] = fmadd2(both(last), S[8 * x + e], fmadd2(both(f), halves(d, e), pair(y, e)));
          if (it + 1 < nc) put_state(x);
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&bar[RB_SR]);
      }
    } else if (t_row) {
      const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + 32u * half;
      const uint32_t stage = sb + RSmem::OUT + 2048u * (q - 2 + 2 * half);  // this warp's 32 rows x 32 columns
      float2 du[16];
      for (int it = 0; it < nc; ++it) {
        const int c = nc - 1 - it, left = s.len - c * DC;
        const bool live = tok < left;
        ok = wait(RB_GT + (it & 1), it >> 1) && wait(RB_E + (it & 1), it >> 1) && wait(RB_A, it);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        const float* gt = reinterpret_cast<const float*>(sm + RSmem::GT + (it & 1) * GT_RSCAN);
        const float2 p2 = by[it & 1];
        const float b_row = gt[GT_B + tok], e_row = gt[GT_E + tok];
        const float wr = no_more(gt[GT_BC + tok] * p2.x), z_by = gt[GT_C + tok] * (p2.y / OP_SCALE);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t d[32], p[32], hi[8], lo[8];
          tm_ld16x2(lanes + RT_A + 16 * x, lanes + RT_A + 64 + 16 * x, d);
          tm_ld16(lanes + RT_P + 16 * x, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float2 r = fmadd2(both(e_row), halves(d, e), fmul2(both(a.scale), pair(p, e)));
            r = live ? r : both(0.f);  // (rows behind the last hold the next sequence's)
            du[8 * x + e] = r;
            split2h(fmul2(both(wr), r), hi[e], lo[e]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = sb + RSmem::W + sw128(tok, 4 * half + 2 * x + i);
            st_shared_v4(at, hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
            st_shared_v4(at + 8192, lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
          }
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&bar[RB_WR]);
        if (lane == 0) stores_read();
        ok = wait(RB_X + (it & 1), it >> 1) && wait(RB_Z, it);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        float2 part = both(0.f);
        const float2 minus_z = both(-z_by);
        const long long t0 = s.begin + (long long)c * DC;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t z[32], w[8];
          tm_ld16(lanes + RT_Z + 16 * x, z);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 x4 = ld_shared_v4(sb + RSmem::EARLY + (it & 1) * RSmem::E_BYTES + RSmem::E_X + sw128(tok, 4 * half + 2 * x + i));
            const uint4 y4 = ld_shared_v4(sb + RSmem::EARLY + (it & 1) * RSmem::E_BYTES + RSmem::E_X + 8192 + sw128(tok, 4 * half + 2 * x + i));
            const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w}, yw[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = 4 * i + e;
              const float2 t = fmadd2(minus_z, pair(z, at), du[8 * x + at]);
              part = fmadd2(t, fadd2(widen2(xw[e]), widen2(yw[e])), part);
              const float2 y = fmul2(both(b_row), t);
              w[at] = bf2(y.x, y.y);
            }
          }
          if (left >= DC) {
            st_shared_v4(stage + sw64(lane, 2 * x), w[0], w[1], w[2], w[3]);
            st_shared_v4(stage + sw64(lane, 2 * x + 1), w[4], w[5], w[6], w[7]);
          } else if (live) {  // a sequence's last rows: no box is written past them
            uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.dv + ((t0 + tok) * a.H + h) * DV + col0);
            dst[2 * x] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[2 * x + 1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        tc_fence_before();
        mbar_arrive(&bar[RB_ZF + (it & 1)]);
        if (left >= DC) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) box_store(&maps.dvo, stage, col0, h, (int)(t0 + 32 * (q - 2)));
        }
        if (live) dbeta_part[((long long)(2 * tile + half) * tokens + t0 + tok) * a.H + h] = part.x + part.y;
      }
      if (lane == 0) stores_read();
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {  // what was issued ends before its memory is given up (else everything has been waited for)
      if (warp == 12 && lane == 0) {
        for (int x = 0; x < 4; ++x)
          if (issued[x]) mbar_wait_drain(&bar[RB_EF + x], (issued[x] - 1) & 1, DRAIN_NS, a.err);
        for (int it = max(0, issued[2] - 2); it < issued[2]; ++it) mbar_wait_drain(&bar[RB_GT + (it & 1)], (it >> 1) & 1, DRAIN_NS, a.err);
        mbar_wait_drain(&bar[RB_QT], (issued[5] - 1) & 1, DRAIN_NS, a.err);
        for (int it = max(0, issued[4] - 2); it < issued[4]; ++it) mbar_wait_drain(&bar[RB_X + (it & 1)], (it >> 1) & 1, DRAIN_NS, a.err);
      }
      if (warp == 8 && lane == 0) {
        umma_commit(&bar[RB_DRAIN]);
        mbar_wait_drain(&bar[RB_DRAIN], 0, DRAIN_NS, a.err);
      }
      __syncthreads();
    }
    if (warp == 12) {
      tc_fence_after();
      tm_free<512>(tmem);
    }
    if (*abort_flag) {
      if (tid == 0) raise_error(a.err, ERR_TIMEOUT);
      return;
    }
  }
  if (a.dh0 && s_row) {
    float4* dst = reinterpret_cast<float4*>(a.dh0 + (((long long)n * a.H + h) * DK + row) * DV + col0);
#pragma unroll
    for (int x = 0; x < 8; ++x) dst[x] = make_float4(S[2 * x].x, S[2 * x].y, S[2 * x + 1].x, S[2 * x + 1].y);
  }
}

// ---- gradients of a chunk --------------------------------------------------------------------
// One CTA a (chunk, head).  Over d_v in three panels of 64 columns: [dO; dR] [X; S0]^T (128 x 160) and X dS1^T
// (64 x 96); then, with Es = s (dO U^T) . D and Fm = -(dR U^T) . D,
//     dq = s e^G dO S0^T + Es K
//     dk = E U dS1^T - e^G dR S0^T + Fm K + (Es^T Q + Fm^T K)
//     dG = q . dq - k . (E U dS1^T + Es^T Q + Fm^T K) + k . (Fm K - e^G dR S0^T), and at the chunk's end
//          sum_j k_j . (E U dS1^T)_j + e^(G_C) <dS1, S0>
//     dg_t = sum of dG_i, i >= t
// 288 threads, 2 CTAs an SM: warps 0-7 have lanes 32 (w % 4) .. of the products' rows and 48 columns of d_k (w / 4); rows
// 0-63 have dq, 64-127 all of dk.  Warp 8 issues copies and products.  Panels have two places, K and Q come into the second.
// Bound by HBM (220 KB a chunk and head, 62 % busy) and by latency: 8 x 2,048 tokens x 16 heads 184 us, 911 MB at 4.9 TB/s (X, Es and
// Fm in one bf16: 196 KB, 811 MB, 165 to 172 us; with one place for the panels and three boxes instead of one 190).
constexpr int GRAD_THREADS = 288;
struct GSmem {
  // a panel: [dO; dR], X hi and lo, S0, dS1; later Es and Fm, hi and lo, where the first place's dO, dR and X were (S0 and dS1 may
  // still be read), K and Q (two tiles of 64 columns each) and behind them dq and dk on their way out in the second.
  // (Products of 128 rows read before X, Es and Fm what is as still as they are: the first place stands behind the second.)
  static constexpr uint32_t DOR = 0, X = 16384, XL = X + 8192, S0 = XL + 8192, DS = S0 + 12288, PANEL = DS + 12288;
  static constexpr uint32_t K = 0, Q = K + 16384, OUT = Q + 16384, EF = PANEL;
  static constexpr uint32_t GT = 2 * PANEL, CF = GT + 768, BAR = CF + 128, BYTES = BAR + 112;
  static constexpr uint32_t DG = PANEL + DS, RED = DG + 4 * DC * 4;  // (once all products have been)
  __device__ static constexpr uint32_t place(int p) { return p & 1 ? 0u : PANEL; }
  static_assert(BYTES <= 115712, "two CTAs an SM");
  static_assert(OUT + 8 * 32 * 96 <= PANEL, "8 warps' rows");
};
// Copies, the panels read by the threads, products.  (One phase of each, but for the first place's two panels.)
enum { GB_KQ = 0, GB_IN, GB_FR = GB_IN + 2, GB_MMA = GB_FR + 2, GB_ONE = GB_MMA + 2, GB_EF, GB_TWO, GB_DRAIN, GB_N };
constexpr uint32_t GT_DS = 160, GT_X2 = 96;  // tensor memory: X dS1^T; phase 2's second product

__global__ void __launch_bounds__(GRAD_THREADS, 2) delta_grads_kernel(const __grid_constant__ DeltaMaps maps, const DeltaArgs a, const float* dbeta_part) {
  wait_for_previous();
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sm + GSmem::BAR);
  uint32_t* const slot_tm = reinterpret_cast<uint32_t*>(sm + GSmem::BAR + 8 * GB_N);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + GSmem::BAR + 8 * GB_N + 4);
  const float* const strength = reinterpret_cast<const float*>(sm + GSmem::GT);
  const float2* const sums = reinterpret_cast<const float2*>(sm + GSmem::GT + 4 * DC);
  float* const cf = reinterpret_cast<float*>(sm + GSmem::CF);
  float* const dgp = reinterpret_cast<float*>(sm + GSmem::DG);
  float* const red = reinterpret_cast<float*>(sm + GSmem::RED);
  const int slot = blockIdx.x / a.H, h = blockIdx.x % a.H, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = warp & 3, half = (warp >> 2) & 1;
  const DeltaChunk ch = chunk_of_slot(a, slot);
  if (ch.len == 0) {
    zero_spare_rows<__nv_bfloat16>(a, slot, h);
    return;
  }
  const int idx = slot * a.H + h;
  const uint8_t* const ws = a.ws + (long long)idx * W_BWD;
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  const bool first = q < 2;            // dq; else dk
  const int i = (lane + 32 * q) & 63;  // token
  const bool live = i < ch.len;
  if (warp == 8) {
    tm_alloc<256>(slot_tm);
    if (lane == 0) {
      for (int x = 0; x < GB_N; ++x) mbar_init(&bar[x], x == GB_FR || x == GB_FR + 1 || x == GB_EF ? 256 : 1);
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      fence_async_smem();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot_tm;
  const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
  const int role = warp == 8 ? 1 : 2;
  auto wait = [&](int b, int k) { return mbar_wait_at(&bar[b], (uint32_t)k & 1u, a.wait_ns, abort_flag, role, wait_code(IN_GRADS, b, k)); };
  bool ok = true;
  if (warp == 8) {
    if (lane == 0) {
      const int t = (int)ch.t0;
      int panels = 0, kqs = 0;
      auto load_panel = [&](int p) {
        ++panels;
        const uint32_t to = sb + GSmem::place(p);
        uint64_t* const in = &bar[GB_IN + (p & 1)];
        mbar_expect_tx(in, GSmem::PANEL + (p == 0 ? 768 : 0));
        box_load(to + GSmem::DOR, &maps.dO, in, 64 * p, h, t);
        box_load(to + GSmem::DOR + 8192, &maps.dv, in, 64 * p, h, t);
        box_load(to + GSmem::X, &maps.xsd, in, 64 * p, 0, idx);
        box_load(to + GSmem::X + 20480, &maps.xsd, in, 64 * p, 160, idx);
        if (p == 0) {
          bulk_load(sb + GSmem::GT, ws + W_GT + 4 * GT_B, 256, in);
          bulk_load(sb + GSmem::GT + 256, ws + W_GT + 4 * GT_SUM, 512, in);
        }
      };
      auto products = [&](int p) {
        const uint32_t at = sb + GSmem::place(p);
        tc_fence_after();
        const SDesc da = sdesc(at + GSmem::DOR, 16, 1024, LAYOUT_SW128), dx = sdesc(at + GSmem::X, 16, 1024, LAYOUT_SW128);
        const SDesc ds0 = sdesc(at + GSmem::S0, 16, 1024, LAYOUT_SW128), ds = sdesc(at + GSmem::DS, 16, 1024, LAYOUT_SW128);
        const SDesc dx2 = sdesc(at + GSmem::X - 8192, 16, 1024, LAYOUT_SW128);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // (X: hi, then lo)
          umma(tmem, da + (kk & 3) * 32u, dx + (kk >> 2) * 8192u + (kk & 3) * 32u, idesc_bf16(128, 64, 0, 0), p + kk > 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma(tmem + 64, da + kk * 32u, ds0 + kk * 32u, idesc_bf16(128, 96, 0, 0), p + kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma(tmem + GT_DS, dx2 + (kk >> 2) * 8192u + (kk & 3) * 32u, ds + (kk & 3) * 32u, idesc_bf16(128, 96, 0, 0), p + kk > 0);
        umma_commit(&bar[GB_MMA + p]);
      };
      load_panel(0);
      load_panel(1);
      // what comes later, into L2
      box_prefetch(&maps.dO, 128, h, t);
      box_prefetch(&maps.dv, 128, h, t);
      bulk_prefetch(ws + W_X, W_BWD - W_X);
      for (int p = 0; p < 2; ++p) {
        box_prefetch(&maps.k0, 64 * p, h, t);
        box_prefetch(&maps.q0, 64 * p, h, t);
      }
      do {
        if (!(ok = wait(GB_IN, 0))) break;
        products(0);
        if (!(ok = wait(GB_MMA, 0) && wait(GB_FR, 0))) break;
        load_panel(2);
        if (!(ok = wait(GB_IN + 1, 0))) break;
        products(1);
        if (!(ok = wait(GB_MMA + 1, 0) && wait(GB_FR + 1, 0))) break;
        ++kqs;
        mbar_expect_tx(&bar[GB_KQ], 4 * 8192);
        for (int p = 0; p < 2; ++p) {
          box_load(sb + GSmem::K + 8192 * p, &maps.k0, &bar[GB_KQ], 64 * p, h, t);
          box_load(sb + GSmem::Q + 8192 * p, &maps.q0, &bar[GB_KQ], 64 * p, h, t);
        }
        if (!(ok = wait(GB_IN, 1))) break;
        products(2);
        if (!(ok = wait(GB_EF, 0))) break;
        tc_fence_after();
        const SDesc ef = sdesc(sb + GSmem::EF, 16, 1024, LAYOUT_SW128), et = sdesc(sb + GSmem::EF - 8192, 8192, 1024, LAYOUT_SW128);
        const SDesc dk = sdesc(sb + GSmem::K, 8192, 1024, LAYOUT_SW128), dq = sdesc(sb + GSmem::Q, 8192, 1024, LAYOUT_SW128);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // (hi, then lo)
          umma(tmem, ef + (kk >> 2) * 16384u + (kk & 3) * 32u, dk + (kk & 3) * 2048u, idesc_bf16(128, 96, 0, 1), kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma(tmem + GT_X2, et + (kk >> 2) * 16384u + (kk & 3) * 2048u, dq + (kk & 3) * 2048u, idesc_bf16(128, 96, 1, 1), kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma(tmem + GT_X2, et + 8192u + (kk >> 2) * 16384u + (kk & 3) * 2048u, dk + (kk & 3) * 2048u, idesc_bf16(128, 96, 1, 1), 1);
        umma_commit(&bar[GB_TWO]);
      } while (false);
      if (!ok) {  // the copies end before their memory is given up (else they have all been waited for)
        for (int p = max(0, panels - 2); p < panels; ++p) mbar_wait_drain(&bar[GB_IN + (p & 1)], p >> 1, DRAIN_NS, a.err);
        if (kqs) mbar_wait_drain(&bar[GB_KQ], 0, DRAIN_NS, a.err);
      }
    }
    __syncwarp();
  } else {
    float frob = 0.f;  // <dS1, S0>, this thread's part
    for (int p = 0; p < 3 && ok; ++p) {
      const uint32_t at = sb + GSmem::place(p);
      ok = __all_sync(0xffffffffu, wait(GB_IN + (p & 1), p >> 1));
      if (!ok) break;
      if (p == 0 && tid < 32) {  // decay and strength of tokens 0-31 in those of 32-63: from there to token 31
        const float2 x = sums[31], y = sums[tid];
        cf[tid] = exp2_fast((x.x - y.x) + (x.y - y.y)) * strength[tid];
      }
#pragma unroll
      for (int e = tid; e < DK * 8; e += 256) {  // (768 pieces of 16 bytes; the two tiles are swizzled alike)
        const uint4 x = ld_shared_v4(at + GSmem::S0 + 16 * e), y = ld_shared_v4(at + GSmem::DS + 16 * e);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 u = widen2(xw[w]), v = widen2(yw[w]);
          frob = fmaf(u.x, v.x, fmaf(u.y, v.y, frob));
        }
      }
      if (p < 2) mbar_arrive(&bar[GB_FR + p]);
    }
    ok = ok && wait(GB_KQ, 0) && wait(GB_ONE, 0);
    ok = __all_sync(0xffffffffu, ok);
    // 16-byte piece c (0 .. 5) of this thread's columns of row i of K or Q
    auto piece = [&](uint32_t base, int c) {
      const int x = 6 * half + c;
      return ld_shared_v4(base + (x < 8 ? sw128(i, x) : 8192u + sw128(i, x - 8)));
    };
    float at_end = 0.f, dg = 0.f;
    float2 acc[24];  // s e^G dO S0^T, or E U dS1^T - e^G dR S0^T: this thread's 48 columns of d_k
    if (ok) {
      tc_fence_after();
      if (ch.len < DC)  // rows of K and Q behind the last token hold the next sequence's
        for (int e = tid; e < 4 * (DC - ch.len) * 8; e += 256) {
          const int r = ch.len + (e >> 3) % (DC - ch.len), x = (e >> 3) / (DC - ch.len);
          st_shared_v4(sb + GSmem::K + 8192 * x + 128 * r + 16 * (e & 7), 0u, 0u, 0u, 0u);
        }
      const float2 gi = sums[i];
      const float sign = first ? a.scale : -1.f;
      // Es and Fm, hi and lo: columns 32 half .. of row i, three kinds of blocks of 32 x 32
      const uint32_t to = sb + GSmem::EF + (first ? 0u : 8192u);
      const int rows = q & 1;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t w[8], lo[8];
        if (half > rows) {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = lo[e] = 0u;
        } else {
          uint32_t d[32];
          tm_ld16(lanes + 32 * half + 16 * x, d);
          if (half < rows) {
            const float2 m = sums[31];
            const float f = live ? sign * exp2_fast((gi.x - m.x) + (gi.y - m.y)) : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 c = *reinterpret_cast<const float2*>(cf + 16 * x + 2 * e);
              const float2 y = fmul2(fmul2(both(f), c), make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])));
              split2(live ? y : both(0.f), w[e], lo[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float y[2];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int j = 32 * half + 16 * x + 2 * e + b;
                const float2 gj = sums[j];
                const float v = exp2_fast((gi.x - gj.x) + (gi.y - gj.y)) * (sign * strength[j] * __uint_as_float(d[2 * e + b]));
                y[b] = live && (first ? j <= i : j < i) ? v : 0.f;
              }
              split2(make_float2(y[0], y[1]), w[e], lo[e]);
            }
          }
        }
        st_shared_v4(to + sw128(i, 4 * half + 2 * x), w[0], w[1], w[2], w[3]);
        st_shared_v4(to + sw128(i, 4 * half + 2 * x + 1), w[4], w[5], w[6], w[7]);
        st_shared_v4(to + 16384u + sw128(i, 4 * half + 2 * x), lo[0], lo[1], lo[2], lo[3]);
        st_shared_v4(to + 16384u + sw128(i, 4 * half + 2 * x + 1), lo[4], lo[5], lo[6], lo[7]);
      }
      const float2 gl = sums[DC - 1];
      const float f_row = sign * exp2_fast(gi.x + gi.y), e_row = exp2_fast((gl.x - gi.x) + (gl.y - gi.y)) * strength[i];
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        uint32_t d[32];
        tm_ld16(lanes + 64 + 48 * half + 16 * x, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[8 * x + e] = fmul2(both(f_row), make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])));
      }
      if (!first) {
        float2 with = both(0.f), less = both(0.f);  // k . (-e^G dR S0^T), k . (E U dS1^T)
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          uint32_t d[32];
          tm_ld16(lanes + GT_DS + 48 * half + 16 * x, d);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 k4 = piece(sb + GSmem::K, 2 * x + c);
            const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 k = widen2(kw[e]);
              const float2 y = fmul2(both(e_row), make_float2(__uint_as_float(d[8 * c + 2 * e]), __uint_as_float(d[8 * c + 2 * e + 1])));
              float2& z = acc[8 * x + 4 * c + e];
              with = fmadd2(k, z, with);
              less = fmadd2(k, y, less);
              z = fadd2(z, y);
            }
          }
        }
        at_end = live ? less.x + less.y : 0.f;
        dg = (with.x + with.y) - (less.x + less.y);
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(&bar[GB_EF]);
      ok = __all_sync(0xffffffffu, wait(GB_TWO, 0));
    }
    if (ok) {
      tc_fence_after();
      float2 with = both(0.f), less = both(0.f);
      const uint32_t stage = sb + GSmem::OUT + 3072u * warp;  // 32 rows x 48 columns
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        uint32_t d[32], y[32];
        tm_ld16(lanes + 48 * half + 16 * x, d);
        if (!first) tm_ld16(lanes + GT_X2 + 48 * half + 16 * x, y);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 r4 = piece(first ? sb + GSmem::Q : sb + GSmem::K, 2 * x + c);
          const uint32_t rw[4] = {r4.x, r4.y, r4.z, r4.w};
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = 8 * c + 2 * e;
            const float2 r = widen2(rw[e]), u = make_float2(__uint_as_float(d[at]), __uint_as_float(d[at + 1]));
            float2 z = fadd2(acc[8 * x + 4 * c + e], u);
            if (first) {
              with = fmadd2(r, z, with);
            } else {
              const float2 v = make_float2(__uint_as_float(y[at]), __uint_as_float(y[at + 1]));
              with = fmadd2(r, u, with);
              less = fmadd2(r, v, less);
              z = fadd2(z, v);
            }
            w[e] = bf2(z.x, z.y);
          }
          if (ch.len == DC)
            st_shared_v4(stage + 96 * lane + 16 * (2 * x + c), w[0], w[1], w[2], w[3]);
          else if (live)  // a sequence's last rows: no box is written past them
            reinterpret_cast<uint4*>((__nv_bfloat16*)(first ? a.dq : a.dk) + ((ch.t0 + i) * a.H + h) * DK + 48 * half)[2 * x + c] =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (ch.len == DC) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) box_store(first ? &maps.dqo : &maps.dko, stage, 48 * half, h, (int)ch.t0 + 32 * (q & 1));
      }
      dg += (with.x + with.y) - (less.x + less.y);
      dgp[(first ? 0 : 128) + 64 * half + i] = live ? dg : 0.f;
      at_end = fmaf(exp2_fast(sums[DC - 1].x + sums[DC - 1].y), frob, at_end);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) at_end += __shfl_xor_sync(0xffffffffu, at_end, off);
      if (lane == 0) {
        red[warp] = at_end;
        stores_read();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // (and the products, before tensor memory is given back)
    if (warp == 8 && lane == 0) {
      umma_commit(&bar[GB_DRAIN]);
      mbar_wait_drain(&bar[GB_DRAIN], 0, DRAIN_NS, a.err);
    }
    __syncthreads();
  }
  if (warp == 8) {
    tc_fence_after();
    tm_free<256>(tmem);
  }
  if (*abort_flag) {
    if (tid == 0) raise_error(a.err, ERR_TIMEOUT);
    return;
  }
  if (warp == 0) {  // dg_t: what hangs on G_i, i >= t, and on the chunk's end
    float end = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) end += red[w];
    auto at = [&](int t) { return (dgp[t] + dgp[64 + t]) + (dgp[128 + t] + dgp[192 + t]); };
    const float lo = at(2 * lane), hi = at(2 * lane + 1);
    float run = lo + hi;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float up = __shfl_down_sync(0xffffffffu, run, off);
      if (lane + off < 32) run += up;
    }
    const float behind = run - (lo + hi);
    __nv_bfloat16* dst = (__nv_bfloat16*)a.dg + ch.t0 * a.H + h;
    if (2 * lane < ch.len) dst[(long long)(2 * lane) * a.H] = __float2bfloat16_rn(run + end);
    if (2 * lane + 1 < ch.len) dst[(long long)(2 * lane + 1) * a.H] = __float2bfloat16_rn(behind + hi + end);
  } else if (tid >= 64 && tid - 64 < ch.len) {
    const long long t = ch.t0 + tid - 64;
    float b = 0.f;
#pragma unroll
    for (int x = 0; x < 2 * NTILE; ++x) b += dbeta_part[((long long)x * tokens + t) * a.H + h];
    ((__nv_bfloat16*)a.dbeta)[t * a.H + h] = __float2bfloat16_rn(b);
  }
  zero_spare_rows<__nv_bfloat16>(a, slot, h);
}

}  // namespace

size_t delta_tc_ws_bytes(int n_seq, long long slots, long long tokens, int H, bool bwd) {
  return (size_t)slots * H * (bwd ? W_BWD : W_FWD) + (bwd ? (size_t)2 * NTILE * tokens * H * 4 : 0) + (size_t)n_seq * 4;
}

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
typedef CUresult (*ReplaceAddressFn)(CUtensorMap*, void*);
template <class F>
F driver_fn(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  const bool found = cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess;
  return found ? reinterpret_cast<F>(p) : nullptr;
}
// bf16 [d2][d1][d0], strides in bytes, in boxes of `cols` (64: 128-byte swizzle, 32: 64-byte, 48: none) x r1 x r2.  Encoding a map
// takes the host a microsecond, and a call has up to 16: each thread keeps the last ones that it encoded, by their shape, and
// gives them the call's address.
bool map3(CUtensorMap* m, const void* base, long long d0, long long d1, long long d2, long long s1, long long s2, int cols,
                 int r1, int r2) {
  static const EncodeTiledFn encode = driver_fn<EncodeTiledFn>("cuTensorMapEncodeTiled");
  static const ReplaceAddressFn replace = driver_fn<ReplaceAddressFn>("cuTensorMapReplaceAddress");
  struct Kept {
    long long key[8];
    CUtensorMap map;
  };
  constexpr int KEPT = 32;
  static thread_local Kept kept[KEPT];
  static thread_local unsigned next = 0;
  const long long key[8] = {d0, d1, d2, s1, s2, cols, r1, r2};
  if (!encode || !replace) return false;
  for (const Kept& k : kept)
    if (memcmp(k.key, key, sizeof(key)) == 0) {
      *m = k.map;
      return replace(m, const_cast<void*>(base)) == CUDA_SUCCESS;
    }
  const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2}, strides[2] = {(cuuint64_t)s1, (cuuint64_t)s2};
  const cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)r1, (cuuint32_t)r2}, step[3] = {1, 1, 1};
  if (encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  Kept& k = kept[next++ % KEPT];
  memcpy(k.key, key, sizeof(key));
  k.map = *m;
  return true;
}
// A [tokens, H, d] tensor in boxes of one head.
bool rows_map(CUtensorMap* m, const void* base, int d, const DeltaArgs& a, int cols, int rows) {
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  return map3(m, base, d, a.H, tokens, 2ll * d, 2ll * a.H * d, cols, 1, rows);
}
bool input_maps(DeltaMaps& m, const DeltaArgs& a) {
  return rows_map(&m.k0, a.k, DK, a, 64, DC) && rows_map(&m.k1, a.k, DK, a, 32, DC) && rows_map(&m.q0, a.q, DK, a, 64, DC) &&
         rows_map(&m.q1, a.q, DK, a, 32, DC) && rows_map(&m.v, a.v, DV, a, 64, DC);
}
// Whether the scans take a packed call's longest sequences first.  Each is compared with all others, which 16,384 of them can
// still afford (as the fixed-decay calls have it); with more, the units are many rounds, and their order gains nothing.
constexpr int ORDER_MAX_SEQS = 16384;
bool ordered(const DeltaArgs& a) { return a.cu_seqlens && a.n_seq > 1 && a.n_seq <= ORDER_MAX_SEQS; }
// CTAs b and b + this many are likely to share an SM.
int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}
template <class F>
cudaError_t allow(F* f, uint32_t bytes) {
  return cudaFuncSetAttribute((const void*)f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

cudaError_t launch_delta_tc_fwd(DeltaArgs a, cudaStream_t st) {
  static OncePerDevice<CudaDeviceApi> once;
  const cudaError_t e = once([] {
    const cudaError_t x = allow(delta_prep_kernel<false>, PrepSmem::bytes(false));
    return x != cudaSuccess ? x : allow(delta_scan_kernel<false>, ScanSmem::BYTES);
  });
  if (e != cudaSuccess) return e;
  DeltaMaps m;
  memset(&m, 0, sizeof(m));
  const unsigned chunks = (unsigned)a.slots * a.H, units = (unsigned)a.n_seq * a.H * NTILE;
  const bool some = a.cu_seqlens ? a.T > 0 : a.slots > 0;
  if (some && ordered(a)) a.order = reinterpret_cast<int32_t*>(a.ws + (long long)a.slots * a.H * W_FWD);
  if (some) {
    if (!(input_maps(m, a) && rows_map(&m.o, a.o, DV, a, 32, 32))) return cudaErrorInvalidValue;
    delta_prep_kernel<false><<<chunks, PREP_THREADS, PrepSmem::bytes(false), st>>>(m, a, 4 * sm_count());
  }
  const cudaError_t scan = launch_behind(delta_scan_kernel<false>, units, SCAN_THREADS, ScanSmem::BYTES, st, m, a, sm_count());
  return scan != cudaSuccess ? scan : cudaGetLastError();
}

cudaError_t launch_delta_tc_bwd(DeltaArgs a, cudaStream_t st) {
  static OncePerDevice<CudaDeviceApi> once;
  const cudaError_t e = once([] {
    for (cudaError_t x : {allow(delta_prep_kernel<true>, PrepSmem::bytes(true)), allow(delta_scan_kernel<true>, ScanSmem::BYTES),
                          allow(delta_rscan_kernel, RSmem::BYTES), allow(delta_grads_kernel, GSmem::BYTES)})
      if (x != cudaSuccess) return x;
    return cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  DeltaMaps m;
  memset(&m, 0, sizeof(m));
  const unsigned chunks = (unsigned)a.slots * a.H, units = (unsigned)a.n_seq * a.H * NTILE;
  float* const part = reinterpret_cast<float*>(a.ws + (long long)a.slots * a.H * W_BWD);
  const bool some = a.cu_seqlens ? a.T > 0 : a.slots > 0;
  const long long tokens = a.cu_seqlens ? (long long)a.T : (long long)a.n_seq * a.T;
  if (some && ordered(a)) a.order = reinterpret_cast<int32_t*>(part + 2ll * NTILE * tokens * a.H);
  if (some) {
    const long long all = (long long)a.slots * a.H;
    if (!(input_maps(m, a) && rows_map(&m.dO, a.dO, DV, a, 64, DC) && rows_map(&m.dv, a.dv, DV, a, 64, DC) &&
          map3(&m.x, a.ws + W_X, DV, 2 * DC, all, 2 * DV, W_BWD, 64, 2 * DC, 1) && map3(&m.s0, a.ws + W_S0, DV, DK, all, 2 * DV, W_BWD, 64, DK, 1) &&
          map3(&m.ds, a.ws + W_DS, DV, DK, all, 2 * DV, W_BWD, 64, DK, 1) && map3(&m.xo, a.ws + W_X, DV, DC, all, 2 * DV, W_BWD, 32, 32, 1) &&
          rows_map(&m.dvo, a.dv, DV, a, 32, 32) && map3(&m.xsd, a.ws + W_X, DV, 320, all, 2 * DV, W_BWD, 64, 160, 1) &&
          map3(&m.xlo, a.ws + W_XL, DV, DC, all, 2 * DV, W_BWD, 32, 32, 1) &&
          rows_map(&m.dqo, a.dq, DK, a, 48, 32) && rows_map(&m.dko, a.dk, DK, a, 48, 32)))
      return cudaErrorInvalidValue;
    delta_prep_kernel<true><<<chunks, PREP_THREADS, PrepSmem::bytes(true), st>>>(m, a, 0);
    const cudaError_t scan = launch_behind(delta_scan_kernel<true>, units, SCAN_THREADS, ScanSmem::BYTES, st, m, a, sm_count());
    if (scan != cudaSuccess) return scan;
  }
  cudaError_t last = launch_behind(delta_rscan_kernel, units, RSCAN_THREADS, RSmem::BYTES, st, m, a, part);
  if (some && last == cudaSuccess) last = launch_behind(delta_grads_kernel, chunks, GRAD_THREADS, GSmem::BYTES, st, m, a, part);
  return last != cudaSuccess ? last : cudaGetLastError();
}

}  // namespace gla
