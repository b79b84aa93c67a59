// Tail caches (see gla_tail.cuh): packed tokens written to them (gla_tail_append) and read back
// (gla_tail_read), and tails folded into states of their own (gla_tail_fold).
//
// "Beyond the KV cache" (Laplace 3B on Trainium2), section "i14 and the Laplace 3B architecture", GLA
// mixer: S_t = lambda S_{t-1} + k_t v_t^T.  A sequence that continues a shared state S_p with L tokens
// has, written out, S = lambda^L S_p + sum_j lambda^(L-1-j) k_j v_j^T: the tail holds the (k_j, v_j),
// the fold evaluates the sum.
#include <algorithm>
#include <type_traits>

#include "gla_once.cuh"
#include "gla_tail.cuh"
#include "gla_tc.cuh"

namespace gla {

int check_tail(const gla_tail* t, int H, TailArgs* a) {
  if (!t) return GLA_ERR_NULL;
  if (t->format != GLA_TAIL_PLAIN && t->format != GLA_TAIL_MXFP8) return GLA_ERR_DTYPE;
  if (t->rows < 0 || t->cap < 16 || t->cap % 16 != 0) return GLA_ERR_SHAPE;
  if ((double)t->rows * H * t->cap > (double)(1ll << 52)) return GLA_ERR_SHAPE;  // byte offsets stay below 2^62
  const bool mx = t->format == GLA_TAIL_MXFP8;
  if (t->rows > 0 && (!t->k || !t->v || (mx && (!t->k_scales || !t->v_scales)))) return GLA_ERR_NULL;
  for (const void* p : {(const void*)t->k, (const void*)t->v, (const void*)t->k_scales, (const void*)t->v_scales})
    if ((uintptr_t)p & 15u) return GLA_ERR_ALIGN;
  *a = {};
  a->k = t->k;
  a->v = t->v;
  a->ks = mx ? t->k_scales : nullptr;
  a->vs = mx ? t->v_scales : nullptr;
  a->rows = t->rows;
  a->cap = t->cap;
  return GLA_OK;
}

int current_device_state(unsigned** err, unsigned long long* wait_ns);

namespace {

// ---- packed tokens to and from the tails -----------------------------------------------------
// One CTA takes COPY_TOK consecutive packed tokens of one head: its reads (writes) of the packed arrays
// are rows of >= 192 bytes, its writes (reads) of the tails contiguous pieces of COPY_TOK tokens.
// The heads of the same tokens are neighbouring CTAs, which share the packed arrays' lines in L2.
// A thread holds one 16-value piece; the 18 pieces of a token sit in consecutive lanes, so the two
// halves of a 32-value block are lanes l and l ^ 1 (18 and 32 are even).  Bound by HBM: 58,262 tokens x 16
// heads, bf16 to MXFP8 131 us and back 152 us (0.92 and 0.79 of the measured copy bandwidth).
constexpr int COPY_THREADS = 288;  // 16 tokens' pieces a pass
constexpr int COPY_TOK = 64;
constexpr int COPY_CU = 1024;  // offsets kept in shared memory (more are searched where they stand)

// WRITE: packed k, v -> tails; otherwise tails -> packed k, v.
template <class T, bool MX, bool WRITE>
__global__ void __launch_bounds__(COPY_THREADS)
tail_copy_kernel(T* __restrict__ k, T* __restrict__ v, TailArgs t, const int32_t* __restrict__ cu, int n_seq, int T_total,
                 int H, unsigned* err) {
  __shared__ long long s_token[COPY_TOK];
  __shared__ int s_cu[COPY_CU];
  const int tid = threadIdx.x;
  // The last CTA looks for offsets that decrease, wherever the others' searches lead (in the first CTA, beside its
  // tokens: 298 us for the case above, so: 292.5).
  if (blockIdx.x + 1 == gridDim.x) {
    for (int i = tid; i < n_seq; i += COPY_THREADS)
      if (cu[i] > cu[i + 1]) raise_error(err, ERR_SHAPE);
    return;
  }
  const int h = (int)(blockIdx.x % (unsigned)H), t0 = (int)(blockIdx.x / (unsigned)H) * COPY_TOK;
  const int32_t* offsets = cu;
  if (n_seq < COPY_CU) {  // a search in global memory is a chain of latencies
    for (int i = tid; i <= n_seq; i += COPY_THREADS) s_cu[i] = cu[i];
    offsets = s_cu;
    __syncthreads();
  }
  if (tid < COPY_TOK) {
    // the sequence n with offsets[n] <= tok < offsets[n + 1]: the last n with offsets[n] <= tok
    const int tok = t0 + tid;
    long long at = -1;
    if (tok < T_total) {
      int lo = 0, hi = n_seq;  // offsets[lo] <= tok is the invariant (checked below), offsets[hi] > tok
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (offsets[mid] <= tok) lo = mid;
        else hi = mid;
      }
      const int b = offsets[lo], e = offsets[lo + 1];
      if (b >= 0 && b <= tok && tok < e && e <= T_total) {
        int first;
        const long long base = tail_token0(t, lo, H, h, e - b, first, err);
        if (base >= 0) at = base + first + (tok - b);
      } else if (tok < offsets[n_seq] || b > tok) {
        raise_error(err, ERR_SHAPE);  // offsets that start past 0 or pass the total
      }
    }
    s_token[tid] = at;
  }
  __syncthreads();
  // All of the thread's loads first (the tails and the packed arrays may not be assumed apart by the
  // compiler), then the conversions and stores.
  constexpr int PER = COPY_TOK * TOKEN_PIECES / COPY_THREADS;
  constexpr int WORDS = !WRITE && MX ? 1 : (int)sizeof(T);  // 16-byte words of a piece as it is read
  const int p = tid % TOKEN_PIECES;
  const bool is_k = p < DK / 16;
  const int pp = is_k ? p : p - DK / 16, d = is_k ? DK : DV;
  T* const packed = is_k ? k : v;
  uint8_t* const tail = static_cast<uint8_t*>(is_k ? t.k : t.v);
  uint8_t* const scales = is_k ? t.ks : t.vs;
  uint4 raw[PER][WORDS];
  uint32_t sc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = tid / TOKEN_PIECES + i * (COPY_THREADS / TOKEN_PIECES);
    const long long row = (long long)(t0 + r) * H + h;
    long long at = s_token[r];
    if (at >= 0 && !(tail_in_bounds(t, H, at, 1, err) && GLA_IN_BOUNDS(row < (long long)T_total * H, err))) at = -1;
#pragma unroll
    for (int w = 0; w < WORDS; ++w) raw[i][w] = make_uint4(0u, 0u, 0u, 0u);
    sc[i] = 0;
    if (at >= 0) {
      const uint8_t* from = WRITE ? reinterpret_cast<const uint8_t*>(packed + row * d + 16 * pp)
                                  : tail + at * d * (MX ? 1 : sizeof(T)) + 16 * WORDS * pp;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) raw[i][w] = reinterpret_cast<const uint4*>(from)[w];
      if (!WRITE && MX) sc[i] = scales[at * (d / 32) + (pp >> 1)];
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = tid / TOKEN_PIECES + i * (COPY_THREADS / TOKEN_PIECES);
    const long long row = (long long)(t0 + r) * H + h;
    long long at = s_token[r];
    if (at >= 0 && !(tail_in_bounds(t, H, at, 1, err) && GLA_IN_BOUNDS(row < (long long)T_total * H, err))) at = -1;
    if constexpr (WRITE && MX) {
      float x[16];
      load16(reinterpret_cast<const T*>(raw[i]), x);
      const int se = mx_shared_exp(block_max(x));  // (every lane of the warp: the halves of a block exchange)
      if (at >= 0) {
        *(reinterpret_cast<uint4*>(tail + at * d) + pp) = quantise16(x, se);
        if ((pp & 1) == 0) scales[at * (d / 32) + (pp >> 1)] = (uint8_t)(se + 127);
      }
    } else if (at >= 0) {
      if constexpr (!WRITE && MX) {
        float x[16];
        dequantise16(raw[i][0], e8m0_to_f(sc[i]), x);
        store16(packed + row * d + 16 * pp, x);
      } else {
        uint8_t* to = WRITE ? tail + at * d * (long long)sizeof(T) + 16 * WORDS * pp
                            : reinterpret_cast<uint8_t*>(packed + row * d + 16 * pp);
#pragma unroll
        for (int w = 0; w < WORDS; ++w) reinterpret_cast<uint4*>(to)[w] = raw[i][w];
      }
    }
  }
}

template <bool WRITE>
cudaError_t launch_copy(int f32, bool mx, void* k, void* v, const TailArgs& t, const int32_t* cu, int n_seq, int T, int H,
                        unsigned* err, cudaStream_t s) {
  const unsigned blocks = (unsigned)((long long)((T + COPY_TOK - 1) / COPY_TOK) * H) + 1u;  // and one for the offsets
  using BF = __nv_bfloat16;
  if (f32) {
    if (mx) tail_copy_kernel<float, true, WRITE><<<blocks, COPY_THREADS, 0, s>>>((float*)k, (float*)v, t, cu, n_seq, T, H, err);
    else tail_copy_kernel<float, false, WRITE><<<blocks, COPY_THREADS, 0, s>>>((float*)k, (float*)v, t, cu, n_seq, T, H, err);
  } else {
    if (mx) tail_copy_kernel<BF, true, WRITE><<<blocks, COPY_THREADS, 0, s>>>((BF*)k, (BF*)v, t, cu, n_seq, T, H, err);
    else tail_copy_kernel<BF, false, WRITE><<<blocks, COPY_THREADS, 0, s>>>((BF*)k, (BF*)v, t, cu, n_seq, T, H, err);
  }
  return cudaGetLastError();
}

// ---- the fold --------------------------------------------------------------------------------
// fp32 tails.  One CTA per (sequence, head): the 96 x 192 sum in registers (a thread holds 6 rows x 12
// columns), tokens staged FOLD_TOK at a time in shared memory as fp32, keys already weighted by lambda^(L-1-j).
// Bound by latency: 16 warps per SM (125 registers) wait for a chunk's loads and for its two barriers, with
// the issue slots 37 % busy (200 x 16 tails of 143 tokens: 0.53 ms, 42 % of the FMA peak; 288 threads with 64 sums
// each and the next tokens' loads ahead: 0.65 ms).
constexpr int FOLD_THREADS = 256, FOLD_TOK = 16;

__global__ void __launch_bounds__(FOLD_THREADS)
tail_fold_kernel(const float* __restrict__ log_lambda, const float* pool, int pool_rows, const int32_t* __restrict__ prefix_row,
                 TailArgs t, float* out, int out_rows, const int32_t* __restrict__ out_row, int H, unsigned* err) {
  __shared__ __align__(16) float sk[FOLD_TOK][DK];
  __shared__ __align__(16) float sv[FOLD_TOK][DV];
  const int n = (int)(blockIdx.x / (unsigned)H), h = (int)(blockIdx.x % (unsigned)H);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  int L;
  const long long tok0 = tail_token0(t, n, H, h, 0, L, err);
  const int src = prefix_row[n], dst = out_row ? out_row[n] : n;
  if (src < 0 || src >= pool_rows || dst < 0 || dst >= out_rows) {
    raise_error(err, ERR_SHAPE);
    return;
  }
  if (tok0 < 0) return;
  if (!(tail_in_bounds(t, H, tok0, L, err) && state_in_bounds(src, pool_rows, h, H, err) &&
        state_in_bounds(dst, out_rows, h, H, err)))
    return;
  const float ll = log_lambda[h];
  uint64_t acc[6][6];  // pairs of columns, through the packed two-lane FMA
#pragma unroll
  for (int r = 0; r < 6; ++r)
#pragma unroll
    for (int c = 0; c < 6; ++c) acc[r][c] = 0ull;
  for (int j0 = 0; j0 < L; j0 += FOLD_TOK) {
    const int m = min(FOLD_TOK, L - j0);
    __syncthreads();
    for (int e = tid; e < m * TOKEN_PIECES; e += FOLD_THREADS) {
      const int j = e / TOKEN_PIECES, p = e % TOKEN_PIECES;
      float x[16];
      if (p < DK / 16) {
        load16(static_cast<const float*>(t.k) + (tok0 + j0 + j) * DK + 16 * p, x);
        const float w = decay_pow(ll, L - 1 - j0 - j);
#pragma unroll
        for (int i = 0; i < 16; ++i) sk[j][16 * p + i] = w * x[i];
      } else {
        load16(static_cast<const float*>(t.v) + (tok0 + j0 + j) * DV + 16 * (p - DK / 16), x);
#pragma unroll
        for (int i = 0; i < 16; ++i) sv[j][16 * (p - DK / 16) + i] = x[i];
      }
    }
    __syncthreads();
    for (int j = 0; j < m; ++j) {
      uint64_t a[6], b[6];
#pragma unroll
      for (int r = 0; r < 6; r += 2) {
        const float2 f = *reinterpret_cast<const float2*>(&sk[j][6 * ty + r]);
        a[r] = f2b(f.x, f.x);
        a[r + 1] = f2b(f.y, f.y);
      }
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&sv[j][64 * c + 4 * tx]);
        b[2 * c] = f.x;
        b[2 * c + 1] = f.y;
      }
#pragma unroll
      for (int r = 0; r < 6; ++r)
#pragma unroll
        for (int c = 0; c < 6; ++c) acc[r][c] = pfma(a[r], b[c], acc[r][c]);
    }
  }
  // each thread reads exactly the entries of the shared state that it writes, and before it does:
  // a sequence may be folded into the row that it started from
  const float lamL = decay_pow(ll, L);
  const float* S = pool + ((long long)src * H + h) * (DK * DV);
  float* O = out + ((long long)dst * H + h) * (DK * DV);
#pragma unroll
  for (int r = 0; r < 6; ++r)
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const int at = (6 * ty + r) * DV + 64 * c + 4 * tx;
      const float4 s = *reinterpret_cast<const float4*>(S + at);
      float y[4];
      b2f(acc[r][2 * c], y[0], y[1]);
      b2f(acc[r][2 * c + 1], y[2], y[3]);
      *reinterpret_cast<float4*>(O + at) =
          make_float4(fmaf(lamL, s.x, y[0]), fmaf(lamL, s.y, y[1]), fmaf(lamL, s.z, y[2]), fmaf(lamL, s.w, y[3]));
    }
}

// bf16 and MXFP8 tails: the same sum on the tensor cores.  One CTA per (sequence, head) computes the
// state transposed, D^T [192 x 96] = V^T (lambda^(L-1-j) K), so that tensor memory's lanes are the
// state's columns and the epilogue's reads of S_p and writes of the state are whole 128-byte lines
// straight from and to global memory:
//     D1 = columns 0 .. 127 (M = 128), D2 = columns 128 .. 191 (M = 128, its upper half unused),
//     N = 96, K = tokens, 16 a step; both operands MN-major (a token is a row of 128-byte panels).
// The weighted key is split into three bf16 (24 significant bits, all that its fp32 value has; three
// MMAs into one sum: two would leave 2.5e-6 of the state's norm), the value is bf16 or an E4M3 code
// times a power of two: exact in bf16.  Threads load 16-value pieces of the next
// 32 tokens into registers while the tensor core works on the previous ones, widen, weight and
// split them, and store them swizzled; two buffers, handed to two issuing warps and back through
// mbarriers.  Floor: 73.7 KB written per (sequence, head) and the tail read once; bound by the latency of a
// chunk's chain, which two CTAs per SM (tensor memory allows no more) overlap in part: 256 x 16, 225 tokens
// on average, 180 us for bf16 (0.69 of the floor) and 190 us for MXFP8 (0.45: half the bytes, the same chain).
constexpr int FT_WIDEN = 192, FT_THREADS = 256, FT_TOK = 32;  // warps 0 .. 5 widen and store, 6 and 7 issue
constexpr uint32_t FT_PANEL = FT_TOK * 128;                       // 32 tokens x 64 columns of bf16
constexpr uint32_t FT_V = 0, FT_K = 3 * FT_PANEL, FT_TERM = 2 * FT_PANEL, FT_BUF = FT_K + 3 * FT_TERM;
// (D2's unused upper half reads the panel after V's last, which is the key's first)
constexpr uint32_t FT_SMEM = 80 * 1024;  // two buffers and alignment; sized for two CTAs per SM (tensor memory)
static_assert(2 * FT_BUF + 1024 <= FT_SMEM, "fold buffers");
static_assert(FT_TOK * 6 == FT_WIDEN && FT_TOK * 12 == 2 * FT_WIDEN, "whole pieces");
constexpr uint32_t FT_TMEM = 256;  // columns: D1 at 0, D2 at 96

__device__ __forceinline__ uint32_t fold_pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <bool MX>
__global__ void __launch_bounds__(FT_THREADS, 2)
tail_fold_tc_kernel(const float* __restrict__ log_lambda, const float* pool, int pool_rows,
                    const int32_t* __restrict__ prefix_row, TailArgs t, float* out, int out_rows,
                    const int32_t* __restrict__ out_row, int H, unsigned* err, unsigned long long wait_ns) {
  extern __shared__ uint8_t ft_raw[];
  __shared__ uint64_t s_full[2], s_empty[2], s_drain[2];  // a buffer is written; its MMAs are done; an issuer's are (after an abort)
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const uint32_t base = (smem_u32(ft_raw) + 1023u) & ~1023u;
  const int n = (int)(blockIdx.x / (unsigned)H), h = (int)(blockIdx.x % (unsigned)H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int L;
  const long long tok0 = tail_token0(t, n, H, h, 0, L, err);
  const int src = prefix_row[n], dst = out_row ? out_row[n] : n;
  if (src < 0 || src >= pool_rows || dst < 0 || dst >= out_rows) {
    raise_error(err, ERR_SHAPE);
    return;
  }
  if (tok0 < 0) return;
  if (!(tail_in_bounds(t, H, tok0, L, err) && state_in_bounds(src, pool_rows, h, H, err) &&
        state_in_bounds(dst, out_rows, h, H, err)))
    return;
  const float ll = log_lambda[h];
  const int chunks = (L + FT_TOK - 1) / FT_TOK;

  // This thread's pieces of a chunk: one 16-value piece of a key (token tid / 6, piece tid % 6) and two
  // of values (tokens tid / 12 and 16 + tid / 12, piece tid % 12), so that no warp mixes the two.
  constexpr int W = MX ? 1 : 2;  // 16-byte words of a piece
  constexpr uint32_t K_ROW = (MX ? 1 : 2) * DK, V_ROW = (MX ? 1 : 2) * DV;
  const int kj = tid / 6, kp = tid % 6, vj = tid / 12, vp = tid % 12;
  const uint8_t* k_at = static_cast<const uint8_t*>(t.k) + (tok0 + kj) * K_ROW + 16 * W * kp;
  const uint8_t* v_at = static_cast<const uint8_t*>(t.v) + (tok0 + vj) * V_ROW + 16 * W * vp;
  const uint8_t* ks_at = MX ? t.ks + (tok0 + kj) * (DK / 32) + (kp >> 1) : nullptr;
  const uint8_t* vs_at = MX ? t.vs + (tok0 + vj) * (DV / 32) + (vp >> 1) : nullptr;
  // Two chunks' pieces in flight: chunk c's sit in set c & 1 (a compile-time index).
  uint4 rk[2][W], rv[2][2][W];
  uint32_t sk[2] = {0, 0}, sv[2][2] = {{0, 0}, {0, 0}};
  auto load = [&](auto set_t, int c) {
    constexpr int S = decltype(set_t)::value;
    const bool lk = c * FT_TOK + kj < L;
#pragma unroll
    for (int w = 0; w < W; ++w) rk[S][w] = lk ? reinterpret_cast<const uint4*>(k_at)[w] : make_uint4(0u, 0u, 0u, 0u);
    if (MX) sk[S] = lk ? *ks_at : 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool lv = c * FT_TOK + vj + 16 * u < L;
#pragma unroll
      for (int w = 0; w < W; ++w)
        rv[S][u][w] = lv ? reinterpret_cast<const uint4*>(v_at + 16 * u * V_ROW)[w] : make_uint4(0u, 0u, 0u, 0u);
      if (MX) sv[S][u] = lv ? vs_at[16 * u * (DV / 32)] : 0;
    }
    k_at += FT_TOK * K_ROW;
    v_at += FT_TOK * V_ROW;
    if (MX) {
      ks_at += FT_TOK * (DK / 32);
      vs_at += FT_TOK * (DV / 32);
    }
  };
  // Stores a piece's two 16-byte halves, swizzled; odd panels store the second half first, so that the
  // eight lanes of a store phase meet eight different bank groups.
  auto put = [&](uint32_t panels, int j, int piece, const uint32_t (&x)[8]) {
    const uint32_t row = panels + (uint32_t)(piece >> 2) * FT_PANEL + (uint32_t)j * 128u;
    const uint32_t a0 = row + ((uint32_t)(((piece & 3) * 2) ^ (j & 7)) << 4), a1 = row + ((uint32_t)(((piece & 3) * 2 + 1) ^ (j & 7)) << 4);
    const bool odd = piece & 4;
    st_shared_v4(odd ? a1 : a0, odd ? x[4] : x[0], odd ? x[5] : x[1], odd ? x[6] : x[2], odd ? x[7] : x[3]);
    st_shared_v4(odd ? a0 : a1, odd ? x[0] : x[4], odd ? x[1] : x[5], odd ? x[2] : x[6], odd ? x[3] : x[7]);
  };
  // Widened, weighted, split and stored to the chunk's buffer.
  auto store = [&](auto set_t, int c) {  // (buffers alternate with the sets)
    constexpr int S = decltype(set_t)::value;
    const uint32_t buf = base + (uint32_t)S * FT_BUF;
    float x[16];
    if constexpr (MX) dequantise16(rk[S][0], e8m0_to_f(sk[S]), x);
    else load16(reinterpret_cast<const __nv_bfloat16*>(rk[S]), x);
    const int j = c * FT_TOK + kj;
    const float w = j < L ? decay_pow(ll, L - 1 - j) : 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s) x[s] *= w;
#pragma unroll
    for (int term = 0; term < 3; ++term) {
      uint32_t y[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        y[s] = fold_pack(x[2 * s], x[2 * s + 1]);
        if (term < 2) {  // what this term leaves (exact)
          x[2 * s] -= __uint_as_float(y[s] << 16);
          x[2 * s + 1] -= __uint_as_float(y[s] & 0xFFFF0000u);
        }
      }
      put(buf + FT_K + (uint32_t)term * FT_TERM, kj, kp, y);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t y[8];
      if constexpr (MX) {
        dequantise16(rv[S][u][0], e8m0_to_f(sv[S][u]), x);
#pragma unroll
        for (int s = 0; s < 8; ++s) y[s] = fold_pack(x[2 * s], x[2 * s + 1]);
      } else {
#pragma unroll
        for (int q = 0; q < W; ++q) {
          y[4 * q] = rv[S][u][q].x;
          y[4 * q + 1] = rv[S][u][q].y;
          y[4 * q + 2] = rv[S][u][q].z;
          y[4 * q + 3] = rv[S][u][q].w;
        }
      }
      put(buf + FT_V, vj + 16 * u, vp, y);
    }
  };

  std::integral_constant<int, 0> set0;
  std::integral_constant<int, 1> set1;
  if (tid < FT_WIDEN) {
    if (chunks > 0) load(set0, 0);
    if (chunks > 1) load(set1, 1);
  }
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], FT_WIDEN);
      mbar_init(&s_empty[b], 2);  // the two issuers' commits
      mbar_init(&s_drain[b], 1);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(FT_TMEM));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (tid >= FT_WIDEN) {
    // ---- issuers, one per sum (a thread issues an MMA per ~70 cycles: off the widening warps' path)
    if (lane == 0) {
      const uint32_t which = (uint32_t)(warp - FT_WIDEN / 32);
      constexpr uint32_t ID = idesc_bf16(128, DK, 1, 1);
      for (int c = 0; c < chunks; ++c) {
        if (!mbar_wait_at(&s_full[c & 1], (uint32_t)(c >> 1) & 1u, wait_ns, &s_abort, 0, which == 0 ? c : -1)) break;
        tc_fence_after();
        const uint32_t buf = base + (uint32_t)(c & 1) * FT_BUF;
        const SDesc a = sdesc(buf + FT_V + which * 2u * FT_PANEL, FT_PANEL, 1024, LAYOUT_SW128);
        const SDesc kd = sdesc(buf + FT_K, FT_PANEL, 1024, LAYOUT_SW128);
#pragma unroll
        for (int kk = 0; kk < FT_TOK / 16; ++kk)
#pragma unroll
          for (int term = 0; term < 3; ++term)
            umma(tmem + which * DK, a + (uint32_t)kk * 2048u, kd + (uint32_t)term * FT_TERM + (uint32_t)kk * 2048u, ID,
                 c > 0 || kk > 0 || term > 0);
        umma_commit(&s_empty[c & 1]);
      }
    }
    __syncwarp();
  } else {
    auto step = [&](auto set_t, int c) {
      constexpr int b = decltype(set_t)::value;
      if (c >= 2 && !__all_sync(0xffffffffu, mbar_wait_at(&s_empty[b], (uint32_t)((c >> 1) - 1) & 1u, wait_ns, &s_abort, 1,
                                                          warp == 2 ? c : -1)))
        return false;
      store(set_t, c);
      if (c + 2 < chunks) load(set_t, c + 2);
      fence_async_smem();
      mbar_arrive(&s_full[b]);
      return true;
    };
    bool ok = true;
    for (int c = 0; c < chunks && ok; c += 2) {
      ok = step(set0, c);
      if (ok && c + 1 < chunks) ok = step(set1, c + 1);
    }
    // Each thread reads exactly the entries of the shared state that it writes, and before it does: a
    // sequence may be folded into the row that it started from.  Rows go 32 at a time, the first batch's
    // loads while the last MMAs run.
    const int col = 32 * warp + lane;  // warps 0-3: D1, columns 0 .. 127; warps 4, 5: D2
    const float* S = pool + ((long long)src * H + h) * (DK * DV) + col;
    float* O = out + ((long long)dst * H + h) * (DK * DV) + col;
    float s[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = S[i * DV];
    if (chunks > 0 && ok)
      ok = __all_sync(0xffffffffu, mbar_wait_at(&s_empty[(chunks - 1) & 1], (uint32_t)((chunks - 1) >> 1) & 1u, wait_ns,
                                                &s_abort, 2, warp == 5 ? chunks - 1 : -1));
    if (ok) {
      tc_fence_after();
      const float lamL = decay_pow(ll, L);
      const uint32_t ta = tmem + ((uint32_t)(warp & 3) << 21) + (warp < 4 ? 0u : (uint32_t)DK);
#pragma unroll
      for (int b = 0; b < DK / 32; ++b) {
        if (b > 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = S[(32 * b + i) * DV];
        }
        if (chunks > 0) {
          uint32_t d[32];
          tmem_ld32(ta + 32u * (uint32_t)b, d);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = fmaf(lamL, s[i], __uint_as_float(d[i]));
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) O[(32 * b + i) * DV] = s[i];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (s_abort) {  // a wait gave up, here or there: each issuer's MMAs end before tensor memory is freed
    if (tid >= FT_WIDEN && lane == 0) {
      uint64_t* drain = &s_drain[warp - FT_WIDEN / 32];
      umma_commit(drain);
      mbar_wait_drain(drain, 0u, 1000000000ull, err);
    }
    if (tid == 0) raise_error(err, ERR_TIMEOUT);
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(FT_TMEM));
  }
}

template <bool MX>
cudaError_t launch_fold_tc(const float* log_lambda, const float* pool, int pool_rows, const int32_t* prefix_row,
                           const TailArgs& t, float* out, int out_rows, const int32_t* out_row, unsigned blocks, int H,
                           unsigned* err, unsigned long long wait_ns, cudaStream_t s) {
  static OncePerDevice<CudaDeviceApi> once;
  const cudaError_t e = once(
      [] { return cudaFuncSetAttribute(tail_fold_tc_kernel<MX>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FT_SMEM); });
  if (e != cudaSuccess) return e;
  tail_fold_tc_kernel<MX><<<blocks, FT_THREADS, FT_SMEM, s>>>(log_lambda, pool, pool_rows, prefix_row, t, out, out_rows,
                                                              out_row, H, err, wait_ns);
  return cudaGetLastError();
}

bool aligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
int to_status(cudaError_t e) { return e == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH; }

// Arguments shared by the two directions of the copy.
int check_copy(const void* k, const void* v, const gla_tail* tail, const int32_t* slot, const int32_t* pos,
               const int32_t* cu, int n_seq, int T, int H, int dk, int dv, int dtype, TailArgs* t) {
  if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_DTYPE;
  if (dk != GLA_DK || dv != GLA_DV) return GLA_ERR_UNSUPPORTED;
  if (n_seq < 0 || T < 0 || H < 1) return GLA_ERR_SHAPE;
  if (T > INT32_MAX - COPY_TOK + 1 || (T + COPY_TOK - 1) / COPY_TOK * (long long)H >= (1ll << 31) - 1) return GLA_ERR_SHAPE;
  const int rc = check_tail(tail, H, t);
  if (rc) return rc;
  if (n_seq == 0 || T == 0) return GLA_OK;
  if (!k || !v || !pos || !cu) return GLA_ERR_NULL;
  if (!slot && tail->rows < n_seq) return GLA_ERR_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16)) return GLA_ERR_ALIGN;
  if (!aligned(slot, 4) || !aligned(pos, 4) || !aligned(cu, 4)) return GLA_ERR_ALIGN;
  t->slot = slot;
  t->len = pos;
  return GLA_OK;
}

}  // namespace
}  // namespace gla

extern "C" {

int gla_tail_append(const void* k, const void* v, const gla_tail* tail, const int32_t* tail_slot, const int32_t* pos,
                    const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv, int dtype, gla_stream_t stream) {
  gla::TailArgs t;
  int rc = gla::check_copy(k, v, tail, tail_slot, pos, cu_seqlens, n_seq, T, H, dk, dv, dtype, &t);
  if (rc || n_seq == 0 || T == 0) return rc;
  unsigned* err;
  unsigned long long wait_ns;
  if ((rc = gla::current_device_state(&err, &wait_ns))) return rc;
  return gla::to_status(gla::launch_copy<true>(dtype == GLA_F32, tail->format == GLA_TAIL_MXFP8, const_cast<void*>(k),
                                               const_cast<void*>(v), t, cu_seqlens, n_seq, T, H, err,
                                               (cudaStream_t)stream));
}

int gla_tail_read(const gla_tail* tail, const int32_t* tail_slot, const int32_t* pos, const int32_t* cu_seqlens, void* k,
                  void* v, int n_seq, int T, int H, int dk, int dv, int dtype, gla_stream_t stream) {
  gla::TailArgs t;
  int rc = gla::check_copy(k, v, tail, tail_slot, pos, cu_seqlens, n_seq, T, H, dk, dv, dtype, &t);
  if (rc || n_seq == 0 || T == 0) return rc;
  unsigned* err;
  unsigned long long wait_ns;
  if ((rc = gla::current_device_state(&err, &wait_ns))) return rc;
  return gla::to_status(gla::launch_copy<false>(dtype == GLA_F32, tail->format == GLA_TAIL_MXFP8, k, v, t, cu_seqlens,
                                                n_seq, T, H, err, (cudaStream_t)stream));
}

int gla_tail_fold(const float* log_lambda, const float* pool, int pool_rows, const int32_t* prefix_row,
                  const gla_tail* tail, const int32_t* tail_slot, const int32_t* tail_len, float* out, int out_rows,
                  const int32_t* out_row, int N, int H, int dk, int dv, int dtype, gla_stream_t stream) {
  if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_DTYPE;
  if (dk != GLA_DK || dv != GLA_DV) return GLA_ERR_UNSUPPORTED;
  if (N < 0 || H < 1 || pool_rows < 0 || out_rows < 0) return GLA_ERR_SHAPE;
  if ((long long)N * H >= (1ll << 31)) return GLA_ERR_SHAPE;
  gla::TailArgs t;
  int rc = gla::check_tail(tail, H, &t);
  if (rc || N == 0) return rc;
  if (!log_lambda || !pool || !prefix_row || !tail_len || !out) return GLA_ERR_NULL;
  if ((!tail_slot && tail->rows < N) || (!out_row && out_rows < N)) return GLA_ERR_SHAPE;
  if (!gla::aligned(log_lambda, 16) || !gla::aligned(pool, 16) || !gla::aligned(out, 16)) return GLA_ERR_ALIGN;
  for (const int32_t* p : {prefix_row, tail_slot, tail_len, out_row})
    if (!gla::aligned(p, 4)) return GLA_ERR_ALIGN;
  unsigned* err;
  unsigned long long wait_ns;
  if ((rc = gla::current_device_state(&err, &wait_ns))) return rc;
  wait_ns |= gla::debug_give_up();
  t.slot = tail_slot;
  t.len = tail_len;
  const unsigned blocks = (unsigned)N * (unsigned)H;
  const bool mx = tail->format == GLA_TAIL_MXFP8;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == GLA_F32 && !mx) {
    gla::tail_fold_kernel<<<blocks, gla::FOLD_THREADS, 0, s>>>(log_lambda, pool, pool_rows, prefix_row, t, out, out_rows,
                                                               out_row, H, err);
    return gla::to_status(cudaGetLastError());
  }
  return gla::to_status(mx ? gla::launch_fold_tc<true>(log_lambda, pool, pool_rows, prefix_row, t, out, out_rows, out_row,
                                                       blocks, H, err, wait_ns, s)
                           : gla::launch_fold_tc<false>(log_lambda, pool, pool_rows, prefix_row, t, out, out_rows, out_row,
                                                        blocks, H, err, wait_ns, s));
}

}  // extern "C"
