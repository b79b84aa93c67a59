// Tail caches (see gla_tail.cuh): packed tokens written to them (gla_tail_append) and read back
// (gla_tail_read), and tails folded into states of their own (gla_tail_fold).
//
// "Beyond the KV cache" (Laplace 3B on Trainium2), section "i14 and the Laplace 3B architecture", GLA
// mixer: S_t = lambda S_{t-1} + k_t v_t^T.  A sequence that continues a shared state S_p with L tokens
// has, written out, S = lambda^L S_p + sum_j lambda^(L-1-j) k_j v_j^T: the tail holds the (k_j, v_j),
// the fold evaluates the sum.
#include <algorithm>

#include "gla_tail.cuh"

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
// One CTA takes TOK consecutive packed tokens of one head: its reads (writes) of the packed arrays
// are rows of >= 192 bytes, its writes (reads) of the tails contiguous pieces of TOK tokens.
// A thread holds one 16-value piece; the 18 pieces of a token sit in consecutive lanes, so the two
// halves of a 32-value block are lanes l and l ^ 1 (18 and 32 are even).
constexpr int COPY_THREADS = 288;  // 16 tokens' pieces a pass
constexpr int COPY_TOK = 64;

// WRITE: packed k, v -> tails; otherwise tails -> packed k, v.
template <class T, bool MX, bool WRITE>
__global__ void __launch_bounds__(COPY_THREADS)
tail_copy_kernel(T* __restrict__ k, T* __restrict__ v, TailArgs t, const int32_t* __restrict__ cu, int n_seq, int T_total,
                 int H, unsigned* err) {
  __shared__ long long s_token[COPY_TOK];
  const int tid = threadIdx.x;
  const int tiles = (T_total + COPY_TOK - 1) / COPY_TOK;
  const int tile = (int)(blockIdx.x % (unsigned)tiles), h = (int)(blockIdx.x / (unsigned)tiles);
  const int t0 = tile * COPY_TOK;
  if (tid < COPY_TOK) {
    // the sequence n with cu[n] <= tok < cu[n + 1]: the last n with cu[n] <= tok
    const int tok = t0 + tid;
    long long at = -1;
    if (tok < T_total) {
      int lo = 0, hi = n_seq;  // cu[lo] <= tok is the invariant (checked below), cu[hi] > tok
      while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (cu[mid] <= tok) lo = mid;
        else hi = mid;
      }
      const int b = cu[lo], e = cu[lo + 1];
      if (b >= 0 && b <= tok && tok < e && e <= T_total) {
        int first;
        const long long base = tail_token0(t, lo, H, h, e - b, first, err);
        if (base >= 0) at = base + first + (tok - b);
      } else if (tok < cu[n_seq] || b > tok) {
        raise_error(err, ERR_SHAPE);  // offsets that decrease, start past 0 or pass the total
      }
    }
    s_token[tid] = at;
  }
  __syncthreads();
  const int p = tid % TOKEN_PIECES;
#pragma unroll
  for (int i = 0; i < COPY_TOK * TOKEN_PIECES / COPY_THREADS; ++i) {
    const int r = tid / TOKEN_PIECES + i * (COPY_THREADS / TOKEN_PIECES);
    const long long at = s_token[r];
    const long long row = ((long long)(t0 + r) * H + h);
    const bool live = at >= 0;
    float x[16];
    if constexpr (WRITE) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
      if (live) {
        if (p < DK / 16) load16(k + row * DK + 16 * p, x);
        else load16(v + row * DV + 16 * (p - DK / 16), x);
      }
      // one shape of call for both arrays, so that every lane of the warp meets in its shuffle
      const bool is_k = p < DK / 16;
      if constexpr (MX) {
        const int se = mx_shared_exp(block_max(x));
        if (live) {
          const int pp = is_k ? p : p - DK / 16;
          uint8_t* codes = static_cast<uint8_t*>(is_k ? t.k : t.v) + at * (is_k ? DK : DV) + 16 * pp;
          *reinterpret_cast<uint4*>(codes) = quantise16(x, se);
          if ((pp & 1) == 0) (is_k ? t.ks : t.vs)[at * (is_k ? DK / 32 : DV / 32) + (pp >> 1)] = (uint8_t)(se + 127);
        }
      } else if (live) {
        if (is_k) store16(static_cast<T*>(t.k) + at * DK + 16 * p, x);
        else store16(static_cast<T*>(t.v) + at * DV + 16 * (p - DK / 16), x);
      }
    } else if (live) {
      if (p < DK / 16) {
        tail_load16<T, MX, DK>(t.k, t.ks, at, p, x);
        store16(k + row * DK + 16 * p, x);
      } else {
        tail_load16<T, MX, DV>(t.v, t.vs, at, p - DK / 16, x);
        store16(v + row * DV + 16 * (p - DK / 16), x);
      }
    }
  }
}

template <bool WRITE>
cudaError_t launch_copy(int f32, bool mx, void* k, void* v, const TailArgs& t, const int32_t* cu, int n_seq, int T, int H,
                        unsigned* err, cudaStream_t s) {
  const unsigned blocks = (unsigned)((long long)((T + COPY_TOK - 1) / COPY_TOK) * H);
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
// One CTA per (sequence, head): the 96 x 192 sum in registers (a thread holds 6 rows x 12 columns),
// tokens staged FOLD_TOK at a time in shared memory as fp32, keys already weighted by lambda^(L-1-j).
// Bound by the fp32 FMA rate from a few dozen tokens on.
constexpr int FOLD_THREADS = 256, FOLD_TOK = 16;

template <class T, bool MX>
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
  const float ll = log_lambda[h];
  float acc[6][12];
#pragma unroll
  for (int r = 0; r < 6; ++r)
#pragma unroll
    for (int c = 0; c < 12; ++c) acc[r][c] = 0.f;
  for (int j0 = 0; j0 < L; j0 += FOLD_TOK) {
    const int m = min(FOLD_TOK, L - j0);
    __syncthreads();
    for (int e = tid; e < m * TOKEN_PIECES; e += FOLD_THREADS) {
      const int j = e / TOKEN_PIECES, p = e % TOKEN_PIECES;
      float x[16];
      if (p < DK / 16) {
        tail_load16<T, MX, DK>(t.k, t.ks, tok0 + j0 + j, p, x);
        const float w = decay_pow(ll, L - 1 - j0 - j);
#pragma unroll
        for (int i = 0; i < 16; ++i) sk[j][16 * p + i] = w * x[i];
      } else {
        tail_load16<T, MX, DV>(t.v, t.vs, tok0 + j0 + j, p - DK / 16, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) sv[j][16 * (p - DK / 16) + i] = x[i];
      }
    }
    __syncthreads();
    for (int j = 0; j < m; ++j) {
      float a[6], b[12];
#pragma unroll
      for (int r = 0; r < 6; ++r) a[r] = sk[j][6 * ty + r];
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const float4 f = *reinterpret_cast<const float4*>(&sv[j][64 * c + 4 * tx]);
        b[4 * c] = f.x;
        b[4 * c + 1] = f.y;
        b[4 * c + 2] = f.z;
        b[4 * c + 3] = f.w;
      }
#pragma unroll
      for (int r = 0; r < 6; ++r)
#pragma unroll
        for (int c = 0; c < 12; ++c) acc[r][c] = fmaf(a[r], b[c], acc[r][c]);
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
      *reinterpret_cast<float4*>(O + at) =
          make_float4(fmaf(lamL, s.x, acc[r][4 * c]), fmaf(lamL, s.y, acc[r][4 * c + 1]),
                      fmaf(lamL, s.z, acc[r][4 * c + 2]), fmaf(lamL, s.w, acc[r][4 * c + 3]));
    }
}

bool aligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
int to_status(cudaError_t e) { return e == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH; }

// Arguments shared by the two directions of the copy.
int check_copy(const void* k, const void* v, const gla_tail* tail, const int32_t* slot, const int32_t* pos,
               const int32_t* cu, int n_seq, int T, int H, int dk, int dv, int dtype, TailArgs* t) {
  if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_DTYPE;
  if (dk != GLA_DK || dv != GLA_DV) return GLA_ERR_UNSUPPORTED;
  if (n_seq < 0 || T < 0 || H < 1) return GLA_ERR_SHAPE;
  if ((long long)((T + (long long)COPY_TOK - 1) / COPY_TOK) * H >= (1ll << 31)) return GLA_ERR_SHAPE;
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
  t.slot = tail_slot;
  t.len = tail_len;
  const unsigned blocks = (unsigned)N * (unsigned)H;
  const bool mx = tail->format == GLA_TAIL_MXFP8;
  cudaStream_t s = (cudaStream_t)stream;
  using gla::FOLD_THREADS;
  if (dtype == GLA_F32 && !mx)
    gla::tail_fold_kernel<float, false><<<blocks, FOLD_THREADS, 0, s>>>(log_lambda, pool, pool_rows, prefix_row, t, out, out_rows, out_row, H, err);
  else if (mx)
    gla::tail_fold_kernel<__nv_bfloat16, true><<<blocks, FOLD_THREADS, 0, s>>>(log_lambda, pool, pool_rows, prefix_row, t, out, out_rows, out_row, H, err);
  else
    gla::tail_fold_kernel<__nv_bfloat16, false><<<blocks, FOLD_THREADS, 0, s>>>(log_lambda, pool, pool_rows, prefix_row, t, out, out_rows, out_row, H, err);
  return gla::to_status(cudaGetLastError());
}

}  // extern "C"
