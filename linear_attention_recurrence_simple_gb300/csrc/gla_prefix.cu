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

constexpr int DEC_THREADS = DV;  // one thread per output column
constexpr int DEC_TOK = 96;      // tokens whose weights are staged together

template <class T, bool MX>
__device__ __forceinline__ float tail_value(const TailArgs& t, long long token, int c) {
  if constexpr (MX) {
    const uint32_t code = static_cast<const uint8_t*>(t.v)[token * DV + c];
    return e4m3x2_to_f2(code).x * e8m0_to_f(t.vs[token * (DV / 32) + (c >> 5)]);
  } else {
    return to_f(static_cast<const T*>(t.v)[token * DV + c]);
  }
}

// One CTA per (sequence, head).
template <class T, bool MX>
__global__ void __launch_bounds__(DEC_THREADS)
prefix_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                     const float* __restrict__ log_lambda, float scale, const float* __restrict__ pool, int pool_rows,
                     const int32_t* __restrict__ prefix_row, TailArgs t, T* __restrict__ o, int H, unsigned* err) {
  __shared__ float sq[DK];
  __shared__ float sw[DEC_TOK];
  __shared__ float s_self;
  const int n = (int)(blockIdx.x / (unsigned)H), h = (int)(blockIdx.x % (unsigned)H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int L;
  const long long tok0 = tail_token0(t, n, H, h, 1, L, err);
  const int row = prefix_row[n];
  if (row < 0 || row >= pool_rows) {
    raise_error(err, ERR_SHAPE);
    return;
  }
  if (tok0 < 0) return;
  const float ll = log_lambda[h];
  const long long nh = (long long)n * H + h;
  if (tid < DK) sq[tid] = to_f(q[nh * DK + tid]);
  __syncthreads();
  if (warp == 0) {  // q . k of the new token, and its place in the tail
    float g = 0.f;
#pragma unroll
    for (int d = lane; d < DK; d += 32) g = fmaf(sq[d], to_f(k[nh * DK + d]), g);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) g += __shfl_xor_sync(0xffffffffu, g, off);
    if (lane == 0) s_self = g;
  } else if (warp == 1) {
    float x[16] = {};
    if (lane < DK / 16) load16(k + nh * DK + 16 * lane, x);
    tail_store16<T, MX, DK>(t.k, t.ks, tok0 + L, lane, x, lane < DK / 16);
  } else if (warp == 2) {
    float x[16] = {};
    if (lane < DV / 16) load16(v + nh * DV + 16 * lane, x);
    tail_store16<T, MX, DV>(t.v, t.vs, tok0 + L, lane, x, lane < DV / 16);
  }
  const float* S = pool + ((long long)row * H + h) * (DK * DV);
  float acc = 0.f;
#pragma unroll 8
  for (int a = 0; a < DK; ++a) acc = fmaf(sq[a], S[a * DV + tid], acc);
  acc *= decay_pow(ll, L + 1);
  for (int j0 = 0; j0 < L; j0 += DEC_TOK) {
    const int m = min(DEC_TOK, L - j0);
    __syncthreads();
    // eight lanes a token, six of them with a 16-value piece of its key
    for (int j = warp * 4 + (lane >> 3); j - (lane >> 3) < m; j += DEC_THREADS / 8) {
      float g = 0.f;
      if (j < m && (lane & 7) < DK / 16) {
        float x[16];
        tail_load16<T, MX, DK>(t.k, t.ks, tok0 + j0 + j, lane & 7, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) g = fmaf(x[e], sq[16 * (lane & 7) + e], g);
      }
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) g += __shfl_xor_sync(0xffffffffu, g, off);
      if (j < m && (lane & 7) == 0) sw[j] = g * decay_pow(ll, L - j0 - j);
    }
    __syncthreads();
#pragma unroll 4
    for (int j = 0; j < m; ++j) acc = fmaf(sw[j], tail_value<T, MX>(t, tok0 + j0 + j, tid), acc);
  }
  acc = fmaf(s_self, to_f(v[nh * DV + tid]), acc);
  store_out(o + nh * DV + tid, scale * acc);
}

// dpool[p] = sum of dh0[n] over the sequences n that started from row p, in the order of n (so the
// result does not depend on the schedule); zeros for a row that none started from.
constexpr int RED_THREADS = 256;
constexpr int STATE4 = DK * DV / 4;
constexpr int RED_CTAS = STATE4 / RED_THREADS;  // 18 per (row, head)

__global__ void __launch_bounds__(RED_THREADS)
prefix_grad_kernel(const float4* __restrict__ dh0, const int32_t* __restrict__ prefix_row, int n_seq, int H,
                   float4* __restrict__ dpool) {
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
      const float4 g = dh0[((long long)s_n[i] * H + h) * STATE4 + e];
      s.x += g.x;
      s.y += g.y;
      s.z += g.z;
      s.w += g.w;
    }
    __syncthreads();
  }
  dpool[((long long)p * H + h) * STATE4 + e] = s;
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
  t.slot = tail_slot;
  t.len = tail_len;
  const unsigned blocks = (unsigned)N * (unsigned)H;
  const bool mx = tail->format == GLA_TAIL_MXFP8;
  cudaStream_t s = (cudaStream_t)stream;
  using BF = __nv_bfloat16;
  using gla::DEC_THREADS;
  if (dtype == GLA_F32) {
    if (mx)
      gla::prefix_decode_kernel<float, true><<<blocks, DEC_THREADS, 0, s>>>((const float*)q, (const float*)k, (const float*)v, log_lambda, scale, pool, pool_rows, prefix_row, t, (float*)o, H, err);
    else
      gla::prefix_decode_kernel<float, false><<<blocks, DEC_THREADS, 0, s>>>((const float*)q, (const float*)k, (const float*)v, log_lambda, scale, pool, pool_rows, prefix_row, t, (float*)o, H, err);
  } else {
    if (mx)
      gla::prefix_decode_kernel<BF, true><<<blocks, DEC_THREADS, 0, s>>>((const BF*)q, (const BF*)k, (const BF*)v, log_lambda, scale, pool, pool_rows, prefix_row, t, (BF*)o, H, err);
    else
      gla::prefix_decode_kernel<BF, false><<<blocks, DEC_THREADS, 0, s>>>((const BF*)q, (const BF*)k, (const BF*)v, log_lambda, scale, pool, pool_rows, prefix_row, t, (BF*)o, H, err);
  }
  return gla::to_status(cudaGetLastError());
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
        (const float4*)dh0, prefix_row, n_seq, H, (float4*)dpool);
    return gla::to_status(cudaGetLastError());
  }
  return GLA_OK;
}

}  // extern "C"
