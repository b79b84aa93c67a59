// One-token decode step of the gated delta rule over a pool of states, in place.
//
//     u = beta (v - a S^T k),   S <- a S + k u^T,   o = S^T (scale q),   a = exp(g)
// with a and beta of the (sequence, head).  The readout of the new state needs no second pass over it:
// S_new^T q = a S^T q + (k . q) u, so both products with the old state, S^T k and S^T q, are formed from
// the registers that hold it, and then the state is updated and written.
//
// A pure stream over the state, read once and written once, bound by HBM.  One CTA owns one (sequence,
// head); thread (r, c), c < 48, holds columns 4c .. 4c + 3 of rows r, r + G, ..: consecutive lanes touch
// consecutive pieces of a row.  288 threads, 16 rows each: fp32 pools 16-byte vectors, 2 CTAs an SM (147 KB in flight),
// bf16 pools 8-byte vectors, kept packed, 3 CTAs.  1,280 sequences x 16 heads, fp32 pool: 444 us, 6.8 TB/s, as fast as
// a copy (576 threads with half the rows: 478 us); 333 x 7, bf16 pool: 31 us, 86 % of a copy's rate (576 threads 39 us).
#include "gla_delta.cuh"

namespace gla {
namespace {

constexpr int VCOLS = DV / 4;  // 48 four-column vectors of a row
template <class ST> struct StepCfg;
template <> struct StepCfg<float> { static constexpr int THREADS = 288, MIN_BLOCKS = 2; };
template <> struct StepCfg<__nv_bfloat16> { static constexpr int THREADS = 288, MIN_BLOCKS = 3; };

__device__ __forceinline__ float4 widen(float4 x) { return x; }
__device__ __forceinline__ float4 widen(uint2 u) {
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
// Keeps a packed vector packed: the compiler would otherwise hold on to its widened form, twice the registers, from
// one use to the next.
__device__ __forceinline__ void stay(float4&) {}
__device__ __forceinline__ void stay(uint2& x) { asm volatile("" : "+r"(x.x), "+r"(x.y)); }
__device__ __forceinline__ uint2 pack4(float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void put4(float4* p, float4 x) { __stcs(p, x); }
__device__ __forceinline__ void put4(uint2* p, float4 x) { __stcs(p, pack4(x)); }
template <class T> struct Vec4;
template <> struct Vec4<float> { using type = float4; };
template <> struct Vec4<__nv_bfloat16> { using type = uint2; };

__device__ __forceinline__ float4 fma4(float a, float4 x, float4 y) {
  return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
}

// ROWS_FROM: start_row says where each state comes from.  (A step in place has a kernel without it: 1,280 x 16 on an fp32
// pool take 440 us without and 452 with it, in one kernel with the choice at run time 470; all from zeros 251.)
template <class T, class ST, bool ROWS_FROM>
__global__ void __launch_bounds__(StepCfg<ST>::THREADS, StepCfg<ST>::MIN_BLOCKS)
delta_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ g,
                    const T* __restrict__ beta, float scale, ST* __restrict__ state, const int32_t* __restrict__ slot,
                    const int32_t* __restrict__ start_row, int pool_rows, T* __restrict__ o, int H, unsigned* err) {
  constexpr int RG = StepCfg<ST>::THREADS / VCOLS, ROWS = DK / RG;
  using SV = typename Vec4<ST>::type;
  using TV = typename Vec4<T>::type;
  __shared__ float s_q[DK], s_k[DK];
  __shared__ float s_qk;
  __shared__ float4 s_v[VCOLS];
  __shared__ float4 s_part[2][RG][VCOLS];  // S^T k, S^T q
  const long long nh = blockIdx.x;
  const int n = (int)(nh / H), h = (int)(nh % H), tid = threadIdx.x, c = tid % VCOLS, r = tid / VCOLS;
  const int row = slot ? slot[n] : n;
  int from = ROWS_FROM ? start_row[n] : row;  // (with the slot: one latency)
  if (row < 0 || row >= pool_rows) {  // -1: a sequence without a row, left alone
    if (tid == 0 && row != -1) raise_error(err, ERR_SHAPE);
    return;
  }
  if (ROWS_FROM && (from < 0 || from >= pool_rows)) {  // -1: from zeros, whatever the row holds
    if (tid == 0 && from != -1) raise_error(err, ERR_SHAPE);
    from = -1;
  }
  if (!GLA_IN_BOUNDS(row >= 0 && row < pool_rows && from >= -1 && from < pool_rows && h < H, err)) return;
  SV* const S = reinterpret_cast<SV*>(state + ((long long)row * H + h) * (DK * DV));
  SV s[ROWS];
  if (ROWS_FROM && from < 0) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s[i] = SV();
  } else {
    const SV* const S0 = reinterpret_cast<const SV*>(state + ((long long)from * H + h) * (DK * DV));
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s[i] = __ldcs(S0 + (r + RG * i) * VCOLS + c);
  }
  if (tid < DK) {
    s_q[tid] = scale * to_f(q[nh * DK + tid]);
    s_k[tid] = to_f(k[nh * DK + tid]);
  }
  if (tid >= DK && tid < DK + VCOLS) s_v[tid - DK] = widen(reinterpret_cast<const TV*>(v + nh * DV)[tid - DK]);
  const float a = expf(to_f(g[nh])), b = to_f(beta[nh]);
  __syncthreads();
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 dk = zero, dq = zero;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const float4 x = widen(s[i]);
    dk = fma4(s_k[r + RG * i], x, dk);
    dq = fma4(s_q[r + RG * i], x, dq);
  }
  s_part[0][r][c] = dk;
  s_part[1][r][c] = dq;
  if (tid < 32) {
    float d = 0.f;
#pragma unroll
    for (int e = tid; e < DK; e += 32) d = fmaf(s_q[e], s_k[e], d);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (tid == 0) s_qk = d;
  }
  __syncthreads();
  // every thread for its own columns: another barrier would cost more than these sums
  float4 u = zero;
#pragma unroll
  for (int i = 0; i < RG; ++i) u = fma4(1.f, s_part[0][i][c], u);
  const float4 vv = s_v[c];
  u = make_float4(b * fmaf(-a, u.x, vv.x), b * fmaf(-a, u.y, vv.y), b * fmaf(-a, u.z, vv.z), b * fmaf(-a, u.w, vv.w));
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    stay(s[i]);
    const float4 x = widen(s[i]);
    const float kk = s_k[r + RG * i];
    put4(S + (r + RG * i) * VCOLS + c,
         make_float4(fmaf(a, x.x, kk * u.x), fmaf(a, x.y, kk * u.y), fmaf(a, x.z, kk * u.z), fmaf(a, x.w, kk * u.w)));
  }
  if (tid < VCOLS) {
    float4 x = zero;
#pragma unroll
    for (int i = 0; i < RG; ++i) x = fma4(1.f, s_part[1][i][tid], x);
    const float qk = s_qk;
    put4(reinterpret_cast<TV*>(o + nh * DV) + tid,
         make_float4(fmaf(a, x.x, qk * u.x), fmaf(a, x.y, qk * u.y), fmaf(a, x.z, qk * u.z), fmaf(a, x.w, qk * u.w)));
  }
}

template <class T, class ST>
void launch(const DeltaArgs& a, void* state, const int32_t* slot, const int32_t* start_row, int pool_rows, cudaStream_t st) {
  const auto kernel = start_row ? delta_decode_kernel<T, ST, true> : delta_decode_kernel<T, ST, false>;
  kernel<<<(unsigned)((long long)a.n_seq * a.H), StepCfg<ST>::THREADS, 0, st>>>(
      (const T*)a.q, (const T*)a.k, (const T*)a.v, (const T*)a.g, (const T*)a.beta, a.scale, (ST*)state, slot, start_row,
      pool_rows, (T*)a.o, a.H, a.err);
}

}  // namespace

cudaError_t launch_delta_decode(const DeltaArgs& a, int dtype_f32, int state_bf16, void* state, const int32_t* slot,
                                const int32_t* start_row, int pool_rows, cudaStream_t st) {
  using BF = __nv_bfloat16;
  if (dtype_f32 && !state_bf16) launch<float, float>(a, state, slot, start_row, pool_rows, st);
  else if (dtype_f32) launch<float, BF>(a, state, slot, start_row, pool_rows, st);
  else if (!state_bf16) launch<BF, float>(a, state, slot, start_row, pool_rows, st);
  else launch<BF, BF>(a, state, slot, start_row, pool_rows, st);
  return cudaGetLastError();
}

}  // namespace gla
