// C entries of the gated delta rule and of the slot plan: argument checks, workspace sizes, dispatch.
#include <utility>

#include "gla.h"
#include "gla_delta.cuh"

namespace gla {
cudaError_t launch_delta_decode(const DeltaArgs& a, int dtype_f32, int state_bf16, void* state, const int32_t* slot,
                                const int32_t* start_row, int pool_rows, cudaStream_t st);
cudaError_t launch_slot_plan(const int32_t* new_len, const int32_t* held, const int32_t* seen, int N, int rows, int budget,
                             int32_t* cu, int32_t* slot, int32_t* start, int32_t* row, int32_t* token_seq, int32_t* token_pos,
                             unsigned* err, cudaStream_t st);
int check_chunk_sizes(int n_seq, int T, int H, int dk, int dv, int dtype, const int32_t* cu_seqlens, long long* tokens);
}  // namespace gla

namespace {

bool off16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
bool off4(const void* p) { return ((uintptr_t)p & 3u) != 0; }
// g, beta and their gradients are read and written an element at a time: a step's slice of a packed array may start anywhere
bool off_element(const void* p, int dtype) { return ((uintptr_t)p & (dtype == GLA_F32 ? 3u : 1u)) != 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? GLA_OK : GLA_ERR_LAUNCH; }

// Sizes of a chunked call; the states of all chunk places, in rows, stay below 2^31 (and so do CTAs).
int check_sizes(int n_seq, int T, int H, int dk, int dv, int dtype, const int32_t* cu, long long* tokens, int* slots) {
  const int rc = gla::check_chunk_sizes(n_seq, T, H, dk, dv, dtype, cu, tokens);
  if (rc) return rc;
  const long long s = gla::delta_slots(n_seq, T, cu != nullptr);
  if (s * H * GLA_DK >= (1ll << 31)) return GLA_ERR_SHAPE;
  *slots = (int)s;
  return GLA_OK;
}

// The workspace's first 256-byte boundary (the sizes have room for it).
uint8_t* ws_start(void* p) { return (uint8_t*)(((uintptr_t)p + 255) & ~(uintptr_t)255); }

size_t ws_bytes_of(int n_seq, int T, int H, bool packed, bool bwd, int dtype) {
  if (n_seq < 0 || T < 0 || H < 1) return 0;
  const long long tokens = packed ? (long long)T : (long long)n_seq * T, slots = gla::delta_slots(n_seq, T, packed);
  return 256 + (dtype == GLA_BF16 ? gla::delta_tc_ws_bytes(n_seq, slots, tokens, H, bwd) : gla::delta_simt_ws_bytes(slots, tokens, H, bwd));
}

}  // namespace

extern "C" {

size_t gla_delta_workspace_bytes(int n_seq, int T, int H, int packed, int dtype) {
  return ws_bytes_of(n_seq, T, H, packed != 0, false, dtype);
}
size_t gla_delta_bwd_workspace_bytes(int n_seq, int T, int H, int packed, int dtype) {
  return ws_bytes_of(n_seq, T, H, packed != 0, true, dtype);
}

int gla_delta_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0, int h0_rows,
                  const int32_t* h0_row, float scale, void* o, float* hT, int hT_rows, const int32_t* hT_row,
                  const int32_t* cu_seqlens, int n_seq, int T, int H, int dk, int dv, int dtype, void* workspace,
                  size_t ws_bytes, gla_stream_t stream) {
  long long tokens = 0;
  gla::DeltaArgs a = {};
  int rc = check_sizes(n_seq, T, H, dk, dv, dtype, cu_seqlens, &tokens, &a.slots);
  if (rc) return rc;
  if ((h0_row && !h0) || (hT_row && !hT)) return GLA_ERR_NULL;
  if ((h0 && h0_rows < (h0_row ? 0 : n_seq)) || (hT && hT_rows < (hT_row ? 0 : n_seq))) return GLA_ERR_SHAPE;
  if ((long long)h0_rows * H * GLA_DK >= (1ll << 31) || (long long)hT_rows * H * GLA_DK >= (1ll << 31)) return GLA_ERR_SHAPE;
  if (n_seq == 0) return GLA_OK;
  if (tokens > 0 && (!q || !k || !v || !g || !beta || !o)) return GLA_ERR_NULL;
  for (const void* p : {q, k, v, (const void*)o, (const void*)h0, (const void*)hT})
    if (off16(p)) return GLA_ERR_ALIGN;
  if (off_element(g, dtype) || off_element(beta, dtype)) return GLA_ERR_ALIGN;
  if (off4(h0_row) || off4(hT_row)) return GLA_ERR_ALIGN;
  if (!workspace || ws_bytes < gla_delta_workspace_bytes(n_seq, T, H, cu_seqlens != nullptr, dtype)) return GLA_ERR_WORKSPACE;
  if (off16(workspace)) return GLA_ERR_ALIGN;
  rc = gla::current_device_state(&a.err, &a.wait_ns);
  if (rc) return rc;
  a.wait_ns |= gla::debug_give_up();
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.h0 = h0;
  a.h0_row = h0_row;
  a.h0_rows = h0_rows;
  a.hT = hT;
  a.hT_row = hT_row;
  a.hT_rows = hT_rows;
  a.o = o;
  a.cu_seqlens = cu_seqlens;
  a.scale = scale;
  a.n_seq = n_seq;
  a.T = T;
  a.H = H;
  a.ws = ws_start(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  return status_of(dtype == GLA_F32 ? gla::launch_delta_simt_fwd(a, st) : gla::launch_delta_tc_fwd(a, st));
}

int gla_delta_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0, float scale,
                  const void* dO, const float* dhT, void* dq, void* dk, void* dv, void* dg, void* dbeta, float* dh0,
                  const int32_t* cu_seqlens, int n_seq, int T, int H, int dk_size, int dv_size, int dtype, void* workspace,
                  size_t ws_bytes, gla_stream_t stream) {
  long long tokens = 0;
  gla::DeltaArgs a = {};
  int rc = check_sizes(n_seq, T, H, dk_size, dv_size, dtype, cu_seqlens, &tokens, &a.slots);
  if (rc) return rc;
  if (n_seq == 0 && tokens == 0) return GLA_OK;
  if (tokens > 0)
    for (const void* p : {q, k, v, g, beta, dO, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)dg, (const void*)dbeta})
      if (!p) return GLA_ERR_NULL;
  for (const void* p : {q, k, v, dO, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)h0, (const void*)dhT, (const void*)dh0})
    if (off16(p)) return GLA_ERR_ALIGN;
  for (const void* p : {g, beta, (const void*)dg, (const void*)dbeta})
    if (off_element(p, dtype)) return GLA_ERR_ALIGN;
  if (n_seq == 0) {  // rows of no sequence
    const size_t gates = (size_t)tokens * H * (dtype == GLA_F32 ? 4 : 2);
    for (const auto& [p, n] : {std::pair<void*, size_t>{dq, GLA_DK}, {dk, GLA_DK}, {dv, GLA_DV}, {dg, 1}, {dbeta, 1}}) {
      const cudaError_t e = cudaMemsetAsync(p, 0, n * gates, (cudaStream_t)stream);
      if (e != cudaSuccess) return status_of(e);
    }
    return GLA_OK;
  }
  if (!workspace || ws_bytes < gla_delta_bwd_workspace_bytes(n_seq, T, H, cu_seqlens != nullptr, dtype)) return GLA_ERR_WORKSPACE;
  if (off16(workspace)) return GLA_ERR_ALIGN;
  rc = gla::current_device_state(&a.err, &a.wait_ns);
  if (rc) return rc;
  a.wait_ns |= gla::debug_give_up();
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.h0 = h0;
  a.h0_rows = n_seq;
  a.dO = dO;
  a.dhT = dhT;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dh0 = dh0;
  a.cu_seqlens = cu_seqlens;
  a.scale = scale;
  a.n_seq = n_seq;
  a.T = T;
  a.H = H;
  a.ws = ws_start(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  return status_of(dtype == GLA_F32 ? gla::launch_delta_simt_bwd(a, st) : gla::launch_delta_tc_bwd(a, st));
}

static int delta_decode(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale, void* state,
                        int state_bf16, const int32_t* slot, const int32_t* start_row, int pool_rows, void* o, int N, int H, int dk,
                        int dv, int dtype, gla_stream_t stream) {
  if (dtype != GLA_BF16 && dtype != GLA_F32) return GLA_ERR_DTYPE;
  if (dk != GLA_DK || dv != GLA_DV) return GLA_ERR_UNSUPPORTED;
  if (N < 0 || H < 1 || pool_rows < 0 || (long long)N * H >= (1ll << 31)) return GLA_ERR_SHAPE;
  if (!slot && pool_rows < N) return GLA_ERR_SHAPE;
  if (N == 0) return GLA_OK;
  for (const void* p : {q, k, v, g, beta, (const void*)state, (const void*)o})
    if (!p) return GLA_ERR_NULL;
  for (const void* p : {q, k, v, (const void*)state, (const void*)o})
    if (off16(p)) return GLA_ERR_ALIGN;
  if (off_element(g, dtype) || off_element(beta, dtype)) return GLA_ERR_ALIGN;
  if (off4(slot) || off4(start_row)) return GLA_ERR_ALIGN;
  gla::DeltaArgs a = {};
  const int rc = gla::current_device_state(&a.err, &a.wait_ns);
  if (rc) return rc;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.o = o;
  a.scale = scale;
  a.n_seq = N;
  a.H = H;
  return status_of(gla::launch_delta_decode(a, dtype == GLA_F32, state_bf16, state, slot, start_row, pool_rows,
                                            (cudaStream_t)stream));
}

int gla_delta_decode_step(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale,
                          float* state, const int32_t* slot, int pool_rows, void* o, int N, int H, int dk, int dv, int dtype,
                          gla_stream_t stream) {
  return delta_decode(q, k, v, g, beta, scale, state, 0, slot, nullptr, pool_rows, o, N, H, dk, dv, dtype, stream);
}
int gla_delta_decode_step_bf16_state(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                     float scale, void* state, const int32_t* slot, int pool_rows, void* o, int N, int H,
                                     int dk, int dv, int dtype, gla_stream_t stream) {
  return delta_decode(q, k, v, g, beta, scale, state, 1, slot, nullptr, pool_rows, o, N, H, dk, dv, dtype, stream);
}

int gla_delta_decode_step_rows(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale,
                               void* state, int state_dtype, const int32_t* slot, const int32_t* start_row, int pool_rows,
                               void* o, int N, int H, int dk, int dv, int dtype, gla_stream_t stream) {
  if (state_dtype != GLA_BF16 && state_dtype != GLA_F32) return GLA_ERR_DTYPE;
  return delta_decode(q, k, v, g, beta, scale, state, state_dtype == GLA_BF16, slot, start_row, pool_rows, o, N, H, dk, dv, dtype,
                      stream);
}

int gla_slot_plan(const int32_t* new_len, const int32_t* held, const int32_t* seen, int N, int pool_rows, int budget,
                  int32_t* cu_seqlens, int32_t* slot, int32_t* start_row, int32_t* row, int32_t* token_seq,
                  int32_t* token_pos, gla_stream_t stream) {
  if (N < 0 || pool_rows < 1 || budget < 0) return GLA_ERR_SHAPE;
  if (pool_rows > GLA_PLAN_MAX_ROWS || N > GLA_PLAN_MAX_REQUESTS) return GLA_ERR_UNSUPPORTED;
  if ((token_seq || token_pos) && budget > GLA_PLAN_MAX_BUDGET) return GLA_ERR_UNSUPPORTED;
  if (!cu_seqlens || !token_seq != !token_pos) return GLA_ERR_NULL;
  if (N > 0 && (!new_len || !held || !slot || !start_row || !row)) return GLA_ERR_NULL;
  for (const void* p : {(const void*)new_len, (const void*)held, (const void*)seen, (const void*)cu_seqlens,
                        (const void*)slot, (const void*)start_row, (const void*)row, (const void*)token_seq,
                        (const void*)token_pos})
    if (off4(p)) return GLA_ERR_ALIGN;
  unsigned* err;
  unsigned long long wait_ns;
  const int rc = gla::current_device_state(&err, &wait_ns);
  if (rc) return rc;
  return status_of(gla::launch_slot_plan(new_len, held, seen, N, pool_rows, budget, cu_seqlens, slot, start_row, row,
                                         token_seq, token_pos, err, (cudaStream_t)stream));
}

}  // extern "C"
