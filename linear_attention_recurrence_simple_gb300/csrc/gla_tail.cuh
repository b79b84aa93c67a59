// Tail caches: per (row, head) the keys and values of a sequence's tokens after its shared prefix,
//   keys [rows, H, cap, 96], values [rows, H, cap, 192],
// in the element type of the call, or as MXFP8 (E4M3 codes of the same shape, one E8M0 scale byte per
// 32 values: [rows, H, cap, 3] and [rows, H, cap, 6]).  The head stands before the token, so that the
// tokens of one (row, head) are one contiguous piece of each array: what the readout streams.
#pragma once

#include "gla.h"
#include "gla_common.cuh"
#include "gla_mx.cuh"

namespace gla {

struct TailArgs {
  void* k;
  void* v;
  uint8_t* ks;  // MXFP8 only
  uint8_t* vs;
  const int32_t* slot;  // tail row of each sequence, or null: row n
  const int32_t* len;   // tokens of each sequence that the tail holds (or the first place to access)
  int rows;
  int cap;
};

// lambda^n from log lambda; n = 0 gives 1 for every lambda (log lambda = -inf included).
__device__ __forceinline__ float decay_pow(float ll, int n) { return n == 0 ? 1.f : expf((float)n * ll); }

// First token index of (sequence n's tail row, head h) in the tail arrays, when places
// [len[n], len[n] + extra) lie inside the row; otherwise -1, and ERR_SHAPE is recorded.
__device__ __forceinline__ long long tail_token0(const TailArgs& t, int n, int H, int h, int extra, int& len,
                                                 unsigned* err) {
  const int row = t.slot ? t.slot[n] : n;
  len = t.len[n];
  if (row < 0 || row >= t.rows || len < 0 || len > t.cap || extra > t.cap - len) {
    raise_error(err, ERR_SHAPE);
    return -1;
  }
  return ((long long)row * H + h) * t.cap;
}

// Debug-bounds build: a piece of `count` tokens from token index `at` lies inside the tail arrays, a (row, head) inside
// a pool (always true in the release build).
__device__ __forceinline__ bool tail_in_bounds([[maybe_unused]] const TailArgs& t, [[maybe_unused]] int H,
                                               [[maybe_unused]] long long at, [[maybe_unused]] int count,
                                               [[maybe_unused]] unsigned* err) {
  return GLA_IN_BOUNDS(at >= 0 && count >= 0 && at + count <= (long long)t.rows * H * t.cap &&
                           (count == 0 || at / t.cap == (at + count - 1) / t.cap),
                       err);
}
__device__ __forceinline__ bool state_in_bounds([[maybe_unused]] int row, [[maybe_unused]] int rows, [[maybe_unused]] int h,
                                                [[maybe_unused]] int H, [[maybe_unused]] unsigned* err) {
  return GLA_IN_BOUNDS(row >= 0 && row < rows && h >= 0 && h < H, err);
}

template <class T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]);
template <>
__device__ __forceinline__ void store16<float>(float* p, const float (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    reinterpret_cast<float4*>(p)[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[8 * j + 2 * e], x[8 * j + 2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(p)[j] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Writes 16 values to a token's row, quantised where the tail is MXFP8.  Every lane of the warp
// calls it (the block's maximum is exchanged between lanes l and l ^ 1, which hold its two halves:
// even pieces sit in even lanes); `live` says whether this lane's piece is written.
template <class T, bool MX, int D>
__device__ __forceinline__ void tail_store16(void* base, uint8_t* scales, long long token, int p,
                                             const float (&x)[16], bool live) {
  if constexpr (MX) {
    const int se = mx_shared_exp(block_max(x));
    if (live) {
      *(reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + token * D) + p) = quantise16(x, se);
      if ((p & 1) == 0) scales[token * (D / 32) + (p >> 1)] = (uint8_t)(se + 127);
    }
  } else {
    if (live) store16(static_cast<T*>(base) + token * D + 16 * p, x);
  }
}

constexpr int TOKEN_PIECES = (DK + DV) / 16;  // 18 16-value pieces per token and head: 6 of k, 12 of v

// Checks of a tail shared by every call that takes one; fills `a`.
int check_tail(const gla_tail* t, int H, TailArgs* a);

}  // namespace gla
