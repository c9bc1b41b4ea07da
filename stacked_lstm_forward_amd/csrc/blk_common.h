// What the block operators' kernels share: parameters, addressing of sequences,
// conversions.  Addresses and strides are those of elements of 2 or 4 bytes, so
// vectors are loaded and stored through memcpy (the hardware takes any alignment).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dec_grid.h"
#include "lstm_common.h"

namespace lstm {

struct SeqStride {
  long long b, t;  // elements
};

struct NormParams {
  const void *x, *r, *w, *b, *dy, *ds;
  void *s, *y, *dx;
  float *mean, *rstd;
  float *dw, *db;
  float* part;  // backward: partial sums of dw and db
  const int32_t* lengths;
  SeqStride sx, sr, ss, sy, sdy, sds, sdx;
  int B, T, N;
  float eps;
  int blocks;  // workgroups of the launch that make partial sums
};

struct GlrParams {
  const void *f, *u, *o, *dy;
  void *y, *df, *du, *dout_o;
  const float *c0, *dcT;
  float *cT, *dc0;
  float* reserve;
  void* ws;
  const int32_t* lengths;
  SeqStride sf, su, so, sy, sdy, sdf, sdu, sdo;
  int B, T, H;
  int tanh;
  long long wait;  // a wait's limit, ticks of 10 ns
};

hipError_t norm_fwd_launch(const NormParams& p, bool bf16, hipStream_t stream);
hipError_t norm_bwd_launch(const NormParams& p, bool bf16, bool grad_bf16, hipStream_t stream);
size_t norm_bwd_parts(const NormParams& p);  // floats
hipError_t glr_fwd_launch(const GlrParams& p, bool bf16, hipStream_t stream);
hipError_t glr_bwd_launch(const GlrParams& p, bool bf16, bool grad_bf16, hipStream_t stream);
size_t glr_reserve(const GlrParams& p, bool bf16);  // floats
size_t glr_workspace(const GlrParams& p, bool bf16);  // bytes
bool glr_waits(const GlrParams& p, bool bf16, bool train);  // the workspace begins with an error word

// Steps of sentence b that are its own.
__device__ __forceinline__ int steps_of(const int32_t* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : n > T ? T : n;
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// N consecutive elements as they lie in memory, and as fp32.
template <bool BF, int N>
struct Raw {
  static constexpr int kWords = BF ? (N + 1) / 2 : N;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* p) { __builtin_memcpy(w, p, N * (BF ? 2 : 4)); }
  __device__ __forceinline__ void store(void* p) const { __builtin_memcpy(p, w, N * (BF ? 2 : 4)); }
  // (written past the caches)
  __device__ __forceinline__ void store_once(void* p) const {
    typedef uint32_t W __attribute__((ext_vector_type(kWords), aligned(2)));
    W v;
    __builtin_memcpy(&v, w, sizeof(v));
    __builtin_nontemporal_store(v, (W*)p);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    return __uint_as_float(w[i]);
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (BF) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        w[i] = __builtin_bit_cast(
            uint32_t, __builtin_convertvector((f32x2_t){v[2 * i], 2 * i + 1 < N ? v[2 * i + 1] : 0.f}, bf16x2_t));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
    }
  }
  // What follows takes the values from these registers again, not from what was made of them before.
  __device__ __forceinline__ void hide() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // the first n of N elements (0 behind them), one by one
  __device__ __forceinline__ void load_part(const void* p, int n) {
    clear();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        if constexpr (BF)
          w[i / 2] |= (uint32_t)((const uint16_t*)p)[i] << (i & 1 ? 16 : 0);
        else
          w[i] = ((const uint32_t*)p)[i];
      }
  }
  __device__ __forceinline__ void store_part(void* p, int n) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) {
        if constexpr (BF)
          ((uint16_t*)p)[i] = (uint16_t)(w[i / 2] >> (i & 1 ? 16 : 0));
        else
          ((uint32_t*)p)[i] = w[i];
      }
  }
};

// Sums over groups of 2, 4, 8, 16 (lanes next to each other), 32 or 64 lanes; every lane gets its
// group's, the same bits in each: both partners of a step add the same two values.
template <int CTRL>
__device__ __forceinline__ float lane_pair(float v) {
  const int x = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false));
}
template <int N>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (N >= 2) v += lane_pair<0xb1>(v);   // quad_perm [1, 0, 3, 2]
  if constexpr (N >= 4) v += lane_pair<0x4e>(v);   // quad_perm [2, 3, 0, 1]
  if constexpr (N >= 8) v += lane_pair<0x141>(v);  // row_half_mirror
  if constexpr (N >= 16) v += lane_pair<0x140>(v); // row_mirror
  if constexpr (N >= 32) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t x = r[0], y = r[1];
    v = __uint_as_float(x) + __uint_as_float(y);
  }
  if constexpr (N >= 64) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t x = r[0], y = r[1];
    v = __uint_as_float(x) + __uint_as_float(y);
  }
  return v;
}

}  // namespace lstm
