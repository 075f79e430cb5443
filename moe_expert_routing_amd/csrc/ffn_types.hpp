// ffn_types.hpp - element types, activations and the shared argument block of
// the feed-forward kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_ffn.h"

namespace moe_ffn {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// The two element types: conversions (to nearest even) and their MFMA.
struct Bf16 {
  typedef __bf16 scalar;
  typedef bf16x4 v4;
  typedef bf16x8 v8;
  static __device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
struct F16 {
  typedef _Float16 scalar;
  typedef f16x4 v4;
  typedef f16x8 v8;
  static __device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <class D>
__device__ __forceinline__ float to_f(uint16_t v) {
  return (float)__builtin_bit_cast(typename D::scalar, v);
}
template <class D>
__device__ __forceinline__ uint16_t from_f(float v) {
  return __builtin_bit_cast(uint16_t, (typename D::scalar)v);
}
template <class D>
__device__ __forceinline__ s16x4 pack4(f32x4 v) {
  return __builtin_bit_cast(s16x4, __builtin_convertvector(v, typename D::v4));
}
template <class D>
__device__ __forceinline__ f32x4 unpack4(s16x4 v) {
  return __builtin_convertvector(__builtin_bit_cast(typename D::v4, v), f32x4);
}
template <class D>
__device__ __forceinline__ s16x8 pack8(f32x8 v) {
  return __builtin_bit_cast(s16x8, __builtin_convertvector(v, typename D::v8));
}
template <class D>
__device__ __forceinline__ f32x8 unpack8(s16x8 v) {
  return __builtin_convertvector(__builtin_bit_cast(typename D::v8, v), f32x8);
}

// act(z) and act'(z) in fp32. silu' = s (1 + z (1 - s)) with s = sigmoid(z);
// gelu' = Phi(z) + z phi(z), where Phi is taken through erfc, so that both stay
// accurate where Phi is small. e^-z overflows to infinity below -88, where
// 1 / (1 + e^-z) is 0.
__device__ __forceinline__ float sigmoid_f(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}
__device__ __forceinline__ float phi_cdf(float z) { return 0.5f * erfcf(-0.70710678118654752f * z); }
__device__ __forceinline__ float act_value(float z, int act) {
  if (act == MOE_ACT_SILU) return z * sigmoid_f(z);
  if (act == MOE_ACT_GELU) return z * phi_cdf(z);
  return z;
}
__device__ __forceinline__ void act_value_slope(float z, int act, float &value, float &slope) {
  if (act == MOE_ACT_SILU) {
    const float s = sigmoid_f(z);
    value = z * s;
    slope = s * (1.f + z * (1.f - s));
  } else if (act == MOE_ACT_GELU) {
    const float c = phi_cdf(z);
    value = z * c;
    slope = c + z * 0.39894228040143268f * __expf(-0.5f * z * z);
  } else {
    value = z;
    slope = 1.f;
  }
}

// The expert of a row's tile and whether one row holds an entry of it.
struct Rows {
  const int32_t *counts, *padded_offsets, *m_indices, *row_entry;
  int64_t rows;        // rows of the row-wise matrices
  int32_t num_experts; // 0: dense
  int32_t top_k;
};

// The uses of the product kernel.
enum Mode { GATED = 0, LINEAR = 1, DGRAD = 2, WGRAD = 3 };

// What one product kernel gets. C[m, n] = sum over k of A(m, k) B(n, k).
struct GemmArgs {
  const uint16_t *a;       // M side
  int64_t lda, a_rows;     // a_rows: rows of A that exist (tokens), gathers stay below it
  const uint16_t *b0, *b1; // N side; b1: second projection
  int64_t ldb0, ldb1, b_stride0, b_stride1;
  uint16_t *c0, *c1;
  int64_t ldc0, ldc1, c_stride0, c_stride1;
  uint16_t *pre;
  int64_t ldp;
  const uint16_t *bias;
  int64_t bias_stride;
  const uint16_t *res;
  int64_t ldr;
  Rows r;
  int32_t M, N, K;         // of one segment
  int64_t a_seg;           // elements between the A columns of two segments
  int32_t segs;            // 1, or 2 for the two projections of a gated block
  int32_t act;
  int32_t m_tiles, n_tiles;
};

}  // namespace moe_ffn
