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
__device__ __forceinline__ s16x8 pack8(f32x8 v) {
  return __builtin_bit_cast(s16x8, __builtin_convertvector(v, typename D::v8));
}
template <class D>
__device__ __forceinline__ f32x8 unpack8(s16x8 v) {
  return __builtin_convertvector(__builtin_bit_cast(typename D::v8, v), f32x8);
}

// act(z) and act'(z) in fp32. silu' = s (1 + z (1 - s)) with s = sigmoid(z);
// gelu' = Phi(z) + z phi(z). e^-z overflows to infinity below -88, where
// 1 / (1 + e^-z) is 0.
__device__ __forceinline__ float sigmoid_f(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}
// Phi(z), the normal distribution function, from `e` = exp(-z^2 / 2):
// Phi(-a) = e t q(t) for a >= 0 with t = 1 / (1 + 0.28 a). q, of degree 8, is a
// least-squares fit of exp(a^2 / 2) Phi(-a) / t in t over (0, 1], reweighted
// towards the smallest largest relative error: 1.7e-7, and 5.1e-7 evaluated in
// fp32. The tail keeps its relative accuracy, and the cost is a
// reciprocal and 9 multiply-adds where a library erfc takes several branches
// (the epilogue of 8192 x 2048 -> 7168 with gelu).
__device__ __forceinline__ float phi_cdf(float z, float e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.28f, fabsf(z), 1.f));
  float q = 2.472378500e-02f;
  q = fmaf(q, t, -9.360811114e-02f);
  q = fmaf(q, t, 9.245216101e-02f);
  q = fmaf(q, t, -6.469420623e-03f);
  q = fmaf(q, t, 7.278459519e-02f);
  q = fmaf(q, t, 8.362825215e-02f);
  q = fmaf(q, t, 1.030850187e-01f);
  q = fmaf(q, t, 1.116997823e-01f);
  q = fmaf(q, t, 1.117038578e-01f);
  const float tail = e * t * q;
  return z < 0.f ? tail : 1.f - tail;
}
// Whole vectors, so that the branch on the activation is taken once and their
// elements' long chains of dependent operations run beside each other.
template <class V>
__device__ __forceinline__ V act_value(V z, int act) {
  constexpr int N = sizeof(V) / sizeof(float);
  if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = z[i] * sigmoid_f(z[i]);
  } else if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = z[i] * phi_cdf(z[i], __expf(-0.5f * z[i] * z[i]));
  }
  return z;
}
template <class V>
__device__ __forceinline__ void act_value_slope(V z, int act, V &value, V &slope) {
  constexpr int N = sizeof(V) / sizeof(float);
  if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = sigmoid_f(z[i]);
      value[i] = z[i] * s;
      slope[i] = s * (1.f + z[i] * (1.f - s));
    }
  } else if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = __expf(-0.5f * z[i] * z[i]), c = phi_cdf(z[i], e);
      value[i] = z[i] * c;
      slope[i] = c + z[i] * 0.39894228040143268f * e;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) value[i] = z[i], slope[i] = 1.f;
  }
}

// Eight elements at column c of a row that has n columns; zeros past n. Global
// memory takes 16-byte accesses at any element's address.
typedef s16x8 s16x8_any __attribute__((aligned(2)));
__device__ __forceinline__ s16x8 load8_raw(const uint16_t *row, int c, int n) {
  if (c + 8 <= n) return *reinterpret_cast<const s16x8_any *>(row + c);
  s16x8 w = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) w[i] = (short)row[c + i];
  return w;
}
template <class D>
__device__ __forceinline__ f32x8 load8(const uint16_t *row, int c, int n) {
  return unpack8<D>(load8_raw(row, c, n));
}
__device__ __forceinline__ void store8_raw(uint16_t *row, int c, int n, s16x8 w) {
  if (c + 8 <= n) {
    *reinterpret_cast<s16x8_any *>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = (uint16_t)w[i];
  }
}
template <class D>
__device__ __forceinline__ void store8(uint16_t *row, int c, int n, f32x8 v) {
  store8_raw(row, c, n, pack8<D>(v));
}

typedef f32x8 f32x8_any __attribute__((aligned(4)));
__device__ __forceinline__ void store8_f32(float *row, int c, int n, f32x8 v) {
  if (c + 8 <= n) {
    *reinterpret_cast<f32x8_any *>(row + c) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < n) row[c + i] = v[i];
  }
}
__device__ __forceinline__ f32x8 load8_f32(const float *row, int c, int n) {
  if (c + 8 <= n) return *reinterpret_cast<const f32x8_any *>(row + c);
  f32x8 v = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) v[i] = row[c + i];
  return v;
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
  // over experts, where the tile does not divide the layout's alignment: rows
  // [x, y) of each m-tile, then in element m_tiles the number of those with an
  // expert; else NULL
  const int4 *tile_map;
  // dense only: K in `splits` ranges of k_split (a multiple of 64), each summed
  // into its own partial [splits][WGRAD: segs][M][N, GATED: 2 N]; NULL: one range
  int32_t splits, k_split;
  float *partial;
  uint32_t top_k_magic, top_k_shift; // entry / top_k as a product; magic 0: top_k is 1
  uint32_t block0;         // number of the launch's first block
};

}  // namespace moe_ffn
