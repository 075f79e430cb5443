// block_rows.hpp - the row-wise kernels around the feed-forward block: the
// root-mean-square norm with the residual's addition and its backward pass,
// dropout, and the values of MXFP8 codes. All of them are bound by the bytes they
// move, 16 a lane.
#pragma once

#include "../../include/moe_block.h"
#include "ffn_types.hpp"

namespace moe_block {

using namespace moe_ffn;

// Eight elements at column c < n of a row of n columns, zeros past n. The last ones of a
// row whose n is no multiple of 8 come from the row's last 16 bytes, shifted: load
// by load, as load8_raw takes them, every row waited for them (30000 rows of 1001,
// norm's backward pass 72 us).
__device__ __forceinline__ s16x8 load_row8(const uint16_t *row, int c, int n) {
  if (n < 8) return load8_raw(row, c, n);
  const int at = min(c, n - 8);
  s16x8 w = *reinterpret_cast<const s16x8_any *>(row + at);
  if (at < c) w = without_first(w, c - at);
  return w;
}

// ------------------------------------------------------------------- dropout

// Dropout of one call; level 0: none.
struct Drop {
  const uint64_t *state;
  uint32_t level, site;
  float times;  // 2^16 / (2^16 - level), 0 where all are dropped
};

// The key and offset, read once by a kernel.
struct Numbers {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ Numbers numbers_of(const Drop &d) {
  if (!d.level) return {0, 0, 0, 0};
  const uint64_t seed = d.state[0], offset = d.state[1];
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

// drop() of the 8 elements of chunk c of row t. Philox4x32-10: ten rounds, each of
// two 32 x 32 -> 64 products (one instruction each); 16 bits an element make one
// counter serve 8 of them: 60 operations an element would be the kernel's bound
// with a 32-bit number for each, and the level's step of 2^-16 is finer than the
// probabilities in use.
__device__ __forceinline__ f32x8 drop8(f32x8 v, uint32_t t, uint32_t c, const Drop &d,
                                       const Numbers &n) {
  uint32_t x0 = c + (d.site << 17), x1 = t, x2 = n.o0, x3 = n.o1, k0 = n.k0, k1 = n.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)x0 * 0xD2511F53u, p1 = (uint64_t)x2 * 0xCD9E8D57u;
    x0 = (uint32_t)(p1 >> 32) ^ x1 ^ k0;
    x2 = (uint32_t)(p0 >> 32) ^ x3 ^ k1;
    x1 = (uint32_t)p1;
    x3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {x0, x1, x2, x3};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu;
    v[i] = u >= d.level ? v[i] * d.times : 0.f;
  }
  return v;
}

struct DropoutArgs {
  const uint16_t *x, *res;
  uint16_t *out;
  int64_t ld_x, ld_res, ld_out, tokens;
  int32_t width;
  Drop drop;
};

// A thread takes one 8-element chunk of a row, and goes down the rows. blockDim.x
// chunks of blockDim.y rows, so that short rows leave no lanes idle. Bound by memory: 8192
// x 7168 with the residual 69 us, 5.1 TB/s, the ten rounds of numbers hidden behind the loads.
template <class D>
__global__ __launch_bounds__(256) void dropout_kernel(const DropoutArgs a) {
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (c >= a.width) return;
  const Numbers n = numbers_of(a.drop);
  for (int64_t t = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; t < a.tokens;
       t += (int64_t)gridDim.y * blockDim.y) {
    const s16x8 raw = load_row8(a.x + t * a.ld_x, c, a.width);
    s16x8 rest = {0, 0, 0, 0, 0, 0, 0, 0};
    if (a.res) rest = load_row8(a.res + t * a.ld_res, c, a.width);
    f32x8 v = unpack8<D>(raw);
    if (a.drop.level) v = drop8(v, (uint32_t)t, (uint32_t)c >> 3, a.drop, n);
    if (a.res) {
      const f32x8 r = unpack8<D>(rest);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    store8<D>(a.out + t * a.ld_out, c, a.width, v);
  }
}

// ----------------------------------------------------------- sums over lanes

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __uint_as_float(dpp_u<CTRL>(__float_as_uint(v)));
}
constexpr int XOR1 = 0xB1, XOR2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140;

// The sum over 16 adjacent lanes, or over the wave, in every one of them.
__device__ __forceinline__ float sum16(float v) {
  v += dpp_f<XOR1>(v);
  v += dpp_f<XOR2>(v);
  v += dpp_f<HALF_MIRROR>(v);
  return v + dpp_f<MIRROR>(v);
}
__device__ __forceinline__ float sum64(float v) {
  const int b = __float_as_int(sum16(v));
  return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) +
          __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(b, 32)) +
          __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}
// Over the L lanes of a row. With several waves through LDS: `slot` alternates
// from row to row, so that one barrier a row is enough.
template <int L>
__device__ __forceinline__ float row_sum(float v, float (*slots)[16], int slot) {
  if constexpr (L == 16) return sum16(v);
  v = sum64(v);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) slots[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < L / 64; ++w) v += slots[slot][w];
  }
  return v;
}

// ---------------------------------------------------------------------- norm

// Makes the compiler unpack a row's elements again where they are used again, in
// place of keeping them in fp32 across the row's sum, which takes twice the registers.
__device__ __forceinline__ void keep_packed(s16x8 &v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
}

struct NormArgs {
  const uint16_t *x, *res, *weight;
  uint16_t *h, *y;
  float *rstd;
  uint8_t *q, *q_scale;
  const uint16_t *dy, *dh;  // backward
  uint16_t *dx, *dres;
  float *part;  // [blocks][width] sums of dy n over the block's rows, or NULL
  int64_t ld_x, ld_res, ld_h, ld_y, ld_dy, ld_dh, ld_dx, ld_dres, tokens;
  int32_t width;
  float eps;
  Drop drop;
};

// E4M3 codes of v[0..7] 2^-shared: to nearest even, saturating, NaN kept.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
__device__ __forceinline__ u32x2_any e4m3_codes(f32x8 v, int shared) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __builtin_amdgcn_ldexpf(v[i], -shared);
    s[i] = t != t ? t : __builtin_amdgcn_fmed3f(t, -448.f, 448.f);
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], hi, true);
  return u32x2_any{(uint32_t)lo, (uint32_t)hi};
}
// The exponent of the scale of 32 values, 8 of them in each of 4 adjacent lanes.
__device__ __forceinline__ int mx_exponent(f32x8 v) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  most = max(most, dpp_u<XOR1>(most));
  most = max(most, dpp_u<XOR2>(most));
  const int e = (int)(most >> 23);
  return e == 0 ? -127 : max(e - 135, -127);
}

// Lanes of a row and chunks of 8 elements of a lane: the least that hold the width.
template <int L_, int CH_>
struct RowShape {
  static constexpr int L = L_, CH = CH_, THREADS = L < 256 ? 256 : L, ROWS = THREADS / L;
  static constexpr int WIDTH = L * CH * 8;
  // The backward pass keeps its columns' sums of dweight in registers, or, where the
  // threads have none left for them, in LDS. (4096 rows of 32768 with 1024 threads, whose
  // 128 registers hold neither: 772 us, with the sums in LDS 655.)
  static constexpr bool SUMS_IN_LDS = CH > 4;
};

// A row stays in registers from its loads to its stores: one pass over memory (but
// for the shape of more than 16384 columns, of which the compiler spills 20 registers a lane). The
// blocks go down the rows with the weight in registers. h is rounded before it
// is squared: y is the norm of the h that is stored, which the backward pass
// reads. Bound by memory: 16384 x 7168 with residual and h, y as E4M3 codes, 830 MB in 165
// us (5.0 TB/s); 131071 x 128 13.4 us (5.0). 8 x 7168 takes 5.7 us, a launch and one row's
// loads, sum and stores after each other.
template <class D, class S>
__global__ __launch_bounds__(S::THREADS) void norm_kernel(const NormArgs a) {
  constexpr int L = S::L, CH = S::CH;
  __shared__ float slots[2][16];
  const int lane = threadIdx.x % L;
  const Numbers n = numbers_of(a.drop);
  const float inv_width = 1.f / (float)a.width;
  s16x8 weight[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * L + lane) * 8;
    if (c < a.width) weight[i] = load_row8(a.weight, c, a.width);
  }
  int slot = 0;
  for (int64_t t = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / L; t < a.tokens;
       t += (int64_t)gridDim.x * S::ROWS, slot ^= 1) {
    s16x8 row[CH], rest[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * L + lane) * 8;
      row[i] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
      if (c < a.width) {
        row[i] = load_row8(a.x + t * a.ld_x, c, a.width);
        if (a.res) rest[i] = load_row8(a.res + t * a.ld_res, c, a.width);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * L + lane) * 8;
      if (c < a.width && (a.res || a.drop.level)) {
        f32x8 v = unpack8<D>(row[i]);
        if (a.drop.level) v = drop8(v, (uint32_t)t, (uint32_t)c >> 3, a.drop, n);
        if (a.res) {
          const f32x8 r = unpack8<D>(rest[i]);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] += r[k];
        }
        row[i] = pack8<D>(v);
      }
      if (c < a.width && a.h) store8_raw(a.h + t * a.ld_h, c, a.width, row[i]);
      const f32x8 v = unpack8<D>(row[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
    }
    sum = row_sum<L>(sum, slots, slot);
    float total = fmaf(sum, inv_width, a.eps), unit = 1.f;
    if constexpr (D::MAX_EXPONENT >= 127) {
      // squares past fp32's range, or below what it holds precisely: again, of
      // elements times a power of two (the same branch in all threads of a row)
      if (total > 3e38f || total < 0x1p-100f) {
        unit = total < 1.f ? 0x1p96f : 0x1p-96f;
        slot ^= 1;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          keep_packed(row[i]);
          const f32x8 v = unpack8<D>(row[i]);
#pragma unroll
          for (int k = 0; k < 8; ++k) sum = fmaf(v[k] * unit, v[k] * unit, sum);
        }
        sum = row_sum<L>(sum, slots, slot);
        total = fmaf(sum, inv_width, a.eps * unit * unit);
      }
    }
    const float rstd = unit / sqrtf(total);
    if (a.rstd && lane == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int i = 0; i < CH; ++i) keep_packed(row[i]), keep_packed(weight[i]);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * L + lane) * 8;
      if (c >= a.width) continue;  // whole groups of 4 lanes where q is written
      f32x8 v = unpack8<D>(row[i]);
      const f32x8 w = unpack8<D>(weight[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * rstd * w[k];
      if (a.y) store8<D>(a.y + t * a.ld_y, c, a.width, v);
      if (a.q) {
        const int shared = mx_exponent(v);
        const int64_t at = t * a.width + c;
        *reinterpret_cast<u32x2_any *>(a.q + at) = e4m3_codes(v, shared);
        if ((lane & 3) == 0) a.q_scale[at >> 5] = (uint8_t)(shared + 127);
      }
    }
  }
}

// The backward pass: a row in registers again, and each lane keeps its columns' sums
// of dy n over all rows of its block (fp32, written once a block and added by
// norm_weight_kernel in the order of the blocks). Bound by memory: 8192 x 7168 with dh 94.5 us
// (5.0 TB/s). Rows of more than 16384 columns, whose sums go through LDS, do not fit the registers:
// 113 of a lane are spilled, and 4096 x 32768 takes 396 us (2.7 TB/s), bound by that.
template <class D, class S>
__global__ __launch_bounds__(S::THREADS) void norm_backward_kernel(const NormArgs a) {
  constexpr int L = S::L, CH = S::CH;
  __shared__ float slots[2][16];
  __shared__ __attribute__((aligned(16))) float join[S::ROWS > 1 ? S::ROWS : 1]
                                                   [S::ROWS > 1 || S::SUMS_IN_LDS ? S::WIDTH : 1];
  const int lane = threadIdx.x % L;
  const Numbers n = numbers_of(a.drop);
  const float inv_width = 1.f / (float)a.width;
  s16x8 weight[CH];
  const f32x8 zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  f32x8 dw[S::SUMS_IN_LDS ? 1 : CH];
  auto sums = [&](int i) -> f32x8 * { return reinterpret_cast<f32x8 *>(&join[0][(i * L + lane) * 8]); };
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * L + lane) * 8;
    weight[i] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
    if (c < a.width) weight[i] = load_row8(a.weight, c, a.width);
    if constexpr (S::SUMS_IN_LDS) *sums(i) = zero; else dw[i] = zero;
  }
  int slot = 0;
  for (int64_t t = (int64_t)blockIdx.x * S::ROWS + threadIdx.x / L; t < a.tokens;
       t += (int64_t)gridDim.x * S::ROWS, slot ^= 1) {
    s16x8 dy[CH], h[CH], rest[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * L + lane) * 8;
      dy[i] = h[i] = rest[i] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
      if (c < a.width) {
        dy[i] = load_row8(a.dy + t * a.ld_dy, c, a.width);
        h[i] = load_row8(a.h + t * a.ld_h, c, a.width);
        if (a.dh) rest[i] = load_row8(a.dh + t * a.ld_dh, c, a.width);
      }
    }
    const float rstd = a.rstd[t];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const f32x8 d = unpack8<D>(dy[i]), f = unpack8<D>(h[i]), w = unpack8<D>(weight[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(d[k] * (f[k] * rstd), w[k], sum);
      if constexpr (S::SUMS_IN_LDS) {
        if (a.part) {
          f32x8 t = *sums(i);
#pragma unroll
          for (int k = 0; k < 8; ++k) t[k] += d[k] * (f[k] * rstd);
          *sums(i) = t;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[i][k] += d[k] * (f[k] * rstd);
      }
    }
    const float mean = row_sum<L>(sum, slots, slot) * inv_width;
    if (!a.dx && !a.dres) continue;
#pragma unroll
    for (int i = 0; i < CH; ++i) keep_packed(dy[i]), keep_packed(h[i]), keep_packed(weight[i]);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * L + lane) * 8;
      if (c >= a.width) continue;
      const f32x8 d = unpack8<D>(dy[i]), f = unpack8<D>(h[i]), w = unpack8<D>(weight[i]);
      f32x8 v = unpack8<D>(rest[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += rstd * (d[k] * w[k] - f[k] * rstd * mean);
      if (a.dres) store8<D>(a.dres + t * a.ld_dres, c, a.width, v);
      if (a.dx) {
        if (a.drop.level) v = drop8(v, (uint32_t)t, (uint32_t)c >> 3, a.drop, n);
        store8<D>(a.dx + t * a.ld_dx, c, a.width, v);
      }
    }
  }
  if (!a.part) return;
  float *part = a.part + (int64_t)blockIdx.x * a.width;
  if constexpr (S::ROWS > 1) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) join[threadIdx.x / L][(i * L + lane) * 8 + k] = dw[i][k];
    __syncthreads();
    for (int c = threadIdx.x; c < a.width; c += S::THREADS) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < S::ROWS; ++g) v += join[g][c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * L + lane) * 8;
      if (c < a.width) store8_f32(part, c, a.width, S::SUMS_IN_LDS ? *sums(i) : dw[S::SUMS_IN_LDS ? 0 : i]);
    }
  }
}

// dweight[c] = the sum over the blocks' partial sums: 64 columns a block, 16 lanes to
// a column, whose sums are added in their order. Bound by latency: 512 x 7168 sums 4.8 us.
constexpr int NORM_SUM_ROWS = 16;
template <class D>
__global__ __launch_bounds__(64 * NORM_SUM_ROWS) void norm_weight_kernel(
    const float *__restrict__ part, int blocks, int width, uint16_t *__restrict__ dw) {
  __shared__ float sums[NORM_SUM_ROWS][64];
  const int c = blockIdx.x * 64 + threadIdx.x;
  float v = 0.f;
  if (c < width)
#pragma unroll 8
    for (int b = threadIdx.y; b < blocks; b += NORM_SUM_ROWS) v += part[(int64_t)b * width + c];
  sums[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < width) {
    v = 0.f;
#pragma unroll
    for (int r = 0; r < NORM_SUM_ROWS; ++r) v += sums[r][threadIdx.x];
    dw[c] = from_f<D>(v);
  }
}

// -------------------------------------------------------------- MXFP8 values

// Values of MXFP8 codes, exact in bf16 but for scales beyond its range. Bound by memory:
// 16384 x 7168 68 us, 5.2 TB/s.
__device__ __forceinline__ float e4m3_value(uint32_t code, int exponent) {
  const int e = (code >> 3) & 15, m = code & 7;
  if ((code & 0x7F) == 0x7F) return __uint_as_float(0x7FC00000u);
  const float v = __builtin_amdgcn_ldexpf(e ? (float)(8 + m) : (float)m, (e ? e : 1) - 10 + exponent);
  return code & 0x80 ? -v : v;
}
template <class D>
__global__ __launch_bounds__(256) void mx_values_kernel(const uint8_t *__restrict__ q,
                                                        const uint8_t *__restrict__ q_scale,
                                                        int64_t chunks, uint16_t *__restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks;
       i += (int64_t)gridDim.x * 256) {
    const u32x2_any codes = *reinterpret_cast<const u32x2_any *>(q + i * 8);
    const int scale = q_scale[i >> 2];
    f32x8 v;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = e4m3_value(codes[k >> 2] >> (8 * (k & 3)) & 0xFF, scale - 127);
      if (scale == 255) v[k] = __uint_as_float(0x7FC00000u);
    }
    *reinterpret_cast<s16x8_any *>(out + i * 8) = pack8<D>(v);
  }
}

}  // namespace moe_block
