// adapter_expand.hpp - the low-rank term of a product, s B_a^T with the adapter a of
// each row, added to the sums that the product kernels hold before their epilogue.
//
// s is fp32. The matrix cores take it in three parts of the matrices' type, which hold
// its 24 bits between them, so that y is the same sum in fp32 here as where few tokens
// multiply s itself; each part costs 1/(in / 32) of the product's operations. (Two parts
// hold 16 bits in bf16: enough beside one rounding of y, not where x W^T and s B^T cancel.)
// In fp16, whose range s may pass, a row's values are taken at a power of two that makes the
// largest of 32 of them lie in [2^14, 2^15); its smallest step, 2^-24, is then 2^-38 of it.
//
// A row takes only its own adapter's result, by a selection and not by factors of zero:
// infinities or NaN in one adapter stay out of the other requests' rows.
#pragma once

#include <type_traits>

#include "ffn_types.hpp"

namespace moe_ffn {

// v in three parts of the type, the largest first. What is no finite number stays in
// the first.
template <class D>
__device__ __forceinline__ void three_parts(f32x8 v, s16x8 (&part)[3]) {
  part[0] = pack8<D>(v);
  const f32x8 h = unpack8<D>(part[0]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_isfinite(h[i]) ? v[i] - h[i] : 0.f;
  part[1] = pack8<D>(v);
  part[2] = pack8<D>(v - unpack8<D>(part[1]));
}
// The power of two that takes `most`, the largest of some magnitudes, into [2^14, 2^15).
__device__ __forceinline__ int exponent_for(float most) {
  const int e = (int)(__float_as_uint(most) >> 23 & 0xff);
  return e == 0 || e == 255 ? 0 : 14 + 127 - e;
}

// acc[i][j] of a wave: rows row0 + 16 i + fr, columns col0 + 16 j + 4 fq .. 4 fq + 3 in
// a lane (fr = lane & 15, fq = lane >> 4). For every 16 rows the adapters among them
// are taken one after the other; the fragments of B stay from one 16 rows to the next
// while the adapter is the same, as in a prompt's rows. A prompt's rows pay next to
// nothing (8192 rows, 7168 -> 2048, rank 16: 180 us, without the term 182). 1200 rows of one token
// each, 14 adapters among 16, pay some 35 us beside 59 (4096 -> 4096): the scan, loads, matrix
// instructions and selections of an adapter follow each other. (The order of the loads' lanes is
// not what it waits for: all lanes on one address take as long.)
template <class D, int FM, int FN>
__device__ __forceinline__ void add_low_rank(f32x4 (&acc)[FM][FN], const LowRank &g, int row0,
                                             int row_end, int col0, int N) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool SCALED = D::MAX_EXPONENT < 127;
  const int lane = threadIdx.x & 63, fr = lane & 15, fq = lane >> 4;
  // rows whose values of s are loaded together, and adapters whose B is. The waves of the
  // largest tiles have no registers for more (two adapters: 221 us for 217); with 4 and 8 adapters
  // in the others 1200 rows of one token each take 119 and 121 us, 1024 rows of 8 prompts 47 and 49.
  constexpr int GROUP = FM < 4 ? FM : FM > 4 ? 2 : 4, AT_ONCE = FN <= 2 ? 4 : 1;
  // up to rank 16 one matrix instruction takes two parts, 16 elements of its 32 each
  const bool both = g.rank <= 16;
  int64_t row_b[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) row_b[j] = (int64_t)min(col0 + 16 * j + fr, N - 1) * g.ldb;
#pragma unroll 1
  for (int k0 = 0; k0 < g.rank; k0 += 32) {
    const int k = k0 + (both ? fq & 1 : fq) * 8, at = min(k, g.rank - 8);
    int have = -1;  // the adapter of fb[0], where it is there alone
    s16x8 fb[AT_ONCE][FN];
#pragma unroll
    for (int i0 = 0; i0 < FM; i0 += GROUP) {
      int id[GROUP];
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        const int m = row0 + 16 * (i0 + i) + fr;
        id[i] = g.ids[min(m, row_end - 1)];
        if (m >= row_end || (uint32_t)id[i] >= (uint32_t)g.n) id[i] = -1;
      }
      f32x8 v[GROUP];
      if ((g.rank & 7) == 0) {
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
          v[i] = *reinterpret_cast<const f32x8_any *>(
              g.s + (int64_t)min(row0 + 16 * (i0 + i) + fr, row_end - 1) * g.lds + at);
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
#pragma unroll
          for (int t = 0; t < 8; ++t) v[i][t] = at == k ? v[i][t] : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
          v[i] = load8_f32(g.s + (int64_t)min(row0 + 16 * (i0 + i) + fr, row_end - 1) * g.lds, k, g.rank);
      }
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        uint32_t todo = (uint32_t)__ballot(id[i] >= 0) & 0xffffu;
        if (!todo) continue;
        int power = 0;
        if constexpr (SCALED) {
          float most = 0.f;
#pragma unroll
          for (int t = 0; t < 8; ++t) most = fmaxf(most, fabsf(v[i][t]));
          most = fmaxf(most, __shfl_xor(most, 16));
          most = fmaxf(most, __shfl_xor(most, 32));
          power = exponent_for(most);
#pragma unroll
          for (int t = 0; t < 8; ++t) v[i][t] = __builtin_amdgcn_ldexpf(v[i][t], power);
        }
        s16x8 part[3];
        three_parts<D>(v[i], part);
        if (both && fq >= 2) part[0] = part[1], part[2] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
        while (todo) {
          // the next adapters' fragments are loaded together: a decode batch's rows
          // have one each
          int a[AT_ONCE];
#pragma unroll
          for (int q = 0; q < AT_ONCE; ++q) {
            const int next = __builtin_amdgcn_readlane(id[i], __builtin_ctz(todo | 0x8000u));
            a[q] = todo ? next : -2;  // -2: no row's
            todo &= ~(uint32_t)__ballot(id[i] == next);
          }
          // B of the first adapters (a[0] for those there are not), without a branch between
          // the loads, which would wait for one after the other
          auto load_b = [&](auto count) MOE_INLINE {
            constexpr int Q = decltype(count)::value;
            if (g.rank < 8) {
#pragma unroll
              for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                  fb[q][j] = load8_raw(g.b + (a[q] < 0 ? a[0] : a[q]) * g.stride + row_b[j], k, g.rank);
              return;
            }
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
              for (int j = 0; j < FN; ++j)
                fb[q][j] = *reinterpret_cast<const s16x8_any *>(
                    g.b + (a[q] < 0 ? a[0] : a[q]) * g.stride + row_b[j] + at);
            if (k0 + (both ? 16 : 32) <= g.rank) return;
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
              for (int j = 0; j < FN; ++j) fb[q][j] = without_first(fb[q][j], k - at);
          };
          const bool several = AT_ONCE > 1 && a[AT_ONCE > 1] >= 0;
          if (several)
            load_b(std::integral_constant<int, AT_ONCE>());
          else if (a[0] != have)
            load_b(std::integral_constant<int, 1>());
          have = several ? -1 : a[0];
          auto add = [&](int q) MOE_INLINE {
            const bool mine = id[i] == a[q];
            f32x4 sum[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < FN; ++j) sum[j] = D::mfma(fb[q][j], part[2], sum[j]);
            if (!both)
#pragma unroll
              for (int j = 0; j < FN; ++j) sum[j] = D::mfma(fb[q][j], part[1], sum[j]);
#pragma unroll
            for (int j = 0; j < FN; ++j) sum[j] = D::mfma(fb[q][j], part[0], sum[j]);
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float t = sum[j][e];
                if constexpr (SCALED) t = __builtin_amdgcn_ldexpf(t, -power);
                acc[i0 + i][j][e] = mine ? acc[i0 + i][j][e] + t : acc[i0 + i][j][e];
              }
          };
          add(0);
          if (several)
#pragma unroll
            for (int q = 1; q < AT_ONCE; ++q) add(q);
        }
      }
    }
  }
#endif
}

}  // namespace moe_ffn
