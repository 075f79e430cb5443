// ffn_gemm.hpp - the tiled products of the feed-forward operators on the
// gfx950 matrix cores.
//
// One kernel template computes C[m, n] = sum over k of A(m, k) B(n, k) for
// four uses, which differ in how the operands lie in memory and in what the
// epilogue does:
//   GATED   A = x rows (gathered by token), B = Wg and Wu rows; epilogue
//           h = act(g) u, optionally g and u themselves
//   LINEAR  A = x rows, B = W rows; epilogue bias, activation, residual
//   DGRAD   A = dz rows, B(n, k) = W[k, n]; one or two segments of k
//           (gate, up) summed
//   WGRAD   A(m, k) = dz[k, m], B(n, k) = x[k, n] (gathered by token), k = the
//           rows of one expert
// An operand whose k is contiguous is staged as rows of 64 k (128 bytes, 8
// chunks of 16 bytes; chunk c of row r at position c ^ (r & 7), so that the 8
// rows that one pass of a fragment read touches hit 8 different bank quads).
// One whose m or n is contiguous is staged as 64 k-rows as they lie in memory
// and read through the transposing LDS load (4 k-rows x 16 columns per 16
// lanes); chunk c of k-row k sits at c ^ swz(k), which puts the 4 rows and the
// two 16-lane groups of a pass on different banks.
//
// Both operands go from global memory straight into LDS, NS stages of 64 k
// deep: stage s + NS is issued as soon as every wave has read stage s. The
// fragments of one MFMA k-step are read from LDS while the previous step's
// MFMAs run.
//
// The weights are the MFMA's first operand: a lane then holds 4 consecutive n
// of one row m, and the two projections of a gated block meet in the same lane
// (their rows are interleaved by 16).
//
// What bounds it, on one MI355X, and what was measured on the way:
//  - 256 x 256 tiles, 8 waves of 128 x 64 (gated block of 4096 x 7168 -> 2048 in
//    training, 240 GFLOP): 180-190 us, 1.27-1.33 PFLOP/s; the MFMA pipes are busy
//    65 % of the time at 1.9 GHz, where the power limit holds the clock. Its 112
//    stages take 153 us; the rest is the first loads and the stores, with every
//    compute unit on one tile. 4 waves of 128 x 128 took 205 us: with one wave
//    on a SIMD nothing covers its other instructions. Stages of 32 k, four or
//    five deep: 200 us, as half lines are twice the requests.
//  - The loop has no branches: stages past the last load zeros by an offset
//    past the buffer. With a branch for the tail, or 64-bit addresses for
//    each piece, the accumulators spilled.
//  - Linear 8192 x 2048 -> 7168: 214 us plain, 255 with gelu, 270 with gelu,
//    bias and residual, and 285-300 with all of it on other inputs each call: 3.5
//    tiles a compute unit take 4 rounds of 43 us for the stages, 4 for the stores,
//    5.5 for gelu and 4 for the residual, whose loads are issued together (one at
//    a time: 304 us where together took 285).
//  - 112 experts with about 146 rows, 2048 -> 1024, 128 x 256 tiles: 265 us
//    for 137 GFLOP (about 190 with the rows that fill up tiles) and 1 GB. Blocks
//    that stay and go from tile to tile, the next tile's loads under the stores,
//    were no faster (274 us; weight gradients 502 against 446).
//  - Weight gradients of these experts, 256 x 256 tiles: 410-460 us, of which
//    writing 940 MB could take 140: with three stages a tile, the first loads
//    (4 us), the stages (5.7) and the stores (3.4) follow each other. 128 x 128
//    and 256 x 128 tiles, two or three blocks to a compute unit, took the same.
#pragma once

#include <type_traits>
#include <utility>

#include "ffn_types.hpp"

namespace moe_ffn {

typedef __attribute__((address_space(3))) void *lds_ptr_t;
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4_ptr_t;
typedef __attribute__((address_space(1))) void *gbl_ptr_t;

#define MOE_INLINE __attribute__((always_inline))  // the kernel's lambdas hold its registers

// Offset past a buffer's end: loads zeros.
constexpr uint32_t PAST = 0xffffffffu;

// The device pass alone knows the buffer builtins.
#if defined(__HIP_DEVICE_COMPILE__)
// 16 bytes a lane from byte offset `o` of the 4 GB - 1 at p into LDS: lane i
// writes at dst + 16 i; p and dst are uniform. With TRANSPOSED the compiler
// is not told of the write to LDS: before every transposing LDS read it
// would wait for all such loads in flight, while the kernel's own waits already
// order a stage's loads before its reads. (s_nop: one wait state between writing
// m0 and an LDS load that reads it.)
template <bool TRANSPOSED>
__device__ __forceinline__ void lds_piece(const uint8_t *p, uint32_t o, uint8_t *dst) {
  if constexpr (TRANSPOSED) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    const uint64_t at = (uint64_t)p;
    const i32x4 rsrc = {(int)(uint32_t)at, (int)(at >> 32) & 0xffff, (int)PAST, 0x00020000};
    const uint32_t to = (uint32_t)(uintptr_t)(lds_ptr_t)dst;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(o),
                 "s"(rsrc)
                 : "m0");
  } else {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, PAST, 0x00020000),
        (lds_ptr_t)dst, 16, o, 0, 0, 0);
  }
}
#endif

constexpr int TK = 64;  // k of a stage: two MFMA k-steps

template <int BM_, int BN_, int WM_, int WN_, int NS_, int BLOCKS_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int BLOCKS = BLOCKS_;  // blocks per compute unit
  static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  static constexpr int NTHREADS = 64 * NW;
  static constexpr int FM = WM / 16, FN = WN / 16;
  static constexpr int A_INSTR = BM * TK / 512, B_INSTR = BN * TK / 512;  // 1 KB pieces
  // pieces of one wave, where they do not come out even the most; and what
  // every wave has at least
  static constexpr int A_LOADS = (A_INSTR + NW - 1) / NW, B_LOADS = (B_INSTR + NW - 1) / NW;
  static constexpr int LOADS = A_LOADS + B_LOADS, LOADS_MIN = A_INSTR / NW + B_INSTR / NW;
  static constexpr int A_BYTES = BM * TK * 2, STAGE_BYTES = (BM + BN) * TK * 2;
  static_assert(A_INSTR * 512 == BM * TK && B_INSTR * 512 == BN * TK, "whole pieces");
  static_assert((NS - 1) * LOADS_MIN <= 63, "vmcnt range");
  static_assert(BLOCKS * NS * STAGE_BYTES <= 160 * 1024, "LDS of a compute unit");
};

// f(0) .. f(N - 1) with compile-time arguments: unrolled whatever the size.
template <class F, int... I>
__device__ __forceinline__ void unrolled(F &&f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(F &&f) {
  unrolled(f, std::make_integer_sequence<int, N>());
}

template <int N>
__device__ __forceinline__ void wait_vmcnt_imm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Position of 16-byte chunk c in k-row k of an operand staged as it lies in
// memory, R columns wide.
template <int R>
__device__ __forceinline__ int swz(int k) {
  return R >= 128 ? ((k & 3) << 1) | (((k >> 3) & 1) << 3) : R >= 64 ? (k & 3) << 1 : (k & 1) << 1;
}

// Number of this block's tile among `total`. The hardware sends block b to XCD
// b % 8: each XCD takes a contiguous run of the first `live` tiles, and then
// of the others, so that the live ones are spread evenly.
__device__ __forceinline__ int tile_of_block(int b, int total, int live) {
  const int x = b % 8, j = b / 8;
  const int live_before = x * (live / 8) + min(x, live % 8);
  const int live_here = live / 8 + (x < live % 8);
  if (j < live_here) return live_before + j;
  const int before = x * (total / 8) + min(x, total % 8);
  return live + before - live_before + (j - live_here);
}
// Tiles go in columns of 8 m-tiles, so that those in flight on one XCD share
// operand rows in its L2.
__device__ __forceinline__ void tile_at(int t, int m_tiles, int n_tiles, int &mt, int &nt) {
  constexpr int GROUP = 8;
  const int full = GROUP * n_tiles;
  const int g = t / full, first = g * GROUP, size = min(GROUP, m_tiles - first);
  t -= g * full;
  mt = first + t % size;
  nt = t / size;
}

template <class D, int MODE, class C, bool GATHER>
__global__ __launch_bounds__(C::NTHREADS, (C::BLOCKS * C::NW + 3) / 4) void gemm_kernel(
    const GemmArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int BM = C::BM, BN = C::BN, NS = C::NS;
  constexpr bool A_TR = MODE == WGRAD, B_TR = MODE == DGRAD || MODE == WGRAD;
  static_assert((!A_TR || BM >= 32) && (!B_TR || BN >= 32), "chunks for swz to permute");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * C::STAGE_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool grouped = g.r.num_experts > 0;

  const uint32_t block = blockIdx.x + g.block0;
  int mt, nt, e = 0, seg0 = 0;
  int64_t k_row0 = 0;  // WGRAD: first row of the expert, or of the k range
  int split = 0, k0 = 0;  // the others: first k of the range
  int K = g.K;
  if constexpr (MODE == WGRAD) {
    // one expert and projection after the other, all its tiles together
    const int per = g.m_tiles * g.n_tiles;
    const int chunk = block / per % (g.segs * max(1, g.r.num_experts));
    split = block / per / (g.segs * max(1, g.r.num_experts));
    tile_at(tile_of_block(block % per, per, per), g.m_tiles, g.n_tiles, mt, nt);
    e = chunk / g.segs;
    seg0 = chunk % g.segs;
    if (grouped) {
      const int64_t p0 = g.r.padded_offsets[e], cnt = g.r.counts[e];
      k_row0 = min(max(p0, (int64_t)0), g.r.rows);
      K = (int)min(max(cnt, (int64_t)0), g.r.rows - k_row0);
      if (GATHER && g.a_rows == 0) K = 0;  // not even a row 0 to gather
    }
  } else {
    int live = g.m_tiles;  // m-tiles with rows of the experts here
    if (g.tile_map) {
      live = g.tile_map[g.m_tiles].x;
    } else if (grouped) {
      const int64_t end = g.r.padded_offsets[g.r.num_experts];
      live = (int)min((int64_t)g.m_tiles, (max(end, (int64_t)0) + BM - 1) / BM);
    }
    const int per = g.m_tiles * g.n_tiles;  // split: all tiles of one k range together
    split = block / per;
    const int t = tile_of_block(block % per, per, live * g.n_tiles);
    if (t < live * g.n_tiles) {
      tile_at(t, live, g.n_tiles, mt, nt);
    } else {
      mt = t / g.n_tiles;
      nt = t % g.n_tiles;
    }
  }
  int m0 = mt * BM, m_end = g.M;  // rows of the tile that are its own: below m_end
  if (MODE != WGRAD && g.tile_map) {
    const int4 tile = g.tile_map[mt];
    m0 = tile.x;
    m_end = tile.y;
    if (m0 >= m_end) return;
  }
  const int n0 = nt * (MODE == GATED ? BN / 2 : BN);  // column of C

  if constexpr (MODE != WGRAD) {
    if (grouped) {
      e = g.r.m_indices[m0];
      if (e < 0 || e >= g.r.num_experts || g.a_rows == 0) {  // no entry here: zeros
        constexpr int RUNS = (MODE == GATED ? BN / 2 : BN) / 8;
        const s16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int i = threadIdx.x; i < BM * RUNS; i += C::NTHREADS) {
          const int64_t m = m0 + i / RUNS;
          const int n = n0 + i % RUNS * 8;
          if (m >= m_end || n >= g.N) continue;
          store8_raw(g.c0 + m * g.ldc0, n, g.N, zero);
          if (MODE <= LINEAR && g.pre) {
            store8_raw(g.pre + m * g.ldp, n, g.N, zero);
            if (MODE == GATED) store8_raw(g.pre + m * g.ldp + g.N, n, g.N, zero);
          }
        }
        return;
      }
    }
  }
  if (g.partial) {
    if (MODE == WGRAD) k_row0 = split * (int64_t)g.k_split; else k0 = split * g.k_split;
    K = min(g.k_split, K - split * g.k_split);
  }
  const uint16_t *b0 = g.b0, *b1 = g.b1;
  if (MODE != WGRAD) {
    b0 += e * g.b_stride0;
    b1 += e * g.b_stride1;
  }
  const int seg_stages = (K + TK - 1) / TK;
  const int nk = seg_stages * (MODE == DGRAD ? g.segs : 1);
  // last 8-element piece of an operand whose m or n is contiguous
  const int m_last = ((g.M + 7) & ~7) - 8, n_last = ((g.N + 7) & ~7) - 8;
  const uint32_t magic = g.top_k_magic, shift = g.top_k_shift;
  auto gathered_row = [&](int32_t entry) MOE_INLINE {  // a bad entry reads row 0, in bounds
    const uint32_t t = magic ? __umulhi((uint32_t)entry, magic) >> shift : (uint32_t)entry;
    return t < (uint64_t)g.a_rows ? t : 0u;
  };

  // Where this wave's pieces come from. A piece is 1 KB, 16 bytes a lane:
  // number q * NW + wave of the A side for q < A_LOADS, of the B side after
  // those. A lane reads at the operand's base of the stage (uniform, advanced
  // by a stage at a time) plus off[q] bytes.
  auto is_a = [&](int q) MOE_INLINE { return q < C::A_LOADS; };
  auto number = [&](int q) MOE_INLINE {
    return (is_a(q) ? q : q - C::A_LOADS) * C::NW + wave;
  };
  auto exists = [&](int q) MOE_INLINE {
    return is_a(q) ? C::A_INSTR % C::NW == 0 || number(q) < C::A_INSTR
                   : C::B_INSTR % C::NW == 0 || number(q) < C::B_INSTR;
  };
  // GATED: B rows alternate, 16 of the gate's and 16 of the other's. A wave's
  // pieces are all of one projection.
  static_assert(MODE != GATED || C::NW * 8 % 32 == 0, "one projection for a wave");
  const bool up = MODE == GATED && ((wave * 8) >> 4 & 1);
  const int64_t ldb = up ? g.ldb1 : g.ldb0;
  const uint8_t *a_base, *b_base, *b_next = nullptr;
  int64_t a_step, b_step;
  if constexpr (A_TR) {
    a_base = reinterpret_cast<const uint8_t *>(g.a + k_row0 * g.lda + seg0 * g.a_seg);
    a_step = TK * g.lda * 2;
  } else {
    a_base = reinterpret_cast<const uint8_t *>(g.a + (GATHER ? 0 : m0 * g.lda) + k0);
    a_step = TK * 2;
  }
  if constexpr (MODE == WGRAD) {
    b_base = reinterpret_cast<const uint8_t *>(b0 + (GATHER ? 0 : k_row0 * ldb));
    b_step = GATHER ? 0 : TK * ldb * 2;
  } else if constexpr (MODE == DGRAD) {
    b_base = reinterpret_cast<const uint8_t *>(b0 + k0 * ldb);
    b_next = reinterpret_cast<const uint8_t *>(b1 + k0 * ldb);
    b_step = TK * ldb * 2;
  } else {
    b_base = reinterpret_cast<const uint8_t *>((up ? b1 : b0) + n0 * ldb + k0);
    b_step = TK * 2;
  }
  // a lane's row and 8-element chunk in a piece of an operand with contiguous
  // k: 128-byte rows, chunk c at c ^ (row & 7)
  const int piece_row = lane >> 3, piece_chunk = (lane & 7) ^ (lane >> 3);
  uint32_t off[C::LOADS];
  auto start = [&]() MOE_INLINE {
#pragma unroll
    for (int q = 0; q < C::LOADS; ++q) {
      const int id = number(q);
      if (is_a(q) && A_TR) {
        constexpr int PER = BM / 8;  // chunks of a k-row
        const int k = (id * 64 + lane) / PER, c = (lane % PER) ^ swz<BM>(k);
        off[q] = (uint32_t)(k * g.lda + min(m0 + c * 8, m_last)) * 2;
      } else if (is_a(q)) {
        const int row = min(m0 + id * 8 + piece_row, g.M - 1);
        const int64_t at = GATHER ? gathered_row(g.r.row_entry[row]) : row - m0;
        off[q] = (uint32_t)(at * g.lda + piece_chunk * 8) * 2;
      } else if (B_TR) {
        constexpr int PER = BN / 8;
        const int k = (id * 64 + lane) / PER, c = (lane % PER) ^ swz<BN>(k);
        // gathered: the row is added when its entry is known
        off[q] = (uint32_t)((MODE == WGRAD && GATHER ? 0 : k * ldb) + min(n0 + c * 8, n_last)) * 2;
      } else {
        int j = id * 8 + piece_row;
        if (MODE == GATED) j = (j >> 5) * 16 + (j & 15);
        off[q] = (uint32_t)(min(j, g.N - 1 - n0) * ldb + piece_chunk * 8) * 2;
      }
    }
  };
  // Whether piece q of a stage with `left` k from its start on lies past them:
  // such pieces, a stage's tail or stages after the last, load zeros.
  auto past = [&](int q, int left) MOE_INLINE {
    if (is_a(q) && A_TR) return lane / (BM / 8) >= left - number(q) * (512 / BM);
    if (!is_a(q) && B_TR) return lane / (BN / 8) >= left - number(q) * (512 / BN);
    return piece_chunk * 8 >= left;
  };
  // WGRAD with gathered x: the entry of the row that piece q of stage s reads,
  // and those of the next stage to be issued
  int32_t entry[C::B_LOADS];
  auto entry_of = [&](int s, int q) MOE_INLINE {
    const int k = number(q) * (512 / BN) + lane / (BN / 8);
    return g.r.row_entry[k_row0 + min(s * TK + k, K - 1)];
  };
  auto fetch_entries = [&](int s) MOE_INLINE {
    if constexpr (MODE == WGRAD && GATHER) {
#pragma unroll
      for (int q = C::A_LOADS; q < C::LOADS; ++q) entry[q - C::A_LOADS] = entry_of(s, q);
    }
  };
  // Stages are issued in order, each followed by next_stage.
  int left = K;  // of the segment, from the next stage to be issued on
  auto issue_piece = [&](int s, int q) MOE_INLINE {
    if (!exists(q)) return;
    uint32_t o = off[q];
    if (MODE == WGRAD && GATHER && !is_a(q))
      o += (uint32_t)(gathered_row(entry[q - C::A_LOADS]) * ldb) * 2;
    o = past(q, left) ? PAST : o;
    lds_piece<A_TR || B_TR>(is_a(q) ? a_base : b_base, o,
                            smem + (s % NS) * C::STAGE_BYTES + (is_a(q) ? 0 : C::A_BYTES) +
                                number(q) * 1024);
  };
  auto next_stage = [&](int s) MOE_INLINE {  // after stage s
    a_base += a_step;
    b_base += b_step;
    left -= TK;
    if (MODE == DGRAD) {
      const bool second = g.segs > 1 && s + 1 == seg_stages;
      a_base = second ? reinterpret_cast<const uint8_t *>(g.a + m0 * g.lda + k0 + g.a_seg)
                      : a_base;
      b_base = second ? b_next : b_base;
      left = second ? K : left;
    }
  };

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int wm = (wave / C::WAVES_N) * C::WM, wn = (wave % C::WAVES_N) * C::WN;
  const int fr = lane & 15, fq = lane >> 4;

  s16x8 fa[2][C::FM], fb[2][C::FN];
  auto frag_k = [&](const uint8_t *t, int row, int ks) MOE_INLINE {
    return *reinterpret_cast<const s16x8 *>(t + (row + fr) * 128 +
                                            (((ks * 4 + fq) ^ (fr & 7)) * 16));
  };
  auto frag_tr = [&](const uint8_t *t, uint32_t lane_off, int f, int ks, auto width) MOE_INLINE {
    constexpr int R = decltype(width)::value;
    const uint8_t *p = t + (lane_off ^ (f * 32)) + ks * 32 * (R * 2);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr_t)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr_t)(p + 4 * (R * 2)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // a lane's k-row and swizzled chunk of the first fragment, transposed reads
  auto lane_tr = [&](int first, auto width) MOE_INLINE {
    constexpr int R = decltype(width)::value;
    const int k = fq * 8 + (fr >> 2);
    return (uint32_t)(k * (R * 2) + (((first >> 3) + ((fr & 3) >> 1)) ^ swz<R>(k)) * 16 +
                      (fr & 1) * 8);
  };
  const uint32_t a_lane = lane_tr(wm, std::integral_constant<int, BM>());
  const uint32_t b_lane = lane_tr(wn, std::integral_constant<int, BN>());
  // fragment f of a k-step: the N side's first, then the M side's
  auto read_frag = [&](int s, int ks, int set, int f) MOE_INLINE {
    const uint8_t *As = smem + (s % NS) * C::STAGE_BYTES, *Bs = As + C::A_BYTES;
    if (f < C::FN) {
      if constexpr (B_TR)
        fb[set][f] = frag_tr(Bs, b_lane, f, ks, std::integral_constant<int, BN>());
      else
        fb[set][f] = frag_k(Bs, wn + 16 * f, ks);
    } else {
      const int i = f - C::FN;
      if constexpr (A_TR)
        fa[set][i] = frag_tr(As, a_lane, i, ks, std::integral_constant<int, BM>());
      else
        fa[set][i] = frag_k(As, wm + 16 * i, ks);
    }
  };
  // The wait in wait_stage has drained this set's LDS reads, which the
  // compiler cannot see: naming the registers here keeps it from waiting
  // for the next set's reads as well.
  auto settle = [&](int set) MOE_INLINE {
#pragma unroll
    for (int i = 0; i < C::FM; ++i) asm volatile("" : "+v"(fa[set][i]));
#pragma unroll
    for (int j = 0; j < C::FN; ++j) asm volatile("" : "+v"(fb[set][j]));
  };
  // The entries too: the compiler counts only the loads it knows, so it would
  // wait for pieces issued after the entries before it uses them.
  auto settle_entries = [&]() MOE_INLINE {
    if constexpr (MODE == WGRAD && GATHER) {
#pragma unroll
      for (int q = 0; q < C::B_LOADS; ++q) asm volatile("" : "+v"(entry[q]));
    }
  };
  // One MFMA k-step on `set`. Between the MFMAs, one at a time, go the fragment
  // reads of k-step rks of stage rs (over the first three quarters) and, with
  // ISSUE, the pieces of stage `is`: an MFMA holds its pipe for 16 cycles, in
  // which the wave can issue the few other instructions.
  auto step = [&](int set, int rs, int rks, auto issue_tag, int is) MOE_INLINE {
    constexpr bool ISSUE = decltype(issue_tag)::value;
    constexpr int FRAGS = C::FM + C::FN, MFMAS = C::FM * C::FN;
    constexpr int SPAN = MFMAS > FRAGS ? MFMAS * 3 / 4 : MFMAS;
    unrolled<MFMAS>([&](auto tc) MOE_INLINE {
      constexpr int t = decltype(tc)::value, i = t / C::FN, j = t % C::FN;
      // read f goes before MFMA f * SPAN / FRAGS, piece q before q * MFMAS / LOADS
      constexpr int F0 = (t * FRAGS + SPAN - 1) / SPAN, F1 = ((t + 1) * FRAGS + SPAN - 1) / SPAN;
#pragma unroll
      for (int f = F0; f < (F1 < FRAGS ? F1 : FRAGS); ++f) read_frag(rs, rks, set ^ 1, f);
      if constexpr (ISSUE) {
        constexpr int Q0 = (t * C::LOADS + MFMAS - 1) / MFMAS,
                      Q1 = ((t + 1) * C::LOADS + MFMAS - 1) / MFMAS;
#pragma unroll
        for (int q = Q0; q < (Q1 < C::LOADS ? Q1 : C::LOADS); ++q) issue_piece(is, q);
      }
      acc[i][j] = D::mfma(fb[set][j], fa[set][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (ISSUE) {
      fetch_entries(is + 1);
      next_stage(is);
    }
  };
  // The oldest stage in flight has landed for every wave (NS - 2 younger ones
  // may not have), and every wave has read the buffer that is filled next.
  auto wait_stage = [&]() MOE_INLINE {
    wait_vmcnt_imm<C::LOADS_MIN *(NS - 2)>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  if (nk > 0) {
    start();
    // all buffers are free: NS stages at once, their entries before them
    int32_t first[NS][C::B_LOADS];
    if constexpr (MODE == WGRAD && GATHER) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int q = C::A_LOADS; q < C::LOADS; ++q) first[s][q - C::A_LOADS] = entry_of(s, q);
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int q = 0; q < C::B_LOADS; ++q) asm volatile("" : "+v"(first[s][q]));
    }
    unrolled<NS>([&](auto sc) MOE_INLINE {
      constexpr int s = decltype(sc)::value;
      if constexpr (MODE == WGRAD && GATHER) {
#pragma unroll
        for (int q = 0; q < C::B_LOADS; ++q) entry[q] = first[s][q];
      }
#pragma unroll
      for (int q = 0; q < C::LOADS; ++q) issue_piece(s, q);
      next_stage(s);
    });
    fetch_entries(NS);
    wait_vmcnt_imm<C::LOADS_MIN *(NS - 1)>();
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int f = 0; f < C::FM + C::FN; ++f) read_frag(0, 0, 0, f);
    // The second k-step of a stage reads the next stage's first fragments and
    // issues the stage NS ahead. After the last stage both go on with zeros,
    // so that the loop has no branches.
#pragma unroll 1
    for (int s = 0; s < nk; ++s) {
      step(0, s, 1, std::false_type(), 0);
      wait_stage();
      settle(1);
      settle_entries();
      step(1, s + 1, 0, std::true_type(), s + NS);
    }
  }

  // Epilogue. A lane holds row fr and columns 4 fq .. 4 fq + 3 of every 16 x 16
  // tile. Each wave turns 16 rows at a time through LDS of its own (fp32, 16-byte
  // chunk c of row r at c ^ r) so that a lane gets 8 consecutive columns of
  // a row: 16-byte loads and stores that fill whole lines, and the epilogue's
  // column vectors stay the same for all rows. What it reads for its rows is
  // loaded before the first of them: one latency, not one for each run of rows.
  constexpr int OUT = MODE == GATED ? C::WN / 2 : C::WN;  // columns of a wave
  constexpr int CH = OUT / 4, LPR = OUT / 8;               // chunks, lanes in a row
  constexpr int PASSES = LPR > 4 ? LPR / 4 : 1, ROWS = 16 / PASSES;
  static_assert(C::NW * 16 * OUT * 4 <= NS * C::STAGE_BYTES, "the waves' LDS");
  float *turn_lds = reinterpret_cast<float *>(smem) + wave * (16 * OUT);
  const int tr = lane / LPR, tc = lane % LPR;  // row of a pass, 8-column run
  const bool on = LPR * 16 >= 64 || lane < LPR * 16;
  auto turn_in = [&](int j, f32x4 v) MOE_INLINE {
    *reinterpret_cast<f32x4 *>(turn_lds + fr * OUT + (((4 * j + fq) ^ fr) & (CH - 1)) * 4) = v;
  };
  auto turn_out = [&](int p) MOE_INLINE {
    const int r = (p * ROWS + tr) & 15;
    const float *row = turn_lds + r * OUT;
    const f32x4 a = *reinterpret_cast<const f32x4 *>(row + (((2 * tc) ^ r) & (CH - 1)) * 4);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(row + (((2 * tc + 1) ^ r) & (CH - 1)) * 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // LDS keeps a wave's accesses in order; the compiler must too, between what
  // other lanes wrote and this lane reads.
  auto turn_order = [&]() MOE_INLINE {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  const int n = n0 + (MODE == GATED ? wn >> 1 : wn) + tc * 8;  // this lane's columns
  const bool cols = on && n < g.N;
  auto row_of = [&](int i, int p) MOE_INLINE {
    return (int64_t)m0 + wm + 16 * i + p * ROWS + tr;
  };
  uint32_t real = 0xffffffffu;  // a bit a run: the row holds an entry
  if (MODE != WGRAD && grouped) {
    real = 0;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (row_of(i, p) < m_end && g.r.m_indices[row_of(i, p)] == e) real |= 1u << (i * PASSES + p);
  }
  auto is_real = [&](int i, int p) MOE_INLINE { return (real >> (i * PASSES + p) & 1) != 0; };
  static_assert(C::FM * PASSES <= 32, "a bit a run");
  s16x8 residual[MODE == LINEAR ? C::FM * PASSES : 1];
  if (MODE == LINEAR && g.res && !g.partial) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int p = 0; p < PASSES; ++p)
        if (cols && row_of(i, p) < m_end)
          residual[i * PASSES + p] = load8_raw(g.res + row_of(i, p) * g.ldr, n, g.N);
  }
  wait_vmcnt_imm<0>();  // with them the zeros still on their way to LDS
  __syncthreads();
  const f32x8 zero8 = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  uint16_t *out = MODE == WGRAD ? (seg0 ? g.c1 + e * g.c_stride1 : g.c0 + e * g.c_stride0) : g.c0;
  const int64_t ldc = MODE == WGRAD && seg0 ? g.ldc1 : g.ldc0;
  if (g.partial) {  // a range's sums as they are; join_kernel does the rest
    const int width = MODE == GATED ? 2 * g.N : g.N;
    float *part = g.partial + (split * (int64_t)(MODE == WGRAD ? g.segs : 1) + seg0) * g.M * width;
    constexpr int SIDES = MODE == GATED ? 2 : 1;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int side = 0; side < SIDES; ++side) {
        turn_order();
#pragma unroll
        for (int j = 0; j < C::FN / SIDES; ++j) turn_in(j, acc[i][SIDES * j + side]);
        turn_order();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
          const f32x8 v = turn_out(p);
          if (cols && row_of(i, p) < m_end)
            store8_f32(part + row_of(i, p) * width + side * g.N, n, g.N, v);
        }
      }
    return;
  }
  if constexpr (MODE == GATED) {
    // what is turned: h, and with pre the two projections as well
    auto rows_out = [&](int i, auto value, uint16_t *to, int64_t ld, int width, int col)
        MOE_INLINE {
      turn_order();
#pragma unroll
      for (int j = 0; j < C::FN / 2; ++j) turn_in(j, value(acc[i][2 * j], acc[i][2 * j + 1]));
      turn_order();
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const f32x8 v = turn_out(p);
        const int64_t m = row_of(i, p);
        if (cols && m < m_end)
          store8<D>(to + m * ld, col, width, is_real(i, p) ? v : zero8);
      }
    };
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      rows_out(i, [&](f32x4 gt, f32x4 up4) MOE_INLINE {
        f32x4 h = act_value(gt, g.act);
#pragma unroll
        for (int v = 0; v < 4; ++v) h[v] *= up4[v];
        return h;
      }, out, ldc, g.N, n);
      if (g.pre) {
        rows_out(i, [&](f32x4 gt, f32x4) MOE_INLINE { return gt; }, g.pre, g.ldp, g.N, n);
        rows_out(i, [&](f32x4, f32x4 up4) MOE_INLINE { return up4; }, g.pre + g.N, g.ldp, g.N, n);
      }
    }
  } else {
    f32x8 bias = zero8;
    if (MODE == LINEAR && g.bias && cols) bias = load8<D>(g.bias + e * g.bias_stride, n, g.N);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      turn_order();
#pragma unroll
      for (int j = 0; j < C::FN; ++j) turn_in(j, acc[i][j]);
      turn_order();
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        f32x8 z = turn_out(p);
        const int64_t m = row_of(i, p);
        if (!cols || m >= m_end) continue;
        if constexpr (MODE == LINEAR) {
#pragma unroll
          for (int v = 0; v < 8; ++v) z[v] += bias[v];
          if (g.pre) store8<D>(g.pre + m * g.ldp, n, g.N, is_real(i, p) ? z : zero8);
          z = act_value(z, g.act);
          if (g.res) {
            const f32x8 r = unpack8<D>(residual[i * PASSES + p]);
#pragma unroll
            for (int v = 0; v < 8; ++v) z[v] += r[v];
          }
        }
        store8<D>(out + m * ldc, n, g.N, is_real(i, p) ? z : zero8);
      }
    }
  }
#endif
}

}  // namespace moe_ffn
