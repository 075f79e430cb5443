// ffn_host.hpp - the host side that the entry points share: workspaces, operands of
// products, plans, checks of matrices.
#pragma once

#include "ffn.hpp"

namespace moe_ffn {

constexpr int64_t MAX_ROWS = MOE_FFN_MAX_ROWS;

inline int round8(int v) { return (v + 7) & ~7; }
inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// Hands out the workspace in 256-byte aligned parts. A dry one only counts
// them: the same code sizes the workspace and then runs the call.
struct Arena {
  uint8_t *base;
  bool dry;
  size_t used;
  uint16_t *take(size_t bytes) {
    uint8_t *p = dry ? nullptr : base + used;
    used += align256(bytes);
    return reinterpret_cast<uint16_t *>(p);
  }
};

// An operand of a product: the matrix itself where its 16-byte pieces are
// aligned, else a padded copy in the workspace. `mats` matrices of [rows,
// cols].
struct Operand {
  const uint16_t *p;
  int64_t ld, stride;
};
Operand operand(const moe_matrix &m, int64_t rows, int cols, int mats, Arena &a, hipStream_t st,
                int *status, bool copy = false);

// How a product runs: its tile, and the ranges that its k is split into.
struct Plan {
  int kind, splits;
};
// Plan of a product whose M is the call's rows; forward: one with rows of W as its
// second operand.
Plan row_plan(const moe_expert_rows &r, bool forward, int64_t M, int64_t N, int64_t K);
// Runs a product by its plan. `width`: the partial sums of a row of C. `tile_m`: the
// alignment of the layout, 0 for a dense product.
int run_product(int dtype, int mode, const Plan &plan, GemmArgs &g, int width, int tile_m,
                Arena &ws, hipStream_t st);

int check_matrix(const moe_matrix &m, int64_t rows, int cols, int mats, bool optional);

#define MOE_TRY(x)              \
  do {                          \
    const int st_ = (x);        \
    if (st_ != MOE_OK) return st_; \
  } while (0)

template <class Args>
static int64_t sized(const Args *a, int check, int (*run)(const Args *, Arena &, hipStream_t)) {
  if (check != MOE_OK) return -1;
  Arena ws = {nullptr, true, 0};
  run(a, ws, nullptr);
  return (int64_t)ws.used;
}
template <class Args>
static int checked_run(const Args *a, int check, int (*run)(const Args *, Arena &, hipStream_t),
                       void *workspace, size_t bytes, void *stream) {
  MOE_TRY(check);
  const int64_t need = sized(a, MOE_OK, run);
  if (need > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || bytes < (size_t)need))
    return MOE_ERR_WORKSPACE;
  Arena ws = {(uint8_t *)workspace, false, 0};
  return run(a, ws, (hipStream_t)stream);
}

}  // namespace moe_ffn
