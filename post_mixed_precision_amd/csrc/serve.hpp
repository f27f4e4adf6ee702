// Host-side launchers of the serving kernels: 4-bit products, the same grouped
// by expert, and token log probabilities (internal to libslim).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4_plan.hpp"

namespace slim {

// ---- 4-bit products ----
hipError_t launch_pack4(const uint8_t *codes, const float *scale, const float *zero, int64_t e, int64_t n, int64_t m,
                        int group, uint32_t *packed, int32_t *info, hipStream_t st);

struct Q4Args {
  const void *X;             // [xrows, m]
  int64_t xrows, m;
  const uint32_t *W;         // e packed matrices
  int64_t n, r;              // output rows of a matrix; rows of Y
  const int32_t *offsets;    // e + 1 row bounds, or null: one matrix for all rows
  const int32_t *rows;       // r rows of X, or null: row i reads X's row i
  const float *row_scale;    // r factors, or null
  void *Y;                   // [r, n]
  int e, group;
  bool xbf16, ybf16;
};
// gather: `rows` may be given (the workspace then does for calls without it as well)
size_t q4_ws_bytes(int64_t xrows, int64_t r, int64_t e, int64_t n, int64_t m, int group, bool xbf16, bool gather);
hipError_t launch_q4(const Q4Args &a, void *ws, hipStream_t st);

// ---- Token log probabilities ----
struct LogprobPlan {
  bool wide;                 // workgroups of 16 waves, not 4
  int nseg;                  // segments a row is split into
  size_t ws_bytes;           // their statistics and best entries (0 for one segment)
};
LogprobPlan logprob_plan(int64_t t, int64_t v, int top, bool bf16);
hipError_t launch_logprobs(const void *L, bool bf16, int64_t t, int64_t v, int64_t ld, const int64_t *ids, int top,
                           float *logprob, float *entropy, float *top_logprob, int32_t *top_id, void *ws,
                           const LogprobPlan &p, hipStream_t st);

}  // namespace slim
