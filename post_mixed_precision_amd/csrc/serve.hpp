// Host-side launchers of the serving kernels: 4-bit products, the same grouped
// by expert, token log probabilities, the 4-bit key/value cache with its
// attention, and the verification of drafted tokens (internal to libslim).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kv4_plan.hpp"
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

// ---- 4-bit key/value cache ----
struct Kv4Rows {             // [t, heads, dim] of the call's type, strides in elements
  const void *p;
  int64_t heads, row, head;
  bool vec;                  // rows and heads start at 16-byte boundaries
};
struct Kv4Append {
  Kv4Rows q, k, v;           // q.p may be null (q.heads 0)
  void *q_out;               // [t, q.heads, dim]
  const int32_t *slots, *positions;
  const float *rotary;       // [npos, rot] or null: cosines, then sines
  uint32_t *cache;
  int64_t t, pages, npos;
  int dim, group, page, page_log, rot;
  bool bf16, interleaved;
  bool rvec;                 // the table's rows start at 16-byte boundaries
};
hipError_t launch_kv4_append(const Kv4Append &a, hipStream_t st);
hipError_t launch_kv4_read(const int32_t *slots, int64_t t, const uint32_t *cache, int64_t pages, int64_t heads,
                           int dim, int group, int page, void *k, void *v, bool bf16, hipStream_t st);

struct Kv4Args {
  const void *q;             // [tq, hq, dim]
  void *out;                 // [tq, hq, dim]
  const uint32_t *cache;
  const int32_t *table;      // [b, per] pages of each sequence
  const int32_t *lengths;    // [b]
  const int32_t *offsets;    // b + 1 bounds of the sequences' query tokens, or null: ql each
  int b, tq, ql, hq, hkv, g, pages, per;   // g = hq / hkv
  int cap;                   // tokens a row of the table can name
  int dim, group, page;
  float scale;
  bool causal, qbf16, obf16;
};
struct Kv4Cut {
  float *part;               // partial results
  int tm, tm_log;            // a power of two
  int tiles;                 // row tiles a sequence, without offsets
  int slots, extra, least;
};
hipError_t launch_kv4_attention(const Kv4Args &a, void *ws, const Kv4Plan &p, hipStream_t st);

// ---- Verification of drafted tokens ----
struct DraftArgs {
  const void *target, *draft;          // [b, k + 1, v] and [b, k, v] or null, strides in elements
  int64_t t_seq, t_row, d_seq, d_row;
  const int64_t *tokens;               // [b, k]
  const float *uniform;                // [b, k + 1]
  int32_t *accepted;                   // [b]
  int64_t *ids;                        // [b, k + 1]
  int64_t b, v;
  int k;
  double temperature;
  bool bf16;
};
struct DraftPlan {
  bool few;                  // segments of 2048 entries, not 8192
  int nseg;                  // segments a row is cut into
  int runs, each;            // runs its masses are summed over; of those, a workgroup's
  size_t ws_bytes;
};
DraftPlan draft_plan(int64_t b, int k, int64_t v);
hipError_t launch_verify_draft(const DraftArgs &a, void *ws, const DraftPlan &p, hipStream_t st);

}  // namespace slim
