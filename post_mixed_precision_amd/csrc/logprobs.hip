// Log probabilities of given tokens, the entropy of their rows and the best
// entries of each row, in one pass over the logits (gfx950).
//
//   M = max_j x_j,  S = sum_j e^(x_j - M),  W = sum_j e^(x_j - M) (x_j - M)
//   logprob = x_id - M - ln S,   entropy = ln S - W / S,
//   top: the entries with the largest x_j, equal ones by ascending j.
//
// Running sums: a lane keeps (M, S, W) of what it has read; when its maximum
// moves by D = M - M', S' = S e^D and W' = (W + D S) e^D, which is also how
// lanes, waves and the segments of a row are joined.  Everything is float32.
// An entry of -inf adds nothing (its product with e^-inf is kept from becoming
// NaN by bounding x - M from below); a row with a NaN or +inf makes S NaN, and
// a row of -inf only leaves S = 0: such a row has no distribution and gives NaN.
//
// Best entries: every wave keeps the largest 64 keys (ordered value bits, then
// the inverted index, so that a larger key is a better entry) sorted over its
// lanes.  A candidate above the top-th key is broadcast and inserted by
// shifting the lanes below it; of N values in random order only about
// top ln(N / top) get that far.  The set and its order depend on the keys alone.
#include "common.hpp"
#include "serve.hpp"

namespace slim {

namespace {

constexpr int LP_WAVES = 4;
constexpr float LOG2E = 1.44269504088896340736f;

typedef unsigned long long key_t64;

struct Stats {
  float m, s, w;
};

__device__ __forceinline__ float exp_diff(float d) { return __builtin_amdgcn_exp2f(d * LOG2E); }

// a joined with b.  A side that has added nothing (s = 0) does not count: its
// maximum is the start value.
__device__ __forceinline__ Stats join(const Stats &a, const Stats &b) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf(a.m - m, -1e30f), db = fmaxf(b.m - m, -1e30f);
  const float ea = exp_diff(a.m - m), eb = exp_diff(b.m - m);
  Stats r;
  r.m = m;
  r.s = fmaf(a.s, ea, b.s * eb);
  r.w = fmaf(fmaf(da, a.s, a.w), ea, fmaf(db, b.s, b.w) * eb);
  return r;
}

__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);          // -0 counts as 0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ key_t64 make_key(float v, uint32_t idx) {
  return ((key_t64)order_bits(v) << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ key_t64 lane_key(key_t64 k, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)k, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(k >> 32), lane);
  return ((key_t64)hi << 32) | lo;
}

// The wave's best keys, descending over the lanes; thr = key number top - 1.
struct Best {
  key_t64 list, thr;
  __device__ __forceinline__ void clear() { list = 0, thr = 0; }
  __device__ __forceinline__ void insert(key_t64 c, int top) {
    const int lane = threadIdx.x & 63;
    const int pos = __popcll(__ballot(list > c));
    const key_t64 up = ((key_t64)(uint32_t)__shfl_up((int)(uint32_t)(list >> 32), 1, 64) << 32) |
                       (uint32_t)__shfl_up((int)(uint32_t)list, 1, 64);
    list = lane < pos ? list : lane == pos ? c : up;
    thr = lane_key(list, top - 1);
  }
  // Every lane offers one key (0: none).
  __device__ __forceinline__ void offer(key_t64 mine, int top) {
    uint64_t left = __ballot(mine > thr);
    while (left) {
      const int src = __ffsll((unsigned long long)left) - 1;
      const key_t64 c = lane_key(mine, src);
      insert(c, top);
      left &= left - 1;
      left &= __ballot(mine > thr);
    }
  }
};

template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const void *p, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (BF16) x[0] = bf16_bits_to_f32(*(const uint16_t *)p);
    else x[0] = *(const float *)p;
  } else if constexpr (BF16) {
    const uint4 v = *(const uint4 *)p;
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(u[e] << 16);
      x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  } else {
    const float4 v = *(const float4 *)p;
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
}

// VEC entries of this lane, the first of them entry idx of the row.
template <int VEC>
__device__ __forceinline__ void take(const float (&x)[VEC], uint32_t idx, bool has, int top, Stats &st, Best &best) {
  float b = x[0];
#pragma unroll
  for (int e = 1; e < VEC; ++e) b = fmaxf(b, x[e]);
  if (has) {
    if (b > st.m) {
      const float d = st.m - b, ed = exp_diff(d);
      st.w = fmaf(fmaxf(d, -1e30f), st.s, st.w) * ed;
      st.s *= ed;
      st.m = b;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = x[e] - st.m;
      const float ex = exp_diff(d);
      st.s += ex;
      st.w = fmaf(ex, fmaxf(d, -1e30f), st.w);
    }
  }
  if (top) {
    const float thr = from_order_bits((uint32_t)(best.thr >> 32));   // NaN while the list is not full
    if (__any(has && !(b < thr))) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) best.offer(has && !(x[e] != x[e]) ? make_key(x[e], idx + e) : 0, top);
    }
  }
}

__device__ __forceinline__ Stats wave_join(Stats st) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    Stats o;
    o.m = __shfl_xor(st.m, d, 64);
    o.s = __shfl_xor(st.s, d, 64);
    o.w = __shfl_xor(st.w, d, 64);
    st = join(st, o);
  }
  return st;
}

// Row results from its joined statistics (one wave).
template <bool BF16>
__device__ __forceinline__ void finish(const Stats &st, const Best &best, const void *row, int64_t v, int64_t a,
                                       const int64_t *ids, int top, float *logprob, float *entropy,
                                       float *top_logprob, int32_t *top_id) {
  const int lane = threadIdx.x & 63;
  const float nan = __uint_as_float(0x7fc00000u);
  const bool ok = st.s > 0.0f;                     // false for 0 and for NaN
  const float ls = logf(st.s);
  if (lane == 0) {
    if (entropy) entropy[a] = ok ? ls - st.w / st.s : nan;
    if (logprob) {
      const int64_t id = ids[a];
      float lp = nan;
      if (id < 0) {
        lp = 0.0f;
      } else if (id < v && ok) {
        float x[1];
        load_vec<BF16, 1>((const char *)row + id * (BF16 ? 2 : 4), x);
        lp = (x[0] - st.m) - ls;
      }
      logprob[a] = lp;
    }
  }
  if (lane < top) {
    const float x = from_order_bits((uint32_t)(best.list >> 32));
    top_logprob[a * top + lane] = ok ? (x - st.m) - ls : nan;
    top_id[a * top + lane] = ok ? (int32_t)~(uint32_t)best.list : -1;
  }
}

// One workgroup per (row, segment).  The row's 16-byte aligned vectors are cut
// into nseg runs; the entries before and after them (rows need not be aligned)
// go to segment 0.
template <bool BF16>
__global__ __launch_bounds__(64 * LP_WAVES) void logprob_kernel(const void *__restrict__ L, int64_t v, int64_t ld,
                                                               const int64_t *__restrict__ ids, int top, int nseg,
                                                               float *logprob, float *entropy, float *top_logprob,
                                                               int32_t *top_id, float *__restrict__ ws_stats,
                                                               key_t64 *__restrict__ ws_keys) {
  constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
  __shared__ Stats s_stats[LP_WAVES];
  __shared__ key_t64 s_keys[LP_WAVES][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t a = blockIdx.x;
  const int seg = blockIdx.y;
  const char *row = (const char *)L + a * ld * ES;
  int64_t head = (int64_t)((16 - ((uintptr_t)row & 15)) & 15) / ES;
  if (head > v) head = v;
  const int64_t nv = (v - head) / VEC, tail = v - head - nv * VEC;
  const int64_t v0 = nv * seg / nseg, v1 = nv * (seg + 1) / nseg;

  Stats st = {-3.402823466e38f, 0.0f, 0.0f};
  Best best;
  best.clear();
  if (seg == 0 && wave == 0) {
    // lanes 0 .. 7 the head, 8 .. 15 the tail
    const int64_t idx = lane < 8 ? lane : v - tail + (lane - 8);
    const bool has = lane < 8 ? lane < head : lane - 8 < tail;
    float x[1] = {-__builtin_inff()};
    if (has) load_vec<BF16, 1>(row + idx * ES, x);
    take<1>(x, (uint32_t)idx, has, top, st, best);
  }
  const char *body = row + head * ES;
  for (int64_t j = v0 + wave * 64; j < v1; j += 64 * LP_WAVES) {
    const bool has = j + lane < v1;
    float x[VEC];
    load_vec<BF16, VEC>(body + (has ? j + lane : v0) * 16, x);
    take<VEC>(x, (uint32_t)(head + (j + lane) * VEC), has, top, st, best);
  }
  st = wave_join(st);
  if (lane == 0) s_stats[wave] = st;
  s_keys[wave][lane] = best.list;
  __syncthreads();
  if (wave) return;
  for (int w = 1; w < LP_WAVES; ++w) {
    st = join(st, s_stats[w]);
    if (top) best.offer(lane < top ? s_keys[w][lane] : 0, top);
  }
  if (nseg == 1) {
    finish<BF16>(st, best, row, v, a, ids, top, logprob, entropy, top_logprob, top_id);
  } else {
    const int64_t o = a * nseg + seg;
    if (lane == 0) {
      ws_stats[3 * o] = st.m;
      ws_stats[3 * o + 1] = st.s;
      ws_stats[3 * o + 2] = st.w;
    }
    if (lane < top) ws_keys[o * top + lane] = best.list;
  }
}

// One wave per row joins its segments.
template <bool BF16>
__global__ __launch_bounds__(64) void logprob_join_kernel(const void *__restrict__ L, int64_t v, int64_t ld,
                                                          const int64_t *__restrict__ ids, int top, int nseg,
                                                          float *logprob, float *entropy, float *top_logprob,
                                                          int32_t *top_id, const float *__restrict__ ws_stats,
                                                          const key_t64 *__restrict__ ws_keys) {
  const int lane = threadIdx.x & 63;
  const int64_t a = blockIdx.x;
  Stats st = {-3.402823466e38f, 0.0f, 0.0f};
  for (int s = lane; s < nseg; s += 64) {
    const float *p = ws_stats + 3 * (a * nseg + s);
    st = join(st, Stats{p[0], p[1], p[2]});
  }
  st = wave_join(st);
  Best best;
  best.clear();
  if (top) {
    const key_t64 *p = ws_keys + a * nseg * top;
    for (int i = 0; i < nseg * top; i += 64) best.offer(i + lane < nseg * top ? p[i + lane] : 0, top);
  }
  finish<BF16>(st, best, (const char *)L + a * ld * (BF16 ? 2 : 4), v, a, ids, top, logprob, entropy, top_logprob,
               top_id);
}

}  // namespace

LogprobPlan logprob_plan(int64_t t, int64_t v, int top) {
  LogprobPlan p;
  int64_t seg = t > 0 ? (1024 + t - 1) / t : 1;
  const int64_t most = (v + 4095) / 4096;
  if (seg > most) seg = most;
  if (seg > 64) seg = 64;
  p.nseg = (int)seg;
  p.ws_bytes = seg > 1 ? (((size_t)t * seg * 12 + 15) & ~(size_t)15) + (size_t)t * seg * top * 8 : 0;
  return p;
}

template <bool BF16>
static hipError_t go(const void *L, int64_t t, int64_t v, int64_t ld, const int64_t *ids, int top, float *logprob,
                     float *entropy, float *top_logprob, int32_t *top_id, void *ws, const LogprobPlan &p,
                     hipStream_t st) {
  float *stats = (float *)ws;
  key_t64 *keys = (key_t64 *)((char *)ws + (((size_t)t * p.nseg * 12 + 15) & ~(size_t)15));
  logprob_kernel<BF16><<<dim3((uint32_t)t, p.nseg), 64 * LP_WAVES, 0, st>>>(L, v, ld, ids, top, p.nseg, logprob, entropy,
                                                                           top_logprob, top_id, stats, keys);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nseg == 1) return e;
  logprob_join_kernel<BF16><<<(uint32_t)t, 64, 0, st>>>(L, v, ld, ids, top, p.nseg, logprob, entropy, top_logprob,
                                                        top_id, stats, keys);
  return hipGetLastError();
}

hipError_t launch_logprobs(const void *L, bool bf16, int64_t t, int64_t v, int64_t ld, const int64_t *ids, int top,
                           float *logprob, float *entropy, float *top_logprob, int32_t *top_id, void *ws,
                           const LogprobPlan &p, hipStream_t st) {
  return bf16 ? go<true>(L, t, v, ld, ids, top, logprob, entropy, top_logprob, top_id, ws, p, st)
              : go<false>(L, t, v, ld, ids, top, logprob, entropy, top_logprob, top_id, ws, p, st);
}

}  // namespace slim
