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
// lanes.  The first threshold is the top-th of the lanes' largest entries;
// what passes the threshold is collected in LDS and offered together: a few keys
// are broadcast and inserted one by one, shifting the lanes below; more are
// sorted over the lanes and merged (a bitonic network of 21 and 7 lane
// exchanges, all by DPP and lane swaps).  Of N values in random order only
// about top ln(N / top) get that far.  Waves and segments are joined by the
// same merge.  The set and its order depend on the keys alone.
//
// Bound by reading the logits where there are many: 2048 rows of 32000 float32
// 48.2 us where other logits pass between calls (262 MB, 5.4 TB/s; 41.4 again and
// again, part of them in the last-level cache), 333 rows of 100003 32 us (133 MB, 4.2
// TB/s) and 4.6 for the join.  bfloat16 halves the bytes but not the work of an entry
// (seven vector operations and a power, which costs four): 2048 rows of 32000 30 to 33 us.
// The best entries add the first threshold of every wave (a sort, 0.8 us) and
// the joins: at 2048 x 32000, float32 +4 us for one entry and +20 for 20,
// bfloat16 +9 and +28.  Few rows are latency: 16 rows of 131072 bfloat16 with 20
// entries 10.4 + 5.1 us, one row of 32000 float32 with five 11.2.
#include <algorithm>

#include "common.hpp"
#include "serve.hpp"

namespace slim {

namespace {

constexpr int LP_UN = 4;
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

// Lane exchanges: the value of lane l ^ X.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
template <int X>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  if constexpr (X == 0) return v;
  else if constexpr (X >= 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);   // both halves' values in every lane
    return lane_xor<X & 31>((threadIdx.x & 32) ? (uint32_t)r[0] : (uint32_t)r[1]);
  } else if constexpr (X >= 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return lane_xor<X & 15>((threadIdx.x & 16) ? (uint32_t)r[0] : (uint32_t)r[1]);
  } else if constexpr (X == 1) return dpp<0xB1>(v);      // quad_perm 1 0 3 2
  else if constexpr (X == 2) return dpp<0x4E>(v);        // quad_perm 2 3 0 1
  else if constexpr (X == 3) return dpp<0x1B>(v);        // quad_perm 3 2 1 0
  else if constexpr (X == 7) return dpp<0x141>(v);       // half row mirrored
  else if constexpr (X == 15) return dpp<0x140>(v);      // row mirrored
  else if constexpr (X == 8) return dpp<0x128>(v);       // row rotated by 8
  else {
    static_assert(X == 4, "not needed");
    return dpp<0x1B>(dpp<0x141>(v));
  }
}
// Lanes l and l ^ X compare keys; the lane without bit B keeps the larger.  The
// lane with it compares the complements: with a condition per lane in place of
// that, every step would wait for the scalar unit.
template <int X, int B>
__device__ __forceinline__ key_t64 exchange(key_t64 k) {
  const key_t64 o = ((key_t64)lane_xor<X>((uint32_t)(k >> 32)) << 32) | lane_xor<X>((uint32_t)k);
  const uint32_t m = (uint32_t)-(int32_t)((threadIdx.x & B) != 0);
  const key_t64 flip = ((key_t64)m << 32) | m;
  return (k ^ flip) > (o ^ flip) ? k : o;
}
// A bitonic sequence over the 64 lanes to descending order.
__device__ __forceinline__ key_t64 merge64(key_t64 k) {
  k = exchange<32, 32>(k);
  k = exchange<16, 16>(k);
  k = exchange<8, 8>(k);
  k = exchange<4, 4>(k);
  k = exchange<2, 2>(k);
  return exchange<1, 1>(k);
}
__device__ __forceinline__ key_t64 sort64(key_t64 k) {
  k = exchange<1, 1>(k);
  k = exchange<3, 2>(k);
  k = exchange<1, 1>(k);
  k = exchange<7, 4>(k);
  k = exchange<2, 2>(k);
  k = exchange<1, 1>(k);
  k = exchange<15, 8>(k);
  k = exchange<4, 4>(k);
  k = exchange<2, 2>(k);
  k = exchange<1, 1>(k);
  k = exchange<31, 16>(k);
  k = exchange<8, 8>(k);
  k = exchange<4, 4>(k);
  k = exchange<2, 2>(k);
  k = exchange<1, 1>(k);
  k = exchange<63, 32>(k);
  k = exchange<16, 16>(k);
  k = exchange<8, 8>(k);
  k = exchange<4, 4>(k);
  k = exchange<2, 2>(k);
  return exchange<1, 1>(k);
}

// The wave's best keys, descending over the lanes; thr = key number top - 1.
struct Best {
  key_t64 list, thr;
  __device__ __forceinline__ void clear() { list = 0, thr = 0; }
  // 64 keys in descending order over the lanes.
  __device__ __forceinline__ void merge(key_t64 k, int top) {
    const key_t64 o = ((key_t64)lane_xor<63>((uint32_t)(k >> 32)) << 32) | lane_xor<63>((uint32_t)k);
    list = merge64(list > o ? list : o);
    thr = lane_key(list, top - 1);
  }
  __device__ __forceinline__ void insert(key_t64 c, int top) {
    const int lane = threadIdx.x & 63;
    const int pos = __popcll(__ballot(list > c));
    const key_t64 up = ((key_t64)dpp<0x138>((uint32_t)(list >> 32)) << 32) | dpp<0x138>((uint32_t)list);   // lane l - 1
    list = lane < pos ? list : lane == pos ? c : up;
    thr = lane_key(list, top - 1);
  }
  // Every lane offers one key (0: none).
  __device__ __forceinline__ void offer(key_t64 mine, int top) {
    uint64_t left = __ballot(mine > thr);
    if (__popcll(left) > 6) {
      mine = sort64(mine);
      if (thr) {
        merge(mine, top);
      } else {                                   // nothing but zeros so far, or fewer than top keys
        const key_t64 had = lane_key(list, 0);
        if (had) {
          merge(mine, top);
        } else {
          list = mine;
          thr = lane_key(list, top - 1);
        }
      }
      return;
    }
    while (left) {
      const int src = __ffsll((unsigned long long)left) - 1;
      insert(lane_key(mine, src), top);
      left &= left - 1;
      left &= __ballot(mine > thr);
    }
  }
};

template <bool BF16>
__device__ __forceinline__ float load_one(const void *p) {
  if constexpr (BF16) return bf16_bits_to_f32(*(const uint16_t *)p);
  else return *(const float *)p;
}
// The entries of a 16-byte vector.
template <bool BF16, int VEC>
__device__ __forceinline__ void unpack(const uint4 &v, float *x) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (BF16) {
      x[2 * e] = __uint_as_float(u[e] << 16);
      x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    } else {
      x[e] = __uint_as_float(u[e]);
    }
  }
}

// N entries of every lane: e is entry idx(e) of the row, rising with e, and one
// that does not exist is -inf and idx(e) >= v.  shared: a threshold of the
// workgroup's other waves; s_thr: where this one's goes.  The waves see each
// other's at different times, but it only spares work: what it keeps out has
// top larger keys in some wave's list.
template <int N, class Idx>
__device__ __forceinline__ void take(const float (&x)[N], Idx idx, uint32_t v, int top, uint32_t shared, Stats &st,
                                     Best &best, uint32_t *s_thr, key_t64 *room) {
  float b = x[0];
#pragma unroll
  for (int e = 1; e < N; ++e) b = fmaxf(b, x[e]);
  if (b > st.m) {
    const float d = st.m - b, ed = exp_diff(d);
    st.w = fmaf(fmaxf(d, -1e30f), st.s, st.w) * ed;
    st.s *= ed;
    st.m = b;
  }
  float s[2] = {0.0f, 0.0f}, w[2] = {0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float d = x[e] - st.m;
    const float ex = exp_diff(d);
    s[e & 1] += ex;
    w[e & 1] = fmaf(ex, fmaxf(d, -1e30f), w[e & 1]);
  }
  st.s += s[0] + s[1];
  st.w += w[0] + w[1];
  if (!top) return;
  // A value below any wave's threshold is not among the row's best.
  if (shared > (uint32_t)(best.thr >> 32)) best.thr = (key_t64)shared << 32;
  float thr = from_order_bits((uint32_t)(best.thr >> 32));   // NaN while no list is full
  if (!__ballot(!(b < thr))) return;
  auto key = [&](float val, int e) __attribute__((always_inline)) {
    const uint32_t i = idx(e);
    return val == val && i < v ? make_key(val, i) : (key_t64)0;
  };
  auto largest = [&](const float (&y)[N]) __attribute__((always_inline)) {   // where y is b, the lowest of equals
    int at = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) at = y[N - 1 - e] == b ? N - 1 - e : at;
    return at;
  };
  key_t64 first = 0;
  if (N > 1 && !best.thr) {                                  // no threshold yet: the lanes' largest set one
    first = key(b, largest(x));
    best.offer(first, top);
    thr = from_order_bits((uint32_t)(best.thr >> 32));
  }
  // The entries that pass it, side by side in `room`, 64 keys of LDS.
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (!__ballot(!(x[e] < thr))) continue;
    const key_t64 k = key(x[e], e);
    const bool in = k > best.thr && k != first;
    const uint64_t who = __ballot(in);
    const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
    if (in && at < 64) room[at] = k;
    n += __popcll(who);
  }
  if (n > 0 && n <= 64) {
    __builtin_amdgcn_wave_barrier();
    best.offer(lane < n ? room[lane] : 0, top);
    __builtin_amdgcn_wave_barrier();
  } else if (n > 64) {
    // More than fit (rising rows, ties, or no threshold): the lanes' largest,
    // then their next ones, until no lane's passes.
    float y[N];
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = first && key(x[e], e) == first ? __uint_as_float(0x7fc00000u) : x[e];
    for (int round = 0; round < N; ++round) {
      b = __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int e = 0; e < N; ++e) b = fmaxf(b, y[e]);
      const int at = largest(y);
      const key_t64 k = key(b, at);
      if (!__ballot(k > best.thr)) break;
      best.offer(k, top);
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = e == at ? __uint_as_float(0x7fc00000u) : y[e];
    }
  }
  if ((threadIdx.x & 63) == 0) atomicMax(s_thr, (uint32_t)(best.thr >> 32));
}

__device__ __forceinline__ float lane_xor_f(float v, int d) {
  const uint32_t u = __float_as_uint(v);
  return __uint_as_float(d == 1    ? lane_xor<1>(u)
                         : d == 2  ? lane_xor<2>(u)
                         : d == 4  ? lane_xor<4>(u)
                         : d == 8  ? lane_xor<8>(u)
                         : d == 16 ? lane_xor<16>(u)
                                   : lane_xor<32>(u));
}
__device__ __forceinline__ Stats wave_join(Stats st) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1)
    st = join(st, Stats{lane_xor_f(st.m, d), lane_xor_f(st.s, d), lane_xor_f(st.w, d)});
  return st;
}

// The waves' lists, each in keys[wave], joined by halves into wave 0's.
template <int LP_WAVES>
__device__ __forceinline__ void join_lists(key_t64 (&keys)[LP_WAVES][64], Best &best, int top) {
  if (!top) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for (int w = LP_WAVES / 2; w >= 1; w /= 2) {
    if (wave < w) {
      best.merge(keys[wave + w][lane], top);
      keys[wave][lane] = best.list;
    }
    __syncthreads();
  }
}

// The given token's logit, read ahead of the results that need it: NaN for an
// id past the row, and anything for a negative one.
template <bool BF16>
__device__ __forceinline__ float given_logit(const void *row, int64_t v, int64_t id) {
  return id >= 0 && id < v ? load_one<BF16>((const char *)row + id * (BF16 ? 2 : 4)) : __uint_as_float(0x7fc00000u);
}

// Row results from its joined statistics (one wave).
__device__ __forceinline__ void finish(const Stats &st, const Best &best, int64_t a, int64_t id, float given, int top,
                                       float *logprob, float *entropy, float *top_logprob, int32_t *top_id) {
  const int lane = threadIdx.x & 63;
  const float nan = __uint_as_float(0x7fc00000u);
  const bool ok = st.s > 0.0f;                     // false for 0 and for NaN
  const float ls = logf(st.s);
  if (lane == 0) {
    if (entropy) entropy[a] = ok ? ls - st.w / st.s : nan;
    if (logprob) logprob[a] = id < 0 ? 0.0f : ok ? (given - st.m) - ls : nan;
  }
  if (lane < top) {
    const float x = from_order_bits((uint32_t)(best.list >> 32));
    top_logprob[a * top + lane] = ok ? (x - st.m) - ls : nan;
    top_id[a * top + lane] = ok ? (int32_t)~(uint32_t)best.list : -1;
  }
}

// One workgroup per (row, segment).  The row's 16-byte aligned vectors are cut
// into nseg runs; the entries before and after them (rows need not be aligned)
// go to segment 0.  A wave reads LP_UN vectors a lane at a time, 256 vectors
// apart, the next ones in flight while these are summed.
template <bool BF16, int LP_WAVES>
__global__ __launch_bounds__(64 * LP_WAVES) void logprob_kernel(const void *__restrict__ L, int64_t v, int64_t ld,
                                                               const int64_t *__restrict__ ids, int top, int nseg,
                                                               float *logprob, float *entropy, float *top_logprob,
                                                               int32_t *top_id, float *__restrict__ ws_stats,
                                                               key_t64 *__restrict__ ws_keys) {
  constexpr int ES = BF16 ? 2 : 4, VEC = 16 / ES;
  constexpr int STEP = 64 * LP_WAVES;
  __shared__ Stats s_stats[LP_WAVES];
  __shared__ key_t64 s_keys[LP_WAVES][64];
  __shared__ uint32_t s_thr;                     // largest threshold of the waves so far (ordered value bits)
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t a = blockIdx.x;
  const int seg = blockIdx.y;
  const char *row = (const char *)L + a * ld * ES;
  int head = (int)((16 - ((uintptr_t)row & 15)) & 15) / ES;
  if (head > v) head = (int)v;
  const int nv = (int)((v - head) / VEC), tail = (int)(v - head - (int64_t)nv * VEC);
  const int v0 = (int)((uint32_t)nv * seg / (uint32_t)nseg);   // nv < 2^23, nseg <= 64
  const int v1 = (int)((uint32_t)nv * (seg + 1) / (uint32_t)nseg);

  int64_t id = -1;
  float given = 0.0f;
  if (nseg == 1 && wave == 0 && logprob) {
    id = ids[a];
    given = given_logit<BF16>(row, v, id);
  }
  Stats st = {-3.402823466e38f, 0.0f, 0.0f};
  Best best;
  best.clear();
  const char *body = row + head * ES;
  int j = v0 + wave * 64 + lane;
  const int last = v1 - 1;
  uint4 cur[LP_UN], nxt[LP_UN];
  auto fetch = [&](int at, uint4 (&r)[LP_UN]) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < LP_UN; ++u)              // past the end: the last vector, not counted
      r[u] = *(const uint4 *)(body + (int64_t)(at + u * STEP < v1 ? at + u * STEP : last) * 16);
  };
  uint32_t shared = 0;
  if (top) {
    if (threadIdx.x == 0) s_thr = 0;
    __syncthreads();
  }
  auto batch = [&]() __attribute__((always_inline)) {
    float x[LP_UN * VEC];
#pragma unroll
    for (int u = 0; u < LP_UN; ++u) {
      unpack<BF16, VEC>(cur[u], x + u * VEC);
      if (j + u * STEP >= v1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[u * VEC + e] = -__builtin_inff();
      }
    }
    take<LP_UN * VEC>(
        x,
        [&](int e) __attribute__((always_inline)) {
          const int at = j + e / VEC * STEP;
          return at < v1 ? (uint32_t)(head + at * VEC + e % VEC) : 0xffffffffu;
        },
        (uint32_t)v, top, shared, st, best, &s_thr, s_keys[wave]);
  };
  if (v0 < v1) {
    fetch(j, cur);
    while (j - lane < v1) {
      fetch(j + LP_UN * STEP, nxt);
      // one value for all lanes, whatever other waves do to it meanwhile: it decides
      // branches around the lane exchanges
      if (top) shared = __builtin_amdgcn_readfirstlane(*(volatile uint32_t *)&s_thr);
      batch();
      j += LP_UN * STEP;
#pragma unroll
      for (int u = 0; u < LP_UN; ++u) cur[u] = nxt[u];
    }
  }
  if (seg == 0 && wave == 0) {
    // lanes 0 .. 7 the head, 8 .. 15 the tail
    const bool has = lane < 8 ? lane < head : lane - 8 < tail;
    const int64_t at = lane < 8 ? lane : v - tail + (lane - 8);
    float x[1] = {-__builtin_inff()};
    if (has) x[0] = load_one<BF16>(row + at * ES);
    take<1>(x, [&](int) __attribute__((always_inline)) { return has ? (uint32_t)at : 0xffffffffu; }, (uint32_t)v, top,
            0u, st, best, &s_thr, s_keys[wave]);
  }
  st = wave_join(st);
  if (lane == 0) s_stats[wave] = st;
  s_keys[wave][lane] = best.list;
  __syncthreads();
  join_lists<LP_WAVES>(s_keys, best, top);
  if (wave) return;
  if (LP_WAVES <= 4) {
    for (int w = 1; w < LP_WAVES; ++w) st = join(st, s_stats[w]);
  } else {
    st = wave_join(lane < LP_WAVES ? s_stats[lane] : Stats{-3.402823466e38f, 0.0f, 0.0f});
  }
  if (nseg == 1) {
    finish(st, best, a, id, given, top, logprob, entropy, top_logprob, top_id);
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

// One workgroup per row joins its segments: their lists by turns over the waves,
// then the waves' own.
template <bool BF16, int LP_WAVES>
__global__ __launch_bounds__(64 * LP_WAVES) void logprob_join_kernel(
    const void *__restrict__ L, int64_t v, int64_t ld, const int64_t *__restrict__ ids, int top, int nseg,
    float *logprob, float *entropy, float *top_logprob, int32_t *top_id, const float *__restrict__ ws_stats,
    const key_t64 *__restrict__ ws_keys) {
  __shared__ key_t64 s_keys[LP_WAVES][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t a = blockIdx.x;
  int64_t id = -1;
  float given = 0.0f;
  if (wave == 0 && logprob) {
    id = ids[a];
    given = given_logit<BF16>((const char *)L + a * ld * (BF16 ? 2 : 4), v, id);
  }
  Best best;
  best.clear();
  if (top) {
    const key_t64 *p = ws_keys + a * nseg * top;
    for (int s = wave; s < nseg; s += LP_WAVES) best.merge(lane < top ? p[s * top + lane] : 0, top);
    s_keys[wave][lane] = best.list;
    __syncthreads();
    join_lists<LP_WAVES>(s_keys, best, top);
  }
  if (wave) return;
  Stats st = {-3.402823466e38f, 0.0f, 0.0f};
  for (int s = lane; s < nseg; s += 64) {
    const float *p = ws_stats + 3 * (a * nseg + s);
    st = join(st, Stats{p[0], p[1], p[2]});
  }
  st = wave_join(st);
  finish(st, best, a, id, given, top, logprob, entropy, top_logprob, top_id);
}

}  // namespace

LogprobPlan logprob_plan(int64_t t, int64_t v, int top, bool bf16) {
  LogprobPlan p;
  const int64_t rows = t > 0 ? t : 1;
  // Few rows: workgroups of 16 waves, whose lists are joined by halves, each with
  // 16384 entries or a short row to itself, which then takes a single launch (one
  // float32 row of 131072, top 5: 12.8 us, by 4 waves 16.7).  More rows, and long
  // bfloat16 ones (16 rows of 131072: 15.1 against 12.9: 16 waves read 32768 of
  // its entries at once), are cut for workgroups of 4 waves.
  p.wide = (rows <= 32 && !bf16) || (rows <= 64 && v <= 32768);
  const int64_t wide = v <= 32768 ? 1 : std::min((256 + rows - 1) / rows, (v + 16383) / 16384);
  // Those pieces: 2048 entries at least until 512 workgroups share the rows, and
  // of 16384 until 1536 do, so that the last workgroups of the card end together
  // (333 rows of 100003: 5 segments 31.4 us, 2 segments 35).
  const int64_t few = std::min((512 + rows - 1) / rows, (v + 2047) / 2048);
  const int64_t even = std::min((1536 + rows - 1) / rows, (v + 16383) / 16384);
  const int64_t seg = std::min<int64_t>(64, p.wide ? wide : std::max(few, even));
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
  const dim3 grid((uint32_t)t, p.nseg);
  if (p.wide)
    logprob_kernel<BF16, 16><<<grid, 64 * 16, 0, st>>>(L, v, ld, ids, top, p.nseg, logprob, entropy, top_logprob, top_id,
                                                       stats, keys);
  else
    logprob_kernel<BF16, 4><<<grid, 64 * 4, 0, st>>>(L, v, ld, ids, top, p.nseg, logprob, entropy, top_logprob, top_id,
                                                     stats, keys);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nseg == 1) return e;
  logprob_join_kernel<BF16, 4><<<(uint32_t)t, 64 * 4, 0, st>>>(L, v, ld, ids, top, p.nseg, logprob, entropy,
                                                               top_logprob, top_id, stats, keys);
  return hipGetLastError();
}

hipError_t launch_logprobs(const void *L, bool bf16, int64_t t, int64_t v, int64_t ld, const int64_t *ids, int top,
                           float *logprob, float *entropy, float *top_logprob, int32_t *top_id, void *ws,
                           const LogprobPlan &p, hipStream_t st) {
  return bf16 ? go<true>(L, t, v, ld, ids, top, logprob, entropy, top_logprob, top_id, ws, p, st)
              : go<false>(L, t, v, ld, ids, top, logprob, entropy, top_logprob, top_id, ws, p, st);
}

}  // namespace slim
