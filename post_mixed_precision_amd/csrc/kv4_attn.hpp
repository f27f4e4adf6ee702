// Attention over the 4-bit key/value cache on the matrix cores of gfx950.
//
//   S[r, t] = scale sum_c q[r, c] k[t, c],  o[r] = sum_t softmax_t(S[r, t]) v[t]   over t < limit(r),
//   k[t, c] = code[t, c] step[t, j] + low[t, j]   (j the group of c; v alike)
//
// Codes are exact in bfloat16, so with Q_j the sum of q over group j
//   S[r, t] = scale sum_j (step[t, j] (sum_{c in j} q[r, c] code[t, c]) + low[t, j] Q_j[r]),
//   o[r, c] = sum_t (P[r, t] step[t, j]) code[t, c] + sum_t P[r, t] low[t, j],
// where the products with codes go to the matrix cores and the rest is float32:
// nothing is dequantized.  P step is the one thing that is rounded: to two
// bfloat16 terms where q and the output are bfloat16, to three elsewhere.
// For many rows of bfloat16 the second product is one of float16 weights with
// float16 values instead, wherever the values' range allows that.
//
// Rows are the query tokens of a sequence times the query heads of one key
// head, 16 a tile.  S is formed transposed (tokens by rows): its accumulator
// then holds, in lane 16 lg + r, row r's entries of tokens 4 lg .. +3 of a
// record, which is what the second product wants of its operand when the
// contraction runs over the same tokens in the same order.  So P never leaves
// its lane, and the cache's layout gives each lane its 4 tokens of a channel
// as one word.  A row's statistics are per lane as well; only the maximum
// crosses lanes.
#pragma once
#include <type_traits>

#include "mma16.hpp"
#include "serve.hpp"

namespace slim {
namespace kv4 {

constexpr float kNaN = __builtin_nanf("");
constexpr float kNegInf = -__builtin_inff();

// 2^x (v_exp_f32: 1 ulp; results below 2^-126 may be 0).
__device__ __forceinline__ float exp2_any(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pk_bf16(float lo, float hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// What a workgroup works on: a tile of a sequence's rows, for one key head,
// over one of `nsplit` runs of the sequence's tokens.
struct Work {
  int64_t q0;                // the sequence's first query token
  int seq, ql, len;          // its number, query tokens, tokens
  int tile, split, nsplit;
  int first;                 // number of the tile's first run, per head
  int slot, slots;           // the tile's number over all sequences; how many there are
  bool over;                 // its length is past its row of the page table
  bool none, bad;            // nothing here; bounds out of order
};

// Tokens of a sequence, 0 if there is nothing to attend to.
__device__ __forceinline__ int length_of(const Kv4Args &a, int seq, bool &over) {
  const int n = a.lengths[seq];
  over = n > a.cap;
  return over || n < 0 ? 0 : n;
}

// Running sums over the wave's lanes, by data-parallel moves (a shuffle
// through LDS costs ten times as much, and every workgroup starts with these).
template <class T>
__device__ __forceinline__ T moved(T x, T none, int which) {
  const int o = __builtin_bit_cast(int, none), v = __builtin_bit_cast(int, x);
  int r;
  switch (which) {
    case 0: r = __builtin_amdgcn_update_dpp(o, v, 0x111, 0xf, 0xf, false); break;   // from 1, 2, 4, 8 lanes below
    case 1: r = __builtin_amdgcn_update_dpp(o, v, 0x112, 0xf, 0xf, false); break;
    case 2: r = __builtin_amdgcn_update_dpp(o, v, 0x114, 0xf, 0xf, false); break;
    case 3: r = __builtin_amdgcn_update_dpp(o, v, 0x118, 0xf, 0xf, false); break;
    case 4: r = __builtin_amdgcn_update_dpp(o, v, 0x142, 0xa, 0xf, false); break;   // the row's sum to the next row,
    default: r = __builtin_amdgcn_update_dpp(o, v, 0x143, 0xc, 0xf, false); break;  // two rows' to the next two
  }
  return __builtin_bit_cast(T, r);
}
template <class T>
__device__ __forceinline__ T running_sum(T x) {
#pragma unroll
  for (int i = 0; i < 6; ++i) x += moved<T>(x, (T)0, i);
  return x;
}
template <class T>
__device__ __forceinline__ T of_lane(T x, int lane) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// ceil(x / y) for x < 2^26: the quotient by a reciprocal, put right.
__device__ __forceinline__ int ceil_div(int x, int y) {
  int r = (int)((float)x * __builtin_amdgcn_rcpf((float)y));
  while ((int64_t)r * y < x) ++r;
  while (r > 0 && (int64_t)(r - 1) * y >= x) --r;
  return r;
}

// How the work is cut is worked out here, by every wave for itself, from the
// lengths and bounds on the device (lane l takes consecutive sequences): a
// tile's tokens go to one workgroup for every `chunk` of them, chunk being
// a share of all tokens that spreads them over `slots` + `extra` workgroups.  So
// sequences of uneven lengths end together, no table or copy to the host is
// needed, and at most slots + extra workgroups are used.  i: number of the run.
__device__ __forceinline__ Work find_work(const Kv4Args &a, const Kv4Cut &cut, int i) {
  Work w = {};
  const int lane = threadIdx.x & 63, per = (a.b + 63) >> 6;
  auto bounds = [&](int s, int &lo, int &hi) __attribute__((always_inline)) {
    lo = a.offsets ? a.offsets[s] : s * a.ql;
    hi = a.offsets ? a.offsets[s + 1] : lo + a.ql;
  };
  auto tiles_of = [&](int lo, int hi) __attribute__((always_inline)) {
    return a.offsets ? (int)((unsigned)((hi - lo) * a.g + cut.tm - 1) >> cut.tm_log) : cut.tiles;
  };
  const bool cuts = cut.extra > 0;
  if (!cuts && !a.offsets) {                   // a run a tile, as many for each sequence
    w.seq = (int)((unsigned)i / (unsigned)cut.tiles);
    w.q0 = (int64_t)w.seq * a.ql, w.ql = a.ql, w.nsplit = 1, w.first = i;
    w.tile = cut.tiles - 1 - (i - w.seq * cut.tiles);
    w.len = length_of(a, w.seq, w.over);
    return w;
  }
  float work = 0.0f;
  bool wrong = false;
  int t0 = 0;                       // records' tiles and row tiles of the lane's first sequence
  int n0 = 0;
  for (int x = 0; x < per; ++x) {
    const int s = lane * per + x;
    if (s >= a.b) break;
    int lo, hi;
    bounds(s, lo, hi);
    wrong |= lo < 0 || hi < lo || hi > a.tq;
    bool over;
    const int n = hi < lo ? 0 : tiles_of(lo, hi), t = cuts ? (length_of(a, s, over) + 31) >> 5 : 0;
    work += (float)n * (float)t;
    if (x == 0) t0 = t, n0 = n;
  }
  if (a.offsets && __any(wrong)) {
    w.bad = true;
    return w;
  }
  int chunk = 1 << 26;
  auto runs_of = [&](int t) __attribute__((always_inline)) { return t <= chunk ? 1 : ceil_div(t, chunk); };
  int tiles = n0;
  for (int x = 1; x < per; ++x) {
    const int s = lane * per + x;
    if (s >= a.b) break;
    int lo, hi;
    bounds(s, lo, hi);
    tiles += tiles_of(lo, hi);
  }
  const int tsum = running_sum(tiles);
  w.slots = of_lane(tsum, 63);
  int runs = 0, rsum = 0;
  auto count = [&]() __attribute__((always_inline)) {
    runs = n0 * runs_of(t0);
    for (int x = 1; x < per; ++x) {
      const int s = lane * per + x;
      if (s >= a.b) break;
      int lo, hi;
      bounds(s, lo, hi);
      bool over;
      runs += tiles_of(lo, hi) * runs_of(cuts ? (length_of(a, s, over) + 31) >> 5 : 0);
    }
    rsum = running_sum(runs);
  };
  if (!cuts) {
    count();
  } else {
    // Every tile's number of runs is rounded up, so spread over `extra` the runs are never too many,
    // and spread over all of them just enough where the tiles divide evenly: the smallest size of three
    // that fits (4000 tokens, 512 float32 queries: 309 TFLOP/s, the last alone 239; 3 sequences of up to
    // 3000: 414 and 362), or the last where a lane has several sequences.  The sum's rounding is
    // below (per + 6) 2^-24 of it, far inside the factor.
    const float all = of_lane(running_sum(work), 63) * 1.01f;
    for (int i = per == 1 ? 2 : 0;; --i) {
      const float share = all / (float)(cut.extra + (w.slots * i >> 1));
      chunk = share < (float)cut.least ? cut.least : (int)fminf(share, (float)(1 << 26)) + 1;
      count();
      if (i <= 0 || of_lane(rsum, 63) <= cut.slots + cut.extra) break;
    }
  }
  const uint64_t past = __ballot(rsum > i);
  if (!past) {
    w.none = true;
    return w;
  }
  const int own = __ffsll((unsigned long long)past) - 1;
  int first = of_lane(rsum - runs, own), slot = of_lane(tsum - tiles, own);
  for (int s = own * per; s < a.b; ++s) {   // lane `own` has run i
    int lo, hi;
    bounds(s, lo, hi);
    w.len = length_of(a, s, w.over);
    const int n = tiles_of(lo, hi), r = cuts ? runs_of((w.len + 31) >> 5) : 1;
    if (i >= first + n * r) {
      first += n * r, slot += n;
      continue;
    }
    const int t = r == 1 ? i - first : (i - first) / r;
    w.q0 = lo, w.seq = s, w.ql = hi - lo, w.nsplit = r;
    w.first = first + t * r;
    w.split = i - w.first;
    w.slot = slot + t;
    w.tile = n - 1 - t;             // the longest first
    return w;
  }
  w.none = true;                    // lengths written to meanwhile: still an end
  return w;
}

// What the join reads of a tile, in the workspace behind the partial results.
struct __attribute__((aligned(16))) Joint {
  int q0, ql, m0, first, runs;   // runs: 0 where there is no tile, -1 for bounds out of order
  int pad[3];
};
__device__ __forceinline__ Joint *joints(const Kv4Args &a, const Kv4Cut &cut, int dim) {
  return (Joint *)(cut.part + (int64_t)(cut.slots + cut.extra) * a.hkv * cut.tm * (dim + 2));
}
// Written by the first head's workgroups: a tile's first one, and for the numbers past the last tile any.
__device__ __forceinline__ void note_joint(const Kv4Args &a, const Kv4Cut &cut, const Work &w, int run, int h, int dim) {
  if (cut.extra == 0 || h != 0 || threadIdx.x != 0) return;
  Joint j = {};
  if (w.bad || run >= w.slots) {
    j.runs = w.bad ? -1 : 0;
    if (run < cut.slots) joints(a, cut, dim)[run] = j;
    if (w.bad) return;
  }
  if (!w.none && w.split == 0) {
    j.q0 = (int)w.q0, j.ql = w.ql, j.m0 = w.tile * cut.tm, j.first = w.first, j.runs = w.nsplit;
    joints(a, cut, dim)[w.slot] = j;
  }
}

// Tokens row i (a query token of ql) of a sequence attends to.
__device__ __forceinline__ int limit_of(const Kv4Args &a, int len, int ql, int i) {
  const int n = a.causal ? len - ql + i + 1 : len;
  return n < 0 ? 0 : n;
}

__device__ __forceinline__ void store_out(const Kv4Args &a, int64_t at, float x) {
  if (a.obf16) ((uint16_t *)a.out)[at] = (uint16_t)f32_to_bf16_bits(x);
  else ((float *)a.out)[at] = x;
}

// Bounds out of order: the first `shares` workgroups of a head share the rows out and make them NaN.
__device__ __forceinline__ void nan_share(const Kv4Args &a, int i, int shares, int h, int dim) {
  const int each = (a.tq + shares - 1) / shares;
  const int64_t lo = (int64_t)i * each, hi = lo + each < a.tq ? lo + each : a.tq;
  for (int64_t x = lo * a.g * dim + threadIdx.x; x < hi * a.g * dim; x += blockDim.x) {
    const int64_t c = x % dim, r = x / dim;
    store_out(a, (r / a.g * a.hq + h * a.g + r % a.g) * dim + c, kNaN);
  }
}

// Partial results, by number of the run, head, row: sums, then (behind all sums) reference and sum of weights.
__device__ __forceinline__ float *part_sum(const Kv4Args &a, const Kv4Cut &cut, int run, int h, int m, int dim) {
  return cut.part + (((int64_t)run * a.hkv + h) * cut.tm + m) * dim;
}
__device__ __forceinline__ float2 *part_ml(const Kv4Args &a, const Kv4Cut &cut, int run, int h, int m, int dim) {
  return (float2 *)(cut.part + (int64_t)(cut.slots + cut.extra) * a.hkv * cut.tm * dim) +
         (((int64_t)run * a.hkv + h) * cut.tm + m);
}

// Row m of a sequence's for head h, query token i = m / g: its place among q's and out's heads.
template <class K>
__device__ __forceinline__ int64_t row_at(const Kv4Args &a, const K &k, int h, int m, int i) {
  return (int64_t)(k.q0 + i) * a.hq + h * a.g + (m - i * a.g);
}

// What a wave keeps of its 16 NQ rows, and one step of the attention: 32
// tokens (two records) for all of them.
//
// Weights are 2^(S - m) with S in powers of two and m the row's reference: the
// maximum of the row's first tokens less kLift, moved up only once a weight
// would exceed 2^kMost.  So a step needs no maximum across lanes and no
// rescaling, but for the first ones: each lane compares its own scores.
//
// Few rows: weights times steps are rounded to the sum of two bfloat16 terms
// (2^-16): with one term (2^-9) the outputs' error was twice that of their own
// rounding to bfloat16.  Weights of float32
// outputs, and float32 queries and their weights, enter as three terms.
//
// Those have codes less 8 in the second product, with low ends plus 8 steps: low
// ends are some two deviations of the values, and their sum over thousands of tokens
// and that of the codes would cancel to a hundredth (80 rows over 20000 tokens were off by
// 4.2e-6 of the output's norm, 1.6e-6 so, elementary operations 1.8e-6; it takes 6 to 10% longer).
//
// Many rows of bfloat16: values are dequantized after all, once for the
// workgroup, to float16 (step, low end and value each within 2^-11 of themselves), and
// weights are float16 too (2^-11, or 2^-33 of the row's largest weight, by the
// lift; a lift of 11 took 3%, of 14 10% longer, as references then move more often).  The products of codes with weights in two terms cost twice the
// matrix instructions and six vector instructions more a weight: 8 sequences
// of 4096, causal, 32 + 8 heads of 128, took 1702 us by them, 1548 us so (and
// 1408 with what came after).
constexpr float kLift = 8.0f, kMost = 15.0f;
// What rows are held by: bfloat16 queries and outputs, bfloat16 queries with float32 outputs, float32 queries.
constexpr int kBf16 = 0, kMixed = 1, kF32 = 2;

// 8 numbers as two bfloat16 terms, the first truncated, the second rounded.
__device__ __forceinline__ void split2(const float (&x)[8], uint4 (&t)[2]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t a = __float_as_uint(x[2 * e]), b = __float_as_uint(x[2 * e + 1]);
    h[e] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    l[e] = pk_bf16(x[2 * e] - __uint_as_float(a & 0xffff0000u), x[2 * e + 1] - __uint_as_float(b & 0xffff0000u));
  }
  t[0] = make_uint4(h[0], h[1], h[2], h[3]);
  t[1] = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ uint32_t pk_half(float lo, float hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

template <int DIM, int GROUP, int NQ, int X>
struct Rows {
  static constexpr int NG = DIM / GROUP, W = DIM / 32, GS = GROUP / 32, NTQ = X == kF32 ? 3 : 1, NTP = X == kBf16 ? 2 : 3;
  uint4 qf[NQ][W][NTQ];      // the rows' queries as operands
  float qs[NQ][NG];          // their sums over each group, times scale log2 e
  int lim[NQ];               // tokens a row attends to
  float m[NQ], thr[NQ];      // reference; what a score may exceed it by (-inf: no reference yet)
  float ls[NQ], pl[NQ][NG];  // this lane's share of sum P and of sum P low
  f32x4_t o[NQ][DIM / 16];   // sum P step code (or P value), channels by rows
  f32x4_t lh[NQ];            // sum P of the steps by float16, in every entry

  // Rows m0 + 16 n + lane % 16 of the sequence, those from `rows` on as zeros that attend to nothing.
  __device__ __forceinline__ void start(const Kv4Args &a, const Work &k, int h, int m0, int rows, float c) {
    const int r16 = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int mm = m0 + 16 * n + r16;
      const bool real = mm < rows;
      const int i = (int)((unsigned)(real ? mm : 0) / (unsigned)a.g);
      lim[n] = real ? limit_of(a, k.len, k.ql, i) : 0;
      const int64_t at = row_at(a, k, h, real ? mm : 0, i) * DIM + 8 * lg;
#pragma unroll
      for (int j = 0; j < NG; ++j) qs[n][j] = pl[n][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if constexpr (X == kF32) {
          const float4 *p = (const float4 *)((const float *)a.q + at + 32 * j);
          float4 u = p[0], w = p[1];
          if (!real) u = w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          split3(__builtin_bit_cast(uint4, u), __builtin_bit_cast(uint4, w), qf[n][j]);
          qs[n][j / GS] += ((u.x + u.y) + (u.z + u.w)) + ((w.x + w.y) + (w.z + w.w));
        } else {
          uint4 u = *(const uint4 *)((const uint16_t *)a.q + at + 32 * j);
          if (!real) u = make_uint4(0u, 0u, 0u, 0u);
          qf[n][j][0] = u;
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) s += __uint_as_float(w[e] << 16) + __uint_as_float(w[e] & 0xffff0000u);
          qs[n][j / GS] += s;
        }
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        qs[n][j] += __shfl_xor(qs[n][j], 16, 64);
        qs[n][j] += __shfl_xor(qs[n][j], 32, 64);
        qs[n][j] *= c;
      }
      m[n] = 0.0f, thr[n] = kNegInf, ls[n] = 0.0f;
      lh[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i2 = 0; i2 < DIM / 16; ++i2) o[n][i2] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // Weights of 32 tokens, tok the lane's first one (entry 4 b + v: token tok + 16 b + v).  Src: codes
  // and pairs of the two records; a key's step is given times scale log2 e.  EDGE: some row does
  // not attend to all of them.  HALF: the sums are those by float16, the others are not yet there.
  template <bool EDGE, bool HALF, class Src>
  __device__ __forceinline__ void weigh(Src &src, int tok, float (&x)[NQ][8]) {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[n][e] = -m[n];
    src.keys();
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        f32x4_t acc[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) acc[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = GS * j; w < GS * (j + 1); ++w) {
          const uint4 k = src.kcode(b, w);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int t = NTQ - 1; t >= 0; --t) acc[n] = mfma16(k, qf[n][w][t], acc[n]);
        }
        float step[4], low[4];
        src.kpair(b, j, step, low);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            x[n][4 * b + v] = __builtin_fmaf(low[v], qs[n][j], x[n][4 * b + v]);
            x[n][4 * b + v] = __builtin_fmaf(step[v], acc[n][v], x[n][4 * b + v]);
          }
      }
    float top[NQ];
    bool up = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if (EDGE) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (tok + 16 * (e >> 2) + (e & 3) >= lim[n]) x[n][e] = kNegInf;
      }
      top[n] = fmaxf(fmaxf(fmaxf(x[n][0], x[n][1]), fmaxf(x[n][2], x[n][3])),
                     fmaxf(fmaxf(x[n][4], x[n][5]), fmaxf(x[n][6], x[n][7])));
      up |= top[n] > thr[n];
    }
    if (__any(up)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) raise<HALF>(n, top[n], x[n]);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[n][e] = exp2_any(x[n][e]);
  }

  // 32 tokens from token `first` on, values by their codes.
  template <bool EDGE, class Src>
  __device__ __forceinline__ void attend(Src &src, int first) {
    const int tok = first + 4 * ((threadIdx.x & 63) >> 4);
    float x[NQ][8];
    weigh<EDGE, false>(src, tok, x);
    src.values();
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) ls[n] += x[n][e];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float step[2][4], low[2][4];
      src.vpair(0, j, step[0], low[0]);
      src.vpair(1, j, step[1], low[1]);
      uint4 pf[NQ][NTP];     // weight times step, 4 tokens of either record
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[e] = x[n][e] * step[e >> 2][e & 3];
          float z = low[e >> 2][e & 3];
          if (X != kBf16) z = __builtin_fmaf(8.0f, step[e >> 2][e & 3], z);
          if (EDGE && tok + 16 * (e >> 2) + (e & 3) >= lim[n]) y[e] = z = 0.0f;   // NaN pairs of masked tokens
          pl[n][j] = __builtin_fmaf(x[n][e], z, pl[n][j]);
        }
        if constexpr (X != kBf16)
          split3(make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])),
                 make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7])),
                 pf[n]);
        else
          split2(y, pf[n]);
      }
      if constexpr (X != kBf16) {   // codes less 8: their sum so far moves by -8 P step
        const uint4 m8 = make_uint4(0xc100c100u, 0xc100c100u, 0xc100c100u, 0xc100c100u);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          f32x4_t by = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int t = NTP - 1; t >= 0; --t) by = mfma16(m8, pf[n][t], by);
#pragma unroll
          for (int i = 2 * GS * j; i < 2 * GS * (j + 1); ++i) o[n][i] += by;
        }
      }
#pragma unroll
      for (int w = GS * j; w < GS * (j + 1); ++w) {
        uint4 even, odd;
        src.vcode(w, even, odd);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int t = NTP - 1; t >= 0; --t) {
            o[n][2 * w] = mfma16(even, pf[n][t], o[n][2 * w]);
            o[n][2 * w + 1] = mfma16(odd, pf[n][t], o[n][2 * w + 1]);
          }
      }
    }
  }

  // The same with the values themselves, finite, as float16.
  template <bool EDGE, class Src>
  __device__ __forceinline__ void attend_half(Src &src, int first) {
    float x[NQ][8];
    weigh<EDGE, true>(src, first + 4 * ((threadIdx.x & 63) >> 4), x);
    const uint4 ones = make_uint4(0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u);
    uint4 pf[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      pf[n] = make_uint4(pk_half(x[n][0], x[n][1]), pk_half(x[n][2], x[n][3]), pk_half(x[n][4], x[n][5]),
                         pk_half(x[n][6], x[n][7]));
      lh[n] = mfma16_half(ones, pf[n], lh[n]);   // the sum of the weights as they are multiplied
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint4 even, odd;
      src.vcode(w, even, odd);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        o[n][2 * w] = mfma16_half(even, pf[n], o[n][2 * w]);
        o[n][2 * w + 1] = mfma16_half(odd, pf[n], o[n][2 * w + 1]);
      }
    }
  }
  // From sums of values times `unit` by float16 to sums of values.
  __device__ __forceinline__ void leave_half(float unit) {
    const bool first = (threadIdx.x & 63) < 16;   // the other lanes of a row have the same sum of weights
    const float f = 1.0f / unit;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      ls[n] = first ? lh[n][0] : 0.0f;
#pragma unroll
      for (int j = 0; j < NG; ++j) pl[n][j] = 0.0f;
#pragma unroll
      for (int i = 0; i < DIM / 16; ++i) o[n][i] *= f;
    }
  }

  // A new reference for the rows that need one: the maximum over the step's tokens.
  template <bool HALF>
  __device__ __forceinline__ void raise(int n, float top, float (&x)[8]) {
    asm volatile("" : "+v"(top));   // nothing of this is done ahead of the branch
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const bool up = top > thr[n];
    const float by = up ? top - kLift : 0.0f;
    const float f = !up ? 1.0f : thr[n] == kNegInf ? 0.0f : exp2_any(-by);   // sums of no token are 0
    m[n] += by;
    if (up) thr[n] = kMost;
    if (HALF) {
      lh[n] *= f;
    } else {
      ls[n] *= f;
#pragma unroll
      for (int j = 0; j < NG; ++j) pl[n][j] *= f;
    }
#pragma unroll
    for (int i = 0; i < DIM / 16; ++i) o[n][i] *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] -= by;
  }

  // The sums of the four lanes of a row; o then holds sum P v.
  __device__ __forceinline__ void finish(bool over) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      ls[n] += __shfl_xor(ls[n], 16, 64);
      ls[n] += __shfl_xor(ls[n], 32, 64);
      if (over) ls[n] = kNaN;
      if (thr[n] == kNegInf) m[n] = kNegInf;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        float x = pl[n][j];
        x += __shfl_xor(x, 16, 64);
        x += __shfl_xor(x, 32, 64);
#pragma unroll
        for (int i = 2 * GS * j; i < 2 * GS * (j + 1); ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) o[n][i][v] += x;
      }
    }
  }
  // Channels 32 w + 8 (lane / 16) .. +7 of row n's lane, in order.
  __device__ __forceinline__ void channels(int n, int w, float (&y)[8]) const {
#pragma unroll
    for (int v = 0; v < 4; ++v) y[2 * v] = o[n][2 * w][v], y[2 * v + 1] = o[n][2 * w + 1][v];
  }
};

__device__ __forceinline__ float half_of(uint32_t w, bool high) {
  return __uint_as_float(high ? w & 0xffff0000u : w << 16);
}

// The pages of a run of records: lane i holds that of record base + i (-1: outside the cache).
struct Pages {
  const int32_t *table;
  const char *cache;         // the head's first record
  unsigned bytes;            // of a page, all heads
  int pages, last, shift, base, page;
  __device__ __forceinline__ void load(int from) {
    base = from;
    const int b = from + (int)(threadIdx.x & 63);
    page = table[(b < last ? b : last) >> shift];
    if (page < 0 || page >= pages) page = -1;
  }
  // Of record b (past the last one: of the last); uniform over the wave.
  __device__ __forceinline__ int of(int b) const { return __builtin_amdgcn_readlane(page, b - base); }
  // Where record b of a page (that of(b) gave; of a lost one: of page 0) lies.
  template <int RECB>
  __device__ __forceinline__ const char *at(int page_of, int b) const {
    const unsigned in = (unsigned)(b < last ? b : last) & ((1u << shift) - 1);
    return cache + (uint64_t)(unsigned)(page_of < 0 ? 0 : page_of) * bytes + in * RECB;
  }
};

// Greatest over aligned groups of 16 lanes.
__device__ __forceinline__ uint32_t over_row(uint32_t x) {
  auto with = [&](uint32_t y) __attribute__((always_inline)) { x = x > y ? x : y; };
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xb1, 0xf, 0xf, true));    // lane ^ 1
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4e, 0xf, 0xf, true));    // lane ^ 2
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xf, 0xf, true));   // lane ^ 7 of 8
  with((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xf, 0xf, true));   // lane ^ 15 of 16
  return x;
}

// Two float16 numbers x y + z, each rounded once.
__device__ __forceinline__ uint32_t fma_half(uint32_t x, uint32_t y, uint32_t z) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, x),
                                                               __builtin_bit_cast(f16x2_t, y),
                                                               __builtin_bit_cast(f16x2_t, z)));
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <int N>
__device__ __forceinline__ void load_words(const uint32_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const uint2 u = *(const uint2 *)p;
    w[0] = u.x, w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = ((const uint4 *)p)[i];
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
}

typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(1))) void global_void_t;

// N 16-byte pieces of LDS at `at` + O..., read and waited for in one block: the
// compiler would wait for every load in flight to LDS before a read of its own.
template <int O0, int O1>
__device__ __forceinline__ void lds_get(uint32_t at, uint4 &a, uint4 &b) {
  u32x4_t x, y;
  asm volatile("ds_read_b128 %0, %2 offset:%3\n\tds_read_b128 %1, %2 offset:%4\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x), "=&v"(y)
               : "v"(at), "n"(O0), "n"(O1)
               : "memory");
  a = __builtin_bit_cast(uint4, x), b = __builtin_bit_cast(uint4, y);
}
template <int O0, int O1>
__device__ __forceinline__ void lds_get(uint32_t at, uint2 &a, uint2 &b) {
  u32x2_t x, y;
  asm volatile("ds_read_b64 %0, %2 offset:%3\n\tds_read_b64 %1, %2 offset:%4\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x), "=&v"(y)
               : "v"(at), "n"(O0), "n"(O1)
               : "memory");
  a = __builtin_bit_cast(uint2, x), b = __builtin_bit_cast(uint2, y);
}
// Two at `at` and two at `pair`.
template <int O0, int O1, int P0, int P1>
__device__ __forceinline__ void lds_get(uint32_t at, uint4 &a, uint4 &b, uint32_t pair, uint4 &c, uint4 &d) {
  u32x4_t x, y, z, w;
  asm volatile("ds_read_b128 %0, %4 offset:%6\n\tds_read_b128 %1, %4 offset:%7\n\t"
               "ds_read_b128 %2, %5 offset:%8\n\tds_read_b128 %3, %5 offset:%9\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(x), "=&v"(y), "=&v"(z), "=&v"(w)
               : "v"(at), "v"(pair), "n"(O0), "n"(O1), "n"(P0), "n"(P1)
               : "memory");
  a = __builtin_bit_cast(uint4, x), b = __builtin_bit_cast(uint4, y);
  c = __builtin_bit_cast(uint4, z), d = __builtin_bit_cast(uint4, w);
}

// Waits until at most VM of this wave's loads are in flight (they complete in order).
template <int VM>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | (VM >> 4) << 14);
  asm volatile("" ::: "memory");
}

// Two records as they lie in the cache, in LDS; a wave's own.
template <int DIM, int GROUP>
struct Ring {
  static constexpr int NG = DIM / GROUP, W = DIM / 32, RECB = 16 * DIM + 128 * NG, TILEB = 2 * RECB;
  static constexpr int LOADS = 2 * (DIM / 64 + 1);         // of a tile
  static constexpr int STAGES = 2;
  // The record at p to LDS at `to`, 16 bytes a lane.
  static __device__ __forceinline__ void load(const char *p, char *to) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < DIM / 64; ++i)
      __builtin_amdgcn_global_load_lds((global_void_t *)(p + 1024 * i + 16 * lane), (lds_void_t *)(to + 1024 * i), 16, 0,
                                       0);
    if (lane < 8 * NG)
      __builtin_amdgcn_global_load_lds((global_void_t *)(p + 16 * DIM + 16 * lane), (lds_void_t *)(to + 16 * DIM), 16, 0,
                                       0);
  }
};

// The same as a source of operands: codes come from LDS when their turn comes and are expanded as they are used.
template <int DIM, int GROUP>
struct RingTile {
  typedef Ring<DIM, GROUP> R;
  static constexpr int NG = R::NG, W = R::W, RECB = R::RECB;
  uint32_t codes, pairs;     // LDS addresses of this lane's codes and of its four tokens' pairs
  int lost;                  // bit b: record b's page lies outside the cache
  float c;
  uint32_t k[2][W], v[2][W];
  uint4 kp[2][NG], vp[2][NG];

  template <int OFF>
  __device__ __forceinline__ void words(uint32_t (&x)[2][W]) {
    if constexpr (W == 2) {
      uint2 a, b;
      lds_get<OFF, OFF + RECB>(codes, a, b);
      x[0][0] = a.x, x[0][1] = a.y, x[1][0] = b.x, x[1][1] = b.y;
    } else if constexpr (W == 8) {
      uint4 a, b, d, e;
      lds_get<OFF, OFF + 16, OFF + RECB, OFF + RECB + 16>(codes, a, b, codes, d, e);
      put(x[0], 0, a), put(x[0], 4, b), put(x[1], 0, d), put(x[1], 4, e);
    }
  }
  static __device__ __forceinline__ void put(uint32_t (&x)[W], int at, const uint4 &a) {
    x[at] = a.x, x[at + 1] = a.y, x[at + 2] = a.z, x[at + 3] = a.w;
  }
  template <int CODES, int PAIRS>
  __device__ __forceinline__ void get(uint32_t (&x)[2][W], uint4 (&p)[2][NG]) {
    if constexpr (W == 4) {
      uint4 a, b;
      lds_get<CODES, CODES + RECB, PAIRS, PAIRS + RECB>(codes, a, b, pairs, p[0][0], p[1][0]);
      put(x[0], 0, a), put(x[1], 0, b);
    } else {
      words<CODES>(x);
      lds_get<PAIRS, PAIRS + RECB>(pairs, p[0][0], p[1][0]);
    }
    more<PAIRS, 1>(p);
    if (lost) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (lost >> b & 1) {
#pragma unroll
          for (int j = 0; j < NG; ++j) p[b][j] = make_uint4(0x7fc0u, 0x7fc0u, 0x7fc0u, 0x7fc0u);
        }
    }
  }
  template <int PAIRS, int J>
  __device__ __forceinline__ void more(uint4 (&p)[2][NG]) {
    if constexpr (J < NG) {
      lds_get<PAIRS + 64 * J, PAIRS + 64 * J + RECB>(pairs, p[0][J], p[1][J]);
      more<PAIRS, J + 1>(p);
    }
  }
  __device__ __forceinline__ void keys() { get<0, 16 * DIM>(k, kp); }
  __device__ __forceinline__ void values() { get<8 * DIM, 16 * DIM + 64 * NG>(v, vp); }
  __device__ __forceinline__ uint4 kcode(int b, int w) const { return q4_codes(k[b][w]); }
  __device__ __forceinline__ void vcode(int w, uint4 &even, uint4 &odd) const {
    const uint4 u = q4_codes(v[0][w]), y = q4_codes(v[1][w]);   // x, y: 4 tokens of the even channel; z, w: odd
    even = make_uint4(u.x, u.y, y.x, y.y), odd = make_uint4(u.z, u.w, y.z, y.w);
  }
  __device__ __forceinline__ void kpair(int b, int j, float (&step)[4], float (&low)[4]) const {
    const uint32_t w[4] = {kp[b][j].x, kp[b][j].y, kp[b][j].z, kp[b][j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) step[i] = half_of(w[i], false) * c, low[i] = half_of(w[i], true);
  }
  __device__ __forceinline__ void vpair(int b, int j, float (&step)[4], float (&low)[4]) const {
    const uint32_t w[4] = {vp[b][j].x, vp[b][j].y, vp[b][j].z, vp[b][j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) step[i] = half_of(w[i], false), low[i] = half_of(w[i], true);
  }
};

template <int RECB>
__device__ __forceinline__ Pages pages_of(const Kv4Args &a, int seq, int h, int kend) {
  Pages p;
  p.bytes = (unsigned)(a.page >> 4) * RECB * a.hkv;      // below 2^27: 1024 heads of 16 records of 5 KB
  p.cache = (const char *)a.cache + (unsigned)h * ((unsigned)(a.page >> 4) * RECB);
  p.table = a.table + (int64_t)seq * a.per;
  p.pages = a.pages;
  p.last = (kend - 1) >> 4;
  p.shift = 31 - __builtin_clz((unsigned)a.page >> 4);
  p.base = p.page = 0;
  return p;
}

// Where share i of n equal shares of `all` (below 2^26) begins.
__device__ __forceinline__ int share_of(int all, int i, int n) {
  const unsigned each = (unsigned)all / (unsigned)n, rest = (unsigned)all - each * n;   // the first `rest` have one more
  return (int)(each * i + (i < (int)rest ? i : rest));
}

// Few rows: every wave streams its own run of tokens for the same 16 NQ rows,
// its records a tile ahead, straight to LDS (in registers they would leave
// room for half the waves); the waves' sums meet in LDS.  16 sequences of up to
// 8192, 64 + 8 heads of 128: 29 us for 106 MB, of which 21 are left without
// computing; the vector unit (42% busy) expands codes and applies pairs.
template <int DIM, int NQ, int X>
constexpr int stream_waves() {   // of a SIMD: what the registers allow
  return X == kF32 ? (DIM == 64 ? 3 : DIM == 128 ? 2 : 1) : DIM == 64 ? (NQ == 1 ? 4 : 2) : DIM == 128 && NQ == 1 ? 3 : 2;
}
template <int DIM, int GROUP, int NQ, int X>
__global__ __launch_bounds__(256, (stream_waves<DIM, NQ, X>())) void kv4_stream_kernel(const Kv4Args a, const Kv4Cut cut) {
  typedef Ring<DIM, GROUP> R;
  constexpr int TM = 16 * NQ, W = DIM / 32, LDO = DIM + 4, ST = R::STAGES;
  union Lds {
    char ring[4][ST][R::TILEB];
    struct {
      float o[4][16][LDO];
      float ml[4][16][2];
    } end;
  };
  __shared__ __attribute__((aligned(16))) Lds s;

  const unsigned run = blockIdx.x / (unsigned)a.hkv;
  const int h = (int)(blockIdx.x - run * a.hkv);     // heads are neighbours: a head's rows meet in one XCD's L2
  const Work k = find_work(a, cut, (int)run);
  note_joint(a, cut, k, (int)run, h, DIM);
  if (k.none) return;
  if (k.bad) {
    if ((int)run < cut.slots && cut.extra == 0) nan_share(a, (int)run, cut.slots, h, DIM);
    return;
  }
  const int rows_all = k.ql * a.g, m0 = k.tile * TM;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int mrows = rows_all - m0 < TM ? rows_all - m0 : TM;
  const float c = a.scale * 1.44269504088896340736f;
  const int kend = limit_of(a, k.len, k.ql, (int)((unsigned)(m0 + mrows - 1) / (unsigned)a.g));   // the last row's
  const int kall = limit_of(a, k.len, k.ql, (int)((unsigned)m0 / (unsigned)a.g));   // every row reaches these
  const int tiles = (kend + 31) >> 5, parts = k.nsplit * 4, mine = k.split * 4 + wave;
  const int t0 = share_of(tiles, mine, parts), t1 = share_of(tiles, mine + 1, parts);

  Pages pg = pages_of<R::RECB>(a, k.seq, h, kend);
  int lost = 0;                                // two bits a tile, the newest lowest
  // The last stages load the last tile again, so that every step has as many loads in flight.
  auto fetch = [&](int t, int stage) __attribute__((always_inline)) {
    if (t >= t1) t = t1 - 1;
    if (2 * t - pg.base >= 64) pg.load(2 * t);
    lost <<= 2;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int page = pg.of(2 * t + b);
      if (page < 0) lost |= 1 << b;
      R::load(pg.template at<R::RECB>(page, 2 * t + b), s.ring[wave][stage] + b * R::RECB);
    }
  };
  if (t0 < t1) {
    pg.load(2 * t0);
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(t0 + i, i);
  }
  Rows<DIM, GROUP, NQ, X> rows;
  rows.start(a, k, h, m0, rows_all, c);
  if (t0 < t1) {
    RingTile<DIM, GROUP> src;
    src.c = c;
    const uint32_t base = (uint32_t)(uintptr_t)(lds_void_t *)s.ring[wave][0];
    int now = 0, next = ST - 1;
    for (int t = t0; t < t1; ++t) {
      fetch(t + ST - 1, next);                 // over the tile of the step before, whose reads have returned
      wait_loads<(ST - 1) * R::LOADS>();
      src.codes = base + now * R::TILEB + lane * (W * 4);
      src.pairs = base + now * R::TILEB + lg * 16;
      src.lost = lost >> (2 * (ST - 1)) & 3;
      if (32 * t + 32 <= kall) rows.template attend<false>(src, 32 * t);
      else rows.template attend<true>(src, 32 * t);
      now = now + 1 == ST ? 0 : now + 1;
      next = next + 1 == ST ? 0 : next + 1;
    }
    wait_loads<0>();
  }

  rows.finish(k.over);
  __syncthreads();                             // the rings are read out and nothing is in flight to them
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (n > 0) __syncthreads();
    if (lg == 0) s.end.ml[wave][r16][0] = rows.m[n], s.end.ml[wave][r16][1] = rows.ls[n];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float y[8];
      rows.channels(n, w, y);
      float4 *p = (float4 *)&s.end.o[wave][r16][32 * w + 8 * lg];
      p[0] = make_float4(y[0], y[1], y[2], y[3]);
      p[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
    __syncthreads();
    // thread: one row, every 16th group of four channels
    const int r = threadIdx.x >> 4, m = 16 * n + r;
    if (m < mrows) {
      float top = s.end.ml[0][r][0];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, s.end.ml[w][r][0]);
      const float ref = top == kNegInf ? 0.0f : top;
      float f[4], l2 = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = exp2_any(s.end.ml[w][r][0] - ref);
        l2 = __builtin_fmaf(f[w], s.end.ml[w][r][1], l2);
      }
      const float inv = k.nsplit > 1 ? 1.0f : l2 == 0.0f ? 0.0f : 1.0f / l2;
      const int mm = m0 + m;
      const int64_t at = row_at(a, k, h, mm, (int)((unsigned)mm / (unsigned)a.g)) * DIM;
      float *to = part_sum(a, cut, (int)run, h, m, DIM);
#pragma unroll
      for (int i = 0; i < DIM / 64; ++i) {
        const int ch = 64 * i + 4 * (threadIdx.x & 15);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 z = *(const float4 *)&s.end.o[w][r][ch];
          y[0] = __builtin_fmaf(f[w], z.x, y[0]), y[1] = __builtin_fmaf(f[w], z.y, y[1]);
          y[2] = __builtin_fmaf(f[w], z.z, y[2]), y[3] = __builtin_fmaf(f[w], z.w, y[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= inv;
        if (k.nsplit > 1) *(float4 *)(to + ch) = make_float4(y[0], y[1], y[2], y[3]);
        else if (a.obf16) *(uint2 *)((uint16_t *)a.out + at + ch) = make_uint2(pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3]));
        else *(float4 *)((float *)a.out + at + ch) = make_float4(y[0], y[1], y[2], y[3]);
      }
      if (k.nsplit > 1 && (threadIdx.x & 15) == 0) *part_ml(a, cut, (int)run, h, m, DIM) = make_float2(top, l2);
    }
  }
}

// TOK tokens in LDS, codes expanded once for the workgroup, as operands: 64
// lanes' 16 bytes each, so every read is 1 KB in order.
template <int DIM, int GROUP>
struct LdsTile {
  static constexpr int NG = DIM / GROUP, W = DIM / 32, TB = DIM == 256 ? 2 : 4, TOK = 16 * TB;
  uint4 k[TB * W][64];
  uint4 v[TB / 2 * (DIM / 16)][64];          // or values, float16
  float pair[4][NG][TOK];    // keys' steps (times scale log2 e) and low ends, values' steps and low ends
  __attribute__((aligned(16))) uint32_t note[4];          // of each wave, on its records' values: greatest magnitude as bits, then whether float16 fits
};
template <int DIM, int GROUP>
struct LdsPart {             // 32 tokens of it
  static constexpr int W = DIM / 32;
  const LdsTile<DIM, GROUP> &t;
  int p;
  __device__ __forceinline__ void keys() {}
  __device__ __forceinline__ void values() {}
  __device__ __forceinline__ uint4 kcode(int b, int w) const { return t.k[(2 * p + b) * W + w][threadIdx.x & 63]; }
  __device__ __forceinline__ void vcode(int w, uint4 &even, uint4 &odd) const {
    even = t.v[p * 2 * W + 2 * w][threadIdx.x & 63];
    odd = t.v[p * 2 * W + 2 * w + 1][threadIdx.x & 63];
  }
  __device__ __forceinline__ void take(const float (&from)[LdsTile<DIM, GROUP>::TOK], int b, float (&x)[4]) const {
    const float4 u = *(const float4 *)&from[32 * p + 16 * b + 4 * ((threadIdx.x & 63) >> 4)];
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
  }
  __device__ __forceinline__ void kpair(int b, int j, float (&step)[4], float (&low)[4]) const {
    take(t.pair[0][j], b, step), take(t.pair[1][j], b, low);
  }
  __device__ __forceinline__ void vpair(int b, int j, float (&step)[4], float (&low)[4]) const {
    take(t.pair[2][j], b, step), take(t.pair[3][j], b, low);
  }
};

// Many rows: four waves of 16 NQ rows each share the tokens.  A tile's codes
// come to registers while the tile before is worked on, and are expanded into
// the other half of LDS behind it: keys to bfloat16 codes; values, for bfloat16
// queries and outputs, to float16 numbers in a unit that makes the first tile's greatest
// one 8 to 16.  Should a tile not fit that (a value past 2^14 units; a token's whole group
// below 2^-9 units, where its step would run out of float16's bits, or 0: if that token has
// a row's whole weight, what is left are weights that float16 rounds to 2^-33 of it; a
// NaN, which must not meet a weight of 0), the rest is done by the values' codes,
// as for float32 queries.  Two loops, not a branch in one: that spilled registers.
// 8 sequences of 4096, causal, 32 + 8 heads of 128: 1408 us, 781 TFLOP/s; the
// matrix unit is 26% and the vector unit 45% busy (two prompts of 1024 and 657).
constexpr float kHalfMost = 0x1p14f, kHalfLeast = 0x1p-9f;
template <int DIM, int GROUP, int NQ, int X>
__global__ __launch_bounds__(256, 2) void kv4_tile_kernel(const Kv4Args a, const Kv4Cut cut) {
  typedef LdsTile<DIM, GROUP> Lds;
  constexpr int NG = Lds::NG, W = Lds::W, TB = Lds::TB, TOK = Lds::TOK, TM = 64 * NQ, REC = 4 * DIM + 32 * NG;
  constexpr int WPW = TB * W / 4;            // words of a record's lane that a wave expands
  constexpr int SW = TB == 4 ? 32 * NG : 16 * NG, NS = (SW + 63) / 64;   // pairs a wave brings
  __shared__ __attribute__((aligned(16))) Lds s[2];

  const unsigned run = blockIdx.x / (unsigned)a.hkv;
  const int h = (int)(blockIdx.x - run * a.hkv);     // heads are neighbours: a head's rows meet in one XCD's L2
  const Work k = find_work(a, cut, (int)run);
  note_joint(a, cut, k, (int)run, h, DIM);
  if (k.none) return;
  if (k.bad) {
    if ((int)run < cut.slots && cut.extra == 0) nan_share(a, (int)run, cut.slots, h, DIM);
    return;
  }
  const int rows_all = k.ql * a.g, m0 = k.tile * TM;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int last = m0 + TM < rows_all ? m0 + TM : rows_all;              // past the workgroup's last row
  const int w0 = m0 + 16 * NQ * wave, w1 = w0 + 16 * NQ < last ? w0 + 16 * NQ : last;
  const float c = a.scale * 1.44269504088896340736f;
  Rows<DIM, GROUP, NQ, X> rows;
  rows.start(a, k, h, w0, rows_all, c);

  auto limit = [&](int m) __attribute__((always_inline)) {
    return limit_of(a, k.len, k.ql, (int)((unsigned)m / (unsigned)a.g));
  };
  const int kend = limit(last - 1);
  const int wend = w1 > w0 ? limit(w1 - 1) : 0, wall = w1 > w0 ? limit(w0) : 0;   // one, all of this wave's rows reach these
  const int tiles = (kend + TOK - 1) / TOK;
  const int t0 = share_of(tiles, k.split, k.nsplit), t1 = share_of(tiles, k.split + 1, k.nsplit);
  if (t0 < t1) {
    Pages pg = pages_of<4 * REC>(a, k.seq, h, kend);
    const int blk = TB == 4 ? wave : wave >> 1, off = TB == 4 ? 0 : WPW * (wave & 1);
    const int soff = TB == 4 ? 0 : 16 * NG * (wave & 1);
    constexpr int GS = GROUP / 32, NV = WPW > GS ? WPW / GS : 1;   // groups of the words that a wave expands
    uint32_t kw[WPW], vw[WPW], sw[NS];
    uint4 vp[X == kBf16 ? NV : 1];                 // their pairs of this lane's four tokens
    float unit = 1.0f;
    auto fetch = [&](int t) __attribute__((always_inline)) {
      if (TB * t - pg.base >= 64) pg.load(TB * t);
      const int page = pg.of(TB * t + blk);
      const uint32_t *p = (const uint32_t *)pg.template at<4 * REC>(page, TB * t + blk);
      load_words(p + lane * W + off, kw);
      load_words(p + 2 * DIM + lane * W + off, vw);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int x = lane + 64 * i;
        sw[i] = x < SW ? p[4 * DIM + soff + x] : 0u;
        if (page < 0) sw[i] = 0x7fc0u;
      }
      if constexpr (X == kBf16) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          vp[i] = *(const uint4 *)(p + 4 * DIM + 16 * NG + 16 * (off / GS + i) + 4 * lg);
          if (page < 0) vp[i] = make_uint4(0x7fc0u, 0x7fc0u, 0x7fc0u, 0x7fc0u);
        }
      }
    };
    // Magnitude, as bits, of the greatest value of a group of one token (NaN: above infinity's; 0: float32's
    // least number, which float16 does not fit; of keys and of tokens that nobody attends to: 0), by the lane that
    // holds its pair.
    auto size_of = [&](int t, int i) __attribute__((always_inline)) {
      const int x = soff + lane + 64 * i;
      const float step = half_of(sw[i], false), low = half_of(sw[i], true);
      const float far = __builtin_fmaf(15.0f, step, low);          // a NaN step makes it one
      const uint32_t u = __float_as_uint(far) & 0x7fffffffu, l = __float_as_uint(low) & 0x7fffffffu;
      const bool counts = lane + 64 * i < SW && x >= 16 * NG && TOK * t + 16 * blk + (x & 15) < kend;
      return !counts ? 0u : (u > l ? u : l) | 1u;
    };
    // CODES: values as bfloat16 codes, else as float16 numbers.
    auto expand = [&](Lds &d, int t, auto codes) __attribute__((always_inline)) {
      constexpr bool CODES = decltype(codes)::value;
      uint32_t st[NV][2], lo[NV][2];
      if constexpr (!CODES) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint32_t w[4] = {vp[i].x, vp[i].y, vp[i].z, vp[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (TOK * t + 16 * blk + 4 * lg + e >= kend) w[e] = 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            st[i][e] = pk_half(half_of(w[2 * e], false) * unit, half_of(w[2 * e + 1], false) * unit);
            lo[i][e] = pk_half(half_of(w[2 * e], true) * unit, half_of(w[2 * e + 1], true) * unit);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < WPW; ++i) {
        const int w = off + i;
        d.k[blk * W + w][lane] = q4_codes(kw[i]);
        uint4 y;
        if constexpr (CODES) {
          y = q4_codes(vw[i]);
        } else {
          y = q4_codes_half(vw[i]);
          const int j = WPW > GS ? i / GS : 0;
          y.x = fma_half(y.x, st[j][0], lo[j][0]), y.y = fma_half(y.y, st[j][1], lo[j][1]);
          y.z = fma_half(y.z, st[j][0], lo[j][0]), y.w = fma_half(y.w, st[j][1], lo[j][1]);
        }
        uint2 *e = (uint2 *)&d.v[(blk >> 1) * (DIM / 16) + 2 * w][lane];
        uint2 *o = (uint2 *)&d.v[(blk >> 1) * (DIM / 16) + 2 * w + 1][lane];
        e[blk & 1] = make_uint2(y.x, y.y);
        o[blk & 1] = make_uint2(y.z, y.w);
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int x = soff + lane + 64 * i;
        const int kv = x / (16 * NG), j = x / 16 % NG;
        if (lane + 64 * i < SW && (CODES || kv == 0)) {
          d.pair[2 * kv][j][16 * blk + (x & 15)] = half_of(sw[i], false) * (kv ? 1.0f : c);
          d.pair[2 * kv + 1][j][16 * blk + (x & 15)] = half_of(sw[i], true);
        }
      }
      if constexpr (!CODES) {
        bool fits = true;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const uint32_t u = size_of(t, i);
          const float x = __uint_as_float(u) * unit;
          fits &= u == 0u || (x < kHalfMost && x >= kHalfLeast);
        }
        const bool all = __all(fits);
        if (lane == 0) d.note[wave] = all;
      }
    };
    constexpr std::integral_constant<bool, true> kCodes{};
    constexpr std::integral_constant<bool, false> kNumbers{};

    pg.load(TB * t0);
    fetch(t0);
    int t = t0;
    if constexpr (X == kBf16) {
      uint32_t most = 0u;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const uint32_t u = size_of(t0, i);
        most = most > u ? most : u;
      }
      most = over_row(most);
#pragma unroll
      for (int i = 0; i < 64; i += 16) {
        const uint32_t u = of_lane(most, i);
        most = most > u ? most : u;
      }
      if (lane == 0) s[1].note[wave] = most;   // that of s[0] is written next
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = s[1].note[i];
        most = most > u ? most : u;
      }
      // 2^(130 - e) for the biased exponent e of the greatest, within 2^+-100 (nothing finite, nothing but 0: 1)
      const int e = (int)(most >> 23);
      const int up = e == 0 || e == 255 ? 0 : 130 - e < -100 ? -100 : 130 - e > 100 ? 100 : 130 - e;
      unit = __uint_as_float((uint32_t)(up + 127) << 23);
      expand(s[0], t0, kNumbers);
      __syncthreads();
      for (; t < t1; ++t) {
        const Lds &d = s[(t - t0) & 1];
        const uint4 fits = *(const uint4 *)d.note;
        if (!__builtin_amdgcn_readfirstlane(fits.x & fits.y & fits.z & fits.w)) break;   // all waves
        if (t + 1 < t1) fetch(t + 1);
#pragma unroll
        for (int p = 0; p < TB / 2; ++p) {
          const int first = t * TOK + 32 * p;
          LdsPart<DIM, GROUP> src = {d, p};
          if (first + 32 <= wall) rows.template attend_half<false>(src, first);
          else if (first < wend) rows.template attend_half<true>(src, first);
        }
        if (t + 1 < t1) expand(s[(t + 1 - t0) & 1], t + 1, kNumbers);   // read last before the barrier of the step before
        __syncthreads();
      }
      rows.leave_half(unit);
    }
    if (t < t1) {                            // the registers still hold tile t; of what it is in LDS only `note` is read
      expand(s[(t - t0) & 1], t, kCodes);
      __syncthreads();
    }
    for (; t < t1; ++t) {
      const Lds &d = s[(t - t0) & 1];
      if (t + 1 < t1) fetch(t + 1);
      constexpr int U = X == kBf16 ? 1 : TB / 2;
#pragma unroll U
      for (int p = 0; p < TB / 2; ++p) {
        const int first = t * TOK + 32 * p;
        LdsPart<DIM, GROUP> src = {d, p};
        if (X != kBf16 && first + 32 <= wall) rows.template attend<false>(src, first);
        else if (first < wend) rows.template attend<true>(src, first);
      }
      if (t + 1 < t1) expand(s[(t + 1 - t0) & 1], t + 1, kCodes);
      __syncthreads();
    }
  }

  rows.finish(k.over);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int mm = w0 + 16 * n + r16;
    if (mm >= w1) continue;
    const int64_t at = row_at(a, k, h, mm, (int)((unsigned)mm / (unsigned)a.g)) * DIM + 8 * lg;
    float *p = part_sum(a, cut, (int)run, h, mm - m0, DIM);
    const float inv = rows.ls[n] == 0.0f ? 0.0f : 1.0f / rows.ls[n];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float y[8];
      rows.channels(n, w, y);
      if (k.nsplit > 1) {
        float4 *z = (float4 *)(p + 32 * w + 8 * lg);
        z[0] = make_float4(y[0], y[1], y[2], y[3]);
        z[1] = make_float4(y[4], y[5], y[6], y[7]);
      } else if (a.obf16) {
        uint32_t z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = pk_bf16(y[2 * e] * inv, y[2 * e + 1] * inv);
        *(uint4 *)((uint16_t *)a.out + at + 32 * w) = make_uint4(z[0], z[1], z[2], z[3]);
      } else {
        float4 *z = (float4 *)((float *)a.out + at + 32 * w);
        z[0] = make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
        z[1] = make_float4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
      }
    }
    if (k.nsplit > 1 && lg == 0) *part_ml(a, cut, (int)run, h, mm - m0, DIM) = make_float2(rows.m[n], rows.ls[n]);
  }
}

// Joins the runs of a row where they are few: 16 lanes a row, 16 rows a
// workgroup, lane l takes channels 4 l .. +3 of every 64.  (A wave a row, as for
// many runs, took 15.8 us for 1681 query tokens of 32 heads, this 8.1.)
template <int DIM>
__global__ __launch_bounds__(256) void kv4_join_few_kernel(const Kv4Args a, const Kv4Cut cut) {
  constexpr int CH = DIM / 64;
  const int l16 = threadIdx.x & 15;
  // tm is a multiple of 16: the rows of a workgroup are of one tile
  const unsigned row = blockIdx.x * 16, x = row >> cut.tm_log;
  const int m0 = (int)(row & (cut.tm - 1)), m = m0 + (int)(threadIdx.x >> 4);
  const unsigned slot = x / (unsigned)a.hkv;
  const int h = (int)(x - slot * a.hkv);
  const Joint k = joints(a, cut, DIM)[slot];
  const int mm = k.m0 + m, n = k.runs;
  if (n < 0 && m0 == 0) nan_share(a, (int)slot, cut.slots, h, DIM);
  if (n <= 1 || mm >= k.ql * a.g) return;         // uniform over a row's lanes
  const int64_t next = (int64_t)a.hkv * cut.tm;   // rows from one run to the next
  const float2 *ml = part_ml(a, cut, k.first, h, m, DIM);
  const float2 u0 = l16 < n ? ml[l16 * next] : make_float2(kNegInf, 0.0f);
  float top = u0.x;
  for (int s = 16 + l16; s < n; s += 16) top = fmaxf(top, ml[s * next].x);
  top = group_max<16>(top);
  const float ref = top == kNegInf ? 0.0f : top;
  float l = 0.0f;
  f32x4_t o[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) o[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const float *p = part_sum(a, cut, k.first, h, m, DIM) + 4 * l16;
  for (int s0 = 0; s0 < n; s0 += 16) {
    const float2 u = s0 == 0 ? u0 : s0 + l16 < n ? ml[(s0 + l16) * next] : make_float2(kNegInf, 0.0f);
    const float f = exp2_any(u.x - ref);
    l += f * u.y;
    const int s1 = n - s0 < 16 ? n - s0 : 16;
#pragma unroll 4
    for (int s = 0; s < s1; ++s) {
      const float fs = __shfl(f, s, 16);
      const float *q = p + (s0 + s) * next * DIM;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const f32x4_t z = *(const f32x4_t *)(q + 64 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = __builtin_fmaf(fs, z[e], o[i][e]);
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) l += __shfl_xor(l, d, 64);
  const int64_t at = row_at(a, k, h, mm, (int)((unsigned)mm / (unsigned)a.g)) * DIM + 4 * l16;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const f32x4_t y = o[i] * inv;
    if (a.obf16) *(uint2 *)((uint16_t *)a.out + at + 64 * i) = make_uint2(pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3]));
    else *(f32x4_t *)((float *)a.out + at + 64 * i) = y;
  }
}

// Where they may be many: PARTS waves share them, lane l takes the DIM / 64
// channels from DIM / 64 l on.  A wave has 64 runs' factors before the first of
// their sums is read, so the reads do not wait for each other.
template <int DIM, int PARTS>
__global__ __launch_bounds__(64 * PARTS) void kv4_join_kernel(const Kv4Args a, const Kv4Cut cut) {
  constexpr int CH = DIM / 64;
  __shared__ float s_o[PARTS][DIM];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned row = blockIdx.x, x = row >> cut.tm_log;
  const int m = (int)(row & (cut.tm - 1)), y = wave;
  const unsigned slot = x / (unsigned)a.hkv;
  const int h = (int)(x - slot * a.hkv);
  const Joint k = joints(a, cut, DIM)[slot];
  const int mm = k.m0 + m, n = k.runs;
  if (n < 0 && m == 0) nan_share(a, (int)slot, cut.slots, h, DIM);
  if (n <= 1 || mm >= k.ql * a.g) return;         // uniform over what shares LDS
  const int64_t next = (int64_t)a.hkv * cut.tm;   // rows from one run to the next
  const float2 *ml = part_ml(a, cut, k.first, h, m, DIM);
  const float2 u0 = lane < n ? ml[lane * next] : make_float2(kNegInf, 0.0f);
  float top = u0.x;
  for (int s = 64 + lane; s < n; s += 64) top = fmaxf(top, ml[s * next].x);
  top = group_max<64>(top);
  const float ref = top == kNegInf ? 0.0f : top;
  float l = 0.0f, o[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) o[i] = 0.0f;
  const float *p = part_sum(a, cut, k.first, h, m, DIM) + CH * lane;
  for (int s0 = 0; s0 < n; s0 += 64) {
    const float2 u = s0 == 0 ? u0 : s0 + lane < n ? ml[(s0 + lane) * next] : make_float2(kNegInf, 0.0f);
    const float f = exp2_any(u.x - ref);
    l += f * u.y;
    const int s1 = n - s0 < 64 ? n - s0 : 64;
#pragma unroll 8
    for (int s = y; s < s1; s += PARTS) {
      const float fs = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), s));
      const float *q = p + (s0 + s) * next * DIM;
      float z[CH];
      if constexpr (CH == 1) {
        z[0] = q[0];
      } else if constexpr (CH == 2) {
        const float2 v = *(const float2 *)q;
        z[0] = v.x, z[1] = v.y;
      } else {
        const float4 v = *(const float4 *)q;
        z[0] = v.x, z[1] = v.y, z[2] = v.z, z[3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) o[i] = __builtin_fmaf(fs, z[i], o[i]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d, 64);
#pragma unroll
  for (int i = 0; i < CH; ++i) s_o[y][CH * lane + i] = o[i];
  __syncthreads();
  if (y > 0) return;
#pragma unroll
  for (int i = 0; i < CH; ++i)
    for (int w = 1; w < PARTS; ++w) o[i] += s_o[w][CH * lane + i];
  const int64_t at = row_at(a, k, h, mm, (int)((unsigned)mm / (unsigned)a.g)) * DIM + CH * lane;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < CH; ++i) store_out(a, at + i, o[i] * inv);
}

template <int DIM, int GROUP>
hipError_t launch_group(const Kv4Args &a, const Kv4Cut &cut, const Kv4Plan &p, hipStream_t st) {
  constexpr bool WIDE = DIM < 256;      // as kv4_plan has it
  const unsigned grid = (unsigned)((int64_t)(p.slots + p.extra) * a.hkv);
#define RUN(KERNEL, NQ, X) KERNEL<DIM, GROUP, NQ, X><<<grid, 256, 0, st>>>(a, cut)
  const bool mixed = a.qbf16 && !a.obf16;
  if (p.tile) {
    if (!a.qbf16) RUN(kv4_tile_kernel, 1, kF32);
    else if (mixed) RUN(kv4_tile_kernel, 1, kMixed);
    else if constexpr (WIDE && DIM / GROUP < 4) RUN(kv4_tile_kernel, 2, kBf16);
    else RUN(kv4_tile_kernel, 1, kBf16);
  } else {
    if (!a.qbf16) RUN(kv4_stream_kernel, 1, kF32);
    else if (mixed) RUN(kv4_stream_kernel, 1, kMixed);
    else if (p.nq == 1) RUN(kv4_stream_kernel, 1, kBf16);
    else if constexpr (WIDE) RUN(kv4_stream_kernel, 2, kBf16);
    else return hipErrorInvalidValue;
  }
#undef RUN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.extra == 0) return e;
  const int64_t rows = (int64_t)p.slots * a.hkv * p.tm;
  if (p.most > 16) kv4_join_kernel<DIM, 16><<<(unsigned)rows, 1024, 0, st>>>(a, cut);
  else if (p.most > 8) kv4_join_kernel<DIM, 4><<<(unsigned)rows, 256, 0, st>>>(a, cut);
  else kv4_join_few_kernel<DIM><<<(unsigned)(rows / 16), 256, 0, st>>>(a, cut);
  return hipGetLastError();
}

hipError_t launch_dim64(const Kv4Args &a, const Kv4Cut &cut, const Kv4Plan &p, hipStream_t st);
hipError_t launch_dim128(const Kv4Args &a, const Kv4Cut &cut, const Kv4Plan &p, hipStream_t st);
hipError_t launch_dim256(const Kv4Args &a, const Kv4Cut &cut, const Kv4Plan &p, hipStream_t st);

}  // namespace kv4
}  // namespace slim
