// Attention over the 4-bit key/value cache on the matrix cores of gfx950.
//
//   S[r, t] = scale sum_c q[r, c] k[t, c],  o[r] = sum_t softmax_t(S[r, t]) v[t]   over t < limit(r),
//   k[t, c] = code[t, c] step[t, j] + low[t, j]   (j the group of c; v alike)
//
// Nothing is dequantized.  Codes are exact in bfloat16, so with Q_j the sum
// of q over group j
//   S[r, t] = scale sum_j (step[t, j] (sum_{c in j} q[r, c] code[t, c]) + low[t, j] Q_j[r]),
//   o[r, c] = sum_t (P[r, t] step[t, j]) code[t, c] + sum_t P[r, t] low[t, j],
// where the products with codes go to the matrix cores and the rest is float32.
// P step is the one thing that is rounded: to bfloat16 where q is bfloat16
// (as the outputs are), to three bfloat16 terms where q is float32.
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

// The row tile of a slot: sequence, its first query token, its query tokens,
// the tile's number inside it.
struct RowTile {
  int64_t q0;
  int seq, ql, tile;
  bool none, bad;            // no tile in this slot; bounds out of order
};

// Uneven queries: every wave works the tiles out from the bounds (lane l
// takes consecutive sequences), so no table or copy to the host is needed.
__device__ __forceinline__ RowTile find_tile(const Kv4Args &a, int64_t slot, int tm) {
  RowTile t = {};
  const int64_t g = a.hq / a.hkv;
  if (!a.offsets) {
    const int64_t ql = a.tq / a.b;
    const int tiles = (int)((ql * g + tm - 1) / tm);
    t.seq = (int)(slot / tiles);
    t.tile = tiles - 1 - (int)(slot - (int64_t)t.seq * tiles);   // the longest first
    t.ql = (int)ql;
    t.q0 = t.seq * ql;
    return t;
  }
  const int lane = threadIdx.x & 63, b = (int)a.b, per = (b + 63) >> 6;
  int64_t mine = 0;
  bool wrong = false;
  for (int i = 0; i < per; ++i) {
    const int s = lane * per + i;
    if (s >= b) break;
    const int64_t lo = a.offsets[s], hi = a.offsets[s + 1];
    wrong |= lo < 0 || hi < lo || hi > a.tq;
    mine += ((hi - lo) * g + tm - 1) / tm;
  }
  if (__any(wrong)) {
    t.bad = true;
    return t;
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t up = __shfl_up(incl, d, 64);
    if (lane >= d) incl += up;
  }
  const uint64_t past = __ballot(incl > slot);
  if (!past) {
    t.none = true;
    return t;
  }
  const int own = __ffsll((unsigned long long)past) - 1;
  int64_t left = slot - __shfl(incl - mine, own, 64);
  int s = own * per;
  for (;; ++s) {             // ends: lane `own` has more than `left` tiles
    const int64_t lo = a.offsets[s], hi = a.offsets[s + 1];
    const int64_t n = ((hi - lo) * g + tm - 1) / tm;
    if (left < n) {
      t.seq = s, t.q0 = lo, t.ql = (int)(hi - lo), t.tile = (int)(n - 1 - left);
      return t;
    }
    left -= n;
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

// Bounds out of order: the slots share the rows out and make them NaN.
__device__ __forceinline__ void nan_share(const Kv4Args &a, int64_t slot, int64_t slots, int h, int dim) {
  const int64_t each = (a.tq + slots - 1) / slots, g = a.hq / a.hkv;
  const int64_t lo = slot * each, hi = lo + each < a.tq ? lo + each : a.tq;
  for (int64_t i = lo * g * dim + threadIdx.x; i < hi * g * dim; i += blockDim.x) {
    const int64_t c = i % dim, r = i / dim;
    store_out(a, (r / g * a.hq + h * g + r % g) * dim + c, kNaN);
  }
}

// What a wave keeps of its 16 NQ rows, and one step of the attention: 32
// tokens (two records) for all of them.
//
// Weights are 2^(S - m) with S in powers of two and m the row's reference: the
// maximum of the row's first tokens, moved up only once a score exceeds it by
// `kSlack` (weights then reach 2^kSlack at most, far inside float32 and
// bfloat16).  So a step needs no maximum across lanes and no rescaling, but
// for the first ones: each lane compares its own scores.
//
// Weights times steps are rounded to the sum of two bfloat16 terms (2^-16):
// with one term (2^-9) the outputs' error was twice that of their own
// rounding to bfloat16.  Float32 queries and weights enter as three terms.
constexpr float kSlack = 10.0f;

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

template <int DIM, int GROUP, int NQ, bool XF32>
struct Rows {
  static constexpr int NG = DIM / GROUP, W = DIM / 32, GS = GROUP / 32, NTQ = XF32 ? 3 : 1, NTP = XF32 ? 3 : 2;
  uint4 qf[NQ][W][NTQ];      // the rows' queries as operands
  float qs[NQ][NG];          // their sums over each group, times scale log2 e
  int lim[NQ];               // tokens a row attends to
  float m[NQ], thr[NQ];      // reference; what a score may exceed it by (-inf: no reference yet)
  float ls[NQ], pl[NQ][NG];  // this lane's share of sum P and of sum P low
  f32x4_t o[NQ][DIM / 16];   // sum P step code, rows (tokens' channels) by columns (rows)

  // Rows m0 + 16 n + lane % 16 of the sequence, those from `rows` on as zeros that attend to nothing.
  __device__ __forceinline__ void start(const Kv4Args &a, const RowTile &rt, int h, int g, int len, int m0, int rows,
                                        float c) {
    const int r16 = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int mm = m0 + 16 * n + r16;
      const bool real = mm < rows;
      const int i = (real ? mm : 0) / g;
      lim[n] = real ? limit_of(a, len, rt.ql, i) : 0;
      const int64_t at = ((rt.q0 + i) * a.hq + (int64_t)h * g + ((real ? mm : 0) - i * g)) * DIM + 8 * lg;
#pragma unroll
      for (int j = 0; j < NG; ++j) qs[n][j] = pl[n][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        if constexpr (XF32) {
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
#pragma unroll
      for (int i2 = 0; i2 < DIM / 16; ++i2) o[n][i2] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // 32 tokens from token `first` on.  Src: codes and pairs of the two records; a key's step is
  // given times scale log2 e.  EDGE: some row does not attend to all of them.
  template <bool EDGE, class Src>
  __device__ __forceinline__ void attend(const Src &src, int first) {
    const int tok = first + 4 * ((threadIdx.x & 63) >> 4);   // of entry 0; entry 4 b + v: + 16 b + v
    float x[NQ][8];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[n][e] = -m[n];
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
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if (EDGE) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (tok + 16 * (e >> 2) + (e & 3) >= lim[n]) x[n][e] = kNegInf;
      }
      float top = fmaxf(fmaxf(fmaxf(x[n][0], x[n][1]), fmaxf(x[n][2], x[n][3])),
                        fmaxf(fmaxf(x[n][4], x[n][5]), fmaxf(x[n][6], x[n][7])));
      if (__any(top > thr[n])) raise(n, top, x[n]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[n][e] = exp2_any(x[n][e]);
        ls[n] += x[n][e];
      }
    }
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
          if (EDGE && tok + 16 * (e >> 2) + (e & 3) >= lim[n]) y[e] = z = 0.0f;   // NaN pairs of masked tokens
          pl[n][j] = __builtin_fmaf(x[n][e], z, pl[n][j]);
        }
        if constexpr (XF32)
          split3(make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3])),
                 make_uint4(__float_as_uint(y[4]), __float_as_uint(y[5]), __float_as_uint(y[6]), __float_as_uint(y[7])),
                 pf[n]);
        else
          split2(y, pf[n]);
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

  // A new reference for the rows that need one: the maximum over the step's tokens.
  __device__ __forceinline__ void raise(int n, float top, float (&x)[8]) {
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const bool up = top > thr[n];
    const float f = !up ? 1.0f : thr[n] == kNegInf ? 0.0f : exp2_any(-top);   // sums of no token are 0
    const float by = up ? top : 0.0f;
    m[n] += by;
    if (up) thr[n] = kSlack;
    ls[n] *= f;
#pragma unroll
    for (int j = 0; j < NG; ++j) pl[n][j] *= f;
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
        pl[n][j] += __shfl_xor(pl[n][j], 16, 64);
        pl[n][j] += __shfl_xor(pl[n][j], 32, 64);
#pragma unroll
        for (int w = GS * j; w < GS * (j + 1); ++w) o[n][2 * w] += pl[n][j], o[n][2 * w + 1] += pl[n][j];
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
  int64_t pages;
  int last, shift, base, page;
  __device__ __forceinline__ void load(int from) {
    base = from;
    const int b = from + (int)(threadIdx.x & 63);
    page = table[(b < last ? b : last) >> shift];
    if (page < 0 || page >= pages) page = -1;
  }
  // Of record b (past the last one: of the last); uniform over the wave.
  __device__ __forceinline__ int of(int b) const { return __builtin_amdgcn_readlane(page, b - base); }
};

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

// Two records in a wave's registers, codes expanded as they are used.
template <int DIM, int GROUP>
struct RegTile {
  static constexpr int NG = DIM / GROUP, W = DIM / 32, REC = 4 * DIM + 32 * NG;
  uint32_t k[2][W], v[2][W];
  uint4 kp[2][NG], vp[2][NG];
  bool lost[2];
  float c;
  __device__ __forceinline__ void load(const uint32_t *cache, int64_t heads, int h, int pb, const Pages &pg, int blk) {
    const int lane = threadIdx.x & 63, lg = lane >> 4;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int page = pg.of(blk + b), at = blk + b < pg.last ? blk + b : pg.last;
      lost[b] = page < 0;
      const uint32_t *p = cache + (((int64_t)(page < 0 ? 0 : page) * heads + h) * pb + (at & (pb - 1))) * REC;
      load_words(p + lane * W, k[b]);
      load_words(p + 2 * DIM + lane * W, v[b]);
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        kp[b][j] = *(const uint4 *)(p + 4 * DIM + 16 * j + 4 * lg);
        vp[b][j] = *(const uint4 *)(p + 4 * DIM + 16 * NG + 16 * j + 4 * lg);
      }
    }
  }
  __device__ __forceinline__ void spoil() {
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (lost[b]) {
#pragma unroll
        for (int j = 0; j < NG; ++j) kp[b][j] = vp[b][j] = make_uint4(0x7fc0u, 0x7fc0u, 0x7fc0u, 0x7fc0u);
      }
  }
  __device__ __forceinline__ uint4 kcode(int b, int w) const { return q4_codes(k[b][w]); }
  __device__ __forceinline__ void vcode(int w, uint4 &even, uint4 &odd) const {
    const uint4 u = q4_codes(v[0][w]), y = q4_codes(v[1][w]);   // x, y: 4 tokens of the even channel; z, w: odd
    even = make_uint4(u.x, u.y, y.x, y.y), odd = make_uint4(u.z, u.w, y.z, y.w);
  }
  __device__ __forceinline__ void kpair(int b, int j, float (&step)[4], float (&low)[4]) const {
    const uint32_t w[4] = {kp[b][j].x, kp[b][j].y, kp[b][j].z, kp[b][j].w};
#pragma unroll
    for (int v2 = 0; v2 < 4; ++v2) step[v2] = half_of(w[v2], false) * c, low[v2] = half_of(w[v2], true);
  }
  __device__ __forceinline__ void vpair(int b, int j, float (&step)[4], float (&low)[4]) const {
    const uint32_t w[4] = {vp[b][j].x, vp[b][j].y, vp[b][j].z, vp[b][j].w};
#pragma unroll
    for (int v2 = 0; v2 < 4; ++v2) step[v2] = half_of(w[v2], false), low[v2] = half_of(w[v2], true);
  }
};

// What a workgroup works on.
struct Unit {
  RowTile rt;
  int64_t unit;
  int split, h, g, rows, m0, len;
  bool over, skip;
};
__device__ __forceinline__ Unit unit_of(const Kv4Args &a, int64_t slots, int nsplit, int tm, int dim) {
  Unit u;
  const int64_t units = slots * a.hkv;
  u.split = (int)(blockIdx.x / units);
  u.unit = blockIdx.x - u.split * units;
  const int64_t slot = u.unit / a.hkv;
  u.h = (int)(u.unit - slot * a.hkv);     // heads are neighbours: a head's rows meet in one XCD's L2
  u.g = (int)(a.hq / a.hkv);
  u.rt = find_tile(a, slot, tm);
  u.skip = u.rt.none || u.rt.bad;
  if (u.rt.bad && nsplit == 1) nan_share(a, slot, slots, u.h, dim);
  if (u.skip) return u;
  u.rows = u.rt.ql * u.g, u.m0 = u.rt.tile * tm;
  const int given = a.lengths[u.rt.seq];
  u.over = given > a.per * a.page;
  u.len = u.over || given < 0 ? 0 : given;
  return u;
}

__device__ __forceinline__ Pages pages_of(const Kv4Args &a, int seq, int kend) {
  Pages p;
  p.table = a.table + seq * a.per;
  p.pages = a.pages;
  p.last = (kend - 1) >> 4;
  p.shift = 31 - __builtin_clz((unsigned)a.page >> 4);
  p.base = p.page = 0;
  return p;
}

// Few rows: every wave streams its own run of tokens for the same 16 NQ rows,
// records ahead in registers; the waves' sums meet in LDS.
template <int DIM, int GROUP, int NQ, bool XF32>
__global__ __launch_bounds__(256) void kv4_stream_kernel(const Kv4Args a, const int64_t slots, const int nsplit,
                                                         float *__restrict__ part) {
  constexpr int TM = 16 * NQ, W = DIM / 32, LDO = DIM + 4;
  __shared__ __attribute__((aligned(16))) float s_o[4][16][LDO];
  __shared__ float s_ml[4][16][2];

  const Unit u = unit_of(a, slots, nsplit, TM, DIM);
  if (u.skip) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4, g = u.g;
  const int mrows = u.rows - u.m0 < TM ? u.rows - u.m0 : TM;
  const float c = a.scale * 1.44269504088896340736f;
  Rows<DIM, GROUP, NQ, XF32> rows;
  rows.start(a, u.rt, u.h, g, u.len, u.m0, u.rows, c);

  const int kend = limit_of(a, u.len, u.rt.ql, (u.m0 + mrows - 1) / g);   // of the last row, the longest
  const int kall = limit_of(a, u.len, u.rt.ql, u.m0 / g);                 // every row reaches these
  const int tiles = (kend + 31) >> 5, parts = nsplit * 4, mine = u.split * 4 + wave;
  const int t0 = (int)((int64_t)tiles * mine / parts), t1 = (int)((int64_t)tiles * (mine + 1) / parts);
  if (t0 < t1) {
    Pages pg = pages_of(a, u.rt.seq, kend);
    const int pb = a.page >> 4;
    typedef RegTile<DIM, GROUP> Tile;
    Tile d0, d1;
    d0.c = d1.c = c;
    auto fetch = [&](int t, Tile &d) __attribute__((always_inline)) {
      if (2 * t - pg.base >= 64) pg.load(2 * t);
      d.load(a.cache, a.hkv, u.h, pb, pg, 2 * t);
    };
    auto step = [&](int t, Tile &d, Tile &next) __attribute__((always_inline)) {
      if (t + 1 < t1) fetch(t + 1, next);
      d.spoil();
      if (32 * t + 32 <= kall) rows.template attend<false>(d, 32 * t);
      else rows.template attend<true>(d, 32 * t);
    };
    pg.load(2 * t0);
    fetch(t0, d0);
    for (int t = t0; t < t1; t += 2) {
      step(t, d0, d1);
      if (t + 1 < t1) step(t + 1, d1, d0);
    }
  }

  rows.finish(u.over);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (n > 0) __syncthreads();
    if (lg == 0) s_ml[wave][r16][0] = rows.m[n], s_ml[wave][r16][1] = rows.ls[n];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float y[8];
      rows.channels(n, w, y);
      float4 *p = (float4 *)&s_o[wave][r16][32 * w + 8 * lg];
      p[0] = make_float4(y[0], y[1], y[2], y[3]);
      p[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * DIM; i += 256) {
      const int r = i / DIM, ch = i % DIM, m = 16 * n + r;
      if (m >= mrows) continue;
      float top = s_ml[0][r][0];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, s_ml[w][r][0]);
      const float ref = top == kNegInf ? 0.0f : top;
      float sum = 0.0f, l2 = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2_any(s_ml[w][r][0] - ref);
        l2 += f * s_ml[w][r][1];
        sum += f * s_o[w][r][ch];
      }
      if (nsplit == 1) {
        const int mm = u.m0 + m, q = mm / g;
        store_out(a, ((u.rt.q0 + q) * a.hq + (int64_t)u.h * g + (mm - q * g)) * DIM + ch, l2 == 0.0f ? 0.0f : sum / l2);
      } else {
        float *p = part + ((u.unit * nsplit + u.split) * TM + m) * (DIM + 2);
        p[ch] = sum;
        if (ch == 0) p[DIM] = top, p[DIM + 1] = l2;
      }
    }
  }
}

// TOK tokens in LDS, codes expanded once for the workgroup, as operands: 64
// lanes' 16 bytes each, so every read is 1 KB in order.
template <int DIM, int GROUP>
struct LdsTile {
  static constexpr int NG = DIM / GROUP, W = DIM / 32, TB = DIM == 256 ? 2 : 4, TOK = 16 * TB;
  uint4 k[TB * W][64];
  uint4 v[TB / 2 * (DIM / 16)][64];
  float pair[4][NG][TOK];    // keys' steps (times scale log2 e) and low ends, values' steps and low ends
};
template <int DIM, int GROUP>
struct LdsPart {             // 32 tokens of it
  const LdsTile<DIM, GROUP> &t;
  int p;
  __device__ __forceinline__ uint4 kcode(int b, int w) const {
    return t.k[(2 * p + b) * (DIM / 32) + w][threadIdx.x & 63];
  }
  __device__ __forceinline__ void vcode(int w, uint4 &even, uint4 &odd) const {
    even = t.v[p * (DIM / 16) + 2 * w][threadIdx.x & 63];
    odd = t.v[p * (DIM / 16) + 2 * w + 1][threadIdx.x & 63];
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
// the other half of LDS behind it.
template <int DIM, int GROUP, int NQ, bool XF32>
__global__ __launch_bounds__(256, 2) void kv4_tile_kernel(const Kv4Args a, const int64_t slots, const int nsplit,
                                                          float *__restrict__ part) {
  typedef LdsTile<DIM, GROUP> Lds;
  constexpr int NG = Lds::NG, W = Lds::W, TB = Lds::TB, TOK = Lds::TOK, TM = 64 * NQ, REC = 4 * DIM + 32 * NG;
  constexpr int WPW = TB * W / 4;            // words of a record's lane that a wave expands
  constexpr int SW = TB == 4 ? 32 * NG : 16 * NG, NS = (SW + 63) / 64;   // pairs a wave brings
  __shared__ __attribute__((aligned(16))) Lds s[2];

  const Unit u = unit_of(a, slots, nsplit, TM, DIM);
  if (u.skip) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4, g = u.g;
  const int last = u.m0 + TM < u.rows ? u.m0 + TM : u.rows;              // past the workgroup's last row
  const int w0 = u.m0 + 16 * NQ * wave, w1 = w0 + 16 * NQ < last ? w0 + 16 * NQ : last;
  const float c = a.scale * 1.44269504088896340736f;
  Rows<DIM, GROUP, NQ, XF32> rows;
  rows.start(a, u.rt, u.h, g, u.len, w0, u.rows, c);

  const int kend = limit_of(a, u.len, u.rt.ql, (last - 1) / g);
  const int wend = w1 > w0 ? limit_of(a, u.len, u.rt.ql, (w1 - 1) / g) : 0;   // this wave's rows reach this far,
  const int wall = w1 > w0 ? limit_of(a, u.len, u.rt.ql, w0 / g) : 0;         // all of them this far
  const int tiles = (kend + TOK - 1) / TOK;
  const int t0 = (int)((int64_t)tiles * u.split / nsplit), t1 = (int)((int64_t)tiles * (u.split + 1) / nsplit);
  if (t0 < t1) {
    Pages pg = pages_of(a, u.rt.seq, kend);
    const int pb = a.page >> 4;
    const int blk = TB == 4 ? wave : wave >> 1, off = TB == 4 ? 0 : WPW * (wave & 1);
    const int soff = TB == 4 ? 0 : 16 * NG * (wave & 1);
    uint32_t kw[WPW], vw[WPW], sw[NS];
    auto fetch = [&](int t) __attribute__((always_inline)) {
      if (TB * t - pg.base >= 64) pg.load(TB * t);
      const int b = TB * t + blk, page = pg.of(b), at = b < pg.last ? b : pg.last;
      const uint32_t *p = a.cache + (((int64_t)(page < 0 ? 0 : page) * a.hkv + u.h) * pb + (at & (pb - 1))) * REC;
      load_words(p + lane * W + off, kw);
      load_words(p + 2 * DIM + lane * W + off, vw);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int x = lane + 64 * i;
        sw[i] = x < SW ? p[4 * DIM + soff + x] : 0u;
        if (page < 0) sw[i] = 0x7fc0u;
      }
    };
    auto expand = [&](Lds &d) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < WPW; ++i) {
        const int w = off + i;
        d.k[blk * W + w][lane] = q4_codes(kw[i]);
        const uint4 y = q4_codes(vw[i]);
        uint2 *e = (uint2 *)&d.v[(blk >> 1) * (DIM / 16) + 2 * w][lane];
        uint2 *o = (uint2 *)&d.v[(blk >> 1) * (DIM / 16) + 2 * w + 1][lane];
        e[blk & 1] = make_uint2(y.x, y.y);
        o[blk & 1] = make_uint2(y.z, y.w);
      }
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int x = soff + lane + 64 * i;
        if (lane + 64 * i < SW) {
          const int kv = x / (16 * NG), j = x / 16 % NG;
          d.pair[2 * kv][j][16 * blk + (x & 15)] = half_of(sw[i], false) * (kv ? 1.0f : c);
          d.pair[2 * kv + 1][j][16 * blk + (x & 15)] = half_of(sw[i], true);
        }
      }
    };
    pg.load(TB * t0);
    fetch(t0);
    expand(s[0]);
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
      const Lds &d = s[(t - t0) & 1];
      if (t + 1 < t1) fetch(t + 1);
#pragma unroll
      for (int p = 0; p < TB / 2; ++p) {
        const int first = t * TOK + 32 * p;
        const LdsPart<DIM, GROUP> src = {d, p};
        if (first + 32 <= wall) rows.template attend<false>(src, first);
        else if (first < wend) rows.template attend<true>(src, first);
      }
      if (t + 1 < t1) expand(s[(t + 1 - t0) & 1]);   // read last before the barrier of the step before
      __syncthreads();
    }
  }

  rows.finish(u.over);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int mm = w0 + 16 * n + r16;
    if (mm >= w1) continue;
    const int q = mm / g;
    const int64_t at = ((u.rt.q0 + q) * a.hq + (int64_t)u.h * g + (mm - q * g)) * DIM + 8 * lg;
    float *p = part + ((u.unit * nsplit + u.split) * TM + (mm - u.m0)) * (DIM + 2);
    const float inv = rows.ls[n] == 0.0f ? 0.0f : 1.0f / rows.ls[n];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float y[8];
      rows.channels(n, w, y);
      if (nsplit > 1) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) *(float2 *)(p + 32 * w + 8 * lg + e) = make_float2(y[e], y[e + 1]);
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
    if (nsplit > 1 && lg == 0) p[DIM] = rows.m[n], p[DIM + 1] = rows.ls[n];
  }
}

// Joins the splits of one row: thread (x, y) takes two channels of every
// PARTS-th split, then the PARTS results meet in LDS.
template <int DIM>
__global__ __launch_bounds__(256) void kv4_join_kernel(const Kv4Args a, const int64_t slots, const int nsplit,
                                                       const int tm, const float *__restrict__ part) {
  constexpr int LANES = DIM / 2, PARTS = 256 / LANES;
  __shared__ float s_m[PARTS], s_l[PARTS];
  __shared__ float2 s_o[PARTS][LANES];
  const int64_t unit = blockIdx.x / (unsigned)tm;
  const int m = (int)(blockIdx.x % (unsigned)tm);
  const int64_t slot = unit / a.hkv;
  const int h = (int)(unit - slot * a.hkv);
  const int g = (int)(a.hq / a.hkv);
  const RowTile rt = find_tile(a, slot, tm);
  if (rt.none) return;
  if (rt.bad) {
    if (m == 0) nan_share(a, slot, slots, h, DIM);
    return;
  }
  const int mm = rt.tile * tm + m;
  if (mm >= rt.ql * g) return;
  const int x = threadIdx.x % LANES, y = threadIdx.x / LANES;
  const float *p = part + (unit * nsplit * tm + m) * (DIM + 2);
  const int64_t stride = (int64_t)tm * (DIM + 2);
  float top = kNegInf, l = 0.0f;
  float2 o = make_float2(0.0f, 0.0f);
  for (int s = y; s < nsplit; s += PARTS) {
    const float *q = p + s * stride;
    const float ms = q[DIM], lq = q[DIM + 1];
    const float2 u = *(const float2 *)(q + 2 * x);
    const float m2 = fmaxf(top, ms), ref = m2 == kNegInf ? 0.0f : m2;
    const float f0 = exp2_any(top - ref), f1 = exp2_any(ms - ref);
    top = m2;
    l = l * f0 + lq * f1;
    o.x = o.x * f0 + u.x * f1;
    o.y = o.y * f0 + u.y * f1;
  }
  if (x == 0) s_m[y] = top, s_l[y] = l;
  s_o[y][x] = o;
  __syncthreads();
  if (y > 0) return;
  float all = kNegInf;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) all = fmaxf(all, s_m[i]);
  const float ref = all == kNegInf ? 0.0f : all;
  float l2 = 0.0f, u = 0.0f, w = 0.0f;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const float f = exp2_any(s_m[i] - ref);
    l2 += f * s_l[i];
    u += f * s_o[i][x].x;
    w += f * s_o[i][x].y;
  }
  const int q = mm / g;
  const int64_t at = ((rt.q0 + q) * a.hq + (int64_t)h * g + (mm - q * g)) * DIM + 2 * x;
  store_out(a, at, l2 == 0.0f ? 0.0f : u / l2);
  store_out(a, at + 1, l2 == 0.0f ? 0.0f : w / l2);
}

template <int DIM, int GROUP>
hipError_t launch_group(const Kv4Args &a, float *ws, const Kv4Plan &p, hipStream_t st) {
  const unsigned grid = (unsigned)(p.slots * a.hkv * p.nsplit);
#define RUN(KERNEL, NQ, X) KERNEL<DIM, GROUP, NQ, X><<<grid, 256, 0, st>>>(a, p.slots, p.nsplit, ws)
  if (p.tile) {
    if (!a.qbf16) RUN(kv4_tile_kernel, 1, true);
    else if constexpr (DIM == 256) RUN(kv4_tile_kernel, 1, false);
    else RUN(kv4_tile_kernel, 2, false);
  } else {
    if (!a.qbf16) RUN(kv4_stream_kernel, 1, true);
    else if (p.nq == 1) RUN(kv4_stream_kernel, 1, false);
    else if constexpr (DIM < 256) RUN(kv4_stream_kernel, 2, false);
    else return hipErrorInvalidValue;
  }
#undef RUN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nsplit == 1) return e;
  kv4_join_kernel<DIM><<<(unsigned)(p.slots * a.hkv * p.tm), 256, 0, st>>>(a, p.slots, p.nsplit, p.tm, ws);
  return hipGetLastError();
}

hipError_t launch_dim64(const Kv4Args &a, float *ws, const Kv4Plan &p, hipStream_t st);
hipError_t launch_dim128(const Kv4Args &a, float *ws, const Kv4Plan &p, hipStream_t st);
hipError_t launch_dim256(const Kv4Args &a, float *ws, const Kv4Plan &p, hipStream_t st);

}  // namespace kv4
}  // namespace slim
