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

// 2^x for x <= 0 or NaN.
__device__ __forceinline__ float exp2_neg(float x) { return __builtin_amdgcn_exp2f(x); }

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
    t.tile = (int)(slot - (int64_t)t.seq * tiles);
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
      t.seq = s, t.q0 = lo, t.ql = (int)(hi - lo), t.tile = (int)left;
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

template <int DIM, int GROUP>
struct Tile32 {              // two records as a wave holds them
  static constexpr int NG = DIM / GROUP, W = DIM / 32;
  uint32_t k[2][W], v[2][W];
  uint4 kp[2][NG], vp[2][NG];
  bool lost[2];              // its page lies outside the cache
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

template <int DIM, int GROUP, int NQ, bool XF32>
__global__ __launch_bounds__(256) void kv4_attn_kernel(const Kv4Args a, const int64_t slots, const int nsplit,
                                                       float *__restrict__ part) {
  constexpr int NG = DIM / GROUP, W = DIM / 32, GS = GROUP / 32, NT = XF32 ? 3 : 1, TM = 16 * NQ;
  constexpr int REC = 4 * DIM + 32 * NG, LDO = DIM + 4;
  __shared__ __attribute__((aligned(16))) float s_o[4][16][LDO];
  __shared__ float s_ml[4][16][2];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int split = (int)(blockIdx.x % (unsigned)nsplit);
  const int64_t unit = blockIdx.x / (unsigned)nsplit;
  const int64_t slot = unit % slots;
  const int h = (int)(unit / slots);
  const int g = (int)(a.hq / a.hkv);
  const RowTile rt = find_tile(a, slot, TM);
  if (rt.none) return;
  if (rt.bad) {
    if (nsplit == 1) nan_share(a, slot, slots, h, DIM);
    return;
  }
  const int rows = rt.ql * g, m0 = rt.tile * TM;
  const int mrows = rows - m0 < TM ? rows - m0 : TM;
  const int given = a.lengths[rt.seq];
  const bool over = given > a.per * a.page;
  const int len = over || given < 0 ? 0 : given;

  // this lane's rows: their queries as operands, their groups' sums, their limits
  uint4 qf[NQ][W][NT];
  float qs[NQ][NG];
  int lim[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int m = 16 * n + r16, mm = m0 + (m < mrows ? m : 0);
    const int i = mm / g;
    lim[n] = m < mrows ? limit_of(a, len, rt.ql, i) : 0;
    const int64_t at = ((rt.q0 + i) * a.hq + (int64_t)h * g + (mm - i * g)) * DIM + 8 * lg;
#pragma unroll
    for (int j = 0; j < NG; ++j) qs[n][j] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (XF32) {
        const float4 *p = (const float4 *)((const float *)a.q + at + 32 * j);
        float4 u = p[0], w = p[1];
        if (m >= mrows) u = w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        split3(__builtin_bit_cast(uint4, u), __builtin_bit_cast(uint4, w), qf[n][j]);
        qs[n][j / GS] += ((u.x + u.y) + (u.z + u.w)) + ((w.x + w.y) + (w.z + w.w));
      } else {
        uint4 u = *(const uint4 *)((const uint16_t *)a.q + at + 32 * j);
        if (m >= mrows) u = make_uint4(0u, 0u, 0u, 0u);
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
    }
  }

  const int kend = limit_of(a, len, rt.ql, (m0 + mrows - 1) / g);   // of the last row, the longest
  const int kall = limit_of(a, len, rt.ql, m0 / g);                 // every row reaches these
  const int tiles = (kend + 31) >> 5, parts = nsplit * 4, mine = split * 4 + wave;
  const int t0 = (int)((int64_t)tiles * mine / parts), t1 = (int)((int64_t)tiles * (mine + 1) / parts);

  f32x4_t o[NQ][DIM / 16];
  float mx[NQ], ls[NQ], pl[NQ][NG];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    mx[n] = kNegInf, ls[n] = 0.0f;
#pragma unroll
    for (int j = 0; j < NG; ++j) pl[n][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < DIM / 16; ++i) o[n][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int32_t *table = a.table + rt.seq * a.per;
  const int pb = a.page >> 4, last = (kend - 1) >> 4;
  const int shift = 31 - __builtin_clz((unsigned)pb);
  const float c = a.scale * 1.44269504088896340736f;
  int page = 0, base = 0;

  auto pages = [&](int from) __attribute__((always_inline)) {       // lane i: the page of record from + i
    base = from;
    const int b = from + lane < last ? from + lane : last;
    page = table[b >> shift];
    if (page < 0 || page >= a.pages) page = -1;
  };
  auto load = [&](int t, Tile32<DIM, GROUP> &d) __attribute__((always_inline)) {
    if (2 * t - base >= 64) pages(2 * t);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int pg = __builtin_amdgcn_readlane(page, 2 * t + b - base);
      const int blk = 2 * t + b < last ? 2 * t + b : last;
      d.lost[b] = pg < 0;
      const int64_t rec = ((int64_t)(pg < 0 ? 0 : pg) * a.hkv + h) * pb + (blk & (pb - 1));
      const uint32_t *p = a.cache + rec * REC;
      load_words(p + lane * W, d.k[b]);
      load_words(p + 2 * DIM + lane * W, d.v[b]);
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        d.kp[b][j] = *(const uint4 *)(p + 4 * DIM + 16 * j + 4 * lg);
        d.vp[b][j] = *(const uint4 *)(p + 4 * DIM + 16 * NG + 16 * j + 4 * lg);
      }
    }
  };
  auto compute = [&](int t, Tile32<DIM, GROUP> &d) __attribute__((always_inline)) {
    const bool edge = 32 * t + 32 > kall;
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (d.lost[b]) {
#pragma unroll
        for (int j = 0; j < NG; ++j) d.kp[b][j] = d.vp[b][j] = make_uint4(0x7fc0u, 0x7fc0u, 0x7fc0u, 0x7fc0u);
      }
    float s[NQ][8];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x4_t acc[NQ][NG];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int j = 0; j < NG; ++j) acc[n][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint4 k = q4_codes(d.k[b][j]);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int x = NT - 1; x >= 0; --x) acc[n][j / GS] = mfma16(k, qf[n][j][x], acc[n][j / GS]);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][4 * b + v] = 0.0f;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const uint32_t w = v == 0 ? d.kp[b][j].x : v == 1 ? d.kp[b][j].y : v == 2 ? d.kp[b][j].z : d.kp[b][j].w;
          const float step = __uint_as_float(w << 16), low = __uint_as_float(w & 0xffff0000u);
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            s[n][4 * b + v] = __builtin_fmaf(low, qs[n][j], s[n][4 * b + v]);
            s[n][4 * b + v] = __builtin_fmaf(step, acc[n][j][v], s[n][4 * b + v]);
          }
        }
      }
    }
    const int tok = 32 * t + 4 * lg;                   // of entry 0; entry 4 b + v: + 16 b + v
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = kNegInf;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[n][e] *= c;
        if (edge && tok + 16 * (e >> 2) + (e & 3) >= lim[n]) s[n][e] = kNegInf;
        top = fmaxf(top, s[n][e]);
      }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      if (__any(top > mx[n])) {
        const float m = fmaxf(mx[n], top);
        const float f = exp2_neg(mx[n] - (m == kNegInf ? 0.0f : m));
        mx[n] = m;
        ls[n] *= f;
#pragma unroll
        for (int j = 0; j < NG; ++j) pl[n][j] *= f;
#pragma unroll
        for (int i = 0; i < DIM / 16; ++i) o[n][i] *= f;
      }
      const float m = mx[n] == kNegInf ? 0.0f : mx[n];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s[n][e] = exp2_neg(s[n][e] - m);
        ls[n] += s[n][e];
      }
    }
    // P step of each group as the second product's operand: 4 tokens of either record
    uint4 pf[NQ][NG][NT];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float step[8], low[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint4 &u = d.vp[e >> 2][j];
        const uint32_t w = (e & 3) == 0 ? u.x : (e & 3) == 1 ? u.y : (e & 3) == 2 ? u.z : u.w;
        step[e] = __uint_as_float(w << 16), low[e] = __uint_as_float(w & 0xffff0000u);
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = s[n][e] * step[e];
          float y = s[n][e] * low[e];
          if (edge && tok + 16 * (e >> 2) + (e & 3) >= lim[n]) x[e] = y = 0.0f;   // NaN pairs of masked tokens
          pl[n][j] += y;
        }
        if constexpr (XF32) {
          split3(make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])),
                 make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7])),
                 pf[n][j]);
        } else {
          pf[n][j][0] = make_uint4(pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7]));
        }
      }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint4 u = q4_codes(d.v[0][w]), y = q4_codes(d.v[1][w]);   // x, y: 4 tokens of the even channel; z, w: odd
      const uint4 even = make_uint4(u.x, u.y, y.x, y.y), odd = make_uint4(u.z, u.w, y.z, y.w);
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int x = NT - 1; x >= 0; --x) {
          o[n][2 * w] = mfma16(even, pf[n][w / GS][x], o[n][2 * w]);
          o[n][2 * w + 1] = mfma16(odd, pf[n][w / GS][x], o[n][2 * w + 1]);
        }
    }
  };

  if (t0 < t1) {
    pages(2 * t0);
    Tile32<DIM, GROUP> d;
    for (int t = t0; t < t1; ++t) {
      load(t, d);
      compute(t, d);
    }
  }

  // the waves' results of 16 rows at a time, joined in LDS
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float l = ls[n];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (over) l = kNaN;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      pl[n][j] += __shfl_xor(pl[n][j], 16, 64);
      pl[n][j] += __shfl_xor(pl[n][j], 32, 64);
    }
    if (n > 0) __syncthreads();
    if (lg == 0) s_ml[wave][r16][0] = mx[n], s_ml[wave][r16][1] = l;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float z = pl[n][w / GS];
      const f32x4_t e = o[n][2 * w], d = o[n][2 * w + 1];
      float4 *p = (float4 *)&s_o[wave][r16][32 * w + 8 * lg];
      p[0] = make_float4(e[0] + z, d[0] + z, e[1] + z, d[1] + z);
      p[1] = make_float4(e[2] + z, d[2] + z, e[3] + z, d[3] + z);
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
        const float f = exp2_neg(s_ml[w][r][0] - ref);
        l2 += f * s_ml[w][r][1];
        sum += f * s_o[w][r][ch];
      }
      if (nsplit == 1) {
        const int mm = m0 + m, q = mm / g;
        store_out(a, ((rt.q0 + q) * a.hq + (int64_t)h * g + (mm - q * g)) * DIM + ch, l2 == 0.0f ? 0.0f : sum / l2);
      } else {
        float *p = part + ((unit * nsplit + split) * TM + m) * (DIM + 2);
        p[ch] = sum;
        if (ch == 0) p[DIM] = top, p[DIM + 1] = l2;
      }
    }
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
  const int64_t slot = unit % slots;
  const int h = (int)(unit / slots);
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
    const float f0 = exp2_neg(top - ref), f1 = exp2_neg(ms - ref);
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
    const float f = exp2_neg(s_m[i] - ref);
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
#define RUN(NQ, X) kv4_attn_kernel<DIM, GROUP, NQ, X><<<grid, 256, 0, st>>>(a, p.slots, p.nsplit, ws)
  if (a.qbf16) {
    if (p.nq == 1) RUN(1, false);
    else if (p.nq == 2) RUN(2, false);
    else if constexpr (DIM < 256) RUN(4, false);
    else return hipErrorInvalidValue;
  } else {
    if (p.nq == 1) RUN(1, true);
    else if constexpr (DIM == 64) RUN(2, true);
    else return hipErrorInvalidValue;
  }
#undef RUN
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.nsplit == 1) return e;
  kv4_join_kernel<DIM><<<(unsigned)(p.slots * a.hkv * 16 * p.nq), 256, 0, st>>>(a, p.slots, p.nsplit, 16 * p.nq, ws);
  return hipGetLastError();
}

hipError_t launch_dim64(const Kv4Args &a, float *ws, const Kv4Plan &p, hipStream_t st);
hipError_t launch_dim128(const Kv4Args &a, float *ws, const Kv4Plan &p, hipStream_t st);
hipError_t launch_dim256(const Kv4Args &a, float *ws, const Kv4Plan &p, hipStream_t st);

}  // namespace kv4
}  // namespace slim
