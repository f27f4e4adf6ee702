// Linear layers from 4-bit codes with group scales, one matrix or one per
// expert, on the matrix cores of gfx950.
//
//   Y[a, i] = sum_j s[i, j] (P[a, i, j] - z[i, j] Xs[a, j]),
//   P[a, i, j] = sum_{c in group j} X[a, c] q[i, c],   Xs[a, j] = sum_{c in group j} X[a, c].
//
// A code below 16 is exact in bfloat16, X enters as stored (float32 X as three
// bfloat16 terms whose sum is exact from 2^-110 on), and P and Xs come from the
// bfloat16 MFMA with float32 sums, so nothing is rounded before the float32 group
// sums; Y is rounded once at the end.  Folding s into a bfloat16 weight would save the
// per-group scaling but round every weight to 8 bits.
//
// Layout (pack4_kernel).  A record holds 16 rows x 128 columns: word 4 l + i
// (lane l = 16 lg + r, i < 4) has the codes of row r, columns 32 i + 8 lg ..
// +7; byte b of it is the code of column b in its low and of column b + 4 in
// its high nibble.  After the 256 code words come (scale, zero) pairs, 16 rows
// per group.  Records of one row block follow each other along the columns, so
// a wave reads one record as 64 consecutive 16-byte loads and its pairs with
// one 8-byte load per group: a pure stream.  Rows past n and columns past m
// are stored as zeros.
#include <type_traits>

#include "common.hpp"
#include "mma16.hpp"
#include "serve.hpp"

namespace slim {

namespace {

// ---------------------------------------------------------------- packing
// A wave per record: lane l packs the 32 codes of its 16 bytes, the first
// 16 (128 / g) lanes copy a (scale, zero) pair each.  Run once per layer; bound
// by reading the codes (28672 x 8192: 92 us, 4.0 TB/s in and out).
__global__ __launch_bounds__(256) void pack4_kernel(const uint8_t *__restrict__ codes, const float *__restrict__ scale,
                                                    const float *__restrict__ zero, int64_t n, int64_t m, int g,
                                                    int64_t nrb, int64_t nch, int64_t nrec,
                                                    uint32_t *__restrict__ packed, int32_t *__restrict__ info) {
  const int lane = threadIdx.x & 63, r = lane & 15, lg = lane >> 4;
  const int gpc = 128 / g;
  const int64_t k = m / g;
  for (int64_t rec = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); rec < nrec; rec += (int64_t)gridDim.x * 4) {
    const int64_t ch = rec % nch, rb = rec / nch % nrb, ex = rec / (nch * nrb);
    uint32_t *out = packed + rec * (256 + 32 * gpc);
    const int64_t row = rb * 16 + r;
    uint32_t w[4], high = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = ch * 128 + 32 * i + 8 * lg;
      uint2 v = make_uint2(0u, 0u);
      if (row < n && c < m) v = *(const uint2 *)(codes + (ex * n + row) * m + c);
      high |= (v.x | v.y) & 0xf0f0f0f0u;
      w[i] = (v.x & 0x0f0f0f0fu) | ((v.y & 0x0f0f0f0fu) << 4);
    }
    *(uint4 *)(out + 4 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    if (high && info) *info = 1;
    if (lg < gpc) {
      const int64_t j = ch * gpc + lg;
      float s = 0.0f, z = 0.0f;
      if (row < n && j < k) {
        s = scale[(ex * n + row) * k + j];
        z = zero[(ex * n + row) * k + j];
      }
      *(float2 *)(out + 256 + 2 * (16 * lg + r)) = make_float2(s, z);
    }
  }
}

// ---------------------------------------------------------------- row tiles
// The experts' row ranges cut into tiles of TOK rows, in order.  Every wave
// works this out for itself from the bounds (lane l takes consecutive
// experts), so no table, extra launch or host copy of the bounds is needed.
// Bounds out of order make every tile bad; tiles then cut the plain row range.
struct RowTile {
  int expert;
  int row0;        // first row of Y (rows are below 2^20)
  int cnt;         // rows in the tile
};

template <int TOK>
struct Tiles {
  int total;       // tiles of this call
  bool bad;        // offsets are not nondecreasing inside [0, r]
  int mine, incl;
  int lo0, hi0;    // bounds of this lane's first expert

  __device__ __forceinline__ void scan(const Q4Args &a) {
    const int r = (int)a.r;
    bad = false;
    mine = incl = lo0 = hi0 = 0;
    total = (r + TOK - 1) / TOK;
    if (!a.offsets) return;
    const int lane = threadIdx.x & 63;
    const int per = (a.e + 63) >> 6;
    bool wrong = false;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < a.e) {
        const int lo = a.offsets[e], hi = a.offsets[e + 1];
        if (i == 0) lo0 = lo, hi0 = hi;
        if (lo < 0 || hi < lo || hi > r) wrong = true;
        else mine += (int)((uint32_t)(hi - lo + TOK - 1) / TOK);
      }
    }
    bad = __builtin_amdgcn_ballot_w64(wrong) != 0;   // uniform, unlike __any, for the compiler too
    if (bad) return;
    incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    total = __builtin_amdgcn_readlane(incl, 63);
  }

  // Tile idx < total.
  __device__ __forceinline__ RowTile locate(const Q4Args &a, int idx) const {
    RowTile t;
    t.expert = 0;
    t.row0 = idx * TOK;
    int end = (int)a.r;
    if (a.offsets && !bad) {
      const int per = (a.e + 63) >> 6;
      int ex = -1;
      int row0 = 0, hi1 = 0;
      int left = idx - (incl - mine);
      if (left >= 0 && left < mine) {
        for (int i = 0; i < per; ++i) {
          const int e = (threadIdx.x & 63) * per + i;
          if (e >= a.e) break;
          const int lo = i ? a.offsets[e] : lo0, hi = i ? a.offsets[e + 1] : hi0;
          const int tl = (int)((uint32_t)(hi - lo + TOK - 1) / TOK);
          if (left < tl) {
            ex = e;
            row0 = lo + left * TOK;
            hi1 = hi;
            break;
          }
          left -= tl;
        }
      }
      const int src = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(ex >= 0)) - 1;
      t.expert = __builtin_amdgcn_readlane(ex, src);
      t.row0 = __builtin_amdgcn_readlane(row0, src);
      end = __builtin_amdgcn_readlane(hi1, src);
    }
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.cnt = __builtin_amdgcn_readfirstlane(end - t.row0 < TOK ? end - t.row0 : TOK);
    return t;
  }
};

__device__ __forceinline__ void store_y(const Q4Args &a, int64_t row, int64_t i, float v) {
  if (a.ybf16) ((uint16_t *)a.Y)[row * a.n + i] = (uint16_t)f32_to_bf16_bits(v);
  else ((float *)a.Y)[row * a.n + i] = v;
}

// What row `row` of Y is multiplied by: NaN where its row of X is out of range, or
// the bounds are.
__device__ __forceinline__ float row_factor(const Q4Args &a, bool bad, int64_t row) {
  float f = a.row_scale ? a.row_scale[row] : 1.0f;
  bool ok = !bad;
  if (a.rows) {
    const int32_t xr = a.rows[row];
    ok = ok && xr >= 0 && xr < a.xrows;
  }
  return ok ? f : __uint_as_float(0x7fc00000u);
}

// A record's scale and zero pairs of row l % 16, for lanes that loaded group
// (l / 16) % GPC's: one load and a few lane swaps in place of a load per group.
// A value swapped with itself leaves both rows' (halves') values in every lane.
template <int GPC>
__device__ __forceinline__ void spread(float2 v, float2 (&o)[GPC]) {
  if constexpr (GPC == 1) {
    o[0] = v;
  } else {
    float2 half[GPC / 2];
    if constexpr (GPC == 2) {
      half[0] = v;
    } else {
      const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v.x), __float_as_uint(v.x), false, false);
      const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(v.y), __float_as_uint(v.y), false, false);
#pragma unroll
      for (int h = 0; h < 2; ++h) half[h] = make_float2(__uint_as_float(x[h]), __uint_as_float(y[h]));
    }
#pragma unroll
    for (int h = 0; h < GPC / 2; ++h) {
      const uint32_t s = __float_as_uint(half[h].x), z = __float_as_uint(half[h].y);
      const auto x = __builtin_amdgcn_permlane16_swap(s, s, false, false);
      const auto y = __builtin_amdgcn_permlane16_swap(z, z, false, false);
#pragma unroll
      for (int q = 0; q < 2; ++q) o[2 * h + q] = make_float2(__uint_as_float(x[q]), __uint_as_float(y[q]));
    }
  }
}

// ---------------------------------------------------------------- streaming kernel
// A workgroup owns 16 R output rows of one matrix and a tile of 16 TT rows of
// Y; its NW waves take the 128-column records in turn (wave w: w, w + NW, ...;
// U of them at a time, whose loads are all in flight together, or AHEAD: the next
// one's while this one is multiplied) and their sums
// are joined through LDS in wave order, so the result does not depend on timing.
// Bound by the stream of records: one token through 28672 x 8192 takes 26.2 us
// where other weights pass between calls (132 MB, 5.1 TB/s; 22.6 us with the same
// ones, from the last-level cache), 16 tokens through 13824 x 5120, g = 64, 11.5 us
// (45 MB, 3.9 TB/s: 216 workgroups leave 40 CUs idle), 1024 rows over 64 experts of
// 1024 x 2048, g = 64, 28.4 us (84 MB once; an expert with more than 16 rows is read
// again for each 16).  Splitting the columns over the waves of a workgroup rather than over
// workgroups keeps it one launch without partial sums in memory.
// MFMA operands (v_mfma_f32_16x16x32_bf16): A = X (row l % 16, columns
// 8 (l / 16) .. +7), B = codes (column l % 16 = output row), D element j =
// (row 4 (l / 16) + j, output row l % 16): one lane keeps one output row, so a
// group's scale and zero are one pair per lane.  Row a of A is token
// 4 (a % 4) + a / 4 of its 16, which puts the first four tokens in element 0.
template <bool XBF16, int G, int R, int TT, int NW, int U, bool AHEAD>
__global__ __launch_bounds__(64 * NW) void q4_stream_kernel(Q4Args a, int nrb, int nch) {
  constexpr int GPC = 128 / G, SPG = G / 32;     // groups per record, K slices per group
  constexpr int RECW = 256 + 32 * GPC;
  constexpr int NT = XBF16 ? 1 : 3;              // bfloat16 terms of X
  constexpr int XL = XBF16 ? 1 : 2;              // 16-byte loads for 8 columns of X
  constexpr int TOK = 16 * TT;
  __shared__ float part[NW][R * TT * 256];
  __shared__ float factor[TOK];
  const int lane = threadIdx.x & 63, r16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  Tiles<TOK> tiles;
  tiles.scan(a);
  const int tile = (int)(blockIdx.z * gridDim.y + blockIdx.y);
  if (tile >= tiles.total) return;
  const RowTile tl = tiles.locate(a, tile);
  const int rb0 = blockIdx.x * R;

  const char *xp[TT];
#pragma unroll
  for (int u = 0; u < TT; ++u) {
    const int tok = 16 * u + 4 * (r16 & 3) + (r16 >> 2);
    int64_t row = tl.row0 + (tok < tl.cnt ? tok : 0);    // rows past the tile repeat its first
    if (a.rows) {
      row = a.rows[row];
      if (row < 0 || row >= a.xrows) row = 0;
    }
    xp[u] = (const char *)a.X + (row * a.m + 8 * lg) * (XBF16 ? 2 : 4);
  }
  if ((int)threadIdx.x < tl.cnt) factor[threadIdx.x] = row_factor(a, tiles.bad, tl.row0 + threadIdx.x);
  const uint32_t *wp[R];                         // row blocks past the last repeat it
#pragma unroll
  for (int b = 0; b < R; ++b)
    wp[b] = a.W + ((int64_t)tl.expert * nrb + (rb0 + b < nrb ? rb0 + b : nrb - 1)) * nch * RECW;

  f32x4_t tot[R][TT];
#pragma unroll
  for (int b = 0; b < R; ++b)
#pragma unroll
    for (int u = 0; u < TT; ++u) tot[b][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);

  // N records of the wave.
  struct Regs {
    uint4 w[U][R];
    float2 pair[U][R];
    uint4 x[U][TT][4][XL];
  };
  auto fetch = [&](int ch0, auto count, Regs &rg) __attribute__((always_inline)) {
    constexpr int N = decltype(count)::value;
    auto &w = rg.w;
    auto &pair = rg.pair;
    auto &x = rg.x;
#pragma unroll
    for (int v = 0; v < N; ++v) {
      const int ch = ch0 + v * NW;
#pragma unroll
      for (int b = 0; b < R; ++b) {
        const uint32_t *rec = wp[b] + (int64_t)ch * RECW;
        w[v][b] = *(const uint4 *)(rec + 4 * lane);
        pair[v][b] = *(const float2 *)(rec + 256 + 2 * (16 * (lg & (GPC - 1)) + r16));
      }
#pragma unroll
      for (int u = 0; u < TT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)              // a record past m holds zeros there: any finite X will do
#pragma unroll
          for (int e = 0; e < XL; ++e)
            x[v][u][i][e] = *(const uint4 *)(xp[u] + (ch * 128 + 32 * i < a.m ? (ch * 128 + 32 * i) * (2 * XL) : 0) + 16 * e);
    }
  };
  auto compute = [&](int ch0, auto count, const Regs &rg) __attribute__((always_inline)) {
    constexpr int N = decltype(count)::value;
    auto &w = rg.w;
    auto &pair = rg.pair;
    auto &x = rg.x;
#pragma unroll
    for (int v = 0; v < N; ++v) {
      const int ch = ch0 + v * NW;
      float2 sz[R][GPC];
#pragma unroll
      for (int b = 0; b < R; ++b) spread<GPC>(pair[v][b], sz[b]);
#pragma unroll
      for (int q = 0; q < GPC; ++q) {
        if (ch * 128 + q * G >= a.m) break;
        f32x4_t acc[R][TT], sx[TT];
#pragma unroll
        for (int u = 0; u < TT; ++u) {
          sx[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < R; ++b) acc[b][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int s = 0; s < SPG; ++s) {
          const int i = q * SPG + s;
          uint4 c[R];
#pragma unroll
          for (int b = 0; b < R; ++b)
            c[b] = q4_codes(i == 0 ? w[v][b].x : i == 1 ? w[v][b].y : i == 2 ? w[v][b].z : w[v][b].w);
#pragma unroll
          for (int u = 0; u < TT; ++u) {
            uint4 xt[NT];
            if constexpr (XBF16) xt[0] = x[v][u][i][0];
            else split3(x[v][u][i][0], x[v][u][i][1], xt);
#pragma unroll
            for (int e = 0; e < NT; ++e) {
              sx[u] = mfma16(xt[e], ones, sx[u]);
#pragma unroll
              for (int b = 0; b < R; ++b) acc[b][u] = mfma16(xt[e], c[b], acc[b][u]);
            }
          }
        }
        auto add = [&](int j) __attribute__((always_inline)) {
#pragma unroll
          for (int b = 0; b < R; ++b)
#pragma unroll
            for (int u = 0; u < TT; ++u)
              tot[b][u][j] = fmaf(sz[b][q].x, fmaf(-sz[b][q].y, sx[u][j], acc[b][u][j]), tot[b][u][j]);
        };
        // up to four tokens have no more than element 0 (t = 1, 28672 x 8192: 28.1 against
        // 28.7 us; where two records are taken at a time the branch costs more than it saves)
        add(0);
        if (TT > 1 || U > 1 || G == 32 || tl.cnt > 4) {
          add(1);
          add(2);
          add(3);
        }
      }
    }
  };
  if (!tiles.bad) {
    int ch = wave;
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, U> all;
    Regs p, q;
    if constexpr (AHEAD) {
      if (ch < nch) {
        fetch(ch, one, p);
        for (;;) {
          bool more = ch + NW < nch;
          if (more) fetch(ch + NW, one, q);
          __builtin_amdgcn_sched_barrier(0);     // these loads before the products
          compute(ch, one, p);
          if (!more) break;
          ch += NW;
          more = ch + NW < nch;
          if (more) fetch(ch + NW, one, p);
          __builtin_amdgcn_sched_barrier(0);
          compute(ch, one, q);
          if (!more) break;
          ch += NW;
        }
      }
    } else {
      for (; ch + (U - 1) * NW < nch; ch += U * NW) {
        fetch(ch, all, p);
        compute(ch, all, p);
      }
      if constexpr (U > 1)
        for (; ch < nch; ch += NW) {
          fetch(ch, one, p);
          compute(ch, one, p);
        }
    }
  }
  // part[wave][(u * 4 + j) * 4 + lg][b][r16]: token 16 u + 4 j + lg, output row 16 b + r16
#pragma unroll
  for (int u = 0; u < TT; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (16 * u + 4 * j >= tl.cnt) break;       // no such token in the tile
#pragma unroll
      for (int b = 0; b < R; ++b) part[wave][((16 * u + 4 * j + lg) * R + b) * 16 + r16] = tot[b][u][j];
    }
  __syncthreads();
  for (int idx = threadIdx.x; idx < tl.cnt * R * 16; idx += 64 * NW) {
    const int tok = idx / (16 * R), col = idx % (16 * R);
    const int64_t i = (int64_t)rb0 * 16 + col;
    if (i >= a.n) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += part[w][idx];
    store_y(a, tl.row0 + tok, i, v * factor[tok]);
  }
}

// ---------------------------------------------------------------- tile kernel
// Large row tiles.  The zero term -z Xs is formed by the matrix cores too: Xs
// (float32, from q4_sums_kernel) and z are split into three bfloat16 terms
// each and eight of their nine products are summed as one more K slice of the
// group,
//   A: sh sm sh sm sh sl sm sl    B: -zh -zh -zm -zm -zl -zh -zl -zm
// (the missing zl sl is below 2^-32 of the product), so a group costs one
// vector operation per output, the scaling.
__device__ __forceinline__ void split_sum(float v, uint32_t &h, uint32_t &m, uint32_t &l) {
  h = __float_as_uint(v) & 0xffff0000u;
  const float r1 = v - __uint_as_float(h);
  m = __float_as_uint(r1) & 0xffff0000u;
  l = __float_as_uint(r1 - __uint_as_float(m));
}
__device__ __forceinline__ uint32_t pack_hi(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// 2048 x 11008 bfloat16: 12.3 us, 3.7 TB/s.
// Group sums of X, sums[row][kp] (kp: groups in whole records), and float32 X
// as three bfloat16 planes side by side, planes[row][3][nch * 128], both zero
// past m; of bfloat16 X a copy if planes is given.  With `rows` row i is X's
// row rows[i].  A thread takes 8 columns; a
// group's G / 8 threads are neighbours.
template <bool XBF16, int G>
__global__ __launch_bounds__(256) void q4_sums_kernel(const void *__restrict__ Xv, const int32_t *__restrict__ rows,
                                                      int64_t xrows, int64_t nrow, int64_t m, int nch,
                                                      float *__restrict__ sums, uint4 *__restrict__ planes) {
  const int64_t m8 = m / 8, p8 = (int64_t)nch * 16, all = nrow * p8;
  for (int64_t base = (int64_t)blockIdx.x * 256; base < all; base += (int64_t)gridDim.x * 256) {
    const int64_t id = base + threadIdx.x;
    const int64_t i = id / p8, c = id - i * p8;
    const bool has = id < all && c < m8;
    float sum = 0.0f;
    if (has) {
      int64_t row = i;
      if (rows) {
        row = rows[i];
        if (row < 0 || row >= xrows) row = 0;
      }
      const int64_t at = row * m8 + c;
      float v[8];
      if constexpr (XBF16) {
        const uint4 x = ((const uint4 *)Xv)[at];
        if (planes) planes[i * p8 + c] = x;
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __uint_as_float(u[e] << 16);
          v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        }
      } else {
        const uint4 x = ((const uint4 *)Xv)[2 * at], y = ((const uint4 *)Xv)[2 * at + 1];
        const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
        uint4 t[3];
        split3(x, y, t);
#pragma unroll
        for (int p = 0; p < 3; ++p) planes[(i * 3 + p) * p8 + c] = t[p];
      }
      sum = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    } else if (planes && id < all) {
#pragma unroll
      for (int p = 0; p < (XBF16 ? 1 : 3); ++p) planes[(i * (XBF16 ? 1 : 3) + p) * p8 + c] = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int d = 1; d < G / 8; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (id < all && (threadIdx.x & (G / 8 - 1)) == 0) sums[i * (nch * (128 / G)) + c / (G / 8)] = sum;
  }
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void q4_lds_t;
typedef const __attribute__((address_space(1))) void q4_global_t;

// BYTES (4 or 16) per lane from base + voff + soff straight to LDS, 64 lanes in
// a row from `to`.
template <int BYTES>
__device__ __forceinline__ void load_lds(const void *base, uint32_t limit, void *to, uint32_t voff, int soff) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, (int)limit, 0x00020000);
  if constexpr (BYTES == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (q4_lds_t *)to, 16, (int)voff, soff, 0, 0);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (q4_lds_t *)to, 4, (int)voff, soff, 0, 0);
}

// Stores that drop what lies past `limit` bytes from `base`.
__device__ __forceinline__ void store_pair(void *base, uint32_t limit, bool half, uint32_t at0, uint32_t at1, float y0,
                                           float y1) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(base, (short)0, (int)limit, 0x00020000);
  if (half) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const uint32_t p = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)y0, (__bf16)y1});
    __builtin_amdgcn_raw_buffer_store_b16((short)p, r, (int)at0, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b16((short)(p >> 16), r, (int)at1, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(y0), r, (int)at0, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(y1), r, (int)at1, 0, 0);
  }
}

// Waits until at most VM of this wave's loads are in flight (loads complete in
// order, so what was issued before the last VM is in LDS) and its LDS reads
// have returned.  The builtin, not inline text: the compiler then knows which
// LDS loads have landed and adds no full wait before the next stage is read.
template <int VM>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | (VM >> 4) << 14);
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void meet() { asm volatile("s_barrier" ::: "memory"); }

// 128 rows of Y x 256 output rows per workgroup (WT = 2, WN = 4) or 64 x 512 (1, 8),
// a 64 x 64 piece of it per wave (2 x 2 blocks of 32 x 32).  Every operand goes straight to LDS, 128 columns
// (a record per 16 output rows) to a stage, two stages ahead of the products:
// X's rows with their 16-byte slots XOR-swizzled by row (16 rows of a column
// slice then lie in different banks), the records, and the group sums.
//
// The two waves of a SIMD take turns.  Half a stage is a load phase (the last
// group's scaling, LDS reads, expansion of the codes: vector unit) and a
// product phase (16 MFMAs and the zero term: matrix unit) with a barrier after
// each, and waves 4 .. 7 run one phase behind waves 0 .. 3, so that at any
// time one wave of each pair keeps the matrix unit busy while the other
// prepares.  In slots of one phase, a leading wave works on stage c in slots
// 4 c (load), 4 c + 1 (products), 4 c + 2, 4 c + 3, a trailing one a slot
// later.  Stage c + 2 is loaded from slot 4 c (4 c + 1) on into the buffer of
// stage c - 1, last read in slot 4 c - 1 (4 c for its own); every wave waits for
// its own loads of stage c + 1 at the end of its first product phase (4 c + 1,
// 4 c + 2), and stage c + 1 is first read in slot 4 c + 3: X is read into
// registers during the product phase before its own.
//
// 2048 rows through 4096 x 11008, g = 128: 171 us, 1.08 PFLOP/s of the product
// (1.21 with the zero term), the matrix unit busy 65% of the cycles at 1.8 GHz;
// a plain bfloat16 library product of that shape takes 151 us.  A phase takes
// 700 to 850 cycles where its products need 512 (640 with the zero term): the
// load phases (the scaling's 256 cycles, LDS latency) are as long as the
// products.  Without the phases, both waves of a SIMD alike, it was 218 us; one
// load and one product phase a stage (g = 128) measured the same 178 us.
// A workgroup's start and end run beside no product, so they are kept short: tile
// arithmetic in 32 bits, the rows' factors fetched at the start, stores whose bounds
// the buffer descriptor checks (8 experts of 11008 x 4096 over 4096 rows: 472 -> 418 us
// when that was done; 390 to 412 by card, group sums included).
template <int G, int WT, int WN>
__global__ __launch_bounds__(64 * WT * WN, 2) void q4_tile_kernel(Q4Args a, const uint16_t *__restrict__ X,
                                                                  int64_t ldx, int nt, bool gather, bool compact,
                                                                  const float *__restrict__ sums, int nrb, int nch,
                                                                  int nnb, float *__restrict__ partial) {
  constexpr int NW = WT * WN, TOK = 64 * WT;
  static_assert(WT * WN == 8 && WN >= 4, "the phases pair waves w and w + 4");
  constexpr int GPC = 128 / G;                   // groups per record
  constexpr int RECW = 256 + 32 * GPC;
  constexpr int XL = 16 / WN;                    // loads per wave and stage: X (1 KB each),
  constexpr int RL = 4 / WT;                     //   codes of a record,
  constexpr int ZP = WN / 4, ZL = ZP * GPC;      //   scales and zeros,
  constexpr int SL = (WT * GPC + NW - 1) / NW;   //   group sums of 64 rows
  constexpr int LOADS = XL + RL + ZL + SL;
  constexpr int RST = (G == 32 || (G == 64 && WN == 8)) ? 2 : 3;   // stages of records, as many as fit
  struct Stage {
    unsigned char x[TOK * 256];
    float s[GPC * TOK];
  };
  struct Recs {
    // codes, then scales and zeros
    unsigned char b[4 * WN * (1024 + 128 * GPC)];
  };
  constexpr int ZAT = 4 * WN * 1024;
  __shared__ __align__(16) Stage st0, st1, st2;
  __shared__ __align__(16) Recs rc0, rc1;
  __shared__ float factor[TOK];
  __shared__ __align__(16) typename std::conditional<RST == 3, Recs, uint4>::type rc2;
  const int lane = threadIdx.x & 63, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wt = wave / WN, wn = wave % WN;

  // Consecutive workgroups go to different XCDs: each XCD takes a contiguous
  // eighth of the tiles, walked four row tiles at a time over the output
  // blocks, so the workgroups sharing an L2 share X tiles and codes.
  Tiles<TOK> tiles;
  tiles.scan(a);
  const uint32_t all = (uint32_t)tiles.total * nnb, per = (all + 7) / 8;   // below 2^27
  const uint32_t idx = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (blockIdx.x >> 3 >= per || idx >= all) return;
  const uint32_t strip = idx / (4 * nnb), in = idx - strip * 4 * nnb;
  const uint32_t wide = tiles.total - 4 * strip < 4 ? tiles.total - 4 * strip : 4;
  const int nb = (int)(in / wide);
  const RowTile tl = tiles.locate(a, (int)(4 * strip + in % wide));

  // Operands come by buffer loads: one descriptor each with its base at this
  // tile, a 32-bit offset per lane that stays, and the stage as scalar offset.
  auto x_row = [&](int tok) __attribute__((always_inline)) {   // row of X, from the tile's base
    const int64_t row = tok < tl.cnt ? tok : 0;
    if (!gather) return row;
    const int64_t g = a.rows[tl.row0 + row];
    return g < 0 || g >= a.xrows ? 0 : g;
  };
  // Stages of this workgroup (blockIdx.y takes a run of them, and its sums go to
  // `partial`, where the columns are split); float32 X passes its three planes in turn.
  const int c0 = nt * nch * (int)blockIdx.y / (int)gridDim.y;
  const int n = nt * nch * ((int)blockIdx.y + 1) / (int)gridDim.y;
  const uint16_t *xbase = X + (gather ? 0 : (int64_t)tl.row0 * ldx);
  const float *sbase = sums + (gather && !compact ? 0 : (int64_t)tl.row0 * (nch * GPC));
  const uint32_t xbytes = (uint32_t)((gather ? a.xrows : tl.cnt) * ldx * 2);
  const uint32_t sbytes = (uint32_t)((gather && !compact ? a.xrows : tl.cnt) * (nch * GPC) * 4);
  uint32_t xo[XL];                              // this lane's 16 bytes of each of its rows, stage 0
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int tok = (wave * XL + i) * 4 + (lane >> 4);
    xo[i] = (uint32_t)(x_row(tok) * ldx * 2) + ((lane & 15) ^ (tok & 15)) * 16;
  }
  uint32_t so[SL];                              // waves beyond the rows load a piece again
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int j = (wave + i * NW) % (WT * GPC), tok = (j % WT) * 64 + lane;
    so[i] = (uint32_t)((compact ? (tok < tl.cnt ? tok : 0) : x_row(tok)) * (nch * GPC) + j / WT) * 4;
  }
  // One of the loads of X's stage c, the sums with the last.
  static_assert(XL <= 4, "one load to a K step of a product phase at most");
  auto load_x = [&](int c, int part, Stage &st) __attribute__((always_inline)) {
    load_lds<16>(xbase, xbytes, st.x + (wave * XL + part) * 1024, xo[part], c * 256);
    if (part < XL - 1) return;
    const int ch = c < nch ? c : 0;             // used with the first plane only
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int j = (wave + i * NW) % (WT * GPC);
      load_lds<4>(sbase, sbytes, st.s + (j / WT) * TOK + (j % WT) * 64, so[i], ch * GPC * 4);
    }
  };
  // Records, as byte offsets from the tile's first; row blocks past the last
  // repeat it.  A wave loads the codes of records RL wave .. and the scales and
  // zeros of the pairs p = wave (and wave + 8): records j and j + 2, j = 4 (p / 2)
  // + p % 2, which one lane reads together.
  const int rb0 = nb * WN * 4;
  auto rec = [&](int j) __attribute__((always_inline)) {
    return (rb0 + j < nrb ? j : nrb - 1 - rb0) * nch * (RECW * 4);
  };
  const uint32_t *wbase = a.W + ((int64_t)tl.expert * nrb + rb0) * nch * RECW;
  const uint32_t limit = (uint32_t)(rec(WN * 4 - 1) + nch * (RECW * 4));
  // scale and zero words in LDS: [pair][group][row][record][2]
  uint32_t zo[ZP];
#pragma unroll
  for (int i = 0; i < ZP; ++i) {
    const int p = wave + 8 * i;
    zo[i] = (uint32_t)(rec(p / 2 * 4 + p % 2 + (lane & 2)) + 1024 + (lane >> 2) * 8 + (lane & 1) * 4);
  }
  auto load_rec = [&](int c, Recs &rc) __attribute__((always_inline)) {
    const int at = (nt > 1 ? c % nch : c) * (RECW * 4);
#pragma unroll
    for (int i = 0; i < RL; ++i)
      load_lds<16>(wbase, limit, rc.b + (wave * RL + i) * 1024, lane * 16, at + rec(wave * RL + i));
#pragma unroll
    for (int i = 0; i < ZP; ++i)
#pragma unroll
      for (int q = 0; q < GPC; ++q)
        load_lds<4>(wbase, limit, rc.b + ZAT + ((wave + 8 * i) * GPC + q) * 256, zo[i], at + q * 128);
  };

  // of this wave's 64 rows, for the end (the waves with the same rows write the same)
  factor[wt * 64 + lane] =
      partial ? 1.0f : row_factor(a, tiles.bad, tl.row0 + (wt * 64 + lane < tl.cnt ? wt * 64 + lane : 0));

  f32x16_t tot[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) tot[i][b][v] = 0.0f;

  const int xrow0 = (wt * 64 + (lane & 31)) * 256 + ((hi ^ (lane & 15)) << 4);
  const int rec0 = wn * 4 + ((lane >> 4) & 1);   // record of this lane's output row in block 0
  constexpr int GH = G == 32 ? 2 : 1;            // groups that end in a half stage (G = 128: in the second)
  f32x16_t acc[2][2];                            // sums of the group at hand
  float sc[GH][2];                               // its scales
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int g = 0; g < GH; ++g) sc[g][b] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][b][v] = 0.0f;
  }
  auto scale_group = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) tot[i][b][v] = fmaf(sc[g][b], acc[i][b][v], tot[i][b][v]);
    // here, and not later, when the next group's sums need the registers
#pragma unroll
    for (int i = 0; i < 2; ++i) asm volatile("" : "+v"(tot[i][0]), "+v"(tot[i][1]));
  };

  u32x4_t x[4][2];                               // X of half a stage, [K step][block]
  uint2 cw[2][2];                                // its codes, [16 columns of 32][block]
  u32x4_t w[2][2];                               // and those of one K step, expanded
  uint4 aa[GH][2], ba[GH][2];                    // and of its zero terms
  auto expand = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
      w[u & 1][b] = __builtin_bit_cast(u32x4_t, q4_codes(u < 2 ? cw[u & 1][b].x : cw[u & 1][b].y));
  };
  float su[GH][2];                               // sums of X, scales and zeros as read
  float4 sz[GH];
  constexpr bool BOTH = G != 128;                // a group ends in either half of a stage
  // Load phase h of stage c: its reads, issued before anything else of the phase,
  auto read = [&](int h, const Stage &st, const Recs &rc) __attribute__((always_inline)) {
    // addresses formed anew: kept over the loop, those of all stages would
    // take more registers than there are
    int rrow = rec0;
    // (an offset the compiler does not know, too, for the scales: seeing that
    // they cannot be what the first load of the stage writes, it would wait for
    // every load in flight)
    int zrow = ZAT + (wn * 2 + ((lane >> 4) & 1)) * GPC * 256 + (lane & 15) * 16;
    asm volatile("" : "+v"(rrow), "+v"(zrow));
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int o = 0; o < 2; ++o)
        cw[o][b] = *(const uint2 *)(rc.b + (rrow + 2 * b) * 1024 + (16 * (hi + 2 * o) + (lane & 15)) * 16 + 8 * h);
    if (BOTH || h == 1) {
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        const int q = BOTH ? h * GH + g : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) su[g][i] = st.s[q * TOK + wt * 64 + i * 32 + (lane & 31)];
        sz[g] = *(const float4 *)(rc.b + zrow + q * 256);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto read_x = [&](int h, int u, const Stage &st) __attribute__((always_inline)) {
    int arow = xrow0;
    asm volatile("" : "+v"(arow));
#pragma unroll
    for (int i = 0; i < 2; ++i) x[u][i] = *(const u32x4_t *)(st.x + (arow ^ ((4 * h + u) << 5)) + i * 8192);
  };
  // and what is computed from them.
  auto prepare = [&](int c, int h) __attribute__((always_inline)) {
    expand(0);
    if (BOTH || h == 1) {
      // K slots 8 .. 15 (the upper lanes) and the later planes of float32 X add nothing
      const uint32_t keep = (uint32_t)(((hi | (c < nch ? 0 : 1)) - 1) >> 31);
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        uint32_t p, r, l;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          split_sum(__uint_as_float(__float_as_uint(su[g][i]) & keep), p, r, l);
          aa[g][i] = make_uint4(pack_hi(p, r), pack_hi(p, r), pack_hi(p, l), pack_hi(r, l));
        }
        sc[g][0] = sz[g].x;
        sc[g][1] = sz[g].z;
        split_sum(-sz[g].y, p, r, l);
        ba[g][0] = make_uint4(pack_hi(p, p), pack_hi(r, r), pack_hi(l, p), pack_hi(l, r));
        split_sum(-sz[g].w, p, r, l);
        ba[g][1] = make_uint4(pack_hi(p, p), pack_hi(r, r), pack_hi(l, p), pack_hi(l, r));
      }
    }
    // keeps this phase's work out of the product phase
    asm volatile("" : "+v"(w[0][0]), "+v"(w[0][1]));
  };
  // Product phase h.  X of the next half stage is read into the registers that a
  // K step has used.
  auto multiply = [&](int h, const Stage &nst, int cl, Stage &lst) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (u < 3) expand(u + 1);
      const bool first = G == 128 ? h == 0 && u == 0 : u % (G / 16) == 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          f32x16_t z;
#pragma unroll
          for (int v = 0; v < 16; ++v) z[v] = 0.0f;
          acc[i][b] = mfma_bf16(__builtin_bit_cast(uint4, x[u][i]), __builtin_bit_cast(uint4, w[u & 1][b]),
                                first ? z : acc[i][b]);
        }
      read_x(1 - h, u, nst);
      if (h == 0 && u < XL) load_x(cl, u, lst);
      if (G == 128 ? h == 1 && u == 3 : u % (G / 16) == G / 16 - 1) {
        const int g = G == 32 ? u / 2 : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b) acc[i][b] = mfma_bf16(aa[g][i], ba[g][b], acc[i][b]);
        if (G == 32 && u == 1) scale_group(0);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {               // the next step's expansion among this step's MFMAs
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (h == 0 && u < XL && j == 1) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  if (!tiles.bad) {
    constexpr int AHEAD = RST == 3 ? LOADS : XL + SL;   // loads that may still fly at the end of a stage
    // The last stages load the last one again: no stage differs from the others.
    auto stage = [&](int c, Stage &st, Stage &st1, Stage &st2, Recs &rc, Recs &rnxt) __attribute__((always_inline)) {
      read(0, st, rc);
      load_rec(c + RST - 1 < n ? c + RST - 1 : n - 1, rnxt);
      scale_group(GH - 1);
      prepare(c, 0);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      meet();
      multiply(0, st, c + 2 < n ? c + 2 : n - 1, st2);
      wait_loads<AHEAD>();
      __builtin_amdgcn_sched_barrier(0);
      meet();
      read(1, st, rc);
      if (BOTH) scale_group(GH - 1);
      prepare(c, 1);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      meet();
      multiply(1, st1, 0, st1);
      __builtin_amdgcn_sched_barrier(0);
      meet();
    };
    load_rec(c0, rc0);
#pragma unroll
    for (int u = 0; u < XL; ++u) load_x(c0, u, st0);
    if (RST == 3) load_rec(c0 + 1 < n ? c0 + 1 : c0, rc1);
#pragma unroll
    for (int u = 0; u < XL; ++u) load_x(c0 + 1 < n ? c0 + 1 : c0, u, st1);
    wait_loads<0>();
    meet();
#pragma unroll
    for (int u = 0; u < 4; ++u) read_x(0, u, st0);
    if (wave >= 4) meet();
    if constexpr (RST == 3) {
      for (int c = c0;;) {
        stage(c, st0, st1, st2, rc0, rc2);
        if (++c == n) break;
        stage(c, st1, st2, st0, rc1, rc0);
        if (++c == n) break;
        stage(c, st2, st0, st1, rc2, rc1);
        if (++c == n) break;
      }
    } else {
      for (int c = c0;;) {
        stage(c, st0, st1, st2, rc0, rc1);
        if (++c == n) break;
        stage(c, st1, st2, st0, rc1, rc0);
        if (++c == n) break;
        stage(c, st2, st0, st1, rc0, rc1);
        if (++c == n) break;
        stage(c, st0, st1, st2, rc1, rc0);
        if (++c == n) break;
        stage(c, st1, st2, st0, rc0, rc1);
        if (++c == n) break;
        stage(c, st2, st0, st1, rc1, rc0);
        if (++c == n) break;
      }
    }
    if (wave < 4) meet();
    scale_group(GH - 1);
    wait_loads<0>();                             // nothing may still write to this workgroup's LDS
  }
  // The tile's rows of Y (or of the split columns' sums): rows past it lie past the
  // limit, and so does the offset of a column past n (the rows are below 2^30 bytes).
  const bool half = !partial && a.ybf16;
  const uint32_t line = (uint32_t)a.n * (half ? 2 : 4);
  char *to = partial ? (char *)(partial + ((int64_t)blockIdx.y * a.r + tl.row0) * a.n)
                     : (char *)a.Y + tl.row0 * (int64_t)line;
  uint32_t at[2];
  int l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));   // `lane` anew: the loop needs its registers
  asm volatile("" : "+v"(l));
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t col = (int64_t)(nb * WN + wn) * 64 + b * 32 + (l & 31);
    at[b] = col < a.n ? (uint32_t)(wt * 64 + acc32_row(0, l)) * line + (uint32_t)col * (half ? 2 : 4) : 0x80000000u;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const uint32_t down = (uint32_t)(i * 32 + acc32_row(v, 0)) * line;
      const float f = factor[wt * 64 + i * 32 + acc32_row(v, l)];
      store_pair(to, tl.cnt * line, half, at[0] + down, at[1] + down, tot[i][0][v] * f, tot[i][1][v] * f);
    }
}

// Sums of a tile kernel whose columns were split, added in order, to Y.  A
// workgroup takes 1024 outputs of one row; rows outside the experts' ranges are
// left alone.
__global__ __launch_bounds__(256) void q4_join_kernel(Q4Args a, const float *__restrict__ partial, int parts) {
  Tiles<128> tiles;
  tiles.scan(a);
  const int64_t row = blockIdx.x;
  if (a.offsets && !tiles.bad && (row < a.offsets[0] || row >= a.offsets[a.e])) return;
  const float f = row_factor(a, tiles.bad, row);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t i = (int64_t)blockIdx.y * 1024 + u * 256 + threadIdx.x;
    if (i >= a.n) return;
    float v = 0.0f;
    for (int p = 0; p < parts; ++p) v += partial[(p * a.r + row) * a.n + i];
    store_y(a, row, i, v * f);
  }
}

template <bool XBF16, int G, int R, int TT, int NW, int U, bool AHEAD>
hipError_t stream_go(const Q4Args &a, hipStream_t st) {
  const int nrb = (int)q4_row_blocks(a.n), nch = (int)q4_chunks(a.m);
  const int64_t tiles = max_tiles(a.r, a.offsets ? a.e : 1, 16 * TT);
  const int64_t gz = (tiles + 65534) / 65535, gy = (tiles + gz - 1) / gz;   // grid limits of 65535
  q4_stream_kernel<XBF16, G, R, TT, NW, U, AHEAD>
      <<<dim3((nrb + R - 1) / R, (uint32_t)gy, (uint32_t)gz), 64 * NW, 0, st>>>(a, nrb, nch);
  return hipGetLastError();
}

template <int G, int WT, int WN>
hipError_t tile_go(const Q4Args &a, const TileWs &w, void *ws, hipStream_t st) {
  const int nrb = (int)q4_row_blocks(a.n), nch = (int)q4_chunks(a.m);
  const int nnb = (nrb + 4 * WN - 1) / (4 * WN);
  const int64_t all = max_tiles(a.r, a.offsets ? a.e : 1, 64 * WT) * nnb;
  const int64_t blocks = (all + 7) / 8 * 8;
  if (blocks * 64 * WT * WN > 0xffffffffll) return hipErrorInvalidConfiguration;
  float *sums = (float *)ws;
  const bool own = !a.xbf16 || w.copy;            // X is read from the workspace
  uint4 *planes = own ? (uint4 *)((char *)ws + w.planes) : nullptr;
  const int64_t sum_blocks = (w.nrow * nch * 16 + 255) / 256;
  const uint32_t sb = (uint32_t)(sum_blocks < 16384 ? sum_blocks : 16384);
  const int32_t *rows = w.compact ? a.rows : nullptr;
  if (a.xbf16) q4_sums_kernel<true, G><<<sb, 256, 0, st>>>(a.X, rows, a.xrows, w.nrow, a.m, nch, sums, planes);
  else q4_sums_kernel<false, G><<<sb, 256, 0, st>>>(a.X, rows, a.xrows, w.nrow, a.m, nch, sums, planes);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float *partial = w.parts > 1 ? (float *)((char *)ws + w.partial) : nullptr;
  q4_tile_kernel<G, WT, WN><<<dim3((uint32_t)blocks, w.parts), 64 * WT * WN, 0, st>>>(
      a, own ? (const uint16_t *)planes : (const uint16_t *)a.X,
      !own ? a.m : (a.xbf16 ? 1 : 3) * (int64_t)nch * 128, a.xbf16 ? 1 : 3, a.rows && !(own && w.compact), w.compact,
      sums, nrb, nch, nnb, partial);
  e = hipGetLastError();
  if (e != hipSuccess || !partial) return e;
  q4_join_kernel<<<dim3((uint32_t)a.r, (uint32_t)((a.n + 1023) / 1024)), 256, 0, st>>>(a, partial, w.parts);
  return hipGetLastError();
}

template <bool XBF16, int G>
hipError_t stream_pick(const Q4Args &a, hipStream_t st) {
  const StreamShape s = stream_shape(a.r, a.e, a.n, a.m, G, XBF16);
  const auto is = [&s](int blocks, int tiles, int waves, int records, bool ahead) {
    return s.blocks == blocks && s.tiles == tiles && s.waves == waves && s.records == records && s.ahead == ahead;
  };
  if constexpr (XBF16)
    if (is(4, 2, 4, 1, true)) return stream_go<XBF16, G, 4, 2, 4, 1, true>(a, st);
  if constexpr (!XBF16 && G == 128)
    if (is(4, 1, 8, 1, false)) return stream_go<XBF16, G, 4, 1, 8, 1, false>(a, st);
  if (is(4, 1, 16, 1, false)) return stream_go<XBF16, G, 4, 1, 16, 1, false>(a, st);
  if (is(4, 1, 4, 1, true)) return stream_go<XBF16, G, 4, 1, 4, 1, true>(a, st);
  if (is(2, 1, 8, 2, false)) return stream_go<XBF16, G, 2, 1, 8, 2, false>(a, st);
  if (is(1, 1, 8, 2, false)) return stream_go<XBF16, G, 1, 1, 8, 2, false>(a, st);
  return hipErrorInvalidDeviceFunction;            // a shape of the rules that is not compiled here
}

template <int G>
hipError_t pick(const Q4Args &a, void *ws, hipStream_t st) {
  if (use_tiles(a.r, a.e, a.n, a.m, a.xbf16)) {
    const TileWs w = tile_ws(a.xrows, a.r, a.e, a.n, a.m, G, a.xbf16, a.rows != nullptr);
    if (narrow_tiles(a.r, a.e, a.n)) return tile_go<G, 1, 8>(a, w, ws, st);
    return tile_go<G, 2, 4>(a, w, ws, st);
  }
  return a.xbf16 ? stream_pick<true, G>(a, st) : stream_pick<false, G>(a, st);
}

}  // namespace

hipError_t launch_pack4(const uint8_t *codes, const float *scale, const float *zero, int64_t e, int64_t n, int64_t m,
                        int group, uint32_t *packed, int32_t *info, hipStream_t st) {
  const int64_t nrb = q4_row_blocks(n), nch = q4_chunks(m), nrec = e * nrb * nch;
  const int64_t blocks = (nrec + 3) / 4 < 65536 ? (nrec + 3) / 4 : 65536;
  pack4_kernel<<<(uint32_t)blocks, 256, 0, st>>>(codes, scale, zero, n, m, group, nrb, nch, nrec, packed, info);
  return hipGetLastError();
}

size_t q4_ws_bytes(int64_t xrows, int64_t r, int64_t e, int64_t n, int64_t m, int group, bool xbf16, bool gather) {
  return r > 0 && use_tiles(r, e, n, m, xbf16) ? tile_ws(xrows, r, e, n, m, group, xbf16, gather).bytes : 0;
}

hipError_t launch_q4(const Q4Args &a, void *ws, hipStream_t st) {
  if (a.group == 128) return pick<128>(a, ws, st);
  if (a.group == 64) return pick<64>(a, ws, st);
  return pick<32>(a, ws, st);
}

}  // namespace slim
