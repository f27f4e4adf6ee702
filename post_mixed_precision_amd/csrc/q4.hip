// Linear layers from 4-bit codes with group scales, one matrix or one per
// expert, on the matrix cores of gfx950.
//
//   Y[a, i] = sum_j s[i, j] (P[a, i, j] - z[i, j] Xs[a, j]),
//   P[a, i, j] = sum_{c in group j} X[a, c] q[i, c],   Xs[a, j] = sum_{c in group j} X[a, c].
//
// A code below 16 is exact in bfloat16, X enters as stored (float32 X as three
// bfloat16 terms whose sum is exact), and P and Xs come from the bfloat16 MFMA
// with float32 sums, so nothing is rounded before the float32 group sums; Y is
// rounded once at the end.  Folding s into a bfloat16 weight would save the
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
#include "common.hpp"
#include "serve.hpp"

namespace slim {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;

__device__ __forceinline__ f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// ---------------------------------------------------------------- packing
// A wave per record: lane l packs the 32 codes of its 16 bytes, the first
// 16 (128 / g) lanes copy a (scale, zero) pair each.  Run once per layer.
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

// ---------------------------------------------------------------- operands
// The 8 codes of one word as bfloat16, in column order.  A byte below 16 read
// as an e4m3 pattern is q 2^-9 exactly, so the scaled pair conversion gives
// two bfloat16 codes at once.
__device__ __forceinline__ uint4 q4_codes(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  return r;
}

// 8 columns of a float32 row as three bfloat16 terms whose sum is exact
// (truncation leaves 16, then 8 significant bits).
__device__ __forceinline__ void split3(const float *p, uint4 (&t)[3]) {
  const float4 a = *(const float4 *)p, b = *(const float4 *)(p + 4);
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t h[8], m[8], l[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h[e] = __float_as_uint(v[e]) & 0xffff0000u;
    const float r1 = v[e] - __uint_as_float(h[e]);
    m[e] = __float_as_uint(r1) & 0xffff0000u;
    l[e] = __float_as_uint(r1 - __uint_as_float(m[e]));
  }
  auto pk = [](uint32_t lo, uint32_t hi) __attribute__((always_inline)) {
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);   // upper halves of two words
  };
  t[0] = make_uint4(pk(h[0], h[1]), pk(h[2], h[3]), pk(h[4], h[5]), pk(h[6], h[7]));
  t[1] = make_uint4(pk(m[0], m[1]), pk(m[2], m[3]), pk(m[4], m[5]), pk(m[6], m[7]));
  t[2] = make_uint4(pk(l[0], l[1]), pk(l[2], l[3]), pk(l[4], l[5]), pk(l[6], l[7]));
}

// ---------------------------------------------------------------- row tiles
struct RowTile {
  int expert;      // -1: this workgroup has no rows
  int64_t row0;    // first row of Y
  int cnt;         // rows in the tile
  bool bad;        // offsets are not nondecreasing inside [0, r]
};

// The idx-th tile of TOK rows when the experts' row ranges are cut into tiles
// in order.  Every wave works it out for itself from the bounds (lane l takes
// per consecutive experts), so no table, extra launch or host copy of the
// bounds is needed.  Bounds out of order make every tile bad; idx then counts
// tiles of the plain row range.
template <int TOK>
__device__ __forceinline__ RowTile find_tile(const Q4Args &a, int64_t idx) {
  RowTile t;
  t.bad = false;
  t.expert = -1;
  t.row0 = idx * TOK;
  t.cnt = 0;
  if (!a.offsets) {
    t.expert = 0;
  } else {
    const int lane = threadIdx.x & 63;
    const int per = (a.e + 63) >> 6;
    const int e0 = lane * per;
    int64_t mine = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
      const int e = e0 + i;
      if (e < a.e) {
        const int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
        if (lo < 0 || hi < lo || hi > a.r) bad = true;
        else mine += (hi - lo + TOK - 1) / TOK;
      }
    }
    if (__any(bad)) {
      t.bad = true;
      t.expert = 0;
    } else {
      int64_t incl = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(incl, d, 64);
        if (lane >= d) incl += o;
      }
      int ex = -1;
      int64_t row0 = 0, end = 0;
      int64_t left = idx - (incl - mine);
      if (left >= 0 && left < mine) {
        for (int i = 0; i < per; ++i) {
          const int e = e0 + i;
          if (e >= a.e) break;
          const int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
          const int64_t tl = (hi - lo + TOK - 1) / TOK;
          if (left < tl) {
            ex = e;
            row0 = lo + left * TOK;
            end = hi;
            break;
          }
          left -= tl;
        }
      }
      const uint64_t who = __ballot(ex >= 0);
      if (who) {
        const int src = __ffsll((unsigned long long)who) - 1;
        t.expert = __builtin_amdgcn_readfirstlane(__shfl(ex, src, 64));
        t.row0 = __shfl(row0, src, 64);
        end = __shfl(end, src, 64);
        t.cnt = (int)(end - t.row0 < TOK ? end - t.row0 : TOK);
      }
      return t;
    }
  }
  const int64_t left = a.r - t.row0;
  if (left <= 0) t.expert = -1;
  t.cnt = (int)(left < 0 ? 0 : left < TOK ? left : TOK);
  return t;
}

__device__ __forceinline__ void store_y(const Q4Args &a, int64_t row, int64_t i, float v) {
  if (a.ybf16) ((uint16_t *)a.Y)[row * a.n + i] = (uint16_t)f32_to_bf16_bits(v);
  else ((float *)a.Y)[row * a.n + i] = v;
}

// ---------------------------------------------------------------- streaming kernel
// A workgroup owns 16 R output rows of one matrix and a tile of 16 TT rows of
// Y; its NW waves take the 128-column records in turn (wave w: w, w + NW, ...)
// and their sums are joined through LDS in wave order, so the result does not
// depend on timing.
// MFMA operands (v_mfma_f32_16x16x32_bf16): A = X (row l % 16, columns
// 8 (l / 16) .. +7), B = codes (column l % 16 = output row), D element j =
// (row 4 (l / 16) + j, output row l % 16): one lane keeps one output row, so a
// group's scale and zero are one pair per lane.  Row a of A is token
// 4 (a % 4) + a / 4 of its 16, which puts the first four tokens in element 0.
template <bool XBF16, int G, int R, int TT, int NW>
__global__ __launch_bounds__(64 * NW) void q4_stream_kernel(Q4Args a, int nrb, int nch) {
  constexpr int GPC = 128 / G, SPG = G / 32;     // groups per record, K slices per group
  constexpr int RECW = 256 + 32 * GPC;
  constexpr int NT = XBF16 ? 1 : 3;
  constexpr int TOK = 16 * TT;
  __shared__ float part[NW][R * TT * 256];
  const int lane = threadIdx.x & 63, r16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const RowTile tl = find_tile<TOK>(a, blockIdx.y);
  if (tl.expert < 0) return;
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
  const uint32_t *wp = a.W + (int64_t)tl.expert * nrb * nch * RECW + 4 * lane;

  f32x4_t tot[R][TT];
#pragma unroll
  for (int b = 0; b < R; ++b)
#pragma unroll
    for (int u = 0; u < TT; ++u) tot[b][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);

  if (!tl.bad) {
    for (int ch = wave; ch < nch; ch += NW) {
      uint4 w[R];
#pragma unroll
      for (int b = 0; b < R; ++b) {
        const int rb = rb0 + b < nrb ? rb0 + b : nrb - 1;
        w[b] = *(const uint4 *)(wp + ((int64_t)rb * nch + ch) * RECW);
      }
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
          for (int b = 0; b < R; ++b) c[b] = q4_codes(i == 0 ? w[b].x : i == 1 ? w[b].y : i == 2 ? w[b].z : w[b].w);
#pragma unroll
          for (int u = 0; u < TT; ++u) {
            uint4 x[NT];
            const char *p = xp[u] + (int64_t)(ch * 128 + 32 * i) * (XBF16 ? 2 : 4);
            if constexpr (XBF16) x[0] = *(const uint4 *)p;
            else split3((const float *)p, x);
#pragma unroll
            for (int e = 0; e < NT; ++e) {
              sx[u] = mfma16(x[e], ones, sx[u]);
#pragma unroll
              for (int b = 0; b < R; ++b) acc[b][u] = mfma16(x[e], c[b], acc[b][u]);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < R; ++b) {
          const int rb = rb0 + b < nrb ? rb0 + b : nrb - 1;
          const float2 sz = *(const float2 *)(wp - 4 * lane + ((int64_t)rb * nch + ch) * RECW + 256 + 2 * (16 * q + r16));
#pragma unroll
          for (int u = 0; u < TT; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tot[b][u][j] = fmaf(sz.x, fmaf(-sz.y, sx[u][j], acc[b][u][j]), tot[b][u][j]);
        }
      }
    }
  }
  // part[wave][(u * 4 + j) * 4 + lg][b][r16]: token 16 u + 4 j + lg, output row 16 b + r16
#pragma unroll
  for (int u = 0; u < TT; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int b = 0; b < R; ++b) part[wave][((16 * u + 4 * j + lg) * R + b) * 16 + r16] = tot[b][u][j];
  __syncthreads();
  for (int idx = threadIdx.x; idx < R * TT * 256; idx += 64 * NW) {
    const int tok = idx / (16 * R), col = idx % (16 * R);
    const int64_t i = (int64_t)rb0 * 16 + col;
    if (tok >= tl.cnt || i >= a.n) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += part[w][idx];
    const int64_t row = tl.row0 + tok;
    bool ok = !tl.bad;
    if (a.rows && ok) {
      const int32_t xr = a.rows[row];
      ok = xr >= 0 && xr < a.xrows;
    }
    if (a.row_scale) v *= a.row_scale[row];
    store_y(a, row, i, ok ? v : __uint_as_float(0x7fc00000u));
  }
}

// Most tiles of tok rows that e ranges covering at most r rows can be cut into.
int64_t max_tiles(int64_t r, int64_t e, int64_t tok) {
  const int64_t whole = (r + tok - 1) / tok;
  if (e <= 1) return whole;
  const int64_t ragged = (r + e * (tok - 1)) / tok;
  const int64_t most = ragged < r ? ragged : r;
  return most > whole ? most : whole;
}

template <bool XBF16, int G, int R, int TT, int NW>
hipError_t stream_go(const Q4Args &a, hipStream_t st) {
  const int nrb = (int)q4_row_blocks(a.n), nch = (int)q4_chunks(a.m);
  const int64_t tiles = max_tiles(a.r, a.offsets ? a.e : 1, 16 * TT);
  if (tiles > 65535) return hipErrorInvalidConfiguration;
  q4_stream_kernel<XBF16, G, R, TT, NW><<<dim3((nrb + R - 1) / R, (uint32_t)tiles), 64 * NW, 0, st>>>(a, nrb, nch);
  return hipGetLastError();
}

template <bool XBF16, int G>
hipError_t stream_pick(const Q4Args &a, hipStream_t st) {
  const int64_t per = a.offsets ? (a.r + a.e - 1) / a.e : a.r;
  if (per <= 16) return stream_go<XBF16, G, 1, 1, 8>(a, st);
  return stream_go<XBF16, G, 2, 4, 4>(a, st);
}

}  // namespace

hipError_t launch_pack4(const uint8_t *codes, const float *scale, const float *zero, int64_t e, int64_t n, int64_t m,
                        int group, uint32_t *packed, int32_t *info, hipStream_t st) {
  const int64_t nrb = q4_row_blocks(n), nch = q4_chunks(m), nrec = e * nrb * nch;
  const int64_t blocks = (nrec + 3) / 4 < 65536 ? (nrec + 3) / 4 : 65536;
  pack4_kernel<<<(uint32_t)blocks, 256, 0, st>>>(codes, scale, zero, n, m, group, nrb, nch, nrec, packed, info);
  return hipGetLastError();
}

size_t q4_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int, bool) { return 0; }

hipError_t launch_q4(const Q4Args &a, void *, hipStream_t st) {
  if (a.xbf16) {
    if (a.group == 128) return stream_pick<true, 128>(a, st);
    if (a.group == 64) return stream_pick<true, 64>(a, st);
    return stream_pick<true, 32>(a, st);
  }
  if (a.group == 128) return stream_pick<false, 128>(a, st);
  if (a.group == 64) return stream_pick<false, 64>(a, st);
  return stream_pick<false, 32>(a, st);
}

}  // namespace slim
