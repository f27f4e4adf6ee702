// Keys and values in 4 bits: appended to a paged cache with the position
// rotation applied on the way, and read back.
//
// A token's key (and value) of one head is cut into groups of g channels.  A
// group is held as its low end and a step, both bfloat16, and 4-bit codes:
//   low  = min x rounded down,  step = fl((max x - low) / 15) rounded up,
//   code = clamp(rint(fl(fl(x - low) fl(1 / step))), 0, 15),  value = fl(code step + low),
// all in float32 without contraction.  Down and up, so that the grid covers
// every entry: rounding to nearest would clip the ends by up to 15 half steps
// of the bfloat16 step.  16-bit pairs, not the float32 pairs of the weights'
// layout: a pair is read again for every token generated, and 4 bytes of 68
// (g = 128) or of 20 (g = 32) are read where it would be 8 of 72 or of 24.
// A step of 0 (a constant group) has codes 0; smaller steps than 2^-126 are
// raised to it (its reciprocal is then finite).  A group with an infinity or
// a NaN, or whose step or low end would be infinite, has step NaN and stands
// for NaN throughout.
//
// The rotation is computed in float64 from the float32 tables (products of
// float32 numbers are exact there, so a pair costs one rounding) and rounded
// to float32 once: every code is a function of the inputs alone, whatever
// kernel or order computed it.
#include <type_traits>

#include "common.hpp"
#include "serve.hpp"

namespace slim {

namespace {

// 8 consecutive channels c.. of a row as float32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t at, bool vec, float (&x)[8]) {
  if (BF16) {
    const uint16_t *s = (const uint16_t *)p + at;
    uint32_t w[4];
    if (vec) {
      const uint4 u = *(const uint4 *)s;
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)s[2 * i] | (uint32_t)s[2 * i + 1] << 16;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float *s = (const float *)p + at;
    if (vec) {
      const float4 a = ((const float4 *)s)[0], b = ((const float4 *)s)[1];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = s[i];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void *p, int64_t at) {
  return BF16 ? bf16_bits_to_f32(((const uint16_t *)p)[at]) : ((const float *)p)[at];
}

// Channels c0 .. c0 + 7 (x) of the head at `at` turned by the row of the
// table; `half` = rot / 2.
template <bool BF16>
__device__ __forceinline__ void rotate8(const Kv4Append &a, const Kv4Rows &s, int64_t at, int c0, const float *row,
                                        float (&x)[8]) {
  const int half = a.rot >> 1;
  if (c0 >= a.rot) return;
  // products of float32 numbers are exact in float64, so a fused sum rounds as a separate one would
  if (a.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const int i = (c0 + e) >> 1;
      if (c0 + e < a.rot) {
        const double c = row[i], n = row[half + i], u = x[e], w = x[e + 1];
        x[e] = (float)__builtin_fma(u, c, -(w * n));
        x[e + 1] = (float)__builtin_fma(w, c, u * n);
      }
    }
    return;
  }
  float y[8];
  if ((half & 7) == 0) {                    // the partners, and the angles, are 8 consecutive ones too
    const bool low = c0 < half;
    const int i = low ? c0 : c0 - half;
    float co[8], si[8];
    load8<BF16>(s.p, at + (low ? c0 + half : c0 - half), s.vec, y);
    load8<false>(row, i, a.rvec, co);
    load8<false>(row, half + i, a.rvec, si);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double w = low ? -y[e] : y[e];
      x[e] = (float)__builtin_fma((double)x[e], (double)co[e], w * (double)si[e]);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = c0 + e;
    y[e] = c < a.rot ? load1<BF16>(s.p, at + (c < half ? c + half : c - half)) : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = c0 + e;
    if (c < a.rot) {
      const int i = c < half ? c : c - half;
      const double co = row[i], si = row[half + i], u = x[e], w = y[e];
      x[e] = (float)__builtin_fma(u, co, c < half ? -(w * si) : w * si);
    }
  }
}

// Least and greatest over aligned groups of W = 4, 8 or 16 lanes by data-parallel moves.
template <int W, class Op>
__device__ __forceinline__ float over_lanes(float x, Op op) {
  auto from = [&](auto ctrl) __attribute__((always_inline)) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  x = op(x, from(std::integral_constant<int, 0xb1>()));                 // lane ^ 1
  x = op(x, from(std::integral_constant<int, 0x4e>()));                 // lane ^ 2
  if (W >= 8) x = op(x, from(std::integral_constant<int, 0x141>()));    // lane ^ 7 of 8
  if (W >= 16) x = op(x, from(std::integral_constant<int, 0x140>()));   // lane ^ 15 of 16
  return x;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

struct Pair {
  float step, low;
  uint32_t word;             // both as bfloat16
};

// Step and low end of the group that W lanes' 8 channels make up.
template <int W>
__device__ __forceinline__ Pair group_pair(const float (&x)[8]) {
  float lo = x[0], hi = x[0];
  bool fin = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
    fin &= fabsf(x[e]) < __uint_as_float(0x7f800000u);
  }
  if (!fin) hi = __uint_as_float(0x7f800000u);             // carries through the maximum
  lo = over_lanes<W>(lo, [](float a, float b) { return fminf(a, b); });
  hi = over_lanes<W>(hi, [](float a, float b) { return fmaxf(a, b); });
  uint32_t u = __float_as_uint(lo);
  u = (u >> 31 ? u + 0xffffu : u) & 0xffff0000u;
  Pair p;
  p.low = __uint_as_float(u);
  float s = (hi - p.low) / 15.0f;
  s = __uint_as_float((__float_as_uint(s) + 0xffffu) & 0xffff0000u);
  if (s > 0.0f) s = fmaxf(s, 0x1p-126f);
  if (!(s < __uint_as_float(0x7f800000u)) || !(fabsf(p.low) < __uint_as_float(0x7f800000u))) {
    p.step = __uint_as_float(0x7fc00000u);
    p.low = 0.0f;
  } else {
    p.step = s;
  }
  p.word = (__float_as_uint(p.step) >> 16) | __float_as_uint(p.low);
  return p;
}

// A lane takes 8 channels of a head of a token: dim / 8 lanes a head, so a
// wave 4 heads of 128.  Items run over the heads of q, k and v of a token.
// Nothing is shared between lanes but the groups' extremes, and every word or
// byte of the cache is written by one lane, so no write reads what another
// token wrote.  2048 tokens of 64 + 8 heads of 128, g = 64: 79 MB in 25 us, 3.2
// TB/s (a copy of 4 GiB has 4.7, that would be 17 us).  The vector unit is 47%
// busy, and a lane waits for its one load of 16 bytes, its partner's, which is
// loaded twice, and the table's, loaded again for every head.  Few tokens:
// one chain of reads (3.8 us).
template <bool BF16, int DIM, int GROUP>
__global__ __launch_bounds__(256) void kv4_append_kernel(const Kv4Append a) {
  constexpr int L = DIM / 8, W = GROUP / 8, NG = DIM / GROUP, REC = 4 * DIM + 32 * NG;
  const unsigned item = blockIdx.x * (256 / L) + threadIdx.x / L;
  const int l = threadIdx.x % L;
  const unsigned per = (unsigned)(a.q.heads + 2 * a.k.heads);
  const unsigned tok = item / per;
  if (tok >= a.t) return;
  int h = (int)(item - tok * per);
  const int kind = h < a.q.heads ? 0 : h < a.q.heads + a.k.heads ? 1 : 2;
  h -= (int)(kind == 0 ? 0 : kind == 1 ? a.q.heads : a.q.heads + a.k.heads);
  const Kv4Rows &s = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  int64_t slot = 0;
  if (kind > 0) {
    slot = a.slots[tok];
    if (slot < 0 || slot >= a.pages * a.page) return;
  }
  const int64_t at = tok * s.row + h * s.head;
  const int c0 = 8 * l;
  float x[8];
  load8<BF16>(s.p, at + c0, s.vec, x);
  if (kind < 2 && a.rotary) {
    const int64_t pos = a.positions[tok];
    if (pos < 0 || pos >= a.npos) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(0x7fc00000u);
    } else {
      rotate8<BF16>(a, s, at, c0, a.rotary + pos * a.rot, x);
    }
  }
  if (kind == 0) {
    const int64_t o = (tok * a.q.heads + h) * DIM + c0;
    if (BF16) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      *(uint4 *)((uint16_t *)a.q_out + o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      ((float4 *)((float *)a.q_out + o))[0] = make_float4(x[0], x[1], x[2], x[3]);
      ((float4 *)((float *)a.q_out + o))[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    return;
  }
  const Pair p = group_pair<W>(x);
  const float inv = p.step > 0.0f ? 1.0f / p.step : 0.0f;
  uint32_t code[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)   // a NaN step gives NaN here, which the clamp makes 0
    code[e] = (uint32_t)fminf(fmaxf(rintf((x[e] - p.low) * inv), 0.0f), 15.0f);
  const int log = a.page_log, in = (int)slot & (a.page - 1), t16 = in & 15;
  uint32_t *rec = a.cache + ((((slot >> log) * a.k.heads + h) << (log - 4)) + (in >> 4)) * REC;
  if (kind == 1) {
    uint32_t w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) w |= (code[b] | code[b + 4] << 4) << (8 * b);
    rec[(16 * (l & 3) + t16) * (DIM / 32) + (l >> 2)] = w;
  } else {
    uint8_t *o = (uint8_t *)(rec + 2 * DIM) + (t16 & 3);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      o[4 * ((16 * (t16 >> 2) + 4 * (l & 3) + b) * (DIM / 32) + (l >> 2))] = (uint8_t)(code[2 * b] | code[2 * b + 1] << 4);
  }
  if (l % W == 0) rec[4 * DIM + (kind == 2 ? 16 * NG : 0) + 16 * (l / W) + t16] = p.word;
}

// The values of given slots.  A lane reads 8 channels, as above.  2048 slots of 8
// heads of 128 as float32: 19 MB in 7.4 to 8.0 us (4 at the copy's rate).  The
// value codes are read byte by byte, and neighbouring tokens, whose bytes share a
// word, go to workgroups of other XCDs: 14 MB are fetched for 2.4.
template <int DIM, int GROUP>
__global__ __launch_bounds__(256) void kv4_read_kernel(const int32_t *__restrict__ slots, int64_t t,
                                                       const uint32_t *__restrict__ cache, int64_t pages,
                                                       int heads, int page_log, void *__restrict__ k,
                                                       void *__restrict__ v, bool bf16) {
  constexpr int L = DIM / 8, W = GROUP / 8, NG = DIM / GROUP, REC = 4 * DIM + 32 * NG;
  const unsigned item = blockIdx.x * (256 / L) + threadIdx.x / L;
  const int l = threadIdx.x % L;
  const unsigned tok = item / (unsigned)(2 * heads);
  if (tok >= t) return;
  const int hh = (int)(item - tok * 2 * heads);
  const bool val = hh >= heads;
  const int h = val ? hh - heads : hh;
  const int64_t slot = slots[tok];
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= pages << page_log) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(0x7fc00000u);
  } else if (slot >= 0) {
    const int in = (int)slot & ((1 << page_log) - 1), t16 = in & 15;
    const uint32_t *rec = cache + ((((slot >> page_log) * heads + h) << (page_log - 4)) + (in >> 4)) * REC;
    const uint32_t pair = rec[4 * DIM + (val ? 16 * NG : 0) + 16 * (l / W) + t16];
    const float step = __uint_as_float(pair << 16), low = __uint_as_float(pair & 0xffff0000u);
    uint32_t code[8];
    if (!val) {
      const uint32_t w = rec[(16 * (l & 3) + t16) * (DIM / 32) + (l >> 2)];
#pragma unroll
      for (int b = 0; b < 4; ++b) code[b] = w >> (8 * b) & 15u, code[b + 4] = w >> (8 * b + 4) & 15u;
    } else {
      const uint8_t *o = (const uint8_t *)(rec + 2 * DIM) + (t16 & 3);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t w = o[4 * ((16 * (t16 >> 2) + 4 * (l & 3) + b) * (DIM / 32) + (l >> 2))];
        code[2 * b] = w & 15u, code[2 * b + 1] = w >> 4;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)code[e] * step + low;
  }
  const int64_t o = ((int64_t)tok * heads + h) * DIM + 8 * l;
  void *out = val ? v : k;
  if (bf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    *(uint4 *)((uint16_t *)out + o) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    ((float4 *)((float *)out + o))[0] = make_float4(x[0], x[1], x[2], x[3]);
    ((float4 *)((float *)out + o))[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// f<DIM, GROUP> for the call's sizes (kv4_shape holds).
#define KV4_BY_SHAPE(dim, group, F)              \
  do {                                           \
    if (dim == 64) {                             \
      if (group == 32) F(64, 32);                \
      else F(64, 64);                            \
    } else if (dim == 128) {                     \
      if (group == 32) F(128, 32);               \
      else if (group == 64) F(128, 64);          \
      else F(128, 128);                          \
    } else {                                     \
      if (group == 32) F(256, 32);               \
      else if (group == 64) F(256, 64);          \
      else F(256, 128);                          \
    }                                            \
  } while (0)

}  // namespace

// Tokens a launch takes: it has less than 2^32 threads, and items are counted in 32 bits.
static int64_t tokens_a_launch(int64_t heads, int dim) { return ((int64_t)1 << 31) / (heads * (dim / 8)); }

hipError_t launch_kv4_append(const Kv4Append &all, hipStream_t st) {
  const int64_t heads = all.q.heads + 2 * all.k.heads, per = 256 / (all.dim / 8), most = tokens_a_launch(heads, all.dim);
  const int64_t size = all.bf16 ? 2 : 4;
  for (int64_t t0 = 0; t0 < all.t; t0 += most) {
    Kv4Append a = all;
    a.t = all.t - t0 < most ? all.t - t0 : most;
    a.k.p = (const char *)all.k.p + t0 * all.k.row * size;
    a.v.p = (const char *)all.v.p + t0 * all.v.row * size;
    if (all.q.p) {
      a.q.p = (const char *)all.q.p + t0 * all.q.row * size;
      a.q_out = (char *)all.q_out + t0 * all.q.heads * all.dim * size;
    }
    a.slots = all.slots + t0;
    if (all.positions) a.positions = all.positions + t0;
    const unsigned grid = (unsigned)((a.t * heads + per - 1) / per);
#define F(D, G)                                                                \
  do {                                                                         \
    if (a.bf16) kv4_append_kernel<true, D, G><<<grid, 256, 0, st>>>(a);        \
    else kv4_append_kernel<false, D, G><<<grid, 256, 0, st>>>(a);              \
  } while (0)
    KV4_BY_SHAPE(a.dim, a.group, F);
#undef F
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv4_read(const int32_t *slots, int64_t t, const uint32_t *cache, int64_t pages, int64_t heads,
                           int dim, int group, int page, void *k, void *v, bool bf16, hipStream_t st) {
  const int64_t per = 256 / (dim / 8), most = tokens_a_launch(2 * heads, dim), row = heads * dim * (bf16 ? 2 : 4);
  for (int64_t t0 = 0; t0 < t; t0 += most) {
    const int64_t n = t - t0 < most ? t - t0 : most;
    const unsigned grid = (unsigned)((n * 2 * heads + per - 1) / per);
#define F(D, G)                                                                                              \
  kv4_read_kernel<D, G><<<grid, 256, 0, st>>>(slots + t0, n, cache, pages, (int)heads, __builtin_ctz(page), \
                                              (char *)k + t0 * row, (char *)v + t0 * row, bf16)
    KV4_BY_SHAPE(dim, group, F);
#undef F
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace slim
