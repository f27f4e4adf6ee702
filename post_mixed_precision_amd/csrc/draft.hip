// Verification of drafted tokens against the target's probabilities.
//
//   p_j = softmax(target[j] / T), q_j = softmax(draft[j] / T)   (no draft: q_j is 1 at the drafted token)
//   token x_j is taken while u_j q_j(x_j) < p_j(x_j);  at the first that is not, the next token is drawn from
//   max(p_j - q_j, 0) (0 up to 2^-44 p_j), after the last from p:  the first entry whose running sum exceeds u_k times the whole.
//
// The drawn token is an index: with 10^5 entries a running sum moves by 10^-5
// an entry and less, so float32 sums (off by 10^-7 and more) would draw a
// neighbour once in a hundred.  Powers, sums and comparisons are float64
// throughout; the index is then a function of the inputs but for borders
// nearer than 10^-13.
//
// Three launches: statistics of every row by segments, then the decision and
// the segment masses of the row to draw from, then the segment and the entry.
// The first one reads all logits once and forms a float64 power of each (17
// vector instructions, 9 of them float64, which run at the rate of float32's
// here): 352 rows of 131072 bfloat16 logits take 37 us, their loads alone 23.  Segments twice as long
// took as long, half as long 41 us, and so did workgroups that go on to the next
// segment with its loads in flight (46); all but the powers' work: 41 with six instructions more a power.
#include "common.hpp"
#include "serve.hpp"
#include "slim.h"

namespace slim {

namespace {

constexpr double kNegInf = -__builtin_inf();
constexpr double kLog2e = 1.4426950408889634074;

// 2^t for t up to 1023 (0 for -inf): t = n + f, |f| <= 1/2, and the polynomial
// that meets 2^f at the 11 Chebyshev points of [-1/2, 1/2] (off by 3.2e-16 of the value at most).
__device__ __forceinline__ double exp2_64(double t) {
  t = fmax(t, -1100.0);
  const double n = __builtin_rint(t), f = t - n;
  double p = 0x1.e6063f7217bc6p-28;
  p = __builtin_fma(p, f, 0x1.b675bca4eeebbp-24);
  p = __builtin_fma(p, f, 0x1.62bfd47773353p-20);
  p = __builtin_fma(p, f, 0x1.ffcb54062e698p-17);
  p = __builtin_fma(p, f, 0x1.430913096fd9fp-13);
  p = __builtin_fma(p, f, 0x1.5d87fe9d7a584p-10);
  p = __builtin_fma(p, f, 0x1.3b2ab6fba1ddap-7);
  p = __builtin_fma(p, f, 0x1.c6b08d703ce49p-5);
  p = __builtin_fma(p, f, 0x1.ebfbdff82c598p-3);
  p = __builtin_fma(p, f, 0x1.62e42fefa3a19p-1);
  p = __builtin_fma(p, f, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// 2^(t / 256) for t = n + g, n whole, |g| <= 1/2, from a table of 2^(i / 256): the polynomial that meets
// (2^(g / 256) - 1) / g at the 3 Chebyshev points of [-1/2, 1/2] is off by 3.5e-14 at most.  n is the low
// word of kMagic + t; added to an entry's high word 12 bits up it sets the
// exponent (n >= -1022 * 256), its own low 8 bits being taken off in the table.
constexpr double kMagic = 0x1.8p52, kLowest = -1020.0 * 256.0;
typedef double PowTable[256];
__device__ __forceinline__ void make_table(PowTable &table) {   // by 256 threads, seen after the next barrier
  uint2 w = __builtin_bit_cast(uint2, exp2_64(threadIdx.x * (1.0 / 256.0)));
  w.y -= threadIdx.x << 12;
  table[threadIdx.x] = __builtin_bit_cast(double, w);
}
__device__ __forceinline__ double exp2_256th(double magic_t, double g, const PowTable &table) {
  const uint32_t i = (uint32_t)__double2loint(magic_t);
  double p = 0x1.c6b08f7c960adp-29;
  p = __builtin_fma(p, g, 0x1.ebfbe3a9ac80bp-19);
  p = __builtin_fma(p, g, 0x1.62e42fefa39efp-9);
  uint2 w = __builtin_bit_cast(uint2, table[i & 255]);
  asm("v_lshl_add_u32 %0, %1, 12, %2" : "=v"(w.y) : "v"(i), "v"(w.y));   // else three instructions of 64 bits
  const double s = __builtin_bit_cast(double, w);
  return __builtin_fma(p * g, s, s);
}
// 2^(t / 256), 0 below 2^-1020 and for NaN.
__device__ __forceinline__ double exp2_256th(double t, const PowTable &table) {
  const double u = fmax(t, kLowest), y = u + kMagic, z = exp2_256th(y, u - (y - kMagic), table);
  return t > kLowest ? z : 0.0;
}
// max(x, y) for a y that is a number; fmaxf also makes a signalling x quiet, by an instruction of its own.
__device__ __forceinline__ float at_least(float x, float y) {
  float z;
  asm("v_max_f32 %0, %1, %2" : "=v"(z) : "v"(x), "v"(y));
  return z;
}

template <bool BF16>
__device__ __forceinline__ float logit(const void *p, int64_t at) {
  return BF16 ? bf16_bits_to_f32(((const uint16_t *)p)[at]) : ((const float *)p)[at];
}

// What a logit's difference to its row's maximum is multiplied by (finite: 0 stays 0).
__device__ __forceinline__ double power_of(const DraftArgs &a) { return fmin(kLog2e / a.temperature, 1e300); }

__device__ __forceinline__ double wave_sum(double v) { return group_sum<64>(v); }

// Rows of a sequence: k + 1 of the target, then k of the draft.
struct RowOf {
  const void *p;
  int64_t at;
};
__device__ __forceinline__ RowOf row_of(const DraftArgs &a, int64_t seq, int j) {
  if (j <= a.k) return {a.target, seq * a.t_seq + j * a.t_row};
  return {a.draft, seq * a.d_seq + (j - a.k - 1) * a.d_row};
}

// One segment's maximum m and sum of 2^((x - m) log2 e / T), as (m, sum); a
// NaN or +inf makes the sum NaN.  A thread takes 16-byte pieces (on the row's
// own 16-byte grid: rows may start anywhere), the ragged ones at the row's
// ends entry by entry.
template <bool BF16, int PIECES>
__global__ __launch_bounds__(256) void draft_stats_kernel(const DraftArgs a, const int nseg, double2 *__restrict__ st) {
  constexpr int PER = BF16 ? 8 : 4, SIZE = BF16 ? 2 : 4;
  __shared__ float s_m[4];
  __shared__ double s_z[4];
  __shared__ PowTable s_pow;
  make_table(s_pow);
  const unsigned nr = a.draft ? 2 * a.k + 1 : a.k + 1;
  const unsigned row = blockIdx.x / (unsigned)nseg, seq = row / nr;
  const int s = (int)(blockIdx.x - row * nseg);
  const RowOf r = row_of(a, seq, (int)(row - seq * nr));
  const char *first = (const char *)r.p + r.at * SIZE;
  const int lead = (int)((uintptr_t)first & 15) / SIZE;    // entries of the grid before the row
  float x[PIECES][PER];
  const int64_t v0 = (int64_t)s * PIECES * 256 * PER - lead;
  uint4 u[PIECES];
  if (v0 >= 0 && v0 + PIECES * 256 * PER <= a.v) {         // all loads at once
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      u[i] = *(const uint4 *)(first + (v0 + (i * 256 + (int)threadIdx.x) * PER) * SIZE);
  } else {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int64_t v = v0 + (i * 256 + (int)threadIdx.x) * PER;
      if (v >= 0 && v + PER <= a.v) {
        u[i] = *(const uint4 *)(first + v * SIZE);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const uint32_t f = v + e >= 0 && v + e < a.v ? __float_as_uint(logit<BF16>(first, v + e)) : 0xff800000u;
          if constexpr (!BF16) w[e] = f;
          else if (e & 1) w[e >> 1] |= f;
          else w[e >> 1] = f >> 16;
        }
        u[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  float m = -__builtin_inff();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (BF16) {
        x[i][2 * e] = __uint_as_float(w[e] << 16), x[i][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      } else {
        x[i][e] = __uint_as_float(w[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      bad |= !(x[i][e] < __builtin_inff());
      m = fmaxf(m, x[i][e]);
    }
  }
  m = group_max<64>(m);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) s_m[wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const double c = 256.0 * power_of(a), md = m == -__builtin_inff() || bad ? 0.0 : (double)m;
  double z = 0.0;
  const double whole = __builtin_rint(-md * c), low = md + kLowest / c;
  const float least = (float)low;
  if (fabs(whole) < 0x1p45 && low > -0x1p127 && fabs((double)least - low) * c < 256.0) {
    // about a whole number `whole` near -m c: fma(x, c, kMagic + whole) is then n in the low word, and g takes
    // one more; entries below `least`, -inf too, become 2^-1020, or that and its rounding, beside a sum of 1 and more
    const double base = kMagic + whole;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const double xd = (double)at_least(x[i][e], least), y = __builtin_fma(xd, c, base);
        z += exp2_256th(y, __builtin_fma(xd, c, base - y), s_pow);
      }
    z *= exp2_64(__builtin_fma(md, -c, -whole) * (1.0 / 256.0));
  } else {   // logits of 10^11 (of the type's lowest, say), or no float between m and `low`: x - m first
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int e = 0; e < PER; ++e) z += exp2_256th(((double)x[i][e] - md) * c, s_pow);
  }
  if (bad) z = __builtin_nan("");
  z = wave_sum(z);
  if ((threadIdx.x & 63) == 0) s_z[wave] = z;
  __syncthreads();
  if (threadIdx.x == 0) st[blockIdx.x] = make_double2((double)m, (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]));
}

// What is drawn from: p, or max(p - q, 0) with q of the draft's row or 1 at `token`.
struct Mass {
  int64_t token;             // of a draft without probabilities, else -1
  double c, tm, tz, dm, dz;  // 256 log2 e / T; the rows' maxima and reciprocal sums
  int taken, minus;
  int64_t pad;
};
// Of entry v with logits x (target) and y (draft; any number if there is none).
__device__ __forceinline__ double mass_of(const Mass &m, float x, float y, int64_t v, const PowTable &table) {
  const double p = exp2_256th(((double)x - m.tm) * m.c, table) * m.tz;
  if (!m.minus) return p;
  if (m.token >= 0) return v == m.token ? 0.0 : p;
  // the rows' sums differ in their last bits even for equal rows (their grids differ), and of those nothing is drawn
  const double d = p - exp2_256th(((double)y - m.dm) * m.c, table) * m.dz;
  return d > 0x1p-44 * p ? d : 0.0;
}
// The masses of 8 entries first, first + STEP, ...; 0 from `end` on.  All loads before the first power.
template <bool BF16, int STEP>
__device__ __forceinline__ void masses(const DraftArgs &a, int64_t seq, const Mass &m, int64_t first, int64_t end,
                                       const PowTable &table, double (&z)[8]) {
  const RowOf t = row_of(a, seq, m.taken), d = m.minus && a.draft ? row_of(a, seq, a.k + 1 + m.taken) : t;
  float x[8], y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t v = first + STEP * e, in = v < end ? v : end - 1;
    x[e] = logit<BF16>(t.p, t.at + in);
    y[e] = logit<BF16>(d.p, d.at + in);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t v = first + STEP * e;
    z[e] = v < end ? mass_of(m, x[e], y[e], v, table) : 0.0;
  }
}

// Every workgroup of a sequence decides for itself: 16 lanes join the segments
// of a row, then lane j of each wave judges token j.
template <bool BF16>
__device__ __forceinline__ Mass decide(const DraftArgs &a, int64_t seq, const double2 *st, int nseg,
                                       double2 (&s_row)[2 * SLIM_DRAFT_MAX_K + 1]) {
  const int nr = a.draft ? 2 * a.k + 1 : a.k + 1, lane = threadIdx.x & 63;
  const double c = power_of(a);        // a power's argument is (x - m) c: exact where x is m, however large
  const int64_t x = lane < a.k ? a.tokens[seq * a.k + lane] : -1;
  const float u = lane < a.k ? a.uniform[seq * (a.k + 1) + lane] : 0.0f;
  float tx = 0.0f, dx = 0.0f;                    // asked for here, needed after the rows
  if (x >= 0 && x < a.v) {
    const RowOf t = row_of(a, seq, lane);
    tx = logit<BF16>(t.p, t.at + x);
    if (a.draft) {
      const RowOf d = row_of(a, seq, a.k + 1 + lane);
      dx = logit<BF16>(d.p, d.at + x);
    }
  }
  for (int j0 = 0; j0 < nr; j0 += 16) {
    const int j = j0 + (threadIdx.x >> 4), l = threadIdx.x & 15;
    if (j < nr) {
      const double2 *p = st + (seq * nr + j) * nseg;
      const double2 f = l < nseg ? p[l] : make_double2(kNegInf, 0.0);
      double m = f.x;
      for (int s = 16 + l; s < nseg; s += 16) m = fmax(m, p[s].x);
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) m = fmax(m, __shfl_xor(m, x, 64));
      if (m == kNegInf) m = 0.0;
      double z = f.y * exp2_64((f.x - m) * c);
      for (int s = 16 + l; s < nseg; s += 16) z += p[s].y * exp2_64((p[s].x - m) * c);
      z = group_sum<16>(z);
      if (l == 0) s_row[j] = make_double2(m, 1.0 / z);   // nothing but -inf: 1 / 0, and 0 * inf is a NaN below
    }
  }
  __syncthreads();
  bool good = false;
  if (x >= 0 && x < a.v) {                       // lanes below k
    const double p = exp2_64(((double)tx - s_row[lane].x) * c) * s_row[lane].y;
    double q = 1.0;
    if (a.draft) q = exp2_64(((double)dx - s_row[a.k + 1 + lane].x) * c) * s_row[a.k + 1 + lane].y;
    good = (double)u * q < p;
  }
  const uint64_t no = ~__ballot(good);           // lanes from k on are in it
  Mass m = {};
  m.taken = __ffsll((unsigned long long)no) - 1;
  const int j = m.taken;
  const int64_t refused = __shfl(x, j, 64);      // lane k: -1
  m.minus = refused >= 0;
  m.token = m.minus && !a.draft ? refused : -1;
  m.c = 256.0 * c, m.tm = s_row[j].x, m.tz = s_row[j].y;
  if (m.minus && a.draft) m.dm = s_row[a.k + 1 + j].x, m.dz = s_row[a.k + 1 + j].y;
  return m;
}

// The masses of runs of kRun entries, `each` of them a workgroup (several
// where there are many: every workgroup decides first).
constexpr int kRun = 2048;
template <bool BF16>
__global__ __launch_bounds__(256) void draft_mass_kernel(const DraftArgs a, const int nseg, const int runs,
                                                         const int each, const double2 *__restrict__ st,
                                                         double *__restrict__ mass, Mass *__restrict__ drawn) {
  __shared__ double2 s_row[2 * SLIM_DRAFT_MAX_K + 1];
  __shared__ double s_z[2][4];
  __shared__ PowTable s_pow;
  make_table(s_pow);
  const unsigned per = (unsigned)(runs + each - 1) / (unsigned)each, seq = blockIdx.x / per;
  const int s0 = (int)(blockIdx.x - seq * per) * each, s1 = s0 + each < runs ? s0 + each : runs;
  const Mass m = decide<BF16>(a, seq, st, nseg, s_row);
  if (s0 == 0 && threadIdx.x == 0) drawn[seq] = m;
  for (int s = s0; s < s1; ++s) {
    double x[8];
    masses<BF16, 256>(a, seq, m, (int64_t)s * kRun + threadIdx.x, a.v, s_pow, x);
    const double z = wave_sum(((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])));
    if ((threadIdx.x & 63) == 0) s_z[s & 1][threadIdx.x >> 6] = z;
    __syncthreads();                             // one a run: the next run's sums go to the other half
    if (threadIdx.x == 0)
      mass[(int64_t)seq * runs + s] = (s_z[s & 1][0] + s_z[s & 1][1]) + (s_z[s & 1][2] + s_z[s & 1][3]);
  }
}

__device__ __forceinline__ double wave_running_sum(double x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double up = __shfl_up(x, d, 64);
    if (lane >= d) x += up;
  }
  return x;
}

template <bool BF16>
__global__ __launch_bounds__(256) void draft_pick_kernel(const DraftArgs a, const int runs,
                                                         const double *__restrict__ mass,
                                                         const Mass *__restrict__ drawn) {
  __shared__ double s_z[4];
  __shared__ PowTable s_pow;
  __shared__ int s_hit[4], s_last[4];
  const int64_t seq = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  make_table(s_pow);
  __syncthreads();
  const Mass m = drawn[seq];
  const double *ms = mass + seq * runs;
  // every wave finds the run: the first whose running mass exceeds what is wanted (with a uniform of 1 or
  // more: the last that has any)
  const double first = lane < runs ? ms[lane] : 0.0;
  double all = first;
  for (int s = 64 + lane; s < runs; s += 64) all += ms[s];
  all = wave_sum(all);
  const double want = (double)a.uniform[seq * (a.k + 1) + a.k] * all;
  int hs = -1, last = -1;
  double left = 0.0, run = 0.0, lastleft = 0.0;
  if (all > 0.0) {                               // a NaN: a row without a distribution
    for (int s0 = 0; s0 < runs && hs < 0; s0 += 64) {
      const double x = s0 == 0 ? first : s0 + lane < runs ? ms[s0 + lane] : 0.0, incl = wave_running_sum(x);
      const uint64_t over = __ballot(x > 0.0 && run + incl > want), some = __ballot(x > 0.0);
      const int at = over ? __ffsll((unsigned long long)over) - 1 : some ? 63 - __clzll((long long)some) : -1;
      if (at >= 0) {
        const double before = want - (run + __shfl(incl - x, at, 64));
        if (over) hs = s0 + at, left = before;
        else last = s0 + at, lastleft = before;
      }
      run += __shfl(incl, 63, 64);
    }
    if (hs < 0) hs = last, left = lastleft;
  }
  int64_t pick = -1;
  if (hs >= 0) {                                 // the same in every wave
    double x[8], sum = 0.0;
    masses<BF16, 1>(a, seq, m, (int64_t)hs * kRun + 8 * tid, a.v, s_pow, x);
    int lastpos = -1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (x[e] > 0.0) lastpos = 8 * tid + e;
      sum += x[e];
    }
    const double incl = wave_running_sum(sum);
    if (lane == 63) s_z[wave] = incl;
    __syncthreads();
    double at = incl - sum;
    for (int w = 0; w < wave; ++w) at += s_z[w];
    int hit = kRun;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      at += x[e];
      if (hit == kRun && x[e] > 0.0 && at > left) hit = 8 * tid + e;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      hit = min(hit, __shfl_xor(hit, d, 64));
      lastpos = max(lastpos, __shfl_xor(lastpos, d, 64));
    }
    if (lane == 0) s_hit[wave] = hit, s_last[wave] = lastpos;
    __syncthreads();
    hit = min(min(s_hit[0], s_hit[1]), min(s_hit[2], s_hit[3]));
    lastpos = max(max(s_last[0], s_last[1]), max(s_last[2], s_last[3]));
    // rounding can leave the run's running sum just short of its mass: its last entry then
    const int in = hit < kRun ? hit : lastpos;
    if (in >= 0) pick = (int64_t)hs * kRun + in;
  }
  if (tid <= a.k)
    a.ids[seq * (a.k + 1) + tid] = tid < m.taken ? a.tokens[seq * a.k + tid] : tid == m.taken ? pick : -1;
  if (tid == 0) a.accepted[seq] = m.taken;
}

// Logits a thread of the first kernel holds: 8 (few rows: more workgroups) or 32.
template <bool BF16>
hipError_t launch(const DraftArgs &a, void *ws, const DraftPlan &p, hipStream_t st) {
  const int nr = a.draft ? 2 * a.k + 1 : a.k + 1;
  Mass *drawn = (Mass *)ws;
  double2 *stat = (double2 *)(drawn + a.b);
  double *mass = (double *)(stat + a.b * nr * p.nseg);
  const unsigned rows = (unsigned)(a.b * nr * p.nseg);
  constexpr int PIECE = BF16 ? 8 : 4;
  if (p.few) draft_stats_kernel<BF16, 8 / PIECE><<<rows, 256, 0, st>>>(a, p.nseg, stat);
  else draft_stats_kernel<BF16, 32 / PIECE><<<rows, 256, 0, st>>>(a, p.nseg, stat);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned groups = (unsigned)(a.b * ((p.runs + p.each - 1) / p.each));
  draft_mass_kernel<BF16><<<groups, 256, 0, st>>>(a, p.nseg, p.runs, p.each, stat, mass, drawn);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  draft_pick_kernel<BF16><<<(unsigned)a.b, 256, 0, st>>>(a, p.runs, mass, drawn);
  return hipGetLastError();
}

}  // namespace

DraftPlan draft_plan(int64_t b, int k, int64_t v) {
  DraftPlan p;
  const int64_t rows = b * (2 * k + 1), wide = v + 7;         // a row's 16-byte grid may start 7 entries before it
  p.few = rows * ((wide + 2047) / 2048) <= 1024;
  const int64_t seg = p.few ? 2048 : 8192;
  p.nseg = (int)((wide + seg - 1) / seg);
  p.runs = (int)((v + kRun - 1) / kRun);
  const int64_t each = b * p.runs / 768;                       // three workgroups a CU
  p.each = (int)(each < 1 ? 1 : each > 8 ? 8 : each);
  p.ws_bytes = (size_t)b * sizeof(Mass) + (size_t)rows * p.nseg * 16 + (size_t)b * p.runs * 8;
  return p;
}

hipError_t launch_verify_draft(const DraftArgs &a, void *ws, const DraftPlan &p, hipStream_t st) {
  return a.bf16 ? launch<true>(a, ws, p, st) : launch<false>(a, ws, p, st);
}

}  // namespace slim
