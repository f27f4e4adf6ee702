// Verification of drafted tokens against the target's probabilities.
//
//   p_j = softmax(target[j] / T), q_j = softmax(draft[j] / T)   (no draft: q_j is 1 at the drafted token)
//   token x_j is taken while u_j q_j(x_j) < p_j(x_j);  at the first that is not, the next token is drawn from
//   max(p_j - q_j, 0), after the last from p:  the first entry whose running sum exceeds u_k times the whole.
//
// The drawn token is an index: with 10^5 entries a running sum moves by 10^-5
// an entry and less, so float32 sums (off by 10^-7 and more) would draw a
// neighbour once in a hundred.  Powers, sums and comparisons are float64
// throughout; the index is then a function of the inputs but for borders
// nearer than 10^-15.
//
// Three launches: statistics of every row by segments (bound by reading the
// logits and by the float64 powers), then the decision and the segment masses
// of the row to draw from, then the segment and the entry.
#include "common.hpp"
#include "serve.hpp"
#include "slim.h"

namespace slim {

namespace {

constexpr double kNegInf = -__builtin_inf();

template <bool BF16>
__device__ __forceinline__ float logit(const void *p, int64_t at) {
  return BF16 ? bf16_bits_to_f32(((const uint16_t *)p)[at]) : ((const float *)p)[at];
}

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

// One segment's maximum and sum of powers, (max, sum); a NaN or +inf makes the sum NaN.
template <bool BF16, int E>
__global__ __launch_bounds__(256) void draft_stats_kernel(const DraftArgs a, const int nseg, double2 *__restrict__ st) {
  __shared__ float s_m[4];
  __shared__ double s_z[4];
  const int nr = a.draft ? 2 * a.k + 1 : a.k + 1;
  const int64_t row = blockIdx.x / (unsigned)nseg;
  const int s = (int)(blockIdx.x % (unsigned)nseg);
  const int64_t seq = row / nr;
  const RowOf r = row_of(a, seq, (int)(row - seq * nr));
  const int64_t v0 = (int64_t)s * (256 * E);
  float x[E];
  float m = -__builtin_inff();
  bool bad = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t v = v0 + 256 * e + threadIdx.x;
    x[e] = v < a.v ? logit<BF16>(r.p, r.at + v) : -__builtin_inff();
    bad |= !(x[e] < __builtin_inff());
    m = fmaxf(m, x[e]);
  }
  m = group_max<64>(m);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) s_m[wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  const double it = 1.0 / a.temperature, ref = m == -__builtin_inff() ? 0.0 : (double)m;
  double z = 0.0;
#pragma unroll
  for (int e = 0; e < E; ++e) z += exp(((double)x[e] - ref) * it);
  if (bad) z = __builtin_nan("");
  z = wave_sum(z);
  if ((threadIdx.x & 63) == 0) s_z[wave] = z;
  __syncthreads();
  if (threadIdx.x == 0) st[(int64_t)blockIdx.x] = make_double2((double)m, (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]));
}

// A row's maximum and sum from its segments'; every lane of the wave has them.
__device__ __forceinline__ double2 row_stat(const double2 *st, int nseg, double it) {
  const int lane = threadIdx.x & 63;
  double m = kNegInf;
  for (int s = lane; s < nseg; s += 64) m = fmax(m, st[s].x);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmax(m, __shfl_xor(m, d, 64));
  const double ref = m == kNegInf ? 0.0 : m;
  double z = 0.0;
  for (int s = lane; s < nseg; s += 64) z += st[s].y * exp((st[s].x - ref) * it);
  return make_double2(ref, wave_sum(z));
}

// What is drawn from: p, or max(p - q, 0) with q of the draft's row or 1 at `token`.
struct Mass {
  RowOf t, d;
  double tm, tz, dm, dz, it;
  int64_t token;             // of a draft without probabilities, else -1
  bool minus;
  template <bool BF16>
  __device__ __forceinline__ double at(int64_t v) const {
    const double p = exp(((double)logit<BF16>(t.p, t.at + v) - tm) * it) / tz;
    if (!minus) return p;
    if (v == token) return 0.0;
    if (token >= 0) return p;
    return fmax(p - exp(((double)logit<BF16>(d.p, d.at + v) - dm) * it) / dz, 0.0);
  }
};

// Decided by every workgroup of a sequence for itself (its rows' statistics are a few KB).
struct Decision {
  Mass mass;
  int taken;
};
template <bool BF16>
__device__ __forceinline__ Decision decide(const DraftArgs &a, int64_t seq, const double2 *st, int nseg,
                                           double2 (&s_row)[2 * SLIM_DRAFT_MAX_K + 1]) {
  const int nr = a.draft ? 2 * a.k + 1 : a.k + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const double it = 1.0 / a.temperature;
  for (int j = wave; j < nr; j += 4) {
    const double2 r = row_stat(st + (seq * nr + j) * nseg, nseg, it);
    if (lane == 0) s_row[j] = r;
  }
  __syncthreads();
  bool good = false;
  if (lane < a.k) {
    const int64_t x = a.tokens[seq * a.k + lane];
    if (x >= 0 && x < a.v) {
      const RowOf t = row_of(a, seq, lane);
      const double2 ts = s_row[lane];
      const double p = exp(((double)logit<BF16>(t.p, t.at + x) - ts.x) * it) / ts.y;
      double q = 1.0;
      if (a.draft) {
        const RowOf d = row_of(a, seq, a.k + 1 + lane);
        const double2 ds = s_row[a.k + 1 + lane];
        q = exp(((double)logit<BF16>(d.p, d.at + x) - ds.x) * it) / ds.y;
      }
      good = (double)a.uniform[seq * (a.k + 1) + lane] * q < p;
    }
  }
  const uint64_t no = ~__ballot(good);
  Decision c;
  c.taken = no ? __ffsll((unsigned long long)no) - 1 : 64;
  if (c.taken > a.k) c.taken = a.k;
  const int j = c.taken;
  const int64_t x = j < a.k ? a.tokens[seq * a.k + j] : -1;
  Mass &m = c.mass;
  m.minus = x >= 0;
  m.token = m.minus && !a.draft ? x : -1;
  m.t = row_of(a, seq, j);
  m.tm = s_row[j].x, m.tz = s_row[j].y, m.it = it;
  m.d = m.t, m.dm = m.dz = 0.0;
  if (m.minus && a.draft) {
    m.d = row_of(a, seq, a.k + 1 + j);
    m.dm = s_row[a.k + 1 + j].x, m.dz = s_row[a.k + 1 + j].y;
  }
  return c;
}

template <bool BF16>
__global__ __launch_bounds__(256) void draft_mass_kernel(const DraftArgs a, const int nseg, const int64_t seg,
                                                         const double2 *__restrict__ st, double *__restrict__ mass) {
  __shared__ double2 s_row[2 * SLIM_DRAFT_MAX_K + 1];
  __shared__ double s_z[4];
  const int64_t seq = blockIdx.x / (unsigned)nseg;
  const int s = (int)(blockIdx.x % (unsigned)nseg);
  const Decision c = decide<BF16>(a, seq, st, nseg, s_row);
  const int64_t v0 = s * seg, v1 = v0 + seg < a.v ? v0 + seg : a.v;
  double z = 0.0;
  for (int64_t v = v0 + threadIdx.x; v < v1; v += 256) z += c.mass.template at<BF16>(v);
  z = wave_sum(z);
  if ((threadIdx.x & 63) == 0) s_z[threadIdx.x >> 6] = z;
  __syncthreads();
  if (threadIdx.x == 0) mass[blockIdx.x] = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
}

template <bool BF16>
__global__ __launch_bounds__(256) void draft_pick_kernel(const DraftArgs a, const int nseg, const int64_t seg,
                                                         const double2 *__restrict__ st,
                                                         const double *__restrict__ mass) {
  __shared__ double2 s_row[2 * SLIM_DRAFT_MAX_K + 1];
  __shared__ double s_z[4];
  __shared__ double s_left;
  __shared__ int s_seg;
  __shared__ unsigned long long s_hit, s_last;
  const int64_t seq = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Decision c = decide<BF16>(a, seq, st, nseg, s_row);
  const double *ms = mass + seq * nseg;
  if (tid == 0) {
    double all = 0.0;
    for (int s = 0; s < nseg; ++s) all += ms[s];
    const double want = (double)a.uniform[seq * (a.k + 1) + a.k] * all;
    double run = 0.0;
    int hit = -1, last = -1;
    double at = 0.0, lastat = 0.0;
    for (int s = 0; s < nseg; ++s) {
      if (ms[s] > 0.0) last = s, lastat = run;
      if (hit < 0 && run + ms[s] > want) hit = s, at = run;
      run += ms[s];
    }
    if (hit < 0) hit = last, at = lastat;
    s_seg = all > 0.0 ? hit : -1;       // NaN: a row without a distribution
    s_left = want - at;
    s_hit = s_last = ~0ull;
  }
  __syncthreads();
  int64_t pick = -1;
  const int hs = s_seg;
  if (hs >= 0) {
    const int64_t v0 = hs * seg, v1 = v0 + seg < a.v ? v0 + seg : a.v;
    const double left = s_left;
    double before = 0.0;
    for (int64_t b = v0; b < v1; b += 2048) {
      double x[8], sum = 0.0;
      int lastpos = -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t v = b + 8 * tid + e;
        x[e] = v < v1 ? c.mass.template at<BF16>(v) : 0.0;
        if (x[e] > 0.0) lastpos = e;
        sum += x[e];
      }
      double incl = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(incl, d, 64);
        if (lane >= d) incl += up;
      }
      if (lane == 63) s_z[wave] = incl;
      __syncthreads();
      double run = before + (incl - sum);
      for (int w = 0; w < wave; ++w) run += s_z[w];
      int hit = -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        run += x[e];
        if (hit < 0 && x[e] > 0.0 && run > left) hit = e;
      }
      if (hit >= 0) atomicMin(&s_hit, (unsigned long long)(b + 8 * tid + hit));
      if (lastpos >= 0) atomicMin(&s_last, ~0ull - 1 - (unsigned long long)(b + 8 * tid + lastpos));
      before += (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
      __syncthreads();
      if (s_hit != ~0ull) break;
    }
    // rounding can leave the segment's running sum just short of its mass: its last entry then
    pick = s_hit != ~0ull ? (int64_t)s_hit : s_last != ~0ull ? (int64_t)(~0ull - 1 - s_last) : -1;
  }
  if (tid <= a.k)
    a.ids[seq * (a.k + 1) + tid] = tid < c.taken ? a.tokens[seq * a.k + tid] : tid == c.taken ? pick : -1;
  if (tid == 0) a.accepted[seq] = c.taken;
}

template <bool BF16>
hipError_t launch(const DraftArgs &a, void *ws, const DraftPlan &p, hipStream_t st) {
  const int nr = a.draft ? 2 * a.k + 1 : a.k + 1;
  double2 *stat = (double2 *)ws;
  double *mass = (double *)(stat + a.b * nr * p.nseg);
  const unsigned rows = (unsigned)(a.b * nr * p.nseg);
  if (p.seg == 2048) draft_stats_kernel<BF16, 8><<<rows, 256, 0, st>>>(a, p.nseg, stat);
  else draft_stats_kernel<BF16, 32><<<rows, 256, 0, st>>>(a, p.nseg, stat);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  draft_mass_kernel<BF16><<<(unsigned)(a.b * p.nseg), 256, 0, st>>>(a, p.nseg, p.seg, stat, mass);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  draft_pick_kernel<BF16><<<(unsigned)a.b, 256, 0, st>>>(a, p.nseg, p.seg, stat, mass);
  return hipGetLastError();
}

}  // namespace

DraftPlan draft_plan(int64_t b, int k, int64_t v) {
  DraftPlan p;
  const int64_t rows = b * (2 * k + 1);
  p.seg = rows * ((v + 2047) / 2048) <= 1024 ? 2048 : 8192;   // few rows: more workgroups
  p.nseg = (int)((v + p.seg - 1) / p.seg);
  p.ws_bytes = (size_t)rows * p.nseg * 16 + (size_t)b * p.nseg * 8;
  return p;
}

hipError_t launch_verify_draft(const DraftArgs &a, void *ws, const DraftPlan &p, hipStream_t st) {
  return a.bf16 ? launch<true>(a, ws, p, st) : launch<false>(a, ws, p, st);
}

}  // namespace slim
