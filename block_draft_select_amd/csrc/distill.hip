// dflash_distill and dflash_distill_grad: the divergence of a student's row
// of logits from a teacher known by its K top logits, and its gradient.
//
// With x_j = s_j / tau, lse = log sum_j e^x_j, and the teacher's listed
// probabilities p_k = e^(t_k / tau - c) (c: the teacher's log-sum-exp over its
// whole vocabulary if given, else over the list),
//   D = sum_k p_k (log p_k - x_{i_k} + lse)
//     + p_rest (log p_rest - lse_rest + lse)     p_rest = 1 - sum p_k,
// where the second line (teacher's log-sum-exp given) treats all unlisted
// tokens as one class and lse_rest is their log-sum-exp.  It is summed over
// the unlisted tokens directly, never as total minus listed: a student that
// puts nearly everything on the list leaves a rest far below the total's
// rounding.  The gradient, with A = sum p + p_rest, is
//   dD/dx_j = A e^(x_j - lse) - p_j                      listed,
//           = e^(x_j - lse_rest) (A e^(lse_rest - lse) - p_rest)  unlisted,
// which stays finite for any gap between the two sums.
//
// distill_sum_kernel streams a row segment once into (maximum, sum);
// distill_loss_kernel, one block per row, joins the segments and the list.
// distill_grad_kernel recomputes the exponentials from lse (one read, one
// write), treats every token as unlisted, then rewrites the listed ones of its
// segment after a barrier.
//
// Sums are fp64: lse is returned in fp64 and the two passes must agree.
#include "rows_blocks.hpp"

namespace dfk {

namespace {

constexpr int kThreads = kDistillThreads;
constexpr int kWaves = kThreads / kWave;
constexpr double kLog2e64 = 1.4426950408889634;
constexpr double kLn2 = 0.6931471805599453;

// Where |x_j| log2 e reaches this, fp64 no longer holds lse beside x_j: a row
// that lies below (all of it the type's lowest value) is empty, a logit above
// counts as +inf
constexpr double kRange = 0x1p40;

// The forward pass sums 2^t, t = (x - m) log2 e, in fp64 for every logit, so its
// time is that of the instructions a term takes (16; fp64 and fp32 issue
// alike here).  With n = floor(512 t) and g the rest,
// 2^t = 2^(n >> 9) 2^((n & 511 + 1/2) / 512) e^v, v = (g - 1/2) ln 2 / 512: the middle
// factor comes from a table in LDS, the last from a parabola (the Taylor
// series with its third term spread over the first, v^3 ~ 3/4 h^2 v on
// |v| <= h = 6.8e-4: within 1.3e-11), the first is added to the table entry's
// exponent.  512 t is shifted by kShift so that truncation is the floor and
// everything below 2^-960 (and -inf) ends at the range's foot.  Measured on
// 2048 x 151936 against 64 entries and degree 3, over a few calls: 148 us to 160.
constexpr int kTabBits = 9, kTab = 1 << kTabBits;
constexpr double kShift = (double)kTab * 960.0;

// k0 + k1 g + k2 g^2 = e^v as above
constexpr double kL = 0.6931471805599453 / kTab;
constexpr double kU = -0.5 * kL;  // v at g = 0
constexpr double kA1 = 1.0 + kU * kU / 8.0;
constexpr double kP2 = 0.5 * kL * kL;
constexpr double kP1 = kL * (kA1 + kU);
constexpr double kP0 = 1.0 + kA1 * kU + 0.5 * kU * kU;

// entry k of the table: 2^((k + 1/2) / 512 - 960), by the Taylor series of e^x, |x| <= 0.3466, to degree 13
__device__ __forceinline__ double table_entry(int k) {
  const double x = ((double)k + 0.5 - 0.5 * kTab) * kL;
  double p = 1.0 / 6227020800.0;
  p = fma(p, x, 1.0 / 479001600.0);
  p = fma(p, x, 1.0 / 39916800.0);
  p = fma(p, x, 1.0 / 3628800.0);
  p = fma(p, x, 1.0 / 362880.0);
  p = fma(p, x, 1.0 / 40320.0);
  p = fma(p, x, 1.0 / 5040.0);
  p = fma(p, x, 1.0 / 720.0);
  p = fma(p, x, 1.0 / 120.0);
  p = fma(p, x, 1.0 / 24.0);
  p = fma(p, x, 1.0 / 6.0);
  p = fma(p, x, 0.5);
  p = fma(p, x, 1.0);
  p = fma(p, x, 1.0);
  return ldexp(p * 1.4142135623730951, -960);
}

// adds 2^(ts / 512 - 960) to the sum (ts = 512 t + kShift).  exp_unit is 2^20, an
// exponent's last bit in the upper word; it is a kernel argument because the
// compiler turns the product with a constant back into a shift, a mask and an
// addition (one instruction of 17 more, 8 per cent)
__device__ __forceinline__ double add_term(double sum, double ts, const double* tab, uint32_t exp_unit) {
  ts = fmax(ts, 0.0);
  const uint32_t n = (uint32_t)ts;
  const double g = __builtin_amdgcn_fract(ts);
  const double e = tab[n & (uint32_t)(kTab - 1)];
  const double f = __hiloint2double((int)(__umul24(n >> kTabBits, exp_unit) + (uint32_t)__double2hiint(e)), __double2loint(e));
  return fma(f, fma(fma(g, kP2, kP1), g, kP0), sum);
}

struct Red {
  double d[kWaves];
};

// over the block's T threads
template <int T>
__device__ __forceinline__ double block_sum(Red& s, double v) {
  v = wave_sum_dpp_f64(v);
  if constexpr (T > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.d[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.d[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v += s.d[w];
  }
  return v;
}

template <int T>
__device__ __forceinline__ double block_max(Red& s, double v) {
  v = fmax(v, dpp_f64<kDppRowShr1>(v, -INFINITY));
  v = fmax(v, dpp_f64<kDppRowShr2>(v, -INFINITY));
  v = fmax(v, dpp_f64<kDppRowShr4>(v, -INFINITY));
  v = fmax(v, dpp_f64<kDppRowShr8>(v, -INFINITY));
  v = fmax(v, dpp_f64<kDppRowBcast15, 0xA>(v, -INFINITY));
  v = fmax(v, dpp_f64<kDppRowBcast31, 0xC>(v, -INFINITY));
  v = readlane_f64(v, 63);
  if constexpr (T > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s.d[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.d[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v = fmax(v, s.d[w]);
  }
  return v;
}

// a list entry counts unless its index lies outside the vocabulary (padding)
__device__ __forceinline__ bool listed(const DistillArgs& a, int64_t row, int k, int& idx) {
  idx = a.t_idx[row * a.K + k];
  return idx >= 0 && idx < a.V;
}

// t_k / tau of a list entry; +inf is no logit: NaN
__device__ __forceinline__ double scaled(const DistillArgs& a, int64_t row, int k) {
  const float t = a.t_logit[row * a.K + k];
  return t < INFINITY ? (double)t / a.tau : (double)NAN;
}

// the largest t_k / tau of a list: -inf if it lies below the range, NaN above it
__device__ __forceinline__ double in_range(double m) {
  return m <= -kRange * kLn2 ? -INFINITY : m < kRange * kLn2 ? m : (double)NAN;
}

// the teacher's normaliser c (natural log); -inf: the teacher's row is empty
template <int T>
__device__ __forceinline__ double teacher_lse(Red& red, const DistillArgs& a, int64_t row) {
  if (a.t_lse) {
    const double c = a.t_lse[row];
    return c < INFINITY ? c : (c != c ? c : -INFINITY);
  }
  double m = -INFINITY;
  int idx;
  for (int k = threadIdx.x; k < a.K; k += T)
    if (listed(a, row, k, idx)) {
      const double t = scaled(a, row, k);
      m = t != t ? INFINITY : fmax(m, t);
    }
  m = in_range(block_max<T>(red, m));
  if (!(fabs(m) < INFINITY)) return m;
  double s = 0.0;
  for (int k = threadIdx.x; k < a.K; k += T)
    if (listed(a, row, k, idx)) s += exp(scaled(a, row, k) - m);
  return m + log(block_sum<T>(red, s));
}

// ---------------------------------------------------------------- forward

// a thread's largest logit; whether one is NaN or +inf
template <int DT, int N>
__device__ __forceinline__ float largest(const Slot (&x)[N], bool& odd) {
  float m = kNegInf;
  odd = false;
  if constexpr (DT == DFLASH_BF16) {
    // signed and unsigned maxima of the raw patterns, two a word: the signed one
    // is the largest logit unless all are negative (then the unsigned minimum
    // is), and a NaN of either sign stands over its infinity
    uint32_t hi = 0x80008000u, up = 0;
#pragma unroll
    for (int l = 0; l < N; ++l)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        hi = smax_i16x2(hi, x[l].w[d]);
        up = max_u16x2(up, x[l].w[d]);
      }
    const int h = max((int)(int16_t)(hi & 0xFFFFu), (int)(int16_t)(hi >> 16));
    odd = h >= 0x7F80 || max(up & 0xFFFFu, up >> 16) > 0xFF80u;
    uint32_t best = (uint32_t)h;
    if (h < 0) {
      uint32_t lo = 0xFFFFFFFFu;
#pragma unroll
      for (int l = 0; l < N; ++l)
#pragma unroll
        for (int d = 0; d < 4; ++d) lo = min_u16x2(lo, x[l].w[d]);
      best = min(lo & 0xFFFFu, lo >> 16);
    }
    m = __uint_as_float(best << 16);
  } else {
#pragma unroll
    for (int l = 0; l < N; ++l)
#pragma unroll
      for (int i = 0; i < RowType<DT>::VE; ++i) {
        const float v = slot_value<DT>(x[l], i);
        m = fmaxf(m, v);
        odd |= !(v < INFINITY);
      }
  }
  return m;
}

// A block sums a row segment of `units` times kDistillUnit slots; each of its
// waves on its own, four slots a lane at a time, relative to the largest logit
// so far (rounded to a power of two, so that a new one only moves exponents).
// 2048 x 151936 bf16: 154 us at best, 4.0 TB/s; 166 at the median of 24 calls.
template <int DT, bool REST>
__global__ __launch_bounds__(kThreads) void distill_sum_kernel(DistillArgs a, int n_seg, int units, uint32_t exp_unit,
                                                               DistillPart* __restrict__ parts) {
  constexpr int VE = RowType<DT>::VE, U = kDistillUnit / kThreads;
  __shared__ double tab[kTab];
  __shared__ double wave_m[kWaves], wave_s[kWaves];
  __shared__ uint32_t mask[REST ? kDistillMaxUnits * kDistillUnit * VE / 32 : 1];
  const int tid = threadIdx.x, seg = blockIdx.x % n_seg;
  const int64_t row = blockIdx.x / n_seg;
  if (a.weight && a.weight[row] == 0.0f) return;
  const RowRef<DT> z(a.S, row, a.stride, a.V);
  const int s0 = seg * units * kDistillUnit, s1 = min(s0 + units * kDistillUnit, z.slots());
  for (int i = tid; i < kTab; i += kThreads) tab[i] = table_entry(i);
  if constexpr (REST) {
    for (int i = tid; i < units * kDistillUnit * VE / 32; i += kThreads) mask[i] = 0;
    __syncthreads();
    const int e0 = s0 * VE, e1 = s1 * VE;
    int idx;
    for (int k = tid; k < a.K; k += kThreads)
      if (listed(a, row, k, idx) && idx >= e0 && idx < e1) atomicOr(&mask[(idx - e0) >> 5], 1u << ((idx - e0) & 31));
  }
  __syncthreads();
  const double c = kLog2e64 / a.tau;
  double M = -INFINITY, s = 0.0;
  bool any_odd = false;
#pragma unroll 1
  for (int u0 = s0; u0 < s1; u0 += kDistillUnit) {
    Slot x[U];
#pragma unroll
    for (int l = 0; l < U; ++l) x[l] = z.template load<true>(min(u0 + l * kThreads + tid, z.slots()));
    if constexpr (REST) {
#pragma unroll
      for (int l = 0; l < U; ++l) {  // listed tokens leave the sums
        const int bit = (u0 - s0 + l * kThreads + tid) * VE;
        const uint32_t mk = (mask[bit >> 5] >> (bit & 31)) & ((1u << VE) - 1u);
        if (mk) {
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if ((mk >> i) & 1u) {
              if constexpr (DT == DFLASH_BF16)
                x[l].w[i >> 1] = (i & 1) ? (x[l].w[i >> 1] & 0x0000FFFFu) | 0xFF800000u : (x[l].w[i >> 1] & 0xFFFF0000u) | 0x0000FF80u;
              else
                x[l].w[i] = 0xFF800000u;
            }
        }
      }
    }
    bool odd;
    const float m = wave_max_dpp_f32(largest<DT>(x, odd));
    const double Mu = rint((double)m * c);
    any_odd |= __ballot(odd) != 0 || Mu >= kRange;
    if (Mu > M && fabs(Mu) < kRange) {
      s = M > -INFINITY ? ldexp(s, (int)fmax(M - Mu, -4000.0)) : 0.0;
      M = Mu;
    }
    if (M > -INFINITY) {
      const double ct = (double)kTab * c, off = kShift - (double)kTab * M;
#pragma unroll
      for (int l = 0; l < U; ++l)
#pragma unroll
        for (int i = 0; i < VE; ++i) s = add_term(s, fma((double)slot_value<DT>(x[l], i), ct, off), tab, exp_unit);
    }
  }
  s = wave_sum_dpp_f64(s);
  if ((tid & 63) == 0) {
    wave_m[tid >> 6] = any_odd ? INFINITY : M;
    wave_s[tid >> 6] = s;
  }
  __syncthreads();
  if (tid == 0) {
    double BM = wave_m[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) BM = fmax(BM, wave_m[w]);
    double sum = 0.0;
    if (BM == INFINITY) {
      sum = NAN;
    } else {
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        if (wave_m[w] > -INFINITY) sum += ldexp(wave_s[w], (int)fmax(wave_m[w] - BM, -4000.0));
    }
    parts[blockIdx.x] = DistillPart{BM, sum};
  }
}

// log-sum-exp (natural) of terms s * 2^m
__device__ __forceinline__ double join_log(double m, double s) {
  if (s == 0.0) return -INFINITY;
  return (m + log2(s)) * kLn2;
}

// T threads a row: a wave for short lists (no barriers; 2048 rows of K = 16 in
// 10 us, 15 with a block each), a block for long ones, whose repeated entries
// are searched for pair by pair
template <int DT, int T, bool REST>
__global__ __launch_bounds__(T) void distill_loss_kernel(DistillArgs a, int n_seg, const DistillPart* __restrict__ parts,
                                                                float* __restrict__ loss, double* __restrict__ lse_out,
                                                                double* __restrict__ rest_out) {
  __shared__ Red red;
  __shared__ int seen[DFLASH_DISTILL_K_MAX];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float w = a.weight ? a.weight[row] : 1.0f;
  if (w == 0.0f) {
    if (tid == 0) {
      if (loss) loss[row] = 0.0f;
      lse_out[row] = 0.0;
      if (REST) rest_out[row] = 0.0;
    }
    return;
  }
  const RowRef<DT> z(a.S, row, a.stride, a.V);
  const double c2 = kLog2e64 / a.tau;
  const double c = teacher_lse<T>(red, a, row);

  // the segments' sums: maxima first, then the terms in segment order
  const DistillPart* part = parts + row * n_seg;
  double M = -INFINITY;
  for (int g = tid; g < n_seg; g += T)
    if (part[g].s != 0.0) M = fmax(M, part[g].m);
  M = block_max<T>(red, M);
  double s = 0.0;
  for (int g = tid; g < n_seg; g += T)
    if (part[g].s != 0.0) s += part[g].s == part[g].s ? ldexp(part[g].s, (int)fmax(part[g].m - M, -4000.0)) : (double)NAN;
  s = block_sum<T>(red, s);
  const double rest = join_log(M, s);  // natural
  double lse = rest;

  if constexpr (REST) {
    // the listed tokens' own terms, each token once
    for (int k = tid; k < a.K; k += T) {
      int idx;
      seen[k] = listed(a, row, k, idx) ? idx : -1;
    }
    __syncthreads();
    double lm = -INFINITY;
    for (int k = tid; k < a.K; k += T) {
      const int idx = seen[k];
      bool first = idx >= 0;
      for (int q = 0; q < k && first; ++q) first = seen[q] != idx;
      if (first) {
        const float v = row_value<DT>(z, idx);
        lm = v != v ? INFINITY : fmax(lm, (double)v);
      }
    }
    lm = block_max<T>(red, lm);
    const double LM = rint(lm * c2);
    if (LM > -kRange) {
      double ls = 0.0;
      for (int k = tid; k < a.K; k += T) {
        const int idx = seen[k];
        bool first = idx >= 0;
        for (int q = 0; q < k && first; ++q) first = seen[q] != idx;
        if (first) {
          const float v = row_value<DT>(z, idx);
          if (v != kNegInf) ls += LM < kRange ? exp2(fma((double)v, c2, -LM)) : (double)NAN;
        }
      }
      ls = block_sum<T>(red, ls);
      const double top = s > 0.0 ? fmax(M, LM) : LM;
      const double all = (s == 0.0 ? 0.0 : ldexp(s, (int)fmax(M - top, -4000.0))) + ldexp(ls, (int)fmax(LM - top, -4000.0));
      lse = s != s ? s : join_log(top, all);
    }
  }

  // D over the listed entries
  double d = 0.0, p_sum = 0.0;
  if (c > -INFINITY || c != c)
    for (int k = tid; k < a.K; k += T) {
      int idx;
      if (!listed(a, row, k, idx)) continue;
      const double logp = scaled(a, row, k) - c;
      const double p = exp(logp);
      p_sum += p;
      if (p != 0.0) d += p * (logp - (double)row_value<DT>(z, idx) / a.tau + lse);
    }
  d = block_sum<T>(red, d);
  p_sum = block_sum<T>(red, p_sum);
  if constexpr (REST) {
    const double p_rest = 1.0 - p_sum;
    if (c > -INFINITY && rest > -INFINITY && p_rest > 0.0) d += p_rest * (log(p_rest) - rest + lse);
    if (rest != rest) d = rest;
  }
  if (c == -INFINITY || lse == -INFINITY) d = 0.0;  // an empty row on either side
  if (tid == 0) {
    if (loss) loss[row] = (float)((double)w * d);
    lse_out[row] = lse;
    if (REST) rest_out[row] = rest;
  }
}

// ---------------------------------------------------------------- backward

// One read and one write of the row at the memory's rate: 2048 x 151936 bf16 in
// 213 to 218 us, 5.8 TB/s (torch's copy of 2 GiB: 4.9).  The exponentials are fp32,
// the exponent in two pieces (off by (|t| + 4) 2^-23, and by the low pieces'
// roundings, 2^-43 |x_j|): the forward pass's fp64 terms alone take 154 us.
template <int DT, int NL, bool REST>
__global__ __launch_bounds__(kThreads) void distill_grad_kernel(DistillArgs a, int n_seg, const float* __restrict__ grad_loss,
                                                                const double* __restrict__ lse_in,
                                                                const double* __restrict__ rest_in, void* dS,
                                                                int64_t d_stride) {
  using E = typename RowType<DT>::elem;
  constexpr int VE = RowType<DT>::VE;
  constexpr int kPerThread = DFLASH_DISTILL_K_MAX / kThreads;
  __shared__ Red red;
  __shared__ int seen[DFLASH_DISTILL_K_MAX];
  __shared__ double prob[DFLASH_DISTILL_K_MAX];
  const int tid = threadIdx.x, seg = blockIdx.x % n_seg;
  const int64_t row = blockIdx.x / n_seg;
  const RowRef<DT> z(a.S, row, a.stride, a.V);
  E* o = static_cast<E*>(dS) + row * d_stride;
  const int s0 = seg * (kThreads * NL), e0 = s0 * VE, e1 = e0 + kThreads * NL * VE;
  double f = (a.weight ? (double)a.weight[row] : 1.0) * (grad_loss ? (double)grad_loss[row] : 1.0);
  const bool off = (a.weight && a.weight[row] == 0.0f) || (grad_loss && grad_loss[row] == 0.0f);
  f /= a.tau;
  const double lse = off ? 0.0 : lse_in[row];
  const double rest = REST && !off ? rest_in[row] : 0.0;

  Slot x[NL];
  if (!off) {
#pragma unroll
    for (int l = 0; l < NL; ++l) x[l] = z.template load<true>(s0 + l * kThreads + tid);
  }
  double c = -INFINITY, p_sum = 0.0;
  float own[kPerThread];  // the listed tokens' logits of this segment, read before anything is stored (dS may be S)
  if (!off && a.K <= kWave) {
    // a short list: one wave, one barrier (61 x 50021 fp32, K = 64: 11.8 us, 13.3
    // with the block's reductions)
    if (tid < kWave) {
      int idx = -1;
      const bool in = tid < a.K && listed(a, row, tid, idx);
      const double t = in ? scaled(a, row, tid) : -INFINITY;
      double p;
      if (a.t_lse) {
        c = teacher_lse<kWave>(red, a, row);
        p = in && c != -INFINITY ? exp(t - c) : 0.0;
      } else {
        c = in_range(block_max<kWave>(red, t != t ? INFINITY : t));
        const double e = in && c != -INFINITY ? exp(t - c) : 0.0;
        const double all = block_sum<kWave>(red, e);
        p = in ? e / all : 0.0;
      }
      if (tid < a.K) {
        seen[tid] = in ? idx : -1;
        prob[tid] = p;
      }
      if (in && idx >= e0 && idx < e1) own[0] = row_value<DT>(z, idx);
      p_sum = block_sum<kWave>(red, p);
      if (tid == 0) {
        red.d[0] = p_sum;
        red.d[1] = c;
      }
    }
    __syncthreads();
    p_sum = red.d[0];
    c = red.d[1];
  } else if (!off) {
    c = teacher_lse<kThreads>(red, a, row);
    if (c != -INFINITY) {
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        const int k = j * kThreads + tid;
        if (k < a.K) {
          int idx;
          const bool in = listed(a, row, k, idx);
          const double p = in ? exp(scaled(a, row, k) - c) : 0.0;
          p_sum += p;
          seen[k] = in ? idx : -1;
          prob[k] = p;
          if (in && idx >= e0 && idx < e1) own[j] = row_value<DT>(z, idx);
        }
      }
    }
    p_sum = block_sum<kThreads>(red, p_sum);
  }
  if (off || c == -INFINITY || lse == -INFINITY) {  // no gradient: weight zero, or an empty row on either side
#pragma unroll
    for (int l = 0; l < NL; ++l) store_slot<DT>(o, a.V, s0 + l * kThreads + tid, Slot{{0, 0, 0, 0}});
    return;
  }
  const bool with_rest = REST && rest != -INFINITY;
  const double p_rest = with_rest ? fmax(1.0 - p_sum, 0.0) : 0.0;
  const double A = p_sum + p_rest;
  const double base = with_rest ? rest : lse;
  double G64 = f * (with_rest ? A * exp(rest - lse) - p_rest : A);
  const double c2 = kLog2e64 / a.tau;
  double b2 = base * kLog2e64;
  // a factor near fp32's end leaves its power of two to the exponent, so that
  // unlikely tokens' gradients, which fit, do not become inf times 0
  if (fabs(G64) >= 0x1p100 && fabs(G64) < INFINITY) {
    const int up = ilogb(G64);
    G64 = ldexp(G64, -up);
    b2 -= up;
  }
  const float G = (float)G64;
  // x_j - base in two pieces of fp32: the product s c and its difference from
  // the base are rounded once (fma), the low halves are added after.  Those stay
  // finite: logits whose exponential is 0 are raised there to 2^-256 of the base's
  // (or below, by as much as rounding moves the border), else a mask of finite
  // lowest values over a small tau would leave fp32 in both pieces, with either sign
  const float ch = (float)c2, cl = (float)(c2 - (double)ch), bh = (float)b2, bl = (float)(b2 - (double)bh);
  const float least = (float)fmax((b2 - 256.0 - fabs(b2) * 0x1p-22) * kLn2 * a.tau, -3.4028234663852886e38);
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    Slot y;
#pragma unroll
    for (int k = 0; k < 4; ++k) y.w[k] = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float v = slot_value<DT>(x[l], i);
      const float t = fmaf(v, ch, -bh) + fmaf(fmaxf(v, least), cl, -bl);
      const float g = G * __builtin_amdgcn_exp2f(t);  // -inf: 0
      if constexpr (DT == DFLASH_BF16)
        y.w[i >> 1] |= bf16_round(g) << ((i & 1) * 16);
      else
        y.w[i] = __float_as_uint(g);
    }
    store_slot<DT>(o, a.V, s0 + l * kThreads + tid, y);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int k = j * kThreads + tid;
    if (k < a.K && seen[k] >= e0 && seen[k] < e1) {
      double p = 0.0;  // every entry of this token, in list order
      for (int q = 0; q < a.K; ++q)
        if (seen[q] == seen[k]) p += prob[q];
      const double sm = own[j] == kNegInf ? 0.0 : exp((double)own[j] / a.tau - lse);
      o[seen[k]] = to_elem<DT>((float)(f * (A * sm - p)));
    }
  }
}

template <int DT, bool REST>
hipError_t run_forward(const DistillArgs& a, float* loss, double* lse, double* rest, char* ws, const DistillPlan& pl,
                       hipStream_t st) {
  DistillPart* parts = reinterpret_cast<DistillPart*>(ws);
  const dim3 rows((unsigned)a.R);
  launch(distill_sum_kernel<DT, REST>, dim3((unsigned)(a.R * pl.n_seg)), dim3(kThreads), st, a, pl.n_seg, pl.units, 0x100000u,
         parts);
  if (a.K <= 128)
    launch(distill_loss_kernel<DT, 64, REST>, rows, dim3(64), st, a, pl.n_seg, (const DistillPart*)parts, loss, lse, rest);
  else
    launch(distill_loss_kernel<DT, kThreads, REST>, rows, dim3(kThreads), st, a, pl.n_seg, (const DistillPart*)parts, loss, lse,
           rest);
  return hipGetLastError();
}

template <int DT, int NL>
hipError_t run_grad(const DistillArgs& a, const float* grad_loss, const double* lse, const double* rest, void* dS,
                    int64_t d_stride, const DistillPlan& pl, hipStream_t st) {
  const dim3 grid((unsigned)(a.R * pl.grad_seg)), block(kThreads);
  if (rest)
    launch(distill_grad_kernel<DT, NL, true>, grid, block, st, a, pl.grad_seg, grad_loss, lse, rest, dS, d_stride);
  else
    launch(distill_grad_kernel<DT, NL, false>, grid, block, st, a, pl.grad_seg, grad_loss, lse, rest, dS, d_stride);
  return hipGetLastError();
}

template <int DT>
hipError_t run_grad_typed(const DistillArgs& a, const float* grad_loss, const double* lse, const double* rest, void* dS,
                          int64_t d_stride, const DistillPlan& pl, hipStream_t st) {
  switch (pl.grad_loads) {
    case 1: return run_grad<DT, 1>(a, grad_loss, lse, rest, dS, d_stride, pl, st);
    case 2: return run_grad<DT, 2>(a, grad_loss, lse, rest, dS, d_stride, pl, st);
    case 4: return run_grad<DT, 4>(a, grad_loss, lse, rest, dS, d_stride, pl, st);
    default: return run_grad<DT, 8>(a, grad_loss, lse, rest, dS, d_stride, pl, st);
  }
}

}  // namespace

hipError_t launch_distill(int32_t dtype, const DistillArgs& a, float* loss, double* lse, double* rest, char* ws,
                          const DistillPlan& pl, hipStream_t st) {
  if (dtype == DFLASH_BF16)
    return rest ? run_forward<DFLASH_BF16, true>(a, loss, lse, rest, ws, pl, st)
                : run_forward<DFLASH_BF16, false>(a, loss, lse, rest, ws, pl, st);
  return rest ? run_forward<DFLASH_F32, true>(a, loss, lse, rest, ws, pl, st)
              : run_forward<DFLASH_F32, false>(a, loss, lse, rest, ws, pl, st);
}

hipError_t launch_distill_grad(int32_t dtype, const DistillArgs& a, const float* grad_loss, const double* lse,
                               const double* rest, void* dS, int64_t d_stride, const DistillPlan& pl, hipStream_t st) {
  if (dtype == DFLASH_BF16) return run_grad_typed<DFLASH_BF16>(a, grad_loss, lse, rest, dS, d_stride, pl, st);
  return run_grad_typed<DFLASH_F32>(a, grad_loss, lse, rest, dS, d_stride, pl, st);
}

}  // namespace dfk
