// dflash_sample and dflash_filter: rows of logits under temperature, top-k,
// top-p and min-p.
//
// With w_i = exp((z_i - max z) / T), the tokens of a row ordered by (z
// descending, index ascending) and W(n) the sum of the first n weights, every
// filter keeps a prefix of that order: top-k the first k, top-p the first n
// with W(n) >= top_p W(k), min-p those with w_i >= min_p.  The kept tokens are
// the shortest of the three, and a token is drawn by inverting W at
// u W(kept) along the same order.  So a cut and a draw are the same question:
// at which token does a running count or sum cross a value.
//
// It is answered without sorting the row.  In units of an eighth of an octave
// a weight is 2^(t / 8), t = z 8 log2(e) / T, and floor(t) bins the tokens in
// their order: (1) sample_hist_kernel counts the tokens and sums the weights
// of each bin of a row segment; (2) sample_finalize_kernel, one block per
// row, adds the segments' bins, scans them, finds the bin of the crossing
// and gathers and sorts that bin's tokens alone, from the row.  A bin of more tokens
// than the list holds is split again by key ranges first; if one value alone
// has that many tokens, its tokens share one weight and the crossing is a
// division.  (3) sample_apply_kernel (dflash_filter) copies the kept tokens.
//
// Counts are exact and sums do not depend on the order of the atomics: a bin
// adds the mantissas of 2^frac(t / 8) as 64-bit integers (the fraction bits of
// a double in [1, 1.0906) stay below 2^48.6, so 32768 of them fit), which keeps
// 52 bits below each token's own weight.  Decisions next to a border need
// such sums: they compare running sums over the whole vocabulary.
#include "rows_blocks.hpp"

// t = z c8 is one rounded product wherever it is formed: fused into the
// subtraction of its own floor it would differ from the value that was binned
#pragma clang fp contract(off)

namespace dfk {

namespace {

constexpr int kThreads = kSampleThreads;
constexpr int kWaves = kThreads / kWave;
constexpr int kBins = kSampleBins;  // 64 octaves; the last bin collects everything below (weight under 2^-63.9)
constexpr int kTail = kBins - 1;
constexpr int kCols = 4;            // copies of the bins a wave's lanes spread over
constexpr int kCap = 4096;          // tokens the sorted list holds
constexpr int kPer = kCap / kThreads;
static_assert(kThreads == kBins, "one thread per bin");

constexpr uint32_t kKeyLowest = 0x00800000u;  // ordered key of the lowest finite fp32
constexpr uint64_t kOneBits = 0x3FF0000000000000ull;

constexpr double kLn2Eighth = 0.08664339756999316;  // ln 2 / 8

// 2^(f / 8) for f in [0, 1): Taylor series to degree 8, truncation below
// 8e-16; exactly 1 at f = 0 and never below 1
__device__ __forceinline__ double exp2_eighth(double f) {
  const double x = f * kLn2Eighth;
  double p = 1.0 / 40320.0;
  p = fma(p, x, 1.0 / 5040.0);
  p = fma(p, x, 1.0 / 720.0);
  p = fma(p, x, 1.0 / 120.0);
  p = fma(p, x, 1.0 / 24.0);
  p = fma(p, x, 1.0 / 6.0);
  p = fma(p, x, 0.5);
  p = fma(p, x, 1.0);
  return fma(p, x, 1.0);
}

// 2^(e / 8), e <= 0 an integer
__device__ __forceinline__ double pow2_eighth(int e) {
  const int r = e & 7;
  double v = (r & 4) ? 1.4142135623730951 : 1.0;
  v *= (r & 2) ? 1.189207115002721 : 1.0;
  v *= (r & 1) ? 1.0905077326652577 : 1.0;
  return ldexp(v, e >> 3);
}

struct RowParams {
  double c8;  // 8 log2(e) / T
  int64_t k;  // top-k; INT64_MAX: off
  double p;   // top-p; >= 1: off
  double m;   // min-p; <= 0: off
};

__device__ __forceinline__ RowParams row_params(const SampleArgs& a, int64_t row) {
  const int64_t g = row / a.group;
  const float T = a.T ? a.T[g] : 1.0f;
  const bool greedy = !(T > 0.0f);
  RowParams r;
  r.c8 = 8.0 * 1.4426950408889634 / (greedy ? 1.0 : (double)T);
  const int32_t k = a.top_k ? a.top_k[g] : 0;
  r.k = greedy ? 1 : (k > 0 ? (int64_t)k : INT64_MAX);
  const float p = a.top_p ? a.top_p[g] : 1.0f;
  r.p = !greedy && p < 1.0f ? fmax((double)p, 0.0) : 1.0;
  const float m = a.min_p ? a.min_p[g] : 0.0f;
  r.m = !greedy && m > 0.0f ? fmin((double)m, 1.0) : 0.0;
  return r;
}

// ---------------------------------------------------------------- block helpers (kThreads threads)

struct Red {
  double d[kWaves];
  uint32_t u[kWaves];
  int first;
};

// smallest thread index whose predicate holds (kThreads if none)
__device__ __forceinline__ int block_first(Red& s, bool pred) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) s.first = kThreads;
  __syncthreads();
  const int f = first_lane(pred);
  if ((tid & 63) == 0 && f < 64) atomicMin(&s.first, tid + f);
  __syncthreads();
  return s.first;
}

__device__ __forceinline__ int block_min(Red& s, int v) {
  const int tid = threadIdx.x;
  v = wave_min_i32(v);
  __syncthreads();
  if (tid == 0) s.first = 0x7FFFFFFF;
  __syncthreads();
  if ((tid & 63) == 0) atomicMin(&s.first, v);
  __syncthreads();
  return s.first;
}

__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t v) {
  const int lane = lane_id();
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const uint32_t w = __shfl_up(v, o);
    v += lane >= o ? w : 0u;
  }
  return v;
}

// inclusive scans over the block, in fixed order
__device__ __forceinline__ uint32_t block_scan_u32(Red& s, uint32_t v) {
  const int w = threadIdx.x >> 6;
  v = wave_scan_u32(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.u[w] = v;
  __syncthreads();
  uint32_t off = 0;
  for (int i = 0; i < w; ++i) off += s.u[i];
  return v + off;
}

__device__ __forceinline__ double block_scan_f64(Red& s, double v) {
  const int w = threadIdx.x >> 6;
  v = wave_scan_f64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.d[w] = v;
  __syncthreads();
  double off = 0.0;
  for (int i = 0; i < w; ++i) off += s.d[i];
  return v + off;
}

// ---------------------------------------------------------------- (1) bins of a segment

template <int DT, int NL>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(SampleArgs a, int64_t row0, int n_seg,
                                                               SamplePart* __restrict__ parts) {
  constexpr int VE = RowType<DT>::VE;
  __shared__ uint64_t mass[kBins * kCols];
  __shared__ uint32_t cnt[kBins * kCols];
  __shared__ float wmax[kWaves];
  __shared__ Red red;
  const int tid = threadIdx.x, seg = blockIdx.x % n_seg;
  const int64_t row = row0 + blockIdx.x / n_seg;
  const RowRef<DT> z(a.Z, row, a.stride, a.V);
  const double c8 = row_params(a, row).c8;

  Slot x[NL];
  const int s0 = seg * (kThreads * NL) + tid;
#pragma unroll
  for (int l = 0; l < NL; ++l) x[l] = z.template load<true>(s0 + l * kThreads);

#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    mass[c * kBins + tid] = 0;
    cnt[c * kBins + tid] = 0;
  }
  float m = kNegInf;
#pragma unroll
  for (int l = 0; l < NL; ++l)
#pragma unroll
    for (int i = 0; i < VE; ++i) m = fmaxf(m, slot_value<DT>(x[l], i));  // NaN drops out
  m = wave_max_f32(fminf(m, RowType<DT>::kMax));
  if ((tid & 63) == 0) wmax[tid >> 6] = m;
  __syncthreads();
  m = wmax[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, wmax[w]);

  SamplePart& out = parts[blockIdx.x];
  if (m == kNegInf) {
    if (tid == 0) {
      out.J = -INFINITY;
      out.max = kNegInf;
      out.n = 0;
      out.nb = 0;
    }
    return;
  }
  const double J = floor((double)m * c8);
  const int col = tid & (kCols - 1);
#pragma unroll
  for (int l = 0; l < NL; ++l)
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float v = slot_value<DT>(x[l], i);
      if (v > kNegInf) {
        const double t = (double)fminf(v, RowType<DT>::kMax) * c8, fl = floor(t);
        const int b = (int)fmin(J - fl, (double)kTail);
        atomicAdd(&cnt[b * kCols + col], 1u);
        if (b < kTail)
          atomicAdd((unsigned long long*)&mass[b * kCols + col], (unsigned long long)__double_as_longlong(exp2_eighth(t - fl)));
      }
    }
  __syncthreads();
  uint32_t c = 0;
  uint64_t f = 0;
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    c += cnt[tid * kCols + k];
    f += mass[tid * kCols + k];
  }
  f -= (uint64_t)c * kOneBits;  // modulo 2^64: the fraction bits' sum
  const uint32_t n = block_scan_u32(red, c);
  uint32_t mirror = 0;  // the bin counted from the far end: the bins in use end where the first of these is not empty
#pragma unroll
  for (int k = 0; k < kCols; ++k) mirror += cnt[(kBins - 1 - tid) * kCols + k];
  const int nb = kBins - block_first(red, mirror != 0);
  if (tid < nb) {
    out.cnt[tid] = c;
    out.mass[tid] = tid < kTail ? (double)c + (double)f * 0x1p-52 : 0.0;
  }
  if (tid == kThreads - 1) {
    out.J = J;
    out.max = m;
    out.n = n;
    out.nb = nb;
  }
}

// ---------------------------------------------------------------- (2) cuts and draw of a row

enum { kByCount, kByMassGe, kByMassGt, kByWeight };

struct FinLds {
  uint64_t comp[kCap];    // the list: (~key, index), ascending = the row's order
  uint64_t mass[kBins];   // bins of a split
  uint32_t cnt[kBins];
  uint32_t cc[kBins + 1];  // tokens before each bin
  double cm[kBins + 1];    // their weight
  uint32_t rc[kBins + 1];  // the same inside a split
  double rm[kBins + 1];
  Red red;
  uint32_t n_list;
  double cum;
  uint64_t at;
};

// where a running count or sum crosses a value
struct Cross {
  uint32_t n;    // tokens up to and including the crossing one (kByWeight: tokens that pass)
  double cum;    // their weight
  uint64_t cut;  // a token is among them iff its (~key, index) is below this
  uint64_t at;   // (~key, index) of the last of them (not for kByWeight)
};

template <int DT>
struct Finalize {
  static constexpr int VE = RowType<DT>::VE;
  FinLds& s;
  const RowRef<DT> z;
  const double c8, J;
  const int tid;
  const uint32_t kmax;  // the row's largest key
  // the list's tokens: rank base + 1 .. base + n, of bins b0 .. b1 (b0 > b1: part of a bin)
  uint32_t base, n;
  double bmass;
  int b0, b1;
  uint32_t lo;
  double cum[kPer];

  __device__ Finalize(FinLds& s_, const RowRef<DT>& z_, double c8_, double J_, uint32_t kmax_)
      : s(s_), z(z_), c8(c8_), J(J_), tid(threadIdx.x), kmax(kmax_), base(0), n(0), bmass(0.0), b0(1), b1(0), lo(0) {}

  // weight of a key relative to 2^(J / 8)
  __device__ double weight(uint32_t key) const {
    const double t = (double)__uint_as_float(unord32(key)) * c8, fl = floor(t);
    return exp2_eighth(t - fl) * pow2_eighth((int)fmax(fl - J, -16000.0));
  }
  // smallest key whose t reaches `j` (a floor value)
  __device__ uint32_t lowest_key(double j) const {
    uint32_t l = kKeyLowest, h = 0xFF800000u;  // t(h) >= j or no finite key reaches it
    while (l < h) {
      const uint32_t mid = l + ((h - l) >> 1);
      if ((double)__uint_as_float(unord32(mid)) * c8 >= j) h = mid; else l = mid + 1;
    }
    return l;
  }

  template <class F>
  __device__ void each(F f) const {  // f(key, index) of every unmasked token of the row
    const int n_slots = (z.V + z.phase + VE - 1) / VE;
    for (int sl = tid; sl < n_slots; sl += kThreads) {
      const Slot x = z.load(sl);
      const int e = z.first(sl);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float v = slot_value<DT>(x, i);
        if (v > kNegInf) f(ord32_canon(__float_as_uint(fminf(v, RowType<DT>::kMax))), (uint32_t)(e + i));
      }
    }
  }

  // gather the tokens with lo <= key <= hi (at most kCap) into the list, sort
  // it and sum its weights
  __device__ void load(uint32_t lo_, uint32_t hi, uint32_t base_, double bmass_, int b0_, int b1_) {
    lo = lo_, base = base_, bmass = bmass_, b0 = b0_, b1 = b1_;
    __syncthreads();
    if (tid == 0) s.n_list = 0;
    __syncthreads();
    each([&](uint32_t key, uint32_t idx) {
      if (key >= lo && key <= hi) {
        const uint32_t i = atomicAdd(&s.n_list, 1u);
        if (i < kCap) s.comp[i] = ((uint64_t)~key << 32) | idx;
      }
    });
    sort();
  }

  __device__ void sort() {
    __syncthreads();
    n = min(s.n_list, (uint32_t)kCap);
    int P = 2;
    while (P < (int)n) P *= 2;
    for (int i = (int)n + tid; i < P; i += kThreads) s.comp[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= P; k *= 2)
      for (int j = k / 2; j > 0; j /= 2) {
        for (int q = tid; q < P / 2; q += kThreads) {
          const int i = ((q & ~(j - 1)) << 1) | (q & (j - 1)), l = i | j;
          const uint64_t x = s.comp[i], y = s.comp[l];
          if ((x > y) == ((i & k) == 0)) {
            s.comp[i] = y;
            s.comp[l] = x;
          }
        }
        __syncthreads();
      }
    double carry = bmass;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (e * kThreads >= (int)n) break;
      const int i = e * kThreads + tid;
      const double w = i < (int)n ? weight(~(uint32_t)(s.comp[i] >> 32)) : 0.0;
      cum[e] = carry + block_scan_f64(s.red, w);
      __syncthreads();
      if (tid == kThreads - 1) s.cum = cum[e];
      __syncthreads();
      carry = s.cum;
    }
  }

  __device__ Cross from_list(int kind, double amount) {
    int pos = (int)n;
#pragma unroll
    for (int e = kPer - 1; e >= 0; --e) {
      const int i = e * kThreads + tid;
      if (i < (int)n) {
        const bool hit = kind == kByCount    ? (double)(base + i + 1) >= amount
                         : kind == kByMassGe ? cum[e] >= amount
                         : kind == kByMassGt ? cum[e] > amount
                                             : weight(~(uint32_t)(s.comp[i] >> 32)) < amount;
        if (hit) pos = i;
      }
    }
    pos = block_min(s.red, pos);
    if (kind != kByWeight) pos = min(pos, (int)n - 1) + 1;  // pos tokens of the list are in
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (pos > 0 && e * kThreads + tid == pos - 1) s.cum = cum[e];
    __syncthreads();
    Cross r;
    r.n = base + pos;
    r.cum = pos > 0 ? s.cum : bmass;
    r.at = pos > 0 ? s.comp[pos - 1] : 0;
    r.cut = pos < (int)n ? s.comp[pos] : ((uint64_t)~lo + 1) << 32;
    return r;
  }

  // index of the r-th (from 1) token with this key, in index order: the waves
  // count contiguous pieces, the one that holds it walks its piece again
  __device__ uint32_t tie_index(uint32_t key, uint32_t r) {
    const int n_slots = (z.V + z.phase + VE - 1) / VE, lane = tid & 63, w = tid >> 6;
    const int per = ((n_slots + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int sb = w * per, se = min(n_slots, sb + per);
    auto count = [&](int sl, uint32_t* mask) {
      const Slot x = z.load(sl);
      uint32_t c = 0, mk = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float v = slot_value<DT>(x, i);
        const bool hit = v > kNegInf && ord32_canon(__float_as_uint(fminf(v, RowType<DT>::kMax))) == key;
        c += hit;
        mk |= (uint32_t)hit << i;
      }
      *mask = mk;
      return c;
    };
    uint32_t c = 0, mk;
    for (int sl = sb + lane; sl < se; sl += 64) c += count(sl, &mk);
    c = wave_sum_u32(c);
    __syncthreads();
    if (lane == 0) s.red.u[w] = c;
    if (tid == 0) s.at = 0;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < w; ++i) before += s.red.u[i];
    if (r > before && r <= before + s.red.u[w]) {
      uint32_t left = r - before;
      for (int b = sb; b < se; b += 64) {
        const uint32_t cl = b + lane < se ? count(b + lane, &mk) : 0;
        const uint32_t sc = wave_scan_u32(cl), total = __shfl(sc, 63);
        if (left <= total) {
          uint32_t k = left - (sc - cl);  // from 1 inside this lane's slot, if it is here
          if (left > sc - cl && left <= sc) {
            int i = -1;
            do {
              ++i;
              if ((mk >> i) & 1u) --k;
            } while (k);
            s.at = (uint64_t)(z.first(b + lane) + i);
          }
          break;
        }
        left -= total;
      }
    }
    __syncthreads();
    return (uint32_t)s.at;
  }

  // a bin (keys lo..hi, more tokens than the list holds): split its key range
  // until the part with the crossing fits, or is one value
  __device__ Cross split(int kind, double amount, uint32_t klo, uint32_t khi, uint32_t cb, double mb, bool tail) {
    for (;;) {
      const uint32_t range = khi - klo;
      const int sh = max(0, 32 - (range ? __builtin_clz(range) : 32) - 9);
      __syncthreads();
      s.cnt[tid] = 0;
      s.mass[tid] = 0;
      __syncthreads();
      each([&](uint32_t key, uint32_t) {
        if (key >= klo && key <= khi) {
          const uint32_t b = (khi - key) >> sh;
          atomicAdd(&s.cnt[b], 1u);
          if (!tail) {
            const double t = (double)__uint_as_float(unord32(key)) * c8;
            // 46 bits of the mantissa: sums of 2^21 tokens fit 64 bits
            atomicAdd((unsigned long long*)&s.mass[b],
                      (unsigned long long)((__double_as_longlong(exp2_eighth(t - floor(t))) - kOneBits) >> 6));
          }
        }
      });
      __syncthreads();
      // one bin holds one eighth of an octave: its unit is that of its lowest key
      const double unit = tail ? 0.0 : pow2_eighth((int)fmax(floor((double)__uint_as_float(unord32(klo)) * c8) - J, -16000.0));
      const uint32_t c = s.cnt[tid];
      const double mass = unit * ((double)c + (double)s.mass[tid] * 0x1p-46);
      const uint32_t c1 = cb + block_scan_u32(s.red, c);
      const double m1 = mb + block_scan_f64(s.red, mass);
      __syncthreads();
      s.rc[tid + 1] = c1;
      s.rm[tid + 1] = m1;
      if (tid == 0) {
        s.rc[0] = cb;
        s.rm[0] = mb;
      }
      const uint32_t top = khi - ((uint32_t)tid << sh);  // highest key of part tid (if it exists)
      const uint32_t n_part = (range >> sh) + 1;
      const uint32_t low = (uint32_t)tid + 1 >= n_part ? klo : top - ((1u << sh) - 1u);
      const bool hit = (uint32_t)tid < n_part &&
                       (kind == kByCount    ? (double)c1 >= amount
                        : kind == kByMassGe ? m1 >= amount
                        : kind == kByMassGt ? m1 > amount
                                            : weight(low) < amount);
      int b = block_first(s.red, hit);
      if (b >= (int)n_part) {
        // by rounding past the last token, or every key passes
        if (kind == kByWeight) {
          Cross r;
          r.n = s.rc[n_part];
          r.cum = s.rm[n_part];
          r.cut = ((uint64_t)~klo + 1) << 32;
          r.at = 0;
          return r;
        }
        kind = kByCount;
        amount = (double)s.rc[n_part];
        b = block_first(s.red, (uint32_t)tid < n_part && (double)c1 >= amount);
      }
      const uint32_t nc = s.rc[b + 1] - s.rc[b];
      const uint32_t nhi = khi - ((uint32_t)b << sh);
      const uint32_t nlo = (uint32_t)b + 1 >= n_part ? klo : nhi - ((1u << sh) - 1u);
      cb = s.rc[b];
      mb = s.rm[b];
      klo = nlo;
      khi = nhi;
      __syncthreads();
      if (nc <= kCap) {
        load(klo, khi, cb, mb, 1, 0);
        return from_list(kind, amount);
      }
      if (klo == khi) {  // one value: every token weighs w
        const double w = tail ? 0.0 : weight(klo);
        double r = (double)nc;
        if (kind == kByCount) r = amount - cb;
        if (kind == kByMassGe || kind == kByMassGt) {
          r = fmin(fmax(floor((amount - mb) / w), 0.0), (double)nc);
          // the quotient is off by rounding only: settle it on the sums themselves
          while (r > 0.0 && (kind == kByMassGe ? fma(r, w, mb) >= amount : fma(r, w, mb) > amount)) r -= 1.0;
          while (r < (double)nc && !(kind == kByMassGe ? fma(r, w, mb) >= amount : fma(r, w, mb) > amount)) r += 1.0;
          r = fmax(r, 1.0);
        }
        if (kind == kByWeight) r = weight(klo) < amount ? 0.0 : (double)nc;
        Cross x;
        x.n = cb + (uint32_t)r;
        x.cum = fma(r, w, mb);
        x.at = 0;
        x.cut = ((uint64_t)~klo) << 32;
        if (r > 0.0) {
          x.at = ((uint64_t)~klo << 32) | tie_index(klo, (uint32_t)r);
          x.cut = x.at + 1;
        }
        return x;
      }
    }
  }

  __device__ Cross locate(int kind, double amount) {
    // a sum within 2^-44 of the value counts as equal to it: rows of equal
    // logits meet dyadic settings exactly, and the sums round (below 2^-47)
    if (kind == kByMassGe) amount *= 1.0 - 0x1p-44;
    if (kind == kByMassGt) amount *= 1.0 + 0x1p-44;
    const bool hit = kind == kByCount    ? (double)s.cc[tid + 1] >= amount
                     : kind == kByMassGe ? s.cm[tid + 1] >= amount
                     : kind == kByMassGt ? s.cm[tid + 1] > amount
                                         : pow2_eighth(-tid) <= amount;
    int b = block_first(s.red, hit);
    if (b >= kBins) {
      b = kTail;
      if (kind != kByWeight) {  // a sum that rounding left short: the last token above the tail
        kind = kByCount;
        amount = (double)s.cc[kTail];
        b = block_first(s.red, (double)s.cc[tid + 1] >= amount);
      }
    }
    const uint32_t c = s.cc[b + 1] - s.cc[b];
    if (!(b >= b0 && b <= b1)) {
      const uint32_t klo = b == kTail ? kKeyLowest : lowest_key(J - b);
      const uint32_t khi = b == 0 ? kmax : lowest_key(J - b + 1.0) - 1u;
      if (c == 0) {  // kByWeight only: nothing in the threshold's own bin
        Cross r;
        r.n = s.cc[b];
        r.cum = s.cm[b];
        r.cut = ((uint64_t)~(khi + 1u) + 1) << 32;
        r.at = 0;
        return r;
      }
      if (c > kCap) return split(kind, amount, klo, khi, s.cc[b], s.cm[b], b == kTail);
      load(klo, khi, s.cc[b], s.cm[b], b, b);
    }
    return from_list(kind, amount);
  }
};

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_finalize_kernel(SampleArgs a, int64_t row0, int n_seg,
                                                                   const SamplePart* __restrict__ parts,
                                                                   const double* __restrict__ u, int32_t* __restrict__ token,
                                                                   float* __restrict__ prob, int32_t* __restrict__ kept,
                                                                   uint64_t* __restrict__ cuts) {
  __shared__ FinLds s;
  const int tid = threadIdx.x;
  const int64_t row = row0 + blockIdx.x;
  const RowParams rp = row_params(a, row);
  const SamplePart* part = parts + (size_t)blockIdx.x * n_seg;

  double J = -INFINITY;
  float m = kNegInf;
  uint32_t N = 0;
  for (int g = 0; g < n_seg; ++g) {
    J = fmax(J, part[g].J);
    m = fmaxf(m, part[g].max);
    N += part[g].n;
  }
  if (N == 0) {  // every token masked
    if (tid == 0) {
      if (token) token[row] = -1;
      if (prob) prob[row] = 0.0f;
      if (kept) kept[row] = 0;
      if (cuts) cuts[blockIdx.x] = 0;
    }
    return;
  }
  // the segments' bins on the row's grid, in segment order
  uint32_t c = 0;
  double mass = 0.0;
  for (int g = 0; g < n_seg; ++g) {
    if (part[g].n == 0) continue;
    const int shift = (int)fmin(J - part[g].J, (double)kBins), b = tid - shift;
    if (tid < kTail && b >= 0 && b < min(part[g].nb, kTail)) {
      c += part[g].cnt[b];
      mass += part[g].mass[b];
    }
  }
  uint32_t cs = block_scan_u32(s.red, c);
  const double ms = block_scan_f64(s.red, mass * pow2_eighth(-tid));
  if (tid == kTail) cs = N;  // the tail bin: whatever is left
  __syncthreads();
  s.cc[tid + 1] = cs;
  s.cm[tid + 1] = ms;
  if (tid == 0) {
    s.cc[0] = 0;
    s.cm[0] = 0.0;
  }
  __syncthreads();

  const uint32_t kmax = ord32_canon(__float_as_uint(m));
  Finalize<DT> f(s, RowRef<DT>(a.Z, row, a.stride, a.V), rp.c8, J, kmax);
  uint32_t n = N;
  double Z = s.cm[kBins];
  uint64_t cut = ~0ull;
  auto take = [&](const Cross& x) {
    if (x.n < n) {
      n = x.n;
      Z = x.cum;
      cut = x.cut;
    }
  };
  if (rp.k < (int64_t)N) take(f.locate(kByCount, (double)rp.k));
  if (rp.p < 1.0) take(f.locate(kByMassGe, rp.p * Z));
  if (rp.m > 0.0) take(f.locate(kByWeight, rp.m * f.weight(kmax)));
  if (kept && tid == 0) kept[row] = (int32_t)n;
  if (cuts && tid == 0) cuts[blockIdx.x] = cut;
  if (!token) return;
  double x = u[row];
  x = x > 0.0 ? fmin(x, 1.0 - 0x1p-53) : 0.0;  // NaN: 0
  Cross d = f.locate(kByMassGt, x * Z);
  if (d.n > n) d = f.locate(kByCount, (double)n);
  if (tid == 0) {
    token[row] = (int32_t)(uint32_t)d.at;
    if (prob) prob[row] = (float)(f.weight(~(uint32_t)(d.at >> 32)) / Z);
  }
}

// ---------------------------------------------------------------- (3) the filtered row

template <int DT, int NL>
__global__ __launch_bounds__(kThreads) void sample_apply_kernel(SampleArgs a, int64_t row0, int n_seg,
                                                                const uint64_t* __restrict__ cuts, uint32_t fill,
                                                                void* out, int64_t out_stride) {
  using E = typename RowType<DT>::elem;
  constexpr int VE = RowType<DT>::VE;
  const int tid = threadIdx.x, seg = blockIdx.x % n_seg;
  const int64_t r = blockIdx.x / n_seg, row = row0 + r;
  const RowRef<DT> z(a.Z, row, a.stride, a.V);
  E* o = static_cast<E*>(out) + row * out_stride;
  const bool same = (reinterpret_cast<uintptr_t>(o) & 15u) == (reinterpret_cast<uintptr_t>(z.p) & 15u);
  const uint64_t cut = cuts[r];
  const int s0 = seg * (kThreads * NL) + tid;
  Slot x[NL];
#pragma unroll
  for (int l = 0; l < NL; ++l) x[l] = z.load(s0 + l * kThreads);
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    const int e = z.first(s0 + l * kThreads);
    Slot y;
#pragma unroll
    for (int k = 0; k < 4; ++k) y.w[k] = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float v = slot_value<DT>(x[l], i);
      const uint32_t key = ord32_canon(__float_as_uint(fminf(v, RowType<DT>::kMax)));
      const bool in = v > kNegInf && (((uint64_t)~key << 32) | (uint32_t)(e + i)) < cut;
      if constexpr (DT == DFLASH_BF16) {
        const uint32_t raw = (i & 1) ? x[l].w[i >> 1] >> 16 : x[l].w[i >> 1] & 0xFFFFu;
        y.w[i >> 1] |= (in ? raw : fill) << ((i & 1) * 16);
      } else {
        y.w[i] = in ? x[l].w[i] : fill;
      }
    }
    store_slot<DT>(o, z, s0 + l * kThreads, y, same);
  }
}

template <int DT, int NL>
hipError_t run(const SampleArgs& a, const SampleOut& o, char* ws, const SamplePlan& pl, hipStream_t st) {
  SamplePart* parts = reinterpret_cast<SamplePart*>(ws + pl.parts);
  uint64_t* cuts = reinterpret_cast<uint64_t*>(ws + pl.cuts);
  for (int64_t r0 = 0; r0 < a.R; r0 += pl.batch) {
    const unsigned nr = (unsigned)(a.R - r0 < pl.batch ? a.R - r0 : pl.batch), nb = nr * (unsigned)pl.n_seg;
    launch(sample_hist_kernel<DT, NL>, dim3(nb), dim3(kThreads), st, a, r0, pl.n_seg, parts);
    launch(sample_finalize_kernel<DT>, dim3(nr), dim3(kThreads), st, a, r0, pl.n_seg, (const SamplePart*)parts, o.u,
                 o.token, o.prob, o.kept, o.out ? cuts : (uint64_t*)nullptr);
    if (o.out)
      launch(sample_apply_kernel<DT, NL>, dim3(nb), dim3(kThreads), st, a, r0, pl.n_seg, (const uint64_t*)cuts, o.fill,
                   o.out, o.out_stride);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t run_nl(const SampleArgs& a, const SampleOut& o, char* ws, const SamplePlan& pl, hipStream_t st) {
  switch (pl.loads) {
    case 1: return run<DT, 1>(a, o, ws, pl, st);
    case 2: return run<DT, 2>(a, o, ws, pl, st);
    case 4: return run<DT, 4>(a, o, ws, pl, st);
    default: return run<DT, 8>(a, o, ws, pl, st);
  }
}

}  // namespace

hipError_t launch_sample(int32_t dtype, const SampleArgs& a, const SampleOut& o, char* ws, const SamplePlan& pl,
                         hipStream_t st) {
  return dtype == DFLASH_BF16 ? run_nl<DFLASH_BF16>(a, o, ws, pl, st) : run_nl<DFLASH_F32>(a, o, ws, pl, st);
}

}  // namespace dfk
