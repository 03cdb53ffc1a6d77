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
// It is answered without sorting the row, in two ways.
//
// bf16 rows (few distinct values): sample_values_kernel counts each value of a
// row segment in LDS; sample_finalize_values_kernel, one block per row, adds
// the segments' counts in the row's order, weighs each value present once and
// scans.  A crossing is a value and a place among its equal tokens, which
// share one weight; that token's index is looked up in its own segment.
//
// fp32 rows: in units of an eighth of an octave a weight is 2^(t / 8), t = z
// 8 log2(e) / T, and rint(t) bins the tokens in their order.
// (1) sample_hist_kernel counts the tokens and sums the weights of each bin of
//     a row segment, and lists the segment's largest tokens in the order of
//     their bins.
// (2) sample_finalize_kernel, one block per row, adds the segments' bins,
//     scans them, finds the bin of the crossing and ranks that bin's tokens
//     alone: a window of at most 512 tokens; a fuller bin is narrowed by key
//     ranges first, and tokens of one value share one weight, so that their
//     crossing is a division.
// (3) Of few tokens all are listed.  Else rows whose cut or draw falls outside
//     the lists ask for the bins they need;
//     sample_gather_kernel collects those from all segments at once, and
//     the row is finished by a second run of (2).
// A bf16 row with values out of the counters' range goes the second way, in
// one block that reads the row as often as it needs.
//
// sample_apply_kernel (dflash_filter) copies the kept tokens.  Short rows of
// either type take (1) and (2) in one launch, a block a row: sample_row_kernel.
//
// Counts are exact and sums do not depend on the order of the atomics: every
// 2^((t - rint(t)) / 8) is rounded to a multiple of 2^-42 (off by 2^-43 of
// itself, and by 2^-51 |z| / T as t is rounded) wherever it is used, and summed
// as an integer.  Decisions next to a border need such sums: they compare running
// sums over the whole vocabulary.  Only min-p asks for single weights; it takes
// them from the logits in full precision.
#include "rows_blocks.hpp"

// t = z c8 is one rounded product wherever it is formed: fused into the
// subtraction of rint(t) it would differ from the value that was binned
#pragma clang fp contract(off)

namespace dfk {

namespace {

constexpr int kThreads = kSampleThreads;
constexpr int kWaves = kThreads / kWave;
constexpr int kBins = kSampleBins;  // 64 octaves; the last bin collects everything below (weight under 2^-63.9)
constexpr int kTail = kBins - 1;
constexpr int kCols = 4;            // copies of the bins that lanes spread over
static_assert(kThreads == kBins, "one thread per bin");

constexpr uint32_t kKeyLowest = 0x00800000u;  // ordered key of the lowest finite fp32
constexpr uint32_t kKeyZero = 0x80000000u;    // of zero

constexpr double kLn2Eighth = 0.08664339756999316;  // ln 2 / 8

// an fp64 constant in scalar registers: an fma takes one as its addend, where a
// literal would be moved into the vector registers that it accumulates in
__device__ __forceinline__ double scalar(double c) {
  asm("" : "+s"(c));
  return c;
}

// 2^(f / 8), |f| <= 1/2, plus 1024: the Taylor series to degree 6 (truncation
// below 2^-43.9), rounded to a multiple of 2^-42
__device__ __forceinline__ double exp2_eighth_1024(double f) {
  constexpr double L = kLn2Eighth, L2 = L * L, L3 = L2 * L;
  double p = fma(f, scalar(L3 * L3 / 720.0), L3 * L2 / 120.0);
  p = fma(p, f, scalar(L2 * L2 / 24.0));
  p = fma(p, f, scalar(L3 / 6.0));
  p = fma(p, f, scalar(L2 / 2.0));
  p = fma(p, f, scalar(L));
  return fma(p, f, scalar(1025.0));
}
__device__ __forceinline__ double exp2_eighth(double f) { return exp2_eighth_1024(f) - 1024.0; }
// in units of 2^-42
__device__ __forceinline__ unsigned long long exp2_eighth_units(double f) {
  return (unsigned long long)__double_as_longlong(exp2_eighth_1024(f)) & ((1ull << 52) - 1);
}

// 2^(e / 8), e <= 0 an integer
__device__ __forceinline__ double pow2_eighth(int e) {
  const int r = e & 7;
  double v = (r & 4) ? 1.4142135623730951 : 1.0;
  v *= (r & 2) ? 1.189207115002721 : 1.0;
  v *= (r & 1) ? 1.0905077326652577 : 1.0;
  return ldexp(v, e >> 3);
}

// 2^t, t <= 0, to fp64's precision: by the nearest integer and the Taylor series
// of e^(f ln 2), |f| <= 1/2, to degree 12 (truncation below 2e-16)
__device__ __forceinline__ double exp2_full(double t) {
  t = fmax(t, -1100.0);
  const double n = rint(t), x = (t - n) * 0.6931471805599453;
  double p = fma(x, scalar(1.0 / 479001600.0), 1.0 / 39916800.0);
  p = fma(p, x, scalar(1.0 / 3628800.0));
  p = fma(p, x, scalar(1.0 / 362880.0));
  p = fma(p, x, scalar(1.0 / 40320.0));
  p = fma(p, x, scalar(1.0 / 5040.0));
  p = fma(p, x, scalar(1.0 / 720.0));
  p = fma(p, x, scalar(1.0 / 120.0));
  p = fma(p, x, scalar(1.0 / 24.0));
  p = fma(p, x, scalar(1.0 / 6.0));
  p = fma(p, x, 0.5);
  p = fma(p, x, 1.0);
  return ldexp(fma(p, x, 1.0), (int)n);
}

struct RowParams {
  double c8;  // 8 log2(e) / T
  double t8;  // T ln(2) / 8
  int64_t k;  // top-k; INT64_MAX: off
  double p;   // top-p; >= 1: off
  double m;   // min-p; <= 0: off
};

__device__ __forceinline__ RowParams row_params(const SampleArgs& a, int64_t row) {
  const uint32_t g = (uint32_t)row / (uint32_t)a.group;  // rows fit 23 bits
  const float T = a.T ? a.T[g] : 1.0f;
  const bool greedy = !(T > 0.0f);
  RowParams r;
  r.c8 = 8.0 * 1.4426950408889634 / (greedy ? 1.0 : (double)T);
  r.t8 = kLn2Eighth * (greedy ? 1.0 : (double)T);
  const int32_t k = a.top_k ? a.top_k[g] : 0;
  r.k = greedy ? 1 : (k > 0 ? (int64_t)k : INT64_MAX);
  const float p = a.top_p ? a.top_p[g] : 1.0f;
  r.p = !greedy && p < 1.0f ? fmax((double)p, 0.0) : 1.0;
  const float m = a.min_p ? a.min_p[g] : 0.0f;
  r.m = !greedy && m > 0.0f ? fmin((double)m, 1.0) : 0.0;
  return r;
}

// ---------------------------------------------------------------- block helpers (kThreads threads)

// inclusive prefix sums, over the 16 lanes of a row and over all 64
__device__ __forceinline__ uint32_t row16_scan_u32(uint32_t v) {
  v += dpp_u32<kDppRowShr1>(v, 0u);
  v += dpp_u32<kDppRowShr2>(v, 0u);
  v += dpp_u32<kDppRowShr4>(v, 0u);
  v += dpp_u32<kDppRowShr8>(v, 0u);
  return v;
}
__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t v) {
  v = row16_scan_u32(v);
  v += dpp_u32<kDppRowBcast15, 0xA>(v, 0u);
  v += dpp_u32<kDppRowBcast31, 0xC>(v, 0u);
  return v;
}

// Reductions over the block with one barrier each: successive calls alternate
// between two buffers, so a buffer is rewritten only after the barrier of the
// call between, which every thread reaches after it has read the buffer.  What
// is equal on all lanes goes to scalar registers.
struct Red {
  double d[2][kWaves];
  uint32_t u[2][kWaves];
};

struct BlockOps {
  Red& s;
  int flip;
  __device__ explicit BlockOps(Red& r) : s(r), flip(0) {}

  // smallest thread index whose predicate holds (kThreads if none)
  __device__ __forceinline__ int first(bool pred) {
    const int tid = threadIdx.x, f = first_lane(pred);
    flip ^= 1;
    if ((tid & 63) == 0) s.u[flip][tid >> 6] = f < 64 ? (uint32_t)(tid + f) : (uint32_t)kThreads;
    __syncthreads();
    uint32_t r = s.u[flip][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) r = min(r, s.u[flip][w]);
    return (int)__builtin_amdgcn_readfirstlane(r);
  }
  // inclusive scans, in fixed order
  __device__ __forceinline__ uint32_t scan(uint32_t v) {
    const int w = threadIdx.x >> 6;
    v = wave_scan_u32(v);
    flip ^= 1;
    if ((threadIdx.x & 63) == 63) s.u[flip][w] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i) v += i < w ? s.u[flip][i] : 0u;
    return v;
  }
  // both, with one barrier
  __device__ __forceinline__ void scan(uint32_t& n, double& v) {
    const int w = threadIdx.x >> 6;
    n = wave_scan_u32(n);
    v = wave_scan_f64(v);
    flip ^= 1;
    if ((threadIdx.x & 63) == 63) {
      s.u[flip][w] = n;
      s.d[flip][w] = v;
    }
    __syncthreads();
    double off = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i) {
      n += i < w ? s.u[flip][i] : 0u;
      off += i < w ? s.d[flip][i] : 0.0;
    }
    v += off;
  }
  __device__ __forceinline__ double scan(double v) {
    const int w = threadIdx.x >> 6;
    v = wave_scan_f64(v);
    flip ^= 1;
    if ((threadIdx.x & 63) == 63) s.d[flip][w] = v;
    __syncthreads();
    double off = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i) off += i < w ? s.d[flip][i] : 0.0;
    return v + off;
  }
  __device__ __forceinline__ double max(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o));
    flip ^= 1;
    if ((threadIdx.x & 63) == 0) s.d[flip][threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.d[flip][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v = fmax(v, s.d[flip][w]);
    return readlane_f64(v, 0);
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    v = ::max(v, dpp_u32<kDppRowShr1>(v, 0u));
    v = ::max(v, dpp_u32<kDppRowShr2>(v, 0u));
    v = ::max(v, dpp_u32<kDppRowShr4>(v, 0u));
    v = ::max(v, dpp_u32<kDppRowShr8>(v, 0u));
    v = ::max(v, dpp_u32<kDppRowBcast15, 0xA>(v, 0u));
    v = ::max(v, dpp_u32<kDppRowBcast31, 0xC>(v, 0u));
    flip ^= 1;
    if ((threadIdx.x & 63) == 63) s.u[flip][threadIdx.x >> 6] = v;
    __syncthreads();
    v = s.u[flip][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v = ::max(v, s.u[flip][w]);
    return __builtin_amdgcn_readfirstlane(v);
  }
  __device__ __forceinline__ uint32_t sum(uint32_t v) {
    v = wave_scan_u32(v);
    flip ^= 1;
    if ((threadIdx.x & 63) == 63) s.u[flip][threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s.u[flip][w];
    return __builtin_amdgcn_readfirstlane(v);
  }

};

__device__ __forceinline__ uint32_t key_of(float v, float max_finite) {
  return ord32_canon(__float_as_uint(fminf(v, max_finite)));
}
__device__ __forceinline__ double key_value(uint32_t key) { return (double)__uint_as_float(unord32(key)); }

// smallest ordered key >= kKeyLowest whose t = z c8 rounds to `j` or more
// (0xFF800000, above every finite key, if none does).  One round of the wave's
// 64 lanes around (j - 1/2) t8, t8 = 1 / c8, which rounding moves by a few
// keys; a search where that guess does not bracket it (j or c8 extreme).
__device__ __forceinline__ uint32_t lowest_key(double j, double c8, double t8) {
  const double z = fmin(fmax((j - 0.5) * t8, -3.4028234663852886e38), 3.4028234663852886e38);
  const uint32_t g = max(ord32_canon(__float_as_uint((float)z)), kKeyLowest + 32u);
  const uint32_t cand = min(g - 32u + (uint32_t)lane_id(), 0xFF7FFFFFu);
  const uint64_t hit = __ballot(rint(key_value(cand) * c8) >= j);
  if (hit && !(hit & 1)) return __shfl(cand, __builtin_ctzll(hit));
  uint32_t l = kKeyLowest, h = 0xFF800000u;
  while (l < h) {
    const uint32_t mid = l + ((h - l) >> 1);
    if (rint(key_value(mid) * c8) >= j) h = mid; else l = mid + 1;
  }
  return l;
}

// min-p on the logits themselves: the least key whose weight, in full precision
// relative to the largest key's, is at least m (0: min-p is off).  As above: a
// round of 64 lanes around zmax + T ln m, and a search of 64 lanes a round
// otherwise (the border near zero, where keys are dense).
__device__ __forceinline__ uint32_t least_key(double m, uint32_t kmax, double c8, double t8) {
  if (!(m > 0.0)) return 0;
  const double zmax = key_value(kmax), c = c8 * 0.125;
  const double z = fmin(fmax(zmax + 8.0 * (double)__builtin_amdgcn_logf((float)m) * t8, -3.4028234663852886e38), zmax);
  const uint32_t g = max(ord32_canon(__float_as_uint((float)z)), kKeyLowest + 32u);
  uint32_t cand = min(g - 32u + (uint32_t)lane_id(), kmax);
  uint64_t hit = __ballot(exp2_full((key_value(cand) - zmax) * c) >= m);
  if (hit && !(hit & 1)) return (uint32_t)__builtin_amdgcn_readlane(cand, __builtin_ctzll(hit));
  uint32_t l = kKeyLowest, h = kmax;  // kmax weighs 1
  while (l < h) {
    const uint32_t step = (h - l + 63u) / 64u;
    cand = min(l + (uint32_t)lane_id() * step, h);
    hit = __ballot(exp2_full((key_value(cand) - zmax) * c) >= m);
    const int f = hit ? __builtin_ctzll(hit) : 64;
    if (f > 0) l = min(l + (uint32_t)(f - 1) * step, h) + 1u;
    if (f < 64) h = (uint32_t)__builtin_amdgcn_readlane(cand, f);
    if (f == 0) break;
  }
  return h;
}
// the bin of a key at or below the row's largest
__device__ __forceinline__ int bin_of(uint32_t key, double c8, double J) {
  return (int)fmin(J - rint(key_value(key) * c8), (double)kTail);
}

__device__ __forceinline__ uint32_t comp_key(uint64_t c) { return ~(uint32_t)(c >> 32); }
__device__ __forceinline__ uint64_t comp_of(uint32_t key, uint32_t index) { return ((uint64_t)~key << 32) | index; }

// ---------------------------------------------------------------- (1) bins of a segment

// A bin's cell takes a token in one 64-bit atomic: 1 from bit 51 on, and below
// it the token's weight over 15/16, in units of 2^-42 (0.02 to 0.107).  Four
// cells a bin, so one takes at most 128 threads' 32 tokens: 2^12, whose sum
// stays below 2^50.8.  Beside a separate count this saves a third of the LDS
// work.
constexpr int kCellCount = 51;
constexpr unsigned long long kCellLess = 15ull << 38;  // 15/16 in units of 2^-42
static_assert(kThreads / kCols * kSampleMaxLoads * 4 <= 4096, "");

template <int NL, bool ALL>
struct HistLds {
  unsigned long long cell[kBins * kCols];
  uint32_t next[kBins];                                 // the list's next place for each bin
  uint16_t pick[kWaves][ALL ? 1 : sample_cap(NL, false)];  // a wave's slots with tokens to be listed
  Red red;
};

__device__ __forceinline__ unsigned long long cell_of(double f) {
  // the constants touch the upper word alone
  constexpr uint32_t kUpper = (uint32_t)((((1ull << kCellCount) - kCellLess) >> 32) - 0x40900000u);
  const unsigned long long w = (unsigned long long)__double_as_longlong(exp2_eighth_1024(f));
  return (unsigned long long)((uint32_t)(w >> 32) + kUpper) << 32 | (uint32_t)w;
}

// a thread's tokens into the bins' cells; J: the maximum's bin
template <int DT, int NL>
__device__ __forceinline__ void add_cells(unsigned long long* cells, const Slot (&x)[NL], double J, const RowParams& rp) {
  constexpr int VE = RowType<DT>::VE;
  constexpr float kMax = RowType<DT>::kMax;
  const double c8 = rp.c8;
  unsigned long long* cell = cells + (threadIdx.x & (kCols - 1));
  uint32_t tail = 0;  // counted aside: a mask of finite lowest values would queue up at one address
  if (fabs(J) <= 0x1p20) {
    // rint by adding 3 2^51, whose sum's lower word is the integer.  Tokens far
    // below the maximum are raised to 1000 bins below it: the tail all the same
    constexpr double kMagic = 0x1.8p52;
    const float lowest = (float)((J - 1000.0) * rp.t8);
    const int j = (int)J;
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float v = slot_value<DT>(x[l], i);
        if (v > kNegInf) {
          const double t = (double)__builtin_amdgcn_fmed3f(v, lowest, kMax) * c8, r = t + kMagic;
          const uint32_t b = (uint32_t)(j - (int)(uint32_t)__double_as_longlong(r));
          if (b < (uint32_t)kTail)
            atomicAdd(&cell[b * kCols], cell_of(t - (r - kMagic)));
          else
            ++tail;
        }
      }
  } else {
    // |max| / T over 9e4: t's integer does not fit the sum's lower word.  Few rows
    // have it, so the registers of a loop matter and its time does not (each token
    // is picked by NL VE comparisons)
#pragma unroll 1
    for (int e = 0; e < NL * VE; ++e) {
      float v = kNegInf;
#pragma unroll
      for (int k = 0; k < NL * VE; ++k)
        if (k == e) v = slot_value<DT>(x[k / VE], k % VE);
      if (v > kNegInf) {
        const double t = (double)fminf(v, kMax) * c8, n = rint(t);
        if (J - n < (double)kTail)
          atomicAdd(&cell[(int)(J - n) * kCols], cell_of(t - n));
        else
          ++tail;
      }
    }
  }
  if (__ballot(tail != 0)) {
    tail = wave_sum_u32(tail);
    if (lane_id() == 0) atomicAdd(&cells[kTail * kCols + ((threadIdx.x >> 6) & (kCols - 1))], (unsigned long long)tail << kCellCount);
  }
}

// a bin's tokens c, and their weight in units of 2^-42
__device__ __forceinline__ unsigned long long read_cells(const unsigned long long* cells, int bin, uint32_t& c) {
  c = 0;
  unsigned long long f = 0;
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    const unsigned long long w = cells[bin * kCols + k];
    c += (uint32_t)(w >> kCellCount);
    f += w & ((1ull << kCellCount) - 1);
  }
  return f + (unsigned long long)c * kCellLess;
}

// a token into the list, which is in the order of its bins
__device__ __forceinline__ void list_token(uint32_t* next, uint64_t* list, double c8, double J, uint64_t c) {
  list[atomicAdd(&next[bin_of(comp_key(c), c8, J)], 1u)] = c;
}

// Bound by instructions, about twenty a token, eleven of them fp64 (t, its bin,
// the weight): 256 x 262144 fp32 in 88 us, 3.1 TB/s.  Counting the tail aside is
// 8 of them (80 with one atomic for either), for the sake of rows under a mask of
// finite values (512 x 262144 masked by -1e4: a call of 193 us, 300 with it).  In a
// build of 74 us the weight took 21, the list 10; the one atomic a token hides
// behind them.
template <int NL, bool ALL>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(SampleArgs a, int64_t row0, int n_seg, int cap,
                                                               SamplePart* __restrict__ parts, uint64_t* __restrict__ lists) {
  constexpr int VE = RowType<DFLASH_F32>::VE;
  constexpr float kMax = RowType<DFLASH_F32>::kMax;
  __shared__ HistLds<NL, ALL> s;
  BlockOps ops(s.red);
  const int tid = threadIdx.x, seg = blockIdx.x % n_seg;
  const int64_t row = row0 + blockIdx.x / n_seg;
  const RowRef<DFLASH_F32> z(a.Z, row, a.stride, a.V);
  const RowParams rp = row_params(a, row);
  const double c8 = rp.c8;
  const int s0 = seg * (kThreads * NL) + tid;
  Slot x[NL];
#pragma unroll
  for (int l = 0; l < NL; ++l) x[l] = z.load<true>(s0 + l * kThreads);
#pragma unroll
  for (int c = 0; c < kCols; ++c) s.cell[c * kBins + tid] = 0;
  float m = kNegInf, most[NL];  // the slots' largest
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    most[l] = kNegInf;
#pragma unroll
    for (int i = 0; i < VE; ++i) most[l] = fmaxf(most[l], slot_value<DFLASH_F32>(x[l], i));  // NaN drops out
    m = fmaxf(m, most[l]);
  }
  m = (float)ops.max((double)fminf(m, kMax));
  SamplePart& out = parts[blockIdx.x];
  if (m == kNegInf) {
    if (tid == 0) {
      out.J = -INFINITY;
      out.max = kNegInf;
      out.n = 0;
      out.nb = 0;
      out.listed = kBins;
    }
    return;
  }
  const double J = rint((double)m * c8);
  add_cells<DFLASH_F32>(s.cell, x, J, rp);
  __syncthreads();
  uint32_t c, far;  // far: the bin counted from the other end
  const unsigned long long f = read_cells(s.cell, tid, c);
  read_cells(s.cell, kBins - 1 - tid, far);
  const uint32_t upto = ops.scan(c);
  const int nb = kBins - ops.first(far != 0);       // bins in use
  const int listed = ops.first(upto > (uint32_t)cap);  // leading bins with at most `cap` tokens together
  s.next[tid] = upto - c;
  if (tid < nb) {
    out.upto[tid] = upto;
    out.mass[tid] = tid < kTail ? (double)f * 0x1p-42 : 0.0;
  }
  if (tid == kThreads - 1) {
    out.J = J;
    out.max = m;
    out.n = upto;
    out.nb = nb;
    out.listed = listed;
  }
  __syncthreads();
  if (listed == 0) return;
  uint64_t* list = lists + (size_t)blockIdx.x * cap;
  const int first = seg * (kThreads * NL) * VE;
  if constexpr (ALL) {  // cap holds the whole segment
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float v = slot_value<DFLASH_F32>(x[l], i);
        if (v > kNegInf) list_token(s.next, list, c8, J, comp_of(key_of(v, kMax), (uint32_t)(first + (tid + l * kThreads) * VE + i)));
      }
  } else {
    // few tokens: a wave picks the slots that hold one, then reads them again,
    // four lanes a slot
    const float least = listed >= kBins ? -kMax : __uint_as_float(unord32(lowest_key(J - (double)(listed - 1), c8, rp.t8)));
    uint16_t* pick = s.pick[tid >> 6];
    int n = 0;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const uint64_t hits = __ballot(most[l] >= least);
      if (hits) {
        const int at = n + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(hits >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)hits, 0));
        if (most[l] >= least && at < sample_cap(NL, false)) pick[at] = (uint16_t)(tid + l * kThreads);
        n += __popcll(hits);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    n = min(n, sample_cap(NL, false));
    for (int i = lane_id(); i < n * VE; i += kWave) {
      const int slot = pick[i / VE];
      const Slot y = z.load(seg * (kThreads * NL) + slot);
      const int k = i % VE;
      const float v = __uint_as_float(k == 0 ? y.w[0] : k == 1 ? y.w[1] : k == 2 ? y.w[2] : y.w[3]);
      if (v >= least) list_token(s.next, list, c8, J, comp_of(key_of(v, kMax), (uint32_t)(first + slot * VE + k)));  // not NaN, not masked
    }
  }
}

// ---------------------------------------------------------------- (2) cuts and draw of a row

enum { kByCount, kByMassGe, kByMassGt, kByWeight };
// kAll: the lists hold every token.  kFirst: they hold the largest; rows that
// need others ask for them.  kSecond: the rows that asked.  kSelf: no lists,
// the row itself is read.  kOne: a row of one block, which holds the list of
// all its tokens.
enum { kAll, kFirst, kSecond, kSelf, kOne };
constexpr int kMaxSeg = kSampleMaxSeg;

struct FinLds {
  uint64_t win[kThreads];   // the window: sorted (~key, index), ascending = the row's order
  double wcum[kThreads];    // and the running sums at its tokens
  uint64_t mass[kBins];     // parts of a key range
  uint32_t cnt[kBins];
  uint32_t cc[kBins + 1];   // tokens before each bin
  double cm[kBins + 1];     // their weight
  int16_t shift[kMaxSeg];   // a segment's first bin on the row's grid
  int16_t nb[kMaxSeg];      // its bins
  uint32_t n_seg[kMaxSeg];  // its unmasked tokens
  uint32_t from[kMaxSeg];   // its listed tokens of some bins: from .. to - 1
  uint32_t to[kMaxSeg];
  Red red;
  uint32_t n;
  uint32_t before_n;
  double before_m;
};

// where a running count or sum crosses a value (kByWeight: where keys fall below
// one, in fp64 as the others)
struct Cross {
  uint32_t n;    // tokens up to and including the crossing one (kByWeight: tokens that pass)
  double cum;    // their weight
  uint64_t cut;  // a token is among them iff its (~key, index) is below this
  uint64_t at;   // (~key, index) of the last of them (not for kByWeight); 0: none at hand (a bin that kFirst has not listed)
};

template <int DT, int MODE>
struct Finalize {
  static constexpr int VE = RowType<DT>::VE;
  FinLds& s;
  BlockOps& ops;
  const RowRef<DT> z;
  const SamplePart* part;
  const uint64_t* lists;
  const uint64_t* asked;  // the row's asked-for tokens
  const SampleAsk* ask;
  const uint32_t ask_cap;
  const int n_seg, cap;
  const double c8, t8, J;
  const int tid;
  const uint32_t kmax;  // the row's largest key
  const uint32_t kmin;  // the least that min-p keeps; 0: off
  const int listed;     // bins 0 .. listed - 1 are in the segments' lists
  // the window's tokens: rank base + 1 .. base + n, of bins b0 .. b1 (b0 > b1: part of a bin)
  uint32_t base, n;
  double bmass;
  int b0, b1;
  uint32_t lo;
  uint32_t seen_lo, seen_hi;  // the last pass's least and largest key

  // weight of a key relative to 2^(J / 8)
  __device__ __forceinline__ double weight(uint32_t key) const {
    const double t = key_value(key) * c8, n = rint(t);
    return exp2_eighth(t - n) * pow2_eighth((int)fmax(n - J, -16000.0));
  }

  // f((~key, index)) of every token of bins B0 .. B1, and of others
  template <class F>
  __device__ __forceinline__ void each(int B0, int B1, F f) {
    if constexpr (MODE == kOne) {
      const int end = (int)s.cc[B1 + 1];
      for (int j = (int)s.cc[B0] + tid; j < end; j += kThreads) f(lists[j]);
    } else if (MODE != kSelf && (MODE == kAll || B1 < listed)) {
      // a segment's list is in the order of its bins, so its part is one run
      __syncthreads();
      if (tid < n_seg) {
        const int l0 = B0 - s.shift[tid], l1 = B1 - s.shift[tid], nb = s.nb[tid];
        const uint32_t* upto = part[tid].upto;
        const uint32_t n_all = s.n_seg[tid];
        s.from[tid] = l0 <= 0 ? 0u : l0 > nb ? n_all : upto[l0 - 1];
        s.to[tid] = B1 == kTail || l1 >= nb ? n_all : l1 < 0 ? 0u : upto[l1];  // the last bin: all that is left
      }
      __syncthreads();
      const bool lots = s.cc[B1 + 1] - s.cc[B0] > 1024u * (uint32_t)n_seg;  // then all threads on one segment after the other
      const int per = lots ? 9 : n_seg <= 16 ? 5 : 4;  // log2 of the threads a segment
      for (int g = tid >> per; g < n_seg; g += kThreads >> per) {
        const uint64_t* list = lists + (size_t)g * cap;
        const int end = (int)s.to[g];
#pragma unroll 4
        for (int j = (int)s.from[g] + (tid & ((1 << per) - 1)); j < end; j += 1 << per) f(list[j]);
      }
    } else if constexpr (MODE == kSecond || MODE == kSelf) {
      if (MODE == kSecond && ask->kind == kSampleAskBins && ((B0 >= ask->b0[0] && B1 <= ask->b1[0]) || (B0 >= ask->b0[1] && B1 <= ask->b1[1]))) {
        const int end = (int)min(ask->n, ask_cap);
#pragma unroll 4
        for (int j = tid; j < end; j += kThreads) f(asked[j]);
      } else {
        const int n_slots = z.slots();
#pragma unroll 2
        for (int sl = tid; sl < n_slots; sl += kThreads) {
          const Slot x = z.load(sl);
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const float v = slot_value<DT>(x, i);
            if (v > kNegInf) f(comp_of(key_of(v, RowType<DT>::kMax), (uint32_t)(sl * VE + i)));
          }
        }
      }
    }
  }

  // One pass over bins B0 .. B1: the tokens with klo <= key <= khi and ilo <=
  // index <= ihi go into the window (sh < 0), or are counted and weighed in
  // parts of 2^sh keys from the highest down (of 2^sh indices if by_index)
  __device__ __forceinline__ void pass(int B0, int B1, uint32_t klo, uint32_t khi, uint32_t ilo, uint32_t ihi, int sh, bool by_index) {
    __syncthreads();
    s.cnt[tid] = 0;
    s.mass[tid] = 0;
    if (tid == 0) s.n = 0;
    __syncthreads();
    const bool weigh = !by_index && B1 != kTail;
    uint32_t least = 0xFFFFFFFFu, most = 0;
    // so many tokens in one bin that equal ones may queue up at one address
    const bool queue = (MODE == kAll || MODE == kSecond) && s.cc[B1 + 1] - s.cc[B0] > 16384u;
    each(B0, B1, [&](uint64_t c) {
      const uint32_t key = comp_key(c), idx = (uint32_t)c;
      if (key < klo || key > khi || idx < ilo || idx > ihi) return;
      if (sh < 0) {
        const uint32_t i = atomicAdd(&s.n, 1u);
        if (i < (uint32_t)kThreads) s.win[i] = c;
      } else {
        const uint32_t b = (by_index ? idx - ilo : khi - key) >> sh;
        least = min(least, key);
        most = max(most, key);
        uint32_t many = 1;
        if (queue) {  // one addition for a wave of equal tokens
          const uint64_t lanes = __ballot(1);
          if (__ballot(b != (uint32_t)__builtin_amdgcn_readfirstlane(b) || key != (uint32_t)__builtin_amdgcn_readfirstlane(key)) == 0)
            many = lane_id() == __builtin_ctzll(lanes) ? (uint32_t)__popcll(lanes) : 0u;
        }
        if (many) {
          atomicAdd(&s.cnt[b], many);
          if (weigh) {
            const double t = key_value(key) * c8;
            atomicAdd((unsigned long long*)&s.mass[b], many * exp2_eighth_units(t - rint(t)));  // sums of 2^21 tokens fit 64 bits
          }
        }
      }
    });
    if (sh >= 0 && !by_index) {
      seen_lo = ~ops.max(~least);
      seen_hi = ops.max(most);
    }
    __syncthreads();
  }

  // s.win[0 .. s.n - 1] holds the window's tokens (keys lo_ .. hi) in any order:
  // sort them and sum their weights.  A token's rank is counted against all
  // others if they are few, else against those of its own of 512 key ranges
  // (512 tokens against all: 15 thousand cycles, 6 us)
  __device__ __forceinline__ void open_window(uint32_t lo_, uint32_t hi, uint32_t base_, double bmass_, int b0_, int b1_) {
    lo = lo_, base = base_, bmass = bmass_, b0 = b0_, b1 = b1_;
    n = min((uint32_t)__builtin_amdgcn_readfirstlane(s.n), (uint32_t)kThreads);
    const bool in = tid < (int)n;
    const uint64_t mine = in ? s.win[tid] : 0;
    uint32_t from = 0, to = n, rank = 0;
    if (n > 64) {
      const uint32_t range = hi - lo;
      const int sh = max(0, 32 - (range ? __builtin_clz(range) : 32) - 9);
      const uint32_t b = in ? min((hi - comp_key(mine)) >> sh, (uint32_t)kThreads - 1u) : 0u;
      s.cnt[tid] = 0;
      __syncthreads();
      if (in) atomicAdd(&s.cnt[b], 1u);
      __syncthreads();
      const uint32_t c = s.cnt[tid], upto = ops.scan(c);
      s.cnt[tid] = upto - c;
      s.mass[tid] = (uint64_t)upto << 32 | (upto - c);
      __syncthreads();
      if (in) {
        from = (uint32_t)s.mass[b];
        to = (uint32_t)(s.mass[b] >> 32);
        s.win[atomicAdd(&s.cnt[b], 1u)] = mine;
      }
      __syncthreads();
    }
    if (in) {
      rank = from;
#pragma unroll 4
      for (uint32_t j = from; j < to; ++j) rank += s.win[j] < mine;
    }
    __syncthreads();
    if (in) s.win[rank] = mine;
    const double c = bmass + [&] {  // the scan's barrier also closes the writes above
      __syncthreads();
      return ops.scan(in ? weight(comp_key(s.win[tid])) : 0.0);
    }();
    if (in) s.wcum[tid] = c;
    __syncthreads();
  }

  // kOne: bins b0 .. b1 into the window; a token's rank is its bin's place in
  // the list and its rank among the bin's own tokens
  __device__ __forceinline__ void open_bins(uint32_t lo_, uint32_t base_, double bmass_, int b0_, int b1_, uint32_t n_) {
    lo = lo_, base = base_, bmass = bmass_, b0 = b0_, b1 = b1_, n = n_;
    __syncthreads();  // the last window's readers
    const uint64_t* list = lists + s.cc[b0];
    const bool in = tid < (int)n;
    double w = 0.0;
    if (in) {
      const uint64_t mine = list[tid];
      const int bin = bin_of(comp_key(mine), c8, J);
      uint32_t rank = s.cc[bin] - s.cc[b0];
      for (uint32_t j = rank, end = s.cc[bin + 1] - s.cc[b0]; j < end; ++j) rank += list[j] < mine;
      s.win[rank] = mine;
    }
    __syncthreads();
    if (in) w = weight(comp_key(s.win[tid]));
    w = bmass + ops.scan(w);
    if (in) s.wcum[tid] = w;
    __syncthreads();
  }

  __device__ __forceinline__ Cross from_window(int kind, double amount) {
    const bool in = tid < (int)n;
    const bool hit = in && (kind == kByCount    ? (double)(base + tid + 1) >= amount
                            : kind == kByMassGe ? s.wcum[tid] >= amount
                            : kind == kByMassGt ? s.wcum[tid] > amount
                                                : (double)comp_key(s.win[tid]) < amount);
    int pos = min(ops.first(hit), (int)n);
    if (kind != kByWeight) pos = min(pos + 1, (int)n);  // pos tokens of the window are in
    Cross r;
    r.n = base + pos;
    r.cum = pos > 0 ? s.wcum[pos - 1] : bmass;
    r.at = pos > 0 ? s.win[pos - 1] : 0;
    r.cut = pos < (int)n ? s.win[pos] : ((uint64_t)~lo + 1) << 32;
    return r;
  }

  // part `b` of a pass: (tokens, weight) before it, and its own tokens
  __device__ __forceinline__ uint32_t part_of(int b, uint32_t upto, double mass_upto, uint32_t c, double mass) {
    if (tid == b) {
      s.before_n = upto - c;
      s.before_m = mass_upto - mass;
      s.n = c;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(s.n);
  }

  __device__ __forceinline__ Cross locate(int kind, double amount) {
    // a sum within 2^-44 of the value counts as equal to it: rows of equal
    // logits meet dyadic settings exactly, and sums of one weight round (below
    // 2^-47)
    if (kind == kByMassGe) amount *= 1.0 - 0x1p-44;
    if (kind == kByMassGt) amount *= 1.0 + 0x1p-44;
    const bool hit = kind == kByCount    ? (double)s.cc[tid + 1] >= amount
                     : kind == kByMassGe ? s.cm[tid + 1] >= amount
                     : kind == kByMassGt ? s.cm[tid + 1] > amount
                                         : tid >= bin_of((uint32_t)amount, c8, J);
    int b = ops.first(hit);
    if (b >= kBins) {
      b = kTail;
      if (kind != kByWeight) {  // a sum that rounding left short: the last token above the tail
        kind = kByCount;
        amount = (double)s.cc[kTail];
        b = ops.first((double)s.cc[tid + 1] >= amount);
      }
    }
    if (b < b0 || b > b1) {
      uint32_t klo = b == kTail ? kKeyLowest : lowest_key(J - b, c8, t8);
      uint32_t khi = b == 0 ? kmax : lowest_key(J - b + 1.0, c8, t8) - 1u;
      uint32_t cb = __builtin_amdgcn_readfirstlane(s.cc[b]), nc = __builtin_amdgcn_readfirstlane(s.cc[b + 1]) - cb;
      double mb = readlane_f64(s.cm[b], 0);
      if (nc == 0) return Cross{cb, mb, ((uint64_t)~khi) << 32, 0};  // kByWeight: nothing in the threshold's own bin
      int B0 = b;
      bool whole = true;
      if (MODE != kSelf && (MODE == kAll || MODE == kOne || b < listed) && s.cc[b + 1] <= (uint32_t)kThreads) {  // everything down to this bin fits a window
        B0 = 0;
        khi = kmax;
        nc += cb;
        cb = 0;
        mb = 0.0;
      }
      while (nc > (uint32_t)kThreads) {
        whole = false;
        if (klo == khi) {  // one value: every token weighs w
          const double w = b == kTail ? 0.0 : weight(klo);
          double r = (double)nc;
          if (kind == kByCount) r = amount - cb;
          if (kind == kByMassGe || kind == kByMassGt) {
            r = fmin(fmax(floor((amount - mb) / w), 0.0), (double)nc);
            // the quotient is off by rounding only: settle it on the sums themselves
            if (r > 0.0 && (kind == kByMassGe ? fma(r - 1.0, w, mb) >= amount : fma(r - 1.0, w, mb) > amount)) r -= 1.0;
            if (r < (double)nc && !(kind == kByMassGe ? fma(r, w, mb) >= amount : fma(r, w, mb) > amount)) r += 1.0;
            r = fmax(r, 1.0);
          }
          if (kind == kByWeight && (double)klo < amount) return Cross{cb, mb, ((uint64_t)~klo) << 32, 0};
          const Cross x{cb + (uint32_t)r, fma(r, w, mb), 0, 0};
          // the index of the r-th of them
          uint32_t left = (uint32_t)r, ilo = 0, ihi = (uint32_t)z.V - 1;
          for (;;) {
            const uint32_t range = ihi - ilo;
            const int sh = max(0, 32 - (range ? __builtin_clz(range) : 32) - 9);
            pass(B0, b, klo, khi, ilo, ihi, sh, true);
            const uint32_t c = s.cnt[tid], upto = ops.scan(c);
            const int q = min(ops.first(upto >= left), kThreads - 1);
            part_of(q, upto, 0.0, c, 0.0);
            left -= s.before_n;
            ilo += (uint32_t)q << sh;
            if (sh == 0) break;
            ihi = min(ihi, ilo + ((1u << sh) - 1u));
          }
          const uint64_t at = ((uint64_t)~klo << 32) | ilo;
          return Cross{x.n, x.cum, at + 1, at};
        }
        const uint32_t range = khi - klo;
        const int sh = max(0, 32 - __builtin_clz(range) - 9);
        pass(B0, b, klo, khi, 0, 0xFFFFFFFFu, sh, false);
        // one bin holds one eighth of an octave: its unit is that of its lowest key
        const double unit = b == kTail ? 0.0 : pow2_eighth((int)fmax(rint(key_value(klo) * c8) - J, -16000.0)) * 0x1p-42;
        const uint32_t c = s.cnt[tid];
        const double mass = unit * (double)s.mass[tid];
        const uint32_t c1 = cb + ops.scan(c);
        const double m1 = mb + ops.scan(mass);
        const uint32_t n_part = (range >> sh) + 1;  // parts, from the highest key down
        const uint32_t low = (uint32_t)tid + 1 >= n_part ? klo : khi - ((uint32_t)tid << sh) - ((1u << sh) - 1u);
        const bool part_hit = (uint32_t)tid < n_part &&
                              (kind == kByCount    ? (double)c1 >= amount
                               : kind == kByMassGe ? m1 >= amount
                               : kind == kByMassGt ? m1 > amount
                                                   : (double)low < amount);
        int q = ops.first(part_hit);
        if (q >= (int)n_part) {  // every key passes, or rounding left the sum short of the last token
          part_of((int)n_part - 1, c1, m1, c, mass);
          if (kind == kByWeight) return Cross{s.before_n + s.n, s.before_m, ((uint64_t)~klo + 1) << 32, 0};
          kind = kByCount;
          amount = (double)(s.before_n + s.n);
          q = ops.first((uint32_t)tid < n_part && (double)c1 >= amount);
        }
        nc = part_of(q, c1, m1, c, mass);
        cb = __builtin_amdgcn_readfirstlane(s.before_n);
        mb = readlane_f64(s.before_m, 0);
        khi -= (uint32_t)q << sh;
        if ((uint32_t)q + 1 < n_part) klo = khi - ((1u << sh) - 1u);
        if (nc == 0) return Cross{cb, mb, ((uint64_t)~khi) << 32, 0};  // kByWeight: the threshold falls between tokens
        khi = min(khi, seen_hi);
        klo = max(klo, seen_lo);
      }
      if (MODE == kOne && whole) {
        open_bins(klo, cb, mb, B0, b, nc);
      } else {
        pass(B0, b, klo, khi, 0, 0xFFFFFFFFu, -1, false);
        open_window(klo, khi, cb, mb, whole ? B0 : 1, whole ? b : 0);
      }
    }
    return from_window(kind, amount);
  }

  // the row's cuts and draw, once s.cc and s.cm hold its bins
  __device__ __forceinline__ void answer(const RowParams& rp, uint32_t N, double u, int64_t row, const SampleOut& o,
                                         uint64_t* cut_out) {
    uint32_t kept = N;
    double Z = s.cm[kBins];
    uint64_t cut = ~0ull;
    // the cuts (0: top-k, 1: top-p, 2: min-p), the draw (3), and the last kept
    // token if rounding drew one behind it (4)
#pragma unroll 1
    for (int q = 0; q < 5; ++q) {
      int kind;
      double amount;
      if (q == 0) {
        if (rp.k >= (int64_t)N) continue;
        kind = kByCount, amount = (double)rp.k;
      } else if (q == 1) {
        if (!(rp.p < 1.0)) continue;
        kind = kByMassGe, amount = rp.p * Z;
      } else if (q == 2) {
        if (kmin == 0) continue;
        kind = kByWeight, amount = (double)kmin;
      } else if (q == 3) {
        if (tid == 0) {
          if (o.kept) o.kept[row] = (int32_t)kept;
          if (o.out) *cut_out = cut;
        }
        if (!o.token) break;
        kind = kByMassGt, amount = u * Z;
      } else {
        kind = kByCount, amount = (double)kept;
      }
      const Cross x = locate(kind, amount);
      if (q < 3) {
        if (x.n < kept) {
          kept = x.n;
          Z = x.cum;
          cut = x.cut;
        }
      } else if (q == 4 || (x.n <= kept && x.at != 0)) {
        // (u next to 1 may cross behind the kept tokens, where kFirst need not have
        // listed any: such a crossing counts only those before it)
        if (tid == 0) {
          o.token[row] = (int32_t)(uint32_t)x.at;
          if (o.prob) o.prob[row] = (float)(weight(comp_key(x.at)) / Z);
        }
        break;
      }
    }
  }
};

// The bins that a row's cuts and draw can need, from the bins' sums alone: a
// cut or draw whose amount depends on an earlier cut inside a bin takes the
// bins of that amount's bounds.  True if all are listed; else asks for them.
__device__ __forceinline__ bool bins_listed(FinLds& s, BlockOps& ops, const RowParams& rp, uint32_t N, bool draw,
                                            double u, double J, uint32_t kmax, uint32_t kmin, int listed, uint32_t ask_cap, SampleAsk& ask) {
  const double c8 = rp.c8, t8 = rp.t8;
  constexpr double kLess = 1.0 - 0x1p-40, kMore = 1.0 + 0x1p-40;
  const int tid = threadIdx.x;
  const double total = s.cm[kBins], after = s.cm[tid + 1];
  int need0 = kBins, need1 = -1, cut1 = kTail;  // bins of cuts; the latest bin the kept tokens can end in
  double zlo = total, zhi = total;
  bool any = false;
  int bk = -1;
  if (rp.k < (int64_t)N) {
    bk = ops.first(s.cc[tid + 1] >= (uint32_t)rp.k);
    cut1 = bk;
    zlo = s.cm[bk];
    zhi = s.cm[bk + 1];
    need0 = need1 = bk;
    any = true;
  }
  if (rp.p < 1.0) {
    const int p0 = min(ops.first(after >= rp.p * zlo * kLess), kTail);
    const int p1 = min(ops.first(after >= rp.p * zhi * kMore), kTail);
    need0 = min(need0, p0);
    need1 = max(need1, min(p1, cut1));
    cut1 = min(cut1, p1);
    zlo = fmin(zlo, s.cm[p0]);
    zhi = s.cm[cut1 + 1];
    any = true;
  }
  if (kmin != 0) {
    const int bm = bin_of(kmin, c8, J);
    if (bm <= cut1) {
      need0 = min(need0, bm);
      need1 = max(need1, bm);
      cut1 = bm;
      zlo = fmin(zlo, s.cm[bm]);
      zhi = s.cm[cut1 + 1];
      any = true;
    }
  }
  int d0 = kBins, d1 = -1;
  if (draw) {
    d0 = min(ops.first(after > u * zlo * kLess), cut1);
    d1 = min(ops.first(after > u * zhi * kMore), cut1);
  }
  if (need1 < listed && d1 < listed) return true;
  if (!any) {
    need0 = d0;
    need1 = d1;
  } else if (draw && d1 >= need0 && d0 <= need1) {
    need0 = min(need0, d0);
    need1 = max(need1, d1);
    d1 = -1;
  }
  if (!any) d1 = -1;
  const uint32_t count = s.cc[need1 + 1] - s.cc[need0] + (d1 >= 0 ? s.cc[d1 + 1] - s.cc[d0] : 0u);
  if (d1 < 0) d0 = kBins;
  // keys of the two ranges of bins (an empty second one: none)
  const uint32_t l0 = need1 == kTail ? kKeyLowest : lowest_key(J - need1, c8, t8), h0 = need0 == 0 ? kmax : lowest_key(J - need0 + 1.0, c8, t8) - 1u;
  uint32_t l1 = 1, h1 = 0;
  if (d1 >= 0) {
    l1 = d1 == kTail ? kKeyLowest : lowest_key(J - d1, c8, t8);
    h1 = d0 == 0 ? kmax : lowest_key(J - d0 + 1.0, c8, t8) - 1u;
  }
  if (tid == 0) {
    ask.kind = count <= ask_cap ? kSampleAskBins : kSampleAskRow;
    ask.n = 0;
    ask.b0[0] = need0, ask.b1[0] = need1, ask.klo[0] = l0, ask.khi[0] = h0;
    ask.b0[1] = d0, ask.b1[1] = d1, ask.klo[1] = l1, ask.khi[1] = h1;
  }
  return false;
}

__device__ __forceinline__ void empty_row(int64_t row, const SampleOut& o, uint64_t* cut_out) {
  if (threadIdx.x == 0) {
    if (o.token) o.token[row] = -1;
    if (o.prob) o.prob[row] = 0.0f;
    if (o.kept) o.kept[row] = 0;
    if (o.out) *cut_out = 0;
  }
}
__device__ __forceinline__ double row_uniform(const SampleOut& o, int64_t row) {
  const double u = o.token ? o.u[row] : 0.0;
  return u > 0.0 ? fmin(u, 1.0 - 0x1p-53) : 0.0;  // NaN: 0
}

// One block a row: bound by the latency of its steps (the segments' bins as
// other blocks left them in memory, then scans, windows and searches).  One row
// of 151936 fp32 takes 13 us (top-p); 256 of 262144 14 to 20 in kFirst and 20 in
// kSecond, 1024 of 32000 26 to 35 and 13 to 34 by their settings.  kSecond at 128
// registers keeps two blocks a CU; with one it took a third longer.
template <int MODE>
__global__ __launch_bounds__(kThreads, MODE == kSecond ? 4 : 2) void sample_finalize_kernel(SampleArgs a, int64_t row0, int n_seg, int cap, uint32_t ask_cap,
                                                                   const SamplePart* __restrict__ parts,
                                                                   const uint64_t* __restrict__ lists,
                                                                   SampleAsk* __restrict__ asks, const uint64_t* __restrict__ asked,
                                                                   SampleOut o, uint64_t* __restrict__ cuts) {
  if constexpr (MODE == kSecond) {
    if (asks[blockIdx.x].kind == kSampleAskNone) return;
  }
  __shared__ FinLds s;
  BlockOps ops(s.red);
  const int tid = threadIdx.x;
  const int64_t row = row0 + blockIdx.x;
  const RowParams rp = row_params(a, row);
  const SamplePart* part = parts + (size_t)blockIdx.x * n_seg;
  if (MODE == kFirst && tid == 0) asks[blockIdx.x].kind = kSampleAskNone;

  // the segments' headers, one thread each (n_seg <= kMaxSeg = kThreads)
  const bool have = tid < n_seg;
  const double Js = have ? part[tid].J : -INFINITY;
  const uint32_t ns = have ? part[tid].n : 0;
  const int nbs = have ? part[tid].nb : 0, ls = have ? part[tid].listed : kBins;
  const double ms = have ? (double)part[tid].max : -INFINITY;
  const double u = row_uniform(o, row);
  const double J = ops.max(Js);
  const float m = (float)ops.max(ms);
  const uint32_t N = ops.sum(ns);
  if (N == 0) return empty_row(row, o, cuts + blockIdx.x);  // every token masked
  const int shift = ns ? (int)fmin(J - Js, (double)kBins) : kBins;
  if (have) {
    s.shift[tid] = (int16_t)shift;
    s.nb[tid] = (int16_t)nbs;
    s.n_seg[tid] = ns;
  }
  // bins whose tokens are all listed: as far as every segment's list reaches
  const int listed = kBins - (int)ops.max((double)(kBins - (ls >= kBins ? kBins : min(kBins, ls + shift))));
  // the segments' bins on the row's grid, in segment order
  uint32_t cs = 0;
  double mass = 0.0;
#pragma unroll 8
  for (int g = 0; g < n_seg; ++g) {
    const int b = tid - s.shift[g];
    const bool in = tid < kTail && b >= 0 && b < s.nb[g];
    cs += in ? part[g].upto[b] : b < 0 ? 0u : s.n_seg[g];
    mass += in ? part[g].mass[b] : 0.0;
  }
  const double cum = ops.scan(mass * pow2_eighth(-tid));
  if (tid == kTail) cs = N;  // the tail bin: whatever is left
  s.cc[tid + 1] = cs;
  s.cm[tid + 1] = cum;
  if (tid == 0) {
    s.cc[0] = 0;
    s.cm[0] = 0.0;
  }
  __syncthreads();

  const uint32_t kmax = key_of(m, RowType<DFLASH_F32>::kMax), kmin = least_key(rp.m, kmax, rp.c8, rp.t8);
  Finalize<DFLASH_F32, MODE> f{s, ops, RowRef<DFLASH_F32>(a.Z, row, a.stride, a.V), part, lists + (size_t)blockIdx.x * n_seg * cap,
                               MODE == kSecond ? asked + (size_t)blockIdx.x * ask_cap : nullptr,
                               MODE == kSecond ? asks + blockIdx.x : nullptr, ask_cap, n_seg, cap, rp.c8, rp.t8, J, tid, kmax, kmin, listed,
                               0, 0, 0.0, 1, 0, 0, 0, 0};
  if constexpr (MODE == kFirst) {
    if (!bins_listed(s, ops, rp, N, o.token != nullptr, u, J, kmax, kmin, listed, ask_cap, asks[blockIdx.x])) return;
  }
  f.answer(rp, N, u, row, o, cuts + blockIdx.x);
}

// a slot of the filtered row: the tokens before `cut` stay
template <int DT>
__device__ __forceinline__ void store_filtered(typename RowType<DT>::elem* o, int V, int slot, const Slot& x, uint64_t cut,
                                               uint32_t fill) {
  constexpr int VE = RowType<DT>::VE;
  Slot y;
#pragma unroll
  for (int k = 0; k < 4; ++k) y.w[k] = 0;
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    const float v = slot_value<DT>(x, i);
    const bool in = v > kNegInf && comp_of(key_of(v, RowType<DT>::kMax), (uint32_t)(slot * VE + i)) < cut;
    if constexpr (DT == DFLASH_BF16) {
      const uint32_t raw = (i & 1) ? x.w[i >> 1] >> 16 : x.w[i >> 1] & 0xFFFFu;
      y.w[i >> 1] |= (in ? raw : fill) << ((i & 1) * 16);
    } else {
      y.w[i] = in ? x.w[i] : fill;
    }
  }
  store_slot<DT>(o, V, slot, y);
}

// ---------------------------------------------------------------- short rows in one launch

// A row of up to 8192 tokens in one block, NL slots a thread: bins, list and
// answer stay in LDS, and the filtered row is written at once.  Bound by the
// chain of steps: one row of 1024 fp32 takes 7.5 us (12.9 in two launches), 2048
// of 1000 35 to 43 by their settings (82); one row of 8000 11 (15), 2048 rows 112
// to 175 (180), as the list of four slots a thread leaves a CU one block (96 KB).
template <int DT, int NL>
__global__ __launch_bounds__(kThreads, 4) void sample_row_kernel(SampleArgs a, SampleOut o) {
  constexpr int VE = RowType<DT>::VE;
  constexpr float kMax = RowType<DT>::kMax;
  __shared__ FinLds s;
  __shared__ uint32_t next[kBins];
  __shared__ unsigned long long cell[kBins * kCols > kThreads * NL * VE ? kBins * kCols : kThreads * NL * VE];  // then the list
  __shared__ uint64_t cut;
  BlockOps ops(s.red);
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const RowParams rp = row_params(a, row);
  const RowRef<DT> z(a.Z, row, a.stride, a.V);
  const double c8 = rp.c8, u = row_uniform(o, row);
  Slot x[NL];
#pragma unroll
  for (int l = 0; l < NL; ++l) x[l] = z.load(tid + l * kThreads);
#pragma unroll
  for (int c = 0; c < kCols; ++c) cell[c * kBins + tid] = 0;
  float m = kNegInf;
#pragma unroll
  for (int l = 0; l < NL; ++l)
#pragma unroll
    for (int i = 0; i < VE; ++i) m = fmaxf(m, slot_value<DT>(x[l], i));
  m = (float)ops.max((double)fminf(m, kMax));
  if (m == kNegInf) {
    empty_row(row, o, &cut);
  } else {
    const double J = rint((double)m * c8);
    add_cells<DT>(cell, x, J, rp);
    __syncthreads();
    uint32_t c, cs;
    const unsigned long long f = read_cells(cell, tid, c);
    cs = c;
    double cum = tid < kTail ? (double)f * 0x1p-42 * pow2_eighth(-tid) : 0.0;
    ops.scan(cs, cum);
    s.cc[tid + 1] = cs;
    s.cm[tid + 1] = cum;
    next[tid] = cs - c;
    if (tid == 0) {
      s.cc[0] = 0;
      s.cm[0] = 0.0;
    }
    __syncthreads();
    uint64_t* list = reinterpret_cast<uint64_t*>(cell);
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float v = slot_value<DT>(x[l], i);
        if (v > kNegInf) list_token(next, list, c8, J, comp_of(key_of(v, kMax), (uint32_t)((tid + l * kThreads) * VE + i)));
      }
    __syncthreads();
    const uint32_t kmax = key_of(m, kMax);
    Finalize<DT, kOne> fin{s, ops, z, nullptr, list, nullptr, nullptr, 0, 1, 0, c8, rp.t8, J, tid, kmax, least_key(rp.m, kmax, c8, rp.t8), kBins, 0, 0, 0.0, 1, 0, 0, 0, 0};
    fin.answer(rp, s.cc[kBins], u, row, o, &cut);
  }
  if (o.out) {
    __syncthreads();
    typename RowType<DT>::elem* out = static_cast<typename RowType<DT>::elem*>(o.out) + row * o.out_stride;
#pragma unroll
    for (int l = 0; l < NL; ++l) store_filtered<DT>(out, a.V, tid + l * kThreads, x[l], cut, o.fill);
  }
}

// ---------------------------------------------------------------- (3) the tokens that rows asked for

// Reads the rows that asked a second time (256 x 262144 fp32 if all do: 44 us, 6.1
// TB/s, the memory's rate; 26 of plain temperature, 14 of mixed requests).
template <int NL>
__global__ __launch_bounds__(kThreads) void sample_gather_kernel(SampleArgs a, int64_t row0, int n_seg, uint32_t ask_cap,
                                                                 SampleAsk* __restrict__ asks, uint64_t* __restrict__ asked) {
  constexpr int DT = DFLASH_F32, VE = RowType<DT>::VE;
  const int r = blockIdx.x / n_seg, seg = blockIdx.x % n_seg, tid = threadIdx.x;
  SampleAsk& ask = asks[r];
  if (ask.kind != kSampleAskBins) return;
  __shared__ uint16_t place[kThreads * NL * VE];  // in the segment
  __shared__ uint32_t n, at;
  if (tid == 0) n = 0;
  __syncthreads();
  const RowRef<DT> z(a.Z, row0 + r, a.stride, a.V);
  const int s0 = seg * (kThreads * NL) + tid;
  // a range may hold no key at all: at a tiny T values are bins apart
  const uint32_t l0 = ask.klo[0], w0 = ask.khi[0] - l0, l1 = ask.klo[1], w1 = ask.khi[1] - l1;
  const bool one = ask.khi[0] >= l0, two = ask.khi[1] >= l1;
  Slot x[NL];
#pragma unroll
  for (int l = 0; l < NL; ++l) x[l] = z.load(s0 + l * kThreads);
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float v = slot_value<DT>(x[l], i);
      const uint32_t key = key_of(v, RowType<DT>::kMax);
      hits |= (uint32_t)(v > kNegInf && ((one && key - l0 <= w0) || (two && key - l1 <= w1))) << i;
    }
    if (hits) {
      uint32_t i = atomicAdd(&n, (uint32_t)__popc(hits));
      do {
        place[i++] = (uint16_t)((tid + l * kThreads) * VE + __builtin_ctz(hits));
        hits &= hits - 1;
      } while (hits);
    }
  }
  __syncthreads();
  const uint32_t c = n;
  if (tid == 0) at = atomicAdd(&ask.n, c);  // the tokens' order in the row's buffer does not matter
  __syncthreads();
  uint64_t* out = asked + (size_t)r * ask_cap;
  for (uint32_t i = tid; i < c && at + i < ask_cap; i += kThreads) {
    const uint32_t idx = (uint32_t)(seg * (kThreads * NL * VE)) + place[i];
    out[at + i] = comp_of(key_of(row_value<DT>(z, (int)idx), RowType<DT>::kMax), idx);
  }
}

// ---------------------------------------------------------------- bf16 rows: counts of values
// The items of a segment, in the order of the row's tokens: item 0 counts
// positive values over the range (+inf too), 1 .. kMags the positive values
// downwards, kMid all that lie nearer to zero (zeros are counted, the others
// listed one by one), then the negative values, kLow
// the finite values under the range; masked tokens are not counted.  The range
// depends on T alone, so that a row's segments agree: kMags magnitudes (23
// binades) below a power of two over 100 T, at least 128.  A row whose
// largest logit lies over it, or that has logits under it which still weigh
// (within 512 eighths of an octave of the largest), is not counted but binned.
constexpr int kMags = 2944;
constexpr int kMid = kMags + 1, kLow = 2 * kMags + 2;

// A segment's counters: for either sign kSide by magnitude (0: nearer to zero,
// kMags + 1: over the range), then the tokens under the range.  In memory the
// two near zero hold the listed tokens and the zeros, and added up for a row
// the first of them holds both.
constexpr int kSide = (kMags + 2 + 3) / 4 * 4, kUnder = 2 * kSide;
static_assert(kUnder + 4 <= kSampleItems, "");
__device__ __forceinline__ int counter_of(int item) { return item <= kMid ? kMid - item : kSide + item - kMid; }

// The finish adds up the items in runs, one a thread
constexpr int kRun = 12;
static_assert(kLow < kRun * kThreads && kRun <= 16, "");

// smallest magnitude (bit pattern) with a counter of its own
__device__ __forceinline__ uint32_t value_base(double c8) {
  const double T = 8.0 * 1.4426950408889634 / c8;  // c8 = 0: inf
  const uint32_t e = (__float_as_uint((float)fmin(fmax(100.0 * T, 64.0), 1.7e38)) >> 23) + 1u;
  return min(e << 7, 0x7F80u) - (uint32_t)kMags;
}

// One LDS atomic a token, two tokens a word formed side by side in 16-bit
// halves.  512 x 262144 bf16 take 68 us, 3.9 TB/s; the loads alone 53, without
// the atomics 65, the atomics alone (random addresses) 28: issue slots and LDS
// share the time.  Not faster: nontemporal loads (81), 8 loads in flight (86
// against 84 then), 16.
__global__ __launch_bounds__(kThreads) void sample_values_kernel(SampleArgs a, int64_t row0, int n_seg, int seg_slots,
                                                                 SampleValues* __restrict__ parts) {
  constexpr int VE = 8, U = 4;
  // the tokens under the range have a counter a lane (equal addresses queue up)
  constexpr int kCounters = kUnder + 64;
  __shared__ __align__(16) uint32_t count[kCounters];
  __shared__ uint32_t n_odd, n_zero;
  const int tid = threadIdx.x, lane = tid & 63, seg = blockIdx.x % n_seg;
  const int64_t row = row0 + blockIdx.x / n_seg;
  const RowRef<DFLASH_BF16> z(a.Z, row, a.stride, a.V);
  const int begin = seg * seg_slots, end = min(begin + seg_slots, z.slots());
  const uint32_t base = value_base(row_params(a, row).c8);
  for (int i = tid; i < kCounters; i += kThreads) count[i] = 0;
  if (tid == 0) n_odd = n_zero = 0;
  __syncthreads();
  const uint32_t near2 = (base - 1u) * 0x10001u, over2 = (uint32_t)(kMags + 1) * 0x10001u, side2 = (uint32_t)kSide * 0x10001u;
  auto add = [&](const Slot& x) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t w = x.w[d];
      const uint32_t mag = subsat_u16x2(w & 0x7FFF7FFFu, near2), e = min_u16x2(mag, over2);
      const uint32_t neg = __builtin_bit_cast(uint32_t, __builtin_bit_cast(s16x2, w) >> (s16x2)(15));
      uint32_t i = __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, e) + __builtin_bit_cast(u16x2, neg & side2));
      if (subsat_u16x2(mag, over2 - 0x10001u)) {
        // a token out of the range: masked ones (-inf, NaN) are not counted,
        // those under the range go to the lane's counter
        const uint32_t lo = w & 0xFFFFu, hi = w >> 16;
        const bool ol = (e & 0xFFFFu) > (uint32_t)kMags, oh = (e >> 16) > (uint32_t)kMags;
        const auto masked = [](uint32_t h) { return h == 0xFF80u || (h & 0x7FFFu) > 0x7F80u; };
        if (ol && (lo >> 15)) i = (i & 0xFFFF0000u) | (uint32_t)(kUnder + lane);
        if (oh && (hi >> 15)) i = (i & 0xFFFFu) | (uint32_t)(kUnder + lane) << 16;
        if (!(ol && masked(lo))) atomicAdd(&count[i & 0xFFFFu], 1u);
        if (!(oh && masked(hi))) atomicAdd(&count[i >> 16], 1u);
      } else {
        atomicAdd(&count[i & 0xFFFFu], 1u);
        atomicAdd(&count[i >> 16], 1u);
      }
    }
  };
#pragma unroll 1
  for (int sl = begin + tid; sl < end; sl += U * kThreads) {
    Slot x[U];
#pragma unroll
    for (int l = 0; l < U; ++l) x[l] = z.load(min(sl + l * kThreads, end));
#pragma unroll
    for (int l = 0; l < U; ++l)
      if (sl + l * kThreads < end) add(x[l]);
  }
  __syncthreads();
  SampleValues& out = parts[blockIdx.x];
  if (count[0] + count[kSide] != 0) {  // tokens near zero: find them again
    uint32_t zeros = 0;
#pragma unroll 1
    for (int sl = begin + tid; sl < end; sl += U * kThreads) {
      Slot x[U];
#pragma unroll
      for (int l = 0; l < U; ++l) x[l] = z.load(min(sl + l * kThreads, end));
#pragma unroll
      for (int l = 0; l < U; ++l)
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const uint32_t w = (i & 1) ? x[l].w[i >> 1] >> 16 : x[l].w[i >> 1] & 0xFFFFu;
          if ((w & 0x7FFFu) < base && sl + l * kThreads < end) {
            if ((w & 0x7FFFu) == 0) {
              ++zeros;
            } else {
              const uint32_t at = atomicAdd(&n_odd, 1u);
              if (at < (uint32_t)kSampleOdd) out.odd[at] = w << 16 | (uint32_t)((sl + l * kThreads - begin) * VE + i);
            }
          }
        }
    }
    zeros = wave_sum_u32(zeros);
    if (lane == 0 && zeros) atomicAdd(&n_zero, zeros);
    __syncthreads();  // every thread has read the two counters, too
    if (tid == 0) {
      count[0] = n_odd;
      count[kSide] = n_zero;
    }
    __syncthreads();
  }
  uint2* counts = reinterpret_cast<uint2*>(out.counts);
  for (int j = tid; j < kUnder / 4; j += kThreads) {
    const uint4 c = reinterpret_cast<const uint4*>(count)[j];
    counts[j] = make_uint2(c.x | c.y << 16, c.z | c.w << 16);
  }
  if (tid < 64) {
    const uint32_t under = wave_sum_u32(count[kUnder + tid]);
    if (tid == 0) counts[kUnder / 4] = make_uint2(under, 0);
  }
}

struct ValLds {
  __align__(16) uint32_t c[kSampleItems];  // the row's counters
  uint32_t rc[kThreads + 1];  // tokens before each run
  double rm[kThreads + 1];    // and their weight
  uint64_t win[kThreads];     // the tokens near zero, sorted; the zeros are one entry
  uint32_t ncum[kThreads];    // their running count
  double wcum[kThreads];      // and weight
  Red red;
  uint32_t n;
  uint32_t idx;
};
union RowLds {
  ValLds v;
  FinLds f;
  __device__ RowLds() {}
};

// where a running count or sum crosses a value: an item and a place in it
struct ValueCross {
  uint32_t n;   // tokens up to and including the crossing one (kByWeight: tokens that pass)
  double cum;   // their weight
  int item;
  uint32_t r;   // tokens of this item (kMid: of this entry) among them
  int e;        // kMid: the entry
};

struct Values {
  ValLds& s;
  BlockOps& ops;
  const RowRef<DFLASH_BF16> z;
  const SampleValues* part;
  const int n_seg, seg_slots, tid;
  const double c;        // log2(e) / T
  const uint32_t base;
  double m;              // the largest logit
  int n_mid;             // entries near zero
  uint32_t n_in;         // tokens in the range

  // the logit of a counted value
  __device__ __forceinline__ float value(int item) const {
    const int mag = (int)base + (item < kMid ? kMags - item : item - kMid - 1);
    const float v = __uint_as_float((uint32_t)mag << 16);
    return item < kMid ? v : -v;
  }
  // relative to the row's largest token, whose weight is exactly 1
  __device__ __forceinline__ double weight(double v) const { return exp2_full((v - m) * c); }
  __device__ __forceinline__ double near_value(uint32_t i) const { return key_value(comp_key(s.win[i])); }

  // tokens of an item
  __device__ __forceinline__ uint32_t tokens(int item) const { return s.c[counter_of(item)]; }

  __device__ __forceinline__ ValueCross locate(int kind, double amount) {
    // a sum within 2^-44 of the value counts as equal to it: rows of equal
    // logits meet dyadic settings exactly, and sums of one weight round (below
    // 2^-47)
    if (kind == kByMassGe) amount *= 1.0 - 0x1p-44;
    if (kind == kByMassGt) amount *= 1.0 + 0x1p-44;
    bool hit = false;
    if (tid <= kLow / kRun) {
      const bool some = s.rc[tid + 1] != s.rc[tid];
      if (kind == kByCount) hit = (double)s.rc[tid + 1] >= amount;
      else if (kind == kByMassGe) hit = some && s.rm[tid + 1] >= amount;
      else if (kind == kByMassGt) hit = some && s.rm[tid + 1] > amount;
      else {  // the run's last value passes or not, present or not
        const int item = min(tid * kRun + kRun - 1, kLow - 1);
        hit = weight(item == kMid ? (n_mid ? near_value(n_mid - 1) : 0.0) : (double)value(item)) < amount;
      }
    }
    int g = ops.first(hit);
    const bool none = g >= kThreads;
    if (none) {
      if (kind == kByWeight) return ValueCross{n_in, s.rm[kThreads], -1, 0, 0};
      g = ops.first(s.rc[tid + 1] >= n_in);  // rounding left the sum short: the last token
    }
    // every wave works the run out for itself, an item a lane
    const int lane = lane_id(), item = g * kRun + lane;
    const uint32_t n0 = s.rc[g], in_run = s.rc[g + 1] - n0;
    const double m0 = s.rm[g];
    const bool own = lane < kRun && item < kLow;
    const uint32_t c = own ? tokens(item) : 0u;
    const double w = item != kMid ? weight((double)value(item)) : weight(n_mid ? near_value(n_mid - 1) : 0.0);
    const uint32_t upto = row16_scan_u32(c);
    const double cum = row16_scan_f64(c ? (item != kMid ? (double)c * w : s.wcum[n_mid - 1]) : 0.0);
    bool cross;
    if (kind == kByWeight) {
      cross = own && item > 0 && w < amount;
    } else {
      const bool last = upto == in_run;
      cross = c != 0 && (none ? last
                         : kind == kByCount    ? (double)(n0 + upto) >= amount
                         : kind == kByMassGe ? m0 + cum >= amount || last
                                             : m0 + cum > amount || last);
    }
    const int l = min(first_lane(cross), kRun - 1), li = g * kRun + l;
    const uint32_t lc = __builtin_amdgcn_readlane(c, l), n1 = n0 + __builtin_amdgcn_readlane(upto, l) - lc;  // before the item
    const double lw = readlane_f64(w, l), before = m0 + (l > 0 ? readlane_f64(cum, max(l - 1, 0)) : 0.0);
    if (li == kMid && lc) {  // among the entries near zero
      const bool h = tid < n_mid && (kind == kByCount    ? (double)(n1 + s.ncum[tid]) >= amount
                                     : kind == kByMassGe ? before + s.wcum[tid] >= amount
                                     : kind == kByMassGt ? before + s.wcum[tid] > amount
                                                         : weight(near_value(tid)) < amount);
      int e = ops.first(h);
      if (kind == kByWeight) {  // up to the last entry that passes
        e = min(e, n_mid);
        const uint32_t n = e ? s.ncum[e - 1] : 0u;
        return ValueCross{n1 + n, e ? before + s.wcum[e - 1] : before, kMid, e > 1 ? n - s.ncum[e - 2] : n, max(e - 1, 0)};
      }
      e = none ? n_mid - 1 : min(e, n_mid - 1);
      const uint32_t n = e ? s.ncum[e - 1] : 0u, c1 = s.ncum[e] - n;
      const double b = e ? before + s.wcum[e - 1] : before;
      const double w1 = weight(near_value(e)), r = none ? (double)c1 : place(kind, amount, n1 + n, b, w1, c1);
      return ValueCross{n1 + n + (uint32_t)r, fma(r, w1, b), kMid, (uint32_t)r, e};
    }
    if (kind == kByWeight) return ValueCross{n1, before, li, 0, 0};
    const double r = none ? (double)lc : place(kind, amount, n1, before, lw, lc);
    return ValueCross{n1 + (uint32_t)r, fma(r, lw, before), li, (uint32_t)r, 0};
  }

  // the first of c tokens of weight w, behind n tokens of the weight `before`,
  // at which the crossing falls (from 1)
  __device__ __forceinline__ double place(int kind, double amount, uint32_t n, double before, double w, uint32_t c) const {
    if (kind == kByCount) return amount - (double)n;
    double r = fmin(fmax(floor((amount - before) / w), 0.0), (double)c);
    // the quotient is off by rounding only: settle it on the sums themselves
    if (r > 0.0 && (kind == kByMassGe ? fma(r - 1.0, w, before) >= amount : fma(r - 1.0, w, before) > amount)) r -= 1.0;
    if (r < (double)c && !(kind == kByMassGe ? fma(r, w, before) >= amount : fma(r, w, before) > amount)) r += 1.0;
    return fmax(r, 1.0);
  }

  __device__ __forceinline__ uint32_t item_key(const ValueCross& x) const {
    if (x.item == kMid) return n_mid ? comp_key(s.win[x.e]) : kKeyZero;
    return ord32(__float_as_uint(value(x.item)));
  }

  // index of the r-th (from 1) token of x's item, in index order
  __device__ __forceinline__ uint32_t index_of(const ValueCross& x, uint32_t r) {
    const bool zero = x.item == kMid;
    if (zero && comp_key(s.win[x.e]) != kKeyZero) return (uint32_t)s.win[x.e];
    // its segment, by the segments' own counts (n_seg <= kThreads)
    const uint32_t has = tid < n_seg ? part[tid].counts[zero ? kSide : counter_of(x.item)] : 0u, sc = ops.scan(has);
    const int g = min(ops.first(sc >= r), n_seg - 1);
    if (tid == g) s.n = sc - has;
    __syncthreads();
    r -= s.n;
    const uint32_t want = zero ? 0u : __float_as_uint(value(x.item)) >> 16, bits = zero ? 0x7FFFu : 0xFFFFu;
    // the segment in order, four slots a thread at a time, up to the r-th
    const int end = min((g + 1) * seg_slots, z.slots());
#pragma unroll 1
    for (int s0 = g * seg_slots; s0 < end; s0 += 4 * kThreads) {
      const int sl = s0 + 4 * tid;
      uint32_t mask = 0;
      Slot y[4];
#pragma unroll
      for (int l = 0; l < 4; ++l) y[l] = z.load(min(sl + l, end));
#pragma unroll
      for (int l = 0; l < 4; ++l)
#pragma unroll
        for (int d = 0; d < 4; ++d)
          mask |= ((uint32_t)((y[l].w[d] & bits) == want) | (uint32_t)((y[l].w[d] >> 16 & bits) == want) << 1) << (8 * l + 2 * d);
      if (sl + 4 > end) mask &= sl < end ? (1u << 8 * (end - sl)) - 1u : 0u;
      const uint32_t found = (uint32_t)__popc(mask), upto = ops.scan(found);
      const int t = ops.first(upto >= r);
      if (t < kThreads) {
        if (tid == t) {
          for (uint32_t left = r - (upto - found); left > 1; --left) mask &= mask - 1u;
          s.idx = (uint32_t)(sl * 8 + __builtin_ctz(mask));
        }
        break;
      }
      r -= ops.sum(found);
    }
    __syncthreads();
    return s.idx;
  }
};

// one bf16 row from its segments' counts; false if the row has to be binned
__device__ __forceinline__ bool finalize_values(ValLds& s, const SampleArgs& a, int64_t row, int n_seg, int seg_slots,
                                                const SampleValues* __restrict__ part, const SampleOut& o, uint64_t* cut_out) {
  constexpr int VE = 8, kMine = kSampleItems / 4 / kThreads;
  static_assert(kSampleItems == kMine * 4 * kThreads, "");
  BlockOps ops(s.red);
  const int tid = threadIdx.x;
  const RowParams rp = row_params(a, row);
  const double c8 = rp.c8, u = row_uniform(o, row);
  const uint32_t base = value_base(c8);
  // the segments' counts, four counters a thread at a time (what lies behind
  // the last counter is not used)
  uint4 c[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) c[j] = make_uint4(0, 0, 0, 0);
  constexpr int kBatch = 5;  // segments whose loads are on their way together
#pragma unroll 1
  for (int g0 = 0; g0 < n_seg; g0 += kBatch) {
    uint2 v[kBatch][kMine];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        v[b][j] = g0 + b < n_seg ? reinterpret_cast<const uint2*>(part[g0 + b].counts)[tid + j * kThreads] : make_uint2(0, 0);
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        c[j].x += v[b][j].x & 0xFFFFu;
        c[j].y += v[b][j].x >> 16;
        c[j].z += v[b][j].y & 0xFFFFu;
        c[j].w += v[b][j].y >> 16;
      }
  }
  int top = kLow;  // the first item with a token: the row's largest
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int q = 4 * (tid + j * kThreads);
    reinterpret_cast<uint4*>(s.c)[tid + j * kThreads] = c[j];
    if (q < kUnder) {
      const int sign = q < kSide ? -1 : 1, item = q < kSide ? kMid - q : kMid + q - kSide;
      top = min(top, c[j].x ? item : kLow);
      top = min(top, c[j].y ? item + sign : kLow);
      top = min(top, c[j].z ? item + 2 * sign : kLow);
      top = min(top, c[j].w ? item + 3 * sign : kLow);
    }
  }
  if (tid == 0) s.n = 0;
  top = kLow - (int)ops.max((uint32_t)(kLow - top));
  const uint32_t n_near = s.c[0], n_zero = s.c[kSide], n_low = s.c[kUnder], n_over = s.c[kMags + 1];
  const uint32_t n_mid = n_near + (n_zero != 0);  // entries
  __syncthreads();
  if (tid == 0) s.c[0] = n_near + n_zero;
  if (n_over || n_mid > (uint32_t)kThreads) return false;
  if (n_mid) {
    // from the segments' lists; too many in one segment: not listed
    bool full = false;
    for (int g = tid; g < n_seg; g += kThreads) {
      const uint32_t k = part[g].counts[0];
      full |= k > (uint32_t)kSampleOdd;
      if (k && k <= (uint32_t)kSampleOdd) {
        uint32_t at = atomicAdd(&s.n, k);
#pragma unroll 1
        for (uint32_t j = 0; j < k && at < (uint32_t)kThreads; ++j, ++at) {
          const uint32_t e = part[g].odd[j];
          s.win[at] = comp_of(ord32_canon(e & 0xFFFF0000u), (uint32_t)(g * seg_slots * VE) + (e & 0xFFFFu));
        }
      }
    }
    if (tid == 0 && n_zero) s.win[n_mid - 1] = comp_of(kKeyZero, 0);
    if (ops.first(full) < kThreads) return false;
    __syncthreads();
    const bool in = tid < (int)n_mid;
    const uint64_t me = in ? s.win[tid] : 0;
    uint32_t rank = 0;
    if ((tid & ~63) < (int)n_mid) {
#pragma unroll 4
      for (uint32_t j = 0; j < n_mid; ++j) rank += s.win[j] < me;
    }
    __syncthreads();
    if (in) s.win[rank] = me;
    __syncthreads();
  }
  Values f{s, ops, RowRef<DFLASH_BF16>(a.Z, row, a.stride, a.V), part, n_seg, seg_slots, tid, c8 * 0.125, base, 0.0, (int)n_mid, 0};
  if (top >= kLow) {
    if (n_low) return false;
    empty_row(row, o, cut_out);
    return true;
  }
  const double m = top == kMid ? f.near_value(0) : (double)f.value(top);
  if (n_low && m - 512.0 / c8 < -(double)__uint_as_float(min((base + (uint32_t)kMags) << 16, 0x7F7F0000u))) return false;
  f.m = m;
  if (n_mid) {
    const uint32_t c = tid >= (int)n_mid ? 0u : comp_key(s.win[tid]) == kKeyZero ? n_zero : 1u, nc = ops.scan(c);
    const double wc = ops.scan(c ? (double)c * f.weight(f.near_value(tid)) : 0.0);
    if (c) {
      s.ncum[tid] = nc;
      s.wcum[tid] = wc;
    }
    __syncthreads();
  }
  // each run's tokens and weight, then before each run
  uint32_t n = 0;
  double sum = 0.0;
  if (tid <= kLow / kRun) {
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const int item = tid * kRun + k;
      const uint32_t c = f.tokens(item);
      double all = (double)c * f.weight((double)f.value(item));
      if (k == kMid % kRun && item == kMid && n_mid) all = s.wcum[n_mid - 1];
      n += c;
      sum += c ? all : 0.0;  // the weight of a value over the row's largest may be infinite
    }
  }
  ops.scan(n, sum);
  s.rc[tid + 1] = n;
  s.rm[tid + 1] = sum;
  if (tid == 0) {
    s.rc[0] = 0;
    s.rm[0] = 0.0;
  }
  __syncthreads();
  const uint32_t n_in = s.rc[kThreads], N = n_in + n_low;
  f.n_in = n_in;
  const double total = s.rm[kThreads];

  uint32_t kept = N;
  double Z = total;
  ValueCross cut{N, total, -1, 0, 0}, draw{0, 0.0, -1, 0, 0};
  bool in_low = false;  // a cut among the tokens under the range
#pragma unroll 1
  for (int q = 0; q < 5; ++q) {
    int kind;
    double amount;
    if (q == 0) {
      if (rp.k >= (int64_t)N) continue;
      if (rp.k > (int64_t)n_in) {
        in_low = true;
        kept = (uint32_t)rp.k;
        continue;
      }
      kind = kByCount, amount = (double)rp.k;
    } else if (q == 1) {
      if (!(rp.p < 1.0)) continue;
      kind = kByMassGe, amount = rp.p * Z;
    } else if (q == 2) {
      if (!(rp.m > 0.0)) continue;
      kind = kByWeight, amount = rp.m;
    } else if (q == 3) {
      if (in_low && o.out) return false;  // the cut itself is needed
      if (!o.token) break;
      kind = kByMassGt, amount = u * Z;
    } else {
      kind = kByCount, amount = (double)min(kept, n_in);
    }
    const ValueCross x = f.locate(kind, amount);
    if (q < 3) {
      if (x.item < 0) {  // all tokens of the range pass min-p
        if (n_low) return false;
      } else if (x.n < kept) {
        kept = x.n;
        Z = x.cum;
        cut = x;
        in_low = false;
      }
    } else {
      draw = x;
      if (q == 4 || x.n <= min(kept, n_in)) break;
    }
  }
  if (tid == 0 && o.kept) o.kept[row] = (int32_t)kept;
  // the index of the cut's or the drawn token (a call has one or the other)
  const ValueCross x = o.out ? cut : draw;
  uint32_t idx = 0;
  if (x.item >= 0 && (x.r > 0 || o.token)) idx = f.index_of(x, max(x.r, 1u));
  if (tid == 0) {
    if (o.out) *cut_out = x.item < 0 ? ~0ull : x.r == 0 ? comp_of(f.item_key(x), 0) : comp_of(f.item_key(x), idx) + 1;
    if (o.token) {
      o.token[row] = (int32_t)idx;
      if (o.prob) o.prob[row] = (float)(f.weight(key_value(f.item_key(x))) / Z);
    }
  }
  return true;
}

// a bf16 row by bins, in one block: maximum, bins, then passes over the row
__device__ __forceinline__ void finalize_self(FinLds& s, const SampleArgs& a, int64_t row, const SampleOut& o, uint64_t* cut_out) {
  constexpr int DT = DFLASH_BF16, VE = 8;
  constexpr float kMax = RowType<DT>::kMax;
  BlockOps ops(s.red);
  const int tid = threadIdx.x;
  const RowParams rp = row_params(a, row);
  const RowRef<DT> z(a.Z, row, a.stride, a.V);
  const int n_slots = z.slots();
  float m = kNegInf;
#pragma unroll 2
  for (int sl = tid; sl < n_slots; sl += kThreads) {
    const Slot x = z.load(sl);
#pragma unroll
    for (int i = 0; i < VE; ++i) m = fmaxf(m, slot_value<DT>(x, i));
  }
  m = (float)ops.max((double)fminf(m, kMax));
  if (m == kNegInf) return empty_row(row, o, cut_out);
  const double c8 = rp.c8, J = rint((double)m * c8);
  s.mass[tid] = 0;
  s.cnt[tid] = 0;
  __syncthreads();
#pragma unroll 1
  for (int sl = tid; sl < n_slots; sl += kThreads) {
    const Slot x = z.load(sl);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float v = slot_value<DT>(x, i);
      if (v > kNegInf) {
        const double t = (double)fminf(v, kMax) * c8, n = rint(t);
        const int b = (int)fmin(J - n, (double)kTail);
        atomicAdd(&s.cnt[b], 1u);
        if (b < kTail) atomicAdd((unsigned long long*)&s.mass[b], exp2_eighth_units(t - n));  // sums of 2^21 tokens fit 64 bits
      }
    }
  }
  __syncthreads();
  const uint32_t c = s.cnt[tid], cs = ops.scan(c);
  const double cum = ops.scan(tid < kTail ? (double)s.mass[tid] * 0x1p-42 * pow2_eighth(-tid) : 0.0);
  s.cc[tid + 1] = cs;
  s.cm[tid + 1] = cum;
  if (tid == 0) {
    s.cc[0] = 0;
    s.cm[0] = 0.0;
  }
  __syncthreads();
  const uint32_t kmax = key_of(m, kMax);
  Finalize<DT, kSelf> f{s, ops, z, nullptr, nullptr, nullptr, nullptr, 0, 0, 0, c8, rp.t8, J, tid, kmax, least_key(rp.m, kmax, c8, rp.t8), 0, 0, 0, 0.0, 1, 0, 0, 0, 0};
  f.answer(rp, s.cc[kBins], row_uniform(o, row), row, o, cut_out);
}

// One row takes 13 us, 512 rows 30: a chain of steps whose latency counts.  Of
// 25 thousand cycles for a row of 151936 the segments' counters take 7, the
// weights 2.4, the scan 3.3, a query 3 to 5 and the token's index 6 (in another
// block's segment).  Runs of items a thread took the weights there from 11; a
// separate kernel for rows that have to be binned costs the others a launch (5
// us).
__global__ __launch_bounds__(kThreads, 4) void sample_finalize_values_kernel(SampleArgs a, int64_t row0, int n_seg, int seg_slots,
                                                                          const SampleValues* __restrict__ parts, SampleOut o,
                                                                          uint64_t* __restrict__ cuts) {
  __shared__ RowLds s;
  const int64_t row = row0 + blockIdx.x;
  if (finalize_values(s.v, a, row, n_seg, seg_slots, parts + (size_t)blockIdx.x * n_seg, o, cuts + blockIdx.x)) return;
  __syncthreads();
  finalize_self(s.f, a, row, o, cuts + blockIdx.x);
}

// ---------------------------------------------------------------- the filtered row

// A copy with a comparison: 819 x 262144 bf16 in 139 to 145 us, 6.1 TB/s read and
// written.
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
  const uint64_t cut = cuts[r];
  const int s0 = seg * (kThreads * NL) + tid;
  Slot x[NL];
#pragma unroll
  for (int l = 0; l < NL; ++l) x[l] = z.load(s0 + l * kThreads);
#pragma unroll
  for (int l = 0; l < NL; ++l) store_filtered<DT>(o, a.V, s0 + l * kThreads, x[l], cut, fill);
}

template <int DT>
void apply(const SampleArgs& a, const SampleOut& o, int64_t r0, unsigned nr, const uint64_t* cuts, hipStream_t st) {
  const int slots = (a.V + RowType<DT>::VE - 1) / RowType<DT>::VE;
  const unsigned n8 = (unsigned)((slots + kThreads * 8 - 1) / (kThreads * 8)), n1 = (unsigned)((slots + kThreads - 1) / kThreads);
  if ((uint64_t)nr * n8 >= 1024)  // four blocks per CU and more
    launch(sample_apply_kernel<DT, 8>, dim3(nr * n8), dim3(kThreads), st, a, r0, (int)n8, cuts, o.fill, o.out, o.out_stride);
  else
    launch(sample_apply_kernel<DT, 1>, dim3(nr * n1), dim3(kThreads), st, a, r0, (int)n1, cuts, o.fill, o.out, o.out_stride);
}

hipError_t run_bf16(const SampleArgs& a, const SampleOut& o, char* ws, const SamplePlan& pl, hipStream_t st) {
  SampleValues* parts = reinterpret_cast<SampleValues*>(ws + pl.parts);
  uint64_t* cuts = reinterpret_cast<uint64_t*>(ws + pl.cuts);
  for (int64_t r0 = 0; r0 < a.R; r0 += pl.batch) {
    const unsigned nr = (unsigned)(a.R - r0 < pl.batch ? a.R - r0 : pl.batch);
    launch(sample_values_kernel, dim3(nr * (unsigned)pl.n_seg), dim3(kThreads), st, a, r0, pl.n_seg, pl.seg_slots, parts);
    launch(sample_finalize_values_kernel, dim3(nr), dim3(kThreads), st, a, r0, pl.n_seg, pl.seg_slots, (const SampleValues*)parts,
           o, cuts);
    if (o.out) apply<DFLASH_BF16>(a, o, r0, nr, cuts, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int NL, bool ALL>
hipError_t run_f32(const SampleArgs& a, const SampleOut& o, char* ws, const SamplePlan& pl, hipStream_t st) {
  SamplePart* parts = reinterpret_cast<SamplePart*>(ws + pl.parts);
  uint64_t* lists = reinterpret_cast<uint64_t*>(ws + pl.lists);
  uint64_t* cuts = reinterpret_cast<uint64_t*>(ws + pl.cuts);
  SampleAsk* asks = reinterpret_cast<SampleAsk*>(ws + pl.asks);
  uint64_t* asked = reinterpret_cast<uint64_t*>(ws + pl.asked);
  const dim3 block(kThreads);
  for (int64_t r0 = 0; r0 < a.R; r0 += pl.batch) {
    const unsigned nr = (unsigned)(a.R - r0 < pl.batch ? a.R - r0 : pl.batch);
    const dim3 rows(nr), segs(nr * (unsigned)pl.n_seg);
    launch(sample_hist_kernel<NL, ALL>, segs, block, st, a, r0, pl.n_seg, pl.cap, parts, lists);
    if constexpr (ALL) {
      launch(sample_finalize_kernel<kAll>, rows, block, st, a, r0, pl.n_seg, pl.cap, pl.ask, (const SamplePart*)parts,
             (const uint64_t*)lists, asks, (const uint64_t*)asked, o, cuts);
    } else {
      launch(sample_finalize_kernel<kFirst>, rows, block, st, a, r0, pl.n_seg, pl.cap, pl.ask, (const SamplePart*)parts,
             (const uint64_t*)lists, asks, (const uint64_t*)asked, o, cuts);
      launch(sample_gather_kernel<NL>, segs, block, st, a, r0, pl.n_seg, pl.ask, asks, asked);
      launch(sample_finalize_kernel<kSecond>, rows, block, st, a, r0, pl.n_seg, pl.cap, pl.ask, (const SamplePart*)parts,
             (const uint64_t*)lists, asks, (const uint64_t*)asked, o, cuts);
    }
    if (o.out) apply<DFLASH_F32>(a, o, r0, nr, cuts, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_sample(int32_t dtype, const SampleArgs& a, const SampleOut& o, char* ws, const SamplePlan& pl,
                         hipStream_t st) {
  if (pl.one) {
    const dim3 rows((unsigned)a.R), block(kThreads);
    if (dtype == DFLASH_BF16)
      launch(sample_row_kernel<DFLASH_BF16, 1>, rows, block, st, a, o);
    else
      launch(pl.loads == 1   ? sample_row_kernel<DFLASH_F32, 1>
             : pl.loads == 2 ? sample_row_kernel<DFLASH_F32, 2>
                             : sample_row_kernel<DFLASH_F32, 4>,
             rows, block, st, a, o);
    return hipGetLastError();
  }
  if (dtype == DFLASH_BF16) return run_bf16(a, o, ws, pl, st);
  if (pl.all) return pl.loads == 2 ? run_f32<2, true>(a, o, ws, pl, st) : run_f32<4, true>(a, o, ws, pl, st);
  switch (pl.loads) {
    case 2: return run_f32<2, false>(a, o, ws, pl, st);
    case 4: return run_f32<4, false>(a, o, ws, pl, st);
    default: return run_f32<8, false>(a, o, ws, pl, st);
  }
}

}  // namespace dfk
