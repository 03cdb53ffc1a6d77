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
constexpr int kCap = 4096;          // tokens of one bin held in LDS
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

// Reductions over the block with one barrier each: successive calls alternate
// between two buffers, so a buffer is rewritten only after the barrier of the
// call between, which every thread reaches after it has read the buffer.
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
    return (int)r;
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
    return v;
  }
  __device__ __forceinline__ uint32_t sum(uint32_t v) {
    v = wave_sum_u32(v);
    flip ^= 1;
    if ((threadIdx.x & 63) == 0) s.u[flip][threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s.u[flip][w];
    return v;
  }

 private:
  static __device__ __forceinline__ uint32_t wave_scan_u32(uint32_t v) {
    v += dpp_u32<kDppRowShr1>(v, 0u);
    v += dpp_u32<kDppRowShr2>(v, 0u);
    v += dpp_u32<kDppRowShr4>(v, 0u);
    v += dpp_u32<kDppRowShr8>(v, 0u);
    v += dpp_u32<kDppRowBcast15, 0xA>(v, 0u);
    v += dpp_u32<kDppRowBcast31, 0xC>(v, 0u);
    return v;
  }
};

__device__ __forceinline__ uint32_t key_of(float v, float max_finite) {
  return ord32_canon(__float_as_uint(fminf(v, max_finite)));
}
__device__ __forceinline__ double key_value(uint32_t key) { return (double)__uint_as_float(unord32(key)); }

// smallest ordered key >= kKeyLowest whose t = z c8 reaches `j` (0xFF800000,
// above every finite key, if none does).  One round of the wave's 64 lanes
// around j / c8, which rounding moves by a few keys; a search where that
// guess does not bracket it (j or c8 extreme).
__device__ __forceinline__ uint32_t lowest_key(double j, double c8) {
  const double z = fmin(fmax(j / c8, -3.4028234663852886e38), 3.4028234663852886e38);  // 0/0: some finite value
  const uint32_t g = max(ord32_canon(__float_as_uint((float)z)), kKeyLowest + 32u);
  const uint32_t cand = min(g - 32u + (uint32_t)lane_id(), 0xFF7FFFFFu);
  const uint64_t hit = __ballot(key_value(cand) * c8 >= j);
  if (hit && !(hit & 1)) return __shfl(cand, __builtin_ctzll(hit));
  uint32_t l = kKeyLowest, h = 0xFF800000u;
  while (l < h) {
    const uint32_t mid = l + ((h - l) >> 1);
    if (key_value(mid) * c8 >= j) h = mid; else l = mid + 1;
  }
  return l;
}

// ---------------------------------------------------------------- (1) bins of a segment

template <int DT, int NL>
__global__ __launch_bounds__(kThreads) void sample_hist_kernel(SampleArgs a, int64_t row0, int n_seg,
                                                               SamplePart* __restrict__ parts) {
  constexpr int VE = RowType<DT>::VE;
  __shared__ uint64_t mass[kBins * kCols];
  __shared__ uint32_t cnt[kBins * kCols];
  __shared__ Red red;
  __shared__ uint32_t n_list;
  BlockOps ops(red);
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
  if (tid == 0) n_list = 0;
  float m = kNegInf;
#pragma unroll
  for (int l = 0; l < NL; ++l)
#pragma unroll
    for (int i = 0; i < VE; ++i) m = fmaxf(m, slot_value<DT>(x[l], i));  // NaN drops out
  m = (float)ops.max((double)fminf(m, RowType<DT>::kMax));

  SamplePart& out = parts[blockIdx.x];
  if (m == kNegInf) {
    if (tid == 0) {
      out.J = -INFINITY;
      out.max = kNegInf;
      out.n = 0;
      out.nb = 0;
      out.listed = kBins;
      out.n_list = 0;
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
  uint32_t c = 0, mirror = 0;  // mirror: the bin counted from the far end
  uint64_t f = 0;
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    c += cnt[tid * kCols + k];
    f += mass[tid * kCols + k];
    mirror += cnt[(kBins - 1 - tid) * kCols + k];
  }
  f -= (uint64_t)c * kOneBits;  // modulo 2^64: the fraction bits' sum
  const uint32_t upto = ops.scan(c);
  const int nb = kBins - ops.first(mirror != 0);  // bins in use
  // the first bins with at most kSampleList tokens together are listed
  const int listed = ops.first(upto > (uint32_t)kSampleList);
  if (tid < nb) {
    out.cnt[tid] = c;
    out.mass[tid] = tid < kTail ? (double)c + (double)f * 0x1p-52 : 0.0;
  }
  if (listed > 0) {
    const uint32_t least = listed >= kBins ? kKeyLowest : lowest_key(J - (double)(listed - 1), c8);
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      const int e = z.first(s0 + l * kThreads);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float v = slot_value<DT>(x[l], i);
        const uint32_t key = key_of(v, RowType<DT>::kMax);
        if (v > kNegInf && key >= least) {
          const uint32_t at = atomicAdd(&n_list, 1u);
          if (at < (uint32_t)kSampleList) out.list[at] = ((uint64_t)~key << 32) | (uint32_t)(e + i);
        }
      }
    }
  }
  __syncthreads();
  if (tid == kThreads - 1) {
    out.J = J;
    out.max = m;
    out.n = upto;
    out.nb = nb;
    out.listed = listed;
    out.n_list = (int32_t)min(n_list, (uint32_t)kSampleList);
  }
}

// ---------------------------------------------------------------- (2) cuts and draw of a row

enum { kByCount, kByMassGe, kByMassGt, kByWeight };

constexpr int kMaxSeg = kSampleMaxSeg;

struct FinLds {
  uint64_t big[kCap];       // tokens of one bin as (~key, index), in any order
  uint64_t win[kThreads];   // the window: sorted, ascending = the row's order
  double wcum[kThreads];    // and the running sums at its tokens
  uint64_t mass[kBins];     // bins of a split
  uint32_t cnt[kBins];
  uint32_t cc[kBins + 1];   // tokens before each bin
  double cm[kBins + 1];     // their weight
  uint32_t rc[kBins + 1];   // the same inside a split
  double rm[kBins + 1];
  int16_t shift[kMaxSeg];   // a segment's first bin on the row's grid
  int16_t len[kMaxSeg];     // its bins and its listed tokens
  int16_t n_list[kMaxSeg];
  Red red;
  uint32_t n;
  uint64_t at;
};

// where a running count or sum crosses a value
struct Cross {
  uint32_t n;    // tokens up to and including the crossing one (kByWeight: tokens that pass)
  double cum;    // their weight
  uint64_t cut;  // a token is among them iff its (~key, index) is below this
  uint64_t at;   // (~key, index) of the last of them (not for kByWeight)
};

__device__ __forceinline__ uint32_t comp_key(uint64_t c) { return ~(uint32_t)(c >> 32); }

template <int DT>
struct Finalize {
  static constexpr int VE = RowType<DT>::VE;
  FinLds& s;
  BlockOps& ops;
  const RowRef<DT> z;
  const SamplePart* part;
  const int n_seg;
  const double c8, J;
  const int tid;
  const uint32_t kmax;  // the row's largest key
  const int listed;     // bins 0 .. listed - 1 are in the segments' lists
  // the window's tokens: rank base + 1 .. base + n, of bins b0 .. b1 (b0 > b1: part of a bin)
  uint32_t base, n;
  double bmass;
  int b0, b1;
  uint32_t lo;

  __device__ Finalize(FinLds& s_, BlockOps& o, const RowRef<DT>& z_, const SamplePart* part_, int n_seg_, double c8_, double J_,
                      uint32_t kmax_, int listed_)
      : s(s_), ops(o), z(z_), part(part_), n_seg(n_seg_), c8(c8_), J(J_), tid(threadIdx.x), kmax(kmax_), listed(listed_), base(0),
        n(0), bmass(0.0), b0(1), b1(0), lo(0) {}

  // weight of a key relative to 2^(J / 8)
  __device__ double weight(uint32_t key) const {
    const double t = key_value(key) * c8, fl = floor(t);
    return exp2_eighth(t - fl) * pow2_eighth((int)fmax(fl - J, -16000.0));
  }

  // f((~key, index)) of every token of the row with klo <= key <= khi; eight slots in flight per thread
  template <class F>
  __device__ void each_in_row(uint32_t klo, uint32_t khi, F f) const {
    const int n_slots = (z.V + z.phase + VE - 1) / VE;
    for (int s0 = tid; s0 < n_slots; s0 += 8 * kThreads) {
      Slot x[8];
#pragma unroll
      for (int l = 0; l < 8; ++l) x[l] = z.load(s0 + l * kThreads);
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        const int e = z.first(s0 + l * kThreads);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
          const float v = slot_value<DT>(x[l], i);
          const uint32_t key = key_of(v, RowType<DT>::kMax);
          if (v > kNegInf && key >= klo && key <= khi) f(((uint64_t)~key << 32) | (uint32_t)(e + i));
        }
      }
    }
  }
  // the same over the segments' lists (whole only for listed bins) and over `big`
  template <class F>
  __device__ void each_in_lists(uint32_t klo, uint32_t khi, F f) const {
    for (int i = tid; i < n_seg * kSampleList; i += kThreads) {
      const int g = i / kSampleList, j = i % kSampleList;
      if (j < s.n_list[g]) {
        const uint64_t c = part[g].list[j];
        const uint32_t key = comp_key(c);
        if (key >= klo && key <= khi) f(c);
      }
    }
  }
  template <class F>
  __device__ void each_in_big(uint32_t nbig, uint32_t klo, uint32_t khi, F f) const {
    for (uint32_t i = tid; i < nbig; i += kThreads) {
      const uint64_t c = s.big[i];
      const uint32_t key = comp_key(c);
      if (key >= klo && key <= khi) f(c);
    }
  }

  // append to an LDS array through s.n
  __device__ void start_append() {
    __syncthreads();
    if (tid == 0) s.n = 0;
    __syncthreads();
  }

  // s.win[0 .. s.n - 1] holds the window's tokens in any order: sort them (each
  // thread ranks one token against the others) and sum their weights
  __device__ void open_window(uint32_t lo_, uint32_t base_, double bmass_, int b0_, int b1_) {
    lo = lo_, base = base_, bmass = bmass_, b0 = b0_, b1 = b1_;
    __syncthreads();
    n = min(s.n, (uint32_t)kThreads);
    const bool in = tid < (int)n;
    const uint64_t mine = in ? s.win[tid] : 0;
    uint32_t rank = 0;
    if ((tid & ~63) < (int)n) {
      uint32_t j = 0;
      for (; j + 4 <= n; j += 4) {
        const uint64_t a = s.win[j], b = s.win[j + 1], c = s.win[j + 2], d = s.win[j + 3];
        rank += (uint32_t)(a < mine) + (uint32_t)(b < mine) + (uint32_t)(c < mine) + (uint32_t)(d < mine);
      }
      for (; j < n; ++j) rank += s.win[j] < mine;
    }
    __syncthreads();
    if (in) s.win[rank] = mine;
    __syncthreads();
    const double w = in ? weight(comp_key(s.win[tid])) : 0.0;
    const double c = bmass + ops.scan(w);
    if (in) s.wcum[tid] = c;
    __syncthreads();
  }

  __device__ Cross from_window(int kind, double amount) {
    const bool in = tid < (int)n;
    const bool hit = in && (kind == kByCount    ? (double)(base + tid + 1) >= amount
                            : kind == kByMassGe ? s.wcum[tid] >= amount
                            : kind == kByMassGt ? s.wcum[tid] > amount
                                                : weight(comp_key(s.win[tid])) < amount);
    int pos = min(ops.first(hit), (int)n);
    if (kind != kByWeight) pos = min(pos + 1, (int)n);  // pos tokens of the window are in
    Cross r;
    r.n = base + pos;
    r.cum = pos > 0 ? s.wcum[pos - 1] : bmass;
    r.at = pos > 0 ? s.win[pos - 1] : 0;
    r.cut = pos < (int)n ? s.win[pos] : ((uint64_t)~lo + 1) << 32;
    return r;
  }

  // index of the r-th (from 1) token with this key in `big`
  __device__ uint32_t tie_in_big(uint32_t nbig, uint32_t key, uint32_t r) {
    uint32_t ilo = 0, ihi = (uint32_t)z.V - 1;
    for (;;) {
      const uint32_t range = ihi - ilo;
      const int sh = max(0, 32 - (range ? __builtin_clz(range) : 32) - 9);
      __syncthreads();
      s.cnt[tid] = 0;
      __syncthreads();
      each_in_big(nbig, key, key, [&](uint64_t c) {
        const uint32_t i = (uint32_t)c;
        if (i >= ilo && i <= ihi) atomicAdd(&s.cnt[(i - ilo) >> sh], 1u);
      });
      __syncthreads();
      const uint32_t c = s.cnt[tid], upto = ops.scan(c);
      const int b = min(ops.first(upto >= r), kThreads - 1);
      if (tid == b) s.at = upto - c;
      __syncthreads();
      r -= (uint32_t)s.at;
      ilo += (uint32_t)b << sh;
      if (sh == 0) return ilo;
      ihi = min(ihi, ilo + ((1u << sh) - 1u));
    }
  }

  // the same over the row, for more equal tokens than `big` holds: the waves
  // count contiguous pieces, the one that holds it walks its piece again
  __device__ uint32_t tie_in_row(uint32_t key, uint32_t r) {
    const int n_slots = (z.V + z.phase + VE - 1) / VE, lane = tid & 63, w = tid >> 6;
    const int per = ((n_slots + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int sb = w * per, se = min(n_slots, sb + per);
    auto count = [&](int sl, uint32_t* mask) {
      const Slot x = z.load(sl);
      uint32_t mk = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float v = slot_value<DT>(x, i);
        mk |= (uint32_t)(v > kNegInf && key_of(v, RowType<DT>::kMax) == key) << i;
      }
      *mask = mk;
      return (uint32_t)__popc(mk);
    };
    uint32_t c = 0, mk = 0;
    for (int sl = sb + lane; sl < se; sl += 64) c += count(sl, &mk);
    c = wave_sum_u32(c);
    __syncthreads();
    if (lane == 0) s.cnt[w] = c;
    if (tid == 0) s.at = 0;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < w; ++i) before += s.cnt[i];
    if (r > before && r <= before + s.cnt[w]) {
      uint32_t left = r - before;
      for (int b = sb; b < se; b += 64) {
        const uint32_t cl = b + lane < se ? count(b + lane, &mk) : 0;
        uint32_t sc = cl;  // inclusive scan over the wave
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
          const uint32_t t = __shfl_up(sc, o);
          sc += lane >= o ? t : 0u;
        }
        const uint32_t total = __shfl(sc, 63);
        if (left <= total) {
          if (left > sc - cl && left <= sc) {
            uint32_t k = left - (sc - cl);  // from 1 inside this lane's slot
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

  // A bin (keys klo .. khi) of more tokens than a window holds: split its key
  // range until the part with the crossing fits one, or is a single value.
  // The first rounds read the row where the bin does not fit `big` either.
  __device__ Cross split(int kind, double amount, uint32_t klo, uint32_t khi, uint32_t cb, uint32_t nc, double mb, bool tail,
                         bool from_lists) {
    uint32_t nbig = 0;
    for (;;) {
      if (nbig == 0 && nc <= (uint32_t)kCap) {
        start_append();
        auto put = [&](uint64_t c) {
          const uint32_t i = atomicAdd(&s.n, 1u);
          if (i < (uint32_t)kCap) s.big[i] = c;
        };
        if (from_lists)
          each_in_lists(klo, khi, put);
        else
          each_in_row(klo, khi, put);
        __syncthreads();
        nbig = min(s.n, (uint32_t)kCap);
      }
      if (nc <= (uint32_t)kThreads) {
        start_append();
        each_in_big(nbig, klo, khi, [&](uint64_t c) {
          const uint32_t i = atomicAdd(&s.n, 1u);
          if (i < (uint32_t)kThreads) s.win[i] = c;
        });
        open_window(klo, cb, mb, 1, 0);
        return from_window(kind, amount);
      }
      if (klo == khi) {  // one value: every token weighs w
        const double w = tail ? 0.0 : weight(klo);
        double r = (double)nc;
        if (kind == kByCount) r = amount - cb;
        if (kind == kByMassGe || kind == kByMassGt) {
          r = fmin(fmax(floor((amount - mb) / w), 0.0), (double)nc);
          // the quotient is off by rounding only: settle it on the sums themselves
          if (r > 0.0 && (kind == kByMassGe ? fma(r - 1.0, w, mb) >= amount : fma(r - 1.0, w, mb) > amount)) r -= 1.0;
          if (r < (double)nc && !(kind == kByMassGe ? fma(r, w, mb) >= amount : fma(r, w, mb) > amount)) r += 1.0;
          r = fmax(r, 1.0);
        }
        if (kind == kByWeight) r = weight(klo) < amount ? 0.0 : (double)nc;
        Cross x;
        x.n = cb + (uint32_t)r;
        x.cum = fma(r, w, mb);
        x.at = 0;
        x.cut = ((uint64_t)~klo) << 32;
        if (r > 0.0) {
          const uint32_t i = nbig ? tie_in_big(nbig, klo, (uint32_t)r) : tie_in_row(klo, (uint32_t)r);
          x.at = ((uint64_t)~klo << 32) | i;
          x.cut = x.at + 1;
        }
        return x;
      }
      const uint32_t range = khi - klo;
      const int sh = max(0, 32 - __builtin_clz(range) - 9);
      __syncthreads();
      s.cnt[tid] = 0;
      s.mass[tid] = 0;
      __syncthreads();
      auto add = [&](uint64_t cp) {
        const uint32_t key = comp_key(cp), b = (khi - key) >> sh;
        atomicAdd(&s.cnt[b], 1u);
        if (!tail) {
          const double t = key_value(key) * c8;
          // 46 bits of the mantissa: sums of 2^21 tokens fit 64 bits
          atomicAdd((unsigned long long*)&s.mass[b],
                    (unsigned long long)((__double_as_longlong(exp2_eighth(t - floor(t))) - kOneBits) >> 6));
        }
      };
      if (nbig)
        each_in_big(nbig, klo, khi, add);
      else
        each_in_row(klo, khi, add);
      __syncthreads();
      // one bin holds one eighth of an octave: its unit is that of its lowest key
      const double unit = tail ? 0.0 : pow2_eighth((int)fmax(floor(key_value(klo) * c8) - J, -16000.0));
      const uint32_t c = s.cnt[tid];
      const uint32_t c1 = cb + ops.scan(c);
      const double m1 = mb + ops.scan(unit * ((double)c + (double)s.mass[tid] * 0x1p-46));
      s.rc[tid + 1] = c1;
      s.rm[tid + 1] = m1;
      if (tid == 0) {
        s.rc[0] = cb;
        s.rm[0] = mb;
      }
      const uint32_t n_part = (range >> sh) + 1;  // parts, from the highest key down
      const uint32_t low = (uint32_t)tid + 1 >= n_part ? klo : khi - ((uint32_t)tid << sh) - ((1u << sh) - 1u);
      const bool hit = (uint32_t)tid < n_part &&
                       (kind == kByCount    ? (double)c1 >= amount
                        : kind == kByMassGe ? m1 >= amount
                        : kind == kByMassGt ? m1 > amount
                                            : weight(low) < amount);
      int b = ops.first(hit);
      if (b >= (int)n_part) {
        // every key passes, or rounding left the sum short of the last token
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
        b = ops.first((uint32_t)tid < n_part && (double)c1 >= amount);
      }
      nc = s.rc[b + 1] - s.rc[b];
      cb = s.rc[b];
      mb = s.rm[b];
      khi -= (uint32_t)b << sh;
      if ((uint32_t)b + 1 < n_part) klo = khi - ((1u << sh) - 1u);
      if (nc == 0) {  // kByWeight: the threshold falls between tokens
        Cross r;
        r.n = cb;
        r.cum = mb;
        r.cut = ((uint64_t)~khi) << 32;
        r.at = 0;
        return r;
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
    int b = ops.first(hit);
    if (b >= kBins) {
      b = kTail;
      if (kind != kByWeight) {  // a sum that rounding left short: the last token above the tail
        kind = kByCount;
        amount = (double)s.cc[kTail];
        b = ops.first((double)s.cc[tid + 1] >= amount);
      }
    }
    if (b >= b0 && b <= b1) return from_window(kind, amount);
    const uint32_t c = s.cc[b + 1] - s.cc[b];
    const uint32_t klo = b == kTail ? kKeyLowest : lowest_key(J - b, c8);
    if (b < listed && s.cc[b + 1] <= (uint32_t)kThreads) {
      // everything down to this bin fits a window and is in the lists
      start_append();
      each_in_lists(klo, kmax, [&](uint64_t cp) {
        const uint32_t i = atomicAdd(&s.n, 1u);
        if (i < (uint32_t)kThreads) s.win[i] = cp;
      });
      open_window(klo, 0, 0.0, 0, b);
      return from_window(kind, amount);
    }
    const uint32_t khi = b == 0 ? kmax : lowest_key(J - b + 1.0, c8) - 1u;
    if (c == 0) {  // kByWeight only: nothing in the threshold's own bin
      Cross r;
      r.n = s.cc[b];
      r.cum = s.cm[b];
      r.cut = ((uint64_t)~khi) << 32;
      r.at = 0;
      return r;
    }
    if (c > (uint32_t)kThreads) return split(kind, amount, klo, khi, s.cc[b], c, s.cm[b], b == kTail, b < listed);
    start_append();
    auto put = [&](uint64_t cp) {
      const uint32_t i = atomicAdd(&s.n, 1u);
      if (i < (uint32_t)kThreads) s.win[i] = cp;
    };
    if (b < listed)
      each_in_lists(klo, khi, put);
    else
      each_in_row(klo, khi, put);
    open_window(klo, s.cc[b], s.cm[b], b, b);
    return from_window(kind, amount);
  }
};

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_finalize_kernel(SampleArgs a, int64_t row0, int n_seg,
                                                                   const SamplePart* __restrict__ parts,
                                                                   const double* __restrict__ u, int32_t* __restrict__ token,
                                                                   float* __restrict__ prob, int32_t* __restrict__ kept,
                                                                   uint64_t* __restrict__ cuts) {
  __shared__ FinLds s;
  BlockOps ops(s.red);
  const int tid = threadIdx.x;
  const int64_t row = row0 + blockIdx.x;
  const RowParams rp = row_params(a, row);
  const SamplePart* part = parts + (size_t)blockIdx.x * n_seg;

  // the segments' headers, one thread each (n_seg <= kMaxSeg = kThreads)
  const bool have = tid < n_seg;
  const double Js = have ? part[tid].J : -INFINITY;
  const uint32_t ns = have ? part[tid].n : 0;
  const int nbs = have ? part[tid].nb : 0, ls = have ? part[tid].listed : kBins, nl = have ? part[tid].n_list : 0;
  const double ms = have ? (double)part[tid].max : -INFINITY;
  const double J = ops.max(Js);
  const float m = (float)ops.max(ms);
  const uint32_t N = ops.sum(ns);
  if (N == 0) {  // every token masked
    if (tid == 0) {
      if (token) token[row] = -1;
      if (prob) prob[row] = 0.0f;
      if (kept) kept[row] = 0;
      if (cuts) cuts[blockIdx.x] = 0;
    }
    return;
  }
  const int shift = ns ? (int)fmin(J - Js, (double)kBins) : kBins;
  if (have) {
    s.shift[tid] = (int16_t)shift;
    s.len[tid] = (int16_t)min(nbs, kTail);
    s.n_list[tid] = (int16_t)nl;
  }
  // bins whose tokens are all listed: as far as every segment's list reaches
  const int listed = kBins - (int)ops.max((double)(kBins - (ls >= kBins ? kBins : min(kBins, ls + shift))));
  // the segments' bins on the row's grid, in segment order
  uint32_t c = 0;
  double mass = 0.0;
#pragma unroll 8
  for (int g = 0; g < n_seg; ++g) {
    const int b = tid - s.shift[g];
    const bool in = tid < kTail && b >= 0 && b < s.len[g];
    c += in ? part[g].cnt[b] : 0u;
    mass += in ? part[g].mass[b] : 0.0;
  }
  uint32_t cs = ops.scan(c);
  const double cum = ops.scan(mass * pow2_eighth(-tid));
  if (tid == kTail) cs = N;  // the tail bin: whatever is left
  s.cc[tid + 1] = cs;
  s.cm[tid + 1] = cum;
  if (tid == 0) {
    s.cc[0] = 0;
    s.cm[0] = 0.0;
  }
  __syncthreads();

  const uint32_t kmax = key_of(m, RowType<DT>::kMax);
  Finalize<DT> f(s, ops, RowRef<DT>(a.Z, row, a.stride, a.V), part, n_seg, rp.c8, J, kmax, listed);
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
    if (prob) prob[row] = (float)(f.weight(comp_key(d.at)) / Z);
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
      const uint32_t key = key_of(v, RowType<DT>::kMax);
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
