// dflash_logprobs and dflash_logprobs_grad: log probabilities of given tokens
// of a row of logits, its entropy and its largest alternatives; the gradient
// of the first two.
//
// With m = max z, c = log2 e / T and any reference M,
//   t_j = z_j c - M,  s = sum_j 2^t_j,  h = sum_j 2^t_j t_j:
//   log sum_j e^((z_j - m) / T) = ln 2 (log2 s + M - m c),
//   entropy                     = ln 2 (log2 s - h / s).
// t_j is one fma, right to half a step of itself however large M is, so the
// terms that count (t near 0) are right to 2^-23; a thread sums 16 or 32 of
// them in fp32 and adds that to fp64.  M is a whole number, so that a larger
// one scales the sums exactly: m c rounded, so that no t is above 1/2.  Beyond 2^24
// fp32 holds no such number: a row with |m| c there (all of it the type's lowest
// value, or T below 1e-6) is summed again from z_j - m.
//
// The alternatives take nothing from the streaming loop but three maxima a
// thread: of the slots a thread loads at a time (a piece), the two largest maxima
// with their places and the third.  A bound that N threads' maxima reach bounds
// the N-th largest logit from below, so only pieces whose maximum reaches it
// are read again: little more than N of them.
#include "rows_blocks.hpp"

namespace dfk {

namespace {

constexpr double kLog2e64 = 1.4426950408889634;
constexpr double kLn2 = 0.6931471805599453;
constexpr int kPieces = 512;       // pieces that are read again
constexpr int kCap = 1024;         // tokens of those that are ranked; of as many lists of the join
static_assert(kCap >= DFLASH_TOP_MAX * DFLASH_TOP_MAX && kPieces >= kLogprobsMaxSeg, "the join's lists");
constexpr float kHuge = 0x1p24f;   // |m| c beyond this, which fp32 does not hold to 1/2: from z - m

// log2 e over a row's temperature, which lies in [1e-30, 1e30]; 0, below or NaN: 1
__device__ __forceinline__ double row_scale(const float* T, int group, int64_t row) {
  const float t = T ? T[row / group] : 1.0f;
  return t > 0.0f ? kLog2e64 / fmin(fmax((double)t, 1e-30), 1e30) : kLog2e64;
}

template <int T>
struct Shared {
  static constexpr int kMaxima = T < 256 ? T : 256;  // of T / kMaxima neighbouring threads each
  uint32_t tm[kMaxima];        // as ordered keys
  uint64_t key[kCap > T + DFLASH_TOP_MAX ? kCap : T + DFLASH_TOP_MAX];  // value and inverted index of tokens that may be alternatives
  uint32_t piece[kPieces];     // thread | piece << 10
  float wave_m[T / kWave];
  double wave_s[T / kWave], wave_h[T / kWave];
  uint32_t n_piece, n_key, tau;
  uint64_t least;
  uint64_t top[DFLASH_TOP_MAX];
};

__device__ __forceinline__ uint64_t token_key(float v, int idx) {
  return ((uint64_t)ord32_canon(__float_as_uint(v)) << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_value(uint64_t k) { return __uint_as_float(unord32((uint32_t)(k >> 32))); }

// a thread's largest logit; whether one is NaN or +inf (then both are any value);
// low: the most negative logit, or any if there is none below zero
template <int DT, int N>
__device__ __forceinline__ float largest(const Slot (&x)[N], bool& odd, float& low) {
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
    const uint32_t u = max(up & 0xFFFFu, up >> 16);
    odd = h >= 0x7F80 || u > 0xFF80u;
    low = __uint_as_float(u << 16);
    uint32_t best = (uint32_t)h;
    if (h < 0) {
      uint32_t lo = 0xFFFFFFFFu;
#pragma unroll
      for (int l = 0; l < N; ++l)
#pragma unroll
        for (int d = 0; d < 4; ++d) lo = min_u16x2(lo, x[l].w[d]);
      best = min(lo & 0xFFFFu, lo >> 16);
    }
    return __uint_as_float(best << 16);
  } else {
    int hi = INT32_MIN;
    uint32_t up = 0;
#pragma unroll
    for (int l = 0; l < N; ++l)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        hi = max(hi, (int)x[l].w[d]);
        up = max(up, x[l].w[d]);
      }
    odd = hi >= 0x7F800000 || up > 0xFF800000u;
    low = __uint_as_float(up);
    uint32_t best = (uint32_t)hi;
    if (hi < 0) {
      best = 0xFFFFFFFFu;
#pragma unroll
      for (int l = 0; l < N; ++l)
#pragma unroll
        for (int d = 0; d < 4; ++d) best = min(best, x[l].w[d]);
    }
    return __uint_as_float(best);
  }
}

// what a row, or a segment of one, has come to
struct Sums {
  float m;      // the largest logit; -inf: nothing unmasked; NaN: a NaN or +inf among them
  double M;     // the sums' reference
  double s, h;
};

__device__ __forceinline__ double reference(float m, float c) {
  return rint(fmin(fmax((double)m * (double)c, -(double)kHuge), (double)kHuge));
}

// s and h from reference `from` to a larger one
__device__ __forceinline__ void rebase(double from, double to, double& s, double& h) {
  const double d = from - to;  // a whole number
  s = ldexp(s, (int)fmax(d, -4000.0));
  h = ldexp(h, (int)fmax(d, -4000.0));
  h = s > 0.0 ? fma(d, s, h) : 0.0;
}

// the N largest keys of sh.key[0 .. n), in order, to sh.top; the others of sh.top are 0
template <int T>
__device__ void rank_keys(Shared<T>& sh, int n, int N) {
  if (threadIdx.x < DFLASH_TOP_MAX) sh.top[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += T) {
    const uint64_t k = sh.key[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += sh.key[j] > k;
    if (rank < N) sh.top[rank] = k;
  }
  __syncthreads();
}

// The N largest tokens of a segment with no bound on how many tie: slots in the
// order of their index, the tokens above the N-th best so far join it.  One more
// pass over the segment.
template <int DT, int T>
__device__ __noinline__ void top_by_scan(Shared<T>& sh, const RowRef<DT> z, int s0, int s1, int N) {
  constexpr int VE = RowType<DT>::VE;
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) sh.n_key = 0, sh.least = 0;
  __syncthreads();
  for (int b = s0; b < s1; b += T) {
    const Slot x = z.load(b + tid < s1 ? b + tid : z.slots());
    uint64_t least = sh.least;
    bool any = false;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float v = slot_value<DT>(x, i);
      any |= v > kNegInf && token_key(v, (b + tid) * VE + i) > least;
    }
    if (!__syncthreads_or(any)) continue;
#pragma unroll 1
    for (int i = 0; i < VE; ++i) {
      // at most T new keys beside the N kept
      float v = slot_value<DT>(x, 0);
#pragma unroll
      for (int q = 1; q < VE; ++q)
        if (i == q) v = slot_value<DT>(x, q);
      const uint64_t k = token_key(v, (b + tid) * VE + i);
      least = sh.least;
      const bool hit = v > kNegInf && k > least;
      if (!__syncthreads_or(hit)) continue;
      if (hit) sh.key[atomicAdd(&sh.n_key, 1u)] = k;
      __syncthreads();
      const int n = (int)sh.n_key;
      rank_keys(sh, n, N);
      if (tid < N) sh.key[tid] = sh.top[tid];
      if (tid == 0) {
        sh.n_key = (uint32_t)min(n, N);
        if (n >= N) sh.least = sh.top[N - 1];
      }
      __syncthreads();
    }
  }
  rank_keys(sh, (int)sh.n_key, N);
}

__device__ __forceinline__ uint32_t value_key(float v) { return ord32_canon(__float_as_uint(v)); }
constexpr uint32_t kMaskedKey = 0x007FFFFFu;  // of -inf

// The N largest tokens of the segment to sh.top.  m1, m2, m3: the largest maxima of
// this thread's pieces, u1 and u2 where the first two are.
template <int DT, int T, int U>
__device__ __forceinline__ void top_of_segment(Shared<T>& sh, const RowRef<DT>& z, int s0, int s1, int N, float m1, float m2,
                                               float m3, int u1, int u2) {
  constexpr int VE = RowType<DT>::VE;
  const int tid = threadIdx.x;
  const uint32_t k1 = value_key(m1), k2 = value_key(m2), k3 = value_key(m3);
  constexpr int kMaxima = Shared<T>::kMaxima, kShare = T / kMaxima;
  uint32_t shared_max = k1;
#pragma unroll
  for (int w = 1; w < kShare; w *= 2) shared_max = max(shared_max, (uint32_t)__shfl_xor(shared_max, w));
  if (tid % kShare == 0) sh.tm[tid / kShare] = shared_max;
  if (tid == 0) sh.n_piece = 0, sh.n_key = 0;
  __syncthreads();
  if (tid < kWave) {
    // from the highest bit on the largest value that N maxima reach, or one that few more reach
    uint32_t k[kMaxima / kWave], t = 0;
#pragma unroll
    for (int q = 0; q < kMaxima / kWave; ++q) k[q] = sh.tm[q * kWave + tid];
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = t | 1u << bit;
      int n = 0;
#pragma unroll
      for (int q = 0; q < kMaxima / kWave; ++q) n += __popcll(__ballot(k[q] >= c));
      if (n >= N) {
        t = c;
        if (n <= N + 4) break;
      }
    }
    if (tid == 0) sh.tau = max(t, kMaskedKey + 1);
  }
  __syncthreads();
  const uint32_t tau = sh.tau;
  auto note = [&](int u) {
    const uint32_t at = atomicAdd(&sh.n_piece, 1u);
    if (at < (uint32_t)kPieces) sh.piece[at] = (uint32_t)tid | (uint32_t)u << 10;
  };
  const int n_unit = (s1 - s0 + T * U - 1) / (T * U);
  if (k1 >= tau) {
    if (k3 >= tau) {
      for (int u = 0; u < n_unit; ++u) {
        note(u);
        if (*(volatile uint32_t*)&sh.n_piece > (uint32_t)kPieces) break;  // too many: the scan below
      }
    } else {
      note(u1);
      if (k2 >= tau) note(u2);
    }
  }
  __syncthreads();
  const int n_piece = (int)sh.n_piece;
  bool full = n_piece > kPieces;
  if (!full) {
    for (int i = tid; i < n_piece * U; i += T) {
      const uint32_t p = sh.piece[i / U];
      const int slot = s0 + ((int)(p >> 10) * U + i % U) * T + (int)(p & 1023u);
      if (slot >= s1) continue;
      const Slot x = z.load(slot);
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        const float v = slot_value<DT>(x, q);
        if (value_key(v) >= tau) {
          const uint32_t at = atomicAdd(&sh.n_key, 1u);
          if (at < (uint32_t)kCap) sh.key[at] = token_key(v, slot * VE + q);
        }
      }
    }
    __syncthreads();
    full = sh.n_key > (uint32_t)kCap;
  }
  if (full)
    top_by_scan<DT, T>(sh, z, s0, s1, N);
  else
    rank_keys(sh, (int)sh.n_key, N);
}

// adds the terms of U slots to s and h
template <int DT, bool ENT, bool MASKED, int U>
__device__ __forceinline__ void add_terms(Slot (&x)[U], float c, float M, double& s, double& h) {
  constexpr int VE = RowType<DT>::VE;
  float ps[U], ph[U];
#pragma unroll
  for (int l = 0; l < U; ++l) {
    ps[l] = ph[l] = 0.0f;
    if (MASKED) {  // or the compiler takes the words apart before it branches here, into twice the registers
#pragma unroll
      for (int d = 0; d < 4; ++d) asm volatile("" : "+v"(x[l].w[d]));
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      const float t = fmaf(slot_value<DT>(x[l], i), c, -M);
      const float e = __builtin_amdgcn_exp2f(t);
      ps[l] += e;
      if (ENT) ph[l] = fmaf(e, MASKED ? fmaxf(t, -256.0f) : t, ph[l]);  // 0 times -inf
    }
    asm volatile("" : "+v"(ps[l]), "+v"(ph[l]));  // slot by slot: else all terms are kept at once, and spill
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int w = 1; w < U; w *= 2)
#pragma unroll
    for (int l = 0; l < U; l += 2 * w) ps[l] += ps[l + w], ph[l] += ph[l + w];
  s += (double)ps[0];
  if (ENT) h += (double)ph[0];
}

// A slot whose elements' order does not matter: the last one of a row comes as the 16
// bytes that end with the row, what the slot before it holds of them masked;
// slots from s1 on are masked.  Rows of at least one whole slot.
template <int DT>
__device__ __forceinline__ Slot load_unordered(const RowRef<DT>& z, int slot, int s1) {
  constexpr int VE = RowType<DT>::VE;
  const int e = slot * VE, at = min(e, z.V - VE);
  const u32x4_any v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(z.p + at));
  Slot s{{v.x, v.y, v.z, v.w}};
  const int drop = slot < s1 ? e - at : VE;  // elements that do not belong here
  if (drop > 0) {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (i < drop) {
        if constexpr (DT == DFLASH_BF16)
          s.w[i >> 1] = (i & 1) ? (s.w[i >> 1] & 0x0000FFFFu) | 0xFF800000u : (s.w[i >> 1] & 0xFFFF0000u) | 0x0000FF80u;
        else
          s.w[i] = 0xFF800000u;
      }
  }
  return s;
}

// streams slots s0 .. s1 - 1 of a row
template <int DT, int T, int U, bool ENT, bool TOP>
__device__ __forceinline__ Sums sum_segment(Shared<T>& sh, const RowRef<DT>& z, int s0, int s1, float c, int N) {
  const int tid = threadIdx.x;
  float m1 = kNegInf, m2 = kNegInf, m3 = kNegInf, Mf = -kHuge;
  int u1 = 0, u2 = 0, u = 0;
  double s = 0.0, h = 0.0;
  bool any_odd = false;
#pragma unroll 1
  for (int b = s0; b < s1; b += T * U, ++u) {
    Slot x[U];
    if (b + T * U <= s1 && (b + T * U) * RowType<DT>::VE <= z.V) {
#pragma unroll
      for (int l = 0; l < U; ++l) {
        const u32x4_any v =
            __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(z.p + (b + l * T + tid) * RowType<DT>::VE));
        x[l] = Slot{{v.x, v.y, v.z, v.w}};
      }
    } else if (T > kWave || z.V >= RowType<DT>::VE) {
#pragma unroll
      for (int l = 0; l < U; ++l) x[l] = load_unordered<DT>(z, b + l * T + tid, s1);
    } else {
      x[0] = z.load(tid);
#pragma unroll
      for (int l = 1; l < U; ++l) x[l] = Slot{{RowType<DT>::kMasked, RowType<DT>::kMasked, RowType<DT>::kMasked, RowType<DT>::kMasked}};
    }
    bool odd;
    float low;
    const float m = largest<DT>(x, odd, low);
    any_odd |= odd;
    if (TOP) {
      const bool a1 = m > m1, a2 = m > m2;
      m3 = a2 ? m2 : fmaxf(m3, m);
      m2 = a1 ? m1 : a2 ? m : m2;
      u2 = a1 ? u1 : a2 ? u : u2;
      u1 = a1 ? u : u1;
    }
    if (m > m1) {
      m1 = m;
      const float to = (float)reference(m, c);
      rebase((double)Mf, (double)to, s, h);
      Mf = to;
    }
    if (ENT && __any(!(fmaf(low, c, -Mf) > -3e38f)))  // masked, or so low that t leaves fp32
      add_terms<DT, ENT, true>(x, c, Mf, s, h);
    else
      add_terms<DT, ENT, false>(x, c, Mf, s, h);
  }
  // over the block: the largest logit, then sums at its reference
  float bm = wave_max_dpp_f32(any_odd ? INFINITY : m1);
  if constexpr (T > kWave) {
    if ((tid & 63) == 0) sh.wave_m[tid >> 6] = bm;
    __syncthreads();
    bm = sh.wave_m[0];
#pragma unroll
    for (int w = 1; w < T / kWave; ++w) bm = fmaxf(bm, sh.wave_m[w]);
  }
  Sums r{};
  if (bm == INFINITY) {
    r.m = NAN;
    return r;
  }
  r.m = bm;
  if (bm > kNegInf) {
    r.M = reference(bm, c);
    if (m1 > kNegInf) rebase((double)Mf, r.M, s, h); else s = h = 0.0;
    r.s = wave_sum_dpp_f64(s);
    if (ENT) r.h = wave_sum_dpp_f64(h);
    if constexpr (T > kWave) {
      if ((tid & 63) == 0) sh.wave_s[tid >> 6] = r.s, sh.wave_h[tid >> 6] = r.h;
      __syncthreads();
      r.s = r.h = 0.0;
#pragma unroll
      for (int w = 0; w < T / kWave; ++w) r.s += sh.wave_s[w], r.h += sh.wave_h[w];
    }
  }
  if (TOP) top_of_segment<DT, T, U>(sh, z, s0, s1, N, m1, m2, m3, u1, u2);
  return r;
}

// The sums of a row whose |m| c is beyond kHuge, from z - m (reference m c): one more pass over the
// row, of which most slots have nothing to add where c is that large (2048 x 151936 bf16 at T =
// 1e-6: 252 us, 1340 with every exponential, 116 at T = 1; one such row: 22, 190 and 10).
template <int DT, int T>
__device__ __noinline__ void sum_far(Shared<T>& sh, const RowRef<DT> z, float m, double c, double& s, double& h) {
  constexpr int VE = RowType<DT>::VE, U = 2;
  const int tid = threadIdx.x;
  s = h = 0.0;
#pragma unroll 1
  for (int b = tid; b < z.slots(); b += T * U) {
    Slot x[U];
#pragma unroll
    for (int l = 0; l < U; ++l) x[l] = z.load(b + l * T);
#pragma unroll
    for (int l = 0; l < U; ++l) {
      float top = slot_value<DT>(x[l], 0);
#pragma unroll
      for (int i = 1; i < VE; ++i) top = fmaxf(top, slot_value<DT>(x[l], i));
      if (!(((double)top - (double)m) * c > -1100.0)) continue;  // 2^t is 0
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const double t = fmax(((double)slot_value<DT>(x[l], i) - (double)m) * c, -2000.0), e = exp2(t);
        s += e;
        h = fma(e, t, h);
      }
    }
  }
  s = wave_sum_dpp_f64(s);
  h = wave_sum_dpp_f64(h);
  if constexpr (T > kWave) {
    __syncthreads();
    if ((tid & 63) == 0) sh.wave_s[tid >> 6] = s, sh.wave_h[tid >> 6] = h;
    __syncthreads();
    s = h = 0.0;
#pragma unroll
    for (int w = 0; w < T / kWave; ++w) s += sh.wave_s[w], h += sh.wave_h[w];
  }
}

// a thread's first given token: read before the row is, as one load waits for the other
struct Given {
  int t;    // -1: none, or padding
  float v;  // its logit
};
template <int DT>
__device__ __forceinline__ Given first_given(const LogprobsArgs& a, const RowRef<DT>& z, int64_t row) {
  Given g{-1, 0.0f};
  if ((int)threadIdx.x < a.M) {
    const int t = a.tok[row * a.M + threadIdx.x];
    if (t >= 0 && t < a.V) g = Given{t, row_value<DT>(z, t)};
  }
  return g;
}

// a row's outputs from its sums and its alternatives (sh.top)
template <int DT, int T>
__device__ __forceinline__ void write_row(Shared<T>& sh, const LogprobsArgs& a, const LogprobsOut& o, const RowRef<DT>& z, int64_t row,
                                          Sums r, double c, Given first) {
  const int tid = threadIdx.x;
  double l = 0.0, ent = 0.0;
  if (r.m > kNegInf) {
    double off = r.M - (double)r.m * (double)(float)c;
    if (!(fabsf(r.m) * (float)c < kHuge)) {
      sum_far<DT, T>(sh, z, r.m, c, r.s, r.h);
      off = 0.0;
    }
    const double ls = log2(r.s);
    l = kLn2 * (ls + off);
    ent = fmax(kLn2 * (ls - r.h / r.s), 0.0);
  } else if (r.m != r.m) {
    l = ent = NAN;
  }
  if (tid == 0) {
    o.norm[2 * row] = r.m;
    o.norm[2 * row + 1] = (float)l;
    if (o.entropy) o.entropy[row] = (float)ent;
  }
  const double per = c * kLn2;  // 1 / T
  for (int k = tid; k < a.M; k += T) {
    Given g = first;
    if (k != tid) {
      g.t = a.tok[row * a.M + k];
      if (g.t < 0 || g.t >= a.V) g.t = -1; else g.v = row_value<DT>(z, g.t);
    }
    o.logp[row * a.M + k] = g.t < 0 ? 0.0f : r.m == kNegInf ? kNegInf : (float)(((double)g.v - (double)r.m) * per - l);
  }
  if (tid < a.N) {
    const uint64_t k = r.m > kNegInf ? sh.top[tid] : 0;
    o.top_idx[row * a.N + tid] = k ? key_token(k) : -1;
    o.top_logp[row * a.N + tid] =
        r.m != r.m ? NAN : k ? (float)(((double)key_value(k) - (double)r.m) * per - l) : kNegInf;
  }
}

// One row, or one segment of it, a block: streams it once.
// Eight waves a SIMD hide the loads, four of which a thread has in flight; bound by issue
// slots with the entropy (2048 x 151936 bf16: 116 us, 5.4 TB/s; a read alone reaches 7.0).
template <int DT, int T, int U, bool ENT, bool TOP>
__global__ __launch_bounds__(T, 8) void logprobs_kernel(LogprobsArgs a, LogprobsOut o, int n_seg, int seg_slots,
                                                     LogprobsPart* __restrict__ parts, uint64_t* __restrict__ lists) {
  __shared__ Shared<T> sh;
  const int seg = blockIdx.x % n_seg;
  const int64_t row = blockIdx.x / n_seg;
  const RowRef<DT> z(a.Z, row, a.stride, a.V);
  const double c = row_scale(a.T, a.group, row);
  const Given first = n_seg == 1 ? first_given<DT>(a, z, row) : Given{-1, 0.0f};
  const int s0 = seg * seg_slots, s1 = min(s0 + seg_slots, z.slots());
  const Sums r = sum_segment<DT, T, U, ENT, TOP>(sh, z, s0, s1, (float)c, a.N);
  if (n_seg == 1) {
    write_row<DT, T>(sh, a, o, z, row, r, c, first);
  } else {
    if (threadIdx.x == 0) parts[blockIdx.x] = LogprobsPart{r.M, r.s, r.h, r.m};
    if (TOP && threadIdx.x < a.N) lists[(int64_t)blockIdx.x * a.N + threadIdx.x] = r.m == r.m && r.m > kNegInf ? sh.top[threadIdx.x] : 0;
  }
}

// joins a row's segments
template <int DT, int T>
__global__ __launch_bounds__(T) void logprobs_join_kernel(LogprobsArgs a, LogprobsOut o, int n_seg,
                                                          const LogprobsPart* __restrict__ parts,
                                                          const uint64_t* __restrict__ lists) {
  __shared__ Shared<T> sh;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const double c = row_scale(a.T, a.group, row);
  const LogprobsPart* part = parts + row * n_seg;
  // at most T segments
  LogprobsPart p{0.0, 0.0, 0.0, kNegInf};
  if (tid < n_seg) p = part[tid];
  const uint64_t* list = lists + row * n_seg * a.N;
  const uint64_t mine = a.N > 0 && tid < n_seg ? list[(int64_t)tid * a.N] : 0;  // its segment's best
  const RowRef<DT> z(a.Z, row, a.stride, a.V);
  const Given first = first_given<DT>(a, z, row);
  float bm = wave_max_dpp_f32(p.m != p.m ? INFINITY : p.m);
  if ((tid & 63) == 0) sh.wave_m[tid >> 6] = bm;
  __syncthreads();
  bm = sh.wave_m[0];
#pragma unroll
  for (int w = 1; w < T / kWave; ++w) bm = fmaxf(bm, sh.wave_m[w]);
  Sums r{};
  r.m = bm == INFINITY ? NAN : bm;
  if (r.m > kNegInf) {
    r.M = reference(r.m, (float)c);
    if (p.m > kNegInf) rebase(p.M, r.M, p.s, p.h);
    r.s = wave_sum_dpp_f64(p.s);
    r.h = wave_sum_dpp_f64(p.h);
    if ((tid & 63) == 0) sh.wave_s[tid >> 6] = r.s, sh.wave_h[tid >> 6] = r.h;
    __syncthreads();
    r.s = r.h = 0.0;
#pragma unroll
    for (int w = 0; w < T / kWave; ++w) r.s += sh.wave_s[w], r.h += sh.wave_h[w];
  }
  if (a.N > 0 && r.m > kNegInf) {
    // the N-th largest of the segments' best bounds the row's N-th from below: only
    // the lists of those N segments can hold one, what of them reaches it is ranked
    sh.key[tid] = mine;
    if (tid == 0) sh.least = 1, sh.n_key = 0, sh.n_piece = 0;
    __syncthreads();
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n_seg; ++j) rank += sh.key[j] > mine;
    if (mine && rank < a.N) {
      sh.piece[rank] = (uint32_t)tid;
      atomicMax(&sh.n_piece, (uint32_t)rank + 1);
      if (rank == a.N - 1) sh.least = mine;
    }
    __syncthreads();
    const uint64_t least = sh.least;
    const int n = (int)sh.n_piece * a.N;
    for (int i = tid; i < n; i += T) {
      const uint64_t k = list[(int64_t)sh.piece[i / a.N] * a.N + i % a.N];
      if (k >= least) sh.key[atomicAdd(&sh.n_key, 1u)] = k;
    }
    __syncthreads();
    rank_keys(sh, (int)sh.n_key, a.N);
  }
  write_row<DT, T>(sh, a, o, z, row, r, c, first);
}

// ---------------------------------------------------------------- backward

struct GradRed {
  double d[kLogprobsThreads / kWave];
};

// dz_j = p_j (a0 + a1 log2 p_j) + (the given token's own gradients) / T, with
//   a0 = -(sum g + g_H H) / T,  a1 = -g_H ln 2 / T.
// One read and one write of the row, NL slots a thread as in the distillation's gradient.
// Bound by memory: 2048 x 151936 bf16 in 217 us, 5.75 TB/s.
template <int DT, int NL>
__global__ __launch_bounds__(kLogprobsThreads) void logprobs_grad_kernel(LogprobsArgs a, const float* __restrict__ g_logp,
                                                                         const float* __restrict__ g_ent,
                                                                         const float* __restrict__ norm,
                                                                         const float* __restrict__ entropy, void* dZ,
                                                                         int64_t d_stride, int n_seg) {
  using E = typename RowType<DT>::elem;
  constexpr int VE = RowType<DT>::VE, T = kLogprobsThreads;
  constexpr int kPerThread = DFLASH_LOGPROBS_M_MAX / T;
  __shared__ int tok[DFLASH_LOGPROBS_M_MAX];
  __shared__ float grad[DFLASH_LOGPROBS_M_MAX];
  __shared__ GradRed red;
  const int tid = threadIdx.x, seg = blockIdx.x % n_seg;
  const int64_t row = blockIdx.x / n_seg;
  const RowRef<DT> z(a.Z, row, a.stride, a.V);
  E* o = static_cast<E*>(dZ) + row * d_stride;
  const int s0 = seg * (T * NL), e0 = s0 * VE, e1 = e0 + T * NL * VE;
  const double c = row_scale(a.T, a.group, row), per = c * kLn2;
  const float m = norm[2 * row], l = norm[2 * row + 1];
  const double gh = g_ent ? (double)g_ent[row] : 0.0;

  // the given tokens of the row, and the sum of their gradients
  double A = 0.0;
  bool some = gh != 0.0;
  float own[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int k = j * T + tid;
    if (j * T < a.M && k < a.M) {
      const int t = a.tok[row * a.M + k];
      const bool in = t >= 0 && t < a.V;
      const float g = in ? g_logp[row * a.M + k] : 0.0f;
      tok[k] = in ? t : -1;
      grad[k] = g;
      some |= g != 0.0f;
      A += (double)g;
      if (in && t >= e0 && t < e1) own[j] = row_value<DT>(z, t);
    }
  }
  A = wave_sum_dpp_f64(A);
  if ((tid & 63) == 0) red.d[tid >> 6] = A;
  some = __syncthreads_or(some);
  A = red.d[0];
#pragma unroll
  for (int w = 1; w < T / kWave; ++w) A += red.d[w];
  if (!some || m == kNegInf) {  // no gradient comes in, or nothing is unmasked
#pragma unroll
    for (int q = 0; q < NL; ++q) store_slot<DT>(o, a.V, s0 + q * T + tid, Slot{{0, 0, 0, 0}});
    return;
  }
  Slot x[NL];
#pragma unroll
  for (int q = 0; q < NL; ++q) x[q] = z.template load<true>(s0 + q * T + tid);
  const double H = g_ent ? (double)entropy[row] : 0.0;
  const double b0 = m != m ? (double)NAN : -(A + gh * H), a0 = b0 * per, a1 = -gh * kLn2 * per;
  // log2 p in two pieces of fp32 (-inf: NaN at times, which the maximum below replaces)
  const double l2 = (double)l * kLog2e64;
  const float ch = (float)c, cl = (float)(c - (double)ch), lh = (float)l2, ll = (float)(l2 - (double)lh);
  __syncthreads();  // every given token's logit is read (dZ may be Z)
  auto slots = [&](auto from_t) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NL; ++q) {
      Slot y;
#pragma unroll
      for (int k = 0; k < 4; ++k) y.w[k] = 0;
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float d = slot_value<DT>(x[q], i) - m;
        const float g = from_t(fmaf(d, ch, -lh) + fmaf(d, cl, -ll));
        if constexpr (DT == DFLASH_BF16)
          y.w[i >> 1] |= bf16_round(g) << ((i & 1) * 16);
        else
          y.w[i] = __float_as_uint(g);
      }
      store_slot<DT>(o, a.V, s0 + q * T + tid, y);
      __builtin_amdgcn_sched_barrier(0);  // slot by slot: else the two paths below take a block's registers a CU more
    }
  };
  const double big = fmax(fabs(a0), 256.0 * fabs(a1));
  if (big >= 0x1p60 && big < INFINITY) {
    // factors that fp32 may not hold are multiplied in fp64, by the power of two of t's whole part
    // as well: unlikely tokens' gradients may fit fp32, those of masked ones are 0 (a factor is below 2^250)
    slots([&](float t) {
      t = fmaxf(t, -1000.0f);
      const float n = rintf(t);
      return (float)ldexp((double)__builtin_amdgcn_exp2f(t - n) * fma(a1, (double)t, a0), (int)n);
    });
  } else {
    const float f0 = (float)a0, f1 = (float)a1;
    slots([&](float t) {
      t = fmaxf(t, -256.0f);
      return __builtin_amdgcn_exp2f(t) * fmaf(f1, t, f0);
    });
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int k = j * T + tid;
    if (j * T < a.M && k < a.M && tok[k] >= e0 && tok[k] < e1) {
      double g = 0.0;  // every entry of this token, in order
      for (int q = 0; q < a.M; ++q)
        if (tok[q] == tok[k]) g += (double)grad[q];
      const double lp = ((double)own[j] - (double)m) * per - (double)l;
      const double p = exp(lp);
      // all that may cancel comes before 1 / T: a token with p = 1 has exactly 0
      if (p > 0.0) g += p * (b0 - gh * lp);
      if (m != m) g = NAN;
      o[tok[k]] = to_elem<DT>((float)(g * per));
    }
  }
}

template <int DT, int T, int U, bool ENT, bool TOP>
hipError_t run(const LogprobsArgs& a, const LogprobsOut& o, char* ws, const LogprobsPlan& pl, hipStream_t st) {
  LogprobsPart* parts = reinterpret_cast<LogprobsPart*>(ws);
  uint64_t* lists = reinterpret_cast<uint64_t*>(ws + pl.lists);
  launch(logprobs_kernel<DT, T, U, ENT, TOP>, dim3((unsigned)(a.R * pl.n_seg)), dim3(T), st, a, o, pl.n_seg, pl.seg_slots, parts,
         lists);
  if (pl.n_seg > 1)
    launch(logprobs_join_kernel<DT, kLogprobsThreads>, dim3((unsigned)a.R), dim3(kLogprobsThreads), st, a, o, pl.n_seg,
           (const LogprobsPart*)parts, (const uint64_t*)lists);
  return hipGetLastError();
}

template <int DT, int T, int U>
hipError_t run_sized(const LogprobsArgs& a, const LogprobsOut& o, char* ws, const LogprobsPlan& pl, hipStream_t st) {
  if (a.N > 0) return o.entropy ? run<DT, T, U, true, true>(a, o, ws, pl, st) : run<DT, T, U, false, true>(a, o, ws, pl, st);
  return o.entropy ? run<DT, T, U, true, false>(a, o, ws, pl, st) : run<DT, T, U, false, false>(a, o, ws, pl, st);
}

template <int DT>
hipError_t run_typed(const LogprobsArgs& a, const LogprobsOut& o, char* ws, const LogprobsPlan& pl, hipStream_t st) {
  if (pl.threads == kWave) return run_sized<DT, kWave, 4>(a, o, ws, pl, st);
  if (pl.threads == 512) return run_sized<DT, 512, 4>(a, o, ws, pl, st);
  if (pl.threads == 1024) return run_sized<DT, 1024, 4>(a, o, ws, pl, st);
  return pl.unit == 1 ? run_sized<DT, kLogprobsThreads, 1>(a, o, ws, pl, st) : run_sized<DT, kLogprobsThreads, 4>(a, o, ws, pl, st);
}

template <int DT>
hipError_t run_grad(const LogprobsArgs& a, const float* g_logp, const float* g_ent, const float* norm, const float* entropy,
                    void* dZ, int64_t d_stride, const LogprobsPlan& pl, hipStream_t st) {
  const dim3 grid((unsigned)(a.R * pl.grad_seg)), block(kLogprobsThreads);
  switch (pl.grad_loads) {
    case 1: launch(logprobs_grad_kernel<DT, 1>, grid, block, st, a, g_logp, g_ent, norm, entropy, dZ, d_stride, pl.grad_seg); break;
    case 2: launch(logprobs_grad_kernel<DT, 2>, grid, block, st, a, g_logp, g_ent, norm, entropy, dZ, d_stride, pl.grad_seg); break;
    case 4: launch(logprobs_grad_kernel<DT, 4>, grid, block, st, a, g_logp, g_ent, norm, entropy, dZ, d_stride, pl.grad_seg); break;
    default: launch(logprobs_grad_kernel<DT, 8>, grid, block, st, a, g_logp, g_ent, norm, entropy, dZ, d_stride, pl.grad_seg);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(int32_t dtype, const LogprobsArgs& a, const LogprobsOut& o, char* ws, const LogprobsPlan& pl,
                           hipStream_t st) {
  return dtype == DFLASH_BF16 ? run_typed<DFLASH_BF16>(a, o, ws, pl, st) : run_typed<DFLASH_F32>(a, o, ws, pl, st);
}

hipError_t launch_logprobs_grad(int32_t dtype, const LogprobsArgs& a, const float* g_logp, const float* g_ent, const float* norm,
                                const float* entropy, void* dZ, int64_t d_stride, const LogprobsPlan& pl, hipStream_t st) {
  return dtype == DFLASH_BF16 ? run_grad<DFLASH_BF16>(a, g_logp, g_ent, norm, entropy, dZ, d_stride, pl, st)
                              : run_grad<DFLASH_F32>(a, g_logp, g_ent, norm, entropy, dZ, d_stride, pl, st);
}

}  // namespace dfk
