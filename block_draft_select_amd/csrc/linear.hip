// dflash_linear_i8: y_rn = xs_r ws_n sum_k xq_rk wq_nk, rows of 8-bit integers
// with a scale each; the sums are exact in 32 bits.
//
// On the matrix cores (v_mfma_i32_16x16x64_i8): the weights are the A operand,
// the tokens the B operand, so a lane of the result holds four neighbouring
// channels of one token.  Lane l of either operand holds the 16 bytes
// 16 (l / 16) .. of row l % 16 and of 64 bytes of k.  Only the tokens' side is
// cleared past the row's end: what the weights hold there is multiplied by zero.
#include <algorithm>

#include "linear_loads.hpp"
#include "rows_blocks.hpp"

namespace dfk {

namespace {

typedef int v4i32 __attribute__((ext_vector_type(4)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// NV values to a row of any element-aligned address, each rounded to the type
template <int DT, int NV>
__device__ __forceinline__ void store_values(typename RowType<DT>::elem* p, const float (&v)[NV]) {
  constexpr int VE = RowType<DT>::VE;
#pragma unroll
  for (int q = 0; q < NV / VE; ++q) {
    u32x4_any o;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if constexpr (DT == DFLASH_BF16)
        o[d] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[q * 8 + 2 * d], v[q * 8 + 2 * d + 1]}), bf16x2));
      else
        o[d] = __float_as_uint(v[q * 4 + d]);
    }
    *reinterpret_cast<u32x4_any*>(p + q * VE) = o;
  }
}

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// four of them
template <int DT>
__device__ __forceinline__ void store4(typename RowType<DT>::elem* p, const float (&v)[4]) {
  if constexpr (DT == DFLASH_BF16)
    *reinterpret_cast<u32x2_any*>(p) = u32x2_any{__builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[0], v[1]}), bf16x2)),
                                                 __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[2], v[3]}), bf16x2))};
  else
    *reinterpret_cast<u32x4_any*>(p) = u32x4_any{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
}

// Workgroup barrier for LDS hand-offs only: __syncthreads() would also wait for
// every global load in flight
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // vmcnt 63 (no wait), expcnt 7, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// An array of 8-bit rows from `row` on as a buffer
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const int8_t* p, int64_t row, int64_t rows, int64_t stride, int H) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p) + row * stride, 0, buffer_bytes(row, rows, stride, H), 0x00027000);
}

// 16 bytes a lane from a buffer straight into LDS, at 16 l past the wave's address
__device__ __forceinline__ void load_to_lds16(__amdgpu_buffer_rsrc_t b, int offset, unsigned char* l) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, l, 16, offset, 0, 0, 0);
#endif
}

// vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N <= 63, "the field");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
}

// Weights whose rows are a multiple of 4096 bytes apart begin in the same memory channels,
// all of them: blocks that go through k in step then read from a few channels at a time.
// There each begins at a place of its own (sums of integers have no order); elsewhere
// that gains nothing, and costs where rows are 2048 bytes apart (1 x 2048 x 151936: 57 us,
// 53; 1 x 4096 x 100000: 79, 85).
bool shifted(const LinearArgs& a) { return a.wq_stride % 4096 == 0; }

// Few tokens: 16 channels and 16 MT tokens a block, its four waves split k.
// Each wave has eight steps of 64 bytes in flight.  The operands go straight to registers,
// neighbouring lanes in different rows: at 30 to 40 bytes a nanosecond and CU that is the
// slowest way to read, but the one that starts first (1 x 2048 x 2048: the 6.5 us of host
// time that a call takes; 1 x 8192 x 65536, one round of blocks after another: 96 us, 5.6 TB/s).
template <int DT, int MT>
__global__ __launch_bounds__(256) void linear_few_kernel(LinearArgs a) {
  constexpr int U = 8;
  __shared__ int part[4][MT * 4][64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int n_ct = (a.N + 15) / 16;
  const int ch0 = (int)(blockIdx.x % n_ct) * 16;
  const int64_t row0 = (int64_t)(blockIdx.x / n_ct) * 16 * MT;
  const int chunks = (a.H + 15) / 16;                 // 16-byte pieces of a row
  const int steps = (chunks + 3) / 4;                 // of 64 bytes
  const int per = (steps + 3) / 4;                    // steps a wave
  const int st0 = wave * per, st1 = min(st0 + per, steps);
  const int8_t* w = a.wq + (int64_t)min(ch0 + (lane & 15), a.N - 1) * a.wq_stride;
  const int8_t* x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = row0 + m * 16 + (lane & 15);
    x[m] = a.xq + (row < a.R ? row : a.R - 1) * a.xq_stride;
  }
  v4i32 acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = (v4i32){0, 0, 0, 0};
  const int last_valid = a.H - (chunks - 1) * 16;     // bytes of the last piece, 1..16
  for (int s0 = st0; s0 < st1; s0 += U) {
    v4i32 wv[U], xv[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = min((s0 + u) * 4 + (lane >> 4), chunks - 1);
      wv[u] = __builtin_nontemporal_load(reinterpret_cast<const v4i32*>(w + (int64_t)c * 16));
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[u][m] = *reinterpret_cast<const v4i32*>(x[m] + (int64_t)c * 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (s0 + u) * 4 + (lane >> 4);
      // bytes of this piece inside the row and inside this wave's part
      const int valid = s0 + u >= st1 || c >= chunks ? 0 : c == chunks - 1 ? last_valid : 16;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (valid < 16) {
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int b = valid - 4 * d;
            xv[u][m][d] = b <= 0 ? 0 : b >= 4 ? xv[u][m][d] : (int)((uint32_t)xv[u][m][d] & ((1u << (8 * b)) - 1u));
          }
        }
        acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u], xv[u][m], acc[m], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][m * 4 + e][lane] = acc[m][e];
  __syncthreads();
  using E = typename RowType<DT>::elem;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = tid >> 4, c = tid & 15;
    const int from = (c >> 2) * 16 + t, e = m * 4 + (c & 3);
    const int sum = part[0][e][from] + part[1][e][from] + part[2][e][from] + part[3][e][from];
    const int64_t row = row0 + m * 16 + t;
    if (row < a.R && ch0 + c < a.N)
      static_cast<E*>(a.y)[row * a.y_stride + ch0 + c] = to_elem<DT>((float)sum * a.xs[row] * a.ws[ch0 + c]);
  }
}

template <int DT, int MT>
hipError_t run_few(const LinearArgs& a, hipStream_t st) {
  const int64_t blocks = (int64_t)((a.N + 15) / 16) * ((a.R + 16 * MT - 1) / (16 * MT));
  launch(linear_few_kernel<DT, MT>, dim3((unsigned)blocks), dim3(256), st, a);
  return hipGetLastError();
}

// Few tokens and many channels: the tokens' rows stay in LDS, and each of a CU's eight
// waves streams the weights of 16 channels at a time through a ring of its own
// there, 128 bytes of k a step; no wave waits for another.  Rows of 128 bytes (of
// the ring) and of whole 128 bytes (of the tokens) hold piece c of row r at place
// c ^ (r % 8).  What lies behind a token row's end is zero.
// Bound by the weights' bytes: 2048 x 151936 in 53.5 us for one token (5.8 TB/s of the 7.0 that
// a read reaches), 59 for 16, 64 for 32, where the tiles below take 66, 69 and 72.
template <int DT, int MT, int XBYTES, bool SHIFT>
__global__ __launch_bounds__(512, 2) void linear_stream_kernel(LinearArgs a) {
  constexpr int D = (kLdsBytes - XBYTES) / 8 / 2048;  // steps in a wave's ring
  __shared__ __attribute__((aligned(1024))) unsigned char lds[XBYTES + 8 * D * 2048];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int steps = (a.H + 127) / 128, pitch = steps * 128;
  const int n_group = (a.N + 15) / 16, stride = (int)gridDim.x * 8;
  int group = (int)blockIdx.x * 8 + wave;  // a block's waves read neighbouring rows
  const int total = group < n_group ? ((n_group - 1 - group) / stride + 1) * steps : 0;

  unsigned char* ring = lds + XBYTES + wave * (D * 2048);
  const int w_stride = (int)a.wq_stride;
  const int wo[2] = {stream_channel(lane, 0) * w_stride + load_piece(lane), stream_channel(lane, 1) * w_stride + load_piece(lane)};
  const int rot = SHIFT ? (wave * 3 + (int)blockIdx.x) % steps : 0;  // the step that a group begins with
  int load_group = group, load_step = rot, load_slot = 0;
  __amdgpu_buffer_rsrc_t wb = rows_buffer(a.wq, (int64_t)min(group, n_group - 1) * 16, a.N, a.wq_stride, a.H);
  // the next step; behind the last one, the last group's rows again, which no one reads
  auto load = [&]() __attribute__((always_inline)) {
    load_to_lds16(wb, wo[0] + load_step * 128, ring + load_slot * 2048);
    load_to_lds16(wb, wo[1] + load_step * 128, ring + load_slot * 2048 + 1024);
    load_slot = load_slot + 1 == D ? 0 : load_slot + 1;
    if (++load_step == steps) load_step = 0;
    if (load_step == rot) {
      load_group += stride;
      if (load_group < n_group) wb = rows_buffer(a.wq, (int64_t)load_group * 16, a.N, a.wq_stride, a.H);
    }
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) load();

  const int chunks = (a.H + 15) / 16, places = steps * 8;
  for (int q = tid; q < MT * 16 * places; q += 512) {
    const int r = q / places, c = q - r * places;
    v4i32 v = {0, 0, 0, 0};
    if (r < a.R && c < chunks) {
      v = *reinterpret_cast<const v4i32*>(a.xq + r * a.xq_stride + c * 16);
      const int valid = a.H - c * 16;
      if (valid < 16) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int n = valid - 4 * d;
          v[d] = n <= 0 ? 0 : n >= 4 ? v[d] : (int)((uint32_t)v[d] & ((1u << (8 * n)) - 1u));
        }
      }
    }
    *reinterpret_cast<v4i32*>(lds + r * pitch + (c ^ (r & 7)) * 16) = v;
  }
  __syncthreads();

  const int i16 = lane & 15, g4 = lane >> 4;
  int fo[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) fo[ks] = ((4 * ks + g4) ^ (i16 & 7)) * 16;
  v4i32 acc[MT];
  float xs[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    acc[m] = (v4i32){0, 0, 0, 0};
    xs[m] = a.xs[min(m * 16 + i16, (int)a.R - 1)];
  }
  typedef const float __attribute__((address_space(4))) * Scales;
  const Scales ws = (Scales)(uintptr_t)a.ws;
  int step = rot, slot = 0;
#pragma unroll 1
  for (int q = 0; q < total; ++q) {
    asm volatile("" ::: "memory");
    wait_loads<2 * (D - 2)>();  // this step's are done when only those of the D - 2 after it remain
    asm volatile("" ::: "memory");
    v4i32 wv[2], xv[2][MT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      wv[ks] = *reinterpret_cast<const v4i32*>(ring + slot * 2048 + i16 * 128 + fo[ks]);
#pragma unroll
      for (int m = 0; m < MT; ++m) xv[ks][m] = *reinterpret_cast<const v4i32*>(lds + (m * 16 + i16) * pitch + step * 128 + fo[ks]);
    }
    load();  // into the slot that the step before used
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[ks], xv[ks][m], acc[m], 0, 0, 0);
    slot = slot + 1 == D ? 0 : slot + 1;
    if (++step == steps) step = 0;
    if (step != rot) continue;
    const int ch = group * 16 + g4 * 4;
    // the channels' scales through scalar loads: a vector load's wait would drain the ring
    float sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) v[g] = ws[min(group * 16 + g * 4 + j, a.N - 1)];
      sc[j] = g4 < 2 ? (g4 == 0 ? v[0] : v[1]) : g4 == 2 ? v[2] : v[3];
    }
    group += stride;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = m * 16 + i16;
      if (row < a.R) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)acc[m][j] * xs[m] * sc[j];
        typename RowType<DT>::elem* y = static_cast<typename RowType<DT>::elem*>(a.y) + row * a.y_stride + ch;
        if (ch + 4 <= a.N) {
          store4<DT>(y, v);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (ch + j < a.N) y[j] = to_elem<DT>(v[j]);
        }
      }
      acc[m] = (v4i32){0, 0, 0, 0};
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no transfer outlives the wave
}

// A wave's 64 channels from ch on of 16 TT tokens from row on, by way of 16 rows of LDS of its
// own: neighbouring lanes then write one row's line (16 rows' pieces of 16 bytes in an
// instruction, as the products leave them, take 82 us at 1883 x 64 x 53594, these 72).
// All scales are here before the first store: a load between stores waits for them.
template <int DT, int TT>
__device__ __forceinline__ void store_tile(const LinearArgs& a, const v4i32 (&acc)[TT][4], int ch, int64_t row, unsigned char* buf) {
  using E = typename RowType<DT>::elem;
  constexpr int VE = RowType<DT>::VE, LANES = 64 / VE, ROWS = 64 / LANES, PITCH = 64 * (int)sizeof(E) + 16;
  const int lane = threadIdx.x & 63, i16 = lane & 15, g4 = lane >> 4;
  float sc[16], xs[TT];
#pragma unroll
  for (int j = 0; j < 16; ++j) sc[j] = a.ws[ch + g4 * 16 + j];
#pragma unroll
  for (int t = 0; t < TT; ++t) xs[t] = a.xs[min(row + 16 * t + i16, a.R - 1)];
  __builtin_amdgcn_s_waitcnt(0x0F70);
  asm volatile("" ::: "memory");
  unsigned char* put = buf + i16 * PITCH + g4 * 16 * (int)sizeof(E);
  const unsigned char* get = buf + lane / LANES * PITCH + lane % LANES * 16;
  E* y = static_cast<E*>(a.y) + ch + lane % LANES * VE;
#pragma unroll
  for (int t = 0; t < TT; ++t, row += 16) {
    if (row >= a.R) break;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = (float)acc[t][j >> 2][j & 3] * xs[t] * sc[j];
    store_values<DT>(reinterpret_cast<E*>(put), v);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int k = 0; k < 16 / ROWS; ++k) {
      const v4i32 x = *reinterpret_cast<const v4i32*>(get + k * ROWS * PITCH);
      const int64_t to = row + k * ROWS + lane / LANES;
      if (to < a.R) *reinterpret_cast<u32x4_any*>(y + to * a.y_stride) = __builtin_bit_cast(u32x4_any, x);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int DT, int MT, int XBYTES>
hipError_t run_stream(const LinearArgs& a, hipStream_t st) {
  const int want = ((a.N + 15) / 16 + 7) / 8;  // a block a CU, or fewer if the channels do not give each wave some
  const dim3 grid((unsigned)(want < 256 ? want : 256)), block(512);
  if (shifted(a))
    launch(linear_stream_kernel<DT, MT, XBYTES, true>, grid, block, st, a);
  else
    launch(linear_stream_kernel<DT, MT, XBYTES, false>, grid, block, st, a);
  return hipGetLastError();
}

template <int DT, int MT>
hipError_t run_stream_sized(const LinearArgs& a, int bytes, hipStream_t st) {
  if (bytes <= 32768) return run_stream<DT, MT, 32768>(a, st);
  if (bytes <= 65536) return run_stream<DT, MT, 65536>(a, st);
  return run_stream<DT, MT, 98304>(a, st);
}

// Many tokens: a block of eight waves owns 256 channels and 32 TT tokens, a wave 64
// channels and 16 TT tokens.  Stages of 128 bytes of k go from global memory straight
// into a ring of NB in LDS, eight lanes to a row's cache line.  (Loading the
// weights straight into the operand's registers puts neighbouring lanes in different
// rows: 38 bytes a nanosecond and CU against 125 this way, 100 with 64 bytes of a
// row; 1152 x 4096 x 262144 took 1490 us so, 1234 with stages of 64 bytes.)
// A stage in LDS: rows of 128 bytes, piece c of row r at place c ^ (r % 8), so that the
// eight rows that are read at once lie in different banks.  The channels' rows are
// dealt out so that a lane ends up with 16 neighbouring channels: row i of tile c is
// channel 16 (i / 4) + 4 c + i % 4.
// Rows that all begin in the same places of memory: few row tiles begin with a stage of
// their own, where the tokens fit into half an XCD's L2 (64 x 8192 x 65536: 97 us, 132 all
// with the first; 2048 x 4096 x 65536, tokens of 8 MiB: 560, 510).
// A stage is waited for late in the one before it, at a barrier of its own, so that
// the operands it begins with are read before it begins and the loads of the stages
// behind it stay in flight.  By then its own rows are read too: the ring of two takes the
// weights of the stage after next into their place at once (1152 x 4096 x 262144: 1134 us,
// 1202 with all loads a little later; rings of three and four lose 2 % by it).
// What bounds it: with many tokens a stage's LDS traffic and its products each take 0.6
// of its time, at a clock that the load pulls down to 1.9 GHz (1152 x 4096 x 262144: 1100 to
// 1130 us, 2190 to 2250 TOP/s, the matrix cores busy for 62 %).  With fewer, a tile's first
// round trip and its stores, which nothing covers where a block is alone on its CU, and weights at
// half of the memory's rate (256 tokens of 2048 times 151936 channels: 110 us, the bytes 57;
// its 1188 tiles of 16 stages are 4.6 rounds of 256 CUs); for 128 tokens also that 594 tiles
// make three rounds where 2.3 would do (86 us, the bytes 50).
template <int DT, int TT, bool SHIFT>
__global__ __launch_bounds__(512, 2) void linear_tile_kernel(LinearArgs a, int n_rt, int n_ct) {
  using L = TileLoads<TT>;
  constexpr int BM = L::BM, SB = L::SB, NB = L::NB, PER = L::PER, G = TT / 2;
  constexpr int E = NB == 2 ? 4 : 0;  // loads that go out behind the stage's own barrier, into its place
  constexpr int LG = NB == 2 ? (2 * G + 3) / 4 : 2 * G - 1;  // groups that bring loads: early ones if they have to land in this stage
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NB * SB];
  // ids with the same value mod 8 run on one XCD: the row tiles of a channel tile follow one another there
  const int grp = blockIdx.x / (8 * n_rt), rem = blockIdx.x - grp * 8 * n_rt;
  const int rt = rem >> 3, ct = grp * 8 + (rem & 7);
  if (ct >= n_ct) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wc = wave & 3, wm = wave >> 2;
  // the last tiles step back to whole ones: some channels are computed twice, alike (N >= 64)
  const int chb = min(ct * kTileCh, a.N - 64);
  const int64_t row0 = (int64_t)rt * BM;
  const int n_st = (a.H + 127) / 128;

  const int i16 = lane & 15, g4 = lane >> 4;
  const int w_stride = (int)a.wq_stride, x_stride = (int)a.xq_stride;
  const __amdgpu_buffer_rsrc_t wb = rows_buffer(a.wq, chb, a.N, a.wq_stride, a.H);
  const __amdgpu_buffer_rsrc_t xb = rows_buffer(a.xq, row0, a.R, a.xq_stride, a.H);
  const int chw = min(ct * kTileCh + (wave >> 1) * 64, a.N - 64) - chb;
  int lo[PER];  // of the wave's loads, in the first stage
#pragma unroll
  for (int i = 0; i < PER; ++i)
    lo[i] = (i < 4 ? (chw + tile_channel(wave, lane, i)) * w_stride : tile_token<TT>(wave, lane, i) * x_stride) + load_piece(lane);
  const int rot = SHIFT ? (ct >> 3) * 5 % n_st : 0;
  auto place = [&](int s) __attribute__((always_inline)) { return SHIFT ? tile_stage(s, rot, n_st) : s; };
  // the wave's i-th load of stage s
  auto load = [&](int s, int buf, int i) __attribute__((always_inline)) {
    unsigned char* to = lds + buf * SB + (i < 4 ? wave * 4 + i : 32 + wave * (TT / 2) + i - 4) * 1024;
    load_to_lds16(i < 4 ? wb : xb, lo[i] + place(s) * 128, to);
  };
  auto barrier = [&]() __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // the tokens' bytes behind the rows' end, in a stage that holds such
  auto clear = [&](int s, int buf) __attribute__((always_inline)) {
    if (s * 128 + 128 > a.H) {
      const int valid = a.H - s * 128;
      uint32_t* p = reinterpret_cast<uint32_t*>(lds + buf * SB + kTileCh * 128);
#pragma unroll 1
      for (int q = tid; q < BM * 32; q += 512) {  // words
        const int n = valid - (((q >> 2) & 7) ^ ((q >> 5) & 7)) * 16 - (q & 3) * 4;
        if (n < 4) p[q] = n <= 0 ? 0u : p[q] & ((1u << (8 * n)) - 1u);
      }
      lds_barrier();
    }
  };

  int fo[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) fo[ks] = i16 * 128 + ((4 * ks + g4) ^ (i16 & 7)) * 16;
  const unsigned char* wf = lds + wc * 8192;
  const unsigned char* xf = lds + kTileCh * 128 + wm * (TT * 2048);
  v4i32 acc[TT][4], wv[2][4], xv[2][2];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[t][c] = (v4i32){0, 0, 0, 0};

#pragma unroll
  for (int s = 0; s < NB - 1; ++s) {
#pragma unroll
    for (int i = 0; i < PER; ++i) load(s, s, i);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) load(NB - 1, NB - 1, i);
  asm volatile("" ::: "memory");
  wait_loads<PER * (NB - 2) + E>();
  barrier();
  clear(place(0), 0);
#pragma unroll
  for (int c = 0; c < 4; ++c) wv[0][c] = *reinterpret_cast<const v4i32*>(wf + c * 2048 + fo[0]);
#pragma unroll
  for (int t = 0; t < 2; ++t) xv[0][t] = *reinterpret_cast<const v4i32*>(xf + t * 2048 + fo[0]);

  int buf = 0;
#pragma unroll 1
  for (int s = 0; s < n_st; ++s) {
    const int next = buf + 1 == NB ? 0 : buf + 1, refill = buf == 0 ? NB - 1 : buf - 1;
    // The refilled stage s - 1 is read no more: the wait before its barrier was for LDS reads
    // too, and all of them had been issued by then
#pragma unroll
    for (int g = 0; g < 2 * G; ++g) {
      const int ks = g / G;
      __builtin_amdgcn_sched_barrier(0);
      if (g == 2 * G - 1) {
        asm volatile("" ::: "memory");
        wait_loads<PER * (NB - 2)>();  // stage s + 1 has landed, and stage s is read
        barrier();
        if (s + 1 < n_st) clear(place(s + 1), next);
#pragma unroll
        for (int i = 0; i < E; ++i) load(s + NB, buf, i);
      }
      const unsigned char* from = g + 1 < 2 * G ? xf + buf * SB + ((g + 1) % G) * 4096 + fo[(g + 1) / G % 2] : xf + next * SB + fo[0];
#pragma unroll
      for (int t = 0; t < 2; ++t) xv[(g + 1) & 1][t] = *reinterpret_cast<const v4i32*>(from + t * 2048);
      if (g == G - 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) wv[1][c] = *reinterpret_cast<const v4i32*>(wf + buf * SB + c * 2048 + fo[1]);
      }
      if (g == 2 * G - 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) wv[0][c] = *reinterpret_cast<const v4i32*>(wf + next * SB + c * 2048 + fo[0]);
      }
#pragma unroll
      for (int i = E; i < PER; ++i)
        if ((i - E) * LG / PER == g) load(s + NB - 1, refill, i);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[g % G * 2 + t][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[ks][c], xv[g & 1][t], acc[g % G * 2 + t][c], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    buf = next;
  }
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0): no transfer outlives the loop
  barrier();
  store_tile<DT, TT>(a, acc, min(ct * kTileCh + wc * 64, a.N - 64), row0 + wm * TT * 16, lds + wave * 4608);
}

template <int DT, int TT>
hipError_t run_tile(const LinearArgs& a, hipStream_t st) {
  const int n_ct = (a.N + kTileCh - 1) / kTileCh;
  const int n_rt = (int)((a.R + 32 * TT - 1) / (32 * TT));
  const dim3 grid((unsigned)((int64_t)((n_ct + 7) / 8) * 8 * n_rt)), block(512);
  if (shifted(a) && a.R * a.H <= (1 << 21))
    launch(linear_tile_kernel<DT, TT, true>, grid, block, st, a, n_rt, n_ct);
  else
    launch(linear_tile_kernel<DT, TT, false>, grid, block, st, a, n_rt, n_ct);
  return hipGetLastError();
}

struct LinearPlan {
  int few;     // 16-token tiles of the few-tokens kernel, or 0
  int stream;  // of the streaming kernel, or 0
  int tile;    // TT of the tile kernel
  int64_t blocks;
};

constexpr int kStreamBytes = 98304;

int stream_bytes(int tiles, int32_t H) { return tiles * 16 * ((H + 127) / 128 * 128); }

// The streaming kernel wherever its tokens fit and the channels give half of its waves
// 16 (with cold weights within 20 % of the best of 159 shapes: 16 x 1024 x 24000: 10 us, the
// few-tokens kernel 8.5; 16 x 512 x 151936: 18, tiles 24); else the least of the others' times
// in nanoseconds, fitted to them over 405 shapes from 1 x 64 x 100 to 2048 x 512 x 151936 (1.3 %
// above the best one on average, 18 % at most but for 1152 x 64 x 151936, all output).  The few-tokens kernel: a start, and
// the most of a round trip to memory for every eight steps of a wave, its loads at 38
// bytes a CU, and what a block costs.  The tiles: a start, and rounds of 256 blocks at a time a stage
// that grows with the tile, or the weights at half of the memory's rate (a quarter of
// the rounds' time once more, as they do not overlap in whole).
LinearPlan linear_plan(int64_t R, int32_t N, int32_t H) {
  LinearPlan p{};
  const int tiles = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  if (R <= 64 && N >= 16384 && stream_bytes(tiles, H) <= kStreamBytes) {
    p.stream = tiles;
    p.blocks = 256;
    return p;
  }
  const int64_t st = (H + 63) / 64;
  double least = 1e300;
  for (int mt = 1; mt <= 4; mt *= 2) {
    const int64_t blocks = (int64_t)((N + 15) / 16) * ((R + 16 * mt - 1) / (16 * mt));
    const double rounds = (double)((blocks + 255) / 256);
    const double t = 4000.0 + std::max({900.0 * (double)((st + 31) / 32), rounds * (double)((1 + mt) * 1024 * st) / 38.0,
                                        rounds * (500.0 + 900.0 * mt)});
    if (t <= least) {
      least = t;
      p.few = mt;
      p.blocks = blocks;
    }
  }
  if (N < 64) return p;
  for (int tt = 2; tt <= 8; tt *= 2) {
    const int64_t blocks = (int64_t)((N + kTileCh - 1) / kTileCh) * ((R + 32 * tt - 1) / (32 * tt));
    const double stage = tt == 2 ? 250.0 : tt == 4 ? 330.0 : 590.0;
    const double work = (double)((blocks + 255) / 256 * st) * stage, read = (double)N * H / 3700.0;
    const double t = 3500.0 + std::max(work, read) + work / 4;
    if (t < least) {
      least = t;
      p.few = 0;
      p.tile = tt;
      p.blocks = (int64_t)((N + kTileCh * 8 - 1) / (kTileCh * 8)) * 8 * ((R + 32 * tt - 1) / (32 * tt));
    }
  }
  return p;
}

template <int DT>
hipError_t run_typed(const LinearArgs& a, hipStream_t st) {
  const LinearPlan p = linear_plan(a.R, a.N, a.H);
  switch (p.stream) {
    case 0: break;
    case 1: return run_stream_sized<DT, 1>(a, stream_bytes(1, a.H), st);
    case 2: return run_stream_sized<DT, 2>(a, stream_bytes(2, a.H), st);
    default: return run_stream_sized<DT, 4>(a, stream_bytes(4, a.H), st);
  }
  if (p.few == 1) return run_few<DT, 1>(a, st);
  if (p.few == 2) return run_few<DT, 2>(a, st);
  if (p.few == 4) return run_few<DT, 4>(a, st);
  switch (p.tile) {
    case 2: return run_tile<DT, 2>(a, st);
    case 4: return run_tile<DT, 4>(a, st);
    default: return run_tile<DT, 8>(a, st);
  }
}

}  // namespace

int64_t linear_blocks(int64_t R, int32_t N, int32_t H) { return linear_plan(R, N, H).blocks; }

hipError_t launch_linear_i8(int32_t dtype, const LinearArgs& a, hipStream_t st) {
  return dtype == DFLASH_BF16 ? run_typed<DFLASH_BF16>(a, st) : run_typed<DFLASH_F32>(a, st);
}

}  // namespace dfk
