// dflash_linear_i8: y_rn = xs_r ws_n sum_k xq_rk wq_nk, rows of 8-bit integers
// with a scale each; the sums are exact in 32 bits.
//
// On the matrix cores (v_mfma_i32_16x16x64_i8): the weights are the A operand,
// the tokens the B operand, so a lane of the result holds four neighbouring
// channels of one token.  Lane l of either operand holds the 16 bytes
// 16 (l / 16) .. of row l % 16 and of 64 bytes of k.  Only the tokens' side is
// cleared past the row's end: what the weights hold there is multiplied by zero.
#include "rows_blocks.hpp"

namespace dfk {

namespace {

typedef int v4i32 __attribute__((ext_vector_type(4)));

// Few tokens: 16 channels and 16 MT tokens a block, its four waves split k.
// Each wave has eight steps of 64 bytes in flight.
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

// Workgroup barrier for LDS hand-offs only: __syncthreads() would also wait for
// every global load in flight
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // vmcnt 63 (no wait), expcnt 7, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// An array of 8-bit rows from `row` on as a buffer: loads behind its end give 0,
// so neither rows nor pieces of k need a clamp (`last`: rows from there on; strides stay
// below 2^24, and a block uses 256 rows at most)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const int8_t* p, int64_t row, int64_t rows, int64_t stride, int H) {
  const int64_t last = min(rows - 1 - row, (int64_t)511);
  const int64_t bytes = min(last * stride, (int64_t)0x7FFF0000) + (H + 15) / 16 * 16;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p) + row * stride, 0, (int)bytes, 0x00027000);
}

// 16 bytes a lane from a buffer straight into LDS, at 16 l past the wave's address
__device__ __forceinline__ void load_to_lds16(__amdgpu_buffer_rsrc_t b, int lane_offset, int offset, unsigned char* l) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, l, 16, lane_offset, offset, 0, 0);
#endif
}

__device__ __forceinline__ v4i32 load16(__amdgpu_buffer_rsrc_t b, int lane_offset, int offset) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_bit_cast(v4i32, __builtin_amdgcn_raw_buffer_load_b128(b, lane_offset, offset, 0));
#else
  return v4i32{};
#endif
}

// Many tokens: a block of four waves owns 256 channels and 16 TT tokens, each wave
// 64 channels of all its tokens.  The weights go from global memory straight
// into the wave's registers (no other wave of the block needs them), two
// stages of 128 bytes of k ahead; the tokens' rows go straight into a ring of
// three LDS stages that the waves share.  So LDS moves one KB a wave for every four matrix
// instructions, half of what it can.
// A stage in LDS: 128-byte rows, the 16-byte piece c of row r at place c ^ (r % 8), so that
// the eight rows that are read at once lie in different banks.
// The rows of the A operand are dealt out so that a lane ends up with 16
// neighbouring channels: row i of tile c is channel 16 (i / 4) + 4 c + i % 4.
constexpr int kTileCh = 256;

template <int DT, int TT>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(LinearArgs a, int n_rt, int n_ct) {
  constexpr int BM = 16 * TT, NB = 3;
  constexpr int XL = TT / 2;           // loads of a stage's token rows a wave: 8 rows each
  constexpr int PER_STAGE = XL + 8;    // and of weights
  __shared__ __attribute__((aligned(1024))) unsigned char lds[NB * BM * 128];
  // ids with the same value mod 8 run on one XCD: the row tiles of a channel tile follow one another there
  const int grp = blockIdx.x / (8 * n_rt), rem = blockIdx.x - grp * 8 * n_rt;
  const int rt = rem >> 3, ct = grp * 8 + (rem & 7);
  if (ct >= n_ct) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  // the last waves step back to whole tiles: some channels are computed twice, alike (N >= 64)
  const int ch0 = min(ct * kTileCh + wave * 64, a.N - 64);
  const int64_t row0 = (int64_t)rt * BM;
  const int n_st = (a.H + 127) / 128;

  const int i16 = lane & 15, g4 = lane >> 4;
  const int w_stride = (int)a.wq_stride, x_stride = (int)a.xq_stride;
  const __amdgpu_buffer_rsrc_t wb = rows_buffer(a.wq, ch0, a.N, a.wq_stride, a.H);
  const __amdgpu_buffer_rsrc_t xb = rows_buffer(a.xq, row0, a.R, a.xq_stride, a.H);
  const int wo = ((i16 >> 2) * 16 + (i16 & 3)) * w_stride + g4 * 16;
  const int xo = (lane >> 3) * x_stride + ((lane & 7) ^ (lane >> 3)) * 16;  // place l % 8 of a row holds this piece
  auto load_x = [&](int s) {
    unsigned char* to = lds + (s % NB) * (BM * 128) + wave * XL * 1024;
#pragma unroll
    for (int i = 0; i < XL; ++i) load_to_lds16(xb, xo, 8 * (wave * XL + i) * x_stride + s * 128, to + i * 1024);
  };
  v4i32 wv[2][2][4];  // [stage parity][64-byte step][tile]
  auto load_w = [&](int s, int ks, v4i32(&to)[4]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) to[t] = load16(wb, wo, 4 * t * w_stride + s * 128 + ks * 64);
  };

  v4i32 acc[TT][4];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[t][c] = (v4i32){0, 0, 0, 0};
  int fo[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) fo[ks] = i16 * 128 + ((4 * ks + g4) ^ (lane & 7)) * 16;

  auto stage = [&](int s, v4i32(&ws)[2][4]) {
    // this wave's loads of stage s are done when only those of s + 1 remain
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (PER_STAGE & 15) | ((PER_STAGE >> 4) << 14));  // vmcnt(PER_STAGE) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    unsigned char* st = lds + (s % NB) * (BM * 128);
    if (s * 128 + 128 > a.H) {  // the rows end in this stage, or before it: clear the tokens' bytes behind the end
      const int valid = a.H - s * 128;
#pragma unroll 1
      for (int q = tid; q < BM * 32; q += 256) {  // words
        const int n = valid - (((q >> 2) & 7) ^ ((q >> 5) & 7)) * 16 - (q & 3) * 4;
        uint32_t* p = reinterpret_cast<uint32_t*>(st) + q;
        if (n < 4) *p = n <= 0 ? 0u : *p & ((1u << (8 * n)) - 1u);
      }
      lds_barrier();
    }
    load_x(s + 2);  // into the buffer that stage s - 1 used
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const v4i32 xv = *reinterpret_cast<const v4i32*>(st + t * 2048 + fo[ks]);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[t][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(ws[ks][c], xv, acc[t][c], 0, 0, 0);
      }
      // left to itself the scheduler loads the next weights before these are used, into registers that it then spills
      __builtin_amdgcn_sched_barrier(0);
      load_w(s + 2, ks, ws[ks]);
    }
  };

  // in the order that the waits count
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    load_x(s);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) load_w(s, ks, wv[s][ks]);
    __builtin_amdgcn_sched_barrier(0);
  }
  // an odd last stage takes one behind the end with it, whose tokens are cleared
  for (int s = 0; s < n_st; s += 2) {
    stage(s, wv[0]);
    stage(s + 1, wv[1]);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no transfer outlives the loop

  using E = typename RowType<DT>::elem;
  const int ch = ch0 + g4 * 16;
  float sc[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) sc[j] = a.ws[ch + j];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t row = row0 + t * 16 + i16;
    if (row >= a.R) continue;
    const float xs = a.xs[row];
    E* y = static_cast<E*>(a.y) + row * a.y_stride + ch;
    E v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = to_elem<DT>((float)acc[t][j >> 2][j & 3] * xs * sc[j]);
    constexpr int VE = RowType<DT>::VE;
#pragma unroll
    for (int q = 0; q < 16 / VE; ++q) {
      u32x4_any o;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if constexpr (DT == DFLASH_BF16)
          o[d] = (uint32_t)v[q * 8 + 2 * d] | (uint32_t)v[q * 8 + 2 * d + 1] << 16;
        else
          o[d] = v[q * 4 + d];
      }
      *reinterpret_cast<u32x4_any*>(y + q * VE) = o;
    }
  }
}

template <int DT, int TT>
hipError_t run_tile(const LinearArgs& a, hipStream_t st) {
  const int n_ct = (a.N + kTileCh - 1) / kTileCh;
  const int n_rt = (int)((a.R + 16 * TT - 1) / (16 * TT));
  launch(linear_tile_kernel<DT, TT>, dim3((unsigned)((int64_t)((n_ct + 7) / 8) * 8 * n_rt)), dim3(256), st, a, n_rt, n_ct);
  return hipGetLastError();
}

struct LinearPlan {
  int few;   // 16-token tiles of the few-tokens kernel, or 0
  int tile;  // of the tile kernel
  int64_t blocks;
};

LinearPlan linear_plan(int64_t R, int32_t N) {
  LinearPlan p{};
  if (R <= 32 || N < 64) {
    p.few = R <= 16 ? 1 : 2;
    p.blocks = (int64_t)((N + 15) / 16) * ((R + 16 * p.few - 1) / (16 * p.few));
  } else {
    p.tile = R <= 64 ? 4 : 8;
    p.blocks = (int64_t)((N + kTileCh * 8 - 1) / (kTileCh * 8)) * 8 * ((R + 16 * p.tile - 1) / (16 * p.tile));
  }
  return p;
}

template <int DT>
hipError_t run_typed(const LinearArgs& a, hipStream_t st) {
  const LinearPlan p = linear_plan(a.R, a.N);
  if (p.few == 1) return run_few<DT, 1>(a, st);
  if (p.few == 2) return run_few<DT, 2>(a, st);
  return p.tile == 4 ? run_tile<DT, 4>(a, st) : run_tile<DT, 8>(a, st);
}

}  // namespace

int64_t linear_blocks(int64_t R, int32_t N, int32_t) { return linear_plan(R, N).blocks; }

hipError_t launch_linear_i8(int32_t dtype, const LinearArgs& a, hipStream_t st) {
  return dtype == DFLASH_BF16 ? run_typed<DFLASH_BF16>(a, st) : run_typed<DFLASH_F32>(a, st);
}

}  // namespace dfk
