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

int few_tiles(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : 4; }

template <int DT>
hipError_t run_typed(const LinearArgs& a, hipStream_t st) {
  switch (few_tiles(a.R)) {
    case 1: return run_few<DT, 1>(a, st);
    case 2: return run_few<DT, 2>(a, st);
    default: return run_few<DT, 4>(a, st);
  }
}

}  // namespace

int64_t linear_blocks(int64_t R, int32_t N, int32_t) {
  const int mt = few_tiles(R);
  return (int64_t)((N + 15) / 16) * ((R + 16 * mt - 1) / (16 * mt));
}

hipError_t launch_linear_i8(int32_t dtype, const LinearArgs& a, hipStream_t st) {
  return dtype == DFLASH_BF16 ? run_typed<DFLASH_BF16>(a, st) : run_typed<DFLASH_F32>(a, st);
}

}  // namespace dfk
