// dflash_quant_i8: rows in 8 bits with one scale each, s = max |x| / 127 and
// q = x / s to the nearest integer (ties to even).
//
// A row stays in the registers of the threads that load it, so it is read once;
// longer ones are read twice.  q is the exact quotient's nearest integer: with
// n = rint(x (1 / s)), the remainder x - n s (one fma, exact but for its last
// bit) says whether x / s lies so near to the middle of two integers that the
// product's rounding (127 x 2^-22) could decide; those slots divide in fp64.
// Bound by memory: 151936 x 2048 bf16 in 164 us, 5.7 TB/s read and written.  A wave a row
// of up to eight slots a lane needs no barrier; a block a longer one.
#include "rows_blocks.hpp"

namespace dfk {

namespace {

// the largest magnitude of a slot as the ordered bits of |x| (of fp32): NaN and inf stand above the rest
template <int DT>
__device__ __forceinline__ uint32_t magnitude(const Slot& x, uint32_t most) {
  if constexpr (DT == DFLASH_BF16) {
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max_u16x2(m, x.w[d] & 0x7FFF7FFFu);
    return max(most, max(m << 16, m & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d) most = max(most, x.w[d] & 0x7FFFFFFFu);
    return most;
  }
}

struct Scale {
  float s, inv, up;  // up: what the row is multiplied by first, so that x and s are normal numbers
};

__device__ __forceinline__ Scale row_scale_of(uint32_t most, float& out) {
  Scale k{0.0f, 0.0f, 1.0f};
  const float a = __uint_as_float(most);
  if (!(a < INFINITY)) {
    out = NAN;  // no scale holds such a row: q is 0
    return k;
  }
  out = (float)((double)a / 127.0);
  if (a < 0x1p-60f) k.up = 0x1p64f;
  k.s = out * k.up;
  k.inv = k.s > 0.0f ? 1.0f / k.s : 0.0f;
  return k;
}

// a slot's bytes, VE of them
template <int DT>
__device__ __forceinline__ uint2 quant_slot(const Slot& x, const Scale& k) {
  constexpr int VE = RowType<DT>::VE;
  float n[VE], far = 0.0f;
#pragma unroll
  for (int i = 0; i < VE; ++i) {
    const float v = slot_value<DT>(x, i) * k.up;
    n[i] = rintf(v * k.inv);
    far = fmaxf(far, fabsf(fmaf(-n[i], k.s, v)));
  }
  if (far > 0.49995f * k.s) {
#pragma unroll
    for (int i = 0; i < VE; ++i) n[i] = k.s > 0.0f ? (float)rint((double)(slot_value<DT>(x, i) * k.up) / (double)k.s) : 0.0f;
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < VE; ++i) w[i >> 2] |= ((uint32_t)(int)fminf(fmaxf(n[i], -127.0f), 127.0f) & 255u) << ((i & 3) * 8);
  return make_uint2(w[0], w[1]);
}

template <int DT>
__device__ __forceinline__ void store_bytes(int8_t* q, int V, int slot, uint2 b) {
  constexpr int VE = RowType<DT>::VE;
  const int e = slot * VE;
  if (e + VE <= V) {
    if constexpr (VE == 8)
      *reinterpret_cast<uint2*>(q + e) = b;
    else
      *reinterpret_cast<uint32_t*>(q + e) = b.x;
  } else {
#pragma unroll 1
    for (int i = e; i < V; ++i) {
      q[i] = (int8_t)b.x;
      b.x = b.x >> 8 | b.y << 24;
      b.y >>= 8;
    }
  }
}

// a slot of the row, 0 past its end
template <int DT>
__device__ __forceinline__ Slot load_or_zero(const RowRef<DT>& z, int slot) {
  constexpr int VE = RowType<DT>::VE;
  Slot s = z.load(slot);
  if ((slot + 1) * VE > z.V) {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (slot * VE + i >= z.V) {
        if constexpr (DT == DFLASH_BF16)
          s.w[i >> 1] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;
        else
          s.w[i] = 0;
      }
  }
  return s;
}

template <int T>
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v) {
  v = wave_max_u32(v);
  if constexpr (T > kWave) {
    __shared__ uint32_t w[T / kWave];
    if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / kWave; ++i) v = max(v, w[i]);
  }
  return v;
}

// T threads a row, NL slots a thread (0: any number, the row is read twice)
template <int DT, int T, int NL>
__global__ __launch_bounds__(256) void quant_kernel(const void* X, int64_t R, int64_t stride, int H, int8_t* __restrict__ q,
                                                    int64_t q_stride, float* __restrict__ scale) {
  constexpr int kRows = 256 / T;  // rows of a block
  const int tid = threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / T;
  if (row >= R) return;  // whole waves; one row a block where there are barriers
  const RowRef<DT> z(X, row, stride, H);
  int8_t* o = q + row * q_stride;
  uint32_t most = 0;
  Slot x[NL > 0 ? NL : 1];
  if constexpr (NL > 0) {
#pragma unroll
    for (int l = 0; l < NL; ++l) x[l] = load_or_zero<DT>(z, l * T + tid);
#pragma unroll
    for (int l = 0; l < NL; ++l) most = magnitude<DT>(x[l], most);
  } else {
    for (int s = tid; s < z.slots(); s += T) most = magnitude<DT>(load_or_zero<DT>(z, s), most);
  }
  most = block_max_u32<T>(most);
  float out;
  const Scale k = row_scale_of(most, out);
  if (tid == 0) scale[row] = out;
  if constexpr (NL > 0) {
#pragma unroll
    for (int l = 0; l < NL; ++l) store_bytes<DT>(o, H, l * T + tid, out == out ? quant_slot<DT>(x[l], k) : make_uint2(0, 0));
  } else {
    for (int s = tid; s < z.slots(); s += T)
      store_bytes<DT>(o, H, s, out == out ? quant_slot<DT>(load_or_zero<DT>(z, s), k) : make_uint2(0, 0));
  }
}

template <int DT, int T, int NL>
hipError_t run(const QuantArgs& a, hipStream_t st) {
  const int64_t rows = 256 / T;
  launch(quant_kernel<DT, T, NL>, dim3((unsigned)((a.R + rows - 1) / rows)), dim3(256), st, a.X, a.R, a.stride, a.H, a.q,
         a.q_stride, a.scale);
  return hipGetLastError();
}

template <int DT>
hipError_t run_typed(const QuantArgs& a, hipStream_t st) {
  const int slots = (a.H + RowType<DT>::VE - 1) / RowType<DT>::VE;
  if (slots <= kWave) return run<DT, kWave, 1>(a, st);
  if (slots <= 2 * kWave) return run<DT, kWave, 2>(a, st);
  if (slots <= 4 * kWave) return run<DT, kWave, 4>(a, st);
  if (slots <= 8 * kWave) return run<DT, kWave, 8>(a, st);
  if (slots <= 4 * 256) return run<DT, 256, 4>(a, st);
  if (slots <= 8 * 256) return run<DT, 256, 8>(a, st);
  return run<DT, 256, 0>(a, st);
}

}  // namespace

hipError_t launch_quant_i8(int32_t dtype, const QuantArgs& a, hipStream_t st) {
  return dtype == DFLASH_BF16 ? run_typed<DFLASH_BF16>(a, st) : run_typed<DFLASH_F32>(a, st);
}

}  // namespace dfk
