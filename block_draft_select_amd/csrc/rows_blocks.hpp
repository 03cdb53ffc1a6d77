// Device building blocks of the operators on rows of vocabulary logits
// (dflash_sample, dflash_filter, dflash_distill, dflash_distill_grad): 16-byte
// access to rows of any length, stride and alignment, and fp64 weights.
//
// A row starts at any element-aligned address.  Its 16-byte aligned slots
// are numbered from the one holding its first element, so slot s covers
// elements s * VE - phase .. s * VE - phase + VE - 1 (VE elements of 16
// bytes; phase: elements between the slot's start and the row's).  Whole
// slots move as one 16-byte access; the partial first and last ones element
// by element, so nothing outside the row is read or written.
#pragma once

#include "device_util.hpp"
#include "internal.hpp"

namespace dfk {

constexpr float kNegInf = -INFINITY;

template <int DT>
struct RowType;
template <>
struct RowType<DFLASH_BF16> {
  static constexpr int VE = 8;  // elements per 16 bytes
  static constexpr uint32_t kMasked = 0xFF80FF80u;
  static constexpr float kMax = 3.3895313892515355e38f;  // largest finite value
  using elem = uint16_t;
};
template <>
struct RowType<DFLASH_F32> {
  static constexpr int VE = 4;
  static constexpr uint32_t kMasked = 0xFF800000u;
  static constexpr float kMax = 3.4028234663852886e38f;
  using elem = uint32_t;
};

// 16 bytes as four words; element i of a slot (i a compile-time constant
// after unrolling)
struct Slot {
  uint32_t w[4];
};

template <int DT>
__device__ __forceinline__ float slot_value(const Slot& s, int i) {
  if constexpr (DT == DFLASH_BF16)
    return (i & 1) ? bf16_hi(s.w[i >> 1]) : bf16_lo(s.w[i >> 1]);
  else
    return __uint_as_float(s.w[i]);
}

template <int DT>
struct RowRef {
  using E = typename RowType<DT>::elem;
  static constexpr int VE = RowType<DT>::VE;
  const E* p;    // first element
  int phase;     // elements of slot 0 before the row's first
  int V;

  __device__ __forceinline__ RowRef(const void* base, int64_t row, int64_t stride, int V_)
      : p(static_cast<const E*>(base) + row * stride), V(V_) {
    phase = (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(E));
  }
  __device__ __forceinline__ int first(int slot) const { return slot * VE - phase; }  // first element of a slot
  __device__ __forceinline__ bool whole(int slot) const {
    const int e = first(slot);
    return e >= 0 && e + VE <= V;
  }
  // the slot's elements; those outside the row read as masked (-inf)
  template <bool STREAM = false>
  __device__ __forceinline__ Slot load(int slot) const {
    Slot s;
    const int e = first(slot);
    if (e >= 0 && e + VE <= V) {
      uint4 v;
      if constexpr (STREAM)
        v = load_stream16(p + e);
      else
        v = *reinterpret_cast<const uint4*>(p + e);
      s.w[0] = v.x, s.w[1] = v.y, s.w[2] = v.z, s.w[3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) s.w[k] = RowType<DT>::kMasked;
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (e + i >= 0 && e + i < V) {
          if constexpr (DT == DFLASH_BF16) {
            const uint32_t b = p[e + i];
            s.w[i >> 1] = (i & 1) ? ((s.w[i >> 1] & 0x0000FFFFu) | (b << 16)) : ((s.w[i >> 1] & 0xFFFF0000u) | b);
          } else {
            s.w[i] = p[e + i];
          }
        }
    }
    return s;
  }
};

// one element of a row
template <int DT>
__device__ __forceinline__ float row_value(const RowRef<DT>& z, int i) {
  if constexpr (DT == DFLASH_BF16)
    return __uint_as_float((uint32_t)z.p[i] << 16);
  else
    return __uint_as_float(z.p[i]);
}

// ---------------------------------------------------------------- stores

// fp32 -> bf16, nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_round(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return (u >> 16) | 0x0040u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

template <int DT>
__device__ __forceinline__ typename RowType<DT>::elem to_elem(float x) {
  if constexpr (DT == DFLASH_BF16)
    return (uint16_t)bf16_round(x);
  else
    return __float_as_uint(x);
}

// Store a slot that was numbered by `in` to the row `out` of another tensor
// (element for element).  One 16-byte store where the slot is whole and the
// output row has the same alignment, else element by element.
template <int DT>
__device__ __forceinline__ void store_slot(typename RowType<DT>::elem* out, const RowRef<DT>& in, int slot,
                                           const Slot& s, bool same_phase) {
  constexpr int VE = RowType<DT>::VE;
  const int e = in.first(slot);
  if (same_phase && in.whole(slot)) {
    *reinterpret_cast<uint4*>(out + e) = make_uint4(s.w[0], s.w[1], s.w[2], s.w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (e + i >= 0 && e + i < in.V) {
        if constexpr (DT == DFLASH_BF16)
          out[e + i] = (uint16_t)((i & 1) ? s.w[i >> 1] >> 16 : s.w[i >> 1]);
        else
          out[e + i] = s.w[i];
      }
  }
}

}  // namespace dfk
