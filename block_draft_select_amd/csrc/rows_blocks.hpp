// Device building blocks of the operators on rows of vocabulary logits
// (dflash_sample, dflash_filter, dflash_distill, dflash_logprobs, their gradients
// and dflash_quant_i8): 16-byte access to rows of any length, stride and alignment.
//
// A row is cut into slots of 16 bytes from its first element on (VE elements
// each), wherever that element lies: global memory instructions take any
// alignment here, and a wave's 1 KB touches at most one cache line more.  Only
// the last slot of a row can be short; it is read through the 16 bytes that
// end with the row, so nothing outside the row is read or written.
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

// 16 bytes at an address aligned to two bytes only
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <int DT>
struct RowRef {
  using E = typename RowType<DT>::elem;
  static constexpr int VE = RowType<DT>::VE;
  const E* p;
  int V;

  __device__ __forceinline__ RowRef(const void* base, int64_t row, int64_t stride, int V_)
      : p(static_cast<const E*>(base) + row * stride), V(V_) {}
  __device__ __forceinline__ int slots() const { return (V + VE - 1) / VE; }

  // the slot's elements; those past the row's end read as masked (-inf)
  template <bool STREAM = false>
  __device__ __forceinline__ Slot load(int slot) const {
    const int e = slot * VE;
    Slot s;
    if (e + VE <= V) {
      const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p + e);
      u32x4_any v;
      if constexpr (STREAM)
        v = __builtin_nontemporal_load(q);
      else
        v = *q;
      s.w[0] = v.x, s.w[1] = v.y, s.w[2] = v.z, s.w[3] = v.w;
      return s;
    }
    constexpr uint64_t kFill = (uint64_t)RowType<DT>::kMasked << 32 | RowType<DT>::kMasked;
    uint64_t lo = kFill, hi = kFill;
    if (e < V) {
      const int bits = (V - e) * (int)sizeof(E) * 8;  // valid bits, below 128
      uint64_t a = 0, b = 0;
      if (V >= VE) {
        const u32x4_any v = *reinterpret_cast<const u32x4_any*>(p + V - VE);
        a = (uint64_t)v.y << 32 | v.x;
        b = (uint64_t)v.w << 32 | v.z;
        const int sh = 128 - bits;  // move the row's last elements to the slot's start
        if (sh < 64) {
          a = a >> sh | b << (64 - sh);
          b >>= sh;
        } else {
          a = b >> (sh - 64);
          b = 0;
        }
      } else {  // the whole row is shorter than a slot
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
          const int at = i * (int)sizeof(E) * 8;
          if (at < 64) a |= (uint64_t)p[i] << at; else b |= (uint64_t)p[i] << (at - 64);
        }
      }
      lo = bits < 64 ? a | kFill << bits : a;
      hi = bits <= 64 ? kFill : b | kFill << (bits - 64);
    }
    s.w[0] = (uint32_t)lo, s.w[1] = (uint32_t)(lo >> 32), s.w[2] = (uint32_t)hi, s.w[3] = (uint32_t)(hi >> 32);
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

// a slot to a row of V elements
template <int DT>
__device__ __forceinline__ void store_slot(typename RowType<DT>::elem* out, int V, int slot, const Slot& s) {
  using E = typename RowType<DT>::elem;
  constexpr int VE = RowType<DT>::VE;
  const int e = slot * VE;
  if (e + VE <= V) {
    u32x4_any v;
    v.x = s.w[0], v.y = s.w[1], v.z = s.w[2], v.w = s.w[3];
    *reinterpret_cast<u32x4_any*>(out + e) = v;
  } else if (e < V) {
    uint64_t a = (uint64_t)s.w[1] << 32 | s.w[0], b = (uint64_t)s.w[3] << 32 | s.w[2];
#pragma unroll 1
    for (int i = e; i < V; ++i) {
      out[i] = (E)a;
      a = a >> (sizeof(E) * 8) | b << (64 - sizeof(E) * 8);
      b >>= sizeof(E) * 8;
    }
  }
}

}  // namespace dfk
