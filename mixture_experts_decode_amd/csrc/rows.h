// Row helpers of the operators around the layer: rounding and 8-element
// loads and stores of BF16 / FP32 rows, and reductions over lane groups.
#pragma once

#include "device.h"

namespace moe {
namespace {

// Two floats -> two BF16, each rounded once to the nearest (ties to even), a
// NaN kept a NaN (element 0 in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  bf16x2 v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}

// Eight consecutive row elements as stored.
template <bool F32> struct Raw8;
template <> struct Raw8<false> {
  u32x4 a;
  __device__ __forceinline__ float get(int i) const {
    return (i & 1) ? bf16_hi(a[i >> 1]) : bf16_lo(a[i >> 1]);
  }
};
template <> struct Raw8<true> {
  u32x4 a[2];
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(a[i >> 2][i & 3]); }
};

// One element of a row at element index i.
template <bool F32>
__device__ __forceinline__ void store1(void* p, size_t i, float v) {
  if constexpr (F32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<__bf16*>(p)[i] = (__bf16)v;
}

// Stores eight values from element index i on (16-byte aligned).  PAST: with a
// streaming policy, so that rows written do not drive out what is read again.
template <bool F32, bool PAST = false>
__device__ __forceinline__ void store8(void* p, size_t i, const float (&v)[8]) {
  auto put = [&](u32x4* q, u32x4 w) {
    if constexpr (PAST) __builtin_nontemporal_store(w, q);
    else *q = w;
  };
  if constexpr (F32) {
    u32x4* q = reinterpret_cast<u32x4*>(reinterpret_cast<float*>(p) + i);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      put(q + h, u32x4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                       __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])});
  } else {
    put(reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + i),
        u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
              pack_bf16(v[6], v[7])});
  }
}

// Orders a wavefront's LDS accesses: its lanes exchange values through LDS
// without a barrier.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sum and maximum over each aligned group of N lanes (16, 32 or 64); every
// lane of the group gets it.
template <int N>
__device__ __forceinline__ float group_sum(float x) {
  x = row16_sum(x);
  if constexpr (N >= 32) {
    const uint32_t u = __float_as_uint(x);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (N == 64) {
    const uint32_t u = __float_as_uint(x);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

template <int N>
__device__ __forceinline__ float group_max(float x) {
  x = fmaxf(x, dpp_f32<0x128>(x));
  x = fmaxf(x, dpp_f32<0x124>(x));
  x = fmaxf(x, dpp_f32<0x122>(x));
  x = fmaxf(x, dpp_f32<0x121>(x));
  if constexpr (N >= 32) {
    const uint32_t u = __float_as_uint(x);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (N == 64) {
    const uint32_t u = __float_as_uint(x);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return x;
}

}  // namespace
}  // namespace moe
