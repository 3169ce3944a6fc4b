// Rounding and storing eight elements of a row.
#pragma once
#include <cuda_fp16.h>

#include <type_traits>

#include "kv_device.cuh"
#include "w8_device.cuh"

namespace spear {

template <class T>
SPEAR_DEVINL T rounded(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// 32 bytes: a whole sector by one lane (16 a lane, 32 apart, reach L2 as half sectors). p is 32-byte aligned.
SPEAR_DEVINL void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <class T>
SPEAR_DEVINL void store8(T* p, int n, bool vec, const float (&x)[8]) {
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = rounded<T>(x[i]);
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      uint4 w;
      memcpy(&w, reinterpret_cast<const char*>(e) + 16 * i, 16);
      *(reinterpret_cast<uint4*>(p) + i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = e[i];
  }
}

}  // namespace spear
