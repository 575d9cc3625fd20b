// What the kernels with rotary positions share: 16-byte vectors of a head, the
// turn of a pair, and the frequencies as fractions of a turn.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace tt {

constexpr int kMaxHalf = 128;  // rot <= 256
constexpr int kMaxAxes = 4;

// |f|/2π modulo 1 in units of 2^-64 (rope.cu).
uint64_t turns_of(double f);

// VEC consecutive elements of type T as floats.
template <typename T, int VEC>
struct Vec {
  static __device__ __forceinline__ void load(const T* p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
      f[0] = static_cast<float>(*p);
    } else {
      static_assert(VEC * sizeof(T) == 16, "16-byte vectors");
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = static_cast<float>(e[i]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
      *p = static_cast<T>(f[0]);
    } else {
      uint4 u;
      T* e = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = static_cast<T>(f[i]);
      *reinterpret_cast<uint4*>(p) = u;
    }
  }
};

// One pair turned; the order of the roundings is fixed, so that results do not depend on alignment.
__device__ __forceinline__ void turn_pair(float& x1, float& x2, float c, float s) {
  const float p = x1, q = x2;
  x1 = __fmaf_rn(-q, s, __fmul_rn(p, c));
  x2 = __fmaf_rn(p, s, __fmul_rn(q, c));
}

// Two vectors of a head turned: c, s the cosines and sines of their pairs, pair j of u[j] and v[j], or of neighbours.
template <int VEC>
__device__ __forceinline__ void turn_vectors(float (&u)[VEC], float (&v)[VEC], const float* c, const float* s,
                                             bool adjacent) {
  if (!adjacent) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) turn_pair(u[j], v[j], c[j], s[j]);
  } else if constexpr (VEC == 1) {
    turn_pair(u[0], v[0], c[0], s[0]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      turn_pair(u[2 * j], u[2 * j + 1], c[j], s[j]);
      turn_pair(v[2 * j], v[2 * j + 1], c[VEC / 2 + j], s[VEC / 2 + j]);
    }
  }
}

// Sine and cosine of 2π·(turn·2^-64).
__device__ __forceinline__ void trig_of(uint64_t turn, float& s, float& c) {
  sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
}

}  // namespace tt
