// Rows of logits in 16-byte vectors, and their sums S = Σ e^(z − m) and
// U = Σ (z − m)·e^(z − m) around a running maximum m. Everything is local to
// the file that includes this.
#pragma once

#include <cuda_fp16.h>

#include "tc_common.cuh"

namespace tt {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
// Offsets from the maximum below this are taken as this: e^-128 is 0 in fp32,
// and 0·d stays 0 for a masked logit (d = -inf).
constexpr float kFloor = -128.f;

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ------------------------------------------------------------------ 16-byte vectors of a row
// A 16-byte vector's elements as floats: pair i, element i, the largest one,
// and raise(): every element at least the type's lowest finite value (a NaN
// stays).
template <typename T>
struct Pairs;
template <>
struct Pairs<float> {
  static constexpr int N = 2;
  static __device__ __forceinline__ float2 get(const uint4& u, int i) {
    return i ? make_float2(__uint_as_float(u.z), __uint_as_float(u.w))
             : make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
  static __device__ __forceinline__ float element(const uint4& u, int i) {
    return __uint_as_float(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w);
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    return fmaxf(tc::fmax3f(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z)), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ float max(const uint4& a, const uint4& b, const uint4& c, const uint4& d) {
    return fmaxf(tc::fmax3f(max(a), max(b), max(c)), max(d));
  }
};
// The two 16-bit types: W = the packed pair.
template <typename W>
struct PackedPairs {
  static constexpr int N = 4;
  static __device__ __forceinline__ uint32_t word(const uint4& u, int i) {
    return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
  }
  static __device__ __forceinline__ W packed(uint32_t w) { return *reinterpret_cast<const W*>(&w); }
  static __device__ __forceinline__ W max2(const uint4& u) {
    return __hmax2(__hmax2(packed(u.x), packed(u.y)), __hmax2(packed(u.z), packed(u.w)));
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    const W m = max2(u);
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ float max(const uint4& a, const uint4& b, const uint4& c, const uint4& d) {
    const W m = __hmax2(__hmax2(max2(a), max2(b)), __hmax2(max2(c), max2(d)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ uint32_t raise(uint32_t w, uint32_t low2) {
    const W m = __hmax2_nan(packed(w), packed(low2));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
};
template <>
struct Pairs<__nv_bfloat16> : PackedPairs<__nv_bfloat162> {
  static constexpr uint32_t kLow2 = 0xff7fff7fu;      // the lowest finite value, twice
  static constexpr float kPlainLow = -1e38f, kPlainHigh = 1e36f;
  static __device__ __forceinline__ float2 floats(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ float2 get(const uint4& u, int i) { return floats(word(u, i)); }
  static __device__ __forceinline__ float element(const uint4& u, int i) {
    const float2 p = get(u, i >> 1);
    return i & 1 ? p.y : p.x;
  }
};
template <>
struct Pairs<__half> : PackedPairs<__half2> {
  static constexpr uint32_t kLow2 = 0xfbfffbffu;
  static constexpr float kPlainLow = -65000.f, kPlainHigh = INFINITY;
  static __device__ __forceinline__ float2 floats(uint32_t w) { return __half22float2(packed(w)); }
  static __device__ __forceinline__ float2 get(const uint4& u, int i) { return floats(word(u, i)); }
  static __device__ __forceinline__ float element(const uint4& u, int i) {
    const float2 p = get(u, i >> 1);
    return i & 1 ? p.y : p.x;
  }
};

template <typename T>
struct Row {
  static constexpr int VN = 16 / sizeof(T);
  const T* p;    // element 0
  int shift;     // elements between the 16-byte boundary at or below p and p
  int V;
  int nvec;
  __device__ __forceinline__ Row(const T* row, int64_t V_) : p(row), V((int)V_) {
    shift = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    nvec = (V + shift + VN - 1) / VN;
  }
  // first element of vector j (negative for the first vector of an unaligned row)
  __device__ __forceinline__ int first(int j) const { return j * VN - shift; }
  __device__ __forceinline__ bool whole(int j) const { return first(j) >= 0 && first(j) + VN <= V; }
  // the vectors whole_lo() .. whole_hi() - 1 lie inside the row
  __device__ __forceinline__ int whole_lo() const { return shift ? 1 : 0; }
  __device__ __forceinline__ int whole_hi() const { return (V + shift) / VN; }
  __device__ __forceinline__ uint4 load_whole(int j) const { return *reinterpret_cast<const uint4*>(p + first(j)); }
  // vector j; places outside the row read -inf
  __device__ __forceinline__ uint4 load(int j) const {
    if (whole(j)) return load_whole(j);
    const int e = first(j);
    uint4 u;
    T* t = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < VN; ++i) t[i] = (e + i >= 0 && e + i < V) ? p[e + i] : static_cast<T>(-INFINITY);
    return u;
  }
};

// ------------------------------------------------------------------ (m, s, u)
struct Stat {
  float m, s, u;  // maximum, Σ e^(z − m), Σ (z − m)·e^(z − m)
};
__device__ __forceinline__ void rescale(Stat& a, float M) {
  const float d = a.m == M ? 0.f : max_nan(a.m - M, kFloor);  // (two maxima of -inf are one)
  const float f = fast_exp2(d * kLog2e);
  a.u = fmaf(d, a.s, a.u) * f;
  a.s *= f;
  a.m = M;
}
__device__ __forceinline__ void merge(Stat& a, Stat b) {
  const float M = fmaxf(a.m, b.m);
  rescale(a, M);
  rescale(b, M);
  a.s += b.s;
  a.u += b.u;
}

// Masked logits (-inf) must add 0 to Σ d·e^d, not 0·(-inf). The plain way of a 16-bit type raises them to the type's
// lowest finite value first, two elements in one instruction: d stays finite and e^d is 0, unless the row's maximum is
// itself near the lowest value (then the two must be told apart) or so high that d overflows. Such rows, known by their
// maximum at the end, are taken again the wide way, which bounds every d (as fp32 rows always are: two instructions for
// two elements, and half as many elements to the byte).
template <typename T>
__device__ __forceinline__ bool plain_way_holds(float m) {
  if constexpr (sizeof(T) == 4) return true;
  else return (m > Pairs<T>::kPlainLow && m < Pairs<T>::kPlainHigh) || m == -INFINITY;
}
// (A maximum of -inf: nothing but masked logits, or NaN; raised logits would give S > 0.)

// Adds one vector to the sums s, q = Σ e^d, Σ d·e^d around nm = −(reference), l2 = log2 e.
template <typename T, bool WIDE>
__device__ __forceinline__ void fold(float2& s, float2& q, const uint4& u, float2 nm, float2 l2) {
#pragma unroll
  for (int i = 0; i < Pairs<T>::N; ++i) {
    float2 x;
    if constexpr (WIDE || sizeof(T) == 4)
      x = Pairs<T>::get(u, i);
    else
      x = Pairs<T>::floats(Pairs<T>::raise(Pairs<T>::word(u, i), Pairs<T>::kLow2));
    float2 d = __fadd2_rn(x, nm);
    if constexpr (WIDE || sizeof(T) == 4) d = make_float2(max_nan(d.x, kFloor), max_nan(d.y, kFloor));
    const float2 t = __fmul2_rn(d, l2);
    const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
    s = __fadd2_rn(s, e);
    q = __ffma2_rn(e, d, q);
  }
}

// The warp's sums in every lane. Both lanes of a pair join in the same order, so that they agree bitwise.
__device__ __forceinline__ Stat join_warp(Stat t, int lane) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(kAll, t.m, o);
    b.s = __shfl_xor_sync(kAll, t.s, o);
    b.u = __shfl_xor_sync(kAll, t.u, o);
    Stat first = (lane & o) ? b : t, second = (lane & o) ? t : b;
    merge(first, second);
    t = first;
  }
  return t;
}

}  // namespace
}  // namespace tt
