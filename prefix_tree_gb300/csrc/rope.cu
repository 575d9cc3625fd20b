// Rotary positions of Q and K with one or several position axes, and their
// inverse (the rotation is orthogonal, so the inverse is also the backward
// pass).
//
//   θ_i = pos[a(i)][t]·f_i,   (x1, x2) -> (x1·cos θ_i − x2·sin θ_i, x2·cos θ_i + x1·sin θ_i),  i < rot/2
//
// over the pairs (i, i + rot/2) or (2i, 2i + 1) of every head; dimensions >=
// rot pass through.
//
// Angles. f_i/2π modulo 1 is held as a 64-bit binary fraction of a turn, so
// pos·f_i modulo one turn is one wrapping 64-bit product: no large argument
// is ever rounded to fp32 (at position 10^6 an fp32 angle is off by up to
// 0.03 rad), and no fp64 instruction is needed. The fraction comes from the
// digits of 1/2π (turns_of), so that it holds for every frequency: an fp64
// division would leave 2^-53 of the frequency's turns, which the position
// multiplies. The top 32 bits, as a signed fraction of half a turn, go to
// sincospif.
//
// Bound by memory: each of q and k once in, once out. A block forms the sines
// and cosines of its tokens once, in shared memory, for all their heads; a
// thread then takes 2 x 16 bytes of a head in and out. 65,536 tokens of 40 + 8
// heads of 128 bf16 (1.61 GB): 242 us, 0.99 of the measured copy rate; 12,669
// of 32 + 8 fp32, half of each head turned: 81 us, 0.96. Dropped: the next
// item loaded while one is turned (274 and 85 us: the registers cost more
// warps than it hides), two and three items of a thread at once (345, 440).
#include "common.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

namespace tt {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxHalf = 128;  // rot <= 256
constexpr int kMaxAxes = 4;
constexpr int kMaxTokens = 32;  // tokens of a block

struct RopeArgs {
  const void* x[2];  // q, k
  void* y[2];
  int64_t ld[2], ldo[2];
  int heads[2];
  int64_t N;
  int d, half, npv, nrot;  // npv: vector pairs of a head, the first nrot of them rotated
  int tokens;              // of a block
  const int32_t* pos;
  int64_t pos_ld;
  int adjacent, inverse;
  uint64_t turn[kMaxHalf];  // f_i/2π mod 1, in units of 2^-64
  uint8_t axis[kMaxHalf];
};

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

template <typename T, int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float trig[];
  float* cosines = trig;
  float* sines = trig + a.tokens * a.half;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int nt = (int)min((int64_t)a.tokens, a.N - t0);
  for (int i = threadIdx.x; i < nt * a.half; i += kRopeThreads) {
    const int t = i / a.half, f = i - t * a.half;
    const int64_t pos = a.pos[a.axis[f] * a.pos_ld + t0 + t];
    const uint64_t turn = (uint64_t)pos * a.turn[f];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    cosines[i] = c;
    sines[i] = a.inverse ? -s : s;
  }
  __syncthreads();
  const int H = a.heads[0] + a.heads[1];
  for (int i = threadIdx.x; i < nt * H * a.npv; i += kRopeThreads) {
    const int r = i / a.npv, pv = i - r * a.npv;
    const int t = r / H, hh = r - t * H;
    const int w = hh >= a.heads[0];
    const int64_t head = (int64_t)(hh - (w ? a.heads[0] : 0)) * a.d;
    const T* x = static_cast<const T*>(a.x[w]) + (t0 + t) * a.ld[w] + head;
    T* y = static_cast<T*>(a.y[w]) + (t0 + t) * a.ldo[w] + head;
    // the two vectors of this item: half a rotation apart, or next to each other
    const bool rotated = pv < a.nrot;
    const int o1 = a.adjacent || !rotated ? (rotated ? 2 * VEC * pv : 2 * a.half + 2 * VEC * (pv - a.nrot)) : VEC * pv;
    const int o2 = a.adjacent || !rotated ? o1 + VEC : o1 + a.half;
    if (!rotated && x == y) continue;
    float u[VEC], v[VEC];
    Vec<T, VEC>::load(x + o1, u);
    Vec<T, VEC>::load(x + o2, v);
    if (rotated) {
      const float* c = cosines + t * a.half + VEC * pv;
      const float* s = sines + t * a.half + VEC * pv;
      if (!a.adjacent) {
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
    Vec<T, VEC>::store(y + o1, u);
    Vec<T, VEC>::store(y + o2, v);
  }
}

// |f|/2π modulo 1 in units of 2^-64, negated for f < 0, cut off below 2^-64 (then at position 2^31 the angle is off by
// 2^-33 of a turn). As Payne and Hanek reduce large arguments: f = mant·2^s with a whole mant of 53 bits, and of the
// product with 1/2π only the digits that matter are formed: 2^s/2π modulo 1 to 128 binary places, which are 128
// consecutive digits of 1/2π, times mant modulo 2^128.
uint64_t turns_of(double f) {
  // the first 1152 binary digits of 1/2π: a double's exponent leaves out up to 971 of them
  static const uint64_t digits[18] = {
      0x28be60db9391054a, 0x7f09d5f47d4d3770, 0x36d8a5664f10e410, 0x7f9458eaf7aef158, 0x6dc91b8e909374b8,
      0x01924bba82746487, 0x3f877ac72c4a69cf, 0xba208d7d4baed121, 0x3a671c09ad17df90, 0x4e64758e60d4ce7d,
      0x272117e2ef7e4a0e, 0xc7fe25fff7816603, 0xfbcbc462d6829b47, 0xdb4d9fb3c9f2c26d, 0xd3d18fd9a797fa8b,
      0x5d49eeb1faf97c5e, 0xcf41ce7de294a4ba, 0x9afed7ec47e35742};
  typedef unsigned __int128 u128;
  // mant and s from f's bits (frexp and ldexp took 0.7 us for the 64 frequencies of a call)
  uint64_t bits;
  std::memcpy(&bits, &f, 8);
  const int e = (int)(bits >> 52 & 0x7ff);
  const uint64_t mant = (bits & ((uint64_t(1) << 52) - 1)) | (uint64_t)(e != 0) << 52;
  const int s = (e ? e : 1) - 1075;
  u128 x = 0;
  if (s >= 0) {
    const int j = s / 64, o = s % 64;
    x = (u128)digits[j] << 64 | digits[j + 1];
    if (o) x = x << o | digits[j + 2] >> (64 - o);
  } else if (s > -128) {
    x = ((u128)digits[0] << 64 | digits[1]) >> -s;
  }
  const uint64_t t = (uint64_t)((mant * x) >> 64);
  return bits >> 63 ? 0 - t : t;
}

template <typename T>
int launch_rope(RopeArgs& a, int rot, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  bool vec = rot % (2 * VEC) == 0 && a.d % (2 * VEC) == 0;
  for (int w = 0; w < 2; ++w)
    if (a.heads[w] > 0)
      vec = vec && aligned16(a.x[w]) && aligned16(a.y[w]) && a.ld[w] % VEC == 0 && a.ldo[w] % VEC == 0;
  const int step = vec ? VEC : 1;
  a.npv = a.d / (2 * step);
  a.nrot = rot / (2 * step);
  // tokens of a block: six items to a thread (65,536 tokens of 48 bf16 heads: 3 items 250 us, 4 247, 6 242, 8 243;
  // 12,669 of 40 fp32 heads: 79, 80, 81, 82), but four blocks to every SM first (64 tokens of 40 heads: one token a
  // block 3.2 us, four 4.9)
  const int64_t per_token = (int64_t)(a.heads[0] + a.heads[1]) * a.npv;
  const int64_t by_items = (6 * kRopeThreads + per_token - 1) / per_token;
  const int64_t by_blocks = a.N / (4 * (int64_t)sm_count());
  a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({by_items, by_blocks, kMaxTokens}));
  const unsigned grid = (unsigned)((a.N + a.tokens - 1) / a.tokens);
  const size_t smem = 2 * sizeof(float) * a.tokens * a.half;
  if (vec)
    rope_kernel<T, VEC><<<grid, kRopeThreads, smem, st>>>(a);
  else
    rope_kernel<T, 1><<<grid, kRopeThreads, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace
}  // namespace tt

using namespace tt;

TT_API int tt_rope(const void* q, void* q_out, int64_t q_ld, int64_t q_out_ld, const void* k, void* k_out, int64_t k_ld,
                   int64_t k_out_ld, int dtype, int64_t N, int Hq, int Hkv, int d, int rot, const int32_t* pos,
                   int64_t pos_ld, int axes, const uint8_t* axis_host, const double* freq_host, int adjacent,
                   int inverse, tt_stream_t stream) {
  if (N < 0 || Hq < 0 || Hkv < 0 || d < 2 || rot < 2 || rot > d || axes < 1) return TT_ERR_INVALID_ARG;
  if (dtype != TT_DT_BF16 && dtype != TT_DT_F16 && dtype != TT_DT_F32) return TT_ERR_INVALID_ARG;
  if (!axis_host || !freq_host) return TT_ERR_INVALID_ARG;
  if (d % 2 || rot % 2 || d > 1024 || rot > 2 * kMaxHalf || axes > kMaxAxes || Hq > 1024 || Hkv > 1024)
    return TT_ERR_UNSUPPORTED;
  RopeArgs a = {};
  for (int i = 0; i < rot / 2; ++i) {
    if (axis_host[i] >= axes || !std::isfinite(freq_host[i])) return TT_ERR_INVALID_ARG;
    a.turn[i] = turns_of(freq_host[i]);
    a.axis[i] = axis_host[i];
  }
  if (N == 0 || Hq + Hkv == 0) return TT_OK;
  const size_t es = dtype == TT_DT_F32 ? 4 : 2;
  const void* x[2] = {q, k};
  void* y[2] = {q_out, k_out};
  const int64_t ld[2] = {q_ld, k_ld}, ldo[2] = {q_out_ld, k_out_ld};
  const int heads[2] = {Hq, Hkv};
  for (int w = 0; w < 2; ++w) {
    a.x[w] = x[w]; a.y[w] = y[w]; a.ld[w] = ld[w]; a.ldo[w] = ldo[w]; a.heads[w] = heads[w];
    if (heads[w] == 0) continue;
    if (!x[w] || !y[w] || ld[w] < (int64_t)heads[w] * d || ldo[w] < (int64_t)heads[w] * d) return TT_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(x[w]) | reinterpret_cast<uintptr_t>(y[w])) % es) return TT_ERR_INVALID_ARG;
    if (x[w] == y[w] && ld[w] != ldo[w]) return TT_ERR_INVALID_ARG;
  }
  // q and k may each be turned in place, not into one another
  if (Hq > 0 && Hkv > 0 && (q_out == k_out || q_out == k || k_out == q)) return TT_ERR_INVALID_ARG;
  if (!pos || (axes > 1 && pos_ld != 0 && pos_ld < N) || N > (int64_t)INT32_MAX) return TT_ERR_INVALID_ARG;
  a.N = N; a.d = d; a.half = rot / 2; a.pos = pos; a.pos_ld = pos_ld; a.adjacent = adjacent; a.inverse = inverse;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case TT_DT_BF16: return launch_rope<__nv_bfloat16>(a, rot, st);
    case TT_DT_F16: return launch_rope<__half>(a, rot, st);
    default: return launch_rope<float>(a, rot, st);
  }
}
