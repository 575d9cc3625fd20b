// RMS norm of every head of Q and K and the rotary positions behind it, in one
// pass, and the backward pass of both.
//
//   r = (Σ_j x_j²/d + ε)^-1/2,   n_j = w_j·x_j·r,   y = R(pos)·n
//   backward: g = R(−pos)·dy,  h = w∘g,  dx = r·h − x·r³·(Σ_j h_j x_j)/d,  dw = Σ_{tokens, heads} g∘x·r
//
// (R as in rope.cu.) A group of lanes takes a head, each lane the two vectors
// of its pairs, so that the turn stays inside a lane and the sums over the
// head are a few shuffles. A block forms the sines and cosines of its tokens
// once for all their heads, and a group takes heads of one token after one
// another, so that weights, cosines and sines stay in registers. n is not
// rounded between the norm and the turn: everything is fp32 from load to
// store, two elements in one instruction.
//
// Bound by memory: forward x in, y out; backward x and dy in, dx out. A
// thread's vectors come by asynchronous copies, three heads ahead: registers
// ahead instead took 378 us where this takes 234 (65,536 tokens of 40 + 8 heads
// of 128, bf16: 6.9 TB/s). The backward's sums for dw stay in registers over
// all tokens of a block, and its blocks take heads of q or of k, not both, so
// that there is one set of sums; each block leaves one row of parts and a
// second small launch adds the rows in order, so that the result does not
// depend on timing. 12,669 tokens of 16 + 8 heads of 128, bf16: 46 + 3.5 us
// (5.1 TB/s): 128 registers leave 16 warps to an SM, which issue in 0.48 of the
// cycles and wait for shuffles and the copies in the others. Three blocks to an
// SM spill (87 us).
#include "rope.cuh"
#include "tc_common.cuh"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace tt {
namespace {

constexpr int kBwdBlocks = 2;       // blocks to an SM, backward
constexpr int kFwdItems = 12;       // heads of a thread, forward, where there are tokens enough
// Heads of a thread on their way or in use. 65,536 tokens forward, 12,669 backward: three 237 and 46 us, four 234 and 46, five 239
// and 47.5.
constexpr int kDepth = 4;
constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;   // tokens of a block at once (backward of 12,669: 16 49 us, 32 and 64 46)
constexpr int kMaxD = 512;
constexpr int kSmemMost = 200 * 1024;
constexpr int kMaxParts = 1024;  // blocks of the backward: rows of parts of dw

struct NormArgs {
  const void *x[2], *dy[2];  // q, k (dy: backward)
  void* y[2];                // forward: the results; backward: dx
  int64_t x_ld[2], dy_ld[2], y_ld[2];
  const void* w[2];          // NULL: ones
  int w_fp32;
  float* parts;              // [gridDim.x][d], the blocks of q first; NULL: no dw
  int heads[2];
  int64_t N;
  int d, half, npv, nrot;    // npv: vector pairs of a head, the first nrot of them rotated
  int tokens[2];             // of a block at once (backward: of one of q, of k)
  int split[2];              // groups that share a token's heads
  float eps, inv_d;
  const int32_t* pos;
  int64_t pos_ld;
  int adjacent;
  uint64_t turn[kMaxHalf];   // frequencies/2π mod 1, in units of 2^-64
  uint8_t axis[kMaxHalf];
};

template <int LANES>
__device__ __forceinline__ float sum_group(float x) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// r³·mean: r³ alone leaves fp32's range from heads of 1e-13 on, r·mean does not.
__device__ __forceinline__ float cubed(float r, float mean) { return r * (r * (r * mean)); }

__device__ __forceinline__ void copy16(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// A 16-byte vector as pairs of floats and back.
template <typename T>
constexpr int kPairs = 8 / sizeof(T);
template <typename T>
__device__ __forceinline__ void unpack(const uint4& x, float2 (&f)[kPairs<T>]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (sizeof(T) == 4) {
    f[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    f[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value)
        f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float2 (&f)[kPairs<T>]) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = pack_bf16(f[i].x, f[i].y);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The weights of both tensors into shared memory: [2][d].
template <typename T>
__device__ __forceinline__ void load_weights(const NormArgs& a, float* weights) {
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    const int w = i >= a.d, j = i - w * a.d;
    float v = 1.f;
    if (a.w[w]) v = a.w_fp32 ? static_cast<const float*>(a.w[w])[j] : static_cast<float>(static_cast<const T*>(a.w[w])[j]);
    weights[i] = v;
  }
}
// Cosines and sines [nt][half] of the tokens t0 .. t0 + nt − 1. A thread keeps to one frequency: in a table among the parameters
// the lanes of a warp look up their 32 places one after another (a lookup for every angle: the backward of 12,669 tokens 61 us,
// one for a thread's: 50).
__device__ __forceinline__ void load_trig(const NormArgs& a, int64_t t0, int nt, bool back, float* cosines, float* sines) {
  if (!a.half) return;
  const int step = kThreads / a.half, first = (int)threadIdx.x / a.half, f = (int)threadIdx.x - first * a.half;
  if (first >= step) return;
  const uint64_t turn = a.turn[f];
  const int32_t* pos = a.pos + a.axis[f] * a.pos_ld + t0;
  for (int t = first; t < nt; t += step) {
    float s, c;
    trig_of((uint64_t)(int64_t)pos[t] * turn, s, c);
    cosines[t * a.half + f] = c;
    sines[t * a.half + f] = back ? -s : s;
  }
}
// The tensor and the blocks that a block of the backward belongs to: the first ones take q, the others k, in proportion to
// the heads, so that a thread sums one weight's gradient only. Forward: both tensors, all blocks.
template <bool BWD>
struct Role {
  int first, last, block, blocks;
  __device__ __forceinline__ Role(int q_blocks) {
    const int b = blockIdx.x, n = gridDim.x;
    first = BWD && b >= q_blocks;
    last = BWD ? first : 1;
    block = first ? b - q_blocks : b;
    blocks = !BWD ? n : first ? n - q_blocks : q_blocks;
  }
};
// The block's row of parts of dw, from the warps' rows in red [warps][d].
__device__ __forceinline__ void store_parts(const NormArgs& a, const float* red) {
  __syncthreads();
  for (int j = threadIdx.x; j < a.d; j += kThreads) {
    float s = red[j];
    for (int q = 1; q < kThreads / 32; ++q) s += red[q * a.d + j];
    a.parts[(int64_t)blockIdx.x * a.d + j] = s;
  }
}

// Heads in 16-byte vectors, a head by LANES lanes with NV pairs of vectors each.
template <typename T, int LANES, int NV, bool BWD, bool ADJ>
__global__ void __launch_bounds__(kThreads, NV == 1 ? (BWD ? 2 : 3) : 1)
    norm_rope_kernel(const __grid_constant__ NormArgs a, int q_blocks) {
  constexpr int VEC = 16 / sizeof(T), P = kPairs<T>, kGroups = kThreads / LANES;
  constexpr int kEach = BWD ? 4 : 2, kVectors = kEach * NV;  // vectors of a thread's share of a head
  extern __shared__ __align__(16) float shared[];
  const Role<BWD> role(q_blocks);
  const int tokens = a.tokens[role.first];
  float* cosines = shared;                                 // [tokens][half]
  float* sines = cosines + tokens * a.half;
  float* weights = sines + tokens * a.half;                // [2][d]
  float* red = weights + 2 * a.d;                          // backward: [warps][d]
  uint4* ring = reinterpret_cast<uint4*>(red + (BWD ? kThreads / 32 * a.d : 0));  // [kDepth][kVectors][kThreads]
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  // the places of this lane's vectors within a head; a lane that has none goes along on the head's first and adds nothing
  int o1[NV], o2[NV];
  bool rotated[NV], here[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int pv = lane + i * LANES;
    here[i] = pv < a.npv;
    rotated[i] = pv < a.nrot;
    if (rotated[i]) {
      o1[i] = ADJ ? 2 * VEC * pv : VEC * pv;
      o2[i] = ADJ ? o1[i] + VEC : o1[i] + a.half;
    } else {
      o1[i] = here[i] ? 2 * a.half + 2 * VEC * (pv - a.nrot) : 0;
      o2[i] = here[i] ? o1[i] + VEC : 0;
    }
  }
  load_weights<T>(a, weights);
  float2 acc[NV][2][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) acc[i][0][j] = acc[i][1][j] = make_float2(0.f, 0.f);
  for (int64_t t0 = (int64_t)role.block * tokens; t0 < a.N; t0 += (int64_t)role.blocks * tokens) {
    const int nt = (int)min((int64_t)tokens, a.N - t0);
    for (int w = role.first; w <= role.last; ++w) {
      const int H = a.heads[w], split = a.split[w], units = nt * split, rounds = (H + split - 1) / split;
      // A group takes a token's heads `split` apart, then those of another token. Whole warps go round together: their lanes
      // meet in the shuffles.
      const int n = (units + kGroups - 1) / kGroups * rounds, step = split * a.d;
      // a thread's vectors come by asynchronous copies into places of its own, kDepth − 1 heads ahead
      int next_unit = group, next_round = 0, next_h = 0;
      const T *next_x = nullptr, *next_dy = nullptr;
      auto enter = [&]() {  // the token of next_unit
        const int t = next_unit / split;
        next_h = next_unit < units ? next_unit - t * split : H;
        next_x = static_cast<const T*>(a.x[w]) + (t0 + t) * a.x_ld[w] + (int64_t)next_h * a.d;
        if (BWD) next_dy = static_cast<const T*>(a.dy[w]) + (t0 + t) * a.dy_ld[w] + (int64_t)next_h * a.d;
      };
      auto copy = [&](int stage) {
        if (next_h < H) {
          uint4* slot = ring + stage * kVectors * kThreads + threadIdx.x;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            copy16(slot + (kEach * i) * kThreads, next_x + o1[i]);
            copy16(slot + (kEach * i + 1) * kThreads, next_x + o2[i]);
            if constexpr (BWD) {
              copy16(slot + (kEach * i + 2) * kThreads, next_dy + o1[i]);
              copy16(slot + (kEach * i + 3) * kThreads, next_dy + o2[i]);
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next_h += split;
        next_x += step;
        next_dy += step;
        if (++next_round == rounds) {
          next_round = 0;
          next_unit += kGroups;
          enter();
        }
      };
      enter();
      for (int k = 0; k < kDepth - 1; ++k) copy(k);
      if (w == role.first) {  // while they come
        if (BWD) __syncthreads();  // the previous tokens' cosines are no longer read
        load_trig(a, t0, nt, BWD, cosines, sines);
        __syncthreads();
      }
      float2 w1[NV][P], w2[NV][P];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) {
          w1[i][j] = reinterpret_cast<const float2*>(weights + w * a.d + o1[i])[j];
          w2[i][j] = reinterpret_cast<const float2*>(weights + w * a.d + o2[i])[j];
        }
      // Non-adjacent pairs: the cosines, sines and negated sines of two pairs each; adjacent ones: both of a pair.
      float2 c[NV][ADJ ? 2 * P : P], s1[NV][ADJ ? 2 * P : P], s2[NV][ADJ ? 1 : P];
      T* y = nullptr;
      int h = 0, round = 0, unit = group, stage = 0, ahead = kDepth - 1;
      for (int k = 0; k < n; ++k) {
        if (round == 0) {
          const int t = unit < units ? unit / split : 0;
          h = unit < units ? unit - t * split : H;
          y = static_cast<T*>(a.y[w]) + (t0 + t) * a.y_ld[w] + (int64_t)h * a.d;
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (rotated[i]) {
              const int at = t * a.half + VEC * (lane + i * LANES);
              const float2* pc = reinterpret_cast<const float2*>(cosines + at);
              const float2* ps = reinterpret_cast<const float2*>(sines + at);
#pragma unroll
              for (int j = 0; j < P; ++j) {
                const float2 cj = pc[j], sj = ps[j];
                if constexpr (ADJ) {
                  c[i][2 * j] = make_float2(cj.x, cj.x), c[i][2 * j + 1] = make_float2(cj.y, cj.y);
                  s1[i][2 * j] = make_float2(-sj.x, sj.x), s1[i][2 * j + 1] = make_float2(-sj.y, sj.y);
                } else {
                  c[i][j] = cj;
                  s1[i][j] = sj;
                  s2[i][j] = make_float2(-sj.x, -sj.y);
                }
              }
            }
        }
        const bool on = h < H;
        float2 u[NV][P], v[NV][P], gu[NV][P], gv[NV][P];
        copy(ahead);
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        const uint4* slot = ring + stage * kVectors * kThreads + threadIdx.x;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          unpack<T>(slot[(kEach * i) * kThreads], u[i]);
          unpack<T>(slot[(kEach * i + 1) * kThreads], v[i]);
          if constexpr (BWD) {
            unpack<T>(slot[(kEach * i + 2) * kThreads], gu[i]);
            unpack<T>(slot[(kEach * i + 3) * kThreads], gv[i]);
          }
        }
        // both vectors turned
        auto turn = [&](float2 (&p)[P], float2 (&q)[P], int i) {
          if (!rotated[i]) return;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            if constexpr (ADJ) {
              p[j] = __ffma2_rn(make_float2(p[j].y, p[j].x), s1[i][j], __fmul2_rn(p[j], c[i][j]));
              q[j] = __ffma2_rn(make_float2(q[j].y, q[j].x), s1[i][P + j], __fmul2_rn(q[j], c[i][P + j]));
            } else {
              const float2 b = p[j];
              p[j] = __ffma2_rn(q[j], s2[i][j], __fmul2_rn(b, c[i][j]));
              q[j] = __ffma2_rn(b, s1[i][j], __fmul2_rn(q[j], c[i][j]));
            }
          }
        };
        float2 ss = make_float2(0.f, 0.f), sp = ss;
        float2 hu[NV][P], hv[NV][P];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (BWD) turn(gu[i], gv[i], i);
          float2 one = make_float2(0.f, 0.f), two = one;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            one = __ffma2_rn(u[i][j], u[i][j], __ffma2_rn(v[i][j], v[i][j], one));
            if constexpr (BWD) {
              hu[i][j] = __fmul2_rn(gu[i][j], w1[i][j]);
              hv[i][j] = __fmul2_rn(gv[i][j], w2[i][j]);
              two = __ffma2_rn(hu[i][j], u[i][j], __ffma2_rn(hv[i][j], v[i][j], two));
            }
          }
          if (here[i]) {
            ss = __fadd2_rn(ss, one);
            sp = __fadd2_rn(sp, two);
          }
        }
        const float r = rsqrtf(fmaf(sum_group<LANES>(ss.x + ss.y), a.inv_d, a.eps));
        const float2 r2 = make_float2(r, r);
        float2 back = r2;
        if constexpr (BWD) {
          const float shift = -cubed(r, sum_group<LANES>(sp.x + sp.y) * a.inv_d);
          back = make_float2(shift, shift);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!on || !here[i]) continue;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            if constexpr (BWD) {
              acc[i][0][j] = __ffma2_rn(gu[i][j], __fmul2_rn(u[i][j], r2), acc[i][0][j]);
              acc[i][1][j] = __ffma2_rn(gv[i][j], __fmul2_rn(v[i][j], r2), acc[i][1][j]);
              u[i][j] = __ffma2_rn(hu[i][j], r2, __fmul2_rn(u[i][j], back));
              v[i][j] = __ffma2_rn(hv[i][j], r2, __fmul2_rn(v[i][j], back));
            } else {
              u[i][j] = __fmul2_rn(u[i][j], __fmul2_rn(w1[i][j], r2));
              v[i][j] = __fmul2_rn(v[i][j], __fmul2_rn(w2[i][j], r2));
            }
          }
          if constexpr (!BWD) turn(u[i], v[i], i);
          *reinterpret_cast<uint4*>(y + o1[i]) = pack<T>(u[i]);
          *reinterpret_cast<uint4*>(y + o2[i]) = pack<T>(v[i]);
        }
        h += split;
        y += step;
        if (++round == rounds) round = 0, unit += kGroups;
        if (++stage == kDepth) stage = 0;
        if (++ahead == kDepth) ahead = 0;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // (groups without copies)
    }
    if (!BWD) return;  // the forward's grid covers the tokens
  }
  if constexpr (BWD) {
    if (!a.parts) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < P; ++j) {
          float2 s = acc[i][e][j];
#pragma unroll
          for (int o = 16; o >= LANES; o >>= 1)
            s = __fadd2_rn(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
          if ((threadIdx.x & 31) < LANES && here[i])
            reinterpret_cast<float2*>(red + threadIdx.x / 32 * a.d + (e ? o2[i] : o1[i]))[j] = s;
        }
    store_parts(a, red);
  }
}

// Any alignment, head size and number of turned dimensions: element accesses, a warp to a head.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const __grid_constant__ NormArgs a, int q_blocks) {
  constexpr int NV = kMaxD / 64, kGroups = kThreads / 32;
  extern __shared__ __align__(16) float shared[];
  const Role<BWD> role(q_blocks);
  const int tokens = a.tokens[role.first];
  float* cosines = shared;                                 // [tokens][half]
  float* sines = cosines + tokens * a.half;
  float* weights = sines + tokens * a.half;                // [2][d]
  float* red = weights + 2 * a.d;                          // backward: [warps][d]
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  int o1[NV], o2[NV];  // a lane's pairs
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = lane + 32 * i;
    const bool rotated = p < a.half;
    o1[i] = !rotated ? 2 * p : a.adjacent ? 2 * p : p;
    o2[i] = !rotated ? 2 * p + 1 : a.adjacent ? 2 * p + 1 : p + a.half;
  }
  load_weights<T>(a, weights);
  float acc[NV][2] = {};
  for (int64_t t0 = (int64_t)role.block * tokens; t0 < a.N; t0 += (int64_t)role.blocks * tokens) {
    const int nt = (int)min((int64_t)tokens, a.N - t0);
    if (BWD) __syncthreads();
    load_trig(a, t0, nt, BWD, cosines, sines);
    __syncthreads();
    for (int w = role.first; w <= role.last; ++w) {
      const int H = a.heads[w];
      for (int item = group; item < nt * H; item += kGroups) {
        const int t = item / H, h = item - t * H;
        const T* x = static_cast<const T*>(a.x[w]) + (t0 + t) * a.x_ld[w] + (int64_t)h * a.d;
        T* y = static_cast<T*>(a.y[w]) + (t0 + t) * a.y_ld[w] + (int64_t)h * a.d;
        const float* wt = weights + w * a.d;
        float u[NV], v[NV], gu[NV], gv[NV], ss = 0.f, sp = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int p = lane + 32 * i;
          if (p >= a.npv) continue;
          u[i] = static_cast<float>(x[o1[i]]);
          v[i] = static_cast<float>(x[o2[i]]);
          ss = fmaf(u[i], u[i], fmaf(v[i], v[i], ss));
          if constexpr (BWD) {
            const T* dy = static_cast<const T*>(a.dy[w]) + (t0 + t) * a.dy_ld[w] + (int64_t)h * a.d;
            gu[i] = static_cast<float>(dy[o1[i]]);
            gv[i] = static_cast<float>(dy[o2[i]]);
            if (p < a.half) turn_pair(gu[i], gv[i], cosines[t * a.half + p], sines[t * a.half + p]);
            sp = fmaf(gu[i] * wt[o1[i]], u[i], fmaf(gv[i] * wt[o2[i]], v[i], sp));
          }
        }
        const float r = rsqrtf(fmaf(sum_group<32>(ss), a.inv_d, a.eps));
        const float shift = BWD ? cubed(r, sum_group<32>(sp) * a.inv_d) : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int p = lane + 32 * i;
          if (p >= a.npv) continue;
          if constexpr (BWD) {
            acc[i][0] = fmaf(gu[i], u[i] * r, acc[i][0]);
            acc[i][1] = fmaf(gv[i], v[i] * r, acc[i][1]);
            u[i] = fmaf(gu[i] * wt[o1[i]], r, -u[i] * shift);
            v[i] = fmaf(gv[i] * wt[o2[i]], r, -v[i] * shift);
          } else {
            u[i] *= wt[o1[i]] * r;
            v[i] *= wt[o2[i]] * r;
            if (p < a.half) turn_pair(u[i], v[i], cosines[t * a.half + p], sines[t * a.half + p]);
          }
          y[o1[i]] = static_cast<T>(u[i]);
          y[o2[i]] = static_cast<T>(v[i]);
        }
      }
    }
    if (!BWD) return;
  }
  if constexpr (BWD) {
    if (!a.parts) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < a.npv) {
        red[group * a.d + o1[i]] = acc[i][0];
        red[group * a.d + o2[i]] = acc[i][1];
      }
    store_parts(a, red);
  }
}

// dw[j] = Σ over the rows of parts (the first q_rows of q, the others of k), in a fixed order: a warp takes 32 columns of
// every eighth row, four rows at a time.
__global__ void __launch_bounds__(kThreads) norm_dw_kernel(const float* parts, int q_rows, int rows, int d, float* dwq,
                                                           float* dwk) {
  __shared__ float red[kThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (d + 31) / 32, w = blockIdx.x / per, col = (blockIdx.x % per) * 32 + lane;
  const int lo = w ? q_rows : 0, hi = w ? rows : q_rows;
  float* dw = w ? dwk : dwq;
  wait_prerequisites();
  if (!dw) return;
  constexpr int kStep = kThreads / 32, kLoads = 8;
  float s = 0.f;
  if (col < d)
    for (int r = lo + warp; r < hi; r += kLoads * kStep) {
      float x[kLoads];
#pragma unroll
      for (int q = 0; q < kLoads; ++q) x[q] = r + q * kStep < hi ? parts[(int64_t)(r + q * kStep) * d + col] : 0.f;
#pragma unroll
      for (int q = 0; q < kLoads; ++q) s += x[q];
    }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < d) {
    for (int q = 1; q < kThreads / 32; ++q) s += red[q][lane];
    dw[col] = s;
  }
}

// LANES lanes to a head: sets up the blocks' shares of the tokens and launches KERNEL.
template <auto KERNEL, bool BWD>
int launch(NormArgs& a, int lanes, size_t ring, float* dwq, float* dwk, cudaStream_t st) {
  const int64_t sms = sm_count(), H = a.heads[0] + a.heads[1];
  int64_t grid, q_blocks = 0;
  if (BWD) {
    // a tensor's blocks by its heads, and each block's tokens in equal parts of at most kMaxTokens
    const int64_t all = std::min<int64_t>(kBwdBlocks * sms, kMaxParts);
    int64_t blocks[2];
    for (int w = 0; w < 2; ++w) {
      blocks[w] = a.heads[w] ? std::min(a.N, std::max<int64_t>(1, w ? all - blocks[0] : all * a.heads[0] / H)) : 0;
      const int64_t share = blocks[w] ? (a.N + blocks[w] - 1) / blocks[w] : 1, parts = (share + kMaxTokens - 1) / kMaxTokens;
      a.tokens[w] = (int)((share + parts - 1) / parts);
    }
    q_blocks = blocks[0];
    grid = blocks[0] + blocks[1];
  } else {
    const int64_t by_items = (kFwdItems * kThreads + H * lanes - 1) / (H * lanes), by_blocks = a.N / (4 * sms);
    a.tokens[0] = (int)std::max<int64_t>(1, std::min<int64_t>({by_items, by_blocks, kMaxTokens}));
    grid = (a.N + a.tokens[0] - 1) / a.tokens[0];
  }
  const int tokens = std::max(a.tokens[0], a.tokens[1]), groups = kThreads / lanes;
  for (int w = 0; w < 2; ++w) {
    // the groups to a token's heads that leave the fewest heads to the busiest group
    const int nt = a.tokens[BWD ? w : 0], H = a.heads[w];
    int best = INT32_MAX;
    a.split[w] = 1;
    for (int split = 1; split <= std::min(H, groups); ++split) {
      const int heads = (nt * split + groups - 1) / groups * ((H + split - 1) / split);
      if (heads < best) best = heads, a.split[w] = split;
    }
  }
  const size_t smem = sizeof(float) * (2 * (size_t)tokens * a.half + 2 * a.d + (BWD ? kThreads / 32 * a.d : 0)) + ring;
  if (smem > 48 * 1024 && !tc::smem_attr_set<KERNEL>(kSmemMost)) return TT_ERR_CUDA;
  KERNEL<<<(unsigned)grid, kThreads, smem, st>>>(a, (int)q_blocks);
  if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
  if (!BWD || !a.parts) return TT_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * ((a.d + 31) / 32)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, norm_dw_kernel, (const float*)a.parts, (int)q_blocks, (int)grid, a.d, dwq, dwk));
}

template <typename T, int LANES, int NV, bool BWD>
int launch_vectors(NormArgs& a, float* dwq, float* dwk, cudaStream_t st) {
  const size_t ring = (size_t)kDepth * (BWD ? 4 : 2) * NV * kThreads * 16;
  return a.adjacent ? launch<norm_rope_kernel<T, LANES, NV, BWD, true>, BWD>(a, LANES, ring, dwq, dwk, st)
                    : launch<norm_rope_kernel<T, LANES, NV, BWD, false>, BWD>(a, LANES, ring, dwq, dwk, st);
}

template <typename T, bool BWD>
int launch_type(NormArgs& a, int rot, float* dwq, float* dwk, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  bool vec = rot % (2 * VEC) == 0 && a.d % (2 * VEC) == 0;
  for (int w = 0; w < 2; ++w)
    if (a.heads[w] > 0) {
      vec = vec && aligned16(a.x[w]) && aligned16(a.y[w]) && a.x_ld[w] % VEC == 0 && a.y_ld[w] % VEC == 0;
      if (BWD) vec = vec && aligned16(a.dy[w]) && a.dy_ld[w] % VEC == 0;
    }
  const int step = vec ? VEC : 1;
  a.npv = a.d / (2 * step);
  a.nrot = rot / (2 * step);
  if (!vec) return launch<norm_rope_any_kernel<T, BWD>, BWD>(a, 32, 0, dwq, dwk, st);
  if (a.npv <= 4) return launch_vectors<T, 4, 1, BWD>(a, dwq, dwk, st);
  if (a.npv <= 8) return launch_vectors<T, 8, 1, BWD>(a, dwq, dwk, st);
  if (a.npv <= 16) return launch_vectors<T, 16, 1, BWD>(a, dwq, dwk, st);
  if (a.npv <= 32) return launch_vectors<T, 32, 1, BWD>(a, dwq, dwk, st);
  if constexpr (sizeof(T) == 4) return launch_vectors<T, 32, 2, BWD>(a, dwq, dwk, st);
  return TT_ERR_UNSUPPORTED;
}

// The arguments that both directions have; TT_OK with *done = true where there is nothing to do.
int check(NormArgs& a, int dtype, int64_t N, int d, int w_dtype, float eps, int rot, const int32_t* pos, int64_t pos_ld,
          int axes, const uint8_t* axis_host, const double* freq_host, int adjacent, bool bwd) {
  if (N < 0 || a.heads[0] < 0 || a.heads[1] < 0 || d < 2 || rot < 0 || rot > d) return TT_ERR_INVALID_ARG;
  if (dtype != TT_DT_BF16 && dtype != TT_DT_F16 && dtype != TT_DT_F32) return TT_ERR_INVALID_ARG;
  if (w_dtype != dtype && w_dtype != TT_DT_F32) return TT_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return TT_ERR_INVALID_ARG;
  if (rot && (!axis_host || !freq_host || axes < 1)) return TT_ERR_INVALID_ARG;
  if (d % 2 || rot % 2 || d > kMaxD || rot > 2 * kMaxHalf || axes > kMaxAxes || a.heads[0] > 1024 || a.heads[1] > 1024)
    return TT_ERR_UNSUPPORTED;
  for (int i = 0; i < rot / 2; ++i) {
    if (axis_host[i] >= axes || !std::isfinite(freq_host[i])) return TT_ERR_INVALID_ARG;
    a.turn[i] = turns_of(freq_host[i]);
    a.axis[i] = axis_host[i];
  }
  a.N = N; a.d = d; a.half = rot / 2; a.eps = eps; a.inv_d = 1.f / (float)d; a.pos = pos; a.pos_ld = pos_ld;
  a.adjacent = adjacent; a.w_fp32 = w_dtype == TT_DT_F32;
  if (N == 0 || a.heads[0] + a.heads[1] == 0) return TT_OK;
  if (N > (int64_t)INT32_MAX) return TT_ERR_INVALID_ARG;
  const size_t es = dtype == TT_DT_F32 ? 4 : 2;
  for (int w = 0; w < 2; ++w) {
    if (a.heads[w] == 0) continue;
    const int64_t least = (int64_t)a.heads[w] * d;
    const void* ptr[3] = {a.x[w], a.y[w], bwd ? a.dy[w] : a.x[w]};
    const int64_t ld[3] = {a.x_ld[w], a.y_ld[w], bwd ? a.dy_ld[w] : a.x_ld[w]};
    for (int i = 0; i < 3; ++i)
      if (!ptr[i] || reinterpret_cast<uintptr_t>(ptr[i]) % es || ld[i] < least) return TT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a.w[w]) % (a.w_fp32 ? 4 : es)) return TT_ERR_INVALID_ARG;
    // an output may be an input of its own, with that one's stride
    if (a.y[w] == a.x[w] && a.y_ld[w] != a.x_ld[w]) return TT_ERR_INVALID_ARG;
    if (bwd && a.y[w] == a.dy[w] && a.y_ld[w] != a.dy_ld[w]) return TT_ERR_INVALID_ARG;
  }
  if (a.heads[0] && a.heads[1]) {  // ... not one of the other tensor's
    if (a.y[0] == a.y[1] || a.y[0] == a.x[1] || a.y[1] == a.x[0]) return TT_ERR_INVALID_ARG;
    if (bwd && (a.y[0] == a.dy[1] || a.y[1] == a.dy[0])) return TT_ERR_INVALID_ARG;
  }
  if (reinterpret_cast<uintptr_t>(pos) % 4) return TT_ERR_INVALID_ARG;
  if (rot && (!pos || (axes > 1 && pos_ld != 0 && pos_ld < N))) return TT_ERR_INVALID_ARG;
  return TT_OK;
}

}  // namespace
}  // namespace tt

using namespace tt;

TT_API int tt_qk_norm_rope(const void* q, void* q_out, int64_t q_ld, int64_t q_out_ld, const void* k, void* k_out,
                           int64_t k_ld, int64_t k_out_ld, int dtype, int64_t N, int Hq, int Hkv, int d,
                           const void* q_weight, const void* k_weight, int w_dtype, float eps, int rot,
                           const int32_t* pos, int64_t pos_ld, int axes, const uint8_t* axis_host,
                           const double* freq_host, int adjacent, tt_stream_t stream) {
  NormArgs a = {};
  a.x[0] = q; a.x[1] = k; a.x_ld[0] = q_ld; a.x_ld[1] = k_ld;
  a.y[0] = q_out; a.y[1] = k_out; a.y_ld[0] = q_out_ld; a.y_ld[1] = k_out_ld;
  a.w[0] = q_weight; a.w[1] = k_weight; a.heads[0] = Hq; a.heads[1] = Hkv;
  const int rc = check(a, dtype, N, d, w_dtype, eps, rot, pos, pos_ld, axes, axis_host, freq_host, adjacent, false);
  if (rc || N == 0 || Hq + Hkv == 0) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case TT_DT_BF16: return launch_type<__nv_bfloat16, false>(a, rot, nullptr, nullptr, st);
    case TT_DT_F16: return launch_type<__half, false>(a, rot, nullptr, nullptr, st);
    default: return launch_type<float, false>(a, rot, nullptr, nullptr, st);
  }
}

TT_API size_t tt_qk_norm_rope_bwd_workspace_bytes(int d) {
  return d < 2 || d > kMaxD ? 0 : (size_t)kMaxParts * d * sizeof(float);
}

TT_API int tt_qk_norm_rope_bwd(const void* dq_out, int64_t dq_out_ld, const void* q, int64_t q_ld, void* dq, int64_t dq_ld,
                               const void* dk_out, int64_t dk_out_ld, const void* k, int64_t k_ld, void* dk,
                               int64_t dk_ld, int dtype, int64_t N, int Hq, int Hkv, int d, const void* q_weight,
                               const void* k_weight, int w_dtype, float eps, int rot, const int32_t* pos,
                               int64_t pos_ld, int axes, const uint8_t* axis_host, const double* freq_host,
                               int adjacent, float* dq_weight, float* dk_weight, void* ws, size_t ws_bytes,
                               tt_stream_t stream) {
  NormArgs a = {};
  a.x[0] = q; a.x[1] = k; a.x_ld[0] = q_ld; a.x_ld[1] = k_ld;
  a.dy[0] = dq_out; a.dy[1] = dk_out; a.dy_ld[0] = dq_out_ld; a.dy_ld[1] = dk_out_ld;
  a.y[0] = dq; a.y[1] = dk; a.y_ld[0] = dq_ld; a.y_ld[1] = dk_ld;
  a.w[0] = q_weight; a.w[1] = k_weight; a.heads[0] = Hq; a.heads[1] = Hkv;
  int rc = check(a, dtype, N, d, w_dtype, eps, rot, pos, pos_ld, axes, axis_host, freq_host, adjacent, true);
  if (rc) return rc;
  const bool want = dq_weight || dk_weight;
  if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) % 4) return TT_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0 || Hq + Hkv == 0) {  // sums over nothing
    cudaError_t e = cudaSuccess;
    if (dq_weight) e = cudaMemsetAsync(dq_weight, 0, sizeof(float) * d, st);
    if (dk_weight && e == cudaSuccess) e = cudaMemsetAsync(dk_weight, 0, sizeof(float) * d, st);
    return cuda_status(e);
  }
  if (want) {
    if (!ws || !aligned16(ws)) return TT_ERR_INVALID_ARG;
    if (ws_bytes < tt_qk_norm_rope_bwd_workspace_bytes(d)) return TT_ERR_WORKSPACE;
    a.parts = static_cast<float*>(ws);
  }
  switch (dtype) {
    case TT_DT_BF16: return launch_type<__nv_bfloat16, true>(a, rot, dq_weight, dk_weight, st);
    case TT_DT_F16: return launch_type<__half, true>(a, rot, dq_weight, dk_weight, st);
    default: return launch_type<float, true>(a, rot, dq_weight, dk_weight, st);
  }
}
