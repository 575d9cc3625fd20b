// RMS norm of every head of Q and K and the rotary positions behind it, in one
// pass, and the backward pass of both.
//
//   r = (Σ_j x_j²/d + ε)^-1/2,   n_j = w_j·x_j·r,   y = R(pos)·n
//   backward: g = R(−pos)·dy,  h = w∘g,  dx = r·h − x·r³·(Σ_j h_j x_j)/d,  dw = Σ_{tokens, heads} g∘x·r
//
// (R as in rope.cu.) A group of lanes takes a head, each lane the two vectors
// of its pairs, so that the turn stays inside a lane and the sums over the
// head are a few shuffles. A block forms the sines and cosines of its tokens
// once for all their heads. n is not rounded between the norm and the turn:
// everything is fp32 from load to store.
//
// Bound by memory: forward x in, y out; backward x and dy in, dx out. The
// backward's sums for dw stay in registers over all tokens of a block; each
// block leaves one row of parts and a second small launch adds the rows in
// order, so that the result does not depend on timing.
#include "rope.cuh"

#include <algorithm>
#include <cmath>

namespace tt {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;   // tokens of a block at once
constexpr int kMaxD = 512;
constexpr int kMaxParts = 512;   // blocks of the backward: rows of parts of dw

struct NormArgs {
  const void *x[2], *dy[2];  // q, k (dy: backward)
  void* y[2];                // forward: the results; backward: dx
  int64_t x_ld[2], dy_ld[2], y_ld[2];
  const void* w[2];          // NULL: ones
  int w_fp32;
  float* parts;              // [2][gridDim.x][d], NULL: no dw
  int heads[2];
  int64_t N;
  int d, half, npv, nrot;    // npv: vector pairs of a head, the first nrot of them rotated
  int tokens;                // of a block at once
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

// T: type of the heads. VEC: elements of a vector (16 bytes, or one). A head is taken by LANES lanes with NV pairs of
// vectors each.
template <typename T, int VEC, int LANES, int NV, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ float shared[];
  float* cosines = shared;                                 // [tokens][half]
  float* sines = cosines + a.tokens * a.half;
  float* weights = sines + a.tokens * a.half;              // [2][d]
  float* red = weights + 2 * a.d;                          // backward: [warps][d]
  constexpr int kGroups = kThreads / LANES;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  // the places of this lane's vectors within a head, and of their cosines
  int o1[NV], o2[NV];
  bool rotated[NV], here[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int pv = lane + i * LANES;
    here[i] = pv < a.npv;
    rotated[i] = pv < a.nrot;
    if (rotated[i]) {
      o1[i] = a.adjacent ? 2 * VEC * pv : VEC * pv;
      o2[i] = a.adjacent ? o1[i] + VEC : o1[i] + a.half;
    } else {
      o1[i] = 2 * a.half + 2 * VEC * (pv - a.nrot);
      o2[i] = o1[i] + VEC;
    }
  }
  for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
    const int w = i >= a.d, j = i - w * a.d;
    float v = 1.f;
    if (a.w[w]) v = a.w_fp32 ? static_cast<const float*>(a.w[w])[j] : static_cast<float>(static_cast<const T*>(a.w[w])[j]);
    weights[i] = v;
  }
  float acc[2][NV][2][VEC];
  if constexpr (BWD) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[w][i][0][j] = acc[w][i][1][j] = 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * a.tokens; t0 < a.N; t0 += (int64_t)gridDim.x * a.tokens) {
    const int nt = (int)min((int64_t)a.tokens, a.N - t0);
    if (BWD) __syncthreads();  // the previous tokens' cosines are no longer read
    for (int i = threadIdx.x; i < nt * a.half; i += kThreads) {
      const int t = i / a.half, f = i - t * a.half;
      const int64_t pos = a.pos[a.axis[f] * a.pos_ld + t0 + t];
      float s, c;
      trig_of((uint64_t)pos * a.turn[f], s, c);
      cosines[i] = c;
      sines[i] = BWD ? -s : s;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int H = a.heads[w], items = nt * H;
      const float* wt = weights + w * a.d;
      // whole warps go round together: their lanes meet in the shuffles
      for (int i0 = 0; i0 < items; i0 += kGroups) {
        const int item = i0 + group;
        const bool on = item < items;
        const int t = on ? item / H : 0, h = on ? item - t * H : 0;
        const T* x = static_cast<const T*>(a.x[w]) + (t0 + t) * a.x_ld[w] + (int64_t)h * a.d;
        float u[NV][VEC], v[NV][VEC], gu[NV][VEC], gv[NV][VEC];
        float ss = 0.f, sp = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) u[i][j] = v[i][j] = gu[i][j] = gv[i][j] = 0.f;
          if (on && here[i]) {
            Vec<T, VEC>::load(x + o1[i], u[i]);
            Vec<T, VEC>::load(x + o2[i], v[i]);
            if constexpr (BWD) {
              const T* dy = static_cast<const T*>(a.dy[w]) + (t0 + t) * a.dy_ld[w] + (int64_t)h * a.d;
              Vec<T, VEC>::load(dy + o1[i], gu[i]);
              Vec<T, VEC>::load(dy + o2[i], gv[i]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) ss = fmaf(u[i][j], u[i][j], fmaf(v[i][j], v[i][j], ss));
          if constexpr (BWD) {
            if (on && here[i]) {
              if (rotated[i])
                turn_vectors<VEC>(gu[i], gv[i], cosines + t * a.half + VEC * (lane + i * LANES),
                                  sines + t * a.half + VEC * (lane + i * LANES), a.adjacent);
#pragma unroll
              for (int j = 0; j < VEC; ++j)
                sp = fmaf(gu[i][j] * wt[o1[i] + j], u[i][j], fmaf(gv[i][j] * wt[o2[i] + j], v[i][j], sp));
            }
          }
        }
        ss = sum_group<LANES>(ss);
        const float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
        float shift = 0.f;
        if constexpr (BWD) shift = r * r * r * sum_group<LANES>(sp) * a.inv_d;
        T* y = static_cast<T*>(a.y[w]) + (t0 + t) * a.y_ld[w] + (int64_t)h * a.d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!on || !here[i]) continue;
          if constexpr (BWD) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              acc[w][i][0][j] = fmaf(gu[i][j], u[i][j] * r, acc[w][i][0][j]);
              acc[w][i][1][j] = fmaf(gv[i][j], v[i][j] * r, acc[w][i][1][j]);
              u[i][j] = fmaf(gu[i][j] * wt[o1[i] + j], r, -u[i][j] * shift);
              v[i][j] = fmaf(gv[i][j] * wt[o2[i] + j], r, -v[i][j] * shift);
            }
          } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              u[i][j] *= r * wt[o1[i] + j];
              v[i][j] *= r * wt[o2[i] + j];
            }
            if (rotated[i])
              turn_vectors<VEC>(u[i], v[i], cosines + t * a.half + VEC * (lane + i * LANES),
                                sines + t * a.half + VEC * (lane + i * LANES), a.adjacent);
          }
          Vec<T, VEC>::store(y + o1[i], u[i]);
          Vec<T, VEC>::store(y + o2[i], v[i]);
        }
      }
    }
    if (!BWD) return;  // the forward's grid covers the tokens
  }
  if constexpr (BWD) {
    if (!a.parts) return;
    const int warp = threadIdx.x / 32;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            float s = acc[w][i][e][j];
#pragma unroll
            for (int o = 16; o >= LANES; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if ((threadIdx.x & 31) < LANES && here[i]) red[warp * a.d + (e ? o2[i] : o1[i]) + j] = s;
          }
      __syncthreads();
      for (int j = threadIdx.x; j < a.d; j += kThreads) {
        float s = red[j];
        for (int q = 1; q < kThreads / 32; ++q) s += red[q * a.d + j];
        a.parts[((int64_t)w * gridDim.x + blockIdx.x) * a.d + j] = s;
      }
    }
  }
}

// dw[w][j] = Σ over the rows of parts, in a fixed order: a warp takes 32 columns of every eighth row.
__global__ void __launch_bounds__(kThreads) norm_dw_kernel(const float* parts, int rows, int d, float* dwq, float* dwk) {
  __shared__ float red[kThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (d + 31) / 32, w = blockIdx.x / per, col = (blockIdx.x % per) * 32 + lane;
  float* dw = w ? dwk : dwq;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!dw) return;
  float s = 0.f;
  if (col < d)
    for (int r = warp; r < rows; r += kThreads / 32) s += parts[((int64_t)w * rows + r) * d + col];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < d) {
    for (int q = 1; q < kThreads / 32; ++q) s += red[q][lane];
    dw[col] = s;
  }
}

template <typename T, int VEC, int LANES, int NV, bool BWD>
int launch(NormArgs& a, int rot, float* dwq, float* dwk, cudaStream_t st) {
  a.npv = a.d / (2 * VEC);
  a.nrot = rot / (2 * VEC);
  const int64_t sms = sm_count();
  const int64_t per_token = (int64_t)(a.heads[0] + a.heads[1]) * LANES;
  const int64_t by_items = (6 * kThreads + per_token - 1) / per_token;
  const int64_t by_blocks = a.N / (4 * sms);
  a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({by_items, by_blocks, kMaxTokens}));
  const int64_t tiles = (a.N + a.tokens - 1) / a.tokens;
  const int64_t grid = BWD ? std::min<int64_t>({tiles, 2 * sms, kMaxParts}) : tiles;
  const size_t smem = sizeof(float) * (2 * (size_t)a.tokens * a.half + 2 * a.d + (BWD ? kThreads / 32 * a.d : 0));
  norm_rope_kernel<T, VEC, LANES, NV, BWD><<<(unsigned)grid, kThreads, smem, st>>>(a);
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
  return cuda_status(cudaLaunchKernelEx(&cfg, norm_dw_kernel, (const float*)a.parts, (int)grid, a.d, dwq, dwk));
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
  if (!vec) return launch<T, 1, 32, kMaxD / 64, BWD>(a, rot, dwq, dwk, st);
  const int npv = a.d / (2 * VEC);
  if (npv <= 4) return launch<T, VEC, 4, 1, BWD>(a, rot, dwq, dwk, st);
  if (npv <= 8) return launch<T, VEC, 8, 1, BWD>(a, rot, dwq, dwk, st);
  if (npv <= 16) return launch<T, VEC, 16, 1, BWD>(a, rot, dwq, dwk, st);
  if (npv <= 32) return launch<T, VEC, 32, 1, BWD>(a, rot, dwq, dwk, st);
  if constexpr (sizeof(T) == 4) return launch<T, VEC, 32, 2, BWD>(a, rot, dwq, dwk, st);
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
  return d < 2 || d > kMaxD ? 0 : (size_t)2 * kMaxParts * d * sizeof(float);
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
