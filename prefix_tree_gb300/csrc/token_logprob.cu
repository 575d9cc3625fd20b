// Log-probability of a given token, entropy and top alternatives of every row
// of logits, and the gradient of any function of them.
//
//   lse = log Σ_v e^{z_v};   logp = z_y − lse;   top: the k largest z (ties to the lower index)
//   H   = lse − Σ_v p_v z_v = log S − U/S,   S = Σ_v e^{d_v},  U = Σ_v d_v e^{d_v},  d_v = z_v − max z
// (S >= 1 and U <= 0: the two terms of H have one sign, nothing cancels).
//
// Forward: one pass over the row. A thread takes 16-byte vectors and folds
// them into (m, s, u) with a running maximum; beside it it keeps the vector
// that holds its largest logit. The k largest logits of the row all lie with
// the k threads whose largest (value, position) are the row's k best: a
// thread outside them has k better elements elsewhere for each of its own.
// So the top alternatives cost the pass one comparison per vector; after it,
// the k threads are found (a bitonic sort per warp, sorted lists merged) and
// only their elements, k/threads of the row, are read again.
//
// Backward: dz_v = p_v·(g_lse − G − g_H·(logp_v + H)) + g_logp·[v = y] + Σ_j g_top_j·[v = id_j],
// with G = g_logp + Σ_j g_top_j: one read and one write of the row.
#include <cooperative_groups.h>

#include <cuda_fp16.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace tt {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Offsets from the maximum below this are taken as this: e^-128 is 0 in fp32,
// and 0·d stays 0 for a masked logit (d = -inf).
constexpr float kFloor = -128.f;
constexpr int kTopMax = 32;
constexpr int kBlock = 256;

typedef unsigned long long u64;

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ------------------------------------------------------------------ 16-byte vectors of a row
template <typename T>
struct Row {
  static constexpr int VN = 16 / sizeof(T);
  const T* p;    // element 0
  int shift;     // elements between the 16-byte boundary at or below p and p
  int64_t V;
  int nvec;
  __device__ __forceinline__ Row(const T* row, int64_t V_) : p(row), V(V_) {
    shift = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    nvec = (int)((V + shift + VN - 1) / VN);
  }
  // first element of vector j (negative for the first vector of an unaligned row)
  __device__ __forceinline__ int64_t first(int j) const { return (int64_t)j * VN - shift; }
  __device__ __forceinline__ bool whole(int j) const { return first(j) >= 0 && first(j) + VN <= V; }
  // vector j as floats; places outside the row read -inf
  __device__ __forceinline__ void load(int j, float (&f)[VN]) const {
    const int64_t e = first(j);
    if (e >= 0 && e + VN <= V) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + e);
      const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < VN; ++i) f[i] = static_cast<float>(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i) f[i] = (e + i >= 0 && e + i < V) ? static_cast<float>(p[e + i]) : -INFINITY;
    }
  }
};

// ------------------------------------------------------------------ ordered keys
// (value, position) as one integer: larger value first, then the lower position. 0 = no entry.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 and 0 are one value
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(u64 key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ u64 make_key(float x, uint32_t pos) { return ((u64)ordered(x) << 32) | (uint32_t)~pos; }
__device__ __forceinline__ uint32_t pos_of(u64 key) { return ~(uint32_t)key; }

constexpr uint32_t kAll = 0xffffffffu;

// Descending over the warp's lanes.
__device__ __forceinline__ u64 sort_warp(u64 key, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o; o >>= 1) {
      const u64 other = __shfl_xor_sync(kAll, key, o);
      const bool up = ((lane & o) == 0) == ((lane & size) == 0);  // this lane keeps the larger one
      key = (up == (key > other)) ? key : other;
    }
  return key;
}
// The 32 largest of two descending lists (lane i holds entry i of each), descending.
__device__ __forceinline__ u64 merge_warp(u64 a, u64 b, int lane) {
  const u64 r = __shfl_sync(kAll, b, 31 - lane);
  a = a > r ? a : r;  // the 32 largest, bitonic
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const u64 other = __shfl_xor_sync(kAll, a, o);
    a = (((lane & o) == 0) == (a > other)) ? a : other;
  }
  return a;
}

// ------------------------------------------------------------------ (m, s, u)
struct Stat {
  float m, s, u;  // maximum, Σ e^(z − m), Σ (z − m)·e^(z − m)
};
__device__ __forceinline__ void rescale(Stat& a, float M) {
  const float d = max_nan(a.m - M, kFloor);
  const float f = fast_exp2(d * kLog2e);
  a.u = fmaf(d, a.s, a.u) * f;
  a.s *= f;
  a.m = M;
}
__device__ __forceinline__ void merge(Stat& a, Stat b) {
  const float M = fmaxf(a.m, b.m);
  if (M != -INFINITY) {  // else both hold nothing but masked logits (0) or a NaN
    rescale(a, M);
    rescale(b, M);
  }
  a.s += b.s;
  a.u += b.u;
}

// One thread's share of vectors lo + tid, lo + tid + kGroup, ... < hi; with TOP also its largest logit and the (first)
// vector that holds it.
template <typename T, int kGroup, bool TOP>
__device__ __forceinline__ Stat scan(const Row<T>& z, int lo, int hi, int tid, float& best, int& best_j) {
  constexpr int VN = Row<T>::VN;
  Stat t = {-INFINITY, 0.f, 0.f};
  best = -INFINITY;
  best_j = lo + tid;
  for (int j = lo + tid; j < hi; j += kGroup) {
    float x[VN];
    z.load(j, x);
    float vm = x[0];
#pragma unroll
    for (int i = 1; i < VN; ++i) vm = fmaxf(vm, x[i]);
    if (TOP && vm > best) {
      best = vm;
      best_j = j;
    }
    const float M = fmaxf(t.m, vm);
    if (M > t.m) rescale(t, M);
    const float mb = t.m == -INFINITY ? 0.f : t.m;
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const float d = max_nan(x[i] - mb, kFloor);
      const float e = fast_exp2(d * kLog2e);
      t.s += e;
      t.u = fmaf(e, d, t.u);
    }
  }
  return t;
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

struct FwdArgs {
  const void* z;
  int64_t N, V, ld;
  const int32_t* y;
  int k;
  float *logp, *entropy, *lse;
  int32_t* top_ids;
  float* top_logp;
  int32_t* err;
};

// A row is taken by a group of WARPS warps of each of the CTAs of a cluster
// (cluster size 1: one group per row). WARPS = 1: the warps of a block take
// rows of their own.
template <typename T, int WARPS, bool TOP>
__global__ void __launch_bounds__(kBlock) token_logprob_kernel(const FwdArgs a, int CL) {
  constexpr int kGroup = WARPS * 32;
  constexpr int VN = Row<T>::VN;
  __shared__ Stat part[kBlock / 32];
  __shared__ u64 lists[kBlock / 32][32];
  __shared__ Stat cta_stat;
  __shared__ u64 cta_list[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARPS == 1 ? lane : (int)threadIdx.x;
  const int64_t row = WARPS == 1 ? (int64_t)blockIdx.x * (kBlock / 32) + warp : (int64_t)(blockIdx.x / CL);
  const int rank = WARPS == 1 ? 0 : (int)(blockIdx.x % CL);
  if (WARPS == 1 && row >= a.N) return;
  const Row<T> z(static_cast<const T*>(a.z) + row * a.ld, a.V);
  const int lo = (int)((int64_t)z.nvec * rank / CL), hi = (int)((int64_t)z.nvec * (rank + 1) / CL);

  float best;
  int best_j;
  Stat t = join_warp(scan<T, kGroup, TOP>(z, lo, hi, tid, best, best_j), lane);

  // ---------------------------------------------------------------- the top alternatives
  u64 list = 0;  // lane i: the i-th best of what has been seen
  if (TOP) {
    const u64 mine = lo + tid < hi ? make_key(best, (uint32_t)best_j) : 0;
    u64 s = sort_warp(mine, lane);
    if (WARPS > 1) {
      lists[warp][lane] = s;
      __syncthreads();
#pragma unroll
      for (int w = WARPS / 2; w; w >>= 1) {
        if (warp < w) lists[warp][lane] = merge_warp(lists[warp][lane], lists[warp + w][lane], lane);
        __syncthreads();
      }
      s = lists[0][lane];
      __syncthreads();
    }
    const u64 tau = __shfl_sync(kAll, s, a.k - 1);  // the k-th best of the threads' best
    const float tau_v = tau ? value_of(tau) : -INFINITY;
    uint32_t chosen = __ballot_sync(kAll, mine != 0 && mine >= tau);
    u64 kth = 0;
    while (chosen) {
      const int src = __ffs(chosen) - 1;
      chosen &= chosen - 1;
      const int j0 = lo + tid - lane + src;  // first vector of the chosen thread
      for (int jb = j0; jb < hi; jb += 32 * kGroup) {
        const int j = jb + lane * kGroup;
        float x[VN];
        bool any = false;
        if (j < hi) {
          z.load(j, x);
#pragma unroll
          for (int i = 0; i < VN; ++i) any |= !(x[i] < tau_v);
        }
        if (!__any_sync(kAll, any)) continue;
        const int64_t e0 = z.first(j);
#pragma unroll
        for (int i = 0; i < VN; ++i) {
          const bool in = any && e0 + i >= 0 && e0 + i < z.V && !(x[i] < tau_v);
          u64 key = in ? make_key(x[i], (uint32_t)(e0 + i)) : 0;
          uint32_t c = __ballot_sync(kAll, key > kth);
          while (c) {
            const u64 add = __shfl_sync(kAll, key, __ffs(c) - 1);
            const int at = __popc(__ballot_sync(kAll, list > add));
            const u64 up = __shfl_up_sync(kAll, list, 1);
            list = lane < at ? list : lane == at ? add : up;
            kth = __shfl_sync(kAll, list, a.k - 1);
            if (key == add) key = 0;
            c = __ballot_sync(kAll, key > kth);
          }
        }
      }
    }
  }

  // ---------------------------------------------------------------- join the group's and the cluster's warps
  if (WARPS > 1) {
    if (lane == 0) part[warp] = t;
    if (TOP) lists[warp][lane] = list;
    __syncthreads();
    if (TOP) {
#pragma unroll
      for (int w = WARPS / 2; w; w >>= 1) {
        if (warp < w) lists[warp][lane] = merge_warp(lists[warp][lane], lists[warp + w][lane], lane);
        __syncthreads();
      }
      list = lists[0][lane];
    }
    t = part[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) merge(t, part[w]);
    if (CL > 1) {
      cg::cluster_group cluster = cg::this_cluster();
      if (threadIdx.x == 0) cta_stat = t;
      if (TOP && warp == 0) cta_list[lane] = list;
      cluster.sync();
      if (rank == 0 && warp == 0) {
        for (int r = 1; r < CL; ++r) {
          merge(t, *cluster.map_shared_rank(&cta_stat, r));
          if (TOP) list = merge_warp(list, cluster.map_shared_rank(cta_list, r)[lane], lane);
        }
      }
      cluster.sync();  // the peers' shared memory lives until it has been read
      if (rank != 0) return;
    }
    if (warp != 0) return;
  }

  // ---------------------------------------------------------------- results
  const float log_s = logf(t.s);
  const bool empty = t.m == -INFINITY && t.s == 0.f;  // every logit is -inf: no distribution
  const float lse = t.m + log_s;
  if (lane == 0) {
    const float h = log_s - t.u / t.s;
    a.lse[row] = empty ? -INFINITY : lse;
    a.entropy[row] = empty || h < 0.f ? 0.f : h;
    if (a.y) {
      const int y = a.y[row];
      if (y < 0 || y >= a.V) {
        set_err(a.err, TT_ERR_INVALID_ARG);
        a.logp[row] = __int_as_float(0x7fc00000);
      } else {
        a.logp[row] = empty ? -INFINITY : (static_cast<float>(z.p[y]) - t.m) - log_s;
      }
    }
  }
  if (TOP && lane < a.k) {
    const float v = value_of(list);
    a.top_ids[row * a.k + lane] = list ? (int32_t)pos_of(list) : lane;
    a.top_logp[row * a.k + lane] = empty ? -INFINITY : (v - t.m) - log_s;
  }
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
  const void* z;
  void* dz;
  int64_t N, V, ld;
  const int32_t* y;
  const float *lse, *entropy, *dlogp, *dentropy, *dlse;
  const int32_t* top_ids;
  const float* dtop;
  int k;
  int32_t* err;
};

// lse in fp32 is off by up to |lse|·2^-24, and e^(z − lse) by as much: from here on (6e-5) the row's own maximum and
// sum are taken again. Such are rows that are masked throughout with the type's lowest value.
constexpr float kWideLse = 1024.f;

// Each CTA of a cluster takes one slice of one row. The entries with a term of
// their own (the target, the top alternatives) are formed by one thread each
// after the slice is written, from logits read before it, so that dz may
// overwrite z; a CTA reads no slice but its own.
template <typename T>
__global__ void __launch_bounds__(kBlock) token_logprob_bwd_kernel(const BwdArgs a, int slices) {
  constexpr int VN = Row<T>::VN;
  __shared__ int ids[kTopMax + 1];
  __shared__ float gs[kTopMax + 1];
  __shared__ Stat part[kBlock / 32];
  __shared__ Stat cta_stat;
  const int64_t row = blockIdx.x / slices;
  const int slice = (int)(blockIdx.x % slices);
  const Row<T> z(static_cast<const T*>(a.z) + row * a.ld, a.V);
  T* out = static_cast<T*>(a.dz) + row * a.ld;
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(z.p) & 15);
  const int lo = (int)((int64_t)z.nvec * slice / slices), hi = (int)((int64_t)z.nvec * (slice + 1) / slices);
  const float lse = a.lse[row];
  const bool empty = lse == -INFINITY;  // no distribution: its gradient is 0
  float m = lse, log_s = 0.f;           // log p = (z − m) − log_s
  if (!empty && fabsf(lse) >= kWideLse && fabsf(lse) < INFINITY) {
    float best;
    int best_j;
    Stat t = join_warp(scan<T, kBlock, false>(z, lo, hi, (int)threadIdx.x, best, best_j), threadIdx.x & 31);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
    __syncthreads();
    t = part[0];
    for (int w = 1; w < kBlock / 32; ++w) merge(t, part[w]);
    if (slices > 1) {  // every CTA of the cluster is here: lse is the row's
      cg::cluster_group cluster = cg::this_cluster();
      if (threadIdx.x == 0) cta_stat = t;
      cluster.sync();
      t = *cluster.map_shared_rank(&cta_stat, 0);
      for (int r = 1; r < slices; ++r) merge(t, *cluster.map_shared_rank(&cta_stat, r));
      cluster.sync();
    }
    m = t.m;
    log_s = logf(t.s);
  }
  const float glp = a.dlogp ? a.dlogp[row] : 0.f;
  const float gh = a.dentropy ? a.dentropy[row] : 0.f;
  // entries with a term of their own: place 0 the target, then the alternatives
  if (threadIdx.x <= a.k) {
    int id = -1;
    float g = 0.f;
    if (threadIdx.x == 0) {
      if (a.dlogp) {
        id = a.y[row];
        g = glp;
      }
    } else {
      id = a.top_ids[row * a.k + threadIdx.x - 1];
      g = a.dtop[row * a.k + threadIdx.x - 1];
    }
    if ((threadIdx.x > 0 || a.dlogp) && (id < 0 || id >= a.V)) {
      set_err(a.err, TT_ERR_INVALID_ARG);
      id = -1;
    }
    ids[threadIdx.x] = id;
    gs[threadIdx.x] = g;
  }
  __syncthreads();
  float whole = glp;
  for (int i = 1; i <= a.k; ++i) whole += gs[i];
  if (a.dlse) whole -= a.dlse[row];
  const float b = fmaf(gh, a.dentropy ? a.entropy[row] : 0.f, whole);
  auto grad = [&](float x) {
    const float lp = max_nan((x - m) - log_s, kFloor);
    return -fast_exp2(lp * kLog2e) * fmaf(gh, lp, b);
  };
  float own = 0.f;
  int own_id = -1;
  if (threadIdx.x <= a.k && ids[threadIdx.x] >= 0) {
    const int id = ids[threadIdx.x];
    const int j = (id + z.shift) / VN;
    bool first = j >= lo && j < hi;
    for (int i = 0; i < (int)threadIdx.x; ++i) first = first && ids[i] != id;
    if (first) {
      own_id = id;
      float g = 0.f;
      for (int i = threadIdx.x; i <= a.k; ++i) g += ids[i] == id ? gs[i] : 0.f;
      own = empty ? 0.f : grad(static_cast<float>(z.p[id])) + g;
    }
  }
  __syncthreads();  // the logits of these entries are read
  for (int j = lo + threadIdx.x; j < hi; j += kBlock) {
    float x[VN];
    z.load(j, x);
#pragma unroll
    for (int i = 0; i < VN; ++i) x[i] = empty ? 0.f : grad(x[i]);
    const int64_t e = z.first(j);
    if (same && z.whole(j)) {
      uint4 u;
      T* t = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < VN; ++i) t[i] = static_cast<T>(x[i]);
      *reinterpret_cast<uint4*>(out + e) = u;
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i)
        if (e + i >= 0 && e + i < z.V) out[e + i] = static_cast<T>(x[i]);
    }
  }
  __syncthreads();
  if (own_id >= 0) out[own_id] = static_cast<T>(own);
}

int check_logits(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, size_t* es) {
  if (dtype != TT_DT_BF16 && dtype != TT_DT_F16 && dtype != TT_DT_F32) return TT_ERR_INVALID_ARG;
  *es = dtype == TT_DT_F32 ? 4 : 2;
  if (N < 0 || V < 1 || ld < V || N > INT32_MAX / 64 || V > INT32_MAX / 2) return TT_ERR_INVALID_ARG;
  if (N && (!logits || reinterpret_cast<uintptr_t>(logits) % *es)) return TT_ERR_INVALID_ARG;
  return TT_OK;
}

template <typename T, bool TOP>
int launch_fwd(const FwdArgs& a, cudaStream_t st) {
  token_logprob_kernel<T, 8, TOP><<<(unsigned)a.N, kBlock, 0, st>>>(a, 1);
  return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}
template <typename T>
int launch_bwd(const BwdArgs& a, cudaStream_t st) {
  token_logprob_bwd_kernel<T><<<(unsigned)a.N, kBlock, 0, st>>>(a, 1);
  return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace
}  // namespace tt

using namespace tt;

TT_API int tt_token_logprob(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* targets,
                            int k, float* logp, float* entropy, float* lse, int32_t* top_ids, float* top_logp,
                            int32_t* err, tt_stream_t stream) {
  size_t es;
  const int rc = check_logits(logits, dtype, N, V, ld, &es);
  if (rc) return rc;
  if (k < 0 || k > V) return TT_ERR_INVALID_ARG;
  if (k > kTopMax) return TT_ERR_UNSUPPORTED;
  if (N == 0) return TT_OK;
  if (!entropy || !lse || !err || (targets && !logp) || (k && (!top_ids || !top_logp))) return TT_ERR_INVALID_ARG;
  const FwdArgs a = {logits, N, V, ld, targets, k, logp, entropy, lse, top_ids, top_logp, err};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case TT_DT_BF16: return k ? launch_fwd<__nv_bfloat16, true>(a, st) : launch_fwd<__nv_bfloat16, false>(a, st);
    case TT_DT_F16: return k ? launch_fwd<__half, true>(a, st) : launch_fwd<__half, false>(a, st);
    default: return k ? launch_fwd<float, true>(a, st) : launch_fwd<float, false>(a, st);
  }
}

TT_API int tt_token_logprob_bwd(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const float* lse,
                                const float* entropy, const int32_t* targets, const float* dlogp,
                                const float* dentropy, const float* dlse, const int32_t* top_ids, const float* dtop,
                                int k, void* dlogits, int32_t* err, tt_stream_t stream) {
  size_t es;
  const int rc = check_logits(logits, dtype, N, V, ld, &es);
  if (rc) return rc;
  if (k < 0) return TT_ERR_INVALID_ARG;
  if (k > kTopMax) return TT_ERR_UNSUPPORTED;
  if (N == 0) return TT_OK;
  if (!lse || !dlogits || !err || reinterpret_cast<uintptr_t>(dlogits) % es || (dlogp && !targets) ||
      (dentropy && !entropy) || (k && (!top_ids || !dtop)))
    return TT_ERR_INVALID_ARG;
  const BwdArgs a = {logits, dlogits, N, V, ld, targets, lse, entropy, dlogp, dentropy, dlse, top_ids, dtop, k, err};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case TT_DT_BF16: return launch_bwd<__nv_bfloat16>(a, st);
    case TT_DT_F16: return launch_bwd<__half>(a, st);
    default: return launch_bwd<float>(a, st);
  }
}
