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
// So the top alternatives cost the pass one comparison per vector; after it a
// lower bound of the k-th best of the threads' best is taken, and only the
// elements of the threads that reach it, little more than k/threads of the
// row, are read again: those that reach the bound are gathered and sorted.
//
// Backward: dz_v = p_v·(g_lse − G − g_H·(logp_v + H)) + g_logp·[v = y] + Σ_j g_top_j·[v = id_j],
// with G = g_logp + Σ_j g_top_j: one read and one write of the row.
#include <cooperative_groups.h>

#include <cuda_fp16.h>

#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace tt {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Offsets from the maximum below this are taken as this: e^-128 is 0 in fp32,
// and 0·d stays 0 for a masked logit (d = -inf).
constexpr float kFloor = -128.f;
constexpr int kTopMax = 32;
constexpr int kBlock = 256;
constexpr int kWarpRow = 512;  // vectors of a row up to which a warp takes a row of its own

typedef unsigned long long u64;

// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ------------------------------------------------------------------ 16-byte vectors of a row
// Element pairs of a 16-byte vector as floats, and its packed maximum.
template <typename T>
struct Pairs;
template <>
struct Pairs<float> {
  static constexpr int N = 2;
  static __device__ __forceinline__ float2 get(const uint4& u, int i) {
    return i ? make_float2(__uint_as_float(u.z), __uint_as_float(u.w))
             : make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    return fmaxf(tc::fmax3f(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z)), __uint_as_float(u.w));
  }
};
template <>
struct Pairs<__nv_bfloat16> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float2 get(const uint4& u, int i) {
    const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <>
struct Pairs<__half> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float2 get(const uint4& u, int i) {
    const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ float max(const uint4& u) {
    const __half2* h = reinterpret_cast<const __half2*>(&u);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};

// The order of a 16-bit type's values in 16 bits (-0 as 0), and back.
__device__ __forceinline__ uint32_t order16(uint32_t bits) {
  return (bits ^ ((bits & 0x8000u) ? 0xffffu : 0x8000u)) & 0xffffu;
}
template <typename T>
__device__ __forceinline__ uint32_t half_order(float x) {
  const T h = static_cast<T>(x + 0.f);  // exact: x is a value of type T
  return order16(*reinterpret_cast<const unsigned short*>(&h));
}
template <typename T>
__device__ __forceinline__ float half_value(uint32_t o) {
  const unsigned short b = (unsigned short)(o ^ ((o & 0x8000u) ? 0x8000u : 0xffffu));
  return static_cast<float>(*reinterpret_cast<const T*>(&b));
}

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
  __device__ __forceinline__ void load(int j, float (&f)[VN]) const {
    const uint4 u = load(j);
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      const float2 x = Pairs<T>::get(u, i);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
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

// Vectors that a thread folds in at once: one rescaling for all of them.
constexpr int kBatch = 4;

// Folds kBatch vectors (bm: their largest element) into t.
template <typename T>
__device__ __forceinline__ void fold(Stat& t, const uint4 (&u)[kBatch], float bm) {
  rescale(t, fmaxf(t.m, bm));
  const float mb = t.m == -INFINITY ? 0.f : t.m;
  const float2 nm = make_float2(-mb, -mb), l2 = make_float2(kLog2e, kLog2e);
  float2 s = make_float2(0.f, 0.f), q = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < kBatch; ++v)
#pragma unroll
    for (int i = 0; i < Pairs<T>::N; ++i) {
      float2 d = __fadd2_rn(Pairs<T>::get(u[v], i), nm);
      d = make_float2(max_nan(d.x, kFloor), max_nan(d.y, kFloor));
      const float2 x = __fmul2_rn(d, l2);
      const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      s = __fadd2_rn(s, e);
      q = __ffma2_rn(e, d, q);
    }
  t.s += s.x + s.y;
  t.u += q.x + q.y;
}

// One thread's share of vectors lo + tid, lo + tid + kGroup, ... < hi; with TOP also its largest logit and the (first)
// vector that holds it.
template <typename T, int kGroup, bool TOP>
__device__ __forceinline__ Stat scan(const Row<T>& z, int lo, int hi, int tid, float& best, int& best_j) {
  Stat t = {-INFINITY, 0.f, 0.f};
  best = -INFINITY;
  best_j = lo + tid;
  const T none = static_cast<T>(-INFINITY);
  uint4 pad;
#pragma unroll
  for (int i = 0; i < Row<T>::VN; ++i) reinterpret_cast<T*>(&pad)[i] = none;
  const int wlo = z.whole_lo(), whi = min(hi, z.whole_hi());
  auto load = [&](int j, uint4(&u)[kBatch]) {
    if (j >= wlo && j + (kBatch - 1) * kGroup < whi) {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) u[v] = z.load_whole(j + v * kGroup);
    } else {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) u[v] = j + v * kGroup < hi ? z.load(j + v * kGroup) : pad;
    }
  };
  uint4 cur[kBatch], next[kBatch];
  int j = lo + tid;
  if (j < hi) load(j, cur);
  while (j < hi) {
    const int jn = j + kBatch * kGroup;
    if (jn < hi) load(jn, next);
    float bm = -INFINITY;
#pragma unroll
    for (int v = 0; v < kBatch; ++v) {
      const float vm = Pairs<T>::max(cur[v]);
      if (TOP && vm > best) {
        best = vm;
        best_j = j + v * kGroup;
      }
      bm = fmaxf(bm, vm);
    }
    fold<T>(t, cur, bm);
#pragma unroll
    for (int v = 0; v < kBatch; ++v) cur[v] = next[v];
    j = jn;
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

// ------------------------------------------------------------------ top alternatives of a slice
// What the threads of a group share while they look for the top alternatives.
template <int WARPS>
struct TopShared {
  static constexpr int kGroup = WARPS * 32;
  static constexpr int kRounds = 8;                   // most of a warp's best that enter the bound
  static constexpr int kRoom = WARPS == 1 ? 64 : 32 * WARPS;  // candidates kept
  uint32_t bests[WARPS == 1 ? 1 : WARPS * kRounds];
  uint32_t bound;
  int chosen, found;  // entries of `threads` and candidates found (possibly more than kRoom)
  uint16_t threads[kGroup];
  u64 keys[kRoom];
};

template <int WARPS>
__device__ __forceinline__ void group_sync() {
  if (WARPS == 1)
    __syncwarp();
  else
    __syncthreads();
}

// Descending over the lanes.
__device__ __forceinline__ uint32_t sort_warp32(uint32_t key, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o; o >>= 1) {
      const uint32_t other = __shfl_xor_sync(kAll, key, o);
      const bool up = ((lane & o) == 0) == ((lane & size) == 0);
      key = up ? max(key, other) : min(key, other);
    }
  return key;
}

// The k largest logits of vectors [lo, hi) as keys, lane i of warp 0 the i-th (0 = none; other warps: unspecified).
// best, best_j: the thread's from scan(). Every thread of the group takes part.
//
// 1. A 32-bit key of every thread's best (16-bit types: value and vector, so that ties count by position; fp32: the
//    value alone), 0 = none. A lower bound of the k-th largest of them: the k-th largest of each warp's first few
//    (exact unless one warp holds more than that many of the k; 4 to a warp for k <= 16, else 8: at least k values).
// 2. The threads that reach the bound; their vectors, spread over the whole group, are read again, and the elements
//    that reach it are gathered.
// 3. More candidates than there is room for (long ties, or rows laid out against the threads): the k-th best of those
//    kept is a higher bound; read again with it. Each time at least kRoom − k >= 32 candidates fall away.
template <typename T, int WARPS>
__device__ __forceinline__ u64 top_of_slice(TopShared<WARPS>& sh, const Row<T>& z, int lo, int hi, int tid, int k,
                                            float best, int best_j) {
  using S = TopShared<WARPS>;
  constexpr int VN = Row<T>::VN;
  const int lane = tid & 31, warp = tid >> 5;
  const bool has = lo + tid < hi, by_place = sizeof(T) == 2 && hi - lo <= 65536;
  uint32_t mine = 0;
  if (has) {
    if (sizeof(T) == 2)
      mine = (half_order<T>(best) << 16) | (by_place ? 0xffffu - (uint32_t)(best_j - lo) : 0xffffu);
    else
      mine = ordered(best);
  }
  if (tid == 0) sh.chosen = sh.found = 0;
  uint32_t bound = 0;
  if constexpr (WARPS == 1) {
    bound = __shfl_sync(kAll, sort_warp32(mine, lane), k - 1);
    __syncwarp();
  } else {
    const int rounds = k <= 4 * WARPS / 2 ? S::kRounds / 2 : S::kRounds;
    uint32_t left = mine;
    for (int r = 0; r < rounds; ++r) {
      const uint32_t top = __reduce_max_sync(kAll, left);
      if (lane == 0) sh.bests[warp * rounds + r] = top;
      if (lane == __ffs(__ballot_sync(kAll, left == top)) - 1) left = 0;
    }
    __syncthreads();
    // each warp ranks its own entries among all
    const uint32_t a = lane < WARPS * rounds ? sh.bests[lane] : 0;
    const uint32_t b = 32 + lane < WARPS * rounds ? sh.bests[32 + lane] : 0;
    for (int r = 0; r < rounds; ++r) {
      const uint32_t v = sh.bests[warp * rounds + r];
      const int above = __popc(__ballot_sync(kAll, a > v)) + __popc(__ballot_sync(kAll, b > v));
      const int reach = __popc(__ballot_sync(kAll, a >= v)) + __popc(__ballot_sync(kAll, b >= v));
      if (above < k && k <= reach && lane == 0) sh.bound = v;  // (equal entries write the same)
    }
    __syncthreads();
    bound = sh.bound;
  }
  if (has && mine >= bound) sh.threads[atomicAdd(&sh.chosen, 1)] = (uint16_t)tid;
  // the same bound on elements
  u64 tau = 0;
  if (bound) {
    if (sizeof(T) == 4) {
      tau = (u64)bound << 32;
    } else {
      const int j = by_place ? lo + (int)(0xffffu - (bound & 0xffffu)) : z.nvec;  // elements of vector j and before
      tau = make_key(half_value<T>(bound >> 16), (uint32_t)(z.first(j) + VN - 1));
    }
  }
  group_sync<WARPS>();
  const int chosen = sh.chosen, per = (hi - lo + S::kGroup - 1) / S::kGroup;
  u64 list;
  for (;;) {
    const float tau_v = tau ? value_of(tau) : -INFINITY;
    for (int f = tid; f < chosen * per; f += S::kGroup) {
      const int c = f / per, j = lo + sh.threads[c] + (f - c * per) * S::kGroup;
      if (j >= hi) continue;
      const uint4 u = z.load(j);
      if (Pairs<T>::max(u) < tau_v) continue;
      const int e0 = z.first(j);
#pragma unroll
      for (int i = 0; i < VN; ++i) {
        const float2 pair = Pairs<T>::get(u, i / 2);
        const u64 key = make_key(i & 1 ? pair.y : pair.x, (uint32_t)(e0 + i));
        if (key >= tau && e0 + i >= 0 && e0 + i < z.V) {
          const int at = atomicAdd(&sh.found, 1);
          if (at < S::kRoom) sh.keys[at] = key;
        }
      }
    }
    group_sync<WARPS>();
    const int found = sh.found, kept = min(found, S::kRoom);
    // sort what was kept: 32 to a warp, then the lists joined
    if constexpr (WARPS == 1) {
      list = sort_warp(lane < kept ? sh.keys[lane] : 0, lane);
      if (kept > 32) list = merge_warp(list, sort_warp(32 + lane < kept ? sh.keys[32 + lane] : 0, lane), lane);
    } else {
      list = 0;
      if (32 * warp < kept) list = sort_warp(tid < kept ? sh.keys[tid] : 0, lane);
      if (kept > 32) {
        sh.keys[tid] = list;  // each warp's own 32 places
#pragma unroll
        for (int w = WARPS / 2; w; w >>= 1) {
          __syncthreads();
          if (warp < w) {
            list = merge_warp(list, sh.keys[tid + 32 * w], lane);
            sh.keys[tid] = list;
          }
        }
        __syncthreads();
      }
    }
    if (found <= S::kRoom) break;
    tau = sh.keys[k - 1];
    if constexpr (WARPS == 1) tau = __shfl_sync(kAll, list, k - 1);
    group_sync<WARPS>();
    if (tid == 0) sh.found = 0;
    group_sync<WARPS>();
  }
  return list;
}

// A row is taken by a group of WARPS warps of each of the CTAs of a cluster
// (cluster size 1: one group per row). WARPS = 1: the warps of a block take
// rows of their own.
template <typename T, int WARPS, bool TOP>
__global__ void __launch_bounds__(kBlock) token_logprob_kernel(const FwdArgs a, int CL) {
  constexpr int kGroup = WARPS * 32;
  constexpr int kGroups = kBlock / kGroup;
  __shared__ Stat part[kBlock / 32];
  __shared__ TopShared<WARPS> top[TOP ? kGroups : 1];
  __shared__ Stat cta_stat;
  __shared__ u64 cta_list[WARPS > 1 && TOP ? 32 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARPS == 1 ? lane : (int)threadIdx.x;
  const int64_t row = WARPS == 1 ? (int64_t)blockIdx.x * kGroups + warp : (int64_t)(blockIdx.x / CL);
  const int rank = WARPS == 1 ? 0 : (int)(blockIdx.x % CL);
  if (WARPS == 1 && row >= a.N) return;
  const Row<T> z(static_cast<const T*>(a.z) + row * a.ld, a.V);
  const int lo = (int)((int64_t)z.nvec * rank / CL), hi = (int)((int64_t)z.nvec * (rank + 1) / CL);

  float best;
  int best_j;
  Stat t = join_warp(scan<T, kGroup, TOP>(z, lo, hi, tid, best, best_j), lane);
  u64 list = 0;  // lane i: the i-th best
  if (WARPS > 1 && lane == 0) part[warp] = t;
  if constexpr (TOP) {
    list = top_of_slice<T, WARPS>(top[WARPS == 1 ? warp : 0], z, lo, hi, tid, a.k, best, best_j);
  } else {
    group_sync<WARPS>();
  }
  if constexpr (WARPS > 1) {
    if (CL == 1) {
      if (warp != 0) return;
      t = part[0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) merge(t, part[w]);
    } else {
      cg::cluster_group cluster = cg::this_cluster();
      if (warp == 0) {
        t = part[0];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) merge(t, part[w]);
        if (lane == 0) cta_stat = t;
        if (TOP) cta_list[lane] = list;
      }
      cluster.sync();
      if (rank == 0) {  // warp r takes CTA r's results; the lists are joined pairwise
        static_assert(WARPS == 8, "a warp for each CTA of a cluster");
        if (warp < CL) {
          if (lane == 0) part[warp] = *cluster.map_shared_rank(&cta_stat, warp);
          if constexpr (TOP) top[0].keys[tid] = list = cluster.map_shared_rank(cta_list, warp)[lane];
        }
        if constexpr (TOP) {
          for (int w = CL / 2; w; w >>= 1) {
            __syncthreads();
            if (warp < w) top[0].keys[tid] = list = merge_warp(list, top[0].keys[tid + 32 * w], lane);
          }
        } else {
          __syncthreads();
        }
        t = part[0];
        for (int w = 1; w < CL; ++w) merge(t, part[w]);
      }
      cluster.sync();  // the peers' shared memory lives until it has been read
      if (rank != 0 || warp != 0) return;
    }
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

// A row is taken by a group of WARPS warps of each of the CTAs of a cluster
// (WARPS = 1: the warps of a block take rows of their own). The entries with a
// term of their own (the target, the top alternatives) are formed by one
// thread each after the slice is written, from logits read before it, so that
// dz may overwrite z; a CTA reads no slice but its own.
template <typename T, int WARPS>
__global__ void __launch_bounds__(kBlock) token_logprob_bwd_kernel(const BwdArgs a, int CL) {
  constexpr int VN = Row<T>::VN;
  constexpr int kGroup = WARPS * 32;
  constexpr int kGroups = kBlock / kGroup;
  __shared__ int all_ids[kGroups][kTopMax + 1];
  __shared__ float all_gs[kGroups][kTopMax + 1];
  __shared__ Stat part[kBlock / 32];
  __shared__ Stat cta_stat;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARPS == 1 ? lane : (int)threadIdx.x;
  const int64_t row = WARPS == 1 ? (int64_t)blockIdx.x * kGroups + warp : (int64_t)(blockIdx.x / CL);
  const int rank = WARPS == 1 ? 0 : (int)(blockIdx.x % CL);
  if (WARPS == 1 && row >= a.N) return;
  int* ids = all_ids[WARPS == 1 ? warp : 0];
  float* gs = all_gs[WARPS == 1 ? warp : 0];
  const Row<T> z(static_cast<const T*>(a.z) + row * a.ld, a.V);
  T* out = static_cast<T*>(a.dz) + row * a.ld;
  const int lo = (int)((int64_t)z.nvec * rank / CL), hi = (int)((int64_t)z.nvec * (rank + 1) / CL);
  const float lse = a.lse[row];
  const bool empty = lse == -INFINITY;  // no distribution: its gradient is 0
  float m = lse, log_s = 0.f;           // log p = (z − m) − log_s
  if (!empty && fabsf(lse) >= kWideLse && fabsf(lse) < INFINITY) {
    float best;
    int best_j;
    Stat t = join_warp(scan<T, kGroup, false>(z, lo, hi, tid, best, best_j), lane);
    if constexpr (WARPS > 1) {
      if (lane == 0) part[warp] = t;
      __syncthreads();
      t = part[0];
      for (int w = 1; w < WARPS; ++w) merge(t, part[w]);
      if (CL > 1) {  // every CTA of the cluster is here: lse is the row's
        cg::cluster_group cluster = cg::this_cluster();
        if (tid == 0) cta_stat = t;
        cluster.sync();
        t = *cluster.map_shared_rank(&cta_stat, 0);
        for (int r = 1; r < CL; ++r) merge(t, *cluster.map_shared_rank(&cta_stat, r));
        cluster.sync();
      }
    }
    m = t.m;
    log_s = logf(t.s);
  }
  const float glp = a.dlogp ? a.dlogp[row] : 0.f;
  const float gh = a.dentropy ? a.dentropy[row] : 0.f;
  // entries with a term of their own: place 0 the target, then the alternatives
  for (int i = tid; i <= a.k; i += kGroup) {
    int id = -1;
    float g = 0.f;
    const bool given = i > 0 || a.dlogp;
    if (given) {
      id = i ? a.top_ids[row * a.k + i - 1] : a.y[row];
      g = i ? a.dtop[row * a.k + i - 1] : glp;
      if (id < 0 || id >= a.V) {
        set_err(a.err, TT_ERR_INVALID_ARG);
        id = -1;
      }
    }
    ids[i] = id;
    gs[i] = g;
  }
  group_sync<WARPS>();
  float whole = glp;
  for (int i = 1; i <= a.k; ++i) whole += gs[i];
  if (a.dlse) whole -= a.dlse[row];
  const float b = fmaf(gh, a.dentropy ? a.entropy[row] : 0.f, whole);
  const float2 nm = make_float2(-m, -m), ns = make_float2(-log_s, -log_s), l2 = make_float2(kLog2e, kLog2e),
               nh = make_float2(-gh, -gh), nb = make_float2(-b, -b);
  auto grad = [&](float2 x) {
    float2 lp = __fadd2_rn(__fadd2_rn(x, nm), ns);
    lp = make_float2(max_nan(lp.x, kFloor), max_nan(lp.y, kFloor));
    const float2 t = __fmul2_rn(lp, l2);
    return __fmul2_rn(make_float2(fast_exp2(t.x), fast_exp2(t.y)), __ffma2_rn(nh, lp, nb));
  };
  // at most two entries to a thread (a warp has 32 threads for up to 33)
  float own[2];
  int own_id[2] = {-1, -1};
#pragma unroll
  for (int q = 0; q < (WARPS == 1 ? 2 : 1); ++q) {
    const int i = tid + q * kGroup;
    if (i > a.k || ids[i] < 0) continue;
    const int id = ids[i], j = (id + z.shift) / VN;
    bool first = j >= lo && j < hi;
    for (int o = 0; o < i; ++o) first = first && ids[o] != id;
    if (!first) continue;
    own_id[q] = id;
    float g = 0.f;
    for (int o = i; o <= a.k; ++o) g += ids[o] == id ? gs[o] : 0.f;
    const float x = static_cast<float>(z.p[id]);
    own[q] = empty ? 0.f : grad(make_float2(x, x)).x + g;
  }
  group_sync<WARPS>();  // the logits of these entries are read

  auto put = [&](int j, const uint4& u) {  // vector j, element by element where it is not whole
    const int e = z.first(j);
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < VN; ++i)
      if (e + i >= 0 && e + i < z.V) out[e + i] = t[i];
  };
  auto turn = [&](const uint4& u) {
    uint4 r;
    T* t = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      const float2 g = empty ? make_float2(0.f, 0.f) : grad(Pairs<T>::get(u, i));
      t[2 * i] = static_cast<T>(g.x);
      t[2 * i + 1] = static_cast<T>(g.y);
    }
    return r;
  };
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(z.p) & 15);
  const int wlo = z.whole_lo(), whi = min(hi, z.whole_hi());
  for (int j = lo + tid; j < hi; j += kBatch * kGroup) {
    if (same && j >= wlo && j + (kBatch - 1) * kGroup < whi) {
      uint4 u[kBatch];
#pragma unroll
      for (int v = 0; v < kBatch; ++v) u[v] = z.load_whole(j + v * kGroup);
#pragma unroll
      for (int v = 0; v < kBatch; ++v) *reinterpret_cast<uint4*>(out + z.first(j + v * kGroup)) = turn(u[v]);
    } else {
      for (int v = 0; v < kBatch && j + v * kGroup < hi; ++v) {
        const int jj = j + v * kGroup;
        const uint4 r = turn(z.load(jj));
        if (same && z.whole(jj))
          *reinterpret_cast<uint4*>(out + z.first(jj)) = r;
        else
          put(jj, r);
      }
    }
  }
  group_sync<WARPS>();
#pragma unroll
  for (int q = 0; q < (WARPS == 1 ? 2 : 1); ++q)
    if (own_id[q] >= 0) out[own_id[q]] = static_cast<T>(own[q]);
}

int check_logits(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, size_t* es) {
  if (dtype != TT_DT_BF16 && dtype != TT_DT_F16 && dtype != TT_DT_F32) return TT_ERR_INVALID_ARG;
  *es = dtype == TT_DT_F32 ? 4 : 2;
  if (N < 0 || V < 1 || ld < V || N > INT32_MAX / 64 || V > INT32_MAX / 2) return TT_ERR_INVALID_ARG;
  if (N && (!logits || reinterpret_cast<uintptr_t>(logits) % *es)) return TT_ERR_INVALID_ARG;
  return TT_OK;
}

// grid CTAs in clusters of CL.
template <typename... P, typename... A>
int launch(void (*kernel)(P...), int64_t grid, int CL, cudaStream_t st, A... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CL;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kBlock);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  (void)cudaGetLastError();
  return cuda_status(e);
}

// CTAs to a row: as many (a power of two up to 8) as leave each at least `least` vectors a thread while the rows
// alone do not fill the GPU's SMs twice.
int ctas_per_row(int64_t N, int64_t nvec, int least) {
  int CL = 1;
  while (CL < 8 && 2 * CL * N <= 2 * (int64_t)sm_count() && nvec >= 2 * (int64_t)CL * kBlock * least) CL *= 2;
  return CL;
}

template <typename T, bool TOP>
int launch_fwd(const FwdArgs& a, cudaStream_t st) {
  const int64_t nvec = a.V / Row<T>::VN + 1;
  if (nvec <= kWarpRow && a.N >= 4 * (int64_t)sm_count())
    return launch(token_logprob_kernel<T, 1, TOP>, (a.N + kBlock / 32 - 1) / (kBlock / 32), 1, st, a, 1);
  const int CL = ctas_per_row(a.N, nvec, 1);
  return launch(token_logprob_kernel<T, kBlock / 32, TOP>, a.N * CL, CL, st, a, CL);
}
template <typename T>
int launch_bwd(const BwdArgs& a, cudaStream_t st) {
  const int64_t nvec = a.V / Row<T>::VN + 1;
  if (nvec <= kWarpRow && a.N >= 4 * (int64_t)sm_count())
    return launch(token_logprob_bwd_kernel<T, 1>, (a.N + kBlock / 32 - 1) / (kBlock / 32), 1, st, a, 1);
  const int CL = ctas_per_row(a.N, nvec, 1);
  return launch(token_logprob_bwd_kernel<T, kBlock / 32>, a.N * CL, CL, st, a, CL);
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
