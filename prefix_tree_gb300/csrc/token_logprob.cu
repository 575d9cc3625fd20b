// Log-probability of a given token, entropy and top alternatives of every row
// of logits, and the gradient of any function of them.
//
//   lse = log Σ_v e^{z_v};   logp = z_y − lse;   top: the k largest z (ties to the lower index)
//   H   = lse − Σ_v p_v z_v = log S − U/S,   S = Σ_v e^{d_v},  U = Σ_v d_v e^{d_v},  d_v = z_v − max z
// (S >= 1 and U <= 0: the two terms of H have one sign, nothing cancels).
//
// Forward: one pass over the row. A thread takes 16-byte vectors and folds
// them into (m, s, u) with a running maximum. Over the first part of the row
// it also keeps the vector that holds its largest logit: the k largest logits
// of that part lie with the k threads whose largest (value, position) are its
// k best, since a thread outside them has k better elements elsewhere for each
// of its own. So after that part a lower bound of the row's k-th best is
// known; the elements of the few threads that reach it are read again (from
// the L2 cache) and kept where they reach it, and over the rest of the row
// whatever exceeds it is kept as it passes: one comparison per vector. What
// was kept, a few times k, is sorted at the end.
//
// Backward: dz_v = p_v·(g_lse − G − g_H·(logp_v + H)) + g_logp·[v = y] + Σ_j g_top_j·[v = id_j],
// with G = g_logp + Σ_j g_top_j: one read and one write of the row.
//
// Bound by memory where rows are many and long: 12,669 x 151,936 bf16 (3.85
// GB) in 564 us without alternatives, 580 with 8 (1.02 and 0.99 of the
// measured copy rate), 632 with 20 (issue slots: about 34,000 warp
// instructions a row for the pass, 500 for each alternative); the gradient
// (7.7 GB) in 1125 us. Few or short rows are bound by latency: 4.6 us one row
// in 8 CTAs, 9.3 with 20 alternatives (the joins and the sort); 60,000 rows of
// 1000 in 42 and, with 8, 77 us.
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
constexpr int kMostCtas = 8;   // CTAs to a row: the portable cluster size
// A row's first part, for the bound on its alternatives: one in so many. A smaller part makes the bound on the rest
// looser (candidates kept: k times this), a larger one has more to read again.
constexpr int kFirstPart = 4;
// Threads of a block: a group of WARPS warps, or eight groups of one.
template <int WARPS>
constexpr int kBlockOf = WARPS == 1 ? 256 : 32 * WARPS;
// CTAs to an SM that the registers are held to: 32 warps (with 40 or 48, spills cost more than the warps give).
template <int WARPS>
constexpr int kMinCtas = 1024 / kBlockOf<WARPS>;

typedef unsigned long long u64;

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

// Batches of a thread on their way from memory or in use. (3 and 4 took as long where four warps take a row of 1000 to
// 151,936 logits; three for eight warps are 48 KB, more than there is beside the alternatives' lists.)
constexpr int kDepth = 2;

// Shared memory that a group's vectors pass through: each thread its own places, so no thread waits for another.
template <int WARPS>
struct Ring {
  uint4 at[kDepth][kBatch][WARPS * 32];
};

// One thread's way over vectors lo + tid, lo + tid + kGroup, ... < hi of a row, kBatch at a time, through asynchronous
// copies kDepth − 1 batches ahead.
template <typename T, int WARPS>
struct Scan {
  static constexpr int kGroup = WARPS * 32, kD = kDepth;
  const Row<T>& z;
  Ring<WARPS>& ring;
  const int hi, wlo, whi, tid;
  int j, stage;
  Stat t;
  float best;  // largest logit of the batches taken with TRACK, and the first vector that holds it
  int best_j;

  __device__ __forceinline__ Scan(const Row<T>& z_, Ring<WARPS>& ring_, int lo, int hi_, int tid_)
      : z(z_), ring(ring_), hi(hi_), wlo(z_.whole_lo()), whi(min(hi_, z_.whole_hi())), tid(tid_), j(lo + tid_), stage(0),
        t{-INFINITY, 0.f, 0.f}, best(-INFINITY), best_j(lo + tid_) {
#pragma unroll
    for (int d = 0; d < kD - 1; ++d) fetch(j + d * kBatch * kGroup, d);
  }
  // Starts the batch at vector `at` on its way into `st`.
  __device__ __forceinline__ void fetch(int at, int st) {
    if (at >= wlo && at + (kBatch - 1) * kGroup < whi) {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) copy(at + v * kGroup, st, v);
    } else {  // the row's ends: only a vector that is not whole is waited for
#pragma unroll
      for (int v = 0; v < kBatch; ++v) {
        const int jv = at + v * kGroup;
        if (jv >= wlo && jv < whi) {
          copy(jv, st, v);
        } else {
          uint4 u;
#pragma unroll
          for (int i = 0; i < Row<T>::VN; ++i) reinterpret_cast<T*>(&u)[i] = static_cast<T>(-INFINITY);
          if (jv < hi) u = z.load(jv);
          ring.at[st][v][tid] = u;
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void copy(int jv, int st, int v) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&ring.at[st][v][tid])), "l"(z.p + z.first(jv))
                 : "memory");
  }
  // The batches before vector `end` (all the thread's with end = hi). The lanes of a warp stay together (those past the
  // end take masked logits). With OVER, over(src) is called by the whole warp for each lane src whose batch has a logit
  // above `above`.
  template <bool TRACK, bool OVER, typename F>
  __device__ __forceinline__ void take(int end, float above, F over) {
    const int lane = threadIdx.x & 31;
    while (j - lane < end) {
      const int ahead = stage == 0 ? kD - 1 : stage - 1;
      fetch(j + (kD - 1) * kBatch * kGroup, ahead);
      asm volatile("cp.async.wait_group %0;" ::"n"(kD - 1) : "memory");
      uint4 u[kBatch];
#pragma unroll
      for (int v = 0; v < kBatch; ++v) u[v] = ring.at[stage][v][tid];
      float bm;
      if (TRACK) {
        bm = -INFINITY;
#pragma unroll
        for (int v = 0; v < kBatch; ++v) {
          const float vm = Pairs<T>::max(u[v]);
          if (vm > best) {
            best = vm;
            best_j = j + v * kGroup;
          }
          bm = fmaxf(bm, vm);
        }
      } else {
        static_assert(kBatch == 4, "four vectors");
        bm = Pairs<T>::max(u[0], u[1], u[2], u[3]);
      }
      if (OVER) {
        uint32_t m = __ballot_sync(kAll, bm > above);
        if (m) {
          __syncwarp();  // the lanes' copies are there for the warp
          do {
            over(__ffs(m) - 1);
            m &= m - 1;
          } while (m);
          __syncwarp();
        }
      }
      rescale(t, fmaxf(t.m, bm));
      const float mb = t.m == -INFINITY ? 0.f : t.m;
      const float2 nm = make_float2(-mb, -mb), l2 = make_float2(kLog2e, kLog2e);
      float2 s = make_float2(0.f, 0.f), q = make_float2(0.f, 0.f);
#pragma unroll
      for (int v = 0; v < kBatch; ++v) fold<T, false>(s, q, u[v], nm, l2);
      t.s += s.x + s.y;
      t.u += q.x + q.y;
      j += kBatch * kGroup;
      stage = stage == kD - 1 ? 0 : stage + 1;
    }
  }
  template <bool TRACK>
  __device__ __forceinline__ void take_all() {
    take<TRACK, false>(hi, 0.f, [](int) {});
  }
};

// The sums of a thread's vectors taken again the wide way.
template <typename T, int WARPS>
__device__ __noinline__ Stat wide_sums(const Row<T>& z, int lo, int hi, int tid) {
  Stat t = {-INFINITY, 0.f, 0.f};
  for (int j = lo + tid; j < hi; j += WARPS * 32) {
    const uint4 u = z.load(j);
    rescale(t, fmaxf(t.m, Pairs<T>::max(u)));
    const float mb = t.m == -INFINITY ? 0.f : t.m;
    float2 s = make_float2(0.f, 0.f), q = make_float2(0.f, 0.f);
    fold<T, true>(s, q, u, make_float2(-mb, -mb), make_float2(kLog2e, kLog2e));
    t.s += s.x + s.y;
    t.u += q.x + q.y;
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
  static constexpr int kEntries = 64;                        // most of the warps' best that enter the bound
  static constexpr int kLists = WARPS < 4 ? 4 : 2 * WARPS;   // candidates are sorted 32 at a time
  static constexpr int kRoom = 32 * kLists;                  // candidates kept
  uint32_t bests[WARPS == 1 ? 1 : kEntries];
  uint32_t bound;
  int chosen, found;  // entries of `threads`, and candidates found (possibly more than kRoom)
  uint16_t threads[kGroup];
  u64 keys[kRoom];

  __device__ __forceinline__ void keep(u64 key) {
    const int at = atomicAdd(&found, 1);
    if (at < kRoom) keys[at] = key;
  }
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

// A lower bound of the k-th largest key (value, element) of vectors [lo, hi), 0 if there are fewer than k elements'
// worth; best, best_j: the thread's from a Scan over them. Lists the threads that reach it in sh.threads and clears
// sh.found. Every thread of the group takes part.
//
// A 32-bit key of every thread's best (16-bit types: value and vector, so that ties count by position; fp32: the value
// alone), 0 = none. Of these, the k-th largest of each warp's first few, 2·k or more in all: exact unless one warp
// holds more than its share of the k.
template <typename T, int WARPS>
__device__ __forceinline__ u64 bound_of(TopShared<WARPS>& sh, const Row<T>& z, int lo, int hi, int tid, int k,
                                        float best, int best_j) {
  using S = TopShared<WARPS>;
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
    const int rounds = max(4, (2 * k + WARPS - 1) / WARPS);  // entries of a warp: 64 in all at most
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
  group_sync<WARPS>();
  if (!bound) return 0;
  if (sizeof(T) == 4) return (u64)bound << 32;
  const int j = by_place ? lo + (int)(0xffffu - (bound & 0xffffu)) : z.nvec;  // elements of vector j and before
  return make_key(half_value<T>(bound >> 16), (uint32_t)(z.first(j) + Row<T>::VN - 1));
}

// Keeps the elements that reach tau of the batch that lane src is at. The whole warp takes part, a lane to an element.
template <typename T, int WARPS>
__device__ __forceinline__ void look(TopShared<WARPS>& sh, const Scan<T, WARPS>& scan, int src, u64 tau) {
  constexpr int VN = Row<T>::VN;
  const int lane = threadIdx.x & 31;
  static_assert(kBatch * VN <= 32, "an element to a lane");
  if (lane < kBatch * VN) {
    const int v = lane / VN, i = lane % VN;
    const int e = scan.z.first(scan.j - lane + src + v * (WARPS * 32)) + i;
    const T x = reinterpret_cast<const T*>(&scan.ring.at[scan.stage][v][scan.tid - lane + src])[i];
    const u64 key = make_key(static_cast<float>(x), (uint32_t)e);
    if (key >= tau && e >= 0 && e < scan.z.V) sh.keep(key);
  }
}

// Keeps the elements of vectors [lo, hi) of the listed threads whose keys reach tau.
template <typename T, int WARPS>
__device__ __forceinline__ void gather(TopShared<WARPS>& sh, const Row<T>& z, int lo, int hi, int tid, u64 tau) {
  constexpr int kGroup = WARPS * 32, VN = Row<T>::VN;
  const int per = (hi - lo + kGroup - 1) / kGroup, all = sh.chosen * per;
  const float tau_v = tau ? value_of(tau) : -INFINITY;
  constexpr int kAtOnce = 4;  // loads of a thread under way together
  for (int f0 = tid; f0 < all; f0 += kAtOnce * kGroup) {
    uint4 u[kAtOnce];
    int at[kAtOnce];
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      const int f = f0 + n * kGroup, c = f / per;
      at[n] = f < all ? lo + sh.threads[c] + (f - c * per) * kGroup : hi;
      if (at[n] < hi) u[n] = z.load(at[n]);
    }
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      if (at[n] >= hi) continue;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < VN; ++i) m |= (Pairs<T>::element(u[n], i) >= tau_v) ? 1u << i : 0u;
      while (m) {
        const int i = __ffs(m) - 1, e = z.first(at[n]) + i;
        m &= m - 1;
        const u64 key = make_key(Pairs<T>::element(u[n], i), (uint32_t)e);
        if (key >= tau && e >= 0 && e < z.V) sh.keep(key);
      }
    }
  }
}

// The 32 largest of what was kept (after a group_sync), descending over the lanes of warp 0 and, where there was more
// than one list to sort, in sh.keys.
template <int WARPS>
__device__ __forceinline__ u64 sort_kept(TopShared<WARPS>& sh, int tid) {
  using S = TopShared<WARPS>;
  const int lane = tid & 31, warp = tid >> 5, kept = min(sh.found, S::kRoom);
  u64 list = 0;
  for (int at = 32 * warp; at < kept; at += 32 * WARPS) {
    const u64 more = sort_warp(at + lane < kept ? sh.keys[at + lane] : 0, lane);
    list = at == 32 * warp ? more : merge_warp(list, more, lane);
  }
  if (WARPS > 1 && kept > 32) {
    sh.keys[tid] = list;  // each warp's own 32 places
#pragma unroll
    for (int w = WARPS / 2; w; w >>= 1) {
      __syncthreads();
      if (warp < w) sh.keys[tid] = list = merge_warp(list, sh.keys[tid + 32 * w], lane);
    }
    __syncthreads();
  }
  return list;
}

// The k largest logits of vectors [lo, hi), lane i of warp 0 the i-th, wherever they lie: for rows where more reached
// the bound than there is room for (ascending rows, long ties). The thread's best of the whole slice give a bound that
// only the elements of its threads can reach; while these are still too many, the k-th best of those kept is a higher
// one. Each time at least kRoom − k >= 96 candidates fall away.
template <typename T, int WARPS>
__device__ __noinline__ u64 top_of_slice(TopShared<WARPS>& sh, const Row<T>& z, Ring<WARPS>& ring, int lo, int hi, int tid,
                                         int k) {
  Scan<T, WARPS> scan(z, ring, lo, hi, tid);
  scan.template take_all<true>();
  group_sync<WARPS>();
  u64 tau = bound_of<T, WARPS>(sh, z, lo, hi, tid, k, scan.best, scan.best_j);
  for (;;) {
    gather<T, WARPS>(sh, z, lo, hi, tid, tau);
    group_sync<WARPS>();
    const u64 list = sort_kept<WARPS>(sh, tid);
    if (sh.found <= TopShared<WARPS>::kRoom) return list;
    tau = WARPS == 1 ? __shfl_sync(kAll, list, k - 1) : sh.keys[k - 1];
    group_sync<WARPS>();
    if (tid == 0) sh.found = 0;
    group_sync<WARPS>();
  }
}

// A row is taken by a group of WARPS warps of each of the CTAs of a cluster
// (cluster size 1: one group per row). WARPS = 1: the warps of a block take
// rows of their own.
template <typename T, int WARPS, bool TOP>
__global__ void __launch_bounds__(kBlockOf<WARPS>, kMinCtas<WARPS>) token_logprob_kernel(const FwdArgs a, int CL) {
  constexpr int kGroup = WARPS * 32;
  constexpr int kGroups = kBlockOf<WARPS> / kGroup;
  __shared__ Stat part[WARPS];
  __shared__ Ring<WARPS> rings[kGroups];
  __shared__ TopShared<WARPS> top[TOP ? kGroups : 1];
  __shared__ Stat cta_stat;
  __shared__ u64 cta_list[WARPS > 1 && TOP ? 32 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARPS == 1 ? lane : (int)threadIdx.x;
  const int64_t row = WARPS == 1 ? (int64_t)blockIdx.x * kGroups + warp : (int64_t)(blockIdx.x / CL);
  const int rank = WARPS == 1 ? 0 : (int)(blockIdx.x % CL);
  if (WARPS == 1 && row >= a.N) return;
  Ring<WARPS>& ring = rings[WARPS == 1 ? warp : 0];
  const Row<T> z(static_cast<const T*>(a.z) + row * a.ld, a.V);
  const int lo = (int)((int64_t)z.nvec * rank / CL), hi = (int)((int64_t)z.nvec * (rank + 1) / CL);

  Scan<T, WARPS> scan(z, ring, lo, hi, tid);
  // the target, and after the pass its logit: loads that nothing waits for
  const int y = a.y && rank == 0 && tid == 0 ? a.y[row] : -1;
  if constexpr (TOP) {
    TopShared<WARPS>& sh = top[WARPS == 1 ? warp : 0];
    // the first part: whole rounds of batches
    constexpr int kRound = kBatch * kGroup;
    const int parts = (hi - lo) / kRound;
    const int mid = parts < 2 ? hi : lo + (a.k <= 16 ? (parts + kFirstPart - 1) / kFirstPart : (parts + 1) / 2) * kRound;
    scan.template take<true, false>(mid, 0.f, [](int) {});
    const u64 tau = bound_of<T, WARPS>(sh, z, lo, mid, tid, a.k, scan.best, scan.best_j);
    gather<T, WARPS>(sh, z, lo, mid, tid, tau);
    // (an equal logit further on comes after the k that are known)
    scan.template take<false, true>(hi, tau ? value_of(tau) : -INFINITY, [&](int src) {
      look<T, WARPS>(sh, scan, src, tau);
    });
  } else {
    scan.template take_all<false>();
  }
  const float zy = y >= 0 && y < z.V ? static_cast<float>(z.p[y]) : 0.f;
  Stat t = join_warp(scan.t, lane);
  if (!plain_way_holds<T>(t.m)) t = join_warp(wide_sums<T, WARPS>(z, lo, hi, tid), lane);
  if (WARPS > 1 && lane == 0) part[warp] = t;
  group_sync<WARPS>();
  u64 list = 0;  // lane i of the first warp: the i-th best
  if constexpr (TOP) {
    TopShared<WARPS>& sh = top[WARPS == 1 ? warp : 0];
    list = sh.found <= TopShared<WARPS>::kRoom ? sort_kept<WARPS>(sh, tid)
                                               : top_of_slice<T, WARPS>(sh, z, ring, lo, hi, tid, a.k);
  }
  if constexpr (WARPS > 1) {
    if (CL == 1) {
      if (warp != 0) return;
      t = part[0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) merge(t, part[w]);
    } else if constexpr (WARPS == kMostCtas) {
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
      if (y < 0 || y >= z.V) {
        set_err(a.err, TT_ERR_INVALID_ARG);
        a.logp[row] = __int_as_float(0x7fc00000);
      } else {
        a.logp[row] = empty ? -INFINITY : (zy - t.m) - log_s;
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
__global__ void __launch_bounds__(kBlockOf<WARPS>) token_logprob_bwd_kernel(const BwdArgs a, int CL) {
  constexpr int VN = Row<T>::VN;
  constexpr int kGroup = WARPS * 32;
  constexpr int kGroups = kBlockOf<WARPS> / kGroup;
  __shared__ int all_ids[kGroups][kTopMax + 1];
  __shared__ float all_gs[kGroups][kTopMax + 1];
  __shared__ Stat part[WARPS];
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
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(z.p) & 15);
  const int wlo = z.whole_lo(), whi = min(hi, z.whole_hi());
  // the first vectors, before the loads that wait for one another
  auto plain = [&](int j) { return same && j >= wlo && j + (kBatch - 1) * kGroup < whi; };
  uint4 next[kBatch];
  auto fetch = [&](int j) {
    if (j >= wlo && j + (kBatch - 1) * kGroup < whi) {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) next[v] = z.load_whole(j + v * kGroup);
    } else {
#pragma unroll
      for (int v = 0; v < kBatch; ++v)
        if (j + v * kGroup < hi) next[v] = z.load(j + v * kGroup);
    }
  };
  fetch(lo + tid);
  const float lse = a.lse[row];
  const bool empty = lse == -INFINITY;  // no distribution: its gradient is 0
  float m = lse, log_s = 0.f;           // log p = (z − m) − log_s
  if (!empty && fabsf(lse) >= kWideLse && fabsf(lse) < INFINITY) {
    Stat t = join_warp(wide_sums<T, WARPS>(z, lo, hi, tid), lane);
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
  for (int j = lo + tid; j < hi; j += kBatch * kGroup) {
    uint4 u[kBatch];
#pragma unroll
    for (int v = 0; v < kBatch; ++v) u[v] = next[v];
    fetch(j + kBatch * kGroup);
    if (plain(j)) {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) *reinterpret_cast<uint4*>(out + z.first(j + v * kGroup)) = turn(u[v]);
    } else {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) {
        const int jv = j + v * kGroup;
        if (jv >= hi) continue;
        const uint4 r = turn(u[v]);
        if (same && z.whole(jv))
          *reinterpret_cast<uint4*>(out + z.first(jv)) = r;
        else
          put(jv, r);
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

// grid CTAs of `block` threads in clusters of CL.
template <typename... P, typename... A>
int launch(void (*kernel)(P...), int64_t grid, int block, int CL, cudaStream_t st, A... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CL;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(block);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  (void)cudaGetLastError();
  return cuda_status(e);
}

// How the rows are taken: by a warp each, by a CTA of four or eight warps each, or by 2, 4 or 8 CTAs each. nvec: 16-byte
// vectors of a row. Measured on bf16 rows of 1000 to 151,936 logits, us for the choice and the next one:
//   forward, 8 alternatives   60,000 x 1000: warp 81, four warps 293;   3000 x 32,000: warp 47, four 48;
//                             2000 x 50,000: four 45, eight 49;         12,669 x 151,936: eight 592, four 597;
//                             1000 x 8000 (rows too few for warps): four 9.3, warp 24.5;
//                             10,000 x 8000, 20 alternatives: warp 69, four 80; 6000 x 16,000: four 75, warp 90
//                             1 x 151,936: 8 CTAs 8.0, one 12.5; 76 x 151,936: 2 CTAs 12.2, 4 CTAs 13.6
//   backward                  60,000 x 1000: warp 78, four 134;         10,000 x 8000: warp 63, four 70;
//                             2000 x 50,000: eight 78, four 86;         76 x 151,936: 8 CTAs 8.3, 4 CTAs 9.6
struct Plan {
  int warps, CL;
};
Plan plan_fwd(int64_t N, int64_t nvec, int k) {
  const int64_t sms = sm_count();
  if (N >= 16 * sms && nvec <= (k <= 16 ? 4096 : 1024)) return {1, 1};
  if (N >= 4 * sms && nvec <= 12288) return {nvec <= 256 ? 1 : 4, 1};
  int CL = 1;  // more CTAs only while each finds an SM of its own
  while (CL < kMostCtas && 2 * CL * N <= sms + sms / 16 && nvec >= 2 * (int64_t)CL * 1024) CL *= 2;
  return {8, CL};
}
Plan plan_bwd(int64_t N, int64_t nvec) {
  const int64_t sms = sm_count();
  if (N >= 16 * sms && nvec <= 4096) return {1, 1};
  if (N >= 4 * sms && nvec <= 2048) return {4, 1};
  int CL = 1;
  while (CL < kMostCtas && 2 * CL * N <= 4 * sms && nvec >= 2 * (int64_t)CL * 128) CL *= 2;
  return {8, CL};
}

template <typename T, bool TOP>
int launch_fwd(const FwdArgs& a, cudaStream_t st) {
  const Plan p = plan_fwd(a.N, a.V / Row<T>::VN + 1, a.k);
  if (p.warps == 1) return launch(token_logprob_kernel<T, 1, TOP>, (a.N + 7) / 8, kBlockOf<1>, 1, st, a, 1);
  if (p.warps == 4) return launch(token_logprob_kernel<T, 4, TOP>, a.N, kBlockOf<4>, 1, st, a, 1);
  return launch(token_logprob_kernel<T, 8, TOP>, a.N * p.CL, kBlockOf<8>, p.CL, st, a, p.CL);
}
template <typename T>
int launch_bwd(const BwdArgs& a, cudaStream_t st) {
  const Plan p = plan_bwd(a.N, a.V / Row<T>::VN + 1);
  if (p.warps == 1) return launch(token_logprob_bwd_kernel<T, 1>, (a.N + 7) / 8, kBlockOf<1>, 1, st, a, 1);
  if (p.warps == 4) return launch(token_logprob_bwd_kernel<T, 4>, a.N, kBlockOf<4>, 1, st, a, 1);
  return launch(token_logprob_bwd_kernel<T, 8>, a.N * p.CL, kBlockOf<8>, p.CL, st, a, p.CL);
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
