// Attention of the next token of every running rollout of a tree.
//
//   O_b = Σ_{segments s that list query b} Σ_{k in s} softmax(scale·q_b·k)·v_k,   LSE_b likewise
//
// The keys of a prompt or a common turn are shared by all rollouts below it:
// they lie once in the pool and are read once for all of their queries, where
// attention sequence by sequence would read them again for each. The rows of a
// segment's product are its queries times the query heads of a key head.
//
// Work is counted in blocks of 128 keys of one key head against one tile of
// rows. All blocks of the step, in the order segment, head, tile, block, are
// cut into equal runs, one for each CTA (one CTA to an SM): a CTA may end one
// tile's keys, take others whole and begin another's. It leaves for each tile
// that it met the unnormalised sums, the maxima and the sums of weights of
// its rows (fp32); a second kernel joins the parts of every query and head in
// a fixed order. With row_base(tile) + 128·CTA as the place of a part, the
// parts of different tiles and CTAs cannot meet: along the runs one of the two
// grows at every step, by at least the rows that the part before takes.
#include "tc_common.cuh"

#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace tt {
namespace {

using namespace tc;

constexpr int64_t kPlanMagic = 0x7474646563706c31LL;  // "ttdecpl1"
constexpr int kKeys = 128;       // keys of a block
constexpr int kMostRows = 128;   // rows of a tile at most
constexpr int kMostCtas = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Plan: header, first segment of every CTA, and two int4 for each segment that has keys and queries:
// {first row of the pool, keys, first query, queries}, {blocks before it, tiles of a head, rows of a tile, partial rows
// before it}.
struct PlanHeader {
  int64_t magic;
  int32_t S, B, Hq, Hkv, d, ctas, valid, code;  // code: the error where valid = 0
  int64_t rows, pairs;
  int32_t blocks, quota, segments;
};
constexpr size_t kPlanCtas = 128, kPlanSegs = kPlanCtas + sizeof(int32_t) * kMostCtas;
static_assert(sizeof(PlanHeader) <= kPlanCtas, "header");

struct PlanArgs {
  const int32_t *kv_begin, *kv_len, *q_begin, *q_end;
  int S, B, Hq, Hkv, d, ctas;
  int64_t rows, pairs;
  void* plan;
  int32_t* err;
};

constexpr int kPlanThreads = 1024;

struct Count {
  int64_t blocks, rows;
  int n;
};
__device__ __forceinline__ Count operator+(Count a, Count b) { return {a.blocks + b.blocks, a.rows + b.rows, a.n + b.n}; }

// Exclusive sums over the block's threads, and the total.
__device__ __forceinline__ Count scan_block(Count x, Count* room, Count& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Count in = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Count y = {__shfl_up_sync(~0u, in.blocks, o), __shfl_up_sync(~0u, in.rows, o), __shfl_up_sync(~0u, in.n, o)};
    if (lane >= o) in = in + y;
  }
  if (lane == 31) room[warp] = in;
  __syncthreads();
  Count before = {0, 0, 0};
  total = {0, 0, 0};
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w == warp) before = total;
    total = total + room[w];
  }
  __syncthreads();
  return {before.blocks + in.blocks - x.blocks, before.rows + in.rows - x.rows, before.n + in.n - x.n};
}

// One CTA: two passes over the segments, the first for the totals.
__global__ void __launch_bounds__(kPlanThreads) decode_plan_kernel(const PlanArgs a) {
  __shared__ Count room[kPlanThreads / 32];
  __shared__ int code;
  PlanHeader* hdr = static_cast<PlanHeader*>(a.plan);
  int32_t* cta_seg = reinterpret_cast<int32_t*>(static_cast<char*>(a.plan) + kPlanCtas);
  int4* segs = reinterpret_cast<int4*>(static_cast<char*>(a.plan) + kPlanSegs);
  if (threadIdx.x == 0) code = 0;
  __syncthreads();
  const int G = a.Hq / a.Hkv;
  int quota = 1;
  Count sum = {0, 0, 0};
  for (int pass = 0; pass < 2; ++pass) {
    sum = {0, 0, 0};
    for (int s0 = 0; s0 < a.S; s0 += kPlanThreads) {
      const int s = s0 + (int)threadIdx.x;
      int kb = 0, n = 0, q0 = 0, q1 = 0;
      if (s < a.S) {
        kb = a.kv_begin[s], n = a.kv_len[s], q0 = a.q_begin[s], q1 = a.q_end[s];
        if (kb < 0 || n < 0 || (int64_t)kb + n > a.rows || q0 < 0 || q1 < q0 || q1 > a.B) {
          atomicCAS(&code, 0, TT_ERR_INVALID_ARG);
          n = 0;
        }
      }
      Count c = {0, 0, 0};
      const int rows = (q1 - q0) * G, tile_rows = 16;
      const int tiles = (rows + tile_rows - 1) / tile_rows;
      if (n > 0 && rows > 0) c = {(int64_t)((n + kKeys - 1) / kKeys) * tiles * a.Hkv, (int64_t)rows * a.Hkv, 1};
      Count total;
      const Count at = sum + scan_block(c, room, total);
      if (pass == 1 && c.n) {
        segs[2 * at.n] = make_int4(kb, n, q0, q1 - q0);
        segs[2 * at.n + 1] = make_int4((int)at.blocks, tiles, tile_rows, (int)at.rows);
        // the CTAs whose run begins in it
        for (int64_t r = (at.blocks + quota - 1) / quota; r * quota < at.blocks + c.blocks; ++r) cta_seg[r] = at.n;
      }
      sum = sum + total;
    }
    if (pass == 0) {
      if (threadIdx.x == 0 && sum.rows > a.pairs * a.Hq) atomicCAS(&code, 0, TT_ERR_WORKSPACE);
      if (threadIdx.x == 0 && sum.blocks > INT32_MAX / 2) atomicCAS(&code, 0, TT_ERR_UNSUPPORTED);
      __syncthreads();
      if (code) break;
      quota = (int)((sum.blocks + a.ctas - 1) / a.ctas);
      if (quota < 1) quota = 1;
    }
  }
  if (threadIdx.x == 0) {
    *hdr = {kPlanMagic, a.S, a.B, a.Hq, a.Hkv, a.d, a.ctas, code == 0, code, a.rows, a.pairs, (int)sum.blocks, quota, sum.n};
    if (code) set_err(a.err, code);
  }
}

struct DecodeArgs {
  const void* plan;
  const void* q;
  int64_t q_ld;
  int B, Hq, Hkv, S, ctas;
  int64_t rows, pairs;
  float scale_log2;
  float* part_o;   // [parts' rows][D]
  float2* part_ml; // [parts' rows] maximum (log2 units) and sum of weights
  void* o;
  float* lse;
  int32_t* err;
};

// 0 where the plan is one of this call's sizes; sets err otherwise.
__device__ __forceinline__ int plan_error(const DecodeArgs& a, int D) {
  const PlanHeader* h = static_cast<const PlanHeader*>(a.plan);
  if (h->magic != kPlanMagic || h->S != a.S || h->B != a.B || h->Hq != a.Hq || h->Hkv != a.Hkv || h->d != D ||
      h->ctas != a.ctas || h->rows != a.rows || h->pairs != a.pairs)
    return TT_ERR_INVALID_ARG;
  return h->valid ? 0 : h->code;
}

// A run's way over its blocks: segment, head, tile, block.
struct Walk {
  const int4* segs;
  int Hkv, G;
  int seg, h, tile, blk;            // where it is
  int kv, len, q0, rows, nb;        // the segment's first key row, keys, first query, rows of a head, blocks of a tile
  int tiles, tile_rows, row_base;
  __device__ __forceinline__ void load() {
    const int4 x = segs[2 * seg], y = segs[2 * seg + 1];
    kv = x.x, len = x.y, q0 = x.z, rows = x.w * G, nb = (len + kKeys - 1) / kKeys;
    tiles = y.y, tile_rows = y.z, row_base = y.w;
  }
  __device__ __forceinline__ Walk(const int4* segs_, int Hkv_, int G_, int first_seg, int w) : segs(segs_), Hkv(Hkv_), G(G_) {
    seg = first_seg;
    load();
    const int at = w - segs[2 * seg + 1].x, unit = at / nb;
    blk = at - unit * nb;
    h = unit / tiles;
    tile = unit - h * tiles;
  }
  // to the next block; `more`: there is one in this run
  __device__ __forceinline__ void next(bool more) {
    if (++blk < nb) return;
    blk = 0;
    if (++tile < tiles) return;
    tile = 0;
    if (++h < Hkv) return;
    h = 0;
    ++seg;
    if (more) load();
  }
  // place of row 0 of the current tile among the partial rows, for CTA c
  __device__ __forceinline__ int64_t part_row(int c) const {
    return (int64_t)row_base + (int64_t)h * rows + tile * tile_rows + (int64_t)c * kMostRows;
  }
};

// ------------------------------------------------------------------ warp-level products of 16 rows
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16(lo, hi);
  }
}

constexpr int kWarps = 8;                  // that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 3;                 // K tiles and V tiles in shared memory, each

template <int D>
struct Smem {
  static constexpr uint32_t kBox = kKeys * 128;            // 64 columns of a block's keys, 128-byte swizzle
  static constexpr uint32_t kTile = (D / 64) * kBox;
  static constexpr uint32_t k0 = 0;
  static constexpr uint32_t v0 = kStages * kTile;
  static constexpr uint32_t kPLd = kKeys * 2 + 16;         // bytes of a row of weights: rows fall in different banks
  static constexpr uint32_t p = v0 + kStages * kTile;
  static constexpr uint32_t max = p + 16 * kPLd;           // [kWarps][16] f32
  static constexpr uint32_t sum = max + kWarps * 16 * 4;   // [kWarps][16] f32
  static constexpr uint32_t row_max = sum + kWarps * 16 * 4;  // [16] f32
  static constexpr uint32_t bars = row_max + 16 * 4;
  static constexpr uint32_t abort = bars + 4 * kStages * 8;
  static constexpr uint32_t total = abort + 16 + 1024;     // + slack for the alignment to 1024 bytes
};
constexpr int K_FULL = 0, V_FULL = kStages, K_EMPTY = 2 * kStages, V_EMPTY = 3 * kStages;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecodeArgs a) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::bars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::abort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PlanHeader* hdr = static_cast<const PlanHeader*>(a.plan);
  if (const int e = plan_error(a, D)) {
    if (threadIdx.x == 0) set_err(a.err, e);
    return;
  }
  const int c = blockIdx.x;
  const int64_t w0 = (int64_t)c * hdr->quota, w1 = min((int64_t)hdr->blocks, w0 + hdr->quota);
  if (w0 >= w1) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar[K_FULL + i], 1);
      mbar_init(&bar[V_FULL + i], 1);
      mbar_init(&bar[K_EMPTY + i], kWarps);
      mbar_init(&bar[V_EMPTY + i], kWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int n = (int)(w1 - w0), G = a.Hq / a.Hkv;
  const int4* segs = reinterpret_cast<const int4*>(static_cast<const char*>(a.plan) + kPlanSegs);
  Walk at(segs, a.Hkv, G, reinterpret_cast<const int32_t*>(static_cast<const char*>(a.plan) + kPlanCtas)[c], (int)w0);

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer: lane 0 the K tiles, lane 1 the V tiles
    if (lane < 2) {
      const CUtensorMap* map = lane ? &tmV : &tmK;
      const int full = lane ? V_FULL : K_FULL, empty = lane ? V_EMPTY : K_EMPTY;
      uint8_t* dst = sm + (lane ? L::v0 : L::k0);
      prefetch_tmap(map);
      int i = 0;
      for (; i < n; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !mbar_wait(&bar[empty + st], (i / kStages - 1) & 1, abort_flag, 50 + lane)) break;
        mbar_expect_tx(&bar[full + st], L::kTile);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_2d(dst + st * L::kTile + x * L::kBox, map, &bar[full + st], at.h * D + x * 64, at.kv + at.blk * kKeys);
        at.next(i + 1 < n);
      }
      // every copy issued has landed before the CTA may leave
      for (int j = i - 1; j >= 0 && j >= i - kStages; --j) mbar_drain(&bar[full + j % kStages], (j / kStages) & 1, abort_flag);
    }
  } else {
    // ------------------------------------------------------------ 16 rows against the blocks, all warps on every block
    constexpr int kCols = D / kWarps;     // columns of O of a warp
    constexpr int kOut = kCols / 8;
    const int r0 = lane >> 2, cc = (lane & 3) * 2;
    const int mi = lane >> 3, mr = lane & 7;
    uint32_t qa[D / 16][4];
    float o[kOut][4], m[2], l[2];
    float* smax = reinterpret_cast<float*>(sm + L::max);
    float* ssum = reinterpret_cast<float*>(sm + L::sum);
    float* srow = reinterpret_cast<float*>(sm + L::row_max);
    const uint32_t pbase = smem_u32(sm + L::p);
    for (int i = 0; i < n; ++i) {
      const int st = i % kStages;
      const uint32_t par = (i / kStages) & 1;
      const int tile_n = min(at.tile_rows, at.rows - at.tile * at.tile_rows);  // rows of this tile
      if (i == 0 || at.blk == 0) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = r0 + 8 * half, rr = at.tile * at.tile_rows + r;
          const T* q = static_cast<const T*>(a.q) + (int64_t)(at.q0 + rr / G) * a.q_ld + (int64_t)(at.h * G + rr % G) * D + cc;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            qa[k][half] = r < tile_n ? *reinterpret_cast<const uint32_t*>(q + k * 16) : 0u;
            qa[k][half + 2] = r < tile_n ? *reinterpret_cast<const uint32_t*>(q + k * 16 + 8) : 0u;
          }
          m[half] = -INFINITY;
          l[half] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kOut; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
      }
      // S of this warp's 16 keys
      float s[2][4] = {};
      mbar_wait(&bar[K_FULL + st], par, abort_flag, 52);
      {
        const uint32_t kt = smem_u32(sm + L::k0 + st * L::kTile);
        const int key = warp * 16 + (mi >> 1) * 8 + mr;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int unit = (k & 3) * 2 + (mi & 1);  // 16 bytes of the row within its box
          uint32_t b[4];
          ldsm4(b, kt + (k >> 2) * L::kBox + key * 128 + ((unit ^ (key & 7)) << 4));
          mma16816<T>(s[0], qa[k], b[0], b[1]);
          mma16816<T>(s[1], qa[k], b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[K_EMPTY + st]);
      const int valid = at.len - at.blk * kKeys;  // keys of the segment in this block, possibly more than there are
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = warp * 16 + t * 8 + cc + (e & 1);
          s[t][e] = key < valid ? s[t][e] * a.scale_log2 : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], s[t][e]);
        }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        mx[half] = fmaxf(mx[half], __shfl_xor_sync(~0u, mx[half], 1));
        mx[half] = fmaxf(mx[half], __shfl_xor_sync(~0u, mx[half], 2));
        if ((lane & 3) == 0) smax[warp * 16 + r0 + 8 * half] = mx[half];
      }
      named_barrier(1, 32 * kWarps);  // the maxima are there; the weights of the block before are used
      float f[2], mu[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x = m[half];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x = fmaxf(x, smax[w * 16 + r0 + 8 * half]);
        mu[half] = x == -INFINITY ? 0.f : x;
        f[half] = fast_exp2(m[half] - mu[half]);
        m[half] = x;
        l[half] *= f[half];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[t][e] = fast_exp2(s[t][e] - mu[e >> 1]);
          l[e >> 1] += s[t][e];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
          *reinterpret_cast<uint32_t*>(sm + L::p + (r0 + 8 * half) * L::kPLd + (warp * 16 + t * 8 + cc) * 2) =
              pack2<T>(s[t][2 * half], s[t][2 * half + 1]);
      }
#pragma unroll
      for (int t = 0; t < kOut; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] *= f[e >> 1];
      mbar_wait(&bar[V_FULL + st], par, abort_flag, 53);
      if (valid < kKeys) {
        // rows behind the segment's end are another segment's, or not yet written: a weight of 0 times what lies there
        // must be 0
        for (int e = (int)threadIdx.x; e < (kKeys - valid) * (D / 8); e += 32 * kWarps) {
          const int key = valid + e / (D / 8), u = e % (D / 8);
          *reinterpret_cast<uint4*>(sm + L::v0 + st * L::kTile + (u >> 3) * L::kBox + key * 128 + ((u & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into this stage
      }
      named_barrier(1, 32 * kWarps);  // the weights are there
      {
        const uint32_t vt = smem_u32(sm + L::v0 + st * L::kTile);
        const uint32_t pt = pbase + ((mi & 1) * 8 + mr) * L::kPLd + (mi >> 1) * 16;
        if constexpr (kOut == 2) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k) {
            const int key = k * 16 + (mi & 1) * 8 + mr, unit = warp * 2 + (mi >> 1);  // 8 columns
            uint32_t pa[4], b[4];
            ldsm4(pa, pt + k * 32);
            ldsm4t(b, vt + (unit >> 3) * L::kBox + key * 128 + (((unit & 7) ^ (key & 7)) << 4));
            mma16816<T>(o[0], pa, b[0], b[1]);
            mma16816<T>(o[1], pa, b[2], b[3]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kKeys / 32; ++k) {
            const int key = k * 32 + mi * 8 + mr;
            uint32_t pa[4], pb[4], b[4];
            ldsm4(pa, pt + k * 64);
            ldsm4(pb, pt + k * 64 + 32);
            ldsm4t(b, vt + key * 128 + ((warp ^ (key & 7)) << 4));
            mma16816<T>(o[0], pa, b[0], b[1]);
            mma16816<T>(o[0], pb, b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[V_EMPTY + st]);
      if (i + 1 == n || at.blk + 1 == at.nb) {
        // the tile's part: every warp its columns of the sums, the first 16 threads maxima and sums of weights
        const int64_t row = at.part_row(c);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = r0 + 8 * half;
          l[half] += __shfl_xor_sync(~0u, l[half], 1);
          l[half] += __shfl_xor_sync(~0u, l[half], 2);
          if ((lane & 3) == 0) {
            ssum[warp * 16 + r] = l[half];
            if (warp == 0) srow[r] = m[half];
          }
          if (r < tile_n)
#pragma unroll
            for (int t = 0; t < kOut; ++t)
              *reinterpret_cast<float2*>(a.part_o + (row + r) * D + warp * kCols + t * 8 + cc) =
                  make_float2(o[t][2 * half], o[t][2 * half + 1]);
        }
        named_barrier(1, 32 * kWarps);
        if (threadIdx.x < 16 && (int)threadIdx.x < tile_n) {
          float x = 0.f;
          for (int w = 0; w < kWarps; ++w) x += ssum[w * 16 + threadIdx.x];
          a.part_ml[row + threadIdx.x] = make_float2(srow[threadIdx.x], x);
        }
      }
      at.next(i + 1 < n);
    }
  }
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) set_err(a.err, TT_ERR_TIMEOUT);
}

// Joins the parts of a query and a head (a warp each): M = max m, O = Σ 2^(m − M)·O_part / Σ 2^(m − M)·l. The segments
// that list the query are found by going over all of them, a chunk at a time, in order.
constexpr int kJoinWarps = 8, kJoinChunk = 32 * kJoinWarps, kJoinParts = 64;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) decode_join_kernel(const DecodeArgs a) {
  __shared__ int list[kJoinChunk], counts[kJoinWarps];
  __shared__ int rows[kJoinWarps][kJoinParts];
  __shared__ float weights[kJoinWarps][kJoinParts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (plan_error(a, D)) return;
  const PlanHeader* hdr = static_cast<const PlanHeader*>(a.plan);
  const int4* segs = reinterpret_cast<const int4*>(static_cast<const char*>(a.plan) + kPlanSegs);
  const int b = blockIdx.x, hq = blockIdx.y * kJoinWarps + warp, G = a.Hq / a.Hkv, h = hq / G, quota = hdr->quota;
  constexpr int kE = D / 32;  // columns of a lane
  float M = -INFINITY, Ls = 0.f, acc[kE] = {};
  // takes the n parts whose rows are listed
  auto take = [&](int n) {
    __syncwarp();
    float mx = M;
    float2 ml[kJoinParts / 32];
#pragma unroll
    for (int u = 0; u < kJoinParts / 32; ++u) {
      const int e = lane + 32 * u;
      ml[u] = e < n ? a.part_ml[rows[warp][e]] : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, ml[u].x);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, s));
    const float mu = mx == -INFINITY ? 0.f : mx, f = fast_exp2(M - mu);
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < kJoinParts / 32; ++u) {
      const float w = fast_exp2(ml[u].x - mu);
      weights[warp][lane + 32 * u] = w;
      sum += w * ml[u].y;
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(~0u, sum, s);
    Ls = Ls * f + sum;
    M = mx;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] *= f;
    __syncwarp();
#pragma unroll 4
    for (int e = 0; e < n; ++e) {
      const float w = weights[warp][e];
      const float* p = a.part_o + (int64_t)rows[warp][e] * D + lane * kE;
      if constexpr (kE == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        acc[0] += w * x.x, acc[1] += w * x.y, acc[2] += w * x.z, acc[3] += w * x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        acc[0] += w * x.x, acc[1] += w * x.y;
      }
    }
    __syncwarp();
  };
  int kept = 0;
  for (int s0 = 0; s0 < hdr->segments; s0 += kJoinChunk) {
    // the chunk's segments with this query, in order
    const int s = s0 + (int)threadIdx.x;
    bool on = false;
    if (s < hdr->segments) {
      const int4 x = segs[2 * s];
      on = b >= x.z && b < x.z + x.w;
    }
    const uint32_t ballot = __ballot_sync(~0u, on);
    if (lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int before = 0, found = 0;
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w == warp) before = found;
      found += counts[w];
    }
    if (on) list[before + __popc(ballot & ((1u << lane) - 1))] = s;
    __syncthreads();
    if (hq < a.Hq)
      for (int e = 0; e < found; ++e) {
        const int4 x = segs[2 * list[e]], y = segs[2 * list[e] + 1];
        const int nb = (x.y + kKeys - 1) / kKeys, r = (b - x.z) * G + (hq - h * G), tile = r / y.z;
        const int first = y.x + (h * y.y + tile) * nb;  // the tile's first block
        const int c0 = first / quota, c1 = (first + nb - 1) / quota;
        for (int c = c0; c <= c1; c += 32) {
          if (kept + 32 > kJoinParts) {
            take(kept);
            kept = 0;
          }
          if (c + lane <= c1) rows[warp][kept + lane] = y.w + h * x.w * G + r + (c + lane) * kMostRows;
          kept += min(32, c1 - c + 1);
        }
      }
    __syncthreads();
  }
  if (hq >= a.Hq) return;
  take(kept);
  const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
  T* o = static_cast<T*>(a.o) + ((int64_t)b * a.Hq + hq) * D + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) a.lse[(int64_t)hq * a.B + b] = Ls > 0.f ? (M + __log2f(Ls)) * kLn2 : -INFINITY;
}

int check_sizes(int32_t S, int32_t B, int64_t rows, int64_t pairs, int Hq, int Hkv, int d) {
  if (S < 0 || B < 0 || rows < 0 || pairs < 0 || Hq < 1 || Hkv < 1) return TT_ERR_INVALID_ARG;
  if (rows > INT32_MAX / 2 || S > (1 << 24)) return TT_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hq % Hkv || Hq > 1024 || B > (1 << 20)) return TT_ERR_UNSUPPORTED;
  if (pairs > (INT32_MAX / 2) / Hq) return TT_ERR_INVALID_ARG;
  return TT_OK;
}
int ctas() { return std::min(sm_count(), kMostCtas); }
int64_t part_rows(int64_t pairs, int Hq) { return pairs * Hq + (int64_t)kMostCtas * kMostRows; }

template <typename T, int D>
int launch_decode(const DecodeArgs& a, const void* k, const void* v, int64_t kv_ld, cudaStream_t st) {
  const uint64_t rows = std::max<int64_t>(a.rows, 1);
  CUtensorMap mk, mv;
  if (!make_tmap_bf16_ld(&mk, k, (uint64_t)a.Hkv * D, rows, kv_ld, kKeys) ||
      !make_tmap_bf16_ld(&mv, v, (uint64_t)a.Hkv * D, rows, kv_ld, kKeys))
    return TT_ERR_CUDA;
  const int smem = (int)Smem<D>::total;
  if (!smem_attr_set<decode_kernel<T, D>>(smem)) return TT_ERR_CUDA;
  decode_kernel<T, D><<<a.ctas, kThreads, smem, st>>>(mk, mv, a);
  if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B, (a.Hq + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, decode_join_kernel<T, D>, a));
}

}  // namespace
}  // namespace tt

using namespace tt;

TT_API size_t tt_tree_decode_plan_bytes(int32_t S) {
  return S < 0 || S > (1 << 24) ? 0 : kPlanSegs + (size_t)S * 2 * sizeof(int4);
}

TT_API int tt_tree_decode_plan(const int32_t* kv_begin, const int32_t* kv_len, const int32_t* q_begin,
                               const int32_t* q_end, int32_t S, int32_t B, int64_t rows, int64_t pairs, int Hq, int Hkv,
                               int d, void* plan, size_t plan_bytes, int32_t* err, tt_stream_t stream) {
  const int rc = check_sizes(S, B, rows, pairs, Hq, Hkv, d);
  if (rc) return rc;
  if ((S && (!kv_begin || !kv_len || !q_begin || !q_end)) || !plan || !aligned16(plan) || !err) return TT_ERR_INVALID_ARG;
  if (plan_bytes < tt_tree_decode_plan_bytes(S)) return TT_ERR_WORKSPACE;
  const PlanArgs a = {kv_begin, kv_len, q_begin, q_end, S, B, Hq, Hkv, d, ctas(), rows, pairs, plan, err};
  decode_plan_kernel<<<1, kPlanThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

TT_API size_t tt_tree_decode_attn_workspace_bytes(int64_t pairs, int Hq, int d) {
  if (pairs < 0 || Hq < 1 || (d != 64 && d != 128) || pairs > (INT32_MAX / 2) / Hq) return 0;
  return (size_t)part_rows(pairs, Hq) * (d * sizeof(float) + sizeof(float2));
}

TT_API int tt_tree_decode_attn(const void* plan, const void* Q, int64_t q_ld, const void* K, const void* V, int64_t kv_ld,
                               int dtype, int32_t S, int32_t B, int64_t rows, int64_t pairs, int Hq, int Hkv, int d,
                               float scale, void* O, float* LSE, void* ws, size_t ws_bytes, int32_t* err,
                               tt_stream_t stream) {
  const int rc = check_sizes(S, B, rows, pairs, Hq, Hkv, d);
  if (rc) return rc;
  if (dtype == TT_DT_F32) return TT_ERR_UNSUPPORTED;
  if (dtype != TT_DT_BF16 && dtype != TT_DT_F16) return TT_ERR_INVALID_ARG;
  if (!plan || !aligned16(plan) || !err || !std::isfinite(scale)) return TT_ERR_INVALID_ARG;
  if (B == 0) return TT_OK;
  if (!Q || !aligned16(Q) || !O || !aligned16(O) || !LSE || q_ld < (int64_t)Hq * d || q_ld % 8) return TT_ERR_INVALID_ARG;
  if (rows && (!K || !V || !aligned16(K) || !aligned16(V) || kv_ld < (int64_t)Hkv * d || kv_ld % 8))
    return TT_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return TT_ERR_INVALID_ARG;
  if (ws_bytes < tt_tree_decode_attn_workspace_bytes(pairs, Hq, d)) return TT_ERR_WORKSPACE;
  DecodeArgs a = {plan, Q, q_ld, B, Hq, Hkv, S, ctas(), rows, pairs, scale * kLog2e, nullptr, nullptr, O, LSE, err};
  a.part_o = static_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + part_rows(pairs, Hq) * d);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {  // no pool: the plan has no keys, and a tensor map needs some memory to name
    K = V = Q;
    kv_ld = q_ld;
  }
  if (dtype == TT_DT_F16) return d == 64 ? launch_decode<__half, 64>(a, K, V, kv_ld, st) : launch_decode<__half, 128>(a, K, V, kv_ld, st);
  return d == 64 ? launch_decode<__nv_bfloat16, 64>(a, K, V, kv_ld, st) : launch_decode<__nv_bfloat16, 128>(a, K, V, kv_ld, st);
}
