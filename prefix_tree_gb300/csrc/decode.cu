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
// A segment with more rows than this is taken by tiles of 128 rows on the tensor cores' asynchronous path, one with
// fewer by tiles of 16 on the warps' own.
#ifndef TT_WIDE
#define TT_WIDE 32
#endif
constexpr int kWideFrom = TT_WIDE;
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
      const int rows = (q1 - q0) * G, tile_rows = rows > kWideFrom ? kMostRows : 16;
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
constexpr int kThreads = 32 * (kWarps + 2);  // and one that copies, one that issues the tensor-core products
constexpr int kKStages = 3, kVStages = 2;  // K and V tiles in shared memory
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256, kColP = 384;  // S and P twice: 128 and 64 columns each
// The running maximum of a row moves only when it grows by more than this (log2 units): weights stay below 2^8.
constexpr float kRescale = 8.0f;

template <int D>
struct Smem {
  static constexpr uint32_t kBox = kKeys * 128;            // 64 columns of a block's keys, 128-byte swizzle
  static constexpr uint32_t kTile = (D / 64) * kBox;
  static constexpr uint32_t q = 0;                         // the 128 rows of a wide tile, laid out as a K tile
  static constexpr uint32_t kQLd = D * 2 + 16;             // bytes of a row of Q of a narrow tile
  static constexpr uint32_t k0 = q + kTile;
  static constexpr uint32_t v0 = k0 + kKStages * kTile;
  static constexpr uint32_t kPLd = kKeys * 2 + 16;         // bytes of a row of weights: rows fall in different banks
  static constexpr uint32_t p = v0 + kVStages * kTile;     // narrow tiles: [16] rows of weights
  static constexpr uint32_t max = p + 16 * kPLd;           // [kWarps][16] f32
  static constexpr uint32_t sum = max + kWarps * 16 * 4;   // [kWarps][16] f32
  static constexpr uint32_t row_max = sum + kWarps * 16 * 4;  // [16] f32
  static constexpr uint32_t wide = row_max + 16 * 4;       // wide tiles: [2][128] f32 of the two halves of a row
  static constexpr uint32_t bars = wide + 2 * 128 * 4;
  static constexpr uint32_t misc = bars + 32 * 8;
  static constexpr uint32_t total = misc + 16 + 1024;      // + slack for the alignment to 1024 bytes
};
// Barriers. EMPTY: the eight computing warps and the issuing one; a warp arrives for a block after it has seen the
// block's FULL, so that it cannot be a phase ahead.
constexpr int K_FULL = 0, V_FULL = K_FULL + kKStages, K_EMPTY = V_FULL + kVStages, V_EMPTY = K_EMPTY + kKStages,
              Q_READY = V_EMPTY + kVStages, S_FULL = Q_READY + 1, S_FREE = S_FULL + 2, P_READY = S_FREE + 2,
              P_FREE = P_READY + 2, FINAL = P_FREE + 2, NBAR = FINAL + 1;
static_assert(NBAR <= 32, "barriers");

// kind::f16 instruction descriptor for type T.
template <typename T>
constexpr uint32_t idesc_of(int M, int N, int a_mn, int b_mn) {
  return idesc_bf16(M, N, a_mn, b_mn) & (std::is_same<T, __half>::value ? ~((1u << 7) | (1u << 10)) : ~0u);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecodeArgs a) {
  using L = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::misc + 4);
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
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bar[K_FULL + i], 1);
      mbar_init(&bar[K_EMPTY + i], kWarps + 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bar[V_FULL + i], 1);
      mbar_init(&bar[V_EMPTY + i], kWarps + 1);
    }
    mbar_init(&bar[Q_READY], 32 * kWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[S_FULL + i], 1);
      mbar_init(&bar[S_FREE + i], 32 * kWarps);
      mbar_init(&bar[P_READY + i], 32 * kWarps);
      mbar_init(&bar[P_FREE + i], 1);
    }
    mbar_init(&bar[FINAL], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kWarps + 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const int n = (int)(w1 - w0), G = a.Hq / a.Hkv;
  const int4* segs = reinterpret_cast<const int4*>(static_cast<const char*>(a.plan) + kPlanSegs);
  Walk at(segs, a.Hkv, G, reinterpret_cast<const int32_t*>(static_cast<const char*>(a.plan) + kPlanCtas)[c], (int)w0);

  if (warp == kWarps) {
    // ------------------------------------------------------------ copies: lane 0 the K tiles, lane 1 the V tiles
    if (lane < 2) {
      const CUtensorMap* map = lane ? &tmV : &tmK;
      const int full = lane ? V_FULL : K_FULL, empty = lane ? V_EMPTY : K_EMPTY, stages = lane ? kVStages : kKStages;
      uint8_t* dst = sm + (lane ? L::v0 : L::k0);
      prefetch_tmap(map);
      int i = 0, st = 0, phase = 0;
      for (; i < n; ++i) {
        if (i >= stages && !mbar_wait(&bar[empty + st], phase ^ 1, abort_flag, 50 + lane)) break;
        mbar_expect_tx(&bar[full + st], L::kTile);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
          tma_load_2d(dst + st * L::kTile + x * L::kBox, map, &bar[full + st], at.h * D + x * 64, at.kv + at.blk * kKeys);
        at.next(i + 1 < n);
        if (++st == stages) st = 0, phase ^= 1;
      }
      // every copy issued has landed before the CTA may leave
      for (int j = i - 1; j >= 0 && j >= i - stages; --j) mbar_drain(&bar[full + j % stages], (j / stages) & 1, abort_flag);
    }
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------ tensor-core products of the wide tiles
    if (lane == 0) {
      constexpr uint32_t idS = idesc_of<T>(128, 128, 0, 0), idPV = idesc_of<T>(128, D, 0, 1);
      const uint64_t dq = smem_desc(smem_u32(sm + L::q), 16, 1024);
      int j = 0, tiles = 0;              // wide blocks and wide tiles so far
      int pv_st = -1, pv_phase = 0;      // the block whose second product is still to be issued: its V stage,
      bool pv_first = false;             // and whether it is its tile's first
      bool ok = true;
      auto issue_pv = [&]() -> bool {    // of wide block j − 1
        const int bb = (j - 1) & 1;
        if (!mbar_wait(&bar[P_READY + bb], ((j - 1) >> 1) & 1, abort_flag, 54)) return false;
        if (!mbar_wait(&bar[V_FULL + pv_st], pv_phase, abort_flag, 55)) return false;
        tc_fence_after();
        const uint64_t dv = smem_desc(smem_u32(sm + L::v0 + pv_st * L::kTile), L::kBox, 1024);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          umma_ts(tbase + kColO, tbase + kColP + bb * 64 + k * 8, desc_at(dv, k * 2048), idPV, !pv_first || k > 0);
        umma_commit(&bar[P_FREE + bb]);
        umma_commit(&bar[V_EMPTY + pv_st]);
        pv_st = -1;
        return true;
      };
      int kst = 0, kphase = 0, vst = 0, vphase = 0;
      for (int i = 0; i < n; ++i) {
        if (!mbar_wait(&bar[K_FULL + kst], kphase, abort_flag, 56)) { ok = false; break; }
        if (at.tile_rows == kMostRows) {
          const int bb = j & 1;
          const bool first = i == 0 || at.blk == 0;
          if (first && !mbar_wait(&bar[Q_READY], tiles++ & 1, abort_flag, 57)) { ok = false; break; }
          if (j >= 2 && !mbar_wait(&bar[S_FREE + bb], ((j - 2) >> 1) & 1, abort_flag, 58)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dk = smem_desc(smem_u32(sm + L::k0 + kst * L::kTile), 16, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k >> 2) * L::kBox + (k & 3) * 32;
            umma_ss(tbase + kColS + bb * 128, desc_at(dq, off), desc_at(dk, off), idS, k > 0);
          }
          umma_commit(&bar[S_FULL + bb]);
          umma_commit(&bar[K_EMPTY + kst]);
          if (pv_st >= 0 && !issue_pv()) { ok = false; break; }
          pv_st = vst, pv_phase = vphase, pv_first = first;
          ++j;
          // a tile's last block is finished here: the computing warps wait for it before they turn to the next tile
          if ((i + 1 == n || at.blk + 1 == at.nb) && !issue_pv()) { ok = false; break; }
        } else {  // the computing warps' alone
          mbar_arrive(&bar[K_EMPTY + kst]);
          if (!mbar_wait(&bar[V_FULL + vst], vphase, abort_flag, 59)) { ok = false; break; }
          mbar_arrive(&bar[V_EMPTY + vst]);
        }
        at.next(i + 1 < n);
        if (++kst == kKStages) kst = 0, kphase ^= 1;
        if (++vst == kVStages) vst = 0, vphase ^= 1;
      }
      // completes after every product of this CTA, also after an abort: shared and tensor memory outlive them
      (void)ok;
      umma_commit(&bar[FINAL]);
      mbar_drain(&bar[FINAL], 0, abort_flag);
    }
  } else {
    // ------------------------------------------------------------ 16 rows against the blocks, all warps on every block
    constexpr int kCols = D / kWarps;     // columns of O of a warp
    constexpr int kOut = kCols / 8;
    const int r0 = lane >> 2, cc = (lane & 3) * 2;
    const int mi = lane >> 3, mr = lane & 7;
    float o[kOut][4], m[2], l[2];
    float* smax = reinterpret_cast<float*>(sm + L::max);
    float* ssum = reinterpret_cast<float*>(sm + L::sum);
    float* srow = reinterpret_cast<float*>(sm + L::row_max);
    const uint32_t pbase = smem_u32(sm + L::p);
    const uint32_t qbase = smem_u32(sm + L::q) + ((mi & 1) * 8 + mr) * L::kQLd + (mi >> 1) * 16;
    float* half_of_row = reinterpret_cast<float*>(sm + L::wide);
    int j = 0;                            // wide blocks so far
    int kst = 0, kphase = 0, vst = 0, vphase = 0;
    for (int i = 0; i < n; ++i) {
      const int tile_n = min(at.tile_rows, at.rows - at.tile * at.tile_rows);  // rows of this tile
      const bool first = i == 0 || at.blk == 0, last = i + 1 == n || at.blk + 1 == at.nb;
      const int valid = at.len - at.blk * kKeys;  // keys of the segment in this block, possibly more than there are
      // rows behind the segment's end are another segment's, or not yet written: a weight of 0 times what lies there must
      // be 0
      auto clear_behind = [&]() {
        if (valid >= kKeys) return;
        for (int e = (int)threadIdx.x; e < (kKeys - valid) * (D / 8); e += 32 * kWarps) {
          const int key = valid + e / (D / 8), u = e % (D / 8);
          *reinterpret_cast<uint4*>(sm + L::v0 + vst * L::kTile + (u >> 3) * L::kBox + key * 128 + ((u & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the products, and the next copy
      };
      if (at.tile_rows == kMostRows) {
        // ---------------------------------------------------------- 128 rows: a thread one row and half of the keys
        const int wq = warp & 3, hf = warp >> 2, r = wq * 32 + lane, bb = j & 1;
        const uint32_t lanes = tbase + ((uint32_t)(wq * 32) << 16);
        if (first) {
          // the rows of Q into shared memory, in the swizzled layout that the products read
          for (int e = (int)threadIdx.x; e < kMostRows * (D / 8); e += 32 * kWarps) {
            const int row = e / (D / 8), u = e % (D / 8), rr = at.tile * kMostRows + row;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (row < tile_n)
              x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (int64_t)(at.q0 + rr / G) * a.q_ld +
                                                  (int64_t)(at.h * G + rr % G) * D + u * 8);
            *reinterpret_cast<uint4*>(sm + L::q + (u >> 3) * L::kBox + row * 128 + (((u & 7) ^ (row & 7)) << 4)) = x;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          mbar_arrive(&bar[Q_READY]);
          m[0] = -INFINITY;
          l[0] = 0.f;
        }
        mbar_wait(&bar[K_FULL + kst], kphase, abort_flag, 60);
        mbar_wait(&bar[S_FULL + bb], (j >> 1) & 1, abort_flag, 61);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[K_EMPTY + kst]);
        tc_fence_after();
        uint32_t x[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_ld32(lanes + kColS + bb * 128 + 64 * hf + q * 32, x[q]);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_pin(x[q]);
        tc_fence_before();
        mbar_arrive(&bar[S_FREE + bb]);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const int seen = valid - 64 * hf;  // keys of this half that are there
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int col = q * 32 + 2 * e;
            const float2 y = __fmul2_rn(make_float2(__uint_as_float(x[q][2 * e]), __uint_as_float(x[q][2 * e + 1])),
                                        make_float2(a.scale_log2, a.scale_log2));
            const float y0 = col < seen ? y.x : -INFINITY, y1 = col + 1 < seen ? y.y : -INFINITY;
            x[q][2 * e] = __float_as_uint(y0);
            x[q][2 * e + 1] = __float_as_uint(y1);
            mx[e & 3] = fmax3f(mx[e & 3], y0, y1);
          }
        const float pm = fmax3f(mx[0], mx[1], fmaxf(mx[2], mx[3]));
        half_of_row[hf * 128 + r] = pm;
        named_barrier(2 + wq, 64);
        const float top = fmaxf(pm, half_of_row[(hf ^ 1) * 128 + r]);
        named_barrier(2 + wq, 64);  // (read before the next block writes)
        bool moved = false;
        float f = 1.f;
        if (top > m[0] + kRescale) {
          f = fast_exp2(m[0] - top);  // 0 at the tile's first keys
          l[0] *= f;
          moved = !first;
          m[0] = top;
        }
        const float mu = m[0] == -INFINITY ? 0.f : m[0];
        const float2 nm = make_float2(-mu, -mu);
        float2 rs = make_float2(0.f, 0.f);
        uint32_t pk[32];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 d = __fadd2_rn(make_float2(__uint_as_float(x[q][2 * e]), __uint_as_float(x[q][2 * e + 1])), nm);
            const float2 w = make_float2(fast_exp2(d.x), fast_exp2(d.y));
            rs = __fadd2_rn(rs, w);
            pk[q * 16 + e] = pack2<T>(w.x, w.y);
          }
        l[0] += rs.x + rs.y;
        if (j >= 2) mbar_wait(&bar[P_FREE + bb], ((j - 2) >> 1) & 1, abort_flag, 62);
        if (__any_sync(~0u, moved)) {
          mbar_wait(&bar[P_FREE + (bb ^ 1)], ((j - 1) >> 1) & 1, abort_flag, 63);  // O of the block before
          tc_fence_after();
          const float g = moved ? f : 1.f;
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            const uint32_t col = lanes + kColO + (D / 2) * hf + q * 32;
            uint32_t y[32];
            tmem_ld32(col, y);
            tmem_ld_wait();
            tmem_pin(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * g);
            tmem_st32(col, y);
          }
        }
        tmem_st32(lanes + kColP + bb * 64 + 32 * hf, pk);
        tmem_st_wait();
        mbar_wait(&bar[V_FULL + vst], vphase, abort_flag, 64);
        clear_behind();
        tc_fence_before();
        mbar_arrive(&bar[P_READY + bb]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[V_EMPTY + vst]);
        if (last) {
          // the tile's part: the row's sums from tensor memory
          half_of_row[hf * 128 + r] = l[0];
          named_barrier(2 + wq, 64);
          const float sum = l[0] + half_of_row[(hf ^ 1) * 128 + r];
          named_barrier(2 + wq, 64);
          mbar_wait(&bar[P_FREE + bb], (j >> 1) & 1, abort_flag, 65);
          tc_fence_after();
          const int64_t row = at.part_row(c) + r;
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            uint32_t y[32];
            tmem_ld32(lanes + kColO + (D / 2) * hf + q * 32, y);
            tmem_ld_wait();
            tmem_pin(y);
            if (r < tile_n) {
              float4* dst = reinterpret_cast<float4*>(a.part_o + row * D + (D / 2) * hf + q * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                dst[e] = make_float4(__uint_as_float(y[4 * e]), __uint_as_float(y[4 * e + 1]),
                                     __uint_as_float(y[4 * e + 2]), __uint_as_float(y[4 * e + 3]));
            }
          }
          tc_fence_before();
          if (hf == 0 && r < tile_n) a.part_ml[row] = make_float2(m[0], sum);
        }
        ++j;
        at.next(i + 1 < n);
        if (++kst == kKStages) kst = 0, kphase ^= 1;
        if (++vst == kVStages) vst = 0, vphase ^= 1;
        continue;
      }
      if (first) {
        // the rows of Q into shared memory (where wide tiles keep theirs)
        for (int e = (int)threadIdx.x; e < 16 * (D / 8); e += 32 * kWarps) {
          const int row = e / (D / 8), u = e % (D / 8), rr = at.tile * 16 + row;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row < tile_n)
            x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (int64_t)(at.q0 + rr / G) * a.q_ld +
                                                (int64_t)(at.h * G + rr % G) * D + u * 8);
          *reinterpret_cast<uint4*>(sm + L::q + row * L::kQLd + u * 16) = x;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          m[half] = -INFINITY;
          l[half] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kOut; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
        named_barrier(1, 32 * kWarps);
      }
      // S of this warp's 16 keys
      float s[2][4] = {};
      mbar_wait(&bar[K_FULL + kst], kphase, abort_flag, 52);
      {
        const uint32_t kt = smem_u32(sm + L::k0 + kst * L::kTile);
        const int key = warp * 16 + (mi >> 1) * 8 + mr;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int unit = (k & 3) * 2 + (mi & 1);  // 16 bytes of the row within its box
          uint32_t b[4], qa[4];
          ldsm4(qa, qbase + k * 32);
          ldsm4(b, kt + (k >> 2) * L::kBox + key * 128 + ((unit ^ (key & 7)) << 4));
          mma16816<T>(s[0], qa, b[0], b[1]);
          mma16816<T>(s[1], qa, b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[K_EMPTY + kst]);
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
      mbar_wait(&bar[V_FULL + vst], vphase, abort_flag, 53);
      clear_behind();
      named_barrier(1, 32 * kWarps);  // the weights are there
      {
        const uint32_t vt = smem_u32(sm + L::v0 + vst * L::kTile);
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
      if (lane == 0) mbar_arrive(&bar[V_EMPTY + vst]);
      if (last) {
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
      if (++kst == kKStages) kst = 0, kphase ^= 1;
      if (++vst == kVStages) vst = 0, vphase ^= 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
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
