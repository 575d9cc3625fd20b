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
// that it met the unnormalised sums, the references and the sums of weights of
// its rows (fp32); a second kernel joins the parts of every query and head in
// a fixed order. With row_base(tile) + 128·CTA as the place of a part, the
// parts of different tiles and CTAs cannot meet: along the runs one of the two
// grows at every step, by at least the rows that the part before takes.
//
// Bound by memory where most keys are the rollouts' own (32 heads to 8 key
// heads of 128, bf16; this kernel + the joining one): 500 rollouts of 2048 keys
// 630 + 15 us for 4.19 GB (6.7 TB/s in the first), 480 of 384 keys 126 + 14 us
// for 755 MB (6.0). With heads of 64 a block has half the bytes and the same
// waits, and the same rollouts take 470 and 97 us (4.5 and 3.9 TB/s). Where a
// long prompt has many rows its products and exponentials bound it: a wide
// block whose keys lie in the L2 cache takes 1.35 us, a narrow one 0.9. A group
// of 64 rollouts of 8192 shared and about 1150 own keys: 57 to 62 + 6 us for 325
// MB; a deep tree of 16,001 shared keys, six common turns and 120 rollouts of
// 1500, 40 heads to 8: 150 to 163 + 9 us for 842 MB.
//
// A segment is a tile of its own, with a start, a part and at least one block,
// and the join looks at every segment for each query and eight heads. Small
// pages are therefore dear: 64 rollouts of 8192 shared and 1024 own keys 59 + 6
// us (302 MB), the same in pages of 256 rows 83 + 31, of 64 rows 276 + 126, of 16
// rows 1073 + 473; the plan, one CTA, 61 us for 16,000 segments.
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
constexpr int kMostRows = 128;   // rows of a wide tile
constexpr int kNarrow = 16;      // and of a narrow one
constexpr int kMostCtas = 1024;
constexpr int kMostSegs = (1 << 24) - 1;
constexpr int kPiece = 32;       // rows of a copy
// Work is shared out by cost: of a block, and of a tile's start (its queries have to be fetched first and its sums
// written last). Measured on a group of 64 rollouts, a deep tree and 40 groups of six, bf16 and fp16. A narrow block at 2.5 or
// 3.5 in place of 3: with heads of 64 2 to 5 % slower either way, with heads of 128 up to 5 % slower at 2.5, between 4 % slower
// and 5 % faster at 3.5; at 4: up to 13 % slower. Starts of 12 and 2, or 16 and 8, in place of 12 and 4: the groups of six 23 %
// slower, or 14 % (heads of 64), the others within 3 %.
constexpr int kBlockWide = 4, kBlockNarrow = 3, kStartWide = 12, kStartNarrow = 4;
// A segment with more rows than this is taken by tiles of 128 rows on the tensor cores' asynchronous path, one with
// fewer by tiles of 16 on the warps' own: 40 segments of 3000 keys with 24 rows take 110 us by one wide tile and 186 by two
// narrow ones (with their rollouts' own keys; heads of 64: 90 and 130).
constexpr int kWideFrom = 16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Plan: header, first segment of every CTA, and two int4 for each segment that has keys and queries:
// {first row of the pool, keys, first query, queries}, {blocks before it, tiles of a head, rows of a tile, partial rows
// before it}.
struct PlanHeader {
  int64_t magic;
  int32_t S, B, Hq, Hkv, d, ctas, valid, code;  // code: the error where valid = 0
  int64_t rows, pairs;
  int32_t cost, quota, segments;
};
constexpr size_t kPlanCtas = 128, kPlanSegs = kPlanCtas + sizeof(int32_t) * kMostCtas;
static_assert(sizeof(PlanHeader) <= kPlanCtas, "header");

__host__ __device__ constexpr int block_cost(int tile_rows) { return tile_rows == kMostRows ? kBlockWide : kBlockNarrow; }
__host__ __device__ constexpr int start_cost(int tile_rows) { return tile_rows == kMostRows ? kStartWide : kStartNarrow; }

struct PlanArgs {
  const int32_t *kv_begin, *kv_len, *q_begin, *q_end;
  int S, B, Hq, Hkv, d, ctas;
  int64_t rows, pairs;
  void* plan;
  int32_t* err;
};

constexpr int kPlanThreads = 1024;

// Exclusive sums of x and y over the block's threads, and the totals. `room`: one place per warp.
__device__ __forceinline__ void scan_block(int64_t& x, int64_t& y, int64_t& all_x, int64_t& all_y, longlong2* room) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t x0 = x, y0 = y;
  auto scan_warp = [&](int64_t& u, int64_t& v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(~0u, u, o), q = __shfl_up_sync(~0u, v, o);
      if (lane >= o) u += p, v += q;
    }
  };
  scan_warp(x, y);
  if (lane == 31) room[warp] = make_longlong2(x, y);
  __syncthreads();
  int64_t u = lane < warps ? room[lane].x : 0, v = lane < warps ? room[lane].y : 0;
  scan_warp(u, v);
  all_x = __shfl_sync(~0u, u, 31);
  all_y = __shfl_sync(~0u, v, 31);
  const int64_t bx = __shfl_sync(~0u, u, (warp + 31) & 31), by = __shfl_sync(~0u, v, (warp + 31) & 31);
  x += (warp ? bx : 0) - x0;
  y += (warp ? by : 0) - y0;
}

// One CTA; a thread takes consecutive segments.
__global__ void __launch_bounds__(kPlanThreads) decode_plan_kernel(const PlanArgs a) {
  __shared__ longlong2 room[kPlanThreads / 32];
  __shared__ int code;
  PlanHeader* hdr = static_cast<PlanHeader*>(a.plan);
  int32_t* cta_seg = reinterpret_cast<int32_t*>(static_cast<char*>(a.plan) + kPlanCtas);
  int4* segs = reinterpret_cast<int4*>(static_cast<char*>(a.plan) + kPlanSegs);
  if (threadIdx.x == 0) code = 0;
  __syncthreads();
  const int G = a.Hq / a.Hkv, each = (a.S + (int)blockDim.x - 1) / (int)blockDim.x;
  const int s0 = min((int64_t)a.S, (int64_t)threadIdx.x * each), s1 = min(a.S, s0 + each);
  // a segment's first row, keys, queries, and its cost, or 0 where it has no work
  auto read = [&](int s, int4& x, int& tiles, int& tile_rows) -> int64_t {
    const int q1 = a.q_end[s];
    x = make_int4(a.kv_begin[s], a.kv_len[s], a.q_begin[s], 0);
    if (x.x < 0 || x.y < 0 || (int64_t)x.x + x.y > a.rows || x.z < 0 || q1 < x.z || q1 > a.B) {
      atomicCAS(&code, 0, TT_ERR_INVALID_ARG);
      return 0;
    }
    x.w = q1 - x.z;
    const int64_t rows = (int64_t)x.w * G;
    if (!x.y || !rows) return 0;
    tile_rows = rows > kWideFrom ? kMostRows : kNarrow;
    tiles = (int)((rows + tile_rows - 1) / tile_rows);
    return ((int64_t)((x.y + kKeys - 1) / kKeys) * block_cost(tile_rows) + start_cost(tile_rows)) * tiles * a.Hkv;
  };
  int64_t cost = 0, rows_n = 0;  // rows_n: partial rows << 24, and segments
  int4 x;
  int tiles, tile_rows;
  // (a thread's sum is cut off where it is too large already, so that the block's cannot wrap; a partial row costs an eighth
  // and more, so that the rows of a step that is not too large cannot either)
  for (int s = s0; s < s1; ++s)
    if (const int64_t c = read(s, x, tiles, tile_rows)) {
      cost = min(cost + c, (int64_t)INT32_MAX);
      rows_n += ((int64_t)x.w * a.Hq << 24) + 1;
    }
  int64_t all_cost, all_rows_n;
  scan_block(cost, rows_n, all_cost, all_rows_n, room);
  if (threadIdx.x == 0 && all_cost > INT32_MAX / 2) atomicCAS(&code, 0, TT_ERR_UNSUPPORTED);
  if (threadIdx.x == 0 && (all_rows_n >> 24) > a.pairs * a.Hq) atomicCAS(&code, 0, TT_ERR_WORKSPACE);
  __syncthreads();
  if (threadIdx.x == 0) {
    const int n = (int)(all_rows_n & 0xffffff);
    const int64_t quota = max((all_cost + a.ctas - 1) / a.ctas, (int64_t)1);
    *hdr = {kPlanMagic, a.S, a.B, a.Hq, a.Hkv, a.d, a.ctas, code == 0, code, a.rows, a.pairs, (int)all_cost, (int)quota, n};
    if (code) set_err(a.err, code);
  }
  if (code) return;
  const int quota = (int)max((all_cost + a.ctas - 1) / a.ctas, (int64_t)1);
  for (int s = s0; s < s1; ++s) {
    const int64_t c = read(s, x, tiles, tile_rows);
    if (!c) continue;
    const int n = (int)(rows_n & 0xffffff);
    segs[2 * n] = x;
    segs[2 * n + 1] = make_int4((int)cost, tiles, tile_rows, (int)(rows_n >> 24));
    // the CTAs whose run begins in it
    for (int64_t r = (cost + quota - 1) / quota; r * quota < cost + c; ++r) cta_seg[r] = n;
    cost += c;
    rows_n += ((int64_t)x.w * a.Hq << 24) + 1;
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
  float2* part_ml; // [parts' rows] reference (log2 units) and sum of weights
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

// A run's way over its blocks: segment, head, tile, block. Tiles follow one another on a line of costs, each its start
// and then its blocks; a block belongs to the run [w, end) in which its place begins.
struct Walk {
  const int4* segs;
  int Hkv, G, w, end;
  int seg, h, tile, blk;            // where it is; w: the block's place
  int kv, len, q0, rows, nb;        // the segment's first key row, keys, first query, rows of a head, blocks of a tile
  int tiles, tile_rows, row_base, cost, start;
  __device__ __forceinline__ int load() {
    const int4 x = segs[2 * seg], y = segs[2 * seg + 1];
    kv = x.x, len = x.y, q0 = x.z, rows = x.w * G, nb = (len + kKeys - 1) / kKeys;
    tiles = y.y, tile_rows = y.z, row_base = y.w;
    cost = block_cost(tile_rows), start = start_cost(tile_rows);
    return y.x;
  }
  __device__ __forceinline__ Walk(const int4* segs_, int Hkv_, int G_, int first_seg, int w_, int end_)
      : segs(segs_), Hkv(Hkv_), G(G_), w(w_), end(end_), seg(first_seg) {
    const int at = w - load(), whole = nb * cost + start, unit = at / whole, off = at - unit * whole - start;
    blk = off <= 0 ? 0 : (off + cost - 1) / cost;
    w += blk * cost - off;
    h = unit / tiles;
    tile = unit - h * tiles;
    if (blk == nb) next_tile();
  }
  __device__ __forceinline__ bool done() const { return w >= end; }
  // blocks of this tile in the run, from here on
  __device__ __forceinline__ int stretch() const { return min(nb - blk, (end - w + cost - 1) / cost); }
  // past n of them
  __device__ __forceinline__ void pass(int n) {
    w += n * cost;
    blk += n;
    if (blk == nb) next_tile();
  }
  __device__ __forceinline__ void next_tile() {
    blk = 0;
    if (++tile == tiles) {
      tile = 0;
      if (++h == Hkv) {
        h = 0;
        ++seg;
        if (w < end) load();
      }
    }
    w += start;
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
// and four more: one copies the K tiles, one the V tiles (a thread suspended in a wait holds up the others of its warp), one
// issues the tensor-core products.
constexpr int kThreads = 32 * (kWarps + 4), kCopyK = kWarps, kCopyV = kWarps + 1, kIssue = kWarps + 2;
// Twelve warps launch with 168 registers each; those four give some back for the computing ones:
// 128·136 + 256·184 = 64,512 = 384·168 = 64,512 launched.
constexpr uint32_t kRegsControl = 136, kRegsCompute = 184;
static_assert(128 * kRegsControl + 256 * kRegsCompute <= kThreads * 168, "register split exceeds the launch's registers");
constexpr int kKStages = 3, kVStages = 2;  // K and V tiles in shared memory
// Tensor memory: each of two groups of four warps has 128 columns for S, whose places its weights take, and up to 128
// for O.
constexpr uint32_t kTmemCols = 512, kGroupCols = 256, kColO = 128;
// The weights enter the second product in the type of V, each off by up to half a step (bf16 2^-8, fp16 2^-11): the product
// of two factors of one 16-bit type is what the tensor cores have, and 32 bits of weight (as a high and a low part) would
// double it. The sum of weights is that of the unrounded ones.
// A row's weights are 2^(score − reference), the reference kLift below a maximum that moves only when the scores grow by more
// than kRescale above it (log2 units): they stay below 2^(kRescale + kLift). fp16 has room for 2^15 and ends at 2^-24, so that
// lifted by 2^7 the weights of far keys are rounded to multiples of 2^-31 of the largest (the sum counts them in any case). The
// bound is put to the difference, which is exact: reference and bound added would round to more from scores of 2^26 on.
constexpr float kRescale = 8.0f;
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 7.0f : 0.0f;

template <int D>
struct Smem {
  static constexpr uint32_t kBox = kKeys * 128;            // 64 columns of a block's keys, 128-byte swizzle
  static constexpr uint32_t kTile = (D / 64) * kBox;
  static constexpr uint32_t q = 0;                         // the 128 rows of a wide tile, laid out as a K tile
  static constexpr uint32_t k0 = q + kTile;
  static constexpr uint32_t v0 = k0 + kKStages * kTile;
  // wide tiles: reference and sum [2][2][128] f32 of the two groups' rows; narrow tiles: twice [kWarps][16] f32
  static constexpr uint32_t rows = v0 + kVStages * kTile;
  static constexpr uint32_t bars = rows + 4 * 128 * 4;
  static constexpr uint32_t misc = bars + 32 * 8;
  static constexpr uint32_t total = misc + 16;             // with the start aligned to 1024 bytes
  static_assert(kWarps * 8 * D * 4 <= kTile, "the joining rows exceed the place of Q");
};
// Barriers. EMPTY: one arrival of each computing warp after a narrow block; after a wide one all from the issuing thread,
// the last of them when its products are done.
constexpr int K_FULL = 0, V_FULL = K_FULL + kKStages, K_EMPTY = V_FULL + kVStages, V_EMPTY = K_EMPTY + kKStages,
              Q_READY = V_EMPTY + kVStages, S_FULL = Q_READY + 1, P_READY = S_FULL + 2, O_DONE = P_READY + 2,
              FINAL = O_DONE + 1, NBAR = FINAL + 1;
static_assert(NBAR <= 32, "barriers");

__device__ __forceinline__ void arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// A copy whose lines the L2 cache keeps as `policy` says.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], [%2], "
      "%5;" ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
// The keys of a segment whose rows take several tiles are read again for each, by CTAs at different times; those of the others
// once, and they are not to drive the first ones out of the L2 cache. Four layers of a deep tree (16,001 shared rows, 600 of
// their queries' heads to a key head; 120 rollouts of 1500 rows): no policy 703 to 722 us, this one 634 to 648; with the first
// ones marked to be evicted last 632, but these would stay in the way of the kernels that follow.
__device__ __forceinline__ uint64_t cache_policy(bool again) {
  uint64_t p;
  if (again)
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  else
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// A ring's stage and phase n blocks on.
__device__ __forceinline__ void pass_stages(int n, int& stage, int& phase, int stages) {
  stage += n;
  phase ^= (stage / stages) & 1;
  stage %= stages;
}

// kind::f16 instruction descriptor for type T.
template <typename T>
constexpr uint32_t idesc_of(int M, int N, int a_mn, int b_mn) {
  return idesc_bf16(M, N, a_mn, b_mn) & (std::is_same<T, __half>::value ? ~((1u << 7) | (1u << 10)) : ~0u);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecodeArgs a) {
  using L = Smem<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&bar[K_FULL + i], 1);
      mbar_init(&bar[K_EMPTY + i], kWarps);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&bar[V_FULL + i], 1);
      mbar_init(&bar[V_EMPTY + i], kWarps);
    }
    mbar_init(&bar[Q_READY], 32 * kWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[S_FULL + i], 1);
      mbar_init(&bar[P_READY + i], 128);
    }
    mbar_init(&bar[O_DONE], 1);
    mbar_init(&bar[FINAL], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  wait_prerequisites();  // the kernels before this one: the plan, Q, K and V, and tensor memory that they may hold
  if (warp == kIssue) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const PlanHeader* hdr = static_cast<const PlanHeader*>(a.plan);
  int e = plan_error(a, D);
  if (smem_u32(sm) & 1023) e = TT_ERR_UNSUPPORTED;  // (the layout of the tiles rests on it)
  if (e && threadIdx.x == 0) set_err(a.err, e);
  const int c = blockIdx.x;
  const int64_t w0 = e ? 0 : (int64_t)c * hdr->quota, cost = e ? 0 : hdr->cost;
  if (w0 >= cost) {  // nothing for this CTA
    __syncthreads();
    if (warp == kIssue) tmem_dealloc(tbase, kTmemCols);
    return;
  }
  const int w1 = (int)min(cost, w0 + hdr->quota);
  const int G = a.Hq / a.Hkv;
  const int4* segs = reinterpret_cast<const int4*>(static_cast<const char*>(a.plan) + kPlanSegs);
  Walk at(segs, a.Hkv, G, reinterpret_cast<const int32_t*>(static_cast<const char*>(a.plan) + kPlanCtas)[c], (int)w0, w1);

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if ((warp == kCopyK || warp == kCopyV) && lane == 0) {
      // ---------------------------------------------------------- copies
      const bool v = warp == kCopyV;
      const CUtensorMap* map = v ? &tmV : &tmK;
      const int full = v ? V_FULL : K_FULL, empty = v ? V_EMPTY : K_EMPTY, stages = v ? kVStages : kKStages;
      uint8_t* dst = sm + (v ? L::v0 : L::k0);
      prefetch_tmap(map);
      const uint64_t once = cache_policy(false), again = cache_policy(true);
      int i = 0, st = 0, phase = 0;
      for (bool ok = true; ok && !at.done();) {
        const int n = at.stretch();
        int y0 = at.kv + at.blk * kKeys, left = at.len - at.blk * kKeys;
        const uint64_t policy = at.tiles > 1 ? again : once;
        for (int t = 0; t < n; ++t, ++i, y0 += kKeys, left -= kKeys) {
          if (i >= stages && !mbar_wait(&bar[empty + st], phase ^ 1, abort_flag, 50)) {
            ok = false;
            break;
          }
          // the pieces that hold keys of the segment
          const int pieces = (min(kKeys, left) + kPiece - 1) / kPiece;
          mbar_expect_tx(&bar[full + st], pieces * kPiece * D * 2);
          for (int y = 0; y < pieces; ++y)
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tma_load_2d(dst + st * L::kTile + x * L::kBox + y * kPiece * 128, map, &bar[full + st], at.h * D + x * 64,
                          y0 + y * kPiece, policy);
          if (++st == stages) st = 0, phase ^= 1;
        }
        at.pass(n);
      }
      // every copy issued has landed before the CTA may leave
      for (int j = i - 1; j >= 0 && j >= i - stages; --j) mbar_drain(&bar[full + j % stages], (j / stages) & 1, abort_flag);
    } else if (warp == kIssue && lane == 0) {
      // ---------------------------------------------------------- tensor-core products of the wide tiles
      constexpr uint32_t idS = idesc_of<T>(128, 128, 0, 0), idPV = idesc_of<T>(128, D, 0, 1);
      const uint64_t dq = smem_desc(smem_u32(sm + L::q), 16, 1024);
      int tiles = 0, blocks[2] = {0, 0};  // wide tiles so far, and blocks of each group
      int kst = 0, kphase = 0, vst = 0, vphase = 0;
      // the block whose second product is still to be issued: its V stage and group, and whether it is the group's first
      int pv_st = -1, pv_phase = 0, pv_group = 0;
      bool pv_first = false, ok = true;
      auto issue_pv = [&]() -> bool {
        if (!mbar_wait(&bar[P_READY + pv_group], (blocks[pv_group] - 1) & 1, abort_flag, 54)) return false;
        if (!mbar_wait(&bar[V_FULL + pv_st], pv_phase, abort_flag, 55)) return false;
        tc_fence_after();
        const uint64_t dv = smem_desc(smem_u32(sm + L::v0 + pv_st * L::kTile), L::kBox, 1024);
        const uint32_t cols = tbase + pv_group * kGroupCols;
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          umma_ts(cols + kColO, cols + k * 8, desc_at(dv, k * 2048), idPV, !pv_first || k > 0);
        arrive_n(&bar[V_EMPTY + pv_st], kWarps - 1);
        umma_commit(&bar[V_EMPTY + pv_st]);
        pv_st = -1;
        return true;
      };
      while (ok && !at.done()) {
        const int n = at.stretch();
        if (at.tile_rows == kMostRows) {
          ok = mbar_wait(&bar[Q_READY], tiles++ & 1, abort_flag, 57);
          for (int t = 0; ok && t < n; ++t) {  // the groups take the blocks in turn
            const int g = t & 1;
            if (!mbar_wait(&bar[K_FULL + kst], kphase, abort_flag, 56)) { ok = false; break; }
            // (S of this group's block before was read before its weights were ready, and those were used by the product
            // issued before this one)
            tc_fence_after();
            const uint64_t dk = smem_desc(smem_u32(sm + L::k0 + kst * L::kTile), 16, 1024);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * L::kBox + (k & 3) * 32;
              umma_ss(tbase + g * kGroupCols, desc_at(dq, off), desc_at(dk, off), idS, k > 0);
            }
            umma_commit(&bar[S_FULL + g]);
            arrive_n(&bar[K_EMPTY + kst], kWarps - 1);
            umma_commit(&bar[K_EMPTY + kst]);
            if (pv_st >= 0) ok = issue_pv();
            ++blocks[g];
            pv_st = vst, pv_phase = vphase, pv_group = g, pv_first = t < 2;
            if (++kst == kKStages) kst = 0, kphase ^= 1;
            if (++vst == kVStages) vst = 0, vphase ^= 1;
          }
          ok = ok && issue_pv();
          umma_commit(&bar[O_DONE]);
        } else {
          pass_stages(n, kst, kphase, kKStages);
          pass_stages(n, vst, vphase, kVStages);
        }
        at.pass(n);
      }
      // completes after every product of this CTA, also after an abort: shared and tensor memory outlive them
      umma_commit(&bar[FINAL]);
      mbar_drain(&bar[FINAL], 0, abort_flag);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    // ------------------------------------------------------------ the computing warps, tile by tile
    // Rows behind the segment's end are another segment's, or not yet written: a weight of 0 times what lies there must be
    // 0. Zeroes rows [lo, hi) of a V tile, by `threads` threads.
    auto clear_rows = [](uint8_t* tile, int lo, int hi, int thread, int threads) {
      for (int e = thread; e < (hi - lo) * (D / 8); e += threads) {
        const int key = lo + e / (D / 8), u = e % (D / 8);
        *reinterpret_cast<uint4*>(tile + (u >> 3) * L::kBox + key * 128 + ((u & 7) << 4)) = make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the products, and the next copy
    };
    float* shared_rows = reinterpret_cast<float*>(sm + L::rows);
    int j = 0, wide_tiles = 0;            // blocks of this warp's group and wide tiles so far
    int kst = 0, kphase = 0, vst = 0, vphase = 0;
    while (!at.done()) {
      const int tile_n = min(at.tile_rows, at.rows - at.tile * at.tile_rows);  // rows of this tile
      const int64_t part = at.part_row(c);
      const int n = at.stretch();
      int left = at.len - at.blk * kKeys;  // keys of the segment from this block on
      if (at.tile_rows == kMostRows) {
        // ---------------------------------------------------------- 128 rows: two groups of four warps take the blocks
        // in turn, a thread one row; while one group is at its exponentials the other's products run
        const int wq = warp & 3, g = warp >> 2, r = wq * 32 + lane;
        const uint32_t lanes = tbase + ((uint32_t)(wq * 32) << 16), cols = lanes + g * kGroupCols;
        // the rows of Q into shared memory, in the swizzled layout that the products read
        constexpr int kUnits = kMostRows * (D / 8) / (32 * kWarps);  // 16-byte pieces of a thread, all under way at once
        uint4 piece[kUnits];
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
          const int at_e = (int)threadIdx.x + e * 32 * kWarps, row = at_e / (D / 8), u = at_e % (D / 8);
          const int rr = at.tile * kMostRows + row;
          piece[e] = make_uint4(0, 0, 0, 0);
          if (row < tile_n)
            piece[e] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (int64_t)(at.q0 + rr / G) * a.q_ld +
                                                       (int64_t)(at.h * G + rr % G) * D + u * 8);
        }
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
          const int at_e = (int)threadIdx.x + e * 32 * kWarps, row = at_e / (D / 8), u = at_e % (D / 8);
          *reinterpret_cast<uint4*>(sm + L::q + (u >> 3) * L::kBox + row * 128 + (((u & 7) ^ (row & 7)) << 4)) = piece[e];
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(&bar[Q_READY]);
        float m = -INFINITY, l = 0.f;  // the row's reference, and its sum of weights
        const float size = fabsf(a.scale_log2);
        for (int t = 0; t < n; ++t, left -= kKeys) {
          if ((t & 1) == g) {
            const int valid = left;  // possibly more than a block's
            mbar_wait(&bar[S_FULL + g], j & 1, abort_flag, 61);
            tc_fence_after();
            // 32 scores of the row; a negative scale turns them round, so that the maximum is the largest weight's; keys
            // that are not there become -inf
            auto scores = [&](int q, uint32_t (&x)[32]) {
              if (a.scale_log2 < 0.f) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] ^= 0x80000000u;
              }
              if (valid < kKeys) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (q * 32 + e >= valid) x[e] = 0xff800000u;
              }
            };
            // (loaded again for the weights: a thread has no registers for a whole row)
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              uint32_t x[2][32];
#pragma unroll
              for (int q = 0; q < 2; ++q) tmem_ld32(cols + half * 64 + q * 32, x[q]);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                tmem_pin(x[q]);
                scores(2 * half + q, x[q]);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  mx[e & 3] = fmax3f(mx[e & 3], __uint_as_float(x[q][2 * e]), __uint_as_float(x[q][2 * e + 1]));
              }
            }
            const float top = __fmul_rn(fmax3f(mx[0], mx[1], fmaxf(mx[2], mx[3])), size);  // (rounded here, not in an fma)
            bool moved = false;
            float f = 1.f;
            if (top - m > kRescale + kLift<T>) {
              f = fast_exp2(m - (top - kLift<T>));  // 0 at the group's first keys
              l *= f;
              moved = t >= 2;
              m = top - kLift<T>;
            }
            if (__any_sync(~0u, moved)) {  // (the products into O that were issued before this S are done, as it is)
              const float by = moved ? f : 1.f;
#pragma unroll
              for (int q = 0; q < D / 32; ++q) {
                uint32_t y[32];
                tmem_ld32(cols + kColO + q * 32, y);
                tmem_ld_wait();
                tmem_pin(y);
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * by);
                tmem_st32(cols + kColO + q * 32, y);
              }
            }
            const float mu = m == -INFINITY ? 0.f : m;
            // The maximum is a rounded product, the differences below are not: from scores of 2^24 on they part by more than
            // half a unit, which soon leaves fp16's range (2^28) and then fp32's (2^31). There the scores are scaled, and
            // rounded, by themselves.
            const bool far = __any_sync(~0u, !(fabsf(mu) < 16777216.f));
            const float2 nm = make_float2(-mu, -mu), by = make_float2(far ? 1.f : size, far ? 1.f : size);
            float2 rs = make_float2(0.f, 0.f);
            // the weights of 32 scores take half of the columns of those: never ones that are still to be read
            auto weigh = [&](int q, const uint32_t (&y)[32]) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 d = __ffma2_rn(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), by, nm);
                const float2 w = make_float2(fast_exp2(d.x), fast_exp2(d.y));
                rs = __fadd2_rn(rs, w);
                pk[e] = pack2<T>(w.x, w.y);
              }
              tmem_st16(cols + q * 16, pk);
            };
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              uint32_t x[2][32];
#pragma unroll
              for (int q = 0; q < 2; ++q) tmem_ld32(cols + half * 64 + q * 32, x[q]);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                tmem_pin(x[q]);
                scores(2 * half + q, x[q]);
                if (far) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) x[q][e] = __float_as_uint(__fmul_rn(__uint_as_float(x[q][e]), size));
                }
                weigh(2 * half + q, x[q]);
              }
            }
            l += rs.x + rs.y;
            tmem_st_wait();
            if (valid < kKeys) {
              mbar_wait(&bar[V_FULL + vst], vphase, abort_flag, 64);
              clear_rows(sm + L::v0 + vst * L::kTile, valid, kKeys, threadIdx.x & 127, 128);
            }
            tc_fence_before();
            mbar_arrive(&bar[P_READY + g]);
            ++j;
          }
          if (++vst == kVStages) vst = 0, vphase ^= 1;
        }
        pass_stages(n, kst, kphase, kKStages);
        // the tile's part: both groups' sums of a row from tensor memory, each thread half of the columns
        shared_rows[(g * 2) * 128 + r] = m;
        shared_rows[(g * 2 + 1) * 128 + r] = l;
        mbar_wait(&bar[O_DONE], wide_tiles++ & 1, abort_flag, 65);
        tc_fence_after();
        named_barrier(2 + wq, 64);
        const float m0 = shared_rows[r], m1 = shared_rows[256 + r], l0 = shared_rows[128 + r], l1 = shared_rows[384 + r];
        const float top = fmaxf(m0, m1), mu = top == -INFINITY ? 0.f : top;
        const float f0 = fast_exp2(m0 - mu), f1 = fast_exp2(m1 - mu);
        const int64_t row = part + r;
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
          const int col = (D / 2) * g + q * 32;
          uint32_t y[32], z[32];
          tmem_ld32(lanes + kColO + col, y);
          if (n > 1) tmem_ld32(lanes + kGroupCols + kColO + col, z);  // (a single block was the first group's)
          tmem_ld_wait();
          tmem_pin(y);
          tmem_pin(z);
          if (r < tile_n) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + row * D + col);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(y[4 * e + i]) * f0;
                if (n > 1) v[i] = fmaf(__uint_as_float(z[4 * e + i]), f1, v[i]);
              }
              dst[e] = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        tc_fence_before();
        if (g == 0 && r < tile_n) a.part_ml[row] = make_float2(top, l0 * f0 + l1 * f1);
        named_barrier(2 + wq, 64);  // (read before the next tile's are written, or O again)
      } else {
        // ---------------------------------------------------------- 16 rows: a warp 16 keys of every block, by itself
        named_barrier(1, 32 * kWarps);  // a wide tile before it is done with the shared rows
        const int r0 = lane >> 2, cc = (lane & 3) * 2, mi = lane >> 3, mr = lane & 7;
        // the rows of Q into shared memory (where wide tiles keep theirs): held in registers they would cost 32
        constexpr int kQLd = D * 2 + 16;  // bytes of a row: rows fall in different banks
        for (int e = (int)threadIdx.x; e < kNarrow * (D / 8); e += 32 * kWarps) {
          const int row = e / (D / 8), u = e % (D / 8), rr = at.tile * kNarrow + row;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row < tile_n)
            x = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (int64_t)(at.q0 + rr / G) * a.q_ld +
                                                (int64_t)(at.h * G + rr % G) * D + u * 8);
          *reinterpret_cast<uint4*>(sm + L::q + row * kQLd + u * 16) = x;
        }
        const uint32_t qbase = smem_u32(sm + L::q) + ((mi & 1) * 8 + mr) * kQLd + (mi >> 1) * 16;
        float o[D / 8][4], m[2], l[2];  // (m: references)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          m[half] = -INFINITY;
          l[half] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
        named_barrier(1, 32 * kWarps);
        const int key0 = warp * 16;
        for (int t = 0; t < n; ++t, left -= kKeys) {
          const int seen = left - key0;  // keys of the segment from this warp's first on
          float s[2][4] = {};
          mbar_wait(&bar[K_FULL + kst], kphase, abort_flag, 52);
          if (seen > 0) {
            const uint32_t kt = smem_u32(sm + L::k0 + kst * L::kTile);
            const int key = key0 + (mi >> 1) * 8 + mr;
            float s2[2][4] = {};  // a second chain of products
#pragma unroll
            for (int k0 = 0; k0 < D / 16; k0 += 2) {
              uint32_t qa[2][4], b[2][4];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                ldsm4(qa[k], qbase + (k0 + k) * 32);
                ldsm4(b[k], kt + ((k0 + k) >> 2) * L::kBox + key * 128 + (((((k0 + k) & 3) * 2 + (mi & 1)) ^ (key & 7)) << 4));
              }
              mma16816<T>(s[0], qa[0], b[0][0], b[0][1]);
              mma16816<T>(s[1], qa[0], b[0][2], b[0][3]);
              mma16816<T>(s2[0], qa[1], b[1][0], b[1][1]);
              mma16816<T>(s2[1], qa[1], b[1][2], b[1][3]);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[t][e] = __fmul_rn(s[t][e] + s2[t][e], a.scale_log2);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[K_EMPTY + kst]);
          uint32_t pa[4];
          if (seen > 0) {
            if (seen < 16) {
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (t * 8 + cc + (e & 1) >= seen) s[t][e] = -INFINITY;
            }
            float f[2] = {1.f, 1.f};
            bool moved = false;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (half * 8 >= tile_n) break;  // (rows that are not there: their scores are 0 or were cleared)
              float x = fmaxf(fmaxf(s[0][2 * half], s[0][2 * half + 1]), fmaxf(s[1][2 * half], s[1][2 * half + 1]));
              x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
              x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
              if (x - m[half] > kRescale + kLift<T>) {
                f[half] = fast_exp2(m[half] - (x - kLift<T>));  // 0 at the first keys
                l[half] *= f[half];
                m[half] = x - kLift<T>;
                moved = true;
              }
              const float mu = m[half] == -INFINITY ? 0.f : m[half];
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  s[t][2 * half + e] = fast_exp2(s[t][2 * half + e] - mu);
                  l[half] += s[t][2 * half + e];
                }
            }
            if (__any_sync(~0u, moved)) {
#pragma unroll
              for (int t = 0; t < D / 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][e] *= f[e >> 1];
            }
            pa[0] = pack2<T>(s[0][0], s[0][1]);
            pa[1] = pack2<T>(s[0][2], s[0][3]);
            pa[2] = pack2<T>(s[1][0], s[1][1]);
            pa[3] = pack2<T>(s[1][2], s[1][3]);
          }
          mbar_wait(&bar[V_FULL + vst], vphase, abort_flag, 53);
          if (seen > 0) {
            if (seen < 16) clear_rows(sm + L::v0 + vst * L::kTile, key0 + seen, key0 + 16, lane, 32);
            __syncwarp();
            const uint32_t vt = smem_u32(sm + L::v0 + vst * L::kTile);
            const int key = key0 + (mi & 1) * 8 + mr;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) {
              const int unit = 2 * u + (mi >> 1);  // 8 columns
              uint32_t b[4];
              ldsm4t(b, vt + (unit >> 3) * L::kBox + key * 128 + (((unit & 7) ^ (key & 7)) << 4));
              mma16816<T>(o[2 * u], pa, b[0], b[1]);
              mma16816<T>(o[2 * u + 1], pa, b[2], b[3]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[V_EMPTY + vst]);
          if (++kst == kKStages) kst = 0, kphase ^= 1;
          if (++vst == kVStages) vst = 0, vphase ^= 1;
        }
        // The tile's part: the warps' sums are joined, eight rows at a time, in shared memory (where wide tiles keep their
        // Q), with the columns of a row turned so that rows fall in different banks.
        float* stage = reinterpret_cast<float*>(sm + L::q);          // [kWarps][8][D]
        float* max_of = reinterpret_cast<float*>(sm + L::rows);      // [kWarps][16]
        float* sum_of = max_of + kWarps * 16;
        named_barrier(1, 32 * kWarps);  // no warp reads Q any more
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half * 8 >= tile_n) break;
          l[half] += __shfl_xor_sync(~0u, l[half], 1);
          l[half] += __shfl_xor_sync(~0u, l[half], 2);
          if ((lane & 3) == 0) {
            max_of[warp * 16 + r0 + 8 * half] = m[half];
            sum_of[warp * 16 + r0 + 8 * half] = l[half];
          }
#pragma unroll
          for (int t = 0; t < D / 8; ++t)
            *reinterpret_cast<float2*>(stage + (warp * 8 + r0) * D + ((t * 8 + cc) ^ (r0 * 8))) =
                make_float2(o[t][2 * half], o[t][2 * half + 1]);
          named_barrier(1, 32 * kWarps);
          const int r = half * 8 + warp;  // this warp's row
          if (r < tile_n) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, max_of[w * 16 + r]);
            const float mu = top == -INFINITY ? 0.f : top;
            constexpr int kE = D / 32;  // columns of a lane
            float acc[kE] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float g = fast_exp2(max_of[w * 16 + r] - mu);
              sum = fmaf(g, sum_of[w * 16 + r], sum);
              const float* src = stage + (w * 8 + warp) * D + ((lane * kE) ^ (warp * 8));
#pragma unroll
              for (int e = 0; e < kE; ++e) acc[e] = fmaf(g, src[e], acc[e]);
            }
            float* dst = a.part_o + (part + r) * D + lane * kE;
            if constexpr (kE == 4)
              *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            else
              *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
            if (lane == 0) a.part_ml[part + r] = make_float2(top, sum);
          }
          named_barrier(1, 32 * kWarps);  // read before it is written again
        }
      }
      at.pass(n);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssue) {
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
  __shared__ int4 list[kJoinChunk][2];
  __shared__ int counts[kJoinWarps];
  __shared__ int rows[kJoinWarps][kJoinParts];
  __shared__ float weights[kJoinWarps][kJoinParts];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_prerequisites();
  const PlanHeader* hdr = static_cast<const PlanHeader*>(a.plan);
  const int4* segs = reinterpret_cast<const int4*>(static_cast<const char*>(a.plan) + kPlanSegs);
  if (plan_error(a, D)) return;  // (before any segment is read: the bytes may hold a plan of fewer of them, or none)
  int4 x = make_int4(0, 0, 0, 0), y = x;
  if ((int)threadIdx.x < hdr->segments) x = segs[2 * threadIdx.x], y = segs[2 * threadIdx.x + 1];
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
    if (s0 && s < hdr->segments) x = segs[2 * s], y = segs[2 * s + 1];
    const bool on = s < hdr->segments && b >= x.z && b < x.z + x.w;
    const uint32_t ballot = __ballot_sync(~0u, on);
    if (lane == 0) counts[warp] = __popc(ballot);
    __syncthreads();
    int before = 0, found = 0;
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w == warp) before = found;
      found += counts[w];
    }
    if (on) {
      const int at = before + __popc(ballot & ((1u << lane) - 1));
      list[at][0] = x;
      list[at][1] = y;
    }
    __syncthreads();
    if (hq < a.Hq)
      for (int e = 0; e < found; ++e) {
        const int4 x = list[e][0], y = list[e][1];
        const int nb = (x.y + kKeys - 1) / kKeys, r = (b - x.z) * G + (hq - h * G), tile = r / y.z;
        const int cost = block_cost(y.z), start = start_cost(y.z);
        const int first = y.x + (h * y.y + tile) * (nb * cost + start) + start;  // place of the tile's first block
        const int c0 = first / quota, c1 = (first + (nb - 1) * cost) / quota;
        for (int c = c0; c <= c1; c += 32) {
          if (kept + 32 > kJoinParts) {
            take(kept);
            kept = 0;
          }
          // whether a block's place begins in the run of CTA c + lane
          const int64_t run = (int64_t)(c + lane) * quota;
          const int64_t blk = run <= first ? 0 : (run - first + cost - 1) / cost;
          const bool has = c + lane <= c1 && blk < nb && first + blk * cost < run + quota;
          const uint32_t with = __ballot_sync(~0u, has);
          if (has) rows[warp][kept + __popc(with & ((1u << lane) - 1))] = y.w + h * x.w * G + r + (c + lane) * kMostRows;
          kept += __popc(with);
        }
      }
    __syncthreads();
  }
  if (hq >= a.Hq) return;
  take(kept);
  const float inv = Ls != 0.f ? 1.f / Ls : 0.f;  // (a NaN stays one)
  T* o = static_cast<T*>(a.o) + ((int64_t)b * a.Hq + hq) * D + lane * kE;
#pragma unroll
  for (int e = 0; e < kE; e += 2) *reinterpret_cast<uint32_t*>(o + e) = pack2<T>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) a.lse[(int64_t)hq * a.B + b] = Ls != 0.f ? (M + __log2f(Ls)) * kLn2 : -INFINITY;
}

int check_sizes(int32_t S, int32_t B, int64_t rows, int64_t pairs, int Hq, int Hkv, int d) {
  if (S < 0 || B < 0 || rows < 0 || pairs < 0 || Hq < 1 || Hkv < 1) return TT_ERR_INVALID_ARG;
  if (rows > INT32_MAX / 2 || S > kMostSegs) return TT_ERR_INVALID_ARG;
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
  if (!make_tmap_bf16_ld(&mk, k, (uint64_t)a.Hkv * D, rows, kv_ld, kPiece) ||
      !make_tmap_bf16_ld(&mv, v, (uint64_t)a.Hkv * D, rows, kv_ld, kPiece))
    return TT_ERR_CUDA;
  const int smem = (int)Smem<D>::total;
  if (!smem_attr_set<decode_kernel<T, D>>(smem)) return TT_ERR_CUDA;
  // Both as programmatic dependents: their launches are prepared while the kernel before runs, and each waits for its
  // predecessors before it reads anything. (Neither lets its own dependents be placed early: CTAs of the joining kernel that
  // wait on SMs took 3 % longer.)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  if (cudaLaunchKernelEx(&cfg, decode_kernel<T, D>, mk, mv, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return TT_ERR_CUDA;
  }
  cfg.gridDim = dim3(a.B, (a.Hq + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, decode_join_kernel<T, D>, a);
  (void)cudaGetLastError();
  return cuda_status(err);
}

}  // namespace
}  // namespace tt

using namespace tt;

TT_API size_t tt_tree_decode_plan_bytes(int32_t S) {
  return S < 0 || S > kMostSegs ? 0 : kPlanSegs + (size_t)S * 2 * sizeof(int4);
}

TT_API int tt_tree_decode_plan(const int32_t* kv_begin, const int32_t* kv_len, const int32_t* q_begin,
                               const int32_t* q_end, int32_t S, int32_t B, int64_t rows, int64_t pairs, int Hq, int Hkv,
                               int d, void* plan, size_t plan_bytes, int32_t* err, tt_stream_t stream) {
  const int rc = check_sizes(S, B, rows, pairs, Hq, Hkv, d);
  if (rc) return rc;
  if ((S && (!kv_begin || !kv_len || !q_begin || !q_end)) || !plan || !aligned16(plan) || !err) return TT_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(kv_begin) | reinterpret_cast<uintptr_t>(kv_len) | reinterpret_cast<uintptr_t>(q_begin) |
       reinterpret_cast<uintptr_t>(q_end)) % 4)
    return TT_ERR_INVALID_ARG;
  if (plan_bytes < tt_tree_decode_plan_bytes(S)) return TT_ERR_WORKSPACE;
  const PlanArgs a = {kv_begin, kv_len, q_begin, q_end, S, B, Hq, Hkv, d, ctas(), rows, pairs, plan, err};
  decode_plan_kernel<<<1, S <= 256 ? 256 : kPlanThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
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
  if (!plan || !aligned16(plan) || !err || !std::isfinite(scale * kLog2e)) return TT_ERR_INVALID_ARG;
  if (B == 0) return TT_OK;
  if (!Q || !aligned16(Q) || !O || !aligned16(O) || !LSE || reinterpret_cast<uintptr_t>(LSE) % 4) return TT_ERR_INVALID_ARG;
  if (q_ld < (int64_t)Hq * d || q_ld % 8) return TT_ERR_INVALID_ARG;
  if (rows && (!K || !V || !aligned16(K) || !aligned16(V) || kv_ld < (int64_t)Hkv * d || kv_ld % 8))
    return TT_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return TT_ERR_INVALID_ARG;
  if (ws_bytes < tt_tree_decode_attn_workspace_bytes(pairs, Hq, d)) return TT_ERR_WORKSPACE;
  // (a scale of 0 times a masked score of -inf would not be -inf; one of 1e-30 makes equal weights as well)
  const float scale_log2 = scale == 0.f ? 1e-30f : scale * kLog2e;
  DecodeArgs a = {plan, Q, q_ld, B, Hq, Hkv, S, ctas(), rows, pairs, scale_log2, nullptr, nullptr, O, LSE, err};
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
