// LM head fused with the weighted log-prob loss on the 5th-generation tensor
// cores: the logits z = H·Wᵀ are formed tile by tile in tensor memory and
// folded into per-row log-sum-exp partials there; they never reach global
// memory.
//
// "Tree Training", Abstract: averaging the per-branch losses equals one pass
// over the tree's tokens in which a token's term is scaled by the share of
// branches through it, so each token's log-probability is computed once:
//   lse_t = log Σ_v exp(z_tv),  logp_t = z_{t,y_t} − lse_t,
//   loss  = −Σ_t w_t·logp_t,    z_tv = <H_t, W_v>.
// The pages give no detail of the LM head itself; this is the plain product
// of the final hidden states H [N][Hd] with the vocabulary matrix W [V][Hd].
//
// lmhead_gemm_kernel<EPI_LSE> (the forward): persistent, one CTA per SM, 6 warps.
//   Tiles of 128 rows x 256 vocabulary entries, vocabulary-major (tile t =
//   v·nR + r): at any time the CTAs work on the row tiles of one or two
//   vocabulary tiles, so each 1 MB slice of W is read from DRAM once and
//   reused from L2 by every row tile, and H (N·Hd·2 bytes) stays in L2.
//   warp 0     TMA producer: per 64-wide K step one [128][64] box of H and
//              one [256][64] box of W into a 4-stage ring (48 KB a stage);
//   warp 1     MMA issuer (one thread): z_tile += A·Bᵀ, M = 128, N = 256,
//              K = 16 per instruction, into one of two TMEM accumulators
//              (256 columns each), so the epilogue of one tile overlaps the
//              MMAs of the next;
//   warps 2..5 epilogue, one thread per row (= TMEM lane): reads the tile's
//              256 fp32 logits in 32-column pieces, masks columns >= V, and
//              keeps an online maximum m of z and rescaled sum
//              s = Σ 2^((z − m)·log2 e); picks the target's raw logit when the
//              target column falls in the tile. Writes (m, s) per (vocab
//              tile, row) and z_{t,y_t} to the workspace. The maximum stays in
//              natural units, so the rounding of log2 e only scales the
//              exponents' offsets from it and does not shift lse.
// lmhead_combine_kernel: per row, merges the nV partials in a fixed order
//   (M = max m_j, S = Σ s_j·e^(m_j − M)), lse = M + ln S, logp.
// The fixed-order loss reduction of the log-prob call follows.
//
// Backward (gradients of g·loss): dz_tv = g·w_t·(e^(z_tv − lse_t) − [v == y_t]),
// dH = dz·W, dW = dzᵀ·H. The same persistent kernel, templated on its
// epilogue and on the major-ness of its operands, runs three GEMMs:
//   dz  = H·Wᵀ with the epilogue above turned into dz (bf16, stored: the
//         3.85 GB gradient of the logits is the one array the backward keeps);
//   dH  = dz·W   (A = dz K-major; B = W read MN-major: [64 vocab rows][64
//         hidden columns] boxes, no transpose);
//   dW  = dzᵀ·H  (A = dz and B = H both read MN-major), fp32 output.
// dz is rounded to bf16 (by up to 2^-8 relative) because an MMA takes both
// operands of one 16-bit type, and W and H are bf16: kind::tf32 would run at
// half the rate on fp32 copies of all three. The rounding puts a relative L2
// error of 0.0016 on dH and dW, as much as their own rounding to bf16 does: at
// 4001 x 32,003 x 1024 the two are 0.0023 from 64 bits together, 0.0017 the
// outputs' alone. A second bf16 array with what the rounding drops would make
// the products dH and dW twice as long (161 + 169 us of the backward's 459)
// and dz's room twice as large. All sums are fp32.
// An MN-major operand is staged as [64 K rows][64 M-or-N columns] boxes with
// 128-byte swizzle: the UMMA descriptor's leading offset is one box (8 KB,
// the next 64 columns), its stride 1024 bytes (8 K rows), and each K = 16
// step advances 2048 bytes. Long sums (dH, dW, and dz of the backward with
// entropy; by_pairs) are made by pairs of CTAs: a tile of 256 x 256 on two
// SMs' tensor cores, each SM holding its 128 rows of A and half of B, 32 KB
// a K step instead of 48. The sums run in the same order: the same bits as
// without. The whole backward (dz, dH, dW) went 547 -> 470 us at 4001 x
// 32,003 x 1024, 16.1 -> 14.1 ms at 12,669 x 151,936 x 2048.
//
// With the entropy (tt_lmhead_token_logprob and its backward): the same
// kernel with two more epilogues. EPI_LSE_H carries u = Σ 2^x·x, x = (z −
// m)·log2 e, beside s; H = ln S − U/S of the joined sums. EPI_DZ_H forms dz =
// −p·(b + g_H·log p) + g_logp·[v == y] with b = g_logp − g_lse + g_H·H per row.
// The added sum costs the forward nothing: 12,669 x 151,936 x 2048 in 4.0 ms
// for a few passes and 4.3 under the power cap, where the log-prob alone takes
// 4.1 and 4.4 (its epilogue masks every column, this one only those of the
// last tile). An epilogue tile takes 2.2 us (EPI_DZ_H 2.8), so up to Hd = 256
// it bounds the GEMM, above it the tensor pipe (80 % busy at Hd = 1024).
#include <algorithm>
#include <atomic>

#include "tc_common.cuh"

namespace tt {
namespace {

using namespace tc;

// ------------------------------------------------------------------ a pair of CTAs (cta_group::2)
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A·B over both CTAs: each holds its rows of A and D and half the columns of B, at the same places.
__device__ __forceinline__ void umma_ss_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs once the tcgen05 operations issued so far by this thread complete.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// TMA load into this CTA's shared memory that signals a barrier of either CTA (an address of the cluster).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// An arrival on a barrier of either CTA. It carries no writes: the waiter takes tensor memory or a slot that was read.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A word for the other CTA, with the arrival on its barrier that the word completes.
__device__ __forceinline__ void send_u64(uint32_t addr, uint64_t v, uint32_t bar) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], 8;" ::"r"(bar) : "memory");
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];" ::"r"(addr), "l"(v), "r"(bar)
               : "memory");
}
// After a wait that the other CTA ended: what it sent is seen. (The phase is complete. A fence in its place waits for the
// warp's own stores too: the backward of 2048 x 65,536 x 2048 took 960 us with fences, 939 so.)
__device__ __forceinline__ void acquire_cluster(uint64_t* bar, uint32_t parity) {
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n}\n" ::"r"(
                   smem_u32(bar)),
               "r"(parity)
               : "memory");
}

constexpr int kLhWarps = 6;
constexpr int kBM = 128, kBN = 256, kBK = 64;
constexpr int kStages = 4;
constexpr uint32_t kABytes = kBM * kBK * 2;  // 16 KB
constexpr uint32_t kBBytes = kBN * kBK * 2;  // 32 KB
constexpr uint32_t kBox = 64 * 64 * 2;       // one [64 K rows][64 columns] box of an MN-major operand
constexpr uint32_t kTmemCols = 512;          // two [128][256] fp32 accumulators
constexpr float kLog2e = 1.4426950408889634f;

// Epilogues: per-row log-sum-exp partials (forward), dz (bf16), plain bf16 / fp32 stores; the partials with an
// entropy sum beside them, and dz of an objective of log-prob and entropy.
// EPI_PART: an fp32 partial product over one of `splits` ranges of K, each to a matrix of its own.
enum { EPI_LSE = 0, EPI_DZ = 1, EPI_BF16 = 2, EPI_F32 = 3, EPI_LSE_H = 4, EPI_DZ_H = 5, EPI_PART = 6 };
// What stands for a column >= V where an entropy is summed: far below any
// logit, and finite, so that 0·(z − m) is 0.
constexpr float kNoColumn = -1e30f;

// mbarriers: FULL[s] (TMA bytes landed), EMPTY[s] (MMAs reading stage s done),
// ACC_FULL[a] (accumulator a holds a finished tile), ACC_EMPTY[a] (the 128
// epilogue threads have read it), FINAL (every MMA of the CTA done).
// TILE_FULL[r] / TILE_EMPTY[r]: the tile index in ring slot r published by
// the producer / read by the MMA thread and the 128 epilogue threads.
// STALL: nothing arrives at it (LhArgs::stall_ns).
constexpr int kTileRing = 4;
template <int STAGES>
struct LhBars {
  static constexpr int FULL = 0, EMPTY = FULL + STAGES, ACC_FULL = EMPTY + STAGES, ACC_EMPTY = ACC_FULL + 2,
                       FINAL = ACC_EMPTY + 2, TILE_FULL = FINAL + 1, TILE_EMPTY = TILE_FULL + kTileRing,
                       STALL = TILE_EMPTY + kTileRing, NBAR = STALL + 1;
};
// A pair of CTAs (a cluster of two, tcgen05 cta_group::2) on one tile of 256
// rows: each holds its 128 rows of A and half the columns of B, so that a K
// step brings 32 KB into an SM instead of 48. The stages are as many as fit.
constexpr int kPairStages = 6;
constexpr int kPairSteps = 32, kPairStepsDz = 16;  // the least K steps to a tile (by_pairs)
constexpr uint32_t kPairBBytes = kBBytes / 2;
static_assert(kPairStages * (kABytes + kPairBBytes) == kStages * (kABytes + kBBytes) &&
                  LhBars<kStages>::NBAR <= LhBars<kPairStages>::NBAR, "one layout for both");

struct LhSmem {
  static constexpr uint32_t a0 = 0;
  static constexpr uint32_t bars = a0 + kStages * (kABytes + kBBytes);
  static constexpr uint32_t ring = bars + LhBars<kPairStages>::NBAR * 8;  // [kTileRing] int64 tile indices
  static constexpr uint32_t misc = ring + kTileRing * 8;
  static constexpr uint32_t total = misc + 16 + 1024;  // + slack for 1024-byte alignment
};
static_assert(LhSmem::total <= 232448, "LM-head shared memory exceeds the per-CTA limit");

struct LhArgs {
  int64_t M, Ncols;  // output rows and columns
  int ksteps;        // ceil(K / 64)
  int nM, nN;        // tiles along M and N
  int64_t tiles;     // nM · nN
  int n_outer;       // tile order: 1 = t -> (n = t / nM, m = t % nM), 0 = (m = t / nN, n = t % nN)
  int* counter;      // tiles claimed so far (zero at launch): CTAs take tiles as they free up; NULL = fixed stride
  const int32_t* targets;  // EPI_LSE, EPI_DZ (M = tokens, N = vocabulary)
  const float* weights;    // EPI_DZ: NULL = ones
  float g;                 // EPI_DZ
  const float* lse;        // EPI_DZ: per row, natural log
  float* pm;               // EPI_LSE: [nN][M] max of z over the tile's columns
  float* ps;               // EPI_LSE: [nN][M] Σ 2^((z − m)·log2 e)
  float* pz;               // EPI_LSE: [M] z_{t, y_t}
  __nv_bfloat16* ob;       // EPI_DZ, EPI_BF16: [M][ldo]
  float* of;               // EPI_F32: [M][ldo]
  int64_t ldo;
  int32_t* err;
  float* pu;             // EPI_LSE_H: [nN][M] Σ 2^x·x, x = (z − m)·log2 e
  const float* entropy;  // EPI_DZ_H, as the next three (each may be NULL): per row
  const float *dlogp, *dentropy, *dlse;
  bool rows32;  // all stores but EPI_DZ's: rows of ob or of begin on 32-byte boundaries (whole sectors to a store)
  int splits;   // EPI_PART: ranges of K (tiles = nM·nN·splits)
  int spread;   // EPI_LSE_H, EPI_DZ_H: A is a few rows laid out by K step, so many to a step (0: plain rows)
  // EPI_DZ_H, a test of the timeout path, 0 in normal calls: the MMA thread waits so long on STALL before the last K
  // step of its first tile, and gives up
  uint64_t stall_ns;
  uint64_t drain_ns;  // a test's limit of the second CTA's wait for FINAL (0: the normal one)
};

// 32 bytes in one store: a whole sector, which halves the L2 writes of a
// thread's row piece against two of 16 (dz of 4001 x 32,003: 202 -> 175 us).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// BN: columns of a tile (kBN, or half where whole tiles would leave most SMs without one).
template <int EPI, bool A_MN, bool B_MN, int BN, bool PAIR>
__global__ void __launch_bounds__(kLhWarps * 32, 1)
    lmhead_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const LhArgs a) {
  using L = LhSmem;
  constexpr bool kLse = EPI == EPI_LSE || EPI == EPI_LSE_H, kDz = EPI == EPI_DZ || EPI == EPI_DZ_H;
  constexpr bool kEnt = EPI == EPI_LSE_H || EPI == EPI_DZ_H;
  // PAIR: CTA 0 of the pair leads: its FULL barriers count both CTAs' copies, its MMA thread issues for both, its
  // ACC_EMPTY and TILE_EMPTY barriers take both CTAs' arrivals; EMPTY, ACC_FULL and FINAL are committed to both.
  constexpr int kStages = PAIR ? kPairStages : tt::kStages;
  constexpr uint32_t kBBytes = PAIR ? kPairBBytes : tt::kBBytes;
  constexpr uint32_t b0 = L::a0 + kStages * kABytes;
  constexpr int kTileM = PAIR ? 2 * kBM : kBM, kCtas = PAIR ? 2 : 1;
  constexpr int kOwnN = BN / kCtas;  // columns of B that a CTA holds
  using Bar = LhBars<kStages>;
  constexpr int FULL = Bar::FULL, EMPTY = Bar::EMPTY, ACC_FULL = Bar::ACC_FULL, ACC_EMPTY = Bar::ACC_EMPTY,
                FINAL = Bar::FINAL, TILE_FULL = Bar::TILE_FULL, TILE_EMPTY = Bar::TILE_EMPTY, STALL = Bar::STALL;
  const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;  // clusters are consecutive CTAs
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::misc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar[FULL + i], 1);
      mbar_init(&bar[EMPTY + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[ACC_FULL + i], 1);
      mbar_init(&bar[ACC_EMPTY + i], PAIR ? 2 * 4 : 128);  // PAIR: one arrival of each epilogue warp
    }
    mbar_init(&bar[FINAL], 1);
    mbar_init(&bar[STALL], 1);
    for (int i = 0; i < kTileRing; ++i) {
      mbar_init(&bar[TILE_FULL + i], 1);
      mbar_init(&bar[TILE_EMPTY + i], PAIR ? 2 * (1 + 4) : 1 + 128);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (PAIR)
      tmem_alloc_pair(tmem_slot, kTmemCols);
    else
      tmem_alloc(tmem_slot, kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_barrier();  // the leader's barriers are there before the other CTA's copies signal them
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const int64_t t_first = blockIdx.x / kCtas, t_step = gridDim.x / kCtas;
  // the leader's barrier (PAIR: as an address of the cluster)
  auto lead = [&](int b) { return dsmem_addr(smem_u32(&bar[b]), 0); };
  // the arrival of a thread, or (whole) of a warp whose lanes are all done
  auto arrive_lead = [&](int b, bool whole) {
    if constexpr (PAIR) {
      if (whole) __syncwarp();
      if (!whole || lane == 0) mbar_arrive_remote(lead(b));
    } else {
      mbar_arrive(&bar[b]);
    }
  };
  // a wait; PAIR: an epilogue warp's lanes give up together, so that its __syncwarp meets them all
  auto wait = [&](uint64_t* b, uint32_t parity, int site) {
    bool ok = mbar_wait(b, parity, abort_flag, site);
    if (PAIR && warp >= 2) ok = __all_sync(~0u, ok);
    return ok;
  };
  volatile int64_t* ring = reinterpret_cast<volatile int64_t*>(sm + L::ring);
  // the tile of this CTA's it-th turn (a value >= tiles ends the loop): with
  // a counter, published by the producer through the ring; else fixed stride
  auto take_tile = [&](int it, int64_t& t, int site) -> bool {
    if (!a.counter) {
      t = t_first + (int64_t)it * t_step;
      return true;
    }
    const int r = it % kTileRing;
    if (!wait(&bar[TILE_FULL + r], (uint32_t)((it / kTileRing) & 1), site)) return false;
    if (PAIR && rank != 0) acquire_cluster(&bar[TILE_FULL + r], (uint32_t)((it / kTileRing) & 1));
    t = ring[r];
    arrive_lead(TILE_EMPTY + r, /*whole=*/warp >= 2);
    return true;
  };
  // the K steps of a tile
  auto k_range = [&](int64_t t, int& k0, int& k1) {
    k0 = 0;
    k1 = a.ksteps;
    if (EPI == EPI_PART) {
      const int s = (int)(t / ((int64_t)a.nM * a.nN));
      k0 = (int)((int64_t)a.ksteps * s / a.splits);
      k1 = (int)((int64_t)a.ksteps * (s + 1) / a.splits);
    }
  };
  auto tile_mn = [&](int64_t t, int& m, int& n) {
    if (EPI == EPI_PART) t %= (int64_t)a.nM * a.nN;
    if (a.n_outer) {
      n = (int)(t / a.nM);
      m = (int)(t % a.nM);
    } else {
      m = (int)(t / a.nN);
      n = (int)(t % a.nN);
    }
  };

  // the [64][64] boxes of an MN-major B that hold columns (the last tile of Hd columns may have fewer than BN)
  // (A pair always takes all: columns past the last read 0.)
  auto tile_boxes = [&](int n) -> uint32_t {
    return PAIR ? kOwnN / 64 : (uint32_t)min((int64_t)(BN / 64), (a.Ncols - (int64_t)n * BN + 63) / 64);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      int64_t kk = 0;  // K steps issued by this CTA (ring position)
      bool ok = true;
      for (int it = 0; ok; ++it) {
        int64_t t = t_first + (int64_t)it * t_step;
        if (PAIR && rank != 0) {
          if (!take_tile(it, t, 8)) break;
        } else if (a.counter) {
          // claim the next tile and publish it to the MMA thread and the epilogue (PAIR: of both CTAs, and the other's
          // producer)
          const int r = it % kTileRing;
          if (it >= kTileRing &&
              !mbar_wait(&bar[TILE_EMPTY + r], (uint32_t)((it / kTileRing - 1) & 1), abort_flag, 5))
            break;
          t = (int64_t)atomicAdd(a.counter, 1);
          ring[r] = t;
          if constexpr (PAIR) {
            send_u64(dsmem_addr(smem_u32(const_cast<const int64_t*>(&ring[r])), 1), (uint64_t)t,
                     dsmem_addr(smem_u32(&bar[TILE_FULL + r]), 1));
          }
          mbar_arrive(&bar[TILE_FULL + r]);
        }
        if (t >= a.tiles) break;
        int m, n, k0, k1;
        tile_mn(t, m, n);
        k_range(t, k0, k1);
        const uint32_t boxes = tile_boxes(n);
        for (int ks = k0; ks < k1; ++ks, ++kk) {
          const int st = (int)(kk % kStages);
          if (kk >= kStages && !mbar_wait(&bar[EMPTY + st], (uint32_t)((kk / kStages - 1) & 1), abort_flag, 1)) {
            ok = false;
            break;
          }
          const bool spread = kEnt && a.spread;
          if (rank == 0)
            mbar_expect_tx(&bar[FULL + st], kCtas * ((spread ? a.spread * kBK * 2 : kABytes) +
                                                     (B_MN ? boxes * kBox : (uint32_t)kOwnN * kBK * 2)));
          uint8_t* sa = sm + L::a0 + st * kABytes;
          uint8_t* sb = sm + b0 + st * kBBytes;
          const int am = m * kTileM + rank * kBM, bn = n * BN + rank * kOwnN;  // this CTA's rows of A, columns of B
          auto load = [&](void* dst, const CUtensorMap* map, int x, int y) {
            if constexpr (PAIR)
              tma_load_2d_pair(dst, map, lead(FULL + st), x, y);
            else
              tma_load_2d(dst, map, &bar[FULL + st], x, y);
          };
          if (A_MN) {  // A stored [K][M]: two [64 K][64 M] boxes
#pragma unroll
            for (int i = 0; i < kBM / 64; ++i) load(sa + i * kBox, &tmA, am + 64 * i, ks * kBK);
          } else if (spread) {  // one [few rows][64 K] box; the tile's other rows give rows that nothing reads
            load(sa, &tmA, 0, ks * a.spread);
          } else {  // A stored [M][K]: one [128 M][64 K] box
            load(sa, &tmA, ks * kBK, am);
          }
          if (B_MN) {  // B stored [K][N]: up to four [64 K][64 N] boxes
#pragma unroll
            for (int i = 0; i < kOwnN / 64; ++i)
              if (i < boxes) load(sb + i * kBox, &tmB, bn + 64 * i, ks * kBK);
          } else {  // B stored [N][K]: one [BN, or half][64 K] box
            load(sb, &tmB, ks * kBK, bn);
          }
        }
      }
      // every copy issued has landed before the CTA may leave
      // (PAIR: the leader waits for both CTAs' copies, and neither leaves before the other)
      for (int64_t j = kk - 1; rank == 0 && j >= 0 && j >= kk - kStages; --j)
        mbar_drain(&bar[FULL + (int)(j % kStages)], (uint32_t)((j / kStages) & 1), abort_flag);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (PAIR: the leader's, for both)
    if (rank == 0 && lane == 0) {
      constexpr uint32_t whole = idesc_bf16(kTileM, BN, A_MN ? 1 : 0, B_MN ? 1 : 0);
      auto commit = [&](int b) {
        if constexpr (PAIR)
          umma_commit_pair(&bar[b]);
        else
          umma_commit(&bar[b]);
      };
      // K-major: 128-byte rows of K, 8-row groups 1024 bytes apart, K = 16 is 32 bytes on.
      // MN-major: 64-column boxes kBox apart, 8 K rows 1024 bytes apart, K = 16 is 2048 bytes on.
      const uint64_t da = A_MN ? smem_desc(smem_u32(sm + L::a0), kBox, 1024) : smem_desc(smem_u32(sm + L::a0), 16, 1024);
      const uint64_t db = B_MN ? smem_desc(smem_u32(sm + b0), kBox, 1024) : smem_desc(smem_u32(sm + b0), 16, 1024);
      constexpr uint32_t ka = A_MN ? 2048 : 32, kb = B_MN ? 2048 : 32;
      int64_t kk = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        int64_t t;
        if (!take_tile(it, t, 6) || t >= a.tiles) break;
        const int acc = it & 1;
        // the epilogue has read this accumulator's previous tile (it − 2)
        if (it >= 2 && !mbar_wait(&bar[ACC_EMPTY + acc], (uint32_t)(((it - 2) >> 1) & 1), abort_flag, 2)) break;
        tc_fence_after();
        const uint32_t dcol = tbase + (uint32_t)acc * BN;
        int k0, k1;
        k_range(t, k0, k1);
        uint32_t idesc = whole;
        if (B_MN && !PAIR) {  // N = the columns that are there
          int m, n;
          tile_mn(t, m, n);
          idesc = idesc_bf16(kBM, 64, A_MN ? 1 : 0, 1) + ((tile_boxes(n) - 1) * 64 / 8 << 17);
        }
        for (int ks = k0; ks < k1; ++ks, ++kk) {
          const int st = (int)(kk % kStages);
          if (!mbar_wait(&bar[FULL + st], (uint32_t)((kk / kStages) & 1), abort_flag, 3) ||
              (EPI == EPI_DZ_H && a.stall_ns && it == 0 && ks == k1 - 1 &&
               !mbar_wait(&bar[STALL], 0, abort_flag, 9, a.stall_ns))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            if constexpr (PAIR)
              umma_ss_pair(dcol, desc_at(da, st * kABytes + k * ka), desc_at(db, st * kBBytes + k * kb), idesc,
                           (ks > k0 || k > 0) ? 1u : 0u);
            else
              umma_ss(dcol, desc_at(da, st * kABytes + k * ka), desc_at(db, st * kBBytes + k * kb), idesc,
                      (ks > k0 || k > 0) ? 1u : 0u);
          commit(EMPTY + st);  // stage st free once these MMAs have read it
        }
        if (ok) commit(ACC_FULL + acc);
      }
      // completes after every MMA of this CTA (waited for even after an abort:
      // TMEM and shared memory must outlive the MMAs)
      commit(FINAL);
      mbar_drain(&bar[FINAL], 0, abort_flag);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int wq = warp & 3;  // TMEM lane quarter this warp may read
    const int rl = wq * 32 + lane;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    for (int it = 0;; ++it) {
      int64_t t;
      if (!take_tile(it, t, 7) || t >= a.tiles) break;
      const int acc = it & 1;
      int m, n;
      tile_mn(t, m, n);
      const int64_t row = (int64_t)m * kTileM + rank * kBM + rl;
      const int64_t c0 = (int64_t)n * BN;  // first column of the tile
      const bool row_ok = row < a.M;
      int y = -1;
      float gw = 0.f, lrow = 0.f;
      if (kLse || kDz) y = row_ok ? a.targets[row] : -1;
      float gh = 0.f, gb = 0.f;  // EPI_DZ_H: dz = −p·(gb + gh·log p) + gw·[column == target]
      if (kDz && row_ok) {
        if (kEnt) {
          gw = a.dlogp ? a.dlogp[row] : 0.f;
          gb = a.dlse ? gw - a.dlse[row] : gw;
          if (a.dentropy) {
            gh = a.dentropy[row];
            gb = fmaf(gh, a.entropy[row], gb);
          }
        } else {
          gw = a.g * (a.weights ? a.weights[row] : 1.f);
        }
        lrow = a.lse[row];
        if ((y < 0 || (int64_t)y >= a.Ncols) && n == 0) set_err(a.err, TT_ERR_INVALID_ARG);
      }
      const int64_t yc = (int64_t)y - c0;  // target column within the tile
      if (!wait(&bar[ACC_FULL + acc], (uint32_t)((it >> 1) & 1), 4)) break;
      tc_fence_after();
      float m_run = -INFINITY, s_run = 0.f, u_run = 0.f, zt = 0.f;
      bool found = false;
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        const int64_t col0 = c0 + c * 32;
        const int64_t nvalid = a.Ncols - col0;  // columns j < nvalid exist
        if ((B_MN || kEnt) && nvalid <= 0) break;
        uint32_t u[32];
        tmem_ld32(tbase + lane_base + (uint32_t)acc * BN + c * 32, u);
        tmem_ld_wait();
        tmem_pin(u);
        if (kLse) {
          float cm = -INFINITY;
          if (kEnt) {
            if (nvalid < 32) {  // the last tile
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j >= nvalid) u[j] = __float_as_uint(kNoColumn);
            }
#pragma unroll
            for (int j = 0; j < 32; j += 2) cm = fmax3f(cm, __uint_as_float(u[j]), __uint_as_float(u[j + 1]));
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float z = j < nvalid ? __uint_as_float(u[j]) : -INFINITY;
              u[j] = __float_as_uint(z);
              cm = fmaxf(cm, z);
            }
          }
          if ((uint64_t)(yc - c * 32) < 32u) {
            // u[jc] by a tree of selects on the bits of jc (no indexed register access)
            const int jc = (int)(yc - c * 32);
            uint32_t sel[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) sel[j] = (jc & 16) ? u[j + 16] : u[j];
#pragma unroll
            for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
              for (int j = 0; j < w; ++j) sel[j] = (jc & w) ? sel[j + w] : sel[j];
            zt = __uint_as_float(sel[0]);
            found = true;
          }
          const float nm = fmaxf(m_run, cm);
          if (kEnt || nm != -INFINITY) {
            // (With the entropy, columns that are NaN throughout have no maximum either, and must reach the sums.)
            const float ref = kEnt && nm == -INFINITY ? 0.f : nm;
            if (kEnt) {  // Σ 2^x·x around the new maximum (its offset kept finite while m_run is still -inf)
              const float dx = fmaxf((m_run - ref) * kLog2e, kNoColumn), f = fast_exp2(dx);
              u_run = fmaf(dx, s_run, u_run) * f;
              s_run *= f;
            } else {
              s_run *= fast_exp2((m_run - nm) * kLog2e);  // 0 while m_run is still -inf (s_run is 0 then)
            }
            const float2 l2 = make_float2(kLog2e, kLog2e), nn = make_float2(-ref, -ref);
            float2 acc2 = make_float2(0.f, 0.f), ent2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 x = __fmul2_rn(
                  __fadd2_rn(make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])), nn), l2);
              const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              acc2 = __fadd2_rn(acc2, e);
              if (kEnt) ent2 = __ffma2_rn(e, x, ent2);
            }
            s_run += acc2.x + acc2.y;
            if (kEnt) u_run += ent2.x + ent2.y;
            m_run = nm;
          }
        } else if (EPI == EPI_F32 || EPI == EPI_PART) {
          if (row_ok) {
            float* dst = a.of + row * a.ldo + col0;
            if (EPI == EPI_PART) dst += t / ((int64_t)a.nM * a.nN) * a.M * a.ldo;
            if (a.rows32) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (8 * q < nvalid) {
                  const uint32_t w8[8] = {u[8 * q],     u[8 * q + 1], u[8 * q + 2], u[8 * q + 3],
                                          u[8 * q + 4], u[8 * q + 5], u[8 * q + 6], u[8 * q + 7]};
                  store32(dst + 8 * q, w8);
                }
            } else
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (4 * q < nvalid)
                *reinterpret_cast<float4*>(dst + 4 * q) =
                    make_float4(__uint_as_float(u[4 * q]), __uint_as_float(u[4 * q + 1]), __uint_as_float(u[4 * q + 2]),
                                __uint_as_float(u[4 * q + 3]));
          }
        } else {
          if (EPI == EPI_DZ_H) {
            const float2 l2 = make_float2(kLog2e, kLog2e), nl = make_float2(-lrow, -lrow);
            const float2 nh = make_float2(-gh, -gh), nb = make_float2(-gb, -gb);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 lp = __fadd2_rn(make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])), nl);
              const float2 x = __fmul2_rn(lp, l2);
              const float2 dz = __fmul2_rn(make_float2(fast_exp2(x.x), fast_exp2(x.y)), __ffma2_rn(nh, lp, nb));
              u[2 * j] = __float_as_uint(dz.x);
              u[2 * j + 1] = __float_as_uint(dz.y);
            }
            if ((uint64_t)(yc - c * 32) < 32u) {
              const int jc = (int)(yc - c * 32);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == jc) u[j] = __float_as_uint(__uint_as_float(u[j]) + gw);
            }
          }
          if (EPI == EPI_DZ) {
            // dz = g·w·(e^(z − lse) − [column == target])
            const float2 l2 = make_float2(kLog2e, kLog2e), nl = make_float2(-lrow, -lrow);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 x = __fmul2_rn(
                  __fadd2_rn(make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])), nl), l2);
              u[2 * j] = __float_as_uint(gw * fast_exp2(x.x));
              u[2 * j + 1] = __float_as_uint(gw * fast_exp2(x.y));
            }
            if ((uint64_t)(yc - c * 32) < 32u) {
              const int jc = (int)(yc - c * 32);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == jc) u[j] = __float_as_uint(__uint_as_float(u[j]) - gw);
            }
          }
          if ((EPI == EPI_DZ_H || EPI == EPI_BF16) && a.rows32) {
            if (row_ok) {
              __nv_bfloat16* dst = a.ob + row * a.ldo + col0;
#pragma unroll
              for (int q = 0; q < 2; ++q)
                if (16 * q < nvalid) {
                  uint32_t w8[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    w8[i] = pack_bf16(__uint_as_float(u[16 * q + 2 * i]), __uint_as_float(u[16 * q + 2 * i + 1]));
                  store32(dst + 16 * q, w8);
                }
            }
          } else if (row_ok) {
            __nv_bfloat16* dst = a.ob + row * a.ldo + col0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (8 * q < nvalid) {
                uint4 w4;
                w4.x = pack_bf16(__uint_as_float(u[8 * q + 0]), __uint_as_float(u[8 * q + 1]));
                w4.y = pack_bf16(__uint_as_float(u[8 * q + 2]), __uint_as_float(u[8 * q + 3]));
                w4.z = pack_bf16(__uint_as_float(u[8 * q + 4]), __uint_as_float(u[8 * q + 5]));
                w4.w = pack_bf16(__uint_as_float(u[8 * q + 6]), __uint_as_float(u[8 * q + 7]));
                *reinterpret_cast<uint4*>(dst + 8 * q) = w4;
              }
          }
        }
      }
      tc_fence_before();
      arrive_lead(ACC_EMPTY + acc, true);
      if (kLse && row_ok) {
        a.pm[(int64_t)n * a.M + row] = m_run;
        a.ps[(int64_t)n * a.M + row] = s_run;
        if (kEnt) a.pu[(int64_t)n * a.M + row] = u_run;
        if (found) a.pz[row] = zt;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // the other CTA's tensor and shared memory are read and written, its barriers signalled, until here
  if constexpr (PAIR) {
    cluster_barrier();
    // The leader has seen its last MMAs complete; their arrival here must not find the CTA gone. (A wait from the
    // kernel's start would put its limit on the whole product, not on what is under way.)
    if (rank != 0 && threadIdx.x == 0) mbar_drain(&bar[FINAL], 0, abort_flag, a.drain_ns ? a.drain_ns : kWaitNs);
  }
  // every role has stopped: a wait that any of them gave up is seen (the producer alone is often done long before)
  if (*abort_flag && threadIdx.x == 0) set_err(a.err, TT_ERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tbase, kTmemCols);
    else
      tmem_dealloc(tbase, kTmemCols);
  }
}

// One persistent launch (one CTA per SM, at most one per tile).
template <int EPI, bool A_MN, bool B_MN, int BN = kBN>
int launch_gemm(const CUtensorMap& ta, const CUtensorMap& tb, const LhArgs& a, cudaStream_t st) {
  const int smem = (int)LhSmem::total;
  if (!smem_attr_set<lmhead_gemm_kernel<EPI, A_MN, B_MN, BN, false>>(smem)) return TT_ERR_CUDA;
  const int64_t grid = std::min<int64_t>(a.tiles, (int64_t)sm_count());
  {
    KtScope kt(TT_KT_LMHEAD, st);
    lmhead_gemm_kernel<EPI, A_MN, B_MN, BN, false><<<(unsigned)grid, kLhWarps * 32, smem, st>>>(ta, tb, a);
  }
  return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

// The same by pairs of CTAs, as many as are resident at once (a: tiles of 256 rows).
template <int EPI, bool A_MN, bool B_MN>
int launch_pairs(const CUtensorMap& ta, const CUtensorMap& tb, const LhArgs& a, cudaStream_t st) {
  constexpr auto kern = lmhead_gemm_kernel<EPI, A_MN, B_MN, kBN, true>;
  const int smem = (int)LhSmem::total;
  if (!smem_attr_set<kern>(smem)) return TT_ERR_CUDA;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kLhWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2);
  static std::atomic<int> resident[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return TT_ERR_CUDA;
  int pairs = resident[dev].load(std::memory_order_relaxed);
  if (pairs == 0) {
    if (cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg) != cudaSuccess || pairs < 1) return TT_ERR_CUDA;
    resident[dev].store(pairs, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(a.tiles, pairs)));
  cudaError_t e;
  {
    KtScope kt(TT_KT_LMHEAD, st);
    e = cudaLaunchKernelEx(&cfg, kern, ta, tb, a);
  }
  (void)cudaGetLastError();
  return cuda_status(e);
}

// Per row: M = max_j m_j, S = Σ_j s_j·e^(m_j − M) over the nV vocabulary
// tiles; lse = M + ln S, logp = z_{t,y_t} − lse. A target outside [0, V)
// sets err = TT_ERR_INVALID_ARG and that row's logp to NaN. A block takes 32
// rows (one per lane: consecutive rows, coalesced loads) and splits their
// tiles over kCombineWarps warps (warp w: tiles w, w + 8, ...); the warps'
// pairs are then merged in warp order, so the sums have a fixed order.
constexpr int kCombineWarps = 8;
__device__ __forceinline__ void lse_merge(float& M, float& S, float m, float s) {
  if (m > M) {
    S = S * expf(M - m) + s;
    M = m;
  } else if (m != -INFINITY) {
    S += s * expf(m - M);
  }
}
__global__ void __launch_bounds__(32 * kCombineWarps)
    lmhead_combine_kernel(const float* pm, const float* ps, const float* pz, int64_t N, int nV, int64_t V,
                          const int32_t* targets, float* logp, float* lse, int32_t* err) {
  __shared__ float2 part[kCombineWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  float M = -INFINITY, S = 0.f;
  if (row < N)
    for (int j = w; j < nV; j += kCombineWarps) lse_merge(M, S, pm[(int64_t)j * N + row], ps[(int64_t)j * N + row]);
  part[w][lane] = make_float2(M, S);
  __syncthreads();
  if (w != 0 || row >= N) return;
  M = -INFINITY;
  S = 0.f;
#pragma unroll
  for (int k = 0; k < kCombineWarps; ++k) lse_merge(M, S, part[k][lane].x, part[k][lane].y);
  const float l = M + logf(S);
  const int y = targets[row];
  float lp;
  if (y < 0 || (int64_t)y >= V) {
    set_err(err, TT_ERR_INVALID_ARG);
    lp = __int_as_float(0x7fc00000);
  } else {
    lp = pz[row] - l;
  }
  if (lse) lse[row] = l;
  logp[row] = lp;
}

// The same with the entropy: per row, (m, s, u) of the nV tiles joined around
// the row's maximum M as S = Σ s_j·f_j, U = Σ (u_j·ln 2 + (m_j − M)·s_j)·f_j,
// f_j = e^(m_j − M); H = ln S − U/S, lse = M + ln S, logp = (z_{t,y_t} − M) −
// ln S.
struct LhStat {
  float m, s, u;
};
__device__ __forceinline__ void stat_merge(LhStat& a, const LhStat& b) {
  const float M = fmaxf(a.m, b.m);
  if (M == -INFINITY) {  // nothing yet (0), or nothing but NaN
    a.s += b.s;
    return;
  }
  const float da = fmaxf(a.m - M, kNoColumn), db = fmaxf(b.m - M, kNoColumn);
  const float fa = expf(da), fb = expf(db);
  a.u = fmaf(da, a.s, a.u) * fa + fmaf(db, b.s, b.u) * fb;
  a.s = a.s * fa + b.s * fb;
  a.m = M;
}
// A block of 1024 threads takes ROWS consecutive rows and splits their tiles over 1024/ROWS threads each, four of a
// thread's tiles under way at once; the threads' sums are joined pairwise. (61 rows of 594 tiles: ROWS = 8 7 us, 32
// 10 us, one tile at a time over 8 warps 57 us.)
template <int ROWS>
__global__ void __launch_bounds__(1024)
    lmhead_combine_entropy_kernel(const float* pm, const float* ps, const float* pu, const float* pz, int64_t N, int nV,
                                  int64_t V, const int32_t* targets, float* logp, float* entropy, float* lse,
                                  int32_t* err) {
  constexpr int kShares = 1024 / ROWS;
  __shared__ LhStat part[kShares][ROWS];
  const int r = threadIdx.x % ROWS, w = threadIdx.x / ROWS;
  const int64_t row = (int64_t)blockIdx.x * ROWS + r;
  LhStat t = {-INFINITY, 0.f, 0.f};
  if (row < N)
    for (int j = w; j < nV; j += 4 * kShares) {
      LhStat p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ji = j + i * kShares;
        const int64_t at = (int64_t)ji * N + row;
        p[i] = ji < nV ? LhStat{pm[at], ps[at], pu[at]} : LhStat{-INFINITY, 0.f, 0.f};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i].u *= 0.6931471805599453f;
        stat_merge(t, p[i]);
      }
    }
  part[w][r] = t;
#pragma unroll
  for (int d = kShares / 2; d; d >>= 1) {
    __syncthreads();
    if (w < d) {
      stat_merge(t, part[w + d][r]);
      part[w][r] = t;
    }
  }
  if (w != 0 || row >= N) return;
  const float log_s = logf(t.s);
  const float h = log_s - t.u / t.s;
  entropy[row] = h < 0.f ? 0.f : h;
  lse[row] = t.m + log_s;
  const int y = targets[row];
  if (y < 0 || (int64_t)y >= V) {
    set_err(err, TT_ERR_INVALID_ARG);
    logp[row] = __int_as_float(0x7fc00000);
  } else {
    logp[row] = (pz[row] - t.m) - log_s;
  }
}

// A few rows of H laid out for the GEMM's CTAs, which all read the same ones: [K step][row][64] with each row of 128
// bytes kSpreadPitch after the one before. Close together they lie in few slices of the L2 cache, whose queues then
// hold up the reads of W as well (1 x 151,936 x 2048: 134 us, spread 99; 16 rows 116 and 101; from 32 rows on there is
// no difference). Only where reading W takes long enough (134 MB, about 20 us) to pay for the copy's launch.
constexpr int kSpreadRows = 31;
constexpr int64_t kSpreadW = 1 << 26;  // entries of W
constexpr int kSpreadPitch = 4096 + 128;
inline int spread_rows(int64_t N, int64_t V, int Hd) {
  return N <= kSpreadRows && V * Hd >= kSpreadW ? (int)((N + 7) / 8 * 8) : 0;
}
inline size_t spread_bytes(int64_t N, int64_t V, int Hd) {
  return (size_t)spread_rows(N, V, Hd) * (size_t)(Hd / kBK) * kSpreadPitch;
}
__global__ void __launch_bounds__(256) lmhead_spread_kernel(const __nv_bfloat16* h, int N, int Hd, int rows, char* out) {
  const int i = blockIdx.x * 256 + threadIdx.x;  // 16-byte vectors: 8 to a row of a step
  if (i >= Hd / kBK * rows * 8) return;
  const int line = i / 8, ks = line / rows, r = line - ks * rows;
  const uint4 v = r < N ? *reinterpret_cast<const uint4*>(h + (int64_t)r * Hd + ks * kBK + (i % 8) * 8)
                        : make_uint4(0, 0, 0, 0);
  *reinterpret_cast<uint4*>(out + (int64_t)line * kSpreadPitch + (i % 8) * 16) = v;
}

struct LhWs {
  size_t pm, ps, pz, total;
  size_t pu, spread, total_u;  // with the entropy sums and the spread rows behind the rest
};
// Tiles of half the columns for the z product where whole ones would not give half the SMs (of kSplitSms) one each:
// 374 x 2150 x 1728, 27 tiles: 15.5 us, with 51 half tiles 13.1; 28 x 14,782 x 448, 58 tiles: 9.6 and 8.9.
constexpr int kSplitSms = 152;
inline bool half_tiles(int64_t N, int64_t V) {
  return (N + kBM - 1) / kBM * ((V + kBN - 1) / kBN) <= kSplitSms / 2;
}
LhWs lh_layout(int64_t N, int64_t V, int Hd = 0, int BN = kBN) {
  const int64_t nV = (V + BN - 1) / BN;
  LhWs w;
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t r = o; o = align_up(o + bytes, 256); return r; };
  w.pm = take(sizeof(float) * (size_t)nV * (size_t)N);
  w.ps = take(sizeof(float) * (size_t)nV * (size_t)N);
  w.pz = take(sizeof(float) * (size_t)N);
  w.total = o;
  w.pu = take(sizeof(float) * (size_t)nV * (size_t)N);
  w.spread = take(spread_bytes(N, V, Hd));
  w.total_u = o;
  return w;
}

// The sum of a split product's parts [splits][n], to bf16 (n a multiple of 4). Four entries to a thread; WARPS > 1: the
// warps of a block share the parts of 128 entries, and their sums are joined in warp order. Many parts (then there are
// few entries): 16 warps, 3 x 384 entries of 152 parts 4.0 us, with one 21; few parts: one, 374 x 1728 entries of 4
// parts 4.7 us, with 16 11.8.
template <int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 256 : 32 * WARPS)
    lmhead_sum_parts_kernel(const float* part, int64_t n, int splits, __nv_bfloat16* out) {
  __shared__ float4 sums[WARPS][32];
  const int lane = threadIdx.x & 31, w = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const int64_t i = (WARPS == 1 ? (int64_t)blockIdx.x * 256 + threadIdx.x : (int64_t)blockIdx.x * 32 + lane) * 4;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < n) {
#pragma unroll 4
    for (int s = w; s < splits; s += WARPS) {
      const float4 p = *reinterpret_cast<const float4*>(part + s * n + i);
      t.x += p.x; t.y += p.y; t.z += p.z; t.w += p.w;
    }
  }
  if constexpr (WARPS > 1) {
    sums[w][lane] = t;
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int k = 1; k < WARPS; ++k) {
      const float4 p = sums[k][lane];
      t.x += p.x; t.y += p.y; t.z += p.z; t.w += p.w;
    }
  }
  if (i < n) *reinterpret_cast<uint2*>(out + i) = make_uint2(pack_bf16(t.x, t.y), pack_bf16(t.z, t.w));
}

}  // namespace
}  // namespace tt

using namespace tt;

TT_API size_t tt_lmhead_logprob_workspace_bytes(int64_t N, int64_t V) {
  if (N < 1 || V < 1) return 0;
  return lh_layout(N, V).total;
}

namespace {
// Whether pairs of CTAs take a product [M][Ncols] with `steps` K steps: where a tile's sum is long enough (`least` steps)
// and tiles of 256 rows need no more than 7/6 of the waves. With pairs the full GPU takes 680 to 700 cycles a K step
// whichever the product (32 KB from L2 for each SM: 12 to 14 TB/s), a CTA alone 736 (dH), 829 (dW), 762 (dz), 655 (the forward,
// where SMs that want the same lines at the same time get them once). 4001 x 32,003 x 1024: dH 196 -> 161 us, dW 195 ->
// 169 (from kPairSteps on), dz 180 -> 164 (from 16 steps on; 9000 x 4001 x 512, 8 steps: the backward 115 -> 117). The
// forward is not made by pairs: 157 -> 164 us there, 313 -> 305 at 2048 x 65,536 x 2048, 4.1 -> 4.4 ms at 12,669 x 151,936.
// path: a test's choice (kByRule: this rule; one or the other wherever it can).
enum { kByRule = 0, kSingles = 1, kPairs = 2 };
bool by_pairs(int path, int64_t M, int64_t Ncols, int64_t steps, int64_t least) {
  const int64_t cols = (Ncols + kBN - 1) / kBN, sms = sm_count();
  if (M <= kBM || sms < 2 || path == kSingles) return false;
  if (path == kPairs) return true;
  if (steps < least) return false;
  const int64_t one = (M + kBM - 1) / kBM * cols, two = (M + 2 * kBM - 1) / (2 * kBM) * cols;
  return ((two + sms / 2 - 1) / (sms / 2)) * 6 <= ((one + sms - 1) / sms) * 7;
}

LhArgs lh_args(int64_t M, int64_t Ncols, int64_t K, int n_outer, int32_t* err, int BN = kBN, int BM = kBM) {
  LhArgs a = {};
  a.M = M; a.Ncols = Ncols; a.ksteps = (int)((K + kBK - 1) / kBK);
  a.nM = (int)((M + BM - 1) / BM);
  a.nN = (int)((Ncols + BN - 1) / BN);
  a.tiles = (int64_t)a.nM * a.nN;
  a.n_outer = n_outer;
  a.err = err;
  return a;
}
int lh_check(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V, int Hd, const int32_t* targets,
             const int32_t* err) {
  if (!hidden || !w_vocab || !targets || !err || N < 1 || V < 1 || Hd < 1) return TT_ERR_INVALID_ARG;
  if (Hd % kBK != 0) return TT_ERR_UNSUPPORTED;
  if (N > (int64_t)INT32_MAX - kBM || V > (int64_t)INT32_MAX - kBN) return TT_ERR_INVALID_ARG;
  if (!aligned16(hidden) || !aligned16(w_vocab)) return TT_ERR_INVALID_ARG;
  return TT_OK;
}
}  // namespace

TT_API int tt_lmhead_logprob(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V, int Hd,
                             const int32_t* targets, const float* weights, float* logp, float* lse, double* loss,
                             void* ws, size_t ws_bytes, int32_t* err, tt_stream_t stream) {
  int rc = lh_check(hidden, w_vocab, N, V, Hd, targets, err);
  if (rc) return rc;
  if (!logp || !loss || !ws || !aligned16(ws)) return TT_ERR_INVALID_ARG;
  const LhWs Lw = lh_layout(N, V);
  if (ws_bytes < Lw.total) return TT_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap mh, mw;
  if (!make_tmap_bf16(&mh, hidden, (uint64_t)Hd, (uint64_t)N, kBM) ||
      !make_tmap_bf16(&mw, w_vocab, (uint64_t)Hd, (uint64_t)V, kBN))
    return TT_ERR_CUDA;
  // z = H·Wᵀ: M = tokens, columns = vocabulary, K = Hd; vocabulary-major tiles
  LhArgs a = lh_args(N, V, Hd, 1, err);
  a.targets = targets;
  a.pm = ws_at<float>(ws, Lw.pm);
  a.ps = ws_at<float>(ws, Lw.ps);
  a.pz = ws_at<float>(ws, Lw.pz);
  // 58,806 equal tiles at the benchmarked shape: a fixed stride leaves no tail
  rc = launch_gemm<EPI_LSE, false, false>(mh, mw, a, st);
  if (rc) return rc;
  lmhead_combine_kernel<<<(unsigned)((N + 31) / 32), 32 * kCombineWarps, 0, st>>>(a.pm, a.ps, a.pz, N, a.nN, V,
                                                                                 targets, logp, lse, err);
  TT_LAUNCH_CHECK();
  return cuda_status(launch_weighted_loss(logp, weights, N, loss, st));
}

// dz [N][ldz] bf16 with ldz = V rounded up to 8 (16-byte rows for the tensor maps).
static inline int64_t dz_ld(int64_t V) { return (V + 7) / 8 * 8; }

// Backward scratch: dz, then the three GEMMs' tile counters.
static inline size_t dz_bytes(int64_t N, int64_t V) { return align_up((size_t)N * (size_t)dz_ld(V) * 2, 256); }

TT_API size_t tt_lmhead_logprob_bwd_workspace_bytes(int64_t N, int64_t V) {
  if (N < 1 || V < 1) return 0;
  return dz_bytes(N, V) + 256;
}

namespace {
// Whether pairs make dH and dW. (A tile by pairs has no columns left out; a split dH is made by single CTAs.)
bool pairs_dh(int path, int64_t N, int64_t V, int Hd, int splits) {
  return Hd % kBN == 0 && splits == 1 && by_pairs(path, N, Hd, V / kBK, kPairSteps);
}
bool pairs_dw(int path, int64_t N, int64_t V, int Hd) {
  return Hd % kBN == 0 && by_pairs(path, V, Hd, N / kBK, kPairSteps);
}
// Whether a product [M][Ncols] has more tiles (of BN columns, in `splits` parts) than CTAs, or pairs, that run at once.
bool has_waves(int64_t M, int64_t Ncols, int BN, bool pairs, int splits) {
  const int64_t rows = pairs ? 2 * kBM : kBM;
  return (M + rows - 1) / rows * ((Ncols + BN - 1) / BN) * splits > sm_count() / (pairs ? 2 : 1);
}

// Rows of `bytes` bytes from p begin on 32-byte boundaries.
bool rows_on_32(const void* p, int64_t bytes) { return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)bytes) % 32 == 0; }

// dH = dz·W (bf16) and dW = dzᵀ·H (fp32, or bf16 with dw_dtype = TT_DT_BF16) from dz [N][ldz]; ctr[1], ctr[2]: their
// tile counters (0 at launch; ctr NULL: tiles at a fixed stride). parts: room for `splits` fp32 matrices [N][Hd] where
// dH's sum over the vocabulary is to be split (splits > 1). fork: dW on a second stream beside dH.
int lh_products(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V, int Hd, const __nv_bfloat16* dz,
                int64_t ldz, int* ctr, tt_bf16* d_hidden, void* d_w_vocab, int dw_dtype, float* parts, int splits,
                bool fork_dw, int path, int32_t* err, cudaStream_t st) {
  // 2. dH = dz·W: A = dz [N][V] (K-major, K = V); B = W [V][Hd] read MN-major; token-major tiles
  CUtensorMap mdz, mw_mn;
  if (!make_tmap_bf16_ld(&mdz, dz, (uint64_t)V, (uint64_t)N, (uint64_t)ldz, kBM) ||
      !make_tmap_bf16(&mw_mn, w_vocab, (uint64_t)Hd, (uint64_t)V, 64))
    return TT_ERR_CUDA;
  const bool dh_pairs = pairs_dh(path, N, V, Hd, splits), dw_pairs = pairs_dw(path, N, V, Hd);
  LhArgs b = lh_args(N, Hd, V, 0, err, kBN, dh_pairs ? 2 * kBM : kBM);
  b.ob = reinterpret_cast<__nv_bfloat16*>(d_hidden); b.ldo = Hd; b.counter = ctr ? ctr + 1 : nullptr;
  b.rows32 = rows_on_32(b.ob, 2 * Hd);
  if (splits > 1) {
    b.of = parts;
    b.rows32 = rows_on_32(parts, 4 * Hd);
    b.splits = splits;
    b.tiles *= splits;
  }
  // 3. dW = dzᵀ·H: A = dz read MN-major ([K = tokens][M = vocabulary]), B = H [N][Hd] read MN-major
  CUtensorMap mdz_mn, mh_mn;
  if (!make_tmap_bf16_ld(&mdz_mn, dz, (uint64_t)V, (uint64_t)N, (uint64_t)ldz, 64) ||
      !make_tmap_bf16(&mh_mn, hidden, (uint64_t)Hd, (uint64_t)N, 64))
    return TT_ERR_CUDA;
  LhArgs c = lh_args(V, Hd, N, 0, err, kBN, dw_pairs ? 2 * kBM : kBM);
  const bool dw_bf16 = dw_dtype == TT_DT_BF16;
  if (dw_bf16)
    c.ob = static_cast<__nv_bfloat16*>(d_w_vocab);
  else
    c.of = static_cast<float*>(d_w_vocab);
  c.rows32 = rows_on_32(d_w_vocab, (dw_bf16 ? 2 : 4) * Hd);
  c.ldo = Hd; c.counter = ctr ? ctr + 2 : nullptr;
  // dH and dW both only read dz: dW runs on a second stream forked after dz,
  // so that its CTAs (which claim tiles as they free up) take the SMs that
  // dH's last round of tiles (792 tiles of K = V at the benchmarked shape,
  // 5.2 per SM) leaves idle; joined back before returning. Not while the
  // caller's stream is being captured into a graph (the second stream is
  // destroyed here, before such a capture would end).
  cudaStream_t side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  const bool two = fork_dw && cudaStreamIsCapturing(st, &cap) == cudaSuccess && cap == cudaStreamCaptureStatusNone &&
                   cudaStreamCreateWithFlags(&side, cudaStreamNonBlocking) == cudaSuccess &&
                   cudaEventCreateWithFlags(&fork, cudaEventDisableTiming) == cudaSuccess &&
                   cudaEventCreateWithFlags(&join, cudaEventDisableTiming) == cudaSuccess &&
                   cudaEventRecord(fork, st) == cudaSuccess && cudaStreamWaitEvent(side, fork, 0) == cudaSuccess;
  if (!two) (void)cudaGetLastError();
  int rc = splits > 1 ? launch_gemm<EPI_PART, false, true>(mdz, mw_mn, b, st)
           : dh_pairs ? launch_pairs<EPI_BF16, false, true>(mdz, mw_mn, b, st)
                      : launch_gemm<EPI_BF16, false, true>(mdz, mw_mn, b, st);
  if (!rc && splits > 1) {
    const int64_t n = N * Hd;
    if (splits >= 16)
      lmhead_sum_parts_kernel<16><<<(unsigned)((n + 127) / 128), 512, 0, st>>>(parts, n, splits, b.ob);
    else
      lmhead_sum_parts_kernel<1><<<(unsigned)((n / 4 + 255) / 256), 256, 0, st>>>(parts, n, splits, b.ob);
    if (cudaGetLastError() != cudaSuccess) rc = TT_ERR_CUDA;
  }
  int rc2 = rc;
  if (!rc)
    rc2 = dw_pairs ? (dw_bf16 ? launch_pairs<EPI_BF16, true, true>(mdz_mn, mh_mn, c, two ? side : st)
                              : launch_pairs<EPI_F32, true, true>(mdz_mn, mh_mn, c, two ? side : st))
          : dw_bf16 ? launch_gemm<EPI_BF16, true, true>(mdz_mn, mh_mn, c, two ? side : st)
                    : launch_gemm<EPI_F32, true, true>(mdz_mn, mh_mn, c, two ? side : st);
  if (two && (cudaEventRecord(join, side) != cudaSuccess || cudaStreamWaitEvent(st, join, 0) != cudaSuccess))
    rc2 = rc2 ? rc2 : TT_ERR_CUDA;
  if (join) cudaEventDestroy(join);
  if (fork) cudaEventDestroy(fork);
  if (side) cudaStreamDestroy(side);
  return rc ? rc : rc2;
}
}  // namespace

TT_API int tt_lmhead_logprob_bwd(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V, int Hd,
                                 const int32_t* targets, const float* weights, float g, const float* lse,
                                 tt_bf16* d_hidden, float* d_w_vocab, void* ws, size_t ws_bytes, int32_t* err,
                                 tt_stream_t stream) {
  int rc = lh_check(hidden, w_vocab, N, V, Hd, targets, err);
  if (rc) return rc;
  if (!lse || !d_hidden || !d_w_vocab || !ws || !aligned16(ws) || !aligned16(d_hidden) || !aligned16(d_w_vocab))
    return TT_ERR_INVALID_ARG;
  if (ws_bytes < tt_lmhead_logprob_bwd_workspace_bytes(N, V)) return TT_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(ws);
  const int64_t ldz = dz_ld(V);
  int* ctr = ws_at<int>(ws, dz_bytes(N, V));  // [3]: dz, dH, dW
  if (cudaMemsetAsync(ctr, 0, 3 * sizeof(int), st) != cudaSuccess) return TT_ERR_CUDA;
  // 1. dz = g·w·(softmax(H·Wᵀ) − onehot): the forward's tiles with the dz epilogue
  CUtensorMap mh, mw;
  if (!make_tmap_bf16(&mh, hidden, (uint64_t)Hd, (uint64_t)N, kBM) ||
      !make_tmap_bf16(&mw, w_vocab, (uint64_t)Hd, (uint64_t)V, kBN))
    return TT_ERR_CUDA;
  LhArgs a = lh_args(N, V, Hd, 1, err);
  a.targets = targets; a.weights = weights; a.g = g; a.lse = lse; a.ob = dz; a.ldo = ldz; a.counter = ctr;
  rc = launch_gemm<EPI_DZ, false, false>(mh, mw, a, st);
  if (rc) return rc;
  return lh_products(hidden, w_vocab, N, V, Hd, dz, ldz, ctr, d_hidden, d_w_vocab, TT_DT_F32, nullptr, 1, true,
                     kByRule, err, st);
}

namespace {
// The tensor map of H for the z product: plain rows, or the few rows spread into `room` first.
int map_hidden(const tt_bf16* hidden, int64_t N, int64_t V, int Hd, void* room, LhArgs* a, CUtensorMap* map, cudaStream_t st) {
  a->spread = spread_rows(N, V, Hd);
  if (!a->spread)
    return make_tmap_bf16(map, hidden, (uint64_t)Hd, (uint64_t)N, kBM) ? TT_OK : TT_ERR_CUDA;
  const int lines = Hd / kBK * a->spread;
  lmhead_spread_kernel<<<(lines * 8 + 255) / 256, 256, 0, st>>>(reinterpret_cast<const __nv_bfloat16*>(hidden), (int)N,
                                                               Hd, a->spread, static_cast<char*>(room));
  if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
  return make_tmap_bf16_ld(map, room, kBK, (uint64_t)lines, kSpreadPitch / 2, (uint32_t)a->spread) ? TT_OK : TT_ERR_CUDA;
}
}  // namespace

TT_API size_t tt_lmhead_token_logprob_workspace_bytes(int64_t N, int64_t V, int Hd) {
  if (N < 1 || V < 1 || Hd < 1) return 0;
  return lh_layout(N, V, Hd, half_tiles(N, V) ? kBN / 2 : kBN).total_u;
}

TT_API int tt_lmhead_token_logprob(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V, int Hd,
                                   const int32_t* targets, float* logp, float* entropy, float* lse, void* ws,
                                   size_t ws_bytes, int32_t* err, tt_stream_t stream) {
  int rc = lh_check(hidden, w_vocab, N, V, Hd, targets, err);
  if (rc) return rc;
  if (!logp || !entropy || !lse || !ws || !aligned16(ws)) return TT_ERR_INVALID_ARG;
  const bool half = half_tiles(N, V);
  const int BN = half ? kBN / 2 : kBN;
  const LhWs Lw = lh_layout(N, V, Hd, BN);
  if (ws_bytes < Lw.total_u) return TT_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  CUtensorMap mh, mw;
  if (!make_tmap_bf16(&mw, w_vocab, (uint64_t)Hd, (uint64_t)V, BN)) return TT_ERR_CUDA;
  LhArgs a = lh_args(N, V, Hd, 1, err, BN);
  if ((rc = map_hidden(hidden, N, V, Hd, ws_at<char>(ws, Lw.spread), &a, &mh, st)) != TT_OK) return rc;
  a.targets = targets;
  a.pm = ws_at<float>(ws, Lw.pm);
  a.ps = ws_at<float>(ws, Lw.ps);
  a.pz = ws_at<float>(ws, Lw.pz);
  a.pu = ws_at<float>(ws, Lw.pu);
  rc = half ? launch_gemm<EPI_LSE_H, false, false, kBN / 2>(mh, mw, a, st)
            : launch_gemm<EPI_LSE_H, false, false>(mh, mw, a, st);
  if (rc) return rc;
  const int rows = N <= 512 ? 8 : 32;
  auto* combine = rows == 8 ? lmhead_combine_entropy_kernel<8> : lmhead_combine_entropy_kernel<32>;
  combine<<<(unsigned)((N + rows - 1) / rows), 1024, 0, st>>>(a.pm, a.ps, a.pu, a.pz, N, a.nN, V, targets, logp, entropy,
                                                             lse, err);
  TT_LAUNCH_CHECK();
  return TT_OK;
}

namespace {
// Scratch of the backward with entropy: dz [N][ldz] (rows on 32-byte
// boundaries), the tile counters, and the parts of a split dH. dH = dz·W has
// ceil(N/128)·ceil(Hd/256) tiles, each a sum over the whole vocabulary: where
// these are few the sum is split so that about every SM has a part, of 8 K
// steps or more (61 x 151,936 x 2048: 8 tiles alone take 790 us). The split
// goes by sizes alone, on any device as on one of kSplitSms SMs: the
// workspace and the order of the sums do not depend on the device.
struct LhBwdWs {
  int64_t ldz;
  int splits;
  size_t ctr, spread, parts, total;
};
LhBwdWs lh_bwd_layout(int64_t N, int64_t V, int Hd) {
  LhBwdWs w;
  w.ldz = (V + 15) / 16 * 16;
  const int64_t tiles = (N + kBM - 1) / kBM * ((Hd + kBN - 1) / kBN), ksteps = (V + kBK - 1) / kBK;
  w.splits = (int)std::max<int64_t>(1, std::min<int64_t>(kSplitSms / tiles, ksteps / 8));
  w.ctr = align_up((size_t)N * (size_t)w.ldz * 2, 256);
  w.spread = w.ctr + 256;
  w.parts = w.spread + align_up(spread_bytes(N, V, Hd), 256);
  w.total = w.parts + (w.splits > 1 ? sizeof(float) * (size_t)w.splits * (size_t)N * (size_t)Hd : 0);
  return w;
}
}  // namespace

TT_API size_t tt_lmhead_token_logprob_bwd_workspace_bytes(int64_t N, int64_t V, int Hd) {
  if (N < 1 || V < 1 || Hd < 1) return 0;
  return lh_bwd_layout(N, V, Hd).total;
}

namespace {
int token_logprob_bwd(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V, int Hd,
                      const int32_t* targets, const float* lse, const float* entropy, const float* dlogp,
                      const float* dentropy, const float* dlse, tt_bf16* d_hidden, void* d_w_vocab, int dw_dtype,
                      void* ws, size_t ws_bytes, int path, uint64_t stall_ns, uint64_t drain_ns, int32_t* err,
                      tt_stream_t stream) {
  int rc = lh_check(hidden, w_vocab, N, V, Hd, targets, err);
  if (rc) return rc;
  if (!lse || (dentropy && !entropy) || !d_hidden || !d_w_vocab || !ws || !aligned16(ws) || !aligned16(d_hidden) ||
      !aligned16(d_w_vocab) || (dw_dtype != TT_DT_F32 && dw_dtype != TT_DT_BF16))
    return TT_ERR_INVALID_ARG;
  const LhBwdWs Lw = lh_bwd_layout(N, V, Hd);
  if (ws_bytes < Lw.total) return TT_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(ws);
  int* ctr = ws_at<int>(ws, Lw.ctr);  // [3]: dz, dH, dW
  CUtensorMap mh, mw;
  const bool half = half_tiles(N, V);
  const int BN = half ? kBN / 2 : kBN;
  const bool pairs = !half && by_pairs(path, N, V, Hd / kBK, kPairStepsDz);
  if (!make_tmap_bf16(&mw, w_vocab, (uint64_t)Hd, (uint64_t)V, pairs ? kBN / 2 : BN)) return TT_ERR_CUDA;
  LhArgs a = lh_args(N, V, Hd, 1, err, BN, pairs ? 2 * kBM : kBM);
  if ((rc = map_hidden(hidden, N, V, Hd, ws_at<char>(ws, Lw.spread), &a, &mh, st)) != TT_OK) return rc;
  // a product with a tile or less to a CTA (pair) needs no claims, and leaves no last round of tiles for dW to run
  // beside: where all three are such, no counters and no second stream
  if (!has_waves(N, V, BN, pairs, 1) && !has_waves(N, Hd, kBN, pairs_dh(path, N, V, Hd, Lw.splits), Lw.splits) &&
      !has_waves(V, Hd, kBN, pairs_dw(path, N, V, Hd), 1))
    ctr = nullptr;
  else if (cudaMemsetAsync(ctr, 0, 3 * sizeof(int), st) != cudaSuccess)
    return TT_ERR_CUDA;
  a.targets = targets; a.lse = lse; a.entropy = entropy; a.dlogp = dlogp; a.dentropy = dentropy; a.dlse = dlse;
  a.ob = dz; a.ldo = Lw.ldz; a.counter = ctr; a.rows32 = rows_on_32(dz, 2 * Lw.ldz);
  a.stall_ns = stall_ns;
  a.drain_ns = drain_ns;
  rc = pairs ? launch_pairs<EPI_DZ_H, false, false>(mh, mw, a, st)
       : half ? launch_gemm<EPI_DZ_H, false, false, kBN / 2>(mh, mw, a, st)
              : launch_gemm<EPI_DZ_H, false, false>(mh, mw, a, st);
  if (rc) return rc;
  return lh_products(hidden, w_vocab, N, V, Hd, dz, Lw.ldz, ctr, d_hidden, d_w_vocab, dw_dtype,
                     ws_at<float>(ws, Lw.parts), Lw.splits, /*fork_dw=*/Lw.splits == 1 && ctr, path, err, st);
}
}  // namespace

TT_API int tt_lmhead_token_logprob_bwd(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V, int Hd,
                                       const int32_t* targets, const float* lse, const float* entropy,
                                       const float* dlogp, const float* dentropy, const float* dlse,
                                       tt_bf16* d_hidden, void* d_w_vocab, int dw_dtype, void* ws, size_t ws_bytes,
                                       int32_t* err, tt_stream_t stream) {
  return token_logprob_bwd(hidden, w_vocab, N, V, Hd, targets, lse, entropy, dlogp, dentropy, dlse, d_hidden, d_w_vocab,
                           dw_dtype, ws, ws_bytes, kByRule, 0, 0, err, stream);
}

TT_API int tt_lmhead_token_logprob_bwd_path_test(const tt_bf16* hidden, const tt_bf16* w_vocab, int64_t N, int64_t V,
                                                 int Hd, const int32_t* targets, const float* lse, const float* entropy,
                                                 const float* dlogp, const float* dentropy, const float* dlse,
                                                 tt_bf16* d_hidden, void* d_w_vocab, int dw_dtype, void* ws,
                                                 size_t ws_bytes, int path, int64_t stall_ns, int64_t drain_ns,
                                                 int32_t* err, tt_stream_t stream) {
  constexpr int64_t kMost = 10000000000LL;
  if (path < kByRule || path > kPairs || stall_ns < 0 || stall_ns > kMost || drain_ns < 0 || drain_ns > kMost)
    return TT_ERR_INVALID_ARG;
  return token_logprob_bwd(hidden, w_vocab, N, V, Hd, targets, lse, entropy, dlogp, dentropy, dlse, d_hidden, d_w_vocab,
                           dw_dtype, ws, ws_bytes, path, (uint64_t)stall_ns, (uint64_t)drain_ns, err, stream);
}
