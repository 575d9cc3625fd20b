// Clipped policy objective with a KL term and an entropy bonus over the tokens
// of rollout trees, from per-token log-probs, or from logits together with the
// gradient with respect to them.
//
//   r = e^{logp − old},  x = ref − logp
//   L = Σ_t w·( −gain·min(r, 1 + ε_hi) + cost·min(max(r, 1 − ε_lo), c) + β·(e^x − 1 − x) − γ·H )
//   dlogp = g·w·( −gain·r·[r <= 1 + ε_hi] + cost·r·[1 − ε_lo <= r <= c] − β·(e^x − 1) ),   dH = −g·w·γ
//   dz_v = p_v·(−dlogp − dH·(log p_v + H)) + dlogp·[v = y]
//
// A token of a shared prefix belongs to several rollouts with advantages A_b
// of both signs; min(r·A, clip(r)·A) is A·min(r, 1 + ε_hi) for A > 0 and
// A·max(r, 1 − ε_lo) for A < 0, so the sum over them needs two numbers only:
// gain = Σ A_b over the positive, cost = Σ |A_b| over the negative ones.
//
// The form on log-probs is elementwise plus three sums: bound by latency up to
// some 10^5 tokens, then by memory. The form on logits reads a row once into
// shared memory, takes (max, Σe^d, Σd·e^d) there, joins them over the CTAs
// of the row's cluster, and forms dz from the same shared memory: one read of
// the logits and one write of the gradient, bound by memory: 12,669 rows of
// 151,936 bf16 (a sixth masked) 1184 us, 6.0 TB/s and 0.88 of a plain
// copy's rate: a CTA's reads, joins and writes follow one another, and only the
// other CTAs of the SM fill the gaps. 1537 fp32 rows of 32,003 70 us, for the
// same reason (three CTAs to an SM; issue slots busy in 0.39 of the cycles). A
// masked row's first batches are read too: they are on their way before its
// weight is known. Streaming stores and loads that the L2 cache drops first were
// slower (by 0.5, 2.5 %).
//
// Where the numbers need it: logp − old is formed from (z_y − m), log S and
// old by exact two-sums, with log S as a pair, since rounding logp (about 12)
// to fp32 first would leave 5e-7 in the ratio; e^x − 1 − x by its series
// below 1/2, where the difference cancels. The sums over tokens are carried as
// pairs of floats (about 48 bits), in a fixed order; every token's ratio and
// policy term too, since terms of both signs cancel (524,288 tokens 11 us, with
// ratios as single floats 8.7).
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "logit_rows.cuh"

namespace cg = cooperative_groups;

namespace tt {
namespace {

// ------------------------------------------------------------------ sums in pairs of floats
struct F2 {
  float hi, lo;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = a + b, bb = s - a;
  return {s, (a - (s - bb)) + (b - bb)};
}
__device__ __forceinline__ F2 add(F2 x, F2 y) {
  F2 s = two_sum(x.hi, y.hi);
  if (!(fabsf(s.hi) < INFINITY)) return {s.hi, 0.f};  // (there the rounding errors are NaN)
  s.lo += x.lo + y.lo;
  return two_sum(s.hi, s.lo);
}
__device__ __forceinline__ void add(F2& x, float y) {
  const F2 s = two_sum(x.hi, y);
  x.hi = s.hi;
  x.lo += s.lo;
}
// a·x
__device__ __forceinline__ F2 scaled(float a, F2 x) {
  const float p = a * x.hi;
  return {p, fmaf(a, x.lo, fmaf(a, x.hi, -p))};
}
// e^x to about 2^-35: x = k·ln 2 + f (Cody and Waite's reduction: ln 2 is split so that k times its first part is exact), e^(f/8)
// − 1 by its series with the first two terms as pairs, then squared three times.
__device__ __forceinline__ F2 exp_pair(F2 x) {
  if (!(fabsf(x.hi) < 80.f)) return {expf(x.hi), 0.f};
  constexpr float kHi = 0.693145751953125f, kLo = 1.42860682e-6f;  // ln 2 to 15 bits, and the rest
  const float k = rintf(x.hi * 1.44269504f), p = k * kLo;
  const F2 f = two_sum(fmaf(-k, kHi, x.hi), -p);
  const float g = 0.125f * f.hi, gl = 0.125f * (f.lo - fmaf(k, kLo, -p) + x.lo);
  const float g2 = g * g, g2l = fmaf(2.f * g, gl, fmaf(g, g, -g2));
  const float rest = g * g2 * fmaf(g, fmaf(g, fmaf(g, 1.f / 720, 1.f / 120), 1.f / 24), 1.f / 6);
  F2 u = two_sum(g, 0.5f * g2);
  u.lo += gl + 0.5f * g2l + rest;
#pragma unroll
  for (int i = 0; i < 3; ++i) {  // (1 + u)² − 1
    const float q = u.hi * u.hi, ql = fmaf(2.f * u.hi, u.lo, fmaf(u.hi, u.hi, -q));
    const F2 v = two_sum(2.f * u.hi, q);
    u = two_sum(v.hi, v.lo + fmaf(2.f, u.lo, ql));
  }
  F2 e = two_sum(1.f, u.hi);
  e.lo += u.lo;
  const float scale = __int_as_float(((int)k + 127) << 23);
  return {e.hi * scale, e.lo * scale};
}

// Policy, KL and entropy terms.
struct Sums {
  F2 v[3];
};

// The warp's sums in lane 0.
__device__ __forceinline__ void sum_warp(Sums& s) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i)
      s.v[i] = add(s.v[i], {__shfl_down_sync(kAll, s.v[i].hi, o), __shfl_down_sync(kAll, s.v[i].lo, o)});
}
// The block's sums in thread 0. A multiple of 32 threads, up to 1024; `room`: a Sums per warp.
__device__ __forceinline__ void sum_block(Sums& s, Sums* room) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  sum_warp(s);
  if (lane == 0) room[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = lane < warps ? room[lane] : Sums{};
    sum_warp(s);
  }
}

// ------------------------------------------------------------------ the objective of one token
struct Policy {
  float lo, hi, dual, kl, ent, g;  // 1 − ε_lo, 1 + ε_hi, c, β, γ, g
  float lo_rest, hi_rest;          // of the first two to more than fp32
};
struct Inputs {  // per token, fp32 [N] each
  const float *old_logp, *adv, *adv_neg, *ref_logp, *weights;
};
__device__ __forceinline__ void split(float adv, bool two_sided, float adv_neg, float& gain, float& cost) {
  gain = two_sided || !(adv < 0.f) ? adv : 0.f;
  cost = two_sided ? adv_neg : adv < 0.f ? -adv : 0.f;
}

// e^x − 1 − x
__device__ __forceinline__ float exp_rest(float x, float em1) {
  if (fabsf(x) >= 0.5f) return em1 - x;
  // x²·Σ x^i/(i + 2)!: the first term left out is below 2^-25 of the sum
  float p = 2.48015873e-5f;
  p = fmaf(p, x, 1.98412698e-4f);
  p = fmaf(p, x, 1.38888889e-3f);
  p = fmaf(p, x, 8.33333333e-3f);
  p = fmaf(p, x, 4.16666667e-2f);
  p = fmaf(p, x, 1.66666667e-1f);
  p = fmaf(p, x, 0.5f);
  return p * x * x;
}

// The slope of the policy term with respect to logp, r = e^(logp − old): r times one factor, so that gain and cost may cancel.
// Comparisons are such that a NaN stays one.
__device__ __forceinline__ float policy_slope(const Policy& c, float gain, float cost, float r) {
  const float by = (!(r < c.lo) && !(r > c.dual) ? cost : 0.f) - (r > c.hi ? 0.f : gain);
  return by != 0.f || !(r > c.hi) ? r * by : 0.f;
}
// The term itself, as a pair: over many tokens the terms of both signs cancel, and their roundings do not.
__device__ __forceinline__ F2 policy_term(const Policy& c, float gain, float cost, F2 r) {
  const F2 term = scaled(-gain, r.hi > c.hi ? F2{c.hi, c.hi_rest} : r);
  if (cost == 0.f) return term;
  return add(term, scaled(cost, r.hi > c.dual ? F2{c.dual, 0.f} : r.hi < c.lo ? F2{c.lo, c.lo_rest} : r));
}
// The KL term and its part of the slope, x = ref − logp.
__device__ __forceinline__ float kl_term(const Policy& c, float x, float& slope) {
  const float em1 = expm1f(x);
  if (c.kl != 0.f) slope = fmaf(-c.kl, em1, slope);
  return exp_rest(x, em1);
}

// sums[4] = loss, policy, KL, entropy
__device__ __forceinline__ void finish(const Sums& s, const Policy& c, float* sums) {
  const double p = (double)s.v[0].hi + (double)s.v[0].lo, k = (double)s.v[1].hi + (double)s.v[1].lo,
               h = (double)s.v[2].hi + (double)s.v[2].lo;
  double loss = p;
  if (c.kl != 0.f) loss += (double)c.kl * k;
  if (c.ent != 0.f) loss -= (double)c.ent * h;
  sums[0] = (float)loss;
  sums[1] = (float)p;
  sums[2] = (float)k;
  sums[3] = (float)h;
}

// ------------------------------------------------------------------ on log-probs
struct LogpArgs {
  const float *logp, *entropy;
  Inputs in;
  int64_t N;
  Policy c;
  float *sums, *dlogp, *dentropy;
  Sums* parts;
};
constexpr int kTokenThreads = 256, kPerThread = 4, kTokens = kTokenThreads * kPerThread;
constexpr int kOneLaunch = 8;  // blocks whose sums one launch joins (a cluster)

// VEC: 16-byte accesses (all arrays aligned to 16 bytes).
template <bool VEC>
__global__ void __launch_bounds__(kTokenThreads) policy_tokens_kernel(const LogpArgs a) {
  __shared__ Sums room[kTokenThreads / 32];
  __shared__ Sums of_ctas[kOneLaunch];
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  Sums s = {};
  auto get = [&](const float* p, float (&v)[kPerThread], int64_t t, bool whole) {
    if (VEC && whole) {
      const float4 f = *reinterpret_cast<const float4*>(p + t);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const int64_t u = VEC ? t + i : t + i * kTokenThreads;
        v[i] = u < a.N ? p[u] : 0.f;
      }
    }
  };
  auto put = [&](float* p, const float (&v)[kPerThread], int64_t t, bool whole) {
    if (VEC && whole) {
      *reinterpret_cast<float4*>(p + t) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const int64_t u = VEC ? t + i : t + i * kTokenThreads;
        if (u < a.N) p[u] = v[i];
      }
    }
  };
  const int64_t t = t0 + (VEC ? kPerThread * (int)threadIdx.x : (int)threadIdx.x);
  const bool whole = VEC && t + kPerThread <= a.N;
  float lp[kPerThread], old[kPerThread], adv[kPerThread], dl[kPerThread], dh[kPerThread];
  float neg[kPerThread] = {}, ref[kPerThread] = {}, w[kPerThread] = {}, h[kPerThread] = {};
  get(a.logp, lp, t, whole);
  get(a.in.old_logp, old, t, whole);
  get(a.in.adv, adv, t, whole);
  if (a.in.adv_neg) get(a.in.adv_neg, neg, t, whole);
  if (a.in.ref_logp) get(a.in.ref_logp, ref, t, whole);
  if (a.in.weights) get(a.in.weights, w, t, whole);
  if (a.entropy) get(a.entropy, h, t, whole);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t u = VEC ? t + i : t + i * kTokenThreads;
    const float wt = u < a.N ? (a.in.weights ? w[i] : 1.f) : 0.f;
    dl[i] = dh[i] = 0.f;
    if (wt == 0.f) continue;  // a masked token, whatever its other inputs hold
    float gain, cost;
    split(adv[i], a.in.adv_neg != nullptr, neg[i], gain, cost);
    const F2 r = exp_pair(two_sum(lp[i], -old[i]));
    float slope = policy_slope(a.c, gain, cost, r.hi);
    s.v[0] = add(s.v[0], scaled(wt, policy_term(a.c, gain, cost, r)));
    if (a.in.ref_logp) add(s.v[1], wt * kl_term(a.c, ref[i] - lp[i], slope));
    if (a.entropy) add(s.v[2], wt * h[i]);
    dl[i] = a.c.g * wt * slope;
    dh[i] = a.c.ent != 0.f ? -a.c.g * wt * a.c.ent : 0.f;
  }
  if (a.dlogp) put(a.dlogp, dl, t, whole);
  if (a.dentropy) put(a.dentropy, dh, t, whole);
  sum_block(s, room);
  if (gridDim.x == 1) {
    if (threadIdx.x == 0) finish(s, a.c, a.sums);
  } else if (a.parts) {
    if (threadIdx.x == 0) a.parts[blockIdx.x] = s;
  } else {  // the grid is one cluster: its first CTA adds up
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // every CTA has started
    if (threadIdx.x == 0) *cluster.map_shared_rank(&of_ctas[blockIdx.x], 0) = s;
    cluster.sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      for (unsigned r = 1; r < gridDim.x; ++r)
#pragma unroll
        for (int i = 0; i < 3; ++i) s.v[i] = add(s.v[i], of_ctas[r].v[i]);
      finish(s, a.c, a.sums);
    }
  }
}

// The sums of n parts in order: of blocks of tokens (ROWS = false), or of rows of logits (a float4 each).
constexpr int kSumThreads = 1024;
template <bool ROWS>
__global__ void __launch_bounds__(kSumThreads) policy_sum_kernel(const void* parts, int64_t n, const Policy c, float* sums) {
  __shared__ Sums room[kSumThreads / 32];
  wait_prerequisites();
  Sums s = {};
  constexpr int kLoads = 8;  // of a thread under way together
  for (int64_t i = threadIdx.x; ROWS && i < n; i += kLoads * kSumThreads) {
    float4 f[kLoads];
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      f[q] = i + q * kSumThreads < n ? static_cast<const float4*>(parts)[i + q * kSumThreads] : make_float4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      s.v[0] = add(s.v[0], {f[q].x, f[q].w});
      add(s.v[1], f[q].y);
      add(s.v[2], f[q].z);
    }
  }
  if (!ROWS) {
    for (int64_t i = threadIdx.x; i < n; i += kSumThreads) {
      const Sums p = static_cast<const Sums*>(parts)[i];
#pragma unroll
      for (int q = 0; q < 3; ++q) s.v[q] = add(s.v[q], p.v[q]);
    }
  }
  sum_block(s, room);
  if (threadIdx.x == 0) finish(s, c, sums);
}

// ------------------------------------------------------------------ on logits
struct LogitsArgs {
  const void* z;
  void* dz;  // NULL: no gradient
  int64_t N, V, ld;
  const int32_t* y;
  Inputs in;
  Policy c;
  float *logp, *entropy;
  float4* rows;  // the row's terms: policy (its first part), KL, entropy; the policy term's second part
  int32_t* err;
};

// log s for s >= 1 (or 0, inf, NaN) as a pair: s = 2^k·f with f in [1/√2, √2), log s = k·ln 2 + log f (Cody and
// Waite's reduction): ln 2 is split so that k times its first part is exact.
__device__ __forceinline__ F2 log_pair(float s) {
  const uint32_t b = __float_as_uint(s);
  if (!(s > 0.f) || s == INFINITY) return {logf(s), 0.f};
  const int k = (int)((b - 0x3f3504f3u) & 0xff800000u) >> 23;  // (the bits of 1/√2)
  const float f = __uint_as_float(b - ((uint32_t)k << 23));
  constexpr float kHi = 0.693145751953125f, kLo = 1.42860682e-6f;  // ln 2 to 15 bits, and the rest
  F2 l = two_sum((float)k * kHi, logf(f));
  l.lo = fmaf((float)k, kLo, l.lo);
  return l;
}

// What every thread needs of its row.
struct RowOf {
  float m, nl;             // nl: −log2 S
  float gl, slope_t, at0;  // dlogp; and −dlogp − dH·(log p + H) as slope_t·(log2 p) + at0
  int none, wide;          // no gradient; every difference to the maximum has to be bounded (see turns_plainly)
};

constexpr int kBatch = 4;   // vectors of a thread at once: one rescaling for all of them
constexpr int kAhead = 2;   // batches on their way beside the one in use (four: no faster)
constexpr int kCtasMost = 8;
template <int WARPS>
constexpr int kGroups = WARPS == 1 ? 4 : 1;  // groups of a block: each takes rows of its own

// (m, s, u) of all lanes, the same bits in every one.
__device__ __forceinline__ Stat sum_stats(Stat t) {
  float M = t.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
  rescale(t, M);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    t.s += __shfl_xor_sync(kAll, t.s, o);
    t.u += __shfl_xor_sync(kAll, t.u, o);
  }
  return t;
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float2 g);
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float2 g) { return pack_bf16(g.x, g.y); }
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float2 g) {
  const __half2 h = __floats2half2_rn(g.x, g.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ uint32_t pack_twice_down(float x);  // x rounded towards -inf, twice
template <>
__device__ __forceinline__ uint32_t pack_twice_down<__nv_bfloat16>(float x) {
  return 0x10001u * __bfloat16_as_ushort(__float2bfloat16_rd(x));
}
template <>
__device__ __forceinline__ uint32_t pack_twice_down<__half>(float x) {
  return 0x10001u * __half_as_ushort(__float2half_rd(x));
}

// A row's inputs as they are loaded, before its sums: nothing waits for them there.
struct RowInputs {
  float old_logp, adv, adv_neg, ref_logp, w;
};
__device__ __forceinline__ RowInputs inputs_of(const Inputs& in, int64_t row, float w) {
  return {in.old_logp[row], in.adv[row], in.adv_neg ? in.adv_neg[row] : 0.f, in.ref_logp ? in.ref_logp[row] : 0.f, w};
}

// Whether a row of 16-bit logits with maximum m can be turned with its elements raised to Turn::low. That bound, about
// m − |m|/64, has to be finite in the type (fp16: from m = −64,496 down it is −inf; the sums hold on to −65,000, since they
// raise to the lowest value itself), and p = 0 times the line there has to be 0: the line's slope times 2^-6·|m| below fp32's
// largest value.
template <typename T>
__device__ __forceinline__ bool turns_plainly(float m) {
  if constexpr (sizeof(T) == 4) return true;
  else if constexpr (std::is_same<T, __half>::value) return m > -64000.f && m < INFINITY;
  else return fabsf(m) < 1e30f;
}

// A row's terms, log-prob and entropy written (by `writer`), and what its gradient needs.
template <typename T>
__device__ __forceinline__ RowOf row_of(const LogitsArgs& a, int64_t row, const RowInputs& in, const Stat& t, float zy, bool y_ok,
                                        bool writer) {
  const float w = in.w;
  const bool empty = t.m == -INFINITY && t.s == 0.f;  // every logit is -inf: no distribution
  const F2 ls = log_pair(t.s);
  const float log_s = ls.hi + ls.lo;
  const float h = empty ? 0.f : ls.hi - t.u / t.s + ls.lo, H = h < 0.f ? 0.f : h;
  // log-prob, and its difference to another one, by exact sums
  const F2 a0 = two_sum(zy, -t.m), a1 = two_sum(a0.hi, -ls.hi);
  const float logp = !y_ok ? __int_as_float(0x7fc00000)
                     : empty ? -INFINITY : zy == -INFINITY ? zy - log_s : a1.hi + (a0.lo + a1.lo - ls.lo);
  auto from = [&](float other) -> F2 {  // logp − other
    if (!(fabsf(logp) < INFINITY && fabsf(other) < INFINITY)) return {logp - other, 0.f};
    const F2 b0 = two_sum(a0.hi, -other), b1 = two_sum(b0.hi, -ls.hi);
    return two_sum(b1.hi, a0.lo + b0.lo + b1.lo - ls.lo);
  };
  float gain, cost;
  split(in.adv, a.in.adv_neg != nullptr, in.adv_neg, gain, cost);
  const F2 r = exp_pair(from(in.old_logp)), policy = scaled(w, policy_term(a.c, gain, cost, r));
  float slope = policy_slope(a.c, gain, cost, r.hi);
  const float kl = a.in.ref_logp ? kl_term(a.c, -from(in.ref_logp).hi, slope) : 0.f;
  if (writer) {
    if (!y_ok) set_err(a.err, TT_ERR_INVALID_ARG);
    a.logp[row] = logp;
    a.entropy[row] = H;
    a.rows[row] = make_float4(policy.hi, w * kl, w * H, policy.lo);
  }
  const float gl = a.c.g * w * slope, gh = a.c.ent != 0.f ? -a.c.g * w * a.c.ent : 0.f;
  constexpr float kLn2 = 0.6931471805599453f;
  // −log2 S rounded (about 16: to 1e-6); the rest of it goes into the line, and as a factor of p into both of its numbers
  const float nl = -ls.hi * kLog2e, rest = -fmaf(ls.hi, kLog2e, nl) - ls.lo * kLog2e, more = fmaf(rest, kLn2, 1.f);
  const float by = -gh * kLn2;
  return {t.m, nl, gl, by * more, fmaf(by, rest, -fmaf(gh, H, gl)) * more, empty || !y_ok, !turns_plainly<T>(t.m)};
}

// dz of vectors of a row.
template <typename T>
struct Turn {
  float2 nm, nl, sl, b0;
  uint32_t low;
  __device__ __forceinline__ Turn(const RowOf& r)
      : nm(make_float2(-r.m, -r.m)), nl(make_float2(r.nl, r.nl)),
        sl(make_float2(r.slope_t, r.slope_t)), b0(make_float2(r.at0, r.at0)), low(0) {
    // so far below the maximum that p is 0, and at least a step of the type below it
    if constexpr (sizeof(T) == 2) low = pack_twice_down<T>(r.m - fmaxf(130.f, fabsf(r.m) * 0.015625f));
  }
  __device__ __forceinline__ float2 line(float2 d) const {  // d = z − m
    const float2 lp = __ffma2_rn(d, make_float2(kLog2e, kLog2e), nl);  // log2 p
    return __fmul2_rn(make_float2(fast_exp2(lp.x), fast_exp2(lp.y)), __ffma2_rn(sl, lp, b0));
  }
  // d bounded: a masked logit's p is 0, and 0 times the line has to be 0
  __device__ __forceinline__ float2 bounded(float2 x) const {
    const float2 d = __fadd2_rn(x, nm);
    return make_float2(max_nan(d.x, kFloor), max_nan(d.y, kFloor));
  }
  __device__ __forceinline__ uint4 wide(const uint4& u) const {
    if constexpr (sizeof(T) == 4) {
      const float2 x = line(bounded(Pairs<T>::get(u, 0))), y = line(bounded(Pairs<T>::get(u, 1)));
      return make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
    } else {
      return make_uint4(pack_pair<T>(line(bounded(Pairs<T>::get(u, 0)))), pack_pair<T>(line(bounded(Pairs<T>::get(u, 1)))),
                        pack_pair<T>(line(bounded(Pairs<T>::get(u, 2)))), pack_pair<T>(line(bounded(Pairs<T>::get(u, 3)))));
    }
  }
  // 16-bit types, unless the row is a wide one: both elements of a pair bounded at once, before they are floats
  __device__ __forceinline__ uint32_t pair(uint32_t w) const {
    return pack_pair<T>(line(__fadd2_rn(Pairs<T>::floats(Pairs<T>::raise(w, low)), nm)));
  }
  __device__ __forceinline__ uint4 plain(const uint4& u) const {
    if constexpr (sizeof(T) == 4)
      return wide(u);
    else
      return make_uint4(pair(u.x), pair(u.y), pair(u.z), pair(u.w));
  }
  __device__ __forceinline__ T target(float zy, float gl) const {
    return static_cast<T>(line(bounded(make_float2(zy, zy))).x + gl);
  }
};

// Adds vectors to (m, s, u) with one rescaling.
template <typename T, bool WIDE, int N>
__device__ __forceinline__ void add_vectors(Stat& t, const uint4 (&u)[N]) {
  float bm;
  if constexpr (N == 4)
    bm = Pairs<T>::max(u[0], u[1], u[2], u[3]);
  else
    bm = Pairs<T>::max(u[0]);
  rescale(t, fmaxf(t.m, bm));
  const float mb = t.m == -INFINITY ? 0.f : t.m;
  const float2 nm = make_float2(-mb, -mb), l2 = make_float2(kLog2e, kLog2e);
  float2 s = make_float2(0.f, 0.f), q = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < N; ++v) fold<T, WIDE>(s, q, u[v], nm, l2);
  t.s += s.x + s.y;
  t.u += q.x + q.y;
}

// That a CTA has started says nothing about memory: with the release that the cluster barrier has by default 12,669 rows of
// 151,936 took 1211 us, not 1179. Not the aligned forms: a masked row's lanes come out of their last stores one by one.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Blocks to an SM that the registers are held to: left alone the compiler takes 90 (a tree's rows 1200 -> 1470 us).
template <int WARPS, bool CLUSTER>
constexpr int kMinBlocks = WARPS == 8 ? (CLUSTER ? 4 : 6) : WARPS == 2 ? 20 : 10;

// A row is taken by a group of WARPS warps, or (CLUSTER) of eight warps of each of the CL CTAs of a cluster, CL a power of two.
// `room`: vectors of a group's slice in shared memory; a thread copies, sums and turns its own vectors, so that the
// copies need no barrier. The sums are joined and the row's scalars formed by one warp of every CTA.
template <typename T, int WARPS, bool CLUSTER>
__global__ void __launch_bounds__(32 * WARPS * kGroups<WARPS>, kMinBlocks<WARPS, CLUSTER>)
    policy_logits_kernel(const LogitsArgs a, int CL, int log_CL, int room) {
  constexpr int VN = Row<T>::VN, kGroup = 32 * WARPS;
  extern __shared__ __align__(16) uint4 slices[];
  __shared__ Stat part[WARPS];
  __shared__ __align__(16) float4 of_ctas[kCtasMost];  // (m, s, u) of the slice, the target's logit where it lies there
  __shared__ float zy_shared;
  __shared__ RowOf row_shared;
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : (int)threadIdx.x >> 5;
  const int group = WARPS == 1 ? (int)threadIdx.x >> 5 : 0;
  const int tid = WARPS == 1 ? lane : (int)threadIdx.x;
  const int64_t row = WARPS == 1 ? (int64_t)blockIdx.x * kGroups<WARPS> + group : (int64_t)(blockIdx.x >> log_CL);
  const int rank = CLUSTER ? (int)blockIdx.x & (CL - 1) : 0;
  if (row >= a.N) return;  // (groups of one warp only)
  if (CLUSTER) cluster_arrive_relaxed();  // waited for before the CTAs write to one another
  const float w = a.in.weights ? a.in.weights[row] : 1.f;
  const Row<T> z(static_cast<const T*>(a.z) + row * a.ld, a.V);
  T* out = static_cast<T*>(a.dz) + row * a.ld;
  const int per = (z.nvec + CL - 1) >> log_CL, lo = rank * per, hi = min(z.nvec, lo + per);
  const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(z.p) & 15);
  const int wlo = z.whole_lo(), whi = min(hi, z.whole_hi());
  auto put_ends = [&](int j, const uint4& u) {
    const int e = z.first(j);
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < VN; ++i)
      if (e + i >= 0 && e + i < z.V) out[e + i] = t[i];
  };
  auto put = [&](int j, const uint4& u) {
    if (same && j >= wlo && j < whi)
      *reinterpret_cast<uint4*>(out + z.first(j)) = u;
    else
      put_ends(j, u);
  };
  uint4* buf = slices + group * room - lo;  // buf[j]: vector j
  const int y = a.y[row];
  const bool y_ok = y >= 0 && y < z.V;
  const int jy = y_ok ? (y + z.shift) / VN : -1;
  auto copy = [&](int j) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(buf + j)), "l"(z.p + z.first(j)) : "memory");
  };
  auto fetch = [&](int at) {
    if (at >= wlo && at + (kBatch - 1) * kGroup < whi) {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) copy(at + v * kGroup);
    } else {
#pragma unroll
      for (int v = 0; v < kBatch; ++v) {
        const int j = at + v * kGroup;
        if (j >= wlo && j < whi)
          copy(j);
        else if (j < hi)
          buf[j] = z.load(j);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int b = 0; b < kAhead; ++b) fetch(lo + tid + b * kBatch * kGroup);
  if (w == 0.f) {
    asm volatile("cp.async.wait_all;" ::: "memory");  // a masked row, whatever the logits that came hold
    if (a.dz)
      for (int j = lo + tid; j < hi; j += kGroup) put(j, make_uint4(0, 0, 0, 0));
    if (rank == 0 && tid == 0) {
      a.logp[row] = a.entropy[row] = 0.f;
      a.rows[row] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (CLUSTER) cluster_wait();
    return;
  }
  RowInputs in = {};
  if (warp == 0) in = inputs_of(a.in, row, w);
  Stat t = {-INFINITY, 0.f, 0.f};
  int j = lo + tid;
  for (; j + (kBatch - 1) * kGroup < hi; j += kBatch * kGroup) {
    fetch(j + kAhead * kBatch * kGroup);
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
    uint4 u[kBatch];
#pragma unroll
    for (int v = 0; v < kBatch; ++v) u[v] = buf[j + v * kGroup];
    add_vectors<T, false>(t, u);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (; j < hi; j += kGroup) {
    const uint4 u[1] = {buf[j]};
    add_vectors<T, false>(t, u);
  }
  t = sum_stats(t);
  if (!plain_way_holds<T>(t.m)) {  // (see fold: extreme rows, again with every difference bounded)
    t = {-INFINITY, 0.f, 0.f};
    for (int i = lo + tid; i < hi; i += kGroup) {
      const uint4 u[1] = {buf[i]};
      add_vectors<T, true>(t, u);
    }
    t = sum_stats(t);
  }
  // the target's logit, by the thread that holds it
  const bool here = jy >= lo && jy < hi, mine = here && ((jy - lo) & (kGroup - 1)) == tid;
  float zy = -INFINITY;
  if (mine) zy = static_cast<float>(reinterpret_cast<const T*>(buf + jy)[(y + z.shift) & (VN - 1)]);
  RowOf r;
  if constexpr (WARPS == 1) {
    zy = __shfl_sync(kAll, zy, here ? (jy - lo) & 31 : 0);
    r = row_of<T>(a, row, in, t, zy, y_ok, lane == 0);
  } else {
    if (lane == 0) part[warp] = t;
    if (mine) zy_shared = zy;
    __syncthreads();
    if (warp == 0) {
      t = lane < WARPS ? part[lane] : Stat{-INFINITY, 0.f, 0.f};
      t = sum_stats(t);
    }
    if (CLUSTER) {
      cg::cluster_group cluster = cg::this_cluster();
      cluster_wait();  // every CTA has started
      if (warp == 0 && lane < CL)
        *cluster.map_shared_rank(&of_ctas[rank], lane) = make_float4(t.m, t.s, t.u, here ? zy_shared : 0.f);
      cluster.sync();
      if (warp == 0) {
        const float4 f = lane < CL ? of_ctas[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        t = sum_stats({f.x, f.y, f.z});
      }
    }
    if (warp == 0) {
      const float target = CLUSTER ? of_ctas[y_ok ? jy / per : 0].w : zy_shared;
      const RowOf mine_too = row_of<T>(a, row, in, t, target, y_ok, rank == 0 && lane == 0);
      if (lane == 0) row_shared = mine_too;
    }
    __syncthreads();
    r = row_shared;
  }
  if (!a.dz) return;
  // ---------------------------------------------------------------- the gradient
  const Turn<T> turn(r);
  if (r.none) {
    for (int i = lo + tid; i < hi; i += kGroup) put(i, make_uint4(0, 0, 0, 0));
    return;
  }
  if (sizeof(T) == 4 || r.wide)
    for (int i = lo + tid; i < hi; i += kGroup) put(i, turn.wide(buf[i]));
  else
    for (int i = lo + tid; i < hi; i += kGroup) put(i, turn.plain(buf[i]));
  if (mine) out[y] = turn.target(zy, r.gl);  // behind this thread's own store
}

int check_policy(const tt_policy* p, Policy* c) {
  if (!p) return TT_ERR_INVALID_ARG;
  const float v[5] = {p->clip_lo, p->clip_hi, p->kl_coef, p->entropy_coef, p->g};
  for (float f : v)
    if (!std::isfinite(f)) return TT_ERR_INVALID_ARG;
  if (p->clip_lo < 0.f || p->clip_lo > 1.f || p->clip_hi < 0.f) return TT_ERR_INVALID_ARG;
  if (p->dual_clip != 0.f && !(p->dual_clip >= 1.f)) return TT_ERR_INVALID_ARG;
  const double lo = 1.0 - p->clip_lo, hi = 1.0 + p->clip_hi;
  *c = {(float)lo, (float)hi, p->dual_clip == 0.f ? INFINITY : p->dual_clip, p->kl_coef, p->entropy_coef, p->g,
        (float)(lo - (float)lo), (float)(hi - (float)hi)};
  return TT_OK;
}

template <typename... P, typename... A>
int launch(void (*kernel)(P...), int64_t grid, int block, size_t smem, int CL, bool dependent, cudaStream_t st, A... args) {
  cudaLaunchAttribute at[2];
  int n = 0;
  if (CL > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = CL;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {  // may be scheduled while the kernel before it runs; it waits at its first instruction
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  (void)cudaGetLastError();
  return cuda_status(e);
}

// Most shared memory of a CTA for its slice: what is left of 227 KB beside the static part.
constexpr int kSliceMost = 224 * 1024;

template <typename T, int WARPS, bool CLUSTER>
int launch_rows(const LogitsArgs& a, int log_CL, cudaStream_t st) {
  const int CL = 1 << log_CL, nvec = (int)(a.V / Row<T>::VN + 2);
  const int room = (nvec + CL - 1) / CL;
  const size_t smem = (size_t)room * 16 * kGroups<WARPS>;
  if (smem > kSliceMost) return TT_ERR_UNSUPPORTED;
  if (smem > 48 * 1024 && !tc::smem_attr_set<policy_logits_kernel<T, WARPS, CLUSTER>>(kSliceMost)) return TT_ERR_CUDA;
  return launch(policy_logits_kernel<T, WARPS, CLUSTER>, (a.N + kGroups<WARPS> - 1) / kGroups<WARPS> * CL,
                32 * WARPS * kGroups<WARPS>, smem, CL, false, st, a, CL, log_CL, room);
}

// How rows are taken: by a warp or two each while they are short and many, by a CTA of eight warps, or by 2, 4 or 8 CTAs. A
// slice of up to 80 KB leaves two CTAs and more to an SM, one's copies under way during another's joins. Few rows are cut
// further while every slice finds an SM of its own. Measured, us for the choice and the next one (bf16):
//   20,000 x 1000: warp 30, two warps 43;        20,000 x 8000: two warps 112, eight 142;
//   20,000 x 16,000: one CTA 206, two 376;       12,669 x 151,936 (16 % masked): 4 CTAs 1184, 8 CTAs 1320, 1 persistent CTA
//   to an SM with part of the row read again 1440, persistent clusters that copy the next row ahead 1590.
constexpr int64_t kSliceVectors = 5120;
template <typename T>
int launch_logits(const LogitsArgs& a, cudaStream_t st) {
  const int64_t nvec = a.V / Row<T>::VN + 1, sms = sm_count();
  if (nvec <= 512 && a.N >= 8 * sms) return launch_rows<T, 1, false>(a, 0, st);
  if (nvec <= 1024 && a.N >= 8 * sms) return launch_rows<T, 2, false>(a, 0, st);
  int log_CL = 0;
  while (log_CL < 3 &&
         (nvec > kSliceVectors << log_CL || ((2 * a.N << log_CL) <= 4 * sms && nvec >= (int64_t)512 << log_CL)))
    ++log_CL;
  return log_CL ? launch_rows<T, 8, true>(a, log_CL, st) : launch_rows<T, 8, false>(a, 0, st);
}

}  // namespace
}  // namespace tt

using namespace tt;

TT_API size_t tt_policy_loss_workspace_bytes(int64_t N) {
  return N <= kOneLaunch * kTokens ? 0 : (size_t)((N + kTokens - 1) / kTokens) * sizeof(Sums);
}

TT_API int tt_policy_loss(const float* logp, const float* entropy, const float* old_logp, const float* adv,
                          const float* adv_neg, const float* ref_logp, const float* weights, int64_t N,
                          const tt_policy* policy, float* sums, float* dlogp, float* dentropy, void* ws,
                          size_t ws_bytes, tt_stream_t stream) {
  Policy c;
  const int rc = check_policy(policy, &c);
  if (rc) return rc;
  if (N < 0 || N > (int64_t)INT32_MAX || !sums || reinterpret_cast<uintptr_t>(sums) % 4) return TT_ERR_INVALID_ARG;
  if (N && (!logp || !old_logp || !adv)) return TT_ERR_INVALID_ARG;
  if (N && c.ent != 0.f && !entropy) return TT_ERR_INVALID_ARG;
  const void* all[9] = {logp, entropy, old_logp, adv, adv_neg, ref_logp, weights, dlogp, dentropy};
  uintptr_t bits = 0;
  for (const void* p : all) bits |= reinterpret_cast<uintptr_t>(p);
  if (bits % 4) return TT_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return cuda_status(cudaMemsetAsync(sums, 0, 4 * sizeof(float), st));
  const int64_t blocks = (N + kTokens - 1) / kTokens;
  LogpArgs a = {logp, entropy, {old_logp, adv, adv_neg, ref_logp, weights}, N, c, sums, dlogp, dentropy, nullptr};
  auto kernel = bits % 16 ? policy_tokens_kernel<false> : policy_tokens_kernel<true>;
  if (blocks <= kOneLaunch) {
    int CL = 1;
    while (CL < blocks) CL *= 2;
    return launch(kernel, CL, kTokenThreads, 0, CL, false, st, a);
  }
  if (!ws || !aligned16(ws)) return TT_ERR_INVALID_ARG;
  if (ws_bytes < tt_policy_loss_workspace_bytes(N)) return TT_ERR_WORKSPACE;
  a.parts = static_cast<Sums*>(ws);
  const int r = launch(kernel, blocks, kTokenThreads, 0, 1, false, st, a);
  if (r) return r;
  return launch(policy_sum_kernel<false>, 1, kSumThreads, 0, 1, true, st, (const void*)ws, blocks, c, sums);
}

TT_API size_t tt_policy_loss_logits_workspace_bytes(int64_t N) { return N < 1 ? 0 : (size_t)N * sizeof(float4); }

TT_API int tt_policy_loss_logits(const void* logits, int dtype, int64_t N, int64_t V, int64_t ld, const int32_t* targets,
                                 const float* old_logp, const float* adv, const float* adv_neg, const float* ref_logp,
                                 const float* weights, const tt_policy* policy, float* sums, float* logp,
                                 float* entropy, void* dlogits, void* ws, size_t ws_bytes, int32_t* err,
                                 tt_stream_t stream) {
  Policy c;
  const int rc = check_policy(policy, &c);
  if (rc) return rc;
  if (dtype != TT_DT_BF16 && dtype != TT_DT_F16 && dtype != TT_DT_F32) return TT_ERR_INVALID_ARG;
  const size_t es = dtype == TT_DT_F32 ? 4 : 2;
  if (N < 0 || V < 1 || ld < V || N > INT32_MAX / 64 || V > INT32_MAX / 2) return TT_ERR_INVALID_ARG;
  if (!sums || reinterpret_cast<uintptr_t>(sums) % 4) return TT_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) return cuda_status(cudaMemsetAsync(sums, 0, 4 * sizeof(float), st));
  if (!logits || !targets || !old_logp || !adv || !logp || !entropy || !err) return TT_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits)) % es) return TT_ERR_INVALID_ARG;
  const void* words[9] = {targets, old_logp, adv, adv_neg, ref_logp, weights, logp, entropy, err};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) % 4) return TT_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return TT_ERR_INVALID_ARG;
  if (ws_bytes < tt_policy_loss_logits_workspace_bytes(N)) return TT_ERR_WORKSPACE;
  const LogitsArgs a = {logits, dlogits, N, V, ld, targets, {old_logp, adv, adv_neg, ref_logp, weights}, c, logp, entropy,
                        static_cast<float4*>(ws), err};
  int r;
  switch (dtype) {
    case TT_DT_BF16: r = launch_logits<__nv_bfloat16>(a, st); break;
    case TT_DT_F16: r = launch_logits<__half>(a, st); break;
    default: r = launch_logits<float>(a, st);
  }
  if (r) return r;
  return launch(policy_sum_kernel<true>, 1, kSumThreads, 0, 1, true, st, (const void*)ws, N, c, sums);
}
