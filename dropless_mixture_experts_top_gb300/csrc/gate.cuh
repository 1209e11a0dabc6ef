// gate.cuh -- the gate's choice: from the router's logits to the chosen experts, their
// weights and their places.  gate_logit.cu, gate_sigmoid.cu and gate_softmax.cu hold the
// kernel's variants (apart, so that they compile side by side), gate.cu the rest of the gate.
//
// Per token, l = its E logits:
//   s = softmax(l) or sigmoid(l),  c = s + bias  (no bias: the order of l)
//   a group's score: the sum of its 1 or 2 largest c;  the best `top_groups` groups
//   S = the k largest c in those groups (ties: lower expert)
//   w_j = scale s_{S_j} / (sum_i s_{S_i} or 1)
//
// Exact choice.  Two scores can be closer than fp32 resolves, and a choice that
// depends on the roundings of an exponential differs from program to program.  The
// choice made here is that of the exact scores: fp32 scores carry an error that
// is bounded (kNearSigmoid, kNearSoftmax below), and a token whose order is not
// decided by more than that is chosen again from scores in 64 bits.  Without a bias the
// logits themselves are compared.
//
// LPT lanes have a token (8, 16 or 32: four, two or one token per warp), with NV of its
// experts each.  A score becomes a 23-bit fixed-point number above the expert's index in
// one 32-bit key, so that keys are unique and one maximum over the token's lanes gives
// both the next score and whose it is.  Each lane sorts its keys once and hands out its
// largest.  Without a bias the key is the upper 24 bits of the logit.  Where the lanes hold
// all experts in whole vectors, a lane's experts are neighbours (VEC): whole sectors per
// load, and groups are runs of lanes.
//
// Bound by instructions (131072 x 256 in 8 groups: 314 a token) and by the few warps that its registers leave: fewer lanes per
// token share the steps between lanes among more tokens, at the price of longer lists to sort, and four
// blocks an SM without loads ahead hide more than two with (131072 x 256 in 8 groups 72 and 94 us; 16 lanes a token 104).
#pragma once

#include <float.h>
#include <limits.h>
#include <math.h>

#include "abi.h"
#include "common.cuh"

namespace moe {

struct GateArgs {
  const float *logits;  // [T,E]
  const float *bias;    // [E] or null
  int T, E, k;
  int groups, top_groups, group_best, group_size;
  bool sigmoid, renormalise;
  float scale;
  int32_t *topk_idx;
  float *topk_w;
  int32_t *counts, *offsets, *row_of_slot, *slot_of_row;
  float *w_row;
  int chunks;           // runs of tokens, a block each
  int chunk_tokens, longer;  // of a chunk; of the first `longer`, one more
  int cluster;          // chunks per cluster
  int32_t *before;      // [chunks][E]: the slots of expert e in the cluster's earlier chunks
  int32_t *count;       // [chunks][E]: its own
  int32_t *total;       // [clusters][E]
  int32_t *flags;       // [clusters]
  int32_t *status;
};

constexpr int kGateThreads = 256;
constexpr int kGateTok = 320;      // tokens of one round of a block at most
constexpr int kGateCluster = 8;    // blocks of a cluster at most

enum GateKey : int { kKeyLogit = 0, kKeySigmoid = 1, kKeySoftmax = 2 };
// The choice, by the key that orders the experts; one cluster: everything.
template <int KEY>
cudaError_t launch_gate_select(const GateArgs &a, cudaStream_t s);

__device__ __forceinline__ int gate_first(const GateArgs &a, int chunk) {
  const int c = min(chunk, a.chunks);
  return c * a.chunk_tokens + min(c, a.longer);
}

__device__ __forceinline__ int32_t ld_peer(const int32_t *p, int rank) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_smem_addr(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ float clean_logit(float l, bool &bad) {
  bad |= !(l <= FLT_MAX);
  return l != l ? -INFINITY : fminf(l, FLT_MAX);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Exclusive prefix of v over the block's first kMaxExperts threads (thread = expert); the
// total to *total.  s_w: 8 ints.
__device__ __forceinline__ int expert_prefix(int v, int *s_w, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31 && warp < kMaxExperts / 32) s_w[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 32; ++w) {
    before += w < warp ? s_w[w] : 0;
    all += s_w[w];
  }
  *total = all;
  return before + incl - v;
}

}  // namespace moe

#ifdef MOE_GATE_SELECT
namespace moe {
namespace {

constexpr int kWarps = kGateThreads / 32;

// Fixed point: c in [-B, 1 + B], B the largest finite |bias|, as 8 + O + c * scale in
// 23 bits, O = ceil(B scale).  A unit is (1 + 2B) 2^-23 or a little more.
// How far the number may be from that of the exact c, in units:
//   sigmoid: 1 / (1 + e), e = 2^(-l log2 e) by the part's ex2: off by 2^-22 of itself, and by |l| 2^-23 for the
//   rounded argument, of which s (1 - s) reaches s (at most 1/4, with the |l| 0.23); the sum by half an ulp, the
//   reciprocal by one: 2^-24 + 0.23 2^-23 + s (2^-24 + 2^-23), 2.2 units; bias * scale + base rounded,
//   half a unit, the product rounded, half: 3.2.  Two numbers that differ by more than 6.4 are in the order
//   of the exact ones.
//   softmax: s = e / Z, e = 2^((l - m) log2 e). Two numbers of one token are compared. They share the error of 1 / Z, which
//   enters their difference by |s_i - s_j| <= 1; their own errors go with s_i + s_j <= 1. In units:
//     shared: half for each rounding of Z, NV - 1 in a lane and log2 LPT across the lanes (34 of 32 experts on 8 lanes:
//     17); its terms, off by 2^-22 of themselves for the exponential (2) and by |l - m| 2.25 2^-24 for the argument
//     (difference, constant and product), whose mean over the scores is at most 3.34 2.25 2^-24 with 256 experts (F of
//     F e^F = 255 / e: one at the top, the others 1 + F below; 3.8); the reciprocal's ulp (1);
//     own: the exponential (2), the argument (|l - m| e^-|l - m| <= 0.37 for each of the two: 0.9), the product (0.5);
//     both numbers' roundings as above (2).
//   12.2 and half for each rounding of Z: 29.2. Sums of two scores have 2 more for their numbers, and twice the distance.
constexpr int kNearSigmoid = 7, kNearSoftmax = 35;
constexpr bool softmax_bound_holds(int lanes, int experts) {
  int roundings = experts - 1;
  for (; lanes > 1; lanes /= 2) ++roundings;
  return 2 * kNearSoftmax >= roundings + 25;
}
constexpr float kFixOne = 8388608.f;       // 2^23
constexpr float kFixLeast = 8.f;           // the least number of an expert that may be chosen; 0: it may not
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid_fast(float l) { return rcp(1.f + ex2(-kLog2e * l)); }

// A logit's order as an unsigned number (both zeros alike).
__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// Sorts NV keys, largest first; of 16 and 32, the first 8.
template <int NV>
__device__ __forceinline__ void sort_keys(uint32_t *v) {
  auto cas = [&](int a, int b) {
    const uint32_t hi = max(v[a], v[b]), lo = min(v[a], v[b]);
    v[a] = hi;
    v[b] = lo;
  };
  if constexpr (NV == 2) {
    cas(0, 1);
  } else if constexpr (NV == 4) {
    cas(0, 1), cas(2, 3), cas(0, 2), cas(1, 3), cas(1, 2);
  } else if constexpr (NV == 8) {
    cas(0, 1), cas(2, 3), cas(4, 5), cas(6, 7);
    cas(0, 2), cas(1, 3), cas(4, 6), cas(5, 7);
    cas(1, 2), cas(5, 6), cas(0, 4), cas(3, 7);
    cas(1, 5), cas(2, 6);
    cas(1, 4), cas(3, 6);
    cas(2, 4), cas(3, 5);
    cas(3, 4);
  } else if constexpr (NV >= 16) {
    constexpr int H = NV / 2;
    sort_keys<H>(v);
    sort_keys<H>(v + H);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = max(v[i], v[H + 7 - i]);  // the 8 largest, falling and rising
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & d) == 0) cas(i, i + d);
  }
}

// What the block keeps of the bias.
struct BiasInfo {
  float scale;  // units per 1
  float base;   // 2^23 + 8 + O
  int off;      // 8 + O: the number of c = 0
  bool odd;     // some entry is not finite
  float most;   // the largest |bias| (inf: some entry is not finite)
};

// A token whose order fp32 does not decide.  runs: which runs of `run` experts may be used
// (bit e / run), or 0 to choose the groups as well; only experts whose fp32 number is at least
// `least` can be among the chosen (0: every one).  extra: where it is known that none but the chosen k and one more come into
// question, that one (-1: not even one more, -2: unknown).
struct Undecided {
  uint32_t runs;
  int least, extra;
};

// ---- Scores as pairs of floats (hi + lo, about 48 bits), from error-free sums and products: the part's 64-bit
// unit is a hundredth as fast as this.  (Dekker, Knuth: two_sum, two_prod by a fused multiply-add.)  What follows is run by
// few warps, once or twice per SM: its time is that of fetching its instructions (some 60 cycles each), so it
// is written as loops, nothing unrolled, and its functions are not inlined twice.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair quick_two_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  return quick_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);
  return quick_two_sum(p, __fmaf_rn(a.h, b.h, -p) + __fmaf_rn(a.h, b.l, a.l * b.h));
}
__device__ __noinline__ Pair pair_div(Pair a, Pair b) {
  const float q = __fdiv_rn(a.h, b.h);
  const float r = __fmaf_rn(-q, b.h, a.h) + __fmaf_rn(-q, b.l, a.l);
  return quick_two_sum(q, __fdiv_rn(r, b.h));
}
// 1 / 6!, 1 / 5!, ... 1 / 0!
__constant__ Pair kFactorials[7] = {{1.3888889225e-03f, -3.3631094437e-11f}, {8.3333337680e-03f, -4.3461720333e-10f},
                                    {4.1666667908e-02f, -1.2417634698e-09f}, {1.6666667163e-01f, -4.9670538794e-09f},
                                    {0.5f, 0.f}, {1.f, 0.f}, {1.f, 0.f}};
// e^-(a + b) for a >= 0, b at most half an ulp of a; 0 from a = 40 on (4e-18).
// n ln 2 comes off in three parts (15, 17 and 24 bits: the first two products are exact), then the series:
// to r^6 / 6! in pairs, the rest, below 2e-7 of the sum, in single floats: off by 2^-45 at most.
__device__ __noinline__ Pair pair_exp_neg(float a, float b) {
  if (!(a < 40.f)) return {0.f, 0.f};
  const float n = rintf(a * 1.4426950408889634f);
  const Pair t = two_sum(__fmaf_rn(n, 0.693145751953125f, -a), __fmul_rn(n, 1.428605173714459e-06f));  // n ln 2 - a
  const Pair r = quick_two_sum(t.h, t.l + __fmaf_rn(n, 1.6465949582897e-12f, -b));
  float q = 1.f / 6227020800.f;  // 1 / 13!
  q = fmaf(q, r.h, 1.f / 479001600.f);
  q = fmaf(q, r.h, 1.f / 39916800.f);
  q = fmaf(q, r.h, 1.f / 3628800.f);
  q = fmaf(q, r.h, 1.f / 362880.f);
  q = fmaf(q, r.h, 1.f / 40320.f);
  q = fmaf(q, r.h, 1.f / 5040.f);
  Pair s = {q, 0.f};
#pragma unroll 1
  for (int k = 0; k < 7; ++k) s = pair_add(pair_mul(s, r), kFactorials[k]);
  const float f = __int_as_float((127 - static_cast<int>(n)) << 23);  // 2^-n
  return {s.h * f, s.l * f};
}
__device__ __forceinline__ Pair pair_sigmoid(float l) {
  const Pair e = pair_exp_neg(fabsf(l), 0.f), d = pair_add({1.f, 0.f}, e);
  return pair_div(l < 0.f ? e : Pair{1.f, 0.f}, d);
}
// In units of 2^-42, from pairs: off by under 8 (2^-39; the exponential's 2^-45, those of Z and the quotient, the
// conversions').  Scores that differ by more than twice that are in the order of the exact ones.
constexpr long long kNearFixed = 16;
constexpr float kFixedOne = 4398046511104.f;  // 2^42
constexpr float kFixedMost = 1024.f;          // of a bias
__device__ __forceinline__ long long to_fixed(Pair s, float b) {
  return __float2ll_rn(s.h * kFixedOne) + __float2ll_rn(s.l * kFixedOne) + __float2ll_rn(b * kFixedOne);
}

// An undecided token's choice by one warp: from fixed-point scores, or, without a bias, from the logits'
// order.  Whether these decide it (logits do); if not, nothing is written.  val: E numbers of this warp, list: E bytes;
// slot: the token's k slots, bit 15 set where an expert had no score.
template <int KEY>
__device__ __noinline__ bool resolve_fixed(const GateArgs &a, const float *row, const float *s_bias, BiasInfo bi, Undecided u,
                                           int run, long long *val, uint8_t *list, uint16_t *slot) {
  const int lane = threadIdx.x & 31, E = a.E;
  const bool biased = KEY != kKeyLogit && a.bias != nullptr;
  const long long least = LLONG_MIN;
  bool bad = false, in_range = true, whole = true;  // whole: biases that are whole numbers of units
  uint32_t scored = 0;                              // by a lane's experts lane + 32 i
  float top = -FLT_MAX, low = FLT_MAX;
  const bool few = KEY != kKeySoftmax && u.extra > -2 && bi.most <= kFixedMost;
  if (!few && lane * 8 < E) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + lane * 8));
#pragma unroll 1
  for (int e = lane, i = 0; e < E && !few; e += 32, ++i) {
    const float l = clean_logit(__ldg(row + e), bad), b = biased ? s_bias[e] : 0.f;
    top = fmaxf(top, l);
    if (l >= -FLT_MAX && b > -INFINITY) {
      scored |= 1u << i;
      low = fminf(low, l);
      in_range = in_range && fabsf(b) <= kFixedMost;
      whole = whole && rintf(b * kFixedOne) == b * kFixedOne;
    }
  }
  if (!__all_sync(0xffffffffu, in_range)) return false;
  // Equal logits (rows of zeros: padding): the scores are one number, which says the same of all, and the biases are exact.
  const bool even = !few && __all_sync(0xffffffffu, whole) && warp_max(-low) == -warp_max(top);
  const long long near = KEY == kKeyLogit || even ? 0 : kNearFixed;
  Pair z = {0.f, 0.f};
  if (KEY == kKeySoftmax) {
    top = warp_max(top);
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
      const float x = clean_logit(__ldg(row + e), bad);
      const Pair d = two_sum(top, -x);
      if (x >= -FLT_MAX) z = pair_add(z, pair_exp_neg(d.h, d.l));
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1)
      z = pair_add(z, {__shfl_xor_sync(0xffffffffu, z.h, o), __shfl_xor_sync(0xffffffffu, z.l, o)});
  }
  // the number of a logit and a bias in the order of the experts (order) or of the groups
  auto number = [&](float x, float c, bool order) -> long long {
    if (KEY == kKeyLogit || (order && !biased)) return static_cast<long long>(order_of(x));
    if (KEY == kKeySigmoid) return to_fixed(pair_sigmoid(x), c);
    const Pair d = two_sum(top, -x);
    return to_fixed(pair_div(pair_exp_neg(d.h, d.l), z), c);
  };
  if (u.runs == 0) {  // the groups as well
    float last = NAN;
    long long v = 0;
#pragma unroll 1
    for (int e = lane, i = 0; e < E; e += 32, ++i) {
      const float x = clean_logit(__ldg(row + e), bad), c = biased ? s_bias[e] : 0.f;
      if (x != last) v = number(x, 0.f, false);  // (rows of equal logits take one)
      last = x;
      val[e] = (scored >> i) & 1u ? v + (KEY == kKeyLogit ? 0 : __float2ll_rn(c * kFixedOne)) : least;
    }
    __syncwarp();
    long long g1 = least, g2 = least;
    if (lane < a.groups)
      for (int m = 0; m < a.group_size; ++m) {
        const long long v = val[lane * a.group_size + m];
        g2 = max(g2, min(g1, v));
        g1 = max(g1, v);
      }
    const long long gv = a.group_best == 2 && g2 > least ? g1 + g2 : g1;
    int before = 0;
    long long next = least;  // the best of those behind
    for (int h = 0; h < a.groups; ++h) {
      const long long o = __shfl_sync(0xffffffffu, gv, h);
      const bool first = o > gv || (o == gv && h < lane);
      before += first ? 1 : 0;
      if (!first && h != lane) next = max(next, o);
    }
    const bool open = lane < a.groups && before == a.top_groups - 1 && next > least && gv - next <= 2 * near && near > 0;
    if (__any_sync(0xffffffffu, open)) return false;
    u.runs = __ballot_sync(0xffffffffu, lane < a.groups && before < a.top_groups);
    u.least = 0;
    run = a.group_size;
    __syncwarp();
  }
  // the experts in question
  int n = 0;
  if (few) {
    if (lane < a.k) list[lane] = static_cast<uint8_t>(slot[lane]);
    if (lane == a.k) list[lane] = static_cast<uint8_t>(u.extra);
    n = a.k + (u.extra >= 0 ? 1 : 0);
  }
#pragma unroll 1
  for (int e0 = 0, i = 0; e0 < E && !few; e0 += 32, ++i) {
    const int e = e0 + lane;
    bool use = (scored >> i & 1u) && ((u.runs >> (e / run & 31)) & 1u);
    if (KEY != kKeyLogit && use && u.least > 0) {
      // the fp32 number once more, with the distance that decides off for safety
      const float l = clean_logit(__ldg(row + e), bad), b = biased ? s_bias[e] : 0.f;
      const float s = KEY == kKeySigmoid ? sigmoid_fast(l) : ex2((l - top) * kLog2e) * rcp(z.h);
      use = fmaf(s + b, bi.scale, static_cast<float>(bi.off)) >= static_cast<float>(u.least) - kNearSoftmax;
    }
    const uint32_t set = __ballot_sync(0xffffffffu, use);
    if (use) list[n + __popc(set & ((1u << lane) - 1u))] = static_cast<uint8_t>(e);
    n += __popc(set);
  }
  __syncwarp();
  {
    float last = NAN;
    long long v = 0;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) {
      const int e = list[i];
      const float x = clean_logit(__ldg(row + e), bad);
      if (x != last) v = number(x, 0.f, true);
      last = x;
      val[i] = v + (KEY == kKeyLogit || !biased ? 0 : __float2ll_rn(s_bias[e] * kFixedOne));
    }
  }
  __syncwarp();
  // lane j keeps the j-th of the order
  const int found = min(n, a.k);
  const long long tie = biased && KEY != kKeyLogit ? near : 0;  // (logits alone decide exactly)
  long long mine = least, end = least;
  int at_mine = 0;
  if (n <= 32) {  // every lane counts those in front of its own
    const long long v = lane < n ? val[lane] : least;
    const int e = lane < n ? list[lane] : 0;
    int before = 0;
#pragma unroll 1
    for (int o = 0; o < n; ++o) {
      const long long other = __shfl_sync(0xffffffffu, v, o);
      const int other_e = __shfl_sync(0xffffffffu, e, o);
      before += other > v || (other == v && other_e < e) ? 1 : 0;
    }
    __syncwarp();
    if (lane < n) val[before] = (v << 8) | lane;  // (numbers below 2^54)
    __syncwarp();
    if (lane < n) {
      mine = val[lane] >> 8;
      at_mine = static_cast<int>(val[lane] & 0xff);
    }
    end = __shfl_sync(0xffffffffu, mine, max(0, found - 1));
    __syncwarp();
    if (lane < n) val[at_mine] = lane < found ? least : mine;
    __syncwarp();
  } else {  // k times the best of what is left
    for (int j = 0; j < found; ++j) {
      long long best = least;
      int at = INT_MAX;
      for (int i = lane; i < n; i += 32) {
        const long long v = val[i];
        if (v > best) best = v, at = i;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const long long ov = __shfl_xor_sync(0xffffffffu, best, o);
        const int oa = __shfl_xor_sync(0xffffffffu, at, o);
        if (ov > best || (ov == best && oa < at)) best = ov, at = oa;
      }
      if (lane == j) mine = best, at_mine = at;
      end = best;
      if ((at & 31) == lane) val[at] = least;
      __syncwarp();
    }
  }
  bool open = false;
  if (tie > 0) {
    auto same = [&](int e0, int e1) { return __ldg(row + e0) == __ldg(row + e1) && s_bias[e0] == s_bias[e1]; };
    const long long next = __shfl_down_sync(0xffffffffu, mine, 1);
    const int at_next = __shfl_down_sync(0xffffffffu, at_mine, 1);
    if (lane + 1 < found && mine - next <= tie) open = !same(list[at_mine], list[at_next]);
    const int at_end = __shfl_sync(0xffffffffu, at_mine, max(0, found - 1));
    for (int i = lane; i < n; i += 32)  // those behind the last one
      if (val[i] > least && end - val[i] <= tie) open |= !same(list[at_end], list[i]);
  }
  if (__any_sync(0xffffffffu, open)) return false;
  if (lane < found) slot[lane] = list[at_mine];
  if (lane == 0) {  // fewer than k: the others by index
    int i = 0, e = 0;
    for (int j = found; j < a.k; ++e) {
      if (i < n && list[i] == e)
        ++i;
      else
        slot[j++] = static_cast<uint16_t>(e | 0x8000);
    }
  }
  __syncwarp();
  return true;
}

// The same in 64 bits: scores that are equal to 2^-38, biases past 1024.
template <int KEY>
__device__ __noinline__ void resolve_token(const GateArgs &a, const float *row, const float *s_bias, BiasInfo bi, Undecided u,
                                           int run, double *val, uint8_t *list, uint16_t *slot) {
  const int lane = threadIdx.x & 31, E = a.E;
  const bool biased = a.bias != nullptr;
  bool bad = false;
  double top = -DBL_MAX, z = 1.0;
  float top32 = -FLT_MAX, z32 = 1.f;
  if (KEY == kKeySoftmax) {
    for (int e = lane; e < E; e += 32) top32 = fmaxf(top32, clean_logit(__ldg(row + e), bad));
    top32 = warp_max(top32);
    top = top32;
    z = 0.0;
    for (int e = lane; e < E; e += 32) z += exp(static_cast<double>(clean_logit(__ldg(row + e), bad)) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z32 = static_cast<float>(z);
  }
  // the score of an expert in the order of the experts (order) or of the groups; a lane keeps the last
  // exponential, which serves rows of equal logits
  float last_l = NAN;
  double last_s = 0.0;
  auto exact = [&](float l, float b, bool order) -> double {
    if (KEY == kKeyLogit || (order && !biased)) return static_cast<double>(l);
    if (l != last_l) {
      last_l = l;
      last_s = KEY == kKeySigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l))) : exp(static_cast<double>(l) - top) / z;
    }
    return biased ? last_s + static_cast<double>(b) : last_s;
  };
  auto scored = [&](float l, float b) { return l >= -FLT_MAX && b > -INFINITY; };  // (not where b is NaN)
  if (u.runs == 0) {
    for (int e = lane; e < E; e += 32) {
      const float l = clean_logit(__ldg(row + e), bad), b = biased ? s_bias[e] : 0.f;
      val[e] = scored(l, b) ? exact(l, b, false) : -INFINITY;
    }
    __syncwarp();
    double g1 = -INFINITY, g2 = -INFINITY;
    if (lane < a.groups)
      for (int m = 0; m < a.group_size; ++m) {
        const double v = val[lane * a.group_size + m];
        g2 = fmax(g2, fmin(g1, v));
        g1 = fmax(g1, v);
      }
    const double gv = a.group_best == 2 && g2 > -INFINITY ? g1 + g2 : g1;
    int before = 0;
    for (int h = 0; h < a.groups; ++h) {
      const double o = __shfl_sync(0xffffffffu, gv, h);
      before += (o > gv || (o == gv && h < lane)) ? 1 : 0;
    }
    u.runs = __ballot_sync(0xffffffffu, lane < a.groups && before < a.top_groups);
    u.least = 0;
    run = a.group_size;
    __syncwarp();
  }
  // the experts in question, by index
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    bool use = false;
    if (e < E) {
      const float l = clean_logit(__ldg(row + e), bad), b = biased ? s_bias[e] : 0.f;
      use = scored(l, b) && ((u.runs >> (e / run)) & 1u);
      if (KEY != kKeyLogit && use && u.least > 0) {
        // the fp32 number once more, with the distance that decides off for safety
        const float s = KEY == kKeySigmoid ? sigmoid_fast(l) : ex2((l - top32) * kLog2e) * rcp(z32);
        use = fmaf(s + b, bi.scale, static_cast<float>(bi.off)) >= static_cast<float>(u.least) - kNearSoftmax;
      }
    }
    const uint32_t set = __ballot_sync(0xffffffffu, use);
    if (use) list[n + __popc(set & ((1u << lane) - 1u))] = static_cast<uint8_t>(e);
    n += __popc(set);
  }
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const int e = list[i];
    val[i] = exact(clean_logit(__ldg(row + e), bad), biased ? s_bias[e] : 0.f, true);
  }
  __syncwarp();
  // k times the best of what is left; taken ones become NaN, which no comparison prefers
  const int found = min(n, a.k);
  for (int j = 0; j < found; ++j) {
    double best = -INFINITY;
    int at = INT_MAX;
    for (int i = lane; i < n; i += 32) {
      const double v = val[i];
      if (v > best || (v == best && i < at)) best = v, at = i;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (ov > best || (ov == best && oa < at)) best = ov, at = oa;
    }
    if ((at & 31) == lane) {
      val[at] = NAN;
      slot[j] = list[at];
    }
    __syncwarp();
  }
  if (lane == 0) {  // fewer than k: the others by index
    int i = 0, e = 0;
    for (int j = found; j < a.k; ++e) {
      if (i < n && list[i] == e)
        ++i;
      else
        slot[j++] = static_cast<uint16_t>(e | 0x8000);
    }
  }
  __syncwarp();
}

// LPT lanes per token, NV experts per lane: with l the lane's place among the token's, e = l + LPT i, or NV l + i
// (VEC; E = LPT NV).  KMAX: k at most.
template <int LPT, int NV, bool VEC, int KEY, bool GROUPS, int KMAX>
__global__ void __launch_bounds__(kGateThreads, 4) gate_select_kernel(const GateArgs a) {
  constexpr int kNear = KEY == kKeyLogit ? 0 : (KEY == kKeySigmoid ? kNearSigmoid : kNearSoftmax);
  constexpr bool KEYS = GROUPS && !VEC;                  // groups by way of shared memory
  static_assert(!KEYS || LPT == 32, "a lane per group");
  static_assert(KEY != kKeySoftmax || softmax_bound_holds(LPT, NV), "the sum over the experts has too many roundings");
  constexpr int TPW = 32 / LPT, kStep = kWarps * TPW;    // tokens of a warp, of the block, at once
  constexpr int ND = NV < 8 ? NV : 8;                    // a lane's sorted keys
  constexpr int kWords = kGateTok / 32;
  __shared__ union {                                     // one after the other:
    uint32_t keys[KEYS ? kWarps : 1][KEYS ? kMaxExperts : 1];  // the choice's
    double val[kWarps][kMaxExperts];                     // for undecided tokens
    struct {
      uint32_t emask[kWords][kMaxExperts];               // tokens of this round that chose expert e
      uint16_t before[kWords][kMaxExperts];              // how many in the words in front
    } rank;
  } sh;
  __shared__ float s_bias[kMaxExperts];
  __shared__ __align__(16) float s_add[kMaxExperts];     // the bias' part of the number (of -inf, NaN, inf: itself)
  __shared__ int32_t s_run[kMaxExperts];                 // the chunk's slots of expert e in earlier rounds
  __shared__ uint16_t s_slot[kGateTok * KMAX];           // expert of each slot; bit 15: without a score
  __shared__ float2 s_soft[kGateTok];                    // softmax weights: a token's largest logit, and its sum
  __shared__ Undecided s_und[kGateTok];
  __shared__ uint16_t s_list[kGateTok];                  // undecided tokens
  __shared__ uint8_t s_cand[kWarps][kMaxExperts];
  __shared__ int32_t s_count, s_flag, s_bodd;
  __shared__ float s_bmax[kWarps];
  __shared__ int32_t s_base[kMaxExperts];
  __shared__ int s_w[kMaxExperts / 32];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = lane % LPT;
  const int E = a.E, k = a.k;
  const int first = gate_first(a, blockIdx.x), last = min(a.T, gate_first(a, blockIdx.x + 1));
  if (tid == 0) s_count = 0, s_flag = 0, s_bodd = 0;
  s_run[tid] = 0;  // (kGateThreads == kMaxExperts)
  asm volatile("" ::"r"(first), "r"(last));  // before the wait
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();

  auto expert = [&](int i) { return VEC ? l * NV + i : l + LPT * i; };
  auto load = [&](int t, float (&v)[NV]) {
    const float *row = a.logits + static_cast<size_t>(t) * E;
    if constexpr (VEC) {
      if (t < last) {
#pragma unroll
        for (int i = 0; i < NV; i += 8)
          asm volatile("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]), "=f"(v[i + 4]), "=f"(v[i + 5]),
                         "=f"(v[i + 6]), "=f"(v[i + 7])
                       : "l"(row + l * NV + i));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = t < last && expert(i) < E ? __ldg(row + expert(i)) : 0.f;
    }
  };

  BiasInfo bi{kFixOne - 32.f, kFixOne + kFixLeast, static_cast<int>(kFixLeast), false, 0.f};
  __syncthreads();
  if (KEY != kKeyLogit) {
    const float b = a.bias && tid < E ? __ldg(a.bias + tid) : 0.f;
    s_bias[tid] = b;
    if (a.bias) {
      const bool odd = !(fabsf(b) <= FLT_MAX);
      if (odd) s_bodd = 1;
      float m = warp_max(odd ? 0.f : fabsf(b));
      if (lane == 0) s_bmax[warp] = m;
      __syncthreads();
      m = s_bmax[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_bmax[w]);
      bi.scale = (kFixOne - 32.f) / (1.f + 2.f * m);
      const float O = ceilf(m * bi.scale);
      bi.base = kFixOne + kFixLeast + O;
      bi.off = static_cast<int>(kFixLeast + O);
      bi.odd = s_bodd != 0;
      bi.most = bi.odd ? INFINITY : m;
    }
    // (VEC: in the order in which the lanes read vectors of four)
    const int at = VEC ? (tid % NV / 4) * (LPT * 4) + tid / NV * 4 + tid % 4 : tid;
    if (!VEC || tid < LPT * NV) s_add[at] = fmaf(b, bi.scale, bi.base);
    __syncthreads();
  }
  // groups: VEC: runs of lanes; else by way of shared memory, with gP lanes for each
  const int gs = a.group_size, G = a.groups;
  int gP = 1, gits = 0;
  if constexpr (KEYS) {
    while (2 * gP * G <= 32) gP *= 2;
    gits = (gs + gP - 1) / gP;
  }
  const int my_g = VEC ? l * NV / gs : lane % G, my_p = VEC ? 0 : lane / G;
  const int shift = 32 - __clz(k - 1), width = 1 << shift;  // a token's slots in a power of two of threads
  const bool whole_sum = !a.sigmoid && !a.renormalise;  // the weights need the softmax' sum over all experts
  bool bad = false;

  auto top_of = [](uint32_t v) {  // over the token's lanes
    if constexpr (LPT == 32) {
      return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
      for (int o = LPT / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
      return v;
    }
  };

  for (int t0 = first; t0 < last; t0 += kGateTok) {
    // ---- choice: a warp's tokens, kStep apart
#pragma unroll 1
    for (int tw = warp * TPW; tw < kGateTok && t0 + tw < last; tw += kStep) {
      const int tl = tw + lane / LPT, t = t0 + tl;
      const bool valid = t < last;
      float x[NV] = {}, fin = 0.f;
      load(t, x);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        fin = fmaf(x[i], 0.f, fin);  // NaN where one is not finite
      }
      const bool odd = __any_sync(0xffffffffu, fin != 0.f);
      uint32_t off = 0;  // experts that may not be chosen
      if (odd) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          x[i] = clean_logit(x[i], bad);
          off |= static_cast<uint32_t>(!(x[i] >= -FLT_MAX)) << i;
        }
      }
      uint32_t key[NV];
      if (KEY == kKeySoftmax || (KEY == kKeyLogit && whole_sum)) {
        float m = -FLT_MAX, z = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = VEC || expert(i) < E ? fmaxf(m, x[i]) : m;
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float e = VEC || expert(i) < E ? ex2((x[i] - m) * kLog2e) : 0.f;
          if (KEY == kKeySoftmax) x[i] = e;
          z += e;
        }
#pragma unroll
        for (int o = LPT / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (l == 0 && valid) s_soft[tl] = make_float2(m, z);
        if (KEY == kKeySoftmax) {
          const float rz = rcp(z);
#pragma unroll
          for (int i = 0; i < NV; ++i) x[i] *= rz;
        }
      }
      if constexpr (KEY == kKeyLogit) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = (order_of(x[i]) & 0xFFFFFF00u) | (255u - expert(i));
      } else {
        float add[NV];
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < NV; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(s_add + i / 4 * (LPT * 4) + l * 4);
            add[i] = q.x, add[i + 1] = q.y, add[i + 2] = q.z, add[i + 3] = q.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i) add[i] = s_add[expert(i) & (kMaxExperts - 1)];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float s = KEY == kKeySigmoid ? sigmoid_fast(x[i]) : x[i];
          x[i] = fmaf(s, bi.scale, add[i]);  // a whole number in [2^23, 2^24), or inf
        }
        if (bi.odd) {  // a bias of -inf or NaN: the number 0
#pragma unroll
          for (int i = 0; i < NV; ++i) x[i] = fmaxf(x[i], kFixOne);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)  // the number's three bytes over the index
          key[i] = __byte_perm(__float_as_uint(x[i]), 255u - expert(i), 0x2104);
      }
      if (odd) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = (off >> i) & 1u ? 0u : key[i];
      }
      if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = expert(i) < E ? key[i] : 0u;
      }
      Undecided u{0xffffffffu, 0, -2};
      bool open_groups = false;
      if constexpr (GROUPS) {
        uint32_t k1, k2;
        if constexpr (VEC) {
          sort_keys<NV>(key);
          k1 = key[0];
          k2 = key[1];
          for (int o = 1; o * NV < gs; o <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o), o2 = __shfl_xor_sync(0xffffffffu, k2, o);
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i) sh.keys[warp][lane + 32 * i] = key[i];
          __syncwarp();
          k1 = k2 = 0;
          if (my_p < gP) {
            int it = my_g % gits;  // each group starts elsewhere: other banks
            for (int n = 0; n < gits; ++n) {
              const int j = my_p + gP * it;
              const uint32_t v = j < gs ? sh.keys[warp][my_g * gs + j] : 0u;
              k2 = max(k2, min(k1, v));
              k1 = max(k1, v);
              if (++it == gits) it = 0;
            }
          }
          for (int o = gP / 2; o > 0; o >>= 1) {
            const uint32_t o1 = __shfl_down_sync(0xffffffffu, k1, o * G), o2 = __shfl_down_sync(0xffffffffu, k2, o * G);
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
          }
          __syncwarp();
        }
        // a group's number (its second score, where it has none: that of c = 0) over its index
        uint32_t gq = k1 >> 8;
        if (KEY != kKeyLogit && a.group_best == 2 && gq) gq += (k2 >> 8) ? k2 >> 8 : static_cast<uint32_t>(bi.off);
        uint32_t gkey = VEC || lane < G ? (gq << 5) | (31u - my_g) : 0u;
        bool kept = false;
        if constexpr (VEC) {  // a lane counts the groups in front of its own
          const int lanes = gs / NV;
          uint32_t below = 0;
          int before = 0;
          for (int o = lanes; o < LPT; o += lanes) {
            const uint32_t other = __shfl_sync(0xffffffffu, gkey, (lane - l) + ((l + o) & (LPT - 1)));
            before += other > gkey ? 1 : 0;
            below = max(below, other < gkey ? other : 0u);
          }
          kept = before < a.top_groups;
          const bool near = before == a.top_groups - 1 && (below >> 5) != 0 &&
                            (bi.odd || (gkey >> 5) - (below >> 5) <= 2 * kNear);
          open_groups = (__ballot_sync(0xffffffffu, near) >> (lane - l) & ((1u << LPT) - 1u)) != 0;
        } else {
          uint32_t r = 0;
          for (int j = 0; j < a.top_groups; ++j) {
            r = top_of(gkey);
            if (gkey == r) {
              kept = true;
              gkey = 0;
            }
          }
          const uint32_t next = top_of(gkey);
          open_groups = a.top_groups < G && (next >> 5) != 0 && (bi.odd || (r >> 5) - (next >> 5) <= 2 * kNear);
        }
        const uint32_t runs = __ballot_sync(0xffffffffu, kept && (VEC || lane < G));
        u.runs = open_groups ? 0u : (VEC ? runs >> (lane - l) & ((1u << (LPT & 31)) - 1u) : runs);
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < ND; ++i) key[i] = kept ? key[i] : 0u;
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i) key[i] = (runs >> (expert(i) / gs & 31)) & 1u ? key[i] : 0u;
        }
      }
      if constexpr (!(GROUPS && VEC)) sort_keys<NV>(key);
      uint32_t gap = 0xffffffffu, end = 0;  // the least distance of neighbours; the k-th
      bool undecided = open_groups;
      if constexpr (LPT < 32) {
        // the lanes' sorted lists merged in pairs, 8 kept: of two falling lists, the larger of v[i] and w[7 - i] are the
        // 8 largest, and fall and rise
        static_assert(KMAX == 8, "lists of 8");
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < ND ? key[i] : 0u;
#pragma unroll
        for (int o = 1; o < LPT; o <<= 1) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = max(v[i], w[7 - i]);
#pragma unroll
          for (int d = 4; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((i & d) == 0) {
                const uint32_t hi = max(v[i], v[i + d]), lo = min(v[i], v[i + d]);
                v[i] = hi;
                v[i + d] = lo;
              }
        }
        uint32_t ninth = 0;
        if (k == 8) {
#pragma unroll
          for (int i = 0; i < ND; ++i) ninth = max(ninth, key[i] < v[7] ? key[i] : 0u);
          ninth = top_of(ninth);
          // (a lane whose whole list is among the 8 may have one behind it that was not sorted)
          if (NV > ND) undecided |= (__ballot_sync(0xffffffffu, key[ND - 1] == v[7]) >> (lane - l) & ((1u << LPT) - 1u)) != 0;
        }
        uint32_t got = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j < k) {
            gap = min(gap, v[j] - (j < 7 ? v[j + 1] : ninth));
            end = v[j];
          }
          got = l == j ? v[j] : got;
        }
        if (l < k && valid) s_slot[tl * k + l] = static_cast<uint16_t>(255u - (got & 255u));
        if (__any_sync(0xffffffffu, gap < (kNear + 1) * 256u)) {  // who comes into question
          uint32_t next = ninth;
#pragma unroll
          for (int j = 1; j < 8; ++j) next = j == k ? v[j] : next;
          const uint32_t bound = end - min(end, (kNear + 1) * 256u);
          bool more = ND < NV && key[ND - 1] >= bound;
#pragma unroll
          for (int i = 0; i < ND; ++i) more |= key[i] < next && key[i] >= bound;
          if ((__ballot_sync(0xffffffffu, more) >> (lane - l) & ((1u << LPT) - 1u)) == 0)
            u.extra = next >= bound && (next >> 8) ? static_cast<int>(255u - (next & 255u)) : -1;
        }
      } else {
        uint32_t prev = 0xffffffffu;
#pragma unroll
        for (int j = 0; j <= KMAX; ++j) {
          if (j > k) break;
          const uint32_t r = top_of(key[0]);
          gap = min(gap, prev - r);
          prev = r;
          if (j < k) end = r;
          if (key[0] == r) {
            if (j < k && valid) s_slot[tl * k + j] = static_cast<uint16_t>(255u - (r & 255u));
#pragma unroll
            for (int i = 0; i + 1 < ND; ++i)
              if (i < KMAX - j) key[i] = key[i + 1];  // (further back none is needed any more)
            if (ND <= KMAX - j || ND == 1) key[ND - 1] = 0;
          }
        }
      }
      // two neighbours too near to tell, or fewer than k that may be chosen
      undecided |= gap < (kNear + 1) * 256u || (end >> 8) == 0;
      if (undecided && l == 0 && valid) {
        const int q = static_cast<int>(end >> 8);
        u.least = q > 2 * kNear + 1 ? q - 2 * kNear : 0;
        if (open_groups || q == 0) u.extra = -2;
        s_und[tl] = u;
        s_list[atomicAdd(&s_count, 1)] = static_cast<uint16_t>(tl);
      }
    }
    __syncthreads();

    // ---- what is left to decide
    const int count = s_count;
    for (int i = warp; i < count; i += kWarps) {
      const int tl = s_list[i], run = GROUPS ? (VEC ? NV : gs) : E;
      const float *row = a.logits + static_cast<size_t>(t0 + tl) * E;
      const bool done = resolve_fixed<KEY>(a, row, s_bias, bi, s_und[tl], run, reinterpret_cast<long long *>(sh.val[warp]),
                                           s_cand[warp], s_slot + tl * k);
      if (KEY != kKeyLogit && !done)
        resolve_token<KEY>(a, row, s_bias, bi, s_und[tl], run, sh.val[warp], s_cand[warp], s_slot + tl * k);
    }
    __syncthreads();
    const int ntok = min(kGateTok, last - t0), words = (ntok + 31) / 32;
    if (tid == 0) s_count = 0;
    for (int w = 0; w < words; ++w) sh.rank.emask[w][tid] = 0u;
    __syncthreads();

    // ---- weights: a thread per slot, the slots of a token side by side in a power of two of lanes
    for (int p = tid; p < words * 32 * width; p += kGateThreads) {
      const int tl = p >> shift, j = p & (width - 1);
      const bool in = tl < ntok && j < k;
      const int v = in ? s_slot[tl * k + j] : 0x8000, e = v & 0x7FFF;
      bool unused = false;
      const float l = v & 0x8000 ? -INFINITY : clean_logit(__ldg(a.logits + static_cast<size_t>(t0 + tl) * E + e), unused);
      float top = l;
      for (int o = width / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // Renormalised, scores enter by their ratios: relative to e^top, which keeps scores that
      // underflow (sigmoid: relative to e^min(top, 0), since s <= 1).
      const bool none = top == -INFINITY;
      float w;
      if (a.sigmoid) {
        const float ref = a.renormalise && !none ? fminf(top, 0.f) : 0.f;
        const float x = expf(-fabsf(l));  // e^(l - ref) / (1 + e^l), by the exponential that does not overflow
        w = l > 0.f ? 1.f / (1.f + x) : expf(l - ref) / (1.f + x);
      } else {
        w = none ? 0.f : expf(l - (whole_sum && in ? s_soft[tl].x : top));
      }
      float sum = w;
      for (int o = width / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (whole_sum && in) sum = s_soft[tl].y;
      if (in) {
        const size_t at = static_cast<size_t>(t0 + tl) * k + j;
        a.topk_idx[at] = e;
        a.topk_w[at] = none ? 0.f : w * (a.scale / (a.sigmoid && !a.renormalise ? 1.f : sum));
        atomicOr(&sh.rank.emask[tl >> 5][e], 1u << (tl & 31));
      }
    }
    __syncthreads();

    // ---- ranks: a slot's place among the chunk's slots of its expert
    int run = s_run[tid];
    for (int w = 0; w < words; ++w) {
      sh.rank.before[w][tid] = static_cast<uint16_t>(run - s_run[tid]);
      run += __popc(sh.rank.emask[w][tid]);
    }
    __syncthreads();
    for (int p = tid; p < ntok * width; p += kGateThreads) {
      const int tl = p >> shift, j = p & (width - 1), sl = tl * k + j;
      if (j >= k) continue;
      const int e = s_slot[sl] & 0x7FFF, w = tl >> 5;
      a.row_of_slot[static_cast<size_t>(t0) * k + sl] =
          s_run[e] + sh.rank.before[w][e] + __popc(sh.rank.emask[w][e] & ((1u << (tl & 31)) - 1u));
    }
    __syncthreads();
    s_run[tid] = run;
  }
  if (bad) s_flag = 1;
  __syncthreads();

  // ---- the cluster's chunks in front of this one
  if (a.cluster > 1) cluster_sync();
  const int rank = blockIdx.x % a.cluster, cluster = blockIdx.x / a.cluster;
  int before = 0, all = 0, n;
  if (tid < E)
    for (int c = 0; c < a.cluster; ++c) {
      const int v = a.cluster > 1 ? ld_peer(&s_run[tid], c) : s_run[tid];
      before += c < rank ? v : 0;
      all += v;
    }
  int flag = 0;
  if (tid == 0 && rank == 0)
    for (int c = 0; c < a.cluster; ++c) flag |= (a.cluster > 1 ? ld_peer(&s_flag, c) : s_flag) ? kDevNonfiniteLogit : 0;
  if (static_cast<int>(gridDim.x) > a.cluster) {  // the second kernel goes on
    if (tid < E) {
      a.before[static_cast<size_t>(blockIdx.x) * E + tid] = before;
      a.count[static_cast<size_t>(blockIdx.x) * E + tid] = s_run[tid];
      if (rank == 0) a.total[static_cast<size_t>(cluster) * E + tid] = all;
    }
    if (tid == 0 && rank == 0) a.flags[cluster] = flag;
  } else {
    const int off = expert_prefix(all, s_w, &n);
    s_base[tid] = off + before;
    if (rank == 0) {
      if (tid < E) {
        a.counts[tid] = all;
        a.offsets[tid] = off;
      }
      if (tid == 0) {
        a.offsets[E] = n;
        *a.status = flag;
      }
    }
    __syncthreads();
    for (int64_t s = static_cast<int64_t>(first) * k + tid; s < static_cast<int64_t>(last) * k; s += kGateThreads) {
      const int row = s_base[a.topk_idx[s]] + a.row_of_slot[s];  // (this block's own writes)
      a.row_of_slot[s] = row;
      a.slot_of_row[row] = static_cast<int32_t>(s);
      a.w_row[row] = a.topk_w[s];
    }
  }
  if (a.cluster > 1) cluster_sync();  // before a block leaves that others read
}

template <int LPT, int NV, bool VEC, int KEY, bool GROUPS, int KMAX>
cudaError_t launch_variant(const GateArgs &a, cudaStream_t s) {
  const int blocks = (a.chunks + a.cluster - 1) / a.cluster * a.cluster;
  return launch_pdl(gate_select_kernel<LPT, NV, VEC, KEY, GROUPS, KMAX>, dim3(blocks), dim3(kGateThreads), 0, s, a.cluster, a);
}
template <int KEY, bool GROUPS>
cudaError_t launch_wide(const GateArgs &a, cudaStream_t s) {  // a warp per token
  if (a.E <= 32) return launch_variant<32, 1, false, KEY, GROUPS, kMaxTopK>(a, s);
  if (a.E <= 64) return launch_variant<32, 2, false, KEY, GROUPS, kMaxTopK>(a, s);
  if (a.E <= 128) return launch_variant<32, 4, false, KEY, GROUPS, kMaxTopK>(a, s);
  return launch_variant<32, 8, false, KEY, GROUPS, kMaxTopK>(a, s);
}

}  // namespace

// Several tokens per warp up to k = 8, whole vectors where a token's row and a group are made of a lane's.
template <int KEY>
cudaError_t launch_gate_select(const GateArgs &a, cudaStream_t s) {
  const bool sectors = (reinterpret_cast<uintptr_t>(a.logits) & 31) == 0;
  auto runs = [&](int nv) {  // groups of a power of two of lanes
    const int lanes = a.group_size / nv;
    return a.group_size % nv == 0 && (lanes & (lanes - 1)) == 0;
  };
  if (a.k <= 8 && a.groups == 1) {
    if (a.E <= 8) return launch_variant<8, 1, false, KEY, false, 8>(a, s);
    if (a.E <= 32) return launch_variant<8, 4, false, KEY, false, 8>(a, s);
    if (a.E == 64 && sectors) return launch_variant<8, 8, true, KEY, false, 8>(a, s);
    if (a.E <= 64) return launch_variant<8, 8, false, KEY, false, 8>(a, s);
    if (a.E == 128 && sectors) return launch_variant<8, 16, true, KEY, false, 8>(a, s);
    if (a.E <= 128) return launch_variant<8, 16, false, KEY, false, 8>(a, s);
    if (a.E == 256 && sectors) return launch_variant<8, 32, true, KEY, false, 8>(a, s);
    return launch_variant<8, 32, false, KEY, false, 8>(a, s);
  }
  if (a.k <= 8 && sectors) {
    if (a.E == 64 && runs(8)) return launch_variant<8, 8, true, KEY, true, 8>(a, s);
    if (a.E == 128 && runs(16)) return launch_variant<8, 16, true, KEY, true, 8>(a, s);
    if (a.E == 256 && runs(32)) return launch_variant<8, 32, true, KEY, true, 8>(a, s);
    if (a.E == 256 && runs(16)) return launch_variant<16, 16, true, KEY, true, 8>(a, s);
  }
  return a.groups > 1 ? launch_wide<KEY, true>(a, s) : launch_wide<KEY, false>(a, s);
}

}  // namespace moe
#endif  // MOE_GATE_SELECT
