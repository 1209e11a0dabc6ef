// gate.cu -- the gate: from the router's logits to a routing, with softmax or
// sigmoid scores, a bias that steers the choice and not the weights, groups of
// experts of which a token may use a few, and weights that are renormalised or not;
// its gradient for the logits; the step of the bias.
//
// Per token, l = its E logits:
//   s = softmax(l) or sigmoid(l),  c = s + bias  (no bias: the order of l)
//   a group's score: the sum of its 1 or 2 largest c;  the best `top_groups` groups
//   S = the k largest c in those groups (ties: lower expert)
//   w_j = scale s_{S_j} / (sum_i s_{S_i} or 1)
// and the dispatch indices of the chosen slots, expert by expert, tokens ascending.
//
// Exact choice.  Two scores can be closer than fp32 resolves, and a choice that
// depends on the roundings of an exponential differs from program to program.  The
// choice made here is that of the exact scores: fp32 scores carry an error that
// is bounded (kNearSigmoid, kNearSoftmax below), and a token whose order is not
// decided by more than that is chosen again from scores in 64 bits.  Of 131072 x 256
// normal logits 0.4% are.  Without a bias the logits themselves are compared.
//
// One warp per token, expert e in register e / 32 of lane e % 32.  A score becomes a
// 23-bit fixed-point number above the expert's index in one 32-bit key, so that keys
// are unique and one warp-wide maximum (redux) gives both the next score and whose it
// is.  Each lane sorts its keys once and hands out its largest.  Without a bias the key
// is the upper 24 bits of the logit.
//
// The dispatch indices take two kernels: the first also leaves every slot's rank
// among its chunk's slots of the same expert and the chunk's histogram (a chunk: the
// tokens of one block); in the second every block adds up the histograms in front of
// its chunk.  No block waits for another and nothing has to be zero before a call.  Up
// to eight chunks run as one cluster, which exchanges its histograms itself.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTok = 64;           // tokens of one round of a block
constexpr int kTokWords = kTok / 32;
constexpr int kMaxGroups = 32;
constexpr int kMaxCluster = 8;
constexpr int kIndexThreads = 1024;
constexpr int kIndexSplit = kIndexThreads / kMaxExperts;  // threads that share an expert's column of histograms

// Fixed point: c in [-B, 1 + B], B the largest finite |bias|, as 8 + O + c * scale in
// 23 bits, O = ceil(B scale).  A unit is (1 + 2B) 2^-23 or a little more.
// How far the number may be from that of the exact c, in units:
//   sigmoid: 1 / (1 + e), e = expf(-l) off by 2 ulp (2^-22 of itself, which moves s by
//   s (1 - s) times that), the sum by half an ulp, the reciprocal by one, c = s + b by half:
//   at most s (2^-22 + 2^-24 + 2^-23) + |c| 2^-24 <= (1 + B) 4.8e-7, under 4.1 units, and
//   half for the rounding to fixed point: under 5.  Two numbers that differ by more than
//   10 are in the order of the exact ones.
//   softmax: e = expf(l - m) off by 2 ulp and |l - m| 2^-24 for the difference, which with
//   the e^-|l - m| of its size is at most 0.37 2^-24; the sum Z by 13 roundings and its
//   terms, 1.1e-6; the quotient by 2 ulp: 1.7e-6 in all, 14.3 units, with the rounding
//   under 15: 30.
constexpr int kNearSigmoid = 10, kNearSoftmax = 30;
constexpr float kFixOne = 8388608.f;       // 2^23
constexpr uint32_t kUnscored = 1;          // the number of an expert that may not be chosen
constexpr float kFixLeast = 8.f;           // a scored one's is above

enum GateKey : int { kKeyLogit = 0, kKeySigmoid = 1, kKeySoftmax = 2 };

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
  int chunk;            // tokens per chunk, a multiple of kTok
  int chunks;
  int32_t *hist;        // [chunks][E]
  int32_t *flags;       // [chunks]
  int32_t *status;
};

__device__ __forceinline__ float clean_logit(float l, bool &bad) {
  bad |= !(l <= FLT_MAX);
  return l != l ? -INFINITY : fminf(l, FLT_MAX);
}

// A logit's order as an unsigned number (both zeros alike).
__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t u = __float_as_uint(l + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float sigmoid_fast(float l) { return __fdividef(1.f, 1.f + expf(-l)); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sorts NV keys, largest first.
template <int NV>
__device__ __forceinline__ void sort_keys(uint32_t (&v)[NV]) {
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
  }
}

// What the block keeps of the bias.
struct BiasInfo {
  float scale;  // units per 1
  float base;   // 2^23 + 8 + O
  int off;      // 8 + O: the number of c = 0
  bool odd;     // some entry is not finite
};

// The choice of one token from 64-bit scores, by one warp.  kept: the groups that may be
// used, or all_groups to choose those as well; only experts whose fp32 number is at least
// `least` can be among the chosen (0: every one).  val: E doubles of this warp.  Lane
// j < k returns its expert, with bit 15 where that had no score.
template <int KEY>
__device__ __noinline__ int resolve_token(const GateArgs &a, const float *row, const float *s_bias, BiasInfo bi,
                                          uint32_t kept, bool choose_groups, int least, double *val) {
  const int lane = threadIdx.x & 31, E = a.E;
  const bool biased = a.bias != nullptr;
  bool bad = false;
  double top = -DBL_MAX, z = 1.0;
  float top32 = -FLT_MAX, z32 = 1.f;
  if (!a.sigmoid && KEY != kKeyLogit) {
    for (int e = lane; e < E; e += 32) top32 = fmaxf(top32, clean_logit(__ldg(row + e), bad));
    top32 = warp_max(top32);
    top = top32;
    z = 0.0;
    for (int e = lane; e < E; e += 32) z += exp(static_cast<double>(clean_logit(__ldg(row + e), bad)) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z32 = static_cast<float>(z);
  }
  // the score of expert e as the order of the experts (order) or of the groups uses it
  auto exact = [&](float l, float b, bool order) -> double {
    if (KEY == kKeyLogit || (order && !biased)) return static_cast<double>(l);
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l))) : exp(static_cast<double>(l) - top) / z;
    return biased ? s + static_cast<double>(b) : s;
  };
  auto scored = [&](float l, float b) { return l >= -FLT_MAX && b > -INFINITY; };  // (not where b is NaN)
  if (choose_groups) {
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
    kept = __ballot_sync(0xffffffffu, lane < a.groups && before < a.top_groups);
    least = 0;
  }
  for (int e = lane; e < E; e += 32) {
    const float l = clean_logit(__ldg(row + e), bad), b = biased ? s_bias[e] : 0.f;
    bool use = scored(l, b) && ((kept >> (e / a.group_size)) & 1u);
    if (KEY != kKeyLogit && use && least > 0) {
      // the fp32 number once more; half of the distance that decides on top for safety
      const float s = a.sigmoid ? sigmoid_fast(l) : __fdividef(expf(l - top32), z32);
      use = fmaf(s + b, bi.scale, static_cast<float>(bi.off)) >= static_cast<float>(least) - kNearSoftmax;
    }
    val[e] = use ? exact(l, b, true) : -INFINITY;
  }
  __syncwarp();
  // k times the best of what is left; taken ones become NaN, which no comparison prefers
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int at = INT_MAX;
    for (int e = lane; e < E; e += 32) {
      const double v = val[e];
      if (v > best || (v == best && e < at)) best = v, at = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (ov > best || (ov == best && oa < at)) best = ov, at = oa;
    }
    if (lane == j) mine = at | (best == -INFINITY ? 0x8000 : 0);
    if ((at & 31) == lane) val[at] = NAN;
    __syncwarp();
  }
  return mine;
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

__device__ __forceinline__ int32_t ld_peer(const int32_t *p, int rank) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_smem_addr(p, rank)) : "memory");
  return v;
}

// NV = experts per lane.  ONE: the chunks are one cluster, one round each, and leave nothing for
// a second kernel.
template <int NV, int KEY, bool GROUPS, bool ONE>
__global__ void __launch_bounds__(kThreads) gate_select_kernel(const GateArgs a) {
  __shared__ float s_bias[kMaxExperts];
  __shared__ uint32_t s_emask[kMaxExperts][kTokWords];  // tokens of this round that chose expert e
  __shared__ int32_t s_run[kMaxExperts];                // the chunk's slots of expert e so far
  __shared__ uint16_t s_slot[kTok * kMaxTopK];          // expert of each slot; bit 15: without a score
  __shared__ uint32_t s_keys[GROUPS ? kWarps : 1][GROUPS ? kMaxExperts : 1];
  __shared__ double s_val[kWarps][kMaxExperts];
  __shared__ float2 s_soft[kTok];                       // softmax weights: a token's largest logit, and its sum
  __shared__ int32_t s_flag;
  __shared__ float s_bmax[kWarps];
  __shared__ int32_t s_bodd;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.E, k = a.k;
  const int first = blockIdx.x * a.chunk, last = min(a.T, first + a.chunk);
  if (tid == 0) s_flag = 0, s_bodd = 0;
  for (int i = tid; i < E * kTokWords; i += kThreads) (&s_emask[0][0])[i] = 0u;
  if (tid < E) s_run[tid] = 0;
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();

  BiasInfo bi{kFixOne - 32.f, kFixOne + kFixLeast, static_cast<int>(kFixLeast), false};
  __syncthreads();
  if (KEY != kKeyLogit && a.bias) {
    float b = tid < E ? __ldg(a.bias + tid) : 0.f;
    if (tid < E) s_bias[tid] = b;
    const bool odd = !(fabsf(b) <= FLT_MAX);
    if (odd) s_bodd = 1;
    float m = odd ? 0.f : fabsf(b);
    m = warp_max(m);
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
  }
  float bias[NV];
  uint32_t gid[GROUPS ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    bias[i] = KEY != kKeyLogit && a.bias && e < E ? s_bias[e] : 0.f;
    if (GROUPS) gid[i] = e / a.group_size;
  }
  const bool whole_sum = !a.sigmoid && !a.renormalise;  // the weights need the softmax' sum over all experts
  constexpr int kNear = KEY == kKeyLogit ? 0 : (KEY == kKeySigmoid ? kNearSigmoid : kNearSoftmax);

  auto load = [&](int t, float (&v)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      v[i] = t < last && e < E ? __ldg(a.logits + static_cast<size_t>(t) * E + e) : -INFINITY;
    }
  };
  float ahead[NV];
  load(first + warp, ahead);
  bool bad = false;

  for (int t0 = first; t0 < last; t0 += kTok) {
    // ---- choice: this warp's tokens, kWarps apart
#pragma unroll 1
    for (int tl = warp; tl < kTok; tl += kWarps) {
      const int t = t0 + tl;
      if (t >= last) break;
      float l[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = ahead[i];
      load(t + kWarps, ahead);  // (of the next round after the last)
      bool odd = false;
#pragma unroll
      for (int i = 0; i < NV; ++i) odd |= (lane + 32 * i < E) && !(fabsf(l[i]) <= FLT_MAX);
      odd = __any_sync(0xffffffffu, odd);
      if (odd) {
#pragma unroll
        for (int i = 0; i < NV; ++i) l[i] = clean_logit(l[i], bad);
      }
      uint32_t key[NV];
      if constexpr (KEY == kKeyLogit) {
        if (whole_sum) {
          float m = -FLT_MAX, z = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i]);
          m = warp_max(m);
#pragma unroll
          for (int i = 0; i < NV; ++i) z += expf(l[i] - m);
          z = warp_sum(z);
          if (lane == 0) s_soft[tl] = make_float2(m, z);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = (order_of(l[i]) & 0xFFFFFF00u) | (255u - (lane + 32 * i));
      } else {
        float s[NV];
        if constexpr (KEY == kKeySigmoid) {
#pragma unroll
          for (int i = 0; i < NV; ++i) s[i] = sigmoid_fast(l[i]);
        } else {
          float m = -FLT_MAX, z = 0.f;
#pragma unroll
          for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i]);
          m = warp_max(m);
#pragma unroll
          for (int i = 0; i < NV; ++i) z += s[i] = expf(l[i] - m);
          z = warp_sum(z);
          if (lane == 0) s_soft[tl] = make_float2(m, z);
#pragma unroll
          for (int i = 0; i < NV; ++i) s[i] = __fdividef(s[i], z);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float x = fmaf(s[i] + bias[i], bi.scale, bi.base);  // a whole number in [2^23, 2^24)
          key[i] = (__float_as_uint(x) << 8) | (255u - (lane + 32 * i));
          if (bi.odd && bias[i] > FLT_MAX) key[i] = 0x7FFFFF00u | (255u - (lane + 32 * i));
        }
      }
      // what may not be chosen: after everything else, by index; past E: never
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        const bool without = (odd && !(l[i] >= -FLT_MAX)) || (KEY != kKeyLogit && bi.odd && !(bias[i] > -INFINITY));
        if (without) key[i] = (kUnscored << 8) | (255u - e);
        if (32 * (i + 1) > E && e >= E) key[i] = 0;
      }
      bool undecided = false, choose_groups = false;
      uint32_t kept = 0xffffffffu;
      if constexpr (GROUPS) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s_keys[warp][lane + 32 * i] = key[i];
        __syncwarp();
        const int G = a.groups, gs = a.group_size;
        int P = 1;
        while (2 * P * G <= 32) P *= 2;
        const int g = lane % G, p = lane / G;
        const int its = (gs + P - 1) / P;
        uint32_t k1 = 0, k2 = 0;
        if (p < P) {
          int it = g % its;  // each group starts elsewhere: other banks
          for (int n = 0; n < its; ++n) {
            const int m = p + P * it;
            const uint32_t v = m < gs ? s_keys[warp][g * gs + m] : 0u;
            k2 = max(k2, min(k1, v));
            k1 = max(k1, v);
            if (++it == its) it = 0;
          }
        }
        for (int o = P / 2; o > 0; o >>= 1) {
          const uint32_t o1 = __shfl_down_sync(0xffffffffu, k1, o * G), o2 = __shfl_down_sync(0xffffffffu, k2, o * G);
          k2 = max(max(k2, o2), min(k1, o1));
          k1 = max(k1, o1);
        }
        __syncwarp();
        int gv = INT_MIN;
        if (lane < G && (k1 >> 8) > kUnscored) {
          if (KEY == kKeyLogit) {
            gv = static_cast<int>(k1 >> 8);
          } else {
            gv = static_cast<int>(k1 >> 8) - bi.off;
            if (a.group_best == 2 && (k2 >> 8) > kUnscored) gv += static_cast<int>(k2 >> 8) - bi.off;
          }
        }
        int before = 0;
        for (int h = 0; h < G; ++h) {
          const int o = __shfl_sync(0xffffffffu, gv, h);
          before += (o > gv || (o == gv && h < lane)) ? 1 : 0;
        }
        kept = __ballot_sync(0xffffffffu, lane < G && before < a.top_groups);
        if (a.top_groups < G) {
          const uint32_t in = __ballot_sync(0xffffffffu, lane < G && before == a.top_groups - 1);
          const uint32_t out = __ballot_sync(0xffffffffu, lane < G && before == a.top_groups);
          const int vi = __shfl_sync(0xffffffffu, gv, __ffs(in) - 1), vo = __shfl_sync(0xffffffffu, gv, __ffs(out) - 1);
          // (in 64 bits: the lowest value stands for a group without any score)
          choose_groups = vo != INT_MIN && (bi.odd || static_cast<int64_t>(vi) - vo <= 2 * kNear);
        }
        undecided = choose_groups;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (!((kept >> (gid[i] & 31)) & 1u) && key[i]) key[i] = (kUnscored << 8) | (255u - (lane + 32 * i));
      }
      int mine = 0;
      uint32_t got = 0;
      if (!undecided) {
        sort_keys<NV>(key);
        for (int j = 0; j <= k; ++j) {
          const uint32_t r = __reduce_max_sync(0xffffffffu, key[0]);
          if (lane == j) got = r;
          if (key[0] == r) {
#pragma unroll
            for (int i = 0; i + 1 < NV; ++i) key[i] = key[i + 1];
            key[NV - 1] = 0;
          }
        }
        const uint32_t next = __shfl_down_sync(0xffffffffu, got, 1);
        const int q = static_cast<int>(got >> 8), qn = static_cast<int>(next >> 8);
        mine = static_cast<int>(255u - (got & 255u)) | (q <= static_cast<int>(kUnscored) ? 0x8000 : 0);
        bool near = lane < k && qn > static_cast<int>(kUnscored) && q - qn <= kNear;
        if (__any_sync(0xffffffffu, near)) {
          const float *row = a.logits + static_cast<size_t>(t) * E;
          // equal in logit and bias: an exact tie, which the index has decided
          auto same = [&](int e0, int e1) {
            return __ldg(row + e0) == __ldg(row + e1) && (KEY == kKeyLogit || !a.bias || s_bias[e0] == s_bias[e1]);
          };
          if (near) near = !same(255 - (got & 255u), 255 - (next & 255u));
          // and none of those behind may be as near to the last one chosen without being its equal
          const uint32_t end = __shfl_sync(0xffffffffu, got, k - 1);
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if ((key[i] >> 8) > kUnscored && static_cast<int>(end >> 8) - static_cast<int>(key[i] >> 8) <= kNear)
              near |= !same(255 - (end & 255u), 255 - (key[i] & 255u));
          undecided = __any_sync(0xffffffffu, near);
        }
      }
      if (undecided) {
        const int least = choose_groups ? 0 : static_cast<int>(__shfl_sync(0xffffffffu, got, k - 1) >> 8);
        mine = resolve_token<KEY>(a, a.logits + static_cast<size_t>(t) * E, s_bias, bi, kept, choose_groups,
                                  least > static_cast<int>(kUnscored) ? max(1, least - 2 * kNear) : 0, s_val[warp]);
      }
      if (lane < k) s_slot[tl * k + lane] = static_cast<uint16_t>(mine);
    }
    __syncthreads();

    // ---- weights: one thread per token
    const int ntok = min(kTok, last - t0);
    if (tid < ntok) {
      const float *row = a.logits + static_cast<size_t>(t0 + tid) * E;
      const size_t at = static_cast<size_t>(t0 + tid) * k;
      float l[kMaxTopK];
      float top = -INFINITY;
      bool bad_here = false;
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j) {
        if (j < k) {
          const int v = s_slot[tid * k + j], e = v & 0x7FFF;
          l[j] = v & 0x8000 ? -INFINITY : clean_logit(__ldg(row + e), bad_here);
          top = fmaxf(top, l[j]);
          a.topk_idx[at + j] = e;
          atomicOr(&s_emask[e][tid >> 5], 1u << (tid & 31));
        }
      }
      // Renormalised, scores enter by their ratios: relative to e^top, which keeps scores that
      // underflow (sigmoid: relative to e^min(top, 0), since s <= 1).
      const bool none = top == -INFINITY;
      float sum = 0.f;
      if (a.sigmoid) {
        const float m = a.renormalise && !none ? fminf(top, 0.f) : 0.f;
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
          if (j < k) {  // e^(l - m) / (1 + e^l), by the exponential that does not overflow
            const float x = expf(-fabsf(l[j]));
            l[j] = l[j] > 0.f ? 1.f / (1.f + x) : expf(l[j] - m) / (1.f + x);
            sum += l[j];
          }
        }
      } else {
        if (whole_sum) top = s_soft[tid].x;
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
          if (j < k) {
            l[j] = none ? 0.f : expf(l[j] - top);
            sum += l[j];
          }
        }
        if (whole_sum) sum = s_soft[tid].y;
      }
      const float f = none ? 0.f : a.scale / (a.sigmoid && !a.renormalise ? 1.f : sum);
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j)
        if (j < k) {
          l[j] = l[j] * f;
          a.topk_w[at + j] = l[j];
        }
    }
    __syncthreads();

    // ---- ranks: a slot's place among the chunk's slots of its expert
    for (int sl = tid; sl < ntok * k; sl += kThreads) {
      const int tl = sl / k, e = s_slot[sl] & 0x7FFF;
      const uint32_t *mk = s_emask[e];
      int r = s_run[e] + __popc(mk[tl >> 5] & ((1u << (tl & 31)) - 1u));
#pragma unroll
      for (int w = 0; w < kTokWords - 1; ++w) r += w < (tl >> 5) ? __popc(mk[w]) : 0;
      a.row_of_slot[static_cast<size_t>(t0) * k + sl] = r;
    }
    __syncthreads();
    if (tid < E) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < kTokWords; ++w) {
        c += __popc(s_emask[tid][w]);
        s_emask[tid][w] = 0u;
      }
      s_run[tid] += c;
    }
    __syncthreads();
  }
  if (bad) s_flag = 1;
  if constexpr (!ONE) {
    if (tid < E) a.hist[static_cast<size_t>(blockIdx.x) * E + tid] = s_run[tid];
    __syncthreads();
    if (tid == 0) a.flags[blockIdx.x] = s_flag ? kDevNonfiniteLogit : 0;
  } else {
    __shared__ int32_t s_base[kMaxExperts];
    __shared__ int s_w[kMaxExperts / 32];
    cluster_sync();  // every block's histogram
    int before = 0, all = 0, n;
    if (tid < E)
      for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
        const int v = ld_peer(&s_run[tid], c);
        before += c < static_cast<int>(blockIdx.x) ? v : 0;
        all += v;
      }
    const int off = expert_prefix(tid < E ? all : 0, s_w, &n);
    if (tid < E) s_base[tid] = off + before;
    if (blockIdx.x == 0) {
      if (tid < E) {
        a.counts[tid] = all;
        a.offsets[tid] = off;
      }
      if (tid == 0) {
        a.offsets[E] = n;
        int f = 0;
        for (int c = 0; c < static_cast<int>(gridDim.x); ++c) f |= ld_peer(&s_flag, c);
        *a.status = f ? kDevNonfiniteLogit : 0;
      }
    }
    __syncthreads();
    const int slots = max(0, last - first) * k;
    for (int sl = tid; sl < slots; sl += kThreads) {
      const size_t s = static_cast<size_t>(first) * k + sl;
      const int row = s_base[s_slot[sl] & 0x7FFF] + a.row_of_slot[s];  // (this block's own write)
      a.row_of_slot[s] = row;
      a.slot_of_row[row] = static_cast<int32_t>(s);
      a.w_row[row] = a.topk_w[s];
    }
    cluster_sync();  // before a block leaves that others read
  }
}

// The second kernel: a block takes the chunks `per` at a time.
__global__ void __launch_bounds__(kIndexThreads) gate_index_kernel(const GateArgs a, int per) {
  __shared__ int32_t s_part[2][kIndexSplit][kMaxExperts];  // per thread: rows in front of the block's chunks, and all
  __shared__ int32_t s_base[kMaxExperts];
  __shared__ int s_w[kMaxExperts / 32];
  const int tid = threadIdx.x, E = a.E;
  const int c0 = blockIdx.x * per, c1 = min(a.chunks, c0 + per);
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  {
    const int e = tid % kMaxExperts, part = tid / kMaxExperts;
    int before = 0, all = 0;
    if (e < E) {
      constexpr int kBatch = 16;
      for (int c = part; c < a.chunks; c += kIndexSplit * kBatch) {
        int h[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int cc = c + i * kIndexSplit;
          h[i] = cc < a.chunks ? __ldcg(a.hist + static_cast<size_t>(cc) * E + e) : 0;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          before += c + i * kIndexSplit < c0 ? h[i] : 0;
          all += h[i];
        }
      }
    }
    s_part[0][part][e] = before;
    s_part[1][part][e] = all;
  }
  __syncthreads();
  int before = 0, all = 0, n;
  if (tid < kMaxExperts) {
#pragma unroll
    for (int p = 0; p < kIndexSplit; ++p) {
      before += s_part[0][p][tid];
      all += s_part[1][p][tid];
    }
  }
  const int off = expert_prefix(all, s_w, &n);  // (threads past the experts: zeros)
  if (tid < E) {
    s_base[tid] = off + before;
    if (blockIdx.x == 0) {
      a.counts[tid] = all;
      a.offsets[tid] = off;
      if (tid == 0) a.offsets[E] = n;
    }
  }
  if (blockIdx.x == 0) {
    int f = 0;
    for (int c = tid; c < a.chunks; c += kIndexThreads) f |= a.flags[c];
    f = __syncthreads_or(f);
    if (tid == 0) *a.status = f ? kDevNonfiniteLogit : 0;
  }
  __syncthreads();
  for (int c = c0; c < c1; ++c) {
    const int64_t s0 = static_cast<int64_t>(c) * a.chunk * a.k;
    const int64_t s1 = min(static_cast<int64_t>(a.T) * a.k, s0 + static_cast<int64_t>(a.chunk) * a.k);
    for (int64_t s = s0 + tid; s < s1; s += kIndexThreads) {
      const int row = s_base[__ldg(a.topk_idx + s)] + a.row_of_slot[s];
      a.row_of_slot[s] = row;
      a.slot_of_row[row] = static_cast<int32_t>(s);
      a.w_row[row] = __ldg(a.topk_w + s);
    }
    if (c + 1 < c1) {  // the next chunk's bases
      __syncthreads();
      if (tid < E) s_base[tid] += __ldcg(a.hist + static_cast<size_t>(c) * E + tid);
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- gradient
//
// With g = d w, n_j = w_j / scale, for the chosen experts:
//   softmax, renormalised   dl_j = w_j (g_j - sum_i n_i g_i)
//   sigmoid, renormalised   dl_j = w_j (1 - s_j) (g_j - sum_i n_i g_i)
//   sigmoid                 dl_j = w_j (1 - s_j) g_j
// and zero for the others; softmax that is not renormalised gives every expert a gradient:
//   dl_e = w_e g_e - p_e sum_i w_i g_i       (w_e = 0 for the others)
// A slot of weight zero has none.  Bound by the gradient's bytes (and the dense kind's
// logits): a block builds whole rows in shared memory and one bulk copy takes them out.

constexpr int kGradThreads = 256;
constexpr int kGradBytes = 16 * 1024;  // rows of one buffer at most

struct GradArgs {
  const float *logits;
  const int32_t *topk_idx;
  const float *topk_w, *d_topk_w;
  float *d_logits;
  int T, E, k;
  int rows;  // tokens per round, a multiple of 4
  bool sigmoid, renormalise;
  float scale;
};

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

template <bool DENSE>
__global__ void __launch_bounds__(kGradThreads) gate_grad_kernel(const GradArgs a) {
  extern __shared__ __align__(128) float s_rows[];  // [2][rows * E]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.E, k = a.k, span = a.rows * E;
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  int buf = 0;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.rows; t0 < a.T; t0 += static_cast<int64_t>(gridDim.x) * a.rows) {
    const int n = static_cast<int>(min(static_cast<int64_t>(a.rows), a.T - t0));
    float *rows = s_rows + buf * span;
    // the copy before the last has read this buffer
    if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncthreads();
    if constexpr (!DENSE) {
      for (int i = tid * 4; i < span; i += kGradThreads * 4) *reinterpret_cast<float4 *>(rows + i) = make_float4(0, 0, 0, 0);
      __syncthreads();
    }
    if constexpr (DENSE) {
      for (int r = warp; r < n; r += kGradThreads / 32) {  // a warp per token
        const int64_t t = t0 + r;
        const float *lr = a.logits + t * E;
        float wg = 0.f;
        int e = -1;
        if (lane < k) {
          e = __ldg(a.topk_idx + t * k + lane);
          if (e < 0 || e >= E) e = -1;
          if (e >= 0) wg = __ldg(a.topk_w + t * k + lane) * __ldg(a.d_topk_w + t * k + lane);
        }
        float v[kMaxExperts / 32];
        float top = -INFINITY, z = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
          const int c = lane + 32 * i;
          v[i] = c < E ? clean_logit(__ldg(lr + c), bad) : -INFINITY;
          top = fmaxf(top, v[i]);
        }
        top = warp_max(top);
        const bool none = top == -INFINITY;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
          v[i] = none ? 0.f : expf(v[i] - top);
          z += v[i];
        }
        const float dot = warp_sum(wg);
        z = warp_sum(z);
        const float f = none ? 0.f : -dot / z;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i)
          if (lane + 32 * i < E) rows[r * E + lane + 32 * i] = v[i] * f;
        __syncwarp();
        if (e >= 0) rows[r * E + e] += wg;
      }
    } else {
      for (int r = tid; r < n; r += kGradThreads) {  // a thread per token
        const int64_t at = (t0 + r) * k;
        const float *lr = a.logits + (t0 + r) * E;
        float w[kMaxTopK], g[kMaxTopK];
        int e[kMaxTopK];
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
          if (j < k) {
            e[j] = __ldg(a.topk_idx + at + j);
            w[j] = __ldg(a.topk_w + at + j);
            g[j] = __ldg(a.d_topk_w + at + j);
            if (e[j] < 0 || e[j] >= E || w[j] == 0.f) e[j] = -1;
            if (e[j] >= 0) dot = fmaf(w[j] / a.scale, g[j], dot);
          }
        }
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) {
          if (j < k && e[j] >= 0) {
            float d = w[j] * (a.renormalise ? g[j] - dot : g[j]);
            if (a.sigmoid) {  // 1 - s = 1 / (1 + e^l)
              const float l = __ldg(lr + e[j]);
              d *= 1.f / (1.f + expf(l));
            }
            rows[r * E + e[j]] = d;
          }
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    // whole 16-byte vectors go out in one copy (t0 * E is a multiple of four); what is left of
    // the tensor's end as single elements
    const int len = n * E, whole = len & ~3;
    float *dst = a.d_logits + t0 * E;
    if (tid == 0) {
      if (whole)
        bulk_store(dst, rows, static_cast<uint32_t>(whole) * 4);
      else
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    if (tid < len - whole) dst[whole + tid] = rows[whole + tid];
    buf ^= 1;
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// bias_e += rate * sign(mean load - load of e), the counts of all rows added up; compared as
// whole numbers: sum_e' c_e' against E c_e.
__global__ void __launch_bounds__(kIndexThreads) gate_bias_kernel(const int32_t *counts, int rows, int E, float rate,
                                                                  float *bias) {
  __shared__ unsigned long long s_load[kMaxExperts], s_all;
  const int e = threadIdx.x % kMaxExperts, part = threadIdx.x / kMaxExperts;
  if (threadIdx.x < kMaxExperts) s_load[threadIdx.x] = 0;
  if (threadIdx.x == 0) s_all = 0;
  __syncthreads();
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  long long c = 0;
  if (e < E)
    for (int r = part; r < rows; r += kIndexSplit) c += __ldg(counts + static_cast<size_t>(r) * E + e);
  atomicAdd(&s_load[e], static_cast<unsigned long long>(c));
  atomicAdd(&s_all, static_cast<unsigned long long>(c));
  __syncthreads();
  if (threadIdx.x >= E) return;
  const long long d = static_cast<long long>(s_all) - static_cast<long long>(s_load[e]) * E;
  if (d != 0) bias[e] += d > 0 ? rate : -rate;
}

// ---------------------------------------------------------------- host side

bool gate_ok(const moe_gate_config *c) {
  if (!c) return false;
  if (c->T < 0 || c->T > (1 << 30) || c->E < 1 || c->E > kMaxExperts || c->k < 1 || c->k > kMaxTopK || c->k > c->E) return false;
  if (static_cast<int64_t>(c->T) * c->k >= (int64_t{1} << 31)) return false;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return false;
  if (c->groups < 1 || c->groups > kMaxGroups || c->E % c->groups) return false;
  if (c->top_groups < 1 || c->top_groups > c->groups) return false;
  if (c->group_best < 1 || c->group_best > 2) return false;
  if (c->top_groups * (c->E / c->groups) < c->k) return false;
  return c->scale > 0.f && c->scale <= FLT_MAX;  // (not where it is NaN)
}

// Chunks: one round of tokens each while that fills two blocks an SM, then as many rounds as
// make two blocks for each of 152 SMs (their histograms are read by every block of the second kernel).
constexpr int kMostChunks = 304;
struct GateLayout {
  int chunk, chunks;
  size_t flags, hist, total;
};
GateLayout gate_layout(const moe_gate_config *c) {
  GateLayout L;
  const int64_t rounds = (static_cast<int64_t>(c->T) + kTok - 1) / kTok;
  const int64_t per = (rounds + kMostChunks - 1) / kMostChunks;
  L.chunk = static_cast<int>(per < 1 ? 1 : per) * kTok;
  L.chunks = static_cast<int>((static_cast<int64_t>(c->T) + L.chunk - 1) / L.chunk);
  L.flags = kHeader;
  L.hist = L.flags + align256(kMostChunks * 4);
  L.total = L.hist + align256(static_cast<size_t>(L.chunks > 0 ? L.chunks : 1) * c->E * 4);
  return L;
}

template <int NV, int KEY, bool GROUPS>
cudaError_t launch_select(const GateArgs &a, cudaStream_t s) {
  if (a.chunks <= kMaxCluster)
    return launch_pdl(gate_select_kernel<NV, KEY, GROUPS, true>, dim3(a.chunks), dim3(kThreads), 0, s, a.chunks, a);
  return launch_pdl(gate_select_kernel<NV, KEY, GROUPS, false>, dim3(a.chunks), dim3(kThreads), 0, s, 1, a);
}
template <int KEY, bool GROUPS>
cudaError_t launch_by_width(const GateArgs &a, cudaStream_t s) {
  if (a.E <= 32) return launch_select<1, KEY, GROUPS>(a, s);
  if (a.E <= 64) return launch_select<2, KEY, GROUPS>(a, s);
  if (a.E <= 128) return launch_select<4, KEY, GROUPS>(a, s);
  return launch_select<8, KEY, GROUPS>(a, s);
}
template <int KEY>
cudaError_t launch_by_groups(const GateArgs &a, cudaStream_t s) {
  return a.groups > 1 ? launch_by_width<KEY, true>(a, s) : launch_by_width<KEY, false>(a, s);
}

bool gate_routing_ok(const moe_routing *r, int T) {
  if (!r || !r->counts || !r->offsets) return false;
  return T == 0 || (r->topk_idx && r->topk_w && r->row_of_slot && r->slot_of_row && r->w_row);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_gate_workspace(const moe_gate_config *cfg, size_t *fwd_scratch) {
  if (!gate_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (fwd_scratch) *fwd_scratch = gate_layout(cfg).total;
  return MOE_OK;
}

moe_status moe_gate_forward(const moe_gate_config *cfg, const float *logits, const float *bias,
                            const moe_routing *routing, void *scratch, size_t scratch_bytes, void *stream) {
  if (!gate_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!gate_routing_ok(routing, cfg->T) || !scratch || (cfg->T > 0 && !logits)) return MOE_ERR_INVALID_ARG;
  if (!al16(logits) || !al16(bias) || !al16(scratch) || !al16(routing->topk_idx) || !al16(routing->topk_w) ||
      !al16(routing->counts) || !al16(routing->offsets) || !al16(routing->row_of_slot) ||
      !al16(routing->slot_of_row) || !al16(routing->w_row))
    return MOE_ERR_ALIGNMENT;
  const GateLayout L = gate_layout(cfg);
  if (scratch_bytes < L.total) return MOE_ERR_WORKSPACE;
  DevInfo di;
  MOE_TRY(device_info(&di));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t *sc = static_cast<uint8_t *>(scratch);
  GateArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.T = cfg->T;
  a.E = cfg->E;
  a.k = cfg->k;
  a.groups = cfg->groups;
  a.top_groups = cfg->top_groups;
  a.group_best = cfg->group_best;
  a.group_size = cfg->E / cfg->groups;
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.renormalise = cfg->renormalise != 0;
  a.scale = cfg->scale;
  a.topk_idx = routing->topk_idx;
  a.topk_w = routing->topk_w;
  a.counts = routing->counts;
  a.offsets = routing->offsets;
  a.row_of_slot = routing->row_of_slot;
  a.slot_of_row = routing->slot_of_row;
  a.w_row = routing->w_row;
  a.chunk = L.chunk;
  a.chunks = L.chunks;
  a.hist = reinterpret_cast<int32_t *>(sc + L.hist);
  a.flags = reinterpret_cast<int32_t *>(sc + L.flags);
  a.status = reinterpret_cast<int32_t *>(sc);
  if (a.T > 0) {
    // the logits' own order, unless a bias or a sum of two scores enters
    const bool by_logit = !bias && (a.groups == 1 || a.group_best == 1);
    MOE_TRY(timed("gate_select", s, [&] {
      if (by_logit) return launch_by_groups<kKeyLogit>(a, s);
      return a.sigmoid ? launch_by_groups<kKeySigmoid>(a, s) : launch_by_groups<kKeySoftmax>(a, s);
    }));
    if (a.chunks <= kMaxCluster) return MOE_OK;
  }
  return timed("gate_index", s, [&] {
    const int per = (a.chunks + di.sms - 1) / di.sms;
    const int blocks = per ? (a.chunks + per - 1) / per : 1;  // (no tokens: one block writes zeros)
    return launch_pdl(gate_index_kernel, dim3(blocks), dim3(kIndexThreads), 0, s, 1, a, per);
  });
}

moe_status moe_gate_backward(const moe_gate_config *cfg, const float *logits, const int32_t *topk_idx,
                             const float *topk_w, const float *d_topk_w, float *d_logits, void *stream) {
  if (!gate_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!logits || !topk_idx || !topk_w || !d_topk_w || !d_logits)) return MOE_ERR_INVALID_ARG;
  if (!al16(logits) || !al16(topk_idx) || !al16(topk_w) || !al16(d_topk_w) || !al16(d_logits)) return MOE_ERR_ALIGNMENT;
  DevInfo di;
  MOE_TRY(device_info(&di));
  if (cfg->T == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GradArgs a{};
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.d_topk_w = d_topk_w;
  a.d_logits = d_logits;
  a.T = cfg->T;
  a.E = cfg->E;
  a.k = cfg->k;
  a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
  a.renormalise = cfg->renormalise != 0;
  a.scale = cfg->scale;
  const int most = kGradBytes / (4 * a.E) / 4 * 4;  // at least 16
  const int even = static_cast<int>((static_cast<int64_t>(a.T) + 4 * di.sms - 1) / (4 * di.sms) + 3) / 4 * 4;
  a.rows = even < most ? even : most;
  const int64_t rounds = (static_cast<int64_t>(a.T) + a.rows - 1) / a.rows;
  const int blocks = static_cast<int>(rounds < 6 * di.sms ? rounds : 6 * di.sms);
  const size_t smem = 2 * static_cast<size_t>(a.rows) * a.E * 4;
  const bool dense = !a.sigmoid && !a.renormalise;
  return timed("gate_backward", s, [&] {
    return dense ? launch_pdl(gate_grad_kernel<true>, dim3(blocks), dim3(kGradThreads), smem, s, 1, a)
                 : launch_pdl(gate_grad_kernel<false>, dim3(blocks), dim3(kGradThreads), smem, s, 1, a);
  });
}

moe_status moe_gate_update_bias(const moe_gate_config *cfg, float *bias, const int32_t *counts, int32_t rows, float rate,
                                void *stream) {
  if (!gate_ok(cfg) || rows < 0) return MOE_ERR_INVALID_ARG;
  if (!bias || (rows > 0 && !counts)) return MOE_ERR_INVALID_ARG;
  if (!al16(bias) || !al16(counts)) return MOE_ERR_ALIGNMENT;
  DevInfo di;
  MOE_TRY(device_info(&di));
  if (rows == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return timed("gate_bias", s, [&] {
    return launch_pdl(gate_bias_kernel, dim3(1), dim3(kIndexThreads), 0, s, 1, counts, static_cast<int>(rows),
                      static_cast<int>(cfg->E), rate, bias);
  });
}

}  // extern "C"
