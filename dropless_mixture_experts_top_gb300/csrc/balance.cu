// balance.cu -- the router's auxiliary losses with per-expert counts, and their
// gradient.
//
// T tokens are S sequences of T/S tokens.  p_t = softmax(logits_t); c_se counts
// the slots of sequence s's valid tokens that chose expert e, N_s its valid
// tokens, S' the sequences that have any, N = sum N_s:
//   f_se = c_se / (k N_s),  P_se = sum_t p_te / N_s
//   balance loss = (1/S') sum_s E sum_e f_se P_se
//   z loss       = (1/N) sum_t lse_t^2,       lse_t = log sum_e exp logits_te
// The counts are constants to the gradient (top-k has none):
//   d/dlogits_te = g_b E / (S' N_s) p_te (f_se - sum_e' f_se' p_te')
//                  + g_z (2/N) lse_t p_te
// A token whose mask is zero, or whose logits are all -inf, has no part in any
// sum; its lse is stored as +inf, by which the backward knows it.
//
// Both directions read the logits once, in fp32, G lanes (a power of two) per
// token holding its row in registers, the next token's loads issued before this
// one is worked on.  The forward's blocks stay inside one sequence and leave their
// column sums, counts and z sums as one partial row each; a second kernel reduces
// them in a fixed order, so losses are the same bits every time (counts are
// integers, added in any order).  A single short sequence is one block and one
// kernel.
//
// Bounds, measured: the backward moves 12 bytes per logit at 98% of the copy rate
// (131072 x 250: 59 us).  The forward of as many (4 bytes per logit, 20 us at that
// rate) takes 35 to 51 us and is bound by its instructions: 72% of the issue slots are
// taken at 57% of DRAM's rate, and of the 7.6 cycles between two instructions of a warp
// 0.4 are waits for memory (3.1 for earlier results, 2.1 for a free slot or pipe).  Below
// some 20,000 tokens it is the latency of its two kernels (16384 x 128 in four
// sequences: 12 us) or its one (512 x 8: 6).
#include <math.h>

#include <type_traits>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBwdBlocksPerSm = 4;  // backward blocks at most (eight: 16384 x 128 10.3 us against 8.2)
// forward blocks over all sequences at most, unless there are more sequences: three per SM
// (131072 x 250 in 32 sequences 55 us against 66 with two; four are no faster)
constexpr int kMaxBlocks = 456;

struct SeqSum {  // one sequence, or one block's share of it
  float bal, z;
  int n, flags;
};

struct BalArgs {
  const float *logits;      // [T,E]
  const int32_t *topk_idx;  // [T,k]
  const uint8_t *mask;      // [T] or null
  int T, E, k, S, L;        // L = T / S
  int nbs, per;             // blocks per sequence, tokens per block
  int G;                    // lanes per token
  float *loss;              // [2]
  int32_t *counts;          // [S,E]
  float *probs;             // [S,E]
  int32_t *tokens;          // [S]
  float *lse;               // [T]
  float *psum;              // scratch [S*nbs][E]
  int32_t *pcnt;            // scratch [S*nbs][E]
  SeqSum *pblk;             // scratch [S*nbs]
  SeqSum *pseq;             // scratch [S]
  int32_t *ticket, *status;
  float g_bal, g_z;         // backward
  const float *lse_in;
  float *d_logits;
};

// A lane's columns: W consecutive ones (the widest of 4, 2, 1 that divides E, so
// that a row's vectors are aligned), then the next W, G lanes further.
template <int W>
__device__ __forceinline__ int col_of(int j, int lane, int G) {
  return ((j / W) * G + lane) * W + j % W;
}
template <int W> struct VecOf;
template <> struct VecOf<4> { using type = float4; };
template <> struct VecOf<2> { using type = float2; };
template <> struct VecOf<1> { using type = float; };

template <int W, int NV>
__device__ __forceinline__ void load_row(const float *row, int E, int G, int lane, bool in, float fill,
                                         float (&v)[NV]) {
  using Vt = typename VecOf<W>::type;
#pragma unroll
  for (int j = 0; j < NV; j += W) {
    const int c = col_of<W>(j, lane, G);
    if (in && c < E) {
      const Vt q = *reinterpret_cast<const Vt *>(row + c);
      memcpy(&v[j], &q, sizeof(q));
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[j + i] = fill;
    }
  }
}
template <int W, int NV>
__device__ __forceinline__ void store_row(float *row, int E, int G, int lane, const float (&v)[NV]) {
  using Vt = typename VecOf<W>::type;
#pragma unroll
  for (int j = 0; j < NV; j += W) {
    const int c = col_of<W>(j, lane, G);
    if (c < E) {
      Vt q;
      memcpy(&q, &v[j], sizeof(q));
      *reinterpret_cast<Vt *>(row + c) = q;
    }
  }
}

__device__ __forceinline__ float group_sum(float v, int G) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < G) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float group_max(float v, int G) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < G) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// v = exp(v - at) in pairs: 2^((v - at) log2 e) with the difference taken first, so
// that rows of the type's lowest value stay exact.  The product with log2 e is rounded,
// which at a distance of d from `at` is 2^-24 d log2 e of the result (5e-7 at 10, 4e-6 at
// 80, where the result is 2e-35), and what is below 2^-126 is zero: both far below the
// last place of a sum that has 1 in it.  131072 x 256 forward takes 38 us with it, 43 with
// expf; 131072 x 250 51 and 55.
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float exp2_flush(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <int NV>
__device__ __forceinline__ void exp_row(float (&v)[NV], float at) {
  if constexpr (NV == 1) {
    v[0] = exp2_flush((v[0] - at) * kLog2e);
  } else {
    const F2 a2 = f2(at, at), l2 = f2(kLog2e, kLog2e);
#pragma unroll
    for (int j = 0; j < NV; j += 2) {
      const float2 x = f2_get(f2_mul(f2_sub(f2(v[j], v[j + 1]), a2), l2));
      v[j] = exp2_flush(x.x);
      v[j + 1] = exp2_flush(x.y);
    }
  }
}
// a = v s + a, and the sum of v.
template <int NV>
__device__ __forceinline__ void add_scaled(float (&a)[NV], const float (&v)[NV], float s) {
  if constexpr (NV == 1) {
    a[0] = fmaf(v[0], s, a[0]);
  } else {
    const F2 s2 = f2(s, s);
#pragma unroll
    for (int j = 0; j < NV; j += 2) {
      const float2 x = f2_get(f2_fma(f2(v[j], v[j + 1]), s2, f2(a[j], a[j + 1])));
      a[j] = x.x;
      a[j + 1] = x.y;
    }
  }
}
template <int NV>
__device__ __forceinline__ float row_sum(const float (&v)[NV]) {
  if constexpr (NV == 1) {
    return v[0];
  } else {
    F2 t = f2(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < NV; j += 2) t = f2_add(t, f2(v[j], v[j + 1]));
    const float2 x = f2_get(t);
    return x.x + x.y;
  }
}

// One sequence's outputs by its only block: thread e holds expert e's probability
// sum and count (0 past E).  r: its z sum, tokens and flags; thread 0 gets the
// sequence's balance term in r.bal.  Every thread of the block calls it.
__device__ __forceinline__ void finish_seq(const BalArgs &a, int s, float sum, int cnt, SeqSum &r, float *s_w) {
  const float inv_n = r.n > 0 ? 1.f / static_cast<float>(r.n) : 0.f;
  const int e = threadIdx.x;
  if (e < 256) {
    const float P = sum * inv_n;
    if (e < a.E) {
      a.counts[static_cast<size_t>(s) * a.E + e] = cnt;
      a.probs[static_cast<size_t>(s) * a.E + e] = P;
    }
    const float fp = warp_sum(e < a.E ? static_cast<float>(cnt) * P : 0.f);
    if ((e & 31) == 0) s_w[e >> 5] = fp;
  }
  __syncthreads();
  if (e == 0) {
    float b = 0.f;
    for (int w = 0; w < 8; ++w) b += s_w[w];
    r.bal = b * static_cast<float>(a.E) / static_cast<float>(a.k) * inv_n;
    a.tokens[s] = r.n;
  }
}
__device__ __forceinline__ void finish_all(const BalArgs &a, float bal, float z, int n, int used, int flags) {
  a.loss[0] = used > 0 ? bal / static_cast<float>(used) : 0.f;
  a.loss[1] = n > 0 ? z / static_cast<float>(n) : 0.f;
  *a.status = flags;
}

template <int W, int NV, bool SOLO>
__global__ void __launch_bounds__(kThreads) balance_fwd_kernel(const BalArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  if (!SOLO) griddep_launch_dependents();  // the finishing kernel may be set up meanwhile
  __shared__ int s_cnt[kMaxExperts];
  __shared__ float s_col[kWarps][kMaxExperts];
  __shared__ SeqSum s_blk[kWarps];
  __shared__ float s_w[kWarps];
  const int warp = threadIdx.x >> 5, l32 = threadIdx.x & 31;
  const int E = a.E, G = a.G, lane = l32 & (G - 1), sub = l32 / G, tpw = 32 / G;
  const int seq = blockIdx.x / a.nbs, blk = blockIdx.x - seq * a.nbs;
  const int i0 = blk * a.per, i1 = min(i0 + a.per, a.L);  // tokens of the sequence
  const size_t tbase = static_cast<size_t>(seq) * a.L;
  const int step = kWarps * tpw;  // tokens of one pass of the block
  // the next token's logits, mask and first slots are loaded before this one is
  // worked on
  constexpr int kAhead = 2;  // slots per lane that are loaded ahead
  float v[NV], next[NV];
  int slot[kAhead], next_slot[kAhead];
  bool next_ok;
  auto fetch = [&](int i) {
    const bool in = i < i1;
    load_row<W>(a.logits + (tbase + i) * E, E, G, lane, in, -INFINITY, next);
    next_ok = in && (!a.mask || a.mask[tbase + i] != 0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int q = lane + G * u;
      next_slot[u] = in && q < a.k ? a.topk_idx[(tbase + i) * a.k + q] : -1;
    }
  };
  int ib = i0 + warp * tpw;
  fetch(ib + sub);
  if (!SOLO && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  for (int e = threadIdx.x; e < E; e += kThreads) s_cnt[e] = 0;
  __syncthreads();
  float col[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) col[j] = 0.f;
  float z = 0.f;
  int n = 0, flags = 0;
  for (; ib < i1; ib += step) {
    const int i = ib + sub;
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = next[j];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) slot[u] = next_slot[u];
    bool ok = next_ok;
    fetch(i + step);
    float mx = v[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) mx = fmaxf(mx, v[j]);
    mx = group_max(mx, G);  // NaNs are passed over here, and show in the sum
    if (__any_sync(0xffffffffu, ok && mx == -INFINITY)) {  // -inf throughout: no part in the losses
      float nan = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) nan = v[j] != v[j] ? 1.f : nan;
      nan = group_max(nan, G);  // by every lane of the warp: its shuffles name them all
      if (mx == -INFINITY && nan == 0.f) ok = false;
    }
    exp_row(v, mx);
    const float sum = group_sum(row_sum(v), G);
    const float lse = mx + logf(sum);  // NaN with a NaN or +inf logit
    if (ok) {
      add_scaled(col, v, 1.f / sum);
      if (lane == 0) {
        z = fmaf(lse, lse, z);
        n += 1;
        if (lse != lse) flags |= kDevNonfiniteLogit;
      }
      auto count = [&](int e) {
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E))
          atomicAdd(&s_cnt[e], 1);
        else
          flags |= kDevBadIndex;
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (lane + G * u < a.k) count(slot[u]);
      for (int q = lane + G * kAhead; q < a.k; q += G) count(a.topk_idx[(tbase + i) * a.k + q]);
    }
    if (lane == 0 && i < i1) a.lse[tbase + i] = ok ? lse : INFINITY;
  }
  // the warp's token groups, then the block's warps, in a fixed order
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float c = col[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o >= G) c += __shfl_xor_sync(0xffffffffu, c, o);
    const int e = col_of<W>(j, lane, G);
    if (sub == 0 && e < E) s_col[warp][e] = c;
  }
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (l32 == 0) s_blk[warp] = SeqSum{0.f, z, n, flags};
  __syncthreads();
  SeqSum r = s_blk[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    r.z += s_blk[w].z;
    r.n += s_blk[w].n;
    r.flags |= s_blk[w].flags;
  }
  float c = 0.f;
  const int e = threadIdx.x;  // kThreads >= E
  if (e < E) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) c += s_col[w][e];
  }
  if constexpr (SOLO) {  // the only block: the results themselves
    finish_seq(a, 0, e < E ? c : 0.f, e < E ? s_cnt[e] : 0, r, s_w);
    if (threadIdx.x == 0) finish_all(a, r.n > 0 ? r.bal : 0.f, r.z, r.n, r.n > 0 ? 1 : 0, r.flags);
  } else {
    if (e < E) {
      a.psum[static_cast<size_t>(blockIdx.x) * E + e] = c;
      a.pcnt[static_cast<size_t>(blockIdx.x) * E + e] = s_cnt[e];
    }
    if (threadIdx.x == 0) a.pblk[blockIdx.x] = r;
  }
}

// The blocks' partial rows added: a cluster of blocks per sequence, 32 experts per
// block (a warp of columns, 32 interleaved runs of rows); the first block of the
// cluster gets the others' part of the balance term through distributed shared
// memory.  Of several sequences, the last cluster to finish (a ticket) adds them.
constexpr int kFinThreads = 1024, kFinCols = 32, kFinRuns = kFinThreads / kFinCols;
__global__ void __launch_bounds__(kFinThreads) balance_finish_kernel(const BalArgs a) {
  cluster_arrive();  // waited for below, before the first block's shared memory is written
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s_sum[kFinRuns][kFinCols + 1];
  __shared__ int s_cnt[kFinRuns][kFinCols + 1];
  __shared__ SeqSum s_warp[kFinRuns];
  __shared__ float s_bal[kMaxExperts / kFinCols];
  __shared__ int s_last;
  const int E = a.E, groups = (E + kFinCols - 1) / kFinCols;
  const int s = blockIdx.x / groups, cg = blockIdx.x - s * groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = cg * kFinCols + lane;
  const size_t row0 = static_cast<size_t>(s) * a.nbs;
  float sum = 0.f;
  int cnt = 0;
  constexpr int U = 10;  // loads of each kind in flight
  for (int b0 = warp; b0 < a.nbs; b0 += kFinRuns * U) {
    float v[U];
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + kFinRuns * u;
      const bool in = b < a.nbs && e < E;
      v[u] = in ? a.psum[(row0 + b) * E + e] : 0.f;
      c[u] = in ? a.pcnt[(row0 + b) * E + e] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      sum += v[u];
      cnt += c[u];
    }
  }
  SeqSum r{0.f, 0.f, 0, 0};
  for (int b = threadIdx.x; b < a.nbs; b += kFinThreads) {
    const SeqSum q = a.pblk[row0 + b];
    r.z += q.z;
    r.n += q.n;
    r.flags |= q.flags;
  }
  r.z = warp_sum(r.z);
  r.n = __reduce_add_sync(0xffffffffu, r.n);
  r.flags = __reduce_or_sync(0xffffffffu, r.flags);
  s_sum[warp][lane] = sum;
  s_cnt[warp][lane] = cnt;
  if (lane == 0) s_warp[warp] = r;
  __syncthreads();
  cluster_wait();  // every block of the cluster runs: its shared memory may be reached
  if (warp == 0) {  // lane = expert
    r = s_warp[lane];  // kFinRuns == 32
    r.z = warp_sum(r.z);
    r.n = __reduce_add_sync(0xffffffffu, r.n);
    r.flags = __reduce_or_sync(0xffffffffu, r.flags);
#pragma unroll
    for (int q = 1; q < kFinRuns; ++q) {
      sum += s_sum[q][lane];
      cnt += s_cnt[q][lane];
    }
    const float inv_n = r.n > 0 ? 1.f / static_cast<float>(r.n) : 0.f;
    const float P = sum * inv_n;
    if (e < E) {
      a.counts[static_cast<size_t>(s) * E + e] = cnt;
      a.probs[static_cast<size_t>(s) * E + e] = P;
    }
    const float fp = warp_sum(static_cast<float>(cnt) * P);
    if (lane == 0) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_smem_addr(s_bal + cg, 0)), "f"(fp) : "memory");
    __syncwarp();
  }
  cluster_sync();
  if (cg != 0) return;
  if (threadIdx.x == 0) {
    float b = 0.f;
    for (int q = 0; q < groups; ++q) b += s_bal[q];
    r.bal = r.n > 0 ? b * static_cast<float>(E) / static_cast<float>(a.k) / static_cast<float>(r.n) : 0.f;
    a.tokens[s] = r.n;
    if (a.S == 1) {
      finish_all(a, r.bal, r.z, r.n, r.n > 0 ? 1 : 0, r.flags);
    } else {
      a.pseq[s] = r;
      __threadfence();
      s_last = atomicAdd(a.ticket, 1) == a.S - 1;
      if (s_last) __threadfence();
    }
  }
  if (a.S == 1) return;
  __syncthreads();
  if (!s_last || threadIdx.x >= 32) return;
  float bal = 0.f, z = 0.f;
  int n = 0, used = 0, flags = 0;
  for (int q = threadIdx.x; q < a.S; q += 32) {
    const int4 w = __ldcg(reinterpret_cast<const int4 *>(a.pseq + q));
    bal += __int_as_float(w.x);
    z += __int_as_float(w.y);
    n += w.z;
    used += w.z > 0;
    flags |= w.w;
  }
  bal = warp_sum(bal);
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  used = __reduce_add_sync(0xffffffffu, used);
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (threadIdx.x == 0) finish_all(a, bal, z, n, used, flags);
}

// MANY: as many blocks as run at once, each going through several sequences.  A block
// adds up the tokens of all sequences, so with a block per sequence that is S^2 reads.
// Measured with a block per sequence and with this, one token each: 131072 sequences 3230
// and 957 us, 32768 322 and 249, 16384 130 and 131, 4096 31 and 36; of 16 tokens, 32768
// 401 and 420, 16384 170 and 210.  So from kManySequences on.  Without MANY the loop around
// the sequences is not there: with it 131072 x 250 in 32 sequences took 81 us instead of 59.
constexpr int kManySequences = 32768;
template <int W, int NV, bool ADD, bool MANY>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(const BalArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ int s_n[kWarps], s_used[kWarps];
  const int warp = threadIdx.x >> 5, l32 = threadIdx.x & 31;
  const int E = a.E, G = a.G, lane = l32 & (G - 1), sub = l32 / G, tpw = 32 / G;
  int seq = blockIdx.x / a.nbs;
  const int blk = blockIdx.x - seq * a.nbs;
  const int i0 = blk * a.per, i1 = min(i0 + a.per, a.L);
  const int step = kWarps * tpw, i_first = i0 + warp * tpw;
  float next[NV], old[NV], lse_next;
  size_t tbase = static_cast<size_t>(seq) * a.L;
  auto fetch = [&](int i) {  // the next token's logits, before this one is worked on
    load_row<W>(a.logits + (tbase + i) * E, E, G, lane, i < i1, -INFINITY, next);
    lse_next = i < i1 ? a.lse_in[tbase + i] : INFINITY;
  };
  fetch(i_first + sub);
  int ns = a.tokens[seq];
  int n = ns, used = ns > 0 ? 1 : 0;
  if (a.S > 1) {
    n = used = 0;
    for (int q = threadIdx.x; q < a.S; q += kThreads) {
      const int t = a.tokens[q];
      n += t;
      used += t > 0;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    used = __reduce_add_sync(0xffffffffu, used);
    if (l32 == 0) {
      s_n[warp] = n;
      s_used[warp] = used;
    }
    __syncthreads();
    n = used = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      n += s_n[w];
      used += s_used[w];
    }
  }
  const float cz = n > 0 ? 2.f * a.g_z / static_cast<float>(n) : 0.f;
  while (true) {
    const float inv = ns > 0 ? 1.f / static_cast<float>(ns) : 0.f;
    const float cb = used > 0 ? a.g_bal * static_cast<float>(E) / static_cast<float>(used) * inv : 0.f;
    float f[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = col_of<W>(j, lane, G);
      f[j] = e < E ? static_cast<float>(a.counts[static_cast<size_t>(seq) * E + e]) * inv / static_cast<float>(a.k) : 0.f;
    }
    for (int ib = i_first; ib < i1; ib += step) {
      const int i = ib + sub;
      float p[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) p[j] = next[j];
      const float lse = lse_next;
      float *row = a.d_logits + (tbase + i) * E;
      if (ADD) load_row<W>(row, E, G, lane, i < i1, 0.f, old);
      fetch(i + step);
      const bool some = lse != INFINITY;  // the token has a part in the losses
      // softmax from the row itself: lse only keeps the exponentials in range (they are at
      // most e^6, where its last place is as much as log E).  exp(v - lse) alone would carry
      // lse's rounding into p, 5e-4 of it at 1e4.  The sum rides along with the dot product.
      exp_row(p, lse);
      float dot = 0.f, sum = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        p[j] = some ? p[j] : 0.f;
        dot = fmaf(f[j], p[j], dot);
        sum += p[j];
      }
      dot = group_sum(dot, G);
      sum = group_sum(sum, G);
      const float r = some ? 1.f / sum : 0.f, cbr = cb * r, zt = some ? cz * lse * r : 0.f;
      dot *= r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float d = p[j] * fmaf(cbr, f[j] - dot, zt);
        p[j] = ADD ? old[j] + d : d;
      }
      if (i < i1 && (some || !ADD)) store_row<W>(row, E, G, lane, p);
    }
    if (!MANY) break;
    seq += gridDim.x;
    if (seq >= a.S) break;
    tbase = static_cast<size_t>(seq) * a.L;
    fetch(i_first + sub);
    ns = a.tokens[seq];
  }
}

bool bal_ok(const moe_balance_config *c) {
  return c && c->T >= 0 && c->T <= (1 << 30) && c->E >= 1 && c->E <= kMaxExperts && c->k >= 1 && c->k <= kMaxTopK &&
         c->k <= c->E && c->sequences >= 1 && c->T % c->sequences == 0;
}

// Values per lane and lanes per token.  Whole float4s: up to `most` values per
// lane, so that few lanes share a token and its sums take few shuffles; narrower
// vectors: 8, so that the lanes of a warp read whole lines.
int width_of(int E) { return E % 4 == 0 ? 4 : (E % 2 == 0 ? 2 : 1); }
int values_per_lane(int E, int most) {
  if (E % 4 != 0) most = 8;
  int nv = width_of(E);
  while (nv < most && nv * 32 < (E % 4 == 0 ? 32 * E : E)) nv *= 2;
  return nv;
}
int lanes_per_token(int E, int most) {
  const int nv = values_per_lane(E, most);
  int G = 1;
  while (G * nv < E) G *= 2;
  return G;
}
constexpr int kFwdValues = 16, kBwdValues = 8;  // (the backward's 16 took 110 registers: 12.5 against 9 us)

// Blocks per sequence (at most `most` over all of them, at least one each) and
// tokens per block, whole passes of its warps.
// A single sequence of up to kSoloPasses goes to one block, which needs no
// second kernel.
constexpr int kSoloPasses = 4;
void split(const moe_balance_config *c, int most, int G, bool solo, int *nbs, int *per) {
  const int L = c->T / c->sequences, pass = kWarps * (32 / G);
  int n = (L + pass - 1) / pass;
  if (solo && c->sequences == 1 && n <= kSoloPasses) n = 1;
  most = most / c->sequences > 1 ? most / c->sequences : 1;
  if (n > most) n = most;
  if (n < 1) n = 1;
  *per = ((L + n - 1) / n + pass - 1) / pass * pass;
  *nbs = L > 0 ? (L + *per - 1) / *per : 1;
}

struct BalLayout {
  size_t ticket, psum, pcnt, pblk, pseq, total;
};
BalLayout bal_layout(const moe_balance_config *c) {
  int nbs, per;
  split(c, kMaxBlocks, lanes_per_token(c->E, kFwdValues), true, &nbs, &per);
  const size_t rows = static_cast<size_t>(c->sequences) * nbs;
  BalLayout L;
  L.ticket = 64;  // inside the header
  L.psum = kHeader;
  L.pcnt = L.psum + align256(rows * c->E * 4);
  L.pblk = L.pcnt + align256(rows * c->E * 4);
  L.pseq = L.pblk + align256(rows * sizeof(SeqSum));
  L.total = L.pseq + align256(static_cast<size_t>(c->sequences) * sizeof(SeqSum));
  return L;
}

BalArgs bal_args(const moe_balance_config *c, int most, int values, bool solo) {
  BalArgs a{};
  a.T = c->T;
  a.E = c->E;
  a.k = c->k;
  a.S = c->sequences;
  a.L = c->T / c->sequences;
  a.G = lanes_per_token(c->E, values);
  split(c, most, a.G, solo, &a.nbs, &a.per);
  return a;
}

template <int W, int NV>
cudaError_t launch_fwd(const BalArgs &a, cudaStream_t s) {
  const bool solo = a.S * a.nbs == 1;
  return launch_pdl(solo ? balance_fwd_kernel<W, NV, true> : balance_fwd_kernel<W, NV, false>, dim3(a.S * a.nbs),
                    dim3(kThreads), 0, s, 1, a);
}
template <int W, int NV>
cudaError_t launch_bwd(const BalArgs &a, int most, bool add, cudaStream_t s) {
  const bool many = a.S >= kManySequences && a.S > most;  // then nbs is 1
  auto kernel = many ? (add ? balance_bwd_kernel<W, NV, true, true> : balance_bwd_kernel<W, NV, false, true>)
                     : (add ? balance_bwd_kernel<W, NV, true, false> : balance_bwd_kernel<W, NV, false, false>);
  return launch_pdl(kernel, dim3(many ? most : a.S * a.nbs), dim3(kThreads), 0, s, 1, a);
}
template <int MOST, class F>
cudaError_t by_width(int E, F &&f) {
  const int nv = values_per_lane(E, MOST);
  auto narrow = [&](auto w) {
    if (nv == 8) return f(w, std::integral_constant<int, 8>{});
    if (nv == 4) return f(w, std::integral_constant<int, 4>{});
    return f(w, std::integral_constant<int, 2>{});
  };
  if (E % 4 == 0) {
    if constexpr (MOST == 16)
      if (nv == 16) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 16>{});
    if (nv == 8) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
  }
  if (E % 2 == 0) return narrow(std::integral_constant<int, 2>{});
  if (nv == 1) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
  return narrow(std::integral_constant<int, 1>{});
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_balance_workspace(const moe_balance_config *cfg, size_t *fwd_scratch) {
  if (!bal_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (fwd_scratch) *fwd_scratch = bal_layout(cfg).total;
  return MOE_OK;
}

moe_status moe_balance_forward(const moe_balance_config *cfg, const float *logits, const int32_t *topk_idx,
                               const uint8_t *mask, float *loss, int32_t *counts, float *probs, int32_t *tokens,
                               float *lse, void *scratch, size_t scratch_bytes, void *stream) {
  if (!bal_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!loss || !counts || !probs || !tokens || !scratch || (cfg->T > 0 && (!logits || !topk_idx || !lse)))
    return MOE_ERR_INVALID_ARG;
  if (!al16(logits) || !al16(topk_idx) || !al16(mask) || !al16(loss) || !al16(counts) || !al16(probs) ||
      !al16(tokens) || !al16(lse) || !al16(scratch))
    return MOE_ERR_ALIGNMENT;
  const BalLayout L = bal_layout(cfg);
  if (scratch_bytes < L.total) return MOE_ERR_WORKSPACE;
  DevInfo di;
  MOE_TRY(device_info(&di));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t *sc = static_cast<uint8_t *>(scratch);
  BalArgs a = bal_args(cfg, kMaxBlocks, kFwdValues, true);
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.mask = mask;
  a.loss = loss;
  a.counts = counts;
  a.probs = probs;
  a.tokens = tokens;
  a.lse = lse;
  a.psum = reinterpret_cast<float *>(sc + L.psum);
  a.pcnt = reinterpret_cast<int32_t *>(sc + L.pcnt);
  a.pblk = reinterpret_cast<SeqSum *>(sc + L.pblk);
  a.pseq = reinterpret_cast<SeqSum *>(sc + L.pseq);
  a.ticket = reinterpret_cast<int32_t *>(sc + L.ticket);
  a.status = reinterpret_cast<int32_t *>(sc);
  // with no tokens the blocks find empty sequences and write zeros
  MOE_TRY(timed("balance_forward", s, [&] {
    return by_width<kFwdValues>(a.E, [&](auto w, auto nv) {
      return launch_fwd<decltype(w)::value, decltype(nv)::value>(a, s);
    });
  }));
  if (a.S * a.nbs == 1) return MOE_OK;
  return timed("balance_finish", s, [&] {
    const int groups = (a.E + kFinCols - 1) / kFinCols;
    return launch_pdl(balance_finish_kernel, dim3(a.S * groups), dim3(kFinThreads), 0, s, groups, a);
  });
}

moe_status moe_balance_backward(const moe_balance_config *cfg, const float *logits, const int32_t *counts,
                                const int32_t *tokens, const float *lse, float g_balance, float g_z,
                                float *d_logits, int32_t accumulate, void *stream) {
  if (!bal_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!counts || !tokens || (cfg->T > 0 && (!logits || !lse || !d_logits))) return MOE_ERR_INVALID_ARG;
  if (!al16(logits) || !al16(counts) || !al16(tokens) || !al16(lse) || !al16(d_logits)) return MOE_ERR_ALIGNMENT;
  DevInfo di;
  MOE_TRY(device_info(&di));
  if (cfg->T == 0) return MOE_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int most = di.sms * kBwdBlocksPerSm;
  BalArgs a = bal_args(cfg, most, kBwdValues, false);
  a.logits = logits;
  a.counts = const_cast<int32_t *>(counts);
  a.tokens = const_cast<int32_t *>(tokens);
  a.lse_in = lse;
  a.g_bal = g_balance;
  a.g_z = g_z;
  a.d_logits = d_logits;
  const bool add = accumulate != 0;
  return timed("balance_backward", s, [&] {
    return by_width<kBwdValues>(a.E, [&](auto w, auto nv) {
      return launch_bwd<decltype(w)::value, decltype(nv)::value>(a, most, add, s);
    });
  });
}

}  // extern "C"
