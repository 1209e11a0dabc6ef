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
// token holding its row in registers.  The forward's blocks stay inside one
// sequence and leave their column sums, counts and z sums as one partial row
// each; a second kernel (one block per sequence, the last to finish adds the
// sequences) reduces them in a fixed order, so losses are the same bits every
// time.  Counts are integers, added in any order.
#include <math.h>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 304;  // forward blocks over all sequences at most, unless there are more sequences
constexpr int kUnroll = 4;       // tokens whose loads a lane group has in flight

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

// A lane's columns: four consecutive ones (VEC, E % 4 == 0) or one, G apart.
template <bool VEC>
__device__ __forceinline__ int col_of(int j, int lane, int G) {
  return VEC ? ((j >> 2) * G + lane) * 4 + (j & 3) : j * G + lane;
}

template <bool VEC, int NV>
__device__ __forceinline__ void load_row(const float *row, int E, int G, int lane, bool in, float fill,
                                         float (&v)[NV]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      const int c = (j * G + lane) * 4;
      const float4 q = in && c < E ? *reinterpret_cast<const float4 *>(row + c) : make_float4(fill, fill, fill, fill);
      v[4 * j] = q.x;
      v[4 * j + 1] = q.y;
      v[4 * j + 2] = q.z;
      v[4 * j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = j * G + lane;
      v[j] = in && c < E ? row[c] : fill;
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

template <bool VEC, int NV>
__global__ void __launch_bounds__(kThreads) balance_fwd_kernel(const BalArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ int s_cnt[kMaxExperts];
  __shared__ float s_col[kWarps][kMaxExperts];
  __shared__ SeqSum s_blk[kWarps];
  const int warp = threadIdx.x >> 5, l32 = threadIdx.x & 31;
  const int E = a.E, G = a.G, lane = l32 & (G - 1), sub = l32 / G, tpw = 32 / G;
  const int seq = blockIdx.x / a.nbs, blk = blockIdx.x - seq * a.nbs;
  const int i0 = blk * a.per, i1 = min(i0 + a.per, a.L);  // tokens of the sequence
  const size_t tbase = static_cast<size_t>(seq) * a.L;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  for (int e = threadIdx.x; e < E; e += kThreads) s_cnt[e] = 0;
  __syncthreads();
  float col[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) col[j] = 0.f;
  float z = 0.f;
  int n = 0, flags = 0;
  const int step = kWarps * tpw;  // tokens of one pass of the block
  for (int ib = i0 + warp * tpw; ib < i1; ib += step * kUnroll) {
    float v[kUnroll][NV];
    bool ok[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = ib + u * step + sub;
      const bool in = i < i1;
      load_row<VEC>(a.logits + (tbase + i) * E, E, G, lane, in, -INFINITY, v[u]);
      ok[u] = in && (!a.mask || a.mask[tbase + i] != 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = ib + u * step + sub;
      float mx = -INFINITY, bad = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        mx = fmaxf(mx, v[u][j]);
        if (v[u][j] != v[u][j] || v[u][j] == INFINITY) bad = 1.f;
      }
      mx = group_max(mx, G);
      bad = group_max(bad, G);
      if (bad == 0.f && mx == -INFINITY) ok[u] = false;  // no finite logit
      float sum = 0.f, ex[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        ex[j] = ok[u] ? expf(v[u][j] - mx) : 0.f;
        sum += ex[j];
      }
      sum = group_sum(sum, G);
      const float lse = bad != 0.f ? NAN : mx + logf(sum);
      if (ok[u]) {
        const float inv = bad != 0.f ? NAN : 1.f / sum;
#pragma unroll
        for (int j = 0; j < NV; ++j) col[j] = fmaf(ex[j], inv, col[j]);
        if (lane == 0) {
          z = fmaf(lse, lse, z);
          n += 1;
          if (bad != 0.f) flags |= kDevNonfiniteLogit;
        }
        for (int q = lane; q < a.k; q += G) {
          const int e = a.topk_idx[(tbase + i) * a.k + q];
          if (static_cast<unsigned>(e) < static_cast<unsigned>(E))
            atomicAdd(&s_cnt[e], 1);
          else
            flags |= kDevBadIndex;
        }
      }
      if (lane == 0 && i < i1) a.lse[tbase + i] = ok[u] ? lse : INFINITY;
    }
  }
  // the warp's token groups, then the block's warps, in a fixed order
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float c = col[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o >= G) c += __shfl_xor_sync(0xffffffffu, c, o);
    const int e = col_of<VEC>(j, lane, G);
    if (sub == 0 && e < E) s_col[warp][e] = c;
  }
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (l32 == 0) s_blk[warp] = SeqSum{0.f, z, n, flags};
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float c = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) c += s_col[w][e];
    a.psum[static_cast<size_t>(blockIdx.x) * E + e] = c;
    a.pcnt[static_cast<size_t>(blockIdx.x) * E + e] = s_cnt[e];
  }
  if (threadIdx.x == 0) {
    SeqSum r = s_blk[0];
    for (int w = 1; w < kWarps; ++w) {
      r.z += s_blk[w].z;
      r.n += s_blk[w].n;
      r.flags |= s_blk[w].flags;
    }
    a.pblk[blockIdx.x] = r;
  }
}

// One block per sequence; the last one to finish adds the sequences.
constexpr int kFinThreads = 1024;
__global__ void __launch_bounds__(kFinThreads) balance_finish_kernel(const BalArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s_sum[kFinThreads];
  __shared__ int s_cnt[kFinThreads];
  __shared__ SeqSum s_seq;
  __shared__ float s_w[8];
  __shared__ int s_last;
  const int E = a.E, s = blockIdx.x;
  int ep = 32;
  while (ep < E) ep *= 2;
  const int e = threadIdx.x & (ep - 1), run = threadIdx.x / ep, runs = kFinThreads / ep;
  const size_t row0 = static_cast<size_t>(s) * a.nbs;
  float sum = 0.f;
  int cnt = 0;
  constexpr int U = 16;  // loads of each kind in flight
  for (int b0 = run; b0 < a.nbs; b0 += runs * U) {
    float v[U];
    int c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + runs * u;
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
  s_sum[threadIdx.x] = sum;
  s_cnt[threadIdx.x] = cnt;
  if (threadIdx.x < 32) {
    SeqSum r{0.f, 0.f, 0, 0};
    for (int b = threadIdx.x; b < a.nbs; b += 32) {
      const SeqSum q = a.pblk[row0 + b];
      r.z += q.z;
      r.n += q.n;
      r.flags |= q.flags;
    }
    r.z = warp_sum(r.z);
    r.n = __reduce_add_sync(0xffffffffu, r.n);
    r.flags = __reduce_or_sync(0xffffffffu, r.flags);
    if (threadIdx.x == 0) s_seq = r;
  }
  __syncthreads();
  const float inv_n = s_seq.n > 0 ? 1.f / static_cast<float>(s_seq.n) : 0.f;
  if (threadIdx.x < 256) {  // E <= 256
    float fp = 0.f;
    if (threadIdx.x < E) {
      for (int r = 1; r < runs; ++r) {
        sum += s_sum[r * ep + threadIdx.x];
        cnt += s_cnt[r * ep + threadIdx.x];
      }
      const float P = sum * inv_n;
      a.counts[static_cast<size_t>(s) * E + e] = cnt;
      a.probs[static_cast<size_t>(s) * E + e] = P;
      fp = static_cast<float>(cnt) * P;
    }
    fp = warp_sum(fp);
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = fp;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float b = 0.f;
    for (int w = 0; w < 8; ++w) b += s_w[w];
    SeqSum r = s_seq;
    r.bal = b * static_cast<float>(E) / static_cast<float>(a.k) * inv_n;
    a.tokens[s] = r.n;
    a.pseq[s] = r;
    __threadfence();
    s_last = atomicAdd(a.ticket, 1) == a.S - 1;
    if (s_last) __threadfence();
  }
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
  if (threadIdx.x == 0) {
    a.loss[0] = used > 0 ? bal / static_cast<float>(used) : 0.f;
    a.loss[1] = n > 0 ? z / static_cast<float>(n) : 0.f;
    *a.status = flags;
  }
}

template <bool VEC, int NV, bool ADD>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(const BalArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ int s_n[kWarps], s_used[kWarps];
  const int warp = threadIdx.x >> 5, l32 = threadIdx.x & 31;
  const int E = a.E, G = a.G, lane = l32 & (G - 1), sub = l32 / G, tpw = 32 / G;
  const int seq = blockIdx.x / a.nbs, blk = blockIdx.x - seq * a.nbs;
  const int i0 = blk * a.per, i1 = min(i0 + a.per, a.L);
  const size_t tbase = static_cast<size_t>(seq) * a.L;
  int n = 0, used = 0;
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
  const int ns = a.tokens[seq];
  const float inv = ns > 0 ? 1.f / static_cast<float>(ns) : 0.f;
  const float cb = used > 0 ? a.g_bal * static_cast<float>(E) / static_cast<float>(used) * inv : 0.f;
  const float cz = n > 0 ? 2.f * a.g_z / static_cast<float>(n) : 0.f;
  float f[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = col_of<VEC>(j, lane, G);
    f[j] = e < E ? static_cast<float>(a.counts[static_cast<size_t>(seq) * E + e]) * inv / static_cast<float>(a.k) : 0.f;
  }
  const int step = kWarps * tpw;
  constexpr int U = kUnroll / 2;
  for (int ib = i0 + warp * tpw; ib < i1; ib += step * U) {
    float v[U][NV], old[U][NV], lse[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = ib + u * step + sub;
      const bool in = i < i1;
      load_row<VEC>(a.logits + (tbase + i) * E, E, G, lane, in, -INFINITY, v[u]);
      if (ADD) load_row<VEC>(a.d_logits + (tbase + i) * E, E, G, lane, in, 0.f, old[u]);
      lse[u] = in ? a.lse_in[tbase + i] : INFINITY;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = ib + u * step + sub;
      const bool some = lse[u] != INFINITY;  // the token has a part in the losses
      float p[NV], dot = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        p[j] = some ? expf(v[u][j] - lse[u]) : 0.f;
        dot = fmaf(f[j], p[j], dot);
      }
      dot = group_sum(dot, G);
      const float zt = some ? cz * lse[u] : 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float d = p[j] * fmaf(cb, f[j] - dot, zt);
        p[j] = ADD ? old[u][j] + d : d;
      }
      if (i < i1 && (some || !ADD)) {
        float *row = a.d_logits + (tbase + i) * E;
        if constexpr (VEC) {
#pragma unroll
          for (int j = 0; j < NV / 4; ++j) {
            const int c = (j * G + lane) * 4;
            if (c < E)
              *reinterpret_cast<float4 *>(row + c) = make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (j * G + lane < E) row[j * G + lane] = p[j];
        }
      }
    }
  }
}

bool bal_ok(const moe_balance_config *c) {
  return c && c->T >= 0 && c->T <= (1 << 30) && c->E >= 1 && c->E <= kMaxExperts && c->k >= 1 && c->k <= kMaxTopK &&
         c->k <= c->E && c->sequences >= 1 && c->T % c->sequences == 0;
}

int lanes_per_token(int E) {
  const int units = E % 4 == 0 ? E / 4 : E;
  int G = 1;
  while (G < units && G < 32) G *= 2;
  return G;
}

// Blocks per sequence and tokens per block: enough blocks to fill the part, but
// none with less than two passes of its warps.
void split(const moe_balance_config *c, int *nbs, int *per) {
  const int L = c->T / c->sequences, pass = kWarps * (32 / lanes_per_token(c->E));
  int n = (L + 2 * pass - 1) / (2 * pass);
  const int most = kMaxBlocks / c->sequences > 1 ? kMaxBlocks / c->sequences : 1;
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
  split(c, &nbs, &per);
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

BalArgs bal_args(const moe_balance_config *c) {
  BalArgs a{};
  a.T = c->T;
  a.E = c->E;
  a.k = c->k;
  a.S = c->sequences;
  a.L = c->T / c->sequences;
  a.G = lanes_per_token(c->E);
  split(c, &a.nbs, &a.per);
  return a;
}

template <bool VEC, int NV>
cudaError_t launch_fwd(const BalArgs &a, cudaStream_t s) {
  return launch_pdl(balance_fwd_kernel<VEC, NV>, dim3(a.S * a.nbs), dim3(kThreads), 0, s, 1, a);
}
template <bool VEC, int NV>
cudaError_t launch_bwd(const BalArgs &a, bool add, cudaStream_t s) {
  return launch_pdl(add ? balance_bwd_kernel<VEC, NV, true> : balance_bwd_kernel<VEC, NV, false>, dim3(a.S * a.nbs),
                    dim3(kThreads), 0, s, 1, a);
}
// Values per lane: float4s where rows are whole ones, else single columns.
template <class Vec4, class Vec8, class S1, class S2, class S4, class S8>
cudaError_t by_width(int E, Vec4 &&v4, Vec8 &&v8, S1 &&s1, S2 &&s2, S4 &&s4, S8 &&s8) {
  if (E % 4 == 0) return E <= 128 ? v4() : v8();
  return E <= 32 ? s1() : E <= 64 ? s2() : E <= 128 ? s4() : s8();
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
  BalArgs a = bal_args(cfg);
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
    return by_width(
        a.E, [&] { return launch_fwd<true, 4>(a, s); }, [&] { return launch_fwd<true, 8>(a, s); },
        [&] { return launch_fwd<false, 1>(a, s); }, [&] { return launch_fwd<false, 2>(a, s); },
        [&] { return launch_fwd<false, 4>(a, s); }, [&] { return launch_fwd<false, 8>(a, s); });
  }));
  return timed("balance_finish", s, [&] {
    return launch_pdl(balance_finish_kernel, dim3(a.S), dim3(kFinThreads), 0, s, 1, a);
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
  BalArgs a = bal_args(cfg);
  a.logits = logits;
  a.counts = const_cast<int32_t *>(counts);
  a.tokens = const_cast<int32_t *>(tokens);
  a.lse_in = lse;
  a.g_bal = g_balance;
  a.g_z = g_z;
  a.d_logits = d_logits;
  const bool add = accumulate != 0;
  return timed("balance_backward", s, [&] {
    return by_width(
        a.E, [&] { return launch_bwd<true, 4>(a, add, s); }, [&] { return launch_bwd<true, 8>(a, add, s); },
        [&] { return launch_bwd<false, 1>(a, add, s); }, [&] { return launch_bwd<false, 2>(a, add, s); },
        [&] { return launch_bwd<false, 4>(a, add, s); }, [&] { return launch_bwd<false, 8>(a, add, s); });
  });
}

}  // extern "C"
