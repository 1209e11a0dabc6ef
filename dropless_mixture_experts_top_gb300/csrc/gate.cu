// gate.cu -- the gate around its choice (gate.cuh): the dispatch indices, the gradient for the
// logits, the step of the bias, and the C entry points.
//
// The dispatch indices take two kernels: the choice also leaves every slot's rank among
// its chunk's slots of the same expert (a chunk: the tokens of one block), the slots in
// front of the chunk in its cluster of blocks, and the cluster's totals; the second
// kernel adds up the totals in front of the cluster.  No block waits for one outside its cluster
// and nothing has to be zero before a call.  Few tokens are one cluster, which needs no
// second kernel.
#include "gate.cuh"

namespace moe {
namespace {

constexpr int kBiasThreads = 1024;
constexpr int kMaxGroups = 32;

// A block per chunk, in the clusters of the first kernel: they share the adding of the totals.
__global__ void __launch_bounds__(kGateThreads) gate_index_kernel(const GateArgs a, int clusters) {
  __shared__ int32_t s_sum[2][kMaxExperts];  // this block's part of the totals: the clusters in front, and all
  __shared__ int32_t s_base[kMaxExperts];
  __shared__ int s_w[kMaxExperts / 32];
  const int tid = threadIdx.x, E = a.E;
  const int rank = blockIdx.x % a.cluster, mine = blockIdx.x / a.cluster;
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  int before = 0, all = 0, n;
  const int here = tid < E && clusters ? __ldcg(a.before + static_cast<size_t>(blockIdx.x) * E + tid) : 0;
  if (tid < E) {
    constexpr int kBatch = 8;  // 57 clusters over 8 blocks
    for (int c = rank; c < clusters; c += a.cluster * kBatch) {
      int h[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int cc = c + i * a.cluster;
        h[i] = cc < clusters ? __ldcg(a.total + static_cast<size_t>(cc) * E + tid) : 0;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        before += c + i * a.cluster < mine ? h[i] : 0;
        all += h[i];
      }
    }
  }
  s_sum[0][tid] = before;
  s_sum[1][tid] = all;
  if (a.cluster > 1)
    cluster_sync();
  else
    __syncthreads();
  if (a.cluster > 1) {
    before = all = 0;
    for (int c = 0; c < a.cluster; ++c) {
      before += ld_peer(&s_sum[0][tid], c);
      all += ld_peer(&s_sum[1][tid], c);
    }
    cluster_arrive();  // (the others may leave after this block has read)
  }
  const int off = expert_prefix(all, s_w, &n);  // (threads past the experts: zeros)
  s_base[tid] = off + before + here;
  if (blockIdx.x == 0) {
    if (tid < E) {
      a.counts[tid] = all;
      a.offsets[tid] = off;
    }
    int f = 0;
    for (int c = tid; c < clusters; c += kGateThreads) f |= a.flags[c];
    f = __syncthreads_or(f);
    if (tid == 0) {
      a.offsets[E] = n;
      *a.status = f;
    }
  }
  __syncthreads();
  if (clusters) {
    const int64_t s1 = static_cast<int64_t>(gate_first(a, blockIdx.x + 1)) * a.k;
    constexpr int kBatch = 4;
    for (int64_t s0 = static_cast<int64_t>(gate_first(a, blockIdx.x)) * a.k + tid; s0 < s1; s0 += kGateThreads * kBatch) {
      int e[kBatch], r[kBatch];
      float w[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t s = s0 + i * kGateThreads;
        if (s < s1) {
          e[i] = __ldcg(a.topk_idx + s);
          r[i] = __ldcg(a.row_of_slot + s);
          w[i] = __ldcg(a.topk_w + s);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t s = s0 + i * kGateThreads;
        if (s < s1) {
          const int row = s_base[e[i]] + r[i];
          a.row_of_slot[s] = row;
          a.slot_of_row[row] = static_cast<int32_t>(s);
          a.w_row[row] = w[i];
        }
      }
    }
  }
  if (a.cluster > 1) cluster_wait();
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
__global__ void __launch_bounds__(kBiasThreads) gate_bias_kernel(const int32_t *counts, int rows, int E, float rate,
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
    for (int r = part; r < rows; r += (kBiasThreads / kMaxExperts)) c += __ldg(counts + static_cast<size_t>(r) * E + e);
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

// Chunks: 32 tokens each while that makes at most three blocks for each of 152 SMs, then more each; up to
// 64 tokens for each of one cluster's blocks are one launch.
constexpr int kLeastTok = 32, kMostChunks = 456;
struct GateLayout {
  int chunks, cluster;
  size_t flags, before, total, bytes;
};
GateLayout gate_layout(const moe_gate_config *c) {
  GateLayout L;
  const int parts = (c->T + kLeastTok - 1) / kLeastTok, most = parts <= 2 * kGateCluster ? kGateCluster : kMostChunks;
  L.chunks = parts < most ? parts : most;
  L.cluster = L.chunks < kGateCluster ? (L.chunks < 1 ? 1 : L.chunks) : kGateCluster;
  const size_t clusters = static_cast<size_t>(L.chunks + L.cluster - 1) / L.cluster;
  L.flags = kHeader;
  L.before = L.flags + align256(clusters * 4 + 4);
  L.total = L.before + align256(clusters * L.cluster * c->E * 4 + 4);
  L.bytes = L.total + align256(clusters * c->E * 4 + 4);
  return L;
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
  if (fwd_scratch) *fwd_scratch = gate_layout(cfg).bytes;
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
  if (scratch_bytes < L.bytes) return MOE_ERR_WORKSPACE;
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
  a.chunks = L.chunks;
  a.cluster = L.cluster;
  a.before = reinterpret_cast<int32_t *>(sc + L.before);
  a.total = reinterpret_cast<int32_t *>(sc + L.total);
  a.flags = reinterpret_cast<int32_t *>(sc + L.flags);
  a.status = reinterpret_cast<int32_t *>(sc);
  if (a.T > 0) {
    // the logits' own order, unless a bias or a sum of two scores enters
    const bool by_logit = !bias && (a.groups == 1 || a.group_best == 1);
    MOE_TRY(timed("gate_select", s, [&] {
      if (by_logit) return launch_gate_select<kKeyLogit>(a, s);
      return a.sigmoid ? launch_gate_select<kKeySigmoid>(a, s) : launch_gate_select<kKeySoftmax>(a, s);
    }));
    if (a.chunks <= a.cluster) return MOE_OK;
  }
  return timed("gate_index", s, [&] {
    const int clusters = (a.chunks + a.cluster - 1) / a.cluster;  // (no tokens: one block writes zeros)
    return launch_pdl(gate_index_kernel, dim3(clusters ? clusters * a.cluster : 1), dim3(kGateThreads), 0, s, a.cluster, a,
                      clusters);
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
    return launch_pdl(gate_bias_kernel, dim3(1), dim3(kBiasThreads), 0, s, 1, counts, static_cast<int>(rows),
                      static_cast<int>(cfg->E), rate, bias);
  });
}

}  // extern "C"
