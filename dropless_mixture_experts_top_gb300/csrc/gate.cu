// gate.cu -- the gate around its choice (gate.cuh): the dispatch indices, the gradient for the
// logits, the step of the bias, and the C entry points.
//
// The dispatch indices take two kernels: the choice also leaves every slot's rank among
// its chunk's slots of the same expert (a chunk: the tokens of one block), the slots in
// front of the chunk in its cluster of blocks, and the cluster's totals; the second
// kernel adds up the totals in front of the cluster.  No block waits for one outside its cluster
// and nothing has to be zero before a call.  Few tokens are one cluster, which needs no
// second kernel.  Measured in graphs: 131072 x 256 in 8 groups 96 us (the choice 72 of them), 16384 x 128 with a
// bias 18.6, 512 x 8 5.7; backward 100000 x 250 dense 39.6, 16384 x 128 with the bias' step 4.9.
#include "gate.cuh"

namespace moe {
namespace {

constexpr int kBiasThreads = 1024;
constexpr int kMaxGroups = 32;

// A block per chunk, in the clusters of the first kernel: they share the adding of the totals.  The chunk's slots are put
// in the order of their rows in shared memory first, where they fit: an expert's are neighbours in the rows' arrays, and
// written one by one each would be a sector of its own (131072 x 8 slots: 116 us for the gate instead of 96).
constexpr int kSorted = 4096;
__global__ void __launch_bounds__(kGateThreads) gate_index_kernel(const GateArgs a, int clusters) {
  __shared__ int32_t s_sum[2][kMaxExperts];  // this block's part of the totals: the clusters in front, and all
  __shared__ int32_t s_base[kMaxExperts], s_first[kMaxExperts];  // an expert's first row, and place in the order, of the chunk
  __shared__ int s_w[2][kMaxExperts / 32];
  __shared__ int32_t q_slot[kSorted];
  __shared__ float q_w[kSorted];
  __shared__ uint8_t q_e[kSorted];
  const int tid = threadIdx.x, E = a.E;
  const int rank = blockIdx.x % a.cluster, mine = blockIdx.x / a.cluster;
  constexpr int kSlots = 4;
  const int64_t first = clusters ? static_cast<int64_t>(gate_first(a, blockIdx.x)) * a.k : 0,
                last = clusters ? static_cast<int64_t>(gate_first(a, blockIdx.x + 1)) * a.k : 0;
  asm volatile("" ::"l"(first), "l"(last), "r"(rank), "r"(mine));  // before the wait
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  // the block's first slots, on their way during what follows
  int slot_e[kSlots], slot_r[kSlots];
  float slot_w[kSlots];
  auto load = [&](int64_t s0) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int64_t s = s0 + i * kGateThreads;
      if (s < last) {
        slot_e[i] = __ldcg(a.topk_idx + s);
        slot_r[i] = __ldcg(a.row_of_slot + s);
        slot_w[i] = __ldcg(a.topk_w + s);
      }
    }
  };
  load(first + tid);
  int before = 0, all = 0, n, slots;
  const bool some = tid < E && clusters;
  const int here = some ? __ldcg(a.before + static_cast<size_t>(blockIdx.x) * E + tid) : 0;
  const int own = some ? __ldcg(a.count + static_cast<size_t>(blockIdx.x) * E + tid) : 0;
  if (tid < E) {
    constexpr int kBatch = 10;  // 76 clusters over 8 blocks
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
  const int off = expert_prefix(all, s_w[0], &n);  // (threads past the experts: zeros)
  s_base[tid] = off + before + here;
  s_first[tid] = expert_prefix(own, s_w[1], &slots);
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
  const bool sorted = slots <= kSorted;
  for (int64_t s0 = first + tid; s0 < last; s0 += kGateThreads * kSlots) {
    if (s0 > first + tid) load(s0);
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int64_t s = s0 + i * kGateThreads;
      if (s < last) {
        const int e = slot_e[i], row = s_base[e] + slot_r[i], at = s_first[e] + slot_r[i];
        a.row_of_slot[s] = row;
        if (sorted) {
          q_slot[at] = static_cast<int32_t>(s);
          q_w[at] = slot_w[i];
          q_e[at] = static_cast<uint8_t>(e);
        } else {
          a.slot_of_row[row] = static_cast<int32_t>(s);
          a.w_row[row] = slot_w[i];
        }
      }
    }
  }
  if (sorted) {
    __syncthreads();
    for (int at = tid; at < slots; at += kGateThreads) {
      const int e = q_e[at], row = s_base[e] + at - s_first[e];
      a.slot_of_row[row] = q_slot[at];
      a.w_row[row] = q_w[at];
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
// A slot of weight zero has none.  Bound by the gradient's bytes (and the dense kind's logits).  A warp has a
// token: it writes the row without the chosen experts, then their elements over it, in lanes that hold a slot each;
// the next token's inputs are on their way meanwhile.

constexpr int kGradThreads = 256;
constexpr int kGradBlocks = 6, kDenseBlocks = 4;  // per SM

struct GradArgs {
  const float *logits;
  const int32_t *topk_idx;
  const float *topk_w, *d_topk_w;
  float *d_logits;
  int T, E, k;
  bool sigmoid, renormalise;
  float scale;
};

// VW: elements per access, by the rows' alignment.
template <int VW>
__device__ __forceinline__ void load_vec(const float *p, float *v) {
  if constexpr (VW == 4) {
    const float4 q = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else if constexpr (VW == 2) {
    const float2 q = __ldg(reinterpret_cast<const float2 *>(p));
    v[0] = q.x, v[1] = q.y;
  } else {
    v[0] = __ldg(p);
  }
}
template <int VW>
__device__ __forceinline__ void store_vec(float *p, const float *v, float f) {
  if constexpr (VW == 4)
    *reinterpret_cast<float4 *>(p) = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
  else if constexpr (VW == 2)
    *reinterpret_cast<float2 *>(p) = make_float2(v[0] * f, v[1] * f);
  else
    *p = v[0] * f;
}

template <bool DENSE, int VW>
__global__ void __launch_bounds__(kGradThreads, DENSE ? kDenseBlocks : kGradBlocks) gate_grad_kernel(const GradArgs a) {
  constexpr int NV = kMaxExperts / 32;
  const int lane = threadIdx.x & 31, E = a.E, k = a.k;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kGradThreads / 32);
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  // a slot's expert (-1: none), weight and gradient, its logit, and the dense kind's row
  struct Slot {
    int e;
    float w, g;
  };
  auto slot_of = [&](int64_t t) {
    Slot s{-1, 0.f, 0.f};
    if (t < a.T && lane < k) {
      s.e = __ldg(a.topk_idx + t * k + lane);
      s.w = __ldg(a.topk_w + t * k + lane);
      s.g = __ldg(a.d_topk_w + t * k + lane);
      if (s.e < 0 || s.e >= E || s.w == 0.f) s.e = -1;
    }
    return s;
  };
  auto row_of = [&](int64_t t, float (&v)[NV]) {
    const float *lr = a.logits + t * E;
#pragma unroll
    for (int i = 0; i < NV; i += VW) {
      const int c = VW * lane + 32 * i;
#pragma unroll
      for (int q = 0; q < VW; ++q) v[i + q] = -INFINITY;
      if (t < a.T && c < E) load_vec<VW>(lr + c, v + i);
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * (kGradThreads / 32) + (threadIdx.x >> 5);
  Slot next = slot_of(t);
  float ahead[DENSE ? NV : 1];
  if constexpr (DENSE) row_of(t, ahead);
  for (; t < a.T; t += step) {
    const Slot s = next;
    float *out = a.d_logits + t * E;
    bool bad = false;
    float l = s.e >= 0 ? clean_logit(__ldg(a.logits + t * E + s.e), bad) : 0.f;
    float d;
    if constexpr (DENSE) {
      float v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = clean_logit(ahead[i], bad);
      next = slot_of(t + step);
      row_of(t + step, ahead);
      float top = -FLT_MAX, z = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) top = fmaxf(top, v[i]);
      top = warp_max(top);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = __expf(v[i] - top);
        z += v[i];
      }
      z = warp_sum(z);
      const float own = s.e >= 0 ? s.w * s.g : 0.f;
      const float f = z > 0.f ? -warp_sum(own) / z : 0.f;  // (z is the same in all lanes)
#pragma unroll
      for (int i = 0; i < NV; i += VW)
        if (VW * lane + 32 * i < E) store_vec<VW>(out + VW * lane + 32 * i, v + i, f);
      d = fmaf(__expf(l - top), f, own);
    } else {
      const float zero[VW] = {};
#pragma unroll
      for (int i = 0; i < NV; i += VW)
        if (VW * lane + 32 * i < E) store_vec<VW>(out + VW * lane + 32 * i, zero, 0.f);
      next = slot_of(t + step);
      float dot = 0.f;
      if (a.renormalise) {
        dot = s.e >= 0 ? s.w / a.scale * s.g : 0.f;
#pragma unroll
        for (int o = kMaxTopK / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      d = s.w * (s.g - dot);
      if (a.sigmoid) d *= 1.f / (1.f + expf(l));  // 1 - s
    }
    __syncwarp();  // the row's other writes come first
    if (s.e >= 0) out[s.e] = d;
  }
}

// bias_e += rate * sign(mean load - load of e), the counts of all rows added up; compared as
// whole numbers: sum_e' c_e' against E c_e.
// Threads: the experts, times the parts of the rows.
__global__ void __launch_bounds__(kBiasThreads) gate_bias_kernel(const int32_t *counts, int rows, int E, float rate,
                                                                 float *bias) {
  __shared__ long long s_load[kBiasThreads], s_all[kMaxExperts / 32];
  const int e = threadIdx.x % kMaxExperts, part = threadIdx.x / kMaxExperts, parts = blockDim.x / kMaxExperts;
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  long long c = 0;
  if (e < E)
    for (int r = part; r < rows; r += parts) c += __ldg(counts + static_cast<size_t>(r) * E + e);
  const float was = e < E ? bias[e] : 0.f;
  s_load[threadIdx.x] = c;
  __syncthreads();
  if (part > 0) return;
  for (int p = 1; p < parts; ++p) c += s_load[p * kMaxExperts + e];
  long long all = c;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if ((e & 31) == 0) s_all[e >> 5] = all;
  asm volatile("bar.sync 1, 256;" ::: "memory");  // (the first kMaxExperts threads)
  all = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 32; ++w) all += s_all[w];
  if (e >= E) return;
  const long long d = all - c * E;
  if (d != 0) bias[e] = was + (d > 0 ? rate : -rate);
}
static_assert(kMaxExperts == 256, "the barrier's threads");

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

// Chunks: one cluster of blocks up to 512 tokens, which needs no second kernel; then 16 tokens each up to two blocks for each
// of 152 SMs (4096 x 128, the choice alone, in 128, 256 and 512 chunks: 9.2, 7.3 and 9.7 us), 32 each up to four
// (16384 x 128 in 304, 512 and 608: 18, 14 and 17 us), then more each (131072 x 256 in 608, 912 and 1216: 89, 98 and 105).
constexpr int kOneCluster = 512, kTwoBlocks = 304, kFourBlocks = 608;
struct GateLayout {
  int chunks, cluster;
  size_t flags, before, count, total, bytes;
};
GateLayout gate_layout(const moe_gate_config *c) {
  GateLayout L;
  auto parts = [&](int tokens) { return (c->T + tokens - 1) / tokens; };
  if (c->T <= kOneCluster)
    L.chunks = parts(32) < kGateCluster ? parts(32) : kGateCluster;
  else if (parts(32) >= kTwoBlocks)
    L.chunks = parts(32) < kFourBlocks ? parts(32) : kFourBlocks;
  else
    L.chunks = parts(16) < kTwoBlocks ? parts(16) : kTwoBlocks;
  L.cluster = L.chunks < kGateCluster ? (L.chunks < 1 ? 1 : L.chunks) : kGateCluster;
  const size_t clusters = static_cast<size_t>(L.chunks + L.cluster - 1) / L.cluster;
  L.flags = kHeader;
  L.before = L.flags + align256(clusters * 4 + 4);
  L.count = L.before + align256(clusters * L.cluster * c->E * 4 + 4);
  L.total = L.count + align256(clusters * L.cluster * c->E * 4 + 4);
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
  if (L.chunks) a.chunk_tokens = cfg->T / L.chunks, a.longer = cfg->T % L.chunks;
  a.cluster = L.cluster;
  a.before = reinterpret_cast<int32_t *>(sc + L.before);
  a.count = reinterpret_cast<int32_t *>(sc + L.count);
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
  const bool dense = !a.sigmoid && !a.renormalise, two = a.E % 2 == 0, four = a.E % 4 == 0;
  const int64_t wanted = (static_cast<int64_t>(a.T) + kGradThreads / 32 - 1) / (kGradThreads / 32);
  const int most = (dense ? kDenseBlocks : kGradBlocks) * di.sms, blocks = static_cast<int>(wanted < most ? wanted : most);
  return timed("gate_backward", s, [&] {
    auto go = [&](auto kernel) { return launch_pdl(kernel, dim3(blocks), dim3(kGradThreads), 0, s, 1, a); };
    if (dense) return four ? go(gate_grad_kernel<true, 4>) : two ? go(gate_grad_kernel<true, 2>) : go(gate_grad_kernel<true, 1>);
    return four ? go(gate_grad_kernel<false, 4>) : two ? go(gate_grad_kernel<false, 2>) : go(gate_grad_kernel<false, 1>);
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
    return launch_pdl(gate_bias_kernel, dim3(1), dim3(rows < 4 ? kMaxExperts : kBiasThreads), 0, s, 1, counts, static_cast<int>(rows),
                      static_cast<int>(cfg->E), rate, bias);
  });
}

}  // extern "C"
