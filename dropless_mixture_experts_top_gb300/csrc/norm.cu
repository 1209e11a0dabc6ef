// norm.cu -- layer norm and RMS norm, forward and backward, with the residual
// sum in front of the norm and the reduction of the weight's gradient.
//
// Forward, row t of H elements:  h = x (+ residual, rounded to the type and
// written), mu = mean h (RMS: 0), r = 1 / sqrt(mean (h - mu)^2 + eps),
// y = (h - mu) r w + b.  The row stays in registers between its two sums, so
// the variance is that of the centred values and memory is read once.
// Backward, with xh = (h - mu) r and g = dy w:
//   dx = r (g - mean g - xh mean(g xh)) (+ d_sum)      (RMS: no mean g)
//   dw = sum_t dy xh,  db = sum_t dy
// Both are bound by memory: every input is read and every output written once.
//
// Layout: a row is shared by TPR threads (a power of two, 8 to 512), each
// holding kElems elements in V vectors that lie TPR vectors apart, so a warp's
// accesses are contiguous.  Blocks are persistent over rows: a thread's columns
// stay the same, so the weight (and in the backward the column sums of dy xh
// and dy) stay in its registers, while asynchronous copies bring the coming rows
// into a ring in shared memory.  The backward's blocks leave one partial row of
// column sums each, which a second kernel adds in a fixed order: no atomics, the
// same bits every time.
#include <type_traits>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxH = 8192;
constexpr int kElems = 16;         // elements of a row per thread
constexpr int kThreads = 256;      // threads per block (a wider row takes one block of its own)
constexpr int kBwdBlocks = 304;    // the backward's partial rows at most: two blocks on each of 152 SMs

struct NormArgs {
  const void *x, *res, *w, *b;  // forward input (backward: h), residual or d_sum, weight, bias
  const void *dy;
  void *y, *sum;                // forward: y, h; backward: dx, -
  float2 *stats;                // [T] mu, r
  float *part;                  // backward: [blocks][2][H] column sums of dy xh and dy
  float eps;
  int T, H, tpr;
  bool layer;
};

// Vectors of VB bytes holding elements of type El (uint16_t: bf16 bits).
template <int VB> struct RawOf;
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<2> { using type = uint16_t; };

template <class El, int VB>
struct Vec {
  using Raw = typename RawOf<VB>::type;
  static constexpr int N = VB / static_cast<int>(sizeof(El));
  static __device__ __forceinline__ Raw zero() {
    Raw r;
    memset(&r, 0, sizeof(r));
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw &r, float *f) {
    if constexpr (sizeof(El) == 4) {
      memcpy(f, &r, VB);
    } else if constexpr (VB == 2) {
      f[0] = __uint_as_float(static_cast<uint32_t>(r) << 16);
    } else {
      uint32_t w[VB / 4];
      memcpy(w, &r, VB);
#pragma unroll
      for (int i = 0; i < VB / 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
  static __device__ __forceinline__ Raw pack(const float *f) {
    Raw r;
    if constexpr (sizeof(El) == 4) {
      memcpy(&r, f, VB);
    } else if constexpr (VB == 2) {
      r = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
      uint32_t w[VB / 4];
#pragma unroll
      for (int i = 0; i < VB / 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
      memcpy(&r, w, VB);
    }
    return r;
  }
};

// Sums of a and b over the tpr threads of a row; every thread gets them.  buf:
// two floats per warp of the block; `turn` alternates so that one barrier per
// sum is enough (a thread writes the other half while slower ones still read).
__device__ __forceinline__ float2 row_sum(float2 v, int tpr, float2 (*buf)[32], int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o < tpr) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
  }
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5, per = tpr >> 5;
    if ((threadIdx.x & 31) == 0) buf[turn][warp] = v;
    __syncthreads();
    const int w0 = warp / per * per;
    v = buf[turn][w0];
    for (int i = 1; i < per; ++i) {
      v.x += buf[turn][w0 + i].x;
      v.y += buf[turn][w0 + i].y;
    }
    turn ^= 1;
  }
  return v;
}

// A thread's own vectors of the coming rows: a ring of D rows in shared memory
// (Q inputs, V vectors per thread), filled by asynchronous copies of VB bytes and
// read back by the same thread, so no barrier is needed.  Rows of an odd number of
// bf16 elements have no copies that small; they are stored by the thread itself.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int VB, class Raw>
__device__ __forceinline__ void copy_vec(Raw *dst, const Raw *src) {
  if constexpr (VB == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
  else if constexpr (VB == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
  else
    *dst = *src;
}

// Rows in flight: what fits 64 to 96 KB of a block.
template <class El, int Q>
__host__ __device__ constexpr int ring_depth() {
  return sizeof(El) == 2 ? (Q == 1 ? 4 : 3) : (Q == 1 ? 4 : 2);
}
template <class El, int Q>
__host__ __device__ constexpr int ring_bytes(int threads) {
  return ring_depth<El, Q>() * Q * kElems * static_cast<int>(sizeof(El)) * threads;
}

template <class El, int VB, bool RES, int TH>
__global__ void __launch_bounds__(TH, 1024 / TH) norm_fwd_kernel(const NormArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  using Vc = Vec<El, VB>;
  using Raw = typename Vc::Raw;
  constexpr int N = Vc::N, V = kElems / N, Q = RES ? 2 : 1, D = ring_depth<El, Q>();
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float2 s_red[2][32];
  Raw *ring = reinterpret_cast<Raw *>(s_dyn) + threadIdx.x;  // vector (d, q, u) is ((d Q + q) V + u) TH further
  int turn = 0;
  const int tpr = a.tpr, rows = TH / tpr, lane = threadIdx.x % tpr, g = threadIdx.x / tpr;
  const int nv = a.H / N;
  const float inv = 1.f / static_cast<float>(a.H);
  const Raw *x = static_cast<const Raw *>(a.x), *res = static_cast<const Raw *>(a.res);
  const int step = gridDim.x * rows, t0 = blockIdx.x * rows + g;
  auto fetch = [&](int t, int d) {
    if (t < a.T) {
      const size_t at = static_cast<size_t>(t) * nv + lane;
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (lane + tpr * u < nv) {
          copy_vec<VB>(ring + ((d * Q) * V + u) * TH, x + at + tpr * u);
          if (RES) copy_vec<VB>(ring + ((d * Q + 1) * V + u) * TH, res + at + tpr * u);
        }
    }
    copies_commit();
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) fetch(t0 + d * step, d);
  Raw wr[V], br[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int v = lane + tpr * u;
    wr[u] = v < nv ? static_cast<const Raw *>(a.w)[v] : Vc::zero();
    br[u] = v < nv && a.b ? static_cast<const Raw *>(a.b)[v] : Vc::zero();
  }
  int d = 0;
  for (int r0 = blockIdx.x * rows; r0 < a.T; r0 += step) {
    const int t = r0 + g;
    fetch(t + (D - 1) * step, d == 0 ? D - 1 : d - 1);
    copies_wait<D - 1>();
    const size_t at = static_cast<size_t>(t) * nv;
    float f[kElems];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int v = lane + tpr * u;
      const bool in = t < a.T && v < nv;
      Vc::unpack(in ? ring[((d * Q) * V + u) * TH] : Vc::zero(), f + N * u);
      if (RES) {
        float q[N];
        Vc::unpack(in ? ring[((d * Q + 1) * V + u) * TH] : Vc::zero(), q);
#pragma unroll
        for (int i = 0; i < N; ++i) f[N * u + i] += q[i];
        const Raw h = Vc::pack(f + N * u);
        Vc::unpack(h, f + N * u);  // the norm is that of the stored sum
        if (in) static_cast<Raw *>(a.sum)[at + v] = h;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) s.x += f[N * u + i];
    }
    if (++d == D) d = 0;
    float mu = 0.f;
    if (a.layer) mu = row_sum(s, tpr, s_red, turn).x * inv;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (lane + tpr * u < nv) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          f[N * u + i] -= mu;
          s.x = fmaf(f[N * u + i], f[N * u + i], s.x);
        }
      }
    const float r = 1.f / sqrtf(fmaf(row_sum(s, tpr, s_red, turn).x, inv, a.eps));
    if (t < a.T) {
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int v = lane + tpr * u;
        if (v < nv) {
          float w[N], b[N], o[N];
          Vc::unpack(wr[u], w);
          Vc::unpack(br[u], b);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = fmaf(f[N * u + i] * r, w[i], b[i]);
          static_cast<Raw *>(a.y)[at + v] = Vc::pack(o);
        }
      }
      if (lane == 0) a.stats[t] = make_float2(mu, r);
    }
  }
}

template <class El, int VB, bool RES, int TH>
__global__ void __launch_bounds__(TH, 512 / TH) norm_bwd_kernel(const NormArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  using Vc = Vec<El, VB>;
  using Raw = typename Vc::Raw;
  constexpr int N = Vc::N, V = kElems / N, Q = RES ? 3 : 2, D = ring_depth<El, Q>();
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float2 s_red[2][32];
  Raw *ring = reinterpret_cast<Raw *>(s_dyn) + threadIdx.x;
  int turn = 0;
  const int tpr = a.tpr, rows = TH / tpr, lane = threadIdx.x % tpr, g = threadIdx.x / tpr;
  const int nv = a.H / N;
  const float inv = 1.f / static_cast<float>(a.H);
  const Raw *x = static_cast<const Raw *>(a.x), *dy = static_cast<const Raw *>(a.dy);
  const Raw *ds = static_cast<const Raw *>(a.res);
  const int step = gridDim.x * rows, t0 = blockIdx.x * rows + g;
  auto fetch = [&](int t, int d) {
    if (t < a.T) {
      const size_t at = static_cast<size_t>(t) * nv + lane;
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (lane + tpr * u < nv) {
          copy_vec<VB>(ring + ((d * Q) * V + u) * TH, x + at + tpr * u);
          copy_vec<VB>(ring + ((d * Q + 1) * V + u) * TH, dy + at + tpr * u);
          if (RES) copy_vec<VB>(ring + ((d * Q + 2) * V + u) * TH, ds + at + tpr * u);
        }
    }
    copies_commit();
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) fetch(t0 + d * step, d);
  Raw wr[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int v = lane + tpr * u;
    wr[u] = v < nv ? static_cast<const Raw *>(a.w)[v] : Vc::zero();
  }
  float aw[kElems], ab[kElems];
#pragma unroll
  for (int i = 0; i < kElems; ++i) aw[i] = ab[i] = 0.f;
  float2 next = t0 < a.T ? a.stats[t0] : make_float2(0.f, 0.f);
  int d = 0;
  for (int r0 = blockIdx.x * rows; r0 < a.T; r0 += step) {
    const int t = r0 + g;
    fetch(t + (D - 1) * step, d == 0 ? D - 1 : d - 1);
    const float mu = next.x, r = next.y;
    if (t + step < a.T) next = a.stats[t + step];
    copies_wait<D - 1>();
    const size_t at = static_cast<size_t>(t) * nv;
    float xh[kElems], gw[kElems];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float w[N], e[N];
      const bool in = t < a.T && lane + tpr * u < nv;
      Vc::unpack(in ? ring[((d * Q) * V + u) * TH] : Vc::zero(), xh + N * u);
      Vc::unpack(in ? ring[((d * Q + 1) * V + u) * TH] : Vc::zero(), e);
      Vc::unpack(wr[u], w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = N * u + i;
        xh[j] = in ? (xh[j] - mu) * r : 0.f;
        gw[j] = e[i] * w[i];
        s.x += gw[j];
        s.y = fmaf(gw[j], xh[j], s.y);
        aw[j] = fmaf(e[i], xh[j], aw[j]);
        ab[j] += e[i];
      }
    }
    s = row_sum(s, tpr, s_red, turn);
    const float c1 = s.y * inv, c2 = a.layer ? s.x * inv : 0.f;
    if (t < a.T) {
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int v = lane + tpr * u;
        if (v < nv) {
          float o[N];
          Vc::unpack(RES ? ring[((d * Q + 2) * V + u) * TH] : Vc::zero(), o);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int j = N * u + i;
            o[i] = fmaf(r, gw[j] - c2 - xh[j] * c1, o[i]);
          }
          static_cast<Raw *>(a.y)[at + v] = Vc::pack(o);
        }
      }
    }
    if (++d == D) d = 0;
  }
  // the block's column sums: its row groups added in order, one after another
  copies_wait<0>();
  __syncthreads();  // the ring is no longer read: it holds the sums
  float *s_col = reinterpret_cast<float *>(s_dyn);  // [2][H] when several rows share the block (H <= TH kElems / 2)
  float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.H;
  for (int q = 0; q < rows; ++q) {
    if (q > 0) __syncthreads();
    if (g == q) {
      float *out = q == rows - 1 ? part : s_col;
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int v = lane + tpr * u;
        if (v < nv) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int c = v * N + i;
            out[c] = q > 0 ? s_col[c] + aw[N * u + i] : aw[N * u + i];
            out[a.H + c] = q > 0 ? s_col[a.H + c] + ab[N * u + i] : ab[N * u + i];
          }
        }
      }
    }
  }
}

// dw[c] and db[c] = the sum over the blocks' partial rows in a fixed order: 8
// columns x 32 interleaved runs of rows per block, the runs added in a tree.
__global__ void __launch_bounds__(256) norm_colsum_kernel(const float *__restrict__ part, int nb, int H,
                                                          float *__restrict__ dw, float *__restrict__ db) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s[32][9];
  const int cl = threadIdx.x & 7, run = threadIdx.x >> 3;
  const int c = blockIdx.x * 8 + cl;
  const float *src = part + static_cast<size_t>(blockIdx.y) * H + c;
  float acc = 0.f;
  if (c < H) {
#pragma unroll 10
    for (int b = run; b < nb; b += 32) acc += src[static_cast<size_t>(b) * 2 * H];
  }
  s[run][cl] = acc;
  __syncthreads();
  if (threadIdx.x < 32) {  // lane = run here: a tree over the 32 runs of each column
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = warp_sum(s[threadIdx.x][i]);
      if (static_cast<int>(threadIdx.x) == i) acc = v;
    }
    const int o = blockIdx.x * 8 + threadIdx.x;
    if (threadIdx.x < 8 && o < H) (blockIdx.y == 0 ? dw : db)[o] = acc;
  }
}

int tpr_of(int H) {
  int tpr = 8;
  while (tpr * kElems < H) tpr *= 2;
  return tpr;
}

// The widest vectors that divide a row (all base pointers are 16-byte aligned,
// so every row then starts on a vector).
int vector_bytes(int H, int el) {
  const int row = H * el;
  return row % 16 == 0 ? 16 : (row % 4 == 0 ? 4 : 2);
}

// Blocks of a kernel that fit the part at once, after its shared-memory opt-in.
template <class K>
cudaError_t resident(DeviceOnce &once, K kernel, int threads, int smem, int sms, int *blocks) {
  return once.get(
      [&](int *out) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, kernel, threads, smem);
        *out *= sms;
        return e != cudaSuccess || *out > 0 ? e : cudaErrorInvalidConfiguration;
      },
      blocks);
}

template <class El, int VB, bool RES, int TH>
cudaError_t launch_fwd(const NormArgs &a, int sms, cudaStream_t s) {
  static DeviceOnce once;
  constexpr int smem = ring_bytes<El, RES ? 2 : 1>(TH);
  int most = 0;
  const cudaError_t e = resident(once, norm_fwd_kernel<El, VB, RES, TH>, TH, smem, sms, &most);
  if (e != cudaSuccess) return e;
  const int rows = TH / a.tpr, need = (a.T + rows - 1) / rows;
  return launch_pdl(norm_fwd_kernel<El, VB, RES, TH>, dim3(need < most ? need : most), dim3(TH), smem, s, 1, a);
}

template <class El, int VB, bool RES, int TH>
cudaError_t launch_bwd(const NormArgs &a, int sms, float *dw, float *db, cudaStream_t s) {
  static DeviceOnce once;
  constexpr int smem = ring_bytes<El, RES ? 3 : 2>(TH);
  int most = 0;
  cudaError_t e = resident(once, norm_bwd_kernel<El, VB, RES, TH>, TH, smem, sms, &most);
  if (e != cudaSuccess) return e;
  if (most > kBwdBlocks) most = kBwdBlocks;
  const int rows = TH / a.tpr, need = (a.T + rows - 1) / rows, nb = need < most ? need : most;
  e = launch_pdl(norm_bwd_kernel<El, VB, RES, TH>, dim3(nb), dim3(TH), smem, s, 1, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_colsum_kernel, dim3((a.H + 7) / 8, db ? 2 : 1), dim3(256), 0, s, 1, a.part, nb, a.H, dw, db);
}

// The variant for a configuration: vectors as wide as the rows allow, 512 threads
// only where a row takes them.
template <class F>
cudaError_t by_form(bool bf, int H, bool res, F &&f) {
  const bool wide = tpr_of(H) > kThreads;
  auto pick = [&](auto el, auto vb) {
    if (res)
      return wide ? f(el, vb, std::true_type{}, std::integral_constant<int, 512>{})
                  : f(el, vb, std::true_type{}, std::integral_constant<int, 256>{});
    return wide ? f(el, vb, std::false_type{}, std::integral_constant<int, 512>{})
                : f(el, vb, std::false_type{}, std::integral_constant<int, 256>{});
  };
  const int vb = vector_bytes(H, bf ? 2 : 4);
  if (bf) {
    if (vb == 16) return pick(uint16_t{}, std::integral_constant<int, 16>{});
    return vb == 4 ? pick(uint16_t{}, std::integral_constant<int, 4>{})
                   : pick(uint16_t{}, std::integral_constant<int, 2>{});
  }
  return vb == 16 ? pick(float{}, std::integral_constant<int, 16>{}) : pick(float{}, std::integral_constant<int, 4>{});
}

bool norm_ok(const moe_norm_config *c) {
  return c && c->T >= 0 && c->T <= (1 << 30) && c->H >= 1 && c->H <= kMaxH && (c->kind == MOE_NORM_LAYER || c->kind == MOE_NORM_RMS) &&
         (c->dtype == MOE_DTYPE_BF16 || c->dtype == MOE_DTYPE_FP32) && c->eps >= 0.f;
}

NormArgs norm_args(const moe_norm_config *c) {
  NormArgs a{};
  a.T = c->T;
  a.H = c->H;
  a.eps = c->eps;
  a.layer = c->kind == MOE_NORM_LAYER;
  a.tpr = tpr_of(c->H);
  return a;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_norm_workspace(const moe_norm_config *cfg, size_t *bwd_scratch) {
  if (!norm_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (bwd_scratch) *bwd_scratch = align256(static_cast<size_t>(kBwdBlocks) * 2 * cfg->H * sizeof(float));
  return MOE_OK;
}

moe_status moe_norm_forward(const moe_norm_config *cfg, const void *x, const void *residual, const void *weight,
                            const void *bias, void *y, void *sum, float *stats, void *stream) {
  if (!norm_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!weight || (!residual != !sum) || (cfg->T > 0 && (!x || !y || !stats))) return MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(residual) || !al16(weight) || !al16(bias) || !al16(y) || !al16(sum) || !al16(stats))
    return MOE_ERR_ALIGNMENT;
  DevInfo di;
  MOE_TRY(device_info(&di));
  if (cfg->T == 0) return MOE_OK;
  NormArgs a = norm_args(cfg);
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.sum = sum;
  a.stats = reinterpret_cast<float2 *>(stats);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return timed("norm_forward", s, [&] {
    return by_form(cfg->dtype == MOE_DTYPE_BF16, cfg->H, residual != nullptr, [&](auto el, auto vb, auto res, auto th) {
      return launch_fwd<decltype(el), decltype(vb)::value, decltype(res)::value, decltype(th)::value>(a, di.sms, s);
    });
  });
}

moe_status moe_norm_backward(const moe_norm_config *cfg, const void *dy, const void *h, const void *weight,
                             const float *stats, const void *d_sum, void *dx, float *dweight, float *dbias,
                             void *scratch, size_t scratch_bytes, void *stream) {
  if (!norm_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!weight || !dweight || !scratch || (cfg->T > 0 && (!dy || !h || !stats || !dx))) return MOE_ERR_INVALID_ARG;
  if (!al16(dy) || !al16(h) || !al16(weight) || !al16(stats) || !al16(d_sum) || !al16(dx) || !al16(dweight) ||
      !al16(dbias) || !al16(scratch))
    return MOE_ERR_ALIGNMENT;
  size_t need = 0;
  moe_norm_workspace(cfg, &need);
  if (scratch_bytes < need) return MOE_ERR_WORKSPACE;
  DevInfo di;
  MOE_TRY(device_info(&di));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cfg->T == 0) {
    if (cudaMemsetAsync(dweight, 0, sizeof(float) * cfg->H, s) != cudaSuccess ||
        (dbias && cudaMemsetAsync(dbias, 0, sizeof(float) * cfg->H, s) != cudaSuccess))
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  NormArgs a = norm_args(cfg);
  a.x = h;
  a.dy = dy;
  a.res = d_sum;
  a.w = weight;
  a.y = dx;
  a.stats = const_cast<float2 *>(reinterpret_cast<const float2 *>(stats));
  a.part = static_cast<float *>(scratch);
  return timed("norm_backward", s, [&] {
    return by_form(cfg->dtype == MOE_DTYPE_BF16, cfg->H, d_sum != nullptr, [&](auto el, auto vb, auto res, auto th) {
      return launch_bwd<decltype(el), decltype(vb)::value, decltype(res)::value, decltype(th)::value>(
          a, di.sms, dweight, dbias, s);
    });
  });
}

}  // extern "C"
