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
// and dy) stay in its registers, and the next row's loads are issued before
// this row's sums.  The backward's blocks leave one partial row of column sums
// each, which a second kernel adds in a fixed order: no atomics, the same bits
// every time.
#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxH = 8192;
constexpr int kElems = 16;         // elements of a row per thread
constexpr int kMaxTpr = kMaxH / kElems;
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

template <class El, int VB>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  using Vc = Vec<El, VB>;
  using Raw = typename Vc::Raw;
  constexpr int N = Vc::N, V = kElems / N;
  __shared__ float2 s_red[2][32];
  int turn = 0;
  const int tpr = a.tpr, rows = blockDim.x / tpr, lane = threadIdx.x % tpr, g = threadIdx.x / tpr;
  const int nv = a.H / N;
  const float inv = 1.f / static_cast<float>(a.H);
  const Raw *x = static_cast<const Raw *>(a.x), *res = static_cast<const Raw *>(a.res);
  Raw wr[V], br[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int v = lane + tpr * u;
    wr[u] = v < nv ? static_cast<const Raw *>(a.w)[v] : Vc::zero();
    br[u] = v < nv && a.b ? static_cast<const Raw *>(a.b)[v] : Vc::zero();
  }
  Raw cx[V], cr[V];
  auto load = [&](int t) {
    const size_t at = static_cast<size_t>(t) * nv;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int v = lane + tpr * u;
      const bool in = t < a.T && v < nv;
      cx[u] = in ? x[at + v] : Vc::zero();
      cr[u] = in && res ? res[at + v] : Vc::zero();
    }
  };
  const int step = gridDim.x * rows;
  load(blockIdx.x * rows + g);
  for (int r0 = blockIdx.x * rows; r0 < a.T; r0 += step) {
    const int t = r0 + g;
    const size_t at = static_cast<size_t>(t) * nv;
    float f[kElems];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      Vc::unpack(cx[u], f + N * u);
      if (res) {
        float q[N];
        Vc::unpack(cr[u], q);
#pragma unroll
        for (int i = 0; i < N; ++i) f[N * u + i] += q[i];
        const Raw h = Vc::pack(f + N * u);
        Vc::unpack(h, f + N * u);  // the norm is that of the stored sum
        const int v = lane + tpr * u;
        if (t < a.T && v < nv) static_cast<Raw *>(a.sum)[at + v] = h;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) s.x += f[N * u + i];
    }
    load(t + step);  // the next row, while this one is summed
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
        if (v >= nv) break;
        float w[N], b[N], o[N];
        Vc::unpack(wr[u], w);
        Vc::unpack(br[u], b);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(f[N * u + i] * r, w[i], b[i]);
        static_cast<Raw *>(a.y)[at + v] = Vc::pack(o);
      }
      if (lane == 0) a.stats[t] = make_float2(mu, r);
    }
  }
}

template <class El, int VB>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  using Vc = Vec<El, VB>;
  using Raw = typename Vc::Raw;
  constexpr int N = Vc::N, V = kElems / N;
  extern __shared__ float s_col[];  // [2][H] when several rows share the block
  __shared__ float2 s_red[2][32];
  int turn = 0;
  const int tpr = a.tpr, rows = blockDim.x / tpr, lane = threadIdx.x % tpr, g = threadIdx.x / tpr;
  const int nv = a.H / N;
  const float inv = 1.f / static_cast<float>(a.H);
  const Raw *x = static_cast<const Raw *>(a.x), *dy = static_cast<const Raw *>(a.dy);
  const Raw *ds = static_cast<const Raw *>(a.res);
  Raw wr[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int v = lane + tpr * u;
    wr[u] = v < nv ? static_cast<const Raw *>(a.w)[v] : Vc::zero();
  }
  float aw[kElems], ab[kElems];
#pragma unroll
  for (int i = 0; i < kElems; ++i) aw[i] = ab[i] = 0.f;
  Raw cx[V], cd[V], cs[V];
  float2 st = make_float2(0.f, 0.f);
  auto load = [&](int t) {
    const size_t at = static_cast<size_t>(t) * nv;
    st = t < a.T ? a.stats[t] : make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int v = lane + tpr * u;
      const bool in = t < a.T && v < nv;
      cx[u] = in ? x[at + v] : Vc::zero();
      cd[u] = in ? dy[at + v] : Vc::zero();
      cs[u] = in && ds ? ds[at + v] : Vc::zero();
    }
  };
  const int step = gridDim.x * rows;
  load(blockIdx.x * rows + g);
  for (int r0 = blockIdx.x * rows; r0 < a.T; r0 += step) {
    const int t = r0 + g;
    const size_t at = static_cast<size_t>(t) * nv;
    const float mu = st.x, r = st.y;
    float xh[kElems], gw[kElems];
    Raw sv[V];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float w[N], d[N];
      Vc::unpack(cx[u], xh + N * u);
      Vc::unpack(cd[u], d);
      Vc::unpack(wr[u], w);
      sv[u] = cs[u];
      const bool in = t < a.T && lane + tpr * u < nv;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = N * u + i;
        xh[j] = in ? (xh[j] - mu) * r : 0.f;
        gw[j] = d[i] * w[i];
        s.x += gw[j];
        s.y = fmaf(gw[j], xh[j], s.y);
        aw[j] = fmaf(d[i], xh[j], aw[j]);
        ab[j] += d[i];
      }
    }
    load(t + step);  // the next row, while this one is summed
    s = row_sum(s, tpr, s_red, turn);
    const float c1 = s.y * inv, c2 = a.layer ? s.x * inv : 0.f;
    if (t < a.T) {
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int v = lane + tpr * u;
        if (v >= nv) break;
        float o[N];
        Vc::unpack(sv[u], o);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int j = N * u + i;
          o[i] = fmaf(r, gw[j] - c2 - xh[j] * c1, o[i]);
        }
        static_cast<Raw *>(a.y)[at + v] = Vc::pack(o);
      }
    }
  }
  // the block's column sums: its row groups added in order, one after another
  float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * a.H;
  float *dst = rows > 1 ? s_col : part;
  for (int q = 0; q < rows; ++q) {
    if (q > 0) __syncthreads();
    if (g == q) {
      float *out = q == rows - 1 ? part : dst;
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int v = lane + tpr * u;
        if (v >= nv) break;
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

// dw[c] and db[c] = the sum over the blocks' partial rows in a fixed order: 32
// columns x 8 interleaved runs of rows per block, the runs added in order.
__global__ void __launch_bounds__(256) norm_colsum_kernel(const float *__restrict__ part, int nb, int H,
                                                          float *__restrict__ dw, float *__restrict__ db) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s[8][33];
  const int cl = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cl;
  const float *src = part + static_cast<size_t>(blockIdx.y) * H + c;
  float acc = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int b = run; b < nb; b += 8) acc += src[static_cast<size_t>(b) * 2 * H];
  }
  s[run][cl] = acc;
  __syncthreads();
  if (run == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += s[i][cl];
    (blockIdx.y == 0 ? dw : db)[c] = acc;
  }
}

struct Shape {
  int tpr, threads, rows;
};
Shape shape_of(int H) {
  Shape s;
  s.tpr = 8;
  while (s.tpr * kElems < H) s.tpr *= 2;
  s.threads = s.tpr > kThreads ? s.tpr : kThreads;
  s.rows = s.threads / s.tpr;
  return s;
}

// The widest vectors that divide a row (all base pointers are 16-byte aligned,
// so every row then starts on a vector).
int vector_bytes(int H, int el) {
  const int row = H * el;
  return row % 16 == 0 ? 16 : (row % 4 == 0 ? 4 : 2);
}

template <class El, int VB>
cudaError_t launch_fwd(const NormArgs &a, int sms, cudaStream_t s) {
  const Shape sh = shape_of(a.H);
  const int need = (a.T + sh.rows - 1) / sh.rows, most = sms * (2048 / sh.threads);
  return launch_pdl(norm_fwd_kernel<El, VB>, dim3(need < most ? need : most), dim3(sh.threads), 0, s, 1, a);
}

template <class El, int VB>
cudaError_t launch_bwd(const NormArgs &a, float *dw, float *db, cudaStream_t s) {
  const Shape sh = shape_of(a.H);
  const int need = (a.T + sh.rows - 1) / sh.rows, nb = need < kBwdBlocks ? need : kBwdBlocks;
  const size_t smem = sh.rows > 1 ? static_cast<size_t>(2) * a.H * sizeof(float) : 0;  // H <= 2048 there
  cudaError_t e = launch_pdl(norm_bwd_kernel<El, VB>, dim3(nb), dim3(sh.threads), smem, s, 1, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_colsum_kernel, dim3((a.H + 31) / 32, db ? 2 : 1), dim3(256), 0, s, 1, a.part, nb, a.H, dw,
                    db);
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
  a.tpr = shape_of(c->H).tpr;
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
  const bool bf = cfg->dtype == MOE_DTYPE_BF16;
  const int vb = vector_bytes(cfg->H, bf ? 2 : 4);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return timed("norm_forward", s, [&] {
    if (bf) {
      if (vb == 16) return launch_fwd<uint16_t, 16>(a, di.sms, s);
      return vb == 4 ? launch_fwd<uint16_t, 4>(a, di.sms, s) : launch_fwd<uint16_t, 2>(a, di.sms, s);
    }
    return vb == 16 ? launch_fwd<float, 16>(a, di.sms, s) : launch_fwd<float, 4>(a, di.sms, s);
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
  const bool bf = cfg->dtype == MOE_DTYPE_BF16;
  const int vb = vector_bytes(cfg->H, bf ? 2 : 4);
  return timed("norm_backward", s, [&] {
    if (bf) {
      if (vb == 16) return launch_bwd<uint16_t, 16>(a, dweight, dbias, s);
      return vb == 4 ? launch_bwd<uint16_t, 4>(a, dweight, dbias, s) : launch_bwd<uint16_t, 2>(a, dweight, dbias, s);
    }
    return vb == 16 ? launch_bwd<float, 16>(a, dweight, dbias, s) : launch_bwd<float, 4>(a, dweight, dbias, s);
  });
}

}  // extern "C"
