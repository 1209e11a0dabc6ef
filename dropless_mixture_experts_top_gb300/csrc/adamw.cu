// adamw.cu -- one AdamW step over a list of tensors in one launch, with states in
// 32 bits or in 8.
//
// Per element, t the step's number:
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2        (g times the gradients' scale)
//   p <- p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
// and, for fp32 parameters, a bf16 copy of p.  8-bit states hold m and sqrt(v) as e4m3
// values times one fp32 scale per 256 elements (a block's largest is 448); the step
// itself uses m and v as they are before that rounding (half of 2^-3 of a value at
// most: the state that a step leaves is what the next one starts from).  The root is
// held instead of v because e4m3 spans 2^18: v then spans 2^36 within a block, and a
// positive root is never rounded to zero, since a zero under a nonzero m would make
// an update as large as m / eps.
//
// Bound by memory: fp32 states with bf16 gradients and copies move 28 bytes per element, 8-bit
// ones 16.  A warp takes 256 elements (a block of the states) in 16-byte accesses of
// whole lines and reduces the block's largest by redux; with 32 warps an SM holds 115
// (64) KB of loads in flight, enough for HBM without staging.  The tensors' addresses
// travel in the launch's parameters: no table on the device, nothing to copy.
//
// The number of steps is device memory, so that a captured step counts on: every
// block reads it, the last one to finish (a ticket that wraps to zero) advances it.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 4;
constexpr int kBlock = 256;       // elements of a warp's unit, which share a scale
constexpr int kPerLaunch = 64;    // tensors of one launch (its parameters stay below 4 KB)
constexpr float kTiny = 1e-30f;   // the least largest value of a block that a scale is made for
constexpr float kCodeMax = 448.f;
constexpr float kCodeLeast = 1.f / 512.f;

struct Entry {
  void *p;
  const void *g;
  uint16_t *copy;
  int64_t n;
  int64_t first;  // the launch's units in front of it
  int64_t unit;   // its first unit in the states
  float decay;
};
struct StepArgs {
  Entry e[kPerLaunch];
  int64_t units;
  void *m, *v;
  float *m_scale, *v_scale;
  int32_t *step;  // status, steps, arrivals, flags
  const float *lr_dev, *scale;
  float lr, b1, c1, b2, c2, log_b1, log_b2, eps;
  int tensors;
  bool last;      // of the call's launches
};
static_assert(sizeof(StepArgs) <= 4096, "the launch's parameters");

// Eight elements of a lane: four from `at`, four from at + 128, of which `left` are in the tensor.
template <class El>
__device__ __forceinline__ void load4(const El *src, int left, float *f) {
  if (left >= 4) {
    if constexpr (sizeof(El) == 4) {
      const float4 q = __ldcs(reinterpret_cast<const float4 *>(src));
      f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
    } else {
      const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(src));
      f[0] = bf16_lo(q.x), f[1] = bf16_hi(q.x), f[2] = bf16_lo(q.y), f[3] = bf16_hi(q.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = 0.f;
      if (i < left) {
        if constexpr (sizeof(El) == 4)
          f[i] = src[i];
        else
          f[i] = __uint_as_float(static_cast<uint32_t>(src[i]) << 16);
      }
    }
  }
}
template <class El>
__device__ __forceinline__ void store4(El *dst, int left, const float *f) {
  if (left >= 4) {
    if constexpr (sizeof(El) == 4)
      __stcs(reinterpret_cast<float4 *>(dst), make_float4(f[0], f[1], f[2], f[3]));
    else
      __stcs(reinterpret_cast<uint2 *>(dst), make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) {
        if constexpr (sizeof(El) == 4)
          dst[i] = f[i];
        else
          dst[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
      }
  }
}

// Four e4m3 codes in a word.
__device__ __forceinline__ void decode4(uint32_t c, float *f) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
  const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}
__device__ __forceinline__ uint32_t encode4(const float *f) {
  uint32_t c;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(c)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]));
  return c;
}
__device__ __forceinline__ void load_codes(const uint8_t *src, int left, float *f) {
  uint32_t c = 0;
  if (left >= 4) {
    c = __ldcs(reinterpret_cast<const uint32_t *>(src));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) c |= static_cast<uint32_t>(src[i]) << (8 * i);
  }
  decode4(c, f);
}
__device__ __forceinline__ void store_codes(uint8_t *dst, int left, const float *f) {
  const uint32_t c = encode4(f);
  if (left >= 4) {
    __stcs(reinterpret_cast<uint32_t *>(dst), c);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < left) dst[i] = static_cast<uint8_t>(c >> (8 * i));
  }
}

// The largest finite |x| of the warp's 256, at least kTiny.
__device__ __forceinline__ float block_most(const float (&x)[8]) {
  float m = kTiny;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fabsf(x[i]) <= FLT_MAX ? fmaxf(m, fabsf(x[i])) : m;
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// Products and sums are rounded one by one (no fused multiply-add) where they enter the 8-bit
// codes, so that a code is the same wherever the formula is written out in fp32.
template <class P, class G, bool EIGHT>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) adamw_kernel(const __grid_constant__ StepArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int steps = __ldcg(a.step + 1) + 1;
  const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
  const float gs = a.scale ? __ldg(a.scale) : 1.f;
  const bool skip = !(fabsf(gs) <= FLT_MAX);
  // 1 - b^t = -expm1(t log b), which is exact to a few ulp (the logarithm is rounded once)
  const float corr1 = -expm1f(static_cast<float>(steps) * a.log_b1), corr2 = -expm1f(static_cast<float>(steps) * a.log_b2);
  const float rate = lr / corr1, root = rsqrtf(corr2);
  bool bad = skip;
  int at = 0;
  if (!skip) {
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < a.units; u += static_cast<int64_t>(gridDim.x) * kWarps) {
      while (at + 1 < a.tensors && u >= a.e[at + 1].first) ++at;
      const Entry &e = a.e[at];
      const int64_t x0 = (u - e.first) * kBlock + lane * 4;  // the lane's first element in the tensor
      const int64_t s0 = (e.unit + (u - e.first)) * kBlock + lane * 4;
      P *p = static_cast<P *>(e.p) + x0;
      const G *g = static_cast<const G *>(e.g) + x0;
      float pv[8], gv[8], mv[8], vv[8];
      int left[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t n = e.n - x0 - 128 * h;
        left[h] = n >= 4 ? 4 : (n > 0 ? static_cast<int>(n) : 0);
      }
      float sm = 0.f, sv = 0.f;
      if constexpr (EIGHT) {
        sm = __ldg(a.m_scale + s0 / kBlock);
        sv = __ldg(a.v_scale + s0 / kBlock);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        load4(p + 128 * h, left[h], pv + 4 * h);
        load4(g + 128 * h, left[h], gv + 4 * h);
        if constexpr (EIGHT) {
          load_codes(static_cast<const uint8_t *>(a.m) + s0 + 128 * h, left[h], mv + 4 * h);
          load_codes(static_cast<const uint8_t *>(a.v) + s0 + 128 * h, left[h], vv + 4 * h);
        } else {
          load4(static_cast<const float *>(a.m) + s0 + 128 * h, left[h], mv + 4 * h);
          load4(static_cast<const float *>(a.v) + s0 + 128 * h, left[h], vv + 4 * h);
        }
      }
      const float keep = 1.f - lr * e.decay;
      float r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (EIGHT) {
          mv[i] = __fmul_rn(mv[i], sm);
          vv[i] = __fmul_rn(vv[i], sv);
          vv[i] = __fmul_rn(vv[i], vv[i]);
        }
        const float gr = __fmul_rn(gv[i], gs);
        mv[i] = __fadd_rn(__fmul_rn(a.b1, mv[i]), __fmul_rn(a.c1, gr));
        vv[i] = __fadd_rn(__fmul_rn(a.b2, vv[i]), __fmul_rn(a.c2, __fmul_rn(gr, gr)));
        r[i] = __fsqrt_rn(vv[i]);
        pv[i] = fmaf(pv[i], keep, -__fdividef(rate * mv[i], fmaf(r[i], root, a.eps)));
        bad |= (i & 3) < left[i >> 2] && !(fabsf(pv[i]) <= FLT_MAX && vv[i] <= FLT_MAX);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        store4(p + 128 * h, left[h], pv + 4 * h);
        if constexpr (sizeof(P) == 4)
          if (e.copy) store4(e.copy + x0 + 128 * h, left[h], pv + 4 * h);
      }
      if constexpr (EIGHT) {
        const float most_m = block_most(mv), most_r = block_most(r);
        const float im = __fdiv_rn(kCodeMax, most_m), ir = __fdiv_rn(kCodeMax, most_r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // (what is not finite becomes e4m3's NaN)
          mv[i] = fabsf(mv[i]) <= FLT_MAX ? __fmul_rn(mv[i], im) : NAN;
          const float q = r[i] <= FLT_MAX ? __fmul_rn(r[i], ir) : NAN;
          r[i] = r[i] > 0.f && q < kCodeLeast ? kCodeLeast : q;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          store_codes(static_cast<uint8_t *>(a.m) + s0 + 128 * h, left[h], mv + 4 * h);
          store_codes(static_cast<uint8_t *>(a.v) + s0 + 128 * h, left[h], r + 4 * h);
        }
        if (lane == 0) {
          a.m_scale[s0 / kBlock] = __fmul_rn(most_m, 1.f / kCodeMax);
          a.v_scale[s0 / kBlock] = __fmul_rn(most_r, 1.f / kCodeMax);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          store4(static_cast<float *>(a.m) + s0 + 128 * h, left[h], mv + 4 * h);
          store4(static_cast<float *>(a.v) + s0 + 128 * h, left[h], vv + 4 * h);
        }
      }
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    if (any) atomicOr(a.step + 3, kDevNonfiniteUpdate);
    if (a.last) {
      __threadfence();  // this block's reading of the steps and its flag come before its ticket
      const unsigned had = atomicInc(reinterpret_cast<unsigned *>(a.step + 2), gridDim.x - 1);
      if (had == gridDim.x - 1) {
        __threadfence();
        a.step[0] = atomicExch(a.step + 3, 0);
        if (!skip) a.step[1] = steps;
      }
    }
  }
}

bool adamw_ok(const moe_adamw_config *c) {
  if (!c || c->tensors < 0) return false;
  if (c->param_dtype != MOE_DTYPE_BF16 && c->param_dtype != MOE_DTYPE_FP32) return false;
  if (c->grad_dtype != MOE_DTYPE_BF16 && c->grad_dtype != MOE_DTYPE_FP32) return false;
  if (c->state_bits != 8 && c->state_bits != 32) return false;
  return c->beta1 >= 0 && c->beta1 < 1 && c->beta2 >= 0 && c->beta2 < 1 && c->eps >= 0 && c->eps <= FLT_MAX;
}

constexpr int64_t kMostElements = int64_t{1} << 40;  // of all tensors
bool sizes_ok(const moe_adamw_config *c, const int64_t *n) {
  if (c->tensors && !n) return false;
  int64_t all = 0;
  for (int i = 0; i < c->tensors; ++i) {
    if (n[i] < 0 || n[i] > kMostElements) return false;
    all += (n[i] + kBlock - 1) / kBlock * kBlock;
    if (all > kMostElements) return false;
  }
  return true;
}

template <class P, class G>
cudaError_t launch_step(const StepArgs &a, bool eight, int blocks, cudaStream_t s) {
  return eight ? launch_pdl(adamw_kernel<P, G, true>, dim3(blocks), dim3(kThreads), 0, s, 1, a)
               : launch_pdl(adamw_kernel<P, G, false>, dim3(blocks), dim3(kThreads), 0, s, 1, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_adamw_state_elements(const moe_adamw_config *cfg, const int64_t *n, int64_t *elements) {
  if (!adamw_ok(cfg) || !sizes_ok(cfg, n) || !elements) return MOE_ERR_INVALID_ARG;
  *elements = 0;
  for (int i = 0; i < cfg->tensors; ++i) *elements += (n[i] + kBlock - 1) / kBlock * kBlock;
  return MOE_OK;
}

moe_status moe_adamw_step(const moe_adamw_config *cfg, const int64_t *n, const double *decay, void *const *params,
                          const void *const *grads, void *const *copies, const moe_adamw_state *state, double lr,
                          const float *lr_device, const float *grad_scale, void *stream) {
  if (!adamw_ok(cfg) || !sizes_ok(cfg, n) || !state || !state->step) return MOE_ERR_INVALID_ARG;
  if (!lr_device && !(lr >= 0 && lr <= FLT_MAX)) return MOE_ERR_INVALID_ARG;
  if (cfg->tensors && (!params || !grads)) return MOE_ERR_INVALID_ARG;
  if (copies && cfg->param_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
  const bool eight = cfg->state_bits == 8;
  bool some = false, aligned = al16(state->m) && al16(state->v) && al16(state->m_scale) && al16(state->v_scale) &&
                               al16(state->step);
  for (int i = 0; i < cfg->tensors; ++i) {
    if (decay && !(decay[i] >= 0 && decay[i] <= FLT_MAX)) return MOE_ERR_INVALID_ARG;
    if (n[i] == 0) continue;
    some = true;
    if (!params[i] || !grads[i]) return MOE_ERR_INVALID_ARG;
    aligned = aligned && al16(params[i]) && al16(grads[i]) && (!copies || al16(copies[i]));
  }
  if (some && (!state->m || !state->v || (eight && (!state->m_scale || !state->v_scale)))) return MOE_ERR_INVALID_ARG;
  if (!aligned || (reinterpret_cast<uintptr_t>(lr_device) & 3) || (reinterpret_cast<uintptr_t>(grad_scale) & 3))
    return MOE_ERR_ALIGNMENT;
  DevInfo di;
  MOE_TRY(device_info(&di));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  StepArgs a;
  a.m = state->m;
  a.v = state->v;
  a.m_scale = state->m_scale;
  a.v_scale = state->v_scale;
  a.step = state->step;
  a.lr_dev = lr_device;
  a.scale = grad_scale;
  a.lr = static_cast<float>(lr);
  a.b1 = static_cast<float>(cfg->beta1);
  a.c1 = static_cast<float>(1 - cfg->beta1);
  a.b2 = static_cast<float>(cfg->beta2);
  a.c2 = static_cast<float>(1 - cfg->beta2);
  a.log_b1 = static_cast<float>(log(cfg->beta1));  // (of 0: -inf, and 1 - 0^t is 1)
  a.log_b2 = static_cast<float>(log(cfg->beta2));
  a.eps = static_cast<float>(cfg->eps);
  int i = 0;
  int64_t unit = 0;
  do {
    a.tensors = 0;
    a.units = 0;
    for (; i < cfg->tensors && a.tensors < kPerLaunch; ++i) {
      if (n[i] == 0) continue;
      Entry &e = a.e[a.tensors++];
      e.p = params[i];
      e.g = grads[i];
      e.copy = copies ? static_cast<uint16_t *>(copies[i]) : nullptr;
      e.n = n[i];
      e.first = a.units;
      e.unit = unit;
      e.decay = decay ? static_cast<float>(decay[i]) : 0.f;
      const int64_t u = (n[i] + kBlock - 1) / kBlock;
      a.units += u;
      unit += u;
    }
    a.last = i == cfg->tensors;
    const int64_t wanted = (a.units + kWarps - 1) / kWarps, most = static_cast<int64_t>(di.sms) * kBlocksPerSm;
    const int blocks = static_cast<int>(wanted < 1 ? 1 : (wanted < most ? wanted : most));
    const bool p32 = cfg->param_dtype == MOE_DTYPE_FP32, g32 = cfg->grad_dtype == MOE_DTYPE_FP32;
    MOE_TRY(timed("adamw_step", s, [&] {
      if (p32) return g32 ? launch_step<float, float>(a, eight, blocks, s) : launch_step<float, uint16_t>(a, eight, blocks, s);
      return g32 ? launch_step<uint16_t, float>(a, eight, blocks, s) : launch_step<uint16_t, uint16_t>(a, eight, blocks, s);
    }));
  } while (i < cfg->tensors);
  return MOE_OK;
}

}  // extern "C"
