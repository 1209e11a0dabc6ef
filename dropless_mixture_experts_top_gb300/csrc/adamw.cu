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
// Bound by memory: fp32 states with bf16 gradients and copies move 28 bytes per element (302 million elements: 1270 to 1290
// us, 98 to 99% of what a copy moves in that time), 8-bit ones 16 (780 to 794 us, 91 to 93%).  A warp takes 256 elements (a block of the states)
// in accesses of whole lines and reduces the block's largest by redux; with 8-bit states it has the next 256 under way
// meanwhile (without that, and with checks and choices for every element, it was bound by its instructions: 1260 us).
// The tensors' addresses
// travel in the launch's parameters: no table on the device, nothing to copy.
//
// The number of steps is device memory, so that a captured step counts on: every
// block reads it, the last one to finish (a ticket that wraps to zero) advances it.
#include <cuda_fp16.h>
#include <float.h>
#include <math.h>

#include <type_traits>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Blocks per SM, by the states' bits.  Measured, 302 million elements: 32 bits 2, 3 and 4 blocks 1277, 1297 and 1347 us (4
// spill); 8 bits 2, 3 and 4 blocks 803, 794 and 900 us.
constexpr int kBlocks32 = 2, kBlocks8 = 3;
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

// A lane's eight elements of a unit: four from 4 lane on, four from 4 lane + 128; `left`: how many of each four the
// tensor has.  As they come from memory (El: float, uint16_t bf16 bits, uint8_t e4m3 codes):
template <class El>
struct Eight {
  static constexpr int W = static_cast<int>(sizeof(El));  // words of four elements
  uint32_t r[2 * W];
  __device__ __forceinline__ void load(const El *src, const int (&left)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const El *s = src + 128 * h;
      if (left[h] == 4) {
        if constexpr (W == 4) {
          const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(s));
          r[4 * h] = q.x, r[4 * h + 1] = q.y, r[4 * h + 2] = q.z, r[4 * h + 3] = q.w;
        } else if constexpr (W == 2) {
          const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(s));
          r[2 * h] = q.x, r[2 * h + 1] = q.y;
        } else {
          r[h] = __ldcs(reinterpret_cast<const uint32_t *>(s));
        }
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) r[W * h + w] = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < left[h]) {
            if constexpr (W == 4)
              r[4 * h + i] = __float_as_uint(s[i]);
            else
              r[W * h + i * W / 4] |= static_cast<uint32_t>(s[i]) << (8 * W * i % 32);
          }
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (W == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * h + i] = __uint_as_float(r[4 * h + i]);
      } else if constexpr (W == 2) {
        f[4 * h] = bf16_lo(r[2 * h]), f[4 * h + 1] = bf16_hi(r[2 * h]);
        f[4 * h + 2] = bf16_lo(r[2 * h + 1]), f[4 * h + 3] = bf16_hi(r[2 * h + 1]);
      } else {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(r[h]));
        const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo)), b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
        f[4 * h] = a.x, f[4 * h + 1] = a.y, f[4 * h + 2] = b.x, f[4 * h + 3] = b.y;
      }
    }
  }
};
template <class El>
__device__ __forceinline__ void store_eight(El *dst, const int (&left)[2], const float (&f)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    El *d = dst + 128 * h;
    const float *v = f + 4 * h;
    if constexpr (sizeof(El) == 4) {
      if (left[h] == 4) {
        __stcs(reinterpret_cast<float4 *>(d), make_float4(v[0], v[1], v[2], v[3]));
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < left[h]) d[i] = v[i];
      }
    } else if constexpr (sizeof(El) == 2) {
      const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
      if (left[h] == 4) {
        __stcs(reinterpret_cast<uint2 *>(d), make_uint2(lo, hi));
      } else {
        if (left[h] > 0) d[0] = static_cast<uint16_t>(lo);
        if (left[h] > 1) d[1] = static_cast<uint16_t>(lo >> 16);
        if (left[h] > 2) d[2] = static_cast<uint16_t>(hi);
      }
    } else {
      uint32_t c;
      asm("{\n\t.reg .b16 a, b;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
          "mov.b32 %0, {a, b};\n\t}"
          : "=r"(c)
          : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
      if (left[h] == 4) {
        __stcs(reinterpret_cast<uint32_t *>(d), c);
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (i < left[h]) d[i] = static_cast<uint8_t>(c >> (8 * i));
      }
    }
  }
}

__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest |x| of the warp's 256, at least kTiny (NaN left out).
__device__ __forceinline__ float block_most(const float (&x)[8]) {
  float m = kTiny;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}

// Where the u-th unit of a launch lies.
struct Place {
  int64_t x0, s0;  // the lane's first element in the tensor, in the states
  int have;        // elements of the unit in the tensor
  __device__ __forceinline__ Place(const Entry &e, int64_t u, int lane) {
    x0 = (u - e.first) * kBlock;
    const int64_t n = e.n - x0;
    have = n >= kBlock ? kBlock : static_cast<int>(n);
    s0 = e.unit * kBlock + x0 + lane * 4;
    x0 += lane * 4;
  }
};
// f(left) with what the lane has of a unit: constants for a whole one.
template <class F>
__device__ __forceinline__ void with_left(int have, int lane, F &&f) {
  if (have == kBlock) {
    const int left[2] = {4, 4};
    f(left);
  } else {
    const int left[2] = {max(0, min(4, have - 4 * lane)), max(0, min(4, have - 128 - 4 * lane))};
    f(left);
  }
}

// A unit as it comes from memory.
template <class P, class G, bool EIGHT>
struct Unit {
  using S = typename std::conditional<EIGHT, uint8_t, float>::type;
  Eight<P> p;
  Eight<G> g;
  Eight<S> m, v;
  float sm, sv;
  int at;  // its tensor
  __device__ __forceinline__ void load(const StepArgs &a, int64_t u, int lane) {
    if (u >= a.units) return;
    while (at + 1 < a.tensors && u >= a.e[at + 1].first) ++at;
    const Entry &e = a.e[at];
    const Place l(e, u, lane);
    with_left(l.have, lane, [&](const int(&left)[2]) {
      p.load(static_cast<const P *>(e.p) + l.x0, left);
      g.load(static_cast<const G *>(e.g) + l.x0, left);
      m.load(static_cast<const S *>(a.m) + l.s0, left);
      v.load(static_cast<const S *>(a.v) + l.s0, left);
    });
    if constexpr (EIGHT) {
      // (not by the read-only path, since this launch writes the neighbours; around the L1 302 million elements take 915 us
      // instead of 782: a line's scales are read one by one)
      sm = a.m_scale[l.s0 / kBlock];
      sv = a.v_scale[l.s0 / kBlock];
    }
  }
};

// A parameter is finite if what is stored of it is: bf16 rounds what is at least 2^128 - 2^119 to infinity.
template <class P>
constexpr float kMostParam = sizeof(P) == 2 ? 0x1.fefffep127f : FLT_MAX;

// Products and sums are rounded one by one (no fused multiply-add), and the root is the exact one, where they enter the
// 8-bit codes: a code is then the same wherever the formula is written out in fp32, as in a run that goes on from a
// checkpoint elsewhere.
template <class P, class G, bool EIGHT>
__global__ void __launch_bounds__(kThreads, EIGHT ? kBlocks8 : kBlocks32) adamw_kernel(const __grid_constant__ StepArgs a) {
  using U = Unit<P, G, EIGHT>;
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  U next;
  next.at = 0;
  if (EIGHT) next.load(a, u, lane);
  const int steps = __ldcg(a.step + 1) + 1;
  const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
  const float gs = a.scale ? __ldg(a.scale) : 1.f;
  const bool skip = !(fabsf(gs) <= FLT_MAX);
  // 1 - b^t = -expm1(t log b), which is exact to a few ulp (the logarithm is rounded once)
  const float corr1 = -expm1f(static_cast<float>(steps) * a.log_b1), corr2 = -expm1f(static_cast<float>(steps) * a.log_b2);
  const float rate = lr / corr1, root = rsqrtf(corr2);
  bool bad = skip;
  auto advance = [&](const U &x, int64_t u) {
    using S = typename U::S;
    const Entry &e = a.e[x.at];
    float pv[8], gv[8], mv[8], vv[8], r[8];
    x.p.get(pv);
    x.g.get(gv);
    x.m.get(mv);
    x.v.get(vv);
    const float keep = 1.f - lr * e.decay;
    float fin = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (EIGHT) {
        mv[i] = __fmul_rn(mv[i], x.sm);
        vv[i] = __fmul_rn(vv[i], x.sv);
        vv[i] = __fmul_rn(vv[i], vv[i]);
      }
      const float gr = __fmul_rn(gv[i], gs);
      mv[i] = __fadd_rn(__fmul_rn(a.b1, mv[i]), __fmul_rn(a.c1, gr));
      vv[i] = __fadd_rn(__fmul_rn(a.b2, vv[i]), __fmul_rn(a.c2, __fmul_rn(gr, gr)));
      const float root_v = EIGHT ? __fsqrt_rn(vv[i]) : sqrt_fast(vv[i]);
      if (EIGHT) r[i] = root_v;
      pv[i] = fmaf(pv[i], keep, -__fdividef(rate * mv[i], fmaf(root_v, root, a.eps)));
      // NaN where one is not finite (of bf16, from 1.98 2^127 on)
      fin = fmaf(vv[i], 0.f, fmaf(sizeof(P) == 2 ? pv[i] * 1.01f : pv[i], 0.f, fin));
    }
    const Place l(e, u, lane);
    // An element whose parameter or v is not finite.  In 8 bits it becomes e4m3's NaN and has no part in its block's
    // scales, though its m, or its root, be finite: a gradient of 1e20 makes v infinite and m so large that the other 255
    // would all be rounded to zero.
    if (fin != 0.f) {  // (elements past a tensor's end are zeros, of which eps = 0 makes NaN)
      with_left(l.have, lane, [&](const int(&left)[2]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool odd = !(fabsf(pv[i]) <= kMostParam<P> && vv[i] <= FLT_MAX);
          bad |= odd && (i & 3) < left[i >> 2];
          if (EIGHT && odd) mv[i] = r[i] = NAN;
        }
      });
    }
    if constexpr (EIGHT) {
      const float most_m = block_most(mv), most_r = block_most(r);
      const float im = __fmul_rn(__frcp_rn(most_m), kCodeMax), ir = __fmul_rn(__frcp_rn(most_r), kCodeMax);
      if (lane == 0) {
        a.m_scale[l.s0 / kBlock] = __fmul_rn(most_m, 1.f / kCodeMax);
        a.v_scale[l.s0 / kBlock] = __fmul_rn(most_r, 1.f / kCodeMax);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mv[i] *= im;
        vv[i] = r[i] > 0.f ? fmaxf(r[i] * ir, kCodeLeast) : r[i];
      }
    }
    with_left(l.have, lane, [&](const int(&left)[2]) {
      store_eight(static_cast<P *>(e.p) + l.x0, left, pv);
      if constexpr (sizeof(P) == 4)
        if (e.copy) store_eight(e.copy + l.x0, left, pv);
      store_eight(static_cast<S *>(a.m) + l.s0, left, mv);
      store_eight(static_cast<S *>(a.v) + l.s0, left, vv);
    });
  };
  if (!skip) {
    for (; u < a.units; u += step) {
      if constexpr (EIGHT) {  // the next unit's loads are under way meanwhile
        const U x = next;
        next.load(a, u + step, lane);
        advance(x, u);
      } else {
        next.load(a, u, lane);
        advance(next, u);
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
    for (; i < cfg->tensors; ++i) {
      if (n[i] == 0) continue;
      if (a.tensors == kPerLaunch) break;
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
    const int64_t wanted = (a.units + kWarps - 1) / kWarps, most = static_cast<int64_t>(di.sms) * (eight ? kBlocks8 : kBlocks32);
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
