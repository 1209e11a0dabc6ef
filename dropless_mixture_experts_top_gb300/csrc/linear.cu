// linear.cu -- a dense layer: a matrix product with bias, activation and residual
// in its epilogue, and its backward pass.
//
//   forward   z = x W + bias,   y = act(z) + residual        x [T,K], W [K,N]
//   backward  dz = dy act'(z),  dx = dz W^T,  dW = x^T dz,  dbias = sum_t dz
// x, W, bias, residual, z, y, dy, dx and dW are bf16, sums fp32.  dz is rounded to bf16 as
// an operand of the two products (dbias adds it up unrounded): dx and dW are then 2.3e-3 of
// themselves off in the mean square where their own rounding alone makes 1.7e-3; the tensor core
// multiplies bf16 by bf16, so that dz as the sum of two would be each product twice.
//
// Activations, in fp32:  relu;  silu z s(z);  gelu z s(2 sqrt(2/pi) (z + 0.044715 z^3)), the
// tanh form written with the sigmoid s, which takes one exponential and one reciprocal.
//
// No transposes: the tensor core reads either operand with its reduction axis
// contiguous (K-major boxes) or strided (MN-major): x . W reads W strided, dz . W^T
// contiguous, x^T . dz both strided.
//
// The products run on CTA pairs (tcgen05 cta_group::2, 256 x 256 tiles) or single
// CTAs (128 x 128), persistent over tiles, fp32 accumulators double-buffered in TMEM:
//   warp 0     TMA producer (each CTA): 128B-swizzled boxes, zeros past the ends
//   warp 1     MMA issuer (of a pair: CTA 0's)
//   warps 2-9  epilogue: tcgen05.ld, bias, activation, residual, bf16 rows
// Tiles that do not fill a last round are split along the reduction, so that the round
// is full: their parts leave fp32 sums in the workspace, which a second kernel adds in
// a fixed order before the same epilogue; or, of a single round, split over the blocks of
// a cluster, which add their sums over shared memory.  Where the tiles of dx and dW are one round
// together, one launch takes both, and the second step of dbias.  The forward of a few tokens is a pass over W on the
// CUDA cores (linear_rows_kernel).
//
// What bounds it, measured (graphs of ten calls): 16384 x 4096 x 4096 277 to 280 us, 1980 TFLOP/s (a library's
// product 266 to 269); 16384 x 1536 x 4096 114 us, 101 without the epilogue's stores, 124 to 127 with a residual, 135 with
// bias and gelu (which stores z, too): the tensor pipe is busy 72% of the time with residual.  Back to back the part's
// power cap holds both to 1.4e15 per second.  The backward of 16384 x 4096 x 1536 with silu takes 258 to 262: 117 for each
// product, 27 for dz and dbias.  Few tiles: 4 us and 0.46 us for each 128 of the reduction, 1.5 more in
// clusters, 5 in parts.
// Every wait is bounded; on a timeout the kernel flags the status word, drains its
// copies and MMAs, frees TMEM and returns.
#include <cuda.h>

#include <algorithm>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxDim = 65536;
constexpr int BM = 128;
constexpr int tile_size(int cg) { return BM * cg; }
constexpr int BK = 64;                // reduction elements per box: one 128-byte swizzle row
constexpr int kHalf = 128 * BK * 2;   // one operand's box (or two 64 x 64 boxes) per CTA: 16 KB
constexpr int kBox = 64 * 64 * 2;
constexpr int kStages = 3;
constexpr int kStageBytes = 4 * kHalf;  // two K blocks: [A k0 | A k1 | B k0 | B k1]
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;
constexpr int kGemmSmem = kStages * kStageBytes + 256 + 1024 /*align*/;
static_assert(kGemmSmem <= 227 * 1024, "shared memory budget");
// Products are cut for 152 SMs wherever they run: the workspace's size is known without a GPU, the order of sums goes by the
// sizes alone.
constexpr int kRuleSms = 152;
constexpr int kMaxSplit = 16;
constexpr int kLeastStages = 4;       // of a part of a split reduction

enum Product : int { kFwd = 0, kDx = 1, kDw = 2, kBoth = 3 };  // kBoth: dx and dW in one launch

struct Ends {  // what an epilogue adds and writes
  const uint16_t *bias, *res;
  uint16_t *y, *z;
  int act;
  bool sectors;  // every row of res, y and z starts on 32 bytes
};
struct ProductArgs {
  int M, N, K;    // rows, columns, reduction
  int nm, nn;     // tiles along both
  int full;       // tiles that are computed whole; the others in `split` parts
  int split;
  int units;      // tiles and parts in all
  int cluster;    // blocks that share a tile's reduction, or 1
  float *part;    // the parts' sums (part_at)
  Ends e;
  int32_t *status;
  bool first;     // of the call's kernels: clears the status word
  const float *sums;  // kBoth: dbias' partial rows, which blocks behind the tiles add up
  int sum_rows;
  float *dbias;
};

// The k-th unit of work: its tile, and its stages of the reduction.
struct Unit {
  int m0, n0, ks0, ks1, part;  // part: index of the sums it leaves, or -1
};
template <int CG>
__device__ __forceinline__ Unit unit_of(int u, const ProductArgs &p, int nstage) {
  constexpr int TS = tile_size(CG);
  Unit t;
  int tile = u;
  t.ks0 = 0;
  t.ks1 = nstage;
  t.part = -1;
  if (u >= p.full && p.split > 1) {
    t.part = u - p.full;
    const int s = t.part % p.split;
    tile = p.full + t.part / p.split;
    t.ks0 = static_cast<int>(static_cast<int64_t>(nstage) * s / p.split);
    t.ks1 = static_cast<int>(static_cast<int64_t>(nstage) * (s + 1) / p.split);
  }
  const int mt = tile / p.nn;
  t.m0 = mt * TS;
  t.n0 = (tile - mt * p.nn) * TS;
  return t;
}

// Where a lane's sums of 32 rows x 32 columns of a part lie (row: the lane): eight times four columns, 128 floats apart, so
// that the lanes' 16 bytes are side by side.
template <int CG>
__device__ __forceinline__ int64_t part_at(int part, int row0, int col0) {
  constexpr int TS = tile_size(CG);
  return (static_cast<int64_t>(part) * (TS / 32) + row0 / 32) * TS * 32 + col0 * 32 + (threadIdx.x & 31) * 4;
}

// A lane's 32 columns of a row (64 bytes, eight columns a piece), of which ncols (a multiple of
// eight) exist.
__device__ __forceinline__ void ld_row(const uint16_t *p, int ncols, bool sectors, uint4 (&w)[4]) {
  if (sectors) {
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      if (8 * i < ncols)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w), "=r"(w[i + 1].x), "=r"(w[i + 1].y),
                       "=r"(w[i + 1].z), "=r"(w[i + 1].w)
                     : "l"(p + 8 * i)
                     : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (8 * i < ncols) w[i] = *reinterpret_cast<const uint4 *>(p + 8 * i);
  }
}
__device__ __forceinline__ void st_row(uint16_t *p, int ncols, bool sectors, const float (&v)[32]) {
  uint4 w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    w[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                      pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
  if (sectors) {
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      if (8 * i < ncols)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 8 * i), "r"(w[i].x), "r"(w[i].y),
                     "r"(w[i].z), "r"(w[i].w), "r"(w[i + 1].x), "r"(w[i + 1].y), "r"(w[i + 1].z), "r"(w[i + 1].w)
                     : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (8 * i < ncols) *reinterpret_cast<uint4 *>(p + 8 * i) = w[i];
  }
}
__device__ __forceinline__ void unpack_row(const uint4 (&w)[4], float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t x[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[8 * q + 2 * h] = bf16_lo(x[h]);
      v[8 * q + 2 * h + 1] = bf16_hi(x[h]);
    }
  }
}

// ---------------------------------------------------------------- activations

// The sigmoid by the part's exponential and reciprocal: within a few fp32 ulp, far below the
// bf16 rounding of what it enters.
__device__ __forceinline__ float sigmoid_(float a) { return __fdividef(1.f, 1.f + __expf(-a)); }
constexpr float kGelu1 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.071354816272600252f; // times 0.044715
// Maximum and minimum that are NaN where one of the two is: a NaN of z is one of y and of dz.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Past 20 gelu's sigmoid is 0 or 1 to the last bit, and its slope's polynomial would overflow first.
__device__ __forceinline__ float gelu_clamp(float z) { return min_nan(max_nan(z, -20.f), 20.f); }
__device__ __forceinline__ float gelu_arg(float z) {
  const float c = gelu_clamp(z);
  return c * fmaf(kGelu3 * c, c, kGelu1);
}
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return max_nan(z, 0.f);
    case MOE_ACT_SILU: return z * sigmoid_(z);
    case MOE_ACT_GELU: return z * sigmoid_(gelu_arg(z));
    default: return z;
  }
}
__device__ __forceinline__ float slope(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z > 0.f ? 1.f : max_nan(z, 0.f);  // 0, or NaN
    case MOE_ACT_SILU: {
      const float s = sigmoid_(z);
      return fmaf(z * s, 1.f - s, s);
    }
    case MOE_ACT_GELU: {
      const float c = gelu_clamp(z), s = sigmoid_(gelu_arg(z));
      return fmaf(c * s * (1.f - s), fmaf(3.f * kGelu3 * c, c, kGelu1), s);
    }
    default: return 1.f;
  }
}

// A row's 32 columns from c0 on: bias, activation, residual, and what is stored.  res: the residual's
// 64 bytes where there is one.
template <int KIND>
__device__ __forceinline__ void finish_row(float (&v)[32], const Ends &e, const uint4 (&res)[4], int64_t at, int c0, int ncols) {
  if constexpr (KIND == kFwd) {
    if (e.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (8 * q < ncols) {
          const uint4 b = __ldg(reinterpret_cast<const uint4 *>(e.bias + c0 + 8 * q));
          const uint32_t x[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            v[8 * q + 2 * h] += bf16_lo(x[h]);
            v[8 * q + 2 * h + 1] += bf16_hi(x[h]);
          }
        }
      }
    }
    if (e.z) st_row(e.z + at, ncols, e.sectors, v);
    if (e.act == MOE_ACT_RELU) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate(v[i], MOE_ACT_RELU);
    } else if (e.act == MOE_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate(v[i], MOE_ACT_SILU);
    } else if (e.act == MOE_ACT_GELU) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = activate(v[i], MOE_ACT_GELU);
    }
    if (e.res) {
      float r[32];
      unpack_row(res, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += r[i];
    }
  }
  st_row(e.y + at, ncols, e.sectors, v);
}

// A float, or four, of a block of the cluster.
__device__ __forceinline__ float ld_peer(const float *p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_smem_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer4(const float *p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_smem_addr(p, rank))
               : "memory");
  return v;
}

// ---------------------------------------------------------------- the product

template <int CG>
__device__ __forceinline__ void load_operand(bool mn, uint8_t *dst, const CUtensorMap *map, uint64_t *bar, uint32_t bar0, int k0,
                                             int r0) {
  auto load = [&](uint8_t *to, int x, int y) {
    if constexpr (CG == 2)
      tma_load_2d_pair(to, map, bar0, x, y);
    else
      tma_load_2d(to, map, bar, x, y);
  };
  if (mn) {
    load(dst, r0, k0);
    load(dst + kBox, r0 + 64, k0);
  } else {
    load(dst, k0, r0);
  }
}
// Descriptor of the j-th 16 of K of a block at shared address s.
__device__ __forceinline__ uint64_t operand_desc(uint32_t s, int j, bool mn) {
  return mn ? smem_desc_sw128(s + j * 2048, kBox, 1024) : smem_desc_sw128(s + j * 32, 16, 1024);
}

// dbias of 32 columns: a warp each for every WARPS-th partial row.  s_sum: [WARPS][32]
template <int WARPS>
__device__ __forceinline__ void add_sums(const float *sums, int rows, int N, float *dbias, int columns, float *s_sum) {
  const int lane = threadIdx.x & 31, c = columns * 32 + lane, w = threadIdx.x >> 5;
  float s = 0.f;
  if (c < N) {
#pragma unroll 8
    for (int i = w; i < rows; i += WARPS) s += __ldcg(sums + static_cast<int64_t>(i) * N + c);
  }
  s_sum[w * 32 + lane] = s;
  __syncthreads();
  if (w || c >= N) return;
#pragma unroll
  for (int i = 1; i < WARPS; ++i) s += s_sum[i * 32 + lane];
  dbias[c] = s;
}

template <int KIND, int CG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    linear_product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                          const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmA2,
                          const __grid_constant__ CUtensorMap tmB2, const ProductArgs p1, const ProductArgs p2) {
  constexpr int TS = tile_size(CG);
  constexpr uint32_t kTmemCols = 2 * TS;
  // kBoth: a tile per block, those of dx first; behind them 32 columns of dbias each
  if constexpr (KIND == kBoth) {
    const int columns = static_cast<int>(blockIdx.x) - p1.units - p2.units;
    if (columns >= 0) {
      extern __shared__ float s_sum[];
      griddep_wait();
      griddep_launch_dependents();
      add_sums<kGemmThreads / 32>(p1.sums, p1.sum_rows, p2.N, p1.dbias, columns, s_sum);
      return;
    }
  }
  const bool second = KIND == kBoth && static_cast<int>(blockIdx.x) >= p1.units;
  const ProductArgs &p = second ? p2 : p1;
  const bool amn = KIND == kBoth ? second : KIND == kDw, bmn = KIND == kBoth ? second : KIND != kDx;
  const CUtensorMap *const mA = second ? &tmA2 : &tmA, *const mB = second ? &tmB2 : &tmB;
  constexpr int kChunks = TS / 64;  // 32-column chunks of a warp's half of the columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);  // [kStages] CTA 0: both CTAs' copies
  uint64_t *empty = full + kStages;      // [kStages] the pair's MMAs are done with the stage
  uint64_t *tfull = empty + kStages;     // [2] accumulator ready (both CTAs)
  uint64_t *tempty = tfull + 2;          // [2] CTA 0: both CTAs' epilogues done
  uint64_t *drain = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const int parts = CG == 1 ? p.cluster : 1, part = blockIdx.x % parts;
  const int group = blockIdx.x / CG / parts - (second ? p1.units : 0), ngroups = gridDim.x / CG / parts;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], CG * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(mA);
    if (!amn) tma_prefetch_desc(&tmA32);
    tma_prefetch_desc(mB);
  }
  if (warp == 1) {
    if constexpr (CG == 2)
      tmem_alloc_pair(tmem_slot, kTmemCols);
    else
      tmem_alloc(tmem_slot, kTmemCols);
  }
  const int nkb = (p.K + BK - 1) / BK, nstage = (nkb + 1) / 2;
  auto unit = [&](int u) {
    Unit t = unit_of<CG>(u, p, nstage);
    if (CG == 1 && parts > 1) {
      t.ks0 = nstage * part / parts;
      t.ks1 = nstage * (part + 1) / parts;
    }
    return t;
  };
  const Unit first = unit(group);
  asm volatile("" ::"r"(first.m0), "r"(first.n0), "r"(first.ks0), "r"(first.ks1), "r"(first.part), "r"(nkb));  // here, not later
  griddep_wait();  // the set-up above overlaps the previous kernel's end; its outputs are read below
  // (a wait that runs out takes two seconds: no block flags one before this)
  if (p1.first && blockIdx.x == 0 && threadIdx.x == 0) *p1.status = 0;
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // both CTAs' barriers initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = CG == 2 ? peer_smem_addr(&full[0], 0) : 0;
      int stage = 0;
      uint32_t phase = 0, armed = 0, arm_par = 0;
      bool ok = true;
      for (int u = group; u < p.units && ok; u += ngroups) {
        const Unit t = u == group ? first : unit(u);
        // Rows of A contiguous along K: where they end inside a CTA's 128, only the boxes of 32 that hold some (the MMA
        // reads what was there before in the others, whose sums are never stored).  With whole boxes a single row took
        // 17.4 us for 4096 x 4096.
        auto boxes = [&](int r) { return amn ? 4 : max(0, min(4, (p.M - (t.m0 + BM * r) + 31) / 32)); };
        const int mine = boxes(rank);
        const uint32_t bytes = CG * kStageBytes - (CG * 4 - boxes(0) - (CG == 2 ? boxes(1) : 0)) * (2 * 32 * BK * 2);
        for (int ks = t.ks0; ks < t.ks1; ++ks) {
          if (!(armed >> stage & 1)) {  // its first use
          } else if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t *sa = smem + stage * kStageBytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], bytes);  // the group's
          // a K block past the end is zero fill, and no MMA reads it
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k0 = (ks * 2 + h) * BK;
            if (mine == 4)
              load_operand<CG>(amn, sa + h * kHalf, mA, &full[stage], full0 + 8u * stage, k0, t.m0 + BM * rank);
            else
              for (int b = 0; b < mine; ++b)
                load_operand<CG>(false, sa + h * kHalf + b * (32 * BK * 2), &tmA32, &full[stage], full0 + 8u * stage, k0,
                                 t.m0 + BM * rank + 32 * b);
            load_operand<CG>(bmn, sa + (2 + h) * kHalf, mB, &full[stage], full0 + 8u * stage, k0, t.n0 + BM * rank);
          }
          armed |= 1u << stage;
          arm_par = (arm_par & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      griddep_launch_dependents();  // all loads issued: the next kernel may be launched
      if (*abort_flag && rank == 0) {  // let the pair's copies land before exit
        for (int s = 0; s < kStages; ++s) {
          if (!((armed >> s) & 1u)) continue;
          for (int i = 0; i < (1 << 22) && !mbar_try_wait(&full[s], (arm_par >> s) & 1u); ++i) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
        if constexpr (CG == 2)
          tc_mma_f16_pair(d, a, b, idesc, acc);
        else
          tc_mma_f16_one(d, a, b, idesc, acc);
      };
      auto commit = [](uint64_t *bar) {
        if constexpr (CG == 2)
          tc_commit_pair(bar);
        else
          tc_commit(bar);
      };
      const uint32_t idesc = idesc_bf16(TS, TS, amn, bmn);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = group; u < p.units && ok; u += ngroups, ++it) {
        const Unit t = u == group ? first : unit(u);
        const int buf = it & 1;
        if (!mbar_wait(&tempty[buf], ((it >> 1) & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * TS;
        for (int ks = t.ks0; ks < t.ks1; ++ks) {
          if (!mbar_wait(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ab = smem_addr(smem + stage * kStageBytes), bb = ab + 2 * kHalf;
          const int nblk = min(2, nkb - ks * 2);  // K blocks inside K
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h < nblk) {
#pragma unroll
              for (int j = 0; j < BK / 16; ++j)
                mma(d, operand_desc(ab + h * kHalf, j, amn), operand_desc(bb + h * kHalf, j, bmn), idesc,
                    (ks != t.ks0 || (h | j) != 0) ? 1u : 0u);
            }
          }
          commit(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        commit(&tfull[buf]);
      }
      if (*abort_flag) {  // wait for the pair's MMAs before TMEM is freed
        commit(drain);
        for (int i = 0; i < (1 << 22) && !mbar_try_wait(drain, 0); ++i) {
        }
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;               // TMEM lane quarter
    const int half = (warp - 2) >> 2;     // column half
    const uint32_t tempty0 = CG == 2 ? peer_smem_addr(&tempty[0], 0) : 0;
    int it = 0;
    for (int u = group; u < p.units; u += ngroups, ++it) {
      const Unit t = u == group ? first : unit(u);
      const int buf = it & 1, row = t.m0 + BM * rank + q * 32 + lane, cols0 = t.n0 + half * (TS / 2);
      const int64_t row_at = static_cast<int64_t>(row) * p.N;
      uint4 res[KIND == kFwd ? kChunks : 1][4];
      uint32_t warm = 0;
      if constexpr (KIND == kFwd) {  // while the product runs: the residual, and the bias into the L1
        if (p.e.bias && lane < TS / 16 && cols0 + 8 * lane < p.N)
          warm = __ldg(reinterpret_cast<const uint32_t *>(p.e.bias + cols0 + 8 * lane));
        if (p.e.res && t.part < 0 && parts == 1 && row < p.M) {
#pragma unroll
          for (int j = 0; j < kChunks; ++j)
            if (cols0 + 32 * j < p.N) ld_row(p.e.res + row_at + cols0 + 32 * j, p.N - (cols0 + 32 * j), p.e.sectors, res[j]);
        }
      }
      if (!wait_lane0(&tfull[buf], (it >> 1) & 1, abort_flag)) break;
      __syncwarp();
      asm volatile("" ::"r"(warm));
      tc_fence_after();
      const uint32_t tb = tmem_base + buf * TS + (static_cast<uint32_t>(q * 32) << 16) + half * (TS / 2);
#pragma unroll(KIND == kFwd ? kChunks : 1)
      for (int j = 0; j < kChunks; ++j) {
        const int c0 = cols0 + 32 * j;
        if (c0 >= p.N) break;
        uint32_t acc[32];
        tmem_ld32(tb + 32 * j, acc);
        tmem_ld_wait();
        if (t.part >= 0 || parts > 1) {  // sums of a part, rows and columns past the ends among them
          // (a cluster's stay in shared memory: all that was loaded there has been read)
          float *to = (parts > 1 ? reinterpret_cast<float *>(smem) : p.part) +
                      part_at<CG>(parts > 1 ? 0 : t.part, BM * rank + q * 32, half * (TS / 2) + 32 * j);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(to + i * 128) = make_uint4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
        } else if (row < p.M) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(acc[i]);
          finish_row<KIND>(v, p.e, res[KIND == kFwd ? j : 0], row_at + c0, c0, min(32, p.N - c0));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(tempty0 + 8u * buf);
        else
          mbar_arrive(&tempty[buf]);
      }
    }
  }

  if (CG == 1 && parts > 1) {  // a tile's 16 squares of 32 x 32 among the cluster's blocks, a warp each
    const int square = 16 / parts * part + warp - 2, at0 = square / 4 * 32, at1 = square % 4 * 32;
    const int row = first.m0 + at0 + lane, col = first.n0 + at1;
    const bool mine = warp >= 2 && warp - 2 < 16 / parts && row < p.M && col < p.N;
    const int64_t at = static_cast<int64_t>(row) * p.N + col;
    uint4 res[4];
    if (KIND == kFwd && mine && p.e.res) ld_row(p.e.res + at, p.N - col, p.e.sectors, res);
    __syncwarp();
    cluster_sync();
    if (mine) {
      const float *from = reinterpret_cast<float *>(smem) + part_at<CG>(0, at0, at1);
      float v[32] = {};
      for (int r = 0; r < parts; r += 2) {
        float4 a[2][8];
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i / 8][i % 8] = ld_peer4(from + i % 8 * 128, r + i / 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 x = a[i / 8][i % 8];
          float *const to = v + i % 8 * 4;
          to[0] += x.x, to[1] += x.y, to[2] += x.z, to[3] += x.w;
        }
      }
      finish_row<KIND>(v, p.e, res, at, col, min(32, p.N - col));
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) flag_status(p.status, kDevWaitTimeout);
  // a pair is done with each other's barriers and TMEM, a cluster with each other's sums
  if (CG == 2 || parts > 1) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
  }
}

// The tiles in parts: their sums in the order of the parts, then the epilogue.  A warp has 32 rows x 32 columns.
constexpr int kFinishThreads = 128;
template <int KIND, int CG>
__global__ void __launch_bounds__(kFinishThreads) linear_finish_kernel(const ProductArgs p) {
  constexpr int TS = tile_size(CG), kSide = TS / 32;
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kFinishThreads / 32) + (threadIdx.x >> 5);
  const int r = static_cast<int>(w / (kSide * kSide)), in = static_cast<int>(w % (kSide * kSide)), tile = p.full + r;
  if (tile >= p.nm * p.nn) return;
  const int mt = tile / p.nn, r0 = in / kSide * 32, c0 = in % kSide * 32;
  const int row0 = mt * TS + r0, row = row0 + (threadIdx.x & 31), col = (tile - mt * p.nn) * TS + c0;
  if (row0 >= p.M || col >= p.N) return;
  const int64_t at = static_cast<int64_t>(row) * p.N + col;
  uint4 res[4];
  if (KIND == kFwd && p.e.res && row < p.M) ld_row(p.e.res + at, p.N - col, p.e.sectors, res);
  float v[32] = {};
  constexpr int kBatch = 4;  // parts under way at once
  for (int s0 = 0; s0 < p.split; s0 += kBatch) {
    float4 a[kBatch][8];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (s0 + b < p.split) {
        const float *from = p.part + part_at<CG>(r * p.split + s0 + b, r0, c0);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[b][i] = __ldcg(reinterpret_cast<const float4 *>(from + i * 128));
      }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (s0 + b < p.split)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[4 * i] += a[b][i].x, v[4 * i + 1] += a[b][i].y, v[4 * i + 2] += a[b][i].z, v[4 * i + 3] += a[b][i].w;
  }
  if (row < p.M) finish_row<KIND>(v, p.e, res, at, col, min(32, p.N - col));
}

// a b + c of two floats, one instruction for both.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n.reg .b64 a, b, c;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 c, a, b, c;\nmov.b64 {%0, %1}, c;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// ---------------------------------------------------------------- a few tokens
//
// y of at most TM tokens, on the CUDA cores: a pass over W, which is all that it has to read.  A thread takes 8 columns of 8
// rows of W at a time, CT threads side by side a block's columns; a cluster's blocks share the rows, as many as are one wave.
// Sums over the lanes, the warps and the cluster's blocks, in that order, in fp32.
// Bound by W's bytes, and for small W by the launch: one token and W from HBM, 4096 x 4096 8.4 us, 60% of the copy rate, 7168 x
// 18432 43.4, 91%, 1024 x 1024 2.8; a library's product 8.6, 40.6, 2.8, the tensor cores' tiles 12.5, 46.5, 6.9.

constexpr int kRowThreads = 256;
// For up to two tokens, and up to eight while the products take no longer than the tiles' part sums.  Here and in tiles: 8 x
// 1024 x 1024 4.4 us and 6.9, 8 x 4096 x 1536 8.9 and 9.5, 8 x 4096 x 4096 13.1 and 12.4, 4 x 4096 x 4096 10.5 and 12.5,
// 4 x 7168 x 18432 48.9 and 46.2, 2 x 7168 x 18432 46.4 and 46.0.
bool few_rows(int64_t T, int64_t K, int64_t N) { return T <= 2 || (T <= 8 && T * K * N < 1 << 27); }
// 16 columns a block up to here, else 64: one token, 16384 x 64 4.4 and 5.7 us, 1024 x 1024 2.8 and 3.0, 4096 x 1536 6.8 and 5.7.
constexpr int kNarrow = 1024;
constexpr int rows_per_sm(int tm) { return tm == 1 ? 4 : tm == 2 ? 3 : 2; }  // blocks an SM holds
struct RowArgs {
  const uint16_t *x, *W;
  Ends e;
  int T, K, N;
  int parts, per;  // blocks that share a run of columns, and their 8 rows each
  int32_t *status;
};
template <int TM, int CT>
__global__ void __launch_bounds__(kRowThreads, rows_per_sm(TM)) linear_rows_kernel(const RowArgs a) {
  constexpr int kCols = 8 * CT, kGroups = kRowThreads / CT, kWarps = kRowThreads / 32;
  __shared__ float s_sum[kWarps][TM][kCols];
  __shared__ float s_out[TM * kCols];
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  const int part = blockIdx.x % a.parts, c0 = blockIdx.x / a.parts * kCols, c = c0 + threadIdx.x % CT * 8;
  float2 sum[TM][4] = {};
  if (c < a.N) {
    const int end = min(a.K / 8, (part + 1) * a.per);
    for (int u = part * a.per + threadIdx.x / CT; u < end; u += kGroups) {
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(a.W + (8 * static_cast<int64_t>(u) + i) * a.N + c));
      constexpr int kAt = TM < 4 ? TM : 4;  // tokens whose x is held at once
#pragma unroll
      for (int t0 = 0; t0 < TM; t0 += kAt) {
        uint4 xv[kAt];
#pragma unroll
        for (int t = 0; t < kAt; ++t)
          xv[t] = t0 + t < a.T ? __ldg(reinterpret_cast<const uint4 *>(a.x + static_cast<int64_t>(t0 + t) * a.K + 8 * u)) : uint4{};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t wi[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          float2 wf[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) wf[h] = make_float2(bf16_lo(wi[h]), bf16_hi(wi[h]));
#pragma unroll
          for (int t = 0; t < kAt; ++t) {
            const uint32_t two = i < 2 ? xv[t].x : i < 4 ? xv[t].y : i < 6 ? xv[t].z : xv[t].w;
            const float xi = i & 1 ? bf16_hi(two) : bf16_lo(two);
#pragma unroll
            for (int h = 0; h < 4; ++h) sum[t0 + t][h] = fma2(make_float2(xi, xi), wf[h], sum[t0 + t][h]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TM; ++t) {
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      float v = h & 1 ? sum[t][h / 2].y : sum[t][h / 2].x;
#pragma unroll
      for (int d = CT; d < 32; d *= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
      if ((threadIdx.x & 31) < CT) s_sum[threadIdx.x >> 5][t][(threadIdx.x & 31) * 8 + h] = v;
    }
  }
  __syncthreads();
  const int n = a.T * kCols;
  for (int i = threadIdx.x; i < n; i += kRowThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_sum[w][i / kCols][i % kCols];
    s_out[i] = v;
  }
  if (a.parts > 1)
    cluster_sync();
  else
    __syncthreads();
  const int mine = (n + a.parts - 1) / a.parts;
  for (int i = part * mine + threadIdx.x; i < min(n, (part + 1) * mine); i += kRowThreads) {
    const int col = c0 + i % kCols;
    if (col >= a.N) continue;
    const int64_t at = static_cast<int64_t>(i / kCols) * a.N + col;
    float v = 0.f;
    if (a.parts > 1)
      for (int r = 0; r < a.parts; ++r) v += ld_peer(&s_out[i], r);
    else
      v = s_out[i];
    if (a.e.bias) v += bf16_lo(a.e.bias[col]);
    if (a.e.z) a.e.z[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
    v = activate(v, a.e.act);
    if (a.e.res) v += bf16_lo(a.e.res[at]);
    a.e.y[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
  }
  if (a.parts > 1) cluster_sync();  // before a block leaves that others read
}

// ---------------------------------------------------------------- dz and dbias
//
// dz = dy act'(z) in bf16 (where there is an activation), and the column sums of it unrounded.  A block
// takes 64 columns and every `split`-th run of rows: 8 threads a row, 32 rows at once; its sums over
// those go to a partial row, which the second kernel adds in order.
// Bound by HBM, with its loads in flight: 16384 x 1536 and 16384 x 4096 with silu 26.7 and 64.4 us with the second kernel, 84%
// and 93% of the copy rate.  Three rows ahead at four blocks an SM, which are one wave; with one thread a column in the second
// kernel 28.8 and 65.9, four rows ahead at three blocks an SM 28.7 and 66.4, two at four 29.6 and 69.8; more blocks than fit
// at once 45.0 and 106.5.

constexpr int kDzThreads = 256, kDzCols = 64, kDzRows = kDzThreads / 8, kDzAhead = 3, kDzPerSm = 4;
// how many blocks share a run of 64 columns: one wave, of at least kDzAhead rows a thread
int dz_split(int T, int N) {
  const int cols = (N + kDzCols - 1) / kDzCols, rounds = (T + kDzRows * kDzAhead - 1) / (kDzRows * kDzAhead);
  return std::max(1, std::min(kDzPerSm * kRuleSms / cols, rounds));
}
struct DzArgs {
  const uint16_t *dy, *z;
  uint16_t *dz;    // null: no activation, dy itself; or no product that reads it
  float *part;     // [split][N], or null: no bias
  float *dbias;
  int T, N, split;
  int32_t *status;
};
template <int ACT>
__global__ void __launch_bounds__(kDzThreads, kDzPerSm) linear_dz_kernel(const DzArgs a) {
  __shared__ float s_sum[kDzRows / 4][kDzCols];
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
  const int c = blockIdx.x * kDzCols + (threadIdx.x & 7) * 8;
  const int step = kDzRows * a.split;
  float sum[8] = {};
  if (c < a.N) {
    constexpr int kAhead = ACT != MOE_ACT_NONE ? kDzAhead : 2 * kDzAhead;
    for (int64_t t0 = blockIdx.y * kDzRows + (threadIdx.x >> 3); t0 < a.T; t0 += static_cast<int64_t>(step) * kAhead) {
      uint4 dy[kAhead], z[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t t = t0 + static_cast<int64_t>(i) * step;
        if (t < a.T) {
          dy[i] = __ldg(reinterpret_cast<const uint4 *>(a.dy + t * a.N + c));
          if (ACT != MOE_ACT_NONE) z[i] = __ldg(reinterpret_cast<const uint4 *>(a.z + t * a.N + c));
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t t = t0 + static_cast<int64_t>(i) * step;
        if (t >= a.T) break;
        const uint32_t y[4] = {dy[i].x, dy[i].y, dy[i].z, dy[i].w};
        float v[8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          v[2 * h] = bf16_lo(y[h]);
          v[2 * h + 1] = bf16_hi(y[h]);
        }
        if constexpr (ACT != MOE_ACT_NONE) {
          const uint32_t x[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            v[2 * h] *= slope(bf16_lo(x[h]), ACT);
            v[2 * h + 1] *= slope(bf16_hi(x[h]), ACT);
          }
          if (a.dz)
            *reinterpret_cast<uint4 *>(a.dz + t * a.N + c) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
#pragma unroll
        for (int h = 0; h < 8; ++h) sum[h] += v[h];
      }
    }
  }
  if (!a.part) return;
  // over the four rows of a warp, then over the warps
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 8);
    sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 16);
  }
  if ((threadIdx.x & 31) < 8) {
#pragma unroll
    for (int h = 0; h < 8; ++h) s_sum[threadIdx.x >> 5][(threadIdx.x & 7) * 8 + h] = sum[h];
  }
  __syncthreads();
  const int col = blockIdx.x * kDzCols + threadIdx.x;
  if (threadIdx.x < kDzCols && col < a.N) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kDzThreads / 32; ++w) s += s_sum[w][threadIdx.x];
    (a.split == 1 ? a.dbias : a.part + static_cast<int64_t>(blockIdx.y) * a.N)[col] = s;
  }
}
__global__ void __launch_bounds__(kDzThreads) linear_dbias_kernel(const float *part, int split, int N, float *dbias) {
  __shared__ float s_sum[kDzThreads];
  griddep_wait();  // the previous kernel in the stream has completed
  griddep_launch_dependents();
  add_sums<kDzThreads / 32>(part, split, N, dbias, blockIdx.x, s_sum);
}

// ---------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A row-major bf16 matrix [rows, inner]: boxes of 64 x box_rows, 128-byte swizzle, zeros outside.
bool map2(CUtensorMap *m, const void *ptr, int inner, int rows, int box_rows) {
  auto fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(inner) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product is cut: the whole tiles, and the parts of those that are left.  By the time in us that each way takes
// apart from what they share: a round of tiles 0.58 us a stage of 128 and 1.4 for its ends with pairs, 0.46 and 0.8 with
// single CTAs; parts cost another 5, for their sums and the second kernel.  Measured, single whole, single in parts, pairs
// whole, pairs in parts: 1024 x 1024 x 1024 7.6, 10.3, 10.1, 11.6; 512 x 2048 x 768 11.1, 9.6, 14.2, 11.7; 4096 x 1536 x 1536 22.7,
// 22.5, 20.4, 21.2; 16 x 4096 x 4096 18.4, 11.9, 22.0, 14.9; 2048 x 4096 x 4096 67.4, 64.0, 42.4, 42.2.
// Or a cluster of 2, 4 or 8 single CTAs shares each tile's reduction and adds its sums over shared memory, for another 1.5 us,
// where all of them run at once (as the part's SMs lie, 76, 36 and 15 such clusters do): 16 x 4096 x 4096 9.4 us and 11.3
// without, 777 x 1000 x 520 8.9 and 10.7, 1100 x 2048 x 1024 11.4 and 14.9, 16 x 4096 x 1536 7.8 and 9.1; 16 clusters of 8,
// which are two rounds, 16.5 and 8.5 (256 x 1024 x 1024).
struct Cut {
  int cg, nm, nn, full, split, units, cluster;
  double cost;
};
Cut cut_with(int64_t M, int64_t N, int64_t K, int cg, bool parts) {
  const int ts = tile_size(cg), groups = kRuleSms / cg;
  Cut c;
  c.cg = cg;
  c.nm = static_cast<int>((M + ts - 1) / ts);
  c.nn = static_cast<int>((N + ts - 1) / ts);
  const int64_t tiles = static_cast<int64_t>(c.nm) * c.nn;
  const int nstage = static_cast<int>((K + 2 * BK - 1) / (2 * BK));
  const int left = static_cast<int>(tiles % groups);
  c.split = 1;
  if (left && parts) c.split = std::max(1, std::min({groups / left, kMaxSplit, nstage / kLeastStages}));
  c.full = static_cast<int>(c.split > 1 ? tiles - left : tiles);
  c.units = static_cast<int>(c.split > 1 ? c.full + left * c.split : tiles);
  const int64_t rounds = c.split > 1 ? c.full / groups : (tiles + groups - 1) / groups;
  const double stage = cg == 2 ? 0.58 : 0.46, ends = cg == 2 ? 1.4 : 0.8;
  c.cluster = 1;
  c.cost = rounds * (nstage * stage + ends);
  if (c.split > 1) c.cost += (nstage + c.split - 1) / c.split * stage + ends + 5;
  return c;
}
Cut cut_of(int64_t M, int64_t N, int64_t K) {
  Cut best = cut_with(M, N, K, 2, false);
  for (int way = 1; way < 4; ++way) {
    const Cut c = cut_with(M, N, K, way & 1 ? 1 : 2, way > 1);
    if (c.cost < best.cost) best = c;
  }
  for (int blocks = 2; blocks <= 8; blocks *= 2) {
    Cut c = cut_with(M, N, K, 1, false);
    const int nstage = static_cast<int>((K + 2 * BK - 1) / (2 * BK));
    if (c.units > (blocks == 2 ? 76 : blocks == 4 ? 36 : 15) || nstage < blocks) break;
    c.cluster = blocks;
    c.cost = (nstage + blocks - 1) / blocks * 0.46 + 0.8 + 1.5;
    if (c.cost < best.cost) best = c;
  }
  return best;
}
// The sums that the parts of a cut leave: part_at's, 16 bytes of each lane.  At most a round of pairs, 20 MB; most shapes
// are not cut into parts.
size_t part_bytes(const Cut &c) {
  return static_cast<size_t>(c.units - c.full) * tile_size(c.cg) * tile_size(c.cg) * 4;
}

// The kernel's shared-memory opt-in, and how many groups of CTAs fit at once; once per device.
template <int KIND, int CG>
cudaError_t groups_of(int sms, int *groups) {
  static DeviceOnce once;
  auto kernel = linear_product_kernel<KIND, CG>;
  return once.get(
      [&](int *out) {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
        if (r != cudaSuccess) return r;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = CG;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(sms / CG * CG);
        q.blockDim = dim3(kGemmThreads);
        q.dynamicSmemBytes = kGemmSmem;
        q.attrs = &attr;
        q.numAttrs = 1;
        int n = 0;
        r = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
        if (r != cudaSuccess) return r;
        if (n < 1) return cudaErrorInvalidConfiguration;
        *out = n < sms / CG ? n : sms / CG;
        return cudaSuccess;
      },
      groups);
}

// One product [M,N] over K of a (its rows contiguous along K, or along M for dW) and b: its maps and arguments.
struct Operands {
  CUtensorMap a, a32, b;
  ProductArgs p;
};
bool operands(Operands *o, int kind, const void *a, const void *b, int M, int N, int K, const Cut &c, const Ends &ends,
              float *part, int32_t *status, bool first) {
  if (!(kind == kDw ? map2(&o->a, a, M, K, 64) : map2(&o->a, a, K, M, 128)) ||
      !(kind == kDw ? map2(&o->a32, a, M, K, 64) : map2(&o->a32, a, K, M, 32)) ||
      !(kind == kDx ? map2(&o->b, b, K, N, 128) : map2(&o->b, b, N, K, 64)))
    return false;
  ProductArgs p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.nm = c.nm;
  p.nn = c.nn;
  p.full = c.full;
  p.split = c.split;
  p.units = c.units;
  p.cluster = c.cluster;
  p.part = part;
  p.e = ends;
  auto al32 = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 31) == 0; };
  p.e.sectors = N % 16 == 0 && al32(ends.res) && al32(ends.y) && al32(ends.z);
  p.status = status;
  p.first = first;
  o->p = p;
  return true;
}

template <int KIND, int CG>
cudaError_t launch_cut(const Operands &o, const Cut &c, int sms, cudaStream_t s) {
  int groups = 0;
  cudaError_t e = groups_of<KIND, CG>(sms, &groups);
  if (e != cudaSuccess) return e;
  if (c.cluster > 1)
    return launch_pdl(linear_product_kernel<KIND, CG>, dim3(static_cast<unsigned>(c.units * c.cluster)), dim3(kGemmThreads),
                      kGemmSmem, s, c.cluster, o.a, o.a32, o.b, o.a, o.b, o.p, o.p);
  e = launch_pdl(linear_product_kernel<KIND, CG>, dim3(static_cast<unsigned>(CG * std::min(c.units, groups))),
                 dim3(kGemmThreads), kGemmSmem, s, CG, o.a, o.a32, o.b, o.a, o.b, o.p, o.p);
  if (e != cudaSuccess || c.split == 1) return e;
  constexpr int TS = tile_size(CG);
  const int64_t threads = static_cast<int64_t>(c.nm * c.nn - c.full) * (TS / 32) * (TS / 32) * 32;
  return launch_pdl(linear_finish_kernel<KIND, CG>, dim3(static_cast<unsigned>((threads + kFinishThreads - 1) / kFinishThreads)),
                    dim3(kFinishThreads), 0, s, 1, o.p);
}

template <int KIND>
moe_status product(const char *label, const Cut &c, const void *a, const void *b, int M, int N, int K, const Ends &ends,
                   float *part, int32_t *status, bool first, int sms, cudaStream_t s) {
  Operands o;
  if (!operands(&o, KIND, a, b, M, N, K, c, ends, part, status, first)) return MOE_ERR_CUDA;
  return timed(label, s, [&] { return c.cg == 2 ? launch_cut<KIND, 2>(o, c, sms, s) : launch_cut<KIND, 1>(o, c, sms, s); });
}

// dx and dW in one launch (*done), where their tiles of single CTAs are one round together and that is not longer than the
// two one after the other: tokens, in, out in one and in two launches: 16 x 1024 x 1024 8.4 us and 12.4; 777 x 1000 x 520
// 13.3 and 19.8; 2048 x 512 x 512 15.7 and 16.5; by the rule in two: 3000 x 384 x 384 20.9 and 18.0, 8192 x 128 x 128 42.2
// and 18.0 (their dW is cut along the tokens).
// apart: what the two take one after the other.  *sums_left: dbias' partial rows (sums, rows) are still to be added up;
// where blocks are left for that, this launch does (777 x 1000 x 520 with gelu and bias 11.4 us, with a launch for it in
// front 12.2).
moe_status both_products(double apart, const void *dz, const void *W, const void *x, int T, int K, int N, const Ends &dx,
                         const Ends &dw, const float *sums, int rows, float *dbias, int32_t *status, bool first, int sms,
                         cudaStream_t s, bool *sums_left, bool *done) {
  const Cut cx = cut_with(T, K, N, 1, false), cw = cut_with(K, N, T, 1, false);
  *done = false;
  if (static_cast<int64_t>(cx.units) + cw.units > kRuleSms || std::max(cx.cost, cw.cost) > apart) return MOE_OK;
  int groups = 0;
  if (groups_of<kBoth, 1>(sms, &groups) != cudaSuccess) return MOE_ERR_CUDA;
  if (cx.units + cw.units > groups) return MOE_OK;
  Operands ox, ow;
  if (!operands(&ox, kDx, dz, W, T, K, N, cx, dx, nullptr, status, first) ||
      !operands(&ow, kDw, x, dz, K, N, T, cw, dw, nullptr, status, first))
    return MOE_ERR_CUDA;
  const int columns = (N + 31) / 32, extra = *sums_left && cx.units + cw.units + columns <= groups ? columns : 0;
  if (extra) {
    ox.p.sums = sums;
    ox.p.sum_rows = rows;
    ox.p.dbias = dbias;
    *sums_left = false;
  }
  *done = true;
  return timed("linear_dx_dW", s, [&] {
    return launch_pdl(linear_product_kernel<kBoth, 1>, dim3(static_cast<unsigned>(cx.units + cw.units + extra)), dim3(kGemmThreads),
                      kGemmSmem, s, 1, ox.a, ox.a32, ox.b, ow.a, ow.b, ox.p, ow.p);
  });
}

template <int TM, int CT>
cudaError_t launch_rows(RowArgs a, cudaStream_t s) {
  const int tiles = (a.N + 8 * CT - 1) / (8 * CT), units = a.K / 8;
  a.parts = 1;
  while (a.parts < 8 && 2 * a.parts * tiles <= rows_per_sm(TM) * kRuleSms && units >= 2 * a.parts * (kRowThreads / CT)) a.parts *= 2;
  a.per = (units + a.parts - 1) / a.parts;
  return launch_pdl(linear_rows_kernel<TM, CT>, dim3(static_cast<unsigned>(tiles * a.parts)), dim3(kRowThreads), 0, s, a.parts, a);
}
template <int TM>
cudaError_t rows_of(const RowArgs &a, cudaStream_t s) {
  return a.N > kNarrow ? launch_rows<TM, 8>(a, s) : launch_rows<TM, 2>(a, s);
}

bool linear_ok(const moe_linear_config *c) {
  if (!c || c->T < 0 || c->T > (1 << 30)) return false;
  if (c->K < 8 || c->K > kMaxDim || c->K % 8 || c->N < 8 || c->N > kMaxDim || c->N % 8) return false;
  if (static_cast<int64_t>(c->T) * std::max(c->K, c->N) >= int64_t{1} << 40) return false;  // (tiles are counted in 32 bits)
  return c->act >= MOE_ACT_NONE && c->act <= MOE_ACT_GELU;
}

// The scratch: the status word and the parts' sums; the backward's holds those of any of the three products, so that it
// serves the forward, too, then dz and dbias' partial rows.
size_t fwd_bytes(const moe_linear_config *c, Cut *cut) {  // few rows: *cut is left as it is
  if (few_rows(c->T, c->K, c->N)) return kHeader;
  *cut = cut_of(c->T, c->N, c->K);
  return kHeader + part_bytes(*cut);
}
struct LinearLayout {
  Cut dx, dw;
  size_t dz, sums, bwd;
};
LinearLayout linear_layout(const moe_linear_config *c) {
  LinearLayout L;
  L.dx = cut_of(c->T, c->K, c->N);
  L.dw = cut_of(c->K, c->N, c->T);
  Cut fwd;
  L.dz = align256(std::max(fwd_bytes(c, &fwd), kHeader + std::max(part_bytes(L.dx), part_bytes(L.dw))));
  L.sums = L.dz + (c->act == MOE_ACT_NONE ? 0 : align256(static_cast<size_t>(c->T) * c->N * 2));
  L.bwd = L.sums + align256(static_cast<size_t>(dz_split(c->T, c->N)) * c->N * 4);
  return L;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_linear_workspace(const moe_linear_config *cfg, size_t *fwd_scratch, size_t *bwd_scratch) {
  if (!linear_ok(cfg)) return MOE_ERR_INVALID_ARG;
  Cut cut;
  if (fwd_scratch) *fwd_scratch = fwd_bytes(cfg, &cut);
  if (bwd_scratch) *bwd_scratch = linear_layout(cfg).bwd;
  return MOE_OK;
}

moe_status moe_linear_forward(const moe_linear_config *cfg, const void *x, const void *W, const void *bias,
                              const void *residual, void *y, void *z, void *scratch, size_t scratch_bytes, void *stream) {
  if (!linear_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!W || !scratch || (cfg->T > 0 && (!x || !y)) || (z && cfg->act == MOE_ACT_NONE)) return MOE_ERR_INVALID_ARG;
  if (!al16(x) || !al16(W) || !al16(bias) || !al16(residual) || !al16(y) || !al16(z) || !al16(scratch)) return MOE_ERR_ALIGNMENT;
  Cut cut;
  if (scratch_bytes < fwd_bytes(cfg, &cut)) return MOE_ERR_WORKSPACE;
  DevInfo di;
  MOE_TRY(device_info(&di));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t *sc = static_cast<uint8_t *>(scratch);
  if (cfg->T == 0) return cudaMemsetAsync(sc, 0, kHeader, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  Ends e{};
  e.bias = static_cast<const uint16_t *>(bias);
  e.res = static_cast<const uint16_t *>(residual);
  e.y = static_cast<uint16_t *>(y);
  e.z = static_cast<uint16_t *>(z);
  e.act = cfg->act;
  if (few_rows(cfg->T, cfg->K, cfg->N)) {
    RowArgs a{};
    a.x = static_cast<const uint16_t *>(x);
    a.W = static_cast<const uint16_t *>(W);
    a.e = e;
    a.T = cfg->T;
    a.K = cfg->K;
    a.N = cfg->N;
    a.status = reinterpret_cast<int32_t *>(sc);
    return timed("linear_forward", s, [&] {
      return a.T == 1 ? rows_of<1>(a, s) : a.T == 2 ? rows_of<2>(a, s) : a.T <= 4 ? rows_of<4>(a, s) : rows_of<8>(a, s);
    });
  }
  return product<kFwd>("linear_forward", cut, x, W, cfg->T, cfg->N, cfg->K, e, reinterpret_cast<float *>(sc + kHeader),
                       reinterpret_cast<int32_t *>(sc), true, di.sms, s);
}

moe_status moe_linear_backward(const moe_linear_config *cfg, const void *dy, const void *x, const void *W, const void *z,
                               void *dx, void *dW, float *dbias, void *scratch, size_t scratch_bytes, void *stream) {
  if (!linear_ok(cfg)) return MOE_ERR_INVALID_ARG;
  const bool act = cfg->act != MOE_ACT_NONE;
  if (!scratch || (!dx && !dW && !dbias) || (dx && !W)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!dy || (dW && !x) || (act != (z != nullptr)))) return MOE_ERR_INVALID_ARG;
  if (!al16(dy) || !al16(x) || !al16(W) || !al16(z) || !al16(dx) || !al16(dW) || !al16(dbias) || !al16(scratch))
    return MOE_ERR_ALIGNMENT;
  const LinearLayout L = linear_layout(cfg);
  if (scratch_bytes < L.bwd) return MOE_ERR_WORKSPACE;
  DevInfo di;
  MOE_TRY(device_info(&di));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t *sc = static_cast<uint8_t *>(scratch);
  int32_t *status = reinterpret_cast<int32_t *>(sc);
  const int T = cfg->T, K = cfg->K, N = cfg->N;
  if (T == 0) {
    if (cudaMemsetAsync(sc, 0, kHeader, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (dW && cudaMemsetAsync(dW, 0, static_cast<size_t>(K) * N * 2, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  float *part = reinterpret_cast<float *>(sc + kHeader);
  const void *dz = dy;
  bool first = true, sums_left = false;
  const float *sums = nullptr;  // dbias' partial rows
  int rows = 0;
  if (act || dbias) {
    DzArgs a{};
    a.dy = static_cast<const uint16_t *>(dy);
    a.z = static_cast<const uint16_t *>(z);
    a.dz = act && (dx || dW) ? reinterpret_cast<uint16_t *>(sc + L.dz) : nullptr;
    a.dbias = dbias;
    a.part = dbias ? reinterpret_cast<float *>(sc + L.sums) : nullptr;
    a.T = T;
    a.N = N;
    a.status = status;
    a.split = dz_split(T, N);
    const auto kernel = cfg->act == MOE_ACT_RELU   ? linear_dz_kernel<MOE_ACT_RELU>
                        : cfg->act == MOE_ACT_SILU ? linear_dz_kernel<MOE_ACT_SILU>
                        : cfg->act == MOE_ACT_GELU ? linear_dz_kernel<MOE_ACT_GELU>
                                                   : linear_dz_kernel<MOE_ACT_NONE>;
    MOE_TRY(timed("linear_dz", s, [&] {
      return launch_pdl(kernel, dim3((N + kDzCols - 1) / kDzCols, a.split), dim3(kDzThreads), 0, s, 1, a);
    }));
    sums = a.part;
    rows = a.split;
    sums_left = dbias && rows > 1;
    if (act) dz = a.dz;
    first = false;
  }
  Ends ex{}, ew{};
  ex.y = static_cast<uint16_t *>(dx);
  ew.y = static_cast<uint16_t *>(dW);
  bool done = false;
  if (dx && dW)
    MOE_TRY(both_products(L.dx.cost + L.dw.cost, dz, W, x, T, K, N, ex, ew, sums, rows, dbias, status, first, di.sms, s,
                          &sums_left, &done));
  if (sums_left)
    MOE_TRY(timed("linear_dbias", s, [&] {
      return launch_pdl(linear_dbias_kernel, dim3((N + 31) / 32), dim3(kDzThreads), 0, s, 1, sums, rows, N, dbias);
    }));
  if (dx && !done) {
    MOE_TRY(product<kDx>("linear_dx", L.dx, dz, W, T, K, N, ex, part, status, first, di.sms, s));
    first = false;
  }
  if (dW && !done) MOE_TRY(product<kDw>("linear_dW", L.dw, x, dz, K, N, T, ew, part, status, first, di.sms, s));
  return MOE_OK;
}

}  // extern "C"
