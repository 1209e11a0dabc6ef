// ortho.cu -- the orthogonalised update of a batch of matrices by Newton-Schulz
// products (what the Muon optimiser applies to a weight's momentum).
//
// Per matrix [R, C], n = min(R, C), m = max(R, C), and u the update (optionally
// through a momentum m' = beta m + g):
//   X = u / max(|u|_F, eps);   each step:  S = X X^T  (or X^T X: n x n),
//   P = a I + b S + c S^2,     X <- P X  (or X P);          out = scale X (bf16)
// With the usual coefficients every singular value ends near 1.
//
// Number format: X, S and P are held in fp16 between products (fp32 accumulation
// throughout).  All three are bounded by about 3.5, so fp16's range suffices and
// its 2^-12 rounding is eight times finer than bf16's: the result is within 1.3
// times the error that rounding the exact result to bf16 makes anyway (bf16
// operands: four to seven times).  X carries a factor of 256 that keeps its
// entries (about 1 / sqrt(n m) at first) clear of fp16's subnormals.  a I is part
// of P, so the update is one plain product.
//
// No transposes: the tensor core reads either operand with its reduction axis
// contiguous or strided (K-major or MN-major boxes), S and P are symmetric, and
// only S's and P's upper tiles are computed (the lower ones are stored mirrored).
//
// The products run on CTA pairs (tcgen05 cta_group::2, 256 x 256 tiles, fp32
// accumulators double-buffered in TMEM), persistent over all matrices' tiles:
//   warp 0     TMA producer (both CTAs): 128B-swizzled boxes of 3-D maps, which
//              read zeros past a matrix's own rows and columns
//   warp 1     CTA 0: MMA issuer
//   warps 2-9  epilogue: tcgen05.ld, the polynomial, rounding, coalesced stores
// Every wait is bounded; on a timeout the kernel flags the status word, drains
// its copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_fp16.h>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr float kSigma = 256.f;  // X is stored times this
constexpr int kMaxDim = 16384, kMaxBatch = 65535, kMaxSteps = 64;  // (at most 2^28 tiles in a product)

// ---------------------------------------------------------------- norms and the first X

constexpr int kPrepThreads = 256;
constexpr int kPrepVecs = 8;                                  // 8-element groups per thread
constexpr int kChunk = kPrepThreads * kPrepVecs * 8;          // elements of one block

struct PrepArgs {
  const void *g;
  float *mom;     // [B,R,C] or null
  float beta;
  bool nesterov;
  float eps;
  int64_t numel;  // R * C
  int C, ld;      // columns, and X's row stride
  int chunks;     // blocks per matrix
  float *part;    // [B][chunks] sums of squares
  uint16_t *x;    // [B][R][ld] fp16
  int64_t x_stride;
  int32_t *status;
};

__device__ __forceinline__ float to_f(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float to_f(float v) { return v; }

// Eight (VEC) or one consecutive elements of src.
template <class El, bool VEC>
__device__ __forceinline__ void load_el(const El *src, float (&f)[VEC ? 8 : 1]) {
  if constexpr (!VEC) {
    f[0] = to_f(*src);
  } else if constexpr (sizeof(El) == 2) {
    const uint4 q = *reinterpret_cast<const uint4 *>(src);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
}

// The update from the gradient and the (new) momentum.
__device__ __forceinline__ float update_of(float g, float m, float beta, bool nesterov) {
  return nesterov ? fmaf(beta, m, g) : m;
}

// Sum of squares of one chunk of one matrix's update; the momentum is advanced
// on the way.  VEC: a matrix's elements are whole groups of eight.
template <class El, bool VEC, bool MOM>
__global__ void __launch_bounds__(kPrepThreads) ortho_norm_kernel(const PrepArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s_w[kPrepThreads / 32];
  constexpr int N = VEC ? 8 : 1, IT = kChunk / (kPrepThreads * N), U = VEC ? kPrepVecs : 16;
  const El *g = static_cast<const El *>(a.g) + blockIdx.y * a.numel;
  float *mom = MOM ? a.mom + blockIdx.y * a.numel : nullptr;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x * N;
  float acc = 0.f;
#pragma unroll 1
  for (int it = 0; it < IT; it += U) {
    float f[U][N], m[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = base + static_cast<int64_t>(it + u) * kPrepThreads * N;
      if (at < a.numel) {
        load_el<El, VEC>(g + at, f[u]);
        if constexpr (MOM) load_el<float, VEC>(mom + at, m[u]);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[u][i] = m[u][i] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = base + static_cast<int64_t>(it + u) * kPrepThreads * N;
      if constexpr (MOM) {
#pragma unroll
        for (int i = 0; i < N; ++i) m[u][i] = fmaf(a.beta, m[u][i], f[u][i]);
        if (at < a.numel) {
          if constexpr (VEC) {
            reinterpret_cast<float4 *>(mom + at)[0] = make_float4(m[u][0], m[u][1], m[u][2], m[u][3]);
            reinterpret_cast<float4 *>(mom + at)[1] = make_float4(m[u][4], m[u][5], m[u][6], m[u][7]);
          } else {
            mom[at] = m[u][0];
          }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) f[u][i] = update_of(f[u][i], m[u][i], a.beta, a.nesterov);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) acc = fmaf(f[u][i], f[u][i], acc);
    }
  }
  acc = warp_sum(acc);
  if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kPrepThreads / 32; ++w) acc += s_w[w];
    a.part[static_cast<size_t>(blockIdx.y) * a.chunks + blockIdx.x] = acc;
  }
}

// X = kSigma u / max(|u|, eps) in fp16, rows padded to ld.  VEC: rows are whole
// groups of eight.
template <class El, bool VEC, bool MOM>
__global__ void __launch_bounds__(kPrepThreads) ortho_scale_kernel(const PrepArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s_w[kPrepThreads / 32];
  constexpr int N = VEC ? 8 : 1, IT = kChunk / (kPrepThreads * N);
  float sq = 0.f;  // the matrix's chunks in a fixed order
  for (int i = threadIdx.x; i < a.chunks; i += kPrepThreads)
    sq += a.part[static_cast<size_t>(blockIdx.y) * a.chunks + i];
  sq = warp_sum(sq);
  if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = sq;
  __syncthreads();
  sq = s_w[0];
#pragma unroll
  for (int w = 1; w < kPrepThreads / 32; ++w) sq += s_w[w];
  const bool fine = isfinite(sq);
  if (!fine && blockIdx.x == 0 && threadIdx.x == 0) flag_status(a.status, kDevNonfiniteUpdate);
  const float norm = fmaxf(sqrtf(sq), a.eps);
  const float f0 = fine ? (norm > 0.f ? kSigma / norm : 0.f) : NAN;
  const El *g = static_cast<const El *>(a.g) + blockIdx.y * a.numel;
  const float *mom = MOM ? a.mom + blockIdx.y * a.numel : nullptr;
  uint16_t *x = a.x + blockIdx.y * a.x_stride;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kChunk + threadIdx.x * N;
#pragma unroll 4
  for (int it = 0; it < IT; ++it) {
    const int64_t at = base + static_cast<int64_t>(it) * kPrepThreads * N;
    if (at >= a.numel) break;
    float f[N];
    load_el<El, VEC>(g + at, f);
    if constexpr (MOM) {
      float m[N];
      load_el<float, VEC>(mom + at, m);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = update_of(f[i], m[i], a.beta, a.nesterov);
    }
    const int row = static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(a.C));  // R * C <= 2^28
    const int64_t dst = static_cast<int64_t>(row) * a.ld + (at - static_cast<int64_t>(row) * a.C);
    if constexpr (VEC) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i] * f0, f[2 * i + 1] * f0);
        memcpy(&w[i], &h, 4);
      }
      *reinterpret_cast<uint4 *>(x + dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      x[dst] = __half_as_ushort(__float2half_rn(f[0] * f0));
    }
  }
}

// ---------------------------------------------------------------- products

constexpr int BM = 128;               // rows per CTA of a 256-row tile
constexpr int BN = 256;               // tile columns; 128 of B per CTA
constexpr int BK = 64;                // reduction elements per box: one 128-byte swizzle row
constexpr int kHalf = 128 * BK * 2;   // one operand's box (or two 64 x 64 boxes) per CTA: 16 KB
constexpr int kBox = 64 * 64 * 2;
constexpr int kStages = 3;
constexpr int kStageBytes = 4 * kHalf;  // two K blocks: [A k0 | A k1 | B k0 | B k1]
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;
constexpr int kTileBytes = 32 * 32 * 2;  // an epilogue warp's staging tile
constexpr uint32_t kTmemCols = 2 * BN;
constexpr int kEpiOff = kStages * kStageBytes + 256;
constexpr int kGemmSmem = kEpiOff + kEpiWarps * kTileBytes + 1024 /*align*/;
static_assert(kGemmSmem <= 227 * 1024, "shared memory budget");

enum Product : int {
  kGram = 0,    // X X^T (or X^T X) / sigma^2 -> S
  kSquare = 1,  // a I + b S + c S S -> P
  kUpdate = 2,  // P X (or X P) -> X
  kLast = 3     // the same times scale / sigma -> out, bf16
};

struct ProductArgs {
  int batch, M, N, K;
  int nm, nn;             // tiles of 256 rows, of 256 columns
  int per;                // tiles per matrix (symmetric: mt <= nt)
  float a, b, c;          // kSquare; c also the factor of the other products
  const uint16_t *s;      // kSquare: S
  uint16_t *out;
  int ld;                 // row stride of s and out
  int64_t stride;         // matrix stride of both
  int32_t *status;
};

struct TileAt {
  int b, m0, n0;
  bool mirror;  // symmetric, off the diagonal: stored transposed as well
};

template <int KIND>
__device__ __forceinline__ TileAt tile_of(int tile, const ProductArgs &p) {
  TileAt t;
  t.b = tile / p.per;
  int r = tile - t.b * p.per;
  if constexpr (KIND == kGram || KIND == kSquare) {
    int nt = 0;
    while (r > nt) r -= ++nt;
    t.m0 = r * 2 * BM;
    t.n0 = nt * BN;
    t.mirror = r != nt;
  } else {
    const int mt = r / p.nn;
    t.m0 = mt * 2 * BM;
    t.n0 = (r - mt * p.nn) * BN;
    t.mirror = false;
  }
  return t;
}

// Byte offset of row r's 16-byte piece q (of 4) in a staging tile: the XOR keeps
// rows written by lanes and pieces read by rows free of bank conflicts.
__device__ __forceinline__ uint32_t swz(int r, int q) {
  return static_cast<uint32_t>(r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

// The staging tile's rows [0, nrows) to global rows at g0 (stride ld), pieces of
// eight columns below ncols (a multiple of eight).
__device__ __forceinline__ void tile_to_rows(const uint8_t *tile, uint16_t *g0, int64_t ld, int nrows, int ncols) {
  const int lane = threadIdx.x & 31, q = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 w = *reinterpret_cast<const uint4 *>(tile + swz(r, q));
    if (r < nrows && q * 8 < ncols) *reinterpret_cast<uint4 *>(g0 + r * ld + q * 8) = w;
  }
}

constexpr int kChunks = BN / 64;  // 32-column chunks of a warp's half of the columns

// kSquare: S under the warp's 32 rows and half of the tile's columns, in the
// order its coalesced loads bring it.
struct SChunks {
  uint4 v[kChunks][4];
  __device__ __forceinline__ void load(const TileAt &t, int row0, int part, const ProductArgs &p) {
    const int lane = threadIdx.x & 31, nrows = min(32, p.M - row0);
    const uint16_t *s = p.s + t.b * p.stride;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c0 = t.n0 + part * (BN / 2) + 32 * j;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        v[j][i] = r < nrows && c0 < p.N ? *reinterpret_cast<const uint4 *>(
                                              s + (row0 + r) * static_cast<int64_t>(p.ld) + c0 + (lane & 3) * 8)
                                        : make_uint4(0, 0, 0, 0);
      }
    }
  }
};

// One warp's 32 rows of half a tile's columns.
template <int KIND>
__device__ __forceinline__ void epilogue(const TileAt &t, uint32_t tb, int row0, int part, const ProductArgs &p,
                                         uint8_t *tile, const SChunks &sc) {
  const int lane = threadIdx.x & 31;
  const int nrows = min(32, p.M - row0);
  uint16_t *out = p.out + t.b * p.stride;
#pragma unroll KIND == kSquare ? kChunks : 1
  for (int j = 0; j < kChunks; ++j) {
    const int cc = part * (BN / 2) + 32 * j, c0 = t.n0 + cc;
    if (c0 >= p.N || nrows <= 0) break;
    uint32_t acc[32];
    tmem_ld32(tb + cc, acc);
    float v[32];
    if constexpr (KIND == kSquare) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(tile + swz(8 * i + (lane >> 2), lane & 3)) = sc.v[j][i];
      __syncwarp();
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = *reinterpret_cast<const uint4 *>(tile + swz(lane, q));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          __half2 hh;
          memcpy(&hh, &ww[h], 4);
          const float2 f = __half22float2(hh);
          const int e = 8 * q + 2 * h;
          v[e] = fmaf(p.c, __uint_as_float(acc[e]), p.b * f.x);
          v[e + 1] = fmaf(p.c, __uint_as_float(acc[e + 1]), p.b * f.y);
        }
      }
      if (c0 < row0 + 32 && row0 < c0 + 32) {  // the chunk on the diagonal (both start at multiples of 32)
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e == lane) v[e] += p.a;
      }
      __syncwarp();
    } else {
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(acc[e]) * p.c;
    }
    if constexpr (KIND == kLast) {  // out [M,N] itself, bf16
      const int ncols = min(32, p.N - c0);
      uint16_t *g0 = out + row0 * static_cast<int64_t>(p.ld) + c0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4 *>(tile + swz(lane, q)) =
            make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                       pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
      __syncwarp();
      if ((p.ld & 7) == 0) {
        tile_to_rows(tile, g0, p.ld, nrows, ncols);
      } else {  // rows that start anywhere: a row's columns across the lanes
        for (int r = 0; r < nrows; ++r)
          if (lane < ncols)
            g0[r * static_cast<int64_t>(p.ld) + lane] =
                *reinterpret_cast<const uint16_t *>(tile + swz(r, lane >> 3) + (lane & 7) * 2);
      }
      __syncwarp();
    } else {  // padded rows: whole chunks
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint4 *>(tile + swz(lane, q)) =
            make_uint4(pack_half2(v[8 * q], v[8 * q + 1]), pack_half2(v[8 * q + 2], v[8 * q + 3]),
                       pack_half2(v[8 * q + 4], v[8 * q + 5]), pack_half2(v[8 * q + 6], v[8 * q + 7]));
      __syncwarp();
      tile_to_rows(tile, out + row0 * static_cast<int64_t>(p.ld) + c0, p.ld, nrows, 32);
      __syncwarp();
      if constexpr (KIND == kGram || KIND == kSquare) {
        if (t.mirror) {  // column e of the chunk is row c0 + e of the transpose
#pragma unroll
          for (int e = 0; e < 32; ++e)
            *reinterpret_cast<uint16_t *>(tile + swz(e, lane >> 3) + (lane & 7) * 2) =
                __half_as_ushort(__float2half_rn(v[e]));
          __syncwarp();
          tile_to_rows(tile, out + c0 * static_cast<int64_t>(p.ld) + row0, p.ld, min(32, p.N - c0), 32);
          __syncwarp();
        }
      }
    }
  }
}

// One K block of one operand into this CTA's half of the stage: 128 rows x 64 of
// K (K-major), or 64 of K x 128 columns in two boxes (MN-major).
template <int MN>
__device__ __forceinline__ void load_operand(uint8_t *dst, const CUtensorMap *map, uint32_t bar, int k0, int r0, int b) {
  if constexpr (MN) {
    tma_load_3d_pair(dst, map, bar, r0, k0, b);
    tma_load_3d_pair(dst + kBox, map, bar, r0 + 64, k0, b);
  } else {
    tma_load_3d_pair(dst, map, bar, k0, r0, b);
  }
}

template <int KIND, int AMN, int BMN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ortho_product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const ProductArgs p) {
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
  uint8_t *epi_tiles = smem + kEpiOff;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  griddep_wait();  // the set-up above overlaps the previous kernel's end; its outputs are read below
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = p.batch * p.per;
  const int nkb = (p.K + BK - 1) / BK, nstage = (nkb + 1) / 2;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = peer_smem_addr(&full[0], 0);
      int stage = 0;
      uint32_t phase = 0, armed = 0, arm_par = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs) {
        const TileAt t = tile_of<KIND>(tile, p);
        for (int ks = 0; ks < nstage; ++ks) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t *sa = smem + stage * kStageBytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);  // both CTAs' bytes
          // a K block past the end is zero fill, and no MMA reads it
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k0 = (ks * 2 + h) * BK;
            load_operand<AMN>(sa + h * kHalf, &tmA, full0 + 8u * stage, k0, t.m0 + BM * rank, t.b);
            load_operand<BMN>(sa + (2 + h) * kHalf, &tmB, full0 + 8u * stage, k0, t.n0 + (BN / 2) * rank, t.b);
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
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair; tile < total && ok; tile += npairs, ++it) {
        const int buf = it & 1;
        if (!mbar_wait(&tempty[buf], ((it >> 1) & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * BN;
        for (int ks = 0; ks < nstage; ++ks) {
          if (!mbar_wait(&full[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t ab = smem_addr(smem + stage * kStageBytes), bb = ab + 2 * kHalf;
          const int nk16 = (BK / 16) * min(2, nkb - ks * 2);
#pragma unroll
          for (int k16 = 0; k16 < 2 * (BK / 16); ++k16) {
            if (k16 < nk16) {
              const int h = k16 / (BK / 16), j = k16 % (BK / 16);
              const uint32_t ao = ab + h * kHalf, bo = bb + h * kHalf;
              const uint64_t ad =
                  AMN ? smem_desc_sw128(ao + j * 2048, kBox, 1024) : smem_desc_sw128(ao + j * 32, 16, 1024);
              const uint64_t bd =
                  BMN ? smem_desc_sw128(bo + j * 2048, kBox, 1024) : smem_desc_sw128(bo + j * 32, 16, 1024);
              tc_mma_f16_pair(d, ad, bd, idesc_f16(2 * BM, BN, AMN, BMN), (ks | k16) != 0 ? 1u : 0u);
            }
          }
          tc_commit_pair(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        tc_commit_pair(&tfull[buf]);
      }
      if (*abort_flag) {  // wait for the pair's MMAs before TMEM is freed
        tc_commit_pair(drain);
        for (int i = 0; i < (1 << 22) && !mbar_try_wait(drain, 0); ++i) {
        }
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;               // TMEM lane quarter
    const int part = (warp - 2) >> 2;     // column half
    const uint32_t tempty0 = peer_smem_addr(&tempty[0], 0), tempty1 = peer_smem_addr(&tempty[1], 0);
    uint8_t *stile = epi_tiles + (warp - 2) * kTileBytes;
    int it = 0;
    for (int tile = pair; tile < total; tile += npairs, ++it) {
      const TileAt t = tile_of<KIND>(tile, p);
      const int buf = it & 1, row0 = t.m0 + BM * rank + q * 32;
      SChunks sc;
      if constexpr (KIND == kSquare) sc.load(t, row0, part, p);  // while the product runs
      if (!wait_lane0(&tfull[buf], (it >> 1) & 1, abort_flag)) break;
      __syncwarp();
      tc_fence_after();
      epilogue<KIND>(t, tmem_base + buf * BN + (static_cast<uint32_t>(q * 32) << 16), row0, part, p, stile, sc);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(buf ? tempty1 : tempty0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) flag_status(p.status, kDevWaitTimeout);
  cluster_sync();  // the pair is done with each other's barriers and TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A batch of fp16 matrices [rows, inner] with row stride ld: boxes of 64 x box_rows,
// 128-byte swizzle, zeros outside each matrix.
bool map3(CUtensorMap *m, const void *ptr, int inner, int rows, int batch, int ld, int box_rows) {
  auto fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * 2 * rows};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, int AMN, int BMN>
cudaError_t launch_product(const CUtensorMap &a, const CUtensorMap &b, ProductArgs p, int sms, cudaStream_t s) {
  static DeviceOnce once;  // the shared-memory opt-in, and how many CTA pairs fit at once
  auto kernel = ortho_product_kernel<KIND, AMN, BMN>;
  int pairs = 0;
  cudaError_t e = once.get(
      [&](int *out) {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem);
        if (r != cudaSuccess) return r;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(sms & ~1);
        q.blockDim = dim3(kGemmThreads);
        q.dynamicSmemBytes = kGemmSmem;
        q.attrs = &attr;
        q.numAttrs = 1;
        int n = 0;
        r = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
        if (r != cudaSuccess) return r;
        if (n < 1) return cudaErrorInvalidConfiguration;
        *out = n < sms / 2 ? n : sms / 2;
        return cudaSuccess;
      },
      &pairs);
  if (e != cudaSuccess) return e;
  p.nm = (p.M + 2 * BM - 1) / (2 * BM);
  p.nn = (p.N + BN - 1) / BN;
  p.per = KIND == kGram || KIND == kSquare ? p.nn * (p.nn + 1) / 2 : p.nm * p.nn;
  const int tiles = p.per * p.batch;
  return launch_pdl(kernel, dim3(2 * (tiles < pairs ? tiles : pairs)), dim3(kGemmThreads), kGemmSmem, s, 2, a, b, p);
}

bool ortho_ok(const moe_ortho_config *c) {
  if (!c || c->batch < 0 || c->batch > kMaxBatch || c->R < 1 || c->R > kMaxDim || c->C < 1 || c->C > kMaxDim)
    return false;
  if (c->steps < 1 || c->steps > kMaxSteps || !(c->eps >= 0.f)) return false;
  return c->dtype == MOE_DTYPE_BF16 || c->dtype == MOE_DTYPE_FP32;
}

inline int pad64(int x) { return (x + 63) / 64 * 64; }

struct OrthoLayout {
  int chunks, ldx, lds;
  size_t part, x0, x1, s, p, total;
};
OrthoLayout ortho_layout(const moe_ortho_config *c) {
  OrthoLayout L;
  const size_t B = c->batch, n = c->R < c->C ? c->R : c->C;
  L.chunks = static_cast<int>((static_cast<int64_t>(c->R) * c->C + kChunk - 1) / kChunk);
  L.ldx = pad64(c->C);
  L.lds = pad64(static_cast<int>(n));
  size_t o = kHeader;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  L.part = take(B * L.chunks * 4);
  L.x0 = take(B * c->R * L.ldx * 2);
  L.x1 = take(c->steps > 1 ? B * c->R * L.ldx * 2 : 0);
  L.s = take(B * n * L.lds * 2);
  L.p = take(B * n * L.lds * 2);
  L.total = o;
  return L;
}

template <class El>
cudaError_t launch_prep(const PrepArgs &a, int batch, int C, cudaStream_t s) {
  const dim3 grid(a.chunks, batch), block(kPrepThreads);
  const bool whole = a.numel % 8 == 0, rows = C % 8 == 0;
  cudaError_t e;
  if (a.mom)
    e = launch_pdl(whole ? ortho_norm_kernel<El, true, true> : ortho_norm_kernel<El, false, true>, grid, block, 0, s, 1,
                   a);
  else
    e = launch_pdl(whole ? ortho_norm_kernel<El, true, false> : ortho_norm_kernel<El, false, false>, grid, block, 0, s,
                   1, a);
  if (e != cudaSuccess) return e;
  if (a.mom)
    return launch_pdl(rows ? ortho_scale_kernel<El, true, true> : ortho_scale_kernel<El, false, true>, grid, block, 0,
                      s, 1, a);
  return launch_pdl(rows ? ortho_scale_kernel<El, true, false> : ortho_scale_kernel<El, false, false>, grid, block, 0,
                    s, 1, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_ortho_workspace(const moe_ortho_config *cfg, size_t *scratch) {
  if (!ortho_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (scratch) *scratch = ortho_layout(cfg).total;
  return MOE_OK;
}

moe_status moe_ortho_update(const moe_ortho_config *cfg, const float *coefs, const void *g, float *momentum,
                            float beta, int32_t nesterov, float scale, void *out, void *scratch, size_t scratch_bytes,
                            void *stream) {
  if (!ortho_ok(cfg) || !coefs) return MOE_ERR_INVALID_ARG;
  if (!scratch || (cfg->batch > 0 && (!g || !out))) return MOE_ERR_INVALID_ARG;
  if (!al16(g) || !al16(momentum) || !al16(out) || !al16(scratch)) return MOE_ERR_ALIGNMENT;
  const OrthoLayout L = ortho_layout(cfg);
  if (scratch_bytes < L.total) return MOE_ERR_WORKSPACE;
  DevInfo di;
  MOE_TRY(device_info(&di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t *sc = static_cast<uint8_t *>(scratch);
  if (cudaMemsetAsync(sc, 0, kHeader, st) != cudaSuccess) return MOE_ERR_CUDA;
  if (cfg->batch == 0) return MOE_OK;
  const int B = cfg->batch, R = cfg->R, C = cfg->C;
  const bool tall = R > C;
  const int n = tall ? C : R, m = tall ? R : C;
  int32_t *status = reinterpret_cast<int32_t *>(sc);
  PrepArgs a{};
  a.g = g;
  a.mom = momentum;
  a.beta = beta;
  a.nesterov = nesterov != 0;
  a.eps = cfg->eps;
  a.numel = static_cast<int64_t>(R) * C;
  a.C = C;
  a.ld = L.ldx;
  a.chunks = L.chunks;
  a.part = reinterpret_cast<float *>(sc + L.part);
  a.x = reinterpret_cast<uint16_t *>(sc + L.x0);
  a.x_stride = static_cast<int64_t>(R) * L.ldx;
  a.status = status;
  MOE_TRY(timed("ortho_norm_scale", st, [&] {
    return cfg->dtype == MOE_DTYPE_BF16 ? launch_prep<uint16_t>(a, B, C, st) : launch_prep<float>(a, B, C, st);
  }));
  // X's rows along C with C contiguous: the Gram product reduces over m, the
  // update over n, so one of them reads X K-major and the other MN-major
  uint8_t *xb[2] = {sc + L.x0, sc + L.x1};
  CUtensorMap xk[2], xm[2], ms, mp;
  for (int i = 0; i < (cfg->steps > 1 ? 2 : 1); ++i)
    if (!map3(&xk[i], xb[i], C, R, B, L.ldx, 128) || !map3(&xm[i], xb[i], C, R, B, L.ldx, 64)) return MOE_ERR_CUDA;
  if (!map3(&ms, sc + L.s, n, n, B, L.lds, 128) || !map3(&mp, sc + L.p, n, n, B, L.lds, 128)) return MOE_ERR_CUDA;
  for (int i = 0; i < cfg->steps; ++i) {
    const int cur = i & 1;
    ProductArgs p{};
    p.batch = B;
    p.status = status;
    p.M = p.N = n;
    p.K = m;
    p.ld = L.lds;
    p.stride = static_cast<int64_t>(n) * L.lds;
    p.c = 1.f / (kSigma * kSigma);
    p.out = reinterpret_cast<uint16_t *>(sc + L.s);
    MOE_TRY(timed("ortho_gram", st, [&] {
      return tall ? launch_product<kGram, 1, 1>(xm[cur], xm[cur], p, di.sms, st)
                  : launch_product<kGram, 0, 0>(xk[cur], xk[cur], p, di.sms, st);
    }));
    p.K = n;
    p.a = coefs[3 * i];
    p.b = coefs[3 * i + 1];
    p.c = coefs[3 * i + 2];
    p.s = reinterpret_cast<const uint16_t *>(sc + L.s);
    p.out = reinterpret_cast<uint16_t *>(sc + L.p);
    MOE_TRY(timed("ortho_polynomial", st, [&] { return launch_product<kSquare, 0, 0>(ms, ms, p, di.sms, st); }));
    const bool last = i + 1 == cfg->steps;
    p.M = R;
    p.N = C;
    p.ld = last ? C : L.ldx;
    p.stride = static_cast<int64_t>(R) * p.ld;
    p.c = last ? scale / kSigma : 1.f;
    p.out = last ? static_cast<uint16_t *>(out) : reinterpret_cast<uint16_t *>(xb[cur ^ 1]);
    MOE_TRY(timed("ortho_apply", st, [&] {
      if (last)
        return tall ? launch_product<kLast, 0, 0>(xk[cur], mp, p, di.sms, st)
                    : launch_product<kLast, 0, 1>(mp, xm[cur], p, di.sms, st);
      return tall ? launch_product<kUpdate, 0, 0>(xk[cur], mp, p, di.sms, st)
                  : launch_product<kUpdate, 0, 1>(mp, xm[cur], p, di.sms, st);
    }));
  }
  return MOE_OK;
}

}  // extern "C"
