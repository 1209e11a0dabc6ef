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
// throughout).  With the usual coefficients none is above 3.5, so fp16's range
// suffices and its 2^-12 rounding is eight times finer than bf16's: the result is
// within 1.4 times the error that rounding the exact result to bf16 makes anyway (bf16
// operands: four to seven times).  X carries a factor of 256 that keeps its
// entries (about 1 / sqrt(n m) at first) clear of fp16's subnormals.  a I is part
// of P, so the update is one plain product.  Coefficients with which X passes 255, or
// P (for pairs of steps: P S, P' P) 65504, leave the range: infinities, which reach the
// result and are reported there.
//
// Steps in pairs: S, P and everything made of them commute, so with S the second
// step's S is P S P, and both steps are one product with X by P' P.  A call of five
// steps makes three passes over X instead of five.  P' P reaches a' a = 11.9, where
// fp16's last place is four times that at a: rounding it moves the singular values that a
// pair leaves near 1 by up to that much more, and the result's error is 2.2e-3 of itself
// instead of 2.0e-3.  Longer runs were less exact still (simulated, three steps at once:
// 1.44 times the bf16 rounding against 1.25).
//
// No transposes: the tensor core reads either operand with its reduction axis
// contiguous or strided (K-major or MN-major boxes).  S and P are symmetric: only
// their tiles on and above the diagonal are computed and stored, and where a
// product needs a tile below it, it loads the stored one with the axes exchanged
// (the majorness of an operand is chosen for every 64 of the reduction).
//
// The products run on CTA pairs (tcgen05 cta_group::2, 256 x 256 tiles) or, where
// there are few tiles, on single CTAs (128 x 128), with fp32 accumulators
// double-buffered in TMEM, persistent over all matrices' tiles:
//   warp 0     TMA producer (each CTA): 128B-swizzled boxes of 3-D maps, which
//              read zeros past a matrix's own rows and columns
//   warp 1     MMA issuer (of a pair: CTA 0's)
//   warps 2-9  epilogue: tcgen05.ld, the polynomial, rounding, and whole 32-byte
//              sectors stored by each lane into its own row
// A long Gram reduction of few tiles is split over clusters, and matrices with a
// side of at most 128 stay on chip from the first read to the last write.
//
// What bounds it, measured (five steps, graph replays): 128 x 2048 x 768 takes 1.90
// ms and 16 x 1536 x 4096 with momentum 1.63, of which the first pass over the
// gradient is 131 and 193 us at the copy rate.  The steps in pairs need 2.03e12
// operations; with tiles that reach past the diagonal the products execute 2.4e12, in
// the rest of the time 1.35e15 per second, against a library's 1.9e15 for one
// large product (1.7e15 once the part's power cap holds the clock near 1.5 GHz; back
// to back this update meets the cap too and takes 2.09 to 2.16 ms).  Symmetric products of
// few tiles lose the most: 70 us each at n = 768, with 300 MB moved.  Small calls
// are chains of dependent products of 4 to 6 us: 3 x 1000 x 333 takes 97 us, 8 x
// 128 x 64 on chip 25.
// Every wait is bounded; on a timeout the kernel flags the status word, drains
// its copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr float kSigma = 256.f;  // X is stored times this
constexpr int kMaxDim = 16384, kMaxBatch = 65535, kMaxSteps = 64;  // (at most 2^30 tiles of 128 x 128 in a product)

// ---------------------------------------------------------------- norms and the first X
//
// One pass over the update: the momentum is advanced, the squares are summed and X
// is written, before the norm is known: times a power of two taken from a sample of
// the gradient that every block reads, so that X's root mean square comes out near 1.
// The norm's factor enters the first step's products, where it is exact in fp32.
// Where the sample misled (X's root mean square is not within 2^-6 .. 2^10 of 1, or a
// value does not fit fp16), the second kernel, which otherwise only adds the
// sums, writes X again with a power of two from the norm.  Two passes over 128 x
// 2048 x 768 took 189 us, 16 x 1536 x 4096 with momentum 281; this one 131 and 194.

constexpr int kPrepThreads = 256;
constexpr int kPrepVecs = 8;        // 8-element groups a thread has in flight
constexpr int kPrepSingles = 16;    // or elements, where rows are not whole groups
constexpr int kRescaleBlocks = 4;   // blocks per matrix of the second kernel
constexpr float kFits = 60000.f;    // the largest value stored

struct PrepArgs {
  const void *g;
  float *mom;     // [B,R,C] or null
  float beta;
  bool nesterov;
  float eps;
  int64_t numel;  // R * C
  int C, ld;      // columns, and X's row stride
  int chunk;      // elements per block
  int chunks;     // blocks per matrix
  float *part;    // [B][chunks] sums of squares; negative where a value does not fit
  float *fac;     // [B] what X is to be multiplied with
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

__device__ __forceinline__ float block_sum(float v, float *s_w) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_w[0];
#pragma unroll
  for (int w = 1; w < kPrepThreads / 32; ++w) v += s_w[w];
  return v;
}

// The power of two that brings a root mean square of sqrt(sum / count) to 1 .. 2
// (1 where there is nothing to go by).  The quotient itself may be below fp32's range;
// the power is between 2^-64 and 2^89 for every finite sum.
__device__ __forceinline__ float power_for(float sum, float count) {
  if (!(sum > 0.f && sum < INFINITY)) return 1.f;
  return exp2f(-floorf(0.5f * (log2f(sum) - log2f(count))));
}

// u times f0 into X at element `at` of the matrix (8 elements or one).
template <bool VEC>
__device__ __forceinline__ void store_x(const PrepArgs &a, uint16_t *x, int64_t at, const float *u, float f0) {
  const int row = static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(a.C));  // R * C <= 2^28
  const int64_t dst = static_cast<int64_t>(row) * a.ld + (at - static_cast<int64_t>(row) * a.C);
  if constexpr (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(u[2 * i] * f0, u[2 * i + 1] * f0);
      memcpy(&w[i], &h, 4);
    }
    *reinterpret_cast<uint4 *>(x + dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    x[dst] = __half_as_ushort(__float2half_rn(u[0] * f0));
  }
}

// The scale that a matrix's blocks take from the sample: 8 elements per thread,
// spread evenly (or the whole matrix, where it is smaller).
template <class El, bool VEC>
__device__ __forceinline__ float sample_scale(const El *g, int64_t numel, float *s_w) {
  constexpr int N = VEC ? 8 : 1;
  const int64_t groups = numel / N;
  const int64_t at = groups > kPrepThreads ? groups * threadIdx.x / kPrepThreads : threadIdx.x;
  float f[N], sum = 0.f;
  const bool in = at < groups;
  if (in) {
    load_el<El, VEC>(g + at * N, f);
#pragma unroll
    for (int i = 0; i < N; ++i) sum = fmaf(f[i], f[i], sum);
  }
  const int64_t used = groups < kPrepThreads ? groups : kPrepThreads;
  return power_for(block_sum(sum, s_w), static_cast<float>(used * N));
}

// One chunk of one matrix.  VEC: rows are whole groups of eight.
template <class El, bool VEC, bool MOM>
__global__ void __launch_bounds__(kPrepThreads) ortho_prepare_kernel(const PrepArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s_w[kPrepThreads / 32];
  constexpr int N = VEC ? 8 : 1, U = VEC ? (MOM ? kPrepVecs / 2 : kPrepVecs) : kPrepSingles;
  const El *g = static_cast<const El *>(a.g) + blockIdx.y * a.numel;
  float *mom = MOM ? a.mom + blockIdx.y * a.numel : nullptr;
  uint16_t *x = a.x + blockIdx.y * a.x_stride;
  const float f0 = sample_scale<El, VEC>(g, a.numel, s_w);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * a.chunk + threadIdx.x * N;
  float acc = 0.f, most = 0.f;
#pragma unroll 1
  for (int it = 0; it < a.chunk / (kPrepThreads * N); it += U) {
    if (base + static_cast<int64_t>(it) * kPrepThreads * N >= a.numel) break;
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
      for (int i = 0; i < N; ++i) {
        acc = fmaf(f[u][i], f[u][i], acc);
        most = fmaxf(most, fabsf(f[u][i]));
      }
      if (at < a.numel) store_x<VEC>(a, x, at, f[u], f0);
    }
  }
  acc = block_sum(acc, s_w);
  // a value past fp16's range, marked by the sign (the sum itself is not negative,
  // and a NaN stays one)
  const bool fits = __syncthreads_and(!(most * f0 > kFits));
  if (threadIdx.x == 0)
    a.part[static_cast<size_t>(blockIdx.y) * a.chunks + blockIdx.x] = fits ? acc : -(acc == 0.f ? 1e-45f : acc);
}

// A matrix's factor from its sums; X again, by the blocks of the matrix, where the
// sample misled.
template <class El, bool VEC, bool MOM>
__global__ void __launch_bounds__(kPrepThreads) ortho_rescale_kernel(const PrepArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  __shared__ float s_w[kPrepThreads / 32];
  constexpr int N = VEC ? 8 : 1;
  const El *g = static_cast<const El *>(a.g) + blockIdx.y * a.numel;
  const float *part = a.part + static_cast<size_t>(blockIdx.y) * a.chunks;
  float sq = 0.f;  // the chunks in a fixed order
  bool fits = true;
  for (int i = threadIdx.x; i < a.chunks; i += kPrepThreads) {
    const float v = part[i];
    sq += fabsf(v);
    fits = fits && !(v < 0.f);
  }
  sq = block_sum(sq, s_w);
  fits = __syncthreads_and(fits);
  float f0 = sample_scale<El, VEC>(g, a.numel, s_w);
  const bool fine = isfinite(sq);
  const float rms = sqrtf(sq) * f0 / sqrtf(static_cast<float>(a.numel));
  if (fine && sq > 0.f && !(fits && rms >= 0x1p-6f && rms <= 0x1p10f)) {
    f0 = power_for(sq, static_cast<float>(a.numel));
    const float *mom = MOM ? a.mom + blockIdx.y * a.numel : nullptr;
    uint16_t *x = a.x + blockIdx.y * a.x_stride;
    for (int64_t at = (static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x) * N; at < a.numel;
         at += static_cast<int64_t>(gridDim.x) * kPrepThreads * N) {
      float f[N];
      load_el<El, VEC>(g + at, f);
      if constexpr (MOM) {
        float m[N];
        load_el<float, VEC>(mom + at, m);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = update_of(f[i], m[i], a.beta, a.nesterov);
      }
      store_x<VEC>(a, x, at, f, f0);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (!fine) flag_status(a.status, kDevNonfiniteUpdate);
    const float norm = fmaxf(sqrtf(sq), a.eps);
    a.fac[blockIdx.y] = fine ? (norm > 0.f ? kSigma / (norm * f0) : 0.f) : NAN;
  }
}

// ---------------------------------------------------------------- products

// CG CTAs work on a tile of 128 CG rows and columns: a pair (tcgen05 cta_group::2)
// or one alone, each with 128 rows of A and 128 columns of B in its shared memory.
// A tile of a pair takes half the operand bytes per operation; where a product has
// too few tiles for the part, one of a single CTA takes half the time.
constexpr int BM = 128;
constexpr int tile_size(int cg) { return BM * cg; }
constexpr int BK = 64;                // reduction elements per box: one 128-byte swizzle row
constexpr int kHalf = 128 * BK * 2;   // one operand's box (or two 64 x 64 boxes) per CTA: 16 KB
constexpr int kBox = 64 * 64 * 2;
constexpr int kStages = 3;
constexpr int kStageBytes = 4 * kHalf;  // two K blocks: [A k0 | A k1 | B k0 | B k1]
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;
constexpr int kTileBytes = 32 * 32 * 2;  // an epilogue warp's staging tile
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
  int nm, nn;             // tiles along the rows, along the columns
  int per;                // tiles per matrix (symmetric: mt <= nt)
  bool back;              // the matrices from the last one to the first
  float a, b, c;          // kSquare; c also the factor of the other products
  const float *fac;       // a matrix's factor besides c (the first step's X), or null
  bool sectors;           // kLast: every row of out starts on 32 bytes
  const uint16_t *s;      // kSquare: S
  uint16_t *out;
  int ld;                 // row stride of s and out
  int64_t stride;         // matrix stride of both
  int32_t *status;
};

struct TileAt {
  int b, m0, n0;
};

template <int KIND, int CG>
__device__ __forceinline__ TileAt tile_of(int tile, const ProductArgs &p) {
  constexpr int TS = tile_size(CG);
  TileAt t;
  t.b = tile / p.per;
  int r = tile - t.b * p.per;
  if (p.back) t.b = p.batch - 1 - t.b;
  if constexpr (KIND == kGram || KIND == kSquare) {
    int nt = 0;
    while (r > nt) r -= ++nt;
    t.m0 = r * TS;
    t.n0 = nt * TS;
  } else {
    const int mt = r / p.nn;
    t.m0 = mt * TS;
    t.n0 = (r - mt * p.nn) * TS;
  }
  return t;
}

// Byte offset of row r's 16-byte piece q (of 4) in a staging tile: the XOR keeps
// rows written by lanes and pieces read by rows free of bank conflicts.
__device__ __forceinline__ uint32_t swz(int r, int q) {
  return static_cast<uint32_t>(r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
}

// The same for rows of 128 bytes as the tensor core reads them (128B swizzle).
__device__ __forceinline__ uint32_t swz128(int r, int q) {
  return static_cast<uint32_t>(r * 128 + ((q ^ (r & 7)) << 4));
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

// One 32-byte sector (32-byte aligned) to or from a lane: whole sectors, although
// every lane has a row of its own.
__device__ __forceinline__ void ld_sector(const void *p, uint4 &a, uint4 &b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_sector(void *p, const uint4 &a, const uint4 &b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

constexpr int chunks_of(int cg) { return tile_size(cg) / 64; }  // 32-column chunks of a warp's half of the columns

// kSquare: S under the warp's 32 rows and half of the tile's columns, a row per
// lane as the accumulator comes: its 64-byte pieces are whole sectors.
template <int CG>
struct SChunks {
  static constexpr int kChunks = chunks_of(CG), TS = tile_size(CG);
  uint4 v[kChunks][4];
  __device__ __forceinline__ void load(const TileAt &t, int row0, int part, const ProductArgs &p) {
    const int lane = threadIdx.x & 31;
    const uint16_t *s = p.s + t.b * p.stride + (row0 + lane) * static_cast<int64_t>(p.ld) + t.n0 + part * (TS / 2);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const bool in = row0 + lane < p.M && t.n0 + part * (TS / 2) + 32 * j < p.N;
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        v[j][i] = v[j][i + 1] = make_uint4(0, 0, 0, 0);
        if (in) ld_sector(s + 32 * j + 8 * i, v[j][i], v[j][i + 1]);
      }
    }
  }
};

// Flags a result that is not finite.  What left fp16's range on the way is infinite
// there and reaches the result: every product multiplies it with something, if only
// with zero.  v times 0 is 0 of a finite value and a NaN of any other.
__device__ __forceinline__ void report_bad(const float (&v)[32], int32_t *status) {
  float bad = 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) bad = fmaf(v[e], 0.f, bad);
  if (bad != bad) flag_status(status, kDevNonfiniteUpdate);
}

// One warp's 32 rows of half a tile's columns.
template <int KIND, int CG>
__device__ __forceinline__ void epilogue(const TileAt &t, uint32_t tb, int row0, int part, const ProductArgs &p,
                                         uint8_t *tile, const SChunks<CG> &sc) {
  constexpr int kChunks = chunks_of(CG), TS = tile_size(CG);
  const int lane = threadIdx.x & 31;
  const int nrows = min(32, p.M - row0);
  uint16_t *out = p.out + t.b * p.stride;
  float c = p.c;
  if (KIND != kSquare && p.fac) {
    const float f = p.fac[t.b];
    c *= KIND == kGram ? f * f : f;
  }
#pragma unroll KIND == kSquare ? kChunks : 1
  for (int j = 0; j < kChunks; ++j) {
    const int cc = part * (TS / 2) + 32 * j, c0 = t.n0 + cc;
    if (c0 >= p.N || nrows <= 0) break;
    uint32_t acc[32];
    tmem_ld32(tb + cc, acc);
    float v[32];
    if constexpr (KIND == kSquare) {
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = sc.v[j][q];
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
    } else {
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(acc[e]) * c;
    }
    if constexpr (KIND == kLast) {  // out [M,N] itself, bf16
      report_bad(v, p.status);
      const int ncols = min(32, p.N - c0);
      uint16_t *g0 = out + row0 * static_cast<int64_t>(p.ld) + c0;
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                          pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
      if (p.sectors) {
        if (lane < nrows) {
          uint16_t *row = g0 + lane * static_cast<int64_t>(p.ld);
          st_sector(row, w[0], w[1]);
          if (ncols > 16) st_sector(row + 16, w[2], w[3]);
        }
        continue;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(tile + swz(lane, q)) = w[q];
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
    } else if (lane < nrows) {  // padded rows: whole chunks, a row per lane
      uint16_t *g0 = out + (row0 + lane) * static_cast<int64_t>(p.ld) + c0;
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = make_uint4(pack_half2(v[8 * q], v[8 * q + 1]), pack_half2(v[8 * q + 2], v[8 * q + 3]),
                          pack_half2(v[8 * q + 4], v[8 * q + 5]), pack_half2(v[8 * q + 6], v[8 * q + 7]));
      st_sector(g0, w[0], w[1]);
      st_sector(g0 + 16, w[2], w[3]);
    }
  }
}

// How one operand is read.  kK: its reduction axis is contiguous; kMN: its other
// axis is; kSym: it is symmetric and stored on and above the diagonal of its
// tiles, so contiguous from the diagonal tile on, the other way before it.
enum Major : int { kK = 0, kMN = 1, kSym = 2 };
template <int MAJOR>
__device__ __forceinline__ bool mn_major(int k0, int tile0) {
  return MAJOR == kMN || (MAJOR == kSym && k0 < tile0);
}

// One K block of one operand into this CTA's half of the stage: 128 rows x 64 of
// K (one box), or 64 of K x 128 columns in two boxes.
template <int MAJOR, int CG>
__device__ __forceinline__ void load_operand(uint8_t *dst, const CUtensorMap *map, const CUtensorMap *map_mn,
                                             uint64_t *bar, uint32_t bar0, int k0, int tile0, int r0, int b) {
  auto load = [&](uint8_t *to, const CUtensorMap *m, int x, int y) {
    if constexpr (CG == 2)
      tma_load_3d_pair(to, m, bar0, x, y, b);
    else
      tma_load_3d(to, m, bar, x, y, b);
  };
  if (mn_major<MAJOR>(k0, tile0)) {
    load(dst, map_mn, r0, k0);
    load(dst + kBox, map_mn, r0 + 64, k0);
  } else {
    load(dst, map, k0, r0);
  }
}

// Descriptor of the j-th 16 of K of a block at shared address s.
__device__ __forceinline__ uint64_t operand_desc(uint32_t s, int j, bool mn) {
  return mn ? smem_desc_sw128(s + j * 2048, kBox, 1024) : smem_desc_sw128(s + j * 32, 16, 1024);
}

template <int KIND, int AM, int BMAJ, int CG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ortho_product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmAmn,
                         const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmBmn,
                         const ProductArgs p) {
  constexpr int TS = tile_size(CG);
  constexpr uint32_t kTmemCols = 2 * TS;
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
  const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const int group = blockIdx.x / CG, ngroups = gridDim.x / CG;
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
    tma_prefetch_desc(AM == kMN ? &tmAmn : &tmA);
    tma_prefetch_desc(BMAJ == kMN ? &tmBmn : &tmB);
  }
  if (warp == 1) {
    if constexpr (CG == 2)
      tmem_alloc_pair(tmem_slot, kTmemCols);
    else
      tmem_alloc(tmem_slot, kTmemCols);
  }
  griddep_wait();  // the set-up above overlaps the previous kernel's end; its outputs are read below
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // both CTAs' barriers initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = p.batch * p.per;
  const int nkb = (p.K + BK - 1) / BK, nstage = (nkb + 1) / 2;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = CG == 2 ? peer_smem_addr(&full[0], 0) : 0;
      int stage = 0;
      uint32_t phase = 0, armed = 0, arm_par = 0;
      bool ok = true;
      for (int tile = group; tile < total && ok; tile += ngroups) {
        const TileAt t = tile_of<KIND, CG>(tile, p);
        for (int ks = 0; ks < nstage; ++ks) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t *sa = smem + stage * kStageBytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * kStageBytes);  // the group's bytes
          // a K block past the end is zero fill, and no MMA reads it
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k0 = (ks * 2 + h) * BK;
            load_operand<AM, CG>(sa + h * kHalf, &tmA, &tmAmn, &full[stage], full0 + 8u * stage, k0, t.m0,
                                 t.m0 + BM * rank, t.b);
            load_operand<BMAJ, CG>(sa + (2 + h) * kHalf, &tmB, &tmBmn, &full[stage], full0 + 8u * stage, k0, t.n0,
                                   t.n0 + BM * rank, t.b);
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
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = group; tile < total && ok; tile += ngroups, ++it) {
        const TileAt t = tile_of<KIND, CG>(tile, p);
        const int buf = it & 1;
        if (!mbar_wait(&tempty[buf], ((it >> 1) & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * TS;
        for (int ks = 0; ks < nstage; ++ks) {
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
              const int k0 = (ks * 2 + h) * BK;
              const bool amn = mn_major<AM>(k0, t.m0), bmn = mn_major<BMAJ>(k0, t.n0);
              const uint32_t idesc = idesc_f16(TS, TS, amn, bmn);
#pragma unroll
              for (int j = 0; j < BK / 16; ++j)
                mma(d, operand_desc(ab + h * kHalf, j, amn), operand_desc(bb + h * kHalf, j, bmn), idesc,
                    (ks | h | j) != 0 ? 1u : 0u);
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
    const int part = (warp - 2) >> 2;     // column half
    const uint32_t tempty0 = CG == 2 ? peer_smem_addr(&tempty[0], 0) : 0;
    uint8_t *stile = epi_tiles + (warp - 2) * kTileBytes;
    int it = 0;
    for (int tile = group; tile < total; tile += ngroups, ++it) {
      const TileAt t = tile_of<KIND, CG>(tile, p);
      const int buf = it & 1, row0 = t.m0 + BM * rank + q * 32;
      SChunks<CG> sc;
      if constexpr (KIND == kSquare) sc.load(t, row0, part, p);  // while the product runs
      if (!wait_lane0(&tfull[buf], (it >> 1) & 1, abort_flag)) break;
      __syncwarp();
      tc_fence_after();
      epilogue<KIND, CG>(t, tmem_base + buf * TS + (static_cast<uint32_t>(q * 32) << 16), row0, part, p, stile, sc);
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

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) flag_status(p.status, kDevWaitTimeout);
  if constexpr (CG == 2) cluster_sync();  // the pair is done with each other's barriers and TMEM
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
  }
}

// After a wait has run out: time (bounded) for copies and MMAs in flight to end
// before shared memory and TMEM are given up.
__device__ __forceinline__ void settle() {
  const long long t0 = clock64();
  while (clock64() - t0 < 20000000LL) {
  }
}

// ---------------------------------------------------------------- small matrices
//
// n <= 128: a cluster of CTAs keeps a whole matrix in shared memory from the first
// read to the last write, one launch for the call.  Each CTA holds all n rows (of X,
// or of its transpose when R > C) of up to 256 of the m columns, in blocks of 64
// columns (128 rows of 128 bytes, 128B-swizzled).  Such a block is a K-major operand
// of the Gram product and, unchanged, an MN-major one of the update.  The Gram
// product's partial sums meet through distributed shared memory, each CTA adding a
// share of the rows in the order of the CTAs; S, P and the update are then each
// CTA's own.  What bounds it is the chain of dependent steps: three products, three
// passes TMEM -> registers -> shared memory and two cluster barriers per step.

constexpr int kSmallN = 128, kSlab = 256;     // rows, and columns per CTA at most
constexpr int kSmallCluster = 16;             // CTAs per matrix at most
constexpr int kSmallThreads = 256;
constexpr int kBlk = 128 * 128;               // bytes of a block
constexpr int kPartStride = kSmallN + 4;      // floats of a row of partial sums
constexpr int kSmallS = (kSlab / 64) * kBlk;  // S, then P: two blocks
constexpr int kSmallPart = kSmallS + 2 * kBlk;
constexpr int small_smem(int cluster) {
  return kSmallPart + (cluster > 1 ? kSmallN * kPartStride * 4 : 0) + 1024 /*align*/;
}
static_assert(small_smem(2) <= 227 * 1024, "shared memory budget");

struct SmallArgs {
  const void *g;
  float *mom;
  uint16_t *out;
  int R, C, n, m;
  int cluster, nblk;  // CTAs per matrix, blocks of 64 columns per CTA
  bool tall, vec;     // R > C; rows of g are whole groups of eight
  float beta, eps, scale;
  bool nesterov;
  int steps;
  int32_t *status;
  float coefs[3 * kMaxSteps];
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32x2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Byte of element (row, column c) in blocks of 64 columns.
__device__ __forceinline__ uint32_t blk_byte(int row, int c) {
  return static_cast<uint32_t>((c >> 6) * kBlk) + swz128(row, (c >> 3) & 7) + (c & 7) * 2;
}

template <class El>
__global__ void __launch_bounds__(kSmallThreads, 2) ortho_small_kernel(const __grid_constant__ SmallArgs p) {
  griddep_wait();  // the previous kernel in the stream has completed
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float s_red[kSmallThreads / 32], s_sq;
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *xs = smem, *ss = smem + kSmallS;
  float *part = reinterpret_cast<float *>(smem + kSmallPart);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int b = blockIdx.x / p.cluster;
  const int c0 = rank * p.nblk * 64, cols = max(0, min(p.nblk * 64, p.m - c0));  // this CTA's columns
  const int64_t numel = static_cast<int64_t>(p.R) * p.C;
  const El *g = static_cast<const El *>(p.g) + b * numel;
  float *mom = p.mom ? p.mom + b * numel : nullptr;

  if (threadIdx.x == 0) {
    mbar_init(&s_bar, 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&s_tmem, kSlab);
  // rows past n and columns past m stay zero
  for (int i = threadIdx.x; i < kSmallPart / 16; i += kSmallThreads)
    reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // this CTA's elements in memory order: rows of `width` elements, `stride` apart
  const int rows = p.tall ? cols : p.n, width = p.tall ? p.n : cols;
  const int64_t base = p.tall ? static_cast<int64_t>(c0) * p.C : c0;
  // i / d for i < 2^15 and d <= 256, from 1 / d: what the half keeps from a whole
  // number, 2^-9 at least, is above what i / d rounds away
  auto quotient = [](int i, float inv_d) { return static_cast<int>((static_cast<float>(i) + 0.5f) * inv_d); };
  // pass 0: advance the momentum and sum the squares; pass 1: store the scaled
  // elements.  Groups of eight or, in rows that are not whole groups, single elements,
  // 16 of them in flight (20 x 100 x 252: 75 us, against 39 for 20 x 128 x 256 in groups;
  // with few in flight, and rows stored by the lanes that hold them, 102)
  auto pass_over = [&](auto vec, int pass, float f0) {
    constexpr int N = decltype(vec)::value ? 8 : 1, U = decltype(vec)::value ? 4 : 16;  // U loads in flight
    float acc = 0.f;
    const int per = width / N, total = rows * per;
    const float inv_per = 1.f / static_cast<float>(per);
    for (int i0 = threadIdx.x; i0 < total; i0 += kSmallThreads * U) {
      float f[U][N], mm[U][N];
      int rr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kSmallThreads;
        if (i >= total) break;
        rr[u] = quotient(i, inv_per);
        const int64_t at = base + static_cast<int64_t>(rr[u]) * p.C + (i - rr[u] * per) * N;
        load_el<El, N == 8>(g + at, f[u]);
        if (mom) load_el<float, N == 8>(mom + at, mm[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kSmallThreads;
        if (i >= total) break;
        const int r = rr[u], c = (i - r * per) * N;
        if (mom) {
          float *m = mom + base + static_cast<int64_t>(r) * p.C + c;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            if (pass == 0) m[k] = mm[u][k] = fmaf(p.beta, mm[u][k], f[u][k]);
            f[u][k] = update_of(f[u][k], mm[u][k], p.beta, p.nesterov);
          }
        }
        if (pass == 0) {
#pragma unroll
          for (int k = 0; k < N; ++k) acc = fmaf(f[u][k], f[u][k], acc);
        } else if (N == 1 || p.tall) {
#pragma unroll
          for (int k = 0; k < N; ++k)
            *reinterpret_cast<uint16_t *>(xs + (p.tall ? blk_byte(c + k, r) : blk_byte(r, c + k))) =
                __half_as_ushort(__float2half_rn(f[u][k] * f0));
        } else {  // eight columns are one piece of 16 bytes
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = pack_half2(f[u][2 * k % N] * f0, f[u][(2 * k + 1) % N] * f0);
          *reinterpret_cast<uint4 *>(xs + blk_byte(r, c)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    return acc;
  };
  auto each = [&](int pass, float f0) {
    return p.vec ? pass_over(std::true_type{}, pass, f0) : pass_over(std::false_type{}, pass, f0);
  };
  float sq = warp_sum(each(0, 0.f));
  if (lane == 0) s_red[warp] = sq;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kSmallThreads / 32; ++w) sq += s_red[w];
    s_sq = sq;
  }
  __syncthreads();
  if (p.cluster > 1) {
    cluster_sync();
    sq = 0.f;
    for (int r = 0; r < p.cluster; ++r) sq += ld_cluster_f32(peer_smem_addr(&s_sq, r));
  } else {
    sq = s_sq;
  }
  const bool fine = isfinite(sq);
  if (!fine && rank == 0 && threadIdx.x == 0) flag_status(p.status, kDevNonfiniteUpdate);
  const float norm = fmaxf(sqrtf(sq), p.eps);
  each(1, fine ? (norm > 0.f ? kSigma / norm : 0.f) : NAN);
  fence_async();
  __syncthreads();

  // a product's MMAs by one thread, and the wait for them by all (a wait that runs
  // out is flagged; the kernel goes on, so that no barrier misses a thread)
  uint32_t phase = 0;
  auto product = [&](auto &&issue) {
    if (threadIdx.x == 0) {
      tc_fence_after();
      issue();
      tc_commit(&s_bar);
    }
    if (!mbar_wait(&s_bar, phase, &s_abort) && lane == 0) flag_status(p.status, kDevWaitTimeout);
    phase ^= 1;
    __syncwarp();
    tc_fence_after();
  };
  const int kn = p.n <= 64 ? 1 : 2;  // blocks of 64 that hold n
  const uint32_t xa = smem_addr(xs), sa = smem_addr(ss);
  const int q = warp & 3, half = warp >> 2, row = q * 32 + lane;
  const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);

  for (int step = 0; step < p.steps; ++step) {
    const float ca = p.coefs[3 * step], cb = p.coefs[3 * step + 1], cc = p.coefs[3 * step + 2];
    const float own = 0.5f * ca;  // X's own part of the update, which P leaves out
    // S = X X^T / sigma^2
    product([&] {
      for (int k = 0; k < p.nblk; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t d = smem_desc_sw128(xa + k * kBlk + j * 32, 16, 1024);
          tc_mma_f16_one(tmem, d, d, idesc_f16(128, 128, 0, 0), (k | j) != 0 ? 1u : 0u);
        }
    });
    constexpr float inv = 1.f / (kSigma * kSigma);
    if (half < kn) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t acc[32];
        tmem_ld32(tq + half * 64 + h * 32, acc);
        tmem_ld_wait();
        if (p.cluster > 1) {
          float4 *dst = reinterpret_cast<float4 *>(part + row * kPartStride + half * 64 + h * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(__uint_as_float(acc[4 * e]), __uint_as_float(acc[4 * e + 1]),
                                 __uint_as_float(acc[4 * e + 2]), __uint_as_float(acc[4 * e + 3]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_half2(__uint_as_float(acc[8 * e + 2 * k]) * inv, __uint_as_float(acc[8 * e + 2 * k + 1]) * inv);
            *reinterpret_cast<uint4 *>(ss + half * kBlk + swz128(row, h * 4 + e)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
    tc_fence_before();
    if (p.cluster > 1) {
      cluster_sync();  // every CTA's partial sums are there
      // this CTA's share of the rows: 128 / cluster, four columns at a time, 16 loads
      // in flight (20 x 128 x 512: 52 us; one row at a time 58)
      auto add_parts = [&](auto ctas, auto rows_at_once) {
        constexpr int CC = decltype(ctas)::value, U = decltype(rows_at_once)::value;
        const int groups = kn * 16, total = kSmallN / p.cluster * groups;
        for (int i0 = threadIdx.x; i0 < total; i0 += kSmallThreads * U) {
          float4 t[U];
#pragma unroll
          for (int u = 0; u < U; ++u) t[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int o0 = 0; o0 < p.cluster; o0 += CC) {
            float4 v[U][CC];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int i = min(i0 + u * kSmallThreads, total - 1);
              const int r = rank * (kSmallN / p.cluster) + i / groups, c = i % groups * 4;
#pragma unroll
              for (int o = 0; o < CC; ++o) v[u][o] = ld_cluster_f32x4(peer_smem_addr(part + r * kPartStride + c, o0 + o));
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int o = 0; o < CC; ++o)
                t[u].x += v[u][o].x, t[u].y += v[u][o].y, t[u].z += v[u][o].z, t[u].w += v[u][o].w;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kSmallThreads;
            if (i >= total) break;
            const int r = rank * (kSmallN / p.cluster) + i / groups, c = i % groups * 4;
            const uint32_t lo = pack_half2(t[u].x * inv, t[u].y * inv), hi = pack_half2(t[u].z * inv, t[u].w * inv);
            for (int o = 0; o < p.cluster; ++o) st_cluster_u32x2(peer_smem_addr(ss + blk_byte(r, c), o), lo, hi);
          }
        }
      };
      const std::integral_constant<int, 1> one;
      const std::integral_constant<int, 2> two;
      const std::integral_constant<int, 4> four;
      const std::integral_constant<int, 8> eight;
      if (p.cluster == 2)
        add_parts(two, eight);
      else if (p.cluster == 4)
        add_parts(four, four);
      else if (p.cluster == 8)
        add_parts(eight, two);
      else
        add_parts(eight, one);
      fence_async();
      cluster_sync();
    }
    fence_async();
    __syncthreads();
    // P = a/2 I + b S + c S S, in S's place: P's diagonal runs from a down to about 1, so
    // that its rounding is smaller with half of a taken out (the result of 13 x 94 x 33
    // is off by 2.1e-3 instead of 2.5e-3 of itself, bf16 alone by 1.7e-3, for 1 us)
    product([&] {
      for (int k = 0; k < kn; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t d = smem_desc_sw128(sa + k * kBlk + j * 32, 16, 1024);
          tc_mma_f16_one(tmem, d, d, idesc_f16(128, 128, 0, 0), (k | j) != 0 ? 1u : 0u);
        }
    });
    if (half < kn) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t acc[32];
        tmem_ld32(tq + half * 64 + h * 32, acc);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 *at = reinterpret_cast<uint4 *>(ss + half * kBlk + swz128(row, h * 4 + e));
          const uint4 sv = *at;
          const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            __half2 hh;
            memcpy(&hh, &sw[k], 4);
            const float2 f = __half22float2(hh);
            const int c = half * 64 + h * 32 + 8 * e + 2 * k;
            const float v0 = fmaf(cc, __uint_as_float(acc[8 * e + 2 * k]), cb * f.x) + (c == row ? ca - own : 0.f);
            const float v1 = fmaf(cc, __uint_as_float(acc[8 * e + 2 * k + 1]), cb * f.y) + (c + 1 == row ? ca - own : 0.f);
            w[k] = pack_half2(v0, v1);
          }
          *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    tc_fence_before();
    fence_async();
    __syncthreads();
    // X <- a/2 X + P X
    product([&] {
      for (int k = 0; k < kn; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc_mma_f16_one(tmem, smem_desc_sw128(sa + k * kBlk + j * 32, 16, 1024),
                         smem_desc_sw128(xa + (k * 64 + j * 16) * 128, kBlk, 1024),
                         idesc_f16(128, 64 * p.nblk, 0, 1), (k | j) != 0 ? 1u : 0u);
    });
    const bool last = step + 1 == p.steps;
    for (int k = half; k < p.nblk; k += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t acc[32];
        tmem_ld32(tq + k * 64 + h * 32, acc);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 xv = *reinterpret_cast<const uint4 *>(xs + k * kBlk + swz128(row, h * 4 + e));
          const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __half2 hh;
            memcpy(&hh, &xw[i], 4);
            const float2 f = __half22float2(hh);
            acc[8 * e + 2 * i] = __float_as_uint(fmaf(own, f.x, __uint_as_float(acc[8 * e + 2 * i])));
            acc[8 * e + 2 * i + 1] = __float_as_uint(fmaf(own, f.y, __uint_as_float(acc[8 * e + 2 * i + 1])));
          }
        }
        if (!last) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_half2(__uint_as_float(acc[8 * e + 2 * i]), __uint_as_float(acc[8 * e + 2 * i + 1]));
            *reinterpret_cast<uint4 *>(xs + k * kBlk + swz128(row, h * 4 + e)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (row < p.n) {
          const float f = p.scale / kSigma;
          const int c = c0 + k * 64 + h * 32;  // column of X
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(acc[e]) * f;
          report_bad(v, p.status);
          uint16_t *out = p.out + b * numel;
          if (p.tall) {  // row c + e of out, column `row`: contiguous over the lanes
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e < p.m)
                out[static_cast<int64_t>(c + e) * p.C + row] =
                    __bfloat16_as_ushort(__float2bfloat16_rn(v[e]));
          } else {
            uint16_t *o = out + static_cast<int64_t>(row) * p.C + c;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(v[8 * e + 2 * i], v[8 * e + 2 * i + 1]);
              if (!p.vec)  // rows that start anywhere: through X's place, below
                *reinterpret_cast<uint4 *>(xs + k * kBlk + swz128(row, h * 4 + e)) = make_uint4(w[0], w[1], w[2], w[3]);
              else if (c + 8 * e < p.m)
                *reinterpret_cast<uint4 *>(o + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
    tc_fence_before();
    fence_async();
    __syncthreads();
  }
  if (!p.vec && !p.tall) {
    uint16_t *out = p.out + b * numel + c0;
    const float inv_cols = 1.f / static_cast<float>(cols);
#pragma unroll 8
    for (int i = threadIdx.x; i < p.n * cols; i += kSmallThreads) {
      const int r = quotient(i, inv_cols), c = i - r * cols;
      out[static_cast<int64_t>(r) * p.C + c] = *reinterpret_cast<const uint16_t *>(xs + blk_byte(r, c));
    }
  }
  if (threadIdx.x == 0 && s_abort) settle();
  __syncthreads();
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another may read it
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kSlab);
  }
}

// ---------------------------------------------------------------- Gram products of few tiles
//
// A Gram product reduces over the long side and has only the short side's tiles: two
// 520 x 2452 matrices are 30 tiles of 20 stages each on 152 SMs.  Here a cluster of
// `split` CTAs works on one tile of 128 x 128, each on a share of the reduction; the
// partial sums (in the operand ring, free by then) meet through distributed shared
// memory, each CTA adding a share of the rows in the order of the CTAs.
constexpr int kSplitThreads = 256, kMaxSplit = 8;
constexpr int kSplitStride = BM + 4;  // floats of a row of partial sums
static_assert(BM * kSplitStride * 4 <= kStages * kStageBytes, "the partial sums fit the ring");
constexpr int kSplitSmem = kStages * kStageBytes + 1024 /*align*/;

template <int MAJOR>
__global__ void __launch_bounds__(kSplitThreads, 1)
    ortho_gram_split_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_mn,
                            const ProductArgs p, int split) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t *smem =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float *part = reinterpret_cast<float *>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 1);
    }
    mbar_init(&s_done, 1);
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(MAJOR == kMN ? &tm_mn : &tm);
  }
  if (warp == 1) tmem_alloc(&s_tmem, BM);
  griddep_wait();  // the set-up above overlaps the previous kernel's end; its outputs are read below
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const TileAt t = tile_of<kGram, 1>(static_cast<int>(blockIdx.x) / split, p);
  const int nkb = (p.K + BK - 1) / BK, nst = (nkb + 1) / 2;
  const int st0 = nst * rank / split, st1 = nst * (rank + 1) / split;  // this CTA's stages
  // (a wait that runs out is flagged; the kernel goes on, so that no barrier misses a thread)
  if (warp == 0 && lane == 0) {
    for (int st = st0; st < st1; ++st) {
      const int i = (st - st0) % kStages;
      if (!mbar_wait(&s_empty[i], (((st - st0) / kStages) & 1) ^ 1, &s_abort)) break;
      mbar_arrive_expect_tx(&s_full[i], kStageBytes);
      uint8_t *sa = smem + i * kStageBytes;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k0 = (st * 2 + h) * BK;
        load_operand<MAJOR, 1>(sa + h * kHalf, &tm, &tm_mn, &s_full[i], 0, k0, t.m0, t.m0, t.b);
        load_operand<MAJOR, 1>(sa + (2 + h) * kHalf, &tm, &tm_mn, &s_full[i], 0, k0, t.n0, t.n0, t.b);
      }
    }
  } else if (warp == 1 && lane == 0) {
    for (int st = st0; st < st1; ++st) {
      const int i = (st - st0) % kStages;
      if (!mbar_wait(&s_full[i], ((st - st0) / kStages) & 1, &s_abort)) break;
      tc_fence_after();
      const uint32_t ab = smem_addr(smem + i * kStageBytes), bb = ab + 2 * kHalf;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (st * 2 + h < nkb) {
#pragma unroll
          for (int j = 0; j < BK / 16; ++j)
            tc_mma_f16_one(tmem, operand_desc(ab + h * kHalf, j, MAJOR == kMN),
                           operand_desc(bb + h * kHalf, j, MAJOR == kMN),
                           idesc_f16(BM, BM, MAJOR == kMN, MAJOR == kMN), ((st - st0) | h | j) != 0 ? 1u : 0u);
        }
      tc_commit(&s_empty[i]);
    }
    tc_commit(&s_done);
  }
  __syncwarp();
  if (!mbar_wait(&s_done, 0, &s_abort) && lane == 0) flag_status(p.status, kDevWaitTimeout);
  __syncwarp();
  tc_fence_after();
  {
    const int q = warp & 3, half = warp >> 2, row = q * 32 + lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t acc[32];
      tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 64 + h * 32, acc);
      tmem_ld_wait();
      float4 *dst = reinterpret_cast<float4 *>(part + row * kSplitStride + half * 64 + h * 32);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dst[e] = make_float4(__uint_as_float(acc[4 * e]), __uint_as_float(acc[4 * e + 1]),
                             __uint_as_float(acc[4 * e + 2]), __uint_as_float(acc[4 * e + 3]));
    }
  }
  tc_fence_before();
  cluster_sync();  // every CTA's partial sums are there
  float c = p.c;
  if (p.fac) c *= p.fac[t.b] * p.fac[t.b];
  uint16_t *out = p.out + t.b * p.stride;
  const int share = BM / split;
  for (int i = threadIdx.x; i < share * (BM / 8); i += kSplitThreads) {
    const int r = rank * share + i / (BM / 8), c8 = i % (BM / 8) * 8;
    if (t.m0 + r >= p.M || t.n0 + c8 >= p.ld) continue;
    float4 v[kMaxSplit][2];
#pragma unroll
    for (int o = 0; o < kMaxSplit; ++o)
      if (o < split) {
        const uint32_t at = peer_smem_addr(part + r * kSplitStride + c8, o);
        v[o][0] = ld_cluster_f32x4(at);
        v[o][1] = ld_cluster_f32x4(at + 16);
      }
#pragma unroll
    for (int o = 1; o < kMaxSplit; ++o)
      if (o < split) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[0][h].x += v[o][h].x, v[0][h].y += v[o][h].y, v[0][h].z += v[o][h].z, v[0][h].w += v[o][h].w;
      }
    *reinterpret_cast<uint4 *>(out + (t.m0 + r) * static_cast<int64_t>(p.ld) + t.n0 + c8) =
        make_uint4(pack_half2(v[0][0].x * c, v[0][0].y * c), pack_half2(v[0][0].z * c, v[0][0].w * c),
                   pack_half2(v[0][1].x * c, v[0][1].y * c), pack_half2(v[0][1].z * c, v[0][1].w * c));
  }
  if (threadIdx.x == 0 && s_abort) settle();
  cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, BM);
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

// A matrix's maps: boxes of 128 rows x 64 columns (K-major) and of 64 x 64 (MN-major).
struct Maps {
  CUtensorMap k, mn;
};

template <int KIND, int AM, int BMAJ, int CG>
cudaError_t launch_groups(const Maps &a, const Maps &b, ProductArgs p, int sms, cudaStream_t s) {
  static DeviceOnce once;  // the shared-memory opt-in, and how many groups of CTAs fit at once
  auto kernel = ortho_product_kernel<KIND, AM, BMAJ, CG>;
  int groups = 0;
  const cudaError_t e = once.get(
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
      &groups);
  if (e != cudaSuccess) return e;
  constexpr int TS = tile_size(CG);
  p.nm = (p.M + TS - 1) / TS;
  p.nn = (p.N + TS - 1) / TS;
  p.per = KIND == kGram || KIND == kSquare ? p.nn * (p.nn + 1) / 2 : p.nm * p.nn;
  const int64_t tiles = static_cast<int64_t>(p.per) * p.batch;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(CG * (tiles < groups ? tiles : groups))), dim3(kGemmThreads),
                    kGemmSmem, s, CG, a.k, a.mn, b.k, b.mn, p);
}

// CTAs per tile of a Gram product; 1: no split.  The exchange costs about 5 us, so
// only reductions from kSplitStages stages of 128 on are split, over the CTAs that
// the tiles leave idle.  Measured, split and not: 1 x 4000 x 400 134 and 161 us,
// 1 x 1024 x 4096 184 and 200, 2 x 520 x 2452 156 and 163; but 3 x 1000 x 333 110 and
// 102, 1 x 768 x 768 120 and 113 (both sides of 1 x 2048 x 768 the same).
constexpr int kSplitStages = 17;
int gram_split(int batch, int n, int m, int sms) {
  const int64_t t = (n + BM - 1) / BM, tiles = batch * t * (t + 1) / 2;
  int split = 1;
  if ((m + 2 * BK - 1) / (2 * BK) >= kSplitStages)
    while (split < kMaxSplit && 2 * split * tiles <= sms) split *= 2;
  return split;
}

template <int MAJOR>
cudaError_t launch_gram_split(const Maps &x, ProductArgs p, int split, cudaStream_t s) {
  static DeviceOnce once;
  auto kernel = ortho_gram_split_kernel<MAJOR>;
  const cudaError_t e = once.get(
      [&](int *) { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplitSmem); });
  if (e != cudaSuccess) return e;
  p.nm = p.nn = (p.N + BM - 1) / BM;
  p.per = p.nn * (p.nn + 1) / 2;
  return launch_pdl(kernel, dim3(p.per * p.batch * split), dim3(kSplitThreads), kSplitSmem, s, split, x.k, x.mn, p,
                    split);
}

template <int KIND, int AM, int BMAJ>
cudaError_t launch_product(const Maps &a, const Maps &b, const ProductArgs &p, bool pair, int sms, cudaStream_t s) {
  return pair ? launch_groups<KIND, AM, BMAJ, 2>(a, b, p, sms, s) : launch_groups<KIND, AM, BMAJ, 1>(a, b, p, sms, s);
}

// Pairs of CTAs or single ones, by the rounds of tiles that a step's products take
// on the part's SMs.  A round's length in units of 128 of the reduction, from timings: K + 4
// for pairs, 0.8 K + 2 for single CTAs (half the MMA and epilogue work, but nearly
// the same operand stream).  Both measured: 3 x 1000 x 333 144 us in pairs, 110 in
// single CTAs; 100 x 256 x 256 183 and 131; 4 x 768 x 1536 188 and 157; but
// 8 x 768 x 1536 216 and 244, 24 x 1024 x 1024 538 and 652, 128 x 2048 x 768 2.0 and
// 2.4 ms.
bool use_pairs(int batch, int R, int C, int sms) {
  const int n = R < C ? R : C, m = R < C ? C : R;
  double cost[2];
  for (int cg = 1; cg <= 2; ++cg) {
    const int ts = tile_size(cg), groups = sms / cg;
    auto tiles = [&](int x) { return static_cast<int64_t>((x + ts - 1) / ts); };
    auto rounds = [&](int64_t per) { return static_cast<double>((per * batch + groups - 1) / groups); };
    auto length = [&](int k) { return cg == 2 ? k / 128.0 + 4 : 0.8 * k / 128.0 + 2; };
    const double sym = rounds(tiles(n) * (tiles(n) + 1) / 2), apply = rounds(tiles(R) * tiles(C));
    cost[cg - 1] = sym * length(m) + (sym + apply) * length(n);
  }
  return cost[1] <= cost[0];
}

bool ortho_ok(const moe_ortho_config *c) {
  if (!c || c->batch < 0 || c->batch > kMaxBatch || c->R < 1 || c->R > kMaxDim || c->C < 1 || c->C > kMaxDim)
    return false;
  if (c->steps < 1 || c->steps > kMaxSteps || !(c->eps >= 0.f)) return false;
  return c->dtype == MOE_DTYPE_BF16 || c->dtype == MOE_DTYPE_FP32;
}

// The workspace's size goes by the rules below, and must be known without a GPU: they
// take GB300's SMs as they were measured, not the present part's.
constexpr int kRuleSms = 152;

// Whether clusters hold the matrices on chip.
bool is_small(const moe_ortho_config *c) {
  const int n = std::min(c->R, c->C), m = std::max(c->R, c->C), cluster = (m + kSlab - 1) / kSlab;
  // up to two CTAs per matrix any number of matrices (608 x 128 x 256: 100 against 444
  // us, 304 x 128 x 512: 222 against 305); more only while all matrices are on the part
  // at once (38 x 128 x 1024: 110 against 125 us, but 76 of them 163 against 154)
  return n <= kSmallN && (cluster <= 2 || (cluster <= kSmallCluster && c->batch * cluster <= kRuleSms));
}

// Steps in pairs, where X is long enough and there is enough to save.  A pair
// replaces one Gram product (n^2 m) and one update (2 n^2 m) by three symmetric
// products (n^3 each), which have launches of their own.  Measured against single
// steps: 128 x 2048 x 768 2.01 against 2.33 ms, 24 x 1024 x 1856 722 against 772 us,
// but 24 x 1024 x 1280 626 against 610, and where launches count, 3 x 1000 x 333
// (1.3e9 operations less) 153 against 144; 5 x 500 x 2600 (1.6e10) 191 against 200.
// The nearer the matrices are to square, the more the pairs' roundings show: the error
// is 2.2e-3 at 1024 x 1856 and 2.4e-3 at 1024 x 1536 (651 against 661 us), 2.0e-3 in
// single steps, 1.7e-3 of rounding the result alone; so from m = 1.75 n on.
bool fuse_steps(int batch, int n, int m) {
  const double saved = 6.0 * n * n * (m - n) * batch;
  return 4 * m >= 7 * n && saved >= 1e10;
}

inline int pad64(int x) { return (x + 63) / 64 * 64; }

struct OrthoLayout {
  int chunk, chunks, ldx, lds;
  size_t part, fac, x0, x1, n[3], total;
};
OrthoLayout ortho_layout(const moe_ortho_config *c) {
  OrthoLayout L{};
  const size_t B = c->batch, n = c->R < c->C ? c->R : c->C;
  // a block's share: one round of its threads' loads, or four where that leaves
  // several blocks for every place on the part
  const int64_t numel = static_cast<int64_t>(c->R) * c->C;
  L.chunk = kPrepThreads * (c->C % 8 == 0 ? kPrepVecs * 8 : kPrepSingles);
  if (numel * c->batch >= static_cast<int64_t>(L.chunk) * 4 * kRuleSms * 8) L.chunk *= 4;
  L.chunks = static_cast<int>((numel + L.chunk - 1) / L.chunk);
  L.ldx = pad64(c->C);
  L.lds = pad64(static_cast<int>(n));
  if (is_small(c)) {
    L.total = kHeader;
    return L;
  }
  size_t o = 0;  // from the first multiple of 256 bytes past the header on
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  L.part = take(B * L.chunks * 4);
  L.fac = take(B * 4);
  L.x0 = take(B * c->R * L.ldx * 2);
  L.x1 = take(c->steps > 1 ? B * c->R * L.ldx * 2 : 0);
  const size_t square = B * n * L.lds * 2;
  L.n[0] = take(square);
  L.n[1] = take(square);
  L.n[2] = take(fuse_steps(c->batch, static_cast<int>(n), c->R < c->C ? c->C : c->R) ? square : 0);
  L.total = kHeader + 256 + o;
  return L;
}

template <class El>
cudaError_t launch_small(SmallArgs &a, int batch, cudaStream_t s) {
  static DeviceOnce once;
  auto kernel = ortho_small_kernel<El>;
  const cudaError_t e = once.get([&](int *) {
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, small_smem(2));
    return r != cudaSuccess ? r : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  const int blocks = (a.m + 63) / 64;  // of 64 columns
  a.cluster = 1;
  while (a.cluster * (kSlab / 64) < blocks) a.cluster *= 2;
  a.nblk = (blocks + a.cluster - 1) / a.cluster;
  return launch_pdl(kernel, dim3(batch * a.cluster), dim3(kSmallThreads), small_smem(a.cluster), s, a.cluster, a);
}

template <class El, bool VEC, bool MOM>
cudaError_t launch_prep(const PrepArgs &a, int batch, cudaStream_t s) {
  cudaError_t e =
      launch_pdl(ortho_prepare_kernel<El, VEC, MOM>, dim3(a.chunks, batch), dim3(kPrepThreads), 0, s, 1, a);
  if (e != cudaSuccess) return e;
  const int blocks = a.chunks < kRescaleBlocks ? a.chunks : kRescaleBlocks;
  return launch_pdl(ortho_rescale_kernel<El, VEC, MOM>, dim3(blocks, batch), dim3(kPrepThreads), 0, s, 1, a);
}
template <class El>
cudaError_t launch_prep(const PrepArgs &a, int batch, cudaStream_t s) {
  if (a.C % 8 == 0) return a.mom ? launch_prep<El, true, true>(a, batch, s) : launch_prep<El, true, false>(a, batch, s);
  return a.mom ? launch_prep<El, false, true>(a, batch, s) : launch_prep<El, false, false>(a, batch, s);
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
  if (is_small(cfg)) {
    SmallArgs q{};
    q.g = g;
    q.mom = momentum;
    q.out = static_cast<uint16_t *>(out);
    q.R = R;
    q.C = C;
    q.n = n;
    q.m = m;
    q.tall = tall;
    q.vec = C % 8 == 0;
    q.beta = beta;
    q.eps = cfg->eps;
    q.scale = scale;
    q.nesterov = nesterov != 0;
    q.steps = cfg->steps;
    q.status = status;
    for (int i = 0; i < 3 * cfg->steps; ++i) q.coefs[i] = coefs[i];
    return timed("ortho_small", st, [&] {
      return cfg->dtype == MOE_DTYPE_BF16 ? launch_small<uint16_t>(q, B, st) : launch_small<float>(q, B, st);
    });
  }
  // (sectors are stored, which need 32-byte alignment; the scratch has 16)
  uint8_t *body = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(sc) + kHeader + 255) &
                                              ~static_cast<uintptr_t>(255));
  PrepArgs a{};
  a.g = g;
  a.mom = momentum;
  a.beta = beta;
  a.nesterov = nesterov != 0;
  a.eps = cfg->eps;
  a.numel = static_cast<int64_t>(R) * C;
  a.C = C;
  a.ld = L.ldx;
  a.chunk = L.chunk;
  a.chunks = L.chunks;
  a.part = reinterpret_cast<float *>(body + L.part);
  a.fac = reinterpret_cast<float *>(body + L.fac);
  a.x = reinterpret_cast<uint16_t *>(body + L.x0);
  a.x_stride = static_cast<int64_t>(R) * L.ldx;
  a.status = status;
  MOE_TRY(timed("ortho_norm_scale", st, [&] {
    return cfg->dtype == MOE_DTYPE_BF16 ? launch_prep<uint16_t>(a, B, st) : launch_prep<float>(a, B, st);
  }));
  // X's rows along C with C contiguous: the Gram product reduces over m, the
  // update over n, so one of them reads X K-major and the other MN-major
  const bool pairs = fuse_steps(B, n, m), pair = use_pairs(B, R, C, di.sms);
  uint8_t *xb[2] = {body + L.x0, body + L.x1}, *nb[3] = {body + L.n[0], body + L.n[1], body + L.n[2]};
  Maps mx[2], mn[3];
  auto make = [&](Maps *mm, const void *ptr, int inner, int rows, int ld) {
    return map3(&mm->k, ptr, inner, rows, B, ld, 128) && map3(&mm->mn, ptr, inner, rows, B, ld, 64);
  };
  for (int i = 0; i < (cfg->steps > 1 ? 2 : 1); ++i)
    if (!make(&mx[i], xb[i], C, R, L.ldx)) return MOE_ERR_CUDA;
  for (int i = 0; i < (pairs ? 3 : 2); ++i)
    if (!make(&mn[i], nb[i], n, n, L.lds)) return MOE_ERR_CUDA;
  // Every launch goes through the matrices the other way round, so that it starts with
  // those that the last one left in the L2.
  bool back = true;
  auto turn = [&back] {
    back = !back;
    return !back;
  };
  ProductArgs sym{};  // of the products into an n x n matrix
  sym.batch = B;
  sym.status = status;
  sym.M = sym.N = n;
  sym.ld = L.lds;
  sym.stride = static_cast<int64_t>(n) * L.lds;
  const float *fac = a.fac;  // of the first X
  auto gram = [&](int x) {  // nb[0] <- S
    ProductArgs p = sym;
    p.K = m;
    p.c = 1.f / (kSigma * kSigma);
    p.fac = fac;
    p.back = turn();
    p.out = reinterpret_cast<uint16_t *>(nb[0]);
    const int split = pair ? 1 : gram_split(B, n, m, di.sms);
    return timed("ortho_gram", st, [&] {
      if (split > 1)
        return tall ? launch_gram_split<kMN>(mx[x], p, split, st) : launch_gram_split<kK>(mx[x], p, split, st);
      return tall ? launch_product<kGram, kMN, kMN>(mx[x], mx[x], p, pair, di.sms, st)
                  : launch_product<kGram, kK, kK>(mx[x], mx[x], p, pair, di.sms, st);
    });
  };
  auto polynomial = [&](int step, int in, int to) {  // nb[to] <- a I + b S + c S S
    ProductArgs p = sym;
    p.K = n;
    p.a = coefs[3 * step];
    p.back = turn();
    p.b = coefs[3 * step + 1];
    p.c = coefs[3 * step + 2];
    p.s = reinterpret_cast<const uint16_t *>(nb[in]);
    p.out = reinterpret_cast<uint16_t *>(nb[to]);
    return timed("ortho_polynomial", st,
                 [&] { return launch_product<kSquare, kSym, kSym>(mn[in], mn[in], p, pair, di.sms, st); });
  };
  auto commuting = [&](int x, int y, int to) {  // nb[to] <- nb[x] nb[y], symmetric as they commute
    ProductArgs p = sym;
    p.K = n;
    p.c = 1.f;
    p.out = reinterpret_cast<uint16_t *>(nb[to]);
    p.back = turn();
    return timed("ortho_commuting", st,
                 [&] { return launch_product<kGram, kSym, kSym>(mn[x], mn[y], p, pair, di.sms, st); });
  };
  auto apply = [&](int poly, int x, bool last) {  // X (or out) <- nb[poly] X
    ProductArgs p = sym;
    p.M = R;
    p.N = C;
    p.K = n;
    p.ld = last ? C : L.ldx;
    p.back = turn();
    p.stride = static_cast<int64_t>(R) * p.ld;
    p.c = last ? scale / kSigma : 1.f;
    p.sectors = last && C % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    p.fac = fac;
    p.out = last ? static_cast<uint16_t *>(out) : reinterpret_cast<uint16_t *>(xb[x ^ 1]);
    return timed("ortho_apply", st, [&] {
      if (last)
        return tall ? launch_product<kLast, kK, kSym>(mx[x], mn[poly], p, pair, di.sms, st)
                    : launch_product<kLast, kSym, kMN>(mn[poly], mx[x], p, pair, di.sms, st);
      return tall ? launch_product<kUpdate, kK, kSym>(mx[x], mn[poly], p, pair, di.sms, st)
                  : launch_product<kUpdate, kSym, kMN>(mn[poly], mx[x], p, pair, di.sms, st);
    });
  };
  int cur = 0;
  for (int i = 0; i < cfg->steps;) {
    MOE_TRY(gram(cur));
    MOE_TRY(polynomial(i, 0, 1));  // P
    int poly = 1, taken = 1;
    // steps go in pairs, an odd one by itself in the middle
    const bool alone = cfg->steps % 2 == 1 && i == cfg->steps / 2 / 2 * 2;
    if (pairs && !alone && i + 1 < cfg->steps) {
      MOE_TRY(commuting(1, 0, 2));       // P S
      MOE_TRY(commuting(2, 1, 0));       // P S P: the S of P X
      MOE_TRY(polynomial(i + 1, 0, 2));  // the next P
      MOE_TRY(commuting(2, 1, 0));       // both steps at once
      poly = 0;
      taken = 2;
    }
    i += taken;
    MOE_TRY(apply(poly, cur, i == cfg->steps));
    cur ^= 1;
    fac = nullptr;
  }
  return MOE_OK;
}

}  // extern "C"
