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
// Measured as called, bf16: forward with residual 16384 x 4096 80.6 us, 98% of what a
// copy moves in that time; backward with d_sum 16384 x 2048 47.8 us, 83% (the kernel
// 41.5 and the sums of its blocks' partial rows the rest).  512 x 128 takes 5.2 us,
// the launch.  Forward without residual 16384 x 2048 26.9 us, 74%: 1024 threads per SM
// leave 64 registers, which also hold the weight and the bias, and 8 to 100 bytes a
// thread are spilled.  fp32 16384 x 4096: forward with residual 176 us, 90%, without 96,
// 82%.  Widths far from a power of two leave threads without elements (5120 with
// residual 176 us, 56%), and ragged rows within a vector of 8192 take 1024 threads a
// block, whose kernels spill 40 to 184 bytes a thread forward and 428 to 676 backward.
//
// Layout: a row is shared by TPR threads (a power of two, 8 to 512), each
// holding kElems elements, in vectors of 16 bytes that lie TPR vectors apart, so
// a warp's accesses are contiguous.  Blocks are persistent over rows: a thread's
// columns stay the same, so the weight (and in the backward the column sums of
// dy xh and dy) stay in its registers, while asynchronous copies bring the coming
// rows into a ring in shared memory.  The backward's blocks leave one partial row
// of column sums each, which a second kernel adds in a fixed order: no atomics,
// the same bits every time.
#include <type_traits>

#include "abi.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kMaxH = 8192;
constexpr int kElems = 16;         // elements of a row per thread
constexpr int kThreads = 256;      // threads per block (a wider row takes one block of its own)
constexpr int kBwdBlocks = 304;    // the backward's partial rows at most: two blocks on each of 152 SMs
// The backward of few rows: one cluster of up to eight blocks with a round of rows each,
// which add their column sums themselves instead of a second kernel (5 x 4096 bf16 12.4
// to 9.1 us, 30 x 777 10.2 to 8.4; with four rounds 60 x 2048 went from 10.0 to 12.3).
constexpr int kOneCluster = 8;

struct NormArgs {
  const void *x, *res, *w, *b;  // forward input (backward: h), residual or d_sum, weight, bias
  const void *dy;
  void *y, *sum;                // forward: y, h; backward: dx, -
  float2 *stats;                // [T] mu, r
  float *part;                  // backward: [blocks][2][H] column sums of dy xh and dy
  float *dw, *db;               // backward, a single cluster of blocks: their sums (db or null)
  float eps;
  int T, H, tpr;
  bool layer;
};

// Sixteen-byte vectors of El (uint16_t: bf16 bits) and single elements.
template <class El>
struct Vec {
  static constexpr int N = 16 / static_cast<int>(sizeof(El));
  static __device__ __forceinline__ void unpack(const uint4 &r, float *f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(El) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *f) {
    if constexpr (sizeof(El) == 4)
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
      return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
  }
};
__device__ __forceinline__ float el_get(float v) { return v; }
__device__ __forceinline__ float el_get(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ void el_set(float *p, float v) { *p = v; }
__device__ __forceinline__ void el_set(uint16_t *p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
// The value as El stores it.
__device__ __forceinline__ float el_round(float v, float) { return v; }
__device__ __forceinline__ float el_round(float v, uint16_t) {
  return el_get(__bfloat16_as_ushort(__float2bfloat16_rn(v)));
}
constexpr uint32_t kAllValid = (1u << kElems) - 1;

// A thread's elements as pairs for the paired fp32 instructions: with single ones
// the arithmetic alone keeps the schedulers busy three quarters of the time.
constexpr int kPairs = kElems / 2;
__device__ __forceinline__ void pairs_of(const float (&f)[kElems], F2 (&p)[kPairs]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) p[i] = f2(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void unpair(const F2 (&p)[kPairs], float (&f)[kElems]) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float2 v = f2_get(p[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

// A thread's place: which of the block's rows (g) and where in it (lane).
struct Place {
  int tpr, rows, lane, g;
  int w0, per;  // the row's first warp, and its warps
  __device__ __forceinline__ Place(int tpr_, int threads) : tpr(tpr_) {
    rows = threads / tpr;
    lane = threadIdx.x & (tpr - 1);
    g = threadIdx.x / tpr;
    per = tpr > 32 ? tpr >> 5 : 1;
    w0 = (threadIdx.x >> 5) & ~(per - 1);
  }
};

// The sum of v (one float or two) over the threads of a row; every thread gets
// it.  buf: one value per warp of the block; `turn` alternates so that one barrier
// per sum is enough (a thread writes one half while slower ones read the other).
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float shfl(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ float2 shfl(float2 v, int o) { return make_float2(shfl(v.x, o), shfl(v.y, o)); }
template <class S>
__device__ __forceinline__ S row_sum(S v, const Place &pl, S (*buf)[32], int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < pl.tpr) v = plus(v, shfl(v, o));
  if (pl.per > 1) {
    if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[turn][pl.w0];
    for (int i = 1; i < pl.per; ++i) v = plus(v, buf[turn][pl.w0 + i]);
    turn ^= 1;
  }
  return v;
}

// 1 / sqrt(v): the approximation and one Newton step (v = 0 gives infinity).
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return v > 0.f && v < INFINITY ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}

// Statistics of one row; x2: h in, h - mu out.  valid: which of this thread's
// elements are the row's (the others hold zeros).
struct Stats {
  float mu, r;
};
__device__ __forceinline__ Stats normalise(F2 (&x2)[kPairs], uint32_t valid, const NormArgs &a, float inv,
                                           const Place &pl, float (*buf)[32], int &turn) {
  Stats st{0.f, 0.f};
  if (a.layer) {
    F2 s2 = x2[0];
#pragma unroll
    for (int i = 1; i < kPairs; ++i) s2 = f2_add(s2, x2[i]);
    const float2 s = f2_get(s2);
    st.mu = row_sum(s.x + s.y, pl, buf, turn) * inv;
    const F2 m2 = f2(st.mu, st.mu);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) x2[i] = f2_sub(x2[i], m2);
    if (valid != kAllValid) {  // what is not the row's does not deviate from its mean
      float f[kElems];
      unpair(x2, f);
#pragma unroll
      for (int i = 0; i < kElems; ++i) f[i] = (valid >> i) & 1u ? f[i] : 0.f;
      pairs_of(f, x2);
    }
  }
  F2 q2 = f2_mul(x2[0], x2[0]);
#pragma unroll
  for (int i = 1; i < kPairs; ++i) q2 = f2_fma(x2[i], x2[i], q2);
  const float2 q = f2_get(q2);
  st.r = inv_sqrt(fmaf(row_sum(q.x + q.y, pl, buf, turn), inv, a.eps));
  return st;
}
__device__ __forceinline__ void scale_shift(F2 (&x2)[kPairs], float r, const float (&w)[kElems],
                                            const float (&b)[kElems]) {
  F2 w2[kPairs], b2[kPairs];
  pairs_of(w, w2);
  pairs_of(b, b2);
  const F2 r2 = f2(r, r);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) x2[i] = f2_fma(f2_mul(x2[i], r2), w2[i], b2[i]);
}

// Backward of one row: x and dy in (zeros past the row's end, and for rows past
// the last with r = 0); leaves g = dy w in gw and xh in x2, adds to the column
// sums, and returns mean(g) and mean(g xh).
__device__ __forceinline__ float2 row_grad(F2 (&x2)[kPairs], const F2 (&e2)[kPairs], const float (&w)[kElems],
                                           F2 (&gw)[kPairs], F2 (&aw)[kPairs], F2 (&ab)[kPairs], float2 st, float inv,
                                           const Place &pl, float2 (*buf)[32], int &turn) {
  F2 w2[kPairs];
  pairs_of(w, w2);
  const F2 m2 = f2(st.x, st.x), r2 = f2(st.y, st.y);
  F2 sg = f2(0.f, 0.f), sx = sg;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    x2[i] = f2_mul(f2_sub(x2[i], m2), r2);
    gw[i] = f2_mul(e2[i], w2[i]);
    sg = f2_add(sg, gw[i]);
    sx = f2_fma(gw[i], x2[i], sx);
    aw[i] = f2_fma(e2[i], x2[i], aw[i]);
    ab[i] = f2_add(ab[i], e2[i]);
  }
  const float2 pg = f2_get(sg), px = f2_get(sx);
  const float2 s = row_sum(make_float2(pg.x + pg.y, px.x + px.y), pl, buf, turn);
  return make_float2(s.x * inv, s.y * inv);
}
// o2 (d_sum or zeros) += r (g - c.x - xh c.y)
__device__ __forceinline__ void row_dx(F2 (&o2)[kPairs], const F2 (&gw)[kPairs], const F2 (&xh)[kPairs], float2 c,
                                       float r) {
  const F2 c1 = f2(-c.y, -c.y), c2 = f2(c.x, c.x), r2 = f2(r, r);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) o2[i] = f2_fma(r2, f2_fma(xh[i], c1, f2_sub(gw[i], c2)), o2[i]);
}

// The block's column sums, its row groups added in order: into its partial row, or
// (a single cluster of blocks, dw set) into shared memory, from which the blocks add
// a share of the columns each, in the order of the blocks, into dw and db.
// col(j): the column of a thread's element j (one below 0 or past H: none).  s_col:
// [rows][2][H] in shared memory (at most 128 bytes a thread).
template <class Col>
__device__ __forceinline__ void block_colsum(const NormArgs &a, const Place &pl, const F2 (&aw)[kPairs],
                                             const F2 (&ab)[kPairs], float *s_col, Col &&col) {
  float cw[kElems], cb[kElems];
  unpair(aw, cw);
  unpair(ab, cb);
  const int H = a.H;
  float *part = a.part + static_cast<size_t>(blockIdx.x) * 2 * H;
  float *mine = pl.rows > 1 || a.dw ? s_col + pl.g * 2 * H : part;
#pragma unroll
  for (int j = 0; j < kElems; ++j) {
    const int c = col(j);
    if (c < 0 || c >= H) continue;
    mine[c] = cw[j];
    mine[H + c] = cb[j];
  }
  if (mine == part) return;
  __syncthreads();
  if (pl.rows > 1) {
    for (int c = threadIdx.x; c < 2 * H; c += blockDim.x) {
      float v = s_col[c];
      for (int q = 1; q < pl.rows; ++q) v += s_col[q * 2 * H + c];
      (a.dw ? s_col : part)[c] = v;  // (each thread its own columns)
    }
  }
  if (!a.dw) return;
  const int n = gridDim.x, rank = blockIdx.x;
  if (n > 1)
    cluster_sync();
  else
    __syncthreads();
  for (int c = rank * blockDim.x + threadIdx.x; c < 2 * H; c += n * blockDim.x) {
    float v = s_col[c];
    if (n > 1) {
      float o[kOneCluster];
#pragma unroll
      for (int r = 0; r < kOneCluster; ++r)
        if (r < n)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o[r]) : "r"(peer_smem_addr(s_col + c, r)) : "memory");
      v = o[0];
#pragma unroll
      for (int r = 1; r < kOneCluster; ++r)
        if (r < n) v += o[r];
    }
    if (c < H)
      a.dw[c] = v;
    else if (a.db)
      a.db[c - H] = v;
  }
  if (n > 1) cluster_sync();  // no block leaves while another reads its sums
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Sixteen bytes into shared memory; of which only `bytes` are read, the rest zero.
__device__ __forceinline__ void copy16(void *dst, const void *src, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}

// Rows of a group in flight.  Three of bf16, two of fp32 (twice the bytes), and two
// for a single input, whose blocks are many: more was never faster.  (One where 1024
// threads share the block's shared memory.)
template <class El, int Q, int TH>
__host__ __device__ constexpr int ring_depth() {
  return TH == 1024 ? 1 : (sizeof(El) == 2 && Q > 1 ? 3 : 2);
}

// ---- the rows of one thread.  Memory is read in aligned vectors, and the ring is
// filled and read back by the same thread, so no barrier is needed.  Rows that are
// not whole vectors (SPAN) start `phase` elements into one; a group's rows are a
// multiple of N apart, so its phase, and every thread's columns, stay the same.
// Elements of a thread's first and last vectors that belong to the neighbouring
// rows are masked, and such vectors are stored element by element.
template <class El, bool SPAN>
struct Lane {
  static constexpr int N = Vec<El>::N, V = kElems / N;
  int H, T, tpr, lane, phase;
  int left;        // vectors of the row from this thread's first one on
  uint32_t valid;  // which of its elements are the row's
  __device__ __forceinline__ Lane(const NormArgs &a, const Place &pl, int t0)
      : H(a.H), T(a.T), tpr(pl.tpr), lane(pl.lane), phase(0), valid(0) {
    if constexpr (SPAN) phase = static_cast<int>(static_cast<int64_t>(t0) * H & (N - 1));
    left = (phase + H + N - 1) / N - lane;
#pragma unroll
    for (int j = 0; j < kElems; ++j) valid |= (col(j) >= 0 && col(j) < H ? 1u : 0u) << j;
  }
  __device__ __forceinline__ int col(int j) const { return (lane + tpr * (j / N)) * N + j % N - phase; }
  // vector of row t's first one, this thread's first
  __device__ __forceinline__ size_t first(int t) const { return static_cast<size_t>(t) * H / N + lane; }
  __device__ __forceinline__ void mask(float (&f)[kElems]) const {
    if (SPAN && valid != kAllValid) {
#pragma unroll
      for (int j = 0; j < kElems; ++j) f[j] = (valid >> j) & 1u ? f[j] : 0.f;
    }
  }
  // a vector of length H (weight, bias), as vectors over this thread's columns
  __device__ __forceinline__ void load_cols(const void *base, uint4 (&r)[V]) const {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if constexpr (SPAN) {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
          f[i] = base && ((valid >> (N * u + i)) & 1u) ? el_get(static_cast<const El *>(base)[col(N * u + i)]) : 0.f;
        r[u] = Vec<El>::pack(f);
      } else {
        r[u] = base && tpr * u < left ? static_cast<const uint4 *>(base)[lane + tpr * u] : make_uint4(0, 0, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void store(void *base, int t, const float (&f)[kElems]) const {
    uint4 *dst = static_cast<uint4 *>(base) + first(t);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const uint32_t ok = (valid >> (N * u)) & ((1u << N) - 1);
      if (!SPAN ? tpr * u < left : ok == (1u << N) - 1) {
        dst[tpr * u] = Vec<El>::pack(f + N * u);
      } else if (SPAN && ok) {
        El *e = reinterpret_cast<El *>(dst + tpr * u);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if ((ok >> i) & 1u) el_set(e + i, f[N * u + i]);
      }
    }
  }
};

template <class El, int Q, int TH>
__host__ __device__ constexpr int ring_bytes() {
  return ring_depth<El, Q, TH>() * Q * kElems * static_cast<int>(sizeof(El)) * TH;
}

template <class El, bool SPAN, int Q, int TH>
struct Ring {
  static constexpr int N = Vec<El>::N, V = kElems / N, D = ring_depth<El, Q, TH>();
  uint4 *slot;  // this thread's; vector (d, q, u) is ((d Q + q) V + u) TH further
  const uint4 *src[Q];
  __device__ __forceinline__ Ring(uint8_t *mem, const Lane<El, SPAN> &ln, const void *const (&in)[Q])
      : slot(reinterpret_cast<uint4 *>(mem) + threadIdx.x) {
#pragma unroll
    for (int q = 0; q < Q; ++q) src[q] = static_cast<const uint4 *>(in[q]);
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int u = 0; u < V; ++u)
          if (ln.tpr * u >= ln.left) at(d, q, u) = make_uint4(0, 0, 0, 0);  // past the row: zeros for good
  }
  __device__ __forceinline__ uint4 &at(int d, int q, int u) const { return slot[((d * Q + q) * V + u) * TH]; }
  __device__ __forceinline__ void fetch(int t, int d, const Lane<El, SPAN> &ln) const {
    const size_t v0 = ln.first(t);
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (ln.tpr * u < ln.left) {
        int bytes = 16;
        if (SPAN && ln.T - t <= N) {  // nothing past the end of the last row is read
          const int64_t rest = static_cast<int64_t>(ln.T - t) * ln.H - ln.col(N * u);  // elements from the vector on
          bytes = rest < N ? static_cast<int>(rest) * static_cast<int>(sizeof(El)) : 16;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          if (t < ln.T)
            copy16(&at(d, q, u), src[q] + v0 + ln.tpr * u, bytes);
          else
            at(d, q, u) = make_uint4(0, 0, 0, 0);
        }
      }
    copies_commit();
  }
  __device__ __forceinline__ void get(int d, int q, float (&f)[kElems], const Lane<El, SPAN> &ln) const {
#pragma unroll
    for (int u = 0; u < V; ++u) Vec<El>::unpack(at(d, q, u), f + N * u);
    ln.mask(f);
  }
};

template <class El>
__device__ __forceinline__ void unpack_all(const uint4 *r, float (&f)[kElems]) {
#pragma unroll
  for (int u = 0; u < kElems / Vec<El>::N; ++u) Vec<El>::unpack(r[u], f + Vec<El>::N * u);
}

// Threads per SM that the kernels are built for.  Forward: 1024, or 512 with a
// residual, whose two reads and two writes run faster from fewer rows at once
// (16384 x 4096 bf16: 84 against 102 us; without one, 16384 x 2048: 28 against
// 34 us the other way, although 64 registers are too few there).  Backward: 512 (its column sums take the registers).
constexpr int fwd_threads(bool res) { return res ? 512 : 1024; }
constexpr int at_least_1(int x) { return x > 0 ? x : 1; }

template <class El, bool SPAN, bool RES, int TH>
__global__ void __launch_bounds__(TH, at_least_1(fwd_threads(RES) / TH)) norm_fwd_kernel(const NormArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  constexpr int Q = RES ? 2 : 1, D = ring_depth<El, Q, TH>();
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float s_red[2][32];
  int turn = 0;
  const Place pl(a.tpr, TH);
  const float inv = 1.f / static_cast<float>(a.H);
  const int step = gridDim.x * pl.rows, t0 = blockIdx.x * pl.rows + pl.g;
  const Lane<El, SPAN> ln(a, pl, t0);
  const void *in[Q];
  in[0] = a.x;
  if constexpr (RES) in[1] = a.res;
  const Ring<El, SPAN, Q, TH> ring(s_dyn, ln, in);
#pragma unroll
  for (int d = 0; d < D - 1; ++d) ring.fetch(t0 + d * step, d, ln);
  uint4 wr[ln.V], br[ln.V];
  ln.load_cols(a.w, wr);
  ln.load_cols(a.b, br);
  int d = 0;
  for (int r0 = blockIdx.x * pl.rows; r0 < a.T; r0 += step) {
    const int t = r0 + pl.g;
    ring.fetch(t + (D - 1) * step, d == 0 ? D - 1 : d - 1, ln);
    copies_wait<D - 1>();
    float f[kElems];
    F2 x2[kPairs];
    ring.get(d, 0, f, ln);
    if constexpr (RES) {
      float q[kElems];
      ring.get(d, 1, q, ln);
#pragma unroll
      for (int i = 0; i < kElems; ++i) f[i] = el_round(f[i] + q[i], El{});  // the norm is that of the stored sum
      if (t < a.T) ln.store(a.sum, t, f);
    }
    if (++d == D) d = 0;
    pairs_of(f, x2);
    const Stats st = normalise(x2, ln.valid, a, inv, pl, s_red, turn);
    if (t < a.T) {
      float w[kElems], b[kElems];
      unpack_all<El>(wr, w);
      unpack_all<El>(br, b);
      scale_shift(x2, st.r, w, b);
      unpair(x2, f);
      ln.store(a.y, t, f);
      if (pl.lane == 0) a.stats[t] = make_float2(st.mu, st.r);
    }
  }
}

template <class El, bool SPAN, bool RES, int TH>
__global__ void __launch_bounds__(TH, at_least_1(512 / TH)) norm_bwd_kernel(const NormArgs a) {
  griddep_wait();  // the previous kernel in the stream has completed
  constexpr int Q = RES ? 3 : 2, D = ring_depth<El, Q, TH>();
  extern __shared__ __align__(16) uint8_t s_dyn[];
  __shared__ float2 s_red[2][32];
  int turn = 0;
  const Place pl(a.tpr, TH);
  const float inv = 1.f / static_cast<float>(a.H);
  const int step = gridDim.x * pl.rows, t0 = blockIdx.x * pl.rows + pl.g;
  const Lane<El, SPAN> ln(a, pl, t0);
  const void *in[Q];
  in[0] = a.x;
  in[1] = a.dy;
  if constexpr (RES) in[2] = a.res;
  const Ring<El, SPAN, Q, TH> ring(s_dyn, ln, in);
#pragma unroll
  for (int d = 0; d < D - 1; ++d) ring.fetch(t0 + d * step, d, ln);
  uint4 wr[ln.V];
  ln.load_cols(a.w, wr);
  F2 aw[kPairs], ab[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) aw[i] = ab[i] = f2(0.f, 0.f);
  const float2 none = make_float2(0.f, 0.f);  // rows past the last: xh = 0, dy = 0
  float2 next = t0 < a.T ? a.stats[t0] : none;
  int d = 0;
  for (int r0 = blockIdx.x * pl.rows; r0 < a.T; r0 += step) {
    const int t = r0 + pl.g;
    ring.fetch(t + (D - 1) * step, d == 0 ? D - 1 : d - 1, ln);
    const float2 st = next;
    next = t + step < a.T ? a.stats[t + step] : none;
    copies_wait<D - 1>();
    float f[kElems];
    F2 x2[kPairs], e2[kPairs], gw[kPairs];
    ring.get(d, 0, f, ln);
    pairs_of(f, x2);
    ring.get(d, 1, f, ln);
    pairs_of(f, e2);
    unpack_all<El>(wr, f);
    float2 c = row_grad(x2, e2, f, gw, aw, ab, st, inv, pl, s_red, turn);
    if (!a.layer) c.x = 0.f;
    if (t < a.T) {
      F2 o2[kPairs];
#pragma unroll
      for (int i = 0; i < kElems; ++i) f[i] = 0.f;
      if constexpr (RES) ring.get(d, 2, f, ln);
      pairs_of(f, o2);
      row_dx(o2, gw, x2, c, st.y);
      unpair(o2, f);
      ln.store(a.y, t, f);
    }
    if (++d == D) d = 0;
  }
  copies_wait<0>();
  __syncthreads();  // the ring is no longer read: it holds the sums
  block_colsum(a, pl, aw, ab, reinterpret_cast<float *>(s_dyn), [&](int j) { return ln.col(j); });
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
  constexpr int U = (kBwdBlocks + 31) / 32;  // every load of a run at once
  float v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = c < H && run + 32 * u < nb ? src[static_cast<size_t>(run + 32 * u) * 2 * H] : 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) acc += v[u];
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

// Rows of whole vectors, and threads per row: enough for the vectors that a row
// touches wherever it starts.
bool spans(int H, int el) { return H * el % 16 != 0; }
int tpr_of(int H, int el) {
  const int n = 16 / el, need = spans(H, el) ? (H + n - 1 + n - 1) / n * n : H;
  int tpr = 8;
  while (tpr * kElems < need) tpr *= 2;
  return tpr;
}
// Blocks: those that fit at once, and where rows have a phase, a number that keeps
// a group's rows a multiple of the vector apart.
int blocks_for(const NormArgs &a, int threads, int most, int el) {
  const int rows = threads / a.tpr, need = (a.T + rows - 1) / rows;
  if (need <= most) return need;
  const int n = 16 / el, unit = spans(a.H, el) && rows < n ? n / rows : 1;
  return most / unit * unit;
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

template <class El, bool SPAN, bool RES, int TH>
cudaError_t launch_fwd(const NormArgs &a, int sms, cudaStream_t s) {
  static DeviceOnce once;
  constexpr int smem = ring_bytes<El, RES ? 2 : 1, TH>();
  auto kernel = norm_fwd_kernel<El, SPAN, RES, TH>;
  int most = 0;
  const cudaError_t e = resident(once, kernel, TH, smem, sms, &most);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(blocks_for(a, TH, most, sizeof(El))), dim3(TH), smem, s, 1, a);
}

template <class El, bool SPAN, bool RES, int TH>
cudaError_t launch_bwd(const NormArgs &a, int sms, float *dw, float *db, cudaStream_t s) {
  static DeviceOnce once;
  constexpr int smem = ring_bytes<El, RES ? 3 : 2, TH>();
  auto kernel = norm_bwd_kernel<El, SPAN, RES, TH>;
  int most = 0;
  cudaError_t e = resident(once, kernel, TH, smem, sms, &most);
  if (e != cudaSuccess) return e;
  const int rows = TH / a.tpr, need = (a.T + rows - 1) / rows;
  if (need <= kOneCluster) {
    NormArgs one = a;
    one.dw = dw;
    one.db = db;
    return launch_pdl(kernel, dim3(need), dim3(TH), smem, s, need, one);
  }
  const int nb = blocks_for(a, TH, most < kBwdBlocks ? most : kBwdBlocks, sizeof(El));
  e = launch_pdl(kernel, dim3(nb), dim3(TH), smem, s, 1, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_colsum_kernel, dim3((a.H + 7) / 8, db ? 2 : 1), dim3(256), 0, s, 1, a.part, nb, a.H, dw, db);
}

// The variant for a configuration: 256 threads, or as many as one row takes
// (1024 only where a row of nearly 8192 elements has a phase).
template <class F>
cudaError_t by_form(const NormArgs &a, bool bf, bool res, F &&f) {
  auto threads = [&](auto el, auto sp, auto re) {
    if (a.tpr <= kThreads) return f(el, sp, re, std::integral_constant<int, kThreads>{});
    if constexpr (decltype(sp)::value)
      if (a.tpr > 512) return f(el, sp, re, std::integral_constant<int, 1024>{});
    return f(el, sp, re, std::integral_constant<int, 512>{});
  };
  auto rows = [&](auto el, auto sp) {
    return res ? threads(el, sp, std::true_type{}) : threads(el, sp, std::false_type{});
  };
  auto type = [&](auto el) {
    return spans(a.H, sizeof(el)) ? rows(el, std::true_type{}) : rows(el, std::false_type{});
  };
  return bf ? type(uint16_t{}) : type(float{});
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
  a.tpr = tpr_of(c->H, c->dtype == MOE_DTYPE_BF16 ? 2 : 4);
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
    return by_form(a, cfg->dtype == MOE_DTYPE_BF16, residual != nullptr, [&](auto el, auto span, auto res, auto th) {
      return launch_fwd<decltype(el), decltype(span)::value, decltype(res)::value, decltype(th)::value>(a, di.sms, s);
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
    return by_form(a, cfg->dtype == MOE_DTYPE_BF16, d_sum != nullptr, [&](auto el, auto span, auto res, auto th) {
      return launch_bwd<decltype(el), decltype(span)::value, decltype(res)::value, decltype(th)::value>(
          a, di.sms, dweight, dbias, s);
    });
  });
}

}  // extern "C"
