// Layer norm over the columns, forward and backward: streaming kernels, bound by HBM bandwidth.
//
//   forward   mean = sum x / n, rstd = 1 / sqrt(sum (x - mean)^2 / n + eps), y = (x - mean) rstd gamma + beta
//   backward  h = (x - mean) rstd, g = dy gamma: dx = rstd (g - sum g / n - h sum (g h) / n) + residual,
//             dgamma = sum over the rows of dy h, dbeta = sum over the rows of dy
//
// A row stays on the SM between the passes over it: it is read once. W warps share a row, each lane U
// pieces of 8 columns; wider rows (more than 16 warps' worth) take a block that reads them again from L2.
// Beside HBM the issue of instructions bounds these kernels (67 % of the cycles with W at run time and a
// row widened anew for each pass): so W and U are compile-time, rows that fill their lanes have kernels without
// bounds (FULL), and what is widened once stays in registers where there is room. All arithmetic is fp32, every
// output rounded once.
#include <algorithm>

#include "linear_math.cuh"

namespace zgb {
namespace {

constexpr int kMaxWarps = 16;               // of a row held in registers
constexpr int kWidest = kMaxWarps * 4 * 256;  // columns of four pieces a lane
constexpr int kWideThreads = 512;           // block of the kernels for wider rows

__device__ __forceinline__ void widen8(const uint4& w, f2 (&x)[4]) {
  x[0] = f2_from_bf16x2(w.x), x[1] = f2_from_bf16x2(w.y), x[2] = f2_from_bf16x2(w.z), x[3] = f2_from_bf16x2(w.w);
}
__device__ __forceinline__ uint4 narrow8(const f2 (&x)[4]) {
  return make_uint4(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]), f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
}
__device__ __forceinline__ float f2_sum(f2 v) {
  float a, b;
  f2_split(v, a, b);
  return __fadd_rn(a, b);
}
__device__ __forceinline__ f2 f2_sum4(const f2 (&v)[4]) { return f2_add(f2_add(v[0], v[1]), f2_add(v[2], v[3])); }
// 1 / sqrt(a), off by at most 2^-23 of itself
__device__ __forceinline__ float reciprocal_root(float a) { return __fdiv_rn(1.0f, __fsqrt_rn(a)); }

// gamma or beta of 8 columns; ones or zeros where there is none
__device__ __forceinline__ uint4 param8(const uint16_t* p, int64_t col, bool in, uint32_t otherwise) {
  return p && in ? __ldg(reinterpret_cast<const uint4*>(p + col)) : make_uint4(otherwise, otherwise, otherwise, otherwise);
}
constexpr uint32_t kOnes = 0x3F803F80u;  // two bf16 1.0

__device__ __forceinline__ float warp_sum(float v, int lanes = 32) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < lanes) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
// Two values of each warp of a row, given to the row's W warps: lane w has those of its warp w (0 past the
// last). `turn` alternates: the half written now was last read before the barrier ahead of this one.
template <int N>
struct RowMeet {
  float2 of[2][N][kMaxWarps];
};
template <int W, int N>
__device__ __forceinline__ void row_meet(float (&a)[N], float (&b)[N], RowMeet<N>& s, int& turn, int first) {
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s.of[turn][i][threadIdx.x >> 5] = make_float2(a[i], b[i]);
  // where a block has several groups, the row's warps alone: every one of them takes as many rows
  if constexpr (W >= 8) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + first / W), "n"(32 * W) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 v = lane < W ? s.of[turn][i][first + lane] : make_float2(0.0f, 0.0f);
    a[i] = v.x, b[i] = v.y;
  }
  turn ^= 1;
}
// of lanes 0 .. 15, given to all (lanes 16 .. 31 hold zeros)
__device__ __forceinline__ float low_lanes_sum(float v) { return __shfl_sync(0xffffffffu, warp_sum(v, kMaxWarps), 0); }

// A thread's place: W warps to a row, PER rows of a block at a time; piece u of the thread's is the 8 columns from
// col0 + 256 W u
__host__ __device__ constexpr int rows_of_block(int w) { return w >= 8 ? 1 : 8 / w; }
__host__ __device__ constexpr int threads_of_block(int w) { return 32 * w * rows_of_block(w); }
template <int W>
struct Place {
  static constexpr int PER = rows_of_block(W), STRIDE = W * 256;
  int first, group, col0;
  __device__ __forceinline__ Place() {
    const int warp = threadIdx.x >> 5;
    group = warp / W, first = group * W;
    col0 = ((warp - first) * 32 + (threadIdx.x & 31)) * 8;
  }
};
// columns of warp w of a row; 0 past the last warp
template <int W, int U, bool FULL>
__device__ __forceinline__ float own_columns(int w, int cols) {
  if (w >= W) return 0.0f;
  if (FULL) return 256.0f * U;
  int n = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) n += min(max(cols - (u * W + w) * 256, 0), 256);
  return static_cast<float>(n);
}

// A block takes R rows in each of its groups of W warps: the rows' loads and reductions are in flight together,
// and share gamma and beta. Bound by HBM and, nearly, by instructions: 8192 x 4096 24.1 us, 5.6 TB/s (issue 64 %; with
// 74 registers, three blocks to an SM instead of four, 27.8); 32768 x 768 16.8 us, 6.0 TB/s; 8192 x 8192 43.4 us, 6.2;
// one row of 4096 1.7 us. Rows loaded ahead through shared memory, as in the backward, by three blocks to an SM:
// 8192 x 4096 26.1 us.
template <int W, int U, int R, bool FULL>
__global__ void __launch_bounds__(threads_of_block(W), (U * R > 4 ? 768 : 1024) / threads_of_block(W)) norm_forward_kernel(
    const uint16_t* __restrict__ x, int64_t rows, int cols, const uint16_t* __restrict__ gamma, const uint16_t* __restrict__ beta,
    float eps, float inv_n, uint16_t* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ RowMeet<R> sums;
  allow_next_grid();
  const Place<W> at;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * at.PER + at.group) * R;
  const uint16_t* xr = x + row0 * cols + at.col0;
  const auto in = [&](int u) { return FULL || at.col0 + u * at.STRIDE < cols; };
  int turn = 0;
  wait_for_prior_grids();
  uint4 w[R][U];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[i][u] = make_uint4(0u, 0u, 0u, 0u);
      if (row0 + i < rows && in(u))
        w[i][u] = __ldcs(reinterpret_cast<const uint4*>(xr + static_cast<int64_t>(i) * cols + u * at.STRIDE));
    }
  // each warp's mean and squares about it, joined: with m_w, q_w and n_w the mean, squares and columns of warp w,
  // the row's squares about its mean are sum q_w + n_w (m_w - mean)^2
  const float inv_own = W == 1 ? inv_n : __fdiv_rn(1.0f, fmaxf(own_columns<W, U, FULL>((threadIdx.x >> 5) - at.first, cols), 1.0f));
  f2 v[R][U][4];
  float sum[R], sq[R], mu[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    f2 t = 0ull;
#pragma unroll
    for (int u = 0; u < U; ++u) {  // zeros past the row
      widen8(w[i][u], v[i][u]);
      t = f2_add(t, f2_sum4(v[i][u]));
    }
    sum[i] = f2_sum(t);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) sum[i] = warp_sum(sum[i]), mu[i] = __fmul_rn(sum[i], inv_own);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    f2 t[2] = {0ull, 0ull};
    const f2 m = f2_both(-mu[i]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in(u)) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 c = f2_add(v[i][u][j], m);
        t[j & 1] = f2_fma(c, c, t[j & 1]);
      }
    }
    sq[i] = f2_sum(f2_add(t[0], t[1]));
  }
#pragma unroll
  for (int i = 0; i < R; ++i) sq[i] = warp_sum(sq[i]);
  if constexpr (W > 1) {
    row_meet<W>(sum, sq, sums, turn, at.first);
    const float theirs = own_columns<W, U, FULL>(threadIdx.x & 31, cols), inv_theirs = __fdiv_rn(1.0f, fmaxf(theirs, 1.0f));
#pragma unroll
    for (int i = 0; i < R; ++i) {
      mu[i] = __fmul_rn(low_lanes_sum(sum[i]), inv_n);
      const float off = __fsub_rn(__fmul_rn(sum[i], inv_theirs), mu[i]);
      sq[i] = low_lanes_sum(__fmaf_rn(__fmul_rn(theirs, off), off, sq[i]));
    }
  }
  float r[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    r[i] = reciprocal_root(__fadd_rn(__fmul_rn(sq[i], inv_n), eps));
    if (at.col0 == 0 && mean && row0 + i < rows) mean[row0 + i] = mu[i], rstd[row0 + i] = r[i];
  }
  uint16_t* yr = y + row0 * cols + at.col0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!in(u)) continue;
    f2 g[4], b[4];
    widen8(param8(gamma, at.col0 + u * at.STRIDE, true, kOnes), g);
    widen8(param8(beta, at.col0 + u * at.STRIDE, true, 0u), b);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (row0 + i >= rows) continue;
      const f2 m = f2_both(-mu[i]), k = f2_both(r[i]);
      f2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = f2_fma(f2_mul(f2_add(v[i][u][j], m), k), g[j], b[j]);
      __stcs(reinterpret_cast<uint4*>(yr + static_cast<int64_t>(i) * cols + u * at.STRIDE), narrow8(o));
    }
  }
}

// What a thread of the backward reads, STAGES - 1 rounds ahead of its use, through its own slots of shared memory: x,
// dy and the residual, U pieces of 16 bytes of each for R rows, none of another thread's, so that nothing but
// the thread's own copies is waited for.
template <int W, int U, int R, int BLOCKS>
struct Ahead {
  static constexpr int THREADS = threads_of_block(W);
  static constexpr uint32_t STAGE = 3 * U * R * 16u * THREADS;
  static constexpr int FIT = 216 * 1024 / BLOCKS / STAGE, STAGES = FIT < 4 ? FIT : 4;
  static_assert(STAGES >= 2, "one round in use, one on its way");
  static constexpr uint32_t BYTES = STAGES * STAGE;
  uint4* mine;  // this thread's slots, THREADS apart
  __device__ __forceinline__ uint4* slot(int stage, int t, int u, int i) const {
    return mine + (((stage * 3 + t) * U + u) * R + i) * THREADS;
  }
  static __device__ __forceinline__ void load(uint4* to, const uint16_t* from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 16u : 0u) : "memory");
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory"); }
};

// Backward. partial: nullable, [blocks][2][cols]: a block's sums of dy h and dy over its rows. A group of W warps
// takes R rows a round, whose reductions are in flight together. h and g are made again for the second pass: keeping
// them takes 32 registers a row, and two rows a round are worth more (32768 x 768 with residual: one row, kept,
// 38.6 us; two rows, kept, at half the warps 39.7; two rows, made again 36.6. 8192 x 4096: 47.2, 46.2, 46.4). Bound by
// HBM: 8192 x 4096 with residual 46 us with the launch below, 5.8 TB/s, 40.4 of it this kernel (75 % of the DRAM rate);
// 8192 x 8192 83 us, 6.4 TB/s; narrower rows more by the latency of a round's reductions (8192 x 2304 26 us, 4.4
// TB/s), and past 8192 columns, where a row takes four pieces a lane and a round is one row, by the same (4096 x 14336
// with residual 94 us, 5.0 TB/s).
struct BackwardArgs {
  const uint16_t *dy, *x;
  const float *mean, *rstd;
  int64_t rows;
  int cols;
  const uint16_t* gamma;
  float inv_n;
  const uint16_t* residual;
  uint16_t* dx;
};
template <int W, int U, int R, int BLOCKS, bool FULL, bool PARAMS>
__device__ __forceinline__ void backward_rows(const BackwardArgs& p, int block, int blocks, uint4* ring_mem, float* __restrict__ partial) {
  using Ring = Ahead<W, U, R, BLOCKS>;
  constexpr int STAGES = Ring::STAGES, PER = Place<W>::PER, STRIDE = Place<W>::STRIDE;
  __shared__ RowMeet<R> sums;
  const uint16_t *dy = p.dy, *residual = p.residual;
  const uint16_t* __restrict__ x = p.x;
  const float *__restrict__ mean = p.mean, *__restrict__ rstd = p.rstd;
  const int64_t rows = p.rows;
  const int cols = p.cols;
  const float inv_n = p.inv_n;
  const Place<W> at;
  const Ring ring{ring_mem + threadIdx.x};
  const auto in = [&](int u) { return FULL || at.col0 + u * STRIDE < cols; };
  const int64_t step = static_cast<int64_t>(blocks) * PER * R, first = static_cast<int64_t>(block) * PER * R;
  const auto load = [&](int64_t row0, int stage) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool there = row0 + i < rows;
      const int64_t base = there ? (row0 + i) * cols + at.col0 : 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool some = there && in(u);
        const int64_t j = some ? base + u * STRIDE : 0;  // a place in the tensors, where nothing is read
        ring.load(ring.slot(stage, 0, u, i), x + j, some);
        ring.load(ring.slot(stage, 1, u, i), dy + j, some);
        if (residual) ring.load(ring.slot(stage, 2, u, i), residual + j, some);
      }
    }
    ring.commit();
  };
  int turn = 0, stage = 0;
  const int64_t mine = first + at.group * R;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) load(mine + i * step, i);
  uint4 gw[U];
  f2 dg[U][4], db[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    gw[u] = param8(p.gamma, at.col0 + u * STRIDE, in(u), kOnes);
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[u][j] = db[u][j] = 0ull;
  }
  // the rows' statistics, one round ahead
  const auto stat = [&](const float* from, int64_t row) { return row < rows ? __ldg(from + row) : 0.0f; };
  float next_mu[R], next_r[R];
#pragma unroll
  for (int i = 0; i < R; ++i) next_mu[i] = stat(mean, mine + i), next_r[i] = stat(rstd, mine + i);
  for (int64_t r0 = first; r0 < rows; r0 += step) {
    const int64_t row0 = r0 + at.group * R;
    f2 mu[R], r[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      mu[i] = f2_both(-next_mu[i]), r[i] = f2_both(next_r[i]);
      next_mu[i] = stat(mean, row0 + i + step), next_r[i] = stat(rstd, row0 + i + step);
    }
    load(row0 + (STAGES - 1) * step, (stage + STAGES - 1) % STAGES);
    ring.wait();
    float s0[R], s1[R];
    // h and g of piece u of row i; returns dy
    const auto make = [&](int u, int i, f2 (&h)[4], f2 (&g)[4], f2 (&d)[4]) {
      widen8(*ring.slot(stage, 0, u, i), h);
      widen8(*ring.slot(stage, 1, u, i), d);
      widen8(gw[u], g);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = f2_mul(f2_add(h[j], mu[i]), r[i]), g[j] = f2_mul(g[j], d[j]);
    };
#pragma unroll
    for (int i = 0; i < R; ++i) {
      f2 t0 = 0ull, t1 = 0ull;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f2 h[4], g[4], d[4];
        make(u, i, h, g, d);
        // past the row (and the rows) dy is 0, and so is its part in each sum
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (PARAMS) dg[u][j] = f2_fma(d[j], h[j], dg[u][j]), db[u][j] = f2_add(db[u][j], d[j]);
          t1 = f2_fma(g[j], h[j], t1);
        }
        t0 = f2_add(t0, f2_sum4(g));
      }
      s0[i] = f2_sum(t0), s1[i] = f2_sum(t1);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) s0[i] = warp_sum(s0[i]), s1[i] = warp_sum(s1[i]);
    if constexpr (W > 1) {
      row_meet<W>(s0, s1, sums, turn, at.first);
#pragma unroll
      for (int i = 0; i < R; ++i) s0[i] = low_lanes_sum(s0[i]), s1[i] = low_lanes_sum(s1[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (row0 + i >= rows) continue;
      const f2 a = f2_both(-__fmul_rn(s0[i], inv_n)), b = f2_both(-__fmul_rn(s1[i], inv_n));
      uint16_t* to = p.dx + (row0 + i) * cols + at.col0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!in(u)) continue;
        f2 h[4], g[4], d[4], t[4];
        make(u, i, h, g, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = f2_fma(h[j], b, f2_add(g[j], a));
        if (residual) {
          f2 e[4];
          widen8(*ring.slot(stage, 2, u, i), e);
#pragma unroll
          for (int j = 0; j < 4; ++j) t[j] = f2_fma(t[j], r[i], e[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) t[j] = f2_mul(t[j], r[i]);
        }
        __stcs(reinterpret_cast<uint4*>(to + u * STRIDE), narrow8(t));
      }
    }
    stage = (stage + 1) % STAGES;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!PARAMS || !partial) return;
  float* out = partial + static_cast<int64_t>(block) * 2 * cols;
  if constexpr (PER > 1) {
    // the block's row groups meet in the ring's memory, one after the other
    constexpr int WIDTH = U * STRIDE;
    static_assert(2 * WIDTH * 4 <= Ring::BYTES, "the sums take the ring's place");
    float* meet = reinterpret_cast<float*>(ring_mem);
    __syncthreads();
    for (int g = 0; g < PER; ++g) {
      if (at.group == g) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f2* a = reinterpret_cast<f2*>(meet + at.col0 + u * STRIDE) + j;
            f2* b = reinterpret_cast<f2*>(meet + WIDTH + at.col0 + u * STRIDE) + j;
            *a = g == 0 ? dg[u][j] : f2_add(*a, dg[u][j]);
            *b = g == 0 ? db[u][j] : f2_add(*b, db[u][j]);
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x * 4; c < cols; c += static_cast<int>(blockDim.x) * 4) {
      *reinterpret_cast<float4*>(out + c) = *reinterpret_cast<const float4*>(meet + c);
      *reinterpret_cast<float4*>(out + cols + c) = *reinterpret_cast<const float4*>(meet + WIDTH + c);
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in(u)) continue;
      const int col = at.col0 + u * STRIDE;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        *reinterpret_cast<ulonglong2*>(out + col + 2 * j) = make_ulonglong2(dg[u][j], dg[u][j + 1]);
        *reinterpret_cast<ulonglong2*>(out + cols + col + 2 * j) = make_ulonglong2(db[u][j], db[u][j + 1]);
      }
    }
  }
}

template <int W, int U, int R, int BLOCKS, bool FULL>
__global__ void __launch_bounds__(threads_of_block(W), BLOCKS) norm_backward_kernel(const BackwardArgs p, float* __restrict__ partial) {
  extern __shared__ uint4 ring_mem[];
  allow_next_grid();
  wait_for_prior_grids();
  backward_rows<W, U, R, BLOCKS, FULL, true>(p, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), ring_mem, partial);
}

// Few rows: dgamma and dbeta in the same launch and without a workspace. Blocks from row_blocks on take 64 columns each,
// 8 threads across them, and all rows, which the other blocks have in L2 too; a thread's sums meet the others' in shared
// memory, in the order of the threads.
constexpr int kStrip = 64;
template <int W, int U, int R, int BLOCKS, bool FULL>
__global__ void __launch_bounds__(threads_of_block(W), BLOCKS)
    norm_backward_few_kernel(const BackwardArgs p, int row_blocks, float* __restrict__ dgamma, float* __restrict__ dbeta) {
  extern __shared__ uint4 ring_mem[];
  allow_next_grid();
  wait_for_prior_grids();
  const int block = static_cast<int>(blockIdx.x);
  if (block < row_blocks) {
    backward_rows<W, U, R, BLOCKS, FULL, false>(p, block, row_blocks, ring_mem, nullptr);
    return;
  }
  constexpr int LANES = kStrip / 8, ROWS = threads_of_block(W) / LANES, AHEAD = 4;
  static_assert(2 * ROWS * kStrip * 4 <= Ahead<W, U, R, BLOCKS>::BYTES, "the sums fit into the ring's memory");
  const int row0 = static_cast<int>(threadIdx.x) / LANES, col = (block - row_blocks) * kStrip + (static_cast<int>(threadIdx.x) % LANES) * 8;
  f2 dg[4] = {0ull, 0ull, 0ull, 0ull}, db[4] = {0ull, 0ull, 0ull, 0ull};
  if (col < p.cols) {
    for (int64_t r0 = row0; r0 < p.rows; r0 += AHEAD * ROWS) {
      uint4 xw[AHEAD], yw[AHEAD];
      float mu[AHEAD], r[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int64_t row = r0 + i * ROWS;
        xw[i] = yw[i] = make_uint4(0u, 0u, 0u, 0u);
        mu[i] = r[i] = 0.0f;
        if (row < p.rows) {
          xw[i] = __ldg(reinterpret_cast<const uint4*>(p.x + row * p.cols + col));
          yw[i] = __ldg(reinterpret_cast<const uint4*>(p.dy + row * p.cols + col));
          mu[i] = __ldg(p.mean + row), r[i] = __ldg(p.rstd + row);
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        f2 h[4], d[4];
        widen8(xw[i], h);
        widen8(yw[i], d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dg[j] = f2_fma(d[j], f2_mul(f2_add(h[j], f2_both(-mu[i])), f2_both(r[i])), dg[j]);
          db[j] = f2_add(db[j], d[j]);
        }
      }
    }
  }
  float* meet = reinterpret_cast<float*>(ring_mem);  // [2][ROWS][kStrip]
  float* mine = meet + row0 * kStrip + (static_cast<int>(threadIdx.x) % LANES) * 8;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f2_split(dg[j], mine[2 * j], mine[2 * j + 1]);
    f2_split(db[j], mine[ROWS * kStrip + 2 * j], mine[ROWS * kStrip + 2 * j + 1]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kStrip; i += threads_of_block(W)) {
    const float* part = meet + (i / kStrip) * ROWS * kStrip + i % kStrip;
    float t = part[0];
#pragma unroll 8
    for (int k = 1; k < ROWS; ++k) t = __fadd_rn(t, part[k * kStrip]);
    float* out = i < kStrip ? dgamma : dbeta;
    const int c = (block - row_blocks) * kStrip + i % kStrip;
    if (out && c < p.cols) out[c] = t;
  }
}

// dgamma, dbeta = the sums of `parts` partial sums a column: a block takes 32 of the 2 cols columns, 4 a
// thread; 64 threads share a column (thread y the partials y, y + 64, ..) and are added in order
__global__ void __launch_bounds__(512) norm_params_kernel(const float* __restrict__ partial, int parts, int64_t cols,
                                                          float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float part[64][33];
  allow_next_grid();
  wait_for_prior_grids();
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 32, col = col0 + x * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < 2 * cols) {
#pragma unroll 8
    for (int l = y; l < parts; l += 64) {
      const float4 v = *reinterpret_cast<const float4*>(partial + l * 2 * cols + col);
      s.x = __fadd_rn(s.x, v.x), s.y = __fadd_rn(s.y, v.y), s.z = __fadd_rn(s.z, v.z), s.w = __fadd_rn(s.w, v.w);
    }
  }
  part[y][4 * x] = s.x, part[y][4 * x + 1] = s.y, part[y][4 * x + 2] = s.z, part[y][4 * x + 3] = s.w;
  __syncthreads();
  const int64_t c = col0 + threadIdx.x;
  if (threadIdx.x < 32 && c < 2 * cols) {
    float t = part[0][threadIdx.x];
#pragma unroll
    for (int l = 1; l < 64; ++l) t = __fadd_rn(t, part[l][threadIdx.x]);
    float* out = c < cols ? dgamma : dbeta;
    if (out) out[c < cols ? c : c - cols] = t;
  }
}

// ------------------------------------------------------------------------------------
// rows wider than a block holds: a block a row, read again from L2 for each pass. 2000 x 40000: 75 us, 4.3 TB/s (floor 47):
// three passes over a row, with two sums over the block between them that nothing hides; backward with residual 199 us
// (94): the column sums are a launch that reads X and dY once more from memory, 47 us of it
// ------------------------------------------------------------------------------------
// N values summed over the block, given to all threads
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (&sh)[kWideThreads / 32][N]) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xffffffffu, v[i], d));
  __syncthreads();  // the last sum has been read
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sh[threadIdx.x >> 5][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = sh[0][i];
    for (int w = 1; w < kWideThreads / 32; ++w) v[i] = __fadd_rn(v[i], sh[w][i]);
  }
}

__global__ void __launch_bounds__(kWideThreads) norm_forward_wide_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                         int64_t cols, const uint16_t* __restrict__ gamma,
                                                                         const uint16_t* __restrict__ beta, float eps,
                                                                         float inv_n, uint16_t* __restrict__ y,
                                                                         float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float sh[kWideThreads / 32][1];
  allow_next_grid();
  wait_for_prior_grids();
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const uint16_t* xr = x + row * cols;
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x * 8; c < cols; c += kWideThreads * 8) {
      f2 v[4];
      widen8(__ldg(reinterpret_cast<const uint4*>(xr + c)), v);
      s[0] = __fadd_rn(s[0], f2_sum(f2_sum4(v)));
    }
    block_sum(s, sh);
    const float mu = __fmul_rn(s[0], inv_n);
    s[0] = 0.0f;
    for (int64_t c = threadIdx.x * 8; c < cols; c += kWideThreads * 8) {
      f2 v[4];
      widen8(__ldg(reinterpret_cast<const uint4*>(xr + c)), v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_add(v[j], f2_both(-mu)), v[j] = f2_mul(v[j], v[j]);
      s[0] = __fadd_rn(s[0], f2_sum(f2_sum4(v)));
    }
    block_sum(s, sh);
    const float r = reciprocal_root(__fadd_rn(__fmul_rn(s[0], inv_n), eps));
    if (threadIdx.x == 0 && mean) mean[row] = mu, rstd[row] = r;
    for (int64_t c = threadIdx.x * 8; c < cols; c += kWideThreads * 8) {
      f2 v[4], g[4], b[4];
      widen8(__ldg(reinterpret_cast<const uint4*>(xr + c)), v);
      widen8(param8(gamma, c, true, kOnes), g);
      widen8(param8(beta, c, true, 0u), b);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_fma(f2_mul(f2_add(v[j], f2_both(-mu)), f2_both(r)), g[j], b[j]);
      __stcs(reinterpret_cast<uint4*>(y + row * cols + c), narrow8(v));
    }
  }
}

__global__ void __launch_bounds__(kWideThreads) norm_backward_wide_kernel(
    const uint16_t* dy, const uint16_t* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
    int64_t rows, int64_t cols, const uint16_t* __restrict__ gamma, float inv_n, const uint16_t* residual, uint16_t* dx) {
  __shared__ float sh[kWideThreads / 32][2];
  allow_next_grid();
  wait_for_prior_grids();
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float mu = mean[row], r = rstd[row];
    float s[2] = {0.0f, 0.0f};
    f2 h[4], g[4], d[4];
    const auto load = [&](int64_t c) {
      widen8(__ldg(reinterpret_cast<const uint4*>(x + row * cols + c)), h);
      widen8(*reinterpret_cast<const uint4*>(dy + row * cols + c), d);
      widen8(param8(gamma, c, true, kOnes), g);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = f2_mul(f2_add(h[j], f2_both(-mu)), f2_both(r)), g[j] = f2_mul(g[j], d[j]);
    };
    for (int64_t c = threadIdx.x * 8; c < cols; c += kWideThreads * 8) {
      load(c);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = f2_mul(g[j], h[j]);
      s[0] = __fadd_rn(s[0], f2_sum(f2_sum4(g)));
      s[1] = __fadd_rn(s[1], f2_sum(f2_sum4(h)));
    }
    block_sum(s, sh);
    const f2 a = f2_both(-__fmul_rn(s[0], inv_n)), b = f2_both(-__fmul_rn(s[1], inv_n));
    for (int64_t c = threadIdx.x * 8; c < cols; c += kWideThreads * 8) {
      load(c);
      f2 e[4];
      widen8(residual ? *reinterpret_cast<const uint4*>(residual + row * cols + c) : make_uint4(0u, 0u, 0u, 0u), e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 t = f2_fma(h[j], b, f2_add(g[j], a));
        e[j] = residual ? f2_fma(t, f2_both(r), e[j]) : f2_mul(t, f2_both(r));
      }
      *reinterpret_cast<uint4*>(dx + row * cols + c) = narrow8(e);
    }
  }
}

// the columns' sums of dy h and dy over the rows of block row y: 2048 columns a block, 8 a thread
__global__ void __launch_bounds__(256) norm_columns_wide_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ x,
                                                                const float* __restrict__ mean, const float* __restrict__ rstd,
                                                                int64_t rows, int64_t cols, float* __restrict__ partial) {
  allow_next_grid();
  wait_for_prior_grids();
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (c >= cols) return;
  f2 dg[4] = {0ull, 0ull, 0ull, 0ull}, db[4] = {0ull, 0ull, 0ull, 0ull};
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    f2 h[4], d[4];
    widen8(__ldg(reinterpret_cast<const uint4*>(x + row * cols + c)), h);
    widen8(__ldg(reinterpret_cast<const uint4*>(dy + row * cols + c)), d);
    const f2 mu = f2_both(-mean[row]), r = f2_both(rstd[row]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dg[j] = f2_fma(d[j], f2_mul(f2_add(h[j], mu), r), dg[j]);
      db[j] = f2_add(db[j], d[j]);
    }
  }
  float* out = partial + static_cast<int64_t>(blockIdx.y) * 2 * cols + c;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    *reinterpret_cast<ulonglong2*>(out + 2 * j) = make_ulonglong2(dg[j], dg[j + 1]);
    *reinterpret_cast<ulonglong2*>(out + cols + 2 * j) = make_ulonglong2(db[j], db[j + 1]);
  }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// f(integral constants W, U) for rows of P pieces of 256 columns
template <int W, int U>
struct Shape {
  static constexpr int warps = W, pieces = U;
};
int pieces_of(int64_t cols) { return static_cast<int>((cols + 255) / 256); }
bool few_rows(int64_t rows, int64_t cols) { return rows * pieces_of(cols) <= static_cast<int64_t>(num_sms()) * 16; }
// forward: two or three pieces a lane; one where there are few rows, whose latency counts
template <class F>
auto with_forward_shape(int64_t rows, int64_t cols, F&& f) {
  const int p = pieces_of(cols);
  if (few_rows(rows, cols)) {
    if (p <= 1) return f(Shape<1, 1>{});
    if (p <= 4) return f(Shape<4, 1>{});
    if (p <= 8) return f(Shape<8, 1>{});
    if (p <= 16) return f(Shape<16, 1>{});
  }
  if (p <= 1) return f(Shape<1, 1>{});
  if (p <= 2) return f(Shape<1, 2>{});
  if (p <= 3) return f(Shape<1, 3>{});
  if (p <= 4) return f(Shape<2, 2>{});
  if (p <= 6) return f(Shape<2, 3>{});
  if (p <= 8) return f(Shape<4, 2>{});
  if (p <= 9) return f(Shape<3, 3>{});
  if (p <= 12) return f(Shape<4, 3>{});
  if (p <= 16) return f(Shape<8, 2>{});
  if (p <= 24) return f(Shape<8, 3>{});
  if (p <= 32) return f(Shape<8, 4>{});
  if (p <= 48) return f(Shape<16, 3>{});
  return f(Shape<16, 4>{});
}
// backward: two pieces a lane and rounds of two rows, as far as sixteen warps reach; 512 threads on an SM
template <int W, int U>
struct BackwardShape {
  static constexpr int warps = W, pieces = U, rows = U <= 2 ? 2 : 1;
  static constexpr int blocks = threads_of_block(W) > 256 ? 1 : 512 / threads_of_block(W);
};
template <class F>
auto with_backward_shape(int64_t cols, F&& f) {
  const int p = pieces_of(cols);
  if (p <= 1) return f(BackwardShape<1, 1>{});
  if (p <= 2) return f(BackwardShape<1, 2>{});
  if (p <= 4) return f(BackwardShape<2, 2>{});
  if (p <= 6) return f(BackwardShape<3, 2>{});
  if (p <= 8) return f(BackwardShape<4, 2>{});
  if (p <= 10) return f(BackwardShape<5, 2>{});
  if (p <= 12) return f(BackwardShape<6, 2>{});
  if (p <= 16) return f(BackwardShape<8, 2>{});
  if (p <= 20) return f(BackwardShape<10, 2>{});
  if (p <= 24) return f(BackwardShape<12, 2>{});
  if (p <= 32) return f(BackwardShape<16, 2>{});
  if (p <= 48) return f(BackwardShape<16, 3>{});
  return f(BackwardShape<16, 4>{});
}

// dgamma and dbeta in the launch that computes dX: up to 1024 rows. With residual, in one launch and in two: 1 x 4096
// 2.2 and 4.7 us, 777 x 2304 8.3 and 9.6, 777 x 14336 22 and 31, 1024 x 4096 12.2 and 13.4, 2048 x 4096 22.4 and 18.0.
// Rows alone do not quite decide: 1024 x 2304 takes 12.3 in one launch and would take 10.8 in two, since its rows no
// longer fit beside the columns' blocks in one round.
constexpr int64_t kFewRows = 1024;
bool few_rows_backward(int64_t rows, int64_t cols) { return rows <= kFewRows && cols <= kWidest; }
// blocks of the backward kernel, and so partial sums a column
int64_t backward_blocks(int64_t rows, int64_t cols) {
  if (cols > kWidest) return std::min<int64_t>(rows, 64);
  return with_backward_shape(cols, [&](auto shape) {
    using S = decltype(shape);
    constexpr int PER = rows_of_block(S::warps) * S::rows;
    return std::min<int64_t>((rows + PER - 1) / PER, static_cast<int64_t>(num_sms()) * S::blocks);
  });
}

int check_shape(int64_t rows, int64_t cols, const char* who) {
  if (rows < 1 || cols < 1 || rows > (1 << 30) || cols > (1 << 30))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: rows %lld and cols %lld must be in 1..2^30", who, (long long)rows,
                     (long long)cols);
  if (cols % 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: cols %lld must be a multiple of 8 (16-byte rows)", who, (long long)cols);
  return ZERO_OK;
}

}  // namespace
}  // namespace zgb

using namespace zgb;

extern "C" int fsdp_layernorm_forward(const zero_bf16* X, int64_t rows, int64_t cols, const zero_bf16* gamma,
                                      const zero_bf16* beta, float eps, zero_bf16* Y, float* mean, float* rstd,
                                      zero_stream_t stream) {
  const char* who = "fsdp_layernorm_forward";
  const int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  if (!X || !Y) return set_error(ZERO_ERR_INVALID_ARG, "%s: X or Y is NULL", who);
  if ((mean != nullptr) != (rstd != nullptr))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: pass both mean and rstd, or neither", who);
  if (!(eps >= 0.0f) || !(eps - eps == 0.0f))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if (!aligned16(X) || !aligned16(gamma) || !aligned16(beta) || !aligned16(Y))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: X, gamma, beta and Y must be 16-byte aligned", who);
  if (!aligned4(mean) || !aligned4(rstd))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: mean and rstd must be 4-byte aligned", who);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const float inv_n = 1.0f / static_cast<float>(cols);
  cudaError_t e;
  if (cols > kWidest) {
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(rows, static_cast<int64_t>(num_sms()) * 4));
    e = launch_overlapped(norm_forward_wide_kernel, dim3(grid), dim3(kWideThreads), 0, 1, st, X, rows, cols, gamma, beta,
                          eps, inv_n, Y, mean, rstd);
  } else {
    e = with_forward_shape(rows, cols, [&](auto shape) {
      constexpr int W = decltype(shape)::warps, U = decltype(shape)::pieces, R = (U == 1 && W > 1) || U == 4 || W == 16 ? 1 : 2, PER = rows_of_block(W) * R;
      const auto kernel = cols == W * U * 256 ? norm_forward_kernel<W, U, R, true> : norm_forward_kernel<W, U, R, false>;
      return launch_overlapped(kernel, dim3(static_cast<unsigned>((rows + PER - 1) / PER)), dim3(threads_of_block(W)), 0, 1, st, X,
                               rows, static_cast<int>(cols), gamma, beta, eps, inv_n, Y, mean, rstd);
    });
  }
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

extern "C" int fsdp_layernorm_backward_workspace(int64_t rows, int64_t cols, uint64_t* bytes) {
  const char* who = "fsdp_layernorm_backward_workspace";
  if (!bytes) return set_error(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  const int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  *bytes = few_rows_backward(rows, cols) ? 0 : 8 * static_cast<uint64_t>(backward_blocks(rows, cols)) * static_cast<uint64_t>(cols);
  return ZERO_OK;
}

extern "C" int fsdp_layernorm_backward(const zero_bf16* dY, const zero_bf16* X, const float* mean, const float* rstd,
                                       int64_t rows, int64_t cols, const zero_bf16* gamma, const zero_bf16* residual,
                                       zero_bf16* dX, float* dgamma, float* dbeta, void* workspace,
                                       uint64_t workspace_bytes, zero_stream_t stream) {
  const char* who = "fsdp_layernorm_backward";
  int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  if (!dY || !X || !mean || !rstd || !dX)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: dY, X, mean, rstd or dX is NULL", who);
  if (!aligned16(dY) || !aligned16(X) || !aligned16(gamma) || !aligned16(residual) || !aligned16(dX) ||
      !aligned16(workspace))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: dY, X, gamma, residual, dX and workspace must be 16-byte aligned", who);
  if (!aligned4(mean) || !aligned4(rstd) || !aligned4(dgamma) || !aligned4(dbeta))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: mean, rstd, dgamma and dbeta must be 4-byte aligned", who);
  const bool params = dgamma || dbeta;
  const bool few = params && few_rows_backward(rows, cols);
  float* partial = nullptr;
  if (params && !few) {
    uint64_t need = 0;
    if ((rc = fsdp_layernorm_backward_workspace(rows, cols, &need))) return rc;
    if (!workspace || workspace_bytes < need)
      return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                       workspace ? (unsigned long long)workspace_bytes : 0ull, (unsigned long long)need);
    partial = static_cast<float*>(workspace);
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const float inv_n = 1.0f / static_cast<float>(cols);
  const int64_t blocks = backward_blocks(rows, cols);
  cudaError_t e = cudaSuccess;
  if (cols > kWidest) {
    if (params)  // before dX, which may be dY
      e = launch_overlapped(norm_columns_wide_kernel,
                            dim3(static_cast<unsigned>((cols + 2047) / 2048), static_cast<unsigned>(blocks)), dim3(256), 0, 1, st,
                            dY, X, mean, rstd, rows, cols, partial);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(rows, static_cast<int64_t>(num_sms()) * 4));
    if (e == cudaSuccess)
      e = launch_overlapped(norm_backward_wide_kernel, dim3(grid), dim3(kWideThreads), 0, 1, st, dY, X, mean, rstd, rows,
                            cols, gamma, inv_n, residual, dX);
  } else {
    e = with_backward_shape(cols, [&](auto shape) {
      using S = decltype(shape);
      constexpr int W = S::warps, U = S::pieces, R = S::rows;
      constexpr uint32_t smem = Ahead<W, U, R, S::blocks>::BYTES;
      const bool full = cols == W * U * 256;
      const BackwardArgs p{dY, X, mean, rstd, rows, static_cast<int>(cols), gamma, inv_n, residual, dX};
      const auto go = [&](auto kernel, OncePerDevice& once, int64_t grid, auto... more) {
        int dev = 0;
        cudaError_t q = cudaGetDevice(&dev);
        if (q == cudaSuccess)
          q = once.run(dev, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
          });
        if (q != cudaSuccess) return q;
        return launch_overlapped(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads_of_block(W)), smem, 1, st, p, more...);
      };
      static OncePerDevice once[4];
      if (few) {
        const int64_t strips = (cols + kStrip - 1) / kStrip;
        const auto launch = [&](int64_t grid, int64_t row_blocks) {
          const int n = static_cast<int>(row_blocks);
          return full ? go(norm_backward_few_kernel<W, U, R, S::blocks, true>, once[0], grid, n, dgamma, dbeta)
                      : go(norm_backward_few_kernel<W, U, R, S::blocks, false>, once[1], grid, n, dgamma, dbeta);
        };
        if (dX != dY) return launch(blocks + strips, blocks);
        const cudaError_t q = launch(strips, 0);  // which read dY, before it is written
        return q == cudaSuccess ? launch(blocks, blocks) : q;
      }
      return full ? go(norm_backward_kernel<W, U, R, S::blocks, true>, once[2], blocks, partial)
                  : go(norm_backward_kernel<W, U, R, S::blocks, false>, once[3], blocks, partial);
    });
  }
  if (e == cudaSuccess && params && !few)
    e = launch_overlapped(norm_params_kernel, dim3(static_cast<unsigned>((2 * cols + 31) / 32)), dim3(512), 0, 1, st, partial,
                          static_cast<int>(blocks), cols, dgamma, dbeta);
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}
