// Layer norm over the columns, forward and backward: streaming kernels, bound by HBM bandwidth.
//
//   forward   mean = sum x / n, rstd = 1 / sqrt(sum (x - mean)^2 / n + eps), y = (x - mean) rstd gamma + beta
//   backward  h = (x - mean) rstd, g = dy gamma: dx = rstd (g - sum g / n - h sum (g h) / n) + residual,
//             dgamma = sum over the rows of dy h, dbeta = sum over the rows of dy
//
// A row stays in registers between the passes over it: it is read once. W warps share a row, each lane
// U pieces of 8 columns; wider rows (more than 16 warps' worth) take a block that reads them again from
// L2. All arithmetic is fp32, every output rounded once.
#include <algorithm>

#include "linear_math.cuh"

namespace zgb {
namespace {

constexpr int kMaxWarps = 16;               // of a row held in registers
constexpr int kMaxPieces = 4;               // of a lane
constexpr int kWidest = kMaxWarps * kMaxPieces * 256;
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

// sums over the warps of a row (W consecutive warps of the block), given to all their threads
template <int W, int N>
struct RowSum {
  float part[2][kMaxWarps][N];
};
template <int W, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], RowSum<W, N>& s, int& turn) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xffffffffu, v[i], d));
  if constexpr (W > 1) {
    const int warp = threadIdx.x >> 5, first = warp & ~(W - 1);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s.part[turn][warp][i] = v[i];
    __syncthreads();  // the other half was last read before the barrier ahead of this one
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = s.part[turn][first][i];
#pragma unroll
      for (int w = 1; w < W; ++w) t = __fadd_rn(t, s.part[turn][first + w][i]);
      v[i] = t;
    }
    turn ^= 1;
  }
}

__host__ __device__ constexpr int block_threads(int w) { return w == 16 ? 512 : 256; }

template <int W, int U>
__global__ void __launch_bounds__(block_threads(W)) norm_forward_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                            const uint16_t* __restrict__ gamma,
                                                            const uint16_t* __restrict__ beta, float eps, float inv_n,
                                                            uint16_t* __restrict__ y, float* __restrict__ mean,
                                                            float* __restrict__ rstd) {
  constexpr int PER = block_threads(W) / 32 / W;  // rows of a block at a time
  __shared__ RowSum<W, 1> sums;
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = ((warp % W) * 32 + lane) * 8;
  int turn = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * PER;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * PER; r0 < rows; r0 += step) {
    const int64_t row = r0 + warp / W;
    const bool there = row < rows;
    uint4 in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in[u] = make_uint4(0u, 0u, 0u, 0u);
      if (there && col0 + u * W * 256 < cols) in[u] = __ldcs(reinterpret_cast<const uint4*>(x + row * cols + col0 + u * W * 256));
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f2 v[4];
      widen8(in[u], v);
      s[0] = __fadd_rn(s[0], f2_sum(f2_sum4(v)));
    }
    row_sum<W, 1>(s, sums, turn);
    const float mu = __fmul_rn(s[0], inv_n);
    s[0] = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (col0 + u * W * 256 >= cols) continue;
      f2 v[4];
      widen8(in[u], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_add(v[j], f2_both(-mu)), v[j] = f2_mul(v[j], v[j]);
      s[0] = __fadd_rn(s[0], f2_sum(f2_sum4(v)));
    }
    row_sum<W, 1>(s, sums, turn);
    const float r = reciprocal_root(__fadd_rn(__fmul_rn(s[0], inv_n), eps));
    if (!there) continue;
    if (lane == 0 && warp % W == 0 && mean) mean[row] = mu, rstd[row] = r;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = col0 + u * W * 256;
      if (col >= cols) continue;
      f2 v[4], g[4], b[4];
      widen8(in[u], v);
      widen8(param8(gamma, col, true, kOnes), g);
      widen8(param8(beta, col, true, 0u), b);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_fma(f2_mul(f2_add(v[j], f2_both(-mu)), f2_both(r)), g[j], b[j]);
      __stcs(reinterpret_cast<uint4*>(y + row * cols + col), narrow8(v));
    }
  }
}

// Backward. partial: nullable, [blocks][2][cols]: a block's sums of dy h and dy over its rows.
template <int W, int U>
__global__ void __launch_bounds__(block_threads(W)) norm_backward_kernel(
    const uint16_t* dy, const uint16_t* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
    int64_t rows, int cols, const uint16_t* __restrict__ gamma, float inv_n, const uint16_t* residual, uint16_t* dx,
    float* __restrict__ partial) {
  constexpr int PER = block_threads(W) / 32 / W;
  __shared__ RowSum<W, 2> sums;
  __shared__ __align__(16) float meet[PER > 1 ? 2 * W * U * 256 : 4];
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = ((warp % W) * 32 + lane) * 8;
  uint4 gw[U];
  f2 dg[U][4], db[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    gw[u] = param8(gamma, col0 + u * W * 256, col0 + u * W * 256 < cols, kOnes);
#pragma unroll
    for (int j = 0; j < 4; ++j) dg[u][j] = db[u][j] = 0ull;
  }
  int turn = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * PER;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * PER; r0 < rows; r0 += step) {
    const int64_t row = r0 + warp / W;
    const bool there = row < rows;
    uint4 xw[U], yw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xw[u] = yw[u] = make_uint4(0u, 0u, 0u, 0u);
      const int col = col0 + u * W * 256;
      if (there && col < cols) {
        xw[u] = __ldcs(reinterpret_cast<const uint4*>(x + row * cols + col));
        yw[u] = __ldcs(reinterpret_cast<const uint4*>(dy + row * cols + col));
      }
    }
    const float mu = there ? mean[row] : 0.0f, r = there ? rstd[row] : 0.0f;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (col0 + u * W * 256 >= cols) continue;
      f2 h[4], g[4], d[4];
      widen8(xw[u], h);
      widen8(yw[u], d);
      widen8(gw[u], g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = f2_mul(f2_add(h[j], f2_both(-mu)), f2_both(r));
        dg[u][j] = f2_fma(d[j], h[j], dg[u][j]);
        db[u][j] = f2_add(db[u][j], d[j]);
        g[j] = f2_mul(g[j], d[j]);
        h[j] = f2_mul(g[j], h[j]);
      }
      s[0] = __fadd_rn(s[0], f2_sum(f2_sum4(g)));
      s[1] = __fadd_rn(s[1], f2_sum(f2_sum4(h)));
    }
    row_sum<W, 2>(s, sums, turn);
    if (!there) continue;
    const f2 a = f2_both(__fmul_rn(s[0], inv_n)), b = f2_both(-__fmul_rn(s[1], inv_n));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = col0 + u * W * 256;
      if (col >= cols) continue;
      f2 h[4], g[4], d[4], e[4];
      widen8(xw[u], h);
      widen8(yw[u], d);
      widen8(gw[u], g);
      const uint4 rw = residual ? __ldcs(reinterpret_cast<const uint4*>(residual + row * cols + col)) : make_uint4(0u, 0u, 0u, 0u);
      widen8(rw, e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = f2_mul(f2_add(h[j], f2_both(-mu)), f2_both(r));
        const f2 t = f2_fma(h[j], b, f2_add(f2_mul(g[j], d[j]), f2_mul(a, f2_both(-1.0f))));
        e[j] = residual ? f2_fma(t, f2_both(r), e[j]) : f2_mul(t, f2_both(r));
      }
      __stcs(reinterpret_cast<uint4*>(dx + row * cols + col), narrow8(e));
    }
  }
  if (!partial) return;
  // the block's row groups meet in shared memory, one after the other
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
  if constexpr (PER > 1) {
    constexpr int WIDTH = W * U * 256;
    for (int g = 0; g < PER; ++g) {
      if (warp / W == g) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f2* a = reinterpret_cast<f2*>(meet + col0 + u * W * 256) + j;
            f2* b = reinterpret_cast<f2*>(meet + WIDTH + col0 + u * W * 256) + j;
            *a = g == 0 ? dg[u][j] : f2_add(*a, dg[u][j]);
            *b = g == 0 ? db[u][j] : f2_add(*b, db[u][j]);
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x * 4; c < cols; c += blockDim.x * 4) {
      *reinterpret_cast<float4*>(out + c) = *reinterpret_cast<const float4*>(meet + c);
      *reinterpret_cast<float4*>(out + cols + c) = *reinterpret_cast<const float4*>(meet + WIDTH + c);
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = col0 + u * W * 256;
      if (col >= cols) continue;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        *reinterpret_cast<ulonglong2*>(out + col + 2 * j) = make_ulonglong2(dg[u][j], dg[u][j + 1]);
        *reinterpret_cast<ulonglong2*>(out + cols + col + 2 * j) = make_ulonglong2(db[u][j], db[u][j + 1]);
      }
    }
  }
}

// dgamma, dbeta = the sums of `parts` partial sums a column: a block takes 32 of the 2 cols columns, 4 a
// thread; 32 threads share a column (thread y the partials y, y + 32, ..) and are added in order
__global__ void __launch_bounds__(256) norm_params_kernel(const float* __restrict__ partial, int parts, int64_t cols,
                                                          float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float part[32][33];
  allow_next_grid();
  wait_for_prior_grids();
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 32, col = col0 + x * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < 2 * cols) {
#pragma unroll 4
    for (int l = y; l < parts; l += 32) {
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
    for (int l = 1; l < 32; ++l) t = __fadd_rn(t, part[l][threadIdx.x]);
    float* out = c < cols ? dgamma : dbeta;
    if (out) out[c < cols ? c : c - cols] = t;
  }
}

// ------------------------------------------------------------------------------------
// rows wider than the registers: a block a row, read again from L2 for each pass
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

// Warps of a row (0: wider than the registers) and pieces of a lane. The fewest warps whose lanes hold the
// row in kMaxPieces pieces, so that most rows' sums stay inside a warp; more where there are few rows.
struct Shape {
  int warps, pieces;
};
Shape shape_of(int64_t rows, int64_t cols) {
  if (cols > kWidest) return {0, 0};
  int w = 1;
  while (w * kMaxPieces * 256 < cols) w *= 2;
  const int64_t warps = static_cast<int64_t>(num_sms()) * 16;
  while (w < kMaxWarps && w * 256 < cols && rows * w * 2 <= warps) w *= 2;
  return {w, static_cast<int>((cols + w * 256 - 1) / (w * 256))};
}
int64_t rows_at_once(int w) { return block_threads(w) / 32 / w; }

// blocks of the backward kernel, and so partial sums a column
constexpr int kBackwardBlocks = 2;  // per SM
int backward_blocks(int64_t rows, int64_t cols) {
  const Shape s = shape_of(rows, cols);
  const int64_t most = static_cast<int64_t>(num_sms()) * kBackwardBlocks;
  if (s.warps == 0) return static_cast<int>(std::min<int64_t>(rows, 64));
  const int64_t per = rows_at_once(s.warps);
  return static_cast<int>(std::min<int64_t>((rows + per - 1) / per, s.warps == 16 ? most / 2 : most));
}

// f(integral constants W, U)
template <int W, class F>
cudaError_t with_pieces(int pieces, F&& f) {
  switch (pieces) {
    case 1: return f(ActTag<W>{}, ActTag<1>{});
    case 2: return f(ActTag<W>{}, ActTag<2>{});
    case 3: return f(ActTag<W>{}, ActTag<3>{});
    default: return f(ActTag<W>{}, ActTag<4>{});
  }
}
template <class F>
cudaError_t with_shape(const Shape& s, F&& f) {
  switch (s.warps) {
    case 1: return with_pieces<1>(s.pieces, f);
    case 2: return with_pieces<2>(s.pieces, f);
    case 4: return with_pieces<4>(s.pieces, f);
    case 8: return with_pieces<8>(s.pieces, f);
    default: return with_pieces<16>(s.pieces, f);
  }
}

int check_shape(int64_t rows, int64_t cols, const char* who) {
  if (rows < 1 || cols < 1 || rows > (int64_t(1) << 40) || cols > (1 << 30) || rows > (int64_t(1) << 61) / cols)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: rows %lld and cols %lld must be >= 1 (at most 2^40 and 2^30)", who,
                     (long long)rows, (long long)cols);
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
  const Shape s = shape_of(rows, cols);
  cudaError_t e;
  if (s.warps == 0) {
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(rows, static_cast<int64_t>(num_sms()) * 4));
    e = launch_overlapped(norm_forward_wide_kernel, dim3(grid), dim3(kWideThreads), 0, 1, st, X, rows, cols, gamma, beta,
                          eps, inv_n, Y, mean, rstd);
  } else {
    const int64_t per = rows_at_once(s.warps);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((rows + per - 1) / per, static_cast<int64_t>(num_sms()) * 64));
    e = with_shape(s, [&](auto w, auto u) {
      constexpr int W = decltype(w)::value, U = decltype(u)::value;
      return launch_overlapped(norm_forward_kernel<W, U>, dim3(grid), dim3(block_threads(W)), 0, 1, st, X, rows,
                               static_cast<int>(cols), gamma, beta, eps, inv_n, Y, mean, rstd);
    });
  }
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

extern "C" int fsdp_layernorm_backward_workspace(int64_t rows, int64_t cols, uint64_t* bytes) {
  const char* who = "fsdp_layernorm_backward_workspace";
  if (!bytes) return set_error(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  const int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  *bytes = 8 * static_cast<uint64_t>(backward_blocks(rows, cols)) * static_cast<uint64_t>(cols);
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
  float* partial = nullptr;
  if (params) {
    uint64_t need = 0;
    if ((rc = fsdp_layernorm_backward_workspace(rows, cols, &need))) return rc;
    if (!workspace || workspace_bytes < need)
      return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                       workspace ? (unsigned long long)workspace_bytes : 0ull, (unsigned long long)need);
    partial = static_cast<float*>(workspace);
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const float inv_n = 1.0f / static_cast<float>(cols);
  const Shape s = shape_of(rows, cols);
  const int blocks = backward_blocks(rows, cols);
  cudaError_t e = cudaSuccess;
  if (s.warps == 0) {
    if (params)  // before dX, which may be dY
      e = launch_overlapped(norm_columns_wide_kernel, dim3(static_cast<unsigned>((cols + 2047) / 2048), blocks), dim3(256), 0,
                            1, st, dY, X, mean, rstd, rows, cols, partial);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(rows, static_cast<int64_t>(num_sms()) * 4));
    if (e == cudaSuccess)
      e = launch_overlapped(norm_backward_wide_kernel, dim3(grid), dim3(kWideThreads), 0, 1, st, dY, X, mean, rstd, rows,
                            cols, gamma, inv_n, residual, dX);
  } else {
    e = with_shape(s, [&](auto w, auto u) {
      constexpr int W = decltype(w)::value, U = decltype(u)::value;
      return launch_overlapped(norm_backward_kernel<W, U>, dim3(static_cast<unsigned>(blocks)), dim3(block_threads(W)), 0, 1,
                               st, dY, X, mean, rstd, rows, static_cast<int>(cols), gamma, inv_n, residual, dX, partial);
    });
  }
  if (e == cudaSuccess && params)
    e = launch_overlapped(norm_params_kernel, dim3(static_cast<unsigned>((2 * cols + 31) / 32)), dim3(256), 0, 1, st, partial,
                          blocks, cols, dgamma, dbeta);
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}
