// 8-bit activation checkpoints (pack, unpack) and the activation's backward, which reads
// them: streaming kernels, bound by HBM bandwidth.
//
//   pack     x [rows, cols] bf16 -> codes int8, one power-of-two scale byte per 32 columns
//   unpack   act(code * 2^(byte - 127)) -> bf16
//   act_backward   dZ = bf16(dY act'(Z)), db = column sums of dY act'(Z) in fp32
//
// A thread has 8 columns, four threads a group; where the last group of a row is cut short, its
// threads past the row hold zeros.
#include <algorithm>

#include "linear_math.cuh"

namespace zgb {
namespace {

constexpr int kThreads = 256;

// 8 values as 4 pairs
__device__ __forceinline__ void widen8(const uint4& w, f2 (&x)[4]) {
  x[0] = f2_from_bf16x2(w.x), x[1] = f2_from_bf16x2(w.y), x[2] = f2_from_bf16x2(w.z), x[3] = f2_from_bf16x2(w.w);
}
__device__ __forceinline__ uint4 narrow8(const f2 (&x)[4]) {
  return make_uint4(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]), f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
}
__device__ __forceinline__ void decode8(const uint2& c, uint32_t byte, f2 (&x)[4]) {
  const float s = ckpt_scale(byte);
#pragma unroll
  for (int j = 0; j < 2; ++j) x[j] = ckpt_values2(c.x, j, s), x[2 + j] = ckpt_values2(c.y, j, s);
}
// codes of 8 values whose group has scale byte b
__device__ __forceinline__ uint2 encode8(f2 (&v)[4], uint32_t b) {
  if (b >= 248u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = ckpt_clamped(v[j], b);
  }
  const float inv = ckpt_inv_scale(b);
  return make_uint2(ckpt_code4(v[0], v[1], inv), ckpt_code4(v[2], v[3], inv));
}
__device__ __forceinline__ float amax8(const f2 (&v)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = amax2(m, v[j]);
  return m;
}

// ------------------------------------------------------------------------------------
// one sweep over memory: pack, unpack, activation backward without column sums
// ------------------------------------------------------------------------------------
constexpr int kWalkBlocks = 48;  // blocks per SM at most; 32 and 16: pack 8192 x 14336 57.4 and 62 us, 56.1
// units a thread has in flight (4 and 3: pack 8192 x 14336 56.1 and 58.9 us, 8192 x 14344 77.8 and 70.9)
__host__ __device__ constexpr int walk_units(bool flat) { return flat ? 4 : 3; }

// A matrix as units of 8 columns, four to a group of the checkpoint, walked by all threads together:
// a warp's accesses are contiguous. FLAT: widths of whole groups, rows need not be known (also where
// there is no checkpoint). Otherwise a row has units up to the end of its last group, those past its
// columns without data, and a thread steps by whole rows and units instead of dividing.
struct WalkDims {
  int64_t rows, cols, units;        // units: of a row, or (flat) of the matrix
  int64_t step_rows, step_units;    // a step of all threads
};
template <bool FLAT>
struct Walk {
  int64_t row, unit;
  __device__ __forceinline__ explicit Walk(const WalkDims& d) {
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;  // below 2^31
    row = 0, unit = i;
    if (!FLAT && d.units <= unit) {
      row = i / static_cast<uint32_t>(d.units);
      unit = i - static_cast<uint32_t>(row) * static_cast<uint32_t>(d.units);
    }
  }
  // the four units of a group are there together, though some may have no data
  __device__ __forceinline__ bool there(const WalkDims& d) const { return FLAT ? unit < d.units : row < d.rows; }
  __device__ __forceinline__ bool data(const WalkDims& d) const { return there(d) && (FLAT || 8 * unit < d.cols); }
  __device__ __forceinline__ int64_t at(const WalkDims& d) const { return FLAT ? 8 * unit : row * d.cols + 8 * unit; }
  __device__ __forceinline__ int64_t group(const WalkDims& d) const {
    return FLAT ? unit >> 2 : row * (d.units >> 2) + (unit >> 2);
  }
  __device__ __forceinline__ void step(const WalkDims& d) {
    unit += d.step_units;
    if constexpr (!FLAT) {
      row += d.step_rows;
      if (unit >= d.units) unit -= d.units, ++row;
    }
  }
};

// Bound by HBM: 8192 x 14336 56 us, 6.4 TB/s (with the codes written); 8192 x 14344, groups cut
// short, 71 us; 33 x 1160 2.8 us, a launch.
template <bool FLAT>
__global__ void __launch_bounds__(kThreads) ckpt8_pack_kernel(const uint16_t* __restrict__ x, const WalkDims d,
                                                              int8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  allow_next_grid();
  Walk<FLAT> w(d);
  wait_for_prior_grids();
  constexpr int UN = walk_units(FLAT);
  while (w.there(d)) {
    uint4 in[UN];
    Walk<FLAT> a = w;
#pragma unroll
    for (int k = 0; k < UN; ++k, a.step(d)) {
      in[k] = make_uint4(0u, 0u, 0u, 0u);
      if (a.data(d)) in[k] = __ldcs(reinterpret_cast<const uint4*>(x + a.at(d)));
    }
#pragma unroll
    for (int k = 0; k < UN; ++k, w.step(d)) {
      if (!w.there(d)) return;
      f2 v[4];
      widen8(in[k], v);
      float amax = amax8(v);
      // units and steps are multiples of 4: a group's lanes are in the loop together
      const uint32_t four = 0xFu << (threadIdx.x & 28u);
      amax = max_nan(amax, __shfl_xor_sync(four, amax, 1));
      amax = max_nan(amax, __shfl_xor_sync(four, amax, 2));
      const uint32_t byte = ckpt_byte(amax);
      const uint2 c = encode8(v, byte);
      if (w.data(d)) {
        *reinterpret_cast<uint2*>(codes + w.at(d)) = c;
        if ((w.unit & 3) == 0) scales[w.group(d)] = static_cast<uint8_t>(byte);
      }
    }
  }
}

// Bound by HBM: 8192 x 14336 54 us, 6.6 TB/s; 8192 x 14344 59 us. With erf's GELU by its instructions (the
// polynomial; 70 % of the issue slots, half of the DRAM rate): 74-77 us.
template <int ACT, bool FLAT>
__global__ void __launch_bounds__(kThreads) ckpt8_unpack_kernel(const int8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, const WalkDims d,
                                                                uint16_t* __restrict__ out) {
  allow_next_grid();
  Walk<FLAT> w(d);
  wait_for_prior_grids();
  constexpr int UN = walk_units(FLAT);
  while (w.there(d)) {
    uint2 in[UN];
    uint32_t byte[UN];
    Walk<FLAT> a = w;
#pragma unroll
    for (int k = 0; k < UN; ++k, a.step(d)) {
      if (a.data(d)) {
        in[k] = __ldcs(reinterpret_cast<const uint2*>(codes + a.at(d)));
        byte[k] = scales[a.group(d)];
      }
    }
#pragma unroll
    for (int k = 0; k < UN; ++k, w.step(d)) {
      if (w.data(d)) {
        f2 v[4];
        decode8(in[k], byte[k], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = act_fwd<ACT>(v[j]);
        __stcs(reinterpret_cast<uint4*>(out + w.at(d)), narrow8(v));
      }
    }
  }
}

// Activation backward without column sums. 8192 x 14336 from 8 bits 91 us, 106 us in the strips below.
template <int ACT, bool Z8, bool FLAT>
__global__ void __launch_bounds__(kThreads) act_backward_walk_kernel(const uint16_t* dy, const uint16_t* __restrict__ z,
                                                                     const int8_t* __restrict__ codes,
                                                                     const uint8_t* __restrict__ scales,
                                                                     const WalkDims d, uint16_t* dz) {
  constexpr int UN = 2;
  allow_next_grid();
  Walk<FLAT> w(d);
  wait_for_prior_grids();
  while (w.there(d)) {
    uint4 gw[UN], zw[UN];
    uint2 cw[UN];
    uint32_t byte[UN];
    Walk<FLAT> a = w;
#pragma unroll
    for (int k = 0; k < UN; ++k, a.step(d)) {
      if (a.data(d)) {
        gw[k] = __ldcs(reinterpret_cast<const uint4*>(dy + a.at(d)));
        if constexpr (Z8) {
          cw[k] = __ldcs(reinterpret_cast<const uint2*>(codes + a.at(d)));
          byte[k] = scales[a.group(d)];
        } else {
          zw[k] = __ldcs(reinterpret_cast<const uint4*>(z + a.at(d)));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < UN; ++k, w.step(d)) {
      if (w.data(d)) {
        f2 g[4], v[4];
        widen8(gw[k], g);
        if constexpr (Z8) decode8(cw[k], byte[k], v);
        else widen8(zw[k], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = f2_mul(g[j], act_grad<ACT>(v[j]));
        __stcs(reinterpret_cast<uint4*>(dz + w.at(d)), narrow8(g));
      }
    }
  }
}

// Activation backward with the column sums over a large matrix: the same sweep, by a number of
// threads that is a multiple of the 8-column units of a row, so that a thread stays in its columns
// and sums them over its rows. `lanes` rows are swept at a time and leave as many partial sums a
// column in the workspace, [lanes][cols] fp32.
constexpr int kSweepBlocks = 4;  // blocks per SM, all resident
template <int ACT, bool Z8>
__global__ void __launch_bounds__(kThreads, kSweepBlocks) act_backward_sweep_kernel(
    const uint16_t* dy, const uint16_t* __restrict__ z, const int8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, int64_t rows, int64_t cols, int lanes, uint16_t* dz, float* __restrict__ partial) {
  constexpr int UN = 2;
  allow_next_grid();
  wait_for_prior_grids();
  const int row_units = static_cast<int>(cols / 8), tid = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
  const int lane = tid / row_units, col = (tid - lane * row_units) * 8;
  if (lane >= lanes) return;
  const int64_t groups = (cols + kCkptGroup - 1) / kCkptGroup, step = static_cast<int64_t>(lanes) * row_units;
  int64_t i0 = tid, s0 = lane * groups + (col >> 5);  // this thread's unit of row r0, and its group
  f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
  for (int64_t r0 = lane; r0 < rows; r0 += UN * lanes, i0 += UN * step, s0 += UN * lanes * groups) {
    uint4 gw[UN], zw[UN];
    uint2 cw[UN];
    uint32_t byte[UN];
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (r0 + k * lanes < rows) {
        gw[k] = __ldcs(reinterpret_cast<const uint4*>(dy) + i0 + k * step);
        if constexpr (Z8) {
          cw[k] = __ldcs(reinterpret_cast<const uint2*>(codes) + i0 + k * step);
          byte[k] = scales[s0 + k * lanes * groups];
        } else {
          zw[k] = __ldcs(reinterpret_cast<const uint4*>(z) + i0 + k * step);
        }
      }
#pragma unroll
    for (int k = 0; k < UN; ++k)
      if (r0 + k * lanes < rows) {
        f2 g[4], v[4];
        widen8(gw[k], g);
        if constexpr (Z8) decode8(cw[k], byte[k], v);
        else widen8(zw[k], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = f2_mul(g[j], act_grad<ACT>(v[j]));
        if (dz) __stcs(reinterpret_cast<uint4*>(dz) + i0 + k * step, narrow8(g));
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = f2_add(sum[j], g[j]);
      }
  }
  ulonglong2* out = reinterpret_cast<ulonglong2*>(partial + static_cast<int64_t>(lane) * cols + col);
  out[0] = make_ulonglong2(sum[0], sum[1]);
  out[1] = make_ulonglong2(sum[2], sum[3]);
}

// db = the sum of `lanes` partial sums a column: a block takes 32 columns, 4 a thread; 32 threads share
// a column (thread y the partials y, y + 32, ..) and are added in order
__global__ void __launch_bounds__(kThreads) sum_partials_kernel(const float* __restrict__ partial, int lanes,
                                                                int64_t cols, float* __restrict__ db) {
  __shared__ float part[32][33];
  allow_next_grid();
  wait_for_prior_grids();
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * 32, col = col0 + x * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < cols) {
#pragma unroll 4
    for (int l = y; l < lanes; l += 32) {
      const float4 v = *reinterpret_cast<const float4*>(partial + l * cols + col);
      s.x = __fadd_rn(s.x, v.x), s.y = __fadd_rn(s.y, v.y), s.z = __fadd_rn(s.z, v.z), s.w = __fadd_rn(s.w, v.w);
    }
  }
  part[y][4 * x] = s.x, part[y][4 * x + 1] = s.y, part[y][4 * x + 2] = s.z, part[y][4 * x + 3] = s.w;
  __syncthreads();
  if (threadIdx.x < 32 && col0 + threadIdx.x < cols) {
    float t = part[0][threadIdx.x];
#pragma unroll
    for (int l = 1; l < 32; ++l) t = __fadd_rn(t, part[l][threadIdx.x]);
    db[col0 + threadIdx.x] = t;
  }
}

// Activation backward with the column sums, without a workspace, for smaller matrices, where one
// launch counts more. A cluster of blocks takes a strip of 8 LANES columns, each block a run of its
// rows: LANES threads across the strip (8 columns each),
// kThreads / LANES rows at a time, four of a thread's rows in flight. A thread sums its rows in
// order; a block adds its row lanes in order through shared memory, and block c of the cluster
// the columns c, c + blocks, .. of all blocks' sums, in block order: the same bits every call, and no
// memory between launches.
constexpr int kActBlocks = 2;  // resident blocks per SM of act_backward_kernel (its registers allow no more)
template <int ACT, bool Z8, int LANES>
__global__ void __launch_bounds__(kThreads, kActBlocks) act_backward_kernel(const uint16_t* dy, const uint16_t* __restrict__ z,
                                                                   const int8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales, int64_t rows,
                                                                   int64_t cols, int64_t rows_per_block, int64_t strip0,
                                                                   uint16_t* dz, float* __restrict__ db) {
  constexpr int RL = kThreads / LANES, STRIP = 8 * LANES, UN = ACT == FSDP_ACT_NONE ? 4 : 2;
  __shared__ float part[RL][STRIP + 1];
  __shared__ float sums[STRIP];
  allow_next_grid();
  wait_for_prior_grids();
  const int64_t groups = (cols + kCkptGroup - 1) / kCkptGroup;
  const int lane = threadIdx.x % LANES, rl = threadIdx.x / LANES;
  const int64_t col0 = (strip0 + blockIdx.y) * STRIP, col = col0 + lane * 8;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * rows_per_block, last = min(first + rows_per_block, rows);
  f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
  if (col < cols) {
    struct Batch {
      uint4 g[UN], z[Z8 ? 1 : UN];
      uint2 c[Z8 ? UN : 1];
      uint32_t byte[Z8 ? UN : 1];
    };
    const auto load = [&](int64_t r0, Batch& t) {
#pragma unroll
      for (int k = 0; k < UN; ++k) {
        const int64_t row = r0 + k * RL;
        if (row < last) {
          t.g[k] = *reinterpret_cast<const uint4*>(dy + row * cols + col);
          if constexpr (ACT != FSDP_ACT_NONE) {
            if constexpr (Z8) {
              t.c[k] = __ldg(reinterpret_cast<const uint2*>(codes + row * cols + col));
              t.byte[k] = scales[row * groups + (col >> 5)];
            } else {
              t.z[k] = __ldg(reinterpret_cast<const uint4*>(z + row * cols + col));
            }
          }
        }
      }
    };
    const auto use = [&](int64_t r0, const Batch& t) {
#pragma unroll
      for (int k = 0; k < UN; ++k) {
        const int64_t row = r0 + k * RL;
        if (row < last) {
          f2 g[4], v[4];
          widen8(t.g[k], g);
          if constexpr (ACT != FSDP_ACT_NONE) {
            if constexpr (Z8) decode8(t.c[k], t.byte[k], v);
            else widen8(t.z[k], v);
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = f2_mul(g[j], act_grad<ACT>(v[j]));
          }
          if (dz) *reinterpret_cast<uint4*>(dz + row * cols + col) = narrow8(g);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[j] = f2_add(sum[j], g[j]);
        }
      }
    };
    // two batches of rows: one is loaded while the other is used
    Batch t[2];
    load(first + rl, t[0]);
    for (int64_t r0 = first + rl; r0 < last; r0 += 2 * UN * RL) {
      load(r0 + UN * RL, t[1]);
      use(r0, t[0]);
      load(r0 + 2 * UN * RL, t[0]);
      use(r0 + UN * RL, t[1]);
    }
  }
  if (!db) return;  // the same for every block of a cluster
#pragma unroll
  for (int j = 0; j < 4; ++j) f2_split(sum[j], part[rl][lane * 8 + 2 * j], part[rl][lane * 8 + 2 * j + 1]);
  __syncthreads();
  if (threadIdx.x < STRIP) {
    float s = part[0][threadIdx.x];
#pragma unroll 8
    for (int i = 1; i < RL; ++i) s = __fadd_rn(s, part[i][threadIdx.x]);
    sums[threadIdx.x] = s;
  }
  cluster_sync_all();
  const int blocks = static_cast<int>(gridDim.x);  // one cluster across the rows
  const int c = static_cast<int>(blockIdx.x) + static_cast<int>(threadIdx.x) * blocks;
  if (c < STRIP) {
    float s = 0.0f;
    for (int b = 0; b < blocks; ++b) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&sums[c]), b)) : "memory");
      s = b == 0 ? v : __fadd_rn(s, v);
    }
    if (col0 + c < cols) db[col0 + c] = s;
  }
  cluster_sync_all();  // no block leaves while its sums are read
}

unsigned int grid_for(int64_t threads, int blocks_per_sm) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  return static_cast<unsigned int>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms()) * blocks_per_sm));
}

// a walk over a [rows, cols] matrix, with its checkpoint's groups or without
struct Walking {
  bool flat;
  unsigned int blocks;
  WalkDims d;
  Walking(int64_t rows, int64_t cols, bool groups) {
    flat = !groups || cols % kCkptGroup == 0;
    const int64_t row_units = flat ? cols / 8 : (cols + kCkptGroup - 1) / kCkptGroup * 4;
    // one unit a thread until there are four blocks per SM, then as many as a thread has in flight (more
    // blocks that use part of it: pack 4096 x 4096 8.2 -> 12.9 us)
    const int64_t units = rows * row_units;
    blocks = std::max(grid_for(units, 4), grid_for(units / walk_units(flat), kWalkBlocks));
    const int64_t step = static_cast<int64_t>(blocks) * kThreads;
    d = {rows, cols, flat ? rows * row_units : row_units, flat ? 0 : step / row_units, flat ? step : step % row_units};
  }
};

constexpr int kMaxCluster = 16;  // blocks; more than 8 a kernel has to allow
// Clusters of 1 .. kMaxCluster blocks of one kernel that are resident at once, asked for once per device
class ResidentClusters {
 public:
  template <class... P>
  cudaError_t get(int dev, void (*kernel)(P...), const int** per_size) {
    int* known = known_[dev & 63];
    *per_size = known;
    return once_.run(dev, [&] {
      cudaError_t q = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (q != cudaSuccess) return q;
      for (unsigned int n = 1; n <= kMaxCluster; ++n) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n), cfg.blockDim = dim3(kThreads);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = n, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr, cfg.numAttrs = 1;
        if ((q = cudaOccupancyMaxActiveClusters(&known[n], kernel, &cfg)) != cudaSuccess) return q;
      }
      return cudaSuccess;
    });
  }

 private:
  OncePerDevice once_;
  int known_[64][kMaxCluster + 1] = {};
};

struct Strips {
  int lanes = 0, blocks = 1;
  float score = 0.0f;
};
// `best`, or strips of 8 LANES columns with n blocks across the rows (one cluster; no fewer than four
// rows a thread), whichever scores higher: the share of the GPU's block slots that work over
// the waves taken, less for larger clusters, whose sums take longer to meet, and for narrower strips,
// whose rows are shorter runs of memory (32 columns: 64 bytes). Measured against a strip width by
// thresholds of the columns: column sums of 8192 x 4096 alone 10.4 us, 20.1 (32 columns); 8192 x 6144
// 16.9, 21.0 (256 columns); from 8 bits 16384 x 1536 33.5, 47.1 (clusters of 6, of which 46 and not 50
// are resident); 400 x 10240 7.8, 12.3; level where the threshold was right (8192 x 14336 40). Clusters of
// up to 16 against up to 8: 9879 x 544 with GELU 11.6, 15.5; 16384 x 512 with SiLU 11.4, 14.6.
template <int ACT, bool Z8, int LANES>
cudaError_t consider_strips(int dev, int slots, int64_t rows, int64_t cols, Strips* best) {
  static ResidentClusters resident;
  const int* per_size = nullptr;
  const cudaError_t e = resident.get(dev, act_backward_kernel<ACT, Z8, LANES>, &per_size);
  if (e != cudaSuccess) return e;
  constexpr int RL = kThreads / LANES, STRIP = 8 * LANES;
  constexpr float WIDE = LANES == 32 ? 1.2f : LANES == 16 ? 1.1f : LANES == 8 ? 1.0f : 0.9f;
  const int64_t strips = (cols + STRIP - 1) / STRIP;
  for (int n = 1; n <= kMaxCluster && (n == 1 || rows > static_cast<int64_t>(n - 1) * RL * 4); ++n) {
    if (per_size[n] < 1) continue;
    const int64_t waves = (strips + per_size[n] - 1) / per_size[n];
    const float busy = static_cast<float>(strips * n) / static_cast<float>(waves * slots);
    const float score = busy * (1.0f - 0.03f * n) * WIDE;
    if (score > best->score) best->score = score, best->lanes = LANES, best->blocks = n;
  }
  return cudaSuccess;
}

template <int ACT, bool Z8, int LANES>
cudaError_t launch_strips(const uint16_t* dy, const uint16_t* z, const int8_t* codes, const uint8_t* scales,
                          int64_t rows, int64_t cols, int blocks, uint16_t* dz, float* db, cudaStream_t st) {
  constexpr int STRIP = 8 * LANES;
  const int64_t per = (rows + blocks - 1) / blocks;
  // strips in launches of at most 65535 (the grid's y limit)
  for (int64_t s0 = 0, strips = (cols + STRIP - 1) / STRIP; s0 < strips; s0 += 65535) {
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(std::min<int64_t>(strips - s0, 65535)), 1);
    const cudaError_t e = launch_overlapped(act_backward_kernel<ACT, Z8, LANES>, grid, dim3(kThreads), 0,
                                            static_cast<unsigned>(blocks), st, dy, z, codes, scales, rows, cols, per, s0,
                                            dz, db);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int ACT, bool Z8>
cudaError_t launch_act(const uint16_t* dy, const uint16_t* z, const int8_t* codes, const uint8_t* scales, int64_t rows,
                       int64_t cols, uint16_t* dz, float* db, cudaStream_t st) {
  Strips s;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int slots = num_sms() * kActBlocks;
  if ((e = consider_strips<ACT, Z8, 32>(dev, slots, rows, cols, &s)) != cudaSuccess) return e;
  if ((e = consider_strips<ACT, Z8, 16>(dev, slots, rows, cols, &s)) != cudaSuccess) return e;
  if ((e = consider_strips<ACT, Z8, 8>(dev, slots, rows, cols, &s)) != cudaSuccess) return e;
  if ((e = consider_strips<ACT, Z8, 4>(dev, slots, rows, cols, &s)) != cudaSuccess) return e;
  switch (s.lanes) {
    case 32: return launch_strips<ACT, Z8, 32>(dy, z, codes, scales, rows, cols, s.blocks, dz, db, st);
    case 16: return launch_strips<ACT, Z8, 16>(dy, z, codes, scales, rows, cols, s.blocks, dz, db, st);
    case 8: return launch_strips<ACT, Z8, 8>(dy, z, codes, scales, rows, cols, s.blocks, dz, db, st);
    default: return launch_strips<ACT, Z8, 4>(dy, z, codes, scales, rows, cols, s.blocks, dz, db, st);
  }
}

// Rows that the sweep takes at a time, and so partial sums a column; 0: the matrix is for the strips.
// Past 2^24 elements and from 1024 columns on the sweep wins (from 8 bits 8192 x 14336: 107 us against
// 114, 8192 x 3584 32 against 34, 16384 x 1536 29.4 against 33.3, with GELU 34 against 50; level at 4096 x
// 4096 and 32768 x 1024; 1024 x 8192 12.3 against 10.7). Without an activation, where only dY is read, the strips are ahead
// (8192 x 14336 40 us against 45).
int sweep_lanes(int64_t rows, int64_t cols) {
  if (rows * cols <= (int64_t(1) << 24) || cols < 1024) return 0;
  return static_cast<int>(std::min<int64_t>(static_cast<int64_t>(num_sms()) * kSweepBlocks * kThreads / (cols / 8), rows));
}

template <int ACT, bool Z8>
cudaError_t launch_sweep(const uint16_t* dy, const uint16_t* z, const int8_t* codes, const uint8_t* scales, int64_t rows,
                         int64_t cols, int lanes, uint16_t* dz, float* db, float* partial, cudaStream_t st) {
  const int64_t threads = lanes * (cols / 8);
  const cudaError_t e = launch_overlapped(act_backward_sweep_kernel<ACT, Z8>,
                                          dim3(static_cast<unsigned>((threads + kThreads - 1) / kThreads)),
                                          dim3(kThreads), 0, 1, st, dy, z, codes, scales, rows, cols, lanes, dz, partial);
  if (e != cudaSuccess) return e;
  return launch_overlapped(sum_partials_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(kThreads), 0, 1, st,
                           partial, lanes, cols, db);
}

template <int ACT>
cudaError_t launch_act_backward(const uint16_t* dy, const uint16_t* z, const int8_t* codes, const uint8_t* scales,
                                int64_t rows, int64_t cols, uint16_t* dz, float* db, float* partial, cudaStream_t st) {
  if constexpr (ACT != FSDP_ACT_NONE) {
    const int lanes = db && partial ? sweep_lanes(rows, cols) : 0;
    if (lanes && codes) return launch_sweep<ACT, true>(dy, z, codes, scales, rows, cols, lanes, dz, db, partial, st);
    if (lanes) return launch_sweep<ACT, false>(dy, z, codes, scales, rows, cols, lanes, dz, db, partial, st);
  }
  if constexpr (ACT != FSDP_ACT_NONE) {
    if (!db) {
      const Walking w(rows, cols, codes != nullptr);
      const auto kernel = !codes ? act_backward_walk_kernel<ACT, false, true>
                          : w.flat ? act_backward_walk_kernel<ACT, true, true>
                                   : act_backward_walk_kernel<ACT, true, false>;
      return launch_overlapped(kernel, dim3(w.blocks), dim3(kThreads), 0, 1, st, dy, z, codes, scales, w.d, dz);
    }
  }
  if constexpr (ACT != FSDP_ACT_NONE)
    if (codes) return launch_act<ACT, true>(dy, z, codes, scales, rows, cols, dz, db, st);
  return launch_act<ACT, false>(dy, z, codes, scales, rows, cols, dz, db, st);
}

cudaError_t launch_pack(const uint16_t* x, int64_t rows, int64_t cols, int8_t* codes, uint8_t* scales, cudaStream_t st) {
  const Walking w(rows, cols, true);
  return launch_overlapped(w.flat ? ckpt8_pack_kernel<true> : ckpt8_pack_kernel<false>, dim3(w.blocks), dim3(kThreads),
                           0, 1, st, x, w.d, codes, scales);
}

template <int ACT>
cudaError_t launch_unpack(const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* out,
                          cudaStream_t st) {
  const Walking w(rows, cols, true);
  return launch_overlapped(w.flat ? ckpt8_unpack_kernel<ACT, true> : ckpt8_unpack_kernel<ACT, false>, dim3(w.blocks),
                           dim3(kThreads), 0, 1, st, codes, scales, w.d, out);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// rows and cols of a checkpoint call: cols % 8, and every count of elements and units in
// 62 bits
int check_shape(int64_t rows, int64_t cols, const char* who) {
  if (rows < 1 || cols < 1 || rows > (int64_t(1) << 40) || cols > (1 << 30) || rows > (int64_t(1) << 61) / cols)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: rows %lld and cols %lld must be >= 1 (below 2^40 and 2^30)", who,
                     (long long)rows, (long long)cols);
  if (cols % 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: cols %lld must be a multiple of 8 (16-byte rows)", who,
                     (long long)cols);
  return ZERO_OK;
}

}  // namespace

int check_kept_activation(const uint16_t* z, const int8_t* codes, const uint8_t* scales, int act, const char* who) {
  if (act < FSDP_ACT_NONE || act > FSDP_ACT_SILU)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: act %d is not one of FSDP_ACT_*", who, act);
  if (act == FSDP_ACT_NONE) return ZERO_OK;  // not read
  if ((codes != nullptr) != (scales != nullptr) || (z != nullptr) == (codes != nullptr))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: pass the kept activation as z, or as both z_codes and z_scales", who);
  if (!aligned16(z) || !aligned16(codes) || !aligned16(scales))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: z, z_codes and z_scales must be 16-byte aligned", who);
  return ZERO_OK;
}

}  // namespace zgb

using namespace zgb;

extern "C" int fsdp_checkpoint8_pack(const zero_bf16* x, int64_t rows, int64_t cols, int8_t* codes, uint8_t* scales,
                                     zero_stream_t stream) {
  const char* who = "fsdp_checkpoint8_pack";
  int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  if (!x || !codes || !scales) return set_error(ZERO_ERR_INVALID_ARG, "%s: NULL argument", who);
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: x, codes and scales must be 16-byte aligned", who);
  const cudaError_t e = launch_pack(x, rows, cols, codes, scales, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

extern "C" int fsdp_checkpoint8_unpack(const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int act,
                                       zero_bf16* out, zero_stream_t stream) {
  const char* who = "fsdp_checkpoint8_unpack";
  int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  if (act < FSDP_ACT_NONE || act > FSDP_ACT_SILU)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: act %d is not one of FSDP_ACT_*", who, act);
  if (!codes || !scales || !out) return set_error(ZERO_ERR_INVALID_ARG, "%s: NULL argument", who);
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: codes, scales and out must be 16-byte aligned", who);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (act) {
    case FSDP_ACT_RELU: e = launch_unpack<FSDP_ACT_RELU>(codes, scales, rows, cols, out, st); break;
    case FSDP_ACT_GELU: e = launch_unpack<FSDP_ACT_GELU>(codes, scales, rows, cols, out, st); break;
    case FSDP_ACT_GELU_TANH: e = launch_unpack<FSDP_ACT_GELU_TANH>(codes, scales, rows, cols, out, st); break;
    case FSDP_ACT_SILU: e = launch_unpack<FSDP_ACT_SILU>(codes, scales, rows, cols, out, st); break;
    default: e = launch_unpack<FSDP_ACT_NONE>(codes, scales, rows, cols, out, st); break;
  }
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

extern "C" int fsdp_act_backward_workspace(int64_t rows, int64_t cols, uint64_t* bytes) {
  const char* who = "fsdp_act_backward_workspace";
  if (!bytes) return set_error(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  const int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  *bytes = 4 * static_cast<uint64_t>(sweep_lanes(rows, cols)) * static_cast<uint64_t>(cols);
  return ZERO_OK;
}

extern "C" int fsdp_act_backward(const zero_bf16* dY, const zero_bf16* z, const int8_t* z_codes, const uint8_t* z_scales,
                                 int64_t rows, int64_t cols, int act, zero_bf16* dZ, float* db, void* workspace,
                                 uint64_t workspace_bytes, zero_stream_t stream) {
  const char* who = "fsdp_act_backward";
  int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  if (!dY) return set_error(ZERO_ERR_INVALID_ARG, "%s: dY is NULL", who);
  if (!dZ && !db) return set_error(ZERO_ERR_INVALID_ARG, "%s: dZ and db are both NULL", who);
  if ((rc = check_kept_activation(z, z_codes, z_scales, act, who))) return rc;
  if (!aligned16(dY) || !aligned16(dZ) || !aligned16(db) || !aligned16(workspace))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: dY, dZ, db and workspace must be 16-byte aligned", who);
  uint64_t need = 0;
  if (workspace && (rc = fsdp_act_backward_workspace(rows, cols, &need))) return rc;
  if (workspace && workspace_bytes < need)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                     (unsigned long long)workspace_bytes, (unsigned long long)need);
  float* partial = static_cast<float*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (act) {
    case FSDP_ACT_RELU: e = launch_act_backward<FSDP_ACT_RELU>(dY, z, z_codes, z_scales, rows, cols, dZ, db, partial, st); break;
    case FSDP_ACT_GELU: e = launch_act_backward<FSDP_ACT_GELU>(dY, z, z_codes, z_scales, rows, cols, dZ, db, partial, st); break;
    case FSDP_ACT_GELU_TANH:
      e = launch_act_backward<FSDP_ACT_GELU_TANH>(dY, z, z_codes, z_scales, rows, cols, dZ, db, partial, st);
      break;
    case FSDP_ACT_SILU: e = launch_act_backward<FSDP_ACT_SILU>(dY, z, z_codes, z_scales, rows, cols, dZ, db, partial, st); break;
    default: e = launch_act_backward<FSDP_ACT_NONE>(dY, nullptr, nullptr, nullptr, rows, cols, dZ, db, partial, st); break;
  }
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}
