// The linear unit with its epilogue on the 5th-generation tensor cores: forward (bias,
// activation, residual, the kept pre-activation), input gradient (activation's derivative,
// residual gradient) and weight gradient (from bf16 or 8-bit activations).
//
//   forward  Y [m, r]  = epilogue(X [m, k] W^T)       contraction over k,  both K-major
//   dx       dX [m, k] = epilogue(dZ [m, r] W)        contraction over r,  W read MN-major
//   dw       dW [r, k] = scale dZ^T X                 contraction over m,  both MN-major
//
// Every operand is read where it lies: W from its row shards, transposed operands as
// MN-major tiles. Two kernels:
//   linear_wide_kernel    256 x 256 output tiles on CTA pairs (tcgen05.mma.cta_group::2),
//                         persistent, the epilogue of one tile beside the main loop of the next;
//   linear_narrow_kernel  128 output columns x TN output rows per tile, the contraction split
//                         over the CTAs of a cluster, whose parts meet in distributed shared
//                         memory and are added in a fixed order. For outputs of too few 256 x
//                         256 tiles to fill the GPU.
// All sums are fp32 in tensor memory; every output is rounded once. Every mbarrier wait is
// bounded: after one gives up the CTA's roles leave their loops, copies and MMAs in flight
// are waited for, and zero_device_status reports it.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "linear_math.cuh"
#include "tcgen05.cuh"

namespace zgb {

ZGB_DECLARE_ERROR_WORD();

namespace {

enum { OP_FWD, OP_DX, OP_DW };

constexpr int BK = 64;                        // contraction elements of one stage (128 bytes of bf16)
constexpr uint32_t kHalf = 128 * BK * 2;      // 128 rows (or MN-major columns) of one operand: 16 KiB
constexpr uint32_t kChunk = 64 * BK * 2;      // 64 columns of an MN-major operand: 8 KiB

constexpr unsigned int kErrEmpty = (5u << 8) | 1u;  // producer waiting for a free stage
constexpr unsigned int kErrFull = (5u << 8) | 2u;   // MMA waiting for a filled stage
constexpr unsigned int kErrAccE = (5u << 8) | 3u;   // MMA waiting for a drained accumulator
constexpr unsigned int kErrAccF = (5u << 8) | 4u;   // epilogue waiting for a finished accumulator
constexpr unsigned int kErrDrain = (5u << 8) | 5u;  // waiting for copies or MMAs in flight

struct LinearParams {
  // fwd, dx: the row shards of W, boxes of 64 columns x w_box rows; where they are cut to fit (w_levels > 1),
  // again with boxes of 4 w_box, 16 w_box rows
  CUtensorMap w[kGemmMaxPieces];
  CUtensorMap a;                  // fwd: X, dx: dZ (K-major, box 64 x 128 or TN rows); dw: dZ (MN-major, box 64 x 64)
  CUtensorMap b;                  // dw: X (MN-major, box 64 x 64)
  CUtensorMap out;                // wide kernel, fp32 dW: the output, boxes of 32 columns x 32 rows
  int m, n, k;                    // the product: out [m, n], contraction over k
  int n_shards, shard_rows;       // fwd, dx
  int w_levels;
  int w_box, w_box_log;           // rows of W per copy: the largest power of two <= 128 (fwd) or 64 (dx) that divides shard_rows
  const uint16_t *bias, *res;     // fwd: bias; fwd, dx: residual
  int act;
  const uint16_t* z_in;           // dx: the kept pre-activation
  const int8_t* zc_in;
  const uint8_t* zs_in;
  uint16_t* y;                    // bf16 output
  float* y32;                     // dw: fp32 output
  uint16_t* z;                    // fwd: pre-activation kept in bf16
  int8_t* zc;                     // fwd: ... in 8 bits
  uint8_t* zs;
  float scale;                    // dw
  int chunks, chunk_blocks;       // dw, fp32: the contraction in chunks of chunk_blocks K blocks (1 chunk otherwise)
};

// ------------------------------------------------------------------------------------
// waits: bounded as everywhere in the library. The barrier queries suspend the thread for up to 20
// us: queries that return at once keep their threads issuing, which at the power limit costs clock
// rate (forward, dx and dw at 8192 tokens, 14336 x 4096: 591, 605 and 555 us, suspended 555, 584 and
// 540). The global timer is read after 64 queries, not at each miss: a read takes long enough that
// the MMA thread then runs 10 % behind.
// ------------------------------------------------------------------------------------
template <bool CLUSTER>  // CLUSTER: arrivals come from the other CTA of the pair too
__device__ __forceinline__ bool try_wait_suspended(uint32_t bar, uint32_t parity) {
  uint32_t done;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
  return done != 0;
}
// false: gave up after kWaitTimeoutNs (recorded in the error word) or because another thread of the
// CTA did
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort, unsigned int code) {
  unsigned long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (try_wait_suspended<CLUSTER>(bar, parity)) return true;
    if (*abort) return false;
    if ((it & 63u) != 0) continue;
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitTimeoutNs) {
      atomicCAS(&g_zgb_dev_error, 0u, code);
      *abort = 1;
      return false;
    }
  }
}
// one lane of a warp waits, the whole warp gets the result
__device__ __forceinline__ bool warp_wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort, unsigned int code) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_bounded(bar, parity, abort, code) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// ------------------------------------------------------------------------------------
// operand copies: what one lane of the producer warp loads for each stage
// ------------------------------------------------------------------------------------
struct Copy {
  const CUtensorMap* map;
  uint32_t dst;   // byte offset in the stage
  int x, y;       // coordinates of the first K block
  bool k_major;   // x advances with K, y otherwise
  bool w_rows;    // y walks W's rows through the shards (dx)
  int shard;
  // W cut to fit: shard and row are where the K block's rows (dx) or the tile's columns (fwd) start
  int row, piece;
  uint32_t base;
};
// W cut to fit: copy number c.piece of ROWS rows from row c.row of shard c.shard, each as high as the
// shard allows of w_box, 4 w_box, .., ROWS; false if there are fewer. Rows past the last one count to
// the last shard, past its end (they read zeros).
template <int ROWS>
__device__ __forceinline__ bool w_piece(const LinearParams& p, Copy& c) {
  int shard = c.shard, y = c.row, at = 0, level = p.w_levels - 1;
  const auto box = [&](int l) { return min(p.w_box << (2 * l), ROWS); };
  if (shard + 1 == p.n_shards || p.shard_rows - y >= ROWS) {
    at = c.piece * box(level), y += at;
  } else {
    for (int i = c.piece; at < ROWS; --i) {
      const bool last = shard + 1 == p.n_shards;
      const int left = last ? ROWS - at : min(ROWS - at, p.shard_rows - y);
      for (level = p.w_levels - 1; level > 0 && box(level) > left;) --level;
      if (i == 0) break;
      at += box(level), y += box(level);
      if (!last && y >= p.shard_rows) y = 0, ++shard;
    }
  }
  if (at >= ROWS) return false;
  c.map = &p.w[level * p.n_shards + shard];
  c.y = y, c.dst = c.base + static_cast<uint32_t>(at) * 128u;
  return true;
}
// to the next K block; false: this lane has nothing to copy for it
template <bool CUT>
__device__ __forceinline__ bool copy_advance(const LinearParams& p, Copy& c) {
  if (c.k_major) {
    c.x += BK;
  } else if (CUT && c.w_rows) {
    c.row += BK;
    while (c.row >= p.shard_rows && c.shard + 1 < p.n_shards) c.row -= p.shard_rows, ++c.shard;
    return w_piece<BK>(p, c);
  } else {
    c.y += BK;
    if (c.w_rows)
      while (c.y >= p.shard_rows && c.shard + 1 < p.n_shards) c.y -= p.shard_rows, ++c.shard, ++c.map;
  }
  return true;
}
// the shard that holds row `row` of W; rows past the last one stay in the last shard, past
// its end (they read zeros)
__device__ __forceinline__ void copy_seek(const LinearParams& p, Copy& c, int row) {
  c.shard = min(row / p.shard_rows, p.n_shards - 1);
  c.map = &p.w[c.shard];
  c.y = row - c.shard * p.shard_rows;
}
// copies of W (fwd): 128 output columns from n0, K-major, 128 / w_box copies of w_box rows, or (CUT) up to
// as many lanes with `has` true
template <bool CUT>
__device__ __forceinline__ int w_copies_k_major(const LinearParams& p, int i, int n0, int kb0, uint32_t dst, Copy& c,
                                                bool& has) {
  const int count = 128 >> p.w_box_log;
  if (i >= 0 && i < count) {
    c.k_major = true, c.w_rows = false;
    c.x = kb0 * BK;
    if constexpr (CUT) {
      copy_seek(p, c, n0);
      c.row = c.y, c.piece = i, c.base = dst;
      has = w_piece<128>(p, c);
    } else {
      copy_seek(p, c, n0 + i * p.w_box);
      c.dst = dst + static_cast<uint32_t>(i * p.w_box) * 128u;
      has = true;
    }
  }
  return count;
}
// copies of W (dx): 128 output columns from n0, MN-major: two chunks of 64 columns, the 64 rows
// of a K block in 64 / w_box copies each, or (CUT) up to as many
template <bool CUT>
__device__ __forceinline__ int w_copies_mn_major(const LinearParams& p, int i, int n0, int kb0, uint32_t dst, Copy& c,
                                                 bool& has) {
  const int per = 64 >> p.w_box_log, count = 2 * per;
  if (i >= 0 && i < count) {
    const int chunk = i / per, sub = i - chunk * per;
    c.k_major = false, c.w_rows = true;
    c.x = n0 + 64 * chunk;
    dst += static_cast<uint32_t>(chunk) * kChunk;
    if constexpr (CUT) {
      copy_seek(p, c, kb0 * BK);
      c.row = c.y, c.piece = sub, c.base = dst;
      has = w_piece<BK>(p, c);
    } else {
      copy_seek(p, c, kb0 * BK + sub * p.w_box);
      c.dst = dst + static_cast<uint32_t>(sub * p.w_box) * 128u;
      has = true;
    }
  }
  return count;
}
// an MN-major operand in one piece: `chunks` chunks of 64 columns from c0
__device__ __forceinline__ int mn_copies(const CUtensorMap* map, int chunks, int i, int c0, int kb0, uint32_t dst, Copy& c,
                                         bool& has) {
  if (i >= 0 && i < chunks) {
    c.map = map, c.k_major = false, c.w_rows = false, c.shard = 0;
    c.x = c0 + 64 * i, c.y = kb0 * BK;
    c.dst = dst + static_cast<uint32_t>(i) * kChunk;
    has = true;
  }
  return chunks;
}
// a K-major operand in one piece: one box of rows from r0
__device__ __forceinline__ int k_copies(const CUtensorMap* map, int i, int r0, int kb0, uint32_t dst, Copy& c, bool& has) {
  if (i == 0)
    c.map = map, c.k_major = true, c.w_rows = false, c.shard = 0, c.x = kb0 * BK, c.y = r0, c.dst = dst, has = true;
  return 1;
}

// ------------------------------------------------------------------------------------
// epilogues
// ------------------------------------------------------------------------------------
__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void unpack8(const uint4& w, f2* x) {
  x[0] = f2_from_bf16x2(w.x), x[1] = f2_from_bf16x2(w.y), x[2] = f2_from_bf16x2(w.z), x[3] = f2_from_bf16x2(w.w);
}

// A 4 KiB staging buffer holds 32 rows x 64 bf16 columns, the 16-byte piece j of row i at slot j ^
// (i % 8): a thread's own row and the warp's rows in order are both free of bank conflicts.
// The epilogue moves it to and from global memory with ordinary accesses, eight lanes to a row of
// 128 bytes: bulk copies would need a proxy fence by every thread, which waits for the warp's
// stores in flight (about 1000 cycles, twice a tile).
__device__ __forceinline__ uint32_t staged_at(int i, int j) { return static_cast<uint32_t>(i * 128 + ((j ^ (i & 7)) * 16)); }
// rows r0 .., columns c0 .. c0 + 63 of src [m, n] to the buffer, asynchronously; zeros outside
__device__ __forceinline__ void stage_load(uint32_t buf, const uint16_t* src, int r0, int c0, int m, int n, int lane) {
  const int j = lane & 7, col = c0 + 8 * j;
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int i = it * 4 + (lane >> 3);
    const bool in = r0 + i < m && col < n;
    const uint16_t* at = in ? src + static_cast<size_t>(r0 + i) * n + col : src;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(buf + staged_at(i, j)), "l"(at), "r"(in ? 16u : 0u)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// the buffer to rows r0 .., columns c0 .. of dst [m, n]
__device__ __forceinline__ void stage_store(const uint8_t* buf, uint16_t* dst, int r0, int c0, int m, int n, int lane) {
  const int j = lane & 7, col = c0 + 8 * j, i0 = lane >> 3;  // rows i0, i0 + 4, ..: two alternating slots
  const int left = col < n ? m - r0 - i0 : 0;
  uint16_t* to = dst + static_cast<size_t>(r0 + i0) * n + col;
  const size_t step = static_cast<size_t>(4) * n;
  const uint8_t *even = buf + staged_at(i0, j), *odd = buf + staged_at(i0 + 4, j);
#pragma unroll
  for (int it = 0; it < 8; ++it, to += step) {
    const uint4 w = *reinterpret_cast<const uint4*>(((it & 1) ? odd : even) + (it >> 1) * 1024);
    if (4 * it < left) __stcs(reinterpret_cast<uint4*>(to), w);
  }
}

// half h of the buffer, 32 columns, from each thread's row, and on to global memory: 64 bytes a row,
// four lanes to one (the two rows of every eight lanes are four apart: no bank conflicts)
__device__ __forceinline__ void stage_store_half(uint8_t* buf, const uint4 (&w)[4], int h, uint16_t* dst, int r0, int c0,
                                                 int m, int n, int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(buf + staged_at(lane, 4 * h + j)) = w[j];
  __syncwarp();
  const int j = 4 * h + (lane & 3), col = c0 + 8 * j, i0 = ((lane >> 2) & 1) * 4 + (lane >> 3);
  const int left = col < n ? m - r0 - i0 : 0;
  uint16_t* to = dst + static_cast<size_t>(r0 + i0) * n + col;
#pragma unroll
  for (int it = 0; it < 4; ++it, to += static_cast<size_t>(8) * n) {
    const uint4 v = *reinterpret_cast<const uint4*>(buf + staged_at(i0, j) + it * 1024);
    if (8 * it < left) __stcs(reinterpret_cast<uint4*>(to), v);
  }
  __syncwarp();
}

// 32 codes of a row, in accesses of 16 bytes where rows allow, else 8
__device__ __forceinline__ void load_codes32(const LinearParams& p, size_t at, int col0, uint32_t (&c)[8]) {
  if (col0 + 32 <= p.n && (p.n & 15) == 0) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.zc_in + at) + q);
      c[4 * q] = w.x, c[4 * q + 1] = w.y, c[4 * q + 2] = w.z, c[4 * q + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint2 w = make_uint2(0u, 0u);
      if (col0 + 8 * q < p.n) w = __ldg(reinterpret_cast<const uint2*>(p.zc_in + at + 8 * q));
      c[2 * q] = w.x, c[2 * q + 1] = w.y;
    }
  }
}

// wide kernel: 32 columns col0 .. of output row `row`, one thread, v their fp32 sums in pairs: the
// output's values in place. 32 columns are one group of the 8-bit checkpoint: the forward stores
// its codes and returns its scale byte in `byte`; for dx from 8 bits `byte` is the kept
// activation's. side: the 32 columns' bf16 words of the tensor read beside the sums (forward: the
// residual; dx: the kept activation in bf16, or else the residual). bias: the columns' biases in
// shared memory. buf, h: the staging buffer's half through which a bf16 pre-activation leaves.
// Sums past column n are zero. Called by whole warps, thread `lane` with row r0 + lane.
template <int OP>
__device__ __forceinline__ void epilogue32(const LinearParams& p, int row, int col0, int r0, const uint4* bias,
                                           const uint4 (&side)[4], uint8_t* buf, int h, int lane, uint32_t& byte,
                                           f2 (&v)[16]) {
  static_assert(OP != OP_DW, "a weight gradient is only scaled, by its caller");
  const size_t at = static_cast<size_t>(row) * p.n + col0;
  const bool live = row < p.m;
  bool side_is_res = p.res != nullptr;
  // dx: a residual beside a bf16 kept activation, which has the staging buffers: on its way while the
  // activation's derivative is computed
  const bool own_res = OP == OP_DX && p.res && p.z_in;
  uint4 res[4];
  if (own_res) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      res[q] = make_uint4(0u, 0u, 0u, 0u);
      if (live && col0 + 8 * q < p.n) res[q] = ldg16(p.res + at + 8 * q);
    }
  }
  if constexpr (OP == OP_FWD) {
    if (p.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f2 b[4];
        unpack8(bias[q], b);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * q + j] = f2_add(v[4 * q + j], b[j]);
      }
    }
    if (p.z) {
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = make_uint4(f2_to_bf16x2(v[4 * q]), f2_to_bf16x2(v[4 * q + 1]), f2_to_bf16x2(v[4 * q + 2]),
                          f2_to_bf16x2(v[4 * q + 3]));
      stage_store_half(buf, w, h, p.z, r0, col0 - 32 * h, p.m, p.n, lane);
    }
    if (p.zc) {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = amax2(amax, v[j]);
      byte = ckpt_byte(amax);
      const float inv = ckpt_inv_scale(byte);
      uint32_t w[8];
      if (byte < 248u) {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = ckpt_code4(v[2 * q], v[2 * q + 1], inv);
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          w[q] = ckpt_code4(ckpt_clamped(v[2 * q], byte), ckpt_clamped(v[2 * q + 1], byte), inv);
      }
      if (live) {
        if (col0 + 32 <= p.n && (p.n & 15) == 0) {
          __stcs(reinterpret_cast<uint4*>(p.zc + at), make_uint4(w[0], w[1], w[2], w[3]));
          __stcs(reinterpret_cast<uint4*>(p.zc + at) + 1, make_uint4(w[4], w[5], w[6], w[7]));
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (col0 + 8 * q < p.n) *reinterpret_cast<uint2*>(p.zc + at + 8 * q) = make_uint2(w[2 * q], w[2 * q + 1]);
        }
      }
    }
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = act_fwd<decltype(act)::value>(v[j]);
    });
  } else {
    if (p.act != FSDP_ACT_NONE) {
      f2 z[16];
      if (p.zc_in) {
        uint32_t c[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        if (live) load_codes32(p, at, col0, c);
        const float s = ckpt_scale(byte);
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = ckpt_values2(c[j >> 1], j & 1, s);
      } else {
        side_is_res = false;
#pragma unroll
        for (int q = 0; q < 4; ++q) unpack8(side[q], z + 4 * q);
      }
      with_act(p.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = f2_mul(v[j], act_grad<decltype(act)::value>(z[j]));
      });
    }
  }
  if (side_is_res || own_res) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f2 r[4];
      unpack8(own_res ? res[q] : side[q], r);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * q + j] = f2_add(v[4 * q + j], r[j]);
    }
  }
}

// narrow kernel: what 4 columns of a row read beside their sums, loaded while the main loop runs.
// Volatile: the compiler would move the loads down to their use.
template <int OP>
struct Side4 {
  uint2 res, z;   // z: bf16, or codes in z.x
  uint32_t byte;  // the group's scale byte
  __device__ __forceinline__ void load(const LinearParams& p, int row, int col) {
    if (OP == OP_DW || row >= p.m || col >= p.n) return;
    const size_t at = static_cast<size_t>(row) * p.n + col;
    if (p.res) load8(p.res + at, res);
    if (OP == OP_DX && p.zc_in) {
      asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(z.x) : "l"(p.zc_in + at));
      asm volatile("ld.global.nc.u8 %0, [%1];"
                   : "=r"(byte)
                   : "l"(p.zs_in + static_cast<size_t>(row) * ((p.n + 31) / 32) + (col >> 5)));
    } else if (OP == OP_DX && p.z_in) {
      load8(p.z_in + at, z);
    }
  }
  static __device__ __forceinline__ void load8(const uint16_t* src, uint2& w) {
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(src));
  }
};

// 4 columns of one output row per lane, 32 lanes across 128 columns; the 8 lanes of a group of 32
// columns share its scale byte through shuffles. bias: the columns' biases (fwd, where there are
// any). Called by whole warps.
template <int OP, int ACT>
__device__ __forceinline__ void epilogue4(const LinearParams& p, int row, int col, uint2 bias, const Side4<OP>& side,
                                          f2 (&v)[2]) {
  const size_t at = static_cast<size_t>(row) * p.n + col;
  const bool live = row < p.m && col < p.n;
  if constexpr (OP == OP_DW) {
    v[0] = f2_mul(v[0], f2_both(p.scale)), v[1] = f2_mul(v[1], f2_both(p.scale));
    if (!live) return;
    if (p.y32) __stcs(reinterpret_cast<ulonglong2*>(p.y32 + at), make_ulonglong2(v[0], v[1]));
    else *reinterpret_cast<uint2*>(p.y + at) = make_uint2(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]));
    return;
  }
  if constexpr (OP == OP_FWD) {
    if (p.bias) v[0] = f2_add(v[0], f2_from_bf16x2(bias.x)), v[1] = f2_add(v[1], f2_from_bf16x2(bias.y));
    if (p.z && live)
      *reinterpret_cast<uint2*>(p.z + at) = make_uint2(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]));
    if (p.zc) {
      float amax = amax2(amax2(0.0f, v[0]), v[1]);
#pragma unroll
      for (int d = 1; d < 8; d *= 2) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
      const uint32_t byte = ckpt_byte(amax);
      const float inv = ckpt_inv_scale(byte);
      const uint32_t w = byte < 248u ? ckpt_code4(v[0], v[1], inv)
                                     : ckpt_code4(ckpt_clamped(v[0], byte), ckpt_clamped(v[1], byte), inv);
      if (live) {
        *reinterpret_cast<uint32_t*>(p.zc + at) = w;
        if ((col & 31) == 0)
          p.zs[static_cast<size_t>(row) * ((p.n + 31) / 32) + (col >> 5)] = static_cast<uint8_t>(byte);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = act_fwd<ACT>(v[j]);
  } else if (ACT != FSDP_ACT_NONE && live) {
    f2 z[2];
    if (p.zc_in) {
      const float s = ckpt_scale(side.byte);
      z[0] = ckpt_values2(side.z.x, 0, s), z[1] = ckpt_values2(side.z.x, 1, s);
    } else {
      z[0] = f2_from_bf16x2(side.z.x), z[1] = f2_from_bf16x2(side.z.y);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = f2_mul(v[j], act_grad<ACT>(z[j]));
  }
  if (!live) return;
  if (p.res) v[0] = f2_add(v[0], f2_from_bf16x2(side.res.x)), v[1] = f2_add(v[1], f2_from_bf16x2(side.res.y));
  *reinterpret_cast<uint2*>(p.y + at) = make_uint2(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]));
}

// ------------------------------------------------------------------------------------
// wide kernel
// ------------------------------------------------------------------------------------
// A cluster of two CTAs on two SMs per 256 x 256 output tile: each CTA loads 128 rows of the
// first operand and 128 columns of the second, and the even CTA's MMA (M = N = 256) reads both
// CTAs' shared memory. Persistent, two accumulators in tensor memory.
//   warp 0       producer: lane i issues the i-th copy of a stage (TMA), both CTAs
//   warp 1       MMA issuer (even CTA), tensor-memory allocation
//   then 8 (dw: 4) epilogue warps, two (one) per tensor-memory lane quarter, sharing its columns
// What bounds it: at 8192 tokens, 14336 x 4096, tensor work at the power limit (forward with bias,
// SiLU and 8-bit Z 512-656 us by the board's temperature, 1.47-1.88 PFLOP/s; alone and cool 505-516 us,
// tensor pipe 86-88 % active; dx with the derivative from 8 bits 507; dW 490 us, 93-97 %, to fp32 515). The pair tile
// is the least that an SM's reads from L2 can feed: 32 KB per 64 contraction elements, about 51
// bytes a clock at the measured tensor rate, near the most an SM reads. At 768 contraction elements
// a tile's products take 4 us and its epilogue up to 6 (GELU with 8-bit Z; the eight warps issue in
// 36 % of the cycles, stalled mostly on fixed latencies), so the epilogue bounds it: 8192 x 2304
// from 768 24.0 us bare, 30.1 with both. Sixteen epilogue warps have 112 registers and spill: 36.1.
// Loading the next 32 sums ahead of their use needs 64 registers more than there are: 38.5.
// COPIES_ONE: every operand of a stage is one copy (W's shards of whole 128-row, dx: 64-row blocks,
// MN-major widths of whole 64-column chunks), issued by one lane. COPIES_EQUAL: lane i of the
// producer warp issues the i-th of a few; COPIES_CUT: W's shards end at multiples of 8 or 16 rows only, and
// its copies are cut to fit (4096 x 3480 from 4096, five shards: 87 us, in equal copies of 8 rows 139; dx
// 130 and 186; one shard 63 and 73). Where equal copies have 32 rows or more they are faster, above all
// for dx, whose cuts change from K block to K block (4096 x 768 from 2304, eight shards: 20, cut 27).
template <int OP> struct Wide {
  static constexpr int EPI_WARPS = OP == OP_DW ? 4 : 8;     // dw's epilogue is a scale and a store
  static constexpr int EPI_COLS = 1024 / EPI_WARPS;         // output columns of one epilogue warp
  static constexpr int STAGES = OP == OP_DW ? 6 : 5;
  static constexpr int THREADS = 32 * (2 + EPI_WARPS);
  static constexpr uint32_t STAGE = 2 * kHalf;
  static constexpr uint32_t EPI = EPI_WARPS * 2u * 4096u;   // two 4 KiB staging buffers per warp
  static constexpr uint32_t BIAS = OP == OP_FWD ? 2u * 256u * 2u : 0u;  // a tile's biases, twice
  static constexpr uint32_t SMEM = STAGES * STAGE + EPI + BIAS + 1024;
};

// tile order: bands of 12 row blocks, down the rows of one tile column, then the next: the
// tiles in flight share few operand tiles, which stay in L2
__device__ __forceinline__ void wide_tile_coords(int tile, int num_m, int num_n, int& mb, int& nb) {
  constexpr int kBand = 12;
  const int rows_in_band = kBand < num_m ? kBand : num_m;
  const int band = tile / (rows_in_band * num_n), in_band = tile - band * rows_in_band * num_n;
  const int rows = min(rows_in_band, num_m - band * rows_in_band);
  mb = band * rows_in_band + in_band % rows;
  nb = in_band / rows;
}

// a box of global memory to L2
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(tmap), "r"(x), "r"(y) : "memory");
}

// fp32 add of a shared-memory box to global memory, in L2
__device__ __forceinline__ void tma_reduce_add_2d(const void* tmap, int32_t x, int32_t y, uint32_t src_smem) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tmap),
               "r"(x), "r"(y), "r"(src_smem)
               : "memory");
}

// A barrier of 128 threads (whole warps): whether any of them says `mine`. Warps of a role meet only at
// barriers that tell all of them when one gave up a wait, so that they leave together: one whose query of
// the same barrier succeeded a moment later would else wait here for a warp that has left.
__device__ __forceinline__ bool any_of_128(int id, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(mine ? 1u : 0u)
      : "memory");
  return any != 0;
}

// The epilogue warps' role. A thread has a row of the tile; a warp's 64-column chunk of bf16 output
// goes through one of its staging buffers. A bf16 tensor that the epilogue reads beside the sums
// (residual, kept activation) is loaded into the buffers before the sums are ready, and each thread
// replaces its row by the output.
template <int OP>
__device__ __forceinline__ void wide_epilogue(const LinearParams& p, uint8_t* smem, uint32_t tmem_base, uint32_t accf_bar,
                                              uint32_t acce_bar, volatile int* abort, int warp, int lane, uint32_t rank,
                                              int pair, int pairs, int num_m, int num_n) {
  using C = Wide<OP>;
  const int q = warp & 3;            // the tensor-memory lane quarter this warp may read
  const int part = (warp - 2) >> 2;  // which of the quarter's warps
  uint8_t* stage = smem + C::STAGES * C::STAGE + static_cast<uint32_t>(warp - 2) * 8192u;
  uint8_t* bias_sm = smem + C::STAGES * C::STAGE + C::EPI;
  const int groups = (p.n + 31) / 32;
  const uint16_t* side_src = nullptr;
  if constexpr (OP != OP_DW) side_src = OP == OP_DX && p.z_in ? p.z_in : p.res;
  uint32_t i = 0, bias_turn = 0;
  // fp32 dW: bulk stores this warp has made. The two buffers alternate over all of them, across tiles: a
  // buffer is written again once all stores but the newest, which reads the other one, have read theirs.
  // Counted by a tile's own columns, two stores in a row would leave from buffer 0 where a tile at the
  // right edge has an odd number of 32-column blocks.
  uint32_t stores = 0;
  const bool shared_bias = OP == OP_FWD && p.bias;
  bool stop = false;  // this warp gave up a wait
  for (int tile = pair; tile < num_m * num_n && (shared_bias || !stop); tile += pairs, bias_turn ^= 1u) {
    int mb, nb;
    wide_tile_coords(tile, num_m, num_n, mb, nb);
    const int r0 = mb * 256 + static_cast<int>(rank) * 128 + q * 32, row = r0 + lane;
    const int c0 = nb * 256 + part * C::EPI_COLS;
    uint32_t bytes = 0;  // the row's scale bytes of four groups
    const uint4* bias = nullptr;
    if constexpr (OP == OP_FWD) {
      if (shared_bias) {
        // one warp of the four that share these 128 columns copies them; the other half of the
        // area is the last tile's, so one barrier is enough. Every warp comes to it at every tile until
        // all leave, one that has given up without the rest of its tile
        uint8_t* at = bias_sm + bias_turn * 512u + part * 256u;
        if (q == 0 && lane < 16) {
          const int col = c0 + 8 * lane;
          reinterpret_cast<uint4*>(at)[lane] = col < p.n ? ldg16(p.bias + col) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (any_of_128(1 + part, stop)) break;
        bias = reinterpret_cast<const uint4*>(at);
      }
    }
    if constexpr (OP != OP_DW) {
      if (side_src)
        for (int b = 0; b < 2; ++b) stage_load(smem_u32(stage) + 4096u * b, side_src, r0, c0 + 64 * b, p.m, p.n, lane);
      if (OP == OP_DX && p.zc_in && row < p.m) {
        const uint8_t* zs = p.zs_in + static_cast<size_t>(row) * groups + (c0 >> 5);
        if ((groups & 3) == 0) {
          if (c0 < p.n) bytes = __ldg(reinterpret_cast<const uint32_t*>(zs));
        } else {
          for (int g = 0; g < 4; ++g)
            if (c0 + 32 * g < p.n) bytes |= static_cast<uint32_t>(__ldg(zs + g)) << (8 * g);
        }
      }
    }
    for (int chunk = 0; chunk < p.chunks; ++chunk, ++i) {
      const uint32_t a = i & 1u, u = i >> 1;
      if (!warp_wait_bounded(accf_bar + 8u * a, u & 1u, abort, kErrAccF)) {
        stop = true;
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * 256 + part * C::EPI_COLS;
      if (OP == OP_DW && p.y32) {
        if (chunk > 0 && lane == 0) bulk_wait_group_all();  // this tile's earlier sums are in memory
  #pragma unroll 1
        for (int c = 0; c < C::EPI_COLS; c += 32) {
          uint32_t r[32];
          tmem_ld_32cols(taddr + c, r);
          if (c0 + c >= p.n) continue;
          const f2 s = f2_both(p.scale);
          uint8_t* buf = stage + (stores++ & 1u) * 4096u;
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
  #pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<ulonglong2*>(buf + staged_at(lane, j)) =
                make_ulonglong2(f2_mul(f2_make(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1])), s),
                                f2_mul(f2_make(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])), s));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (chunk == 0) tma_store_2d(&p.out, c0 + c, r0, smem_u32(buf));
            else tma_reduce_add_2d(&p.out, c0 + c, r0, smem_u32(buf));
            bulk_commit_group();
          }
        }
      } else {
        // 32 columns at a time, rolled: unrolled by two the code is twice as long for the instruction
        // cache that the producer and MMA loops share (8192 x 2304 from 768: 32.2 us, rolled 30.0). The
        // activation is a switch in it for the same reason: the role once per activation cost 4096 x
        // 2304 from 4096 6 %.
#pragma unroll 1
        for (int c = 0; c < C::EPI_COLS; c += 32) {
          const int h = (c >> 5) & 1, col0 = c0 + c;
          uint8_t* buf = stage + ((c >> 6) & 1) * 4096;
          if (h == 0) {
            if (OP != OP_DW && side_src) {
              if (c == 0) asm volatile("cp.async.wait_group 1;" ::: "memory");
              else asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncwarp();  // the buffer is loaded, or its last store has read it
          }
          uint32_t r[32];
          tmem_ld_32cols(taddr + c, r);
          if (col0 >= p.n) continue;  // warp-uniform
          f2 v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = f2_make(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
          uint4 w[4];
          if constexpr (OP == OP_DW) {
            const f2 s = f2_both(p.scale);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = f2_mul(v[j], s);
          } else {
            if (side_src) {
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint4*>(buf + staged_at(lane, 4 * h + j));
            }
            uint32_t byte = OP == OP_DX ? (bytes >> (c >> 2)) & 0xFFu : 0u;
            epilogue32<OP>(p, row, col0, r0, bias + (c >> 3), w, buf, h, lane, byte, v);
            if (OP == OP_FWD) bytes |= byte << (c >> 2);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(buf + staged_at(lane, 4 * h + j)) =
                make_uint4(f2_to_bf16x2(v[4 * j]), f2_to_bf16x2(v[4 * j + 1]), f2_to_bf16x2(v[4 * j + 2]),
                           f2_to_bf16x2(v[4 * j + 3]));
          if (h == 1 || col0 + 32 >= p.n) {
            __syncwarp();
            stage_store(buf, p.y, r0, col0 - 32 * h, p.m, p.n, lane);
          }
        }
        __syncwarp();  // before the next tile's loads into the buffers
        if (OP == OP_FWD && p.zc && row < p.m) {
          uint8_t* zs = p.zs + static_cast<size_t>(row) * groups + (c0 >> 5);
          if ((groups & 3) == 0) {
            if (c0 < p.n) *reinterpret_cast<uint32_t*>(zs) = bytes;
          } else {
            for (int g = 0; g < 4; ++g)
              if (c0 + 32 * g < p.n) zs[g] = static_cast<uint8_t>(bytes >> (8 * g));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      // relaxed: the arrival only says that the tensor-memory loads are done (ordered by the fence
      // above); a release at cluster scope would wait for every store the epilogue just made
      if (lane == 0)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         mapa_shared(acce_bar + 8u * a, 0))
                     : "memory");
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // no copy may still write this CTA's shared memory
  if (lane == 0) bulk_wait_group_all();             // and no store still read it
}

enum { COPIES_EQUAL, COPIES_ONE, COPIES_CUT };
template <int OP, int COPIES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide<OP>::THREADS, 1)
    linear_wide_kernel(const __grid_constant__ LinearParams p) {
  using C = Wide<OP>;
  constexpr bool A_MN = OP == OP_DW, B_MN = OP != OP_FWD;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t accf_bar[2];
  __shared__ __align__(8) uint64_t acce_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const int num_m = (p.m + 255) / 256, num_n = (p.n + 255) / 256, num_k = (p.k + BK - 1) / BK;
  // work items: a tile's chunks one after the other on the same pair
  const int tiles = num_m * num_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&accf_bar[a]), 1);
      mbar_init(smem_u32(&acce_bar[a]), 2 * C::EPI_WARPS);
    }
    mbar_init(smem_u32(&drain_bar), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_base_sh), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers initialised and tensor memory allocated before any copy
  tc_fence_after();
  allow_next_grid();
  wait_for_prior_grids();
  const uint32_t tmem_base = tmem_base_sh;

  if (warp == 0) {
    // ---------------- producer (both CTAs) ----------------
    uint32_t it = 0, s = 0, ph = 0;  // K blocks issued; their stage and its phase parity
    bool stop = false;
    if constexpr (COPIES == COPIES_ONE) {
      if (lane == 0) {
        for (int tile = pair; tile < tiles && !stop; tile += pairs) {
          int mb, nb;
          wide_tile_coords(tile, num_m, num_n, mb, nb);
          const int m0 = mb * 256 + static_cast<int>(rank) * 128, n0 = nb * 256 + static_cast<int>(rank) * 128;
          int shard = 0, row = 0;  // W: the shard and its row of this tile (fwd) or K block (dx)
          if constexpr (OP == OP_FWD) shard = min(n0 / p.shard_rows, p.n_shards - 1), row = n0 - shard * p.shard_rows;
          for (int kb = 0; kb < num_k; ++kb, ++it) {
            if (it >= static_cast<uint32_t>(C::STAGES) &&
                !wait_bounded(smem_u32(&empty_bar[s]), ph ^ 1u, abort, kErrEmpty)) {
              stop = true;
              break;
            }
            const uint32_t fb = mapa_shared(smem_u32(&full_bar[s]), 0);
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), 4 * kHalf);
            const uint32_t sa = smem_u32(smem) + s * C::STAGE;
            if constexpr (A_MN) tma_load_3d_pair(sa, &p.a, 0, kb * BK, m0 / 64, fb);
            else tma_load_2d_pair(sa, &p.a, kb * BK, m0, fb);
            if constexpr (OP == OP_FWD) {
              tma_load_2d_pair(sa + kHalf, &p.w[shard], kb * BK, row, fb);
            } else if constexpr (OP == OP_DX) {
              tma_load_3d_pair(sa + kHalf, &p.w[shard], 0, row, n0 / 64, fb);
              if ((row += BK) >= p.shard_rows && shard + 1 < p.n_shards) row = 0, ++shard;
            } else {
              tma_load_3d_pair(sa + kHalf, &p.b, 0, kb * BK, n0 / 64, fb);
            }
            if (++s == C::STAGES) s = 0, ph ^= 1u;
          }
        }
      }
    } else
    for (int tile = pair; tile < tiles && !stop; tile += pairs) {
      int mb, nb;
      wide_tile_coords(tile, num_m, num_n, mb, nb);
      const int m0 = mb * 256 + static_cast<int>(rank) * 128, n0 = nb * 256 + static_cast<int>(rank) * 128;
      Copy c;
      int i = lane;
      bool has = false;  // a copy of this K block
      constexpr bool CUT = COPIES == COPIES_CUT;
      if constexpr (A_MN) i -= mn_copies(&p.a, 2, i, m0, 0, 0, c, has);
      else i -= k_copies(&p.a, i, m0, 0, 0, c, has);
      if constexpr (OP == OP_FWD) i -= w_copies_k_major<CUT>(p, i, n0, 0, kHalf, c, has);
      else if constexpr (OP == OP_DX) i -= w_copies_mn_major<CUT>(p, i, n0, 0, kHalf, c, has);
      else i -= mn_copies(&p.b, 2, i, n0, 0, kHalf, c, has);
      const bool mine = CUT && OP == OP_DX ? i < 0 : has;
      for (int kb = 0; kb < num_k; ++kb, ++it) {
        bool ok = true;
        if (it >= static_cast<uint32_t>(C::STAGES))
          ok = wait_bounded(smem_u32(&empty_bar[s]), ph ^ 1u, abort, kErrEmpty);
        if (!__all_sync(0xffffffffu, ok)) {
          stop = true;
          break;
        }
        if (rank == 0 && lane == 0)
          mbar_arrive_expect_tx(smem_u32(&full_bar[s]), 4 * kHalf);
        if (mine) {
          if (!(CUT && OP == OP_DX) || has)
            tma_load_2d_pair(smem_u32(smem) + s * C::STAGE + c.dst, c.map, c.x, c.y,
                             mapa_shared(smem_u32(&full_bar[s]), 0));
          has = copy_advance<CUT>(p, c);
        }
        __syncwarp();
        if (++s == C::STAGES) s = 0, ph ^= 1u;
      }
    }
    // every stage this CTA filled is read by the even CTA's MMAs: wait until they released it
    if (lane == 0) {
      int never = 0;
      const uint32_t first = it > static_cast<uint32_t>(C::STAGES) ? it - C::STAGES : 0u;
      for (uint32_t j = first; j < it; ++j)
        wait_bounded(smem_u32(&empty_bar[j % C::STAGES]), (j / C::STAGES) & 1u, &never, kErrDrain);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (even CTA) ----------------
    if (rank == 0 && lane == 0) {
      // the next 16 contraction elements: +32 bytes K-major, +2048 bytes MN-major
      constexpr uint32_t a_step = A_MN ? 128u : 2u, b_step = B_MN ? 128u : 2u;
      constexpr uint32_t idesc = idesc_bf16_f32(256, 256, A_MN, B_MN);
      uint32_t i = 0, s = 0, ph = 0;
      bool stop = false, issued = false;
      for (int tile = pair; tile < tiles && !stop; tile += pairs) {
        for (int kb = 0; kb < num_k && !stop; ++i) {  // one accumulator per chunk
          const int kb_end = min(kb + p.chunk_blocks, num_k), kb_first = kb;
          const uint32_t a = i & 1u, u = i >> 1;
          if (u >= 1 && !wait_bounded<true>(smem_u32(&acce_bar[a]), (u - 1) & 1u, abort, kErrAccE)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + a * 256;
          for (; kb < kb_end; ++kb) {
            if (!wait_bounded(smem_u32(&full_bar[s]), ph, abort, kErrFull)) {
              stop = true;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem) + s * C::STAGE;
            const uint64_t ad = A_MN ? sw128_mnmajor_desc(sa, kChunk) : sw128_kmajor_desc(sa);
            const uint64_t bd = B_MN ? sw128_mnmajor_desc(sa + kHalf, kChunk) : sw128_kmajor_desc(sa + kHalf);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              umma_bf16_pair(d, ad + a_step * k, bd + b_step * k, idesc, (kb != kb_first || k != 0) ? 1u : 0u);
            umma_commit_pair(smem_u32(&empty_bar[s]), 0x3);
            issued = true;
            if (++s == C::STAGES) s = 0, ph ^= 1u;
          }
          if (!stop) umma_commit_pair(smem_u32(&accf_bar[a]), 0x3);
        }
      }
      if (*abort && issued) {
        int never = 0;
        umma_commit_pair(smem_u32(&drain_bar), 0x1);
        wait_bounded(smem_u32(&drain_bar), 0, &never, kErrDrain);
      }
    }
  } else if (warp < 2 + C::EPI_WARPS) {
    // ---------------- epilogue (both CTAs, own 128 rows) ----------------
    wide_epilogue<OP>(p, smem, tmem_base, smem_u32(&accf_bar[0]), smem_u32(&acce_bar[0]), abort, warp, lane, rank, pair,
                      pairs, num_m, num_n);
  }

  tc_fence_before();
  cluster_sync_all();  // neither CTA's copies, MMAs or arrivals still target the other
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ------------------------------------------------------------------------------------
// narrow kernel
// ------------------------------------------------------------------------------------
// One tile per cluster: 128 output columns (the MMA's M side) x TN output rows (its N side, so
// a few tokens cost a narrow MMA and a small copy). The cluster's CTAs split the K blocks. CTA c
// finishes rows c TN / S .. of the tile: every CTA stores its fp32 part of them into CTA c's shared
// memory (as [row][128 columns]; stores to a neighbour need no answer, where loads from it take most
// of a microsecond), and CTA c adds the parts in CTA order and runs the epilogue, 4 columns a lane.
//   warp 0      producer: lane i issues the i-th copy of a stage
//   warp 1      MMA issuer, tensor-memory allocation
//   all warps   the sum over the parts and the epilogue
// What bounds it: launch, first loads and the exchange of the parts, about 4 us of every call (one
// token, 2304 from 768: 4.4 us, of which reading the weights takes 0.5); then the weights' bytes (one
// token, 4096 from 4096: 9.2 us; 14336 from 4096: 22.9 us, 5.1 TB/s), and with many rows the reads from
// L2, 24 KB per 64 contraction elements of a 128 x 64 tile (2041 x 768 from 768: 7.0 us).
template <int TN> struct Narrow {
  static constexpr uint32_t QB = TN * BK * 2;               // the row-side operand of a stage
  static constexpr uint32_t STAGE = kHalf + QB;
  static constexpr int STAGES = TN == 128 ? 3 : TN == 64 ? 4 : 5;  // two CTAs per SM
  static constexpr uint32_t SMEM = STAGES * STAGE + 1024;
  static constexpr uint32_t TMEM_COLS = TN;
  static_assert(STAGES * STAGE >= TN * 128 * 4, "the fp32 part takes the stages' place");
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// What follows the main loop, for S CTAs to a tile, by all eight warps: the parts to their owners,
// their sum and the epilogue. `wait` returns once the accumulator is complete.
template <int OP, int TN, int S, class Wait>
__device__ __forceinline__ void finish_tile(const LinearParams& p, uint8_t* smem, uint32_t tmem_base, int rank, int m0,
                                            int n0, int warp, int lane, Wait&& wait) {
  constexpr int ROWS = TN / S;                         // rows this CTA finishes
  constexpr int MINE = ROWS < 8 ? 1 : ROWS / 8;        // rows of a warp: warp, warp + 8, ..
  constexpr int AHEAD = MINE < 8 ? MINE : 8;           // of them, with their side tensors loaded ahead
  const int col = n0 + lane * 4, row0 = m0 + rank * ROWS;
  uint2 bias = make_uint2(0u, 0u);
  if (OP == OP_FWD && p.bias && col < p.n) Side4<OP>::load8(p.bias + col, bias);
  Side4<OP> side[AHEAD];
#pragma unroll
  for (int j = 0; j < AHEAD; ++j)
    if (warp + 8 * j < ROWS) side[j].load(p, row0 + warp + 8 * j, col);

  wait();
  __syncthreads();
  tc_fence_after();
  if (S > 1) cluster_arrive();  // this CTA's stages are free for the others' parts
  // tensor memory lane l = output column n0 + l, column t = output row m0 + t
  const int q = warp & 3, half = warp >> 2;
  const uint32_t base = smem_u32(smem), taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
  if (S > 1) cluster_wait();
#pragma unroll
  for (int t0 = half * 32; t0 < TN; t0 += 64) {
    uint32_t r[32];
    tmem_ld_32cols(taddr + t0, r);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int t = t0 + j;
      const uint32_t at = static_cast<uint32_t>(((rank * ROWS + t % ROWS) * 128 + q * 32 + lane) * 4);
      if (S > 1)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(base, t / ROWS) + at), "r"(r[j]) : "memory");
      else
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + at), "r"(r[j]) : "memory");
    }
  }
  tc_fence_before();
  if (S > 1) cluster_sync_all();  // every part is in its owner's shared memory
  else __syncthreads();
  const float4* part = reinterpret_cast<const float4*>(smem);
  with_act(OP == OP_DW ? FSDP_ACT_NONE : p.act, [&](auto act) {
#pragma unroll
    for (int j = 0; j < MINE; ++j) {
      const int t = warp + 8 * j;
      if (t < ROWS && row0 + t < p.m) {  // the same for the whole warp
        if (j >= AHEAD) side[j % AHEAD].load(p, row0 + t, col);
        f2 v[2];
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const float4 f = part[(s * ROWS + t) * 32 + lane];
          const f2 lo = f2_make(f.x, f.y), hi = f2_make(f.z, f.w);
          v[0] = s == 0 ? lo : f2_add(v[0], lo), v[1] = s == 0 ? hi : f2_add(v[1], hi);
        }
        epilogue4<OP, decltype(act)::value>(p, row0 + t, col, bias, side[j % AHEAD], v);
      }
    }
  });
}

template <int OP, int TN, bool CUT>
__global__ void __launch_bounds__(256, 2) linear_narrow_kernel(const __grid_constant__ LinearParams p) {
  using C = Narrow<TN>;
  constexpr bool P_MN = OP != OP_FWD, Q_MN = OP == OP_DW;  // P: the column side, Q: the row side
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::STAGES];
  __shared__ __align__(8) uint64_t empty_bar[C::STAGES];
  __shared__ __align__(8) uint64_t acc_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);  // one cluster per tile
  const int n0 = static_cast<int>(blockIdx.y) * 128, m0 = static_cast<int>(blockIdx.z) * TN;
  const int num_k = (p.k + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<int64_t>(num_k) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(num_k) * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(&acc_bar), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_sh), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  allow_next_grid();
  const uint32_t tmem_base = tmem_base_sh;

  int issued = 0;  // K blocks, warp 0
  if (warp != 0) wait_for_prior_grids();
  if (warp == 0) {
    Copy c;
    int i = lane;
    bool has = false;  // a copy of this K block
    if constexpr (OP == OP_FWD) i -= w_copies_k_major<CUT>(p, i, n0, kb0, 0, c, has);
    else if constexpr (OP == OP_DX) i -= w_copies_mn_major<CUT>(p, i, n0, kb0, 0, c, has);
    else i -= mn_copies(&p.b, 2, i, n0, kb0, 0, c, has);
    if constexpr (Q_MN) i -= mn_copies(&p.a, TN / 64, i, m0, kb0, kHalf, c, has);
    else i -= k_copies(&p.a, i, m0, kb0, kHalf, c, has);
    const bool mine = CUT && OP == OP_DX ? i < 0 : has;
    if (mine) {
      // While the stream's earlier kernels finish: the copy's map (dW 2304 x 768 from 1024 tokens 8.5 -> 7.6
      // us), and, where W is read by one row of tiles, its first stages to L2, which an earlier kernel's
      // writes to W reach too (one token, repeated calls: 2304 from 768 4.9 -> 4.4 us, 4096 from 4096 10.0
      // -> 9.2; by sixteen rows of tiles 1003 x 1160 from 520 10.1 -> 11.1, so not there).
      if (has) prefetch_tmap(c.map);
      if (OP != OP_DW && gridDim.z == 1 && (!has || c.dst < kHalf)) {
        Copy ahead = c;
        bool some = has;
        for (int kb = kb0; kb < min(kb1, kb0 + C::STAGES); ++kb, some = copy_advance<CUT>(p, ahead))
          if (some) tma_prefetch_2d(ahead.map, ahead.x, ahead.y);
      }
    }
    wait_for_prior_grids();
    uint32_t s = 0, ph = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++issued) {
      bool ok = true;
      if (issued >= C::STAGES)
        ok = wait_bounded(smem_u32(&empty_bar[s]), ph ^ 1u, abort, kErrEmpty);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_arrive_expect_tx(smem_u32(&full_bar[s]), C::STAGE);
      if (mine) {
        if (!(CUT && OP == OP_DX) || has)
          tma_load_2d(smem_u32(smem) + s * C::STAGE + c.dst, c.map, c.x, c.y, smem_u32(&full_bar[s]));
        has = copy_advance<CUT>(p, c);
      }
      __syncwarp();
      if (++s == C::STAGES) s = 0, ph ^= 1u;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t p_step = P_MN ? 128u : 2u, q_step = Q_MN ? 128u : 2u;
      constexpr uint32_t idesc = idesc_bf16_f32(128, TN, P_MN, Q_MN);
      uint32_t s = 0, ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bounded(smem_u32(&full_bar[s]), ph, abort, kErrFull)) break;
        tc_fence_after();
        const uint32_t sp = smem_u32(smem) + s * C::STAGE;
        const uint64_t pd = P_MN ? sw128_mnmajor_desc(sp, kChunk) : sw128_kmajor_desc(sp);
        const uint64_t qd = Q_MN ? sw128_mnmajor_desc(sp + kHalf, kChunk) : sw128_kmajor_desc(sp + kHalf);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          umma_bf16(tmem_base, pd + p_step * k, qd + q_step * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
        umma_commit(smem_u32(&empty_bar[s]));
        if (++s == C::STAGES) s = 0, ph ^= 1u;
      }
      umma_commit(smem_u32(&acc_bar));  // every MMA issued, also after a wait that gave up
    }
    __syncwarp();
  }

  // the accumulator is complete (or, after an abort, no MMA runs any more)
  const auto wait = [&] {
    int never = 0;
    wait_bounded(smem_u32(&acc_bar), 0, &never, kErrAccF);
    if (*abort && warp == 0)  // copies in flight still write this CTA's shared memory
      for (int j = max(0, issued - C::STAGES); j < issued; ++j)
        wait_bounded(smem_u32(&full_bar[j % C::STAGES]), static_cast<uint32_t>(j / C::STAGES) & 1u, &never, kErrDrain);
  };
  switch (splits) {
    case 1: finish_tile<OP, TN, 1>(p, smem, tmem_base, rank, m0, n0, warp, lane, wait); break;
    case 2: finish_tile<OP, TN, 2>(p, smem, tmem_base, rank, m0, n0, warp, lane, wait); break;
    case 4: finish_tile<OP, TN, 4>(p, smem, tmem_base, rank, m0, n0, warp, lane, wait); break;
    default:  // 128-row tiles are split in 8 only for long fp32 weight gradients
      if constexpr (TN != 128 || OP == OP_DW) finish_tile<OP, TN, 8>(p, smem, tmem_base, rank, m0, n0, warp, lane, wait);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

int encoder(const char* who) {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", who);
}

// row-major [rows, cols] of bf16 or fp32, boxes of box_cols x box_rows (128 bytes wide) in the
// 128-byte swizzle; out of range reads zeros, writes nothing
int encode(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_cols, int box_rows, bool fp32,
           const char* who) {
  const int rc = encoder(who);
  if (rc) return rc;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * (fp32 ? 4 : 2)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(ZERO_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", who, (int)r);
  return ZERO_OK;
}

// row-major [rows, cols] bf16 (cols % 64 == 0) read MN-major: element (x, y, z) is row y, column 64 z +
// x; boxes of 64 x BK x 2 land as two chunks of 64 columns
int encode_mn(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, const char* who) {
  int rc = encoder(who);
  if (rc) return rc;
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(BK), 2};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(ZERO_ERR_CUDA, "%s: cuTensorMapEncodeTiled (MN-major) failed (%d)", who, (int)r);
  return ZERO_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class K>
int set_smem(OncePerDevice& once, K kernel, uint32_t bytes, const char* who) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = once.run(dev, [&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    });
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

template <int OP, int COPIES>
int launch_wide(const LinearParams& p, cudaStream_t st, const char* who) {
  using C = Wide<OP>;
  static OncePerDevice once;
  int rc = set_smem(once, linear_wide_kernel<OP, COPIES>, C::SMEM, who);
  if (rc) return rc;
  const int64_t tiles = static_cast<int64_t>((p.m + 255) / 256) * ((p.n + 255) / 256);
  if (tiles > INT32_MAX / 2)
    return set_error(ZERO_ERR_UNSUPPORTED, "%s: an output of %d x %d is more than 2^30 tiles", who, p.m, p.n);
  const unsigned int pairs = static_cast<unsigned int>(std::min<int64_t>(tiles, std::max(1, num_sms() / 2)));
  const cudaError_t e =
      launch_overlapped(linear_wide_kernel<OP, COPIES>, dim3(2 * pairs), dim3(C::THREADS), C::SMEM, 1, st, p);
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

template <int OP, int TN, bool CUT>
int launch_narrow(const LinearParams& p, int splits, cudaStream_t st, const char* who) {
  using C = Narrow<TN>;
  static OncePerDevice once;
  int rc = set_smem(once, linear_narrow_kernel<OP, TN, CUT>, C::SMEM, who);
  if (rc) return rc;
  const dim3 grid(static_cast<unsigned>(splits), static_cast<unsigned>((p.n + 127) / 128),
                  static_cast<unsigned>((p.m + TN - 1) / TN));
  const cudaError_t e = launch_overlapped(linear_narrow_kernel<OP, TN, CUT>, grid, dim3(256), C::SMEM,
                                          static_cast<unsigned>(splits), st, p);
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

// fp32 weight gradients: the tensor cores add to the accumulator with truncation, about
// 2^-24 of it per step, always toward zero (measured: 1.9e-5 of the result's norm over 16384
// terms, 4.4e-6 over 4096). So an fp32 result is summed in parts of at most 64 blocks (4096
// tokens), which are added with rounding to nearest: the narrow kernel's splits, or the wide
// kernel's chunks, added in memory by the same warp in order. bf16 results round 2^-8 anyway
// and take one part.
constexpr int kMaxChunkBlocks = 64;

// Kernel choice, from both kernels timed over 35 shapes (forward, dx, dw; every tile height and
// split), repeated calls in a graph. The narrow kernel while its 128 x 128 tiles, split in two, are
// resident at once (two CTAs per SM: up to 38 wide tiles; 36 of them, 1024 x 2304 from 768: 9.9 us
// against 11.6) and for up to 128 rows, which leave half of a 256-row tile or more empty; else the
// wide one (48 tiles, 4096 x 768 from 768: 11.9 against 14.4).
//   splits: doubled while every CTA keeps two K blocks and the CTAs are resident at once, beyond
// one CTA per SM only if three blocks are left to each (72 tiles of 8 blocks: 2 splits 5.3 us, 4
// splits 6.2; of 32 blocks: 9.3 and 8.1).
//   rows of a tile: 32 for up to 32 rows (16 x 768 from 768: 4.8 us). A tile of 64 rows passes on half
// of what one of 128 does and needs fewer splits for as many CTAs, but loads the column side for 64
// rows only. So 64 if that leaves 4 splits or more (dW 768 x 768 from 4096: 10.9 us, 128 rows with 8
// splits 14.2, with 4 12.3), or if it loads at most 240 KB per SM more (1024 x 2304 from 768, 182
// KB: 9.9 us against 11.5; dW 2304 x 768 from 1500, 273 KB: 11.4 against 11.0; from 2048, 364 KB: 14.2
// against 12.5).
struct Choice {
  bool wide;
  int tn, splits;
};
Choice choose(int op, int64_t m, int64_t n, int64_t k, bool fp32) {
  const int64_t wide_tiles = ((m + 255) / 256) * ((n + 255) / 256), sms = num_sms();
  const int64_t blocks = (k + BK - 1) / BK, col_tiles = (n + 127) / 128;
  const bool few_rows = op != OP_DW && m <= 128;
  Choice c{true, 128, 1};
  if ((wide_tiles * 4 > sms && !few_rows) || (fp32 && blocks > 8 * kMaxChunkBlocks) || col_tiles > 65535) return c;
  c.wide = false;
  const int64_t tiles64 = ((m + 63) / 64) * col_tiles, tiles128 = ((m + 127) / 128) * col_tiles;
  const auto splits_of = [&](int64_t tiles) {
    int splits = 1;
    while (splits < 8 && blocks >= 4 * splits) {
      const int64_t next = 2 * splits, ctas = tiles * next;
      if (ctas > sms && (ctas > 2 * sms || blocks < 3 * next)) break;
      splits = static_cast<int>(next);
    }
    return splits;
  };
  const int64_t kb = BK * 2 * (128 + 64) / 1024, kb128 = BK * 2 * (128 + 128) / 1024;  // KB of a stage
  if (op != OP_DW && m <= 32)
    c.tn = 32, c.splits = splits_of(col_tiles);
  else if (tiles64 <= 2 * sms &&
           (splits_of(tiles64) >= 4 || blocks * (tiles64 * kb - tiles128 * kb128) <= 240 * sms))
    c.tn = 64, c.splits = splits_of(tiles64);
  else
    c.splits = splits_of(tiles128);
  while (fp32 && c.splits < 8 && blocks > static_cast<int64_t>(c.splits) * kMaxChunkBlocks) c.splits *= 2;
  return c;
}

// the product's operands as the entry points get them
struct Operands {
  int n_shards;
  const uint16_t* const* w;  // fwd, dx
  const uint16_t* a;         // X, dZ, dZ
  const uint16_t* x;         // dw: X
};

template <int OP>
int launch(LinearParams& p, const Operands& o, cudaStream_t st, const char* who) {
  const bool fp32 = p.y32 != nullptr;
  const Choice c = choose(OP, p.m, p.n, p.k, fp32);
  const int blocks = (p.k + BK - 1) / BK;
  p.chunk_blocks = c.wide && fp32 ? kMaxChunkBlocks : blocks;
  p.chunks = (blocks + p.chunk_blocks - 1) / p.chunk_blocks;
  int rc;
  bool fast = c.wide;  // one copy per operand and stage
  if constexpr (OP == OP_DW) {
    fast = fast && p.m % 64 == 0 && p.n % 64 == 0;
    if ((rc = fast ? encode_mn(&p.a, o.a, p.k, p.m, who) : encode(&p.a, o.a, p.k, p.m, 64, BK, false, who))) return rc;
    if ((rc = fast ? encode_mn(&p.b, o.x, p.k, p.n, who) : encode(&p.b, o.x, p.k, p.n, 64, BK, false, who)))
      return rc;
  } else {
    if ((rc = encode(&p.a, o.a, p.m, p.k, BK, c.wide ? 128 : c.tn, false, who))) return rc;
    const int most = OP == OP_FWD ? 128 : BK;
    p.n_shards = o.n_shards;
    // shards that lie back to back are one matrix: one map, and boxes of any height
    const int64_t shard_elems = static_cast<int64_t>(p.shard_rows) * (OP == OP_FWD ? p.k : p.n);
    bool joined = true;
    for (int s = 1; s < o.n_shards; ++s) joined = joined && o.w[s] == o.w[0] + s * shard_elems;
    if (joined) p.shard_rows *= p.n_shards, p.n_shards = 1;
    // one shard: rows past the last are zeros in any box, so it may be whole
    p.w_box = p.n_shards == 1 ? most : std::min(p.shard_rows & -p.shard_rows, most);
    for (p.w_box_log = 3; (1 << p.w_box_log) < p.w_box;) ++p.w_box_log;
    // copies below 32 rows keep the producer behind: as many as fit in a copy of 4, 16 times the rows
    p.w_levels = 1;
    if (p.w_box < 32)
      while ((p.w_levels + 1) * p.n_shards <= kGemmMaxPieces && (p.w_box << (2 * (p.w_levels - 1))) < most) ++p.w_levels;
    fast = fast && p.w_box == most && (OP == OP_FWD || p.n % 64 == 0);
    const int64_t w_cols = OP == OP_FWD ? p.k : p.n;
    for (int i = 0; i < p.w_levels * p.n_shards; ++i) {
      const int s = i % p.n_shards, box = std::min(p.w_box << (2 * (i / p.n_shards)), most);
      rc = OP == OP_DX && fast ? encode_mn(&p.w[i], o.w[s], p.shard_rows, w_cols, who)
                               : encode(&p.w[i], o.w[s], p.shard_rows, w_cols, 64, box, false, who);
      if (rc) return rc;
    }
  }
  if (c.wide && fp32 && (rc = encode(&p.out, p.y32, p.m, p.n, 32, 32, true, who))) return rc;
  if constexpr (OP != OP_DW)
    if (p.w_levels > 1) {
      if (c.wide) return launch_wide<OP, COPIES_CUT>(p, st, who);
      if (c.tn == 32) return launch_narrow<OP, 32, true>(p, c.splits, st, who);
      if (c.tn == 64) return launch_narrow<OP, 64, true>(p, c.splits, st, who);
      return launch_narrow<OP, 128, true>(p, c.splits, st, who);
    }
  if (c.wide)
    return fast ? launch_wide<OP, COPIES_ONE>(p, st, who) : launch_wide<OP, COPIES_EQUAL>(p, st, who);
  if constexpr (OP != OP_DW)
    if (c.tn == 32) return launch_narrow<OP, 32, false>(p, c.splits, st, who);
  if (c.tn == 64) return launch_narrow<OP, 64, false>(p, c.splits, st, who);
  return launch_narrow<OP, 128, false>(p, c.splits, st, who);
}

int check_sizes(int64_t m, int64_t r, int64_t k, const char* who) {
  const int64_t most = 1 << 30;
  if (m < 1 || r < 1 || k < 1 || m > most || r > most || k > most)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: m_tokens, rows_out and k_in must be in 1..2^30", who);
  if (r % 8 || k % 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: rows_out %lld and k_in %lld must be multiples of 8 (16-byte rows)", who,
                     (long long)r, (long long)k);
  return ZERO_OK;
}

int check_shards(LinearParams* p, int n, const zero_bf16* const w_shards[], int64_t rows_out, const char* who) {
  if (n < 1 || n > kGemmMaxPieces)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: n_ranks %d outside 1..%d", who, n, kGemmMaxPieces);
  if (rows_out % n || (rows_out / n) % 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: rows_out / n_ranks (%lld / %d) must be a multiple of 8", who,
                     (long long)rows_out, n);
  if (!w_shards) return set_error(ZERO_ERR_INVALID_ARG, "%s: w_shards is NULL", who);
  for (int q = 0; q < n; ++q) {
    if (!w_shards[q])
      return set_error(ZERO_ERR_INVALID_ARG, "%s: w_shards[%d] is NULL (missing rank)", who, q);
    if (!aligned16(w_shards[q]))
      return set_error(ZERO_ERR_INVALID_ARG, "%s: w_shards[%d] must be 16-byte aligned", who, q);
  }
  p->shard_rows = static_cast<int>(rows_out / n);
  return ZERO_OK;
}


}  // namespace

unsigned int fsdp_linear_read_clear_error() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_zgb_dev_error, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v) cudaMemcpyToSymbol(g_zgb_dev_error, &zero, sizeof(zero));
  return v;
}

}  // namespace zgb

using namespace zgb;

extern "C" int fsdp_linear_forward(int n_ranks, const zero_bf16* const w_shards[], int64_t rows_out, int64_t k_in,
                                   const zero_bf16* X, int64_t m_tokens, const zero_bf16* bias, int act,
                                   const zero_bf16* residual, zero_bf16* Y, zero_bf16* z, int8_t* z_codes,
                                   uint8_t* z_scales, zero_stream_t stream) {
  const char* who = "fsdp_linear_forward";
  LinearParams p;
  memset(&p, 0, sizeof(p));
  int rc;
  if ((rc = check_sizes(m_tokens, rows_out, k_in, who))) return rc;
  if ((rc = check_shards(&p, n_ranks, w_shards, rows_out, who))) return rc;
  if (act < FSDP_ACT_NONE || act > FSDP_ACT_SILU)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: act %d is not one of FSDP_ACT_*", who, act);
  if (!X || !Y) return set_error(ZERO_ERR_INVALID_ARG, "%s: X or Y is NULL", who);
  if ((z_codes != nullptr) != (z_scales != nullptr) || (z && z_codes))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: keep Z as z, or as both z_codes and z_scales, or not at all", who);
  if (!aligned16(X) || !aligned16(bias) || !aligned16(residual) || !aligned16(Y) || !aligned16(z) ||
      !aligned16(z_codes) || !aligned16(z_scales))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: every buffer must be 16-byte aligned", who);
  p.m = static_cast<int>(m_tokens), p.n = static_cast<int>(rows_out), p.k = static_cast<int>(k_in);
  p.bias = bias, p.res = residual, p.act = act;
  p.y = Y, p.z = z, p.zc = z_codes, p.zs = z_scales;
  const Operands o{n_ranks, w_shards, X, nullptr};
  return launch<OP_FWD>(p, o, reinterpret_cast<cudaStream_t>(stream), who);
}

extern "C" int fsdp_linear_dx(int n_ranks, const zero_bf16* const w_shards[], int64_t rows_out, int64_t k_in,
                              const zero_bf16* dZ, int64_t m_tokens, const zero_bf16* z, const int8_t* z_codes,
                              const uint8_t* z_scales, int act, const zero_bf16* residual, zero_bf16* dX,
                              zero_stream_t stream) {
  const char* who = "fsdp_linear_dx";
  LinearParams p;
  memset(&p, 0, sizeof(p));
  int rc;
  if ((rc = check_sizes(m_tokens, rows_out, k_in, who))) return rc;
  if ((rc = check_shards(&p, n_ranks, w_shards, rows_out, who))) return rc;
  if (!dZ || !dX) return set_error(ZERO_ERR_INVALID_ARG, "%s: dZ or dX is NULL", who);
  if ((rc = check_kept_activation(z, z_codes, z_scales, act, who))) return rc;
  if (!aligned16(dZ) || !aligned16(residual) || !aligned16(dX))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: every buffer must be 16-byte aligned", who);
  p.m = static_cast<int>(m_tokens), p.n = static_cast<int>(k_in), p.k = static_cast<int>(rows_out);
  p.res = residual, p.act = act, p.y = dX;
  if (act != FSDP_ACT_NONE) p.z_in = z, p.zc_in = z_codes, p.zs_in = z_scales;
  const Operands o{n_ranks, w_shards, dZ, nullptr};
  return launch<OP_DX>(p, o, reinterpret_cast<cudaStream_t>(stream), who);
}

// X from an 8-bit checkpoint is unpacked into the workspace first, 3 bytes of traffic per element
// against 2 rows_out flops: 3 % of the product's time at rows_out = 4096. Converting codes inside
// the product's operand loads saves that traffic but repeats the conversion for every 256 rows of
// dW: measured 2.5 times the whole product's time at rows_out = 14336.
extern "C" int fsdp_linear_dw_workspace(int64_t m_tokens, int64_t k_in, uint64_t* bytes) {
  const char* who = "fsdp_linear_dw_workspace";
  if (!bytes) return set_error(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  const int rc = check_sizes(m_tokens, 8, k_in, who);
  if (rc) return rc;
  *bytes = (2 * static_cast<uint64_t>(m_tokens) * static_cast<uint64_t>(k_in) + 255) & ~uint64_t(255);
  return ZERO_OK;
}

extern "C" int fsdp_linear_dw(const zero_bf16* dZ, const zero_bf16* x, const int8_t* x_codes, const uint8_t* x_scales,
                              int64_t m_tokens, int64_t rows_out, int64_t k_in, float scale, float* dW,
                              zero_bf16* dW_bf16, void* workspace, uint64_t workspace_bytes, zero_stream_t stream) {
  const char* who = "fsdp_linear_dw";
  LinearParams p;
  memset(&p, 0, sizeof(p));
  int rc;
  if ((rc = check_sizes(m_tokens, rows_out, k_in, who))) return rc;
  if (!dZ) return set_error(ZERO_ERR_INVALID_ARG, "%s: dZ is NULL", who);
  if ((x_codes != nullptr) != (x_scales != nullptr) || (x != nullptr) == (x_codes != nullptr))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: pass X as x, or as both x_codes and x_scales", who);
  if ((dW != nullptr) == (dW_bf16 != nullptr))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: pass one of dW and dW_bf16", who);
  if (!(scale - scale == 0.0f)) return set_error(ZERO_ERR_INVALID_ARG, "%s: scale must be finite", who);
  if (!aligned16(dZ) || !aligned16(x) || !aligned16(x_codes) || !aligned16(x_scales) || !aligned16(dW) ||
      !aligned16(dW_bf16) || (x_codes && !aligned16(workspace)))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: every buffer must be 16-byte aligned", who);
  if (x_codes) {
    uint64_t need = 0;
    if ((rc = fsdp_linear_dw_workspace(m_tokens, k_in, &need))) return rc;
    if (!workspace || workspace_bytes < need)
      return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                       workspace ? (unsigned long long)workspace_bytes : 0ull, (unsigned long long)need);
    if ((rc = fsdp_checkpoint8_unpack(x_codes, x_scales, m_tokens, k_in, FSDP_ACT_NONE,
                                      static_cast<zero_bf16*>(workspace), stream)))
      return rc;
    x = static_cast<const zero_bf16*>(workspace);
  }
  p.m = static_cast<int>(rows_out), p.n = static_cast<int>(k_in), p.k = static_cast<int>(m_tokens);
  p.scale = scale, p.y32 = dW, p.y = dW_bf16;
  const Operands o{0, nullptr, dZ, x};
  return launch<OP_DW>(p, o, reinterpret_cast<cudaStream_t>(stream), who);
}
