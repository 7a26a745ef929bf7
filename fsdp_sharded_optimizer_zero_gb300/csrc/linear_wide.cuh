// The CTA-pair tensor-core kernel of the linear unit and of the loss over the vocabulary: its
// operand copies, its waits, its main loop and the staging its epilogues share. The epilogue of
// each operation is in the file that launches it.
#pragma once

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

// The products. What an operation loads: like the forward (both operands K-major, the second W's row
// shards), like dx (W's shards read MN-major along the contraction) or like dw (both MN-major).
//   OP_LSE, OP_DLOGITS      the loss over the vocabulary: its forward's and backward's logits
//   OP_LSE_PARTS, OP_DLOGITS_PARTS    the same, their contraction summed in parts
//   OP_DX_SPLIT             an input gradient whose contraction is split over pairs
//   OP_DW_SHORT             a bf16 weight gradient of few tokens, bound by its stores: eight epilogue warps, not four
enum { OP_FWD, OP_DX, OP_DW, OP_DW_SHORT, OP_LSE, OP_LSE_PARTS, OP_DLOGITS, OP_DLOGITS_PARTS, OP_DX_SPLIT };
__host__ __device__ constexpr bool is_lse(int op) { return op == OP_LSE || op == OP_LSE_PARTS; }
__host__ __device__ constexpr bool is_dlogits(int op) { return op == OP_DLOGITS || op == OP_DLOGITS_PARTS; }
__host__ __device__ constexpr bool is_logits(int op) { return is_lse(op) || is_dlogits(op); }
__host__ __device__ constexpr bool loads_as_fwd(int op) { return op == OP_FWD || is_logits(op); }
__host__ __device__ constexpr bool is_dw(int op) { return op == OP_DW || op == OP_DW_SHORT; }
__host__ __device__ constexpr bool loads_as_dx(int op) { return op == OP_DX || op == OP_DX_SPLIT; }

constexpr int BK = 64;                        // contraction elements of one stage (128 bytes of bf16)
constexpr uint32_t kHalf = 128 * BK * 2;      // 128 rows (or MN-major columns) of one operand: 16 KiB
constexpr uint32_t kChunk = 64 * BK * 2;      // 64 columns of an MN-major operand: 8 KiB

constexpr unsigned int kErrEmpty = (5u << 8) | 1u;  // producer waiting for a free stage
constexpr unsigned int kErrFull = (5u << 8) | 2u;   // MMA waiting for a filled stage
constexpr unsigned int kErrAccE = (5u << 8) | 3u;   // MMA waiting for a drained accumulator
constexpr unsigned int kErrAccF = (5u << 8) | 4u;   // epilogue waiting for a finished accumulator
constexpr unsigned int kErrDrain = (5u << 8) | 5u;  // waiting for copies or MMAs in flight

struct ProductParams {
  CUtensorMap a;                  // fwd: X, dx: dZ (K-major, box 64 x 128 or TN rows); dw: dZ (MN-major, box 64 x 64)
  CUtensorMap b;                  // dw: X (MN-major, box 64 x 64)
  CUtensorMap out;                // wide kernel, fp32 dW: the output, boxes of 32 columns x 32 rows
  int m, n, k;                    // the product: out [m, n], contraction over k
  int n_shards, shard_rows;       // fwd, dx
  int w_levels, w_shift;          // heights of W's copies: w_box, w_box << w_shift, ..
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
  const float* count;             // dw: nullable, what the scale is divided by (1 at least)
  int chunks, chunk_blocks;       // fp32 dw, logits: the contraction in chunks of chunk_blocks K blocks (1 chunk otherwise)
};
// fwd, dx: the row shards of W, boxes of 64 columns x w_box rows; where they are cut to fit (w_levels > 1), again with
// boxes of the other heights
struct LinearParams : ProductParams {
  CUtensorMap w[kGemmMaxPieces];
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
// shard allows of the heights up to ROWS; false if there are fewer. Rows past the last one count to
// the last shard, past its end (they read zeros).
template <int ROWS, class P>
__device__ __forceinline__ bool w_piece(const P& p, Copy& c) {
  int shard = c.shard, y = c.row, at = 0, level = p.w_levels - 1;
  const auto box = [&](int l) { return min(p.w_box << (p.w_shift * l), ROWS); };
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
// to the next K block; false: this lane has nothing to copy for it (had: whether it had for this one)
template <bool CUT, class P>
__device__ __forceinline__ bool copy_advance(const P& p, Copy& c, bool had) {
  if (c.k_major) {
    c.x += BK;
  } else if (CUT && c.w_rows) {
    // inside a shard a block's copies are the last one's, further down (a new cut for each block keeps the
    // producer behind: 0.51 us a block where the products take 0.34)
    const bool whole = c.row + BK <= p.shard_rows;
    c.row += BK;
    if (whole && c.row + BK <= p.shard_rows) {
      c.y += BK;
      return had;
    }
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
template <class P>
__device__ __forceinline__ void copy_seek(const P& p, Copy& c, int row) {
  c.shard = min(row / p.shard_rows, p.n_shards - 1);
  c.map = &p.w[c.shard];
  c.y = row - c.shard * p.shard_rows;
}
// copies of W (fwd): 128 output columns from n0, K-major, 128 / w_box copies of w_box rows, or (CUT) up to
// as many lanes with `has` true
template <bool CUT, class P>
__device__ __forceinline__ int w_copies_k_major(const P& p, int i, int n0, int kb0, uint32_t dst, Copy& c,
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
template <bool CUT, class P>
__device__ __forceinline__ int w_copies_mn_major(const P& p, int i, int n0, int kb0, uint32_t dst, Copy& c,
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
// the buffer to rows r0 .., columns c0 .. of dst [m, n], whose rows are ld apart
__device__ __forceinline__ void stage_store(const uint8_t* buf, uint16_t* dst, int r0, int c0, int m, int n, int ld,
                                            int lane) {
  const int j = lane & 7, col = c0 + 8 * j, i0 = lane >> 3;  // rows i0, i0 + 4, ..: two alternating slots
  const int left = col < n ? m - r0 - i0 : 0;
  uint16_t* to = dst + static_cast<size_t>(r0 + i0) * ld + col;
  const size_t step = static_cast<size_t>(4) * ld;
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

// ------------------------------------------------------------------------------------
// wide kernel
// ------------------------------------------------------------------------------------
// A cluster of two CTAs on two SMs per 256 x 256 output tile: each CTA loads 128 rows of the
// first operand and 128 columns of the second, and the even CTA's MMA (M = N = 256) reads both
// CTAs' shared memory. Persistent, two accumulators in tensor memory.
//   warp 0       producer: lane i issues the i-th copy of a stage (TMA), both CTAs
//   warp 1       MMA issuer (even CTA), tensor-memory allocation
//   then 8 (dw: 4, of few tokens 8) epilogue warps, two (one) per tensor-memory lane quarter, sharing its columns
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
  using Params = LinearParams;
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

// what a weight gradient's sums are multiplied by
__device__ __forceinline__ float dw_scale(float scale, const float* count) {
  return count ? __fdiv_rn(scale, fmaxf(__ldg(count), 1.0f)) : scale;
}

// fp32 output: this warp's 32 rows (from row `row` of `out`) and COLS columns (from c0, those below n) of
// an accumulator, scaled, through two staging buffers. `stores` counts the bulk stores that this warp has
// made: the two buffers alternate over all of them, across tiles, and a buffer is written again once all
// stores but the newest, which reads the other one, have read theirs. Counted by a tile's own columns, two
// stores in a row would leave from buffer 0 where a tile at the right edge has an odd number of 32-column
// blocks. add: to what is there. live: whether this thread's row is anything but zeros.
template <int COLS>
__device__ __forceinline__ void store_sums(const CUtensorMap* out, uint32_t taddr, int row, int c0, int n, float scale,
                                           bool add, uint8_t* stage, uint32_t& stores, int lane, bool live = true) {
#pragma unroll 1
  for (int c = 0; c < COLS; c += 32) {
    uint32_t r[32];
    tmem_ld_32cols(taddr + c, r);
    if (c0 + c >= n) continue;
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = live ? r[j] : 0u;
    const f2 s = f2_both(scale);
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
      if (add) tma_reduce_add_2d(out, c0 + c, row, smem_u32(buf));
      else tma_store_2d(out, c0 + c, row, smem_u32(buf));
      bulk_commit_group();
    }
  }
}

// The epilogue warps' role, defined beside each operation.
template <int OP>
__device__ __forceinline__ void wide_epilogue(const typename Wide<OP>::Params& p, uint8_t* smem, uint32_t tmem_base,
                                              uint32_t accf_bar, uint32_t acce_bar, volatile int* abort, int warp,
                                              int lane, uint32_t rank, int pair, int pairs, int num_m, int num_n);
// What else the loss over the vocabulary sets: where in W its columns (logits) or its
// contraction (OP_DX_SPLIT) begin, and in how many parts the contraction is summed.
template <int OP>
__device__ __forceinline__ int first_w_row(const typename Wide<OP>::Params& p) {
  if constexpr (is_logits(OP) || OP == OP_DX_SPLIT) return p.w_row0;
  return 0;
}
// A work item of the persistent loop: an output tile, and (OP_DX_SPLIT) the K blocks of one part
template <int OP>
struct WideItem {
  int tile, kb0, kb1;
  __device__ __forceinline__ WideItem(const typename Wide<OP>::Params& p, int item, int tiles, int num_k)
      : tile(item), kb0(0), kb1(num_k) {
    if constexpr (OP == OP_DX_SPLIT) {
      const int part = item / tiles;
      tile = item - part * tiles;
      kb0 = static_cast<int>(static_cast<int64_t>(num_k) * part / p.splits);
      kb1 = static_cast<int>(static_cast<int64_t>(num_k) * (part + 1) / p.splits);
    }
  }
};
template <int OP>
__device__ __forceinline__ int wide_items(const typename Wide<OP>::Params& p, int tiles) {
  if constexpr (OP == OP_DX_SPLIT) return tiles * p.splits;
  return tiles;
}

enum { COPIES_EQUAL, COPIES_ONE, COPIES_CUT };
template <int OP, int COPIES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide<OP>::THREADS, 1)
    linear_wide_kernel(const __grid_constant__ typename Wide<OP>::Params p) {
  using C = Wide<OP>;
  constexpr bool A_MN = is_dw(OP), B_MN = !loads_as_fwd(OP);
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
  const int tiles = num_m * num_n, items = wide_items<OP>(p, tiles);

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
        for (int item = pair; item < items && !stop; item += pairs) {
          const WideItem<OP> w(p, item, tiles, num_k);
          int mb, nb;
          wide_tile_coords(w.tile, num_m, num_n, mb, nb);
          const int m0 = mb * 256 + static_cast<int>(rank) * 128, n0 = nb * 256 + static_cast<int>(rank) * 128;
          int shard = 0, row = 0;  // W: the shard and its row of this tile (fwd) or K block (dx)
          if constexpr (loads_as_fwd(OP) || OP == OP_DX_SPLIT) {
            row = first_w_row<OP>(p) + (loads_as_fwd(OP) ? n0 : w.kb0 * BK);
            shard = min(row / p.shard_rows, p.n_shards - 1), row -= shard * p.shard_rows;
          }
          for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
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
            if constexpr (loads_as_fwd(OP)) {
              tma_load_2d_pair(sa + kHalf, &p.w[shard], kb * BK, row, fb);
            } else if constexpr (loads_as_dx(OP)) {
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
    for (int item = pair; item < items && !stop; item += pairs) {
      const WideItem<OP> w(p, item, tiles, num_k);
      int mb, nb;
      wide_tile_coords(w.tile, num_m, num_n, mb, nb);
      const int m0 = mb * 256 + static_cast<int>(rank) * 128, n0 = nb * 256 + static_cast<int>(rank) * 128;
      Copy c;
      int i = lane;
      bool has = false;  // a copy of this K block
      constexpr bool CUT = COPIES == COPIES_CUT;
      if constexpr (A_MN) i -= mn_copies(&p.a, 2, i, m0, 0, 0, c, has);
      else i -= k_copies(&p.a, i, m0, w.kb0, 0, c, has);
      if constexpr (loads_as_fwd(OP)) i -= w_copies_k_major<CUT>(p, i, first_w_row<OP>(p) + n0, 0, kHalf, c, has);
      else if constexpr (loads_as_dx(OP))
        i -= w_copies_mn_major<CUT>(p, i, n0, first_w_row<OP>(p) / BK + w.kb0, kHalf, c, has);
      else i -= mn_copies(&p.b, 2, i, n0, 0, kHalf, c, has);
      const bool mine = CUT && loads_as_dx(OP) ? i < 0 : has;
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
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
          if (!(CUT && loads_as_dx(OP)) || has)
            tma_load_2d_pair(smem_u32(smem) + s * C::STAGE + c.dst, c.map, c.x, c.y,
                             mapa_shared(smem_u32(&full_bar[s]), 0));
          has = copy_advance<CUT>(p, c, has);
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
      for (int item = pair; item < items && !stop; item += pairs) {
        const WideItem<OP> w(p, item, tiles, num_k);
        for (int kb = w.kb0; kb < w.kb1 && !stop; ++i) {  // one accumulator per chunk
          const int kb_end = min(kb + p.chunk_blocks, w.kb1), kb_first = kb;
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

// row-major [rows, cols] of bf16 or fp32, rows ld elements apart, boxes of box_cols x box_rows (128 bytes
// wide) in the 128-byte swizzle; out of range reads zeros, writes nothing
int encode(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_cols, int box_rows,
           bool fp32, const char* who) {
  const int rc = encoder(who);
  if (rc) return rc;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * (fp32 ? 4 : 2)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = g_encode(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(ZERO_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", who, (int)r);
  return ZERO_OK;
}

// row-major [rows, cols] bf16 (cols % 64 == 0), rows ld elements apart, read MN-major: element (x, y, z) is
// row y, column 64 z + x; boxes of 64 x BK x 2 land as two chunks of 64 columns
int encode_mn(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, const char* who) {
  int rc = encoder(who);
  if (rc) return rc;
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, 128};
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

// The maps of W, given as n row shards of p.shard_rows rows, as a forward (K-major, rows of k elements) or dx
// (MN-major, rows of n elements) loads it: p.w, p.n_shards, p.shard_rows, p.w_box and p.w_levels. Of its rows
// those from `rows` on are not there (they read zeros): the last shard's end may be padding. cut_from: copies of
// fewer rows than this are cut to fit, as many heights as there are maps for: each four times the one before, or
// (long_shards, whose rows are cut at few places) the lowest and the highest only. one_copy: whether an operand of a
// stage may be one copy; cleared where W's shards do not allow it.
template <class P>
int encode_w(P& p, int n, const uint16_t* const* w, int64_t rows, bool fwd, int cut_from, bool long_shards, bool* one_copy,
             const char* who) {
  const int most = fwd ? 128 : BK, maps = long_shards ? static_cast<int>(sizeof(p.w) / sizeof(p.w[0])) : kGemmMaxPieces;
  const int64_t cols = fwd ? p.k : p.n;
  p.n_shards = n;
  // shards that lie back to back are one matrix: one map, and boxes of any height
  const int64_t shard_elems = static_cast<int64_t>(p.shard_rows) * cols;
  bool joined = true;
  for (int s = 1; s < n; ++s) joined = joined && w[s] == w[0] + s * shard_elems;
  if (joined) p.shard_rows *= p.n_shards, p.n_shards = 1;
  // one shard: rows past the last are zeros in any box, so it may be whole
  p.w_box = p.n_shards == 1 ? most : std::min(p.shard_rows & -p.shard_rows, most);
  for (p.w_box_log = 3; (1 << p.w_box_log) < p.w_box;) ++p.w_box_log;
  p.w_levels = 1, p.w_shift = 2;
  if (p.w_box < cut_from) {
    if (long_shards)
      for (; p.w_box << p.w_shift < most;) ++p.w_shift;
    while ((p.w_levels + 1) * p.n_shards <= maps && (p.w_box << (p.w_shift * (p.w_levels - 1))) < most) ++p.w_levels;
  }
  *one_copy = *one_copy && p.w_box == most && (fwd || p.n % 64 == 0);
  for (int i = 0; i < p.w_levels * p.n_shards; ++i) {
    const int s = i % p.n_shards, box = std::min(p.w_box << (p.w_shift * (i / p.n_shards)), most);
    const int64_t left = std::min<int64_t>(p.shard_rows, rows - static_cast<int64_t>(s) * p.shard_rows);
    const int rc = !fwd && *one_copy ? encode_mn(&p.w[i], w[s], left, cols, cols, who)
                                     : encode(&p.w[i], w[s], left, cols, cols, 64, box, false, who);
    if (rc) return rc;
  }
  return ZERO_OK;
}

template <int OP, int COPIES>
int launch_wide(const typename Wide<OP>::Params& p, cudaStream_t st, const char* who) {
  using C = Wide<OP>;
  static OncePerDevice once;
  int rc = set_smem(once, linear_wide_kernel<OP, COPIES>, C::SMEM, who);
  if (rc) return rc;
  const int64_t tiles = static_cast<int64_t>((p.m + 255) / 256) * ((p.n + 255) / 256);
  if (tiles > INT32_MAX / 2)
    return set_error(ZERO_ERR_UNSUPPORTED, "%s: an output of %d x %d is more than 2^30 tiles", who, p.m, p.n);
  int64_t items = tiles;
  if constexpr (OP == OP_DX_SPLIT) items *= p.splits;
  const unsigned int pairs = static_cast<unsigned int>(std::min<int64_t>(items, std::max(1, num_sms() / 2)));
  const cudaError_t e =
      launch_overlapped(linear_wide_kernel<OP, COPIES>, dim3(2 * pairs), dim3(C::THREADS), C::SMEM, 1, st, p);
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
}

}  // namespace
}  // namespace zgb
