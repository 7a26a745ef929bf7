// The loss over the vocabulary on the 5th-generation tensor cores: softmax cross entropy of the logits
// Z = X W^T, W the output layer held as row shards, without keeping Z.
//
//   forward   lse_i = log sum_v exp Z_iv, loss_i = lse_i - Z_i[label]: each 256 x 256 tile of Z leaves, per
//             row and 128 columns, its maximum and the sum of exponentials below it (2 fp32), joined after
//   backward  in pieces of the vocabulary: Z again from X and the piece of W, dZ = exp(Z - lse) - onehot in bf16,
//             then the piece's rows of dW = dZ^T (c g X), and dX += c g dZ W; c what all tokens share (the loss's
//             scale, one over the count), g a token's own factor
//
// The products run in linear_wide_kernel, of few tokens in linear_narrow_kernel; what is here are their epilogues and the
// joining passes. Softmax
// statistics and all sums are fp32. dZ is rounded to bf16, as the gradient of a linear unit's output is
// everywhere in the library: the tensor cores multiply bf16, and its gradients are bf16. The factors are left out of it:
// the label's element is about -1 and so hardly rounded, while with c it would be rounded alike for every token, which
// biases every gradient by up to 2^-9 (8192 x 32000 from 4096: 3.7e-3 of the gradients' norm off, without 1.7e-3, the
// outputs' own rounding). c and g multiply fp32 sums; only for dW, whose sums are over the tokens, g (and c with it) goes
// into X, rounded to bf16 once more: a word that is the label of one token gets that product, which the output no longer
// rounds (777 x 50257 from 768: dW 2.2e-3 off, with g in dZ 2.4e-3; where words are many tokens' labels up to 2.6e-3; the
// output's rounding alone 1.7e-3). What that rounds off, as a second part of X, would take dW's product once more, a third
// of the call.
//
// Bound by tensor work. On the device, in a graph of a few ms, W as 8 shards back to back: forward 8192 x 50257 from 768
// 347-357 us (1.78-1.82 PFLOP/s; tensor pipe 82 % active), of which joining the parts takes about 10, from 4096 (vocabulary
// 32000) 1128 us (1.90); gradients 8192 x 32000 from 4096 3.52-3.62 ms (1.78-1.83), 8192 x 50257 from 768 1.13-1.19 ms
// (1.59-1.69: dZ's product 394 us, held up by the 824 MB that it writes, tensor pipe 73 %; dW's 361, dX's 340). Called
// again and again the board is at its power limit: the first 385-402 us, the third 3.9-4.1 ms. Shards that lie apart and end
// inside tiles cost copies: 50257 x 768 361 us and 1.25 ms. Of few tokens: W's bytes, one of 32000 x 4096 45 us (5.8 TB/s;
// shards apart 51), its gradients 157 (W read twice, dW written). One of 50257 x 768 23 and 69 us: 393 tiles of 128 words
// are more than the 304 CTAs that are resident, so a second round has 89, and one lane of the joining pass has all 393 parts.
#include "linear_narrow.cuh"

namespace zgb {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

struct VocabParams : ProductParams {
  CUtensorMap w[2 * kGemmMaxPieces];  // as LinearParams', for two heights of any number of shards
  int w_row0;              // the row of W where this launch's columns (dx: contraction) begin
  int splits, slot_rows;   // dx: parts of the contraction, each its own [slot_rows, n] of y32
  bool add;                // dx: to what y32 holds
  int vocab;
  int cols, ld;            // dlogits: columns of y to write (the rest of n is none), and its row distance
  const void* labels;
  int labels_wide;         // 8-byte labels
  float2* part;            // lse: [2 ceil(n / 256)][m]: maximum, sum of exp(z - maximum)
  unsigned int* ticket;    // lse: set to 0 for the kernel that joins the parts
  float* z_label;          // lse: [m]
  const float *lse, *dloss;  // dlogits; dx
};

template <> struct Wide<OP_LSE> {
  using Params = VocabParams;
  static constexpr int EPI_WARPS = 8, EPI_COLS = 128, STAGES = 6, THREADS = 32 * (2 + EPI_WARPS);
  static constexpr uint32_t STAGE = 2 * kHalf, SMEM = STAGES * STAGE + 1024;
};
template <> struct Wide<OP_LSE_PARTS> : Wide<OP_LSE> {};
template <> struct Wide<OP_DLOGITS> {
  using Params = VocabParams;
  static constexpr int EPI_WARPS = 8, EPI_COLS = 128, STAGES = 6, THREADS = 32 * (2 + EPI_WARPS);
  static constexpr uint32_t STAGE = 2 * kHalf, EPI = EPI_WARPS * 4096u, SMEM = STAGES * STAGE + EPI + 1024;
};
template <> struct Wide<OP_DLOGITS_PARTS> : Wide<OP_DLOGITS> {};
template <> struct Wide<OP_DX_SPLIT> {
  using Params = VocabParams;
  static constexpr int EPI_WARPS = 4, EPI_COLS = 256, STAGES = 6, THREADS = 32 * (2 + EPI_WARPS);
  static constexpr uint32_t STAGE = 2 * kHalf, EPI = EPI_WARPS * 8192u, SMEM = STAGES * STAGE + EPI + 1024;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// label i, or -1 where it is none (outside 0 .. vocab - 1): the token is not counted
__device__ __forceinline__ int label_at(const void* labels, int wide, int64_t i, int vocab) {
  const int64_t t = wide ? __ldg(static_cast<const long long*>(labels) + i) : __ldg(static_cast<const int*>(labels) + i);
  return t >= 0 && t < vocab ? static_cast<int>(t) : -1;
}
__device__ __forceinline__ float finite_or_0(float x) { return fabsf(x) < __int_as_float(0x7f800000) ? x : 0.0f; }

// e^d of d = z - maximum (or lse). The difference is made first, and is exact where it is small: the largest term is exactly 1,
// and a token that is all but sure keeps its loss, where z log2 e less a rounded maximum log2 e is off by half a step of the
// maximum (logits of 100: losses of 0 came out between -7.6e-6 and 7.6e-6). It costs an operation a pair: the loss of 8192 x
// 50257 from 768 351 us (347), its gradients 1136 (1120).
__device__ __forceinline__ float exp_fast(float d) { return exp2_fast(__fmul_rn(d, kLog2e)); }

// A row's maximum and sum of exp(z - maximum). An infinite maximum is subtracted as 0: -inf throughout leaves the sum 0,
// +inf makes it infinite, and NaN stays.
struct Softmax {
  float top, sum;
  template <int N>
  __device__ __forceinline__ void join(const float2 (&v)[N]) {
    float t = top;
#pragma unroll
    for (int i = 0; i < N; ++i) t = max_nan(t, v[i].x);
    const float r = finite_or_0(t);
    // a sum of 0 has no terms: its maximum says nothing
    const auto scaled = [&](float s, float m) { return s == 0.0f ? 0.0f : __fmul_rn(s, exp_fast(__fsub_rn(finite_or_0(m), r))); };
    sum = scaled(sum, top);
#pragma unroll
    for (int i = 0; i < N; ++i) sum = __fadd_rn(sum, scaled(v[i].y, v[i].x));
    top = t;
  }
};

// The epilogue warps' role: as in the linear unit, a thread has a row of the tile and a warp 32 rows.
template <int OP>
__device__ __forceinline__ void wide_epilogue(const typename Wide<OP>::Params& p, uint8_t* smem, uint32_t tmem_base,
                                              uint32_t accf_bar, uint32_t acce_bar, volatile int* abort, int warp,
                                              int lane, uint32_t rank, int pair, int pairs, int num_m, int num_n) {
  using C = Wide<OP>;
  const int q = warp & 3;            // the tensor-memory lane quarter this warp may read
  const int part = (warp - 2) >> 2;  // which of the quarter's warps
  // staging: two buffers of 4 KiB a warp for dX, one for dZ (the forward: none)
  uint8_t* stage = smem + C::STAGES * C::STAGE + static_cast<uint32_t>(warp - 2) * (is_dlogits(OP) ? 4096u : 8192u);
  uint32_t i = 0, stores = 0;
  const float scale = OP == OP_DX_SPLIT ? dw_scale(p.scale, p.count) : 1.0f;
  if (is_lse(OP) && pair == 0 && rank == 0 && warp == 2 && lane == 0) *p.ticket = 0u;
  const int tiles = num_m * num_n, items = wide_items<OP>(p, tiles);
  for (int item = pair; item < items; item += pairs) {
    const int part_k = OP == OP_DX_SPLIT ? item / tiles : 0;
    int mb, nb;
    wide_tile_coords(item - part_k * tiles, num_m, num_n, mb, nb);
    const int r0 = mb * 256 + static_cast<int>(rank) * 128 + q * 32, row = r0 + lane;
    const int c0 = nb * 256 + part * C::EPI_COLS;
    // while the products run: the row's label, as a column of this launch
    int target = -1;
    bool counted = false;  // not: dZ and dX are 0, selected and not multiplied, whatever X and W hold
    float lse = 0.0f, own = scale;  // own: dx, of this row
    if (row < p.m) {
      const int label = label_at(p.labels, p.labels_wide, row, p.vocab);
      counted = label >= 0;
      target = counted ? label - p.w_row0 : -1;
      if (is_dlogits(OP) && counted) lse = __ldg(p.lse + row);
      if (OP == OP_DX_SPLIT && counted && p.dloss) own = __fmul_rn(scale, __ldg(p.dloss + row));
    }
    // 32 logits of the row, of columns col0 ..: joined to s
    Softmax s{__int_as_float(0xff800000), 0.0f};
    const auto join_32 = [&](int col0, uint32_t (&r)[32]) {
      if (static_cast<uint32_t>(target - col0) < 32u) {
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) z = target - col0 == j ? __uint_as_float(r[j]) : z;
        p.z_label[row] = z;
      }
      if (col0 + 32 > p.n) {
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = col0 + j < p.n ? r[j] : 0xff800000u;
      }
      float top = __uint_as_float(r[0]);
#pragma unroll
      for (int j = 1; j < 32; ++j) top = max_nan(top, __uint_as_float(r[j]));
      const f2 base = f2_both(-finite_or_0(top));
      f2 sum = 0ull;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float x, y;
        f2_split(f2_mul(f2_add(f2_make(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), base), f2_both(kLog2e)), x, y);
        sum = f2_add(sum, f2_make(exp2_fast(x), exp2_fast(y)));
      }
      float x, y;
      f2_split(sum, x, y);
      s.join({make_float2(top, __fadd_rn(x, y))});
    };
    // ... or written as dZ, at column c of this warp's (the buffer takes two of them)
    const auto put_32 = [&](int c, uint32_t (&r)[32]) {
      const int h = (c >> 5) & 1, col0 = c0 + c;
      uint8_t* buf = stage;
      // few instructions a pair: what concerns single elements (the label's, those past the vocabulary) is
      // put right in the packed words and in the buffer
      uint4 w[4];
      uint32_t* word = reinterpret_cast<uint32_t*>(w);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float x, y;
        f2_split(f2_mul(f2_add(f2_make(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), f2_both(-lse)), f2_both(kLog2e)), x, y);
        word[j >> 1] = f2_to_bf16x2(f2_make(exp2_fast(x), exp2_fast(y)));
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) word[j] = counted ? word[j] : 0u;  // whatever the logits are
      if (col0 + 32 > p.n) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          word[j] = col0 + 2 * j >= p.n ? 0u : col0 + 2 * j + 1 >= p.n ? word[j] & 0xFFFFu : word[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(buf + staged_at(lane, 4 * h + j)) = w[j];
      const int at = target - col0;
      if (static_cast<uint32_t>(at) < 32u) {
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) z = at == j ? __uint_as_float(r[j]) : z;
        const float v = __fsub_rn(exp_fast(__fsub_rn(z, lse)), 1.0f);
        *reinterpret_cast<uint16_t*>(buf + staged_at(lane, 4 * h + (at >> 3)) + 2 * (at & 7)) = f32_to_bf16_bits(v);
      }
      if (h == 1 || col0 + 32 >= p.cols) {
        __syncwarp();
        stage_store(buf, p.y, r0, col0 - 32 * h, p.m, p.cols, p.ld, lane);
      }
    };
    const auto put_part = [&] {
      if (row < p.m && c0 < p.n) p.part[static_cast<size_t>(nb * 2 + part) * p.m + row] = make_float2(s.top, s.sum);
    };
    // relaxed: the arrival only says that the tensor-memory loads are done (ordered by the fence before it)
    const auto drained = [&](uint32_t a) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(acce_bar + 8u * a, 0))
                     : "memory");
    };
    if constexpr (OP == OP_LSE_PARTS || OP == OP_DLOGITS_PARTS) {
      // the row's 128 logits, added up part by part with rounding to nearest: 128 of the 168 registers that ten warps leave a
      // thread, so some spill (bytes stored and loaded a thread: dZ 532 and 564, the loss 40 and 72), once a tile. Half the
      // columns a warp needs sixteen epilogue warps, 112 registers
      f2 z[C::EPI_COLS / 2];
#pragma unroll
      for (int j = 0; j < C::EPI_COLS / 2; ++j) z[j] = 0ull;
      bool stop = false;
#pragma unroll 1
      for (int chunk = 0; chunk < p.chunks; ++chunk, ++i) {
        const uint32_t a = i & 1u, u = i >> 1;
        if (!warp_wait_bounded(accf_bar + 8u * a, u & 1u, abort, kErrAccF)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * 256 + part * C::EPI_COLS;
#pragma unroll
        for (int c = 0; c < C::EPI_COLS; c += 32) {
          uint32_t r[32];
          tmem_ld_32cols(taddr + c, r);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            z[c / 2 + j] = f2_add(z[c / 2 + j], f2_make(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])));
        }
        drained(a);
      }
      if (stop) break;
#pragma unroll
      for (int c = 0; c < C::EPI_COLS; c += 32) {
        if (is_dlogits(OP) && ((c >> 5) & 1) == 0) __syncwarp();  // the buffer's last store has read it
        if (c0 + c >= (is_lse(OP) ? p.n : p.cols)) continue;  // warp-uniform
        uint32_t r[32];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float x, y;
          f2_split(z[c / 2 + j], x, y);
          r[2 * j] = __float_as_uint(x), r[2 * j + 1] = __float_as_uint(y);
        }
        if constexpr (is_lse(OP)) join_32(c0 + c, r);
        else put_32(c, r);
      }
      if constexpr (is_lse(OP)) put_part();
      else __syncwarp();
      continue;
    }
    const uint32_t a = i & 1u, u = i >> 1;
    ++i;
    if (!warp_wait_bounded(accf_bar + 8u * a, u & 1u, abort, kErrAccF)) break;
    tc_fence_after();
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + a * 256 + part * C::EPI_COLS;
    if constexpr (OP == OP_DX_SPLIT) {
      if (p.y32) {
        if (r0 < p.m)
          store_sums<C::EPI_COLS>(&p.out, taddr, part_k * p.slot_rows + r0, c0, p.n, own, p.add, stage, stores, lane, counted);
      } else {
#pragma unroll 1
        for (int c = 0; c < C::EPI_COLS; c += 32) {
          const int h = (c >> 5) & 1, col0 = c0 + c;
          uint8_t* buf = stage + ((c >> 6) & 1) * 4096;
          if (h == 0) __syncwarp();  // the buffer's last store has read it
          uint32_t r[32];
          tmem_ld_32cols(taddr + c, r);
          if (col0 >= p.n) continue;
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = counted ? r[j] : 0u;
          const auto two = [&](int i) {
            return f2_to_bf16x2(f2_mul(f2_make(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), f2_both(own)));
          };
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(buf + staged_at(lane, 4 * h + j)) =
                make_uint4(two(8 * j), two(8 * j + 2), two(8 * j + 4), two(8 * j + 6));
          if (h == 1 || col0 + 32 >= p.n) {
            __syncwarp();
            stage_store(buf, p.y, r0, col0 - 32 * h, p.m, p.n, p.n, lane);
          }
        }
        __syncwarp();
      }
    }
    if constexpr (OP == OP_LSE) {
#pragma unroll 1
      for (int c = 0; c < C::EPI_COLS; c += 32) {
        uint32_t r[32];
        tmem_ld_32cols(taddr + c, r);
        if (c0 + c < p.n) join_32(c0 + c, r);  // warp-uniform
      }
      put_part();
    }
    if constexpr (OP == OP_DLOGITS) {
#pragma unroll 1
      for (int c = 0; c < C::EPI_COLS; c += 32) {
        if (((c >> 5) & 1) == 0) __syncwarp();  // the buffer's last store has read it
        uint32_t r[32];
        tmem_ld_32cols(taddr + c, r);
        if (c0 + c < p.cols) put_32(c, r);  // warp-uniform
      }
      __syncwarp();
    }
    drained(a);
  }
  if (lane == 0) bulk_wait_group_all();  // no store still reads shared memory
}

// ------------------------------------------------------------------------------------
// few tokens: the narrow kernel's epilogue, a row's 128 columns in a warp, 4 a lane
// ------------------------------------------------------------------------------------
struct RowOfLoss {  // loaded while the main loop runs, all lanes the same
  long long label;
  float lse;
  __device__ __forceinline__ void load(const VocabParams& p, int row, int) {
    if (row >= p.m) return;
    if (p.labels_wide) {
      asm volatile("ld.global.nc.s64 %0, [%1];" : "=l"(label) : "l"(static_cast<const long long*>(p.labels) + row));
    } else {
      int l;
      asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(l) : "l"(static_cast<const int*>(p.labels) + row));
      label = l;
    }
    if (p.lse) asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(lse) : "l"(p.lse + row));
  }
};
template <> struct Side4<OP_LSE> : RowOfLoss {};
template <> struct Side4<OP_DLOGITS> : RowOfLoss {};

template <int OP, int ACT>
__device__ __forceinline__ void epilogue4(const typename Wide<OP>::Params& p, int row, int col, uint2, const Side4<OP>& side,
                                          f2 (&v)[2]) {
  float z[4];
  f2_split(v[0], z[0], z[1]);
  f2_split(v[1], z[2], z[3]);
  const bool counted = side.label >= 0 && side.label < p.vocab;
  const int at = counted ? static_cast<int>(side.label) - p.w_row0 - col : -1;  // the label's, of this lane's columns
  if constexpr (OP == OP_LSE) {
    if (row == 0 && col == 0) *p.ticket = 0u;
    if (at >= 0 && at < 4) p.z_label[row] = at == 0 ? z[0] : at == 1 ? z[1] : at == 2 ? z[2] : z[3];
    float top = __int_as_float(0xff800000);
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = col + j < p.n ? z[j] : __int_as_float(0xff800000), top = max_nan(top, z[j]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float base = finite_or_0(top);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum = __fadd_rn(sum, exp_fast(__fsub_rn(z[j], base)));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
    if ((threadIdx.x & 31) == 0) p.part[static_cast<size_t>(col >> 7) * p.m + row] = make_float2(top, sum);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float e = exp_fast(__fsub_rn(z[j], side.lse));
      z[j] = counted && col + j < p.n ? (at == j ? __fsub_rn(e, 1.0f) : e) : 0.0f;
    }
    if (col < p.cols)
      *reinterpret_cast<uint2*>(p.y + static_cast<size_t>(row) * p.ld + col) =
          make_uint2(f2_to_bf16x2(f2_make(z[0], z[1])), f2_to_bf16x2(f2_make(z[2], z[3])));
  }
}

// lse and loss from the parts of a row: a block takes 32 rows, its warps the parts in turn, kAtOnce of them in
// flight; their largest maximum is found first. With total, a block also leaves its rows' sum of losses and count,
// and the block that comes last (a ticket, left at 0 by the product before) adds them, in the order of the
// blocks.
constexpr int kThreads = 256;
constexpr int kJoinWarps = 16, kAtOnce = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) join_parts_kernel(const float2* __restrict__ part, int parts, int m,
                                                                     const float* __restrict__ z_label, const void* labels,
                                                                     int wide, int vocab, float* __restrict__ loss,
                                                                     float* __restrict__ lse, float2* __restrict__ block_total,
                                                                     unsigned int* ticket, float* __restrict__ total) {
  __shared__ float2 meet[kJoinWarps][32];
  __shared__ bool last;
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const float none = __int_as_float(0xff800000);
  Softmax s{none, 0.0f};
  if (row < m)
    for (int i0 = warp; i0 < parts; i0 += kJoinWarps * kAtOnce) {
      float2 v[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * kJoinWarps;
        v[j] = i < parts ? part[static_cast<size_t>(i) * m + row] : make_float2(none, 0.0f);
      }
      s.join(v);
    }
  meet[warp][lane] = make_float2(s.top, s.sum);
  __syncthreads();
  if (warp == 0) {
    float2 v[kJoinWarps];
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) v[w] = meet[w][lane];
    s = {none, 0.0f};
    s.join(v);
    float mine = 0.0f;
    int count = 0;
    if (row < m) {
      // the loss not from lse, which is rounded to the size of the logits: neither of its terms is below 0
      const float log2_sum = log2f(s.sum), top = finite_or_0(s.top);
      count = label_at(labels, wide, row, vocab) >= 0 ? 1 : 0;
      mine = count ? __fmaf_rn(log2_sum, kLn2, __fsub_rn(top, z_label[row])) : 0.0f;
      lse[row] = __fmaf_rn(log2_sum, kLn2, top), loss[row] = mine;
    }
    if (total) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        mine = __fadd_rn(mine, __shfl_xor_sync(0xffffffffu, mine, d));
        count += __shfl_xor_sync(0xffffffffu, count, d);
      }
      if (lane == 0) {
        block_total[blockIdx.x] = make_float2(mine, __int_as_float(count));
        __threadfence();
        last = atomicAdd(ticket, 1u) + 1u == gridDim.x;
      }
    }
  }
  if (!total) return;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float sum = 0.0f, lost = 0.0f;  // a thread keeps what its additions round off, as long as the sum is finite
  int count = 0;
  for (int64_t i = threadIdx.x; i < gridDim.x; i += 32 * kJoinWarps) {
    const float2 v = __ldcg(block_total + i);
    const float x = __fsub_rn(v.x, lost), t = __fadd_rn(sum, x);
    lost = finite_or_0(__fsub_rn(__fsub_rn(t, sum), x));
    sum = t;
    count += __float_as_int(v.y);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
    count += __shfl_xor_sync(0xffffffffu, count, d);
  }
  if (lane == 0) meet[0][warp] = make_float2(sum, __int_as_float(count));
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kJoinWarps; ++w) sum = __fadd_rn(sum, meet[0][w].x), count += __float_as_int(meet[0][w].y);
    total[0] = sum, total[1] = static_cast<float>(count);
  }
}

// dX = bf16 of the sum of `slots` parts, in order
__global__ void __launch_bounds__(kThreads) sum_slots_kernel(const float* __restrict__ slot, int slots, int64_t slot_elems,
                                                             int64_t n8, uint16_t* __restrict__ dx) {
  allow_next_grid();
  wait_for_prior_grids();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n8; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    f2 v[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 4
    for (int s = 0; s < slots; ++s) {
      const ulonglong2* a = reinterpret_cast<const ulonglong2*>(slot + s * slot_elems + 8 * i);
      const ulonglong2 x = a[0], y = a[1];
      v[0] = f2_add(v[0], x.x), v[1] = f2_add(v[1], x.y), v[2] = f2_add(v[2], y.x), v[3] = f2_add(v[3], y.y);
    }
    reinterpret_cast<uint4*>(dx)[i] =
        make_uint4(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]), f2_to_bf16x2(v[2]), f2_to_bf16x2(v[3]));
  }
}

// c g X in bf16, a warp up to 1024 columns of a row, as many pieces of 8 as it has lanes at once; zeros where the token is
// not counted. Latency: 3 us of a call (100 x 4096).
constexpr int kWeighPieces = 128;
__global__ void __launch_bounds__(kThreads) weigh_rows_kernel(const uint16_t* __restrict__ x, int m, int pieces, const void* labels,
                                                              int wide, int vocab, const float* __restrict__ dloss, float scale,
                                                              const float* count, uint16_t* __restrict__ out) {
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  const float c = dw_scale(scale, count);
  const int64_t slices = (pieces + kWeighPieces - 1) / kWeighPieces, items = m * slices;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); item < items;
       item += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
    const int64_t row = item / slices;
    const int first = static_cast<int>(item - row * slices) * kWeighPieces, last = min(first + kWeighPieces, pieces);
    const bool counted = label_at(labels, wide, row, vocab) >= 0;
    const f2 w = f2_both(__fmul_rn(c, __ldg(dloss + row)));
    const uint4* from = reinterpret_cast<const uint4*>(x) + row * pieces;
    uint4* to = reinterpret_cast<uint4*>(out) + row * pieces;
#pragma unroll 4
    for (int j = first + lane; j < last; j += 32) {
      f2 v[4];
      unpack8(__ldg(from + j), v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = counted ? f2_mul(v[i], w) : 0ull;
      to[j] = make_uint4(f2_to_bf16x2(v[0]), f2_to_bf16x2(v[1]), f2_to_bf16x2(v[2]), f2_to_bf16x2(v[3]));
    }
  }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
uint64_t up256(uint64_t n) { return (n + 255) & ~uint64_t(255); }

// The tensor cores add to an accumulator with truncation, about 2^-24 of it a step and always toward zero. The loss is
// an fp32 result, so its logits are summed in parts of 16 K blocks (1024 elements), which are added with rounding
// to nearest: at 8192 elements lse is 6.4e-6 of itself off in one part, 3.3e-7 in eight, at 1024 3.6e-7 (8192 x 32000
// from 4096: 1077 us in one part, 1135 in four). The backward's logits are summed the same way: they have to be the
// forward's, bit for bit, for exp(Z - lse) to add up to 1, or what is left of a sure token's gradient is wrong.
constexpr int kPartBlocks = 16;

// W as the launches see it: the shards that hold rows of the vocabulary
struct Weights {
  int n, shard_rows;
  const uint16_t* w[kGemmMaxPieces];
};

// Shards for which there would be one height of copies only, that of 8 rows for a vocabulary of odd size, in 16 maps: the
// lowest and the highest, in up to 32, where they are long enough to be cut at few of the tiles (16 shards, in one height:
// 8192 of 50257 x 768 353 us (455-497), gradients 1.15-1.18 ms (1.57); 2000 of 4900 x 768, 312 rows a shard, 29 (33), of
// 2700 x 768, 176 rows, 21.6 (19.7)). Up to 8 shards, 16 maps do as well.
bool long_shards(const Weights& w) { return w.n > kGemmMaxPieces / 2 && w.shard_rows >= 256; }

template <int OP>
int launch_product(VocabParams& p, const Weights& w, bool one_copy, cudaStream_t st, const char* who) {
  p.shard_rows = w.shard_rows;
  const int blocks = (p.k + BK - 1) / BK;
  p.chunk_blocks = OP == OP_LSE_PARTS || OP == OP_DLOGITS_PARTS ? kPartBlocks : blocks;
  p.chunks = (blocks + p.chunk_blocks - 1) / p.chunk_blocks;
  int rc;
  // a vocabulary's shards are long: copies as high as they can be, cut at the few places where a shard ends
  const bool fwd = OP != OP_DX_SPLIT;
  if ((rc = encode_w(p, w.n, w.w, p.vocab, fwd, fwd ? 128 : BK, long_shards(w), &one_copy, who))) return rc;
  if (p.w_levels > 1) return launch_wide<OP, COPIES_CUT>(p, st, who);
  return one_copy ? launch_wide<OP, COPIES_ONE>(p, st, who) : launch_wide<OP, COPIES_EQUAL>(p, st, who);
}

template <int OP, int TN>
int launch_few(const VocabParams& p, int splits, cudaStream_t st, const char* who) {
  return p.w_levels > 1 ? launch_narrow<OP, TN, true>(p, splits, st, who) : launch_narrow<OP, TN, false>(p, splits, st, who);
}

// X's logits (p.a's map is set here too). The kernel follows from m, the whole vocabulary and k, so that the forward and
// each of the backward's pieces sum alike. The narrow kernel (wide in brackets, us) for up to 32 tokens: one of 50257 x
// 768 21 (28), of 32000 x 4096 45 (77), 16 of 131072 x 1024 55 (58); for up to 64 while its tiles are resident at once:
// 64 of 32000 x 4096 48 (55), but of 50257 x 2048 48 (46); and where so few that the contraction is split: 100 of 2000 x
// 4096 13 (27), 256 of 1157 x 520 12.1 (12.4), unsplit 1003 of 1157 x 520 14.8 (12.8), 128 of 32000 x 4096 62 (55).
template <int OP, int OP_PARTS>
int launch_logits(VocabParams& p, const Weights& w, const zero_bf16* x, cudaStream_t st, const char* who) {
  int rc;
  const int blocks = (p.k + BK - 1) / BK;
  Choice c = choose(OP_FWD, p.m, p.vocab, p.k, false);
  const bool resident = (p.vocab + 127) / 128 <= 2 * num_sms();
  c.wide = c.wide || (c.splits == 1 && p.m > (resident ? 64 : 32));
  // its accumulators and splits have to make parts of kPartBlocks
  while (!c.wide && (blocks + c.splits - 1) / c.splits > kPartBlocks * (kLogitCols / c.tn)) {
    c.splits *= 2;
    c.wide = c.splits > (c.tn == 128 ? 4 : 8);
  }
  if ((rc = encode(&p.a, x, p.m, p.k, p.k, BK, c.wide ? 128 : c.tn, false, who))) return rc;
  if (c.wide) return blocks > kPartBlocks ? launch_product<OP_PARTS>(p, w, true, st, who) : launch_product<OP>(p, w, true, st, who);
  bool one_copy = false;
  p.shard_rows = w.shard_rows, p.chunk_blocks = kPartBlocks;
  if ((rc = encode_w(p, w.n, w.w, p.vocab, true, kCutFrom, long_shards(w), &one_copy, who))) return rc;
  return c.tn == 32   ? launch_few<OP, 32>(p, c.splits, st, who)
         : c.tn == 64 ? launch_few<OP, 64>(p, c.splits, st, who)
                      : launch_few<OP, 128>(p, c.splits, st, who);
}

// The backward's pieces and its workspace: dZ of a piece [m, ld], c g X, and where dX is summed in parts, those.
// The default piece is as much of the vocabulary as a dZ of kPieceBytes holds: each piece is three launches,
// and more of them than one share dX through memory.
constexpr uint64_t kPieceBytes = uint64_t(1) << 30;
struct BackwardPlan {
  int64_t piece, pieces, ld, slot_rows;
  int splits;      // of dX's contraction over a piece
  bool slots;      // dX is summed in slots, else written by the product
  uint64_t x_at, slots_at, bytes;
  BackwardPlan(int64_t m, int64_t vocab, int64_t k, int64_t asked) {
    piece = asked;
    if (piece == 0) {
      const int64_t most = std::max<int64_t>(256, static_cast<int64_t>(kPieceBytes / (2 * static_cast<uint64_t>(m))) / 256 * 256);
      const int64_t n = (vocab + most - 1) / most;
      piece = ((vocab + n - 1) / n + 255) / 256 * 256;
    }
    pieces = (vocab + piece - 1) / piece;
    ld = std::min(piece, (vocab + 63) / 64 * 64);
    // splits: each pair of SMs takes whole (tile, part) items, so the time is the rounds times a part's K
    // blocks, and the parts' way through memory (256 KB a tile and part, out and in, against 0.34 us a block)
    const int64_t tiles = ((m + 255) / 256) * ((k + 255) / 256), pairs = std::max(1, num_sms() / 2);
    const int64_t blocks = (std::min(piece, vocab) + BK - 1) / BK;
    slot_rows = (m + 31) / 32 * 32;
    double best = 0.0;
    splits = 1;
    for (int s = 1; s <= 32 && s <= blocks && s * slot_rows <= INT32_MAX; ++s) {
      const int64_t rounds = (tiles * s + pairs - 1) / pairs;
      const double t = static_cast<double>(rounds) * (static_cast<double>((blocks + s - 1) / s) + 4.0) +
                       (s > 1 || pieces > 1 ? 0.25 * static_cast<double>(tiles * (s + 0.5)) + 8.0 : 0.0);
      if (s == 1 || t < best) best = t, splits = s;
    }
    slots = splits > 1 || pieces > 1;
    x_at = up256(2 * static_cast<uint64_t>(m) * static_cast<uint64_t>(ld));
    slots_at = x_at + up256(2 * static_cast<uint64_t>(m) * static_cast<uint64_t>(k));
    bytes = slots_at + (slots ? up256(4 * static_cast<uint64_t>(splits) * static_cast<uint64_t>(slot_rows) * static_cast<uint64_t>(k)) : 0);
  }
};

int check_sizes(int64_t m, int64_t rows, int64_t vocab, int64_t k, int label_bytes, const char* who) {
  const int64_t most = 1 << 30;
  if (m < 1 || rows < 1 || k < 1 || m > most || rows > most || k > most)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: m_tokens, rows_out and k_in must be in 1..2^30", who);
  if (k % 8) return set_error(ZERO_ERR_INVALID_ARG, "%s: k_in %lld must be a multiple of 8 (16-byte rows)", who, (long long)k);
  if (vocab < 1 || vocab > rows)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: vocab %lld outside 1..%lld (the rows of W)", who, (long long)vocab, (long long)rows);
  if (label_bytes != 4 && label_bytes != 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: label_bytes %d is not 4 or 8", who, label_bytes);
  if (((m + 255) / 256) * ((vocab + 255) / 256) > (1 << 30))
    return set_error(ZERO_ERR_UNSUPPORTED, "%s: logits of %lld x %lld are more than 2^30 tiles", who, (long long)m, (long long)vocab);
  return ZERO_OK;
}

int check_shards(Weights* out, int n, const zero_bf16* const w_shards[], int64_t rows, int64_t vocab, const char* who) {
  if (n < 1 || n > kGemmMaxPieces)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: n_ranks %d outside 1..%d", who, n, kGemmMaxPieces);
  if (rows % n || (rows / n) % 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: rows_out / n_ranks (%lld / %d) must be a multiple of 8", who, (long long)rows, n);
  if (!w_shards) return set_error(ZERO_ERR_INVALID_ARG, "%s: w_shards is NULL", who);
  for (int q = 0; q < n; ++q) {
    if (!w_shards[q]) return set_error(ZERO_ERR_INVALID_ARG, "%s: w_shards[%d] is NULL (missing rank)", who, q);
    if (!aligned16(w_shards[q]))
      return set_error(ZERO_ERR_INVALID_ARG, "%s: w_shards[%d] must be 16-byte aligned", who, q);
    out->w[q] = w_shards[q];
  }
  out->shard_rows = static_cast<int>(rows / n);
  out->n = static_cast<int>((vocab + out->shard_rows - 1) / out->shard_rows);
  return ZERO_OK;
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

}  // namespace

unsigned int fsdp_vocab_loss_read_clear_error() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_zgb_dev_error, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (v) cudaMemcpyToSymbol(g_zgb_dev_error, &zero, sizeof(zero));
  return v;
}

}  // namespace zgb

using namespace zgb;

// The forward's workspace: the parts of each row, the labels' logits, the blocks' totals and their ticket
namespace {
struct ForwardSpace {
  int parts;
  uint64_t z_label, totals, ticket, bytes;
  ForwardSpace(int64_t m, int64_t vocab) {
    parts = static_cast<int>((vocab + 127) / 128);  // 128 columns each
    z_label = up256(8 * static_cast<uint64_t>(parts) * static_cast<uint64_t>(m));
    totals = z_label + up256(4 * static_cast<uint64_t>(m));
    ticket = totals + up256(8 * static_cast<uint64_t>((m + 31) / 32));
    bytes = ticket + 256;
  }
};
}  // namespace

extern "C" int fsdp_vocab_loss_forward_workspace(int64_t m_tokens, int64_t vocab, uint64_t* bytes) {
  const char* who = "fsdp_vocab_loss_forward_workspace";
  if (!bytes) return set_error(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  const int rc = check_sizes(m_tokens, vocab, vocab, 8, 4, who);
  if (rc) return rc;
  *bytes = ForwardSpace(m_tokens, vocab).bytes;
  return ZERO_OK;
}

extern "C" int fsdp_vocab_loss_forward(int n_ranks, const zero_bf16* const w_shards[], int64_t rows_out, int64_t vocab,
                                       int64_t k_in, const zero_bf16* X, int64_t m_tokens, const void* labels,
                                       int label_bytes, float* loss, float* lse, float* total, void* workspace,
                                       uint64_t workspace_bytes, zero_stream_t stream) {
  const char* who = "fsdp_vocab_loss_forward";
  int rc;
  if ((rc = check_sizes(m_tokens, rows_out, vocab, k_in, label_bytes, who))) return rc;
  Weights w;
  if ((rc = check_shards(&w, n_ranks, w_shards, rows_out, vocab, who))) return rc;
  if (!X || !labels || !loss || !lse) return set_error(ZERO_ERR_INVALID_ARG, "%s: X, labels, loss or lse is NULL", who);
  if (!aligned16(X) || !aligned16(workspace))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: X and workspace must be 16-byte aligned", who);
  if (!aligned(labels, label_bytes) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(total, 4))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: labels, loss, lse and total must be aligned to their elements", who);
  const ForwardSpace sp(m_tokens, vocab);
  if (!workspace || workspace_bytes < sp.bytes)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                     workspace ? (unsigned long long)workspace_bytes : 0ull, (unsigned long long)sp.bytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  VocabParams p;
  memset(static_cast<void*>(&p), 0, sizeof(p));
  p.m = static_cast<int>(m_tokens), p.n = static_cast<int>(vocab), p.k = static_cast<int>(k_in);
  p.vocab = p.n, p.labels = labels, p.labels_wide = label_bytes == 8;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part = static_cast<float2*>(workspace);
  p.z_label = reinterpret_cast<float*>(ws + sp.z_label);
  p.ticket = reinterpret_cast<unsigned int*>(ws + sp.ticket);
  if ((rc = launch_logits<OP_LSE, OP_LSE_PARTS>(p, w, X, st, who))) return rc;
  const cudaError_t e =
      launch_overlapped(join_parts_kernel, dim3(static_cast<unsigned>((m_tokens + 31) / 32)), dim3(32 * kJoinWarps), 0, 1, st, p.part,
                        sp.parts, p.m, p.z_label, labels, p.labels_wide, p.vocab, loss, lse,
                        reinterpret_cast<float2*>(ws + sp.totals), p.ticket, total);
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

namespace {
int check_piece(int64_t piece, const char* who) {
  if (piece < 0 || piece % 256 || piece > (1 << 30))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: piece %lld must be 0 or a multiple of 256 up to 2^30", who, (long long)piece);
  return ZERO_OK;
}
}  // namespace

extern "C" int fsdp_vocab_loss_backward_workspace(int64_t m_tokens, int64_t vocab, int64_t k_in, int64_t piece,
                                                  uint64_t* bytes) {
  const char* who = "fsdp_vocab_loss_backward_workspace";
  if (!bytes) return set_error(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  int rc;
  if ((rc = check_sizes(m_tokens, vocab, vocab, k_in, 4, who)) || (rc = check_piece(piece, who))) return rc;
  *bytes = BackwardPlan(m_tokens, vocab, k_in, piece).bytes;
  return ZERO_OK;
}

extern "C" int fsdp_vocab_loss_backward(int n_ranks, const zero_bf16* const w_shards[], int64_t rows_out, int64_t vocab,
                                        int64_t k_in, const zero_bf16* X, int64_t m_tokens, const void* labels,
                                        int label_bytes, const float* lse, const float* dloss, const float* total,
                                        float scale, zero_bf16* dX, zero_bf16* dW, int64_t piece, void* workspace,
                                        uint64_t workspace_bytes, zero_stream_t stream) {
  const char* who = "fsdp_vocab_loss_backward";
  int rc;
  if ((rc = check_sizes(m_tokens, rows_out, vocab, k_in, label_bytes, who)) || (rc = check_piece(piece, who))) return rc;
  Weights w;
  if ((rc = check_shards(&w, n_ranks, w_shards, rows_out, vocab, who))) return rc;
  if (!X || !labels || !lse) return set_error(ZERO_ERR_INVALID_ARG, "%s: X, labels or lse is NULL", who);
  if (!dX && !dW) return set_error(ZERO_ERR_INVALID_ARG, "%s: dX and dW are both NULL", who);
  if (!(scale - scale == 0.0f)) return set_error(ZERO_ERR_INVALID_ARG, "%s: scale must be finite", who);
  if (!aligned16(X) || !aligned16(dX) || !aligned16(dW) || !aligned16(workspace))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: X, dX, dW and workspace must be 16-byte aligned", who);
  if (!aligned(labels, label_bytes) || !aligned(lse, 4) || !aligned(dloss, 4) || !aligned(total, 4))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: labels, lse, dloss and total must be aligned to their elements", who);
  const BackwardPlan plan(m_tokens, vocab, k_in, piece);
  if (!workspace || workspace_bytes < plan.bytes)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                     workspace ? (unsigned long long)workspace_bytes : 0ull, (unsigned long long)plan.bytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint16_t* dz = static_cast<uint16_t*>(workspace);
  float* slots = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.slots_at);
  uint16_t* xw = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + plan.x_at);
  const int m = static_cast<int>(m_tokens), k = static_cast<int>(k_in), ld = static_cast<int>(plan.ld);
  const float* count = total ? total + 1 : nullptr;
  cudaError_t e = cudaSuccess;
  if (dW && rows_out > vocab)  // the padding's rows
    e = cudaMemsetAsync(dW + vocab * k_in, 0, static_cast<size_t>(rows_out - vocab) * static_cast<size_t>(k_in) * 2, st);
  if (e != cudaSuccess) return set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  if (dW && dloss) {
    const int64_t items = m_tokens * ((k / 8 + kWeighPieces - 1) / kWeighPieces);
    const int64_t blocks = std::min<int64_t>((items + kThreads / 32 - 1) / (kThreads / 32), static_cast<int64_t>(num_sms()) * 8);
    e = launch_overlapped(weigh_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, 1, st, X, m, k / 8, labels,
                          label_bytes == 8 ? 1 : 0, static_cast<int>(vocab), dloss, scale, count, xw);
    if (e != cudaSuccess) return set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  for (int64_t c0 = 0; c0 < vocab; c0 += plan.piece) {
    const int cols = static_cast<int>(std::min(plan.piece, vocab - c0));
    VocabParams p;
    memset(static_cast<void*>(&p), 0, sizeof(p));
    p.m = m, p.n = cols, p.k = k;
    p.w_row0 = static_cast<int>(c0), p.vocab = static_cast<int>(vocab);
    p.cols = (cols + 7) / 8 * 8, p.ld = ld, p.y = dz;
    p.labels = labels, p.labels_wide = label_bytes == 8;
    p.lse = lse;
    if ((rc = launch_logits<OP_DLOGITS, OP_DLOGITS_PARTS>(p, w, X, st, who))) return rc;
    if (dW && (rc = dloss ? launch_linear_dw(dz, ld, xw, m, cols, k, 1.0f, nullptr, dW + c0 * k_in, st, who)
                          : launch_linear_dw(dz, ld, X, m, cols, k, scale, count, dW + c0 * k_in, st, who)))
      return rc;
    if (!dX) continue;
    VocabParams d;
    memset(static_cast<void*>(&d), 0, sizeof(d));
    d.m = m, d.n = k, d.k = cols;
    d.w_row0 = p.w_row0, d.vocab = p.vocab, d.scale = scale, d.count = count;
    d.labels = labels, d.labels_wide = p.labels_wide, d.dloss = dloss;
    // a shorter last piece may have fewer K blocks than there are parts: a part has one at least
    d.splits = static_cast<int>(std::min<int64_t>(plan.splits, (cols + BK - 1) / BK));
    d.slot_rows = static_cast<int>(plan.slot_rows), d.add = c0 > 0;
    if (plan.slots) d.y32 = slots;
    else d.y = dX;
    if ((rc = encode(&d.a, dz, m, cols, ld, BK, 128, false, who))) return rc;
    if (plan.slots && (rc = encode(&d.out, slots, plan.splits * plan.slot_rows, k, k, 32, 32, true, who))) return rc;
    if ((rc = launch_product<OP_DX_SPLIT>(d, w, true, st, who))) return rc;
  }
  if (dX && plan.slots) {
    const int64_t n8 = m_tokens * k_in / 8;
    const int64_t blocks = std::min<int64_t>((n8 + kThreads - 1) / kThreads, static_cast<int64_t>(num_sms()) * 16);
    e = launch_overlapped(sum_slots_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, 1, st, slots, plan.splits,
                          plan.slot_rows * k_in, n8, dX);
  }
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}
