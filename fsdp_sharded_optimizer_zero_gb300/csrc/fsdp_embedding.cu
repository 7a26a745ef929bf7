// Token embedding from a table held as row shards, and its gradient.
//
//   forward   Y[i] = scale E[t_i]
//   backward  dE[v] = scale * sum over i with t_i = v of dY[i], every row of dE (or added to it)
//
// The backward brings the rows of one token together, in the order of their positions, and sums them in registers
// in that order, without atomics: the same bits every call. Up to 4096 tokens each block looks for its rows' tokens
// itself, in one launch; more are ordered by a stable sort. Bound by writing dE (8192 tokens of 50257 x 768 fp32: 39 us,
// 23 of them the 154 MB of dE, beside which the sort runs, then 16 the latency of the two launches that sum; 4096
// tokens 33 us) and by the rows of dY (65536 tokens: 65 us, 3.9 TB/s). A token outside 0 .. vocab - 1 is none:
// zeros, no gradient.
#include <algorithm>

#include "linear_math.cuh"

namespace zgb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct TableShards {
  const uint16_t* p[16];
};

__device__ __forceinline__ void widen8(const uint4& w, f2 (&x)[4]) {
  x[0] = f2_from_bf16x2(w.x), x[1] = f2_from_bf16x2(w.y), x[2] = f2_from_bf16x2(w.z), x[3] = f2_from_bf16x2(w.w);
}
__device__ __forceinline__ uint4 narrow8(const f2 (&x)[4]) {
  return make_uint4(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]), f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
}
// token i, or -1 where it is none
__device__ __forceinline__ int token_at(const void* tokens, int wide, int64_t i, int vocab) {
  const int64_t t = wide ? __ldg(static_cast<const long long*>(tokens) + i) : __ldg(static_cast<const int*>(tokens) + i);
  return t >= 0 && t < vocab ? static_cast<int>(t) : -1;
}

// tokens i0, i0 + 32, .. below m (-1 behind), all on their way at once: a branch on their width at each would wait for
// one after the other
template <int N>
__device__ __forceinline__ void tokens_at(const void* tokens, int wide, int64_t i0, int64_t m, int vocab, int (&t)[N]) {
  int64_t raw[N];
  if (wide) {
#pragma unroll
    for (int j = 0; j < N; ++j) raw[j] = i0 + 32 * j < m ? __ldg(static_cast<const long long*>(tokens) + i0 + 32 * j) : -1;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) raw[j] = i0 + 32 * j < m ? __ldg(static_cast<const int*>(tokens) + i0 + 32 * j) : -1;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) t[j] = raw[j] >= 0 && raw[j] < vocab ? static_cast<int>(raw[j]) : -1;
}

// A warp takes up to 1024 columns of a token's row at a time: four pieces of 8 columns a lane, in flight together.
// Bound by HBM, less what tokens that come again find in L2: 8192 tokens of 32000 x 4096 15.9 us (134 MB, 8.4 TB/s);
// one token of 768 columns 1.4 us.
constexpr int kPieces = 4;
__global__ void __launch_bounds__(kThreads) embedding_forward_kernel(const __grid_constant__ TableShards e, int shard_rows,
                                                                     int vocab, int64_t cols, const void* tokens, int wide,
                                                                     int64_t m, int slices, float scale,
                                                                     uint16_t* __restrict__ y) {
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t items = m * slices, step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items; item += step) {
    const int64_t i = item / slices, col0 = (item - i * slices) * (kPieces * 256) + lane * 8;
    const int t = token_at(tokens, wide, i, vocab);
    const int shard = t < 0 ? 0 : t / shard_rows;
    const uint16_t* row = e.p[shard] + (t < 0 ? 0 : static_cast<int64_t>(t - shard * shard_rows) * cols);
    uint4 w[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      if (t >= 0 && col0 + u * 256 < cols) w[u] = __ldg(reinterpret_cast<const uint4*>(row + col0 + u * 256));
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if (col0 + u * 256 >= cols) continue;
      f2 v[4];
      widen8(w[u], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = t < 0 ? 0ull : f2_mul(v[j], f2_both(scale));
      __stcs(reinterpret_cast<uint4*>(y + i * cols + col0 + u * 256), narrow8(v));
    }
  }
}

// ------------------------------------------------------------------------------------
// positions in order of their tokens
// ------------------------------------------------------------------------------------
constexpr int kNone = 0x7fffffff;  // key of a position without a token: behind all others
struct Sorted {
  int* key;    // [m] tokens in order
  int* order;  // [m] their positions
};

// zeros to `n16` pieces of 16 bytes, by block `block` of `blocks`
__device__ __forceinline__ void fill_zeros(uint4* out, int64_t n16, int64_t block, int64_t blocks) {
  for (int64_t i = block * blockDim.x + threadIdx.x; i < n16; i += blocks * blockDim.x) __stcs(out + i, make_uint4(0u, 0u, 0u, 0u));
}

// More than kFewTokens: a stable radix sort, a digit of kDigitBits a pass from the lowest, in two or three launches a
// pass. Block b has the positions from b kSortTile on, a warp a run of them. They are few blocks: the others of each
// launch fill a share of dE with zeros.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kSortTile = 2048, kSortRun = kSortTile / kSortWarps, kSortRounds = kSortRun / 32;
struct SortPass {
  const void* tokens;  // first pass: the tokens themselves; else null
  int wide, vocab, shift;
  Sorted in, out;
  int64_t m;
  int blocks;
  int* count;  // [blocks][kDigits]; scanned: [kDigits][blocks], the places where they begin
  bool scanned;
  uint4* zero;  // this launch's share to fill
  int64_t zero16;
};
// positions without a token have the digits of `vocab`, which no token has: behind the others
__device__ __forceinline__ int sort_digit(const SortPass& p, int key) {
  return (min(key, p.vocab) >> p.shift) & (kDigits - 1);
}
// the keys of a lane's positions of its warp's run, all on their way at once
__device__ __forceinline__ void load_keys(const SortPass& p, int64_t first, int (&key)[kSortRounds], int (&digit)[kSortRounds]) {
  if (p.tokens) {
    tokens_at(p.tokens, p.wide, first, p.m, p.vocab, key);
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) key[r] = key[r] < 0 ? kNone : key[r];
  } else {
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) key[r] = first + r * 32 < p.m ? p.in.key[first + r * 32] : kNone;
  }
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) digit[r] = first + r * 32 < p.m ? sort_digit(p, key[r]) : -1;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortPass p) {
  __shared__ int count[kDigits];
  allow_next_grid();
  wait_for_prior_grids();
  if (static_cast<int>(blockIdx.x) >= p.blocks) {
    fill_zeros(p.zero, p.zero16, blockIdx.x - p.blocks, gridDim.x - p.blocks);
    return;
  }
  int key[kSortRounds], digit[kSortRounds];
  load_keys(p, static_cast<int64_t>(blockIdx.x) * kSortTile + (threadIdx.x >> 5) * kSortRun + (threadIdx.x & 31), key, digit);
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) count[d] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    if (digit[r] >= 0) atomicAdd(&count[digit[r]], 1);
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads)
    p.count[p.scanned ? static_cast<int64_t>(d) * p.blocks + blockIdx.x : static_cast<int64_t>(blockIdx.x) * kDigits + d] = count[d];
}

// exclusive sums over all of count, in place, by one block: where there are so many blocks that each of them cannot
// add up the others' counts itself. One block is slow at that, 4096 counts a round: 262144 tokens into 50257 x 768 fp32 take
// 199 us (floor 82), 1048576 641 (261); without it 131072 take 98 (53).
constexpr int kOwnScan = 64;
__global__ void __launch_bounds__(1024) sort_scan_kernel(int* count, int64_t n) {
  __shared__ int warp_sum[32];
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int base = 0;
  for (int64_t i0 = 0; i0 < n; i0 += 4096) {
    const int64_t i = i0 + static_cast<int64_t>(threadIdx.x) * 4;
    int v[4], mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? count[i + j] : 0, mine += v[j];
    int run = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int t = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += t;
    }
    __syncthreads();  // the last round's sums have been read
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    int ahead = 0, all = 0;
    for (int w = 0; w < 32; ++w) ahead += w < warp ? warp_sum[w] : 0, all += warp_sum[w];
    int at = base + ahead + run - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i + j < n) count[i + j] = at;
      at += v[j];
    }
    base += all;
  }
}

// A warp finds each position's place among its own of the same digit: those ahead of it in its round of 32, and
// those of earlier rounds, which next[digit] counts. The lanes of the same digit are found by a vote for each of its
// bits.
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const SortPass p) {
  static_assert(kDigits == kSortThreads, "a thread a digit");
  __shared__ int next[kSortWarps][kDigits];  // per warp: counts, then where its positions of a digit go
  __shared__ int warp_sum[kSortWarps];
  allow_next_grid();
  wait_for_prior_grids();
  if (static_cast<int>(blockIdx.x) >= p.blocks) {
    fill_zeros(p.zero, p.zero16, blockIdx.x - p.blocks, gridDim.x - p.blocks);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSortTile + warp * kSortRun + lane;
  int key[kSortRounds], digit[kSortRounds], order[kSortRounds], place[kSortRounds];
  load_keys(p, first, key, digit);
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) order[r] = static_cast<int>(first + r * 32);
  if (!p.tokens) {
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) order[r] = first + r * 32 < p.m ? p.in.order[first + r * 32] : 0;
  }
  // where this block's positions of digit threadIdx.x begin
  int begin = 0;
  if (p.scanned) {
    begin = p.count[static_cast<int64_t>(threadIdx.x) * p.blocks + blockIdx.x];
  } else {
    int all = 0;
#pragma unroll 16
    for (int b = 0; b < p.blocks; ++b) {
      const int n = p.count[b * kDigits + static_cast<int>(threadIdx.x)];
      begin += b < static_cast<int>(blockIdx.x) ? n : 0;
      all += n;
    }
    int run = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int t = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += t;
    }
    if (lane == 31) warp_sum[warp] = run;
    begin += run - all;
  }
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) next[w][threadIdx.x] = 0;
  __syncthreads();
  if (!p.scanned)
    for (int w = 0; w < warp; ++w) begin += warp_sum[w];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    uint32_t same = __ballot_sync(0xffffffffu, digit[r] >= 0);  // a digit of -1: no position
#pragma unroll
    for (int bit = 0; bit < kDigitBits; ++bit) {
      const bool one = (digit[r] >> bit) & 1;
      const uint32_t ones = __ballot_sync(0xffffffffu, one);
      same &= one ? ones : ~ones;
    }
    const int ahead = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (digit[r] >= 0) at = next[warp][digit[r]];
    __syncwarp();
    if (digit[r] >= 0 && ahead == 0) next[warp][digit[r]] = at + __popc(same);
    __syncwarp();
    place[r] = at + ahead;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    const int n = next[w][threadIdx.x];
    next[w][threadIdx.x] = begin;
    begin += n;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    if (digit[r] >= 0) {
      const int at = next[warp][digit[r]] + place[r];
      p.out.key[at] = key[r], p.out.order[at] = order[r];
    }
}

// ------------------------------------------------------------------------------------
// sums over the ordered positions
// ------------------------------------------------------------------------------------
// A warp takes a run of RUN ordered positions and 256 columns. The stretches of one token that lie inside
// the run are finished; the one that goes on at its end (and came from ahead or not) leaves its fp32 sum in
// `open`, slot 1, and one that came from ahead and ends here in slot 0. All rows of the run are on their way at
// once, each lane's 16 bytes of each through its own slots of shared memory, so that the loop over them is
// rolled (with the rows in registers and the loop unrolled, its end of a stretch 17 times in the code, 65536
// positions of 768 columns took 33 us).
constexpr int kShortRun = 16, kLongRun = 32;
int run_of(int64_t m) { return m <= 16384 ? kShortRun : kLongRun; }
__host__ __device__ constexpr int warps_of_run(int run) { return 128 / run; }
struct SumArgs {
  Sorted s;
  int64_t m;
  const uint16_t* dy;
  int64_t cols;
  int slices;  // of 256 columns
  float scale;
  float* de32;
  uint16_t* de16;
  bool add;
  float* open;  // [runs][2][cols]
};

__device__ __forceinline__ void put_row(const SumArgs& p, int64_t row, int64_t col, f2 (&v)[4]) {
  const int64_t at = row * p.cols + col;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = f2_mul(v[j], f2_both(p.scale));
  if (p.de32) {
    ulonglong2* to = reinterpret_cast<ulonglong2*>(p.de32 + at);
    if (p.add) {
      const ulonglong2 a = to[0], b = to[1];
      v[0] = f2_add(v[0], a.x), v[1] = f2_add(v[1], a.y), v[2] = f2_add(v[2], b.x), v[3] = f2_add(v[3], b.y);
    }
    to[0] = make_ulonglong2(v[0], v[1]), to[1] = make_ulonglong2(v[2], v[3]);
  } else {
    uint4* to = reinterpret_cast<uint4*>(p.de16 + at);
    if (p.add) {  // one rounding, of the sum
      f2 old[4];
      widen8(*to, old);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f2_add(v[j], old[j]);
    }
    *to = narrow8(v);
  }
}

// Up to kFewTokens positions: one launch and no workspace. A block has a group of dE's rows; its warps look through
// all tokens, a share each, for those of its rows. The first blocks have 256 columns too: they keep what they found, in
// order; a warp takes a row, collects its positions and sums them. The others mark the rows that they found and fill
// the rest with zeros, whole rows in one sweep (a warp to a row and 256 columns fills half as fast).
// Rows of more than kFewRows positions are left for all warps together, each a share of the positions, whose sums meet
// in shared memory, in order. In which order rows are taken changes no result.
constexpr int kTokenBits = 12, kFewTokens = 1 << kTokenBits, kFewShare = kFewTokens / kWarps, kFewRows = 64;
constexpr int kFewGroup = 1 << 13;  // rows of a group at most
// Blocks per SM that sum and that fill, of five that are resident. 50257 x 768 fp32, 4096 and 1000 tokens, and 1003 of
// 1157 x 520: with 1 and 4 39.1, 26.8 and 7.7 us; 3 and 4 32.8, 28.5 and 7.9; 5 and 8 31.5, 28.7 and 9.0.
constexpr int kSumBlocks = 3, kFillBlocks = 4;
struct FewGroups {
  int sum_blocks, sum_rows, fill_rows;  // blocks that sum, rows of one's group; rows of a block that fills
};
__global__ void __launch_bounds__(kThreads) sum_few_kernel(const void* tokens, int wide, int m, int vocab, int64_t rows,
                                                           const FewGroups groups, const SumArgs p) {
  __shared__ __align__(16) uint32_t found[kWarps][kFewShare];  // (row of the block's, position), in order; later: its rows
  __shared__ uint32_t list[kFewTokens];                        // the same, without gaps
  __shared__ uint16_t at[kWarps][kFewShare];                   // a warp's positions
  __shared__ uint32_t seen[kFewGroup / 32];                    // a bit a row
  __shared__ int count[kWarps];
  __shared__ int many[kFewTokens / kFewRows], n_many, n_rows;
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int block = static_cast<int>(blockIdx.x);
  const bool fill = block >= groups.sum_blocks;
  const int group = fill ? block - groups.sum_blocks : block / p.slices, per = fill ? groups.fill_rows : groups.sum_rows;
  const int64_t row0 = static_cast<int64_t>(group) * per;
  const int mine_rows = static_cast<int>(min(static_cast<int64_t>(per), rows - row0));
  const uint32_t below = (1u << lane) - 1u;
  for (int i = threadIdx.x; i < (mine_rows + 31) / 32; i += kThreads) seen[i] = 0u;
  if (threadIdx.x == 0) n_many = n_rows = 0;
  __syncthreads();
  {
    constexpr int ROUNDS = kFewShare / 32;
    const int each = (m + kWarps * 32 - 1) / (kWarps * 32) * 32, first = warp * each;
    int t[ROUNDS], n = 0;
    tokens_at(tokens, wide, first + lane, min(m, first + each), vocab, t);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const bool mine = t[r] >= row0 && t[r] < row0 + mine_rows;
      const uint32_t row = mine ? static_cast<uint32_t>(t[r] - row0) : 0u;
      const uint32_t all = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        if (fill) atomicOr(&seen[row >> 5], 1u << (row & 31));
        else found[warp][n + __popc(all & below)] = (row << kTokenBits) | static_cast<uint32_t>(first + r * 32 + lane);
      }
      n += __popc(all);
    }
    if (lane == 0) count[warp] = n;
  }
  __syncthreads();
  if (fill) {
    const int64_t row16 = p.cols * (p.de32 ? 4 : 2) / 16;
    uint4* out = reinterpret_cast<uint4*>(p.de32 ? static_cast<void*>(p.de32) : p.de16) + row0 * row16;
    int row = 0;
    int64_t i = threadIdx.x;  // of the row
    while (true) {
      while (i >= row16 && row < mine_rows) i -= row16, ++row;
      if (row >= mine_rows) return;
      if (!((seen[row >> 5] >> (row & 31)) & 1u)) __stcs(out + row * row16 + i, make_uint4(0u, 0u, 0u, 0u));
      i += kThreads;
    }
  }
  const int64_t col = static_cast<int64_t>(block - group * p.slices) * 256 + lane * 8;
  const bool in = col < p.cols;
  int ahead = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) ahead += w < warp ? count[w] : 0, all += count[w];
  if (all == 0) return;
  for (int i = lane; i < count[warp]; i += 32) list[ahead + i] = found[warp][i];
  __syncthreads();
  uint32_t* present = &found[0][0];
  for (int i = threadIdx.x; i < all; i += kThreads) {
    const uint32_t row = list[i] >> kTokenBits, bit = 1u << (row & 31);
    if (!(atomicOr(&seen[row >> 5], bit) & bit)) present[atomicAdd(&n_rows, 1)] = row;
  }
  __syncthreads();
  // the positions of `row` among list[from .. to), to this warp's `at` as far as there is room: how many there are
  const auto collect = [&](uint32_t row, int from, int to, int room) {
    int n = 0;
    for (int i0 = from; i0 < to; i0 += 32) {
      const uint32_t e = i0 + lane < to ? list[i0 + lane] : 0u;
      const bool mine = i0 + lane < to && (e >> kTokenBits) == row;
      const uint32_t hits = __ballot_sync(0xffffffffu, mine);
      const int i = n + __popc(hits & below);
      if (mine && i < room) at[warp][i] = static_cast<uint16_t>(e & (kFewTokens - 1));
      n += __popc(hits);
    }
    __syncwarp();
    return n;
  };
  const auto sum_rows = [&](int n, f2 (&sum)[4]) {
    sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
    if (in)
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        f2 v[4];
        widen8(__ldg(reinterpret_cast<const uint4*>(p.dy + at[warp][j] * p.cols + col)), v);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = f2_add(sum[k], v[k]);
      }
    __syncwarp();  // before the next positions
  };
  f2 sum[4];
  for (int i = warp; i < n_rows; i += kWarps) {
    const uint32_t row = present[i];
    const int n = collect(row, 0, all, kFewRows);
    if (n > kFewRows) {
      if (lane == 0) many[atomicAdd(&n_many, 1)] = static_cast<int>(row);
      continue;
    }
    sum_rows(n, sum);
    if (in) put_row(p, row0 + row, col, sum);
  }
  __syncthreads();
  f2(*part)[32][4] = reinterpret_cast<f2(*)[32][4]>(present);  // its rows are done with
  static_assert(sizeof(f2[kWarps][32][4]) <= sizeof(found), "the warps' sums take their place");
  for (int i = 0; i < n_many; ++i) {
    const int n = collect(static_cast<uint32_t>(many[i]), all * warp / kWarps, all * (warp + 1) / kWarps, kFewShare);
    sum_rows(n, sum);
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][lane][j] = sum[j];
    __syncthreads();
    if (warp == 0 && in) {
#pragma unroll
      for (int w = 1; w < kWarps; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = f2_add(sum[j], part[w][lane][j]);
      put_row(p, row0 + many[i], col, sum);
    }
    __syncthreads();  // before the next row's sums
  }
}

template <int RUN>
__global__ void __launch_bounds__(32 * warps_of_run(RUN)) sum_runs_kernel(const SumArgs p) {
  constexpr int WARPS = warps_of_run(RUN);
  extern __shared__ uint4 run_mem[];
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4* rows = run_mem + warp * RUN * 32 + lane;  // 32 apart
  const int64_t runs = (p.m + RUN - 1) / RUN, items = runs * p.slices, step = static_cast<int64_t>(gridDim.x) * WARPS;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * WARPS + warp; item < items; item += step) {
    const int64_t run = item / p.slices, col = (item - run * p.slices) * 256 + lane * 8, first = run * RUN;
    const bool there = lane < RUN && first + lane < p.m;
    const int key = there ? p.s.key[first + lane] : kNone, at = there ? p.s.order[first + lane] : 0;
    const int before = first > 0 ? p.s.key[first - 1] : -1, behind = first + RUN < p.m ? p.s.key[first + RUN] : -1;
    const bool in = col < p.cols;
    // those without a token are behind the others
    const int real = __popc(__ballot_sync(0xffffffffu, key != kNone));
    if (real == 0) continue;
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      const int pos = __shfl_sync(0xffffffffu, at, j);
      if (in && j < real)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(rows + j * 32)), "l"(p.dy + pos * p.cols + col)
                     : "memory");
    }
    // bit j: a stretch ends with position j of the run
    const int next = __shfl_down_sync(0xffffffffu, key, 1);
    const uint32_t ends = __ballot_sync(0xffffffffu, lane < real && (lane + 1 == real || next != key));
    bool from_ahead = __shfl_sync(0xffffffffu, key, 0) == before;
    const bool goes_on = real == RUN && __shfl_sync(0xffffffffu, key, RUN - 1) == behind;
    float* open = p.open + run * 2 * p.cols + col;
    asm volatile("cp.async.wait_all;" ::: "memory");
    f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 2
    for (int j = 0; j < real; ++j) {
      if (in) {
        f2 v[4];
        widen8(rows[j * 32], v);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = f2_add(sum[k], v[k]);
      }
      if (!((ends >> j) & 1u)) continue;  // the same for the whole warp
      const int token = __shfl_sync(0xffffffffu, key, j);
      const bool leaves = goes_on && j == RUN - 1;
      if (in) {
        if (leaves || from_ahead) {
          ulonglong2* to = reinterpret_cast<ulonglong2*>(open + (leaves ? p.cols : 0));
          to[0] = make_ulonglong2(sum[0], sum[1]), to[1] = make_ulonglong2(sum[2], sum[3]);
        } else {
          put_row(p, token, col, sum);
        }
      }
      sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
      from_ahead = false;
    }
  }
}

// The tokens whose stretch crosses from one run into the next, 256 columns at a time: where it touches up to
// kFewRuns runs, by a warp, at the boundary where it crosses first; where it touches more, by a block, at the first of
// its runs whose number is a multiple of kFewRuns / 2 (it has one that starts with it), the runs shared among its
// warps, whose sums meet in shared memory. The first few_blocks blocks are of the first kind.
constexpr int kFewRuns = 16, kCrossThreads = 512, kCrossWarps = kCrossThreads / 32;
// the sums that runs from .. to - 1 left of a stretch: it goes on behind every run but `last`, where it left its sum
// as one that ends there
__device__ __forceinline__ void add_open(const SumArgs& p, int64_t from, int64_t to, int64_t last, int64_t col, f2 (&sum)[4]) {
  sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
#pragma unroll 8
  for (int64_t r = from; r < to; ++r) {
    const ulonglong2* a = reinterpret_cast<const ulonglong2*>(p.open + (r * 2 + (r < last ? 1 : 0)) * p.cols + col);
    const ulonglong2 x = a[0], y = a[1];
    sum[0] = f2_add(sum[0], x.x), sum[1] = f2_add(sum[1], x.y), sum[2] = f2_add(sum[2], y.x), sum[3] = f2_add(sum[3], y.y);
  }
}
template <int RUN>
__global__ void __launch_bounds__(kCrossThreads) sum_crossing_kernel(const SumArgs p, int64_t few_blocks) {
  __shared__ f2 part[kCrossWarps][32][4];
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t runs = (p.m + RUN - 1) / RUN;
  const int* key = p.s.key;
  f2 sum[4];
  if (blockIdx.x < few_blocks) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kCrossWarps + warp, b = 1 + item / p.slices;  // between b - 1 and b
    if (b >= runs) return;
    const int64_t first = b * RUN, col = (item - (b - 1) * p.slices) * 256 + lane * 8;
    // whether the runs from b on begin with the token; lanes in order: the first that does not
    const int64_t r = b + lane;
    const int mine = r < runs ? key[r * RUN] : -1, token = __shfl_sync(0xffffffffu, mine, 0);
    const int before = key[first - 1], earlier = b > 1 ? key[first - RUN - 1] : -1;
    if (token == kNone || before != token || earlier == token) return;  // none crosses here, or it crossed before
    const uint32_t other = ~__ballot_sync(0xffffffffu, mine == token);
    const int more = other ? __ffs(other) - 1 : 32;  // runs from b on that it touches
    if (1 + more > kFewRuns || col >= p.cols) return;
    add_open(p, b - 1, b + more, b + more - 1, col, sum);
    put_row(p, token, col, sum);
    return;
  }
  const int64_t item = blockIdx.x - few_blocks, at = item / p.slices * (kFewRuns / 2);  // a run
  const int64_t col = (item - item / p.slices * p.slices) * 256 + lane * 8;
  const int token = key[at * RUN];
  if (token == kNone) return;
  // the runs ahead that it touches
  const int64_t r = at - 1 - lane;
  const uint32_t other = ~__ballot_sync(0xffffffffu, r >= 0 && key[r * RUN + RUN - 1] == token);
  const int ahead = other ? __ffs(other) - 1 : 32;
  // that one's, if it begins the run kFewRuns / 2 ahead too: sure where it touches runs before that
  if (ahead > kFewRuns / 2 || (ahead == kFewRuns / 2 && key[(at - kFewRuns / 2) * RUN] == token)) return;
  int64_t last = at;
  for (int64_t r0 = at + 1;; r0 += kCrossThreads) {
    const int64_t q = r0 + threadIdx.x;
    const int n = __syncthreads_count(q < runs && key[q * RUN] == token);
    last += n;
    if (n < kCrossThreads) break;
  }
  const int64_t from = at - ahead, parts = last - from + 1;
  if (parts <= kFewRuns) return;
  const bool in = col < p.cols;
  if (in) add_open(p, from + parts * warp / kCrossWarps, from + parts * (warp + 1) / kCrossWarps, last, col, sum);
#pragma unroll
  for (int j = 0; j < 4; ++j) part[warp][lane][j] = in ? sum[j] : 0ull;
  __syncthreads();
  if (warp == 0 && in) {
#pragma unroll
    for (int w = 1; w < kCrossWarps; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = f2_add(sum[j], part[w][lane][j]);
    put_row(p, token, col, sum);
  }
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_sizes(int64_t m, int64_t rows, int64_t vocab, int64_t cols, int token_bytes, const char* who) {
  const int64_t most = 1 << 30;
  if (m < 1 || rows < 1 || m > most || rows > most)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: m_tokens and rows must be in 1..2^30", who);
  if (cols < 1 || cols > (1 << 20)) return set_error(ZERO_ERR_INVALID_ARG, "%s: cols must be in 1..2^20", who);
  if (m * cols > (int64_t(1) << 42))
    return set_error(ZERO_ERR_UNSUPPORTED, "%s: %lld x %lld is more than 2^42 elements", who, (long long)m, (long long)cols);
  if (cols % 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: cols %lld must be a multiple of 8 (16-byte rows)", who, (long long)cols);
  if (vocab < 1 || vocab > rows)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: vocab %lld outside 1..%lld (the table's rows)", who, (long long)vocab,
                     (long long)rows);
  if (token_bytes != 4 && token_bytes != 8)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: token_bytes %d is not 4 or 8", who, token_bytes);
  return ZERO_OK;
}

// The backward's workspace: the ordered positions (twice, where they are sorted in passes, with their counts),
// and the open sums of the runs.
struct BackwardSpace {
  int64_t sort_blocks;
  int passes;
  uint64_t key[2], order[2], count, open, bytes;
  BackwardSpace(int64_t m, int64_t vocab, int64_t cols) {
    const auto take = [&](uint64_t n) {
      const uint64_t at = bytes;
      bytes += (n + 255) & ~uint64_t(255);
      return at;
    };
    bytes = 0, passes = 0, sort_blocks = 0, count = 0;
    key[0] = key[1] = order[0] = order[1] = open = 0;
    if (m <= kFewTokens) return;
    key[0] = key[1] = take(4 * static_cast<uint64_t>(m));
    order[0] = order[1] = take(4 * static_cast<uint64_t>(m));
    int bits = 1;
    while (bits < 31 && (vocab >> bits) != 0) ++bits;  // of keys 0 .. vocab
    passes = (bits + kDigitBits - 1) / kDigitBits;
    sort_blocks = (m + kSortTile - 1) / kSortTile;
    if (passes > 1) key[1] = take(4 * static_cast<uint64_t>(m)), order[1] = take(4 * static_cast<uint64_t>(m));
    count = take(4 * static_cast<uint64_t>(sort_blocks) * kDigits);
    open = take(8 * static_cast<uint64_t>((m + run_of(m) - 1) / run_of(m)) * static_cast<uint64_t>(cols));
  }
};

}  // namespace
}  // namespace zgb

using namespace zgb;

extern "C" int fsdp_embedding_forward(int n_ranks, const zero_bf16* const e_shards[], int64_t rows, int64_t vocab,
                                      int64_t cols, const void* tokens, int token_bytes, int64_t m_tokens, float scale,
                                      zero_bf16* Y, zero_stream_t stream) {
  const char* who = "fsdp_embedding_forward";
  int rc = check_sizes(m_tokens, rows, vocab, cols, token_bytes, who);
  if (rc) return rc;
  if (n_ranks < 1 || n_ranks > 16) return set_error(ZERO_ERR_INVALID_ARG, "%s: n_ranks %d outside 1..16", who, n_ranks);
  if (rows % n_ranks)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: rows %lld must be a multiple of n_ranks %d", who, (long long)rows, n_ranks);
  if (!e_shards) return set_error(ZERO_ERR_INVALID_ARG, "%s: e_shards is NULL", who);
  if (!tokens || !Y) return set_error(ZERO_ERR_INVALID_ARG, "%s: tokens or Y is NULL", who);
  TableShards e = {};
  for (int q = 0; q < n_ranks; ++q) {
    if (!e_shards[q]) return set_error(ZERO_ERR_INVALID_ARG, "%s: e_shards[%d] is NULL (missing rank)", who, q);
    if (!aligned16(e_shards[q]))
      return set_error(ZERO_ERR_INVALID_ARG, "%s: e_shards[%d] must be 16-byte aligned", who, q);
    e.p[q] = e_shards[q];
  }
  if (!aligned16(Y)) return set_error(ZERO_ERR_INVALID_ARG, "%s: Y must be 16-byte aligned", who);
  if (reinterpret_cast<uintptr_t>(tokens) % token_bytes)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: tokens must be aligned to their %d bytes", who, token_bytes);
  if (!(scale - scale == 0.0f)) return set_error(ZERO_ERR_INVALID_ARG, "%s: scale must be finite", who);
  const int slices = static_cast<int>((cols + kPieces * 256 - 1) / (kPieces * 256));
  const int64_t blocks = std::min<int64_t>((m_tokens * slices + kWarps - 1) / kWarps, static_cast<int64_t>(num_sms()) * 64);
  const cudaError_t err = launch_overlapped(embedding_forward_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, 1,
                                            reinterpret_cast<cudaStream_t>(stream), e, static_cast<int>(rows / n_ranks),
                                            static_cast<int>(vocab), cols, tokens, token_bytes == 8 ? 1 : 0, m_tokens, slices,
                                            scale, Y);
  return err == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(err));
}

extern "C" int fsdp_embedding_backward_workspace(int64_t m_tokens, int64_t vocab, int64_t cols, uint64_t* bytes) {
  const char* who = "fsdp_embedding_backward_workspace";
  if (!bytes) return set_error(ZERO_ERR_INVALID_ARG, "%s: bytes is NULL", who);
  const int rc = check_sizes(m_tokens, vocab, vocab, cols, 4, who);
  if (rc) return rc;
  *bytes = BackwardSpace(m_tokens, vocab, cols).bytes;
  return ZERO_OK;
}

extern "C" int fsdp_embedding_backward(const zero_bf16* dY, const void* tokens, int token_bytes, int64_t m_tokens,
                                       int64_t rows, int64_t vocab, int64_t cols, float scale, int accumulate, float* dE,
                                       zero_bf16* dE_bf16, void* workspace, uint64_t workspace_bytes, zero_stream_t stream) {
  const char* who = "fsdp_embedding_backward";
  const int rc = check_sizes(m_tokens, rows, vocab, cols, token_bytes, who);
  if (rc) return rc;
  if (!dY || !tokens) return set_error(ZERO_ERR_INVALID_ARG, "%s: dY or tokens is NULL", who);
  if ((dE != nullptr) == (dE_bf16 != nullptr)) return set_error(ZERO_ERR_INVALID_ARG, "%s: pass one of dE and dE_bf16", who);
  if (!(scale - scale == 0.0f)) return set_error(ZERO_ERR_INVALID_ARG, "%s: scale must be finite", who);
  if (!aligned16(dY) || !aligned16(dE) || !aligned16(dE_bf16) || !aligned16(workspace))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: dY, dE and workspace must be 16-byte aligned", who);
  if (reinterpret_cast<uintptr_t>(tokens) % token_bytes)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: tokens must be aligned to their %d bytes", who, token_bytes);
  const BackwardSpace sp(m_tokens, vocab, cols);
  if (sp.bytes && (!workspace || workspace_bytes < sp.bytes))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                     workspace ? (unsigned long long)workspace_bytes : 0ull, (unsigned long long)sp.bytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const auto ints = [&](uint64_t at) { return reinterpret_cast<int*>(ws + at); };
  uint4* zero = reinterpret_cast<uint4*>(dE ? static_cast<void*>(dE) : dE_bf16);
  const int64_t zero16 = accumulate ? 0 : rows * cols * (dE ? 4 : 2) / 16;
  const int wide = token_bytes == 8 ? 1 : 0;
  Sorted sorted{ints(sp.key[0]), ints(sp.order[0])};
  const int64_t slices = (cols + 255) / 256;
  SumArgs a;
  a.s = sorted, a.m = m_tokens, a.dy = dY, a.cols = cols, a.slices = static_cast<int>(slices), a.scale = scale;
  a.de32 = dE, a.de16 = dE_bf16, a.add = accumulate != 0, a.open = reinterpret_cast<float*>(ws + sp.open);
  cudaError_t e = cudaSuccess;
  if (m_tokens <= kFewTokens) {
    const auto rows_each = [&](int64_t blocks) {
      return std::min<int64_t>((rows + blocks - 1) / blocks, kFewGroup);
    };
    const int64_t sms = num_sms();
    const int64_t sum_rows = rows_each(std::max<int64_t>(1, std::min(rows, kSumBlocks * sms / slices)));
    const int64_t fill_rows = rows_each(std::max<int64_t>(1, std::min(std::min(rows, kFillBlocks * sms), zero16 / (2 * kThreads))));
    const int64_t sum_blocks = (rows + sum_rows - 1) / sum_rows * slices, fill_blocks = zero16 ? (rows + fill_rows - 1) / fill_rows : 0;
    const FewGroups groups{static_cast<int>(sum_blocks), static_cast<int>(sum_rows), static_cast<int>(fill_rows)};
    e = launch_overlapped(sum_few_kernel, dim3(static_cast<unsigned>(sum_blocks + fill_blocks)), dim3(kThreads), 0, 1, st, tokens,
                          wide, static_cast<int>(m_tokens), static_cast<int>(vocab), rows, groups, a);
    return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  for (int pass = 0; pass < sp.passes && e == cudaSuccess; ++pass) {
    SortPass p;
    p.tokens = pass == 0 ? tokens : nullptr;
    p.wide = wide, p.vocab = static_cast<int>(vocab), p.shift = pass * kDigitBits, p.m = m_tokens;
    p.blocks = static_cast<int>(sp.sort_blocks);
    // the last pass ends in the first buffer
    const int to = (sp.passes - 1 - pass) & 1;
    p.in = {ints(sp.key[to ^ 1]), ints(sp.order[to ^ 1])};
    p.out = {ints(sp.key[to]), ints(sp.order[to])};
    p.count = ints(sp.count), p.scanned = sp.sort_blocks > kOwnScan;
    // of every four parts of a pass's share of dE, one beside the counts and three beside the placing, which takes
    // three times as long
    const auto part = [&](int64_t i) { return zero16 * (4 * pass + i) / (4 * sp.passes); };
    const auto share = [&](int64_t from, int64_t to) {
      p.zero = zero + from, p.zero16 = to - from;
      return static_cast<unsigned>(sp.sort_blocks + std::min<int64_t>((p.zero16 + 4 * kSortThreads - 1) / (4 * kSortThreads),
                                                                     static_cast<int64_t>(num_sms()) * 4));
    };
    const unsigned counting = share(part(0), part(1));
    e = launch_overlapped(sort_count_kernel, dim3(counting), dim3(kSortThreads), 0, 1, st, p);
    if (e == cudaSuccess && p.scanned)
      e = launch_overlapped(sort_scan_kernel, dim3(1), dim3(1024), 0, 1, st, p.count, sp.sort_blocks * kDigits);
    const unsigned placing = share(part(1), part(4));
    if (e == cudaSuccess)
      e = launch_overlapped(sort_scatter_kernel, dim3(placing), dim3(kSortThreads), 0, 1, st, p);
  }
  const int run = run_of(m_tokens);
  const int64_t runs = (m_tokens + run - 1) / run;
  const auto sums = [&](auto length) {
    constexpr int RUN = decltype(length)::value, WARPS = warps_of_run(RUN);
    constexpr uint32_t smem = WARPS * RUN * 512;
    const int64_t blocks = std::min<int64_t>((runs * slices + WARPS - 1) / WARPS, static_cast<int64_t>(num_sms()) * 64);
    static OncePerDevice once;
    int dev = 0;
    cudaError_t q = cudaGetDevice(&dev);
    if (q == cudaSuccess)
      q = once.run(dev, [] {
        return cudaFuncSetAttribute(sum_runs_kernel<RUN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      });
    if (q == cudaSuccess)
      q = launch_overlapped(sum_runs_kernel<RUN>, dim3(static_cast<unsigned>(blocks)), dim3(32 * WARPS), smem, 1, st, a);
    if (q == cudaSuccess && runs > 1) {
      const int64_t few = ((runs - 1) * slices + kCrossWarps - 1) / kCrossWarps;
      const int64_t many = (runs + kFewRuns / 2 - 1) / (kFewRuns / 2) * slices;
      q = launch_overlapped(sum_crossing_kernel<RUN>, dim3(static_cast<unsigned>(few + many)), dim3(kCrossThreads), 0, 1, st, a, few);
    }
    return q;
  };
  if (e == cudaSuccess) e = run == kShortRun ? sums(ActTag<kShortRun>{}) : sums(ActTag<kLongRun>{});
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}
