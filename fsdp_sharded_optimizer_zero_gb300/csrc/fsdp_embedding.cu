// Token embedding from a table held as row shards, and its gradient.
//
//   forward   Y[i] = scale E[t_i]
//   backward  dE[v] = scale * sum over i with t_i = v of dY[i], every row of dE (or added to it)
//
// The backward orders the positions by token first (stably: the positions of one token stay in order),
// so that the rows of one token lie one after the other and are summed in registers in a fixed order,
// without atomics: the same bits every call. A token outside 0 .. vocab - 1 is none: zeros, no gradient.
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

// A warp takes up to 1024 columns of a token's row at a time: four pieces of 8 columns a lane, in flight together.
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

__device__ __forceinline__ int key_at(const void* tokens, int wide, int64_t i, int vocab) {
  const int t = token_at(tokens, wide, i, vocab);
  return t < 0 ? kNone : t;
}

// zeros to `n16` pieces of 16 bytes, by block `block` of `blocks`
__device__ __forceinline__ void fill_zeros(uint4* out, int64_t n16, int64_t block, int64_t blocks) {
  for (int64_t i = block * kThreads + threadIdx.x; i < n16; i += blocks * kThreads) __stcs(out + i, make_uint4(0u, 0u, 0u, 0u));
}

// Up to kRankMost positions: a position's place is the number of smaller keys and of equal ones ahead of it,
// counted over all keys, kRankSplit threads to a position. m^2 comparisons, but one launch, and beside it the
// rest of the blocks fill dE with zeros.
constexpr int kRankMost = 16384;
constexpr int kRankSplit = 8;
constexpr int kRankTile = 2048;  // keys in shared memory at a time
__global__ void __launch_bounds__(kThreads) rank_kernel(const void* tokens, int wide, int m, int vocab, Sorted s,
                                                        int rank_blocks, uint4* zero, int64_t zero16) {
  __shared__ int keys[kRankTile];
  allow_next_grid();
  wait_for_prior_grids();
  if (static_cast<int>(blockIdx.x) >= rank_blocks) {
    fill_zeros(zero, zero16, blockIdx.x - rank_blocks, gridDim.x - rank_blocks);
    return;
  }
  const int i = (static_cast<int>(blockIdx.x) * kThreads + static_cast<int>(threadIdx.x)) / kRankSplit;
  const int part = threadIdx.x % kRankSplit;
  const int mine = i < m ? key_at(tokens, wide, i, vocab) : kNone;
  int count = 0;
  for (int t0 = 0; t0 < m; t0 += kRankTile) {
    __syncthreads();
    for (int j = threadIdx.x; j < kRankTile; j += kThreads) keys[j] = t0 + j < m ? key_at(tokens, wide, t0 + j, vocab) : kNone;
    __syncthreads();
    const int last = min(kRankTile, m - t0);
    for (int j = part; j < last; j += kRankSplit) {
      const int k = keys[j];
      count += (k < mine || (k == mine && t0 + j < i)) ? 1 : 0;
    }
  }
#pragma unroll
  for (int d = 1; d < kRankSplit; d *= 2) count += __shfl_xor_sync(0xffffffffu, count, d);
  if (i < m && part == 0) s.key[count] = mine, s.order[count] = i;
}

// More positions: a radix sort, a digit of kDigitBits a pass from the lowest, each pass stable. Block b has the
// positions from b kSortTile on, a warp a run of them.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortTile = 4096, kSortRun = kSortTile / kWarps;
struct SortPass {
  const void* tokens;  // first pass: the tokens themselves; else null
  int wide, vocab, shift;
  Sorted in, out;
  int64_t m;
  int blocks;
  int* count;  // [kDigits][blocks], then the places where they begin
};
__device__ __forceinline__ int sort_key(const SortPass& p, int64_t i) {
  return p.tokens ? key_at(p.tokens, p.wide, i, p.vocab) : p.in.key[i];
}
// positions without a token have the digits of `vocab`, which no token has: behind the others
__device__ __forceinline__ int sort_digit(const SortPass& p, int key) {
  return (min(key, p.vocab) >> p.shift) & (kDigits - 1);
}

__global__ void __launch_bounds__(kThreads) sort_count_kernel(const SortPass p, uint4* zero, int64_t zero16) {
  __shared__ int count[kDigits];
  allow_next_grid();
  wait_for_prior_grids();
  if (static_cast<int>(blockIdx.x) >= p.blocks) {
    fill_zeros(zero, zero16, blockIdx.x - p.blocks, gridDim.x - p.blocks);
    return;
  }
  for (int d = threadIdx.x; d < kDigits; d += kThreads) count[d] = 0;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSortTile;
  for (int j = threadIdx.x; j < kSortTile; j += kThreads)
    if (first + j < p.m) atomicAdd(&count[sort_digit(p, sort_key(p, first + j))], 1);
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kThreads) p.count[static_cast<int64_t>(d) * p.blocks + blockIdx.x] = count[d];
}

// exclusive sums over all of count, in place, by one block
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

__global__ void __launch_bounds__(kThreads) sort_scatter_kernel(const SortPass p) {
  __shared__ int next[kWarps][kDigits];  // per warp: counts, then where its next position of a digit goes
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int d = threadIdx.x; d < kWarps * kDigits; d += kThreads) (&next[0][0])[d] = 0;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kSortTile + warp * kSortRun;
  for (int j = lane; j < kSortRun; j += 32)
    if (first + j < p.m) atomicAdd(&next[warp][sort_digit(p, sort_key(p, first + j))], 1);
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kThreads) {
    int at = p.count[static_cast<int64_t>(d) * p.blocks + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int n = next[w][d];
      next[w][d] = at;
      at += n;
    }
  }
  __syncthreads();
  for (int j = lane; j < kSortRun; j += 32) {  // the same number of rounds for every lane
    const bool there = first + j < p.m;
    const int key = there ? sort_key(p, first + j) : 0;
    const int digit = there ? sort_digit(p, key) : kDigits;  // those past the end among themselves
    const uint32_t same = __match_any_sync(0xffffffffu, digit);
    const int ahead = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (there) at = next[warp][digit] + ahead;
    __syncwarp();
    if (there && ahead == 0) next[warp][digit] += __popc(same);
    __syncwarp();
    if (there) {
      p.out.key[at] = key;
      p.out.order[at] = p.tokens ? static_cast<int>(first + j) : p.in.order[first + j];
    }
  }
}

// ------------------------------------------------------------------------------------
// sums over the ordered positions
// ------------------------------------------------------------------------------------
// A warp takes a run of RUN ordered positions and 256 columns. The stretches of one token that lie inside
// the run are finished; the one that goes on at its end (and came from ahead or not) leaves its fp32 sum in
// `open`, slot 1, and one that came from ahead and ends here in slot 0.
constexpr int kShortRun = 16, kLongRun = 32;
int run_of(int64_t m) { return m <= kRankMost ? kShortRun : kLongRun; }
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

__device__ __forceinline__ void put_row(const SumArgs& p, int key, int64_t col, f2 (&v)[4]) {
  const int64_t at = static_cast<int64_t>(key) * p.cols + col;
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

template <int RUN>
__global__ void __launch_bounds__(kThreads) sum_runs_kernel(const SumArgs p) {
  allow_next_grid();
  wait_for_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t runs = (p.m + RUN - 1) / RUN, items = runs * p.slices, step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items; item += step) {
    const int64_t run = item / p.slices, col = (item - run * p.slices) * 256 + lane * 8, first = run * RUN;
    const int count = static_cast<int>(min(p.m - first, static_cast<int64_t>(RUN)));
    const int key = lane < count ? p.s.key[first + lane] : kNone;
    const int at = lane < count ? p.s.order[first + lane] : 0;
    const int before = first > 0 ? p.s.key[first - 1] : -1, after = first + count < p.m ? p.s.key[first + count] : -1;
    const bool in = col < p.cols;
    f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
    int now = __shfl_sync(0xffffffffu, key, 0);
    bool from_ahead = now == before;
    float* open = p.open + run * 2 * p.cols + col;
    const auto leave = [&](int slot) {
      if (in) {
        ulonglong2* to = reinterpret_cast<ulonglong2*>(open + slot * p.cols);
        to[0] = make_ulonglong2(sum[0], sum[1]), to[1] = make_ulonglong2(sum[2], sum[3]);
      }
    };
    // all rows of the run are on their way before the first is used
    constexpr int AHEAD = RUN < 16 ? RUN : 16;
    for (int j0 = 0; j0 < count && now != kNone; j0 += AHEAD) {
      uint4 w[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int k = __shfl_sync(0xffffffffu, key, (j0 + j) & 31), pos = __shfl_sync(0xffffffffu, at, (j0 + j) & 31);
        w[j] = make_uint4(0u, 0u, 0u, 0u);
        if (j0 + j < count && k != kNone && in) w[j] = __ldg(reinterpret_cast<const uint4*>(p.dy + pos * p.cols + col));
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int k = j0 + j < count ? __shfl_sync(0xffffffffu, key, (j0 + j) & 31) : now;
        if (k != now) {  // the same for the whole warp
          if (from_ahead) leave(0);
          else if (in) put_row(p, now, col, sum);
          sum[0] = sum[1] = sum[2] = sum[3] = 0ull;
          now = k, from_ahead = false;
        }
        f2 v[4];
        widen8(w[j], v);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = f2_add(sum[i], v[i]);  // zeros past the run
      }
    }
    if (now == kNone) continue;
    if (now == after) leave(1);
    else if (from_ahead) leave(0);
    else if (in) put_row(p, now, col, sum);
  }
}

// The tokens whose stretch crosses from one run into the next: a block takes a boundary where a stretch
// crosses for the first time and 256 columns, its warps consecutive parts of the runs it touches.
template <int RUN>
__global__ void __launch_bounds__(kThreads) sum_crossing_kernel(const SumArgs p) {
  __shared__ f2 part[kWarps][32][4];
  allow_next_grid();
  wait_for_prior_grids();
  const int64_t b = blockIdx.x + 1, first = b * RUN, runs = (p.m + RUN - 1) / RUN;  // between runs b - 1 and b
  const int key = p.s.key[first], before = p.s.key[first - 1], earlier = b > 1 ? p.s.key[first - RUN - 1] : -1;
  // which of the next runs begin with the key, 256 at a time: keys are in order
  int64_t last = b;
  for (int64_t r0 = b + 1;; r0 += kThreads) {
    const int64_t r = r0 + threadIdx.x;
    const bool same = r < runs && p.s.key[r * RUN] == key;
    if (r0 == b + 1 && (key == kNone || before != key || earlier == key)) return;  // none crosses here, or crossed before
    const int n = __syncthreads_count(same);
    last += n;
    if (n < kThreads) break;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * 256 + lane * 8;
  const bool in = col < p.cols;
  const int64_t parts = last - b + 2, from = b - 1 + parts * warp / kWarps, to = b - 1 + parts * (warp + 1) / kWarps;
  f2 sum[4] = {0ull, 0ull, 0ull, 0ull};
  if (in)
#pragma unroll 8
    for (int64_t r = from; r < to; ++r) {
      // it goes on behind every run but the last, where it left its sum as one that ends there
      const ulonglong2* a = reinterpret_cast<const ulonglong2*>(p.open + (r * 2 + (r < last ? 1 : 0)) * p.cols + col);
      const ulonglong2 x = a[0], y = a[1];
      sum[0] = f2_add(sum[0], x.x), sum[1] = f2_add(sum[1], x.y), sum[2] = f2_add(sum[2], y.x), sum[3] = f2_add(sum[3], y.y);
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) part[warp][lane][j] = sum[j];
  __syncthreads();
  if (warp == 0 && in) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = f2_add(sum[j], part[w][lane][j]);
    put_row(p, key, col, sum);
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
    key[0] = key[1] = take(4 * static_cast<uint64_t>(m));
    order[0] = order[1] = take(4 * static_cast<uint64_t>(m));
    if (m > kRankMost) {
      int bits = 1;
      while (bits < 31 && (vocab >> bits) != 0) ++bits;  // of keys 0 .. vocab
      passes = (bits + kDigitBits - 1) / kDigitBits;
      sort_blocks = (m + kSortTile - 1) / kSortTile;
      if (passes > 1) key[1] = take(4 * static_cast<uint64_t>(m)), order[1] = take(4 * static_cast<uint64_t>(m));
      count = take(4 * static_cast<uint64_t>(sort_blocks) * kDigits);
    }
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
  if (!workspace || workspace_bytes < sp.bytes)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: workspace of %llu bytes is below the %llu needed", who,
                     workspace ? (unsigned long long)workspace_bytes : 0ull, (unsigned long long)sp.bytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const auto ints = [&](uint64_t at) { return reinterpret_cast<int*>(ws + at); };
  uint4* zero = reinterpret_cast<uint4*>(dE ? static_cast<void*>(dE) : dE_bf16);
  const int64_t zero16 = accumulate ? 0 : rows * cols * (dE ? 4 : 2) / 16;
  const int64_t zero_blocks = std::min<int64_t>((zero16 + 4 * kThreads - 1) / (4 * kThreads), static_cast<int64_t>(num_sms()) * 8);
  const int wide = token_bytes == 8 ? 1 : 0;
  Sorted sorted{ints(sp.key[0]), ints(sp.order[0])};
  cudaError_t e = cudaSuccess;
  if (sp.passes == 0) {
    const int64_t rank_blocks = (m_tokens * kRankSplit + kThreads - 1) / kThreads;
    e = launch_overlapped(rank_kernel, dim3(static_cast<unsigned>(rank_blocks + zero_blocks)), dim3(kThreads), 0, 1, st, tokens,
                          wide, static_cast<int>(m_tokens), static_cast<int>(vocab), sorted, static_cast<int>(rank_blocks),
                          zero, zero16);
  } else {
    for (int pass = 0; pass < sp.passes && e == cudaSuccess; ++pass) {
      SortPass p;
      p.tokens = pass == 0 ? tokens : nullptr;
      p.wide = wide, p.vocab = static_cast<int>(vocab), p.shift = pass * kDigitBits, p.m = m_tokens;
      p.blocks = static_cast<int>(sp.sort_blocks);
      // the last pass ends in the first buffer
      const int to = (sp.passes - 1 - pass) & 1;
      p.in = {ints(sp.key[to ^ 1]), ints(sp.order[to ^ 1])};
      p.out = {ints(sp.key[to]), ints(sp.order[to])};
      p.count = ints(sp.count);
      const int64_t more = pass == 0 ? zero_blocks : 0;
      e = launch_overlapped(sort_count_kernel, dim3(static_cast<unsigned>(sp.sort_blocks + more)), dim3(kThreads), 0, 1, st, p,
                            zero, zero16);
      if (e == cudaSuccess)
        e = launch_overlapped(sort_scan_kernel, dim3(1), dim3(1024), 0, 1, st, p.count, sp.sort_blocks * kDigits);
      if (e == cudaSuccess)
        e = launch_overlapped(sort_scatter_kernel, dim3(static_cast<unsigned>(sp.sort_blocks)), dim3(kThreads), 0, 1, st, p);
    }
  }
  const int run = run_of(m_tokens);
  const int64_t runs = (m_tokens + run - 1) / run, slices = (cols + 255) / 256;
  SumArgs a;
  a.s = sorted, a.m = m_tokens, a.dy = dY, a.cols = cols, a.slices = static_cast<int>(slices), a.scale = scale;
  a.de32 = dE, a.de16 = dE_bf16, a.add = accumulate != 0, a.open = reinterpret_cast<float*>(ws + sp.open);
  if (e == cudaSuccess) {
    const int64_t blocks = std::min<int64_t>((runs * slices + kWarps - 1) / kWarps, static_cast<int64_t>(num_sms()) * 64);
    e = launch_overlapped(run == kShortRun ? sum_runs_kernel<kShortRun> : sum_runs_kernel<kLongRun>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, 1, st, a);
  }
  if (e == cudaSuccess && runs > 1)
    e = launch_overlapped(run == kShortRun ? sum_crossing_kernel<kShortRun> : sum_crossing_kernel<kLongRun>,
                          dim3(static_cast<unsigned>(runs - 1), static_cast<unsigned>(slices)), dim3(kThreads),
                          0, 1, st, a);
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}
