// The narrow kernel: products of few or small outputs, 128 output columns x TN output rows per tile, the contraction
// split over the CTAs of a cluster, whose parts meet in distributed shared memory and are added in a fixed order. Used by
// the linear unit and by the loss over the vocabulary.
#pragma once
#include "linear_wide.cuh"

namespace zgb {
namespace {

// What 4 columns of a row read beside their sums: load(p, row, col), called while the main loop runs. Volatile loads: the
// compiler would move them down to their use.
template <int OP> struct Side4;
__device__ __forceinline__ void load8(const uint16_t* src, uint2& w) {
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(src));
}
// 4 columns of one output row per lane, 32 lanes across 128 columns. bias: the columns' biases (fwd, where there are any).
// Called by whole warps, for rows of the output.
template <int OP, int ACT>
__device__ __forceinline__ void epilogue4(const typename Wide<OP>::Params& p, int row, int col, uint2 bias,
                                          const Side4<OP>& side, f2 (&v)[2]);

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
  static_assert(STAGES * STAGE >= TN * 128 * 4, "the fp32 part takes the stages' place");
};

// logits have an accumulator for each part of the contraction; two CTAs share the 512 columns
constexpr int kLogitCols = 256;
template <int OP, int TN>
__host__ __device__ constexpr uint32_t tmem_cols() { return is_logits(OP) ? kLogitCols : TN; }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// What follows the main loop, for S CTAs to a tile, by all eight warps: the parts to their owners,
// their sum and the epilogue. `wait` returns once the accumulator is complete.
template <int OP, int TN, int S, class Wait>
__device__ __forceinline__ void finish_tile(const typename Wide<OP>::Params& p, int parts, uint8_t* smem, uint32_t tmem_base, int rank, int m0,
                                            int n0, int warp, int lane, Wait&& wait) {
  constexpr int ROWS = TN / S;                         // rows this CTA finishes
  constexpr int MINE = ROWS < 8 ? 1 : ROWS / 8;        // rows of a warp: warp, warp + 8, ..
  constexpr int AHEAD = MINE < 8 ? MINE : 8;           // of them, with their side tensors loaded ahead
  const int col = n0 + lane * 4, row0 = m0 + rank * ROWS;
  uint2 bias = make_uint2(0u, 0u);
  if (OP == OP_FWD && p.bias && col < p.n) load8(p.bias + col, bias);
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
    if constexpr (is_logits(OP)) {
      for (int i = 1; i < parts; ++i) {
        uint32_t more[32];
        tmem_ld_32cols(taddr + i * TN + t0, more);
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__fadd_rn(__uint_as_float(r[j]), __uint_as_float(more[j])));
      }
    }
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
  with_act(OP == OP_FWD || OP == OP_DX ? p.act : FSDP_ACT_NONE, [&](auto act) {
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
__global__ void __launch_bounds__(256, 2) linear_narrow_kernel(const __grid_constant__ typename Wide<OP>::Params p) {
  using C = Narrow<TN>;
  constexpr bool P_MN = !loads_as_fwd(OP), Q_MN = OP == OP_DW;  // P: the column side, Q: the row side
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
    tmem_alloc(smem_u32(&tmem_base_sh), tmem_cols<OP, TN>());
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
    if constexpr (loads_as_fwd(OP)) i -= w_copies_k_major<CUT>(p, i, n0 + first_w_row<OP>(p), kb0, 0, c, has);
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
        for (int kb = kb0; kb < min(kb1, kb0 + C::STAGES); ++kb, some = copy_advance<CUT>(p, ahead, some))
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
        has = copy_advance<CUT>(p, c, has);
      }
      __syncwarp();
      if (++s == C::STAGES) s = 0, ph ^= 1u;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t p_step = P_MN ? 128u : 2u, q_step = Q_MN ? 128u : 2u;
      constexpr uint32_t idesc = idesc_bf16_f32(128, TN, P_MN, Q_MN);
      uint32_t s = 0, ph = 0, acc = tmem_base;
      int part0 = kb0;  // where this accumulator's part begins
      for (int kb = kb0; kb < kb1; ++kb) {
        if (is_logits(OP) && kb == part0 + p.chunk_blocks) acc += TN, part0 = kb;
        if (!wait_bounded(smem_u32(&full_bar[s]), ph, abort, kErrFull)) break;
        tc_fence_after();
        const uint32_t sp = smem_u32(smem) + s * C::STAGE;
        const uint64_t pd = P_MN ? sw128_mnmajor_desc(sp, kChunk) : sw128_kmajor_desc(sp);
        const uint64_t qd = Q_MN ? sw128_mnmajor_desc(sp + kHalf, kChunk) : sw128_kmajor_desc(sp + kHalf);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k)
          umma_bf16(acc, pd + p_step * k, qd + q_step * k, idesc, (kb != part0 || k != 0) ? 1u : 0u);
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
  const int parts = is_logits(OP) ? (kb1 - kb0 + p.chunk_blocks - 1) / p.chunk_blocks : 1;
  switch (splits) {
    case 1: finish_tile<OP, TN, 1>(p, parts, smem, tmem_base, rank, m0, n0, warp, lane, wait); break;
    case 2: finish_tile<OP, TN, 2>(p, parts, smem, tmem_base, rank, m0, n0, warp, lane, wait); break;
    case 4: finish_tile<OP, TN, 4>(p, parts, smem, tmem_base, rank, m0, n0, warp, lane, wait); break;
    default:  // 128-row tiles are split in 8 only for long fp32 weight gradients
      if constexpr (TN != 128 || OP == OP_DW) finish_tile<OP, TN, 8>(p, parts, smem, tmem_base, rank, m0, n0, warp, lane, wait);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols<OP, TN>());
  }
}

template <int OP, int TN, bool CUT>
int launch_narrow(const typename Wide<OP>::Params& p, int splits, cudaStream_t st, const char* who) {
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

constexpr int kCutFrom = 32;  // copies of W below 32 rows keep the producer behind

}  // namespace
}  // namespace zgb
