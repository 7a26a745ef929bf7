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
#include "linear_narrow.cuh"

namespace zgb {
namespace {

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

// narrow kernel: what 4 columns of a row read beside their sums
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
};

// 4 columns of one output row per lane, 32 lanes across 128 columns; the 8 lanes of a group of 32
// columns share its scale byte through shuffles. bias: the columns' biases (fwd, where there are
// any). Called by whole warps.
template <int OP, int ACT>
__device__ __forceinline__ void epilogue4(const typename Wide<OP>::Params& p, int row, int col, uint2 bias, const Side4<OP>& side,
                                          f2 (&v)[2]) {
  const size_t at = static_cast<size_t>(row) * p.n + col;
  const bool live = row < p.m && col < p.n;
  if constexpr (OP == OP_DW) {
    const f2 scale = f2_both(dw_scale(p.scale, p.count));
    v[0] = f2_mul(v[0], scale), v[1] = f2_mul(v[1], scale);
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

// The epilogue warps' role. A thread has a row of the tile; a warp's 64-column chunk of bf16 output
// goes through one of its staging buffers. A bf16 tensor that the epilogue reads beside the sums
// (residual, kept activation) is loaded into the buffers before the sums are ready, and each thread
// replaces its row by the output.
template <int OP>
__device__ __forceinline__ void wide_epilogue(const typename Wide<OP>::Params& p, uint8_t* smem, uint32_t tmem_base,
                                              uint32_t accf_bar, uint32_t acce_bar, volatile int* abort, int warp,
                                              int lane, uint32_t rank, int pair, int pairs, int num_m, int num_n) {
  using C = Wide<OP>;
  const int q = warp & 3;            // the tensor-memory lane quarter this warp may read
  const int part = (warp - 2) >> 2;  // which of the quarter's warps
  uint8_t* stage = smem + C::STAGES * C::STAGE + static_cast<uint32_t>(warp - 2) * 8192u;
  uint8_t* bias_sm = smem + C::STAGES * C::STAGE + C::EPI;
  const int groups = (p.n + 31) / 32;
  const uint16_t* side_src = nullptr;
  if constexpr (!is_dw(OP)) side_src = OP == OP_DX && p.z_in ? p.z_in : p.res;
  uint32_t i = 0, bias_turn = 0;
  uint32_t stores = 0;  // fp32 dW: bulk stores this warp has made
  const float scale = is_dw(OP) ? dw_scale(p.scale, p.count) : 1.0f;
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
    if constexpr (!is_dw(OP)) {
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
        store_sums<C::EPI_COLS>(&p.out, taddr, r0, c0, p.n, scale, chunk > 0, stage, stores, lane);
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
            if (!is_dw(OP) && side_src) {
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
          if constexpr (is_dw(OP)) {
            const f2 s = f2_both(scale);
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
            stage_store(buf, p.y, r0, col0 - 32 * h, p.m, p.n, p.n, lane);
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

// the product's operands as the entry points get them
struct Operands {
  int n_shards;
  const uint16_t* const* w;  // fwd, dx
  const uint16_t* a;         // X, dZ, dZ
  int64_t lda;               // its rows' distance
  const uint16_t* x;         // dw: X
};

// dW in bf16 of few tokens, us with eight epilogue warps (with four): 32000 x 4096 from 1 49 (68), from 128 51 (71), from
// 256 60 (76), from 512 89 (88); 50257 x 768 from 256 23.4 (26.4), from 400 30.3 (29.1)
constexpr int kShortBlocks = 4;

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
    if ((rc = fast ? encode_mn(&p.a, o.a, p.k, p.m, o.lda, who) : encode(&p.a, o.a, p.k, p.m, o.lda, 64, BK, false, who)))
      return rc;
    if ((rc = fast ? encode_mn(&p.b, o.x, p.k, p.n, p.n, who) : encode(&p.b, o.x, p.k, p.n, p.n, 64, BK, false, who)))
      return rc;
  } else {
    if ((rc = encode(&p.a, o.a, p.m, p.k, o.lda, BK, c.wide ? 128 : c.tn, false, who))) return rc;
    if ((rc = encode_w(p, o.n_shards, o.w, static_cast<int64_t>(o.n_shards) * p.shard_rows, OP == OP_FWD, kCutFrom, false, &fast,
                       who)))
      return rc;
  }
  if (c.wide && fp32 && (rc = encode(&p.out, p.y32, p.m, p.n, p.n, 32, 32, true, who))) return rc;
  if constexpr (OP != OP_DW)
    if (p.w_levels > 1) {
      if (c.wide) return launch_wide<OP, COPIES_CUT>(p, st, who);
      if (c.tn == 32) return launch_narrow<OP, 32, true>(p, c.splits, st, who);
      if (c.tn == 64) return launch_narrow<OP, 64, true>(p, c.splits, st, who);
      return launch_narrow<OP, 128, true>(p, c.splits, st, who);
    }
  if constexpr (OP == OP_DW)
    if (c.wide && !fp32 && blocks <= kShortBlocks)
      return fast ? launch_wide<OP_DW_SHORT, COPIES_ONE>(p, st, who) : launch_wide<OP_DW_SHORT, COPIES_EQUAL>(p, st, who);
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

int launch_linear_dw(const uint16_t* dZ, int64_t ldz, const uint16_t* x, int64_t m_tokens, int64_t rows_out, int64_t k_in,
                     float scale, const float* count, uint16_t* dW, cudaStream_t st, const char* who) {
  LinearParams p;
  memset(&p, 0, sizeof(p));
  p.m = static_cast<int>(rows_out), p.n = static_cast<int>(k_in), p.k = static_cast<int>(m_tokens);
  p.scale = scale, p.count = count, p.y = dW;
  return launch<OP_DW>(p, Operands{0, nullptr, dZ, ldz, x}, st, who);
}

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
  const Operands o{n_ranks, w_shards, X, k_in, nullptr};
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
  const Operands o{n_ranks, w_shards, dZ, rows_out, nullptr};
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
  const Operands o{0, nullptr, dZ, rows_out, x};
  return launch<OP_DW>(p, o, reinterpret_cast<cudaStream_t>(stream), who);
}
