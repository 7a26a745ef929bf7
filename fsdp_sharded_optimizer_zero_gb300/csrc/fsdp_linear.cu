// The linear unit with its epilogue: forward (bias, activation, residual, the kept
// pre-activation), input gradient (activation's derivative, residual gradient) and weight
// gradient (from bf16 or 8-bit activations).
//
// One simple kernel for the three products: a 32 x 32 output tile per block of 256 threads,
// operands staged in shared memory as fp32, fp32 fused multiply-adds. 32 columns are one
// group of the 8-bit checkpoint, so the epilogue runs row by row over the staged tile.
#include <string.h>

#include <algorithm>

#include "linear_math.cuh"

namespace zgb {
namespace {

enum { OP_FWD, OP_DX, OP_DW };

struct LinearParams {
  const uint16_t* w[kGemmMaxPieces];  // row shards of W [rows_out, k_in]
  int shard_rows;
  int m, n, k;                // the product: out [m, n], contraction over k
  const uint16_t *a, *b;      // fwd: X; dx: dZ; dw: a = dZ, b = X (bf16)
  const int8_t* b_codes;      // dw: X in 8 bits
  const uint8_t* b_scales;
  const uint16_t *bias, *res;
  int act;
  const uint16_t* z_in;       // dx: the kept pre-activation
  const int8_t* zc_in;
  const uint8_t* zs_in;
  uint16_t* out;              // bf16 output
  float* out32;               // dw: fp32 output
  uint16_t* z;                // fwd: kept pre-activation
  int8_t* zc;
  uint8_t* zs;
  float scale;
};

template <int OP>
__device__ __forceinline__ float load_a(const LinearParams& p, int i, int k) {
  if (i >= p.m || k >= p.k) return 0.0f;
  if constexpr (OP == OP_DW) return bf16_bits_to_f32(p.a[static_cast<size_t>(k) * p.m + i]);
  return bf16_bits_to_f32(p.a[static_cast<size_t>(i) * p.k + k]);
}
template <int OP>
__device__ __forceinline__ float load_b(const LinearParams& p, int j, int k) {
  if (j >= p.n || k >= p.k) return 0.0f;
  if constexpr (OP == OP_FWD) {
    const int s = j / p.shard_rows;
    return bf16_bits_to_f32(p.w[s][static_cast<size_t>(j - s * p.shard_rows) * p.k + k]);
  } else if constexpr (OP == OP_DX) {
    const int s = k / p.shard_rows;
    return bf16_bits_to_f32(p.w[s][static_cast<size_t>(k - s * p.shard_rows) * p.n + j]);
  } else {
    const size_t at = static_cast<size_t>(k) * p.n + j;
    if (!p.b_codes) return bf16_bits_to_f32(p.b[at]);
    const float s = ckpt_scale(p.b_scales[static_cast<size_t>(k) * ((p.n + 31) / 32) + j / 32]);
    return __fmul_rn(static_cast<float>(p.b_codes[at]), s);
  }
}

// the 32 columns col0 .. of one output row, from their fp32 sums
template <int OP>
__device__ void epilogue_row(const LinearParams& p, int row, int col0, const float* acc) {
  const int n = min(32, p.n - col0);
  const size_t at = static_cast<size_t>(row) * p.n + col0;
  const size_t group = static_cast<size_t>(row) * ((p.n + 31) / 32) + col0 / 32;
  if constexpr (OP == OP_DW) {
    for (int j = 0; j < n; ++j) {
      const float v = __fmul_rn(acc[j], p.scale);
      if (p.out32) p.out32[at + j] = v;
      else p.out[at + j] = f32_to_bf16_bits(v);
    }
  } else {
    float amax = 0.0f;
    for (int j = 0; j < n; ++j) {
      float v = acc[j];
      if constexpr (OP == OP_FWD) {
        if (p.bias) v = __fadd_rn(v, bf16_bits_to_f32(p.bias[col0 + j]));
        if (p.z) p.z[at + j] = f32_to_bf16_bits(v);
        amax = max_nan(amax, fabsf(v));
        with_act(p.act, [&](auto a) { v = act_fwd<decltype(a)::value>(v); });
      } else if (p.act != FSDP_ACT_NONE) {
        const float z = p.z_in ? bf16_bits_to_f32(p.z_in[at + j])
                               : __fmul_rn(static_cast<float>(p.zc_in[at + j]), ckpt_scale(p.zs_in[group]));
        with_act(p.act, [&](auto a) { v = __fmul_rn(v, act_grad<decltype(a)::value>(z)); });
      }
      if (p.res) v = __fadd_rn(v, bf16_bits_to_f32(p.res[at + j]));
      p.out[at + j] = f32_to_bf16_bits(v);
    }
    if (OP == OP_FWD && p.zc) {
      const uint32_t b = ckpt_byte(amax);
      const float inv = ckpt_inv_scale(b);
      for (int j = 0; j < n; ++j) {
        float v = acc[j];
        if (p.bias) v = __fadd_rn(v, bf16_bits_to_f32(p.bias[col0 + j]));
        if (b >= 248u) v = ckpt_clamped(v, b);
        p.zc[at + j] = static_cast<int8_t>(ckpt_code_word(v, inv) & 0xFFu);
      }
      p.zs[group] = static_cast<uint8_t>(b);
    }
  }
}

template <int OP>
__global__ void __launch_bounds__(256) linear_kernel(const __grid_constant__ LinearParams p) {
  __shared__ float sa[32][33], sb[32][33];  // [k][row], [k][column]
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int tiles_n = (p.n + 31) / 32;
  const int64_t tiles = static_cast<int64_t>((p.m + 31) / 32) * tiles_n;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int i0 = static_cast<int>(tile / tiles_n) * 32, j0 = static_cast<int>(tile % tiles_n) * 32;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};  // rows ty + 8 q, column tx
    for (int k0 = 0; k0 < p.k; k0 += 32) {
      for (int q = 0; q < 4; ++q) {
        const int t = ty + 8 * q;
        // lanes along the operand's contiguous index
        if constexpr (OP == OP_DW) sa[t][tx] = load_a<OP>(p, i0 + tx, k0 + t);
        else sa[tx][t] = load_a<OP>(p, i0 + t, k0 + tx);
        if constexpr (OP == OP_FWD) sb[tx][t] = load_b<OP>(p, j0 + t, k0 + tx);
        else sb[t][tx] = load_b<OP>(p, j0 + tx, k0 + t);
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int q = 0; q < 4; ++q) acc[q] = __fmaf_rn(sa[k][ty + 8 * q], sb[k][tx], acc[q]);
      __syncthreads();
    }
    for (int q = 0; q < 4; ++q) sa[ty + 8 * q][tx] = acc[q];
    __syncthreads();
    if (threadIdx.x < 32 && i0 + static_cast<int>(threadIdx.x) < p.m)
      epilogue_row<OP>(p, i0 + threadIdx.x, j0, sa[threadIdx.x]);
    __syncthreads();
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int OP>
int launch(const LinearParams& p, cudaStream_t st, const char* who) {
  const int64_t tiles = static_cast<int64_t>((p.m + 31) / 32) * ((p.n + 31) / 32);
  linear_kernel<OP><<<static_cast<unsigned int>(std::min<int64_t>(tiles, 1 << 20)), 256, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
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

int load_shards(LinearParams* p, int n, const zero_bf16* const w_shards[], int64_t rows_out, const char* who) {
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
    p->w[q] = w_shards[q];
  }
  p->shard_rows = static_cast<int>(rows_out / n);
  return ZERO_OK;
}

}  // namespace
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
  if ((rc = load_shards(&p, n_ranks, w_shards, rows_out, who))) return rc;
  if (act < FSDP_ACT_NONE || act > FSDP_ACT_SILU)
    return set_error(ZERO_ERR_INVALID_ARG, "%s: act %d is not one of FSDP_ACT_*", who, act);
  if (!X || !Y) return set_error(ZERO_ERR_INVALID_ARG, "%s: X or Y is NULL", who);
  if ((z_codes != nullptr) != (z_scales != nullptr) || (z && z_codes))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: keep Z as z, or as both z_codes and z_scales, or not at all", who);
  if (!aligned16(X) || !aligned16(bias) || !aligned16(residual) || !aligned16(Y) || !aligned16(z) ||
      !aligned16(z_codes) || !aligned16(z_scales))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: every buffer must be 16-byte aligned", who);
  p.m = static_cast<int>(m_tokens), p.n = static_cast<int>(rows_out), p.k = static_cast<int>(k_in);
  p.a = X, p.bias = bias, p.res = residual, p.act = act;
  p.out = Y, p.z = z, p.zc = z_codes, p.zs = z_scales;
  return launch<OP_FWD>(p, reinterpret_cast<cudaStream_t>(stream), who);
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
  if ((rc = load_shards(&p, n_ranks, w_shards, rows_out, who))) return rc;
  if (!dZ || !dX) return set_error(ZERO_ERR_INVALID_ARG, "%s: dZ or dX is NULL", who);
  if ((rc = check_kept_activation(z, z_codes, z_scales, act, who))) return rc;
  if (!aligned16(dZ) || !aligned16(residual) || !aligned16(dX))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: every buffer must be 16-byte aligned", who);
  p.m = static_cast<int>(m_tokens), p.n = static_cast<int>(k_in), p.k = static_cast<int>(rows_out);
  p.a = dZ, p.res = residual, p.act = act, p.out = dX;
  if (act != FSDP_ACT_NONE) p.z_in = z, p.zc_in = z_codes, p.zs_in = z_scales;
  return launch<OP_DX>(p, reinterpret_cast<cudaStream_t>(stream), who);
}

extern "C" int fsdp_linear_dw(const zero_bf16* dZ, const zero_bf16* x, const int8_t* x_codes, const uint8_t* x_scales,
                              int64_t m_tokens, int64_t rows_out, int64_t k_in, float scale, float* dW,
                              zero_bf16* dW_bf16, zero_stream_t stream) {
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
      !aligned16(dW_bf16))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: every buffer must be 16-byte aligned", who);
  p.m = static_cast<int>(rows_out), p.n = static_cast<int>(k_in), p.k = static_cast<int>(m_tokens);
  p.a = dZ, p.b = x, p.b_codes = x_codes, p.b_scales = x_scales, p.scale = scale;
  p.out32 = dW, p.out = dW_bf16;
  return launch<OP_DW>(p, reinterpret_cast<cudaStream_t>(stream), who);
}
