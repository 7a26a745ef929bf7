// 8-bit activation checkpoints (pack, unpack) and the activation's backward, which reads
// them: streaming kernels, bound by HBM bandwidth.
//
//   pack     x [rows, cols] bf16 -> codes int8, one power-of-two scale byte per 32 columns
//   unpack   act(code * 2^(byte - 127)) -> bf16
//   act_backward   dZ = bf16(dY act'(Z)), db = column sums of dY act'(Z) in fp32
//
// A thread works on 8 columns (16 bytes of bf16, 8 codes), four neighbouring lanes on one
// group of 32. cols is a multiple of 8, so each 8-column unit is whole; the last group of a
// row may have fewer than four units, and the lanes past it hold zeros.
#include <algorithm>

#include "linear_math.cuh"

namespace zgb {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(v[j]), x[2 * j + 1] = bf16_hi(v[j]);
}
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void decode8(const uint2& c, uint32_t byte, float (&x)[8]) {
  const float s = ckpt_scale(byte);
  const uint32_t lo = c.x ^ 0x80808080u, hi = c.y ^ 0x80808080u;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = ckpt_value(lo, j, s), x[4 + j] = ckpt_value(hi, j, s);
}

__global__ void __launch_bounds__(kThreads) ckpt8_pack_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                              int64_t cols, int8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  const int64_t groups = (cols + kCkptGroup - 1) / kCkptGroup, per_row = 4 * groups, total = rows * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  // total and stride are multiples of 4: the four lanes of a group stay together
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += stride) {
    const int64_t row = i / per_row, u = i - row * per_row;
    const bool valid = u * 8 < cols;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (valid) widen8(__ldcs(reinterpret_cast<const uint4*>(x + row * cols + u * 8)), v);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(v[j]));
    const uint32_t four = 0xFu << (threadIdx.x & 28u);
    amax = max_nan(amax, __shfl_xor_sync(four, amax, 1));
    amax = max_nan(amax, __shfl_xor_sync(four, amax, 2));
    const uint32_t b = ckpt_byte(amax);
    if (b >= 248u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = ckpt_clamped(v[j], b);
    }
    const float inv = ckpt_inv_scale(b);
    if (valid)
      *reinterpret_cast<uint2*>(codes + row * cols + u * 8) =
          make_uint2(ckpt_code4(v[0], v[1], v[2], v[3], inv), ckpt_code4(v[4], v[5], v[6], v[7], inv));
    if ((u & 3) == 0) scales[row * groups + (u >> 2)] = static_cast<uint8_t>(b);
  }
}

template <int ACT>
__global__ void __launch_bounds__(kThreads) ckpt8_unpack_kernel(const int8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                                int64_t cols, uint16_t* __restrict__ out) {
  const int64_t groups = (cols + kCkptGroup - 1) / kCkptGroup, units = cols / 8, total = rows * units;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += stride) {
    const int64_t row = i / units, u = i - row * units;
    float v[8];
    decode8(__ldcs(reinterpret_cast<const uint2*>(codes + row * cols + u * 8)), scales[row * groups + (u >> 2)], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_fwd<ACT>(v[j]);
    __stcs(reinterpret_cast<uint4*>(out + row * cols + u * 8), narrow8(v));
  }
}

// One block per strip of 64 columns: 8 lanes across a row's strip, 32 rows at a time. Each
// thread sums its rows in order; the 32 row lanes are then summed in order in shared memory.
template <int ACT, bool Z8>
__global__ void __launch_bounds__(kThreads) act_backward_kernel(const uint16_t* __restrict__ dy,
                                                                const uint16_t* __restrict__ z,
                                                                const int8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                                int64_t cols, uint16_t* dz, float* __restrict__ db) {
  __shared__ float part[32][65];
  const int64_t groups = (cols + kCkptGroup - 1) / kCkptGroup;
  const int lane = threadIdx.x & 7, rl = threadIdx.x >> 3;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane * 8;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (col < cols) {
    for (int64_t row = rl; row < rows; row += 32) {
      float g[8], v[8];
      widen8(*reinterpret_cast<const uint4*>(dy + row * cols + col), g);
      if constexpr (ACT != FSDP_ACT_NONE) {
        if constexpr (Z8)
          decode8(__ldcs(reinterpret_cast<const uint2*>(codes + row * cols + col)), scales[row * groups + (col >> 5)],
                  v);
        else
          widen8(__ldcs(reinterpret_cast<const uint4*>(z + row * cols + col)), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __fmul_rn(g[j], act_grad<ACT>(v[j]));
      }
      if (dz) *reinterpret_cast<uint4*>(dz + row * cols + col) = narrow8(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] = __fadd_rn(sum[j], g[j]);
    }
  }
  if (!db) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[rl][lane * 8 + j] = sum[j];
  __syncthreads();
  if (threadIdx.x < 64) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    float s = part[0][threadIdx.x];
    for (int i = 1; i < 32; ++i) s = __fadd_rn(s, part[i][threadIdx.x]);
    if (c < cols) db[c] = s;
  }
}

unsigned int grid_streaming(int64_t units) {
  const int64_t blocks = (units + kThreads - 1) / kThreads;
  return static_cast<unsigned int>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms()) * 8));
}

template <int ACT>
cudaError_t launch_act_backward(const uint16_t* dy, const uint16_t* z, const int8_t* codes, const uint8_t* scales,
                                int64_t rows, int64_t cols, uint16_t* dz, float* db, cudaStream_t st) {
  const unsigned int grid = static_cast<unsigned int>((cols + 63) / 64);
  if (codes && ACT != FSDP_ACT_NONE)
    act_backward_kernel<ACT, true><<<grid, kThreads, 0, st>>>(dy, z, codes, scales, rows, cols, dz, db);
  else
    act_backward_kernel<ACT, false><<<grid, kThreads, 0, st>>>(dy, z, codes, scales, rows, cols, dz, db);
  return cudaGetLastError();
}

template <int ACT>
cudaError_t launch_unpack(const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* out,
                          cudaStream_t st) {
  ckpt8_unpack_kernel<ACT><<<grid_streaming(rows * (cols / 8)), kThreads, 0, st>>>(codes, scales, rows, cols, out);
  return cudaGetLastError();
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
  const int64_t units = rows * (4 * ((cols + kCkptGroup - 1) / kCkptGroup));
  ckpt8_pack_kernel<<<grid_streaming(units), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, rows, cols,
                                                                                                    codes, scales);
  const cudaError_t e = cudaGetLastError();
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

extern "C" int fsdp_act_backward(const zero_bf16* dY, const zero_bf16* z, const int8_t* z_codes, const uint8_t* z_scales,
                                 int64_t rows, int64_t cols, int act, zero_bf16* dZ, float* db, zero_stream_t stream) {
  const char* who = "fsdp_act_backward";
  int rc = check_shape(rows, cols, who);
  if (rc) return rc;
  if (!dY) return set_error(ZERO_ERR_INVALID_ARG, "%s: dY is NULL", who);
  if (!dZ && !db) return set_error(ZERO_ERR_INVALID_ARG, "%s: dZ and db are both NULL", who);
  if ((rc = check_kept_activation(z, z_codes, z_scales, act, who))) return rc;
  if (!aligned16(dY) || !aligned16(dZ) || !aligned16(db))
    return set_error(ZERO_ERR_INVALID_ARG, "%s: dY, dZ and db must be 16-byte aligned", who);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (act) {
    case FSDP_ACT_RELU: e = launch_act_backward<FSDP_ACT_RELU>(dY, z, z_codes, z_scales, rows, cols, dZ, db, st); break;
    case FSDP_ACT_GELU: e = launch_act_backward<FSDP_ACT_GELU>(dY, z, z_codes, z_scales, rows, cols, dZ, db, st); break;
    case FSDP_ACT_GELU_TANH:
      e = launch_act_backward<FSDP_ACT_GELU_TANH>(dY, z, z_codes, z_scales, rows, cols, dZ, db, st);
      break;
    case FSDP_ACT_SILU: e = launch_act_backward<FSDP_ACT_SILU>(dY, z, z_codes, z_scales, rows, cols, dZ, db, st); break;
    default: e = launch_act_backward<FSDP_ACT_NONE>(dY, nullptr, nullptr, nullptr, rows, cols, dZ, db, st); break;
  }
  return e == cudaSuccess ? ZERO_OK : set_error(ZERO_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}
