// Device-side arithmetic of the linear unit's epilogues and of the 8-bit activation
// checkpoints: the activations and their derivatives, and the coding of a group of 32
// values. Everything is fp32; the library is built with -fmad=false, so the fused
// multiply-adds are written out.
#pragma once

#include "device_common.cuh"

namespace zgb {

// ------------------------------------------------------------------------------------
// activations
// ------------------------------------------------------------------------------------
// min / max that return NaN when an operand is one (the IEEE-754 2019 minimum / maximum)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 1 / (1 + exp(-x)) = (x >= 0 ? 1 : t) / (1 + t) with t = exp(-|x|): the denominator stays in
// [1, 2], so the approximate reciprocal needs no scaling, and small results keep their
// precision down to the subnormals: t is the square of 2^(-|x| log2(e) / 2), which is normal
// for every t that is not zero. Relative error a few 2^-22 for |x| < 20, |x| 2^-24 beyond,
// far inside the bf16 rounding of what it goes into; 0 and 1 at the ends, NaN for NaN.
__device__ __forceinline__ float sigmoid_fast(float x) {
  float h, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(__fmul_rn(fabsf(x), -0.72134752f)));
  const float t = __fmul_rn(h, h);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, t)));
  return __fmul_rn(x >= 0.0f ? 1.0f : t, r);
}

constexpr float kGeluA = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;                // the cubic term of the tanh form
constexpr float kSqrtHalf = 0.70710678118654752f;  // 1 / sqrt(2)
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// act(x). The tanh form of GELU uses (1 + tanh u) / 2 = 1 / (1 + exp(-2u)): one exponential,
// no cancellation for negative x.
template <int ACT>
__device__ __forceinline__ float act_fwd(float x) {
  if constexpr (ACT == FSDP_ACT_RELU) return x < 0.0f ? 0.0f : x;  // NaN stays
  if constexpr (ACT == FSDP_ACT_GELU) return __fmul_rn(__fmul_rn(0.5f, x), erfcf(__fmul_rn(-kSqrtHalf, x)));
  if constexpr (ACT == FSDP_ACT_GELU_TANH) {
    const float u = __fmul_rn(__fmul_rn(kGeluA, x), __fmaf_rn(__fmul_rn(kGeluB, x), x, 1.0f));
    return __fmul_rn(x, sigmoid_fast(u));
  }
  if constexpr (ACT == FSDP_ACT_SILU) return __fmul_rn(x, sigmoid_fast(x));
  return x;
}

// act'(x); NaN for NaN, so that a checkpoint's NaN group never looks like a zero gradient
template <int ACT>
__device__ __forceinline__ float act_grad(float x) {
  if constexpr (ACT == FSDP_ACT_RELU) return x > 0.0f ? 1.0f : x != x ? x : 0.0f;
  if constexpr (ACT == FSDP_ACT_GELU) {
    const float pdf = __fmul_rn(kInvSqrt2Pi, __expf(__fmul_rn(__fmul_rn(-0.5f, x), x)));
    return __fmaf_rn(x, pdf, __fmul_rn(0.5f, erfcf(__fmul_rn(-kSqrtHalf, x))));
  }
  if constexpr (ACT == FSDP_ACT_GELU_TANH) {
    // past |x| = 30 the sigmoid is 0 or 1 exactly: clamping keeps x^2 * 0 from being inf * 0
    const float c = min_nan(max_nan(x, -30.0f), 30.0f), c2 = __fmul_rn(c, c);
    const float s = sigmoid_fast(__fmul_rn(__fmul_rn(kGeluA, c), __fmaf_rn(kGeluB, c2, 1.0f)));
    const float du = __fmul_rn(kGeluA, __fmaf_rn(3.0f * kGeluB, c2, 1.0f));
    return __fmaf_rn(__fmul_rn(__fmul_rn(c, s), __fsub_rn(1.0f, s)), du, s);
  }
  if constexpr (ACT == FSDP_ACT_SILU) {
    const float s = sigmoid_fast(x);
    return __fmul_rn(s, __fmaf_rn(x, __fsub_rn(1.0f, s), 1.0f));
  }
  return 1.0f;
}

// f(integral constant) for the run-time activation (already checked on the host)
template <int V>
struct ActTag {
  static constexpr int value = V;
};
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case FSDP_ACT_RELU: f(ActTag<FSDP_ACT_RELU>{}); break;
    case FSDP_ACT_GELU: f(ActTag<FSDP_ACT_GELU>{}); break;
    case FSDP_ACT_GELU_TANH: f(ActTag<FSDP_ACT_GELU_TANH>{}); break;
    case FSDP_ACT_SILU: f(ActTag<FSDP_ACT_SILU>{}); break;
    default: f(ActTag<FSDP_ACT_NONE>{}); break;
  }
}

// ------------------------------------------------------------------------------------
// 8-bit checkpoint: a group of 32 columns of one row shares the power of two 2^e, e = b -
// 127 with b the stored byte; a value is code * 2^e with code in [-127, 127]. 2^e is the
// least power of two with amax / 2^e < 127.5, so rounding to the nearest code is off by at
// most 2^e / 2 and never past 127. A 7-bit integer times a power of two is exact in bf16.
// b is kept in 1 .. 248: below, values under 2^-126 round to its multiples (also off by
// half of one at most); above, amax from 127.5 * 2^121 on is coded as 127 * 2^121. A group
// with an infinity or a NaN has b = 255 and zero codes: 0 * inf reads back as NaN.
// ------------------------------------------------------------------------------------
constexpr int kCkptGroup = 32;
constexpr float kRoundMagic = 12582912.0f;   // 1.5 * 2^23: x + magic holds rint(x) in its low bits
constexpr float kCodeLimit = 0x1.FCp+127f;   // 127 * 2^121

// the scale byte of a group whose largest magnitude is amax (NaN if it holds one)
__device__ __forceinline__ uint32_t ckpt_byte(float amax) {
  if (!(amax < __int_as_float(0x7f800000))) return 255u;
  const int b = static_cast<int>((__float_as_uint(amax) + 0x10000u) >> 23) - 6;
  return static_cast<uint32_t>(min(max(b, 1), 248));
}
// 2^(127 - b), which a value is multiplied by before rounding; 0 for b = 255
__device__ __forceinline__ float ckpt_inv_scale(uint32_t b) { return __uint_as_float(b == 255u ? 0u : (254u - b) << 23); }
// 2^(b - 127); inf for b = 255
__device__ __forceinline__ float ckpt_scale(uint32_t b) { return __uint_as_float(b << 23); }
// the code of x in a word whose low byte holds it (the other bytes: the magic number)
__device__ __forceinline__ uint32_t ckpt_code_word(float x, float inv) {
  return __float_as_uint(__fmaf_rn(x, inv, kRoundMagic));
}
// four codes, first in the lowest byte
__device__ __forceinline__ uint32_t ckpt_code4(float a, float b, float c, float d, float inv) {
  const uint32_t lo = __byte_perm(ckpt_code_word(a, inv), ckpt_code_word(b, inv), 0x0040);
  const uint32_t hi = __byte_perm(ckpt_code_word(c, inv), ckpt_code_word(d, inv), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
// value `i` of a word of four codes (biased: word ^ 0x80808080) with scale s = 2^e: the byte
// in a float's low mantissa bits is 2^23 + 128 + code; both operations are exact (removing
// the offset after scaling, in one fused multiply-add, would overflow for large s)
__device__ __forceinline__ float ckpt_value(uint32_t biased, int i, float s) {
  const uint32_t w = __byte_perm(biased, 0x4B000000u, 0x7540 + i);
  return __fmul_rn(__fsub_rn(__uint_as_float(w), 8388736.0f), s);
}

// values past the largest code of b = 248, held to it; inputs that are not finite (b = 255)
// are zeroed, so that their codes are 0
__device__ __forceinline__ float ckpt_clamped(float x, uint32_t b) {
  return b == 255u ? 0.0f : fminf(fmaxf(x, -kCodeLimit), kCodeLimit);
}

}  // namespace zgb
