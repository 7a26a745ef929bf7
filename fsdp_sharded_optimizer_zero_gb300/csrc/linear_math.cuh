// Device-side arithmetic of the linear unit's epilogues and of the 8-bit activation
// checkpoints: the activations and their derivatives, and the coding of a group of 32
// values. Everything is fp32; the library is built with -fmad=false, so the fused
// multiply-adds are written out.
#pragma once

#include "device_common.cuh"

namespace zgb {

// ------------------------------------------------------------------------------------
// pairs of fp32: one instruction for two lanes' worth of add, multiply and fused multiply-add.
// The epilogues run beside tensor-core work at the power limit, where each instruction's issue
// is paid in clock rate as much as in time.
// ------------------------------------------------------------------------------------
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 f2_both(float x) { return f2_make(x, x); }
__device__ __forceinline__ void f2_split(f2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t f2_to_bf16x2(f2 v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ f2 f2_from_bf16x2(uint32_t w) { return f2_make(bf16_lo(w), bf16_hi(w)); }

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
// max(m, |a|, |b|)
__device__ __forceinline__ float amax2(float m, f2 v) {
  float a, b, r;
  f2_split(v, a, b);
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

constexpr float kHalfLog2e = 0.72134752044448170f;  // log2(e) / 2
constexpr float kGeluA = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;                 // the cubic term of the tanh form
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// 2^8 / (1 + exp(-x)) from m = -x log2(e) / 2 - 4: with h = 2^m, h^2 = 2^-8 exp(-x), so
// 1 / (h^2 + 2^-8). The factor 2^8 keeps the reciprocal normal wherever the sigmoid is more than
// the smallest subnormal bf16; halving the exponent keeps h in range. Fast exponential and
// reciprocal, and the 4 in the argument, whose rounding it makes 2^-22: relative error within
// 2^-20 + |x| 2^-22 (measured over every bf16 number, derivatives in fp32: 2^-21.4 near 0, 2^-18.1
// at -64 .. -90). That is far inside the bf16 rounding of most of what it goes into; db sums it
// unrounded. h -> inf gives 0, h -> 0 gives 2^8, NaN stays.
__device__ __forceinline__ f2 sigmoid256(f2 m) {
  float a, b, ra, rb;
  f2_split(m, a, b);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ra) : "f"(a));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(rb) : "f"(b));
  const f2 h = f2_make(ra, rb);
  f2_split(f2_fma(h, h, f2_both(0.00390625f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ra) : "f"(a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rb) : "f"(b));
  return f2_make(ra, rb);
}

// Phi(a) - 1 for a = |x| held to 60 (where it is 0), and e = exp(-a^2 / 2), which the density shares.
// 1 - Phi(a) = e / 2 * erfcx(a / sqrt 2), and erfcx(a / sqrt 2) = t P(t) with t = 1 / (1 + 0.36 a), P of
// degree 8 (here times -1/2), fitted here for the least largest relative error over 0 <= a <= 40
// (weighted least squares, weights iterated): 9.1e-8. So the tail keeps its relative precision, at
// one exponential and one reciprocal.
__device__ __forceinline__ f2 normal_tail(f2 a, f2& e) {
  float u, v, ta, tb, ea, eb;
  f2_split(f2_fma(a, f2_both(0.36f), f2_both(1.0f)), u, v);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ta) : "f"(u));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(tb) : "f"(v));
  const f2 t = f2_make(ta, tb);
  f2_split(f2_mul(f2_mul(a, a), f2_both(-kHalfLog2e)), ea, eb);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ea) : "f"(ea));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(eb) : "f"(eb));
  e = f2_make(ea, eb);
  f2 p = f2_both(-0.5f * -0.060481980f);
  p = f2_fma(p, t, f2_both(-0.5f * 0.27903997f));
  p = f2_fma(p, t, f2_both(-0.5f * -0.44723977f));
  p = f2_fma(p, t, f2_both(-0.5f * 0.21477633f));
  p = f2_fma(p, t, f2_both(-0.5f * -0.00079324538f));
  p = f2_fma(p, t, f2_both(-0.5f * 0.19208115f));
  p = f2_fma(p, t, f2_both(-0.5f * 0.24801837f));
  p = f2_fma(p, t, f2_both(-0.5f * 0.28736386f));
  p = f2_fma(p, t, f2_both(-0.5f * 0.28723533f));
  return f2_mul(f2_mul(p, t), e);
}
__device__ __forceinline__ f2 abs_to_60(f2 x) {
  float a, b;
  f2_split(x, a, b);
  return f2_make(fminf(fabsf(a), 60.0f), fminf(fabsf(b), 60.0f));
}

// act(x). The tanh form of GELU uses (1 + tanh u) / 2 = 1 / (1 + exp(-2u)): one exponential,
// no cancellation for negative x; where x^2 overflows the argument is infinite with the right
// sign.
template <int ACT>
__device__ __forceinline__ f2 act_fwd(f2 x) {
  if constexpr (ACT == FSDP_ACT_RELU) {
    float a, b;
    f2_split(x, a, b);
    return f2_make(a < 0.0f ? 0.0f : a, b < 0.0f ? 0.0f : b);  // NaN stays
  }
  if constexpr (ACT == FSDP_ACT_GELU) {  // max(x, 0) - |x| (1 - Phi(|x|)); a NaN comes through the maximum
    float a, b;
    f2 e;
    f2_split(x, a, b);
    const f2 m = abs_to_60(x);
    return f2_fma(m, normal_tail(m, e), f2_make(max_nan(a, 0.0f), max_nan(b, 0.0f)));
  }
  if constexpr (ACT == FSDP_ACT_GELU_TANH) {
    const f2 w = f2_fma(f2_mul(x, x), f2_both(-kGeluA * kGeluB * kHalfLog2e), f2_both(-kGeluA * kHalfLog2e));
    return f2_mul(f2_mul(x, f2_both(0.00390625f)), sigmoid256(f2_fma(x, w, f2_both(-4.0f))));
  }
  if constexpr (ACT == FSDP_ACT_SILU)
    return f2_mul(f2_mul(x, f2_both(0.00390625f)), sigmoid256(f2_fma(x, f2_both(-kHalfLog2e), f2_both(-4.0f))));
  return x;
}

// act'(x); NaN for NaN, so that a checkpoint's NaN group never looks like a zero gradient
template <int ACT>
__device__ __forceinline__ f2 act_grad(f2 x) {
  if constexpr (ACT == FSDP_ACT_RELU) {
    float a, b;
    f2_split(x, a, b);
    return f2_make(a > 0.0f ? 1.0f : a != a ? a : 0.0f, b > 0.0f ? 1.0f : b != b ? b : 0.0f);
  }
  if constexpr (ACT == FSDP_ACT_GELU) {  // Phi(x) + x phi(x)
    float a, b, qa, qb, ua, ub;
    f2 e;
    const f2 q = normal_tail(abs_to_60(x), e);
    f2_split(q, qa, qb);
    f2_split(f2_add(q, f2_both(1.0f)), ua, ub);
    f2_split(x, a, b);
    return f2_fma(f2_mul(x, e), f2_both(kInvSqrt2Pi), f2_make(a < 0.0f ? -qa : ua, b < 0.0f ? -qb : ub));
  }
  if constexpr (ACT == FSDP_ACT_GELU_TANH) {
    // s + x s (1 - s) du with du = A (1 + 3 B x^2). Past |x| = 100 s is 0 or 1: holding x^2
    // there keeps the last term from being 0 * inf.
    float a, b;
    f2_split(f2_mul(x, x), a, b);
    const f2 p = f2_make(min_nan(a, 1e4f), min_nan(b, 1e4f));
    const f2 w = f2_fma(p, f2_both(-kGeluA * kGeluB * kHalfLog2e), f2_both(-kGeluA * kHalfLog2e));
    const f2 r = sigmoid256(f2_fma(x, w, f2_both(-4.0f)));
    const f2 s = f2_mul(r, f2_both(0.00390625f)), q = f2_fma(r, f2_both(-0.00390625f), f2_both(1.0f));
    const f2 du = f2_fma(p, f2_both(3.0f * kGeluA * kGeluB), f2_both(kGeluA));
    return f2_fma(f2_mul(f2_mul(x, s), q), du, s);
  }
  if constexpr (ACT == FSDP_ACT_SILU) {  // s (1 + x (1 - s))
    const f2 r = sigmoid256(f2_fma(x, f2_both(-kHalfLog2e), f2_both(-4.0f)));
    const f2 q = f2_fma(r, f2_both(-0.00390625f), f2_both(1.0f));
    return f2_mul(f2_mul(r, f2_both(0.00390625f)), f2_fma(x, q, f2_both(1.0f)));
  }
  return f2_both(1.0f);
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
// four codes of two pairs, first in the lowest byte: x / 2^e + 1.5 * 2^23 holds the rounded
// integer in its low byte
__device__ __forceinline__ uint32_t ckpt_code4(f2 x, f2 y, float inv) {
  float a, b, c, d;
  f2_split(f2_fma(x, f2_both(inv), f2_both(kRoundMagic)), a, b);
  f2_split(f2_fma(y, f2_both(inv), f2_both(kRoundMagic)), c, d);
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
// the pair of values of codes 2 i, 2 i + 1 of a word with scale s = 2^e: the biased code in a
// float's low mantissa bits is 2^23 + 128 + code. Both operations are exact; they are separate
// because removing the offset after scaling, in one fused multiply-add, overflows for large s.
__device__ __forceinline__ f2 ckpt_values2(uint32_t word, int i, float s) {
  const uint32_t v = word ^ 0x80808080u;
  const f2 w = f2_make(__uint_as_float(__byte_perm(v, 0x4B000000u, 0x7540 + 2 * i)),
                       __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7541 + 2 * i)));
  return f2_mul(f2_add(w, f2_both(-8388736.0f)), f2_both(s));
}

// values past the largest code of b = 248, held to it; inputs that are not finite (b = 255)
// are zeroed, so that their codes are 0
__device__ __forceinline__ f2 ckpt_clamped(f2 v, uint32_t b) {
  float x, y;
  f2_split(v, x, y);
  return b == 255u ? 0ull : f2_make(fminf(fmaxf(x, -kCodeLimit), kCodeLimit), fminf(fmaxf(y, -kCodeLimit), kCodeLimit));
}

}  // namespace zgb
