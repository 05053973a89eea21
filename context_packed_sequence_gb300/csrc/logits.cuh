// Arithmetic shared by the kernels over rows of logits: element types, the
// running maximum and sum of a softmax, and pairs of floats for the row
// scalars that are differences of close numbers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "thd_internal.cuh"

namespace thd {

// log2(e) / temperature as the sum of two floats.  hi is rounded towards zero,
// so lo > 0 and d*hi + d*lo never mixes infinities of both signs.  A softmax
// scaled by hi alone is the softmax of a temperature up to 6e-8 off: the same
// error in every row, which sums of log-probabilities over a document add up.
struct LogitScale {
  float hi, lo;
  float tau, inv_tau;
};

inline LogitScale make_logit_scale(float temperature) {
  LogitScale s;
  const double c = 1.4426950408889634 / static_cast<double>(temperature);
  s.hi = static_cast<float>(c);
  if (static_cast<double>(s.hi) >= c) s.hi = std::nextafterf(s.hi, 0.0f);
  s.lo = static_cast<float>(c - static_cast<double>(s.hi));
  s.tau = temperature;
  s.inv_tau = static_cast<float>(1.0 / static_cast<double>(temperature));
  return s;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(d * log2(e) / temperature) = exp(d / temperature)
__device__ __forceinline__ float exp_scaled(float d, LogitScale c) { return ex2(fmaf(d, c.hi, d * c.lo)); }

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// ---------------------------------------------------------------------------
// softmax statistics
// ---------------------------------------------------------------------------

// Running maximum m of some logits and the sum s of exp((z - shift(m)) / tau).
// The shift is m itself, or 0 while m is not finite: a set whose logits are
// all -inf then has s = 0, one that holds +inf has s = +inf, and a NaN makes
// s NaN, without a case of its own.
struct SoftmaxStat {
  float m, s;
};

__device__ __forceinline__ float softmax_shift(float m) { return fabsf(m) < INFINITY ? m : 0.0f; }

__device__ __forceinline__ SoftmaxStat empty_stat() { return {-INFINITY, 0.0f}; }

// s of a set with maximum m, rescaled to the shift of the larger maximum `to`
__device__ __forceinline__ float rescaled(float m, float s, float to, LogitScale c) {
  if (m == to || s == 0.0f) return s;
  return s * exp_scaled(softmax_shift(m) - softmax_shift(to), c);
}

__device__ __forceinline__ SoftmaxStat join(SoftmaxStat a, SoftmaxStat b, LogitScale c) {
  const float m = fmaxf(a.m, b.m);
  return {m, rescaled(a.m, a.s, m, c) + rescaled(b.m, b.s, m, c)};
}

// A row none of whose logits is above -inf: its probabilities are taken as 0.
__device__ __forceinline__ bool stat_is_empty(SoftmaxStat t) { return t.m == -INFINITY && t.s == 0.0f; }

__device__ __forceinline__ SoftmaxStat warp_join(SoftmaxStat t, LogitScale c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    SoftmaxStat u;
    u.m = __shfl_xor_sync(kFullMask, t.m, o);
    u.s = __shfl_xor_sync(kFullMask, t.s, o);
    t = join(t, u, c);
  }
  return t;
}

// ---------------------------------------------------------------------------
// float pairs: an unevaluated sum hi + lo with |lo| at most an ulp of hi
// ---------------------------------------------------------------------------

struct Pair {
  float hi, lo;
};

// a + b exactly (Knuth, "The Art of Computer Programming", volume 2, 4.2.2);
// with an infinity or a NaN in it lo is 0
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  const float e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return {s, fabsf(s) < INFINITY ? e : 0.0f};
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}

// p * k for a constant k = k_hi + k_lo
__device__ __forceinline__ Pair scaled(Pair p, float k_hi, float k_lo) {
  const float h = p.hi * k_hi;
  const float e = fmaf(p.hi, k_hi, -h) + (p.hi * k_lo + p.lo * k_hi);
  return {h, fabsf(h) < INFINITY ? e : 0.0f};
}

constexpr float kLn2Hi = 0.693147182464599609375f;  // ln 2 rounded to a float
constexpr float kLn2Lo = -1.904654299957767e-9f;    // ln 2 - kLn2Hi

// log2(s) as a whole number plus the logarithm of a number near 1, whose
// error is relative to itself
__device__ __forceinline__ Pair log2_pair(float s) {
  if (!(s >= 1.17549435e-38f && s < INFINITY)) return {log2f(s), 0.0f};
  int32_t bits = __float_as_int(s);
  int32_t ex = (bits >> 23) - 127;
  float f = __int_as_float((bits & 0x007fffff) | 0x3f800000);
  if (f > 1.41421354f) {
    f *= 0.5f;
    ++ex;
  }
  return two_sum(static_cast<float>(ex), log2f(f));
}

// A row's log of its sum (relative to the shift), kept for its scalars.
struct RowNorm {
  float shift;  // softmax_shift(m)
  Pair log_sum;
};

__device__ __forceinline__ RowNorm row_norm(SoftmaxStat t) {
  return {softmax_shift(t.m), scaled(log2_pair(t.s), kLn2Hi, kLn2Lo)};
}

// x / tau for a pair x
__device__ __forceinline__ Pair over_tau(Pair x, LogitScale c) {
  const float q = x.hi / c.tau;
  const float e = (fmaf(-q, c.tau, x.hi) + x.lo) * c.inv_tau;
  return {q, fabsf(q) < INFINITY ? e : 0.0f};
}

// Logarithm of the probability of a logit z, as a pair.  Its error is that of
// the sum: the large numbers z and m are subtracted before anything is rounded.
__device__ __forceinline__ Pair log_prob(float z, const RowNorm& r, LogitScale c) {
  return add(over_tau(two_sum(z, -r.shift), c), {-r.log_sum.hi, -r.log_sum.lo});
}

__device__ __forceinline__ float log_sum_exp(const RowNorm& r, LogitScale c) {
  const Pair n = add(over_tau({r.shift, 0.0f}, c), r.log_sum);
  return n.hi + n.lo;
}

}  // namespace thd
