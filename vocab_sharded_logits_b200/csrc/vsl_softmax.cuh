// vsl_softmax.cuh - the softmax statistics of a row of vocab-sliced logits,
// shared by the kernels that score given tokens.
//
// For a row of logits l_j at temperature T one pass gives, with e_j =
// exp((l_j - m) / T) for some reference m,
//   z = sum_j e_j,   and where the entropy is asked for   w = sum_j e_j (l_j - m) / T,
// from which, for a token t,
//   log p_t = (l_t - m) / T - log z,     H = log z - w / z.
//
// The token's own term is left out of the sums and added to them at the end, in
// 64 bits: where it is nearly all of z, log p_t is what the others leave, and
// that keeps its digits.
//
// The fast form.  e_j = 2^(c l_j - k) with c = log2(e) / T in float32 and k an
// integer, so a logit costs one fused multiply-add, one ex2 and one addition
// (and a bound and another multiply-add for w): no running maximum is kept.
// k is taken from the largest of the first logits each thread of the CTA
// reads: near the row's maximum, as a rule.  A thread that meets logits far
// above it (its next sixteen sum to more than 2^5) renews its k and takes them
// again: an exponent c l_j - k of up to 40 would have a rounding of up to 2^-19
// in its exponential, one below 5 has 2^-22 at most.  Different k are powers of
// two apart, so bringing sums together costs no rounding.  What it rests on is
// checked afterwards: a row whose sums left [2^-40, 2^60] (a NaN or +inf logit;
// none above -inf) or whose k exceeds 2^20 is done again in the careful form.  c's rounding is a temperature off by at
// most 2^-24, used consistently: log p_t moves by at most 2^-24 of its distance
// from the mean of x.
//
// The careful form keeps each thread's running maximum, e_j = exp((l_j - m) /
// T) with c as a sum of two floats, and rescales when the maximum grows.
#pragma once

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "vsl_internal.h"

namespace vsl {

constexpr double kLn2 = 0.69314718055994530941723212145818;

// log2(e) / T: nearest float (fast form), and as hi + lo with hi <= c, lo > 0
// (careful form: both positive, so l = -inf gives -inf).
struct ExpScale {
  float c, hi, lo;
  double inv_t;      // 1 / T
  double inv_t_fast; // 1 / T as c has it: c ln 2
};

inline ExpScale exp_scale(float temperature) {
  const double c = 1.4426950408889634073599246810019 / static_cast<double>(temperature);
  ExpScale r;
  r.c = static_cast<float>(c);
  r.hi = r.c;
  if (static_cast<double>(r.hi) > c) r.hi = std::nextafterf(r.hi, 0.0f);
  r.lo = static_cast<float>(c - static_cast<double>(r.hi));
  if (!(r.lo > 0.0f)) r.lo = FLT_MIN;
  r.inv_t = 1.0 / static_cast<double>(temperature);
  r.inv_t_fast = static_cast<double>(r.c) * kLn2;
  return r;
}

// ex2.approx is off by at most 1.43e-7 relative on this part and, over a
// binade, by -5.16e-8 in the mean (measured on 2^18 arguments in each of 30
// binades; the errors repeat from one to the next).  A sum of many
// exponentials keeps the mean error, so it is taken out of z, w and p (but not of
// the token's own term, which is exact).
constexpr double kExpMean = 1.0 + 5.16e-8;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// two float32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ------------------------------------------------------------------ fast form

// A thread's sums: z, and w in units of log2 (sum of e times its exponent), as
// two float32 partial sums each.
struct FastSums {
  float2 z, w;
};

// The CTA's k from the largest of the logits its threads read first (0 where
// that is lower than k may be, as masked ones are).
constexpr float kFastMaxK = 1048576.0f;
__device__ __forceinline__ float fast_reference(float top, float c) {
  const float k = rintf(top * c);
  return k < -kFastMaxK ? 0.0f : k;
}

// Four logits.
template <bool ENT>
__device__ __forceinline__ void fast_add(FastSums& s, const float4& x, float c, float k) {
  const float2 cc = make_float2(c, c), kk = make_float2(-k, -k);
  float2 y0 = fma2(make_float2(x.x, x.y), cc, kk), y1 = fma2(make_float2(x.z, x.w), cc, kk);
  if (ENT) {  // an exponential of 0 times a bounded exponent is 0
    y0 = make_float2(max_nan(y0.x, -200.0f), max_nan(y0.y, -200.0f));
    y1 = make_float2(max_nan(y1.x, -200.0f), max_nan(y1.y, -200.0f));
  }
  const float2 e0 = make_float2(exp2_fast(y0.x), exp2_fast(y0.y)), e1 = make_float2(exp2_fast(y1.x), exp2_fast(y1.y));
  s.z = add2(s.z, add2(e0, e1));
  if (ENT) s.w = fma2(e1, y1, fma2(e0, y0, s.w));
}

// A thread's sums brought from k to a larger integer, without rounding (w: but
// for the product's).
template <bool ENT>
__device__ __forceinline__ void fast_rebase(FastSums& s, float k, float to) {
  const float d = k - to;
  const float f = d < -126.0f ? 0.0f : __int_as_float((127 + static_cast<int>(d)) << 23);  // 2^d
  if (ENT) {
    s.w.x = __fmaf_rn(d, s.z.x, s.w.x) * f;
    s.w.y = __fmaf_rn(d, s.z.y, s.w.y) * f;
  }
  s.z.x *= f;
  s.z.y *= f;
}

// 4 N logits.  Sixteen near k sum to 2^4.5 at most (an exponent of 2^(1/2) each);
// above 2^5 k is renewed from the largest of them and they are taken again.
constexpr float kFastBatchMost = 32.0f;
template <bool ENT, int N>
__device__ __forceinline__ void fast_batch(FastSums& s, float& k, const float4 (&v)[N], float c) {
  FastSums b{};
#pragma unroll
  for (int u = 0; u < N; ++u) fast_add<ENT>(b, v[u], c, k);
  if (b.z.x + b.z.y > kFastBatchMost) {
    float top = -FLT_MAX;
#pragma unroll
    for (int u = 0; u < N; ++u) top = fmaxf(top, fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w)));
    const float to = rintf(top * c);
    if (to > k && to <= kFastMaxK) {
      fast_rebase<ENT>(s, k, to);
      k = to;
      b = FastSums{};
#pragma unroll
      for (int u = 0; u < N; ++u) fast_add<ENT>(b, v[u], c, k);
    }
  }
  s.z = add2(s.z, b.z);
  if (ENT) s.w = add2(s.w, b.w);
}

// ------------------------------------------------------------------ careful form

// exp(t / T) (0 for -inf, NaN for NaN).
__device__ __forceinline__ float exp_of(float t, const ExpScale& c) {
  return exp2_fast(__fmaf_rn(t, c.hi, t * c.lo));
}
// t bounded from below, so that its product with an exponential of 0 is 0: at
// -1e18 the exponential is 0 for every T up to 1e6, and a factor of up to 1e20
// (a sum of exponentials, a gradient's coefficient) still gives a finite value.
__device__ __forceinline__ float finite_low(float t) { return fmaxf(t, -1e18f); }

// A thread's sums relative to its running maximum m (w in units of l).  m
// starts at the lowest finite value, so l - m is never inf - inf unless a
// logit is +inf, which makes z a NaN like a NaN logit does; z = 0 means that
// every logit is -inf.
struct CarefulSums {
  float m, z, w;
};
__device__ __forceinline__ CarefulSums careful_empty() { return {-FLT_MAX, 0.0f, 0.0f}; }

__device__ __forceinline__ void careful_rebase(CarefulSums& s, float m, const ExpScale& c) {
  const float d = finite_low(s.m - m);
  const float f = exp_of(d, c);
  s.w = (s.w + d * s.z) * f;
  s.z *= f;
  s.m = m;
}
__device__ __forceinline__ void careful_add(CarefulSums& s, const float4& x, const ExpScale& c) {
  const float v[4] = {x.x, x.y, x.z, x.w};
  const float m = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
  if (m > s.m) careful_rebase(s, m, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float t = v[i] - s.m;
    const float e = exp_of(t, c);
    s.z += e;
    s.w = __fmaf_rn(e, finite_low(t), s.w);
  }
}

// ------------------------------------------------------------------ parts of a row

// A CTA's part of a row, or the row: z and w (w in units of (l - m) / T)
// relative to a reference: 2^(c l - ref) (fast) or exp((l - ref) / T) (careful).
struct PartStats {
  double z, w;
  float ref;
};

// 2^n for an integer n <= 0 (0 below -1000).
__device__ __forceinline__ double exp2_int(double n) {
  return n < -1000.0 ? 0.0 : __hiloint2double((1023 + static_cast<int>(n)) << 20, 0);
}

// The parts in lanes 0 .. N - 1 (an empty one: z = w = 0, ref the lowest
// value), brought to the largest reference; lanes 0 .. N - 1 hold the result.
// FAST: the references are exponents of 2.
template <bool FAST, int N>
__device__ __forceinline__ PartStats merge_parts(PartStats p, const ExpScale& c) {
  float ref = p.ref;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, o));
  double d = static_cast<double>(p.ref) - static_cast<double>(ref);  // <= 0 (NaN: both infinite)
  double f = 0.0;
  if (FAST) {
    if (d > -1000.0) {
      f = exp2_int(d);
      d *= kLn2;
    } else {
      d = 0.0;  // a far lower part adds 0
    }
  } else {
    d *= c.inv_t;
    if (d > -1000.0) {
      f = exp(d);
    } else {
      d = 0.0;
    }
  }
  p.w = (p.w + d * p.z) * f;
  p.z *= f;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    p.z += __shfl_xor_sync(0xFFFFFFFFu, p.z, o);
    p.w += __shfl_xor_sync(0xFFFFFFFFu, p.w, o);
  }
  p.ref = ref;
  return p;
}

// Whether a CTA's fast sums hold (a row's, when its parts' and its token's do and
// it is not below kFastLeast).
__device__ __forceinline__ bool fast_holds(const PartStats& p) { return p.z <= 0x1p60 && fabsf(p.ref) <= kFastMaxK; }
constexpr double kFastLeast = 0x1p-40;

// The token's own term relative to an integer exponent of 2, in 64 bits (0: its
// logit is -inf, or so low that the term is nothing beside a row that holds).
struct TokenTerm {
  double e;
  float k;
  bool holds;
};
__device__ __forceinline__ TokenTerm token_term(float logit, const ExpScale& c) {
  TokenTerm t;
  t.k = rintf(logit * c.c);
  t.holds = t.k <= kFastMaxK;  // no for +inf and NaN
  t.e = 0.0;
  if (t.holds && t.k >= -kFastMaxK)
    t.e = exp(static_cast<double>(logit) * c.inv_t_fast - static_cast<double>(t.k) * kLn2);
  else
    t.k = -FLT_MAX;
  return t;
}

// A row's sums with the token's term among them, and z without it; the
// exponentials' mean error is taken out of the others'.
struct RowStats {
  double z, w, rest;
  float ref;
};
__device__ __forceinline__ RowStats add_token(const PartStats& p, const TokenTerm& t, float logit, const ExpScale& c) {
  RowStats r;
  r.ref = fmaxf(p.ref, t.k);
  const double d = static_cast<double>(p.ref) - static_cast<double>(r.ref), f = kExpMean * exp2_int(d);
  const double e = t.e * exp2_int(static_cast<double>(t.k) - static_cast<double>(r.ref));
  r.w = (p.w + d * kLn2 * p.z) * f;
  if (e > 0.0) r.w += e * (static_cast<double>(logit) * c.inv_t_fast - static_cast<double>(r.ref) * kLn2);
  r.rest = p.z * f;
  r.z = r.rest + e;
  return r;
}
__device__ __forceinline__ RowStats add_token_careful(const PartStats& p, float logit, const ExpScale& c) {
  RowStats r;
  r.ref = fmaxf(p.ref, logit);
  const double d = (static_cast<double>(p.ref) - static_cast<double>(r.ref)) * c.inv_t;
  const double x = (static_cast<double>(logit) - static_cast<double>(r.ref)) * c.inv_t;
  const double f = d > -1000.0 ? kExpMean * exp(d) : 0.0;
  const double e = logit < INFINITY ? (x > -1000.0 ? exp(x) : 0.0) : static_cast<double>(NAN);
  r.w = (p.w + (d > -1000.0 ? d * p.z : 0.0)) * f;
  if (e > 0.0) r.w += e * x;
  r.rest = p.z * f;
  r.z = r.rest + e;
  return r;
}

// A row's results in 64 bits (a difference of two logprobs, a ratio near a
// border and the KL estimate near 0 all lose digits in 32), from its sums with
// the token's term.
struct RowScore {
  double logprob, z, log_z, entropy;
};
template <bool FAST, bool ENT>
__device__ __forceinline__ RowScore row_score(const RowStats& s, float token_logit, const ExpScale& c) {
  RowScore r;
  r.z = s.z > 0.0 ? s.z : static_cast<double>(NAN);  // 0: every logit is -inf; NaN: a NaN or +inf logit
  r.log_z = log(r.z);
  const double l = token_logit, ref = s.ref;
  const double x = FAST ? l * c.inv_t_fast - ref * kLn2 : (l - ref) * c.inv_t;
  r.logprob = x - r.log_z;
  r.entropy = 0.0;
  if (ENT) {
    r.entropy = r.log_z - s.w / r.z;  // less the mean of x under p
    if (r.entropy < 0.0) r.entropy = 0.0;
  }
  if (r.logprob > 0.0) r.logprob = 0.0;
  return r;
}

// Position of a thread in the slices of a row, in units of four logits: the
// thread visits every `step`-th unit from its first.
struct SliceCursor {
  int slice, at;  // unit `at` of slice `slice`
  __device__ __forceinline__ void start(int first, int per_slice) {
    slice = first / per_slice;
    at = first - slice * per_slice;
  }
  __device__ __forceinline__ void advance(int step, int per_slice) {
    at += step;
    while (at >= per_slice) {
      at -= per_slice;
      ++slice;
    }
  }
};

}  // namespace vsl
