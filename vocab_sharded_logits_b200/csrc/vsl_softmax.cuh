// vsl_softmax.cuh - the running softmax statistics of a row of vocab-sliced
// logits, shared by the kernels that score given tokens.
//
// For a row of logits l_j at temperature T, x_j = l_j / T, one pass keeps
//   m = max_j l_j,  z = sum_j exp((l_j - m) / T),  w = sum_j exp((l_j - m) / T) (l_j - m),
// from which, for a token t,
//   log p_t = (l_t - m) / T - log z,     H = log z - w / (z T)  (the entropy).
// exp((l - m) / T) is 2^(c (l - m)) with c = log2(e) / T.  c is carried as a
// sum of two floats, hi <= c and lo > 0: the rounding of a single float c would
// put the same relative error, |l - m| / T times 2^-24, on every far term of z.
// Both parts are positive, so l = -inf gives -inf and an exponential of 0, and
// a NaN stays one.  m starts at the lowest finite value, so l - m is never
// inf - inf unless a logit is +inf, which makes z a NaN like a NaN logit does;
// z = 0 means that every logit is -inf.
#pragma once

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "vsl_internal.h"

namespace vsl {

// c = log2(e) / T as hi + lo, hi <= c, lo > 0.
struct ExpScale {
  float hi, lo;
};

inline ExpScale exp_scale(float temperature) {
  const double c = 1.4426950408889634073599246810019 / static_cast<double>(temperature);
  ExpScale r;
  r.hi = static_cast<float>(c);
  if (static_cast<double>(r.hi) > c) r.hi = std::nextafterf(r.hi, 0.0f);
  r.lo = static_cast<float>(c - static_cast<double>(r.hi));
  if (!(r.lo > 0.0f)) r.lo = FLT_MIN;
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(t / T) for t <= 0 (0 for -inf, NaN for NaN).
__device__ __forceinline__ float exp_of(float t, ExpScale c) { return exp2_fast(__fmaf_rn(t, c.hi, t * c.lo)); }
// t bounded from below, so that its product with an exponential of 0 is 0: at
// -1e18 the exponential is 0 for every T up to 1e6, and a factor of up to 1e20
// (a sum of exponentials, a gradient's coefficient) still gives a finite value.
__device__ __forceinline__ float finite_low(float t) { return fmaxf(t, -1e18f); }

struct SoftmaxStats {
  float m, z, w;
};

__device__ __forceinline__ SoftmaxStats stats_empty() { return {-FLT_MAX, 0.0f, 0.0f}; }

// The statistics of two disjoint parts of a row.  ENT: w is kept.
template <bool ENT>
__device__ __forceinline__ SoftmaxStats stats_merge(const SoftmaxStats& a, const SoftmaxStats& b, ExpScale c) {
  SoftmaxStats r;
  r.m = fmaxf(a.m, b.m);
  const float da = finite_low(a.m - r.m), db = finite_low(b.m - r.m);
  const float fa = exp_of(da, c), fb = exp_of(db, c);
  r.z = a.z * fa + b.z * fb;
  r.w = 0.0f;
  if (ENT) r.w = (a.w + da * a.z) * fa + (b.w + db * b.z) * fb;
  return r;
}

// Adds N logits to a thread's statistics: their maximum first (one rescaling
// when it grows), then the exponentials.
template <bool ENT, int N>
__device__ __forceinline__ void stats_add(SoftmaxStats& s, const float (&v)[N], ExpScale c) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  if (m > s.m) {
    const float d = finite_low(s.m - m);
    const float f = exp_of(d, c);
    if (ENT) s.w = (s.w + d * s.z) * f;
    s.z *= f;
    s.m = m;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float t = v[i] - s.m;
    const float e = exp_of(t, c);
    s.z += e;
    if (ENT) s.w = __fmaf_rn(e, finite_low(t), s.w);
  }
}

template <bool ENT>
__device__ __forceinline__ SoftmaxStats stats_warp(SoftmaxStats s, ExpScale c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    SoftmaxStats b;
    b.m = __shfl_xor_sync(0xFFFFFFFFu, s.m, o);
    b.z = __shfl_xor_sync(0xFFFFFFFFu, s.z, o);
    b.w = ENT ? __shfl_xor_sync(0xFFFFFFFFu, s.w, o) : 0.0f;
    s = stats_merge<ENT>(s, b, c);
  }
  return s;
}

// A row's results in 64 bits (a difference of two logprobs, a ratio near a
// border and the KL estimate near 0 all lose digits in 32).
struct RowScore {
  double logprob, log_z, entropy;
};
template <bool ENT>
__device__ __forceinline__ RowScore row_score(const SoftmaxStats& s, float token_logit, float temperature) {
  RowScore r;
  const double inv_t = 1.0 / static_cast<double>(temperature);
  const double z = s.z > 0.0f ? static_cast<double>(s.z) : static_cast<double>(NAN);  // all -inf, NaN or +inf
  r.log_z = log(z);
  r.logprob = (static_cast<double>(token_logit) - static_cast<double>(s.m)) * inv_t - r.log_z;
  r.entropy = ENT ? r.log_z - static_cast<double>(s.w) / z * inv_t : 0.0;
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
