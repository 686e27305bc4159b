// vsl_preference.cu - preference loss of pairs of sequences (paired log
// ratios) over the logprobs of their tokens, with its gradient.
//
// Sequence i owns rows [offsets[i], offsets[i + 1]); pair q prefers sequence 2q
// (chosen) to 2q + 1 (rejected).  With s_i = beta sum_rows (logprob - ref) and
// h = s_chosen - s_rejected,
//   loss = w [ -(1 - e) log sigmoid(h) - e log sigmoid(-h) ],
//   dloss / dh = w [ e sigmoid(h) - (1 - e) sigmoid(-h) ],
// and a row's derivative is +beta dloss/dh (chosen) or -beta dloss/dh
// (rejected).  Sums and the loss are kept in 64 bits: s_chosen - s_rejected
// cancels.
//
// One CTA per pair: 8 bytes read and 4 written per row, bound by launch latency
// and the chain of offsets, sums and loss (a pair of 256 rows each: 3.4 us in a
// graph's replay, 6.5 alone and cold).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "vsl_internal.h"

namespace vsl {

namespace {

constexpr int kPairThreads = 128;

struct PreferenceArgs {
  const float* logprob;
  const float* ref;      // may be null: 0
  const int32_t* offsets;
  const float* weights;  // may be null: 1
  float* loss;
  float* rewards;    // may be null
  float* d_logprob;  // may be null
  double beta, smoothing;
  int R, pairs;
};

__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kPairThreads / 32; ++i) v += shared[i];
  return v;
}

__device__ __forceinline__ double log_sigmoid(double h) {
  return h >= 0.0 ? -log1p(exp(-h)) : h - log1p(exp(h));
}
__device__ __forceinline__ double sigmoid(double h) {
  if (h >= 0.0) return 1.0 / (1.0 + exp(-h));
  const double e = exp(h);
  return e / (1.0 + e);
}

__device__ __forceinline__ void fill_rows(float* p, int first, int last, float v) {
  for (int r = first + static_cast<int>(threadIdx.x); r < last; r += kPairThreads) p[r] = v;
}

__global__ void __launch_bounds__(kPairThreads) preference_kernel(const __grid_constant__ PreferenceArgs a) {
  __shared__ double shared[kPairThreads / 32];
  const int q = static_cast<int>(blockIdx.x);
  // offsets come from device memory: kept inside the rows whatever they are
  int at[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) at[i] = min(max(a.offsets[2 * q + i], 0), a.R);
  const double w = a.weights != nullptr ? a.weights[q] : 1.0f;
  double s[2] = {0.0, 0.0}, loss = 0.0, d = 0.0;
  if (w != 0.0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      double v = 0.0;
      for (int r = at[i] + static_cast<int>(threadIdx.x); r < at[i + 1]; r += kPairThreads)
        v += static_cast<double>(a.logprob[r]) - (a.ref != nullptr ? static_cast<double>(a.ref[r]) : 0.0);
      s[i] = a.beta * block_sum(v, shared);
    }
    const double h = s[0] - s[1];
    // a factor of 0 leaves its term out, an infinite one too
    loss = w * -((a.smoothing != 1.0 ? (1.0 - a.smoothing) * log_sigmoid(h) : 0.0) +
                 (a.smoothing != 0.0 ? a.smoothing * log_sigmoid(-h) : 0.0));
    d = w * a.beta * (a.smoothing * sigmoid(h) - (1.0 - a.smoothing) * sigmoid(-h));
  }
  if (threadIdx.x == 0) {
    a.loss[q] = static_cast<float>(loss);
    if (a.rewards != nullptr) {
      a.rewards[2 * q] = static_cast<float>(s[0]);
      a.rewards[2 * q + 1] = static_cast<float>(s[1]);
    }
  }
  if (a.d_logprob != nullptr) {
    fill_rows(a.d_logprob, at[0], at[1], static_cast<float>(d));
    fill_rows(a.d_logprob, at[1], at[2], static_cast<float>(-d));
    // rows before the first sequence and behind the last belong to no pair
    if (q == 0) fill_rows(a.d_logprob, 0, at[0], 0.0f);
    if (q == a.pairs - 1) fill_rows(a.d_logprob, at[2], a.R, 0.0f);
  }
}

}  // namespace

cudaError_t launch_preference(const float* logprob, const float* ref, const int32_t* offsets, const float* weights,
                              int R, int pairs, float beta, float smoothing, float* loss, float* rewards,
                              float* d_logprob, cudaStream_t stream) {
  PreferenceArgs a{};
  a.logprob = logprob;
  a.ref = ref;
  a.offsets = offsets;
  a.weights = weights;
  a.loss = loss;
  a.rewards = rewards;
  a.d_logprob = d_logprob;
  a.beta = beta;
  a.smoothing = smoothing;
  a.R = R;
  a.pairs = pairs;
  preference_kernel<<<pairs, kPairThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace vsl
