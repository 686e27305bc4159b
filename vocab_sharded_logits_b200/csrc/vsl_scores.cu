// vsl_scores.cu - logprobs of given tokens over vocab-sliced logits, their
// gradient, and the clipped policy loss with its gradient.
//
// The sampler returns the raw logprob of the token it draws; these calls score
// tokens that are given, at a temperature, and take derivatives back to the
// logits.  With p_j the softmax of l / T over the row, t its token and H the
// entropy,
//   d log p_t / d l_j = (1[j = t] - p_j) / T,
//   d H / d l_j       = -p_j (log p_j + H) / T,
// so the gradient of any function of a row's logprob and entropy is
//   G_j = (g 1[j = t] - p_j (g + h (log p_j + H))) / T,  g = df / dlogp, h = df / dH,
// and with p_j = e_j / z, log p_j = (l_j - m) / T - log z:
//   G_j = e_j (alpha + gamma (l_j - m)) + (g / T) 1[j = t].
// Clipped policy loss of a row with ratio r = exp(logp - old):
//   w [ -min(r A, clip(r, 1 - lo, 1 + hi) A) + beta (exp(d) - d - 1) - c H ],  d = ref - logp.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "vsl_internal.h"
#include "vsl_ptx.cuh"
#include "vsl_softmax.cuh"

namespace vsl {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;  // units of four logits a thread has in flight

struct SliceArgs {
  const float* slices[VSL_MAX_SLICES];
  int per_slice;  // V_s / 4
  int units;      // S * V_s / 4
  int V_s;
  ExpScale c;
  float temperature;
};

__device__ __forceinline__ const float* unit_ptr(const SliceArgs& a, int row, const SliceCursor& k) {
  return a.slices[k.slice] + static_cast<size_t>(row) * a.V_s + 4 * static_cast<size_t>(k.at);
}

// 16-byte load of data read once (not the read-only path: the gradient may be
// written over the logits by the same kernel).
__device__ __forceinline__ float4 ldg_once4(const float* p) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
  return v;
}

// Statistics of units [first, last) of a row by the whole CTA.
template <bool ENT>
__device__ __forceinline__ SoftmaxStats part_stats(const SliceArgs& a, int row, int first, int last) {
  SoftmaxStats s = stats_empty();
  int i = first + static_cast<int>(threadIdx.x);
  SliceCursor k;
  k.start(i < last ? i : first, a.per_slice);
  const int step = static_cast<int>(blockDim.x);
  while (i < last) {
    float v[4 * kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (i < last) {
        x = ldg_once4(unit_ptr(a, row, k));
        i += step;
        if (i < last) k.advance(step, a.per_slice);
      }
      v[4 * u] = x.x;
      v[4 * u + 1] = x.y;
      v[4 * u + 2] = x.z;
      v[4 * u + 3] = x.w;
    }
    stats_add<ENT>(s, v, a.c);
  }
  return s;
}

// Block-wide merge; every thread returns the result.  `shared` holds a slot per warp.
template <bool ENT>
__device__ __forceinline__ SoftmaxStats block_stats(SoftmaxStats s, SoftmaxStats* shared, ExpScale c) {
  s = stats_warp<ENT>(s, c);
  const int warps = static_cast<int>(blockDim.x) >> 5;
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = s;
  __syncthreads();
  s = shared[0];
  for (int i = 1; i < warps; ++i) s = stats_merge<ENT>(s, shared[i], c);
  __syncthreads();
  return s;
}

__device__ __forceinline__ float token_logit(const SliceArgs& a, int row, int token) {
  const int s = token / a.V_s;
  return a.slices[s][static_cast<size_t>(row) * a.V_s + (token - s * a.V_s)];
}

__device__ __forceinline__ void store_unit(float* p, const float (&g)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(g[0], g[1], g[2], g[3]);
}
__device__ __forceinline__ void store_unit(__nv_bfloat16* p, const float (&g)[4]) {
  // one rounding to bf16 at the end: the next step is a bf16 matrix product
  __nv_bfloat162 lo = __floats2bfloat162_rn(g[0], g[1]), hi = __floats2bfloat162_rn(g[2], g[3]);
  uint2 v;
  v.x = reinterpret_cast<uint32_t&>(lo);
  v.y = reinterpret_cast<uint32_t&>(hi);
  *reinterpret_cast<uint2*>(p) = v;
}

// A row's gradient coefficients (see the file's head).
struct GradCoef {
  float m, alpha, gamma, at_token;
  int token;  // -1: the row does not count, its gradient is 0
};

__device__ __forceinline__ GradCoef grad_coef(double g, double h, double m, double z, double log_z, double entropy,
                                              double temperature, int token) {
  const double inv_t = 1.0 / temperature;
  GradCoef k;
  k.m = static_cast<float>(m);
  k.gamma = 0.0f;
  double alpha = -g * inv_t / z;
  if (h != 0.0) {
    alpha -= h * (entropy - log_z) * inv_t / z;
    k.gamma = static_cast<float>(-h * inv_t * inv_t / z);
  }
  k.alpha = static_cast<float>(alpha);
  k.at_token = static_cast<float>(g * inv_t);
  k.token = token;
  return k;
}

struct GradArgs {
  void* grad[VSL_MAX_SLICES];
};

// Gradient of units [first, last) of a row by the whole CTA.
template <typename T>
__device__ __forceinline__ void part_grad(const SliceArgs& a, const GradArgs& out, const GradCoef& k, int row,
                                          int first, int last) {
  int i = first + static_cast<int>(threadIdx.x);
  SliceCursor cur;
  cur.start(i < last ? i : first, a.per_slice);
  const int step = static_cast<int>(blockDim.x);
  for (; i < last; i += step) {
    T* dst = static_cast<T*>(out.grad[cur.slice]) + static_cast<size_t>(row) * a.V_s + 4 * static_cast<size_t>(cur.at);
    float g[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (k.token >= 0) {
      // a plain load: the gradient may be written over the logits
      const float4 x = *reinterpret_cast<const float4*>(unit_ptr(a, row, cur));
      const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float t = v[j] - k.m;
        g[j] = exp_of(t, a.c) * __fmaf_rn(k.gamma, finite_low(t), k.alpha);
        if (4 * i + j == k.token) g[j] += k.at_token;
      }
    }
    store_unit(dst, g);
    if (i + step < last) cur.advance(step, a.per_slice);
  }
}

struct LogprobArgs {
  SliceArgs in;
  const int32_t* tokens;
  float* logprob;
  float* entropy;  // may be null
  float2* stats;   // may be null
};

template <bool ENT>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ SoftmaxStats shared[kWarps];
  const int row = static_cast<int>(blockIdx.x);
  const int token = a.tokens[row];
  const bool on = token >= 0 && token < 4 * a.in.units;
  SoftmaxStats s{0.0f, 1.0f, 0.0f};
  RowScore r{0.0, 0.0, 0.0};
  if (on) {
    s = block_stats<ENT>(part_stats<ENT>(a.in, row, 0, a.in.units), shared, a.in.c);
    if (threadIdx.x == 0) r = row_score<ENT>(s, token_logit(a.in, row, token), a.in.temperature);
  }
  if (threadIdx.x == 0) {
    a.logprob[row] = static_cast<float>(r.logprob);
    if (ENT) a.entropy[row] = static_cast<float>(r.entropy);
    if (a.stats != nullptr) a.stats[row] = make_float2(s.m, s.z);
  }
}

struct LogprobGradArgs {
  SliceArgs in;
  GradArgs out;
  const int32_t* tokens;
  const float2* stats;
  const float* entropy;
  const float* d_logprob;
  const float* d_entropy;  // may be null
  int per_part;            // units per CTA
  int parts;               // CTAs per row
};

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
  const int row = static_cast<int>(blockIdx.x) / a.parts;
  const int first = (static_cast<int>(blockIdx.x) - row * a.parts) * a.per_part;
  const int last = min(a.in.units, first + a.per_part);
  const int token = a.tokens[row];
  GradCoef k{};
  k.token = -1;
  const double g = a.d_logprob[row], h = a.d_entropy != nullptr ? a.d_entropy[row] : 0.0f;
  if (token >= 0 && token < 4 * a.in.units && (g != 0.0 || h != 0.0)) {
    const float2 s = a.stats[row];
    const double z = s.y > 0.0f ? s.y : NAN;
    k = grad_coef(g, h, s.x, z, log(z), h != 0.0 ? a.entropy[row] : 0.0, a.in.temperature, token);
  }
  part_grad<T>(a.in, a.out, k, row, first, last);
}

struct PolicyArgs {
  SliceArgs in;
  GradArgs out;
  const int32_t* tokens;
  const float* old_logprob;
  const float* ref_logprob;  // may be null
  const float* advantages;
  const float* weights;      // may be null
  float* loss;
  float* logprob;  // may be null
  float* kl;       // may be null
  float* entropy;  // may be null
  float clip_low, clip_high, kl_coef, entropy_coef;
  int grad;
};

// The row's loss and outputs (one thread), and its gradient coefficients.
__device__ __forceinline__ GradCoef policy_row(const PolicyArgs& a, int row, int token, const SoftmaxStats& s,
                                               float logit, bool write) {
  const RowScore r = row_score<true>(s, logit, a.in.temperature);
  const double w = a.weights != nullptr ? a.weights[row] : 1.0f;
  const double adv = a.advantages[row];
  const double ratio = exp(r.logprob - static_cast<double>(a.old_logprob[row]));
  const double low = 1.0 - static_cast<double>(a.clip_low), high = 1.0 + static_cast<double>(a.clip_high);
  const double free_term = ratio * adv, clip_term = fmin(fmax(ratio, low), high) * adv;
  double loss = free_term != free_term ? NAN : -(free_term <= clip_term ? free_term : clip_term);
  double g = free_term != free_term ? NAN : free_term <= clip_term ? -adv * ratio : 0.0;
  double kl = 0.0;
  if (a.ref_logprob != nullptr) {
    const double d = static_cast<double>(a.ref_logprob[row]) - r.logprob;
    kl = d > 700.0 ? INFINITY : expm1(d) - d;  // not inf - inf
    if (a.kl_coef != 0.0f) {
      loss += static_cast<double>(a.kl_coef) * kl;
      g -= static_cast<double>(a.kl_coef) * expm1(d);
    }
  }
  double h = 0.0;
  if (a.entropy_coef != 0.0f) {
    loss -= static_cast<double>(a.entropy_coef) * r.entropy;
    h = -w * static_cast<double>(a.entropy_coef);
  }
  if (write) {
    a.loss[row] = static_cast<float>(w * loss);
    if (a.logprob != nullptr) a.logprob[row] = static_cast<float>(r.logprob);
    if (a.kl != nullptr) a.kl[row] = static_cast<float>(kl);
    if (a.entropy != nullptr) a.entropy[row] = static_cast<float>(r.entropy);
  }
  const double z = s.z > 0.0f ? s.z : NAN;
  return grad_coef(w * g, h, s.m, z, r.log_z, r.entropy, a.in.temperature, token);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) policy_loss_kernel(const __grid_constant__ PolicyArgs a) {
  __shared__ SoftmaxStats shared[kWarps];
  __shared__ GradCoef coef;
  const int row = static_cast<int>(blockIdx.x);
  const int token = a.tokens[row];
  const bool on = token >= 0 && token < 4 * a.in.units && (a.weights == nullptr || a.weights[row] != 0.0f);
  if (on) {
    const SoftmaxStats s = block_stats<true>(part_stats<true>(a.in, row, 0, a.in.units), shared, a.in.c);
    if (threadIdx.x == 0) coef = policy_row(a, row, token, s, token_logit(a.in, row, token), true);
  } else if (threadIdx.x == 0) {
    coef = GradCoef{};
    coef.token = -1;
    a.loss[row] = 0.0f;
    if (a.logprob != nullptr) a.logprob[row] = 0.0f;
    if (a.kl != nullptr) a.kl[row] = 0.0f;
    if (a.entropy != nullptr) a.entropy[row] = 0.0f;
  }
  if (!a.grad) return;
  __syncthreads();
  part_grad<T>(a.in, a.out, coef, row, 0, a.in.units);
}

SliceArgs slice_args(const float* const* logits, int S, int V_s, float temperature) {
  SliceArgs in{};
  for (int s = 0; s < S; ++s) in.slices[s] = logits[s];
  in.per_slice = V_s / 4;
  in.units = S * (V_s / 4);
  in.V_s = V_s;
  in.c = exp_scale(temperature);
  in.temperature = temperature;
  return in;
}

}  // namespace

cudaError_t launch_token_logprobs(const float* const* logits, int R, int S, int V_s, const int32_t* token_ids,
                                  float temperature, float* logprob, float* entropy, float* row_stats,
                                  cudaStream_t stream) {
  LogprobArgs a{};
  a.in = slice_args(logits, S, V_s, temperature);
  a.tokens = token_ids;
  a.logprob = logprob;
  a.entropy = entropy;
  a.stats = reinterpret_cast<float2*>(row_stats);
  if (entropy != nullptr)
    token_logprobs_kernel<true><<<R, kThreads, 0, stream>>>(a);
  else
    token_logprobs_kernel<false><<<R, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_token_logprobs_grad(const float* const* logits, int R, int S, int V_s, const int32_t* token_ids,
                                       float temperature, const float* row_stats, const float* entropy,
                                       const float* d_logprob, const float* d_entropy, void* const* grad,
                                       int grad_type, cudaStream_t stream) {
  LogprobGradArgs a{};
  a.in = slice_args(logits, S, V_s, temperature);
  for (int s = 0; s < S; ++s) a.out.grad[s] = grad[s];
  a.tokens = token_ids;
  a.stats = reinterpret_cast<const float2*>(row_stats);
  a.entropy = entropy;
  a.d_logprob = d_logprob;
  a.d_entropy = d_entropy;
  a.per_part = kThreads * 8;
  a.parts = (a.in.units + a.per_part - 1) / a.per_part;
  const long long grid_size = static_cast<long long>(R) * a.parts;
  if (grid_size > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(grid_size);
  if (grad_type == VSL_GRAD_BF16)
    token_logprobs_grad_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  else
    token_logprobs_grad_kernel<float><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_policy_loss(const float* const* logits, int R, int S, int V_s, const vsl_policy_inputs& in,
                               const vsl_policy_outputs& out, cudaStream_t stream) {
  PolicyArgs a{};
  a.in = slice_args(logits, S, V_s, in.temperature);
  a.grad = out.grad_slices != nullptr;
  if (a.grad)
    for (int s = 0; s < S; ++s) a.out.grad[s] = out.grad_slices[s];
  a.tokens = in.token_ids;
  a.old_logprob = in.old_logprob;
  a.ref_logprob = in.ref_logprob;
  a.advantages = in.advantages;
  a.weights = in.weights;
  a.loss = out.loss;
  a.logprob = out.logprob;
  a.kl = out.kl;
  a.entropy = out.entropy;
  a.clip_low = in.clip_low;
  a.clip_high = in.clip_high;
  a.kl_coef = in.kl_coef;
  a.entropy_coef = in.entropy_coef;
  if (out.grad_type == VSL_GRAD_BF16)
    policy_loss_kernel<__nv_bfloat16><<<R, kThreads, 0, stream>>>(a);
  else
    policy_loss_kernel<float><<<R, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace vsl
