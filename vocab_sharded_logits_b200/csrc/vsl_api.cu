// vsl_api.cu - the extern "C" entry points of libvsl: host-side argument
// validation, then a launch of the call's kernels.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "vsl_internal.h"

namespace vsl {

// Device error word: kernels OR a site bit into it when a bounded wait gives up.
__device__ uint32_t g_device_error = 0;

uint32_t* device_error_word() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
  return static_cast<uint32_t*>(p);
}

namespace {
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The checks every call that reads logits slices and scores tokens makes.
vsl_status check_slices(const float* const* logits, int32_t R, int32_t S, int32_t V_s) {
  if (logits == nullptr || R <= 0 || S <= 0 || V_s <= 0) return VSL_ERR_INVALID_ARG;
  if (S > VSL_MAX_SLICES || static_cast<long long>(S) * V_s > VSL_MAX_VOCAB) return VSL_ERR_UNSUPPORTED;
  if (V_s % 4 != 0) return VSL_ERR_ALIGNMENT;
  for (int s = 0; s < S; ++s) {
    if (logits[s] == nullptr) return VSL_ERR_INVALID_ARG;
    if (!aligned16(logits[s])) return VSL_ERR_ALIGNMENT;
  }
  return VSL_OK;
}

// Output slices: aligned, distinct, and no alias of the logits but (where
// allowed) the slice of the same index.
vsl_status check_out_slices(const float* const* logits, void* const* out, int32_t S, bool in_place_allowed) {
  for (int s = 0; s < S; ++s) {
    if (out[s] == nullptr) return VSL_ERR_INVALID_ARG;
    if (!aligned16(out[s])) return VSL_ERR_ALIGNMENT;
    for (int o = 0; o < S; ++o) {
      if (out[s] == static_cast<const void*>(logits[o]) && !(in_place_allowed && o == s)) return VSL_ERR_INVALID_ARG;
      if (o < s && out[o] == out[s]) return VSL_ERR_INVALID_ARG;
    }
  }
  return VSL_OK;
}

bool temperature_ok(float t) { return t >= 1e-6f && t <= 1e6f; }
}  // namespace

}  // namespace vsl

extern "C" {

const char* vsl_version(void) { return "libvsl 0.1 (sm_100a)"; }

const char* vsl_status_string(vsl_status status) {
  switch (status) {
    case VSL_OK: return "ok";
    case VSL_ERR_INVALID_ARG: return "invalid argument";
    case VSL_ERR_ALIGNMENT: return "pointer or row pitch not 16-byte aligned";
    case VSL_ERR_UNSUPPORTED: return "size beyond the library's limits";
    case VSL_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case VSL_ERR_CUDA: return "CUDA call failed";
    case VSL_ERR_DEVICE_TIMEOUT: return "a kernel gave up a bounded wait";
  }
  return "unknown status";
}

size_t vsl_tile_stats_floats(int32_t R, int32_t S, int32_t V_s) {
  if (R <= 0 || S <= 0 || V_s <= 0) return 0;
  return static_cast<size_t>(R) * static_cast<size_t>(S) * ((static_cast<size_t>(V_s) + 127) / 128) * 8;
}

vsl_status vsl_tile_stats(const float* const* logits_slices, int32_t R, int32_t S, int32_t V_s, float* tile_stats,
                          void* stream) {
  if (logits_slices == nullptr || tile_stats == nullptr) return VSL_ERR_INVALID_ARG;
  if (R <= 0 || S <= 0 || V_s <= 0) return VSL_ERR_INVALID_ARG;
  if (S > VSL_MAX_SLICES) return VSL_ERR_UNSUPPORTED;
  if (V_s % 4 != 0 || !vsl::aligned32(tile_stats)) return VSL_ERR_ALIGNMENT;
  for (int s = 0; s < S; ++s) {
    if (logits_slices[s] == nullptr) return VSL_ERR_INVALID_ARG;
    if (!vsl::aligned16(logits_slices[s])) return VSL_ERR_ALIGNMENT;
  }
  const cudaError_t e = vsl::launch_tile_stats(logits_slices, R, S, V_s, tile_stats, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

vsl_status vsl_logits_local(const void* hidden_bf16, const void* const* w_slices_bf16, float* const* logits_slices,
                            int32_t R, int32_t H, int32_t S, int32_t V_s, void* stream) {
  return vsl_logits_local_ex(hidden_bf16, w_slices_bf16, logits_slices, R, H, S, V_s, nullptr, stream);
}

vsl_status vsl_logits_local_ex(const void* hidden_bf16, const void* const* w_slices_bf16, float* const* logits_slices,
                               int32_t R, int32_t H, int32_t S, int32_t V_s, float* tile_stats, void* stream) {
  if (hidden_bf16 == nullptr || w_slices_bf16 == nullptr || logits_slices == nullptr) return VSL_ERR_INVALID_ARG;
  if (R <= 0 || H <= 0 || S <= 0 || V_s <= 0) return VSL_ERR_INVALID_ARG;
  if (S > VSL_MAX_SLICES) return VSL_ERR_UNSUPPORTED;
  if (H % 8 != 0 || V_s % 4 != 0) return VSL_ERR_ALIGNMENT;
  if (!vsl::aligned16(hidden_bf16)) return VSL_ERR_ALIGNMENT;
  for (int s = 0; s < S; ++s) {
    if (w_slices_bf16[s] == nullptr || logits_slices[s] == nullptr) return VSL_ERR_INVALID_ARG;
    if (!vsl::aligned16(w_slices_bf16[s]) || !vsl::aligned16(logits_slices[s])) return VSL_ERR_ALIGNMENT;
  }
  if (tile_stats != nullptr && !vsl::aligned32(tile_stats)) return VSL_ERR_ALIGNMENT;
  const cudaError_t e = vsl::launch_logits_local(hidden_bf16, w_slices_bf16, logits_slices, R, H, S, V_s, tile_stats,
                                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

size_t vsl_sample_workspace_bytes(int32_t R, int32_t S, int32_t V_s, int32_t n_logprobs) {
  (void)R;
  (void)S;
  (void)V_s;
  (void)n_logprobs;
  return 0;  // every intermediate lives in shared memory
}

int32_t vsl_sample_launches(int32_t R, int32_t S, int32_t V_s) {
  if (R <= 0 || S <= 0 || S > VSL_MAX_SLICES || V_s <= 0 || V_s % 4 != 0) return -1;
  return vsl::sample_launches(R, static_cast<long long>(S) * V_s);
}

vsl_status vsl_sample_plan_for(int32_t R, int32_t S, int32_t V_s, int32_t sms, int32_t max_cluster,
                               vsl_sample_plan* out) {
  if (out == nullptr || R <= 0 || S <= 0 || V_s <= 0 || sms <= 0 || max_cluster <= 0) return VSL_ERR_INVALID_ARG;
  if (S > VSL_MAX_SLICES) return VSL_ERR_UNSUPPORTED;
  if (V_s % 4 != 0) return VSL_ERR_ALIGNMENT;
  const long long V = static_cast<long long>(S) * V_s;
  if (V > 0x7FFFFFFFLL || !vsl::sample_plan(R, V, sms, max_cluster, out)) return VSL_ERR_UNSUPPORTED;
  return VSL_OK;
}

vsl_status vsl_sample_ex(const float* const* logits_slices, int32_t R, int32_t S, int32_t V_s,
                         const vsl_row_params* params_dev, uint64_t seed, int32_t n_logprobs, int32_t* token_ids,
                         float* token_logprob, int32_t* topn_ids, float* topn_logprob, uint32_t* row_flags,
                         void* workspace, size_t workspace_bytes, const vsl_sample_extras* extras, void* stream) {
  (void)workspace;
  if (logits_slices == nullptr || params_dev == nullptr || token_ids == nullptr || token_logprob == nullptr ||
      row_flags == nullptr)
    return VSL_ERR_INVALID_ARG;
  if (R <= 0 || S <= 0 || V_s <= 0 || n_logprobs < 0) return VSL_ERR_INVALID_ARG;
  if (S > VSL_MAX_SLICES || n_logprobs > VSL_MAX_LOGPROBS) return VSL_ERR_UNSUPPORTED;
  const long long V = static_cast<long long>(S) * V_s;
  if (n_logprobs > V) return VSL_ERR_INVALID_ARG;
  if (n_logprobs > 0 && (topn_ids == nullptr || topn_logprob == nullptr)) return VSL_ERR_INVALID_ARG;
  if (V_s % 4 != 0) return VSL_ERR_ALIGNMENT;
  for (int s = 0; s < S; ++s) {
    if (logits_slices[s] == nullptr) return VSL_ERR_INVALID_ARG;
    if (!vsl::aligned16(logits_slices[s])) return VSL_ERR_ALIGNMENT;
  }
  float* kept_theta = extras != nullptr ? extras->kept_theta : nullptr;
  if (kept_theta != nullptr && (reinterpret_cast<uintptr_t>(kept_theta) & 7u) != 0) return VSL_ERR_ALIGNMENT;
  float* p_token = extras != nullptr ? extras->processed_logprob : nullptr;
  int32_t* p_topn_ids = extras != nullptr ? extras->processed_topn_ids : nullptr;
  float* p_topn = extras != nullptr ? extras->processed_topn_logprob : nullptr;
  if (p_token == nullptr && (p_topn_ids != nullptr || p_topn != nullptr)) return VSL_ERR_INVALID_ARG;
  if (p_token != nullptr && kept_theta == nullptr) return VSL_ERR_INVALID_ARG;
  if (p_token != nullptr && n_logprobs > 0 && (p_topn_ids == nullptr || p_topn == nullptr)) return VSL_ERR_INVALID_ARG;
  const float* tile_stats = extras != nullptr ? extras->tile_stats : nullptr;
  if (tile_stats != nullptr && !vsl::aligned32(tile_stats)) return VSL_ERR_ALIGNMENT;
  if (V > vsl::sample_max_vocab()) return VSL_ERR_UNSUPPORTED;
  int maxc = 0, c = 0, part = 0;
  if (vsl::sample_max_cluster(&maxc) != cudaSuccess) return VSL_ERR_CUDA;
  if (!vsl::sample_geometry_for(V, maxc, &c, &part)) return VSL_ERR_UNSUPPORTED;
  if (workspace_bytes < vsl_sample_workspace_bytes(R, S, V_s, n_logprobs)) return VSL_ERR_WORKSPACE_TOO_SMALL;
  cudaError_t e = vsl::launch_sample(logits_slices, R, S, V_s, params_dev, seed, n_logprobs, token_ids,
                                     token_logprob, topn_ids, topn_logprob, row_flags, kept_theta, tile_stats,
                                     static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess && p_token != nullptr)
    e = vsl::launch_processed(logits_slices, R, S, V_s, params_dev, n_logprobs, token_ids, topn_ids, row_flags,
                              kept_theta, p_token, p_topn_ids, p_topn, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

vsl_status vsl_sample(const float* const* logits_slices, int32_t R, int32_t S, int32_t V_s,
                      const vsl_row_params* params_dev, uint64_t seed, int32_t n_logprobs, int32_t* token_ids,
                      float* token_logprob, int32_t* topn_ids, float* topn_logprob, uint32_t* row_flags,
                      void* workspace, size_t workspace_bytes, void* stream) {
  return vsl_sample_ex(logits_slices, R, S, V_s, params_dev, seed, n_logprobs, token_ids, token_logprob, topn_ids,
                       topn_logprob, row_flags, workspace, workspace_bytes, nullptr, stream);
}

vsl_status vsl_verify_drafts(const int32_t* token_ids, const float* token_logprob, const int32_t* draft_ids,
                             int32_t requests, int32_t spec, int32_t* out_ids, float* out_logprob,
                             int32_t* accepted, void* stream) {
  if (token_ids == nullptr || out_ids == nullptr || accepted == nullptr) return VSL_ERR_INVALID_ARG;
  if (requests <= 0 || spec < 0 || spec > VSL_MAX_SPEC) return VSL_ERR_INVALID_ARG;
  if (spec > 0 && draft_ids == nullptr) return VSL_ERR_INVALID_ARG;
  if ((out_logprob == nullptr) != (token_logprob == nullptr)) return VSL_ERR_INVALID_ARG;
  if (static_cast<long long>(requests) * (spec + 1) > 0x7FFFFFFFLL) return VSL_ERR_UNSUPPORTED;
  const cudaError_t e = vsl::launch_verify(token_ids, token_logprob, draft_ids, requests, spec, out_ids,
                                           out_logprob, accepted, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

size_t vsl_adapters_workspace_bytes(int32_t R, int32_t n_adapters, int32_t rank) {
  if (R <= 0 || n_adapters <= 0 || rank <= 0 || rank > VSL_MAX_RANK || R > VSL_MAX_ADAPTER_ROWS)
    return 0;
  return vsl::adapters_workspace_bytes(R, n_adapters, rank);
}

vsl_status vsl_adapters_add(const float* const* logits_slices, float* const* out_slices, const void* hidden_bf16,
                            int32_t R, int32_t H, int32_t S, int32_t V_s, const void* a_bf16,
                            const void* const* b_slices_bf16, const float* scale, int32_t n_adapters, int32_t rank,
                            const int32_t* adapter_ids, float* tile_stats, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (out_slices == nullptr || hidden_bf16 == nullptr || a_bf16 == nullptr || b_slices_bf16 == nullptr ||
      adapter_ids == nullptr)
    return VSL_ERR_INVALID_ARG;
  if (H <= 0 || n_adapters <= 0 || rank <= 0) return VSL_ERR_INVALID_ARG;
  vsl_status st = vsl::check_slices(logits_slices, R, S, V_s);
  if (st != VSL_OK) return st;
  if (rank > VSL_MAX_RANK || R > VSL_MAX_ADAPTER_ROWS) return VSL_ERR_UNSUPPORTED;
  if (H % 8 != 0 || rank % 8 != 0) return VSL_ERR_ALIGNMENT;
  if (!vsl::aligned16(hidden_bf16) || !vsl::aligned16(a_bf16)) return VSL_ERR_ALIGNMENT;
  for (int s = 0; s < S; ++s) {
    if (b_slices_bf16[s] == nullptr) return VSL_ERR_INVALID_ARG;
    if (!vsl::aligned16(b_slices_bf16[s])) return VSL_ERR_ALIGNMENT;
  }
  void* out[VSL_MAX_SLICES];
  for (int s = 0; s < S; ++s) out[s] = out_slices[s];
  st = vsl::check_out_slices(logits_slices, out, S, true);
  if (st != VSL_OK) return st;
  if (tile_stats != nullptr && !vsl::aligned32(tile_stats)) return VSL_ERR_ALIGNMENT;
  if (workspace == nullptr) return VSL_ERR_INVALID_ARG;
  if (!vsl::aligned16(workspace)) return VSL_ERR_ALIGNMENT;
  if (workspace_bytes < vsl_adapters_workspace_bytes(R, n_adapters, rank)) return VSL_ERR_WORKSPACE_TOO_SMALL;
  const cudaError_t e =
      vsl::launch_adapters_add(logits_slices, out_slices, hidden_bf16, R, H, S, V_s, a_bf16, b_slices_bf16, scale,
                               n_adapters, rank, adapter_ids, tile_stats, workspace, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

vsl_status vsl_token_logprobs(const float* const* logits_slices, int32_t R, int32_t S, int32_t V_s,
                              const int32_t* token_ids, float temperature, float* logprob, float* entropy,
                              float* row_stats, void* stream) {
  if (token_ids == nullptr || logprob == nullptr || !vsl::temperature_ok(temperature)) return VSL_ERR_INVALID_ARG;
  const vsl_status st = vsl::check_slices(logits_slices, R, S, V_s);
  if (st != VSL_OK) return st;
  if (row_stats != nullptr && !vsl::aligned8(row_stats)) return VSL_ERR_ALIGNMENT;
  const cudaError_t e = vsl::launch_token_logprobs(logits_slices, R, S, V_s, token_ids, temperature, logprob, entropy,
                                                   row_stats, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

vsl_status vsl_token_logprobs_grad(const float* const* logits_slices, int32_t R, int32_t S, int32_t V_s,
                                   const int32_t* token_ids, float temperature, const float* row_stats,
                                   const float* entropy, const float* d_logprob, const float* d_entropy,
                                   void* const* grad_slices, int32_t grad_type, void* stream) {
  if (token_ids == nullptr || row_stats == nullptr || d_logprob == nullptr || grad_slices == nullptr)
    return VSL_ERR_INVALID_ARG;
  if (d_entropy != nullptr && entropy == nullptr) return VSL_ERR_INVALID_ARG;
  if (!vsl::temperature_ok(temperature)) return VSL_ERR_INVALID_ARG;
  if (grad_type != VSL_GRAD_FP32 && grad_type != VSL_GRAD_BF16) return VSL_ERR_INVALID_ARG;
  vsl_status st = vsl::check_slices(logits_slices, R, S, V_s);
  if (st != VSL_OK) return st;
  st = vsl::check_out_slices(logits_slices, grad_slices, S, grad_type == VSL_GRAD_FP32);
  if (st != VSL_OK) return st;
  if (!vsl::aligned8(row_stats)) return VSL_ERR_ALIGNMENT;
  const cudaError_t e =
      vsl::launch_token_logprobs_grad(logits_slices, R, S, V_s, token_ids, temperature, row_stats, entropy, d_logprob,
                                      d_entropy, grad_slices, grad_type, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

vsl_status vsl_policy_loss(const float* const* logits_slices, int32_t R, int32_t S, int32_t V_s,
                           const vsl_policy_inputs* inputs, const vsl_policy_outputs* outputs, void* stream) {
  if (inputs == nullptr || outputs == nullptr) return VSL_ERR_INVALID_ARG;
  if (inputs->token_ids == nullptr || inputs->old_logprob == nullptr || inputs->advantages == nullptr ||
      outputs->loss == nullptr)
    return VSL_ERR_INVALID_ARG;
  if (!vsl::temperature_ok(inputs->temperature)) return VSL_ERR_INVALID_ARG;
  // written so that a NaN is refused
  if (!(inputs->clip_low >= 0.0f && inputs->clip_low <= 1.0f) || !(inputs->clip_high >= 0.0f)) return VSL_ERR_INVALID_ARG;
  if (!std::isfinite(inputs->kl_coef) || !std::isfinite(inputs->entropy_coef)) return VSL_ERR_INVALID_ARG;
  if (inputs->kl_coef != 0.0f && inputs->ref_logprob == nullptr) return VSL_ERR_INVALID_ARG;
  if (outputs->grad_type != VSL_GRAD_FP32 && outputs->grad_type != VSL_GRAD_BF16) return VSL_ERR_INVALID_ARG;
  vsl_status st = vsl::check_slices(logits_slices, R, S, V_s);
  if (st != VSL_OK) return st;
  if (outputs->grad_slices != nullptr) {
    st = vsl::check_out_slices(logits_slices, outputs->grad_slices, S, outputs->grad_type == VSL_GRAD_FP32);
    if (st != VSL_OK) return st;
  }
  const cudaError_t e =
      vsl::launch_policy_loss(logits_slices, R, S, V_s, *inputs, *outputs, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

vsl_status vsl_preference_loss(const float* logprob, const float* ref_logprob, const int32_t* offsets,
                               const float* weights, int32_t R, int32_t pairs, float beta, float label_smoothing,
                               float* loss, float* rewards, float* d_logprob, void* stream) {
  if (offsets == nullptr || loss == nullptr || R < 0 || pairs <= 0) return VSL_ERR_INVALID_ARG;
  if (R > 0 && logprob == nullptr) return VSL_ERR_INVALID_ARG;
  if (!std::isfinite(beta) || !(label_smoothing >= 0.0f && label_smoothing <= 1.0f)) return VSL_ERR_INVALID_ARG;
  if (pairs > 0x3FFFFFFF) return VSL_ERR_UNSUPPORTED;  // 2 * pairs + 1 offsets
  const cudaError_t e = vsl::launch_preference(logprob, ref_logprob, offsets, weights, R, pairs, beta, label_smoothing,
                                               loss, rewards, d_logprob, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VSL_OK : VSL_ERR_CUDA;
}

vsl_status vsl_device_error(uint32_t* code_out) {
  if (cudaDeviceSynchronize() != cudaSuccess) return VSL_ERR_CUDA;
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, vsl::g_device_error, sizeof(v)) != cudaSuccess) return VSL_ERR_CUDA;
  const uint32_t zero = 0;
  if (cudaMemcpyToSymbol(vsl::g_device_error, &zero, sizeof(zero)) != cudaSuccess) return VSL_ERR_CUDA;
  if (code_out) *code_out = v;
  return v ? VSL_ERR_DEVICE_TIMEOUT : VSL_OK;
}

}  // extern "C"
