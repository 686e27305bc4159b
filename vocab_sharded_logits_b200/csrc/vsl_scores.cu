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
// and with p_j = e_j / z, log p_j = log e_j - log z:
//   G_j = e_j (alpha + gamma log e_j) + (g / T) 1[j = t].
// Clipped policy loss of a row with ratio r = exp(logp - old):
//   w [ -min(r A, clip(r, 1 - lo, 1 + hi) A) + beta (exp(d) - d - 1) - c H ],  d = ref - logp.
//
// Times below, but where another is named: calls replayed back to back from a
// graph over the same tensors, the median of five allocations.  One allocation
// differs from another by up to 5 % above 100 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "vsl_internal.h"
#include "vsl_ptx_rows.cuh"
#include "vsl_softmax.cuh"

namespace vsl {

namespace {

constexpr int kThreads = 512;       // of a CTA of the gradient kernel
constexpr int kRowThreads = 1536;   // threads of a row kernel that stand on an SM (40 registers each)
constexpr int kLogprobThreads = 1280;  // at least as many of the logprobs' stand on an SM (48 registers)
constexpr int kBatch = 4;      // units of four logits a thread has in flight
constexpr int kMaxCluster = 8;

struct SliceArgs {
  const float* slices[VSL_MAX_SLICES];
  int per_slice;  // V_s / 4
  int units;      // S * V_s / 4
  int V_s;
  ExpScale c;
};

__device__ __forceinline__ const float* unit_ptr(const SliceArgs& a, int row, const SliceCursor& k) {
  return a.slices[k.slice] + static_cast<size_t>(row) * a.V_s + 4 * static_cast<size_t>(k.at);
}

// Position and loads of a thread over units [first, last) of a row.
struct UnitReader {
  SliceCursor k;
  int i, last, step;
  __device__ __forceinline__ UnitReader(const SliceArgs& a, int first, int last_, int thread, int threads)
      : i(first + thread), last(last_), step(threads) {
    k.start(i < last ? i : 0, a.per_slice);
  }
  // The next kBatch units (-inf past the end).
  __device__ __forceinline__ void load(const SliceArgs& a, int row, float4 (&v)[kBatch], uint64_t policy) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      v[u] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (i < last) {
        v[u] = ldg_hint4(unit_ptr(a, row, k), policy);
        i += step;
        if (i < last) k.advance(step, a.per_slice);
      }
    }
  }
};

// The token, where it is one of the thread's own among units [first, last), else
// -1 (threads: a power of two).
__device__ __forceinline__ int own_token(int token, int first, int last, int thread, int threads) {
  const int u = token >> 2;
  return u >= first && u < last && ((u - first) & (threads - 1)) == thread ? token : -1;
}
// Leaves the own token out of the batch whose first unit is i.
__device__ __forceinline__ void drop_token(float4 (&v)[kBatch], int own, int i, int step) {
  const int unit = own >> 2;
  if (unit >= i && unit < i + kBatch * step) {  // rare; never for -1
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (unit == i + u * step) {
        const int j = own & 3;
        v[u] = make_float4(j == 0 ? -INFINITY : v[u].x, j == 1 ? -INFINITY : v[u].y, j == 2 ? -INFINITY : v[u].z,
                           j == 3 ? -INFINITY : v[u].w);
      }
  }
}

// A CTA's threads bring their sums together: each warp's into shared memory,
// then warp 0 (after a barrier) adds them up.  k0: the exponent the threads
// began with.
struct WarpSums {
  float z, w, k;
};
template <bool ENT>
__device__ __forceinline__ void fast_warp_sums(FastSums s, float k, float k0, WarpSums* shared, int warp, int lane) {
  const float top = __all_sync(0xFFFFFFFFu, k == k0) ? k0 : warp_max(k);
  if (k != top) fast_rebase<ENT>(s, k, top);
  const float z = warp_sum(s.z.x + s.z.y);
  const float w = ENT ? warp_sum(s.w.x + s.w.y) : 0.0f;
  if (lane == 0) shared[warp] = WarpSums{z, w, top};
}
template <bool ENT, int WARPS>
__device__ __forceinline__ PartStats fast_part(const WarpSums* shared, int lane) {
  static_assert(WARPS <= 16, "lanes 0 .. 15 hold the result");
  PartStats p{0.0, 0.0, shared[0].k};
  if (lane < WARPS) {
    p.z = shared[lane].z;
    p.w = shared[lane].w;
    p.ref = shared[lane].k;
  }
  if (!__all_sync(0xFFFFFFFFu, p.ref == shared[0].k)) {  // rare: a warp renewed its k
    float ref = p.ref;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xFFFFFFFFu, ref, o));
    const double d = fmax(static_cast<double>(p.ref) - static_cast<double>(ref), -2000.0), f = exp2_int(d);
    p.w = (p.w + d * p.z) * f;
    p.z *= f;
    p.ref = ref;
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    p.z += __shfl_xor_sync(0xFFFFFFFFu, p.z, o);
    if (ENT) p.w += __shfl_xor_sync(0xFFFFFFFFu, p.w, o);
  }
  p.w *= kLn2;
  return p;
}

// The careful sums of units [first, last) but the token, by `threads` threads;
// each warp's first lane leaves them in `shared`.
__device__ __noinline__ void careful_warp_sums(const SliceArgs& a, int row, int token, int first, int last, int thread,
                                               int threads, CarefulSums* shared) {
  UnitReader reader(a, first, last, thread, threads);
  CarefulSums s = careful_empty();
  const uint64_t policy = policy_evict_last();
  const int own = own_token(token, first, last, thread, threads);
  while (reader.i < last) {
    float4 v[kBatch];
    const int i = reader.i;
    reader.load(a, row, v, policy);
    drop_token(v, own, i, threads);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) careful_add(s, v[u], a.c);
  }
  __syncwarp();
  const float m = warp_max(s.m);
  if (s.m != m) careful_rebase(s, m, a.c);
  s.z = warp_sum(s.z);
  s.w = warp_sum(s.w);
  if ((thread & 31) == 0) shared[thread >> 5] = s;
}
__device__ __forceinline__ PartStats careful_part(const CarefulSums* shared, int lane, int warps, const ExpScale& c) {
  PartStats p{0.0, 0.0, -FLT_MAX};
  if (lane < warps) {
    p.z = shared[lane].z;
    p.w = static_cast<double>(shared[lane].w) * c.inv_t;
    p.ref = shared[lane].m;
  }
  return merge_parts<false, 32>(p, c);
}

// One CTA's part of a row, as the CTAs of a cluster exchange it.
struct alignas(16) PartSlot {
  double z, w;
  float ref, pad[3];
};
__device__ __forceinline__ void send_part(PartSlot* slot, uint32_t rank, const PartStats& p) {
  const uint32_t at = mapa(smem_u32(slot), rank);
  st_dsmem_f64(at, p.z);
  st_dsmem_f64(at + 8, p.w);
  st_dsmem_u32(at + 16, __float_as_uint(p.ref));
}
__device__ __forceinline__ PartStats lane_part(const PartSlot* slots, int lane, int parts) {
  PartStats p{0.0, 0.0, -FLT_MAX};
  if (lane < parts) {
    p.z = slots[lane].z;
    p.w = slots[lane].w;
    p.ref = slots[lane].ref;
  }
  return p;
}

__device__ __forceinline__ float token_logit(const SliceArgs& a, int row, int token) {
  const int s = token / a.V_s;
  return a.slices[s][static_cast<size_t>(row) * a.V_s + (token - s * a.V_s)];
}

__device__ __forceinline__ void store_unit(float* p, const float4& g, uint64_t policy) {
  stg_hint4(p, __float_as_uint(g.x), __float_as_uint(g.y), __float_as_uint(g.z), __float_as_uint(g.w), policy);
}
__device__ __forceinline__ void store_unit(__nv_bfloat16* p, const float4& g, uint64_t policy) {
  // one rounding to bf16 at the end: the next step is a bf16 matrix product
  __nv_bfloat162 lo = __floats2bfloat162_rn(g.x, g.y), hi = __floats2bfloat162_rn(g.z, g.w);
  stg_hint2(p, reinterpret_cast<uint32_t&>(lo), reinterpret_cast<uint32_t&>(hi), policy);
}

// A row's gradient coefficients (see the file's head): G_j = e_j (alpha + gamma
// y_j), where y_j is what e_j is taken from: the exponent c l_j - ref of 2
// (fast), or l_j - ref (careful).  at_token: what comes to it at the token, or,
// where the row's sums are at hand in 64 bits (token_grad), its value.
struct GradCoef {
  float ref, alpha, gamma, at_token;
  int token;  // -1: the row does not count, its gradient is 0
  int careful;
};

// From df / dlogp = g and df / dH = h.
template <bool FAST>
__device__ __forceinline__ GradCoef grad_coef(double g, double h, double z, double log_z, double entropy, float ref,
                                              const ExpScale& c, int token) {
  GradCoef k;
  k.ref = ref;
  k.token = token;
  k.careful = !FAST;
  const double f = -c.inv_t * kExpMean / z;  // 1 / z of the exponentials as they are computed
  k.alpha = static_cast<float>(f * (h != 0.0 ? g + h * (entropy - log_z) : g));
  k.gamma = h != 0.0 ? static_cast<float>(f * h * (FAST ? kLn2 : c.inv_t)) : 0.0f;
  k.at_token = static_cast<float>(g * c.inv_t);
  return k;
}

// The gradient at the token, in 64 bits: 1 - p (`rest`) of a token that is nearly
// certain is no difference of two numbers near 1.
__device__ __forceinline__ float token_grad(double g, double h, double logprob, double rest, double entropy,
                                            const ExpScale& c) {
  double v = g * rest;
  if (h != 0.0 && rest != 1.0) v -= h * (1.0 - rest) * (logprob + entropy);
  return static_cast<float>(v * c.inv_t);
}

struct GradArgs {
  void* grad[VSL_MAX_SLICES];
};

// What at_token is to the gradient at the token: its value, or what is added.
template <bool SET>
__device__ __forceinline__ void at_the_token(const GradCoef& k, int i, float4& g) {
  const int at = k.token - 4 * i;
  if (at >= 0 && at < 4) {
    if (at == 0) g.x = SET ? k.at_token : g.x + k.at_token;
    if (at == 1) g.y = SET ? k.at_token : g.y + k.at_token;
    if (at == 2) g.z = SET ? k.at_token : g.z + k.at_token;
    if (at == 3) g.w = SET ? k.at_token : g.w + k.at_token;
  }
}

// Gradient of one unit (the i-th of the row) from its logits.
template <bool SET>
__device__ __forceinline__ float4 unit_grad(const float4& x, const GradCoef& k, const ExpScale& c, int i) {
  const float v[4] = {x.x, x.y, x.z, x.w};
  float g[4];
  if (!k.careful && k.gamma == 0.0f) {  // no entropy in it: alpha e_j
    const float2 cc = make_float2(c.c, c.c), kk = make_float2(-k.ref, -k.ref), alpha = make_float2(k.alpha, k.alpha);
    const float2 y0 = fma2(make_float2(x.x, x.y), cc, kk), y1 = fma2(make_float2(x.z, x.w), cc, kk);
    const float2 g0 = mul2(make_float2(exp2_fast(y0.x), exp2_fast(y0.y)), alpha);
    const float2 g1 = mul2(make_float2(exp2_fast(y1.x), exp2_fast(y1.y)), alpha);
    g[0] = g0.x;
    g[1] = g0.y;
    g[2] = g1.x;
    g[3] = g1.y;
  } else if (!k.careful) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = max_nan(__fmaf_rn(v[j], c.c, -k.ref), -200.0f);
      g[j] = exp2_fast(y) * __fmaf_rn(k.gamma, y, k.alpha);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = v[j] - k.ref;
      g[j] = exp_of(t, c) * __fmaf_rn(k.gamma, finite_low(t), k.alpha);
    }
  }
  float4 r = make_float4(g[0], g[1], g[2], g[3]);
  at_the_token<SET>(k, i, r);
  return r;
}

// Gradient of units [first, last) of a row from global memory, a slice's run
// at a time.
template <typename T, bool SET, int BATCH = kBatch>
__device__ __forceinline__ void part_grad(const SliceArgs& a, const GradArgs& out, const GradCoef& k, int row,
                                          int first, int last, int thread, int threads) {
  SliceCursor run;
  run.start(min(first, a.units - 1), a.per_slice);
  const size_t row_at = static_cast<size_t>(row) * a.V_s;
  const uint64_t once = policy_evict_first();
  for (int u = first; u < last;) {
    const int n = min(last - u, a.per_slice - run.at);
    const size_t at = row_at + 4 * static_cast<size_t>(run.at);
    const float* src = a.slices[run.slice] + at;
    T* dst = static_cast<T*>(out.grad[run.slice]) + at;
    for (int i = thread; i < n; i += BATCH * threads) {
      float4 x[BATCH];
      if (k.token >= 0) {
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
          if (i + b * threads < n) x[b] = ldg_hint4(src + 4 * (i + b * threads), once);
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
          if (i + b * threads < n) x[b] = unit_grad<SET>(x[b], k, a.c, u + i + b * threads);
      } else {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) x[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
        if (i + b * threads < n) store_unit(dst + 4 * (i + b * threads), x[b], once);
    }
    u += n;
    run.at = 0;
    ++run.slice;
  }
}

struct LogprobArgs {
  SliceArgs in;
  const int32_t* tokens;
  float* logprob;
  float* entropy;  // may be null
  float2* stats;   // may be null
  int cluster;     // CTAs per row
  int per_part;    // units per CTA
};

// A cluster per row: each CTA streams a part of the row once; the CTAs exchange
// their sums over distributed shared memory.  Bound by DRAM where there are rows
// enough (2,048 of 151,936: 194 us, 6.4 TB/s; 512: 51 us, 6.1 TB/s, the last,
// partial set of CTAs in it), by the chain of load, sums, exchange and the row's
// arithmetic where there are few (64 rows of 248,320: 12.7 us; 4 of 1,024: 4.5 us).
template <bool ENT, int THREADS>
__global__ void __launch_bounds__(THREADS, kLogprobThreads / THREADS)
    token_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int kWarps = THREADS / 32;
  __shared__ float first_max[kWarps];
  __shared__ WarpSums warps[kWarps];
  __shared__ CarefulSums careful_warps[kWarps];
  __shared__ PartSlot slots[2][kMaxCluster];
  __shared__ float logit;  // the token's
  __shared__ int redo;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int row = static_cast<int>(blockIdx.x) / a.cluster;
  const int token = a.tokens[row];
  if (token < 0 || token >= 4 * a.in.units) {  // the whole cluster's: the row does not count
    if (rank == 0 && threadIdx.x == 0) {
      a.logprob[row] = 0.0f;
      if (ENT) a.entropy[row] = 0.0f;
      if (a.stats != nullptr) a.stats[row] = make_float2(0.0f, 1.0f);
    }
    return;
  }
  cluster_arrive();  // this CTA runs; waited for before the first access to another's memory
  const int first = min(a.in.units, rank * a.per_part), last = min(a.in.units, first + a.per_part);
  const uint64_t policy = policy_evict_first();
  UnitReader reader(a.in, first, last, threadIdx.x, THREADS);
  const int own = own_token(token, first, last, threadIdx.x, THREADS);
  float4 v[kBatch];
  int at = reader.i;
  reader.load(a.in, row, v, policy);
  drop_token(v, own, at, THREADS);
  if (threadIdx.x == 0) logit = token_logit(a.in, row, token);
  float m = -FLT_MAX;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) m = fmaxf(m, fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w)));
  m = warp_max(m);
  if (lane == 0) first_max[warp] = m;
  __syncthreads();
  const float k0 = fast_reference(warp_max(first_max[lane % kWarps]), a.in.c.c);
  float k = k0;
  FastSums s{};
#pragma unroll
  for (int u = 0; u < kBatch; ++u) fast_add<ENT>(s, v[u], a.in.c.c, k);
  while (reader.i < last) {
    at = reader.i;
    reader.load(a.in, row, v, policy);
    drop_token(v, own, at, THREADS);
    fast_batch<ENT>(s, k, v, a.in.c.c);
  }
  fast_warp_sums<ENT>(s, k, k0, warps, warp, lane);
  __syncthreads();
  cluster_wait();  // every CTA of the cluster runs
  if (warp == 0) {
    const PartStats p = fast_part<ENT, kWarps>(warps, lane);
    if (lane < a.cluster) send_part(&slots[0][rank], lane, p);
  }
  cluster_arrive();
  TokenTerm term{};
  if (warp == 0) term = token_term(logit, a.in.c);  // while the sums travel
  cluster_wait();  // also: no CTA leaves while another may write to it
  if (warp == 0) {
    const PartStats part = lane_part(slots[0], lane, a.cluster);
    bool ok = __all_sync(0xFFFFFFFFu, lane >= a.cluster || fast_holds(part)) && term.holds;
    const RowStats p = add_token(merge_parts<true, kMaxCluster>(part, a.in.c), term, logit, a.in.c);
    ok = ok && __shfl_sync(0xFFFFFFFFu, p.z, 0) >= kFastLeast;  // the whole warp's decision
    if (ok && rank == 0) {
      const RowScore r = row_score<true, ENT>(p, logit, a.in.c);
      if (lane == 0) {
        a.logprob[row] = static_cast<float>(r.logprob);
        if (ENT) a.entropy[row] = static_cast<float>(r.entropy);
        if (a.stats != nullptr) a.stats[row] = make_float2(p.ref, static_cast<float>(r.z));
      }
    }
    if (lane == 0) redo = !ok;
  }
  __syncthreads();
  if (!redo) return;  // the cluster's CTAs agree: they saw the same sums
  careful_warp_sums(a.in, row, token, first, last, threadIdx.x, THREADS, careful_warps);
  __syncthreads();
  if (warp == 0) {
    const PartStats p = careful_part(careful_warps, lane, kWarps, a.in.c);
    if (lane < a.cluster) send_part(&slots[1][rank], lane, p);
  }
  cluster_sync();
  if (rank != 0 || warp != 0) return;
  const RowStats p =
      add_token_careful(merge_parts<false, kMaxCluster>(lane_part(slots[1], lane, a.cluster), a.in.c), logit, a.in.c);
  const RowScore r = row_score<false, ENT>(p, logit, a.in.c);
  if (lane == 0) {
    a.logprob[row] = static_cast<float>(r.logprob);
    if (ENT) a.entropy[row] = static_cast<float>(r.entropy);
    if (a.stats != nullptr) a.stats[row] = make_float2(p.ref, -static_cast<float>(r.z));  // the sign: careful
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

// Four CTAs of 512 threads an SM, each 8 units of a row a thread, two loads in
// flight: no sum is shared, so the work is cut finely.  Bound by DRAM: 512 rows of
// 151,936 100 us to float32 (6.2 TB/s of one read and one write), 85 us to bf16
// (5.5); with the entropy's derivative 103 and 89.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_grad_kernel(const __grid_constant__ LogprobGradArgs a) {
  const int row = static_cast<int>(blockIdx.x) / a.parts;
  const int first = (static_cast<int>(blockIdx.x) - row * a.parts) * a.per_part;
  const int last = min(a.in.units, first + a.per_part);
  const int token = a.tokens[row];
  GradCoef k{};
  k.token = -1;
  const double g = a.d_logprob[row], h = a.d_entropy != nullptr ? a.d_entropy[row] : 0.0f;
  if (token >= 0 && token < 4 * a.in.units && (g != 0.0 || h != 0.0)) {
    const float2 s = a.stats[row];
    const double z = fabs(static_cast<double>(s.y)), ent = h != 0.0 ? a.entropy[row] : 0.0f;
    k = s.y < 0.0f ? grad_coef<false>(g, h, z, log(z), ent, s.x, a.in.c, token)
                   : grad_coef<true>(g, h, z, log(z), ent, s.x, a.in.c, token);
  }
  part_grad<T, false, 2>(a.in, a.out, k, row, first, last, threadIdx.x, kThreads);
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
  int cluster;   // CTAs per row
  int per_part;  // units per CTA
};

// A row's own inputs, read before its sums are ready.
struct RowInputs {
  float logit, old_logprob, ref_logprob, advantage, weight;
};
__device__ __forceinline__ void row_inputs(const PolicyArgs& a, int row, int token, RowInputs& r) {
  // the token's logit, before any CTA may write the gradient over it
  r.logit = token_logit(a.in, row, token);
  r.old_logprob = a.old_logprob[row];
  r.ref_logprob = a.ref_logprob != nullptr ? a.ref_logprob[row] : 0.0f;
  r.advantage = a.advantages[row];
  r.weight = a.weights != nullptr ? a.weights[row] : 1.0f;
}

// The row's loss and outputs, and its gradient coefficients, by one warp (every
// lane holds p, the row's sums with the token's term).
template <bool FAST, bool ENT>
__device__ __forceinline__ GradCoef policy_row(const PolicyArgs& a, int row, int token, const RowInputs& in,
                                               const RowStats& p, int lane, bool write) {
  const RowScore r = row_score<FAST, ENT>(p, in.logit, a.in.c);
  const double w = in.weight, adv = in.advantage;
  const double d = static_cast<double>(in.ref_logprob) - r.logprob;
  // exp(logprob - old) - 1 and exp(ref - logprob) - 1 side by side
  const double em = expm1(lane == 1 ? d : r.logprob - static_cast<double>(in.old_logprob));
  const double ratio = __shfl_sync(0xFFFFFFFFu, em, 0) + 1.0, em_d = __shfl_sync(0xFFFFFFFFu, em, 1);
  const double low = 1.0 - static_cast<double>(a.clip_low), high = 1.0 + static_cast<double>(a.clip_high);
  const double free_term = ratio * adv, clip_term = fmin(fmax(ratio, low), high) * adv;
  double loss = free_term != free_term ? NAN : -(free_term <= clip_term ? free_term : clip_term);
  double g = free_term != free_term ? NAN : free_term <= clip_term ? -adv * ratio : 0.0;
  double kl = 0.0;
  if (a.ref_logprob != nullptr) {
    kl = d > 700.0 ? INFINITY : em_d - d;  // not inf - inf
    if (a.kl_coef != 0.0f) {
      loss += static_cast<double>(a.kl_coef) * kl;
      g -= static_cast<double>(a.kl_coef) * em_d;
    }
  }
  double h = 0.0;
  if (a.entropy_coef != 0.0f) {
    loss -= static_cast<double>(a.entropy_coef) * r.entropy;
    h = -w * static_cast<double>(a.entropy_coef);
  }
  if (write && lane == 0) {
    a.loss[row] = static_cast<float>(w * loss);
    if (a.logprob != nullptr) a.logprob[row] = static_cast<float>(r.logprob);
    if (a.kl != nullptr) a.kl[row] = static_cast<float>(kl);
    if (a.entropy != nullptr) a.entropy[row] = static_cast<float>(r.entropy);
  }
  GradCoef k = grad_coef<FAST>(w * g, h, r.z, r.log_z, r.entropy, p.ref, a.in.c, token);
  k.at_token = token_grad(w * g, h, r.logprob, p.rest / r.z, r.entropy, a.in.c);
  return k;
}

// A cluster per row.  KEEP: its threads hold the row in registers between the
// two passes.  Else its CTAs stream the row once for the sums, exchange them
// over distributed shared memory, and read their parts again for the gradient,
// out of the L2 cache: the first reading asks it to keep the lines, the second
// and the gradient's stores to let theirs go first (2,048 rows of 151,936: 517 us,
// 519 if the first asks nothing).
//
// DRAM sees the row once (512 rows of 151,936: 347 MB read of 311 without the
// second reading, 259 MB written): 135 us to float32, 115 to bf16; 2,048 rows
// 517 and 432 us, 4.8 and 4.3 TB/s.  What bounds it is that a row's phases wait
// on one another (read, exchange, the row's arithmetic in 64 bits, read and
// write): the rows beside it on the SM fill the gaps only in part.  A form that
// kept the row in a cluster's shared memory, fed by TMA through a ring, took 588
// us for the 2,048 rows where this took 495 then: fewer rows at a time, longer gaps.
template <typename T, bool ENT, bool KEEP, int THREADS>
__global__ void __launch_bounds__(THREADS, (KEEP ? 1024 : kRowThreads) / THREADS)
    policy_loss_kernel(const __grid_constant__ PolicyArgs a) {
  constexpr int kWarps = THREADS / 32;
  __shared__ float first_max[kWarps];
  __shared__ WarpSums warps[kWarps];
  __shared__ CarefulSums careful_warps[kWarps];
  __shared__ PartSlot slots[2][kMaxCluster];
  __shared__ RowInputs in;
  __shared__ GradCoef coef;
  __shared__ int redo;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int row = static_cast<int>(blockIdx.x) / a.cluster;
  const int first = min(a.in.units, rank * a.per_part), last = min(a.in.units, first + a.per_part);
  const int token = a.tokens[row];
  if (token < 0 || token >= 4 * a.in.units || (a.weights != nullptr && a.weights[row] == 0.0f)) {
    if (rank == 0 && threadIdx.x == 0) {
      a.loss[row] = 0.0f;
      if (a.logprob != nullptr) a.logprob[row] = 0.0f;
      if (a.kl != nullptr) a.kl[row] = 0.0f;
      if (a.entropy != nullptr) a.entropy[row] = 0.0f;
    }
    GradCoef off{};
    off.token = -1;
    if (a.grad) part_grad<T, true>(a.in, a.out, off, row, first, last, threadIdx.x, THREADS);
    return;
  }
  cluster_arrive();  // this CTA runs; waited for before the first access to another's memory
  const uint64_t keep = KEEP ? policy_evict_first() : policy_evict_last();
  UnitReader reader(a.in, first, last, threadIdx.x, THREADS);
  const int own = own_token(token, first, last, threadIdx.x, THREADS);
  float4 v[kBatch];
  int at = reader.i;
  reader.load(a.in, row, v, keep);
  drop_token(v, own, at, THREADS);
  if (threadIdx.x == 0) row_inputs(a, row, token, in);
  float m = -FLT_MAX;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) m = fmaxf(m, fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w)));
  m = warp_max(m);
  if (lane == 0) first_max[warp] = m;
  __syncthreads();
  const float k0 = fast_reference(warp_max(first_max[lane % kWarps]), a.in.c.c);
  float k = k0;
  FastSums s{};
#pragma unroll
  for (int u = 0; u < kBatch; ++u) fast_add<ENT>(s, v[u], a.in.c.c, k);
  while (!KEEP && reader.i < last) {
    at = reader.i;
    reader.load(a.in, row, v, keep);
    drop_token(v, own, at, THREADS);
    fast_batch<ENT>(s, k, v, a.in.c.c);
  }
  fast_warp_sums<ENT>(s, k, k0, warps, warp, lane);
  __syncthreads();
  cluster_wait();  // every CTA of the cluster runs
  if (warp == 0) {
    const PartStats p = fast_part<ENT, kWarps>(warps, lane);
    if (lane < a.cluster) send_part(&slots[0][rank], lane, p);
  }
  cluster_arrive();
  TokenTerm term{};
  if (warp == 0) term = token_term(in.logit, a.in.c);  // while the sums travel
  cluster_wait();  // also: no CTA leaves while another may write to it
  if (warp == 0) {
    const PartStats part = lane_part(slots[0], lane, a.cluster);
    bool ok = __all_sync(0xFFFFFFFFu, lane >= a.cluster || fast_holds(part)) && term.holds;
    const RowStats p = add_token(merge_parts<true, kMaxCluster>(part, a.in.c), term, in.logit, a.in.c);
    ok = ok && __shfl_sync(0xFFFFFFFFu, p.z, 0) >= kFastLeast;  // the whole warp's decision
    if (ok) {
      const GradCoef g = policy_row<true, ENT>(a, row, token, in, p, lane, rank == 0);
      if (lane == 0) coef = g;
    }
    if (lane == 0) redo = !ok;
  }
  __syncthreads();
  if (redo) {  // the cluster's CTAs agree: they saw the same sums
    careful_warp_sums(a.in, row, token, first, last, threadIdx.x, THREADS, careful_warps);
    __syncthreads();
    if (warp == 0) {
      const PartStats p = careful_part(careful_warps, lane, kWarps, a.in.c);
      if (lane < a.cluster) send_part(&slots[1][rank], lane, p);
    }
    cluster_sync();
    if (warp == 0) {
      const RowStats p =
          add_token_careful(merge_parts<false, kMaxCluster>(lane_part(slots[1], lane, a.cluster), a.in.c), in.logit, a.in.c);
      const GradCoef g = policy_row<false, ENT>(a, row, token, in, p, lane, rank == 0);
      if (lane == 0) coef = g;
    }
    __syncthreads();
  }
  if (!a.grad) return;
  if (KEEP) {
    const GradCoef g = coef;
    const uint64_t once = policy_evict_first();
    const int i0 = first + static_cast<int>(threadIdx.x);
    SliceCursor to;
    to.start(min(i0, a.in.units - 1), a.in.per_slice);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * THREADS;
      if (i < last) {
        store_unit(static_cast<T*>(a.out.grad[to.slice]) + static_cast<size_t>(row) * a.in.V_s + 4 * static_cast<size_t>(to.at),
                   unit_grad<true>(v[u], g, a.in.c, i), once);
        if (i + THREADS < last) to.advance(THREADS, a.in.per_slice);
      }
    }
  } else {
    part_grad<T, true>(a.in, a.out, coef, row, first, last, threadIdx.x, THREADS);
  }
}

SliceArgs slice_args(const float* const* logits, int S, int V_s, float temperature) {
  SliceArgs in{};
  for (int s = 0; s < S; ++s) in.slices[s] = logits[s];
  in.per_slice = V_s / 4;
  in.units = S * (V_s / 4);
  in.V_s = V_s;
  in.c = exp_scale(temperature);
  return in;
}

// The SM count of the current device, read once per device.
constexpr int kMaxDevices = 64;
cudaError_t device_sms(int* sms) {
  static std::once_flag once[kMaxDevices];
  static cudaError_t status[kMaxDevices];
  static int count[kMaxDevices];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev],
                 [&] { status[dev] = cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev); });
  *sms = count[dev];
  return status[dev];
}

// Threads of a CTA of the row kernels.  CTAs of 256 finish and make room in
// smaller steps than of 512 (logprobs of 512 rows of 151,936: 51 us, 64 with
// 512; of 2,048: 194 us, 207; policy loss of 300 rows of 51,012: 30 us, 32), of
// 128 only pay on short rows where there are many (logprobs of 4,000 rows of
// 2,000: 11 us with 128, 19 with 256; of 8,000 25, 30; but of 512 rows 5.1 and
// 6.1 with 128, 4.3 and 5.6 with 256; policy loss of 512 rows of 151,936: 149 us
// with 128, 135 with 256).  512 where the rows are so few that a CTA each SM's
// worth would not fill them (policy loss of 16 rows of 262,144: 15.6 us, 16.8
// with 256), and in the policy loss where 256 would leave more rows in flight
// than the L2 cache holds (1,024 rows of 262,144: 450 us, 465).
constexpr float kL2Room = 96.0f * 1048576.0f;  // of 126 MB
int row_threads(int R, int units, bool cached, int sms) {
  if (units <= 2048) return 128;
  const long long places = static_cast<long long>(kRowThreads) * sms;
  if (static_cast<long long>(R) * kMaxCluster * 512 <= places) return 512;
  const float rows = fminf(static_cast<float>(R), static_cast<float>(places / (256 * kMaxCluster)));
  return cached && rows * units * 16.0f > kL2Room ? 512 : 256;
}

// CTAs per row (a power of two): the fewest microseconds by a rough count.  The
// SMs hold kRowThreads threads each, `places` CTAs in all; a full set of CTAs
// takes `per_unit` for each unit a thread has, bound by memory, and `fixed` for
// the steps that wait on one another; a last, partial set goes faster by its
// share, but not faster than a third.  Both constants are fits to measured
// times, and only their ratio matters: it keeps, say, 148 rows from taking 4
// CTAs each, a third more than there are places (policy loss of 148 rows of
// 151,936, CTAs of 512: 50 us with 4, 44 with 2).  `cached`: the rows being worked on at a
// time must leave the L2 cache room, at most 96 MB of its 126 (2,048 rows of
// 151,936: 517 us; 550 with room for 140 MB, 610 with 64).
cudaError_t choose_cluster(int R, int units, float per_unit, float fixed, bool cached, int* cluster, int* threads_out) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int threads = *threads_out = row_threads(R, units, cached, sms);
  const float places = static_cast<float>(kRowThreads) * sms / threads;
  float best = 0.0f;
  *cluster = 0;
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    if (c > 1 && units / c < threads) break;  // a part has a unit or more per thread
    const float sets = static_cast<float>(R) * c / places, whole = floorf(sets), rest = sets - whole;
    const float rows = fminf(static_cast<float>(R), places / c);
    if (cached && c < kMaxCluster && units / (2 * c) >= threads && rows * units * 16.0f > kL2Room) continue;
    const float stream = per_unit * units / (static_cast<float>(c) * threads);
    const float time = whole * (stream + fixed) + (rest > 0.0f ? stream * fmaxf(rest, 0.35f) + fixed : 0.0f);
    if (*cluster == 0 || time < best) {
      best = time;
      *cluster = c;
    }
  }
  return static_cast<long long>(R) * *cluster > 0x7FFFFFFFLL ? cudaErrorInvalidConfiguration : cudaSuccess;
}

cudaError_t row_cluster(int R, int units, int* cluster, int* threads) {
  return choose_cluster(R, units, 0.55f, 5.0f, false, cluster, threads);
}

// keep: the threads hold their parts in registers between the two passes,
// which pays where all CTAs run at once and time is latency (4 rows of 1,024:
// 5.2 us, 5.6 without; 64 rows 5.4, 5.9), not where it halves how many do (300
// rows of 51,012, eight CTAs of 512: 66 us, 55 without).
cudaError_t policy_cluster(int R, int units, int* cluster, int* threads, bool* keep) {
  const cudaError_t e = choose_cluster(R, units, 1.1f, 6.0f, true, cluster, threads);
  if (e != cudaSuccess) return e;
  int sms = 0;
  *keep = units <= *cluster * kBatch * *threads && device_sms(&sms) == cudaSuccess &&
          static_cast<long long>(R) * *cluster * *threads <= 1024LL * sms;
  return cudaSuccess;
}

template <typename Args>
cudaError_t launch_clusters(void (*kernel)(Args), const Args& a, int R, int cluster, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  cfg.gridDim = dim3(static_cast<unsigned>(R) * cluster);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int THREADS>
cudaError_t launch_policy(const PolicyArgs& a, int R, bool ent, bool keep, cudaStream_t stream) {
  auto kernel = ent ? keep ? policy_loss_kernel<T, true, true, THREADS> : policy_loss_kernel<T, true, false, THREADS>
                    : keep ? policy_loss_kernel<T, false, true, THREADS> : policy_loss_kernel<T, false, false, THREADS>;
  return launch_clusters(kernel, a, R, a.cluster, THREADS, stream);
}
template <typename T>
cudaError_t launch_policy(const PolicyArgs& a, int R, int threads, bool ent, bool keep, cudaStream_t stream) {
  return threads == 512   ? launch_policy<T, 512>(a, R, ent, keep, stream)
         : threads == 256 ? launch_policy<T, 256>(a, R, ent, keep, stream)
                          : launch_policy<T, 128>(a, R, ent, keep, stream);
}

template <int THREADS>
cudaError_t launch_logprobs(const LogprobArgs& a, int R, cudaStream_t stream) {
  return launch_clusters(a.entropy != nullptr ? token_logprobs_kernel<true, THREADS> : token_logprobs_kernel<false, THREADS>,
                         a, R, a.cluster, THREADS, stream);
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
  int threads = 0;
  const cudaError_t e = row_cluster(R, a.in.units, &a.cluster, &threads);
  if (e != cudaSuccess) return e;
  a.per_part = (a.in.units + a.cluster - 1) / a.cluster;
  return threads == 512   ? launch_logprobs<512>(a, R, stream)
         : threads == 256 ? launch_logprobs<256>(a, R, stream)
                          : launch_logprobs<128>(a, R, stream);
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
  bool keep = false;
  int threads = 0;
  const cudaError_t e = policy_cluster(R, a.in.units, &a.cluster, &threads, &keep);
  if (e != cudaSuccess) return e;
  a.per_part = (a.in.units + a.cluster - 1) / a.cluster;
  const bool ent = a.entropy != nullptr || a.entropy_coef != 0.0f;
  if (out.grad_type == VSL_GRAD_BF16) return launch_policy<__nv_bfloat16>(a, R, threads, ent, keep, stream);
  return launch_policy<float>(a, R, threads, ent, keep, stream);
}

}  // namespace vsl
