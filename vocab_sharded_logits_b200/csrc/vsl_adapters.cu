// vsl_adapters.cu - low-rank adapters of many requests beside the shared
// vocab-slice projection.
//
// The projection gives every row the base model's logits.  A row r whose
// request uses adapter a adds its own low-rank term:
//   u[r][k]        = scale[a] sum_h hidden[r][h] A[a][k][h],
//   out_s[r][j]    = logits_s[r][j] + sum_k B_s[a][j][k] u[r][k].
// Two kernels: u first (a few hundred KB), then one pass over the logits.
//
// Both products run on the tensor cores with bf16 operands and fp32 sums over
// groups of 16 rows: for each adapter that occurs in a group the product is
// taken for all 16 rows, and each row keeps the result of its own adapter (a
// selection, not a multiplication by 0, so that one request's infinities or
// NaNs never reach another's row).  u is not rounded to bf16: it is carried as
// three bf16 terms (8 + 8 + 8 bits), each multiplied with B.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "vsl_internal.h"
#include "vsl_ptx.cuh"

namespace vsl {

namespace {

constexpr int kGroup = 16;        // rows per tensor-core product
constexpr int kShrinkWarps = 8;
constexpr int kExpandWarps = 4;
constexpr int kTerms = 3;         // bf16 terms of u

__host__ __device__ constexpr int padded_rank(int rank) { return (rank + 15) / 16 * 16; }

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The adapter of row r (-1: none, or an id outside the pool).
__device__ __forceinline__ int adapter_of(const int32_t* ids, int r, int R, int n) {
  const int a = r < R ? ids[r] : -1;
  return a >= 0 && a < n ? a : -1;
}

struct ShrinkArgs {
  const __nv_bfloat16* hidden;
  const __nv_bfloat16* a;
  const float* scale;  // may be null: 1
  const int32_t* ids;
  __nv_bfloat16* u;    // [R][kTerms][padded rank]
  int R, H, n, rank;
};

// u of the rows of one group that use its blockIdx.y-th adapter, ranks 16
// blockIdx.z ..: the warps split H.
__global__ void __launch_bounds__(kShrinkWarps * 32) adapters_shrink_kernel(const __grid_constant__ ShrinkArgs p) {
  __shared__ float part[kShrinkWarps][kGroup][16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int row0 = static_cast<int>(blockIdx.x) * kGroup;
  const int mine = adapter_of(p.ids, row0 + (lane & 15), p.R, p.n);
  uint32_t left = __ballot_sync(0xFFFFFFFFu, mine >= 0) & 0xFFFFu, rows = 0;
  int adapter = -1;
  for (int i = 0; i <= static_cast<int>(blockIdx.y) && left; ++i) {
    adapter = __shfl_sync(0xFFFFFFFFu, mine, __ffs(left) - 1);
    rows = __ballot_sync(0xFFFFFFFFu, mine == adapter) & 0xFFFFu;
    left &= ~rows;
    if (i < static_cast<int>(blockIdx.y)) rows = 0;
  }
  if (rows == 0) return;  // the group has fewer adapters
  const int k0 = static_cast<int>(blockIdx.z) * 16;
  const bool row_ok[2] = {((rows >> g) & 1u) != 0, ((rows >> (g + 8)) & 1u) != 0};
  const bool rank_ok[2] = {k0 + g < p.rank, k0 + 8 + g < p.rank};
  const __nv_bfloat16* h_row[2];
  const __nv_bfloat16* a_row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    h_row[i] = p.hidden + static_cast<size_t>(row_ok[i] ? row0 + g + 8 * i : row0) * p.H;
    a_row[i] = p.a + (static_cast<size_t>(adapter) * p.rank + (rank_ok[i] ? k0 + 8 * i + g : 0)) * p.H;
  }
  float d[2][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // 32 columns of H a step: a lane's 8 consecutive ones serve two products
  // (the order of the summed index is free, the same on both sides)
  // (the loop's bound is the warp's, not the lane's: every lane takes part in
  // a product, with zeros past the end of H)
#pragma unroll 4
  for (int h0 = warp * 32; h0 < p.H; h0 += kShrinkWarps * 32) {
    const int h = h0 + 8 * t;
    const bool in = h < p.H;
    uint4 x[2], y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[i] = in && row_ok[i] ? __ldg(reinterpret_cast<const uint4*>(h_row[i] + h)) : zero;
      y[i] = in && rank_ok[i] ? __ldg(reinterpret_cast<const uint4*>(a_row[i] + h)) : zero;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mma_16816(d[i], x[0].x, x[1].x, x[0].y, x[1].y, y[i].x, y[i].y);
      mma_16816(d[i], x[0].z, x[1].z, x[0].w, x[1].w, y[i].z, y[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    part[warp][g][8 * i + 2 * t] = d[i][0];
    part[warp][g][8 * i + 2 * t + 1] = d[i][1];
    part[warp][g + 8][8 * i + 2 * t] = d[i][2];
    part[warp][g + 8][8 * i + 2 * t + 1] = d[i][3];
  }
  __syncthreads();
  const int r = threadIdx.x >> 4, k = threadIdx.x & 15;
  if (!((rows >> r) & 1u)) return;
  float u = 0.0f;
#pragma unroll
  for (int w = 0; w < kShrinkWarps; ++w) u += part[w][r][k];
  if (p.scale != nullptr) u *= p.scale[adapter];
  const int rp = padded_rank(p.rank);
  __nv_bfloat16* out = p.u + static_cast<size_t>(row0 + r) * kTerms * rp + k0 + k;
#pragma unroll
  for (int i = 0; i < kTerms; ++i) {
    const __nv_bfloat16 term = __float2bfloat16_rn(u);
    out[i * rp] = term;
    const float f = __bfloat162float(term);
    u = isfinite(f) ? u - f : 0.0f;  // exact
  }
}

struct ExpandArgs {
  const float* logits[VSL_MAX_SLICES];
  float* out[VSL_MAX_SLICES];
  const __nv_bfloat16* b[VSL_MAX_SLICES];
  const __nv_bfloat16* u;
  const int32_t* ids;
  float* stats;  // may be null
  int R, V_s, n, rank, S, B;
  int groups;       // row groups
  int cta_groups;   // row groups per CTA (1, 2 or 4 of its warps)
  int in_place;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tile statistics of a row of the block: the row's 4 lanes (same g) hold 8
// logits of each quarter (v[b] = ids 16 b + 4 t ..), -inf past the slice's end.
__device__ __forceinline__ void row_stats(const float4 (&v)[8], float* rec, int t, bool write) {
  constexpr float kLog2e = 1.4426950408889634f;
  float q[4], mn = INFINITY, am = INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = -INFINITY;
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const float x[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[b >> 1] = fmaxf(q[b >> 1], x[j]);
      mn = fminf(mn, isfinite(x[j]) ? x[j] : INFINITY);
      am = fminf(am, x[j] != 0.0f ? fabsf(x[j]) : INFINITY);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fmaxf(q[i], __shfl_xor_sync(0xFFFFFFFFu, q[i], o));
    mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
    am = fminf(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
  }
  const float top = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3]));
  const float c = isfinite(top) ? top : 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int b = 0; b < 8; ++b)
    sum += ex2((v[b].x - c) * kLog2e) + ex2((v[b].y - c) * kLog2e) + ex2((v[b].z - c) * kLog2e) +
           ex2((v[b].w - c) * kLog2e);
  sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
  sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
  if (write && t == 0) {
    reinterpret_cast<float4*>(rec)[0] = make_float4(q[0], q[1], q[2], q[3]);
    reinterpret_cast<float4*>(rec)[1] = make_float4(sum, mn, am, 0.0f);
  }
}

// A warp takes 16 rows x 128 ids (one block of a slice).  The products' N index
// is laid over the ids so that a lane's sums are 4 consecutive ids of a row:
// column n of the i-th product of 8 is id 16 (i / 2) + 4 (n / 2) + 2 (i mod 2) + n mod 2.
__global__ void __launch_bounds__(kExpandWarps * 32) adapters_expand_kernel(const __grid_constant__ ExpandArgs p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int group_ctas = (p.groups + p.cta_groups - 1) / p.cta_groups;
  const int group = static_cast<int>(blockIdx.x % group_ctas) * p.cta_groups + warp % p.cta_groups;
  const int block = static_cast<int>(blockIdx.x / group_ctas) * (kExpandWarps / p.cta_groups) + warp / p.cta_groups;
  if (group >= p.groups || block >= p.S * p.B) return;
  const int slice = block / p.B;
  const int j0 = (block - slice * p.B) * 128;
  const int row0 = group * kGroup;
  const int mine = adapter_of(p.ids, row0 + (lane & 15), p.R, p.n);
  uint32_t left = __ballot_sync(0xFFFFFFFFu, mine >= 0) & 0xFFFFu;
  if (p.in_place && left == 0 && p.stats == nullptr) return;  // the base logits stay as they are
  const int r[2] = {row0 + g, row0 + g + 8};
  const size_t base[2] = {static_cast<size_t>(r[0]) * p.V_s + j0 + 4 * t, static_cast<size_t>(r[1]) * p.V_s + j0 + 4 * t};
  float4 x[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      x[i][b] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (r[i] < p.R && j0 + 16 * b + 4 * t < p.V_s)
        x[i][b] = *reinterpret_cast<const float4*>(p.logits[slice] + base[i] + 16 * b);
    }
  const int rp = padded_rank(p.rank);
  const uint2 zero = make_uint2(0, 0);
  const __nv_bfloat16* u_row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    u_row[i] = p.u + static_cast<size_t>(r[i] < p.R ? r[i] : row0) * kTerms * rp + 4 * t;
  const int n_id = 4 * (g >> 1) + (g & 1);  // the id of this lane's column, within 16 ids, of an even product
  while (left) {
    const int adapter = __shfl_sync(0xFFFFFFFFu, mine, __ffs(left) - 1);
    const uint32_t rows = __ballot_sync(0xFFFFFFFFu, mine == adapter) & 0xFFFFu;
    left &= ~rows;
    const bool own[2] = {((rows >> g) & 1u) != 0, ((rows >> (g + 8)) & 1u) != 0};
    const __nv_bfloat16* b_base = p.b[slice] + (static_cast<size_t>(adapter) * p.V_s + j0) * p.rank + 4 * t;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float d[8][4] = {};
      for (int k = 0; k < rp; k += 16) {
        uint2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = 64 * half + 16 * (i >> 1) + 2 * (i & 1) + n_id;
          y[i] = j0 + j < p.V_s && k + 4 * t < p.rank
                     ? __ldg(reinterpret_cast<const uint2*>(b_base + static_cast<size_t>(j) * p.rank + k))
                     : zero;
        }
#pragma unroll
        for (int e = 0; e < kTerms; ++e) {
          // a row of another adapter is computed too and not kept: zeros stand in for a row that has no u
          const uint2 u0 = own[0] ? *reinterpret_cast<const uint2*>(u_row[0] + e * rp + k) : zero;
          const uint2 u1 = own[1] ? *reinterpret_cast<const uint2*>(u_row[1] + e * rp + k) : zero;
#pragma unroll
          for (int i = 0; i < 8; ++i) mma_16816(d[i], u0.x, u1.x, u0.y, u1.y, y[i].x, y[i].y);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (own[i]) {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float4& v = x[i][4 * half + b];
            v.x += d[2 * b][2 * i];
            v.y += d[2 * b][2 * i + 1];
            v.z += d[2 * b + 1][2 * i];
            v.w += d[2 * b + 1][2 * i + 1];
          }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 8; ++b)
      if (r[i] < p.R && j0 + 16 * b + 4 * t < p.V_s)
        *reinterpret_cast<float4*>(p.out[slice] + base[i] + 16 * b) = x[i][b];
  if (p.stats != nullptr) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      row_stats(x[i], p.stats + (static_cast<size_t>(r[i]) * p.S * p.B + block) * 8, t, r[i] < p.R);
  }
}

}  // namespace

size_t adapters_workspace_bytes(int R, int rank) {
  return (static_cast<size_t>(R) * kTerms * padded_rank(rank) * sizeof(__nv_bfloat16) + 15) / 16 * 16;
}

cudaError_t launch_adapters_add(const float* const* logits, float* const* out, const void* hidden, int R, int H, int S,
                                int V_s, const void* a, const void* const* b, const float* scale, int n, int rank,
                                const int32_t* ids, float* stats, void* workspace, cudaStream_t stream) {
  const int groups = (R + kGroup - 1) / kGroup;
  ShrinkArgs sa{};
  sa.hidden = static_cast<const __nv_bfloat16*>(hidden);
  sa.a = static_cast<const __nv_bfloat16*>(a);
  sa.scale = scale;
  sa.ids = ids;
  sa.u = static_cast<__nv_bfloat16*>(workspace);
  sa.R = R;
  sa.H = H;
  sa.n = n;
  sa.rank = rank;
  const int distinct = R < kGroup ? R : kGroup;
  const dim3 shrink_grid(groups, n < distinct ? n : distinct, padded_rank(rank) / 16);
  adapters_shrink_kernel<<<shrink_grid, kShrinkWarps * 32, 0, stream>>>(sa);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ExpandArgs ea{};
  ea.in_place = 1;
  for (int s = 0; s < S; ++s) {
    ea.logits[s] = logits[s];
    ea.out[s] = out[s];
    ea.b[s] = static_cast<const __nv_bfloat16*>(b[s]);
    if (logits[s] != out[s]) ea.in_place = 0;
  }
  ea.u = sa.u;
  ea.ids = ids;
  ea.stats = stats;
  ea.R = R;
  ea.V_s = V_s;
  ea.n = n;
  ea.rank = rank;
  ea.S = S;
  ea.B = (V_s + 127) / 128;
  ea.groups = groups;
  ea.cta_groups = groups >= 4 ? 4 : groups >= 2 ? 2 : 1;
  const long long group_ctas = (groups + ea.cta_groups - 1) / ea.cta_groups;
  const long long block_ctas = (static_cast<long long>(S) * ea.B + kExpandWarps / ea.cta_groups - 1) /
                               (kExpandWarps / ea.cta_groups);
  if (group_ctas * block_ctas > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  adapters_expand_kernel<<<static_cast<unsigned>(group_ctas * block_ctas), kExpandWarps * 32, 0, stream>>>(ea);
  return cudaGetLastError();
}

}  // namespace vsl
