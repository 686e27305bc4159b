// vsl_adapters.cu - low-rank adapters of many requests beside the shared
// vocab-slice projection.
//
// The projection gives every row the base model's logits.  A row r whose
// request uses adapter a adds its own low-rank term:
//   u[r][k]        = scale[a] sum_h hidden[r][h] A[a][k][h],
//   out_s[r][j]    = logits_s[r][j] + sum_k B_s[a][j][k] u[r][k].
// Two kernels.  The first sorts the rows of a tile of 256 by adapter and forms
// units: up to 16 rows of one adapter (or of none); it computes u of each unit
// and leaves the units' rows behind as a plan.  The second passes over the
// logits, a warp to a unit and 128 ids.  Both products run on the tensor cores
// (mma.sync: the 16 rows of a unit are its M, and what bounds the work is the
// logits' and the B's bytes) with bf16 operands and fp32 sums.  A unit's rows
// share one adapter, so no row ever meets another adapter's numbers: one
// request's infinities or NaNs never reach another's row, and no product is
// computed to be thrown away.  u is not rounded to bf16: it is carried as three
// bf16 terms (8 + 8 + 8 bits), each multiplied with B.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "vsl_internal.h"
#include "vsl_ptx.cuh"

namespace vsl {

namespace {

constexpr int kUnitRows = 16;     // rows per tensor-core product
constexpr int kTile = 256;        // rows sorted together
constexpr int kShrinkWarps = 8;   // kShrinkWarps * 32 == kTile: a thread sorts a row
constexpr int kExpandWarps = 4;
constexpr int kTerms = 3;         // bf16 terms of u
constexpr int kFragment = 32 * 4; // 32-bit registers of one A operand (16 x 16 bf16) over a warp
constexpr int kMaxSplit = 4;      // CTAs that share H
constexpr int kFewRows = 2;       // a unit of so few rows is done with float32 multiply-adds

// Products of 16 ranks: one, or an even number (a lane then loads 8 ranks of B
// at a time, which serve two).
__host__ __device__ constexpr int rank_steps(int rank) { return rank <= 16 ? 1 : (rank + 31) / 32 * 2; }
// Units a tile of `rows` rows over n adapters can have: full ones, a ragged one
// per adapter and one of rows without an adapter.
__host__ __device__ constexpr int unit_slots(int rows, int n) {
  const int distinct = n < rows ? n + 1 : rows;
  return rows / kUnitRows + distinct < rows ? rows / kUnitRows + distinct : rows;
}

// The plan of a tile: its units' number, then of each unit the adapter (-1:
// none), the number of rows and (from the fifth word on) the rows, -1 past them.
constexpr int kPlanUnit = 1 + kUnitRows;
__host__ __device__ constexpr size_t plan_ints(int slots) { return 4 + static_cast<size_t>(slots) * (kPlanUnit + 3); }
__device__ __forceinline__ int32_t* plan_unit(int32_t* plan, int slot) { return plan + 4 + slot * (kPlanUnit + 3); }

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 operands, fp32 sums.  Every lane of
// the warp takes part.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct ShrinkArgs {
  const __nv_bfloat16* hidden;
  const __nv_bfloat16* a;
  const float* scale;  // may be null: 1
  const int32_t* ids;
  int32_t* plan;       // [tiles][plan_ints(slots)]
  uint32_t* u;         // [tiles][slots][steps][kTerms][kFragment]: as the second kernel's lanes hold it, or
                       // in a unit of few rows [row][rank] float32
  int R, H, n, rank, slots, split;
};

// CTA (tile, unit, up to 16 GROUPS ranks x a part of H): the warps split the
// part, the CTAs of a cluster share H.
template <int GROUPS>
__global__ void __launch_bounds__(kShrinkWarps * 32) adapters_shrink_kernel(const __grid_constant__ ShrinkArgs p) {
  __shared__ int key[kTile];
  __shared__ int order[kTile];        // sorted position -> row of the tile
  __shared__ int within[kTile];       // sorted position -> rows of its adapter before it
  __shared__ int starts[kTile + 1];   // unit -> its first sorted position
  __shared__ int warp_units[kShrinkWarps];
  constexpr int kRanks = 16 * GROUPS;
  __shared__ float part[kShrinkWarps / 2][kUnitRows][kRanks];
  __shared__ float parts[kMaxSplit][kUnitRows][kRanks];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int slot = static_cast<int>(blockIdx.y), tile = static_cast<int>(blockIdx.x);
  const int split_rank = static_cast<int>(cluster_ctarank());
  const int k0 = static_cast<int>(blockIdx.z) / p.split * kRanks;
  const int row0 = tile * kTile, rows = min(kTile, p.R - row0);

  // ---- sort: rows by (adapter, row), those without an adapter last
  int mine = 0x7FFFFFFF;  // past the tile's end
  if (tid < rows) {
    mine = p.ids[row0 + tid];
    if (mine < 0 || mine >= p.n) mine = p.n;
  }
  key[tid] = mine;
  __syncthreads();
  int before = 0, same = 0;  // rows of smaller adapters; rows of mine before me
  for (int j = 0; j < rows; ++j) {
    const int other = key[j];
    before += other < mine;
    same += (other == mine) & (j < tid);
  }
  const int at = before + same;
  if (tid < rows) {
    order[at] = tid;
    within[at] = same;
  }
  __syncthreads();
  // a unit starts at every 16th row of an adapter; its number: the starts before it
  const bool begins = tid < rows && within[tid] % kUnitRows == 0;
  const uint32_t ballot = __ballot_sync(0xFFFFFFFFu, begins);
  if (lane == 0) warp_units[warp] = __popc(ballot);
  __syncthreads();
  int unit = __popc(ballot & ((1u << lane) - 1u));
  int units = 0;
  for (int w = 0; w < kShrinkWarps; ++w) {
    if (w < warp) unit += warp_units[w];
    units += warp_units[w];
  }
  if (begins) starts[unit] = tid;
  if (tid == 0) starts[units] = rows;
  __syncthreads();
  if (slot >= units) return;  // the whole cluster's
  const int first = starts[slot], count = starts[slot + 1] - first;
  const int adapter = key[order[first]] < p.n ? key[order[first]] : -1;

  // ---- the plan, by the first CTA of the unit
  if (blockIdx.z == 0) {
    int32_t* plan = p.plan + tile * plan_ints(p.slots);
    if (slot == 0 && tid == 0) plan[0] = units;
    int32_t* entry = plan_unit(plan, slot);
    if (tid < kUnitRows) entry[4 + tid] = tid < count ? row0 + order[first + tid] : -1;
    if (tid == kUnitRows) entry[0] = adapter;
    if (tid == kUnitRows + 1) entry[1] = count;
  }
  if (adapter < 0) return;

  // ---- u of the unit: 16 rows x kRanks ranks
  const int g = lane >> 2, t = lane & 3;
  const bool row_ok[2] = {g < count, g + 8 < count};
  const __nv_bfloat16* h_row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    h_row[i] = p.hidden + static_cast<size_t>(row0 + order[first + (row_ok[i] ? g + 8 * i : 0)]) * p.H;
  const __nv_bfloat16* a_row = p.a + (static_cast<size_t>(adapter) * p.rank + k0 + g) * p.H;
  float d[2 * GROUPS][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // 32 columns of H a step: a lane's 8 consecutive ones serve two products
  // (the order of the summed index is free, the same on both sides).  The
  // loop's bound is the warp's, not the lane's: every lane takes part in a
  // product, with zeros past the end of H.
#pragma unroll (GROUPS > 2 ? 2 : 4)
  for (int h0 = (split_rank * kShrinkWarps + warp) * 32; h0 < p.H; h0 += p.split * kShrinkWarps * 32) {
    const int h = h0 + 8 * t;
    const bool in = h < p.H;
    uint4 x[2], y[2 * GROUPS];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = in && row_ok[i] ? __ldg(reinterpret_cast<const uint4*>(h_row[i] + h)) : zero;
#pragma unroll
    for (int i = 0; i < 2 * GROUPS; ++i)
      y[i] = in && k0 + 8 * i + g < p.rank
                 ? __ldg(reinterpret_cast<const uint4*>(a_row + static_cast<size_t>(8 * i) * p.H + h))
                 : zero;
#pragma unroll
    for (int i = 0; i < 2 * GROUPS; ++i) {
      mma_16816(d[i], x[0].x, x[1].x, x[0].y, x[1].y, y[i].x, y[i].y);
      mma_16816(d[i], x[0].z, x[1].z, x[0].w, x[1].w, y[i].z, y[i].w);
    }
  }
  // the warps' sums: the upper four's first, then the lower four add theirs
  float* mine_part = &part[warp % (kShrinkWarps / 2)][0][0];
#pragma unroll
  for (int round = 0; round < 2; ++round) {
    if (warp / (kShrinkWarps / 2) == 1 - round) {
#pragma unroll
      for (int i = 0; i < 2 * GROUPS; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float& to = mine_part[(g + 8 * (q >> 1)) * kRanks + 8 * i + 2 * t + (q & 1)];
          to = round == 0 ? d[i][q] : to + d[i][q];
        }
    }
    __syncthreads();
  }
  for (int e = tid; e < kUnitRows * kRanks; e += kShrinkWarps * 32) {
    float u = 0.0f;
#pragma unroll
    for (int w = 0; w < kShrinkWarps / 2; ++w) u += (&part[w][0][0])[e];
    *cluster_ptr(&parts[split_rank][0][0] + e, 0) = u;
  }
  cluster_sync();  // no access to another CTA's memory follows
  if (split_rank != 0) return;
  const int steps = rank_steps(p.rank);
  uint32_t* unit_u = p.u + (static_cast<size_t>(tile) * p.slots + slot) * steps * kTerms * kFragment;
  for (int e = tid; e < kUnitRows * kRanks; e += kShrinkWarps * 32) {
    const int r = e / kRanks, rank = k0 + e % kRanks;
    if (rank >= 16 * steps) continue;
    float u = (&parts[0][0][0])[e];
    for (int c = 1; c < p.split; ++c) u += (&parts[c][0][0])[e];
    if (p.scale != nullptr) u *= p.scale[adapter];
    if (count <= kFewRows) {  // kept as it is, [row][padded rank]
      if (r < count) reinterpret_cast<float*>(unit_u)[r * steps * 16 + rank] = u;
      continue;
    }
    // Where the second kernel's A operand has this rank.  A lane's B holds 4
    // consecutive ranks (one step: operand columns 2 t, 2 t + 1, 2 t + 8, 2 t + 9)
    // or 8 (two steps, 4 each); the operand's registers are (row g, columns 2 t ..),
    // (row g + 8, 2 t ..), (row g, 2 t + 8 ..), (row g + 8, 2 t + 8 ..).
    const int in_block = rank & 31;
    const int of_lane = steps == 1 ? rank & 3 : in_block & 7, quad = steps == 1 ? rank >> 2 : in_block >> 3;
    const int step = steps == 1 ? 0 : rank / 32 * 2 + (of_lane >> 2);
    const int reg = (r >> 3) + 2 * ((of_lane >> 1) & 1);
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(unit_u + step * kTerms * kFragment) +
                         2 * (4 * (4 * (r & 7) + quad) + reg) + (rank & 1);
#pragma unroll
    for (int i = 0; i < kTerms; ++i) {
      const __nv_bfloat16 term = __float2bfloat16_rn(u);
      out[2 * i * kFragment] = term;
      const float v = __bfloat162float(term);
      u = isfinite(v) ? u - v : 0.0f;  // exact
    }
  }
}

struct ExpandArgs {
  const float* logits[VSL_MAX_SLICES];
  float* out[VSL_MAX_SLICES];
  const __nv_bfloat16* b[VSL_MAX_SLICES];
  const int32_t* plan;
  const uint32_t* u;
  float* stats;  // may be null
  int V_s, rank, S, B, slots;
  int slot_ctas;   // CTAs over the slots of all tiles
  int warp_blocks; // blocks of 128 ids a warp takes
  int tiles;
  int in_place;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tile statistics of half a block (64 ids) of a row: the row's 4 lanes (same g)
// hold 8 logits of each of its two quarters (v[b] = ids 16 b + 4 t ..), -inf
// past the slice's end.  Every lane of the four holds the result.
struct HalfStats {
  float q[2], sum, mn, am;
};
__device__ __forceinline__ HalfStats half_stats(const float4 (&v)[4]) {
  constexpr float kLog2e = 1.4426950408889634f;
  HalfStats s;
  s.mn = INFINITY;
  s.am = INFINITY;
  s.q[0] = s.q[1] = -INFINITY;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float x[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s.q[b >> 1] = fmaxf(s.q[b >> 1], x[j]);
      s.mn = fminf(s.mn, isfinite(x[j]) ? x[j] : INFINITY);
      s.am = fminf(s.am, x[j] != 0.0f ? fabsf(x[j]) : INFINITY);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    s.q[0] = fmaxf(s.q[0], __shfl_xor_sync(0xFFFFFFFFu, s.q[0], o));
    s.q[1] = fmaxf(s.q[1], __shfl_xor_sync(0xFFFFFFFFu, s.q[1], o));
    s.mn = fminf(s.mn, __shfl_xor_sync(0xFFFFFFFFu, s.mn, o));
    s.am = fminf(s.am, __shfl_xor_sync(0xFFFFFFFFu, s.am, o));
  }
  const float top = fmaxf(s.q[0], s.q[1]);
  const float c = isfinite(top) ? top : 0.0f;
  s.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    s.sum += ex2((v[b].x - c) * kLog2e) + ex2((v[b].y - c) * kLog2e) + ex2((v[b].z - c) * kLog2e) +
             ex2((v[b].w - c) * kLog2e);
  s.sum += __shfl_xor_sync(0xFFFFFFFFu, s.sum, 1);
  s.sum += __shfl_xor_sync(0xFFFFFFFFu, s.sum, 2);
  return s;
}
__device__ __forceinline__ void write_stats(const HalfStats& a, const HalfStats& b, float* rec) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float ta = fmaxf(a.q[0], a.q[1]), tb = fmaxf(b.q[0], b.q[1]), top = fmaxf(ta, tb);
  const float c = isfinite(top) ? top : 0.0f;
  // a half without a finite maximum has the sum 0, +inf or NaN whatever it is taken relative to
  const float sum = a.sum * (isfinite(ta) ? ex2((ta - c) * kLog2e) : 1.0f) +
                    b.sum * (isfinite(tb) ? ex2((tb - c) * kLog2e) : 1.0f);
  reinterpret_cast<float4*>(rec)[0] = make_float4(a.q[0], a.q[1], b.q[0], b.q[1]);
  reinterpret_cast<float4*>(rec)[1] = make_float4(sum, fminf(a.mn, b.mn), fminf(a.am, b.am), 0.0f);
}

// A lane's part of B for 64 ids: 4 ranks of an id's row to a load, or 8.
template <int STEPS>
struct BLoad {
  uint4 v[8];
};
template <>
struct BLoad<1> {
  uint2 v[8];
};

__device__ __forceinline__ void load_b(uint2& v, const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ void load_b(uint4& v, const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }

// Operand i of u: from registers, shared memory or global memory.
template <int STEPS, typename Reg, typename Shared>
__device__ __forceinline__ uint4 operand(const Reg& reg, const Shared& shared, const uint4* u, int warp, int lane, int i) {
  if constexpr (STEPS == 1 || STEPS == 2) return reg[i];
  if constexpr (STEPS == 4) return shared[warp][i][lane];
  return u[i * 32];
}
template <int STEPS, typename Reg, typename Shared>
__device__ __forceinline__ void second_step(float (&d)[8][4], const BLoad<STEPS>& y, const Reg& reg,
                                            const Shared& shared, const uint4* u, int warp, int lane, int k) {
  if constexpr (STEPS != 1) {
#pragma unroll
    for (int e = 0; e < kTerms; ++e) {
      const uint4 a = operand<STEPS>(reg, shared, u, warp, lane, (k + 1) * kTerms + e);
#pragma unroll
      for (int i = 0; i < 8; ++i) mma_16816(d[i], a.x, a.y, a.z, a.w, y.v[i].z, y.v[i].w);
    }
  }
}

// Tile statistics of a row of a block whose quarter m is spread over the warp
// as v[m] (-inf past the slice's end).
__device__ __forceinline__ void warp_stats(const float (&v)[4], float* rec, int lane) {
  constexpr float kLog2e = 1.4426950408889634f;
  float q[4], mn = INFINITY, am = INFINITY;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    q[m] = v[m];
    mn = fminf(mn, isfinite(v[m]) ? v[m] : INFINITY);
    am = fminf(am, v[m] != 0.0f ? fabsf(v[m]) : INFINITY);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int m = 0; m < 4; ++m) q[m] = fmaxf(q[m], __shfl_xor_sync(0xFFFFFFFFu, q[m], o));
    mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
    am = fminf(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
  }
  const float top = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3]));
  const float c = isfinite(top) ? top : 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int m = 0; m < 4; ++m) sum += ex2((v[m] - c) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) {
    reinterpret_cast<float4*>(rec)[0] = make_float4(q[0], q[1], q[2], q[3]);
    reinterpret_cast<float4*>(rec)[1] = make_float4(sum, mn, am, 0.0f);
  }
}

__device__ __forceinline__ float dot8(const uint4& b, const float (&u)[8], float sum) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum = __fmaf_rn(__uint_as_float(w[i] << 16), u[2 * i], sum);
    sum = __fmaf_rn(__uint_as_float(w[i] & 0xFFFF0000u), u[2 * i + 1], sum);
  }
  return sum;
}

// Up to ROWS rows of a unit of at most kFewRows over blocks of 128 ids: 15 of 16 rows of a
// tensor-core product would be empty, and what counts is that B, which no other
// row shares, streams in.  LANES lanes hold an id's row of B, 8 ranks each: a
// quarter (32 ids) is LANES loads of 512 contiguous bytes.  The lanes' sums are
// added and dealt out in one butterfly, after which every lane holds one id of
// the quarter: LANES' lane `sub` of the ids' group `at` id (32 / LANES) sub + at.
template <int LANES, int ROWS>
__device__ __forceinline__ void few_rows(const ExpandArgs& p, int adapter, const int32_t* rows, int count, const float* u_rows,
                                         int padded, int block0, int last_block, int lane) {
  constexpr int kPer = 32 / LANES;              // ids of one load
  constexpr int kLoads = LANES < 8 ? LANES : 8; // loads of a quarter in flight
  constexpr int kQuarters = LANES < 8 ? (LANES < 2 ? 4 : 8 / LANES) : 1;  // quarters in flight
  const int sub = lane % LANES, at = lane / LANES;
  const bool ranks_in = 8 * sub < p.rank;
  float u[ROWS][8];
  int row[ROWS];
#pragma unroll
  for (int c = 0; c < ROWS; ++c) {
    row[c] = rows[c < count ? c : 0];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[c][i] = c < count && ranks_in ? u_rows[c * padded + 8 * sub + i] : 0.0f;
  }
  int slice = block0 / p.B, in_slice = block0 - slice * p.B;
#pragma unroll 1
  for (int block = block0; block < last_block; ++block, ++in_slice) {
    if (in_slice == p.B) {
      in_slice = 0;
      ++slice;
    }
    const int j0 = in_slice * 128, most = p.V_s - 1 - j0;
    const __nv_bfloat16* b = p.b[slice] + (static_cast<size_t>(adapter) * p.V_s + j0) * p.rank + 8 * sub;
    const int mine = kPer * sub + at;  // this lane's id of a quarter
    float v[ROWS][4];
#pragma unroll
    for (int c = 0; c < ROWS; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        v[c][m] = -INFINITY;
        if (c < count && 32 * m + mine <= most)
          v[c][m] = p.logits[slice][static_cast<size_t>(row[c]) * p.V_s + j0 + 32 * m + mine];
      }
#pragma unroll
    for (int m0 = 0; m0 < 4; m0 += kQuarters) {
      float part[ROWS][kQuarters][LANES];
#pragma unroll
      for (int i0 = 0; i0 < LANES; i0 += kLoads) {
        uint4 y[kQuarters][kLoads];
#pragma unroll
        for (int q = 0; q < kQuarters; ++q)
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            y[q][i] = make_uint4(0, 0, 0, 0);
            // ids past the slice's end read its last one's row instead (their sums are not kept)
            if (ranks_in) load_b(y[q][i], b + min(32 * (m0 + q) + kPer * (i0 + i) + at, most) * p.rank);
          }
#pragma unroll
        for (int q = 0; q < kQuarters; ++q)
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            part[0][q][i0 + i] = dot8(y[q][i], u[0], 0.0f);
#pragma unroll
            for (int c = 1; c < ROWS; ++c) part[c][q][i0 + i] = count > c ? dot8(y[q][i], u[c], 0.0f) : 0.0f;
          }
      }
#pragma unroll
      for (int c = 0; c < ROWS; ++c)
        if (c < count) {  // the warp's: a butterfly takes all its lanes
#pragma unroll
          for (int q = 0; q < kQuarters; ++q) {
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
              for (int i = 0; i < o; ++i) {
                const float keep = (sub & o) ? part[c][q][i + o] : part[c][q][i];
                const float give = (sub & o) ? part[c][q][i] : part[c][q][i + o];
                part[c][q][i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
              }
            v[c][m0 + q] += part[c][q][0];
          }
        }
    }
#pragma unroll
    for (int c = 0; c < ROWS; ++c)
      if (c < count) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (32 * m + mine <= most)
            p.out[slice][static_cast<size_t>(row[c]) * p.V_s + j0 + 32 * m + mine] = v[c][m];
        if (p.stats != nullptr) warp_stats(v[c], p.stats + (static_cast<size_t>(row[c]) * p.S * p.B + block) * 8, lane);
      }
  }
}

// A warp takes a unit's 16 rows and runs over blocks of 128 ids (of a slice),
// 64 ids at a time.  The products' N index is laid over the ids so that a
// lane's sums are 4 consecutive ids of a row: column n of the i-th product of 8
// is id 16 (i / 2) + 4 (n / 2) + 2 (i mod 2) + n mod 2.  The units of a CTA's
// warps follow one another, so those of one adapter share its B in L1.
template <int STEPS, int LANES>  // rank_steps (0: any even number), lanes of 8 ranks in few_rows
__global__ void __launch_bounds__(kExpandWarps * 32, STEPS == 1 || STEPS == 2 ? 4 : 3)
    adapters_expand_kernel(const __grid_constant__ ExpandArgs p) {
  // u stays in registers for one or two steps, in shared memory for four
  constexpr bool kInRegs = STEPS == 1 || STEPS == 2;
  __shared__ uint4 u_shared[STEPS == 4 ? kExpandWarps : 1][STEPS == 4 ? 4 * kTerms : 1][STEPS == 4 ? 32 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int item = static_cast<int>(blockIdx.x % p.slot_ctas) * kExpandWarps + warp;
  const int block0 = static_cast<int>(blockIdx.x / p.slot_ctas) * p.warp_blocks;
  const int tile = item / p.slots, slot = item - tile * p.slots;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tile >= p.tiles) return;
  const int32_t* plan = p.plan + tile * plan_ints(p.slots);
  const int32_t* entry = plan + 4 + slot * (kPlanUnit + 3);
  if (slot >= plan[0]) return;
  const int adapter = entry[0];
  if (adapter < 0 && p.in_place && p.stats == nullptr) return;  // the base logits stay as they are
  const int last_block = min(block0 + p.warp_blocks, p.S * p.B);
  const int steps = STEPS > 0 ? STEPS : rank_steps(p.rank);
  if (adapter >= 0 && entry[1] <= kFewRows) {  // the whole warp's
    const float* u_rows =
        reinterpret_cast<const float*>(p.u + (static_cast<size_t>(tile) * p.slots + slot) * steps * kTerms * kFragment);
    constexpr int kAtOnce = LANES < 16 ? kFewRows : 1;  // as many as the registers hold
    for (int c = 0; c < entry[1]; c += kAtOnce)
      few_rows<LANES, kAtOnce>(p, adapter, entry + 4 + c, min(entry[1] - c, kAtOnce), u_rows + c * steps * 16, steps * 16,
                               block0, last_block, lane);
    return;
  }
  const int r[2] = {entry[4 + g], entry[4 + g + 8]};
  const uint4* u = reinterpret_cast<const uint4*>(
      p.u + (static_cast<size_t>(tile) * p.slots + slot) * steps * kTerms * kFragment) + lane;
  uint4 u_reg[kInRegs ? STEPS * kTerms : 1];
  if (adapter >= 0) {
    if (kInRegs) {
#pragma unroll
      for (int i = 0; i < STEPS * kTerms; ++i) u_reg[i] = u[i * 32];
    }
    if (STEPS == 4) {
#pragma unroll
      for (int i = 0; i < 4 * kTerms; ++i) u_shared[warp][i][lane] = u[i * 32];  // a lane reads its own back
    }
  }
  const int n_id = 4 * (g >> 1) + (g & 1);  // the id of this lane's column, within 16 ids, of an even product
  constexpr int kLaneRanks = STEPS == 1 ? 4 : 8;  // of one load
  int slice = block0 / p.B, in_slice = block0 - slice * p.B;
#pragma unroll 1
  for (int block = block0; block < last_block; ++block, ++in_slice) {
    if (in_slice == p.B) {
      in_slice = 0;
      ++slice;
    }
    const int j0 = in_slice * 128;
    const size_t base[2] = {static_cast<size_t>(r[0]) * p.V_s + j0 + 4 * t,
                            static_cast<size_t>(r[1]) * p.V_s + j0 + 4 * t};
    const float* src = p.logits[slice];
    float* dst = p.out[slice];
    HalfStats stats[2][2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int jh = j0 + 64 * half;
      float4 x[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          x[i][b] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
          if (r[i] >= 0 && jh + 16 * b + 4 * t < p.V_s)
            x[i][b] = *reinterpret_cast<const float4*>(src + base[i] + 64 * half + 16 * b);
        }
      if (adapter >= 0) {
        // ids past the slice's end read its last one's row instead (their sums are not kept)
        const int most = p.V_s - 1 - jh;
        const __nv_bfloat16* b_base = p.b[slice] + (static_cast<size_t>(adapter) * p.V_s + jh) * p.rank + kLaneRanks * t;
        float d[8][4] = {};
#pragma unroll
        for (int k = 0; k < steps; k += STEPS == 1 ? 1 : 2) {
          BLoad<STEPS> y;
          const bool ranks_in = 16 * k + kLaneRanks * t < p.rank;  // past the rank: zeros
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = min(16 * (i >> 1) + 2 * (i & 1) + n_id, most);
            y.v[i] = {};
            if (ranks_in) load_b(y.v[i], b_base + j * p.rank + 16 * k);
          }
#pragma unroll
          for (int e = 0; e < kTerms; ++e) {
            const uint4 a = operand<STEPS>(u_reg, u_shared, u, warp, lane, k * kTerms + e);
#pragma unroll
            for (int i = 0; i < 8; ++i) mma_16816(d[i], a.x, a.y, a.z, a.w, y.v[i].x, y.v[i].y);
          }
          second_step<STEPS>(d, y, u_reg, u_shared, u, warp, lane, k);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            x[i][b].x += d[2 * b][2 * i];
            x[i][b].y += d[2 * b][2 * i + 1];
            x[i][b].z += d[2 * b + 1][2 * i];
            x[i][b].w += d[2 * b + 1][2 * i + 1];
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (r[i] >= 0 && jh + 16 * b + 4 * t < p.V_s)
            *reinterpret_cast<float4*>(dst + base[i] + 64 * half + 16 * b) = x[i][b];
      if (p.stats != nullptr) {
        stats[0][half] = half_stats(x[0]);
        stats[1][half] = half_stats(x[1]);
      }
    }
    if (p.stats != nullptr && t == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (r[i] >= 0)
          write_stats(stats[i][0], stats[i][1], p.stats + (static_cast<size_t>(r[i]) * p.S * p.B + block) * 8);
    }
  }
}

}  // namespace

namespace {

struct AdapterSizes {
  int tiles, slots;
  size_t plan_bytes, u_bytes;  // each a multiple of 16
};
AdapterSizes adapter_sizes(int R, int n, int rank) {
  AdapterSizes z;
  z.tiles = (R + kTile - 1) / kTile;
  z.slots = unit_slots(R < kTile ? R : kTile, n);
  z.plan_bytes = static_cast<size_t>(z.tiles) * plan_ints(z.slots) * sizeof(int32_t);
  z.u_bytes = static_cast<size_t>(z.tiles) * z.slots * rank_steps(rank) * kTerms * kFragment * sizeof(uint32_t);
  return z;
}

template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), const Args& a, unsigned grid, cudaStream_t stream) {
  // may start before the kernel ahead of it ends; waits for its results itself
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kExpandWarps * 32);
  cfg.stream = stream;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t adapters_workspace_bytes(int R, int n, int rank) {
  const AdapterSizes z = adapter_sizes(R, n, rank);
  return z.plan_bytes + z.u_bytes;
}

cudaError_t launch_adapters_add(const float* const* logits, float* const* out, const void* hidden, int R, int H, int S,
                                int V_s, const void* a, const void* const* b, const float* scale, int n, int rank,
                                const int32_t* ids, float* stats, void* workspace, cudaStream_t stream) {
  const AdapterSizes z = adapter_sizes(R, n, rank);
  ShrinkArgs sa{};
  sa.hidden = static_cast<const __nv_bfloat16*>(hidden);
  sa.a = static_cast<const __nv_bfloat16*>(a);
  sa.scale = scale;
  sa.ids = ids;
  sa.plan = static_cast<int32_t*>(workspace);
  sa.u = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + z.plan_bytes);
  sa.R = R;
  sa.H = H;
  sa.n = n;
  sa.rank = rank;
  sa.slots = z.slots;
  // up to 64 ranks to a CTA; the CTAs of a cluster share longer rows of H while
  // the units are few
  const int steps = rank_steps(rank);
  const int groups = steps < 4 ? steps : 4, ctas = z.tiles * z.slots * ((steps + groups - 1) / groups);
  sa.split = H < 4 * 256 || ctas > 296 ? 1 : ctas > 148 ? 2 : kMaxSplit;
  {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    cfg.gridDim = dim3(z.tiles, z.slots, (steps + groups - 1) / groups * sa.split);
    cfg.blockDim = dim3(kShrinkWarps * 32);
    cfg.stream = stream;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = sa.split;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    auto kernel = groups == 1   ? adapters_shrink_kernel<1>
                  : groups == 2 ? adapters_shrink_kernel<2>
                                : adapters_shrink_kernel<4>;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, sa);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  ExpandArgs ea{};
  ea.in_place = 1;
  for (int s = 0; s < S; ++s) {
    ea.logits[s] = logits[s];
    ea.out[s] = out[s];
    ea.b[s] = static_cast<const __nv_bfloat16*>(b[s]);
    if (logits[s] != out[s]) ea.in_place = 0;
  }
  ea.plan = sa.plan;
  ea.u = sa.u;
  ea.stats = stats;
  ea.V_s = V_s;
  ea.rank = rank;
  ea.S = S;
  ea.B = (V_s + 127) / 128;
  ea.slots = z.slots;
  ea.tiles = z.tiles;
  ea.slot_ctas = static_cast<int>((static_cast<long long>(z.tiles) * z.slots + kExpandWarps - 1) / kExpandWarps);
  // a warp keeps its unit's u over several blocks, while there are warps enough to fill the SMs some times over
  ea.warp_blocks = 1;
  while (ea.warp_blocks < 8 && static_cast<long long>(ea.slot_ctas) * S * ea.B / ea.warp_blocks > 8 * 148 * 4)
    ea.warp_blocks *= 2;
  const long long grid =
      static_cast<long long>(ea.slot_ctas) * ((static_cast<long long>(S) * ea.B + ea.warp_blocks - 1) / ea.warp_blocks);
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  auto kernel = rank <= 8     ? adapters_expand_kernel<1, 1>
                : rank <= 16  ? adapters_expand_kernel<1, 2>
                : rank <= 32  ? adapters_expand_kernel<2, 4>
                : rank <= 64  ? adapters_expand_kernel<4, 8>
                : rank <= 128 ? adapters_expand_kernel<0, 16>
                              : adapters_expand_kernel<0, 32>;
  return launch_after(kernel, ea, static_cast<unsigned>(grid), stream);
}

}  // namespace vsl
