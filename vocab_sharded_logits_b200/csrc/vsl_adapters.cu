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
// bf16 terms (8 + 8 + 8 bits, cut off one after another), each multiplied with B.
//
// What it cannot do without: one read and one write of the logits and one read
// of each used adapter's A and B.  Measured (H = 4,096 but where stated, of the
// time those bytes take at the 6.56 TB/s of a copy): one row of rank 16 over
// 151,936 ids 7.5 us (two launches, one of which waits for the other's end); 64
// rows of as many adapters of rank 16 73 us, 83 %; 512 rows over 18 adapters of
// rank 32 159 us, 78 %, 184 with tile statistics, 68 %; 2,048 rows over 8
// adapters of rank 64 (H = 5,120) 631 us, 65 %.
//
// Times here and below, but where another is named: calls with given outputs,
// replayed back to back from a graph over the same tensors, the median of five
// allocations.  One allocation differs from another by up to 5 % above 100 us.  A
// program that calls from Python over changing inputs sees 10 us for the one row
// and 672 for the 2,048.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstddef>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "vsl_internal.h"
#include "vsl_ptx_rows.cuh"

namespace vsl {

namespace {

constexpr int kUnitRows = 16;     // rows per tensor-core product
constexpr int kTile = 256;        // rows sorted together
constexpr int kShrinkWarps = 8;   // kShrinkWarps * 32 == kTile: a thread sorts a row
constexpr int kWideWarps = 4;     // most warps of a CTA of the second kernel above rank 64
constexpr int kTerms = 3;         // bf16 terms of u
constexpr int kFragment = 32 * 4; // 32-bit registers of one A operand (16 x 16 bf16) over a warp
constexpr int kMaxSplit = 4;      // CTAs that share H
constexpr int kFewRows = 2;       // see few_rows_of

// Products of 16 ranks: one, or an even number (a lane then loads 8 ranks of B
// at a time, which serve two).
__host__ __device__ constexpr int rank_steps(int rank) { return rank <= 16 ? 1 : (rank + 31) / 32 * 2; }
// Units of at most so many rows are done with float32 multiply-adds: of 16 rows
// of a product 14 or more would be empty, and u is as long as a lane's own share
// of it.  64 rows of as many adapters of rank 16: 73 us, 102 by products; 32
// adapters of two rows 52, 65; at rank 32 126 and 139, but 79 and 77; at rank 64
// the products are as fast, 245 us (245), or faster, 135 (151).
__host__ __device__ constexpr int few_rows_of(int rank) { return rank <= 32 ? kFewRows : 0; }
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

// D = A B.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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

// CTA (tile, unit, 16 ranks x a part of H): the warps split the
// part, the CTAs of a cluster share H.  Every CTA sorts the tile itself, by
// counting, which costs less than a launch that does it once.  Bound by the
// latency of its chain (ids, sort, one run over H, the warps' sums, the
// cluster's): 21 us for 512 rows over 18 adapters of rank 32, 45 us for 2,048
// over 8 of rank 64 (H = 5,120), each alone under the profiler; the second
// kernel's CTAs are already there when it ends.
__global__ void __launch_bounds__(kShrinkWarps * 32) adapters_shrink_kernel(const __grid_constant__ ShrinkArgs p) {
  __shared__ int key[kTile];
  __shared__ int order[kTile];        // sorted position -> row of the tile
  __shared__ int within[kTile];       // sorted position -> rows of its adapter before it
  __shared__ int starts[kTile + 1];   // unit -> its first sorted position
  __shared__ int warp_units[kShrinkWarps];
  constexpr int kRanks = 16;
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
  cluster_arrive();  // this CTA runs; waited for before the first access to another's memory

  // ---- u of the unit: 16 rows x kRanks ranks
  const int g = lane >> 2, t = lane & 3;
  const bool row_ok[2] = {g < count, g + 8 < count};
  const __nv_bfloat16* h_row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    h_row[i] = p.hidden + static_cast<size_t>(row0 + order[first + (row_ok[i] ? g + 8 * i : 0)]) * p.H;
  const __nv_bfloat16* a_row = p.a + (static_cast<size_t>(adapter) * p.rank + k0 + g) * p.H;
  float d[2][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // 32 columns of H a step: a lane's 8 consecutive ones serve two products
  // (the order of the summed index is free, the same on both sides).  The
  // loop's bound is the warp's, not the lane's: every lane takes part in a
  // product, with zeros past the end of H.
#pragma unroll 4
  for (int h0 = (split_rank * kShrinkWarps + warp) * 32; h0 < p.H; h0 += p.split * kShrinkWarps * 32) {
    const int h = h0 + 8 * t;
    const bool in = h < p.H;
    uint4 x[2], y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = in && row_ok[i] ? __ldg(reinterpret_cast<const uint4*>(h_row[i] + h)) : zero;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      y[i] = in && k0 + 8 * i + g < p.rank
                 ? __ldg(reinterpret_cast<const uint4*>(a_row + static_cast<size_t>(8 * i) * p.H + h))
                 : zero;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
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
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float& to = mine_part[(g + 8 * (q >> 1)) * kRanks + 8 * i + 2 * t + (q & 1)];
          to = round == 0 ? d[i][q] : to + d[i][q];
        }
    }
    __syncthreads();
  }
  cluster_wait();  // every CTA of the cluster runs
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
    if (rank >= p.rank) u = 0.0f;  // padding: an infinite hidden state or scale times its zeros is no number
    if (count <= few_rows_of(p.rank)) {  // kept as it is, [row][padded rank]
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
      const __nv_bfloat16 term = __float2bfloat16_rz(u);  // cut off: of a finite u never infinite
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

// Tile statistics of a row of a block, a quarter (32 ids) after another: the
// row's 4 lanes (same g) hold 8 logits of the quarter (v[b] = ids 16 b + 4 t ..),
// -inf past the slice's end.  Sums and minima stay a lane's own until the end.

// The largest of a lane's logits, the smallest finite one, the smallest nonzero
// |l| (infinite ones count as +inf).
template <int N>
__device__ __forceinline__ void lane_extremes(const float (&x)[N], float& top, float& mn, float& am) {
  top = x[0];
  mn = x[0];
  am = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) {
    top = fmaxf(top, x[i]);  // (NaN: dropped by all three)
    mn = fminf(mn, x[i]);
    am = fminf(am, fabsf(x[i]));
  }
  if (mn == -INFINITY || am == 0.0f || mn != mn) {  // rare: what does not count is among them
    top = -INFINITY;
    mn = INFINITY;
    am = INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top = fmaxf(top, x[i]);
      mn = fminf(mn, isfinite(x[i]) ? x[i] : INFINITY);
      am = fminf(am, x[i] != 0.0f ? fabsf(x[i]) : INFINITY);
    }
  }
}
struct BlockStats {
  float q[4], sum[4], mn, am;  // sum[i] relative to q[i] where that is finite
};
__device__ __forceinline__ void quarter_stats(BlockStats& s, int quarter, const float4 (&v)[2]) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
  float top, mn, am;
  lane_extremes(x, top, mn, am);
  if (quarter != 0) {
    mn = fminf(mn, s.mn);
    am = fminf(am, s.am);
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  const float c = isfinite(top) ? top : 0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int b = 0; b < 2; ++b)
    sum += ex2((v[b].x - c) * kLog2e) + ex2((v[b].y - c) * kLog2e) + ex2((v[b].z - c) * kLog2e) +
           ex2((v[b].w - c) * kLog2e);
  s.mn = mn;
  s.am = am;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // static registers
    if (i == quarter) {
      s.q[i] = top;
      s.sum[i] = sum;
    }
}
// By all lanes of the warp; the row's first one writes.
__device__ __forceinline__ void write_stats(const BlockStats& s, float* rec, bool write) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float top = fmaxf(fmaxf(s.q[0], s.q[1]), fmaxf(s.q[2], s.q[3]));
  const float c = isfinite(top) ? top : 0.0f;
  float sum = 0.0f, mn = s.mn, am = s.am;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // a quarter without a finite maximum has the sum 0, +inf or NaN whatever it is relative to
    sum += s.sum[i] * (isfinite(s.q[i]) ? ex2((s.q[i] - c) * kLog2e) : 1.0f);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
    am = fminf(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
  }
  if (write) {
    reinterpret_cast<float4*>(rec)[0] = make_float4(s.q[0], s.q[1], s.q[2], s.q[3]);
    reinterpret_cast<float4*>(rec)[1] = make_float4(sum, mn, am, 0.0f);
  }
}

__device__ __forceinline__ void load_b(uint4& v, const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }

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

// The rows of a unit of at most kFewRows over blocks of 128 ids: what counts is
// that B, which no other row shares, streams in.  LANES lanes hold an id's row
// of B, 8 ranks each: a quarter (32 ids) is LANES loads of 512 contiguous bytes.
// The lanes' sums are added and dealt out in one butterfly, after which every
// lane holds one id of the quarter: LANES' lane `sub` of the ids' group `at` id
// (32 / LANES) sub + at.
template <int LANES>
__device__ __forceinline__ void few_rows(const ExpandArgs& p, int adapter, const int32_t* rows, int count, const float* u_rows,
                                         int padded, int block0, int last_block, int lane) {
  constexpr int ROWS = kFewRows;
  constexpr int kPer = 32 / LANES;                      // ids of one load
  constexpr int kQuarters = LANES < 2 ? 4 : 8 / LANES;  // quarters in flight, LANES loads each
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
      uint4 y[kQuarters][LANES];
#pragma unroll
      for (int q = 0; q < kQuarters; ++q)
#pragma unroll
        for (int i = 0; i < LANES; ++i) {
          y[q][i] = make_uint4(0, 0, 0, 0);
          // ids past the slice's end read its last one's row instead (their sums are not kept)
          if (ranks_in) load_b(y[q][i], b + min(32 * (m0 + q) + kPer * i + at, most) * p.rank);
        }
#pragma unroll
      for (int q = 0; q < kQuarters; ++q)
#pragma unroll
        for (int i = 0; i < LANES; ++i) {
          part[0][q][i] = dot8(y[q][i], u[0], 0.0f);
#pragma unroll
          for (int c = 1; c < ROWS; ++c) part[c][q][i] = count > c ? dot8(y[q][i], u[c], 0.0f) : 0.0f;
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
        if (p.stats != nullptr) {
#pragma unroll
          for (int m = 0; m < 4; ++m)  // past the slice's end: -inf again, where an infinite product made it a NaN
            if (32 * m + mine > most) v[c][m] = -INFINITY;
          warp_stats(v[c], p.stats + (static_cast<size_t>(row[c]) * p.S * p.B + block) * 8, lane);
        }
      }
  }
}

// 16 or 8 bytes from src + FROM to shared memory at dst + TO, in the
// background.  16: past L1; 8: through it.
template <int BYTES, int TO, int FROM>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(TO), "n"(FROM) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0 + %2], [%1 + %3], 8;" ::"r"(dst), "l"(src), "n"(TO), "n"(FROM) : "memory");
}
// The same where `valid`, else zeros (nothing is read).
template <int BYTES, int TO, int FROM>
__device__ __forceinline__ void copy_async_or_zero(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16, %4;" ::"r"(dst), "l"(src), "n"(TO), "n"(FROM), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0 + %2], [%1 + %3], 8, %4;" ::"r"(dst), "l"(src), "n"(TO), "n"(FROM), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// What a warp has in flight: the 16 rows' logits and the B of a quarter (32
// ids), a lane's own parts of both, so that a lane waits for its own copies
// only.  B: 4 ranks of an id's row to a copy (one step), or 8.
template <int STEPS>
struct ExpandStage {
  static constexpr int kCopies = STEPS == 1 ? 4 : 4 * STEPS / 2;  // of B
  static constexpr int kBytes = STEPS == 1 ? 8 : 16;              // of one
  uint4 x[4][32];
  typename std::conditional<STEPS == 1, uint2, uint4>::type b[kCopies][32];
};
constexpr int kStages = 3;
template <int STEPS>
constexpr size_t expand_smem() {
  return kStages * sizeof(ExpandStage<STEPS>);
}
// CTAs that the registers let stand on an SM (512 rows of rank 32 with statistics:
// 184 us with 13, 195 with 16, 198 with 12, rank 64 no different with fewer).
constexpr int expand_ctas(int steps) { return steps == 4 ? 12 : steps == 2 ? 13 : 16; }

// A warp's unit: its plan entry, and where its u is.
struct WarpUnit {
  const int32_t* entry;
  const uint32_t* u;
  int adapter, count, block0, last_block;
  bool work;
};
__device__ __forceinline__ WarpUnit warp_unit(const ExpandArgs& p, int warp, int warps, int steps) {
  WarpUnit w{};
  const int item = static_cast<int>(blockIdx.x % p.slot_ctas) * warps + warp;
  w.block0 = static_cast<int>(blockIdx.x / p.slot_ctas) * p.warp_blocks;
  w.last_block = min(w.block0 + p.warp_blocks, p.S * p.B);
  const int tile = item / p.slots, slot = item - tile * p.slots;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tile >= p.tiles) return w;
  const int32_t* plan = p.plan + tile * plan_ints(p.slots);
  if (slot >= plan[0]) return w;
  w.entry = plan + 4 + slot * (kPlanUnit + 3);
  w.adapter = w.entry[0];
  w.count = w.entry[1];
  w.u = p.u + (static_cast<size_t>(tile) * p.slots + slot) * steps * kTerms * kFragment;
  // (in place, rows without an adapter: the base logits stay as they are)
  w.work = !(w.adapter < 0 && p.in_place && p.stats == nullptr);
  return w;
}

// A step's products of 32 ids: y, a lane's B of the four products; a, u's
// operands of the step; FIRST: the sums begin with it.  The large term's sums and
// the two small ones' apart.
template <bool FIRST>
__device__ __forceinline__ void step_products(float (&d)[2][4][4], const uint4 (&a)[kTerms], const uint2 (&y)[4]) {
#pragma unroll
  for (int e = 0; e < kTerms; ++e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float(&to)[4] = d[e == 0 ? 0 : 1][i];
      if (FIRST && e < 2)
        mma_16816_first(to, a[e].x, a[e].y, a[e].z, a[e].w, y[i].x, y[i].y);
      else
        mma_16816(to, a[e].x, a[e].y, a[e].z, a[e].w, y[i].x, y[i].y);
    }
}

// The sums of 32 ids onto the rows' logits, the large terms' first: where those
// cancel the logit the sum is exact, and the small terms are what is left.  An
// infinity in B times a small term of 0 makes the small terms' sum a NaN, which
// says nothing: the large ones' is what it should be, and a number is added.
// (Terms of a u have one sign, so an infinite sum of small ones agrees.)
__device__ __forceinline__ float small_sum(float d) { return fmaxf(d, -FLT_MAX); }
__device__ __forceinline__ void add_sums(float4 (&x)[2][2], const float (&d)[2][4][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      x[i][b].x = (x[i][b].x + d[0][2 * b][2 * i]) + small_sum(d[1][2 * b][2 * i]);
      x[i][b].y = (x[i][b].y + d[0][2 * b][2 * i + 1]) + small_sum(d[1][2 * b][2 * i + 1]);
      x[i][b].z = (x[i][b].z + d[0][2 * b + 1][2 * i]) + small_sum(d[1][2 * b + 1][2 * i]);
      x[i][b].w = (x[i][b].w + d[0][2 * b + 1][2 * i + 1]) + small_sum(d[1][2 * b + 1][2 * i + 1]);
    }
}

// Stores a quarter of the unit's rows, j its first id; a lane's logits past the
// slice's end become -inf (for the statistics).
__device__ __forceinline__ void store_quarter(float* dst, const size_t (&row_at)[2], const int (&r)[2], int j, int V_s,
                                              int t, float4 (&x)[2][2]) {
  dst += j + 4 * t;
  if (j + 32 <= V_s) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (r[i] >= 0) {
        *reinterpret_cast<float4*>(dst + row_at[i]) = x[i][0];
        *reinterpret_cast<float4*>(dst + row_at[i] + 16) = x[i][1];
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (j + 16 * b + 4 * t >= V_s)
        x[i][b] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      else if (r[i] >= 0)
        *reinterpret_cast<float4*>(dst + row_at[i] + 16 * b) = x[i][b];
    }
}

// A CTA is one warp: a unit whose rows are few, or a slot that is empty, holds no
// other warp's place (when it was chosen, of this kernel's form then: one row of
// rank 16 8.3 us, 10.4 with four warps a CTA; 64 requests 76 us, 78).
//
// The warp takes a unit's 16 rows and runs over blocks of 128 ids (of a slice), a
// quarter at a time, the next quarters' logits and B on their way meanwhile.
// The products' N index is laid over the ids so that a lane's sums are 4
// consecutive ids of a row: column n of the i-th product of 4 is id
// 16 (i / 2) + 4 (n / 2) + 2 (i mod 2) + n mod 2.
//
// Under the profiler, alone: 512 rows over 18 adapters of rank 32 with statistics
// 172 us, 0.78 GB of DRAM traffic (4.5 TB/s), the issue slots 57 % used; 2,048
// rows over 8 adapters of rank 64 565 us, 2.64 GB (4.7 TB/s), the tensor pipe 45 %
// active, 5.6 GB read out of the L2 cache (176 M sectors), where the B's of 155 MB
// are read once for each unit of 16 rows.  What is left is the overlap within a
// warp, which waits for copies, products and sums in turn, and that reading of B.
// Units of 32 rows, which read B half as often, need twice the registers: when
// they were tried 612 us where this took 591; more warps, more stages or B
// through L1 left the time as it was or cost up to 10 %.
template <int STEPS, int LANES>  // rank_steps, lanes of 8 ranks in few_rows (0: no unit comes there)
__global__ void __launch_bounds__(32, expand_ctas(STEPS))
    adapters_expand_kernel(const __grid_constant__ ExpandArgs p) {
  extern __shared__ uint4 expand_stages[];
  using Stage = ExpandStage<STEPS>;
  const int lane = threadIdx.x, g = lane >> 2, t = lane & 3;
  const WarpUnit w = warp_unit(p, 0, 1, STEPS);
  if (!w.work) return;
  if constexpr (LANES > 0) {
    if (w.adapter >= 0 && w.count <= kFewRows) {  // the whole warp's
      few_rows<LANES>(p, w.adapter, w.entry + 4, w.count, reinterpret_cast<const float*>(w.u), STEPS * 16, w.block0,
                      w.last_block, lane);
      return;
    }
  }
  Stage* stages = reinterpret_cast<Stage*>(expand_stages);
  const int r[2] = {w.entry[4 + g], w.entry[4 + g + 8]};
  const size_t row_at[2] = {static_cast<size_t>(max(r[0], 0)) * p.V_s, static_cast<size_t>(max(r[1], 0)) * p.V_s};
  uint4 u[STEPS * kTerms];
  if (w.adapter >= 0) {
#pragma unroll
    for (int i = 0; i < STEPS * kTerms; ++i) u[i] = reinterpret_cast<const uint4*>(w.u)[i * 32 + lane];
  }
  const int n_id = 4 * (g >> 1) + (g & 1);  // the id of this lane's column, within 16 ids, of an even product
  constexpr int kLaneRanks = Stage::kBytes / 2;
  const int slice0 = w.block0 / p.B;
  const bool even_ranks = p.rank == 16 * STEPS;
  // this lane's places in what quarter h of the warp's blocks copies: two rows'
  // logits, and the B of its ids, whose rows are 0, 2, 16 and 18 from the first
  int load_slice = slice0, load_j = 128 * (w.block0 - slice0 * p.B);
  const int two = 2 * p.rank;
  const float *x0, *x1;
  const __nv_bfloat16* b0;
  auto place = [&] {
    const float* src = p.logits[load_slice] + load_j + 4 * t;
    x0 = src + row_at[0];
    x1 = src + row_at[1];
    b0 = p.b[load_slice] +
         (static_cast<size_t>(w.adapter >= 0 ? w.adapter : 0) * p.V_s + load_j + n_id) * p.rank + kLaneRanks * t;
  };
  place();
  uint32_t to = smem_u32(stages) + 16 * lane;  // the stage that is copied to, this lane's 16 bytes
  const uint32_t to_end = to + kStages * sizeof(Stage);
  auto issue = [&](int h) {
    const uint32_t x_to = to, b_to = to + offsetof(Stage, b) - (16 - Stage::kBytes) * lane;
    to += sizeof(Stage);
    if (to == to_end) to -= kStages * sizeof(Stage);
    constexpr int kB = Stage::kBytes, kRow = 32 * kB;  // a copy over the warp's lanes
    if (load_j + 32 <= p.V_s) {
      if (r[0] >= 0) {
        copy_async<16, 0, 0>(x_to, x0);
        copy_async<16, 512, 64>(x_to, x0);
      }
      if (r[1] >= 0) {
        copy_async<16, 1024, 0>(x_to, x1);
        copy_async<16, 1536, 64>(x_to, x1);
      }
      if (w.adapter >= 0) {
        if (even_ranks) {
          constexpr int kId = 2 * 16 * STEPS;  // bytes of an id's row
          copy_async<kB, 0, 0>(b_to, b0);
          copy_async<kB, kRow, 2 * kId>(b_to, b0);
          copy_async<kB, 2 * kRow, 16 * kId>(b_to, b0);
          copy_async<kB, 3 * kRow, 18 * kId>(b_to, b0);
          if constexpr (STEPS == 4) {
            copy_async<kB, 4 * kRow, 64>(b_to, b0);
            copy_async<kB, 5 * kRow, 2 * kId + 64>(b_to, b0);
            copy_async<kB, 6 * kRow, 16 * kId + 64>(b_to, b0);
            copy_async<kB, 7 * kRow, 18 * kId + 64>(b_to, b0);
          }
        } else {
          const __nv_bfloat16* id[4] = {b0, b0 + two, b0 + 8 * two, b0 + 9 * two};
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // past the rank: zeros
            copy_async_or_zero<kB, 0, 0>(b_to + i * kRow, id[i], kLaneRanks * t < p.rank);
            if constexpr (STEPS == 4) copy_async_or_zero<kB, 4 * kRow, 64>(b_to + i * kRow, id[i], 32 + 8 * t < p.rank);
          }
        }
      }
    } else {  // the slice's end
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (load_j + 16 * q + 4 * t < p.V_s) {
          if (r[0] >= 0) copy_async<16, 0, 0>(x_to + q * 512, x0 + 16 * q);
          if (r[1] >= 0) copy_async<16, 0, 0>(x_to + (2 + q) * 512, x1 + 16 * q);
        }
      if (w.adapter >= 0) {
        // ids past it take its last one's row instead (their sums are not kept)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat16* id = b0 + min(16 * (i >> 1) + 2 * (i & 1), p.V_s - 1 - load_j - n_id) * p.rank;
          copy_async_or_zero<kB, 0, 0>(b_to + i * kRow, id, kLaneRanks * t < p.rank);
          if constexpr (STEPS == 4) copy_async_or_zero<kB, 4 * kRow, 64>(b_to + i * kRow, id, 32 + 8 * t < p.rank);
        }
      }
    }
    load_j += 32;
    x0 += 32;
    x1 += 32;
    b0 += 16 * two;
    if ((h & 3) == 3 && load_j >= p.V_s && ++load_slice < p.S) {  // (the last slice's end: no more is issued)
      load_j = 0;
      place();
    }
  };
  const int quarters = 4 * (w.last_block - w.block0);
  const Stage* at = stages;  // the stage that is read
#pragma unroll
  for (int h = 0; h < kStages - 1; ++h) {
    issue(h);  // (a warp has four quarters at least)
    copy_commit();
  }
  int slice = slice0, in_slice = w.block0 - slice0 * p.B;
  BlockStats stats[2];
#pragma unroll 1
  for (int h = 0; h < quarters; ++h) {
    if (h + kStages - 1 < quarters) issue(h + kStages - 1);
    copy_commit();  // a group a quarter, empty ones at the end
    copy_wait<kStages - 1>();
    const Stage& st = *at;
    if (++at == stages + kStages) at = stages;
    const int j = in_slice * 128 + 32 * (h & 3);
    float4 x[2][2];
    float d[2][4][4];
    if (w.adapter >= 0) {
      if constexpr (STEPS == 1) {
        uint2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = st.b[i][lane];
        const uint4 a[kTerms] = {u[0], u[1], u[2]};
        step_products<true>(d, a, y);
      } else {
#pragma unroll
        for (int k = 0; k < STEPS; k += 2) {
          uint2 y0[4], y1[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = st.b[2 * k + i][lane];
            y0[i] = make_uint2(v.x, v.y);
            y1[i] = make_uint2(v.z, v.w);
          }
          const uint4 a0[kTerms] = {u[k * kTerms], u[k * kTerms + 1], u[k * kTerms + 2]};
          const uint4 a1[kTerms] = {u[(k + 1) * kTerms], u[(k + 1) * kTerms + 1], u[(k + 1) * kTerms + 2]};
          if (k == 0)
            step_products<true>(d, a0, y0);
          else
            step_products<false>(d, a0, y0);
          step_products<false>(d, a1, y1);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint4 v = st.x[2 * i + b][lane];
        x[i][b] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
      }
    if (w.adapter >= 0) add_sums(x, d);
    store_quarter(p.out[slice], row_at, r, j, p.V_s, t, x);
    if (p.stats != nullptr) {
      quarter_stats(stats[0], h & 3, x[0]);
      quarter_stats(stats[1], h & 3, x[1]);
      if ((h & 3) == 3) {
        const int block = w.block0 + (h >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          write_stats(stats[i], p.stats + (static_cast<size_t>(max(r[i], 0)) * p.S * p.B + block) * 8,
                      r[i] >= 0 && t == 0);
      }
    }
    if ((h & 3) == 3 && ++in_slice == p.B) {
      in_slice = 0;
      ++slice;
    }
  }
}

// The same for ranks above 64: B and u are loaded as they are used, so that the
// time is the loads' latency over the warps that stand on an SM (512 rows over 8
// adapters: 356 us at rank 128, 599 at rank 256; 2.6 and 2.1 TB/s).  The small
// terms' sums stay apart here too; their 16 registers cost a tenth (called from
// Python 324 us became 354, 525 590), but one sum loses them where the large terms
// cancel the logit.
__global__ void __launch_bounds__(kWideWarps * 32, 16 / kWideWarps) adapters_expand_wide_kernel(const __grid_constant__ ExpandArgs p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int steps = rank_steps(p.rank);
  const WarpUnit w = warp_unit(p, warp, static_cast<int>(blockDim.x >> 5), steps);
  if (!w.work) return;
  const int r[2] = {w.entry[4 + g], w.entry[4 + g + 8]};
  const size_t row_at[2] = {static_cast<size_t>(max(r[0], 0)) * p.V_s, static_cast<size_t>(max(r[1], 0)) * p.V_s};
  const uint4* u = reinterpret_cast<const uint4*>(w.u) + lane;
  const int n_id = 4 * (g >> 1) + (g & 1);
  int slice = w.block0 / p.B, in_slice = w.block0 - slice * p.B;
  BlockStats stats[2];
#pragma unroll 1
  for (int h = 0; h < 4 * (w.last_block - w.block0); ++h) {
    const int j = in_slice * 128 + 32 * (h & 3);
    float4 x[2][2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (r[i] >= 0 && j + 16 * b + 4 * t < p.V_s)
          x[i][b] = *reinterpret_cast<const float4*>(p.logits[slice] + row_at[i] + j + 16 * b + 4 * t);
    if (w.adapter >= 0) {
      const __nv_bfloat16* id0 = p.b[slice] + (static_cast<size_t>(w.adapter) * p.V_s + j + n_id) * p.rank + 8 * t;
      const int most = p.V_s - 1 - j - n_id;  // ids past the slice's end take its last one's row instead
      float d[2][4][4] = {};
#pragma unroll 2
      for (int k = 0; k < steps; k += 2) {
        uint2 y0[4], y1[4];
        const bool ranks_in = 16 * k + 8 * t < p.rank;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (ranks_in) load_b(v, id0 + min(16 * (i >> 1) + 2 * (i & 1), most) * p.rank + 16 * k);
          y0[i] = make_uint2(v.x, v.y);
          y1[i] = make_uint2(v.z, v.w);
        }
        const uint4* a_at = u + k * kTerms * 32;
        const uint4 a0[kTerms] = {a_at[0], a_at[32], a_at[64]};
        const uint4 a1[kTerms] = {a_at[96], a_at[128], a_at[160]};
        step_products<false>(d, a0, y0);
        step_products<false>(d, a1, y1);
      }
      add_sums(x, d);
    }
    store_quarter(p.out[slice], row_at, r, j, p.V_s, t, x);
    if (p.stats != nullptr) {
      quarter_stats(stats[0], h & 3, x[0]);
      quarter_stats(stats[1], h & 3, x[1]);
      if ((h & 3) == 3) {
        const int block = w.block0 + (h >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          write_stats(stats[i], p.stats + (static_cast<size_t>(max(r[i], 0)) * p.S * p.B + block) * 8,
                      r[i] >= 0 && t == 0);
      }
    }
    if ((h & 3) == 3 && ++in_slice == p.B) {
      in_slice = 0;
      ++slice;
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

// The second kernel: may start before the one ahead of it ends, waits for its
// results itself.
cudaError_t launch_after(void (*kernel)(ExpandArgs), const ExpandArgs& a, unsigned grid, int warps, size_t smem,
                         cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The shared-memory attributes of the second kernel's variants, once per
// device, with it current.
cudaError_t prepare_expand() {
  constexpr int kMaxDevices = 64;
  static std::once_flag once[kMaxDevices];
  static cudaError_t status[kMaxDevices];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    constexpr int kCarveout = 72;  // percent: 164 KB
    const auto allow = [&](void (*kernel)(ExpandArgs), size_t smem) {
      if (status[dev] == cudaSuccess)
        status[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      // The rest is L1, which the multiply-adds' loads need (64 requests of rank
      // 32: 126 us, 144 with 196 KB; of rank 16 73 us, 87), and no case wants
      // more warps than fit (2,048 rows of rank 64: 631 us, 638 with 228 KB).
      if (status[dev] == cudaSuccess)
        status[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, kCarveout);
    };
    status[dev] = cudaSuccess;
    allow(adapters_expand_kernel<1, 1>, expand_smem<1>());
    allow(adapters_expand_kernel<1, 2>, expand_smem<1>());
    allow(adapters_expand_kernel<2, 4>, expand_smem<2>());
    allow(adapters_expand_kernel<4, 0>, expand_smem<4>());
  });
  return status[dev];
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
  // the CTAs of a cluster share longer rows of H while the units are few (one row
  // of rank 16 over H = 4,096: 7.5 us, 12.4 by one CTA; 512 rows over 18 adapters
  // of rank 32 with statistics: 184 us, 191)
  const int steps = rank_steps(rank);
  const long long ctas = static_cast<long long>(z.tiles) * z.slots * steps;
  sa.split = H < 4 * 256 || ctas > 296 ? 1 : ctas > 148 ? 2 : kMaxSplit;
  {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    cfg.gridDim = dim3(z.tiles, z.slots, steps * sa.split);
    cfg.blockDim = dim3(kShrinkWarps * 32);
    cfg.stream = stream;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = sa.split;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, adapters_shrink_kernel, sa);
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
  // Above rank 64 the warps of a CTA, next units, read the same B out of L1 where
  // adapters have units enough (512 rows over 8 adapters of rank 128: 356 us, 375
  // by single warps; 16 over 16: 160, 164; one row of rank 256: 46, 32).
  const int warps = rank > 64 && R > kUnitRows * static_cast<long long>(n) ? kWideWarps : 1;
  ea.slot_ctas = static_cast<int>((static_cast<long long>(z.tiles) * z.slots + warps - 1) / warps);
  // A warp keeps its unit's u over several blocks, while there are warps enough
  // to fill the SMs some times over (64 requests of rank 16: 73 us, 87 with a
  // block a warp; 2,048 rows over 8 adapters of rank 64: 631 us, 719).  Above
  // rank 64 it keeps no u (512 rows of rank 256: 599 us, 626 with four blocks).
  ea.warp_blocks = 1;
  while (rank <= 64 && ea.warp_blocks < 8 && static_cast<long long>(ea.slot_ctas) * S * ea.B / ea.warp_blocks > 8 * 148 * 16)
    ea.warp_blocks *= 2;
  const long long grid =
      static_cast<long long>(ea.slot_ctas) * ((static_cast<long long>(S) * ea.B + ea.warp_blocks - 1) / ea.warp_blocks);
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  const unsigned g = static_cast<unsigned>(grid);
  if (rank > 64) return launch_after(adapters_expand_wide_kernel, ea, g, warps, 0, stream);
  const cudaError_t e = prepare_expand();
  if (e != cudaSuccess) return e;
  if (rank > 32) return launch_after(adapters_expand_kernel<4, 0>, ea, g, 1, expand_smem<4>(), stream);
  if (rank > 16) return launch_after(adapters_expand_kernel<2, 4>, ea, g, 1, expand_smem<2>(), stream);
  if (rank > 8) return launch_after(adapters_expand_kernel<1, 2>, ea, g, 1, expand_smem<1>(), stream);
  return launch_after(adapters_expand_kernel<1, 1>, ea, g, 1, expand_smem<1>(), stream);
}

}  // namespace vsl
