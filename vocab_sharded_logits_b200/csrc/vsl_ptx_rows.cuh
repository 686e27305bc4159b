// vsl_ptx_rows.cuh - inline-PTX wrappers of the row operators (adapters, token
// logprobs, losses) beside those of vsl_ptx.cuh: loads and stores with an L2
// policy, a store to distributed shared memory.
#pragma once

#include "vsl_ptx.cuh"

namespace vsl {

// 16-byte load that does not allocate in L1, with an L2 policy (not the
// read-only path: the kernel may write the same memory later).
__device__ __forceinline__ float4 ldg_hint4(const float* p, uint64_t policy) {
  float4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p), "l"(policy));
  return v;
}
__device__ __forceinline__ void stg_hint4(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.b32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void stg_hint2(void* p, uint32_t a, uint32_t b, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v2.b32 [%0], {%1, %2}, %3;" ::"l"(p), "r"(a), "r"(b), "l"(policy) : "memory");
}
__device__ __forceinline__ void st_dsmem_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

}  // namespace vsl
