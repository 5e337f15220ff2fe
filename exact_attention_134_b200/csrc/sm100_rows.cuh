// sm100_rows.cuh — instructions of the kernels that stream rows (norm with
// rotation, 4-bit cache) beside those of sm100_ptx.cuh.
#pragma once

#include "sm100_ptx.cuh"

namespace attn_sm100 {

// ---------------------------------------------------------------- plain asynchronous copies
// 16 bytes from global to shared memory, both 16-byte aligned; a lane waits for
// its own groups, the warp's copies need a __syncwarp() behind that.
__device__ __forceinline__ void cp_async16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the last N groups of the lane have landed.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- packed fp32
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return bits_f2(r);
}

// Halves of a word as fp32: bf16 values.
__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace attn_sm100
