// What the kernels of the grouped-query layer share: powers of two, E4M3 codes, the
// token axis of a step, launches.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "dsa_internal.cuh"

namespace dsa {
namespace gqa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kExpMin = -64, kExpMax = 120;  // exponents of a scale

// 2^x, -126 <= x <= 127
__device__ __forceinline__ float pow2(int x) {
  return __uint_as_float((uint32_t)(127 + x) << 23);
}
// The exponent of a scale (a power of two; anything else is brought into the range).
__device__ __forceinline__ int exponent_of(float scale) {
  const int e = (int)((__float_as_uint(scale) >> 23) & 0xffu) - 127;
  return min(max(e, kExpMin), kExpMax);
}
// The least exponent e >= kExpMin with top <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ int exponent_for(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kExpMin);
}
// The values of two codes.
__device__ __forceinline__ float2 codes2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// The same as a pair of fp16 (exact).
__device__ __forceinline__ uint32_t codes2_f16(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The last sequence that begins at or before row t of the token axis cu [B + 1] (the one
// that owns it, if any does).
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  int b = 0;
  for (int hi = B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (cu[mid] <= t) b = mid; else hi = mid;
  }
  return b;
}

// The rows cu0 .. cu1 - 1 of a step of n_t, as far as the step has them.  (Clamped before anything
// is subtracted: faulty boundaries may lie 2^32 apart.)
struct StepRows {
  int first, n;  // n < 0: cu falls
};
__device__ __forceinline__ StepRows rows_between(int cu0, int cu1, int n_t) {
  const int c0 = min(max(cu0, 0), n_t);
  return {c0, min(max(cu1, 0), n_t) - c0};
}

// Positions that the block table has room for.
__host__ __device__ inline int table_cap(int max_pages, int page_size) {
  const long long n = (long long)max_pages * page_size;
  return n < 0x7fffff00ll ? (int)n : 0x7fffff00;  // (and a few tiles more are still below 2^31)
}

// Block j, forced into the selection of a token whose own block is `mine`.
__device__ __forceinline__ bool forced(const GqaScoreArgs& a, int mine, int j) {
  return j <= mine && (j < a.sink_blocks || (long long)j > (long long)mine - a.local_blocks);
}

struct Launch {  // a launch that may start while the kernel before it ends
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg;
  Launch(dim3 grid, int threads, size_t smem, cudaStream_t stream) : cfg{} {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  Launch(const Launch&) = delete;
  Launch& operator=(const Launch&) = delete;
};

}  // namespace gqa
}  // namespace dsa
