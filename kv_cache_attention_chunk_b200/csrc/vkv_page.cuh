// Shared by the paged-cache kernels: element types, row lengths, host checks.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "vkv_internal.h"
#include "vkv_ptx.cuh"

namespace vkv {

// The tokens of a row as the kernels count them: kv_len, or -2 (after raising
// VKV_DEVERR_BAD_OFFSETS) for a length that the table cannot hold.
__device__ __forceinline__ int page_row_len(int len, int W, int page, int* err) {
  if (len >= -1 && (long long)len <= (long long)W * page) return len;
  if (err) atomicCAS(err, 0, VKV_DEVERR_BAD_OFFSETS);
  return -2;
}

// Eight 16-bit values (T = __nv_bfloat16 or __half) of a 16-byte load as fp32.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4 v, float* f);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void unpack8<__half>(const uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
    f[2 * e] = p.x;
    f[2 * e + 1] = p.y;
  }
}

// Two e4m3 values (low byte first) as f16x2; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}

// Two fp32 -> two e4m3 bytes (lo in the low byte): round to nearest even,
// magnitudes above 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// n / d for 0 <= n < 2^31 by a multiplication: (umulhi(n, mul) + n) >> shift, with
// 2^shift >= d the next power of two and mul = floor(2^32 (2^shift - d) / d) + 1
// (Granlund and Montgomery, Division by Invariant Integers using Multiplication, 1994).
struct FastDiv {
  uint32_t mul, shift;
  __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
};
inline FastDiv fast_div(int d) {
  FastDiv f;
  f.shift = 0;
  while ((1ll << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((1ull << f.shift) - (uint32_t)d) << 32) / (uint32_t)d + 1);
  return f;
}

// Launches a kernel that calls griddep_wait() before it touches memory: its blocks may take
// their places while the stream's last kernel ends (programmatic dependent launch).
// All its loads are ordinary ones, never the read-only path's: that is for memory which nobody
// writes while the kernel is there, and here the last kernel may still be writing lengths, table,
// selection or queries; the compiler may also move such a load ahead of the wait.  The
// kernels let the next one in with griddep_launch_dependents() once their loads are done, not
// when they begin: waiting blocks hold shared memory, several launches pile up, and what comes
// next is crowded onto few SMs (one row of 1560 tokens 12 us if let in at the start, 10.7 at the
// end; 59 rows' selection and attention of 12 pages of 16 tokens 51 and 38 us).
template <typename P>
cudaError_t launch_ahead(void (*fn)(const P), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t rc = cudaLaunchKernelEx(&cfg, fn, p);
  if (rc != cudaSuccess) cudaGetLastError();
  return rc;
}

// Bytes of one element.
inline int dtype_bytes(int dt) { return dt == VKV_E4M3 ? 1 : 2; }

// The 16-byte rule for a tensor of `dt`: pointer and the strides that are read.
inline bool page_tensor_aligned(const vkv_tensor& t, int dt) {
  const int64_t m = 16 / dtype_bytes(dt);
  return (reinterpret_cast<uintptr_t>(t.ptr) & 15u) == 0 && t.sb % m == 0 && t.st % m == 0 && t.sh % m == 0;
}

}  // namespace vkv
