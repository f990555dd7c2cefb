// Pieces shared by the kernels of the paged 8-bit KV cache (kv8_*.cu).
//
// A block holds block_size consecutive keys of one sequence for every KV head; a key's
// 256 values are e4m3 numbers times one power of two per (block, KV head), K and V
// apart.  With power-of-two scales a product q * scale is exact in fp32, and moving a
// block to a larger scale only rounds values that become e4m3 subnormals.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace gqa {
namespace {

// The cache's kernels are launched as programmatic dependents, one after another: each lets
// the next be scheduled early, and waits for the last before it touches global memory.  (The
// merge alone reads inputs of the call before its wait, so the split kernel before it lets it
// start only after its own.)
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_last() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

constexpr int kMinScaleExp = -126;   // an all-zero run's scale: the smallest normal power of two

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// 2^-e for the same range; 2^-127 is a subnormal.
__device__ __forceinline__ float inv_pow2f(int e) {
  return e == 127 ? __uint_as_float(0x400000u) : pow2f(-e);
}

// Least e >= -126 with a <= 448 * 2^e, from the bits of a finite a >= 0.  448 is
// 1.75 * 2^8, so with a = m * 2^x (1 <= m < 2) e is x - 8 for m <= 1.75, else x - 7.
__device__ __forceinline__ int scale_exp(uint32_t a_bits) {
  const int x = int(a_bits >> 23) - 127;               // -127 for zero and subnormals
  const int e = x - 8 + ((a_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kMinScaleExp);
}

// Least e in [-126, 127] with 2^e >= s for a stored scale (e itself for 2^e); -126 for
// a scale that is no positive finite number.
__device__ __forceinline__ int stored_exp(float s) {
  const uint32_t b = __float_as_uint(s);
  if (!(s > 0.f) || b >= 0x7F800000u) return kMinScaleExp;
  return min(max(int(b >> 23) - 127 + ((b & 0x7FFFFFu) ? 1 : 0), kMinScaleExp), 127);
}

// Two values (|x| <= 448 when finite) rounded to e4m3, nearest even; NaN and infinities
// (e4m3 has none) become NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint32_t v = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
  if (isinf(lo)) v |= 0x007Fu;
  if (isinf(hi)) v |= 0x7F00u;
  return v;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Eight e4m3 values (little-endian bytes) to fp32.
__device__ __forceinline__ void from_e4m3x8(uint2 u, float (&f)[8]) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = from_e4m3x2(w[i]), b = from_e4m3x2(w[i] >> 16);
    f[4 * i] = a.x;
    f[4 * i + 1] = a.y;
    f[4 * i + 2] = b.x;
    f[4 * i + 3] = b.y;
  }
}

__device__ __forceinline__ uint2 to_e4m3x8(const float (&f)[8]) {
  return make_uint2(to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16),
                    to_e4m3x2(f[4], f[5]) | (to_e4m3x2(f[6], f[7]) << 16));
}

// The same for values that are all finite.
__device__ __forceinline__ uint2 finite_to_e4m3x8(const float (&f)[8]) {
  const auto two = [](float lo, float hi) -> uint32_t {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
  };
  return make_uint2(two(f[0], f[1]) | (two(f[2], f[3]) << 16),
                    two(f[4], f[5]) | (two(f[6], f[7]) << 16));
}

// Largest |x| of eight values as fp32 bits, NaN and infinities left out.
__device__ __forceinline__ uint32_t finite_amax_bits(const float (&f)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0x7FFFFFFFu;
    m = max(m, b < 0x7F800000u ? b : 0u);
  }
  return m;
}

}  // namespace

// Host check shared by the entry points: block sizes are 16, 32, 64 or 128 keys, and a
// slot (block * block_size + row) and a pool row ((block * Hkv + head) * block_size +
// row) both fit an int.
inline int check_kv8_pool(int num_blocks, int Hkv, int block_size) {
  if (num_blocks < 1 || Hkv < 1 ||
      (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128))
    return GQA_ERR_INVALID_ARG;
  if ((long long)num_blocks * Hkv * block_size >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

inline bool aligned_to(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace gqa
