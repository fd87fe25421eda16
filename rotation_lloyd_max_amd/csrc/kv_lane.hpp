// How a cache row lies on the lanes of a wave, for the paged cache's write and read-back
// kernels: a row of D = 64, 128 or 256 elements on D / 8 neighbouring lanes, eight elements
// (a chunk) per lane.
//
// Lane L of a row holds chunk  c = L ^ 3 * ((L >> 2) & 1).  With that order the partner of a
// Sylvester stage on chunk bit 0, 1, 2, 3 is the lane L ^ 1, L ^ 2, L ^ 7, L ^ 8, and each of
// those moves is one DPP operand (quad permutations, half-row mirror, row rotation by 8), no
// LDS traffic; only bit 4 (D = 256) goes through a swizzle. Lanes whose chunks share a group of 32,
// 64 or 128 elements are closed under {1, 2}, {1, 2, 7}, {1, 2, 7, 8}.
#pragma once

#include "device_common.hpp"

namespace tq {

__device__ __forceinline__ int kv_chunk(int L) { return L ^ (3 * ((L >> 2) & 1)); }

// x of the partner lane for chunk bit B.
template <int B>
__device__ __forceinline__ int kv_swap(int x) {
  if constexpr (B == 4) {
    return __builtin_amdgcn_ds_swizzle(x, 0x401f);  // lane ^ 16
  } else {
    constexpr int ctrl = B == 0 ? 0xB1 : B == 1 ? 0x4E : B == 2 ? 0x141 : 0x128;
    return __builtin_amdgcn_update_dpp(0, x, ctrl, 0xf, 0xf, true);
  }
}
template <int B>
__device__ __forceinline__ float kv_swap(float x) {
  return __int_as_float(kv_swap<B>(__float_as_int(x)));
}
template <int B>
__device__ __forceinline__ double kv_swap(double x) {
  return __hiloint2double(kv_swap<B>(__double2hiint(x)), kv_swap<B>(__double2loint(x)));
}

__device__ __forceinline__ float kv_flip(float x, uint32_t m) {
  return __uint_as_float(__float_as_uint(x) ^ m);
}
__device__ __forceinline__ double kv_flip(double x, uint32_t m) {
  return __hiloint2double(__double2hiint(x) ^ static_cast<int>(m), __double2loint(x));
}

// One stage across lanes: the lower chunk keeps the sum, the upper partner - own.
template <int B, typename T>
__device__ __forceinline__ void kv_stage(T (&v)[8], int c) {
  const uint32_t m = (c >> B) & 1 ? 0x80000000u : 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const T o = kv_swap<B>(v[j]);
    v[j] = o + kv_flip(v[j], m);
  }
}

// The unnormalized Sylvester transform of the row.
template <int D, typename T>
__device__ __forceinline__ void kv_transform(T (&v)[8], int c) {
#pragma unroll
  for (int s = 1; s < 8; s <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j & s) continue;
      const T a = v[j], b = v[j | s];
      v[j] = a + b;
      v[j | s] = a - b;
    }
  kv_stage<0>(v, c);
  kv_stage<1>(v, c);
  kv_stage<2>(v, c);
  if constexpr (D >= 128) kv_stage<3>(v, c);
  if constexpr (D >= 256) kv_stage<4>(v, c);
}

}  // namespace tq
