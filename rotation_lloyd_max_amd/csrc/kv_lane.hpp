// How a cache row lies on the lanes of a wave, for the paged cache's write and read-back
// kernels: a row of D = 64, 128 or 256 elements on D / 8 neighbouring lanes, eight elements
// (a chunk) per lane.
//
// Lane L of a row holds chunk  c = L ^ 3 * ((L >> 2) & 1).  With that order the partner of a
// Sylvester stage on chunk bit 0, 1, 2, 3 is the lane L ^ 1, L ^ 2, L ^ 7, L ^ 8, and each of
// those moves is one DPP operand (quad permutations, half-row mirror, row rotation by 8), no
// LDS traffic; bits 4 and 5 are the row and half-wave swaps of gfx950 (v_permlane16_swap and
// v_permlane32_swap: with both operands x they give the lower rows' x in one result and the upper
// rows' in the other, for both partners). Lanes whose chunks share a group of 32,
// 64 or 128 elements are closed under {1, 2}, {1, 2, 7}, {1, 2, 7, 8}.
#pragma once

#include "device_common.hpp"

namespace tq {

__device__ __forceinline__ int kv_chunk(int L) { return L ^ (3 * ((L >> 2) & 1)); }

// x of the partner lane for chunk bit B < 4.
template <int B>
__device__ __forceinline__ int kv_swap(int x) {
  constexpr int ctrl = B == 0 ? 0xB1 : B == 1 ? 0x4E : B == 2 ? 0x141 : 0x128;
  return __builtin_amdgcn_update_dpp(0, x, ctrl, 0xf, 0xf, true);
}
template <int B>
__device__ __forceinline__ float kv_swap(float x) {
  return __int_as_float(kv_swap<B>(__float_as_int(x)));
}
template <int B>
__device__ __forceinline__ double kv_swap(double x) {
  return __hiloint2double(kv_swap<B>(__double2hiint(x)), kv_swap<B>(__double2loint(x)));
}
// x of the lower and of the upper partner for chunk bit B = 4, 5, in both of them.
template <int B>
__device__ __forceinline__ void kv_both(uint32_t x, uint32_t& lower, uint32_t& upper) {
  const auto r = B == 4 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                        : __builtin_amdgcn_permlane32_swap(x, x, false, false);
  lower = r[0];
  upper = r[1];
}
template <int B>
__device__ __forceinline__ void kv_both(float x, float& lower, float& upper) {
  uint32_t a, b;
  kv_both<B>(__float_as_uint(x), a, b);
  lower = __uint_as_float(a);
  upper = __uint_as_float(b);
}
template <int B>
__device__ __forceinline__ void kv_both(double x, double& lower, double& upper) {
  uint32_t a, b, c, d;
  kv_both<B>(static_cast<uint32_t>(__double2loint(x)), a, b);
  kv_both<B>(static_cast<uint32_t>(__double2hiint(x)), c, d);
  lower = __hiloint2double(static_cast<int>(c), static_cast<int>(a));
  upper = __hiloint2double(static_cast<int>(d), static_cast<int>(b));
}

__device__ __forceinline__ float kv_flip(float x, uint32_t m) {
  return __uint_as_float(__float_as_uint(x) ^ m);
}
__device__ __forceinline__ double kv_flip(double x, uint32_t m) {
  return __hiloint2double(__double2hiint(x) ^ static_cast<int>(m), __double2loint(x));
}

// One stage across lanes. B < 4: own + k partner with k = 1 in the lower chunk and -1 in the upper,
// which there is -(lower - upper): one fused operation (with the lane move as its DPP operand in
// fp32) instead of a sign change and an addition. Both partners of every later stage carry the
// same sign, so it stays a factor of the lane: kv_sign. B >= 4: the sum in the lower chunk, lower -
// upper in the upper.
template <int B, int N, typename T>
__device__ __forceinline__ void kv_stage(T (&v)[N], int c) {
  const T k = (c >> B) & 1 ? static_cast<T>(-1) : static_cast<T>(1);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if constexpr (B < 4) {
      v[j] = __builtin_fma(kv_swap<B>(v[j]), k, v[j]);
    } else {
      T lower, upper;
      kv_both<B>(v[j], lower, upper);
      v[j] = __builtin_fma(upper, k, lower);
    }
  }
}
template <int B, int N>
__device__ __forceinline__ void kv_stage(float (&v)[N], int c) {
  const float k = (c >> B) & 1 ? -1.f : 1.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if constexpr (B < 4) {
      v[j] = __builtin_fmaf(kv_swap<B>(v[j]), k, v[j]);
    } else {
      float lower, upper;
      kv_both<B>(v[j], lower, upper);
      v[j] = __builtin_fmaf(upper, k, lower);
    }
  }
}
// 1 where the transforms below leave the lane's values negated.
__device__ __forceinline__ uint32_t kv_sign(int c) { return __builtin_popcount(c & 15) & 1; }

// The maximum over the wave, in every lane.
__device__ __forceinline__ float kv_wave_max(float x) {
  x = fmaxf(x, kv_swap<0>(x));
  x = fmaxf(x, kv_swap<1>(x));
  x = fmaxf(x, kv_swap<2>(x));
  x = fmaxf(x, kv_swap<3>(x));
  float a, b;
  kv_both<4>(x, a, b);
  kv_both<5>(fmaxf(a, b), a, b);
  return fmaxf(a, b);
}

// The unnormalized Sylvester transform of a row of 64 N elements on a whole wave, lane L holding
// elements N kv_chunk(L) + j; negated where kv_sign says so.
template <int N>
__device__ __forceinline__ void kv_wave_transform(float (&v)[N], int c) {
#pragma unroll
  for (int s = 1; s < N; s <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j & s) continue;
      const float a = v[j], b = v[j | s];
      v[j] = a + b;
      v[j | s] = a - b;
    }
  kv_stage<0>(v, c);
  kv_stage<1>(v, c);
  kv_stage<2>(v, c);
  kv_stage<3>(v, c);
  kv_stage<4>(v, c);
  kv_stage<5>(v, c);
}

// The unnormalized Sylvester transform of a row on D / 8 lanes; negated where kv_sign says so.
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
