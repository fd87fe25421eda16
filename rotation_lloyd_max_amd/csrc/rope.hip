// Rotary positions: pairs of elements of every head turned by the angle of the token's position,
//     (a, b) -> gain * (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i].
//
// The angle is formed in fp64 in turns and reduced there (position * inv_freq passes 2^24 turns
// of fp32 resolution long before the longest texts end), and so are its sine and cosine, times the
// gain, before they are rounded to fp32 (fp32 sines leave fp32 outputs half as much again off and are no
// faster: one token 8.7 us a call either way, 8192 tokens 29.0 us against 29.4). All
// heads of a token share them, so a workgroup makes the cosines and sines of its tokens once, in
// LDS, and its threads then stream the heads: the call is bound by reading x and writing out.
// 8192 tokens of 32 + 8 heads of 128 in bf16 (168 MB): 28.4 us, 5.9 TB/s, the rate of a copy
// whose data partly stays in the last cache; one token 2.9 us.
#include "device_common.hpp"
#include "internal.hpp"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 512;  // cosines and sines a workgroup holds
constexpr int64_t kRopeBlocks = 1 << 23;  // workgroups of a launch, at most: 2^32 threads wrap around

struct RopeParams {
  const char* x;
  char* out;
  const int32_t* positions;
  const double* inv_freq;
  int64_t tokens, xts, xhs, ots, ohs;  // strides in elements
  int heads, D, rot, tpb, hpb;         // tokens and heads of a workgroup
  double gain;
  bool transposed, copy;  // copy: elements from rot on are copied (not in place)
};

template <int DT, int V>
__device__ __forceinline__ void rope_get(const char* p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = load_elem<DT>(p, 0);
  } else if constexpr (DT == 0) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  } else {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (DT == 1) {
        f[2 * k] = __uint_as_float(a[k] << 16);
        f[2 * k + 1] = __uint_as_float(a[k] & 0xffff0000u);
      } else {
        f[2 * k] = half_bits_to_float(static_cast<uint16_t>(a[k] & 0xffffu));
        f[2 * k + 1] = half_bits_to_float(static_cast<uint16_t>(a[k] >> 16));
      }
    }
  }
}

template <int DT, int V>
__device__ __forceinline__ void rope_put(char* p, const float (&f)[V]) {
  if constexpr (V == 1) {
    store_any(p, DT, 0, f[0]);
  } else if constexpr (DT == 0) {
    *reinterpret_cast<u32x4_t*>(p) = u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]),
                                             __float_as_uint(f[2]), __float_as_uint(f[3])};
  } else {
    uint32_t a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = DT == 1 ? float_to_bf16_rne(f[2 * k]) : float_to_half_rne(f[2 * k]);
      const uint32_t hi = DT == 1 ? float_to_bf16_rne(f[2 * k + 1]) : float_to_half_rne(f[2 * k + 1]);
      a[k] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x4_t*>(p) = u32x4_t{a[0], a[1], a[2], a[3]};
  }
}

// VEC: 16-byte accesses. A head is cut into units: V pairs (two accesses) in the half layout, V
// elements (V / 2 pairs) interleaved, V copied elements behind rot; without VEC a unit is one
// pair or one copied element.
template <int DT, bool VEC, bool IL>
__global__ __launch_bounds__(kRopeThreads) void k_rope(RopeParams p) {
  constexpr int SZ = DT == 0 ? 4 : 2;
  constexpr int V = VEC ? 16 / SZ : 1;
  __shared__ float2 cs[kRopeAngles];
  const int half = p.rot >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tpb;
  const int nt = static_cast<int>(p.tokens - t0 < p.tpb ? p.tokens - t0 : p.tpb);
  const int h0 = blockIdx.y * p.hpb;
  const int nh = p.heads - h0 < p.hpb ? p.heads - h0 : p.hpb;
  for (int a = threadIdx.x; a < nt * half; a += kRopeThreads) {
    const int t = a / half, i = a - t * half;
    const double turns = static_cast<double>(p.positions[t0 + t]) * (p.inv_freq[i] * 0.15915494309189533577);
    double sn, cn;
    sincospi(2.0 * (turns - rint(turns)), &sn, &cn);
    cs[a] = make_float2(static_cast<float>(cn * p.gain), static_cast<float>((p.transposed ? -sn : sn) * p.gain));
  }
  __syncthreads();
  // units of a head: those that turn, then those that copy
  const int nr = IL ? (VEC ? p.rot / V : half) : half / V;
  const int nu = nr + (p.copy ? (p.D - p.rot) / V : 0);
  const int total = nt * nh * nu;
  for (int u = threadIdx.x; u < total; u += kRopeThreads) {
    const int row = u / nu, k = u - row * nu;
    const int t = row / nh, h = h0 + (row - t * nh);
    const char* xr = p.x + ((t0 + t) * p.xts + h * p.xhs) * SZ;
    char* orow = p.out + ((t0 + t) * p.ots + h * p.ohs) * SZ;
    if (k >= nr) {
      const int d = p.rot + (k - nr) * V;
      float f[V];
      rope_get<DT, V>(xr + d * SZ, f);
      rope_put<DT, V>(orow + d * SZ, f);
    } else if constexpr (IL && VEC) {
      float f[V], o[V];
      rope_get<DT, V>(xr + k * V * SZ, f);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 a = cs[t * half + (k * V + e) / 2];
        o[e] = f[e] * a.x - f[e + 1] * a.y;
        o[e + 1] = f[e + 1] * a.x + f[e] * a.y;
      }
      rope_put<DT, V>(orow + k * V * SZ, o);
    } else {
      const int d0 = IL ? 2 * k : k * V, d1 = IL ? 2 * k + 1 : k * V + half;
      float f[V], g[V], o[V], q[V];
      rope_get<DT, V>(xr + d0 * SZ, f);
      rope_get<DT, V>(xr + d1 * SZ, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 a = cs[t * half + k * V + e];
        o[e] = f[e] * a.x - g[e] * a.y;
        q[e] = g[e] * a.x + f[e] * a.y;
      }
      rope_put<DT, V>(orow + d0 * SZ, o);
      rope_put<DT, V>(orow + d1 * SZ, q);
    }
  }
}

template <int DT>
void rope_run(const RopeParams& p, bool vec, bool il, dim3 grid, hipStream_t s) {
  if (vec && il) hipLaunchKernelGGL((k_rope<DT, true, true>), grid, dim3(kRopeThreads), 0, s, p);
  else if (vec) hipLaunchKernelGGL((k_rope<DT, true, false>), grid, dim3(kRopeThreads), 0, s, p);
  else if (il) hipLaunchKernelGGL((k_rope<DT, false, true>), grid, dim3(kRopeThreads), 0, s, p);
  else hipLaunchKernelGGL((k_rope<DT, false, false>), grid, dim3(kRopeThreads), 0, s, p);
}

}  // namespace

hipError_t launch_rope(const void* x, int dt, int64_t tokens, int heads, int D, int64_t xts,
                       int64_t xhs, const RopeArgs& r, bool transposed, void* out, int64_t ots,
                       int64_t ohs, hipStream_t s) {
  RopeParams p{};
  p.inv_freq = r.inv_freq;
  p.xts = xts; p.xhs = xhs; p.ots = ots; p.ohs = ohs;
  p.heads = heads; p.D = D; p.rot = r.rot;
  p.gain = r.gain;
  p.transposed = transposed;
  p.copy = x != out;
  const int V = dt == 0 ? 4 : 8, half = r.rot / 2;
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                   xts % V == 0 && xhs % V == 0 && ots % V == 0 && ohs % V == 0 && D % V == 0 &&
                   (r.interleaved ? r.rot % V == 0 : half % V == 0);
  // a workgroup takes as many tokens as give its threads one angle each, fewer while that
  // leaves CUs without a workgroup; a few tokens are split by heads as well
  int tpb = half < 256 ? 256 / half : 1;
  while (tpb > 1 && (tokens + tpb - 1) / tpb < 1024) tpb >>= 1;
  p.tpb = tpb;
  int hpb = heads;
  const int64_t nb = (tokens + tpb - 1) / tpb;
  while (hpb > 4 && nb * ((heads + hpb - 1) / hpb) < 256) hpb = (hpb + 1) / 2;
  p.hpb = hpb;
  const int size = dt == 0 ? 4 : 2;
  for (int64_t b0 = 0; b0 < nb; b0 += kRopeBlocks) {
    const int64_t t0 = b0 * tpb, n = nb - b0 < kRopeBlocks ? nb - b0 : kRopeBlocks;
    p.x = static_cast<const char*>(x) + t0 * xts * size;
    p.out = static_cast<char*>(out) + t0 * ots * size;
    p.positions = r.positions + t0;
    p.tokens = tokens - t0 < n * tpb ? tokens - t0 : n * tpb;
    const dim3 grid(static_cast<uint32_t>(n), (heads + hpb - 1) / hpb);
    switch (dt) {
      case 0: rope_run<0>(p, vec, r.interleaved, grid, s); break;
      case 1: rope_run<1>(p, vec, r.interleaved, grid, s); break;
      default: rope_run<2>(p, vec, r.interleaved, grid, s); break;
    }
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tq
