// Attention over the paged compressed cache.
//     out = R_v^T sum_j p_j v'_j,  p = softmax_j(scale * (R_k q) . k'_j)
// with k', v' the decoded rows in the rotated bases (R orthonormal: q . k = (R q) . (R k)).
//
// One workgroup per (query row, query head): its waves take the tokens in turn, a lane holding
// D / 64 elements; each wave keeps a running maximum and sum, and the waves' partial sums are
// joined at the end.
#include "device_common.hpp"
#include "internal.hpp"

namespace tq {
namespace {

constexpr int kAtWaves = 4;

struct SimpleParams {
  AttendArgs a;
  float lut[2][256];
};

__device__ __forceinline__ uint32_t code_at(const uint32_t* w, int bits, int e) {
  const int bp = bits * e;
  uint32_t x = w[bp >> 5] >> (bp & 31);
  if ((bp & 31) + bits > 32) x |= w[(bp >> 5) + 1] << (32 - (bp & 31));
  return x & ((1u << bits) - 1u);
}

template <int D>
__device__ void row_transform(float* buf) {
  for (int h = 1; h < D; h <<= 1) {
    for (int i = threadIdx.x; i < D / 2; i += blockDim.x) {
      const int j = (i / h) * 2 * h + (i % h);
      const float a = buf[j], b = buf[j + h];
      buf[j] = a + b;
      buf[j + h] = a - b;
    }
    __syncthreads();
  }
}

template <int D>
__global__ __launch_bounds__(64 * kAtWaves) void k_attend_simple(SimpleParams p) {
  constexpr int EL = D / 64;
  const AttendArgs& a = p.a;
  __shared__ float lut[2][256];
  __shared__ float qs[D];
  __shared__ float po[kAtWaves][D];
  __shared__ float pm[kAtWaves], pl[kAtWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = blockIdx.x;
  const int qh = blockIdx.y, kh = qh / (a.q_heads / a.c.heads);
  for (int k = threadIdx.x; k < 256; k += blockDim.x) {
    lut[0][k] = p.lut[0][k];
    lut[1][k] = p.lut[1][k];
  }
  // the sequence of row m
  int b, start, n;
  if (a.q_offsets) {
    int lo = 0, hi = a.B;  // first b with q_offsets[b + 1] > m
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.q_offsets[mid + 1] > m) hi = mid;
      else lo = mid + 1;
    }
    if (lo >= a.B) return;
    b = lo;
    start = a.q_offsets[b];
    n = a.q_offsets[b + 1] - start;
  } else {
    n = static_cast<int>(a.M / a.B);
    b = static_cast<int>(m / n);
    start = b * n;
  }
  const int i = static_cast<int>(m) - start;
  const int64_t cap = static_cast<int64_t>(a.table_width) * a.c.page;
  int len = a.kv_lens[b];
  len = len < 0 ? 0 : static_cast<int>(len < cap ? len : cap);
  const int before = len - n;
  const int end = a.tree ? len : (before + i + 1 < len ? before + i + 1 : len);

  const float inv = 1.f / __builtin_sqrtf(static_cast<float>(D));
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    const float x = load_any(a.q, a.qdt, m * a.q_stride + qh * D + d);
    qs[d] = (a.c.k.signs[d >> 5] >> (d & 31)) & 1u ? -x : x;
  }
  __syncthreads();
  row_transform<D>(qs);
  float q[EL], o[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    q[e] = qs[lane * EL + e] * inv * a.scale;
    o[e] = 0.f;
  }
  float top = -__builtin_inff(), sum = 0.f;
  for (int j = wave; j < end; j += kAtWaves) {
    if (a.tree && j >= before) {
      const int x = j - before;
      if (x < 0 || x >= a.tree_words * 32 || !((a.tree[m * a.tree_words + (x >> 5)] >> (x & 31)) & 1u)) continue;
    }
    const int pg = a.page_table[static_cast<int64_t>(b) * a.table_width + j / a.c.page];
    const bool ok = pg >= 0 && pg < a.c.pages;
    const int64_t row = (static_cast<int64_t>(ok ? pg : 0) * a.c.heads + kh) * a.c.page + j % a.c.page;
    const uint32_t* kw = a.c.k.codes + row * a.c.k.wpr;
    const uint32_t* vw = a.c.v.codes + row * a.c.v.wpr;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      const int d = lane * EL + e;
      s += q[e] * lut[0][code_at(kw, a.c.k.bits, d)] *
           half_bits_to_float(a.c.k.scales[row * (D / a.c.k.group) + d / a.c.k.group]);
    }
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) s += __shfl_xor(s, x);
    if (!ok) s = __builtin_nanf("");
    const float nt = (s > top || s != s) ? s : top;
    const float f = __expf(top - nt), w = __expf(s - nt);
    top = nt;
    sum = sum * f + w;
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      const int d = lane * EL + e;
      o[e] = o[e] * f + w * lut[1][code_at(vw, a.c.v.bits, d)] *
                            half_bits_to_float(a.c.v.scales[row * (D / a.c.v.group) + d / a.c.v.group]);
    }
  }
  if (lane == 0) {
    pm[wave] = top;
    pl[wave] = sum;
  }
#pragma unroll
  for (int e = 0; e < EL; ++e) po[wave][lane * EL + e] = o[e];
  __syncthreads();
  float all = -__builtin_inff();
  for (int w = 0; w < kAtWaves; ++w) all = (pm[w] > all || pm[w] != pm[w]) ? pm[w] : all;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float x = 0.f, l = 0.f;
    for (int w = 0; w < kAtWaves; ++w) {
      if (pm[w] == -__builtin_inff()) continue;
      const float f = __expf(pm[w] - all);
      x += po[w][d] * f;
      l += pl[w] * f;
    }
    qs[d] = l == 0.f ? 0.f : x / l;
  }
  __syncthreads();
  row_transform<D>(qs);
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    const float x = qs[d] * inv;
    store_any(a.out, a.odt, (m * a.q_heads + qh) * D + d, (a.c.v.signs[d >> 5] >> (d & 31)) & 1u ? -x : x);
  }
}

}  // namespace

size_t kv_attend_workspace(const KvCacheArgs&, int, int, int64_t) { return 0; }

hipError_t launch_kv_attend(const AttendArgs& a, hipStream_t s) {
  SimpleParams p{};
  p.a = a;
  for (int i = 0; i < 2; ++i) {
    const int levels = i ? a.c.v.levels : a.c.k.levels;
    const float* cb = levels == 256 ? codebook256()->c : codebook_for(levels)->c;
    for (int k = 0; k < levels; ++k) p.lut[i][k] = cb[k];
  }
  const dim3 grid(static_cast<uint32_t>(a.M), a.q_heads), block(64 * kAtWaves);
  if (a.c.D == 64) hipLaunchKernelGGL((k_attend_simple<64>), grid, block, 0, s, p);
  else if (a.c.D == 128) hipLaunchKernelGGL((k_attend_simple<128>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((k_attend_simple<256>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace tq
