// Tokens read back from the paged cache by slot: out[t][h] = R^T (c[code] * scale), the rows of
// kv_fetch.hip in the order of a slot list ("your SSD is a GPU": dequantize, de-rotate on the
// way out). fp32, rounded once.
//
// A row lies on D / 8 lanes (kv_lane.hpp): a lane reads its eight codes (b bytes), does three
// transform stages in registers and the others with DPP moves, and writes 16 (or 32) bytes;
// a wave's rows are neighbouring heads of a token, so its store covers consecutive bytes.
#include "internal.hpp"
#include "kv_lane.hpp"

namespace tq {
namespace {

struct LoadHalf {
  const uint32_t* codes;
  const uint16_t* scales;
  const uint32_t* signs;
  void* out;
  int levels, bits, wpr, lg_group;
  float lut[256];
};

struct LoadParams {
  LoadHalf half[2];
  const int64_t* slots;
  int64_t tokens, capacity;
  int heads, page;
  float inv_sqrt_d;
};

template <int ODT, int D>
__global__ __launch_bounds__(256) void k_kv_load(LoadParams p) {
  constexpr int LR = D / 8, LGR = D == 64 ? 3 : D == 128 ? 4 : 5;
  __shared__ float lut[256];
  const LoadHalf& hf = p.half[blockIdx.y];
  for (int k = threadIdx.x; k < hf.levels; k += 256) lut[k] = hf.lut[k];
  const int c = kv_chunk(threadIdx.x & (LR - 1)), d0 = 8 * c;
  const uint32_t sg = (hf.signs[d0 >> 5] >> (d0 & 31)) & 0xffu;
  const int bits = hf.bits;
  const uint32_t mask = (1u << bits) - 1u;
  __syncthreads();
  const int64_t rows = p.tokens * p.heads;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * (256 >> LGR); r0 < rows;
       r0 += static_cast<int64_t>(gridDim.x) * (256 >> LGR)) {
    int64_t r = r0 + (threadIdx.x >> LGR);
    const bool live = r < rows;
    r = live ? r : rows - 1;
    const int64_t t = r / p.heads;
    const int h = static_cast<int>(r - t * p.heads);
    const int64_t slot = p.slots[t];
    const bool ok = slot >= 0 && slot < p.capacity;
    const int64_t page = (ok ? slot : 0) / p.page;
    const int64_t src = (page * p.heads + h) * p.page + ((ok ? slot : 0) - page * p.page);
    const uint32_t* w = hf.codes + src * hf.wpr;
    uint32_t lo, hi = 0;
    if (bits == 8) {
      const u32x2_t x = *reinterpret_cast<const u32x2_t*>(w + 2 * c);
      lo = x.x;
      hi = x.y;
    } else if (bits == 4) {
      lo = w[c];
    } else if (bits == 3) {  // 24 bits at byte 3 c: inside one word, or across two
      const int wi = (3 * c) >> 2, sh = 8 * ((3 * c) & 3);
      const uint32_t a = w[wi], b = w[wi + 1 < hf.wpr ? wi + 1 : wi];
      lo = static_cast<uint32_t>((static_cast<uint64_t>(b) << 32 | a) >> sh);
    } else {
      lo = w[c >> 1] >> (16 * (c & 1));
    }
    const float sc = ok ? half_bits_to_float(hf.scales[src * (D >> hf.lg_group) + (d0 >> hf.lg_group)]) * p.inv_sqrt_d
                        : __builtin_nanf("");
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = bits == 8 ? ((e < 4 ? lo : hi) >> (8 * (e & 3))) : (lo >> (bits * e));
      v[e] = lut[x & mask] * sc;
    }
    kv_transform<D>(v, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = kv_flip(v[e], ((sg >> e) & 1u) << 31);
    if (live) {
      u32x4_t* dst = reinterpret_cast<u32x4_t*>(static_cast<char*>(hf.out) + (r * D + d0) * (ODT == 0 ? 4 : 2));
      if constexpr (ODT == 0) {
        dst[0] = u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        dst[1] = u32x4_t{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
      } else {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = ODT == 1 ? float_to_bf16_rne(v[2 * k]) : float_to_half_rne(v[2 * k]);
          const uint32_t b = ODT == 1 ? float_to_bf16_rne(v[2 * k + 1]) : float_to_half_rne(v[2 * k + 1]);
          u[k] = a | (b << 16);
        }
        dst[0] = u32x4_t{u[0], u[1], u[2], u[3]};
      }
    }
  }
}

template <int ODT>
void load_run(const LoadParams& p, int D, dim3 grid, hipStream_t s) {
  if (D == 64) hipLaunchKernelGGL((k_kv_load<ODT, 64>), grid, dim3(256), 0, s, p);
  else if (D == 128) hipLaunchKernelGGL((k_kv_load<ODT, 128>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((k_kv_load<ODT, 256>), grid, dim3(256), 0, s, p);
}

}  // namespace

hipError_t launch_kv_load(const KvCacheArgs& c, const int64_t* slots, int64_t tokens, void* k_out,
                          void* v_out, int odt, hipStream_t s) {
  LoadParams p{};
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    void* out = i ? v_out : k_out;
    if (!out) continue;
    const KvHalf& h = i ? c.v : c.k;
    LoadHalf& o = p.half[n++];
    o.codes = h.codes; o.scales = h.scales; o.signs = h.signs; o.out = out;
    o.levels = h.levels; o.bits = h.bits; o.wpr = h.wpr;
    o.lg_group = __builtin_ctz(h.group);
    const float* cb = h.levels == 256 ? codebook256()->c : codebook_for(h.levels)->c;
    for (int k = 0; k < h.levels; ++k) o.lut[k] = cb[k];
  }
  p.slots = slots; p.tokens = tokens; p.capacity = c.pages * c.page;
  p.heads = c.heads; p.page = c.page;
  p.inv_sqrt_d = static_cast<float>(1.0 / __builtin_sqrt(static_cast<double>(c.D)));
  const int64_t per = 256 / (c.D / 8);
  const int64_t want = (tokens * c.heads + per - 1) / per;
  const dim3 grid(static_cast<uint32_t>(want < 2048 ? want : 2048), n);
  switch (odt) {
    case 0: load_run<0>(p, c.D, grid, s); break;
    case 1: load_run<1>(p, c.D, grid, s); break;
    default: load_run<2>(p, c.D, grid, s); break;
  }
  return hipGetLastError();
}

}  // namespace tq
