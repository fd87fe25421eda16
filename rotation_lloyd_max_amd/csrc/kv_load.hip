// Tokens read back from the paged cache by slot: out[t][h] = R^T (c[code] * scale), the rows of
// kv_fetch.hip in the order of a slot list ("your SSD is a GPU": dequantize, de-rotate on the
// way out). fp32, rounded once.
//
// A row lies on D / 8 lanes (kv_lane.hpp): a lane reads its eight codes (b bytes), does three
// transform stages in registers and the others with DPP moves, and writes 16 (or 32) bytes;
// a wave's rows are neighbouring heads of a token, so its store covers consecutive bytes.
//
// Bound by vector instructions, 203 for the 64 chunks of a wave (their issue is full): 32768 tokens of 8
// heads of 128, 8-bit keys and 3-bit values, to bf16 (183 MB) 48 us, 3.8 TB/s of the 5.2 that a large copy
// reaches (62 us before the next row's codes were loaded a row ahead and divisions left the loop); 301
// tokens of 5 heads of 64 to fp32 4.0 us, latency.
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
  uint32_t page16, page_mul;  // page / 16 and ceil(2^32 / page16) (0 for 1)
  float inv_sqrt_d;
};

// Row of a slot: 64-bit division only for caches of 2^31 tokens and more (elsewhere the quotient of
// slot / 16 by page / 16 <= 2^12 from a 32-bit product, at most one too large).
__device__ __forceinline__ int64_t load_row(const LoadParams& p, int64_t slot, int h) {
  int64_t page;
  if (p.capacity <= 0x7fffffff) {
    const uint32_t u = static_cast<uint32_t>(slot) >> 4;
    uint32_t y = p.page_mul ? __umulhi(u, p.page_mul) : u;
    y -= static_cast<uint64_t>(y) * p.page16 > u ? 1u : 0u;
    page = y;
  } else {
    page = slot / p.page;
  }
  return (page * p.heads + h) * p.page + (slot - page * p.page);
}

// A lane's codes and scale; none: the slot is outside the cache.
struct LoadIn {
  uint32_t lo, hi;
  uint16_t scale;
  bool none;
};

// Each wave takes rows (token, head) in turn; the next row's codes and the slot of the one after
// are requested before this one is transformed.
template <int ODT, int D>
__global__ __launch_bounds__(256) void k_kv_load(LoadParams p) {
  constexpr int LR = D / 8, LGR = D == 64 ? 3 : D == 128 ? 4 : 5;
  __shared__ float lut[256];
  const LoadHalf& hf = p.half[blockIdx.y];
  if (threadIdx.x < hf.levels) lut[threadIdx.x] = hf.lut[threadIdx.x];
  const int c = kv_chunk(threadIdx.x & (LR - 1)), d0 = 8 * c;
  // the row's signs, and the transform's
  const uint32_t sg = ((hf.signs[d0 >> 5] >> (d0 & 31)) & 0xffu) ^ (kv_sign(c) ? 0xffu : 0u);
  uint32_t flip[4];  // of packed pairs of 16-bit outputs
#pragma unroll
  for (int k = 0; k < 4; ++k) flip[k] = ((sg >> (2 * k)) & 1u) << 15 | ((sg >> (2 * k + 1)) & 1u) << 31;
  const int bits = hf.bits, lgg = hf.lg_group;
  const uint32_t* const codes = hf.codes;
  const uint16_t* const scales = hf.scales;
  const uint32_t woff = bits == 8 ? 2 * c : bits == 4 ? c : bits == 3 ? (3 * c) >> 2 : c >> 1;
  const uint32_t wnext = bits == 8 ? 1 : bits == 3 && woff + 1 < static_cast<uint32_t>(hf.wpr) ? 1 : 0;
  const int shift = bits == 3 ? 8 * ((3 * c) & 3) : bits == 2 ? 16 * (c & 1) : 0;
  const uint32_t soff = d0 >> lgg;
  const int64_t rows = p.tokens * p.heads;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (256 >> LGR);
  int64_t r = static_cast<int64_t>(blockIdx.x) * (256 >> LGR) + (threadIdx.x >> LGR);
  // (token, head) of row r + stride from those of row r, without a division
  const int64_t dt = stride / p.heads;
  const int dh = static_cast<int>(stride - dt * p.heads);
  auto advance = [&](int64_t& t, int& h) {
    t += dt;
    h += dh;
    if (h >= p.heads) {
      h -= p.heads;
      ++t;
    }
  };
  int64_t t = r / p.heads;
  int h = static_cast<int>(r - t * p.heads);
  auto slot_of = [&](int64_t t) { return p.slots[t < p.tokens ? t : p.tokens - 1]; };
  auto get = [&](int64_t slot, int h) {
    LoadIn x;
    x.none = slot < 0 || slot >= p.capacity;
    const int64_t row = load_row(p, x.none ? 0 : slot, h);
    const uint32_t* w = codes + row * hf.wpr + woff;
    if (bits == 8) {
      const u32x2_t y = *reinterpret_cast<const u32x2_t*>(w);
      x.lo = y.x;
      x.hi = y.y;
    } else {
      x.lo = w[0];
      x.hi = w[wnext];
    }
    x.scale = scales[row * (D >> lgg) + soff];
    return x;
  };
  int64_t t1 = t;
  int h1 = h;
  advance(t1, h1);
  LoadIn nxt = get(slot_of(t), h);
  int64_t slot1 = slot_of(t1);
  __syncthreads();
  for (; r - (threadIdx.x >> LGR) < rows; r += stride) {
    const LoadIn in = nxt;
    nxt = get(slot1, h1);
    advance(t1, h1);
    slot1 = slot_of(t1);
    const float sc = in.none ? __builtin_nanf("") : half_bits_to_float(in.scale) * p.inv_sqrt_d;
    float v[8];
    // the codes' addresses in the table: four times the code
    if (bits == 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(lut) +
                                               __builtin_amdgcn_udot4(e < 4 ? in.lo : in.hi, 4u << (8 * (e & 3)), 0, false));
    } else {
      const uint32_t x = static_cast<uint32_t>((static_cast<uint64_t>(in.hi) << 32 | in.lo) >> shift);
      const uint32_t mask = ((1u << bits) - 1u) << 2;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t y = e == 0 ? x << 2 : x >> (bits * e - 2);
        v[e] = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(lut) + (y & mask));
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= sc;
    kv_transform<D>(v, c);
    if (r < rows) {
      u32x4_t* dst = reinterpret_cast<u32x4_t*>(static_cast<char*>(hf.out) + (r * D + d0) * (ODT == 0 ? 4 : 2));
      if constexpr (ODT == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = kv_flip(v[e], ((sg >> e) & 1u) << 31);
        dst[0] = u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        dst[1] = u32x4_t{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
      } else {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a = ODT == 1 ? float_to_bf16_rne(v[2 * k]) : float_to_half_rne(v[2 * k]);
          const uint32_t b = ODT == 1 ? float_to_bf16_rne(v[2 * k + 1]) : float_to_half_rne(v[2 * k + 1]);
          u[k] = (a | (b << 16)) ^ flip[k];  // the rounding to nearest is the same for both signs
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
  p.page16 = c.page / 16;
  p.page_mul = p.page16 == 1 ? 0 : static_cast<uint32_t>((0x100000000ull + p.page16 - 1) / p.page16);
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
