// New tokens into the paged cache: each head's key and value rotated, quantized and packed into
// the row of its token's slot ("How it works", "The KV cache": the weights' rotation and
// codebook; "your SSD is a GPU": rotate, quantize, store).
//
// Mathematics of tq_encode: v = H (s * x) in fp64 (x after its rotary turn, also fp64, so that a
// value near a threshold falls where exact arithmetic puts it), r = sqrt(mean_g v^2),
// scale = fp16(r / sqrt(D)), u = v / r (0 when r = 0), code = #{k : u > t_k} in binary32.
//
// A row lies on D / 8 lanes (kv_lane.hpp), so one decoded token already spreads over several
// waves. The code comes from a bucket table instead of a search: |u| * 64 is exact, each bucket
// of width 1/64 holds at most one positive threshold (neighbours are more than 1/64 apart even
// at 256 levels), so one LDS read gives the count below the bucket and the threshold to compare.
//
// Bound by vector instructions (fp64 transform of five to eight stages; 2900 wave instructions per
// 4 x 256 elements of a key or value): 3001 tokens of 4 heads of 256 in fp16, 4 bits, turned (31 MB):
// 21.5 us, 1.4 TB/s; 16 tokens of 8 heads of 128: 6.0 us, latency. 1024 workgroups a half instead of
// 2048 23 us; next token's rows loaded ahead spilled and took 59 us.
#include "kv_lane.hpp"

#include <mutex>

#include "encode_lane.hpp"
#include "internal.hpp"

namespace tq {
namespace {

constexpr int kStoreBuckets = 320;  // buckets of 1/64 up to 5.0; the last one is open

// One half's decision data: positive thresholds (binary32 bits, the last one a sentinel no key
// exceeds) and the buckets that hold one, as bits, with the number of bits before each word: the
// thresholds below bucket b are as many as the bits below b.
struct SnapTable {
  uint32_t thr[128];
  uint32_t held[kStoreBuckets / 32], before[kStoreBuckets / 32];
};

struct StoreHalf {
  const char* x;
  int64_t ts, hs;  // strides in elements
  uint32_t* codes;
  uint16_t* scales;
  const uint32_t* signs;
  int levels, bits, wpr, lg_group;
  SnapTable snap;
};

struct StoreParams {
  StoreHalf half[2];
  const int64_t* slots;
  const int32_t* positions;
  const double* inv_freq;  // null: no rotary positions
  const uint8_t* axis;     // null: one axis (RopeArgs)
  int64_t axis_stride;
  int64_t tokens, capacity;
  int heads, page, rot, axes;
  bool interleaved;
  double gain, inv_sqrt_d;
};

template <int DT, bool VEC>
__device__ __forceinline__ void store_load(const char* row, int d0, double (&v)[8]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<double>(load_elem<DT>(row, d0 + e));
  } else if constexpr (DT == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(row + (d0 + 4 * k) * 4);
      v[4 * k] = __uint_as_float(w.x); v[4 * k + 1] = __uint_as_float(w.y);
      v[4 * k + 2] = __uint_as_float(w.z); v[4 * k + 3] = __uint_as_float(w.w);
    }
  } else {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(row + d0 * 2);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint16_t lo = static_cast<uint16_t>(a[k] & 0xffffu), hi = static_cast<uint16_t>(a[k] >> 16);
      v[2 * k] = DT == 1 ? bf16_bits_to_float(lo) : half_bits_to_float(lo);
      v[2 * k + 1] = DT == 1 ? bf16_bits_to_float(hi) : half_bits_to_float(hi);
    }
  }
}

// The rotary turn of the lane's eight elements d0 .. d0 + 7 of a key row; cs holds
// gain * (cos, sin) of the token's angles.
template <int DT, bool VEC>
__device__ __forceinline__ void store_turn(const char* row, int d0, int rot, bool interleaved,
                                           const double2* cs, double (&v)[8]) {
  if (d0 >= rot) return;
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      if (d0 + e >= rot) break;
      const double2 a = cs[(d0 + e) >> 1];
      const double x = v[e], y = v[e + 1];
      v[e] = x * a.x - y * a.y;
      v[e + 1] = y * a.x + x * a.y;
    }
    return;
  }
  const int half = rot >> 1;
  double o[8];
  if (VEC && half % 8 == 0) {
    store_load<DT, VEC>(row, d0 < half ? d0 + half : d0 - half, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      o[e] = d < rot ? static_cast<double>(load_elem<DT>(row, d < half ? d + half : d - half)) : 0.0;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = d0 + e;
    if (d >= rot) break;
    const bool first = d < half;
    const double2 a = cs[first ? d : d - half];
    v[e] = v[e] * a.x + o[e] * (first ? -a.y : a.y);
  }
}

// grid (workgroups over tokens, half): heads * D / 8 threads of a workgroup take a token's
// rows, the workgroup going from token to token. AX: positions of several axes (a branch at run time cost
// calls without them 1.5 %).
template <int DT, int D, bool VEC, bool AX>
__global__ __launch_bounds__(256) void k_kv_store(StoreParams p) {
  constexpr int LR = D / 8, LGR = D == 64 ? 3 : D == 128 ? 4 : 5;
  __shared__ u32x2_t tab[kStoreBuckets];
  __shared__ double2 cs[2][D / 2];
  const int part = blockIdx.y;
  const StoreHalf& hf = p.half[part];
  const int c = kv_chunk(threadIdx.x & (LR - 1)), d0 = 8 * c;
  const uint32_t sg = (hf.signs[d0 >> 5] >> (d0 & 31)) & 0xffu;
  const int rows_per_pass = blockDim.x >> LGR;
  const int lg_gl = hf.lg_group - 3;  // log2 of the lanes of a group
  const int bits = hf.bits;
  const int cpos = hf.levels / 2;
  const bool turn = part == 0 && p.inv_freq;
  int flip = 0;
  static_assert(kStoreBuckets % 64 == 0, "whole waves");
  for (int b = threadIdx.x; b < kStoreBuckets; b += blockDim.x) {
    const int w = __builtin_amdgcn_readfirstlane(b >> 5);  // a wave's buckets: two words
    const uint32_t held = b & 32 ? hf.snap.held[w + 1] : hf.snap.held[w];
    const uint32_t before = b & 32 ? hf.snap.before[w + 1] : hf.snap.before[w];
    const uint32_t base = before + __builtin_popcount(held & ((1u << (b & 31)) - 1u));
    tab[b] = u32x2_t{hf.snap.thr[base], base};
  }
  __syncthreads();
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const int64_t slot = p.slots[t];
    if (slot < 0 || slot >= p.capacity) continue;
    const int64_t page = slot / p.page;
    const int tok = static_cast<int>(slot - page * p.page);
    if (turn) {
      // two buffers: the next token's angles may be written while this one's are read
      double pos = 0.0;
      if constexpr (!AX) pos = static_cast<double>(p.positions[t]);
      for (int i = threadIdx.x; i < (p.rot >> 1); i += blockDim.x) {
        if constexpr (AX) {
          const int ax = p.axis[i];
          pos = static_cast<double>(ax < p.axes ? p.positions[ax * p.axis_stride + t] : 0);
        }
        const double turns = pos * (p.inv_freq[i] * 0.15915494309189533577);
        double s, co;
        sincospi(2.0 * (turns - rint(turns)), &s, &co);
        cs[flip][i] = make_double2(co * p.gain, s * p.gain);
      }
      __syncthreads();
    }
    for (int h0 = 0; h0 < p.heads; h0 += rows_per_pass) {
      const int hh = h0 + (threadIdx.x >> LGR);
      const bool live = hh < p.heads;
      const int h = live ? hh : p.heads - 1;  // idle lanes repeat a row (lane moves need them)
      const char* row = hf.x + (t * hf.ts + h * hf.hs) * (DT == 0 ? 4 : 2);
      double v[8];
      store_load<DT, VEC>(row, d0, v);
      if (turn) {
        int dt = d0;  // the angles are read again for each row: held over the rows they took 100 registers
        asm volatile("" : "+v"(dt));
        store_turn<DT, VEC>(row, dt, p.rot, p.interleaved, cs[flip], v);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = kv_flip(v[e], ((sg >> e) & 1u) << 31);
      kv_transform<D>(v, c);
      double sq = 0.0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = __builtin_fma(v[e], v[e], sq);
      sq += kv_swap<0>(sq);
      sq += kv_swap<1>(sq);
      if (lg_gl >= 3) sq += kv_swap<2>(sq);
      if (lg_gl >= 4) sq += kv_swap<3>(sq);
      const double rr = __builtin_sqrt(sq / (8 << lg_gl));
      const double rinv = kv_flip(rr > 0.0 ? 1.0 / rr : 0.0, kv_sign(c) << 31);
      uint32_t code[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t ub = __float_as_uint(static_cast<float>(v[e] * rinv));
        const bool pos = static_cast<int32_t>(ub) > 0;
        const uint32_t mag = ub & 0x7fffffffu;
        // NaN takes the last bucket (fminf drops it), where the count is the largest
        const int b = static_cast<int>(fminf(__uint_as_float(mag) * 64.f, kStoreBuckets - 1.f));
        const u32x2_t tb = tab[b];
        const uint32_t cnt = tb.y + (mag + (pos ? 0u : 1u) > tb.x ? 1u : 0u);
        code[e] = pos ? cpos + cnt : cpos - 1 - cnt;
      }
      const int64_t r = (page * p.heads + h) * p.page + tok;
      if (live && (c & ((1 << lg_gl) - 1)) == 0)
        hf.scales[r * (D >> hf.lg_group) + (c >> lg_gl)] = double_to_half_rne_sat(rr * p.inv_sqrt_d);
      uint32_t* dst = hf.codes + r * hf.wpr;
      if (bits == 8) {
        const u32x2_t w{code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24,
                        code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24};
        if (live) *reinterpret_cast<u32x2_t*>(dst + 2 * c) = w;
      } else {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= code[e] << (bits * e);
        // the next chunk's word: one lane up in the quad, or down where the order is reversed
        const int up = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), 0xF9, 0xf, 0xf, true);  // [1,2,3,3]
        const int dn = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), 0x90, 0xf, 0xf, true);  // [0,0,1,2]
        const uint32_t nx = static_cast<uint32_t>((threadIdx.x & 4) ? dn : up);
        if (bits == 4) {
          if (live) dst[c] = w;
        } else if (bits == 3) {  // four chunks of 24 bits make three words
          const int j = c & 3;
          if (live && j < 3) dst[3 * (c >> 2) + j] = (w >> (8 * j)) | (nx << (24 - 8 * j));
        } else {  // two chunks of 16 bits make a word
          if (live && (c & 1) == 0) dst[c >> 1] = w | (nx << 16);
        }
      }
    }
    flip ^= 1;
  }
}

template <int DT, int D, bool AX>
void store_run_ax(const StoreParams& p, bool vec, dim3 grid, int threads, hipStream_t s) {
  if (vec) hipLaunchKernelGGL((k_kv_store<DT, D, true, AX>), grid, dim3(threads), 0, s, p);
  else hipLaunchKernelGGL((k_kv_store<DT, D, false, AX>), grid, dim3(threads), 0, s, p);
}
template <int DT, int D>
void store_run(const StoreParams& p, bool vec, dim3 grid, int threads, hipStream_t s) {
  if (p.axis) store_run_ax<DT, D, true>(p, vec, grid, threads, s);
  else store_run_ax<DT, D, false>(p, vec, grid, threads, s);
}
template <int DT>
void store_run_d(const StoreParams& p, int D, bool vec, dim3 grid, int threads, hipStream_t s) {
  if (D == 64) store_run<DT, 64>(p, vec, grid, threads, s);
  else if (D == 128) store_run<DT, 128>(p, vec, grid, threads, s);
  else store_run<DT, 256>(p, vec, grid, threads, s);
}

SnapTable g_snap[4];
bool g_snap_ok = false;
std::once_flag g_snap_once;

void init_snap() {
  bool ok = true;
  const int levels[4] = {4, 8, 16, 256};
  for (int i = 0; i < 4; ++i) {
    SnapTable& t = g_snap[i];
    const int n = levels[i] / 2 - 1;
    uint32_t bits[128];
    ok = ok && positive_threshold_bits(levels[i], bits);
    for (int k = 0; k < 128; ++k) t.thr[k] = k < n ? bits[k] : 0xffffffffu;
    for (int b = 0; b < kStoreBuckets; ++b) {
      int in = 0;
      for (int k = 0; k < n; ++k) {
        const float x = __builtin_bit_cast(float, bits[k]) * 64.f;
        in += x >= b && (b + 1 == kStoreBuckets || x < b + 1) ? 1 : 0;
      }
      ok = ok && in <= 1 && !(in && b + 1 == kStoreBuckets);
      if (in) t.held[b >> 5] |= 1u << (b & 31);
    }
    for (int w = 1; w < kStoreBuckets / 32; ++w) t.before[w] = t.before[w - 1] + __builtin_popcount(t.held[w - 1]);
  }
  g_snap_ok = ok;
}

}  // namespace

hipError_t launch_kv_store(const KvCacheArgs& c, const void* k, const void* v, int dt,
                           int64_t tokens, const int64_t (&strides)[4], const int64_t* slots,
                           const RopeArgs& r, hipStream_t s) {
  std::call_once(g_snap_once, init_snap);
  if (!g_snap_ok) return hipErrorInvalidValue;
  StoreParams p{};
  bool vec = true;
  for (int i = 0; i < 2; ++i) {
    const KvHalf& h = i ? c.v : c.k;
    StoreHalf& o = p.half[i];
    o.x = static_cast<const char*>(i ? v : k);
    o.ts = strides[2 * i];
    o.hs = strides[2 * i + 1];
    o.codes = h.codes; o.scales = h.scales; o.signs = h.signs;
    o.levels = h.levels; o.bits = h.bits; o.wpr = h.wpr;
    o.lg_group = __builtin_ctz(h.group);
    o.snap = g_snap[h.bits == 8 ? 3 : h.bits - 2];
    const int V = dt == 0 ? 4 : 8;
    vec = vec && reinterpret_cast<uintptr_t>(o.x) % 16 == 0 && o.ts % V == 0 && o.hs % V == 0;
  }
  p.slots = slots; p.tokens = tokens; p.capacity = c.pages * c.page;
  p.heads = c.heads; p.page = c.page;
  p.positions = r.positions; p.inv_freq = r.inv_freq; p.rot = r.rot;
  p.interleaved = r.interleaved; p.gain = r.gain;
  p.axis = r.axis; p.axis_stride = r.axis_stride; p.axes = r.axes;
  p.inv_sqrt_d = 1.0 / __builtin_sqrt(static_cast<double>(c.D));
  int threads = (c.heads * (c.D / 8) + 63) & ~63;
  if (threads > 256) threads = 256;
  const dim3 grid(static_cast<uint32_t>(tokens < 2048 ? tokens : 2048), 2);
  switch (dt) {
    case 0: store_run_d<0>(p, c.D, vec, grid, threads, s); break;
    case 1: store_run_d<1>(p, c.D, vec, grid, threads, s); break;
    default: store_run_d<2>(p, c.D, vec, grid, threads, s); break;
  }
  return hipGetLastError();
}

}  // namespace tq
