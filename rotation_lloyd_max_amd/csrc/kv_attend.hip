// Attention over the paged compressed cache: dispatch, workspace, and the join of units that
// several workgroups share (the kernels are in kv_attend.hpp).
#include "kv_attend_wide.hpp"

namespace tq {

extern template hipError_t at_launch_k<2>(const AttendParams& p, int vbits, int D, int rows, hipStream_t s);
extern template hipError_t at_launch_k<3>(const AttendParams& p, int vbits, int D, int rows, hipStream_t s);
extern template hipError_t at_launch_k<4>(const AttendParams& p, int vbits, int D, int rows, hipStream_t s);
extern template hipError_t at_launch_k<8>(const AttendParams& p, int vbits, int D, int rows, hipStream_t s);

namespace {

constexpr size_t kMetaBytes = sizeof(AttendMeta) * kAtMaxGrid;

// Query rows of a tile, and the workgroups of a launch. By the rows that share a key head of a sequence
// (8 sequences of 4096 tokens, 8 key heads of 128, 8-bit keys, 3-bit values; whole call, us):
//   rows                              8   32   64  128  132  256  2048 (4 sequences)
//   tiles of 16: waves share rows,   28   38   57
//       each decoding its own tokens
//   tiles of 128: waves split the    50   50   52   66   93   94   294
//       rows and share each block
//   tiles of 256                               66   86   85   87   216
int tile_rows(int D, int share, int B, int64_t M) {
  const int64_t rows = (M * share + B - 1) / B;
  return rows <= 48 ? 16 : rows <= 128 || D == 256 ? 128 : 256;
}
int workgroups(int D, int rows) { return (rows > 16 ? 1 : D <= 128 ? 3 : 2) * kAtCus; }

// What the join needs of the arguments.
struct JoinParams {
  const AttendMeta* meta;
  const float* parts;
  const uint32_t* vsigns;
  uint16_t* out;
  int q_heads, odt, rows;
  uint32_t hb_mul;
  int hb;
  float inv_sqrt_d;
};

// Normalises, rotates back and stores one output row held as in kv_wave_transform; sg: the
// lane's sign bits.
template <int D, typename P>
__device__ __forceinline__ void at_finish(P p, float (&v)[D / 64], float l, int64_t m, int head, uint32_t sg, int lane) {
  constexpr int EL = D / 64;
  const float f = p->inv_sqrt_d / l;
  sg ^= 0u - kv_sign(kv_chunk(lane));
#pragma unroll
  for (int e = 0; e < EL; ++e) v[e] = l == 0.f ? 0.f : v[e] * f;
  const int c = kv_chunk(lane);
  kv_wave_transform<EL>(v, c);
  const int odt = p->odt;
  uint16_t* dst = p->out + (m * p->q_heads + head) * D + c * EL;
  uint16_t x[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    const float y = (sg >> e) & 1u ? -v[e] : v[e];
    x[e] = odt == 1 ? float_to_bf16_rne(y) : float_to_half_rne(y);
  }
  __builtin_memcpy(__builtin_assume_aligned(dst, 2 * EL), x, 2 * EL);
}

// The query rows of units whose parts lie in several workgroups' slots, the parts added in the order
// of the tokens. Few parts each: many rows, and what bounds it is the instructions of a row, so a wave
// takes several (65536 rows of 128: 22 us with a row per wave, 15 us so). Many parts: few rows, one per
// wave.
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(JoinParams p) {
  constexpr int EL = D / 64;
  __shared__ float wt[4][kAtMaxGrid];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const AttendMeta m = p.meta[blockIdx.x];
  if (m.parts == 0) return;
  const int n = m.parts + 1;
  const int64_t slot = static_cast<int64_t>(p.rows) * (D + 2);
  // part 0 is the second slot of its workgroup, the others the first of theirs
  const float* const base = p.parts + 2 * static_cast<int64_t>(blockIdx.x) * slot;
  auto part = [&](int i) { return base + (i == 0 ? slot : 2 * i * slot); };
  // K parts, everything at once (past the last part: that one again, unused)
  auto few = [&](auto count) {
    constexpr int K = decltype(count)::value;
    const AtRows<D> rows;
    const int r = (blockIdx.y * 4 + wave) * AtRows<D>::N + rows.sub;
    if (r >= p.rows) return;
    const int tk = (static_cast<uint32_t>(r) * p.hb_mul) >> 16, hd = r - tk * p.hb;
    f32x4_t x[K][2];
    float a[K], b[K], v[8] = {}, top = kAtNone, l = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float* s = part(k < n ? k : n - 1);
      a[k] = s[p.rows * D + r];
      b[k] = s[p.rows * D + p.rows + r];
#pragma unroll
      for (int e = 0; e < 2; ++e) x[k][e] = *reinterpret_cast<const f32x4_t*>(s + r * D + 8 * rows.c + 4 * e);
    }
    const uint32_t sg = rows.signs(p.vsigns);
#pragma unroll
    for (int k = 0; k < K; ++k) top = fmaxf(top, a[k]);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k >= n) break;
      const float f = a[k] == kAtNone ? 0.f : at_exp2(a[k] - top);
      l += b[k] != b[k] ? b[k] : b[k] * f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(f, x[k][e >> 2][e & 3], v[e]);
    }
    at_store<D>(&p, v, l, static_cast<int64_t>(m.row0) + tk, m.head0 + hd, sg, rows.c, tk < m.nrows && hd < m.nh);
  };
  if (n <= 4) return few(AtInt<4>{});
  if (n <= 8) return few(AtInt<8>{});
  const int r = blockIdx.y * 4 + wave, tk = (static_cast<uint32_t>(r) * p.hb_mul) >> 16, hd = r - tk * p.hb;
  if (tk >= m.nrows || hd >= m.nh) return;
  const int d0 = kv_chunk(lane) * EL;
  const uint32_t sg = p.vsigns[d0 >> 5] >> (d0 & 31);
  float top = kAtNone, l = 0.f;
  float v[EL] = {};
  for (int i = lane; i < n; i += 64) {
    const float a = part(i)[p.rows * D + r];
    wt[wave][i] = a;
    top = fmaxf(top, a);
  }
  top = kv_wave_max(top);
  for (int i = lane; i < n; i += 64) {
    const float a = wt[wave][i], b = part(i)[p.rows * D + p.rows + r];
    const float f = a == kAtNone ? 0.f : at_exp2(a - top);
    wt[wave][i] = f;
    l += b != b ? b : b * f;
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
  wave_lds_sync();
  // sixteen parts' loads at a time
  for (int i0 = 0; i0 < n; i0 += 16) {
    float x[16][EL];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float* s = part(i0 + k < n ? i0 + k : n - 1) + r * D + d0;
#pragma unroll
      for (int e = 0; e < EL; ++e) x[k][e] = s[e];
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float f = i0 + k < n ? wt[wave][i0 + k] : 0.f;
#pragma unroll
      for (int e = 0; e < EL; ++e) v[e] = __builtin_fmaf(f, x[k][e], v[e]);
    }
  }
  at_finish<D>(&p, v, l, static_cast<int64_t>(m.row0) + tk, m.head0 + hd, sg, lane);
}

uint32_t div_mul(uint32_t d) { return d == 1 ? 0 : static_cast<uint32_t>((0x100000000ull + d - 1) / d); }

}  // namespace

size_t kv_attend_workspace(const KvCacheArgs& c, int q_heads, int B, int64_t M) {
  if (B == 0 || M == 0) return 0;
  const int rows = tile_rows(c.D, q_heads / c.heads, B, M);
  return kMetaBytes + 2 * static_cast<size_t>(workgroups(c.D, rows)) * rows * (c.D + 2) * sizeof(float);
}

hipError_t launch_kv_attend(const AttendArgs& a, hipStream_t s) {
  AttendParams p{};
  const int D = a.c.D;
  p.kcodes = a.c.k.codes; p.vcodes = a.c.v.codes; p.ksigns = a.c.k.signs; p.vsigns = a.c.v.signs;
  p.kscales = a.c.k.scales; p.vscales = a.c.v.scales;
  p.q = static_cast<const uint16_t*>(a.q);
  p.out = static_cast<uint16_t*>(a.out);
  p.q_offsets = a.q_offsets; p.kv_lens = a.kv_lens; p.page_table = a.page_table; p.tree = a.tree;
  p.q_stride = a.q_stride; p.qdt = a.qdt; p.odt = a.odt; p.q_heads = a.q_heads; p.B = a.B;
  p.M = static_cast<int>(a.M); p.table_width = a.table_width; p.tree_words = a.tree_words;
  p.heads = a.c.heads; p.pages = static_cast<int>(a.c.pages); p.page = a.c.page;
  p.page16 = a.c.page / 16;
  p.page_mul = div_mul(p.page16);
  p.lg_kg = __builtin_ctz(a.c.k.group); p.lg_vg = __builtin_ctz(a.c.v.group);
  p.lg_gk = __builtin_ctz(D / a.c.k.group); p.lg_gv = __builtin_ctz(D / a.c.v.group);
  p.share = a.q_heads / a.c.heads;
  const int rows = tile_rows(D, p.share, a.B, a.M);
  p.hb = p.share < rows ? p.share : rows;
  p.nhb = (p.share + p.hb - 1) / p.hb;
  p.a_tok = rows / p.hb;
  p.hb_mul = (65536 + p.hb - 1) / p.hb;  // r hb < 2^16 for the rows r: the product is exact
  p.a_mul = div_mul(p.a_tok);
  p.hu_n = a.c.heads * p.nhb;
  p.cap = a.table_width * a.c.page;
  p.n_each = static_cast<int>(a.M / a.B);
  p.negate = a.scale < 0.f;
  p.inv_sqrt_d = static_cast<float>(1.0 / __builtin_sqrt(static_cast<double>(D)));
  p.c1 = __builtin_fabsf(a.scale) * 1.44269504f * p.inv_sqrt_d;
  p.meta = static_cast<AttendMeta*>(a.ws);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kMetaBytes);
  for (int i = 0; i < 2; ++i) {
    const int levels = i ? a.c.v.levels : a.c.k.levels;
    const uint16_t* hb = levels == 256 ? codebook256()->h : codebook_for(levels)->h;
    for (int k = 0; k < levels; ++k) (i ? p.hv : p.hk)[k] = hb[k];
  }
  hipError_t e;
  switch (a.c.k.bits) {
    case 2: e = at_launch_k<2>(p, a.c.v.bits, D, rows, s); break;
    case 3: e = at_launch_k<3>(p, a.c.v.bits, D, rows, s); break;
    case 4: e = at_launch_k<4>(p, a.c.v.bits, D, rows, s); break;
    default: e = at_launch_k<8>(p, a.c.v.bits, D, rows, s); break;
  }
  if (e != hipSuccess) return e;
  JoinParams j{p.meta, p.parts, p.vsigns, p.out, p.q_heads, p.odt, rows, p.hb_mul, p.hb, p.inv_sqrt_d};
  const dim3 grid(workgroups(D, rows), rows / 4);
  if (D == 64) hipLaunchKernelGGL((k_attend_join<64>), grid, dim3(256), 0, s, j);
  else if (D == 128) hipLaunchKernelGGL((k_attend_join<128>), grid, dim3(256), 0, s, j);
  else hipLaunchKernelGGL((k_attend_join<256>), grid, dim3(256), 0, s, j);
  return hipGetLastError();
}

}  // namespace tq
