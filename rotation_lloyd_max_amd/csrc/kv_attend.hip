// Attention over the paged compressed cache: dispatch, workspace, and the join of units that
// several workgroups share (the kernels are in kv_attend.hpp).
#include "encode_lane.hpp"
#include "kv_attend.hpp"

namespace tq {

extern template hipError_t at_launch_k<2>(const AttendParams& p, int R, hipStream_t s);
extern template hipError_t at_launch_k<3>(const AttendParams& p, int R, hipStream_t s);
extern template hipError_t at_launch_k<4>(const AttendParams& p, int R, hipStream_t s);
extern template hipError_t at_launch_k<8>(const AttendParams& p, int R, hipStream_t s);

namespace {

constexpr size_t kMetaBytes = sizeof(AttendMeta) * kAtMaxGrid;

// 16-row blocks of a tile.
int workgroups(int D, int R) { return (R == 1 && D <= 128 ? 3 : 2) * kAtCus; }
int tile_blocks(int D, int share, int B, int64_t M) {
  const int64_t rows = (M * share + B - 1) / (B > 0 ? B : 1);  // query rows per key head and sequence
  return rows <= 16 ? 1 : D == 256 ? 2 : 4;
}

// One wave per query row of a unit whose parts lie in several workgroups' slots, in the
// order of the tokens.
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(AttendParams p, int rows) {
  constexpr int EL = D / 64;
  __shared__ float wt[4][kAtMaxGrid];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const AttendMeta m = p.meta[blockIdx.x];
  if (m.parts == 0) return;
  const int r = blockIdx.y * 4 + wave, tk = r / p.hb, hd = r - tk * p.hb;
  if (tk >= m.nrows || hd >= m.hb) return;
  const int n = m.parts + 1;
  const int64_t slot = static_cast<int64_t>(rows) * (D + 2);
  auto part = [&](int i) { return p.parts + (2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * slot; };
  float top = -__builtin_inff(), l = 0.f;
  for (int i = lane; i < n; i += 64) top = fmaxf(top, part(i)[rows * D + r]);
  top = kv_wave_max(top);
  for (int i = lane; i < n; i += 64) {
    const float a = part(i)[rows * D + r], b = part(i)[rows * D + rows + r];
    const float f = a == -__builtin_inff() ? 0.f : at_exp2(a - top);
    wt[wave][i] = f;
    l += b != b ? b : b * f;
  }
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) l += __shfl_xor(l, x);
  wave_lds_sync();
  float v[EL] = {};
  for (int i = 0; i < n; ++i) {
    const float f = wt[wave][i];
    const float* s = part(i) + r * D + kv_chunk(lane) * EL;
#pragma unroll
    for (int e = 0; e < EL; ++e) v[e] += f == 0.f ? 0.f : f * s[e];
  }
  at_finish<D>(p, v, l, m.row0 + tk, m.head0 + hd, lane);
}

}  // namespace

size_t kv_attend_workspace(const KvCacheArgs& c, int q_heads, int B, int64_t M) {
  if (B == 0 || M == 0) return 0;
  const int R = tile_blocks(c.D, q_heads / c.heads, B, M);
  const size_t rows = 16 * R;
  return kMetaBytes + 2 * workgroups(c.D, R) * rows * (c.D + 2) * sizeof(float);
}

hipError_t launch_kv_attend(const AttendArgs& a, hipStream_t s) {
  AttendParams p{};
  p.a = a;
  p.share = a.q_heads / a.c.heads;
  const int R = tile_blocks(a.c.D, p.share, a.B, a.M), rows = 16 * R;
  p.hb = p.share < rows ? p.share : rows;
  p.nhb = (p.share + p.hb - 1) / p.hb;
  p.a_tok = rows / p.hb;
  p.grid = workgroups(a.c.D, R);
  p.n_each = static_cast<int>(a.M / a.B);
  p.inv_sqrt_d = static_cast<float>(1.0 / __builtin_sqrt(static_cast<double>(a.c.D)));
  p.page16 = a.c.page / 16;
  p.page_mul = p.page16 == 1 ? 0 : static_cast<uint32_t>((0x100000000ull + p.page16 - 1) / p.page16);
  p.meta = static_cast<AttendMeta*>(a.ws);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a.ws) + kMetaBytes);
  for (int i = 0; i < 2; ++i) {
    const int levels = i ? a.c.v.levels : a.c.k.levels;
    const uint16_t* hb = levels == 256 ? codebook256()->h : codebook_for(levels)->h;
    for (int k = 0; k < levels; ++k) (i ? p.hv : p.hk)[k] = hb[k];
  }
  hipError_t e;
  switch (a.c.k.bits) {
    case 2: e = at_launch_k<2>(p, R, s); break;
    case 3: e = at_launch_k<3>(p, R, s); break;
    case 4: e = at_launch_k<4>(p, R, s); break;
    default: e = at_launch_k<8>(p, R, s); break;
  }
  if (e != hipSuccess) return e;
  const dim3 grid(p.grid, rows / 4);
  if (a.c.D == 64) hipLaunchKernelGGL((k_attend_join<64>), grid, dim3(256), 0, s, p, rows);
  else if (a.c.D == 128) hipLaunchKernelGGL((k_attend_join<128>), grid, dim3(256), 0, s, p, rows);
  else hipLaunchKernelGGL((k_attend_join<256>), grid, dim3(256), 0, s, p, rows);
  return hipGetLastError();
}

}  // namespace tq
