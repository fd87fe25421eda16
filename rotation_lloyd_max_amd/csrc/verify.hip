// Verification of drafted tokens against the target's distribution (tq_verify).
//
// The walk. At row c, with target p and draft q, the children are tried in their order; after k of them
// went, what is left of p is proportional to (p - a_k q)+ with a_0 = 0, a_{k+1} = a_k + S_k, S_k = sum
// (p - a_k q)+ (S_0 = 1): if r = (p - a q)+ / S, then (r - q)+ = (p - (a + S) q)+ / S. So the state is one
// number, a, and its sum, and no distribution is ever stored. Without a draft the tried tokens are taken
// out of p one by one. Children have larger indices than their parents and are tried in ascending
// order: one ascending scan of a sequence's rows is the walk.
//
// Everything that decides is fp64: the new token is found at u sum(w) in the cumulative sum of w, and
// each of 10^5 borders in it that is off by 10^-8 gives a neighbour now and then.
//
// Two launches. k_verify_stats: largest value and sum of exponentials of every row of logits that can
// be looked at, a wave per piece of a row. k_verify_pick: each workgroup of a sequence joins the pieces and
// walks (all do the same: cheaper than another launch), sums w over its share of the vocabulary, and
// the one that comes last finds the token. Where siblings are tried against a draft, sums S are needed
// during the walk: k_verify_walk, a workgroup per sequence, goes first.
#include "device_common.hpp"
#include "internal.hpp"

namespace tq {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kBlockElems = 512;    // a wave's step: 8 elements a lane
constexpr int kWindow = 256;        // rows whose probabilities are in LDS at a time
constexpr int kGone = 256;          // tried tokens in LDS
constexpr int kTable = 256;         // 2^(i / 256)

// Of a piece of a row, in units of the largest value: z = sum 2^((x - top) c), c = log2(e) / T. Where
// it holds NaN or +infinity z is NaN. at: the index of its first largest value (greedy rows).
struct StatPart {
  double z;
  float top;
  int at;
};

struct Side {  // target or draft
  const char* data;
  int64_t stride;  // bytes
  int dt;
  bool probs;
  const StatPart* stat;  // [rows][parts]
};

// What the walk found (k_verify_walk to k_verify_pick).
struct Walked {
  double al;
  int cur, kept, tried;
};

struct VerifyParams {
  VerifyArgs a;
  Side t, d;
  int parts, part_blocks;  // pieces of a row of logits, and kBlockElems in each
  int shares, share_blocks;  // the same of k_verify_pick's workgroups
  double* sums;            // [B][blocks]
  int* tickets;            // [B]
  Walked* walked;          // [B] where k_verify_walk runs
};

typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements from i on (all inside the row), at any alignment of the type.
template <int DT>
__device__ __forceinline__ void load8(const char* row, int i, float (&f)[8]) {
  if constexpr (DT == 0) {
    const u32x4_a2 a = *reinterpret_cast<const u32x4_a2*>(row + static_cast<int64_t>(i) * 4);
    const u32x4_a2 b = *reinterpret_cast<const u32x4_a2*>(row + static_cast<int64_t>(i) * 4 + 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = __uint_as_float(a[k]);
      f[4 + k] = __uint_as_float(b[k]);
    }
  } else {
    const u32x4_a2 a = *reinterpret_cast<const u32x4_a2*>(row + static_cast<int64_t>(i) * 2);
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
// The same at the end of a row: `none` behind it.
template <int DT>
__device__ __forceinline__ void load8_end(const char* row, int i, int V, float none, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = i + k < V ? load_elem<DT>(row, i + k) : none;
}
__device__ __forceinline__ void load8_any(const char* row, int dt, int i, int V, float none, float (&f)[8]) {
  const bool whole = i + 8 <= V;
  if (dt == 0) whole ? load8<0>(row, i, f) : load8_end<0>(row, i, V, none, f);
  else if (dt == 1) whole ? load8<1>(row, i, f) : load8_end<1>(row, i, V, none, f);
  else whole ? load8<2>(row, i, f) : load8_end<2>(row, i, V, none, f);
}

__device__ __forceinline__ void fill_table(double* tab) {
  for (int i = threadIdx.x; i < kTable; i += blockDim.x) tab[i] = exp2(i * (1.0 / kTable));
  __syncthreads();
}

// s + 2^t for t < 1000, to 2e-14 of 2^t; t below -1000 counts as -1000, NaN too. 2^t = 2^k 2^(i / 256) 2^r,
// |r| <= 1 / 512: k and i from the low bits of t + 1.5 2^44, 2^r = e^y by the polynomial of degree 3 with
// the least error on |y| <= h = ln 2 / 512 (y^4 / 24 replaced by its nearest of degree 2, h^2 y^2 - h^4 / 8).
__device__ __forceinline__ double add_exp2(double t, double s, const double* tab) {
  constexpr double kMagic = 26388279066624.0;  // 1.5 2^44: steps of 1 / 256
  constexpr double kLn2 = 0.69314718055994530942, kH = kLn2 / 512;
  t = __builtin_fmax(t, -1000.0);
  const double z = t + kMagic;
  const double r = t - (z - kMagic);
  const uint32_t i = static_cast<uint32_t>(__double2loint(z));
  double p = __builtin_fma(r, kLn2 * kLn2 * kLn2 / 6, kLn2 * kLn2 * (0.5 + kH * kH / 24));
  p = __builtin_fma(p, r, kLn2);
  p = __builtin_fma(p, r, 1.0 - kH * kH * kH * kH / 192);
  const double w = tab[i & (kTable - 1)];
  return __builtin_fma(__hiloint2double(__double2hiint(w) + ((i & ~(kTable - 1u)) << 12), __double2loint(w)), p, s);
}

__device__ __forceinline__ double temperature_of(const VerifyArgs& a, int b) { return a.temperature ? a.temperature[b] : 1.0; }
__device__ __forceinline__ double scale_of(double T) { return 1.4426950408889634074 / T; }

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int s = 32; s; s >>= 1) x = __builtin_elementwise_maximum(x, __shfl_xor(x, s));
  return x;
}
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
  return x;
}

// The largest b with offsets[b] <= row, by all lanes of a wave.
__device__ __forceinline__ int seq_of(const int32_t* offsets, int B, int row) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6, i = lo + lane * step;
    const int below = __popcll(__ballot(i < hi && offsets[i] <= row));
    lo += (below > 1 ? below - 1 : 0) * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  return lo;
}

// Bounds of a sequence's rows, inside [0, M].
__device__ __forceinline__ void seq_rows(const VerifyArgs& a, int b, int& lo, int& hi) {
  lo = a.offsets[b];
  hi = a.offsets[b + 1];
  lo = lo < 0 ? 0 : lo < a.M ? lo : a.M;
  hi = hi < lo ? lo : hi < a.M ? hi : a.M;
}

// ---- statistics of the rows ---------------------------------------------------------------

template <int DT>
__device__ __forceinline__ StatPart stat_piece(const char* row, int V, int i0, int i1, double c, const double* tab) {
  const int lane = threadIdx.x & 63;
  const float inf = __builtin_inff();
  float f[8], top = -inf, ref = 0.f;
  double s0 = 0.0, s1 = 0.0, base = 0.0;
  bool first = true;
  // relative to the lane's first eight values, which may turn out to be far below the others
  for (int i = i0 + 8 * lane; i < i1; i += kBlockElems) {
    if (i + 8 <= V) load8<DT>(row, i, f);
    else load8_end<DT>(row, i, V, -inf, f);
    float m = __builtin_elementwise_maximum(f[0], f[1]);
#pragma unroll
    for (int k = 2; k < 8; k += 2)
      m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, f[k]), f[k + 1]);
    top = __builtin_elementwise_maximum(top, m);
    if (first) {
      ref = __builtin_fabsf(m) < inf ? m : 0.f;
      base = ref;
      first = false;
    }
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      s0 = add_exp2((f[k] - base) * c, s0, tab);
      s1 = add_exp2((f[k + 1] - base) * c, s1, tab);
    }
  }
  double s = s0 + s1;
  if (!((static_cast<double>(top) - base) * c < 900.0) || s < 0x1p-900) {
    // ... or far above them; or none is finite
    s = 0.0;
    ref = top;
    if (top != top || top == inf) {
      s = __builtin_nan("");
    } else if (top > -inf) {
      for (int i = i0 + 8 * lane; i < i1; i += kBlockElems) {
        load8_end<DT>(row, i, V, -inf, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) s = add_exp2((f[k] - static_cast<double>(ref)) * c, s, tab);
      }
    }
  }
  StatPart p;
  p.top = wave_max(top);
  p.at = 0;
  if (s != 0.0) s *= add_exp2((static_cast<double>(ref) - p.top) * c, 0.0, tab);
  p.z = wave_sum(s);
  if (p.top != p.top || p.top == inf) p.z = __builtin_nan("");
  return p;
}

// Greedy rows: the first largest value.
template <int DT>
__device__ __forceinline__ StatPart stat_largest(const char* row, int V, int i0, int i1) {
  const int lane = threadIdx.x & 63;
  const float inf = __builtin_inff();
  float f[8], top = -inf;
  int at = 0x7fffffff;
  bool bad = false;
  for (int i = i0 + 8 * lane; i < i1; i += kBlockElems) {
    if (i + 8 <= V) load8<DT>(row, i, f);
    else load8_end<DT>(row, i, V, -inf, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      bad |= !(f[k] < inf);
      if (f[k] > top) {
        top = f[k];
        at = i + k;
      }
    }
  }
  StatPart p;
  p.top = wave_max(top);
  if (top != p.top) at = 0x7fffffff;
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const int o = __shfl_xor(at, s);
    at = o < at ? o : at;
  }
  p.at = at;
  p.z = __ballot(bad) ? __builtin_nan("") : 0.0;
  return p;
}

// A wave per piece of a row: the target's rows, then (of logits) the draft's.
__global__ __launch_bounds__(kVerifyThreads) void k_verify_stats(VerifyParams p, int64_t unit0, int64_t units) {
  __shared__ double tab[kTable];
  const VerifyArgs& a = p.a;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.B; i += kVerifyThreads) p.tickets[i] = 0;
  fill_table(tab);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int lim = a.offsets[a.B] < a.M ? a.offsets[a.B] : a.M;
  for (int64_t unit = unit0 + static_cast<int64_t>(blockIdx.x) * (kVerifyThreads / 64) + wave; unit < units;
       unit += static_cast<int64_t>(gridDim.x) * (kVerifyThreads / 64)) {
    const int line = static_cast<int>(unit / p.parts), part = static_cast<int>(unit - static_cast<int64_t>(line) * p.parts);
    const bool draft = line >= a.M;
    const int row = draft ? line - a.M : line;
    if (row >= lim) continue;
    const Side& s = draft ? p.d : p.t;
    double T = 1.0;
    if (a.temperature || draft) {
      const int b = seq_of(a.offsets, a.B, row);
      T = temperature_of(a, b);
      if (draft) {  // rows without children are not looked at
        if (!(T > 0.0)) continue;
        const int lo = a.offsets[b], hi = a.offsets[b + 1] < lim ? a.offsets[b + 1] : lim;
        bool child = row + 1 < hi;
        if (a.parents) {
          child = false;
          for (int r = row + 1; r < hi && !child; r += 64) child = __ballot(r + lane < hi && a.parents[r + lane] == row - lo) != 0;
        }
        if (!child) continue;
      }
    }
    const bool greedy = !(T > 0.0);
    if (s.probs && !greedy) continue;
    const char* x = s.data + row * s.stride;
    const int i0 = part * p.part_blocks * kBlockElems;
    const int64_t end = static_cast<int64_t>(i0) + p.part_blocks * kBlockElems;
    const int i1 = end < a.V ? static_cast<int>(end) : a.V;
    StatPart r;
    if (greedy) {
      r = s.dt == 0 ? stat_largest<0>(x, a.V, i0, i1) : s.dt == 1 ? stat_largest<1>(x, a.V, i0, i1) : stat_largest<2>(x, a.V, i0, i1);
    } else {
      const double c = scale_of(T);
      r = s.dt == 0 ? stat_piece<0>(x, a.V, i0, i1, c, tab) : s.dt == 1 ? stat_piece<1>(x, a.V, i0, i1, c, tab)
                                                                      : stat_piece<2>(x, a.V, i0, i1, c, tab);
    }
    if (lane == 0) const_cast<StatPart*>(s.stat)[static_cast<int64_t>(row) * p.parts + part] = r;
  }
}

// ---- rows as distributions ------------------------------------------------------------------

struct Dist {
  const char* row;
  double c, ref, zinv;  // logits: 2^((x - ref) c) zinv; NaN for a row that is none
};

__device__ __forceinline__ double value_of(const Side& s, const Dist& d, int i, const double* tab) {
  const double x = load_any(d.row, s.dt, i);
  if (s.probs) return x;
  const double t = (x - d.ref) * d.c;
  return (t <= -1000.0 || x == -__builtin_inf() ? 0.0 : add_exp2(t, 0.0, tab)) * d.zinv;
}

// Row `row` of one side from its pieces, by `lanes` neighbouring lanes (a power of two).
__device__ __forceinline__ Dist dist_of(const VerifyParams& p, const Side& s, int row, double c, int lanes, const double* tab) {
  Dist d;
  d.row = s.data + row * s.stride;
  d.c = c;
  d.ref = 0.0;
  d.zinv = 1.0;
  if (s.probs) return d;
  const StatPart* st = s.stat + static_cast<int64_t>(row) * p.parts;
  const int l = threadIdx.x & (lanes - 1);
  float top = -__builtin_inff();
  for (int k = l; k < p.parts; k += lanes) top = __builtin_elementwise_maximum(top, st[k].top);
  for (int m = lanes >> 1; m; m >>= 1) top = __builtin_elementwise_maximum(top, __shfl_xor(top, m));
  double z = 0.0;
  for (int k = l; k < p.parts; k += lanes) {
    const StatPart q = st[k];
    if (q.z != 0.0) z += q.z * add_exp2((static_cast<double>(q.top) - top) * c, 0.0, tab);
  }
  for (int m = lanes >> 1; m; m >>= 1) z += __shfl_xor(z, m);
  d.ref = top;
  d.zinv = z > 0.0 && z < __builtin_inf() ? 1.0 / z : __builtin_nan("");
  return d;
}

// The first largest value of a greedy row: its index, or -1. By a wave.
__device__ __forceinline__ int largest_of(const VerifyParams& p, int row) {
  const StatPart* st = p.t.stat + static_cast<int64_t>(row) * p.parts;
  const int lane = threadIdx.x & 63;
  float top = -__builtin_inff();
  bool bad = false;
  for (int k = lane; k < p.parts; k += 64) {
    bad |= st[k].z != 0.0;
    top = __builtin_elementwise_maximum(top, st[k].top);
  }
  top = wave_max(top);
  int at = 0x7fffffff;
  for (int k = lane; k < p.parts; k += 64)
    if (st[k].top == top && st[k].at < at) at = st[k].at;
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const int o = __shfl_xor(at, s);
    at = o < at ? o : at;
  }
  if (__ballot(bad) || !(top > (p.t.probs ? 0.f : -__builtin_inff()))) return -1;
  return at;
}

// ---- weights ----------------------------------------------------------------------------------

// What the new token is drawn from (or S is summed over).
struct Weights {
  Dist p, q;
  double al;        // (p - al q)+ where drafted
  bool drafted;
  int ngone;        // tokens taken out of p; more than kGone: look among the rows
};

// w of elements i .. i + 7 (0 behind the row).
__device__ __forceinline__ void weights8(const VerifyParams& p, const Weights& w, int i, const double* tab, double (&v)[8]) {
  const float none = -__builtin_inff();
  float f[8];
  load8_any(w.p.row, p.t.dt, i, p.a.V, p.t.probs ? 0.f : none, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (p.t.probs) {
      v[k] = f[k];
    } else {
      const double t = (f[k] - w.p.ref) * w.p.c;
      v[k] = t <= -1000.0 || f[k] == none ? 0.0 : add_exp2(t, 0.0, tab) * w.p.zinv;
    }
  }
  if (w.drafted) {
    load8_any(w.q.row, p.d.dt, i, p.a.V, p.d.probs ? 0.f : none, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      double q = f[k];
      if (!p.d.probs) {
        const double t = (f[k] - w.q.ref) * w.q.c;
        q = t <= -1000.0 || f[k] == none ? 0.0 : add_exp2(t, 0.0, tab) * w.q.zinv;
      }
      v[k] = __builtin_fma(-w.al, q, v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = v[k] < 0.0 ? 0.0 : v[k];
}

// ---- the walk -----------------------------------------------------------------------------

struct WalkShared {
  double px[kWindow], qx[kWindow], u[kWindow];
  int parent[kWindow], token[kWindow], gone[kGone];
  double tab[kTable], red[64];
};

__device__ __forceinline__ int parent_of(const VerifyArgs& a, int lo, int r) { return a.parents ? a.parents[lo + r] : r - 1; }

// Whether a child of cur before row `end` has token x, by all lanes of a wave.
__device__ __forceinline__ bool tried_before(const VerifyArgs& a, const WalkShared& sh, int lo, int n, int cur, int end, int x) {
  const int lane = threadIdx.x & 63;
  bool found = false;
  for (int r = cur + 1; r < end && !found; r += 64) {
    const int i = r + lane;
    bool hit = false;
    if (i < end) hit = n <= kWindow ? sh.parent[i] == cur && sh.token[i] == x : parent_of(a, lo, i) == cur && a.tokens[lo + i] == x;
    found = __ballot(hit) != 0;
  }
  return found;
}

// The walk of sequence b, by all waves of the workgroup alike; `writes`: this workgroup writes the
// outputs but the new token. `sum(cur, al)`: S of a row, called by all threads (SUMS only).
template <int NT, bool SUMS, typename F>
__device__ __forceinline__ Walked walk(const VerifyParams& p, WalkShared& sh, int lo, int n, double T, bool writes, F sum) {
  const VerifyArgs& a = p.a;
  const int lane = threadIdx.x & 63;
  const bool greedy = !(T > 0.0), drafted = a.draft && !greedy;
  const double c = scale_of(T);
  Walked w{0.0, 0, 1, 0};
  double S = 1.0;
  int largest = greedy ? largest_of(p, lo) : -1;
  bool over = false;
  for (int w0 = 0; w0 < n && !over; w0 += kWindow) {
    const int w1 = n - w0 < kWindow ? n : w0 + kWindow;
    // the probabilities of the window's tokens under their parents
    if (w0) __syncthreads();
    constexpr int LANES = 16;
    for (int r = w0 + static_cast<int>(threadIdx.x) / LANES; r < w1; r += NT / LANES) {
      const int up = parent_of(a, lo, r), x = a.tokens[lo + r];
      const bool any = r > 0 && up >= 0 && up < r && x >= 0 && x < a.V;
      double px = 0.0, qx = 0.0;
      if (any && !greedy) {
        const Dist t = dist_of(p, p.t, lo + up, c, LANES, sh.tab);
        px = value_of(p.t, t, x, sh.tab);
        if (drafted) {
          const Dist q = dist_of(p, p.d, lo + up, c, LANES, sh.tab);
          qx = value_of(p.d, q, x, sh.tab);
        }
      }
      if ((threadIdx.x & (LANES - 1)) == 0) {
        sh.parent[r - w0] = any ? up : -1;
        sh.token[r - w0] = x;
        sh.px[r - w0] = px;
        sh.qx[r - w0] = qx;
        sh.u[r - w0] = a.uniforms[lo + r];
      }
    }
    __syncthreads();
    for (int next = w0;;) {
      // the next child of cur in the window
      int r = w1;
      for (int i = next; i < w1; i += 64) {
        const uint64_t m = __ballot(i + lane < w1 && sh.parent[i + lane - w0] == w.cur);
        if (m) {
          r = i + __builtin_ctzll(m);
          break;
        }
      }
      if (r >= w1) break;
      next = r + 1;
      const int x = sh.token[r - w0];
      const double u = sh.u[r - w0], px = sh.px[r - w0], qx = sh.qx[r - w0];
      bool yes, taken = false;
      if (greedy) {
        yes = x == largest;
      } else if (drafted) {
        yes = u * S * qx < px - w.al * qx;
      } else {
        taken = w.tried && tried_before(a, sh, lo, n, w.cur, r, x);
        yes = u * S < (taken ? 0.0 : px);
      }
      if (yes) {
        if (writes && threadIdx.x == 0) {
          a.out_tokens[lo + w.kept - 1] = x;
          a.path[lo + w.kept] = r;
        }
        w.cur = r;
        ++w.kept;
        w.tried = 0;
        w.al = 0.0;
        S = 1.0;
        if (greedy) largest = largest_of(p, lo + r);
      } else {
        ++w.tried;
        if (drafted) {
          w.al += S;
          if constexpr (SUMS) {
            // (of use only if another child follows)
            bool more = false;
            for (int i = r + 1; i < n && !more; i += 64) more = __ballot(i + lane < n && parent_of(a, lo, i + lane) == w.cur) != 0;
            if (more) S = sum(w.cur, w.al);
          }
        } else if (!taken) {
          S -= px;
        }
        if (!a.parents) over = true;
        if (over) break;
      }
    }
  }
  if (writes) {
    for (int i = w.kept + threadIdx.x; i < n; i += NT) {
      a.out_tokens[lo + i] = -1;
      a.path[lo + i] = -1;
    }
    if (threadIdx.x == 0) a.path[lo] = 0;
  }
  return w;
}

// Rows with siblings tried against a draft: S of the rows on the way takes passes over the vocabulary.
constexpr int kWalkThreads = 1024;
__global__ __launch_bounds__(kWalkThreads) void k_verify_walk(VerifyParams p) {
  __shared__ WalkShared sh;
  const VerifyArgs& a = p.a;
  const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int lo, hi;
  seq_rows(a, b, lo, hi);
  if (hi == lo) return;
  fill_table(sh.tab);
  const double T = temperature_of(a, b);
  auto sum = [&](int cur, double al) {
    Weights w;
    w.p = dist_of(p, p.t, lo + cur, scale_of(T), 64, sh.tab);
    w.q = dist_of(p, p.d, lo + cur, scale_of(T), 64, sh.tab);
    w.al = al;
    w.drafted = true;
    double s = 0.0, v[8];
    for (int i = threadIdx.x * 8; i < a.V; i += kWalkThreads * 8) {
      weights8(p, w, i, sh.tab, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
    s = wave_sum(s);
    __syncthreads();
    if (lane == 0) sh.red[wave] = s;
    __syncthreads();
    s = 0.0;
    for (int k = 0; k < kWalkThreads / 64; ++k) s += sh.red[k];
    return s;
  };
  const Walked w = walk<kWalkThreads, true>(p, sh, lo, hi - lo, T, true, sum);
  if (threadIdx.x == 0) {
    p.walked[b] = w;
    a.kept[b] = w.kept;
  }
}

// ---- the new token ----------------------------------------------------------------------------

// The first k < count with get(0) + .. + get(k) > u total (the last with get(k) > 0 if there is none), and
// the sum before it; -1 if the total is not above 0 and finite. By all threads of the workgroup.
template <typename F>
__device__ __forceinline__ int locate(WalkShared& sh, int count, F get, double u, double& total, double& before, double& goal) {
  constexpr int NT = kVerifyThreads, W = NT / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int each = (count + NT - 1) / NT;
  const int k0 = threadIdx.x * each < count ? threadIdx.x * each : count, k1 = k0 + each < count ? k0 + each : count;
  double own = 0.0;
  int last = -1;
  for (int k = k0; k < k1; ++k) {
    const double x = get(k);
    own += x;
    if (x > 0.0) last = k;
  }
  double incl = own;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const double o = __shfl_up(incl, s);
    if (lane >= s) incl += o;
  }
  double excl = __shfl_up(incl, 1);
  if (lane == 0) excl = 0.0;
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const int o = __shfl_xor(last, s);
    last = o > last ? o : last;
  }
  __syncthreads();
  if (lane == 63) sh.red[wave] = incl;
  if (lane == 0) sh.gone[wave] = last;
  __syncthreads();
  total = 0.0;
  last = -1;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    if (k == wave) {
      excl += total;
      incl += total;
    }
    total += sh.red[k];
    last = sh.gone[k] > last ? sh.gone[k] : last;
  }
  goal = (u > 0.0 ? u : 0.0) * total;
  const uint64_t m = __ballot(incl > goal);
  __syncthreads();
  if (lane == 0) sh.gone[wave] = m ? wave * 64 + __builtin_ctzll(m) : NT;
  __syncthreads();
  int hit = NT;
#pragma unroll
  for (int k = W - 1; k >= 0; --k) hit = sh.gone[k] < NT ? sh.gone[k] : hit;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) == hit) {
    int k = k0, found = k0;
    double run = excl, at = excl;
    for (; k < k1; ++k) {
      const double x = get(k);
      if (x > 0.0) {  // (rounding may leave the last of the thread's own as the one)
        found = k;
        at = run;
        if (run + x > goal) break;
      }
      run += x;
    }
    sh.gone[0] = found;
    sh.red[0] = at;
  }
  __syncthreads();
  int res = hit < NT ? sh.gone[0] : last;
  before = hit < NT ? sh.red[0] : __builtin_inf();  // (no border above the goal: take the last there)
  if (!(total > 0.0) || total == __builtin_inf()) res = -1;
  __syncthreads();
  return res;
}

// The workgroups of a sequence (`shares` of them) sum w over their blocks; the last finds the token.
template <bool WALKED>
__global__ __launch_bounds__(kVerifyThreads) void k_verify_pick(VerifyParams p) {
  __shared__ WalkShared sh;
  __shared__ int s_gone[kGone], s_last;
  const VerifyArgs& a = p.a;
  const int b = blockIdx.x / p.shares, share = blockIdx.x - b * p.shares;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const bool first = share == 0;
  int lo, hi;
  seq_rows(a, b, lo, hi);
  const int n = hi - lo;
  if (n == 0) {
    if (first && threadIdx.x == 0) a.kept[b] = 0;
    return;
  }
  fill_table(sh.tab);
  const double T = temperature_of(a, b), c = scale_of(T);
  Walked k;
  if constexpr (WALKED) {
    k = p.walked[b];
  } else {
    k = walk<kVerifyThreads, false>(p, sh, lo, n, T, first, [](int, double) { return 0.0; });
    if (first && threadIdx.x == 0) a.kept[b] = k.kept;
  }
  int32_t* const token = a.out_tokens + lo + k.kept - 1;
  if (!(T > 0.0)) {
    const int at = largest_of(p, lo + k.cur);
    if (first && threadIdx.x == 0) *token = at;
    return;
  }
  Weights w;
  w.p = dist_of(p, p.t, lo + k.cur, c, 64, sh.tab);
  w.al = k.al;
  w.drafted = a.draft && k.al != 0.0;
  if (w.drafted) w.q = dist_of(p, p.d, lo + k.cur, c, 64, sh.tab);
  w.ngone = 0;
  if (!a.draft && k.tried) {
    for (int r0 = k.cur + 1; r0 < n; r0 += 64) {
      const int r = r0 + lane;
      const bool child = r < n && parent_of(a, lo, r) == k.cur;
      const uint64_t m = __ballot(child);
      const int at = w.ngone + __popcll(m & ((1ull << lane) - 1));
      if (wave == 0 && child && at < kGone) s_gone[at] = a.tokens[lo + r];
      w.ngone += __popcll(m);
    }
    __syncthreads();
  }
  const int blocks = (a.V + kBlockElems - 1) / kBlockElems;
  const double u = a.uniforms[lo];
  double* const sums = p.sums + static_cast<int64_t>(b) * blocks;
  auto weights = [&](int i, double (&v)[8]) {
    weights8(p, w, i, sh.tab, v);
    if (w.ngone) {
      if (w.ngone <= kGone) {
        for (int g = 0; g < w.ngone; ++g) {
          const int x = s_gone[g];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = x == i + e ? 0.0 : v[e];
        }
      } else {
        for (int r = k.cur + 1; r < n; ++r) {
          if (parent_of(a, lo, r) != k.cur) continue;
          const int x = a.tokens[lo + r];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = x == i + e ? 0.0 : v[e];
        }
      }
    }
  };
  auto block_sum = [&](int block) {  // by a wave
    double v[8], s = 0.0;
    const int i = block * kBlockElems + 8 * lane;
    if (i < a.V) {
      weights(i, v);
      s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    return wave_sum(s);
  };
  auto sum_blocks = [&](int k0, int k1) {
    for (int block = k0 + wave; block < k1; block += kVerifyThreads / 64) {
      const double s = block_sum(block);
      if (lane == 0) __hip_atomic_store(sums + block, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __threadfence();
  };
  auto put = [&](int at, double before, double goal) {  // the token in block `at`, by the first wave
    if (wave) return;
    int res = -1;
    if (at >= 0) {
      double v[8], own = 0.0;
      const int i = at * kBlockElems + 8 * lane;
      if (i < a.V) weights(i, v);
      int last = -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (i >= a.V) v[e] = 0.0;
        own += v[e];
        if (v[e] > 0.0) last = i + e;
      }
      double incl = own;
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const double o = __shfl_up(incl, s);
        if (lane >= s) incl += o;
      }
      double run = before + (incl - own);
      int hit = 0x7fffffff;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        run += v[e];
        if (v[e] > 0.0 && run > goal && hit == 0x7fffffff) hit = i + e;
      }
#pragma unroll
      for (int s = 32; s; s >>= 1) {
        const int o = __shfl_xor(hit, s), l = __shfl_xor(last, s);
        hit = o < hit ? o : hit;
        last = l > last ? l : last;
      }
      // (none above the goal in the block where its sum passed it: rounding; the last one there)
      res = hit < 0x7fffffff && before < __builtin_inf() ? hit : last;
    }
    if (lane == 0) *token = res;
  };
  double total, before, goal;
  if (w.p.zinv != w.p.zinv || (w.drafted && w.q.zinv != w.q.zinv)) {  // no distribution
    if (first) put(-1, 0.0, 0.0);
    return;
  }
  if (!p.t.probs && !w.drafted && !w.ngone) {
    // p itself: its pieces are summed already
    if (!first) return;
    const StatPart* st = p.t.stat + static_cast<int64_t>(lo + k.cur) * p.parts;
    auto piece = [&](int i) {
      const StatPart q = st[i];
      return q.z == 0.0 ? 0.0 : q.z * add_exp2((static_cast<double>(q.top) - w.p.ref) * c, 0.0, sh.tab) * w.p.zinv;
    };
    const int at = locate(sh, p.parts, piece, u, total, before, goal);
    if (at < 0) return put(-1, 0.0, 0.0);
    const int k0 = at * p.part_blocks, k1 = k0 + p.part_blocks < blocks ? k0 + p.part_blocks : blocks;
    for (int block = k0 + wave; block < k1; block += kVerifyThreads / 64) {
      const double s = block_sum(block);
      if (lane == 0) sh.px[block - k0] = s;
    }
    __syncthreads();
    int hit = -1;
    double run = before, start = before;
    for (int i = 0; i < k1 - k0; ++i) {
      if (!(sh.px[i] > 0.0)) continue;
      hit = i;
      start = run;
      if (before < __builtin_inf() && run + sh.px[i] > goal) break;
      run += sh.px[i];
    }
    return put(hit < 0 ? -1 : k0 + hit, start, goal);
  }
  const int k0 = share * p.share_blocks < blocks ? share * p.share_blocks : blocks;
  const int k1 = k0 + p.share_blocks < blocks ? k0 + p.share_blocks : blocks;
  sum_blocks(k0, k1);
  __syncthreads();
  if (threadIdx.x == 0) s_last = __hip_atomic_fetch_add(p.tickets + b, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (s_last != p.shares - 1) return;
  __threadfence();
  auto get = [&](int i) { return __hip_atomic_load(sums + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  int at = locate(sh, blocks, get, u, total, before, goal);
  if (total == 0.0 && (w.drafted || w.ngone)) {  // nothing is left: p itself
    w.drafted = false;
    w.ngone = 0;
    sum_blocks(0, blocks);
    __syncthreads();
    at = locate(sh, blocks, get, u, total, before, goal);
  }
  put(at, before, goal);
}

// The workspace: statistics, then what the workgroups of a sequence share.
struct VerifyLayout {
  int parts, part_blocks, shares, share_blocks, blocks;
  size_t sums, tickets, walked, bytes;  // offsets
};

// Pieces of rows: as long as 4096 waves get one each, up to 16 blocks (a wave joins its sum over the lanes
// once per piece); workgroups of a sequence: 1024 in all, with a block for each wave at least.
VerifyLayout layout(int V, int B, int M, bool tprobs, bool drafted, bool dprobs) {
  VerifyLayout l{};
  l.blocks = (V + kBlockElems - 1) / kBlockElems;
  const bool drows = drafted && !dprobs;
  const int64_t rows = static_cast<int64_t>(M) * ((tprobs ? 0 : 1) + (drows ? 1 : 0));
  l.part_blocks = 16;
  while (l.part_blocks > 1 && rows * ((l.blocks + l.part_blocks - 1) / l.part_blocks) < 4096) l.part_blocks >>= 1;
  l.parts = (l.blocks + l.part_blocks - 1) / l.part_blocks;
  int shares = B > 0 ? (1024 + B - 1) / B : 1;
  if (shares > (l.blocks + 3) / 4) shares = (l.blocks + 3) / 4;
  l.share_blocks = (l.blocks + shares - 1) / shares;
  l.shares = (l.blocks + l.share_blocks - 1) / l.share_blocks;
  size_t at = static_cast<size_t>(M) * (drows ? 2 : 1) * l.parts * sizeof(StatPart);
  l.sums = at;
  at += static_cast<size_t>(B) * l.blocks * sizeof(double);
  l.walked = at;
  at += static_cast<size_t>(B) * sizeof(Walked);
  l.tickets = at;
  at += static_cast<size_t>(B) * sizeof(int);
  l.bytes = M > 0 && B > 0 ? at : 0;
  return l;
}

}  // namespace

size_t verify_workspace(int V, int B, int M, bool tprobs, bool drafted, bool dprobs) {
  return layout(V, B, M, tprobs, drafted, dprobs).bytes;
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  const VerifyLayout l = layout(a.V, a.B, a.M, a.tprobs, a.draft != nullptr, a.dprobs);
  VerifyParams p{};
  char* const ws = static_cast<char*>(a.ws);
  p.a = a;
  StatPart* const stat = reinterpret_cast<StatPart*>(ws);
  p.t = Side{static_cast<const char*>(a.target), a.tstride * (a.tdt == 0 ? 4 : 2), a.tdt, a.tprobs, stat};
  p.d = Side{static_cast<const char*>(a.draft), a.dstride * (a.ddt == 0 ? 4 : 2), a.ddt, a.dprobs,
             stat + static_cast<size_t>(a.M) * l.parts};
  p.parts = l.parts; p.part_blocks = l.part_blocks; p.shares = l.shares; p.share_blocks = l.share_blocks;
  p.sums = reinterpret_cast<double*>(ws + l.sums);
  p.tickets = reinterpret_cast<int*>(ws + l.tickets);
  p.walked = reinterpret_cast<Walked*>(ws + l.walked);
  if (a.M > 0) {
    // (rows of probabilities have statistics only where they may be greedy)
    const int first = a.tprobs && !a.temperature ? a.M : 0, end = a.draft && !a.dprobs ? 2 * a.M : a.M;
    const int64_t u0 = static_cast<int64_t>(first) * l.parts, u1 = static_cast<int64_t>(end) * l.parts;
    int64_t blocks = (u1 - u0 + 3) / 4;
    blocks = blocks < 1 ? 1 : blocks < (1 << 22) ? blocks : 1 << 22;
    hipLaunchKernelGGL(k_verify_stats, dim3(static_cast<uint32_t>(blocks)), dim3(kVerifyThreads), 0, s, p, u0, u1);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (a.M > 0 && a.draft && a.parents) {
    hipLaunchKernelGGL(k_verify_walk, dim3(a.B), dim3(kWalkThreads), 0, s, p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    hipLaunchKernelGGL(k_verify_pick<true>, dim3(a.B * l.shares), dim3(kVerifyThreads), 0, s, p);
  } else {
    hipLaunchKernelGGL(k_verify_pick<false>, dim3(a.B * l.shares), dim3(kVerifyThreads), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace tq
