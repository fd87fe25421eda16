// Verification of drafted tokens against the target's distribution (tq_verify).
//
// The walk. At row c, with target p and draft q, the children are tried in their order; after k of them
// went, what is left of p is proportional to (p - a_k q)+ with a_0 = 0, a_{k+1} = a_k + S_k, S_k = sum
// (p - a_k q)+ (S_0 = 1): if r = (p - a q)+ / S, then (r - q)+ = (p - (a + S) q)+ / S. So the state is one
// number, a, and its sum, and no distribution is ever stored. Without a draft the tried tokens are taken
// out of p one by one. Children have larger indices than their parents and are tried in ascending
// order: one ascending scan of a sequence's rows is the walk.
//
// Where a rounding matters. A test of a row's first child compares two numbers: single precision's errors
// (1e-6) matter where they are that close, and then the row is summed in fp64 (row_factors). Later siblings are tested against a small S. The new token is found at u sum(w) in the cumulative sum of w: each of
// its 10^5 borders that is off by 10^-8 gives a neighbour now and then, so w, its sums and the rows' sums
// that it is made of are fp64. The rows' sums that the first tests need, of all rows, are of exponentials
// in fp32; the passes that sum S and w sum their row once more, in fp64 (see Sums), and later siblings take that.
//
// Launches. k_verify_stats: largest value and sum of exponentials of every row of logits that can be
// looked at, a wave per piece of a row. k_verify_pick: each workgroup of a sequence joins the pieces and walks
// (all do the same: cheaper than another launch), sums w over its share of the vocabulary, and the one that
// comes last finds the token. Where siblings are tried against a draft, S is such a sum too: the last
// workgroup walks on with it, and the next launch of k_verify_pick sums what the walk needs then. kPasses - 1 more
// launches follow, in which sequences that are done end at once; what is still open in the last one its last
// workgroup sums alone (20 rows of 8 sequences, 60000 tokens: 105 us when the first launch's did so, 55 now; each sibling
// turned away behind the fourth 52 us more, 130 over 131072 tokens).
//
// Bounds and figures. 64 sequences of 9 rows, 131072 tokens in bf16, a draft: k_verify_stats reads 285 MB in 54 us,
// 5.3 TB/s, bound by memory; k_verify_pick, 30 us, reads 64 of these rows again: 5 us for the walk, 1 for the row's
// constants, 15 for the sums (8 to 10 of them vector instructions: 32 for a token of both rows, 60 more for 512), 5 for
// the meeting and the last block. One sequence of 4 rows, 32000 tokens: 14.8 us in a stream of launches, 4.6 of them launches and the rows'
// sums, about 3 the walk, 3 the sums, 1.5 until the block is found, 1.5 the token: the latency of some ten loads that
// wait for each other and of fp64 chains in waves that have a SIMD to themselves.
#include <type_traits>

#include "internal.hpp"
#include "kv_lane.hpp"

namespace tq {
namespace {

#define TQ_INLINE __attribute__((always_inline))

constexpr int kVerifyThreads = 256;
constexpr int kBlockElems = 512;    // a wave's step: 8 elements a lane
constexpr int kWindow = 256;        // rows whose probabilities are in LDS at a time
constexpr int kGone = 256;          // tried tokens in LDS
constexpr int kTable = 256;         // 2^(i / 256)
constexpr int kPieces = 32;         // pieces of a row that the lanes of a row hold at once
constexpr int kPasses = 4;          // launches of k_verify_pick for trees with a draft

// Of a piece of a row: z = sum 2^((x - top) c), c = log2(e) / T, top a value with x - top below 100 / c for every
// x. Where it holds NaN or +infinity z is NaN. Greedy rows: top the largest value, at its first index.
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

// A token may be on the wrong side of p = a q where a q is this close to p by the rows' fp32 sums (if these are off by
// more, all are), and what is summed over such tokens may be off by so much of the sum of p + a q.
constexpr double kClose = 0x1p-18, kBorder = 1e-9;

// What w is summed from. Let p~ = p P, q~ = q Q be a row's values with their own sums P, Q (2^((x - ref) c) of
// logits; probabilities as they are, P = Q = 1), and rho = a P / Q by the rows' sums of k_verify_stats, which is
// right to 1e-6. (p - a q)+ is summed over the tokens with p~ > rho q~ instead of p > a q: the ones on the
// other side add 1e-6 of themselves. So one pass gives all:
//     p = sum of p~, q = sum of q~ over those tokens, and P, Q:   sum w = p / P - a q / Q.
// Two rows that are alike nearly everywhere may have most of p on the other side. So tokens that may be there are seen
// (add gives true), and their p is summed: with how far rho was off, known with P and Q, it says whether the pass
// has to be made again.
struct Sums {
  double p, q, P, Q;
  __device__ __forceinline__ bool add(const double (&pv)[8], const double (&qv)[8], double rho) {
    bool close = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double d = __builtin_fma(-rho, qv[k], pv[k]);
      const double in = d <= 0.0 ? 0.0 : 1.0;  // (NaN goes in)
      close |= __builtin_fabs(d) < __builtin_fma(kClose, pv[k], -1e-200);  // (masked tokens, p~ of 1e-301, do not count)
      p = __builtin_fma(in, pv[k], p);
      q = __builtin_fma(in, qv[k], q);
      P += pv[k];
      Q += qv[k];
    }
    return close;
  }
};
__device__ __forceinline__ double close_to_border(const double (&pv)[8], const double (&qv)[8], double rho) {
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += __builtin_fabs(__builtin_fma(-rho, qv[k], pv[k])) < kClose * pv[k] ? pv[k] : 0.0;
  return s;
}
// Whether too much may be on the wrong side (close to the border, in 2^-30), or rho is off by more than that counts; rp,
// rq: 1 / P and 1 / Q.
__device__ __forceinline__ bool border_open(double rho, double al, double rp, double rq, uint64_t close) {
  const double off = __builtin_fabs(rho * rp - al * rq), whole = al * rq;
  return off * (static_cast<double>(close) * 0x1p-30 + kBorder / kClose) > kBorder * whole;
}
// A sequence's ticket: workgroups that have come in the upper bits, what they have close to the border in the lower
// (whole numbers: their sum does not depend on the order).
constexpr uint64_t kArrival = 1ull << 52;

// A walk that has come to a row.
struct Walk {
  double al, S;   // (without a draft al is the p of those that went, by the sums of k_verify_stats)
  double fp, fq;  // 1 / P and 1 / Q of cur by those of k_verify_stats, once its sums are made in fp64 (till then 1)
  int cur, kept, tried;  // tried: the last child of cur that went (0: none)
  int next;              // the first row that it has not looked at
  int known;             // the rows before it are in VerifyParams::rows (trees with a draft)
};
// What the walk needs of a row.
struct Dist {  // probabilities of a row of logits: 2^((x - ref) c) zinv; zinv NaN: the row is no distribution
  double ref, zinv;
};
struct RowInfo {
  double px, qx, u;   // its token's probabilities under its parent, its number
  Dist p, q;          // of its parent
  int parent, token;  // parent -1: a row that is no child of any
};
// What one launch of k_verify_pick leaves to the next.
struct Pending {
  Walk w;
  int state;  // kDone, or what has to be summed for cur: kLeft: S, kToken: w
};
enum { kDone = 0, kLeft = 1, kToken = 2 };

struct VerifyParams {
  VerifyArgs a;
  Side t, d;
  int parts, part_blocks;  // pieces of a row of logits, and kBlockElems in each
  int shares, share_blocks;  // the same of k_verify_pick's workgroups
  double* sums;            // [B][blocks][2]: Sums::p and Sums::q of a block
  Sums* totals;            // [B][shares * waves]: P and Q; p and q where S is summed
  uint64_t* tickets;       // [kPasses][B]
  Pending* pending;        // [B], and
  RowInfo* rows;           // [M], of trees with a draft
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
// The same for a type known at run time; one piece of code for all types and ends. The loads, and the values.
struct Raw8 {
  uint32_t x[8];
};
template <int DT>
__device__ __forceinline__ Raw8 load8_any(const char* row, int dt, int i, int V) {
  if (DT >= 0) dt = DT;
  Raw8 r;
  if (dt == 0 && i + 8 <= V) {
    const u32x4_a2 a = *reinterpret_cast<const u32x4_a2*>(row + static_cast<int64_t>(i) * 4);
    const u32x4_a2 b = *reinterpret_cast<const u32x4_a2*>(row + static_cast<int64_t>(i) * 4 + 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r.x[k] = a[k];
      r.x[4 + k] = b[k];
    }
  } else if (dt == 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.x[k] = reinterpret_cast<const uint32_t*>(row)[i + k < V ? i + k : V - 1];
  } else if (i + 8 <= V) {
    const u32x4_a2 a = *reinterpret_cast<const u32x4_a2*>(row + static_cast<int64_t>(i) * 2);
#pragma unroll
    for (int k = 0; k < 4; ++k) r.x[k] = a[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint16_t* const h = reinterpret_cast<const uint16_t*>(row);
      r.x[k] = h[i + 2 * k < V ? i + 2 * k : V - 1] | static_cast<uint32_t>(h[i + 2 * k + 1 < V ? i + 2 * k + 1 : V - 1]) << 16;
    }
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void values_any(const Raw8& r, int dt, int i, int V, float none, float (&f)[8]) {
  if (DT >= 0) dt = DT;
  if (dt == 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(r.x[k]);
  } else if (dt == 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(r.x[k] << 16);
      f[2 * k + 1] = __uint_as_float(r.x[k] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = half_bits_to_float(static_cast<uint16_t>(r.x[k] & 0xffffu));
      f[2 * k + 1] = half_bits_to_float(static_cast<uint16_t>(r.x[k] >> 16));
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = i + k < V ? f[k] : none;
}

// 2^(i / 256), the upper word less i << 12: adding j << 12 for any j = 256 k + i leaves 2^(j / 256).
__device__ __forceinline__ void fill_table(double* tab, uint64_t* close) {
  if (threadIdx.x == 0) *close = 0;
  for (int i = threadIdx.x; i < kTable; i += blockDim.x) {
    const double x = exp2(i * (1.0 / kTable));
    tab[i] = __hiloint2double(__double2hiint(x) - (i << 12), __double2loint(x));
  }
  __syncthreads();
}

// Exponentials: 2^t = 2^k 2^(i / 256) 2^r, |r| <= 1 / 512. Adding 1.5 2^44 rounds t to steps of 1 / 256 and leaves
// 256 k + i in the low word; 2^r = e^y by the polynomial of degree 3 with the least error on |y| <= h =
// ln 2 / 512 (y^4 / 24 replaced by its nearest of degree 2, h^2 y^2 - h^4 / 8): 2e-14 of 2^t in all.
constexpr double kMagic = 26388279066624.0;
__device__ __forceinline__ double add_pow2(double z, double r, double s, const double* tab) {
  constexpr double kLn2 = 0.69314718055994530942, kH = kLn2 / 512;
  const uint32_t j = static_cast<uint32_t>(__double2loint(z));
  double p = __builtin_fma(r, kLn2 * kLn2 * kLn2 / 6, kLn2 * kLn2 * (0.5 + kH * kH / 24));
  p = __builtin_fma(p, r, kLn2);
  p = __builtin_fma(p, r, 1.0 - kH * kH * kH * kH / 192);
  u32x2_t w = __builtin_bit_cast(u32x2_t, tab[j & (kTable - 1)]);
  w.y += j << 12;
  return __builtin_fma(__builtin_bit_cast(double, w), p, s);
}
// s + 2^t for t < 1000; t below -1000 counts as -1000, NaN too.
__device__ __forceinline__ double add_exp2(double t, double s, const double* tab) {
  t = __builtin_fmax(t, -1000.0);
  const double z = t + kMagic;
  return add_pow2(z, t - (z - kMagic), s, tab);
}

// 2^((x - ref) c) for many x: with ref c rounded to steps of 1 / 256 (a factor that every x has alike), x c
// is rounded and its step counted from ref in one fused operation. x is held above `cut`, where the
// result is about 2^-1000 (NaN stays NaN, and its result is anything). Not `ok`: a scale or a reference for
// which single precision cannot place the cut (temperatures below 1e-7 or above 1e35 or so).
struct Exp2Near {
  double c, magic, base;  // magic = 1.5 2^44 - base; base: ref c, rounded
  float cut;
  bool ok;
};
__device__ __forceinline__ Exp2Near exp2_near(double ref, double c, double reach) {  // reach = 1000 / c
  Exp2Near e;
  e.c = c;
  const double rc = ref * c;
  e.base = (rc + kMagic) - kMagic;
  e.magic = kMagic - e.base;
  e.cut = static_cast<float>(ref - reach);
  e.ok = __builtin_fabs(rc) < 0x1p27 && e.cut > -3e38f;
  return e;
}
__device__ __forceinline__ double add_exp2_near(const Exp2Near& e, float x, double s, const double* tab) {
  const double v = __builtin_elementwise_maximum(x, e.cut);
  const double z = __builtin_fma(v, e.c, e.magic);
  return add_pow2(z, __builtin_fma(v, e.c, e.magic - z), s, tab);
}

__device__ __forceinline__ double temperature_of(const VerifyArgs& a, int b) { return a.temperature ? a.temperature[b] : 1.0; }
__device__ __forceinline__ double scale_of(double T) { return 1.4426950408889634074 / T; }
__device__ __forceinline__ double reach_of(double T) { return 693.14718055994530942 * T; }  // 1000 / scale

// Over rows of 8 or 16 lanes and over the wave, in every lane, by lane moves that need no LDS (kv_lane.hpp); NaN
// where any is.
template <int LANES = 16>
__device__ __forceinline__ float row_max(float x) {
  x = __builtin_elementwise_maximum(x, kv_swap<0>(x));
  x = __builtin_elementwise_maximum(x, kv_swap<1>(x));
  x = __builtin_elementwise_maximum(x, kv_swap<2>(x));
  return LANES == 8 ? x : __builtin_elementwise_maximum(x, kv_swap<3>(x));
}
__device__ __forceinline__ float wave_max(float x) {
  float a, b;
  kv_both<4>(row_max(x), a, b);
  kv_both<5>(__builtin_elementwise_maximum(a, b), a, b);
  return __builtin_elementwise_maximum(a, b);
}
template <int LANES = 16>
__device__ __forceinline__ double row_sum(double x) {
  x += kv_swap<0>(x);
  x += kv_swap<1>(x);
  x += kv_swap<2>(x);
  return LANES == 8 ? x : x + kv_swap<3>(x);
}
__device__ __forceinline__ double wave_sum(double x) {
  double a, b;
  kv_both<4>(row_sum(x), a, b);
  kv_both<5>(a + b, a, b);
  return a + b;
}
// x and all before it, over the wave: within rows of 16 by shifts, then the rows before by broadcasts.
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double x) {
  const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(x), CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(x), CTRL, ROWS, 0xf, false);
  return x + __hiloint2double(hi, lo);
}
__device__ __forceinline__ double wave_scan(double x) {
  x = scan_step<0x111, 0xf>(x);  // row_shr:1, 2, 4, 8
  x = scan_step<0x112, 0xf>(x);
  x = scan_step<0x114, 0xf>(x);
  x = scan_step<0x118, 0xf>(x);
  x = scan_step<0x142, 0xa>(x);  // lane 15 of rows 0 and 2 to rows 1 and 3
  return scan_step<0x143, 0xc>(x);  // lane 31 to rows 2 and 3
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

// Elements [i0, i1) of a row by a wave: fp32 exponentials (a step off in 2^23, a test compares numbers that are
// off by 1e-6 then), eight at a time summed in fp32, then fp64. Relative to a value of the piece, not to
// its largest: that one need not be looked for. Two loads at a time: 54 us for 285 MB; one 56, four 55; with
// the largest value and (x - ref) c in three roundings 60.
template <int DT>
__device__ __forceinline__ StatPart stat_piece(const char* row, int V, int i0, int i1, double T) {
  const int lane = threadIdx.x & 63;
  const float inf = __builtin_inff(), c = static_cast<float>(scale_of(T));
  const bool usual = c > 1e-30f && c < 1e30f;
  float f[8], top = -inf, ref = 0.f;
  double s = 0.0;
  auto load = [&](int i, float (&f)[8]) TQ_INLINE {
    if (i + 8 <= V) load8<DT>(row, i, f);
    else load8_end<DT>(row, i, V, -inf, f);
  };
  auto most = [&](const float (&f)[8]) TQ_INLINE {
    float m = __builtin_elementwise_maximum(f[0], f[1]);
#pragma unroll
    for (int k = 2; k < 8; k += 2) m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, f[k]), f[k + 1]);
    return m;
  };
  auto sum8 = [&](const float (&e)[8]) TQ_INLINE { return ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])); };
  const int first = i0 + 8 * lane;
  bool done = first >= i1;
  if (usual && !done) {
    // relative to the lane's first eight values: x c - base is rounded once, so base may be any value near ref c
    load(first, f);
    const float m = most(f);
    const bool near = __builtin_fabsf(m) * c < 0x1p24f;
    top = near ? m : 0.f;
    const float base = top * c;
    auto sum_near = [&](const float (&f)[8]) TQ_INLINE {
      float e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(f[k], c, -base));
      return sum8(e);
    };
    s = sum_near(f);
    int i = first + kBlockElems;
    constexpr int U = 2;
    for (; i + (U - 1) * kBlockElems + 8 <= i1; i += U * kBlockElems) {
      float g[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) load8<DT>(row, i + u * kBlockElems, g[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) s += sum_near(g[u]);
    }
    for (; i < i1; i += kBlockElems) {
      load(i, f);
      s += sum_near(f);
    }
    done = s > 0x1p-100 && s < 0x1p100;
    // (in units of 2^base: of `top`)
    if (done) s *= exp2(static_cast<double>(base) - static_cast<double>(top) * c);
    ref = top;
  }
  if (!done) {
    // ... or far above them or below, or none is finite, or the temperature is extreme: relative to the largest
    top = -inf;
    for (int i = first; i < i1; i += kBlockElems) {
      load(i, f);
      top = __builtin_elementwise_maximum(top, most(f));
    }
    ref = top;
    s = 0.0;
    if (top != top || top == inf) {
      s = __builtin_nan("");
    } else if (top > -inf) {
      for (int i = first; i < i1; i += kBlockElems) {
        load(i, f);
        if (usual) {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = __builtin_amdgcn_exp2f((f[k] - ref) * c);
          s += sum8(f);
        } else {
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            const float x = load_elem<DT>(row, i + k < V ? i + k : V - 1);
            s += i + k < V && x > -inf ? exp2((static_cast<double>(x) - top) * scale_of(T)) : 0.0;
          }
        }
      }
    }
  }
  StatPart p;
  p.top = wave_max(top);
  p.at = 0;
  if (s != 0.0) s *= exp2((static_cast<double>(ref) - p.top) * scale_of(T));
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
  const VerifyArgs& a = p.a;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kPasses * a.B; i += kVerifyThreads) p.tickets[i] = 0;
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
      r = s.dt == 0 ? stat_piece<0>(x, a.V, i0, i1, T) : s.dt == 1 ? stat_piece<1>(x, a.V, i0, i1, T) : stat_piece<2>(x, a.V, i0, i1, T);
    }
    if (lane == 0) const_cast<StatPart*>(s.stat)[static_cast<int64_t>(row) * p.parts + part] = r;
  }
}

// ---- rows as distributions ------------------------------------------------------------------

__device__ __forceinline__ double probability(const Side& s, const Dist& d, double c, float x, const double* tab) {
  if (s.probs) return x;
  const double t = (x - d.ref) * c;
  return (t <= -1000.0 || x == -__builtin_inff() ? 0.0 : add_exp2(t, 0.0, tab)) * d.zinv;
}

// Row `row` of one side from its pieces, by LANES neighbouring lanes.
template <int LANES>
__device__ __forceinline__ Dist dist_of(const VerifyParams& p, const Side& s, int row, double c, const double* tab) {
  Dist d{0.0, 1.0};
  if (s.probs) return d;
  static_assert(LANES == 8 || LANES == 16 || LANES == 64, "rows of lanes, or the wave");
  constexpr int HELD = kPieces / (LANES == 64 ? 16 : LANES);
  const StatPart* st = s.stat + static_cast<int64_t>(row) * p.parts;
  const int l = threadIdx.x & (LANES - 1);
  const float inf = __builtin_inff();
  StatPart held[HELD];
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    held[k] = StatPart{0.0, -inf, 0};
    if (l + k * LANES < p.parts) held[k] = st[l + k * LANES];
  }
  float top = -inf;
#pragma unroll
  for (int k = 0; k < HELD; ++k) top = __builtin_elementwise_maximum(top, held[k].top);
  for (int k = l + HELD * LANES; k < p.parts; k += LANES) top = __builtin_elementwise_maximum(top, st[k].top);
  top = LANES < 64 ? row_max<LANES>(top) : wave_max(top);
  double z = 0.0;
#pragma unroll
  for (int k = 0; k < HELD; ++k) {
    const double f = add_exp2((static_cast<double>(held[k].top) - top) * c, 0.0, tab);
    z += held[k].z == 0.0 ? 0.0 : held[k].z * f;
  }
  for (int k = l + HELD * LANES; k < p.parts; k += LANES) {
    const StatPart q = st[k];
    if (q.z != 0.0) z += q.z * add_exp2((static_cast<double>(q.top) - top) * c, 0.0, tab);
  }
  z = LANES < 64 ? row_sum<LANES>(z) : wave_sum(z);
  d.ref = top;
  d.zinv = z > 0.0 && z < __builtin_inf() ? 1.0 / z : __builtin_nan("");
  return d;
}

// The first largest value of a greedy row: its index, or -1. By a wave.
__device__ __forceinline__ int largest_of(const VerifyParams& p, int row) {
  const StatPart* st = p.t.stat + static_cast<int64_t>(row) * p.parts;
  const int lane = threadIdx.x & 63;
  float top = -__builtin_inff();
  int at = 0x7fffffff;
  bool bad = false;
  for (int k = lane; k < p.parts; k += 64) {  // (ascending: the first of equal ones stays)
    const StatPart q = st[k];
    bad |= q.z != 0.0;
    if (q.top > top) {
      top = q.top;
      at = q.at;
    }
  }
  const float most = wave_max(top);
  if (top != most) at = 0x7fffffff;
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const int o = __shfl_xor(at, s);
    at = o < at ? o : at;
  }
  return __ballot(bad) || !(most > (p.t.probs ? 0.f : -__builtin_inff())) ? -1 : at;
}

// ---- weights ----------------------------------------------------------------------------------

// Weights up to here count as nothing: masked tokens come out as about 2^-1000, not 0.
constexpr double kNothing = 1e-280;
// So much left of p, or less, is nothing: the rounding of the sums of p and of a q, ten times over. Sums of 10^5 terms
// are off by 10^-15 or so, of logits the exponentials by 2 10^-14 too, and by 2^-52 of the exponent.
__device__ __forceinline__ double little(bool probs) { return probs ? 1e-14 : 1e-12; }
// With less left than this the tokens that the rows' fp32 sums put on the wrong side of p = a q (10^-6 of them) may
// matter: the sums are made once more, with P and Q as they were found (a sequence comes here as often as that).
constexpr double kAgain = 1e-4;

// So close, relative to what they are made of, two numbers may be for the rows' fp32 sums to tell them apart (2.6e-5
// for both sides together).
constexpr double kNear = 3e-5;

__device__ __forceinline__ bool near_border(double l, double r) {  // (single precision is enough to see it)
  const float x = static_cast<float>(l), y = static_cast<float>(r);
  return __builtin_fabsf(x - y) < static_cast<float>(kNear) * (x + y);
}

// One side of what the new token is drawn from (or S is summed over): values p~ of Sums.
struct WeightSide {
  const char* row;
  Dist d;
  Exp2Near e;
  double inv;  // 1 / P by k_verify_stats (probabilities: 1)
};
struct Weights {
  WeightSide p, q;
  double c;
};

// A value that all lanes hold, in scalar registers.
__device__ __forceinline__ double uniform(double x) {
  return __hiloint2double(__builtin_amdgcn_readfirstlane(__double2hiint(x)), __builtin_amdgcn_readfirstlane(__double2loint(x)));
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ Walk uniform(const Walk& w) {
  return Walk{uniform(w.al), uniform(w.S), uniform(w.fp), uniform(w.fq), uniform(w.cur), uniform(w.kept), uniform(w.tried), uniform(w.next), uniform(w.known)};
}

__device__ __forceinline__ WeightSide weight_side(const Side& s, int row, const Dist& d, double T, const double* tab) {
  WeightSide w;
  const double c = scale_of(T);
  w.row = s.data + row * s.stride;
  w.d = Dist{uniform(d.ref), uniform(d.zinv)};
  w.e = exp2_near(w.d.ref, c, reach_of(T));
  w.inv = uniform(s.probs ? 1.0 : w.e.ok ? d.zinv * add_exp2(w.e.base - d.ref * c, 0.0, tab) : d.zinv);
  w.e.c = uniform(c);
  w.e.base = uniform(w.e.base);
  w.e.magic = uniform(w.e.magic);
  w.e.cut = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(w.e.cut)));
  w.e.ok = __builtin_amdgcn_readfirstlane(w.e.ok);
  return w;
}

template <int DT>
__device__ __forceinline__ void values8(const Side& s, const WeightSide& w, const Raw8& raw, double c, int i, int V, const double* tab,
                                               double (&v)[8]) {
  float f[8];
  values_any<DT>(raw, s.dt, i, V, s.probs ? 0.f : -__builtin_inff(), f);
  if (s.probs) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = f[k];
  } else if (w.e.ok) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = add_exp2_near(w.e, f[k], 0.0, tab);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = f[k] == -__builtin_inff() ? 0.0 : add_exp2((f[k] - w.d.ref) * c, 0.0, tab);
    }
  }
}

// ---- the walk -----------------------------------------------------------------------------

struct WalkShared {
  RowInfo row[kWindow];
  double tab[kTable], red[4 * 16];
  uint64_t close;
  int pick[32];
};

template <bool TREE>
__device__ __forceinline__ int parent_of(const VerifyArgs& a, int lo, int r) { return TREE ? a.parents[lo + r] : r - 1; }

// Whether a child of cur before row `end` has token x, by all lanes of a wave.
__device__ __forceinline__ bool tried_before(const VerifyArgs& a, const WalkShared& sh, int lo, int n, int cur, int end, int x) {
  const int lane = threadIdx.x & 63;
  bool found = false;
  for (int r = cur + 1; r < end && !found; r += 64) {
    const int i = r + lane;
    bool hit = false;
    if (i < end) hit = n <= kWindow ? sh.row[i].parent == cur && sh.row[i].token == x : parent_of<true>(a, lo, i) == cur && a.tokens[lo + i] == x;
    found = __ballot(hit) != 0;
  }
  return found;
}

// Rows [w0, w1) into LDS: their tokens' probabilities under their parents, some lanes a row (trees, which have
// more rows, 8: 24 rows at once; 8 trees of these 21.7 -> 20.6 us). kept: where a
// launch before has left them (load), or where they are left for the next (null: not).
template <bool TREE, bool DRAFT>
__device__ __forceinline__ void fill_window(const VerifyParams& p, WalkShared& sh, int lo, int w0, int w1, double T, RowInfo* kept,
                                            bool load) {
  const VerifyArgs& a = p.a;
  const bool greedy = !(T > 0.0), drafted = DRAFT && !greedy;
  const double c = scale_of(T);
  constexpr int LANES = TREE ? 8 : 16;
  if (load) {
    for (int r = w0 + static_cast<int>(threadIdx.x); r < w1; r += kVerifyThreads) sh.row[r - w0] = kept[lo + r];
  } else {
    for (int r = w0 + static_cast<int>(threadIdx.x) / LANES; r < w1; r += kVerifyThreads / LANES) {
      const int up = parent_of<TREE>(a, lo, r), x = a.tokens[lo + r];
      const float u = a.uniforms[lo + r];
      const bool any = r > 0 && up >= 0 && up < r && x >= 0 && x < a.V;
      RowInfo i{0.0, 0.0, u, {0.0, 1.0}, {0.0, 1.0}, any ? up : -1, x};
      if (any && !greedy) {
        const float xt = load_any(p.t.data + (lo + up) * p.t.stride, p.t.dt, x);
        float xd = 0.f;
        if (drafted) xd = load_any(p.d.data + (lo + up) * p.d.stride, p.d.dt, x);
        i.p = dist_of<LANES>(p, p.t, lo + up, c, sh.tab);
        i.px = probability(p.t, i.p, c, xt, sh.tab);
        if (!(i.px < __builtin_inf())) i.px = __builtin_nan("");  // no distribution: it stays under no number
        if (drafted) {
          i.q = dist_of<LANES>(p, p.d, lo + up, c, sh.tab);
          i.qx = probability(p.d, i.q, c, xd, sh.tab);
        }
      }
      if ((threadIdx.x & (LANES - 1)) == 0) {
        sh.row[r - w0] = i;
        if (kept) kept[lo + r] = i;
      }
    }
  }
  __syncthreads();
}

// 1 / P and 1 / Q of the row that `r` follows by sums of fp64 exponentials, relative to those of k_verify_stats; by all
// threads of the workgroup, in every workgroup of the sequence. For a test that the rows' fp32 sums cannot decide: one
// in some 10^4 (65 us over 131072 tokens; four loads together instead of one 48, and 0.3 us more where none is made), and
// where siblings that went have left little of p.
template <bool DRAFT, int DT>
__device__ __forceinline__ void row_factors(const VerifyParams& p, WalkShared& sh, int row, const RowInfo& r, double T, double& fp,
                                            double& fq) {
  fp = fq = 1.0;
#pragma unroll 1
  for (int side = 0; side < (DRAFT ? 2 : 1); ++side) {
    const Side& s = side ? p.d : p.t;
    if (s.probs) continue;
    const Dist d = side ? r.q : r.p;
    const char* const x = s.data + row * s.stride;
    double sum = 0.0;
    for (int i = 8 * static_cast<int>(threadIdx.x); i < p.a.V; i += 8 * kVerifyThreads) {
      float f[8];
      values_any<DT>(load8_any<DT>(x, s.dt, i, p.a.V), s.dt, i, p.a.V, -__builtin_inff(), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = add_exp2((f[k] - d.ref) * scale_of(T), sum, sh.tab);
    }
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) sh.red[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = (sh.red[0] + sh.red[1]) + (sh.red[2] + sh.red[3]);
    __syncthreads();
    (side ? fq : fp) = 1.0 / (sum * d.zinv);
  }
}

// Walks on, all waves of the workgroup alike, until S of cur is needed (true) or no child stays (false).
// `writes`: this workgroup writes the tokens that stay. held: the window in LDS, -1 for none. later: not the first launch.
template <bool TREE, bool DRAFT, int DT>
__device__ __forceinline__ bool walk(const VerifyParams& p, WalkShared& sh, int lo, int n, double T, bool writes, Walk& w, int& held,
                                     bool later) {
  constexpr bool SUMS = TREE && DRAFT;
  const VerifyArgs& a = p.a;
  const int lane = threadIdx.x & 63;
  const bool greedy = !(T > 0.0), drafted = DRAFT && !greedy;
  const bool sums = !p.t.probs || (drafted && !p.d.probs);  // tests are made with rows' sums
  int largest = greedy ? largest_of(p, lo + w.cur) : -1;
  while (w.next < n) {
    const int w0 = w.next / kWindow * kWindow, w1 = n - w0 < kWindow ? n : w0 + kWindow;
    if (held != w0) {
      if (held >= 0) __syncthreads();
      fill_window<TREE, DRAFT>(p, sh, lo, w0, w1, T, SUMS && (later || writes) ? p.rows : nullptr, SUMS && later && w0 < w.known);
      held = w0;
      if (w.known < w1) w.known = w1;
    }
    if (!TREE && !greedy) {
      // A chain: no test depends on another's, so 64 rows at a time (nine rows that stay one by one: 7 us).
      for (int sure = 0;;) {  // the rows up to `sure` that are near their border have exact numbers
        const int i = w.next + lane;
        bool row = false, yes = false, near = false;
        int x = 0;
        if (i < w1) {
          const RowInfo& f = sh.row[i - w0];
          x = f.token;
          row = f.parent >= 0;
          const double l = drafted ? f.u * f.qx : f.u;
          yes = row && l < f.px;
          near = row && i > sure && near_border(l, f.px);
        }
        const uint64_t m = ~__ballot(yes);
        const int run = m ? __builtin_ctzll(m) : 64;
        const uint64_t open = __ballot(near) & (run < 63 ? (2ull << run) - 1 : ~0ull);
        if (__builtin_expect(open && sums, 0)) {  // the first of them that the walk comes to
          sure = w.next + __builtin_ctzll(open);
          RowInfo& f = sh.row[sure - w0];
          double fp, fq;
          row_factors<DRAFT, DT>(p, sh, lo + sure - 1, f, T, fp, fq);
          if (threadIdx.x == 0) {  // (all waves have read it: row_factors waits for them)
            f.px *= fp;
            f.qx *= fq;
          }
          __syncthreads();
          continue;
        }
        if (writes && threadIdx.x < 64 && lane < run) {
          a.out_tokens[lo + w.kept - 1 + lane] = x;
          a.path[lo + w.kept + lane] = i;
        }
        w.kept += run;
        w.next += run;
        w.cur = w.next - 1;
        if (run == 64 && w.next < w1) continue;
        if (w.next < w1) {
          if (__ballot(row) >> run & 1) {
            w.tried = w.next;
            w.al = 1.0;
            if (!DRAFT) w.S -= sh.row[w.next - w0].px;
          }
          w.next = n;
        }
        break;
      }
      continue;
    }
    // the next child of cur in the window
    int r = w1;
    for (int i = w.next; i < w1; i += 64) {
      const uint64_t m = __ballot(i + lane < w1 && sh.row[i + lane - w0].parent == w.cur);
      if (m) {
        r = i + __builtin_ctzll(m);
        break;
      }
    }
    w.next = r;
    if (r == w1) continue;
    w.next = r + 1;
    const RowInfo& row = sh.row[r - w0];
    const int x = row.token;
    // (where siblings have gone S may be as small as the rows' sums are off)
    const double u = row.u;
    double px = row.px * w.fp, qx = row.qx * w.fq;
    bool yes, taken = false;
    if (greedy) {
      yes = x == largest;
    } else if (drafted) {
      if (__builtin_expect(sums && w.al == 0.0 && near_border(u * qx, px), 0)) {
        row_factors<DRAFT, DT>(p, sh, lo + w.cur, row, T, w.fp, w.fq);
        px = row.px * w.fp;
        qx = row.qx * w.fq;
      }
      yes = w.S > 0.0 && u * w.S * qx < px - w.al * qx;  // (nothing left: the difference is rounding)
    } else {
      taken = TREE && w.tried && tried_before(a, sh, lo, n, w.cur, r, x);
      if (__builtin_expect(sums && w.fp == 1.0 && !taken && __builtin_fabs(u * w.S - px) < kNear * (u * w.al + px), 0)) {
        row_factors<DRAFT, DT>(p, sh, lo + w.cur, row, T, w.fp, w.fq);
        px = row.px * w.fp;
        w.S = 1.0 - w.al * w.fp;
      }
      yes = !taken && u * w.S < px;
    }
    if (yes) {
      if (writes && threadIdx.x == 0) {
        a.out_tokens[lo + w.kept - 1] = x;
        a.path[lo + w.kept] = r;
      }
      w = Walk{0.0, 1.0, 1.0, 1.0, r, w.kept + 1, 0, r + 1, w.known};
      if (greedy) largest = largest_of(p, lo + r);
    } else {
      w.tried = r;
      if (!TREE) {  // a chain has no siblings
        w.next = n;
      } else if (drafted) {
        w.al += w.S;
        // (S is of use only if another child follows)
        bool more = false;
        for (int i = r + 1; i < n && !more; i += 64) more = __ballot(i + lane < n && parent_of<TREE>(a, lo, i + lane) == w.cur) != 0;
        if (more) return true;
      } else if (!taken) {
        w.S -= px;
        w.al += row.px;
      }
    }
  }
  return false;
}

// ---- the new token ----------------------------------------------------------------------------

// What other workgroups have written, from where it was written through to.
__device__ __forceinline__ double shared_load(const double* x) {
  return __hip_atomic_load(x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The block that the new token is in, from the blocks' sums, by all threads of the workgroup.
struct Found {
  int at;          // the first block that takes the cumulative sum above goal; the last with weight if
                   // there is none (before = infinity then); -1 if nothing is left
  double total, goal, before;  // sum of all, u of it, sum before the block
  double rp, rq;   // 1 / P, 1 / Q
};
template <bool DRAFT>
__device__ __forceinline__ Found locate(WalkShared& sh, const double* sums, int blocks, const Sums* totals, int ntotals, bool drafted,
                                        bool plogits, bool qlogits, double al, double u) {
  constexpr int NT = kVerifyThreads, W = NT / 64;
  drafted = DRAFT && drafted;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int each = (blocks + NT - 1) / NT;
  const int k0 = static_cast<int>(threadIdx.x) * each < blocks ? threadIdx.x * each : blocks, k1 = k0 + each < blocks ? k0 + each : blocks;
  // (all first loads before any wait; a thread with one block does not read it again)
  Sums s{};
  if (k0 < k1) s.p = shared_load(sums + 2 * k0);
  if (drafted) {
    const int t = threadIdx.x;
    if (k0 < k1) s.q = shared_load(sums + 2 * k0 + 1);
    if (t < ntotals) s.P = shared_load(&totals[t].P);
    if (t < ntotals) s.Q = shared_load(&totals[t].Q);
    for (int k = t + NT; k < ntotals; k += NT) {
      s.P += shared_load(&totals[k].P);
      s.Q += shared_load(&totals[k].Q);
    }
  }
  for (int k = k0 + 1; k < k1; ++k) {
    s.p += shared_load(sums + 2 * k);
    if (drafted) s.q += shared_load(sums + 2 * k + 1);
  }
  const double ip = wave_scan(s.p);
  double iq = 0.0;
  if (drafted) {
    iq = wave_scan(s.q);
    s.P = wave_sum(s.P);
    s.Q = wave_sum(s.Q);
  }
  if (lane == 63) {
    sh.red[4 * wave] = ip;
    sh.red[4 * wave + 1] = iq;
    sh.red[4 * wave + 2] = s.P;
    sh.red[4 * wave + 3] = s.Q;
  }
  __syncthreads();
  Sums all{}, left{};  // of all threads, of the waves before
#pragma unroll
  for (int k = 0; k < W; ++k) {
    if (k == wave) left = all;
    all.p += sh.red[4 * k];
    all.q += sh.red[4 * k + 1];
    all.P += sh.red[4 * k + 2];
    all.Q += sh.red[4 * k + 3];
  }
  Found f;
  f.rp = drafted && plogits ? 1.0 / all.P : 1.0;
  f.rq = drafted && qlogits ? 1.0 / all.Q : 1.0;
  auto weight = [&](double p, double q) TQ_INLINE { return p * f.rp - al * (q * f.rq); };
  f.total = weight(all.p, all.q);
  f.goal = (u > 0.0 ? u : 0.0) * f.total;
  // a block's own weight; rounding may leave a block of nothing a little
  auto block = [&](int k) TQ_INLINE {
    const double x = each == 1 ? weight(s.p, s.q) : weight(shared_load(sums + 2 * k), drafted ? shared_load(sums + 2 * k + 1) : 0.0);
    return x <= kNothing ? 0.0 : x;
  };
  const uint64_t m = __ballot(weight(left.p + ip, left.q + iq) > f.goal);
  if (lane == 0) sh.pick[wave] = m ? wave * 64 + __builtin_ctzll(m) : NT;
  __syncthreads();
  int hit = NT;
#pragma unroll
  for (int k = W - 1; k >= 0; --k) hit = sh.pick[k] < NT ? sh.pick[k] : hit;
  if (static_cast<int>(threadIdx.x) == hit) {
    int found = -1;
    double run = weight(left.p + (ip - s.p), left.q + (iq - s.q)), at = run;
    for (int k = k0; k < k1; ++k) {
      const double x = block(k);
      if (x > 0.0) {  // (rounding may leave the last of the thread's own as the one)
        found = k;
        at = run;
        if (run + x > f.goal) break;
      }
      run += x;
    }
    sh.pick[W] = found;
    sh.red[4 * W] = at;
  }
  __syncthreads();
  f.at = hit < NT ? sh.pick[W] : -1;
  f.before = sh.red[4 * W];
  __syncthreads();
  if (f.at < 0) {
    f.before = __builtin_inf();
    int last = -1;
    for (int k = k0; k < k1; ++k)
      if (block(k) > 0.0) last = k;
#pragma unroll
    for (int k = 32; k; k >>= 1) {
      const int o = __shfl_xor(last, k);
      last = o > last ? o : last;
    }
    if (lane == 0) sh.pick[wave] = last;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) f.at = sh.pick[k] > f.at ? sh.pick[k] : f.at;
    __syncthreads();
  }
  return f;
}

// The workgroups of a sequence (`shares` of them) sum w over their blocks; the last finds the token, or walks on.
// Trees with a draft take several launches. Chains, trees, drafts and the rows' type (DT, as in load_elem; -1: two
// of them) are told apart at compile time: a wave that has a SIMD to itself pays for every branch and spilled
// register (one sequence of 4 rows 14.0 us, 14.9 with all of it in one kernel; 8 trees of 24 rows 20.3, 23.6; 64
// sequences of 9 rows 80.5, 84.5; before tests near their border were made again). Trees with a draft want 200 registers: at three waves a SIMD they spilled (8
// sequences of 20 rows 61 us a call against 57).
template <bool TREE, bool DRAFT, int DT>
__global__ __launch_bounds__(kVerifyThreads, TREE && DRAFT ? 2 : 3) void k_verify_pick(VerifyParams p, int pass, int passes) {
  constexpr bool SUMS = TREE && DRAFT;
  __shared__ WalkShared sh;
  __shared__ int s_gone[kGone];
  __shared__ uint64_t s_ticket;
  const VerifyArgs& a = p.a;
  const int b = blockIdx.x / p.shares, share = blockIdx.x - b * p.shares;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  bool writes = share == 0;  // this workgroup writes outputs
  Pending st;
  if (SUMS && pass) {
    st = p.pending[b];
    if (st.state == kDone) return;
  }
  int lo, hi;
  const float temperature = a.temperature ? a.temperature[b] : 1.f;
  seq_rows(a, b, lo, hi);
  fill_table(sh.tab, &sh.close);  // (while these are on their way)
  const int n = hi - lo;
  if (n == 0) {
    if (writes && threadIdx.x == 0) {
      a.kept[b] = 0;
      if (SUMS) p.pending[b].state = kDone;
    }
    return;
  }
  const double T = uniform(static_cast<double>(temperature)), nothing = little(p.t.probs && p.d.probs);
  const float u = a.uniforms[lo];
  int held = -1;
  if (!SUMS || !pass) st.w = Walk{0.0, 1.0, 1.0, 1.0, 0, 1, 0, 1, 0};
  if constexpr (!SUMS) {
    walk<TREE, DRAFT, DT>(p, sh, lo, n, T, writes, st.w, held, false);
    st.w = uniform(st.w);
    st.state = kToken;
  }
  const int blocks = (a.V + kBlockElems - 1) / kBlockElems, ntotals = p.shares * (kVerifyThreads / 64);
  double* const sums = p.sums + 2 * static_cast<int64_t>(b) * blocks;
  Sums* const totals = p.totals + static_cast<int64_t>(b) * ntotals;
  int k0 = share * p.share_blocks < blocks ? share * p.share_blocks : blocks;
  int k1 = k0 + p.share_blocks < blocks ? k0 + p.share_blocks : blocks;
  bool alone = false;              // the others have ended
  bool walks = SUMS && !pass, fresh = true;  // to walk on; to begin with the row that the walk has come to
  bool drafted = false, exact = false;  // exact: rho is made of sums in fp64
  int ngone = 0;
  double al = 0.0, rho = 0.0;
  Weights w;
  Found f{-1, 0.0, 0.0, 0.0, 1.0, 1.0};
  double pv[8], qv[8];
  // Begins with the row that the walk has come to; false: the token needs no sums, and is written.
  auto begin = [&]() TQ_INLINE {
    al = DRAFT ? st.w.al : 0.0;
    int res = -2;  // a token that needs no sums
    if (st.state == kToken) {
      if (writes) {
        for (int i = st.w.kept + threadIdx.x; i < n; i += kVerifyThreads) {
          a.out_tokens[lo + i] = -1;
          a.path[lo + i] = -1;
        }
        if (threadIdx.x == 0) {
          a.path[lo] = 0;
          a.kept[b] = st.w.kept;
        }
      }
      if (!(T > 0.0)) res = largest_of(p, lo + st.w.cur);
    }
    const int row = lo + st.w.cur;
    w.c = scale_of(T);
    drafted = DRAFT && al != 0.0;
    Dist dp, dq{0.0, 1.0};
    if (res == -2) {
      if (st.w.tried && held == 0 && n <= kWindow) {  // (the last child's parent is this row)
        dp = sh.row[st.w.tried].p;
        dq = sh.row[st.w.tried].q;
      } else if (SUMS && pass && st.w.tried) {
        dp = p.rows[lo + st.w.tried].p;
        dq = p.rows[lo + st.w.tried].q;
      } else {
        dp = dist_of<64>(p, p.t, row, w.c, sh.tab);
        if (drafted) dq = dist_of<64>(p, p.d, row, w.c, sh.tab);
      }
      // no distribution: of logits, or a tried token's probability (with a draft w has it too)
      if (st.state == kToken && (dp.zinv != dp.zinv || (drafted && dq.zinv != dq.zinv) || (!DRAFT && st.w.S != st.w.S))) res = -1;
    }
    if (res != -2) {
      if (writes && threadIdx.x == 0) {
        a.out_tokens[lo + st.w.kept - 1] = res;
        if (SUMS) p.pending[b].state = kDone;
      }
      return false;
    }
    w.p = weight_side(p.t, row, dp, T, sh.tab);
    w.q = w.p;
    if (drafted) w.q = weight_side(p.d, row, dq, T, sh.tab);
    rho = al * (w.q.inv / w.p.inv);
    if (SUMS) rho *= st.w.fq / st.w.fp;
    exact = (p.t.probs || st.w.fp != 1.0) && (p.d.probs || st.w.fq != 1.0);
    // tokens that were taken out of p
    ngone = 0;
    if (!DRAFT && st.w.tried) {
      for (int r0 = st.w.cur + 1; r0 < n; r0 += 64) {
        const int r = r0 + lane;
        const bool child = r < n && parent_of<TREE>(a, lo, r) == st.w.cur;
        const uint64_t m = __ballot(child);
        const int at = ngone + __popcll(m & ((1ull << lane) - 1));
        if (wave == 0 && child && at < kGone) s_gone[at] = a.tokens[lo + r];
        ngone += __popcll(m);
      }
      __syncthreads();
    }
    return true;
  };
  if constexpr (!SUMS)
    if (!begin()) return;
  // The same loop sums blocks and, at last, looks at the block that the token is in: the code is in the
  // instruction cache then, where a copy of it took 2 us to come.
  for (;;) {
    if (SUMS && walks) {
      st.state = walk<TREE, DRAFT, DT>(p, sh, lo, n, T, writes, st.w, held, pass > 0) ? kLeft : kToken;
      st.w = uniform(st.w);
      walks = false;
      fresh = true;
      if (alone && pass + 1 < passes) {  // the next launch goes on
        if (threadIdx.x == 0) p.pending[b] = st;
        return;
      }
    }
    if (SUMS && fresh) {
      fresh = false;
      if (!begin()) return;
    }
    Sums s{}, all{};
    for (int block = k0 + wave; block < k1; block += kVerifyThreads / 64) {
      const int i = block * kBlockElems + 8 * lane;
      s.p = s.q = 0.0;
      bool close = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) pv[e] = qv[e] = 0.0;
      if (i < a.V) {
        const Raw8 praw = load8_any<DT>(w.p.row, p.t.dt, i, a.V);
        Raw8 qraw{};
        if (drafted) qraw = load8_any<DT>(w.q.row, p.d.dt, i, a.V);
        values8<DT>(p.t, w.p, praw, w.c, i, a.V, sh.tab, pv);
        if (drafted) values8<DT>(p.d, w.q, qraw, w.c, i, a.V, sh.tab, qv);
        // (more of them than LDS holds: looked for among the rows again)
        const int g0 = ngone <= kGone ? 0 : st.w.cur + 1, g1 = ngone <= kGone ? ngone : n;
        for (int g = g0; g < g1; ++g) {
          const int x = ngone <= kGone ? s_gone[g] : parent_of<TREE>(a, lo, g) == st.w.cur ? a.tokens[lo + g] : -1;
#pragma unroll
          for (int e = 0; e < 8; ++e) pv[e] = x == i + e ? 0.0 : pv[e];
        }
        if (f.at >= 0) break;
        if (drafted) {
          close = s.add(pv, qv, rho);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) s.p += pv[e] < 0.0 ? 0.0 : pv[e];
        }
      }
      if (f.at >= 0) break;
      if (DRAFT && __builtin_expect(__ballot(close) != 0, 0)) {
        const double x = __builtin_fmin(wave_sum(close_to_border(pv, qv, rho)) * w.p.inv, 1.0);
        if (lane == 0) __hip_atomic_fetch_add(&sh.close, static_cast<uint64_t>(x * 0x1p30) + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      }
      if (SUMS && st.state == kLeft) {
        all.p += s.p;
        all.q += s.q;
        continue;
      }
      const double ps = wave_sum(s.p);
      if (lane == 0) __hip_atomic_store(sums + 2 * block, ps <= kNothing ? 0.0 : ps, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (drafted) {
        const double qs = wave_sum(s.q);
        if (lane == 0) __hip_atomic_store(sums + 2 * block + 1, qs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (f.at >= 0) break;
    if (drafted) {
      all = Sums{wave_sum(all.p), wave_sum(all.q), wave_sum(s.P), wave_sum(s.Q)};
      // (a workgroup alone: the others' are nothing)
      for (int k = alone ? wave : share * (kVerifyThreads / 64) + wave; k < ntotals; k += kVerifyThreads / 64) {
        if (lane == 0) {
          __hip_atomic_store(&totals[k].p, all.p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(&totals[k].q, all.q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(&totals[k].P, all.P, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(&totals[k].Q, all.Q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        all = Sums{};
        if (!alone) break;
      }
    }
    // The sums are written through to where every XCD sees them, and read from there: the wave waits
    // for its stores before it meets the others, and no cache has to be written back (a release fence
    // does that, for the whole L2: 90 us more in the largest batch).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (!alone) {
      if (threadIdx.x == 0) {
        const uint64_t mine = kArrival + (DRAFT ? sh.close : 0);
        s_ticket = mine + __hip_atomic_fetch_add(p.tickets + pass * a.B + b, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (DRAFT) sh.close = s_ticket & (kArrival - 1);
      }
      __syncthreads();
      if (s_ticket / kArrival != static_cast<uint32_t>(p.shares)) return;
      alone = writes = true;
      k0 = 0;
      k1 = blocks;
    }
    if (SUMS && st.state == kLeft) {
      // S, by every wave for itself
      Sums t{};
      for (int k = lane; k < ntotals; k += 64) {
        t.p += shared_load(&totals[k].p);
        t.q += shared_load(&totals[k].q);
        t.P += shared_load(&totals[k].P);
        t.Q += shared_load(&totals[k].Q);
      }
      const uint64_t close = sh.close;
      __syncthreads();  // (they may be written again)
      if (threadIdx.x == 0) sh.close = 0;
      t = Sums{wave_sum(t.p), wave_sum(t.q), wave_sum(t.P), wave_sum(t.Q)};
      if (!p.t.probs) st.w.fp = 1.0 / (t.P * w.p.inv);
      if (!p.d.probs) st.w.fq = 1.0 / (t.Q * w.q.inv);
      const double left = (p.t.probs ? t.p : t.p / t.P) - al * (p.d.probs ? t.q : t.q / t.Q);
      __syncthreads();
      if (!exact && (left < kAgain || border_open(rho, al, st.w.fp * w.p.inv, st.w.fq * w.q.inv, close))) {
        exact = true;
        rho = al * ((w.q.inv * st.w.fq) / (w.p.inv * st.w.fp));
        continue;
      }
      st.w.S = left < nothing ? 0.0 : left;
      walks = true;
      continue;
    }
    f = locate<DRAFT>(sh, sums, blocks, totals, ntotals, drafted, !p.t.probs, !p.d.probs, al, u);
    if (DRAFT && drafted && !exact && (f.total < kAgain || border_open(rho, al, f.rp, f.rq, sh.close))) {
      exact = true;
      rho = al * (f.rq / f.rp);
      f.at = -1;
      continue;
    }
    if ((drafted && f.total < nothing) || (ngone && f.total == 0.0)) {
      // nothing is left, or no more than the rounding of the rows' sums: p itself, by this workgroup
      f.at = -1;
      drafted = false;
      ngone = 0;
      continue;
    }
    if (SUMS && threadIdx.x == 0) p.pending[b].state = kDone;
    if (f.at < 0 || !(f.total > 0.0) || f.total == __builtin_inf()) {
      if (threadIdx.x == 0) a.out_tokens[lo + st.w.kept - 1] = -1;
      return;
    }
    k0 = f.at;
    k1 = f.at + 1;
  }
  if (wave) return;
  double own = 0.0;
  const int i = f.at * kBlockElems + 8 * lane;
  int last = -1;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double x = drafted ? pv[e] * f.rp - al * (qv[e] * f.rq) : pv[e];
    pv[e] = x <= kNothing ? 0.0 : x;
    own += pv[e];
    if (pv[e] > 0.0) last = i + e;
  }
  double run = f.before + (wave_scan(own) - own);
  int hit = 0x7fffffff;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    run += pv[e];
    if (pv[e] > 0.0 && run > f.goal && hit == 0x7fffffff) hit = i + e;
  }
#pragma unroll
  for (int s = 32; s; s >>= 1) {
    const int o = __shfl_xor(hit, s), l = __shfl_xor(last, s);
    hit = o < hit ? o : hit;
    last = l > last ? l : last;
  }
  // (none above the goal in the block where its sum passed it: rounding; the last one there)
  if (lane == 0) a.out_tokens[lo + st.w.kept - 1] = hit < 0x7fffffff && f.before < __builtin_inf() ? hit : last;
}

// The workspace: statistics, then what the workgroups of a sequence share.
struct VerifyLayout {
  int parts, part_blocks, shares, share_blocks, blocks;
  size_t sums, totals, tickets, pending, rows, bytes;  // offsets
};

// Pieces of rows: as long as 4096 waves get one each, up to 16 blocks (a wave joins its sum over the lanes
// once per piece), and of no more than kPieces to a row, which its lanes join without a loop (256 of them took
// the walk of 8 rows 17 us instead of 4). Workgroups of a sequence: 768 in all, three to a CU, with a block for each wave
// at least (200 sequences of 5 rows of 32000: 55.0 us, 58.7 with 1024, 55.9 with 512; 64 of 9 of 131072: 84.5, 84.5, 85.6;
// before the kernels were told apart).
VerifyLayout layout(int V, int B, int M, bool tprobs, bool drafted, bool dprobs) {
  VerifyLayout l{};
  l.blocks = (V + kBlockElems - 1) / kBlockElems;
  const bool drows = drafted && !dprobs;
  const int64_t rows = static_cast<int64_t>(M) * ((tprobs ? 0 : 1) + (drows ? 1 : 0));
  const auto pieces = [&](int part_blocks) { return (l.blocks + part_blocks - 1) / part_blocks; };
  l.part_blocks = 16;
  while (l.part_blocks > 1 && rows * pieces(l.part_blocks) < 4096 && pieces(l.part_blocks / 2) <= kPieces) l.part_blocks /= 2;
  l.parts = pieces(l.part_blocks);
  int shares = B > 0 ? (768 + B - 1) / B : 1;
  if (shares > (l.blocks + 3) / 4) shares = (l.blocks + 3) / 4;
  l.share_blocks = (l.blocks + shares - 1) / shares;
  l.shares = (l.blocks + l.share_blocks - 1) / l.share_blocks;
  size_t at = static_cast<size_t>(M) * (drows ? 2 : 1) * l.parts * sizeof(StatPart);
  l.sums = at;
  at += static_cast<size_t>(B) * l.blocks * 2 * sizeof(double);
  l.totals = at;
  at += static_cast<size_t>(B) * l.shares * (kVerifyThreads / 64) * sizeof(Sums);
  l.pending = at;
  at += static_cast<size_t>(B) * sizeof(Pending);
  l.rows = at;
  at += drafted ? static_cast<size_t>(M) * sizeof(RowInfo) : 0;
  l.tickets = at;
  at += static_cast<size_t>(B) * kPasses * sizeof(uint64_t);
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
  p.totals = reinterpret_cast<Sums*>(ws + l.totals);
  p.tickets = reinterpret_cast<uint64_t*>(ws + l.tickets);
  p.pending = reinterpret_cast<Pending*>(ws + l.pending);
  p.rows = reinterpret_cast<RowInfo*>(ws + l.rows);
  if (a.M > 0) {
    // (rows of probabilities have statistics only where they may be greedy)
    const int first = a.tprobs && !a.temperature ? a.M : 0, end = a.draft && !a.dprobs ? 2 * a.M : a.M;
    const int64_t u0 = static_cast<int64_t>(first) * l.parts, u1 = static_cast<int64_t>(end) * l.parts;
    int64_t blocks = (u1 - u0 + 3) / 4;
    blocks = blocks < 1 ? 1 : blocks < (1 << 22) ? blocks : 1 << 22;
    hipLaunchKernelGGL(k_verify_stats, dim3(static_cast<uint32_t>(blocks)), dim3(kVerifyThreads), 0, s, p, u0, u1);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (a.draft && a.parents) {  // two workgroups of these to a CU: no more than run at once (48 sequences of 12 rows: 77 -> 74 us)
    int shares = (512 + a.B - 1) / a.B;
    if (shares > l.shares) shares = l.shares;
    p.share_blocks = (l.blocks + shares - 1) / shares;
    p.shares = (l.blocks + p.share_blocks - 1) / p.share_blocks;
  }
  const dim3 grid(a.B * p.shares);
  // (no rows: nothing is read of either, and the kernels without a draft are of one type)
  const int dt = a.M > 0 && a.draft && a.ddt != a.tdt ? -1 : a.tdt;
  const auto pick = [&](auto tree, auto draft, int pass, int passes) {
    constexpr bool TREE = decltype(tree)::value, DRAFT = decltype(draft)::value;
    const dim3 threads(kVerifyThreads);
    if (dt == 0) hipLaunchKernelGGL((k_verify_pick<TREE, DRAFT, 0>), grid, threads, 0, s, p, pass, passes);
    else if (dt == 1) hipLaunchKernelGGL((k_verify_pick<TREE, DRAFT, 1>), grid, threads, 0, s, p, pass, passes);
    else if (dt == 2) hipLaunchKernelGGL((k_verify_pick<TREE, DRAFT, 2>), grid, threads, 0, s, p, pass, passes);
    else if constexpr (DRAFT) hipLaunchKernelGGL((k_verify_pick<TREE, true, -1>), grid, threads, 0, s, p, pass, passes);
    else return hipErrorInvalidValue;
    return hipGetLastError();
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (!a.parents) return a.draft ? pick(No{}, Yes{}, 0, 1) : pick(No{}, No{}, 0, 1);
  if (!a.draft || a.M == 0) return pick(Yes{}, No{}, 0, 1);
  for (int pass = 0; pass < kPasses; ++pass)
    if (const hipError_t e = pick(Yes{}, Yes{}, pass, kPasses); e != hipSuccess) return e;
  return hipGetLastError();
}

}  // namespace tq
