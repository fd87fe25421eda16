// Attention over the paged compressed cache: the kernel (instantiated per key format in
// kv_attend_*.hip, dispatched in kv_attend.hip).
//     out = R_v^T sum_j p_j v'_j,  p = softmax_j(scale * (R_k q) . k'_j)
// with k', v' the decoded rows in the rotated bases (R orthonormal: q . k = (R q) . (R k)).
//
// Work. A unit is (sequence, key head, tile of up to 16 R query rows that share the head). All
// units lie on one line of work, each as long as the tokens it reads plus a constant for its
// set-up, cut into equal shares, one per workgroup: uneven lengths balance, and a few long
// sequences still fill the chip. A share boundary inside a unit leaves partial sums in the
// workspace, which k_attend_join adds up in a fixed order. Workgroups are small (four waves), so
// that two or three share a CU and one's set-up hides behind another's stream.
//
// A wave takes blocks of 32 tokens. Scores come as S^T = K Q^T on v_mfma_f32_16x16x32_f16: lane l
// supplies a quarter row of token l % 16 (elements D / 4 * (l / 16) + ..., one contiguous load and
// one group scale) and receives, for query row l % 16, the tokens 4 (l / 16) + i: exactly the
// layout in which P^T is the B operand of O^T += V^T P^T, so probabilities never leave their lane. The V operand wants eight tokens of one element per
// lane: lane l loads the same piece of eight tokens' rows (D / 16 codes at element D / 16 * (l % 16))
// and pairs equal positions of two tokens by bit operations. Decoded values are never stored.
//
// Decoding is an LDS table of fp16 centroids. Codes of 8 bits (and pairs of 4-bit codes) use a
// table with 32 columns, entry e for lane l at 128 e + 4 (l % 32): the lanes that the LDS serves
// together never meet in a bank, and one v_dot4 makes the address from a byte of the word. Pairs of 3- and 2-bit codes need 64 and 16 entries, which
// lie in different banks by themselves.
//
// Group scales multiply the centroids in fp16, kept in range by powers of two per wave that follow
// the largest scales met. Softmax in base 2 with a reference that moves only when a score passes it
// by 2^8 (p then stays within fp16: 2^7 at the reference, at most 2^15), so the running maximum
// needs neither lane exchange nor rescaling in the common step. Sums are fp32.
#pragma once

#include "internal.hpp"
#include "kv_lane.hpp"

namespace tq {

constexpr int kAtCus = 256;
constexpr int kAtMaxGrid = 3 * kAtCus;  // workgroups of a launch, at most
constexpr int kAtUnit = 256;            // a unit's set-up in tokens of work
constexpr int kAtMinShare = 512;        // least work of a share
constexpr float kAtLazy = 8.f;      // log2 of how far a score may pass the reference

struct AttendMeta {                 // of a workgroup whose last unit goes on in the next ones
  int32_t parts;                    // following workgroups that hold a part; 0: nothing to join
  int32_t row0, nrows;              // first query row (of M) of the unit, rows per (token, head)
  int32_t head0, hb, pad[3];        // first query head, heads per token of the tile
};

struct AttendParams {
  AttendArgs a;
  int share, hb, nhb, a_tok;  // query heads per key head; heads, head blocks, tokens of a tile
  int grid, n_each;           // workgroups; queries of a sequence without q_offsets
  float inv_sqrt_d;
  uint32_t page16, page_mul;  // page_tokens / 16 and ceil(2^32 / page16) (0 for 1)
  AttendMeta* meta;
  float* parts;
  uint16_t hk[256], hv[256];  // fp16 centroids
};

template <int KB, int VB, int D, int R>
struct AtCfg {
  static constexpr int W = 4;               // waves
  static constexpr int T = 64 * W;
  static constexpr int ROWS = 16 * R;
  static constexpr int NS = D / 32;         // 32-element steps of a key row
  static constexpr int CH = D / 16;         // codes of a lane's piece of a value row
  static constexpr bool KWIDE = KB == 8 || (KB == 4 && VB != 8);
  static constexpr bool VWIDE = VB == 8 || (VB == 4 && KB != 8);
  static constexpr int KROW = D * KB / 8, VROW = D * VB / 8;  // row bytes
  static constexpr int KW = (KROW / 4 + 3) / 4;               // words of a quarter key row
  static constexpr int KS = D == 256 ? 2 : 1;                 // key scales of a quarter row, at most
  static constexpr int VW = (VB * CH + 31) / 32;              // words of a value piece
  static constexpr int WGS = R == 1 && D <= 128 ? 3 : 2;      // workgroups per CU
  // LDS; the joined sums take the place of q
  static constexpr int WIDE = (KWIDE || VWIDE) ? 32768 : 0;
  static constexpr int TK = WIDE, TV = TK + 1024;
  static constexpr int C1 = TV + 1024, ML = C1 + ROWS * 4, SC = ML + W * ROWS * 8, QS = SC + 64;
  static constexpr int QP = D * 2 + 16;                       // padded row of q
  static constexpr int PER_N = W * ROWS * 16 * 4;             // bytes of one O block of all waves
  static constexpr int NL = PER_N >= 16384 ? 1 : 16384 / PER_N;  // O blocks joined per round
  static constexpr int FP = D + 1;                            // padded row of the joined sums
  static constexpr int RED = QS;
  static constexpr int max3(int a, int b, int c) { return a > b ? (a > c ? a : c) : b > c ? b : c; }
  static constexpr int LDS = QS + max3(ROWS * QP, PER_N * NL, ROWS * FP * 4);
  static_assert(LDS * WGS <= 163840, "LDS of a CU");
  static_assert(CH % NL == 0, "whole rounds");
};

// A word of LDS at a byte address (the kernel's LDS is all dynamic and begins at address 0: no base
// is added to an address that the lookup just computed).
__device__ __forceinline__ uint32_t at_lds(uint32_t off) {
  return *(const __attribute__((address_space(3))) uint32_t*)(uintptr_t)(off);
}
__device__ __forceinline__ int at_uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t at_uniform(int64_t x) {
  return static_cast<int64_t>(at_uniform(static_cast<int>(x >> 32))) << 32 |
         static_cast<uint32_t>(at_uniform(static_cast<int>(x)));
}
__device__ __forceinline__ uint32_t at_pack(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x05040100);
}
// base + m * (byte k of x)
template <int MUL>
__device__ __forceinline__ uint32_t at_byte(uint32_t x, int k, uint32_t base) {
  return __builtin_amdgcn_udot4(x, static_cast<uint32_t>(MUL) << (8 * k), base, false);
}
__device__ __forceinline__ float at_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
// base + bytes as a pointer that stays in scalar registers (loads then take a scalar base and the
// lane's 32-bit offset)
typedef const __attribute__((address_space(1))) char* AtPtr;
__device__ __forceinline__ AtPtr at_base(const void* base, int64_t bytes) {
  return (AtPtr)(at_uniform(reinterpret_cast<int64_t>(base) + bytes));
}
template <typename T>
__device__ __forceinline__ T at_get(AtPtr base, uint32_t off) {
  return *(const __attribute__((address_space(1))) T*)(base + off);
}
// a load at any byte address
template <typename T>
__device__ __forceinline__ T at_load(AtPtr base, uint32_t off) {
  typedef T __attribute__((aligned(1))) U;
  return *(const __attribute__((address_space(1))) U*)(base + off);
}

// Normalises, rotates back and stores one output row held as in kv_wave_transform.
template <int D>
__device__ __forceinline__ void at_finish(const AttendParams& p, float (&v)[D / 64], float l, int64_t m,
                                          int head, int lane) {
  constexpr int EL = D / 64;
  const float f = l == 0.f ? 0.f : p.inv_sqrt_d / l;
#pragma unroll
  for (int e = 0; e < EL; ++e) v[e] = l == 0.f ? 0.f : v[e] * f;
  const int c = kv_chunk(lane), d0 = c * EL;
  const uint32_t sg = p.a.c.v.signs[d0 >> 5] >> (d0 & 31);
  kv_wave_transform<EL>(v, c);
  const int64_t o = (m * p.a.q_heads + head) * D + d0;
  uint16_t* dst = static_cast<uint16_t*>(p.a.out) + o;
  uint16_t x[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    const float y = (sg >> e) & 1u ? -v[e] : v[e];
    x[e] = p.a.odt == 1 ? float_to_bf16_rne(y) : float_to_half_rne(y);
  }
  __builtin_memcpy(__builtin_assume_aligned(dst, 2 * EL), x, 2 * EL);
}

// ---- work ---------------------------------------------------------------------------------
// One sequence as the schedule sees it. Tile t of a head costs the tokens its last row sees and
// kAtUnit; block k of it lies kAtUnit + 32 k from the unit's begin on the line.
struct AtSeq {
  int row0, n, len, tiles;
  bool flat;         // every tile reads the whole length (trees; more queries than tokens)
  int64_t per_head;  // cost of all tiles of one head
};

__device__ __forceinline__ int64_t at_before(const AtSeq& s, int a, int t) {  // cost of tiles < t, t < tiles
  if (s.flat) return static_cast<int64_t>(t) * ((s.len > 1 ? s.len : 1) + kAtUnit);
  return static_cast<int64_t>(t) * (s.len - s.n + kAtUnit) + static_cast<int64_t>(a) * t * (t + 1) / 2;
}
__device__ __forceinline__ int at_reads(const AtSeq& s, int a, int t) {
  if (s.flat) return s.len > 1 ? s.len : 1;
  const int q = (t + 1) * a < s.n ? (t + 1) * a : s.n;
  return s.len - s.n + q;
}
// U: b is the same in every lane of the wave, and so is what comes of it.
template <bool U>
__device__ __forceinline__ AtSeq at_seq(const AttendParams& p, int b) {
  AtSeq s;
  const int M = static_cast<int>(p.a.M);
  int len = p.a.kv_lens[b];
  if constexpr (U) len = at_uniform(len);
  if (p.a.q_offsets) {
    int lo = p.a.q_offsets[b], hi = p.a.q_offsets[b + 1];
    if constexpr (U) {
      lo = at_uniform(lo);
      hi = at_uniform(hi);
    }
    lo = lo < 0 ? 0 : lo > M ? M : lo;
    hi = hi < lo ? lo : hi > M ? M : hi;
    s.row0 = lo;
    s.n = hi - lo;
  } else {
    s.n = p.n_each;
    s.row0 = b * s.n;
  }
  const int cap = p.a.table_width * p.a.c.page;
  s.len = len < 0 ? 0 : len < cap ? len : cap;
  s.tiles = s.n <= p.a_tok ? (s.n > 0 ? 1 : 0) : (s.n + p.a_tok - 1) / p.a_tok;
  s.flat = p.a.tree != nullptr || s.n > s.len;
  s.per_head = s.tiles == 0 ? 0 : at_before(s, p.a_tok, s.tiles - 1) + at_reads(s, p.a_tok, s.tiles - 1) + kAtUnit;
  return s;
}

// Page of token j (a multiple of 16): a product estimate, at most one too large because j / 16 < 2^27
// and page16 <= 2^12, put right by one step.
__device__ __forceinline__ int at_page(const AttendParams& p, int j) {
  const uint32_t u = static_cast<uint32_t>(j) >> 4;
  uint32_t x = p.page_mul ? __umulhi(u, p.page_mul) : u;
  x -= x * p.page16 > u ? 1u : 0u;
  return static_cast<int>(x);
}

// ---- decoding -----------------------------------------------------------------------------
// Eight key codes (number st of the lane's quarter row) as four fp16 pairs.
template <typename C, int KB>
__device__ __forceinline__ void at_decode_k(const uint32_t* w, int st, uint32_t lane4, uint32_t (&o)[4]) {
  if constexpr (KB == 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = w[2 * st + (k >> 1)];
      const uint32_t a = at_lds(at_byte<128>(x, 2 * (k & 1), lane4));
      const uint32_t b = at_lds(at_byte<128>(x, 2 * (k & 1) + 1, lane4));
      o[k] = at_pack(a, b);
    }
  } else if constexpr (KB == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (C::KWIDE) o[k] = at_lds(at_byte<128>(w[st], k, lane4));
      else o[k] = at_lds(C::TK + (at_byte<4>(w[st], k, 0)));
    }
  } else {
    // pairs of 2 KB bits of the bitstream; a table index times four
    constexpr uint32_t M = ((1u << (2 * KB)) - 1u) << 2;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int bp = 2 * KB * (4 * st + k), wi = bp >> 5, sh = bp & 31;
      uint32_t x;
      if (sh + 2 * KB > 32) x = static_cast<uint32_t>((static_cast<uint64_t>(w[wi + 1]) << 32 | w[wi]) >> (sh - 2));
      else x = sh < 2 ? w[wi] << (2 - sh) : w[wi] >> (sh - 2);
      o[k] = at_lds(C::TK + (x & M));
    }
  }
}

// Element n of a value piece of the tokens with words w0 and w1, as an fp16 pair. e and o are
// the words combined by at_pair (codes below 8 bits).
template <int VB>
__device__ __forceinline__ void at_pair(uint32_t w0, uint32_t w1, uint32_t& even, uint32_t& odd) {
  constexpr uint32_t M = VB == 4 ? 0x0f0f0f0fu : VB == 3 ? 0x001c71c7u : 0x33333333u;
  constexpr uint32_t M3 = VB == 3 ? 0x00e38e38u : ~M;  // the upper code of each field
  even = (w0 & M) | ((w1 << VB) & M3);
  odd = ((w0 >> VB) & M) | (w1 & M3);
}
template <typename C, int VB>
__device__ __forceinline__ uint32_t at_pair_at(uint32_t x, int q, uint32_t lane4) {
  if constexpr (VB == 4) {
    if constexpr (C::VWIDE) return at_lds(at_byte<128>(x, q, lane4));
    return at_lds(C::TV + (at_byte<4>(x, q, 0)));
  } else if constexpr (VB == 3) {
    return at_lds(C::TV + ((q == 0 ? x << 2 : x >> (6 * q - 2)) & 0xfcu));
  } else {
    return at_lds(C::TV + ((q == 0 ? x << 2 : x >> (4 * q - 2)) & 0x3cu));
  }
}

__device__ __forceinline__ uint32_t at_mul(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, a) * __builtin_bit_cast(half2_t, b));
}
// 2^-e in both halves, -15 <= e <= 14; 2^-15 as the subnormal it is
__device__ __forceinline__ uint32_t at_pow2(int e) {
  const uint32_t x = e < 15 ? static_cast<uint32_t>(15 - e) << 10 : 0x0200u;
  return x | (x << 16);
}
__device__ __forceinline__ f32x4_t at_mfma(const uint32_t (&a)[4], const uint32_t (&b)[4], f32x4_t c) {
  const u32x4_t x{a[0], a[1], a[2], a[3]}, y{b[0], b[1], b[2], b[3]};
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, x), __builtin_bit_cast(f16x8_t, y), c, 0, 0, 0);
}

template <int KB, int VB, int D, int R>
__global__ __launch_bounds__((AtCfg<KB, VB, D, R>::T), (AtCfg<KB, VB, D, R>::WGS)) void k_attend(AttendParams p) {
  using C = AtCfg<KB, VB, D, R>;
  constexpr int W = C::W, T = C::T, ROWS = C::ROWS, NS = C::NS, CH = C::CH, EL = D / 64;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = at_uniform(tid >> 6);
  const int col = lane & 15, h = lane >> 4;
  const uint32_t lane4 = (lane & 31) * 4;

  // this workgroup's share of the work: a scan over the sequences' costs, each thread taking
  // neighbouring ones; the thread that holds the share's begin finds its unit
  const int hu_n = p.a.c.heads * p.nhb;
  const int per = (p.a.B + T - 1) / T;
  const int b0 = tid * per, b1 = b0 + per < p.a.B ? b0 + per : p.a.B;
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += at_seq<false>(p, b).per_head * hu_n;

  // centroid tables
  if constexpr (C::WIDE > 0) {
    // a wave's entries are uniform: scalar loads of the arguments, two 128-byte rows per store
    constexpr int TB = KB == 8 || VB == 8 ? 8 : 4;
    const uint16_t* hc = KB == TB ? p.hk : p.hv;
    constexpr int PW = 256 / W;
#pragma unroll
    for (int k = 0; k < PW; k += 2) {
      const int e = wave * PW + k;
      const uint32_t x = TB == 8 ? hc[e] : (hc[e & 15] | static_cast<uint32_t>(hc[e >> 4]) << 16);
      const uint32_t y = TB == 8 ? hc[e + 1] : (hc[(e + 1) & 15] | static_cast<uint32_t>(hc[e >> 4]) << 16);
      *reinterpret_cast<uint32_t*>(smem + 128 * e + 4 * lane) = lane < 32 ? x : y;
    }
  }
  if constexpr (KB < 8 && !C::KWIDE)
    for (int e = tid; e < (1 << (2 * KB)); e += T)
      *reinterpret_cast<uint32_t*>(smem + C::TK + 4 * e) =
          p.hk[e & ((1 << KB) - 1)] | static_cast<uint32_t>(p.hk[e >> KB]) << 16;
  if constexpr (VB < 8 && !C::VWIDE)
    for (int e = tid; e < (1 << (2 * VB)); e += T)
      *reinterpret_cast<uint32_t*>(smem + C::TV + 4 * e) =
          p.hv[e & ((1 << VB) - 1)] | static_cast<uint32_t>(p.hv[e >> VB]) << 16;

  int64_t* sc = reinterpret_cast<int64_t*>(smem + C::SC);  // [W] wave sums, then the begin
  int64_t incl = sum;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int64_t o = __shfl_up(incl, m);
    incl += lane >= m ? o : 0;
  }
  if (lane == 63) sc[wave] = incl;
  if (tid == 0) p.meta[blockIdx.x].parts = 0;
  __syncthreads();
  int64_t total = 0, base = incl - sum;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int64_t x = sc[w];
    base += w < wave ? x : 0;
    total += x;
  }
  total = at_uniform(total);
  int64_t q = total / p.grid + 1;
  q = at_uniform(q < kAtMinShare ? kAtMinShare : q);
  const int64_t w0 = q * blockIdx.x, w1 = w0 + q < total ? w0 + q : total;
  if (w0 >= total) return;
  if (w0 >= base && w0 < base + sum) {
    int64_t rem = w0 - base;
    int b = b0;
    AtSeq x = at_seq<false>(p, b);
    while (rem >= x.per_head * hu_n) {
      rem -= x.per_head * hu_n;
      x = at_seq<false>(p, ++b);
    }
    // head and tile: rem < 2^53, so the quotient in fp64 is at most one off
    int64_t hd = static_cast<int64_t>(static_cast<double>(rem) / static_cast<double>(x.per_head));
    hd -= hd * x.per_head > rem ? 1 : 0;
    hd += (hd + 1) * x.per_head <= rem ? 1 : 0;
    rem -= hd * x.per_head;
    int lo = 0, hi = x.tiles - 1;  // last tile with at_before <= rem
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (at_before(x, p.a_tok, mid) <= rem) lo = mid;
      else hi = mid - 1;
    }
    sc[4] = static_cast<int64_t>(hd) << 32 | b;
    sc[5] = lo;
    sc[6] = w0 - (rem - at_before(x, p.a_tok, lo));
  }
  __syncthreads();
  int b = at_uniform(static_cast<int>(sc[4])), hu = at_uniform(static_cast<int>(sc[4] >> 32));
  int t = at_uniform(static_cast<int>(sc[5]));
  int64_t u0 = at_uniform(sc[6]);  // the unit's begin
  AtSeq sq = at_seq<true>(p, b);

  const int page = p.a.c.page;
  const int kg = p.a.c.k.group, vg = p.a.c.v.group;
  const int gk = D / kg, gv = D / vg;
  const uint32_t koff = col * C::KROW + (C::KROW / 4) * h;
  // scales of the quarter row's first and (D = 256) second half
  const uint32_t ksoff = (col * gk + (D / 4 * h) / kg) * 2, ksoff2 = (col * gk + (D / 4 * h + D / 8) / kg) * 2;
  const uint32_t voff = 4 * h * C::VROW + (VB * CH * col) / 8;
  const uint32_t vsoff = 4 * h * gv * 2 + ((col * CH) / vg) * 2;

  for (int64_t w = w0; w < w1;) {
    // what steers the wave is the same in all its lanes; said so, it lives in scalar registers
    w = at_uniform(w);
    u0 = at_uniform(u0);
    b = at_uniform(b);
    hu = at_uniform(hu);
    t = at_uniform(t);
    sq.row0 = at_uniform(sq.row0);
    sq.n = at_uniform(sq.n);
    sq.len = at_uniform(sq.len);
    sq.tiles = at_uniform(sq.tiles);
    sq.flat = at_uniform(sq.flat ? 1 : 0) != 0;
    const int reads = at_reads(sq, p.a_tok, t);
    const int64_t x0 = w - u0 - kAtUnit, x1 = w1 - u0 - kAtUnit < reads ? w1 - u0 - kAtUnit : reads;
    const int k0 = x0 <= 0 ? 0 : static_cast<int>((x0 + 31) >> 5);
    const int k1 = x1 <= 0 ? 0 : static_cast<int>((x1 + 31) >> 5);
    const int nblk = (reads + 31) >> 5;
    if (k0 < k1) {
      const int kh = hu / p.nhb, hblk = hu - kh * p.nhb;
      const int head0 = kh * p.share + hblk * p.hb;
      const int nh = p.share - hblk * p.hb < p.hb ? p.share - hblk * p.hb : p.hb;
      const int tok0 = t * p.a_tok;
      const int ntok = sq.n - tok0 < p.a_tok ? sq.n - tok0 : p.a_tok;
      const int before = sq.len - sq.n;

      // ---- blocks of 32 tokens ----
      uint32_t kraw[2][C::KW] = {}, vraw[8][C::VW] = {}, ksr[2][C::KS] = {}, vsr[4] = {};
      const int32_t* table = p.a.page_table + static_cast<int64_t>(b) * p.a.table_width;
      const int64_t khead = static_cast<int64_t>(kh) * page, prow = static_cast<int64_t>(p.a.c.heads) * page;
      int64_t row_of[2] = {};
      bool bad[2] = {};
      // page ids of a block's halves (a half past the end stands for the first one), read one
      // block ahead; constant memory, so that they come by scalar loads
      typedef const int32_t __attribute__((address_space(4))) * ConstIds;
      const ConstIds ids = (ConstIds)reinterpret_cast<uintptr_t>(table);
      int id[2] = {}, in[2] = {};
      auto look = [&](int blk) {
        const int j = blk * 32, j2 = j + 16 < sq.len ? j + 16 : j;
        const int pi = at_page(p, j), pi2 = at_page(p, j2);
        in[0] = j - pi * page;
        in[1] = j2 - pi2 * page;
        id[0] = sq.len > 0 ? ids[pi] : -1;
        id[1] = sq.len > 0 ? ids[pi2] : -1;
      };
      auto locate = [&]() {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          bad[x] = id[x] < 0 || id[x] >= p.a.c.pages;
          row_of[x] = (bad[x] ? 0 : id[x]) * prow + khead + in[x];
        }
      };
      auto load_k = [&]() {
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
          const AtPtr kc = at_base(p.a.c.k.codes, row_of[sb] * C::KROW);
          constexpr int L = C::KW % 4 == 0 ? 4 : C::KW % 3 == 0 ? 3 : C::KW % 2 == 0 ? 2 : 1;  // words of a load
          if constexpr (C::KROW % 16 != 0) {  // six bytes
            kraw[sb][0] = at_load<uint32_t>(kc, koff);
            kraw[sb][1] = at_load<uint16_t>(kc, koff + 4);
          } else {
#pragma unroll
          for (int k = 0; k < C::KW; k += L) {
            if constexpr (L == 4) {
              const u32x4_t x = at_get<u32x4_t>(kc, koff + 4 * k);
              kraw[sb][k] = x.x; kraw[sb][k + 1] = x.y; kraw[sb][k + 2] = x.z; kraw[sb][k + 3] = x.w;
            } else if constexpr (L == 3) {
              const u32x3_t x = at_get<u32x3_t>(kc, koff + 4 * k);
              kraw[sb][k] = x.x; kraw[sb][k + 1] = x.y; kraw[sb][k + 2] = x.z;
            } else if constexpr (L == 2) {
              const u32x2_t x = at_get<u32x2_t>(kc, koff + 4 * k);
              kraw[sb][k] = x.x; kraw[sb][k + 1] = x.y;
            } else {
              kraw[sb][k] = at_get<uint32_t>(kc, koff + 4 * k);
            }
          }
          }
          const AtPtr sp = at_base(p.a.c.k.scales, row_of[sb] * gk * 2);
          ksr[sb][0] = at_get<uint16_t>(sp, ksoff);
          if constexpr (C::KS == 2) ksr[sb][1] = at_get<uint16_t>(sp, ksoff2);
        }
      };
      auto load_v = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int sb = i >> 2;
          const AtPtr vc = at_base(p.a.c.v.codes, row_of[sb] * C::VROW);
          const uint32_t off = voff + (i & 3) * C::VROW;
          if constexpr (VB == 3) {
            if constexpr (CH == 4) {
              vraw[i][0] = at_load<uint16_t>(vc, off) >> (4 * (col & 1));
            } else if constexpr (CH == 8) {
              const uint32_t back = col == 15 ? 1 : 0;
              vraw[i][0] = at_load<uint32_t>(vc, off - back) >> (8 * back);
            } else {
              const uint32_t a = at_load<uint32_t>(vc, off), c = at_load<uint16_t>(vc, off + 4);
              vraw[i][0] = a;
              vraw[i][1] = (a >> 24) | (c << 8);
            }
          } else if constexpr (VB * CH == 8) {
            vraw[i][0] = at_get<uint8_t>(vc, off);
          } else if constexpr (VB * CH == 16) {
            vraw[i][0] = at_get<uint16_t>(vc, off);
          } else {
#pragma unroll
            for (int k = 0; k < C::VW; ++k) vraw[i][k] = at_get<uint32_t>(vc, off + 4 * k);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const AtPtr sp = at_base(p.a.c.v.scales, row_of[i >> 1] * gv * 2);
          const uint32_t off = vsoff + (2 * (i & 1)) * gv * 2;
          const uint32_t a = at_get<uint16_t>(sp, off);
          const uint32_t c = at_get<uint16_t>(sp, off + gv * 2);
          vsr[i] = a | (c << 16);
        }
      };

      int blk = k0 + wave;
      bool kbad[2] = {false, false};
      if (blk < k1) {
        look(blk);
        locate();
        load_k();
        load_v();
        kbad[0] = bad[0];
        kbad[1] = bad[1];
        if (blk + W < k1) look(blk + W);
      }
      // ---- q: rotated, scaled by a power of two to fp16's upper range, into LDS ----
      __syncthreads();  // the last unit's readers of this memory are done
      {
        constexpr int RW = ROWS / W < 4 ? ROWS / W : 4;  // rows of a wave at a time
        const int ch = kv_chunk(lane), d0 = ch * EL;
        const uint32_t sg = p.a.c.k.signs[d0 >> 5] >> (d0 & 31);
#pragma unroll 1
        for (int r0 = wave * (ROWS / W); r0 < (wave + 1) * (ROWS / W); r0 += RW) {
          float v[RW][EL];
#pragma unroll
          for (int x = 0; x < RW; ++x) {
            const int tk = (r0 + x) / p.hb, hd = r0 + x - tk * p.hb;
            const bool ok = tk < ntok && hd < nh && p.a.scale != 0.f;
            const uint16_t* src = static_cast<const uint16_t*>(p.a.q) +
                                  (static_cast<int64_t>(sq.row0) + tok0 + (ok ? tk : 0)) * p.a.q_stride +
                                  static_cast<int64_t>(head0 + (ok ? hd : 0)) * D + d0;
            uint16_t raw[EL];
            __builtin_memcpy(raw, __builtin_assume_aligned(src, 2 * EL), 2 * EL);
#pragma unroll
            for (int e = 0; e < EL; ++e) {
              const float y = p.a.qdt == 1 ? bf16_bits_to_float(raw[e]) : half_bits_to_float(raw[e]);
              v[x][e] = !ok ? 0.f : ((sg >> e) & 1u) != (p.a.scale < 0.f ? 1u : 0u) ? -y : y;
            }
          }
#pragma unroll
          for (int x = 0; x < RW; ++x) {
            kv_wave_transform<EL>(v[x], ch);
            float mx = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) mx = fmaxf(mx, fabsf(v[x][e]));
            mx = kv_wave_max(mx);
            // the largest magnitude comes to [2^13, 2^14): exponent 127 + 13 of the scaled value
            const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
            int k = mx > 0.f && ex < 255 ? 140 - ex : 0;
            k = k > 100 ? 100 : k;
            const float f = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
            _Float16 y[EL];
#pragma unroll
            for (int e = 0; e < EL; ++e) y[e] = static_cast<_Float16>(v[x][e] * f);
            __builtin_memcpy(__builtin_assume_aligned(smem + C::QS + (r0 + x) * C::QP + 2 * d0, 2 * EL), y, 2 * EL);
            if (lane == 0)
              *reinterpret_cast<float*>(smem + C::C1 + 4 * (r0 + x)) =
                  p.a.scale == 0.f ? 1.f : fabsf(p.a.scale) * 1.44269504f * p.inv_sqrt_d *
                                               __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
          }
        }
      }
      __syncthreads();
      float c1[R];
      int lim[R], tok_row[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = 16 * r + col, tk = row / p.hb, hd = row - tk * p.hb;
        c1[r] = *reinterpret_cast<const float*>(smem + C::C1 + 4 * row);  // times 2^kexp
        const bool ok = tk < ntok && hd < nh;
        tok_row[r] = sq.row0 + tok0 + (ok ? tk : 0);
        int x = p.a.tree ? before : before + tok0 + tk + 1;
        x = x < 0 ? 0 : x;
        lim[r] = !ok || x > sq.len ? sq.len : x;
      }
      // from this token on some row's mask may cut
      int cut = p.a.tree ? before : before + tok0 + 1;
      cut = cut < 0 ? 0 : cut;

      float mref[R], mo[R], l[R];
      f32x4_t o[R][CH];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mref[r] = -__builtin_inff();
        mo[r] = 0.f;
        l[r] = 0.f;
#pragma unroll
        for (int n = 0; n < CH; ++n) o[r][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      // Scales are held times 2^-kexp and 2^-vexp. They start at 1, are set by the first block if
      // its scales are small (below 2^-4), and grow when one passes 2^13.
      int kexp = 0, vexp = 0;

      for (; blk < k1; blk += W) {
        const bool more = blk + W < k1;
        const bool b0_ = kbad[0], b1_ = kbad[1];
        // ---- scores ----
        f32x4_t s[R][2];
        uint32_t kd[2][C::KS];  // scales times 2^-kexp, in both halves; no number for a bad page
        auto key_scales = [&]() {
          uint32_t big = 0;
#pragma unroll
          for (int sb = 0; sb < 2; ++sb)
#pragma unroll
            for (int x = 0; x < C::KS; ++x) {
              uint32_t y = ksr[sb][x] | (ksr[sb][x] << 16);
              if (sb ? b1_ : b0_) y = 0;
              kd[sb][x] = at_mul(y, at_pow2(kexp));
              big = kd[sb][x] > big ? kd[sb][x] : big;
            }
          return big;
        };
        const uint32_t kbig = key_scales();
        if (__any(kbig > 0x7000ffffu) || (blk == k0 + wave && !__any(kbig > 0x2c00ffffu))) {  // beyond 2^13, no number, or small
          float top = 0.f;
#pragma unroll
          for (int sb = 0; sb < 2; ++sb)
#pragma unroll
            for (int x = 0; x < C::KS; ++x)
              if ((ksr[sb][x] & 0x7c00u) != 0x7c00u && !(sb ? b1_ : b0_))
                top = fmaxf(top, fabsf(half_bits_to_float(static_cast<uint16_t>(ksr[sb][x]))));
          int ne = static_cast<int>(__float_as_uint(kv_wave_max(top)) >> 23) - 127;
          ne = at_uniform(ne < -15 ? -15 : ne);
          if (ne > kexp || blk == k0 + wave) {
            const float f = at_exp2(static_cast<float>(ne - kexp));
            kexp = ne;
#pragma unroll
            for (int r = 0; r < R; ++r) c1[r] *= f;
          }
          key_scales();
        }
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
#pragma unroll
          for (int r = 0; r < R; ++r) s[r][sb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int st = 0; st < NS; ++st) {
            uint32_t a[4];
            at_decode_k<C, KB>(kraw[sb], st, lane4, a);
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = at_mul(a[k], kd[sb][C::KS == 2 ? st / (NS / 2) : 0]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const u32x4_t qv = *reinterpret_cast<const u32x4_t*>(smem + C::QS + (16 * r + col) * C::QP + (D / 2) * h + 16 * st);
              const uint32_t qb[4] = {qv.x, qv.y, qv.z, qv.w};
              s[r][sb] = at_mfma(a, qb, s[r][sb]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          if (sb ? b1_ : b0_) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[r][sb][i] = __builtin_nanf("");
          }
        }
        if (more) {
          locate();
          load_k();
          kbad[0] = bad[0];
          kbad[1] = bad[1];
          if (blk + 2 * W < k1) look(blk + 2 * W);
        }
        // ---- masks ----
        const int j0 = blk * 32 + 4 * h;
        if (blk * 32 + 32 > cut) {
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int sb = 0; sb < 2; ++sb)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = j0 + 16 * sb + i;
                bool see = j < lim[r];
                if (p.a.tree && !see && j < sq.len) {
                  const int x = j - before;
                  if (x >= 0 && x < p.a.tree_words * 32)
                    see = (p.a.tree[static_cast<int64_t>(tok_row[r]) * p.a.tree_words + (x >> 5)] >> (x & 31)) & 1u;
                }
                s[r][sb][i] = see ? s[r][sb][i] : -__builtin_inff();
              }
        }
        // ---- softmax against a lazily moved reference ----
        float mx[R];
        bool move = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          mx[r] = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3]))) * c1[r];
          move = move || mx[r] > mref[r] + kAtLazy;
        }
        if (__any(move)) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float x, y;
            kv_both<4>(mx[r], x, y);
            kv_both<5>(fmaxf(x, y), x, y);
            x = fmaxf(x, y);
            if (x > mref[r] + kAtLazy) {  // the same in the four lanes of a row
              const float f = at_exp2(mref[r] - x);
              mref[r] = x;
              mo[r] = x - 7.f;
              l[r] *= f;
#pragma unroll
              for (int n = 0; n < CH; ++n) o[r][n] *= f;
            }
          }
        }
        uint32_t pb[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            e[i] = at_exp2(__builtin_fmaf(s[r][i >> 2][i & 3], c1[r], -mo[r]));
            l[r] += e[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const half2_t x{static_cast<_Float16>(e[2 * i]), static_cast<_Float16>(e[2 * i + 1])};
            pb[r][i] = __builtin_bit_cast(uint32_t, x);
          }
        }
        // ---- value scales: dead tokens and bad pages to zero, held times 2^-vexp ----
        uint32_t vs[4];
        if (blk * 32 + 32 > sq.len || b0_ || b1_) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + 16 * (i >> 1) + 2 * (i & 1);
            const bool dead = i < 2 ? b0_ : b1_;
            const uint32_t m = (dead || j >= sq.len ? 0u : 0xffffu) | (dead || j + 1 >= sq.len ? 0u : 0xffff0000u);
            vsr[i] &= m;
          }
        }
        uint32_t big = 0;
        {
          const uint32_t sc2 = at_pow2(vexp);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            vs[i] = at_mul(vsr[i], sc2);
            const uint32_t a = vs[i] & 0xffffu, c = vs[i] >> 16;
            big = a > big ? a : big;
            big = c > big ? c : big;
          }
        }
        if (__any(big > 0x7000u) || (blk == k0 + wave && !__any(big > 0x2c00u))) {
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t bits = (vsr[i >> 1] >> (16 * (i & 1))) & 0xffffu;
            const bool none = (bits & 0x7c00u) == 0x7c00u;
            const uint64_t who = __ballot(none);
            if ((who >> (16 * h)) & 0xffffu) {
              // this token's value is no number: rows that see it become NaN, others stay
              vsr[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
#pragma unroll
              for (int r = 0; r < R; ++r)
                if (s[r][i >> 2][i & 3] != -__builtin_inff()) l[r] = __builtin_nanf("");
            } else {
              top = fmaxf(top, fabsf(half_bits_to_float(static_cast<uint16_t>(bits))));
            }
          }
          int ne = static_cast<int>(__float_as_uint(kv_wave_max(top)) >> 23) - 127;
          ne = at_uniform(ne < -15 ? -15 : ne);
          if (ne > vexp || blk == k0 + wave) {
            const float f = at_exp2(static_cast<float>(vexp - ne));
            vexp = ne;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int n = 0; n < CH; ++n) o[r][n] *= f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) vs[i] = at_mul(vsr[i], at_pow2(vexp));
        }
        // ---- values ----
#pragma unroll
        for (int half = 0; half < (VB == 8 ? 1 : VB == 3 && CH == 16 ? 2 : C::VW); ++half) {
          constexpr int PN = VB == 8 ? CH : VB == 3 ? (CH == 16 ? 8 : CH) : (CH < 32 / VB ? CH : 32 / VB);
          uint32_t ev[4], od[4];
          if constexpr (VB < 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) at_pair<VB>(vraw[2 * i][half], vraw[2 * i + 1][half], ev[i], od[i]);
          }
#pragma unroll
          for (int n = 0; n < PN; ++n) {
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t x;
              if constexpr (VB == 8) {
                const uint32_t y = at_lds(at_byte<128>(vraw[2 * i][n >> 2], n & 3, lane4));
                const uint32_t z = at_lds(at_byte<128>(vraw[2 * i + 1][n >> 2], n & 3, lane4));
                x = at_pack(y, z);
              } else {
                x = at_pair_at<C, VB>((n & 1) ? od[i] : ev[i], n >> 1, lane4);
              }
              a[i] = at_mul(x, vs[i]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) o[r][half * PN + n] = at_mfma(a, pb[r], o[r][half * PN + n]);
            if (n & 1) __builtin_amdgcn_sched_barrier(0);
          }
        }
        if (more) load_v();
      }

      // ---- join the waves ----
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x, y;
        kv_both<4>(l[r], x, y);
        kv_both<5>(x + y, x, y);
        l[r] = x + y;
        if (h == 0)
          *reinterpret_cast<float2*>(smem + C::ML + 8 * (wave * ROWS + 16 * r + col)) = make_float2(mref[r], l[r]);
      }
      __syncthreads();
      float f[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float top = -__builtin_inff();
#pragma unroll
        for (int x = 0; x < W; ++x) top = fmaxf(top, *reinterpret_cast<const float*>(smem + C::ML + 8 * (x * ROWS + 16 * r + col)));
        f[r] = mref[r] == -__builtin_inff() ? 0.f : at_exp2(mref[r] - top + static_cast<float>(vexp));
      }
      constexpr int OUT = C::NL * 16 * ROWS / T;  // sums of a thread per round
      constexpr int RND = CH / C::NL;
      static_assert(C::NL * 16 * ROWS % T == 0, "whole sums per thread");
      float res[RND * OUT];
      float* red = reinterpret_cast<float*>(smem + C::RED);
#pragma unroll
      for (int rd = 0; rd < RND; ++rd) {
        if (rd) __syncthreads();
#pragma unroll
        for (int nl = 0; nl < C::NL; ++nl)
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              red[((wave * C::NL + nl) * 16 + 4 * h + i) * ROWS + 16 * r + col] = o[r][rd * C::NL + nl][i] * f[r];
        __syncthreads();
#pragma unroll
        for (int x = 0; x < OUT; ++x) {
          float acc = 0.f;
#pragma unroll
          for (int y = 0; y < W; ++y) acc += red[y * C::NL * 16 * ROWS + x * T + tid];
          res[rd * OUT + x] = acc;
        }
      }
      __syncthreads();
#pragma unroll
      for (int rd = 0; rd < RND; ++rd)
#pragma unroll
        for (int x = 0; x < OUT; ++x) {
          const int idx = x * T + tid, row = idx % ROWS, dc = (idx / ROWS) % 16, nl = idx / (16 * ROWS);
          red[row * C::FP + CH * dc + rd * C::NL + nl] = res[rd * OUT + x];
        }
      __syncthreads();
      const bool whole = k0 == 0 && k1 == nblk;
      float* slot = p.parts + static_cast<int64_t>(2 * blockIdx.x + (k0 > 0 ? 0 : 1)) * ROWS * (D + 2);
      for (int r = wave; r < ROWS; r += W) {
        const int tk = r / p.hb, hd = r - tk * p.hb;
        if (tk >= ntok || hd >= nh) continue;
        float top = -__builtin_inff(), ls = 0.f;
#pragma unroll
        for (int x = 0; x < W; ++x) top = fmaxf(top, *reinterpret_cast<const float*>(smem + C::ML + 8 * (x * ROWS + r)));
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const float2 ml = *reinterpret_cast<const float2*>(smem + C::ML + 8 * (x * ROWS + r));
          ls += ml.x == -__builtin_inff() ? (ml.y != ml.y ? ml.y : 0.f) : ml.y * at_exp2(ml.x - top);
        }
        float v[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = red[r * C::FP + kv_chunk(lane) * EL + e];
        if (whole) {
          at_finish<D>(p, v, ls, sq.row0 + tok0 + tk, head0 + hd, lane);
        } else {
#pragma unroll
          for (int e = 0; e < EL; ++e) slot[r * D + kv_chunk(lane) * EL + e] = v[e];
          if (lane == 0) {
            slot[ROWS * D + r] = top;
            slot[ROWS * D + ROWS + r] = ls;
          }
        }
      }
      if (!whole && k0 == 0 && tid == 0) {
        // the workgroups that go on with this unit: shares that hold the start of one of its blocks
        const int64_t last = u0 + kAtUnit + static_cast<int64_t>(nblk - 1) * 32;  // the last block's place on the line
        AttendMeta m{};
        m.parts = static_cast<int>(last / q) - static_cast<int>(blockIdx.x);
        m.row0 = sq.row0 + tok0;
        m.nrows = ntok;
        m.head0 = head0;
        m.hb = nh;
        p.meta[blockIdx.x] = m;
      }
    }
    // ---- next unit ----
    u0 += reads + kAtUnit;
    w = u0;
    if (w >= w1) break;
    if (++t == sq.tiles) {
      t = 0;
      if (++hu == hu_n) {
        hu = 0;
        do {
          ++b;
          sq = at_seq<true>(p, b);
        } while (sq.tiles == 0);
      }
    }
  }
}

template <int KB, int VB, int D, int R>
hipError_t at_launch(const AttendParams& p, hipStream_t s) {
  using C = AtCfg<KB, VB, D, R>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend<KB, VB, D, R>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attend<KB, VB, D, R>), dim3(p.grid), dim3(C::T), C::LDS, s, p);
  return hipGetLastError();
}

template <int KB, int VB>
hipError_t at_launch_d(const AttendParams& p, int R, hipStream_t s) {
  switch (p.a.c.D) {
    case 64: return R == 1 ? at_launch<KB, VB, 64, 1>(p, s) : at_launch<KB, VB, 64, 4>(p, s);
    case 128: return R == 1 ? at_launch<KB, VB, 128, 1>(p, s) : at_launch<KB, VB, 128, 4>(p, s);
    default: return R == 1 ? at_launch<KB, VB, 256, 1>(p, s) : at_launch<KB, VB, 256, 2>(p, s);
  }
}

// One key format's kernels.
template <int KB>
hipError_t at_launch_k(const AttendParams& p, int R, hipStream_t s) {
  switch (p.a.c.v.bits) {
    case 2: return at_launch_d<KB, 2>(p, R, s);
    case 3: return at_launch_d<KB, 3>(p, R, s);
    case 4: return at_launch_d<KB, 4>(p, R, s);
    default: return at_launch_d<KB, 8>(p, R, s);
  }
}

}  // namespace tq
