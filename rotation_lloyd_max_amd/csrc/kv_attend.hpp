// Attention over the paged compressed cache: the kernel (instantiated per key format in
// kv_attend_*.hip, dispatched in kv_attend.hip).
//     out = R_v^T sum_j p_j v'_j,  p = softmax_j(scale * (R_k q) . k'_j)
// with k', v' the decoded rows in the rotated bases (R orthonormal: q . k = (R q) . (R k)).
//
// Work. A unit is (sequence, key head, tile of query rows that share the head). All units lie on
// one line of work, each as long as the tokens it reads plus a constant for its set-up, cut into
// shares, one per workgroup: uneven lengths balance, and a few long sequences still fill the chip.
// With few units each is cut evenly into its own workgroups (AtWork). A cut inside a unit leaves
// partial sums in the workspace, which k_attend_join adds up in a fixed order. The schedule is made
// on the device, by every workgroup for itself: lengths and offsets may change between replays.
//
// This kernel is for few rows (tiles of 16; many: kv_attend_wide.hpp). Workgroups are small (four
// waves), so that two or three share a CU and one's set-up hides behind another's stream; the waves
// share the rows and split the tokens.
//
// A wave takes blocks of 32 tokens. Scores come as S^T = K Q^T on v_mfma_f32_16x16x32_f16: lane l
// supplies a quarter row of token l % 16 (elements D / 4 * (l / 16) + ..., one contiguous load and
// one group scale) and receives, for query row l % 16, the tokens 4 (l / 16) + i: exactly the
// layout in which P^T is the B operand of O^T += V^T P^T, so probabilities never leave their lane.
// The V operand wants eight tokens of one element per lane: lane l loads the same piece of eight
// tokens' rows (D / 16 codes at element D / 16 * (l % 16)) and pairs equal positions of two tokens
// by bit operations. Decoded values are never stored.
//
// Decoding is an LDS table of fp16 centroids. Codes of 8 bits (and pairs of 4-bit codes) use a
// table with 32 columns, entry e for lane l at 128 e + 4 (l % 32): the lanes that the LDS serves
// together never meet in a bank (2.8 cycles of a CU per wave's read; 4.7 from one copy of 256
// entries), and one v_dot4 makes the address from a byte of the word. Pairs of 3- and 2-bit codes
// need 64 and 16 entries, which lie in different banks by themselves (3.4 cycles).
//
// Group scales multiply the centroids in fp16. Scales from 2^-12 up to 2^13 enter as they are: products
// stay below fp16's largest, and what its subnormals cut is less than 2^-13 of a scale. In a block that
// holds another scale each token is held times one of two powers of two, by its own largest scale
// (kAtLoud). Keys' come off their scores in fp32; a block with values of both kinds is multiplied twice, once
// for the tokens of either kind, with the sums brought to their power of two in between. So no token costs
// its neighbours bits, seen or not, and in the common step scales cost one comparison. (32 sequences of 61
// to 8191, whole call: all scales in range 37 us, all values below 2^-12 47, one token of 64 at 3e4 45.)
//
// Softmax in base 2 with a reference that moves only when a score passes it by 2^8 (p then stays within
// fp16: 2^7 at the reference, at most 2^15, so that its subnormals cut 2^-32 of a weight), so the
// running maximum needs neither lane exchange nor rescaling in the common step. Sums are fp32. What is
// rounded to fp16 (the rotated q, centroids, their products with scales, p) is what the matrix cores
// take: half a step each, 2^-11, against 2^-8 of a bf16 output and 6e-3 that the quantization of an 8-bit
// cache costs. (More bits would take fp32 products in the decoding, two vector instructions for one, or
// twice the matrix products.)
//
// Measured, 8 key heads of 128 shared by 4 query heads, 8-bit keys and 3-bit values, kernel and join:
// one token over 337 11.1 + 3.6 us; over 131071 (193 MB) 55.0 + 7.3 us, 3.5 TB/s of the 6.0 that a
// large read reaches; 32 sequences of 61 to 8191 (82 MB) 32.8 + 4.1 us. No one part bounds the long ones:
// about 370 vector instructions for a block of 32 tokens take half of the cycles, LDS 39 %, a wave waits
// 45 % of its time (with no table reads 92 % of the time remained, with no loads 85 %): what a wave does
// for a block follows one another, and three waves per SIMD overlap it in part. The short ones are bound
// by the chain of memory latencies of schedule, q, page ids, codes and join.
#pragma once

#include "exact_div.hpp"
#include "internal.hpp"
#include "kv_lane.hpp"

namespace tq {

constexpr int kAtCus = 256;
constexpr int kAtMaxGrid = 3 * kAtCus;  // workgroups of a launch, at most
// a unit's set-up in tokens of work, and the least work of a share (32 sequences of 61 to 8191, whole
// call: set-up 96 42.9 us, 256 40.0, 448 40.2, 704 42.4; share 256 40.2, 512 40.0, 1024 42.1)
constexpr int kAtUnit = 256;
constexpr int kAtMinShare = 512;
// least blocks of a part (one token over 337 and 4096, whole call: 1 12.9 and 18.9 us, 4 12.9 and 14.5,
// 8 14.8 and 15.5, 16 16.7 and 20.5)
constexpr int kAtMinBlocks = 4;
constexpr float kAtLazy = 8.f;          // log2 of how far a score may pass the reference
// Exponents are one fused operation, score times factor minus reference. The reference was rounded, the
// fused product is not: from 2^28 on half a step of fp32 between them would take weights out of fp16. From
// this size on a row's factor is cut to a power of two, whose products are exact. (That scales score
// differences by up to 2, where the fp16 operands leave the scores themselves off by 2^-11 of 2^25.)
constexpr float kAtHuge = 0x1p25f;
constexpr float kAtNone = -3e38f;       // reference of a row that has seen nothing
// fp16 bits of scales: they enter as they are from kAtLow up to below kAtLow + kAtSpan (2^-12, 2^13). In a
// block with others (0 among them), tokens whose largest scale is from kAtLoud (2^-4) on are held times 2^-6, the rest
// times 2^12: both bring every token's largest to 2^-12 .. 2^10.
constexpr uint32_t kAtLow = 0x0c00, kAtSpan = 0x6400, kAtLoud = 0x2c00;
constexpr int kAtLoudExp = 6, kAtQuietExp = -12;

struct AttendMeta {                 // of a workgroup whose last unit goes on in the next ones
  int32_t parts;                    // following workgroups that hold a part; 0: nothing to join
  int32_t row0, nrows;              // first query row (of M) of the unit, tokens of the tile
  int32_t head0, nh, pad[3];        // first query head, heads per token
};

struct AttendParams {
  const uint32_t *kcodes, *vcodes, *ksigns, *vsigns;
  const uint16_t *kscales, *vscales;
  const uint16_t* q;
  uint16_t* out;
  const int32_t *q_offsets, *kv_lens, *page_table;
  const uint32_t* tree;
  AttendMeta* meta;
  float* parts;
  int64_t q_stride;
  int qdt, odt, q_heads, B, M, table_width, tree_words;
  int heads, pages, page;
  uint32_t page16, page_mul;        // page_tokens / 16 and ceil(2^32 / page16) (0 for 1)
  int lg_gk, lg_gv, lg_kg, lg_vg;   // log2 of scales per row and of the groups
  int share, hb, nhb, a_tok;        // query heads per key head; heads, head blocks, tokens of a tile
  uint32_t hb_mul, a_mul;           // ceil(2^16 / hb), ceil(2^32 / a_tok) (0 for 1)
  int hu_n, cap, n_each, negate;    // heads * nhb; tokens of a table row; queries without q_offsets
  float inv_sqrt_d, c1;             // c1: |scale| log2(e) / sqrt(D); 0 for scale 0
  uint16_t hk[256], hv[256];        // fp16 centroids
};

// The arguments are read where they are used, by scalar loads of the kernel's argument block:
// held in registers from the start they would not fit beside the block loop's scalars. at_again
// makes a point before which no read may be moved.
typedef const __attribute__((address_space(4))) AttendParams* AtArgs;
__device__ __forceinline__ AtArgs at_again(AtArgs p) {
  asm volatile("" : "+s"(p));
  return p;
}

template <int KB, int VB, int D>
struct AtCfg {
  static constexpr int W = 4;               // waves
  static constexpr int T = 64 * W;
  static constexpr int ROWS = 16;
  static constexpr int NS = D / 32;         // 32-element steps of a key row
  static constexpr int CH = D / 16;         // codes of a lane's piece of a value row
  static constexpr bool KWIDE = KB == 8 || (KB == 4 && VB != 8);
  static constexpr bool VWIDE = VB == 8 || (VB == 4 && KB != 8);
  static constexpr int KROW = D * KB / 8, VROW = D * VB / 8;  // row bytes
  static constexpr int KW = (KROW / 4 + 3) / 4;               // words of a quarter key row
  static constexpr int KS = D == 256 ? 2 : 1;                 // key scales of a quarter row, at most
  static constexpr int VW = (VB * CH + 31) / 32;              // words of a value piece
  static constexpr int WGS = D <= 128 ? 3 : 2;  // workgroups per CU
  static constexpr int GRID = WGS * kAtCus;
  // LDS; the joined sums take the place of q
  static constexpr int WIDE = (KWIDE || VWIDE) ? 32768 : 0;
  static constexpr int TK = WIDE, TV = TK + 1024;
  static constexpr int C1 = TV + 1024, LIM = C1 + ROWS * 4, ML = LIM + ROWS * 4, QS = ML + W * ROWS * 8;
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
// (constants go to `base`, where they become the load's immediate offset)
template <typename T>
__device__ __forceinline__ T at_get(AtPtr base, uint32_t off) {
  return *(const __attribute__((address_space(1))) T*)(base + off);
}
// x as a value the compiler knows nothing of: what is computed from it is not kept from one place
// to another
__device__ __forceinline__ int at_fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
// A row's softmax reference: mo, 7 below the score it was set by, in units of the factor fc; c1 is the
// row's own factor, which fc is unless the scores are huge.
__device__ __forceinline__ float at_ratio(float c1) {  // c1 over its power of two
  return __uint_as_float((__float_as_uint(c1) & 0x007fffffu) | 0x3f800000u);
}
__device__ __forceinline__ float at_reference(float c1, float fc, float mo) {  // mo in units of c1
  return fc == c1 ? mo : mo * at_ratio(c1);
}
// To the score x; what was summed so far is to be multiplied by the result.
__device__ __forceinline__ float at_refer(float x, float c1, float& fc, float& mo) {
  const float t = x * c1, old = at_reference(c1, fc, mo);
  const bool huge = fabsf(t) > kAtHuge;
  fc = huge ? __uint_as_float(__float_as_uint(c1) & 0x7f800000u) : c1;
  mo = x * fc - 7.f;
  return at_exp2(fminf(old - (huge ? t - 7.f : mo), 0.f));
}
// a load at any byte address
template <typename T>
__device__ __forceinline__ T at_load(AtPtr base, uint32_t off) {
  typedef T __attribute__((aligned(1))) U;
  return *(const __attribute__((address_space(1))) U*)(base + off);
}

// x / d for 0 <= x < 2^31 with mul = ceil(2^32 / d) (0 for d = 1): the product is at most one too
// large while d <= 2^12 (x (mul d - 2^32) < 2^31 d), put right by one step.
__device__ __forceinline__ int at_div(int x, int d, uint32_t mul) {
  const uint32_t u = static_cast<uint32_t>(x);
  uint32_t y = mul ? __umulhi(u, mul) : u;
  y -= static_cast<uint64_t>(y) * d > u ? 1u : 0u;
  return static_cast<int>(y);
}

// ceil(x / d) for 0 < x <= 2^27, 1 <= d <= 2^27
__device__ __forceinline__ int at_ceil_div(int x, int d) {
  return ceil_div_by(x, d, __builtin_amdgcn_rcpf(static_cast<float>(d)));
}

// ---- work ---------------------------------------------------------------------------------
// One sequence as the schedule sees it. Tile t of a head costs the tokens its last row sees and
// kAtUnit; block k of it lies kAtUnit + 32 k from the unit's begin on the line.
struct AtSeq {
  int row0, n, len, tiles;
  int flat;          // 1: every tile reads the whole length (trees; more queries than tokens)
  int64_t per_head;  // cost of all tiles of one head
  __device__ __forceinline__ int blocks() const { return len > 1 ? (len + 31) >> 5 : 1; }  // of a tile, if flat or alone
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
// What the schedule reads of a sequence: length and query rows [lo, hi).
struct AtRaw {
  int len, lo, hi;
};
__device__ __forceinline__ AtRaw at_raw(AtArgs p, int b) {
  AtRaw r;
  r.len = p->kv_lens[b];
  if (p->q_offsets) {
    r.lo = p->q_offsets[b];
    r.hi = p->q_offsets[b + 1];
  } else {
    r.lo = b * p->n_each;
    r.hi = r.lo + p->n_each;
  }
  return r;
}
__device__ __forceinline__ AtRaw at_uniform(AtRaw r) {
  return AtRaw{at_uniform(r.len), at_uniform(r.lo), at_uniform(r.hi)};
}
__device__ __forceinline__ AtSeq at_seq(AtArgs p, const AtRaw& r) {
  AtSeq s;
  const int M = p->M, a = p->a_tok;
  s.row0 = r.lo < 0 ? 0 : r.lo > M ? M : r.lo;
  const int hi = r.hi < s.row0 ? s.row0 : r.hi > M ? M : r.hi;
  s.n = hi - s.row0;
  s.len = r.len < 0 ? 0 : r.len < p->cap ? r.len : p->cap;
  s.tiles = at_div(s.n + a - 1, a, p->a_mul);
  s.flat = p->tree != nullptr || s.n > s.len ? 1 : 0;
  s.per_head = s.tiles == 0 ? 0 : at_before(s, a, s.tiles - 1) + at_reads(s, a, s.tiles - 1) + kAtUnit;
  return s;
}

template <int V>
struct AtInt {
  static constexpr int value = V;
};
// Inclusive sum over the lanes of a wave (row shifts, then the rows' last lanes broadcast).
template <int CTRL, int ROWS>
__device__ __forceinline__ int at_shift(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float at_shift(float x) {
  return __int_as_float(at_shift<CTRL, ROWS>(__float_as_int(x)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t at_shift(int64_t x) {
  return static_cast<int64_t>(at_shift<CTRL, ROWS>(static_cast<int>(x >> 32))) << 32 |
         static_cast<uint32_t>(at_shift<CTRL, ROWS>(static_cast<int>(x)));
}
template <typename T>
__device__ __forceinline__ T at_scan(T x) {
  x += at_shift<0x111, 0xf>(x);
  x += at_shift<0x112, 0xf>(x);
  x += at_shift<0x114, 0xf>(x);
  x += at_shift<0x118, 0xf>(x);
  x += at_shift<0x142, 0xa>(x);
  x += at_shift<0x143, 0xc>(x);
  return x;
}
__device__ __forceinline__ int64_t at_lane(int64_t x, int lane) {
  return static_cast<int64_t>(__builtin_amdgcn_readlane(static_cast<int>(x >> 32), lane)) << 32 |
         static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}

// A workgroup's part of the work: the sequence, head and tile it begins with, and what of the line.
struct AtWork {
  bool own;          // cut unit by unit: this is part `part` of np; else [w, w1) of the line
  int b, hu, t, part, np;
  AtSeq sq;
  int64_t q, w, w1, u0;  // shares of the line; the unit's begin on it
  // what steers a wave is the same in all its lanes; said so, it lives in scalar registers
  __device__ __forceinline__ void uniform() {
    w = at_uniform(w);
    u0 = at_uniform(u0);
    b = at_uniform(b);
    hu = at_uniform(hu);
    t = at_uniform(t);
    sq.row0 = at_uniform(sq.row0);
    sq.n = at_uniform(sq.n);
    sq.len = at_uniform(sq.len);
    sq.tiles = at_uniform(sq.tiles);
    sq.flat = at_uniform(sq.flat);
  }
  // the blocks [k0, k1) of the unit's nblk that are this workgroup's
  __device__ __forceinline__ void blocks(int reads, int nblk, int& k0, int& k1) const {
    if (own) {
      const int each = at_ceil_div(nblk, np);  // evenly; the last part may be short or empty
      k0 = part * each < nblk ? part * each : nblk;
      k1 = k0 + each < nblk ? k0 + each : nblk;
    } else {
      const int64_t x0 = w - u0 - kAtUnit, x1 = w1 - u0 - kAtUnit < reads ? w1 - u0 - kAtUnit : reads;
      k0 = x0 <= 0 ? 0 : static_cast<int>((x0 + 31) >> 5);
      k1 = x1 <= 0 ? 0 : static_cast<int>((x1 + 31) >> 5);
    }
    k0 = at_uniform(k0);
    k1 = at_uniform(k1);
  }
  // the workgroups that go on with this unit: its other parts, or the shares of the line that hold
  // the begin of one of its blocks
  __device__ __forceinline__ int more(int nblk, int wg) const {
    return own ? at_ceil_div(nblk, at_ceil_div(nblk, np)) - 1
               : static_cast<int>((u0 + kAtUnit + static_cast<int64_t>(nblk - 1) * 32) / q) - wg;
  }
  // to the next unit, if any of it is this workgroup's
  __device__ __forceinline__ bool next(AtArgs p, int reads, int hu_n) {
    if (own) return false;
    u0 += reads + kAtUnit;
    w = u0;
    if (w >= w1) return false;
    if (++t == sq.tiles) {
      t = 0;
      if (++hu == hu_n) {
        hu = 0;
        do {
          ++b;
          sq = at_seq(p, at_uniform(at_raw(p, b)));
        } while (sq.tiles == 0);
      }
    }
    return true;
  }
};

// Workgroup wg's part of GRID, found by every wave for itself: a scan over the sequences' costs, a
// lane taking `per` neighbouring ones from b0 on, of which raw0 is the first. False: nothing to do.
template <int GRID>
__device__ __forceinline__ bool at_plan(AtArgs p, int wg, int lane, int per, int b0, const AtRaw& raw0, AtWork& o) {
  const int a_tok = p->a_tok, hu_n = p->hu_n;
  const AtSeq seq0 = at_seq(p, raw0);
  const int b1 = b0 + per < p->B ? b0 + per : p->B;
  // units and blocks of the lane's sequences; even: every tile of a head costs the same
  int units = 0;
  float blocks = 0.f;
  bool even = true;
  for (int b = b0; b < b1; ++b) {
    const AtSeq x = b == b0 ? seq0 : at_seq(p, at_raw(p, b));
    const int u = x.tiles * hu_n;
    units = units + u < GRID ? units + u : GRID;
    blocks += static_cast<float>(u) * static_cast<float>(x.blocks());
    even = even && (x.flat || x.tiles <= 1);
  }
  const int all_units = __builtin_amdgcn_readlane(at_scan(units), 63);
  // With few units, each is cut into parts of at most `chunk` blocks, one part per workgroup:
  // sum ceil(blocks / chunk) <= sum blocks / chunk + units <= GRID (the sum in fp32 is rounded up).
  // Otherwise the line is cut every q. Parts start sooner, shares balance better; whole call with
  // either, 4096 tokens, units of workgroups: 8 of 768 14 and 20 us, 64 of 768 28 and 31, 256 of 768
  // 60 and 56; tiles of 128, 32 of 256 44 and 50, 64 of 256 50 and 47.
  o.own = !__any(!even) && all_units <= GRID / 6;
  const bool own = o.own;
  int chunk = 0;
  int64_t q = 0, w0, w1, excl;
  int src;
  if (own) {
    const float all = at_scan(blocks) * (1.f + 0x1p-16f) / static_cast<float>(GRID - all_units);
    chunk = static_cast<int>(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(all), 63))) + 1;
    chunk = chunk < kAtMinBlocks ? kAtMinBlocks : chunk;
    int parts = 0;
    for (int b = b0; b < b1; ++b) {
      const AtSeq x = b == b0 ? seq0 : at_seq(p, at_raw(p, b));
      parts += x.tiles * hu_n * at_ceil_div(x.blocks(), chunk);
    }
    const int incl = at_scan(parts);
    w0 = wg;
    w1 = wg + 1;
    if (wg >= __builtin_amdgcn_readlane(incl, 63)) return false;
    src = __builtin_ctzll(__ballot(incl > wg));
    excl = __builtin_amdgcn_readlane(incl - parts, src);
  } else {
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += (b == b0 ? seq0 : at_seq(p, at_raw(p, b))).per_head * hu_n;
    const int64_t incl = at_scan(sum), total = at_lane(incl, 63);
    q = total / GRID + 1;
    q = q < kAtMinShare ? kAtMinShare : q;
    w0 = q * wg;
    w1 = w0 + q < total ? w0 + q : total;
    if (w0 >= total) return false;
    src = __builtin_ctzll(__ballot(incl > w0));
    excl = at_lane(incl - sum, src);
  }
  // the sequence, among those of the lane that holds w0
  int64_t rem = at_uniform(w0 - excl);
  int b = src * per;
  AtSeq sq = at_seq(p, AtRaw{__builtin_amdgcn_readlane(raw0.len, src), __builtin_amdgcn_readlane(raw0.lo, src),
                             __builtin_amdgcn_readlane(raw0.hi, src)});
  auto work_of = [&](const AtSeq& x) {
    return own ? static_cast<int64_t>(x.tiles * hu_n * at_ceil_div(x.blocks(), chunk)) : x.per_head * hu_n;
  };
  if (per > 1)
    for (int64_t x = work_of(sq); rem >= x; x = work_of(sq)) {
      rem = at_uniform(rem - x);
      ++b;
      sq = at_seq(p, at_uniform(at_raw(p, b)));
    }
  int hu, t, part = 0, np = 1;
  int64_t u0 = 0;  // the unit's begin on the line
  if (own) {
    np = at_uniform(at_ceil_div(sq.blocks(), chunk));
    const int unit = at_uniform(at_ceil_div(static_cast<int>(rem) + 1, np) - 1);
    part = static_cast<int>(rem) - unit * np;
    hu = sq.tiles == 1 ? unit : at_ceil_div(unit + 1, sq.tiles) - 1;
    t = unit - hu * sq.tiles;
  } else {
    // rem < 2^53, so the quotient in fp64 is at most one off
    hu = static_cast<int>(static_cast<double>(rem) / static_cast<double>(sq.per_head));
    hu -= hu * sq.per_head > rem ? 1 : 0;
    hu += (hu + 1) * sq.per_head <= rem ? 1 : 0;
    rem -= hu * sq.per_head;
    int lo = 0, hi = sq.tiles - 1;  // last tile with at_before <= rem
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (at_before(sq, a_tok, mid) <= rem) lo = mid;
      else hi = mid - 1;
    }
    t = lo;
    u0 = w0 - (rem - at_before(sq, a_tok, t));
  }
  o.q = q; o.w = w0; o.w1 = w1; o.u0 = u0;
  o.b = b; o.hu = hu; o.t = t; o.part = part; o.np = np;
  o.sq = sq;
  return true;
}

// The centroid tables. A wave's entries are uniform: scalar loads of the arguments, two 128-byte
// rows per store.
template <typename C, int KB, int VB>
__device__ __forceinline__ void at_tables(AtArgs p, char* smem, int tid, int lane, int wave) {
  if constexpr (C::WIDE > 0) {
    constexpr int TB = KB == 8 || VB == 8 ? 8 : 4;
    const __attribute__((address_space(4))) uint16_t* hc = KB == TB ? p->hk : p->hv;
    constexpr int PW = 256 / C::W;
#pragma unroll
    for (int k = 0; k < PW; k += 2) {
      const int e = wave * PW + k;
      const uint32_t x = TB == 8 ? hc[e] : (hc[e & 15] | static_cast<uint32_t>(hc[e >> 4]) << 16);
      const uint32_t y = TB == 8 ? hc[e + 1] : (hc[(e + 1) & 15] | static_cast<uint32_t>(hc[e >> 4]) << 16);
      *reinterpret_cast<uint32_t*>(smem + 128 * e + 4 * lane) = lane < 32 ? x : y;
    }
  }
  if constexpr (KB < 8 && !C::KWIDE)
    for (int e = tid; e < (1 << (2 * KB)); e += C::T)
      *reinterpret_cast<uint32_t*>(smem + C::TK + 4 * e) =
          p->hk[e & ((1 << KB) - 1)] | static_cast<uint32_t>(p->hk[e >> KB]) << 16;
  if constexpr (VB < 8 && !C::VWIDE)
    for (int e = tid; e < (1 << (2 * VB)); e += C::T)
      *reinterpret_cast<uint32_t*>(smem + C::TV + 4 * e) =
          p->hv[e & ((1 << VB) - 1)] | static_cast<uint32_t>(p->hv[e >> VB]) << 16;

}

// Rows of a tile as a wave takes them in and out: N at a time, each on D / 8 lanes, eight elements
// of a lane (kv_lane.hpp). A row on the whole wave costs four times the instructions: what is done
// once per row is then done by every lane for one row only.
template <int D>
struct AtRows {
  static constexpr int LR = D / 8, N = 64 / LR;
  int sub, c;  // the lane's row of the N, its chunk
  __device__ __forceinline__ AtRows() {
    const int lane = at_fresh(threadIdx.x & 63);
    sub = lane / LR;
    c = kv_chunk(lane & (LR - 1));
  }
  __device__ __forceinline__ uint32_t signs(const uint32_t* bits) const { return (bits[c >> 2] >> (8 * (c & 3))) & 0xffu; }
  __device__ __forceinline__ static float most(float x) {  // the maximum over the row's lanes
    x = fmaxf(x, kv_swap<0>(x));
    x = fmaxf(x, kv_swap<1>(x));
    x = fmaxf(x, kv_swap<2>(x));
    if constexpr (LR >= 16) x = fmaxf(x, kv_swap<3>(x));
    if constexpr (LR >= 32) {
      float a, b;
      kv_both<4>(x, a, b);
      x = fmaxf(a, b);
    }
    return x;
  }
};

// A tile's queries: rotated, scaled by a power of two to fp16's upper range, into LDS as rows of QP
// bytes, with each row's score factor and the token its mask ends at (a tree's: begins at).
template <int D>
struct AtQuery : AtRows<D> {
  int tok0, ntok, nh, hb, row0, head0;
  uint32_t hb_mul;
  uint32_t sg;
  float c1;
  u32x4_t raw;
  __device__ __forceinline__ AtQuery(AtArgs p, int row0_, int head0_, int tok0_, int ntok_, int nh_)
      : tok0(tok0_), ntok(ntok_), nh(nh_), hb(p->hb), row0(row0_), head0(head0_), hb_mul(p->hb_mul),
        sg(this->signs(p->ksigns)), c1(p->c1) {}
  // whether row r of the tile is a query's
  __device__ __forceinline__ bool row(int r, int& tk, int& hd) const {
    tk = (static_cast<uint32_t>(r) * hb_mul) >> 16;
    hd = r - tk * hb;
    return tk < ntok && hd < nh;
  }
  __device__ __forceinline__ void load(AtArgs p, int r0) {
    int tk, hd;
    const bool ok = row(r0 + this->sub, tk, hd);
    raw = *reinterpret_cast<const u32x4_t*>(p->q + (static_cast<int64_t>(row0) + (ok ? tk : 0)) * p->q_stride +
                                            static_cast<int64_t>(head0 + (ok ? hd : 0)) * D + 8 * this->c);
  }
  // the rows loaded last, rows r0 on; those from `next` on are loaded meanwhile (next < 0: none)
  __device__ __forceinline__ void rotate(AtArgs p, char* smem, int r0, int dst, int QP, int C1, int LIM, int before, int len, int next) {
    const int c = this->c, r = r0 + this->sub, qdt = p->qdt;
    int tk, hd;
    const bool ok = row(r, tk, hd), use = ok && c1 != 0.f;
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8], mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint16_t x = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
      const float y = qdt == 1 ? bf16_bits_to_float(x) : half_bits_to_float(x);
      v[e] = !use ? 0.f : (sg >> e) & 1u ? -y : y;
    }
    if (next >= 0) load(p, next);
    kv_transform<D>(v, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
    mx = this->most(mx);
    // the largest magnitude comes to [2^13, 2^14): exponent 127 + 13 of the scaled value
    const int ex = static_cast<int>(__float_as_uint(mx) >> 23);
    int k = mx > 0.f && ex < 255 ? 140 - ex : 0;
    k = k > 100 ? 100 : k;
    const bool neg = (kv_sign(c) != 0) != (p->negate != 0);  // the transform's sign, and the scale's
    const float f = __uint_as_float(static_cast<uint32_t>(127 + k) << 23 | (neg ? 0x80000000u : 0u));
    uint32_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const half2_t x{static_cast<_Float16>(v[2 * e] * f), static_cast<_Float16>(v[2 * e + 1] * f)};
      y[e] = __builtin_bit_cast(uint32_t, x);
    }
    *reinterpret_cast<u32x4_t*>(smem + dst + this->sub * QP + 16 * c) = u32x4_t{y[0], y[1], y[2], y[3]};
    if (c == 0) {
      *reinterpret_cast<float*>(smem + C1 + 4 * r) = c1 == 0.f ? 1.f : c1 * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      int lim = p->tree ? before : before + tok0 + tk + 1;
      lim = lim < 0 ? 0 : lim;
      *reinterpret_cast<int*>(smem + LIM + 4 * r) = !ok || lim > len ? len : lim;
    }
  }
};

// The lane's part v of a row's sums, l the sum of its weights: normalised, rotated back and (if ok)
// stored.
template <int D, typename P>
__device__ __forceinline__ void at_store(P p, float (&v)[8], float l, int64_t m, int head, uint32_t sg, int c, bool ok) {
  const float f = p->inv_sqrt_d / l;
  sg ^= 0u - kv_sign(c);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = l == 0.f ? 0.f : v[e] * f;
  kv_transform<D>(v, c);
  const int odt = p->odt;
  uint32_t x[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = (sg >> e) & 1u ? -v[e] : v[e];
    const uint32_t b = odt == 1 ? float_to_bf16_rne(y) : float_to_half_rne(y);
    x[e >> 1] = e & 1 ? x[e >> 1] | b << 16 : b;
  }
  if (ok) *reinterpret_cast<u32x4_t*>(p->out + (m * p->q_heads + head) * D + 8 * c) = u32x4_t{x[0], x[1], x[2], x[3]};
}

// The lowest n bits; none for n <= 0, all from 32 on.
__device__ __forceinline__ uint32_t at_low(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// The tokens j0 .. j0 + 31 that row `row` of the tile sees, as bits: those before lim and, of a tree,
// those of its mask's words. row0: first query row of the tile, ntok its tokens.
__device__ __forceinline__ uint32_t at_seen(AtArgs p, int lim, int j0, int before, int len, int row0, int row, int ntok) {
  uint32_t see = at_low(lim - j0);
  if (p->tree) {
    const int tk = (static_cast<uint32_t>(row) * p->hb_mul) >> 16, words = p->tree_words;
    const uint32_t* bits = p->tree + static_cast<int64_t>(row0 + (tk < ntok ? tk : 0)) * words;
    const int w = (j0 - before) >> 5, sh = (j0 - before) & 31;
    const uint32_t w0 = w >= 0 && w < words ? bits[w] : 0u, w1 = w >= -1 && w + 1 < words ? bits[w + 1] : 0u;
    see |= static_cast<uint32_t>((static_cast<uint64_t>(w1) << 32 | w0) >> sh) & at_low(len - j0);
  }
  return see;
}

// The lane's part of a row's sums into a slot of the workspace: [rows][D] sums, references, weights.
template <int D>
__device__ __forceinline__ void at_put(float* slot, int rows, int r, int c, const float (&v)[8], float top, float l) {
  f32x4_t* const dst = reinterpret_cast<f32x4_t*>(slot + r * D + 8 * c);
  dst[0] = f32x4_t{v[0], v[1], v[2], v[3]};
  dst[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  if (c == 0) {
    slot[rows * D + r] = top;
    slot[rows * D + rows + r] = l;
  }
}

// ---- decoding -----------------------------------------------------------------------------
// the larger of each half, as unsigned numbers
typedef uint16_t AtU16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t at_max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(AtU16x2, a), __builtin_bit_cast(AtU16x2, b)));
}
// how far two scales lie above kAtLow, those below it farthest; in range: less than kAtSpan
__device__ __forceinline__ uint32_t at_range(uint32_t pair) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(AtU16x2, pair) - __builtin_bit_cast(AtU16x2, kAtLow | kAtLow << 16));
}
// whether a scale of any lane's four pairs is out of range (a wave's answer)
__device__ __forceinline__ bool at_far(const uint32_t (&pair)[4]) {
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) big = at_max_u16(at_range(pair[i]), big);
  big = big > (big << 16) ? big : big << 16;
  return __any(big >= (kAtSpan << 16));
}
// Which of the 16 tokens of a half block are loud, lane l holding the largest of its scales (without
// sign) of token l % 16.
__device__ __forceinline__ uint32_t at_loud(uint32_t largest) {
  uint64_t who = __ballot(largest >= kAtLoud);
  who |= who >> 32;
  return static_cast<uint32_t>(who | who >> 16) & 0xffffu;
}
// a if the bit is set, else b, by bit operations (a comparison per bit would take a pair of scalar
// registers each)
__device__ __forceinline__ float at_pick(uint32_t bits, int bit, float a, float b) {
  const uint32_t m = static_cast<uint32_t>(static_cast<int32_t>(bits << (31 - bit)) >> 31);
  return __uint_as_float((__float_as_uint(a) & m) | (__float_as_uint(b) & ~m));
}
// The lane's scores of a half block back from the power of two of their tokens' keys; loud: bits of its
// 16 tokens.
__device__ __forceinline__ void at_back(f32x4_t& s, uint32_t loud, int h) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s[i] *= at_pick(loud >> (4 * h), i, static_cast<float>(1 << kAtLoudExp), 1.f / static_cast<float>(1 << -kAtQuietExp));
}
__device__ __forceinline__ uint32_t at_mul(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, a) * __builtin_bit_cast(half2_t, b));
}
// 2^-e in both halves, -15 <= e <= 14
__device__ __forceinline__ uint32_t at_pow2(int e) { return static_cast<uint32_t>(15 - e) * 0x04000400u; }
__device__ __forceinline__ f32x4_t at_mfma(const uint32_t (&a)[4], const uint32_t (&b)[4], f32x4_t c) {
  const u32x4_t x{a[0], a[1], a[2], a[3]}, y{b[0], b[1], b[2], b[3]};
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, x), __builtin_bit_cast(f16x8_t, y), c, 0, 0, 0);
}

// The table reads for eight key codes (number st of the lane's quarter row): one per code of 8
// bits, one per pair of smaller ones.
template <int KB>
struct AtLook {
  static constexpr int N = KB == 8 ? 8 : 4;
  uint32_t t[N];
};
template <typename C, int KB>
__device__ __forceinline__ void at_look_k(const uint32_t* w, int st, uint32_t lane4, AtLook<KB>& o) {
  if constexpr (KB == 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) o.t[k] = at_lds(at_byte<128>(w[2 * st + (k >> 2)], k & 3, lane4));
  } else if constexpr (KB == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (C::KWIDE) o.t[k] = at_lds(at_byte<128>(w[st], k, lane4));
      else o.t[k] = at_lds(C::TK + at_byte<4>(w[st], k, 0));
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
      o.t[k] = at_lds(C::TK + (x & M));
    }
  }
}
// What was read as four fp16 pairs, times the scale.
template <int KB>
__device__ __forceinline__ void at_pairs_k(const AtLook<KB>& x, uint32_t scale, uint32_t (&o)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = at_mul(KB == 8 ? at_pack(x.t[(2 * k) % AtLook<KB>::N], x.t[(2 * k + 1) % AtLook<KB>::N]) : x.t[k], scale);
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

// A block's codes and scales as loaded: a quarter row of token l % 16 of each half for the scores,
// a piece of eight tokens' rows for the sums.
template <typename C>
struct AtBlock {
  uint32_t k[2][C::KW], v[8][C::VW], ks[2][C::KS], vs[8];  // vs: see load_v and pair_scales
  uint32_t bad;  // uniform; bit x: the page of half x is none
};

template <int KB, int VB, int D>
__global__ __launch_bounds__((AtCfg<KB, VB, D>::T), (AtCfg<KB, VB, D>::WGS * AtCfg<KB, VB, D>::W / 4)) void k_attend(AttendParams) {
  using C = AtCfg<KB, VB, D>;
  constexpr int W = C::W, T = C::T, ROWS = C::ROWS, NS = C::NS, CH = C::CH;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  AtArgs p = (AtArgs)__builtin_amdgcn_kernarg_segment_ptr();
  const int tid = threadIdx.x, lane = tid & 63, wave = at_uniform(tid >> 6);
  const int col = lane & 15, h = lane >> 4;
  const uint32_t lane4 = (lane & 31) * 4;
  const int wg = blockIdx.x;

  const int per = (p->B + 63) >> 6;
  const int b0 = lane * per;
  AtRaw raw0{0, 0, 0};
  if (b0 < p->B) raw0 = at_raw(p, b0);

  at_tables<C, KB, VB>(p, smem, tid, lane, wave);  // while those loads are on their way
  const int a_tok = p->a_tok, hu_n = p->hu_n;
  if (tid == 0) p->meta[wg].parts = 0;
  AtWork wk;
  if (!at_plan<C::GRID>(p, wg, lane, per, b0, raw0, wk)) return;

  const uint32_t koff = col * C::KROW + (C::KROW / 4) * h;
  const uint32_t voff = 4 * h * C::VROW + (VB * CH * col) / 8, vback = voff - (col == 15 ? 1 : 0);
  // scales of the quarter row's first and (D = 256) second half, and of the value piece
  const uint32_t ksoff = ((col << p->lg_gk) + ((D / 4 * h) >> p->lg_kg)) * 2;
  const uint32_t ksoff2 = ((col << p->lg_gk) + ((D / 4 * h + D / 8) >> p->lg_kg)) * 2;
  const uint32_t vsoff = ((4 * h << p->lg_gv) + ((col * CH) >> p->lg_vg)) * 2;

  while (true) {
    wk.uniform();
    p = at_again(p);
    const int reads = at_reads(wk.sq, a_tok, wk.t);
    const int nblk = (reads + 31) >> 5;
    int k0, k1;
    wk.blocks(reads, nblk, k0, k1);
    const AtSeq& sq = wk.sq;
    const int hu = wk.hu, t = wk.t, b = wk.b;
    if (k0 < k1) {
      const int kh = p->nhb == 1 ? hu : hu / p->nhb, hblk = hu - kh * p->nhb;
      const int hb = p->hb, head0 = kh * p->share + hblk * hb;
      const int nh = p->share - hblk * hb < hb ? p->share - hblk * hb : hb;
      const int tok0 = t * a_tok;
      const int ntok = sq.n - tok0 < a_tok ? sq.n - tok0 : a_tok;
      const int before = sq.len - sq.n;
      const int len = sq.len;

      // ---- the stream of blocks ----
      const int page = p->page, pages = p->pages;
      const uint32_t page16 = p->page16, page_mul = p->page_mul;
      const uint32_t prow = static_cast<uint32_t>(p->heads) * page;
      const int lgk = p->lg_gk, lgv = p->lg_gv;
      const char* const kcodes = reinterpret_cast<const char*>(p->kcodes) + static_cast<int64_t>(kh) * page * C::KROW;
      const char* const vcodes = reinterpret_cast<const char*>(p->vcodes) + static_cast<int64_t>(kh) * page * C::VROW;
      const char* const kscales = reinterpret_cast<const char*>(p->kscales) + ((static_cast<int64_t>(kh) * page) << (lgk + 1));
      const char* const vscales = reinterpret_cast<const char*>(p->vscales) + ((static_cast<int64_t>(kh) * page) << (lgv + 1));
      // page ids of a block's halves (a half past the end stands for the first one), read one
      // block ahead; constant memory, so that they come by scalar loads
      typedef const int32_t __attribute__((address_space(4))) * ConstIds;
      const ConstIds ids = (ConstIds)reinterpret_cast<uintptr_t>(p->page_table + static_cast<int64_t>(b) * p->table_width);
      int id[2] = {}, in[2] = {};
      auto look = [&](int blk) {
        const int j = blk * 32, j2 = j + 16 < len ? j + 16 : j;
        const int pi = at_div(j >> 4, page16, page_mul), pi2 = at_div(j2 >> 4, page16, page_mul);
        in[0] = j - pi * page;
        in[1] = j2 - pi2 * page;
        id[0] = len > 0 ? ids[pi] : -1;
        id[1] = len > 0 ? ids[pi2] : -1;
      };
      int64_t row_of[2] = {};
      auto locate = [&](AtBlock<C>& x) {
        x.bad = 0;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const bool none = static_cast<uint32_t>(id[y]) >= static_cast<uint32_t>(pages);
          x.bad |= none ? 1u << y : 0u;
          row_of[y] = static_cast<int64_t>(static_cast<uint64_t>(none ? 0u : static_cast<uint32_t>(id[y])) * prow) + in[y];
        }
      };
      auto load_k = [&](AtBlock<C>& x) {
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
          const AtPtr kc = at_base(kcodes, row_of[sb] * C::KROW);
          constexpr int L = C::KW % 4 == 0 ? 4 : C::KW % 3 == 0 ? 3 : C::KW % 2 == 0 ? 2 : 1;  // words of a load
          if constexpr (C::KROW % 16 != 0) {  // six bytes
            x.k[sb][0] = at_load<uint32_t>(kc, koff);
            x.k[sb][1] = at_load<uint16_t>(kc + 4, koff);
          } else {
#pragma unroll
            for (int k = 0; k < C::KW; k += L) {
              if constexpr (L == 4) {
                const u32x4_t y = at_get<u32x4_t>(kc + 4 * k, koff);
                x.k[sb][k] = y.x; x.k[sb][k + 1] = y.y; x.k[sb][k + 2] = y.z; x.k[sb][k + 3] = y.w;
              } else if constexpr (L == 3) {
                const u32x3_t y = at_get<u32x3_t>(kc + 4 * k, koff);
                x.k[sb][k] = y.x; x.k[sb][k + 1] = y.y; x.k[sb][k + 2] = y.z;
              } else if constexpr (L == 2) {
                const u32x2_t y = at_get<u32x2_t>(kc + 4 * k, koff);
                x.k[sb][k] = y.x; x.k[sb][k + 1] = y.y;
              } else {
                x.k[sb][k] = at_get<uint32_t>(kc + 4 * k, koff);
              }
            }
          }
          const AtPtr sp = at_base(kscales, row_of[sb] << (lgk + 1));
          x.ks[sb][0] = at_get<uint16_t>(sp, ksoff);
          if constexpr (C::KS == 2) x.ks[sb][1] = at_get<uint16_t>(sp, ksoff2);
        }
      };
      auto load_v = [&](AtBlock<C>& x) {
        auto one = [&](auto half) {
          constexpr int sb = decltype(half)::value;
          const AtPtr vc = at_base(vcodes, row_of[sb] * C::VROW);
          const AtPtr sp = at_base(vscales, row_of[sb] << (lgv + 1));
#pragma unroll
          for (int i = 4 * sb; i < 4 * sb + 4; ++i) {
            const AtPtr vr = vc + (i & 3) * C::VROW;
            if constexpr (VB == 3) {
              // a piece of 12, 24 or 48 bits; of 24, the row's last one is read one byte earlier,
              // inside the row (shifted down where it is used)
              if constexpr (CH == 4) {
                x.v[i][0] = at_load<uint16_t>(vr, voff);
              } else if constexpr (CH == 8) {
                x.v[i][0] = at_load<uint32_t>(vr, vback);
              } else {
                x.v[i][0] = at_load<uint32_t>(vr, voff);
                x.v[i][1] = at_load<uint16_t>(vr + 4, voff);
              }
            } else if constexpr (VB * CH == 8) {
              x.v[i][0] = at_get<uint8_t>(vr, voff);
            } else if constexpr (VB * CH == 16) {
              x.v[i][0] = at_get<uint16_t>(vr, voff);
            } else if constexpr (C::VW == 4) {
              const u32x4_t y = at_get<u32x4_t>(vr, voff);
              x.v[i][0] = y.x; x.v[i][1] = y.y; x.v[i][2] = y.z; x.v[i][3] = y.w;
            } else if constexpr (C::VW == 2) {
              const u32x2_t y = at_get<u32x2_t>(vr, voff);
              x.v[i][0] = y.x; x.v[i][1] = y.y;
            } else {
              x.v[i][0] = at_get<uint32_t>(vr, voff);
            }
          }
          // scales of the four tokens: all groups' of up to two, else of the piece's group alone;
          // nothing is done to them here, which would wait for the loads
          uint32_t y0, y1, y2 = 0, y3 = 0;
          if (lgv == 0) {
            const u32x2_t y = at_get<u32x2_t>(sp, 8 * h);
            y0 = y.x; y1 = y.y;
          } else if (lgv == 1) {
            typedef uint32_t U4 __attribute__((ext_vector_type(4), aligned(8)));
            const U4 y = at_get<U4>(sp, 16 * h);
            y0 = y.x; y1 = y.y; y2 = y.z; y3 = y.w;
          } else {
            y0 = at_get<uint16_t>(sp, vsoff);
            y1 = at_get<uint16_t>(sp + (2 << lgv), vsoff);
            y2 = at_get<uint16_t>(sp + (4 << lgv), vsoff);
            y3 = at_get<uint16_t>(sp + (6 << lgv), vsoff);
          }
          x.vs[4 * sb] = y0; x.vs[4 * sb + 1] = y1; x.vs[4 * sb + 2] = y2; x.vs[4 * sb + 3] = y3;
        };
        one(AtInt<0>{});
        one(AtInt<1>{});
      };
      // the scales of the piece's group, tokens 2 i and 2 i + 1 in a word
      const uint32_t vsel = ((col * CH) >> p->lg_vg) & 1 ? 0x07060302u : 0x05040100u;
      auto pair_scales = [&](const AtBlock<C>& x, uint32_t (&o)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t pair = x.vs[4 * (i >> 1) + (i & 1)];
          const uint32_t a = x.vs[4 * (i >> 1) + 2 * (i & 1)], c = x.vs[4 * (i >> 1) + 2 * (i & 1) + 1];
          o[i] = lgv == 0 ? pair : __builtin_amdgcn_perm(c, a, lgv == 1 ? vsel : 0x05040100u);
        }
      };
      // ---- q: rotated, scaled by a power of two to fp16's upper range, into LDS ----
      AtQuery<D> qs(p, sq.row0 + tok0, head0, tok0, ntok, nh);
      constexpr int RN = AtRows<D>::N;  // rows of a wave at a time
      if (wave * RN < ROWS) qs.load(p, wave * RN);
      AtBlock<C> blk0 = {};
      int blk = k0 + wave;
      if (blk < k1) {
        look(blk);
        locate(blk0);
        load_k(blk0);
        load_v(blk0);
        if (blk + W < k1) look(blk + W);
      }

      const bool masked = p->tree != nullptr;
      __syncthreads();  // the last unit's readers of this memory are done
#pragma unroll 1
      for (int r0 = wave * RN; r0 < ROWS; r0 += W * RN)
        qs.rotate(p, smem, r0, C::QS + r0 * C::QP, C::QP, C::C1, C::LIM, before, len, r0 + W * RN < ROWS ? r0 + W * RN : -1);
      __syncthreads();
      // from this token on some row's mask may cut
      int cut = masked ? before : before + tok0 + 1;
      cut = cut < 0 ? 0 : cut;

      float fc = *reinterpret_cast<const float*>(smem + C::C1 + 4 * col);  // score factor
      float mo = kAtNone, l = 0.f;                                         // reference - 7; sum
      int oexp = 0;                                                        // the sums are held times 2^-oexp
      f32x4_t o[CH];
#pragma unroll
      for (int n = 0; n < CH; ++n) o[n] = f32x4_t{0.f, 0.f, 0.f, 0.f};

      auto scores = [&](AtBlock<C>& x, int blk, f32x4_t (&s)[2]) {
        if (blk * 32 + 32 > len || x.bad) {  // rows that hold no token hold anything: as if 1
          const int j = blk * 32 + (at_fresh(threadIdx.x & 63) & 15);
#pragma unroll
          for (int sb = 0; sb < 2; ++sb)
#pragma unroll
            for (int y = 0; y < C::KS; ++y)
              x.ks[sb][y] = j + 16 * sb < len && !((x.bad >> sb) & 1u) ? x.ks[sb][y] : 0x3c00u;
        }
        uint32_t kd[2][C::KS];  // scales in both halves
        uint32_t far = 0;
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
#pragma unroll
          for (int y = 0; y < C::KS; ++y) {
            kd[sb][y] = x.ks[sb][y] | (x.ks[sb][y] << 16);
            const uint32_t z = x.ks[sb][y] - kAtLow;
            far = z > far ? z : far;
          }
        const bool apart = __any(far >= kAtSpan);
        auto loud = [&](int sb) {
          return at_loud((C::KS == 2 && (x.ks[sb][C::KS - 1] & 0x7fffu) > (x.ks[sb][0] & 0x7fffu) ? x.ks[sb][C::KS - 1] : x.ks[sb][0]) & 0x7fffu);
        };
        if (__builtin_expect(apart, 0)) {
#pragma unroll
          for (int sb = 0; sb < 2; ++sb) {
            const uint32_t f = (loud(sb) >> col) & 1u ? at_pow2(kAtLoudExp) : at_pow2(kAtQuietExp);
#pragma unroll
            for (int y = 0; y < C::KS; ++y) kd[sb][y] = at_mul(kd[sb][y], f);
          }
        }
        s[0] = s[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        // the next step's table reads are on their way while this one's results are multiplied
        constexpr int PF = 1;
        AtLook<KB> ring[PF + 1];
#pragma unroll
        for (int y = 0; y < PF; ++y) at_look_k<C, KB>(x.k[y / NS], y % NS, lane4, ring[y]);
#pragma unroll
        for (int y = 0; y < 2 * NS; ++y) {
          const int sb = y / NS, st = y % NS;
          if (y + PF < 2 * NS) at_look_k<C, KB>(x.k[(y + PF) / NS], (y + PF) % NS, lane4, ring[(y + PF) % (PF + 1)]);
          const u32x4_t qv = *reinterpret_cast<const u32x4_t*>(smem + C::QS + col * C::QP + (D / 2) * h + 16 * st);
          __builtin_amdgcn_sched_barrier(0);
          uint32_t a[4];
          at_pairs_k<KB>(ring[y % (PF + 1)], kd[sb][C::KS == 2 ? st / (NS / 2) : 0], a);
          const uint32_t qb[4] = {qv.x, qv.y, qv.z, qv.w};
          s[sb] = at_mfma(a, qb, s[sb]);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (__builtin_expect(apart, 0)) {
          at_back(s[0], loud(0), h);
          at_back(s[1], loud(1), h);
        }
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
          if ((x.bad >> sb) & 1u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[sb][i] = __builtin_nanf("");
          }
      };
      auto softmax = [&](const f32x4_t (&s)[2], uint32_t (&pb)[4]) {
        // against a lazily moved reference
        const float mx = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                               fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        if (__any(__builtin_fmaf(mx, fc, -mo) > 7.f + kAtLazy)) {
          const float c1 = *reinterpret_cast<const float*>(smem + C::C1 + 4 * col);
          float x, y;
          kv_both<4>(mx, x, y);
          kv_both<5>(fmaxf(x, y), x, y);
          x = fmaxf(x, y);
          if (__builtin_fmaf(x, fc, -mo) > 7.f + kAtLazy) {  // the same in the four lanes of a row
            const float f = at_refer(x, c1, fc, mo);
            l *= f;
#pragma unroll
            for (int n = 0; n < CH; ++n) o[n] *= f;
          }
        }
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = at_exp2(__builtin_fmaf(s[i >> 2][i & 3], fc, -mo));
        l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const half2_t x{static_cast<_Float16>(e[2 * i]), static_cast<_Float16>(e[2 * i + 1])};
          pb[i] = __builtin_bit_cast(uint32_t, x);
        }
      };
      auto values = [&](AtBlock<C>& x, const uint32_t (&vs)[4], const uint32_t (&pb)[4]) {
        if constexpr (VB == 3) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if constexpr (CH == 4) x.v[i][0] >>= 4 * (col & 1);
            else if constexpr (CH == 8) x.v[i][0] >>= col == 15 ? 8 : 0;
            else x.v[i][1] = (x.v[i][0] >> 24) | (x.v[i][1] << 8);
          }
        }
        constexpr int HALVES = VB == 8 ? 1 : C::VW, PN = CH / HALVES;  // words of a piece, elements of a word
        uint32_t ev[HALVES][4], od[HALVES][4];
        if constexpr (VB < 8) {
#pragma unroll
          for (int y = 0; y < HALVES; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) at_pair<VB>(x.v[2 * i][y], x.v[2 * i + 1][y], ev[y][i], od[y][i]);
        }
        // element n of the eight tokens: the table reads, one element ahead of the products
        constexpr int NT = VB == 8 ? 8 : 4;
        auto look_v = [&](int n, uint32_t (&tb)[NT]) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if constexpr (VB == 8) tb[i] = at_lds(at_byte<128>(x.v[i][n >> 2], n & 3, lane4));
            else tb[i] = at_pair_at<C, VB>((n & 1) ? od[n / PN][i] : ev[n / PN][i], (n % PN) >> 1, lane4);
          }
        };
        constexpr int STEP = NT == 8 ? 1 : 2;  // elements of a step: eight table reads
        constexpr int SV = CH / STEP, PV = SV > 1 ? 1 : 0;
        uint32_t tb[PV + 1][STEP][NT];
#pragma unroll
        for (int z = 0; z < PV; ++z)
#pragma unroll
          for (int y = 0; y < STEP; ++y) look_v(z * STEP + y, tb[z][y]);
#pragma unroll
        for (int n = 0; n < CH; n += STEP) {
          if (n + PV * STEP < CH) {
#pragma unroll
            for (int y = 0; y < STEP; ++y) look_v(n + PV * STEP + y, tb[(n / STEP + PV) % (PV + 1)][y]);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int y = 0; y < STEP; ++y) {
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* z = tb[(n / STEP) % (PV + 1)][y];
              a[i] = at_mul(VB == 8 ? at_pack(z[(2 * i) % NT], z[(2 * i + 1) % NT]) : z[i], vs[i]);
            }
            o[n + y] = at_mfma(a, pb, o[n + y]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };

      {
        // the registers hold one block: its keys' make room for the next keys after the scores, its
        // values' after the sums
        bool again = false;  // the block comes a second time, see below
        while (blk < k1) {
          const bool more = blk + W < k1;
          AtBlock<C>& x = blk0;
          f32x4_t s[2];
          uint32_t pb[4], vs[4];
          const uint32_t bad = x.bad;
          scores(x, blk, s);
          if (more) {
            locate(x);
            load_k(x);
            if (blk + 2 * W < k1) look(blk + 2 * W);
          }
          uint32_t nbad = x.bad;
          if (blk * 32 + 32 > cut) {
            const int lane = at_fresh(threadIdx.x & 63), col = lane & 15;
            const uint32_t see = at_seen(p, *reinterpret_cast<const int*>(smem + C::LIM + 4 * col), blk * 32, before, len,
                                         sq.row0 + tok0, col, ntok) >> (4 * (lane >> 4));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              s[i >> 2][i & 3] = (see >> (16 * (i >> 2) + (i & 3))) & 1u ? s[i >> 2][i & 3] : -__builtin_inff();
          }
          pair_scales(x, vs);
          if (blk * 32 + 32 > len || bad) {  // as if 1: their weights are 0 (or, of a bad page, no numbers)
            const int j0 = blk * 32 + 4 * (at_fresh(threadIdx.x & 63) >> 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 16 * (i >> 1) + 2 * (i & 1);
              const bool dead = (bad >> (i >> 1)) & 1u;
              const uint32_t none = (dead || j >= len ? 0xffffu : 0u) | (dead || j + 1 >= len ? 0xffff0000u : 0u);
              vs[i] = (vs[i] & ~none) | (0x3c003c00u & none);
            }
          }
          // A block with values of both kinds is taken twice, for the loud ones and then for the others,
          // what is not of the kind masked.
          bool once_more = false;
          int e = 0;
          if (__builtin_expect(at_far(vs), 0)) {
            bool some_loud = false, some_quiet = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t bits = (vs[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
              const bool loud = (__ballot(bits >= kAtLoud) >> (16 * h)) & 0xffffu;
              some_loud = some_loud || loud;
              some_quiet = some_quiet || !loud;
            }
            const bool any_loud = __any(some_loud), quiet = again || !any_loud;  // quiet: the kind of this time
            once_more = any_loud && __any(some_quiet) && !again;
            e = quiet ? kAtQuietExp : kAtLoudExp;
            uint32_t f[4] = {};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t bits = (vs[i >> 1] >> (16 * (i & 1))) & 0x7fffu, half = i & 1 ? 0xffff0000u : 0x0000ffffu;
              const bool none = (__ballot(bits >= 0x7c00u) >> (16 * h)) & 0xffffu, loud = (__ballot(bits >= kAtLoud) >> (16 * h)) & 0xffffu;
              const float y = s[i >> 2][i & 3];
              // a token whose value is no number: rows that see it become NaN, others stay
              l = none && y != -__builtin_inff() ? __builtin_nanf("") : l;
              vs[i >> 1] &= none ? ~half : 0xffffffffu;
              f[i >> 1] |= (loud ? at_pow2(kAtLoudExp) : at_pow2(kAtQuietExp)) & half;
              s[i >> 2][i & 3] = loud != quiet ? y : -__builtin_inff();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) vs[i] = at_mul(vs[i], f[i]);
            if (once_more) {  // its keys instead of the next ones; those are looked for again
              look(blk);
              locate(x);
              load_k(x);
              nbad = x.bad;
              if (more) look(blk + W);
            }
          }
          if (__builtin_expect(e != oexp, 0)) {
            const float f = at_exp2(static_cast<float>(oexp - e));
            oexp = e;
#pragma unroll
            for (int n = 0; n < CH; ++n) o[n] *= f;
          }
          softmax(s, pb);
          values(x, vs, pb);
          x.bad = nbad;
          if (more || once_more) load_v(x);
          again = once_more;
          if (!again) blk += W;
        }
      }

      // ---- join the waves ----
      p = at_again(p);
      {
      const int tid = at_fresh(threadIdx.x), lane = tid & 63, col = lane & 15, h = lane >> 4;
      float x, y;
      kv_both<4>(l, x, y);
      kv_both<5>(x + y, x, y);
      l = x + y;
      mo = at_reference(*reinterpret_cast<const float*>(smem + C::C1 + 4 * col), fc, mo);
      if (h == 0)
        *reinterpret_cast<float2*>(smem + C::ML + 8 * (wave * ROWS + col)) = make_float2(mo, l);
      __syncthreads();
      float f;
      float top = kAtNone;
#pragma unroll
      for (int x = 0; x < W; ++x) top = fmaxf(top, *reinterpret_cast<const float*>(smem + C::ML + 8 * (x * ROWS + col)));
      f = mo == kAtNone ? 0.f : at_exp2(mo - top + static_cast<float>(oexp));
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
          for (int i = 0; i < 4; ++i)
            red[((wave * C::NL + nl) * 16 + 4 * h + i) * ROWS + col] = o[rd * C::NL + nl][i] * f;
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
      float* slot = p->parts + static_cast<int64_t>(2 * wg + (k0 > 0 ? 0 : 1)) * ROWS * (D + 2);
      const AtRows<D> rows;
      const uint32_t vsg = rows.signs(p->vsigns);
#pragma unroll 1
      for (int r0 = wave * RN; r0 < ROWS; r0 += W * RN) {
        const int r = r0 + rows.sub;
        const int tk = (static_cast<uint32_t>(r) * p->hb_mul) >> 16, hd = r - tk * hb;
        const bool ok = tk < ntok && hd < nh;
        float2 ml[W];
        float top = kAtNone, ls = 0.f;
#pragma unroll
        for (int x = 0; x < W; ++x) {
          ml[x] = *reinterpret_cast<const float2*>(smem + C::ML + 8 * (x * ROWS + r));
          top = fmaxf(top, ml[x].x);
        }
#pragma unroll
        for (int x = 0; x < W; ++x)  // a wave that saw nothing adds nothing, unless its sum is no number
          ls += ml[x].x == kAtNone ? (ml[x].y != ml[x].y ? ml[x].y : 0.f) : ml[x].y * at_exp2(ml[x].x - top);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = red[r * C::FP + 8 * rows.c + e];
        if (whole) {
          at_store<D>(p, v, ls, static_cast<int64_t>(sq.row0) + tok0 + tk, head0 + hd, vsg, rows.c, ok);
        } else if (ok) {
          at_put<D>(slot, C::ROWS, r, rows.c, v, top, ls);
        }
      }
      if (!whole && k0 == 0 && tid == 0) {
        AttendMeta m{};
        m.parts = wk.more(nblk, wg);
        m.row0 = sq.row0 + tok0;
        m.nrows = ntok;
        m.head0 = head0;
        m.nh = nh;
        p->meta[wg] = m;
      }
      }
    }
    if (!wk.next(p, reads, hu_n)) break;
  }
}

template <int KB, int VB, int D>
hipError_t at_launch(const AttendParams& p, hipStream_t s) {
  using C = AtCfg<KB, VB, D>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend<KB, VB, D>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attend<KB, VB, D>), dim3(C::GRID), dim3(C::T), C::LDS, s, p);
  return hipGetLastError();
}

}  // namespace tq
