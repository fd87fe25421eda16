// Attention over the paged compressed cache for many query rows per key head (prompt chunks, trees
// of drafted tokens): the kernel of kv_attend.hpp with its roles exchanged. There each wave decodes
// its own tokens for all of a tile's rows; here the rows are spread over eight waves and each
// decoded block serves all of them, through shared memory.
//
// A chunk of NB blocks (32 NB tokens) is decoded once, by four waves its keys and by four its
// values, straight into the order in which the matrix instructions take them: 1 KB pieces, 16 bytes
// per lane. Two buffers alternate: while a chunk is multiplied the next one is decoded, the table
// reads and their use spread over the products, and the one after that is on its way from memory.
// A wave holds 16 R rows: their rotated queries and sums stay in its registers (R = 2 of D = 128: 236
// of 256), and no sums are joined across waves.
//
// The powers of two of a block's tokens (kv_attend.hpp) follow from its scales alone, so that the waves
// that decode parts of it agree without asking each other; they travel with the block.
//
// Measured: two chunks of 2047 tokens over texts of 4095 to 8190, 8 key heads of 128 shared by 4 query
// heads, 8-bit keys and 3-bit values (300 Gflop): 459 us a call in a stream of calls, 655 Tflop/s against
// 1180 of a large library product in bf16 (traced, which takes longer: kernel 515, join 15). Of a call of
// 523 us between events 87 were set-up, join and launch; without the decoding 436 remained, without the
// softmax 471, without the loads 465, with the products alone 367: bound by the matrix products (28 % of
// the cycles) and the vector instructions (49 %) that two waves of a SIMD overlap only in part. Four trees
// of 24 tokens over 1500 to 6007: 41 us a call, 28 of them set-up and join.
#pragma once

#include <cstddef>
#include <type_traits>

#include "encode_lane.hpp"
#include "kv_attend.hpp"

namespace tq {

template <int KB, int VB, int D, int R>
struct AwCfg {
  static constexpr int W = 8;               // waves
  static constexpr int T = 64 * W;
  static constexpr int ROWS = 16 * W * R;
  static constexpr int NS = D / 32;         // 32-element steps of a key row
  static constexpr int CH = D / 16;         // codes of a lane's piece of a value row
  static constexpr bool KWIDE = KB == 8 || (KB == 4 && VB != 8);
  static constexpr bool VWIDE = VB == 8 || (VB == 4 && KB != 8);
  static constexpr int KROW = D * KB / 8, VROW = D * VB / 8;  // row bytes
  static constexpr int NB = D == 256 ? 1 : 2;                 // blocks of a chunk
  static constexpr int KP = 2 / NB, VP = 4 / NB;              // waves of a half block's keys, of a block's values
  static constexpr int SPP = NS / KP, EPP = CH / VP;          // steps and value elements of such a wave
  static constexpr int KBYTES = SPP * KB, KW = (KBYTES + 3) / 4;  // its bytes of a quarter key row
  static constexpr int VBITS = EPP * VB;                          // its bits of a value piece
  using Piece = std::conditional_t<VB == 3 || VBITS == 16, uint16_t, std::conditional_t<VBITS <= 8, uint8_t, uint32_t>>;
  static constexpr int KS = D == 256 ? 2 : 1;                 // key scales of a quarter row, at most
  static constexpr int GRID = kAtCus;
  // LDS; the queries on their way in and the sums on their way out take the place of the buffers
  static constexpr int WIDE = (KWIDE || VWIDE) ? 32768 : 0;
  static constexpr int TK = WIDE, TV = TK + 1024;
  static constexpr int C1 = TV + 1024, LIM = C1 + ROWS * 4, HDR = LIM + ROWS * 4;
  static constexpr int BUF = HDR + 2 * NB * 32;  // (32: an AwHeader)
  static constexpr int VOFF = NB * 2 * NS * 1024, BYTES = VOFF + NB * CH * 1024;  // of a buffer
  static constexpr int QP = D * 2 + 16;                       // padded row of q
  static constexpr int FR = D == 256 ? 8 : 16, FP = D + 1;    // rows of a wave that go out at a time, padded row
  static constexpr int max3(int a, int b, int c) { return a > b ? (a > c ? a : c) : b > c ? b : c; }
  static constexpr int LDS = BUF + max3(2 * BYTES, W * 16 * QP, W * FR * FP * 4);
  static_assert(LDS <= 163840, "LDS of a CU");
  static_assert(NB * 2 * KP == 4 && NB * VP == 4, "four waves each");
};

// What a block of a buffer needs besides its values. Keys and values: whether scales are out of the
// range that enters as it is, and if so which tokens are loud (kv_attend.hpp); vbad: the tokens whose
// value is no number.
struct AwHeader {
  uint32_t k[2];  // of a half: 0, or 1 << 16 and the loud ones of its 16 tokens
  uint32_t vapart, pad, vloud, vbad, pad2[2];
};
static_assert(sizeof(AwHeader) == 32 && offsetof(AwHeader, vloud) % 8 == 0, "as it is read");

template <int KB, int VB, int D, int R>
__global__ __launch_bounds__((AwCfg<KB, VB, D, R>::T), 2) void k_attend_wide(AttendParams) {
  using C = AwCfg<KB, VB, D, R>;
  constexpr int W = C::W, NS = C::NS, CH = C::CH, NB = C::NB;
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

  // this wave's part of a chunk's decoding: waves 0 - 3 keys, 4 - 7 values
  const bool keys = wave < 4;
  const int pb = keys ? (wave & 3) / (2 * C::KP) : (wave & 3) / C::VP;  // block of the chunk
  const int sbk = (wave / C::KP) & 1, kp = wave % C::KP, vp = wave % C::VP;
  const uint32_t koff = col * C::KROW + (C::KROW / 4) * h + C::KBYTES * kp;
  // a value piece's part begins at any bit; of 3-bit rows two bytes are read, inside the row
  const int vbit = VB * (CH * col + C::EPP * vp);
  const int vbyte = VB == 3 && (vbit >> 3) > C::VROW - 2 ? C::VROW - 2 : vbit >> 3;
  const int vshift = vbit - 8 * vbyte;
  const uint32_t voff = 4 * h * C::VROW + vbyte;
  // scales: of the quarter key row's first and (D = 256) second half, or of the value piece
  const uint32_t soff = keys ? ((col << p->lg_gk) + ((D / 4 * h) >> p->lg_kg)) * 2
                             : ((4 * h << p->lg_gv) + ((col * CH) >> p->lg_vg)) * 2;
  const uint32_t soff2 = ((col << p->lg_gk) + ((D / 4 * h + D / 8) >> p->lg_kg)) * 2;

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
      // of this wave's half: codes and scales of the head, bytes of a row, log2 of a row's scales
      const uint32_t rbytes = keys ? C::KROW : C::VROW;
      const int lg = keys ? p->lg_gk : p->lg_gv;
      const char* const codes = reinterpret_cast<const char*>(keys ? p->kcodes : p->vcodes) + static_cast<int64_t>(kh) * page * rbytes;
      const char* const scales = reinterpret_cast<const char*>(keys ? p->kscales : p->vscales) + ((static_cast<int64_t>(kh) * page) << (lg + 1));
      typedef const int32_t __attribute__((address_space(4))) * ConstIds;
      const ConstIds ids = (ConstIds)reinterpret_cast<uintptr_t>(p->page_table + static_cast<int64_t>(b) * p->table_width);
      // page ids of a block's halves (a half past the end stands for the first one), read a chunk ahead
      int id[2] = {}, in[2] = {};
      auto look = [&](int blk) __attribute__((always_inline)) {
        const int j = blk * 32, j2 = j + 16 < len ? j + 16 : j;
        const int pi = at_div(j >> 4, page16, page_mul), pi2 = at_div(j2 >> 4, page16, page_mul);
        in[0] = j - pi * page;
        in[1] = j2 - pi2 * page;
        id[0] = len > 0 ? ids[pi] : -1;
        id[1] = len > 0 ? ids[pi2] : -1;
      };
      // codes and scales of this wave's part, of the block being decoded and of the next one, in the
      // types they are loaded as: widened at once, they would be waited for at once
      uint32_t kx[8], kx1[8];
      uint16_t ks[C::KS], vs[8], ks1[C::KS], vs1[8];
      typename C::Piece vx[8], vx1[8];
      uint32_t bad = 0, bad1 = 0;  // bit y: the page of half y is none
      auto load = [&](auto role) __attribute__((always_inline)) {
        int64_t row_of[2];
        bad1 = 0;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const bool none = static_cast<uint32_t>(id[y]) >= static_cast<uint32_t>(pages);
          bad1 |= none ? 1u << y : 0u;
          row_of[y] = static_cast<int64_t>(static_cast<uint64_t>(none ? 0u : static_cast<uint32_t>(id[y])) * prow) + in[y];
        }
        if constexpr (decltype(role)::value) {
          const int64_t row = sbk ? row_of[1] : row_of[0];
          const uint32_t ko = at_fresh(koff), so = at_fresh(soff);
          const AtPtr kc = at_base(codes, row * C::KROW);
          constexpr int L = C::KW % 4 == 0 ? 4 : C::KW % 3 == 0 ? 3 : C::KW % 2 == 0 ? 2 : 1;  // words of a load
          if constexpr (C::KBYTES == 6) {
            kx1[0] = at_load<uint32_t>(kc, ko);
            kx1[1] = at_load<uint16_t>(kc + 4, ko);
          } else {
#pragma unroll
            for (int k = 0; k < C::KW; k += L) {
              if constexpr (L == 4) {
                const u32x4_t y = at_get<u32x4_t>(kc + 4 * k, ko);
                kx1[k] = y.x; kx1[k + 1] = y.y; kx1[k + 2] = y.z; kx1[k + 3] = y.w;
              } else if constexpr (L == 3) {
                const u32x3_t y = at_get<u32x3_t>(kc + 4 * k, ko);
                kx1[k] = y.x; kx1[k + 1] = y.y; kx1[k + 2] = y.z;
              } else if constexpr (L == 2) {
                const u32x2_t y = at_get<u32x2_t>(kc + 4 * k, ko);
                kx1[k] = y.x; kx1[k + 1] = y.y;
              } else {
                kx1[k] = at_get<uint32_t>(kc + 4 * k, ko);
              }
            }
          }
          const AtPtr sp = at_base(scales, row << (lg + 1));
          ks1[0] = at_get<uint16_t>(sp, so);
          if constexpr (C::KS == 2) ks1[1] = at_get<uint16_t>(sp, at_fresh(soff2));
        } else {
          const uint32_t vo = at_fresh(voff), so = at_fresh(soff);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const AtPtr vc = at_base(codes, row_of[y] * C::VROW), sp = at_base(scales, row_of[y] << (lg + 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const AtPtr vr = vc + i * C::VROW;
              if constexpr (VB == 3) vx1[4 * y + i] = at_load<uint16_t>(vr, vo);
              else vx1[4 * y + i] = at_get<typename C::Piece>(vr, vo);
              vs1[4 * y + i] = at_get<uint16_t>(sp + (static_cast<int64_t>(i) << (lg + 1)), so);
            }
          }
        }
      };

      auto take = [&](auto role) __attribute__((always_inline)) {
        bad = bad1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (decltype(role)::value) {
            if (i < C::KW) kx[i] = kx1[i];
            if (i < C::KS) ks[i] = ks1[i];
          } else {
            vx[i] = vx1[i];
            vs[i] = vs1[i];
          }
        }
      };
      // A round's decoding: what was loaded, of block blk, into buffer `buf`, in STEPS steps (of keys:
      // 32-element steps; of values: elements) of a table lookup and, later, its use.
      constexpr int STEPS = C::SPP;
      static_assert(C::SPP == C::EPP, "as many for either role");
      uint32_t mul[4], ev[4], od[4], tb[8];  // scales, value pairs of even and odd elements, table words
      uint32_t dst;                          // LDS address
      auto prepare = [&](auto role, int buf, int blk) __attribute__((always_inline)) {
        const int lane = at_fresh(threadIdx.x & 63), h = lane >> 4;
        AwHeader* const hdr = reinterpret_cast<AwHeader*>(smem + C::HDR) + buf * NB + pb;
        dst = C::BUF + buf * C::BYTES + 16 * lane;
        if constexpr (decltype(role)::value) {
          dst += ((pb * 2 + sbk) * NS + kp * C::SPP) * 1024;
          uint32_t z[C::KS], far = 0, most = 0;
#pragma unroll
          for (int y = 0; y < C::KS; ++y) {
            z[y] = (bad >> sbk) & 1u ? 0x7e00u : ks[y];  // scores of a bad page are NaN
            // rows that hold no token hold anything: as if 1
            if (blk * 32 + 32 > len) z[y] = blk * 32 + 16 * sbk + (lane & 15) < len ? z[y] : 0x3c00u;
            far = z[y] - kAtLow > far ? z[y] - kAtLow : far;
            most = (z[y] & 0x7fffu) > most ? z[y] & 0x7fffu : most;
          }
          mul[0] = C::KS == 2 && kp ? z[C::KS - 1] : z[0];
          mul[0] |= mul[0] << 16;
          uint32_t word = 0;
          if (__any(far >= kAtSpan)) {
            const uint32_t loud = at_loud(most);
            mul[0] = at_mul(mul[0], (loud >> (lane & 15)) & 1u ? at_pow2(kAtLoudExp) : at_pow2(kAtQuietExp));
            word = 0x10000u | loud;
          }
          if (lane == 0) hdr->k[sbk] = word;
        } else {
          dst += C::VOFF + (pb * CH + vp * C::EPP) * 1024;
#pragma unroll
          for (int i = 0; i < 4; ++i) mul[i] = at_pack(vs[2 * i], vs[2 * i + 1]);  // scales of tokens 2 i and 2 i + 1
          if (blk * 32 + 32 > len || bad) {  // as if 1: their weights are 0 (or, of a bad page, no numbers)
            const int j0 = blk * 32 + 4 * h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + 16 * (i >> 1) + 2 * (i & 1);
              const bool dead = (bad >> (i >> 1)) & 1u;
              const uint32_t none = (dead || j >= len ? 0xffffu : 0u) | (dead || j + 1 >= len ? 0xffff0000u : 0u);
              mul[i] = (mul[i] & ~none) | (0x3c003c00u & none);
            }
          }
          uint32_t vapart = 0, vloud = 0, vbad = 0;
          if (at_far(mul)) {
            vapart = 1;
            uint32_t f[4] = {};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t bits = (mul[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
              // the lanes of a token's groups: 16 y to 16 y + 15 of tokens 4 y + (i & 3)
              const uint64_t none = __ballot(bits >= 0x7c00u), who = __ballot(bits >= kAtLoud);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t bit = 1u << (16 * (i >> 2) + 4 * y + (i & 3));
                if ((none >> (16 * y)) & 0xffffu) vbad |= bit;
                if ((who >> (16 * y)) & 0xffffu) vloud |= bit;
              }
              if ((none >> (16 * h)) & 0xffffu) mul[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
              const uint32_t two = (who >> (16 * h)) & 0xffffu ? at_pow2(kAtLoudExp) : at_pow2(kAtQuietExp);
              f[i >> 1] |= two & ((i & 1) ? 0xffff0000u : 0x0000ffffu);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) mul[i] = at_mul(mul[i], f[i]);
          }
          if (lane == 0) {
            hdr->vapart = vapart;
            hdr->vloud = vloud;
            hdr->vbad = vbad;
          }
          if constexpr (VB < 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) at_pair<VB>(vx[2 * i] >> vshift, vx[2 * i + 1] >> vshift, ev[i], od[i]);
          }
        }
      };
      auto look_up = [&](auto role, int n) __attribute__((always_inline)) {
        if constexpr (decltype(role)::value) {
          AtLook<KB> x;
          at_look_k<C, KB>(kx, n, lane4, x);
#pragma unroll
          for (int i = 0; i < AtLook<KB>::N; ++i) tb[i] = x.t[i];
        } else if constexpr (VB == 8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) tb[i] = at_lds(at_byte<128>(vx[i], n, lane4));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) tb[i] = at_pair_at<C, VB>((n & 1) ? od[i] : ev[i], n >> 1, lane4);
        }
      };
      auto finish = [&](auto role, int n) __attribute__((always_inline)) {
        constexpr bool single = decltype(role)::value ? KB == 8 : VB == 8;  // a word per code, not per pair
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = at_mul(single ? at_pack(tb[2 * i], tb[2 * i + 1]) : tb[i], decltype(role)::value ? mul[0] : mul[i]);
        *reinterpret_cast<u32x4_t*>(smem + dst + n * 1024) = u32x4_t{a[0], a[1], a[2], a[3]};
      };

      // ---- q: row group wave + 8 r of the tile to this wave, by way of LDS ----
      AtQuery<D> qs(p, sq.row0 + tok0, head0, tok0, ntok, nh);
      qs.load(p, 16 * wave);
      constexpr int RN = AtRows<D>::N;  // rows of a wave at a time
      // past its last block a wave repeats it, into buffers that nothing reads
      const auto next_of = [&](int x) { return x + NB < k1 ? x + NB : x; };
      int blk = k0 + pb < k1 ? k0 + pb : k0;
      {
        look(blk);
        if (keys) load(AtInt<1>{});
        else load(AtInt<0>{});
        look(next_of(blk));
      }
      uint32_t q[R][NS][4];
      float fc[R], mo[R], l[R];  // score factor; reference - 7; sum
      f32x4_t o[R][CH];
      __syncthreads();  // the last unit's readers of this memory are done
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int r0 = 16 * (wave + W * r), at = C::BUF + wave * 16 * C::QP;
        wave_lds_sync();
#pragma unroll 1
        for (int y = 0; y < 16; y += RN)
          qs.rotate(p, smem, r0 + y, at + y * C::QP, C::QP, C::C1, C::LIM, before, len,
                    y + RN < 16 ? r0 + y + RN : r + 1 < R ? r0 + 16 * W : -1);
        wave_lds_sync();
#pragma unroll
        for (int st = 0; st < NS; ++st) {
          const u32x4_t x = *reinterpret_cast<const u32x4_t*>(smem + at + col * C::QP + (D / 2) * h + 16 * st);
          q[r][st][0] = x.x; q[r][st][1] = x.y; q[r][st][2] = x.z; q[r][st][3] = x.w;
        }
        fc[r] = *reinterpret_cast<const float*>(smem + C::C1 + 4 * (r0 + col));
        mo[r] = kAtNone;
        l[r] = 0.f;
#pragma unroll
        for (int n = 0; n < CH; ++n) o[r][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      __syncthreads();
      const bool masked = p->tree != nullptr;
      int cut = masked ? before : before + tok0 + 1;  // from this token on some row's mask may cut
      cut = cut < 0 ? 0 : cut;
      const uint32_t hb_mul = p->hb_mul;
      const bool live = ((static_cast<uint32_t>(16 * wave) * hb_mul) >> 16) < static_cast<uint32_t>(ntok);

      int oexp = 0;  // the sums are held times 2^-oexp
      uint32_t state = 0;  // 1: a chunk's second time; 2: it needs one; see multiply

      // Scores, weights and sums of block x of the chunk. Pieces are read G at a time, AHEAD groups before
      // their products; z holds those on their way.
      constexpr int G = 2, KG = 2 * NS / G, VG = CH / G, BG = KG + VG, AHEAD = 1;
      u32x4_t z[AHEAD + 1][G];
      auto read = [&](const char* src, int g) __attribute__((always_inline)) {  // group g of the chunk's NB * BG
        if (g >= NB * BG) return;
        const int x = g / BG, k = g % BG, at = (k < KG ? x * KG + k : NB * KG + x * VG + k - KG) * G;
#pragma unroll
        for (int y = 0; y < G; ++y) z[g % (AHEAD + 1)][y] = *reinterpret_cast<const u32x4_t*>(src + (at + y) * 1024);
      };
      auto multiply = [&](int buf, int x, int blk, auto side) __attribute__((always_inline)) {
        const int lane = at_fresh(threadIdx.x & 63), h = lane >> 4;
        const char* const src = smem + C::BUF + buf * C::BYTES + 16 * lane;
        const AwHeader* const hdr = reinterpret_cast<const AwHeader*>(smem + C::HDR) + buf * NB + x;
        f32x4_t s[R][2];
        if (x == 0) {
#pragma unroll
          for (int g = 0; g < AHEAD; ++g) read(src, g);
        }
#pragma unroll
        for (int g = 0; g < KG; ++g) {
          read(src, x * BG + g + AHEAD);
          side(g);
#pragma unroll
          for (int y = 0; y < G; ++y) {
            const int n = G * g + y, sb = n / NS, st = n % NS;
            const u32x4_t w = z[(x * BG + g) % (AHEAD + 1)][y];
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][sb] = at_mfma(a, q[r][st], st == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : s[r][sb]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        const u32x4_t hd = *reinterpret_cast<const u32x4_t*>(hdr);
        const uint32_t apart = static_cast<uint32_t>(at_uniform(static_cast<int>(hd.x | hd.y | hd.z)));
        if (blk * 32 + 32 > cut) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const int row = 16 * (wave + W * r) + (lane & 15);
            const uint32_t see = at_seen(p, *reinterpret_cast<const int*>(smem + C::LIM + 4 * row), blk * 32, before, len,
                                         sq.row0 + tok0, row, ntok) >> (4 * h);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              s[r][i >> 2][i & 3] = (see >> (16 * (i >> 2) + (i & 3))) & 1u ? s[r][i >> 2][i & 3] : -__builtin_inff();
          }
        }
        if (__builtin_expect((apart | static_cast<uint32_t>(oexp) | state) != 0, 0)) {
          const uint32_t ka = static_cast<uint32_t>(at_uniform(static_cast<int>(hd.x))), kb = static_cast<uint32_t>(at_uniform(static_cast<int>(hd.y)));
          const bool vapart = at_uniform(static_cast<int>(hd.z)) != 0;
          // A block with values of both kinds is multiplied twice, for the loud ones and then for the others,
          // what is not of the kind masked; beside it other blocks have nothing left the second time.
          const uint2 hv = *reinterpret_cast<const uint2*>(&hdr->vloud);
          const uint32_t vloud = static_cast<uint32_t>(at_uniform(static_cast<int>(hv.x))), vbad = static_cast<uint32_t>(at_uniform(static_cast<int>(hv.y)));
          const bool both = vapart && vloud != 0 && vloud != ~0u, again = (state & 1u) != 0;
          const uint32_t kind = (both ? (again ? ~vloud : vloud) : again ? 0u : ~0u) >> (4 * h), none = vapart ? vbad >> (4 * h) : 0u;
          state |= both ? 2u : 0u;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (ka) at_back(s[r][0], ka, h);
            if (kb) at_back(s[r][1], kb, h);
          }
          if (both || again || (vapart && vbad)) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int bit = 16 * (i >> 2) + (i & 3);
                const float y = s[r][i >> 2][i & 3];
                // tokens whose value is no number: rows that see one become NaN, others stay
                l[r] = (none >> bit) & 1u && y != -__builtin_inff() ? __builtin_nanf("") : l[r];
                s[r][i >> 2][i & 3] = at_pick(kind, bit, y, -__builtin_inff());
              }
          }
          const int e = !vapart ? 0 : again || !vloud ? kAtQuietExp : kAtLoudExp;
          if (e != oexp) {
            const float f = at_exp2(static_cast<float>(oexp - e));
            oexp = e;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int n = 0; n < CH; ++n) o[r][n] *= f;
          }
        }
        float mx[R];
        bool move = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          mx[r] = fmaxf(fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3])),
                        fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
          move = move || __builtin_fmaf(mx[r], fc[r], -mo[r]) > 7.f + kAtLazy;
        }
        if (__builtin_expect(__any(move), 0)) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float c1 = *reinterpret_cast<const float*>(smem + C::C1 + 4 * (16 * (wave + W * r) + (lane & 15)));
            float y, w;
            kv_both<4>(mx[r], y, w);
            kv_both<5>(fmaxf(y, w), y, w);
            y = fmaxf(y, w);
            if (__builtin_fmaf(y, fc[r], -mo[r]) > 7.f + kAtLazy) {  // the same in the four lanes of a row
              const float f = at_refer(y, c1, fc[r], mo[r]);
              l[r] *= f;
#pragma unroll
              for (int n = 0; n < CH; ++n) o[r][n] *= f;
            }
          }
        }
        uint32_t pr[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = at_exp2(__builtin_fmaf(s[r][i >> 2][i & 3], fc[r], -mo[r]));
          l[r] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const half2_t y{static_cast<_Float16>(e[2 * i]), static_cast<_Float16>(e[2 * i + 1])};
            pr[r][i] = __builtin_bit_cast(uint32_t, y);
          }
        }
#pragma unroll
        for (int g = 0; g < VG; ++g) {
          read(src, x * BG + KG + g + AHEAD);
          side(KG + g);
#pragma unroll
          for (int y = 0; y < G; ++y) {
            const u32x4_t w = z[(x * BG + KG + g) % (AHEAD + 1)][y];
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int r = 0; r < R; ++r) o[r][G * g + y] = at_mfma(a, pr[r], o[r][G * g + y]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };

      // One loop for the waves of keys and one for those of values: with both roles in one, the loads
      // in flight would be copied, and so waited for, where its paths meet. Each ends its rounds with
      // the same barriers. A round decodes a chunk while it multiplies the one before, the steps of
      // one spread over the products of the other.
      auto rounds = [&](auto role) __attribute__((always_inline)) {
        auto begin = [&](int buf) __attribute__((always_inline)) {
          take(role);
          const int now = blk;
          blk = next_of(blk);
          load(role);
          look(next_of(blk));
          prepare(role, buf, now);
        };
        auto plain = [&]() __attribute__((always_inline)) {
#pragma unroll
          for (int n = 0; n < STEPS; ++n) {
            look_up(role, n);
            finish(role, n);
          }
        };
        begin(0);
        plain();
        __syncthreads();
        int buf = 0;
        for (int c = k0; c < k1;) {
          if (__builtin_expect(state == 0, 1)) begin(buf ^ 1);
          if (live) {
            constexpr int SB = STEPS / NB, EVERY = BG / (2 * SB);
#pragma unroll
            for (int x = 0; x < NB; ++x)
              if (x == 0 || c + x < k1)  // (without it there is no next chunk either)
                multiply(buf, x, c + x, [&](int slot) __attribute__((always_inline)) {
                  if (slot % EVERY == 0) {
                    const int y = slot / EVERY, n = x * SB + (y >> 1);
                    if (y & 1) finish(role, n);
                    else look_up(role, n);
                  }
                });
          } else {
            plain();
          }
          state = state == 2u ? 1u : 0u;
          if (__builtin_expect(state != 0, 0)) continue;  // the decoding's steps then do again what they did
          __syncthreads();
          buf ^= 1;
          c += NB;
        }
      };
      if (keys) rounds(AtInt<1>{});
      else rounds(AtInt<0>{});

      // ---- out: a wave's rows, transposed by way of LDS ----
      p = at_again(p);
      const int lane = at_fresh(threadIdx.x & 63), col = lane & 15, h = lane >> 4;
      const AtRows<D> rows;
      const uint32_t vsg = rows.signs(p->vsigns);
      const bool whole = k0 == 0 && k1 == nblk;
      float* const slot = p->parts + static_cast<int64_t>(2 * wg + (k0 > 0 ? 0 : 1)) * C::ROWS * (D + 2);
      float* const red = reinterpret_cast<float*>(smem + C::BUF) + wave * C::FR * C::FP;
      const float fo = at_exp2(static_cast<float>(oexp));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x, y;
        kv_both<4>(l[r], x, y);
        kv_both<5>(x + y, x, y);
        l[r] = x + y;
        mo[r] = at_reference(*reinterpret_cast<const float*>(smem + C::C1 + 4 * (16 * (wave + W * r) + col)), fc[r], mo[r]);
#pragma unroll
        for (int r1 = 0; r1 < 16; r1 += C::FR) {
          wave_lds_sync();
          if (col >= r1 && col < r1 + C::FR)
#pragma unroll
            for (int n = 0; n < CH; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) red[(col - r1) * C::FP + CH * (4 * h + i) + n] = o[r][n][i] * fo;
          wave_lds_sync();
#pragma unroll 1
          for (int z0 = r1; z0 < r1 + C::FR; z0 += RN) {
            const int z = z0 + rows.sub, row = 16 * (wave + W * r) + z;
            const int tk = (static_cast<uint32_t>(row) * hb_mul) >> 16, hd = row - tk * hb;
            const bool ok = tk < ntok && hd < nh;
            const float ls = __shfl(l[r], z), top = __shfl(mo[r], z);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = red[(z - r1) * C::FP + 8 * rows.c + e];
            if (whole) at_store<D>(p, v, ls, static_cast<int64_t>(sq.row0) + tok0 + tk, head0 + hd, vsg, rows.c, ok);
            else if (ok) at_put<D>(slot, C::ROWS, row, rows.c, v, top, ls);
          }
        }
      }
      if (!whole && k0 == 0 && threadIdx.x == 0) {
        AttendMeta m{};
        m.parts = wk.more(nblk, wg);
        m.row0 = sq.row0 + tok0;
        m.nrows = ntok;
        m.head0 = head0;
        m.nh = nh;
        p->meta[wg] = m;
      }
    }
    if (!wk.next(p, reads, hu_n)) break;
  }
}

template <int KB, int VB, int D, int R>
hipError_t aw_launch(const AttendParams& p, hipStream_t s) {
  using C = AwCfg<KB, VB, D, R>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend_wide<KB, VB, D, R>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attend_wide<KB, VB, D, R>), dim3(C::GRID), dim3(C::T), C::LDS, s, p);
  return hipGetLastError();
}

template <int KB, int VB>
hipError_t at_launch_d(const AttendParams& p, int D, int rows, hipStream_t s) {
  switch (D) {
    case 64: return rows == 16 ? at_launch<KB, VB, 64>(p, s) : rows == 128 ? aw_launch<KB, VB, 64, 1>(p, s) : aw_launch<KB, VB, 64, 2>(p, s);
    case 128: return rows == 16 ? at_launch<KB, VB, 128>(p, s) : rows == 128 ? aw_launch<KB, VB, 128, 1>(p, s) : aw_launch<KB, VB, 128, 2>(p, s);
    default: return rows == 16 ? at_launch<KB, VB, 256>(p, s) : aw_launch<KB, VB, 256, 1>(p, s);
  }
}

// One key format's kernels, by the rows of a tile.
template <int KB>
hipError_t at_launch_k(const AttendParams& p, int vbits, int D, int rows, hipStream_t s) {
  switch (vbits) {
    case 2: return at_launch_d<KB, 2>(p, D, rows, s);
    case 3: return at_launch_d<KB, 3>(p, D, rows, s);
    case 4: return at_launch_d<KB, 4>(p, D, rows, s);
    default: return at_launch_d<KB, 8>(p, D, rows, s);
  }
}

}  // namespace tq
