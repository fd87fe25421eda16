// The tables of a decoding step from the requests' lengths, and what stays of the step in the paged
// cache (tq_kv_plan and tq_kv_keep).
//
// Plan. Sequence b, with n tokens in ceil(n / page) pages, gets c rows, its tokens n .. n + c, and
//     w_b = ceil((n + c) / page) - ceil(n / page)
// pages off the top of the pool's list: page j of them is entry count - 1 - (W_b + j), W_b the sum of
// the w before. Every workgroup scans all sequences (rows and pages, two sums that saturate, so 32 bits
// hold them), 1024 at a time in LDS, and takes its share of the rows and of the new table entries, which
// it finds in the sums by bisection: uneven counts balance, and no workgroup waits for another. New
// pages are read from the list, not from the table, so the table's new entries may be written at the
// same time.
//
// Keep. Rows of an accepted branch go to the places behind the sequence's tokens, each thread moving
// one column of 8 bytes (scales: 2) of a head for all of the branch's rows in their order. A row moves to a
// place at or before its own, so a place is overwritten only after it was read. Pages behind the new
// length go back in the order that undoes the plan.
//
// Both change the pool's count at their end, by the workgroup that arrives last: all others have read it.
//
// Bounds and figures. Kilobytes pass (keep's moves aside), so both are bound by a launch and by loads that wait for each
// other, 0.6 us each: state, lengths, table or list, for trees the parents and then LDS from row to row. In a
// stream of launches: 16 sequences of one row 5.3 us, 5 prompts of 48,000 rows in all 5.1, 192 trees of 24 rows 10.0 (the
// page's number is fetched before the way to the root: 0.2 more when after); keep 3.8, with 4 rows each of 192 branches
// moved (2.8 MB) 5.5.
#include "device_common.hpp"
#include "internal.hpp"

namespace tq {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepPer = 4;                           // sequences of a thread
constexpr int kStepTile = kStepThreads * kStepPer;    // sequences in LDS
constexpr int kStepParents = 2048;                    // parents in LDS
constexpr uint32_t kStepLong = 256;                   // rows of a tree that are still walked one by one
constexpr uint32_t kStepCap = (1u << 30) + 1;         // sums stop here, above every limit

__device__ __forceinline__ uint32_t step_add(uint32_t a, uint32_t b) {
  return a + b < kStepCap ? a + b : kStepCap;
}

// Exclusive prefix sums over the workgroup of two values per thread; the totals in ta, tb.
__device__ __forceinline__ void step_scan(uint32_t& a, uint32_t& b, uint32_t& ta, uint32_t& tb,
                                          uint32_t (&waves)[2][kStepThreads / 64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = a, y = b;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const uint32_t u = __shfl_up(x, s), v = __shfl_up(y, s);
    if (lane >= s) {
      x = step_add(x, u);
      y = step_add(y, v);
    }
  }
  if (lane == 63) {
    waves[0][wave] = x;
    waves[1][wave] = y;
  }
  const uint32_t px = __shfl_up(x, 1), py = __shfl_up(y, 1);
  __syncthreads();
  a = lane ? px : 0;
  b = lane ? py : 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kStepThreads / 64; ++w) {
    if (w == wave) {
      a = step_add(a, ta);
      b = step_add(b, tb);
    }
    ta = step_add(ta, waves[0][w]);
    tb = step_add(tb, waves[1][w]);
  }
  __syncthreads();
}

// The largest i < n with s[i] <= x (s ascending, s[0] <= x).
__device__ __forceinline__ int step_find(const uint32_t* s, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t step_pages(uint32_t tokens, uint32_t page) { return (tokens + page - 1) / page; }

__device__ __forceinline__ uint32_t step_free(const int32_t* state, int pages) {
  const int n = state[0];
  return n < 0 ? 0 : n < pages ? n : pages;
}

// Whether this workgroup is the last of the launch to come here. Nothing passes between them but the order:
// what the last one overwrites the others have read.
__device__ __forceinline__ bool step_last(int32_t* state, int& shared) {
  __syncthreads();
  if (threadIdx.x == 0)
    shared = __hip_atomic_fetch_add(state + 1, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return shared == static_cast<int>(gridDim.x) - 1;
}

// Trees of more than kStepLong rows, whose walks to the root would be as long (time grew with the square of the
// length). Their first rows, as far as they are a chain, which prompts among trees are throughout, are known without a
// walk: every workgroup looks how far that is, up to its own rows. The rows behind are made by one workgroup of the
// sequence, 256 at a time: a row's steps and mask within these by doubling the way to its ancestors, 8 times at most, and
// the rest from its first ancestor before, which is done. 191 trees of 24 rows and a prompt of 4000, masks of 125 words:
// 49 us (830 walked); a tree of 4000 rows that each follow the last but one instead, without masks 111 (320), with them
// 574 (429: the words, 2 MB, are copied by one workgroup).
struct LongShared {
  int ptr[kStepThreads], anc[kStepThreads];  // the ancestor 2^k steps up within the 256, -1: none; the first before them, -1: none
  uint32_t depth[kStepThreads];              // steps to it, or to the root
  uint32_t mask[kStepThreads][kStepThreads / 32];
};

// Bits 0 .. last of a mask, word k.
__device__ __forceinline__ uint32_t step_ones(int64_t last, int k) {
  return last >= 32ll * k + 31 ? ~0u : last >= 32ll * k ? (2u << (last - 32ll * k)) - 1 : 0;
}

// The first row in [1, n) that does not follow the one before it; n if there is none. parents: of the sequence.
__device__ __forceinline__ uint32_t step_chain(const int32_t* parents, uint32_t n, uint32_t& shared) {
  constexpr uint32_t U = 8;
  if (threadIdx.x == 0) shared = n;
  __syncthreads();
  for (uint32_t t = 1; t < n; t += U * kStepThreads) {
    uint32_t first = n;
#pragma unroll
    for (int u = U - 1; u >= 0; --u) {
      const uint32_t a = t + u * kStepThreads + threadIdx.x;
      if (a < n && parents[a] != static_cast<int>(a - 1)) first = a;
    }
    if (__syncthreads_or(first < n)) {
      if (first < n) atomicMin(&shared, first);
      break;
    }
  }
  __syncthreads();
  const uint32_t e = shared;
  __syncthreads();
  return e;
}

// Depths and masks of rows e .. n of a sequence whose rows before e are a chain. put(a, depth): slot and position;
// depth_of(a): of a row before, from its position. tree: of the sequence, null without masks.
template <class Put, class Depth>
__device__ __forceinline__ void step_long(const int32_t* parents, uint32_t n, uint32_t e, uint32_t* tree, int words, LongShared& sh,
                                          Put put, Depth depth_of) {
  constexpr int W = kStepThreads / 32, U = 4;
  const int l = threadIdx.x;
  for (uint32_t t = e & ~(kStepThreads - 1u); t < n; t += kStepThreads) {
    const uint32_t a = t + l;
    int ptr = -1, anc = -1;
    uint32_t depth = 0, mask[W];
#pragma unroll
    for (int k = 0; k < W; ++k) mask[k] = (l >> 5) == k ? 1u << (l & 31) : 0;
    if (a < e) {
      depth = a;
      anc = static_cast<int>(t) - 1;
#pragma unroll
      for (int k = 0; k < W; ++k) mask[k] = step_ones(l, k);
    } else if (a < n && a > 0) {
      const int up = parents[a];
      if (up >= 0 && static_cast<uint32_t>(up) < a) {
        if (static_cast<uint32_t>(up) >= t) {
          ptr = up - static_cast<int>(t);
          depth = 1;
        } else {
          anc = up;
          depth = 1 + (static_cast<uint32_t>(up) < e ? up : depth_of(up));
        }
      }
    }
    auto share = [&]() {
      sh.ptr[l] = ptr;
      sh.anc[l] = anc;
      sh.depth[l] = depth;
#pragma unroll
      for (int k = 0; k < W; ++k) sh.mask[l][k] = mask[k];
    };
    share();
    while (__syncthreads_or(ptr >= 0)) {
      if (ptr >= 0) {
        depth += sh.depth[ptr];
        anc = sh.anc[ptr];
#pragma unroll
        for (int k = 0; k < W; ++k) mask[k] |= sh.mask[ptr][k];
        ptr = sh.ptr[ptr];
      }
      __syncthreads();
      share();
    }
    __syncthreads();
    if (a >= e && a < n) put(a, depth);
    // the masks, words next to each other by threads next to each other
    const uint32_t skip = e > t ? e - t : 0, rows = n - t < kStepThreads ? n - t : kStepThreads, base = t >> 5;
    for (uint32_t x0 = skip * words + l; x0 < rows * words; x0 += U * kStepThreads) {
      uint32_t v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t x = x0 + u * kStepThreads, row = x / words, k = x - row * words;
        v[u] = 0;
        if (row >= rows) continue;
        if (k >= base) {
          if (k < base + W) v[u] = sh.mask[row][k - base];
        } else if (const int up = sh.anc[row]; up >= 0) {
          v[u] = static_cast<uint32_t>(up) < e ? step_ones(up, k) : tree[static_cast<int64_t>(up) * words + k];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t x = x0 + u * kStepThreads;
        if (x < rows * words) tree[static_cast<int64_t>(t) * words + x] = v[u];
      }
    }
    __syncthreads();  // (what these rows got is read by the next)
  }
}

// TREE: with parents. LONG: more rows than kStepLong, so a tree may be that long.
template <bool TREE, bool LONG>
__global__ __launch_bounds__(kStepThreads) void k_kv_plan(PlanArgs p, int rows_each) {
  __shared__ uint32_t s_row[kStepTile + 1], s_new[kStepTile + 1];
  __shared__ int s_len[kStepTile];  // -1: refused
  __shared__ int s_parent[kStepParents];
  __shared__ uint32_t s_wave[2][kStepThreads / 64];
  __shared__ uint32_t s_granted;
  __shared__ int s_arrived;
  __shared__ int s_long;  // there are trees of more than kStepLong rows
  __shared__ uint32_t s_chain;
  __shared__ LongShared s_tile;
  const uint32_t page = p.page, M = p.M, free_count = step_free(p.state, p.pages);
  const uint32_t cap = page * static_cast<uint32_t>(p.width);
  const uint32_t lo_row = blockIdx.x * rows_each;
  const uint32_t hi_row = lo_row + rows_each < M ? lo_row + rows_each : M;
  uint32_t row0 = 0, new0 = 0, granted = 0;
  if (threadIdx.x == 0) s_granted = 0;
  if (LONG && threadIdx.x == 0) s_long = 0;
  // the parents of its rows and of those before, as many as fit, while the lengths are on their way
  const uint32_t first = hi_row > kStepParents ? hi_row - kStepParents : 0;
  if (TREE)
    for (uint32_t r = first + threadIdx.x; r < hi_row; r += kStepThreads) s_parent[r - first] = p.parents[r];
  for (int b0 = 0; b0 < p.B; b0 += kStepTile) {
    const int nb = p.B - b0 < kStepTile ? p.B - b0 : kStepTile;
    uint32_t n[kStepPer], c[kStepPer], w[kStepPer], rows = 0, fresh = 0;
    bool wide[kStepPer];
#pragma unroll
    for (int k = 0; k < kStepPer; ++k) {
      const int i = threadIdx.x * kStepPer + k;
      const int len = i < nb ? p.lens[b0 + i] : 0, count = i < nb ? p.counts[b0 + i] : 0;
      n[k] = len < 0 ? 0 : len;
      c[k] = count < 0 ? 0 : count;
      wide[k] = n[k] + c[k] > cap;  // (two numbers below 2^31)
      w[k] = wide[k] ? 0 : step_pages(n[k] + c[k], page) - step_pages(n[k], page);
      rows = step_add(rows, c[k] < kStepCap ? c[k] : kStepCap);
      fresh = step_add(fresh, w[k]);
    }
    uint32_t all_rows, all_new;
    step_scan(rows, fresh, all_rows, all_new, s_wave);
    rows = step_add(rows, row0);
    fresh = step_add(fresh, new0);
#pragma unroll
    for (int k = 0; k < kStepPer; ++k) {
      const int i = threadIdx.x * kStepPer + k;
      const uint32_t end = step_add(rows, c[k] < kStepCap ? c[k] : kStepCap), last = step_add(fresh, w[k]);
      const int status = wide[k] ? 2 : c[k] && end > M ? 3 : w[k] && last > free_count ? 1 : 0;
      if (i < nb) {
        s_row[i] = rows < M ? rows : M;
        s_new[i] = fresh;
        s_len[i] = status == 0 ? static_cast<int>(n[k]) : -1;
        if (status == 0 && w[k]) granted = last;
        if (LONG && status == 0 && c[k] > kStepLong) s_long = 1;
        if ((b0 / kStepTile) % gridDim.x == blockIdx.x) {
          p.q_offsets[b0 + i] = rows < M ? rows : M;
          p.kv_lens[b0 + i] = status == 0 ? n[k] + c[k] : 0;
          p.status[b0 + i] = status;
        }
      }
      rows = end;
      fresh = last;
    }
    row0 = step_add(row0, all_rows);
    new0 = step_add(new0, all_new);
    if (threadIdx.x == 0) {
      s_row[nb] = row0 < M ? row0 : M;
      s_new[nb] = new0;
    }
    __syncthreads();
    // new pages into the table
    const uint32_t top = s_new[nb] < free_count ? s_new[nb] : free_count;
    for (uint32_t x = s_new[0] + blockIdx.x * kStepThreads + threadIdx.x; x < top; x += gridDim.x * kStepThreads) {
      const int i = step_find(s_new, nb, x);
      if (s_len[i] < 0) continue;
      const uint32_t j = step_pages(s_len[i], page) + (x - s_new[i]);
      p.table[static_cast<int64_t>(b0 + i) * p.width + j] = p.free_pages[free_count - 1 - x];
    }
    // rows
    const uint32_t lo = s_row[0] < lo_row ? lo_row : s_row[0], hi = s_row[nb] < hi_row ? s_row[nb] : hi_row;
    // slot and position of row `own` of sequence i, at `depth`
    auto put = [&](int i, uint32_t own, uint32_t depth, int number, uint32_t shift) {
      const uint32_t r = s_row[i] + own, len = s_len[i], token = len + own;
      p.positions[r] = static_cast<int>(len + depth + shift);
      p.slots[r] = number >= 0 && number < p.pages ? static_cast<int64_t>(number) * page + token % page : -1;
    };
    auto number_of = [&](int i, uint32_t own) {  // of its page
      const uint32_t len = s_len[i], j = (len + own) / page, held = step_pages(len, page);
      return j < held ? p.table[static_cast<int64_t>(b0 + i) * p.width + j] : p.free_pages[free_count - 1 - (s_new[i] + (j - held))];
    };
    auto shift_of = [&](int i) { return p.shift ? static_cast<uint32_t>(p.shift[b0 + i]) : 0u; };
    auto is_long = [&](int i) { return s_len[i] >= 0 && s_row[i + 1] - s_row[i] > kStepLong; };
    const bool longs = LONG && s_long;
    for (uint32_t r = lo + threadIdx.x; r < hi; r += kStepThreads) {
      const int i = step_find(s_row, nb, r), len = s_len[i];
      const uint32_t start = s_row[i], own = r - start;
      uint32_t* mask = p.words ? p.tree + static_cast<int64_t>(r) * p.words : nullptr;
      if (LONG && __builtin_expect(longs, 0) && is_long(i)) continue;
      if (len < 0) {
        p.slots[r] = -1;
        p.positions[r] = 0;
        for (int k = 0; k < p.words; ++k) mask[k] = 0;
        continue;
      }
      const int number = number_of(i, own);
      const uint32_t shift = shift_of(i);
      // to the root (while the page's number is on its way): its steps, and a bit for each row on the way (they descend, so a word is done when
      // the next one is below it)
      uint32_t depth = own;
      if (TREE) {
        const bool near = start >= first;
        depth = 0;
        int k = p.words - 1;
        uint32_t bits = 0;
        for (uint32_t a = own;;) {
          const int word = a >> 5;
          if (word < p.words) {
            for (; k > word; --k) {
              mask[k] = bits;
              bits = 0;
            }
            bits |= 1u << (a & 31);
          }
          if (a == 0) break;
          const int up = near ? s_parent[start + a - first] : p.parents[start + a];
          if (up < 0 || static_cast<uint32_t>(up) >= a) break;
          a = up;
          ++depth;
        }
        for (; k >= 0; --k) {
          mask[k] = bits;
          bits = 0;
        }
      } else {
        for (int k = 0; k < p.words; ++k) mask[k] = step_ones(own, k);  // a chain: rows 0 .. own
      }
      put(i, own, depth, number, shift);
    }
    if (LONG && __builtin_expect(longs, 0) && lo < hi) {  // of the trees that are not walked, the rows of this workgroup that begin with a chain
      for (int i = step_find(s_row, nb, lo); i < nb && s_row[i] < hi; ++i) {
        if (!is_long(i)) continue;
        const uint32_t start = s_row[i], end = s_row[i + 1] < hi ? s_row[i + 1] : hi, shift = shift_of(i);
        const uint32_t e = step_chain(p.parents + start, end - start, s_chain), from = lo > start ? lo - start : 0;
        for (uint32_t own = from + threadIdx.x; own < e; own += kStepThreads) put(i, own, own, number_of(i, own), shift);
        const int64_t words = p.words;
        for (int64_t x = from * words + threadIdx.x; x < e * words; x += kStepThreads)
          p.tree[start * words + x] = step_ones(x / words, static_cast<int>(x % words));
      }
    }
    if (LONG && __builtin_expect(longs, 0)) {  // and of every one of them that is this workgroup's the rows behind
      for (int i = 0; i < nb; ++i) {
        if ((b0 + i) % gridDim.x != blockIdx.x || !is_long(i)) continue;
        const uint32_t start = s_row[i], n = s_row[i + 1] - start, shift = shift_of(i), base = static_cast<uint32_t>(s_len[i]) + shift;
        const uint32_t e = step_chain(p.parents + start, n, s_chain);
        if (e == n) continue;
        step_long(p.parents + start, n, e, p.words ? p.tree + static_cast<int64_t>(start) * p.words : nullptr, p.words, s_tile,
                  [&](uint32_t a, uint32_t depth) { put(i, a, depth, number_of(i, a), shift); },
                  [&](uint32_t a) { return static_cast<uint32_t>(p.positions[start + a]) - base; });
      }
    }
    __syncthreads();
  }
  // rows behind the last sequence's
  const uint32_t used = row0 < M ? row0 : M;
  for (uint32_t r = (used < lo_row ? lo_row : used) + threadIdx.x; r < hi_row; r += kStepThreads) {
    p.slots[r] = -1;
    p.positions[r] = 0;
    for (int k = 0; k < p.words; ++k) p.tree[static_cast<int64_t>(r) * p.words + k] = 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.q_offsets[p.B] = used;
  if (granted) atomicMax(&s_granted, granted);
  __syncthreads();
  const bool takes = p.left == p.state;
  if (takes && gridDim.x > 1) {
    if (step_last(p.state, s_arrived) && threadIdx.x == 0) {
      p.state[0] = free_count - s_granted;
      p.state[1] = 0;
    }
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.left[0] = free_count - s_granted;
  }
}

// A sequence at the end of a step: tokens before it, its rows, those that stay, pages that go back.
struct KeepSeq {
  uint32_t len, rows, kept, end, from, back;  // back: pages from .. from + back
  int first;                                  // of the rows, in the step
};
__device__ __forceinline__ KeepSeq keep_seq(const KeepArgs& p, int b) {
  KeepSeq s;
  const uint32_t page = p.page, cap = page * static_cast<uint32_t>(p.width);
  const int len = p.lens[b], kept = p.kept[b];
  s.len = len < 0 ? 0 : len;
  s.len = s.len < cap ? s.len : cap;
  int rows = 0;
  s.first = 0;
  if (p.q_offsets && !(p.status && p.status[b])) {
    const int lo = p.q_offsets[b], hi = p.q_offsets[b + 1];
    s.first = lo < 0 ? 0 : lo < p.M ? lo : p.M;
    rows = (hi < p.M ? hi : p.M) - s.first;
    rows = rows < 0 ? 0 : rows;
  }
  s.rows = static_cast<uint32_t>(rows) < cap - s.len ? rows : cap - s.len;
  s.kept = kept < 0 ? 0 : static_cast<uint32_t>(kept) < s.rows ? kept : s.rows;
  s.end = kept < 0 ? 0 : s.len + s.kept;
  s.from = step_pages(s.end, page);
  s.back = step_pages(s.len + s.rows, page) - s.from;
  return s;
}

// Column `col` of head h of the kept rows of sequence b, moved to their places.
__device__ __forceinline__ void keep_move(const KeepArgs& p, int b, const KeepSeq& s, int item) {
  const int kc = p.c.k.wpr >> 1, vc = p.c.v.wpr >> 1, ks = p.c.D / p.c.k.group, vs = p.c.D / p.c.v.group;
  const int cols = kc + vc + ks + vs, h = item / cols;
  int col = item - h * cols;
  const bool scale = col >= kc + vc;
  if (scale) col -= kc + vc;
  const bool value = col >= (scale ? ks : kc);
  if (value) col -= scale ? ks : kc;
  const KvHalf& half = value ? p.c.v : p.c.k;
  const int64_t step = scale ? (value ? vs : ks) * 2 : half.wpr * 4;  // bytes of a row
  char* base = scale ? reinterpret_cast<char*>(half.scales) + col * 2 : reinterpret_cast<char*>(half.codes) + col * 8;
  const int32_t* path = p.path + s.first;
  const int32_t* table = p.table + static_cast<int64_t>(b) * p.width;
  auto row = [&](uint32_t token) -> int64_t {  // byte offset of its row, -1 outside the cache
    const uint32_t j = token / static_cast<uint32_t>(p.page);
    const int number = table[j];
    if (number < 0 || number >= p.pages) return -1;
    return ((static_cast<int64_t>(number) * p.c.heads + h) * p.page + (token - j * p.page)) * step;
  };
  for (uint32_t j = 1; j < s.kept; ++j) {
    const int from = path[j];
    if (from <= static_cast<int>(j) || from >= static_cast<int>(s.rows)) continue;
    const int64_t a = row(s.len + from), d = row(s.len + j);
    if (a < 0 || d < 0) continue;
    if (scale) *reinterpret_cast<uint16_t*>(base + d) = *reinterpret_cast<const uint16_t*>(base + a);
    else *reinterpret_cast<u32x2_t*>(base + d) = *reinterpret_cast<const u32x2_t*>(base + a);
  }
}

// Workgroup 0: pages and lengths; the others: `each` of them per sequence move its rows.
__global__ __launch_bounds__(kStepThreads) void k_kv_keep(KeepArgs p, int each, int items) {
  __shared__ uint32_t s_back[kStepTile + 1];
  __shared__ int s_from[kStepTile];
  __shared__ uint32_t s_wave[2][kStepThreads / 64];
  __shared__ int s_arrived;
  const uint32_t free_count = step_free(p.state, p.pages);
  // in place, the last workgroup writes what the others read
  const bool late = gridDim.x > 1 && (p.left == p.state || p.lens_out == p.lens);
  uint32_t total = 0;
  auto sum_all = [&]() {  // pages that go back; as every thread's result
    uint32_t a = 0, b = 0, ta, tb;
    for (int s = threadIdx.x; s < p.B; s += kStepThreads) a = step_add(a, keep_seq(p, s).back);
    step_scan(a, b, ta, tb, s_wave);
    return ta;
  };
  auto put_left = [&](uint32_t back) {
    const uint32_t now = step_add(free_count, back);
    p.left[0] = now < static_cast<uint32_t>(p.pages) ? now : p.pages;
  };
  if (blockIdx.x > 0) {
    for (int unit = blockIdx.x - 1; unit < p.B * each; unit += gridDim.x - 1) {
      const int b = unit / each, item = (unit - b * each) * kStepThreads + threadIdx.x;
      if (item < items) keep_move(p, b, keep_seq(p, b), item);
    }
  } else {
    total = sum_all();
    uint32_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += kStepTile) {
      const int nb = p.B - b0 < kStepTile ? p.B - b0 : kStepTile;
      uint32_t back[kStepPer], sum = 0, none = 0, all, zero;
#pragma unroll
      for (int k = 0; k < kStepPer; ++k) {
        const int i = threadIdx.x * kStepPer + k;
        back[k] = 0;
        if (i < nb) {
          const KeepSeq s = keep_seq(p, b0 + i);
          back[k] = s.back;
          s_from[i] = s.from;
          if (!late) p.lens_out[b0 + i] = s.end;
        }
        sum = step_add(sum, back[k]);
      }
      step_scan(sum, none, all, zero, s_wave);
      sum = step_add(sum, before);
#pragma unroll
      for (int k = 0; k < kStepPer; ++k) {
        const int i = threadIdx.x * kStepPer + k;
        if (i < nb) s_back[i] = sum;
        sum = step_add(sum, back[k]);
      }
      before = step_add(before, all);
      if (threadIdx.x == 0) s_back[nb] = before;
      __syncthreads();
      for (uint32_t x = s_back[0] + threadIdx.x; x < s_back[nb]; x += kStepThreads) {
        const int i = step_find(s_back, nb, x);
        const uint32_t at = free_count + total - 1 - x;
        const uint32_t j = s_from[i] + (x - s_back[i]);
        if (at < static_cast<uint32_t>(p.pages)) p.free_pages[at] = p.table[static_cast<int64_t>(b0 + i) * p.width + j];
      }
      __syncthreads();
    }
    if (!late && threadIdx.x == 0) put_left(total);
  }
  if (!late || !step_last(p.state, s_arrived)) return;
  total = sum_all();
  for (int b = threadIdx.x; b < p.B; b += kStepThreads) p.lens_out[b] = keep_seq(p, b).end;
  if (threadIdx.x == 0) {
    put_left(total);
    p.state[1] = 0;
  }
}

}  // namespace

hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s) {
  int blocks = (a.M + kStepThreads - 1) / kStepThreads;
  blocks = blocks < 1 ? 1 : blocks > 256 ? 256 : blocks;
  const int each = (a.M + blocks - 1) / blocks;
  const auto plan = !a.parents ? k_kv_plan<false, false> : a.M <= static_cast<int>(kStepLong) ? k_kv_plan<true, false> : k_kv_plan<true, true>;
  hipLaunchKernelGGL(plan, dim3(blocks), dim3(kStepThreads), 0, s, a, each);
  return hipGetLastError();
}

hipError_t launch_kv_keep(const KeepArgs& a, hipStream_t s) {
  int each = 0, items = 0;
  if (a.path) {
    items = a.c.heads * (a.c.k.wpr / 2 + a.c.v.wpr / 2 + a.c.D / a.c.k.group + a.c.D / a.c.v.group);
    each = (items + kStepThreads - 1) / kStepThreads;
  }
  const int units = a.B * each;  // (at most 65536 * 320)
  hipLaunchKernelGGL(k_kv_keep, dim3(1 + (units < 65536 ? units : 65536)), dim3(kStepThreads), 0, s, a, each, items);
  return hipGetLastError();
}

}  // namespace tq
