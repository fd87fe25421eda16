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
#include "device_common.hpp"
#include "internal.hpp"

namespace tq {
namespace {

constexpr int kVerifyThreads = 256;

// Of a row of logits: exp((x - ref) / T) = 2^((x - ref) c) with c = log2(e) / T; z the sum (NaN: not a
// distribution); top the index of the largest value (-1: none).
struct RowStat {
  double ref, z;
  int top, pad;
};

struct Side {  // target or draft
  const char* data;
  int dt;
  int64_t stride;
  bool probs;
  RowStat* stat;  // [M], of logits and greedy rows
};
struct VerifyParams {
  VerifyArgs a;
  Side t, d;
};

__device__ __forceinline__ double temperature_of(const VerifyArgs& a, int b) { return a.temperature ? a.temperature[b] : 1.0; }

__device__ __forceinline__ const char* row_of(const Side& s, int row) {
  return s.data + row * s.stride * (s.dt == 0 ? 4 : 2);
}

// The probability of one token of a row.
struct Dist {
  const char* row;
  int dt, top;  // top: greedy rows are point masses
  bool probs, greedy;
  double c, ref, zinv;
  __device__ __forceinline__ double at(int i) const {
    if (greedy) return i == top ? 1.0 : top < 0 ? __builtin_nan("") : 0.0;
    const double x = load_any(row, dt, i);
    if (probs) return x;
    return x == -__builtin_inf() ? 0.0 * zinv : exp2((x - ref) * c) * zinv;
  }
};

__device__ __forceinline__ Dist dist_of(const Side& s, int row, double T, bool greedy) {
  Dist d;
  d.row = row_of(s, row);
  d.dt = s.dt;
  d.probs = s.probs;
  d.greedy = greedy;
  d.top = -1;
  d.c = d.ref = d.zinv = 0.0;
  if (greedy) d.top = s.stat[row].top;
  else if (!s.probs) {
    d.c = 1.4426950408889634074 / T;
    d.ref = s.stat[row].ref;
    d.zinv = 1.0 / s.stat[row].z;
  }
  return d;
}

__device__ __forceinline__ int seq_of(const int32_t* offsets, int B, int row) {
  int lo = 0, hi = B;  // the largest b with offsets[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= row) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <typename T, typename F>
__device__ __forceinline__ T block_join(T x, T* shared, F f) {
  __syncthreads();
  shared[threadIdx.x] = x;
  __syncthreads();
  for (int s = kVerifyThreads / 2; s; s >>= 1) {
    if (static_cast<int>(threadIdx.x) < s) shared[threadIdx.x] = f(shared[threadIdx.x], shared[threadIdx.x + s]);
    __syncthreads();
  }
  return shared[0];
}

// Statistics of the rows of one side: a workgroup per row.
__global__ __launch_bounds__(kVerifyThreads) void k_verify_stats(VerifyParams p, bool draft) {
  __shared__ double sd[kVerifyThreads];
  __shared__ int si[kVerifyThreads];
  const VerifyArgs& a = p.a;
  const Side& s = draft ? p.d : p.t;
  const int row = blockIdx.x;
  const int lim = a.offsets[a.B] < a.M ? a.offsets[a.B] : a.M;
  if (row >= lim) return;
  const double T = temperature_of(a, seq_of(a.offsets, a.B, row));
  const bool greedy = !(T > 0.0);
  if (greedy ? draft : s.probs) return;
  const char* x = row_of(s, row);
  double top = -__builtin_inf(), bad = 0.0;
  int at = 0x7fffffff;
  for (int i = threadIdx.x; i < a.V; i += kVerifyThreads) {
    const double v = load_any(x, s.dt, i);
    if (v != v || v == __builtin_inf()) bad = 1.0;
    if (v > top) {
      top = v;
      at = i;
    }
  }
  bad = block_join(bad, sd, [](double u, double v) { return u > v ? u : v; });
  const double most = block_join(top, sd, [](double u, double v) { return u > v ? u : v; });
  const int first = block_join(top == most ? at : 0x7fffffff, si, [](int u, int v) { return u < v ? u : v; });
  RowStat r{};
  const bool none = bad > 0.0 || (s.probs ? !(most > 0.0) : most == -__builtin_inf());
  r.top = none ? -1 : first;
  if (!greedy) {
    const double c = 1.4426950408889634074 / T;
    r.ref = most;
    double z = 0.0;
    if (!none)
      for (int i = threadIdx.x; i < a.V; i += kVerifyThreads) {
        const double v = load_any(x, s.dt, i);
        if (v != -__builtin_inf()) z += exp2((v - r.ref) * c);
      }
    z = block_join(z, sd, [](double u, double v) { return u + v; });
    r.z = none ? __builtin_nan("") : z;
  }
  if (threadIdx.x == 0) s.stat[row] = r;
}

// The walk and the new token: a workgroup per sequence.
__global__ __launch_bounds__(kVerifyThreads) void k_verify_walk(VerifyParams p) {
  __shared__ double sd[kVerifyThreads];
  __shared__ int si[kVerifyThreads];
  const VerifyArgs& a = p.a;
  const int b = blockIdx.x, V = a.V;
  int lo = a.offsets[b], hi = a.offsets[b + 1];
  lo = lo < 0 ? 0 : lo < a.M ? lo : a.M;
  hi = hi < lo ? lo : hi < a.M ? hi : a.M;
  const int n = hi - lo;
  if (n == 0) {
    if (threadIdx.x == 0) a.kept[b] = 0;
    return;
  }
  for (int i = threadIdx.x; i < n; i += kVerifyThreads) {
    a.out_tokens[lo + i] = -1;
    a.path[lo + i] = i == 0 ? 0 : -1;
  }
  __syncthreads();
  const double T = temperature_of(a, b);
  const bool greedy = !(T > 0.0), drafted = a.draft && !greedy;
  int cur = 0, kept = 1, tried = 0;  // tried: children of cur that went
  double al = 0.0, S = 1.0;
  Dist t = dist_of(p.t, lo, T, greedy), q{};
  if (drafted && n > 1) q = dist_of(p.d, lo, T, false);
  // (a child tried before with the same token took it out)
  auto gone = [&](int x, int end) {
    for (int r = cur + 1; r < end; ++r)
      if ((a.parents ? a.parents[lo + r] : r - 1) == cur && a.tokens[lo + r] == x) return true;
    return false;
  };
  auto weight = [&](int i, bool fresh, int end) {
    double w = t.at(i);
    if (!fresh) {
      if (drafted) w -= al * q.at(i);
      else if (tried && gone(i, end)) w = 0.0;
    }
    return w < 0.0 ? 0.0 : w;
  };
  auto sum = [&](bool fresh, int end) {
    double w = 0.0;
    for (int i = threadIdx.x; i < V; i += kVerifyThreads) w += weight(i, fresh, end);
    return block_join(w, sd, [](double u, double v) { return u + v; });
  };
  for (int r = 1; r < n; ++r) {
    if ((a.parents ? a.parents[lo + r] : r - 1) != cur) continue;
    const int x = a.tokens[lo + r];
    if (x < 0 || x >= V) continue;
    const double u = a.uniforms[lo + r], px = t.at(x);
    bool yes;
    if (greedy) {
      yes = x == t.top;
    } else if (drafted) {
      const double qx = q.at(x);
      yes = u * S * qx < px - al * qx;
    } else {
      yes = u * S < (gone(x, r) ? 0.0 : px);
    }
    if (yes) {
      if (threadIdx.x == 0) {
        a.out_tokens[lo + kept - 1] = x;
        a.path[lo + kept] = r;
      }
      cur = r;
      ++kept;
      tried = 0;
      al = 0.0;
      S = 1.0;
      t = dist_of(p.t, lo + r, T, greedy);
      if (drafted && r + 1 < n) q = dist_of(p.d, lo + r, T, false);
    } else {
      ++tried;
      if (drafted) {
        al += S;
        if (a.parents) S = sum(false, n);
      } else if (!gone(x, r)) {
        S -= px;
      }
    }
  }
  // the new token: threads take neighbouring pieces of the row
  bool fresh = drafted ? al == 0.0 : tried == 0;
  const int each = (V + kVerifyThreads - 1) / kVerifyThreads;
  const int i0 = threadIdx.x * each < V ? threadIdx.x * each : V, i1 = i0 + each < V ? i0 + each : V;
  double own, total;
  for (;;) {
    own = 0.0;
    for (int i = i0; i < i1; ++i) own += weight(i, fresh, n);
    total = block_join(own, sd, [](double u, double v) { return u + v; });
    if (total == 0.0 && !fresh) fresh = true;
    else break;
  }
  __syncthreads();
  sd[threadIdx.x] = own;
  __syncthreads();
  double before = 0.0;
  for (int k = 0; k < static_cast<int>(threadIdx.x); ++k) before += sd[k];
  int pick = 0x7fffffff, lastw = -1;
  const double u = a.uniforms[lo], goal = (u > 0.0 ? u : 0.0) * total;
  for (int i = i0; i < i1; ++i) {
    const double w = weight(i, fresh, n);
    before += w;
    if (w > 0.0) {
      lastw = i;
      if (before > goal && pick == 0x7fffffff) pick = i;
    }
  }
  pick = block_join(pick, si, [](int u, int v) { return u < v ? u : v; });
  lastw = block_join(lastw, si, [](int u, int v) { return u > v ? u : v; });
  if (threadIdx.x == 0) {
    a.kept[b] = kept;
    a.out_tokens[lo + kept - 1] = !(total > 0.0) || total == __builtin_inf() ? -1 : pick < V ? pick : lastw;
  }
}

VerifyParams make_params(const VerifyArgs& a) {
  VerifyParams p{};
  p.a = a;
  p.t = Side{static_cast<const char*>(a.target), a.tdt, a.tstride, a.tprobs, static_cast<RowStat*>(a.ws)};
  p.d = Side{static_cast<const char*>(a.draft), a.ddt, a.dstride, a.dprobs, static_cast<RowStat*>(a.ws) + a.M};
  return p;
}

}  // namespace

size_t verify_workspace(int V, int B, int M, bool tprobs, bool drafted, bool dprobs) {
  return 2 * static_cast<size_t>(M) * sizeof(RowStat);
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  const VerifyParams p = make_params(a);
  if (a.M > 0) {
    hipLaunchKernelGGL(k_verify_stats, dim3(a.M), dim3(kVerifyThreads), 0, s, p, false);
    if (a.draft && !a.dprobs) hipLaunchKernelGGL(k_verify_stats, dim3(a.M), dim3(kVerifyThreads), 0, s, p, true);
  }
  hipLaunchKernelGGL(k_verify_walk, dim3(a.B), dim3(kVerifyThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace tq
