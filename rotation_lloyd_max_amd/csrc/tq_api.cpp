// Host side of libtq: the C entry points declared in include/tq.h.
//
// Every call validates its arguments before launching anything, reports failures through a
// negative status and a thread-local message, and never throws or aborts across the C
// interface. The Lloyd-Max codebooks are computed here once, in double precision, by
// Lloyd's iteration on the N(0,1) density (turboquant-mlx "How it works", "Quantizing a
// weight, with no data", third bullet: one fixed codebook per bit width, a mathematical
// constant; "The ternary tier (1.58 bits)": levels {-c, 0, +c}).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/tq.h"
#include "../../include/tq_kv.h"
#include "../../include/tq_step.h"
#include "internal.hpp"

namespace tq {
namespace {

thread_local std::string g_err;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return TQ_OK;
  return fail(TQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// ---- Lloyd-Max codebooks ---------------------------------------------------------------
double normal_pdf(double x) {
  if (std::isinf(x)) return 0.0;
  return std::exp(-0.5 * x * x) / std::sqrt(2.0 * M_PI);
}
// P(X > x)
double normal_sf(double x) {
  if (x == INFINITY) return 0.0;
  if (x == -INFINITY) return 1.0;
  return 0.5 * std::erfc(x / std::sqrt(2.0));
}
// P(a < X <= b), evaluated on the side of 0 where it does not cancel
double cell_mass(double a, double b) {
  if (a >= 0.0) return normal_sf(a) - normal_sf(b);
  if (b <= 0.0) return normal_sf(-b) - normal_sf(-a);
  return 1.0 - normal_sf(-a) - normal_sf(b);
}

void lloyd(int L, double* c, double* t) {
  for (int k = 0; k < L; ++k) c[k] = -2.0 + 4.0 * (k + 0.5) / L;
  double nc[16];
  for (int it = 0; it < 200000; ++it) {
    for (int k = 0; k + 1 < L; ++k) t[k] = 0.5 * (c[k] + c[k + 1]);
    for (int k = 0; k < L; ++k) {
      const double a = k == 0 ? -INFINITY : t[k - 1];
      const double b = k == L - 1 ? INFINITY : t[k];
      nc[k] = (normal_pdf(a) - normal_pdf(b)) / cell_mass(a, b);
    }
    double delta = 0.0;
    for (int k = 0; k < L; ++k) {
      const double v = 0.5 * (nc[k] - nc[L - 1 - k]);  // keep the exact symmetry
      delta = std::fmax(delta, std::fabs(v - c[k]));
      c[k] = v;
    }
    if (delta < 1e-15) break;
  }
  for (int k = 0; k + 1 < L; ++k) t[k] = 0.5 * (c[k] + c[k + 1]);
}

// The 256-level codebook (8-bit KV-cache keys): the same fixed point, but plain Lloyd
// iteration contracts at about 0.99985 per step there and the fixed point amplifies the
// map's rounding errors about 10^4 times, so it is computed in 80-bit long double: Lloyd
// steps from the same start, then Newton's method on lloyd(c) - c = 0 with the tridiagonal
// Jacobian of the map (d mean / d b = pdf(b) (b - mean) / P, d mean / d a = pdf(a)
// (mean - a) / P, each threshold the midpoint of its neighbours).
typedef long double ldbl;
ldbl pdf_l(ldbl x) { return std::exp(-0.5L * x * x) / std::sqrt(2.0L * 3.14159265358979323846264338327950288L); }
ldbl sf_l(ldbl x) { return 0.5L * std::erfc(x / std::sqrt(2.0L)); }
ldbl mass_l(ldbl a, ldbl b, bool a_inf, bool b_inf) {
  const ldbl Qa = a_inf ? 1.0L : sf_l(a), Qb = b_inf ? 0.0L : sf_l(b);
  if (!a_inf && a >= 0) return Qa - Qb;
  if (!b_inf && b <= 0) return (b_inf ? 1.0L : sf_l(-b)) - (a_inf ? 0.0L : sf_l(-a));
  return 1.0L - (a_inf ? 0.0L : sf_l(-a)) - Qb;
}

void lloyd_big(int L, double* c_out, double* t_out) {
  std::vector<ldbl> c(L), nc(L), t(L - 1), g(L), sub(L), dia(L), sup(L), cp(L), dp(L), d(L);
  for (int k = 0; k < L; ++k) c[k] = -2.0L + 4.0L * (k + 0.5L) / L;
  auto step = [&](bool jac) {
    for (int k = 0; k + 1 < L; ++k) t[k] = 0.5L * (c[k] + c[k + 1]);
    for (int k = 0; k < L; ++k) {
      const bool ai = k == 0, bi = k == L - 1;
      const ldbl a = ai ? 0.0L : t[k - 1], b = bi ? 0.0L : t[k];
      const ldbl pa = ai ? 0.0L : pdf_l(a), pb = bi ? 0.0L : pdf_l(b);
      const ldbl P = mass_l(a, b, ai, bi);
      const ldbl m = (pa - pb) / P;
      nc[k] = m;
      if (jac) {
        const ldbl da = ai ? 0.0L : pa * (m - a) / P;
        const ldbl db = bi ? 0.0L : pb * (b - m) / P;
        sub[k] = da / 2;
        dia[k] = (da + db) / 2 - 1;
        sup[k] = db / 2;
      }
    }
  };
  for (int it = 0; it < 2000; ++it) {
    step(false);
    for (int k = 0; k < L; ++k) c[k] = 0.5L * (nc[k] - nc[L - 1 - k]);
  }
  for (int it = 0; it < 40; ++it) {
    step(true);
    for (int k = 0; k < L; ++k) g[k] = nc[k] - c[k];
    cp[0] = sup[0] / dia[0];
    dp[0] = -g[0] / dia[0];
    for (int k = 1; k < L; ++k) {
      const ldbl den = dia[k] - sub[k] * cp[k - 1];
      cp[k] = sup[k] / den;
      dp[k] = (-g[k] - sub[k] * dp[k - 1]) / den;
    }
    d[L - 1] = dp[L - 1];
    for (int k = L - 2; k >= 0; --k) d[k] = dp[k] - cp[k] * d[k + 1];
    ldbl dmax = 0;
    for (int k = 0; k < L; ++k) {
      c[k] += d[k];
      dmax = std::fmax(dmax, std::fabs(d[k]));
    }
    for (int k = 0; k < L; ++k) nc[k] = 0.5L * (c[k] - c[L - 1 - k]);
    for (int k = 0; k < L; ++k) c[k] = nc[k];
    if (dmax < 1e-17L) break;
  }
  for (int k = 0; k < L; ++k) c_out[k] = static_cast<double>(c[k]);
  for (int k = 0; k + 1 < L; ++k) t_out[k] = static_cast<double>(0.5L * (c[k] + c[k + 1]));
}

CodebookArgs g_books[4];
BigCodebook g_big;
std::once_flag g_books_once;

void init_books() {
  const int levels[4] = {3, 4, 8, 16};
  for (int i = 0; i < 4; ++i) {
    CodebookArgs& b = g_books[i];
    std::memset(&b, 0, sizeof b);
    const int L = levels[i];
    double c[16], t[15];
    lloyd(L, c, t);
    b.levels = L;
    for (int k = 0; k < L; ++k) {
      b.c[k] = static_cast<float>(c[k]);
      const _Float16 h = static_cast<_Float16>(c[k]);
      std::memcpy(&b.h[k], &h, 2);
    }
    for (int k = 0; k + 1 < L; ++k) b.t[k] = static_cast<float>(t[k]);
  }
  {
    std::vector<double> c(256), t(255);
    lloyd_big(256, c.data(), t.data());
    for (int k = 0; k < 256; ++k) {
      g_big.c[k] = static_cast<float>(c[k]);
      const _Float16 h = static_cast<_Float16>(c[k]);
      std::memcpy(&g_big.h[k], &h, 2);
    }
    for (int k = 0; k < 255; ++k) g_big.t[k] = static_cast<float>(t[k]);
  }
}

int64_t words_per_row(int64_t K, int levels) {
  switch (levels) {
    case 3: return (K + 19) / 20;
    case 4: return (2 * K + 31) / 32;
    case 8: return (3 * K + 31) / 32;
    case 16: return (4 * K + 31) / 32;
    case 256: return (8 * K + 31) / 32;
    default: return 0;
  }
}

bool valid_dtype(int d) { return d == TQ_F32 || d == TQ_BF16 || d == TQ_F16; }
size_t dtype_size(int d) { return d == TQ_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// allow256: the 8-bit codebook (KV-cache rows), for power-of-two K up to 4096 only;
// any_k: no Hadamard transform is applied (pre-rotated inputs, dense rotations,
// dequantization), so K need only be a multiple of 32 in [64, 8192]
int check_shape(int64_t K, int levels, int group, int* m, int* P, bool allow256 = false,
                bool any_k = false) {
  if (levels == 256 && allow256) {
    if (K < 64 || K > 4096 || (K & (K - 1)) != 0)
      return fail(TQ_ERR_UNSUPPORTED, "256 levels need K a power of two in [64, 4096] (got %lld)",
                  static_cast<long long>(K));
  } else if (levels != 3 && levels != 4 && levels != 8 && levels != 16) {
    return fail(TQ_ERR_UNSUPPORTED, "n_levels must be 3, 4, 8 or 16%s (got %d)",
                allow256 ? " (or 256)" : "", levels);
  }
  if (group != 16 && group != 32 && group != 64 && group != 128)
    return fail(TQ_ERR_UNSUPPORTED, "group must be 16, 32, 64 or 128 (got %d)", group);
  if (K < 64 || K > 8192 || K % 32 != 0)
    return fail(TQ_ERR_UNSUPPORTED, "K must be a multiple of 32 in [64, 8192] (got %lld)",
                static_cast<long long>(K));
  if (!split_dim(K, m, P)) {
    if (!any_k)
      return fail(TQ_ERR_UNSUPPORTED,
                  "K=%lld is not m*2^k with m in {1, 12, 20, 28} (a dense rotation and "
                  "TQ_X_ROTATED inputs take any multiple of 32)",
                  static_cast<long long>(K));
    *m = 1;
    *P = static_cast<int>(K);
  }
  if (K % group != 0)
    return fail(TQ_ERR_UNSUPPORTED, "group %d does not divide K=%lld", group,
                static_cast<long long>(K));
  return TQ_OK;
}

// rotated: the call applies no rotation of its own (TQ_X_ROTATED inputs, dequantization), so
// K may be any multiple of 32 in [64, 8192] and the sign bits are not needed
int check_weight(const tq_qweight* w, WeightArgs* out, bool allow256 = false,
                 bool rotated = false) {
  if (!w) return fail(TQ_ERR_ARG, "weight descriptor is NULL");
  int m = 1, P = 1;
  const int rc = check_shape(w->K, w->n_levels, w->group, &m, &P, allow256, rotated);
  if (rc != TQ_OK) return rc;
  if (w->N < 0 || w->N > (1 << 24)) return fail(TQ_ERR_ARG, "N out of range");
  if (w->E < 1 || w->E > 8192) return fail(TQ_ERR_ARG, "E must be in [1, 8192]");
  if (w->N > 0) {
    if (!w->codes || !w->scales || (!w->signs && !rotated))
      return fail(TQ_ERR_ARG, "codes, scales and signs must be non-NULL");
    if (!aligned(w->codes, 16)) return fail(TQ_ERR_ALIGN, "codes must be 16-byte aligned");
    if (!aligned(w->scales, 2) || (w->signs && !aligned(w->signs, 4)))
      return fail(TQ_ERR_ALIGN, "scales/signs misaligned");
  }
  out->codes = w->codes;
  out->scales = w->scales;
  out->signs = w->signs;
  out->levels = w->n_levels;
  out->group = w->group;
  out->K = static_cast<int>(w->K);
  out->N = static_cast<int>(w->N);
  out->E = static_cast<int>(w->E);
  out->wpr = static_cast<int>(words_per_row(w->K, w->n_levels));
  out->m = m;
  out->P = P;
  return TQ_OK;
}

// x is read with 16-byte loads (rows of K elements, K a multiple of 32, stay aligned).
int check_io(const void* x, int xdt, const void* y, int ydt, bool need) {
  if (!valid_dtype(xdt) || !valid_dtype(ydt)) return fail(TQ_ERR_ARG, "bad dtype");
  if (!need) return TQ_OK;
  if (!x || !y) return fail(TQ_ERR_ARG, "x and y must be non-NULL");
  if (!aligned(x, 16)) return fail(TQ_ERR_ALIGN, "x must be 16-byte aligned");
  if (!aligned(y, dtype_size(ydt))) return fail(TQ_ERR_ALIGN, "y misaligned for its dtype");
  return TQ_OK;
}

// The two halves of a paged cache: their own limits on levels, group, head dimension and
// pages (tq_kv_cache), the rest as any weight.
int check_half(const tq_qweight& w, const char* name, int64_t rows, KvHalf* out) {
  if (w.n_levels != 4 && w.n_levels != 8 && w.n_levels != 16 && w.n_levels != 256)
    return fail(TQ_ERR_UNSUPPORTED, "cache %s: n_levels must be 4, 8, 16 or 256 (got %d)", name,
                w.n_levels);
  if (w.K != 64 && w.K != 128 && w.K != 256)
    return fail(TQ_ERR_UNSUPPORTED, "cache %s: the head dimension must be 64, 128 or 256 (got %lld)",
                name, static_cast<long long>(w.K));
  if ((w.group != 32 && w.group != 64 && w.group != 128) || w.K % w.group != 0)
    return fail(TQ_ERR_UNSUPPORTED,
                "cache %s: group must be 32, 64 or 128 and divide the head dimension (got %d)",
                name, w.group);
  if (w.N != rows)
    return fail(TQ_ERR_ARG, "cache %s: N must be heads * page_tokens = %lld (got %lld)", name,
                static_cast<long long>(rows), static_cast<long long>(w.N));
  if (w.E < 1 || w.E > 0x7fffffffll) return fail(TQ_ERR_ARG, "cache %s: pages out of range", name);
  if (!w.codes || !w.scales || !w.signs)
    return fail(TQ_ERR_ARG, "cache %s: codes, scales and signs must be non-NULL", name);
  if (!aligned(w.codes, 16) || !aligned(w.scales, 8) || !aligned(w.signs, 4))
    return fail(TQ_ERR_ALIGN, "cache %s: codes must be 16-byte, scales 8-byte and signs 4-byte aligned",
                name);
  out->codes = const_cast<uint32_t*>(w.codes);
  out->scales = const_cast<uint16_t*>(w.scales);
  out->signs = w.signs;
  out->levels = w.n_levels;
  out->bits = w.n_levels == 256 ? 8 : w.n_levels == 16 ? 4 : w.n_levels == 8 ? 3 : 2;
  out->group = w.group;
  out->wpr = static_cast<int>(w.K) * out->bits / 32;
  return TQ_OK;
}

int check_cache(const tq_kv_cache* c, KvCacheArgs* out) {
  if (!c) return fail(TQ_ERR_ARG, "cache descriptor is NULL");
  if (c->heads < 1 || c->heads > 1024) return fail(TQ_ERR_ARG, "cache heads must be in [1, 1024]");
  if (c->page_tokens < 16 || c->page_tokens > 65536 || c->page_tokens % 16 != 0)
    return fail(TQ_ERR_ARG, "page_tokens must be a multiple of 16 in [16, 65536] (got %d)",
                c->page_tokens);
  const int64_t rows = static_cast<int64_t>(c->heads) * c->page_tokens;
  int rc = check_half(c->k, "keys", rows, &out->k);
  if (rc != TQ_OK) return rc;
  rc = check_half(c->v, "values", rows, &out->v);
  if (rc != TQ_OK) return rc;
  if (c->k.K != c->v.K || c->k.E != c->v.E)
    return fail(TQ_ERR_ARG, "cache keys and values differ in head dimension or pages");
  out->D = static_cast<int>(c->k.K);
  out->heads = c->heads;
  out->page = c->page_tokens;
  out->pages = c->k.E;
  return TQ_OK;
}

int check_rope(const tq_rope_params* r, const int32_t* positions, int head_dim, RopeArgs* out) {
  if (!r) return fail(TQ_ERR_ARG, "rope is NULL");
  if (r->rot_dim < 2 || r->rot_dim > head_dim || r->rot_dim % 2 != 0)
    return fail(TQ_ERR_ARG, "rot_dim must be even and in [2, head_dim] (got %d)", r->rot_dim);
  if (r->interleaved != 0 && r->interleaved != 1)
    return fail(TQ_ERR_ARG, "interleaved must be 0 or 1");
  if (!r->inv_freq || !positions) return fail(TQ_ERR_ARG, "inv_freq and positions must be non-NULL");
  if (!aligned(r->inv_freq, 8) || !aligned(positions, 4))
    return fail(TQ_ERR_ALIGN, "inv_freq or positions misaligned");
  out->inv_freq = r->inv_freq;
  out->positions = positions;
  out->rot = r->rot_dim;
  out->interleaved = r->interleaved != 0;
  out->gain = r->gain;
  return TQ_OK;
}

int check_axes(const uint8_t* axis, int64_t axis_stride, int32_t axes, RopeArgs* out) {
  if (!axis) return fail(TQ_ERR_ARG, "axis is NULL");
  if (axes < 1 || axes > 255) return fail(TQ_ERR_ARG, "axes must be in [1, 255] (got %d)", axes);
  if (axis_stride < 0) return fail(TQ_ERR_ARG, "axis_stride must be >= 0");
  out->axis = axis;
  out->axis_stride = axis_stride;
  out->axes = axes;
  return TQ_OK;
}

}  // namespace

const BigCodebook* codebook256() {
  std::call_once(g_books_once, init_books);
  return &g_big;
}

const CodebookArgs* codebook_for(int levels) {
  std::call_once(g_books_once, init_books);
  switch (levels) {
    case 3: return &g_books[0];
    case 4: return &g_books[1];
    case 8: return &g_books[2];
    case 16: return &g_books[3];
    default: return nullptr;
  }
}

bool split_dim(int64_t K, int* m, int* P) {
  const int ms[4] = {1, 12, 20, 28};
  for (int i = 0; i < 4; ++i) {
    if (K % ms[i] != 0) continue;
    const int64_t p = K / ms[i];
    if (p >= 1 && (p & (p - 1)) == 0) {
      *m = ms[i];
      *P = static_cast<int>(p);
      return true;
    }
  }
  return false;
}

}  // namespace tq

using namespace tq;

extern "C" {

int64_t tq_words_per_row(int64_t K, int32_t n_levels) {
  if (K <= 0) return 0;
  return words_per_row(K, n_levels);
}

int tq_codebook(int32_t n_levels, float* centroids, float* thresholds) {
  if (n_levels == 256) {
    if (!centroids) return fail(TQ_ERR_ARG, "centroids is NULL");
    const BigCodebook* g = codebook256();
    std::memcpy(centroids, g->c, sizeof(float) * 256);
    if (thresholds) std::memcpy(thresholds, g->t, sizeof(float) * 255);
    return TQ_OK;
  }
  const CodebookArgs* b = codebook_for(n_levels);
  if (!b) return fail(TQ_ERR_UNSUPPORTED, "n_levels must be 3, 4, 8 or 16 (got %d)", n_levels);
  if (!centroids) return fail(TQ_ERR_ARG, "centroids is NULL");
  std::memcpy(centroids, b->c, sizeof(float) * n_levels);
  if (thresholds) std::memcpy(thresholds, b->t, sizeof(float) * (n_levels - 1));
  return TQ_OK;
}

int tq_signs(uint64_t seed, int64_t K, uint32_t* bits, void* stream) {
  if (K <= 0 || K > (1 << 24)) return fail(TQ_ERR_ARG, "K out of range");
  if (!bits) return fail(TQ_ERR_ARG, "bits is NULL");
  if (!aligned(bits, 4)) return fail(TQ_ERR_ALIGN, "bits must be 4-byte aligned");
  return hip_status(launch_signs(seed, static_cast<int>(K), bits, static_cast<hipStream_t>(stream)),
                    "tq_signs");
}

int tq_encode(const void* W, tq_dtype w_dtype, int64_t rows, int64_t K, int32_t n_levels,
              int32_t group, uint64_t seed, uint32_t* codes, uint16_t* scales, void* stream) {
  int m = 1, P = 1;
  const int rc = check_shape(K, n_levels, group, &m, &P, /*allow256=*/true);
  if (rc != TQ_OK) return rc;
  if (!valid_dtype(w_dtype)) return fail(TQ_ERR_ARG, "bad weight dtype");
  if (rows < 0) return fail(TQ_ERR_ARG, "rows must be >= 0");
  if (rows == 0) return TQ_OK;
  if (!W || !codes || !scales) return fail(TQ_ERR_ARG, "W, codes and scales must be non-NULL");
  if (!aligned(W, dtype_size(w_dtype)) || !aligned(codes, 4) || !aligned(scales, 2))
    return fail(TQ_ERR_ALIGN, "W, codes or scales misaligned");
  if (n_levels == 256 && !aligned(W, 16))
    return fail(TQ_ERR_ALIGN, "256-level encode reads W with 16-byte loads: W must be 16-byte aligned");
  return hip_status(launch_encode(W, w_dtype, rows, static_cast<int>(K), m, P, n_levels, group,
                                  seed, codes, scales, static_cast<hipStream_t>(stream)),
                    "tq_encode");
}

int tq_encode_stream(const void* W_host, tq_dtype w_dtype, int64_t rows, int64_t K,
                     int32_t n_levels, int32_t group, uint64_t seed, uint32_t* codes,
                     uint16_t* scales, void* staging, size_t staging_bytes, void* stream,
                     void* copy_stream) {
  int m = 1, P = 1;
  const int rc = check_shape(K, n_levels, group, &m, &P, /*allow256=*/true);
  if (rc != TQ_OK) return rc;
  if (!valid_dtype(w_dtype)) return fail(TQ_ERR_ARG, "bad weight dtype");
  if (rows < 0) return fail(TQ_ERR_ARG, "rows must be >= 0");
  if (rows == 0) return TQ_OK;
  if (!W_host || !codes || !scales || !staging)
    return fail(TQ_ERR_ARG, "W_host, codes, scales and staging must be non-NULL");
  if (!aligned(W_host, dtype_size(w_dtype)) || !aligned(codes, 4) || !aligned(scales, 2))
    return fail(TQ_ERR_ALIGN, "W_host, codes or scales misaligned");
  if (!aligned(staging, 256)) return fail(TQ_ERR_ALIGN, "staging must be 256-byte aligned");
  // each half of the staging buffer holds `chunk` whole rows and starts 256-byte aligned
  const size_t row_bytes = static_cast<size_t>(K) * dtype_size(w_dtype);
  const size_t half = (staging_bytes / 2) & ~static_cast<size_t>(255);
  const int64_t chunk = static_cast<int64_t>(half / row_bytes);
  if (chunk < 1)
    return fail(TQ_ERR_ARG, "staging of %zu bytes holds fewer than two rows of %zu bytes",
                staging_bytes, row_bytes);
  const int64_t wpr = words_per_row(K, n_levels);
  const int64_t ngk = K / group;
  const hipStream_t cs = static_cast<hipStream_t>(stream);
  const hipStream_t xs = copy_stream ? static_cast<hipStream_t>(copy_stream) : cs;
  // filled[b]: half b holds its chunk (copy done); freed[b]: its encode is done; entry:
  // everything enqueued on `stream` before this call (which may still read `staging`)
  hipEvent_t filled[2] = {nullptr, nullptr}, freed[2] = {nullptr, nullptr}, entry = nullptr;
  hipError_t e = hipSuccess;
  for (int b = 0; b < 2 && e == hipSuccess; ++b) {
    e = hipEventCreateWithFlags(&filled[b], hipEventDisableTiming);
    if (e == hipSuccess) e = hipEventCreateWithFlags(&freed[b], hipEventDisableTiming);
  }
  if (e == hipSuccess && xs != cs) {
    e = hipEventCreateWithFlags(&entry, hipEventDisableTiming);
    if (e == hipSuccess) e = hipEventRecord(entry, cs);
    if (e == hipSuccess) e = hipStreamWaitEvent(xs, entry, 0);
  }
  const char* src = static_cast<const char*>(W_host);
  char* stage = static_cast<char*>(staging);
  for (int64_t i = 0, r0 = 0; e == hipSuccess && r0 < rows; ++i, r0 += chunk) {
    const int b = static_cast<int>(i & 1);
    const int64_t n = rows - r0 < chunk ? rows - r0 : chunk;
    char* buf = stage + b * half;
    // the half is reused once the encode of the chunk it held two steps ago is done
    if (i >= 2) e = hipStreamWaitEvent(xs, freed[b], 0);
    if (e == hipSuccess)
      e = hipMemcpyAsync(buf, src + static_cast<size_t>(r0) * row_bytes,
                         static_cast<size_t>(n) * row_bytes, hipMemcpyHostToDevice, xs);
    if (e == hipSuccess) e = hipEventRecord(filled[b], xs);
    if (e == hipSuccess) e = hipStreamWaitEvent(cs, filled[b], 0);
    if (e == hipSuccess)
      e = launch_encode(buf, w_dtype, n, static_cast<int>(K), m, P, n_levels, group, seed,
                        codes + r0 * wpr, scales + r0 * ngk, cs);
    if (e == hipSuccess) e = hipEventRecord(freed[b], cs);
  }
  for (int b = 0; b < 2; ++b) {
    if (filled[b]) (void)hipEventDestroy(filled[b]);
    if (freed[b]) (void)hipEventDestroy(freed[b]);
  }
  if (entry) (void)hipEventDestroy(entry);
  return hip_status(e, "tq_encode_stream");
}

int tq_fwht(const void* x, tq_dtype x_dtype, int64_t rows, int64_t K, uint64_t seed, void* out,
            tq_dtype out_dtype, void* stream) {
  int m = 1, P = 1;
  if (K < 64 || K > 8192 || K % 32 != 0 || !split_dim(K, &m, &P))
    return fail(TQ_ERR_UNSUPPORTED, "K must be m*2^k (m in {1,12,20,28}), a multiple of 32 in [64, 8192]");
  if (rows < 0) return fail(TQ_ERR_ARG, "rows must be >= 0");
  const int rc = check_io(x, x_dtype, out, out_dtype, rows > 0);
  if (rc != TQ_OK) return rc;
  if (rows == 0) return TQ_OK;
  return hip_status(launch_fwht(x, x_dtype, rows, static_cast<int>(K), m, P, nullptr, seed, out,
                                out_dtype, static_cast<hipStream_t>(stream)),
                    "tq_fwht");
}

size_t tq_workspace_bytes(int32_t op, const tq_qweight* w, int64_t count, int64_t T) {
  WeightArgs a{};
  if (check_weight(w, &a, false, /*rotated=*/true) != TQ_OK || count < 0 || T < 0) return SIZE_MAX;
  switch (op) {
    case TQ_OP_QMV:
    case TQ_OP_GATHER_QMV: return 0;
    case TQ_OP_MULTI_GATHER_QMV: return multi_gather_workspace(a, count);
    case TQ_OP_GATHER_QMM: return gather_qmm_workspace(a, count, T);
    case TQ_OP_ENCODE_DENSE: return static_cast<size_t>(count) * a.K * 8;
    default: fail(TQ_ERR_ARG, "unknown op %d", op); return SIZE_MAX;
  }
}

int tq_qmv(const tq_qweight* w, const void* x, tq_dtype x_dtype, void* y, tq_dtype y_dtype,
           uint32_t flags, void* ws, size_t ws_bytes, void* stream) {
  (void)ws;
  (void)ws_bytes;
  WeightArgs a{};
  int rc = check_weight(w, &a, false, (flags & TQ_X_ROTATED) != 0);
  if (rc != TQ_OK) return rc;
  if (a.E != 1) return fail(TQ_ERR_ARG, "tq_qmv needs E = 1 (use tq_gather_qmv for experts)");
  rc = check_io(x, x_dtype, y, y_dtype, a.N > 0);
  if (rc != TQ_OK) return rc;
  return hip_status(launch_qmv(a, nullptr, 1, x, x_dtype, (flags & TQ_X_ROTATED) != 0, y, y_dtype,
                               static_cast<hipStream_t>(stream)),
                    "tq_qmv");
}

int tq_gather_qmv(const tq_qweight* w, const int32_t* ids, int32_t n, const void* x,
                  tq_dtype x_dtype, void* y, tq_dtype y_dtype, uint32_t flags, void* ws,
                  size_t ws_bytes, void* stream) {
  (void)ws;
  (void)ws_bytes;
  WeightArgs a{};
  int rc = check_weight(w, &a, false, (flags & TQ_X_ROTATED) != 0);
  if (rc != TQ_OK) return rc;
  if (n < 0) return fail(TQ_ERR_ARG, "n must be >= 0");
  if (n > 0 && !ids) return fail(TQ_ERR_ARG, "ids is NULL");
  if (n > 0 && !aligned(ids, 4)) return fail(TQ_ERR_ALIGN, "ids misaligned");
  rc = check_io(x, x_dtype, y, y_dtype, n > 0 && a.N > 0);
  if (rc != TQ_OK) return rc;
  return hip_status(launch_qmv(a, ids, n, x, x_dtype, (flags & TQ_X_ROTATED) != 0, y, y_dtype,
                               static_cast<hipStream_t>(stream)),
                    "tq_gather_qmv");
}

int tq_gather_qmv_pair(const tq_qweight* w1, const tq_qweight* w2, const int32_t* ids, int32_t n,
                       const void* x, tq_dtype x_dtype, void* y, tq_dtype y_dtype, uint32_t flags,
                       void* stream) {
  const bool rotated = (flags & TQ_X_ROTATED) != 0;
  WeightArgs a{}, b{};
  int rc = check_weight(w1, &a, false, rotated);
  if (rc != TQ_OK) return rc;
  rc = check_weight(w2, &b, false, rotated);
  if (rc != TQ_OK) return rc;
  if (a.levels != b.levels || a.group != b.group || a.K != b.K || a.N != b.N || a.E != b.E)
    return fail(TQ_ERR_ARG, "tq_gather_qmv_pair: the two weights differ in format or shape");
  if (!rotated && w1->signs != w2->signs)
    return fail(TQ_ERR_ARG, "tq_gather_qmv_pair: the two weights must share one signs array");
  if (n < 0 || n > 65535) return fail(TQ_ERR_ARG, "n must be in [0, 65535]");
  if (n > 0 && !ids) return fail(TQ_ERR_ARG, "ids is NULL");
  if (n > 0 && !aligned(ids, 4)) return fail(TQ_ERR_ALIGN, "ids misaligned");
  rc = check_io(x, x_dtype, y, y_dtype, n > 0 && a.N > 0);
  if (rc != TQ_OK) return rc;
  return hip_status(launch_qmv(a, ids, n, x, x_dtype, rotated, y, y_dtype,
                               static_cast<hipStream_t>(stream), &b),
                    "tq_gather_qmv_pair");
}

int tq_multi_gather_qmv(const tq_qweight* w, const int32_t* ids, int64_t P, const void* x,
                        tq_dtype x_dtype, void* y, tq_dtype y_dtype, uint32_t flags, void* ws,
                        size_t ws_bytes, void* stream) {
  WeightArgs a{};
  int rc = check_weight(w, &a, false, (flags & TQ_X_ROTATED) != 0);
  if (rc != TQ_OK) return rc;
  if (P < 0 || P > (1 << 30)) return fail(TQ_ERR_ARG, "P out of range");
  if (P > 0 && !ids) return fail(TQ_ERR_ARG, "ids is NULL");
  if (P > 0 && !aligned(ids, 4)) return fail(TQ_ERR_ALIGN, "ids misaligned");
  rc = check_io(x, x_dtype, y, y_dtype, P > 0 && a.N > 0);
  if (rc != TQ_OK) return rc;
  if (P == 0 || a.N == 0) return TQ_OK;
  const size_t need = multi_gather_workspace(a, P);
  if (!ws || ws_bytes < need)
    return fail(TQ_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (!aligned(ws, 16)) return fail(TQ_ERR_ALIGN, "workspace must be 16-byte aligned");
  return hip_status(launch_multi_gather(a, ids, P, x, x_dtype, (flags & TQ_X_ROTATED) != 0, y,
                                        y_dtype, ws, static_cast<hipStream_t>(stream)),
                    "tq_multi_gather_qmv");
}

int tq_multi_gather_qmv_pair(const tq_qweight* w1, const tq_qweight* w2, const int32_t* ids,
                             int64_t P, const void* x, tq_dtype x_dtype, void* y,
                             tq_dtype y_dtype, uint32_t flags, void* ws, size_t ws_bytes,
                             void* stream) {
  const bool rotated = (flags & TQ_X_ROTATED) != 0;
  WeightArgs a{}, b{};
  int rc = check_weight(w1, &a, false, rotated);
  if (rc != TQ_OK) return rc;
  rc = check_weight(w2, &b, false, rotated);
  if (rc != TQ_OK) return rc;
  if (a.levels != b.levels || a.group != b.group || a.K != b.K || a.N != b.N || a.E != b.E)
    return fail(TQ_ERR_ARG, "tq_multi_gather_qmv_pair: the two weights differ in format or shape");
  if (!rotated && w1->signs != w2->signs)
    return fail(TQ_ERR_ARG, "tq_multi_gather_qmv_pair: the two weights must share one signs array");
  if (P < 0 || P > (1 << 29)) return fail(TQ_ERR_ARG, "P out of range");
  if (P > 0 && !ids) return fail(TQ_ERR_ARG, "ids is NULL");
  if (P > 0 && !aligned(ids, 4)) return fail(TQ_ERR_ALIGN, "ids misaligned");
  rc = check_io(x, x_dtype, y, y_dtype, P > 0 && a.N > 0);
  if (rc != TQ_OK) return rc;
  if (P == 0 || a.N == 0) return TQ_OK;
  const size_t need = multi_gather_workspace(a, P);
  if (!ws || ws_bytes < need)
    return fail(TQ_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (!aligned(ws, 16)) return fail(TQ_ERR_ALIGN, "workspace must be 16-byte aligned");
  return hip_status(launch_multi_gather(a, ids, P, x, x_dtype, rotated, y, y_dtype, ws,
                                        static_cast<hipStream_t>(stream), &b),
                    "tq_multi_gather_qmv_pair");
}

int tq_multi_gather_qmv_static(const tq_qweight* w, const int32_t* ids, int64_t P,
                               const void* x, tq_dtype x_dtype, void* y, tq_dtype y_dtype,
                               uint32_t flags, void* stream) {
  WeightArgs a{};
  int rc = check_weight(w, &a, false, (flags & TQ_X_ROTATED) != 0);
  if (rc != TQ_OK) return rc;
  if (P < 0 || P > (1 << 30)) return fail(TQ_ERR_ARG, "P out of range");
  if (P > 0 && !ids) return fail(TQ_ERR_ARG, "ids is NULL");
  if (P > 0 && !aligned(ids, 4)) return fail(TQ_ERR_ALIGN, "ids misaligned");
  rc = check_io(x, x_dtype, y, y_dtype, P > 0 && a.N > 0);
  if (rc != TQ_OK) return rc;
  if (P == 0 || a.N == 0) return TQ_OK;
  const size_t need = multi_gather_workspace(a, P);
  if (need > kStaticScratchBytes)
    return fail(TQ_ERR_WORKSPACE,
                "tq_multi_gather_qmv_static: %lld pairs of K=%d need %zu bytes of workspace, "
                "above the fixed %zu (use tq_multi_gather_qmv with a workspace)",
                static_cast<long long>(P), a.K, need, kStaticScratchBytes);
  void* ws = nullptr;
  rc = hip_status(static_scratch(&ws), "tq_multi_gather_qmv_static");
  if (rc != TQ_OK) return rc;
  return hip_status(launch_multi_gather(a, ids, P, x, x_dtype, (flags & TQ_X_ROTATED) != 0, y,
                                        y_dtype, ws, static_cast<hipStream_t>(stream)),
                    "tq_multi_gather_qmv_static");
}

int tq_rotate_dense(const void* x, tq_dtype x_dtype, int64_t rows, int64_t K, const float* R,
                    void* out, tq_dtype out_dtype, void* stream) {
  if (K < 64 || K > 8192 || K % 32 != 0)
    return fail(TQ_ERR_UNSUPPORTED, "K must be a multiple of 32 in [64, 8192] (got %lld)",
                static_cast<long long>(K));
  if (rows < 0) return fail(TQ_ERR_ARG, "rows must be >= 0");
  if (!valid_dtype(x_dtype) || !valid_dtype(out_dtype)) return fail(TQ_ERR_ARG, "bad dtype");
  if (rows == 0) return TQ_OK;
  if (!x || !R || !out) return fail(TQ_ERR_ARG, "x, R and out must be non-NULL");
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(R, 4) || !aligned(out, dtype_size(out_dtype)))
    return fail(TQ_ERR_ALIGN, "x, R or out misaligned");
  if ((rows + 63) / 64 > 65535) return fail(TQ_ERR_ARG, "rows must be below 64 * 65536");
  return hip_status(launch_dense_rot(x, x_dtype, rows, static_cast<int>(K), R, out, out_dtype,
                                     static_cast<hipStream_t>(stream)),
                    "tq_rotate_dense");
}

int tq_encode_dense(const void* W, tq_dtype w_dtype, int64_t rows, int64_t K, const float* R,
                    int32_t n_levels, int32_t group, uint32_t* codes, uint16_t* scales,
                    void* ws, size_t ws_bytes, void* stream) {
  int m = 1, P = 1;
  const int rc = check_shape(K, n_levels, group, &m, &P, false, /*any_k=*/true);
  if (rc != TQ_OK) return rc;
  if (!valid_dtype(w_dtype)) return fail(TQ_ERR_ARG, "bad weight dtype");
  if (rows < 0) return fail(TQ_ERR_ARG, "rows must be >= 0");
  if (rows == 0) return TQ_OK;
  if (!W || !R || !codes || !scales) return fail(TQ_ERR_ARG, "W, R, codes and scales must be non-NULL");
  if (!aligned(W, dtype_size(w_dtype)) || !aligned(R, 4) || !aligned(codes, 4) ||
      !aligned(scales, 2))
    return fail(TQ_ERR_ALIGN, "W, R, codes or scales misaligned");
  const size_t row_bytes = static_cast<size_t>(K) * 8;
  if (!ws || ws_bytes < row_bytes)
    return fail(TQ_ERR_WORKSPACE, "workspace of at least %zu bytes (one fp64 row) needed", row_bytes);
  if (!aligned(ws, 8)) return fail(TQ_ERR_ALIGN, "workspace must be 8-byte aligned");
  int64_t chunk = static_cast<int64_t>(ws_bytes / row_bytes);
  if (chunk > 64 * 65535) chunk = 64 * 65535;
  const int64_t wpr = words_per_row(K, n_levels), ngk = K / group;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const char* src = static_cast<const char*>(W);
  hipError_t e = hipSuccess;
  for (int64_t r0 = 0; r0 < rows && e == hipSuccess; r0 += chunk) {
    const int64_t n = rows - r0 < chunk ? rows - r0 : chunk;
    e = launch_dense_rot(src + static_cast<size_t>(r0) * K * dtype_size(w_dtype), w_dtype, n,
                         static_cast<int>(K), R, ws, 3, st);
    if (e == hipSuccess)
      e = launch_encode_rotated(static_cast<const double*>(ws), n, static_cast<int>(K), n_levels,
                                group, codes + r0 * wpr, scales + r0 * ngk, st);
  }
  return hip_status(e, "tq_encode_dense");
}

int tq_kv_fetch(const tq_qweight* w, void* out, tq_dtype out_dtype, void* stream) {
  WeightArgs a{};
  int rc = check_weight(w, &a, /*allow256=*/true);
  if (rc != TQ_OK) return rc;
  if (!kv_fetch_supported(a.K, a.levels))
    return fail(TQ_ERR_UNSUPPORTED,
                "tq_kv_fetch needs a bit format (4, 8, 16 or 256 levels) and K a power of two "
                "in [64, 2048] (got %d levels, K=%d)", a.levels, a.K);
  if (!valid_dtype(out_dtype)) return fail(TQ_ERR_ARG, "bad dtype");
  const int64_t rows = static_cast<int64_t>(a.E) * a.N;
  if (rows == 0) return TQ_OK;
  if (!out) return fail(TQ_ERR_ARG, "out is NULL");
  if (!aligned(out, 16)) return fail(TQ_ERR_ALIGN, "out must be 16-byte aligned");
  return hip_status(launch_kv_fetch(a, rows, out, out_dtype, static_cast<hipStream_t>(stream)),
                    "tq_kv_fetch");
}

int tq_dequant(const tq_qweight* w, const int32_t* ids, int64_t n, void* out,
               tq_dtype out_dtype, void* stream) {
  WeightArgs a{};
  int rc = check_weight(w, &a, false, /*rotated=*/true);
  if (rc != TQ_OK) return rc;
  if (!valid_dtype(out_dtype)) return fail(TQ_ERR_ARG, "bad dtype");
  if (n < 0 || n > 65535) return fail(TQ_ERR_ARG, "n must be in [0, 65535]");
  if (!ids && n > a.E) return fail(TQ_ERR_ARG, "without ids n must be at most E");
  if (n == 0 || a.N == 0) return TQ_OK;
  if (ids && !aligned(ids, 4)) return fail(TQ_ERR_ALIGN, "ids misaligned");
  if (!out) return fail(TQ_ERR_ARG, "out is NULL");
  if (!aligned(out, 16)) return fail(TQ_ERR_ALIGN, "out must be 16-byte aligned");
  return hip_status(launch_dequant(a, ids, static_cast<int>(n), out, out_dtype,
                                   static_cast<hipStream_t>(stream)),
                    "tq_dequant");
}

int tq_gather_qmm(const tq_qweight* w, const void* x, tq_dtype x_dtype, int64_t T,
                  const int32_t* row_token, const int32_t* expert_offsets, int64_t M, void* y,
                  tq_dtype y_dtype, uint32_t flags, void* ws, size_t ws_bytes, void* stream) {
  WeightArgs a{};
  int rc = check_weight(w, &a, false, (flags & TQ_X_ROTATED) != 0);
  if (rc != TQ_OK) return rc;
  if (T < 0 || M < 0 || M > (1ll << 31) - 1 || T > (1ll << 31) - 1)
    return fail(TQ_ERR_ARG, "T and M must be in [0, 2^31)");
  rc = check_io(x, x_dtype, y, y_dtype, M > 0 && a.N > 0);
  if (rc != TQ_OK) return rc;
  if (M == 0 || a.N == 0) return TQ_OK;
  if (T == 0) return fail(TQ_ERR_ARG, "T must be > 0 when M > 0");
  if (!row_token || !expert_offsets) return fail(TQ_ERR_ARG, "row_token and expert_offsets needed");
  if (!aligned(row_token, 4) || !aligned(expert_offsets, 4))
    return fail(TQ_ERR_ALIGN, "row_token/expert_offsets misaligned");
  const bool rotated = (flags & TQ_X_ROTATED) != 0;
  if (rotated && x_dtype == TQ_BF16 && !aligned(x, 16))
    return fail(TQ_ERR_ALIGN, "rotated bf16 x must be 16-byte aligned");
  const size_t need = gather_qmm_workspace(a, M, T);
  if (!ws || ws_bytes < need)
    return fail(TQ_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (!aligned(ws, 256)) return fail(TQ_ERR_ALIGN, "workspace must be 256-byte aligned");
  return hip_status(launch_gather_qmm(a, x, x_dtype, T, row_token, expert_offsets, M, rotated, y,
                                      y_dtype, ws, static_cast<hipStream_t>(stream)),
                    "tq_gather_qmm");
}

int tq_gather_qmm_pair(const tq_qweight* w1, const tq_qweight* w2, const void* x,
                       tq_dtype x_dtype, int64_t T, const int32_t* row_token,
                       const int32_t* expert_offsets, int64_t M, void* y, tq_dtype y_dtype,
                       uint32_t flags, void* ws, size_t ws_bytes, void* stream) {
  const bool rotated = (flags & TQ_X_ROTATED) != 0;
  WeightArgs a{}, b{};
  int rc = check_weight(w1, &a, false, rotated);
  if (rc != TQ_OK) return rc;
  rc = check_weight(w2, &b, false, rotated);
  if (rc != TQ_OK) return rc;
  if (a.levels != b.levels || a.group != b.group || a.K != b.K || a.N != b.N || a.E != b.E)
    return fail(TQ_ERR_ARG, "tq_gather_qmm_pair: the two weights differ in format or shape");
  if (!rotated && w1->signs != w2->signs)
    return fail(TQ_ERR_ARG, "tq_gather_qmm_pair: the two weights must share one signs array");
  if (T < 0 || M < 0 || M > (1ll << 30) - 1 || T > (1ll << 31) - 1)
    return fail(TQ_ERR_ARG, "T must be in [0, 2^31) and M in [0, 2^30)");
  rc = check_io(x, x_dtype, y, y_dtype, M > 0 && a.N > 0);
  if (rc != TQ_OK) return rc;
  if (M == 0 || a.N == 0) return TQ_OK;
  if (T == 0) return fail(TQ_ERR_ARG, "T must be > 0 when M > 0");
  if (!row_token || !expert_offsets) return fail(TQ_ERR_ARG, "row_token and expert_offsets needed");
  if (!aligned(row_token, 4) || !aligned(expert_offsets, 4))
    return fail(TQ_ERR_ALIGN, "row_token/expert_offsets misaligned");
  if (rotated && x_dtype == TQ_BF16 && !aligned(x, 16))
    return fail(TQ_ERR_ALIGN, "rotated bf16 x must be 16-byte aligned");
  const size_t need = gather_qmm_workspace(a, M, T);
  if (!ws || ws_bytes < need)
    return fail(TQ_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (!aligned(ws, 256)) return fail(TQ_ERR_ALIGN, "workspace must be 256-byte aligned");
  return hip_status(launch_gather_qmm(a, x, x_dtype, T, row_token, expert_offsets, M, rotated, y,
                                      y_dtype, ws, static_cast<hipStream_t>(stream), &b),
                    "tq_gather_qmm_pair");
}

int tq_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double stretch,
                        double original, double* inv_freq, double* gain) {
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0)
    return fail(TQ_ERR_ARG, "rot_dim must be even and in [2, 1024] (got %d)", rot_dim);
  if (!(base > 0.0) || !std::isfinite(base)) return fail(TQ_ERR_ARG, "base must be positive");
  if (!(stretch >= 1.0) || !std::isfinite(stretch)) return fail(TQ_ERR_ARG, "stretch must be at least 1");
  if (scaling < TQ_ROPE_NONE || scaling > TQ_ROPE_YARN)
    return fail(TQ_ERR_UNSUPPORTED, "unknown rope scaling %d", scaling);
  if (scaling == TQ_ROPE_YARN && (!(original > 0.0) || !std::isfinite(original)))
    return fail(TQ_ERR_ARG, "original must be positive");
  if (scaling == TQ_ROPE_NTK && rot_dim == 2)
    return fail(TQ_ERR_UNSUPPORTED, "NTK scaling needs rot_dim above 2");
  if (!inv_freq || !gain) return fail(TQ_ERR_ARG, "inv_freq and gain must be non-NULL");
  const double d = rot_dim;
  const double b = scaling == TQ_ROPE_NTK ? base * std::pow(stretch, d / (d - 2.0)) : base;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / d);
    if (scaling == TQ_ROPE_LINEAR) f /= stretch;
    if (scaling == TQ_ROPE_YARN) {
      const double turns = original * f / (2.0 * M_PI);
      const double g = std::fmin(std::fmax((turns - 1.0) / 31.0, 0.0), 1.0);
      f *= g + (1.0 - g) / stretch;
    }
    inv_freq[i] = f;
  }
  *gain = scaling == TQ_ROPE_YARN ? 0.1 * std::log(stretch) + 1.0 : 1.0;
  return TQ_OK;
}

namespace {
// tq_rope and tq_rope_axes (r holds the axes of the latter already)
int rope_call(const char* name, const void* x, tq_dtype dtype, int64_t tokens, int32_t heads, int32_t head_dim,
              int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions, RopeArgs r,
              const tq_rope_params* rope, uint32_t flags, void* out, int64_t out_token_stride,
              int64_t out_head_stride, void* stream) {
  if (!valid_dtype(dtype)) return fail(TQ_ERR_ARG, "bad dtype");
  if (head_dim < 2 || head_dim > 1024 || head_dim % 2 != 0)
    return fail(TQ_ERR_UNSUPPORTED, "head_dim must be even and in [2, 1024] (got %d)", head_dim);
  if (tokens < 0 || tokens > (1 << 30) || heads < 0 || heads > 65536)
    return fail(TQ_ERR_ARG, "tokens must be in [0, 2^30] and heads in [0, 65536]");
  if (flags & ~static_cast<uint32_t>(TQ_ROPE_TRANSPOSED)) return fail(TQ_ERR_ARG, "unknown flags");
  if (tokens == 0 || heads == 0) return TQ_OK;
  if (!x || !out) return fail(TQ_ERR_ARG, "x and out must be non-NULL");
  if (!aligned(x, dtype_size(dtype)) || !aligned(out, dtype_size(dtype)))
    return fail(TQ_ERR_ALIGN, "x or out misaligned for its dtype");
  if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
    return fail(TQ_ERR_ARG, "in place, x and out must have the same strides");
  if ((tokens > 1 && out_token_stride == 0) || (heads > 1 && out_head_stride == 0))
    return fail(TQ_ERR_ARG, "out must not overlap itself");
  const int rc = check_rope(rope, positions, head_dim, &r);
  if (rc != TQ_OK) return rc;
  return hip_status(launch_rope(x, dtype, tokens, heads, head_dim, x_token_stride, x_head_stride, r,
                                (flags & TQ_ROPE_TRANSPOSED) != 0, out, out_token_stride,
                                out_head_stride, static_cast<hipStream_t>(stream)),
                    name);
}

// tq_kv_store and tq_kv_store_axes
int store_call(const char* name, const tq_kv_cache* cache, const void* k, const void* v, tq_dtype dtype,
               int64_t tokens, const int64_t (&strides)[4], const int64_t* slots, RopeArgs r,
               const tq_rope_params* rope, const int32_t* positions, void* stream) {
  KvCacheArgs c{};
  int rc = check_cache(cache, &c);
  if (rc != TQ_OK) return rc;
  if (!valid_dtype(dtype)) return fail(TQ_ERR_ARG, "bad dtype");
  if (tokens < 0 || tokens > (1 << 30)) return fail(TQ_ERR_ARG, "tokens must be in [0, 2^30]");
  if (tokens == 0) return TQ_OK;
  if (!k || !v || !slots) return fail(TQ_ERR_ARG, "k, v and slots must be non-NULL");
  if (!aligned(k, dtype_size(dtype)) || !aligned(v, dtype_size(dtype)) || !aligned(slots, 8))
    return fail(TQ_ERR_ALIGN, "k, v or slots misaligned");
  if (rope) {
    rc = check_rope(rope, positions, c.D, &r);
    if (rc != TQ_OK) return rc;
  }
  return hip_status(launch_kv_store(c, k, v, dtype, tokens, strides, slots, r,
                                    static_cast<hipStream_t>(stream)),
                    name);
}
}  // namespace

int tq_rope(const void* x, tq_dtype dtype, int64_t tokens, int32_t heads, int32_t head_dim,
            int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
            const tq_rope_params* rope, uint32_t flags, void* out, int64_t out_token_stride,
            int64_t out_head_stride, void* stream) {
  return rope_call("tq_rope", x, dtype, tokens, heads, head_dim, x_token_stride, x_head_stride, positions,
                   RopeArgs{}, rope, flags, out, out_token_stride, out_head_stride, stream);
}

int tq_rope_axes(const void* x, tq_dtype dtype, int64_t tokens, int32_t heads, int32_t head_dim,
                 int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
                 int64_t axis_stride, int32_t axes, const uint8_t* axis, const tq_rope_params* rope,
                 uint32_t flags, void* out, int64_t out_token_stride, int64_t out_head_stride,
                 void* stream) {
  RopeArgs r{};
  const int rc = check_axes(axis, axis_stride, axes, &r);
  if (rc != TQ_OK) return rc;
  return rope_call("tq_rope_axes", x, dtype, tokens, heads, head_dim, x_token_stride, x_head_stride,
                   positions, r, rope, flags, out, out_token_stride, out_head_stride, stream);
}

int tq_kv_store(const tq_kv_cache* cache, const void* k, const void* v, tq_dtype dtype,
                int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                const tq_rope_params* rope, const int32_t* positions, void* stream) {
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  return store_call("tq_kv_store", cache, k, v, dtype, tokens, strides, slots, RopeArgs{}, rope, positions,
                    stream);
}

int tq_kv_store_axes(const tq_kv_cache* cache, const void* k, const void* v, tq_dtype dtype,
                     int64_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                     int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                     const tq_rope_params* rope, const int32_t* positions, int64_t axis_stride,
                     int32_t axes, const uint8_t* axis, void* stream) {
  RopeArgs r{};
  const int rc = check_axes(axis, axis_stride, axes, &r);
  if (rc != TQ_OK) return rc;
  if (!rope) return fail(TQ_ERR_ARG, "rope is NULL");
  const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  return store_call("tq_kv_store_axes", cache, k, v, dtype, tokens, strides, slots, r, rope, positions,
                    stream);
}

int tq_kv_load(const tq_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k_out,
               void* v_out, tq_dtype dtype, void* stream) {
  KvCacheArgs c{};
  const int rc = check_cache(cache, &c);
  if (rc != TQ_OK) return rc;
  if (!valid_dtype(dtype)) return fail(TQ_ERR_ARG, "bad dtype");
  if (tokens < 0 || tokens > (1 << 30)) return fail(TQ_ERR_ARG, "tokens must be in [0, 2^30]");
  if (tokens == 0 || (!k_out && !v_out)) return TQ_OK;
  if (!slots) return fail(TQ_ERR_ARG, "slots is NULL");
  if (!aligned(slots, 8)) return fail(TQ_ERR_ALIGN, "slots misaligned");
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(TQ_ERR_ALIGN, "k_out and v_out must be 16-byte aligned");
  return hip_status(launch_kv_load(c, slots, tokens, k_out, v_out, dtype,
                                   static_cast<hipStream_t>(stream)),
                    "tq_kv_load");
}

namespace {
int check_attend_shape(const KvCacheArgs& c, int32_t q_heads, int32_t B, int64_t M) {
  if (q_heads < 1 || q_heads > 65536 || q_heads % c.heads != 0)
    return fail(TQ_ERR_ARG, "q_heads must be a multiple of the cache's %d heads, at most 65536 (got %d)",
                c.heads, q_heads);
  if (B < 0 || B > 65536) return fail(TQ_ERR_ARG, "B must be in [0, 65536]");
  if (M < 0 || M > (1 << 24)) return fail(TQ_ERR_ARG, "M must be in [0, 2^24]");
  return TQ_OK;
}
}  // namespace

size_t tq_kv_attend_workspace(const tq_kv_cache* cache, int32_t q_heads, int32_t B, int64_t M) {
  KvCacheArgs c{};
  if (check_cache(cache, &c) != TQ_OK || check_attend_shape(c, q_heads, B, M) != TQ_OK)
    return SIZE_MAX;
  return kv_attend_workspace(c, q_heads, B, M);
}

int tq_kv_attend(const tq_kv_cache* cache, const void* q, tq_dtype q_dtype, int32_t q_heads,
                 int64_t q_token_stride, int32_t B, const int32_t* q_offsets, int64_t M,
                 const int32_t* kv_lens, const int32_t* page_table, int32_t table_width,
                 const uint32_t* tree, int32_t tree_words, float scale, void* out,
                 tq_dtype out_dtype, void* ws, size_t ws_bytes, void* stream) {
  AttendArgs a{};
  int rc = check_cache(cache, &a.c);
  if (rc != TQ_OK) return rc;
  rc = check_attend_shape(a.c, q_heads, B, M);
  if (rc != TQ_OK) return rc;
  if ((q_dtype != TQ_BF16 && q_dtype != TQ_F16) || (out_dtype != TQ_BF16 && out_dtype != TQ_F16))
    return fail(TQ_ERR_UNSUPPORTED, "tq_kv_attend takes bf16 or fp16 queries and outputs");
  if (table_width < 0) return fail(TQ_ERR_ARG, "table_width must be >= 0");
  if (tree ? tree_words < 1 || tree_words > 65536 : tree_words != 0)
    return fail(TQ_ERR_ARG, "tree_words must be in [1, 65536] with a tree and 0 without");
  if (static_cast<int64_t>(table_width) * a.c.page > 0x7fffffffll - 65536)
    return fail(TQ_ERR_ARG, "table_width * page_tokens must be below 2^31 - 65536");
  // what the schedule counts: units in 32 bits, tokens read by all of them below 2^53
  const int64_t heads_of_rows = (M + B) * q_heads, tokens = static_cast<int64_t>(table_width) * a.c.page + 256;
  if (heads_of_rows > 0x7fffffffll || heads_of_rows > (1ll << 53) / tokens)
    return fail(TQ_ERR_ARG, "(M + B) * q_heads must be below 2^31, and 2^53 with the table's tokens");
  if (!q_offsets && (B == 0 ? M > 0 : M % B != 0))
    return fail(TQ_ERR_ARG, "without q_offsets B must divide M");
  if (B == 0 || M == 0) return TQ_OK;
  if (!q || !out || !kv_lens || (table_width > 0 && !page_table))
    return fail(TQ_ERR_ARG, "q, out, kv_lens and page_table must be non-NULL");
  if (!std::isfinite(scale)) return fail(TQ_ERR_ARG, "scale must be finite");
  if (!aligned(q, 16) || q_token_stride % 8 != 0 || !aligned(out, 16))
    return fail(TQ_ERR_ALIGN, "q and its rows, and out, must be 16-byte aligned");
  if (!aligned(kv_lens, 4) || (page_table && !aligned(page_table, 4)) ||
      (q_offsets && !aligned(q_offsets, 4)) || (tree && !aligned(tree, 4)))
    return fail(TQ_ERR_ALIGN, "kv_lens, page_table, q_offsets or tree misaligned");
  const size_t need = kv_attend_workspace(a.c, q_heads, B, M);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(TQ_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (need > 0 && !aligned(ws, 256)) return fail(TQ_ERR_ALIGN, "workspace must be 256-byte aligned");
  a.q = q; a.qdt = q_dtype; a.q_heads = q_heads; a.q_stride = q_token_stride; a.B = B;
  a.q_offsets = q_offsets; a.M = M; a.kv_lens = kv_lens; a.page_table = page_table;
  a.table_width = table_width; a.tree = tree; a.tree_words = tree_words; a.scale = scale;
  a.out = out; a.odt = out_dtype; a.ws = ws;
  return hip_status(launch_kv_attend(a, static_cast<hipStream_t>(stream)), "tq_kv_attend");
}

namespace {
int check_pool(const tq_kv_pool* pool, int32_t page_tokens, int32_t B, int32_t table_width) {
  if (!pool) return fail(TQ_ERR_ARG, "pool is NULL");
  if (pool->pages < 1 || pool->pages > (1 << 30)) return fail(TQ_ERR_ARG, "pool pages must be in [1, 2^30]");
  if (!pool->free_pages || !pool->state) return fail(TQ_ERR_ARG, "the pool's free_pages and state must be non-NULL");
  if (!aligned(pool->free_pages, 4) || !aligned(pool->state, 4))
    return fail(TQ_ERR_ALIGN, "the pool's free_pages or state misaligned");
  if (page_tokens < 1 || page_tokens > 65536) return fail(TQ_ERR_ARG, "page_tokens must be in [1, 65536]");
  if (B < 0 || B > 65536) return fail(TQ_ERR_ARG, "B must be in [0, 65536]");
  if (table_width < 0 || static_cast<int64_t>(table_width) * page_tokens > 0x7fffffffll - 65536)
    return fail(TQ_ERR_ARG, "table_width must be >= 0, table_width * page_tokens below 2^31 - 65536");
  return TQ_OK;
}

// Memory of a call: `rows` pieces of `bytes`, `stride` bytes apart.
struct Piece {
  const char* name;
  const void* at;
  int64_t bytes, rows = 1, stride = 0;
};
// Whether [lo, hi) shares a byte with p. Addresses are compared as numbers.
bool meets(int64_t lo, int64_t hi, const Piece& p) {
  const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p.at));
  if (!p.at || p.bytes <= 0 || p.rows <= 0 || lo >= hi) return false;
  if (p.rows > 1 && p.stride >= p.bytes) {  // the last row that begins before hi
    if (at >= hi) return false;
    const int64_t r = (hi - 1 - at) / p.stride, last = r < p.rows ? r : p.rows - 1;
    return lo < at + last * p.stride + p.bytes;
  }
  const int64_t all = (p.rows - 1) * p.stride;
  return lo < at + (all > 0 ? all : 0) + p.bytes && hi > at + (all < 0 ? all : 0);
}
// Refuses outputs (one piece each) that meet an input or each other.
int check_apart(std::initializer_list<Piece> outputs, std::initializer_list<Piece> inputs) {
  for (const Piece* o = outputs.begin(); o != outputs.end(); ++o) {
    const int64_t lo = static_cast<int64_t>(reinterpret_cast<uintptr_t>(o->at)), hi = lo + o->bytes;
    if (!o->at || o->bytes <= 0) continue;
    for (const Piece& i : inputs)
      if (meets(lo, hi, i)) return fail(TQ_ERR_ARG, "%s and %s overlap", o->name, i.name);
    for (const Piece* p = o + 1; p != outputs.end(); ++p)
      if (meets(lo, hi, *p)) return fail(TQ_ERR_ARG, "%s and %s overlap", o->name, p->name);
  }
  return TQ_OK;
}

bool all_aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p && !aligned(p, 4)) return false;
  return true;
}
}  // namespace

int tq_kv_plan(const tq_kv_pool* pool, int32_t page_tokens, int32_t B, const int32_t* lens,
               const int32_t* counts, int32_t* page_table, int32_t table_width, int64_t M,
               const int32_t* parents, const int32_t* shift, int64_t* slots, int32_t* positions,
               int32_t* q_offsets, int32_t* kv_lens, int32_t* status, uint32_t* tree,
               int32_t tree_words, int32_t* left, void* stream) {
  int rc = check_pool(pool, page_tokens, B, table_width);
  if (rc != TQ_OK) return rc;
  if (M < 0 || M > (1 << 24)) return fail(TQ_ERR_ARG, "M must be in [0, 2^24]");
  if (tree ? tree_words < 1 || tree_words > 65536 : tree_words != 0)
    return fail(TQ_ERR_ARG, "tree_words must be in [1, 65536] with a tree and 0 without");
  if (!q_offsets || (B > 0 && (!lens || !counts || !kv_lens || !status || (table_width > 0 && !page_table))) ||
      (M > 0 && (!slots || !positions)))
    return fail(TQ_ERR_ARG, "lens, counts, page_table and the outputs must be non-NULL");
  if (!aligned(slots, 8) || !all_aligned4({lens, counts, page_table, parents, shift, positions, q_offsets,
                                           kv_lens, status, tree, left}))
    return fail(TQ_ERR_ALIGN, "slots must be 8-byte, the other arrays 4-byte aligned");
  const int64_t per = 4 * static_cast<int64_t>(B), table_bytes = per * table_width;
  rc = check_apart({{"page_table", page_table, table_bytes}, {"slots", slots, 8 * M}, {"positions", positions, 4 * M},
                    {"q_offsets", q_offsets, per + 4}, {"kv_lens", kv_lens, per}, {"status", status, per},
                    {"tree", tree, 4 * M * tree_words}, {"left", left == pool->state ? nullptr : left, 4},
                    {"the pool's state", pool->state, 8}},
                   {{"lens", lens, per}, {"counts", counts, per}, {"parents", parents, 4 * M}, {"shift", shift, per},
                    {"the pool's free_pages", pool->free_pages, 4 * static_cast<int64_t>(pool->pages)}});
  if (rc != TQ_OK) return rc;
  PlanArgs a{};
  a.free_pages = pool->free_pages; a.state = pool->state; a.pages = pool->pages; a.page = page_tokens;
  a.B = B; a.lens = lens; a.counts = counts; a.table = page_table; a.width = table_width;
  a.M = static_cast<int>(M); a.parents = parents; a.words = tree_words; a.shift = shift;
  a.slots = slots; a.positions = positions; a.q_offsets = q_offsets; a.kv_lens = kv_lens;
  a.status = status; a.tree = tree; a.left = left ? left : pool->state;
  return hip_status(launch_kv_plan(a, static_cast<hipStream_t>(stream)), "tq_kv_plan");
}

int tq_kv_keep(const tq_kv_pool* pool, const tq_kv_cache* cache, int32_t page_tokens, int32_t B,
               const int32_t* lens, const int32_t* q_offsets, const int32_t* status,
               const int32_t* kept, const int32_t* path, int64_t M, const int32_t* page_table,
               int32_t table_width, int32_t* lens_out, int32_t* left, void* stream) {
  int rc = check_pool(pool, page_tokens, B, table_width);
  if (rc != TQ_OK) return rc;
  KeepArgs a{};
  if (path) {
    rc = check_cache(cache, &a.c);
    if (rc != TQ_OK) return rc;
    if (a.c.page != page_tokens || a.c.pages != pool->pages)
      return fail(TQ_ERR_ARG, "the cache and the pool differ in pages or page_tokens");
    if (!q_offsets) return fail(TQ_ERR_ARG, "a path needs q_offsets");
    if (M < 0 || M > (1 << 24)) return fail(TQ_ERR_ARG, "M must be in [0, 2^24]");
  }
  if (B == 0 && (!left || left == pool->state)) return TQ_OK;
  if (B > 0 && (!lens || !kept || !lens_out || (table_width > 0 && !page_table)))
    return fail(TQ_ERR_ARG, "lens, kept, page_table and lens_out must be non-NULL");
  if (!all_aligned4({lens, q_offsets, status, kept, path, page_table, lens_out, left}))
    return fail(TQ_ERR_ALIGN, "the arrays must be 4-byte aligned");
  const int64_t per = 4 * static_cast<int64_t>(B), cache_rows = path ? a.c.pages * a.c.heads * a.c.page : 0;
  const auto codes = [&](const KvHalf& h) { return cache_rows * h.wpr * 4; };
  const auto scales = [&](const KvHalf& h) { return cache_rows * (a.c.D / (path ? h.group : 1)) * 2; };
  rc = check_apart({{"lens_out", lens_out, per}, {"left", left == pool->state ? nullptr : left, 4},
                    {"the pool's free_pages", pool->free_pages, 4 * static_cast<int64_t>(pool->pages)},
                    {"the pool's state", pool->state, 8}, {"the cache's key codes", a.c.k.codes, codes(a.c.k)},
                    {"the cache's key scales", a.c.k.scales, scales(a.c.k)},
                    {"the cache's value codes", a.c.v.codes, codes(a.c.v)},
                    {"the cache's value scales", a.c.v.scales, scales(a.c.v)}},
                   {{"lens", lens_out == lens ? nullptr : lens, per}, {"q_offsets", q_offsets, per + 4}, {"status", status, per},
                    {"kept", kept, per}, {"path", path, 4 * M}, {"page_table", page_table, per * table_width}});
  if (rc != TQ_OK) return rc;
  a.free_pages = pool->free_pages; a.state = pool->state; a.pages = pool->pages; a.page = page_tokens;
  a.B = B; a.lens = lens; a.q_offsets = q_offsets; a.status = status; a.kept = kept; a.path = path;
  a.M = path ? static_cast<int>(M) : 0x7fffffff;
  a.table = page_table; a.width = table_width; a.lens_out = lens_out;
  a.left = left ? left : pool->state;
  return hip_status(launch_kv_keep(a, static_cast<hipStream_t>(stream)), "tq_kv_keep");
}

namespace {
int check_verify(int64_t vocab, int32_t B, int64_t M, uint32_t flags) {
  if (vocab < 1 || vocab > (1 << 28)) return fail(TQ_ERR_ARG, "vocab must be in [1, 2^28]");
  if (B < 0 || B > 65536) return fail(TQ_ERR_ARG, "B must be in [0, 65536]");
  if (M < 0 || M > (1 << 24)) return fail(TQ_ERR_ARG, "M must be in [0, 2^24]");
  if (flags & ~static_cast<uint32_t>(TQ_TARGET_PROBS | TQ_DRAFT_PROBS)) return fail(TQ_ERR_ARG, "unknown flags");
  return TQ_OK;
}
}  // namespace

size_t tq_verify_workspace(int64_t vocab, int32_t B, int64_t M, int32_t drafted, uint32_t flags) {
  if (check_verify(vocab, B, M, flags) != TQ_OK) return SIZE_MAX;
  if (drafted != 0 && drafted != 1) {
    fail(TQ_ERR_ARG, "drafted must be 0 or 1");
    return SIZE_MAX;
  }
  return verify_workspace(static_cast<int>(vocab), B, static_cast<int>(M), (flags & TQ_TARGET_PROBS) != 0,
                          drafted != 0, (flags & TQ_DRAFT_PROBS) != 0);
}

int tq_verify(const void* target, tq_dtype target_dtype, int64_t target_stride, const void* draft,
              tq_dtype draft_dtype, int64_t draft_stride, uint32_t flags, int64_t vocab, int32_t B,
              const int32_t* offsets, int64_t M, const int32_t* tokens, const int32_t* parents,
              const float* uniforms, const float* temperature, int32_t* kept, int32_t* out_tokens,
              int32_t* path, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_verify(vocab, B, M, flags);
  if (rc != TQ_OK) return rc;
  if (!valid_dtype(target_dtype) || (draft && !valid_dtype(draft_dtype))) return fail(TQ_ERR_ARG, "bad dtype");
  if (B == 0) return TQ_OK;
  if (!offsets || !kept) return fail(TQ_ERR_ARG, "offsets and kept must be non-NULL");
  if (M > 0 && (!target || !tokens || !uniforms || !out_tokens || !path))
    return fail(TQ_ERR_ARG, "target, tokens, uniforms, out_tokens and path must be non-NULL");
  if (!aligned(target, dtype_size(target_dtype)) || (draft && !aligned(draft, dtype_size(draft_dtype))))
    return fail(TQ_ERR_ALIGN, "target or draft misaligned for its dtype");
  if (!all_aligned4({offsets, tokens, parents, uniforms, temperature, kept, out_tokens, path}))
    return fail(TQ_ERR_ALIGN, "the arrays must be 4-byte aligned");
  VerifyArgs a{};
  a.target = target; a.draft = draft; a.tdt = target_dtype; a.ddt = draft ? draft_dtype : TQ_F32;
  a.tstride = target_stride; a.dstride = draft_stride;
  a.tprobs = (flags & TQ_TARGET_PROBS) != 0; a.dprobs = (flags & TQ_DRAFT_PROBS) != 0;
  a.V = static_cast<int>(vocab); a.B = B; a.M = static_cast<int>(M);
  a.offsets = offsets; a.tokens = tokens; a.parents = parents; a.uniforms = uniforms;
  a.temperature = temperature; a.kept = kept; a.out_tokens = out_tokens; a.path = path; a.ws = ws;
  const size_t need = verify_workspace(a.V, B, a.M, a.tprobs, draft != nullptr, a.dprobs);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(TQ_ERR_WORKSPACE, "workspace of %zu bytes needed (got %zu)", need, ws_bytes);
  if (need > 0 && !aligned(ws, 256)) return fail(TQ_ERR_ALIGN, "workspace must be 256-byte aligned");
  const int64_t per = 4 * static_cast<int64_t>(B), tsize = dtype_size(target_dtype), dsize = draft ? dtype_size(draft_dtype) : 0;
  rc = check_apart({{"kept", kept, per}, {"out_tokens", out_tokens, 4 * M}, {"path", path, 4 * M},
                    {"the workspace", ws, static_cast<int64_t>(need)}},
                   {{"target", target, vocab * tsize, M, target_stride * tsize}, {"draft", draft, vocab * dsize, M, draft_stride * dsize},
                    {"offsets", offsets, per + 4}, {"tokens", tokens, 4 * M}, {"parents", parents, 4 * M},
                    {"uniforms", uniforms, 4 * M}, {"temperature", temperature, per}});
  if (rc != TQ_OK) return rc;
  return hip_status(launch_verify(a, static_cast<hipStream_t>(stream)), "tq_verify");
}

// ---- expert cache ------------------------------------------------------------------------
// Host state (caller-owned memory): a header, then slot_expert[slots] (int32, -1 = empty),
// slot_tick[slots] (uint64, the call that last used the slot), expert_slot[E] (int32, -1 =
// not resident).
namespace {
constexpr uint64_t kCacheMagic = 0x7471657863616368ull;  // "tqexcach"
struct CacheHeader {
  uint64_t magic;
  int64_t E;
  uint64_t tick;
  int64_t hits, misses;
  int32_t slots, pad;
};
size_t align8(size_t n) { return (n + 7) & ~static_cast<size_t>(7); }
size_t cache_bytes(int64_t slots, int64_t E) {
  return sizeof(CacheHeader) + align8(static_cast<size_t>(slots) * 4) +
         static_cast<size_t>(slots) * 8 + align8(static_cast<size_t>(E) * 4);
}
struct CacheView {
  CacheHeader* h;
  int32_t* slot_expert;
  uint64_t* slot_tick;
  int32_t* expert_slot;
};
CacheView cache_view(void* state) {
  CacheView v{};
  v.h = static_cast<CacheHeader*>(state);
  char* p = static_cast<char*>(state) + sizeof(CacheHeader);
  v.slot_expert = reinterpret_cast<int32_t*>(p);
  p += align8(static_cast<size_t>(v.h->slots) * 4);
  v.slot_tick = reinterpret_cast<uint64_t*>(p);
  p += static_cast<size_t>(v.h->slots) * 8;
  v.expert_slot = reinterpret_cast<int32_t*>(p);
  return v;
}
}  // namespace

size_t tq_expert_cache_bytes(int32_t slots, int64_t E) {
  if (slots < 1 || slots > 8192 || E < 1 || E > 8192) return SIZE_MAX;
  return cache_bytes(slots, E);
}

int tq_expert_cache_init(void* state, size_t state_bytes, int32_t slots, int64_t E) {
  if (slots < 1 || slots > 8192 || E < 1 || E > 8192)
    return fail(TQ_ERR_ARG, "slots and E must be in [1, 8192]");
  if (!state) return fail(TQ_ERR_ARG, "state is NULL");
  if (!aligned(state, 8)) return fail(TQ_ERR_ALIGN, "state must be 8-byte aligned");
  if (state_bytes < cache_bytes(slots, E))
    return fail(TQ_ERR_ARG, "state of %zu bytes needed (got %zu)", cache_bytes(slots, E),
                state_bytes);
  CacheHeader* h = static_cast<CacheHeader*>(state);
  std::memset(h, 0, sizeof *h);
  h->magic = kCacheMagic;
  h->E = E;
  h->slots = slots;
  CacheView v = cache_view(state);
  for (int32_t s = 0; s < slots; ++s) {
    v.slot_expert[s] = -1;
    v.slot_tick[s] = 0;
  }
  for (int64_t e = 0; e < E; ++e) v.expert_slot[e] = -1;
  return TQ_OK;
}

int tq_expert_cache_fetch(void* state, const tq_qweight* host, const tq_qweight* pool,
                          const int32_t* ids_host, int32_t n, int32_t* slot_ids_dev,
                          int32_t* slot_ids_host, int32_t* copied, void* stream,
                          void* copy_stream) {
  if (!state || !aligned(state, 8) || static_cast<CacheHeader*>(state)->magic != kCacheMagic)
    return fail(TQ_ERR_ARG, "state was not set up by tq_expert_cache_init");
  CacheView v = cache_view(state);
  WeightArgs hw{}, pw{};
  int rc = check_weight(host, &hw);
  if (rc != TQ_OK) return rc;
  rc = check_weight(pool, &pw);
  if (rc != TQ_OK) return rc;
  if (hw.levels != pw.levels || hw.group != pw.group || hw.K != pw.K || hw.N != pw.N)
    return fail(TQ_ERR_ARG, "host weight and slot pool differ in levels, group, K or N");
  if (hw.E != v.h->E || pw.E != v.h->slots)
    return fail(TQ_ERR_ARG, "host weight must have the cache's E experts and the pool its slots");
  if (n < 0 || n > kMaxSlotIds) return fail(TQ_ERR_ARG, "n must be in [0, %d]", kMaxSlotIds);
  if (n > 0 && (!ids_host || !slot_ids_dev)) return fail(TQ_ERR_ARG, "ids_host and slot_ids_dev needed");
  if (n > 0 && !aligned(slot_ids_dev, 4)) return fail(TQ_ERR_ALIGN, "slot_ids_dev misaligned");
  for (int32_t k = 0; k < n; ++k)
    if (ids_host[k] < 0 || ids_host[k] >= hw.E)
      return fail(TQ_ERR_ARG, "ids_host[%d] = %d is outside [0, %d)", k, ids_host[k], hw.E);
  // distinct experts of this call must fit the pool
  {
    int32_t distinct = 0;
    for (int32_t k = 0; k < n; ++k) {
      bool seen = false;
      for (int32_t j = 0; j < k && !seen; ++j) seen = ids_host[j] == ids_host[k];
      distinct += seen ? 0 : 1;
    }
    if (distinct > pw.E)
      return fail(TQ_ERR_ARG, "%d distinct experts do not fit %d slots", distinct, pw.E);
  }
  // residency: hits first (so that no expert this call needs is evicted), then misses take
  // the least recently used slots that this call does not use
  const uint64_t tick = ++v.h->tick;
  for (int32_t k = 0; k < n; ++k) {
    const int32_t s = v.expert_slot[ids_host[k]];
    if (s >= 0) v.slot_tick[s] = tick;
  }
  int32_t load_e[kMaxSlotIds], load_s[kMaxSlotIds];
  int32_t nload = 0;
  SlotIds out{};
  out.n = n;
  for (int32_t k = 0; k < n; ++k) {
    const int32_t e = ids_host[k];
    int32_t s = v.expert_slot[e];
    if (s < 0) {
      int32_t best = -1;
      for (int32_t c = 0; c < pw.E; ++c) {
        if (v.slot_tick[c] == tick) continue;
        if (best < 0 || v.slot_tick[c] < v.slot_tick[best]) best = c;
      }
      s = best;  // exists: distinct experts <= slots
      if (v.slot_expert[s] >= 0) v.expert_slot[v.slot_expert[s]] = -1;
      v.slot_expert[s] = e;
      v.expert_slot[e] = s;
      v.slot_tick[s] = tick;
      load_e[nload] = e;
      load_s[nload] = s;
      ++nload;
      ++v.h->misses;
    } else {
      ++v.h->hits;
    }
    out.v[k] = s;
    if (slot_ids_host) slot_ids_host[k] = s;
  }
  if (copied) *copied = nload;
  const hipStream_t cs = static_cast<hipStream_t>(stream);
  const hipStream_t xs = copy_stream ? static_cast<hipStream_t>(copy_stream) : cs;
  hipError_t e = hipSuccess;
  if (nload > 0) {
    const size_t cb = static_cast<size_t>(hw.N) * hw.wpr * 4;
    const size_t sb = static_cast<size_t>(hw.N) * (hw.K / hw.group) * 2;
    hipEvent_t entry = nullptr, done = nullptr;
    // a slot being refilled may still be read by work already on `stream`
    if (xs != cs) {
      e = hipEventCreateWithFlags(&entry, hipEventDisableTiming);
      if (e == hipSuccess) e = hipEventRecord(entry, cs);
      if (e == hipSuccess) e = hipStreamWaitEvent(xs, entry, 0);
    }
    for (int32_t i = 0; i < nload && e == hipSuccess; ++i) {
      const char* hc = reinterpret_cast<const char*>(hw.codes) + cb * load_e[i];
      const char* hs = reinterpret_cast<const char*>(hw.scales) + sb * load_e[i];
      char* dc = reinterpret_cast<char*>(const_cast<uint32_t*>(pw.codes)) + cb * load_s[i];
      char* ds = reinterpret_cast<char*>(const_cast<uint16_t*>(pw.scales)) + sb * load_s[i];
      e = hipMemcpyAsync(dc, hc, cb, hipMemcpyHostToDevice, xs);
      if (e == hipSuccess) e = hipMemcpyAsync(ds, hs, sb, hipMemcpyHostToDevice, xs);
    }
    if (xs != cs && e == hipSuccess) {
      e = hipEventCreateWithFlags(&done, hipEventDisableTiming);
      if (e == hipSuccess) e = hipEventRecord(done, xs);
      if (e == hipSuccess) e = hipStreamWaitEvent(cs, done, 0);
    }
    if (entry) (void)hipEventDestroy(entry);
    if (done) (void)hipEventDestroy(done);
  }
  if (e == hipSuccess) e = launch_put_ids(out, slot_ids_dev, cs);
  return hip_status(e, "tq_expert_cache_fetch");
}

int tq_expert_cache_stats(const void* state, int64_t* hits, int64_t* misses) {
  if (!state || !aligned(state, 8) || static_cast<const CacheHeader*>(state)->magic != kCacheMagic)
    return fail(TQ_ERR_ARG, "state was not set up by tq_expert_cache_init");
  const CacheHeader* h = static_cast<const CacheHeader*>(state);
  if (hits) *hits = h->hits;
  if (misses) *misses = h->misses;
  return TQ_OK;
}

const char* tq_last_error(void) { return g_err.c_str(); }

}  // extern "C"
