// Declarations shared by the host entry points (tq_api.cpp) and the kernel launchers
// (*.hip). Nothing here is part of the public interface in include/tq.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tq {

// A codebook as the kernels see it: centroids and thresholds in binary32, centroids also
// as fp16 bit patterns (for the packed-fp16 decode tables). Passed by value.
struct CodebookArgs {
  float c[16];
  float t[15];
  uint16_t h[16];
  int levels;
};

// Lloyd-Max codebook for `levels` in {3, 4, 8, 16}; nullptr otherwise.
const CodebookArgs* codebook_for(int levels);

// The 256-level codebook (8-bit codes of KV-cache rows), binary32 and fp16.
struct BigCodebook {
  float c[256];
  float t[255];
  uint16_t h[256];
};
const BigCodebook* codebook256();

// K = m * P with m in {1, 12, 20, 28}, P a power of two.
bool split_dim(int64_t K, int* m, int* P);

// Everything a qmv-family launch needs about the weight, resolved on the host.
struct WeightArgs {
  const uint32_t* codes;
  const uint16_t* scales;
  const uint32_t* signs;
  int levels, group, K, N, E, wpr, m, P;
};

hipError_t launch_signs(uint64_t seed, int K, uint32_t* bits, hipStream_t s);

// out[r] = R x[r]; `signbits` (device) or, when null, signs computed from `seed`.
hipError_t launch_fwht(const void* x, int xdt, int64_t rows, int K, int m, int P,
                       const uint32_t* signbits, uint64_t seed, void* out, int odt,
                       hipStream_t s);

hipError_t launch_encode(const void* W, int wdt, int64_t rows, int K, int m, int P,
                         int levels, int group, uint64_t seed, uint32_t* codes,
                         uint16_t* scales, hipStream_t s);
// Encode of rows already rotated (fp64): group RMS, fp16 scale, snap, pack.
hipError_t launch_encode_rotated(const double* V, int64_t rows, int K, int levels, int group,
                                 uint32_t* codes, uint16_t* scales, hipStream_t s);
// out = x R^T (dense rotation, fp64 matrix cores); odt 3 = fp64 output.
hipError_t launch_dense_rot(const void* x, int xdt, int64_t rows, int K, const float* R, void* out,
                            int odt, hipStream_t s);

// The register-resident encode for K = 2^p, 64 <= K <= 4096 (W 16-byte aligned).
// rows of m * 2^k (m = 12, 20, 28; 32 <= 2^k <= 256) with the rotation in registers
bool encode_m_supported(int K, int m);
hipError_t launch_encode_m(const void* W, int wdt, int64_t rows, int K, int m, int levels,
                           int group, uint64_t seed, uint32_t* codes, uint16_t* scales,
                           hipStream_t s);
bool encode_p2_supported(int K, int m, int levels);
hipError_t launch_encode_p2(const void* W, int wdt, int64_t rows, int K, int levels, int group,
                            uint64_t seed, uint32_t* codes, uint16_t* scales, hipStream_t s);

// qmv (ids == nullptr, n = 1) and gather_qmv.
// out[k] = decoded weights of expert ids[k] (k when ids is null) in the rotated basis.
hipError_t launch_dequant(const WeightArgs& w, const int32_t* ids, int n, void* out, int odt,
                          hipStream_t s);

// With w2 (same format, shape and experts as w, rotated alike), 2n slots: slot k < n
// reads w at ids[k], slot n + k reads w2 at ids[k]; y holds 2n rows.
hipError_t launch_qmv(const WeightArgs& w, const int32_t* ids, int n, const void* x, int xdt,
                      bool x_rotated, void* y, int ydt, hipStream_t s,
                      const WeightArgs* w2 = nullptr);

// Rotate nrows input rows (input row rows[r], or r when rows is null) into fp16 rows in
// the layout of rot16.hpp, then write zero_rows rows of zeros after them; with a bucket job
// (bucket.hpp), one more workgroup of the same launch sorts the pairs by expert.
struct BucketJob;
hipError_t launch_rot16(const void* x, int xdt, const int32_t* rows, int64_t nrows,
                        int64_t zero_rows, const WeightArgs& w, bool x_rotated, _Float16* out,
                        float* scale, const BucketJob* bucket, hipStream_t s);
size_t multi_gather_workspace(const WeightArgs& w, int64_t P);
// The fixed per-GPU workspace of tq_multi_gather_qmv_static (device address on the current
// device, resolved once per device).
constexpr size_t kStaticScratchBytes = size_t(8) << 20;
hipError_t static_scratch(void** ptr);
// With w2 (same format, shape and experts as w, rotated alike): both weights over the same
// pairs, one rotation and one bucketing; y holds 2P rows (w2's from row P).
hipError_t launch_multi_gather(const WeightArgs& w, const int32_t* ids, int64_t P,
                               const void* x, int xdt, bool x_rotated, void* y, int ydt,
                               void* ws, hipStream_t s, const WeightArgs* w2 = nullptr);

size_t gather_qmm_workspace(const WeightArgs& w, int64_t M, int64_t T);
// With w2 (same format, shape and experts as w, rotated alike): y holds 2M rows, w2's
// from row M; the rows are rotated and the tiles scheduled once.
hipError_t launch_gather_qmm(const WeightArgs& w, const void* x, int xdt, int64_t T,
                             const int32_t* row_token, const int32_t* offsets, int64_t M,
                             bool x_rotated, void* y, int ydt, void* ws, hipStream_t s,
                             const WeightArgs* w2 = nullptr);

// KV-cache fetch: out[r] = R^T (c[idx] * scale) for `rows` rows of a power-of-two K <= 2048.
bool kv_fetch_supported(int K, int levels);
hipError_t launch_kv_fetch(const WeightArgs& w, int64_t rows, void* out, int odt, hipStream_t s);

// A paged KV cache (tq_kv_cache), resolved on the host.
struct KvHalf {
  uint32_t* codes;
  uint16_t* scales;
  const uint32_t* signs;
  int levels, bits, group, wpr;  // wpr: words per row
};
struct KvCacheArgs {
  KvHalf k, v;
  int D, heads, page;  // page: tokens of a page
  int64_t pages;
};
struct RopeArgs {
  const double* inv_freq;  // null: no rotary positions
  const int32_t* positions;
  int rot;
  bool interleaved;
  double gain;
  const uint8_t* axis;  // null: one axis; else the axis of each pair, `axes` rows of positions
  int64_t axis_stride;
  int axes;
};
hipError_t launch_rope(const void* x, int dt, int64_t tokens, int heads, int D, int64_t xts,
                       int64_t xhs, const RopeArgs& r, bool transposed, void* out, int64_t ots,
                       int64_t ohs, hipStream_t s);
hipError_t launch_kv_store(const KvCacheArgs& c, const void* k, const void* v, int dt,
                           int64_t tokens, const int64_t (&strides)[4], const int64_t* slots,
                           const RopeArgs& r, hipStream_t s);
hipError_t launch_kv_load(const KvCacheArgs& c, const int64_t* slots, int64_t tokens, void* k_out,
                          void* v_out, int odt, hipStream_t s);
struct AttendArgs {
  KvCacheArgs c;
  const void* q;
  int qdt, q_heads;
  int64_t q_stride;
  int B;
  const int32_t* q_offsets;
  int64_t M;
  const int32_t *kv_lens, *page_table;
  int table_width;
  const uint32_t* tree;
  int tree_words;
  float scale;
  void* out;
  int odt;
  void* ws;
};
size_t kv_attend_workspace(const KvCacheArgs& c, int q_heads, int B, int64_t M);
hipError_t launch_kv_attend(const AttendArgs& a, hipStream_t s);

// A decoding step (tq_step.h), resolved on the host.
struct PlanArgs {
  int32_t *free_pages, *state;
  int pages, page, B;
  const int32_t *lens, *counts;
  int32_t* table;
  int width;
  int M;
  const int32_t* parents;  // null: chains
  int words;               // of a row's tree mask
  const int32_t* shift;    // null: none
  int64_t* slots;
  int32_t *positions, *q_offsets, *kv_lens, *status;
  uint32_t* tree;
  int32_t* left;  // state itself, or another word
};
hipError_t launch_kv_plan(const PlanArgs& a, hipStream_t s);
struct KeepArgs {
  KvCacheArgs c;  // read where path is not null
  int32_t *free_pages, *state;
  int pages, page, B;
  const int32_t *lens, *q_offsets, *status, *kept, *path;  // q_offsets, status, path may be null
  int M;  // q_offsets are cut to [0, M]
  const int32_t* table;
  int width;
  int32_t *lens_out, *left;
};
hipError_t launch_kv_keep(const KeepArgs& a, hipStream_t s);
struct VerifyArgs {
  const void *target, *draft;  // draft may be null: point masses
  int tdt, ddt;
  int64_t tstride, dstride;  // elements
  bool tprobs, dprobs;
  int V, B, M;
  const int32_t *offsets, *tokens, *parents;  // parents null: chains
  const float *uniforms, *temperature;        // temperature null: 1
  int32_t *kept, *out_tokens, *path;
  void* ws;
};
size_t verify_workspace(int V, int B, int M, bool tprobs, bool drafted, bool dprobs);
hipError_t launch_verify(const VerifyArgs& a, hipStream_t s);

// Up to kMaxSlotIds int32 values passed by value to a kernel (tq_expert_cache_fetch).
constexpr int kMaxSlotIds = 512;
struct SlotIds {
  int32_t n;
  int32_t v[kMaxSlotIds];
};
hipError_t launch_put_ids(const SlotIds& ids, int32_t* dst, hipStream_t s);

}  // namespace tq
