// C ABI of the paged 8-bit and 4-bit caches (include/idx_cache.h, include/idx_cache4.h):
// host-side argument validation, workspace layout and dispatch. As in api.cpp, validation
// makes no HIP call.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "idx_cache.h"
#include "idx_cache4.h"
#include "launch.h"

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;  // of a launch
constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int hip_status(int e) { return e == 0 ? IDX_OK : IDX_ERR_HIP; }

bool page_size_built(int page_size) {
  return page_size == 16 || page_size == 32 || page_size == 64;
}

// partial results of `rows` rows cut into `splits`: sums, then (maximum, weight)
size_t partial_bytes(int64_t rows, int Hq, int splits) {
  if (splits <= 1) return 0;
  const size_t n = (size_t)rows * Hq * splits;
  return round_up(n * IDX_HEAD_DIM * sizeof(float), 256) + round_up(n * 2 * sizeof(float), 256);
}

// 16-token units of the longest row a call may hold
int64_t row_units(int max_pages, int K, int page_size) {
  return (int64_t)(K > 0 ? K : max_pages) * (page_size / 16);
}

bool shape_ok(int64_t rows, int B, int Hq, int Hkv, int max_pages, int page_size) {
  return rows >= 0 && rows <= kMaxInt && B >= 1 && Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 &&
         Hq / Hkv <= IDX_MAX_GROUP && max_pages >= 1 && page_size_built(page_size) &&
         (int64_t)max_pages * page_size <= kMaxInt;
}

// What the attention calls check; the workspace and the rows' own arrays apart. Scales are
// aligned to `scale_align` bytes.
int check_attend(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                 const void* k_scale, const void* v_scale, int scale_align,
                 const int32_t* kv_indptr,
                 const int32_t* kv_indices, const int32_t* kv_len, const float* slopes,
                 const void* out, int rows, int B, int Hq, int Hkv, int D, int n_pages,
                 int64_t n_indices, int max_pages, int page_size, float scale, float softcap,
                 idx_dtype dt) {
  if (rows < 0 || B < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || D < 1 || n_pages < 1 ||
      n_indices < 0 || max_pages < 1 || page_size < 1)
    return IDX_ERR_INVALID_ARG;
  if (dt != IDX_F32 && dt != IDX_BF16) return IDX_ERR_INVALID_ARG;
  if (!isfinite(scale) || !isfinite(softcap) || softcap < 0.f) return IDX_ERR_INVALID_ARG;
  if (softcap > 0.f && (softcap < IDX_MIN_SOFTCAP || softcap > IDX_MAX_SOFTCAP))
    return IDX_ERR_UNSUPPORTED;
  if (D != IDX_HEAD_DIM || dt != IDX_BF16 || Hq / Hkv > IDX_MAX_GROUP ||
      !page_size_built(page_size))
    return IDX_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * Hkv > kMaxInt || (int64_t)max_pages * page_size > kMaxInt ||
      (int64_t)Hq * D > kMaxInt)
    return IDX_ERR_INVALID_ARG;
  if (rows > 0) {
    if (q == nullptr || out == nullptr || kv_len == nullptr) return IDX_ERR_INVALID_ARG;
    if (q_stride < (int64_t)Hq * D || q_stride % 8 != 0) return IDX_ERR_INVALID_ARG;
    if (k_cache == nullptr || v_cache == nullptr || k_scale == nullptr || v_scale == nullptr ||
        kv_indptr == nullptr || (kv_indices == nullptr && n_indices > 0))
      return IDX_ERR_INVALID_ARG;
  }
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scale, scale_align) || !aligned(v_scale, scale_align) ||
      !aligned(kv_indptr, 4) || !aligned(kv_indices, 4) || !aligned(kv_len, 4) || !aligned(slopes, 4))
    return IDX_ERR_INVALID_ARG;
  return IDX_OK;
}

idxk::AttnArgs attend_args(int bits, const void* q, int64_t q_stride, const uint8_t* k_cache,
                           const uint8_t* v_cache, const void* k_scale, const void* v_scale,
                           const int32_t* kv_indptr, const int32_t* kv_indices,
                           const int32_t* kv_len, const float* slopes, void* out, int rows, int B,
                           int Hq, int Hkv, int n_pages, int64_t n_indices, int max_pages,
                           int page_size, float scale, float softcap, int splits, void* ws) {
  idxk::AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  if (bits == 8) {
    a.k_scale = static_cast<const float*>(k_scale);
    a.v_scale = static_cast<const float*>(v_scale);
  } else {
    a.k_exp = static_cast<const uint8_t*>(k_scale);
    a.v_exp = static_cast<const uint8_t*>(v_scale);
  }
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.kv_len = kv_len;
  a.slopes = slopes;
  a.out = static_cast<uint16_t*>(out);
  a.n_indices = n_indices;
  a.R = rows;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.page_size = page_size;
  a.score_scale = softcap > 0.f ? scale : scale * kLog2e;
  a.softcap = softcap;
  if (splits > 1) {
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float*>(
        static_cast<char*>(ws) +
        round_up((size_t)rows * Hq * splits * IDX_HEAD_DIM * sizeof(float), 256));
  }
  return a;
}

int check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned(ws, 256)))
    return IDX_ERR_WORKSPACE;
  return IDX_OK;
}

// How the rows of a call are cut.
idxk::AttnSplit single_split(int bits, int R, int Hq, int Hkv, int64_t units) {
  return bits == 8 ? idxk::attend_rows_split(R, Hkv, units)
                   : idxk::attend4_rows_split(R, Hkv, Hq / Hkv, units);
}
idxk::AttnSplit packed_split(int bits, int n_tok, int B, int Hq, int Hkv, int64_t units) {
  return bits == 8 ? idxk::attend_prefill_split(n_tok, B, Hq, Hkv, units)
                   : idxk::attend4_prefill_split(n_tok, B, Hq, Hkv, units);
}

size_t single_bytes(int bits, int R, int Hq, int Hkv, int max_pages, int K, int page_size) {
  if (R < 1 || K < 0 || !shape_ok(R, 1, Hq, Hkv, max_pages, page_size)) return 0;
  return partial_bytes(
      R, Hq, single_split(bits, R, Hq, Hkv, row_units(max_pages, K, page_size)).splits);
}

// idx_attend over the cache of so many bits, and idx_attend_prefill
int attend_single(int bits, const void* q, int64_t q_stride, const uint8_t* k_cache,
                  const uint8_t* v_cache, const void* k_scale, const void* v_scale,
                  const int32_t* kv_indptr, const int32_t* kv_indices, const int32_t* kv_len,
                  const int32_t* row_req, const int32_t* ids, const float* slopes, void* out, int R,
                  int B, int Hq, int Hkv, int D, int n_pages, int64_t n_indices, int max_pages,
                  int page_size, int K, float scale, float softcap, idx_dtype dt, void* ws,
                  size_t ws_bytes, void* stream) {
  const int st = check_attend(q, q_stride, k_cache, v_cache, k_scale, v_scale, bits == 8 ? 4 : 16,
                              kv_indptr, kv_indices, kv_len, slopes, out, R, B, Hq, Hkv, D,
                              n_pages, n_indices, max_pages, page_size, scale, softcap, dt);
  if (st != IDX_OK) return st;
  if (!aligned(row_req, 4) || !aligned(ids, 4)) return IDX_ERR_INVALID_ARG;
  if (K < 0 || (ids != nullptr) != (K > 0) || (row_req == nullptr && R > B))
    return IDX_ERR_INVALID_ARG;
  if ((int64_t)K * page_size > kMaxInt) return IDX_ERR_INVALID_ARG;
  if (R == 0) return IDX_OK;
  const idxk::AttnSplit sp = single_split(bits, R, Hq, Hkv, row_units(max_pages, K, page_size));
  // 256 threads for each of at most two workgroups a row, KV head and split (rows are cut,
  // and joined, only where rows times KV heads are a few hundred)
  if ((int64_t)R * Hkv * sp.splits * (Hq / Hkv > 32 ? 2 : 1) * 256 > kMaxThreads)
    return IDX_ERR_INVALID_ARG;
  const int wst = check_workspace(ws, ws_bytes, partial_bytes(R, Hq, sp.splits));
  if (wst != IDX_OK) return wst;
  idxk::AttnArgs a = attend_args(bits, q, q_stride, k_cache, v_cache, k_scale, v_scale, kv_indptr,
                                 kv_indices, kv_len, slopes, out, R, B, Hq, Hkv, n_pages,
                                 n_indices, max_pages, page_size, scale, softcap, sp.splits, ws);
  a.row_req = row_req;
  a.ids = ids;
  a.K = K;
  return hip_status(bits == 8 ? idxk::launch_attend_rows(a, sp, stream)
                              : idxk::launch_attend4_rows(a, sp, stream));
}

size_t packed_bytes(int bits, int n_tok, int B, int Hq, int Hkv, int max_pages, int page_size) {
  if (n_tok < 1 || !shape_ok(n_tok, B, Hq, Hkv, max_pages, page_size)) return 0;
  return partial_bytes(
      n_tok, Hq, packed_split(bits, n_tok, B, Hq, Hkv, row_units(max_pages, 0, page_size)).splits);
}

int attend_packed(int bits, const void* q, int64_t q_stride, const uint8_t* k_cache,
                  const uint8_t* v_cache, const void* k_scale, const void* v_scale,
                  const int32_t* kv_indptr, const int32_t* kv_indices, const int32_t* tok_indptr,
                  const int32_t* kv_len, const float* slopes, void* out, int n_tok, int B, int Hq,
                  int Hkv, int D, int n_pages, int64_t n_indices, int max_pages, int page_size,
                  float scale, float softcap, idx_dtype dt, void* ws, size_t ws_bytes,
                  void* stream) {
  const int st = check_attend(q, q_stride, k_cache, v_cache, k_scale, v_scale, bits == 8 ? 4 : 16,
                              kv_indptr, kv_indices, kv_len, slopes, out, n_tok, B, Hq, Hkv, D,
                              n_pages, n_indices, max_pages, page_size, scale, softcap, dt);
  if (st != IDX_OK) return st;
  if ((n_tok > 0 && tok_indptr == nullptr) || !aligned(tok_indptr, 4)) return IDX_ERR_INVALID_ARG;
  if (B > IDX_MAX_REQUESTS) return IDX_ERR_UNSUPPORTED;
  if (n_tok == 0) return IDX_OK;
  const idxk::AttnSplit sp =
      packed_split(bits, n_tok, B, Hq, Hkv, row_units(max_pages, 0, page_size));
  // up to 512 threads for each row tile, KV head and split
  if (idxk::attend_prefill_tiles(n_tok, B, Hq / Hkv, sp.rows) * Hkv * sp.splits * 512 >
      kMaxThreads)
    return IDX_ERR_INVALID_ARG;
  const int wst = check_workspace(ws, ws_bytes, partial_bytes(n_tok, Hq, sp.splits));
  if (wst != IDX_OK) return wst;
  idxk::AttnArgs a = attend_args(bits, q, q_stride, k_cache, v_cache, k_scale, v_scale, kv_indptr,
                                 kv_indices, kv_len, slopes, out, n_tok, B, Hq, Hkv, n_pages,
                                 n_indices, max_pages, page_size, scale, softcap, sp.splits, ws);
  a.tok_indptr = tok_indptr;
  return hip_status(bits == 8 ? idxk::launch_attend_prefill(a, sp, stream)
                              : idxk::launch_attend4_prefill(a, sp, stream));
}

// What the write and the read of a cache check; the caller's own scales apart.
int check_rows(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
               const int32_t* slots, const void* k_cache, const void* v_cache,
               const void* k_scale, const void* v_scale, int scale_align, int n_tok, int Hkv,
               int D, int n_pages, int page_size, idx_dtype dt, bool both) {
  if (n_tok < 0 || Hkv < 1 || D < 1 || n_pages < 1 || page_size < 1) return IDX_ERR_INVALID_ARG;
  if (dt != IDX_F32 && dt != IDX_BF16) return IDX_ERR_INVALID_ARG;
  if (D != IDX_HEAD_DIM || !page_size_built(page_size)) return IDX_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * Hkv > kMaxInt || (int64_t)n_pages * page_size > kMaxInt ||
      (int64_t)Hkv * D > kMaxInt ||
      ((int64_t)n_tok / 16 + 1) * (((int64_t)Hkv + 1) / 2) * 256 > kMaxThreads)
    return IDX_ERR_INVALID_ARG;
  if (n_tok > 0) {
    if (((k == nullptr || v == nullptr) && both) || slots == nullptr || k_cache == nullptr ||
        v_cache == nullptr || k_scale == nullptr || v_scale == nullptr)
      return IDX_ERR_INVALID_ARG;
    for (int64_t stride : {k != nullptr ? k_stride : (int64_t)Hkv * D,
                           v != nullptr ? v_stride : (int64_t)Hkv * D})
      if (stride < (int64_t)Hkv * D || stride % 8 != 0) return IDX_ERR_INVALID_ARG;
  }
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(k_scale, scale_align) || !aligned(v_scale, scale_align))
    return IDX_ERR_INVALID_ARG;
  return IDX_OK;
}

}  // namespace

extern "C" {

int idx_page_tables(const int32_t* seq_len, const int32_t* n_new, const int32_t* cursor,
                    int32_t* table, int32_t* free_ring, int32_t* seq_out, int32_t* cursor_out,
                    int32_t* kv_indptr, int32_t* kv_indices, int32_t* tok_indptr, int32_t* slots,
                    int32_t* tok_req, int32_t* tok_len, int B, int max_pages, int page_size,
                    int n_pages, int64_t n_indices, int n_tokens, void* stream) {
  const void* all[] = {seq_len,   n_new,     cursor,     table,      free_ring, seq_out,
                       cursor_out, kv_indptr, tok_indptr, kv_indices, slots,     tok_req,
                       tok_len};
  for (int i = 0; i < 9; ++i)
    if (all[i] == nullptr) return IDX_ERR_INVALID_ARG;
  for (const void* p : all)
    if (!aligned(p, 4)) return IDX_ERR_INVALID_ARG;
  if (B < 1 || max_pages < 1 || page_size < 1 || n_pages < 1 || n_indices < 0 || n_tokens < 0)
    return IDX_ERR_INVALID_ARG;
  if ((kv_indices == nullptr && n_indices > 0) ||
      (n_tokens > 0 && (slots == nullptr || tok_req == nullptr || tok_len == nullptr)))
    return IDX_ERR_INVALID_ARG;
  if ((int64_t)B * max_pages > kMaxInt || (int64_t)max_pages * page_size > kMaxInt ||
      (int64_t)n_pages * page_size > kMaxInt)
    return IDX_ERR_INVALID_ARG;
  if (seq_out == seq_len || cursor_out == cursor) return IDX_ERR_INVALID_ARG;
  if (B > IDX_MAX_REQUESTS) return IDX_ERR_UNSUPPORTED;
  return hip_status(idxk::launch_page_tables(seq_len, n_new, cursor, table, free_ring, seq_out,
                                             cursor_out, kv_indptr, kv_indices, tok_indptr, slots,
                                             tok_req, tok_len, B, max_pages, page_size, n_pages,
                                             n_indices, n_tokens, stream));
}

int idx_cache_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                    const int32_t* slots, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                    float* v_scale, int n_tok, int Hkv, int D, int n_pages, int page_size,
                    idx_dtype dt, void* stream) {
  const int st = check_rows(k, v, k_stride, v_stride, slots, k_cache, v_cache, k_scale, v_scale, 4,
                            n_tok, Hkv, D, n_pages, page_size, dt, true);
  if (st != IDX_OK) return st;
  if (n_tok == 0) return IDX_OK;
  return hip_status(idxk::launch_cache_write(k, v, k_stride, v_stride, slots, k_cache, v_cache,
                                             k_scale, v_scale, n_tok, Hkv, n_pages, page_size,
                                             dt == IDX_BF16, stream));
}

int idx_cache4_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                     const int32_t* slots, uint8_t* k_cache, uint8_t* v_cache, uint8_t* k_scale,
                     uint8_t* v_scale, int n_tok, int Hkv, int D, int n_pages, int page_size,
                     idx_dtype dt, void* stream) {
  const int st = check_rows(k, v, k_stride, v_stride, slots, k_cache, v_cache, k_scale, v_scale,
                            16, n_tok, Hkv, D, n_pages, page_size, dt, true);
  if (st != IDX_OK) return st;
  if (n_tok == 0) return IDX_OK;
  return hip_status(idxk::launch_cache4_write(k, v, k_stride, v_stride, slots, k_cache, v_cache,
                                              k_scale, v_scale, n_tok, Hkv, n_pages, page_size,
                                              dt == IDX_BF16, stream));
}

int idx_cache4_read(const int32_t* slots, const uint8_t* k_cache, const uint8_t* v_cache,
                    const uint8_t* k_scale, const uint8_t* v_scale, void* k, void* v,
                    int64_t k_stride, int64_t v_stride, int n_tok, int Hkv, int D, int n_pages,
                    int page_size, idx_dtype dt, void* stream) {
  const int st = check_rows(k, v, k_stride, v_stride, slots, k_cache, v_cache, k_scale, v_scale,
                            16, n_tok, Hkv, D, n_pages, page_size, dt, false);
  if (st != IDX_OK) return st;
  if (n_tok == 0 || (k == nullptr && v == nullptr)) return IDX_OK;
  return hip_status(idxk::launch_cache4_read(slots, k_cache, v_cache, k_scale, v_scale, k, v,
                                             k_stride, v_stride, n_tok, Hkv, n_pages, page_size,
                                             dt == IDX_BF16, stream));
}

size_t idx_attend_workspace_bytes(int R, int Hq, int Hkv, int max_pages, int K, int page_size) {
  return single_bytes(8, R, Hq, Hkv, max_pages, K, page_size);
}

int idx_attend(const void* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
               const float* k_scale, const float* v_scale, const int32_t* kv_indptr,
               const int32_t* kv_indices, const int32_t* kv_len, const int32_t* row_req,
               const int32_t* ids, const float* slopes, void* out, int R, int B, int Hq, int Hkv,
               int D, int n_pages, int64_t n_indices, int max_pages, int page_size, int K,
               float scale, float softcap, idx_dtype dt, void* ws, size_t ws_bytes, void* stream) {
  return attend_single(8, q, q_stride, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                       kv_len, row_req, ids, slopes, out, R, B, Hq, Hkv, D, n_pages, n_indices,
                       max_pages, page_size, K, scale, softcap, dt, ws, ws_bytes, stream);
}

size_t idx_attend4_workspace_bytes(int R, int Hq, int Hkv, int max_pages, int K, int page_size) {
  return single_bytes(4, R, Hq, Hkv, max_pages, K, page_size);
}

int idx_attend4(const void* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* kv_indptr,
                const int32_t* kv_indices, const int32_t* kv_len, const int32_t* row_req,
                const int32_t* ids, const float* slopes, void* out, int R, int B, int Hq, int Hkv,
                int D, int n_pages, int64_t n_indices, int max_pages, int page_size, int K,
                float scale, float softcap, idx_dtype dt, void* ws, size_t ws_bytes,
                void* stream) {
  return attend_single(4, q, q_stride, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                       kv_len, row_req, ids, slopes, out, R, B, Hq, Hkv, D, n_pages, n_indices,
                       max_pages, page_size, K, scale, softcap, dt, ws, ws_bytes, stream);
}

size_t idx_attend_prefill_workspace_bytes(int n_tok, int B, int Hq, int Hkv, int max_pages,
                                          int page_size) {
  return packed_bytes(8, n_tok, B, Hq, Hkv, max_pages, page_size);
}

int idx_attend_prefill(const void* q, int64_t q_stride, const uint8_t* k_cache,
                       const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* kv_indptr, const int32_t* kv_indices,
                       const int32_t* tok_indptr, const int32_t* kv_len, const float* slopes,
                       void* out, int n_tok, int B, int Hq, int Hkv, int D, int n_pages,
                       int64_t n_indices, int max_pages, int page_size, float scale,
                       float softcap, idx_dtype dt, void* ws, size_t ws_bytes, void* stream) {
  return attend_packed(8, q, q_stride, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                       tok_indptr, kv_len, slopes, out, n_tok, B, Hq, Hkv, D, n_pages, n_indices,
                       max_pages, page_size, scale, softcap, dt, ws, ws_bytes, stream);
}

size_t idx_attend4_prefill_workspace_bytes(int n_tok, int B, int Hq, int Hkv, int max_pages,
                                           int page_size) {
  return packed_bytes(4, n_tok, B, Hq, Hkv, max_pages, page_size);
}

int idx_attend4_prefill(const void* q, int64_t q_stride, const uint8_t* k_cache,
                        const uint8_t* v_cache, const uint8_t* k_scale, const uint8_t* v_scale,
                        const int32_t* kv_indptr, const int32_t* kv_indices,
                        const int32_t* tok_indptr, const int32_t* kv_len, const float* slopes,
                        void* out, int n_tok, int B, int Hq, int Hkv, int D, int n_pages,
                        int64_t n_indices, int max_pages, int page_size, float scale,
                        float softcap, idx_dtype dt, void* ws, size_t ws_bytes, void* stream) {
  return attend_packed(4, q, q_stride, k_cache, v_cache, k_scale, v_scale, kv_indptr, kv_indices,
                       tok_indptr, kv_len, slopes, out, n_tok, B, Hq, Hkv, D, n_pages, n_indices,
                       max_pages, page_size, scale, softcap, dt, ws, ws_bytes, stream);
}

}  // extern "C"
