// extern "C" entry points of the paged serving step (page planning, rotary
// positions, page writes, attention, drafted trees) and of e4m3 products:
// argument checks on the host, then asynchronous launches on the caller's stream.
#include <stdint.h>

#include "misa.h"
#include "misa_launch.h"

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 26;
constexpr int64_t kMaxSlots = (int64_t)1 << 31;   // pool rows are numbered in 31 bits

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline misa_status from_hip(hipError_t e) { return e == hipSuccess ? MISA_OK : MISA_ERR_HIP; }

#define MISA_TRY(expr)              \
  do {                              \
    misa_status _st = (expr);       \
    if (_st != MISA_OK) return _st; \
  } while (0)

misa_status check_rope(const misa_rope_spec* r, int32_t head_dim) {
  if (r == nullptr || r->inv_freq == nullptr || r->positions == nullptr) return MISA_ERR_INVALID_ARG;
  if (r->rotary_dim < 2 || r->rotary_dim > 1024 || (r->rotary_dim & 1) != 0) return MISA_ERR_INVALID_ARG;
  if (r->rot_start < 0 || r->rot_start > head_dim - r->rotary_dim) return MISA_ERR_INVALID_ARG;
  if (r->layout != MISA_ROPE_HALF && r->layout != MISA_ROPE_INTERLEAVED) return MISA_ERR_INVALID_ARG;
  if (!(r->mscale == r->mscale)) return MISA_ERR_INVALID_ARG;
  return MISA_OK;
}

// strides that keep the head_dim values of every (token, head) apart: either
// dimension may be the outer one
bool strides_apart(int64_t n_tokens, int64_t n_heads, int64_t head_dim, int64_t st, int64_t sh) {
  if (st < 0 || sh < 0) return false;
  if (n_heads > 1 && sh < head_dim) return false;
  if (n_tokens > 1 && st < head_dim) return false;
  if (n_tokens > 1 && n_heads > 1) return st >= sh * (n_heads - 1) + head_dim || sh >= st * (n_tokens - 1) + head_dim;
  return true;
}

struct Span {
  const void* at;
  int64_t bytes;   // 0: nothing there
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
  return a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

misa_status check_pool(int64_t n_pages, int32_t page_keys) {
  if (n_pages < 1 || page_keys < 1) return MISA_ERR_INVALID_ARG;
  if (n_pages >= kMaxSlots || n_pages * page_keys >= kMaxSlots) return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

misa_status check_attn(const misa_attn_shape* s, const misa_kv_pages* p) {
  if (s == nullptr || p == nullptr) return MISA_ERR_INVALID_ARG;
  if (s->n_seq < 1 || s->n_tokens < 0 || s->n_kv_heads < 1 || s->n_heads < 1 || s->max_new < 0)
    return MISA_ERR_INVALID_ARG;
  if (s->n_heads % s->n_kv_heads != 0) return MISA_ERR_INVALID_ARG;
  if (!(s->scale == s->scale) || s->scale - s->scale != 0.f) return MISA_ERR_INVALID_ARG;
  if (s->q_stride_token < 0 || s->q_stride_head < 0 || s->q_stride_token % 8 != 0 || s->q_stride_head % 8 != 0)
    return MISA_ERR_INVALID_ARG;
  if (s->head_dim != 64 && s->head_dim != 128) return MISA_ERR_UNSUPPORTED;
  if (s->n_seq > 65535 || s->n_heads > 1024 || s->n_tokens > kMaxTokens) return MISA_ERR_UNSUPPORTED;
  if (p->kdtype != MISA_K_BF16 && p->kdtype != MISA_K_FP8_E4M3) return MISA_ERR_INVALID_ARG;
  if (p->max_pages < 1) return MISA_ERR_INVALID_ARG;
  if (p->max_pages >= kMaxSlots || p->max_pages * p->page_keys >= kMaxSlots) return MISA_ERR_UNSUPPORTED;
  return check_pool(p->n_pages, p->page_keys);
}

misa_status check_attn_pointers(const misa_kv_pages* p, const void* q, const void* q_start, const void* kv_lens,
                                const void* out) {
  if (p->k == nullptr || p->v == nullptr || !aligned16(p->k) || !aligned16(p->v) || p->block_table == nullptr)
    return MISA_ERR_INVALID_ARG;
  if (p->kdtype == MISA_K_FP8_E4M3 && (p->k_scale == nullptr || p->v_scale == nullptr)) return MISA_ERR_INVALID_ARG;
  if (q == nullptr || !aligned16(q) || out == nullptr || !aligned16(out)) return MISA_ERR_INVALID_ARG;
  if (q_start == nullptr || kv_lens == nullptr) return MISA_ERR_INVALID_ARG;
  return MISA_OK;
}

misa_status attention(const misa_attn_shape* s, const misa_kv_pages* p, const uint16_t* q, const int32_t* q_start,
                      const int32_t* kv_lens, const int32_t* idx, int32_t topk, const uint32_t* mask, int32_t words,
                      uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  MISA_TRY(check_attn_pointers(p, q, q_start, kv_lens, out));
  if (!misa::attn_fits(*s, *p, topk, mask != nullptr)) return MISA_ERR_UNSUPPORTED;
  const size_t need = misa::attn_workspace_bytes(*s, *p, topk, mask != nullptr);
  if (need > 0 && (ws == nullptr || !aligned16(ws) || ws_bytes < need)) return MISA_ERR_WORKSPACE;
  if (s->n_tokens == 0) return MISA_OK;
  return from_hip(misa::launch_attention(*s, *p, q, q_start, kv_lens, idx, topk, mask, words, out, lse, ws,
                                         (hipStream_t)stream));
}

constexpr int32_t kMaxTreeWords = 1024;
constexpr int64_t kMaxCols = (int64_t)1 << 20;
constexpr int64_t kMaxBlocks = (int64_t)1 << 27;    // quantised in one call
constexpr int64_t kMaxStride = (int64_t)1 << 22;   // of rows of codes: a tile of 256 stays within 32 bits

misa_status check_matmul(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 1 || k < 1) return MISA_ERR_INVALID_ARG;
  if (k % 16 != 0 || k > kMaxCols || n > kMaxTokens || m > kMaxTokens) return MISA_ERR_UNSUPPORTED;
  if (!misa::matmul_q8_fits(m, n, k)) return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

}  // namespace

extern "C" {

misa_status misa_plan_pages(int32_t n_seq, const int32_t* cached_lens, const int32_t* new_lens, int32_t page_keys,
                            const int32_t* free_pages, int32_t n_free, int32_t* block_table, int64_t max_pages,
                            int32_t* q_start, int32_t* kv_lens, int64_t* slots, int32_t* positions, int64_t n_tokens,
                            int32_t* n_taken, void* stream) {
  if (n_seq < 1 || page_keys < 1 || max_pages < 1 || n_free < 0 || n_tokens < 0) return MISA_ERR_INVALID_ARG;
  if (cached_lens == nullptr || new_lens == nullptr || block_table == nullptr || q_start == nullptr ||
      kv_lens == nullptr || n_taken == nullptr)
    return MISA_ERR_INVALID_ARG;
  if (n_free > 0 && free_pages == nullptr) return MISA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (slots == nullptr || positions == nullptr)) return MISA_ERR_INVALID_ARG;
  if (n_seq > 65535 || n_tokens > kMaxTokens || max_pages >= kMaxSlots) return MISA_ERR_UNSUPPORTED;
  // workgroups read the inputs while others write
  const Span in[] = {{cached_lens, 4 * (int64_t)n_seq}, {new_lens, 4 * (int64_t)n_seq}, {free_pages, 4 * (int64_t)n_free}};
  const Span out[] = {{block_table, 4 * n_seq * max_pages}, {q_start, 4 * ((int64_t)n_seq + 1)}, {kv_lens, 4 * (int64_t)n_seq},
                      {slots, 8 * n_tokens}, {positions, 4 * n_tokens}, {n_taken, 4}};
  for (const Span& o : out) {
    for (const Span& i : in)
      if (overlap(o, i)) return MISA_ERR_INVALID_ARG;
    for (const Span& p : out)
      if (&p != &o && overlap(o, p)) return MISA_ERR_INVALID_ARG;
  }
  return from_hip(misa::launch_plan_pages(n_seq, cached_lens, new_lens, page_keys, free_pages, n_free, block_table,
                                          max_pages, q_start, kv_lens, slots, positions, n_tokens, n_taken,
                                          (hipStream_t)stream));
}

misa_status misa_rope(const misa_rope_spec* spec, const void* x, misa_dtype dtype, int64_t n_tokens, int32_t n_heads,
                      int32_t head_dim, int64_t x_stride_token, int64_t x_stride_head, void* out,
                      int64_t out_stride_token, int64_t out_stride_head, void* stream) {
  if (n_tokens < 0 || n_heads < 1 || head_dim < 2) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_T_BF16 && dtype != MISA_T_FP16 && dtype != MISA_T_FP32) return MISA_ERR_INVALID_ARG;
  MISA_TRY(check_rope(spec, head_dim));
  if (x == nullptr || out == nullptr) return MISA_ERR_INVALID_ARG;
  if (!strides_apart(n_tokens, n_heads, head_dim, out_stride_token, out_stride_head)) return MISA_ERR_INVALID_ARG;
  if (x_stride_token < 0 || x_stride_head < 0) return MISA_ERR_INVALID_ARG;
  if (x == out && (x_stride_token != out_stride_token || x_stride_head != out_stride_head))
    return MISA_ERR_INVALID_ARG;
  if (n_tokens > kMaxTokens || (int64_t)n_heads * head_dim > (1 << 20)) return MISA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MISA_OK;
  return from_hip(misa::launch_rope(*spec, x, dtype, n_tokens, n_heads, head_dim, x_stride_token, x_stride_head, out,
                                    out_stride_token, out_stride_head, (hipStream_t)stream));
}

misa_status misa_write_pages(int64_t n_tokens, int32_t n_heads, int32_t head_dim, const uint16_t* k,
                             int64_t k_stride_token, int64_t k_stride_head, const uint16_t* v,
                             int64_t v_stride_token, int64_t v_stride_head, const int64_t* slots,
                             const misa_rope_spec* spec, void* k_pages, void* v_pages, misa_kdtype kdtype,
                             float* k_scale_pages, float* v_scale_pages, int64_t n_pages, int32_t page_keys,
                             void* stream) {
  if (n_tokens < 0 || n_heads < 1 || head_dim < 1) return MISA_ERR_INVALID_ARG;
  if (kdtype != MISA_K_BF16 && kdtype != MISA_K_FP8_E4M3) return MISA_ERR_INVALID_ARG;
  if (k == nullptr || !aligned16(k) || slots == nullptr || k_pages == nullptr || !aligned16(k_pages))
    return MISA_ERR_INVALID_ARG;
  if ((v == nullptr) != (v_pages == nullptr) || !aligned16(v) || !aligned16(v_pages)) return MISA_ERR_INVALID_ARG;
  if (kdtype == MISA_K_FP8_E4M3 && (k_scale_pages == nullptr || (v != nullptr && v_scale_pages == nullptr)))
    return MISA_ERR_INVALID_ARG;
  if (k_stride_token < 0 || k_stride_head < 0 || k_stride_token % 8 != 0 || k_stride_head % 8 != 0)
    return MISA_ERR_INVALID_ARG;
  if (v != nullptr && (v_stride_token < 0 || v_stride_head < 0 || v_stride_token % 8 != 0 || v_stride_head % 8 != 0))
    return MISA_ERR_INVALID_ARG;
  if (spec != nullptr) {
    MISA_TRY(check_rope(spec, head_dim));
    if (spec->backward != 0) return MISA_ERR_INVALID_ARG;
  }
  MISA_TRY(check_pool(n_pages, page_keys));
  if (head_dim % 8 != 0 || head_dim > 512 || n_tokens > kMaxTokens || (int64_t)n_heads * head_dim > (1 << 20))
    return MISA_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MISA_OK;
  return from_hip(misa::launch_write_pages(n_tokens, n_heads, head_dim, k, k_stride_token, k_stride_head, v,
                                           v_stride_token, v_stride_head, slots, spec, k_pages, v_pages, kdtype,
                                           k_scale_pages, v_scale_pages, n_pages * page_keys, (hipStream_t)stream));
}

size_t misa_attention_paged_workspace_bytes(const misa_attn_shape* shape, const misa_kv_pages* pages) {
  if (check_attn(shape, pages) != MISA_OK) return 0;
  return misa::attn_workspace_bytes(*shape, *pages, 0, false);
}

misa_status misa_attention_paged(const misa_attn_shape* shape, const misa_kv_pages* pages, const uint16_t* q,
                                 const int32_t* q_start, const int32_t* kv_lens, uint16_t* out, float* lse, void* ws,
                                 size_t ws_bytes, void* stream) {
  MISA_TRY(check_attn(shape, pages));
  return attention(shape, pages, q, q_start, kv_lens, nullptr, 0, nullptr, 0, out, lse, ws, ws_bytes, stream);
}

size_t misa_attention_selected_workspace_bytes(const misa_attn_shape* shape, const misa_kv_pages* pages,
                                               int32_t topk) {
  if (check_attn(shape, pages) != MISA_OK || topk < 1 || topk > MISA_MAX_TOPK) return 0;
  return misa::attn_workspace_bytes(*shape, *pages, topk, false);
}

misa_status misa_attention_selected(const misa_attn_shape* shape, const misa_kv_pages* pages, const uint16_t* q,
                                    const int32_t* q_start, const int32_t* kv_lens, const int32_t* idx, int32_t topk,
                                    uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  MISA_TRY(check_attn(shape, pages));
  if (idx == nullptr || topk < 1 || topk > MISA_MAX_TOPK) return MISA_ERR_INVALID_ARG;
  return attention(shape, pages, q, q_start, kv_lens, idx, topk, nullptr, 0, out, lse, ws, ws_bytes, stream);
}

misa_status misa_plan_tree(int32_t n_seq, const int32_t* parents, const int32_t* q_start, const int32_t* kv_lens,
                           int64_t n_tokens, int32_t words, uint32_t* mask, int32_t* positions, void* stream) {
  if (n_seq < 1 || n_tokens < 0 || words < 1) return MISA_ERR_INVALID_ARG;
  if (q_start == nullptr || kv_lens == nullptr) return MISA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (parents == nullptr || mask == nullptr || positions == nullptr)) return MISA_ERR_INVALID_ARG;
  if (n_seq > 65535 || n_tokens > kMaxTokens || words > kMaxTreeWords) return MISA_ERR_UNSUPPORTED;
  const Span in[] = {{parents, 4 * n_tokens}, {q_start, 4 * ((int64_t)n_seq + 1)}, {kv_lens, 4 * (int64_t)n_seq}};
  const Span out[] = {{mask, 4 * n_tokens * words}, {positions, 4 * n_tokens}};
  for (const Span& o : out)
    for (const Span& i : in)
      if (overlap(o, i)) return MISA_ERR_INVALID_ARG;
  if (overlap(out[0], out[1])) return MISA_ERR_INVALID_ARG;
  if (n_tokens == 0) return MISA_OK;
  return from_hip(misa::launch_plan_tree(n_seq, parents, q_start, kv_lens, n_tokens, words, mask, positions,
                                         (hipStream_t)stream));
}

size_t misa_attention_tree_workspace_bytes(const misa_attn_shape* shape, const misa_kv_pages* pages) {
  if (check_attn(shape, pages) != MISA_OK) return 0;
  return misa::attn_workspace_bytes(*shape, *pages, 0, true);
}

misa_status misa_attention_tree(const misa_attn_shape* shape, const misa_kv_pages* pages, const uint16_t* q,
                                const int32_t* q_start, const int32_t* kv_lens, const uint32_t* mask, int32_t words,
                                uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  MISA_TRY(check_attn(shape, pages));
  if (mask == nullptr || words < 1) return MISA_ERR_INVALID_ARG;
  if (words > kMaxTreeWords) return MISA_ERR_UNSUPPORTED;
  return attention(shape, pages, q, q_start, kv_lens, nullptr, 0, mask, words, out, lse, ws, ws_bytes, stream);
}

misa_status misa_keep_path(int32_t n_seq, const int32_t* path, int32_t max_path, const int32_t* q_start,
                           const int32_t* kv_lens, const int32_t* block_table, int64_t max_pages, int32_t n_heads,
                           int32_t head_dim, void* k_pages, void* v_pages, misa_kdtype kdtype, float* k_scale_pages,
                           float* v_scale_pages, int64_t n_pages, int32_t page_keys, int32_t* kept_lens, void* stream) {
  if (n_seq < 1 || max_path < 1 || max_pages < 1 || n_heads < 1 || head_dim < 1) return MISA_ERR_INVALID_ARG;
  if (kdtype != MISA_K_BF16 && kdtype != MISA_K_FP8_E4M3) return MISA_ERR_INVALID_ARG;
  if (path == nullptr || q_start == nullptr || kv_lens == nullptr || block_table == nullptr || kept_lens == nullptr)
    return MISA_ERR_INVALID_ARG;
  if (k_pages == nullptr || !aligned16(k_pages) || !aligned16(v_pages)) return MISA_ERR_INVALID_ARG;
  const bool fp8 = kdtype == MISA_K_FP8_E4M3;
  if (fp8 && (k_scale_pages == nullptr || (v_pages != nullptr && v_scale_pages == nullptr))) return MISA_ERR_INVALID_ARG;
  MISA_TRY(check_pool(n_pages, page_keys));
  if (n_seq > 65535 || max_path > (1 << 20) || max_pages >= kMaxSlots) return MISA_ERR_UNSUPPORTED;
  if (head_dim % 8 != 0 || head_dim > 512 || (int64_t)n_heads * head_dim > (1 << 20)) return MISA_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)n_heads * head_dim * (fp8 ? 1 : 2), slots = n_pages * page_keys;
  const Span lens{kept_lens, 4 * (int64_t)n_seq};
  const Span others[] = {{path, 4 * (int64_t)n_seq * max_path}, {q_start, 4 * ((int64_t)n_seq + 1)},
                         {kv_lens, 4 * (int64_t)n_seq}, {block_table, 4 * n_seq * max_pages}, {k_pages, slots * row},
                         {v_pages, v_pages != nullptr ? slots * row : 0}, {k_scale_pages, fp8 ? 4 * slots * n_heads : 0},
                         {v_scale_pages, fp8 && v_pages != nullptr ? 4 * slots * n_heads : 0}};
  for (const Span& o : others)   // workgroups read the lengths while others write theirs
    if (overlap(lens, o)) return MISA_ERR_INVALID_ARG;
  for (int i = 4; i < 8; ++i)    // the pools are apart, from each other and from what says where rows go
    for (int j = 0; j < i; ++j)
      if (overlap(others[i], others[j])) return MISA_ERR_INVALID_ARG;
  const misa::KeepArgs a{path, q_start, kv_lens, block_table, max_path, max_pages, n_pages, page_keys,
                         static_cast<char*>(k_pages), static_cast<char*>(v_pages), (int)row,
                         fp8 ? k_scale_pages : nullptr, fp8 ? v_scale_pages : nullptr, n_heads, kept_lens};
  return from_hip(misa::launch_keep_path(n_seq, a, (hipStream_t)stream));
}

misa_status misa_quantize_blocks(const void* x, misa_dtype dtype, int64_t rows, int64_t cols, int64_t x_stride,
                                 int32_t block_rows, uint8_t* codes, float* scale, void* stream) {
  if (rows < 0 || cols < 1 || x_stride < 0) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_T_BF16 && dtype != MISA_T_FP16 && dtype != MISA_T_FP32) return MISA_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != 128) return MISA_ERR_INVALID_ARG;
  if (x == nullptr || !aligned16(x) || codes == nullptr || !aligned16(codes) || scale == nullptr)
    return MISA_ERR_INVALID_ARG;
  if (x_stride % (dtype == MISA_T_FP32 ? 4 : 8) != 0) return MISA_ERR_INVALID_ARG;
  if (cols % 16 != 0 || cols > kMaxCols || rows > kMaxTokens || rows * ((cols + 127) / 128) > kMaxBlocks)
    return MISA_ERR_UNSUPPORTED;
  if (rows == 0) return MISA_OK;
  const int64_t size = dtype == MISA_T_FP32 ? 4 : 2;
  const Span in{x, ((rows - 1) * x_stride + cols) * size};
  const Span out[] = {{codes, rows * cols}, {scale, 4 * ((rows + block_rows - 1) / block_rows) * ((cols + 127) / 128)}};
  if (overlap(in, out[0]) || overlap(in, out[1]) || overlap(out[0], out[1])) return MISA_ERR_INVALID_ARG;
  return from_hip(misa::launch_quantize_blocks(x, dtype, rows, cols, x_stride, block_rows, codes, scale, (hipStream_t)stream));
}

size_t misa_matmul_q8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (check_matmul(m, n, k) != MISA_OK) return 0;
  return misa::matmul_q8_workspace_bytes(m, n, k);
}

misa_status misa_matmul_q8(int64_t m, int64_t n, int64_t k, const uint8_t* x, int64_t x_stride, const float* x_scale,
                           const uint8_t* w, int64_t w_stride, const float* w_scale, uint16_t* out, int64_t out_stride,
                           void* ws, size_t ws_bytes, void* stream) {
  MISA_TRY(check_matmul(m, n, k));
  if (x == nullptr || !aligned16(x) || w == nullptr || !aligned16(w) || x_scale == nullptr || w_scale == nullptr ||
      out == nullptr)
    return MISA_ERR_INVALID_ARG;
  if (x_stride < 0 || w_stride < 0 || x_stride % 16 != 0 || w_stride % 16 != 0) return MISA_ERR_INVALID_ARG;
  if (m > 1 && out_stride < n) return MISA_ERR_INVALID_ARG;
  if (x_stride > kMaxStride || w_stride > kMaxStride || out_stride > ((int64_t)1 << 40)) return MISA_ERR_UNSUPPORTED;
  const size_t need = misa::matmul_q8_workspace_bytes(m, n, k);
  if (need > 0 && (ws == nullptr || !aligned16(ws) || ws_bytes < need)) return MISA_ERR_WORKSPACE;
  if (m == 0) return MISA_OK;
  const Span y{out, 2 * ((m - 1) * out_stride + n)};
  const int64_t across = (k + 127) / 128;
  const Span in[] = {{x, (m - 1) * x_stride + k}, {w, (n - 1) * w_stride + k}, {x_scale, 4 * m * across},
                     {w_scale, 4 * ((n + 127) / 128) * across}};
  for (const Span& i : in)
    if (overlap(y, i)) return MISA_ERR_INVALID_ARG;
  return from_hip(misa::launch_matmul_q8(misa::MatmulArgs{x, w, x_scale, w_scale, out, x_stride, w_stride, out_stride, m, n, k},
                                         ws, (hipStream_t)stream));
}

}  // extern "C"
