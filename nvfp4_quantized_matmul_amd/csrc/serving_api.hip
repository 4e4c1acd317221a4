// C ABI of the serving operators (cache append, paged attention, sampling):
// argument checks and launches.  Every check runs on the host before anything
// is enqueued; sequence lengths, row offsets and page tables live on the
// device and are bounded by the kernels.
#include <climits>
#include <cstdint>

#include "nvfp4_internal.hpp"

namespace {

bool mul_ok(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r) && *r >= 0; }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid_dtype(int dt) { return dt == NVFP4_F32 || dt == NVFP4_BF16 || dt == NVFP4_F16; }

int64_t dtype_size(nvfp4_dtype_t dt) { return dt == NVFP4_F32 ? 4 : 2; }

int launched() { return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

// Positions are 32-bit in the kernels, with room for a tile past the end.
constexpr int64_t kMaxPositions = 1LL << 30;
// A block of the append turns up to four tokens' query heads, of up to 128 items
// each, in a 32-bit index.
constexpr int64_t kMaxTurnedHeads = 1LL << 20;

// Elements from the first to behind the last one of [tokens, heads, dim] with
// these strides.
bool extent(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs, int64_t* n) {
  int64_t a, b;
  return mul_ok(tokens - 1, ts, &a) && mul_ok(heads - 1, hs, &b) && !__builtin_add_overflow(a, b, n) &&
         !__builtin_add_overflow(*n, dim, n);
}

bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

int check_page(int64_t page, int64_t dim) {
  if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256) return NVFP4_ERR_UNSUPPORTED;
  if (dim != 64 && dim != 128 && dim != 192 && dim != 256) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

int check_cache(const nvfp4_kv_cache_t* c, int64_t* bytes) {
  if (!c) return NVFP4_ERR_NULLPTR;
  if (c->pages < 0 || c->heads < 1 || c->pages > INT_MAX || c->heads > INT_MAX) return NVFP4_ERR_SHAPE;
  const int st = check_page(c->page, c->dim);
  if (st != NVFP4_OK) return st;
  int64_t t;
  if (!mul_ok(c->pages, c->heads, &t) || !mul_ok(t, c->page * c->dim, bytes)) return NVFP4_ERR_SHAPE;
  if (c->pages == 0) return NVFP4_OK;
  if (!c->k || !c->v || !c->k_scales || !c->v_scales) return NVFP4_ERR_NULLPTR;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int check_sizes(int64_t heads_q, int64_t heads, int64_t page, int64_t tokens, int64_t batch, int64_t max_q,
                int64_t width) {
  if (tokens < 0 || batch < 0 || max_q < 0 || width < 0 || heads_q < 0) return NVFP4_ERR_SHAPE;
  if (tokens > INT_MAX || batch > INT_MAX || heads_q > INT_MAX || max_q > kMaxPositions) return NVFP4_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(width, page, &t) || t > kMaxPositions) return NVFP4_ERR_SHAPE;
  // rows of a sequence and head count in 32 bits
  if (!mul_ok(max_q, heads_q, &t) || t > kMaxPositions || !mul_ok(tokens, heads_q, &t) || t > INT_MAX) return NVFP4_ERR_SHAPE;
  if (!mul_ok(tokens, heads, &t) || t > INT_MAX) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

int check_sequences(const int32_t* cu_q, int64_t tokens, int64_t batch, const int32_t* table, int64_t width,
                    const int32_t* lens) {
  if (!cu_q && tokens != batch) return NVFP4_ERR_SHAPE;
  if (!lens || (width > 0 && !table)) return NVFP4_ERR_NULLPTR;
  if (!aligned(lens, 4) || !aligned(table, 4) || !aligned(cu_q, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_kv_append(const nvfp4_kv_cache_t* cache, const void* k, int64_t k_token, int64_t k_head,
                    const void* v, int64_t v_token, int64_t v_head, const void* q, int64_t q_token,
                    int64_t q_head, int64_t heads_q, void* q_out, nvfp4_dtype_t dtype, int64_t tokens,
                    const int32_t* cu_q, int64_t batch, int64_t max_q, const int32_t* table,
                    int64_t table_width, const int32_t* lens, const float* inv_freq, int64_t rot,
                    int interleaved, hipStream_t stream) {
  int64_t cache_bytes = 0, nk, nv, nq = 0, no = 0;
  int st = check_cache(cache, &cache_bytes);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(dtype)) return NVFP4_ERR_DTYPE;
  st = check_sizes(heads_q, cache->heads, cache->page, tokens, batch, max_q, table_width);
  if (st != NVFP4_OK) return st;
  if (rot < 0 || rot % 2 != 0 || rot > cache->dim || (rot > 0) != (inv_freq != nullptr)) return NVFP4_ERR_SHAPE;
  if ((q != nullptr) != (q_out != nullptr)) return NVFP4_ERR_SHAPE;
  if (k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0 || q_token < 0 || q_head < 0) return NVFP4_ERR_SHAPE;
  if (!q) heads_q = 0;
  if (heads_q > kMaxTurnedHeads) return NVFP4_ERR_SHAPE;
  if (!cu_q && tokens != batch) return NVFP4_ERR_SHAPE;
  if (tokens == 0 || batch == 0) return NVFP4_OK;
  if (max_q == 0) return NVFP4_ERR_SHAPE;   // new tokens, and none in any sequence
  st = check_sequences(cu_q, tokens, batch, table, table_width, lens);
  if (st != NVFP4_OK) return st;
  if (!k || !v) return NVFP4_ERR_NULLPTR;
  const int64_t size = dtype_size(dtype);
  if (!aligned(k, size) || !aligned(v, size) || !aligned(inv_freq, 4) || (q && (!aligned(q, size) || !aligned(q_out, 16))))
    return NVFP4_ERR_ALIGN;
  if (!extent(tokens, cache->heads, cache->dim, k_token, k_head, &nk) || !mul_ok(nk, size, &nk) ||
      !extent(tokens, cache->heads, cache->dim, v_token, v_head, &nv) || !mul_ok(nv, size, &nv))
    return NVFP4_ERR_SHAPE;
  if (heads_q > 0) {
    if (!extent(tokens, heads_q, cache->dim, q_token, q_head, &nq) || !mul_ok(nq, size, &nq) ||
        !mul_ok(tokens * heads_q, cache->dim * size, &no))
      return NVFP4_ERR_SHAPE;
    if (overlaps(q_out, no, q, nq) || overlaps(q_out, no, k, nk) || overlaps(q_out, no, v, nv)) return NVFP4_ERR_SHAPE;
    if (overlaps(q_out, no, cache->k, cache_bytes) || overlaps(q_out, no, cache->v, cache_bytes)) return NVFP4_ERR_SHAPE;
  }
  if (nvfp4host::kv_append_blocks(cache->page, cache->heads, heads_q, tokens, batch, max_q) > nvfp4host::kMaxGrid256)
    return NVFP4_ERR_GRID;
  nvfp4host::launch_kv_append(*cache, k, k_token, k_head, v, v_token, v_head, q, q_token, q_head, heads_q, q_out, dtype,
                              tokens, cu_q, batch, max_q, table, table_width, lens, inv_freq, rot, interleaved != 0, stream);
  return launched();
}

int64_t nvfp4_paged_attention_workspace_size(int64_t tokens, int64_t heads_q, int64_t heads, int64_t dim,
                                             int64_t page, int64_t batch, int64_t max_q,
                                             int64_t table_width, int64_t window, nvfp4_dtype_t dtype) {
  int st = check_page(page, dim);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(dtype)) return NVFP4_ERR_DTYPE;
  if (heads < 1 || heads_q % heads != 0) return NVFP4_ERR_SHAPE;
  st = check_sizes(heads_q, heads, page, tokens, batch, max_q, table_width);
  if (st != NVFP4_OK) return st;
  if (tokens == 0 || batch == 0 || heads_q == 0 || max_q == 0) return 0;
  return nvfp4host::paged_attention_bytes(tokens, heads_q, heads, dim, page, batch, max_q, table_width, window, dtype);
}

int nvfp4_paged_attention(const nvfp4_kv_cache_t* cache, const void* q, int64_t q_token, int64_t q_head,
                          int64_t heads_q, nvfp4_dtype_t dtype, int64_t tokens, const int32_t* cu_q,
                          int64_t batch, int64_t max_q, const int32_t* table, int64_t table_width,
                          const int32_t* lens, int64_t window, float scale, void* workspace,
                          int64_t workspace_bytes, void* out, hipStream_t stream) {
  int64_t cache_bytes = 0, nq, no;
  int st = check_cache(cache, &cache_bytes);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(dtype)) return NVFP4_ERR_DTYPE;
  if (heads_q % cache->heads != 0) return NVFP4_ERR_SHAPE;
  st = check_sizes(heads_q, cache->heads, cache->page, tokens, batch, max_q, table_width);
  if (st != NVFP4_OK) return st;
  if (q_token < 0 || q_head < 0) return NVFP4_ERR_SHAPE;
  if (workspace_bytes < 0 || (workspace_bytes > 0 && !workspace)) return NVFP4_ERR_SHAPE;
  if (!cu_q && tokens != batch) return NVFP4_ERR_SHAPE;
  if (tokens == 0 || batch == 0 || heads_q == 0) return NVFP4_OK;
  if (max_q == 0) return NVFP4_ERR_SHAPE;   // new tokens, and none in any sequence
  st = check_sequences(cu_q, tokens, batch, table, table_width, lens);
  if (st != NVFP4_OK) return st;
  if (!q || !out) return NVFP4_ERR_NULLPTR;
  const int64_t size = dtype_size(dtype);
  if (!aligned(q, size) || !aligned(out, 16) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  if (!extent(tokens, heads_q, cache->dim, q_token, q_head, &nq) || !mul_ok(nq, size, &nq) ||
      !mul_ok(tokens * heads_q, cache->dim * size, &no))
    return NVFP4_ERR_SHAPE;
  if (overlaps(out, no, q, nq) || overlaps(out, no, cache->k, cache_bytes) || overlaps(out, no, cache->v, cache_bytes))
    return NVFP4_ERR_SHAPE;
  if (workspace && (overlaps(workspace, workspace_bytes, out, no) || overlaps(workspace, workspace_bytes, q, nq) ||
                    overlaps(workspace, workspace_bytes, cache->k, cache_bytes) ||
                    overlaps(workspace, workspace_bytes, cache->v, cache_bytes)))
    return NVFP4_ERR_SHAPE;
  if (nvfp4host::paged_attention_blocks(tokens, heads_q, cache->heads, cache->dim, cache->page, batch, max_q, table_width, window,
                                        dtype) > nvfp4host::kMaxGrid256)
    return NVFP4_ERR_GRID;
  nvfp4host::launch_paged_attention(*cache, q, q_token, q_head, heads_q, dtype, tokens, cu_q, batch, max_q, table,
                                    table_width, lens, window, scale, workspace, workspace_bytes, out, stream);
  return launched();
}

int64_t nvfp4_sample_workspace_size(int64_t batch, int64_t vocab, nvfp4_dtype_t dtype) {
  if (batch < 0 || vocab < 0 || vocab > kMaxPositions) return NVFP4_ERR_SHAPE;
  if (!valid_dtype(dtype)) return NVFP4_ERR_DTYPE;
  int64_t t;
  if (!mul_ok(batch, vocab, &t)) return NVFP4_ERR_SHAPE;
  if (batch == 0 || vocab == 0) return 0;
  return nvfp4host::sample_bytes(batch, vocab, dtype);
}

int nvfp4_sample(const void* logits, nvfp4_dtype_t dtype, int64_t batch, int64_t vocab, int64_t row_stride,
                 const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                 const float* min_p, void* workspace, int64_t workspace_bytes, int32_t* token, float* prob,
                 hipStream_t stream) {
  const int64_t need = nvfp4_sample_workspace_size(batch, vocab, dtype);
  if (need < 0) return (int)need;
  if (row_stride < vocab || workspace_bytes < 0 || (workspace_bytes > 0 && !workspace)) return NVFP4_ERR_SHAPE;
  if (batch == 0) return NVFP4_OK;
  if (vocab == 0) return NVFP4_ERR_SHAPE;   // rows without a token to choose
  const int64_t size = dtype_size(dtype);
  int64_t n;
  if (!mul_ok(batch, row_stride, &n) || !mul_ok(n, size, &n)) return NVFP4_ERR_SHAPE;
  if (!logits || !u || !token) return NVFP4_ERR_NULLPTR;
  if (!aligned(logits, size) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(token, 4) || !aligned(prob, 4) || !aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  if (batch > nvfp4host::kMaxGridY) return NVFP4_ERR_GRID;
  nvfp4host::launch_sample(logits, dtype, batch, vocab, row_stride, u, temperature, top_k, top_p, min_p, workspace,
                           workspace_bytes, token, prob, stream);
  return launched();
}

}  // extern "C"
