// New keys and values into the paged 8-bit cache, with the position rotation
// of keys and queries.
//
// One launch.  A block owns one side (keys or values) of one page and head
// that a sequence's new tokens reach, so that the page's scale -- the smallest
// power of two that holds the largest new value, or the present one if the
// page holds earlier tokens at a larger scale -- is one block's maximum and
// nothing is written twice.  The remaining blocks rotate queries.
//
// Rotation: (a, b) -> (a cos - b sin, b cos + a sin) with the angle position *
// inv_freq.  The product is formed in a double, where it is exact for positions
// below 2^29 (29 bits and a float's 24; behind, it is off by 2^-53 of itself);
// it is reduced and its sine and cosine formed there, since in 32 bits a
// position of 100000 would leave an angle with an error of 0.004.  The products
// are in 64 bits too, so each rotated value is rounded to 32 bits once (the
// sines' and cosines' error of up to 4e-13 moves that rounding in 1 of 10^5
// values at most) and the largest value of a page falls on the right side of a
// power of two.
//
// Bound by memory where there is much to do: three ragged prompts of up to 4096
// tokens, 42 + 2 x 6 heads of 128 (234 MB), take 61 us, 3.8 TB/s (in bf16 with
// split halves 47 us, 4.7 TB/s).  A decode step is a chain of dependent loads
// and 64-bit sums: 6 us for one sequence, 11 us for 64, 32 + 2 x 8 heads of 128.
#include <climits>

#include "kv_append.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

constexpr int kThreads = 256;
// Rotated items that a thread keeps between the two passes over a page (16
// values each): 4 hold a page of 16384 values, what is over is rotated twice.
constexpr int kHeld = 4;
// Tokens of a query block, and items that a thread loads before it turns them.
constexpr int kTokensWide = 4, kQueryItems = 3;

template <int W, bool INTER, typename CS>
__device__ __forceinline__ void rotate_item(float (&a)[W], float (&b)[W], const CS& cs_of) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    double sn, cs;
    cs_of(i, &sn, &cs);
    float& xr = INTER ? (2 * i < W ? a[(2 * i) % W] : b[(2 * i) % W]) : a[i];
    float& yr = INTER ? (2 * i + 1 < W ? a[(2 * i + 1) % W] : b[(2 * i + 1) % W]) : b[i];
    const double x = xr, y = yr;
    xr = rounded(x * cs - y * sn);
    yr = rounded(y * cs + x * sn);
  }
}

template <typename T, int W, bool INTER>
__device__ void append_keys(const AppendArgs& A, const T* k, uint8_t* codes, uint8_t* scale, int pos0, int begin,
                            int end, uint32_t* shared) {
  // k: the head's row of the token at position `begin`; codes: the page; pos0: its first position
  const int per = A.dim / (2 * W), items = (end - begin) * per, turning = A.rot / (2 * W);
  const int old = *scale;
  float xa[kHeld][W], xb[kHeld][W];

  auto value = [&](int it, float (&a)[W], float (&b)[W]) {
    const int t = it / per, j = it - t * per;
    int ca, cb;
    item_channels<W, INTER>(j, A.rot, &ca, &cb);
    const T* row = k + (int64_t)t * A.k_token;
    load_group<T, W>(row + ca, a);
    load_group<T, W>(row + cb, b);
    if (j < turning) {
      const double p = begin + t;
      rotate_item<W, INTER>(a, b, [&](int i, double* sn, double* cs) {
        sin_cos(p * (double)A.inv_freq[W * j + i], sn, cs);
      });
    }
  };
  uint32_t top = 0;
  auto largest = [&](const float (&a)[W], const float (&b)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t u = finite_bits(a[i]), w = finite_bits(b[i]);
      top = u > top ? u : top;
      top = w > top ? w : top;
    }
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r) {
    const int it = r * kThreads + threadIdx.x;
    if (it < items) {
      value(it, xa[r], xb[r]);
      largest(xa[r], xb[r]);
    }
  }
  for (int it = kHeld * kThreads + threadIdx.x; it < items; it += kThreads) {
    float a[W], b[W];
    value(it, a, b);
    largest(a, b);
  }
  const int fresh = scale_byte(block_max<kThreads>(top, shared));
  const int held = begin - pos0;
  const int byte = held > 0 && old > fresh ? old : fresh;
  const int up = 127 - byte;

  auto write = [&](int it, const float (&a)[W], const float (&b)[W]) {
    const int t = it / per, j = it - t * per;
    int ca, cb;
    item_channels<W, INTER>(j, A.rot, &ca, &cb);
    store_codes<W>(codes + (int64_t)(held + t) * A.dim, ca, cb, a, b, up);
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r) {
    const int it = r * kThreads + threadIdx.x;
    if (it < items) write(it, xa[r], xb[r]);
  }
  for (int it = kHeld * kThreads + threadIdx.x; it < items; it += kThreads) {
    float a[W], b[W];
    value(it, a, b);
    write(it, a, b);
  }
  if (held > 0 && byte > old) recode_keys<kThreads>(codes, held * A.dim, old - byte);
  if (threadIdx.x == 0) *scale = (uint8_t)byte;   // every thread read `old` before the barrier in block_max
}

template <typename T, int W, bool INTER>
__device__ void rotate_queries(const AppendArgs& A, int64_t block, double2* turn, int* pos) {
  // turn [q_tokens][rot / 2]: (sin, cos); pos [q_tokens]
  const int t0 = (int)block * A.q_tokens;
  const int n = A.s.tokens - t0 < A.q_tokens ? A.s.tokens - t0 : A.q_tokens;
  if ((int)threadIdx.x < n) pos[threadIdx.x] = row_position(A, t0 + threadIdx.x);
  __syncthreads();
  uint32_t left_out = 0;   // a bit per row
#pragma unroll
  for (int t = 0; t < kTokensWide; ++t) left_out |= t < n && pos[t] == kLeftOut ? 1u << t : 0u;
  left_out = __builtin_amdgcn_readfirstlane(left_out);
  const int half = A.rot / 2;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    double sn, cs;
    const int p = pos[t];
    sin_cos((double)(p < 0 ? 0 : p) * (double)A.inv_freq[f], &sn, &cs);
    turn[i] = make_double2(sn, cs);
  }
  __syncthreads();
  const int per = A.dim / (2 * W), turning = A.rot / (2 * W), row_items = A.heads_q * per;
  // rows [ta, tb), the loads of several items in flight at a time
  const auto rows = [&](int ta, int tb) {
    const int all = tb * row_items;
    for (int it0 = ta * row_items + threadIdx.x; it0 < all; it0 += kQueryItems * kThreads) {
      float a[kQueryItems][W], b[kQueryItems][W];
#pragma unroll
      for (int r = 0; r < kQueryItems; ++r) {
        const int it = it0 + r * kThreads;
        if (it < all) {
          const int t = it / row_items, rest = it - t * row_items, h = rest / per;
          int ca, cb;
          item_channels<W, INTER>(rest - h * per, A.rot, &ca, &cb);
          const T* row = (const T*)A.q + (int64_t)(t0 + t) * A.q_token + (int64_t)h * A.q_head;
          load_group<T, W>(row + ca, a[r]);
          load_group<T, W>(row + cb, b[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < kQueryItems; ++r) {
        const int it = it0 + r * kThreads;
        if (it < all) {
          const int t = it / row_items, rest = it - t * row_items, h = rest / per, j = rest - h * per;
          int ca, cb;
          item_channels<W, INTER>(j, A.rot, &ca, &cb);
          if (j < turning)
            rotate_item<W, INTER>(a[r], b[r], [&](int i, double* sn, double* cs) {
              const double2 d = turn[t * half + W * j + i];
              *sn = d.x;
              *cs = d.y;
            });
          T* out = (T*)A.q_out + ((int64_t)(t0 + t) * A.heads_q + h) * A.dim;
          store_group<T, W>(out + ca, a[r]);
          store_group<T, W>(out + cb, b[r]);
        }
      }
    }
  };
  if (!left_out) {
    rows(0, n);
  } else {
    for (int t = 0; t < n; ++t)
      if (!((left_out >> t) & 1)) rows(t, t + 1);
  }
}

template <typename T, int W, bool INTER>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs A) {
  __shared__ double2 turn[kTokensWide * 128];
  __shared__ uint32_t shared[kThreads / 64];
  const int64_t block = blockIdx.x;
  if (block >= A.kv_blocks) {
    rotate_queries<T, W, INTER>(A, block - A.kv_blocks, turn, (int*)shared);
    return;
  }
  PagePart p;
  if (!page_part(A, block, &p)) return;
  const int64_t page_bytes = (int64_t)A.dim << A.c.page_shift;
  if (p.side == 0)
    append_keys<T, W, INTER>(A, (const T*)A.k + p.row * A.k_token + p.head * A.k_head, A.c.k + p.ph * page_bytes,
                             A.c.ks + p.ph, p.pos0, p.begin, p.end, shared);
  else
    append_values<T, W, kThreads>(A, (const T*)A.v + p.row * A.v_token + p.head * A.v_head, A.c.v + p.ph * page_bytes,
                                  A.c.vs + p.ph, p.pos0, p.begin, p.end, shared);
}

template <typename T, int W>
void launch(const AppendArgs& A, bool inter, int64_t blocks, hipStream_t s) {
  if (inter) append_kernel<T, W, true><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(A);
  else append_kernel<T, W, false><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(A);
}

// Page slots that get a block a head and side.  A sequence of n new tokens
// touches at most ceil(n / page) + 1 pages, one more than they fill when they
// start inside one; so many for each sequence is little work for a block but
// many blocks where max_q is far above most sequences' tokens (or not known).
// Then sequence b has the slots from cu_q[b] / page + 2 b on, at least n / page
// + 2 of them, and blocks search the sequences for theirs: some dependent loads,
// taken when they spare more than half of the blocks.  (32 ragged prompts of
// 8192 tokens together, 8 heads of 128, pages of 16: 58 us searched; 60 us not,
// with the longest one's tokens as max_q, 239 us with all tokens.  16 of 256: 6.5
// us, and 7 and 9.)
struct Slots {
  int64_t all, each;   // each 0: searched
};
Slots page_slots(int64_t page, int64_t tokens, int64_t batch, int64_t max_q) {
  const int64_t each = (max_q + page - 1) / page + 1, packed = tokens / page + 2 * batch;
  if (batch * each > 2 * packed) return {packed, 0};
  return {batch * each, each};
}

int query_tokens(int64_t tokens) { return tokens > 1024 ? kTokensWide : 1; }

bool wide(const void* p, int64_t a, int64_t b, int64_t size) {
  return ((uintptr_t)p & 15) == 0 && (a * size) % 16 == 0 && (b * size) % 16 == 0;
}

}  // namespace

namespace nvfp4host {

int64_t kv_append_blocks(int64_t page, int64_t dim, int64_t heads, int64_t heads_q, int64_t tokens, int64_t batch,
                         int64_t max_q, bool norm) {
  int64_t n;
  if (__builtin_mul_overflow(page_slots(page, tokens, batch, max_q).all, heads * 2, &n)) return INT64_MAX;
  if (n > kMaxGrid256) return n;
  if (norm) return kv_append_norm_blocks(n, page, dim, heads_q, tokens, max_q);
  return n + (heads_q > 0 ? (tokens + query_tokens(tokens) - 1) / query_tokens(tokens) : 0);
}

void launch_kv_append(const nvfp4_kv_cache_t& c, const void* k, int64_t k_token, int64_t k_head, const void* v,
                      int64_t v_token, int64_t v_head, const void* q, int64_t q_token, int64_t q_head,
                      int64_t heads_q, void* q_out, nvfp4_dtype_t dt, int64_t tokens, const int32_t* cu,
                      int64_t batch, int64_t max_q, const int32_t* table, int64_t width, const int32_t* lens,
                      const float* inv_freq, int64_t rot, bool inter, const float* q_norm, int64_t q_norm_head,
                      const float* k_norm, int64_t k_norm_head, double eps, hipStream_t s) {
  AppendArgs A;
  A.c = {c.k, c.v, c.k_scales, c.v_scales, (int32_t)c.pages, (int32_t)c.heads, __builtin_ctz((unsigned)c.page)};
  A.s = {table, lens, cu, width, (int32_t)batch, (int32_t)tokens, (int32_t)max_q};
  A.k = k; A.v = v; A.q = q;
  A.k_token = k_token; A.k_head = k_head; A.v_token = v_token; A.v_head = v_head; A.q_token = q_token; A.q_head = q_head;
  A.q_out = q_out;
  A.inv_freq = inv_freq;
  A.q_norm = heads_q ? q_norm : nullptr; A.q_norm_head = A.q_norm ? q_norm_head : 0;
  A.k_norm = k_norm; A.k_norm_head = k_norm ? k_norm_head : 0;
  A.eps = eps; A.inv_dim = 1.0 / (double)c.dim;
  A.heads_q = (int32_t)heads_q; A.dim = (int32_t)c.dim; A.rot = (int32_t)rot;
  const Slots slots = page_slots(c.page, tokens, batch, max_q);
  A.slots = (int32_t)slots.each;
  A.kv_blocks = slots.all * c.heads * 2;
  A.q_tokens = query_tokens(tokens);
  // 16-byte accesses where every row and half of a rotated head starts on one
  const int64_t size = dt == NVFP4_F32 ? 4 : 2;
  const bool vec = rot % 16 == 0 && wide(k, k_token, k_head, size) && wide(v, v_token, v_head, size) &&
                   (!heads_q || wide(q, q_token, q_head, size));
  if (A.q_norm || k_norm) return launch_kv_append_norm(A, dt, vec, inter, max_q, s);
  const int64_t blocks = kv_append_blocks(c.page, c.dim, c.heads, heads_q, tokens, batch, max_q, false);
  switch (dt) {
    case NVFP4_F32: vec ? launch<float, 8>(A, inter, blocks, s) : launch<float, 1>(A, inter, blocks, s); break;
    case NVFP4_BF16: vec ? launch<__bf16, 8>(A, inter, blocks, s) : launch<__bf16, 1>(A, inter, blocks, s); break;
    case NVFP4_F16: vec ? launch<_Float16, 8>(A, inter, blocks, s) : launch<_Float16, 1>(A, inter, blocks, s); break;
  }
}

}  // namespace nvfp4host
