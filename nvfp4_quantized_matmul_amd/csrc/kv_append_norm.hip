// The append to the paged 8-bit cache with norms of the queries' and keys'
// heads before their rotation: x -> x / sqrt(mean(x^2) + eps) * weight over a
// head's channels.
//
// Blocks, scales, codes and rotation are those of the append without norms.
// The sum of squares, the root and both products are in 64 bits as well: the
// sum is good to 2^-46 and cannot leave the range, and a value is rounded to
// 32 bits once, behind its rotation.
//
// A head's row lies with a group of lanes that sum their squares among
// themselves, 8 channels a lane.  Sines and cosines are formed by all lanes
// together into LDS, in the order in which the rows' lanes read them, which
// keeps the code short: what a small call waits for is its instructions.
#include <algorithm>
#include <climits>

#include "kv_append.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

// Rounds of a page's keys that stay in registers between the two passes over
// it; what is over is formed twice.
constexpr int kHeld = 2;
// Rounds of queries that are loaded ahead.
constexpr int kAhead = 3;

// W = 4 or 1 consecutive elements as they are loaded.
template <typename T, int W>
struct Raw {
  typedef T V __attribute__((ext_vector_type(W)));
  V v;
  __device__ __forceinline__ void load(const T* p) { v = *(const V*)p; }
  __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
};

// 1 / sqrt(x).  The instruction is good to some 2^-23; with e = 1 - x y^2,
// 1 / sqrt(x) = y (1 - e)^(-1/2), whose sum up to e^2 is off by e^3 5 / 16.
__device__ __forceinline__ double inverse_root(double x) {
  const double y = __builtin_amdgcn_rsq(x);
  const double e = __builtin_fma(-(x * y), y, 1.0);
  const double r = __builtin_fma(y * e, __builtin_fma(e, 0.375, 0.5), y);
  return x > 0.0 && x < __builtin_inf() ? r : y;
}

template <int CTRL>
__device__ __forceinline__ double moved(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The sum over groups of 8, 16, 32 or 64 lanes; each of them gets it.  Lanes
// meet their neighbour, the other pair, the other four and the other eight
// (mirrored, which is one lane of them) in registers.
__device__ __forceinline__ double row_sum(double s, int lanes) {
  s += moved<0xb1>(s);      // lanes 1 0 3 2 of four
  s += moved<0x4e>(s);      // 2 3 0 1
  s += moved<0x141>(s);     // 7 .. 0 of eight
  if (lanes >= 16) s += moved<0x140>(s);   // 15 .. 0 of sixteen
  if (lanes >= 32) s += __shfl_xor(s, 16, 64);
  if (lanes >= 64) s += __shfl_xor(s, 32, 64);
  return s;
}

// A row's lanes: a group of a power of two of them, the first `units` with two
// groups of W channels each (of single channels with two times two, so that a
// row fits a wave).
template <typename T, int W, bool INTER>
struct Row {
  static constexpr int kItems = W == 1 ? 2 : 1;
  int units, lanes, lane, turning;   // turning: the items of a row that rotate
  int item[kItems], ca[kItems], cb[kItems];
  bool active;
  float w[kItems][2][W];     // the weights of the lane's channels

  static __device__ __host__ __forceinline__ int group(int dim) {
    const int units = dim / (2 * W * kItems);
    return units <= 8 ? 8 : units <= 16 ? 16 : units <= 32 ? 32 : 64;
  }
  __device__ __forceinline__ explicit Row(const AppendArgs& A) {
    units = A.dim / (2 * W * kItems);
    lanes = group(A.dim);
    lane = threadIdx.x & (lanes - 1);
    turning = A.rot / (2 * W);
    active = lane < units;
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
      item[r] = (active ? lane : 0) + r * units;   // lanes without items load others' and drop them
      item_channels<W, INTER>(item[r], A.rot, &ca[r], &cb[r]);
    }
  }
  // Without a branch around single loads, which would wait for one another.
  __device__ __forceinline__ void weights(const float* norm) {
#pragma unroll
    for (int r = 0; r < kItems; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        w[r][0][i] = norm ? norm[ca[r] + i] : 1.0f;
        w[r][1][i] = norm ? norm[cb[r] + i] : 1.0f;
      }
  }
};

template <typename T, int W>
struct RowData {
  static constexpr int kItems = W == 1 ? 2 : 1;
  Raw<T, W> a[kItems], b[kItems];
  template <bool INTER>
  __device__ __forceinline__ void load(const Row<T, W, INTER>& row, const T* p) {
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
      a[r].load(p + row.ca[r]);
      b[r].load(p + row.cb[r]);
    }
  }
};

// The row's values normed (or not) and rotated.  turn: sine and cosine of pair
// i of item j at [i * stride + j].
template <typename T, int W, bool INTER>
__device__ __forceinline__ void norm_row(const AppendArgs& A, const Row<T, W, INTER>& row, const RowData<T, W>& x, bool normed,
                                         const double2* turn, int stride, float (&a)[Row<T, W, INTER>::kItems][W],
                                         float (&b)[Row<T, W, INTER>::kItems][W]) {
  constexpr int ITEMS = Row<T, W, INTER>::kItems;
  double factor = 1.0;
  if (normed) {
    double s = 0.0;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s = __builtin_fma((double)x.a[r][i], (double)x.a[r][i], s);
        s = __builtin_fma((double)x.b[r][i], (double)x.b[r][i], s);
      }
    s = row.active ? s : 0.0;
    s = row_sum(s, row.lanes);
    factor = inverse_root(__builtin_fma(s, A.inv_dim, A.eps));
  }
  // channel i of group g
  const auto at = [&](int r, int g, int i) { return (double)(g ? x.b[r][i] : x.a[r][i]) * (factor * (double)row.w[r][g][i]); };
#pragma unroll
  for (int r = 0; r < ITEMS; ++r) {
    if (row.item[r] < row.turning) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int gx = INTER && 2 * i >= W, gy = !INTER || 2 * i + 1 >= W, ix = INTER ? 2 * i % W : i, iy = INTER ? (2 * i + 1) % W : i;
        const double2 t = turn[i * stride + row.item[r]];
        const double u = at(r, gx, ix), v = at(r, gy, iy);
        (gx ? b : a)[r][ix] = rounded(u * t.y - v * t.x);
        (gy ? b : a)[r][iy] = rounded(v * t.y + u * t.x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        a[r][i] = rounded(at(r, 0, i));
        b[r][i] = rounded(at(r, 1, i));
      }
    }
  }
}

template <typename T, int W, bool INTER, int THREADS>
__device__ void norm_keys(const AppendArgs& A, const T* k, const float* norm, uint8_t* codes, uint8_t* scale, int pos0,
                          int begin, int end, double2* turn, uint32_t* shared) {
  // k: the head's row of the token at position `begin`; codes: the page; pos0: its first position
  constexpr int ITEMS = Row<T, W, INTER>::kItems;
  Row<T, W, INTER> row(A);
  const int tokens = end - begin, each = THREADS / row.lanes, mine = threadIdx.x / row.lanes;   // each: tokens of a round
  const int old = *scale;
  // rows behind the last one are the last one again
  const auto load = [&](int t, RowData<T, W>& x) { x.load(row, k + (int64_t)(t < tokens ? t : tokens - 1) * A.k_token); };
  RowData<T, W> x[kHeld];
#pragma unroll
  for (int r = 0; r < kHeld; ++r) load(r * each + mine, x[r]);
  row.weights(norm);
  uint32_t top = 0;
  const auto value = [&](int t0, const RowData<T, W>& x, float (&a)[ITEMS][W], float (&b)[ITEMS][W]) {
    const int cells = each * row.turning;
    if (row.turning > 0) {
      __syncthreads();   // the round before has read
      for (int at = threadIdx.x; at < W * cells; at += THREADS) {
        const int i = at / cells, rest = at - i * cells, t = rest / row.turning, j = rest - t * row.turning;
        double sn, cs;
        sin_cos((double)(begin + t0 + t) * (double)A.inv_freq[W * j + i], &sn, &cs);
        turn[at] = make_double2(sn, cs);
      }
      __syncthreads();
    }
    norm_row<T, W, INTER>(A, row, x, norm != nullptr, turn + mine * row.turning, cells, a, b);
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t u = finite_bits(a[r][i]), w = finite_bits(b[r][i]);
        const uint32_t m = t0 + mine < tokens ? (u > w ? u : w) : 0u;
        top = m > top ? m : top;
      }
  };
  float a[kHeld][ITEMS][W], b[kHeld][ITEMS][W];
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r * each < tokens) value(r * each, x[r], a[r], b[r]);
  for (int t0 = kHeld * each; t0 < tokens; t0 += each) {
    load(t0 + mine, x[0]);
    float c[ITEMS][W], d[ITEMS][W];
    value(t0, x[0], c, d);
  }
  const int fresh = scale_byte(block_max<THREADS>(top, shared));
  const int held = begin - pos0;
  const int byte = held > 0 && old > fresh ? old : fresh;
  const int up = 127 - byte;
  const auto write = [&](int t, const float (&a)[ITEMS][W], const float (&b)[ITEMS][W]) {
    if (!row.active || t >= tokens) return;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) store_codes<W>(codes + (int64_t)(held + t) * A.dim, row.ca[r], row.cb[r], a[r], b[r], up);
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r * each < tokens) write(r * each + mine, a[r], b[r]);
  for (int t0 = kHeld * each; t0 < tokens; t0 += each) {
    load(t0 + mine, x[0]);
    value(t0, x[0], a[0], b[0]);
    write(t0 + mine, a[0], b[0]);
  }
  if (held > 0 && byte > old) recode_keys<THREADS>(codes, held * A.dim, old - byte);
  if (threadIdx.x == 0) *scale = (uint8_t)byte;   // every thread read `old` before the barrier in block_max
}

// A wave has the heads [part * q_heads, + q_heads) of a token.
template <typename T, int W, bool INTER, int THREADS>
__device__ void norm_queries(const AppendArgs& A, int64_t block, int q_heads, int q_parts, double2* turn) {
  constexpr int ITEMS = Row<T, W, INTER>::kItems;
  Row<T, W, INTER> row(A);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t unit = block * (THREADS / 64) + wave;
  const int64_t t = unit / q_parts;
  const int h0 = (int)(unit - t * q_parts) * q_heads, each = 64 / row.lanes, mine = lane / row.lanes;
  const int h1 = h0 + q_heads < A.heads_q ? h0 + q_heads : A.heads_q;
  const bool there = t < A.s.tokens;
  turn += wave * 128;   // half of a row of 256 channels
  RowData<T, W> x[kAhead];
  const T* q = (const T*)A.q + (there ? t : 0) * A.q_token;
  const auto load = [&](int h, RowData<T, W>& x) { x.load(row, q + (int64_t)(h < h1 ? h : h1 - 1) * A.q_head); };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(h0 + i * each + mine, x[i]);
  if (A.q_norm_head == 0) row.weights(A.q_norm);
  const int p = there ? row_position(A, (int)t) : kLeftOut;
  const double at = p < 0 ? 0 : p;
  for (int c = lane; c < A.rot / 2; c += 64) {
    const int i = c / row.turning, j = c - i * row.turning;
    double sn, cs;
    sin_cos(at * (double)A.inv_freq[W * j + i], &sn, &cs);
    turn[c] = make_double2(sn, cs);
  }
  __syncthreads();
  if (p == kLeftOut) return;
  for (int h = h0; h < h1; h += each) {
    if (A.q_norm_head != 0) row.weights(A.q_norm + (h + mine < h1 ? h + mine : h1 - 1) * A.q_norm_head);
    float a[ITEMS][W], b[ITEMS][W];
    norm_row<T, W, INTER>(A, row, x[0], A.q_norm != nullptr, turn, row.turning, a, b);
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) x[i] = x[i + 1];
    load(h + kAhead * each + mine, x[kAhead - 1]);
    if (row.active && h + mine < h1) {
      T* out = (T*)A.q_out + (t * A.heads_q + h + mine) * A.dim;
#pragma unroll
      for (int r = 0; r < ITEMS; ++r) {
        store_group<T, W>(out + row.ca[r], a[r]);
        store_group<T, W>(out + row.cb[r], b[r]);
      }
    }
  }
}

template <typename T, int W, bool INTER, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_append_kernel(AppendArgs A, int q_heads, int q_parts) {
  // rounds of keys: up to four pairs a lane; queries: up to 128 a wave
  __shared__ double2 turn[THREADS * 4];
  __shared__ uint32_t shared[THREADS / 64];
  const int64_t block = blockIdx.x;
  if (block >= A.kv_blocks) {
    norm_queries<T, W, INTER, THREADS>(A, block - A.kv_blocks, q_heads, q_parts, turn);
    return;
  }
  PagePart p;
  if (!page_part(A, block, &p)) return;
  const int64_t page_bytes = (int64_t)A.dim << A.c.page_shift;
  if (p.side == 0)
    norm_keys<T, W, INTER, THREADS>(A, (const T*)A.k + p.row * A.k_token + p.head * A.k_head,
                                    A.k_norm ? A.k_norm + p.head * A.k_norm_head : nullptr, A.c.k + p.ph * page_bytes,
                                    A.c.ks + p.ph, p.pos0, p.begin, p.end, turn, shared);
  else
    append_values<T, W == 1 ? 1 : 8, THREADS>(A, (const T*)A.v + p.row * A.v_token + p.head * A.v_head, A.c.v + p.ph * page_bytes,
                                 A.c.vs + p.ph, p.pos0, p.begin, p.end, shared);
}

// Few new tokens a sequence have few rows a page: blocks of one wave then, and
// a token's queries in parts of one round.
struct Plan {
  bool few;
  int64_t q_heads, q_parts, q_blocks;
};
template <int W>
Plan make_plan(int64_t dim, int64_t heads_q, int64_t tokens, int64_t max_q) {
  Plan p;
  const int lanes = Row<float, W, false>::group((int)dim);
  p.few = max_q * lanes <= 64 * kHeld;
  p.q_heads = p.few && tokens <= 256 ? 64 / lanes : heads_q;
  p.q_parts = heads_q ? (heads_q + p.q_heads - 1) / p.q_heads : 0;
  const int64_t units = tokens * p.q_parts;
  p.q_blocks = p.few ? units : (units + 3) / 4;
  return p;
}

template <typename T, int W, bool INTER>
void launch(const AppendArgs& A, int64_t max_q, hipStream_t s) {
  const Plan p = make_plan<W>(A.dim, A.heads_q, A.s.tokens, max_q);
  const dim3 grid((uint32_t)(A.kv_blocks + p.q_blocks));
  if (p.few) norm_append_kernel<T, W, INTER, 64><<<grid, dim3(64), 0, s>>>(A, (int)p.q_heads, (int)p.q_parts);
  else norm_append_kernel<T, W, INTER, 256><<<grid, dim3(256), 0, s>>>(A, (int)p.q_heads, (int)p.q_parts);
}

template <typename T>
void launch_type(const AppendArgs& A, bool vec, bool inter, int64_t max_q, hipStream_t s) {
  if (vec) inter ? launch<T, 4, true>(A, max_q, s) : launch<T, 4, false>(A, max_q, s);
  else inter ? launch<T, 1, true>(A, max_q, s) : launch<T, 1, false>(A, max_q, s);
}

}  // namespace

namespace nvfp4host {

int64_t kv_append_norm_q_blocks(int64_t dim, int64_t heads_q, int64_t tokens, int64_t max_q) {
  return std::max(make_plan<4>(dim, heads_q, tokens, max_q).q_blocks, make_plan<1>(dim, heads_q, tokens, max_q).q_blocks);
}

void launch_kv_append_norm(const nvfp4dev::AppendArgs& A, nvfp4_dtype_t dt, bool vec, bool inter, int64_t max_q, hipStream_t s) {
  switch (dt) {
    case NVFP4_F32: launch_type<float>(A, vec, inter, max_q, s); break;
    case NVFP4_BF16: launch_type<__bf16>(A, vec, inter, max_q, s); break;
    case NVFP4_F16: launch_type<_Float16>(A, vec, inter, max_q, s); break;
  }
}

}  // namespace nvfp4host
