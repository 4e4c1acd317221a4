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
// themselves, 8 channels of a key or 16 of a query a lane.  Sines and cosines
// are formed by all lanes together into LDS, which keeps the code short: what a
// small call waits for is its instructions, read once.
//
// Decode batch: bound by its chain of loads and 64-bit operations, 6.1 us in a
// graph (64 sequences, 32 + 2 x 8 heads of 128; 25 us in blocks of 256 threads
// with 16 channels a lane and angles formed by each, whose 190 registers left two
// waves a SIMD).  Prompts: bound by memory and, close behind, by the vector
// units' 64-bit operations.  Three ragged prompts of up to 4096 tokens, over four
// sets of inputs in turn: 32 + 2 x 8 heads of 128 in bf16 (183 MB) 49 us, 3.8
// TB/s; 42 + 2 x 6 heads (234 MB) 56; in f16 with a weight for each head and a
// rotation of 96 channels (272 MB) 79 us, 3.4 TB/s.  Over one set, which the
// last-level cache holds in part, 42, 50 and 71.
#include <algorithm>
#include <climits>

#include "kv_append.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

// Rounds of a page's keys that stay in registers between the two passes over
// it; what is over is formed twice.
constexpr int kHeld = 4;

// W = 8, 4 or 1 consecutive elements as they are loaded.
template <typename T, int W>
struct Raw {
  typedef T V __attribute__((ext_vector_type(W), aligned(W * sizeof(T) < 16 ? W * sizeof(T) : 16)));
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

// The sum over groups of 4, 8, 16, 32 or 64 lanes; each of them gets it.  Lanes
// meet their neighbour, the other pair, the other four and the other eight
// (mirrored, which is one lane of them) in registers.
__device__ __forceinline__ double row_sum(double s, int lanes) {
  s += moved<0xb1>(s);      // lanes 1 0 3 2 of four
  s += moved<0x4e>(s);      // 2 3 0 1
  if (lanes >= 8) s += moved<0x141>(s);    // 7 .. 0 of eight
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

  static __device__ __host__ __forceinline__ int group(int dim) {
    const int units = dim / (2 * W * kItems);
    return units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : units <= 32 ? 32 : 64;
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
};

// The weights of a lane's channels.
template <int W, int ITEMS>
struct Weights {
  float a[ITEMS][W], b[ITEMS][W];
  // (Loads behind a branch each would wait for one another.)
  template <typename R>
  __device__ __forceinline__ void load(const R& row, const float* norm) {
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        a[r][i] = norm[row.ca[r] + i];
        b[r][i] = norm[row.cb[r] + i];
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

// The row's values normed (or not) and rotated; turn(r, i): sine and cosine of
// pair i of the lane's item r.
template <typename T, int W, bool INTER, int ITEMS, typename TURN>
__device__ __forceinline__ void norm_row(const AppendArgs& A, const Row<T, W, INTER>& row, const RowData<T, W>& x,
                                         const Weights<W, ITEMS>& w, bool normed, const TURN& turn,
                                         float (&a)[ITEMS][W], float (&b)[ITEMS][W]) {
  double u[ITEMS][W], v[ITEMS][W];   // the groups' channels
#pragma unroll
  for (int r = 0; r < ITEMS; ++r)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      u[r][i] = (double)x.a[r][i];
      v[r][i] = (double)x.b[r][i];
    }
  if (normed) {
    double s = 0.0;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s = __builtin_fma(u[r][i], u[r][i], s);
        s = __builtin_fma(v[r][i], v[r][i], s);
      }
    const double factor = inverse_root(__builtin_fma(row_sum(row.active ? s : 0.0, row.lanes), A.inv_dim, A.eps));
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        u[r][i] *= factor * (double)w.a[r][i];
        v[r][i] *= factor * (double)w.b[r][i];
      }
  }
#pragma unroll
  for (int r = 0; r < ITEMS; ++r) {
    if (row.item[r] < row.turning) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        double& p = INTER && 2 * i >= W ? v[r][2 * i % W] : u[r][INTER ? 2 * i % W : i];
        double& q = !INTER || 2 * i + 1 >= W ? v[r][INTER ? (2 * i + 1) % W : i] : u[r][(2 * i + 1) % W];
        const double2 t = turn(r, i);
        const double p0 = p;
        p = p0 * t.y - q * t.x;
        q = q * t.y + p0 * t.x;
      }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a[r][i] = rounded(u[r][i]);
      b[r][i] = rounded(v[r][i]);
    }
  }
}

// The codes of finite values that are at most 448 at the scale.
template <int W, int ITEMS>
__device__ __forceinline__ void store_finite_codes(uint8_t* row, int c, const float (&x)[ITEMS][W], int r, int up) {
  if constexpr (W == 1) {
    row[c] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(x[r][0], up), 0.0f, 0, false);
  } else {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(x[r][0], up), __builtin_ldexpf(x[r][1], up), 0, false);
    *(int*)(row + c) = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(x[r][2], up), __builtin_ldexpf(x[r][3], up), lo, true);
  }
}

// Angles: the first round's sines and cosines are formed by all threads into
// LDS, and those of the step from a round to the next.  Each lane takes its
// pairs' into registers and turns them on from round to round, up to 63 times:
// that adds 2^-52 or so each time, since the step has sums of two more terms
// (with those of the first round, off by up to 4e-13, each turn would add that).
template <typename T, int W, bool INTER, int THREADS>
__device__ void norm_keys(const AppendArgs& A, const T* k, const float* norm, uint8_t* codes, uint8_t* scale, int pos0,
                          int begin, int end, double2* turn, double2* step, uint32_t* shared) {
  // k: the head's row of the token at position `begin`; codes: the page; pos0: its first position
  constexpr int ITEMS = Row<T, W, INTER>::kItems;
  Row<T, W, INTER> row(A);
  const int tokens = end - begin, each = THREADS / row.lanes, mine = threadIdx.x / row.lanes;   // each: tokens of a round
  const int half = A.rot / 2;
  const int old = *scale;
  // rows behind the last one are the last one again
  const auto load = [&](int t, RowData<T, W>& x) { x.load(row, k + (int64_t)(t < tokens ? t : tokens - 1) * A.k_token); };
  RowData<T, W> x[kHeld];
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r == 0 || r * each < tokens) load(r * each + mine, x[r]);
  Weights<W, ITEMS> weights;
  if (norm) weights.load(row, norm);

  for (int at = threadIdx.x; at < each * half; at += THREADS) {
    const int t = at / half, f = at - t * half;
    double sn, cs;
    sin_cos((double)(begin + t) * (double)A.inv_freq[f], &sn, &cs);
    turn[at] = make_double2(sn, cs);
  }
  if (each < tokens) {
    for (int f = threadIdx.x; f < half; f += THREADS) {
      double sn, cs;
      sin_cos<true>((double)each * (double)A.inv_freq[f], &sn, &cs);
      step[f] = make_double2(sn, cs);
    }
  }
  __syncthreads();
  double sn[ITEMS][W], cs[ITEMS][W];
  const auto first_angles = [&]() {
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const double2 d = row.item[r] < row.turning ? turn[mine * half + W * row.item[r] + i] : make_double2(0.0, 1.0);
        sn[r][i] = d.x;
        cs[r][i] = d.y;
      }
  };
  const auto turn_on = [&]() {
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (row.item[r] < row.turning) {
          const double2 d = step[W * row.item[r] + i];
          const double s = sn[r][i];
          sn[r][i] = s * d.y + cs[r][i] * d.x;
          cs[r][i] = cs[r][i] * d.y - s * d.x;
        }
      }
  };
  uint32_t top = 0;
  bool finite = true;      // all values of the lane's rows are
  const auto value = [&](int t0, const RowData<T, W>& x, float (&a)[ITEMS][W], float (&b)[ITEMS][W]) {
    norm_row<T, W, INTER>(A, row, x, weights, norm != nullptr, [&](int r, int i) { return make_double2(sn[r][i], cs[r][i]); }, a, b);
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) m = max(m, max(fbits(a[r][i]) & 0x7fffffffu, fbits(b[r][i]) & 0x7fffffffu));
    if (m >= 0x7f800000u) {
      finite = false;
      m = 0;
#pragma unroll
      for (int r = 0; r < ITEMS; ++r)
#pragma unroll
        for (int i = 0; i < W; ++i) m = max(m, max(finite_bits(a[r][i]), finite_bits(b[r][i])));
    }
    top = t0 + mine < tokens ? max(top, m) : top;
  };
  float a[kHeld][ITEMS][W], b[kHeld][ITEMS][W];
  first_angles();
#pragma unroll
  for (int r = 0; r < kHeld; ++r) {
    if (r * each < tokens) {
      if (r > 0) turn_on();
      value(r * each, x[r], a[r], b[r]);
    }
  }
  for (int t0 = kHeld * each; t0 < tokens; t0 += each) {
    float c[ITEMS][W], d[ITEMS][W];
    load(t0 + mine, x[0]);
    turn_on();
    value(t0, x[0], c, d);
  }
  const int fresh = scale_byte(block_max<THREADS>(top, shared));
  const int held = begin - pos0;
  const int byte = held > 0 && old > fresh ? old : fresh;
  const int up = 127 - byte;
  const auto write = [&](int t, const float (&a)[ITEMS][W], const float (&b)[ITEMS][W]) {
    if (!row.active || t >= tokens) return;
    uint8_t* to = codes + (int64_t)(held + t) * A.dim;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      if (finite) {
        store_finite_codes<W>(to, row.ca[r], a, r, up);
        store_finite_codes<W>(to, row.cb[r], b, r, up);
      } else {
        store_codes<W>(to, row.ca[r], row.cb[r], a[r], b[r], up);
      }
    }
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r * each < tokens) write(r * each + mine, a[r], b[r]);
  if (kHeld * each < tokens) {
    first_angles();
#pragma unroll 1
    for (int r = 1; r < kHeld; ++r) turn_on();
  }
  for (int t0 = kHeld * each; t0 < tokens; t0 += each) {
    load(t0 + mine, x[0]);
    turn_on();
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
  // a grid has less than 2^26 waves
  const uint32_t unit = (uint32_t)block * (THREADS / 64) + (uint32_t)wave, token = unit / (uint32_t)q_parts;
  const int64_t t = token;
  const int h0 = (int)(unit - token * (uint32_t)q_parts) * q_heads, each = 64 / row.lanes, mine = lane / row.lanes;
  const int h1 = h0 + q_heads < A.heads_q ? h0 + q_heads : A.heads_q;
  const bool there = t < A.s.tokens;
  turn += wave * 128;   // half of a row of 256 channels
  RowData<T, W> x;
  const T* q = (const T*)A.q + (there ? t : 0) * A.q_token;
  const auto load = [&](int h, RowData<T, W>& x) { x.load(row, q + (int64_t)(h < h1 ? h : h1 - 1) * A.q_head); };
  load(h0 + mine, x);
  const auto load_weights = [&](int h, Weights<W, ITEMS>& w) { w.load(row, A.q_norm + (h < h1 ? h : h1 - 1) * A.q_norm_head); };
  Weights<W, ITEMS> weights;
  if (A.q_norm) load_weights(h0 + mine, weights);
  const int p = there ? row_position(A, (int)t) : kLeftOut;
  const double at = p < 0 ? 0 : p;
  for (int f = lane; f < A.rot / 2; f += 64) {
    double sn, cs;
    sin_cos(at * (double)A.inv_freq[f], &sn, &cs);
    turn[f % W * row.turning + f / W] = make_double2(sn, cs);   // the lanes' pairs i side by side: no bank twice
  }
  // a wave reads what it wrote itself: in order, if the compiler keeps it
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  if (p == kLeftOut) return;
  for (int h = h0; h < h1; h += each) {
    float a[ITEMS][W], b[ITEMS][W];
    norm_row<T, W, INTER>(A, row, x, weights, A.q_norm != nullptr, [&](int r, int i) { return turn[i * row.turning + row.item[r]]; }, a, b);
    // the next round's, behind the last one that one's again
    load(h + each + mine, x);
    if (A.q_norm_head != 0) load_weights(h + each + mine, weights);
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
  __shared__ double2 turn[THREADS * 4], step[128];
  __shared__ uint32_t shared[THREADS / 64];
  const int64_t block = blockIdx.x;
  if (block >= A.kv_blocks) {
    norm_queries<T, W == 1 ? 1 : 8, INTER, THREADS>(A, block - A.kv_blocks, q_heads, q_parts, turn);
    return;
  }
  PagePart p;
  if (!page_part(A, block, &p)) return;
  const int64_t page_bytes = (int64_t)A.dim << A.c.page_shift;
  if (p.side == 0)
    norm_keys<T, W, INTER, THREADS>(A, (const T*)A.k + p.row * A.k_token + p.head * A.k_head,
                                    A.k_norm ? A.k_norm + p.head * A.k_norm_head : nullptr, A.c.k + p.ph * page_bytes,
                                    A.c.ks + p.ph, p.pos0, p.begin, p.end, turn, step, shared);
  else
    append_values<T, W == 1 ? 1 : 8, THREADS>(A, (const T*)A.v + p.row * A.v_token + p.head * A.v_head, A.c.v + p.ph * page_bytes,
                                 A.c.vs + p.ph, p.pos0, p.begin, p.end, shared);
}

// Blocks of 256 threads, or of one wave where the rows of a page that new
// tokens can fill are two rounds of it at most; then a token's queries go in
// parts of one round.  (Blocks of 512 threads hold pages of 16384 values for the
// second pass, where 256 form half of them again: three prompts of up to 4096
// tokens in pages of 128, 42 + 2 x 6 heads of 128, one set of inputs, 85 us with
// them and 80 without, in bf16 with shared weights 59 and 55, in float32 81 and 77.)
struct Plan {
  int threads;
  int64_t q_heads, q_parts, q_blocks;
};
template <int W>
Plan make_plan(int64_t page, int64_t dim, int64_t heads_q, int64_t tokens, int64_t max_q) {
  Plan p;
  const int lanes = Row<float, W, false>::group((int)dim);
  p.threads = (max_q < page ? max_q : page) * lanes <= 2 * 64 ? 64 : 256;
  p.q_heads = p.threads == 64 && tokens <= 256 ? 64 / Row<float, W == 1 ? 1 : 8, false>::group((int)dim) : heads_q;
  p.q_parts = heads_q ? (heads_q + p.q_heads - 1) / p.q_heads : 0;
  const int64_t waves = p.threads / 64;
  p.q_blocks = (tokens * p.q_parts + waves - 1) / waves;
  return p;
}

template <typename T, int W, bool INTER, int THREADS>
void launch_threads(const AppendArgs& A, const Plan& p, hipStream_t s) {
  norm_append_kernel<T, W, INTER, THREADS><<<dim3((uint32_t)(A.kv_blocks + p.q_blocks)), dim3(THREADS), 0, s>>>(A, (int)p.q_heads, (int)p.q_parts);
}

template <typename T, int W, bool INTER>
void launch(const AppendArgs& A, int64_t max_q, hipStream_t s) {
  const Plan p = make_plan<W>(1 << A.c.page_shift, A.dim, A.heads_q, A.s.tokens, max_q);
  if (p.threads == 64) launch_threads<T, W, INTER, 64>(A, p, s);
  else launch_threads<T, W, INTER, 256>(A, p, s);
}

template <typename T>
void launch_type(const AppendArgs& A, bool vec, bool inter, int64_t max_q, hipStream_t s) {
  if (vec) inter ? launch<T, 4, true>(A, max_q, s) : launch<T, 4, false>(A, max_q, s);
  else inter ? launch<T, 1, true>(A, max_q, s) : launch<T, 1, false>(A, max_q, s);
}

}  // namespace

namespace nvfp4host {

int64_t kv_append_norm_blocks(int64_t page_blocks, int64_t page, int64_t dim, int64_t heads_q, int64_t tokens, int64_t max_q) {
  const Plan a = make_plan<4>(page, dim, heads_q, tokens, max_q), b = make_plan<1>(page, dim, heads_q, tokens, max_q);
  return page_blocks + std::max(a.q_blocks, b.q_blocks);
}

void launch_kv_append_norm(const nvfp4dev::AppendArgs& A, nvfp4_dtype_t dt, bool vec, bool inter, int64_t max_q, hipStream_t s) {
  switch (dt) {
    case NVFP4_F32: launch_type<float>(A, vec, inter, max_q, s); break;
    case NVFP4_BF16: launch_type<__bf16>(A, vec, inter, max_q, s); break;
    case NVFP4_F16: launch_type<_Float16>(A, vec, inter, max_q, s); break;
  }
}

}  // namespace nvfp4host
