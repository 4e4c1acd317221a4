// New keys and values into the paged 8-bit cache, with the position rotation
// of keys and queries, and before it, if wanted, the norms of their heads.
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
// Norms: x -> x / sqrt(mean(x^2) + eps) * weight over a head's channels, in 64
// bits too: the sum of squares is exact to 2^-52 and cannot leave the range,
// and a value is rounded to 32 bits once, behind its rotation.
//
// Bound by memory where there is much to do: three ragged prompts of up to 4096
// tokens, 42 + 2 x 6 heads of 128 (234 MB), take 61 us, 3.8 TB/s (in bf16 with
// split halves 47 us, 4.7 TB/s).  A decode step is a chain of dependent loads
// and 64-bit sums: 6 us for one sequence, 11 us for 64, 32 + 2 x 8 heads of 128.
#include <climits>

#include "kv_cache.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

constexpr int kThreads = 256;
// Rotated items that a thread keeps between the two passes over a page (16
// values each): 4 hold a page of 16384 values, what is over is rotated twice.
constexpr int kHeld = 4;
// Tokens of a query block, and items that a thread loads before it turns them.
constexpr int kTokensWide = 4, kQueryItems = 3;

struct AppendArgs {
  CacheView c;
  SequenceView s;
  const void *k, *v, *q;
  int64_t k_token, k_head, v_token, v_head, q_token, q_head;
  void* q_out;
  const float* inv_freq;
  int64_t kv_blocks;
  int32_t heads_q, dim, rot, q_tokens;
  const float *q_norm, *k_norm;          // weights, or null
  int64_t q_norm_head, k_norm_head;      // from one head's to the next's
  double eps;
  int32_t slots;   // page slots of a sequence; 0: as the offsets tell
};

// sin and cos of x >= 0 (below 2^52): x minus the nearest multiple of pi/2 in
// two parts, then the Taylor sums to x^13 and x^12, whose first left-out terms
// are below 2.1e-14 and 4e-13 for |x| <= pi/4.
__device__ __forceinline__ void sin_cos(double x, double* sn, double* cs) {
  const double n = __builtin_rint(x * 0.63661977236758134308);
  double r = __builtin_fma(-n, 1.57079632679489661923, x);
  r = __builtin_fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double s = 1.0 / 6227020800.0;
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  s = __builtin_fma(s * z, r, r);
  double c = 1.0 / 479001600.0;
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  // the quadrant is n mod 4, taken in 64 bits: n passes 31 bits at far positions
  const int quad = (int)((int64_t)n & 3);
  const double a = quad & 1 ? c : s, b = quad & 1 ? s : c;
  *sn = quad & 2 ? -a : a;
  *cs = (quad == 1 || quad == 2) ? -b : b;
}

// W consecutive elements as floats; W = 8 reads 16 bytes at a time.
template <typename T, int W>
__device__ __forceinline__ void load_group(const T* p, float (&x)[W]) {
  if constexpr (W == 1) {
    x[0] = load_x(p);
  } else if constexpr (sizeof(T) == 4) {
    const f32x4_t lo = *(const f32x4_t*)p, hi = *((const f32x4_t*)p + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = lo[i]; x[4 + i] = hi[i]; }
  } else {
    typedef T vec8 __attribute__((ext_vector_type(8)));
    const vec8 u = *(const vec8*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)u[i];
  }
}

template <typename T, int W>
__device__ __forceinline__ void store_group(T* p, const float (&x)[W]) {
  if constexpr (W == 1) {
    store_out(p, x[0]);
  } else if constexpr (sizeof(T) == 4) {
    *(f32x4_t*)p = f32x4_t{x[0], x[1], x[2], x[3]};
    *((f32x4_t*)p + 1) = f32x4_t{x[4], x[5], x[6], x[7]};
  } else {
    typedef T vec8 __attribute__((ext_vector_type(8)));
    vec8 u;
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (T)x[i];
    *(vec8*)p = u;
  }
}

__device__ __forceinline__ bool finite(float x) { return (fbits(x) & 0x7f800000u) != 0x7f800000u; }

// The E4M3 code of x * 2^up (nearest, ties to even); NaN's code where x is not
// finite.  The product is at most 448 by the choice of the scale.
__device__ __forceinline__ uint32_t encode(float x, int up) {
  const uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(x, up), 0.0f, 0, false) & 0xffu;
  return finite(x) ? c : (((fbits(x) >> 24) & 0x80u) | 0x7fu);
}

// Four codes of one word rounded anew at a scale 2^down times as fine (down <
// 0); NaN codes stay.
__device__ __forceinline__ uint32_t recode(uint32_t w, int down) {
  uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(e4m3<0>(w), down), __builtin_ldexpf(e4m3<1>(w), down), 0, false);
  uint32_t r = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_ldexpf(e4m3<2>(w), down), __builtin_ldexpf(e4m3<3>(w), down), (int)lo, true);
  const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // bit 7 of each byte whose code is NaN
  const uint32_t keep = nan | (nan - (nan >> 7));                          // 0xff in those bytes
  return (r & ~keep) | (w & keep);
}

// An item is 2 W channels of one token: two groups of W.  The first rot / (2 W)
// items of a token rotate (pair i of the item has the frequency W * item + i),
// the rest are copied.  Split halves: the groups lie rot / 2 apart and pair
// up element by element.  Interleaved: the groups are neighbours and their 2 W
// channels pair up in turn.
template <int W, bool INTER>
__device__ __forceinline__ void item_channels(int item, int rot, int* ca, int* cb) {
  const int turning = rot / (2 * W);
  if (item < turning && !INTER) {
    *ca = W * item;
    *cb = rot / 2 + W * item;
  } else {
    *ca = 2 * W * item;
    *cb = *ca + W;
  }
}

// x rounded to 32 bits and no further: seen together with the rounding to a
// 2-byte type the compiler makes one of the two, by some 20 instructions.
__device__ __forceinline__ float rounded(double x) {
  float r = (float)x;
  asm("" : "+v"(r));
  return r;
}

// `of` makes a double of channel i of a group (0: a, 1: b) from what was loaded.
template <int W, bool INTER, typename OF, typename CS>
__device__ __forceinline__ void rotate_item(float (&a)[W], float (&b)[W], const OF& of, const CS& cs_of) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    double sn, cs;
    cs_of(i, &sn, &cs);
    const int gx = INTER && 2 * i >= W, gy = !INTER || 2 * i + 1 >= W, ix = INTER ? 2 * i % W : i, iy = INTER ? (2 * i + 1) % W : i;
    float& xr = gx ? b[ix] : a[ix];
    float& yr = gy ? b[iy] : a[iy];
    const double x = of(xr, gx, ix), y = of(yr, gy, iy);
    xr = rounded(x * cs - y * sn);
    yr = rounded(y * cs + x * sn);
  }
}

// Of channels without a norm.
struct Plain {
  __device__ __forceinline__ double operator()(float x, int, int) const { return x; }
};

// A head's row lies with a group of lanes, a power of two that holds its units;
// a lane has ITEMS items of the row (one of 16 channels; of two channels, of
// which a row has up to 128, two).
template <int W>
struct RowLanes {
  static constexpr int kItems = W == 1 ? 2 : 1;
  int units, lanes;   // lanes with items, and all of the group
  __device__ __forceinline__ explicit RowLanes(int dim) : units(dim / (2 * W * kItems)) {
    lanes = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : units <= 32 ? 32 : 64;
  }
};

// Sums of a row's lanes; each lane gets it.
__device__ __forceinline__ double row_sum(double v, int lanes) {
  for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// The items of a lane: their norm, and each rotated by cs_of(item, i) or not.
template <int W, int ITEMS>
struct Normed {
  float w[ITEMS][2][W];   // the weights of a head's channels, that the lane has
  __device__ __forceinline__ void weights(const float* norm, bool active, const int (&ca)[ITEMS], const int (&cb)[ITEMS]) {
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        w[r][0][i] = norm && active ? norm[ca[r] + i] : 1.0f;
        w[r][1][i] = norm && active ? norm[cb[r] + i] : 1.0f;
      }
  }
  static __device__ __forceinline__ double squares(const float (&a)[ITEMS][W], const float (&b)[ITEMS][W]) {
    double s = 0.0;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s = __builtin_fma((double)a[r][i], (double)a[r][i], s);
        s = __builtin_fma((double)b[r][i], (double)b[r][i], s);
      }
    return s;
  }
  template <bool INTER, typename CS>
  __device__ __forceinline__ void apply(float (&a)[ITEMS][W], float (&b)[ITEMS][W], double factor, const int (&item)[ITEMS],
                                        int turning, const CS& cs_of) const {
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      const auto of = [&](float x, int g, int i) { return (double)x * (factor * (double)w[r][g][i]); };
      if (item[r] < turning) {
        rotate_item<W, INTER>(a[r], b[r], of, [&](int i, double* sn, double* cs) { cs_of(item[r], i, sn, cs); });
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          a[r][i] = rounded(of(a[r][i], 0, i));
          b[r][i] = rounded(of(b[r][i], 1, i));
        }
      }
    }
  }
};

__device__ __forceinline__ double norm_factor(const AppendArgs& A, double squares) {
  return 1.0 / __builtin_sqrt(squares / A.dim + A.eps);
}

// The largest of all threads' values; every thread gets it.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* shared) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, off, 64);
    v = o > v ? o : v;
  }
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
  __syncthreads();
  v = shared[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) v = shared[w] > v ? shared[w] : v;
  return v;
}

__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t u = fbits(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

template <int W>
__device__ __forceinline__ void store_codes(uint8_t* row, int ca, int cb, const float (&a)[W], const float (&b)[W], int up) {
  if constexpr (W == 1) {
    row[ca] = (uint8_t)encode(a[0], up);
    row[cb] = (uint8_t)encode(b[0], up);
  } else {
    uint32_t wa[2] = {0, 0}, wb[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      wa[i / 4] |= encode(a[i], up) << (8 * (i % 4));
      wb[i / 4] |= encode(b[i], up) << (8 * (i % 4));
    }
    *(uint2*)(row + ca) = make_uint2(wa[0], wa[1]);
    *(uint2*)(row + cb) = make_uint2(wb[0], wb[1]);
  }
}

// The first n codes of a page of keys, rounded anew.
__device__ __forceinline__ void recode_keys(uint8_t* codes, int n, int down) {
  uint4* p = (uint4*)codes;
  for (int i = threadIdx.x; i < n / 16; i += kThreads) {
    uint4 w = p[i];
    w.x = recode(w.x, down);
    w.y = recode(w.y, down);
    w.z = recode(w.z, down);
    w.w = recode(w.w, down);
    p[i] = w;
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
      rotate_item<W, INTER>(a, b, Plain(), [&](int i, double* sn, double* cs) {
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
  const int fresh = scale_byte(block_max(top, shared));
  const int held = begin - pos0;
  const int byte = held > 0 && old > fresh ? old : fresh;
  const int up = 127 - byte;

  const auto write = [&](int it, const float (&a)[W], const float (&b)[W]) {
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
  if (held > 0 && byte > old) recode_keys(codes, held * A.dim, old - byte);
  if (threadIdx.x == 0) *scale = (uint8_t)byte;   // every thread read `old` before the barrier in block_max
}

// append_keys with the norm of each token's head: rows lie with groups of
// lanes, which sum their squares among themselves.
template <typename T, int W, bool INTER>
__device__ void append_normed_keys(const AppendArgs& A, const T* k, const float* norm, uint8_t* codes, uint8_t* scale,
                                   int pos0, int begin, int end, uint32_t* shared) {
  constexpr int ITEMS = RowLanes<W>::kItems;
  const RowLanes<W> row(A.dim);
  const int tokens = end - begin, turning = A.rot / (2 * W), each = kThreads / row.lanes;   // tokens of a round
  const int mine = threadIdx.x / row.lanes, lane = threadIdx.x % row.lanes;
  const bool active = lane < row.units;
  const int old = *scale;
  int item[ITEMS], ca[ITEMS], cb[ITEMS];
#pragma unroll
  for (int r = 0; r < ITEMS; ++r) {
    item[r] = lane + r * row.units;
    item_channels<W, INTER>(item[r], A.rot, &ca[r], &cb[r]);
  }
  Normed<W, ITEMS> n;
  n.weights(norm, active, ca, cb);
  const auto load = [&](int t, float (&a)[ITEMS][W], float (&b)[ITEMS][W]) {
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      if (active && t < tokens) {
        load_group<T, W>(k + (int64_t)t * A.k_token + ca[r], a[r]);
        load_group<T, W>(k + (int64_t)t * A.k_token + cb[r], b[r]);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) a[r][i] = b[r][i] = 0.0f;
      }
    }
  };
  uint32_t top = 0;
  const auto value = [&](int t, float (&a)[ITEMS][W], float (&b)[ITEMS][W]) {
    const double squares = row_sum(n.squares(a, b), row.lanes);
    if (!active || t >= tokens) return;
    const double p = begin + t;
    n.template apply<INTER>(a, b, norm ? norm_factor(A, squares) : 1.0, item, turning, [&](int j, int i, double* sn, double* cs) {
      sin_cos(p * (double)A.inv_freq[W * j + i], sn, cs);
    });
#pragma unroll
    for (int r = 0; r < ITEMS; ++r)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t u = finite_bits(a[r][i]), w = finite_bits(b[r][i]);
        top = u > top ? u : top;
        top = w > top ? w : top;
      }
  };
  float xa[kHeld][ITEMS][W], xb[kHeld][ITEMS][W];
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r * each < tokens) load(r * each + mine, xa[r], xb[r]);
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r * each < tokens) value(r * each + mine, xa[r], xb[r]);
  for (int t0 = kHeld * each; t0 < tokens; t0 += each) {
    float a[ITEMS][W], b[ITEMS][W];
    load(t0 + mine, a, b);
    value(t0 + mine, a, b);
  }
  const int fresh = scale_byte(block_max(top, shared));
  const int held = begin - pos0;
  const int byte = held > 0 && old > fresh ? old : fresh;
  const int up = 127 - byte;
  const auto write = [&](int t, const float (&a)[ITEMS][W], const float (&b)[ITEMS][W]) {
    if (!active || t >= tokens) return;
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) store_codes<W>(codes + (int64_t)(held + t) * A.dim, ca[r], cb[r], a[r], b[r], up);
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r * each < tokens) write(r * each + mine, xa[r], xb[r]);
  for (int t0 = kHeld * each; t0 < tokens; t0 += each) {
    float a[ITEMS][W], b[ITEMS][W];
    load(t0 + mine, a, b);
    value(t0 + mine, a, b);
    write(t0 + mine, a, b);
  }
  if (held > 0 && byte > old) recode_keys(codes, held * A.dim, old - byte);
  if (threadIdx.x == 0) *scale = (uint8_t)byte;
}

// Values lie with a channel's tokens side by side: a thread takes four tokens
// (one word of codes) of W channels.  The rows are read again for the second
// pass: they come from the L2, and nothing has to be computed anew.
template <typename T, int W>
__device__ void append_values(const AppendArgs& A, const T* v, uint8_t* codes, uint8_t* scale, int pos0, int begin,
                              int end, uint32_t* shared) {
  const int page = 1 << A.c.page_shift, held = begin - pos0, stop = end - pos0;
  const int groups = A.dim / W, quad0 = held / 4, items = ((stop + 3) / 4 - quad0) * groups;
  const int old = *scale;
  uint32_t top = 0;
  for (int it = threadIdx.x; it < items; it += kThreads) {
    const int qd = quad0 + it / groups, g = it % groups;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * qd + i;
      if (t >= held && t < stop) {
        float x[W];
        load_group<T, W>(v + (int64_t)(t - held) * A.v_token + g * W, x);
#pragma unroll
        for (int c = 0; c < W; ++c) {
          const uint32_t u = finite_bits(x[c]);
          top = u > top ? u : top;
        }
      }
    }
  }
  const int fresh = scale_byte(block_max(top, shared));
  const int byte = held > 0 && old > fresh ? old : fresh;
  const int up = 127 - byte;
  for (int it = threadIdx.x; it < items; it += kThreads) {
    const int qd = quad0 + it / groups, g = it % groups;
    uint32_t w[W];
#pragma unroll
    for (int c = 0; c < W; ++c) w[c] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * qd + i;
      if (t >= held && t < stop) {
        float x[W];
        load_group<T, W>(v + (int64_t)(t - held) * A.v_token + g * W, x);
#pragma unroll
        for (int c = 0; c < W; ++c) w[c] |= encode(x[c], up) << (8 * i);
      }
    }
    uint8_t* at = codes + (int64_t)g * W * page + 4 * qd;
    if (4 * qd >= held && 4 * qd + 4 <= stop) {
#pragma unroll
      for (int c = 0; c < W; ++c) *(uint32_t*)(at + c * page) = w[c];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * qd + i;
        if (t >= held && t < stop) {
#pragma unroll
          for (int c = 0; c < W; ++c) at[c * page + i] = (uint8_t)(w[c] >> (8 * i));
        }
      }
    }
  }
  if (held > 0 && byte > old) {
    // earlier tokens' codes; the last word may hold new ones, written above
    // by other threads, so its bytes go one by one
    const int quads = (held + 3) / 4;
    for (int it = threadIdx.x; it < quads * A.dim; it += kThreads) {
      const int c = it / quads, qd = it - c * quads;
      uint8_t* at = codes + (int64_t)c * page + 4 * qd;
      if (4 * qd + 4 <= held) {
        *(uint32_t*)at = recode(*(const uint32_t*)at, old - byte);
      } else {
        for (int t = 4 * qd; t < held; ++t) at[t - 4 * qd] = (uint8_t)recode(at[t - 4 * qd], old - byte);
      }
    }
  }
  if (threadIdx.x == 0) *scale = (uint8_t)byte;
}

// In place of a position (of a row past the tokens that the call takes).
constexpr int kLeftOut = INT_MIN;

// The n tokens from t0 on: a head's row lies with a group of lanes.
template <typename T, int W, bool INTER>
__device__ __forceinline__ void norm_queries(const AppendArgs& A, int t0, int n, uint32_t left_out, const double2* turn) {
  constexpr int ITEMS = RowLanes<W>::kItems;
  const RowLanes<W> row(A.dim);
  const int turning = A.rot / (2 * W), half = A.rot / 2, rows = n * A.heads_q, each = kThreads / row.lanes;
  const int mine = threadIdx.x / row.lanes, lane = threadIdx.x % row.lanes;
  int item[ITEMS], ca[ITEMS], cb[ITEMS];
#pragma unroll
  for (int r = 0; r < ITEMS; ++r) {
    item[r] = lane + r * row.units;
    item_channels<W, INTER>(item[r], A.rot, &ca[r], &cb[r]);
  }
  Normed<W, ITEMS> norm;
  if (A.q_norm_head == 0) norm.weights(A.q_norm, lane < row.units, ca, cb);
  for (int row0 = 0; row0 < rows; row0 += kQueryItems * each) {
    float a[kQueryItems][ITEMS][W], b[kQueryItems][ITEMS][W];
#pragma unroll
    for (int s = 0; s < kQueryItems; ++s) {
      const int at = row0 + s * each + mine, t = at / A.heads_q, h = at - t * A.heads_q;
      const bool active = lane < row.units && at < rows && !((left_out >> t) & 1);
      const T* p = (const T*)A.q + (int64_t)(t0 + t) * A.q_token + (int64_t)h * A.q_head;
#pragma unroll
      for (int r = 0; r < ITEMS; ++r) {
        if (active) {
          load_group<T, W>(p + ca[r], a[s][r]);
          load_group<T, W>(p + cb[r], b[s][r]);
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i) a[s][r][i] = b[s][r][i] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int s = 0; s < kQueryItems; ++s) {
      const int at = row0 + s * each + mine, t = at / A.heads_q, h = at - t * A.heads_q;
      const bool active = lane < row.units && at < rows && !((left_out >> t) & 1);
      const double squares = row_sum(norm.squares(a[s], b[s]), row.lanes);
      if (!active) continue;
      if (A.q_norm_head != 0) norm.weights(A.q_norm + h * A.q_norm_head, true, ca, cb);
      norm.template apply<INTER>(a[s], b[s], A.q_norm ? norm_factor(A, squares) : 1.0, item, turning,
                                 [&](int j, int i, double* sn, double* cs) {
                                   const double2 d = turn[t * half + W * j + i];
                                   *sn = d.x;
                                   *cs = d.y;
                                 });
      T* out = (T*)A.q_out + ((int64_t)(t0 + t) * A.heads_q + h) * A.dim;
#pragma unroll
      for (int r = 0; r < ITEMS; ++r) {
        store_group<T, W>(out + ca[r], a[s][r]);
        store_group<T, W>(out + cb[r], b[s][r]);
      }
    }
  }
}

template <typename T, int W, bool INTER, bool NORM>
__device__ void rotate_queries(const AppendArgs& A, int64_t block, double2* turn, int* pos) {
  // turn [q_tokens][rot / 2]: (sin, cos); pos [q_tokens]
  const int t0 = (int)block * A.q_tokens;
  const int n = A.s.tokens - t0 < A.q_tokens ? A.s.tokens - t0 : A.q_tokens;
  if ((int)threadIdx.x < n) {
    const int t = t0 + threadIdx.x;
    int b = t;
    if (A.s.cu) {
      // the last sequence that starts at or before row t
      int lo = 0, hi = A.s.batch;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (A.s.cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
      }
      b = lo;
    }
    int p = 0;   // rows of no sequence are copied unturned
    if (b < A.s.batch) {
      const Sequence s = sequence(A.s, b);
      p = t - s.row0 < s.count ? s.first + (t - s.row0) : kLeftOut;
    }
    pos[threadIdx.x] = p;
  }
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
  if constexpr (NORM) {
    norm_queries<T, W, INTER>(A, t0, n, left_out, turn);
    return;
  }
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
            rotate_item<W, INTER>(a[r], b[r], Plain(), [&](int i, double* sn, double* cs) {
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

template <typename T, int W, bool INTER, bool NORM>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs A) {
  __shared__ double2 turn[kTokensWide * 128];
  __shared__ uint32_t shared[kThreads / 64];
  int64_t block = blockIdx.x;
  if (block >= A.kv_blocks) {
    rotate_queries<T, W, INTER, NORM>(A, block - A.kv_blocks, turn, (int*)shared);
    return;
  }
  const int side = (int)(block & 1);
  block >>= 1;
  const int h = (int)(block % A.c.heads);
  block /= A.c.heads;
  int b, slot;
  if (A.slots > 0) {
    slot = (int)(block % A.slots);
    b = (int)(block / A.slots);
  } else {
    // the last sequence whose slots start at or before this one
    const auto start = [&](int i) { return (sequence_row(A.s, i) >> A.c.page_shift) + 2 * i; };
    int lo = 0, hi = A.s.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start(mid) <= (int)block) lo = mid; else hi = mid - 1;
    }
    b = lo;
    slot = (int)block - start(b);
    if (slot < 0) return;
  }
  const Sequence s = sequence(A.s, b);
  const int first = s.first, stop = s.first + s.count, from = first < 0 ? 0 : first;
  const int64_t pi = (int64_t)(from >> A.c.page_shift) + slot;
  const int64_t page0 = pi << A.c.page_shift;
  if (pi >= A.s.width || page0 >= stop) return;
  const int pos0 = (int)page0, page = 1 << A.c.page_shift;
  const int begin = from > pos0 ? from : pos0;
  const int end = stop - pos0 < page ? stop : pos0 + page;
  const int id = A.s.table[(int64_t)b * A.s.width + pi];
  if (begin >= end || id < 0 || id >= A.c.pages) return;
  const int64_t ph = (int64_t)id * A.c.heads + h;
  const int64_t row = s.row0 + (begin - first), page_bytes = (int64_t)A.dim << A.c.page_shift;
  const T* k = (const T*)A.k + row * A.k_token + h * A.k_head;
  if (side == 0 && NORM)
    append_normed_keys<T, W, INTER>(A, k, A.k_norm ? A.k_norm + h * A.k_norm_head : nullptr, A.c.k + ph * page_bytes,
                                    A.c.ks + ph, pos0, begin, end, shared);
  else if (side == 0)
    append_keys<T, W, INTER>(A, k, A.c.k + ph * page_bytes, A.c.ks + ph, pos0, begin, end, shared);
  else
    append_values<T, W>(A, (const T*)A.v + row * A.v_token + h * A.v_head, A.c.v + ph * page_bytes, A.c.vs + ph, pos0,
                        begin, end, shared);
}

template <typename T, int W, bool NORM>
void launch_order(const AppendArgs& A, bool inter, int64_t blocks, hipStream_t s) {
  if (inter) append_kernel<T, W, true, NORM><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(A);
  else append_kernel<T, W, false, NORM><<<dim3((uint32_t)blocks), dim3(kThreads), 0, s>>>(A);
}

template <typename T, int W>
void launch(const AppendArgs& A, bool inter, int64_t blocks, hipStream_t s) {
  if (A.q_norm || A.k_norm) launch_order<T, W, true>(A, inter, blocks, s);
  else launch_order<T, W, false>(A, inter, blocks, s);
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

int64_t kv_append_blocks(int64_t page, int64_t heads, int64_t heads_q, int64_t tokens, int64_t batch, int64_t max_q) {
  int64_t n;
  if (__builtin_mul_overflow(page_slots(page, tokens, batch, max_q).all, heads * 2, &n)) return INT64_MAX;
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
  A.eps = eps;
  A.heads_q = (int32_t)heads_q; A.dim = (int32_t)c.dim; A.rot = (int32_t)rot;
  const Slots slots = page_slots(c.page, tokens, batch, max_q);
  A.slots = (int32_t)slots.each;
  A.kv_blocks = slots.all * c.heads * 2;
  A.q_tokens = query_tokens(tokens);
  const int64_t blocks = kv_append_blocks(c.page, c.heads, heads_q, tokens, batch, max_q);
  // 16-byte accesses where every row and half of a rotated head starts on one
  const int64_t size = dt == NVFP4_F32 ? 4 : 2;
  const bool vec = rot % 16 == 0 && wide(k, k_token, k_head, size) && wide(v, v_token, v_head, size) &&
                   (!heads_q || wide(q, q_token, q_head, size));
  switch (dt) {
    case NVFP4_F32: vec ? launch<float, 8>(A, inter, blocks, s) : launch<float, 1>(A, inter, blocks, s); break;
    case NVFP4_BF16: vec ? launch<__bf16, 8>(A, inter, blocks, s) : launch<__bf16, 1>(A, inter, blocks, s); break;
    case NVFP4_F16: vec ? launch<_Float16, 8>(A, inter, blocks, s) : launch<_Float16, 1>(A, inter, blocks, s); break;
  }
}

}  // namespace nvfp4host
