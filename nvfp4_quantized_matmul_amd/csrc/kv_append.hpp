// What the appends to the paged 8-bit cache share: codes, angles, values, and
// which page a block has.
#pragma once

#include <climits>

#include "kv_cache.hpp"
#include "nvfp4.h"

namespace nvfp4dev {

struct AppendArgs {
  CacheView c;
  SequenceView s;
  const void *k, *v, *q;
  int64_t k_token, k_head, v_token, v_head, q_token, q_head;
  void* q_out;
  const float* inv_freq;
  int64_t kv_blocks;
  int32_t heads_q, dim, rot, q_tokens;
  const float *q_norm, *k_norm;          // weights of the heads' norms, or null
  int64_t q_norm_head, k_norm_head;      // from one head's to the next's
  double eps, inv_dim;
  int32_t slots;   // page slots of a sequence; 0: as the offsets tell
};

// sin and cos of x >= 0 (below 2^52): x minus the nearest multiple of pi/2 in
// two parts, then the Taylor sums to x^13 and x^12, whose first left-out terms
// are below 2.1e-14 and 4e-13 for |x| <= pi/4; FINE: to x^15 and x^16, and
// below 5e-17 and 3e-18.
template <bool FINE = false>
__device__ __forceinline__ void sin_cos(double x, double* sn, double* cs) {
  const double n = __builtin_rint(x * 0.63661977236758134308);
  double r = __builtin_fma(-n, 1.57079632679489661923, x);
  r = __builtin_fma(-n, 6.12323399573676603587e-17, r);
  const double z = r * r;
  double s = 1.0 / 6227020800.0;
  if constexpr (FINE) s = __builtin_fma(-1.0 / 1307674368000.0, z, s);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  s = __builtin_fma(s * z, r, r);
  double c = 1.0 / 479001600.0;
  if constexpr (FINE) c = __builtin_fma(__builtin_fma(1.0 / 20922789888000.0, z, -1.0 / 87178291200.0), z, c);
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
#pragma unroll
    for (int i = 0; i < W; i += 4) *(f32x4_t*)(p + i) = f32x4_t{x[i], x[i + 1], x[i + 2], x[i + 3]};
  } else {
    typedef T vec __attribute__((ext_vector_type(W)));
    vec u;
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = (T)x[i];
    *(vec*)p = u;
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

// The largest of all threads' values; every thread gets it.
template <int THREADS>
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
  for (int w = 1; w < THREADS / 64; ++w) v = shared[w] > v ? shared[w] : v;
  return v;
}

__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t u = fbits(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// A row's codes of an item.
template <int W>
__device__ __forceinline__ void store_codes(uint8_t* row, int ca, int cb, const float (&a)[W], const float (&b)[W], int up) {
  if constexpr (W == 1) {
    row[ca] = (uint8_t)encode(a[0], up);
    row[cb] = (uint8_t)encode(b[0], up);
  } else {
    uint32_t wa[W / 4] = {}, wb[W / 4] = {};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      wa[i / 4] |= encode(a[i], up) << (8 * (i % 4));
      wb[i / 4] |= encode(b[i], up) << (8 * (i % 4));
    }
    if constexpr (W == 4) {
      *(uint32_t*)(row + ca) = wa[0];
      *(uint32_t*)(row + cb) = wb[0];
    } else {
      *(uint2*)(row + ca) = make_uint2(wa[0], wa[1]);
      *(uint2*)(row + cb) = make_uint2(wb[0], wb[1]);
    }
  }
}

// The first n codes of a page of keys, rounded anew.
template <int THREADS>
__device__ __forceinline__ void recode_keys(uint8_t* codes, int n, int down) {
  uint4* p = (uint4*)codes;
  for (int i = threadIdx.x; i < n / 16; i += THREADS) {
    uint4 w = p[i];
    w.x = recode(w.x, down);
    w.y = recode(w.y, down);
    w.z = recode(w.z, down);
    w.w = recode(w.w, down);
    p[i] = w;
  }
}

// Values lie with a channel's tokens side by side: a thread takes four tokens
// (one word of codes) of W channels.  The rows are read again for the second
// pass: they come from the L2, and nothing has to be computed anew.
template <typename T, int W, int THREADS>
__device__ void append_values(const AppendArgs& A, const T* v, uint8_t* codes, uint8_t* scale, int pos0, int begin,
                              int end, uint32_t* shared) {
  const int page = 1 << A.c.page_shift, held = begin - pos0, stop = end - pos0;
  const int groups = A.dim / W, quad0 = held / 4, items = ((stop + 3) / 4 - quad0) * groups;
  const int old = *scale;
  uint32_t top = 0;
  for (int it = threadIdx.x; it < items; it += THREADS) {
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
  const int fresh = scale_byte(block_max<THREADS>(top, shared));
  const int byte = held > 0 && old > fresh ? old : fresh;
  const int up = 127 - byte;
  for (int it = threadIdx.x; it < items; it += THREADS) {
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
    for (int it = threadIdx.x; it < quads * A.dim; it += THREADS) {
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

// What a block of one side of one page and head has to do.
struct PagePart {
  int side, head;
  int pos0, begin, end;      // the page's first position, those of the new tokens in it
  int64_t row, ph;           // the row of the first of them; index of page and head
};

// False: nothing.
__device__ __forceinline__ bool page_part(const AppendArgs& A, int64_t block, PagePart* r) {
  r->side = (int)(block & 1);
  block >>= 1;
  r->head = (int)(block % A.c.heads);
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
    if (slot < 0) return false;
  }
  const Sequence s = sequence(A.s, b);
  const int first = s.first, stop = s.first + s.count, from = first < 0 ? 0 : first;
  const int64_t pi = (int64_t)(from >> A.c.page_shift) + slot;
  const int64_t page0 = pi << A.c.page_shift;
  if (pi >= A.s.width || page0 >= stop) return false;
  const int page = 1 << A.c.page_shift;
  r->pos0 = (int)page0;
  r->begin = from > r->pos0 ? from : r->pos0;
  r->end = stop - r->pos0 < page ? stop : r->pos0 + page;
  const int id = A.s.table[(int64_t)b * A.s.width + pi];
  if (r->begin >= r->end || id < 0 || id >= A.c.pages) return false;
  r->ph = (int64_t)id * A.c.heads + r->head;
  r->row = s.row0 + (r->begin - first);
  return true;
}

// The position of row t among the new tokens; 0 for rows of no sequence, which
// are copied unturned.
__device__ __forceinline__ int row_position(const AppendArgs& A, int t) {
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
  if (b >= A.s.batch) return 0;
  const Sequence s = sequence(A.s, b);
  return t - s.row0 < s.count ? s.first + (t - s.row0) : kLeftOut;
}

}  // namespace nvfp4dev

namespace nvfp4host {

// The append with norms; `vec`: 16-byte accesses of q, k and v.  _blocks: its
// grid, with page_blocks for the pages.
int64_t kv_append_norm_blocks(int64_t page_blocks, int64_t page, int64_t dim, int64_t heads_q, int64_t tokens, int64_t max_q);
void launch_kv_append_norm(const nvfp4dev::AppendArgs& A, nvfp4_dtype_t dt, bool vec, bool inter, int64_t max_q, hipStream_t s);

}  // namespace nvfp4host
