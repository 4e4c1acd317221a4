// Attention of new tokens over the paged 8-bit key/value cache: out =
// softmax(scale q K^T) V, one pass over the cache with a running maximum and
// sum per query row.
//
// Both products run transposed on the matrix cores, S^T = K Q^T and O^T = V^T
// P^T, with a query row per column.  A lane then holds scores of one row only,
// so the running maximum is the lane's own; and its scores are consecutive
// tokens of that row, the very operand that the second product takes, if the
// 16 key rows of a multiply are taken in the right order.  Weights never leave
// their registers.  An E4M3 code is exact in bf16 and f16, so codes are
// converted in registers and multiply 2-byte queries; float32 queries and
// weights multiply as three bf16 parts whose sum is the float.
//
// Scales.  Keys: the score of a token is multiplied by its page's power of
// two.  Values: with s the score in powers of two and e the exponent of the
// value scale, the weight in units of codes is 2^(s + e), so the running
// maximum m is that of s + e, weights are 2^(s + e - r) against a reference r
// that follows m, and the sum of the softmax takes each of them times 2^-e.
//
// What a row does not see gets s = -inf.  A NaN code among its values would
// still spoil the product, as 0 * NaN: a tile that is not seen whole by all
// rows is searched for them, and one that holds any takes a separate path.
#include <algorithm>
#include <climits>

#include "kv_cache.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

constexpr float kLog2e = 1.44269504088896340736f;

struct AttnArgs {
  CacheView c;
  SequenceView s;
  const void* q;
  int64_t q_token, q_head;
  void* out;
  float *part_o, *part_m, *part_l;   // of a split axis: [tokens * heads_q][splits][dim], twice [tokens * heads_q][splits]
  int32_t heads_q, group;
  int32_t window;                    // <= 0: none
  int32_t sinks;                     // first tokens that are seen through any window
  int32_t splits, chunk;             // chunk: tokens of a split, a multiple of 64
  int32_t row_tiles;                 // of a sequence and head, at most
  float scale_log2;                  // |scale| * log2(e)
  float sign;                        // the scale's: the queries take it
  bool vec;                          // 16-byte loads of q
};

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

template <typename T>
struct Mma;
template <>
struct Mma<__bf16> {
  typedef __bf16 E;
  typedef bf16x8_t V8;
  static constexpr int kParts = 1;
  static __device__ __forceinline__ f32x4_t mul(V8 a, V8 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma<float> : Mma<__bf16> {
  static constexpr int kParts = 3;
};
template <>
struct Mma<_Float16> {
  typedef _Float16 E;
  typedef f16x8_t V8;
  static constexpr int kParts = 1;
  static __device__ __forceinline__ f32x4_t mul(V8 a, V8 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// Weights of the 2-byte types are rounded once to their type, as the queries
// are; sums are of the weights as they were.  Against 64 bits a bf16 output is
// then off by 2.1e-3 of its norm, 1.7e-3 of it the output's own rounding (f16
// 2.9e-4, 2.1e-4).  A second part of each weight takes that away, but costs a
// prompt of 4096 tokens 26% (280 us, 42 heads of 128), single tokens 1% at 128
// channels and 12% at 192; a row is to come out alike from either kernel.
//
// The range of weights.  In bf16 and float32 they reach 1 or a little more.  f16
// has its 11 bits down to 2^-14 only and nothing below 2^-25: there r lies below
// m, weights reach 2^15, and one of 2^-25 of the largest still has all its bits;
// a smaller one is off by at most 2^-36 of the largest.  (With weights up to 1
// a row of 20000 tokens beside one of 17 nats more lost them all.)
//
// The exponent of a value scale counts within [kLeast, kLast]: 2^-e has to stay
// in 32 bits, and the weights take the rest.  In f16 they could not take more
// than 1 (and the sum does without: the largest weight is above 2^11).
template <typename T>
struct Range {
  static constexpr float kSetFew = 0.0f, kSetMany = 0.0f, kMostMany = 8.0f, kLeast = -60.0f, kLast = 60.0f;
};
template <>
struct Range<_Float16> {
  static constexpr float kSetFew = 15.0f, kSetMany = 11.0f, kMostMany = 15.0f, kLeast = -60.0f, kLast = 128.0f;
};
// kSet: the exponent of the largest weight when the reference is set, kMostMany
// that at which the many-rows kernel raises it.  Where scores are rounded by
// more than the room to f16's largest number, the reference is the maximum.
template <typename T>
__device__ __forceinline__ float room(float exponent, bool huge) {
  return __is_same(T, _Float16) && huge ? 0.0f : exponent;
}

struct ValueScale {
  float e, rest, back;   // what counts of the exponent, the factor of the weights, 2^-e
};
template <typename T>
__device__ __forceinline__ ValueScale value_scale(int byte) {
  const float all = (float)(byte - 127);
  ValueScale r;
  r.e = all < Range<T>::kLeast ? Range<T>::kLeast : all > Range<T>::kLast ? Range<T>::kLast : all;
  r.rest = __builtin_ldexpf(1.0f, (int)(all - r.e));
  r.back = __builtin_ldexpf(1.0f, -(int)r.e);
  return r;
}

// Eight codes (two words) as an operand, exactly.
template <typename V8>
__device__ __forceinline__ V8 decode8(uint32_t lo, uint32_t hi) {
  uint32_t d[4];
  if constexpr (__is_same(V8, bf16x8_t)) {
    d[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
    d[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
    d[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
    d[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  } else {
    d[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    d[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    d[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    d[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
  }
  return __builtin_bit_cast(V8, d);
}

// 0x80 in each byte of w that is a NaN code.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// 1.0 (code 0x38) where `nan` has 0x80, else 0.
__device__ __forceinline__ uint32_t nan_ones(uint32_t nan) { return (nan >> 2) | (nan >> 3) | (nan >> 4); }

// Eight floats as the parts of an operand: rounded once to a 2-byte type, or
// split into three bf16 parts.
template <typename T>
__device__ __forceinline__ void to_parts(const float (&x)[8], typename Mma<T>::V8 (&p)[Mma<T>::kParts]) {
  if constexpr (Mma<T>::kParts == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[0][i] = (typename Mma<T>::E)x[i];
  } else {
    uint32_t d[3][4];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      uint32_t h0, m0, l0, h1, m1, l1;
      split3_bits(fbits(x[i]), h0, m0, l0);
      split3_bits(fbits(x[i + 1]), h1, m1, l1);
      d[0][i / 2] = __builtin_amdgcn_perm(h1, h0, 0x07060302u);
      d[1][i / 2] = __builtin_amdgcn_perm(m1, m0, 0x07060302u);
      d[2][i / 2] = __builtin_amdgcn_perm(l1, l0, 0x07060302u);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) p[k] = __builtin_bit_cast(bf16x8_t, d[k]);
  }
}

// Eight channels of a query row from element offset 8 c on.
template <typename T>
__device__ __forceinline__ void load_row8(const T* row, bool vec, float (&x)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      const f32x4_t lo = *(const f32x4_t*)row, hi = *((const f32x4_t*)row + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) { x[i] = lo[i]; x[4 + i] = hi[i]; }
    } else {
      typedef T vec8 __attribute__((ext_vector_type(8)));
      const vec8 u = *(const vec8*)row;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (float)u[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = load_x(row + i);
  }
}

// Scaled scores of this size are rounded by 1/16 and more, so weights have to
// come from the same roundings as the maximum.
__device__ __forceinline__ bool huge_score(float x) { return __builtin_fabsf(x) > 1048576.0f; }

__device__ __forceinline__ float pow2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float max_across_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_across_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// The tokens that rows [t0, t1] (token numbers among the new ones) see, and
// where a split axis starts.
struct Span {
  int32_t first, last;   // positions of the first and the last row
  int32_t begin, end;    // cached tokens that any of the rows sees; begin on a tile
  int32_t from;          // where the window's part of them starts
};

// The first position that a row at position p sees through the window.
__device__ __forceinline__ int32_t first_seen(const AttnArgs& A, int32_t p) {
  return A.window > 0 && p >= A.window ? p - A.window + 1 : 0;
}

template <bool SINKS>
__device__ __forceinline__ Span span_of(const AttnArgs& A, const Sequence& s, int t0, int t1) {
  Span r;
  r.first = s.first + t0;
  r.last = s.first + t1;
  const int64_t cap = A.s.width << A.c.page_shift;
  r.end = r.last + 1 < cap ? r.last + 1 : (int32_t)cap;
  const int32_t lo = first_seen(A, r.first);
  // behind the table there is nothing, and positions from there on would pass 32 bits
  r.from = (lo < cap ? lo : (int32_t)cap) & ~63;
  // Sinks: their tiles come right before the window's part, so that what goes
  // along the axis and splits it sees one axis [begin, end); see place_of.  A
  // call costs the tokens seen, not the length: 64 sequences of up to 100003
  // tokens, 32 heads of 128 over 8, 4096 + 4 seen (539 MB) 98 us, 5.5 TB/s; 1024
  // and 264 tokens of two prompts, 42 heads over 6, 2048 + 100 seen 97 us, 612
  // TFLOP/s: 426 blocks, so that 170 units have two and 86 one.
  const int32_t front = A.sinks < r.from ? A.sinks : r.from;
  r.begin = SINKS ? r.from - ((front + 63) & ~63) : r.from;
  return r;
}

// The token at place t of the axis.
template <bool SINKS>
__device__ __forceinline__ int place_of(const Span& sp, int t) { return SINKS && t < sp.from ? t - sp.begin : t; }

// Whether rows whose windows start at `from` or before see the tile at token t0
// whole, as far as window and sinks go.
template <bool SINKS>
__device__ __forceinline__ bool in_reach(const AttnArgs& A, int t0, int from) { return t0 >= from || (SINKS && t0 + 64 <= A.sinks); }

// ---------------------------------------------------------------------------
// Few rows: the waves of a block share the rows and split the tokens
// ---------------------------------------------------------------------------
//
// A tile is 64 tokens.  Lane (n, g) = (lane % 16, lane / 16) holds tokens 16 g
// .. 16 g + 15 of column n, so a 16-byte load of codes is one channel's tokens
// (values) or 16 channels of one token (keys).  Key row m of multiply t is
// token 16 (m / 4) + 4 t + m % 4: with four rows per lane group in the result,
// lane group g gets the tokens 16 g + 4 t + (0..3) from it.  Nothing is shared
// between waves until the end, so K and V go straight from memory to
// registers; the queries lie in LDS as operands.
//
// Bound by memory: 4 sequences of up to 128k tokens (837 MB) take 165 us with
// the join, 5.1 TB/s, where a plain read of as much reaches 6.5 and a copy 4.9;
// 32 of up to 8k 28 us, 3.1 TB/s and 5 us of it the join.  Loads that bypass
// the caches took 193 us for the former: in pages of 128 tokens two waves share
// each line of the values.
constexpr int kFewWaves = 4;

template <int DIM, int NT, int PARTS>
constexpr int few_lds_bytes() {
  constexpr int q = NT * 16 * DIM * 2 * PARTS;          // operands
  constexpr int red = 2 * NT * 16 * DIM * 4 + kFewWaves * NT * 16 * 2 * 4;  // two waves' sums; all waves' maxima and sums
  return q > red ? q : red;
}

// About what registers a lane needs for the running sums, a tile's scores and
// its codes: up to what two blocks a unit leave each there are two.  The
// compiler does not always meet it: 2-byte types with 16 rows of 192 channels
// spill 25 at two blocks (32 sequences of up to 8k tokens, 16 heads, take 38 us,
// 41 with one block and no spill; 4 of up to 87k 199 us, and 183), 32 rows of
// 256 spill 82 in bf16, 94 in f16 and 105 in float32 at one (with sinks 108, 96
// and 109).
constexpr int few_blocks_per_cu(int dim, int nt, int parts) { return nt * dim / 4 + 16 * nt + dim / 2 + 24 * parts * nt + 64 <= 256 ? 2 : 1; }

template <typename T, int DIM, int NT, bool SINKS>
__global__ __launch_bounds__(64 * kFewWaves, few_blocks_per_cu(DIM, NT, Mma<T>::kParts)) void few_rows_kernel(AttnArgs A) {
  typedef Mma<T> M;
  typedef typename M::V8 V8;
  constexpr int PARTS = M::kParts, U = DIM / 64, CB = DIM / 16, ROWS = 16 * NT;
  // Whether tiles that are seen whole scale only their largest score first.  In
  // float32 with 32 rows the second way costs more registers than it spares
  // work: a prompt of 4096 tokens, 8 heads of 128, 279 us with it and 263
  // without; 16 sequences of 6 tokens, 256 channels, 62 and 54 us.  With 16 rows
  // it spares 2%.
  constexpr bool BOTH = PARTS == 1 || NT == 1;
  extern __shared__ __align__(16) uint8_t lds[];

  int64_t block = blockIdx.x;
  const int split = (int)(block % A.splits);
  block /= A.splits;
  const int rt = (int)(block % A.row_tiles);
  block /= A.row_tiles;
  const int h = (int)(block % A.c.heads), b = (int)(block / A.c.heads);
  const Sequence sq = sequence(A.s, b);
  const int rows = sq.count * A.group, row0 = rt * ROWS;
  if (row0 >= rows) return;
  const int nrows = rows - row0 < ROWS ? rows - row0 : ROWS;
  // float32 has the sinks' form of it also without any, which spills less: 32 rows
  // of 256 channels take 55 us with it and 58 without (bf16 44 and 43)
  const Span sp = span_of<SINKS || PARTS == 3>(A, sq, row0 / A.group, (row0 + nrows - 1) / A.group);
  const int64_t lo64 = (int64_t)sp.begin + (int64_t)split * A.chunk;
  // a split behind the end writes nothing: the join counts the splits itself;
  // the first one always writes, so that rows that see nothing become zeros
  if (split > 0 && lo64 >= sp.end) return;
  const int lo = (int)lo64;
  const int hi = sp.end - lo < A.chunk ? sp.end : lo + A.chunk;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;

  // queries as operands: [NT][2 U steps][PARTS][64 lanes] of 16 bytes, the
  // step (u, s) of lane (n, g) holding channels 64 u + 16 g + 8 s .. + 7
  V8* ql = (V8*)lds;
  for (int i = threadIdx.x; i < ROWS * (DIM / 8); i += 64 * kFewWaves) {
    const int r = i / (DIM / 8), c8 = i % (DIM / 8);
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < nrows) {
      const int row = row0 + r, t = row / A.group, hh = h * A.group + row % A.group;
      load_row8((const T*)A.q + (int64_t)(sq.row0 + t) * A.q_token + (int64_t)hh * A.q_head + 8 * c8, A.vec, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= A.sign;
    }
    V8 p[PARTS];
    to_parts<T>(x, p);
    const int u = c8 / 8, gg = (c8 / 2) % 4, s = c8 % 2;
#pragma unroll
    for (int k = 0; k < PARTS; ++k) ql[(((r / 16) * 2 * U + 2 * u + s) * PARTS + k) * 64 + gg * 16 + r % 16] = p[k];
  }
  __syncthreads();

  float m[NT], l[NT];
  f32x4_t o[NT][CB];
  int pos[NT];   // the column's position; -1: no row
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = -__builtin_inff();
    l[nt] = 0.0f;
    const int r = nt * 16 + n;
    pos[nt] = r < nrows ? sp.first - row0 / A.group + (row0 + r) / A.group : -1;
#pragma unroll
    for (int c = 0; c < CB; ++c) o[nt][c] = f32x4_t{0, 0, 0, 0};
  }

  const int from_last = first_seen(A, sp.last);
  const int shift = A.c.page_shift, pmask = (1 << shift) - 1;
  const int32_t* table = A.s.table + (int64_t)b * A.s.width;
  const int64_t page_bytes = (int64_t)DIM << shift;

  // The table's entry of token t (behind the end: the last one), and the page
  // that it means there; -1 where there is none.  Entries are fetched a tile
  // ahead and no load stands behind a branch: waiting for either at once would
  // wait for every load of codes before it.
  auto entry_of = [&](int t) -> int { return table[place_of<SINKS>(sp, t < hi ? t : hi - 1) >> shift]; };
  auto page_of = [&](int entry, int t) -> int { return entry < A.c.pages && t < hi ? entry : -1; };

  constexpr int STEP = 64 * kFewWaves;
  uint4 kreg[4][U], vreg[CB];
  float kscale = 0.0f;
  int kbyte = 0, vbyte = 0;

  // Key rows of lane n come from token group n / 4, values from group g.
  auto load_k = [&](int t0, int id) {
    const int64_t ph = (int64_t)(id < 0 ? 0 : id) * A.c.heads + h;
    const uint8_t* p = A.c.k + ph * page_bytes + (int64_t)((t0 & pmask) + ((n >> 2) * 16 & pmask) + (n & 3)) * DIM + 16 * g;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u) kreg[t][u] = *(const uint4*)(p + 4 * t * DIM + 64 * u);
  };
  auto load_v = [&](int t0, int id) {
    const int64_t ph = (int64_t)(id < 0 ? 0 : id) * A.c.heads + h;
    const uint8_t* p = A.c.v + ph * page_bytes + ((int64_t)n << shift) + ((t0 & pmask) + (g * 16 & pmask));
#pragma unroll
    for (int c = 0; c < CB; ++c) vreg[c] = *(const uint4*)(p + ((int64_t)(16 * c) << shift));
    kbyte = A.c.ks[ph];
    vbyte = A.c.vs[ph];
  };

  int t0 = lo + wave * 64;
  const int tk = (n >> 2) * 16, tv = g * 16;   // the lane's first tokens of a tile, of keys and of values
  int idk = -1, idv = -1, entry_k = -1, entry_v = -1;
  if (t0 < hi) {
    idk = page_of(entry_of(t0 + tk), t0 + tk);
    idv = page_of(entry_of(t0 + tv), t0 + tv);
    entry_k = entry_of(t0 + STEP + tk);
    entry_v = entry_of(t0 + STEP + tv);
    load_k(place_of<SINKS>(sp, t0), idk);
    load_v(place_of<SINKS>(sp, t0), idv);
  }
  for (; t0 < hi; t0 += STEP) {
    const int t_next = t0 + STEP;
    asm volatile("" ::: "memory");   // the query operands are read from LDS in each tile: held, they would fill the registers
    // behind the last tile that one is loaded again
    const bool more = t_next < hi;
    const int t_load = place_of<SINKS>(sp, more ? t_next : t0), at = place_of<SINKS>(sp, t0);
    const int idk_next = more ? page_of(entry_k, t_next + tk) : idk, idv_next = more ? page_of(entry_v, t_next + tv) : idv;
    entry_k = entry_of(t_next + STEP + tk);
    entry_v = entry_of(t_next + STEP + tv);
    kscale = __builtin_ldexpf(A.scale_log2, kbyte - 127);
    const ValueScale vs = value_scale<T>(vbyte);

    // S^T
    f32x4_t sc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int t = 0; t < 4; ++t) sc[nt][t] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        V8 a[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) a[t] = s ? decode8<V8>(kreg[t][u].z, kreg[t][u].w) : decode8<V8>(kreg[t][u].x, kreg[t][u].y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < PARTS; ++k) {
            const V8 bq = ql[((nt * 2 * U + 2 * u + s) * PARTS + k) * 64 + lane];
#pragma unroll
            for (int t = 0; t < 4; ++t) sc[nt][t] = M::mul(a[t], bq, sc[nt][t]);
          }
      }
    }
    load_k(t_load, idk_next);

    // what each row sees; a tile that all rows see whole needs no comparison
    const bool whole = at + 63 <= sp.first && in_reach<SINKS>(A, at, from_last) && t0 + 64 <= hi &&
                       __all(idv >= 0);   // columns without a row may hold anything
    V8 pw[NT][2][PARTS];
    uint32_t seen[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      seen[nt] = 0xffffu;
      if (!whole) {
        seen[nt] = 0;
        const int tg = at + 16 * g;
        // tokens tg + i with i <= last_i and i >= first_i
        const int last_i = (pos[nt] < hi ? pos[nt] : hi - 1) - tg;
        const int first_i = first_seen(A, pos[nt]) - tg, sinks_i = A.sinks - tg;
        if (idv >= 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) seen[nt] |= (i <= last_i && (i >= first_i || (SINKS && i < sinks_i))) ? 1u << i : 0u;
        }
      }
      // a lane's tokens share their scales: of a tile that is seen whole only
      // the largest score is scaled for the maximum (the factor is not negative)
      float w[16], top, mul = kscale, add = vs.e;
      bool scaled = !BOTH || !whole;
      if (BOTH && whole) {
        top = sc[nt][0][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, sc[nt][i / 4][i % 4]);
        top = __builtin_fmaf(top, mul, add);
        scaled = __any(huge_score(top));
      }
      if (scaled) {
        top = -__builtin_inff();
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __builtin_fmaf(sc[nt][i / 4][i % 4], kscale, vs.e);
            sc[nt][i / 4][i % 4] = x;
            top = fmaxf(top, x);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = (seen[nt] >> i) & 1 ? __builtin_fmaf(sc[nt][i / 4][i % 4], kscale, vs.e) : -__builtin_inff();
            sc[nt][i / 4][i % 4] = x;
            top = fmaxf(top, x);
          }
        }
        mul = 1.0f;
        add = 0.0f;
      }
      top = max_across_groups(top);
      const float m_new = fmaxf(m[nt], top - room<T>(Range<T>::kSetFew, huge_score(top)));
      const float base = m_new == -__builtin_inff() ? 0.0f : m_new;
      const float alpha = pow2(m[nt] - base), less = add - base;
      m[nt] = m_new;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        w[i] = pow2(__builtin_fmaf(sc[nt][i / 4][i % 4], mul, less));
        sum += w[i];
      }
      l[nt] = __builtin_fmaf(sum, vs.back, l[nt] * alpha);
#pragma unroll
      for (int c = 0; c < CB; ++c) o[nt][c] *= alpha;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = w[8 * s + i] * vs.rest;
        to_parts<T>(x, pw[nt][s]);
      }
    }

    // O^T
    bool nan = false;
    if (!whole) {
      uint32_t any = 0;
#pragma unroll
      for (int c = 0; c < CB; ++c) any |= nan_bytes(vreg[c].x) | nan_bytes(vreg[c].y) | nan_bytes(vreg[c].z) | nan_bytes(vreg[c].w);
      nan = __any(any != 0);
    }
    if (!nan) {
#pragma unroll
      for (int c = 0; c < CB; ++c) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const V8 a = s ? decode8<V8>(vreg[c].z, vreg[c].w) : decode8<V8>(vreg[c].x, vreg[c].y);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < PARTS; ++k) o[nt][c] = M::mul(a, pw[nt][s][k], o[nt][c]);
        }
      }
    } else {
      // NaN codes as zeros, and beside it the number of NaN codes that a row
      // sees: where there is one, the row's channel is NaN
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        f32x4_t hits[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) hits[nt] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t w0 = s ? vreg[c].z : vreg[c].x, w1 = s ? vreg[c].w : vreg[c].y;
          const uint32_t n0 = nan_bytes(w0), n1 = nan_bytes(w1);
          const V8 a = decode8<V8>(w0 & ~(n0 | (n0 - (n0 >> 7))), w1 & ~(n1 | (n1 - (n1 >> 7))));
          const V8 ones = decode8<V8>(nan_ones(n0), nan_ones(n1));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < PARTS; ++k) o[nt][c] = M::mul(a, pw[nt][s][k], o[nt][c]);
            V8 vis;
#pragma unroll
            for (int i = 0; i < 8; ++i) vis[i] = (typename M::E)(float)((seen[nt] >> (8 * s + i)) & 1);
            hits[nt] = M::mul(ones, vis, hits[nt]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][c][i] = hits[nt][i] > 0.0f ? __builtin_nanf("") : o[nt][c][i];
      }
    }
    load_v(t_load, idv_next);
    idk = idk_next;
    idv = idv_next;
  }

  // join the waves: common maximum, then the sums of waves 2 and 3 through LDS
  // to waves 0 and 1, and of wave 1 to wave 0
  __syncthreads();
  f32x4_t* red = (f32x4_t*)lds;                                 // [2][NT][CB][64]
  float* ml = (float*)(lds + 2 * NT * CB * 64 * 16);            // [waves][NT][16][2]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float sum = sum_across_groups(l[nt]);
    if (g == 0) {
      ml[((wave * NT + nt) * 16 + n) * 2] = m[nt];
      ml[((wave * NT + nt) * 16 + n) * 2 + 1] = sum;
    }
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) top = fmaxf(top, ml[((w * NT + nt) * 16 + n) * 2]);
    const float base = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w)
      sum += ml[((w * NT + nt) * 16 + n) * 2 + 1] * pow2(ml[((w * NT + nt) * 16 + n) * 2] - base);
    const float f = pow2(m[nt] - base);
#pragma unroll
    for (int c = 0; c < CB; ++c) o[nt][c] *= f;
    m[nt] = top;
    l[nt] = sum;
  }
#pragma unroll
  for (int half = kFewWaves / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < CB; ++c) red[(((wave - half) * NT + nt) * CB + c) * 64 + lane] = o[nt][c];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < CB; ++c) o[nt][c] += red[((wave * NT + nt) * CB + c) * 64 + lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 16 + n;
    if (r >= nrows) continue;
    const int row = row0 + r, t = row / A.group, hh = h * A.group + row % A.group;
    const int64_t at = (int64_t)(sq.row0 + t) * A.heads_q + hh;
    if (A.splits == 1) {
      T* out = (T*)A.out + at * DIM;
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        typedef T vec4 __attribute__((ext_vector_type(4)));
        vec4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (T)(l[nt] == 0.0f ? 0.0f : o[nt][c][i] / l[nt]);
        *(vec4*)(out + 16 * c + 4 * g) = y;
      }
    } else {
      const int64_t ps = at * A.splits + split;
      if (g == 0) {
        A.part_m[ps] = m[nt];
        A.part_l[ps] = l[nt];
      }
      float* po = A.part_o + ps * DIM;
#pragma unroll
      for (int c = 0; c < CB; ++c) *(f32x4_t*)(po + 16 * c + 4 * g) = o[nt][c];
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows: the waves of a block share the tokens and split the rows
// ---------------------------------------------------------------------------
//
// 2-byte types.  Each of four waves has 32 rows; a tile of 64 tokens is
// converted once for all of them on its way into LDS, where two tiles
// alternate: while one is multiplied the next one's codes are on their way to
// registers, and one barrier a tile is enough.  The 32x32 multiply reads each
// LDS operand for twice as many rows as the 16x16 one; at 32 rows a wave the
// LDS and the matrix cores are then about equally busy.
//
// Lane (n, hh) = (lane % 32, lane / 32) holds of multiply tt tokens 32 tt + 16
// s + 8 hh + (0..7) of column n, s = 0, 1: an operand of the second product
// per s.  Key rows therefore lie in LDS in the order in which the result has
// them.  Rows of LDS are stored with their 16-byte pieces permuted by the row
// number, so that lanes reading down a column of pieces meet all banks.
//
// The reference is raised only once a score passes it by kMostMany: most tiles
// leave the sums alone.
//
// Bound by the order of a wave's steps, not by a unit: K Q^T, the maximum, the
// weights and V P^T follow one another, and the two or three waves a SIMD that
// the registers leave overlap little of it.  A causal prompt of 4096 tokens, 42
// heads of 128, takes 225 us (803 TFLOP/s), with the matrix cores busy 32% of
// the cycles, the vector units 45%, and waves waiting 31% of theirs; 1024 tokens
// over 32768, 16 heads of 64, 214 us with the join (631 TFLOP/s; 26%, 59% and
// 32%).  Two groups of four waves that took turns at multiplies and weights
// over the same tile took 5% and 19% longer.
constexpr int kManyWaves = 4, kManyRows = 32 * kManyWaves;

template <typename T>
struct Mma32;
template <>
struct Mma32<__bf16> {
  static __device__ __forceinline__ f32x16_t mul(bf16x8_t a, bf16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mma32<_Float16> {
  static __device__ __forceinline__ f32x16_t mul(f16x8_t a, f16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

// What the four groups of 16 tokens of a tile have in common.
struct GroupInfo {
  float kscale;                  // score factor
  float e, rest, back;           // of ValueScale
};

// Where the pieces of 16 bytes of row r lie: 16 lanes read a column of pieces
// of 16 rows in a cycle, 256 bytes of LDS, and meet every bank once.  (With 16
// pieces a row; 24 are three times the pattern of 8.)
template <int PIECES>
__device__ __forceinline__ int swizzle(int r) { return PIECES % 16 == 0 ? r & 15 : (r & 7) ^ ((r >> 3) & 1); }

template <int DIM>
struct ManyTile {
  uint4 k[64 * DIM / 8];   // [64 rows][DIM / 8] pieces of 8 elements
  uint4 v[DIM * 8];        // [DIM channels][8]
};

template <int DIM>
struct ManyShared {
  ManyTile<DIM> tile[2];
  GroupInfo info[2][4];
  uint32_t there[2];   // bit g: group g's page is there
  int32_t nan[2];      // the first token of the last partial tile here that had a NaN code among its values,
  __align__(8) uint16_t nan_tokens[2][DIM][4];   // and which ones: a bit per token
};

// A barrier for what lies in LDS: loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <typename T, int DIM, bool ONE_PAGE, bool SINKS>
__global__ __launch_bounds__(64 * kManyWaves, DIM <= 64 ? 3 : DIM <= 128 ? 2 : 1) void many_rows_kernel(AttnArgs A) {
  typedef typename Mma<T>::V8 V8;
  typedef typename Mma<T>::E E;
  constexpr int KS = DIM / 16, CB = DIM / 32, KP = DIM / 8, THREADS = 64 * kManyWaves;
  constexpr int KLOADS = 64 * DIM / 16 / THREADS;   // 16-byte loads of a thread and tile, of keys and of values
  static_assert(KLOADS * THREADS * 16 == 64 * DIM, "whole rounds");
  extern __shared__ __align__(16) uint8_t lds[];
  ManyShared<DIM>& S = *(ManyShared<DIM>*)lds;

  // the longest row tiles first; splits, heads and sequences side by side
  int64_t block = blockIdx.x;
  const int split = (int)(block % A.splits);
  block /= A.splits;
  const int h = (int)(block % A.c.heads);
  block /= A.c.heads;
  const int b = (int)(block % A.s.batch);
  const int rt = A.row_tiles - 1 - (int)(block / A.s.batch);
  const Sequence sq = sequence(A.s, b);
  const int rows = sq.count * A.group, row0 = rt * kManyRows;
  if (row0 >= rows) return;
  const int nrows = rows - row0 < kManyRows ? rows - row0 : kManyRows;
  const Span sp = span_of<SINKS>(A, sq, row0 / A.group, (row0 + nrows - 1) / A.group);
  const int64_t lo64 = (int64_t)sp.begin + (int64_t)split * A.chunk;
  if (split > 0 && lo64 >= sp.end) return;
  const int lo = (int)lo64;
  const int hi = sp.end - lo < A.chunk ? sp.end : lo + A.chunk;

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, hh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // what goes by the wave stays in scalar registers
  const int shift = A.c.page_shift, pmask = (1 << shift) - 1;
  const int32_t* table = A.s.table + (int64_t)b * A.s.width;
  const int64_t page_bytes = (int64_t)DIM << shift;

  // the wave's queries, in registers: step s holds channels 16 s + 8 hh .. + 7
  const int my = wave * 32 + n, base_pos = sq.first;
  const int pos = my < nrows ? base_pos + (row0 + my) / A.group : -1;
  V8 q[KS];
  {
    const int row = row0 + (my < nrows ? my : 0), t = row / A.group, head = h * A.group + row % A.group;
    const T* p = (const T*)A.q + (int64_t)(sq.row0 + t) * A.q_token + (int64_t)head * A.q_head + 8 * hh;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8];
      load_row8(p + 16 * s, A.vec, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[s][i] = (E)(my < nrows ? x[i] * A.sign : 0.0f);
    }
  }
  // positions of the wave's first and last row: rows are in the order of positions
  const int wave_rows = nrows - wave * 32 < 32 ? nrows - wave * 32 : 32;
  const int wfirst = wave_rows > 0 ? base_pos + (row0 + wave * 32) / A.group : 0;
  const int wlast = wave_rows > 0 ? base_pos + (row0 + wave * 32 + wave_rows - 1) / A.group : -1;
  const int from_wfirst = first_seen(A, wfirst), from_wlast = first_seen(A, wlast), from_last = first_seen(A, sp.last);

  auto page_of = [&](int t) -> int {
    if (t >= hi) return -1;
    const int id = table[t >> shift];
    return id < A.c.pages ? id : -1;
  };
  // a thread's loads: piece i THREADS + tid of the keys, DIM / 16 of them a
  // row; values of channel tid / 4 + i THREADS / 4, tokens 16 (tid % 4)
  const int vch = tid / 4, vg = tid % 4;
  int krow[KLOADS], kc[KLOADS];
#pragma unroll
  for (int i = 0; i < KLOADS; ++i) {
    krow[i] = (i * THREADS + tid) / (DIM / 16);
    kc[i] = (i * THREADS + tid) % (DIM / 16);
  }
  // Entries of the table are fetched a tile before they are looked at, into
  // vector registers (a scalar load would be waited for with the next LDS
  // read), and every load is issued without a branch around it (behind one its
  // register would be copied, and so waited for, at once): what lies behind
  // the end reads the last entry, pages that are not there read page 0.
  // A tile inside one page has one entry, and its addresses are the block's.
  constexpr int IDS = ONE_PAGE ? 1 : KLOADS + 1, VALUES = IDS - 1;
  uint4 kreg[KLOADS], vreg[KLOADS];
  int id[IDS], entry[IDS];   // pages of the keys' loads and of the values', of the next tile; the table's entries of the one after it
  int kbyte = 0, vbyte = 0;
  auto token = [&](int t0, int i) -> int { return ONE_PAGE ? t0 : t0 + (i < KLOADS ? krow[i < KLOADS ? i : 0] : 16 * vg); };
  auto fetch_ids = [&](int t0) {
#pragma unroll
    for (int i = 0; i < IDS; ++i) {
      const int t = token(t0, i);
      int at = place_of<SINKS>(sp, t < hi ? t : hi - 1) >> shift;
      asm("" : "+v"(at));
      entry[i] = table[at];
    }
  };
  auto ids = [&](int t0) {
#pragma unroll
    for (int i = 0; i < IDS; ++i) {
      id[i] = entry[i] < A.c.pages && token(t0, i) < hi ? entry[i] : -1;
      if constexpr (ONE_PAGE) id[i] = __builtin_amdgcn_readfirstlane(id[i]);
    }
  };
  auto load = [&](int place) {
    const int t0 = place_of<SINKS>(sp, place);
#pragma unroll
    for (int i = 0; i < KLOADS; ++i) {
      if constexpr (ONE_PAGE) {
        const uint8_t* base = A.c.k + ((int64_t)(id[0] < 0 ? 0 : id[0]) * A.c.heads + h) * page_bytes + (uint32_t)(t0 & pmask) * DIM;
        kreg[i] = *(const uint4*)(base + 16 * i * THREADS + 16u * (uint32_t)tid);
      } else {
        const int64_t ph = (int64_t)(id[i < IDS ? i : 0] < 0 ? 0 : id[i < IDS ? i : 0]) * A.c.heads + h;
        kreg[i] = *(const uint4*)(A.c.k + ph * page_bytes + (uint32_t)((t0 + krow[i]) & pmask) * DIM + 16 * kc[i]);
      }
    }
    const int64_t ph = (int64_t)(id[VALUES] < 0 ? 0 : id[VALUES]) * A.c.heads + h;
    const uint8_t* base = A.c.v + ph * page_bytes + (ONE_PAGE ? t0 & pmask : 0);
    const uint32_t off = (uint32_t)(vch << shift) + (ONE_PAGE ? 16 * vg : (t0 + 16 * vg) & pmask);
#pragma unroll
    for (int i = 0; i < KLOADS; ++i) vreg[i] = *(const uint4*)(base + ((int64_t)(i * (THREADS / 4)) << shift) + off);
    kbyte = A.c.ks[ph];
    vbyte = A.c.vs[ph];
  };
  // converts the loaded tile into LDS; `part`: some row of the block does not see all of it
  auto store = [&](int at, int t0, bool part) {
    ManyTile<DIM>& t = S.tile[at];
    if (part) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < KLOADS; ++i) {
        uint32_t* w = &vreg[i].x;
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t nan = nan_bytes(w[k]);
          w[k] &= ~(nan | (nan - (nan >> 7)));
          bits |= (((nan >> 7) * 0x10204080u) >> 28) << (4 * k);   // bits 7, 15, 23, 31 side by side
        }
        S.nan_tokens[at][vch + i * (THREADS / 4)][vg] = (uint16_t)bits;
        any |= bits;
      }
      if (__any(any != 0) && lane == 0) S.nan[at] = t0;
    }
#pragma unroll
    for (int i = 0; i < KLOADS; ++i) {
      const int tok = krow[i];
      const int r = (tok & 32) | (tok & 16) | ((tok & 4) << 1) | ((tok & 8) >> 1) | (tok & 3);
      t.k[r * KP + ((2 * kc[i]) ^ swizzle<KP>(r))] = __builtin_bit_cast(uint4, decode8<V8>(kreg[i].x, kreg[i].y));
      t.k[r * KP + ((2 * kc[i] + 1) ^ swizzle<KP>(r))] = __builtin_bit_cast(uint4, decode8<V8>(kreg[i].z, kreg[i].w));
      const int c = vch + i * (THREADS / 4);
      t.v[c * 8 + ((2 * vg) ^ swizzle<8>(c))] = __builtin_bit_cast(uint4, decode8<V8>(vreg[i].x, vreg[i].y));
      t.v[c * 8 + ((2 * vg + 1) ^ swizzle<8>(c))] = __builtin_bit_cast(uint4, decode8<V8>(vreg[i].z, vreg[i].w));
    }
    if (wave == 0) {
      const ValueScale vs = value_scale<T>(vbyte);
      if (tid < 4) S.info[at][tid] = {__builtin_ldexpf(A.scale_log2, kbyte - 127), vs.e, vs.rest, vs.back};
      const uint64_t there = __ballot(id[VALUES] >= 0);
      if (tid == 0) S.there[at] = (uint32_t)there & 0xfu;
    }
  };

  f32x16_t o[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[c][i] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;

  // a tile is partial for the block if a row does not see it whole or a page is missing
  auto partial = [&](int place) -> bool {
    const int t0 = place_of<SINKS>(sp, place);
    return t0 + 63 > sp.first || !in_reach<SINKS>(A, t0, from_last) || place + 64 > hi || __any(id[VALUES] < 0);
  };

  if (tid < 2) S.nan[tid] = -1;
  __syncthreads();
  int at = 0;
  if (lo < hi) {
    fetch_ids(lo);
    ids(lo);
    load(lo);
    fetch_ids(lo + 64);
    store(0, lo, partial(lo));
    ids(lo + 64);
    fetch_ids(lo + 128);
  }
  for (int place = lo; place < hi; place += 64, at ^= 1) {
    lds_barrier();
    load(place + 64);   // also behind the last tile, from page 0
    const bool next_partial = partial(place + 64);
    const int t0 = place_of<SINKS>(sp, place);
    const ManyTile<DIM>& t = S.tile[at];
    const bool unseen = t0 > wlast || (t0 + 63 < from_wfirst && !(SINKS && t0 < A.sinks));
    if (!unseen) {
      f32x16_t sc[2];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[tt][i] = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          const int r = 32 * tt + n;
          sc[tt] = Mma32<T>::mul(__builtin_bit_cast(V8, t.k[r * KP + ((2 * s + hh) ^ swizzle<KP>(r))]), q[s], sc[tt]);
        }
      }
      const uint32_t there = S.there[at];
      const bool whole = t0 + 63 <= wfirst && in_reach<SINKS>(A, t0, from_wlast) && wave_rows == 32 && there == 0xfu;
      // the largest score, and the factor and summand that make weights of
      // scores: of tiles that are seen whole only the largest of each group of
      // 16 tokens is scaled for it (the factors are not negative)
      float top = -__builtin_inff(), mul[4], add[4];
      uint64_t vis = ~0ull;   // the tile's tokens that the lane's row sees
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        mul[g] = S.info[at][g].kscale;
        add[g] = S.info[at][g].e;
      }
      bool scaled = !whole;
      if (whole) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float x = sc[g / 2][8 * (g % 2)];
#pragma unroll
          for (int j = 1; j < 8; ++j) x = fmaxf(x, sc[g / 2][8 * (g % 2) + j]);
          top = fmaxf(top, __builtin_fmaf(x, mul[g], add[g]));
        }
        scaled = __any(huge_score(top));
      }
      if (scaled) {
        top = -__builtin_inff();
        const int last_i = pos - t0, first_i = first_seen(A, pos) - t0;
        vis = last_i < 0 ? 0 : last_i >= 63 ? ~0ull : (2ull << last_i) - 1;
        if constexpr (SINKS) {
          const int sinks_i = A.sinks - t0;
          const uint64_t sinks = sinks_i <= 0 ? 0 : sinks_i >= 64 ? ~0ull : (1ull << sinks_i) - 1;
          vis &= sinks | (first_i > 63 ? 0 : first_i > 0 ? ~0ull << first_i : ~0ull);
        } else if (first_i > 0) {
          vis = first_i > 63 ? 0 : vis & (~0ull << first_i);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) vis &= (there >> g) & 1 ? ~0ull : ~(0xffffull << (16 * g));
        const uint32_t seen[2] = {(uint32_t)vis >> (8 * hh), (uint32_t)(vis >> 32) >> (8 * hh)};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float x = __builtin_fmaf(sc[g / 2][8 * (g % 2) + j], mul[g], add[g]);
            x = (seen[g / 2] >> (16 * (g % 2) + j)) & 1 ? x : -__builtin_inff();
            sc[g / 2][8 * (g % 2) + j] = x;
            top = fmaxf(top, x);
          }
          mul[g] = 1.0f;
          add[g] = 0.0f;
        }
      }
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const bool huge = huge_score(top);
      if (__any(top > m + room<T>(Range<T>::kMostMany, huge))) {
        const float m_new = fmaxf(m, top - room<T>(Range<T>::kSetMany, huge));
        const float alpha = pow2(m - (m_new == -__builtin_inff() ? 0.0f : m_new));
        m = m_new;
        l *= alpha;
#pragma unroll
        for (int c = 0; c < CB; ++c) o[c] *= alpha;
      }
      const float base = m == -__builtin_inff() ? 0.0f : m;
      // rest is 1 but for values of very different scales; a branch around it
      // cost 4% (registers, and weights and multiplies apart in two blocks)
      V8 pw[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float back = S.info[at][g].back, rest = S.info[at][g].rest, less = add[g] - base;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = pow2(__builtin_fmaf(sc[g / 2][8 * (g % 2) + j], mul[g], less));
          sum += w;
          pw[g][j] = (E)(w * rest);
        }
        l = __builtin_fmaf(sum, back, l);
      }
      // one multiply after the other into different sums: into the same one it would wait
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          const int ch = 32 * c + n;
          o[c] = Mma32<T>::mul(__builtin_bit_cast(V8, t.v[ch * 8 + ((2 * g + hh) ^ swizzle<8>(ch))]), pw[g], o[c]);
        }
      if (S.nan[at] == place) {
        // NaN codes lie as zeros in the tile: a channel with one that the row sees is NaN
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t bad = *(const uint64_t*)S.nan_tokens[at][32 * c + 8 * (i / 4) + 4 * hh + i % 4];
            o[c][i] = (bad & vis) ? __builtin_nanf("") : o[c][i];
          }
      }
    }
    store(at ^ 1, place + 64, next_partial);   // its readers have passed this round's barrier
    ids(place + 128);
    fetch_ids(place + 192);
  }

  l += __shfl_xor(l, 32, 64);
  if (my >= nrows) return;
  const int row = row0 + my, tq = row / A.group, head = h * A.group + row % A.group;
  const int64_t out_row = (int64_t)(sq.row0 + tq) * A.heads_q + head;
  if (A.splits == 1) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T* out = (T*)A.out + out_row * DIM;
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        typedef T vec4 __attribute__((ext_vector_type(4)));
        vec4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (T)(l == 0.0f ? 0.0f : o[c][4 * i4 + i] * inv);
        *(vec4*)(out + 32 * c + 8 * i4 + 4 * hh) = y;
      }
  } else {
    const int64_t ps = out_row * A.splits + split;
    if (hh == 0) {
      A.part_m[ps] = m;
      A.part_l[ps] = l;
    }
    float* po = A.part_o + ps * DIM;
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4)
        *(f32x4_t*)(po + 32 * c + 8 * i4 + 4 * hh) = f32x4_t{o[c][4 * i4], o[c][4 * i4 + 1], o[c][4 * i4 + 2], o[c][4 * i4 + 3]};
  }
}

// ---------------------------------------------------------------------------
// Join of a split axis
// ---------------------------------------------------------------------------
//
// WAVES waves per output row, four or one: with few splits there are many
// rows, and a block's start and sums through LDS cost more than its loads
// (16384 rows of 6 splits: 31 us with four, 12 us with one).
template <typename T, int DIM, int WAVES>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs A, int rows_per_tile) {
  __shared__ float sum_o[4][DIM];
  __shared__ float sum_l[4];
  const int64_t at = WAVES == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (at >= (int64_t)A.s.tokens * A.heads_q) return;
  const int t_abs = (int)(at / A.heads_q), hh = (int)(at % A.heads_q);
  int b = t_abs;
  if (A.s.cu) {
    int lo = 0, hi = A.s.batch;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (A.s.cu[mid + 1] <= t_abs) lo = mid + 1; else hi = mid;
    }
    b = lo;
  }
  if (b >= A.s.batch) return;
  const Sequence sq = sequence(A.s, b);
  const int t = t_abs - sq.row0;
  if (t < 0 || t >= sq.count) return;
  const int row = t * A.group + hh % A.group, rows = sq.count * A.group, row0 = row / rows_per_tile * rows_per_tile;
  const int last = (row0 + rows_per_tile < rows ? row0 + rows_per_tile : rows) - 1;
  const Span sp = span_of<true>(A, sq, row0 / A.group, last / A.group);   // (sinks 0: as without)
  int n = sp.end > sp.begin ? (sp.end - sp.begin + A.chunk - 1) / A.chunk : 1;
  n = n < A.splits ? n : A.splits;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* pm = A.part_m + at * A.splits;
  const float* pl = A.part_l + at * A.splits;
  float mx = -__builtin_inff();
  for (int i = lane; i < n; i += 64) mx = fmaxf(mx, pm[i]);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
  const float base = mx == -__builtin_inff() ? 0.0f : mx;
  float acc[DIM / 64], l = 0.0f;
#pragma unroll
  for (int c = 0; c < DIM / 64; ++c) acc[c] = 0.0f;
#pragma unroll 4
  for (int i = WAVES == 4 ? wave : 0; i < n; i += WAVES) {
    const float f = pow2(pm[i] - base);
    l = __builtin_fmaf(pl[i], f, l);
    const float* po = A.part_o + (at * A.splits + i) * DIM;
#pragma unroll
    for (int c = 0; c < DIM / 64; ++c) acc[c] = __builtin_fmaf(po[c * 64 + lane], f, acc[c]);
  }
  if constexpr (WAVES == 1) {
#pragma unroll
    for (int c = 0; c < DIM / 64; ++c) store_out((T*)A.out + at * DIM + c * 64 + lane, l == 0.0f ? 0.0f : acc[c] / l);
    return;
  }
#pragma unroll
  for (int c = 0; c < DIM / 64; ++c) sum_o[wave][c * 64 + lane] = acc[c];
  if (lane == 0) sum_l[wave] = l;
  __syncthreads();
  l = (sum_l[0] + sum_l[1]) + (sum_l[2] + sum_l[3]);
  for (int c = threadIdx.x; c < DIM; c += 256) {
    const float o = (sum_o[0][c] + sum_o[1][c]) + (sum_o[2][c] + sum_o[3][c]);
    store_out((T*)A.out + at * DIM + c, l == 0.0f ? 0.0f : o / l);
  }
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------

struct Plan {
  bool many;          // the many-rows kernel
  int nt;             // columns / 16 of the few-rows kernel
  int rows;           // rows of a tile
  int64_t row_tiles;  // of a sequence and head, at most
  int64_t splits, chunk, blocks;
};

// Splits of many rows whose spans are alike, up to `most`: those of the least
// time by what was measured at 128 channels.  A tile takes a block 1.9 us where
// it has its unit to itself, 2.5 where two share one; splits cost 8 us, and
// their partial sums, written and read, go at 4 TB/s.  (42 heads of 128 over 6,
// 768 new tokens: 20 tiles 44 us whole and 59 halved, 68 tiles 127 and 115; 18
// new tokens 75 whole, 28 in four.)
int64_t many_splits(int64_t tiles, int64_t base, int64_t most, int64_t dim) {
  int64_t best = 1;
  double least = 0.0;
  for (int64_t n = 1; n <= most; ++n) {
    const double tile = (n * base <= 256 ? 1.9 : 2.5) * (double)dim / 128;
    const double sums = n == 1 ? 0.0 : 8.0 + (double)(n * base * kManyRows * dim * 8) / 4e6;
    const double time = (double)((tiles + n - 1) / n) * tile + sums;
    if (n == 1 || time < least) {
      best = n;
      least = time;
    }
  }
  return best;
}

Plan make_plan(int64_t heads_q, int64_t heads, int64_t page, int64_t batch, int64_t max_q, int64_t width,
               int64_t window, int64_t sinks, nvfp4_dtype_t dt, int64_t dim, bool split) {
  Plan p;
  const int64_t group = heads_q / heads, rows = max_q * group;
  p.many = dt != NVFP4_F32 && rows > 32;
  p.nt = rows <= 16 ? 1 : 2;
  p.rows = p.many ? kManyRows : 16 * p.nt;
  p.row_tiles = (rows + p.rows - 1) / p.rows;
  // the longest span of a tile of rows, from a tile boundary on
  int64_t span = width * page;
  if (window > 0 && window < span) {
    const int64_t front = sinks <= 0 ? 0 : sinks < span ? (sinks + 63) / 64 * 64 : span;
    const int64_t w = window - 1 + (p.rows + group - 1) / group + 1 + 63 + front;
    if (w < span) span = w;
  }
  const int64_t tiles = (span + 63) / 64, base = batch * heads * p.row_tiles;   // max_q * heads_q is at most 2^30
  p.splits = 1;
  p.chunk = (tiles > 0 ? tiles : 1) * 64;
  if (split) {
    // few rows: three rounds of blocks on the chip, and four tiles a wave at
    // least; many rows: one round, and eight tiles a block.  With sinks, which
    // go with a window that is short beside the sequences, spans are alike: few
    // rows then take the one round that comes nearest, and two tiles a wave (32
    // heads of 128 over 8, 4096 + 4 tokens: 64 sequences 98 us, 111 with three
    // rounds; 16 28.7 and 36; one 11.7 and 13.8; 16 of 6 tokens 36 and 54).
    // While sequences are shorter than the window theirs are not, and lengths
    // are not known here: with a table of 100000 tokens 16 of up to 4096, window
    // 4096, take 25.9 us and 23.1 with three rounds, of 6 tokens 34 and 39; 4 of
    // up to 4096, window 8192, 17.6 and 14.4; 64 of up to 8192, window 8192, 120
    // and 115, 32 (16 heads over 2) 25.5 and 24.4, of up to 2048 15.8 and 16.5.
    // Windows alone keep the three rounds, so that their results stay as they
    // are to the last bit: 64 sequences 108 us where the one round would take 99,
    // 16 36 and 28.5, one 14.0 and 11.6, 16 of 6 tokens 53 and 37.
    const bool alike = sinks > 0 && window > 0;
    const int64_t unit = p.many ? 1 : kFewWaves, least = p.many ? 8 : (alike ? 2 : 4) * kFewWaves;
    const int64_t round = 256 * few_blocks_per_cu((int)dim, p.nt, dt == NVFP4_F32 ? 3 : 1);
    const int64_t full = p.many ? (dim <= 64 ? 768 : 512) : alike ? round + base / 2 : 3 * 512 + base - 1;
    int64_t want = full / base;
    const int64_t most = (tiles + least - 1) / least;
    if (want > most) want = most;
    if (p.many && alike) want = many_splits(tiles, base, want, dim);
    if (want > 1) {
      p.chunk = ((tiles + want - 1) / want + unit - 1) / unit * unit * 64;
      p.splits = (tiles * 64 + p.chunk - 1) / p.chunk;
    }
  }
  p.blocks = base * p.splits;
  return p;
}

// A wave a row joins up to kFewSplits splits, a block a row more of them.
constexpr int64_t kFewSplits = 16;
int64_t join_blocks(const Plan& p, int64_t rows) { return p.splits == 1 ? 0 : p.splits <= kFewSplits ? (rows + 3) / 4 : rows; }

int64_t partials(const Plan& p, int64_t tokens, int64_t heads_q, int64_t dim) {
  return p.splits > 1 ? tokens * heads_q * p.splits * (dim + 2) * 4 : 0;
}

template <typename T, int DIM, int NT, bool SINKS>
bool launch_few(const AttnArgs& A, int64_t blocks, hipStream_t s) {
  constexpr int bytes = few_lds_bytes<DIM, NT, Mma<T>::kParts>();
  static_assert(bytes <= 160 * 1024, "LDS of a workgroup");
  if constexpr (bytes > 64 * 1024) {
    if (hipFuncSetAttribute((const void*)few_rows_kernel<T, DIM, NT, SINKS>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
      return false;
  }
  few_rows_kernel<T, DIM, NT, SINKS><<<dim3((uint32_t)blocks), dim3(64 * kFewWaves), bytes, s>>>(A);
  return true;
}

template <typename T, int DIM, bool ONE_PAGE, bool SINKS>
bool launch_many(const AttnArgs& A, int64_t blocks, hipStream_t s) {
  constexpr int bytes = (int)sizeof(ManyShared<DIM>);
  static_assert(bytes <= 160 * 1024, "LDS of a workgroup");
  if (bytes > 64 * 1024 &&
      hipFuncSetAttribute((const void*)many_rows_kernel<T, DIM, ONE_PAGE, SINKS>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
    return false;
  many_rows_kernel<T, DIM, ONE_PAGE, SINKS><<<dim3((uint32_t)blocks), dim3(64 * kManyWaves), bytes, s>>>(A);
  return true;
}

template <typename T, int DIM, bool SINKS>
bool launch_rows(const AttnArgs& A, const Plan& p, hipStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (p.many)
      return A.c.page_shift >= 6 ? launch_many<T, DIM, true, SINKS>(A, p.blocks, s) : launch_many<T, DIM, false, SINKS>(A, p.blocks, s);
  return p.nt == 1 ? launch_few<T, DIM, 1, SINKS>(A, p.blocks, s) : launch_few<T, DIM, 2, SINKS>(A, p.blocks, s);
}

template <typename T, int DIM>
void launch_dim(const AttnArgs& A, const Plan& p, hipStream_t s) {
  const bool ok = A.sinks > 0 ? launch_rows<T, DIM, true>(A, p, s) : launch_rows<T, DIM, false>(A, p, s);
  if (ok && p.splits > 1) {
    const dim3 grid((uint32_t)join_blocks(p, (int64_t)A.s.tokens * A.heads_q));
    if (p.splits <= kFewSplits) join_kernel<T, DIM, 1><<<grid, dim3(256), 0, s>>>(A, p.rows);
    else join_kernel<T, DIM, 4><<<grid, dim3(256), 0, s>>>(A, p.rows);
  }
}

template <typename T>
void launch_type(const AttnArgs& A, const Plan& p, int64_t dim, hipStream_t s) {
  switch (dim) {
    case 64: launch_dim<T, 64>(A, p, s); break;
    case 128: launch_dim<T, 128>(A, p, s); break;
    case 192: launch_dim<T, 192>(A, p, s); break;
    case 256: launch_dim<T, 256>(A, p, s); break;
  }
}

}  // namespace

namespace nvfp4host {

int64_t paged_attention_bytes(int64_t tokens, int64_t heads_q, int64_t heads, int64_t dim, int64_t page, int64_t batch,
                              int64_t max_q, int64_t width, int64_t window, int64_t sinks, nvfp4_dtype_t dt) {
  return (partials(make_plan(heads_q, heads, page, batch, max_q, width, window, sinks, dt, dim, true), tokens, heads_q, dim) + 255) / 256 * 256;
}

int64_t paged_attention_blocks(int64_t tokens, int64_t heads_q, int64_t heads, int64_t dim, int64_t page, int64_t batch,
                               int64_t max_q, int64_t width, int64_t window, int64_t sinks, nvfp4_dtype_t dt) {
  const Plan p = make_plan(heads_q, heads, page, batch, max_q, width, window, sinks, dt, dim, true);
  return std::max(p.blocks, join_blocks(p, tokens * heads_q));
}

void launch_paged_attention(const nvfp4_kv_cache_t& c, const void* q, int64_t q_token, int64_t q_head, int64_t heads_q,
                            nvfp4_dtype_t dt, int64_t tokens, const int32_t* cu, int64_t batch, int64_t max_q,
                            const int32_t* table, int64_t width, const int32_t* lens, int64_t window,
                            int64_t sinks, float scale, void* ws, int64_t ws_bytes, void* out, hipStream_t s) {
  Plan p = make_plan(heads_q, c.heads, c.page, batch, max_q, width, window, sinks, dt, c.dim, true);
  if (ws_bytes < partials(p, tokens, heads_q, c.dim)) p = make_plan(heads_q, c.heads, c.page, batch, max_q, width, window, sinks, dt, c.dim, false);
  AttnArgs A;
  A.c = {c.k, c.v, c.k_scales, c.v_scales, (int32_t)c.pages, (int32_t)c.heads, __builtin_ctz((unsigned)c.page)};
  A.s = {table, lens, cu, width, (int32_t)batch, (int32_t)tokens, (int32_t)max_q};
  A.q = q; A.q_token = q_token; A.q_head = q_head;
  A.out = out;
  if (c.pages == 0) A.s.width = 0;   // no page to read: nothing is seen
  const int64_t prow = tokens * heads_q * p.splits;
  A.part_o = (float*)ws;
  A.part_m = p.splits > 1 ? A.part_o + prow * c.dim : nullptr;
  A.part_l = p.splits > 1 ? A.part_m + prow : nullptr;
  A.heads_q = (int32_t)heads_q; A.group = (int32_t)(heads_q / c.heads);
  // none where it passes all positions; lengths may pass the table, so its size says nothing
  A.window = window <= 0 || window > INT_MAX ? 0 : (int32_t)window;
  A.sinks = A.window == 0 || sinks <= 0 ? 0 : (int32_t)std::min<int64_t>(sinks, INT_MAX);
  A.splits = (int32_t)p.splits; A.chunk = (int32_t)p.chunk;
  A.row_tiles = (int32_t)p.row_tiles;
  A.sign = scale < 0.0f ? -1.0f : 1.0f;
  A.scale_log2 = scale * A.sign * kLog2e;
  const int64_t size = dt == NVFP4_F32 ? 4 : 2;
  A.vec = ((uintptr_t)q & 15) == 0 && (q_token * size) % 16 == 0 && (q_head * size) % 16 == 0;
  switch (dt) {
    case NVFP4_F32: launch_type<float>(A, p, c.dim, s); break;
    case NVFP4_BF16: launch_type<__bf16>(A, p, c.dim, s); break;
    case NVFP4_F16: launch_type<_Float16>(A, p, c.dim, s); break;
  }
}

}  // namespace nvfp4host
