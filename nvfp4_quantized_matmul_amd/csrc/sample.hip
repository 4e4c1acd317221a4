// One token per row of logits: temperature, top-k, top-p and min-p, then the
// inverse of the kept weights' running sum at a given random number.
//
// The kept tokens are a prefix of the order (logit falling, index rising), so
// they are told by the last kept logit and, among the tokens that share it, by
// the last kept index.  The row is not sorted.  The distance of a logit from
// the largest, over the row's range, gives one of 2048 bins; a histogram of
// number and weight tells the bins in which top-k and top-p end, and only
// those bins' tokens (some hundreds of a quarter of a million) are gathered,
// sorted and walked.  A row whose border bins hold more than 2048 tokens, as
// where most logits are equal, and one with an infinite largest logit are
// searched by the bits of the logit instead, in one block (row_by_digits).
//
// A row of at most eight rounds of its block's 16-byte loads runs in one block
// and launch if top-k or top-p are asked for: latency counts there.  Others are
// cut into tiles of that size, or smaller while blocks are few, in three or
// five launches (range; histogram and gathering; sums; choice).
//
// Bound by the vector units, 64-bit arithmetic most of it: one row of 32000
// float32 logits with all filters 40 us (the search by digits in one block 53
// us), 16 rows of 50001 f16 logits with min-p 19 us, 64 rows of 262144 bf16 logits 106 us (488 us), of which reading them
// once would be 7: 8 for the range, 28 for the histogram, 28 for gathering, 34
// for the sums, 11 for the choice.
//
// With a quarter of a million tokens a probability is a millionth and the
// place of u among them is decided in the 7th digit and beyond, so weights (good
// to 1e-11) and running sums are in 64 bits.  A histogram's sums are integers,
// which add up the same in any order; everything else is added in a fixed order.
// The place of top-p's border comes from them: with bins a token's weight is
// rounded to 2^-32 of its bin's largest, so that the sums are good to 2e-10;
// by digits to 2^-(62 - bits of the vocabulary), good to vocabulary^2 2^-62 of a
// row's sum (1.5e-8 for a quarter of a million, 2e-10 for 32000).
#include "nvfp4_device.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

constexpr int kThreads = 1024, kWaves = kThreads / 64, kBits = 11, kBins = 1 << kBits;

struct SampleArgs {
  const void* logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* token;
  float* prob;
  int64_t row_stride;
  int32_t vocab;
  int32_t fix;   // fraction bits of the histogram's weights
};

template <typename T>
struct KeyBits;   // significant bits of a type's ordered key
template <>
struct KeyBits<float> { static constexpr int n = 32; };
template <>
struct KeyBits<__bf16> { static constexpr int n = 16; };
template <>
struct KeyBits<_Float16> { static constexpr int n = 19; };   // sign, 8 exponent bits of the float, 10 of mantissa

// NaN counts as -inf, -0 as +0.
__device__ __forceinline__ float clean(float x) { return x != x ? -__builtin_inff() : x + 0.0f; }

// Rises with x; equal for equal values only.
template <typename T>
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = fbits(x);
  return (b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) >> (32 - KeyBits<T>::n);
}

// 2^y, y in [-kFar, kFar]: the power of two of the nearest integer and the
// Taylor sum of the rest to its 9th power, whose first left-out term is below
// 1e-11 of the sum.
constexpr double kFar = 1080.0;   // weights below 2^-kFar are 0
__device__ __forceinline__ double exp2_64(double y) {
  const double n = __builtin_rint(y), f = (y - n) * 0.69314718055994530942;
  double p = 1.0 / 362880.0;
  p = __builtin_fma(p, f, 1.0 / 40320.0);
  p = __builtin_fma(p, f, 1.0 / 5040.0);
  p = __builtin_fma(p, f, 1.0 / 720.0);
  p = __builtin_fma(p, f, 1.0 / 120.0);
  p = __builtin_fma(p, f, 1.0 / 24.0);
  p = __builtin_fma(p, f, 1.0 / 6.0);
  p = __builtin_fma(p, f, 0.5);
  p = __builtin_fma(p, f, 1.0);
  p = __builtin_fma(p, f, 1.0);
  return __builtin_ldexp(p, (int)n);
}

// The same as a call: most of a short row's time goes to fetching
// instructions that run once, so what is off the loops is kept small.
__device__ __noinline__ double exp2_call(double y) { return exp2_64(y); }

// log2(e) / temperature, never negative: weights are at most 1, and their sums
// in 62 bits do not wrap.
__device__ __forceinline__ double rate_of(const SampleArgs& A, int row) {
  const double t = A.temperature ? (double)A.temperature[row] : 1.0;
  return t > 0.0 ? 1.44269504088896340736 / t : __builtin_inf();
}

// exp((x - top) / temperature), with rate = log2(e) / temperature.
__device__ __forceinline__ double weight(float x, float top, double rate) {
  if (x == top) return 1.0;
  const double y = ((double)x - (double)top) * rate;
  if (!(y > -kFar)) return 0.0;
  return exp2_64(y);
}

struct Shared {
  uint32_t count[kBins];
  unsigned long long mass[kBins];
  uint32_t wave_count[kWaves];
  unsigned long long wave_mass[kWaves];
  double part[kWaves];
  uint32_t bin, bin_count;
  unsigned long long before;
};

template <typename V>
__device__ __forceinline__ V wave_inclusive(V v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const V o = __shfl_up(v, off, 64);
    if ((int)(threadIdx.x & 63) >= off) v += o;
  }
  return v;
}

// The bin, from the top down, in which the sum before it is still below
// `target` and the sum with it is not: into S.bin, the sum before it into
// S.before.  There is one, as before0 is below the target and the whole is not,
// and conversions to double keep the order.  `value` gives a bin's amount; bins
// 2 t and 2 t + 1 from the top are thread t's.
template <typename F>
__device__ void find_bin(Shared& S, double target, const F& value, unsigned long long before0) {
  static_assert(kBins == 2 * kThreads, "two bins a thread");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b0 = kBins - 1 - 2 * tid, b1 = b0 - 1;
  const unsigned long long v0 = value(b0), v1 = value(b1);
  const unsigned long long incl = wave_inclusive<unsigned long long>(v0 + v1);
  if (lane == 63) S.wave_mass[wave] = incl;
  __syncthreads();
  unsigned long long before = before0;
  for (int w = 0; w < wave; ++w) before += S.wave_mass[w];
  before += incl - v0 - v1;
  if (v0 && (double)before < target && (double)(before + v0) >= target) { S.bin = b0; S.before = before; }
  const unsigned long long mid = before + v0;
  if (v1 && (double)mid < target && (double)(mid + v1) >= target) { S.bin = b1; S.before = mid; }
  __syncthreads();
}

// Narrows [lo, hi) to the first index whose running sum of f passes a target:
// share * (whole sum) at first, with 0 <= share < 1, or `fixed` if share < 0.
// Returns the index (-1 if f is nowhere positive); the whole sum into *whole.
template <typename F>
__device__ int narrow(Shared& S, const F& f, int lo, int hi, double share, double fixed, double* whole) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double before = 0.0, target = fixed;
  bool first = true;
  while (first || hi - lo > 64) {
    const int part = ((hi - lo + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int from = lo + wave * part;
    const int to = from + part < hi ? from + part : hi;
    double s = 0.0;
    for (int i = from + lane; i < to; i += 64) s += f(i);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
    if (lane == 0) S.part[wave] = s;
    __syncthreads();
    if (first) {
      double all = 0.0;
      for (int w = 0; w < kWaves; ++w) all += S.part[w];
      *whole = all;
      if (share >= 0.0) target = share * all;
      if (!(all > 0.0)) { __syncthreads(); return -1; }
      first = false;
    }
    int pick = -1, last = -1;
    double acc = before, acc_last = before;
    for (int w = 0; w < kWaves; ++w) {
      const double v = S.part[w];
      if (v > 0.0) { last = w; acc_last = acc; }
      if (pick < 0 && v > 0.0 && acc + v > target) { pick = w; before = acc; }
      acc += v;
    }
    if (pick < 0) { pick = last; before = acc_last; }
    if (pick < 0) pick = 0;
    __syncthreads();
    lo += pick * part;
    hi = lo + part < hi ? lo + part : hi;
  }
  const double v = lo + lane < hi ? f(lo + lane) : 0.0;
  const double run = before + wave_inclusive<double>(v);
  const uint64_t over = __ballot(v > 0.0 && run > target), some = __ballot(v > 0.0);
  return over ? lo + __builtin_ctzll(over) : some ? lo + 63 - __builtin_clzll(some) : -1;
}

// ---------------------------------------------------------------------------
// A row by the digits of its keys, in one block
// ---------------------------------------------------------------------------
//
// A logit's bits as an ordered key are searched digit by digit, from the top,
// through a histogram of the tokens whose higher digits agree: of their number
// for top-k, of their weight for top-p.  Right for any row, at several passes
// over it by one block.
template <typename T>
__device__ __noinline__ void row_by_digits(const SampleArgs& A, Shared& S, int row) {
  const int tid = threadIdx.x, V = A.vocab;
  const T* x = (const T*)A.logits + (int64_t)row * A.row_stride;

  uint32_t top_key = 0;
  for (int i = tid; i < V; i += kThreads) {
    const uint32_t k = key_of<T>(clean((float)x[i]));
    top_key = k > top_key ? k : top_key;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top_key, off, 64);
    top_key = o > top_key ? o : top_key;
  }
  if ((tid & 63) == 0) S.wave_count[tid >> 6] = top_key;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) top_key = S.wave_count[w] > top_key ? S.wave_count[w] : top_key;
  const uint32_t full = top_key << (32 - KeyBits<T>::n);
  // the largest logit, from its key (the low bits that a 2-byte type lacks are
  // zero in a value that is not negative, and one before the complement in one that is)
  const uint32_t low = KeyBits<T>::n == 32 ? 0u : (1u << (32 - KeyBits<T>::n)) - 1u;
  const float top = (full >> 31) ? __builtin_bit_cast(float, full ^ 0x80000000u) : __builtin_bit_cast(float, ~(full | low));
  if (top == -__builtin_inff()) {
    if (tid == 0) {
      A.token[row] = -1;
      if (A.prob) A.prob[row] = 0.0f;
    }
    return;
  }
  auto at = [&](int i) -> float { return clean((float)x[i]); };
  const double rate = rate_of(A, row);
  int k = A.top_k ? A.top_k[row] : 0;
  double p = A.top_p ? (double)A.top_p[row] : 1.0;
  const double floor_w = A.min_p ? (double)A.min_p[row] : 0.0;
  if (!(floor_w <= 1.0)) k = 1;   // above the first one's own weight: it stays alone
  const double unit = __builtin_ldexp(1.0, A.fix);
  auto fixed_weight = [&](float v) -> unsigned long long { return (unsigned long long)(weight(v, top, rate) * unit + 0.5); };

  // the last kept key, and how many of the tokens that have it are kept
  uint32_t last_key = 0;
  uint32_t take = 0xffffffffu, ties = 0;
  constexpr int N = KeyBits<T>::n;
  if (k > 0 && k < V) {
    uint32_t prefix = 0;
    unsigned long long before = 0;
    for (int left = N; left > 0;) {
      const int bits = left < kBits ? left : kBits, shift = left - bits;
      for (int i = tid; i < kBins; i += kThreads) S.count[i] = 0;
      __syncthreads();
      for (int i = tid; i < V; i += kThreads) {
        const uint32_t key = key_of<T>(at(i));
        if (left == N || (key >> left) == prefix) atomicAdd(&S.count[(key >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      find_bin(S, (double)k, [&](int b) -> unsigned long long { return S.count[b]; }, before);
      prefix = (prefix << bits) | S.bin;
      before = S.before;
      ties = S.count[S.bin];
      left = shift;
      __syncthreads();
    }
    last_key = prefix;
    take = (uint32_t)(k - (int)before);
  }
  if (!(p >= 1.0)) {
    uint32_t prefix = 0, count = 0;
    unsigned long long before = 0;
    double target = 0.0;
    for (int left = N; left > 0;) {
      const int bits = left < kBits ? left : kBits, shift = left - bits;
      for (int i = tid; i < kBins; i += kThreads) { S.count[i] = 0; S.mass[i] = 0; }
      __syncthreads();
      for (int i = tid; i < V; i += kThreads) {
        const float v = at(i);
        const uint32_t key = key_of<T>(v);
        if (key >= last_key && (left == N || (key >> left) == prefix)) {
          const uint32_t b = (key >> shift) & ((1u << bits) - 1u);
          atomicAdd(&S.count[b], 1u);
          // of the tokens with the last key only `take` weigh; they are added below
          if (key > last_key || take == 0xffffffffu) atomicAdd(&S.mass[b], fixed_weight(v));
        }
      }
      __syncthreads();
      if (tid == 0 && take != 0xffffffffu && (left == N || (last_key >> left) == prefix)) {
        const uint32_t fk = last_key << (32 - N);
        const float v = (fk >> 31) ? __builtin_bit_cast(float, fk ^ 0x80000000u) : __builtin_bit_cast(float, ~(fk | low));
        S.mass[(last_key >> shift) & ((1u << bits) - 1u)] += take * fixed_weight(v);
      }
      __syncthreads();
      if (left == N) {
        // target: top_p of the whole; below half a unit the first token alone
        unsigned long long m = S.mass[2 * tid] + S.mass[2 * tid + 1];
        m = wave_inclusive<unsigned long long>(m);
        if ((tid & 63) == 63) S.wave_mass[tid >> 6] = m;
        __syncthreads();
        unsigned long long all = 0;
        for (int w = 0; w < kWaves; ++w) all += S.wave_mass[w];
        target = p * (double)all;
        target = target > 0.5 ? target : 0.5;
        __syncthreads();
      }
      find_bin(S, target, [&](int b) -> unsigned long long { return S.mass[b]; }, before);
      prefix = (prefix << bits) | S.bin;
      before = S.before;
      count = S.count[S.bin];
      left = shift;
      __syncthreads();
    }
    // tokens of the last key: the j-th (from 0) stays while before + j w < target
    const uint32_t fk = prefix << (32 - N);
    const float v = (fk >> 31) ? __builtin_bit_cast(float, fk ^ 0x80000000u) : __builtin_bit_cast(float, ~(fk | low));
    const double w = (double)fixed_weight(v);
    uint32_t stay = count;
    if (w > 0.0) {
      const double need = __builtin_ceil((target - (double)before) / w);
      stay = need < 1.0 ? 1u : need < (double)count ? (uint32_t)need : count;
    }
    if (prefix == last_key && take < stay) stay = take;
    last_key = prefix;
    take = stay;
    ties = count;
  }
  // the index of the last kept token among those that share the last key
  int last_index = V;
  double whole;
  if (take < ties)
    last_index = narrow(S, [&](int i) -> double { return key_of<T>(at(i)) == last_key ? 1.0 : 0.0; }, 0, V, -1.0,
                        (double)take - 0.5, &whole);
  auto kept = [&](int i) -> double {
    const float v = at(i);
    const uint32_t key = key_of<T>(v);
    if (key < last_key || (key == last_key && i > last_index)) return 0.0;
    const double w = weight(v, top, rate);
    return w >= floor_w || key == top_key ? w : 0.0;
  };
  const int pick = narrow(S, kept, 0, V, (double)A.u[row], 0.0, &whole);
  if (tid == 0) {
    A.token[row] = pick;
    if (A.prob) A.prob[row] = (float)(kept(pick) / whole);
  }
}

// ---------------------------------------------------------------------------
// A row by bins of its logits
// ---------------------------------------------------------------------------

constexpr int kNB = 2048;          // bins
constexpr int kStripes = 8;        // rounds of 16-byte loads of a tile, at most
constexpr int kCands = 2048;       // tokens of the border bins, at most
constexpr int kMaxTiles = 64;      // of a row
constexpr int kParts = kStripes * kWaves;
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);
template <typename T>
constexpr int kStripe = kThreads * kVec<T>;   // tokens of a round

// A histogram's entry: the number of tokens from bit 47 on, and below it the
// sum of 1 - 2^-f in units of 2^-32, where 2^-f is the token's weight relative
// to the largest one of its bin.  With at most 65536 tokens and f at most 1080
// / 2047 (2^-f above 0.69) neither passes its bits.
constexpr int kCountBit = 47;

struct Settings {
  double rate, p, floor_w;
  int k;
  bool ordered;   // top-k or top-p leaves tokens out
};

__device__ __forceinline__ Settings settings(const SampleArgs& A, int row) {
  Settings s;
  s.rate = rate_of(A, row);
  s.p = A.top_p ? (double)A.top_p[row] : 1.0;
  s.p = s.p == s.p ? s.p : 0.0;
  s.floor_w = A.min_p ? (double)A.min_p[row] : 0.0;
  s.k = A.top_k ? A.top_k[row] : 0;
  if (!(s.floor_w <= 1.0)) s.k = 1;   // above the first one's own weight: it stays alone
  s.ordered = (s.k > 0 && s.k < A.vocab) || s.p < 1.0;
  return s;
}

// How the row's logits fall into bins.
struct Bins {
  float top;
  double rate, per_unit, unit;   // bins per power of two, and its inverse
  bool digits;                   // the row takes the other way
};

__device__ __forceinline__ Bins bins_of(float top, float least, double rate) {
  Bins b;
  b.top = top;
  b.rate = rate;
  double range = ((double)top - (double)least) * rate;
  range = range < kFar ? range : kFar;   // also what is not a number: the least one at the top, at temperature 0
  b.per_unit = range > 0.0 ? (kNB - 1) / range : 0.0;
  b.per_unit = b.per_unit < 1e100 ? b.per_unit : 1e100;
  b.unit = b.per_unit > 0.0 ? 1.0 / b.per_unit : 0.0;
  b.digits = top == __builtin_inff();
  return b;
}

// The distance of x from the top in powers of two; past kFar the token has no weight.
__device__ __forceinline__ double distance(const Bins& b, float x) { return x == b.top ? 0.0 : ((double)b.top - (double)x) * b.rate; }
__device__ __forceinline__ int bin_of(const Bins& b, double y) {
  const int i = (int)(y * b.per_unit);
  return i < kNB - 1 ? i : kNB - 1;
}

// Rises with the token's place in the order, from the last to the first; 0 is no token's.
__device__ __forceinline__ unsigned long long place_of(float x, int i) {
  const uint32_t b = fbits(x);
  return ((unsigned long long)(b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u)) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float logit_of(unsigned long long place) {
  const uint32_t k = (uint32_t)(place >> 32);
  return __builtin_bit_cast(float, (k >> 31) ? k ^ 0x80000000u : ~k);
}

struct Borders {
  int bk;                        // the bin in which top-k ends; kNB: none
  uint32_t rest;                 // tokens that top-k keeps of it
  int lo, hi;                    // the bins in one of which top-p ends; lo > hi: none
  uint32_t cands;                // tokens of all these bins
  double before_k, before_lo, total;
};

struct Fast {
  unsigned long long hist[kNB];
  unsigned long long cand[kCands];
  double part[kParts];
  double wave[kWaves];
  uint32_t wave_n[kWaves];
  float wave_f[2][kWaves];
  Borders b;
  uint32_t count;
  int32_t first;
};
union AnyShared {
  Shared digits;
  Fast fast;
  __device__ AnyShared() {}
};

// Eight or four logits from index i on, -inf behind the end; `take` gives the
// first one and moves the others up, so that loops over them stay rolled.
template <typename T>
struct Piece {
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* row, int i, int V) {
    if (i + kVec<T> <= V) {
      __builtin_memcpy(w, row + i, 16);
    } else {
      T x[kVec<T>];
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) x[e] = i + e < V ? row[i + e] : (T)(-__builtin_inff());
      __builtin_memcpy(w, x, 16);
    }
  }
  // logit e as it is
  __device__ __forceinline__ float raw(int e) const {
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(float, w[e]);
    else return (float)__builtin_bit_cast(T, (uint16_t)(w[e / 2] >> (16 * (e % 2))));
  }
  __device__ __forceinline__ float take() {
    if constexpr (sizeof(T) == 4) {
      const float x = __builtin_bit_cast(float, w[0]);
      w[0] = w[1]; w[1] = w[2]; w[2] = w[3];
      return clean(x);
    } else {
      const float x = (float)__builtin_bit_cast(T, (uint16_t)w[0]);
      w[0] = __builtin_amdgcn_alignbit(w[1], w[0], 16);
      w[1] = __builtin_amdgcn_alignbit(w[2], w[1], 16);
      w[2] = __builtin_amdgcn_alignbit(w[3], w[2], 16);
      w[3] >>= 16;
      return clean(x);
    }
  }
};

// f(piece, index) for the block's tokens [from, to); the next round's load is
// in flight while this round's are worked on.  end(round) after each round.
template <typename T, typename F, typename E>
__device__ __forceinline__ void each_piece(const T* row, int from, int to, const F& f, const E& end) {
  Piece<T> next;
  int i = from + (int)threadIdx.x * kVec<T>;
  next.load(row, i, to);
  for (int j = 0, base = from; base < to; ++j, base += kStripe<T>, i += kStripe<T>) {
    Piece<T> now = next;
    if (base + kStripe<T> < to) next.load(row, i + kStripe<T>, to);
    f(now, i);
    end(j);
  }
}
struct Nothing {
  __device__ void operator()(int) const {}
};

// The largest and the least of all threads' values.
__device__ __forceinline__ void block_range(float& hi, float& lo, Fast& S) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    hi = fmaxf(hi, __shfl_xor(hi, off, 64));
    lo = fminf(lo, __shfl_xor(lo, off, 64));
  }
  __syncthreads();
  if (lane == 0) { S.wave_f[0][wave] = hi; S.wave_f[1][wave] = lo; }
  __syncthreads();
  hi = S.wave_f[0][lane & (kWaves - 1)];
  lo = S.wave_f[1][lane & (kWaves - 1)];
#pragma unroll
  for (int off = kWaves / 2; off > 0; off >>= 1) {
    hi = fmaxf(hi, __shfl_xor(hi, off, 64));
    lo = fminf(lo, __shfl_xor(lo, off, 64));
  }
}

// The tile's largest logit and the least one that has weight beside it.
template <typename T>
__device__ void tile_range(const T* row, int from, int to, double rate, Fast& S, float* top, float* least) {
  float hi = -__builtin_inff(), lo = __builtin_inff();
  each_piece<T>(row, from, to, [&](const Piece<T>& p, int) {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
      const float x = p.raw(e);
      hi = fmaxf(hi, x);   // NaN is passed over by both
      lo = x > -__builtin_inff() ? fminf(lo, x) : lo;
    }
  }, Nothing());
  block_range(hi, lo, S);
  if (((double)hi - (double)lo) * rate > kFar) {
    // logits masked by a large negative number, or a low temperature: the
    // least of those that weigh (the limit's rounding to 32 bits keeps them)
    const float limit = (float)((double)hi - kFar * 1.0001 / rate);
    float in = hi;
    each_piece<T>(row, from, to, [&](const Piece<T>& p, int) {
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) in = p.raw(e) >= limit ? fminf(in, p.raw(e)) : in;
    }, Nothing());
    lo = in;
    block_range(hi, lo, S);
  }
  *top = hi;
  *least = lo;
}

template <typename T>
__device__ void tile_histogram(const T* row, int from, int to, const Bins& b, Fast& S) {
  for (int i = threadIdx.x; i < kNB; i += kThreads) S.hist[i] = 0;
  __syncthreads();
  const bool narrow_bins = b.unit < 0.03 / 0.69314718055994530942;
  each_piece<T>(row, from, to, [&](Piece<T>& p, int) {
#pragma unroll 1
    for (int e = 0; e < kVec<T>; ++e) {
      const double y = distance(b, p.take());
      if (y <= kFar) {
        const int i = bin_of(b, y);
        double f = __builtin_fma(-(double)i, b.unit, y) * 0.69314718055994530942;
        f = f > 0.0 ? f : 0.0;
        // 1 - e^-f by its Taylor sum: what is left out is below 0.366^10 / 10! =
        // 1.2e-11, or 0.03^6 / 6! = 1e-12 where the bins are narrow
        double d = 1.0 / 120.0;
        if (!narrow_bins) {
          d = 1.0 / 362880.0;
          d = __builtin_fma(d, -f, 1.0 / 40320.0);
          d = __builtin_fma(d, -f, 1.0 / 5040.0);
          d = __builtin_fma(d, -f, 1.0 / 720.0);
          d = __builtin_fma(d, -f, 1.0 / 120.0);
        }
        d = __builtin_fma(d, -f, 1.0 / 24.0);
        d = __builtin_fma(d, -f, 1.0 / 6.0);
        d = __builtin_fma(d, -f, 0.5);
        d = __builtin_fma(d, -f, 1.0);
        d *= f;
        atomicAdd(&S.hist[i], (1ull << kCountBit) + (uint32_t)(d * 4294967296.0 + 0.5));
      }
    }
  }, Nothing());
  __syncthreads();
}

// The sum of a value of every thread before this one, and of all.
template <typename V>
__device__ __forceinline__ V block_before(V v, V* shared, V* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const V incl = wave_inclusive<V>(v);
  __syncthreads();
  if (lane == 63) shared[wave] = incl;
  __syncthreads();
  // each lane of a row of 16 adds up the waves' sums in the same order
  const V mine = shared[lane & (kWaves - 1)];
  V run = mine;
#pragma unroll
  for (int off = 1; off < kWaves; off <<= 1) {
    const V o = __shfl_up(run, off, kWaves);
    if ((lane & (kWaves - 1)) >= off) run += o;
  }
  *all = __shfl(run, kWaves - 1, 64);
  const V before = wave > 0 ? __shfl(run, wave > 0 ? wave - 1 : 0, 64) : (V)0;
  return before + (incl - v);
}

// The lanes that have a value (>= 0) have rising ones: the last of them counts.
__device__ __forceinline__ void last_of(int* shared, int v) {
  const uint64_t has = __ballot(v >= 0);
  if (has && (int)(threadIdx.x & 63) == 63 - __builtin_clzll(has)) atomicMax(shared, v);
}

// Finds the borders' bins from the numbers and integer deficits of bins 2 tid
// and 2 tid + 1.
__device__ void find_borders(const Settings& set, const Bins& b, const uint32_t (&n)[2], const unsigned long long (&deficit)[2], Fast& S) {
  static_assert(kNB == 2 * kThreads, "two bins a thread");
  const int tid = threadIdx.x;
  double mass[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    mass[i] = n[i] ? ((double)n[i] - (double)deficit[i] * (1.0 / 4294967296.0)) * exp2_call(-(double)(2 * tid + i) * b.unit) : 0.0;
  uint32_t all_n;
  double all;
  const uint32_t n_before = block_before<uint32_t>(n[0] + n[1], S.wave_n, &all_n);
  const double before = block_before<double>(mass[0] + mass[1], S.wave, &all);
  if (tid == 0) {
    S.b.bk = kNB;
    S.b.rest = 0;
    S.b.before_k = all;
    S.b.lo = set.p < 1.0 ? 0 : kNB;
    S.b.hi = set.p < 1.0 ? 0 : -1;
    S.b.before_lo = 0.0;
    S.b.total = all;
  }
  __syncthreads();
  double low = all, high = all;   // what the first k tokens weigh lies between
  if (set.k > 0 && (uint32_t)set.k < all_n) {
    uint32_t nb = n_before;
    double mb = before;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (nb < (uint32_t)set.k && (uint32_t)set.k <= nb + n[i]) {
        S.b.bk = 2 * tid + i;
        S.b.rest = (uint32_t)set.k - nb;
        S.b.before_k = mb;
      }
      nb += n[i];
      mb += mass[i];
    }
    __syncthreads();
    low = S.b.before_k + S.b.rest * exp2_call(-(double)(S.b.bk + 1) * b.unit);
    high = S.b.before_k + S.b.rest * exp2_call(-(double)S.b.bk * b.unit);
  }
  if (set.p < 1.0) {
    // with room for the roundings of both sides: a bin more is only gathered
    // for nothing.  The last bin that starts below a target is the border's.
    const double t_low = set.p * low * (1.0 - 1e-9), t_high = set.p * high * (1.0 + 1e-9);
    double mb = before;
    int lo = -1, hi = -1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (n[i] && mb < t_low) lo = 2 * tid + i;
      if (n[i] && mb < t_high) hi = 2 * tid + i;
      mb += mass[i];
    }
    last_of(&S.b.lo, lo);
    last_of(&S.b.hi, hi);
    __syncthreads();
    if (tid == 0 && S.b.hi > S.b.bk) S.b.hi = S.b.bk;
    if (tid == 0 && S.b.lo > S.b.bk) S.b.lo = S.b.bk;
    __syncthreads();
    if (S.b.lo / 2 == tid) S.b.before_lo = S.b.lo & 1 ? before + mass[0] : before;
  }
  const int lo = S.b.lo, hi = S.b.hi, bk = S.b.bk;
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = 2 * tid + i;
    if ((at >= lo && at <= hi) || at == bk) mine += n[i];
  }
  uint32_t cands;
  block_before<uint32_t>(mine, S.wave_n, &cands);
  if (tid == 0) {
    S.b.cands = cands;
    S.count = 0;
  }
  __syncthreads();
}

// An interval that holds every logit of the bins [lo, hi], nothing if lo > hi.
// In 64 bits the edges are off by parts of 10^-15; rounding to 32 bits keeps
// the order, so a float inside stays inside.
__device__ __forceinline__ void logits_of_bins(const Bins& b, int lo, int hi, float* least, float* most) {
  *least = __builtin_inff();
  *most = -__builtin_inff();
  if (lo > hi) return;
  const double per_logit = b.rate * b.per_unit;
  if (!(per_logit > 0.0 && per_logit < 1e300)) {   // all logits in one bin, or as good as equal
    *least = -__builtin_inff();
    *most = __builtin_inff();
    return;
  }
  const double room = 1e-12 * (1.0 + lo + hi) / per_logit + 1e-12 * __builtin_fabs((double)b.top);
  *most = (float)((double)b.top - lo / per_logit + room);
  *least = hi >= kNB - 1 ? -__builtin_inff() : (float)((double)b.top - (hi + 1) / per_logit - room);
}

// Gathers the tile's tokens of the borders' bins into S.cand, in any order,
// and their number into S.count.
template <typename T>
__device__ void tile_gather(const T* row, int from, int to, const Bins& b, Fast& S) {
  const int lo = S.b.lo, hi = S.b.hi, bk = S.b.bk;
  // the logits between which these bins lie, and a little more: most pieces
  // need no further look.  The last bin is open downwards.
  float from_p, to_p, from_k, to_k;
  logits_of_bins(b, lo, hi, &from_p, &to_p);
  logits_of_bins(b, bk, bk < kNB ? bk : -1, &from_k, &to_k);
  each_piece<T>(row, from, to, [&](Piece<T>& p, int i0) {
    const auto near = [&](float x) { return (x >= from_p && x <= to_p) || (x >= from_k && x <= to_k); };
    bool any = false;
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) any |= near(p.raw(e));
    if (!any) return;
#pragma unroll 1
    for (int e = 0; e < kVec<T>; ++e) {
      const float x = p.take();
      if (!near(x)) continue;
      const double y = distance(b, x);
      const int bin = y <= kFar ? bin_of(b, y) : kNB;
      if ((bin >= lo && bin <= hi) || (bin == bk && bk < kNB)) {
        const uint32_t at = atomicAdd(&S.count, 1u);
        if (at < (uint32_t)kCands) S.cand[at] = place_of(x, i0 + e);
      }
    }
  }, Nothing());
  __syncthreads();
}

// Sorts the n gathered tokens into their order and returns the place of the
// last kept one; tokens at or above it stay.
__device__ unsigned long long last_kept(const Settings& set, const Bins& b, Fast& S, uint32_t n) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (n <= 256) {
    // a token's place among so few is the number of those before it
    unsigned long long mine = 0;
    uint32_t rank = 0;
    if ((uint32_t)tid < n) {
      mine = S.cand[tid];
      for (uint32_t i = 0; i < n; ++i) rank += S.cand[i] > mine ? 1u : 0u;
    }
    __syncthreads();
    if ((uint32_t)tid < n) S.cand[rank] = mine;
    __syncthreads();
  } else {
    int size = 512;
    while (size < (int)n) size *= 2;
    for (int i = n + tid; i < size; i += kThreads) S.cand[i] = 0;
    __syncthreads();
    for (int run = 2; run <= size; run *= 2)
      for (int step = run / 2; step > 0; step /= 2) {
        if (tid < size / 2) {
          const int i = 2 * tid - (tid & (step - 1)), j = i + step;
          const unsigned long long x = S.cand[i], y = S.cand[j];
          const bool falling = (i & run) == 0;
          if ((x < y) == falling) { S.cand[i] = y; S.cand[j] = x; }
        }
        __syncthreads();
      }
  }
  const Borders at = S.b;
  // two tokens a thread, their running sums in order
  constexpr int PER = kCands / kThreads;
  double w[PER], sum = 0.0, sum_k = 0.0;
  int bin[PER];
  uint32_t above_k = 0;   // gathered tokens before top-k's bin
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const uint32_t i = PER * tid + e;
    const float x = i < n ? logit_of(S.cand[i]) : 0.0f;
    bin[e] = i < n ? bin_of(b, distance(b, x)) : kNB;
    w[e] = 0.0;
    if (i < n) w[e] = exp2_call(-distance(b, x));   // all gathered ones weigh
    above_k += bin[e] < at.bk ? 1u : 0u;
    sum += w[e];
  }
  uint32_t first_k;
  block_before<uint32_t>(above_k, S.wave_n, &first_k);
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const uint32_t i = PER * tid + e;
    if (i >= first_k && i - first_k < at.rest) sum_k += w[e];
  }
  double all_k, all;
  block_before<double>(sum_k, S.wave, &all_k);
  const double before = at.before_lo + block_before<double>(sum, S.wave, &all);
  unsigned long long place = 0;
  if (at.bk < kNB) place = S.cand[first_k + at.rest - 1];
  if (set.p < 1.0) {
    const double target = set.p * (at.bk < kNB ? at.before_k + all_k : at.total);
    if (tid == 0) S.first = -1;
    __syncthreads();
    double mb = before;
    int last = -1;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const uint32_t i = PER * tid + e;
      if (i < n && bin[e] <= at.hi && (mb < target || (i == 0 && at.lo == 0))) last = (int)i;
      mb += w[e];
    }
    last_of(&S.first, last);
    __syncthreads();
    // none: the border is the start of the first bin, and all of it goes
    const unsigned long long by_p = S.first >= 0 ? S.cand[S.first] : S.cand[0] + 1;
    place = by_p > place ? by_p : place;
  }
  __syncthreads();
  return place;
}

__device__ __forceinline__ double kept_weight(const Bins& b, unsigned long long last, double floor_w, float x, int i) {
  if (x == -__builtin_inff() || place_of(x, i) < last) return 0.0;
  const double w = weight(x, b.top, b.rate);
  return w >= floor_w || x == b.top ? w : 0.0;
}

// The kept weights' sum of each round and wave of a tile, into part.
template <typename T>
__device__ void tile_sums(const T* row, int from, int to, const Bins& b, unsigned long long last, double floor_w, double* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double sum = 0.0;
  // no token below `least` is kept: most pieces need no further look.  The
  // logarithm is good to 1e-6.
  float least = last ? logit_of(last) : -__builtin_inff();
  if (floor_w > 0.0) {
    const double far = -(double)__builtin_amdgcn_logf((float)floor_w);
    least = fmaxf(least, fminf(b.top, (float)((double)b.top - (far * 1.0001 + 1e-4) / b.rate)));
  }
  each_piece<T>(row, from, to, [&](Piece<T>& p, int i0) {
    bool any = false;
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) any |= p.raw(e) >= least;
    if (!any) return;
#pragma unroll 1
    for (int e = 0; e < kVec<T>; ++e) {
      const float x = p.take();
      if (x >= least) sum += kept_weight(b, last, floor_w, x, i0 + e);
    }
  }, [&](int j) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane == 0) part[j * kWaves + wave] = sum;
    sum = 0.0;
  });
}

// The first token whose running sum passes u times the whole, from the sums of
// all the row's parts, each of 64 kVec tokens.
template <typename T>
__device__ void pick(const SampleArgs& A, const T* x, const Bins& b, unsigned long long last, double floor_w, double u,
                     const double* part, int parts, Fast& S, int row) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int per = (parts + kThreads - 1) / kThreads;
  const int p0 = tid * per < parts ? tid * per : parts, p1 = p0 + per < parts ? p0 + per : parts;
  double sum = 0.0, whole;
  for (int i = p0; i < p1; ++i) sum += part[i];
  if (tid == 0) S.first = INT_MAX;
  if (tid == 0) S.count = 0;
  double before = block_before<double>(sum, S.wave, &whole);
  const double target = u > 0.0 ? u * whole : 0.0;
  int mine = INT_MAX, some = -1;
  {
    double acc = before;
    for (int i = p0; i < p1; ++i) {
      const double v = part[i];
      if (v > 0.0) {
        some = i;
        if (mine == INT_MAX && acc + v > target) mine = i;
      }
      acc += v;
    }
  }
  const uint64_t passes = __ballot(mine != INT_MAX);
  if (passes && lane == __builtin_ctzll(passes)) atomicMin(&S.first, mine);
  last_of((int*)&S.count, some);
  __syncthreads();
  // by rounding alone no part may pass: then the last one that weighs
  const int at = S.first != INT_MAX ? S.first : (int)S.count;
  if (at >= p0 && at < p1) {
    for (int i = p0; i < at; ++i) before += part[i];
    S.wave[0] = before;
  }
  __syncthreads();
  if (tid >= 64) return;
  before = S.wave[0];
  const int i0 = (at * 64 + lane) * kVec<T>;
  Piece<T> piece;
  piece.load(x, i0, A.vocab);
  double w[kVec<T>], own = 0.0;
#pragma unroll
  for (int e = 0; e < kVec<T>; ++e) {
    w[e] = kept_weight(b, last, floor_w, piece.take(), i0 + e);
    own += w[e];
  }
  double acc = before + (wave_inclusive<double>(own) - own);
  int over = -1, final_one = -1;
  double over_w = 0.0, final_w = 0.0;
#pragma unroll
  for (int e = 0; e < kVec<T>; ++e) {
    acc += w[e];
    if (w[e] > 0.0) {
      if (over < 0 && acc > target) { over = i0 + e; over_w = w[e]; }
      final_one = i0 + e;
      final_w = w[e];
    }
  }
  const uint64_t has = __ballot(over >= 0), any = __ballot(final_one >= 0);
  const int winner = has ? __builtin_ctzll(has) : any ? 63 - __builtin_clzll(any) : 0;
  if (lane == winner) {
    A.token[row] = has ? over : final_one;
    if (A.prob) A.prob[row] = (float)((has ? over_w : final_w) / whole);
  }
}

__device__ __forceinline__ void no_token(const SampleArgs& A, int row) {
  if (threadIdx.x == 0) {
    A.token[row] = -1;
    if (A.prob) A.prob[row] = 0.0f;
  }
}

// A row in one block.
template <typename T>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs A) {
  __shared__ AnyShared M;
  Fast& S = M.fast;
  const int row = blockIdx.x;
  const T* x = (const T*)A.logits + (int64_t)row * A.row_stride;
  const Settings set = settings(A, row);
  float top, least;
  tile_range<T>(x, 0, A.vocab, set.rate, S, &top, &least);
  if (top == -__builtin_inff()) return no_token(A, row);
  const Bins b = bins_of(top, least, set.rate);
  unsigned long long last = 0;
  bool digits = b.digits;
  if (!digits && set.ordered) {
    tile_histogram<T>(x, 0, A.vocab, b, S);
    const unsigned long long h0 = S.hist[2 * threadIdx.x], h1 = S.hist[2 * threadIdx.x + 1];
    const unsigned long long mask = (1ull << kCountBit) - 1;
    const uint32_t n[2] = {(uint32_t)(h0 >> kCountBit), (uint32_t)(h1 >> kCountBit)};
    const unsigned long long deficit[2] = {h0 & mask, h1 & mask};
    find_borders(set, b, n, deficit, S);
    const uint32_t cands = S.b.cands;
    digits = cands > (uint32_t)kCands;
    if (!digits && cands > 0) {
      tile_gather<T>(x, 0, A.vocab, b, S);
      last = last_kept(set, b, S, cands);
    }
  }
  __syncthreads();
  if (digits) {
    row_by_digits<T>(A, M.digits, row);
    return;
  }
  tile_sums<T>(x, 0, A.vocab, b, last, set.floor_w, S.part);
  __syncthreads();
  const int rounds = (A.vocab + kStripe<T> - 1) / kStripe<T>;
  pick<T>(A, x, b, last, set.floor_w, (double)A.u[row], S.part, rounds * kWaves, S, row);
}

// A row in several blocks: what the launches hand on.
struct RowWork {
  float* range;               // [tiles][2]
  unsigned long long* hist;   // [tiles][kNB]
  unsigned long long* cand;   // [kCands]
  double* part;               // [tiles * stripes * kWaves]
  unsigned long long* last;
  uint32_t* count;
  Borders* borders;
};

struct SplitArgs {
  uint8_t* ws;
  int64_t row_bytes;
  int32_t tiles, stripes;
  bool ordered;   // there is top-k or top-p
};

__host__ __device__ inline int64_t row_work_bytes(int64_t tiles, int64_t stripes) {
  return (tiles * 8 + 15) / 16 * 16 + tiles * kNB * 8 + kCands * 8 + tiles * stripes * kWaves * 8 + 16 + (sizeof(Borders) + 15) / 16 * 16;
}

__device__ __forceinline__ RowWork row_work(const SplitArgs& P, int row) {
  RowWork w;
  uint8_t* p = P.ws + (int64_t)row * P.row_bytes;
  w.range = (float*)p;
  p += (P.tiles * 8 + 15) / 16 * 16;
  w.hist = (unsigned long long*)p;
  p += (int64_t)P.tiles * kNB * 8;
  w.cand = (unsigned long long*)p;
  p += kCands * 8;
  w.part = (double*)p;
  p += (int64_t)P.tiles * P.stripes * kWaves * 8;
  w.last = (unsigned long long*)p;
  w.count = (uint32_t*)(p + 8);
  w.borders = (Borders*)(p + 16);
  return w;
}

__device__ __forceinline__ Bins split_bins(const SplitArgs& P, const RowWork& w, double rate) {
  static_assert(kMaxTiles <= 64, "a lane per tile");
  const int lane = threadIdx.x & 63;
  float top = -__builtin_inff(), least = __builtin_inff();
  if (lane < P.tiles) {
    const float2 r = *(const float2*)(w.range + 2 * lane);
    top = r.x;
    least = top > -__builtin_inff() ? r.y : least;   // a tile without a token has no least one
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    top = fmaxf(top, __shfl_xor(top, off, 64));
    least = fminf(least, __shfl_xor(least, off, 64));
  }
  return bins_of(top, least, rate);
}

// The borders from all tiles' histograms; every gathering block finds them.
__device__ __forceinline__ void split_borders(const SplitArgs& P, const RowWork& w, const Settings& set, const Bins& b, Fast& S) {
  uint32_t n[2] = {0, 0};
  unsigned long long deficit[2] = {0, 0};
  const unsigned long long mask = (1ull << kCountBit) - 1;
#pragma unroll 4
  for (int i = 0; i < P.tiles; ++i) {
    const ulonglong2 h = *(const ulonglong2*)(w.hist + (int64_t)i * kNB + 2 * threadIdx.x);
    n[0] += (uint32_t)(h.x >> kCountBit);
    n[1] += (uint32_t)(h.y >> kCountBit);
    deficit[0] += h.x & mask;
    deficit[1] += h.y & mask;
  }
  find_borders(set, b, n, deficit, S);
}

enum Phase { kRange, kHistogram, kGather, kSums, kPick };

template <typename T, int PHASE>
__global__ __launch_bounds__(kThreads) void sample_phase_kernel(SampleArgs A, SplitArgs P) {
  __shared__ AnyShared M;
  Fast& S = M.fast;
  const int row = blockIdx.y, tile = blockIdx.x;
  const T* x = (const T*)A.logits + (int64_t)row * A.row_stride;
  const RowWork w = row_work(P, row);
  const Settings set = settings(A, row);
  const int64_t from64 = (int64_t)tile * P.stripes * kStripe<T>;
  const int from = (int)from64, to = from64 + (int64_t)P.stripes * kStripe<T> < A.vocab ? (int)(from64 + (int64_t)P.stripes * kStripe<T>) : A.vocab;
  if constexpr (PHASE == kRange) {
    float top, least;
    tile_range<T>(x, from, to, set.rate, S, &top, &least);
    if (threadIdx.x == 0) {
      w.range[2 * tile] = top;
      w.range[2 * tile + 1] = least;
      if (tile == 0) *w.count = 0;
    }
    return;
  }
  const Bins b = split_bins(P, w, set.rate);
  const bool none = b.top == -__builtin_inff();
  if constexpr (PHASE == kHistogram) {
    if (none || b.digits || !set.ordered) return;
    tile_histogram<T>(x, from, to, b, S);
    for (int i = threadIdx.x; i < kNB; i += kThreads) w.hist[(int64_t)tile * kNB + i] = S.hist[i];
  } else if constexpr (PHASE == kGather) {
    if (none || b.digits || !set.ordered) return;
    split_borders(P, w, set, b, S);
    if (tile == 0 && threadIdx.x == 0) *w.borders = S.b;
    if (S.b.cands <= (uint32_t)kCands && S.b.cands > 0) {
      tile_gather<T>(x, from, to, b, S);
      const uint32_t mine = S.count;
      if (threadIdx.x == 0) S.wave_n[0] = mine ? atomicAdd(w.count, mine) : 0;
      __syncthreads();
      const uint32_t at = S.wave_n[0];
      for (uint32_t i = threadIdx.x; i < mine; i += kThreads)
        if (at + i < (uint32_t)kCands) w.cand[at + i] = S.cand[i];
    }
  } else if constexpr (PHASE == kSums) {
    if (none || b.digits) return;
    unsigned long long last = 0;
    if (set.ordered) {
      if (P.ordered) {
        if (threadIdx.x == 0) S.b = *w.borders;
        __syncthreads();
      }
      // without top-k and top-p a row is ordered only by a min_p above 1
      const uint32_t cands = P.ordered ? S.b.cands : kCands + 1u;
      if (cands > (uint32_t)kCands) {
        if (tile == 0 && threadIdx.x == 0) *w.last = ~0ull;   // for the last launch: by digits
        return;
      }
      if (cands > 0) {
        for (uint32_t i = threadIdx.x; i < cands; i += kThreads) S.cand[i] = w.cand[i];
        last = last_kept(set, b, S, cands);
      }
    }
    if (tile == 0 && threadIdx.x == 0) *w.last = last;
    tile_sums<T>(x, from, to, b, last, set.floor_w, w.part + (int64_t)tile * P.stripes * kWaves);
  } else {
    if (none) return no_token(A, row);
    if (b.digits || *w.last == ~0ull) {
      row_by_digits<T>(A, M.digits, row);
      return;
    }
    const int rounds = (A.vocab + kStripe<T> - 1) / kStripe<T>;
    pick<T>(A, x, b, *w.last, set.floor_w, (double)A.u[row], w.part, rounds * kWaves, S, row);
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_digits_kernel(SampleArgs A) {
  __shared__ Shared S;
  row_by_digits<T>(A, S, blockIdx.x);
}

// Rounds of a tile: all eight once two blocks a unit have work, fewer before
// that, but no more than 16 tiles a row for it (every block reads all tiles'
// histograms).
void tiling(int64_t batch, int64_t vocab, int64_t stripe, int64_t* tiles, int64_t* stripes) {
  const int64_t rounds = (vocab + stripe - 1) / stripe;
  int64_t want = batch < 512 ? 512 / batch : 1;
  want = want > 16 ? 16 : want;
  int64_t s = (rounds + want - 1) / want;
  s = s < kStripes ? s : kStripes;
  *stripes = s;
  *tiles = (rounds + s - 1) / s;
}

// Whether each row runs in one block.  With top-k or top-p five launches are
// not faster before a block's eight rounds are over (32000 float32 logits: 39
// us both ways; 64 such rows 43 us in one block each, 61 us in tiles); without,
// three launches are, from the third round on (16 rows of 50001 f16 logits 19
// us, 35 us in one block each), until the rows alone fill half of the chip.
bool by_rows(int64_t batch, int64_t vocab, int64_t stripe, bool ordered) {
  const int64_t rounds = (vocab + stripe - 1) / stripe;
  return rounds <= (ordered || batch >= 128 ? kStripes : 2);
}

template <typename T>
void launch(const SampleArgs& A, int64_t batch, uint8_t* ws, int64_t ws_bytes, hipStream_t s) {
  const bool ordered = A.top_k || A.top_p;
  int64_t tiles, stripes;
  tiling(batch, A.vocab, kStripe<T>, &tiles, &stripes);
  SplitArgs P{ws, row_work_bytes(tiles, stripes), (int32_t)tiles, (int32_t)stripes, ordered};
  const bool room = tiles <= kMaxTiles && ws_bytes >= batch * P.row_bytes;
  if (by_rows(batch, A.vocab, kStripe<T>, ordered) || (!room && A.vocab <= kStripes * kStripe<T>)) {
    sample_row_kernel<T><<<dim3((uint32_t)batch), dim3(kThreads), 0, s>>>(A);
    return;
  }
  if (!room) {
    sample_digits_kernel<T><<<dim3((uint32_t)batch), dim3(kThreads), 0, s>>>(A);
    return;
  }
  const dim3 grid((uint32_t)tiles, (uint32_t)batch), one(1, (uint32_t)batch);
  sample_phase_kernel<T, kRange><<<grid, dim3(kThreads), 0, s>>>(A, P);
  if (ordered) {
    sample_phase_kernel<T, kHistogram><<<grid, dim3(kThreads), 0, s>>>(A, P);
    sample_phase_kernel<T, kGather><<<grid, dim3(kThreads), 0, s>>>(A, P);
  }
  sample_phase_kernel<T, kSums><<<grid, dim3(kThreads), 0, s>>>(A, P);
  sample_phase_kernel<T, kPick><<<one, dim3(kThreads), 0, s>>>(A, P);
}

template <typename T>
int64_t bytes_of(int64_t batch, int64_t vocab) {
  if (by_rows(batch, vocab, kStripe<T>, false)) return 0;
  int64_t tiles, stripes;
  tiling(batch, vocab, kStripe<T>, &tiles, &stripes);
  return tiles > kMaxTiles ? 0 : batch * row_work_bytes(tiles, stripes);
}

}  // namespace

namespace nvfp4host {

int64_t sample_bytes(int64_t batch, int64_t vocab, nvfp4_dtype_t dt) {
  return dt == NVFP4_F32 ? bytes_of<float>(batch, vocab) : bytes_of<__bf16>(batch, vocab);
}

void launch_sample(const void* logits, nvfp4_dtype_t dt, int64_t batch, int64_t vocab, int64_t row_stride, const float* u,
                   const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p, void* ws,
                   int64_t ws_bytes, int32_t* token, float* prob, hipStream_t s) {
  SampleArgs A{logits, u, temperature, top_p, min_p, top_k, token, prob, row_stride, (int32_t)vocab, 0};
  // a row's weights add up to at most vocab: its integer sum stays below 2^62
  A.fix = 62 - (64 - __builtin_clzll((unsigned long long)vocab));
  switch (dt) {
    case NVFP4_F32: launch<float>(A, batch, (uint8_t*)ws, ws_bytes, s); break;
    case NVFP4_BF16: launch<__bf16>(A, batch, (uint8_t*)ws, ws_bytes, s); break;
    case NVFP4_F16: launch<_Float16>(A, batch, (uint8_t*)ws, ws_bytes, s); break;
  }
}

}  // namespace nvfp4host
