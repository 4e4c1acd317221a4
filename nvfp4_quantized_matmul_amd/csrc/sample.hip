// One token per row of logits: temperature, top-k, top-p and min-p, then the
// inverse of the kept weights' running sum at a given random number.
//
// The kept tokens are a prefix of the order (logit falling, index rising), so
// they are told by the last kept logit and, among the tokens that share it, by
// the last kept index.  Nothing is sorted: a logit's bits as an ordered key
// are searched digit by digit, from the top, through a histogram of the tokens
// whose higher digits agree -- of their number for top-k, of their weight for
// top-p.  The token itself is found by narrowing the row to the part in which
// the running sum passes u times the whole, 16 parts at a time.
//
// With a quarter of a million tokens a probability is a millionth and the
// place of u among them is decided in the 7th digit and beyond, so weights and
// running sums are in 64 bits.  The histogram's weights are integers of 62
// bits for a whole row, which add up the same in any order.
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

// exp((x - top) / temperature), with rate = log2(e) / temperature: 2^y as the
// power of two of the nearest integer and the Taylor sum of the rest to its
// 9th power, whose first left-out term is below 8e-12 of the sum.
__device__ __forceinline__ double weight(float x, float top, double rate) {
  if (x == top) return 1.0;
  const double y = ((double)x - (double)top) * rate;
  if (!(y > -1080.0)) return 0.0;
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
// `target` and the sum with it is not (the last non-empty one if rounding
// leaves none): into S.bin, the sum before it into S.before.  `value` gives a
// bin's amount; bins 2 t and 2 t + 1 from the top are thread t's.
template <typename F>
__device__ void find_bin(Shared& S, double target, const F& value, unsigned long long before0) {
  static_assert(kBins == 2 * kThreads, "two bins a thread");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b0 = kBins - 1 - 2 * tid, b1 = b0 - 1;
  const unsigned long long v0 = value(b0), v1 = value(b1);
  const unsigned long long incl = wave_inclusive<unsigned long long>(v0 + v1);
  if (lane == 63) S.wave_mass[wave] = incl;
  if (tid == 0) S.bin = 0xffffffffu;
  __syncthreads();
  unsigned long long before = before0;
  for (int w = 0; w < wave; ++w) before += S.wave_mass[w];
  before += incl - v0 - v1;
  if (v0 && (double)before < target && (double)(before + v0) >= target) { S.bin = b0; S.before = before; }
  const unsigned long long mid = before + v0;
  if (v1 && (double)mid < target && (double)(mid + v1) >= target) { S.bin = b1; S.before = mid; }
  __syncthreads();
  if (S.bin == 0xffffffffu) {
    // only where the target passes the whole by a rounding: the lowest non-empty bin
    if (tid == 0) {
      unsigned long long sum = before0;
      for (int b = kBins - 1; b >= 0; --b) {
        const unsigned long long v = value(b);
        if (v) { S.bin = b; S.before = sum; }
        sum += v;
      }
      if (S.bin == 0xffffffffu) { S.bin = 0; S.before = sum; }
    }
    __syncthreads();
  }
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

template <typename T, bool HELD>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs A) {
  __shared__ Shared S;
  extern __shared__ __align__(16) uint8_t held[];
  const int row = blockIdx.x, tid = threadIdx.x, V = A.vocab;
  const T* x = (const T*)A.logits + (int64_t)row * A.row_stride;
  T* hx = (T*)held;

  uint32_t top_key = 0;
  for (int i = tid; i < V; i += kThreads) {
    const T e = x[i];
    if constexpr (HELD) hx[i] = e;
    const uint32_t k = key_of<T>(clean((float)e));
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
  auto at = [&](int i) -> float { return clean((float)(HELD ? hx[i] : x[i])); };
  const double rate = 1.44269504088896340736 / (A.temperature ? (double)A.temperature[row] : 1.0);
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

template <typename T>
bool launch(const SampleArgs& A, int64_t batch, hipStream_t s) {
  const int64_t bytes = ((int64_t)A.vocab * sizeof(T) + 15) / 16 * 16;
  // a row that fits beside the histogram is read from memory once
  const int64_t room = 160 * 1024 - (int64_t)sizeof(Shared) - 64;
  if (bytes <= room) {
    if (bytes + (int64_t)sizeof(Shared) > 64 * 1024 &&
        hipFuncSetAttribute((const void*)sample_kernel<T, true>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)room) != hipSuccess)
      return false;
    sample_kernel<T, true><<<dim3((uint32_t)batch), dim3(kThreads), (uint32_t)bytes, s>>>(A);
  } else {
    sample_kernel<T, false><<<dim3((uint32_t)batch), dim3(kThreads), 0, s>>>(A);
  }
  return true;
}

}  // namespace

namespace nvfp4host {

int64_t sample_bytes(int64_t, int64_t, nvfp4_dtype_t) { return 0; }

void launch_sample(const void* logits, nvfp4_dtype_t dt, int64_t batch, int64_t vocab, int64_t row_stride, const float* u,
                   const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p, void*, int64_t,
                   int32_t* token, float* prob, hipStream_t s) {
  SampleArgs A{logits, u, temperature, top_p, min_p, top_k, token, prob, row_stride, (int32_t)vocab, 0};
  // a row's weights add up to at most vocab: its integer sum stays below 2^62
  A.fix = 62 - (64 - __builtin_clzll((unsigned long long)vocab));
  switch (dt) {
    case NVFP4_F32: launch<float>(A, batch, s); break;
    case NVFP4_BF16: launch<__bf16>(A, batch, s); break;
    case NVFP4_F16: launch<_Float16>(A, batch, s); break;
  }
}

}  // namespace nvfp4host
