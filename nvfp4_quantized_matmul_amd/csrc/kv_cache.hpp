// Device view of the paged 8-bit key/value cache and of the new tokens'
// rows, shared by the kernels that write it and read it.
#pragma once

#include "nvfp4_device.hpp"

namespace nvfp4dev {

struct CacheView {
  uint8_t* k;         // [pages, heads, page, dim]
  uint8_t* v;         // [pages, heads, dim, page]
  uint8_t* ks;        // [pages, heads]
  uint8_t* vs;
  int32_t pages, heads;
  int32_t page_shift;  // page = 1 << page_shift
};

// Which rows are a sequence's new tokens, and which pages its tokens.
struct SequenceView {
  const int32_t* table;  // [batch, width]
  const int32_t* lens;   // [batch]
  const int32_t* cu;     // [batch + 1] or nullptr: one new token each
  int64_t width;
  int32_t batch, tokens;
  int32_t most;          // new tokens of a sequence that the call takes
};

struct Sequence {
  int32_t row0, count;  // rows [row0, row0 + count) of q, k and v
  int32_t first;        // position of the first of them; lengths may pass the table
};

// The first row of sequence b.
__device__ __forceinline__ int sequence_row(const SequenceView& sv, int b) {
  const int lo = sv.cu ? sv.cu[b] : b;
  return lo < 0 ? 0 : lo > sv.tokens ? sv.tokens : lo;
}

// Sequence b, its rows cut to the rows that exist and to those that the call takes.
__device__ __forceinline__ Sequence sequence(const SequenceView& sv, int b) {
  Sequence s;
  const int lo = sequence_row(sv, b), len = sv.lens[b];
  int hi = sv.cu ? sv.cu[b + 1] : b + 1;
  hi = hi < lo ? lo : hi > sv.tokens ? sv.tokens : hi;
  s.row0 = lo;
  s.first = (len < 0 ? 0 : len) - (hi - lo);
  s.count = hi - lo < sv.most ? hi - lo : sv.most;
  return s;
}

// exponent + 127 of the smallest power of two p with amax <= 448 p, from the
// bits of amax >= 0 (finite): 448 = 1.75 * 2^8, so p = 2^(E - 8) where amax =
// 1.f * 2^E, or twice that when 1.f > 1.75.  Below 2^-119 the byte stays 0.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 0 ? 0 : e;
}

}  // namespace nvfp4dev
