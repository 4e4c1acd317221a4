// Bookkeeping of the cache's pages on the device: freeing, reserving, sharing
// and compacting them.
//
// A page is free where refs, the number of table entries that name it, is not
// above 0.  That number is the only state, so a result never depends on an
// order: counts change by integer atomics, and pages are handed out by rank,
// the lowest free one first, to entries in the order of (sequence, entry).
//
// Contents move as whole pages, copied for all layers' caches by one launch
// whose pairs (from, to) the launch before it has left in the workspace.
//
// Small calls are the host's (5 us a call with one launch, 12 with two) and a
// chain of a few dependent loads: freeing 2.7 us (16 sequences of 469 entries),
// 6.0 where 64 of 256 sequences of up to 2048 entries end; forking 4.0 and 7.7
// (128 beams of 2048 entries); reserving for 64 sequences 5.2 and the copying
// launch that finds nothing to copy 1.9.
#include <algorithm>
#include <climits>

#include "kv_cache.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

constexpr int kThreads = 256;
// Cells of the table that a block takes.
constexpr int kCells = 4 * kThreads;
// Threads of a block that plans, pages that a thread looks at in a round, and
// those of a round of all of them.
constexpr int kPlan = 1024, kScan = 16, kRound = kPlan * kScan;
// Pools of more pages than these are counted by a launch of many blocks before
// they are planned: one block takes 1.5 us a round of a reserve, and 15 of a
// compaction.  (Calls: a reserve from the end of 65536 pages 21 us either way, of
// 1048576 23 us, 136 by one block; half of 65536 pages of 2 KB compacted 41 us
// and 100.)
constexpr int64_t kReserveAlone = 4 * kRound, kCompactAlone = kRound;
// Bytes of a page's side that a block copies at a time, in 16-byte accesses.
constexpr int kVecs = 4, kPiece = kVecs * kThreads * 16;
// Caches of a copying launch: their addresses are its arguments.
constexpr int kLayers = 32;
// Copying blocks, eight a unit; more copies than that go round.
constexpr int64_t kCopyBlocks = 2048;

__device__ __forceinline__ bool is_page(int32_t id, int32_t pages) { return id >= 0 && id < pages; }

// The sum of the threads' values before this one; *all gets the whole sum.
__device__ __forceinline__ int block_scan(int v, int* shared, int* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off, 64);
    x += lane >= off ? y : 0;
  }
  if (lane == 63) shared[wave] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlan / 64; ++w) {
    before += w < wave ? shared[w] : 0;
    sum += shared[w];
  }
  __syncthreads();   // the next scan writes `shared` again
  *all = sum;
  return before + x - v;
}

// A bit for each of the pages p .. p + kScan - 1 that is free.
__device__ __forceinline__ uint32_t free_pages(const int32_t* refs, int64_t p, int32_t pages, bool vec) {
  int32_t r[kScan];
  if (vec && p + kScan <= pages) {
#pragma unroll
    for (int i = 0; i < kScan / 4; ++i) {
      const int4 x = *((const int4*)(refs + p) + i);
      r[4 * i] = x.x; r[4 * i + 1] = x.y; r[4 * i + 2] = x.z; r[4 * i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kScan; ++i) r[i] = p + i < pages ? refs[p + i] : 1;
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kScan; ++i) m |= r[i] <= 0 ? 1u << i : 0u;
  return m;
}

// The pages of a thread's kScan from p on that are there, and those below `end`.
__device__ __forceinline__ uint32_t pages_below(int64_t p, int64_t end) {
  return p >= end ? 0 : end - p < kScan ? (1u << (end - p)) - 1 : (1u << kScan) - 1;
}

// The free pages of each round.
__global__ __launch_bounds__(kPlan) void count_kernel(const int32_t* refs, int32_t* counts, int32_t pages, bool vec) {
  __shared__ int shared[kPlan / 64];
  const int64_t p = (int64_t)blockIdx.x * kRound + threadIdx.x * kScan;
  int all;
  block_scan(__popc(free_pages(refs, p, pages, vec)), shared, &all);
  if (threadIdx.x == 0) counts[blockIdx.x] = all;
}

// ---------------------------------------------------------------------------
// freeing and sharing: every cell of the table by itself
// ---------------------------------------------------------------------------

struct FreeArgs {
  int32_t* table;
  const int32_t* lens;
  int32_t* refs;
  int64_t keep, sinks;
  int32_t cells, width, pages, page_shift;
};

__global__ __launch_bounds__(kThreads) void free_kernel(FreeArgs A) {
  // a thread's cells at once: their loads wait together
  constexpr int N = kCells / kThreads;
  uint32_t c[N];
  int32_t id[N], len[N], i[N];
#pragma unroll
  for (int r = 0; r < N; ++r) {
    c[r] = blockIdx.x * (uint32_t)kCells + r * kThreads + threadIdx.x;
    const uint32_t at = c[r] < (uint32_t)A.cells ? c[r] : 0, b = at / (uint32_t)A.width;
    i[r] = (int32_t)(at - b * (uint32_t)A.width);
    len[r] = A.lens[b];
    id[r] = A.table[at];
  }
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const int64_t begin = (int64_t)i[r] << A.page_shift, end = begin + (1 << A.page_shift);
    const bool needed = begin < len[r] && (A.keep <= 0 || end > len[r] - A.keep || begin < A.sinks);
    if (c[r] < (uint32_t)A.cells && !needed && is_page(id[r], A.pages)) {
      A.table[c[r]] = -1;
      atomicSub(&A.refs[id[r]], 1);
    }
  }
}

struct ForkArgs {
  const int32_t *table, *lens, *parent;
  int32_t *refs, *table_out, *lens_out;
  int32_t batch, rows, width, pages;
  uint32_t cells;   // of the larger table, and at least its rows
};

__global__ __launch_bounds__(kThreads) void fork_kernel(ForkArgs A) {
  constexpr int N = kCells / kThreads;
  const uint32_t c0 = blockIdx.x * (uint32_t)kCells + threadIdx.x, width = A.width > 0 ? A.width : 1;
  uint32_t b[N], i[N];
  int32_t from[N], to[N], parent[N];
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const uint32_t c = c0 + r * kThreads;
    b[r] = c / width;
    i[r] = c - b[r] * width;
    parent[r] = b[r] < (uint32_t)A.rows && c < A.cells ? A.parent[b[r]] : -1;
    from[r] = A.width > 0 && b[r] < (uint32_t)A.batch ? A.table[c] : -1;
  }
#pragma unroll
  for (int r = 0; r < N; ++r) to[r] = A.width > 0 && is_page(parent[r], A.batch) ? A.table[(int64_t)parent[r] * A.width + i[r]] : -1;
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const uint32_t c = c0 + r * kThreads;
    if (b[r] < (uint32_t)A.rows && c < A.cells) {
      if (A.width > 0) A.table_out[c] = to[r];
      if (i[r] == 0) A.lens_out[b[r]] = is_page(parent[r], A.batch) ? A.lens[parent[r]] : 0;
    }
    // what a row keeps counts as before
    if (from[r] != to[r]) {
      if (is_page(to[r], A.pages)) atomicAdd(&A.refs[to[r]], 1);
      if (is_page(from[r], A.pages)) atomicSub(&A.refs[from[r]], 1);
    }
  }
}

// ---------------------------------------------------------------------------
// reserving: one block
// ---------------------------------------------------------------------------
//
// An item is a page slot of a sequence's new tokens: sequence b has those from
// (first row / page) + 2 b on (one each without offsets).  First every item's
// need, and its rank among them; then as many free pages as are needed, by
// rank; then the entries.  A sequence's items are served together or not at all.

struct ReserveArgs {
  SequenceView s;
  int32_t *table, *refs, *missing;
  int32_t* copies;    // their number, and from [4] on the pairs (from, to)
  int32_t* ranks;     // [items + 1]: needs before an item
  int32_t* fresh;     // [items]: the pages taken, from rank kPlan on
  const int32_t* counts;   // free pages of each round, or null: not counted
  int32_t items, pages, page_shift;
  bool vec;           // 16-byte loads of refs
};

__device__ __forceinline__ int first_item(const ReserveArgs& A, int b) {
  return A.s.cu ? (sequence_row(A.s, b) >> A.page_shift) + 2 * b : b;
}

struct Item {
  int32_t b;
  int32_t old;        // what the entry holds
  int64_t cell;       // of the table; -1: no entry of new tokens
  bool partly;        // the page holds earlier tokens too
};

__device__ __forceinline__ Item item_of(const ReserveArgs& A, int e) {
  Item it;
  it.b = e;
  it.cell = -1;
  it.old = -1;
  it.partly = false;
  int slot = 0;
  if (A.s.cu) {
    int lo = 0, hi = A.s.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_item(A, mid) <= e) lo = mid; else hi = mid - 1;
    }
    it.b = lo;
    slot = e - first_item(A, lo);
  }
  const Sequence s = sequence(A.s, it.b);
  const int first = s.first, stop = s.first + s.count, from = first < 0 ? 0 : first;
  const int64_t i = (int64_t)(from >> A.page_shift) + slot;
  if (slot < 0 || s.count <= 0 || i >= A.s.width || (i << A.page_shift) >= stop) return it;
  it.cell = (int64_t)it.b * A.s.width + i;
  it.old = A.table[it.cell];
  it.partly = (i << A.page_shift) < from;
  return it;
}

__global__ __launch_bounds__(kPlan) void reserve_kernel(ReserveArgs A) {
  __shared__ int shared[kPlan / 64];
  __shared__ int32_t fresh[kPlan];
  __shared__ int copies;
  const int tid = threadIdx.x;
  if (tid == 0) copies = 0;

  // needs, and their ranks; the first round's stay in registers
  Item mine;
  int my_rank = 0, want = 0;
  bool my_need = false;
  for (int base = 0; base < A.items; base += kPlan) {
    const int e = base + tid;
    Item it;
    bool need = false;
    if (e < A.items) {
      it = item_of(A, e);
      need = it.cell >= 0 && (!is_page(it.old, A.pages) || A.refs[it.old] > 1);
    }
    int all;
    const int rank = want + block_scan(need, shared, &all);
    if (e < A.items) A.ranks[e] = rank;
    if (base == 0) {
      mine = it;
      my_rank = rank;
      my_need = need;
    }
    want += all;
  }
  if (tid == 0) A.ranks[A.items] = want;

  // the first `want` free pages
  int have = 0;
  const auto take = [&](int64_t round) {
    const int64_t p = round * kRound + tid * kScan;
    uint32_t m = free_pages(A.refs, p, A.pages, A.vec);
    int all, rank = have + block_scan(__popc(m), shared, &all);
    for (; m && rank < want; m &= m - 1, ++rank) {
      const int32_t id = (int32_t)(p + __builtin_ctz(m));
      if (rank < kPlan) fresh[rank] = id; else A.fresh[rank] = id;
    }
    have += all;
  };
  const int64_t rounds = ((int64_t)A.pages + kRound - 1) / kRound;
  if (!A.counts) {
    for (int64_t r = 0; r < rounds && have < want; ++r) take(r);
  } else {
    // only rounds with free pages, 64 of them looked up at a time
    for (int64_t r0 = 0; r0 < rounds && have < want; r0 += 64) {
      const int64_t r = r0 + (tid & 63);
      uint64_t some = __ballot(r < rounds && A.counts[r] > 0);
      for (; some && have < want; some &= some - 1) take(r0 + __builtin_ctzll(some));
    }
  }
  __syncthreads();

  const bool enough = have >= want;
  const auto needs_until = [&](int b) { return A.ranks[b < A.s.batch ? min(first_item(A, b), A.items) : A.items]; };
  for (int base = 0; base < A.items; base += kPlan) {
    const int e = base + tid;
    if (e >= A.items) continue;
    if (base > 0) {
      my_rank = A.ranks[e];
      my_need = A.ranks[e + 1] != my_rank;
      if (my_need) mine = item_of(A, e);
    }
    if (!my_need || !(enough || needs_until(mine.b + 1) <= have)) continue;
    const int32_t id = my_rank < kPlan ? fresh[my_rank] : A.fresh[my_rank];
    A.table[mine.cell] = id;
    A.refs[id] = 1;
    if (is_page(mine.old, A.pages)) {   // needed though it is there: it is shared
      atomicSub(&A.refs[mine.old], 1);
      if (mine.partly) {
        const int at = atomicAdd(&copies, 1);
        A.copies[4 + 2 * at] = mine.old;
        A.copies[5 + 2 * at] = id;
      }
    }
  }
  for (int b = tid; b < A.s.batch; b += kPlan) {
    int lack = 0;
    if (!enough) {
      const int until = needs_until(b + 1);
      lack = until <= have ? 0 : until - needs_until(b);
    }
    A.missing[b] = lack;
  }
  __syncthreads();
  if (tid == 0) A.copies[0] = copies;
}

// ---------------------------------------------------------------------------
// compacting: a block plans each round, alone for a pool of one
// ---------------------------------------------------------------------------

struct CompactArgs {
  int32_t *refs, *used, *where;
  int32_t* copies;    // their number, and from [4] on the pairs (from, to)
  int32_t pages;
  bool vec;
};

// The round's part of the plan, of the thread's pages from p on, those in
// `empty` free: holes are the free pages below `used`, movers the pages in use
// from there on; `holes` and `movers` are those of earlier rounds.  Gives the
// movers of this round and earlier ones.
__device__ __forceinline__ int plan_round(const CompactArgs& A, int64_t p, uint32_t empty, int used, int holes, int movers, int* shared) {
  const uint32_t inside = pages_below(p, A.pages), low = pages_below(p, used);
  uint32_t hole = empty & low, mover = inside & ~empty & ~low;
#pragma unroll
  for (int i = 0; i < kScan; ++i)
    if ((inside >> i) & 1) A.where[p + i] = (empty >> i) & 1 ? -1 : (int32_t)(p + i);
  int sum;   // a round has at most 2^14 of each
  const int before = block_scan(__popc(hole) | (__popc(mover) << 16), shared, &sum);
  // (k stays in the list also if another stream changes the counts meanwhile)
  const int room = A.pages / 2;
  for (int k = holes + (before & 0xffff); hole && k < room; hole &= hole - 1, ++k) A.copies[5 + 2 * (int64_t)k] = (int32_t)(p + __builtin_ctz(hole));
  for (int k = movers + (before >> 16); mover && k < room; mover &= mover - 1, ++k) A.copies[4 + 2 * (int64_t)k] = (int32_t)(p + __builtin_ctz(mover));
  return movers + (sum >> 16);
}

__device__ __forceinline__ void move_count(const CompactArgs& A, int64_t k) {
  const int32_t from = A.copies[4 + 2 * k], to = A.copies[5 + 2 * k];
  if (!is_page(from, A.pages) || !is_page(to, A.pages)) return;
  A.where[from] = to;
  A.refs[to] = A.refs[from];
  A.refs[from] = 0;
}

// Pools of one round at most.
__global__ __launch_bounds__(kPlan) void compact_kernel(CompactArgs A) {
  __shared__ int shared[kPlan / 64];
  const int tid = threadIdx.x;
  const int64_t p = tid * kScan;
  const uint32_t empty = free_pages(A.refs, p, A.pages, A.vec);
  int used;
  block_scan(__popc(pages_below(p, A.pages)) - __popc(empty), shared, &used);
  int movers = plan_round(A, p, empty, used, 0, 0, shared);
  __syncthreads();
  movers = movers < A.pages / 2 ? movers : A.pages / 2;
  for (int k = tid; k < movers; k += kPlan) move_count(A, k);
  if (tid == 0) {
    A.copies[0] = movers;
    *A.used = used;
  }
}

// The same by a block each round, with the rounds' free pages counted.
__global__ __launch_bounds__(kPlan) void compact_round_kernel(CompactArgs A, const int32_t* counts) {
  __shared__ int shared[kPlan / 64];
  const int rounds = (int)(((int64_t)A.pages + kRound - 1) / kRound);
  const auto sum_to = [&](int end) {
    int v = 0, all;
    for (int r = threadIdx.x; r < end; r += kPlan) v += counts[r];
    block_scan(v, shared, &all);
    return all;
  };
  const int used = A.pages - sum_to(rounds), mine = (int)blockIdx.x, border = used / kRound;
  // the holes before this round and all of them: the free pages below `used`
  const int64_t p = (int64_t)border * kRound + threadIdx.x * kScan;
  int in_border;
  block_scan(__popc(free_pages(A.refs, p, A.pages, A.vec) & pages_below(p, used)), shared, &in_border);
  const int all = sum_to(border < rounds ? border : rounds) + in_border, free_before = sum_to(mine);
  // the movers before this round: pages in use before it but for those below `used`
  const int holes = mine <= border ? free_before : all;
  const int movers = mine <= border ? 0 : mine * kRound - free_before - (used - all);
  if (mine == 0 && threadIdx.x == 0) {
    A.copies[0] = all < A.pages / 2 ? all : A.pages / 2;
    *A.used = used;
  }
  const int64_t at = (int64_t)mine * kRound + threadIdx.x * kScan;
  plan_round(A, at, free_pages(A.refs, at, A.pages, A.vec), used, holes, movers, shared);
}

__global__ __launch_bounds__(kThreads) void move_counts_kernel(CompactArgs A) {
  const int64_t k = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (k < A.copies[0]) move_count(A, k);
}

// ---------------------------------------------------------------------------
// copying
// ---------------------------------------------------------------------------

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct CopyArgs {
  const int32_t* copies;
  int64_t page_bytes;       // of a side
  int32_t heads, layers;
  int32_t pieces, group;    // pieces of a page, or the pages that fit one
  int32_t* table;           // to be rewritten by `where`, by the last row of blocks
  const int32_t* where;
  int32_t cells, pages;
  uint8_t *k[kLayers], *v[kLayers], *ks[kLayers], *vs[kLayers];
};

// A row of blocks for each cache and side, and one for the table.
//
// Bound by memory.  Copies are not read again soon, so they are stored past the
// caches, and with ONCE, where each page is copied to one other alone, loaded
// past them too: half of a pool of 2048 pages compacted in 4 layers (537 MB,
// read and written) 109 us with the plan, 4.9 TB/s, 124 through the caches; 64
// copies of 8 pages in 16 layers (268 MB) 41 us with stores alone past them, 63
// through, 58 with loads past them as well.  GROUPED: a block copies several
// small pages at a time.
template <bool ONCE, bool GROUPED>
__global__ __launch_bounds__(kThreads) void copy_kernel(CopyArgs A) {
  const int layer = blockIdx.y >> 1, side = blockIdx.y & 1;
  if (layer == A.layers) {
    for (uint32_t c = blockIdx.x * kThreads + threadIdx.x; c < (uint32_t)A.cells; c += gridDim.x * kThreads) {
      const int32_t id = A.table[c];
      if (is_page(id, A.pages)) A.table[c] = A.where[id];
    }
    return;
  }
  // pieces of all pages of a pool of 2^31 pages would pass 32 bits, those of one in memory do not
  const uint32_t count = (uint32_t)A.copies[0], vecs = (uint32_t)(A.page_bytes / 16), heads = (uint32_t)A.heads;
  const uint32_t group = GROUPED ? (uint32_t)A.group : 1, all = (count + group - 1) / group * (uint32_t)A.pieces;
  uint8_t* const base = side ? A.v[layer] : A.k[layer];
  uint8_t* const scales = side ? A.vs[layer] : A.ks[layer];
  for (uint32_t at = blockIdx.x; at < all; at += gridDim.x) {
    const uint32_t first = GROUPED ? at : at / (uint32_t)A.pieces, piece = at - first * (uint32_t)A.pieces, pair0 = first * group;
    const int64_t from0 = A.copies[4 + 2 * (int64_t)pair0], to0 = A.copies[5 + 2 * (int64_t)pair0];
    u32x4_t x[kVecs];
    if constexpr (!GROUPED) {
      if (!is_page((int32_t)from0, A.pages) || !is_page((int32_t)to0, A.pages)) continue;
      const u32x4_t* src = (const u32x4_t*)(base + from0 * A.page_bytes);
      u32x4_t* dst = (u32x4_t*)(base + to0 * A.page_bytes);
      const uint32_t v = piece * (kPiece / 16) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (v + i * kThreads < vecs) x[i] = ONCE ? __builtin_nontemporal_load(src + v + i * kThreads) : src[v + i * kThreads];
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (v + i * kThreads < vecs) __builtin_nontemporal_store(x[i], dst + v + i * kThreads);
    } else {
      u32x4_t* dst[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const uint32_t v = i * kThreads + threadIdx.x, local = v / vecs, off = v - local * vecs, pair = pair0 + local;
        dst[i] = nullptr;
        if (local < group && pair < count) {
          const int64_t from = A.copies[4 + 2 * (int64_t)pair], to = A.copies[5 + 2 * (int64_t)pair];
          if (!is_page((int32_t)from, A.pages) || !is_page((int32_t)to, A.pages)) continue;
          const u32x4_t* src = (const u32x4_t*)(base + from * A.page_bytes) + off;
          dst[i] = (u32x4_t*)(base + to * A.page_bytes) + off;
          x[i] = ONCE ? __builtin_nontemporal_load(src) : *src;
        }
      }
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (dst[i]) __builtin_nontemporal_store(x[i], dst[i]);
    }
    if (piece == 0) {
      for (uint32_t h = threadIdx.x; h < heads * group; h += kThreads) {
        const uint32_t local = GROUPED ? h / heads : 0, pair = pair0 + local, head = h - local * heads;
        if (pair < count) {
          const int64_t from = A.copies[4 + 2 * (int64_t)pair], to = A.copies[5 + 2 * (int64_t)pair];
          if (is_page((int32_t)from, A.pages) && is_page((int32_t)to, A.pages)) scales[to * heads + head] = scales[from * heads + head];
        }
      }
    }
  }
}

int64_t blocks_of(int64_t cells) { return (cells + kCells - 1) / kCells; }

template <bool ONCE>
void launch_copies(const nvfp4_kv_cache_t* caches, int64_t count, const int32_t* copies, int64_t most, int32_t* table,
                   const int32_t* where, int64_t cells, hipStream_t s) {
  CopyArgs A;
  A.copies = copies;
  A.page_bytes = caches->heads * caches->page * caches->dim;
  A.heads = (int32_t)caches->heads;
  A.pages = (int32_t)caches->pages;
  A.pieces = (int32_t)((A.page_bytes + kPiece - 1) / kPiece);
  A.group = (int32_t)std::max<int64_t>(kPiece / A.page_bytes, 1);
  A.table = table;
  A.where = where;
  A.cells = (int32_t)cells;
  for (int64_t at = 0; at < count; at += kLayers) {
    A.layers = (int32_t)std::min<int64_t>(kLayers, count - at);
    const bool rewrite = at == 0 && cells > 0;
    for (int i = 0; i < kLayers; ++i) {
      const nvfp4_kv_cache_t& c = caches[at + (i < A.layers ? i : 0)];
      A.k[i] = c.k; A.v[i] = c.v; A.ks[i] = c.k_scales; A.vs[i] = c.v_scales;
    }
    const int64_t row = std::max<int64_t>(kCopyBlocks / (2 * A.layers), 1);
    const int64_t groups = (most + A.group - 1) / A.group;
    int64_t x = groups < row ? std::min(row, groups * std::min<int64_t>(A.pieces, row)) : row;
    if (rewrite) x = std::max(x, std::min(blocks_of(cells), row));
    const dim3 grid((uint32_t)x, (uint32_t)(2 * A.layers + (rewrite ? 1 : 0)));
    if (x > 0 && A.group > 1) copy_kernel<ONCE, true><<<grid, dim3(kThreads), 0, s>>>(A);
    else if (x > 0) copy_kernel<ONCE, false><<<grid, dim3(kThreads), 0, s>>>(A);
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

int64_t rounds_of(int64_t pages) { return (pages + kRound - 1) / kRound; }

}  // namespace

namespace nvfp4host {

int64_t kv_reserve_items(int64_t tokens, int64_t batch, int64_t page, bool offsets) {
  return offsets ? tokens / page + 2 * batch : batch;
}

// The copies and their number, ranks, pages taken, the rounds' free pages.
int64_t kv_reserve_bytes(int64_t items, int64_t batch, int64_t pages) {
  return ((4 + 2 * batch + 2 * items + 1 + (pages > kReserveAlone ? rounds_of(pages) : 0)) * 4 + 255) / 256 * 256;
}

// The copies and their number, the rounds' free pages.
int64_t kv_compact_bytes(int64_t pages) { return ((4 + pages + 1 + rounds_of(pages)) * 4 + 255) / 256 * 256; }

void launch_kv_free(int32_t* table, int64_t batch, int64_t width, const int32_t* lens, int64_t page, int64_t keep,
                    int64_t sinks, int32_t* refs, int64_t pages, hipStream_t s) {
  const FreeArgs A = {table, lens, refs, keep, sinks, (int32_t)(batch * width), (int32_t)width, (int32_t)pages,
                      __builtin_ctz((unsigned)page)};
  free_kernel<<<dim3((uint32_t)blocks_of(A.cells)), dim3(kThreads), 0, s>>>(A);
}

void launch_kv_fork(const int32_t* table, int64_t batch, int64_t width, const int32_t* lens, const int32_t* parent,
                    int64_t rows, int32_t* refs, int64_t pages, int32_t* table_out, int32_t* lens_out, hipStream_t s) {
  const int64_t cells = std::max(std::max(batch, rows) * width, rows);
  const ForkArgs A = {table, lens, parent, refs, table_out, lens_out, (int32_t)batch, (int32_t)rows, (int32_t)width,
                      (int32_t)pages, (uint32_t)cells};
  fork_kernel<<<dim3((uint32_t)blocks_of(cells)), dim3(kThreads), 0, s>>>(A);
}

void launch_kv_reserve(const nvfp4_kv_cache_t* caches, int64_t count, int32_t* table, int64_t batch, int64_t width,
                       const int32_t* lens, const int32_t* cu, int64_t tokens, int32_t* refs, void* ws,
                       int32_t* missing, hipStream_t s) {
  ReserveArgs A;
  const int64_t items = kv_reserve_items(tokens, batch, caches->page, cu != nullptr);
  A.s = {table, lens, cu, width, (int32_t)batch, (int32_t)tokens, INT_MAX};
  A.table = table; A.refs = refs; A.missing = missing;
  A.copies = (int32_t*)ws;
  A.ranks = A.copies + 4 + 2 * batch;
  A.fresh = A.ranks + items + 1;
  A.items = (int32_t)items; A.pages = (int32_t)caches->pages;
  A.page_shift = __builtin_ctz((unsigned)caches->page);
  A.vec = aligned16(refs);
  A.counts = nullptr;
  if (caches->pages > kReserveAlone) {
    int32_t* counts = A.fresh + items;
    count_kernel<<<dim3((uint32_t)rounds_of(caches->pages)), dim3(kPlan), 0, s>>>(refs, counts, A.pages, A.vec);
    A.counts = counts;
  }
  reserve_kernel<<<dim3(1), dim3(kPlan), 0, s>>>(A);
  launch_copies<false>(caches, count, A.copies, batch, nullptr, nullptr, 0, s);
}

void launch_kv_compact(const nvfp4_kv_cache_t* caches, int64_t count, int32_t* table, int64_t batch, int64_t width,
                       int32_t* refs, void* ws, int32_t* used, int32_t* where, hipStream_t s) {
  const CompactArgs A = {refs, used, where, (int32_t*)ws, (int32_t)caches->pages, aligned16(refs)};
  if (caches->pages <= kCompactAlone) {
    compact_kernel<<<dim3(1), dim3(kPlan), 0, s>>>(A);
  } else {
    const int64_t rounds = rounds_of(caches->pages);
    int32_t* counts = A.copies + 4 + caches->pages + 1;
    count_kernel<<<dim3((uint32_t)rounds), dim3(kPlan), 0, s>>>(refs, counts, A.pages, A.vec);
    compact_round_kernel<<<dim3((uint32_t)rounds), dim3(kPlan), 0, s>>>(A, counts);
    move_counts_kernel<<<dim3((uint32_t)((caches->pages / 2 + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(A);
  }
  launch_copies<true>(caches, count, A.copies, caches->pages / 2, table, where, batch * width, s);
}

}  // namespace nvfp4host
