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
#include <algorithm>
#include <climits>

#include "kv_cache.hpp"
#include "nvfp4_internal.hpp"

namespace {

using namespace nvfp4dev;

constexpr int kThreads = 256;
// Cells of the table that a block takes.
constexpr int kCells = 4 * kThreads;
// Threads of the block that plans, and pages that a thread looks at in a round.
constexpr int kPlan = 1024, kScan = 16;
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
  for (int64_t p0 = 0; p0 < A.pages && have < want; p0 += kPlan * kScan) {
    const int64_t p = p0 + tid * kScan;
    uint32_t m = free_pages(A.refs, p, A.pages, A.vec);
    int all, rank = have + block_scan(__popc(m), shared, &all);
    for (; m && rank < want; m &= m - 1, ++rank) {
      const int32_t id = (int32_t)(p + __builtin_ctz(m));
      if (rank < kPlan) fresh[rank] = id; else A.fresh[rank] = id;
    }
    have += all;
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
// compacting: one block plans
// ---------------------------------------------------------------------------

struct CompactArgs {
  int32_t *refs, *used, *where;
  int32_t* copies;    // their number, and from [4] on the pairs (from, to)
  int32_t pages;
  bool vec;
};

__global__ __launch_bounds__(kPlan) void compact_kernel(CompactArgs A) {
  __shared__ int shared[kPlan / 64];
  const int tid = threadIdx.x;
  constexpr int kRound = kPlan * kScan;
  int used = 0;
  for (int64_t p0 = 0; p0 < A.pages; p0 += kRound) {
    const int64_t p = p0 + tid * kScan;
    const int64_t n = p < A.pages ? (A.pages - p < kScan ? A.pages - p : kScan) : 0;
    used += (int)n - __popc(free_pages(A.refs, p, A.pages, A.vec));
  }
  int all;
  block_scan(used, shared, &all);
  used = all;
  // holes below `used` and pages in use from there on: the k-th of these goes to the k-th of those
  int holes = 0, movers = 0;
  for (int64_t p0 = 0; p0 < A.pages; p0 += kRound) {
    const int64_t p = p0 + tid * kScan;
    const uint32_t inside = p >= A.pages ? 0 : A.pages - p < kScan ? (1u << (A.pages - p)) - 1 : (1u << kScan) - 1;
    const uint32_t low = p >= used ? 0 : used - p < kScan ? (1u << (used - p)) - 1 : (1u << kScan) - 1;
    const uint32_t empty = free_pages(A.refs, p, A.pages, A.vec) & inside;
    uint32_t hole = empty & low, mover = inside & ~empty & ~low;
#pragma unroll
    for (int i = 0; i < kScan; ++i)
      if ((inside >> i) & 1) A.where[p + i] = (empty >> i) & 1 ? -1 : (int32_t)(p + i);
    int sum;   // a round has at most 2^14 of each
    const int before = block_scan(__popc(hole) | (__popc(mover) << 16), shared, &sum);
    for (int k = holes + (before & 0xffff); hole; hole &= hole - 1, ++k) A.copies[5 + 2 * k] = (int32_t)(p + __builtin_ctz(hole));
    for (int k = movers + (before >> 16); mover; mover &= mover - 1, ++k) A.copies[4 + 2 * k] = (int32_t)(p + __builtin_ctz(mover));
    holes += sum & 0xffff;
    movers += sum >> 16;
  }
  __syncthreads();
  for (int k = tid; k < movers; k += kPlan) {
    const int32_t from = A.copies[4 + 2 * k], to = A.copies[5 + 2 * k];
    A.where[from] = to;
    A.refs[to] = A.refs[from];
    A.refs[from] = 0;
  }
  if (tid == 0) {
    A.copies[0] = movers;
    *A.used = used;
  }
}

// ---------------------------------------------------------------------------
// copying
// ---------------------------------------------------------------------------

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct CopyArgs {
  const int32_t* copies;
  int64_t page_bytes;       // of a side
  int32_t heads, layers, pieces;
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
// through, 58 with loads past them as well.
template <bool ONCE>
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
  const uint32_t all = (uint32_t)A.copies[0] * (uint32_t)A.pieces;
  uint8_t* const base = side ? A.v[layer] : A.k[layer];
  for (uint32_t at = blockIdx.x; at < all; at += gridDim.x) {
    const uint32_t pair = at / (uint32_t)A.pieces, piece = at - pair * (uint32_t)A.pieces;
    const int64_t from = A.copies[4 + 2 * pair], to = A.copies[5 + 2 * pair];
    const u32x4_t* src = (const u32x4_t*)(base + from * A.page_bytes);
    u32x4_t* dst = (u32x4_t*)(base + to * A.page_bytes);
    const int64_t vecs = A.page_bytes / 16, first = (int64_t)piece * (kPiece / 16) + threadIdx.x;
    u32x4_t x[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const u32x4_t* at = src + first + i * kThreads;
      if (first + i * kThreads < vecs) x[i] = ONCE ? __builtin_nontemporal_load(at) : *at;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (first + i * kThreads < vecs) __builtin_nontemporal_store(x[i], dst + first + i * kThreads);
    if (piece == 0) {
      uint8_t* scales = side ? A.vs[layer] : A.ks[layer];
      for (int h = threadIdx.x; h < A.heads; h += kThreads) scales[to * A.heads + h] = scales[from * A.heads + h];
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
    int64_t x = most < row ? std::min(row, most * std::min<int64_t>(A.pieces, row)) : row;
    if (rewrite) x = std::max(x, std::min(blocks_of(cells), row));
    if (x > 0) copy_kernel<ONCE><<<dim3((uint32_t)x, (uint32_t)(2 * A.layers + (rewrite ? 1 : 0))), dim3(kThreads), 0, s>>>(A);
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

namespace nvfp4host {

int64_t kv_reserve_items(int64_t tokens, int64_t batch, int64_t page, bool offsets) {
  return offsets ? tokens / page + 2 * batch : batch;
}

int64_t kv_reserve_bytes(int64_t items, int64_t batch) { return ((4 + 2 * batch + 2 * items + 1) * 4 + 255) / 256 * 256; }

int64_t kv_compact_bytes(int64_t pages) { return ((4 + pages + 1) * 4 + 255) / 256 * 256; }

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
  reserve_kernel<<<dim3(1), dim3(kPlan), 0, s>>>(A);
  launch_copies<false>(caches, count, A.copies, batch, nullptr, nullptr, 0, s);
}

void launch_kv_compact(const nvfp4_kv_cache_t* caches, int64_t count, int32_t* table, int64_t batch, int64_t width,
                       int32_t* refs, void* ws, int32_t* used, int32_t* where, hipStream_t s) {
  const CompactArgs A = {refs, used, where, (int32_t*)ws, (int32_t)caches->pages, aligned16(refs)};
  compact_kernel<<<dim3(1), dim3(kPlan), 0, s>>>(A);
  launch_copies<true>(caches, count, A.copies, caches->pages / 2, table, where, batch * width, s);
}

}  // namespace nvfp4host
