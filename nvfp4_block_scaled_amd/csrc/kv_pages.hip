// Pages of the key/value cache: copy, fork, resize (free and take), compact.
//
// A pool's state is one reference count per page; a page is free at <= 0 and
// pages are taken lowest id first, so every result is a function of the inputs
// alone (atomic adds only count). The host never waits: what one kernel finds
// (which pages are free, how many move) the next reads from the workspace.
//
// Copying is bound by memory: every page byte is read once and written once, 16
// bytes a lane, four loads in flight per lane: a fork that copies 302 MB takes
// 51.2 us (5.9 TB/s: shared sources come from the caches), a compaction that moves
// 283 MB 57.5 us (4.9 TB/s; a large copy: 4.7). The bookkeeping is bound by the
// latency of a few dependent passes over the counts: 5 to 7 us before a copy, 11.3
// for a resize of 256 sequences in a pool of 65536 pages (three launches).
#include "kv_common.hpp"

namespace nvfp4 {

static constexpr int kScanThreads = 1024;
static constexpr int kPerThread = 16;                       // counts that a thread of a scan holds
static constexpr int kScanSpan = kScanThreads * kPerThread;
static constexpr int kNearStarts = 4096;
static constexpr int kSegment = kScanSpan;                  // counts of one workgroup of the compact scan

// Exclusive prefix sum over the workgroup; *total gets the sum. red: one int per wave, plus one.
__device__ __forceinline__ int block_scan(int v, int *red, int *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63) red[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < waves; w++) {
    const int r = red[w];
    before += w < wave ? r : 0;
    all += r;
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

// Which of the kPerThread counts from `first` on are above zero (LIVE) or not, as bits; none past `end`.
template <bool LIVE>
__device__ __forceinline__ uint32_t count_bits(const int32_t *refs, int64_t first, int64_t end) {
  uint32_t bits = 0;
  if (first + kPerThread <= end) {
    u32x4_t w[kPerThread / 4];
#pragma unroll
    for (int i = 0; i < kPerThread / 4; i++) w[i] = *reinterpret_cast<const u32x4_a4 *>(refs + first + 4 * i);
#pragma unroll
    for (int i = 0; i < kPerThread; i++) bits |= ((int)w[i >> 2][i & 3] > 0) == LIVE ? 1u << i : 0u;
  } else {
    for (int i = 0; i < kPerThread; i++)
      if (first + i < end && (refs[first + i] > 0) == LIVE) bits |= 1u << i;
  }
  return bits;
}

// ---------------------------------------------------------------- copying

struct Pool {
  uint8_t *base;
  int64_t layer_stride, page_stride;
  int32_t layers, num_pages;
  uint32_t units;                  // 16-byte units of a page
};

static constexpr int kCopyThreads = 256;
static constexpr int kCopyUnits = kCopyThreads * 4;         // units that a workgroup copies at a time

// One workgroup's part `part` of copying page src to dst in a layer (ids checked by the caller).
__device__ __forceinline__ void copy_part(const Pool &pool, int layer, int src, int dst, uint32_t part) {
  const u32x4_t *from = reinterpret_cast<const u32x4_t *>(pool.base + layer * pool.layer_stride + src * pool.page_stride);
  u32x4_t *to = reinterpret_cast<u32x4_t *>(pool.base + layer * pool.layer_stride + dst * pool.page_stride);
  const uint32_t u = part * kCopyUnits + threadIdx.x;
  u32x4_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (u + i * kCopyThreads < pool.units) w[i] = __builtin_nontemporal_load(from + u + i * kCopyThreads);
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (u + i * kCopyThreads < pool.units) __builtin_nontemporal_store(w[i], to + u + i * kCopyThreads);
}

// Copies the pairs (src[i], dst[i]), i < n, in all layers; a work item is one part of one page of one layer.
__device__ __forceinline__ void copy_pairs(const Pool &pool, const int32_t *src, const int32_t *dst, int n,
                                           uint32_t block, uint32_t blocks) {
  const uint32_t parts = (pool.units + kCopyUnits - 1) / kCopyUnits;
  const uint64_t per_pair = (uint64_t)parts * pool.layers, items = per_pair * n;
  for (uint64_t it = block; it < items; it += blocks) {
    const int i = (int)(it / per_pair);
    const uint32_t rest = (uint32_t)(it - i * per_pair);
    const int layer = rest / parts;
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= pool.num_pages || d < 0 || d >= pool.num_pages) continue;
    copy_part(pool, layer, s, d, rest - layer * parts);
  }
}

__global__ __launch_bounds__(kCopyThreads) void copy_pages_kernel(const Pool pool, const int32_t *src,
                                                                  const int32_t *dst, int n) {
  copy_pairs(pool, src, dst, n, blockIdx.x, gridDim.x);
}

__global__ __launch_bounds__(256) void copy_counts_kernel(const int32_t *from, int32_t *to, int n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) to[i] = from[i];
}

// ------------------------------------------------------------------- fork

struct ForkArgs {
  Pool pool;
  int32_t log_p, batch, children;
  int64_t width, table_stride, child_stride;
  const int32_t *table, *lens, *parents;
  const int32_t *refs_in;
  int32_t *child_table, *refs, *short_dev;
  int32_t *src, *dst;              // workspace: the page each child copies, and where to (-1: none, -2: not served)
};

// Pages a sequence of n tokens holds, its length taken as 0 .. width * page.
__device__ __forceinline__ int clamp_len(int n, int64_t width, int log_p) {
  const int64_t most = width << log_p;
  return n < 0 ? 0 : (int64_t)n > most ? (int)most : n;
}

// Takes free pages lowest id first for `need` takers: give(rank, page) for each; one workgroup.
// Returns how many were found (at most need).
template <typename Give>
__device__ __forceinline__ int take_pages(const int32_t *refs, int num_pages, int need, int *red, Give give) {
  int found = 0;
  for (int64_t base = 0; base < num_pages && found < need; base += kScanSpan) {
    const int64_t first = base + (int64_t)threadIdx.x * kPerThread;
    uint32_t free_bits = count_bits<false>(refs, first, num_pages);
    int total;
    int rank = found + block_scan(__popc(free_bits), red, &total);
    while (free_bits && rank < need) {
      const int i = __ffs((int)free_bits) - 1;
      free_bits &= free_bits - 1;
      give(rank, (int)(first + i));
      rank++;
    }
    found += total;
  }
  return min(found, need);
}

// One workgroup: which children can be served, and the page that each copies to.
__global__ __launch_bounds__(kScanThreads) void fork_plan_kernel(const ForkArgs A) {
  __shared__ int red[kScanThreads / 64 + 1];
  int need = 0, bad = 0;
  // first the rank of each child among those that need a page, in dst
  for (int base = 0; base < A.children; base += kScanThreads) {
    const int c = base + threadIdx.x;
    int wants = 0, src = -1, ok = 0;
    if (c < A.children) {
      const int p = A.parents[c];
      if (p >= 0 && p < A.batch) {
        const int n = A.lens[p];
        if (n >= 0 && (int64_t)n <= (A.width << A.log_p)) {
          ok = 1;
          const int whole = n >> A.log_p;
          if (n & ((1 << A.log_p) - 1)) {
            src = A.table[p * A.table_stride + whole];
            if (src < 0 || src >= A.pool.num_pages) ok = 0;
            else wants = 1;
          }
        }
      }
      if (!ok) bad++;
    }
    int total;
    const int rank = need + block_scan(wants, red, &total);
    need += total;
    if (c < A.children) {
      A.src[c] = wants ? src : -1;
      A.dst[c] = ok ? (wants ? rank : -1) : -2;
    }
  }
  __syncthreads();
  // pages by rank go to the second half of the dst array
  int32_t *page_of = A.dst + A.children;
  const int found = take_pages(A.refs_in, A.pool.num_pages, need, red, [&](int rank, int page) { page_of[rank] = page; });
  if (A.refs != A.refs_in && A.pool.num_pages <= kScanSpan)      // (a larger pool's counts are copied beforehand)
    for (int i = threadIdx.x; i < A.pool.num_pages; i += kScanThreads) A.refs[i] = A.refs_in[i];
  __syncthreads();
  for (int c = threadIdx.x; c < A.children; c += kScanThreads) {
    const int rank = A.dst[c];
    if (rank < 0) continue;
    if (rank < found) {
      const int page = page_of[rank];
      A.dst[c] = page;
      A.refs[page] = 1;
    } else {
      A.dst[c] = -2;
      bad++;
    }
  }
  int total;
  block_scan(bad, red, &total);
  if (threadIdx.x == 0) *A.short_dev = total;
}

// Copies pages (the first blocks of the grid), writes the children's rows and raises the counts of
// shared pages (the last `children` blocks).
__global__ __launch_bounds__(kCopyThreads) void fork_copy_kernel(const ForkArgs A, int copy_blocks) {
  if ((int)blockIdx.x < copy_blocks) {
    copy_pairs(A.pool, A.src, A.dst, A.children, blockIdx.x, copy_blocks);
    return;
  }
  const int c = blockIdx.x - copy_blocks;
  const int dst = A.dst[c];
  const bool ok = dst != -2;
  const int p = ok ? A.parents[c] : 0;
  const int whole = ok ? A.lens[p] >> A.log_p : 0;
  for (int64_t i = threadIdx.x; i < A.width; i += kCopyThreads) {
    int e = -1;
    if (ok && i < whole) {
      e = A.table[p * A.table_stride + i];
      if (e >= 0 && e < A.pool.num_pages) atomicAdd(A.refs + e, 1);
    } else if (ok && i == whole && dst >= 0) {
      e = dst;
    }
    A.child_table[c * A.child_stride + i] = e;
  }
}

// ----------------------------------------------------------------- resize

struct ResizeArgs {
  int32_t num_pages, log_p, batch;
  int64_t width, table_stride, out_stride;
  const int32_t *table, *lens, *new_lens;
  int32_t *table_out, *refs, *short_dev;
  int32_t *starts;                 // workspace [batch]: entries that sequences before b take,
  int32_t *taken;                  // and [num_pages]: the pages in the order in which they are taken
};

// A workgroup per sequence: gives back what it drops and writes its row: kept entries, -1 elsewhere.
__global__ __launch_bounds__(256) void resize_rows_kernel(const ResizeArgs A) {
  const int b = blockIdx.x;
  const int was = (clamp_len(A.lens[b], A.width, A.log_p) + (1 << A.log_p) - 1) >> A.log_p;
  const int now = (clamp_len(A.new_lens[b], A.width, A.log_p) + (1 << A.log_p) - 1) >> A.log_p;
  const bool in_place = A.table == A.table_out;
  for (int64_t i = (in_place ? min(was, now) : 0) + threadIdx.x; i < (in_place ? max(was, now) : A.width); i += 256) {
    const bool drop = i >= now && i < was, grow = i >= was && i < now;
    const int e = grow ? -1 : A.table[b * A.table_stride + i];
    if (drop && e >= 0 && e < A.num_pages) atomicAdd(A.refs + e, -1);
    A.table_out[b * A.out_stride + i] = (drop || grow) ? -1 : e;
  }
}

// One workgroup: hands free pages out, in the order of sequences and positions.
__global__ __launch_bounds__(kScanThreads) void resize_plan_kernel(const ResizeArgs A) {
  __shared__ int red[kScanThreads / 64 + 1];
  __shared__ int near[kNearStarts];                 // the sequences' starts, where they fit: they are searched
  const bool fits = A.batch <= kNearStarts;
  int need = 0;
  for (int base = 0; base < A.batch; base += kScanThreads) {
    const int b = base + threadIdx.x;
    int grow = 0;
    if (b < A.batch) {
      const int was = (clamp_len(A.lens[b], A.width, A.log_p) + (1 << A.log_p) - 1) >> A.log_p;
      const int now = (clamp_len(A.new_lens[b], A.width, A.log_p) + (1 << A.log_p) - 1) >> A.log_p;
      grow = max(0, now - was);
    }
    int total;
    const int before = need + block_scan(grow, red, &total);
    if (b < A.batch) (fits ? near : A.starts)[b] = before;
    need += total;
  }
  __syncthreads();
  // first which pages, by the threads that find them free; then whose they are, a thread per page
  const int found = take_pages(A.refs, A.num_pages, need, red, [&](int rank, int page) {
    A.taken[rank] = page;
    A.refs[page] = 1;
  });
  __syncthreads();
  for (int rank = threadIdx.x; rank < found; rank += kScanThreads) {
    int lo = 0, hi = A.batch - 1;                 // the last sequence whose start is <= rank
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((fits ? near[mid] : A.starts[mid]) <= rank) lo = mid;
      else hi = mid - 1;
    }
    const int was = (clamp_len(A.lens[lo], A.width, A.log_p) + (1 << A.log_p) - 1) >> A.log_p;
    A.table_out[lo * A.out_stride + was + (rank - (fits ? near[lo] : A.starts[lo]))] = A.taken[rank];
  }
  if (threadIdx.x == 0) *A.short_dev = need - found;
}

// ---------------------------------------------------------------- compact

struct CompactArgs {
  Pool pool;
  int32_t batch, segments;
  int64_t width, table_stride, out_stride;
  const int32_t *table, *refs;
  int32_t *table_out, *refs_out, *live_dev;
  int32_t *counts;                 // workspace [segments]: live pages of each segment
  int32_t *holes, *movers, *rank;  // workspace [num_pages] each; counts[segments] holds how many move
};

__global__ __launch_bounds__(kScanThreads) void compact_count_kernel(const CompactArgs A) {
  __shared__ int red[kScanThreads / 64 + 1];
  const int64_t first = (int64_t)blockIdx.x * kSegment + threadIdx.x * kPerThread;
  int total;
  block_scan(__popc(count_bits<true>(A.refs, first, A.pool.num_pages)), red, &total);
  if (threadIdx.x == 0) A.counts[blockIdx.x] = total;
}

// With n live pages: live id >= n -> the list of movers, free id < n -> the list of holes, both in
// ascending order, so that mover r goes to hole r. A live page's rank among the live ones is the
// prefix sum of the counts; a mover's rank is that less the live pages below n.
__global__ __launch_bounds__(kScanThreads) void compact_plan_kernel(const CompactArgs A) {
  __shared__ int red[kScanThreads / 64 + 1];
  const int64_t first = (int64_t)blockIdx.x * kSegment + threadIdx.x * kPerThread;
  const uint32_t bits = count_bits<true>(A.refs, first, A.pool.num_pages);
  int live, mine = 0, total;
  int rank = block_scan(__popc(bits), red, &total);
  if (A.segments == 1) {
    live = total;
  } else {
    int all = 0, before = 0;
    for (int i = threadIdx.x; i < A.segments; i += kScanThreads) {
      const int c = A.counts[i];
      all += c;
      before += i < (int)blockIdx.x ? c : 0;
    }
    block_scan(all, red, &live);
    block_scan(before, red, &mine);                  // live pages before this segment
    rank += mine;
  }
  // Live pages below `live`: whole segments, then part of one. In a pool with no free page that is all of
  // them, known without the counts (a full pool of one whole segment has none to read).
  int staying = live;
  if (live < A.pool.num_pages) {
    const int cut = live / kSegment;
    int below = 0;
    for (int i = threadIdx.x; i < cut; i += kScanThreads) below += A.counts[i];
    const int64_t part = (int64_t)cut * kSegment + threadIdx.x * kPerThread;
    below += __popc(count_bits<true>(A.refs, part, live));
    block_scan(below, red, &staying);
  }

#pragma unroll
  for (int i = 0; i < kPerThread; i++) {
    const int64_t id = first + i;
    if (id >= A.pool.num_pages) break;
    const bool alive = (bits >> i) & 1u;
    int r = -1;
    if (alive && id >= live) {
      r = rank - staying;
      A.movers[r] = (int)id;
    } else if (!alive && id < live) {
      A.holes[id - rank] = (int)id;
    }
    A.rank[id] = r;
    rank += alive;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    A.counts[A.segments] = live - staying;           // how many move
    *A.live_dev = live;
  }
}

// Three jobs by block ranges: copy the moving pages, renumber the table, write the counts.
__global__ __launch_bounds__(kCopyThreads) void compact_move_kernel(const CompactArgs A, int copy_blocks,
                                                                    int table_blocks) {
  const int moves = A.counts[A.segments];
  int b = blockIdx.x;
  if (b < copy_blocks) {
    copy_pairs(A.pool, A.movers, A.holes, moves, b, copy_blocks);
    return;
  }
  b -= copy_blocks;
  if (b < table_blocks) {
    const int64_t n = A.width * A.batch;
    for (int64_t i = (int64_t)b * kCopyThreads + threadIdx.x; i < n; i += (int64_t)table_blocks * kCopyThreads) {
      const int64_t row = i / A.width, col = i - row * A.width;
      const int e = A.table[row * A.table_stride + col];
      const int r = e >= 0 && e < A.pool.num_pages ? A.rank[e] : -1;
      A.table_out[row * A.out_stride + col] = r >= 0 ? A.holes[r] : e;
    }
    return;
  }
  b -= table_blocks;
  const int blocks = gridDim.x - copy_blocks - table_blocks;
  const int start = b * kCopyThreads + threadIdx.x, step = blocks * kCopyThreads;
  for (int64_t r = start; r < moves; r += step) {
    const int from = A.movers[r];
    const int count = A.refs[from];
    A.refs_out[A.holes[r]] = count;
    A.refs_out[from] = 0;
  }
  // (In place, a mover's count may be read before or after the loop above clears it: neither writes
  // anything but zero there.)
  const int live = *A.live_dev;
  for (int64_t id = start; id < A.pool.num_pages; id += step) {
    const int count = A.refs[id];
    const bool alive = count > 0;
    if (alive && id < live && A.refs_out != A.refs) A.refs_out[id] = count;   // stays
    else if (!alive && id >= live) A.refs_out[id] = 0;                        // free before and after
  }
}

}  // namespace nvfp4

using namespace nvfp4;

namespace {

nvfp4_status pool_of(const nvfp4_kv_pool *p, Pool *out) {
  if (!p) return NVFP4_ERR_NULL;
  if (p->layers < 1 || p->layers > 65535 || p->num_pages < 1 || p->num_pages > 0x3FFFFFFF || p->page_bytes < 16 ||
      p->page_bytes > ((int64_t)1 << 34) || p->page_stride < p->page_bytes)
    return NVFP4_ERR_SHAPE;
  if (p->page_stride > INT64_MAX / p->num_pages || (p->layers > 1 && p->layer_stride < 0)) return NVFP4_ERR_SHAPE;
  if (p->layers > 1 && p->layer_stride > INT64_MAX / p->layers) return NVFP4_ERR_SHAPE;
  if (!p->base) return NVFP4_ERR_NULL;
  if (!aligned(p->base, 16) || p->page_stride % 16 != 0 || p->page_bytes % 16 != 0 ||
      (p->layers > 1 && p->layer_stride % 16 != 0))
    return NVFP4_ERR_ALIGN;
  out->base = p->base;
  out->layer_stride = p->layers > 1 ? p->layer_stride : 0;
  out->page_stride = p->page_stride;
  out->layers = (int32_t)p->layers;
  out->num_pages = (int32_t)p->num_pages;
  out->units = (uint32_t)(p->page_bytes / 16);
  return NVFP4_OK;
}

bool page_size_ok(int32_t p) { return p >= 1 && p <= 65536 && (p & (p - 1)) == 0; }

// A table of rows x width page ids whose lengths fit 31 bits.
nvfp4_status table_ok(const int32_t *table, int64_t stride, int64_t width, int64_t rows, int32_t page_size) {
  if (width < 1 || rows < 1 || rows > (1 << 24) || (rows > 1 && stride < width) ||
      width > 0x7FFFFFFF / page_size)
    return NVFP4_ERR_SHAPE;
  if (!table) return NVFP4_ERR_NULL;
  return aligned(table, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// Whether two tables with rows of `width` entries share none: one lies behind the other, or their rows
// are different columns of one wider table.
bool tables_apart(const int32_t *a, int64_t a_stride, int64_t a_rows, const int32_t *b, int64_t b_stride, int64_t b_rows,
                  int64_t width) {
  const __int128 a0 = (__int128)((uintptr_t)a / 4), b0 = (__int128)((uintptr_t)b / 4);
  if (a0 + (__int128)(a_rows - 1) * a_stride + width <= b0 || b0 + (__int128)(b_rows - 1) * b_stride + width <= a0) return true;
  if ((a_rows == 1 && b_rows == 1) || (a_rows > 1 && b_rows > 1 && a_stride != b_stride)) return false;
  const int64_t stride = a_rows > 1 ? a_stride : b_stride;
  const __int128 off = ((b0 - a0) % stride + stride) % stride;
  return off >= width && off + width <= stride;
}

bool ints_ok(const void *p) { return aligned(p, 4); }

// Blocks for copying `pairs` pages in all layers, eight workgroups for each CU at most.
int copy_grid(const Pool &pool, int64_t pairs, int cus) {
  const int64_t parts = (pool.units + kCopyUnits - 1) / kCopyUnits;
  const int64_t items = parts * pool.layers * pairs;
  const int64_t most = (int64_t)cus * 8;
  return (int)(items < most ? (items < 1 ? 1 : items) : most);
}

// Counts for an operation that changes them elsewhere than in place.
nvfp4_status copy_counts(const int32_t *from, int32_t *to, int64_t n, hipStream_t s) {
  if (from == to) return NVFP4_OK;
  const int64_t blocks = (n + 255) / 256;
  hipLaunchKernelGGL(copy_counts_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, s, from, to,
                     (int)n);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

nvfp4_status ws_ok(void *ws, size_t have, size_t need) {
  if (!ws || have < need) return NVFP4_ERR_WORKSPACE;
  return aligned(ws, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t nvfp4_kv_pages_workspace_bytes(int64_t num_pages, int64_t batch) {
  if (num_pages < 1 || num_pages > 0x3FFFFFFF || batch < 0 || batch > (1 << 24)) return 0;
  const int64_t segments = (num_pages + kSegment - 1) / kSegment;
  const int64_t compact = segments + 4 + 3 * num_pages, rows = 3 * batch + 4;
  return (size_t)((compact > rows ? compact : rows) * 4 + 15) / 16 * 16;
}

nvfp4_status nvfp4_kv_copy_pages(const nvfp4_kv_pool *pool, const int32_t *src, const int32_t *dst, int64_t n,
                                 void *stream) {
  Pool p;
  nvfp4_status st = pool_of(pool, &p);
  if (st != NVFP4_OK) return st;
  if (n < 0 || n > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  if (n == 0) return NVFP4_OK;
  if (!src || !dst) return NVFP4_ERR_NULL;
  if (!ints_ok(src) || !ints_ok(dst)) return NVFP4_ERR_ALIGN;
  DeviceInfo d;
  st = device_info(&d);
  if (st != NVFP4_OK) return st;
  hipLaunchKernelGGL(copy_pages_kernel, dim3(copy_grid(p, n, d.num_cus)), dim3(kCopyThreads), 0, (hipStream_t)stream, p,
                     src, dst, (int)n);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

nvfp4_status nvfp4_kv_fork(const nvfp4_kv_pool *pool, int32_t page_size, const int32_t *table, int64_t table_stride,
                           int64_t width, int64_t batch, const int32_t *lens, const int32_t *refs,
                           const int32_t *parents, int64_t children, int32_t *child_table, int64_t child_stride,
                           int32_t *refs_out, int32_t *short_dev, void *ws, size_t ws_bytes, void *stream) {
  ForkArgs A = {};
  nvfp4_status st = pool_of(pool, &A.pool);
  if (st != NVFP4_OK) return st;
  if (!page_size_ok(page_size)) return NVFP4_ERR_SHAPE;
  if ((st = table_ok(table, table_stride, width, batch, page_size)) != NVFP4_OK) return st;
  if (children < 0 || children > (1 << 24) || (children > 1 && child_stride < width)) return NVFP4_ERR_SHAPE;
  if (!lens || !refs || !refs_out || !short_dev || (children > 0 && (!parents || !child_table))) return NVFP4_ERR_NULL;
  if (!ints_ok(lens) || !ints_ok(refs) || !ints_ok(refs_out) || !ints_ok(short_dev) || !ints_ok(parents) ||
      !ints_ok(child_table))
    return NVFP4_ERR_ALIGN;
  if ((st = ws_ok(ws, ws_bytes, nvfp4_kv_pages_workspace_bytes(pool->num_pages, children))) != NVFP4_OK) return st;
  // a child's row written over a parent's that another child still reads
  if (children > 0 && !tables_apart(table, table_stride, batch, child_table, child_stride, children, width)) return NVFP4_ERR_VALUE;
  DeviceInfo d;
  st = device_info(&d);
  if (st != NVFP4_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  A.log_p = __builtin_ctz((unsigned)page_size);
  A.batch = (int32_t)batch, A.children = (int32_t)children;
  A.width = width, A.table_stride = table_stride, A.child_stride = child_stride;
  A.table = table, A.lens = lens, A.parents = parents;
  A.child_table = child_table, A.refs_in = refs, A.refs = refs_out, A.short_dev = short_dev;
  A.src = (int32_t *)ws, A.dst = A.src + children;
  if (A.pool.num_pages > kScanSpan && (st = copy_counts(refs, refs_out, A.pool.num_pages, s)) != NVFP4_OK) return st;
  hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(kScanThreads), 0, s, A);
  NVFP4_LAUNCH_CHECK();
  if (children == 0) return NVFP4_OK;
  const int copies = copy_grid(A.pool, children, d.num_cus);
  hipLaunchKernelGGL(fork_copy_kernel, dim3((unsigned)(copies + children)), dim3(kCopyThreads), 0, s, A, copies);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

nvfp4_status nvfp4_kv_resize(int64_t num_pages, int32_t page_size, const int32_t *table, int64_t table_stride,
                             int64_t width, int64_t batch, const int32_t *lens, const int32_t *new_lens,
                             const int32_t *refs, int32_t *table_out, int64_t table_out_stride, int32_t *refs_out,
                             int32_t *short_dev, void *ws, size_t ws_bytes, void *stream) {
  if (num_pages < 1 || num_pages > 0x3FFFFFFF || !page_size_ok(page_size)) return NVFP4_ERR_SHAPE;
  nvfp4_status st = table_ok(table, table_stride, width, batch, page_size);
  if (st != NVFP4_OK) return st;
  if ((st = table_ok(table_out, table_out_stride, width, batch, page_size)) != NVFP4_OK) return st;
  if (!lens || !new_lens || !refs || !refs_out || !short_dev) return NVFP4_ERR_NULL;
  if (!ints_ok(lens) || !ints_ok(new_lens) || !ints_ok(refs) || !ints_ok(refs_out) || !ints_ok(short_dev))
    return NVFP4_ERR_ALIGN;
  if (table == table_out && batch > 1 && table_stride != table_out_stride) return NVFP4_ERR_SHAPE;
  if (width > 0x7FFFFFFF / batch) return NVFP4_ERR_SHAPE;         // the plan adds up entries in 32 bits
  if ((st = ws_ok(ws, ws_bytes, nvfp4_kv_pages_workspace_bytes(num_pages, batch))) != NVFP4_OK) return st;
  DeviceInfo d;
  st = device_info(&d);
  if (st != NVFP4_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  ResizeArgs A = {};
  A.num_pages = (int32_t)num_pages, A.log_p = __builtin_ctz((unsigned)page_size), A.batch = (int32_t)batch;
  A.width = width, A.table_stride = table_stride, A.out_stride = table_out_stride;
  A.table = table, A.lens = lens, A.new_lens = new_lens;
  A.table_out = table_out, A.refs = refs_out, A.short_dev = short_dev;
  A.starts = (int32_t *)ws, A.taken = A.starts + batch;    // (batch + num_pages <= 3 max(batch, num_pages))
  if ((st = copy_counts(refs, refs_out, num_pages, s)) != NVFP4_OK) return st;
  hipLaunchKernelGGL(resize_rows_kernel, dim3((unsigned)batch), dim3(256), 0, s, A);
  NVFP4_LAUNCH_CHECK();
  hipLaunchKernelGGL(resize_plan_kernel, dim3(1), dim3(kScanThreads), 0, s, A);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

nvfp4_status nvfp4_kv_compact(const nvfp4_kv_pool *pool, const int32_t *table, int64_t table_stride, int64_t width,
                              int64_t batch, const int32_t *refs, int32_t *table_out, int64_t table_out_stride,
                              int32_t *refs_out, int32_t *live_dev, void *ws, size_t ws_bytes, void *stream) {
  CompactArgs A = {};
  nvfp4_status st = pool_of(pool, &A.pool);
  if (st != NVFP4_OK) return st;
  if ((st = table_ok(table, table_stride, width, batch, 1)) != NVFP4_OK) return st;
  if ((st = table_ok(table_out, table_out_stride, width, batch, 1)) != NVFP4_OK) return st;
  if (!refs || !refs_out || !live_dev) return NVFP4_ERR_NULL;
  if (!ints_ok(refs) || !ints_ok(refs_out) || !ints_ok(live_dev)) return NVFP4_ERR_ALIGN;
  if (table == table_out && batch > 1 && table_stride != table_out_stride) return NVFP4_ERR_SHAPE;
  if ((st = ws_ok(ws, ws_bytes, nvfp4_kv_pages_workspace_bytes(pool->num_pages, batch))) != NVFP4_OK) return st;
  DeviceInfo d;
  st = device_info(&d);
  if (st != NVFP4_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  const int32_t np = A.pool.num_pages;
  A.batch = (int32_t)batch;
  A.segments = (np + kSegment - 1) / kSegment;
  A.width = width, A.table_stride = table_stride, A.out_stride = table_out_stride;
  A.table = table, A.refs = refs, A.table_out = table_out, A.refs_out = refs_out, A.live_dev = live_dev;
  A.holes = (int32_t *)ws, A.movers = A.holes + np, A.rank = A.movers + np, A.counts = A.rank + np;
  if (A.segments > 1) {               // (a single segment's workgroup counts for itself)
    hipLaunchKernelGGL(compact_count_kernel, dim3(A.segments), dim3(kScanThreads), 0, s, A);
    NVFP4_LAUNCH_CHECK();
  }
  hipLaunchKernelGGL(compact_plan_kernel, dim3(A.segments), dim3(kScanThreads), 0, s, A);
  NVFP4_LAUNCH_CHECK();
  const int copies = copy_grid(A.pool, np / 2 + 1, d.num_cus);
  const int64_t tb = (width * batch + 1023) / 1024, rb = ((int64_t)np + 1023) / 1024;
  const int tables = (int)(tb < 512 ? tb : 512), counts = (int)(rb < 512 ? rb : 512);
  hipLaunchKernelGGL(compact_move_kernel, dim3((unsigned)(copies + tables + counts)), dim3(kCopyThreads), 0, s, A, copies,
                     tables);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

}  // extern "C"
