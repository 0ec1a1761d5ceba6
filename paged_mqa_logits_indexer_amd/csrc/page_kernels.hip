// Care of the paged caches' pages (gfx950): requests released and forked, a pool
// compacted, and pages copied in the caches of all layers.
//
// refs[p] counts the requests (and whoever else) that hold page p; a page with no
// holder is free.  All of it stays on the GPU: which pages are free, which are
// copied and where to is found by the kernels, so a serving loop that forks and
// compacts needs no synchronisation.
//
//   release  refs[p] -= 1 for the pages of each request that ends
//   fork     a child shares its parent's full pages (refs + 1 each); the page that
//            the parent has begun is copied to the lowest free page, the requests
//            served in ascending order
//   compact  with L pages held, the i-th held page from L on moves to the i-th free
//            page below L (both ascending), so sources and destinations never meet
//   copy     (source, destination) pages in every cache, whole or their first tokens
//
// Copies are bound by memory (about 114 pages in 24 caches, 62 MB read and written
// together, 11.2 us: 5.5 TB/s, partly from the last-level cache), the rest by its few
// dependent round trips (release 2.4, fork 5.5 us for 64 requests, compact 6.1 us for a
// pool of 478 pages).
//
// The results are whole numbers and do not depend on timing: refs change by atomic
// additions alone, and every list is ordered by a scan.
#include "indexer_common.h"
#include "launches.h"

namespace pmqa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kPerThread = 4;                      // requests (or pages of a chunk) of a thread
constexpr int kPerGo = kPlanThreads * kPerThread;  // 4096: the most requests, and the pages of a chunk

// Exclusive scan over the workgroup of one count per thread; `total` is the sum.
__device__ __forceinline__ int block_scan(int n, int* s_waves, int& total) {
  const int upto = wave_inclusive_scan(n);
  __syncthreads();  // the sums of the call before have been read
  if (lane_id() == kWave - 1) s_waves[threadIdx.x / kWave] = upto;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kPlanWaves; ++i) {
    const int w = s_waves[i];
    before += i < static_cast<int>(threadIdx.x) / kWave ? w : 0;
    total += w;
  }
  return before + upto - n;
}

__device__ __forceinline__ int held_pages(int len, int max_pages) {
  return (max(0, min(len, max_pages * kPage)) + kPage - 1) / kPage;
}

// What every entry of the block table needs: its request, and its column.
struct Entry {
  int b, j;
};
__device__ __forceinline__ Entry entry_at(const PageArgs& a, int e) {
  const int b = e / a.max_pages;
  return {b, e - b * a.max_pages};
}

__device__ __forceinline__ void release_entry(const PageArgs& a, int page) {
  if (page >= 0 && page < a.num_pages) atomicSub(a.new_refs + page, 1);
}
__device__ __forceinline__ void share_entry(const PageArgs& a, int64_t to, int page) {
  a.block_table[to] = page;
  if (page >= 0 && page < a.num_pages) atomicAdd(a.new_refs + page, 1);
}
__device__ __forceinline__ void move_entry(const PageArgs& a, int64_t at, bool held, const int32_t* map) {
  const int page = a.block_table[at];
  a.new_table[at] = held && page >= 0 && page < a.num_pages ? map[page] : page;
}

// A whole release by one workgroup (a small pool).
__global__ __launch_bounds__(kPlanThreads) void release_small_kernel(PageArgs a) {
  const int tid = threadIdx.x;
  if (a.new_refs != a.refs)
    for (int i = tid; i < a.num_pages; i += kPlanThreads) a.new_refs[i] = a.refs[i];
  __syncthreads();
  for (int e = tid; e < a.requests * a.max_pages; e += kPlanThreads) {
    const Entry at = entry_at(a, e);
    if (a.mask[at.b] != 0 && at.j < held_pages(a.lens[at.b], a.max_pages)) release_entry(a, a.block_table[e]);
  }
  __syncthreads();  // (new_lens may be lens)
  for (int b = tid; b < a.requests; b += kPlanThreads) a.new_lens[b] = a.mask[b] != 0 ? 0 : a.lens[b];
}

// A copy of refs, where the result goes elsewhere.
__global__ __launch_bounds__(256) void copy_refs_kernel(const int32_t* __restrict__ refs, int n,
                                                        int32_t* __restrict__ out) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) out[i] = refs[i];
}

// One workgroup per request.
__global__ __launch_bounds__(256) void release_kernel(PageArgs a) {
  const int b = blockIdx.x;
  const bool ends = a.mask[b] != 0;
  const int len = a.lens[b];
  __syncthreads();  // (new_lens may be lens)
  if (threadIdx.x == 0) a.new_lens[b] = ends ? 0 : len;
  if (!ends) return;
  const int32_t* row = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const int n = held_pages(len, a.max_pages);
  for (int j = threadIdx.x; j < n; j += 256) release_entry(a, row[j]);
}

// A pool of many pages is a chunk per workgroup: held pages are counted in each, then
// every workgroup adds up the chunks before its own (and, to compact, those below L).
struct Held {
  int live;    // L: of the whole pool
  int below;   // of the pages below L
  int before;  // of the pages before this chunk
};

__global__ __launch_bounds__(kPlanThreads) void count_held_kernel(PageArgs a, int32_t* __restrict__ chunks) {
  __shared__ int s_waves[kPlanWaves];
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int p = blockIdx.x * kPerGo + i * kPlanThreads + threadIdx.x;
    n += p < a.num_pages && a.refs[p] > 0;
  }
  int total;
  block_scan(n, s_waves, total);
  if (threadIdx.x == 0) chunks[blockIdx.x] = total;
}

__device__ __forceinline__ Held add_up(const PageArgs& a, const int32_t* chunks, int n_chunks, int mine, int* s_waves) {
  Held h;
  int all = 0, before = 0;
  for (int c = threadIdx.x; c < n_chunks; c += kPlanThreads) {
    const int n = chunks[c];
    all += n;
    before += c < mine ? n : 0;
  }
  block_scan(all, s_waves, h.live);
  block_scan(before, s_waves, h.before);
  const int border = h.live / kPerGo;  // the chunk that L lies in: its pages one by one
  int below = 0;
  for (int c = threadIdx.x; c < border; c += kPlanThreads) below += chunks[c];
  for (int p = border * kPerGo + threadIdx.x; p < h.live; p += kPlanThreads) below += a.refs[p] > 0;
  block_scan(below, s_waves, h.below);
  return h;
}

// The first free pages, ascending, as many as there are requests; refs to new_refs.
__global__ __launch_bounds__(kPlanThreads) void free_list_kernel(PageArgs a, const int32_t* __restrict__ chunks,
                                                                 int32_t* __restrict__ free) {
  __shared__ int s_waves[kPlanWaves];
  int held_before = 0, before;
  for (int c = threadIdx.x; c < static_cast<int>(blockIdx.x); c += kPlanThreads) held_before += chunks[c];
  block_scan(held_before, s_waves, before);
  const int p = blockIdx.x * kPerGo + static_cast<int>(threadIdx.x) * kPerThread;
  int r[kPerThread], n = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    r[i] = p + i < a.num_pages ? a.refs[p + i] : 1;
    n += r[i] > 0;
  }
  int total;
  int held = before + block_scan(n, s_waves, total);  // pages held before p + i
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (p + i >= a.num_pages) continue;
    if (r[i] <= 0 && p + i - held < a.requests) free[p + i - held] = p + i;
    held += r[i] > 0;
    if (a.new_refs != a.refs) a.new_refs[p + i] = r[i];
  }
}

// One workgroup.  Which requests are forked, and the page that each takes.  SMALL: it
// finds the free pages, copies refs to new_refs and adds the pages that are shared;
// otherwise free_list_kernel has done the first two (free, of `total` free pages) and
// fork_rows_kernel does the third, with inherit[b]: full pages that b takes over, -1
// for a request that is not forked.
template <bool SMALL>
__global__ __launch_bounds__(kPlanThreads) void fork_plan_kernel(PageArgs a, int32_t* __restrict__ inherit,
                                                                 const int32_t* __restrict__ free,
                                                                 const int32_t* __restrict__ chunks) {
  __shared__ int s_waves[kPlanWaves];
  __shared__ int s_inherit[SMALL ? kPerGo : 1];
  __shared__ int s_free[SMALL ? kPerGo : 1];  // pages for the requests that need one, in their order
  const int tid = threadIdx.x;
  // ---- requests, four in a row per thread
  int parent[kPerThread], len[kPerThread], from[kPerThread], rank[kPerThread];
  int needs = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    parent[i] = b < a.requests ? a.mask[b] : -1;
    len[i] = b < a.requests ? a.lens[b] : 0;
    // a request with tokens of its own, or a parent that is none, is left as it is
    if (parent[i] < 0 || parent[i] >= a.requests || len[i] > 0) parent[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    from[i] = parent[i] >= 0 ? max(0, min(a.lens[parent[i]], a.max_pages * kPage)) : 0;
    rank[i] = needs;
    needs += from[i] % kPage != 0;
  }
  int wanted;
  const int base = block_scan(needs, s_waves, wanted);
  // ---- the first free pages, ascending
  int found = 0;
  if constexpr (SMALL) {
    const bool copies = a.new_refs != a.refs;
    for (int p0 = 0; p0 < a.num_pages && (copies || found < wanted); p0 += kPerGo) {
      const int p = p0 + tid * kPerThread;
      int r[kPerThread], n = 0;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        r[i] = p + i < a.num_pages ? a.refs[p + i] : 1;
        n += r[i] <= 0;
      }
      if (copies) {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i)
          if (p + i < a.num_pages) a.new_refs[p + i] = r[i];
      }
      if (found < wanted) {  // (the same for all threads)
        int total;
        int at = found + block_scan(n, s_waves, total);
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
          if (r[i] > 0) continue;
          if (at < wanted) s_free[at] = p + i;
          ++at;
        }
        found += total;
      }
    }
  } else {
    int held = 0, all;
    for (int c = tid; c < (a.num_pages + kPerGo - 1) / kPerGo; c += kPlanThreads) held += chunks[c];
    block_scan(held, s_waves, all);
    found = a.num_pages - all;
  }
  found = min(found, wanted);
  __syncthreads();  // s_free and new_refs are written (and lens read: new_lens may be lens)
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    if (b >= a.requests) continue;
    const int full = from[i] / kPage, rest = from[i] % kPage;
    const bool takes = rest != 0 && base + rank[i] < found;
    const bool forked = parent[i] >= 0 && (rest == 0 || takes);
    int src = -1, dst = -1;
    if (takes) {
      src = a.block_table[static_cast<int64_t>(parent[i]) * a.max_pages + full];
      dst = SMALL ? s_free[base + rank[i]] : free[base + rank[i]];
      a.block_table[static_cast<int64_t>(b) * a.max_pages + full] = dst;
      a.new_refs[dst] = 1;
    }
    a.src[b] = src;
    a.dst[b] = dst;
    a.tokens[b] = takes ? rest : 0;
    a.new_lens[b] = forked ? from[i] : len[i];
    if constexpr (SMALL) s_inherit[b] = forked ? full : -1;
    else inherit[b] = forked ? full : -1;
  }
  if (tid == 0) {
    a.counts[0] = found;
    a.counts[1] = wanted - found;
  }
  if constexpr (SMALL) {
    __syncthreads();
    for (int e = tid; e < a.requests * a.max_pages; e += kPlanThreads) {
      const Entry at = entry_at(a, e);
      if (at.j < s_inherit[at.b]) share_entry(a, e, a.block_table[static_cast<int64_t>(a.mask[at.b]) * a.max_pages + at.j]);
    }
  }
}

// One workgroup per request: the full pages that it shares with its parent.
__global__ __launch_bounds__(256) void fork_rows_kernel(PageArgs a, const int32_t* __restrict__ inherit) {
  const int b = blockIdx.x;
  const int n = inherit[b];
  if (n <= 0) return;
  const int32_t* from = a.block_table + static_cast<int64_t>(a.mask[b]) * a.max_pages;
  for (int j = threadIdx.x; j < n; j += 256) share_entry(a, static_cast<int64_t>(b) * a.max_pages + j, from[j]);
}

// The moves that begin or end in a chunk, and, apart from them, map and new_refs.
__device__ __forceinline__ void list_chunk(const PageArgs& a, int chunk, const Held& h, int32_t* map, int* s_waves) {
  const int p = chunk * kPerGo + static_cast<int>(threadIdx.x) * kPerThread;
  int r[kPerThread], n = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    r[i] = p + i < a.num_pages ? a.refs[p + i] : 0;
    n += r[i] > 0;
  }
  int total;
  int held = h.before + block_scan(n, s_waves, total);  // pages held before p + i
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (p + i >= a.num_pages) continue;
    if (p + i >= h.live && r[i] > 0) a.src[held - h.below] = p + i;
    if (p + i < h.live && r[i] <= 0) a.dst[p + i - held] = p + i;
    held += r[i] > 0;
    map[p + i] = p + i;
    if (a.new_refs != a.refs) a.new_refs[p + i] = r[i];
  }
}

// Entry i of the list of moves: new_refs and map, or the list's padding.
__device__ __forceinline__ void move_refs(const PageArgs& a, int i, int moved, int32_t* map) {
  if (i >= moved) {
    a.src[i] = a.dst[i] = -1;
    return;
  }
  const int from = a.src[i], to = a.dst[i];
  a.new_refs[to] = a.refs[from];  // (no page is both a source and a destination)
  a.new_refs[from] = 0;
  map[from] = to;
}

__global__ __launch_bounds__(kPlanThreads) void compact_small_kernel(PageArgs a, int32_t* __restrict__ map) {
  __shared__ int s_waves[kPlanWaves];
  const int tid = threadIdx.x, n_chunks = (a.num_pages + kPerGo - 1) / kPerGo;
  int all = 0;
  for (int p = tid; p < a.num_pages; p += kPlanThreads) all += a.refs[p] > 0;
  Held h;
  h.before = 0;
  block_scan(all, s_waves, h.live);
  int below = 0;
  for (int p = tid; p < h.live; p += kPlanThreads) below += a.refs[p] > 0;
  block_scan(below, s_waves, h.below);
  for (int c = 0; c < n_chunks; ++c) {
    list_chunk(a, c, h, map, s_waves);
    int n = 0, total;
    for (int p = c * kPerGo + tid; p < min((c + 1) * kPerGo, a.num_pages); p += kPlanThreads) n += a.refs[p] > 0;
    block_scan(n, s_waves, total);
    h.before += total;
  }
  __syncthreads();
  const int moved = h.live - h.below;
  for (int i = tid; i < a.num_pages; i += kPlanThreads) move_refs(a, i, moved, map);
  if (tid == 0) {
    a.counts[0] = h.live;
    a.counts[1] = moved;
  }
  __syncthreads();
  for (int e = tid; e < a.requests * a.max_pages; e += kPlanThreads) {
    const Entry at = entry_at(a, e);
    move_entry(a, e, at.j < held_pages(a.lens[at.b], a.max_pages), map);
  }
}

__global__ __launch_bounds__(kPlanThreads) void compact_list_kernel(PageArgs a, int32_t* __restrict__ map,
                                                                    const int32_t* __restrict__ chunks) {
  __shared__ int s_waves[kPlanWaves];
  const Held h = add_up(a, chunks, gridDim.x, blockIdx.x, s_waves);
  list_chunk(a, blockIdx.x, h, map, s_waves);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.counts[0] = h.live;
    a.counts[1] = h.live - h.below;
  }
}

__global__ __launch_bounds__(256) void compact_refs_kernel(PageArgs a, int32_t* __restrict__ map) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < a.num_pages) move_refs(a, i, a.counts[1], map);
}

// The block table's held entries through the map.
__global__ __launch_bounds__(256) void compact_table_kernel(PageArgs a, const int32_t* __restrict__ map) {
  const int b = blockIdx.y;
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= a.max_pages) return;
  move_entry(a, static_cast<int64_t>(b) * a.max_pages + j, j < held_pages(a.lens[b], a.max_pages), map);
}

// A workgroup per (pair, cache): 16-byte pieces, eight loads in flight, then the
// four-byte rest of a part page.
__global__ __launch_bounds__(256) void copy_pages_kernel(CopyArgs a) {
  const int n = a.count ? max(0, min(a.n, a.count[0])) : a.n;
  const int64_t units = static_cast<int64_t>(n) * a.caches;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int i = static_cast<int>(u / a.caches), c = static_cast<int>(u - static_cast<int64_t>(i) * a.caches);
    const int src = a.src[i], dst = a.dst[i];
    const int tokens = a.tokens ? max(0, min(a.tokens[i], kPage)) : kPage;
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || src == dst) continue;
    const int row = a.token_bytes[c];
    const int64_t page_bytes = static_cast<int64_t>(row) * kPage;
    const char* from = static_cast<const char*>(a.base[c]) + src * page_bytes;
    char* to = static_cast<char*>(a.base[c]) + dst * page_bytes;
    const int pieces = row * tokens / 16;
    for (int p0 = threadIdx.x; p0 < pieces; p0 += 8 * 256) {
      i32x4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (p0 + k * 256 < pieces) x[k] = reinterpret_cast<const i32x4*>(from)[p0 + k * 256];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (p0 + k * 256 < pieces) reinterpret_cast<i32x4*>(to)[p0 + k * 256] = x[k];
    }
    const int rest = row * tokens / 4 - 4 * pieces;  // 0 .. 3 words
    if (static_cast<int>(threadIdx.x) < rest)
      reinterpret_cast<int*>(to)[4 * pieces + threadIdx.x] = reinterpret_cast<const int*>(from)[4 * pieces + threadIdx.x];
  }
}

constexpr int kCopyGrid = 2048;  // workgroups: eight per CU

// Small pools are one workgroup's, in one launch.  Calls with as many table entries as
// pages, release / fork / compact in us, one workgroup against several launches: 4096
// 7 / 9 / 9 and 10 / 17 / 16; 8192 9 / 13 / 14 and 10 / 17 / 16; 16384 16 / 24 / 26 and
// 10 / 17 / 16 (a million pages: 10 / 17 / 19).
constexpr int kSmallPages = 8192, kSmallEntries = 8192;
bool small_pool(const PageArgs& a) {
  return a.num_pages <= kSmallPages && static_cast<int64_t>(a.requests) * a.max_pages <= kSmallEntries;
}

}  // namespace

// fork: two ints per request; compact: an int per page; both: one per chunk.
size_t ints_bytes(int64_t n) { return (static_cast<size_t>(n) * sizeof(int32_t) + 255) / 256 * 256; }
int chunk_count(int32_t num_pages) { return (num_pages + kPerGo - 1) / kPerGo; }

size_t pages_workspace_size(int32_t requests, int32_t num_pages) {
  if (requests <= 0 || num_pages <= 0) return 0;
  return ints_bytes(requests > num_pages ? requests : num_pages) + ints_bytes(requests) +
         ints_bytes(chunk_count(num_pages));
}

struct PageWorkspace {
  int32_t* first;   // per page or request
  int32_t* second;  // per request
  int32_t* chunks;
};
static PageWorkspace page_workspace(const PageArgs& a) {
  char* p = static_cast<char*>(a.workspace);
  const size_t first = ints_bytes(a.requests > a.num_pages ? a.requests : a.num_pages), second = ints_bytes(a.requests);
  return {reinterpret_cast<int32_t*>(p), reinterpret_cast<int32_t*>(p + first),
          reinterpret_cast<int32_t*>(p + first + second)};
}

hipError_t launch_release_pages(const PageArgs& a, hipStream_t stream, LaunchEvents ev) {
  if (small_pool(a)) {
    launch_kernel(release_small_kernel, dim3(1), dim3(kPlanThreads), stream, ev.start, ev.stop, a);
    return hipGetLastError();
  }
  const bool copies = a.new_refs != a.refs;
  if (copies) {
    const int blocks = (a.num_pages + 255) / 256;
    launch_kernel(copy_refs_kernel, dim3(blocks < 1024 ? blocks : 1024), dim3(256), stream, ev.start, nullptr, a.refs,
                  a.num_pages, a.new_refs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  launch_kernel(release_kernel, dim3(a.requests), dim3(256), stream, copies ? nullptr : ev.start, ev.stop, a);
  return hipGetLastError();
}

hipError_t launch_fork_pages(const PageArgs& a, hipStream_t stream, LaunchEvents ev) {
  const PageWorkspace ws = page_workspace(a);
  const dim3 threads(kPlanThreads);
  if (small_pool(a)) {
    launch_kernel(fork_plan_kernel<true>, dim3(1), threads, stream, ev.start, ev.stop, a, nullptr, nullptr, nullptr);
    return hipGetLastError();
  }
  const dim3 grid(chunk_count(a.num_pages));
  launch_kernel(count_held_kernel, grid, threads, stream, ev.start, nullptr, a, ws.chunks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_kernel(free_list_kernel, grid, threads, stream, nullptr, nullptr, a, ws.chunks, ws.second);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_kernel(fork_plan_kernel<false>, dim3(1), threads, stream, nullptr, nullptr, a, ws.first, ws.second, ws.chunks);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_kernel(fork_rows_kernel, dim3(a.requests), dim3(256), stream, nullptr, ev.stop, a, ws.first);
  return hipGetLastError();
}

hipError_t launch_compact_pages(const PageArgs& a, hipStream_t stream, LaunchEvents ev) {
  const PageWorkspace ws = page_workspace(a);
  int32_t *map = ws.first, *chunks = ws.chunks;
  if (small_pool(a)) {
    launch_kernel(compact_small_kernel, dim3(1), dim3(kPlanThreads), stream, ev.start, ev.stop, a, map);
    return hipGetLastError();
  }
  const dim3 grid(chunk_count(a.num_pages));
  launch_kernel(count_held_kernel, grid, dim3(kPlanThreads), stream, ev.start, nullptr, a, chunks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_kernel(compact_list_kernel, grid, dim3(kPlanThreads), stream, nullptr, nullptr, a, map, chunks);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_kernel(compact_refs_kernel, dim3((a.num_pages + 255) / 256), dim3(256), stream, nullptr, nullptr, a, map);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_kernel(compact_table_kernel, dim3((a.max_pages + 255) / 256, a.requests), dim3(256), stream, nullptr, ev.stop,
                a, map);
  return hipGetLastError();
}

hipError_t launch_copy_pages(const CopyArgs& a, hipStream_t stream, hipEvent_t start, hipEvent_t stop) {
  const int64_t units = static_cast<int64_t>(a.n) * a.caches;
  launch_kernel(copy_pages_kernel, dim3(static_cast<uint32_t>(units < kCopyGrid ? units : kCopyGrid)), dim3(256), stream,
                start, stop, a);
  return hipGetLastError();
}

}  // namespace pmqa
