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
// The results are whole numbers and do not depend on timing: refs change by atomic
// additions alone, and every list is ordered by a scan.
#include "indexer_common.h"
#include "launches.h"

namespace pmqa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kPerThread = 4;                           // pages (or requests) of a thread in one go
constexpr int kPerGo = kPlanThreads * kPerThread;       // 4096: also the most requests

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
  for (int j = threadIdx.x; j < n; j += 256) {
    const int page = row[j];
    if (page >= 0 && page < a.num_pages) atomicSub(a.new_refs + page, 1);
  }
}

// One workgroup.  Which requests are forked, and the page that each takes; then
// refs to new_refs up to the pages that are shared, which fork_rows_kernel adds.
// inherit[b]: full pages that b takes over, -1 for a request that is not forked.
__global__ __launch_bounds__(kPlanThreads) void fork_plan_kernel(PageArgs a, int32_t* __restrict__ inherit) {
  __shared__ int s_waves[kPlanWaves];
  __shared__ int s_free[kPerGo];  // pages for the requests that need one, in their order
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
      dst = s_free[base + rank[i]];
      a.block_table[static_cast<int64_t>(b) * a.max_pages + full] = dst;
      a.new_refs[dst] = 1;
    }
    a.src[b] = src;
    a.dst[b] = dst;
    a.tokens[b] = takes ? rest : 0;
    a.new_lens[b] = forked ? from[i] : len[i];
    inherit[b] = forked ? full : -1;
  }
  if (tid == 0) {
    a.counts[0] = found;
    a.counts[1] = wanted - found;
  }
}

// One workgroup per request: the full pages that it shares with its parent.
__global__ __launch_bounds__(256) void fork_rows_kernel(PageArgs a, const int32_t* __restrict__ inherit) {
  const int b = blockIdx.x;
  const int n = inherit[b];
  if (n <= 0) return;
  const int32_t* from = a.block_table + static_cast<int64_t>(a.mask[b]) * a.max_pages;
  int32_t* row = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  for (int j = threadIdx.x; j < n; j += 256) {
    const int page = from[j];
    row[j] = page;
    if (page >= 0 && page < a.num_pages) atomicAdd(a.new_refs + page, 1);
  }
}

// One workgroup: the moves, new_refs, and where each page goes (map).
__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(PageArgs a, int32_t* __restrict__ map) {
  __shared__ int s_waves[kPlanWaves];
  const int tid = threadIdx.x;
  int held = 0;
  for (int p = tid; p < a.num_pages; p += kPlanThreads) held += a.refs[p] > 0;
  int live;
  block_scan(held, s_waves, live);
  int moved = 0, holes = 0;  // held pages from `live` on, free ones below it: as many of each in the end
  for (int p0 = 0; p0 < a.num_pages; p0 += kPerGo) {
    const int p = p0 + tid * kPerThread;
    int r[kPerThread], n = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const bool in = p + i < a.num_pages;
      r[i] = in ? a.refs[p + i] : 0;
      // two counts of at most 4096 in one scan
      if (in && p + i >= live && r[i] > 0) n += 1 << 16;
      if (in && p + i < live && r[i] <= 0) n += 1;
    }
    int total;
    const int before = block_scan(n, s_waves, total);
    int to_src = moved + (before >> 16), to_dst = holes + (before & 0xFFFF);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (p + i >= a.num_pages) continue;
      if (p + i >= live && r[i] > 0) a.src[to_src++] = p + i;
      if (p + i < live && r[i] <= 0) a.dst[to_dst++] = p + i;
      map[p + i] = p + i;
      if (a.new_refs != a.refs) a.new_refs[p + i] = r[i];
    }
    moved += total >> 16;
    holes += total & 0xFFFF;
  }
  __syncthreads();
  for (int i = tid; i < a.num_pages; i += kPlanThreads) {
    if (i >= moved) {
      a.src[i] = a.dst[i] = -1;
      continue;
    }
    const int from = a.src[i], to = a.dst[i];
    a.new_refs[to] = a.refs[from];  // (no page is both a source and a destination)
    a.new_refs[from] = 0;
    map[from] = to;
  }
  if (tid == 0) {
    a.counts[0] = live;
    a.counts[1] = moved;
  }
}

// The block table's held entries through the map.
__global__ __launch_bounds__(256) void compact_table_kernel(PageArgs a, const int32_t* __restrict__ map) {
  const int b = blockIdx.y;
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= a.max_pages) return;
  const int64_t at = static_cast<int64_t>(b) * a.max_pages + j;
  const int page = a.block_table[at];
  const bool held = j < held_pages(a.lens[b], a.max_pages) && page >= 0 && page < a.num_pages;
  a.new_table[at] = held ? map[page] : page;
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

}  // namespace

// fork: an int per request; compact: an int per page.
size_t pages_workspace_size(int32_t requests, int32_t num_pages) {
  if (requests <= 0 || num_pages <= 0) return 0;
  return (static_cast<size_t>(requests > num_pages ? requests : num_pages) * sizeof(int32_t) + 255) / 256 * 256;
}

hipError_t launch_release_pages(const PageArgs& a, hipStream_t stream, LaunchEvents ev) {
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
  int32_t* inherit = static_cast<int32_t*>(a.workspace);
  launch_kernel(fork_plan_kernel, dim3(1), dim3(kPlanThreads), stream, ev.start, nullptr, a, inherit);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  launch_kernel(fork_rows_kernel, dim3(a.requests), dim3(256), stream, nullptr, ev.stop, a, inherit);
  return hipGetLastError();
}

hipError_t launch_compact_pages(const PageArgs& a, hipStream_t stream, LaunchEvents ev) {
  int32_t* map = static_cast<int32_t*>(a.workspace);
  launch_kernel(compact_plan_kernel, dim3(1), dim3(kPlanThreads), stream, ev.start, nullptr, a, map);
  const hipError_t e = hipGetLastError();
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
