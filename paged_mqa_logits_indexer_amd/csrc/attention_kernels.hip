// Attention over the paged latent cache (gfx950): over a request's pages, over
// pages that a batch shares, and over the keys that the top-k selected.
//
// All heads of a row read the same cache row per key (576 values: 512 latent,
// which are also the value vector, and 64 rotated), so a tile of M (row, head)
// pairs against 64 keys is one matrix product S = K Q^T, an online softmax
// per pair, and a second product O^T += V^T P^T on the same keys.
//
//   z_s = scale q . k_s,  c tanh(z / c),  - slope_h |pos_r - s|
//   m = max z, p_s = exp(z_s - m), l = sum p_s, o = sum p_s k_s[0:512]
//   out = o / l, lse = m + log l;  a row without keys: 0 and -inf
//
// Both products run transposed, keys on the MFMA's rows and pairs on its
// columns: a lane then holds four consecutive keys of ONE pair, which is at
// once the layout the second product takes P in (no exchange through LDS) and
// one in which the softmax of a pair needs two lane exchanges.  The value
// operand V^T comes from the same LDS tile with the transposing 64-bit reads.
//
// Work: the (pair tile, 64-key tile) list of the whole batch is cut into equal
// contiguous shares, one per persistent workgroup (one per CU), whatever the
// requests' lengths.  A share that covers all keys of a pair tile writes its
// output; the pieces of a pair tile that several workgroups share go to the
// workspace as (o, m, l) in float32 and a second kernel joins them, in a fixed
// order.
#include <algorithm>
#include <climits>

#include "indexer_common.h"
#include "launches.h"

namespace pmqa {
namespace {

constexpr int kRowDim = IDX_LATENT_ROW;            // 576
constexpr int kValDim = IDX_LATENT_DIM;            // 512
constexpr int kRowBytes = kRowDim * 2;             // 1152
constexpr int kKSteps = kRowDim / 32;              // 18 MFMA steps of S
constexpr int kDimTiles = kValDim / 16;            // 32 output tiles of 16 dimensions
constexpr int kTile = 64;                          // keys per iteration of a workgroup
constexpr int kBlkBytes = 16 * kRowBytes;          // 16 keys in LDS: 18432
constexpr int kSlotBytes = kTile * kRowBytes;      // 73728
constexpr int kSlots = 2;
constexpr int kAttnThreads = 256;
constexpr int kChunkDims = 128;                    // epilogue: dimensions exchanged at a time
constexpr int kChunkStride = kChunkDims + 4;       // floats; the pad spreads the pairs over all banks
constexpr int kScanChunks = 1056;                  // work-list chunks of 256 pair tiles
constexpr float kMInit = -1.7e38f;                 // running maximum before any key (finite: no inf - inf)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum is raised only when a score passes it by more than this
// (powers of two): P then holds values up to 2^6, exact in the final quotient,
// and the 128 accumulators are rescaled a few times per row instead of at
// every new maximum.
constexpr float kRaise = 6.0f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// P is rounded to the cache's 16-bit type for the second product (an MFMA
// takes both operands in one type): a relative error of at most half a step
// per key, independent over the keys, so it stays below the rounding of the
// output itself; l sums the unrounded values.  FP16 has few exponents, so its
// P is scaled by 2^8 (kShift): keys 2^-22 below the maximum are still normal.
template <int DT>
struct Elem;
template <>
struct Elem<IDX_BF16> {
  static constexpr float kShift = 0.0f;
  static __device__ __forceinline__ f32x4 mfma32(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  static __device__ __forceinline__ f32x4 mfma16(s16x4 a, s16x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ short round(float x) {
    return __builtin_bit_cast(short, static_cast<__bf16>(x));
  }
};
template <>
struct Elem<IDX_FP16> {
  static constexpr float kShift = 8.0f;
  static __device__ __forceinline__ f32x4 mfma32(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  static __device__ __forceinline__ f32x4 mfma16(s16x4 a, s16x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a), __builtin_bit_cast(f16x4, b), c, 0, 0,
                                                 0);
  }
  static __device__ __forceinline__ short round(float x) {
    return __builtin_bit_cast(short, static_cast<_Float16>(x));
  }
};

// Where invalid keys are read from: a row of zeros, so that neither S nor the
// value product meets what the cache holds there.
__device__ __attribute__((aligned(128))) const uint32_t kZeroRow[kRowBytes / 4] = {};

// LDS image of 16 keys (18 KiB): nine 1 KiB pieces per 8 keys, a piece holding
// 128 bytes of each of them -- what one direct-to-LDS load of 64 x 16 bytes
// writes.  Within its 128 bytes a key's 16-byte chunks are exchanged by
// c ^ swz(key), which spreads both kinds of reads over all banks: the K
// operand (16 keys, one chunk) and the transposed V operand (8 keys of one
// parity class, two neighbouring chunks).
__device__ __forceinline__ int swz(int key) { return (((key >> 1) & 3) << 1) | ((key >> 3) & 1); }
__device__ __forceinline__ int key_offset(int key) { return (key >> 3) * (kBlkBytes / 2) + (key & 7) * 128; }

// Issues this wave's 16 keys of a tile into LDS: lane l reads 16-byte pieces of
// keys l / 8 and 8 + l / 8 from the addresses a0 and a1.  The instruction's
// offset advances both the source and the LDS address by 128; M0 supplies the
// rest of the 1 KiB step.  Written in assembly so that the compiler does not
// drain the loads in flight before every LDS access of the other slot; the
// caller waits (vmcnt) before the barrier that publishes the tile.
__device__ __forceinline__ void load_keys(const char* a0, const char* a1, uint32_t lds) {
  constexpr uint32_t kStep = 1024 - 128;
#define PMQA_LOAD(v, j, at)                      \
  "s_add_u32 m0, %[l], " at "\n"                 \
  "s_nop 0\n"                                    \
  "global_load_lds_dwordx4 %[" v "], off offset:" j "\n"
  static_assert(kStep == 896, "offsets below are multiples of 896");
  __asm__ volatile(
      PMQA_LOAD("a", "0", "0") PMQA_LOAD("a", "128", "896") PMQA_LOAD("a", "256", "1792")
      PMQA_LOAD("a", "384", "2688") PMQA_LOAD("a", "512", "3584") PMQA_LOAD("a", "640", "4480")
      PMQA_LOAD("a", "768", "5376") PMQA_LOAD("a", "896", "6272") PMQA_LOAD("a", "1024", "7168")
      PMQA_LOAD("b", "0", "9216") PMQA_LOAD("b", "128", "10112") PMQA_LOAD("b", "256", "11008")
      PMQA_LOAD("b", "384", "11904") PMQA_LOAD("b", "512", "12800") PMQA_LOAD("b", "640", "13696")
      PMQA_LOAD("b", "768", "14592") PMQA_LOAD("b", "896", "15488") PMQA_LOAD("b", "1024", "16384")
      :
      : [l] "s"(lds), [a] "v"(a0), [b] "v"(a1)
      : "memory", "m0", "scc");
#undef PMQA_LOAD
}

__device__ __forceinline__ void wait_all_and_barrier() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0); the compiler counts its own loads as done, too
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

typedef __attribute__((address_space(3))) const s16x8* LdsVec8;
typedef __attribute__((address_space(3))) s16x4* LdsVec4;
__device__ __forceinline__ s16x8 lds_read(uint32_t at) { return *reinterpret_cast<LdsVec8>(at); }
__device__ __forceinline__ s16x4 lds_read_tr(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<LdsVec4>(at));
}

// Maximum of a value over the four lanes (l, l ^ 16, l ^ 32, l ^ 48) of a pair.
__device__ __forceinline__ float pair_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// tanh(x) = 1 - 2 / (1 + e^2x): absolute error of about one float32 step of 1,
// which the cap's factor turns into that of the score; near zero, where the
// difference would lose the argument's digits, the odd series
// x - x^3/3 + 2 x^5/15 - 17 x^7/315 (the next term is below 2^-24 relative for
// |x| < 0.1).
__device__ __forceinline__ float tanh_f32(float x) {
  const float e = __builtin_amdgcn_exp2f(x * (2.0f * kLog2e));
  const float far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e);
  const float y = x * x;
  const float near = x * (1.0f + y * (-1.0f / 3.0f + y * (2.0f / 15.0f - y * (17.0f / 315.0f))));
  return fabsf(x) < 0.1f ? near : far;
}

// One pair tile of the work list: its pairs and the 64-key tiles it reads.
struct Item {
  int request;   // block-table row
  int row0;      // the first row of the request (pair p is row row0 + p / heads)
  int pair0;     // first pair, counted from row0 * heads
  int pairs;     // 1 .. M (0: no such item)
  int tile0;     // first 64-key tile
  int tiles;     // number of tiles (at least 1 when pairs > 0)
  int max_start; // largest first key and smallest end over the rows: tiles inside need no mask
  int min_end;
  int min_start; // keys that some row may see: [min_start, max_end)
  int max_end;
  int key_lo;    // keys of this item: [key_lo, key_hi) (shared: prefix and rest)
  int key_hi;
};

// KIND: what the key tiles are.
enum { kDense = 0, kShared = 1, kSparse = 2 };

__device__ __forceinline__ int clamp_len(int len, int capacity) { return max(0, min(len, capacity)); }

// Rows of request b as [r0, r1), clamped into the batch.
__device__ __forceinline__ void request_rows(const AttentionArgs& a, int b, int& r0, int& r1) {
  if (a.cu_q) {
    r0 = max(0, min(a.cu_q[b], a.rows));
    r1 = max(r0, min(a.cu_q[b + 1], a.rows));
  } else {
    r0 = b * a.next_n;
    r1 = r0 + a.next_n;
  }
}

// First item id of request b of a ragged batch: one id per M pairs of the
// rows before it plus one per request, so every request has enough ids
// (floor((x + n) / M) + 1 - floor(x / M) >= ceil(n / M)) and an id finds its
// request by bisection, without a scan.
template <int M>
__device__ __forceinline__ int ragged_base(const AttentionArgs& a, int b) {
  const int r = max(0, min(a.cu_q[b], a.rows));
  return static_cast<int>(static_cast<int64_t>(r) * a.heads / M) + b;
}

// Key range of rows [r0, r1): every lane of the caller computes it (BY = 1) or
// the lanes of a wave share the rows (BY = 64).
template <int BY>
__device__ __forceinline__ void key_range(const AttentionArgs& a, int r0, int r1, int capacity, Item& it) {
  int lo = INT_MAX, hi = 0, max_start = 0, min_end = INT_MAX;
  for (int r = r0 + (BY > 1 ? lane_id() : 0); r < r1; r += BY) {
    const int end = clamp_len(a.row_lens[r], capacity);
    const int start = a.row_starts ? max(0, a.row_starts[r]) : 0;
    max_start = max(max_start, start);
    min_end = min(min_end, end);
    if (start < end) {
      lo = min(lo, start);
      hi = max(hi, end);
    }
  }
  if constexpr (BY > 1) {
    lo = -wave_max(-lo);
    hi = wave_max(hi);
    max_start = wave_max(max_start);
    min_end = -wave_max(-min_end);
  }
  if (lo > hi) lo = hi;  // no row sees a key
  it.max_start = max(max_start, it.key_lo);
  it.min_end = min(min_end, it.key_hi);
  it.min_start = max(lo, it.key_lo);
  it.max_end = min(hi, it.key_hi);
  it.tile0 = lo / kTile;
  it.tiles = (hi + kTile - 1) / kTile - it.tile0;
}

// Item `id` of the list.  Dense: requests' pair tiles.  Shared: first the pair
// tiles of the whole batch over the prefix pages, then the requests' pair
// tiles over what follows.  Sparse: rows' pair tiles over the selection.
template <int KIND, int M, int BY>
__device__ __forceinline__ Item make_item(const AttentionArgs& a, int id) {
  const int capacity = a.max_pages * kPage;
  Item it{};
  it.key_hi = capacity;
  if constexpr (KIND == kSparse) {
    const int per_row = (a.heads + M - 1) / M;
    const int row = id / per_row, t = id - row * per_row;
    it.row0 = row;
    it.pair0 = t * M;
    it.pairs = min(M, a.heads - it.pair0);
    it.tiles = (a.k + kTile - 1) / kTile;
    if (a.cu_q) {
      // the last request that starts at or before the row
      int lo = 0, hi = a.requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.cu_q[mid] <= row) lo = mid; else hi = mid;
      }
      it.request = lo;
      if (row < a.cu_q[lo] || row >= a.cu_q[lo + 1]) it.pairs = it.tiles = 0;
    } else {
      it.request = row / a.next_n;
    }
    return it;
  } else {
    int prefix_items = 0;
    if constexpr (KIND == kShared) {
      const int64_t all = static_cast<int64_t>(a.rows) * a.heads;
      prefix_items = static_cast<int>((all + M - 1) / M);
      if (id < prefix_items) {
        const int64_t p0 = static_cast<int64_t>(id) * M;
        const int n = static_cast<int>(min(static_cast<int64_t>(M), all - p0));
        it.row0 = static_cast<int>(p0 / a.heads);
        it.key_hi = a.prefix_pages * kPage;
        it.pair0 = static_cast<int>(p0 - static_cast<int64_t>(it.row0) * a.heads);
        it.pairs = n;
        key_range<BY>(a, it.row0, it.row0 + (it.pair0 + n - 1) / a.heads + 1, capacity, it);
        const int end = min(it.tile0 + it.tiles, a.prefix_pages);
        it.tile0 = min(it.tile0, a.prefix_pages - 1);
        it.tiles = max(1, end - it.tile0);
        return it;
      }
      id -= prefix_items;
    }
    int b, t;
    if (a.cu_q) {
      int lo = 0, hi = a.requests;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (ragged_base<M>(a, mid) <= id) lo = mid; else hi = mid;
      }
      b = lo;
      t = id - ragged_base<M>(a, b);
    } else {
      const int per = (a.next_n * a.heads + M - 1) / M;
      b = id / per;
      t = id - b * per;
    }
    int r0, r1;
    request_rows(a, b, r0, r1);
    it.request = b;
    it.row0 = r0;
    it.pair0 = t * M;
    it.pairs = static_cast<int>(min(static_cast<int64_t>(M), static_cast<int64_t>(r1 - r0) * a.heads - static_cast<int64_t>(t) * M));
    if (t < 0 || it.pairs <= 0) {
      it.pairs = 0;
      return it;
    }
    if constexpr (KIND == kShared) it.key_lo = a.prefix_pages * kPage;
    key_range<BY>(a, r0 + it.pair0 / a.heads, r0 + (it.pair0 + it.pairs - 1) / a.heads + 1, capacity, it);
    if constexpr (KIND == kShared) {
      const int end = it.tile0 + it.tiles;
      it.tile0 = max(it.tile0, min(a.prefix_pages, a.max_pages - 1));
      it.tiles = end - it.tile0;
    }
    it.tiles = max(1, it.tiles);
    it.tile0 = min(it.tile0, a.max_pages - 1);
    return it;
  }
}

template <int KIND, int M>
__host__ __device__ __forceinline__ int64_t item_count(const AttentionArgs& a) {
  const int64_t pairs = static_cast<int64_t>(a.rows) * a.heads;
  if (KIND == kSparse) return static_cast<int64_t>(a.rows) * ((a.heads + M - 1) / M);
  const int64_t own = a.cu_q ? pairs / M + a.requests
                             : static_cast<int64_t>(a.requests) * ((static_cast<int64_t>(a.next_n) * a.heads + M - 1) / M);
  return KIND == kShared ? (pairs + M - 1) / M + own : own;
}

// The workgroup's share [t0, t1) of the tile list and the item it starts in.
struct Share {
  int64_t t0, t1;      // tiles
  int64_t total;
  int64_t item_at;     // tile offset of `item`
  int item;
  int groups;          // workgroups with work
};

// Share of workgroup w: as many groups as give each kMinTiles tiles.
__device__ __forceinline__ int64_t share_begin(int64_t total, int groups, int w) {
  return total * w / groups;
}
// The workgroup whose share holds tile t.
__device__ __forceinline__ int share_owner(int64_t total, int groups, int64_t t) {
  int w = static_cast<int>((t * groups + groups - 1) / total);
  while (w > 0 && share_begin(total, groups, w) > t) --w;
  while (w + 1 < groups && share_begin(total, groups, w + 1) <= t) ++w;
  return w;
}

template <int KIND, int M>
__device__ Share find_share(const AttentionArgs& a, int w, int grid, int min_tiles, int* s_scan, int64_t* s_res) {
  Share s;
  const int items = static_cast<int>(item_count<KIND, M>(a));
  const int tid = threadIdx.x;
  if constexpr (KIND == kSparse) {
    if (!a.cu_q) {
      const int n = (a.k + kTile - 1) / kTile;
      s.total = static_cast<int64_t>(items) * n;
      s.groups = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), s.total / min_tiles)));
      s.t0 = w < s.groups ? share_begin(s.total, s.groups, w) : 0;
      s.t1 = w < s.groups ? share_begin(s.total, s.groups, w + 1) : 0;
      s.item = static_cast<int>(s.t0 / n);
      s.item_at = static_cast<int64_t>(s.item) * n;
      return s;
    }
  }
  // Tiles per chunk of 256 items, then their sum, then the chunk that holds t0
  // is walked again.  s_scan: a counter per wave, then the chunk sums.
  const int chunks = (items + kAttnThreads - 1) / kAttnThreads;
  int* s_wave = s_scan;
  int* s_chunk = s_scan + kAttnThreads / kWave;
  for (int c = 0; c < chunks; ++c) {
    const int id = c * kAttnThreads + tid;
    const int n = id < items ? make_item<KIND, M, 1>(a, id).tiles : 0;
    const int sum = wave_sum(n);
    if (lane_id() == 0) s_wave[tid / kWave] = sum;
    __syncthreads();
    if (tid == 0) s_chunk[c] = s_wave[0] + s_wave[1] + s_wave[2] + s_wave[3];
    __syncthreads();
  }
  int64_t total = 0;
  for (int c = 0; c < chunks; ++c) total += s_chunk[c];
  s.total = total;
  s.groups = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(grid), total / min_tiles)));
  if (w >= s.groups || total == 0) {
    s.t0 = s.t1 = 0;
    s.item = 0;
    s.item_at = 0;
    return s;
  }
  s.t0 = share_begin(total, s.groups, w);
  s.t1 = share_begin(total, s.groups, w + 1);
  int64_t at = 0;
  int c = 0;
  while (c + 1 < chunks && at + s_chunk[c] <= s.t0) at += s_chunk[c++];
  const int id = c * kAttnThreads + tid;
  const int n = id < items ? make_item<KIND, M, 1>(a, id).tiles : 0;
  const int upto = wave_inclusive_scan(n);
  if (lane_id() == kWave - 1) s_wave[tid / kWave] = upto;
  __syncthreads();
  int64_t before = at + upto - n;
  for (int i = 0; i < tid / kWave; ++i) before += s_wave[i];
  if (n > 0 && before <= s.t0 && s.t0 < before + n) {
    s_res[0] = id;
    s_res[1] = before;
  }
  __syncthreads();
  s.item = static_cast<int>(s_res[0]);
  s.item_at = s_res[1];
  return s;
}

// What the join kernel needs to know of a pair tile that several workgroups
// share: written by the workgroup that holds the tile's beginning.
struct alignas(16) JoinInfo {
  int first;      // first piece of the list (see piece_id)
  int pieces;     // 0: nothing to join here
  int pairs;
  int pad;
  int64_t pair0;  // first pair, counted over the whole batch
  int64_t pad2;
};

// Pieces in the workspace: float o[M][512], then float2 (m, l)[M].  Dense and
// sparse: two per workgroup, for a pair tile that began before it (2 w) and one
// that ends after it (2 w + 1).  Shared: every (workgroup, item) visit is a
// piece, w + item -- consecutive over a pair tile's workgroups.
__host__ __device__ __forceinline__ int64_t piece_floats(int m) { return static_cast<int64_t>(m) * (kValDim + 2); }

template <int DT, int KIND, int PT, int PG>
__global__ __launch_bounds__(kAttnThreads, 1) void attention_kernel(AttentionArgs a, int min_tiles, JoinInfo* join,
                                                                    float* pieces) {
  using E = Elem<DT>;
  constexpr int kWavePairs = 16 * PT;           // pairs of a wave
  constexpr int M = kWavePairs * PG;            // pairs of the workgroup
  constexpr int TS = 4 / PG;                    // key streams: waves that take different keys of the same pairs
  constexpr int ST = 4 / TS;                    // 16-key blocks of a tile per wave
  __shared__ __attribute__((aligned(1024))) char s_keys[kSlots * kSlotBytes];
  __shared__ int s_tok[kSlots][kTile];          // sparse: logical key of every tile row, -1 for none
  __shared__ float2 s_ml[4][kWavePairs];
  __shared__ int64_t s_res[2];
  __shared__ int s_scan[kAttnThreads / kWave + kScanChunks];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grid = gridDim.x;
  // consecutive shares on one XCD (workgroups are dealt to the 8 XCDs in turn)
  const int w = (grid & 7) ? static_cast<int>(blockIdx.x)
                           : static_cast<int>(blockIdx.x & 7) * (grid >> 3) + static_cast<int>(blockIdx.x >> 3);
  const Share share = find_share<KIND, M>(a, w, grid, min_tiles, s_scan, s_res);
  if (KIND != kShared && tid == 0) join[w].pieces = 0;
  if (share.t0 >= share.t1) return;

  const uint32_t keys_lds = static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)s_keys));
  const int pg = wave / TS, ts = wave % TS;
  const int n16 = lane & 15, g4 = lane >> 4;
  // this lane's places in a 16-key block: K operand (key n16, chunk g4), and
  // the transposed V operand (key 4 g4 + n16 / 4, 4 dimensions n16 % 4)
  const uint32_t k_at = key_offset(n16) + ((g4 ^ swz(n16)) * 16);
  const int vkey = 4 * g4 + (n16 >> 2);
  const uint32_t v_at = key_offset(vkey) + ((((n16 >> 1) & 1) ^ swz(vkey)) * 16) + (n16 & 1) * 8;
  const int src0 = ((lane & 7) ^ swz(lane >> 3)) * 16;        // source chunk of the keys lane / 8 ...
  const int src1 = ((lane & 7) ^ swz(8 + (lane >> 3))) * 16;  // ... and 8 + lane / 8
  const int capacity = a.max_pages * kPage;
  const char* cache = static_cast<const char*>(a.cache);
  const float to_log2 = a.scale * kLog2e;

  int64_t at = share.t0;
  int64_t item_at = share.item_at;
  int item = share.item;
  const int items = static_cast<int>(item_count<KIND, M>(a));
  while (at < share.t1 && item < items) {
    const Item it = make_item<KIND, M, kWave>(a, item);
    if (it.tiles == 0 || item_at + it.tiles <= at) {  // no pairs: nothing to do or to write
      item_at += it.tiles;
      ++item;
      continue;
    }
    const int lo = static_cast<int>(at - item_at);
    const int hi = static_cast<int>(min(static_cast<int64_t>(it.tiles), share.t1 - item_at));
    const bool whole = lo == 0 && hi == it.tiles && KIND != kShared;
    const int32_t* table = a.block_table + static_cast<int64_t>(it.request) * a.max_pages;

    // the pairs of this lane: queries in the B operand's layout
    s16x8 q[PT][kKSteps];
    int p_start[PT], p_end[PT], p_pos[PT];
    float p_slope[PT];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) {
      const int local = min(pg * kWavePairs + pt * 16 + n16, it.pairs - 1);
      const int pair = it.pair0 + local;
      const int row = it.row0 + pair / a.heads;
      const char* qp = static_cast<const char*>(a.q) +
                       (static_cast<int64_t>(it.row0) * a.heads + pair) * kRowBytes + g4 * 16;
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks) q[pt][ks] = *reinterpret_cast<const s16x8*>(qp + ks * 64);
      p_start[pt] = 0;
      p_end[pt] = capacity;
      if constexpr (KIND != kSparse) {
        p_end[pt] = clamp_len(a.row_lens[row], capacity);
        if (a.row_starts) p_start[pt] = max(0, a.row_starts[row]);
      }
      p_slope[pt] = a.slopes ? a.slopes[pair % a.heads] * kLog2e : 0.0f;
      p_pos[pt] = a.row_positions ? a.row_positions[row] : p_end[pt] - 1;
      p_start[pt] = max(p_start[pt], it.key_lo);
      p_end[pt] = min(p_end[pt], it.key_hi);
    }

    // ---- loading: this wave's 16 keys of tile `t` (counted from the item's first)
    int page_window = -1, window_page = 0;  // dense: page ids of 64 tiles, one per lane
    int next_tok0 = -1, next_tok1 = -1;     // sparse: keys of the tile to be issued next ...
    int next_page0 = 0, next_page1 = 0;     // ... and their pages
    int after_tok0 = -1, after_tok1 = -1;   // keys of the tile after it
    auto fetch_tokens = [&](int t, int& tok0, int& tok1) {
      const int c0 = t * kTile + wave * 16 + (lane >> 3);
      const int32_t* list = a.indices + static_cast<int64_t>(it.row0) * a.k;
      tok0 = c0 < a.k ? list[c0] : -1;
      tok1 = c0 + 8 < a.k ? list[c0 + 8] : -1;
      if (tok0 >= capacity) tok0 = -1;
      if (tok1 >= capacity) tok1 = -1;
    };
    auto fetch_pages = [&](int tok0, int tok1, int& page0, int& page1) {
      page0 = table[max(tok0, 0) / kPage];
      page1 = table[max(tok1, 0) / kPage];
    };
    auto issue = [&](int t, int slot) {
      int slot0, slot1;      // cache rows
      bool live0, live1;
      if constexpr (KIND == kSparse) {
        live0 = next_tok0 >= 0;
        live1 = next_tok1 >= 0;
        slot0 = max(0, min(next_page0, a.num_pages - 1)) * kPage + (max(next_tok0, 0) & (kPage - 1));
        slot1 = max(0, min(next_page1, a.num_pages - 1)) * kPage + (max(next_tok1, 0) & (kPage - 1));
        if ((lane & 7) == 0) {
          s_tok[slot][wave * 16 + (lane >> 3)] = live0 ? next_tok0 : -1;
          s_tok[slot][wave * 16 + 8 + (lane >> 3)] = live1 ? next_tok1 : -1;
        }
      } else {
        const int tile = it.tile0 + t;
        if ((tile >> 6) != page_window) {
          page_window = tile >> 6;
          window_page = table[min(page_window * 64 + lane, a.max_pages - 1)];
        }
        const int page = max(0, min(__builtin_amdgcn_readlane(window_page, tile & 63), a.num_pages - 1));
        const int key = wave * 16 + (lane >> 3);
        slot0 = page * kPage + key;
        slot1 = slot0 + 8;
        // keys that no row of the pair tile sees are not read
        live0 = tile * kTile + key >= it.min_start && tile * kTile + key < it.max_end;
        live1 = tile * kTile + key + 8 >= it.min_start && tile * kTile + key + 8 < it.max_end;
      }
      const char* zero = reinterpret_cast<const char*>(kZeroRow);
      const char* a0 = (live0 ? cache + static_cast<int64_t>(slot0) * kRowBytes : zero) + src0;
      const char* a1 = (live1 ? cache + static_cast<int64_t>(slot1) * kRowBytes : zero) + src1;
      if constexpr (KIND == kSparse) {
        // two dependent loads run ahead of each tile: its key ids two issues
        // early, their pages one issue early, so that neither is waited for
        // (and none is waited for with this tile's loads in flight)
        next_tok0 = after_tok0;
        next_tok1 = after_tok1;
        fetch_pages(next_tok0, next_tok1, next_page0, next_page1);
        fetch_tokens(t + 2, after_tok0, after_tok1);
      }
      load_keys(a0, a1, keys_lds + slot * kSlotBytes + wave * kBlkBytes);
    };

    f32x4 acc[PT][kDimTiles];
    float m[PT], l[PT];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) {
      m[pt] = kMInit;
      l[pt] = 0.0f;
#pragma unroll
      for (int d = 0; d < kDimTiles; ++d) acc[pt][d] = f32x4{0, 0, 0, 0};
    }

    __syncthreads();  // the slots are free (the previous item's epilogue used them)
    if constexpr (KIND == kSparse) {
      fetch_tokens(lo, next_tok0, next_tok1);
      fetch_tokens(lo + 1, after_tok0, after_tok1);
      fetch_pages(next_tok0, next_tok1, next_page0, next_page1);
    }
    issue(lo, 0);
    for (int t = lo; t < hi; ++t) {
      const int slot = (t - lo) & 1;
      wait_all_and_barrier();  // tile t is in its slot, and every wave has left the other one
      if (t + 1 < hi) issue(t + 1, slot ^ 1);
      const uint32_t blk0 = keys_lds + slot * kSlotBytes + ts * ST * kBlkBytes;

      // ---- S = K Q^T
      f32x4 s[PT][ST];
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int st = 0; st < ST; ++st) s[pt][st] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks) {
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          const s16x8 kk = lds_read((blk0 + (ks & 1 ? k_at ^ 64 : k_at)) + st * kBlkBytes + (ks >> 1) * 1024);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) s[pt][st] = E::mfma32(kk, q[pt][ks], s[pt][st]);
        }
      }

      // ---- scores in powers of two, masked keys at -inf
      const int key0 = (it.tile0 + t) * kTile + ts * ST * 16 + 4 * g4;  // dense: + 16 st + i
      int tok[ST][4];
#pragma unroll
      for (int st = 0; st < ST; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tok[st][i] = KIND == kSparse ? s_tok[slot][(ts * ST + st) * 16 + 4 * g4 + i] : key0 + st * 16 + i;
      const int tile_lo = (it.tile0 + t) * kTile;
      const bool masked = KIND == kSparse || tile_lo < it.max_start || tile_lo + kTile > it.min_end;
      // some key that is read is hidden from some row
      const bool mixed = KIND != kSparse && (max(tile_lo, it.min_start) < it.max_start ||
                                             min(tile_lo + kTile, it.max_end) > it.min_end);
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          if (a.softcap > 0.0f) {
            const float by = a.scale / a.softcap, cap = a.softcap * kLog2e;
#pragma unroll
            for (int i = 0; i < 4; ++i) s[pt][st][i] = cap * tanh_f32(s[pt][st][i] * by);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[pt][st][i] *= to_log2;
          }
          if (a.slopes) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[pt][st][i] -= p_slope[pt] * fabsf(static_cast<float>(p_pos[pt] - tok[st][i]));
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool seen = KIND == kSparse ? tok[st][i] >= 0 : tok[st][i] >= p_start[pt] && tok[st][i] < p_end[pt];
              s[pt][st][i] = seen ? s[pt][st][i] : -__builtin_inff();
            }
          }
        }

      // ---- running maximum and sum
      s16x4 p[PT][ST];
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        float mx = s[pt][0][0];
#pragma unroll
        for (int st = 0; st < ST; ++st)
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[pt][st][i]);
        mx = pair_max(mx) - E::kShift;
        if (__ballot(mx > m[pt] + kRaise)) {
          const float raised = fmaxf(m[pt], mx);
          const float by = __builtin_amdgcn_exp2f(m[pt] - raised);
          m[pt] = raised;
          l[pt] *= by;
#pragma unroll
          for (int d = 0; d < kDimTiles; ++d) acc[pt][d] *= by;
        }
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = __builtin_amdgcn_exp2f(s[pt][st][i] - m[pt]);
          l[pt] += (e[0] + e[1]) + (e[2] + e[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) p[pt][st][i] = E::round(e[i]);
        }
      }

      // A key that some rows of the pair tile see and others do not may hold an
      // infinity or a NaN; a weight of zero would not take it out of the
      // product.  Rows that see it get their NaN from S.
      if constexpr (KIND != kSparse) {
        if (mixed) {
          __syncthreads();
          for (int i = tid; i < kSlotBytes / 16; i += kAttnThreads) {
            s16x8* v = reinterpret_cast<s16x8*>(s_keys + slot * kSlotBytes) + i;
            s16x8 x = *v;
            constexpr int kExp = DT == IDX_BF16 ? 0x7F80 : 0x7C00;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (x[j] & kExp) == kExp ? 0 : x[j];
            *v = x;
          }
          __syncthreads();
        }
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int d = 0; d < kDimTiles; ++d) {
        const uint32_t va = blk0 + (v_at ^ ((d & 3) * 32)) + (d >> 2) * 1024;
        if constexpr (ST == 1) {
          const s16x4 v = lds_read_tr(va);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) acc[pt][d] = E::mfma16(v, p[pt][0], acc[pt][d]);
        } else {
#pragma unroll
          for (int st = 0; st < ST; st += 2) {
            const s16x4 v0 = lds_read_tr(va + st * kBlkBytes), v1 = lds_read_tr(va + (st + 1) * kBlkBytes);
            const s16x8 v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
              const s16x8 pp = __builtin_shufflevector(p[pt][st], p[pt][st + 1], 0, 1, 2, 3, 4, 5, 6, 7);
              acc[pt][d] = E::mfma32(v, pp, acc[pt][d]);
            }
          }
        }
      }
    }

    // ---- the streams' parts of each pair become one, 128 dimensions at a
    // time through LDS, and leave as whole rows
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) {
      const float sum = pair_sum(l[pt]);
      if (g4 == 0) s_ml[wave][pt * 16 + n16] = make_float2(m[pt], sum);
    }
    __syncthreads();  // every wave has left the last tile, and s_ml is complete
    const int64_t pair_base = static_cast<int64_t>(it.row0) * a.heads + it.pair0;  // over the whole batch
    float* piece = nullptr;
    if (!whole) {
      const int64_t id = KIND == kShared ? static_cast<int64_t>(w) + item : (lo == 0 ? 2 * w + 1 : 2 * w);
      piece = pieces + id * piece_floats(M);
    }
    float* s_o = reinterpret_cast<float*>(s_keys);
    for (int c = 0; c < kValDim / kChunkDims; ++c) {
      if (c) __syncthreads();
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int d = 0; d < kDimTiles; ++d)
          if (d / 8 == c)
            *reinterpret_cast<f32x4*>(s_o + (wave * kWavePairs + pt * 16 + n16) * kChunkStride + (d % 8) * 16 +
                                      4 * g4) = acc[pt][d];
      __syncthreads();
      for (int i = tid; i < M * (kChunkDims / 4); i += kAttnThreads) {
        const int local = i / (kChunkDims / 4), dim = (i % (kChunkDims / 4)) * 4;
        const int group = local / kWavePairs, in = local % kWavePairs;
        if (local >= it.pairs) continue;
        float top = kMInit;
#pragma unroll
        for (int k = 0; k < TS; ++k) top = fmaxf(top, s_ml[group * TS + k][in].x);
        f32x4 o = {0, 0, 0, 0};
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < TS; ++k) {
          const float2 ml = s_ml[group * TS + k][in];
          const float by = TS == 1 ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top);
          sum += ml.y * by;
          o += *reinterpret_cast<const f32x4*>(s_o + ((group * TS + k) * kWavePairs + in) * kChunkStride + dim) * by;
        }
        if (whole) {
          const int64_t pair = pair_base + local;
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          s16x4 r;
#pragma unroll
          for (int j = 0; j < 4; ++j) r[j] = E::round(o[j] * inv);
          *reinterpret_cast<s16x4*>(static_cast<short*>(a.out) + pair * kValDim + c * kChunkDims + dim) = r;
          if (a.lse && c == 0 && dim == 0) a.lse[pair] = (top + __log2f(sum)) * kLn2;
        } else {
          *reinterpret_cast<f32x4*>(piece + static_cast<int64_t>(local) * kValDim + c * kChunkDims + dim) = o;
          if (c == 0 && dim == 0)
            reinterpret_cast<float2*>(piece + M * kValDim)[local] = make_float2(top, sum);
        }
      }
    }
    if (!whole && lo == 0 && tid == 0) {
      const int last = share_owner(share.total, share.groups, item_at + it.tiles - 1);
      JoinInfo j;
      j.pair0 = pair_base;
      j.pairs = it.pairs;
      j.pieces = last - w + 1;
      j.first = w;
      j.pad = 0;
      j.pad2 = 0;
      join[KIND == kShared ? item : w] = j;
    }
    at = item_at + hi;
    item_at += it.tiles;
    ++item;
  }
}

// Joins the pieces of pairs.  One wave per pair; lanes hold 8 dimensions each.
struct JoinArgs {
  const JoinInfo* info;
  const float* pieces;
  void* out;
  float* lse;
};

struct Joined {
  f32x4 o0, o1;
  float m, l;
};

template <class At>
__device__ __forceinline__ void join_list(Joined& j, int n, int M, int local, At at) {
  const int lane = lane_id();
  for (int i = 0; i < n; ++i) {
    const float* piece = at(i);
    const float2 ml = reinterpret_cast<const float2*>(piece + M * kValDim)[local];
    const f32x4* o = reinterpret_cast<const f32x4*>(piece + static_cast<int64_t>(local) * kValDim + lane * 8);
    const f32x4 a = o[0], b = o[1];
    const float top = fmaxf(j.m, ml.x);
    const float mine = __builtin_amdgcn_exp2f(j.m - top), theirs = __builtin_amdgcn_exp2f(ml.x - top);
    j.o0 = j.o0 * mine + a * theirs;
    j.o1 = j.o1 * mine + b * theirs;
    j.l = j.l * mine + ml.y * theirs;
    j.m = top;
  }
}

template <int DT>
__device__ __forceinline__ void write_joined(const Joined& j, int64_t pair, void* out, float* lse) {
  using E = Elem<DT>;
  const float inv = j.l == 0.0f ? 0.0f : 1.0f / j.l;
  s16x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = E::round(j.o0[i] * inv);
    r[4 + i] = E::round(j.o1[i] * inv);
  }
  *reinterpret_cast<s16x8*>(static_cast<short*>(out) + pair * kValDim + lane_id() * 8) = r;
  if (lse && lane_id() == 0) lse[pair] = (j.m + __log2f(j.l)) * kLn2;
}

// Dense and sparse: block (w, y) joins pairs 4 y .. 4 y + 3 of the pair tile
// that workgroup w began and others went on with.
template <int DT>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a, int M) {
  const JoinInfo info = a.info[blockIdx.x];
  const int local = blockIdx.y * 4 + static_cast<int>(threadIdx.x >> 6);
  if (info.pieces == 0 || local >= info.pairs) return;
  Joined j{{0, 0, 0, 0}, {0, 0, 0, 0}, kMInit, 0.0f};
  join_list(j, info.pieces, M, local, [&](int i) {
    return a.pieces + static_cast<int64_t>(i == 0 ? 2 * info.first + 1 : 2 * (info.first + i)) * piece_floats(M);
  });
  write_joined<DT>(j, info.pair0 + local, a.out, a.lse);
}

// Shared: every pair has pieces of its prefix item and of its request's item.
template <int DT>
__global__ __launch_bounds__(256) void join_shared_kernel(JoinArgs a, int M, int64_t pairs, int heads, int next_n) {
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (pair >= pairs) return;
  const int prefix_items = static_cast<int>((pairs + M - 1) / M);
  const int of_request = next_n * heads;
  const int b = static_cast<int>(pair / of_request), in = static_cast<int>(pair - static_cast<int64_t>(b) * of_request);
  const int items[2] = {static_cast<int>(pair / M), prefix_items + b * ((of_request + M - 1) / M) + in / M};
  const int locals[2] = {static_cast<int>(pair % M), in % M};
  Joined j{{0, 0, 0, 0}, {0, 0, 0, 0}, kMInit, 0.0f};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const JoinInfo info = a.info[items[k]];
    join_list(j, info.pieces, M, locals[k], [&](int i) {
      return a.pieces + (static_cast<int64_t>(info.first) + i + items[k]) * piece_floats(M);
    });
  }
  write_joined<DT>(j, pair, a.out, a.lse);
}

// Pairs of a pair tile, by the pairs that one request brings (its rows' heads):
// as few idle matrix columns as possible, and beyond 64 the same keys are read
// again by the next tile.
int tile_pairs(int64_t pairs_per_request) {
  return pairs_per_request <= 16 ? 16 : pairs_per_request <= 32 ? 32 : 64;
}

constexpr int kMaxGrid = 256;  // one persistent workgroup per CU
constexpr int kMinTiles = 2;   // smallest share: below, the join costs more than the split saves

size_t join_bytes(int64_t infos) { return (static_cast<size_t>(infos) * sizeof(JoinInfo) + 255) / 256 * 256; }

template <int DT, int KIND, int PT, int PG>
hipError_t launch(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  constexpr int M = 16 * PT * PG;
  const int64_t items = item_count<KIND, M>(a);
  const int64_t tiles = KIND == kSparse ? (a.k + kTile - 1) / kTile : a.max_pages;
  const int grid = static_cast<int>(std::max(int64_t{1}, std::min(int64_t{kMaxGrid}, items * tiles / kMinTiles)));
  JoinInfo* info = static_cast<JoinInfo*>(a.workspace);
  float* pieces = reinterpret_cast<float*>(static_cast<char*>(a.workspace) +
                                           join_bytes(KIND == kShared ? items : kMaxGrid));
  const bool joins = KIND == kShared || grid > 1;
  launch_kernel(attention_kernel<DT, KIND, PT, PG>, dim3(grid), dim3(kAttnThreads), stream, ev.start,
                joins ? nullptr : ev.stop, a, kMinTiles, info, pieces);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !joins) return e;
  const JoinArgs j{info, pieces, a.out, a.lse};
  if constexpr (KIND == kShared) {
    const int64_t pairs = static_cast<int64_t>(a.rows) * a.heads;
    launch_kernel(join_shared_kernel<DT>, dim3(static_cast<uint32_t>((pairs + 3) / 4)), dim3(256), stream, nullptr,
                  ev.stop, j, M, pairs, a.heads, a.next_n);
  } else {
    launch_kernel(join_kernel<DT>, dim3(grid, M / 4), dim3(256), stream, nullptr, ev.stop, j, M);
  }
  return hipGetLastError();
}

template <int DT, int KIND>
hipError_t launch_kind(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  const int64_t per_request = KIND == kSparse ? a.heads
                                              : (static_cast<int64_t>(a.rows) + a.requests - 1) / a.requests * a.heads;
  switch (tile_pairs(per_request)) {
    case 16: return launch<DT, KIND, 1, 1>(a, stream, ev);
    case 32: return launch<DT, KIND, 1, 2>(a, stream, ev);
    default: return launch<DT, KIND, 1, 4>(a, stream, ev);
  }
}

template <int KIND>
hipError_t launch_type(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return a.dtype == IDX_BF16 ? launch_kind<IDX_BF16, KIND>(a, stream, ev)
                             : launch_kind<IDX_FP16, KIND>(a, stream, ev);
}

}  // namespace

size_t attention_workspace_size(int32_t rows, int32_t heads, int32_t requests) {
  if (rows <= 0 || heads <= 0 || requests <= 0) return 0;
  // whichever of the operators that share this query needs more
  const int64_t per_request = (static_cast<int64_t>(rows) + requests - 1) / requests * heads;
  const int m = std::max(tile_pairs(per_request), tile_pairs(heads));
  return join_bytes(kMaxGrid) + 2 * kMaxGrid * static_cast<size_t>(piece_floats(m)) * sizeof(float);
}

size_t shared_prefix_workspace_size(int32_t rows, int32_t heads, int32_t requests) {
  if (rows <= 0 || heads <= 0 || requests <= 0) return 0;
  const int64_t per_request = (static_cast<int64_t>(rows) + requests - 1) / requests * heads;
  const int m = tile_pairs(per_request);
  const int64_t items = (static_cast<int64_t>(rows) * heads + m - 1) / m + requests * ((per_request + m - 1) / m);
  return join_bytes(items) + (items + kMaxGrid) * static_cast<size_t>(piece_floats(m)) * sizeof(float);
}

hipError_t launch_paged_attention(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kDense>(a, stream, ev);
}
hipError_t launch_shared_prefix_attention(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kShared>(a, stream, ev);
}
hipError_t launch_sparse_attention(const AttentionArgs& a, hipStream_t stream, LaunchEvents ev) {
  return launch_type<kSparse>(a, stream, ev);
}

}  // namespace pmqa
